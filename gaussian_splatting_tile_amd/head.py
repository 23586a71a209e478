"""A network head that predicts Gaussians, and what gives its tokens their
content, on the library's operators.

Token features [m][width] pass through residual blocks

    s' = s + w2 act(w1 norm(s) + b1) + b2

and a last norm and product that writes one plane per Gaussian parameter, the
[rows][m] layout that gs_project reads: 3 means, 3 log-scales, 4 quaternion
components, 1 opacity logit and (degree + 1)^2 x 3 SH coefficients.  The
rasterizer's gradients come back in the same layout, so nothing is copied
between the two (the heads of the GlobalSplat page, step (4) of its pipeline).

Before the head, the scene's tokens may read the feature maps of the input
views (ViewReader): a group norm with SiLU over every map, a product to keys and
values, and cross attention from the tokens (steps (2) and (3) of that
pipeline).

    python -m gaussian_splatting_tile_amd.head

fits a small head to one view of a scene and renders it again with its blocks
in 8 bits.
"""

from __future__ import annotations

from typing import Dict, Optional

import torch

from . import binding as B


class GaussianHead:
    """Weights, activations and buffers for training on `m` tokens; serve()
    takes any number.  `width` and `hidden` are multiples of 32 (the 8-bit
    blocks)."""

    def __init__(self, m: int, width: int, hidden: int, blocks: int, sh_degree: int = 3, act: str = "gelu",
                 dtype=torch.bfloat16, device="cuda", seed: int = 0):
        assert width % 32 == 0 and hidden % 32 == 0 and blocks >= 1
        self.m, self.width, self.hidden, self.blocks, self.act = m, width, hidden, blocks, act
        self.sh_coeffs = (sh_degree + 1) ** 2
        self.rows = 11 + 3 * self.sh_coeffs
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s, scale: (torch.randn(s, generator=gen, device=device) * scale).to(dtype)
        e16 = lambda *s: torch.empty(s, dtype=dtype, device=device)
        f32 = lambda *s: torch.zeros(s, device=device)
        # the blocks' matrices are stacked, so one optimiser call steps all of them
        self.w1, self.w2 = rand(blocks, hidden, width, scale=width ** -0.5), rand(blocks, width, hidden, scale=0.1 * hidden ** -0.5)
        self.w_out = rand(self.rows, width, scale=0.02)
        self.b1, self.b2, self.b_out = f32(blocks, hidden), f32(blocks, width), f32(self.rows)
        self.gamma = torch.ones(blocks + 1, width, device=device)
        self.matrices, self.vectors = ("w1", "w2", "w_out"), ("b1", "b2", "b_out", "gamma")
        self.grads = {k: torch.zeros_like(getattr(self, k)) for k in self.matrices + self.vectors}
        self.momentum = {k: torch.zeros_like(getattr(self, k), dtype=torch.float32) for k in self.matrices}
        # activations: the residual stream before every block and at the end,
        # each block's normed input, pre-activation and hidden values
        self.s, self.normed = [e16(m, width) for _ in range(blocks + 1)], [e16(m, width) for _ in range(blocks + 1)]
        self.rstd = f32(blocks + 1, m)
        self.z, self.h = [e16(m, hidden) for _ in range(blocks)], [e16(m, hidden) for _ in range(blocks)]
        self.planes, self.dplanes = f32(self.rows, m), f32(self.rows, m)
        self.ds, self.dn, self.dh = e16(m, width), e16(m, width), e16(m, hidden)
        # descriptors once: the buffers stay where they are
        self._up = [B.linear_struct(self.normed[i], self.w1[i], self.h[i], bias=self.b1[i], z=self.z[i], act=act) for i in range(blocks)]
        self._down = [B.linear_struct(self.h[i], self.w2[i], self.s[i + 1], bias=self.b2[i], residual=self.s[i]) for i in range(blocks)]
        self._out = B.linear_struct(self.normed[blocks], self.w_out, self.planes, bias=self.b_out, planes=True)
        g = self.grads
        self._d_out = B.linear_grads_struct(self._out, self.dplanes, dx=self.dn, dw=g["w_out"], db=g["b_out"])
        self._d_down = [B.linear_grads_struct(self._down[i], self.ds, dx=self.dh, dw=g["w2"][i], db=g["b2"][i]) for i in range(blocks)]
        self._d_up = [B.linear_grads_struct(self._up[i], self.dh, dx=self.dn, dw=g["w1"][i], db=g["b1"][i]) for i in range(blocks)]
        need = [B.linear_fwd_workspace_bytes(x) for x in self._up + self._down + [self._out]]
        need += [B.linear_bwd_workspace_bytes(x, y) for x, y in zip(self._up + self._down + [self._out], self._d_up + self._d_down + [self._d_out])]
        need += [B.rms_norm_bwd_workspace_bytes(m, width)]
        need += [B.muon_workspace_bytes(self._muon(k, 0.0)) for k in self.matrices]
        self.ws = torch.empty(max(need) + 16, dtype=torch.uint8, device=device)

    # ---- training -----------------------------------------------------------
    def forward(self, tokens: torch.Tensor) -> torch.Tensor:
        """The parameter planes [rows][m] (fp32) of tokens [m][width]."""
        if tokens.shape != (self.m, self.width):
            raise ValueError(f"tokens: expected [{self.m}][{self.width}], got {tuple(tokens.shape)}")
        self.s[0].copy_(tokens)
        for i in range(self.blocks):
            B.rms_norm_fwd(self.s[i], self.normed[i], gamma=self.gamma[i], rstd=self.rstd[i])
            B.linear_fwd(self._up[i], self.ws)
            B.linear_fwd(self._down[i], self.ws)
        last = self.blocks
        B.rms_norm_fwd(self.s[last], self.normed[last], gamma=self.gamma[last], rstd=self.rstd[last])
        B.linear_fwd(self._out, self.ws)
        return self.planes

    def backward(self):
        """Gradients of every weight from `dplanes`."""
        last = self.blocks
        B.linear_bwd(self._out, self._d_out, self.ws)
        B.rms_norm_bwd(self.s[last], self.rstd[last], self.dn, self.ds, gamma=self.gamma[last],
                       dgamma=self.grads["gamma"][last], workspace=self.ws)
        for i in reversed(range(self.blocks)):
            B.linear_bwd(self._down[i], self._d_down[i], self.ws)
            B.linear_bwd(self._up[i], self._d_up[i], self.ws)
            B.rms_norm_bwd(self.s[i], self.rstd[i], self.dn, self.ds, gamma=self.gamma[i], dsum=self.ds,
                           dgamma=self.grads["gamma"][i], workspace=self.ws)

    def _muon(self, k: str, lr: float, beta: float = 0.95) -> B.GsMuon:
        w = getattr(self, k)
        scale = max(1.0, w.shape[-2] / w.shape[-1]) ** 0.5
        return B.muon_struct(self.grads[k], momentum=self.momentum[k], weight=w, lr=lr, beta=beta, scale=scale)

    def step(self, lr: float, lr_vectors: float):
        """One step of every weight: orthogonalised momentum for the
        matrices, the sign of the gradient for biases and gammas."""
        for k in self.matrices:
            B.muon_step(self._muon(k, lr), self.ws)
        for k in self.vectors:
            getattr(self, k).sub_(lr_vectors * torch.sign(self.grads[k]))

    # ---- the rasterizer's side ------------------------------------------------
    def gaussians(self, planes: torch.Tensor) -> Dict[str, torch.Tensor]:
        """The arrays of binding.gaussians_struct; means, quats and SH are the
        planes themselves."""
        return dict(means=planes[0:3], scales=torch.exp(planes[3:6]), quats=planes[6:10],
                    opacities=torch.sigmoid(planes[10]), sh=planes[11:].view(self.sh_coeffs, 3, self.m))

    def gaussian_grads(self) -> Dict[str, torch.Tensor]:
        """dplanes, zeroed, as the arrays the rasterizer's backward adds to."""
        d = self.dplanes.zero_()
        return dict(means=d[0:3], log_scales=d[3:6], quats=d[6:10], opacity_logits=d[10],
                    sh=d[11:].view(self.sh_coeffs, 3, self.m))

    # ---- serving ----------------------------------------------------------------
    def quantize(self):
        """8-bit copies of the blocks' matrices for serve()."""
        self.q = {}
        for k in ("w1", "w2"):
            w = getattr(self, k).reshape(-1, getattr(self, k).shape[-1])
            codes = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=w.device)
            scales = torch.empty((w.shape[0], w.shape[1] // 32), dtype=torch.uint8, device=w.device)
            B.mxfp8_quantize(w, codes, scales)
            shape = getattr(self, k).shape
            self.q[k] = (codes.view(shape), scales.view(*shape[:-1], -1))

    def serve(self, tokens: torch.Tensor) -> torch.Tensor:
        """The planes of any number of tokens, the blocks by 8-bit products
        (quantize() first).  The last product stays in the weights' own type:
        a Gaussian's position has to be good to a fraction of its size."""
        if tokens.dim() != 2 or tokens.shape[1] != self.width:
            raise ValueError(f"tokens: expected [n][{self.width}], got {tuple(tokens.shape)}")
        n, dev = tokens.shape[0], tokens.device
        codes = lambda w: (torch.empty((n, w), dtype=torch.float8_e4m3fn, device=dev), torch.empty((n, w // 32), dtype=torch.uint8, device=dev))
        s, (y, ys), (hq, hs) = tokens.to(self.w1.dtype).clone(), codes(self.width), codes(self.hidden)
        h, planes = torch.empty((n, self.hidden), dtype=s.dtype, device=dev), torch.empty((self.rows, n), device=dev)

        def product(*args, **kw):
            a = B.linear_struct(*args, **kw)
            B.linear_fwd(a, torch.empty(B.linear_fwd_workspace_bytes(a), dtype=torch.uint8, device=dev))

        for i in range(self.blocks):
            B.rms_norm_fwd(s, y, gamma=self.gamma[i], y_scales=ys)
            product(y, self.q["w1"][0][i], h, bias=self.b1[i], act=self.act, x_scales=ys, w_scales=self.q["w1"][1][i])
            B.mxfp8_quantize(h, hq, hs)
            product(hq, self.q["w2"][0][i], s, bias=self.b2[i], residual=s, x_scales=hs, w_scales=self.q["w2"][1][i])
        B.rms_norm_fwd(s, s, gamma=self.gamma[self.blocks])
        product(s, self.w_out, planes, bias=self.b_out, planes=True)
        return planes


class ViewReader:
    """Tokens [m][width] read feature maps [views][pixels][channels]:

        f = silu(group_norm(features)),  [k v] = f w_kv^T + b_kv,  q = norm(tokens) w_q^T + b_q
        tokens' = tokens + attention(q, k, v) w_o^T + b_o

    with `heads` heads of width / heads.  Views whose byte in `seen` is 0 are not
    attended and give no gradient, whatever their maps hold.  For the backward the
    maps are kept in 8 bits; `channels` and `width` are multiples of 32, a head has 128
    channels at most, and `groups` divides `channels`."""

    def __init__(self, m: int, width: int, views: int, pixels: int, channels: int, heads: int, groups: int,
                 dtype=torch.bfloat16, device="cuda", seed: int = 0):
        assert width % 32 == 0 and channels % 32 == 0 and width % heads == 0 and width // heads <= 128 and channels % groups == 0
        self.m, self.width, self.views, self.pixels, self.channels, self.heads, self.groups = m, width, views, pixels, channels, heads, groups
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s, scale: (torch.randn(s, generator=gen, device=device) * scale).to(dtype)
        e16 = lambda *s: torch.empty(s, dtype=dtype, device=device)
        f32 = lambda *s: torch.zeros(s, device=device)
        n = views * pixels
        self.w_kv, self.w_q, self.w_o = rand(2 * width, channels, scale=channels ** -0.5), rand(width, width, scale=width ** -0.5), rand(width, width, scale=0.1 * width ** -0.5)
        self.b_kv, self.b_q, self.b_o = f32(2 * width), f32(width), f32(width)
        self.gamma_f, self.beta_f, self.gamma = torch.ones(channels, device=device), f32(channels), torch.ones(width, device=device)
        self.matrices, self.vectors = ("w_kv", "w_q", "w_o"), ("b_kv", "b_q", "b_o", "gamma_f", "beta_f", "gamma")
        self.grads = {k: torch.zeros_like(getattr(self, k)) for k in self.matrices + self.vectors}
        # activations
        self.f, self.mean, self.rstd_f = e16(views, pixels, channels), f32(views, groups), f32(views, groups)
        self.kept = torch.empty((views, pixels, channels), dtype=torch.float8_e4m3fn, device=device)
        self.kept_scales = torch.empty((views, pixels, channels // 32), dtype=torch.uint8, device=device)
        self.kv, self.normed, self.rstd, self.q = e16(n, 2 * width), e16(m, width), f32(m), e16(m, width)
        self.read, self.lse, self.tokens, self.out = e16(m, width), f32(1, heads, m), e16(m, width), e16(m, width)
        self.mask, self.nothing = torch.ones((1, n), dtype=torch.uint8, device=device), torch.zeros((), dtype=dtype, device=device)
        self.d_out, self.d_read, self.d_q, self.d_kv = e16(m, width), e16(m, width), e16(m, width), e16(n, 2 * width)
        self.d_normed, self.d_tokens, self.d_features = e16(m, width), e16(m, width), e16(views, pixels, channels)
        # descriptors once: the buffers stay where they are
        rows = lambda t: t.view(1, m, heads, width // heads)
        k, v = (self.kv.view(1, n, 2, heads, width // heads)[:, :, i] for i in range(2))
        dk, dv = (self.d_kv.view(1, n, 2, heads, width // heads)[:, :, i] for i in range(2))
        flat, g = self.f.view(n, channels), self.grads
        self._kv = B.linear_struct(flat, self.w_kv, self.kv, bias=self.b_kv)
        self._q = B.linear_struct(self.normed, self.w_q, self.q, bias=self.b_q)
        self._o = B.linear_struct(self.read, self.w_o, self.out, bias=self.b_o, residual=self.tokens)
        self._read = B.attention_struct(rows(self.q), k, v, rows(self.read), lse=self.lse, kv_mask=self.mask)
        self._d_kv = B.linear_grads_struct(self._kv, self.d_kv, dx=self.d_features.view(n, channels), dw=g["w_kv"], db=g["b_kv"])
        self._d_q = B.linear_grads_struct(self._q, self.d_q, dx=self.d_normed, dw=g["w_q"], db=g["b_q"])
        self._d_o = B.linear_grads_struct(self._o, self.d_out, dx=self.d_read, dw=g["w_o"], db=g["b_o"])
        self._d_read = B.attention_grads_struct(self._read, rows(self.d_read), dq=rows(self.d_q), dk=dk, dv=dv)
        need = [B.linear_fwd_workspace_bytes(x) for x in (self._kv, self._q, self._o)]
        need += [B.linear_bwd_workspace_bytes(x, y) for x, y in ((self._kv, self._d_kv), (self._q, self._d_q), (self._o, self._d_o))]
        need += [B.attention_fwd_workspace_bytes(self._read), B.attention_bwd_workspace_bytes(self._read, self._d_read)]
        need += [f(views, pixels, channels, groups) for f in (B.group_norm_fwd_workspace_bytes, B.group_norm_bwd_workspace_bytes)]
        need += [B.rms_norm_bwd_workspace_bytes(m, width)]
        self.ws = torch.empty(max(need) + 16, dtype=torch.uint8, device=device)

    @torch.no_grad()
    def forward(self, tokens: torch.Tensor, features: torch.Tensor, seen: Optional[torch.Tensor] = None) -> torch.Tensor:
        """tokens' [m][width]; seen [views] uint8 or bool, or None: all."""
        if tokens.shape != (self.m, self.width) or features.shape != (self.views, self.pixels, self.channels):
            raise ValueError(f"expected tokens [{self.m}][{self.width}] and features [{self.views}][{self.pixels}][{self.channels}], "
                             f"got {tuple(tokens.shape)} and {tuple(features.shape)}")
        if seen is not None and seen.shape != (self.views,):
            raise ValueError(f"seen: expected [{self.views}], got {tuple(seen.shape)}")
        if features.dtype is not self.f.dtype or features.device != self.f.device:
            raise ValueError(f"features: expected {self.f.dtype} on {self.f.device}, got {features.dtype} on {features.device}")
        mask = self.mask.view(self.views, self.pixels)
        if seen is None:
            mask.fill_(1)
        else:
            there = (seen != 0).to(mask.device)
            mask.copy_(there.view(-1, 1).expand_as(mask))
            # zeros for what is not there: the backward multiplies every view's f and h by
            # gradients of 0, which NaN and infinities would survive
            features = torch.where(there.view(-1, 1, 1), features, self.nothing, out=self.f)
        self.tokens.copy_(tokens)
        B.group_norm_fwd(features, self.f, self.groups, gamma=self.gamma_f, beta=self.beta_f, act="silu", mean=self.mean, rstd=self.rstd_f,
                         kept=self.kept, kept_scales=self.kept_scales, workspace=self.ws)
        B.linear_fwd(self._kv, self.ws)
        B.rms_norm_fwd(self.tokens, self.normed, gamma=self.gamma, rstd=self.rstd)
        B.linear_fwd(self._q, self.ws)
        B.attention_fwd(self._read, self.ws)
        B.linear_fwd(self._o, self.ws)
        return self.out

    def backward(self, d_out: torch.Tensor):
        """Gradients of every weight; returns those of tokens and features."""
        if d_out.shape != (self.m, self.width):
            raise ValueError(f"d_out: expected [{self.m}][{self.width}], got {tuple(d_out.shape)}")
        self.d_out.copy_(d_out)
        B.linear_bwd(self._o, self._d_o, self.ws)
        B.attention_bwd(self._read, self._d_read, self.ws)
        B.linear_bwd(self._q, self._d_q, self.ws)
        B.rms_norm_bwd(self.tokens, self.rstd, self.d_normed, self.d_tokens, gamma=self.gamma, dsum=self.d_out, dgamma=self.grads["gamma"],
                       workspace=self.ws)
        B.linear_bwd(self._kv, self._d_kv, self.ws)
        B.group_norm_bwd(self.kept, self.mean, self.rstd_f, self.d_features, self.d_features, self.groups, gamma=self.gamma_f, beta=self.beta_f,
                         act="silu", dgamma=self.grads["gamma_f"], dbeta=self.grads["beta_f"], x_scales=self.kept_scales, workspace=self.ws)
        return self.d_tokens, self.d_features


def fit(steps: int = 120, n: int = 1000, width: int = 64, hidden: int = 128, blocks: int = 2, say=print):
    """Fits a head to one view of a small scene; returns the losses, the head,
    its tokens, the trained image and the one rendered from serve()."""
    import numpy as np

    from . import scenes
    sc = scenes.tiny(n=n)
    cam = sc.cameras[0]
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    buf = B.ViewBuffers(n, cam, 256 * n)
    target_g = dict(means=up(sc.means), scales=up(sc.scales), quats=up(sc.quats), opacities=up(sc.opacities), sh=up(sc.sh))
    buf.forward(B.gaussians_struct(target_g, sc.sh_degree))
    target = buf.image.clone()

    head = GaussianHead(n, width, hidden, blocks, sh_degree=0)
    tokens = torch.randn((n, width), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    # the head starts at the scene's average Gaussian and spreads them out
    head.b_out[2] = float(target_g["means"][2].mean())
    head.b_out[3:6] = float(torch.log(target_g["scales"]).mean())
    head.b_out[6] = 1.0
    head.w_out[0:3].mul_(15.0)
    bws = buf.backward_workspace()
    losses = []
    for t in range(steps):
        planes = head.forward(tokens)
        g = head.gaussians(planes)
        gs = B.gaussians_struct(g, 0)
        buf.forward(gs)
        diff = buf.image - target
        losses.append(diff.square().mean())
        buf.backward(gs, diff * (2.0 / diff.numel()), head.gaussian_grads(), bws)
        head.backward()
        decay = 1.0 - t / steps
        head.step(0.01 * decay, 0.002 * decay)
    losses = torch.stack(losses).tolist()
    g = head.gaussians(head.forward(tokens))
    buf.forward(B.gaussians_struct(g, 0))
    image = buf.image.clone()
    head.quantize()
    g = head.gaussians(head.serve(tokens))
    buf.forward(B.gaussians_struct(g, 0))
    say(f"loss {losses[0]:.5f} -> {losses[-1]:.5f} in {steps} steps; 8-bit image differs by {float((buf.image - image).square().mean()):.2e} (mean square)")
    return losses, head, tokens, image, buf.image.clone(), target


if __name__ == "__main__":
    fit()
