"""Tokens that read feature maps (gaussian_splatting_tile_amd/head.py,
ViewReader): group norm with its 8-bit checkpoint, products and cross attention
run together, forward and backward, before a head and through the rasterizer."""

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_amd import binding as B
from gaussian_splatting_tile_amd import head as H
from gaussian_splatting_tile_amd import scenes
from oracle import attention as A
from oracle import network as N
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().float().cpu().double().numpy()


def _oracle(r, tokens, features, seen, d_out):
    """(tokens', gradients) in fp64; the maps' gradient from the maps as the
    checkpoint holds them, as the reader has it."""
    m, w, h = r.m, r.width, r.heads
    n, d = r.views * r.pixels, w // h
    P = {k: _np(getattr(r, k)) for k in r.matrices + r.vectors}
    T, F, D = _np(tokens), _np(features), _np(d_out)
    mean, rstd, _, f = A.group_norm(F, r.groups, P["gamma_f"], P["beta_f"], "silu")
    flat = f.reshape(n, -1)
    kv = N.linear(flat, P["w_kv"], P["b_kv"])[1]
    _, rs, normed = N.rms_norm(T, None, P["gamma"])
    q = N.linear(normed, P["w_q"], P["b_q"])[1]
    mask = np.repeat(seen, r.pixels)[None]
    heads = lambda x: x.reshape(1, -1, h, d)
    k, v = heads(kv[:, :w]), heads(kv[:, w:])
    read, lse, _ = A.attention(heads(q), k, v, d ** -0.5, A.seen_keys(1, n, None, mask))
    out = N.linear(read.reshape(m, w), P["w_o"], P["b_o"], "none", T)[1]
    g = {}
    d_read, g["w_o"], g["b_o"], _ = N.linear_grads(read.reshape(m, w), P["w_o"], None, D)
    dq, dk, dv, _ = A.attention_grads(heads(q), k, v, d ** -0.5, A.seen_keys(1, n, None, mask), read, lse, heads(d_read))
    d_normed, g["w_q"], g["b_q"], _ = N.linear_grads(normed, P["w_q"], None, dq.reshape(m, w))
    g["tokens"], g["gamma"] = N.rms_norm_grads(T, rs, d_normed, P["gamma"], D)
    d_kv = np.concatenate([dk.reshape(n, w), dv.reshape(n, w)], axis=1)
    d_f, g["w_kv"], g["b_kv"], _ = N.linear_grads(flat, P["w_kv"], None, d_kv)
    codes, scales = N.mxfp8_quantize(F.reshape(n, -1))
    kept = N.mxfp8_value(codes, scales).reshape(F.shape)
    g["features"], g["gamma_f"], g["beta_f"] = A.group_norm_grads(kept, mean, rstd, d_f.reshape(F.shape), r.groups, P["gamma_f"], P["beta_f"], "silu")
    return out, g


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 3e-5), (torch.float16, 1.5e-2), (torch.bfloat16, 8e-2)])
def test_reader_matches_the_oracle(dtype, tol):
    """Relative (Frobenius) errors: some ten roundings in a chain, each of at
    most u (2^-11, 2^-8), and for fp32 the sums' error bounds."""
    r = H.ViewReader(150, 64, 3, 70, 96, 4, 12, dtype=dtype, seed=3)
    rng = np.random.default_rng(2)
    for k in r.vectors:
        getattr(r, k).add_(torch.from_numpy(rng.standard_normal(getattr(r, k).shape) * 0.1).float().cuda())
    up = lambda *s, scale=1.0: torch.from_numpy(rng.standard_normal(s) * scale).to(dtype).cuda()
    tokens, features, d_out = up(150, 64), up(3, 70, 96, scale=2.0), up(150, 64, scale=0.1)
    features[1] = float("nan")                              # a view that is not there
    seen = torch.tensor([True, False, True], device="cuda")
    clean = features.clone()
    clean[1] = 0.0
    before = r.forward(tokens, features, seen).clone()
    out = r.forward(tokens, clean, seen)
    assert torch.equal(before, out)                         # what it holds has no effect
    got = [_np(out)] + [_np(x) for x in r.backward(d_out)]
    want, g = _oracle(r, tokens, clean, seen.cpu().numpy(), d_out)
    assert np.linalg.norm(got[0] - want) <= tol * np.linalg.norm(want)
    mine = {"tokens": got[1], "features": got[2], **{k: _np(v) for k, v in r.grads.items()}}
    for k, w in g.items():
        err = np.linalg.norm(mine[k] - w) / np.linalg.norm(w)
        say(f"[gpu] reader {dtype} d{k}: {err:.2e}")
        assert err <= tol, (k, err)


def test_reader_before_a_head_and_the_rasterizer():
    """A training step of both, captured in a graph: replays give what the
    eager step gives, with eager work in between."""
    n, sc = 256, scenes.tiny(n=256)
    cam = sc.cameras[0]
    r = H.ViewReader(n, 64, 2, 100, 32, 4, 4, seed=1)
    head = H.GaussianHead(n, 64, 96, 1, sh_degree=0)
    head.b_out[2], head.b_out[3:6], head.b_out[6] = float(sc.means[2].mean()), float(np.log(sc.scales).mean()), 1.0
    gen = torch.Generator("cuda").manual_seed(5)
    tokens = torch.randn((n, 64), generator=gen, device="cuda").bfloat16()
    features = torch.randn((2, 100, 32), generator=gen, device="cuda").bfloat16()
    buf = B.ViewBuffers(n, cam, 256 * n)
    bws = buf.backward_workspace()
    grad = torch.randn(buf.image.shape, generator=gen, device="cuda") * 1e-3

    def step():
        planes = head.forward(r.forward(tokens, features))
        gs = B.gaussians_struct(head.gaussians(planes), 0)
        buf.forward(gs)
        buf.backward(gs, grad, head.gaussian_grads(), bws)
        head.backward()
        return [r.out, planes, head.ds, *r.backward(head.ds), *r.grads.values(), *head.grads.values()]

    want = [x.clone() for x in step()]
    assert all(torch.isfinite(x.float()).all() for x in want) and float(want[4].float().abs().max()) > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for x in got:
            x.zero_()
        torch.randn(1000, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
