"""Attention and group norm at the far end of their sizes, on other streams, in
replayed graphs, and twice over."""

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_amd import binding as B
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def _ws(n):
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device="cuda")


class Attention:
    """A call with everything it needs."""

    def __init__(self, b, nq, nk, h, kv, d, dtype, seed=0, lengths=None, mask=None):
        gen = torch.Generator("cuda").manual_seed(seed)
        e = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)
        self.q, self.k, self.v, self.dout = e(b, nq, h, d), e(b, nk, kv, d), e(b, nk, kv, d), e(b, nq, h, d)
        self.out, self.lse = torch.empty_like(self.q), torch.empty(b, h, nq, device="cuda")
        self.dq, self.dk, self.dv = torch.empty_like(self.q), torch.empty_like(self.k), torch.empty_like(self.v)
        self.a = B.attention_struct(self.q, self.k, self.v, self.out, lse=self.lse, kv_lengths=lengths, kv_mask=mask)
        self.g = B.attention_grads_struct(self.a, self.dout, dq=self.dq, dk=self.dk, dv=self.dv)
        self.ws = _ws(max(B.attention_fwd_workspace_bytes(self.a), B.attention_bwd_workspace_bytes(self.a, self.g)))

    def __call__(self, stream=None):
        B.attention_fwd(self.a, self.ws, stream)
        B.attention_bwd(self.a, self.g, self.ws, stream)

    def results(self):
        return [self.out, self.lse, self.dq, self.dk, self.dv]


class Norm:
    def __init__(self, n, p, c, groups, dtype, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        e = lambda *s: torch.randn(s, generator=gen, device="cuda")
        self.x, self.dy, self.gamma, self.beta, self.groups = e(n, p, c).to(dtype), e(n, p, c).to(dtype), e(c), e(c), groups
        self.y, self.dx, self.mean, self.rstd = torch.empty_like(self.x), torch.empty_like(self.x), torch.empty(n, groups, device="cuda"), torch.empty(n, groups, device="cuda")
        self.kept, self.scales = torch.empty(n, p, c, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(n, p, c // 32, dtype=torch.uint8, device="cuda")
        self.dgamma, self.dbeta = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
        self.ws = _ws(max(B.group_norm_fwd_workspace_bytes(n, p, c, groups), B.group_norm_bwd_workspace_bytes(n, p, c, groups)))

    def __call__(self, stream=None):
        B.group_norm_fwd(self.x, self.y, self.groups, gamma=self.gamma, beta=self.beta, act="gelu", mean=self.mean, rstd=self.rstd, kept=self.kept,
                         kept_scales=self.scales, workspace=self.ws, stream=stream)
        B.group_norm_bwd(self.kept, self.mean, self.rstd, self.dy, self.dx, self.groups, gamma=self.gamma, beta=self.beta, act="gelu", dgamma=self.dgamma,
                         dbeta=self.dbeta, x_scales=self.scales, workspace=self.ws, stream=stream)

    def results(self):
        return [self.y, self.mean, self.rstd, self.kept.view(torch.uint8), self.scales, self.dx, self.dgamma, self.dbeta]


def _calls():
    return [Attention(2, 150, 700, 4, 2, 64, torch.bfloat16, 1), Attention(1, 1, 5000, 4, 4, 40, torch.float16, 2), Attention(1, 40, 300, 2, 1, 128, torch.float32, 3),
            Attention(3, 70, 130, 2, 2, 33, torch.bfloat16, 4, lengths=torch.tensor([130, 0, 64], dtype=torch.int32, device="cuda")),
            Norm(2, 50, 64, 8, torch.bfloat16, 5), Norm(2, 9000, 32, 4, torch.float16, 6), Norm(3, 700, 96, 2, torch.float32, 7)]


def test_repeated_streamed_and_replayed_calls_give_the_same_bits():
    calls = _calls()
    for c in calls:
        c()
    torch.cuda.synchronize()
    want = [[r.clone() for r in c.results()] for c in calls]

    def same(what):
        torch.cuda.synchronize()
        for c, w in zip(calls, want):
            for i, (x, y) in enumerate(zip(c.results(), w)):
                assert torch.equal(x.view(torch.uint8) if x.dtype.is_floating_point else x, y.view(torch.uint8) if y.dtype.is_floating_point else y), (what, type(c).__name__, i)

    def scrub():
        for c in calls:
            for r in c.results():
                r.zero_()
            c.ws.fill_(0xFF)                               # nothing is kept in a workspace from one call to the next
        torch.cuda.synchronize()

    scrub()
    for c in calls:
        c()
    same("again")
    scrub()
    streams = [torch.cuda.Stream() for _ in calls]         # two at once, each on a stream of its own
    for c, s in zip(calls, streams):
        c(s)
    same("streams")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for c in calls:
            c()
    torch.cuda.synchronize()
    graphs = []
    for half in (calls[::2], calls[1::2]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for c in half:
                c()
        graphs.append(g)
    for i in range(3):
        scrub()
        for g in graphs:
            g.replay()
        same(f"replay {i}")
        calls[i]()                                          # eager work between replays


def test_attention_beyond_32_bit_offsets():
    """States whose rows lie past 2^32 bytes of their head's first one, in place
    and packed.  All scores are 0 but the last state's."""
    for d, nk in ((128, (1 << 24) + 70), (124, (1 << 24) + 70)):
        say(f"[gpu] attention over {nk} states of {d}")
        k = torch.zeros(1, nk, 1, d, dtype=torch.bfloat16, device="cuda")
        v = torch.zeros(1, nk, 1, d, dtype=torch.bfloat16, device="cuda")
        k[0, -1], v[0, -1] = 8.0, torch.arange(d, device="cuda").bfloat16()
        v[0, 0] = -7.0
        q = torch.full((1, 3, 1, d), 1.0, dtype=torch.bfloat16, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(1, 1, 3, device="cuda")
        a = B.attention_struct(q, k, v, out, lse=lse, scale=0.125)
        B.attention_fwd(a, _ws(B.attention_fwd_workspace_bytes(a)))
        assert torch.equal(out, v[:, -1:].expand_as(out))   # exp(124) against 2^24 states
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dv.fill_(3.0)
        g = B.attention_grads_struct(a, q, dq=dq, dk=dk, dv=dv)
        B.attention_bwd(a, g, _ws(B.attention_bwd_workspace_bytes(a, g)))
        assert bool((dv[0, -1] == 3.0).all()) and float(dv[0, :-1].float().abs().max()) < 1e-30
        assert bool((dk[0, -1].float().abs() < 1e-2).all()) and bool(torch.isfinite(dq).all())
        del k, v, dk, dv


def test_attention_of_many_rows_of_queries():
    """2^24 queries of two states each; rows of out and of dq past 2^31 elements."""
    nq, d = (1 << 24) + 33, 128
    say(f"[gpu] attention of {nq} queries")
    q = torch.zeros(1, nq, 1, d, dtype=torch.bfloat16, device="cuda")
    q[0, -1] = 1.0
    kv = torch.zeros(1, 2, 1, d, dtype=torch.bfloat16, device="cuda")
    kv[0, 1] = 2.0
    out, lse = torch.empty_like(q), torch.empty(1, 1, nq, device="cuda")
    a = B.attention_struct(q, kv, kv, out, lse=lse, scale=0.25)
    B.attention_fwd(a, _ws(B.attention_fwd_workspace_bytes(a)))
    assert bool((out[0, :-1] == 1.0).all()) and bool((out[0, -1] == 2.0).all())
    dout, dk, dv = torch.zeros_like(q), torch.empty_like(kv), torch.empty_like(kv)
    dout[0, -1], dout[0, 0] = 3.0, 1.0
    g = B.attention_grads_struct(a, dout, dk=dk, dv=dv)
    B.attention_bwd(a, g, _ws(B.attention_bwd_workspace_bytes(a, g)))
    # the first query gives half of 1 to each state, the last all of 3 to the second
    assert bool((dv[0, 0] == 0.5).all()) and bool((dv[0, 1] == 3.5).all()), (dv[0, :, 0, 0], )


@pytest.mark.parametrize("c,groups", [(1024, 4), (4100, 5)])
def test_group_norm_beyond_32_bit_offsets(c, groups):
    """Images past 2^32 bytes: what the last pixels get, against their formula."""
    n, p = 2, (1 << 31) // c + 77
    say(f"[gpu] group norm {n} x {p} x {c}")
    x = torch.empty(n, p, c, dtype=torch.bfloat16, device="cuda")
    for i in range(n):                                      # alternating pixels: mean 1 + i, variance 4
        x[i, ::2], x[i, 1::2] = 3.0 + i, -1.0 + i
    mean, rstd, y = torch.empty(n, groups, device="cuda"), torch.empty(n, groups, device="cuda"), torch.empty_like(x)
    B.group_norm_fwd(x, y, groups, act="relu", mean=mean, rstd=rstd, eps=0.0, workspace=_ws(B.group_norm_fwd_workspace_bytes(n, p, c, groups)))
    odd = p % 2 / p                                         # one pixel more of 3 + i
    assert (mean.cpu() - torch.tensor([[1.0], [2.0]])).abs().max() < 4 * odd + 1e-5 and (rstd.cpu() - 0.5).abs().max() < odd + 1e-5
    assert bool((y[:, ::2] == 1.0).all()) and bool((y[:, 1::2] == 0.0).all())
    dy, dg, db = y, torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    B.group_norm_bwd(x, mean, rstd, dy, x, groups, act="relu", dgamma=dg, dbeta=db, workspace=_ws(B.group_norm_bwd_workspace_bytes(n, p, c, groups)))
    # dz is 1 on half of the pixels, where h is 1: dz - 1/2 - h / 2 is 0 everywhere
    half = n * (p + p % 2) / 2
    assert (dg - half).abs().max() <= 1e-4 * half and (db - half).abs().max() <= 1e-4 * half
    assert float(x.float().abs().max()) < 1e-3


def test_many_small_images():
    n, p, c, groups = 65535, 3, 8, 2
    x = torch.randn(n, p, c, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    y, mean, rstd = torch.empty_like(x), torch.empty(n, groups, device="cuda"), torch.empty(n, groups, device="cuda")
    B.group_norm_fwd(x, y, groups, mean=mean, rstd=rstd, workspace=_ws(B.group_norm_fwd_workspace_bytes(n, p, c, groups)))
    v = x.double().view(n, p, groups, 4)
    m = v.mean((1, 3), keepdim=True)
    want = ((v - m) / (v.var((1, 3), correction=0, keepdim=True) + 1e-5).sqrt()).view(n, p, c)
    assert float((y - want).abs().max()) < 2e-5


def test_many_batches_of_heads():
    """More pairs of batch element and head than a dimension of a launch has."""
    b, h, d = 20000, 8, 8
    say(f"[gpu] attention of {b} x {h} pairs")
    gen = torch.Generator("cuda").manual_seed(1)
    e = lambda n: torch.randn((b, n, h, d), generator=gen, device="cuda")
    q, k, v = e(2), e(5), e(5)
    out, lse = torch.empty_like(q), torch.empty(b, h, 2, device="cuda")
    a = B.attention_struct(q, k, v, out, lse=lse)
    B.attention_fwd(a, _ws(B.attention_fwd_workspace_bytes(a)))
    t = lambda x: x.double().transpose(1, 2).contiguous()
    s = torch.matmul(t(q), t(k).transpose(2, 3).contiguous()) * d ** -0.5
    want = torch.matmul(torch.softmax(s, 3), t(v)).transpose(1, 2)
    assert float((out - want).abs().max()) < 2e-5 and float((lse - torch.logsumexp(s, 3)).abs().max()) < 1e-5
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    g = B.attention_grads_struct(a, q, dq=dq, dk=dk, dv=dv)
    B.attention_bwd(a, g, _ws(B.attention_bwd_workspace_bytes(a, g)))
    assert float((dv - torch.matmul(torch.softmax(s, 3).transpose(2, 3).contiguous(), t(q)).transpose(1, 2)).abs().max()) < 2e-5
