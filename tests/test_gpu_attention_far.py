"""Attention's gradients at the far end of its sizes by value, and fp16
probabilities of little weight in every form of the forward."""

import math

import pytest
import torch

from gaussian_splatting_tile_amd import binding as B
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def _ws(n):
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("d", [128, 124])                  # read in place, and packed first
def test_gradients_of_states_beyond_32_bit_offsets(d):
    """The last two states share all weight (the others have exp(-d) of it, 0 in
    fp32): k is 16 in one half of d or in the other, v the last one's 0, 1, .. and
    0.  With N = sum v: dS = +-N / 4 and dq = +-1/8 x 16 N / 4.  P is off by 8 E d (the
    constants, products and sums in scores and lse), dS and the results by 2^-8 each."""
    nk = (1 << 24) + 70
    say(f"[gpu] attention gradients over {nk} states of {d}")
    k, v = (torch.zeros(1, nk, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    half = torch.arange(d, device="cuda") < d // 2
    k[0, -1, 0], k[0, -2, 0] = half * 16.0, ~half * 16.0
    v[0, -1] = torch.arange(d, device="cuda").bfloat16()
    q = torch.ones(1, 3, 1, d, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(1, 1, 3, device="cuda")
    a = B.attention_struct(q, k, v, out, lse=lse, scale=0.125)
    B.attention_fwd(a, _ws(B.attention_fwd_workspace_bytes(a)))
    assert torch.equal(out, (v[:, -1:].float() / 2).bfloat16().expand_as(out))
    assert float((lse - (d + math.log(2))).abs().max()) <= 8 * E * d
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    g = B.attention_grads_struct(a, q, dq=dq, dk=dk, dv=dv)
    B.attention_bwd(a, g, _ws(B.attention_bwd_workspace_bytes(a, g)))
    ds = d * (d - 1) / 2 / 4
    sign = torch.where(half, 1.0, -1.0).double()
    near = lambda got, want: float((got.double() / want - 1).abs().max()) <= 2.05 * 2.0 ** -8
    assert near(dq[0, :, 0], 0.125 * 16 * ds * sign)
    assert near(dk[0, -1, 0], 3 * 0.125 * ds) and near(dk[0, -2, 0], -3 * 0.125 * ds)
    assert near(dv[0, -2:], 1.5)
    assert bool((dk[0, :-2] == 0).all()) and bool((dv[0, :-2] == 0).all())


def test_gradients_of_many_rows_of_queries():
    """2^24 queries of two states, 0 and 2, which are k and v; rows of dq past 2^31
    elements.  The first query weighs both alike: delta = 128, dS = -+64, dq = 1/4 x 64 x 2.
    The last takes the second state alone, so dS is 0; the others have no dout."""
    nq, d = (1 << 24) + 33, 128
    say(f"[gpu] attention gradients of {nq} queries")
    q = torch.zeros(1, nq, 1, d, dtype=torch.bfloat16, device="cuda")
    q[0, -1] = 1.0
    kv = torch.zeros(1, 2, 1, d, dtype=torch.bfloat16, device="cuda")
    kv[0, 1] = 2.0
    out, lse = torch.empty_like(q), torch.empty(1, 1, nq, device="cuda")
    a = B.attention_struct(q, kv, kv, out, lse=lse, scale=0.25)
    B.attention_fwd(a, _ws(B.attention_fwd_workspace_bytes(a)))
    dout, dq, dk, dv = torch.zeros_like(q), torch.full_like(q, 7.0), torch.empty_like(kv), torch.empty_like(kv)
    dout[0, -1], dout[0, 0] = 3.0, 1.0
    dout[0, -2] = 1.0                                      # like the first, at the far end
    g = B.attention_grads_struct(a, dout, dq=dq, dk=dk, dv=dv)
    B.attention_bwd(a, g, _ws(B.attention_bwd_workspace_bytes(a, g)))
    assert bool((dq[0, 0] == 32.0).all()) and bool((dq[0, -2] == 32.0).all())
    assert bool((dq[0, 1:-2] == 0.0).all()) and bool((dq[0, -1] == 0.0).all())
    assert bool((dv[0, 0] == 1.0).all()) and bool((dv[0, 1] == 4.0).all())
    # q is 0 but in the last row, whose dS is -768 exp(-64) for the first state, 0 for the second
    assert float(dk[0, 0].float().abs().max()) <= 1e-25 and bool((dk[0, 1] == 0).all())


def test_gradients_of_many_batches_of_heads():
    """All three against their formulas, fp32: a score is off by (d + 20) E of its terms'
    magnitudes, dP and delta alike, P by what its score and lse are, and dS and the results' products by
    a few E; three limbs add nothing to that."""
    b, h, d, s = 20000, 8, 8, 8 ** -0.5
    gen = torch.Generator("cuda").manual_seed(1)
    e = lambda n: torch.randn((b, n, h, d), generator=gen, device="cuda")
    q, k, v, dout = e(2), e(5), e(5), e(2)
    out, lse = torch.empty_like(q), torch.empty(b, h, 2, device="cuda")
    a = B.attention_struct(q, k, v, out, lse=lse)
    B.attention_fwd(a, _ws(B.attention_fwd_workspace_bytes(a)))
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    g = B.attention_grads_struct(a, dout, dq=dq, dk=dk, dv=dv)
    B.attention_bwd(a, g, _ws(B.attention_bwd_workspace_bytes(a, g)))
    t = lambda x: x.double().transpose(1, 2).contiguous()
    x = lambda y: y.transpose(2, 3).contiguous()
    Q, K, V, D, O = (t(y) for y in (q, k, v, dout, out))
    S = torch.matmul(Q, x(K)) * s
    P = torch.exp(S - lse.double()[..., None])
    dP = torch.matmul(D, x(V))
    dS = P * (dP - (D * O).sum(3, keepdim=True))
    r = (d + 20) * E * s * torch.matmul(Q.abs(), x(K).abs()) + 4 * E * (4 + S.abs() + lse.double().abs()[..., None])
    off = P * (d + 20) * E * (torch.matmul(D.abs(), x(V).abs()) + (D * O).abs().sum(3, keepdim=True)) + (2 * r + 40 * E) * dS.abs()
    for name, got, want, tol in (("dq", dq, s * torch.matmul(dS, K), s * torch.matmul(off, K.abs())),
                                 ("dk", dk, s * torch.matmul(x(dS), Q), s * torch.matmul(x(off), Q.abs())),
                                 ("dv", dv, torch.matmul(x(P), D), torch.matmul(x(P * (2 * r + 40 * E)), D.abs()))):
        err = ((t(got) - want).abs() / (tol + 1e-30)).max()
        assert float(err) <= 1.0, (name, float(err))


@pytest.mark.parametrize("nq,h,kv,d", [(1, 2, 2, 8), (3, 4, 1, 128), (20, 1, 1, 64), (70, 4, 2, 40), (300, 2, 2, 96), (8192, 4, 4, 64)])
@pytest.mark.parametrize("states", ["all", "masked", "ragged"])
def test_fp16_states_of_little_weight(nq, h, kv, d, states):
    """States 2^-20.5 of the first one's weight make up all of out, in one walk or
    in splits with maxima of their own, by one wave or four, in whole tiles or not.
    Held times 2^6, half a step of the smallest is 2^-10.5 of each; to that come out's
    rounding, 2^-11, and 2^-12 for 4096 additions in fp32.  The sum of lse takes 32 values
    of a tile and then 64 tiles' sums, each addition E of the whole at most."""
    nk, s = 4096, 14.203125
    k, v = torch.zeros(2, nk, kv, d), torch.ones(2, nk, kv, d)
    k[:, 1:, :, 0], v[:, 0] = -s, 0.0
    k, v = k.half().cuda(), v.half().cuda()
    count = torch.full((2,), nk)
    mask = lengths = None
    if states == "masked":
        mask = torch.ones(2, nk, dtype=torch.uint8)
        mask[0, 1::3], mask[1, 700:1900] = 0, 0
        count = mask.sum(1, dtype=torch.int64)
        mask = mask.cuda()
        k[mask == 0], v[mask == 0] = float("nan"), float("inf")
    elif states == "ragged":
        count = torch.tensor([4001, 1030])
        lengths = count.int().cuda()
    q = torch.ones(1, 1, 1, d, dtype=torch.float16, device="cuda").expand(2, nq, h, d)
    out, lse = torch.empty(2, nq, h, d, dtype=torch.float16, device="cuda"), torch.empty(2, h, nq, device="cuda")
    a = B.attention_struct(q, k, v, out, lse=lse, kv_lengths=lengths, kv_mask=mask, scale=1.0)
    B.attention_fwd(a, _ws(B.attention_fwd_workspace_bytes(a)))
    for i in range(2):
        mass = (int(count[i]) - 1) * math.exp(-s)
        want = mass / (1 + mass)
        assert float((out[i].double() - want).abs().max()) <= want * (2.0 ** -10.5 + 2.0 ** -11 + 2.0 ** -12), i
        assert float((lse[i].double() - math.log1p(mass)).abs().max()) <= (nk // 64 + 128) * E, i
