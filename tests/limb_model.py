"""What limb products lose, by a model of them on the CPU, and the bounds that
follow for the tests of the kernels.

A value is held as `nl` bf16 limbs, a product of two is formed from the pairs
i + j < nl, 32 k at a time into an fp32 sum, smallest pairs first.  Relative
Frobenius errors of that model, next to those with a limb fewer:

  products of fp32 (k = 32 .. 13001)       3 limbs 3e-8 .. 9e-7, 2 limbs 4.3e-6 .. 4.7e-6
  orthogonalised noise with strong directions,
    fp32 result                            3 limbs 3e-7 .. 1.5e-6, 2 limbs 3.0e-5 .. 5.7e-5
    bf16 result against the rounded one    2 limbs up to 5.8e-4, 1 limb from 1.7e-2
    fp16 result against the rounded one    2 limbs up to 1.8e-4, 1 limb from 1.7e-2
  orthogonalised rank 1 (errors in the empty directions grow 3.4445^5-fold)
                                           3 limbs up to 3.8e-5, 2 limbs from 1.5e-3

Each bound lies between the two, at about their geometric mean."""

import torch

from oracle import network as N

LINEAR_F32 = 1.8e-6
ORTHO = {torch.float32: 6e-6, torch.bfloat16: 3e-3, torch.float16: 1e-3}
ORTHO_RANK_1 = 2e-4


def limbs(x, nl):
    out, rest = [], x.float()
    for _ in range(nl):
        head = rest.bfloat16().float()
        out.append(head.double())
        rest = rest - head
    return out


def product(a, b, nl):
    """a [r][k] b [q][k]^T in fp32."""
    pa, pb = limbs(a, nl), limbs(b, nl)
    acc = torch.zeros(a.shape[0], b.shape[0])
    for k in range(0, a.shape[1], 32):
        for order in range(nl - 1, -1, -1):
            for i in range(order + 1):
                acc = (acc.double() + pa[i][:, k:k + 32] @ pb[order - i][:, k:k + 32].T).float()
    return acc


def orthogonalize(u, nl, eps=1e-7):
    a, b, c = N.COEFFS
    held = lambda v: sum(limbs(v, nl)).float()
    u = u.double()
    tall = u.shape[0] > u.shape[1]
    x = held((u.T if tall else u) / (u.norm() + eps))
    for _ in range(5):
        p = held(product(x, x, nl))
        q = held(b * p + c * product(p, p, nl))
        last = a * x + product(x.T.contiguous(), q, nl).T
        x = held(last)
    return last.T if tall else last


def error(got, want, t=torch.float32):
    """Relative Frobenius distance of `got` from `want` (fp64), which is rounded
    to t first if that is a 16-bit type."""
    want = torch.as_tensor(want)
    if t is not torch.float32:
        want = want.to(t).double()
    return float((torch.as_tensor(got).double().cpu() - want).norm() / want.norm())
