"""Views that are not there, in ViewReader (gaussian_splatting_tile_amd/head.py):
whatever their maps hold, the result and every gradient are those of maps of
zeros in their place, bit for bit."""

import pytest
import torch

from gaussian_splatting_tile_amd import head as H

pytestmark = pytest.mark.gpu


def _step(r, tokens, features, seen, d_out):
    out = r.forward(tokens, features, seen).clone()
    d_tokens, d_features = r.backward(d_out)
    return {"out": out, "tokens": d_tokens.clone(), "features": d_features.clone(), **{k: v.clone() for k, v in r.grads.items()}}


def _inputs(dtype, views, pixels):
    gen = torch.Generator("cuda").manual_seed(7)
    e = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)
    return e(40, 64), e(views, pixels, 96), e(40, 64) * 0.1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("pixels", [30, 900])              # a map of one workgroup, and of more
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), None])
def test_absent_views_give_no_gradient(dtype, pixels, bad):
    r = H.ViewReader(40, 64, 4, pixels, 96, 4, 6, dtype=dtype, seed=1)
    tokens, features, d_out = _inputs(dtype, 4, pixels)
    seen = torch.tensor([1, 0, 1, 0], dtype=torch.uint8, device="cuda")
    if bad is not None:
        features[1] = bad
        features[3, pixels // 2, 5] = bad
    else:                                                  # finite, but its squares are not
        features[1] = torch.finfo(dtype).max
    clean = features.clone()
    clean[1] = clean[3] = 0.0
    given = features.clone()
    got, want = _step(r, tokens, features, seen, d_out), _step(r, tokens, clean, seen, d_out)
    for k, w in want.items():
        assert bool(torch.isfinite(w.float()).all()) and float(w.float().abs().max()) > 0, k
        assert torch.equal(got[k], w), k
    assert bool((got["features"][1::2] == 0).all())
    assert torch.equal(features.nan_to_num(), given.nan_to_num())          # the caller's maps stay as they were


def test_all_views_seen_or_none():
    r = H.ViewReader(40, 64, 3, 200, 96, 4, 6, seed=1)
    tokens, features, d_out = _inputs(torch.bfloat16, 3, 200)
    want = _step(r, tokens, features, None, d_out)
    for seen in (torch.ones(3, dtype=torch.bool, device="cuda"), torch.full((3,), 255, dtype=torch.uint8, device="cuda"), torch.ones(3, dtype=torch.uint8)):
        got = _step(r, tokens, features, seen, d_out)
        assert all(torch.equal(got[k], w) for k, w in want.items())
    got = _step(r, tokens, torch.full_like(features, float("nan")), torch.zeros(3, dtype=torch.bool, device="cuda"), d_out)
    assert torch.equal(got["out"], (tokens.float() + r.b_o).bfloat16())
    assert all(bool(torch.isfinite(x.float()).all()) for x in got.values())
    assert bool((got["w_kv"] == 0).all()) and bool((got["features"] == 0).all())


def test_absent_views_in_a_graph():
    """The views that are there change between replays, with eager work between."""
    r = H.ViewReader(40, 64, 3, 300, 96, 4, 6, seed=1)
    tokens, features, d_out = _inputs(torch.bfloat16, 3, 300)
    seen = torch.ones(3, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.forward(tokens, features, seen)
        r.backward(d_out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.forward(tokens, features, seen)
        r.backward(d_out)
    for i in range(3):
        seen.fill_(1)
        seen[i] = 0
        held = features[i].clone()
        features[i] = float("nan")
        want = _step(r, tokens, features, seen, d_out)
        for v in r.grads.values():
            v.zero_()
        torch.randn(1000, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        got = {"out": r.out, "tokens": r.d_tokens, "features": r.d_features, **r.grads}
        for k, w in want.items():
            assert bool(torch.isfinite(w.float()).all()) and torch.equal(got[k], w), (i, k)
        features[i] = held


def test_maps_and_tokens_of_an_encoder_that_torch_differentiates():
    """The reader's gradients are its own; what comes with a history is taken as it is."""
    r = H.ViewReader(40, 64, 3, 200, 96, 4, 6, seed=1)
    tokens, features, d_out = _inputs(torch.bfloat16, 3, 200)
    seen = torch.tensor([1, 0, 1], dtype=torch.uint8, device="cuda")
    want = [_step(r, tokens, features, s, d_out) for s in (seen, None)]
    leaf, scale = features.clone().requires_grad_(), torch.ones((), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    for s, w in zip((seen, None), want):
        got = _step(r, tokens * scale, leaf * 1, s, d_out)
        assert all(torch.equal(got[k], w[k]) for k in w)
        assert not any(t.requires_grad for t in (r.tokens, r.f, r.out, *got.values()))
