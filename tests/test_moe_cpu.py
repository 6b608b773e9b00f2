"""The mixture-of-experts operators' refusals and the plain 64-bit references
that the GPU tests compare with (CPU only: no compute call)."""

import ctypes

import numpy as np
import pytest

import moe_ref as ref
from computation_collective_amd import hocf

OK, INVALID, UNSUPPORTED, HIP = 0, hocf.HOCF_ERR_INVALID_ARG, hocf.HOCF_ERR_UNSUPPORTED, hocf.HOCF_ERR_HIP
F32, BF16 = hocf.HOCF_F32, hocf.HOCF_BF16


def addr(n):
    """Fake device addresses a TiB apart, never dereferenced."""
    return (1 << 44) + (n << 40)


def sync(epoch=1, ws=None, nbytes=1 << 24):
    return hocf.sync(epoch, addr(60) if ws is None else ws, nbytes, status=addr(61))


def gpu():
    import torch
    return torch.cuda.is_available()


def valid(st):
    """A valid call passes every check; without a GPU it stops at the device query."""
    if gpu():
        pytest.skip("GPU present")
    assert st == HIP


ROUTE = dict(T=64, E=64, topk=4, dt=F32, logits=addr(1), ld=64, bias=None, score=0, n_group=1, topk_group=1,
             group_top=1, renorm=0, scale=1.0, experts=addr(2), weights=addr(3), counts=addr(4), s=None)


def route(**kw):
    a = dict(ROUTE, **kw)
    s = a.pop("s")
    return hocf.hocf_moe_route(*a.values(), sync() if s is None else s)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(E=0), INVALID), (dict(topk=0), INVALID),
    (dict(topk=65), INVALID), (dict(dt=7), INVALID), (dict(score=2), INVALID), (dict(renorm=2), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID), (dict(ld=63), INVALID),
    (dict(ld=(1 << 24) + 1), INVALID), (dict(n_group=0), INVALID), (dict(n_group=5), INVALID),
    (dict(n_group=4, topk_group=5), INVALID), (dict(n_group=4, topk_group=0), INVALID), (dict(group_top=3), INVALID),
    (dict(E=1024, ld=1024), UNSUPPORTED), (dict(topk=17), UNSUPPORTED),
    (dict(E=256, ld=256, n_group=128, topk_group=1), UNSUPPORTED),
    (dict(logits=None), INVALID), (dict(experts=None), INVALID), (dict(weights=addr(3) + 4), INVALID),
    (dict(weights=addr(2) + 16), INVALID), (dict(counts=addr(1)), INVALID), (dict(bias=addr(4)), INVALID),
    (dict(s=sync(epoch=0)), INVALID), (dict(s=sync(nbytes=64 * 4)), INVALID), (dict(s=sync(ws=0)), INVALID),
    (dict(s=sync(ws=addr(1))), INVALID),
])
def test_route_rejects(kw, expect):
    assert route(**kw) == expect
    assert hocf.last_error().startswith("moe_route") or "s" in kw


def test_route_accepts():
    assert hocf.hocf_moe_route_workspace_bytes(64) == 65 * 4 and hocf.hocf_moe_route_workspace_bytes(0) == 0
    assert route(T=0, counts=None, logits=None, experts=None, weights=None) == OK
    valid(route())
    valid(route(counts=None, s=sync(ws=0, nbytes=0)))      # no counts: no workspace


BWD = dict(T=64, E=64, topk=4, dt=F32, logits=addr(1), ld=64, experts=addr(2), dweights=addr(3), score=0, renorm=0,
           scale=1.0, dlogits=addr(4), s=None)


def route_bwd(**kw):
    a = dict(BWD, **kw)
    s = a.pop("s")
    return hocf.hocf_moe_route_bwd(*a.values(), sync() if s is None else s)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(topk=65), INVALID), (dict(dt=2), INVALID),
    (dict(score=-1), INVALID), (dict(renorm=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(ld=8), INVALID),
    (dict(E=513, ld=513), UNSUPPORTED), (dict(topk=17), UNSUPPORTED), (dict(dlogits=None), INVALID),
    (dict(logits=addr(1) + 2), INVALID), (dict(dlogits=addr(1)), INVALID), (dict(dlogits=addr(3)), INVALID),
    (dict(s=sync(epoch=0)), INVALID),
])
def test_route_bwd_rejects(kw, expect):
    assert route_bwd(**kw) == expect


def test_route_bwd_accepts():
    assert route_bwd(T=0, logits=None, dlogits=None) == OK
    valid(route_bwd())


def test_null_sync_is_refused():
    L = hocf.lib()
    none = ctypes.POINTER(hocf.hocf_sync)()
    assert L.hocf_moe_route(1, 4, 1, F32, addr(1), 4, None, 0, 1, 1, 1, 0, 1.0, addr(2), addr(3), None, none, None) == INVALID
    assert L.hocf_moe_route_bwd(1, 4, 1, F32, addr(1), 4, addr(2), addr(3), 0, 0, 1.0, addr(4), none, None) == INVALID


# ------------------------------------------------------------------ the references themselves

def test_route_reference_by_hand():
    x = np.array([[0.0, 2.0, 2.0, -np.inf], [-np.inf] * 4, [np.nan, 1.0, -np.inf, 1.0]])
    e, w, c = ref.route(x, 2)
    assert e.tolist() == [[1, 2], [-1, -1], [1, 3]] and c.tolist() == [0, 2, 1, 1]
    p = 1 / (2 + np.exp(-2.0))
    assert np.allclose(w, [[p, p], [0, 0], [0.5, 0.5]], rtol=1e-15)
    # groups of two: by their largest, group 1 (3.0); by the sum of two, group 0 (2 + 2 > 3 + 0)
    y = np.array([[2.0, 2.0, 3.0, -9.0]])
    assert ref.route(y, 2, score=ref.SIGMOID, n_group=2, group_top=1)[0].tolist() == [[2, 3]]
    assert ref.route(y, 2, score=ref.SIGMOID, n_group=2, group_top=2)[0].tolist() == [[0, 1]]
    # the bias moves the choice, not the weight
    e, w, _ = ref.route(y, 1, bias=np.array([0, 0, 0, 1.0]), score=ref.SIGMOID, scale=2.0)
    assert e.tolist() == [[3]] and w[0, 0] == pytest.approx(2 / (1 + np.exp(9.0)), rel=1e-15)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_reference_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(3, 7))
    x[0, 2] = -np.inf
    e, _, _ = ref.route(x, 3, score=score, renorm=renorm)
    e[1, 2] = -1
    dw = rng.normal(size=e.shape)
    d, _ = ref.route_bwd(x, e, dw, score, renorm, 2.5)
    h = 1e-6
    for t in range(3):
        for k in range(7):
            up, dn = x.copy(), x.copy()
            up[t, k] += h
            dn[t, k] -= h
            num = ((ref.weights_of(up, e, score, renorm, 2.5) - ref.weights_of(dn, e, score, renorm, 2.5)) * dw).sum() / (2 * h)
            assert d[t, k] == pytest.approx(num, abs=1e-8)
