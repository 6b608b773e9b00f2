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
    assert hocf.hocf_moe_route_workspace_bytes(60) == 9 * 64 * 8 and hocf.hocf_moe_route_workspace_bytes(0) == 0
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


SLOTS = dict(T=100, topk=2, bins=4, per_bin=2, cap=64, experts=addr(1), index=addr(2), pair=addr(3), counts=addr(4),
             s=None)


def slots(**kw):
    a = dict(SLOTS, **kw)
    s = a.pop("s")
    return hocf.hocf_moe_slots(*a.values(), sync() if s is None else s)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INVALID), (dict(T=1 << 30), INVALID), (dict(topk=0), INVALID), (dict(bins=0), INVALID),
    (dict(per_bin=0), INVALID), (dict(bins=64, per_bin=1 << 25), INVALID), (dict(cap=-1), INVALID),
    (dict(cap=1 << 29), INVALID), (dict(bins=65), UNSUPPORTED), (dict(experts=None), INVALID),
    (dict(index=None), INVALID), (dict(pair=None), INVALID), (dict(counts=None), INVALID),
    (dict(counts=addr(4) + 8), INVALID), (dict(pair=addr(1)), INVALID), (dict(index=addr(3) + 1008), INVALID),
    (dict(s=sync(nbytes=16)), INVALID), (dict(s=sync(epoch=0)), INVALID), (dict(s=sync(ws=addr(2))), INVALID),
])
def test_slots_rejects(kw, expect):
    assert slots(**kw) == expect


def test_slots_accepts():
    assert hocf.hocf_moe_slots_workspace_bytes(100, 2, 4) == 64 * 4
    assert hocf.hocf_moe_slots_workspace_bytes(1 << 20, 8, 4) == 256 * 64 * 4
    assert hocf.hocf_moe_slots_workspace_bytes(0, 2, 4) == 0
    valid(slots())
    valid(slots(T=0, experts=None, index=None, s=sync(ws=0, nbytes=0)))
    valid(slots(cap=0, pair=None))


COMBINE = dict(T=10, topk=2, N=64, R=40, dt=BF16, out_dt=F32, rows=addr(1), weights=addr(2), index=addr(3),
               add=addr(4), out=addr(5), s=None)


def combine(**kw):
    a = dict(COMBINE, **kw)
    s = a.pop("s")
    return hocf.hocf_moe_combine(*a.values(), sync() if s is None else s)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INVALID), (dict(R=-1), INVALID), (dict(topk=0), INVALID), (dict(N=-8), INVALID),
    (dict(N=60), INVALID), (dict(dt=3), INVALID), (dict(out_dt=-1), INVALID), (dict(index=None), INVALID),
    (dict(topk=17), UNSUPPORTED), (dict(N=(1 << 24) + 8), UNSUPPORTED), (dict(rows=None), INVALID),
    (dict(weights=None), INVALID), (dict(out=None), INVALID), (dict(rows=addr(1) + 8), INVALID),
    (dict(add=addr(4) + 4), INVALID), (dict(out=addr(4)), INVALID), (dict(out=addr(1)), INVALID),
    (dict(out=addr(3)), INVALID), (dict(s=sync(epoch=0)), INVALID),
])
def test_combine_rejects(kw, expect):
    assert combine(**kw) == expect


def test_combine_accepts():
    assert combine(T=0, rows=None, weights=None, out=None) == OK
    assert combine(N=0) == OK
    valid(combine())
    valid(combine(R=0, rows=None))
    valid(combine(R=20, index=None, add=None))


CBWD = dict(T=10, topk=2, N=64, R=40, dt=BF16, out_dt=F32, rows=addr(1), weights=addr(2), dout=addr(3), index=addr(4),
            pair=addr(5), drows=addr(6), dweights=addr(7), s=None)


def combine_bwd(**kw):
    a = dict(CBWD, **kw)
    s = a.pop("s")
    return hocf.hocf_moe_combine_bwd(*a.values(), sync() if s is None else s)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INVALID), (dict(N=4), INVALID), (dict(dt=2), INVALID), (dict(topk=17), UNSUPPORTED),
    (dict(index=None), INVALID), (dict(pair=None), INVALID), (dict(index=None, pair=None), INVALID),
    (dict(R=20, index=None), INVALID), (dict(T=0, pair=None), INVALID), (dict(rows=None), INVALID),
    (dict(dout=None), INVALID), (dict(drows=None), INVALID), (dict(dweights=None), INVALID),
    (dict(dweights=addr(7) + 4), INVALID), (dict(drows=addr(1)), INVALID), (dict(dweights=addr(2)), INVALID),
    (dict(drows=addr(5)), INVALID), (dict(s=sync(epoch=0)), INVALID),
])
def test_combine_bwd_rejects(kw, expect):
    assert combine_bwd(**kw) == expect


def test_combine_bwd_accepts():
    assert combine_bwd(T=0, R=0, index=None, pair=None) == OK
    valid(combine_bwd())
    valid(combine_bwd(R=20, index=None, pair=None))
    valid(combine_bwd(T=0, index=None, weights=None, dout=None, dweights=None))
    valid(combine_bwd(R=0, rows=None, drows=None, pair=None))


W4 = dict(R=8, rows_per_x=2, E=4, e0=0, N=64, K=256, group=64, out_dt=F32, x=addr(1), experts=addr(2), wq=addr(3),
          scales=addr(4), zeros=addr(5), out=addr(6), s=None)


def w4(**kw):
    a = dict(W4, **kw)
    s = a.pop("s")
    return hocf.hocf_gemv_w4(*a.values(), sync() if s is None else s)


@pytest.mark.parametrize("kw,expect", [
    (dict(R=-2), INVALID), (dict(rows_per_x=0), INVALID), (dict(rows_per_x=3), INVALID), (dict(E=0), INVALID),
    (dict(e0=-1), INVALID), (dict(e0=2 ** 31 - 4), INVALID), (dict(N=60), INVALID), (dict(K=-8), INVALID),
    (dict(K=12), INVALID), (dict(out_dt=5), INVALID), (dict(experts=None), INVALID), (dict(group=16), UNSUPPORTED),
    (dict(group=256), UNSUPPORTED), (dict(R=1026), UNSUPPORTED), (dict(N=(1 << 20) + 8), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(wq=None), INVALID), (dict(scales=None), INVALID), (dict(out=None), INVALID),
    (dict(zeros=addr(5) + 2), INVALID), (dict(out=addr(1)), INVALID), (dict(out=addr(3) + 1024), INVALID),
    (dict(out=addr(2)), INVALID), (dict(s=sync(epoch=0)), INVALID),
])
def test_gemv_w4_rejects(kw, expect):
    assert w4(**kw) == expect


def test_gemv_w4_accepts():
    assert w4(R=0, x=None, out=None) == OK and w4(N=0) == OK
    valid(w4())
    valid(w4(E=1, experts=None, zeros=None))
    valid(w4(K=0, x=None, wq=None, scales=None, zeros=None))


PACK = dict(E=2, N=64, K=256, group=64, codes=addr(1), scales=addr(2), zeros=addr(3), wq=addr(4), scales_out=addr(5),
            zeros_out=addr(6))


@pytest.mark.parametrize("kw,expect", [
    (dict(E=0), INVALID), (dict(N=4), INVALID), (dict(K=4), INVALID), (dict(group=48), UNSUPPORTED),
    (dict(K=(1 << 20) + 8), UNSUPPORTED), (dict(zeros=None), INVALID), (dict(zeros_out=None), INVALID),
    (dict(codes=None), INVALID), (dict(scales_out=None), INVALID), (dict(wq=addr(4) + 4), INVALID),
    (dict(wq=addr(1)), INVALID), (dict(scales_out=addr(2)), INVALID), (dict(zeros_out=addr(5)), INVALID),
])
def test_w4_pack_rejects(kw, expect):
    assert hocf.hocf_w4_pack(*dict(PACK, **kw).values()) == expect


def test_w4_pack_accepts():
    assert hocf.hocf_w4_pack(*dict(PACK, K=0).values()) == OK


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
