"""The 8-bit integer operators' refusals and the plain 64-bit references that
the GPU tests compare with (CPU only: no compute call)."""

import numpy as np
import pytest

import i8_ref as ref
from computation_collective_amd import hocf
from test_moe_cpu import BF16, F32, INVALID, OK, UNSUPPORTED, addr, sync, valid

QUANT = dict(T=64, K=128, dt=BF16, x=addr(1), ld=128, act=0, codes=addr(2), scales=addr(3), pre_codes=None,
             pre_scales=None, s=None)
DEQUANT = dict(T=64, K=128, out_dt=BF16, codes=addr(1), scales=addr(2), out=addr(3), s=None)
WEIGHTS = dict(E=2, N=64, K=128, dt=BF16, W=addr(1), wq=addr(2), scales=addr(3), s=None)
GEMM = dict(E=2, T=64, N=64, K=128, out_dt=BF16, xq=addr(1), xs=addr(2), wq=addr(3), ws=addr(4), offsets=addr(5),
            out=addr(6), s=None)
GEMV = dict(R=8, rows_per_x=2, E=4, e0=0, N=64, K=128, out_dt=F32, xq=addr(1), xs=addr(2), experts=addr(3),
            wq=addr(4), ws=addr(5), out=addr(6), s=None)
DX = dict(E=2, T=64, N=64, K=128, out_dt=BF16, dy=addr(1), wq=addr(2), ws=addr(3), offsets=addr(4), pre_codes=None,
          pre_scales=None, dx=addr(7), s=None)
DW = dict(E=2, T=64, N=64, K=128, out_dt=F32, xq=addr(1), xs=addr(2), dy=addr(3), offsets=addr(4), dw=addr(5), s=None)
ALL = {"quant_i8": QUANT, "dequant_i8": DEQUANT, "weights_i8": WEIGHTS, "gemm_i8": GEMM, "gemv_i8": GEMV,
       "gemm_i8_dx": DX, "gemm_i8_dw": DW}


def call(op, **kw):
    a = dict(ALL[op], **kw)
    s = a.pop("s")
    return getattr(hocf, "hocf_" + op)(*a.values(), sync() if s is None else s)


SIZES = [(dict(K=0), INVALID), (dict(K=-16), INVALID), (dict(K=24), INVALID), (dict(K=65552), UNSUPPORTED),
         (dict(s=sync(epoch=0)), INVALID)]
MATRICES = SIZES + [(dict(E=0), INVALID), (dict(N=0), INVALID), (dict(N=-8), INVALID), (dict(N=12), INVALID),
                    (dict(N=65544), UNSUPPORTED), (dict(E=1025), UNSUPPORTED)]
GROUPED = MATRICES + [(dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(out_dt=2), INVALID),
                      (dict(offsets=None), INVALID), (dict(offsets=addr(5) + 8), INVALID)]
CASES = {
    "quant_i8": SIZES + [
        (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(dt=2), INVALID), (dict(act=2), INVALID),
        (dict(act=-1), INVALID), (dict(ld=112), INVALID), (dict(ld=132), INVALID), (dict(dt=F32, ld=130), INVALID),
        (dict(ld=(1 << 24) + 8), INVALID), (dict(pre_codes=addr(4)), INVALID), (dict(act=1, pre_scales=addr(4)), INVALID),
        (dict(pre_codes=addr(4), pre_scales=addr(5)), INVALID),       # nothing before an activation that is none
        (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
        (dict(x=addr(1) + 8), INVALID), (dict(codes=addr(2) + 8), INVALID), (dict(codes=addr(1)), INVALID),
        (dict(x=addr(1), codes=addr(1) + 64 * 256 - 16), INVALID), (dict(scales=addr(2) + 64 * 128 - 16), INVALID),
        (dict(act=1, pre_codes=addr(2), pre_scales=addr(5)), INVALID)],
    "dequant_i8": SIZES + [
        (dict(T=-1), INVALID), (dict(out_dt=-1), INVALID), (dict(codes=None), INVALID), (dict(out=None), INVALID),
        (dict(out=addr(1)), INVALID), (dict(out=addr(2)), INVALID), (dict(scales=addr(2) + 4), INVALID)],
    "weights_i8": MATRICES + [
        (dict(dt=3), INVALID), (dict(W=None), INVALID), (dict(wq=None), INVALID), (dict(scales=None), INVALID),
        (dict(wq=addr(1)), INVALID), (dict(W=addr(1) + 2), INVALID), (dict(s=sync(nbytes=2 * 64 * 4 - 1)), INVALID),
        (dict(s=sync(ws=0)), INVALID), (dict(s=sync(ws=addr(2))), INVALID)],
    "gemm_i8": GROUPED + [
        (dict(xq=None), INVALID), (dict(ws=None), INVALID), (dict(out=addr(1)), INVALID), (dict(out=addr(4)), INVALID),
        (dict(out=addr(5)), INVALID), (dict(xs=addr(2) + 4), INVALID), (dict(out=addr(61)), INVALID)],
    "gemv_i8": MATRICES + [
        (dict(R=-2), INVALID), (dict(R=9), INVALID), (dict(rows_per_x=0), INVALID), (dict(R=1026), UNSUPPORTED),
        (dict(e0=-1), INVALID), (dict(e0=(1 << 31) - 4), INVALID), (dict(experts=None), INVALID),
        (dict(out_dt=5), INVALID), (dict(out=None), INVALID), (dict(out=addr(3)), INVALID), (dict(wq=addr(4) + 8), INVALID)],
    "gemm_i8_dx": GROUPED + [
        (dict(pre_codes=addr(5)), INVALID), (dict(pre_scales=addr(6)), INVALID), (dict(dy=None), INVALID),
        (dict(dx=addr(1)), INVALID), (dict(pre_codes=addr(5), pre_scales=addr(6), dx=addr(5)), INVALID),
        (dict(pre_codes=addr(5) + 4, pre_scales=addr(6)), INVALID)],
    "gemm_i8_dw": GROUPED + [
        (dict(dw=None), INVALID), (dict(dy=None), INVALID), (dict(dw=addr(1)), INVALID), (dict(dw=addr(3)), INVALID),
        (dict(T=0, dw=None), INVALID)],
}


@pytest.mark.parametrize("op,kw,expect", [(op, kw, e) for op, cases in CASES.items() for kw, e in cases])
def test_rejects(op, kw, expect):
    assert call(op, **kw) == expect
    assert hocf.last_error().startswith(op) or "s" in kw


def test_accepts():
    assert hocf.hocf_weights_i8_workspace_bytes(2, 64, 128) == 2 * 64 * 4
    assert hocf.hocf_weights_i8_workspace_bytes(2, 64, 272) == 2 * 2 * 64 * 4
    assert hocf.hocf_weights_i8_workspace_bytes(0, 64, 128) == 0
    assert call("quant_i8", T=0, x=None, codes=None, scales=None) == OK
    assert call("dequant_i8", T=0, codes=None, out=None) == OK
    assert call("gemm_i8", T=0, xq=None, out=None) == OK
    assert call("gemv_i8", R=0, xq=None, experts=None, E=1, out=None) == OK
    assert call("gemm_i8_dx", T=0, dy=None, dx=None) == OK
    for op in ALL:
        valid(call(op))
    valid(call("quant_i8", act=1, pre_codes=addr(4), pre_scales=addr(5)))
    valid(call("gemm_i8", E=1, offsets=None))
    valid(call("gemm_i8_dw", T=0, xq=None, xs=None, dy=None))       # the gradient of no rows is still written


def test_reference_bf16():
    import torch
    g = np.random.default_rng(1)
    v = np.concatenate([g.standard_normal(4000) * 10.0 ** g.integers(-44, 38, 4000), [0.0, -0.0, 3.4e38, 3.39e38, 1e-40]])
    # (through fp32 first: torch rounds twice from 64 bits, the reference once)
    v = v.astype(np.float32)
    assert np.array_equal(ref.to_bf16(v), torch.from_numpy(v).bfloat16().double().numpy())


def test_reference_quant():
    # 254 x / largest odd: halves, to the even code; the largest gets 127
    a = np.array([[127.0, 0.5, 1.5, -2.5, 126.5, 0.0], [0.0] * 6, [1.0, np.inf, 0, 0, 0, 0], [2.0 ** -130] * 6])
    q, s = ref.quant(a)
    assert q[0].tolist() == [127, 0, 2, -2, 126, 0] and s[0] == 1.0
    assert not q[1].any() and s[1] == 2.0 ** -126
    assert not q[2].any() and np.isnan(s[2])
    assert not q[3].any() and s[3] == 2.0 ** -126               # a sixteenth of the smallest scale
    x = np.random.default_rng(0).standard_normal((50, 64)).astype(np.float32).astype(np.float64)
    q, s = ref.quant(x)
    assert (np.abs(q.astype(int)).max(1) == 127).all()
    assert (np.abs(q * s.astype(np.float64)[:, None] - x) <= s[:, None] / 2 * (1 + 1e-12)).all()


def numerically(f, x, step=1e-4):
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[i] = step
        d[i] = (f(x + e) - f(x - e)) / (2 * step)
    return d


@pytest.mark.parametrize("act", [False, True])
def test_reference_gradients_against_differences(act):
    """The formulas are the gradients of sum(G . (act(h) W)) at h = x's held numbers, for each expert's rows."""
    g = np.random.default_rng(3)
    E, T, K, N, offsets = 2, 7, 16, 8, [1, 4, 6]
    hq, hs = ref.quant(2 * g.standard_normal((T, K)))
    wq, ws = ref.quant(g.standard_normal((E, N, K)))
    G = ref.to_bf16(g.standard_normal((T, N)))
    h, w = ref.held(hq, hs), np.stack([ref.held(wq[e], ws[e]).T for e in range(E)])

    def loss(h, w):
        a = ref.silu(h) if act else h
        return sum((G[lo:hi] * (a[lo:hi] @ w[e])).sum() for e, (lo, hi) in enumerate(ref.groups(offsets, E, T)))

    got, _ = ref.dx(G, wq, ws, offsets, (hq, hs) if act else None)
    want = numerically(lambda v: loss(v, w), h)
    inside = slice(offsets[0], offsets[-1])
    # a central difference is off by step^2 / 6 of the third derivative (SiLU's is below 0.5) and 1e-16 / step of the loss
    assert np.abs(got - want)[inside].max() < 1e-7 and np.isnan(got[0]).all() and np.isnan(got[6]).all()
    if not act:
        got, _ = ref.dw(hq, hs, G, E, offsets)
        assert np.abs(got - numerically(lambda v: loss(h, v), w)).max() < 1e-7


def test_handles_refuse():
    """What the Python handles check before any GPU call."""
    import torch
    from computation_collective_amd import buffers as bf
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        bf.QuantI8(4, 64, x)
    with pytest.raises(ValueError, match="shape"):
        bf.QuantI8(4, 32, x)
    with pytest.raises(ValueError, match="overlap"):
        bf.QuantI8(4, 64, x[:1].expand(4, 64))
    with pytest.raises(ValueError, match="adjacent"):
        bf.QuantI8(4, 32, x[:, ::2])
    with pytest.raises(ValueError, match="GPU"):
        bf.DequantI8(4, 64, q, s)
    with pytest.raises(ValueError, match="GPU"):
        bf.QuantI8(4, 64, x, keep=True)
    with pytest.raises(TypeError):
        bf.DequantI8(4, 64, q.float(), s)
    with pytest.raises(ValueError, match="contiguous"):
        bf.GemmI8(1, 64, 8, 4, q.t(), s, q, s)
    with pytest.raises(TypeError, match="int64"):
        bf.GemmI8(1, 4, 8, 64, q, s, torch.zeros(1, 8, 64, dtype=torch.int8), torch.zeros(1, 8),
                  offsets=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="bfloat16"):
        bf.GemmI8Dw(1, 4, 8, 64, q, s, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="GPU"):
        bf.GemmI8Dx(1, 4, 8, 64, torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(1, 8, 64, dtype=torch.int8),
                    torch.zeros(1, 8))
    with pytest.raises(ValueError, match="4 or 8"):
        from computation_collective_amd import moe_layer
        moe_layer.MoeDecode(1, 4, 2, x, None, None, 64, 64, bits=2)


def test_sums_in_parts_need_their_workspace():
    """dw of few tiles and many rows takes its sums in parts through the workspace: none, or one byte too few, is refused."""
    T, N, K = 9000, 64, 128
    need = hocf.hocf_gemm_i8_dw_workspace_bytes(2, T, N, K)
    assert need == 4 * 2 * N * K * 4
    for s in (sync(ws=0, nbytes=0), sync(ws=0, nbytes=need), sync(nbytes=need - 1)):
        assert call("gemm_i8_dw", T=T, s=s) == INVALID
    valid(call("gemm_i8_dw", T=T, s=sync(nbytes=need)))
