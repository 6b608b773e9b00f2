"""The 8-bit integer operators on the GPU against plain 64-bit implementations
(i8_ref.py), at the sizes, groups and values where they can go wrong.

Codes and scales are equal.  Computed values: half a step of the output's type
relative to the value, plus a stated number of binary32 half steps (2^-24)
relative to the sum of the magnitudes that the value is a sum of.  Outputs are
poisoned first, so an element that is not written shows."""

import numpy as np
import pytest
import torch

import i8_ref as ref
from computation_collective_amd import buffers as bf
from computation_collective_amd import hocf
from computation_collective_amd import moe_layer
from test_gpu_moe import HALF, host, near, run, say

pytestmark = pytest.mark.gpu
F32, BF16, NONE, SILU = hocf.HOCF_F32, hocf.HOCF_BF16, hocf.HOCF_ACT_NONE, hocf.HOCF_ACT_SILU
TORCH = {F32: torch.float32, BF16: torch.bfloat16}
BAD_INDEX = hocf.HOCF_ERR_BAD_INDEX


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def rng(seed):
    return np.random.default_rng(seed)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def same(t, want):
    got = t.cpu().numpy()
    assert np.array_equal(got, want, equal_nan=got.dtype.kind == "f"), np.argwhere(got != want)[:5]


# ------------------------------------------------------------------------------ rows to codes

def rows_of(T, K, dt, seed, ld=None):
    """Normal rows of very different sizes on the device, rows ld apart with NaN between; and themselves in 64 bits."""
    g = rng(seed)
    a = np.full((T, ld or K), np.nan, np.float32)
    a[:, :K] = g.standard_normal((T, K)) * 10.0 ** g.uniform(-3, 3, (T, 1))
    x = dev(a, TORCH[dt])[:, :K]
    return x, host(x)


def check_quant(x, want, **kw):
    h = bf.QuantI8(*x.shape, x, **kw)
    for again in range(2):
        run(h)
        q, s = ref.quant(want)
        same(h.scales, s)
        same(h.codes, q)
    return h


@pytest.mark.parametrize("T,K,ld", [(1, 16, 16), (3, 48, 56), (5, 1040, 1040), (2, 2048, 2064), (7, 2064, 2064), (4, 4096, 4096),
                                    (3, 4112, 4120), (2, 8192, 8192), (3, 8208, 8208), (2, 65536, 65536),
                                    (2050, 16, 24), (2049, 1024, 1024), (2100, 1040, 1040), (2048, 1792, 1792), (2049, 2064, 2072),
                                    (2051, 4096, 4096)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_quant_sizes(T, K, ld, dt):
    say(f"quant T={T} K={K} ld={ld} dt={dt}")
    check_quant(*rows_of(T, K, dt, T + K, ld))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_quant_halves(dt):
    """x = m / 2 of a scale that is 1, a power of two or inexact: exact halves and their neighbours in the type."""
    say(f"quant halves dt={dt}")
    m = np.arange(-254, 255) / 2.0
    rows = []
    for top in (127.0, 127.0 * 2 ** 20, 127.0 * 2 ** -60, 100.0, 3.0, 1.7e-20, 254.0 / 3):
        s = np.float64(np.float32(top) / np.float32(127))
        near_half = (m * s).astype(np.float32)
        for v in (near_half, np.nextafter(near_half, np.float32(np.inf)), np.nextafter(near_half, np.float32(-np.inf))):
            rows.append(np.concatenate([np.clip(v, -top, top), [top, -top, 0.0]]))
    x = dev(np.array(rows, np.float32), TORCH[dt])
    check_quant(x, host(x))


@pytest.mark.parametrize("T", [40, 2050])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_quant_odd_values(T, dt):
    """Zeros, subnormal rows, the largest numbers, and rows that are not finite, one of each kind."""
    say(f"quant odd values T={T} dt={dt}")
    a = rng(1).standard_normal((T, 64)).astype(np.float32)
    a[0] = 0.0
    a[1] = -0.0
    a[2] = 2.0 ** -133
    a[3] = np.float32(2.0 ** -126) * np.linspace(-200, 200, 64)
    a[4] = np.linspace(-3.38e38, 3.38e38, 64)
    a[5, 63] = np.inf
    a[6, 0] = -np.inf
    a[7, 31] = np.nan
    a[8, :] = np.nan
    a[9, 5] = 1e30                                    # all others round to 0
    a[T - 1] = 1.0
    x = dev(a, TORCH[dt])
    h = check_quant(x, host(x))
    assert np.isnan(h.scales[5:9].cpu().numpy()).all()
    # and what they stand for
    d = run_dequant(h.codes, h.scales, dt)
    assert np.isnan(d[5:9]).all() and not d[0].any()


def run_dequant(q, s, dt):
    h = bf.DequantI8(*q.shape, q, s, out_dt=dt)
    h.poison()
    h.run()
    torch.cuda.synchronize()
    return host(h.out)


def silu_bounds(x, dt):
    """SiLU rounded to the type, from values 2^-20 of themselves below and above (bf16; fp32: the rounded value)."""
    a = ref.silu(x)
    if dt == F32:
        a = a.astype(np.float32).astype(np.float64)
        return a, a
    return ref.to_bf16(a * (1 - 2.0 ** -20)), ref.to_bf16(a * (1 + 2.0 ** -20))


@pytest.mark.parametrize("T,K", [(1, 16), (5, 1040), (3, 2064), (3, 8192), (2, 8208), (2049, 1024), (2100, 1792), (2048, 4096)])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("keep", [False, True])
def test_quant_silu(T, K, dt, keep):
    say(f"quant silu T={T} K={K} dt={dt} keep={keep}")
    g = rng(K)
    x = dev((4 * g.standard_normal((T, K))).astype(np.float32), TORCH[dt])
    h = run(bf.QuantI8(T, K, x, act=SILU, keep=keep))
    lo, hi = silu_bounds(host(x), dt)
    # a row whose largest magnitude is certain has a certain scale, and each code lies between those of the bounds
    sure = np.abs(lo).max(1) == np.abs(hi).max(1)
    assert sure.mean() > 0.9
    (ql, sl), (qh, sh) = ref.quant(lo), ref.quant(hi)
    q, s = h.codes.cpu().numpy(), h.scales.cpu().numpy()
    assert np.array_equal(s[sure], sl[sure]) and ((s == sl) | (s == sh)).all()
    assert ((q >= np.minimum(ql, qh)) & (q <= np.maximum(ql, qh)))[sure].all()
    assert (ql == qh)[sure].mean() > 0.99
    if keep:
        q, s = ref.quant(host(x))
        same(h.pre_codes, q)
        same(h.pre_scales, s)


@pytest.mark.parametrize("T,K", [(2049, 16), (2051, 256), (2055, 592), (2049, 768), (2053, 1040), (16385, 1040),
                                 (16389, 1792)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_quant_halves_of_waves(T, K, dt):
    """Odd numbers of rows at lengths where two rows share a wave, each row of its own scale, some not finite."""
    say(f"quant halves of waves T={T} K={K} dt={dt}")
    g = rng(T + K)
    x = g.standard_normal((T, K)).astype(np.float32) * np.exp2(g.integers(-20, 20, (T, 1))).astype(np.float32)
    x[5, 3], x[8, K - 1], x[T - 1, 0], x[10] = np.nan, np.inf, -np.inf, 0
    x = dev(x, TORCH[dt])
    h = run(bf.QuantI8(T, K, x))
    q, s = ref.quant(host(x))
    same(h.codes, q)
    same(h.scales, s)
    h = run(bf.QuantI8(T, K, x, act=SILU, keep=True))
    same(h.pre_codes, q)
    same(h.pre_scales, s)


def test_silu_far():
    """SiLU far from zero: rows that fp32's exponential alone would lose or overflow."""
    say("silu far")
    x = np.zeros((8, 16), np.float32)
    x[0] = np.linspace(-95, -80, 16)
    x[1] = np.linspace(-88, -60, 16)
    x[2] = np.linspace(-1e4, 1e4, 16)
    x[3] = np.linspace(60, 130, 16)
    x[4] = -1e38
    x[5] = np.linspace(-3e38, 3e38, 16)
    x[6] = np.linspace(-1e-30, 1e-30, 16)
    x[7, 3] = -np.inf
    for dt in (F32, BF16):
        t = dev(x, TORCH[dt])
        h = run(bf.QuantI8(8, 16, t, act=SILU))
        with np.errstate(invalid="ignore"):
            lo, hi = silu_bounds(host(t), dt)
        for r in range(7):
            (ql, sl), (qh, sh) = ref.quant(lo[r:r + 1]), ref.quant(hi[r:r + 1])
            s, q = h.scales[r].item(), h.codes[r].cpu().numpy()
            assert min(sl, sh) <= s <= max(sl, sh), r
            # (a scale one step off moves a code's border by 2^-8 of it: one code at most)
            assert (np.abs(q.astype(int) - ql[0]) <= (0 if sl == sh else 1) + (ql != qh)[0]).all(), r
        assert np.isnan(h.scales[7].item()) and not h.codes[7].any()   # -inf / inf


@pytest.mark.parametrize("T,K", [(1, 16), (3, 48), (70, 1040), (1000, 64), (33, 4096), (2, 65536)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_dequant(T, K, dt):
    say(f"dequant T={T} K={K} dt={dt}")
    g = rng(T)
    q = g.integers(-128, 128, (T, K)).astype(np.int8)
    s = (10.0 ** g.uniform(-30, 30, T)).astype(np.float32)
    got = run_dequant(dev(q), dev(s), dt)
    want = (q * s[:, None]).astype(np.float32).astype(np.float64)
    assert np.array_equal(got, want if dt == F32 else ref.to_bf16(want))


@pytest.mark.parametrize("E,K,N", [(1, 16, 8), (2, 48, 64), (3, 1040, 1000), (1, 256, 72), (2, 272, 136), (1, 65536, 8),
                                   (1, 16, 65536), (5, 400, 200), (5, 400, 1032), (161, 1040, 24), (40, 1552, 136),
                                   (170, 2064, 8), (5, 4096, 1032), (4, 4112, 1288)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_weights(E, K, N, dt):
    say(f"weights E={E} K={K} N={N} dt={dt}")
    g = rng(E + K)
    w = dev((g.standard_normal((E, K, N)) * 10.0 ** g.uniform(-2, 2, (E, 1, N))).astype(np.float32), TORCH[dt])
    w[0, :, 1] = 0
    w[-1, K - 1, 2] = float("nan")
    w[-1, 0, 3] = float("inf")
    h = bf.WeightsI8(E, N, K, w)
    for again in range(2):
        run(h)
        q, s = ref.quant(host(w).transpose(0, 2, 1))
        same(h.scales, s)
        same(h.wq, q)


# ------------------------------------------------------------------------------ products

def codes(shape, seed, full=False):
    g = rng(seed)
    if full:
        return np.where(g.random(shape) < 0.5, 127, -128).astype(np.int8)
    return np.clip(np.round(32 * g.standard_normal(shape)), -127, 127).astype(np.int8)


def scales(shape, seed):
    return (10.0 ** rng(seed).uniform(-4, 0, shape)).astype(np.float32)


def gemm_case(E, T, N, K, out_dt, offsets=None, full=False, seed=0):
    xq, wq = codes((T, K), seed + 1, full), codes((E, N, K), seed + 2, full)
    xs, ws = scales(T, seed + 3), scales((E, N), seed + 4)
    off = None if offsets is None else dev(np.array(offsets, np.int64))
    h = run(bf.GemmI8(E, T, N, K, dev(xq), dev(xs), dev(wq), dev(ws), offsets=off, out_dt=out_dt))
    return h, ref.gemm(xq, xs, wq, ws, offsets)


def check_rows(got, want, size, dtype, steps):
    """near() where a group has the row; the others as they were poisoned."""
    got, out = host(got), np.isnan(want).all(1)
    assert np.isnan(got[out]).all(), "rows of no group"
    near(torch.from_numpy(got[~out]), want[~out], size[~out], dtype, steps)


# (the rounding of the sum, and of its products with the two scales)
GEMM_STEPS = 3


@pytest.mark.parametrize("T,N,K", [(1, 8, 16), (2, 8, 144), (63, 72, 128), (64, 64, 256), (65, 1000, 1040), (201, 1000, 272),
                                   (1030, 2056, 384), (1024, 2048, 512), (4100, 2056, 400), (300, 65536, 64), (8200, 1032, 128)])
@pytest.mark.parametrize("out_dt", [F32, BF16])
def test_gemm_sizes(T, N, K, out_dt):
    say(f"gemm T={T} N={N} K={K} out={out_dt}")
    h, want = gemm_case(1, T, N, K, out_dt)
    check_rows(h.out, want, np.abs(want), TORCH[out_dt], GEMM_STEPS)


def test_gemm_largest_sums():
    """Sums of 65536 products of the largest codes fit 32 bits, of either sign."""
    say("gemm largest sums")
    T, N, K = 70, 72, 65536
    for fill in ((-128, -128), (127, -128), (127, 127)):
        xq, wq = np.full((T, K), fill[0], np.int8), np.full((1, N, K), fill[1], np.int8)
        one = np.ones(T, np.float32), np.ones((1, N), np.float32)
        h = run(bf.GemmI8(1, T, N, K, dev(xq), dev(one[0]), dev(wq), dev(one[1]), out_dt=F32))
        assert (host(h.out) == fill[0] * fill[1] * K).all()
        v = run(bf.GemvI8(T, 1, 1, 0, N, K, dev(xq), dev(one[0]), None, dev(wq), dev(one[1]), out_dt=F32))
        assert torch.equal(v.out, h.out)
    h, want = gemm_case(1, T, N, 1024, F32, full=True)
    check_rows(h.out, want, np.abs(want), torch.float32, GEMM_STEPS)


GROUPS = [
    (2, 100, [0, 37, 100]), (4, 300, [0, 0, 131, 131, 300]), (3, 50, [7, 7, 20, 41]), (1, 90, [10, 71]),
    (3, 40, [0, 0, 0, 0]), (2, 64, [64, 64, 64]), (5, 1300, [0, 256, 512, 513, 1027, 1300]),
    (70, 400, list(range(0, 355, 5))), (130, 200, [min(200, 3 * i // 2) for i in range(131)]),
    (1024, 1100, [min(i, 1100) for i in range(1025)]),
]


@pytest.mark.parametrize("E,T,offsets", GROUPS)
@pytest.mark.parametrize("out_dt", [F32, BF16])
def test_gemm_groups(E, T, offsets, out_dt):
    say(f"gemm groups E={E} T={T} out={out_dt}")
    h, want = gemm_case(E, T, 136, 144, out_dt, offsets)
    check_rows(h.out, want, np.abs(want), TORCH[out_dt], GEMM_STEPS)


@pytest.mark.parametrize("E,T,N,offsets", [(4, 5000, 1800, [3, 1300, 1300, 1301, 4990]), (3, 2400, 1032, [0, 1100, 1237, 2400])])
def test_gemm_groups_large_tiles(E, T, N, offsets):
    say(f"gemm groups E={E} T={T} N={N}")
    h, want = gemm_case(E, T, N, 208, BF16, offsets)
    check_rows(h.out, want, np.abs(want), torch.bfloat16, GEMM_STEPS)


BAD_OFFSETS = [[-5, 40, 90], [0, 70, 50], [0, 40, 120], [1 << 62, -(1 << 62), 90], [0, 50, -1], [200, 300, 400]]


@pytest.mark.parametrize("offsets", BAD_OFFSETS)
def test_bad_offsets_are_reported(offsets):
    """Offsets that fall or leave the rows: reported, and nothing outside the outputs is touched."""
    say(f"bad offsets {offsets}")
    E, T, N, K = 2, 90, 72, 64
    off = dev(np.array(offsets, np.int64))
    q, s = dev(codes((T, K), 1)), dev(scales(T, 2))
    wq, ws = dev(codes((E, N, K), 3)), dev(scales((E, N), 4))
    dy = torch.randn(T, N, device="cuda").bfloat16()
    for h in (bf.GemmI8(E, T, N, K, q, s, wq, ws, offsets=off), bf.GemmI8Dx(E, T, N, K, dy, wq, ws, offsets=off),
              bf.GemmI8Dw(E, T, N, K, q, s, dy, offsets=off)):
        h.run()
        torch.cuda.synchronize()
        assert h.status_value() == BAD_INDEX


def test_gemm_scales_that_are_not_finite():
    """A NaN row or channel gives NaN there and nowhere else; an infinite one infinities, and NaN for sums of zero."""
    say("gemm odd scales")
    T, N, K = 70, 72, 64
    xq, wq, xs, ws = codes((T, K), 1), codes((1, N, K), 2), scales(T, 3), scales((1, N), 4)
    xs[[3, 69]] = np.nan
    ws[0, 40] = np.nan
    xs[5] = np.inf
    xq[6], xs[6] = 0, np.inf
    want = None
    with np.errstate(invalid="ignore"):
        want = ref.gemm(xq, xs, wq, ws)
    h = run(bf.GemmI8(1, T, N, K, dev(xq), dev(xs), dev(wq), dev(ws), out_dt=F32))
    got = host(h.out)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
    fine = np.isfinite(want)
    assert (np.abs(got - want)[fine] <= 2.0 ** -22 * np.abs(want[fine])).all()
    v = run(bf.GemvI8(T, 1, 1, 0, N, K, dev(xq), dev(xs), None, dev(wq), dev(ws), out_dt=F32))
    assert np.array_equal(host(v.out), got, equal_nan=True)


# ------------------------------------------------------------------------------ a few rows

@pytest.mark.parametrize("R,rows_per_x,E,e0,N,K", [
    (1, 1, 1, 0, 8, 16), (5, 1, 1, 0, 1000, 1040), (16, 1, 1, 0, 72, 128), (17, 1, 1, 0, 24, 4096), (64, 1, 1, 0, 136, 2064),
    (8, 8, 64, 0, 72, 1792), (6, 2, 8, 4, 40, 144), (32, 2, 4, 0, 1000, 528), (200, 1, 3, 1, 72, 272),
    (1024, 4, 7, 0, 24, 64), (40, 1, 1, 0, 8, 65536)])
@pytest.mark.parametrize("out_dt", [F32, BF16])
def test_gemv(R, rows_per_x, E, e0, N, K, out_dt):
    say(f"gemv R={R} rows_per_x={rows_per_x} E={E} e0={e0} N={N} K={K} out={out_dt}")
    rows = R // rows_per_x
    xq, wq, xs, ws = codes((rows, K), 1), codes((E, N, K), 2), scales(rows, 3), scales((E, N), 4)
    e = None
    if E > 1:
        e = rng(5).integers(e0 - 1, e0 + E + 1, R).astype(np.int32)     # some of other ranks
        e[R // 2] = -1
        if R > 4:
            e[3] = -(1 << 31)
    h = run(bf.GemvI8(R, rows_per_x, E, e0, N, K, dev(xq), dev(xs), None if e is None else dev(e), dev(wq), dev(ws),
                      out_dt=out_dt))
    want = np.zeros((R, N))
    for r in range(R):
        at = 0 if e is None else int(e[r]) - e0
        if 0 <= at < E:
            i = r // rows_per_x
            want[r] = ref.gemm(xq[i:i + 1], xs[i:i + 1], wq[at:at + 1], ws[at:at + 1])[0]
    near(h.out, want, np.abs(want), TORCH[out_dt], GEMM_STEPS)


def test_gemv_gives_the_bits_of_gemm():
    say("gemv and gemm")
    R, N, K, E = 48, 200, 1040, 3
    xq, wq, xs, ws = dev(codes((R, K), 1)), dev(codes((E, N, K), 2)), dev(scales(R, 3)), dev(scales((E, N), 4))
    e = torch.arange(R, dtype=torch.int32, device="cuda") * E // R
    off = torch.tensor([0, 16, 32, 48], device="cuda")
    a = run(bf.GemvI8(R, 1, E, 0, N, K, xq, xs, e, wq, ws, out_dt=F32))
    b = run(bf.GemmI8(E, R, N, K, xq, xs, wq, ws, offsets=off, out_dt=F32))
    assert torch.equal(a.out, b.out)


# ------------------------------------------------------------------------------ gradients

def dx_case(E, T, N, K, out_dt, offsets=None, silu=False):
    dy = dev(rng(1).standard_normal((T, N)).astype(np.float32), torch.bfloat16)
    wq, ws = codes((E, N, K), 2), scales((E, N), 3)
    pre = (codes((T, K), 4), (scales(T, 5) * 0.5).astype(np.float32)) if silu else None
    off = None if offsets is None else dev(np.array(offsets, np.int64))
    kw = dict(pre_codes=dev(pre[0]), pre_scales=dev(pre[1])) if silu else {}
    h = run(bf.GemmI8Dx(E, T, N, K, dy, dev(wq), dev(ws), offsets=off, out_dt=out_dt, **kw))
    return (h, *ref.dx(host(dy), wq, ws, offsets, pre))


@pytest.mark.parametrize("T,N,K", [(1, 8, 16), (3, 72, 48), (64, 64, 64), (65, 136, 80), (333, 1000, 1040), (130, 8, 2064),
                                   (1030, 264, 2048), (4100, 128, 2064), (8200, 72, 1040), (200, 4096, 208)])
@pytest.mark.parametrize("out_dt", [F32, BF16])
def test_dx_sizes(T, N, K, out_dt):
    say(f"dx T={T} N={N} K={K} out={out_dt}")
    h, want, size = dx_case(1, T, N, K, out_dt)
    check_rows(h.out, want, size, TORCH[out_dt], N)


@pytest.mark.parametrize("E,T,offsets", GROUPS)
def test_dx_groups(E, T, offsets):
    say(f"dx groups E={E} T={T}")
    h, want, size = dx_case(E, T, 72, 80, F32, offsets)
    check_rows(h.out, want, size, torch.float32, 72)


@pytest.mark.parametrize("E,T,N,K,offsets", [(1, 5, 16, 16, None), (1, 333, 136, 1040, None), (1, 4200, 72, 2064, None),
                                             (1, 8200, 72, 1040, None), (3, 700, 64, 208, [5, 300, 300, 690]),
                                             (4, 5000, 72, 1808, [3, 1300, 1300, 1301, 4990])])
@pytest.mark.parametrize("out_dt", [F32, BF16])
def test_dx_through_silu(E, T, N, K, offsets, out_dt):
    say(f"dx through silu E={E} T={T} N={N} K={K} out={out_dt}")
    plain = dx_case(E, T, N, K, out_dt, offsets)
    h, want, _ = dx_case(E, T, N, K, out_dt, offsets, silu=True)
    # |slope| and the sizes that its rounding errors are relative to: p (1 + |h| (1 - p)), and h's 64 half steps of exp's argument
    pre = ref.held(codes((T, K), 4), (scales(T, 5) * 0.5).astype(np.float32))
    assert np.abs(pre).max() < 64
    p = 1 / (1 + np.exp(-pre))
    size = plain[2] * p * (1 + np.abs(pre))
    check_rows(h.out, want, size, TORCH[out_dt], N + 64 + 16)


@pytest.mark.parametrize("T,N,K", [(0, 8, 16), (1, 8, 16), (2, 72, 48), (63, 64, 64), (64, 64, 64), (65, 136, 80), (129, 264, 144),
                                   (501, 1000, 1040), (200, 2056, 2064), (96, 4096, 4096), (2000, 72, 80)])
@pytest.mark.parametrize("out_dt", [F32, BF16])
def test_dw_sizes(T, N, K, out_dt):
    say(f"dw T={T} N={N} K={K} out={out_dt}")
    check_dw(1, T, N, K, out_dt)


def check_dw(E, T, N, K, out_dt, offsets=None):
    xq, xs = codes((T, K), 1), scales(T, 2)
    dy = dev(rng(3).standard_normal((T, N)).astype(np.float32), torch.bfloat16)
    clean = host(dy)
    if offsets is not None:                            # what no group has must not matter
        outside = np.ones(T, bool)
        outside[offsets[0]:offsets[-1]] = False
        xs[outside] = np.nan
        dy[dev(outside)] = float("nan")
    off = None if offsets is None else dev(np.array(offsets, np.int64))
    h = run(bf.GemmI8Dw(E, T, N, K, dev(xq), dev(xs), dy, offsets=off, out_dt=out_dt))
    want, size = ref.dw(xq, xs, clean, E, offsets)
    near(h.out, want, size, TORCH[out_dt], max(1, T))
    return h


@pytest.mark.parametrize("E,T,offsets", GROUPS)
@pytest.mark.parametrize("out_dt", [F32, BF16])
def test_dw_groups(E, T, offsets, out_dt):
    say(f"dw groups E={E} T={T} out={out_dt}")
    check_dw(E, T, 72, 80, out_dt, offsets)


def test_dw_sums_in_parts():
    """Few tiles and many rows: the sums go through the workspace in parts, groups of very different lengths too."""
    say("dw, sums in parts")
    assert hocf.hocf_gemm_i8_dw_workspace_bytes(1, 5000, 72, 80) == 4 * 72 * 80 * 4
    assert hocf.hocf_gemm_i8_dw_workspace_bytes(1, 2000, 72, 80) == 0
    check_dw(1, 5000, 72, 80, F32)
    check_dw(1, 4097, 264, 272, BF16)
    check_dw(2, 9000, 136, 80, F32, [10, 20, 8990])       # one group shorter than a step of each part
    check_dw(3, 7000, 72, 144, BF16, [0, 0, 6999, 7000])


def test_dw_groups_large_tiles():
    say("dw groups, large tiles")
    check_dw(3, 500, 2056, 2064, F32, [3, 130, 130, 480])
    check_dw(2, 300, 1032, 1040, BF16, [0, 299, 300])


def test_gradients_keep_rows_apart():
    """NaN and infinities of one row or group stay in what depends on it."""
    say("gradients apart")
    E, T, N, K, offsets = 2, 140, 72, 80, [0, 67, 140]
    off = dev(np.array(offsets, np.int64))
    xq, xs, wq, ws = codes((T, K), 1), scales(T, 2), codes((E, N, K), 3), scales((E, N), 4)
    dy = rng(5).standard_normal((T, N)).astype(np.float32)
    base_x = run(bf.GemmI8Dx(E, T, N, K, dev(dy, torch.bfloat16), dev(wq), dev(ws), offsets=off, out_dt=F32)).out.clone()
    base_w = run(bf.GemmI8Dw(E, T, N, K, dev(xq), dev(xs), dev(dy, torch.bfloat16), offsets=off)).out.clone()
    dy[66, 5], dy[70, 7] = np.nan, np.inf              # the last row of group 0, a row of group 1
    d = dev(dy, torch.bfloat16)
    gx = bf.GemmI8Dx(E, T, N, K, d, dev(wq), dev(ws), offsets=off, out_dt=F32)
    gw = bf.GemmI8Dw(E, T, N, K, dev(xq), dev(xs), d, offsets=off)
    gx.run(), gw.run()
    torch.cuda.synchronize()
    rows = torch.arange(T, device="cuda")
    rest = (rows != 66) & (rows != 70)
    assert torch.equal(gx.out[rest], base_x[rest]) and gx.out[66].isnan().all() and not gx.out[70].isfinite().any()
    cols = torch.arange(N, device="cuda")
    assert gw.out[0][:, 5].isnan().all() and torch.equal(gw.out[0][:, cols != 5], base_w[0][:, cols != 5])
    assert not gw.out[1][:, 7].isfinite().any() and torch.equal(gw.out[1][:, cols != 7], base_w[1][:, cols != 7])


def test_gradient_against_differences():
    """dw and dx of the loss sum(G . out) with the product itself: codes moved by one, exactly linear."""
    say("gradient against differences")
    T, N, K = 6, 8, 16
    xq, wq = codes((T, K), 1), codes((1, N, K), 2)
    xs, ws = np.full(T, 2.0 ** -5, np.float32), np.full((1, N), 2.0 ** -6, np.float32)   # (held numbers are exact)
    G = ref.to_bf16(rng(3).standard_normal((T, N)))
    loss = lambda x, w: (G * host(run(bf.GemmI8(1, T, N, K, dev(x), dev(xs), dev(w), dev(ws), out_dt=F32)).out)).sum()
    dx = host(run(bf.GemmI8Dx(1, T, N, K, dev(G, torch.bfloat16), dev(wq), dev(ws), out_dt=F32)).out)
    dw = host(run(bf.GemmI8Dw(1, T, N, K, dev(xq), dev(xs), dev(G, torch.bfloat16))).out)[0]
    here = loss(xq, wq)
    for r, k in ((0, 0), (5, 15), (3, 7)):
        x = xq.copy()
        x[r, k] += 1
        assert abs((loss(x, wq) - here) / 2.0 ** -5 - dx[r, k]) < 1e-4
    for n, k in ((0, 0), (7, 15), (4, 9)):
        w = wq.copy()
        w[0, n, k] += 1
        assert abs((loss(xq, w) - here) / 2.0 ** -6 - dw[k, n]) < 1e-4


# ------------------------------------------------------------------------------ together

def plain_experts(x, w_up, w_down, dy, offsets):
    """y, dx, dw_up, dw_down of silu(x w_up) w_down with autograd in 64 bits on the CPU (no codes)."""
    x, w_up, w_down = (t.double().cpu().requires_grad_() for t in (x, w_up, w_down))
    y = torch.zeros_like(x)
    parts = [torch.nn.functional.silu(x[a:b] @ w_up[e]) @ w_down[e]
             for e, (a, b) in enumerate(zip(offsets[:-1], offsets[1:]))]
    y = torch.cat([torch.zeros(offsets[0], x.shape[1]).double()] + parts + [torch.zeros(len(x) - offsets[-1], x.shape[1]).double()])
    y.backward(dy.double().cpu())
    return y.detach(), x.grad, w_up.grad, w_down.grad


def normal(shape, seed, std=1.0):
    return (std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).bfloat16().cuda()


@pytest.mark.parametrize("E,rows,K,H,offsets", [(2, 300, 256, 384, [0, 130, 300]), (4, 500, 192, 144, [0, 100, 100, 407, 480])])
def test_experts_layer(E, rows, K, H, offsets):
    """The layer against its stages' references, and near the layer without codes."""
    say(f"experts layer E={E} rows={rows}")
    w_up, w_down = normal((E, K, H), 1, K ** -0.5), normal((E, H, K), 2, H ** -0.5)
    layer = moe_layer.ExpertsI8(E, rows, w_up, w_down)
    off = torch.tensor(offsets, device="cuda")
    x, dy = normal((rows, K), 3), normal((rows, K), 4)
    for again in range(2):
        y = layer.forward(x, off)
        dx, dw_up, dw_down = layer.backward(dy)
        layer.check()
    # every stage from the stage before it
    q = lambda h: (h.codes.cpu().numpy(), h.scales.cpu().numpy())
    up, down = ((w.wq.cpu().numpy(), w.scales.cpu().numpy()) for w in (layer.w_up, layer.w_down))
    assert all(np.array_equal(a, b) for a, b in zip(up, ref.quant(host(w_up).transpose(0, 2, 1))))
    xq = ref.quant(host(x))
    assert all(np.array_equal(a, b) for a, b in zip(q(layer.x_codes), xq))
    zero = lambda v: np.nan_to_num(v)                  # rows of no group hold zeros here
    h = zero(ref.gemm(*xq, *up, offsets))
    near(layer.up.out, h, np.abs(h), torch.bfloat16, GEMM_STEPS)
    pre = ref.quant(host(layer.up.out))
    same(layer.h_codes.pre_codes, pre[0])
    want = zero(ref.gemm(*q(layer.h_codes), *down, offsets))
    near(y, want, np.abs(want), torch.bfloat16, GEMM_STEPS)
    want, size = ref.dw(*q(layer.h_codes), host(dy), E, offsets)
    near(dw_down, want, size, torch.float32, rows)
    want, _ = ref.dx(host(dy), *down, offsets, pre)
    _, size = ref.dx(host(dy), *down, offsets)
    hh = np.abs(ref.held(*pre))
    near(layer.dh.out, zero(want), zero(size) * (1 + hh), torch.bfloat16, K + 64 + 16)
    want, size = ref.dw(*xq, host(layer.dh.out), E, offsets)
    near(dw_up, want, size, torch.float32, rows)
    want, size = ref.dx(host(layer.dh.out), *up, offsets)
    near(dx, zero(want), zero(size), torch.bfloat16, H)
    # The codes' rounding: a code is off by at most half a scale, 1/254 of its row's largest, 2^-8 bf16 steps on
    # top; normal rows of 144 to 384 have their largest within 4.5 deviations, so a factor's relative error is below
    # 4.5 / 254 / sqrt(3) + 2^-9 = 1.3 % rms, and a chain of at most six of them below 6 x 1.3 % even if all add up.
    for got, want in zip((y, dx, dw_up, dw_down), plain_experts(x, w_up, w_down, dy, offsets)):
        got, want = host(got), want.numpy()
        assert np.linalg.norm(got - want) < 0.08 * np.linalg.norm(want)


def test_experts_layer_follows_its_weights():
    """requantise() takes the weights' codes anew; without it the old ones stay."""
    say("experts layer weights")
    w_up, w_down = normal((1, 64, 64), 1, 0.1), normal((1, 64, 64), 2, 0.1)
    layer = moe_layer.ExpertsI8(1, 32, w_up, w_down)
    x, off = normal((32, 64), 3), torch.tensor([0, 32], device="cuda")
    first = layer.forward(x, off).clone()
    w_down.mul_(2)
    assert torch.equal(layer.forward(x, off), first)
    layer.requantise()
    assert torch.equal(layer.forward(x, off), first * 2)
    with pytest.raises(RuntimeError, match="experts"):
        layer.forward(x, torch.tensor([0, 99], device="cuda"))
        layer.check()
    layer.forward(x, off)
    layer.check()


@pytest.mark.parametrize("T,E,topk", [(1, 16, 4), (4, 8, 2), (16, 32, 2)])
def test_decode_in_8_bits(T, E, topk):
    say(f"decode in 8 bits T={T} E={E}")
    K, H = 256, 192
    up, down = (bf.WeightsI8(E, n, k, normal((E, k, n), 10 + k, k ** -0.5)) for k, n in ((K, H), (H, K)))
    up.run(), down.run()
    d = moe_layer.MoeDecode(T, E, topk, normal((K, E), 3, 0.06), (up.wq, up.scales), (down.wq, down.scales), K, H, bits=8)
    x = normal((T, K), 4)
    out = d.step(x)
    torch.cuda.synchronize()
    xq, xs = ref.quant(host(x))
    e = d.route.experts.cpu().numpy()
    (uq, us), (dq, ds) = ((w.wq.cpu().numpy(), w.scales.cpu().numpy()) for w in (up, down))
    for t in range(T):
        for j in range(topk):
            k = e[t, j]
            want = ref.gemm(xq[t:t + 1], xs[t:t + 1], uq[k:k + 1], us[k:k + 1])
            near(d.hidden[t * topk + j], want[0], np.abs(want[0]), torch.bfloat16, GEMM_STEPS)
            hq, hs = (a[t * topk + j:t * topk + j + 1].cpu().numpy() for a in (d.h_codes.codes, d.h_codes.scales))
            want = ref.gemm(hq, hs, dq[k:k + 1], ds[k:k + 1])
            near(d.down.out[t * topk + j], want[0], np.abs(want[0]), torch.bfloat16, GEMM_STEPS)
    rows, w = host(d.down.out).reshape(T, topk, K), d.route.weights.cpu().numpy()
    want = (rows * w[:, :, None]).sum(1) + host(x)
    near(out, want, (np.abs(rows) * w[:, :, None]).sum(1) + np.abs(host(x)), torch.bfloat16, topk + 1)


def test_command(capsys):
    moe_layer.main(["--ranks", "1", "--tokens", "64", "--steps", "1"])
    assert "8-bit integers" in capsys.readouterr().out


# ------------------------------------------------------------------------------ streams and graphs

def test_layer_in_a_graph():
    """Forward and backward in one captured graph, replayed with eager work and other inputs in between."""
    say("experts layer in a graph")
    E, rows, K, H, offsets = 3, 400, 256, 144, [0, 150, 150, 390]
    layer = moe_layer.ExpertsI8(E, rows, normal((E, K, H), 1, 0.06), normal((E, H, K), 2, 0.08))
    eager = moe_layer.ExpertsI8(E, rows, layer.w_up.w, layer.w_down.w)
    off, dy = torch.tensor(offsets, device="cuda"), normal((rows, K), 9)
    layer.forward(normal((rows, K), 3), off)
    layer.backward(dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.experts()
        dx, dw_up, dw_down = layer.backward(dy)
    for i in range(4):
        x = normal((rows, K), 20 + i)
        layer.x.copy_(x)
        if i == 2:
            off = torch.tensor([5, 5, 300, 301], device="cuda")
            layer.offsets.copy_(off)
            for h in (layer, eager):
                for g in (h.up, h.down, h.dh, h.dx):
                    g.out.zero_()
        graph.replay()
        want = eager.forward(x, off), *eager.backward(dy)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, dw_up, dw_down), want)), i
    layer.check()


def test_weights_in_a_graph():
    say("weights in a graph")
    w = normal((2, 528, 200), 1)
    h, eager = bf.WeightsI8(2, 200, 528, w), bf.WeightsI8(2, 200, 528, w)
    run(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.run()
    for i in range(4):
        w.copy_(normal((2, 528, 200), 5 + i, 10.0 ** -i))
        graph.replay()
        run(eager)
        assert torch.equal(h.wq, eager.wq) and torch.equal(h.scales, eager.scales)


def test_two_streams_at_once():
    """Two layers at work on two streams: each has its own buffers, and neither disturbs the other."""
    say("two streams")
    off = torch.tensor([0, 700, 2000], device="cuda")
    layers = [moe_layer.ExpertsI8(2, 2000, normal((2, 512, 528), i, 0.05), normal((2, 528, 512), 9 + i, 0.05)) for i in range(2)]
    xs, dys = [normal((2000, 512), 20 + i) for i in range(2)], [normal((2000, 512), 30 + i) for i in range(2)]
    want = []
    for layer, x, dy in zip(layers, xs, dys):
        y = layer.forward(x, off).clone()
        want.append([y] + [t.clone() for t in layer.backward(dy)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for again in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = [layers[i].forward(xs[i], off), *layers[i].backward(dys[i])]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_run_on_a_given_stream():
    say("given stream")
    x, st = normal((100, 64), 1), torch.cuda.Stream()
    a, b = bf.QuantI8(100, 64, x), bf.QuantI8(100, 64, x)
    run(a)
    b.poison()
    st.wait_stream(torch.cuda.current_stream())
    b.run(st)
    st.synchronize()
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


# ------------------------------------------------------------------------------ far into large buffers

def test_far_rows():
    """Rows of codes beyond 2^31 elements: to codes and back, products and gradients."""
    say("far rows")
    T, K, N = 33000, 65536, 8
    assert (T - 2) * K > 2 ** 31
    few = normal((2, K), 1)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    x[-2:] = few
    h, s = run(bf.QuantI8(T, K, x)), run(bf.QuantI8(2, K, few))
    assert torch.equal(h.codes[-2:], s.codes) and torch.equal(h.scales[-2:], s.scales) and not h.codes[:-2].any()
    d = run(bf.DequantI8(T, K, h.codes, h.scales))
    assert torch.equal(d.out[-2:], run(bf.DequantI8(2, K, s.codes, s.scales)).out)
    del d, x
    torch.cuda.empty_cache()
    wq, ws = dev(codes((1, N, K), 2)), dev(scales((1, N), 3))
    off = torch.tensor([T - 2, T], device="cuda")
    far = run(bf.GemmI8(1, T, N, K, h.codes, h.scales, wq, ws, offsets=off))
    near_ = run(bf.GemmI8(1, 2, N, K, s.codes, s.scales, wq, ws))
    assert torch.equal(far.out[-2:], near_.out)
    dy = normal((T, N), 4)
    dw = run(bf.GemmI8Dw(1, T, N, K, h.codes, h.scales, dy, offsets=off)).out
    assert torch.equal(dw, run(bf.GemmI8Dw(1, 2, N, K, s.codes, s.scales, dy[-2:].contiguous())).out)
    dx = run(bf.GemmI8Dx(1, T, N, K, dy, wq, ws, offsets=off, pre_codes=h.codes, pre_scales=h.scales)).out
    want = run(bf.GemmI8Dx(1, 2, N, K, dy[-2:].contiguous(), wq, ws, pre_codes=s.codes, pre_scales=s.scales)).out
    assert torch.equal(dx[-2:], want)


def test_far_experts():
    """Weights' codes beyond 2^32 bytes."""
    say("far experts")
    E, N, K = 300, 4096, 4096
    assert (E - 1) * N * K > 2 ** 32
    wq = torch.zeros((E, N, K), dtype=torch.int8, device="cuda")
    ws = torch.zeros((E, N), dtype=torch.float32, device="cuda")
    wq[-1], ws[-1] = dev(codes((N, K), 1)), dev(scales(N, 2))
    T = 200
    xq, xs, dy = dev(codes((T, K), 3)), dev(scales(T, 4)), normal((T, N), 5)
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    off[-1] = T
    for make in (lambda e, w, s, o: bf.GemmI8(e, T, N, K, xq, xs, w, s, offsets=o), lambda e, w, s, o: bf.GemmI8Dx(e, T, N, K, dy, w, s, offsets=o)):
        assert torch.equal(run(make(E, wq, ws, off)).out, run(make(1, wq[-1:], ws[-1:], None)).out)
    e = torch.full((4,), E - 1, dtype=torch.int32, device="cuda")
    a = run(bf.GemvI8(4, 1, E, 0, N, K, xq[:4], xs[:4], e, wq, ws))
    b = run(bf.GemvI8(4, 1, 1, 0, N, K, xq[:4], xs[:4], None, wq[-1:], ws[-1:]))
    assert torch.equal(a.out, b.out)


def test_many_rows():
    """More workgroups than one dimension of a grid takes here (2^20): rows to codes, back, and their products."""
    say("many rows")
    T, K, N = 280_000_000, 16, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    few = torch.randn((1000, K), generator=g, device="cuda").bfloat16()
    x = torch.zeros((T // 40, K), dtype=torch.bfloat16, device="cuda")      # 7 million rows, four a workgroup
    at = torch.randint(0, len(x), (1000,), generator=g, device="cuda").unique()
    at[-1] = len(x) - 1
    x[at] = few[:len(at)]
    h, want = run(bf.QuantI8(len(x), K, x)), run(bf.QuantI8(len(at), K, few[:len(at)]))
    assert torch.equal(h.codes[at], want.codes) and torch.equal(h.scales[at], want.scales)
    assert int((h.codes != 0).any(1).sum()) <= len(at) and not h.scales.isnan().any()
    q = torch.zeros((T, K), dtype=torch.int8, device="cuda")
    s = torch.ones(T, dtype=torch.float32, device="cuda")
    at = torch.randint(0, T, (1000,), generator=g, device="cuda").unique()
    at[-1] = T - 1
    q[at] = dev(codes((len(at), K), 2))
    d = run(bf.DequantI8(T, K, q, s))
    assert torch.equal(d.out[at], run(bf.DequantI8(len(at), K, q[at], s[at])).out)
    assert int((d.out != 0).any(1).sum()) <= len(at)
    del d
    torch.cuda.empty_cache()
    wq, ws = dev(codes((1, N, K), 3)), dev(scales((1, N), 4))
    h = run(bf.GemmI8(1, T, N, K, q, s, wq, ws))
    assert torch.equal(h.out[at], run(bf.GemmI8(1, len(at), N, K, q[at], s[at], wq, ws)).out)
    assert int((h.out != 0).any(1).sum()) <= len(at)
