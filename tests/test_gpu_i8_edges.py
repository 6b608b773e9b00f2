"""The 8-bit integer operators on the GPU where test_gpu_i8.py does not reach:
every bf16 number through SiLU, SiLU in every form of the kernel, offsets that
fall over three groups and more, SiLU's derivative far from zero, the decode
products' forms of several blocks of columns, and the layer behind a dispatch."""

import numpy as np
import pytest
import torch

import i8_ref as ref
from computation_collective_amd import buffers as bf
from computation_collective_amd import hocf
from computation_collective_amd import moe_layer
from test_gpu_i8 import BAD_INDEX, BF16, F32, GEMM_STEPS, SILU, TORCH, check_rows, codes, dev, normal, plain_experts, rng, same, scales
from test_gpu_moe import host, near, run, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


# ------------------------------------------------------------------------------ SiLU, rounded to bf16

def silu_quant(x):
    """Codes and scales of SiLU in 64 bits, rounded to bf16 once."""
    with np.errstate(invalid="ignore"):
        return ref.quant(ref.to_bf16(ref.silu(x)))


@pytest.mark.parametrize("rows", [65536, 2047])
@pytest.mark.parametrize("keep", [False, True])
def test_silu_of_every_bf16(rows, keep):
    """Each of the 65536 numbers in a row of its own among zeros: the row's scale, 1/127 of its magnitude, tells
    what it was rounded to (from 2^-119 on, where scales are not the smallest one).  All at once, two rows a
    wave, and 2047 at a time, four waves a row."""
    say(f"silu of every bf16 rows={rows} keep={keep}")
    K = 16
    u = np.arange(65536)
    x = np.zeros((65536, K), np.int16)
    x[u, u * 7 % K] = u.astype(np.uint16).view(np.int16)
    x = dev(x).view(torch.bfloat16)
    for r in range(0, 65536, rows):
        part = x[r:r + rows]
        h = run(bf.QuantI8(len(part), K, part, act=SILU, keep=keep))
        q, s = silu_quant(host(part))
        same(h.scales, s)
        same(h.codes, q)


@pytest.mark.parametrize("T,K", [(1, 16), (5, 1040), (3, 2064), (3, 4096), (3, 8192), (2, 8208), (2049, 1024), (2049, 2048), (2048, 4096),
                                 (2049, 16), (2055, 592), (2053, 1040), (16385, 1040), (16389, 1792)])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("keep", [False, True])
def test_silu_codes_are_the_definitions(T, K, dt, keep):
    """Every form of the kernel: codes and scales of SiLU equal, rows of numbers up to 90 and of several sizes."""
    say(f"silu codes T={T} K={K} dt={dt} keep={keep}")
    g = rng(T + K)
    a = g.standard_normal((T, K)) * np.exp2(g.integers(-8, 5, (T, 1)))
    a[:, 0] = g.uniform(-90, 2, T)
    x = dev(a.astype(np.float32), TORCH[dt])
    h = run(bf.QuantI8(T, K, x, act=SILU, keep=keep))
    x = host(x)
    if dt == F32:
        q, s = ref.quant(ref.silu(x).astype(np.float32).astype(np.float64))
    else:
        q, s = silu_quant(x)
    same(h.scales, s)
    same(h.codes, q)
    if keep:
        q, s = ref.quant(x)
        same(h.pre_codes, q)
        same(h.pre_scales, s)


# ------------------------------------------------------------------------------ offsets that fall

def counted(offsets, T):
    """The offsets that the header has in their place: each the largest of itself and those before it, within [0, T]."""
    return np.maximum.accumulate(np.clip(np.array(offsets, object), 0, T)).astype(np.int64).tolist()


class Guarded:
    """A tensor of `shape` inside a larger one, all NaN: what is written beside it shows."""

    def __init__(self, shape, out_dt):
        n, self.guard = int(np.prod(shape)), 8192
        self.all = torch.full((n + 2 * self.guard,), float("nan"), dtype=TORCH[out_dt], device="cuda")
        self.out = self.all[self.guard:self.guard + n].view(shape)

    def intact(self):
        return bool(self.all[:self.guard].isnan().all() and self.all[-self.guard:].isnan().all())


FALLING = [
    (3, 90, 72, 64, [0, 70, 50, 90]), (4, 90, 72, 64, [-5, 40, 200, 30, 90]), (4, 90, 72, 64, [80, 20, 60, 85, 10]),
    (5, 700, 136, 144, [0, 700, 0, 700, 0, 700]), (5, 700, 136, 144, [0, 300, 100, 400, 350, 1 << 40]),
    (130, 400, 72, 80, [min(400, 4 * i) if i % 50 else -i for i in range(131)]),     # falls at the 64-group borders' sides too
    (200, 900, 72, 80, [900 - 5 * i if 64 <= i < 70 else 5 * (i - 1) for i in range(201)]),
    (4, 5000, 1800, 208, [3, 2600, 2500, 4000, 3990]), (3, 2400, 1032, 272, [0, 1100, 1037, 2400]),
    (3, 9000, 136, 80, [10, 6000, 20, 8990]),                                        # (dw's sums in parts)
    (3, 0, 72, 64, [0, 5, -1, 0]), (2, 90, 72, 64, [-(1 << 63), (1 << 63) - 1, -(1 << 63)])]


@pytest.mark.parametrize("E,T,N,K,offsets", FALLING)
@pytest.mark.parametrize("out_dt", [F32, BF16])
def test_offsets_that_fall(E, T, N, K, offsets, out_dt):
    """The products and both gradients as the header has them, each row in one group, nothing beside the outputs
    written, and the same bits again."""
    say(f"offsets that fall E={E} T={T} out={out_dt} {offsets[:6]}")
    c = counted(offsets, T)
    xq, wq, xs, ws = codes((T, K), 1), codes((E, N, K), 2), scales(T, 3), scales((E, N), 4)
    dy = dev(rng(5).standard_normal((T, N)).astype(np.float32), torch.bfloat16)
    off, word = dev(np.array(offsets, np.int64)), torch.zeros(1, dtype=torch.int32, device="cuda")
    d = [dev(a) for a in (xq, xs, wq, ws)]
    size = hocf.hocf_gemm_i8_dw_workspace_bytes(E, T, N, K)
    space = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream()

    def call(entry, shape, *args):
        got = []
        for again in range(2):
            word.zero_()
            g = Guarded(shape, out_dt)
            hocf.check(entry(E, T, N, K, out_dt, *args, off, *(() if entry is not hocf.hocf_gemm_i8_dx else (None, None)), g.out,
                             hocf.sync(1, space, size, status=word), st))
            torch.cuda.synchronize()
            assert g.intact() and (word.item() == BAD_INDEX or (T == 0 and entry is not hocf.hocf_gemm_i8_dw))
            got.append(g.out)
        assert torch.equal(got[0].isnan(), got[1].isnan()) and torch.equal(got[0].nan_to_num(), got[1].nan_to_num())
        return got[0]

    out = call(hocf.hocf_gemm_i8, (T, N), *d)
    if T:
        want = ref.gemm(xq, xs, wq, ws, c)
        check_rows(out, want, np.abs(want), TORCH[out_dt], GEMM_STEPS)
    dx = call(hocf.hocf_gemm_i8_dx, (T, K), dy, d[2], d[3])
    if T:
        want, room = ref.dx(host(dy), wq, ws, c)
        check_rows(dx, want, room, TORCH[out_dt], N)
    dw = call(hocf.hocf_gemm_i8_dw, (E, K, N), d[0], d[1], dy)
    want, room = ref.dw(xq, xs, host(dy), E, c)
    near(dw, want, room, TORCH[out_dt], max(1, T))


# ------------------------------------------------------------------------------ SiLU's derivative

@pytest.mark.parametrize("T,N,K", [(2, 8, 65536), (300, 16, 1024)])
def test_slope_of_every_code(T, N, K):
    """dx through SiLU at h from -300 to 300, beside its roots and signs: within a fixed number of roundings of the
    formula.  With z = exp(-|h|), i = 1 / (1 + z), p is i or z i and 1 - p the other.  Errors in half steps (2^-24):
    z 5 (the instruction 2, its argument's constant 2, a product 1), 1 + z 1, i 2, z i 1: p and 1 - p 9 at most each; 1 + h (1 - p)
    1 more, the slope 1, its product with the sum 1.  In all 21 of |sum| p (1 + |h| (1 - p)).  A z below 2^-126 is zero."""
    say(f"slope T={T} N={N} K={K}")
    g = rng(T)
    dy = dev(g.standard_normal((T, N)).astype(np.float32), torch.bfloat16)
    wq, ws = codes((1, N, K), 2), scales((1, N), 3)
    pre = g.integers(-127, 128, (T, K)).astype(np.int8)
    pre_s = (10.0 ** g.uniform(-4, np.log10(300 / 127), T)).astype(np.float32)
    pre_s[0] = np.float32(1.0)
    h = run(bf.GemmI8Dx(1, T, N, K, dy, dev(wq), dev(ws), pre_codes=dev(pre), pre_scales=dev(pre_s), out_dt=F32))
    want, _ = ref.dx(host(dy), wq, ws, None, (pre, pre_s))
    plain, size = ref.dx(host(dy), wq, ws)
    at = ref.held(pre, pre_s)
    z = np.exp(-np.abs(at))
    p, rest = np.where(at < 0, z, 1) / (1 + z), np.where(at < 0, 1, z) / (1 + z)
    # the sum's own roundings (N of its terms' sizes) meet the slope, whose roots they do not know
    slope = np.abs(ref.silu_slope(at))
    sums = N * size * 2.0 ** -24
    room = sums * slope + 21 * 2.0 ** -24 * (np.abs(plain) + sums) * p * (1 + np.abs(at) * rest)
    room = room * (1 + 2.0 ** -10) + 2.0 ** -126 * (1 + (1 + np.abs(at)) * size)
    got = host(h.out)
    off = np.abs(got - want) - room
    worst = np.unravel_index(np.argmax(off), off.shape)
    assert off[worst] <= 0, (at[worst], got[worst], want[worst], room[worst])
    assert np.isfinite(got).all()


# ------------------------------------------------------------------------------ a few rows, many column blocks

@pytest.mark.parametrize("R,rows_per_x,E,N,K", [
    # two blocks of columns a workgroup (384 to 767 blocks): the last workgroup has one of them, or eight columns
    (1, 1, 1, 6152, 528), (5, 1, 1, 6168, 1040), (8, 8, 64, 888, 2064), (9, 1, 1, 8200, 4080),
    # four blocks (768 and more): one to four of them in the last
    (1, 1, 1, 12296, 48), (20, 1, 1, 16408, 528), (32, 2, 32, 408, 1040), (17, 1, 1, 12312, 2064), (48, 4, 16, 792, 4080),
    (7, 1, 1, 12328, 4096),
    # K beyond what is at once: one block a workgroup, in turns
    (3, 1, 1, 12296, 4112), (40, 2, 8, 1544, 4112)])
@pytest.mark.parametrize("out_dt", [F32, BF16])
def test_gemv_blocks(R, rows_per_x, E, N, K, out_dt):
    """More than 16 rows on one expert too, rows of other ranks' experts, and nothing behind the rows written."""
    say(f"gemv blocks R={R} E={E} N={N} K={K} out={out_dt}")
    rows, e0 = R // rows_per_x, 3 if E > 1 else 0
    xq, wq, xs, ws = codes((rows, K), 1), codes((E, N, K), 2), scales(rows, 3), scales((E, N), 4)
    e = None
    if E > 1:
        e = rng(5).integers(e0, e0 + E, R).astype(np.int32)
        e[:min(R - 2, 21)] = e0 + E // 2                   # (21 rows on one expert: more than one turn of 16)
        e[R // 2], e[R - 1] = e0 + E, e0 - 1
    guard = 64
    out = torch.full((guard + R * N + guard,), float("nan"), dtype=TORCH[out_dt], device="cuda")
    args = (dev(xq), dev(xs), None if e is None else dev(e), dev(wq), dev(ws))
    hocf.check(hocf.hocf_gemv_i8(R, rows_per_x, E, e0, N, K, out_dt, *args, out[guard:guard + R * N], hocf.sync(1, None, 0),
                                 torch.cuda.current_stream()))
    torch.cuda.synchronize()
    assert out[:guard].isnan().all() and out[-guard:].isnan().all()
    want = np.zeros((R, N))
    for r in range(R):
        at = 0 if e is None else int(e[r]) - e0
        if 0 <= at < E:
            i = r // rows_per_x
            want[r] = ref.gemm(xq[i:i + 1], xs[i:i + 1], wq[at:at + 1], ws[at:at + 1])[0]
    near(out[guard:guard + R * N].view(R, N), want, np.abs(want), TORCH[out_dt], GEMM_STEPS)


# ------------------------------------------------------------------------------ the layer behind a dispatch

def test_experts_take_what_the_dispatch_leaves():
    """hocf_a2a_gemm's received rows (bit patterns, padded with zero rows to 256 a group, NaN behind the last) and offsets go
    into the layer as they are; near the layer without codes, and the same as from the rows as bfloat16."""
    say("experts behind a dispatch")
    P, E, B, topk, K, H, cap = 2, 3, 60, 2, 128, 256, 1100
    n = P * E
    w_up, w_down = normal((E, K, H), 1, K ** -0.5), normal((E, H, K), 2, H ** -0.5)
    X = normal((P, B, K), 3)
    chosen = np.stack([rng(4 + p).permuted(np.tile(np.arange(n), (B, 1)), axis=1)[:, :topk] for p in range(P)]).astype(np.int32)
    d = bf.A2aGemm(P, E, E, B, topk, H, K, BF16, X, dev(chosen), w_up, cap)
    d.poison()
    d.run()
    layer = moe_layer.ExpertsI8(E, cap, w_up, w_down)
    dy = normal((cap, K), 5)
    got = [layer.forward(d.recv, d.offsets).clone()] + [t.clone() for t in layer.backward(dy.view(torch.int16))]
    layer.check()
    off = d.offsets.tolist()
    assert off[0] == 0 and 512 <= off[-1] <= 768 and off[-1] % 256 == 0
    x = d.recv.view(torch.bfloat16).clone()
    again = [layer.forward(x, d.offsets), *layer.backward(dy)]
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    x[off[-1]:] = 0
    # (8 %: the bound of the layer's own test)
    for a, b in zip(got, plain_experts(x, w_up, w_down, dy, off)):
        a, b = host(a), b.numpy()
        assert np.linalg.norm(a - b) < 0.08 * np.linalg.norm(b)


def test_experts_refuse_other_shapes():
    say("experts' refusals")
    layer = moe_layer.ExpertsI8(2, 64, normal((2, 32, 48), 1), normal((2, 48, 32), 2))
    x, off = normal((64, 32), 3), torch.tensor([0, 30, 64], device="cuda")
    want = layer.forward(x, off).clone()
    for bad in (x[:1], x[0], x[:63], x[:, :16]):
        with pytest.raises(ValueError, match="x has shape"):
            layer.forward(bad, off)
        with pytest.raises(ValueError, match="dy has shape"):
            layer.backward(bad)
    for bad in (off[:2], off[:1], off[0]):
        with pytest.raises(ValueError, match="offsets"):
            layer.forward(x, bad)
    for a, o in ((x.int(), off), (x, off.float())):
        with pytest.raises(TypeError):
            layer.forward(a, o)
    assert torch.equal(layer.forward(x, off.int()), want) and torch.equal(layer.forward(x.float(), off), want)
