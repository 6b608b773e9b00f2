"""The mixture-of-experts operators on the GPU against plain 64-bit
implementations (moe_ref.py), at the sizes and masks where they can go wrong.

Choices, slots and counts are equal.  Computed values: half a step of the
output's type relative to the value, plus a stated number of binary32 half
steps (2^-24) relative to the sum of the magnitudes that the value is a sum
of.  Outputs are poisoned first, so an element that is not written shows."""

import numpy as np
import pytest
import torch

import moe_ref as ref
from computation_collective_amd import buffers as bf
from computation_collective_amd import hocf

pytestmark = pytest.mark.gpu
SOFTMAX, SIGMOID = hocf.HOCF_SCORE_SOFTMAX, hocf.HOCF_SCORE_SIGMOID
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def say(msg):
    print(f"\n[case] {msg}", flush=True)


def run(h):
    h.poison()
    h.run()
    torch.cuda.synchronize()
    assert h.status_value() == 0
    return h


def host(t):
    """A result in 64 bits (bf16 bit patterns decoded)."""
    t = t.view(torch.bfloat16) if t.dtype == torch.int16 else t
    return t.detach().cpu().double().numpy()


def near(got, want, size, dtype, steps):
    """|got - want| within half a step of `dtype` of want and `steps` binary32 half steps of `size`."""
    got = host(got)
    assert not np.isnan(got).any(), "unwritten (NaN) elements"
    room = HALF[dtype] * np.abs(want) + ref.rel_steps(steps) * size + 2.0 ** -126
    off = np.abs(got - want) - room
    if off.size == 0:
        return
    at = np.unravel_index(np.argmax(off), off.shape)
    assert off[at] <= 0, (at, got[at], want[at], room[at])


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------------------ routing

def logits(T, E, dtype, seed, ld=None, masked=0.0, spread=1.0):
    g = gen(seed)
    x = torch.full((T, ld or E), float("nan"))
    x[:, :E] = torch.randn(T, E, generator=g) * spread
    if masked:
        x[:, :E][torch.rand(T, E, generator=g) < masked] = float("-inf")
    return x.to(dtype).cuda()[:, :E]


def check_route(x, topk, bias=None, counts=True, **kw):
    T, E = x.shape
    h = bf.MoeRoute(T, E, topk, x, bias=None if bias is None else bias.cuda(), counts=counts, **kw)
    e, w, c = ref.route(x.double().cpu().numpy(), topk, None if bias is None else bias.numpy(), **kw)
    for again in range(2):
        run(h)
        assert np.array_equal(h.experts.cpu().numpy(), e), "experts"
        # distances of logits up to 12 from the row's largest, and 24 roundings of exp, sum and quotient
        near(h.weights, w, np.abs(w), torch.float32, 40)
        if counts:
            assert np.array_equal(h.counts.cpu().numpy(), c), "counts"
            assert not h.ws.any(), "workspace must be left zeroed"
    return h


@pytest.mark.parametrize("T,E,topk,dtype,ld", [
    (1, 1, 1, torch.float32, 1), (1, 8, 8, torch.float32, 8), (5, 7, 3, torch.bfloat16, 7),
    (33, 60, 4, torch.bfloat16, 64), (17, 61, 6, torch.float32, 64), (64, 64, 8, torch.float32, 64),
    (65, 128, 1, torch.bfloat16, 131), (130, 256, 8, torch.float32, 256), (67, 257, 5, torch.bfloat16, 260),
    (35, 512, 16, torch.float32, 515), (1000, 32, 2, torch.float32, 32)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_sizes(T, E, topk, dtype, ld, score):
    say(f"route T={T} E={E} topk={topk} {dtype} ld={ld} score={score}")
    for renorm in (False, True):
        check_route(logits(T, E, dtype, T + E, ld), topk, score=score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("E,n_group,topk_group,group_top,topk", [
    (8, 8, 3, 1, 3), (8, 4, 2, 2, 4), (60, 4, 1, 2, 6), (63, 7, 3, 2, 8), (256, 8, 4, 2, 8), (256, 8, 8, 1, 8),
    (240, 3, 2, 2, 8), (256, 64, 5, 2, 8), (512, 16, 4, 2, 16), (500, 4, 2, 1, 7), (48, 16, 3, 2, 9)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_groups(E, n_group, topk_group, group_top, topk, dtype):
    say(f"route groups E={E} of {n_group} take {topk_group} top {group_top} {dtype}")
    g = gen(E + n_group)
    bias = 0.01 * torch.randint(-20, 21, (E,), generator=g).float()
    for score, b, masked in ((SIGMOID, bias, 0.0), (SOFTMAX, None, 0.2), (SIGMOID, None, 0.5)):
        check_route(logits(70, E, dtype, 5 * E, E + 1, masked), topk, bias=b, score=score, n_group=n_group,
                    topk_group=topk_group, group_top=group_top, renorm=True)


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_masks_and_odd_values(score):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    rows = [[-inf] * 6, [nan] * 6, [nan, 0.0, -inf, -0.0, 0.0, -inf], [low] * 6, [low, -inf, low, 1.0, -inf, 1.0],
            [-inf, -inf, -inf, -inf, -inf, 3.0], [0.0] * 6, [80.0, 80.0, -80.0, 80.0, 1.0, 0.0],
            [-90.0, -91.0, -92.0, -93.0, -94.0, -95.0]]
    x = torch.tensor(rows).cuda()
    say(f"route odd values score={score}")
    # distances beyond 12 (and sums below 2^-126): the weights of the far ones are compared absolutely
    for renorm in (False, True):
        h = run(bf.MoeRoute(9, 6, 4, x, score=score, renorm=renorm, counts=True))
        e, w, c = ref.route(x.double().cpu().numpy(), 4, score=score, renorm=renorm)
        assert np.array_equal(h.experts.cpu().numpy(), e) and np.array_equal(h.counts.cpu().numpy(), c)
        got = host(h.weights)
        assert np.isfinite(got).all()
        assert (np.abs(got - w) <= ref.rel_steps(256) * np.abs(w) + 2.0 ** -126).all(), (got, w)


def test_route_infinite_logits_share():
    inf = float("inf")
    x = torch.tensor([[1.0, inf, 2.0, inf], [inf, -inf, 0.0, float("nan")]]).cuda()
    h = run(bf.MoeRoute(2, 4, 2, x))
    assert h.experts.tolist() == [[1, 3], [0, 2]] and h.weights.tolist() == [[0.5, 0.5], [1.0, 0.0]]


def test_route_near_ties():
    """Scores one binary32 step apart, and biases that put sums a 2^-30 apart or equal: the order of 64 bits."""
    say("route near ties")
    base = torch.tensor([0.7, -1.3, 2.1, 0.01])
    x = base.repeat(50, 16)
    step = torch.arange(64).repeat(50, 1) % 5 - 2
    x = torch.nextafter(x, x + step)            # neighbours: a step up, down, or the same
    x = x.cuda()
    for score in (SOFTMAX, SIGMOID):
        check_route(x, 8, score=score)
        check_route(x, 8, score=score, n_group=8, topk_group=3, group_top=2)
    g = gen(0)
    bias = torch.randint(-3, 4, (64,), generator=g).float() * 2.0 ** -24 + 0.1
    check_route(x, 8, bias=bias, score=SIGMOID)
    check_route(x, 8, bias=bias, score=SIGMOID, n_group=16, topk_group=3, group_top=2)


@pytest.mark.parametrize("E,n_group,topk_group,topk", [
    (16, 1, 1, 16), (30, 1, 1, 8), (64, 8, 3, 12), (100, 1, 1, 16), (128, 4, 2, 8), (256, 1, 1, 16), (256, 8, 4, 8),
    (250, 2, 1, 7), (300, 1, 1, 16), (512, 1, 1, 16), (512, 32, 6, 16), (60, 60, 9, 9)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_crowded(E, n_group, topk_group, topk, dtype):
    """Values that crowd around a few: most tokens are in doubt, more of them than a wave's list holds; the
    largest all in one lane's run, in rising and falling order; runs of equal logits; tiny logits."""
    say(f"route crowded E={E} of {n_group} topk={topk} {dtype}")
    T, g = 160, gen(E + topk)
    few = torch.tensor([0.5, 0.5001, -1.0, 2.0, 1e-3])
    x = few[torch.randint(0, 5, (T, E), generator=g)]
    x[:80] = torch.nextafter(x[:80], x[:80] + torch.randint(-2, 3, (80, E), generator=g))
    e = torch.arange(E).float()
    x[0], x[1], x[2], x[3] = e / 7, -e / 7, 3.0, 0.0
    x[4] = torch.where(e < E // 2, e * 2.0 ** -23 + 1.0, 0.0)
    x[5] = (e % 3) * 2.0 ** -20
    x[6:9] = torch.randn(3, E, generator=g) * 2.0 ** -14
    x[9] = -torch.inf
    x[10, E // 3:] = -torch.inf
    x[11, ::2] = torch.nan
    x = x.to(dtype).cuda()
    size = E // n_group
    for score, top2, bias in ((SOFTMAX, False, None), (SIGMOID, True, None),
                              (SIGMOID, True, torch.randint(-2, 3, (E,), generator=g) * 2.0 ** -10), (SOFTMAX, True, None)):
        check_route(x, topk, bias=bias, score=score, n_group=n_group, topk_group=topk_group,
                    group_top=2 if top2 and size > 1 and n_group > 1 else 1, renorm=True)


@pytest.mark.parametrize("E,n_group,topk_group,topk", [(64, 8, 3, 12), (256, 8, 4, 8), (512, 32, 6, 16), (100, 1, 1, 7)])
@pytest.mark.parametrize("spread", [0.1, 1.0, 4.0])
def test_route_softmax_by_score(E, n_group, topk_group, topk, spread):
    """Softmax scores with biases (all different: sums that are equal but for their rounding have no order), flat rows
    and peaked ones, half of the logits within a few steps of another one."""
    say(f"route softmax by score E={E} of {n_group} spread={spread}")
    T, g = 150, gen(E + topk)
    x = spread * torch.randn(T, E, generator=g)
    x[:, E // 2:] = torch.nextafter(x[:, :E - E // 2], x[:, :E - E // 2] + torch.randint(-1, 2, (T, E - E // 2), generator=g))
    bias = 1e-3 * torch.randn(E, generator=g)
    near_bias = 0.01 + 2.0 ** -30 * torch.randperm(E, generator=g).float()
    for b in (bias, near_bias, None):
        check_route(x.cuda(), topk, bias=b, score=SOFTMAX, n_group=n_group, topk_group=topk_group,
                    group_top=2 if n_group > 1 else 1, renorm=True)


@pytest.mark.parametrize("grid", [1, 3, 9])
def test_route_few_workgroups(grid, monkeypatch):
    """Many tokens a wave, in the last step a part of one; counts from a grid of any size."""
    monkeypatch.setenv("HOCF_MAX_WORKGROUPS", str(grid))
    say(f"route grid={grid}")
    bias = 0.001 * torch.randint(-9, 10, (256,), generator=gen(1)).float()
    check_route(logits(1001, 256, torch.float32, 2), 8, bias=bias, score=SIGMOID, n_group=8, topk_group=4, group_top=2)
    check_route(logits(1003, 40, torch.bfloat16, 3, masked=0.3), 4)
    x = logits(515, 320, torch.float32, 4)
    check_route(x, 3, score=SIGMOID)
    dw = torch.randn(515, 3, generator=gen(5))
    e = ref.route(x.double().cpu().numpy(), 3)[0]
    h = run(bf.MoeRouteBwd(515, 320, 3, x, torch.from_numpy(e).cuda(), dw.cuda()))
    d, size = ref.route_bwd(x.double().cpu().numpy(), e, dw.numpy(), SOFTMAX, False, 1.0)
    near(h.dlogits, d, size, torch.float32, 80)


def test_route_odd_biases():
    """Biases beyond the keys' range, and experts that a NaN or -inf bias rules out."""
    say("route odd biases")
    x = logits(40, 24, torch.float32, 3, masked=0.2)
    for kind in range(4):
        b = 0.1 * torch.randn(24, generator=gen(kind))
        if kind == 0:
            b[::3] += 100.0
        elif kind == 1:
            b -= 3.9
        elif kind == 2:
            b[::2] = -1e30
        else:
            b[5], b[6] = float("nan"), float("-inf")
        e = ref.route(x.double().cpu().numpy(), 6, torch.nan_to_num(b, nan=-np.inf, neginf=-np.inf, posinf=np.inf).numpy(),
                      score=SIGMOID, n_group=4, topk_group=3, group_top=2)[0]
        h = run(bf.MoeRoute(40, 24, 6, x, bias=b.cuda(), score=SIGMOID, n_group=4, topk_group=3, group_top=2))
        assert np.array_equal(h.experts.cpu().numpy(), e), kind


def test_route_far_logits_by_value():
    """Softmax scores that underflow or saturate even in 64 bits tie: the lower index."""
    x = torch.tensor([[0.0, -800.0, -790.0, -900.0, -5.0], [60.0, 50.0, 55.0, 45.0, 70.0]]).cuda()
    h = run(bf.MoeRoute(2, 5, 4, x))
    e, _, _ = ref.route(x.double().cpu().numpy(), 4)
    assert np.array_equal(h.experts.cpu().numpy(), e)
    h = run(bf.MoeRoute(2, 5, 4, x, score=SIGMOID))
    e, _, _ = ref.route(x.double().cpu().numpy(), 4, score=SIGMOID)
    assert np.array_equal(h.experts.cpu().numpy(), e)


def test_route_empty_and_counts():
    x = torch.empty((0, 8), device="cuda")
    h = run(bf.MoeRoute(0, 8, 2, x, counts=True))
    assert not h.counts.any() and not h.ws.any()
    bf.MoeRoute(0, 8, 2, x).run()
    check_route(logits(20000, 40, torch.float32, 1), 5)          # many workgroups add to one table


@pytest.mark.parametrize("T,E,topk,dtype,ld", [
    (1, 1, 1, torch.float32, 1), (3, 9, 4, torch.bfloat16, 9), (33, 60, 4, torch.float32, 64),
    (40, 64, 8, torch.bfloat16, 64), (65, 128, 8, torch.bfloat16, 128), (31, 256, 8, torch.float32, 259),
    (20, 511, 16, torch.bfloat16, 511), (9, 512, 3, torch.float32, 512)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_bwd(T, E, topk, dtype, ld, score, renorm):
    say(f"route_bwd T={T} E={E} topk={topk} {dtype} score={score} renorm={renorm}")
    x = logits(T, E, dtype, T + E, ld, masked=0.1)
    xs = x.double().cpu().numpy()
    e, _, _ = ref.route(xs, topk, score=score)
    dw = torch.randn(T, topk, generator=gen(7))
    if T > 2:
        e[1] = -1                                # a token without experts
        e[2, :topk // 2] = -1
    h = run(bf.MoeRouteBwd(T, E, topk, x, torch.from_numpy(e).cuda(), dw.cuda(), score=score, renorm=renorm, scale=2.5))
    d, size = ref.route_bwd(xs, e, dw.numpy(), score, renorm, 2.5)
    # as the weights (40), the sum over topk places, and the products and differences after them
    near(h.dlogits, d, size, dtype, 80)


def test_route_bwd_against_differences():
    T, E, topk = 6, 24, 4
    x = logits(T, E, torch.float32, 9)
    xs = x.double().cpu().numpy()
    dw = torch.randn(T, topk, generator=gen(8))
    for score in (SOFTMAX, SIGMOID):
        for renorm in (False, True):
            r = run(bf.MoeRoute(T, E, topk, x, score=score, renorm=renorm))
            e = r.experts.cpu().numpy()
            h = run(bf.MoeRouteBwd(T, E, topk, x, r.experts, dw.cuda(), score=score, renorm=renorm))
            got, step = host(h.dlogits), 1e-5
            for k in range(E):
                up, dn = xs.copy(), xs.copy()
                up[:, k] += step
                dn[:, k] -= step
                num = ((ref.weights_of(up, e, score, renorm, 1.0) - ref.weights_of(dn, e, score, renorm, 1.0)) *
                       dw.numpy()).sum(1) / (2 * step)
                # differences: step^2 (third derivatives below 1) and 2^-53 / step; the kernel: 80 half steps of |dw| < 4
                assert np.abs(got[:, k] - num).max() <= 4 * (1e-10 + 2.0 ** -53 / step + ref.rel_steps(80) * 4)


def test_route_bwd_bad_place():
    x = logits(2, 8, torch.float32, 1)
    e = torch.tensor([[1, 8], [-5, 3]], dtype=torch.int32).cuda()
    h = bf.MoeRouteBwd(2, 8, 2, x, e, torch.ones(2, 2).cuda(), score=SIGMOID)
    h.poison()
    h.run()
    torch.cuda.synchronize()
    assert h.status_value() == hocf.HOCF_ERR_BAD_INDEX
    keep = np.array([[1, -1], [-1, 3]])
    d, size = ref.route_bwd(x.double().cpu().numpy(), keep, np.ones((2, 2)), SIGMOID, False, 1.0)
    near(h.dlogits, d, size, torch.float32, 80)


# ------------------------------------------------------------------------------ window rows

def choices(T, topk, E, seed, none=0.0, beyond=0):
    """Random experts; some places empty, some naming experts beyond E."""
    g = gen(seed)
    e = torch.randint(0, E + beyond, (T, topk), generator=g, dtype=torch.int32)
    if none:
        e[torch.rand(T, topk, generator=g) < none] = -1
    return e


@pytest.mark.parametrize("T,topk,bins,per_bin,cap", [
    (0, 2, 3, 2, 5), (1, 1, 1, 1, 1), (1, 1, 64, 1, 1), (31, 3, 5, 3, 20), (64, 1, 2, 1, 64), (513, 2, 8, 4, 200),
    (1000, 8, 16, 16, 700), (2048, 8, 64, 3, 300), (2049, 8, 64, 3, 300), (4097, 5, 7, 1, 0), (9000, 4, 33, 2, 1200),
    (70001, 3, 1, 5, 250000), (300000, 8, 9, 7, 300000)])
def test_slots(T, topk, bins, per_bin, cap):
    say(f"slots T={T} topk={topk} bins={bins}x{per_bin} cap={cap}")
    e = choices(T, topk, bins * per_bin, T, none=0.1, beyond=2)
    if T > 600:
        e[100:400] = e[0, 0]                     # a run on one bin
        e[400:500] = -1
    index, pair, counts = ref.slots(e.numpy(), bins, per_bin, cap)
    h = bf.MoeSlots(T, topk, bins, per_bin, cap, e.cuda())
    h.ws.fill_(-1)                               # the workspace needs no zeroing
    for again in range(2):
        run(h)
        assert np.array_equal(h.counts.cpu().numpy(), counts)
        assert np.array_equal(h.index.cpu().numpy(), index)
        assert np.array_equal(h.pair.cpu().numpy(), pair)


def test_slots_odd_experts():
    e = torch.tensor([[-1, -2], [2 ** 31 - 1, -2 ** 31], [5, 6]], dtype=torch.int32).cuda()
    h = run(bf.MoeSlots(3, 2, 3, 2, 2, e))
    assert h.index.tolist() == [[-1, -1], [-1, -1], [4, -1]] and h.counts.tolist() == [0, 0, 1]


# ------------------------------------------------------------------------------ weighted sum

def combine_inputs(T, topk, N, bins, dt, out_dt, seed, none=0.1):
    """Rows in windows a third larger than needed (bins = 0: in pair order); what no pair names is NaN."""
    g = gen(seed)
    w = torch.rand(T, topk, generator=g) + 0.05
    if bins:
        cap = T * topk // bins + T * topk // (3 * bins) + 9
        e = choices(T, topk, bins, seed, none)
        index, pair, _ = ref.slots(e.numpy(), bins, 1, cap)
        rows = torch.randn(bins * cap, N, generator=g)
        rows[torch.from_numpy(pair) < 0] = float("nan")
    else:
        index = pair = None
        rows = torch.randn(T * topk, N, generator=g)
    return rows.to(dt), w, index, pair, torch.randn(T, N, generator=g).to(out_dt)


def dev(a):
    return None if a is None else (torch.from_numpy(a) if isinstance(a, np.ndarray) else a).cuda()


TYPES = {torch.float32: hocf.HOCF_F32, torch.bfloat16: hocf.HOCF_BF16}
SHAPES = [(1, 1, 8, 0), (3, 2, 16, 2), (4, 2, 4096, 0), (5, 3, 40, 3), (7, 8, 520, 4), (33, 4, 1032, 8), (66, 5, 264, 1),
          (9, 16, 2056, 8), (10, 9, 128, 0), (300, 6, 64, 8), (2050, 7, 24, 8), (2300, 8, 520, 0), (2, 1, 65544, 1)]


@pytest.mark.parametrize("T,topk,N,bins", SHAPES)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out_dt", [torch.float32, torch.bfloat16])
def test_combine(T, topk, N, bins, dt, out_dt):
    say(f"combine T={T} topk={topk} N={N} bins={bins} {dt} -> {out_dt}")
    rows, w, index, _, add = combine_inputs(T, topk, N, bins, dt, out_dt, T + N)
    if index is not None and T > 2:
        index[1] = -1                            # a token without rows
    for a in (None, add):
        h = run(bf.MoeCombine(T, topk, N, dev(rows), dev(w), index=dev(index), add=dev(a), out_dt=TYPES[out_dt]))
        out, size = ref.combine(rows.float().numpy(), w.numpy(), index, None if a is None else a.float().numpy())
        near(h.out, out, size, out_dt, topk + 1)  # one rounding for each product-sum and for add


@pytest.mark.parametrize("T,topk,N,bins", SHAPES)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out_dt", [torch.float32, torch.bfloat16])
def test_combine_bwd(T, topk, N, bins, dt, out_dt):
    say(f"combine_bwd T={T} topk={topk} N={N} bins={bins} {dt} <- {out_dt}")
    rows, w, index, pair, dout = combine_inputs(T, topk, N, bins, dt, out_dt, T + N + 1)
    h = run(bf.MoeCombineBwd(T, topk, N, dev(rows), dev(w), dev(dout), index=dev(index), pair=dev(pair)))
    dr, dw, size = ref.combine_bwd(rows.float().numpy(), w.numpy(), dout.float().numpy(), index)
    near(h.drows, dr, np.abs(dr), dt, 1)
    near(h.dweights, dw, size, torch.float32, N / 64 + 10)    # a lane's run of products, then the folds
    first = h.dweights.clone(), h.drows.clone()
    run(h)
    assert torch.equal(first[0], h.dweights) and torch.equal(first[1], h.drows), "another call, other bits"


def test_combine_gradients_are_the_formulas_differences():
    """<dout, out> is linear in each weight and each row: unit steps give the gradients."""
    T, topk, N = 3, 2, 16
    rows, w, index, pair, dout = combine_inputs(T, topk, N, 2, torch.float32, torch.float32, 3)
    h = run(bf.MoeCombineBwd(T, topk, N, dev(rows), dev(w), dev(dout), index=dev(index), pair=dev(pair)))
    x = np.nan_to_num(rows.numpy())
    for t in range(T):
        for j in range(topk):
            up = w.numpy().astype(np.float64).copy()
            up[t, j] += 1
            num = ((ref.combine(x, up, index)[0] - ref.combine(x, w.numpy(), index)[0]) * dout.numpy()).sum()
            assert abs(host(h.dweights)[t, j] - num) <= 30 * 2.0 ** -24 * N * 9
    for r in range(len(x)):
        up = x.astype(np.float64).copy()
        up[r, 5] += 1
        num = ((ref.combine(up, w.numpy(), index)[0] - ref.combine(x, w.numpy(), index)[0]) * dout.numpy()).sum()
        assert abs(host(h.drows)[r, 5] - num) <= 2.0 ** -22 * 4 + 1e-12


def test_combine_without_rows():
    """R = 0 and T = 0: nothing is read, everything is written."""
    w = torch.ones(3, 2).cuda()
    none = torch.full((3, 2), -1, dtype=torch.int32).cuda()
    rows, add = torch.empty((0, 16)).cuda(), torch.randn(3, 16).cuda()
    h = run(bf.MoeCombine(3, 2, 16, rows, w, index=none, add=add, out_dt=hocf.HOCF_F32))
    assert torch.equal(h.out, add)
    h = run(bf.MoeCombineBwd(3, 2, 16, rows, w, add, index=none, pair=torch.empty(0, dtype=torch.int32).cuda()))
    assert not h.dweights.any()
    e, f = torch.empty((0, 2)).cuda(), torch.empty((0, 2), dtype=torch.int32).cuda()
    rows, pair = torch.randn(5, 16).cuda(), torch.full((5,), -1, dtype=torch.int32).cuda()
    h = run(bf.MoeCombineBwd(0, 2, 16, rows, e, torch.empty((0, 16)).cuda(), index=f, pair=pair))
    assert not h.drows.any()
    run(bf.MoeCombine(0, 2, 16, rows, e, index=f, out_dt=hocf.HOCF_F32))


def test_combine_bad_index():
    rows, w = torch.randn(4, 8).cuda(), torch.ones(2, 2).cuda()
    index = torch.tensor([[0, 4], [-2, 3]], dtype=torch.int32).cuda()
    h = bf.MoeCombine(2, 2, 8, rows, w, index=index, out_dt=hocf.HOCF_F32)
    h.poison()
    h.run()
    torch.cuda.synchronize()
    assert h.status_value() == hocf.HOCF_ERR_BAD_INDEX
    assert torch.equal(h.out, rows[[0, 3]])
    pair = torch.tensor([0, -1, -1, 3], dtype=torch.int32).cuda()
    h = bf.MoeCombineBwd(2, 2, 8, rows, w, torch.ones(2, 8).cuda(), index=index, pair=pair)
    h.poison()
    h.run()
    torch.cuda.synchronize()
    assert h.status_value() == hocf.HOCF_ERR_BAD_INDEX
    assert torch.equal(h.drows, torch.tensor([1.0, 0, 0, 1])[:, None].expand(4, 8).cuda())
    assert h.dweights[0, 1] == 0 and h.dweights[1, 0] == 0


# ------------------------------------------------------------------------------ 4-bit weights

def w4_case(E, N, K, group, zeros, seed):
    g = gen(seed)
    groups = -(-K // group)
    codes = torch.randint(0, 16, (E, K, N), generator=g, dtype=torch.uint8)
    scales = (0.01 * (0.5 + torch.rand(E, groups, N, generator=g))).bfloat16()
    z = torch.randint(0, 16, (E, groups, N), generator=g).bfloat16() if zeros else None
    return codes, scales, z


def w4_steps(K, group):
    """Binary32 half steps, relative to the sum of |x| |scale| (|zero| + 31): the 32 products of a matrix instruction
    in any order, even truncated (64), four chained (8), zero, scale and fold (8), and the sum over groups."""
    return 80 + -(-K // group)


def check_w4(R, per, E, e0, N, K, group, zeros, experts, out_dt, seed=0):
    codes, scales, z = w4_case(E, N, K, group, zeros, seed)
    x = torch.randn(R // per, K, generator=gen(seed + 1)).bfloat16()
    wq, s, zz = bf.w4_pack(codes.cuda(), scales.cuda(), None if z is None else z.cuda(), group)
    h = bf.GemvW4(R, per, E, e0, N, K, group, x.cuda(), dev(experts), wq, s, zz, out_dt=TYPES[out_dt])
    out, size = ref.w4(x.float().numpy(), codes.numpy(), scales.float().numpy(), None if z is None else z.float().numpy(),
                       None if experts is None else experts.numpy(), e0, per, group)
    run(h)
    near(h.out, out, size, out_dt, w4_steps(K, group))
    first = h.out.clone()
    run(h)
    assert torch.equal(h.out, first), "another call, other bits"
    return h


@pytest.mark.parametrize("R,N,K", [(1, 8, 8), (1, 16, 128), (2, 40, 136), (5, 264, 1048), (16, 64, 512), (17, 72, 520),
                                   (32, 128, 1024), (33, 24, 2056), (64, 520, 264), (65, 16, 384), (200, 48, 160),
                                   (1, 4096, 4096), (3, 8, 8192)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_one_matrix(R, N, K, group):
    say(f"w4 R={R} N={N} K={K} group={group}")
    for zeros, out_dt in ((False, torch.bfloat16), (True, torch.float32)):
        check_w4(R, 1, 1, 0, N, K, group, zeros, None, out_dt, R + K)


@pytest.mark.parametrize("T,topk,E,e0,N,K", [
    (1, 8, 64, 0, 48, 256), (1, 1, 8, 3, 16, 128), (4, 2, 4, 2, 40, 648), (16, 2, 32, 0, 264, 384), (20, 4, 3, 0, 24, 1160),
    (40, 2, 2, 1, 72, 136), (128, 8, 5, 0, 16, 64)])
@pytest.mark.parametrize("up", [True, False])
def test_w4_experts(T, topk, E, e0, N, K, up):
    say(f"w4 experts T={T} topk={topk} E={E} from {e0} N={N} K={K} up={up}")
    e = choices(T, topk, E + e0, T + N, none=0.1, beyond=2).reshape(-1)
    if T > 4:
        e[3:3 + T] = e0                          # more rows of one expert than one tile holds
    for group, zeros, out_dt in ((32, True, torch.bfloat16), (128, False, torch.float32)):
        check_w4(T * topk, topk if up else 1, E, e0, N, K, group, zeros, e, out_dt, T)


def test_w4_all_rows_of_other_ranks():
    e = torch.tensor([7, -1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    for E in (2, 6):
        h = check_w4(4, 2, E, 8, 24, 128, 64, True, e, torch.float32)
        assert not h.out.any()


def test_w4_empty():
    check_w4(0, 1, 1, 0, 16, 64, 32, False, None, torch.float32)
    check_w4(3, 1, 1, 0, 16, 0, 32, False, None, torch.float32)


def test_w4_padding_is_not_read_into_results():
    """Codes, scales and zeros beyond K and N may hold anything."""
    N, K, group = 24, 136, 32
    codes, scales, z = w4_case(1, N, K, group, True, 5)
    x = torch.randn(3, K, generator=gen(6)).bfloat16().cuda()
    wq, s, zz = bf.w4_pack(codes.cuda(), scales.cuda(), z.cuda(), group)
    clean = run(bf.GemvW4(3, 1, 1, 0, N, K, group, x, None, wq, s, zz)).out.clone()
    wq[:, 1, :, 8::16] = -1
    wq[:, 1, :, 9::16] = 0x55555555
    wq[:, :, 1, 16:] = -1                        # rows from 136 on
    wq[:, :, 1, :, 1:] = 0x7fffffff
    for n in range(8, 16):
        s[:, 1, :, n] = float("nan")
        zz[:, 1, :, n] = float("inf")
    assert torch.equal(run(bf.GemvW4(3, 1, 1, 0, N, K, group, x, None, wq, s, zz)).out, clean)


def test_w4_pack_places():
    """One code at a time lands in its four bits."""
    N, K = 24, 264
    for n, k in ((0, 0), (3, 1), (17, 130), (23, 263), (5, 39), (15, 127)):
        codes = torch.zeros((1, K, N), dtype=torch.uint8)
        codes[0, k, n] = 13
        wq, _, _ = bf.w4_pack(codes.cuda(), torch.ones(1, 3, N).bfloat16().cuda(), None, 128)
        at = wq.cpu().nonzero().tolist()
        assert at == [[0, n // 16, k // 128, (k % 32 // 8) * 16 + n % 16, k % 128 // 32]]
        bit = (3 + 16 * (k % 2) + 4 * (k % 8 // 2)) % 32
        want = (13 << bit | 13 >> (32 - bit)) & 0xFFFFFFFF if bit else 13
        assert int(wq.cpu()[tuple(at[0])]) & 0xFFFFFFFF == want
