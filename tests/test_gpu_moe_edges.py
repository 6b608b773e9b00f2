"""The mixture-of-experts operators where calls are unusual but allowed: rows
of no elements, scores that are equal in 64 bits, infinities, kernel forms
that only large or odd shapes take, errors that have to end with their call."""

import numpy as np
import pytest
import torch

import moe_ref as ref
from computation_collective_amd import buffers as bf
from computation_collective_amd import hocf
from computation_collective_amd import moe_layer
from test_gpu_moe import (HALF, TYPES, check_route, check_w4, combine_inputs, dev, gen, host, logits, near, run, say,
                          w4_case, w4_steps)

pytestmark = pytest.mark.gpu
SOFTMAX, SIGMOID = hocf.HOCF_SCORE_SOFTMAX, hocf.HOCF_SCORE_SIGMOID


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def entry(fn, *args):
    """A C entry with a sync block of its own on the current stream."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hocf.check(fn(*args, hocf.sync(1, None, 0, status=status), torch.cuda.current_stream()))
    torch.cuda.synchronize()
    assert int(status) == 0


# ------------------------------------------------------------------------------ weighted sum

@pytest.mark.parametrize("T", [3, 2048, 2050])
@pytest.mark.parametrize("dt", [hocf.HOCF_F32, hocf.HOCF_BF16])
def test_combine_bwd_of_rows_without_elements(T, dt):
    """N = 0, with rows that need not be there: the weights' gradients are empty sums, and nothing else is written."""
    topk, R = 2, 2 * T
    say(f"combine_bwd N=0 T={T} dt={dt}")
    index = torch.arange(R, dtype=torch.int32).view(T, topk).cuda()
    w, dw = torch.ones((T, topk)).cuda(), torch.full((T, topk), -7.0).cuda()
    around = torch.full((256,), 3.0).cuda()
    for rows, dout, drows in ((None, None, None), (None, None, around.data_ptr() + 16),
                              (w, w, around.data_ptr() + 128)):
        dw.fill_(-7.0)
        entry(hocf.hocf_moe_combine_bwd, T, topk, 0, R, dt, dt, rows, w, dout, index, index.view(-1), drows, dw)
        assert not dw.any() and (around == 3.0).all()


# ------------------------------------------------------------------------------ 4-bit weights

def test_w4_pack_on_another_stream_of_temporaries():
    """Codes and scales made on the current stream and dropped at once; the packing's stream is busy meanwhile and
    the current one fills the next tensors of the same sizes."""
    E, N, K, group = 4, 512, 1024, 64
    say("w4_pack on another stream")
    g = gen(3)
    codes = torch.randint(0, 16, (E, K, N), generator=g, dtype=torch.uint8).cuda()
    scales, zeros = (torch.rand(2, E, K // group, N, generator=g) + 0.5).bfloat16().cuda()
    want = bf.w4_pack(codes, scales, zeros, group)
    torch.cuda.synchronize()
    side, busy = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, None):
        with torch.cuda.stream(side):
            for _ in range(8):
                busy = busy @ busy * 1e-3
        got = bf.w4_pack(codes.clone(), scales.clone(), zeros.clone(), group, stream=stream)
        other = [torch.full_like(t, 9) for t in (codes, scales, zeros)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(other) == 3


# ------------------------------------------------------------------------------ routing

@pytest.mark.parametrize("E,n_group,topk_group,group_top", [(12, 1, 1, 1), (16, 1, 1, 1), (60, 4, 3, 1), (60, 4, 3, 2),
                                                            (250, 1, 1, 1), (480, 1, 1, 1), (480, 32, 30, 1)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_equal_scores_of_different_logits(E, n_group, topk_group, group_top, score, dtype):
    """Logits too small to move a 64-bit score: the scores are equal and the lower index comes first, whichever of a
    row's other logits are there (large ones take a token through the choice in 64 bits)."""
    say(f"route equal scores E={E} of {n_group} top {group_top} score={score} {dtype}")
    topk, size = min(E, 16), E // n_group
    tiny = torch.tensor([1e-20, 2e-20, -1e-30, 0.0, 3e-25, -0.0, 5e-20, 1e-21])
    x = torch.full((24, E), -3.0)
    for t in range(24):
        n = t % 9 + 2                            # so many tiny logits, spread over the row from expert t % 5 on
        at = (t % 5 + (E - 5) // n * torch.arange(n)).long()
        x[t, at] = tiny[torch.arange(n) % 8]
        if t >= 8:
            x[t, (t * 7) % E] = (2.0, 5.0, 25.0, 40.0)[t % 4]
    x = x.to(dtype).cuda()
    for renorm in (False, True):
        how = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top, renorm=renorm)
        e, w, c = ref.route(x.double().cpu().numpy(), topk, **how)
        h = run(bf.MoeRoute(24, E, topk, x, counts=True, **how))
        assert np.array_equal(h.experts.cpu().numpy(), e)
        assert np.array_equal(h.counts.cpu().numpy(), c)
        near(h.weights, w, np.abs(w), torch.float32, 100)


def test_route_equal_scores_across_keys():
    """Two logits a step apart on both sides of a fixed-point key's border near zero, whose distances to the row's
    largest round to the same 64-bit number."""
    low = torch.tensor(-2.0 ** -26)
    high = torch.nextafter(low, torch.tensor(0.0))
    assert float(low) - 20.0 == float(high) - 20.0 and high > low
    x = torch.full((4, 8), -9.0)
    for t, (a, b, top) in enumerate(((1, 5, 20.0), (5, 1, 20.0), (1, 5, -3.0), (5, 1, -3.0))):
        x[t, a], x[t, b], x[t, 3] = low, high, top
    x = x.cuda()
    e, w, _ = ref.route(x.double().cpu().numpy(), 3)
    for renorm in (False, True):
        h = run(bf.MoeRoute(4, 8, 3, x, renorm=renorm))
        assert h.experts.cpu().tolist() == e.tolist() == [[3, 1, 5], [3, 1, 5], [5, 1, 3], [1, 5, 3]]
    # the same between groups
    x = torch.full((2, 8), -9.0)
    x[:, 6] = 20.0
    x[0, 1], x[0, 3], x[1, 1], x[1, 3] = low, high, high, low
    x = x.cuda()
    e, _, _ = ref.route(x.double().cpu().numpy(), 2, n_group=4, topk_group=2)
    for renorm in (False, True):
        h = run(bf.MoeRoute(2, 8, 2, x, n_group=4, topk_group=2, renorm=renorm))
        assert h.experts.cpu().tolist() == e.tolist() == [[6, 1], [6, 1]]


@pytest.mark.parametrize("R,E,N,K,group", [(1, 1, 24, 136, 32), (5, 1, 40, 1160, 64), (20, 1, 24, 264, 128),
                                           (16, 4, 4104, 640, 64), (3, 40, 72, 4224, 128)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("out_dt", [torch.float32, torch.bfloat16])
def test_w4_values_that_are_not_finite(R, E, N, K, group, zeros, out_dt):
    """Infinities and NaN in x, scales and zero points, and finite values whose sums leave the range of binary32 before
    the zero points are taken off: what the definition gives in 64 bits."""
    inf, nan = float("inf"), float("nan")
    say(f"w4 not finite R={R} E={E} N={N} K={K} group={group} zeros={zeros}")
    for kind in range(6):
        codes, scales, z = w4_case(E, N, K, group, zeros, R + K + kind)
        x = torch.randn(R, K, generator=gen(kind)).bfloat16()
        if kind == 0:
            x[0, K // 2] = inf
        elif kind == 1:
            x[-1, 0], x[-1, K - 1] = -inf, inf
        elif kind == 2:
            x[R // 2, K - 3] = nan
        elif kind == 3:                          # finite, and so are the results: 3e38 * 1e-3 * 15 * K
            x[0] = 3e38 * torch.randn(K, generator=gen(9)).sign()
            x[-1, ::5] = 2e38
            scales *= 2.0 ** -14
        elif kind == 4:
            scales[0, 0, N // 2], scales[-1, -1, 3], scales[0, 0, 0] = inf, nan, 0.0
            x[:, 1] = 1e38
        elif zeros:
            z[0, 0, 5], z[-1, -1, N - 1] = inf, -inf
            z[0, 0, 1] = 1e30
        experts = torch.randint(-1, E + 1, (R,), generator=gen(R), dtype=torch.int32) if E > 1 else None
        if E > 1:
            experts[0], experts[-1] = 0, E - 1
        wq, s, zz = bf.w4_pack(codes.cuda(), scales.cuda(), None if z is None else z.cuda(), group)
        h = run(bf.GemvW4(R, 1, E, 0, N, K, group, x.cuda(), dev(experts), wq, s, zz,
                          out_dt=hocf.HOCF_F32 if out_dt == torch.float32 else hocf.HOCF_BF16))
        with np.errstate(invalid="ignore", over="ignore"):
            want, size = ref.w4(x.float().numpy(), codes.numpy(), scales.float().numpy(),
                                None if z is None else z.float().numpy(), None if experts is None else experts.numpy(),
                                0, 1, group)
        got, fin = host(h.out), np.isfinite(want)
        assert fin.all() or kind != 3
        assert np.array_equal(got[~fin], want[~fin], equal_nan=True), kind
        room = HALF[out_dt] * np.abs(want[fin]) + ref.rel_steps(w4_steps(K, group)) * size[fin] + 2.0 ** -126
        assert (np.abs(got[fin] - want[fin]) <= room).all(), kind


# ------------------------------------------------------------------------------ the layer

def two_way_layer(P, E, B, cap, recv_rows):
    """P * E = 2 experts; a token goes to the first where its first element is positive, else to the second."""
    K = H = 256
    g = gen(11)
    router = torch.zeros(K, 2)
    router[0] = torch.tensor([1.0, -1.0])
    up, down = (0.06 * torch.randn(2, K, H, generator=g)).bfloat16().cuda(), (0.06 * torch.randn(2, H, K, generator=g)).bfloat16().cuda()
    return moe_layer.MoeLayer(P, E, B, 1, router.bfloat16().cuda(), up, down, cap=cap, recv_rows=recv_rows)


def two_way_input(P, B, first):
    """`first` tokens of every rank go to the first expert."""
    x = 0.1 * torch.randn(P, B, 256, generator=gen(12))
    x[:, :, 0] = torch.where(torch.arange(B) < first, 3.0, -3.0)
    return x.bfloat16().cuda()


@pytest.mark.parametrize("P,E,cap,recv_rows,fits,does_not,match", [
    (1, 2, 8, 256, (8, 0), 3, "rank 0.*receive buffer"), (2, 1, 4, 512, (4,), 7, "its window holds 4")])
def test_layer_after_an_input_it_refused(P, E, cap, recv_rows, fits, does_not, match):
    """What a batch overflowed does not stay behind: the next one that fits is computed as by a new layer."""
    B = 8
    say(f"layer after a refused input P={P} cap={cap}")
    layer = two_way_layer(P, E, B, cap, recv_rows)
    for n in fits:
        with pytest.raises(RuntimeError, match=match):
            layer.forward(two_way_input(P, B, does_not))
        x = two_way_input(P, B, n)
        out = layer.forward(x)
        assert torch.equal(out, two_way_layer(P, E, B, cap, recv_rows).forward(x))
        drows, dlogits = layer.backward(x)
        layer.check()
        assert torch.isfinite(dlogits).all()


def test_layer_reports_what_its_operators_found():
    """An error word that an operator sets is raised once, by check() or by the next forward(), and cleared."""
    P, E, B = 2, 1, 8
    layer, x = two_way_layer(P, E, B, 8, 512), two_way_input(P, B, 4)
    say("layer reports")
    want = layer.forward(x)
    layer.check()
    for by_check in (True, False):
        layer.forward(x)
        layer.slots[1].index[3, 0] = 10 ** 6       # a row that no window has
        layer.backward(x)
        with pytest.raises(RuntimeError, match="source 1.*weighted sum.*index"):
            layer.check() if by_check else layer.forward(x)
        layer.check()
        assert torch.equal(layer.forward(x), want)
    layer.route.experts[5, 0] = -7                 # no expert of the row
    layer.backward(x)
    with pytest.raises(RuntimeError, match="router.*index"):
        layer.check()
    layer.check()


# ------------------------------------------------------------------------------ forms of large and odd shapes

@pytest.mark.parametrize("T,topk,N,bins,dt,out_dt", [
    (2048, 2, 64, 0, torch.bfloat16, torch.bfloat16), (2051, 3, 128, 4, torch.bfloat16, torch.float32),
    (2050, 2, 4096, 8, torch.bfloat16, torch.bfloat16), (2049, 8, 96, 8, torch.float32, torch.bfloat16),
    (2053, 9, 192, 5, torch.bfloat16, torch.bfloat16), (2048, 16, 64, 0, torch.float32, torch.float32),
    (2055, 12, 520, 3, torch.bfloat16, torch.bfloat16), (2050, 1, 32, 1, torch.float32, torch.float32)])
def test_combine_of_many_tokens(T, topk, N, bins, dt, out_dt):
    """A wave to a token: rows of whole cache lines (and one of parts of lines with more than eight places)."""
    say(f"combine of many tokens T={T} topk={topk} N={N} bins={bins} {dt} {out_dt}")
    rows, w, index, pair, dout = combine_inputs(T, topk, N, bins, dt, out_dt, T + N)
    if index is not None:
        gone = index[7].copy()
        index[7] = -1                            # a token without rows: theirs have no pair either
        pair[gone[gone >= 0]] = -1
        rows[torch.from_numpy(gone[gone >= 0]).long()] = float("nan")
    h = run(bf.MoeCombine(T, topk, N, dev(rows), dev(w), index=dev(index), out_dt=TYPES[out_dt]))
    out, size = ref.combine(rows.float().numpy(), w.numpy(), index)
    near(h.out, out, size, out_dt, topk + 1)
    h = run(bf.MoeCombineBwd(T, topk, N, dev(rows), dev(w), dev(dout), index=dev(index), pair=dev(pair)))
    dr, dw, size = ref.combine_bwd(rows.float().numpy(), w.numpy(), dout.float().numpy(), index)
    near(h.drows, dr, np.abs(dr), dt, 1)
    near(h.dweights, dw, size, torch.float32, N / 64 + 10)
    first = h.dweights.clone(), h.drows.clone()
    run(h)
    assert torch.equal(first[0], h.dweights) and torch.equal(first[1], h.drows)


@pytest.mark.parametrize("R,E,N,K,group,rows_of_one", [
    (16, 16, 2056, 264, 64, 0),       # 129 blocks of columns x 16 experts: two blocks to a workgroup, the last one alone
    (16, 32, 2056, 264, 128, 3),      # fewer rows than experts: a workgroup to the first row of each
    (32, 32, 1064, 1160, 32, 12),     # 9 to 16 blocks of rows, and passes that hold 12 rows
    (16, 16, 2072, 2184, 128, 9),     # more than 16 blocks of rows
    (64, 16, 2056, 1032, 64, 20),     # more rows of one expert than a tile
    (3, 1, 88, 1288, 128, 0), (4, 1, 264, 2048, 32, 0),   # one block to a workgroup, 9 to 16 blocks of rows, few rows
    (3, 1, 32792, 136, 64, 0), (40, 1, 16648, 392, 64, 0)])   # one matrix of many columns, a few rows and three tiles
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_of_many_blocks(R, E, N, K, group, rows_of_one, zeros):
    say(f"w4 of many blocks R={R} E={E} N={N} K={K} group={group} zeros={zeros}")
    experts = None
    if E > 1:
        experts = torch.randint(-1, E + 1, (R,), generator=gen(R + K), dtype=torch.int32)
        experts[:rows_of_one] = E - 1
    for out_dt in (torch.bfloat16, torch.float32):
        check_w4(R, 1, E, 0, N, K, group, zeros, experts, out_dt, R + N)


@pytest.mark.parametrize("E,n_group,topk_group,group_top,topk", [
    (500, 5, 2, 2, 8), (500, 5, 3, 1, 16), (495, 33, 9, 2, 10), (507, 39, 20, 1, 5), (510, 17, 4, 2, 7), (432, 3, 1, 2, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_long_runs_of_a_wave(E, n_group, topk_group, group_top, topk, dtype):
    """A wave to a token whose lanes hold 9 to 16 experts each."""
    say(f"route E={E} of {n_group} take {topk_group} top {group_top} {dtype}")
    bias = 0.01 * torch.randint(-20, 21, (E,), generator=gen(E)).float()
    for score, b, masked in ((SIGMOID, bias, 0.0), (SOFTMAX, None, 0.2), (SIGMOID, None, 0.5)):
        check_route(logits(70, E, dtype, 5 * E, E + 1, masked), topk, bias=b, score=score, n_group=n_group,
                    topk_group=topk_group, group_top=group_top, renorm=True)
