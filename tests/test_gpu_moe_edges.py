"""The mixture-of-experts operators where calls are unusual but allowed: rows
of no elements, scores that are equal in 64 bits, infinities, kernel forms
that only large or odd shapes take, errors that have to end with their call."""

import numpy as np
import pytest
import torch

import moe_ref as ref
from computation_collective_amd import buffers as bf
from computation_collective_amd import hocf
from test_gpu_moe import dev, gen, host, near, run, say

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
