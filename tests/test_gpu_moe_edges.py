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
