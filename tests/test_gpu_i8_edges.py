"""The 8-bit integer operators on the GPU where test_gpu_i8.py does not reach:
every bf16 number through SiLU, and SiLU in every form of the kernel."""

import numpy as np
import pytest
import torch

import i8_ref as ref
from computation_collective_amd import buffers as bf
from test_gpu_i8 import BF16, F32, SILU, TORCH, dev, rng, same
from test_gpu_moe import host, run, say

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
