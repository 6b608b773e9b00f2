"""Host logic around the mixture-of-experts operators (CPU only): the rules by
which a call's kernel form is chosen, and what the Python handles refuse."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "computation_collective_amd", "csrc")

FORMS = r"""
#include "moe.hpp"
using namespace hocf;
// T, R, N, type, address of the rows' gradients
static_assert(combine_bwd_form(4096, 8192, 4096, kBF16, 1 << 12) == kRows, "whole lines");
static_assert(combine_bwd_form(2048, 1, 64, kBF16, 1 << 12) == kRows, "one line");
static_assert(combine_bwd_form(2048, 1, 32, kF32, 1 << 12) == kRows, "one line");
static_assert(combine_bwd_form(2047, 8192, 4096, kBF16, 1 << 12) == kWide, "few tokens");
static_assert(combine_bwd_form(2048, 8192, 2056, kBF16, 1 << 12) == kShifted, "parts of lines");
static_assert(combine_bwd_form(2048, 8192, 4096, kF32, (1 << 12) + 16) == kShifted, "rows that start inside a line");
static_assert(combine_bwd_form(2048, 0, 2056, kBF16, 1 << 12) == kWide, "no row to read");
// the shifted form reads the eight elements from min(max(.., 0), N - 8) on of dout and of every row: N = 0 has none
static_assert(combine_bwd_form(2048, 8192, 0, kBF16, (1 << 12) + 16) == kWide, "nothing in a row");
static_assert(combine_bwd_form(1 << 20, 8192, 0, kF32, (1 << 12) + 112) == kWide, "nothing in a row");
static_assert(combine_bwd_form(2048, 8192, 0, kBF16, 0) == kWide, "nothing in a row");
"""


def _hipcc():
    for c in (os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc"), shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    return None


def test_combine_bwd_form(tmp_path):
    """The form of the weighted sum's backward pass, at every border of the rule."""
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not found")
    src = tmp_path / "forms.cpp"
    src.write_text(FORMS)
    r = subprocess.run([hipcc, "-x", "hip", "--offload-arch=gfx950", "--cuda-host-only", "-std=c++17", "-fsyntax-only",
                        "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
