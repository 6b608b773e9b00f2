"""Host logic around the mixture-of-experts operators (CPU only): the rules by
which a call's kernel form is chosen, what the Python handles refuse, and that
the other operators' profile summaries stay valid beside them."""

import os
import shutil
import subprocess

import pytest
import torch

from computation_collective_amd import buffers as bf
from computation_collective_amd import profsum

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


def test_logits_rows_may_not_overlap():
    """The row stride is the tensor's own: rows less than E apart (a broadcast row, overlapping views) are refused."""
    E = 8
    one = torch.zeros((1, E))
    store = torch.zeros(64)
    for x in (one.expand(4, E), store.as_strided((4, E), (1, 1)), store.as_strided((2, E), (E - 1, 1)),
              store[:1, None].expand(3, 1)):
        with pytest.raises(ValueError, match="overlap"):
            bf._rows_ld(x, *x.shape)
    assert bf._rows_ld(torch.zeros((4, E)), 4, E) == E
    assert bf._rows_ld(torch.zeros((4, 11))[:, :E], 4, E) == 11
    assert bf._rows_ld(torch.zeros((9, E))[::3], 3, E) == 3 * E
    assert bf._rows_ld(one.expand(1, E), 1, E) == E and bf._rows_ld(torch.zeros((0, E)), 0, E) == E
    assert bf._rows_ld(torch.zeros((5, 1)), 5, 1) == 1
    with pytest.raises(ValueError, match="not adjacent"):
        bf._rows_ld(torch.zeros((E, 4)).t(), 4, E)


def test_route_refuses_overlapping_logits():
    """Both router handles ask before anything is bound."""
    x = torch.zeros((1, 8)).expand(4, 8)
    with pytest.raises(ValueError, match="overlap"):
        bf.MoeRoute(4, 8, 2, x)
    with pytest.raises(ValueError, match="overlap"):
        bf.MoeRouteBwd(4, 8, 2, x, torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2)))


def test_handles_refuse_host_memory():
    """Tensors in host memory are refused by every handle, before a kernel could be given their addresses."""
    T, E, topk, N, K, group = 4, 8, 2, 16, 64, 32
    i, b = torch.int32, torch.bfloat16
    logits, w, x = torch.zeros((T, E)), torch.zeros((T, topk)), torch.zeros((T, K), dtype=b)
    e, rows, index = torch.zeros((T, topk), dtype=i), torch.zeros((T * topk, N)), torch.zeros((T, topk), dtype=i)
    codes, scales = torch.zeros((1, K, N), dtype=torch.uint8), torch.zeros((1, K // group, N), dtype=b)
    words, small = bf.w4_layout(1, N, K, group)
    for make in (lambda: bf.MoeRoute(T, E, topk, logits, counts=True),
                 lambda: bf.MoeRouteBwd(T, E, topk, logits, e, w),
                 lambda: bf.MoeSlots(T, topk, 4, 2, 8, e),
                 lambda: bf.MoeCombine(T, topk, N, rows, w),
                 lambda: bf.MoeCombineBwd(T, topk, N, rows, w, torch.zeros((T, N)), index=index,
                                          pair=torch.zeros(T * topk, dtype=i)),
                 lambda: bf.w4_pack(codes, scales, None, group, stream=0),
                 lambda: bf.GemvW4(T, 1, 1, 0, N, K, group, x, None, torch.zeros(words, dtype=i),
                                   torch.zeros(small, dtype=b))):
        with pytest.raises(ValueError, match="on cpu"):
            make()


# ------------------------------------------------------------------ the bench's memory traffic

def test_committed_summaries_are_current():
    """Every profiled operator's traffic is known from the committed summaries, as bench.py prints it."""
    for op in list(profsum.workloads()) + list(profsum.COMPOSITE):
        if op in profsum.COMPOSITE or os.path.isfile(os.path.join(profsum.PROFILES, profsum.workloads()[op][0] + ".txt")):
            assert profsum.traffic(op), op


def test_summaries_outlive_other_operators_changes(tmp_path, monkeypatch):
    """The hash in a summary covers the profiled kernels' units and the headers they include, and nothing else."""
    src = profsum.source_hash()
    shutil.copytree(os.path.join(ROOT, "computation_collective_amd", "csrc"), tmp_path / "csrc")
    monkeypatch.setattr(profsum, "HERE", str(tmp_path))
    assert profsum.source_hash() == src

    def after(name, text):
        with open(tmp_path / "csrc" / name, "a") as fh:
            fh.write(text)
        return profsum.source_hash()

    for name in ("moe_route.hip", "gemv_w4.hip", "moe.hpp", "abi.cpp", "another.hip"):
        assert after(name, "// more\n") == src
    for name in ("embbag_a2a.hip", "mfma_tile.hpp", "common.hpp"):     # a unit, its header, that header's
        assert after(name, "// more\n") != src
        src = profsum.source_hash()
    with open(tmp_path / "csrc" / "new.hpp", "w") as fh:
        fh.write("// new\n")
    src = after("gemm_rs.hip", '#include "new.hpp"\n')
    assert after("new.hpp", "// more\n") != src
