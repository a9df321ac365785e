"""The choice of kernel for grouped products (csrc/moe_choice.h), compiled for the host (CPU only)."""
import os
import subprocess

import pytest

import moe_cases as C

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "megatron_tensor_mlp_gb300", "csrc")
PAIRS = 76  # of a GB300 of 152 SMs

PROGRAM = r"""
#include <cstdio>
#include "moe_choice.h"
using namespace tpmlp::moe;
int main() {
    long long op, rows, experts, K, N, gathered;
    while (std::scanf("%lld %lld %lld %lld %lld %lld", &op, &rows, &experts, &K, &N, &gathered) == 6)
        std::printf("%d\n", op < 2   ? forward_kernel(rows, experts, K, N, op == 1, gathered, 76)
                            : op < 4 ? dx_kernel(rows, experts, K, N, op == 3, 76)
                                     : dw_kernel(rows, experts, K, N, gathered, 76));
}
"""
OPS = ["forward", "gated", "dx", "gated dx", "dw"]
KERNELS = ["few", "narrow", "wide"]


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    at = tmp_path_factory.mktemp("choice")
    (at / "choice.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(at / "choice.cpp"), "-o", str(at / "choice")], check=True)

    def run(cases):
        text = "\n".join(f"{OPS.index(op)} {rows} {e} {K} {N} {int(g)}" for op, rows, e, K, N, g in cases)
        out = subprocess.run([str(at / "choice")], input=text, capture_output=True, text=True, check=True).stdout.split()
        return [KERNELS[int(v)] for v in out]

    return run


def test_the_measured_products_take_the_faster_kernel(choose):
    """Rows, experts, K, N and the kernel that was faster, as the header's comments have them."""
    measured = [
        ("gated", 8, 64, 1024, 8192, True, "few"), ("forward", 128, 8, 4096, 1024, False, "few"), ("forward", 666, 8, 4096, 1024, False, "few"),
        ("gated", 128, 64, 1024, 8448, True, "wide"), ("forward", 1024, 16, 4096, 1024, False, "narrow"),
        ("dx", 30, 8, 624, 3840, False, "few"), ("dx", 1000, 8, 1024, 2048, False, "narrow"),
        ("gated dx", 8, 8, 4096, 5120, False, "few"), ("gated dx", 1400, 8, 512, 1024, False, "few"),
        ("gated dx", 600, 64, 1024, 1024, False, "narrow"), ("gated dx", 400, 8, 1024, 1024, False, "narrow"),
        ("forward", 16384, 8, 5120, 8192, True, "wide"), ("gated", 8192, 64, 1024, 2048, True, "wide"),
        ("gated", 6000, 8, 5120, 8192, False, "wide"), ("forward", 6000, 8, 5120, 8192, False, "wide"),
        ("gated", 16384, 16, 1024, 4096, False, "narrow"), ("gated", 8192, 8, 2048, 4096, False, "wide"),
        ("dw", 16384, 8, 5120, 8192, True, "wide"), ("dw", 16384, 8, 5120, 8192, False, "wide"), ("dw", 8192, 16, 4096, 2048, False, "narrow"),
    ]
    got = choose([m[:-1] for m in measured])
    wrong = [(m, k) for m, k in zip(measured, got) if k != m[-1]]
    assert not wrong, wrong


def test_the_kernels_tests_run_on_the_kernel_they_name(choose):
    got = choose([(op, sum(counts) + behind, len(counts), K, N, g) for op, _, counts, behind, K, N, g in C.CASES])
    wrong = [(C.name(c), k) for c, k in zip(C.CASES, got) if k != c[1]]
    assert not wrong, wrong
    # every kernel that there is, with rows in order and, where it takes them, gathered
    there = {(c[0], c[1], c[6]) for c in C.CASES}
    for op in ("forward", "gated"):
        assert {(op, k, g) for k in KERNELS for g in (False, True)} <= there
    assert {("dx", k, False) for k in KERNELS} <= there and {("gated dx", k, False) for k in KERNELS[:2]} <= there
    assert {("dw", k, g) for k in KERNELS[1:] for g in (False, True)} <= there


@pytest.mark.parametrize("tn", [64, 256])
def test_the_tiles_of_an_expert_cover_its_rows(tn):
    """tile_tokens of the kernels' tiles: ceil(n / TN) tiles of equal size, a multiple of 16, none empty."""
    for n in range(1, 40 * tn):
        nt = -(-n // tn)
        size = (-(-n // nt) + 15) // 16 * 16
        assert size <= tn and (nt - 1) * size < n <= nt * size, (tn, n)
