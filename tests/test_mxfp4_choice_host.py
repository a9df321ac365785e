"""The choice of kernel and split for MXFP4 products (csrc/mxfp4_choice.h), compiled for the host (CPU only)."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "megatron_tensor_mlp_gb300", "csrc")

# What runs at once on a GB300 of 152 SMs (cudaOccupancyMaxActiveClusters, one CTA an SM), and the plain product's exchange
PAIRS, CLUSTERS = 76, {1: 152, 2: 76, 3: 46, 4: 36, 8: 15}
ROOM = 113 * 1024 - 1280

PROGRAM = r"""
#include <cstdio>
#include "mxfp4_choice.h"
using namespace tpmlp::mx;
int main() {
    Machine on{%d, {}};
    %s
    const Exchange ex{4, 1, %d};
    long long m, n, k;
    while (std::scanf("%%lld %%lld %%lld", &m, &n, &k) == 3) {
        const int kb = static_cast<int>((k + 255) / 256);
        const Choice c = choose(on, ex, {m, (n + 127) / 128 * ((m + 127) / 128), (m + 255) / 256 * ((n + 255) / 256), kb});
        std::printf("%%d %%d %%d\n", c.pair, c.split, ex.fits(c.split, static_cast<int>(m < 128 ? m : 128), kb));
    }
}
"""

# Measured microseconds of products m x n x k, weights out of L2: single CTAs, pairs, and K split 2, 3, 4 and 8 ways (a split
# that does not fit runs as the next smaller one).  On either side of what runs at once: 36, 46 and 76 tiles for one
# CTA an SM, 72 and 92 for two.
MEASURED = [
    (16, 20480, 1024, 6.6, 7.3, 13.0, 14.2, 18.1, 18.1),
    (1024, 1024, 1024, 4.8, 5.5, 6.4, 9.9, 10.4, 10.3),
    (16, 2560, 4096, 7.9, 8.4, 7.3, 7.2, 6.6, 7.9),
    (2048, 4096, 4096, 21.7, 14.7, 40.8, 61.8, 75.5, 75.5),
    (128, 4864, 8192, 15.2, 13.6, 12.2, 11.8, 13.8, 13.6),
    (640, 1024, 8192, 14.0, 13.4, 11.1, 10.4, 13.2, 13.2),
    (2048, 768, 8192, 13.8, 13.3, 13.0, 17.6, 22.6, 22.5),
    (1, 2560, 16384, 18.2, 21.2, 12.8, 11.1, 9.8, 10.9),
    (64, 2560, 16384, 21.3, 21.3, 14.6, 12.3, 11.0, 13.7),
    (65, 2048, 16384, 25.7, 21.2, 16.7, 13.8, 11.9, 13.6),
    (100, 5248, 16384, 26.4, 21.7, 18.2, 16.1, 17.5, 17.5),
    (128, 9728, 16384, 28.4, 23.0, 21.9, 22.6, 32.2, 32.3),
    (256, 4864, 16384, 26.1, 22.1, 18.2, 18.9, 27.5, 27.6),
    (333, 3200, 16384, 25.4, 21.9, 17.3, 17.9, 23.8, 23.8),
    (333, 4096, 16384, 25.9, 22.4, 20.1, 21.4, 29.4, 29.2),
    (800, 768, 16384, 23.4, 21.6, 15.9, 13.6, 15.8, 15.9),
    (1, 5120, 20480, 22.3, 26.1, 16.0, 14.7, 14.3, 20.6),
    (33, 2560, 20480, 24.9, 25.4, 16.2, 13.6, 11.8, 14.1),
    (64, 5120, 20480, 26.2, 25.6, 18.2, 16.0, 16.1, 24.7),
    (64, 6144, 20480, 26.5, 25.8, 19.1, 18.0, 17.5, 27.1),
    (128, 4096, 20480, 31.1, 26.3, 20.6, 17.3, 16.1, 16.1),
    (128, 4864, 20480, 31.4, 26.3, 20.9, 17.8, 18.9, 18.9),
    (128, 5120, 20480, 31.6, 26.6, 21.0, 18.1, 19.5, 19.6),
    (128, 5760, 20480, 31.6, 26.3, 21.3, 18.8, 20.2, 20.3),
    (128, 6144, 20480, 31.9, 26.6, 21.6, 20.5, 20.9, 21.0),
    (128, 8192, 20480, 33.3, 27.2, 24.0, 23.9, 23.9, 24.0),
    (128, 9728, 20480, 34.7, 27.5, 25.8, 25.8, 37.0, 36.9),
    (128, 10240, 20480, 35.0, 28.3, 27.5, 26.7, 37.8, 38.2),
    (200, 5248, 20480, 31.7, 26.3, 22.9, 20.7, 30.7, 30.7),
    (256, 2688, 20480, 29.7, 26.0, 19.3, 16.3, 18.3, 18.5),
    (512, 5120, 20480, 34.0, 27.0, 41.9, 39.4, 49.7, 49.5),
    (800, 5120, 20480, 36.4, 48.5, 47.1, 59.2, 68.7, 68.8),
]


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    d = tmp_path_factory.mktemp("choice")
    src, exe = d / "t.cc", d / "t"
    src.write_text(PROGRAM % (PAIRS, " ".join(f"on.clusters[{s}] = {c};" for s, c in CLUSTERS.items()), ROOM))
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(products):
        text = "\n".join("%d %d %d" % p for p in products)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
        return [tuple(int(x) for x in line.split()) for line in out if line]
    return run


def test_every_cluster_of_a_split_runs_at_once(choose):
    """A few clusters more than fit take another wave, which lasts as long as the first (76 tiles of 16384 split four
    ways took 27 us where two ways take 18)."""
    products = [(m, 128 * t, 256 * kb) for m in (1, 33, 100, 128) for t in range(1, 200) for kb in (1, 4, 16, 32, 64, 80, 256)]
    for (m, n, k), (pair, split, fits) in zip(products, choose(products)):
        tiles = n // 128
        assert fits and split <= max(1, k // 256)
        assert pair or split == 1 or tiles <= 2 * CLUSTERS[split], (m, n, k, split)
        assert m > 32 or not pair


def test_choice_costs_little(choose):
    """Within 15 % of the best measured form on either side of each limit."""
    for (m, n, k, *us), (pair, split, _) in zip(MEASURED, choose([r[:3] for r in MEASURED])):
        took = us[1] if pair else us[{1: 0, 2: 2, 3: 3, 4: 4, 8: 5}[split]]
        assert took <= 1.15 * min(us), (m, n, k, pair, split, us)
