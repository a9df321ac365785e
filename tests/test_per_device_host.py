"""What the launchers keep per device is computed once and seen whole by every thread (CPU only; under the thread
sanitizer where the compiler has it)."""
import glob
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "megatron_tensor_mlp_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"

struct Value { int a = -1, b = -1; };

int main() {
    for (int round = 0; round < 200; ++round) {
        tpmlp::PerDevice<Value> cache;
        std::atomic<int> computed{0}, wrong{0};
        std::vector<std::thread> threads;
        for (int t = 0; t < 8; ++t)
            threads.emplace_back([&, t] {
                for (int i = 0; i < 4; ++i) {
                    const int device = (t + i) % 4;
                    const Value v = cache.get(device, [&](Value& w) { ++computed; w.a = device; w.b = 10 * device; return true; });
                    if (v.a != device || v.b != 10 * device) ++wrong;
                }
            });
        for (auto& t : threads) t.join();
        if (computed != 4 || wrong != 0) return std::printf("computed %d wrong %d\n", computed.load(), wrong.load()), 1;
    }
    // a value that does not hold is computed again; so is one past the last device
    tpmlp::PerDevice<int> cache;
    int n = 0;
    for (int i = 0; i < 3; ++i) cache.get(1, [&](int& v) { v = ++n; return n == 2; });
    if (n != 2 || cache.get(1, [](int&) { return false; }) != 2) return 2;
    for (int i = 0; i < 2; ++i)
        if (cache.get(64, [&](int& v) { v = ++n; return true; }) != 3 + i) return 3;
    return 0;
}
"""


def test_first_use_by_many_threads(tmp_path):
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(PROGRAM)
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-pthread", "-I", CSRC, str(src), "-o", str(exe)]
    if subprocess.run(cmd + ["-fsanitize=thread"], capture_output=True).returncode != 0:
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    if "unexpected memory mapping" in r.stderr:
        pytest.skip("the sanitizer does not run on this kernel")
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu"))), ids=os.path.basename)
def test_launchers_keep_no_plain_flags(path):
    """(a function's own static flag, set and read without synchronisation, is what PerDevice replaces)"""
    assert not re.findall(r"^\s+static (?:bool|int) \w+\[", open(path).read(), flags=re.M)
