"""The adapters of a group of rows as the fused pair gets them, on the CPU (no
GPU needed): an id outside [0, count) of any value means no adapter, and what is
packed for a group comes back as it was.

A host program over the library's own header prints, for every id, the adapter
it stands for, and for every first, split and then of a group what the packed
words decode to.
"""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include "ks_internal.h"
int main() {
    const int counts[] = {1, 6, 65535};
    for (int count : counts) {
        const int ids[] = {INT_MIN, INT_MIN + 1, -131072, -100, -2, -1, 0, 1, count - 1, count, count + 7, 65535, INT_MAX};
        for (int first : ids)
            for (int then : ids)
                for (int split = 0; split <= ks::kPairGroup; ++split) {
                    const int f = ks::adapter_of(first, count), t = ks::adapter_of(then, count);
                    const ks::PairGroup g = ks::PairGroup::of(f, split, t);
                    std::printf("%d %d %d %d %d %d %d\n", count, first, then, split, g.first, g.split(), g.then());
                }
    }
}
"""


def test_packed_groups_come_back(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not found")
    src, exe = tmp_path / "groups.cpp", tmp_path / "groups"
    src.write_text(PROGRAM)
    subprocess.run([HIPCC, "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "kronecker_sparse_structured_amd", "csrc"), str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    assert len(lines) == 3 * 13 * 13 * 5
    for line in lines:
        count, first, then, split, got_first, got_split, got_then = map(int, line.split())
        want = [i if 0 <= i < count else -1 for i in (first, then)]
        assert [got_first, got_then] == want and got_split == split, line
