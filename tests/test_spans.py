"""Which matrices share bytes, against every byte written down (CPU only, a small C++ program)."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_fp8_gemm_gb300", "csrc")
PROGRAM = r"""
#include "spans.h"
#include <cstdio>
#include <set>
using namespace gemmar;
static std::set<int64_t> bytes(int64_t at, int64_t row, int64_t stride, int64_t rows)
{
    std::set<int64_t> all;
    for (int64_t i = 0; i < rows; ++i)
        for (int64_t j = 0; j < row; ++j)
            all.insert(at + i * stride + j);
    return all;
}
int main()
{
    const int64_t shapes[][3] = {{1, 1, 1}, {3, 3, 4}, {2, 5, 3}, {4, 5, 3}, {1, 7, 4}, {3, 8, 2}, {5, 0, 3}, {2, 11, 5}, {6, 6, 1}, {40, 40, 1}, {3, 4, 9}};
    long cases = 0, met = 0;
    for (auto &a : shapes)
        for (auto &b : shapes)
            for (int64_t d = -70; d <= 70; ++d, ++cases) {
                const std::set<int64_t> x = bytes(1000, a[0], a[1], a[2]), y = bytes(1000 + d, b[0], b[1], b[2]);
                bool want = false;
                for (int64_t v : y)
                    want = want || x.count(v);
                const Span s = span_rows((void *)1000, a[0], a[1], a[2]), t = span_rows((void *)(1000 + d), b[0], b[1], b[2]);
                met += want;
                if (meet(s, t) != want || meet(t, s) != want || any_meet({s}, {t}) != want || any_meet({s, t}, {}) != want)
                    return std::printf("%ld %ld %ld | %ld %ld %ld at %ld: %d\n", (long)a[0], (long)a[1], (long)a[2], (long)b[0], (long)b[1], (long)b[2], (long)d, want), 1;
            }
    const Span none = span(nullptr, 100), some = span((void *)16, 1 << 20);
    if (meet(none, some) || meet(some, none) || meet(none, none))
        return 1;
    std::printf("%ld cases, %ld meet\n", cases, met);
}
"""


def test_meetings_of_spans(tmp_path):
    src, exe = tmp_path / "spans.cpp", tmp_path / "spans"
    src.write_text(PROGRAM)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-Wall", "-I", CSRC, str(src), "-o", str(exe)], check=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
    cases, met = (int(w) for w in r.stdout.split() if w.isdigit())
    assert cases == 11 * 11 * 141 and 1000 < met < cases
