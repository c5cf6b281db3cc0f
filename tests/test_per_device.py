"""What is asked of a GPU once: kept for each device, and not where the question failed (CPU only, a small C++ program)."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_fp8_gemm_gb300", "csrc")
PROGRAM = r"""
#include "per_device.h"
#include <cstdio>
using namespace gemmar;
static int asked = 0, fails = 0;
static int here = 0;
static bool ask(int &v)
{
    ++asked;
    v = 100 + here;
    return fails-- <= 0;
}
#define CHECK(c) if (!(c)) return std::printf("%s\n", #c), 1
int main()
{
    PerDevice<int> p;
    int v = 0;
    fails = 2;
    CHECK(!p.get(0, v, ask) && !p.get(0, v, ask) && asked == 2);   // failed: asked again
    CHECK(p.get(0, v, ask) && v == 100 && asked == 3);
    v = 0;
    CHECK(p.get(0, v, ask) && v == 100 && asked == 3);             // kept
    here = 5;
    CHECK(p.get(5, v, ask) && v == 105 && asked == 4);             // another device's own
    CHECK(p.get(0, v, ask) && v == 100 && p.get(5, v, ask) && v == 105 && asked == 4);
    fails = 1;
    here = 7;
    CHECK(!p.get(7, v, ask) && p.get(5, v, ask) && v == 105 && p.get(7, v, ask) && v == 107 && asked == 6);
}
"""


def test_kept_by_device_and_not_after_a_failure(tmp_path):
    src, exe = tmp_path / "per_device.cpp", tmp_path / "per_device"
    src.write_text(PROGRAM)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-Wall", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
