"""The table of how many clusters of a kernel a device holds: one per kernel
(also where two kernels have one type), per device and per cluster size; an
answer is asked for once, a failed query again."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MAIN = r"""
#include <cstdio>
#include "cluster_table.h"
template <int N> void kernel(int) {}
template <int N> int ask(int dev, int csize, int answer, int &asked)
{
    return smoe::cluster_table<kernel<N>>().get(dev, csize, [&] { ++asked; return answer; });
}
#define CHECK(x) if (!(x)) { std::printf("%s\n", #x); return 1; }
int main()
{
    int asked = 0;
    CHECK(ask<1>(0, 2, 76, asked) == 76 && asked == 1);
    CHECK(ask<1>(0, 2, 5, asked) == 76 && asked == 1);   // kept
    CHECK(ask<2>(0, 2, 38, asked) == 38 && asked == 2);  // another kernel of the same type
    CHECK(ask<1>(0, 2, 5, asked) == 76 && asked == 2);
    CHECK(ask<1>(0, 4, 30, asked) == 30 && asked == 3);  // another size, another device
    CHECK(ask<1>(0, 8, 12, asked) == 12 && asked == 4);
    CHECK(ask<1>(1, 2, 70, asked) == 70 && asked == 5);
    CHECK(ask<3>(0, 2, -1, asked) == 0 && asked == 6);   // failed: asked again
    CHECK(ask<3>(0, 2, 0, asked) == 0 && asked == 7);
    CHECK(ask<3>(0, 2, 9, asked) == 9 && asked == 8);
    CHECK(ask<3>(0, 2, 0, asked) == 9 && asked == 8);
    CHECK(ask<1>(-1, 2, 7, asked) == 0 && ask<1>(64, 2, 7, asked) == 0 && asked == 8);
    return 0;
}
"""


def test_cluster_table(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    src, exe = tmp_path / "main.cpp", tmp_path / "main"
    src.write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "moe_expert_ffn_smoe_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_the_product_uses_it():
    with open(os.path.join(ROOT, "moe_expert_ffn_smoe_gb300", "csrc", "q8_tc.cu")) as f:
        text = f.read()
    assert "cluster_table<Kernel>()" in text
