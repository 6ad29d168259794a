"""The serving operators' host arithmetic at the ends of what they accept
(CPU only): numbers of CTAs, and divisions by a launch's divisor."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "serve.cuh"
using namespace q4;
int main()
{
    const int64_t most = 2147483647;
    const int per[] = {1, 4, 512};
    const int64_t n[] = {1, 3, 4, 5, 511, 512, 513, most - 512, most - 511, most - 3, most - 2, most};
    for (int p : per)
        for (int64_t x : n) {
            const int64_t c = ctas_for(x, p);
            if (c < 1 || c * p < x || (c - 1) * p >= x) return printf("%lld things, %d each: %lld\n", (long long)x, p, (long long)c), 1;
        }
    for (int64_t d = 1; d <= 65536; ++d) {
        FastDiv f;
        f.set(static_cast<int>(d));
        for (int64_t k : {int64_t{0}, int64_t{1}, int64_t{2}, most / d / 2, most / d - 1, most / d})
            for (int64_t o : {int64_t{-1}, int64_t{0}, int64_t{1}, d / 2, d - 1}) {
                const int64_t x = k * d + o;
                if (x >= 0 && x <= most && f.div(static_cast<int>(x)) != x / d)
                    return printf("%lld / %lld = %d\n", (long long)x, (long long)d, f.div(static_cast<int>(x))), 1;
            }
    }
    return 0;
}
"""


def test_ctas_and_divisions(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "sizes.cu", tmp_path / "sizes"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "weight_only_int4_group_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
