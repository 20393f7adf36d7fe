"""The launches of a few tokens' experts on devices of any size, without one: kmr_moe_small.cu compiled with its launch call replaced."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <cuda_runtime.h>
static cudaError_t seen(const cudaLaunchConfig_t* c, const void*, void**) {
    std::printf(" %u %u %zu", c->gridDim.x, c->blockDim.x, c->dynamicSmemBytes);
    return cudaSuccess;
}
#define cudaLaunchKernelExC seen
#include "kmr_moe_small.cu"
int main(int, char** a) {
    kmr::MoeSmallParams p = {};
    p.w.E = std::atoi(a[1]), p.w.H = std::atoi(a[2]), p.w.I = std::atoi(a[3]), p.T = std::atoi(a[4]), p.k = std::atoi(a[5]);
    for (const int sms : {1, 16, 64, 127, 128, 148, 152, 160})
        for (const bool bf16 : {false, true}) {
            std::printf("%d %d", sms, int(kmr::moe_small_fits(p.w, bf16, p.T, p.k)));
            std::printf(" %d\n", int(kmr::launch_moe_small(p, bf16, sms, nullptr)));
        }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    nvcc = os.environ.get("NVCC") or ("/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else shutil.which("nvcc"))
    if not nvcc:
        pytest.skip("no nvcc")
    d = tmp_path_factory.mktemp("launch")
    (d / "main.cu").write_text(PROGRAM)
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"),
                        "-I", os.path.join(ROOT, "int4_weight_only_group_gb300", "csrc"), str(d / "main.cu"), "-o", str(d / "main")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(d / "main")


@pytest.mark.parametrize("E,H,I,T,k", [(128, 2048, 768, 1, 8), (1, 128, 128, 1, 1), (1024, 4096, 1024, 4, 3), (60, 2048, 1408, 4, 4)])
def test_every_number_of_sms_is_served(program, E, H, I, T, k):
    """A call that takes the few-token form is launched whatever the device: its shared memory is planned for 128 CTAs at once, and fewer SMs
    run them in turn."""
    r = subprocess.run([program, *map(str, (E, H, I, T, k))], capture_output=True, text=True)
    assert r.returncode == 0
    lines = r.stdout.splitlines()
    assert len(lines) == 16
    work = min(T * k, E) * (I // 8)
    for line in lines:
        sms, fits, g0, t0, m0, g1, t1, m1, rc = map(int, line.split())
        assert fits and rc == 0
        assert g0 == min(work, max(sms, 128)) and g1 == H // 16 and t0 == t1 == 1024
        assert max(m0, m1) <= 227 * 1024 - 512
