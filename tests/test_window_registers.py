"""What the window kernels' hosts check before they launch a kernel that divides its registers anew: the
kernel's own count, as the driver gives it.  The driver's answers are a fake's here."""

import os
import re
import subprocess

from differentiable_gaussian_splatting_gb300 import build

PROGRAM = r"""
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdio>

static int asked = 0, registers = 0;
static cudaError_t answer = cudaSuccess;
static cudaError_t fake_attributes(cudaFuncAttributes* a, const void*) {
    ++asked;
    a->numRegs = registers;
    return answer;
}
#define cudaFuncGetAttributes fake_attributes
#include "gs_attention.cuh"

int main() {
    std::atomic<bool> known{false};
    const auto check = [&](int regs, cudaError_t e) {
        registers = regs;
        answer = e;
        const cudaError_t got = gs::launch_registers_ok(nullptr, &known);
        std::printf("%d %d\n", (int)got, asked);
    };
    check(168, cudaErrorInitializationError);  // a failure that passes
    check(160, cudaSuccess);                   // shares that the launch does not have
    check(168, cudaSuccess);
    check(160, cudaErrorInitializationError);  // found good before: not asked again
    std::printf("%d %d\n", (int)cudaErrorInitializationError, (int)cudaErrorInvalidConfiguration);
}
"""


def test_a_failed_look_at_the_registers_is_not_kept(tmp_path):
    source, program = tmp_path / "registers.cu", tmp_path / "registers"
    source.write_text(PROGRAM)
    subprocess.run([build.nvcc(), "-std=c++17", "-O1", *build.ARCH, "-I", build.CSRC, "-I", build.INCLUDE,
                    str(source), "-o", str(program)], check=True, capture_output=True)
    out = subprocess.run([str(program)], check=True, capture_output=True, text=True).stdout
    *lines, (failed, refused) = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert lines == [(failed, 1), (refused, 2), (0, 3), (0, 3)]


def test_no_failure_is_kept_for_the_process():
    for name in os.listdir(build.CSRC):
        with open(os.path.join(build.CSRC, name)) as f:
            assert not re.search(r"static\s+(const\s+)?(cudaError_t|gs_status)\s+\w+\s*=", f.read()), name
