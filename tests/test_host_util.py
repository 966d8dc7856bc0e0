"""Host-side helpers of the kernels' launches (csrc/host_util.h), against a runtime whose calls
fail on request: no GPU and no CUDA runtime is involved."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "host_util.h"
#include <cstdio>

static int calls = 0;
static cudaError_t answer = cudaSuccess;
extern "C" cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  ++calls;
  if (answer == cudaSuccess) a->numRegs = 128;
  return answer;
}
static void kernel(int) {}
static int failed = 0;
static void expect(bool ok, const char* what) {
  if (!ok) std::printf("%s\n", what), failed = 1;
}

int main() {
  mattn::KernelRegs r;
  int n = -1;
  answer = cudaErrorMemoryAllocation;
  expect(r.get(kernel, n) == cudaErrorMemoryAllocation, "a failed question's error is returned");
  answer = cudaErrorNoDevice;
  expect(r.get(kernel, n) == cudaErrorNoDevice, "each time its own");
  answer = cudaSuccess;
  expect(r.get(kernel, n) == cudaSuccess && n == 128, "a failure is not remembered");
  expect(calls == 3, "asked again after a failure");
  answer = cudaErrorNoDevice;
  n = -1;
  expect(r.get(kernel, n) == cudaSuccess && n == 128 && calls == 3, "an answer is remembered");
  return failed;
}
"""


def test_a_failed_question_for_registers_is_asked_again(tmp_path):
    """A transient failure must not refuse a kernel for the rest of the process, nor hide its
    error."""
    from masked_attention_gb300 import _build
    nvcc = os.path.realpath(_build.nvcc())
    include = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    if not os.path.exists(os.path.join(include, "cuda_runtime.h")) or not shutil.which("g++"):
        pytest.skip("no CUDA headers or g++")
    src, exe = tmp_path / "regs.cpp", tmp_path / "regs"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I", include, "-I", _build.CSRC, str(src), "-o",
                        str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_no_launch_keeps_a_failed_question():
    """Every register question goes through the helper that forgets failures."""
    users = []
    for name in sorted(os.listdir(os.path.join(ROOT, "masked_attention_gb300", "csrc"))):
        with open(os.path.join(ROOT, "masked_attention_gb300", "csrc", name)) as f:
            if "cudaFuncGetAttributes" in f.read():
                users.append(name)
    assert users == ["host_util.h"]
