"""What is asked of or set on a device once (host-only programs over csrc/internal.h)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_attention_prefill_tcgen05_gb300", "csrc")

PROGRAM = r"""
#include "internal.h"
int main()
{
    std::atomic<uint64_t> done{0};
    int calls = 0;
    cudaError_t answer = cudaSuccess;
    auto set = [&] { ++calls; return answer; };
    for (int dev : {0, 1, 0, 63, 1, 63})                // three devices: three calls
        if (idx::once_per_device(done, dev, set) != cudaSuccess)
            return 1;
    if (calls != 3)
        return 2;
    answer = cudaErrorMemoryAllocation;                  // a failure is returned, and not kept
    if (idx::once_per_device(done, 2, set) != answer || calls != 4)
        return 3;
    answer = cudaSuccess;
    if (idx::once_per_device(done, 2, set) != cudaSuccess || calls != 5)
        return 4;
    idx::once_per_device(done, 2, set);
    if (calls != 5)
        return 5;
    for (int dev : {64, 64, 200})                        // past the bits: every time
        idx::once_per_device(done, dev, set);
    return calls == 8 ? 0 : 6;
}
"""


ANSWERS = r"""
#include "internal.h"
int main()
{
    std::atomic<int> known{0};
    int calls = 0, answer = 0;
    auto ask = [&] { ++calls; return answer; };
    if (idx::remembered(known, ask) != 0 || idx::remembered(known, ask) != 0 || calls != 2)
        return 1;                                        // no answer is not one
    answer = -152;
    if (idx::remembered(known, ask) != -152 || calls != 3)
        return 2;
    answer = 7;
    return idx::remembered(known, ask) == -152 && calls == 3 ? 0 : 3;
}
"""


def run(program, tmp_path):
    include = "/usr/local/cuda/include"
    if shutil.which("g++") is None or not os.path.exists(os.path.join(include, "cuda_runtime.h")):
        pytest.skip("no host compiler or CUDA headers")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(program)
    subprocess.run(["g++", "-std=c++17", "-I" + CSRC, "-I" + include, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_a_device_that_comes_later_is_set_up_too(tmp_path):
    run(PROGRAM, tmp_path)


def test_a_device_that_could_not_be_asked_is_asked_again(tmp_path):
    run(ANSWERS, tmp_path)


def test_no_launch_keeps_a_device_attribute_for_the_process():
    """cudaFuncSetAttribute is called at every launch or under once_per_device, never for a static."""
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu"):
            lines = open(os.path.join(CSRC, name)).read().split("\n")
            for i, line in enumerate(lines):
                if "cudaFuncSetAttribute(" in line:
                    before = "\n".join(lines[max(0, i - 14):i])
                    assert "static const cudaError_t" not in before, f"{name}:{i + 1}"
