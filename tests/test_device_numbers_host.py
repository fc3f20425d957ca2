"""What the launch code keeps of the runtime's answers: for each device, and no failed answer (no GPU)."""
import subprocess

from moe_task_scheduling_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include "et_api.h"
int main() {
    static et::DeviceNumbers<3> n;
    int asked = 0, v = -1, bad = 0;
    auto answer = [&](int what, cudaError_t e) { return [&asked, what, e](int* out) { ++asked; *out = what; return e; }; };
    bad |= n.get(0, 1, &v, answer(19, cudaErrorInvalidValue)) != cudaErrorInvalidValue;  // fails: not kept
    bad |= (n.get(0, 1, &v, answer(38, cudaSuccess)) != cudaSuccess || v != 38) << 1;
    bad |= (n.get(0, 1, &v, answer(5, cudaSuccess)) != cudaSuccess || v != 38) << 2;     // kept
    bad |= (n.get(1, 1, &v, answer(5, cudaSuccess)) != cudaSuccess || v != 5) << 3;      // of its own for each device
    bad |= (n.get(63, 2, &v, answer(0, cudaSuccess)) != cudaSuccess || v != 0) << 4;     // 0 is an answer too
    bad |= (n.get(63, 2, &v, answer(7, cudaSuccess)) != cudaSuccess || v != 0) << 5;
    bad |= (n.get(0, 2, &v, answer(7, cudaSuccess)) != cudaSuccess || v != 7) << 6;
    bad |= (asked != 5) << 7;
    std::printf("%d\n", bad);
    return bad;
}
"""


def test_kept_for_each_device_and_only_when_right(tmp_path):
    src, exe = tmp_path / "n.cu", tmp_path / "n"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I", build.CSRC, "-o", str(exe), str(src)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout.strip() == "0"
