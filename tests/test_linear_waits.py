"""What the products' kernels do when a bounded wait runs out: warps stay whole. The waits' helpers run
in a small program of their own; where the kernels use them is read from the sources."""
import os
import re
import subprocess

import pytest

from mixture_experts_layer_05_gb300 import build as build_mod

KERNELS = ("linear_stream.cu", "linear_pair.cu", "linear_fp8.cu")


def _source(name):
    with open(os.path.join(build_mod.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _heads(text, at):
    """The text in front of each open brace around position `at`."""
    depth, heads = 0, []
    for i in range(at - 1, -1, -1):
        if text[i] == "}":
            depth += 1
        elif text[i] == "{":
            depth -= 1
            if depth < 0:
                depth = 0
                heads.append(text[max(text.rfind(c, 0, i) for c in ";{}") + 1:i])
    return heads


@pytest.mark.parametrize("name", KERNELS)
def test_only_single_threads_wait_lane_by_lane(name):
    """A wait that gives up may tell the lanes of a warp different things. Whole warps wait with lin_wait,
    which brings them to one answer; the others are the elected threads that issue copies and MMAs."""
    text = _source(name)
    calls = [m for m in re.finditer(r"\b(wait_fast|wait_bounded)\w*\(", text)]
    assert calls
    for m in calls:
        assert any("lin_elect()" in h for h in _heads(text, m.start())), text[m.start():m.start() + 60]


WAITS = r"""
#include <cstdio>
#include "linear.cuh"
using namespace gbmoe;

// Even lanes wait for a phase that is complete, odd ones for one that nothing completes, with the CTA
// giving up already.
__global__ void lanes(int* out) {
  __shared__ alignas(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(smem_addr(&bar), 1);
    abort_flag = 1;
    fence_mbar_init();
  }
  __syncthreads();
  const int lane = threadIdx.x;
  const uint32_t parity = lane % 2 ? 0u : 1u;
  out[lane] = wait_fast(smem_addr(&bar), parity, &abort_flag, nullptr);
  __syncwarp();
  out[32 + lane] = lin_wait(smem_addr(&bar), parity, &abort_flag, nullptr);
  out[64 + lane] = lin_wait(smem_addr(&bar), 1u, &abort_flag, nullptr);
}

int main() {
  int* out;
  if (cudaMallocManaged(&out, 96 * sizeof(int)) != cudaSuccess) return 2;
  lanes<<<1, 32>>>(out);
  if (cudaDeviceSynchronize() != cudaSuccess) return 3;
  for (int i = 0; i < 96; ++i) printf("%d", out[i]);
  printf("\n");
}
"""


def _run(tmp_path, source):
    (tmp_path / "main.cu").write_text(source)
    subprocess.run([build_mod.nvcc()] + build_mod.flags() + ["-I", build_mod.CSRC, str(tmp_path / "main.cu"),
                                                             "-o", str(tmp_path / "main")], check=True)
    return subprocess.run([str(tmp_path / "main")], capture_output=True, text=True, check=True,
                          timeout=60).stdout.splitlines()


@pytest.mark.gpu
def test_a_warp_waits_as_one(cuda_lib, tmp_path):
    out, = _run(tmp_path, WAITS)
    assert out == "10" * 16 + "0" * 32 + "1" * 32
