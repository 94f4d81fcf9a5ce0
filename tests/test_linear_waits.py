"""The products' waits: those for other CTAs acquire at the cluster's scope; and where a bounded wait runs
out, warps stay whole, and no CTA leaves before what is in flight has landed. The helpers run in small programs of their own; where the kernels use them is
read from the sources."""
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


def test_waits_for_other_ctas_acquire_at_their_scope():
    """Phases that another CTA of the cluster completes: all of the pairs', whose stages and accumulators are
    both CTAs', and the few-row kernel's partial sums (received; taken, so that the next may be sent)."""
    pair = _source("linear_pair.cu")
    assert re.findall(r"\b(wait_\w+|lin_wait)(<true>)?\(", pair) == [
        ("wait_fast_cluster", "")] * 3 + [("lin_wait", "<true>")]
    stream = _source("linear_stream.cu")
    waits = re.findall(r"\b(wait_\w+|lin_wait)(<true>)?\((\w+)", stream)
    assert {bar for _, across, bar in waits if across} == {"rfull_bar", "rempty_bar"}
    assert not {bar for _, across, bar in waits if not across} & {"rfull_bar", "rempty_bar"}


@pytest.mark.parametrize("name", KERNELS)
def test_kernels_end_by_lin_leave(name):
    """The last barrier in front of TMEM's release is the one that stays where a CTA gave up."""
    text = _source(name)
    end = re.findall(r"(\w+)\([^()]*\);\s*if \(warp == 1\) \{\s*tc_fence_after\(\);\s*tmem_dealloc", text)
    assert end == ["lin_leave"]


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


LEAVE = r"""
#include <cstdio>
#include "linear.cuh"
using namespace gbmoe;

// Warp 3 of the last CTA gives up, or none. Per CTA: its flag, and how long it stayed.
__global__ void leave(int C, int gives_up, unsigned long long* out) {
  __shared__ int abort_flag;
  if (threadIdx.x == 0) abort_flag = 0;
  if (C > 1) cluster_sync();
  else __syncthreads();
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  const unsigned long long t0 = globaltimer_ns();
  if (gives_up && rank == C - 1 && threadIdx.x == 100) abort_flag = 1;
  lin_leave(C, &abort_flag);
  const unsigned long long t1 = globaltimer_ns();
  if (threadIdx.x == 0) {
    out[2 * rank] = (unsigned long long)abort_flag;
    out[2 * rank + 1] = t1 - t0;
  }
}

int main() {
  unsigned long long* out;
  if (cudaMallocManaged(&out, 16 * sizeof(*out)) != cudaSuccess) return 2;
  for (int C : {1, 2, 8}) {
    for (int gives_up : {0, 0, 1}) {               // the first call loads the kernel
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(C);
      cfg.blockDim = dim3(160);
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = C;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      if (cudaLaunchKernelEx(&cfg, leave, C, gives_up, out) != cudaSuccess) return 3;
      if (cudaDeviceSynchronize() != cudaSuccess) return 4;
      printf("%d %d", C, gives_up);
      for (int i = 0; i < 2 * C; ++i) printf(" %llu", out[i]);
      printf("\n");
    }
  }
}
"""


@pytest.mark.gpu
def test_a_cluster_stays_where_one_gave_up(cuda_lib, tmp_path):
    lines = [[int(x) for x in l.split()] for l in _run(tmp_path, LEAVE)]
    assert len(lines) == 9
    for C, gave_up, *per in lines:
        assert per[::2] == [gave_up] * C
        # the timer ticks in steps of up to a few microseconds
        assert all(t > 990000 if gave_up else t < 900000 for t in per[1::2]), (C, gave_up, per)
