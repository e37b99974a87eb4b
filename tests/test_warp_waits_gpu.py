"""The bounded wait of a whole warp (GPU): one answer for all lanes, also where the wait runs out at
about the time that the barrier completes.  The wait is compiled from the library's own header into
a small library of its own."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from bit_paged_kv_diag_b200 import build

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "kvq_ptx.cuh"
using namespace kvq;
// Warp 0 waits `limit` ns for a barrier at which warp 1 arrives after delay * blockIdx.x ns (never:
// delay < 0).  answers: [blocks][32], one a lane.  Every loop ends.
__global__ void __launch_bounds__(64) waits(int* answers, long long limit, long long delay) {
  __shared__ __align__(8) unsigned long long bar_mem;
  const unsigned bar = smem_addr(&bar_mem);
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    answers[blockIdx.x * 32 + threadIdx.x] = mbar_wait_warp(bar, 0u, limit);
  } else if (threadIdx.x == 32 && delay >= 0) {
    const unsigned long long t0 = global_timer_ns();
    const unsigned long long stop = static_cast<unsigned long long>(delay) * blockIdx.x;
    for (int i = 0; i < 1000000 && global_timer_ns() - t0 < stop; i++) {}
    mbar_arrive(bar);
  }
  __syncthreads();
}
extern "C" __attribute__((visibility("default"))) int run_waits(int* answers, int blocks, long long limit, long long delay) {
  waits<<<blocks, 64>>>(answers, limit, delay);
  return cudaDeviceSynchronize();
}
"""


def test_all_lanes_get_the_same_answer(tmp_path):
    import torch
    src, so = tmp_path / "waits.cu", tmp_path / "waits.so"
    src.write_text(SOURCE)
    subprocess.run([build._nvcc(), *build.NVCC_FLAGS, "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"),
                    "-shared", "-o", str(so), str(src)], check=True)
    run = ctypes.CDLL(str(so)).run_waits
    run.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_longlong]
    blocks = 2048
    answers = torch.full((blocks, 32), 7, dtype=torch.int32, device="cuda")
    # Nothing arrives: every wait runs out, and the context stays usable.
    assert run(answers.data_ptr(), blocks, 20000, -1) == 0
    assert not answers.any()
    # Arrivals from long before to long after the limit.
    for _ in range(5):
        assert run(answers.data_ptr(), blocks, 200000, 200) == 0
        a = answers.cpu().numpy()
        assert (a == a[:, :1]).all() and np.isin(a, (0, 1)).all()
        assert a[0].all() and not a[-1].any()
