"""The waits of the kernels whose work is dealt out in line end at their limit by the clock: a kernel of one
warp waits for a barrier that nothing completes, and for a count that nothing raises."""
import ctypes as C
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "kvline.cuh"
using namespace eagle;
__global__ void wait_kernel(int which, long long limit, long long* cycles, unsigned* out) {
  __shared__ __align__(8) unsigned long long bar;
  __shared__ unsigned count;
  __shared__ volatile int gave_up;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    count = 5;
    gave_up = which == 3;                    // (another role of the CTA has given up)
    fence_mbar_init();
  }
  __syncwarp();
  const long long t0 = clock64();
  bool ok = true;
  if (which == 0) ok = kx_wait(smem_u32(&bar), 0, out + 1, &gave_up, limit);
  if (which == 1 || which == 3) ok = kx_wait<true>(smem_u32(&bar), 0, out + 1, &gave_up, limit);
  if (which == 2 && threadIdx.x == 0) ok = kx_wait_past(smem_u32(&count), 5, out + 1, &gave_up, limit);
  if (which == 4 && threadIdx.x == 0) ok = kx_wait_past(smem_u32(&count), 4, out + 1, &gave_up, limit);
  if (threadIdx.x == 0) {
    *cycles = clock64() - t0;
    out[0] = (ok ? 1u : 0u) | (gave_up ? 2u : 0u);
  }
}
extern "C" __attribute__((visibility("default"))) int wait_once(int which, long long limit, long long* cycles, unsigned* out) {
  wait_kernel<<<1, 32>>>(which, limit, cycles, out);
  return static_cast<int>(cudaDeviceSynchronize());
}
"""


@pytest.fixture(scope="module")
def wait(tmp_path_factory):
    from eagle_speculative_decoding_03_gb300 import build
    d = tmp_path_factory.mktemp("wait")
    src, so = str(d / "wait.cu"), str(d / "wait.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([build._nvcc(), *build.NVCC_FLAGS, "-I", build.CSRC, "-shared", "-cudart", "static", src, "-o", so], check=True)
    lib = C.CDLL(so)
    lib.wait_once.argtypes = [C.c_int, C.c_int64, C.c_void_p, C.c_void_p]

    def once(which, limit):
        cycles = torch.zeros(1, dtype=torch.int64, device="cuda")
        out = torch.zeros(2, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        assert lib.wait_once(which, limit, cycles.data_ptr(), out.data_ptr()) == 0
        return cycles.item(), out[0].item(), out[1].item()
    return once


@pytest.mark.parametrize("which", [0, 1, 2])
def test_a_wait_in_vain_ends_by_the_clock(wait, which):
    """Not before its limit and not long after (256 polls and sleeps more), with the error bit set."""
    for limit in (1_000_000, 20_000_000):            # 0.5 and 10 ms
        cycles, state, err = wait(which, limit)
        assert state == 2 and err == 1, (state, err)
        assert limit <= cycles <= 2 * limit + 200_000_000


def test_a_wait_ends_where_another_role_gave_up(wait):
    cycles, state, err = wait(3, 2_000_000_000)
    assert state == 2 and err == 0 and cycles < 200_000_000


def test_a_count_that_has_passed_is_not_waited_for(wait):
    cycles, state, err = wait(4, 2_000_000_000)
    assert state == 1 and err == 0 and cycles < 1_000_000
