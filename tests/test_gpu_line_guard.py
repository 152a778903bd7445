"""A CTA of the kernels dealt out in line whose shared memory lies off the tiles' alignment gives up: the
call is flagged, and what the join reads of the CTA is an empty cut, not what the workspace held."""
import ctypes as C
import subprocess

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "kvline.cuh"
using namespace eagle;
__global__ void guard(unsigned ring, float* parts, unsigned* err, int* gave_up) {
  if (misplaced(ring, parts, err) && threadIdx.x == 0) gave_up[blockIdx.x] = 1;
}
extern "C" __attribute__((visibility("default"))) int cut_bytes() { return static_cast<int>(sizeof(Cut)); }
extern "C" __attribute__((visibility("default"))) int run_guard(unsigned ring, float* parts, unsigned* err, int* gave_up) {
  guard<<<4, 64>>>(ring, parts, err, gave_up);
  return static_cast<int>(cudaDeviceSynchronize());
}
"""


def test_a_misplaced_ring_leaves_empty_cuts(tmp_path):
    from eagle_speculative_decoding_03_gb300 import build
    src, so = str(tmp_path / "guard.cu"), str(tmp_path / "guard.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([build._nvcc(), *build.NVCC_FLAGS, "-I", build.CSRC, "-shared", "-cudart", "static", src, "-o", so], check=True)
    lib = C.CDLL(so)
    lib.run_guard.argtypes = [C.c_uint32, C.c_void_p, C.c_void_p, C.c_void_p]
    words = lib.cut_bytes() // 4
    for ring, bad in ((0, 0), (1024, 0), (100 * 1024, 0), (16, 1), (1024 + 512, 1)):
        parts = torch.full((4, words), 7, dtype=torch.int32, device="cuda")
        err, gave_up = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        assert lib.run_guard(ring, parts.data_ptr(), err.data_ptr(), gave_up.data_ptr()) == 0
        assert (gave_up == bad).all() and err.item() == bad
        assert (parts[:, 0] == (0 if bad else 7)).all()      # `last`: 0 is an empty cut
