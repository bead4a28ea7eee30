"""The kernels' bounded wait on an mbarrier: one that nobody arrives on gives up, says so in the error
word, and leaves a larger error that is there already.  A one-warp kernel around the wait itself."""
import ctypes
import os
import subprocess

import pytest

import sparse_moe_02_gb300 as moe
from sparse_moe_02_gb300 import build

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "ptx.cuh"

__global__ void wait_kernel(int* err, int* done) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) moe::mbar_init(&bar, 1);
  moe::fence_mbar_init();
  __syncwarp();
  done[0] = moe::mbar_wait(&bar, 0, err);  // nobody arrives
  if (threadIdx.x == 0) moe::mbar_arrive(&bar);
  __syncwarp();
  done[1] = moe::mbar_wait(&bar, 0, err);
}

extern "C" int run_wait(int* err, int* done) {
  wait_kernel<<<1, 32>>>(err, done);
  return (int)cudaDeviceSynchronize();
}
"""


@pytest.fixture(scope="module")
def run_wait(tmp_path_factory):
    at = tmp_path_factory.mktemp("wait")
    (at / "wait.cu").write_text(SOURCE)
    subprocess.run(["nvcc", *build.FLAGS, *build.ARCH, "-shared", "-o", str(at / "wait.so"),
                    str(at / "wait.cu")], check=True)
    fn = ctypes.CDLL(os.path.join(str(at), "wait.so")).run_wait
    fn.argtypes, fn.restype = [ctypes.c_void_p] * 2, ctypes.c_int
    return fn


@pytest.mark.parametrize("before", [moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_DEVICE,
                                    moe.MOE_ERR_NO_MEMORY])
def test_an_expired_wait_leaves_the_larger_error(run_wait, before):
    import torch
    err = torch.tensor([before], dtype=torch.int32, device="cuda")
    done = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert run_wait(err.data_ptr(), done.data_ptr()) == 0
    assert done.tolist() == [0, 1]
    assert err.item() == max(before, moe.MOE_ERR_TIMEOUT)
