"""A kernel that lets its dependents start at once and then runs longer than the limit of the
kernels' waits (one second): products behind it under PDL wait for it without giving up."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import handle
from test_gpu_fp4 import bound, mx, on_gpu, operand  # noqa: F401

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include <cstdint>
// One block that releases its dependents, spins for `ns` of the global timer, then copies n words.
__global__ void slow(const uint32_t* in, uint32_t* out, int n, uint64_t ns) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  do {
    __nanosleep(1000);
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  } while (t - t0 < ns);
  for (int i = threadIdx.x; i < n; i += blockDim.x) out[i] = in[i];
}
extern "C" int run_slow(const void* in, void* out, int n, unsigned long long ns, void* stream) {
  slow<<<1, 256, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<const uint32_t*>(in), static_cast<uint32_t*>(out), n, ns);
  return cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def slow(tmp_path_factory):
    d = tmp_path_factory.mktemp("slow")
    (d / "slow.cu").write_text(SOURCE)
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-shared", "-Xcompiler", "-fPIC",
                    "-o", str(d / "slow.so"), str(d / "slow.cu")], check=True)
    lib = ctypes.CDLL(str(d / "slow.so"))
    lib.run_slow.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_ulonglong, ctypes.c_void_p]
    return lib


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("m,n,k,splits", [(48, 32768, 2048, False), (300, 8192, 2048, False), (300, 8320, 2048, False),
                                          (16, 1024, 16384, True)])
def test_products_outwait_it(mx, slow, m, n, k, splits, fp4):  # noqa: F811
    """In each form of the kernels (two CTAs to an SM, pairs, one to an SM, K split) the ring is
    shorter than K; the activation comes from the slow kernel."""
    plan = mx.mx_plan_gemm_fp4(m, n, k, fp4_activations=fp4, pdl=True)
    chunks = k // (256 if fp4 else 128)
    assert (plan["splits"] > 1) == splits and plan["stages"] * plan["splits"] < chunks
    rng = np.random.default_rng(m + n)
    aq, as_, av = operand(rng, m, k, fp4)
    wq, ws, wv = operand(rng, n, k, True)
    source, a = on_gpu(aq), torch.zeros(aq.shape, dtype=torch.uint8, device="cuda:0")
    args = [a, on_gpu(oracle.swizzle_scales(as_)), on_gpu(wq), on_gpu(oracle.swizzle_scales(ws))]
    out = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda:0")
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    assert slow.run_slow(source.data_ptr(), a.data_ptr(), aq.size // 4, 1_400_000_000, stream) == 0
    mx.mx_gemm_fp4(handle(), *args, out=out, pdl=True)
    assert mx.mx_device_status(handle()) == mx.MX_OK
    ref = av @ wv.T
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound(av, wv, ref)).all(), (err / bound(av, wv, ref)).max()
