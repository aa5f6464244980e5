"""The feed-forward kernels behind a kernel that lets its successor start at once and then runs on for longer than the
deadline of any wait inside a kernel (2 s): no such wait may be counting while the kernel in front still runs."""
import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# 32 threads that signal and sleep for 2.6 s in steps of at most 1 ms, at most 20,000 of them
SRC = r'''
#include <cstdint>
__global__ void hold() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  for (int i = 0; i < 20000; ++i) {
    __nanosleep(500000);
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (t - t0 > 2600000000ull) break;
  }
}
extern "C" int launch_hold(void* stream) {
  hold<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>();
  return static_cast<int>(cudaGetLastError());
}
'''


@pytest.fixture(scope="module")
def hold(tmp_path_factory):
    from mixture_experts_layer_build_gb300 import build
    d = tmp_path_factory.mktemp("hold")
    src, lib = d / "hold.cu", d / "libhold.so"
    src.write_text(SRC)
    cudalib = os.path.join(os.path.dirname(os.path.dirname(build.NVCC)), "lib64")
    subprocess.run([build.NVCC, *build.ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC", "-cudart", "shared", "-Xlinker",
                    f"-rpath,{cudalib}", str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).launch_hold
    f.argtypes = [ctypes.c_void_p]
    return f


@pytest.mark.parametrize("T,H,I", [(20, 1024, 512), (200, 1024, 512), (1500, 1024, 512)])  # tile kernel (split or not), pairs
def test_no_wait_counts_while_the_kernel_in_front_runs(hold, T, H, I):
    from mixture_experts_layer_build_gb300 import mok
    g = torch.Generator(device="cuda").manual_seed(T)
    x, wg, wu, wd, dy = ((torch.randn(s, generator=g, device="cuda") * 0.05).to(BF)
                         for s in ((T, H), (I, H), (I, H), (H, I), (T, H)))
    want, plan = mok.FFN(T, H, I), mok.FFN(T, H, I)
    want.forward(x, wg, wu, wd)
    want.backward(x, wg, wu, wd, dy)
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    assert hold(stream) == 0
    plan.forward(x, wg, wu, wd)
    assert hold(stream) == 0
    plan.backward(x, wg, wu, wd, dy)
    torch.cuda.synchronize()
    assert plan.device_status() == 0
    assert torch.equal(plan.out, want.out)
    assert all(torch.equal(a, b) for a, b in zip(vars(plan.grads).values(), vars(want.grads).values()))
