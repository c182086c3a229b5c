"""What moe_tree_attention answers when its launch is refused (no GPU: the C entry beside fakes of what it calls)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mxfp4_mixture_experts_route_gb300", "csrc")

FAKES = r'''
#include "kv_abi.cu"
#include <stdio.h>

namespace moe {
static cudaError_t g_launch;
int check_device() { return MOE_OK; }
int cuda_rc(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
cudaError_t launch_kv_plan(const KvDims&, const PlanArgs&, cudaStream_t) { return g_launch; }
cudaError_t launch_kv_append(const KvDims&, const AppendArgs&, cudaStream_t) { return g_launch; }
cudaError_t launch_tree_attn(const KvDims&, const AttnArgs&, cudaStream_t) { return g_launch; }
size_t tree_attn_ws_bytes(const KvDims&) { return 4096; }
}  // namespace moe

int main() {
    moe_kv_shape s = {};
    s.B = 1, s.T = 1, s.Hq = 1, s.Hkv = 1, s.D = 64, s.page = 16, s.n_pages = 4, s.max_pages = 4, s.scale = 1.f;
    void* p = (void*)0x10000;
    for (cudaError_t e : {cudaSuccess, cudaErrorNotSupported, cudaErrorCooperativeLaunchTooLarge, cudaErrorInvalidValue}) {
        moe::g_launch = e;
        printf("%d\n", moe_tree_attention(&s, p, p, p, (int32_t*)p, (int32_t*)p, (int32_t*)p, nullptr, nullptr, nullptr, p,
                                          nullptr, p, 4096, nullptr));
    }
}
'''


def test_too_few_multiprocessors_have_a_code_of_their_own(tmp_path):
    import mxfp4_mixture_experts_route_gb300 as moe
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src = tmp_path / "fakes.cu"
    src.write_text(FAKES)
    exe = str(tmp_path / "fakes")
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                        "-I", CSRC, str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0
    assert [int(x) for x in out.stdout.split()] == [moe.MOE_OK, moe.MOE_ERR_NO_DEVICE, moe.MOE_ERR_NO_DEVICE,
                                                    moe.MOE_ERR_CUDA]
