"""A launch that fails reports it and leaves no CUDA error behind: a pending one
would be taken for the next call's.  Host program linked with the library's
objects and with fakes of the runtime's calls, of which the first few work and
the others fail; nothing reaches a device."""
import glob
import os
import subprocess

from linear_layers_b200 import build as tpbuild

FAKED = ("cudaLaunchKernel", "cudaLaunchKernelExC", "cudaFuncSetAttribute", "cudaGetLastError",
         "cudaOccupancyMaxActiveClusters", "cudaGetDevice")

PROGRAM = r"""
#include <cstdio>
#include <cuda_runtime.h>
#include "internal.h"
using namespace tpl;

int works = 0;                               // so many calls still work
cudaError_t pending = cudaSuccess;
bool failed = false;
cudaError_t answer() {
  if (works-- > 0) return cudaSuccess;
  failed = true;
  return pending = cudaErrorLaunchOutOfResources;
}
extern "C" {
cudaError_t __wrap_cudaLaunchKernel(const void*, dim3, dim3, void**, size_t, cudaStream_t) { return answer(); }
cudaError_t __wrap_cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) { return answer(); }
cudaError_t __wrap_cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return answer(); }
cudaError_t __wrap_cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
  *n = 64;
  return cudaSuccess;
}
cudaError_t __wrap_cudaGetDevice(int* dev) { return *dev = 0, cudaSuccess; }
cudaError_t __wrap_cudaGetLastError() {
  const cudaError_t e = pending;
  pending = cudaSuccess;
  return e;
}
}

int bad = 0;
template <typename F>
void check(const char* what, F call) {
  for (int n = 0;; ++n) {
    works = n;
    failed = false;
    const tp_status s = call();
    if (s != (failed ? TP_ERR_CUDA : TP_OK) || pending != cudaSuccess) {
      std::printf("%s, %d calls work: status %d, pending error %d\n", what, n, int(s), int(pending));
      pending = cudaSuccess;
      ++bad;
    }
    if (!failed) return;
  }
}

int main() {
  void* p = reinterpret_cast<void*>(1 << 20);   // never dereferenced: nothing is launched
  float* f = static_cast<float*>(p);
  check("loss_sum", [&] { return loss_sum_launch(f, 4, f, nullptr); });
  check("loss_sum, early", [&] { return loss_sum_launch(f, 4, f, nullptr, true); });
  for (int dt = 0; dt < 2; ++dt) {
    const tp_dtype t = static_cast<tp_dtype>(dt);
    LogprobsArgs l = {};
    l.logits = p; l.T = 4; l.v = 300; l.scale = 1.0f; l.lse = f;
    check("logprobs_fwd", [&] { return logprobs_fwd_launch(l, t, nullptr); });
    l.top_k = 3; l.top_idx = static_cast<int32_t*>(p); l.top_logprob = f;
    check("logprobs_fwd, top", [&] { return logprobs_fwd_launch(l, t, nullptr); });
    LogprobsBwdArgs b = {};
    b.logits = p; b.lse = f; b.dentropy = f; b.entropy = f; b.T = 4; b.v = 300; b.scale = 1.0f; b.dlogits = p;
    check("logprobs_bwd", [&] { return logprobs_bwd_launch(b, t, t, nullptr); });
    DistillArgs d = {};
    d.logits = p; d.ids = static_cast<int32_t*>(p); d.teacher = f; d.T = 4; d.v = 300; d.K = 8;
    d.scale = d.grad_scale = 1.0f; d.loss = f;
    check("distill, loss alone", [&] { return distill_launch(d, t, t, f, p, nullptr); });
    d.dlogits = p;
    check("distill", [&] { return distill_launch(d, t, t, f, p, nullptr); });
  }
  check("few tokens", [&] {
    return linear_logprobs_few_launch(p, p, nullptr, 1, 64, 300, 1.0f, f, f, f, f, nullptr);
  });
  check("combine", [&] {
    return linear_logprobs_combine_launch(f, f, f, f, nullptr, 1, 300, 10, 1.0f, f, f, f, nullptr, nullptr);
  });
  return bad != 0;
}
"""


def test_no_error_is_left_pending(tmp_path):
    tpbuild.build()
    src, exe = tmp_path / "launches.cu", tmp_path / "launches"
    src.write_text(PROGRAM)
    objects = sorted(glob.glob(os.path.join(tpbuild.BUILD, "*.o")))
    wraps = [a for name in FAKED for a in ("-Xlinker", f"--wrap={name}")]
    subprocess.run([tpbuild._nvcc(), *tpbuild.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-cudart",
                    "static", "-I", tpbuild.CSRC, "-I", tpbuild.INCLUDE, str(src), *objects, *wraps,
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
