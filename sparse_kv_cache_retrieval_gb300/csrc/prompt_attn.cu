// Causal attention over packed prompts: one warp a (row, query head), one key
// at a time, four values of a row a lane.
#include <cuda_runtime.h>

#include "spc_device.cuh"
#include "spc_internal.h"

namespace spc {

__global__ void __launch_bounds__(128) prompt_attn_kernel(PromptAttnCall a) {
  const int lane = threadIdx.x & 31;
  const long long n = (long long)a.T * a.n_q, warps = (long long)gridDim.x * 4;
  for (long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5); w < n; w += warps) {
    const int t = (int)(w / a.n_q), h = (int)(w % a.n_q), g = h / (a.n_q / a.n_kv);
    int first = -1;
    for (int b = 0; b < a.B; ++b) {
      const int s = max(0, min(a.cu[b], a.T)), e = max(s, min(a.cu[b + 1], a.T));
      if (t >= s && t < e) first = s;
    }
    if (first < 0) continue;
    const uint2 qw = *reinterpret_cast<const uint2*>(a.q + t * a.q_stride + (size_t)h * kD + 4 * lane);
    const float q0 = bf_lo(qw.x), q1 = bf_hi(qw.x), q2 = bf_lo(qw.y), q3 = bf_hi(qw.y);
    float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
    for (int j = first; j <= t; ++j) {
      const uint2 k = *reinterpret_cast<const uint2*>(a.k + j * a.k_stride + (size_t)g * kD + 4 * lane);
      const uint2 v = *reinterpret_cast<const uint2*>(a.v + j * a.v_stride + (size_t)g * kD + 4 * lane);
      const float x = a.scale2 * warp_sum(q0 * bf_lo(k.x) + q1 * bf_hi(k.x) + q2 * bf_lo(k.y) + q3 * bf_hi(k.y));
      const float M = fmaxf(m, x);
      const float c = m == -INFINITY ? 0.f : exp2f(m - M), e = exp2f(x - M);
      l = l * c + e;
      o0 = o0 * c + e * bf_lo(v.x);
      o1 = o1 * c + e * bf_hi(v.x);
      o2 = o2 * c + e * bf_lo(v.y);
      o3 = o3 * c + e * bf_hi(v.y);
      m = M;
    }
    const float r = 1.f / l;
    *reinterpret_cast<uint2*>(a.out + ((size_t)t * a.n_q + h) * kD + 4 * lane) =
        make_uint2(pack_bf16(o0 * r, o1 * r), pack_bf16(o2 * r, o3 * r));
  }
}

size_t prompt_attn_workspace(int, int, int, int) { return 256; }

int prompt_attn_launch(const PromptAttnCall& c, void*, void* stream) {
  const long long n = ((long long)c.T * c.n_q + 3) / 4;
  prompt_attn_kernel<<<(int)(n < 152 * 64 ? n : 152 * 64), 128, 0, static_cast<cudaStream_t>(stream)>>>(c);
  return cudaGetLastError() == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

}  // namespace spc
