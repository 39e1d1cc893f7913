// Decode attention over the paged 4-bit cache: one warp a (request, query
// head), one position at a time, four values of K and V a lane.
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "spc_device.cuh"
#include "spc_internal.h"

namespace spc {

__global__ void __launch_bounds__(32) kv4_attn_kernel(Kv4AttnCall a) {
  const int lane = threadIdx.x, b = blockIdx.x / a.n_q, h = blockIdx.x % a.n_q, G = a.n_q / a.n_kv, g = h / G;
  const uint2 qw = *reinterpret_cast<const uint2*>(a.q + (size_t)blockIdx.x * kD + 4 * lane);
  const float q0 = bf_lo(qw.x), q1 = bf_hi(qw.x), q2 = bf_lo(qw.y), q3 = bf_hi(qw.y);
  const int L = max(0, min(a.len[b], a.max_blocks << a.block_shift));
  const int n = a.selected ? a.budget : L;
  const int32_t* sel = a.selected ? a.selected + ((size_t)b * a.n_kv + g) * a.budget : nullptr;
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
  for (int i = 0; i < n; ++i) {
    const int p = sel ? sel[i] : i;
    if (p < 0 || p >= L) continue;
    const int blk = a.table[(size_t)b * a.max_blocks + (p >> a.block_shift)];
    if (blk < 0 || blk >= a.num_blocks) continue;
    const uint8_t* rec = a.cache + ((((size_t)blk * a.n_kv + g) << a.block_shift) + (p & ((1 << a.block_shift) - 1))) * kKv4Rec;
    uint32_t kh[4], vh[4];
    const uint32_t kc = *reinterpret_cast<const uint16_t*>(rec + 2 * lane);
    const uint32_t vc = *reinterpret_cast<const uint16_t*>(rec + kKv4V + 2 * lane);
    e2m1x8_to_f16(kc | vc << 16, kh);
    const uint32_t ks = e4m3_dup_f16(rec[kKv4Scale + (lane >> 2)]), vs = e4m3_dup_f16(rec[kKv4Scale + 8 + (lane >> 2)]);
    vh[0] = hmul2(kh[2], vs);
    vh[1] = hmul2(kh[3], vs);
    kh[0] = hmul2(kh[0], ks);
    kh[1] = hmul2(kh[1], ks);
    const float x = a.scale2 * warp_sum(q0 * f16_lo(kh[0]) + q1 * f16_hi(kh[0]) + q2 * f16_lo(kh[1]) + q3 * f16_hi(kh[1]));
    const float M = fmaxf(m, x);
    const float c = exp2f(m - M), e = exp2f(x - M);
    l = l * c + e;
    o0 = o0 * c + e * f16_lo(vh[0]);
    o1 = o1 * c + e * f16_hi(vh[0]);
    o2 = o2 * c + e * f16_lo(vh[1]);
    o3 = o3 * c + e * f16_hi(vh[1]);
    m = M;
  }
  const float r = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(a.out + (size_t)blockIdx.x * kD + 4 * lane) =
      make_uint2(pack_bf16(o0 * r, o1 * r), pack_bf16(o2 * r, o3 * r));
}

size_t kv4_attn_workspace(int, int, int, int, int, int) { return 256; }

int kv4_attn_launch(const Kv4AttnCall& c, void*, void* stream) {
  kv4_attn_kernel<<<c.B * c.n_q, 32, 0, static_cast<cudaStream_t>(stream)>>>(c);
  return cudaGetLastError() == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

}  // namespace spc
