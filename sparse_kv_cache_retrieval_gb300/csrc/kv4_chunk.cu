// Attention of chunks of new tokens over the paged 4-bit cache:
// out_i = sum_{p <= P_i} softmax_p(scale q_i.K_p) V_p, P_i = len - n + i.
// One warp a (row, query head), one position at a time.
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "spc_device.cuh"
#include "spc_internal.h"

namespace spc {

__global__ void __launch_bounds__(256) kv4_chunk_kernel(const Kv4ChunkCall c) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = (int)(w / c.n_q), h = (int)(w - (long long)t * c.n_q), g = h / (c.n_q / c.n_kv);
  if (t >= c.T) return;
  int b = 0;
  while (b < c.B && !(t >= c.cu[b] && t < c.cu[b + 1])) ++b;
  if (b == c.B) return;
  const int L = max(0, min(c.len[b], c.max_blocks << c.block_shift)), P = L - (c.cu[b + 1] - t);
  const uint2 qw = *reinterpret_cast<const uint2*>(c.q + t * c.q_stride + (size_t)h * kD + 4 * lane);
  const float q[4] = {bf_lo(qw.x), bf_hi(qw.x), bf_lo(qw.y), bf_hi(qw.y)};
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  bool any = false;
  for (int p = 0; p <= P; ++p) {
    const int blk = c.table[(size_t)b * c.max_blocks + (p >> c.block_shift)];
    if ((unsigned)blk >= (unsigned)c.num_blocks) continue;
    const int bs = 1 << c.block_shift;
    const uint8_t* r = c.cache + (((size_t)blk * c.n_kv + g) * bs + (p & (bs - 1))) * kKv4Rec;
    uint32_t k[4], v[4];
    e2m1x8_to_f16(*reinterpret_cast<const uint16_t*>(r + 2 * lane), k);
    e2m1x8_to_f16(*reinterpret_cast<const uint16_t*>(r + kKv4V + 2 * lane), v);
    const float ks = f16_lo(e4m3_dup_f16(r[kKv4Scale + lane / 4])), vs = f16_lo(e4m3_dup_f16(r[kKv4Scale + 8 + lane / 4]));
    const float x = warp_sum(q[0] * (f16_lo(k[0]) * ks) + q[1] * (f16_hi(k[0]) * ks) + q[2] * (f16_lo(k[1]) * ks) +
                             q[3] * (f16_hi(k[1]) * ks)) * c.scale * kLog2e;
    any = true;
    const float M = fmaxf(m, x), al = m == M ? 1.f : exp2f(m - M), e = exp2f(x - M);
    m = M;
    l = l * al + e;
    o[0] = o[0] * al + e * (f16_lo(v[0]) * vs);
    o[1] = o[1] * al + e * (f16_hi(v[0]) * vs);
    o[2] = o[2] * al + e * (f16_lo(v[1]) * vs);
    o[3] = o[3] * al + e * (f16_hi(v[1]) * vs);
  }
  const float r = any ? 1.f / l : 0.f;
  *reinterpret_cast<uint2*>(c.out + ((size_t)t * c.n_q + h) * kD + 4 * lane) =
      make_uint2(pack_bf16(o[0] * r, o[1] * r), pack_bf16(o[2] * r, o[3] * r));
  if (c.lse && lane == 0) c.lse[(size_t)t * c.n_q + h] = any ? (m + log2f(l)) / kLog2e : -INFINITY;
}

size_t kv4_chunk_workspace(int, int, int, int) { return 256; }

int kv4_chunk_launch(const Kv4ChunkCall& c, void*, void* stream) {
  const long long blocks = ((long long)c.T * c.n_q + 7) / 8;
  kv4_chunk_kernel<<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(c);
  return cudaGetLastError() == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

}  // namespace spc
