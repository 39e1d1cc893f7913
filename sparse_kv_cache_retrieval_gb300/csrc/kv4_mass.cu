// The attention weight that the positions of the paged 4-bit cache receive from
// chunks of new tokens: mass_p = keep prev_p + sum_i exp(scale q_i.K_p - lse_i).
// One warp a (request, KV head, position), one row at a time.
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "spc_device.cuh"
#include "spc_internal.h"

namespace spc {

__global__ void __launch_bounds__(256) kv4_mass_kernel(const Kv4ChunkCall c) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y / c.n_kv, g = blockIdx.y - b * c.n_kv, G = c.n_q / c.n_kv;
  const int L = max(0, min(c.len[b], c.max_blocks << c.block_shift)), bs = 1 << c.block_shift;
  const int t0 = max(0, min(c.cu[b], c.T)), n = max(t0, min(c.cu[b + 1], c.T)) - t0;
  for (int p = blockIdx.x * 8 + (threadIdx.x >> 5); p < L; p += gridDim.x * 8) {
    const int blk = c.table[(size_t)b * c.max_blocks + (p >> c.block_shift)];
    float sum = 0.f;
    if ((unsigned)blk < (unsigned)c.num_blocks) {
      const uint8_t* r = c.cache + (((size_t)blk * c.n_kv + g) * bs + (p & (bs - 1))) * kKv4Rec;
      uint32_t kw[4];
      e2m1x8_to_f16(*reinterpret_cast<const uint16_t*>(r + 2 * lane), kw);
      const float ks = f16_lo(e4m3_dup_f16(r[kKv4Scale + lane / 4]));
      const float k[4] = {f16_lo(kw[0]) * ks, f16_hi(kw[0]) * ks, f16_lo(kw[1]) * ks, f16_hi(kw[1]) * ks};
      float part = 0.f;                                // of 16 tokens
      for (int i = max(0, p - (L - n)); i < n; ++i) {
        for (int h = g * G; h < g * G + G; ++h) {
          const float lse = c.lse[(size_t)(t0 + i) * c.n_q + h];
          if (lse == -INFINITY) continue;
          const uint2 qw = *reinterpret_cast<const uint2*>(c.q + (t0 + i) * c.q_stride + (size_t)h * kD + 4 * lane);
          const float s = warp_sum(bf_lo(qw.x) * k[0] + bf_hi(qw.x) * k[1] + bf_lo(qw.y) * k[2] + bf_hi(qw.y) * k[3]);
          part += expf(fmaf(s, c.scale, -lse));
        }
        if ((i & 15) == 15 || i == n - 1) {
          sum += part;
          part = 0.f;
        }
      }
    }
    const size_t at = ((size_t)b * c.n_kv + g) * c.cap + p;
    if (lane == 0) c.mass_next[at] = c.keep != 0.f ? fmaf(c.keep, c.mass_prev[at], sum) : sum;
  }
}

size_t kv4_mass_workspace(int, int, int, int) { return 256; }

int kv4_mass_launch(const Kv4ChunkCall& c, void*, void* stream) {
  const int blocks = ((c.max_blocks << c.block_shift) + 7) / 8;
  kv4_mass_kernel<<<dim3((unsigned)(blocks < 4096 ? blocks : 4096), (unsigned)(c.B * c.n_kv)), 256, 0,
                    static_cast<cudaStream_t>(stream)>>>(c);
  return cudaGetLastError() == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

}  // namespace spc
