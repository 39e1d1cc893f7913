// Rows of K and V into and out of the paged 4-bit cache.
//
// One warp holds one (token, KV head): lanes 0-15 its K row, lanes 16-31 its V
// row, 8 values a lane, so that a group of 16 values is a pair of lanes.
// Rounding: the scale is e4m3(max|x| / 6) of the correctly rounded quotient;
// the codes need e2m1(x / s) of the exact quotient, ties included. x has 8
// significant bits and s has 4, so a quotient that is not a tie of e2m1 is at
// least 2^-8 (relative) away from one; x * (1 / s) in fp32 is within 2^-23 of
// it, and rounding that product to fp16 (11 bits) returns the tie exactly
// where there is one and stays on its side where there is none. The
// conversion of the fp16 value to e2m1 therefore rounds the exact quotient.
// Bound: HBM (512 bytes read and 144 written a row, or the reverse).
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "spc_device.cuh"
#include "spc_internal.h"

namespace spc {

constexpr int kRowThreads = 256;

__device__ __forceinline__ uint8_t* kv4_record(const Kv4RowsCall& a, int slot, int g) {
  const int blk = slot >> a.block_shift, r = slot & ((1 << a.block_shift) - 1);
  return a.cache + ((((size_t)blk * a.n_kv + g) << a.block_shift) + r) * kKv4Rec;
}

// A warp takes kRowBatch consecutive (token, head) pairs at a time and loads
// all of their rows before it works on the first.
constexpr int kRowBatch = 4;

// slot and head of pair i, -1 where there is none
__device__ __forceinline__ int row_slot(const Kv4RowsCall& a, long long i, long long n, int& t, int& g) {
  t = 0;
  g = 0;
  if (i >= n) return -1;
  t = a.n_kv == 1 ? (int)i : (int)(i / a.n_kv);
  g = (int)(i - (long long)t * a.n_kv);
  const int slot = __ldg(a.slot_map + t);
  return slot < a.n_cache_slots ? slot : -1;
}

__global__ void __launch_bounds__(kRowThreads) kv4_store_kernel(Kv4RowsCall a) {
  const int lane = threadIdx.x & 31, hl = lane & 15, isv = lane >> 4;
  const long long n = (long long)a.T * a.n_kv;
  const long long step = (long long)gridDim.x * (kRowThreads / 32) * kRowBatch;
  const uint16_t* base = (isv ? a.v : a.k) + 8 * hl;
  const int64_t stride = isv ? a.v_stride : a.k_stride;
  for (long long i = ((long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * kRowBatch; i < n; i += step) {
    uint4 w[kRowBatch];
    int slot[kRowBatch], g[kRowBatch];
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b) {
      int t;
      slot[b] = row_slot(a, i + b, n, t, g[b]);
      w[b] = make_uint4(0u, 0u, 0u, 0u);
      if (i + b < n) w[b] = ldg_stream(base + t * stride + g[b] * kD);
    }
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b) {
      // largest magnitude of the group: bit patterns without the sign order
      // like the magnitudes, NaN above infinity
      constexpr uint32_t A = 0x7fff7fffu;
      uint32_t m = __vmaxu2(__vmaxu2(w[b].x & A, w[b].y & A), __vmaxu2(w[b].z & A, w[b].w & A));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m & 0xffffu, m >> 16);
      const uint32_t sb = __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(m << 16), 6.f), __NV_SATFINITE, __NV_E4M3);
      const float s = f16_lo(e4m3x2_to_f16(sb));
      const float r = s > 0.f ? __frcp_rn(s) : 0.f;
      float x[8];
      unpack8(w[b], x);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const __half2 h = __floats2half2_rn(x[j] * r, x[j + 1] * r);
        x[j] = __low2float(h);
        x[j + 1] = __high2float(h);
      }
      const uint32_t codes = f32_to_e2m1x8(x);
      // the scales of four groups (eight lanes) as one word
      uint32_t sw = sb | (__shfl_down_sync(0xffffffffu, sb, 2) << 8);
      sw |= __shfl_down_sync(0xffffffffu, sw, 4) << 16;
      if (slot[b] < 0) continue;
      uint8_t* rec = kv4_record(a, slot[b], g[b]);
      *reinterpret_cast<uint32_t*>(rec + isv * kKv4V + 4 * hl) = codes;
      if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(rec + kKv4Scale + 4 * (lane >> 3)) = sw;
    }
  }
}

__global__ void __launch_bounds__(kRowThreads) kv4_load_kernel(Kv4RowsCall a) {
  const int lane = threadIdx.x & 31, hl = lane & 15, isv = lane >> 4;
  const long long n = (long long)a.T * a.n_kv;
  const long long step = (long long)gridDim.x * (kRowThreads / 32) * kRowBatch;
  uint16_t* base = const_cast<uint16_t*>(isv ? a.v : a.k) + 8 * hl;
  const int64_t stride = isv ? a.v_stride : a.k_stride;
  for (long long i = ((long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * kRowBatch; i < n; i += step) {
    uint32_t codes[kRowBatch], sb[kRowBatch];
    uint16_t* dst[kRowBatch];
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b) {
      int t, g;
      const int slot = row_slot(a, i + b, n, t, g);
      dst[b] = nullptr;
      codes[b] = sb[b] = 0;
      if (slot >= 0) {
        const uint8_t* rec = kv4_record(a, slot, g);
        codes[b] = __ldg(reinterpret_cast<const uint32_t*>(rec + isv * kKv4V + 4 * hl));
        sb[b] = __ldg(rec + kKv4Scale + 8 * isv + (hl >> 1));
        dst[b] = base + t * stride + g * kD;
      }
    }
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b) {
      const uint32_t s = e4m3_dup_f16(sb[b]);
      uint32_t h[4];
      e2m1x8_to_f16(codes[b], h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = hmul2(h[j], s);
        h[j] = pack_bf16(f16_lo(h[j]), f16_hi(h[j]));
      }
      if (dst[b]) stg_v4(dst[b], make_uint4(h[0], h[1], h[2], h[3]));
    }
  }
}

static int rows_grid(const Kv4RowsCall& c) {
  const long long n = (long long)c.T * c.n_kv, per = kRowThreads / 32 * kRowBatch;
  const long long g = (n + per - 1) / per;
  return (int)(g < 152 * 8 ? g : 152 * 8);
}

int kv4_store_launch(const Kv4RowsCall& c, void* stream) {
  kv4_store_kernel<<<rows_grid(c), kRowThreads, 0, static_cast<cudaStream_t>(stream)>>>(c);
  return cudaGetLastError() == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

int kv4_load_launch(const Kv4RowsCall& c, void* stream) {
  kv4_load_kernel<<<rows_grid(c), kRowThreads, 0, static_cast<cudaStream_t>(stream)>>>(c);
  return cudaGetLastError() == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

}  // namespace spc
