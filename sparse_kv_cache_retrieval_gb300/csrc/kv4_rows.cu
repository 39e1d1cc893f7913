// Rows of K and V into and out of the paged 4-bit cache.
//
// A group of 16 values, its scale and its 16 codes are one lane's: 8 lanes a K
// or V row, two (token, KV head) pairs a warp, and kRowBatch such steps loaded
// before the first is worked on: 2 where there are more steps than warps
// (65536 tokens of 8 heads, store and load: 122 us, with 1 step 147), else 1
// (8 tokens: 3.3 us, with 2 steps 4.1).
//
// Rounding. The scale is e4m3 of the exact quotient max / 6, the codes are
// e2m1 of the exact quotients x / s, ties to even. Neither division is done:
// x (bf16) has 8 significant bits, s has 4, ties of e4m3 have 5 and ties of
// e2m1 at most 3, so a quotient that is not a tie is at least 2^-8 (relative)
// away from one. max * (1/6) in fp32 is within 2^-22 of the quotient; rounded
// to fp16 (11 bits) it is the tie where there is one and stays on its side
// where there is none, and e4m3 of that is e4m3 of the quotient. In the same
// way x * r, r within 2^-22 of 1/s, is rounded to multiples of 2^-11 (ties of
// e2m1 are multiples of 1/4, and a quotient beside one of at least 1/4 is at
// least 2^-10 away) by adding and subtracting 6144 in fp32.
//
// Bound: HBM (512 bytes read and 144 written a pair, or the reverse).
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "spc_device.cuh"
#include "spc_internal.h"

namespace spc {

constexpr int kRowThreads = 256;
constexpr int kRowCtas = 152 * 8;         // 8 CTAs of 8 warps fill an SM

__device__ __forceinline__ uint8_t* kv4_record(const Kv4RowsCall& a, int slot, int g) {
  const int blk = slot >> a.block_shift, r = slot & ((1 << a.block_shift) - 1);
  return a.cache + ((((size_t)blk * a.n_kv + g) << a.block_shift) + r) * kKv4Rec;
}
// 32 bytes a lane; one instruction where the rows are 32-byte aligned
__device__ __forceinline__ void row_load(const uint16_t* p, bool wide, uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p));
  } else {
    const uint4 x = ldg_stream(p), y = ldg_stream(p + 8);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
  }
}
__device__ __forceinline__ void row_store(uint16_t* p, bool wide, const uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" :: "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
  } else {
    stg_v4(p, make_uint4(w[0], w[1], w[2], w[3]));
    stg_v4(p + 8, make_uint4(w[4], w[5], w[6], w[7]));
  }
}
__device__ __forceinline__ bool rows_wide(const uint16_t* p, int64_t stride) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride * 2) & 31u) == 0;
}

// Steps of two pairs: pair 2 step + (lane / 16), in (token, head) order. The
// division is made once and carried on.
struct RowCursor {
  long long i;
  int t, g;
};
__device__ __forceinline__ RowCursor row_at(const Kv4RowsCall& a, long long i) {
  RowCursor c;
  c.i = i;
  c.t = (int)(i / a.n_kv);
  c.g = (int)(i - (long long)c.t * a.n_kv);
  return c;
}
__device__ __forceinline__ void row_next(const Kv4RowsCall& a, RowCursor& c, int n) {
  c.i += n;
  c.g += n;
  while (c.g >= a.n_kv) {
    c.g -= a.n_kv;
    ++c.t;
  }
}

__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int kRowBatch>
__global__ void __launch_bounds__(kRowThreads) kv4_store_kernel(Kv4RowsCall a) {
  const int lane = threadIdx.x & 31, q = lane & 7, isv = (lane >> 3) & 1, half = lane >> 4;
  const long long n = (long long)a.T * a.n_kv;
  const long long warps = (long long)gridDim.x * (kRowThreads / 32);
  const uint16_t* base = (isv ? a.v : a.k) + 16 * q;
  const int64_t stride = isv ? a.v_stride : a.k_stride;
  const bool wide = rows_wide(base, stride);
  for (long long s0 = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); s0 * 2 * kRowBatch < n; s0 += warps) {
    uint32_t w[kRowBatch][8];
    uint8_t* rec[kRowBatch];
    RowCursor c = row_at(a, s0 * 2 * kRowBatch + half);
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b) {
      rec[b] = nullptr;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[b][j] = 0u;
      if (c.i < n) {
        const int slot = __ldg(a.slot_map + c.t);
        row_load(base + c.t * stride + c.g * kD, wide, w[b]);
        if (slot >= 0 && slot < a.n_cache_slots) rec[b] = kv4_record(a, slot, c.g);
      }
      row_next(a, c, 2);
    }
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b) {
      // largest magnitude: bit patterns without the sign order like the
      // magnitudes, NaN above infinity
      uint32_t m = w[b][0] & 0x7fff7fffu;
#pragma unroll
      for (int j = 1; j < 8; ++j) m = __vmaxu2(m, w[b][j] & 0x7fff7fffu);
      m = max(m & 0xffffu, m >> 16);
      const __half2 a6 = __floats2half2_rn(__uint_as_float(m << 16) * (1.f / 6.f), 0.f);
      const uint32_t sb = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(a6), __NV_SATFINITE, __NV_E4M3) & 0xffu;
      const float s = f16_lo(e4m3x2_to_f16(sb));
      const float r = s > 0.f ? rcp_fast(s) : 0.f;
      const float2 rr = make_float2(r, r), up = make_float2(6144.f, 6144.f), dn = make_float2(-6144.f, -6144.f);
      uint32_t codes[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t v = w[b][4 * e + j];
          const float2 z = make_float2(bf_lo(v), bf_hi(v)), y = add2(fma2(z, rr, up), dn);
          x[2 * j] = copysignf(y.x, z.x);            // what rounds to zero keeps its sign
          x[2 * j + 1] = copysignf(y.y, z.y);
        }
        codes[e] = f32_to_e2m1x8(x);
      }
      if (rec[b]) {
        *reinterpret_cast<uint2*>(rec[b] + isv * kKv4V + 8 * q) = make_uint2(codes[0], codes[1]);
        rec[b][kKv4Scale + 8 * isv + q] = (uint8_t)sb;
      }
    }
  }
}

template <int kRowBatch>
__global__ void __launch_bounds__(kRowThreads) kv4_load_kernel(Kv4RowsCall a) {
  const int lane = threadIdx.x & 31, q = lane & 7, isv = (lane >> 3) & 1, half = lane >> 4;
  const long long n = (long long)a.T * a.n_kv;
  const long long warps = (long long)gridDim.x * (kRowThreads / 32);
  uint16_t* base = const_cast<uint16_t*>(isv ? a.v : a.k) + 16 * q;
  const int64_t stride = isv ? a.v_stride : a.k_stride;
  const bool wide = rows_wide(base, stride);
  for (long long s0 = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); s0 * 2 * kRowBatch < n; s0 += warps) {
    uint2 codes[kRowBatch];
    uint32_t sb[kRowBatch];
    uint16_t* dst[kRowBatch];
    RowCursor c = row_at(a, s0 * 2 * kRowBatch + half);
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b) {
      dst[b] = nullptr;
      codes[b] = make_uint2(0u, 0u);
      sb[b] = 0;
      if (c.i < n) {
        const int slot = __ldg(a.slot_map + c.t);
        if (slot >= 0 && slot < a.n_cache_slots) {
          const uint8_t* rec = kv4_record(a, slot, c.g);
          codes[b] = __ldg(reinterpret_cast<const uint2*>(rec + isv * kKv4V + 8 * q));
          sb[b] = __ldg(rec + kKv4Scale + 8 * isv + q);
          dst[b] = base + c.t * stride + c.g * kD;
        }
      }
      row_next(a, c, 2);
    }
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b) {
      const uint32_t s = e4m3_dup_f16(sb[b]);
      uint32_t h[8];
      e2m1x8_to_f16(codes[b].x, *reinterpret_cast<uint32_t (*)[4]>(h));
      e2m1x8_to_f16(codes[b].y, *reinterpret_cast<uint32_t (*)[4]>(h + 4));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[j] = hmul2(h[j], s);
        h[j] = pack_bf16(f16_lo(h[j]), f16_hi(h[j]));
      }
      if (dst[b]) row_store(dst[b], wide, h);
    }
  }
}

static int rows_launch(void (*one)(Kv4RowsCall), void (*two)(Kv4RowsCall), const Kv4RowsCall& c, void* stream) {
  const long long n = (long long)c.T * c.n_kv, per = kRowThreads / 32 * 2;     // pairs a CTA, a step
  const long long ctas = (n + per - 1) / per;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (ctas <= kRowCtas)
    one<<<(int)ctas, kRowThreads, 0, st>>>(c);
  else
    two<<<(int)((ctas + 1) / 2 < kRowCtas ? (ctas + 1) / 2 : kRowCtas), kRowThreads, 0, st>>>(c);
  return cudaGetLastError() == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

int kv4_store_launch(const Kv4RowsCall& c, void* stream) {
  return rows_launch(kv4_store_kernel<1>, kv4_store_kernel<2>, c, stream);
}

int kv4_load_launch(const Kv4RowsCall& c, void* stream) {
  return rows_launch(kv4_load_kernel<1>, kv4_load_kernel<2>, c, stream);
}

}  // namespace spc
