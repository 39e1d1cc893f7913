// What the kernels over chunks of new tokens in the paged 4-bit cache share:
// the requests' shapes as a warp holds them, and the copies of their records.
#pragma once

#include <stdint.h>

#include "kv4.cuh"
#include "spc_device.cuh"
#include "spc_internal.h"
#include "spc_tc.cuh"

namespace spc {

constexpr int kKcCtas = 152;                          // one per SM; a constant, so that the workspace depends on shapes alone
constexpr int kKcKeys = 128;                          // positions a block
constexpr int kKcHalf = 64;                           // positions of half a block
constexpr uint32_t kKcTile = kKcKeys * kRowBytes;     // 32 KB: 128 rows of 16-bit values
constexpr uint32_t kKcBlock = kKcTile / 2;            // its 64-value half
constexpr long long kKcWait = 4000000000ll;           // clock cycles, some 2 s

// request b of a call: lane b / 2 of a warp has it at index b & 1
struct KcRequests {
  int row0[2], n[2], len[2];                          // first row, new tokens, positions in the cache
  long long end[2];                                   // units of the requests up to and with this one
};
__device__ __forceinline__ void kc_requests(const Kv4ChunkCall& c, KcRequests& r) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int b = 2 * lane + e;
    r.row0[e] = r.n[e] = r.len[e] = 0;
    if (b < c.B) {
      r.row0[e] = max(0, min(c.cu[b], c.T));
      r.n[e] = max(r.row0[e], min(c.cu[b + 1], c.T)) - r.row0[e];
      r.len[e] = max(0, min(c.len[b], c.max_blocks << c.block_shift));
    }
  }
}
// end[] from each request's own units u[]; returns their sum
__device__ __forceinline__ long long kc_prefix(KcRequests& r, long long u0, long long u1) {
  const int lane = threadIdx.x & 31;
  long long s = u0 + u1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  r.end[0] = s - u1;
  r.end[1] = s;
  return __shfl_sync(0xffffffffu, s, 31);
}
template <class T>
__device__ __forceinline__ T kc_of(const T (&v)[2], int b) {
  return __shfl_sync(0xffffffffu, b & 1 ? v[1] : v[0], b >> 1);
}
// the first request with units behind u
__device__ __forceinline__ int kc_find(const KcRequests& r, long long u) {
  return __popc(__ballot_sync(0xffffffffu, r.end[0] <= u)) + __popc(__ballot_sync(0xffffffffu, r.end[1] <= u));
}

// The second of a call's two kernels is launched while the first one runs: the
// first one lets it, once each of its CTAs is there, and the second one waits for
// the end of it before it reads or writes anything (17 tokens behind 1000, call after call in
// a stream: 1.8 us of 20.5 less; no difference in a graph).
__device__ __forceinline__ void kc_let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void kc_wait_first() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <class... P, class... A>
static bool kc_launch_next(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

// a / b of 64 bits each, mostly small: a division of 64 bits takes some 400 cycles, and the plans have chains of them
__device__ __forceinline__ long long kc_div(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The table entries of a request, a window of 32 at a time and the next one on
// its way: lane l holds entry `at` + l, -1 behind the last one.
struct KcTable {
  const int32_t* row;
  int at, n, cur, next;
  __device__ __forceinline__ int get(int i) const { return i < n ? row[i] : -1; }
  __device__ __forceinline__ void start(const int32_t* table_row, int entries, int first) {
    row = table_row;
    n = entries;
    at = first & ~31;
    cur = get(at + (threadIdx.x & 31));
    next = get(at + 32 + (threadIdx.x & 31));
  }
  // the same, where what is there may do: the same row, at its window or the one behind it
  __device__ __forceinline__ void move(const int32_t* table_row, int entries, int first) {
    const int to = first & ~31;
    if (row != table_row || (to != at && to != at + 32)) start(table_row, entries, first);
  }
  // entry i of this lane's choice, all of them in the window of `first` (a warp-uniform index)
  __device__ __forceinline__ int entry(int first, int i) {
    if ((first & ~31) != at) {
      at = first & ~31;
      cur = next;
      next = get(at + 32 + (threadIdx.x & 31));
    }
    return __shfl_sync(0xffffffffu, cur, i & 31);
  }
};

// One warp: the records of positions p0 .. p0 + 63 (p0 a multiple of 64) of a
// request with `len` positions, KV head g, into a stage, one bulk copy a cache
// block (a copy costs its warp some 200 clocks); the positions there are, as
// bits. The stage's barrier has one arrival.
__device__ __forceinline__ void kc_copy(const Kv4ChunkCall& c, KcTable& t, int g, int len, int p0, uint8_t* stage,
                                        uint64_t* bar, uint32_t* mask) {
  const int lane = threadIdx.x & 31, bs = 1 << c.block_shift, run = min(bs, kKcHalf), runs = kKcHalf / run;
  const int p = p0 + lane * run;
  const int blk = t.entry(p0 >> c.block_shift, p >> c.block_shift);
  int n = 0;
  if (lane < runs && (unsigned)blk < (unsigned)c.num_blocks) n = max(0, min(len - p, run));
  if (runs == 1) {
    // one copy: by an elected lane, from uniform values
    const int one = __shfl_sync(0xffffffffu, blk, 0), cnt = __shfl_sync(0xffffffffu, n, 0);
    if (elect_one()) {
      *reinterpret_cast<uint2*>(mask) = make_uint2(cnt >= 32 ? 0xffffffffu : (1u << cnt) - 1u,
                                                   cnt >= 64 ? 0xffffffffu : cnt > 32 ? (1u << (cnt - 32)) - 1u : 0u);
      if (cnt > 0) {
        mbar_arrive_expect_tx(bar, (uint32_t)cnt * kKv4Rec);
        bulk_g2s(stage, c.cache + (((size_t)one * c.n_kv + g) * bs + (p0 & (bs - 1))) * kKv4Rec, (uint32_t)cnt * kKv4Rec, bar);
      } else {
        mbar_arrive(bar);
      }
    }
    __syncwarp();
    return;
  }
  uint32_t m[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int lo = max(0, lane * run - 32 * h), hi = min(32, lane * run + n - 32 * h);   // bits of word h
    m[h] = n > 0 && hi > lo ? (hi - lo == 32 ? 0xffffffffu : ((1u << (hi - lo)) - 1u)) << lo : 0u;
    m[h] = __reduce_or_sync(0xffffffffu, m[h]);
  }
  const uint32_t bytes = __reduce_add_sync(0xffffffffu, (uint32_t)n) * kKv4Rec;
  if (lane == 0) {
    *reinterpret_cast<uint2*>(mask) = make_uint2(m[0], m[1]);
    if (bytes) mbar_arrive_expect_tx(bar, bytes); else mbar_arrive(bar);
  }
  __syncwarp();
  if (n > 0)
    bulk_g2s(stage + lane * run * kKv4Rec, c.cache + (((size_t)blk * c.n_kv + g) * bs + (p & (bs - 1))) * kKv4Rec,
             (uint32_t)n * kKv4Rec, bar);
  __syncwarp();
}

__device__ __forceinline__ uint4 lds_v4(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds_v2(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ void sts_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

}  // namespace spc
