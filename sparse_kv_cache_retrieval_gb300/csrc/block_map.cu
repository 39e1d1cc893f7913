// Block tables and slot maps of a paged cache from request lengths.
//
// Everything follows from three prefix sums over at most 64 requests (new
// positions, blocks given back, blocks taken), so every CTA computes them for
// itself with one warp and the CTAs share nothing: the i-th block taken is
// entry (n_free + given back - 1 - i) of the free stack, which is an old stack
// entry or, above n_free, a table entry of a shrinking request, and neither is
// written by this call. One launch, no atomics but the error word's.
// Bound: latency (two dependent loads and one search of the prefix); the slot
// map is 4 bytes a new token.
#include <cuda_runtime.h>

#include "spc_device.cuh"
#include "spc_internal.h"

namespace spc {

constexpr int kBmThreads = 256;
constexpr int kBmBatch = SPC_MAX_BATCH;
static_assert(kBmBatch == 64, "the prefix sums run two requests a lane");

struct BmShared {
  int old[kBmBatch];            // L0
  int have[kBmBatch];           // blocks held before the call
  int want[kBmBatch];           // and after it
  int cu[kBmBatch + 1];         // new positions before request b
  int pop[kBmBatch + 1];        // blocks taken before request b
  int push[kBmBatch + 1];       // blocks given back before request b
  int n_free;
  int bad;
};

// the request whose run of the exclusive prefix pre[0 .. B] holds item i < pre[B]
__device__ __forceinline__ int bm_find(const int* pre, int B, int i) {
  int lo = 0, hi = B;           // pre[lo] <= i < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// exclusive prefix of two consecutive items a lane into out[0 .. 64]
__device__ __forceinline__ void bm_scan(int a, int b, int lane, int* out) {
  const int incl = warp_incl_scan(a + b);
  out[2 * lane] = incl - a - b;
  out[2 * lane + 1] = incl - b;
  if (lane == 31) out[2 * lane + 2] = incl;
}

__device__ __forceinline__ int bm_popped(const BlockMapCall& a, const BmShared& s, int i) {
  const int pos = s.n_free + s.push[kBmBatch] - 1 - i;
  if (pos < s.n_free) return a.free_list[pos];
  const int r = pos - s.n_free, b = bm_find(s.push, kBmBatch, r);
  return a.table[(size_t)b * a.max_blocks + s.want[b] + (r - s.push[b])];
}

// V consecutive slots a thread: one search, one block entry in most cases.
// V = 4 once there are more slots than threads (1.7 M slots: 5.9 us, with V =
// 1 10.0), else V = 1 (64 slots of 64 requests: 2.6 us, with V = 4 3.5).
template <int V>
__global__ void __launch_bounds__(kBmThreads) block_map_kernel(BlockMapCall a) {
  __shared__ BmShared s;
  const int bs = 1 << a.block_shift;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int n_free = *a.n_free;
    int grow[2], take[2], give[2];
    bool bad = n_free < 0 || n_free > a.num_blocks;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int b = 2 * lane + e;
      int l0 = 0, l1 = 0;
      if (b < a.B) {
        l0 = a.len[b];
        l1 = a.len_next[b];
        const int most = a.max_blocks << a.block_shift;
        if (l0 < 0 || l1 < 0 || l0 > most || l1 > most) {
          bad = true;
          l0 = l1 = 0;
        }
      }
      const int h = (l0 + bs - 1) >> a.block_shift, w = (l1 + bs - 1) >> a.block_shift;
      s.old[b] = l0;
      s.have[b] = h;
      s.want[b] = w;
      grow[e] = max(0, l1 - l0);
      take[e] = max(0, w - h);
      give[e] = max(0, h - w);
    }
    bm_scan(grow[0], grow[1], lane, s.cu);
    bm_scan(take[0], take[1], lane, s.pop);
    bm_scan(give[0], give[1], lane, s.push);
    bad = __any_sync(0xffffffffu, bad);
    __syncwarp();
    if (lane == 0) {
      const long long top = (long long)n_free + s.push[kBmBatch];
      bad = bad || top > a.num_blocks || s.pop[kBmBatch] > top || s.cu[kBmBatch] > a.n_slots;
      s.n_free = n_free;
      s.bad = bad;
      if (blockIdx.x == 0) {
        if (bad) set_status(a.status, SPC_ERR_OVERFLOW);
        *a.n_free_next = bad ? n_free : (int)top - s.pop[kBmBatch];
      }
    }
  }
  __syncthreads();
  const bool bad = s.bad != 0;
  const int tid = blockIdx.x * kBmThreads + threadIdx.x, stride = gridDim.x * kBmThreads;
  if (blockIdx.x == 0 && threadIdx.x <= a.B) a.cu_new[threadIdx.x] = bad ? 0 : s.cu[threadIdx.x];
  const int n_pop = bad ? 0 : s.pop[kBmBatch], n_push = bad ? 0 : s.push[kBmBatch];
  for (int i = tid; i < n_pop; i += stride) {
    const int b = bm_find(s.pop, kBmBatch, i);
    a.table[(size_t)b * a.max_blocks + s.have[b] + (i - s.pop[b])] = bm_popped(a, s, i);
  }
  for (int i = tid; i < n_push; i += stride) {
    const int b = bm_find(s.push, kBmBatch, i);
    a.free_list[s.n_free + i] = a.table[(size_t)b * a.max_blocks + s.want[b] + (i - s.push[b])];
  }
  const int n_new = bad ? 0 : s.cu[kBmBatch];
  const bool wide = (reinterpret_cast<uintptr_t>(a.slot_map) & 15u) == 0;
  for (int t = V * tid; t < a.n_slots; t += V * stride) {
    int out[V];
#pragma unroll
    for (int e = 0; e < V; ++e) out[e] = -1;
    if (t < n_new) {
      int b = bm_find(s.cu, kBmBatch, t), seen = -1, blk = -1;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (t + e >= n_new) break;
        if (t + e >= s.cu[b + 1]) {
          do ++b; while (t + e >= s.cu[b + 1]);
          seen = -1;
        }
        const int p = s.old[b] + (t + e - s.cu[b]), k = p >> a.block_shift;
        if (k != seen) {
          seen = k;
          blk = k < s.have[b] ? a.table[(size_t)b * a.max_blocks + k] : bm_popped(a, s, s.pop[b] + k - s.have[b]);
        }
        if (blk >= 0 && blk < a.num_blocks) out[e] = (blk << a.block_shift) + (p & (bs - 1));
      }
    }
    if (V == 4 && wide && t + 4 <= a.n_slots) {
      *reinterpret_cast<int4*>(a.slot_map + t) = make_int4(out[0], out[V > 1 ? 1 : 0], out[V > 2 ? 2 : 0], out[V > 3 ? 3 : 0]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (t + e < a.n_slots) a.slot_map[t + e] = out[e];
    }
  }
}

int block_map_launch(const BlockMapCall& c, void* stream) {
  constexpr int most = 152 * 4;
  const int v = c.n_slots > most * kBmThreads ? 4 : 1;
  const int grid = min((c.n_slots + v * kBmThreads - 1) / (v * kBmThreads), most);
  if (v == 4)
    block_map_kernel<4><<<grid, kBmThreads, 0, static_cast<cudaStream_t>(stream)>>>(c);
  else
    block_map_kernel<1><<<grid, kBmThreads, 0, static_cast<cudaStream_t>(stream)>>>(c);
  return cudaGetLastError() == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

}  // namespace spc
