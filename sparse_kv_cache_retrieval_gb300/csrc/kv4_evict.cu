// Eviction from the paged 4-bit cache by accumulated attention weight: per
// (request, KV head) the sinks, the recent window and the largest sums are kept
// (ties to the lower position), and their records move to the front in order.
//
// One thread-block cluster per (request, KV head). A rank owns a contiguous
// slice of the positions and, later, a contiguous share of the kept rows:
//  1. the slice's sums become order keys in shared memory (the bits of a
//     non-negative float; forced positions above every sum);
//  2. a radix select over the cluster (11, 10 and 10 bits) finds the key of the
//     last position kept. Counts are added to the rank that owns a bin, and
//     every rank reads all totals, so that all reach the same threshold;
//  3. each rank counts what it keeps, the counts give the ranks their places,
//     and each kept position is written to the list of the rank that moves it;
//  4. every rank copies its share of the rows and sums into shared memory, the
//     cluster meets, and only then is anything written. So a cache that shrinks
//     in place, where row i comes from a place >= i that may be another row's
//     destination, needs no order between the moves.
// Bound: the sums' bytes and the kept records', 144 in and out; small calls by
// the chain of seven cluster barriers.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "spc_device.cuh"
#include "spc_internal.h"

namespace spc {
namespace cg = cooperative_groups;

constexpr int kEvThreads = 512;
constexpr int kEvCluster = 8;
constexpr int kEvBins = 2048 + 1024 + 1024;          // of the three levels
constexpr uint32_t kEvForced = 0xffffffffu;

struct EvShared {
  uint32_t tot[kEvBins];                             // this rank's bins (bin % C == rank) over the cluster
  int scratch[33];
  uint32_t wgt[kEvThreads / 32], weq[kEvThreads / 32];
  uint32_t cgt[kEvCluster], ceq[kEvCluster];         // of every rank
  uint32_t bin, above;
};

struct EvArgs {
  Kv4EvictCall c;
  int slice, share;    // most positions and kept rows a rank
};

__host__ __device__ constexpr size_t ev_rows_bytes(int share) {
  return (size_t)share * kKv4Rec > 8192 ? (size_t)share * kKv4Rec : 8192;
}

__global__ void __launch_bounds__(kEvThreads) kv4_evict_kernel(const EvArgs a) {
  extern __shared__ __align__(16) uint8_t ev_raw[];
  cg::cluster_group cluster = cg::this_cluster();
  constexpr int C = kEvCluster;
  const Kv4EvictCall& c = a.c;
  EvShared& sm = *reinterpret_cast<EvShared*>(ev_raw);
  uint8_t* rows = ev_raw + (sizeof(EvShared) + 15) / 16 * 16;                 // [share][144]; before that,
  uint32_t* hist = reinterpret_cast<uint32_t*>(rows);                         // [2048]
  uint32_t* keys = reinterpret_cast<uint32_t*>(rows + ev_rows_bytes(a.share));  // [slice]
  int* list = reinterpret_cast<int*>(keys + a.slice);                         // [share]
  float* sums = reinterpret_cast<float*>(list + a.share);                     // [share]
  const int rank = (int)cluster.block_rank(), seg = blockIdx.x / C, b = seg / c.n_kv, g = seg - b * c.n_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = 1 << c.block_shift;
  const int L = max(0, min(c.len[b], c.max_blocks << c.block_shift)), K = min(L, c.budget);
  const int32_t* from = c.table + (size_t)b * c.max_blocks;
  const int32_t* to = c.table_next + (size_t)b * c.max_blocks;
  const float* mass = c.mass + (size_t)seg * c.cap;
  float* mass_next = c.mass_next + (size_t)seg * c.cap;
  int32_t* kept = c.kept ? c.kept + (size_t)seg * c.budget : nullptr;

  // the request is left as it was if a block that it uses is not in the pool
  bool bad = false;
  for (int i = tid; i < (L + bs - 1) >> c.block_shift; i += kEvThreads) bad |= (unsigned)from[i] >= (unsigned)c.num_blocks;
  for (int i = tid; i < (K + bs - 1) >> c.block_shift; i += kEvThreads) bad |= (unsigned)to[i] >= (unsigned)c.num_blocks;
  if (__syncthreads_or(bad)) {
    const int t = rank * kEvThreads + tid;
    if (kept)
      for (int i = t; i < c.budget; i += C * kEvThreads) kept[i] = -1;
    if (mass_next != mass)
      for (int i = t; i < L; i += C * kEvThreads) mass_next[i] = mass[i];
    if (t == 0 && g == 0) c.len_next[b] = L;
    if (t == 0) set_status(c.status, SPC_ERR_INVALID_ARG);
    return;
  }

  // ---- order keys of the slice
  const int slice = min(a.slice, ((L + C - 1) / C + 31) & ~31), p0 = min(L, rank * slice), n = min(L, p0 + slice) - p0;
  const bool all = L <= c.budget;
  for (int i = tid; i < n; i += kEvThreads) {
    const int p = p0 + i;
    const float m = mass[p];
    keys[i] = all || p < c.n_sink || p >= L - c.n_recent ? kEvForced : m > 0.f ? __float_as_uint(m) : 0u;
  }
  for (int i = tid; i < kEvBins; i += kEvThreads) sm.tot[i] = 0u;
  __syncthreads();

  // ---- threshold: keys above it are kept, and the first `ties` of those equal to it
  uint32_t thr = kEvForced - 1, ties = 0u;
  const int want = all ? 0 : K - c.n_sink - c.n_recent;
  if (want > 0) {
    uint32_t need = (uint32_t)want, prefix = 0u;
    int base = 0;
#pragma unroll 1
    for (int level = 0; level < 3; ++level) {
      const int bits = level == 0 ? 11 : 10, shift = level == 0 ? 20 : level == 1 ? 10 : 0, bins = 1 << bits;
      for (int i = tid; i < bins; i += kEvThreads) hist[i] = 0u;
      __syncthreads();
      for (int i = tid; i < n; i += kEvThreads) {
        const uint32_t k = keys[i];
        if (k != kEvForced && (level == 0 || k >> (shift + bits) == prefix)) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
      }
      if (level == 0) cluster.sync(); else __syncthreads();          // every rank's totals are zero
      for (int i = tid; i < bins; i += kEvThreads)
        if (hist[i]) atomicAdd(cluster.map_shared_rank(&sm.tot[base + i], i % C), hist[i]);
      cluster.sync();
      // the bins from the highest down, bins / kEvThreads a thread
      const int per = bins / kEvThreads;
      uint32_t v[4], s = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = bins - 1 - (tid * per + j);
        v[j] = j < per ? *cluster.map_shared_rank(&sm.tot[base + i], i % C) : 0u;
        s += v[j];
      }
      int total;
      uint32_t run = (uint32_t)block_excl_scan((int)s, sm.scratch, &total);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (run < need && run + v[j] >= need) {
          sm.bin = (uint32_t)(bins - 1 - (tid * per + j));
          sm.above = run;
        }
        run += v[j];
      }
      __syncthreads();
      prefix = (prefix << bits) | sm.bin;
      need -= sm.above;
      base += bins;
      __syncthreads();
    }
    thr = prefix;
    ties = need;
  }

  // ---- what each warp's part of the slice keeps, and where the rank's places begin
  constexpr int W = kEvThreads / 32;
  const int part = (n + W * 32 - 1) / (W * 32) * 32, w0 = min(n, warp * part), w1 = min(n, w0 + part);
  uint32_t ngt = 0u, neq = 0u;
  for (int i = w0; i < w1; i += 32) {
    const uint32_t k = i + lane < w1 ? keys[i + lane] : 0u;
    const bool in = i + lane < w1;
    ngt += __popc(__ballot_sync(0xffffffffu, in && k > thr));
    neq += __popc(__ballot_sync(0xffffffffu, in && k == thr));
  }
  if (lane == 0) {
    sm.wgt[warp] = ngt;
    sm.weq[warp] = neq;
  }
  __syncthreads();
  if (tid < C) {
    uint32_t gt = 0u, eq = 0u;
    for (int w = 0; w < W; ++w) {
      gt += sm.wgt[w];
      eq += sm.weq[w];
    }
    *cluster.map_shared_rank(&sm.cgt[rank], tid) = gt;
    *cluster.map_shared_rank(&sm.ceq[rank], tid) = eq;
  }
  cluster.sync();
  uint32_t gt = 0u, eq = 0u;                          // kept by their keys, equal to the threshold, before this warp's part
  for (int r = 0; r < rank; ++r) {
    gt += sm.cgt[r];
    eq += sm.ceq[r];
  }
  for (int w = 0; w < warp; ++w) {
    gt += sm.wgt[w];
    eq += sm.weq[w];
  }

  // ---- the kept positions, to the ranks that move them
  const int share = min(a.share, (K + C - 1) / C);
  const uint32_t below = (1u << lane) - 1u;
  for (int i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1;
    const uint32_t k = in ? keys[i + lane] : 0u;
    const uint32_t mg = __ballot_sync(0xffffffffu, in && k > thr), me = __ballot_sync(0xffffffffu, in && k == thr);
    const uint32_t e = eq + __popc(me & below);
    if (in && (k > thr || (k == thr && e < ties))) {
      const int at = (int)(gt + __popc(mg & below) + min(e, ties));
      *cluster.map_shared_rank(&list[at % share], at / share) = p0 + i + lane;
      if (kept) kept[at] = p0 + i + lane;
    }
    gt += __popc(mg);
    eq += __popc(me);
  }
  if (kept)
    for (int i = K + rank * kEvThreads + tid; i < c.budget; i += C * kEvThreads) kept[i] = -1;
  cluster.sync();

  // ---- this rank's rows and sums, all of them read before any is written
  const int i0 = min(K, rank * share), m = min(K, i0 + share) - i0;
  auto record = [&](const int32_t* table, int p) {
    return c.cache + (((size_t)table[p >> c.block_shift] * c.n_kv + g) * bs + (p & (bs - 1))) * kKv4Rec;
  };
  for (int e = tid; e < m * 9; e += kEvThreads) {
    const int i = e / 9, piece = (e - i * 9) * 16;
    const uint8_t* src = record(from, list[i]);
    if (src != record(to, i0 + i)) cp_async16(rows + i * kKv4Rec + piece, src + piece, 16);
  }
  for (int i = tid; i < m; i += kEvThreads) sums[i] = mass[list[i]];
  cp_async_commit();
  cp_async_wait<0>();
  cluster.sync();
  for (int e = tid; e < m * 9; e += kEvThreads) {
    const int i = e / 9, piece = (e - i * 9) * 16;
    uint8_t* dst = record(to, i0 + i);
    if (dst != record(from, list[i])) stg_v4(dst + piece, *reinterpret_cast<const uint4*>(rows + i * kKv4Rec + piece));
  }
  for (int i = tid; i < m; i += kEvThreads) mass_next[i0 + i] = sums[i];
  for (int i = K + rank * kEvThreads + tid; i < L; i += C * kEvThreads) mass_next[i] = 0.f;
  if (g == 0 && rank == 0 && tid == 0) c.len_next[b] = K;
}

int kv4_evict_launch(const Kv4EvictCall& c, void* stream) {
  EvArgs a{};
  a.c = c;
  const int most = c.max_blocks << c.block_shift;
  a.slice = ((most + kEvCluster - 1) / kEvCluster + 31) & ~31;
  a.share = ((most < c.budget ? most : c.budget) + kEvCluster - 1) / kEvCluster;
  const size_t smem = (sizeof(EvShared) + 15) / 16 * 16 + ev_rows_bytes(a.share) + (size_t)a.share * 8 + (size_t)a.slice * 4;
  if (set_func_attr((const void*)kv4_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SPC_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  cfg.gridDim = dim3((unsigned)(c.B * c.n_kv * kEvCluster));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = at;
  cfg.numAttrs = 1;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kEvCluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  return cudaLaunchKernelEx(&cfg, kv4_evict_kernel, a) == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

}  // namespace spc
