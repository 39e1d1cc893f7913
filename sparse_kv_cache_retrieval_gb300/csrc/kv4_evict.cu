// Eviction from the paged 4-bit cache by accumulated attention weight: per
// (request, KV head) the sinks, the recent window and the largest sums are kept
// (ties to the lower position), and their records move to the front in order.
//
// One thread-block cluster per (request, KV head). A rank owns a contiguous
// slice of the positions and, later, a contiguous share of the kept rows:
//  1. the slice's sums become order keys in shared memory (the bits of a
//     non-negative float; forced positions above every sum);
//  2. a radix select over the cluster (11, 10 and 10 bits) finds the key of the
//     last position kept. Every rank adds up all ranks' counts for itself, so
//     that all reach the same threshold with one barrier a level;
//  3. each rank counts what it keeps, the counts give the ranks their places,
//     and each kept position is written to the list of the rank that moves it;
//  4. batches of 256 rows a rank, in the order of the places, go through shared
//     memory, and the cluster meets between the loads of a batch and its stores. A
//     cache that shrinks in place needs no more: row i comes from a place >= i, so
//     that a batch overwrites no source of a later one.
// Ranks: one for each 16384 positions, and while there are few heads more of them, until
// the kept rows are one batch each (both sides at kv4_evict_launch).
// Bound: 8 requests of 65536 positions cut to 4096, 8 heads, take 45 us: 15 of
// them move 38 MB each way (65 MB of DRAM reads, for a record of 144 bytes begins
// at any multiple of 16: 4.3 TB/s), the others are the select's chain, which every
// cluster goes through at the same time: sums and tables 7 us, three levels 11 (a
// barrier of the cluster, the other ranks' counts, two scans), the ranks' counts 3, the list
// 6, the records' places 3. Small calls are that chain alone: 1088 positions cut to
// 1024 take 10.8 us. (Times from a clock trace of the slowest ranks.)
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "spc_device.cuh"
#include "spc_internal.h"

namespace spc {
namespace cg = cooperative_groups;

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvCluster = 8;                        // most ranks (the portable limit)
constexpr int kEvSlice = 16384;                      // positions a rank is meant to have
constexpr int kEvBatch = 256;                        // rows of a batch, a rank
constexpr int kEvBins = 2048 + 1024 + 1024;          // of the three levels
constexpr uint32_t kEvForced = 0xffffffffu;

struct EvShared {
  uint32_t hist[kEvBins];                            // this rank's counts, kept apart: other ranks read them
  uint32_t sums[kEvWarps];
  uint32_t wcnt[kEvWarps];                           // a warp's part: kept by their keys, and (from bit 16) ties
  uint32_t cgt[kEvCluster], ceq[kEvCluster];         // of every rank
  uint32_t bin, above, pad[2];
};
static_assert(sizeof(EvShared) % 16 == 0, "what follows is aligned");

struct EvArgs {
  Kv4EvictCall c;
  int slice, share;        // most positions and kept rows a rank
  uint32_t list;           // offset in shared memory of the lists, behind the keys that become batches of rows
};

// Whether the cluster's other ranks have started: none of them may touch the shared
// memory of one that has not. Requests that select nothing (not longer than the
// budget, or all of it forced) meet no other barrier before they write to each other.
template <int C>
__device__ __forceinline__ void ev_started() {
  if constexpr (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
template <int C>
__device__ __forceinline__ void ev_wait_started() {
  if constexpr (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// a barrier of the cluster, or of the CTA where it is one
template <int C>
__device__ __forceinline__ void ev_sync() {
  if constexpr (C > 1) cg::this_cluster().sync(); else __syncthreads();
}
// rank r's copy of a shared address
template <int C, class T>
__device__ __forceinline__ T* ev_at(T* p, int r) {
  if constexpr (C > 1) return cg::this_cluster().map_shared_rank(p, r); else return p;
}

template <int C>
__global__ void __launch_bounds__(kEvThreads, 2) kv4_evict_kernel(const EvArgs a) {
  extern __shared__ __align__(16) uint8_t ev_raw[];
  ev_started<C>();
  const Kv4EvictCall& c = a.c;
  EvShared& sm = *reinterpret_cast<EvShared*>(ev_raw);
  uint8_t* rows = ev_raw + sizeof(EvShared);                                  // [2][kEvBatch][144]; before that
  uint32_t* keys = reinterpret_cast<uint32_t*>(rows);                         // [slice]
  uint32_t* list = reinterpret_cast<uint32_t*>(ev_raw + a.list);              // [share] kept positions, then their records
  uint32_t* dst = list + a.share;                                             // [share] records they go to
  int rank = 0;
  if constexpr (C > 1) rank = (int)cg::this_cluster().block_rank();
  const int seg = blockIdx.x / C, b = seg / c.n_kv, g = seg - b * c.n_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = 1 << c.block_shift;
  const int L = max(0, min(c.len[b], c.max_blocks << c.block_shift)), K = min(L, c.budget);
  const int32_t* from = c.table + (size_t)b * c.max_blocks;
  const int32_t* to = c.table_next + (size_t)b * c.max_blocks;
  const float* mass = c.mass + (size_t)seg * c.cap;
  float* mass_next = c.mass_next + (size_t)seg * c.cap;
  int32_t* kept = c.kept ? c.kept + (size_t)seg * c.budget : nullptr;

  // the tables' entries are checked below, where the first of them have arrived
  const int nfrom = (L + bs - 1) >> c.block_shift, nto = (K + bs - 1) >> c.block_shift;
  const int from0 = tid < nfrom ? from[tid] : 0, to0 = tid < nto ? to[tid] : 0;

  // ---- order keys of the slice, padded to whole runs of 128 by keys that are never kept
  const int slice = min(a.slice, ((L + C - 1) / C + 127) & ~127), p0 = min(L, rank * slice), n = min(L, p0 + slice) - p0;
  const int whole = (n + 127) & ~127;
  const bool all = L <= c.budget;
  // keys above thr are kept, and the first `ties` of those equal to it; 0 stands for what is not there
  auto key = [&](int p, float m) {
    return p >= L ? 0u : all || p < c.n_sink || p >= L - c.n_recent ? kEvForced : m > 0.f ? __float_as_uint(m) + 1u : 1u;
  };
  constexpr int U = 8;                                // loads in flight a thread
  if ((reinterpret_cast<uintptr_t>(mass + p0) & 15u) == 0) {
    for (int i0 = tid; 4 * i0 < whole; i0 += U * kEvThreads) {
      float4 m[U];
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int i = 4 * (i0 + e * kEvThreads);
        m[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (all || i >= n) continue;
        if (i + 3 < n) {
          m[e] = *reinterpret_cast<const float4*>(mass + p0 + i);
        } else {                                      // nothing behind the request is read
          m[e].x = mass[p0 + i];
          if (i + 1 < n) m[e].y = mass[p0 + i + 1];
          if (i + 2 < n) m[e].z = mass[p0 + i + 2];
        }
      }
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int i = 4 * (i0 + e * kEvThreads), p = p0 + i;
        if (i < whole)
          *reinterpret_cast<uint4*>(keys + i) =
              make_uint4(i < n ? key(p, m[e].x) : 0u, i + 1 < n ? key(p + 1, m[e].y) : 0u, i + 2 < n ? key(p + 2, m[e].z) : 0u,
                         i + 3 < n ? key(p + 3, m[e].w) : 0u);
      }
    }
  } else {
    for (int i0 = tid; i0 < whole; i0 += U * kEvThreads) {
      float m[U];
#pragma unroll
      for (int e = 0; e < U; ++e) m[e] = i0 + e * kEvThreads < n && !all ? mass[p0 + i0 + e * kEvThreads] : 0.f;
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int i = i0 + e * kEvThreads;
        if (i < whole) keys[i] = i < n ? key(p0 + i, m[e]) : 0u;
      }
    }
  }
  for (int i = tid; i < kEvBins / 4; i += kEvThreads) reinterpret_cast<uint4*>(sm.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
  // the request is left as it was if a block that it uses is not in the pool
  bool bad = (tid < nfrom && (unsigned)from0 >= (unsigned)c.num_blocks) || (tid < nto && (unsigned)to0 >= (unsigned)c.num_blocks);
  for (int i = tid + kEvThreads; i < nfrom; i += kEvThreads) bad |= (unsigned)from[i] >= (unsigned)c.num_blocks;
  for (int i = tid + kEvThreads; i < nto; i += kEvThreads) bad |= (unsigned)to[i] >= (unsigned)c.num_blocks;
  ev_wait_started<C>();
  if (__syncthreads_or(bad)) {                        // the same in every rank
    const int t = rank * kEvThreads + tid;
    if (kept)
      for (int i = t; i < c.budget; i += C * kEvThreads) kept[i] = -1;
    if (mass_next != mass)
      for (int i = t; i < L; i += C * kEvThreads) mass_next[i] = mass[i];
    if (t == 0 && g == 0) c.len_next[b] = L;
    if (t == 0) set_status(c.status, SPC_ERR_INVALID_ARG);
    return;
  }

  // ---- threshold
  uint32_t thr = kEvForced - 1u, ties = 0u;
  const int want = all ? 0 : K - c.n_sink - c.n_recent;
  if (want > 0) {
    uint32_t need = (uint32_t)want, prefix = 0u;
#pragma unroll
    for (int level = 0; level < 3; ++level) {
      // keys are 1 .. 2^31 - 2^23 + 1: 11 bits, 10 and 10
      constexpr int kShift[3] = {20, 10, 0}, kBase[3] = {0, 2048, 3072};
      const int bits = level == 0 ? 11 : 10, bins = 1 << bits, shift = kShift[level];
      uint32_t* hist = sm.hist + kBase[level];
      for (int i = 4 * tid; i < whole; i += 4 * kEvThreads) {
        const uint4 k4 = *reinterpret_cast<const uint4*>(keys + i);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (k[e] - 1u < kEvForced - 1u && (level == 0 || k[e] >> (shift + bits) == prefix))
            atomicAdd(&hist[(k[e] >> shift) & (bins - 1)], 1u);
      }
      ev_sync<C>();
      // four bins a thread, from the highest down
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (4 * tid < bins) {
#pragma unroll
        for (int r = 0; r < C; ++r) {
          const uint4 x = *ev_at<C>(reinterpret_cast<uint4*>(hist) + (bins / 4 - 1 - tid), r);
          v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
        }
      }
      const uint32_t mine = v.x + v.y + v.z + v.w;
      const uint32_t incl = (uint32_t)warp_incl_scan((int)mine);
      if (lane == 31) sm.sums[warp] = incl;
      __syncthreads();
      uint32_t run = incl - mine;
#pragma unroll
      for (int w = 0; w < kEvWarps; ++w) run += w < warp ? sm.sums[w] : 0u;
      const uint32_t d[4] = {v.w, v.z, v.y, v.x};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (run < need && run + d[e] >= need) {
          sm.bin = (uint32_t)(bins - 1 - (4 * tid + e));
          sm.above = run;
        }
        run += d[e];
      }
      __syncthreads();
      prefix = (prefix << bits) | sm.bin;
      need -= sm.above;
    }
    thr = prefix;
    ties = need;
  }

  // ---- what each warp's part of the slice keeps, and where the rank's places begin
  const int part = ((whole / 128 + kEvWarps - 1) / kEvWarps) * 128, w0 = min(whole, warp * part), w1 = min(whole, w0 + part);
  // kept by their keys, and from bit 16 on ties
  auto count = [&](const uint4& k) {
    return (uint32_t)(k.x > thr) + (k.y > thr) + (k.z > thr) + (k.w > thr) +
           (((uint32_t)(k.x == thr) + (k.y == thr) + (k.z == thr) + (k.w == thr)) << 16);
  };
  uint32_t cnt = 0u;
#pragma unroll 4
  for (int i = w0 + 4 * lane; i < w1; i += 128) cnt += count(*reinterpret_cast<const uint4*>(keys + i));
  cnt = __reduce_add_sync(0xffffffffu, cnt);
  if (lane == 0) sm.wcnt[warp] = cnt;
  __syncthreads();
  uint32_t gt = 0u, eq = 0u;                          // before this warp's part
#pragma unroll
  for (int w = 0; w < kEvWarps; ++w) {
    gt += w < warp ? sm.wcnt[w] & 0xffffu : 0u;
    eq += w < warp ? sm.wcnt[w] >> 16 : 0u;
  }
  if constexpr (C > 1) {
    if (warp == kEvWarps - 1 && lane < C) {
      *ev_at<C>(&sm.cgt[rank], lane) = gt + (cnt & 0xffffu);
      *ev_at<C>(&sm.ceq[rank], lane) = eq + (cnt >> 16);
    }
    ev_sync<C>();
#pragma unroll
    for (int r = 0; r < C; ++r) {
      gt += r < rank ? sm.cgt[r] : 0u;
      eq += r < rank ? sm.ceq[r] : 0u;
    }
  }

  // ---- the kept positions, to the ranks that move them
  const uint32_t below = (1u << lane) - 1u;
  for (int i = w0 + 4 * lane; i < w1; i += 128) {
    const uint4 k4 = *reinterpret_cast<const uint4*>(keys + i);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    uint32_t x = gt, e = eq;                          // before the lane's four
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const uint32_t above = __ballot_sync(0xffffffffu, k[f] > thr), tie = __ballot_sync(0xffffffffu, k[f] == thr);
      x += __popc(above & below);
      e += __popc(tie & below);
      gt += __popc(above);
      eq += __popc(tie);
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const bool above = k[f] > thr, tie = k[f] == thr;
      if (above || (tie && e < ties)) {
        // place at: batch at / (256 C), rank (at / 256) % C
        const uint32_t at = x + min(e, ties);
        *ev_at<C>(&list[at / (kEvBatch * C) * kEvBatch + at % kEvBatch], at / kEvBatch % C) = (uint32_t)(p0 + i + f);
      }
      x += above;
      e += tie;
    }
  }
  if (kept)
    for (int i = K + rank * kEvThreads + tid; i < c.budget; i += C * kEvThreads) kept[i] = -1;
  ev_sync<C>();

  // ---- this rank's rows: where they are and go to (records' indexes in the pool, below 2^31), and their sums
  const int batches = (K + kEvBatch * C - 1) / (kEvBatch * C);
  auto place = [&](int i) { return i / kEvBatch * (kEvBatch * C) + rank * kEvBatch + i % kEvBatch; };   // of the rank's row i
  auto record = [&](const int32_t* table, int p) {
    return ((uint32_t)table[p >> c.block_shift] * c.n_kv + g) * bs + (p & (bs - 1));
  };
  constexpr int M = SPC_MAX_BUDGET / C / kEvThreads;  // rows a thread looks up
  float sums[M];
#pragma unroll
  for (int e = 0; e < M; ++e) {
    const int i = tid + e * kEvThreads, at = place(i);
    if (i >= batches * kEvBatch || at >= K) continue;
    const int p = (int)list[i];
    sums[e] = mass[p];
    if (kept) kept[at] = p;
    list[i] = record(from, p);
    dst[i] = record(to, at);
  }
  __syncthreads();
  // the 16-byte pieces of batch k, nine a row
  auto moves = [&](int k, auto f) {
    const int m = max(0, min(kEvBatch, K - place(k * kEvBatch)));
    const uint32_t* src_rec = list + k * kEvBatch;
    const uint32_t* dst_rec = dst + k * kEvBatch;
    uint8_t* buf = rows + (k & 1) * kEvBatch * kKv4Rec;
    int i = tid / 9, piece = tid - i * 9;
#pragma unroll
    for (int e = 0; e < (kEvBatch * 9 + kEvThreads - 1) / kEvThreads; ++e) {
      if (i < m && src_rec[i] != dst_rec[i]) f(src_rec[i], dst_rec[i], buf + i * kKv4Rec + piece * 16, piece * 16);
      i += kEvThreads / 9;
      piece += kEvThreads % 9;
      if (piece >= 9) {
        piece -= 9;
        ++i;
      }
    }
  };
  auto load = [&](int k) {
    moves(k, [&](uint32_t from_rec, uint32_t, uint8_t* at, int off) {
      cp_async16(at, c.cache + (size_t)from_rec * kKv4Rec + off, 16);
    });
    cp_async_commit();
  };
  if (batches > 0) load(0);
  for (int k = 0; k < batches; ++k) {
    if (k + 1 < batches) {
      load(k + 1);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    ev_sync<C>();                                     // before the first batch: every sum has been read, too
    moves(k, [&](uint32_t, uint32_t to_rec, uint8_t* at, int off) {
      stg_v4(c.cache + (size_t)to_rec * kKv4Rec + off, *reinterpret_cast<const uint4*>(at));
    });
    if (k + 2 < batches) __syncthreads();             // the next load goes to the same rows
  }
#pragma unroll
  for (int e = 0; e < M; ++e) {
    const int i = tid + e * kEvThreads, at = place(i);
    if (i < batches * kEvBatch && at < K) mass_next[at] = sums[e];
  }
  for (int i = K + rank * kEvThreads + tid; i < L; i += C * kEvThreads) mass_next[i] = 0.f;
  if (g == 0 && rank == 0 && tid == 0) c.len_next[b] = K;
}

template <int C>
static int ev_launch(EvArgs a, void* stream) {
  const Kv4EvictCall& c = a.c;
  const int most = c.max_blocks << c.block_shift, budget = most < c.budget ? most : c.budget;
  a.slice = ((most + C - 1) / C + 127) & ~127;
  a.share = (budget + kEvBatch * C - 1) / (kEvBatch * C) * kEvBatch;
  const uint32_t keys = (uint32_t)a.slice * 4, rows = (a.share > kEvBatch ? 2 : 1) * kEvBatch * kKv4Rec;
  a.list = (uint32_t)sizeof(EvShared) + (keys > rows ? keys : rows);
  const size_t smem = a.list + (size_t)a.share * 8;
  if (set_func_attr((const void*)kv4_evict_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SPC_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  cfg.gridDim = dim3((unsigned)(c.B * c.n_kv * C));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 1 : 0;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  return cudaLaunchKernelEx(&cfg, kv4_evict_kernel<C>, a) == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

int kv4_evict_launch(const Kv4EvictCall& c, void* stream) {
  EvArgs a{};
  a.c = c;
  const int most = c.max_blocks << c.block_shift, budget = most < c.budget ? most : c.budget;
  int C = 1;
  // us with 1, 2, 4 and 8 ranks, 8 heads: one request of 8000 positions to 2048 19.9, 17.9,
  // 13.8, 14.0; four of 12000 22.6, 19.7, 15.5, 23.1; sixteen of 8000 23.9, 28.4, 38.9,
  // 84.0; one of 1088 to 1024 11.4, 12.2, 11.3, 13.5
  while (C < kEvCluster && C * kEvSlice < most) C *= 2;
  while (C < kEvCluster && C * kEvBatch < budget && 2 * C * c.B * c.n_kv <= 152) C *= 2;
  switch (C) {
    case 1: return ev_launch<1>(a, stream);
    case 2: return ev_launch<2>(a, stream);
    case 4: return ev_launch<4>(a, stream);
    default: return ev_launch<8>(a, stream);
  }
}

}  // namespace spc
