// Causal attention over whole packed prompts on the 5th-generation tensor
// cores: out_i = sum_{j <= i} softmax_j(scale q_i.k_j) v_j within a sequence.
//
// Rows are (token, query head of the group) pairs: a 128-row tile holds 128/G
// tokens x G heads of one KV head, so that every group size fills the tile,
// its causal edge is only 128/G tokens wide and K and V are read once for the
// whole group. A work item is two such tiles (A and B, consecutive tokens) of
// one (sequence, KV head) against that head's keys in blocks of 128:
//   S[128][128] = Q K^T     Q, K in shared memory (TMA, 128-byte swizzle)
//   O[128][128] += P V      P in tensor memory over S's columns, V MN-major
// The tensor cores work on one tile while the other one's softmax runs: the
// issue order is S_A S_B, then PV_A(j) S_A(j+1) PV_B(j) S_B(j+1), ...; the
// tensor pipe executes one thread's MMAs in order, so S(j+1) does not
// overwrite P(j) before PV(j) has read it.
// Softmax: one thread a row (no exchange between threads), in base 2. The
// running maximum is raised only when a logit passes it by more than 8 (P stays
// below 2^8), and only then is the row of O rescaled. P is rounded to bf16, V's
// type (relative error at most 2^-8, independent from key to key), its sum is
// that of the fp32 values; S, O, maximum and sum are fp32.
//
// What a row does not see must not reach it, NaN and infinities included. In S
// masked columns are replaced. In P V they meet P = 0, which a non-finite V
// defeats: V rows behind the sequence's end are zeroed in shared memory before
// they are used, and a row whose sum is finite but whose result is not, though
// the V that it sees do not explain that (a non-finite V behind it, or weights
// above 1 on values near the type's largest), is computed again by a warp from
// global memory over exactly the keys it sees. So is a row whose maximum passes 2^26 in
// base 2: a weight is 2^(s scale - m) with m rounded to fp32, and beyond 2^31 that
// rounding alone passes the range of the weights.
//
// One CTA per SM, persistent over items ordered by the number of key blocks,
// longest first, and dealt to the CTAs in a snake:
//   warps 0-3, 4-7  softmax and epilogue of tile A, B
//   warp 8          tensor memory, MMA issue (one lane)
//   warp 9          item schedule, TMA loads (Q per tile, K and V ring)
//   warp 10         gate: passes the loads' arrival on to the MMA warp's barriers
// Bound: the tensor pipe. A block of keys against both tiles is four products
// of 512 cycles; a period was 2650 cycles in a clock trace, of which the chain
// of one tile (its S, 1130 cycles from S to P, the MMA warp's wait, its PV) is
// what is left. Measured, 32 heads on 8 KV heads: one sequence of 16384 tokens
// (2199 GFLOP) 1.20-1.31 ms, 0.88-0.96 of the measured matrix rate, and 1.32-1.35
// ms in a long run, where the power limit lowers the clock (0.94-0.97 of the rate
// measured so); 4096 tokens (137 GFLOP) 91 us, 0.79; 16 sequences of 1 to 700 tokens
// 41 us (their bytes alone are 17):
// an item has one to six blocks, and its first S, its epilogue (about 3000
// cycles) and the sixth item of a few CTAs weigh as much as the blocks.
// Every wait is bounded: a role whose wait gives up records SPC_ERR_TIMEOUT
// and leaves, the others' waits then give up in turn; copies land and MMAs
// complete before the CTA releases its tensor memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <type_traits>

#include "spc_device.cuh"
#include "spc_internal.h"
#include "spc_tc.cuh"

namespace spc {

constexpr int kPaKeys = 128;                          // keys a block
constexpr uint32_t kPaTile = 128 * kRowBytes;         // 32 KiB: a Q, K or V tile
constexpr uint32_t kPaBlock = kPaTile / 2;            // its 64-value half
constexpr int kPaStages = 2;                          // ring of (V of a block, K of the next one)
constexpr int kPaItems = 2;                           // item ring
constexpr int kPaSoftWarps = 8;
constexpr int kPaWarpMma = 8, kPaWarpTma = 9, kPaWarpGate = 10;
constexpr int kPaThreads = 384;                       // warp 11 fills the third warpgroup
// registers a thread: 168 at launch (384 threads); the softmax warpgroups take
// 208, the third keeps 88 (2 * 208 + 88 = 3 * 168)
constexpr int kPaRegSoft = 208, kPaRegRest = 88;
constexpr int kPaCtas = 152;
constexpr float kPaHeadroom = 8.f;
constexpr float kPaLarge = 67108864.f;                // 2^26
// clock cycles, some 4 s: a warp whose 32 rows are all computed again over 262144
// keys takes 1.3 s, for which the other roles wait
constexpr long long kPaWait = 8000000000ll;
constexpr int kPaTmemCols = 512;                      // S_A, S_B, O_A, O_B
constexpr uint32_t kPaColO = 256;
constexpr uint32_t kPaIdescS = umma_idesc_bf16(128, kPaKeys, false);
constexpr uint32_t kPaIdescO = umma_idesc_bf16(128, kD, true);

// shared memory, from a 1024-byte aligned base
constexpr uint32_t kPaOffQ = 0;                                       // [2] tiles
constexpr uint32_t kPaOffKv = kPaOffQ + 2 * kPaTile;
constexpr uint32_t kPaOffK0 = kPaOffKv + kPaStages * 2 * kPaTile;     // an item's first K
constexpr uint32_t kPaOffItem = kPaOffK0 + kPaTile;                   // [kPaItems] PaItem
constexpr uint32_t kPaOffBar = kPaOffItem + kPaItems * 32;
constexpr int kPaBars = 2 * kPaStages + 2 + 2 * kPaItems + 2 * 5 + 1;
constexpr size_t kPaSmem = 1024 + kPaOffBar + kPaBars * 8 + 16;

struct PaArgs {
  PromptAttnCall c;
  int G, gshift, tpm;      // heads a group, its log2, tokens a tile
  int* status;
  long long wait_limit;
  int starve;              // test builds: no copy is issued, so that every wait runs out
};

struct PaItem {
  int start, len;          // the sequence's first row and length; len < 0: no more items
  int g, t0;               // KV head, first token (in the sequence) of tile A
  int nA, nB;              // key blocks of the tiles
};

__device__ __forceinline__ bool pa_wait(const PaArgs& a, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.wait_limit));
}
// A shared-memory matrix descriptor (spc_tc.cuh) in two words: the low one
// holds the address (in 16-byte units) and the leading byte offset, the high
// one is the same for every operand here (1024 bytes between 8-row groups,
// 128-byte swizzle). K-major operands have leading offset 16, V's 64-value
// blocks lie kPaBlock apart.
constexpr uint32_t kPaDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kPaDescVLo = ((kPaBlock >> 4) - 1u) << 16;      // on top of a K-major low word
__device__ __forceinline__ uint32_t pa_desc_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint64_t pa_desc(uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; }
__device__ __forceinline__ float pa_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// tcgen05.wait::ld, with the values it makes valid passed through it
__device__ __forceinline__ void pa_ld_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29])
               :: "memory");
  asm volatile("" : "+f"(v[30]), "+f"(v[31]));
}
// 32 logits of a row: weights 2^(s scale - m) to 16 packed columns, their sum, their largest logit
__device__ __forceinline__ void pa_weights(const float* s, float scale2, float m, float2 (&sum)[2], uint32_t tp) {
  const float2 sc = make_float2(scale2, scale2), nm = make_float2(-m, -m);
  uint32_t p[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float2 x = fma2(make_float2(s[2 * e], s[2 * e + 1]), sc, nm);
    x.x = ex2_approx(x.x);
    x.y = ex2_approx(x.y);
    sum[e & 1] = add2(sum[e & 1], x);
    p[e] = pack_bf16(x.x, x.y);
  }
  tmem_st16(tp, p);
}
__device__ __forceinline__ void pa_max32(const float* s, float (&mx)[4]) {
#pragma unroll
  for (int e = 0; e < 32; e += 8)
#pragma unroll
    for (int f = 0; f < 4; ++f) mx[f] = pa_max3(mx[f], s[e + f], s[e + 4 + f]);
}
__device__ __forceinline__ void pa_tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
               :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool pa_not_finite(uint32_t bf) { return (bf & 0x7f80u) == 0x7f80u; }

// One row by one warp, from global memory, over the keys it sees (h is the
// query head, g its KV head): the result of lane l is dims 4l .. 4l + 3, held
// as a running mean, so that it does not overflow where the mean does not. The
// maximum is that of the products q.k, without the scale.
__device__ void pa_row_again(const PaArgs& a, int start, int qpos, int h, int g) {
  constexpr int U = 8;                                 // keys a step, their loads in flight together
  const PromptAttnCall& c = a.c;
  const int lane = threadIdx.x & 31, t = start + qpos;
  const uint2 qw = *reinterpret_cast<const uint2*>(c.q + t * c.q_stride + (size_t)h * kD + 4 * lane);
  const float q0 = bf_lo(qw.x), q1 = bf_hi(qw.x), q2 = bf_lo(qw.y), q3 = bf_hi(qw.y);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = start; j <= t; j += U) {
    uint2 k[U], v[U];
    float x[U], M = m;
#pragma unroll
    for (int e = 0; e < U; ++e) {
      k[e] = v[e] = make_uint2(0u, 0u);
      if (j + e <= t) {
        k[e] = *reinterpret_cast<const uint2*>(c.k + (j + e) * c.k_stride + (size_t)g * kD + 4 * lane);
        v[e] = *reinterpret_cast<const uint2*>(c.v + (j + e) * c.v_stride + (size_t)g * kD + 4 * lane);
      }
    }
#pragma unroll
    for (int e = 0; e < U; ++e) {
      x[e] = warp_sum(q0 * bf_lo(k[e].x) + q1 * bf_hi(k[e].x) + q2 * bf_lo(k[e].y) + q3 * bf_hi(k[e].y));
      if (j + e > t) x[e] = -INFINITY;
      M = fmaxf(M, x[e]);
    }
    const float Ms = M == -INFINITY ? 0.f : M, old = l * exp2f((m - Ms) * c.scale2);
    l = old;
#pragma unroll
    for (int e = 0; e < U; ++e) l += x[e] = exp2f((x[e] - Ms) * c.scale2);
    m = M;
    if (l == 0.f) continue;                            // nothing but -inf so far
    const float r = 1.f / l;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] *= old * r;
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const float w = x[e] * r;
      if (j + e > t) break;
      o[0] += w * bf_lo(v[e].x);
      o[1] += w * bf_hi(v[e].x);
      o[2] += w * bf_lo(v[e].y);
      o[3] += w * bf_hi(v[e].y);
    }
  }
  if (l == 0.f) o[0] = o[1] = o[2] = o[3] = NAN;
  *reinterpret_cast<uint2*>(c.out + ((size_t)t * c.n_q + h) * kD + 4 * lane) =
      make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
}

// The rows of a warp's lanes in `large` are computed again. Those in `again`
// have results that are not finite: a dim in which a V that the row sees is not
// finite, and none behind it in the row's block of keys, stays; a row with
// another such dim is computed again. One pass over V tells each dim's first
// non-finite key, one over the block the last, for all rows.
__device__ void pa_rows_again(const PaArgs& a, uint32_t again, uint32_t large, int start, int len, int qpos, int h, int g) {
  constexpr int U = 8;
  const PromptAttnCall& c = a.c;
  const int lane = threadIdx.x & 31;
  again &= ~large;
  int first[4] = {INT_MAX, INT_MAX, INT_MAX, INT_MAX}, last[4] = {-1, -1, -1, -1};
  // keys j0 .. j1 - 1, until `first` is known in every dim if that is all that is asked for
  auto scan = [&](int j0, int j1, bool all) {
    for (int j = j0; j < j1; j += U) {
      uint2 v[U];
#pragma unroll
      for (int e = 0; e < U; ++e) {
        v[e] = make_uint2(0u, 0u);
        if (j + e < j1)
          v[e] = *reinterpret_cast<const uint2*>(c.v + (start + j + e) * c.v_stride + (size_t)g * kD + 4 * lane);
      }
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const bool bad[4] = {pa_not_finite(v[e].x), pa_not_finite(v[e].x >> 16), pa_not_finite(v[e].y), pa_not_finite(v[e].y >> 16)};
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          if (!bad[d]) continue;
          first[d] = min(first[d], j + e);
          last[d] = max(last[d], j + e);
        }
      }
      if (!all && __all_sync(0xffffffffu, max(max(first[0], first[1]), max(first[2], first[3])) < INT_MAX)) break;
    }
  };
  if (again) {
    // the tokens of a warp's rows lie in one block of keys
    const int top = __reduce_max_sync(0xffffffffu, again >> lane & 1 ? qpos : 0), b0 = top / kPaKeys * kPaKeys;
    scan(0, b0, false);
    scan(b0, min(b0 + kPaKeys, len), true);
  }
  __syncwarp();                                        // the rows' results are read and written by other lanes
  for (uint32_t rows = again | large; rows; rows &= rows - 1) {
    const int src = __ffs(rows) - 1;
    const int qp = __shfl_sync(0xffffffffu, qpos, src), hh = __shfl_sync(0xffffffffu, h, src);
    if (large >> src & 1) {
      pa_row_again(a, start, qp, hh, g);
      continue;
    }
    const uint2 o = __ldcg(reinterpret_cast<const uint2*>(c.out + ((size_t)(start + qp) * c.n_q + hh) * kD) + lane);
    const uint32_t w[4] = {o.x, o.x >> 16, o.y, o.y >> 16};
    bool open = false;
#pragma unroll
    for (int d = 0; d < 4; ++d) open = open || (pa_not_finite(w[d]) && (first[d] > qp || last[d] > qp));
    if (__any_sync(0xffffffffu, open)) pa_row_again(a, start, qp, hh, g);
  }
}

__global__ void __launch_bounds__(kPaThreads, 1) prompt_attn_kernel(const __grid_constant__ CUtensorMap qmap,
                                                                    const __grid_constant__ CUtensorMap kmap,
                                                                    const __grid_constant__ CUtensorMap vmap,
                                                                    const PaArgs a) {
  extern __shared__ uint8_t pa_raw[];
  const uint32_t raw_addr = smem_u32(pa_raw);
  uint8_t* base = pa_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  volatile PaItem* items = reinterpret_cast<volatile PaItem*>(base + kPaOffItem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + kPaOffBar);
  uint64_t* kvfull = bars;                    // [kPaStages] TMA bytes
  uint64_t* kvfree = kvfull + kPaStages;      // [kPaStages] commit after the last MMA that reads the stage
  uint64_t* k0full = kvfree + kPaStages;      // TMA bytes
  uint64_t* k0free = k0full + 1;              // commit after the item's first S
  uint64_t* ifull = k0free + 1;               // [kPaItems] item written
  uint64_t* ifree = ifull + kPaItems;         // [kPaItems] MMA, gate and softmax warps have read it
  uint64_t* qfull = ifree + kPaItems;         // [2] TMA bytes
  uint64_t* qfree = qfull + 2;                // [2] commit after the tile's last S
  uint64_t* sfull = qfree + 2;                // [2] commit: S in tensor memory
  uint64_t* pfull = sfull + 2;                // [2] 4 softmax warps: P written, O rescaled; gate: V and the next K are there
  uint64_t* ofull = pfull + 2;                // [2] commit: the item's last PV done
  uint64_t* drain = ofull + 2;                // commit after the last MMA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPaStages; ++s) {
      mbar_init(&kvfull[s], 1);
      mbar_init(&kvfree[s], 1);
    }
    mbar_init(k0full, 1);
    mbar_init(k0free, 1);
    for (int s = 0; s < kPaItems; ++s) {
      mbar_init(&ifull[s], 1);
      mbar_init(&ifree[s], kPaSoftWarps + 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&qfull[s], 1);
      mbar_init(&qfree[s], 1);
      mbar_init(&sfull[s], 1);
      mbar_init(&pfull[s], kPaSoftWarps / 2 + 1);
      mbar_init(&ofull[s], 1);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == kPaWarpMma) tmem_alloc<kPaTmemCols>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t qs = smem_u32(base + kPaOffQ), kvs = smem_u32(base + kPaOffKv);
  bool dead = false;

  if (warp == kPaWarpTma) {
    // ================= schedule and loads
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kPaRegRest));
    const PromptAttnCall& c = a.c;
    int start[2], len[2], nb[2];
    const int per = 2 * a.tpm;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int b = 32 * e + lane;
      start[e] = len[e] = 0;
      if (b < c.B) {
        start[e] = max(0, min(c.cu[b], c.T));
        len[e] = max(start[e], min(c.cu[b + 1], c.T)) - start[e];
      }
      nb[e] = (len[e] + per - 1) / per;
    }
    // items with block index >= q, over n_kv
    auto at_least = [&](int q) {
      return (int)__reduce_add_sync(0xffffffffu, (unsigned)(max(0, nb[0] - q) + max(0, nb[1] - q)));
    };
    const int most = (int)__reduce_max_sync(0xffffffffu, (unsigned)max(nb[0], nb[1]));
    const long long n_items = (long long)at_least(0) * c.n_kv;
    int it = 0, nkv = 0, nk0 = 0, nq[2] = {0, 0};
    auto acquire = [&](uint64_t* bar, uint32_t parity) {
      if (!dead && !pa_wait(a, bar, parity)) {
        if (lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
        dead = true;
      }
    };
    for (int round = 0;; ++round, ++it) {
      // snake: even rounds in CTA order, odd ones in reverse
      const int cta = (round & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
      const long long k = (long long)round * gridDim.x + cta;
      PaItem x;
      x.len = -1;
      if (k < n_items && !dead) {
        const int r0 = (int)(k / c.n_kv), g = (int)(k - (long long)r0 * c.n_kv);
        int lo = 0, hi = most;                        // at_least(lo) > r0 >= at_least(hi)
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (at_least(mid) > r0) lo = mid; else hi = mid;
        }
        // the (r0 - at_least(lo + 1))-th sequence that has a block lo
        int r = r0 - at_least(lo + 1);
        const uint32_t m0 = __ballot_sync(0xffffffffu, nb[0] > lo), m1 = __ballot_sync(0xffffffffu, nb[1] > lo);
        const int n0 = __popc(m0), e = r >= n0 ? 1 : 0;
        if (e) r -= n0;
        const int src = __fns(e ? m1 : m0, 0, r + 1);
        x.start = __shfl_sync(0xffffffffu, e ? start[1] : start[0], src);
        x.len = __shfl_sync(0xffffffffu, e ? len[1] : len[0], src);
        x.g = g;
        x.t0 = lo * per;
        x.nA = (min(x.t0 + a.tpm, x.len) + kPaKeys - 1) / kPaKeys;
        x.nB = x.t0 + a.tpm < x.len ? (min(x.t0 + per, x.len) + kPaKeys - 1) / kPaKeys : 0;
      }
      const int is = it % kPaItems;
      acquire(&ifree[is], ((it / kPaItems) & 1) ^ 1);
      if (lane == 0) {
        items[is].start = x.start; items[is].len = x.len; items[is].g = x.g; items[is].t0 = x.t0;
        items[is].nA = x.nA; items[is].nB = x.nB;
        mbar_arrive(&ifull[is]);
      }
      __syncwarp();
      if (x.len < 0) break;
#ifdef SPC_TEST_HOOKS
      if (a.starve) break;
#endif
      const int n = max(x.nA, x.nB);
      auto load_q = [&](int i) {
        acquire(&qfree[i], (nq[i] & 1) ^ 1);
        if (dead) return;
        ++nq[i];
        if (lane == 0) {
          mbar_arrive_expect_tx(&qfull[i], kPaTile);
          const int row = x.start + x.t0 + i * a.tpm;
          pa_tma_3d(qs + i * kPaTile, &qmap, 0, x.g << a.gshift, row, &qfull[i]);
          pa_tma_3d(qs + i * kPaTile + kPaBlock, &qmap, 64, x.g << a.gshift, row, &qfull[i]);
        }
      };
      auto load = [&](const CUtensorMap* map, uint32_t dst, int j, uint64_t* bar) {
        pa_tma_3d(dst, map, 0, x.g, x.start + j * kPaKeys, bar);
        pa_tma_3d(dst + kPaBlock, map, 64, x.g, x.start + j * kPaKeys, bar);
      };
      load_q(0);
      acquire(k0free, (nk0 & 1) ^ 1);
      if (!dead) {
        ++nk0;
        if (lane == 0) {
          mbar_arrive_expect_tx(k0full, kPaTile);
          load(&kmap, qs + (kPaOffK0 - kPaOffQ), 0, k0full);
        }
      }
      if (x.nB) load_q(1);
      for (int j = 0; j < n; ++j) {
        const int st = nkv % kPaStages;
        acquire(&kvfree[st], ((nkv / kPaStages) & 1) ^ 1);
        if (dead) break;
        ++nkv;
        if (lane == 0) {
          const uint32_t dst = kvs + (uint32_t)st * 2 * kPaTile;
          mbar_arrive_expect_tx(&kvfull[st], j + 1 < n ? 2 * kPaTile : kPaTile);
          load(&vmap, dst, j, &kvfull[st]);
          if (j + 1 < n) load(&kmap, dst + kPaTile, j + 1, &kvfull[st]);
        }
      }
    }
    // every copy lands before the CTA ends (they have, unless a role gave up)
    if (lane == 0) {
      for (int k = max(0, nkv - kPaStages); k < nkv; ++k)
        mbar_wait_bounded(&kvfull[k % kPaStages], (k / kPaStages) & 1, a.wait_limit);
      if (nk0 > 0) mbar_wait_bounded(k0full, (nk0 - 1) & 1, a.wait_limit);
      for (int i = 0; i < 2; ++i)
        if (nq[i] > 0) mbar_wait_bounded(&qfull[i], (nq[i] - 1) & 1, a.wait_limit);
    }
    __syncwarp();
  } else if (warp == kPaWarpMma) {
    // ================= MMA issue. The whole warp runs the loop, so that its
    // values stay warp-uniform (operands of tcgen05.mma are uniform registers;
    // built by a single lane they cost about 90 cycles an instruction and held
    // the tensor pipe at 60%); one elected lane issues.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kPaRegRest));
    auto acquire = [&](uint64_t* bar, uint32_t parity) {
      if (!dead && !pa_wait(a, bar, parity)) {
        if (lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
        dead = true;
      }
    };
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    int nkv = 0, nk0 = 0, nq[2] = {0, 0}, np[2] = {0, 0};
    // S of tile i against the K tile whose descriptor is kd; last: of the item
    auto issue_s = [&](auto tile, uint32_t kd, bool last) {
      constexpr int i = decltype(tile)::value;
      if (elect_one()) {
        const uint32_t qd = pa_desc_lo(qs + i * kPaTile);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t off = (uint32_t)(kk >> 2) * (kPaBlock >> 4) + (uint32_t)(kk & 3) * 2;
          umma_f16(tm + i * kPaKeys, pa_desc(qd + off, kPaDescHi), pa_desc(kd + off, kPaDescHi), kPaIdescS, kk ? 1u : 0u);
        }
        umma_commit(&sfull[i]);
        if (last) umma_commit(&qfree[i]);
      }
      __syncwarp();
    };
    // PV of block j of tile i, then S of block j + 1. The tensor pipe queues
    // only a few MMAs, so nothing waits between the two
    auto issue = [&](auto tile, uint32_t st, int j, int n, uint64_t* stage_free) {
      constexpr int i = decltype(tile)::value;
      // mostly there: tested before it is waited for (90 against 190 cycles)
      if (!__all_sync(0xffffffffu, mbar_test(&pfull[i], np[i] & 1))) acquire(&pfull[i], np[i] & 1);
      ++np[i];
      if (dead) return;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t vd = st + kPaDescVLo, kd = st + (kPaTile >> 4), qd = pa_desc_lo(qs + i * kPaTile);
#pragma unroll
        for (int kk = 0; kk < kPaKeys / 16; ++kk)
          umma_f16_tmem_a(tm + kPaColO + i * kD, tm + i * kPaKeys + kk * 8, pa_desc(vd + (uint32_t)kk * 128, kPaDescHi),
                          kPaIdescO, kk ? 1u : (j ? 1u : 0u));
        if (j + 1 < n) {
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk) {
            const uint32_t off = (uint32_t)(kk >> 2) * (kPaBlock >> 4) + (uint32_t)(kk & 3) * 2;
            umma_f16(tm + i * kPaKeys, pa_desc(qd + off, kPaDescHi), pa_desc(kd + off, kPaDescHi), kPaIdescS, kk ? 1u : 0u);
          }
          umma_commit(&sfull[i]);
          if (j + 2 == n) umma_commit(&qfree[i]);
        } else {
          umma_commit(&ofull[i]);
        }
        if (stage_free) umma_commit(stage_free);
      }
      __syncwarp();
    };
    constexpr std::integral_constant<int, 0> tA{};
    constexpr std::integral_constant<int, 1> tB{};
    for (int it = 0;; ++it) {
      const int is = it % kPaItems;
      acquire(&ifull[is], (it / kPaItems) & 1);
      if (dead) break;
      const int nA = items[is].nA, nB = items[is].nB, len = items[is].len;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
      if (len < 0) break;
      const int n = max(nA, nB);
      const uint32_t k0 = pa_desc_lo(qs + (kPaOffK0 - kPaOffQ));
      acquire(k0full, nk0++ & 1);
      acquire(&qfull[0], nq[0]++ & 1);
      if (dead) break;
      tc_fence_after();
      issue_s(tA, k0, nA == 1);
      if (nB) {
        acquire(&qfull[1], nq[1]++ & 1);
        if (dead) break;
        issue_s(tB, k0, nB == 1);
      }
      if (elect_one()) umma_commit(k0free);
      __syncwarp();
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const int st = nkv % kPaStages;
        ++nkv;
        const uint32_t sd = pa_desc_lo(kvs) + (uint32_t)st * (2 * kPaTile >> 4);
        if (j < nA) issue(tA, sd, j, nA, j < nB ? nullptr : &kvfree[st]);
        if (j < nB) issue(tB, sd, j, nB, &kvfree[st]);
      }
      if (dead) break;
    }
    // tensor memory is released below: every MMA has completed (the softmax
    // warps wait for each item's last one, unless something gave up)
    if (elect_one()) umma_commit(drain);
    __syncwarp();
    pa_wait(a, drain, 0);
  } else if (warp < kPaSoftWarps) {
    // ================= softmax and epilogue of tile i, one row a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kPaRegSoft));
    const PromptAttnCall& c = a.c;
    const int i = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + i * kPaKeys, to = tmem + lanes + kPaColO + i * kD;
    int n_s = 0, n_o = 0, nkv = 0;
    auto acquire = [&](uint64_t* bar, uint32_t parity) {
      if (!dead && !pa_wait(a, bar, parity)) {
        if (lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
        dead = true;
      }
    };
    for (int it = 0;; ++it) {
      const int is = it % kPaItems;
      acquire(&ifull[is], (it / kPaItems) & 1);
      if (dead) break;
      const int start = items[is].start, len = items[is].len, g = items[is].g, nA = items[is].nA, nB = items[is].nB;
      const int t0 = items[is].t0 + i * a.tpm;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
      if (len < 0) break;
      const int n = i ? nB : nA, nmax = max(nA, nB);
      const int qpos = t0 + (row >> a.gshift);
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        acquire(&sfull[i], n_s & 1);
        if (dead) break;
        tc_fence_after();
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // raises the row's maximum to M where that is needed
        auto raise = [&](float M) {
          float alpha = 1.f;
          const bool up = M > m + kPaHeadroom;
          if (up) {
            alpha = m == -INFINITY ? 0.f : ex2_approx(m - M);
            l *= alpha;
            m = M;
          }
          if (j > 0 && __any_sync(0xffffffffu, up)) {
            // O holds earlier blocks; their PV is done, for this block's S was
            // issued behind it and the commit it came with covers both
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {
              float o[16];
              tmem_ld16(to + 16 * q, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= alpha;
              tmem_st16(to + 16 * q, o);
            }
          }
        };
        if ((j + 1) * kPaKeys <= t0 + 1 && !__any_sync(0xffffffffu, m == -INFINITY)) {
          // every row sees the whole block and has a maximum: weights against
          // it at once, while the block's own maximum is being found
          float s[128];
          tmem_ld32(ts, *reinterpret_cast<float (*)[32]>(s));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            pa_ld_wait(s + 32 * q);
            if (q < 3) tmem_ld32(ts + 32 * (q + 1), *reinterpret_cast<float (*)[32]>(s + 32 * (q + 1)));
            pa_max32(s + 32 * q, mx);
            pa_weights(s + 32 * q, c.scale2, m, sum, ts + 16 * q);
          }
          const float M = pa_max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * c.scale2;
          if (__any_sync(0xffffffffu, M > m + kPaHeadroom)) {
            // the weights go to the same columns again, and stores to tensor
            // memory are asynchronous: the first ones have to be there
            tmem_st_wait();
            raise(M);
            sum[0] = sum[1] = make_float2(0.f, 0.f);
#pragma unroll
            for (int q = 0; q < 4; ++q) pa_weights(s + 32 * q, c.scale2, m, sum, ts + 16 * q);
          }
        } else {
          // An item's first block and its last one: S is read twice, in chunks
          // of 32 columns, without the chunks that no row of the warp sees (64
          // sequences of 100 tokens: 39.5 -> 35.1 us; all four chunks from
          // registers, 39.5, and in loops, 42.9). Columns 0 .. seen are visible,
          // 0 .. seen0 to every row of the warp, none behind seen1 to any; the
          // tile's tokens lie in one block of keys, so that seen1 >= 0.
          const int w0 = (warp & 3) * 32, at = t0 - j * kPaKeys;
          const int seen = qpos - j * kPaKeys, seen0 = at + (w0 >> a.gshift), seen1 = at + ((w0 + 31) >> a.gshift);
          auto load = [&](int q, float (&v)[32]) {
            tmem_ld32(ts + 32 * q, v);
            pa_ld_wait(v);
            if (seen0 < 32 * q + 31) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * q + e > seen) v[e] = -INFINITY;
            }
          };
          const int nq = min(4, seen1 / 32 + 1);
#pragma unroll 1
          for (int q = 0; q < nq; ++q) {
            float v[32];
            load(q, v);
            pa_max32(v, mx);
          }
          raise(pa_max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * c.scale2);
          const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll 1
          for (int q = 0; q < nq; ++q) {
            float v[32];
            load(q, v);
            pa_weights(v, c.scale2, mm, sum, ts + 16 * q);
          }
          const uint32_t none[16] = {};
#pragma unroll 1
          for (int q = nq; q < 4; ++q) tmem_st16(ts + 16 * q, none);
        }
        l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
        if ((j + 1) * kPaKeys > len) {
          // V rows behind the sequence's end: zeros
          const int v = nkv + j, vs = v % kPaStages;
          acquire(&kvfull[vs], (v / kPaStages) & 1);
          if (dead) break;
          if (row >= len - j * kPaKeys) {
            uint4* r0 = reinterpret_cast<uint4*>(base + kPaOffKv + vs * 2 * kPaTile + row * 128);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              r0[e] = make_uint4(0u, 0u, 0u, 0u);
              r0[e + kPaBlock / 16] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[i]);
        ++n_s;
      }
      if (dead) break;
      nkv += nmax;
      if (n == 0) continue;
      // ---- epilogue
      acquire(&ofull[i], n_o & 1);
      if (dead) break;
      ++n_o;
      tc_fence_after();
      const bool live = qpos < len;
      const int h = (g << a.gshift) + (row & (a.G - 1));
      uint16_t* dst = c.out + ((size_t)(start + qpos) * c.n_q + h) * kD;
      const float r = 1.f / l;
      const bool wide = (reinterpret_cast<uintptr_t>(c.out) & 31u) == 0;   // whole sectors a store
      // (an infinite maximum is the products' own, unless the scale can have made it so)
      const bool large = live && fabsf(m) > kPaLarge && (fabsf(m) < INFINITY || c.scale2 > 1.f);
      bool odd = large;                                // or a value that is not finite
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        float o[32];
        tmem_ld32(to + 32 * q, o);
        tmem_ld_wait();
        if (live) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t w[8];
#pragma unroll
            for (int f = 0; f < 8; ++f) {
              const float x0 = o[16 * e + 2 * f] * r, x1 = o[16 * e + 2 * f + 1] * r;
              odd = odd || !(fabsf(x0) < INFINITY) || !(fabsf(x1) < INFINITY);
              w[f] = pack_bf16(x0, x1);
            }
            uint16_t* d = dst + 32 * q + 16 * e;
            if (wide) {
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" :: "l"(d), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                           "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
            } else {
              stg_v4(d, make_uint4(w[0], w[1], w[2], w[3]));
              stg_v4(d + 8, make_uint4(w[4], w[5], w[6], w[7]));
            }
          }
        }
      }
      tc_fence_before();
      const uint32_t again = __ballot_sync(0xffffffffu, live && odd && (l < INFINITY || large));
      if (again) pa_rows_again(a, again, __ballot_sync(0xffffffffu, large), start, len, qpos, h, g);
    }
  } else if (warp == kPaWarpGate) {
    // ================= gate: passes the arrival of V_j and K_(j+1) on to the
    // tiles' P barriers, so that the MMA warp waits once a batch
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kPaRegRest));
    auto acquire = [&](uint64_t* bar, uint32_t parity) {
      if (!dead && !pa_wait(a, bar, parity)) {
        if (lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
        dead = true;
      }
    };
    int nkv = 0, np[2] = {0, 0};
    for (int it = 0; !dead; ++it) {
      const int is = it % kPaItems;
      acquire(&ifull[is], (it / kPaItems) & 1);
      if (dead) break;
      const int nA = items[is].nA, nB = items[is].nB, len = items[is].len;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
      if (len < 0) break;
      for (int j = 0; j < max(nA, nB); ++j, ++nkv) {
        acquire(&kvfull[nkv % kPaStages], (nkv / kPaStages) & 1);
        if (dead) break;
        // one arrival a phase: the block before's P has been written
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (j >= (i ? nB : nA)) continue;
          if (np[i] > 0) acquire(&pfull[i], (np[i] - 1) & 1);
          if (dead) break;
          ++np[i];
          if (lane == 0) mbar_arrive(&pfull[i]);
        }
        if (dead) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kPaRegRest));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kPaWarpMma) {
    tc_fence_after();
    tmem_dealloc<kPaTmemCols>(tmem);
  }
}

size_t prompt_attn_workspace(int, int, int, int) { return 256; }

int prompt_attn_launch(const PromptAttnCall& c, void* workspace, void* stream) {
  PaArgs a{};
  a.c = c;
  a.G = c.n_q / c.n_kv;
  while ((1 << a.gshift) < a.G) ++a.gshift;
  a.tpm = 128 >> a.gshift;
  a.status = static_cast<int*>(workspace);
  a.wait_limit = kPaWait;
#ifdef SPC_TEST_HOOKS
  a.starve = paged_starve(&a.wait_limit) ? 1 : 0;
#endif
  CUtensorMap qmap, kmap, vmap;
  auto map = [&](CUtensorMap* m, const void* p, int heads, int64_t stride, uint32_t bh, uint32_t bt) {
    const uint64_t dims[3] = {(uint64_t)kD, (uint64_t)heads, (uint64_t)c.T};
    const uint64_t strides[2] = {(uint64_t)kRowBytes, (uint64_t)stride * 2};
    const uint32_t box[3] = {64, bh, bt};
    return tensor_map_bf16_sw128(m, p, 3, dims, strides, box);
  };
  if (!map(&qmap, c.q, c.n_q, c.q_stride, a.G, a.tpm) || !map(&kmap, c.k, c.n_kv, c.k_stride, 1, kPaKeys) ||
      !map(&vmap, c.v, c.n_kv, c.v_stride, 1, kPaKeys))
    return SPC_ERR_CUDA;
  if (set_func_attr((const void*)prompt_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPaSmem) != cudaSuccess)
    return SPC_ERR_CUDA;
  const long long most = ((long long)c.T / (2 * a.tpm) + c.B) * c.n_kv;      // items at most
  const int grid = (int)(most < kPaCtas ? most : kPaCtas);
  prompt_attn_kernel<<<grid, kPaThreads, kPaSmem, static_cast<cudaStream_t>(stream)>>>(qmap, kmap, vmap, a);
  return cudaGetLastError() == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

}  // namespace spc
