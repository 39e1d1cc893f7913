// The attention weight that the positions of the paged 4-bit cache receive from
// chunks of new tokens, on the 5th-generation tensor cores:
// mass_p = keep prev_p + sum_i exp(scale q_i.K_p - lse_i) over the rows that see p.
//
// With the rows' lse known the weights need no second pass, so the positions
// stay put and the rows stream past them. An item is two tiles (A and B) of 128
// positions of one (request, KV head), dequantised once, against the 128-row
// tiles of (token, query head of the group) pairs that see them:
//   S^T[128 positions][N rows] = K Q^T     K in tensor memory, Q in shared memory
// A position is one thread's throughout: one dequantises its record into its own
// tensor memory lane (no swizzle, and the shared memory is left to a ring of row
// tiles that hides their loads), another reads its row of S^T into registers,
// takes the exponentials and adds them up, so that nothing is exchanged
// between threads and every sum has one order. Operands are bf16, the queries'
// own type, in which a record's values are exact: products are exact and their
// sums fp32, so that the weights' errors are those of fp32. The exponent is
// scale s - lse with one rounding, before the factor log2(e). A row tile's sums
// go into the position's total by a compensated addition.
//
// Work: the items' row tiles (and an item's fixed part) form a line
// that is cut into equal runs, one a CTA (persistent, one per SM). The pieces of
// an item that is cut leave their sums in the workspace; of the warps that have
// the same 32 positions the last to arrive adds them in the order of the pieces.
//   warps 0-11      exponentials and sums: three groups take the products in turn, each
//                   from an S of its own (a warp's way through one is some 2000 clocks,
//                   of which it issues for 500: with two groups 904 us at 16K)
//   warps 12-15     dequantisation, a record a thread
//   warp 16         tensor memory, MMA issue
//   warp 17         schedule, copies of the records (cp.async.bulk)
//   warp 18         queries (TMA, or by hand where a tile has few rows) and lse
//   warp 19         gate: waits for all that a product needs, so that the MMA warp waits once
// Every wait is bounded; see kv4_chunk.cu.
// Bound: exponentials and products, 58% of their pipes each, and 62% of the issue
// slots (8192 tokens): 16384 tokens of 32 heads take 783-807 us, 1.36-1.40 PFLOP/s.
// Where an item has few row tiles (64 tokens look back over five prompts: two for
// 256 positions, 79 us), the copies and conversions of K and an item's ends.
#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "kv4_attn.cuh"
#include "kv4_chunk.cuh"
#include "spc_tc.cuh"

namespace spc {

// stages of each dequantising warp's ring of records, and positions a stage: three
// tiles, where with 1.5 (and six Q tiles) 64 tokens' look back took 95 us, not 83
constexpr int kMsRaw = 6, kMsRun = 16;
constexpr uint32_t kMsStage = kMsRun * kKv4Rec;
constexpr int kMsK = 2;                               // ring of dequantised K tiles
constexpr int kMsQ = 5;                               // ring of Q tiles
constexpr int kMsL = 6;                               // ring of the rows' lse
constexpr int kMsItems = 2;
constexpr int kMsGo = 4;                              // products that the gate may be ahead by
constexpr int kMsMasks = 8;                           // tiles whose masks are kept: the ring's items' and those of the one being summed up
static_assert(kMsMasks >= 2 * (kMsItems + 1), "masks of three items");
constexpr int kMsHand = 32;                           // rows up to which a Q tile is loaded without TMA
constexpr int kMsWarpDeq = 12, kMsWarpMma = 16, kMsWarpPlan = 17, kMsWarpQ = 18;
constexpr int kMsThreads = 640;
// registers a thread: 96 at launch (640 threads); the three warpgroups that sum
// 112, dequantisation 80, the rest 64: 3 * 112 + 80 + 64 = 5 * 96
constexpr int kMsRegSum = 112, kMsRegDeq = 80, kMsRegRest = 64;
constexpr int kMsFixed = 12;                          // units (of two products) of an item's fixed part; with 1 a 16K prompt took 823 us, not 804
constexpr int kMsS = 3;                               // ring of S, and groups that sum
constexpr int kMsTmemCols = 512;                      // S, and K tiles of 64 columns
constexpr uint32_t kMsColK = kMsS * 128;
static_assert(kMsColK + kMsK * 64 <= kMsTmemCols, "tensor memory");

constexpr uint32_t kMsOffQ = 0;
constexpr uint32_t kMsOffRaw = kMsOffQ + kMsQ * kKcTile;
constexpr uint32_t kMsOffItem = kMsOffRaw + 4 * kMsRaw * kMsStage;    // [kMsItems] MsItem
constexpr uint32_t kMsOffLse = kMsOffItem + kMsItems * 64;            // [kMsL][128] -lse
constexpr uint32_t kMsOffOdd = kMsOffLse + kMsL * 512;                // [kMsL] whether a row adds nothing, [4 words] which
constexpr uint32_t kMsOffMask = kMsOffOdd + kMsL * 32;                // [kMsMasks][4 words]
constexpr uint32_t kMsOffComb = kMsOffMask + kMsMasks * 16;          // [2 tiles][2 other groups][128] sums
constexpr uint32_t kMsOffBar = kMsOffComb + 2 * 2 * 512;
constexpr int kMsBars = 8 * kMsRaw + 2 * kMsK + 2 * kMsQ + 2 * kMsL + 2 * kMsItems + 2 * kMsS + kMsGo + 2 * 8 + 1;
constexpr size_t kMsSmem = 1024 + kMsOffBar + kMsBars * 8 + 16;
static_assert(kMsSmem <= 227 * 1024, "shared memory of one CTA");

// workspace: status; arrival counters (zeroed by the call's first kernel) of the items that are
// cut first in a CTA, [2 tiles][4 warps]; the sums of a CTA's first and last piece
constexpr size_t kMsOffCount = 256;
constexpr size_t kMsOffPart = kMsOffCount + (size_t)kKcCtas * 8 * 4;
constexpr size_t kMsWorkspace = kMsOffPart + (size_t)kKcCtas * 2 * 256 * 4;
static_assert(kMsOffPart % 256 == 0, "aligned partials");

constexpr int kMfRows = 32;                           // rows up to which a request is the other kernel's

struct MsArgs {
  Kv4ChunkCall c;
  int G, gshift, tpm;      // heads a group, its log2, tokens a row tile
  int* status;
  uint32_t* counters;
  float* part;
  float up, scale;         // of K's scales in tensor memory; of the products
  long long wait_limit;
  int starve;              // test builds: no copy is issued, so that every wait runs out
};

struct MsItem {
  int b, g, p0;            // request (-1: no more items), KV head, first position
  int row0, n, len;        // the request's first row, new tokens and positions
  int tiles;               // of positions: 1 or 2
  int r0, r1;              // the piece's row tiles
  int pieces, piece, first;  // of the item, and its first CTA
  int pad[4];
};
static_assert(sizeof(MsItem) == 64, "item ring");

__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 32 K values of 16 bytes of codes and two scales as bf16 into 16 columns of this
// thread's tensor memory lane. A code as fp16 has at most one bit of mantissa; its bits three
// places further down are bf16's of the value times 2^-112, which the scale, an
// e4m3 number times `up`, takes back: the product is exact. `up` is 2^112, or 2^92 where the
// scale is at most 1 and takes the 2^20 (MsArgs): sums of 128 products of any finite queries,
// up to 2^147, then stay within fp32's range, and what is lost below 2^-126 is nothing in the logit.
// With a larger scale a sum beyond fp32's range is a logit beyond it.
__device__ __forceinline__ void ms_quarter_row(const uint4& codes, uint32_t sc, float up, uint32_t t) {
  uint32_t k[16];
  const uint32_t s2 = e4m3x2_to_f16(sc & 0xffffu);
  const float f0 = f16_lo(s2) * up, f1 = f16_hi(s2) * up;
  const uint32_t s[2] = {pack_bf16(f0, f0), pack_bf16(f1, f1)};
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t h[4];
    e2m1x8_to_f16(w[e], h);
#pragma unroll
    for (int f = 0; f < 4; ++f) k[4 * e + f] = bmul2(((h[f] >> 3) & 0x0fff0fffu) | (h[f] & 0x80008000u), s[e >> 1]);
  }
  tmem_st16(t, k);
}

// ---------------------------------------------------------------- the line of work
// Item i of a request's head holds positions [256 i, 256 i + 256); its row tiles
// are those from the first that sees one of them on, max(0, 2 G i - cd) of nt,
// cd = ceil((len - n) / tpm). Requests with few rows have no items here.
struct MsShape {
  int n, len, nt, cd, items, G2;
};
__device__ __forceinline__ bool ms_few(const MsArgs& a, int n) { return ((long long)n << a.gshift) <= kMfRows; }
__device__ __forceinline__ MsShape ms_shape(const MsArgs& a, int len, int n) {
  const int lt = 7 - a.gshift;
  MsShape s;
  s.n = n;
  s.len = len;
  s.nt = (n + a.tpm - 1) >> lt;
  s.cd = -((n - len) >> lt);
  s.items = ms_few(a, n) ? 0 : (len + 255) >> 8;
  s.G2 = 2 * a.G;
  return s;
}
__device__ __forceinline__ int ms_first(const MsShape& s, int i) { return max(0, s.G2 * i - s.cd); }
__device__ __forceinline__ long long ms_units(const MsShape& s, int k) {   // of the items below k
  // the first item that some row tile does not see, and from there on an arithmetic progression
  const int k0 = s.cd < 0 ? 0 : min(k, s.cd / s.G2 + 1);
  const long long m = k - k0;
  return (long long)k * (kMsFixed + s.nt) - ((long long)s.G2 * (k - 1 + k0) * m / 2 - (long long)s.cd * m);
}

__global__ void __launch_bounds__(kMsThreads, 1) kv4_mass_kernel(const __grid_constant__ CUtensorMap qmap, const MsArgs a) {
  extern __shared__ uint8_t ms_raw[];
  const uint32_t raw_addr = smem_u32(ms_raw);
  uint8_t* base = ms_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  MsItem* items = reinterpret_cast<MsItem*>(base + kMsOffItem);
  float* neglse = reinterpret_cast<float*>(base + kMsOffLse);
  uint32_t* odds = reinterpret_cast<uint32_t*>(base + kMsOffOdd);
  uint32_t* masks = reinterpret_cast<uint32_t*>(base + kMsOffMask);
  float* comb = reinterpret_cast<float*>(base + kMsOffComb);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + kMsOffBar);
  uint64_t* rfull = bars;                     // [4 warps][kMsRaw] bytes of the records
  uint64_t* rfree = rfull + 4 * kMsRaw;       // [4][kMsRaw] the warp has read them
  uint64_t* kfull = rfree + 4 * kMsRaw;       // [kMsK] four dequantising warps have written the tile
  uint64_t* kfree = kfull + kMsK;             // [kMsK] commit after the last MMA that reads it
  uint64_t* qfull = kfree + kMsK;             // [kMsQ] the tile's rows are there
  uint64_t* qfree = qfull + kMsQ;             // [kMsQ] commit after the MMAs that read them
  uint64_t* lfull = qfree + kMsQ;             // [kMsL] the rows' lse are there
  uint64_t* lfree = lfull + kMsL;             // [kMsL] the summing warps have read them
  uint64_t* ifull = lfree + kMsL;             // [kMsItems]
  uint64_t* ifree = ifull + kMsItems;         // [kMsItems]
  uint64_t* sfull = ifree + kMsItems;         // [kMsS] commit: S in tensor memory
  uint64_t* sfree = sfull + kMsS;             // [kMsS] four summing warps have read it
  uint64_t* go = sfree + kMsS;                // [kMsGo] gate: S may be written, its operands are there
  uint64_t* cdone = go + kMsGo;               // [2 tiles][4 warps] the other groups' sums are there
  uint64_t* cread = cdone + 8;                // [2][4] and have been read
  uint64_t* drain = cread + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const Kv4ChunkCall& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 4 * kMsRaw; ++s) {
      mbar_init(&rfull[s], 1);
      mbar_init(&rfree[s], 1);
    }
    for (int s = 0; s < kMsK; ++s) {
      mbar_init(&kfull[s], 4);
      mbar_init(&kfree[s], 1);
    }
    for (int s = 0; s < kMsQ; ++s) {
      mbar_init(&qfull[s], 1);
      mbar_init(&qfree[s], 1);
    }
    for (int s = 0; s < kMsL; ++s) {
      mbar_init(&lfull[s], 1);
      mbar_init(&lfree[s], 8);
    }
    for (int s = 0; s < kMsItems; ++s) {
      mbar_init(&ifull[s], 1);
      mbar_init(&ifree[s], 4 + 12 + 3);
    }
    for (int s = 0; s < kMsS; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sfree[s], 4);
    }
    for (int s = 0; s < kMsGo; ++s) mbar_init(&go[s], 1);
    for (int s = 0; s < 8; ++s) {
      mbar_init(&cdone[s], 2);
      mbar_init(&cread[s], 1);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == kMsWarpMma) tmem_alloc<kMsTmemCols>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  kc_wait_first();
  const uint32_t qs = smem_u32(base + kMsOffQ);
  bool dead = false;
  auto acquire = [&](uint64_t* bar, uint32_t parity) {
    // mostly over: tested before it is waited for
    if (!dead && !__all_sync(0xffffffffu, mbar_test(bar, parity)) &&
        !__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.wait_limit))) {
      if (lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
      dead = true;
    }
  };

  if (warp == kMsWarpPlan) {
    // ================= schedule and copies of the records
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kMsRegRest));
    const int bs = 1 << c.block_shift;
    KcRequests rq;
    kc_requests(c, rq);
    long long own[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const MsShape s = ms_shape(a, rq.len[e], rq.n[e]);
      own[e] = ms_units(s, s.items);
    }
    const long long total = kc_prefix(rq, own[0] * c.n_kv, own[1] * c.n_kv);
    const int ctas = (int)(total < (long long)gridDim.x ? total : (long long)gridDim.x);
    const bool has = (int)blockIdx.x < ctas;
    const long long u0 = has ? kc_div(total * blockIdx.x, ctas) : 0, u1 = has ? kc_div(total * (blockIdx.x + 1), ctas) : 0;
    auto cta_of = [&](long long u) { return (int)kc_div((u + 1) * ctas - 1, total); };
    int b = 0, g = 0, i = 0;
    long long at = 0, whole = 1;
    MsShape s{};
    auto enter = [&](int request) {
      b = request;
      s = ms_shape(a, kc_of(rq.len, b), kc_of(rq.n, b));
      whole = __shfl_sync(0xffffffffu, b & 1 ? own[1] : own[0], b >> 1);
    };
    if (has) {
      enter(kc_find(rq, u0));
      long long r = u0 - (kc_of(rq.end, b) - whole * c.n_kv);
      g = (int)kc_div(r, whole);
      r -= (long long)g * whole;
      int lo = 0, hi = s.items;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ms_units(s, mid) <= r) lo = mid; else hi = mid;
      }
      i = lo;
      at = u0 - r + ms_units(s, i);
    }
    int it = 0, blocks = 0, nraw = 0;
    KcTable t;
    t.row = nullptr;
    for (;;) {
      MsItem x;
      x.b = -1;
      bool skip = false;
      const int nu = has && at < u1 ? s.nt - ms_first(s, i) : 0;
      if (has && at < u1 && !dead) {
        const long long first = at + kMsFixed;
        const int lo = (int)max(0ll, u0 - first), hi = (int)min((long long)nu, u1 - first);
        skip = hi <= lo;
        if (!skip) {
          x.b = b;
          x.g = g;
          x.p0 = i << 8;
          x.row0 = kc_of(rq.row0, b);
          x.n = s.n;
          x.len = s.len;
          x.tiles = x.p0 + 128 < s.len ? 2 : 1;
          x.r0 = s.nt - nu + lo;
          x.r1 = s.nt - nu + hi;
          x.first = lo > 0 ? cta_of(first) : (int)blockIdx.x;
          x.pieces = lo > 0 || hi < nu ? cta_of(first + nu - 1) - x.first + 1 : 1;
          x.piece = (int)blockIdx.x - x.first;
        }
      }
      if (!skip) {
        const int is = it % kMsItems;
        acquire(&ifree[is], ((it / kMsItems) & 1) ^ 1);
        if (lane == 0) {
          items[is] = x;
          mbar_arrive(&ifull[is]);
        }
        __syncwarp();
        ++it;
        if (x.b < 0) break;
#ifdef SPC_TEST_HOOKS
        if (a.starve) break;
#endif
        t.move(c.table + (size_t)b * c.max_blocks, (x.len + bs - 1) >> c.block_shift, x.p0 >> c.block_shift);
        // lane w + 4 h copies half h of dequantising warp w's positions
        const int w = lane & 3, h = lane >> 2 & 1;
        for (int j = 0; j < x.tiles && !dead; ++j, ++blocks, nraw += 2) {
          const int use = nraw + h, st = w * kMsRaw + use % kMsRaw, p = x.p0 + j * 128 + w * 32 + h * kMsRun;
          const int blk = t.entry((x.p0 + j * 128) >> c.block_shift, p >> c.block_shift);
          const int n = (unsigned)blk < (unsigned)c.num_blocks ? max(0, min(x.len - p, kMsRun)) : 0;
          uint32_t mask = ((1u << n) - 1u) << (h * kMsRun);
          mask |= __shfl_xor_sync(0xffffffffu, mask, 4);
          acquire(&rfree[st], ((use / kMsRaw) & 1) ^ 1);
          if (dead) break;
          if (lane < 4) masks[(blocks % kMsMasks) * 4 + lane] = mask;
          __syncwarp();                               // before the arrivals that let them be read
          if (lane < 8) {
            if (n > 0) {
              mbar_arrive_expect_tx(&rfull[st], (uint32_t)n * kKv4Rec);
              bulk_g2s(base + kMsOffRaw + st * kMsStage,
                       c.cache + (((size_t)blk * c.n_kv + x.g) * bs + (p & (bs - 1))) * kKv4Rec, (uint32_t)n * kKv4Rec, &rfull[st]);
            } else {
              mbar_arrive(&rfull[st]);
            }
          }
          __syncwarp();
        }
      }
      // the next item
      at += kMsFixed + nu;
      if (++i == s.items) {
        i = 0;
        if (++g == c.n_kv) {
          g = 0;
          if (at < u1) enter(kc_find(rq, at));
        }
      }
    }
    // every copy lands before the CTA ends (they have, unless a role gave up)
    if (lane < 4)
      for (int k = max(0, nraw - kMsRaw); k < nraw; ++k)
        mbar_wait_bounded(&rfull[lane * kMsRaw + k % kMsRaw], (k / kMsRaw) & 1, a.wait_limit);
    __syncwarp();
  } else if (warp == kMsWarpQ) {
    // ================= queries and lse of the row tiles
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kMsRegRest));
    int nq = 0;
    for (int it = 0;; ++it) {
      const int is = it % kMsItems;
      acquire(&ifull[is], (it / kMsItems) & 1);
      if (dead) break;
      const MsItem x = items[is];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
      if (x.b < 0) break;
#ifdef SPC_TEST_HOOKS
      if (a.starve) break;
#endif
      // row r of a tile whose first token is tok
      auto lse_of = [&](int tok, int r) {
        const int t = tok + (r >> a.gshift);
        return t < x.n ? c.lse[(size_t)(x.row0 + t) * c.n_q + (x.g << a.gshift) + (r & (a.G - 1))] : 0.f;
      };
      float next[4], after[4];                        // of this row tile and the one behind it
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        next[e] = lse_of(x.r0 * a.tpm, 32 * e + lane);
        after[e] = x.r0 + 1 < x.r1 ? lse_of((x.r0 + 1) * a.tpm, 32 * e + lane) : 0.f;
      }
      for (int r = x.r0; r < x.r1; ++r, ++nq) {
        const int st = nq % kMsQ, tok = r * a.tpm, rows = min(128, (x.n - tok) << a.gshift);
        acquire(&qfree[st], ((nq / kMsQ) & 1) ^ 1);
        if (dead) break;
        if (rows > kMsHand) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&qfull[st], kKcTile);
            tma_load_3d(qs + st * kKcTile, &qmap, 0, x.g << a.gshift, x.row0 + tok, &qfull[st]);
            tma_load_3d(qs + st * kKcTile + kKcBlock, &qmap, 64, x.g << a.gshift, x.row0 + tok, &qfull[st]);
          }
          __syncwarp();
        } else {
          // 16 pieces of 16 bytes a row; rows that are not there are zeros up to the MMA's multiple of 16
          const int all = ((rows + 15) & ~15) * 16;
#pragma unroll 1
          for (int e0 = lane; e0 < all; e0 += 4 * 32) {
            uint4 v[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              const int e = e0 + 32 * f, row = e >> 4;
              v[f] = make_uint4(0u, 0u, 0u, 0u);
              if (e < all && row < rows)
                v[f] = *reinterpret_cast<const uint4*>(c.q + (x.row0 + tok + (row >> a.gshift)) * c.q_stride +
                                                       (size_t)((x.g << a.gshift) + (row & (a.G - 1))) * kD + (e & 15) * 8);
            }
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              const int e = e0 + 32 * f, row = e >> 4, u = e & 15;
              if (e < all)
                sts_v4(qs + st * kKcTile + (u >> 3) * kKcBlock + row * 128 + (((u & 7) ^ (row & 7)) << 4), v[f].x, v[f].y, v[f].z,
                       v[f].w);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&qfull[st]);
        }
        const int ls = nq % kMsL;
        acquire(&lfree[ls], ((nq / kMsL) & 1) ^ 1);
        if (dead) break;
        uint32_t any = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          neglse[ls * 128 + 32 * e + lane] = -next[e];
          const uint32_t odd = __ballot_sync(0xffffffffu, next[e] == -INFINITY);
          if (lane == 0) odds[ls * 8 + 1 + e] = odd;
          any |= odd;
        }
        if (lane == 0) odds[ls * 8] = any;
        __syncwarp();
        if (lane == 0) mbar_arrive(&lfull[ls]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          next[e] = after[e];
          if (r + 2 < x.r1) after[e] = lse_of(tok + 2 * a.tpm, 32 * e + lane);
        }
      }
      if (dead) break;
    }
    if (lane == 0)
      for (int k = max(0, nq - kMsQ); k < nq; ++k) mbar_wait_bounded(&qfull[k % kMsQ], (k / kMsQ) & 1, a.wait_limit);
    __syncwarp();
  } else if (warp == kMsWarpMma) {
    // ================= MMA issue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kMsRegRest));
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    int nk = 0, nq = 0, ns = 0;
    for (int it = 0;; ++it) {
      const int is = it % kMsItems;
      acquire(&ifull[is], (it / kMsItems) & 1);
      if (dead) break;
      const int b = items[is].b, n = items[is].n, r0 = items[is].r0, r1 = items[is].r1, tiles = items[is].tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
      if (b < 0) break;
      for (int r = r0; r < r1 && !dead; ++r, ++nq) {
        const int st = nq % kMsQ, N = min(128, (((n - r * a.tpm) << a.gshift) + 15) & ~15);
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
#pragma unroll 1
        for (int j = 0; j < tiles; ++j) {
          const int buf = ns % kMsS;
          acquire(&go[ns % kMsGo], (ns / kMsGo) & 1);
          ++ns;
          if (dead) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t kt = tm + kMsColK + (uint32_t)((nk + j) % kMsK) * 64;
            const uint32_t qd = umma_desc_lo(qs) + (uint32_t)st * (kKcTile >> 4);
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk) {
              const uint32_t off = (uint32_t)(kk >> 2) * (kKcBlock >> 4) + (uint32_t)(kk & 3) * 2;
              umma_f16_tmem_a(tm + (uint32_t)buf * 128, kt + kk * 8, umma_desc(qd + off), idesc, kk ? 1u : 0u);
            }
            umma_commit(&sfull[buf]);
            if (j + 1 == tiles) umma_commit(&qfree[st]);
            if (r + 1 == r1) umma_commit(&kfree[(nk + j) % kMsK]);
          }
          __syncwarp();
        }
      }
      nk += tiles;
      if (dead) break;
    }
    if (elect_one()) umma_commit(drain);
    __syncwarp();
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(drain, 0, a.wait_limit)) && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
  } else if (warp >= kMsWarpDeq && warp < kMsWarpDeq + 4) {
    // ================= dequantisation, a record a thread
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kMsRegDeq));
    const int w = warp - kMsWarpDeq;
    int nk = 0, nread = 0;
    for (int it = 0;; ++it) {
      const int is = it % kMsItems;
      acquire(&ifull[is], (it / kMsItems) & 1);
      if (dead) break;
      const int b = items[is].b, tiles = items[is].tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
      if (b < 0) break;
      for (int j = 0; j < tiles; ++j, ++nk) {
        const int s0 = nread % kMsRaw, s1 = (nread + 1) % kMsRaw;
        acquire(&rfull[w * kMsRaw + s0], (nread / kMsRaw) & 1);
        acquire(&rfull[w * kMsRaw + s1], ((nread + 1) / kMsRaw) & 1);
        if (dead) break;
        nread += 2;
        const uint32_t rec = smem_u32(base + kMsOffRaw) + (uint32_t)(w * kMsRaw + (lane < kMsRun ? s0 : s1)) * kMsStage +
                             (uint32_t)(lane & (kMsRun - 1)) * kKv4Rec;
        const bool there = masks[(nk % kMsMasks) * 4 + w] >> lane & 1;
        const int slot = nk % kMsK;
        acquire(&kfree[slot], ((nk / kMsK) & 1) ^ 1);
        if (dead) break;
        tc_fence_after();
        const uint32_t t = tmem + ((uint32_t)(w * 32) << 16) + kMsColK + (uint32_t)slot * 64;
        // in a loop: one warp an SM's quarter runs this code, and unrolled it waits for its own instructions
        // (64 tokens' look back 79 us, unrolled 83)
        const uint2 sc = lds_v2(rec + kKv4Scale);
        uint4 v = lds_v4(rec);
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          const uint4 next = q < 3 ? lds_v4(rec + 16 * (q + 1)) : v;
          if (!there) v = make_uint4(0u, 0u, 0u, 0u);
          ms_quarter_row(v, there ? (q < 2 ? sc.x : sc.y) >> (16 * (q & 1)) : 0u, a.up, t + 16 * q);
          v = next;
        }
        __syncwarp();
        if (lane < 2) mbar_arrive(&rfree[w * kMsRaw + (lane ? s1 : s0)]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kfull[slot]);
      }
      if (dead) break;
    }
  } else if (warp < kMsWarpDeq) {
    // ================= exponentials and sums, one position a thread: group g takes the
    // products whose number is g modulo 3, and ends up with tile g's sums
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kMsRegSum));
    const int grp = warp >> 2, wq = warp & 3, lt = 7 - a.gshift;
    const uint32_t ts = tmem + ((uint32_t)(wq * 32) << 16) + (uint32_t)grp * 128;
    const float2 sc = make_float2(a.scale, a.scale), l2e = make_float2(kLog2e, kLog2e);
    int ns = 0, nq = 0, nk = 0, nc[2] = {0, 0};
    for (int it = 0;; ++it) {
      const int is = it % kMsItems;
      acquire(&ifull[is], (it / kMsItems) & 1);
      if (dead) break;
      const MsItem x = items[is];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
      if (x.b < 0) break;
      const int two = x.tiles - 1, count = (x.r1 - x.r0) << two, ctx = x.len - x.n;
      const int at0 = x.p0 + wq * 32;                 // the warp's first position in tile A
      const size_t at = ((size_t)x.b * c.n_kv + x.g) * c.cap + at0 + grp * 128 + lane;
      const bool mine = grp < x.tiles && at0 + grp * 128 + lane < x.len;
      const float prev = mine && c.keep != 0.f ? c.mass_prev[at] : 0.f;
      float total[2] = {0.f, 0.f}, lost[2] = {0.f, 0.f};
      // Row tile r's columns are all tokens at or behind the warp's last position
      // of tile j where r >= all[j]; the last row tile may be short.
      int all[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        all[j] = (int)max(0ll, ((long long)at0 + j * 128 + 31 - ctx + a.tpm - 1) >> lt);
      const int whole = x.n >> lt;
      for (int k = (grp + kMsS - ns % kMsS) % kMsS; k < count; k += kMsS) {
        const int r = x.r0 + (k >> two), j = k & two, ls = (nq + (k >> two)) % kMsL;
        acquire(&sfull[grp], ((ns + k) / kMsS) & 1);
        if (dead) break;
        tc_fence_after();
        const float* nl = neglse + ls * 128;
        float y;
        if (r >= (j ? all[1] : all[0]) && r < whole && odds[ls * 8] == 0u) {
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          float s[2][32];
          tmem_ld32(ts, s[0]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tmem_ld_wait32(s[q & 1]);
            if (q < 3) {
              tmem_ld32(ts + 32 * (q + 1), s[(q + 1) & 1]);
            } else {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sfree[grp]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 l4 = *reinterpret_cast<const float4*>(nl + 32 * q + 4 * e);
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                float2 t = fma2(make_float2(s[q & 1][4 * e + 2 * f], s[q & 1][4 * e + 2 * f + 1]), sc,
                                f ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y));
                t = fma2(t, l2e, make_float2(0.f, 0.f));
                t.x = ex2_approx(t.x);
                t.y = ex2_approx(t.y);
                sum[f] = add2(sum[f], t);
              }
            }
          }
          y = (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
        } else {
          const int tok = r * a.tpm, cols = min(128, (x.n - tok) << a.gshift);
          // columns from this one on are tokens at or behind the position
          const long long from = ((long long)at0 + j * 128 + lane - ctx - tok) << a.gshift;
          const uint32_t* odd = odds + ls * 8 + 1;
          float sum[2] = {0.f, 0.f};
#pragma unroll 1
          for (int q = 0; 32 * q < cols; ++q) {
            float s[32];
            tmem_ld32(ts + 32 * q, s);
            tmem_ld_wait32(s);
            const long long lo = from - 32 * q;
            const int hi = cols - 32 * q;
            const uint32_t vis = (lo <= 0 ? 0xffffffffu : lo >= 32 ? 0u : 0xffffffffu << (int)lo) &
                                 (hi >= 32 ? 0xffffffffu : (1u << hi) - 1u) & ~odd[q];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float t = ex2_approx(fmaf(s[e], a.scale, nl[32 * q + e]) * kLog2e);
              sum[e & 1] += vis >> e & 1 ? t : 0.f;
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfree[grp]);
          y = sum[0] + sum[1];
        }
        __syncwarp();
        if (lane <= 1 - two) mbar_arrive(&lfree[ls]);   // eight arrivals a row tile, also where one tile reads it
        // the tile's sum into the total, what the addition loses kept beside it
        const float t0 = j ? total[1] : total[0], u = t0 + y, v = u - t0, w = (t0 - (u - v)) + (y - v);
        if (j) {
          total[1] = u;
          lost[1] += w;
        } else {
          total[0] = u;
          lost[0] += w;
        }
      }
      if (dead) break;
      ns += count;
      nq += x.r1 - x.r0;
      // a tile's sums from the other two groups to the one that has its number
      float sum[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // infinities and NaN are the sum's own; their difference above is not
        sum[j] = total[j] + (fabsf(total[j]) < INFINITY ? lost[j] : 0.f);
        if (j >= x.tiles || j == grp) continue;
        acquire(&cread[j * 4 + wq], (nc[j]++ & 1) ^ 1);
        if (dead) break;
        comb[(j * 2 + (grp == 2 ? 1 : 0)) * 128 + wq * 32 + lane] = sum[j];
        __syncwarp();
        if (lane == 0) mbar_arrive(&cdone[j * 4 + wq]);
      }
      if (dead) break;
      nk += x.tiles;
      if (grp >= x.tiles) continue;
      acquire(&cdone[grp * 4 + wq], nc[grp & 1]++ & 1);
      if (dead) break;
      float y = grp ? sum[1] : sum[0];
#pragma unroll
      for (int e = 0; e < 2; ++e) y += comb[(grp * 2 + e) * 128 + wq * 32 + lane];
      __syncwarp();
      if (lane == 0) mbar_arrive(&cread[grp * 4 + wq]);
      if (!(masks[((nk - x.tiles + grp) % kMsMasks) * 4 + wq] >> lane & 1)) y = 0.f;
      if (x.pieces > 1) {
        float* part = a.part + ((size_t)blockIdx.x * 2 + (x.piece == 0 ? 1 : 0)) * 256 + grp * 128 + wq * 32 + lane;
        *part = y;
        __threadfence();
        __syncwarp();
        uint32_t* arrived = a.counters + x.first * 8 + grp * 4 + wq;
        uint32_t before = 0u;
        if (lane == 0) before = atomicAdd(arrived, 1u);
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before + 1u != (uint32_t)x.pieces) continue;
        __threadfence();
        y = 0.f;
        for (int k = 0; k < x.pieces; ++k)
          y += __ldcg(a.part + ((size_t)(x.first + k) * 2 + (k == 0 ? 1 : 0)) * 256 + grp * 128 + wq * 32 + lane);
      }
      if (mine) c.mass_next[at] = c.keep != 0.f ? fmaf(c.keep, prev, y) : y;
    }
  } else {                                    // warp 19
    // ================= gate
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kMsRegRest));
    int nk = 0, nq = 0, ns = 0;
    for (int it = 0; !dead; ++it) {
      const int is = it % kMsItems;
      acquire(&ifull[is], (it / kMsItems) & 1);
      if (dead) break;
      const int b = items[is].b, steps = items[is].r1 - items[is].r0, tiles = items[is].tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
      if (b < 0) break;
      for (int j = 0; j < tiles; ++j) acquire(&kfull[(nk + j) % kMsK], ((nk + j) / kMsK) & 1);
      for (int r = 0; r < steps && !dead; ++r, ++nq) {
        acquire(&lfull[nq % kMsL], (nq / kMsL) & 1);
        acquire(&qfull[nq % kMsQ], (nq / kMsQ) & 1);
        for (int j = 0; j < tiles; ++j, ++ns) {
          acquire(&sfree[ns % kMsS], ((ns / kMsS) & 1) ^ 1);
          if (dead) break;
          if (lane == 0) mbar_arrive(&go[ns % kMsGo]);
        }
      }
      nk += tiles;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMsWarpMma) {
    tc_fence_after();
    tmem_dealloc<kMsTmemCols>(tmem);
  }
}

// ---------------------------------------------------------------- few rows
// Requests with at most 32 rows (a decode step's token, a few drafted ones, none):
// the records' bytes are what counts, so every warp streams positions for
// itself. 15 warps each have a ring of stages of 32 records that a sixteenth
// fills (k4_copy); the products run on mma.sync with 16 positions as M and 8 rows
// as N. Lane (gid, tig) dequantises dims 32 tig .. 32 tig + 31 of positions gid
// and gid + 8 to fp16, 16 bytes of codes each; the contraction's order is free,
// so these are the fragments of the eight steps as they come, and the queries, in
// registers, are in the same order: bf16 to fp16 times a power of two a row, as in
// kv4_chunk.cu (11 bits down to 2^-28 of the row's largest, so that a bf16 value is
// exact there). Nothing is exchanged but a position's sum over four lanes.
// Bound: HBM. 8 x 65536 positions, 64 heads on 8: 604 MB of records (K's 72 bytes of
// 144 are in every line that is read) and 34 MB of sums in 126 us, 5.1 TB/s; 32768:
// 69 us alone, 4.7 TB/s, the ALU pipe 41% busy with conversions.
constexpr int kMfWarps = 15, kMfStages = 3, kMfTiles = kMfRows / 8;
constexpr uint32_t kMfOffBar = kMfWarps * kMfStages * kK4StageBytes;
constexpr uint32_t kMfOffMask = kMfOffBar + 2 * kMfWarps * kMfStages * 8;
constexpr uint32_t kMfSmem = kMfOffMask + kMfWarps * kMfStages * 4;

struct MfArgs {
  Kv4Args k4;              // the cache, for k4_copy
  MsArgs ms;
};

__global__ void __launch_bounds__(32 * (kMfWarps + 1), 1) kv4_mass_few_kernel(const MfArgs fa) {
  extern __shared__ __align__(128) uint8_t mf_smem[];
  __shared__ K4Line ln;
  const MsArgs& a = fa.ms;
  const Kv4ChunkCall& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  uint64_t* all_full = reinterpret_cast<uint64_t*>(mf_smem + kMfOffBar);
  uint64_t* all_free = all_full + kMfWarps * kMfStages;
  uint32_t* all_masks = reinterpret_cast<uint32_t*>(mf_smem + kMfOffMask);
  if (warp == 1) {
    for (int s = lane; s < kMfWarps * kMfStages; s += 32) {
      mbar_init(&all_full[s], 1);
      mbar_init(&all_free[s], 1);
    }
    fence_mbar_init();
  }
  if (warp == 0) {
    // tiles of 32 positions of the requests with few rows, cut into equal runs
    KcRequests rq;
    kc_requests(c, rq);
    int nt[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      nt[e] = ms_few(a, rq.n[e]) ? (rq.len[e] + kK4Tile - 1) / kK4Tile : 0;
      ln.len[2 * lane + e] = rq.len[e];
      ln.nt[2 * lane + e] = nt[e];
      nt[e] *= c.n_kv;
    }
    const int incl = warp_incl_scan(nt[0] + nt[1]);
    ln.pre[2 * lane] = incl - nt[0] - nt[1];
    ln.pre[2 * lane + 1] = incl - nt[1];
    if (lane == 31) {
      ln.pre[SPC_MAX_BATCH] = incl;
      ln.t0 = (int)((long long)incl * blockIdx.x / gridDim.x);
      ln.t1 = (int)((long long)incl * (blockIdx.x + 1) / gridDim.x);
    }
  }
  __syncthreads();
  const int t0 = ln.t0, t1 = ln.t1;
  // the other kernel's counters, whatever a call that ran out of time has left there
  if (threadIdx.x < 8) a.counters[blockIdx.x * 8 + threadIdx.x] = 0u;
  kc_let_next();
  if (t0 >= t1) return;
  if (warp == kMfWarps) {
#ifdef SPC_TEST_HOOKS
    if (a.starve) return;
#endif
    k4_copy<kMfWarps, kMfStages>(fa.k4, ln, c.n_kv, t0, t1, mf_smem, all_full, all_free, all_masks);
    return;
  }
  const uint32_t ring = smem_u32(mf_smem) + (uint32_t)warp * kMfStages * kK4StageBytes;
  uint64_t* full = all_full + warp * kMfStages;
  uint64_t* empty = all_free + warp * kMfStages;
  const uint32_t* masks = all_masks + warp * kMfStages;
  K4Cursor x = k4_at(fa.k4.c, ln, min(t0 + warp, t1 - 1));
  int seg = -1, tiles = 0, ctx = 0;
  uint32_t q[kMfTiles][16];                           // rows 8 i + gid, the lane's 32 dims
  float f[kMfTiles][2], nl[kMfTiles][2];              // of columns 8 i + 2 tig, + 1: a logit's factor (0: adds nothing), -lse
  for (int t = t0 + warp, k = 0; t < t1; t += kMfWarps, ++k) {
    const int b = x.b, g = x.s, p0 = x.i * kK4Tile;
    if (seg != b * c.n_kv + g) {
      seg = b * c.n_kv + g;
      const int row0 = max(0, min(c.cu[b], c.T)), n = max(row0, min(c.cu[b + 1], c.T)) - row0, rows = n << a.gshift;
      ctx = x.len - n;
      tiles = (rows + 7) >> 3;
#pragma unroll
      for (int i = 0; i < kMfTiles; ++i) {
        const int r = 8 * i + gid;                    // rows that are not there are as those that add nothing
        const size_t tok = row0 + (r >> a.gshift);
        const int h = (g << a.gshift) + (r & (a.G - 1));
        const float lse = r < rows ? c.lse[tok * c.n_q + h] : -INFINITY;
        uint4 w[4];
        uint32_t mx = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // a row that adds nothing is zeros, whatever it holds, and left out of the sums: a
          // K scale that is NaN makes its products NaN
          w[e] = lse != -INFINITY ? *reinterpret_cast<const uint4*>(c.q + tok * c.q_stride + (size_t)h * kD + 32 * tig + 8 * e)
                                  : make_uint4(0u, 0u, 0u, 0u);
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(w[e].x & 0x7fff7fffu, w[e].y & 0x7fff7fffu),
                                     __vmaxu2(w[e].z & 0x7fff7fffu, w[e].w & 0x7fff7fffu)));
        }
        mx = max(mx & 0xffffu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int E = (int)(mx >> 7), e2 = min(141 - E, 126);
        const float up = __int_as_float((e2 + 127) << 23);
        // the scale over the power of two (q.K itself may be beyond fp32's range), kept from zero and from infinity: a
        // row that adds nothing is told by it, and a product of zero stays one
        const float factor = fminf(fmaxf(__int_as_float((127 - e2) << 23) * c.scale, 1.17549435e-38f), 3.40282347e38f);
        auto f16 = [&](uint32_t v) { return pack_f16(bf_lo(v) * up, bf_hi(v) * up); };   // infinities and NaN stay what they are
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q[i][4 * e] = f16(w[e].x);
          q[i][4 * e + 1] = f16(w[e].y);
          q[i][4 * e + 2] = f16(w[e].z);
          q[i][4 * e + 3] = f16(w[e].w);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[i][e] = __shfl_sync(0xffffffffu, lse == -INFINITY ? 0.f : factor, (2 * tig + e) * 4);
          nl[i][e] = -__shfl_sync(0xffffffffu, lse, (2 * tig + e) * 4);
        }
      }
    }
    // lane tig 0 writes position gid of each half, tig 1 position gid + 8
    const size_t at = (size_t)seg * c.cap + p0 + gid + 8 * tig;
    float prev[2] = {0.f, 0.f};
    if (c.keep != 0.f && tig < 2) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (p0 + 16 * m + gid + 8 * tig < x.len) prev[m] = c.mass_prev[at + 16 * m];
    }
    const int st = k % kMfStages;
    if (!__all_sync(0xffffffffu, mbar_test(&full[st], (k / kMfStages) & 1) ||
                                     mbar_wait_bounded(&full[st], (k / kMfStages) & 1, a.wait_limit))) {
      if (lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
      return;
    }
    const uint32_t mask = masks[st];
    const bool seen = p0 + kK4Tile - 1 <= ctx;        // by every row
    // 16 positions against NT row tiles
    auto weigh = [&](auto count, int m) {
      constexpr int NT = decltype(count)::value;
      const uint32_t rec = ring + (uint32_t)st * kK4StageBytes + (uint32_t)(16 * m + gid) * kKv4Rec;
      const uint4 c0 = lds_v4(rec + 16 * tig), c1 = lds_v4(rec + 8 * kKv4Rec + 16 * tig);
      const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
      uint32_t b0, b1;
      asm volatile("ld.shared.u16 %0, [%1];" : "=r"(b0) : "r"(rec + kKv4Scale + 2 * tig));
      asm volatile("ld.shared.u16 %0, [%1];" : "=r"(b1) : "r"(rec + 8 * kKv4Rec + kKv4Scale + 2 * tig));
      const uint32_t h0 = e4m3x2_to_f16(b0), h1 = e4m3x2_to_f16(b1);
      float d[NT][4] = {};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t s0 = __byte_perm(h0, h0, e < 2 ? 0x1010 : 0x3232), s1 = __byte_perm(h1, h1, e < 2 ? 0x1010 : 0x3232);
        uint32_t k0[4], k1[4];
        e2m1x8_to_f16(w0[e], k0);
        e2m1x8_to_f16(w1[e], k1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t av[4] = {hmul2(k0[2 * h], s0), hmul2(k1[2 * h], s1), hmul2(k0[2 * h + 1], s0), hmul2(k1[2 * h + 1], s1)};
#pragma unroll
          for (int i = 0; i < NT; ++i) mma_f16(d[i], av, q[i][4 * e + 2 * h], q[i][4 * e + 2 * h + 1]);
        }
      }
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = ex2_approx(fmaf(d[i][e], f[i][e & 1], nl[i][e & 1]) * kLog2e);
          // column 8 i + 2 tig + (e & 1) adds something and is a token at or behind the position
          const bool vis = f[i][e & 1] != 0.f &&
                           (seen || ctx + ((8 * i + 2 * tig + (e & 1)) >> a.gshift) >= p0 + 16 * m + gid + 8 * (e >> 1));
          sum[e >> 1] += vis ? y : 0.f;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
      }
      const int j = 16 * m + gid + 8 * tig;
      if (tig < 2 && p0 + j < x.len) {
        const float y = mask >> j & 1 ? tig ? sum[1] : sum[0] : 0.f;
        c.mass_next[at + 16 * m] = c.keep != 0.f ? fmaf(c.keep, m ? prev[1] : prev[0], y) : y;
      }
    };
#pragma unroll 1
    for (int m = 0; m < 2; ++m) {
      if (tiles == 1) weigh(std::integral_constant<int, 1>{}, m);
      else if (tiles == 2) weigh(std::integral_constant<int, 2>{}, m);
      else weigh(std::integral_constant<int, kMfTiles>{}, m);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
    if (t + kMfWarps < t1) k4_step(fa.k4.c, ln, c.n_kv, x, kMfWarps);
  }
}

size_t kv4_mass_workspace(int, int, int, int) { return kMsWorkspace; }

int kv4_mass_launch(const Kv4ChunkCall& c, void* workspace, void* stream) {
  MsArgs a{};
  a.c = c;
  a.G = c.n_q / c.n_kv;
  while ((1 << a.gshift) < a.G) ++a.gshift;
  a.tpm = 128 >> a.gshift;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.status = reinterpret_cast<int*>(w);
  a.counters = reinterpret_cast<uint32_t*>(w + kMsOffCount);
  a.part = reinterpret_cast<float*>(w + kMsOffPart);
  a.up = c.scale <= 1.f ? 4.951760157141521e27f : 5.192296858534828e33f;   // 2^92, 2^112
  a.scale = c.scale <= 1.f ? c.scale * 1048576.f : c.scale;
  a.wait_limit = kKcWait;
#ifdef SPC_TEST_HOOKS
  a.starve = paged_starve(&a.wait_limit) ? 1 : 0;
#endif
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  MfArgs f{};
  f.ms = a;
  f.k4.c.cache = c.cache; f.k4.c.table = c.table; f.k4.c.len = c.len;
  f.k4.c.B = c.B; f.k4.c.n_q = c.n_q; f.k4.c.n_kv = c.n_kv; f.k4.c.num_blocks = c.num_blocks;
  f.k4.c.block_shift = c.block_shift; f.k4.c.max_blocks = c.max_blocks;
  f.k4.status = a.status;
  f.k4.wait_limit = a.wait_limit;
  if (set_func_attr((const void*)kv4_mass_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMfSmem) != cudaSuccess)
    return SPC_ERR_CUDA;
  kv4_mass_few_kernel<<<kKcCtas, 32 * (kMfWarps + 1), kMfSmem, st>>>(f);
  if (cudaGetLastError() != cudaSuccess) return SPC_ERR_CUDA;
  // The request's rows decide, up to 32 of them here and more there. us, the one way and the
  // other, G = 4: 8 x 65536 positions, 4 rows 121 and 492, 8 rows 126 and 492, 16 rows
  // 138 and 493, 32 rows 173 and 513; 1 x 1000, 4 rows 4.4 and 10.6, 32 rows 6.1 and
  // 11.0. 64 rows are eight tiles of 8, with 128 registers of queries a lane: not here.
  // No request can have more rows than the call.
  if ((long long)c.T * a.G > kMfRows) {
    CUtensorMap qmap{};
    const uint64_t dims[3] = {(uint64_t)kD, (uint64_t)c.n_q, (uint64_t)c.T};
    const uint64_t strides[2] = {(uint64_t)kRowBytes, (uint64_t)c.q_stride * 2};
    const uint32_t box[3] = {64, (uint32_t)a.G, (uint32_t)a.tpm};
    if (!tensor_map_bf16_sw128(&qmap, c.q, 3, dims, strides, box)) return SPC_ERR_CUDA;
    if (set_func_attr((const void*)kv4_mass_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMsSmem) != cudaSuccess)
      return SPC_ERR_CUDA;
    if (!kc_launch_next(kv4_mass_kernel, dim3(kKcCtas), kMsThreads, kMsSmem, st, qmap, a)) return SPC_ERR_CUDA;
  }
  return SPC_OK;
}

}  // namespace spc
