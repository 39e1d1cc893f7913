// Attention of chunks of new tokens over the paged 4-bit cache, on the
// 5th-generation tensor cores: out_i = sum_{p <= P_i} softmax_p(scale q_i.K_p) V_p,
// P_i = len - n + i, and lse_i.
//
// Rows are (token, query head of the group) pairs: a 128-row tile holds 128/G
// tokens x G heads of one KV head, so that a record that is dequantised serves
// the whole group. An item is two such tiles (A and B, consecutive tokens) of one
// (request, KV head) against that head's positions in blocks of 128:
//   S[128][128] = Q K^T     Q, K in shared memory (128-byte swizzle)
//   O[128][128] += P V      P in tensor memory over S's columns, V MN-major
// The tensor cores work on one tile while the other one's softmax runs. A
// request's last tile, if it has no partner (and with few new tokens every one of
// them), takes both places: A runs over the even blocks and B over the odd
// ones, and A's warps merge what B's have found (a warp of B has the same tensor
// memory lanes, so that only maxima and sums go through shared memory).
//
// Operands are fp16. A record's values are exact there; 11 bits of P instead of
// bf16's 8; and e2m1 to fp16 is one conversion for two values. Queries are scaled
// by a power of two a row (the largest to [2^14, 2^15): a value loses bits only
// below 2^-28 of it), in place, by the softmax thread of the row. P and its sum
// are kept 2^8 times the weights against the running maximum, so that weights keep
// 11 bits down to 2^-22 of the largest and are off by 2^-33 of it below; the
// maximum (of the products q.K, before the scale, so that a large logit's own
// rounding cannot pass the range) is raised when a logit passes it by more than
// 7.75 in base 2, and only then is the row of O rescaled. That costs some 2500
// cycles, for which the other tile's products wait: an earlier state with 2^11 and 4.75, where a raise
// of some row came in a third of the blocks (logits of a deviation of 2), took 3.67 ms
// for 64K x 2048 tokens of 64 heads.
// Sums, maxima, S and O are fp32; a weight's sum is that of the unrounded values.
//
// What a row does not see does not reach it. Masked columns of S are replaced. V
// meets their weight of zero, which a value that is not finite would defeat:
// records that are not there are zeros, and a V scale that is NaN (the only such
// value a record can hold) is taken as zero in the product while the first
// position that has it is noted for its 16 dims; rows at or behind that position
// get NaN there.
//
// Work: the items' blocks (and an item's fixed part), in units of their time, form
// a line that is cut into equal runs, one a CTA (persistent, one per SM). The pieces of
// an item that is cut leave partials (O, maximum, sum) in the workspace, which a
// second kernel merges in the order of the positions.
//   warps 0-3, 4-7  softmax and epilogue of tile A, B
//   warps 8-11      dequantisation (few new tokens: 8-15, and four more below) into a ring of four 32 KB operands: K_j, V_j, K_j+1, ...
//   warp 12         tensor memory, MMA issue
//   warp 13         schedule, copies of the records (cp.async.bulk)
//   warp 14         Q loads (TMA)
//   warp 15         gate: passes the operands' arrival on to the P barriers, so that the MMA
//                   warp waits once a batch
// Bound: 2048 tokens of 64 heads behind 64K take 2.93 ms, 1.48 PFLOP/s, a block of two
// tiles 1.7 us. Its products are 1 024 cycles of the tensor pipe, but S reads both
// operands from shared memory, which takes its half twice as long, and with the operands'
// own 64 KB shared memory is some 70% busy (counted, 2340 of 3250 cycles); the rest is the chain S, softmax, P of a
// tile where the other one does not cover it. With few rows (LONE) a block costs
// what 128 rows cost: 8 x 64K, 32 rows, 265 us, 2.3 TB/s of records.
// Every wait is bounded: a role whose wait gives up records SPC_ERR_TIMEOUT
// and leaves, the others' waits then give up in turn; copies land and MMAs
// complete before the CTA releases its tensor memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <type_traits>

#include "kv4_attn.cuh"
#include "kv4_chunk.cuh"
#include "spc_tc.cuh"

namespace spc {

// Records of the kernel for many new tokens: a ring for each dequantising warp (one
// reader, so that a wait on a phase's parity is never two phases behind), stages of
// 16 positions, which lie in one cache block
constexpr int kKcRaw = 3, kKcRun = 16;
constexpr uint32_t kKcRunBytes = kKcRun * kKv4Rec;
constexpr int kKcSlots = 4;                           // ring of dequantised operands
constexpr int kKcItems = 2;                           // item ring
constexpr int kKcMasks = 16;                          // blocks whose masks are kept: the copies are at most 8 ahead of the softmax
constexpr int kKcWarpDeq = 8;
constexpr float kKcBias = 8.f;                        // log2 of the factor of the weights
constexpr float kKcHeadroom = 7.75f;                  // log2 growth allowed before a maximum is raised
// The line of work: units of a block for two tiles, for one in both places, of an
// item's fixed part, and those a CTA takes at least (more than a block's, so that
// every CTA between an item's first and last one has a piece of it). 16 requests
// with up to 700 tokens take 755 us; with 4 or 6 for a block of one tile 814 or 767;
// with 6 for the fixed part 1.17 times as long. A run of 18 at least: 17 tokens behind
// 1000 took 29 us where a run of 11 took 23.
constexpr int kKcUnitsTwo = 6, kKcUnitsOne = 5, kKcFixed = 42, kKcMinRun = 9;
static_assert(kKcMinRun >= kKcUnitsTwo, "a block begins in every run");
constexpr int kKcTmemCols = 512;                      // S_A, S_B, O_A, O_B
constexpr uint32_t kKcColO = 256;
constexpr uint32_t kKcIdescS = (1u << 4) | ((uint32_t)(kKcKeys >> 3) << 17) | (8u << 24);
constexpr uint32_t kKcIdescO = kKcIdescS | (1u << 16);
constexpr uint32_t kKcDescVLo = umma_mn_lo(kKcBlock);

// What differs where there are few new tokens (LONE), so that every tile takes both
// places and the cache's bytes count: one Q tile; a second group of dequantising
// warps, the groups taking the blocks in turn, each with stages of its own of half a
// block; and fewer registers for the softmax, which then reads S twice.
template <bool LONE>
struct KcCfg {
  static constexpr int kTiles = LONE ? 1 : 2;         // of Q
  static constexpr int kDeq = LONE ? 2 : 1;           // groups of four dequantising warps
  static constexpr int kRaw = LONE ? 2 * kDeq : 4 * kKcRaw;             // stages of records
  static constexpr uint32_t kStage = LONE ? kKcHalf * kKv4Rec : kKcRunBytes;
  static constexpr int kWarpMma = kKcWarpDeq + 4 * kDeq, kWarpCopy = kWarpMma + 1, kWarpQ = kWarpMma + 2;
  static constexpr int kThreads = 32 * (kWarpMma + 4);
  // registers a thread: 128 at launch (512 threads) or 96 (640). Softmax 176 (two
  // warpgroups), dequantisation 88, the rest 72: 2 * 176 + 88 + 72 = 4 * 128; or 128,
  // 72 (two) and 72: 2 * 128 + 2 * 72 + 72 < 5 * 96
  static constexpr int kRegSoft = LONE ? 128 : 176, kRegDeq = LONE ? 72 : 88, kRegRest = 72;
  // shared memory, from a 1024-byte aligned base
  static constexpr uint32_t kOffQ = 0;                                    // [kTiles]
  static constexpr uint32_t kOffKv = kOffQ + kTiles * kKcTile;
  static constexpr uint32_t kOffRaw = kOffKv + kKcSlots * kKcTile;        // [kRaw]
  static constexpr uint32_t kOffItem = kOffRaw + kRaw * kStage;           // [kKcItems] KcItem
  static constexpr uint32_t kOffNan = kOffItem + kKcItems * 64;           // [kKcItems][8] first position with a NaN V scale
  static constexpr uint32_t kOffMask = kOffNan + kKcItems * 32;           // [kKcMasks][4 words]
  static constexpr uint32_t kOffMl = kOffMask + kKcMasks * 16;            // [128] maximum and sum of tile B's row, for tile A
  static constexpr uint32_t kOffInv = kOffMl + 128 * 8;                   // [128] scale of tile A's row, for tile B
  static constexpr uint32_t kOffBar = kOffInv + 128 * 4;
  static constexpr int kBars = 2 * kRaw + 2 * kKcSlots + 2 * kKcItems + 2 * 6 + 2 * 4 + 1;
  static constexpr size_t kSmem = 1024 + kOffBar + kBars * 8 + 16;
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

// workspace: status; for each CTA the item that is cut first there; partials, of
// a CTA's first and last piece, two tiles each
constexpr size_t kKcOffCut = 256;
constexpr size_t kKcOffPart = kKcOffCut + (size_t)kKcCtas * 64;
constexpr int kKcPart = kD + 4;                       // a row's partial: O[128], and maximum, sum, their factor and the queries' scale
static_assert(kKcOffPart % 128 == 0, "aligned partials");
constexpr int kKcMergeThreads = 256;

struct KcItem {
  int row0, n;             // the request's first row and new tokens; n < 0: no more items
  int len, g, t0;          // its positions, KV head, first token of tile A
  int j0, j1;              // the piece's blocks
  int n0, n1;              // how many of them tile A and B take
  int single;              // one tile in both places
  int pieces, piece, first;  // of the item, and its first CTA
  int pad[3];
};
static_assert(sizeof(KcItem) == 64, "item ring");

struct KcArgs {
  Kv4ChunkCall c;
  int G, gshift, tpm;      // heads a group, its log2, tokens a tile
  int part_rows;           // rows of a tile that can be new tokens'
  int* status;
  KcItem* cut;
  float* part;
  long long wait_limit;
  int starve;              // test builds: no copy is issued, so that every wait runs out
};


__device__ __forceinline__ bool kc_wait(const KcArgs& a, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.wait_limit));
}

// 32 products of a row: weights 2^((s - m) f + bias) to 16 packed columns, and their sum
__device__ __forceinline__ void kc_weights(const float* s, float f, float m, float2 (&sum)[2], uint32_t tp) {
  const float2 nm = make_float2(-m, -m), ff = make_float2(f, f), bias = make_float2(kKcBias, kKcBias);
  uint32_t p[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float2 x = fma2(add2(make_float2(s[2 * e], s[2 * e + 1]), nm), ff, bias);
    x.x = ex2_approx(x.x);
    x.y = ex2_approx(x.y);
    sum[e & 1] = add2(sum[e & 1], x);
    p[e] = pack_f16(x.x, x.y);
  }
  tmem_st16(tp, p);
}

// A row of 128 values of 64 bytes of codes and 8 scales into row r of a swizzled tile.
// In a loop: one warp (or two) of an SM's quarter runs this code, and unrolled it
// waits for its own instructions (2048 tokens behind 64K 2.97 ms, unrolled 3.26;
// 16 ragged requests 772 us, unrolled 930)
__device__ __forceinline__ void kc_row(const uint4* codes, uint32_t sc0, uint32_t sc1, uint32_t tile, int r) {
  const uint32_t dst = tile + (uint32_t)r * 128u, r7 = (uint32_t)r & 7u;
  uint4 c0 = codes[0], c1 = codes[1], c2 = codes[2], c3 = codes[3];
  uint32_t at = dst, x = r7;                          // x: the place of four 16-byte units in their row of eight
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    const uint32_t s2 = e4m3x2_to_f16(sc0 & 0xffffu);
    sc0 = __funnelshift_r(sc0, sc1, 16);
    sc1 >>= 16;
    const uint32_t s[2] = {__byte_perm(s2, s2, 0x1010), __byte_perm(s2, s2, 0x3232)};
    const uint32_t ww[4] = {c0.x, c0.y, c0.z, c0.w};
    c0 = c1;
    c1 = c2;
    c2 = c3;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t h[4];
      e2m1x8_to_f16(ww[e], h);
      sts_v4(at + ((x ^ (uint32_t)e) << 4), hmul2(h[0], s[e >> 1]), hmul2(h[1], s[e >> 1]), hmul2(h[2], s[e >> 1]),
             hmul2(h[3], s[e >> 1]));
    }
    x ^= 4u;
    if (q == 1) at += kKcBlock;
  }
}

// A row of queries, bf16 to fp16 times a power of two, in place; returns the
// power's inverse. A row that is not finite becomes NaN: whatever it sees, its
// softmax has no value.
__device__ __forceinline__ float kc_query(uint32_t tile, int r) {
  uint4 w[16];
  uint32_t mx = 0u;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    w[u] = lds_v4(tile + (uint32_t)r * 128u + (u >> 3) * kKcBlock + (u & 7) * 16);
    mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(w[u].x & 0x7fff7fffu, w[u].y & 0x7fff7fffu),
                               __vmaxu2(w[u].z & 0x7fff7fffu, w[u].w & 0x7fff7fffu)));
  }
  const int E = (int)(max(mx & 0xffffu, mx >> 16) >> 7);       // exponent field of the largest
  const bool odd = E == 255;
  const int e = min(141 - E, 126);
  const float up = __int_as_float((e + 127) << 23);
  auto f16 = [&](uint32_t x) { return odd ? 0x7fff7fffu : pack_f16(bf_lo(x) * up, bf_hi(x) * up); };
#pragma unroll
  for (int u = 0; u < 16; ++u)
    sts_v4(tile + (uint32_t)r * 128u + (u >> 3) * kKcBlock + (u & 7) * 16, f16(w[u].x), f16(w[u].y), f16(w[u].z), f16(w[u].w));
  return __int_as_float((127 - e) << 23);
}

// ---------------------------------------------------------------- the line of work
// Items of a request: item i holds tokens [i t, (i + 1) t), two tiles' or one's,
// and sees ceil((ctx + (i + 1) t) / 128) blocks, ctx = len - n, at least one. An
// item's units are its fixed part's, then its blocks'.
struct KcShape {
  int ctx, n, lt, pairs;       // lt: log2 of t; items
};
__device__ __forceinline__ int kc_blocks(const KcShape& s, int i) {
  return max(1, (s.ctx + min(s.n, (i + 1) << s.lt) + kKcKeys - 1) >> 7);
}
// units of a block of item i: it is one tile, or two
template <bool LONE>
__device__ __forceinline__ bool kc_single(const KcShape& s, int i) {
  return LONE || 2 * i + 2 > (s.n + (1 << (s.lt - 1)) - 1) >> (s.lt - 1);
}
template <bool LONE>
__device__ __forceinline__ int kc_unit(const KcShape& s, int i) { return kc_single<LONE>(s, i) ? kKcUnitsOne : kKcUnitsTwo; }
// units of the items below k <= items - 1, none of them the last one
template <bool LONE>
__device__ __forceinline__ long long kc_units(const KcShape& s, int k) {
  constexpr int lb = 7, mask = kKcKeys - 1;
  const int lt = s.lt;
  // the first ones see one block (or nothing), from i0 on the sum of an arithmetic progression's quotients
  const int i0 = max(0, min(k, (mask + 1 - s.ctx) >> lt)), m = k - i0;
  const int each = LONE ? kKcUnitsOne : kKcUnitsTwo;
  const long long u = (long long)k * kKcFixed + (long long)i0 * each;
  if (m == 0) return u;
  const int c = s.ctx + (i0 << lt);
  if (lt >= lb) return u + each * ((long long)m * ((c + mask) >> lb) + ((long long)m * (m + 1) / 2 << (lt - lb)));
  const int ls = lb - lt, w = (1 << ls) - 1 + ((c & ((1 << lt) - 1)) > 0 ? 1 : 0);
  const long long a = (c >> lt) + w;                  // sum of floor((a + i) / 2^ls), i = 1 .. m
  auto below = [&](long long x) {                     // sum of floor(j / 2^ls), j = 0 .. x
    const long long q = (x + 1) >> ls, r = (x + 1) & ((1 << ls) - 1);
    return (q * (q - 1) / 2 << ls) + r * q;
  };
  return u + each * (below(a + m) - below(a));
}
// a row's log-sum-exp; the queries' factor goes to the scale, for q.K itself may be beyond fp32's range (and
// where the two are, a product of zero stays one)
__device__ __forceinline__ float kc_lse(const KcArgs& a, float m, float l, float inv) {
  return l == 0.f ? -INFINITY : m * fminf(inv * a.c.scale, 3.40282347e38f) + (log2f(l) - kKcBias) * 0.6931471805599453f;
}
// A piece's partials of a tile: four dims of O of each row, [32][rows][4], then the
// rows' maxima and so on, [rows][4]: the lanes of a warp have consecutive rows,
// where they are written and where they are read
__device__ __forceinline__ float4* kc_part(const KcArgs& a, int cta, int last, int tile) {
  return reinterpret_cast<float4*>(a.part) + (((size_t)cta * 2 + last) * 2 + tile) * a.part_rows * (kKcPart / 4);
}

// The partials of the items that are cut. A warp has 16 dims of 32 rows, a row a
// lane, and goes through the pieces once, with the running maximum: nothing that
// it loads depends on what it has loaded but the number of pieces. (A warp a row,
// maxima first, then the weights, then O, and four rows in turn: 8.4 us of the 23
// that 17 tokens behind 1000 took.)
__global__ void __launch_bounds__(kKcMergeThreads) kv4_chunk_merge_kernel(const KcArgs a) {
  const Kv4ChunkCall& c = a.c;
  kc_wait_first();
  const KcItem x = a.cut[blockIdx.x];
  const int warp = threadIdx.x >> 5, row = blockIdx.y * 32 + (threadIdx.x & 31), i = blockIdx.z;
  if (x.pieces < 2 || (x.single && i)) return;
  const int t0 = x.t0 + i * a.tpm;
  if (row >= min((long long)(x.n - t0) << a.gshift, 128ll)) return;
  float m = -INFINITY, l = 0.f, f = 0.f, inv = 0.f, o[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] = 0.f;
  constexpr int U = 4;                                // pieces whose loads are in flight together
  for (int k0 = 0; k0 < x.pieces; k0 += U) {
    float4 ml[U], v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u >= x.pieces) continue;
      // piece k is its CTA's last one for k = 0, else its first
      const float4* p = kc_part(a, x.first + k0 + u, k0 + u == 0, i) + row;
      ml[u] = p[(size_t)(kD / 4) * a.part_rows];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[u][e] = p[(size_t)(4 * warp + e) * a.part_rows];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u >= x.pieces) continue;
      f = ml[u].z;
      inv = ml[u].w;
      if (ml[u].y == 0.f) continue;                   // the row saw nothing, and its O may not have been written
      const float M = fmaxf(m, ml[u].x), wo = l == 0.f ? 0.f : ex2_approx((m - M) * f), wn = ex2_approx((ml[u].x - M) * f);
      m = M;
      l = l * wo + ml[u].y * wn;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[4 * e] = o[4 * e] * wo + v[u][e].x * wn;
        o[4 * e + 1] = o[4 * e + 1] * wo + v[u][e].y * wn;
        o[4 * e + 2] = o[4 * e + 2] * wo + v[u][e].z * wn;
        o[4 * e + 3] = o[4 * e + 3] * wo + v[u][e].w * wn;
      }
    }
  }
  const float r = l == 0.f ? 0.f : 1.f / l;
  const size_t at = (size_t)(x.row0 + t0 + (row >> a.gshift)) * c.n_q + (x.g << a.gshift) + (row & (a.G - 1));
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = pack_bf16(o[2 * e] * r, o[2 * e + 1] * r);
  uint16_t* d = c.out + at * kD + 16 * warp;
  stg_v4(d, make_uint4(w[0], w[1], w[2], w[3]));
  stg_v4(d + 8, make_uint4(w[4], w[5], w[6], w[7]));
  if (c.lse && warp == 0) c.lse[at] = kc_lse(a, m, l, inv);
}
static_assert(kKcMergeThreads == 32 * (kD / 16), "a warp for 16 dims");

template <bool LONE>
__global__ void __launch_bounds__(KcCfg<LONE>::kThreads, 1) kv4_chunk_kernel(const __grid_constant__ CUtensorMap qmap, const KcArgs a) {
  using Cfg = KcCfg<LONE>;
  constexpr int kDeqWarps = 4 * Cfg::kDeq;
  extern __shared__ uint8_t kc_raw[];
  const uint32_t raw_addr = smem_u32(kc_raw);
  uint8_t* base = kc_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  KcItem* items = reinterpret_cast<KcItem*>(base + Cfg::kOffItem);
  int* nans = reinterpret_cast<int*>(base + Cfg::kOffNan);
  uint32_t* masks = reinterpret_cast<uint32_t*>(base + Cfg::kOffMask);
  float2* ml_b = reinterpret_cast<float2*>(base + Cfg::kOffMl);
  float* inv_a = reinterpret_cast<float*>(base + Cfg::kOffInv);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + Cfg::kOffBar);
  uint64_t* rfull = bars;                     // [kRaw] bytes of the records ([4 warps][kKcRaw], LONE: [group][half block])
  uint64_t* rfree = rfull + Cfg::kRaw;        // [kRaw] the warp, or the group's four, have read them
  uint64_t* kvfull = rfree + Cfg::kRaw;       // [kKcSlots] four dequantising warps have written the operand
  uint64_t* kvfree = kvfull + kKcSlots;       // [kKcSlots] commit after the last MMA that reads it
  uint64_t* ifull = kvfree + kKcSlots;        // [kKcItems] item written
  uint64_t* ifree = ifull + kKcItems;         // [kKcItems] every role has read it, the softmax warps are done with it
  uint64_t* qfull = ifree + kKcItems;         // [2] TMA bytes
  uint64_t* qready = qfull + 2;               // [2] four softmax warps have converted the tile
  uint64_t* qfree = qready + 2;               // [2] commit after the tile's last S
  uint64_t* sfull = qfree + 2;                // [2] commit: S in tensor memory
  uint64_t* pfull = sfull + 2;                // [2] four softmax warps: P written, O rescaled; gate: the batch's operands are there
  uint64_t* ofull = pfull + 2;                // [2] commit: the piece's last PV done
  uint64_t* bdone = ofull + 2;                // [4] a warp of B: its rows' O, maxima and sums are there
  uint64_t* bread = bdone + 4;                // [4] the warp of A with the same rows has read them
  uint64_t* drain = bread + 4;                // commit after the last MMA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const Kv4ChunkCall& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kRaw; ++s) {
      mbar_init(&rfull[s], 1);
      mbar_init(&rfree[s], LONE ? 4 : 1);
    }
    for (int s = 0; s < kKcSlots; ++s) {
      mbar_init(&kvfull[s], 4);
      mbar_init(&kvfree[s], 1);
    }
    for (int s = 0; s < kKcItems; ++s) {
      mbar_init(&ifull[s], 1);
      mbar_init(&ifree[s], kDeqWarps + 8 + 3);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&qfull[s], 1);
      mbar_init(&qready[s], 4);
      mbar_init(&qfree[s], 1);
      mbar_init(&sfull[s], 1);
      mbar_init(&pfull[s], 5);
      mbar_init(&ofull[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bdone[s], 1);
      mbar_init(&bread[s], 1);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == Cfg::kWarpMma) tmem_alloc<kKcTmemCols>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  kc_let_next();
  const uint32_t qs = smem_u32(base + Cfg::kOffQ), kvs = smem_u32(base + Cfg::kOffKv);
  bool dead = false;
  auto acquire = [&](uint64_t* bar, uint32_t parity) {
    // mostly over: tested before it is waited for (some 90 cycles against 190)
    if (!dead && !__all_sync(0xffffffffu, mbar_test(bar, parity)) && !kc_wait(a, bar, parity)) {
      if (lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
      dead = true;
    }
  };

  if (warp == Cfg::kWarpCopy) {
    // ================= schedule and copies of the records
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(Cfg::kRegRest));
    KcRequests rq;
    kc_requests(c, rq);
    const int lt = (LONE ? 7 : 8) - a.gshift, bs = 1 << c.block_shift;
    auto shape = [&](int len, int n) {
      KcShape s;
      s.ctx = len - n;
      s.n = n;
      s.lt = lt;
      s.pairs = (n + (1 << lt) - 1) >> lt;
      return s;
    };
    auto units = [&](const KcShape& s) {              // of one KV head
      return s.n == 0 ? 0ll : kc_units<LONE>(s, s.pairs - 1) + kKcFixed +
                              (long long)kc_blocks(s, s.pairs - 1) * kc_unit<LONE>(s, s.pairs - 1);
    };
    long long own[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) own[e] = units(shape(rq.len[e], rq.n[e]));
    const long long total = kc_prefix(rq, own[0] * c.n_kv, own[1] * c.n_kv);
    const int ctas = (int)max(min(total, 1ll), min(total / kKcMinRun, (long long)gridDim.x));
    const bool has = (int)blockIdx.x < ctas;
    const long long u0 = has ? kc_div(total * blockIdx.x, ctas) : 0, u1 = has ? kc_div(total * (blockIdx.x + 1), ctas) : 0;
    auto cta_of = [&](long long u) { return (int)kc_div((u + 1) * ctas - 1, total); };
    // the item at u0: request b, head g, pair i; `at` is its first unit
    int b = 0, g = 0, i = 0;
    long long at = 0, whole = 1;
    KcShape s = shape(0, 0);
    auto enter = [&](int request) {                   // its shape and units a head
      b = request;
      s = shape(kc_of(rq.len, b), kc_of(rq.n, b));
      whole = __shfl_sync(0xffffffffu, b & 1 ? own[1] : own[0], b >> 1);
    };
    if (has) {
      enter(kc_find(rq, u0));
      long long r = u0 - (kc_of(rq.end, b) - whole * c.n_kv);
      g = (int)kc_div(r, whole);
      r -= (long long)g * whole;
      int lo = 0, hi = s.pairs;                       // units(lo) <= r
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (kc_units<LONE>(s, mid) <= r) lo = mid; else hi = mid;
      }
      i = lo;
      at = u0 - r + kc_units<LONE>(s, i);
    }
    int it = 0, blocks = 0, nraw = 0;
    if (lane == 0) a.cut[blockIdx.x].pieces = 0;      // unless an item goes on in the next CTA
    for (;; ) {
      KcItem x;
      x.n = -1;
      bool skip = false;
      if (has && at < u1 && !dead) {
        const int nb = kc_blocks(s, i);
        const long long first = at + kKcFixed;        // its first block's unit
        const int each = kc_unit<LONE>(s, i);         // a block is the CTA's in whose run it begins
        const int lo = (int)((max(0ll, u0 - first) + each - 1) / each);
        const int hi = (int)min((long long)nb, (max(0ll, u1 - first) + each - 1) / each);
        skip = hi <= lo;                              // no block begins here
        if (!skip) {
          x.row0 = kc_of(rq.row0, b);
          x.n = s.n;
          x.len = s.ctx + s.n;
          x.g = g;
          x.t0 = i << lt;
          x.single = kc_single<LONE>(s, i);
          x.j0 = lo;
          x.j1 = hi;
          if (x.single) {
            x.n0 = (x.j1 - x.j0 + 1) >> 1;
            x.n1 = (x.j1 - x.j0) >> 1;
          } else {
            // tile A sees the blocks up to its own last token
            const int na = max(1, (s.ctx + min(s.n, x.t0 + a.tpm) + kKcKeys - 1) >> 7);
            x.n0 = max(0, min(x.j1, na) - x.j0);
            x.n1 = x.j1 - x.j0;
          }
          const bool cut = lo > 0 || hi < nb;
          x.first = lo > 0 ? cta_of(first) : (int)blockIdx.x;
          x.pieces = cut ? cta_of(first + (long long)(nb - 1) * each) - x.first + 1 : 1;
          x.piece = (int)blockIdx.x - x.first;
          if (x.pieces > 1 && x.piece == 0 && lane == 0) a.cut[blockIdx.x] = x;
        }
      }
      if (!skip) {
        const int is = it % kKcItems;
        acquire(&ifree[is], ((it / kKcItems) & 1) ^ 1);
        if (lane == 0) items[is] = x;
        if (lane < 8) nans[is * 8 + lane] = INT_MAX;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ifull[is]);
        ++it;
        if (x.n < 0) break;
#ifdef SPC_TEST_HOOKS
        if (a.starve) break;
#endif
        KcTable t;
        t.start(c.table + (size_t)b * c.max_blocks, (x.len + bs - 1) >> c.block_shift, x.j0 * kKcKeys >> c.block_shift);
        if constexpr (LONE) {
          for (int j = x.j0; j < x.j1 && !dead; ++j, ++blocks) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              const int st = (blocks & 1) * 2 + h;
              acquire(&rfree[st], ((blocks >> 1) & 1) ^ 1);
              if (dead) break;
              kc_copy(c, t, x.g, x.len, j * kKcKeys + h * kKcHalf, base + Cfg::kOffRaw + st * Cfg::kStage, &rfull[st],
                      masks + (blocks % kKcMasks) * 4 + 2 * h);
            }
          }
        } else {
          // lane w copies for dequantising warp w
          for (int j = x.j0; j < x.j1 && !dead; ++j, ++blocks) {
            uint32_t mask = 0u;
#pragma unroll 1
            for (int h = 0; h < 2; ++h, ++nraw) {
              const int st = nraw % kKcRaw, p = j * kKcKeys + (lane & 3) * 32 + h * kKcRun;
              const int blk = t.entry(j * kKcKeys >> c.block_shift, p >> c.block_shift);
              const int n = (unsigned)blk < (unsigned)c.num_blocks ? max(0, min(x.len - p, kKcRun)) : 0;
              mask |= ((1u << n) - 1u) << (h * kKcRun);
              const uint32_t parity = ((nraw / kKcRaw) & 1) ^ 1;
              uint64_t* bar = &rfull[(lane & 3) * kKcRaw + st];
              if (!__all_sync(0xffffffffu, mbar_wait_bounded(&rfree[(lane & 3) * kKcRaw + st], parity, a.wait_limit))) {
                if (lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
                dead = true;
                break;
              }
              if (lane < 4) {
                if (h == 1) masks[(blocks % kKcMasks) * 4 + lane] = mask;
                if (n > 0) mbar_arrive_expect_tx(bar, (uint32_t)n * kKv4Rec); else mbar_arrive(bar);
                if (n > 0)
                  bulk_g2s(base + Cfg::kOffRaw + (lane * kKcRaw + st) * kKcRunBytes,
                           c.cache + (((size_t)blk * c.n_kv + x.g) * bs + (p & (bs - 1))) * kKv4Rec, (uint32_t)n * kKv4Rec, bar);
              }
              __syncwarp();
            }
          }
        }
      }
      // the next item
      at += kKcFixed + (long long)kc_blocks(s, i) * kc_unit<LONE>(s, i);
      if (++i == s.pairs) {
        i = 0;
        if (++g == c.n_kv) {
          g = 0;
          if (at < u1) enter(kc_find(rq, at));
        }
      }
    }
    // every copy lands before the CTA ends (they have, unless a role gave up)
    if constexpr (LONE) {
      if (lane == 0)
        for (int k = max(0, 2 * blocks - Cfg::kRaw); k < 2 * blocks; ++k)     // each stage's last use
          mbar_wait_bounded(&rfull[(k >> 1 & 1) * 2 + (k & 1)], (k >> 2) & 1, a.wait_limit);
    } else if (lane < 4) {
      for (int k = max(0, nraw - kKcRaw); k < nraw; ++k)
        mbar_wait_bounded(&rfull[lane * kKcRaw + k % kKcRaw], (k / kKcRaw) & 1, a.wait_limit);
    }
    __syncwarp();
  } else if (warp == Cfg::kWarpQ) {
    // ================= queries
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(Cfg::kRegRest));
    int nq[2] = {0, 0};
    for (int it = 0;; ++it) {
      const int is = it % kKcItems;
      acquire(&ifull[is], (it / kKcItems) & 1);
      if (dead) break;
      const int n = items[is].n, n0 = items[is].n0, n1 = items[is].n1, row = items[is].row0 + items[is].t0, g = items[is].g;
      const int single = items[is].single;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
      if (n < 0) break;
#ifdef SPC_TEST_HOOKS
      if (a.starve) break;
#endif
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        if (i ? LONE || n1 == 0 : n0 == 0) continue;
        acquire(&qfree[i], (nq[i] & 1) ^ 1);
        if (dead) break;
        ++nq[i];
        if (lane == 0) {
          mbar_arrive_expect_tx(&qfull[i], kKcTile);
          const int r = row + (single ? 0 : i * a.tpm);
          tma_load_3d(qs + i * kKcTile, &qmap, 0, g << a.gshift, r, &qfull[i]);
          tma_load_3d(qs + i * kKcTile + kKcBlock, &qmap, 64, g << a.gshift, r, &qfull[i]);
        }
        __syncwarp();
      }
      if (dead) break;
    }
    if (lane == 0)
      for (int i = 0; i < 2; ++i)
        if (nq[i] > 0) mbar_wait_bounded(&qfull[i], (nq[i] - 1) & 1, a.wait_limit);
    __syncwarp();
  } else if (warp == Cfg::kWarpMma) {
    // ================= MMA issue; the whole warp runs the loop, so that its values stay warp-uniform
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(Cfg::kRegRest));
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    int kv = 0, nq[2] = {0, 0}, np[2] = {0, 0};
    auto full = [&](int k) {                          // operand k has been written
      acquire(&kvfull[k % kKcSlots], (k / kKcSlots) & 1);
    };
    // S of tile i against operand k; first: of its Q, last: no further one. `done`: nothing else reads k
    auto issue_s = [&](auto tile, int k, bool first, bool last, bool done) {
      constexpr int i = decltype(tile)::value, qi = LONE ? 0 : i;
      if (first) acquire(&qready[qi], nq[qi]++ & 1);
      if (dead) return;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t qd = umma_desc_lo(qs + qi * kKcTile), kd = umma_desc_lo(kvs) + (uint32_t)(k % kKcSlots) * (kKcTile >> 4);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t off = (uint32_t)(kk >> 2) * (kKcBlock >> 4) + (uint32_t)(kk & 3) * 2;
          umma_f16(tm + i * kKcKeys, umma_desc(qd + off), umma_desc(kd + off), kKcIdescS, kk ? 1u : 0u);
        }
        umma_commit(&sfull[i]);
        if (last) umma_commit(&qfree[qi]);
        if (done) umma_commit(&kvfree[k % kKcSlots]);
      }
      __syncwarp();
    };
    auto issue_pv = [&](auto tile, int k, bool first, bool last, bool done) {
      constexpr int i = decltype(tile)::value;
      acquire(&pfull[i], np[i]++ & 1);
      if (dead) return;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t vd = umma_desc_lo(kvs) + (uint32_t)(k % kKcSlots) * (kKcTile >> 4) + kKcDescVLo;
#pragma unroll
        for (int kk = 0; kk < kKcKeys / 16; ++kk)
          umma_f16_tmem_a(tm + kKcColO + i * kD, tm + i * kKcKeys + kk * 8, umma_desc(vd + (uint32_t)kk * 128), kKcIdescO,
                          kk ? 1u : (first ? 0u : 1u));
        if (done) umma_commit(&kvfree[k % kKcSlots]);
        if (last) umma_commit(&ofull[i]);
      }
      __syncwarp();
    };
    constexpr std::integral_constant<int, 0> tA{};
    constexpr std::integral_constant<int, 1> tB{};
    for (int it = 0;; ++it) {
      const int is = it % kKcItems;
      acquire(&ifull[is], (it / kKcItems) & 1);
      if (dead) break;
      const int n = items[is].n, n0 = items[is].n0, n1 = items[is].n1, nb = items[is].j1 - items[is].j0;
      const int single = items[is].single;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
      if (n < 0) break;
      // operand kv + 2 k is K of the piece's block k, kv + 2 k + 1 its V
      full(kv);
      if (LONE || single) {
        // LONE: the two have one Q, whose last use is the last block's
        issue_s(tA, kv, true, LONE ? nb == 1 : n0 == 1, true);
        if (n1) {
          full(kv + 2);
          issue_s(tB, kv + 2, !LONE, LONE ? nb == 2 : n1 == 1, true);
        }
#pragma unroll 1
        for (int k = 0; k < nb && !dead; k += 2) {
          issue_pv(tA, kv + 2 * k + 1, k == 0, k + 2 >= nb, true);
          if (k + 2 < nb) {
            full(kv + 2 * k + 4);
            issue_s(tA, kv + 2 * k + 4, false, LONE ? k + 3 == nb : k + 4 >= nb, true);
          }
          if (k + 1 < nb) issue_pv(tB, kv + 2 * k + 3, k == 0, k + 3 >= nb, true);
          if (k + 3 < nb) {
            full(kv + 2 * k + 6);
            issue_s(tB, kv + 2 * k + 6, false, LONE ? k + 4 == nb : k + 5 >= nb, true);
          }
        }
      } else {
        if (n0) issue_s(tA, kv, true, n0 == 1, n1 == 0);
        if (n1) issue_s(tB, kv, true, n1 == 1, true);
#pragma unroll 1
        for (int k = 0; k < nb && !dead; ++k) {
          // PV of block k, S of the next one; the tensor pipe queues only a few MMAs, so nothing waits between the two
          const int v = kv + 2 * k + 1;
          if (k < n0) issue_pv(tA, v, k == 0, k + 1 == n0, k >= n1);
          if (k + 1 < n0) issue_s(tA, v + 1, false, k + 2 == n0, k + 1 >= n1);
          if (k < n1) issue_pv(tB, v, k == 0, k + 1 == n1, true);
          if (k + 1 < n1) issue_s(tB, v + 1, false, k + 2 == n1, true);
        }
      }
      kv += 2 * nb;
      if (dead) break;
    }
    // tensor memory is released below: every MMA has completed (the softmax
    // warps wait for each piece's last one, unless something gave up)
    if (elect_one()) umma_commit(drain);
    __syncwarp();
    kc_wait(a, drain, 0);
  } else if (warp >= kKcWarpDeq && warp < Cfg::kWarpMma) {
    // ================= dequantisation, a record a thread
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(Cfg::kRegDeq));
    const int w = warp - kKcWarpDeq, r = threadIdx.x & 127;
    int blocks = 0, kv = 0, nread = 0;
    for (int it = 0;; ++it) {
      const int is = it % kKcItems;
      acquire(&ifull[is], (it / kKcItems) & 1);
      if (dead) break;
      const int n = items[is].n, j0 = items[is].j0, j1 = items[is].j1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
      if (n < 0) break;
      for (int j = j0; j < j1; ++j, ++blocks, kv += 2) {
        // the whole record into registers, so that its stage is free at once
        int s0, s1;
        uint32_t rec;
        if constexpr (LONE) {
          if ((blocks & 1) != w >> 2) continue;
          s0 = (blocks & 1) * 2;
          s1 = s0 + 1;
          acquire(&rfull[s0], (blocks >> 1) & 1);
          acquire(&rfull[s1], (blocks >> 1) & 1);
          rec = smem_u32(base + Cfg::kOffRaw) + (uint32_t)s0 * Cfg::kStage + (uint32_t)r * kKv4Rec;   // the two lie one behind the other
        } else {
          s0 = w * kKcRaw + nread % kKcRaw;
          s1 = w * kKcRaw + (nread + 1) % kKcRaw;
          acquire(&rfull[s0], (nread / kKcRaw) & 1);
          acquire(&rfull[s1], ((nread + 1) / kKcRaw) & 1);
          nread += 2;
          rec = smem_u32(base + Cfg::kOffRaw) + (uint32_t)(lane < kKcRun ? s0 : s1) * Cfg::kStage +
                (uint32_t)(lane & (kKcRun - 1)) * kKv4Rec;
        }
        if (dead) break;
        const bool there = masks[(blocks % kKcMasks) * 4 + (w & 3)] >> lane & 1;
        uint4 v[9];
#pragma unroll
        for (int q = 0; q < 9; ++q) v[q] = lds_v4(rec + 16 * q);
        __syncwarp();
        if (lane < 2) mbar_arrive(&rfree[lane ? s1 : s0]);
        if (!there) {
#pragma unroll
          for (int q = 0; q < 9; ++q) v[q] = make_uint4(0u, 0u, 0u, 0u);
        }
        // scales of V that are NaN: noted, and zero in the product
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t& x = e ? v[8].w : v[8].z;
          const uint32_t bad = ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
          if (bad) {
#pragma unroll
            for (int f = 0; f < 4; ++f)
              if (bad >> (8 * f + 7) & 1) {
                atomicMin(&nans[is * 8 + 4 * e + f], j * kKcKeys + r);
                x &= ~(0xffu << (8 * f));
              }
          }
        }
#pragma unroll
        for (int part = 0; part < 2; ++part) {        // K, then V
          const int slot = (kv + part) % kKcSlots;
          acquire(&kvfree[slot], (((kv + part) / kKcSlots) & 1) ^ 1);
          if (dead) break;
          if (part) kc_row(v + 4, v[8].z, v[8].w, kvs + (uint32_t)slot * kKcTile, r);
          else kc_row(v, v[8].x, v[8].y, kvs + (uint32_t)slot * kKcTile, r);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&kvfull[slot]);
        }
        if (dead) break;
      }
      if (dead) break;
    }
  } else if (warp < kKcWarpDeq) {
    // ================= softmax and epilogue of tile i, one row a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(Cfg::kRegSoft));
    const int i = warp >> 2, wq = warp & 3, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t ts = tmem + lanes + i * kKcKeys, to = tmem + lanes + kKcColO + i * kD;
    int n_q = 0, n_s = 0, n_o = 0, n_b = 0, blocks = 0;
    for (int it = 0;; ++it) {
      const int is = it % kKcItems;
      acquire(&ifull[is], (it / kKcItems) & 1);
      if (dead) break;
      const KcItem x = items[is];
      if (x.n < 0) break;
      const int n = i ? x.n1 : x.n0, t0 = x.t0 + (x.single ? 0 : i * a.tpm);
      const int token = t0 + (row >> a.gshift), qpos = x.len - x.n + token, qpos0 = x.len - x.n + t0;
      const int hq = (x.g << a.gshift) + (row & (a.G - 1));
      float m = -INFINITY, l = 0.f, inv = 1.f;
      if (LONE && i) {
        if (n > 0) {                                  // tile A's rows: their scales are there when an S is
          acquire(&sfull[i], n_s & 1);
          if (dead) break;
          inv = inv_a[row];
        }
      } else if (n > 0) {
        acquire(&qfull[i], n_q & 1);
        if (dead) break;
        ++n_q;
        inv = kc_query(qs + i * kKcTile, row);
        if (LONE) inv_a[row] = inv;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&qready[i]);
      } else if (x.pieces > 1 && !x.single) {
        // a piece without a block of this tile's: the rows' factors, for the merge
        const int t = min(x.row0 + token, c.T - 1);
        uint32_t mx = 0u;
        for (int u = 0; u < 16; ++u) {
          const uint4 w = *reinterpret_cast<const uint4*>(c.q + t * c.q_stride + (size_t)hq * kD + 8 * u);
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                     __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
        }
        inv = __int_as_float((127 - min(141 - (int)(max(mx & 0xffffu, mx >> 16) >> 7), 126)) << 23);
      }
      const float f = k4_factor(inv * c.scale * kLog2e);
      for (int k = 0; k < n; ++k) {
        const int j = x.single ? x.j0 + 2 * k + i : x.j0 + k;
        acquire(&sfull[i], n_s & 1);
        if (dead) break;
        tc_fence_after();
        const uint4 mask = *reinterpret_cast<const uint4*>(masks + ((blocks + j - x.j0) % kKcMasks) * 4);
        const bool there = (mask.x & mask.y & mask.z & mask.w) == 0xffffffffu;
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // raises the row's maximum to M where that is needed
        auto raise = [&](float M) {
          float alpha = 1.f;
          const bool up = (M - m) * f > kKcHeadroom;
          if (up) {
            alpha = m == -INFINITY ? 0.f : ex2_approx((m - M) * f);
            l *= alpha;
            m = M;
          }
          if (k > 0 && __any_sync(0xffffffffu, up)) {
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
        if (there && (j + 1) * kKcKeys <= qpos0 + 1) {
          // every row sees the whole block
          if constexpr (LONE) {
            // twice from tensor memory: there are not the registers to keep a row
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              float v[32];
              tmem_ld32(ts + 32 * q, v);
              tmem_ld_wait32(v);
              max32(v, mx);
            }
            raise(max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]));
            const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              float v[32];
              tmem_ld32(ts + 32 * q, v);
              tmem_ld_wait32(v);
              kc_weights(v, f, mm, sum, ts + 16 * q);
            }
          } else {
            // once (2.93 ms for 2048 tokens behind 64K, in two passes in loops 3.25)
            float s[128];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, *reinterpret_cast<float (*)[32]>(s + 32 * q));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              tmem_ld_wait32(s + 32 * q);
              max32(s + 32 * q, mx);
            }
            raise(max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]));
            const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int q = 0; q < 4; ++q) kc_weights(s + 32 * q, f, mm, sum, ts + 16 * q);
          }
        } else {
          // a block with an end or a gap in it, and the last ones: S is read twice, in chunks of 32 columns, without the
          // chunks behind the last column that a row of the warp sees
          const int seen = qpos - j * kKcKeys, seen1 = qpos0 + ((wq * 32 + 31) >> a.gshift) - j * kKcKeys;
          auto load = [&](int q, float (&v)[32]) {
            tmem_ld32(ts + 32 * q, v);
            tmem_ld_wait32(v);
            const int cols = seen + 1 - 32 * q;
            const uint32_t vis = (q == 0 ? mask.x : q == 1 ? mask.y : q == 2 ? mask.z : mask.w) &
                                 (cols >= 32 ? 0xffffffffu : cols <= 0 ? 0u : (1u << cols) - 1u);
            if (!__all_sync(0xffffffffu, vis == 0xffffffffu)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(vis >> e & 1)) v[e] = -INFINITY;
            }
          };
          const int nq = seen1 < 0 ? 0 : min(4, seen1 / 32 + 1);
#pragma unroll 1
          for (int q = 0; q < nq; ++q) {
            float v[32];
            load(q, v);
            max32(v, mx);
          }
          raise(max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]));
          const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll 1
          for (int q = 0; q < nq; ++q) {
            float v[32];
            load(q, v);
            kc_weights(v, f, mm, sum, ts + 16 * q);
          }
          const uint32_t none[16] = {};
#pragma unroll 1
          for (int q = nq; q < 4; ++q) tmem_st16(ts + 16 * q, none);
        }
        l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[i]);
        ++n_s;
      }
      if (dead) break;
      blocks += x.j1 - x.j0;
      // ---- epilogue
      if (n > 0) {
        acquire(&ofull[i], n_o & 1);
        if (dead) break;
        ++n_o;
        tc_fence_after();
      }
      if (i && x.single) {
        // tile B: its warp's maxima and sums to the warp of A that has the same rows, which reads O as well
        if (n > 0) {
          ml_b[row] = make_float2(m, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bdone[wq]);
          acquire(&bread[wq], n_b++ & 1);
          if (dead) break;
        }
      } else if (n > 0 || x.pieces > 1) {
        const bool live = token < x.n;
        const bool both = x.single && x.n1 > 0;
        float wa = 1.f, wb = 0.f;
        if (both) {
          acquire(&bdone[wq], n_b++ & 1);
          if (dead) break;
          tc_fence_after();
          const float2 ml = ml_b[row];
          const float M = fmaxf(m, ml.x);
          wa = l == 0.f ? 0.f : ex2_approx((m - M) * f);
          wb = ml.y == 0.f ? 0.f : ex2_approx((ml.x - M) * f);
          m = M;
          l = l * wa + ml.y * wb;
        }
        const bool cut = x.pieces > 1;
        float4* p = kc_part(a, blockIdx.x, x.piece == 0, i) + row;
        const float r = cut ? 1.f : l == 0.f ? 0.f : 1.f / l;
        wa *= r;
        wb *= r;
        uint16_t* dst = c.out + ((size_t)(x.row0 + token) * c.n_q + hq) * kD;
        const bool wide = (reinterpret_cast<uintptr_t>(c.out) & 31u) == 0;     // whole sectors a store
        if (n > 0) {
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {               // the 16 dims of a scale
            float o[16];
            tmem_ld16(to + 16 * q, o);
            if (both) {
              float ob[16];
              tmem_ld16(tmem + lanes + kKcColO + kD + 16 * q, ob);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = o[e] * wa + ob[e] * wb;
            } else {
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= wa;
            }
            if (nans[is * 8 + q] <= qpos) {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = NAN;
            }
            if (!live) continue;
            if (cut) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                p[(size_t)(4 * q + e) * a.part_rows] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
              continue;
            }
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = pack_bf16(o[2 * e], o[2 * e + 1]);
            uint16_t* d = dst + 16 * q;
            if (wide) {
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" :: "l"(d), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                           "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
            } else {
              stg_v4(d, make_uint4(w[0], w[1], w[2], w[3]));
              stg_v4(d + 8, make_uint4(w[4], w[5], w[6], w[7]));
            }
          }
          tc_fence_before();
        }
        if (both) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bread[wq]);
        }
        if (live && cut) p[(size_t)(kD / 4) * a.part_rows] = make_float4(m, l, f, inv);
        if (live && !cut && c.lse) c.lse[(size_t)(x.row0 + token) * c.n_q + hq] = kc_lse(a, m, l, inv);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
    }
  } else {                                    // the last warp
    // ================= gate: one arrival a phase of the P barriers, when what the batch behind it reads is there
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(Cfg::kRegRest));
    int kv = 0, np[2] = {0, 0};
    for (int it = 0; !dead; ++it) {
      const int is = it % kKcItems;
      acquire(&ifull[is], (it / kKcItems) & 1);
      if (dead) break;
      const int n = items[is].n, n0 = items[is].n0, n1 = items[is].n1, nb = items[is].j1 - items[is].j0;
      const int single = items[is].single;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ifree[is]);
      if (n < 0) break;
      for (int k = 0; k < nb; ++k) {
        // V of the block, and K of the next one where both tiles take it
        const int v = kv + 2 * k + 1;
        acquire(&kvfull[v % kKcSlots], (v / kKcSlots) & 1);
        if (!single && k + 1 < nb) acquire(&kvfull[(v + 1) % kKcSlots], ((v + 1) / kKcSlots) & 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (single ? (k & 1) != i : k >= (i ? n1 : n0)) continue;
          if (np[i] > 0) acquire(&pfull[i], (np[i] - 1) & 1);      // the phase before is over
          if (dead) break;
          ++np[i];
          if (lane == 0) mbar_arrive(&pfull[i]);
        }
        if (dead) break;
      }
      kv += 2 * nb;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == Cfg::kWarpMma) {
    tc_fence_after();
    tmem_dealloc<kKcTmemCols>(tmem);
  }
}

static int kc_part_rows(int T, int G) { return (long long)T * G < 128 ? T * G : 128; }

size_t kv4_chunk_workspace(int T, int, int n_q, int n_kv) {
  return kKcOffPart + (size_t)kKcCtas * 2 * 2 * kc_part_rows(T, n_q / n_kv) * kKcPart * 4;
}

template <bool LONE>
static int kc_launch(const CUtensorMap& qmap, const KcArgs& a, cudaStream_t st) {
  constexpr size_t smem = KcCfg<LONE>::kSmem;
  if (set_func_attr((const void*)kv4_chunk_kernel<LONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SPC_ERR_CUDA;
  kv4_chunk_kernel<LONE><<<kKcCtas, KcCfg<LONE>::kThreads, smem, st>>>(qmap, a);
  if (cudaGetLastError() != cudaSuccess) return SPC_ERR_CUDA;
  const dim3 grid(kKcCtas, (a.part_rows + 31) / 32, LONE ? 1 : 2);
  return kc_launch_next(kv4_chunk_merge_kernel, grid, kKcMergeThreads, 0, st, a) ? SPC_OK : SPC_ERR_CUDA;
}

int kv4_chunk_launch(const Kv4ChunkCall& c, void* workspace, void* stream) {
  KcArgs a{};
  a.c = c;
  a.G = c.n_q / c.n_kv;
  while ((1 << a.gshift) < a.G) ++a.gshift;
  a.tpm = 128 >> a.gshift;
  a.part_rows = kc_part_rows(c.T, a.G);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.status = reinterpret_cast<int*>(w);
  a.cut = reinterpret_cast<KcItem*>(w + kKcOffCut);
  a.part = reinterpret_cast<float*>(w + kKcOffPart);
  a.wait_limit = kKcWait;
#ifdef SPC_TEST_HOOKS
  a.starve = paged_starve(&a.wait_limit) ? 1 : 0;
#endif
  CUtensorMap qmap;
  const uint64_t dims[3] = {(uint64_t)kD, (uint64_t)c.n_q, (uint64_t)c.T};
  const uint64_t strides[2] = {(uint64_t)kRowBytes, (uint64_t)c.q_stride * 2};
  const uint32_t box[3] = {64, (uint32_t)a.G, (uint32_t)a.tpm};
  if (!tensor_map_bf16_sw128(&qmap, c.q, 3, dims, strides, box)) return SPC_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // One Q tile where a request has at most a tile's rows on average. G = 4, the one
  // way and the other: 8 requests of 32K, 32 tokens (a tile) 144 and 176 us, 33
  // tokens (two) 271 and 210; one of 32K, 35 and 40, 48 and 46; 1 token 32 and 37. One
  // rule for the whole call, measured with requests that are alike: in a batch of many single
  // tokens and one long chunk either kind may take the kernel that is slower for it
  return (long long)c.T * a.G <= 128ll * c.B ? kc_launch<true>(qmap, a, st) : kc_launch<false>(qmap, a, st);
}

}  // namespace spc
