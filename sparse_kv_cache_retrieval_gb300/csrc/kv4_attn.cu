// Decode attention over the paged 4-bit cache, one query token per request.
//
// out = sum_p softmax_p(scale q.K_p) V_p over the context, or over selected
// positions, of (request, KV head) segments. Both products run on mma.sync
// (m16n8k16, fp16 operands, fp32 accumulators) with the cache rows as the
// 16-row operand and up to 8 query heads of the group as the 8 columns:
//   S^T [16 positions][8 heads] = K [16][128] Q^T [128][8]
//   O^T [128 dims][8 heads]    += V^T [128][16 positions] P^T [16][8]
// A 4-bit code times its e4m3 scale is exact in fp16, so dequantised operands
// lose nothing. The queries are scaled per head by a power of two to below 2
// and rounded to fp16 (11 bits; bf16 has 8, so only values 2^-14 below the
// head's largest lose bits, at most 2^-25 of it); maxima, sums and outputs are
// fp32. The weights P are rounded to fp16, whose range is used from its top:
// they are kept 2^14 times those against the running maximum, in the sums as
// well, so that they have 11 bits down to 2^-28 of the largest and are off by at
// most 2^-39 of it below. (Without the factor, 2^-14 and 2^-25: where a position
// with a V near zero takes nearly all the weight, 65536 small weights that the
// sum counts and the products lose are the whole result.)
//
// Layout: a record is 36 words, so 8 consecutive rows start 4 banks apart.
// The 32 positions of a step are dealt to the two 16-row tiles so that both
// the 16-byte K loads (rows 4 apart, mod 8, in a quarter warp) and the 8-byte
// V loads (rows 2 apart in a half warp) touch every bank once: tile t, row
// m = 8h + 2i + o is position 16h + 8o + ((2i + 4o) mod 8) + t.
//   K: lane (gid, tig) reads 16 bytes, values 32 tig .. 32 tig + 31 of a row;
//      the contraction index is permuted the same way in Q's fragments.
//   V: a weight's row pairs must share a register, so the nibbles of two rows
//      are interleaved (two shifts, two selects per 8 values of each) before
//      the conversion; lane (gid, tig) then holds dims 16 gid .. 16 gid + 15,
//      one scale group.
//
// The running maximum of a head is raised only when a logit passes it by more
// than 1.75 in base 2 (weights stay below 2^15.75, under fp16's largest), which
// takes the shuffles out of the common case. It is kept as a product q.K, without
// the factor to base 2: a weight is 2^((q.K - maximum) factor). The rounding of a
// large logit alone (beyond 2^25) would pass the range otherwise.
//
// Work: all segments' 32-position tiles in one line, cut into runs, one per CTA
// (k4_plan; the lengths are read on the device). Tile t of a run belongs to
// computing warp t mod W, which has a ring of its own (kStages tiles) that the
// copying warps fill; warps meet only at the end of a segment, where their
// partial (m, l, O) are merged through shared memory. A segment that several
// CTAs share leaves a partial per CTA in the workspace and the last CTA to
// finish merges them in CTA order (deterministic).
//
// What bounds it: the ALU pipe, at two conversions a cycle and SM -- 128 of the
// 290 ALU instructions a warp spends on a tile are e2m1 conversions, which
// together with 128 fp16 multiplications and 32 MMAs take a tile of 32 records
// (4.6 KB) about 200 cycles of an SM, close to its share of HBM (170). Measured:
// 8 requests of 65536 positions, 64 heads on 8 KV heads, 604 MB: 109 us, 5560
// GB/s, 0.82 of the measured copy rate (with one warp a ring copying for itself
// 123-128 us; with 8 warps of 64-position tiles 142); batch 1 of 32768, 32 heads
// on 8, 38 MB: 16 us; the same 64 segments over 4096 selected positions each, 38
// MB in rows of 144 bytes: 22 us. Below that the fixed part shows: 8 us for one
// request of 1000 positions, of which the launch, the lengths, the table entry
// and the first tile's copy, one after the other, are 4.
#include <cuda_runtime.h>

#include <atomic>

#include "kv4.cuh"
#include "kv4_attn.cuh"
#include "spc_device.cuh"
#include "spc_internal.h"

namespace spc {

constexpr int kK4Tile = 32;                          // positions a tile
constexpr uint32_t kK4StageBytes = kK4Tile * kKv4Rec;
constexpr float kK4Bias = 14.f;                      // log2 of the factor of the weights
constexpr float kK4Headroom = 1.75f;                 // log2 growth allowed before the maximum is raised
static_assert(kK4Bias + kK4Headroom <= 15.9f, "weights within fp16's range");

// The CTA of a kernel for HT head tiles; the last warps copy for the others:
// one where the whole context is read, 5 of 15 (or 2 of 8) where positions are
// gathered (64 segments of 4096: 5 for 10 that compute 21.4 us, 4 for 12 22.9, 3
// for 12 25.3).
template <int HT, bool SEL>
struct K4Cfg {
  static constexpr int kAll = HT > 1 ? 8 : SEL ? 15 : 16;      // warps
  static constexpr int kCopy = !SEL ? 1 : HT == 1 ? 5 : 2;
  static constexpr int kWarps = kAll - kCopy;          // warps that compute
  // Copying warps take the tiles in turn, and a ring's tiles have to be one
  // warp's: a wait on a stage's phase tells the phases of one parity from the
  // other, so that who waits may be one phase ahead and not two.
  static_assert(kWarps % kCopy == 0, "every ring is filled by one copying warp");
  static constexpr int kStages = HT == 1 ? 2 : 4;      // tiles in a warp's ring
  // Tiles up to which a segment is never split, and that a CTA takes at least
  // of one that is. A split costs about 2.5 us (8 segments of 10 tiles: 5.6 us
  // whole, 8.1 split); where one is made, small runs spread the work (8
  // segments of 63 tiles: 8.4 us at 8, 11.0 at 32) until the merge, which grows
  // with the heads, outweighs it (16 heads, 125 tiles: 13.5 us at 12, 17.6 at 4
  // and 13.1 at 16, but 32 tiles 11.6 at 12 and 13.1 at 16; 64 heads, 128
  // selected tiles: 22 us at 16, 31 at 4).
  static constexpr int kWhole = HT == 1 ? 24 : 16;
  static constexpr int kMinRun = HT == 1 ? 8 : HT == 2 ? 12 : 16;
  static constexpr int kSlack = 2 * kAll;              // tiles that a second piece costs a CTA, about
  static constexpr int kThreads = 32 * kAll;
  // shared memory
  static constexpr uint32_t kOffMerge = kWarps * kStages * kK4StageBytes;              // [warps][8 heads][kK4Part]
  static constexpr uint32_t kOffQ = kOffMerge + kWarps * 8 * kK4Part * 4;              // HT > 1: [HT][8 k-steps][32 lanes] x 8 bytes
  static constexpr uint32_t kOffBar = kOffQ + (HT > 1 ? HT * 8 * 32 * 8 : 0);          // [warps][stages] full, then free
  static constexpr uint32_t kOffMask = kOffBar + 2 * kWarps * kStages * 8;
  static constexpr uint32_t kSmem = kOffMask + kWarps * kStages * 4;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Whole context: the copying warp. Lane w serves warp w: tiles t0 + w, t0 + w
// + W, ... go into its ring as its stages fall free, so that one instruction
// stream computes the addresses of W tiles. A lane's table entries are fetched
// one tile ahead.
template <int W, int S>
__device__ __forceinline__ void k4_copy(const Kv4Args& a, const K4Line& ln, int segs, int t0, int t1, uint8_t* ring,
                                        uint64_t* full, uint64_t* empty, uint32_t* masks) {
  const Kv4AttnCall& c = a.c;
  const int lane = threadIdx.x & 31, bs = 1 << c.block_shift, sh = c.block_shift;
  const bool mine = lane < W;
  K4Cursor x = k4_at(c, ln, t0 + (mine ? lane : 0));
  if (!mine) x.t = t1;
  ring += lane * S * kK4StageBytes;
  full += lane * S;
  empty += lane * S;
  masks += lane * S;
  int k = 0, e0 = -1, e1 = -1;
  auto fetch = [&]() {
    if (x.t >= t1) return;
    const int p = x.i * kK4Tile;
    e0 = __ldg(x.table + (p >> sh));
    e1 = (bs < kK4Tile && p + 16 < x.len) ? __ldg(x.table + (p >> sh) + 1) : -1;
  };
  fetch();
  long long idle = clock64();
  while (__any_sync(0xffffffffu, x.t < t1)) {
    const int st = k % S;
    const bool ready = x.t < t1 && (k < S || mbar_test(&empty[st], ((k / S) & 1) ^ 1));
    if (ready) {
      const int p = x.i * kK4Tile, n = min(kK4Tile, x.len - p), g = x.s >> a.hshift;
      const bool ok0 = (unsigned)e0 < (unsigned)c.num_blocks;
      uint8_t* dst = ring + st * kK4StageBytes;
      if (bs >= kK4Tile) {
        masks[st] = ok0 ? 0xffffffffu >> (32 - n) : 0u;
        mbar_arrive_expect_tx(&full[st], ok0 ? (uint32_t)n * kKv4Rec : 0u);
        if (ok0)
          bulk_g2s(dst, c.cache + ((((size_t)e0 * c.n_kv + g) << sh) + (p & (bs - 1))) * kKv4Rec, (uint32_t)n * kKv4Rec,
                   &full[st]);
      } else {
        // two blocks of 16
        const bool ok1 = (unsigned)e1 < (unsigned)c.num_blocks;
        const int n0 = ok0 ? min(16, n) : 0, n1 = ok1 ? max(0, n - 16) : 0;
        masks[st] = ((1u << n0) - 1) | ((1u << n1) - 1) << 16;
        mbar_arrive_expect_tx(&full[st], (uint32_t)(n0 + n1) * kKv4Rec);
        if (n0 > 0)
          bulk_g2s(dst, c.cache + (((size_t)e0 * c.n_kv + g) << sh) * kKv4Rec, (uint32_t)n0 * kKv4Rec, &full[st]);
        if (n1 > 0)
          bulk_g2s(dst + 16 * kKv4Rec, c.cache + (((size_t)e1 * c.n_kv + g) << sh) * kKv4Rec, (uint32_t)n1 * kKv4Rec,
                   &full[st]);
      }
      ++k;
      k4_step(c, ln, segs, x, W);
      fetch();
    }
    if (__any_sync(0xffffffffu, ready)) {
      idle = clock64();
    } else {
      if (__any_sync(0xffffffffu, clock64() - idle > a.wait_limit)) {   // a warp gave up: stop copying
        set_status(a.status, SPC_ERR_TIMEOUT);
        break;
      }
      __nanosleep(40);
    }
  }
  // every copy lands before the CTA ends
  for (int j = max(0, k - S); j < k; ++j) mbar_wait_bounded(&full[j % S], (j / S) & 1, a.wait_limit);
  __syncwarp();
}

// Selected positions: copying warp w of N takes the run's tiles w, w + N, ...,
// one position a lane. A position is fetched four tiles ahead of its copy and
// its table entry two; the 32 records' nine 16-byte words each are dealt to
// the lanes in order, so that an instruction's copies cover whole records.
// (One cp.async.bulk of 144 bytes a record measured 70 cycles each: 74 us
// against 22 at 64 segments of 4096 positions.) Each lane arrives on the stage's
// barrier when its copies have landed, and lane 0 once the mask is written.
template <int W, int S, int N>
__device__ __forceinline__ void k4_gather(const Kv4Args& a, const K4Line& ln, int segs, int t0, int t1, int w, uint8_t* ring,
                                          uint64_t* full, uint64_t* empty, uint32_t* masks) {
  const Kv4AttnCall& c = a.c;
  const int lane = threadIdx.x & 31, sh = c.block_shift;
  constexpr int kWords = kKv4Rec / 16;
  struct Tile {
    int p, blk, len, g;
    const int32_t* table;
  };
  K4Cursor x = k4_at(c, ln, min(t0 + w, max(ln.pre[c.B] - 1, 0)));
  auto position = [&](Tile& y, int t) {             // x is at tile t
    y.p = -1;
    y.blk = -1;
    if (t >= t1) return;
    const int i = x.i * kK4Tile + lane;
    y.len = x.len;
    y.table = x.table;
    y.g = x.s >> a.hshift;
    if (i < c.budget) y.p = __ldg(c.selected + ((size_t)x.b * c.n_kv + y.g) * c.budget + i);
    k4_step(c, ln, segs, x, N);
  };
  auto lookup = [&](Tile& y) {
    if (y.p >= 0 && y.p < y.len) y.blk = __ldg(y.table + (y.p >> sh));
  };
  // word 32 k + lane of a tile: its record and its address in the cache but for the record
  int row[kWords];
  const uint8_t* word[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    row[k] = (32 * k + lane) / kWords;
    word[k] = c.cache + 16 * (32 * k + lane - kWords * row[k]);
  }
  // tiles in flight, by turns without moves (a move would wait for its load)
  Tile q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) position(q[j], t0 + w + j * N);
  lookup(q[0]);
  lookup(q[1]);
  bool dead = false;
  int wp = w, use = 0;                              // the tile is the use-th of warp wp
#pragma unroll 1
  for (int t = t0 + w; t < t1 && !dead;) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (t >= t1 || dead) break;
      lookup(q[(j + 2) & 3]);
      const int slot = wp * S + use % S;
      if (use >= S && !__all_sync(0xffffffffu, mbar_wait_bounded(&empty[slot], ((use / S) & 1) ^ 1, a.wait_limit))) {
        dead = true;
        break;
      }
      const bool ok = (unsigned)q[j].blk < (unsigned)c.num_blocks;
      const uint32_t m = __ballot_sync(0xffffffffu, ok);
      const uint32_t rec = (((uint32_t)q[j].blk * c.n_kv + q[j].g) << sh) + (q[j].p & ((1 << sh) - 1));
      uint8_t* dst = ring + (uint32_t)slot * kK4StageBytes + 16 * lane;
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        if (m == 0) break;
        const uint32_t r = __shfl_sync(0xffffffffu, rec, row[k]);
        if ((m >> row[k]) & 1u) cp_async16(dst + 512 * k, word[k] + (size_t)r * kKv4Rec, 16);
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(&full[slot])) : "memory");
      if (lane == 0) {
        masks[slot] = m;
        mbar_arrive(&full[slot]);
      }
      position(q[j], t + 4 * N);
      t += N;
      wp += N;
      if (wp >= W) {
        wp -= W;
        ++use;
      }
    }
  }
  if (dead && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
  // every copy lands before the CTA ends
  cp_async_commit();
  cp_async_wait<0>();
}

// The 32 positions of a stage: logits, weights, sums.
// FULL: every position of the step counts.
template <int HT, bool FULL>
__device__ __forceinline__ void k4_step32(const uint8_t* rows, uint32_t valid, const uint2* sq, const uint32_t (&qr)[16],
                                          const float (&f)[HT][2], float (&m)[HT][2], float (&l)[HT][2],
                                          float (&o)[HT][8][4]) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int od = gid & 1;
  const int rk = 8 * od + ((2 * (gid >> 1) + 4 * od) & 7);       // this lane's K row (+ 16, + tile)
  float s[HT][2][4];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    uint4 w[2];
    uint32_t sc[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* r = rows + (rk + 16 * h + t) * kKv4Rec;
      w[h] = *reinterpret_cast<const uint4*>(r + 16 * tig);
      const uint32_t e = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(r + kKv4Scale + 2 * tig));
      sc[h][0] = __byte_perm(e, e, 0x1010);
      sc[h][1] = __byte_perm(e, e, 0x3232);
    }
#pragma unroll
    for (int n = 0; n < HT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][t][e] = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t h0[4], h1[4];
      e2m1x8_to_f16(reinterpret_cast<const uint32_t*>(&w[0])[x], h0);
      e2m1x8_to_f16(reinterpret_cast<const uint32_t*>(&w[1])[x], h1);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t av[4] = {hmul2(h0[2 * y], sc[0][x >> 1]), hmul2(h1[2 * y], sc[1][x >> 1]),
                                hmul2(h0[2 * y + 1], sc[0][x >> 1]), hmul2(h1[2 * y + 1], sc[1][x >> 1])};
        const int j = 2 * x + y;
        if constexpr (HT == 1) {
          mma_f16(s[0][t], av, qr[2 * j], qr[2 * j + 1]);
        } else {
#pragma unroll
          for (int n = 0; n < HT; ++n) {
            const uint2 b = sq[(n * 8 + j) * 32 + lane];
            mma_f16(s[n][t], av, b.x, b.y);
          }
        }
      }
    }
  }
  uint32_t p[HT][2][2];
#pragma unroll
  for (int n = 0; n < HT; ++n) {
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!FULL && !((valid >> (rk + 16 * (e >> 1) + t)) & 1u)) s[n][t][e] = -INFINITY;
        mx[e & 1] = fmaxf(mx[e & 1], s[n][t][e]);
      }
    const bool up = (mx[0] - m[n][0]) * f[n][0] > kK4Headroom || (mx[1] - m[n][1]) * f[n][1] > kK4Headroom;
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int k = 4; k <= 16; k <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], k));
        const float M = fmaxf(m[n][e], mx[e]);
        // a first finite maximum takes 0 of what was (nothing)
        const float c = ex2_approx((m[n][e] - (M == -INFINITY ? 0.f : M)) * f[n][e]);
        m[n][e] = M;
        l[n][e] *= c;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[n][j][e] *= c;
          o[n][j][e + 2] *= c;
        }
      }
    }
    const float2 nm = make_float2(m[n][0] == -INFINITY ? 0.f : -m[n][0], m[n][1] == -INFINITY ? 0.f : -m[n][1]);
    const float2 ff = make_float2(f[n][0], f[n][1]), bias = make_float2(kK4Bias, kK4Bias);
    float2 ls = make_float2(l[n][0], l[n][1]);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float2 x = fma2(add2(make_float2(s[n][t][2 * e], s[n][t][2 * e + 1]), nm), ff, bias);
        x.x = ex2_approx(x.x);
        x.y = ex2_approx(x.y);
        ls = add2(ls, x);
        p[n][t][e] = movmatrix(pack_f16(x.x, x.y));
      }
    }
    l[n][0] = ls.x;
    l[n][1] = ls.y;
  }
  const int rv0 = 2 * tig, rv1 = 8 + ((2 * tig + 4) & 7);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    uint2 v[4];
    uint32_t b[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int row = ((h & 1) ? rv1 : rv0) + 16 * (h >> 1) + t;
      const uint8_t* r = rows + row * kKv4Rec;
      v[h] = *reinterpret_cast<const uint2*>(r + kKv4V + 8 * gid);
      b[h] = r[kKv4Scale + 8 + gid];
      // what does not count must not reach the sums: codes are always finite, a scale may be NaN
      if (!FULL && !((valid >> row) & 1u)) b[h] = 0;
    }
    const uint32_t sc0 = e4m3x2_to_f16(b[0] | b[1] << 8), sc1 = e4m3x2_to_f16(b[2] | b[3] << 8);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t ev0[4], od0[4], ev1[4], od1[4];
      const uint32_t a0 = x ? v[0].y : v[0].x, a1 = x ? v[1].y : v[1].x, a2 = x ? v[2].y : v[2].x, a3 = x ? v[3].y : v[3].x;
      constexpr uint32_t M = 0x0f0f0f0fu;
      e2m1x8_to_f16((a0 & M) | ((a1 << 4) & ~M), ev0);
      e2m1x8_to_f16(((a0 >> 4) & M) | (a1 & ~M), od0);
      e2m1x8_to_f16((a2 & M) | ((a3 << 4) & ~M), ev1);
      e2m1x8_to_f16(((a2 >> 4) & M) | (a3 & ~M), od1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t av[4] = {hmul2(ev0[i], sc0), hmul2(od0[i], sc0), hmul2(ev1[i], sc1), hmul2(od1[i], sc1)};
#pragma unroll
        for (int n = 0; n < HT; ++n) mma_f16(o[n][4 * x + i], av, p[n][t][0], p[n][t][1]);
      }
    }
  }
}

template <int HT, bool SEL>
__global__ void __launch_bounds__(K4Cfg<HT, SEL>::kThreads, 1) kv4_attn_kernel(Kv4Args a) {
  using Cfg = K4Cfg<HT, SEL>;
  constexpr int kWarps = Cfg::kWarps, kStages = Cfg::kStages;
  extern __shared__ __align__(128) uint8_t k4_smem[];
  __shared__ K4Line ln;
  __shared__ int s_last;
  const Kv4AttnCall& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int G = c.n_q / c.n_kv, segs = c.n_kv << a.hshift, heads = min(8 * HT, G);
  float* mrg = reinterpret_cast<float*>(k4_smem + Cfg::kOffMerge);
  uint2* sq = reinterpret_cast<uint2*>(k4_smem + Cfg::kOffQ);
  uint64_t* all_full = reinterpret_cast<uint64_t*>(k4_smem + Cfg::kOffBar);
  uint64_t* all_free = all_full + kWarps * kStages;
  uint32_t* all_masks = reinterpret_cast<uint32_t*>(k4_smem + Cfg::kOffMask);

  if (warp == 1) {
    for (int s = lane; s < kWarps * kStages; s += 32) {
      mbar_init(&all_full[s], SEL ? 33 : 1);
      mbar_init(&all_free[s], 1);
    }
    fence_mbar_init();
  }
  if (warp == 0) k4_plan<kK4Tile, Cfg::kWhole, Cfg::kMinRun, Cfg::kSlack>(a, ln, segs, SEL);
  __syncthreads();
  const int total = ln.pre[c.B], t0 = ln.t0, t1 = ln.t1;

  if (warp >= kWarps) {
#ifdef SPC_TEST_HOOKS
    if (a.starve) return;
#endif
    if constexpr (SEL)
      k4_gather<kWarps, kStages, Cfg::kCopy>(a, ln, segs, t0, t1, warp - kWarps, k4_smem, all_full, all_free, all_masks);
    else
      k4_copy<kWarps, kStages>(a, ln, segs, t0, t1, k4_smem, all_full, all_free, all_masks);
    return;
  }
  // the warps that compute
  auto sync = [&]() { asm volatile("bar.sync 1, %0;" :: "n"(32 * kWarps) : "memory"); };
  uint8_t* ring = k4_smem + (uint32_t)warp * kStages * kK4StageBytes;
  uint64_t* full = all_full + warp * kStages;
  uint64_t* empty = all_free + warp * kStages;
  uint32_t* masks = all_masks + warp * kStages;

  bool dead = false;
  int n_wait = 0;                                    // tiles this warp has waited for

  // requests without a tile: zeros
  for (int b = ln.empty ? 0 : c.B; b < c.B; ++b) {
    if (ln.nt[b] != 0) continue;
    uint4* dst = reinterpret_cast<uint4*>(c.out + (size_t)b * c.n_q * kD);
    for (int i = blockIdx.x * 32 * kWarps + threadIdx.x; i < c.n_q * kD / 8; i += gridDim.x * 32 * kWarps)
      dst[i] = make_uint4(0u, 0u, 0u, 0u);
  }

  K4Cursor pc = k4_at(c, ln, min(t0, max(total - 1, 0)));   // the piece at hand
  for (int pt = t0; pt < t1;) {
    const int b = pc.b, sg = pc.s, nt = pc.nt;
    const int pe = min(t1, pt + nt - pc.i);          // end of this CTA's piece of the segment
    const int g = sg >> a.hshift, hh = sg - (g << a.hshift);
    const int h0 = g * G + hh * 8 * HT;              // first query head
    // ---- queries: per head a power of two that brings the largest value below 2
    uint32_t qr[16];
    float f[HT][2];
#pragma unroll
    for (int n = 0; n < HT; ++n) {
      const int h = 8 * n + gid;
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = h < heads ? __ldg(reinterpret_cast<const uint4*>(c.q + ((size_t)b * c.n_q + h0 + h) * kD + 32 * tig) + i)
                         : make_uint4(0u, 0u, 0u, 0u);
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu),
                                   __vmaxu2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu)));
      mx = max(mx & 0xffffu, mx >> 16);
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // exponent of the largest value; 2^e as two factors, each normal (2^-e may be subnormal, and is exact)
      const int e = max((int)(mx >> 7), 1) - 127;
      const int e1 = e / 2, e2 = e - e1;
      const float down = __uint_as_float((uint32_t)(127 - e1) << 23) * __uint_as_float((uint32_t)(127 - e2) << 23);
      const float u1 = __uint_as_float((uint32_t)(127 + e1) << 23), u2 = __uint_as_float((uint32_t)(127 + e2) << 23);
      const float fh = k4_factor(c.scale2 * u1 * u2);           // of head 8 n + gid
      f[n][0] = __shfl_sync(0xffffffffu, fh, 8 * tig);
      f[n][1] = __shfl_sync(0xffffffffu, fh, 8 * tig + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[8];
        unpack8(w[i], x);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t b0 = pack_f16(x[4 * y] * down, x[4 * y + 1] * down);
          const uint32_t b1 = pack_f16(x[4 * y + 2] * down, x[4 * y + 3] * down);
          if constexpr (HT == 1) {
            qr[4 * i + 2 * y] = b0;
            qr[4 * i + 2 * y + 1] = b1;
          } else if (warp == 0) {
            sq[(n * 8 + 2 * i + y) * 32 + lane] = make_uint2(b0, b1);
          }
        }
      }
    }
    if constexpr (HT > 1) sync();

    float m[HT][2], l[HT][2], o[HT][8][4];
#pragma unroll
    for (int n = 0; n < HT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][j][e] = 0.f;
    }
    // this warp's tiles of the piece
    const int k0 = (pt - t0 + kWarps - 1 - warp) / kWarps;
#pragma unroll 1
    for (int t = t0 + warp + k0 * kWarps; t < pe; t += kWarps) {
      const int st = n_wait % kStages;
      if (!dead && !mbar_wait_bounded(&full[st], (n_wait / kStages) & 1, a.wait_limit)) {
        set_status(a.status, SPC_ERR_TIMEOUT);
        dead = true;
      }
      dead = __any_sync(0xffffffffu, dead);
      if (dead) continue;                            // the other warps' barriers are still reached
      ++n_wait;
      const uint8_t* rows = ring + st * kK4StageBytes;
      const uint32_t valid = masks[st];
      if (valid == 0xffffffffu)
        k4_step32<HT, true>(rows, valid, sq, qr, f, m, l, o);
      else if (valid != 0)
        k4_step32<HT, false>(rows, valid, sq, qr, f, m, l, o);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---- merge of the warps' partials, 8 heads at a time
    const int seg = b * segs + sg;
    const int s0 = pt - pc.i, s1 = s0 + nt;          // the segment's tiles in the line
    // CTAs that have a piece of it
    const int run = ln.run, ends = run == 1 << 30;
    const int w0 = ends ? ln.first : s0 / run, w1 = ends ? ln.last : (s1 - 1) / run;
    const bool whole = w0 == w1;
    float* res = a.part + ((size_t)blockIdx.x * 2 + (!ends && s0 > t0 ? 1 : 0)) * (size_t)(8 * HT) * kK4Part;
#pragma unroll 1
    for (int n = 0; n < HT; ++n) {
      float mm[2], ll[2], ff[2];
      float* dst = mrg + (size_t)(warp * 8 + 2 * tig) * kK4Part;
#pragma unroll
      for (int k = 0; k < HT; ++k) {
        if (k != n) continue;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mm[e] = m[k][e];
          ll[e] = l[k][e];
          ff[e] = f[k][e];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            *reinterpret_cast<float4*>(dst + e * kK4Part + 4 + 16 * gid + 4 * y) =
                make_float4(o[k][2 * y][e], o[k][2 * y][e + 2], o[k][2 * y + 1][e], o[k][2 * y + 1][e + 2]);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int k = 4; k <= 16; k <<= 1) ll[e] += __shfl_xor_sync(0xffffffffu, ll[e], k);
        if (gid == 0) {
          dst[e * kK4Part] = mm[e];
          dst[e * kK4Part + 1] = ll[e];
          dst[e * kK4Part + 2] = ff[e];
        }
      }
      sync();
#pragma unroll 1
      for (int e = warp; e < 8; e += kWarps) {       // head e of the eight
        const int h = 8 * n + e;
        if (h >= heads) break;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mrg[(w * 8 + e) * kK4Part]);
        const float Ms = M == -INFINITY ? 0.f : M, fh = mrg[e * kK4Part + 2];
        float L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* src = mrg + (size_t)(w * 8 + e) * kK4Part;
          const float wt = ex2_approx((src[0] - Ms) * fh);
          const float4 x = *reinterpret_cast<const float4*>(src + 4 + 4 * lane);
          L += wt * src[1];
          v.x += wt * x.x; v.y += wt * x.y; v.z += wt * x.z; v.w += wt * x.w;
        }
        if (whole) {
          const float r = L == 0.f ? 0.f : 1.f / L;
          *reinterpret_cast<uint2*>(c.out + ((size_t)b * c.n_q + h0 + h) * kD + 4 * lane) =
              make_uint2(pack_bf16(v.x * r, v.y * r), pack_bf16(v.z * r, v.w * r));
        } else {
          float* p = res + (size_t)h * kK4Part;
          if (lane == 0) *reinterpret_cast<float4*>(p) = make_float4(M, L, fh, 0.f);
          *reinterpret_cast<float4*>(p + 4 + 4 * lane) = v;
        }
      }
      sync();
    }
    if (!whole) {
      __threadfence();
      sync();
      if (threadIdx.x == 0) s_last = atomicAdd(&a.counters[seg], 1u) == (uint32_t)(w1 - w0);
      sync();
      if (s_last) {
        __threadfence();
        k4_merge<HT, kWarps, kWarps * 8 * kK4Part * 4>(a, K4Open{seg, b, h0, s0, w0, w1, run}, heads, mrg);
      }
    }
    k4_step(c, ln, segs, pc, pe - pt);
    pt = pe;
  }
}

#ifdef SPC_TEST_HOOKS
static std::atomic<int> g_starve_calls{0};
static std::atomic<long long> g_starve_wait{0};
bool paged_starve(long long* wait_limit) {
  int n = g_starve_calls.load();
  while (n > 0 && !g_starve_calls.compare_exchange_weak(n, n - 1)) {
  }
  if (n > 0) *wait_limit = g_starve_wait.load();
  return n > 0;
}
#endif

// The whole context of groups of 32 and 64 heads goes to the tcgen05 kernel. Both
// sides measured for 32 and 64 heads on 1, 4 and 8 KV heads, 1 to 64 requests of 16
// to 65536 positions, equal and ragged: it is 1.17 to 3.8 times as fast in all 60
// (us there and here: 64 heads on one, 8 x 65536 47 and 88, 1 x 2000 11 and 22, 64 of
// 1-2000 21 and 63; 32 on one, 39 and 60, 9 and 22, 17 and 25; 32 on each of 8, 8 x
// 65536 235 and 276, 32 of 16-200 12 and 21). 16 heads, 8 x 65536: 35 and 35 on one
// KV head, 108 and 88 on four. Selected positions stay here.
static bool k4_on_tc(int G, int budget) { return G >= 32 && budget == 0; }
// head tiles a segment, and log2 of the segments a group is split into
static int k4_head_tiles(int G, int budget) { return k4_on_tc(G, budget) ? G / 8 : G <= 8 ? 1 : G == 16 ? 2 : 4; }
static int k4_split(int G, int budget) { return !k4_on_tc(G, budget) && G > 32 ? 1 : 0; }

size_t kv4_attn_workspace(int, int n_q, int n_kv, int, int, int budget) {
  return kK4OffPart + (size_t)kK4Ctas * 2 * 8 * k4_head_tiles(n_q / n_kv, budget) * kK4Part * 4;
}

template <int HT, bool SEL>
static int k4_run(const Kv4Args& a, void* stream) {
  cudaError_t e = set_func_attr((const void*)kv4_attn_kernel<HT, SEL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)K4Cfg<HT, SEL>::kSmem);
  if (e != cudaSuccess) return SPC_ERR_CUDA;
  kv4_attn_kernel<HT, SEL><<<kK4Ctas, K4Cfg<HT, SEL>::kThreads, K4Cfg<HT, SEL>::kSmem, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

int kv4_attn_max_kv() { return kK4MaxKv; }

int kv4_attn_launch(const Kv4AttnCall& c, void* workspace, void* stream) {
  const int G = c.n_q / c.n_kv;
  Kv4Args a{};
  a.c = c;
  a.ht = k4_head_tiles(G, c.budget);
  a.hshift = k4_split(G, c.budget);
  a.wait_limit = kK4WaitLimit;
#ifdef SPC_TEST_HOOKS
  a.starve = paged_starve(&a.wait_limit) ? 1 : 0;
#endif
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.status = reinterpret_cast<int*>(ws);
  a.counters = reinterpret_cast<uint32_t*>(ws + kK4OffCount);
  a.segments = ws + kK4OffSeg;
  a.part = reinterpret_cast<float*>(ws + kK4OffPart);
  if (k4_on_tc(G, c.budget)) return kv4_attn_tc_launch(a, G, stream);
  if (!c.selected) return a.ht == 1 ? k4_run<1, false>(a, stream) : k4_run<2, false>(a, stream);
  switch (a.ht) {
    case 1: return k4_run<1, true>(a, stream);
    case 2: return k4_run<2, true>(a, stream);
    default: return k4_run<4, true>(a, stream);
  }
}

}  // namespace spc

#ifdef SPC_TEST_HOOKS
// Test builds only: the next `calls` launches of the 4-bit decode attention or
// the prompt attention issue no copies and give up waiting after `wait_cycles`
// clock cycles.
extern "C" int spc_test_starve_paged(int calls, long long wait_cycles) {
  if (calls < 0 || wait_cycles < 1) return SPC_ERR_INVALID_ARG;
  spc::g_starve_wait.store(wait_cycles);
  spc::g_starve_calls.store(calls);
  return SPC_OK;
}
#endif
