// Decode attention over the paged 4-bit cache for groups of 32 or 64 query
// heads, whole context, on the 5th-generation tensor cores.
//
// With N heads a record feeds 512 N flops; from 32 heads on the mma.sync
// kernel is bound by the reuse of its dequantised operands (8 heads an
// instruction) and by few, register-heavy warps. Here a tile of 128 positions is
// dequantised once, for all heads, and both products are transposed, with the
// positions in the tensor memory lanes:
//   S^T [128 positions][N heads] = K [128][128] Q^T     K in tensor memory
//   O^T [128 dims][N heads]     += V^T [128][128] P^T   V, P in shared memory
// A position is one thread's throughout: it dequantises the K row into its own
// tensor memory lane (no transpose, no swizzle) and the V row into one row of
// an MN-major operand; the softmax thread of the position has its logits of
// all heads and writes one row of P. So nothing is exchanged between positions
// but the heads' maxima (as products q.K, see kv4_attn.cu), and those only when a
// logit passes the running one by more than 4.75 (a barrier's OR tells), and the
// sums, once a segment.
// Operands are fp16: K and V exact, Q scaled per head by a power of two and P
// rounded; logits, maxima, sums and O are fp32. P and the sums are kept 2^11
// times the weights against the running maximum, the top of fp16's range (see
// kv4_attn.cu): 11 bits down to 2^-25 of the largest, off by at most 2^-36 of it
// below. A raise costs about a tile here, which is why more of the range is left
// to growth than there (8 x 65536, 64 heads on one: 46.5 us with a factor of 2^10,
// 46.7 with 2^11, 48.7 with 2^12).
//
// One CTA per SM, 16 warps:
//   0-3    softmax and epilogue (one position, in the epilogue one dim, a thread)
//   4-11   dequantisation, two groups of four that take the tiles by turns
//   12     tensor memory, MMA issue: S(t + 1) ahead of PV(t)
//   13     copies (cp.async.bulk, one a cache block), six tiles ahead
// Bound: a tile is 1.26 us at N = 64 and 1.02 at N = 32 (from 8 requests of 32768
// and of 131072 positions), of which its 18 KB are 0.41 us of an SM's share of HBM.
// No unit is busy (tensor pipe 24%, ALU 26%): without the softmax's arithmetic it
// is 0.99 and 0.82 us, without the conversions 1.21 and 0.97, without both 0.97
// and 0.78. What is left is the chain of a tile, of which two are in flight: V
// dequantised when the PV two tiles back has read its buffer, S, softmax, PV, a
// barrier between each two. Beside its tiles a call has 13 us (N = 32: 11): launch,
// plan, first tile, and 6 for the merge kernel; one request over 128 CTAs has
// more in the merge (20 us) than here (14).
// Measured (8 requests of 65536 positions on one KV head, 27 tiles a CTA, 75 MB,
// floor 11 us): N = 64 46.7 us, N = 32 38.6 us; the mma.sync kernel 88 and 60.
// Every wait is bounded; a warp whose wait gives up records SPC_ERR_TIMEOUT and
// runs on without waiting, so that the softmax warps' barriers are reached.
#include <cuda_runtime.h>

#include "kv4_attn.cuh"
#include "spc_tc.cuh"

namespace spc {

constexpr int kKtTile = 128;                          // positions
constexpr uint32_t kKtRaw = kKtTile * kKv4Rec;        // 18 KB: a tile's records
constexpr int kKtStages = 6;
static_assert(kKtStages % 2 == 0, "every stage is read by one of the two dequantising groups");
constexpr int kKtMasks = 16;                          // tiles whose masks are kept
constexpr float kKtBias = 11.f;                       // log2 of the factor of the weights
constexpr float kKtHeadroom = 4.75f;                  // log2 growth allowed before a maximum is raised
static_assert(kKtBias + kKtHeadroom <= 15.9f, "weights within fp16's range");
// See k4_plan. A tile is 1.0 to 1.3 us of the CTA that has it, the merge some 4 us
// and a little a piece: 64 heads on one, 1 x 2000: 10.6 us with these, 17.9 with
// 8 and 8; 1 x 65536 26.4 and 24.8.
constexpr int kKtWhole = 4, kKtMinRun = 2, kKtSlack = 8;
constexpr uint32_t kKtV = kKtTile * kRowBytes;        // 32 KB: V of a tile, fp16
constexpr uint32_t kKtP = kKtTile * 128;              // 16 KB: P, 64 heads a row
constexpr int kKtWarpMma = 12, kKtWarpCopy = 13;
constexpr int kKtThreads = 512;
// registers a thread: 128 at launch (512 threads); softmax 200, dequantisation
// 112 (two warpgroups), the rest 88: 200 + 2 * 112 + 88 = 4 * 128
constexpr int kKtRegSoft = 200, kKtRegDeq = 112, kKtRegRest = 88;
constexpr uint32_t kKtColS = 128, kKtColO = 256;      // K in columns 0-63 and 64-127, S in 128.. and 192..

// shared memory, from a 1024-byte aligned base
constexpr uint32_t kKtOffV = 0;                                      // [2]
constexpr uint32_t kKtOffP = kKtOffV + 2 * kKtV;                     // [2]
constexpr uint32_t kKtOffQ = kKtOffP + 2 * kKtP;                     // [2 halves of 64 dims][N][128 bytes]
constexpr uint32_t kKtOffRaw = kKtOffQ + 64 * kRowBytes;             // [kKtStages]
constexpr uint32_t kKtOffMf = kKtOffRaw + kKtStages * kKtRaw;        // [32 pairs of heads] float4: logit factors, -maxima
constexpr uint32_t kKtOffM = kKtOffMf + 64 * 8;                      // [64] running maxima
constexpr uint32_t kKtOffAl = kKtOffM + 64 * 4;                      // [64] rescale factors; 1 / sums
constexpr uint32_t kKtOffRed = kKtOffAl + 64 * 4;                    // [4 warps][64]
constexpr uint32_t kKtOffMask = kKtOffRed + 4 * 64 * 4;              // [kKtMasks][4 words]
constexpr uint32_t kKtOffBar = kKtOffMask + kKtMasks * 16;
constexpr int kKtBars = 2 * kKtStages + 2 * 5 + 4;
constexpr size_t kKtSmem = 1024 + kKtOffBar + kKtBars * 8 + 16;

// a segment's partials: its first CTA, their number (0: none), its first tile
// and the tiles a run (2^30: runs end with their segments)
struct KtSegment {
  int w0, np, s0, run;
};
static_assert(sizeof(KtSegment) * SPC_MAX_BATCH * kK4MaxKv <= kK4OffPart - kK4OffSeg, "one entry a segment in the workspace");

template <int N>
constexpr uint32_t kKtIdescS = (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kKtTile >> 4) << 24);
template <int N>
constexpr uint32_t kKtIdescO = kKtIdescS<N> | (1u << 15) | (1u << 16);         // both operands MN-major

// barrier of the four softmax warps, plain and with the OR of a predicate
__device__ __forceinline__ void kt_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool kt_any(bool x) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, 1, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r) : "r"((uint32_t)x) : "memory");
  return r != 0;
}
// N (32 or 64) consecutive fp32 columns of this thread's lane
template <int N>
__device__ __forceinline__ void kt_ld(uint32_t t, float (&v)[N]) {
#pragma unroll
  for (int q = 0; q < N; q += 32) tmem_ld32(t + q, *reinterpret_cast<float (*)[32]>(v + q));
  tmem_ld_wait();
}

// v[h] over the warp's lanes reduced for all N (32 or 64) heads at once, halving
// the heads a lane keeps at each step; the result of head h goes to red[h]
template <int N, class F>
__device__ __forceinline__ void kt_reduce(float (&v)[N], float* red, F f) {
  const int lane = threadIdx.x & 31;
  int h = 0;                                          // first head this lane keeps
#pragma unroll
  for (int s = 0; s < 5; ++s) {
    const int x = 16 >> s, keep = N >> (s + 1);       // lanes apart, heads kept
    const bool up = (lane & x) != 0;
#pragma unroll
    for (int j = 0; j < keep; ++j) {
      const float send = up ? v[j] : v[j + keep], mine = up ? v[j + keep] : v[j];
      v[j] = f(mine, __shfl_xor_sync(0xffffffffu, send, x));
    }
    h += up ? keep : 0;
  }
#pragma unroll
  for (int j = 0; j < N / 32; ++j) red[h + j] = v[j];
}

// 32 codes (four words of 8) times their two scales, as fp16 pairs (exact)
__device__ __forceinline__ void kt_dequant32(const uint4& w, uint32_t scales, uint32_t (&h)[16]) {
  const uint32_t s = e4m3x2_to_f16(scales);
  const uint32_t s0 = __byte_perm(s, s, 0x1010), s1 = __byte_perm(s, s, 0x3232);
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t t[4];
    e2m1x8_to_f16(x[i], t);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[4 * i + j] = hmul2(t[j], i < 2 ? s0 : s1);
  }
}

template <int N>
__global__ void __launch_bounds__(kKtThreads, 1) kv4_attn_tc_kernel(Kv4Args a, KtSegment* segments) {
  extern __shared__ uint8_t kt_raw[];
  __shared__ K4Line ln;
  uint8_t* base = kt_raw + (((smem_u32(kt_raw) + 1023u) & ~1023u) - smem_u32(kt_raw));
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(base + kKtOffBar);   // [kKtStages] copy bytes
  uint64_t* raw_free = raw_full + kKtStages;          // [kKtStages] 4 dequantising warps have read the stage
  uint64_t* kv_full = raw_free + kKtStages;           // [2] 4 warps: K and V of a tile dequantised
  uint64_t* s_full = kv_full + 2;                     // [2] commit: S in tensor memory; its K buffer is free
  uint64_t* s_free = s_full + 2;                      // [2] 4 softmax warps have read S
  uint64_t* p_full = s_free + 2;                      // [2] 4 softmax warps: P written, O rescaled
  uint64_t* pv_done = p_full + 2;                     // [2] commit: PV done; its V and P buffers are free
  uint64_t* q_full = pv_done + 2;                     // 4 softmax warps: a segment's queries written
  uint64_t* drain = q_full + 1;                       // commit after the last MMA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  uint32_t* masks = reinterpret_cast<uint32_t*>(base + kKtOffMask);
  const Kv4AttnCall& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, segs = c.n_kv;

  if (warp == 1 && lane == 0) {
    for (int s = 0; s < kKtStages; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_free[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&kv_full[s], 4);
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], 4);
      mbar_init(&p_full[s], 4);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(q_full, 4);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 0) k4_plan<kKtTile, kKtWhole, kKtMinRun, kKtSlack>(a, ln, segs, false);
  if (warp == kKtWarpMma) tmem_alloc<512>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int t0 = ln.t0, t1 = ln.t1, nt_run = t1 - t0;
  bool dead = false;
  auto acquire = [&](uint64_t* bar, uint32_t parity) {
    if (!dead && !__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.wait_limit))) {
      if (lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
      dead = true;
    }
  };

  if (warp == kKtWarpCopy) {
    // ================= copies. Lane u < 8 sees to rows 16u .. 16u + 15 of a tile
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kKtRegRest));
    const int sh = c.block_shift, bs = 1 << sh, span = min(bs, kKtTile), r0 = 16 * lane;
    K4Cursor x = k4_at(c, ln, min(t0, max(ln.pre[c.B] - 1, 0)));
    auto entry = [&]() {
      const int p = x.i * kKtTile + r0;
      return lane < 8 && x.t < t1 && p < x.len ? __ldg(x.table + (p >> sh)) : -1;
    };
    int e = entry(), i = 0;
    bool starve = false;
#ifdef SPC_TEST_HOOKS
    starve = a.starve != 0;
#endif
#pragma unroll 1
    for (; i < nt_run && !starve; ++i) {
      const int st = i % kKtStages, p = x.i * kKtTile + r0, n = x.len - x.i * kKtTile;     // n: rows left of the context
      const bool ok = (unsigned)e < (unsigned)c.num_blocks;
      const int rows = ok && lane < 8 ? max(0, min(16, n - r0)) : 0;
      const uint8_t* src = c.cache + ((((size_t)(ok ? e : 0) * c.n_kv + x.s) << sh) + (p & (bs - 1))) * kKv4Rec;
      k4_step(c, ln, segs, x, 1);
      e = entry();
      acquire(&raw_free[st], ((i / kKtStages) & 1) ^ 1);
      if (dead) break;
      const uint32_t bits = (1u << rows) - 1, hi = __shfl_down_sync(0xffffffffu, bits, 1);
      if (lane < 8 && !(lane & 1)) masks[i % kKtMasks * 4 + (lane >> 1)] = bits | hi << 16;
      __syncwarp();                                   // lane 0's arrival releases the four lanes' masks
      const uint32_t bytes = __reduce_add_sync(0xffffffffu, (unsigned)rows) * kKv4Rec;
      if (lane == 0) mbar_arrive_expect_tx(&raw_full[st], bytes);
      __syncwarp();
      if (rows > 0 && (r0 & (span - 1)) == 0)
        bulk_g2s(base + kKtOffRaw + (uint32_t)st * kKtRaw + (uint32_t)r0 * kKv4Rec, src, (uint32_t)min(span, n - r0) * kKv4Rec,
                 &raw_full[st]);
      __syncwarp();
    }
    // every copy lands before the CTA ends
    for (int k = max(0, i - kKtStages); k < i; ++k)
      mbar_wait_bounded(&raw_full[k % kKtStages], (k / kKtStages) & 1, a.wait_limit);
    __syncwarp();
  } else if (warp == kKtWarpMma) {
    // ================= MMA issue, warp-uniform, by one elected lane
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kKtRegRest));
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), sm = smem_u32(base);
    constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);             // descriptors' high word (spc_tc.cuh)
    auto desc = [&](uint32_t addr, uint32_t lead) { return (uint64_t)hi << 32 | (addr >> 4) | (lead >> 4) << 16; };
    auto issue_s = [&](int i) {
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk)
          umma_f16_tmem_a(tm + kKtColS + (i & 1) * 64, tm + (i & 1) * 64 + kk * 8,
                          desc(sm + kKtOffQ + (uint32_t)(kk >> 2) * (N * 128) + (uint32_t)(kk & 3) * 32, 16), kKtIdescS<N>,
                          kk ? 1u : 0u);
        umma_commit(&s_full[i & 1]);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int i, bool first) {
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kKtTile / 16; ++kk)
          umma_f16(tm + kKtColO, desc(sm + kKtOffV + (uint32_t)(i & 1) * kKtV + (uint32_t)kk * 2048, kKtV / 2),
                   desc(sm + kKtOffP + (uint32_t)(i & 1) * kKtP + (uint32_t)kk * 2048, 16), kKtIdescO<N>,
                   (first && kk == 0) ? 0u : 1u);
        umma_commit(&pv_done[i & 1]);
      }
      __syncwarp();
    };
    // S up to two tiles ahead of PV, whichever has its operands; the first S
    // of a segment waits for its queries, which are written when the segment
    // before is done
    if (nt_run > 0) {
      K4Cursor x = k4_at(c, ln, t0);
      int is = 0, ip = 0, nq = 0;                     // next S, next PV
      int end = min(nt_run, x.nt - x.i);              // of the segment that S is at
      int begin = 0, pv_end = end, pv_begin = 0;      // and the one that PV is at
      long long idle = clock64();
      while (ip < nt_run) {
        bool s_ok = is < nt_run && is < ip + 2 && mbar_test(&kv_full[is & 1], (is >> 1) & 1) &&
                    mbar_test(&s_free[is & 1], ((is >> 1) & 1) ^ 1) && (is != begin || mbar_test(q_full, nq & 1));
        s_ok = __all_sync(0xffffffffu, s_ok);
        if (s_ok) {
          if (is == begin) ++nq;
          issue_s(is);
          if (++is == end && is < nt_run) {
            k4_step(c, ln, segs, x, end - begin);
            begin = end;
            end = min(nt_run, begin + x.nt);
          }
          idle = clock64();
          continue;
        }
        if (__all_sync(0xffffffffu, ip < is && mbar_test(&p_full[ip & 1], (ip >> 1) & 1))) {
          issue_pv(ip, ip == pv_begin);
          if (++ip == pv_end) {
            pv_begin = pv_end;
            pv_end = end;                             // S is in the next segment by now, or at its start
          }
          idle = clock64();
          continue;
        }
        if (__any_sync(0xffffffffu, clock64() - idle > a.wait_limit)) {
          if (lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
          break;
        }
      }
    }
    // every MMA has completed before tensor memory is released
    if (elect_one()) umma_commit(drain);
    __syncwarp();
    mbar_wait_bounded(drain, 0, a.wait_limit);
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ================= dequantisation of every other tile, one position a thread
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kKtRegDeq));
    const int grp = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
#pragma unroll 1
    for (int i = grp; i < nt_run; i += 2) {
      const int st = i % kKtStages, u = i >> 1;
      acquire(&raw_full[st], (i / kKtStages) & 1);
      const uint8_t* rec = base + kKtOffRaw + (uint32_t)st * kKtRaw + (uint32_t)row * kKv4Rec;
      const bool valid = !dead && ((masks[i % kKtMasks * 4 + (warp & 3)] >> lane) & 1u);
      uint4 w[4];
      uint2 sc;
      auto load = [&](int off, int soff) {
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = *reinterpret_cast<const uint4*>(rec + off + 16 * q);
        sc = *reinterpret_cast<const uint2*>(rec + kKv4Scale + soff);
        if (!valid) {                                 // what does not count is zero, whatever it was
#pragma unroll
          for (int q = 0; q < 4; ++q) w[q] = make_uint4(0u, 0u, 0u, 0u);
          sc = make_uint2(0u, 0u);
        }
      };
      load(0, 0);
      // K: S of tile i - 2 has read this buffer
      if (u > 0) acquire(&s_full[grp], (u - 1) & 1);
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t h[16];
        kt_dequant32(w[q], (q < 2 ? sc.x : sc.y) >> (16 * (q & 1)), h);
        if (!dead) tmem_st16(tmem + lanes + grp * 64 + 16 * q, h);
      }
      load(kKv4V, 8);
      __syncwarp();
      if (lane == 0) mbar_arrive(&raw_free[st]);
      // V: PV of tile i - 2 has read this buffer
      if (u > 0) acquire(&pv_done[grp], (u - 1) & 1);
      const uint32_t vb = smem_u32(base) + kKtOffV + (uint32_t)grp * kKtV + (uint32_t)row * 128;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t h[16];
        kt_dequant32(w[q], (q < 2 ? sc.x : sc.y) >> (16 * (q & 1)), h);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int un = 4 * q + j;                   // 16-byte unit: dims 8 un .. 8 un + 7
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                       :: "r"(vb + (uint32_t)(un >> 3) * (kKtV / 2) + (uint32_t)(((un & 7) ^ (row & 7)) << 4)), "r"(h[4 * j]),
                          "r"(h[4 * j + 1]), "r"(h[4 * j + 2]), "r"(h[4 * j + 3]) : "memory");
        }
      }
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kv_full[grp]);
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kKtRegRest));
  } else {
    // ================= softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kKtRegSoft));
    const int row = threadIdx.x;                      // position of a tile; dim in the epilogue
    const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
    float* mf = reinterpret_cast<float*>(base + kKtOffMf);
    auto mf_at = [](int h) { return (h >> 1) * 4 + (h & 1); };      // of head h's factor; its -maximum is 2 behind
    float* mrun = reinterpret_cast<float*>(base + kKtOffM);
    float* al = reinterpret_cast<float*>(base + kKtOffAl);
    float* red = reinterpret_cast<float*>(base + kKtOffRed);
    // requests without a tile: zeros
    for (int b = ln.empty ? 0 : c.B; b < c.B; ++b) {
      if (ln.nt[b] != 0) continue;
      uint4* dst = reinterpret_cast<uint4*>(c.out + (size_t)b * c.n_q * kD);
      for (int i = blockIdx.x * 128 + row; i < c.n_q * kD / 8; i += gridDim.x * 128) dst[i] = make_uint4(0u, 0u, 0u, 0u);
      for (int i = blockIdx.x * 128 + row; i < segs; i += gridDim.x * 128) segments[b * segs + i] = KtSegment{0, 0, 0, 0};
    }
    K4Cursor pc = k4_at(c, ln, min(t0, max(ln.pre[c.B] - 1, 0)));
    int i = 0;
    while (i < nt_run) {
      const int b = pc.b, g = pc.s, nt = pc.nt, pt = t0 + i, i1 = min(nt_run, i + nt - pc.i), h0 = g * N;
      // ---- queries: per head a power of two that brings the largest value
      // below 2; four dims a lane, one head a warp at a time
      uint2 qw[N / 4];
#pragma unroll
      for (int k = 0; k < N / 4; ++k)
        qw[k] = __ldg(reinterpret_cast<const uint2*>(c.q + ((size_t)b * c.n_q + h0 + warp + 4 * k) * kD) + lane);
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        const int h = warp + 4 * k;
        const uint2 w = qw[k];
        uint32_t mx = __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
        mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
        const int e = max((int)(mx >> 7), 1) - 127, e1 = e / 2, e2 = e - e1;
        const float d1 = __uint_as_float((uint32_t)(127 - e1) << 23), d2 = __uint_as_float((uint32_t)(127 - e2) << 23);
        const uint32_t dst = smem_u32(base) + kKtOffQ + (uint32_t)(lane >> 4) * (N * 128) + (uint32_t)h * 128 +
                             (uint32_t)((((lane & 15) >> 1) ^ (h & 7)) << 4) + (uint32_t)(lane & 1) * 8;
        asm volatile("st.shared.v2.b32 [%0], {%1,%2};"
                     :: "r"(dst), "r"(pack_f16(bf_lo(w.x) * d1 * d2, bf_hi(w.x) * d1 * d2)),
                        "r"(pack_f16(bf_lo(w.y) * d1 * d2, bf_hi(w.y) * d1 * d2)) : "memory");
        if (lane == 0) {
          const float u1 = __uint_as_float((uint32_t)(127 + e1) << 23), u2 = __uint_as_float((uint32_t)(127 + e2) << 23);
          mf[mf_at(h)] = k4_factor(c.scale2 * u1 * u2);
          mf[mf_at(h) + 2] = 0.f;
          mrun[h] = -INFINITY;
        }
      }
      fence_proxy_async_smem();
      kt_sync();
      if (lane == 0) mbar_arrive(q_full);

      float l[N];
#pragma unroll
      for (int h = 0; h < N; ++h) l[h] = 0.f;
      bool first = true, none = true;                 // of the piece; no position counted yet
#pragma unroll 1
      for (; i < i1; ++i) {
        const int u = i >> 1, bf = i & 1;
        float s[N];
        acquire(&s_full[bf], u & 1);
        tc_fence_after();
        const uint4 mk = *reinterpret_cast<const uint4*>(masks + i % kKtMasks * 4);
        const uint32_t word = warp == 0 ? mk.x : warp == 1 ? mk.y : warp == 2 ? mk.z : mk.w;
        const bool some = (mk.x | mk.y | mk.z | mk.w) != 0;
        auto load = [&]() {
          if (!dead) kt_ld<N>(tl + kKtColS + bf * 64, s);
          if (dead || word != 0xffffffffu) {
#pragma unroll
            for (int h = 0; h < N; ++h) s[h] = !dead && ((word >> lane) & 1u) ? s[h] : -INFINITY;
          }
        };
        load();
        // P of tile i - 2 has been read
        if (u > 0) acquire(&pv_done[bf], (u - 1) & 1);
        // s becomes the weights against the maxima at hand, and P; returns the
        // largest exponent of a weight
        const uint32_t pb = smem_u32(base) + kKtOffP + (uint32_t)bf * kKtP + (uint32_t)row * 128;
        auto weights = [&]() {
          float mx = -INFINITY;
#pragma unroll
          for (int n = 0; n < N / 8; ++n) {
            uint32_t p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int h = 8 * n + 2 * j;
              const float4 k = *reinterpret_cast<const float4*>(mf + 2 * h);
              const float2 x = fma2(add2(make_float2(s[h], s[h + 1]), make_float2(k.z, k.w)), make_float2(k.x, k.y),
                                    make_float2(kKtBias, kKtBias));
              mx = fmaxf(mx, fmaxf(x.x, x.y));
              s[h] = ex2_approx(x.x);
              s[h + 1] = ex2_approx(x.y);
              p[j] = pack_f16(s[h], s[h + 1]);
            }
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" :: "r"(pb + (uint32_t)((n ^ (row & 7)) << 4)), "r"(p[0]),
                         "r"(p[1]), "r"(p[2]), "r"(p[3]) : "memory");
          }
          return mx;
        };
        const bool start = none && some;              // the first that counts: no maximum to try
        if (start || kt_any(weights() > kKtBias + kKtHeadroom)) {
          // a maximum to raise: every head's over the tile, 32 heads at a time
          if (!start) load();
#pragma unroll
          for (int hb = 0; hb < N; hb += 32) {
            float v[32];
#pragma unroll
            for (int h = 0; h < 32; ++h) v[h] = s[hb + h];
            kt_reduce<32>(v, red + warp * 64 + hb, [](float x, float y) { return fmaxf(x, y); });
          }
          kt_sync();
          if (row < N) {
            // (finite from the first position that counts on)
            const float tmx = fmaxf(fmaxf(fmaxf(red[row], red[64 + row]), fmaxf(red[128 + row], red[192 + row])), -3e38f);
            const float m = mrun[row], f = mf[mf_at(row)], M = (tmx - m) * f > kKtHeadroom ? tmx : m;
            al[row] = M == m ? 1.f : ex2_approx((m - M) * f);
            mrun[row] = M;
            mf[mf_at(row) + 2] = -M;
          }
          kt_sync();
#pragma unroll
          for (int h = 0; h < N; ++h) l[h] *= al[h];
          if (!first) {
            // O holds this piece's earlier tiles: their PV must be done
            acquire(&pv_done[bf ^ 1], ((i - 1) >> 1) & 1);
            tc_fence_after();
            if (!dead) {
#pragma unroll 1
              for (int q = 0; q < N; q += 16) {
                float o[16];
                tmem_ld16(tl + kKtColO + q, o);
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < 16; ++h) o[h] *= al[q + h];
                tmem_st16(tl + kKtColO + q, o);
              }
              tmem_st_wait();
            }
          }
          weights();
        }
        first = false;
        none = none && !some;
#pragma unroll
        for (int h = 0; h < N; h += 2) {
          const float2 x = add2(make_float2(l[h], l[h + 1]), make_float2(s[h], s[h + 1]));
          l[h] = x.x;
          l[h + 1] = x.y;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s_free[bf]);
          mbar_arrive(&p_full[bf]);
        }
      }

      // ---- the piece's end: sums over the positions, O
      kt_reduce<N>(l, red + warp * 64, [](float x, float y) { return x + y; });
      kt_sync();
      const int seg = b * segs + g, s0 = pt - pc.i, s1 = s0 + nt, run = ln.run, ends = run == 1 << 30;
      const int w0 = ends ? ln.first : s0 / run, w1 = ends ? ln.last : (s1 - 1) / run;
      const bool whole = w0 == w1;
      float* res = a.part + ((size_t)blockIdx.x * 2 + (!ends && s0 > t0 ? 1 : 0)) * (size_t)N * kK4Part;
      if (row < N) {
        const float L = (red[row] + red[64 + row]) + (red[128 + row] + red[192 + row]);
        al[row] = L == 0.f ? 0.f : 1.f / L;
        if (!whole) *reinterpret_cast<float4*>(res + (size_t)row * kK4Part) = make_float4(mrun[row], L, mf[mf_at(row)], 0.f);
      }
      acquire(&pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1);
      tc_fence_after();
      kt_sync();
#pragma unroll 1
      for (int q = 0; q < N; q += 16) {
        float o[16];
        if (!dead) {
          tmem_ld16(tl + kKtColO + q, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int h = 0; h < 16; ++h) o[h] = 0.f;
        }
        if (whole) {
          uint16_t* dst = c.out + ((size_t)b * c.n_q + h0 + q) * kD + row;
#pragma unroll
          for (int h = 0; h < 16; ++h) dst[(size_t)h * kD] = (uint16_t)pack_bf16(o[h] * al[q + h], 0.f);
        } else {
#pragma unroll
          for (int h = 0; h < 16; ++h) res[(size_t)(q + h) * kK4Part + 4 + row] = o[h];
        }
      }
      tc_fence_before();
      // the CTA with the segment's first tile tells the merge kernel where its partials are
      if (pt == s0 && row == 0) segments[seg] = KtSegment{w0, whole ? 0 : w1 - w0 + 1, s0, run};
      kt_sync();
      k4_step(c, ln, segs, pc, i1 - (pt - t0));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kKtWarpMma) {
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

// The partials of the segments that several CTAs share: a warp a head, its
// pieces' weights by lanes, then O four dims a lane with eight loads in flight,
// the first of them ahead of the weights. A kernel of its own, for N heads of
// up to 152 pieces are more than one CTA should read (64 heads of one segment
// of 131072 positions: 549 us when the last CTA to arrive did it).
constexpr int kKmWarps = 8;
template <int N>
__global__ void __launch_bounds__(32 * kKmWarps) kt_merge_kernel(Kv4Args a, const KtSegment* segments) {
  __shared__ float wl[kKmWarps][kK4Ctas];
  const int seg = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y * kKmWarps + warp;
  const KtSegment u = segments[seg];
  if (u.np == 0) return;
  const Kv4AttnCall& c = a.c;
  constexpr int kFly = 8;
  auto piece = [&](int i) {
    const int w = u.w0 + i;
    return a.part + (((size_t)w * 2 + (u.run < (1 << 30) && u.s0 > w * u.run ? 1 : 0)) * N + h) * (size_t)kK4Part;
  };
  float4 x[kFly];
  auto load = [&](int q0) {
#pragma unroll
    for (int q = 0; q < kFly; ++q)
      if (q0 + q < u.np) x[q] = __ldcg(reinterpret_cast<const float4*>(piece(q0 + q) + 4) + lane);
  };
  load(0);
  constexpr int kMl = (kK4Ctas + 31) / 32;
  float4 ml[kMl];
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int k = 0; k < kMl; ++k) {
    ml[k] = lane + 32 * k < u.np ? __ldcg(reinterpret_cast<const float4*>(piece(lane + 32 * k))) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    M = fmaxf(M, ml[k].x);
  }
  M = warp_max(M);
  const float Ms = M == -INFINITY ? 0.f : M, f = __shfl_sync(0xffffffffu, ml[0].z, 0);
#pragma unroll
  for (int k = 0; k < kMl; ++k) {
    const float wt = ex2_approx((ml[k].x - Ms) * f);
    L += wt * ml[k].y;
    if (lane + 32 * k < u.np) wl[warp][lane + 32 * k] = wt;
  }
  L = warp_sum(L);
  __syncwarp();
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int q0 = 0; q0 < u.np; q0 += kFly) {
    if (q0 > 0) load(q0);
#pragma unroll
    for (int q = 0; q < kFly; ++q) {
      if (q0 + q >= u.np) break;
      const float w = wl[warp][q0 + q];
      v.x += w * x[q].x; v.y += w * x[q].y; v.z += w * x[q].z; v.w += w * x[q].w;
    }
  }
  const float r = L == 0.f ? 0.f : 1.f / L;
  const int b = seg / c.n_kv, g = seg - b * c.n_kv;
  *reinterpret_cast<uint2*>(c.out + ((size_t)b * c.n_q + g * N + h) * kD + 4 * lane) =
      make_uint2(pack_bf16(v.x * r, v.y * r), pack_bf16(v.z * r, v.w * r));
}

template <int N>
static int kt_run(const Kv4Args& a, void* stream) {
  if (set_func_attr((const void*)kv4_attn_tc_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kKtSmem) != cudaSuccess)
    return SPC_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  KtSegment* segments = static_cast<KtSegment*>(a.segments);
  kv4_attn_tc_kernel<N><<<kK4Ctas, kKtThreads, kKtSmem, st>>>(a, segments);
  if (cudaGetLastError() != cudaSuccess) return SPC_ERR_CUDA;
  // no segment is split where the table has room for kKtWhole tiles at most
  if ((a.c.max_blocks << a.c.block_shift) <= kKtWhole * kKtTile) return SPC_OK;
  kt_merge_kernel<N><<<dim3((unsigned)(a.c.B * a.c.n_kv), N / kKmWarps), 32 * kKmWarps, 0, st>>>(a, segments);
  return cudaGetLastError() == cudaSuccess ? SPC_OK : SPC_ERR_CUDA;
}

int kv4_attn_tc_launch(const Kv4Args& a, int G, void* stream) {
  switch (G) {
    case 32: return kt_run<32>(a, stream);
    default: return kt_run<64>(a, stream);
  }
}

}  // namespace spc
