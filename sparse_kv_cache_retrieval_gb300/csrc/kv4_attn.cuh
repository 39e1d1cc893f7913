// What the kernels of the decode attention over the 4-bit cache share: the
// line of tiles and how it is cut among the CTAs, and the merge of partials.
#pragma once

#include <stdint.h>

#include "kv4.cuh"
#include "spc_device.cuh"
#include "spc_internal.h"

namespace spc {

constexpr int kK4Ctas = 152;                         // one per SM; a constant, so that the workspace depends on shapes alone
constexpr int kK4Part = kD + 4;                      // a head's partial: m, l, factor of m to base 2, unused, O[128]
constexpr int kK4MaxKv = 128;                        // KV heads
// workspace: status, arrival counters (zero between calls), where a segment's
// partials are (tcgen05 kernel), partials. The offsets do not depend on the
// shapes, so that calls of different shapes may take turns on one workspace.
constexpr size_t kK4OffCount = 256;
constexpr size_t kK4OffSeg = kK4OffCount + (size_t)SPC_MAX_BATCH * kK4MaxKv * 2 * 4;
constexpr size_t kK4OffPart = kK4OffSeg + (size_t)SPC_MAX_BATCH * kK4MaxKv * 16;
constexpr long long kK4WaitLimit = 4000000000ll;     // clock cycles

struct Kv4Args {
  Kv4AttnCall c;
  int ht;            // head tiles (8 heads) a segment
  int hshift;        // log2 of the segments a KV head's group is split into
  int* status;
  uint32_t* counters; // one a segment
  void* segments;     // KtSegment, one a segment
  float* part;
  long long wait_limit;
  int starve;        // test builds: no copy is issued, so that every wait runs out
};

// groups of 32 or 64 heads over the whole context (kv4_attn_tc.cu)
int kv4_attn_tc_launch(const Kv4Args& a, int G, void* stream);

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// A head's logit factor, kept from vanishing (queries of zeros, a small scale):
// masked logits are -inf, and -inf times zero would not be. At this factor every
// logit is zero but for 2^-100. And kept from passing fp32's range (a large scale
// times large queries), where equal logits times infinity would be NaN: products
// q.K are multiples of 2^-34 below 2^20, so that at 2^100 the largest takes all
// and nothing overflows.
__device__ __forceinline__ float k4_factor(float f) { return fminf(fmaxf(f, 1.17549435e-38f), 1.26765060e30f); }
// x / d for 0 <= x <= 2^21 (a request's tiles, or a segment's times the CTAs), d
// >= 1. The approximate quotient is off by less than one there; an integer
// division costs some 150 cycles each in a plan that every CTA waits for.
__device__ __forceinline__ int k4_div(int x, int d) {
  const int q = (int)__fdividef((float)x, (float)d), r = x - q * d;
  return q + (r >= d ? 1 : 0) - (r < 0 ? 1 : 0);
}

// the line of tiles: request b's tiles (of every KV head and head split) start at pre[b]
struct K4Line {
  int pre[SPC_MAX_BATCH + 1];
  int nt[SPC_MAX_BATCH];       // tiles a segment of request b
  int run;                     // tiles a CTA takes; 2^30: runs end with their segments
  int t0, t1;                  // this CTA's run
  int empty;                   // some request has no tile
  int first, last;             // whole runs: the CTAs of its segment
  int len[SPC_MAX_BATCH];
};

// a segment whose tiles several CTAs share: its index, request, first head,
// first tile, first and last CTA, tiles a run
struct K4Open {
  int seg, b, h0, s0, w0, w1, run;
};

// a tile of the line: tile i of segment (b, s), s = (g << hshift) + hh, with what
// its copy needs of the segment
struct K4Cursor {
  int t, i, b, s;
  int nt, len;                 // the segment's tiles, the request's context
  const int32_t* table;        // the request's table row
};
__device__ __forceinline__ void k4_seg(const Kv4AttnCall& c, const K4Line& ln, K4Cursor& x) {
  const int b = min(x.b, c.B - 1);
  x.nt = max(1, ln.nt[b]);
  x.len = ln.len[b];
  x.table = c.table + (size_t)b * c.max_blocks;
}
__device__ __forceinline__ K4Cursor k4_at(const Kv4AttnCall& c, const K4Line& ln, int t) {
  int lo = 0, hi = c.B;        // pre[lo] <= t < pre[hi]; requests without tiles are passed over
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ln.pre[mid] <= t) lo = mid; else hi = mid;
  }
  K4Cursor x;
  x.t = t;
  x.b = lo;
  k4_seg(c, ln, x);
  const int r = t - ln.pre[lo];
  x.s = k4_div(r, x.nt);
  x.i = r - x.s * x.nt;
  return x;
}
__device__ __forceinline__ void k4_step(const Kv4AttnCall& c, const K4Line& ln, int segs, K4Cursor& x, int n) {
  x.t += n;
  x.i += n;
  if (x.i < x.nt) return;
  while (x.b < c.B && x.i >= ln.nt[x.b]) {
    x.i -= ln.nt[x.b];
    if (++x.s == segs) {
      x.s = 0;
      do ++x.b; while (x.b < c.B && ln.nt[x.b] == 0);
    }
  }
  k4_seg(c, ln, x);
}

// One warp: the line of TILE-position tiles and this CTA's part of it.
template <int TILE, int WHOLE, int MIN_RUN, int SLACK>
__device__ __forceinline__ void k4_plan(const Kv4Args& a, K4Line& ln, int segs, bool sel) {
  const Kv4AttnCall& c = a.c;
  const int lane = threadIdx.x & 31;
  // tiles a segment of each request, two requests a lane
  int n[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int b = 2 * lane + e;
    int L = b < c.B ? c.len[b] : 0;
    L = max(0, min(L, c.max_blocks << c.block_shift));
    const int nt = b < c.B ? ((sel ? c.budget : L) + TILE - 1) / TILE : 0;
    ln.len[b] = L;
    ln.nt[b] = nt;
    n[e] = nt * segs;
  }
  const int incl = warp_incl_scan(n[0] + n[1]);
  ln.pre[2 * lane] = incl - n[0] - n[1];
  ln.pre[2 * lane + 1] = incl - n[1];
  if (lane == 31) ln.pre[SPC_MAX_BATCH] = incl;
  // Which tiles of the line this CTA takes. A second piece costs a CTA about
  // SLACK tiles (queries, merge, fence), and a split segment waits for its
  // last piece, so runs end with their segments where they can:
  //  - segments of at most WHOLE tiles are never split: each CTA takes those
  //    that start in its share of a line in which every segment is SLACK longer
  //    (32 requests of 16 to 200 positions, 8 heads: 8.8 us, without about 20);
  //  - runs have MIN_RUN tiles at least;
  //  - with fewer segments than CTAs, each gets a number of CTAs of its own,
  //    if that makes no run longer than SLACK tiles above an equal share;
  //  - else equal runs of the line.
  constexpr int grid = kK4Ctas;
  const int total = __shfl_sync(0xffffffffu, incl, 31), blk = blockIdx.x;
  const int nt0 = ln.nt[2 * lane], nt1 = ln.nt[2 * lane + 1];
  int run = max((total + grid - 1) / grid, MIN_RUN), np0 = 0, np1 = 0;      // np: pieces a segment
  const bool small = (int)__reduce_max_sync(0xffffffffu, (unsigned)max(nt0, nt1)) <= WHOLE;
  bool whole = small;
  for (int k = 0; k <= 2 && !whole; ++k) {
    const int r = run + k * (SLACK / 2);
    np0 = k4_div(nt0 + r - 1, r);
    np1 = k4_div(nt1 + r - 1, r);
    whole = (int)__reduce_add_sync(0xffffffffu, (unsigned)((np0 + np1) * segs)) <= grid;
  }
  const bool empty = __any_sync(0xffffffffu, (2 * lane < c.B && nt0 == 0) || (2 * lane + 1 < c.B && nt1 == 0));
  int t0, t1, first = blk, last = blk;
  __syncwarp();                              // all lanes' ln.pre and ln.nt are read below
  // the last request that starts at or before x (the starts s0, s1 of this lane's two)
  auto find = [&](int s0, int s1, int x) {
    return __popc(__ballot_sync(0xffffffffu, s0 <= x)) + __popc(__ballot_sync(0xffffffffu, s1 <= x)) - 1;
  };
  if (small) {
    const int w0 = nt0 ? nt0 + SLACK : 0, w1 = nt1 ? nt1 + SLACK : 0;
    const int wi = warp_incl_scan((w0 + w1) * segs), s0 = wi - (w0 + w1) * segs, s1 = wi - w1 * segs;
    const int wt = __shfl_sync(0xffffffffu, wi, 31);
    auto start = [&](int x) {                      // of the first segment that starts at or behind x of that line
      const int e = find(s0, s1, x), len = max(1, __shfl_sync(0xffffffffu, e & 1 ? w1 : w0, e >> 1));
      const int p = __shfl_sync(0xffffffffu, e & 1 ? s1 : s0, e >> 1);
      return min(total, ln.pre[e] + k4_div(x - p + len - 1, len) * ln.nt[e]);
    };
    t0 = start((int)((long long)wt * blk / grid));
    t1 = start((int)((long long)wt * (blk + 1) / grid));
  } else if (whole) {
    const int end = warp_incl_scan((np0 + np1) * segs), c0 = end - (np0 + np1) * segs, c1 = end - np1 * segs;
    const int e = find(c0, c1, blk);
    const int np = __shfl_sync(0xffffffffu, e & 1 ? np1 : np0, e >> 1), nt = __shfl_sync(0xffffffffu, e & 1 ? nt1 : nt0, e >> 1);
    const int c0e = __shfl_sync(0xffffffffu, e & 1 ? c1 : c0, e >> 1);
    t0 = t1 = total;
    if (blk < __shfl_sync(0xffffffffu, end, 31)) {
      const int r = blk - c0e, sg = k4_div(r, np), q = r - sg * np, s0 = ln.pre[e] + sg * nt;
      first = blk - q;
      last = first + np - 1;
      t0 = s0 + k4_div(nt * q, np);
      t1 = s0 + k4_div(nt * (q + 1), np);
    }
  } else {
    t0 = min(total, blk * run);
    t1 = min(total, t0 + run);
  }
  if (lane == 0) {
    ln.run = whole ? 1 << 30 : run;
    ln.empty = empty ? 1 : 0;
    ln.t0 = t0;
    ln.t1 = t1;
    ln.first = first;
    ln.last = last;
  }
}

// The last CTA to arrive at a segment merges its CTAs' partials, in CTA order.
// kMg heads at a time: the pieces' (m, l) to shared memory, a weight per (head,
// piece), then O by (head, float4) items, kFly loads in flight, the first of
// them ahead of the weights. W warps, scratch of SCRATCH bytes.
template <int HT, int W, int SCRATCH>
__device__ __forceinline__ void k4_merge(const Kv4Args& a, const K4Open& u, int heads, float* mrg) {
  const Kv4AttnCall& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto sync = [&]() { asm volatile("bar.sync 1, %0;" :: "n"(32 * W) : "memory"); };
  constexpr int kMg = HT == 1 ? 8 : 16, kFly = 8;
  const int np = u.w1 - u.w0 + 1;
  float2* wl = reinterpret_cast<float2*>(mrg);                  // [kMg][kK4Ctas]
  float* lsum = mrg + 2 * kMg * kK4Ctas;                        // [kMg]
  float* fac = lsum + kMg;                                      // [kMg]
  static_assert((2 * kMg * kK4Ctas + 2 * kMg) * 4 <= SCRATCH, "merge scratch");
  auto piece = [&](int i, int h) {
    const int w = u.w0 + i;
    return a.part + (((size_t)w * 2 + (u.run < (1 << 30) && u.s0 > w * u.run ? 1 : 0)) * (8 * HT) + h) * (size_t)kK4Part;
  };
#pragma unroll 1
  for (int hb = 0; hb < heads; hb += kMg) {
    const int nh = min(kMg, heads - hb);
    float4 x[kFly];
    auto load = [&](int i, int q0) {
#pragma unroll
      for (int q = 0; q < kFly; ++q)
        if (q0 + q < np) x[q] = __ldcg(reinterpret_cast<const float4*>(piece(q0 + q, hb + (i >> 5)) + 4) + (i & 31));
    };
    if (threadIdx.x < nh * 32) load(threadIdx.x, 0);
    for (int i = threadIdx.x; i < nh * np; i += 32 * W) {
      const int h = i / np, q = i - h * np;
      const float4 x = __ldcg(reinterpret_cast<const float4*>(piece(q, hb + h)));
      wl[h * kK4Ctas + q] = make_float2(x.x, x.y);
      if (q == 0) fac[h] = x.z;
    }
    sync();
    for (int h = warp; h < nh; h += W) {
      float M = -INFINITY;
      for (int q = lane; q < np; q += 32) M = fmaxf(M, wl[h * kK4Ctas + q].x);
      M = warp_max(M);
      const float Ms = M == -INFINITY ? 0.f : M, f = fac[h];
      float L = 0.f;
      for (int q = lane; q < np; q += 32) {
        const float2 ml = wl[h * kK4Ctas + q];
        const float wt = ex2_approx((ml.x - Ms) * f);
        L += wt * ml.y;
        wl[h * kK4Ctas + q].x = wt;
      }
      L = warp_sum(L);
      if (lane == 0) lsum[h] = L == 0.f ? 0.f : 1.f / L;
    }
    sync();
    for (int i = threadIdx.x; i < nh * 32; i += 32 * W) {
      const int h = i >> 5, f4 = i & 31;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int q0 = 0; q0 < np; q0 += kFly) {
        if (q0 > 0 || i != threadIdx.x) load(i, q0);
#pragma unroll
        for (int q = 0; q < kFly; ++q) {
          if (q0 + q >= np) break;
          const float w = wl[h * kK4Ctas + q0 + q].x;
          v.x += w * x[q].x; v.y += w * x[q].y; v.z += w * x[q].z; v.w += w * x[q].w;
        }
      }
      const float r = lsum[h];
      *reinterpret_cast<uint2*>(c.out + ((size_t)u.b * c.n_q + u.h0 + hb + h) * kD + 4 * f4) =
          make_uint2(pack_bf16(v.x * r, v.y * r), pack_bf16(v.z * r, v.w * r));
    }
    sync();
  }
  if (threadIdx.x == 0) a.counters[u.seg] = 0u;
}

}  // namespace spc
