// Dense attention of a few query rows over a long cache (decode steps, short chunks, and
// every fp32 output), the attention weight per cache slot, and token appends to a cache
// without a tree.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "recsa_dense.cuh"

namespace recsa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;                  // query rows of a tile: queries x heads of a KV group
constexpr int kStep = 16;                  // keys of a step
constexpr int kStages = 2;                 // steps in flight of a warp
constexpr int kStepBytes = kStep * kRowBytes;
constexpr int kTableStride = kHalf * 8 + 64;  // bytes of a table row in shared memory
constexpr int kQStride = kD + 8;              // floats of a query row in shared memory

struct RowsSmem {
  unsigned char stage[kWarps][kStages][2][kStepBytes];  // [K, V]
  unsigned char table[kSpan * kTableStride];
  float q[2][kRows][kQStride];         // [window, sinks], scaled, turned to the tile's base position
  float4 ang[kWarps][kHalf / 2];       // a warp's rotation of the query rows, two frequencies each
  float m[kWarps][kRows], l[kWarps][kRows];
  uint32_t live[kWarps][kStages];      // a step's keys that were loaded
  int pos[kRows];                      // a row's position; 0 or less: nothing visible
  int last;
};

// One step's loads: 16 keys from token T, those outside [lo, hi) or on a page outside the
// pool as zeros.
template <bool PV>
__device__ __forceinline__ uint32_t load_step(const DenseArgs &a, int b, int h, int T, int lo, int hi,
                                              unsigned char (*st)[kStepBytes], int lane) {
  const int t = T + (lane & 15);
  bool live = t >= lo && t < hi;
  int64_t row = 0;
  if (live) {
    row = cache_row(a, b, h, t);
    if (row < 0) {
      row = 0;
      live = false;
      atomicOr(&a.hdr->err, kErrIndex);
    }
  }
  const uint32_t mask = __ballot_sync(0xffffffffu, live) & 0xffffu;
  const uint32_t sk = smem_u32(st[0]), sv = smem_u32(st[1]);
  const int c = lane & 15;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int key = 2 * i + (lane >> 4);
    const int64_t r = __shfl_sync(0xffffffffu, row, key);
    const bool on = (mask >> key) & 1u;
    const uint32_t off = key * kRowBytes + ((c ^ (key & 7)) << 4);
    cp_async16(sk + off, a.k + r * kD + c * 8, on);
    if (PV) cp_async16(sv + off, a.v + r * kD + c * 8, on);
  }
  return mask;
}

// The tile's rows turned to base position + delta, as the A operands of the score product:
// q (and with SPLIT what the rounding to bf16 leaves) for this thread's rows lane/4, lane/4+8.
template <bool SPLIT>
__device__ __forceinline__ void turn_queries(const DenseArgs &a, const float (*q)[kQStride], int delta, float4 *ang,
                                             uint32_t (&qh)[8][4], uint32_t (&ql)[SPLIT ? 8 : 1][4], int lane) {
  const uint64_t *f = ws_freq(a.hdr);
  __syncwarp();
  const float2 r0 = rotation(delta, __ldg(f + 2 * lane)), r1 = rotation(delta, __ldg(f + 2 * lane + 1));
  ang[lane] = make_float4(r0.x, r0.y, r1.x, r1.y);
  __syncwarp();
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int ch = 0; ch < 8; ++ch) {  // 8 dimensions: 16 of a k-step are two of these
    const float4 w = ang[ch * 4 + c];
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const float2 x = *reinterpret_cast<const float2 *>(&q[r + 8 * rr][ch * 8 + 2 * c]);
      const float2 y = *reinterpret_cast<const float2 *>(&q[r + 8 * rr][ch * 8 + 2 * c + kHalf]);
      const float x0 = x.x * w.x - y.x * w.y, x1 = x.y * w.z - y.y * w.w;
      const float y0 = y.x * w.x + x.x * w.y, y1 = y.y * w.z + x.y * w.w;
      const int ks = ch >> 1, reg = (ch & 1) * 2 + rr;
      qh[ks][reg] = cvt_bf16x2(x0, x1);
      qh[ks + 4][reg] = cvt_bf16x2(y0, y1);
      if (SPLIT) {
        ql[ks][reg] = residue_bf16x2(x0, x1, qh[ks][reg]);
        ql[ks + 4][reg] = residue_bf16x2(y0, y1, qh[ks + 4][reg]);
      }
    }
  }
}

// Scores of the step's keys 8 nt .. 8 nt + 7: rotates them by their place in the span and
// multiplies.  With SPLIT both operands are two bf16 parts, hi * hi + lo * hi + hi * lo: what
// is dropped is below 2^-16 of the product of the magnitudes.
template <bool SPLIT>
__device__ __forceinline__ void score_keys(const unsigned char *table, uint32_t sk, int T, int nt,
                                           const uint32_t (&qh)[8][4], const uint32_t (&ql)[SPLIT ? 8 : 1][4],
                                           float (&s)[4], int lane) {
  uint32_t kr[16];
  const int key = nt * 8 + (lane & 7);
#pragma unroll
  for (int g = 0; g < 4; ++g)
    ldsm4(sk + key * kRowBytes + (((4 * g + (lane >> 3)) ^ (key & 7)) << 4), kr[4 * g], kr[4 * g + 1], kr[4 * g + 2],
          kr[4 * g + 3]);
  const unsigned char *tr = table + ((T & (kSpan - 1)) + nt * 8 + (lane >> 2)) * kTableStride + (lane & 3) * 16;
  float hi[4] = {0.f, 0.f, 0.f, 0.f}, lo[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    uint32_t kh[4], kl[4];  // k-step ks: 0, 1; k-step ks + 4: 2, 3
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int ch = 2 * ks + i;
      const float4 w = *reinterpret_cast<const float4 *>(tr + ch * 64);
      const float x0 = bf16_lo(kr[ch]), x1 = bf16_hi(kr[ch]), y0 = bf16_lo(kr[ch + 8]), y1 = bf16_hi(kr[ch + 8]);
      const float u0 = x0 * w.x - y0 * w.y, u1 = x1 * w.z - y1 * w.w;
      const float v0 = y0 * w.x + x0 * w.y, v1 = y1 * w.z + x1 * w.w;
      kh[i] = cvt_bf16x2(u0, u1);
      kh[2 + i] = cvt_bf16x2(v0, v1);
      if (SPLIT) {
        kl[i] = residue_bf16x2(u0, u1, kh[i]);
        kl[2 + i] = residue_bf16x2(v0, v1, kh[2 + i]);
      }
    }
    mma16816(hi, qh[ks], kh[0], kh[1]);
    if (SPLIT) mma16816(lo, ql[SPLIT ? ks : 0], kh[0], kh[1]);
    mma16816(hi, qh[ks + 4], kh[2], kh[3]);
    if (SPLIT) {
      mma16816(lo, qh[ks], kl[0], kl[1]);
      mma16816(lo, ql[SPLIT ? ks + 4 : 0], kh[2], kh[3]);
      mma16816(lo, qh[ks + 4], kl[2], kl[3]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = hi[i] + lo[i];
}

__device__ __forceinline__ bool not_finite(uint32_t bf16x2) {
  return (bf16x2 & 0x7f80u) == 0x7f80u || (bf16x2 & 0x7f800000u) == 0x7f800000u;
}

// What one block of a tile's key range covers.  Steps are numbered over the sinks first, then
// the window's tokens; both start on multiples of 16.
struct Range {
  int n1, first;  // steps of the sinks; first step of the window
  int hi1, lo2, hi2;
  int total;
};
__device__ __forceinline__ Range tile_range(const DenseArgs &a, int p_min, int p_max) {
  Range r;
  r.hi1 = a.window ? max(0, min(a.sinks, p_max)) : 0;
  r.n1 = (r.hi1 + kStep - 1) / kStep;
  r.lo2 = max(0, window_first(a, p_min));
  r.hi2 = max(p_max, 0);
  r.first = r.lo2 / kStep;
  r.total = r.n1 + (r.hi2 > r.lo2 ? (r.hi2 + kStep - 1) / kStep - r.first : 0);
  return r;
}

// One tile of 16 query rows (16 / G queries of one sequence and KV group) against one block's
// share of the keys they see.  Each warp walks its own steps of 16 keys through a private ring
// of cp.async stages with an online softmax, so warps never wait for one another until their
// (max, sum, output) are joined at the end; the last block of a tile joins the blocks.  Reading
// K and V bounds it: at G = 4 a key costs 512 bytes and about 45 issue slots of its SM's ~88.
// PV: values are weighted and summed; without it the rows' log2-sum-exp goes to `lse`.
template <bool SPLIT, bool PV>
__global__ void __launch_bounds__(kThreads, 1) dense_rows_kernel(DenseArgs a, float *lse, const uint32_t *redo, int chunk_tiles) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  RowsSmem &sm = *reinterpret_cast<RowsSmem *>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t item = blockIdx.x / a.nsplit;
  const int split = blockIdx.x % a.nsplit;
  const int tile = item % a.tiles, bh = item / a.tiles;
  const int b = bh / a.hkv, h = bh % a.hkv;
  const int gs = a.group_shift, G = 1 << gs, hq = a.hkv << gs;
  const int q0 = tile * (kRows >> gs), nq = min(kRows >> gs, a.nq - q0);  // the tile's queries
  if (a.hdr->magic != kDenseMagic || a.hdr->rope_base != a.rope_base) {
    if (tid == 0) atomicOr(&a.hdr->err, kErrWs);
    return;
  }
  if (redo) {  // only what the chunk kernel marked
    const int chunk_item = bh * chunk_tiles + chunk_tiles - 1 - q0 / (256 >> gs);
    if (!redo[chunk_item % kMaxShared]) return;
  }
  const int len = dense_length(a, b, tid == 0 && tile == 0 && split == 0 && h == 0);
  const int p_min = dense_position(a, len, q0), p_max = dense_position(a, len, q0 + nq - 1);
  const Range rg = tile_range(a, p_min, p_max);
  const int base_sink = sink_position(a, p_max);

  if (tid < kRows) sm.pos[tid] = (tid >> gs) < nq ? dense_position(a, len, q0 + (tid >> gs)) : 0;
  for (int e = tid; e < kSpan * kHalf / 2; e += kThreads)
    *reinterpret_cast<float4 *>(sm.table + (e / (kHalf / 2)) * kTableStride + (e % (kHalf / 2)) * 16) =
        __ldg(reinterpret_cast<const float4 *>(ws_table(a.hdr)) + e);
  for (int e = tid; e < kRows * kHalf * 2; e += kThreads) {  // query rows, turned to the tile's last position
    const int i = e % kHalf, row = (e / kHalf) % kRows, sink = e / (kHalf * kRows);
    if (sink && !rg.n1) break;
    float x = 0.f, y = 0.f;
    if ((row >> gs) < nq) {
      const uint16_t *src = a.q + (((int64_t)b * a.nq + q0 + (row >> gs)) * hq + h * G + (row & (G - 1))) * kD + i;
      x = __uint_as_float((uint32_t)src[0] << 16) * a.qscale;
      y = __uint_as_float((uint32_t)src[kHalf] << 16) * a.qscale;
      const int p = dense_position(a, len, q0 + (row >> gs));
      const int d = sink ? sink_position(a, p) - base_sink : p - p_max;
      if (d != 0) {
        const float2 w = rotation(d, __ldg(ws_freq(a.hdr) + i));
        const float u = x * w.x - y * w.y;
        y = y * w.x + x * w.y;
        x = u;
      }
    }
    sm.q[sink][row][i] = x;
    sm.q[sink][row][i + kHalf] = y;
  }
  __syncthreads();

  // this warp's steps
  const int64_t parts = (int64_t)a.nsplit * kWarps, part = (int64_t)split * kWarps + warp;
  const int st0 = (int)(rg.total * part / parts), st1 = (int)(rg.total * (part + 1) / parts);
  auto start = [&](int st) {
    const int s = st % kStages;
    const bool sink = st < rg.n1;
    const int T = (sink ? st : rg.first + st - rg.n1) * kStep;
    const uint32_t m = load_step<PV>(a, b, h, T, sink ? 0 : rg.lo2, sink ? rg.hi1 : rg.hi2, sm.stage[warp][s], lane);
    if (lane == 0) sm.live[warp][s] = m;
  };
  const int r = lane >> 2, c = lane & 3;
  const int pa = sm.pos[r], pb = sm.pos[r + 8];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  float o[PV ? 16 : 1][4];
#pragma unroll
  for (int i = 0; i < (PV ? 16 : 1); ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  uint32_t qh[8][4], ql[SPLIT ? 8 : 1][4];
  int turned = -1;  // the span the query rows are turned for (sinks: odd)

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (st0 + i < st1) start(st0 + i);
    cp_async_commit();
  }
  for (int st = st0; st < st1; ++st) {
    if (st + kStages - 1 < st1) start(st + kStages - 1);
    cp_async_commit();
    const bool sink = st < rg.n1;
    const int T = (sink ? st : rg.first + st - rg.n1) * kStep;
    const int span = (T / kSpan) * 2 + (sink ? 1 : 0);
    if (span != turned) {
      turned = span;
      turn_queries<SPLIT>(a, sm.q[sink], (sink ? base_sink : p_max) - (T & ~(kSpan - 1)), sm.ang[warp], qh, ql, lane);
    }
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t sk = smem_u32(sm.stage[warp][st % kStages][0]), sv = sk + kStepBytes;
    const uint32_t live = sm.live[warp][st % kStages];
    // tokens [la, ha) and [lb, hb) are visible to this thread's two rows
    const int la = sink ? 0 : window_first(a, pa), lb = sink ? 0 : window_first(a, pb);
    const int ha = sink ? min(pa, rg.hi1) : pa, hb = sink ? min(pb, rg.hi1) : pb;
    float s[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      score_keys<SPLIT>(sm.table, sk, T, nt, qh, ql, s[nt], lane);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = nt * 8 + 2 * c + i, t = T + j;
        const bool on = (live >> j) & 1u;
        if (!(on && t >= la && t < ha)) s[nt][i] = -INFINITY;
        if (!(on && t >= lb && t < hb)) s[nt][2 + i] = -INFINITY;
      }
    }
    float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
    float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
    }
    const bool up = x0 > m0 || x1 > m1;
    if (__any_sync(0xffffffffu, up)) {
      const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
      const float f0 = m0 == -INFINITY ? 0.f : exp2_approx(m0 - n0), f1 = m1 == -INFINITY ? 0.f : exp2_approx(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= f0;
      l1 *= f1;
      if (PV) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[i][0] *= f0;
          o[i][1] *= f0;
          o[i][2] *= f1;
          o[i][3] *= f1;
        }
      }
    }
    const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
    bool hidden = false;  // some key of the step is not seen by some row of this thread
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        hidden |= s[nt][i] == -INFINITY || s[nt][2 + i] == -INFINITY;
        s[nt][i] = exp2_approx(s[nt][i] - z0);
        s[nt][2 + i] = exp2_approx(s[nt][2 + i] - z1);
        l0 += s[nt][i];
        l1 += s[nt][2 + i];
      }
    if (PV) {
      // A row that does not see a key must not touch its value: a product with a zero weight
      // would carry an infinity or NaN over.  In steps that hide a key from some row, values
      // that are not finite go to the rows that see them one by one and are zeros in the product.
      if (__any_sync(0xffffffffu, hidden)) {
        bool odd = false;
        for (int i = lane; i < kStepBytes / 4; i += 32) {
          uint32_t u;
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(sv + i * 4));
          odd |= not_finite(u);
        }
        if (__any_sync(0xffffffffu, odd)) {
          for (int j = 0; j < kStep; ++j) {
            const int src = (lane & ~3) | ((j & 7) >> 1);
            const float e0 = (j & 8) ? ((j & 1) ? s[1][1] : s[1][0]) : ((j & 1) ? s[0][1] : s[0][0]);
            const float e1 = (j & 8) ? ((j & 1) ? s[1][3] : s[1][2]) : ((j & 1) ? s[0][3] : s[0][2]);
            const float w0 = __shfl_sync(0xffffffffu, e0, src), w1 = __shfl_sync(0xffffffffu, e1, src);
            const bool on = (live >> j) & 1u;
            const bool va = on && T + j >= la && T + j < ha, vb = on && T + j >= lb && T + j < hb;
#pragma unroll
            for (int n = 0; n < 16; ++n) {
              uint32_t u;
              asm volatile("ld.shared.u32 %0, [%1];"
                           : "=r"(u)
                           : "r"(sv + j * kRowBytes + ((n ^ (j & 7)) << 4) + c * 4));
              const float v0 = bf16_lo(u), v1 = bf16_hi(u);
              if (!isfinite(v0)) {
                if (va) o[PV ? n : 0][0] += w0 * v0;
                if (vb) o[PV ? n : 0][2] += w1 * v0;
              }
              if (!isfinite(v1)) {
                if (va) o[PV ? n : 0][1] += w0 * v1;
                if (vb) o[PV ? n : 0][3] += w1 * v1;
              }
            }
          }
          __syncwarp();
          for (int i = lane; i < kStepBytes / 4; i += 32) {
            uint32_t u;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(sv + i * 4));
            if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
            if ((u & 0x7f800000u) == 0x7f800000u) u &= 0xffffu;
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(sv + i * 4), "r"(u) : "memory");
          }
          __syncwarp();
        }
      }
      {
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            ph[nt * 2 + rr] = cvt_bf16x2(s[nt][2 * rr], s[nt][2 * rr + 1]);
            if (SPLIT) pl[nt * 2 + rr] = residue_bf16x2(s[nt][2 * rr], s[nt][2 * rr + 1], ph[nt * 2 + rr]);
          }
        const int key = ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
        for (int d = 0; d < 16; d += 2) {
          uint32_t b0, b1, b2, b3;
          ldsm4_trans(sv + key * kRowBytes + (((d + (lane >> 4)) ^ (key & 7)) << 4), b0, b1, b2, b3);
          if (SPLIT) {
            // The tensor cores cut their fp32 sums off instead of rounding them: over a million
            // keys an output summed there alone came out 5e-5 short.  A step's 16 keys are
            // summed there, the steps in fp32 adds that round.
            float t0[4] = {0.f, 0.f, 0.f, 0.f}, t1[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816(t0, pl, b0, b1);
            mma16816(t1, pl, b2, b3);
            mma16816(t0, ph, b0, b1);
            mma16816(t1, ph, b2, b3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[PV ? d : 0][i] += t0[i];
              o[PV ? d + 1 : 0][i] += t1[i];
            }
          } else {
            mma16816(o[PV ? d : 0], ph, b0, b1);
            mma16816(o[PV ? d + 1 : 0], ph, b2, b3);
          }
        }
      }
    }
    __syncwarp();  // the stage is free for the next load
  }
  cp_async_wait<0>();

  // join the warps: their outputs in the stage memory
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, d);
    l1 += __shfl_xor_sync(0xffffffffu, l1, d);
  }
  if (c == 0) {
    sm.m[warp][r] = m0;
    sm.m[warp][r + 8] = m1;
    sm.l[warp][r] = l0;
    sm.l[warp][r + 8] = l1;
  }
  __syncthreads();
  float *const wo = reinterpret_cast<float *>(sm.stage);  // [warp][16][kQStride]
  if (PV) {
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      float *p = wo + (warp * kRows + r) * kQStride + n * 8 + 2 * c;
      *reinterpret_cast<float2 *>(p) = make_float2(o[PV ? n : 0][0], o[PV ? n : 0][1]);
      *reinterpret_cast<float2 *>(p + 8 * kQStride) = make_float2(o[PV ? n : 0][2], o[PV ? n : 0][3]);
    }
  }
  __syncthreads();
  const int row = tid >> 4, d0 = (tid & 15) * 8;  // a thread: 8 dimensions of a row
  float m = -INFINITY, l = 0.f, acc[8] = {};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[w][row]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float mw = sm.m[w][row];
    if (mw == -INFINITY) continue;
    const float f = exp2_approx(mw - m);
    l += f * sm.l[w][row];
    if (PV) {
      const float4 *p = reinterpret_cast<const float4 *>(wo + (w * kRows + row) * kQStride + d0);
      const float4 u = p[0], v = p[1];
      acc[0] += f * u.x, acc[1] += f * u.y, acc[2] += f * u.z, acc[3] += f * u.w;
      acc[4] += f * v.x, acc[5] += f * v.y, acc[6] += f * v.z, acc[7] += f * v.w;
    }
  }
  if (a.nsplit > 1) {  // leave this block's part; the last block of the tile joins them in order
    float *part_row = ws_part(a.hdr) + ((int64_t)blockIdx.x * kRows + row) * kPartRow;
    if (d0 == 0) *reinterpret_cast<float2 *>(part_row) = make_float2(m, l);
    if (PV) {
      float4 *p = reinterpret_cast<float4 *>(part_row + 4 + d0);
      p[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      p[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      const int done = atomicAdd(ws_count(a.hdr) + item, 1);
      sm.last = done == a.nsplit - 1;
      if (sm.last) ws_count(a.hdr)[item] = 0;  // for the next call
    }
    __syncthreads();
    if (!sm.last) return;
    __threadfence();
    const float *p0 = ws_part(a.hdr) + ((int64_t)item * a.nsplit * kRows + row) * kPartRow;
    const int64_t stride = (int64_t)kRows * kPartRow;
    m = -INFINITY;
    l = 0.f;
    for (int j = 0; j < a.nsplit; ++j) m = fmaxf(m, __ldcg(p0 + j * stride));
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int j = 0; j < a.nsplit; ++j) {
      const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p0 + j * stride));
      const float f = ml.x == -INFINITY ? 0.f : exp2_approx(ml.x - m);
      if (ml.x == -INFINITY) continue;
      l += f * ml.y;
      if (PV) {
        const float4 u = __ldcg(reinterpret_cast<const float4 *>(p0 + j * stride + 4 + d0));
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p0 + j * stride + 8 + d0));
        acc[0] += f * u.x, acc[1] += f * u.y, acc[2] += f * u.z, acc[3] += f * u.w;
        acc[4] += f * v.x, acc[5] += f * v.y, acc[6] += f * v.z, acc[7] += f * v.w;
      }
    }
  }
  if ((row >> gs) >= nq) return;
  const int64_t out_row = ((int64_t)b * a.nq + q0 + (row >> gs)) * hq + h * G + (row & (G - 1));
  if (!PV) {
    if (d0 == 0) lse[out_row] = l > 0.f || !(l == l) ? m + log2f(l) : INFINITY;  // no key: every weight is exp2(-inf)
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] *= inv;
  if (a.out_fp32) {
    float4 *p = reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + out_row * kD + d0);
    p[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    p[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  } else {
    *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(a.out) + out_row * kD + d0) =
        make_uint4(cvt_bf16x2(acc[0], acc[1]), cvt_bf16x2(acc[2], acc[3]), cvt_bf16x2(acc[4], acc[5]),
                   cvt_bf16x2(acc[6], acc[7]));
  }
}

// ---------------------------------------------------------------------------------------
// Weights per slot: w[t] = sum over rows of exp2(s[row][t] - lse[row]).  A block holds keys
// (each warp 64 at a time, one span) and walks the query rows in pieces of 16; keys are
// rotated against a span's table, rows turned to the span, so scores are formed exactly as
// the pass that summed lse formed them.

struct WeightsSmem {
  unsigned char stage[kWarps][kStep * 2][kRowBytes];  // 32 keys of a warp
  unsigned char table[kSpan * kTableStride];
  float q[kRows][kQStride];
  float4 ang[kWarps][kHalf / 2];
  float lse[kRows];
  int pos[kRows];
};

__global__ void __launch_bounds__(kThreads, 1)
    dense_weights_kernel(DenseArgs a, const float *__restrict__ lse, float *__restrict__ weights, int accumulate) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  WeightsSmem &sm = *reinterpret_cast<WeightsSmem *>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x / a.nsplit, split = blockIdx.x % a.nsplit;
  const int b = bh / a.hkv, h = bh % a.hkv;
  const int gs = a.group_shift, G = 1 << gs, hq = a.hkv << gs;
  if (a.hdr->magic != kDenseMagic || a.hdr->rope_base != a.rope_base) {
    if (tid == 0) atomicOr(&a.hdr->err, kErrWs);
    return;
  }
  const int len = dense_length(a, b, tid == 0 && split == 0 && h == 0);
  for (int e = tid; e < kSpan * kHalf / 2; e += kThreads)
    *reinterpret_cast<float4 *>(sm.table + (e / (kHalf / 2)) * kTableStride + (e % (kHalf / 2)) * 16) =
        __ldg(reinterpret_cast<const float4 *>(ws_table(a.hdr)) + e);
  const int steps = (len + 31) / 32;  // 32 keys a warp, 8 warps a round
  const int rounds = (steps + kWarps - 1) / kWarps;
  const int r = lane >> 2, c = lane & 3;
  const int qt = kRows >> gs;
  float *const w_row = weights + ((int64_t)b * a.hkv + h) * a.capacity;

  for (int rd = split; rd < rounds; rd += a.nsplit) {
    const int T = (rd * kWarps + warp) * 32;
    uint32_t live = 0;
    __syncwarp();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int Th = T + half * kStep;
      unsigned char(*st)[kStepBytes] = reinterpret_cast<unsigned char(*)[kStepBytes]>(sm.stage[warp][half * kStep]);
      live |= load_step<false>(a, b, h, Th, 0, len, st, lane) << (16 * half);
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncwarp();
    const uint32_t sk = smem_u32(sm.stage[warp]);
    float sum[4][2];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) sum[nt][0] = sum[nt][1] = 0.f;
    for (int q0 = 0; q0 < a.nq; q0 += qt) {
      const int nq = min(qt, a.nq - q0);
      const int p_max = dense_position(a, len, q0 + nq - 1);
      __syncthreads();
      if (tid < kRows) {
        const bool in = (tid >> gs) < nq;
        sm.pos[tid] = in ? dense_position(a, len, q0 + (tid >> gs)) : 0;
        sm.lse[tid] = in ? lse[((int64_t)b * a.nq + q0 + (tid >> gs)) * hq + h * G + (tid & (G - 1))] : INFINITY;
      }
      for (int e = tid; e < kRows * kHalf; e += kThreads) {
        const int i = e % kHalf, row = e / kHalf;
        float x = 0.f, y = 0.f;
        if ((row >> gs) < nq) {
          const uint16_t *src = a.q + (((int64_t)b * a.nq + q0 + (row >> gs)) * hq + h * G + (row & (G - 1))) * kD + i;
          x = __uint_as_float((uint32_t)src[0] << 16) * a.qscale;
          y = __uint_as_float((uint32_t)src[kHalf] << 16) * a.qscale;
          const int d = dense_position(a, len, q0 + (row >> gs)) - p_max;
          if (d != 0) {
            const float2 w = rotation(d, __ldg(ws_freq(a.hdr) + i));
            const float u = x * w.x - y * w.y;
            y = y * w.x + x * w.y;
            x = u;
          }
        }
        sm.q[row][i] = x;
        sm.q[row][i + kHalf] = y;
      }
      __syncthreads();
      if (T < len && p_max > T) {
        uint32_t qh[8][4], ql[8][4];
        turn_queries<true>(a, sm.q, p_max - (T & ~(kSpan - 1)), sm.ang[warp], qh, ql, lane);
        const int pa = sm.pos[r], pb = sm.pos[r + 8];
        const float za = sm.lse[r], zb = sm.lse[r + 8];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          float s[4];
          score_keys<true>(sm.table, sk, T, nt, qh, ql, s, lane);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int t = T + nt * 8 + 2 * c + i;
            if (t < pa) sum[nt][i] += exp2_approx(s[i] - za);
            if (t < pb) sum[nt][i] += exp2_approx(s[2 + i] - zb);
          }
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = sum[nt][i];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        const int j = nt * 8 + 2 * c + i;
        if (r == 0 && T + j < len) {
          if (!((live >> j) & 1u)) v = 0.f;  // a token on a page outside the pool receives nothing
          w_row[T + j] = accumulate ? w_row[T + j] + v : v;
        }
      }
  }
}

__global__ void append_tokens_kernel(DenseArgs a, uint4 *k, uint4 *v, const uint4 *__restrict__ k_new,
                                     const uint4 *__restrict__ v_new, int64_t at, int count, int64_t limit) {
  const int64_t n16 = (int64_t)a.batch * count * a.hkv * 16;
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n16; e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = e >> 4;
    const int part = (int)(e & 15), h = (int)(row % a.hkv);
    const int64_t bi = row / a.hkv;
    const int i = (int)(bi % count), b = (int)(bi / count);
    int64_t from = at;
    if (a.seq_len) {  // a sequence with no room for the tokens is left as it is
      from = a.seq_len[b];
      if (from < 0 || from + count > limit) {
        if (part == 0 && h == 0 && i == 0) atomicOr(&a.hdr->err, kErrIndex);
        continue;
      }
    }
    const int64_t dst = cache_row(a, b, h, (int)(from + i));
    if (dst < 0) {
      atomicOr(&a.hdr->err, kErrIndex);
      continue;
    }
    k[dst * 16 + part] = k_new[e];
    v[dst * 16 + part] = v_new[e];
  }
}

__global__ void dense_init_kernel(unsigned char *ws, double base) {
  WsHeader *hdr = reinterpret_cast<WsHeader *>(ws);
  const int idx = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = idx % kHalf, r = idx / kHalf;
  const double theta = pow(base, -2.0 * (double)i / (double)kD);
  if (r < kSpan) {
    double s, c;
    sincos((double)r * theta, &s, &c);
    reinterpret_cast<float2 *>(ws + kDenseTable)[idx] = make_float2((float)c, (float)s);
  }
  if (r == 0) {
    const double turns = theta / (2.0 * 3.14159265358979323846);
    reinterpret_cast<uint64_t *>(ws + kDenseFreq)[i] = (uint64_t)((turns - floor(turns)) * 18446744073709551616.0);
  }
  if (idx < kMaxShared) {
    reinterpret_cast<int32_t *>(ws + kDenseCount)[idx] = 0;
    reinterpret_cast<uint32_t *>(ws + kDenseRedo)[idx] = 0u;
  }
  if (idx == 0) {
    hdr->err = 0u;
    hdr->table_rows = kSpan;
    hdr->rope_base = (float)base;
    __threadfence();
    hdr->magic = kDenseMagic;
  }
}

template <typename K>
int opt_in(K kernel, size_t bytes) {
  return (int)cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <bool SPLIT, bool PV>
int run_rows(const DenseArgs &a, unsigned grid, float *lse, void *stream, const uint32_t *redo = nullptr,
             int chunk_tiles = 0) {
  int rc = opt_in(dense_rows_kernel<SPLIT, PV>, sizeof(RowsSmem));
  if (rc) return rc;
  dense_rows_kernel<SPLIT, PV><<<grid, kThreads, sizeof(RowsSmem), (cudaStream_t)stream>>>(a, lse, redo, chunk_tiles);
  return (int)cudaGetLastError();
}

}  // namespace

int dense_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  return n;
}

int launch_dense_init(void *ws, double base, void *stream) {
  static_assert(kSpan * kHalf >= kMaxShared, "one thread per counter");
  dense_init_kernel<<<kSpan * kHalf / 256, 256, 0, (cudaStream_t)stream>>>(reinterpret_cast<unsigned char *>(ws), base);
  return (int)cudaGetLastError();
}

// Blocks a tile's keys are shared among: enough for every SM, in waves as full as possible, as
// long as a block keeps kMinKeys keys (below that the join costs more than the walk it saves).
static int pick_split(int64_t items, int64_t max_keys, int sms) {
  constexpr int64_t kMinKeys = 256;
  if (items > kMaxShared) return 1;
  const int64_t most = std::min<int64_t>({std::max<int64_t>(1, max_keys / kMinKeys), kRowsParts / items, 512});
  int best = 1;
  double cost = 1e30;
  for (int64_t n = 1; n <= most; ++n) {
    const int64_t waves = ceil_div(items * n, sms);
    // a wave's time in keys walked, plus about 1000 keys' worth of a block's start and end
    const double c = (double)waves * ((double)max_keys / (double)n + 1000.0);
    if (c < cost * 0.995) {
      cost = c;
      best = (int)n;
    }
    if (waves > 12) break;
  }
  return best;
}

int launch_dense_rows(DenseArgs a, bool split, int64_t max_keys, float *lse, void *stream) {
  const int per = kRows >> a.group_shift;
  a.tiles = (a.nq + per - 1) / per;
  const int64_t items = (int64_t)a.batch * a.hkv * a.tiles;
  a.nsplit = pick_split(items, max_keys, dense_sm_count());
  const unsigned grid = (unsigned)(items * a.nsplit);
  if (lse) return run_rows<true, false>(a, grid, lse, stream);
  return split ? run_rows<true, true>(a, grid, nullptr, stream) : run_rows<false, true>(a, grid, nullptr, stream);
}

int launch_dense_redo(DenseArgs a, int chunk_tiles, void *stream) {
  const int per = kRows >> a.group_shift;
  a.tiles = (a.nq + per - 1) / per;
  a.nsplit = 1;
  uint32_t *redo = reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(a.hdr) + kDenseRedo);
  int rc = run_rows<true, true>(a, (unsigned)((int64_t)a.batch * a.hkv * a.tiles), nullptr, stream, redo, chunk_tiles);
  if (rc) return rc;
  return (int)cudaMemsetAsync(redo, 0, kMaxShared * sizeof(uint32_t), (cudaStream_t)stream);
}

int launch_dense_weights(DenseArgs a, const float *lse, float *weights, int accumulate, void *stream) {
  int rc = opt_in(dense_weights_kernel, sizeof(WeightsSmem));
  if (rc) return rc;
  const int64_t heads = (int64_t)a.batch * a.hkv;
  const int64_t rounds = ceil_div(a.length, 32 * kWarps);
  a.nsplit = (int)std::min<int64_t>(std::max<int64_t>(rounds, 1), std::max<int64_t>(1, 4 * dense_sm_count() / heads));
  dense_weights_kernel<<<(unsigned)(heads * a.nsplit), kThreads, sizeof(WeightsSmem), (cudaStream_t)stream>>>(
      a, lse, weights, accumulate);
  return (int)cudaGetLastError();
}

int launch_append_tokens(const DenseArgs &a, void *k, void *v, const void *k_new, const void *v_new, int64_t at,
                         int count, int64_t limit, void *stream) {
  const int64_t n16 = (int64_t)a.batch * count * a.hkv * 16;
  const int threads = 256;
  const int64_t grid = std::min<int64_t>(ceil_div(n16, threads), (int64_t)dense_sm_count() * 8);
  append_tokens_kernel<<<(unsigned)grid, threads, 0, (cudaStream_t)stream>>>(
      a, reinterpret_cast<uint4 *>(k), reinterpret_cast<uint4 *>(v), reinterpret_cast<const uint4 *>(k_new),
      reinterpret_cast<const uint4 *>(v_new), at, count, limit);
  return (int)cudaGetLastError();
}

}  // namespace recsa
