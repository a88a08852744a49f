// Dense attention of a few query rows over a long cache (decode steps, short chunks, and
// every fp32 output), and token appends to a cache without a tree.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "recsa_dense.cuh"

namespace recsa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 16;                  // keys of a step
constexpr int kStepBytes = kStep * kRowBytes;
constexpr int kTableStride = kHalf * 8;       // bytes of a table row in shared memory
constexpr int kQStride = kD + 4;              // floats of a query row in shared memory
constexpr int kOStride = kD + 8;              // floats of an output row in shared memory
constexpr int kDealtSequences = kThreads;     // sequences whose steps can be dealt out (a thread counts one's)
constexpr int kDealtSteps = 16;               // steps a block is worth starting for
constexpr float kRowsRescale = 64.f;          // a row's maximum may lag by 2^64 before its output is rescaled
// A row whose output overflows that way (values above 2^63, infinities) is computed once more by
// careful_row, with weights of at most 2^-32: sums of 2^30 of them stay finite.
constexpr float kRowsLarge = 0x1p96f;         // outputs up to here join without overflow
constexpr float kRowsLift = 32.f;

template <int R>  // query rows of a tile: queries x heads of a KV group
struct RowsSmem {
  unsigned char stage[kWarps][2][kStepBytes];  // [K, V]
  // two frequencies: cos, cos', sin, sin'; the pieces of odd rows are moved by four places, so that
  // the two rows a quarter warp reads lie in different banks
  unsigned char table[kSpan * kTableStride];
  float q[2][R][kQStride];             // [window, sinks], scaled, turned to the tile's base position
  float4 ang[kWarps][kHalf / 2];       // a warp's rotation of the query rows, as the table
  float m[kWarps][R], l[kWarps][R];
  int pos[R];                          // a row's position; 0 or less: nothing visible
  int last;
  int range[2];                        // the block's steps of the tile
  int dealt[kDealtSequences + 1];      // steps before each sequence, when steps are dealt out to the blocks
};

// One step's rows: 16 keys from token T, those outside [lo, hi) or on a page outside the pool as
// zeros; `live` are the keys that are there.  T is a multiple of 16, so a contiguous cache and
// pages of 16 tokens or more hold a step in consecutive rows: its first row is enough then;
// smaller pages place a row a lane (key lane % 16).
struct Step {
  uint32_t row;   // fewer than 2^32 rows fit a GPU
  uint32_t live;
};
__device__ __forceinline__ Step place_step(const DenseArgs &a, int b, int h, int T, int lo, int hi, int lane) {
  Step s;
  if (!a.pages || a.page_shift >= 4) {
    const int64_t r = cache_row(a, b, h, T);
    s.live = 0xffffu;
    if (T < lo) s.live &= lo - T >= kStep ? 0u : 0xffffu << (lo - T);
    if (T + kStep > hi) s.live &= hi <= T ? 0u : 0xffffu >> (T + kStep - hi);
    if (r < 0 && s.live) {
      if (lane == 0) atomicOr(&a.hdr->err, kErrIndex);
      s.live = 0;
    }
    s.row = r < 0 ? 0u : (uint32_t)r;
    return s;
  }
  const int t = T + (lane & 15);
  bool on = t >= lo && t < hi;
  s.row = 0;
  if (on) {
    const int64_t r = cache_row(a, b, h, t);
    if (r < 0) {
      on = false;
      atomicOr(&a.hdr->err, kErrIndex);
    } else {
      s.row = (uint32_t)r;
    }
  }
  s.live = __ballot_sync(0xffffffffu, on) & 0xffffu;
  return s;
}
// A lane copies 16 bytes of keys 2 i + lane / 16; `swz` is where those of key lane / 16 go.
__device__ __forceinline__ void load_step(const DenseArgs &a, const uint16_t *cache, const Step &s, uint32_t dst,
                                          int lane) {
  const int c = lane & 15, k0 = lane >> 4;
  const uint32_t swz = dst + k0 * kRowBytes;
  const uint32_t col = (uint32_t)((c ^ k0) << 4);  // piece c of key k goes to place c ^ (k % 8)
  if (!a.pages || a.page_shift >= 4) {
    const char *src = reinterpret_cast<const char *>(cache) + ((int64_t)s.row + k0) * kRowBytes + c * 16;
    if (s.live == 0xffffu) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(swz + i * 2 * kRowBytes + (col ^ ((2 * i & 6) << 4))),
                     "l"(src + i * 2 * kRowBytes)
                     : "memory");
    } else {  // rows outside the range are not touched: their source is the first row of the cache
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool on = (s.live >> (2 * i + k0)) & 1u;
        cp_async16(swz + i * 2 * kRowBytes + (col ^ ((2 * i & 6) << 4)),
                   on ? src + i * 2 * kRowBytes : reinterpret_cast<const char *>(cache), on);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t r = __shfl_sync(0xffffffffu, s.row, 2 * i + k0);
      cp_async16(swz + i * 2 * kRowBytes + (col ^ ((2 * i & 6) << 4)), cache + (int64_t)r * kD + c * 8,
                 (s.live >> (2 * i + k0)) & 1u);
    }
  }
  cp_async_commit();
}

// The rotation table into shared memory (queued; the caller commits and waits).
__device__ __forceinline__ void load_table(const DenseArgs &a, unsigned char *table, bool scaled, int tid) {
  const uint32_t dst = smem_u32(table);
#pragma unroll
  for (int i = 0; i < kSpan * kHalf / 2 / kThreads; ++i) {
    const int e = tid + i * kThreads;
    const int r = e / (kHalf / 2), piece = e % (kHalf / 2);
    cp_async16(dst + r * kTableStride + ((piece ^ ((r & 1) << 2)) << 4), ws_table(a.hdr, scaled) + 2 * e, true);
  }
}

// 8 query rows turned by a further `delta` positions, as the B operands of the score product: each
// value as two parts (q rounded, and what that leaves, rounded).
template <int NR, bool EX>
__device__ __forceinline__ void turn_queries(const DenseArgs &a, const float (*q)[kQStride], int delta, float4 *ang,
                                             uint32_t (&qh)[NR][16], uint32_t (&ql)[NR][16], int lane) {
  const uint64_t *f = ws_freq(a.hdr);
  __syncwarp();
  const float2 r0 = rotation(delta, __ldg(f + 2 * lane)), r1 = rotation(delta, __ldg(f + 2 * lane + 1));
  ang[lane] = make_float4(r0.x, r1.x, r0.y, r1.y);
  __syncwarp();
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int ch = 0; ch < 8; ++ch) {
    const float4 w = ang[ch * 4 + c];
    const F2 cs = f2(w.x, w.y), sn = f2(w.z, w.w);
#pragma unroll
    for (int nt = 0; nt < NR; ++nt) {
      const float2 x = *reinterpret_cast<const float2 *>(&q[nt * 8 + r][ch * 8 + 2 * c]);
      const float2 y = *reinterpret_cast<const float2 *>(&q[nt * 8 + r][ch * 8 + 2 * c + kHalf]);
      const F2 X = f2(x.x, x.y), Y = f2(y.x, y.y);
      split_pair<EX>(f2_fma(Y, f2_neg(sn), f2_mul(X, cs)), qh[nt][ch], ql[nt][ch]);
      split_pair<EX>(f2_fma(X, sn, f2_mul(Y, cs)), qh[nt][ch + 8], ql[nt][ch + 8]);
    }
  }
}

// Scores of a step's 16 keys (rows of the product) with the tile's query rows (columns): the keys
// are rotated by their place in the span.  Both operands are two parts, hi * hi + lo * hi +
// hi * lo: what is dropped is below 2^-16 of the product of the magnitudes with bf16 parts, below
// 2^-22 with fp16 ones (EX: fp32 outputs and weights).  A rotated element beyond fp16's range makes
// the score infinite, and that is made NaN: such a row goes to careful_row.
// The tensor cores cut sums off: with EX they are joined by rounded adds every 32 dimensions.
// s[nt]: keys lane/4 (first two) and lane/4 + 8, query rows nt * 8 + 2 (lane % 4) and one more.
template <int NR, bool EX>
__device__ __forceinline__ void score_step(const unsigned char *table, uint32_t sk, int T, const uint32_t (&qh)[NR][16],
                                           const uint32_t (&ql)[NR][16], float (&s)[NR][4], int lane) {
  const int lrow = lane & 15, lch = lane >> 4;  // ldmatrix: lanes 0-15 the first 8 dimensions' rows, 16-31 the next 8
  const uint32_t lbase = sk + lrow * kRowBytes;
  const unsigned char *tr = table + ((T & (kSpan - 1)) + (lane >> 2)) * kTableStride + (lane & 3) * 16;
  const int odd = ((lane >> 2) & 1) << 6;  // 4 pieces (T is even)
  float lo[NR][4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    uint32_t x[4], y[4];  // [key half][chunk of the k-step]: registers 0: (0, 0), 1: (1, 0), 2: (0, 1), 3: (1, 1)
    ldsm4(lbase + (((2 * ks + lch) ^ (lrow & 7)) << 4), x[0], x[1], x[2], x[3]);
    ldsm4(lbase + (((2 * ks + 8 + lch) ^ (lrow & 7)) << 4), y[0], y[1], y[2], y[3]);
    uint32_t uh[4], ul[4], vh[4], vl[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 w = *reinterpret_cast<const float4 *>(tr + (i & 1) * 8 * kTableStride + (((2 * ks + (i >> 1)) * 64) ^ odd));
      const F2 cs = f2(w.x, w.y), sn = f2(w.z, w.w), X = f2_bf16(x[i]), Y = f2_bf16(y[i]), minus = f2(-1.f, -1.f);
      const F2 U = f2_fma(f2_mul(Y, sn), minus, f2_mul(X, cs)), V = f2_fma(X, sn, f2_mul(Y, cs));
      if (EX) {
        cut_pair(U, uh[i], ul[i]);
        cut_pair(V, vh[i], vl[i]);
      } else {
        split_pair<false>(U, uh[i], ul[i]);
        split_pair<false>(V, vh[i], vl[i]);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NR; ++nt) {
      float t[4];  // EX: these dimensions, small terms first
      if (EX) {
        mma16816_half_zero(t, uh, ql[nt][2 * ks], ql[nt][2 * ks + 1]);
        mma16816_half(t, vh, ql[nt][2 * ks + 8], ql[nt][2 * ks + 9]);
        mma16816_half(t, ul, qh[nt][2 * ks], qh[nt][2 * ks + 1]);
        mma16816_half(t, vl, qh[nt][2 * ks + 8], qh[nt][2 * ks + 9]);
        mma16816_half(t, uh, qh[nt][2 * ks], qh[nt][2 * ks + 1]);
        mma16816_half(t, vh, qh[nt][2 * ks + 8], qh[nt][2 * ks + 9]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = ks == 0 ? t[i] : s[nt][i] + t[i];
      } else {
        if (ks == 0) {
          mma16816_zero(s[nt], uh, qh[nt][0], qh[nt][1]);
          mma16816_zero(lo[nt], uh, ql[nt][0], ql[nt][1]);
        } else {
          mma16816(s[nt], uh, qh[nt][2 * ks], qh[nt][2 * ks + 1]);
          mma16816(lo[nt], uh, ql[nt][2 * ks], ql[nt][2 * ks + 1]);
        }
        mma16816(s[nt], vh, qh[nt][2 * ks + 8], qh[nt][2 * ks + 9]);
        mma16816(lo[nt], vh, ql[nt][2 * ks + 8], ql[nt][2 * ks + 9]);
        mma16816(lo[nt], ul, qh[nt][2 * ks], qh[nt][2 * ks + 1]);
        mma16816(lo[nt], vl, qh[nt][2 * ks + 8], qh[nt][2 * ks + 9]);
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NR; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i)  // EX: an infinity becomes NaN
      s[nt][i] = EX ? __fmaf_rn(s[nt][i], 1.f / (kKeyScale * kQueryScale), s[nt][i] * 0.f) : s[nt][i] + lo[nt][i];
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t ld_shared32(uint32_t addr) {
  uint32_t u;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(addr) : "memory");
  return u;
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
  __device__ __forceinline__ bool sink(int st) const { return st < n1; }
  __device__ __forceinline__ int token(int st) const { return (st < n1 ? st : first + st - n1) * kStep; }
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

// `total` steps dealt out evenly to as many of the grid's blocks as are worth starting.
struct Dealt {
  int total, blocks;
  __device__ __forceinline__ explicit Dealt(int t) : total(t), blocks(min((int)gridDim.x, max(1, t / kDealtSteps))) {}
  __device__ __forceinline__ int begin(int block) const { return (int)((int64_t)total * block / blocks); }
  __device__ __forceinline__ int holder(int step) const {  // the block that holds a step
    int block = (int)((int64_t)step * blocks / total);
    while (begin(block + 1) <= step) ++block;
    while (begin(block) > step) --block;
    return block;
  }
};

// One row over the steps [begin, stop) of its tile by one warp, in fp32: dimensions 4 lane .. 4 lane
// + 3 of the weighted sum of values (without PV: the scores, written), the weights' sum and the
// maximum they are relative to.  Every value is weighed by itself: one that the row does not see is
// not touched, and an infinity does not meet the zero that a weight's second part may be.
template <int R, bool PV, bool EX>
__device__ void careful_row(const DenseArgs &a, RowsSmem<R> &sm, const Range &rg, int row, int b, int h, int p_max,
                            int base_sink, int bh, float (&acc)[4], float &m, float &sum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, p = sm.pos[row];
  float *const turned = reinterpret_cast<float *>(sm.ang[warp]);
  const uint64_t *f = ws_freq(a.hdr);
  float top = -INFINITY;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int st = sm.range[0]; st < sm.range[1]; ++st) {
    const bool sink = rg.sink(st);
    const int T = rg.token(st), delta = (sink ? base_sink : p_max) - a.back - (T & ~(kSpan - 1));
    __syncwarp();
#pragma unroll
    for (int i = lane; i < kHalf; i += 32) {  // the row turned to the span, as the keys' table is
      const float2 w = rotation(delta, __ldg(f + i));
      const float x = sm.q[sink][row][i] * (EX ? 1.f / kQueryScale : 1.f),
                  y = sm.q[sink][row][i + kHalf] * (EX ? 1.f / kQueryScale : 1.f);
      turned[i] = x * w.x - y * w.y;
      turned[i + kHalf] = y * w.x + x * w.y;
    }
    __syncwarp();
    // two lanes a key, half of the dimensions each
    const int t = T + (lane & 15);
    const bool in = sink ? t < min(p, rg.hi1) : t >= window_first(a, p) && t < p;
    const int64_t r = in ? cache_row(a, b, h, t) : -1;
    float s = 0.f;
    if (r >= 0) {
      const uint32_t *key = reinterpret_cast<const uint32_t *>(a.k + r * kD);
      const unsigned char *tr = sm.table + (t & (kSpan - 1)) * kTableStride;
#pragma unroll 4
      for (int i = (lane >> 4) * 16; i < (lane >> 4) * 16 + 16; ++i) {
        float4 w = *reinterpret_cast<const float4 *>(tr + ((i ^ ((t & 1) << 2)) << 4));
        if (EX) w.x *= 1.f / kKeyScale, w.y *= 1.f / kKeyScale, w.z *= 1.f / kKeyScale, w.w *= 1.f / kKeyScale;
        const uint32_t x = __ldg(key + i), y = __ldg(key + i + 32);
        s += turned[2 * i] * (bf16_lo(x) * w.x - bf16_lo(y) * w.z) + turned[2 * i + 1] * (bf16_hi(x) * w.y - bf16_hi(y) * w.w);
        s += turned[2 * i + kHalf] * (bf16_lo(y) * w.x + bf16_lo(x) * w.z) +
             turned[2 * i + 1 + kHalf] * (bf16_hi(y) * w.y + bf16_hi(x) * w.w);
      }
    }
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if (r < 0) s = -INFINITY;
    if (!PV && a.scores && row < a.score_stride && lane < kStep)
      a.scores[((int64_t)(bh - a.bh0) * a.score_pitch + t) * a.score_stride + row] = s;
    float x = s;
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    if (x > top) {
      const float w = top == -INFINITY ? 0.f : exp2_approx(top - x);
      top = x;
      sum *= w;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] *= w;
    }
    const float weight = exp2_approx(s - ((top == -INFINITY ? 0.f : top) + kRowsLift));
    const uint32_t seen = __ballot_sync(0xffffffffu, r >= 0);
#pragma unroll 4
    for (int key = 0; key < kStep; ++key) {
      const float w = __shfl_sync(0xffffffffu, weight, key);
      const int64_t v_row = __shfl_sync(0xffffffffu, r, key);
      if (!((seen >> key) & 1u)) continue;
      sum += w;
      if (!PV) continue;
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(a.v + v_row * kD) + lane);
      acc[0] += w * bf16_lo(v.x), acc[1] += w * bf16_hi(v.x), acc[2] += w * bf16_lo(v.y), acc[3] += w * bf16_hi(v.y);
    }
  }
  m = top == -INFINITY ? top : top + kRowsLift;
}

// One tile of 8 NR query rows (queries x heads of a KV group) against one block's share of the keys
// they see.  Each warp walks its own steps of 16 keys with an online softmax, its keys and values
// fetched one step ahead with cp.async into memory of its own, so warps never wait for one another
// until their (max, sum, output) are joined at the end; the last block of a tile joins the blocks.
// EX: fp32's accuracy (fp32 outputs, weights).  Against two bf16 parts of everything the error of 16
// queries over 4096 tokens fell from 6e-6 to 3.2e-7 (plain fp32 arithmetic: 7.8e-7) at 19.3 us instead
// of 18.4, of the weights of one step over 4 x 65536 tokens from 4.9e-6 to 2.5e-7 at 162 instead of 158.
// Scores, probabilities and outputs are products of the tensor cores with keys (scores) and
// dimensions (outputs) as rows and the query rows as columns, so that one to eight rows - a decode
// step - fill an instruction.  DRAM and issue bound it together: a key of 512 bytes costs about 56
// issue slots of the ~88 its SM has meanwhile (2 x 131072 tokens, 8 KV heads, G = 4: 178 us, 74 % of
// the DRAM peak and 63 % of the slots).
// MODE 0: the output.  MODE 1: the rows' (maximum, 1 / sum) to `lse`.  MODE 2: the output of the tiles
// that the chunk kernel marked in `redo`, if any.
template <int NR, int MODE, bool DEAL, bool EX>
__global__ void __launch_bounds__(kThreads, NR == 1 ? 2 : 1)
    dense_rows_kernel(DenseArgs a, int items, float *lse, uint32_t *redo, int chunk_tiles) {
  constexpr int R = 8 * NR;
  constexpr bool PV = MODE != 1;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  RowsSmem<R> &sm = *reinterpret_cast<RowsSmem<R> *>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gs = a.group_shift, G = 1 << gs, hq = a.hkv << gs;
  const float qscale = EX ? a.qscale * kQueryScale : a.qscale;
  const WsHeader head = *a.hdr;  // checked once the first loads are on their way
  if (MODE == 2) {  // nearly always nothing is marked
    uint32_t any = 0;
    for (int i = tid; i < kMaxShared / 4; i += kThreads) {
      const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(redo) + i);
      any |= u.x | u.y | u.z | u.w;
    }
    if (!__syncthreads_or(any != 0)) return;
  }
  const int r = lane >> 2, c = lane & 3;
  const uint32_t sk = smem_u32(sm.stage[warp][0]), sv = sk + kStepBytes;

  // Sequences of unequal length: their steps (a head's one after the other) are dealt out evenly
  // to the blocks instead of an equal number of blocks a head.
  int at = 0, end = 0;
  if (DEAL) {
    int steps = 0;
    if (tid < a.batch) {
      const int len = dense_length(a, tid, blockIdx.x == 0);
      steps = max(1, tile_range(a, dense_position(a, len, 0), dense_position(a, len, a.nq - 1)).total);
    }
    int incl = steps * a.hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int *const warp_sum = reinterpret_cast<int *>(sm.ang);  // (free until the first turn)
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += warp_sum[w];
    sm.dealt[tid + 1] = incl;
    if (tid == 0) sm.dealt[0] = 0;
    __syncthreads();
    const Dealt d(sm.dealt[a.batch]);
    if ((int)blockIdx.x >= d.blocks) return;
    at = d.begin(blockIdx.x);
    end = d.begin(blockIdx.x + 1);
  }

  bool table = false;
  for (int work = blockIdx.x; DEAL ? at < end : work < items * a.nsplit; work += gridDim.x) {
  int item, split = 0, tile, bh, b, h;
  if (DEAL) {
    int lo = 0, hi = a.batch - 1;  // the sequence that holds step `at`
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (sm.dealt[mid] <= at) lo = mid; else hi = mid - 1;
    }
    b = lo;
    h = (at - sm.dealt[b]) / ((sm.dealt[b + 1] - sm.dealt[b]) / a.hkv);
    item = bh = b * a.hkv + h;
    tile = 0;
  } else {
    item = work / a.nsplit;
    split = work % a.nsplit;
    tile = item % a.tiles;
    bh = a.bh0 + item / a.tiles;
    b = bh / a.hkv;
    h = bh % a.hkv;
  }
  const int q0 = tile * (R >> gs), nq = min(R >> gs, a.nq - q0);  // the tile's queries
  if (MODE == 2 && !redo[redo_slot(bh, chunk_tiles, q0 / (256 >> gs))]) continue;
  const int len = dense_length(a, b, !DEAL && tid == 0 && tile == 0 && split == 0 && h == 0);
  const int p_min = dense_position(a, len, q0), p_max = dense_position(a, len, q0 + nq - 1);
  const Range rg = tile_range(a, p_min, p_max);
  const int base_sink = sink_position(a, p_max);

  int begin, stop;  // the block's steps of the tile
  if (DEAL) {
    const int steps = (sm.dealt[b + 1] - sm.dealt[b]) / a.hkv;
    begin = at - (sm.dealt[b] + h * steps);
    stop = min(steps, begin + end - at);
    at += stop - begin;
    stop = min(stop, rg.total);  // (a tile without keys counts as one step)
  } else {
    begin = (int)((int64_t)rg.total * split / a.nsplit);
    stop = (int)((int64_t)rg.total * (split + 1) / a.nsplit);
  }
  if (tid == 0) sm.range[0] = begin, sm.range[1] = stop;
  // this warp's steps; the first loads are on their way while the query rows are turned
  const int st0 = begin + (int)((int64_t)(stop - begin) * warp / kWarps),
            st1 = begin + (int)((int64_t)(stop - begin) * (warp + 1) / kWarps);
  auto place = [&](int st) {
    const bool sink = rg.sink(st);
    return place_step(a, b, h, rg.token(st), sink ? 0 : rg.lo2, sink ? rg.hi1 : rg.hi2, lane);
  };
  // MODE 1 has no values: its keys alternate between the two halves of the stage
  Step cur = {0, 0u}, next = {0, 0u};
  if (!table) load_table(a, sm.table, EX, tid);  // with the first step's keys
  table = true;
  if (st0 < st1) {
    cur = place(st0);
    load_step(a, a.k, cur, PV || !(st0 & 1) ? sk : sv, lane);
  } else {
    cp_async_commit();
  }
  if (st0 + (PV ? 0 : 1) < st1) {
    if (!PV) next = place(st0 + 1);
    load_step(a, PV ? a.v : a.k, PV ? cur : next, PV || !(st0 & 1) ? sv : sk, lane);
  } else {
    cp_async_commit();
  }
  if (tid < R) sm.pos[tid] = (tid >> gs) < nq ? dense_position(a, len, q0 + (tid >> gs)) : 0;
  for (int e = tid; e < R * kHalf * 2; e += kThreads) {  // query rows, turned to the tile's last position
    const int i = e % kHalf, row = (e / kHalf) % R, sink = e / (kHalf * R);
    if (sink && !rg.n1) break;
    float x = 0.f, y = 0.f;
    if ((row >> gs) < nq) {
      const uint16_t *src = a.q + (((int64_t)b * a.nq + q0 + (row >> gs)) * hq + h * G + (row & (G - 1))) * kD + i;
      x = __uint_as_float((uint32_t)src[0] << 16) * qscale;
      y = __uint_as_float((uint32_t)src[kHalf] << 16) * qscale;
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
  cp_async_wait<1>();  // the table
  __syncthreads();
  if (head.magic != kDenseMagic || head.rope_base != a.rope_base) {
    cp_async_wait<0>();
    if (tid == 0) atomicOr(&a.hdr->err, kErrWs);
    return;
  }

  // this thread's query rows: nt * 8 + 2 c + i
  float m[NR][2], l[NR][2], o[PV ? NR : 1][8][4];
#pragma unroll
  for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[nt][i] = -INFINITY;
      l[nt][i] = 0.f;
    }
    if (PV) {
#pragma unroll
      for (int d = 0; d < 8; ++d) o[nt][d][0] = o[nt][d][1] = o[nt][d][2] = o[nt][d][3] = 0.f;
    }
  }
  uint32_t qh[NR][16], ql[NR][16];
  int turned = -1;  // the span the query rows are turned for (sinks: odd)

  for (int st = st0; st < st1; ++st) {
    const bool sink = rg.sink(st);
    const int T = rg.token(st);
    const int span = (T / kSpan) * 2 + (sink ? 1 : 0);
    if (span != turned) {
      turned = span;
      turn_queries<NR, EX>(a, sm.q[sink], (sink ? base_sink : p_max) - a.back - (T & ~(kSpan - 1)), sm.ang[warp], qh, ql, lane);
    }
    cp_async_wait<1>();
    __syncwarp();
    float s[NR][4];
    const uint32_t keys = PV || !(st & 1) ? sk : sv;
    score_step<NR, EX>(sm.table, keys, T, qh, ql, s, lane);
    __syncwarp();  // the keys' memory is free
    const uint32_t live = cur.live;
    constexpr int kAhead = PV ? 1 : 2;
    if (!PV) cur = next;
    if (st + kAhead < st1) {
      next = place(st + kAhead);
      load_step(a, a.k, next, keys, lane);
    } else {
      cp_async_commit();
    }
    // every row sees every key of the step unless it meets an end of some row's range
    const bool whole = live == 0xffffu && (sink ? T + kStep <= min(p_min, rg.hi1)
                                                : T + kStep <= p_min && T >= window_first(a, p_max));
    bool seen[NR][4];
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) seen[nt][i] = true;
    if (!whole) {
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = r + (i & 2) * 4, t = T + key, p = sm.pos[nt * 8 + 2 * c + (i & 1)];
          const int lo = sink ? 0 : window_first(a, p), hi = sink ? min(p, rg.hi1) : p;
          seen[nt][i] = ((live >> key) & 1u) && t >= lo && t < hi;
          if (!seen[nt][i]) s[nt][i] = -INFINITY;
        }
    }
    if (MODE == 1 && a.scores && 2 * c < a.score_stride) {  // (only with 8 rows or fewer: one tile a head)
      float *dst = a.scores + ((int64_t)(bh - a.bh0) * a.score_pitch + T + r) * a.score_stride + 2 * c;
      *reinterpret_cast<float2 *>(dst) = make_float2(s[0][0], s[0][1]);
      *reinterpret_cast<float2 *>(dst + 8 * a.score_stride) = make_float2(s[0][2], s[0][3]);
    }
    // Weights from the maximum so far: weights, sums and outputs hold numbers up to 2^127 with
    // the same relative precision (a row's output beyond kRowsLarge is computed again below).  Only
    // a row whose maximum has grown by more than 2^64 (or that has none yet) takes a new one.
    bool up = false;
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) up |= s[nt][i] > m[nt][i & 1] + kRowsRescale;
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = fmaxf(s[nt][i], s[nt][2 + i]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          if (x > m[nt][i] + kRowsRescale) {
            const float f = m[nt][i] == -INFINITY ? 0.f : exp2_approx(m[nt][i] - x);
            m[nt][i] = x;
            l[nt][i] *= f;
            if (PV) {
#pragma unroll
              for (int d = 0; d < 8; ++d) {
                o[nt][d][i] *= f;
                o[nt][d][2 + i] *= f;
              }
            }
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float mm = m[nt][i & 1];
        s[nt][i] = exp2_approx(s[nt][i] - (mm == -INFINITY ? 0.f : mm));
        l[nt][i & 1] += s[nt][i];
      }
    if (PV) {
      cp_async_wait<1>();
      __syncwarp();
      // A row that does not see a key must not touch its value: a product with a zero weight
      // would carry an infinity or NaN over.  In steps that hide a key from some row, values
      // that are not finite go to the rows that see them one by one and are zeros in the product.
      if (!whole) {
        bool odd = false;
        for (int i = lane; i < kStepBytes / 4; i += 32) odd |= not_finite(ld_shared32(sv + i * 4));
        if (__any_sync(0xffffffffu, odd)) {
          for (int key = 0; key < kStep; ++key) {
#pragma unroll
            for (int nt = 0; nt < NR; ++nt) {
              // the weights of this key and this thread's rows sit in the lane of key % 8
              const int src = (key & 7) * 4 + c;
              const float w0 = __shfl_sync(0xffffffffu, key & 8 ? s[nt][2] : s[nt][0], src);
              const float w1 = __shfl_sync(0xffffffffu, key & 8 ? s[nt][3] : s[nt][1], src);
              const bool v0 = __shfl_sync(0xffffffffu, (int)(key & 8 ? seen[nt][2] : seen[nt][0]), src);
              const bool v1 = __shfl_sync(0xffffffffu, (int)(key & 8 ? seen[nt][3] : seen[nt][1]), src);
#pragma unroll
              for (int d = 0; d < 8; ++d)
#pragma unroll
                for (int k = 0; k < 2; ++k) {  // dimension 16 d + 8 k + r
                  const uint32_t u = ld_shared32(sv + key * kRowBytes + (((2 * d + k) ^ (key & 7)) << 4) + (r >> 1) * 4);
                  const float v = (r & 1) ? bf16_hi(u) : bf16_lo(u);
                  if (!isfinite(v)) {
                    if (v0) o[PV ? nt : 0][d][2 * k] += w0 * v;
                    if (v1) o[PV ? nt : 0][d][2 * k + 1] += w1 * v;
                  }
                }
            }
          }
          __syncwarp();
          for (int i = lane; i < kStepBytes / 4; i += 32) {
            uint32_t u = ld_shared32(sv + i * 4);
            if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
            if ((u & 0x7f800000u) == 0x7f800000u) u &= 0xffffu;
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(sv + i * 4), "r"(u) : "memory");
          }
          __syncwarp();
        }
      }
      uint32_t ph[NR][2], pl[NR][2], pm[NR][2];  // the weights' parts with keys along the k of the product
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t hi = cvt_bf16x2(s[nt][2 * k], s[nt][2 * k + 1]);
          ph[nt][k] = transpose8x8(hi);
          const uint32_t lo = residue_bf16x2(s[nt][2 * k], s[nt][2 * k + 1], hi);
          pl[nt][k] = transpose8x8(lo);
          if (EX)
            pm[nt][k] = transpose8x8(residue_bf16x2(s[nt][2 * k] - bf16_lo(hi), s[nt][2 * k + 1] - bf16_hi(hi), lo));
        }
      const int key = (lane & 7) + ((lane >> 4) << 3), dch = (lane >> 3) & 1;
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        uint32_t v[4];
        ldsm4_trans(sv + key * kRowBytes + (((2 * d + dch) ^ (key & 7)) << 4), v[0], v[1], v[2], v[3]);
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
          // The tensor cores cut their fp32 sums off instead of rounding them: over a million
          // keys an output summed there alone came out 5e-5 short.  A step's 16 keys are
          // summed there, the steps in fp32 adds that round.
          float t[4];
          if (EX) {
            mma16816_zero(t, v, pm[nt][0], pm[nt][1]);
            mma16816(t, v, pl[nt][0], pl[nt][1]);
          } else {
            mma16816_zero(t, v, pl[nt][0], pl[nt][1]);
          }
          mma16816(t, v, ph[nt][0], ph[nt][1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[PV ? nt : 0][d][i] += t[i];
        }
      }
      __syncwarp();  // the values' memory is free
      if (st + 1 < st1)
        load_step(a, a.v, next, sv, lane);
      else
        cp_async_commit();
    }
    if (PV) cur = next;
  }
  cp_async_wait<0>();

  // join the warps: their outputs in the stage memory
#pragma unroll
  for (int nt = 0; nt < NR; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], d);
      if (r == 0) {
        sm.m[warp][nt * 8 + 2 * c + i] = m[nt][i];
        sm.l[warp][nt * 8 + 2 * c + i] = l[nt][i];
      }
    }
  __syncthreads();
  float *const wo = reinterpret_cast<float *>(sm.stage);  // [warp][R][kOStride], half the warps at a time
  static_assert(sizeof(float) * (kWarps / NR) * R * kOStride <= sizeof(sm.stage), "the outputs fit the stages");
  constexpr int kPer = kD * R / kThreads;  // dimensions of a row that a thread joins
  const int row = tid / (kD / kPer), d0 = (tid % (kD / kPer)) * kPer;
  float mx = -INFINITY, sum = 0.f, acc[kPer] = {};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm.m[w][row]);
#pragma unroll 1
  for (int w0 = 0; w0 < kWarps; w0 += kWarps / NR) {
    if (PV) {
      if (w0 > 0) __syncthreads();
      if (warp >= w0 && warp < w0 + kWarps / NR) {
        float *dst = wo + (warp - w0) * R * kOStride + r;
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int d = 0; d < 8; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[(nt * 8 + 2 * c + (i & 1)) * kOStride + d * 16 + (i >> 1) * 8] = o[PV ? nt : 0][d][i];
      }
      __syncthreads();
    }
#pragma unroll
    for (int w = 0; w < kWarps / NR; ++w) {
      const float mw = sm.m[w0 + w][row];
      if (mw == -INFINITY) {
        sum += sm.l[w0 + w][row];  // 0, or NaN: every score was
        continue;
      }
      const float f = exp2_approx(mw - mx);
      sum += f * sm.l[w0 + w][row];
      if (PV) {
#pragma unroll
        for (int i = 0; i < kPer; i += 4) {
          const float4 u = *reinterpret_cast<const float4 *>(wo + (w * R + row) * kOStride + d0 + i);
          acc[i] += f * u.x, acc[i + 1] += f * u.y, acc[i + 2] += f * u.z, acc[i + 3] += f * u.w;
        }
      }
    }
  }
  {  // (a row's threads are lanes of one warp)
    float size = sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) size += PV ? fabsf(acc[i]) : 0.f;
    const uint32_t large = __ballot_sync(0xffffffffu, !(size <= kRowsLarge));
    if (large) {
#pragma unroll 1
      for (int j = 0; j < NR; ++j) {
        if (!(large >> (j * (32 / NR)) << (32 - 32 / NR))) continue;
        float x[4], xm, xsum;
        careful_row<R, PV, EX>(a, sm, rg, warp * NR + j, b, h, p_max, base_sink, bh, x, xm, xsum);
        const bool mine = row == warp * NR + j;
        if (mine) mx = xm, sum = xsum;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const float y = __shfl_sync(0xffffffffu, x[i & 3], (d0 + i) / 4);
          if (mine) acc[i] = y;
        }
      }
    }
  }
  bool write = true;
  // the blocks that share the tile, and where the part of the j-th of them is
  int sharing = a.nsplit, first_block = 0, item_at = 0;
  const Dealt dealt(DEAL ? sm.dealt[a.batch] : 1);
  if (DEAL) {
    const int steps = (sm.dealt[b + 1] - sm.dealt[b]) / a.hkv;
    item_at = sm.dealt[b] + h * steps;
    first_block = dealt.holder(item_at);
    sharing = dealt.holder(item_at + steps - 1) - first_block + 1;
  }
  auto part_at = [&](int j) {  // dealt out: in a block's first segment or its last
    const int64_t slot = DEAL ? (int64_t)(first_block + j) * 2 + (dealt.begin(first_block + j) >= item_at ? 0 : 1)
                              : (int64_t)item * a.nsplit + j;
    return ws_part(a.hdr) + slot * (R * kPartRow);
  };
  if (sharing > 1) {  // leave this block's part; the last block of the tile joins them in order
    float *part_row =
        part_at(DEAL ? (int)blockIdx.x - first_block : split) + row * kPartRow;
    if (d0 == 0) *reinterpret_cast<float2 *>(part_row) = make_float2(mx, sum);
    if (PV) {
#pragma unroll
      for (int i = 0; i < kPer; i += 4)
        *reinterpret_cast<float4 *>(part_row + 4 + d0 + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      const int done = atomicAdd(ws_count(a.hdr) + item, 1);
      sm.last = done == sharing - 1;
      if (sm.last) ws_count(a.hdr)[item] = 0;  // for the next call
    }
    __syncthreads();
    write = sm.last;
    if (write) {
      __threadfence();
      mx = -INFINITY;
      sum = 0.f;
#pragma unroll 4
      for (int j = 0; j < sharing; ++j) mx = fmaxf(mx, __ldcg(part_at(j) + row * kPartRow));
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll 8
      for (int j = 0; j < sharing; ++j) {
        const float *p = part_at(j) + row * kPartRow;
        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p));
        const float f = ml.x == -INFINITY ? 0.f : exp2_approx(ml.x - mx);
        float4 u[kPer / 4];
        if (PV) {
#pragma unroll
          for (int i = 0; i < kPer / 4; ++i) u[i] = __ldcg(reinterpret_cast<const float4 *>(p + 4 + d0) + i);
        }
        if (ml.x == -INFINITY) {
          sum += ml.y;
          continue;
        }
        sum += f * ml.y;
        if (PV) {
#pragma unroll
          for (int i = 0; i < kPer / 4; ++i) {
            acc[4 * i] += f * u[i].x, acc[4 * i + 1] += f * u[i].y;
            acc[4 * i + 2] += f * u[i].z, acc[4 * i + 3] += f * u[i].w;
          }
        }
      }
    }
  }
  if (write && (row >> gs) < nq) {
    const int64_t out_row = ((int64_t)b * a.nq + q0 + (row >> gs)) * hq + h * G + (row & (G - 1));
    if (!PV) {
      // a key's weight is exp2(score - maximum) / sum: no logarithm of the sum, whose rounding would
      // weigh on every weight of the row
      if (d0 == 0)
        reinterpret_cast<float2 *>(lse)[out_row] = sum == 0.f ? make_float2(0.f, 0.f) : make_float2(mx, 1.f / sum);
    } else {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int i = 0; i < kPer; i += 4) {
        const float x0 = acc[i] * inv, x1 = acc[i + 1] * inv, x2 = acc[i + 2] * inv, x3 = acc[i + 3] * inv;
        if (a.out_fp32)
          *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + out_row * kD + d0 + i) =
              make_float4(x0, x1, x2, x3);
        else
          *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(a.out) + out_row * kD + d0 + i) =
              make_uint2(cvt_bf16x2(x0, x1), cvt_bf16x2(x2, x3));
      }
    }
  }
  __syncthreads();  // the shared memory is free for the next tile
  }
  if (MODE == 2) {  // the last block to finish clears the marks
    __syncthreads();
    if (tid == 0) sm.last = atomicAdd(ws_count(a.hdr) + kMaxShared, 1) == (int)gridDim.x - 1;
    __syncthreads();
    if (sm.last) {
      for (int i = tid; i < kMaxShared; i += kThreads) redo[i] = 0u;
      if (tid == 0) ws_count(a.hdr)[kMaxShared] = 0;
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
    float *w = reinterpret_cast<float *>(ws + kDenseTable) + (r * kHalf + (i & ~1)) * 2 + (i & 1);
    w[0] = (float)c;  // two frequencies: cos, cos', sin, sin'
    w[2] = (float)s;
    w[kDenseTableBytes / sizeof(float)] = (float)(c * kKeyScale);
    w[kDenseTableBytes / sizeof(float) + 2] = (float)(s * kKeyScale);
  }
  if (r == 0) {
    const double turns = theta / (2.0 * 3.14159265358979323846);
    reinterpret_cast<uint64_t *>(ws + kDenseFreq)[i] = (uint64_t)((turns - floor(turns)) * 18446744073709551616.0);
  }
  if (idx < kMaxShared) {
    reinterpret_cast<int32_t *>(ws + kDenseCount)[idx] = 0;
    if (idx == 0) reinterpret_cast<int32_t *>(ws + kDenseCount)[kMaxShared] = 0;
    reinterpret_cast<uint32_t *>(ws + kDenseRedo)[idx] = 0u;
    reinterpret_cast<int32_t *>(ws + kDenseBeyond)[idx] = 0;
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

// Blocks of the rows kernel an SM holds.
constexpr int blocks_per_sm(int nr) { return nr == 1 ? 2 : 1; }

template <int NR, int MODE, bool DEAL, bool EX>
int run_rows(const DenseArgs &a, int64_t items, int64_t grid, float *lse, uint32_t *redo, int chunk_tiles, void *stream) {
  const int rc = opt_in(dense_rows_kernel<NR, MODE, DEAL, EX>, sizeof(RowsSmem<8 * NR>));
  if (rc) return rc;
  dense_rows_kernel<NR, MODE, DEAL, EX><<<(unsigned)grid, kThreads, sizeof(RowsSmem<8 * NR>), (cudaStream_t)stream>>>(
      a, (int)items, lse, redo, chunk_tiles);
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

// Blocks a tile's keys are shared among: enough for every place an SM has for a block, in waves
// as full as possible, as long as a block keeps kMinKeys keys.  (Fewer join more than they save:
// 8 heads of 8192 tokens took 21.4, 18.9 and 16.9 us with at least 128, 256 and 512 keys, 8 heads of 1000
// took 13.1, 14.0 and 20.5, one head of 4096 with 64 rows 21.9, 16.6 and 18.9.)
static int pick_split(int64_t items, int64_t max_keys, int places, int rows) {
  constexpr int64_t kMinKeys = 256;
  if (items > kMaxShared) return 1;
  const int64_t parts = (int64_t)(kDensePartBytes / (rows * kPartRow * sizeof(float)));
  const int64_t most = std::min<int64_t>({std::max<int64_t>(1, max_keys / kMinKeys), parts / items, 512});
  int best = 1;
  double cost = 1e30;
  for (int64_t n = 1; n <= most; ++n) {
    const int64_t waves = ceil_div(items * n, places);
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

template <bool DEAL>
static int run_rows_as(const DenseArgs &a, int nr, int64_t items, int64_t grid, float *lse, void *stream) {
  if (lse) return run_rows<1, 1, DEAL, true>(a, items, grid, lse, nullptr, 0, stream);
  if (a.out_fp32)
    return nr == 1 ? run_rows<1, 0, DEAL, true>(a, items, grid, nullptr, nullptr, 0, stream)
                   : run_rows<2, 0, DEAL, true>(a, items, grid, nullptr, nullptr, 0, stream);
  return nr == 1 ? run_rows<1, 0, DEAL, false>(a, items, grid, nullptr, nullptr, 0, stream)
                 : run_rows<2, 0, DEAL, false>(a, items, grid, nullptr, nullptr, 0, stream);
}

int launch_dense_rows(DenseArgs a, int64_t max_keys, float *lse, void *stream) {
  // Tiles of 8 rows keep two blocks on an SM; more rows than that share a key's fetch and turn.
  const int nr = ((int64_t)a.nq << a.group_shift) <= 8 ? 1 : 2;
  const int per = (8 * nr) >> a.group_shift;
  a.tiles = (a.nq + per - 1) / per;
  const int64_t all = (int64_t)a.batch * a.hkv, items = (a.heads ? a.heads : all) * a.tiles;
  const int places = dense_sm_count() * blocks_per_sm(nr);
  // Per-sequence lengths: what the host knows is their bound, so the steps are dealt out on the device.
  // That costs a block its start and a second segment, so not where blocks have few steps anyway
  // (24 x 4 heads of up to 19001 tokens: 139 -> 125 us; 6 x 2 of 780: 20 -> 30 us).
  const int64_t steps = all * (ceil_div(max_keys, kStep) + 2);
  if (a.seq_len && steps >= 64 * (int64_t)places && steps < (int64_t)1 << 31 && a.tiles == 1 && a.batch <= kDealtSequences && items == all && items <= kMaxShared) {
    a.nsplit = 1;
    return run_rows_as<true>(a, nr, items, places, lse, stream);
  }
  a.nsplit = pick_split(items, max_keys, places, 8 * nr);
  return run_rows_as<false>(a, nr, items, items * a.nsplit, lse, stream);
}

int launch_dense_redo(DenseArgs a, int chunk_tiles, void *stream) {
  const int per = 16 >> a.group_shift;
  a.tiles = (a.nq + per - 1) / per;
  a.nsplit = 1;
  const int64_t items = (int64_t)a.batch * a.hkv * a.tiles;
  uint32_t *redo = reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(a.hdr) + kDenseRedo);
  return run_rows<2, 2, false, false>(a, items, std::min<int64_t>(items, dense_sm_count()), nullptr, redo, chunk_tiles, stream);
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
