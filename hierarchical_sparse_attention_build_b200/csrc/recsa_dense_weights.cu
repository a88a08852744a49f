// The softmax weight each cache slot receives: w[t] = sum over query rows of exp2(s[row][t] - L[row]),
// L[row] the row's log2-sum-exp.  Every weight needs every row's sum, so the scores are needed twice.
//
// A few rows (a decode step: at most 8 a KV group): reading K bounds it.  The rows kernel (in its
// accurate form) leaves its scores (4 bytes a row and key, against the key's 256) with the sums, and
// a second pass turns them into weights: one step's weights over 4 x 65536 tokens took 394 us with K
// read twice.
//
// More rows (a prompt's last queries): the products bound it.  dense_scores_kernel forms them on
// tcgen05 twice, with 128 x 128 tiles of keys and rows that were rotated once into shared-memory
// images.  Pass 1 has the query rows as the product's rows, so that a thread sums a row; pass 2 has
// the keys as rows, so that a thread sums a key over all query rows, in a fixed order and without a
// shuffle or an atomic.  The weights are fp32, so both operands are two fp16 parts (rounded, and what
// that leaves, rounded) of scaled values and three products are summed; what is dropped is below
// 2^-22 of the product of the magnitudes.  The tensor cores cut their sums off, toward zero, by up
// to 2^-23 a product: a score is summed in two accumulators of 64 dimensions each, joined by a
// rounded add.  64 queries' weights over 32768 tokens are off by 1.4e-7 (plain fp32: 1.2e-7), where
// bf16 parts and one accumulator left 1.25e-6; that costs 173 us against 164.  A head with elements
// that fp16 does not hold has its images made again, as two bf16 parts (2^-16).
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "recsa_dense_umma.cuh"

namespace recsa {
namespace {

constexpr int kEpilogueWarps = 8;           // two sets of four, on alternate tiles
constexpr int kScoreThreads = 320;
constexpr int kPartBytes = 2 * kTileBytes;  // a tile's two parts
constexpr int kMaxRange = 40;               // key tiles of a block
constexpr int64_t kCachedImages = (int64_t)80 << 20;  // of the 126 MB of L2
constexpr int kTurnThreads = 128;
constexpr int kTurnRows = 32;               // query rows a block of the images kernel turns
constexpr int kParts = kTile / kTurnRows;   // blocks of a row tile
constexpr int kWideBlocks = 32;             // blocks that make a head's images again
constexpr float kUnscale = 1.f / (kKeyScale * kQueryScale);

struct ScoreArgs {
  DenseArgs d;
  int bh0, heads;              // the launch's (sequence, KV head) pairs
  int row0, row_tiles;         // and the query rows of each: from row0 on, in tiles of 128
  int key0, key_tiles;         // the launch's key tiles of a head, 128 keys
  int nsplit;                  // blocks a head's key tiles are shared among
  int part0, parts;            // this launch's first of all blocks that a head's keys have in turn
  unsigned char *key_images, *query_images;  // [heads][key_tiles], [heads][row_tiles]: two parts each
  uint4 *live;                 // a key tile's tokens that were loaded
  int *beyond;                 // [heads]: some image's rows exceed fp16 (0 between calls)
  int *wide;                   // [heads]: the head's images are bf16 parts
  float2 *sums;                // [heads][row_tiles][2 parts][128]: a row's (maximum, sum) in part of the keys
  float *weights;
  int accumulate;
};

struct ScoreSmem {
  unsigned char q[kPartBytes];
  unsigned char k[2][kPartBytes];
  float acc[kMaxRange * kTile];  // pass 2: the block's keys
  alignas(16) float lse[kTile];
  alignas(16) int pos[kTile];
  alignas(16) uint64_t q_full;
  uint64_t q_empty, k_full[2], k_empty[2], d_full[2], d_empty[2], drain;
  uint32_t tmem, stop;
};
constexpr size_t kScoreSmem = sizeof(ScoreSmem) + 1024;

// One row of 8 + 8 dimensions, times `scale`, turned, as two parts of a tile (fp16, of keys cut off,
// of queries rounded; or WIDE: bf16); `most` keeps the largest magnitude.
template <bool WIDE, bool KEY>
__device__ __forceinline__ void put_parts(unsigned char *tile, int row, int ch, const uint4 &lo, const uint4 &hi,
                                          const Turn &t, float scale, float &most) {
  const uint32_t x[4] = {lo.x, lo.y, lo.z, lo.w}, y[4] = {hi.x, hi.y, hi.z, hi.w};
  uint32_t uh[4], ul[4], vh[4], vl[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    F2 p = f2_bf16(x[i]), q = f2_bf16(y[i]);
    p = f2_mul(p, f2(scale, scale));
    q = f2_mul(q, f2(scale, scale));
    const F2 u = f2_fma(q, f2_neg(t.s[i]), f2_mul(p, t.c[i])), v = f2_fma(p, t.s[i], f2_mul(q, t.c[i]));
    if (!WIDE) {
      const float2 x = f2_get(u), y = f2_get(v);
      most = max3(most, max3(fabsf(x.x), fabsf(x.y), fabsf(y.x)), fabsf(y.y));
    }
    if (!WIDE && KEY) {
      cut_pair(u, uh[i], ul[i]);
      cut_pair(v, vh[i], vl[i]);
    } else {
      split_pair<!WIDE>(u, uh[i], ul[i]);
      split_pair<!WIDE>(v, vh[i], vl[i]);
    }
  }
  put_row(tile, row, ch, make_uint4(uh[0], uh[1], uh[2], uh[3]), make_uint4(vh[0], vh[1], vh[2], vh[3]));
  put_row(tile + kTileBytes, row, ch, make_uint4(ul[0], ul[1], ul[2], ul[3]), make_uint4(vl[0], vl[1], vl[2], vl[3]));
}

// Query row `row` of a KV group is head row % G of query row / G.
__device__ __forceinline__ int row_position(const DenseArgs &d, int len, int row) {
  const int qi = row >> d.group_shift;
  return qi < d.nq ? dense_position(d, len, qi) : 0;
}

// kTurnRows query rows into their image.
template <bool WIDE>
__device__ __forceinline__ void turn_query_rows(const ScoreArgs &a, int hl, int rt, int part, int lt, float &most) {
  const DenseArgs &d = a.d;
  const int ch = lt & 7, r0 = lt >> 3, gs = d.group_shift, G = 1 << gs, hq = d.hkv << gs;
  const uint64_t *f = ws_freq(d.hdr) + ch * 8;
  const int b = (a.bh0 + hl) / d.hkv, h = (a.bh0 + hl) % d.hkv;
  const int len = dense_length(d, b, false);
#pragma unroll
  for (int i = 0; i < kTurnRows / 16; ++i) {
    const int in_tile = part * kTurnRows + r0 + 16 * i, row = a.row0 + rt * kTile + in_tile, qi = row >> gs;
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (qi < d.nq) {
      const uint4 *src =
          reinterpret_cast<const uint4 *>(d.q + (((int64_t)b * d.nq + qi) * hq + h * G + (row & (G - 1))) * kD);
      lo = __ldg(src + ch);
      hi = __ldg(src + ch + 8);
    }
    Turn t;
    t.set(f, dense_position(d, len, qi) - d.back);
    put_parts<WIDE, false>(a.query_images + ((int64_t)hl * a.row_tiles + rt) * kPartBytes, in_tile, ch, lo, hi, t,
                    WIDE ? d.qscale : d.qscale * kQueryScale, most);
  }
}

// A key tile into its image; false where the sequence has no tokens of it.
template <bool WIDE>
__device__ __forceinline__ bool turn_keys(const ScoreArgs &a, int hl, int kt, int lt, float &most) {
  const DenseArgs &d = a.d;
  const int ch = lt & 7, r0 = lt >> 3;
  const uint64_t *f = ws_freq(d.hdr) + ch * 8;
  const int b = (a.bh0 + hl) / d.hkv, h = (a.bh0 + hl) % d.hkv;
  const int len = dense_length(d, b, false), T = (a.key0 + kt) * kTile;
  if (T >= len) return false;
  unsigned char *const tile = a.key_images + ((int64_t)hl * a.key_tiles + kt) * kPartBytes;
  uint32_t word[4] = {0u, 0u, 0u, 0u};
  Turn t, step;
  t.set(f, T + r0);
  step.set(f, 16);
#pragma unroll 1
  for (int i0 = 0; i0 < 8; i0 += 4) {  // four rows in flight
    uint4 xl[4], xh[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = T + r0 + 16 * (i0 + i);
      xl[i] = xh[i] = make_uint4(0, 0, 0, 0);
      if (tok < len) {
        const int64_t r = cache_row(d, b, h, tok);
        if (r >= 0) {
          const uint4 *src = reinterpret_cast<const uint4 *>(d.k + r * kD);
          xl[i] = __ldg(src + ch);
          xh[i] = __ldg(src + ch + 8);
          word[i >> 1] |= i0 ? 0u : 1u << (r0 + 16 * (i & 1));
          word[2 + (i >> 1)] |= i0 ? 1u << (r0 + 16 * (i & 1)) : 0u;
        } else {
          atomicOr(&d.hdr->err, kErrIndex);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      put_parts<WIDE, true>(tile, r0 + 16 * (i0 + i), ch, xl[i], xh[i], t, WIDE ? 1.f : kKeyScale, most);
      t.advance(step);
    }
  }
  if (WIDE) return true;  // (the loaded tokens are noted already)
  __shared__ uint32_t words[4];
  if (lt < 4) words[lt] = 0u;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w)
    if (ch == 0) atomicOr(&words[w], word[w]);
  __syncthreads();
  if (lt == 0) a.live[(int64_t)hl * a.key_tiles + kt] = make_uint4(words[0], words[1], words[2], words[3]);
  return true;
}

// The first heads * key_tiles blocks turn a key tile each, the others kTurnRows query rows.
__global__ void __launch_bounds__(kTurnThreads, 5) dense_score_images_kernel(ScoreArgs a) {
  const DenseArgs &d = a.d;
  if (d.hdr->magic != kDenseMagic || d.hdr->rope_base != d.rope_base) return;  // the score kernel reports it
  const int lt = threadIdx.x, keys = a.heads * a.key_tiles;
  float most = 0.f;
  int hl;
  if ((int)blockIdx.x >= keys) {
    const int e = blockIdx.x - keys, rt = e / kParts % a.row_tiles;
    hl = e / kParts / a.row_tiles;
    turn_query_rows<false>(a, hl, rt, e % kParts, lt, most);
  } else {
    hl = blockIdx.x / a.key_tiles;
    turn_keys<false>(a, hl, blockIdx.x % a.key_tiles, lt, most);
  }
  if (!(most <= 65504.f)) a.beyond[hl] = 1;
}

// The images of a head that exceeds fp16 again, as bf16 parts.
__global__ void __launch_bounds__(kTurnThreads, 5) dense_wide_images_kernel(ScoreArgs a) {
  const DenseArgs &d = a.d;
  if (d.hdr->magic != kDenseMagic || d.hdr->rope_base != d.rope_base) return;
  const int lt = threadIdx.x, hl = blockIdx.x / kWideBlocks;
  const int any = __ldcg(a.beyond + hl);
  if (lt == 0 && blockIdx.x % kWideBlocks == 0) a.wide[hl] = any;
  if (!any) return;
  float most = 0.f;
  for (int i = blockIdx.x % kWideBlocks; i < a.key_tiles + kParts * a.row_tiles; i += kWideBlocks) {
    if (i < a.key_tiles)
      turn_keys<true>(a, hl, i, lt, most);
    else
      turn_query_rows<true>(a, hl, (i - a.key_tiles) / kParts, (i - a.key_tiles) % kParts, lt, most);
  }
}

// A block: a range of key tiles of one (sequence, KV head) against all its query rows, 128 at a
// time.  Warps 0-3 and 4-7 take the products of alternate tiles from TMEM, warp 8 issues them,
// warp 9 copies the images.
template <int PASS>
__global__ void __launch_bounds__(kScoreThreads, 1) dense_scores_kernel(ScoreArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  ScoreSmem &sm = *reinterpret_cast<ScoreSmem *>(smem_raw + (1024u - (smem_u32(smem_raw) & 1023u)) % 1024u);
  const DenseArgs &d = a.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (d.hdr->magic != kDenseMagic || d.hdr->rope_base != d.rope_base) {
    if (tid == 0) atomicOr(&d.hdr->err, kErrWs);
    return;
  }
  const int hl = blockIdx.x / a.nsplit, split = blockIdx.x % a.nsplit;
  if (PASS == 1 && split == 0 && tid == 0) a.beyond[hl] = 0;  // for the next images
  const int b = (a.bh0 + hl) / d.hkv, h = (a.bh0 + hl) % d.hkv;
  const int len = dense_length(d, b, PASS == 1 && tid == 0 && h == 0 && split == 0);
  const int tiles = min(a.key_tiles, max(0, (len + kTile - 1) / kTile - a.key0));
  const int kt0 = (int)((int64_t)tiles * split / a.nsplit), kt1 = (int)((int64_t)tiles * (split + 1) / a.nsplit);
  if (kt0 >= kt1) {  // pass 2 reads every block's sums
    if (PASS == 1)
      for (int e = tid; e < a.row_tiles * 2 * kTile; e += kScoreThreads) {
        const int rt = e / (2 * kTile), set = e / kTile % 2;
        a.sums[(((int64_t)hl * a.row_tiles + rt) * (2 * a.parts) + (a.part0 + split) * 2 + set) * kTile + e % kTile] =
            make_float2(-INFINITY, 0.f);
      }
    return;
  }
  if (tid == 0) {
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.d_full[i], 1);
      mbar_init(&sm.d_empty[i], 4);
    }
    sm.stop = 0;
    mbar_fence_init();
  }
  if (warp == 8) {
    umma::tmem_alloc(&sm.tmem, 512);
    umma::tmem_relinquish();
  }
  if (PASS == 2)
    for (int i = tid; i < (kt1 - kt0) * kTile; i += kScoreThreads) sm.acc[i] = 0.f;
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = sm.tmem;
  const bool wide = a.wide[hl] != 0;
  const float unscale = wide ? 1.f : kUnscale;
  auto wait = [&](uint64_t *bar, uint32_t parity) { bounded_wait(&sm.stop, d.hdr, bar, parity); };
  // key tiles that row tile rt's queries see (at least one, so that every row tile has a product)
  auto last_tile = [&](int rt) {
    const int row = min(a.row0 + (rt + 1) * kTile, d.nq << d.group_shift) - 1;
    const int p = row_position(d, len, row);
    return max(kt0 + 1, min(kt1, (max(p, 0) + kTile - 1) / kTile - a.key0));
  };

  if (warp < kEpilogueWarps) {
    const int set = warp >> 2, trow = (warp & 3) * 32 + lane;
    const uint32_t td = tmem + ((uint32_t)(warp & 3) << 21) + set * 2 * kTile;
    uint32_t n = 0;  // products so far
    for (int rt = 0; rt < a.row_tiles; ++rt) {
      const int end = last_tile(rt);
      if (PASS == 2) {
        asm volatile("bar.sync 1, 256;" ::: "memory");  // the last row tile's values have been read
        if (tid < kTile) {
          const int p = row_position(d, len, a.row0 + rt * kTile + tid);
          const float2 *src = a.sums + ((int64_t)hl * a.row_tiles + rt) * (2 * a.parts) * kTile + tid;
          float m = -INFINITY, l = 0.f;
          constexpr int kAhead = 16;  // parts in flight
          for (int j0 = 0; j0 < 2 * a.parts; j0 += kAhead) {
            float2 v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
              v[j] = j0 + j < 2 * a.parts ? __ldcg(src + (int64_t)(j0 + j) * kTile) : make_float2(-INFINITY, 0.f);
            float top = m;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) top = fmaxf(top, v[j].x);
            if (top > m) {
              l *= m == -INFINITY ? 1.f : exp2_approx(m - top);  // (l is 0 or NaN without a maximum)
              m = top;
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
              l += v[j].x != -INFINITY ? v[j].y * exp2_approx(v[j].x - m) : v[j].y;  // (0, or NaN: every score was)
          }
          // a row that sees nothing gives no weight; neither does a row past the queries
          const bool gives = a.row0 + rt * kTile + tid < (d.nq << d.group_shift) && (l > 0.f || l != l);
          sm.lse[tid] = gives ? m + log2f(l) : INFINITY;
          sm.pos[tid] = p;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
      }
      const int p_row = PASS == 1 ? row_position(d, len, a.row0 + rt * kTile + trow) : 0;
      const int p_least = row_position(d, len, a.row0 + rt * kTile);  // positions grow with the row
      float m = -INFINITY, l = 0.f;
      for (int kt = kt0; kt < end; ++kt, ++n) {
        if ((int)(n & 1) != set) continue;
        const int T = (a.key0 + kt) * kTile;
        const uint4 live = __ldg(a.live + (int64_t)hl * a.key_tiles + kt);
        wait(&sm.d_full[set], (n >> 1) & 1);
        umma::fence_after_sync();
        auto taken = [&]() {  // the accumulator may be overwritten
          umma::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.d_empty[set]);
        };
        if (PASS == 1) {
          const uint32_t lv[4] = {live.x, live.y, live.z, live.w};
          const bool masked = T + kTile > p_row || (live.x & live.y & live.z & live.w) != 0xffffffffu;
          uint32_t u[32], v[32];
          umma::tmem_ld32(td, u);
          umma::tmem_ld32(td + kTile, v);
#pragma unroll
          for (int g = 0; g < 4; ++g) {  // 32 columns, the next 32 on their way
            float s[32];
            umma::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = (__uint_as_float(u[i]) + __uint_as_float(v[i])) * unscale;
            if (g < 3) {
              umma::tmem_ld32(td + (g + 1) * 32, u);
              umma::tmem_ld32(td + kTile + (g + 1) * 32, v);
            } else {
              taken();
            }
            if (masked) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (T + g * 32 + i >= p_row || !((lv[g] >> i) & 1u)) s[i] = -INFINITY;
            }
            float x[2] = {m, m};
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              x[0] = max3(x[0], s[i], s[i + 1]);
              x[1] = max3(x[1], s[i + 2], s[i + 3]);
            }
            const float top = fmaxf(x[0], x[1]);
            if (top > m) {
              l *= m == -INFINITY ? 0.f : exp2_approx(m - top);
              m = top;
            }
            const float z = m == -INFINITY ? 0.f : m;
            float add[4] = {};
#pragma unroll
            for (int i = 0; i < 32; ++i) add[i & 3] += exp2_approx(s[i] - z);
            l += (add[0] + add[1]) + (add[2] + add[3]);
          }
        } else {
          const int t = T + trow;
          const uint32_t lw = trow < 32 ? live.x : trow < 64 ? live.y : trow < 96 ? live.z : live.w;
          // every row of the tile is a query's, and sees every key of the tile
          const bool whole = T + kTile <= p_least && a.row0 + (rt + 1) * kTile <= d.nq << d.group_shift;
          float add[4] = {};
          uint32_t u[32], v[32];
          umma::tmem_ld32(td, u);
          umma::tmem_ld32(td + kTile, v);
#pragma unroll
          for (int g = 0; g < 4; ++g) {  // 32 columns, the next 32 on their way
            float s[32];
            umma::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(u[i]) + __uint_as_float(v[i]);
            if (g < 3) {
              umma::tmem_ld32(td + (g + 1) * 32, u);
              umma::tmem_ld32(td + kTile + (g + 1) * 32, v);
            } else {
              taken();
            }
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 z = *reinterpret_cast<const float4 *>(&sm.lse[g * 32 + i]);
              float e[4] = {exp2_approx(__fmaf_rn(s[i], unscale, -z.x)), exp2_approx(__fmaf_rn(s[i + 1], unscale, -z.y)),
                            exp2_approx(__fmaf_rn(s[i + 2], unscale, -z.z)), exp2_approx(__fmaf_rn(s[i + 3], unscale, -z.w))};
              if (!whole) {
                const int4 p = *reinterpret_cast<const int4 *>(&sm.pos[g * 32 + i]);
                if (t >= p.x) e[0] = 0.f;
                if (t >= p.y) e[1] = 0.f;
                if (t >= p.z) e[2] = 0.f;
                if (t >= p.w) e[3] = 0.f;
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) add[k] += e[k];
            }
          }
          if ((lw >> (trow & 31)) & 1u) sm.acc[(kt - kt0) * kTile + trow] += (add[0] + add[1]) + (add[2] + add[3]);
        }
      }
      if (PASS == 1)
        a.sums[(((int64_t)hl * a.row_tiles + rt) * (2 * a.parts) + (a.part0 + split) * 2 + set) * kTile + trow] =
            make_float2(m, l);
    }
    if (PASS == 2) {
      asm volatile("bar.sync 1, 256;" ::: "memory");
      float *const w = a.weights + ((int64_t)b * d.hkv + h) * d.capacity;
      const int t0 = (a.key0 + kt0) * kTile;
      for (int t = t0 + tid; t < min((a.key0 + kt1) * kTile, len); t += kEpilogueWarps * 32) {
        const float v = sm.acc[t - t0];
        w[t] = a.accumulate ? w[t] + v : v;
      }
    }
  } else if (warp == 8) {
    if (elect_one()) {
      const uint64_t dq = swizzled_desc(smem_u32(sm.q), 16), dk = swizzled_desc(smem_u32(sm.k[0]), 16);
      const uint32_t idesc = wide ? chunk_idesc(kTile, true, false) : chunk_idesc(kTile, false, false);
      uint32_t n = 0;
      for (int rt = 0; rt < a.row_tiles; ++rt) {
        const int end = last_tile(rt);
        wait(&sm.q_full, rt & 1);
        for (int kt = kt0; kt < end; ++kt, ++n) {
          const uint32_t s = n & 1;
          wait(&sm.k_full[s], (n >> 1) & 1);
          if (n >= 2) wait(&sm.d_empty[s], ((n >> 1) - 1) & 1);
          umma::fence_after_sync();
          const uint64_t k = dk + s * (kPartBytes >> 4);
          const uint64_t rows = PASS == 1 ? dq : k, cols = PASS == 1 ? k : dq;
#pragma unroll
          for (int p = 0; p < 3; ++p) {  // small terms first: low x high, high x low, high x high
            // the second accumulator takes the high parts' last 64 dimensions alone
            const uint64_t ra = rows + (p == 0 ? kTileBytes >> 4 : 0), cb = cols + (p == 1 ? kTileBytes >> 4 : 0);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint32_t off = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
              const bool second = p == 2 && ks >= 4;
              umma::mma(tmem + (2 * s + second) * kTile, ra + off, cb + off, idesc, second ? ks > 4 : p + ks > 0);
            }
          }
          umma::commit(&sm.d_full[s]);
          umma::commit(&sm.k_empty[s]);
        }
        umma::commit(&sm.q_empty);
      }
      umma::commit(&sm.drain);  // nothing may be in flight when the tensor memory is freed
      if (!mbar_wait(&sm.drain, 0)) atomicOr(&d.hdr->err, kErrTimeout);
    }
  } else if (elect_one()) {
    uint32_t n = 0;
    for (int rt = 0; rt < a.row_tiles; ++rt) {
      const int end = last_tile(rt);
      if (rt > 0) wait(&sm.q_empty, (rt - 1) & 1);
      mbar_expect(&sm.q_full, kPartBytes);
      bulk_load(smem_u32(sm.q), a.query_images + ((int64_t)hl * a.row_tiles + rt) * kPartBytes, kPartBytes, &sm.q_full);
      for (int kt = kt0; kt < end; ++kt, ++n) {
        const uint32_t s = n & 1;
        if (n >= 2) wait(&sm.k_empty[s], ((n >> 1) - 1) & 1);
        mbar_expect(&sm.k_full[s], kPartBytes);
        bulk_load(smem_u32(sm.k[s]), a.key_images + ((int64_t)hl * a.key_tiles + kt) * kPartBytes, kPartBytes,
                  &sm.k_full[s]);
      }
    }
    // every copy has landed before the block may end
    for (uint32_t i = n > 2 ? n - 2 : 0; i < n; ++i) mbar_wait(&sm.k_full[i & 1], (i >> 1) & 1);
  }
  __syncwarp();
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (warp == 8) umma::tmem_dealloc(tmem, 512);
}

// Weights from the scores that the rows kernel left: a thread a key.
__global__ void __launch_bounds__(256) weights_from_scores_kernel(DenseArgs a, const float2 *__restrict__ sums,
                                                                 float *__restrict__ weights, int accumulate) {
  if (a.hdr->magic != kDenseMagic || a.hdr->rope_base != a.rope_base) return;  // the rows kernel reported it
  const int bh = a.bh0 + blockIdx.y, b = bh / a.hkv, h = bh % a.hkv, gs = a.group_shift, G = 1 << gs;
  const int len = dense_length(a, b, false), rows = a.nq << gs;
  __shared__ float2 z[8];  // a row's maximum and 1 / sum
  __shared__ int pos[8];  // the rows kernel visits no token that no row sees
  if (threadIdx.x < 8) {
    pos[threadIdx.x] = threadIdx.x < rows ? dense_position(a, len, threadIdx.x >> gs) : 0;
    z[threadIdx.x] = threadIdx.x < rows ? sums[((int64_t)b * a.nq + (threadIdx.x >> gs)) * (a.hkv << gs) + h * G +
                                               (threadIdx.x & (G - 1))]
                                        : make_float2(0.f, 0.f);
  }
  __syncthreads();
  const float *s = a.scores + (int64_t)blockIdx.y * a.score_pitch * a.score_stride;
  float *const w = weights + ((int64_t)b * a.hkv + h) * a.capacity;
  for (int t = blockIdx.x * blockDim.x + threadIdx.x; t < len; t += gridDim.x * blockDim.x) {
    float v = 0.f;
    for (int i = 0; i < a.score_stride; i += 2) {
      const float2 x = __ldcs(reinterpret_cast<const float2 *>(s + (int64_t)t * a.score_stride + i));
      if (t < pos[i]) v += exp2_approx(x.x - z[i].x) * z[i].y;
      if (t < pos[i + 1]) v += exp2_approx(x.y - z[i + 1].x) * z[i + 1].y;
    }
    w[t] = accumulate ? w[t] + v : v;
  }
}

int few_rows(DenseArgs d, float *lse, float *weights, int accumulate, int64_t room, void *stream) {
  const int64_t heads = (int64_t)d.batch * d.hkv;
  const int rows = d.nq << d.group_shift;
  d.score_stride = rows <= 2 ? 2 : rows <= 4 ? 4 : 8;
  d.score_pitch = ceil_div(std::max(d.length, 1), 16) * 16;
  const int64_t fit = std::min<int64_t>(room / (d.score_pitch * d.score_stride * (int64_t)sizeof(float)), 65535);
  if (fit < 1) return kNoRoom;
  d.scores = reinterpret_cast<float *>(reinterpret_cast<char *>(d.hdr) + kDenseImages);
  const int64_t step = std::min(heads, fit);
  for (int64_t bh0 = 0; bh0 < heads; bh0 += step) {
    d.bh0 = (int)bh0;
    d.heads = (int)std::min(step, heads - bh0);
    const int rc = launch_dense_rows(d, d.length, lse, stream);
    if (rc) return rc;
    const dim3 grid((unsigned)std::min<int64_t>(ceil_div(d.score_pitch, 256), 4096), (unsigned)d.heads);
    weights_from_scores_kernel<<<grid, 256, 0, (cudaStream_t)stream>>>(d, reinterpret_cast<const float2 *>(lse), weights, accumulate);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return (int)e;
  }
  return 0;
}

}  // namespace

int launch_dense_weights(const DenseArgs &d, float *lse, float *weights, int accumulate, int64_t room, void *stream) {
  const int64_t rows = (int64_t)d.nq << d.group_shift, heads = (int64_t)d.batch * d.hkv;
  if (rows <= 8 && 2 * rows * heads <= kMaxDenseLse) {
    const int rc = few_rows(d, lse, weights, accumulate, room, stream);
    if (rc != kNoRoom) return rc;
  }
  ScoreArgs a = {};
  a.d = d;
  a.weights = weights;
  const int64_t key_tiles = ceil_div(std::max(d.length, 1), kTile);
  // As many heads and rows a launch as the images' room and the sums' hold: an eighth of the room
  // for one head's rows, at least one tile of them.  Later rows add to what earlier ones wrote.  A
  // head whose images do not fit has its keys in slices, turned for pass 1 and again for pass 2.
  constexpr int64_t kKeyBytes = kPartBytes + (int64_t)sizeof(uint4);
  const int64_t sums = (int64_t)kDensePartBytes / (2 * (int64_t)(kTile * sizeof(float2)));  // of a row tile and a part
  const int64_t all_tiles = ceil_div(rows, kTile);
  int64_t slice = 0, slices = 0, least = 0;  // key tiles a launch; launches a pass; fewest blocks a slice
  auto slice_for = [&](int64_t row_tiles) {
    slice = std::min(key_tiles, (room - row_tiles * (int64_t)kPartBytes) / kKeyBytes);
    if (slice < 1) return false;
    slices = ceil_div(key_tiles, slice);
    least = ceil_div(slice, kMaxRange);
    return sums / (least * slices) >= 1;
  };
  if (!slice_for(1)) return kNoRoom;
  int64_t tiles = std::min(all_tiles, std::max<int64_t>(1, room / 8 / kPartBytes));
  while (tiles > 1 && (!slice_for(tiles) || tiles > sums / (least * slices))) tiles = (tiles + 1) / 2;
  slice_for(tiles);
  const int64_t key_bytes = slice * kKeyBytes;
  const int64_t fit = slices > 1 ? 1 : std::min(room / (key_bytes + tiles * (int64_t)kPartBytes), sums / (least * tiles));
  cudaError_t e = cudaFuncSetAttribute(dense_scores_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kScoreSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(dense_scores_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kScoreSmem);
  if (e != cudaSuccess) return (int)e;
  const cudaStream_t st = (cudaStream_t)stream;
  const int sms = dense_sm_count();
  // Both passes read a head's images for every row tile: heads in turn, as many as stay in the L2
  // cache from the turning to the last reading (64 queries over 8 x 32768 tokens, whose images are
  // 134 MB: 167 -> 161 us).
  const int64_t step = std::min({heads, fit, std::max<int64_t>(1, kCachedImages / key_bytes), (int64_t)kMaxShared});
  for (int64_t bh0 = 0; bh0 < heads; bh0 += step) {
    a.bh0 = (int)bh0;
    a.heads = (int)std::min(step, heads - bh0);
    a.key_images = reinterpret_cast<unsigned char *>(d.hdr) + kDenseImages;
    a.query_images = a.key_images + (int64_t)a.heads * slice * kPartBytes;
    a.live = reinterpret_cast<uint4 *>(a.query_images + (int64_t)a.heads * tiles * kPartBytes);
    a.beyond = reinterpret_cast<int *>(reinterpret_cast<char *>(d.hdr) + kDenseBeyond);
    a.wide = a.beyond + kMaxShared;
    a.sums = reinterpret_cast<float2 *>(reinterpret_cast<char *>(d.hdr) + kDensePart);
    for (int64_t rt0 = 0; rt0 < all_tiles; rt0 += tiles) {
      a.row0 = (int)(rt0 * kTile);
      a.row_tiles = (int)std::min(tiles, all_tiles - rt0);
      a.accumulate = accumulate || rt0 > 0;
      // one wave of blocks where that leaves each at most kMaxRange key tiles
      a.nsplit = (int)std::min<int64_t>(
          {std::max<int64_t>(least, sms / a.heads), slice, sums / ((int64_t)a.heads * a.row_tiles * slices)});
      a.parts = (int)(a.nsplit * slices);
      for (int pass = 1; pass <= 2; ++pass) {
        for (int64_t i = 0; i < slices; ++i) {
          a.key0 = (int)(i * slice);
          a.key_tiles = (int)std::min(slice, key_tiles - i * slice);
          a.part0 = (int)(i * a.nsplit);
          if (pass == 1 || slices > 1) {  // once where one slice holds all keys
            dense_score_images_kernel<<<(unsigned)(a.heads * (a.key_tiles + (int64_t)a.row_tiles * kParts)), kTurnThreads, 0,
                                        st>>>(a);
            dense_wide_images_kernel<<<(unsigned)(a.heads * kWideBlocks), kTurnThreads, 0, st>>>(a);
          }
          const unsigned blocks = (unsigned)(a.heads * a.nsplit);
          if (pass == 1)
            dense_scores_kernel<1><<<blocks, kScoreThreads, kScoreSmem, st>>>(a);
          else
            dense_scores_kernel<2><<<blocks, kScoreThreads, kScoreSmem, st>>>(a);
          e = cudaGetLastError();
          if (e != cudaSuccess) return (int)e;
        }
      }
    }
  }
  return 0;
}

}  // namespace recsa
