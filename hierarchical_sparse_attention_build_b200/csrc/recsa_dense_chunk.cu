// Dense attention of a chunk of queries on the 5th-generation tensor cores (bf16 outputs).
//
// dense_images_kernel turns the keys and queries to their positions once and leaves them as the
// tiles' shared-memory images, so that dense_chunk_kernel fetches a tile with one bulk copy
// (turning the keys inside it, once a work item, took as many issue slots as the softmax: a
// chunk of 4096 over 32768 tokens, 32 query heads, took 4.1 ms that way).
//
// dense_chunk_kernel: a work item is 256 query rows (256 / G queries x the G heads of one KV
// group) of one sequence, as two tiles of 128 rows; its keys come in tiles of 128.  One CTA per SM:
//   warps 0-3, 4-7 : softmax of the two row tiles, a thread a row with 64 scores in registers; the
//                    probabilities go over the scores in TMEM.  (Two threads a row were slower:
//                    their exchange of maxima cost more than the shorter rows gave.)
//   warps 8-11     : gather the values with cp.async (any page size) into swizzled tiles;
//   warps 12, 14   : one thread each issues a row tile's products, S = Q K^T (shared x shared) and
//                    O += P V (TMEM x shared).  (One thread for both spent 200 cycles a wait with
//                    the tensor cores idle.)
//   warp 13        : one thread copies the images.
// Steps are half a key tile, 64 keys: a row's softmax has one half while the tensor cores do the
// other half's O += P V and next S, and the other row tile's.
// Measured: 2048 queries over 16384 tokens, 32/8 heads: 465 us, 1108 TFLOP/s, tensor pipe and
// special-function unit each half busy; 4096 over 32768: 2.0 ms in a short burst, 2.3 ms at the
// power limit.  What bounds it is the wait of a row's next scores for its weights and back.
//
// Rounding: rotated queries and keys are rounded to fp16 (half a step is 2^-11 of an element, an
// eighth of bf16's), probabilities to bf16 (the values' type: one product takes one type; half a
// step, 2^-8 of a weight, as the output's own rounding).  A rotated element beyond fp16's range, or
// an output that is not finite (a hidden token's value may hold anything, and a zero weight times
// infinity is NaN), marks the item: the rows kernel, which has neither limit, then computes it again.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "recsa_dense_umma.cuh"

namespace recsa {
namespace {

constexpr int kItemRows = 2 * kTile;
constexpr int kStepKeys = 64;              // keys of a softmax step: half a key tile
constexpr int kSoftWarps = 8;
constexpr int kLoadThreads = 128;
constexpr int kChunkThreads = 512;
constexpr int kQueryBytes = 2 * kTileBytes;
constexpr int kQueryRows = 64;              // query rows a block of the images kernel turns
constexpr int kRing = 2;                    // key and value tiles in shared memory
constexpr int kMaxChunkBlocks = (int)(kDensePartBytes / (2 * kItemRows * kPartRow * sizeof(float)));
constexpr float kRescale = 64.f;            // a row's maximum may lag by 2^64 before its output is rescaled

struct ChunkSmem {
  unsigned char q[2][kTileBytes];
  unsigned char k[kRing][kTileBytes];
  unsigned char v[kRing][kTileBytes];
  uint4 live[4];                            // a key tile's tokens that were loaded, by tile % 4
  int gap[4];                               // whether some token of it before the sequence's end was not
  uint64_t k_full[kRing], k_empty[kRing], v_full[kRing], v_empty[kRing];
  uint64_t s_full[2][2], p_full[2][2];
  uint64_t drain[2];
  uint32_t tmem;
  uint32_t stop;                            // a wait ran out: no role waits any more, all run to their ends
  int scan[kChunkThreads / 32];
  int prefix[kMaxShared + 1];               // key tiles before each item, when items are shared
};
constexpr size_t kChunkSmem = sizeof(ChunkSmem) + 1024;  // the tiles begin on 1024 bytes

struct ChunkArgs {
  DenseArgs d;
  int bh0, heads;   // the launch's (sequence, KV head) pairs
  int tile0, tiles; // and its items of each (of the d.tiles that the chunk has)
  int items;
  int shared;       // 1: the key tiles of all items are dealt out evenly to the blocks
  int key_tiles, query_sets;
  uint32_t *redo;
  int *prefix;
  // rotated rows: keys [heads][key_tiles] and their loaded tokens; queries [items][1 or 2: for the
  // window's tokens, for the sinks][2 row tiles]
  unsigned char *key_images, *query_images;
  uint4 *live;
};

// What a role knows of the item it is at.
struct Item {
  int b, h, q0, nq;       // sequence, KV head, first query, queries
  int len, p_min, p_max;  // tokens; positions of the first and last query
  int hi1, n1;            // sinks: tokens, key tiles
  int lo2, hi2, first;    // the window's tokens; its first key tile
  int tiles;              // key tiles (at least one, which may hold nothing)
  __device__ __forceinline__ bool sink(int j) const { return j < n1; }
  __device__ __forceinline__ int token(int j) const { return (j < n1 ? j : first + j - n1) * kTile; }
};
__device__ __forceinline__ Item chunk_item(const ChunkArgs &a, int item) {
  const DenseArgs &d = a.d;
  Item it;
  const int bh = a.bh0 + item / a.tiles, tile = a.tile0 + a.tiles - 1 - item % a.tiles;  // the longest ranges first
  it.b = bh / d.hkv;
  it.h = bh % d.hkv;
  it.q0 = tile * (kItemRows >> d.group_shift);
  it.nq = min(kItemRows >> d.group_shift, d.nq - it.q0);
  it.len = dense_length(d, it.b, false);
  it.p_min = dense_position(d, it.len, it.q0);
  it.p_max = dense_position(d, it.len, it.q0 + it.nq - 1);
  it.hi1 = d.window ? max(0, min(d.sinks, it.p_max)) : 0;
  it.n1 = (it.hi1 + kTile - 1) / kTile;
  it.lo2 = max(0, window_first(d, it.p_min));
  it.hi2 = max(it.p_max, 0);
  it.first = it.lo2 / kTile;
  it.tiles = max(1, it.n1 + (it.hi2 > it.lo2 ? (it.hi2 + kTile - 1) / kTile - it.first : 0));
  return it;
}
// Whether the item's rows reach into its second row tile.
__device__ __forceinline__ bool two_tiles(const DenseArgs &d, const Item &it) { return (it.nq << d.group_shift) > kTile; }
// Where the rows kernel looks whether to compute a tile of the chunk again.
__device__ __forceinline__ void mark_again(const ChunkArgs &a, int b, int h, int tile) {
  a.redo[redo_slot(b * a.d.hkv + h, a.d.tiles, tile)] = 1u;
}

// The key tiles that some query of the chunk sees: those of the sinks, then the window's.
struct HeadRange {
  int n1, first, count;
};
__device__ __forceinline__ HeadRange head_range(const DenseArgs &d, int len) {
  const int p_min = dense_position(d, len, 0), p_max = dense_position(d, len, d.nq - 1);
  HeadRange r;
  r.n1 = d.window ? (max(0, min(d.sinks, p_max)) + kTile - 1) / kTile : 0;
  r.first = max(0, window_first(d, p_min)) / kTile;
  r.count = r.n1 + max(0, (max(p_max, 0) + kTile - 1) / kTile - r.first);
  return r;
}

// The segments (item, key tiles [j0, j1)) of this block, the same for every role.
struct Segments {
  int item, at, end;  // the item; shared: the next key tile overall and where the block's end
  int begin;          // shared: where the block's begin
  int j0, j1;
};
// Shared: block c of `blocks` holds key tiles [total c / blocks, total (c + 1) / blocks).
__device__ __forceinline__ int dealt(int total, int blocks, int c) { return (int)((int64_t)total * c / blocks); }
__device__ __forceinline__ int sharing_blocks(int total, int grid) { return min(grid, total); }
// A block's part of an item it shares: at most its first segment's and its last's are parts.
__device__ __forceinline__ float *part_of(const DenseArgs &d, int c, bool first) {
  return ws_part(d.hdr) + ((int64_t)c * 2 + (first ? 0 : 1)) * (kItemRows * kPartRow);
}
__device__ __forceinline__ Segments segments_begin(const ChunkArgs &a, const ChunkSmem &sm) {
  Segments s;
  s.j0 = s.j1 = 0;
  s.at = s.end = s.begin = 0;
  s.item = (int)blockIdx.x - (int)gridDim.x;
  if (a.shared) {
    const int total = sm.prefix[a.items], blocks = sharing_blocks(total, gridDim.x);
    if ((int)blockIdx.x >= blocks) return s;
    s.begin = s.at = dealt(total, blocks, blockIdx.x);
    s.end = dealt(total, blocks, blockIdx.x + 1);
    int lo = 0, hi = a.items - 1;  // the item that holds key tile `at`
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (sm.prefix[mid] <= s.at) lo = mid; else hi = mid - 1;
    }
    s.item = lo - 1;
  }
  return s;
}
__device__ __forceinline__ bool segments_next(const ChunkArgs &a, const ChunkSmem &sm, Segments &s, Item &it) {
  if (a.shared) {
    if (s.at >= s.end) return false;
    ++s.item;
    it = chunk_item(a, s.item);
    s.j0 = s.at - sm.prefix[s.item];
    s.j1 = min(it.tiles, s.j0 + s.end - s.at);
    s.at += s.j1 - s.j0;
    return true;
  }
  s.item += gridDim.x;
  if (s.item >= a.items) return false;
  it = chunk_item(a, s.item);
  s.j0 = 0;
  s.j1 = it.tiles;
  return true;
}

__device__ __forceinline__ void wait(ChunkSmem &sm, const ChunkArgs &a, uint64_t *bar, uint32_t parity) {
  bounded_wait(&sm.stop, a.d.hdr, bar, parity);
}

// Query rows row0 + 0 .. kQueryRows - 1 of an item into its image, turned to their positions
// (sinks: to their positions for the sinks).
__device__ __forceinline__ void turn_queries(const ChunkArgs &a, unsigned char *q, const Item &it, bool sink, int row0,
                                             int lt, __half2 &most) {
  const DenseArgs &d = a.d;
  const int ch = lt & 7, gs = d.group_shift, G = 1 << gs, hq = d.hkv << gs, r0 = row0 + (lt >> 3);
  const uint64_t *f = ws_freq(d.hdr) + ch * 8;
  constexpr int kPer = kQueryRows / 16;  // rows r0 + 16 i of a thread
  auto position = [&](int i) {
    const int p = dense_position(d, it.len, it.q0 + ((r0 + 16 * i) >> gs));
    return sink ? sink_position(d, p) : p;
  };
  uint4 lo[kPer], hi[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int row = r0 + 16 * i, qi = row >> gs;
    lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
    if (qi < it.nq) {
      const uint4 *src = reinterpret_cast<const uint4 *>(
          d.q + (((int64_t)it.b * d.nq + it.q0 + qi) * hq + it.h * G + (row & (G - 1))) * kD);
      lo[i] = __ldg(src + ch);
      hi[i] = __ldg(src + ch + 8);
    }
  }
  // the rows' positions advance evenly (16 / G a step, or not at all), except where the sinks'
  // positions stop growing on the way: those are turned one by one
  const int p0 = position(0), by = position(1) - p0;
  bool even = true;
#pragma unroll
  for (int i = 2; i < kPer; ++i) even = even && position(i) == p0 + i * by;
  Turn t, step;
  t.set(f, p0 - d.back);
  if (by != 0) step.set(f, by);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int row = r0 + 16 * i;
    uint4 ol, oh;
    turn_row<true>(lo[i], hi[i], t, d.qscale, ol, oh, most);
    put_row(q + (row >> 7) * kTileBytes, row & 127, ch, ol, oh);
    if (i + 1 < kPer) {
      if (!even)
        t.set(f, position(i + 1) - d.back);
      else if (by != 0)
        t.advance(step);
    }
  }
}

__device__ __forceinline__ bool beyond_half(__half2 most) {
  return __hgt(__hmax(__low2half(most), __high2half(most)), __float2half(65504.f));
}

// Rotated keys (the first `keys` blocks: a key tile each) and queries (kQueryRows rows a block)
// of a launch as the chunk kernel's images.
__global__ void __launch_bounds__(kLoadThreads, 6) dense_images_kernel(ChunkArgs a, int keys) {
  const DenseArgs &d = a.d;
  if (d.hdr->magic != kDenseMagic || d.hdr->rope_base != d.rope_base) return;  // the chunk kernel reports it
  const int lt = threadIdx.x, ch = lt & 7, r0 = lt >> 3;
  __half2 most = __floats2half2_rn(0.f, 0.f);
  if ((int)blockIdx.x >= keys) {
    constexpr int kParts = kItemRows / kQueryRows;
    const int e = blockIdx.x - keys, image = e / kParts, item = image / a.query_sets;
    const Item it = chunk_item(a, item);
    turn_queries(a, a.query_images + (int64_t)image * kQueryBytes, it, image % a.query_sets == 1, e % kParts * kQueryRows,
                 lt, most);
    if (beyond_half(most)) mark_again(a, it.b, it.h, it.q0 / (kItemRows >> d.group_shift));
    return;
  }
  const int hl = blockIdx.x / a.key_tiles, kt = blockIdx.x % a.key_tiles;
  const int b = (a.bh0 + hl) / d.hkv, h = (a.bh0 + hl) % d.hkv;
  const int len = dense_length(d, b, false);
  const HeadRange hr = head_range(d, len);
  if (kt >= hr.count) return;
  const int T = (kt < hr.n1 ? kt : hr.first + kt - hr.n1) * kTile;
  unsigned char *const tile = a.key_images + (int64_t)blockIdx.x * kTileBytes;
  uint32_t word[4] = {0u, 0u, 0u, 0u};
  Turn t, step;
  const uint64_t *f = ws_freq(d.hdr) + ch * 8;
  t.set(f, T + r0);
  step.set(f, 16);
#pragma unroll
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
          word[(i0 + i) >> 1] |= 1u << (r0 + 16 * (i & 1));
        } else {
          atomicOr(&d.hdr->err, kErrIndex);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 ol, oh;
      turn_row<false>(xl[i], xh[i], t, 1.f, ol, oh, most);
      put_row(tile, r0 + 16 * (i0 + i), ch, ol, oh);
      t.advance(step);
    }
  }
  __shared__ uint32_t words[4];
  if (lt < 4) words[lt] = 0u;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w)
    if (ch == 0) atomicOr(&words[w], word[w]);
  __syncthreads();
  if (lt == 0) a.live[blockIdx.x] = make_uint4(words[0], words[1], words[2], words[3]);
  if (beyond_half(most))  // any of the head's items may read this tile
    for (int i = 0; i < d.tiles; ++i) mark_again(a, b, h, i);
}

// bits n .. 31 (none for n >= 32, all for n <= 0)
__device__ __forceinline__ uint32_t bits_from(int n) { return n >= 32 ? 0u : 0xffffffffu << max(n, 0); }

__device__ __forceinline__ float row_max(const uint32_t (&s)[2][32]) {
  float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 32; i += 4)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      x[g] = max3(x[g], __uint_as_float(s[g & 1][i + 2 * (g >> 1)]), __uint_as_float(s[g & 1][i + 2 * (g >> 1) + 1]));
  return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
}

// A row's weights 2^(s - m) of half a key tile, rounded to bf16, over the scores in TMEM; returns
// their sum and takes the scores' maximum into x.
__device__ __forceinline__ float weigh(const uint32_t (&s)[2][32], float m, uint32_t ts, float &x) {
  const float z = m == -INFINITY ? 0.f : m;
  const F2 nz = f2(-z, -z);
  F2 add = f2(0.f, 0.f);
  float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float u = __uint_as_float(s[g][2 * i]), v = __uint_as_float(s[g][2 * i + 1]);
      const float2 d = f2_get(f2_add(f2(u, v), nz));
      const float2 e = make_float2(exp2_approx(d.x), exp2_approx(d.y));
      add = f2_add(add, f2(e.x, e.y));
      pk[i] = cvt_bf16x2(e.x, e.y);
      if (i & 1)
        x1 = max3(x1, u, v);
      else
        x0 = max3(x0, u, v);
    }
    tmem_st16(ts + g * 16, pk);
  }
  x = fmaxf(x0, x1);
  return f2_get(add).x + f2_get(add).y;
}

__global__ void __launch_bounds__(kChunkThreads, 1) dense_chunk_kernel(ChunkArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  ChunkSmem &sm = *reinterpret_cast<ChunkSmem *>(smem_raw + (1024u - (smem_u32(smem_raw) & 1023u)) % 1024u);
  const DenseArgs &d = a.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (d.hdr->magic != kDenseMagic || d.hdr->rope_base != d.rope_base) {
    if (tid == 0) atomicOr(&d.hdr->err, kErrWs);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.v_full[i], kLoadThreads);
      mbar_init(&sm.k_empty[i], 2);
      mbar_init(&sm.v_empty[i], 2);
    }
    for (int u = 0; u < 4; ++u) {
      mbar_init(&sm.s_full[u & 1][u >> 1], 1);
      mbar_init(&sm.p_full[u & 1][u >> 1], kSoftWarps / 2);
    }
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    sm.stop = 0;
    mbar_fence_init();
  }
  if (warp == 12) {
    umma::tmem_alloc(&sm.tmem, 512);
    umma::tmem_relinquish();
  }
  if (a.shared) {  // key tiles before each item: a block-wide prefix sum
    const int per = (a.items + kChunkThreads - 1) / kChunkThreads, i0 = min(a.items, tid * per),
              i1 = min(a.items, i0 + per);
    int sum = 0;
    for (int i = i0; i < i1; ++i) sum += chunk_item(a, i).tiles;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int w = 0; w < warp; ++w) at += sm.scan[w];
    for (int i = i0; i < i1; ++i) {
      sm.prefix[i] = at;
      at += chunk_item(a, i).tiles;
    }
    if (i1 == a.items && i0 < i1) sm.prefix[a.items] = at;
  }
  if (d.seq_len && blockIdx.x == 0)
    for (int b = tid; b < d.batch; b += kChunkThreads) dense_length(d, b, true);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (a.shared && blockIdx.x == 0)  // for dense_join_kernel
    for (int i = tid; i <= a.items; i += kChunkThreads) a.prefix[i] = sm.prefix[i];
  const uint32_t tmem = sm.tmem;
  Segments sg = segments_begin(a, sm);
  Item it;

  // Registers a thread: 512 threads are launched with 128 (65,536); the softmax takes 144, the
  // loaders give theirs down to 96 and the last four warps keep 128 (65,536).
  if (warp < kSoftWarps) {
    // ------------------------------------------------------------------ softmax and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int t = warp >> 2, trow = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const uint32_t ts = tmem + lanes + t * kTile, to = tmem + lanes + 2 * kTile + t * kTile;
    const int row = t * kTile + trow, gs = d.group_shift, G = 1 << gs, hq = d.hkv << gs;
    uint32_t n = 0, n_s = 0;  // key tiles seen; phases of s_full
    while (segments_next(a, sm, sg, it)) {
      const bool busy = t == 0 || two_tiles(d, it);
      const bool in = (row >> gs) < it.nq;
      const int p = in ? dense_position(d, it.len, it.q0 + (row >> gs)) : INT_MAX;  // rows past the chunk: no mask
      const int lo = in ? window_first(d, p) : 0, hi_sink = min(p, it.hi1);
      // every row of the warp sees tokens [lo_all, hi_all) of the window, [0, hi_sink_all) of the sinks
      const int lo_all = __reduce_max_sync(0xffffffffu, lo), hi_all = __reduce_min_sync(0xffffffffu, p),
                hi_sink_all = __reduce_min_sync(0xffffffffu, hi_sink);
      float m = -INFINITY, l = 0.f;
      if (!busy) n += sg.j1 - sg.j0;
      for (int j = sg.j0; busy && j < sg.j1; ++j, ++n, ++n_s) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int T = it.token(j) + h * kStepKeys;
          const bool sink = it.sink(j);
          wait(sm, a, &sm.s_full[t][h], n_s & 1);
          umma::fence_after_sync();
          const uint32_t tsh = ts + h * kStepKeys;
          uint32_t s[2][32];
          umma::tmem_ld32(tsh, s[0]);
          umma::tmem_ld32(tsh + 32, s[1]);
          const bool masked = sm.gap[n & 3] || T + kStepKeys > (sink ? hi_sink_all : hi_all) || (!sink && T < lo_all);
          umma::tmem_wait_ld();
          if (masked) {
            const uint2 live = reinterpret_cast<const uint2 *>(&sm.live[n & 3])[h];
            const int a0 = (sink ? 0 : lo) - T, a1 = (sink ? hi_sink : p) - T;  // visible columns [a0, a1)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const uint32_t seen = (g ? live.y : live.x) & bits_from(a0 - 32 * g) & ~bits_from(a1 - 32 * g);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((seen >> i) & 1u)) s[g][i] = 0xff800000u;
            }
          }
          const bool first = j == sg.j0 && h == 0;
          if (first) m = row_max(s);
          // The weights are taken from the maximum so far, without waiting for this step's:
          // weights, sums and outputs hold numbers up to 2^127 with the same relative precision.
          // Only where a row's maximum has grown by more than 2^kRescale are they taken again
          // (and its output rescaled).
          float x, sum = weigh(s, m, tsh, x);
          const bool up = x > m + kRescale || (m == -INFINITY && x > m);
          if (__any_sync(0xffffffffu, up)) {
            const float f = up ? (m == -INFINITY ? 0.f : exp2_approx(m - x)) : 1.f;
            if (up) m = x;
            l *= f;
            sum = weigh(s, m, tsh, x);
            if (!first) {
              // the last product into the output is complete once the other half's next scores are
              wait(sm, a, &sm.s_full[t][h ^ 1], (n_s + h) & 1);
              umma::fence_after_sync();
#pragma unroll 1
              for (int g = 0; g < 8; ++g) {
                uint32_t o[16];
                tmem_ld16(to + g * 16, o);
                umma::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st16(to + g * 16, o);
              }
            }
          }
          l += sum;
          tmem_wait_st();
          umma::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[t][h]);
        }
      }
      // s_full arrives once more after the segment's last products
      if (busy) {
        wait(sm, a, &sm.s_full[t][0], n_s & 1);
        wait(sm, a, &sm.s_full[t][1], n_s & 1);
        ++n_s;
        umma::fence_after_sync();
      }
      // epilogue: the item's output, or this block's part of it: [32 pieces of 16 bytes][row], then
      // (maximum, sum) [row]
      const bool part = sg.j1 - sg.j0 < it.tiles;
      const int64_t out_row = ((int64_t)it.b * d.nq + it.q0 + (row >> gs)) * hq + it.h * G + (row & (G - 1));
      uint4 *const po = reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(d.out) + out_row * kD);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      bool odd = !(l < INFINITY);
      float *const mypart = part_of(d, blockIdx.x, sg.at - (sg.j1 - sg.j0) == sg.begin);
#pragma unroll 1
      for (int g = 0; busy && g < 4; ++g) {
        uint32_t o[32];
        umma::tmem_ld32(to + g * 32, o);
        umma::tmem_wait_ld();
        if (part) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            reinterpret_cast<uint4 *>(mypart)[(g * 8 + i) * kItemRows + row] =
                make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float u = __uint_as_float(o[8 * i + 2 * c]) * inv, v = __uint_as_float(o[8 * i + 2 * c + 1]) * inv;
              odd |= !(fabsf(u) < INFINITY) || !(fabsf(v) < INFINITY);
              w[c] = cvt_bf16x2(u, v);
            }
            if (in) po[g * 4 + i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      umma::fence_before_sync();
      if (part) {
        if (busy) reinterpret_cast<float2 *>(mypart + kItemRows * kD)[row] = make_float2(m, l);
        odd = false;  // dense_join_kernel joins the parts
      }
      if (odd && in) mark_again(a, it.b, it.h, it.q0 / (kItemRows >> gs));
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ values
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    const int lt = tid - kSoftWarps * 32, ch = lt & 7, r0 = lt >> 3;  // rows r0 + 16 i
    const uint32_t sv = smem_u32(sm.v[0]) + r0 * 128 + ((ch ^ (r0 & 7)) << 4);
    uint32_t n = 0;  // key tiles loaded
    while (segments_next(a, sm, sg, it)) {
      uint32_t rows[8], here = 0;  // rows in the cache (fewer than 2^32 fit a GPU); bit i: row i is a token to load
      auto place = [&](int j) {
        const int T = it.token(j), lo = it.sink(j) ? 0 : it.lo2, hi = it.sink(j) ? it.hi1 : it.hi2;
        here = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = T + r0 + 16 * i;
          const int64_t r = tok >= lo && tok < hi ? cache_row(d, it.b, it.h, tok) : -1;
          rows[i] = r >= 0 ? (uint32_t)r : 0u;
          here |= r >= 0 ? 1u << i : 0u;
        }
      };
      place(sg.j0);
      for (int j = sg.j0; j < sg.j1; ++j, ++n) {
        const int s = n % kRing;
        if (n >= kRing) wait(sm, a, &sm.v_empty[s], (n / kRing - 1) & 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t dst = sv + s * kTileBytes + i * 16 * 128;
          const bool on = (here >> i) & 1u;
          const uint16_t *src = d.v + (int64_t)rows[i] * kD + ch * 8;
          cp_async16(dst, src, on);
          cp_async16(dst + kHalfBytes, src + kHalf, on);
        }
        cp_async_commit();
        if (j + 1 < sg.j1) place(j + 1);
        cp_async_wait<0>();
        umma::fence_async_smem();
        mbar_arrive(&sm.v_full[s]);
      }
    }
  } else {
    if (warp == 13 && elect_one()) {
      // ---------------------------------------------------------------- images
      uint32_t n = 0;
      while (segments_next(a, sm, sg, it)) {
        const HeadRange hr = head_range(d, it.len);
        const int hl = it.b * d.hkv + it.h - a.bh0;
        for (int j = sg.j0; j < sg.j1; ++j, ++n) {
          const bool sink = it.sink(j);
          const int s = n % kRing;
          const int kt = min(sink ? j : hr.n1 + it.first + j - it.n1 - hr.first, a.key_tiles - 1);
          const int64_t image = (int64_t)hl * a.key_tiles + kt;
          const bool queries = j == sg.j0 || (j == it.n1 && j > 0);
          // new queries: the products that read the last ones are done once the previous tile is free
          if (queries && n > 0) wait(sm, a, &sm.k_empty[(n - 1) % kRing], ((n - 1) / kRing) & 1);
          if (n >= kRing) wait(sm, a, &sm.k_empty[s], (n / kRing - 1) & 1);
          const uint4 live = __ldg(a.live + image);
          const int left = it.len - it.token(j);  // tokens of the tile
          const int have = __popc(live.x) + __popc(live.y) + __popc(live.z) + __popc(live.w);
          sm.live[n & 3] = live;
          sm.gap[n & 3] = have < min(left, kTile);
          mbar_expect(&sm.k_full[s], kTileBytes + (queries ? kQueryBytes : 0));
          if (queries)
            bulk_load(smem_u32(sm.q[0]),
                      a.query_images + ((int64_t)sg.item * a.query_sets + (sink && a.query_sets == 2 ? 1 : 0)) * kQueryBytes,
                      kQueryBytes, &sm.k_full[s]);
          bulk_load(smem_u32(sm.k[s]), a.key_images + image * kTileBytes, kTileBytes, &sm.k_full[s]);
        }
      }
      // every copy has landed before the block may end
      if (n > 0) mbar_wait(&sm.k_full[(n - 1) % kRing], ((n - 1) / kRing) & 1);
      if (n > 1) mbar_wait(&sm.k_full[(n - 2) % kRing], ((n - 2) / kRing) & 1);
    }
    if ((warp == 12 || warp == 14) && elect_one()) {
      // ---------------------------------------------------------------- products
      const int t = warp == 14;
      const uint32_t ts = tmem + t * kTile, to = tmem + 2 * kTile + t * kTile;
      const uint64_t dq = swizzled_desc(smem_u32(sm.q[t]), 16), dk = swizzled_desc(smem_u32(sm.k[0]), 16),
                     dv = swizzled_desc(smem_u32(sm.v[0]), kHalfBytes);
      uint32_t n = 0, n_p = 0;  // key tiles; phases of p_full
      auto scores = [&](int h, uint32_t i) {
        const uint64_t k = dk + (i % kRing) * (kTileBytes >> 4) + h * ((kStepKeys * 128) >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t off = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
          umma::mma(ts + h * kStepKeys, dq + off, k + off, chunk_idesc(kStepKeys, false, false), ks > 0);
        }
      };
      while (segments_next(a, sm, sg, it)) {
        const int count = sg.j1 - sg.j0;
        if (t == 1 && !two_tiles(d, it)) {  // the other row tile holds all rows: tiles are let go as they come
          for (int j = 0; j < count; ++j, ++n) {
            wait(sm, a, &sm.k_full[n % kRing], (n / kRing) & 1);
            umma::commit(&sm.k_empty[n % kRing]);
            wait(sm, a, &sm.v_full[n % kRing], (n / kRing) & 1);
            umma::commit(&sm.v_empty[n % kRing]);
          }
          continue;
        }
        wait(sm, a, &sm.k_full[n % kRing], (n / kRing) & 1);
        umma::fence_after_sync();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          scores(h, n);
          umma::commit(&sm.s_full[t][h]);
        }
        umma::commit(&sm.k_empty[n % kRing]);
        for (int j = 0; j < count; ++j, ++n, ++n_p) {
          const uint32_t s = n % kRing, s1 = (n + 1) % kRing;
          const bool more = j + 1 < count;
          wait(sm, a, &sm.v_full[s], (n / kRing) & 1);
          if (more) wait(sm, a, &sm.k_full[s1], ((n + 1) / kRing) & 1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            wait(sm, a, &sm.p_full[t][h], n_p & 1);
            umma::fence_after_sync();
            const uint64_t v = dv + s * (kTileBytes >> 4) + h * ((kStepKeys * 128) >> 4);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_tmem_a(to, ts + h * kStepKeys + ks * 8, v + ks * (2048 >> 4), chunk_idesc(kTile, true, true),
                         j + h + ks > 0);
            if (more) scores(h, n + 1);
            umma::commit(&sm.s_full[t][h]);
          }
          umma::commit(&sm.v_empty[s]);
          if (more) umma::commit(&sm.k_empty[s1]);
        }
      }
      umma::commit(&sm.drain[t]);  // nothing may be in flight when the tensor memory is freed
      if (!mbar_wait(&sm.drain[t], 0)) atomicOr(&d.hdr->err, kErrTimeout);
    }
  }
  __syncwarp();
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (warp == 12) umma::tmem_dealloc(tmem, 512);
}

// Joins the parts of the items that several blocks of the chunk kernel shared, in the blocks' order:
// 32 rows of an item a block, a warp's lanes along the rows.  (Joined by the last of the sharing
// blocks instead, 18 parts took that block 28 us.)
__global__ void __launch_bounds__(256) dense_join_kernel(ChunkArgs a, int chunk_blocks) {
  const DenseArgs &d = a.d;
  if (d.hdr->magic != kDenseMagic || d.hdr->rope_base != d.rope_base) return;
  constexpr int kBlocks = kItemRows / 32;
  const int item = blockIdx.x / kBlocks, row = blockIdx.x % kBlocks * 32 + (threadIdx.x & 31), piece0 = threadIdx.x >> 5;
  const int total = __ldg(a.prefix + a.items), blocks = sharing_blocks(total, chunk_blocks);
  const int w0 = __ldg(a.prefix + item), w1 = __ldg(a.prefix + item + 1);
  auto holder = [&](int w) {  // the block that holds key tile w
    int c = (int)((int64_t)w * blocks / total);
    while (dealt(total, blocks, c + 1) <= w) ++c;
    while (dealt(total, blocks, c) > w) --c;
    return c;
  };
  const int c0 = holder(w0), c1 = holder(w1 - 1);
  if (c0 == c1) return;
  const Item it = chunk_item(a, item);
  const int gs = d.group_shift, G = 1 << gs, hq = d.hkv << gs;
  if ((row >> gs) >= it.nq) return;
  // the item is in block c's first segment if the block begins inside it
  auto from = [&](int c) { return part_of(d, c, dealt(total, blocks, c) >= w0); };
  auto stats = [&](int c) { return __ldcg(reinterpret_cast<const float2 *>(from(c) + kItemRows * kD) + row); };
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) m = fmaxf(m, stats(c).x);
  float4 acc[4] = {};
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const float2 ml = stats(c);
    const float f = ml.x == -INFINITY ? 0.f : exp2_approx(ml.x - m);
    const float4 *src = reinterpret_cast<const float4 *>(from(c)) + row;
    l += f * ml.y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 u = __ldcg(src + (piece0 + 8 * i) * kItemRows);
      acc[i].x += f * u.x, acc[i].y += f * u.y, acc[i].z += f * u.z, acc[i].w += f * u.w;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  bool odd = !(l < INFINITY);
  uint16_t *const out = reinterpret_cast<uint16_t *>(d.out) +
                        (((int64_t)it.b * d.nq + it.q0 + (row >> gs)) * hq + it.h * G + (row & (G - 1))) * kD;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x[4] = {acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv};
#pragma unroll
    for (int k = 0; k < 4; ++k) odd |= !(fabsf(x[k]) < INFINITY);
    *reinterpret_cast<uint2 *>(out + (piece0 + 8 * i) * 4) = make_uint2(cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]));
  }
  if (odd) mark_again(a, it.b, it.h, it.q0 / (kItemRows >> gs));
}

// The most key tiles a head's queries see.
int64_t most_key_tiles(const DenseArgs &d) {
  const int64_t all = ceil_div(std::max(d.length, 1), kTile);
  if (!d.window) return all;
  return std::min<int64_t>(all, ceil_div((int64_t)d.window + (d.causal ? d.nq : 0), kTile) + 1) +
         std::min<int64_t>(all, ceil_div(d.sinks, kTile));
}

}  // namespace

int launch_dense_chunk(const DenseArgs &d, int64_t max_keys, int64_t image_bytes, void *stream) {
  ChunkArgs a = {};
  a.d = d;
  const int per = kItemRows >> d.group_shift;
  const int64_t chunk_tiles = ceil_div(d.nq, per), heads = (int64_t)d.batch * d.hkv;
  a.d.tiles = (int)chunk_tiles;
  a.redo = reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(d.hdr) + kDenseRedo);
  a.prefix = reinterpret_cast<int *>(reinterpret_cast<char *>(d.hdr) + kDensePrefix);
  a.key_tiles = (int)most_key_tiles(d);
  a.query_sets = d.window && d.sinks && d.rank_sinks ? 2 : 1;
  const int sms = std::min(dense_sm_count(), kMaxChunkBlocks);
  cudaError_t e = cudaFuncSetAttribute(dense_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kChunkSmem);
  if (e != cudaSuccess) return (int)e;
  // As many heads and items a launch as the images' room holds: an eighth of it for the queries
  // of one head, at least one item.
  const int64_t key_bytes = a.key_tiles * (int64_t)(kTileBytes + sizeof(uint4)), item_bytes = a.query_sets * (int64_t)kQueryBytes;
  const int64_t head_tiles = std::min(chunk_tiles, std::max<int64_t>(1, image_bytes / 8 / item_bytes));
  const int64_t fit = image_bytes / (key_bytes + head_tiles * item_bytes);
  if (fit < 1) return kNoRoom;
  const int64_t step = std::min(heads, fit), tiles = ceil_div(max_keys, kTile) + 1;
  for (int64_t bh0 = 0; bh0 < heads; bh0 += step) {
    a.bh0 = (int)bh0;
    a.heads = (int)std::min(step, heads - bh0);
    a.key_images = reinterpret_cast<unsigned char *>(d.hdr) + kDenseImages;
    a.query_images = a.key_images + (int64_t)a.heads * a.key_tiles * kTileBytes;
    a.live = reinterpret_cast<uint4 *>(a.query_images + a.heads * head_tiles * item_bytes);
    for (int64_t tile0 = 0; tile0 < chunk_tiles; tile0 += head_tiles) {
      a.tile0 = (int)tile0;
      a.tiles = (int)std::min(head_tiles, chunk_tiles - tile0);
      a.items = a.heads * a.tiles;
      // Dealing the key tiles out evenly costs a part's write and join (about four key tiles'
      // time) and saves the last wave's idle blocks.
      const int64_t plain = ceil_div(a.items, sms) * tiles, dealt = ceil_div(a.items * tiles, sms) + 4;
      a.shared = a.items <= kMaxShared && dealt < plain ? 1 : 0;
      const int keys = tile0 == 0 ? a.heads * a.key_tiles : 0;
      dense_images_kernel<<<(unsigned)(keys + (int64_t)a.items * a.query_sets * (kItemRows / kQueryRows)), kLoadThreads, 0,
                            (cudaStream_t)stream>>>(a, keys);
      e = cudaGetLastError();
      if (e != cudaSuccess) return (int)e;
      const int64_t work = a.shared ? a.items * tiles : a.items;
      const int blocks = (int)std::min<int64_t>(work, sms);
      dense_chunk_kernel<<<(unsigned)blocks, kChunkThreads, kChunkSmem, (cudaStream_t)stream>>>(a);
      if (a.shared) dense_join_kernel<<<(unsigned)(a.items * (kItemRows / 32)), 256, 0, (cudaStream_t)stream>>>(a, blocks);
      e = cudaGetLastError();
      if (e != cudaSuccess) return (int)e;
    }
  }
  return launch_dense_redo(d, a.d.tiles, stream);
}

}  // namespace recsa
