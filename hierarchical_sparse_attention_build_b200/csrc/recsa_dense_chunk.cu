// Dense attention of a chunk of queries on the 5th-generation tensor cores (bf16 outputs).
//
// A work item is 256 query rows (256 / G queries x the G heads of one KV group) of one
// sequence, as two tiles of 128 rows; its keys come in tiles of 128.  One CTA per SM:
//   warps 0-3, 4-7 : softmax of the two row tiles, a thread a row (scores and probabilities in
//                    TMEM), the rescaling of the outputs and the epilogue;
//   warps 8-11     : loaders: rotate the keys to their positions (registers -> swizzled shared
//                    memory), gather the values with cp.async, rotate the queries;
//   warp 12        : one thread issues the products: S = Q K^T (shared x shared) and
//                    O += P V (TMEM x shared).
// While one row tile's softmax runs, the tensor cores do the other's O += P V and next S.
//
// Rounding: rotated queries and keys are rounded to fp16 (11 bits; half the steps of the
// output's bf16 even after the sum over 128 terms), probabilities to bf16 (the values' type: one
// product takes one type).  A rotated element beyond fp16's range, or an output that is not
// finite (a hidden token's value may hold anything, and a zero weight times infinity is NaN),
// marks the item: the rows kernel, which has neither limit, then computes it again.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include <cuda_fp16.h>

#include "recsa_dense.cuh"
#include "recsa_umma.cuh"

namespace recsa {
namespace {

constexpr int kTile = 128;                  // rows of a row tile, keys of a key tile
constexpr int kItemRows = 2 * kTile;
constexpr int kSoftWarps = 8;
constexpr int kLoadThreads = 128;
constexpr int kTileBytes = kTile * kRowBytes;  // 32 KB: [64-element half][row][128 bytes], 16-byte pieces XOR row % 8
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kRing = 2;                    // key and value tiles in shared memory
constexpr int kMaxChunkBlocks = (int)(kDensePartBytes / (2 * kItemRows * kPartRow * sizeof(float)));
constexpr int kImageTiles = 2;              // items a head from which images are made
constexpr float kRescale = 8.f;             // a row's maximum may lag by 2^8 before its output is rescaled

struct ChunkSmem {
  unsigned char q[2][kTileBytes];
  unsigned char k[kRing][kTileBytes];
  unsigned char v[kRing][kTileBytes];
  uint32_t live[4][4][4];                   // a key tile's tokens that were loaded, by tile % 4: a part a loader warp
  alignas(16) uint64_t k_full[kRing], k_empty[kRing], v_full[kRing], v_empty[kRing];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t join, joined, drain;
  uint32_t tmem;
  uint32_t stop;                            // a wait ran out: every role leaves
  int last;
  int scan[16];
  int prefix[kMaxShared + 1];               // key tiles before each item, when items are shared
};

constexpr size_t kChunkSmem = sizeof(ChunkSmem) + 1024;  // the tiles begin on 1024 bytes

struct ChunkArgs {
  DenseArgs d;
  int bh0, heads;  // the launch's (sequence, KV head) pairs
  int items;     // work items
  int shared;    // 1: the key tiles of all items are dealt out evenly to the blocks
  uint32_t *redo;
  // rotated rows as the tiles' shared-memory images (IMG): keys [heads][key_tiles], their loaded
  // tokens, queries [items][1 or 2: for the window's tokens, for the sinks][2 row tiles]
  unsigned char *key_images, *query_images;
  uint4 *live;
  int key_tiles, query_sets;
};
__device__ __forceinline__ uint32_t &redo_mark(const ChunkArgs &a, int item) {
  return a.redo[(a.bh0 * a.d.tiles + item) % kMaxShared];
}

__host__ __device__ constexpr uint32_t chunk_idesc(bool bf16, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(kTile >> 3) << 17) |
         ((uint32_t)(kTile >> 4) << 24);
}
// Descriptor of a 128-byte-swizzled operand: rows of 128 bytes, 8 rows 1024 bytes apart.  K-major
// (queries, keys): a k-step of 16 elements is 32 bytes further into the row.  MN-major (values): the
// rows are keys, the second 64 dimensions lie kHalfBytes further (the leading-dimension step).
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3fffu) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(
          d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// What a role knows of the item it is at.
struct Item {
  int b, h, q0, nq;       // sequence, KV head, first query, queries
  int len, p_min, p_max;  // tokens; positions of the first and last query
  int hi1, n1;            // sinks: tokens, key tiles
  int lo2, hi2, first;    // the window's tokens; its first key tile
  int tiles;              // key tiles (at least one, which may hold nothing)
};
__device__ __forceinline__ Item chunk_item(const ChunkArgs &a, int item) {
  const DenseArgs &d = a.d;
  Item it;
  const int bh = a.bh0 + item / d.tiles, tile = d.tiles - 1 - item % d.tiles;  // the longest ranges first
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
__device__ __forceinline__ int sharing_blocks(int total) { return min((int)gridDim.x, total); }
__device__ __forceinline__ Segments segments_begin(const ChunkArgs &a, const ChunkSmem &sm) {
  Segments s;
  s.j0 = s.j1 = 0;
  s.at = s.end = s.begin = 0;
  s.item = blockIdx.x;
  if (a.shared) {
    const int total = sm.prefix[a.items], blocks = sharing_blocks(total);
    if ((int)blockIdx.x >= blocks) return s;
    s.begin = s.at = dealt(total, blocks, blockIdx.x);
    s.end = dealt(total, blocks, blockIdx.x + 1);
    int lo = 0, hi = a.items - 1;  // the item that holds key tile `at`
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (sm.prefix[mid] <= s.at) lo = mid; else hi = mid - 1;
    }
    s.item = lo - 1;
  } else {
    s.item -= gridDim.x;
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

__device__ __forceinline__ bool wait_or_stop(ChunkSmem &sm, const ChunkArgs &a, uint64_t *bar, uint32_t parity) {
  for (uint32_t i = 0; i < kMbarPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*(volatile uint32_t *)&sm.stop) return false;
  }
  *(volatile uint32_t *)&sm.stop = 1u;
  atomicOr(&a.d.hdr->err, kErrTimeout);
  return false;
}

// Rotation state of eight frequencies: cos and sin of a position, advanced by a fixed step.
struct Turn {
  F2 c[4], s[4];
  __device__ __forceinline__ void set(const uint64_t *f, int pos) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 r0 = rotation(pos, __ldg(f + 2 * i)), r1 = rotation(pos, __ldg(f + 2 * i + 1));
      c[i] = f2(r0.x, r1.x);
      s[i] = f2(r0.y, r1.y);
    }
  }
  __device__ __forceinline__ void advance(const Turn &d) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 u = f2_fma(f2_neg(s[i]), d.s[i], f2_mul(c[i], d.c[i]));
      s[i] = f2_fma(c[i], d.s[i], f2_mul(s[i], d.c[i]));
      c[i] = u;
    }
  }
};

// Dimensions 8 ch .. 8 ch + 7 and 64 more of one bf16 row, turned and rounded to fp16; `most`
// keeps the largest magnitudes.
template <bool SCALE>
__device__ __forceinline__ void turn_row(const uint4 &lo, const uint4 &hi, const Turn &t, float scale, uint4 &out_lo,
                                         uint4 &out_hi, __half2 &most) {
  const uint32_t x[4] = {lo.x, lo.y, lo.z, lo.w}, y[4] = {hi.x, hi.y, hi.z, hi.w};
  uint32_t u[4], v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    F2 p = f2_bf16(x[i]), q = f2_bf16(y[i]);
    if (SCALE) {
      p = f2_mul(p, f2(scale, scale));
      q = f2_mul(q, f2(scale, scale));
    }
    const float2 a2 = f2_get(f2_fma(q, f2_neg(t.s[i]), f2_mul(p, t.c[i])));
    const float2 b2 = f2_get(f2_fma(p, t.s[i], f2_mul(q, t.c[i])));
    const __half2 a = __floats2half2_rn(a2.x, a2.y), b = __floats2half2_rn(b2.x, b2.y);
    most = __hmax2(most, __hmax2(__habs2(a), __habs2(b)));
    u[i] = *reinterpret_cast<const uint32_t *>(&a);
    v[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  out_lo = make_uint4(u[0], u[1], u[2], u[3]);
  out_hi = make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void put_row(unsigned char *tile, int row, int ch, const uint4 &lo, const uint4 &hi) {
  unsigned char *p = tile + row * 128 + ((ch ^ (row & 7)) << 4);
  *reinterpret_cast<uint4 *>(p) = lo;
  *reinterpret_cast<uint4 *>(p + kHalfBytes) = hi;
}

// The item's query rows, turned to their positions (sinks: their positions for the sinks).
__device__ __forceinline__ void load_queries(const ChunkArgs &a, unsigned char *q, const Item &it, bool sink, int lt,
                                             __half2 &most) {
  const DenseArgs &d = a.d;
  const int ch = lt & 7, gs = d.group_shift, G = 1 << gs, hq = d.hkv << gs;
  const uint64_t *f = ws_freq(d.hdr) + ch * 8;
  Turn t, step;
  // rows lt / 8 + 16 i: for the window their positions advance by 16 / G a step
  const bool even = !sink || !d.rank_sinks;
  step.set(f, d.causal ? 16 >> gs : 0);
  t.set(f, dense_position(d, it.len, it.q0 + ((lt >> 3) >> gs)));
#pragma unroll 1
  for (int i = 0; i < kItemRows / 16; ++i) {
    const int row = (lt >> 3) + 16 * i, qi = row >> gs;
    if (!even) t.set(f, sink_position(d, dense_position(d, it.len, it.q0 + qi)));
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (qi < it.nq) {
      const uint4 *src = reinterpret_cast<const uint4 *>(
          d.q + (((int64_t)it.b * d.nq + it.q0 + qi) * hq + it.h * G + (row & (G - 1))) * kD);
      lo = __ldg(src + ch);
      hi = __ldg(src + ch + 8);
    }
    uint4 ol, oh;
    turn_row<true>(lo, hi, t, d.qscale, ol, oh, most);
    put_row(q + (row >> 7) * kTileBytes, row & 127, ch, ol, oh);
    if (even) t.advance(step);
  }
}

__device__ __forceinline__ bool beyond_half(__half2 most) {
  return __hgt(__hmax(__low2half(most), __high2half(most)), __float2half(65504.f));
}

// Rotated keys and queries of a launch as the chunk kernel's shared-memory images, so that it
// fetches a tile with one bulk copy.  A block turns one key tile or one item's query rows.
__global__ void __launch_bounds__(kLoadThreads) dense_images_kernel(ChunkArgs a) {
  const DenseArgs &d = a.d;
  if (d.hdr->magic != kDenseMagic || d.hdr->rope_base != d.rope_base) return;  // the chunk kernel reports it
  const int lt = threadIdx.x, ch = lt & 7, r0 = lt >> 3;
  __half2 most = __floats2half2_rn(0.f, 0.f);
  const int keys = a.heads * a.key_tiles;
  if ((int)blockIdx.x >= keys) {
    const int e = blockIdx.x - keys, item = e / a.query_sets;
    load_queries(a, a.query_images + (int64_t)e * (2 * kTileBytes), chunk_item(a, item), e % a.query_sets == 1, lt, most);
    if (beyond_half(most)) redo_mark(a, item) = 1u;
    return;
  }
  const int hl = blockIdx.x / a.key_tiles, kt = blockIdx.x % a.key_tiles;
  const int b = (a.bh0 + hl) / d.hkv, h = (a.bh0 + hl) % d.hkv;
  const int len = dense_length(d, b, false);
  const HeadRange hr = head_range(d, len);
  if (kt >= hr.count) return;
  const int T = (kt < hr.n1 ? kt : hr.first + kt - hr.n1) * kTile;
  unsigned char *const tile = a.key_images + (int64_t)blockIdx.x * kTileBytes;
  Turn t, step;
  const uint64_t *f = ws_freq(d.hdr) + ch * 8;
  t.set(f, T + r0);
  step.set(f, 16);
  uint32_t word[4] = {0u, 0u, 0u, 0u};
  uint4 xl[8], xh[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int tok = T + r0 + 16 * i;
    xl[i] = xh[i] = make_uint4(0, 0, 0, 0);
    if (tok < len) {
      const int64_t r = cache_row(d, b, h, tok);
      if (r >= 0) {
        const uint4 *src = reinterpret_cast<const uint4 *>(d.k + r * kD);
        xl[i] = __ldg(src + ch);
        xh[i] = __ldg(src + ch + 8);
        word[i >> 1] |= 1u << (r0 + 16 * (i & 1));
      } else {
        atomicOr(&d.hdr->err, kErrIndex);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint4 ol, oh;
    turn_row<false>(xl[i], xh[i], t, 1.f, ol, oh, most);
    put_row(tile, r0 + 16 * i, ch, ol, oh);
    t.advance(step);
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
    for (int tile_i = 0; tile_i < d.tiles; ++tile_i) redo_mark(a, hl * d.tiles + tile_i) = 1u;
}

// One bulk copy of `bytes` (a multiple of 16) into shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// IMG: keys and queries come rotated, as images (dense_images_kernel); otherwise the loaders
// rotate them.  Registers a thread: 16 warps launched with 128 give the softmax 192, the loaders
// 72 and the last four warps 56 (65,536 in all); without images 13 warps launched with 128 give
// 112, 152 and 128 (52,224 of 53,248).
template <bool IMG>
__global__ void __launch_bounds__(IMG ? 512 : 416, 1) dense_chunk_kernel(ChunkArgs a) {
  constexpr int kChunkThreads = IMG ? 512 : 416;
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
      mbar_init(&sm.k_full[i], IMG ? 1 : kLoadThreads);
      mbar_init(&sm.v_full[i], kLoadThreads);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_full[t], 4);
      mbar_init(&sm.o_full[t], 1);
    }
    mbar_init(&sm.join, kSoftWarps);
    mbar_init(&sm.joined, 1);
    mbar_init(&sm.drain, 1);
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
  const uint32_t tmem = sm.tmem;
  Segments sg = segments_begin(a, sm);
  Item it;

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------------ softmax and epilogue
    if constexpr (IMG)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
    const int t = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const uint32_t ts = tmem + lanes + t * kTile, to = tmem + lanes + 2 * kTile + t * kTile;
    const int row = t * kTile + (warp & 3) * 32 + lane, gs = d.group_shift, G = 1 << gs, hq = d.hkv << gs;
    uint32_t n_s = 0, n_o = 0, n_join = 0, n_tile = 0;  // phases of s_full, o_full and join, key tiles seen
    bool ok = true;
    while (ok && segments_next(a, sm, sg, it)) {
      const bool in = (row >> gs) < it.nq;
      const int p = in ? dense_position(d, it.len, it.q0 + (row >> gs)) : 0;
      const int lo = window_first(d, p), hi = p, hi_sink = min(p, it.hi1);
      float m = -INFINITY, l = 0.f;
      for (int j = sg.j0; j < sg.j1; ++j, ++n_tile) {
        const bool sink = j < it.n1;
        const int T = (sink ? j : it.first + j - it.n1) * kTile;
        const int a0 = (sink ? 0 : lo) - T, a1 = (sink ? hi_sink : hi) - T;  // visible columns [a0, a1)
        if (!wait_or_stop(sm, a, &sm.s_full[t], n_s & 1)) {
          ok = false;
          break;
        }
        ++n_s;
        umma::fence_after_sync();
        uint32_t live[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int w = 0; w < (IMG ? 1 : 4); ++w) {
          const uint4 lv = *reinterpret_cast<const uint4 *>(sm.live[n_tile & 3][w]);
          live[0] |= lv.x, live[1] |= lv.y, live[2] |= lv.z, live[3] |= lv.w;
        }
        const bool whole = a0 <= 0 && a1 >= kTile && (live[0] & live[1] & live[2] & live[3]) == 0xffffffffu;
        const bool masked = __any_sync(0xffffffffu, !whole);
        float x = -INFINITY;
        [[maybe_unused]] uint32_t sr[IMG ? 4 : 1][32];  // the row's scores
        if constexpr (IMG) {
#pragma unroll
          for (int g = 0; g < 4; ++g) umma::tmem_ld32(ts + g * 32, sr[g]);
          umma::tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int c = g * 32 + i;
                if (c < a0 || c >= a1 || !((live[g] >> i) & 1u)) sr[g][i] = 0xff800000u;
              }
          }
          float xs[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; i += 2)
#pragma unroll
            for (int g = 0; g < 4; ++g) xs[g] = max3(xs[g], __uint_as_float(sr[g][i]), __uint_as_float(sr[g][i + 1]));
          x = fmaxf(fmaxf(xs[0], xs[1]), fmaxf(xs[2], xs[3]));
        } else {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t s[32];
            umma::tmem_ld32(ts + g * 32, s);
            umma::tmem_wait_ld();
            if (masked) {
              const uint32_t w = live[g];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int c = g * 32 + i;
                if (c < a0 || c >= a1 || !((w >> i) & 1u)) s[i] = 0xff800000u;
              }
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) x = max3(x, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
          }
        }
        const bool up = x > m + kRescale || (m == -INFINITY && x > m);
        if (__any_sync(0xffffffffu, up)) {
          const float f = up ? (m == -INFINITY ? 0.f : exp2_approx(m - x)) : 1.f;
          if (up) {
            m = x;
            l *= f;
          }
          if (j > sg.j0) {
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
              uint32_t o[32];
              umma::tmem_ld32(to + g * 32, o);
              umma::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st32(to + g * 32, o);
            }
            tmem_wait_st();
          }
        }
        const float z = m == -INFINITY ? 0.f : m;
        const F2 nz = f2(-z, -z);
        F2 sum = f2(0.f, 0.f);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t s[32], pk[16];
          if constexpr (IMG) {
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = sr[g][i];
          } else {
            umma::tmem_ld32(ts + g * 32, s);
            umma::tmem_wait_ld();
            if (masked) {
              const uint32_t w = live[g];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int c = g * 32 + i;
                if (c < a0 || c >= a1 || !((w >> i) & 1u)) s[i] = 0xff800000u;
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x2 = f2_get(f2_add(f2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), nz));
            const float e0 = exp2_approx(x2.x), e1 = exp2_approx(x2.y);
            sum = f2_add(sum, f2(e0, e1));
            pk[i] = cvt_bf16x2(e0, e1);
          }
          tmem_st16(ts + g * 16, pk);  // over columns that were read
        }
        l += f2_get(sum).x + f2_get(sum).y;
        tmem_wait_st();
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[t]);
      }
      if (!ok || !wait_or_stop(sm, a, &sm.o_full[t], n_o & 1)) break;
      ++n_o;
      umma::fence_after_sync();
      // epilogue: the item's output, or this block's part of it
      const bool part = sg.j1 - sg.j0 < it.tiles;
      const bool first_seg = sg.at - (sg.j1 - sg.j0) == sg.begin;
      float *const pr = ws_part(d.hdr) + (((int64_t)blockIdx.x * 2 + (first_seg ? 0 : 1)) * kItemRows + row) * kPartRow;
      const int64_t out_row = ((int64_t)it.b * d.nq + it.q0 + (row >> gs)) * hq + it.h * G + (row & (G - 1));
      uint4 *const po = reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(d.out) + out_row * kD);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      bool odd = !(l < INFINITY);
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        uint32_t o[32];
        umma::tmem_ld32(to + g * 32, o);
        umma::tmem_wait_ld();
        if (part) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(pr + 4 + g * 32 + i * 4) =
                make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float u = __uint_as_float(o[2 * i]) * inv, v = __uint_as_float(o[2 * i + 1]) * inv;
            odd |= !(fabsf(u) < INFINITY) || !(fabsf(v) < INFINITY);
            w[i] = cvt_bf16x2(u, v);
          }
          if (in) {
#pragma unroll
            for (int i = 0; i < 4; ++i) po[g * 4 + i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        }
      }
      umma::fence_before_sync();
      if (part) {
        *reinterpret_cast<float2 *>(pr) = make_float2(m, l);
        odd = false;
        // the item's key tiles are spread over blocks c0 .. c1: the last to arrive joins them in order
        const int total = sm.prefix[a.items], blocks = sharing_blocks(total);
        const int w0 = sm.prefix[sg.item], w1 = w0 + it.tiles;
        auto holder = [&](int w) {  // the block that holds key tile w
          int c = (int)((int64_t)w * blocks / total);
          while (dealt(total, blocks, c + 1) <= w) ++c;
          while (dealt(total, blocks, c) > w) --c;
          return c;
        };
        const int c0 = holder(w0), c1 = holder(w1 - 1);
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.join);
        if (!wait_or_stop(sm, a, &sm.join, n_join & 1)) break;
        if (tid == 0) {
          const int done = atomicAdd(ws_count(d.hdr) + sg.item, 1);
          sm.last = done == c1 - c0;
          if (sm.last) ws_count(d.hdr)[sg.item] = 0;  // for the next call
          __threadfence();
          mbar_arrive(&sm.joined);
        }
        if (!wait_or_stop(sm, a, &sm.joined, n_join & 1)) break;
        ++n_join;
        __threadfence();
        if (sm.last) {
          auto from = [&](int c) {
            // the item is in block c's first segment if the block begins inside it
            return ws_part(d.hdr) +
                   (((int64_t)c * 2 + (dealt(total, blocks, c) >= w0 ? 0 : 1)) * kItemRows + row) * kPartRow;
          };
          float mm = -INFINITY, ll = 0.f;
          for (int c = c0; c <= c1; ++c) mm = fmaxf(mm, __ldcg(from(c)));
          for (int c = c0; c <= c1; ++c) {
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(from(c)));
            if (ml.x != -INFINITY) ll += ml.y * exp2_approx(ml.x - mm);
          }
          const float iv = ll == 0.f ? 0.f : 1.f / ll;
          odd = !(ll < INFINITY);
#pragma unroll 1
          for (int g = 0; g < 16; ++g) {
            float acc[8] = {};
            for (int c = c0; c <= c1; ++c) {
              const float *q = from(c);
              const float mc = __ldcg(q);
              if (mc == -INFINITY) continue;
              const float f = exp2_approx(mc - mm) * iv;
              const float4 u = __ldcg(reinterpret_cast<const float4 *>(q + 4 + g * 8));
              const float4 v = __ldcg(reinterpret_cast<const float4 *>(q + 8 + g * 8));
              acc[0] += f * u.x, acc[1] += f * u.y, acc[2] += f * u.z, acc[3] += f * u.w;
              acc[4] += f * v.x, acc[5] += f * v.y, acc[6] += f * v.z, acc[7] += f * v.w;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) odd |= !(fabsf(acc[i]) < INFINITY);
            if (in)
              po[g] = make_uint4(cvt_bf16x2(acc[0], acc[1]), cvt_bf16x2(acc[2], acc[3]), cvt_bf16x2(acc[4], acc[5]),
                                 cvt_bf16x2(acc[6], acc[7]));
          }
        }
      }
      if (odd && in) redo_mark(a, sg.item) = 1u;
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ loaders
    if constexpr (IMG)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    const int lt = tid - kSoftWarps * 32, ch = lt & 7;
    const uint64_t *f = ws_freq(d.hdr) + ch * 8;
    const int r0 = lt >> 3;  // this thread's rows: r0 + 16 i
    [[maybe_unused]] Turn step, t;
    if constexpr (!IMG) step.set(f, 16);
    uint32_t n = 0;  // key tiles loaded
    bool ok = true;
    while (ok && segments_next(a, sm, sg, it)) {
      __half2 most = __floats2half2_rn(0.f, 0.f);
      // Rows of key tile j in the caches (fewer than 2^32 rows fit a GPU); bit i of the result:
      // this thread's row i is a token of the range on a page of the pool.
      uint32_t rows[8], here;
      auto place = [&](int j) {
        const bool sink = j < it.n1;
        const int T = (sink ? j : it.first + j - it.n1) * kTile;
        const int lo = sink ? 0 : it.lo2, hi = sink ? it.hi1 : it.hi2;
        here = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = T + r0 + 16 * i;
          rows[i] = 0;
          if (tok >= lo && tok < hi) {
            const int64_t r = cache_row(d, it.b, it.h, tok);
            if (r >= 0) {
              rows[i] = (uint32_t)r;
              here |= 1u << i;
            } else if (!IMG) {
              atomicOr(&d.hdr->err, kErrIndex);
            }
          }
        }
      };
      [[maybe_unused]] uint4 xl[2][4], xh[2][4];  // raw keys of half a tile, the next half in flight while one is turned
      auto fetch = [&](int hf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool on = (here >> (hf * 4 + i)) & 1u;
          const uint4 *src = reinterpret_cast<const uint4 *>(d.k + (int64_t)rows[hf * 4 + i] * kD);
          xl[hf][i] = on ? __ldg(src + ch) : make_uint4(0, 0, 0, 0);
          xh[hf][i] = on ? __ldg(src + ch + 8) : make_uint4(0, 0, 0, 0);
        }
      };
      auto turn = [&](int hf, int s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 ol, oh;
          turn_row<false>(xl[hf][i], xh[hf][i], t, 1.f, ol, oh, most);
          put_row(sm.k[s], r0 + 16 * (hf * 4 + i), ch, ol, oh);
          t.advance(step);
        }
      };
      place(sg.j0);
      if constexpr (!IMG) fetch(0);
      for (int j = sg.j0; j < sg.j1; ++j, ++n) {
        const bool sink = j < it.n1;
        const int s = n % kRing;
        const uint32_t round = n / kRing;
        if (!IMG && (j == sg.j0 || (j == it.n1 && j > 0))) {
          // the queries of a new segment, or of the window after the sinks: the products that
          // read the last ones are done once the previous key tile is free
          if (n > 0 && !wait_or_stop(sm, a, &sm.k_empty[(n - 1) % kRing], ((n - 1) / kRing) & 1)) {
            ok = false;
            break;
          }
          load_queries(a, sm.q[0], it, sink, lt, most);
        }
        // The rotation goes on from tile to tile (16 positions a row, 128 a tile) and starts anew
        // every 16 tiles: 128 steps of fp32 rounding are below 2^-16, fp16 rounds at 2^-11.
        if (!IMG && (j == sg.j0 || j == it.n1 || ((j - sg.j0) & 15) == 0))
          t.set(f, (sink ? j : it.first + j - it.n1) * kTile + r0);
        if (round > 0 && !wait_or_stop(sm, a, &sm.v_empty[s], (round - 1) & 1)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t dst = smem_u32(sm.v[s]) + (r0 + 16 * i) * 128 + ((ch ^ (r0 & 7)) << 4);
          const bool on = (here >> i) & 1u;
          const uint16_t *src = d.v + (int64_t)rows[i] * kD + ch * 8;
          cp_async16(dst, src, on);
          cp_async16(dst + kHalfBytes, src + kHalf, on);
        }
        cp_async_commit();
        if constexpr (IMG) {
          if (j + 1 < sg.j1) place(j + 1);
          cp_async_wait<0>();
          umma::fence_async_smem();
          mbar_arrive(&sm.v_full[s]);
          continue;
        }
        fetch(1);
        if (round > 0 && !wait_or_stop(sm, a, &sm.k_empty[s], (round - 1) & 1)) {
          ok = false;
          break;
        }
        {  // live tokens, each warp its rows: word w of the tile is tokens 32 w .. 32 w + 31
          uint32_t word[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int i = 0; i < 8; ++i) word[i >> 1] |= ((here >> i) & 1u) << (r0 + 16 * (i & 1));
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            word[w] |= __shfl_xor_sync(0xffffffffu, word[w], 8);
            word[w] |= __shfl_xor_sync(0xffffffffu, word[w], 16);
          }
          if (lane == 0)
            *reinterpret_cast<uint4 *>(sm.live[n & 3][warp - kSoftWarps]) = make_uint4(word[0], word[1], word[2], word[3]);
        }
        turn(0, s);
        if (j + 1 < sg.j1) {
          place(j + 1);
          fetch(0);
        }
        turn(1, s);
        umma::fence_async_smem();
        mbar_arrive(&sm.k_full[s]);
        cp_async_wait<0>();
        umma::fence_async_smem();
        mbar_arrive(&sm.v_full[s]);
      }
      if (!IMG && beyond_half(most)) redo_mark(a, sg.item) = 1u;
    }
    cp_async_wait<0>();
  } else {
    if constexpr (IMG) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (IMG && warp == 13 && lane == 0) {
      // ---------------------------------------------------------------- images
      uint32_t n = 0;
      bool ok = true;
      while (ok && segments_next(a, sm, sg, it)) {
        const HeadRange hr = head_range(d, it.len);
        const int hl = it.b * d.hkv + it.h - a.bh0;
        for (int j = sg.j0; j < sg.j1; ++j, ++n) {
          const bool sink = j < it.n1;
          const int s = n % kRing;
          const int kt = min(sink ? j : hr.n1 + it.first + j - it.n1 - hr.first, a.key_tiles - 1);
          const int64_t image = (int64_t)hl * a.key_tiles + kt;
          const bool queries = j == sg.j0 || (j == it.n1 && j > 0);
          // new queries: the products that read the last ones are done once the previous tile is free
          if (queries && n > 0 && !wait_or_stop(sm, a, &sm.k_empty[(n - 1) % kRing], ((n - 1) / kRing) & 1)) {
            ok = false;
            break;
          }
          if (n >= kRing && !wait_or_stop(sm, a, &sm.k_empty[s], (n / kRing - 1) & 1)) {
            ok = false;
            break;
          }
          *reinterpret_cast<uint4 *>(sm.live[n & 3][0]) = __ldg(a.live + image);
          mbar_expect(&sm.k_full[s], kTileBytes + (queries ? 2 * kTileBytes : 0));
          if (queries)
            bulk_load(smem_u32(sm.q[0]),
                      a.query_images + ((int64_t)sg.item * a.query_sets + (sink ? 1 : 0)) * (2 * kTileBytes),
                      2 * kTileBytes, &sm.k_full[s]);
          bulk_load(smem_u32(sm.k[s]), a.key_images + image * kTileBytes, kTileBytes, &sm.k_full[s]);
        }
      }
      // every copy has landed before the block may end
      if (n > 0) mbar_wait(&sm.k_full[(n - 1) % kRing], ((n - 1) / kRing) & 1);
      if (n > 1) mbar_wait(&sm.k_full[(n - 2) % kRing], ((n - 2) / kRing) & 1);
    }
  }
  if (warp == 12 && lane == 0) {
    // ------------------------------------------------------------------ products
    uint32_t n = 0;         // key tiles
    uint32_t n_p = 0;       // phases of p_full
    bool ok = true;
    auto scores = [&](int t, int s) {
      const uint32_t q = smem_u32(sm.q[t]), k = smem_u32(sm.k[s]);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t off = (ks >> 2) * kHalfBytes + (ks & 3) * 32;
        umma::mma(tmem + t * kTile, swizzled_desc(q + off, 16), swizzled_desc(k + off, 16), chunk_idesc(false, false),
                  ks > 0);
      }
      umma::commit(&sm.s_full[t]);
    };
    while (ok && segments_next(a, sm, sg, it)) {
      const int count = sg.j1 - sg.j0;
      if (!wait_or_stop(sm, a, &sm.k_full[n % kRing], (n / kRing) & 1)) break;
      umma::fence_after_sync();
      scores(0, n % kRing);
      scores(1, n % kRing);
      umma::commit(&sm.k_empty[n % kRing]);
      for (int j = 0; j < count; ++j, ++n, ++n_p) {
        const int s = n % kRing, s1 = (n + 1) % kRing;
        if (!wait_or_stop(sm, a, &sm.v_full[s], (n / kRing) & 1)) {
          ok = false;
          break;
        }
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          if (!wait_or_stop(sm, a, &sm.p_full[t], n_p & 1)) {
            ok = false;
            break;
          }
          umma::fence_after_sync();
          const uint32_t v = smem_u32(sm.v[s]);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_tmem_a(tmem + 2 * kTile + t * kTile, tmem + t * kTile + ks * 8, swizzled_desc(v + ks * 2048, kHalfBytes),
                       chunk_idesc(true, true), j > 0 || ks > 0);
          if (t == 1) umma::commit(&sm.v_empty[s]);
          if (j + 1 < count) {
            if (t == 0) {
              if (!wait_or_stop(sm, a, &sm.k_full[s1], ((n + 1) / kRing) & 1)) {
                ok = false;
                break;
              }
              umma::fence_after_sync();
            }
            scores(t, s1);
            if (t == 1) umma::commit(&sm.k_empty[s1]);
          } else {
            umma::commit(&sm.o_full[t]);
          }
        }
        if (!ok) break;
      }
    }
    umma::commit(&sm.drain);  // nothing may be in flight when the tensor memory is freed
    if (!mbar_wait(&sm.drain, 0)) atomicOr(&d.hdr->err, kErrTimeout);
  }
  __syncwarp();
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (warp == 12) umma::tmem_dealloc(tmem, 512);
}

}  // namespace

namespace {

template <bool IMG>
int run_chunk(const ChunkArgs &a, int64_t tiles, void *stream) {
  const int sms = std::min(dense_sm_count(), kMaxChunkBlocks);
  cudaError_t e = cudaFuncSetAttribute(dense_chunk_kernel<IMG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kChunkSmem);
  if (e != cudaSuccess) return (int)e;
  const int64_t work = a.shared ? a.items * tiles : a.items;
  dense_chunk_kernel<IMG><<<(unsigned)std::min<int64_t>(work, sms), IMG ? 512 : 416, kChunkSmem, (cudaStream_t)stream>>>(a);
  return (int)cudaGetLastError();
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
  a.d.tiles = (d.nq + per - 1) / per;
  const int64_t heads = (int64_t)d.batch * d.hkv;
  a.redo = reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(d.hdr) + kDenseRedo);
  const int sms = std::min(dense_sm_count(), kMaxChunkBlocks);
  const int64_t tiles = ceil_div(max_keys, kTile) + 1;
  // Rotated images pay once two items share a key tile; as many heads a launch as they fit.
  a.key_tiles = (int)most_key_tiles(d);
  a.query_sets = d.window && d.sinks && d.rank_sinks ? 2 : 1;
  const int64_t head_bytes = a.key_tiles * (int64_t)(kTileBytes + sizeof(uint4)) +
                             (int64_t)a.d.tiles * a.query_sets * 2 * kTileBytes;
  const int64_t fit = image_bytes / head_bytes;
  const bool images = a.d.tiles >= kImageTiles && fit >= 1;
  const int64_t step = images ? std::min(heads, fit) : heads;
  for (int64_t bh0 = 0; bh0 < heads; bh0 += step) {
    a.bh0 = (int)bh0;
    a.heads = (int)std::min(step, heads - bh0);
    a.items = a.heads * a.d.tiles;
    // Dealing the key tiles out evenly costs a part's write and join (about four key tiles'
    // time) and saves the last wave's idle blocks.
    const int64_t plain = ceil_div(a.items, sms) * tiles, dealt = ceil_div(a.items * tiles, sms) + 4;
    a.shared = a.items <= kMaxShared && dealt < plain ? 1 : 0;
    int rc;
    if (images) {
      a.key_images = reinterpret_cast<unsigned char *>(d.hdr) + kDenseImages;
      a.query_images = a.key_images + (int64_t)a.heads * a.key_tiles * kTileBytes;
      a.live = reinterpret_cast<uint4 *>(a.query_images + (int64_t)a.items * a.query_sets * 2 * kTileBytes);
      dense_images_kernel<<<(unsigned)(a.heads * a.key_tiles + a.items * a.query_sets), kLoadThreads, 0,
                            (cudaStream_t)stream>>>(a);
      rc = (int)cudaGetLastError();
      if (rc == 0) rc = run_chunk<true>(a, tiles, stream);
    } else {
      rc = run_chunk<false>(a, tiles, stream);
    }
    if (rc) return rc;
  }
  return launch_dense_redo(d, a.d.tiles, stream);
}

}  // namespace recsa
