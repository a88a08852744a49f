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
constexpr int kChunkThreads = 13 * 32;
constexpr int kTileBytes = kTile * kRowBytes;  // 32 KB: [64-element half][row][128 bytes], 16-byte pieces XOR row % 8
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kRing = 2;                    // key and value tiles in shared memory
constexpr int kMaxChunkBlocks = (int)(kDensePartBytes / (2 * kItemRows * kPartRow * sizeof(float)));
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
  int items;     // work items
  int shared;    // 1: the key tiles of all items are dealt out evenly to the blocks
  uint32_t *redo;
};

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
  const int bh = item / d.tiles, tile = d.tiles - 1 - item % d.tiles;  // the longest ranges first
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
  float c[8], s[8];
  __device__ __forceinline__ void set(const uint64_t *f, int pos) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 r = rotation(pos, __ldg(f + i));
      c[i] = r.x;
      s[i] = r.y;
    }
  }
  __device__ __forceinline__ void advance(const Turn &d) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = c[i] * d.c[i] - s[i] * d.s[i];
      s[i] = s[i] * d.c[i] + c[i] * d.s[i];
      c[i] = u;
    }
  }
};

// Dimensions 8 ch .. 8 ch + 7 and 64 more of one bf16 row, turned and rounded to fp16; `most`
// keeps the largest magnitudes.
__device__ __forceinline__ void turn_row(const uint4 &lo, const uint4 &hi, const Turn &t, float scale, uint4 &out_lo,
                                         uint4 &out_hi, __half2 &most) {
  const uint32_t x[4] = {lo.x, lo.y, lo.z, lo.w}, y[4] = {hi.x, hi.y, hi.z, hi.w};
  uint32_t u[4], v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = bf16_lo(x[i]) * scale, x1 = bf16_hi(x[i]) * scale;
    const float y0 = bf16_lo(y[i]) * scale, y1 = bf16_hi(y[i]) * scale;
    const __half2 a = __floats2half2_rn(x0 * t.c[2 * i] - y0 * t.s[2 * i], x1 * t.c[2 * i + 1] - y1 * t.s[2 * i + 1]);
    const __half2 b = __floats2half2_rn(y0 * t.c[2 * i] + x0 * t.s[2 * i], y1 * t.c[2 * i + 1] + x1 * t.s[2 * i + 1]);
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
__device__ __forceinline__ void load_queries(const ChunkArgs &a, ChunkSmem &sm, const Item &it, bool sink, int lt,
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
    turn_row(lo, hi, t, d.qscale, ol, oh, most);
    put_row(sm.q[row >> 7], row & 127, ch, ol, oh);
    if (even) t.advance(step);
  }
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
      mbar_init(&sm.k_full[i], kLoadThreads);
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
        for (int w = 0; w < 4; ++w) {
          const uint4 lv = *reinterpret_cast<const uint4 *>(sm.live[n_tile & 3][w]);
          live[0] |= lv.x, live[1] |= lv.y, live[2] |= lv.z, live[3] |= lv.w;
        }
        const bool whole = a0 <= 0 && a1 >= kTile && (live[0] & live[1] & live[2] & live[3]) == 0xffffffffu;
        const bool masked = __any_sync(0xffffffffu, !whole);
        float x = -INFINITY;
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
          for (int i = 0; i < 32; ++i) x = fmaxf(x, __uint_as_float(s[i]));
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
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t s[32], pk[16];
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
          for (int i = 0; i < 16; ++i) {
            const float e0 = exp2_approx(__uint_as_float(s[2 * i]) - z);
            const float e1 = exp2_approx(__uint_as_float(s[2 * i + 1]) - z);
            l0 += e0;
            l1 += e1;
            pk[i] = cvt_bf16x2(e0, e1);
          }
          tmem_st16(ts + g * 16, pk);  // over columns that were read
        }
        l += l0 + l1;
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
      if (odd && in) a.redo[sg.item % kMaxShared] = 1u;
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ loaders
    const int lt = tid - kSoftWarps * 32, ch = lt & 7;
    const uint64_t *f = ws_freq(d.hdr) + ch * 8;
    Turn step;
    step.set(f, 16);
    uint32_t n = 0;  // key tiles loaded
    bool ok = true;
    while (ok && segments_next(a, sm, sg, it)) {
      __half2 most = __floats2half2_rn(0.f, 0.f);
      for (int j = sg.j0; j < sg.j1; ++j, ++n) {
        const bool sink = j < it.n1;
        const int T = (sink ? j : it.first + j - it.n1) * kTile;
        const int lo = sink ? 0 : it.lo2, hi = sink ? it.hi1 : it.hi2;
        const int s = n % kRing;
        const uint32_t round = n / kRing;
        if (j == sg.j0 || (j == it.n1 && j > 0)) {
          // the queries of a new segment, or of the window after the sinks: the products that
          // read the last ones are done once the previous key tile is free
          if (n > 0 && !wait_or_stop(sm, a, &sm.k_empty[(n - 1) % kRing], ((n - 1) / kRing) & 1)) {
            ok = false;
            break;
          }
          load_queries(a, sm, it, sink, lt, most);
        }
        // rows of the tile: a token's page is looked up once, by the 8 threads of its row
        Turn t;
        t.set(f, T + (lt >> 3));
        if (round > 0 && !wait_or_stop(sm, a, &sm.v_empty[s], (round - 1) & 1)) {
          ok = false;
          break;
        }
        int64_t rows[8];
        uint32_t here = 0;  // bit i: this thread's row i is loaded
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = T + (lt >> 3) + 16 * i;
          rows[i] = 0;
          if (tok >= lo && tok < hi) {
            const int64_t r = cache_row(d, it.b, it.h, tok);
            if (r >= 0) {
              rows[i] = r;
              here |= 1u << i;
            } else {
              atomicOr(&d.hdr->err, kErrIndex);
            }
          }
          const uint32_t dst = smem_u32(sm.v[s]) + ((lt >> 3) + 16 * i) * 128 + ((ch ^ ((lt >> 3) & 7)) << 4);
          const bool on = (here >> i) & 1u;
          cp_async16(dst, d.v + rows[i] * kD + ch * 8, on);
          cp_async16(dst + kHalfBytes, d.v + rows[i] * kD + kHalf + ch * 8, on);
        }
        cp_async_commit();
        if (round > 0 && !wait_or_stop(sm, a, &sm.k_empty[s], (round - 1) & 1)) {
          ok = false;
          break;
        }
        // live tokens: thread row r = lt / 8 holds tokens r + 16 i; word w of the tile is tokens 32 w ..
        {
          uint32_t word[4] = {0u, 0u, 0u, 0u};
          const int r = lt >> 3;
#pragma unroll
          for (int i = 0; i < 8; ++i) word[i >> 1] |= ((here >> i) & 1u) << (r + 16 * (i & 1));
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            word[w] |= __shfl_xor_sync(0xffffffffu, word[w], 8);
            word[w] |= __shfl_xor_sync(0xffffffffu, word[w], 16);
          }
          if (lane == 0)
            *reinterpret_cast<uint4 *>(sm.live[n & 3][warp - kSoftWarps]) = make_uint4(word[0], word[1], word[2], word[3]);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint4 xl[4], xh[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool on = (here >> (hf * 4 + i)) & 1u;
            const uint4 *src = reinterpret_cast<const uint4 *>(d.k + rows[hf * 4 + i] * kD);
            xl[i] = on ? __ldg(src + ch) : make_uint4(0, 0, 0, 0);
            xh[i] = on ? __ldg(src + ch + 8) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 ol, oh;
            turn_row(xl[i], xh[i], t, 1.f, ol, oh, most);
            put_row(sm.k[s], (lt >> 3) + 16 * (hf * 4 + i), ch, ol, oh);
            t.advance(step);
          }
        }
        umma::fence_async_smem();
        mbar_arrive(&sm.k_full[s]);
        cp_async_wait<0>();
        umma::fence_async_smem();
        mbar_arrive(&sm.v_full[s]);
      }
      if (__hgt(__hmax(__low2half(most), __high2half(most)), __float2half(65504.f))) a.redo[sg.item % kMaxShared] = 1u;
    }
    cp_async_wait<0>();
  } else if (lane == 0) {
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

int launch_dense_chunk(const DenseArgs &d, int64_t max_keys, void *stream) {
  ChunkArgs a;
  a.d = d;
  const int per = kItemRows >> d.group_shift;
  a.d.tiles = (d.nq + per - 1) / per;
  const int64_t items = (int64_t)d.batch * d.hkv * a.d.tiles;
  a.items = (int)items;
  a.redo = nullptr;
  const int sms = std::min(dense_sm_count(), kMaxChunkBlocks);
  // Dealing the key tiles out evenly costs a part's write and join (about four key tiles'
  // time) and saves the last wave's idle blocks.
  const int64_t tiles = ceil_div(max_keys, kTile) + 1;
  const int64_t plain = ceil_div(items, sms) * tiles, dealt = ceil_div(items * tiles, sms) + 4;
  a.shared = items <= kMaxShared && dealt < plain ? 1 : 0;
  a.redo = reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(d.hdr) + kDenseRedo);
  cudaError_t e = cudaFuncSetAttribute(dense_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kChunkSmem);
  if (e != cudaSuccess) return (int)e;
  const int64_t work = a.shared ? items * tiles : items;
  dense_chunk_kernel<<<(unsigned)std::min<int64_t>(work, sms), kChunkThreads, kChunkSmem, (cudaStream_t)stream>>>(a);
  e = cudaGetLastError();
  return e != cudaSuccess ? (int)e : launch_dense_redo(d, a.d.tiles, stream);
}

}  // namespace recsa
