// What the dense operators' tensor-core (tcgen05) kernels share: 128 x 128 operand tiles in swizzled
// shared memory, their descriptors and products, bounded waits, bulk copies, and the rotation of
// rows on their way into a tile.
#pragma once

#include <cuda_fp16.h>

#include "recsa_dense.cuh"
#include "recsa_umma.cuh"

namespace recsa {

constexpr int kTile = 128;                  // rows of a row tile, keys of a key tile
constexpr int kTileBytes = kTile * kRowBytes;  // 32 KB: [64-element half][row][128 bytes], 16-byte pieces XOR row % 8
constexpr int kHalfBytes = kTileBytes / 2;

__host__ __device__ constexpr uint32_t chunk_idesc(int n, bool bf16, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kTile >> 4) << 24);
}
// Descriptor of a 128-byte-swizzled operand: rows of 128 bytes, 8 rows 1024 bytes apart.  K-major
// (queries, keys): a k-step of 16 elements is 32 bytes further into the row.  MN-major (values): the
// rows are keys, the second 64 dimensions lie kHalfBytes further (the leading-dimension step).
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3fffu) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// One thread of the warp, chosen so that the compiler knows only one runs on: descriptors then stay
// in uniform registers (branching on the lane number instead doubled the cycles an MMA took).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
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
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Waits for a barrier's phase, within a limit; after a wait ran out nobody waits any more (each
// role's steps are counted, so all of them end) and the timeout is reported.
// A poll without a suspend hint wakes sooner (a 4096-token chunk over 32768: 2.24 -> 2.16 ms).
constexpr uint32_t kChunkPolls = 1u << 20;  // of a microsecond or so each
__device__ __forceinline__ void bounded_wait(uint32_t *stop, WsHeader *hdr, uint64_t *bar, uint32_t parity) {
  for (uint32_t i = 0; i < kChunkPolls; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (done) return;
    if (*(volatile uint32_t *)stop) return;
  }
  *(volatile uint32_t *)stop = 1u;
  atomicOr(&hdr->err, kErrTimeout);
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

// One bulk copy of `bytes` (a multiple of 16) into shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

}  // namespace recsa
