// What the dense operators' kernels share: the workspace layout, the cache they read, which
// tokens a query sees, and the rotation of rows by exact phases.
//
// Rotation.  theta_i = base^(-2i/128).  The workspace holds f_i = theta_i / 2 pi as a 64-bit
// fraction of a turn, so the angle of position t is the wrapped product t * f_i: the range
// reduction is exact integer arithmetic, and f_i, formed in doubles, is good to 2^-55 of a turn
// (a position near 2^20 to 2^-35, one near 2^30 to 2^-25).  cos and sin come from sincospif of the
// top 32 bits as a float, half a step of which is 2^-26 of a turn.  Rotations compose,
// <R_p q, R_t k> = <R_{p-T} q, R_{t-T} k>, so a kernel that walks keys in spans of 64 from an
// aligned T reads the keys' rotations from one table of 64 positions and turns the few query
// rows by p - T once a span.
#pragma once

#include "recsa_dense_internal.h"
#include "recsa_device.cuh"

namespace recsa {

__device__ __forceinline__ const uint64_t *ws_freq(const WsHeader *h) {
  return reinterpret_cast<const uint64_t *>(reinterpret_cast<const char *>(h) + kDenseFreq);
}
__device__ __forceinline__ const float2 *ws_table(const WsHeader *h, bool scaled) {
  return reinterpret_cast<const float2 *>(reinterpret_cast<const char *>(h) + kDenseTable +
                                          (scaled ? kDenseTableBytes : 0));
}
__device__ __forceinline__ int32_t *ws_count(WsHeader *h) {
  return reinterpret_cast<int32_t *>(reinterpret_cast<char *>(h) + kDenseCount);
}
__device__ __forceinline__ float *ws_part(WsHeader *h) {
  return reinterpret_cast<float *>(reinterpret_cast<char *>(h) + kDensePart);
}

// (cos, sin) of position t for a frequency of f turns
__device__ __forceinline__ float2 rotation(int64_t t, uint64_t f) {
  const int32_t turn = (int32_t)((uint32_t)(((uint64_t)t * f) >> 32));
  float s, c;
  sincospif((float)turn * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ int dense_length(const DenseArgs &a, int b, bool report) {
  if (!a.seq_len) return a.length;
  const int64_t n = a.seq_len[b];
  if (n < 0 || n > a.length) {
    if (report) atomicOr(&a.hdr->err, kErrIndex);
    return n < 0 ? 0 : a.length;
  }
  return (int)n;
}

// The p of query i of a sequence of len tokens: it sees tokens t < p (0 or less: nothing) and sits
// at p - back.
__device__ __forceinline__ int dense_position(const DenseArgs &a, int len, int i) {
  return a.causal ? len - a.nq + i + a.own : len;
}
// The bound that a query of bound p has for the sinks (those outside its window).
__device__ __forceinline__ int sink_position(const DenseArgs &a, int p) {
  return a.rank_sinks ? min(p, a.sinks + a.window) : p;
}
// The tokens a query at p sees, besides the first min(sinks, p): [first, p).
__device__ __forceinline__ int window_first(const DenseArgs &a, int p) {
  return a.window ? max(a.sinks, p - a.window) : 0;
}

// Row of token t of (sequence, head) in the caches, or -1 for a page outside the pool.
__device__ __forceinline__ int64_t cache_row(const DenseArgs &a, int b, int h, int t) {
  if (!a.pages) return ((int64_t)b * a.hkv + h) * a.capacity + t;
  const int pg = __ldg(a.pages + (int64_t)b * a.pages_per_seq + (t >> a.page_shift));
  if ((unsigned)pg >= (unsigned)a.num_pages) return -1;
  return (((int64_t)pg * a.hkv + h) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
// c += a (16 x 16, row) * b (16 x 8, column), fp16 operands, fp32 sums
__device__ __forceinline__ void mma16816_half(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c = a * b, fp16 operands
__device__ __forceinline__ void mma16816_half_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
      "%10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// the same with bf16 operands
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c = a * b
__device__ __forceinline__ void mma16816_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
      "%10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// two fp32 -> packed bf16, round to nearest even (lo in the low half)
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// what the rounding of (lo, hi) to the packed pair `r` left over, itself rounded to bf16
__device__ __forceinline__ uint32_t residue_bf16x2(float lo, float hi, uint32_t r) {
  return cvt_bf16x2(lo - bf16_lo(r), hi - bf16_hi(r));
}
// the same for fp16
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two fp32 lanes in one register pair: one instruction an operation on both.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2_get(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 f2_neg(F2 a) { return F2{a.v ^ 0x8000000080000000ull}; }
__device__ __forceinline__ F2 f2_bf16(uint32_t u) { return f2(bf16_lo(u), bf16_hi(u)); }
__device__ __forceinline__ F2 f2_f16(uint32_t u) {
  float lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(u));
  return f2(lo, hi);
}
// Two values as the first part of an operand, rounded, and what that leaves as the second: pairs of
// fp16 or bf16.
template <bool HALF>
__device__ __forceinline__ void split_pair(F2 x, uint32_t &hi, uint32_t &lo) {
  const float2 u = f2_get(x);
  hi = HALF ? cvt_f16x2(u.x, u.y) : cvt_bf16x2(u.x, u.y);
  const float2 d = f2_get(f2_fma(HALF ? f2_f16(hi) : f2_bf16(hi), f2(-1.f, -1.f), x));
  lo = HALF ? cvt_f16x2(d.x, d.y) : cvt_bf16x2(d.x, d.y);
}
// The same in fp16 with the first part cut off instead of rounded: one logical instruction, and no
// conversion back (weights of one step over 4 x 65536 tokens 166.3 -> 162.5 us).  Second parts are up
// to twice as large then; with the other operand's rounded, their dropped product has no bias.
__device__ __forceinline__ void cut_pair(F2 x, uint32_t &hi, uint32_t &lo) {
  const float2 u = f2_get(x);
  const float2 c = make_float2(__uint_as_float(__float_as_uint(u.x) & 0xffffe000u),
                               __uint_as_float(__float_as_uint(u.y) & 0xffffe000u));
  const float2 d = f2_get(f2_fma(f2(c.x, c.y), f2(-1.f, -1.f), x));
  hi = cvt_f16x2(c.x, c.y);
  lo = cvt_f16x2(d.x, d.y);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

}  // namespace recsa
