// Eviction of cache slots by accumulated attention weight: per (sequence, KV head) the `keep`
// heaviest slots are selected and their rows compacted in slot order.
//
// Selection is a radix select over the weights' order keys: three digits of 11, 11 and 10
// bits from the top, each a histogram of the keys that match the digits above, give the
// smallest kept key and how many of its equals (lowest slots first) are kept; a last walk in
// slot order writes the kept indices.  A cluster shares one (sequence, head); its histograms
// are summed over distributed shared memory, so every block finds the same digit.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include <cooperative_groups.h>

#include "recsa_dense.cuh"
#include "recsa_evict.h"

namespace cg = cooperative_groups;

namespace recsa {
namespace {

__device__ uint32_t g_evict_err = 0u;  // kErr* (the call takes no workspace); recsa_check_device_errors reads it

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxBlocks = 8;   // of a cluster

struct SelectSmem {
  int hist[3][kBins];
  int warp_gt[kSelWarps], warp_eq[kSelWarps];  // then: of the warps before
  int gt, eq;          // this block's totals
  int digit, above;    // the digit found, and how many keys lie above it
  int scan[kSelWarps];
};

// larger weight -> larger key; NaN below every number
__device__ __forceinline__ uint32_t weight_key(float w) { return w == w ? order_key(w) : 0u; }

// PER > 0: a thread holds its weights' keys, at most PER of them (two blocks an SM leave it 64
// registers: of 32 keys some lie in local memory, 172 bytes of spill stores); 0: they are read
// again each time.
template <int PER>
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(EvictArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SelectSmem &sm = *reinterpret_cast<SelectSmem *>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int nblk = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int bh = blockIdx.x / nblk, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = bh / a.hkv;
  const int n = evict_length(a, b);
  if (rank == 0 && tid == 0 && evict_bad_length(a, b)) atomicOr(&g_evict_err, kErrIndex);
  int32_t *const kept = a.kept + (int64_t)bh * a.keep;
  if (n <= a.keep) {  // everything stays
    for (int j = rank * kSelThreads + tid; j < a.keep; j += nblk * kSelThreads) kept[j] = j < n ? j : -1;
    return;
  }
  const float *const w = a.weights + (int64_t)bh * a.capacity;
  const int f0 = a.sinks, f1 = n - a.recent;        // the slots that compete
  const int want = a.keep - a.sinks - a.recent;     // how many of them stay: 0 <= want < f1 - f0
  for (int i = tid; i < 3 * kBins; i += kSelThreads) (&sm.hist[0][0])[i] = 0;
  __syncthreads();
  // this block's slots, and this warp's contiguous part of them (in 32s)
  const int64_t span = (int64_t)(f1 - f0 + 31) / 32, parts = (int64_t)nblk * kSelWarps, part = rank * kSelWarps + warp;
  const int w0 = f0 + (int)(span * part / parts) * 32, w1 = min(f1, f0 + (int)(span * (part + 1) / parts) * 32);

  uint32_t held[PER ? PER : 1];
  if (PER) {
    float x[PER ? PER : 1];
#pragma unroll
    for (int j = 0; j < PER; ++j) x[j] = w0 + lane + 32 * j < w1 ? __ldg(w + w0 + lane + 32 * j) : 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) held[j] = weight_key(x[j]);
  }
  // f(slot, key) for each of this lane's slots
  auto each = [&](auto &&f) {
    if (PER) {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (w0 + lane + 32 * j < w1) f(w0 + lane + 32 * j, held[j]);
    } else {
#pragma unroll 8
      for (int i = w0 + lane; i < w1; i += 32) f(i, weight_key(__ldg(w + i)));
    }
  };
  uint32_t floor_key = 0xffffffffu;  // the smallest kept key (none: want = 0)
  int left = want;                   // how many keys equal to it stay
  if (want > 0) {
    uint32_t prefix = 0;
#pragma unroll
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
      const uint32_t mask = d == 2 ? 1023u : 2047u;
      each([&](int, uint32_t key) {
        const bool in = d == 0 || (d == 1 ? (key >> 21) == prefix : (key >> 10) == prefix);
        if (in) atomicAdd(&sm.hist[d][(key >> shift) & mask], 1);
      });
      cluster.sync();
      // bins from the top: thread t sums bins kBins-1-4t down to kBins-4-4t over the cluster
      constexpr int kPer = kBins / kSelThreads;
      static_assert(kPer == 4, "a thread's bins are one 16-byte load");
      const int top = kBins - 1 - kPer * tid;
      int4 part[kMaxBlocks];
#pragma unroll
      for (int k = 0; k < kMaxBlocks; ++k)
        part[k] = k < nblk ? *reinterpret_cast<const int4 *>(cluster.map_shared_rank(&sm.hist[d][top - 3], k))
                           : make_int4(0, 0, 0, 0);
      int c[kPer] = {0, 0, 0, 0};  // the highest bin first
#pragma unroll
      for (int k = 0; k < kMaxBlocks; ++k) c[0] += part[k].w, c[1] += part[k].z, c[2] += part[k].y, c[3] += part[k].x;
      const int own = c[0] + c[1] + c[2] + c[3];
      int incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) sm.scan[warp] = incl;
      __syncthreads();
      const int before_warp = warp_sum_int(lane < warp ? sm.scan[lane] : 0);
      int before = before_warp + incl - own;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (before < left && before + c[i] >= left) sm.digit = top - i, sm.above = before;
        before += c[i];
      }
      __syncthreads();
      prefix = d == 0 ? (uint32_t)sm.digit : d == 1 ? (prefix << 11) | (uint32_t)sm.digit
                                                    : (prefix << 10) | (uint32_t)sm.digit;
      left -= sm.above;
      __syncthreads();
    }
    floor_key = prefix;
  }
  // how many larger and equal keys each warp holds, then each block's place in slot order
  int gt = 0, eq = 0;
  each([&](int, uint32_t key) {
    gt += key > floor_key;
    eq += key == floor_key;
  });
  gt = warp_sum_int(gt);
  eq = warp_sum_int(eq);
  if (lane == 0) sm.warp_gt[warp] = gt, sm.warp_eq[warp] = eq;
  __syncthreads();
  if (tid == 0) {
    int g = 0, e = 0;
    for (int k = 0; k < kSelWarps; ++k) g += sm.warp_gt[k], e += sm.warp_eq[k];
    sm.gt = g;
    sm.eq = e;
  }
  cluster.sync();
  gt = lane < rank ? *cluster.map_shared_rank(&sm.gt, lane) : 0;
  eq = lane < rank ? *cluster.map_shared_rank(&sm.eq, lane) : 0;
  if (lane < warp) gt += sm.warp_gt[lane], eq += sm.warp_eq[lane];
  gt = warp_sum_int(gt);
  eq = warp_sum_int(eq);
  auto write = [&](int i, uint32_t key) {
    const bool is_gt = i < w1 && key > floor_key, is_eq = i < w1 && key == floor_key && left > 0;
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t mg = __ballot_sync(0xffffffffu, is_gt), me = __ballot_sync(0xffffffffu, is_eq);
    const int e = eq + __popc(me & below);  // equals in lower slots
    const int at = a.sinks + gt + __popc(mg & below) + min(e, left);
    if (is_gt || (is_eq && e < left)) kept[at] = i;
    gt += __popc(mg);
    eq += __popc(me);
  };
  if (PER) {
#pragma unroll
    for (int j = 0; j < PER; ++j) write(w0 + lane + 32 * j, held[j]);
  } else {
#pragma unroll 8
    for (int i0 = w0; i0 < w1; i0 += 32) write(i0 + lane, i0 + lane < w1 ? weight_key(__ldg(w + i0 + lane)) : 0u);
  }
  if (rank == 0) {
    for (int j = tid; j < a.sinks; j += kSelThreads) kept[j] = j;
    for (int j = tid; j < a.recent; j += kSelThreads) kept[a.keep - a.recent + j] = f1 + j;
  }
  cluster.sync();  // no block leaves while another may read its shared memory
}

// Rows to another cache: nothing overlaps, 16 threads a row.
__global__ void evict_copy_kernel(EvictArgs a, int64_t *to_len) {
  if (to_len && blockIdx.x == 0)  // the receiving cache's lengths
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x) to_len[b] = min(evict_length(a, b), a.keep);
  const int64_t rows = (int64_t)a.batch * a.hkv * a.keep;
  const int part = threadIdx.x & 15;
  for (int64_t e = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 4; e < rows;
       e += ((int64_t)gridDim.x * blockDim.x) >> 4) {
    const int j = (int)(e % a.keep);
    const int64_t bh = e / a.keep;
    const int b = (int)(bh / a.hkv), h = (int)(bh % a.hkv);
    const int i = __ldg(a.kept + e);
    if (i < 0) continue;
    if (part == 0 && a.to_weights) a.to_weights[bh * a.to_capacity + j] = __ldg(a.weights + bh * a.capacity + i);
    const int64_t src = evict_row(a.from, a.hkv, b, h, i), dst = evict_row(a.to, a.hkv, b, h, j);
    if ((src < 0 || dst < 0) && part == 0) atomicOr(&g_evict_err, kErrIndex);
    if (dst < 0) continue;
    const uint4 none = make_uint4(0, 0, 0, 0);
    a.to.k[dst * 16 + part] = src >= 0 ? __ldg(a.from.k + src * 16 + part) : none;
    a.to.v[dst * 16 + part] = src >= 0 ? __ldg(a.from.v + src * 16 + part) : none;
  }
}

// Rows within one cache.  A block owns a 64-byte column of K or of V (or the weights) of one
// (sequence, head) and walks the kept rows in order: a piece is read whole before it is
// written.  Row j comes from slot kept[j] >= j, so writing rows [j, j + piece) can only touch
// slots below j + piece, which no later piece reads: no block waits for another.
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;  // rows a thread holds
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a) {
  const int col = blockIdx.x % 9;
  const int64_t bh = blockIdx.x / 9;
  const int b = (int)(bh / a.hkv), h = (int)(bh % a.hkv);
  const int n = evict_length(a, b);
  if (n <= a.keep && !(col == 8 && a.to_weights != a.weights)) return;  // nothing moves
  const int count = min(n, a.keep);
  const int32_t *const kept = a.kept + bh * a.keep;
  if (col == 8) {
    if (!a.to_weights) return;
    const float *from = a.weights + bh * a.capacity;
    float *to = a.to_weights + bh * a.to_capacity;
    for (int j0 = 0; j0 < count; j0 += kMoveThreads * kMoveRows) {
      float x[kMoveRows];
#pragma unroll
      for (int r = 0; r < kMoveRows; ++r) {
        const int j = j0 + r * kMoveThreads + threadIdx.x;
        x[r] = j < count ? from[kept[j]] : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kMoveRows; ++r) {
        const int j = j0 + r * kMoveThreads + threadIdx.x;
        if (j < count) to[j] = x[r];
      }
    }
    // the next tokens go to the slots behind: they start without the weights of those that are gone
    for (int j = count + threadIdx.x; j < n; j += kMoveThreads) to[j] = 0.f;
    return;
  }
  uint4 *const rows = col < 4 ? a.to.k : a.to.v;
  const int part = (col & 3) * 4 + (threadIdx.x & 3), r0 = threadIdx.x >> 2;
  constexpr int kPer = kMoveThreads / 4;
  for (int j0 = 0; j0 < count; j0 += kPer * kMoveRows) {
    uint4 x[kMoveRows];
    int64_t src[kMoveRows], dst[kMoveRows];
#pragma unroll
    for (int r = 0; r < kMoveRows; ++r) {
      const int j = j0 + r * kPer + r0;
      src[r] = dst[r] = -1;
      if (j < count) {
        const int i = kept[j];
        if (i != j) {
          src[r] = evict_row(a.from, a.hkv, b, h, i);
          dst[r] = evict_row(a.to, a.hkv, b, h, j);
          if (src[r] < 0 || dst[r] < 0) atomicOr(&g_evict_err, kErrIndex);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kMoveRows; ++r) x[r] = src[r] >= 0 ? rows[src[r] * 16 + part] : make_uint4(0, 0, 0, 0);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kMoveRows; ++r)
      if (dst[r] >= 0) rows[dst[r] * 16 + part] = x[r];
  }
}

// in place, after the rows: the per-sequence lengths
__global__ void evict_lengths_kernel(EvictArgs a, int64_t *to_len) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < a.batch) to_len[b] = min(evict_length(a, b), a.keep);
}

}  // namespace

int read_evict_errors(uint32_t *bits) {
  uint32_t v = 0u, zero = 0u;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_evict_err, sizeof(v));
  if (e == cudaSuccess && v != 0u) e = cudaMemcpyToSymbol(g_evict_err, &zero, sizeof(zero));
  *bits = v;
  return (int)e;
}

int launch_evict(const EvictArgs &a, bool in_place, int64_t *to_len, void *stream) {
  const cudaStream_t st = (cudaStream_t)stream;
  const int64_t heads = (int64_t)a.batch * a.hkv;
  cudaLaunchConfig_t cfg = {};
  const int blocks = a.length > 8192 ? kMaxBlocks : 1;
  cfg.gridDim = dim3((unsigned)(heads * blocks));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = sizeof(SelectSmem);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)blocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  // a thread's slots, as the kernel deals them out: whole 32s a warp
  const int64_t per = ceil_div(ceil_div(a.length, 32), (int64_t)blocks * kSelWarps);
  cudaError_t e = per <= 4    ? cudaLaunchKernelEx(&cfg, evict_select_kernel<4>, a)
                  : per <= 8  ? cudaLaunchKernelEx(&cfg, evict_select_kernel<8>, a)
                  : per <= 16 ? cudaLaunchKernelEx(&cfg, evict_select_kernel<16>, a)
                  : per <= 32 ? cudaLaunchKernelEx(&cfg, evict_select_kernel<32>, a)
                              : cudaLaunchKernelEx(&cfg, evict_select_kernel<0>, a);
  if (e != cudaSuccess) return (int)e;
  if (in_place) {
    evict_move_kernel<<<(unsigned)(heads * 9), kMoveThreads, 0, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || !to_len) return (int)e;
    evict_lengths_kernel<<<(unsigned)ceil_div(a.batch, 128), 128, 0, st>>>(a, to_len);
  } else {
    const int64_t threads = heads * a.keep * 16;
    const int64_t grid = std::min<int64_t>(ceil_div(threads, 256), (int64_t)dense_sm_count() * 16);
    evict_copy_kernel<<<(unsigned)grid, 256, 0, st>>>(a, to_len);
  }
  e = cudaGetLastError();
  return (int)e;
}

}  // namespace recsa
