// Host declarations of the dense cache operators: the workspace layout, the arguments of a
// launch and the launchers.
#pragma once

#include <cstddef>
#include <cstdint>

#include "recsa_dense.h"
#include "recsa_internal.h"

namespace recsa {

constexpr uint32_t kDenseMagic = 0x52534433u;  // "RSD3"
constexpr int kSpan = 64;                      // positions of the rotation table
constexpr int kMaxShared = 4096;               // work items whose key range may be shared by blocks
constexpr size_t kDenseFreq = kWsHeader;                                   // uint64[64] turns
constexpr size_t kDenseTable = kDenseFreq + kHalf * sizeof(uint64_t);      // float4[64][32] (cos, cos', sin, sin')
constexpr size_t kDenseTableBytes = kSpan * kHalf * 2 * sizeof(float);
constexpr size_t kDenseCount = kDenseTable + 2 * kDenseTableBytes;  // (the second table: the first times kKeyScale)
constexpr size_t kDenseRedo = kDenseCount + kMaxShared * sizeof(int32_t) + 256;  // marks of items to compute again
constexpr size_t kDensePrefix = kDenseRedo + kMaxShared * sizeof(uint32_t);  // key tiles before each item of a chunk
constexpr size_t kDenseBeyond = kDensePrefix + (kMaxShared + 64) * sizeof(int32_t);  // heads beyond fp16: found, in use
constexpr size_t kDensePart = kDenseBeyond + 2 * kMaxShared * sizeof(int32_t);  // partial results
constexpr size_t kDensePartBytes = (size_t)40 << 20;
constexpr size_t kDenseLse = kDensePart + kDensePartBytes;                 // two floats a query row
constexpr int64_t kMaxDenseLse = (int64_t)1 << 20;                         // floats: rows of a call that keeps their scores
constexpr size_t kDenseImages = kDenseLse + kMaxDenseLse * sizeof(float);   // rotated rows of a chunk's keys and queries
constexpr size_t kMaxDenseImages = (size_t)320 << 20;   // for many heads together
constexpr size_t kMaxHeadImages = (size_t)1280 << 20;   // for one long head
constexpr int kPartRow = kD + 4;  // floats of a row's partial result: maximum, sum, 2 unused, 128 sums

constexpr float kLog2e = 1.4426950408889634f;
// fp32 outputs and weights are scored from two fp16 parts of rotated rows, 22 bits, of keys and
// queries times these powers of two: the parts' smallest steps are then 2^-29 and 2^-31.
constexpr float kKeyScale = 16.f, kQueryScale = 64.f;

// The cache and the queries of one launch.
struct DenseArgs {
  const uint16_t *k, *v, *q;
  void *out;
  const int64_t *seq_len;
  const int32_t *pages;
  int64_t capacity;
  int32_t pages_per_seq, page_shift, num_pages;
  int32_t batch, hkv, group_shift, nq;
  int32_t length;
  int32_t sinks, window, rank_sinks, causal, own;
  int32_t back;       // a query that sees the tokens t < p sits at p - back
  int32_t out_fp32;
  int32_t tiles, nsplit;
  float qscale;       // softmax scale * log2(e)
  float rope_base;
  WsHeader *hdr;
  int32_t bh0, heads;     // the rows kernel's (sequence, KV head) pairs (heads = 0: all)
  float *scores;          // where its sums' scores go: [heads][score_pitch tokens][score_stride rows]
  int32_t score_stride;
  int64_t score_pitch;
};

// Mark of tile `tile` (256 query rows) of a (sequence, KV head) in the workspace's list; two tiles
// that share a mark are both computed again.
#ifdef __CUDACC__
__host__ __device__
#endif
inline int redo_slot(int bh, int tiles, int tile) { return (int)(((int64_t)bh * tiles + tile) % kMaxShared); }

int dense_sm_count();  // of the current device
int launch_dense_init(void *ws, double base, void *stream);
// The rows kernel: outputs, or with `lse` the rows' (maximum, 1 / sum) (at most 8 rows a KV group).
int launch_dense_rows(DenseArgs a, int64_t max_keys, float *lse, void *stream);
// The chunk kernel (bf16 output), then the rows kernel for the items it marked; kNoRoom, with
// nothing launched, where a head's rotated keys do not fit image_bytes of the workspace.
constexpr int kNoRoom = -1000;
int launch_dense_chunk(const DenseArgs &a, int64_t max_keys, int64_t image_bytes, void *stream);
int launch_dense_redo(DenseArgs a, int chunk_tiles, void *stream);
// Weights per slot; `lse` has room for kMaxDenseLse floats, the images `room` bytes; kNoRoom, with
// nothing launched, where a head's partial sums do not fit theirs.
int launch_dense_weights(const DenseArgs &a, float *lse, float *weights, int accumulate, int64_t room, void *stream);
int launch_append_tokens(const DenseArgs &a, void *k, void *v, const void *k_new, const void *v_new, int64_t at,
                         int count, int64_t limit, void *stream);

}  // namespace recsa
