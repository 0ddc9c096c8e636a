// Host-side interface of the dense causal attention (attend_kernel.cuh) between
// the C-ABI layer and its translation units.  Not part of the public ABI.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace i8kv {

struct AttendParams {
  const __half* q;           // [T, Hq, D], tokens q_stride elements apart
  long long q_stride;
  const void* k;             // packed: [T, Hkv, D] fp16 rows; paged: the cache (MX4: the record cache)
  const void* v;
  long long k_stride, v_stride;  // packed: elements between tokens
  const float* k_scale;      // of a quantised cache, [1] or [Hkv, D]
  const float* v_scale;
  const int32_t* table;      // paged: [B, max_blocks]; nullptr: packed
  const int32_t* lens;       // paged: [B] lengths, new tokens included; nullptr: the new tokens are all
  const int32_t* starts;     // [B + 1] first new token of each sequence
  const float* sink;         // [Hq] or nullptr
  __half* out;               // [T, Hq, D]
  float* lse;                // [T, Hq] or nullptr
  uint32_t* flags;
  // pieces > 0: the batch's blocks cut into so many pieces of equal length, one per CTA, each of which ends inside
  // two (tile, KV head)s at most, whose partials go to the slots 2 * CTA (begun inside) and 2 * CTA + 1
  float* part_acc;           // [2 * pieces, M, D] with M vectors per tile of a CTA
  float* part_m;             // [2 * pieces, M]
  float* part_l;
  int32_t pieces;            // 0: whole tiles
  int32_t T, B, Hq, Hkv, G, D;
  int32_t per_channel;
  int32_t bs, bs_log2, max_blocks;
  int32_t cap;               // max_blocks * bs
  int64_t num_blocks;
  int32_t rows;              // of a plain source: T, or num_blocks * bs
  float sigma, softcap;
  int32_t window;
};

// two_tiles: 256 vectors per CTA (D = 64 or 128); ctas: the grid (pieces, if there are).  Pieces are merged by
// launch_attend_merge on the same parameters.
cudaError_t launch_attend_f16(const AttendParams& p, bool two_tiles, unsigned ctas, cudaStream_t s);
cudaError_t launch_attend_int8(const AttendParams& p, bool two_tiles, unsigned ctas, cudaStream_t s);
cudaError_t launch_attend_fp8(const AttendParams& p, bool two_tiles, unsigned ctas, cudaStream_t s);
cudaError_t launch_attend_mx4(const AttendParams& p, bool two_tiles, unsigned ctas, cudaStream_t s);
cudaError_t launch_attend_merge(const AttendParams& p, bool two_tiles, cudaStream_t s);

}  // namespace i8kv
