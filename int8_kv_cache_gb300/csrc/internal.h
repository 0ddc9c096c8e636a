// Host-side interface between the C-ABI layer (api.cu) and the kernel
// translation units.  Not part of the public ABI.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace i8kv {

enum class Path : int { kDsa = 1, kPaged = 2 };

struct DecodeParams {
  const void* q;             // fp16 [rows, Hq, D]
  const void* k;             // cache base (int8 or fp16)
  const void* v;
  const float* k_scale;      // [1] or [Hkv, D]; unused for an fp16 cache
  const float* v_scale;
  const int32_t* idx;        // DSA: [rows, max_sel]
  const int32_t* block_table;  // paged: [rows, max_blocks]
  const int32_t* seq_lens;     // paged: [rows]
  const float* sink;         // [Hq] or nullptr
  void* out;                 // fp16 [rows, Hq, D]
  float* lse;                // [rows, Hq] or nullptr
  float* ws_acc;             // [units, splits, G, D]
  float* ws_m;               // [units, splits, G]
  float* ws_l;               // [units, splits, G]
  int32_t* slots_out;        // paged debug [rows, cap] or nullptr
  uint32_t* flags;           // or nullptr
  int64_t cache_rows;        // DSA: N; paged: num_blocks (in blocks)
  int32_t rows, Hq, Hkv, G;
  int32_t max_sel;           // DSA list length (cap)
  int32_t bs, max_blocks;    // paged
  int32_t bs_log2;           // log2(bs) when bs is a power of two, else -1
  int32_t num_splits, chunk;
  int32_t per_channel;       // 1: scales [Hkv, D]; 0: one scale
  float sigma;
  float softcap;             // paged: > 0 caps scores to softcap * tanh(s / softcap); 0 off
  int32_t window;            // paged: >= 0 attends [len - 1 - window, len); -1 off
  int32_t lpt;               // paged: longest-first dispatch of the (unit, split) items
  // paged, balanced pieces (chunk 0 on the API): the live lengths are cut on
  // the device into pieces of about equal length across the batch, at most
  // num_splits per row (the partial slots), bal_pieces (row, piece) pairs in
  // all, each a multiple of bal_round positions; the grid has
  // ceil(num_splits / 2) CTAs per unit (decode_kernel.cuh, balanced_item).  MX4: the rule and
  // the grid (at most bal_pieces CTAs) are mx4_kernel.cuh's balanced_piece; bal_round is not used
  int32_t balanced;
  int32_t bal_round;
  int32_t bal_pieces;
  int32_t longest_first;     // MX4 rows: they are taken in the order of falling lengths
  int32_t head_groups;       // MX4 rows and clusters: 2: each half of a group's query heads is a unit of its own
};

// Longest-first dispatch of the paged decode (decode_kernel.cuh, lpt_item):
// batches of at most kLptMaxRows rows, chunks of at least kLptMinChunk tokens.
constexpr int kLptMaxRows = 128;
constexpr int kLptMinChunk = 1280;

// What a CTA of the MX4 decode works on: a piece (or chunk) of a row and KV head, all of it, or
// its part in the cluster of num_splits CTAs that shares it.
enum class Mx4Way : int { kPieces = 0, kRows = 1, kCluster = 2 };

struct KernelKey {
  Path path;
  int D;
  int nt;          // 8-head tiles: 1 (G <= 8) or 2 (G <= 16)
  bool fp16_cache;
  bool fp8_cache;  // float8 e4m3fn codes (same tile as int8, other conversion)
  bool p_lo;       // probability tile as fp16 high + low parts
  bool mx4_cache = false;  // 4-bit records (mx4_kernel.cuh; DecodeParams::k is the record cache)
  Mx4Way way = Mx4Way::kPieces;
  bool wide = false;       // mx4_cache: 8-warp CTAs (clusters always are)
  bool per_channel = false;  // mx4_cache, KernelInfo only: the kernel for scales per channel
};

// What the geometry needs to know of a decode kernel instantiation.
struct KernelInfo {
  int occupancy;  // resident CTAs per SM (the CUDA occupancy API)
  int round;      // positions one round of the CTA's warps covers (warps x step)
  int clusters[4] = {0, 0, 0, 0};  // cluster kernels: resident clusters of 2, 4, 8 CTAs, from [1]
};

// Per-path launchers (one per translation unit): grid (rows * Hkv, num_splits);
// with info != NULL nothing is launched and the selected kernel's KernelInfo
// is returned there instead.
cudaError_t launch_dsa_decode(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                              KernelInfo* info);
cudaError_t launch_dsa_prefill(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                               KernelInfo* info);
cudaError_t launch_paged_int8(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                              KernelInfo* info);
cudaError_t launch_paged_fp16(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                              KernelInfo* info);
cudaError_t launch_paged_fp8(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                             KernelInfo* info);

cudaError_t launch_paged_mx4(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                             KernelInfo* info);
cudaError_t launch_paged_mx4_wide(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                                  KernelInfo* info);
cudaError_t launch_paged_mx4_rows(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                                  KernelInfo* info);
cudaError_t launch_paged_mx4_rows_wide(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                                       KernelInfo* info);
cudaError_t launch_paged_mx4_cluster(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                                     KernelInfo* info);
constexpr int kMx4MaxCluster = 8;  // CTAs of a portable cluster
constexpr int kMx4RankRows = 256;  // rows that longest_first takes at most
constexpr int kMx4Warps = 4, kMx4WideWarps = 8;  // of a CTA

// rope_and_cache and gather_cache (append.cu); the cache type picks the kernel.
struct AppendParams {
  const __half* q;           // [num_tokens, Hq, D], tokens q_stride elements apart
  const __half* k;
  const __half* v;
  long long q_stride, k_stride, v_stride;
  const int32_t* positions;
  const float* cos_sin;      // [max_pos, R]: R / 2 cosines, then the sines
  long long max_pos;
  int32_t R, interleaved;
  const int32_t* slots;
  int32_t num_tokens, Hq, Hkv, D;
  __half* q_out;
  void* k_cache;             // MX4: the record cache
  void* v_cache;
  long long num_slots;
  int32_t bs, bs_shift;      // MX4: block size, its log2 or -1
  const float* k_scale;
  const float* v_scale;
  int32_t per_channel;
  uint32_t* flags;
  // norm_rope_and_cache: [D] weights of the norms (or nullptr), and where keys go besides the cache
  const float* q_weight;
  const float* k_weight;
  float eps;
  __half* k_out;             // [num_tokens, Hkv, D] or nullptr
};
cudaError_t launch_rope_and_cache(const AppendParams& p, int cache_dtype, cudaStream_t stream);
cudaError_t launch_gather_cache(const AppendParams& p, int cache_dtype, void* k_out, void* v_out,
                                cudaStream_t stream);

// The dense tensor-core prefill (prefill_tc.cu): whether it serves a shape
// (and with how much shared memory / how many mask rows), and its launch.
bool prefill_tc_plan(int D, int G, int rows, long long N, int max_sel, int* smem_bytes,
                     int* mask_rows);
// stage: NULL for the converting form; else the staged form's operand images
// and row bitmasks (prefill_stage_bytes of them, 16-byte aligned), written by
// the call itself.
// nsplit > 1 (staged form only): each tile's blocks split over nsplit CTAs,
// whose partials (prefill_partial_bytes at part: acc, then m, then l) the
// combine kernel merges into out and lse.
cudaError_t launch_dsa_prefill_tc(const DecodeParams& p, int D, int smem, int mask_rows,
                                  void* stage, int nsplit, float* part, cudaStream_t s);
size_t prefill_stage_bytes(long long N, int Hkv, int D, int rows);
size_t prefill_partial_bytes(int rows, int Hq, int D, int nsplit);
// The automatic split count of the dense prefill on a device with sms SMs.
int prefill_auto_splits(int rows, int G, int Hkv, int sms);

cudaError_t launch_combine(const float* acc, const float* m, const float* l, int units,
                           int num_splits, int Hq, int Hkv, int D, const float* sink, void* out,
                           float* lse, cudaStream_t stream);
cudaError_t launch_int8_to_fp16(const int8_t* in, uint16_t* out, int64_t n, cudaStream_t stream);
cudaError_t launch_reshape_and_cache(const void* k_new, const void* v_new, const int32_t* slots,
                                     int num_tokens, int Hkv, int D, void* k_cache,
                                     void* v_cache, long long num_slots, const float* ks,
                                     const float* vs, int per_channel, bool fp8, uint32_t* flags,
                                     cudaStream_t stream);
cudaError_t launch_fp8_to_fp16(const uint8_t* in, uint16_t* out, int64_t n, cudaStream_t stream);

}  // namespace i8kv
