/*
 * int8kv.h -- C ABI of libint8kv.so: split-KV GQA decode attention over an
 * INT8-quantized KV cache on GB300 (sm_103a).
 *
 * The operation (all entry points below compute parts of it):
 *   For each query row r and query head h, with KV head g = h / G and
 *   G = Hq / Hkv (contiguous GQA groups):
 *     K_t = k_scale * code_K[t, g, :]   V_t = v_scale * code_V[t, g, :]
 *         (per-tensor scale: one number; per-channel: scale[g, d])
 *     s_t = softmax_scale * dot(Q[r, h, :], K_t)       (natural-log units)
 *     O[r, h, :] = sum_t exp(s_t - m) V_t / sum_t exp(s_t - m),  m = max_t s_t
 *     lse[r, h]  = m + ln sum_t exp(s_t - m)
 *     optional head sink s_h:  O <- O / (1 + exp(s_h - lse))
 *   over the candidate set of the row: the valid entries of a sparse index
 *   list (onnxruntime PR 33707 "INT8-KV DynamicSparseAttention", Summary of
 *   Changes §1-§2) or the first min(seq_len, cap) tokens of a paged
 *   block-table cache (onnxruntime PR 29912 "PagedAttention: quantized KV
 *   cache ...", CUDA kernels: paged decode, ApplyHeadSink).  The decode calls
 *   split each row's candidates into chunks, run an online softmax per chunk
 *   and merge the partials with a log-sum-exp combine (PR 33707 §2); the split
 *   count comes from the capacity and the row count only (onnx-genai PR 1350
 *   "adaptive split-KV sizing", Summary).
 *
 * Conventions shared by every entry point
 *   - Device pointers are CUDA device addresses of the current device.  The
 *     caller owns every buffer; the library allocates nothing, never
 *     synchronises the host and enqueues work only on `stream` (a
 *     cudaStream_t passed as void*; NULL = the legacy default stream).
 *   - fp16 tensors are passed as uint16_t* (IEEE binary16 bit patterns).
 *   - Layouts are dense row-major with the shapes given per argument.
 *   - Alignment: q, out, caches and per-channel scales must be 16-byte
 *     aligned; index lists, block tables, lengths, lse, sinks and flags
 *     4-byte aligned; the workspace 16-byte aligned.
 *   - Argument errors are reported by the return value before anything is
 *     enqueued.  A launch failure returns I8KV_ECUDA.  Data-dependent
 *     conditions found on the device are OR-ed into the optional `flags`
 *     word (I8KV_FLAG_*) and never stop the kernel.
 *   - Every call with the same shapes and geometry enqueues the same
 *     kernels with the same launch configuration, so calls can be captured
 *     in a CUDA graph; live lengths are read on the device.
 */
#ifndef INT8KV_H_
#define INT8KV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
typedef enum {
  I8KV_OK = 0,
  I8KV_EINVAL = 1,        /* bad argument: NULL required pointer, negative size, bad enum,
                             non-finite or negative softmax scale, geometry that misses the cap */
  I8KV_EUNSUPPORTED = 2,  /* valid but not served: head_dim not 64/128/256, G > 16,
                             softmax_scale > 1, block_size not a multiple of 16, ... */
  I8KV_EALIGN = 3,        /* a pointer breaks the alignment rule above */
  I8KV_EWORKSPACE = 4,    /* workspace NULL or smaller than split_workspace_bytes() */
  I8KV_ECUDA = 5          /* a CUDA runtime call or kernel launch failed */
} i8kv_status;

/* ---- enumerations ------------------------------------------------------- */
#define I8KV_SCALE_PER_TENSOR 1  /* k_scale / v_scale: one float                 */
#define I8KV_SCALE_PER_CHANNEL 2 /* k_scale / v_scale: float [Hkv, D]             */

#define I8KV_CACHE_INT8 1 /* codes in [-128, 127], dequantised with the scales */
#define I8KV_CACHE_FP16 2 /* paged_decode only: values taken as is, scales ignored */
#define I8KV_CACHE_FP8 3  /* paged_decode / reshape_and_cache only: float8 e4m3fn codes,
                             dequantised with the scales (onnxruntime PR 29912, Schema:
                             cache element type float8e4m3fn) */

#define I8KV_CACHE_MX4 4  /* paged_decode_mx4 / rope_and_cache / gather_cache only: 4-bit e2m1
                             codes in blocks of 16 channels, an e4m3 scale for each (the record
                             layout below), times the scales */

#define I8KV_ROPE_HALVES 0      /* rope_and_cache: channels i and i + rot_dim / 2 turn together */
#define I8KV_ROPE_INTERLEAVED 1 /* rope_and_cache: channels 2i and 2i + 1 turn together         */

#define I8KV_GEOM_WAVE 0       /* onnx-genai PR 1350 rule (num_splits from one wave)        */
#define I8KV_GEOM_POW2_TILES 1 /* onnxruntime PR 33707 rule (power-of-two tiles per split)  */
#define I8KV_GEOM_BALANCED 2   /* decode_plan, paged path: balanced pieces (see paged_decode) */

#define I8KV_PATH_DSA 1   /* sparse-candidate decode kernel */
#define I8KV_PATH_PAGED 2 /* paged decode kernel            */

#define I8KV_MAX_PIECES 1024 /* paged_prefill: at most 1024 pieces */
#define I8KV_MAX_SPLITS 32 /* at most 32 splits (onnxruntime PR 33707, §2) */

/* bits OR-ed into the optional device `flags` word */
#define I8KV_FLAG_LEN_CLAMPED 0x1u /* a seq_len was > cap (clamped) or < 0 (taken as 0)       */
#define I8KV_FLAG_QUERY_RANGE 0x2u /* some Q*k_scale is not finite or beyond +-65504 (that CTA
                                      took the FP32 path)                                     */
#define I8KV_FLAG_BAD_BLOCK 0x4u   /* a block-table entry inside the live length is outside
                                      [0, num_blocks): those tokens were skipped              */
#define I8KV_FLAG_BAD_SLOT 0x8u    /* reshape_and_cache: a slot >= num_slots was skipped      */
#define I8KV_FLAG_FP32_PATH 0x10u  /* some CTA evaluated its heads on the FP32 path (see the
                                      numerical eligibility rules below)                     */
#define I8KV_FLAG_WAIT_TIMEOUT 0x20u /* dsa_prefill's tensor-core kernel, paged_decode_mx4,
                                        packed_prefill and paged_prefill: a CTA gave up waiting
                                        (about a second) for its own asynchronous copies or
                                        tensor-core products; its outputs are NaN (of the last
                                        two, rows that it had not come to may be as they were) */

#define I8KV_FLAG_BAD_POSITION 0x40u /* rope_and_cache: a position outside [0, max_pos): that token
                                        was skipped                                         */

/* Human-readable name of a status code (static storage). */
const char* i8kv_status_string(int status);

/* Library ABI version (major*100 + minor).  3.0: dsa_prefill_ws and
 * dsa_prefill_workspace_bytes take num_splits; dsa_prefill_auto_splits.  The
 * number names the signatures: functions that are added leave it as it is, and
 * a caller that loads the library finds them by name (rope_and_cache,
 * gather_cache, paged_decode_mx4, mx4_cache_bytes). */
int32_t i8kv_version(void);

/* The cudaError_t value behind the calling thread's most recent I8KV_ECUDA
 * (0 if there was none). */
int32_t i8kv_last_cuda_error(void);

/*
 * split_geometry -- pure host integer arithmetic, no CUDA call.
 *
 * Chooses the number of splits and the chunk length (in candidates or tokens)
 * from the capacity `cap` (list length or max_blocks*block_size) and the number
 * of independent work units `units` (rows x KV heads), never from a live length.
 *   mode I8KV_GEOM_WAVE (onnx-genai PR 1350, Summary):
 *     n = min(ceil(wave_ctas / units), ceil(cap / min_chunk), max_splits);
 *     chunk = ceil(cap / n) rounded up to a multiple of `granule`;
 *     n = ceil(cap / chunk).  override_value > 0 pins the chunk instead:
 *     n = min(ceil(cap / override_value), max_splits), then as above.
 *   mode I8KV_GEOM_POW2_TILES (onnxruntime PR 33707, §2): tiles = ceil(cap /
 *     granule); tiles_per_split = smallest power of two with
 *     ceil(tiles / tps) * units <= wave_ctas (override_value > 0: that tps as a
 *     target); n = min(ceil(tiles / tps), max_splits); tiles_eff = ceil(tiles /
 *     n); n = ceil(tiles / tiles_eff); chunk = tiles_eff * granule.
 *   cap <= 0 gives n = 1, chunk = granule.
 * Outputs: *num_splits in [1, max_splits], *chunk a multiple of granule with
 * num_splits * chunk >= cap and (num_splits - 1) * chunk < cap.
 * Errors: I8KV_EINVAL for units, wave_ctas, granule, min_chunk or max_splits < 1,
 * override_value < 0, an unknown mode or NULL outputs.
 */
i8kv_status split_geometry(int64_t cap, int32_t units, int32_t wave_ctas, int32_t granule,
                           int32_t min_chunk, int32_t max_splits, int32_t mode,
                           int32_t override_value, int32_t* num_splits, int32_t* chunk);

/*
 * split_workspace_bytes -- bytes of the split workspace for `units` work units
 * of G query heads of dimension D and `num_splits` splits.  Layout (fp32):
 *   acc [units, num_splits, G, D]   un-normalised partial outputs, value-scaled
 *   m   [units, num_splits, G]      running maximum (natural log)
 *   l   [units, num_splits, G]      running sum of exp(s - m)
 * The partial vectors come first so that they stay 16-byte aligned
 * (onnxruntime PR 33707, §2).  Returns 0 for num_splits <= 1 or bad sizes.
 */
size_t split_workspace_bytes(int32_t units, int32_t num_splits, int32_t G, int32_t D);

/*
 * decode_plan -- the geometry a decode call uses when it is given
 * num_splits = 0 (automatic), for the current device.
 *   path: I8KV_PATH_DSA or I8KV_PATH_PAGED; cache_dtype: I8KV_CACHE_INT8, or
 *   (paged only) I8KV_CACHE_FP16, I8KV_CACHE_FP8 or I8KV_CACHE_MX4; cap: max_sel
 *   (DSA) or max_blocks*block_size (paged); rows: S (DSA) or B (paged); mode /
 *   override_value as in split_geometry.  wave_ctas = SM count x resident CTAs per SM of the
 *   selected decode kernel (queried from the CUDA occupancy API and cached per
 *   device); granule = 64 (POW2_TILES) or 16 (WAVE); min_chunk = 128;
 *   mode I8KV_GEOM_BALANCED (paged path only, else I8KV_EUNSUPPORTED):
 *   num_splits = min(32, max(2, 2 x the WAVE rule's automatic count)) partial
 *   slots and chunk = 0, for paged_decode's balanced pieces (for an MX4 cache 1,
 *   2, 4 or 8 where spans are short: see paged_decode_mx4);
 *   max_splits = I8KV_MAX_SPLITS.  For the paged path in WAVE mode with
 *   override_value 0 the chunk is then moved to the multiple of one round of
 *   the paged kernel's CTA (4 warps x its step: 128 positions for an int8 or
 *   e4m3fn cache with head_dim <= 128, else 64) nearer to
 *   ceil(cap / num_splits) -- the lower one only if it is >= 128 and gives at
 *   most I8KV_MAX_SPLITS splits -- and num_splits = ceil(cap / chunk).
 * Outputs: *num_splits, *chunk, *workspace_bytes (0 when one split), and, if
 * wave_ctas is not NULL, the wave used.  Errors as for the decode calls'
 * shape checks, I8KV_ECUDA if the device cannot be queried.
 */
i8kv_status decode_plan(int32_t path, int32_t cache_dtype, int64_t cap, int32_t rows,
                        int32_t Hq, int32_t Hkv, int32_t D, int32_t mode,
                        int32_t override_value, int32_t* num_splits, int32_t* chunk,
                        size_t* workspace_bytes, int32_t* wave_ctas);

/*
 * dsa_decode -- sparse-candidate decode (onnxruntime PR 33707, Summary of
 * Changes §2: split-K decode over a per-row candidate list of an INT8 cache).
 *   q        [S, Hq, D] fp16                 query rows
 *   k_cache  [N, Hkv, D] int8, v_cache same  the main cache (token-major)
 *   k_scale, v_scale, scale_kind             fp32 [1] or [Hkv, D]
 *   idx      [S, max_sel] int32              row r attends the entries of
 *            idx[r, :] that lie in [0, N), in list order, duplicates counted;
 *            any other value is skipped (padding: -1)
 *   softmax_scale                            sigma, 0 <= sigma <= 1 (the FP16
 *            query / probability path is bounded for sigma <= 1: PR 33707 §1)
 *   head_sink [Hq] fp32 or NULL              per-head sink logit (PR 29912)
 *   num_splits, chunk                        geometry: split k of row r covers
 *            list positions [k*chunk, (k+1)*chunk); requires num_splits in
 *            [1, 32], chunk > 0 and a multiple of 16, num_splits*chunk >=
 *            max_sel.  num_splits = 0: automatic (decode_plan, POW2_TILES rule,
 *            chunk ignored).
 *   workspace, workspace_bytes               >= split_workspace_bytes(S*Hkv,
 *            num_splits, G, D) when num_splits > 1 (may be NULL otherwise)
 *   out      [S, Hq, D] fp16                 output.  NULL with num_splits > 1:
 *            write the split partials to the workspace only and enqueue no
 *            combine (the caller runs split_combine later, e.g. after gathering
 *            partials of one row computed on several devices)
 *   lse      [S, Hq] fp32 or NULL            log-sum-exp of the attended scores
 *            (without the sink); -inf for an empty candidate set (O = 0)
 *   flags    device uint32 or NULL           I8KV_FLAG_* bits are OR-ed in
 * Work: one kernel over (S*Hkv units) x num_splits CTAs writing partials, then
 * the split_combine kernel; with one split the decode kernel writes O directly.
 * S = 0 or max_sel = 0 enqueues nothing for S = 0 and writes O = 0, lse = -inf
 * for max_sel = 0.
 */
i8kv_status dsa_decode(const uint16_t* q, const int8_t* k_cache, const int8_t* v_cache,
                       const float* k_scale, const float* v_scale, int32_t scale_kind,
                       const int32_t* idx, int32_t S, int32_t Hq, int32_t Hkv, int32_t D,
                       int64_t N, int32_t max_sel, float softmax_scale, const float* head_sink,
                       int32_t num_splits, int32_t chunk, void* workspace,
                       size_t workspace_bytes, uint16_t* out, float* lse, uint32_t* flags,
                       void* stream);

/*
 * dsa_prefill -- the tensor-core multi-row variant over gathered candidates
 * (onnxruntime PR 33707, Summary of Changes §1: grid (rows, KV heads), no
 * splits, the probability tile as a single FP16 tile).  Arguments as for
 * dsa_decode without the geometry and the workspace; any S >= 0.
 */
i8kv_status dsa_prefill(const uint16_t* q, const int8_t* k_cache, const int8_t* v_cache,
                        const float* k_scale, const float* v_scale, int32_t scale_kind,
                        const int32_t* idx, int32_t S, int32_t Hq, int32_t Hkv, int32_t D,
                        int64_t N, int32_t max_sel, float softmax_scale,
                        const float* head_sink, uint16_t* out, float* lse, uint32_t* flags,
                        void* stream);

/*
 * dsa_prefill_workspace_bytes -- bytes of the workspace that lets dsa_prefill_ws
 * take the staged form of the tensor-core kernel for this shape and split
 * count (num_splits as for dsa_prefill_ws; 0 = the automatic count on the
 * current device): Hkv x ceil(N / 128) x 2 x 128 x D x 2 (the cache as fp16
 * operand images) + S x ceil(N / 128) x 16 (every row's candidate bitmask)
 * + S x 4 (every row's repeat flag), plus with more than one split, from the
 * next 256-byte boundary, S x Hq x splits x (D + 2) x 4 (the splits' fp32
 * partials: the accumulators, then m, then l).  0 when the tensor-core kernel does not
 * serve the shape (head_dim other than 128 / 256, 4 * max_sel < N, masks too
 * large for shared memory, S, N or max_sel < 1, bad heads) or num_splits is
 * outside [0, 32].  Host only (the automatic count reads the SM count).
 */
size_t dsa_prefill_workspace_bytes(int32_t S, int32_t Hq, int32_t Hkv, int32_t D, int64_t N,
                                   int32_t max_sel, int32_t num_splits);

/*
 * dsa_prefill_auto_splits -- the automatic split count of the tensor-core
 * prefill (num_splits = 0) on a device with `sms` SMs: with tiles = Hkv x
 * ceil(S x (Hq / Hkv) / 128) tiles of 128 (row, head) vectors, min(8, sms /
 * tiles) where 2 x tiles <= sms, else 1 (a split's partials cost a round trip
 * through the combine kernel, paid back only where tiles leave SMs idle).
 * 0 for S < 1, sms < 1 or bad heads.  Host arithmetic only.
 */
int32_t dsa_prefill_auto_splits(int32_t S, int32_t Hq, int32_t Hkv, int32_t sms);

/*
 * dsa_prefill_ws -- dsa_prefill with an optional workspace (the caller's device
 * memory, 16-byte aligned, workspace_bytes >= dsa_prefill_workspace_bytes for
 * the same num_splits).  With one, where the tensor-core kernel serves the
 * shape, the call first converts the cache once into fp16 operand images in
 * the workspace (a kernel of its own, about 3 bytes written per cache byte
 * read, whose other CTAs also turn each row's list into a bitmask of cache
 * positions) and the prefill kernel copies each block in with one bulk copy
 * instead of converting it in every CTA; unsplit, the results are the same
 * bit for bit.
 *   num_splits  0: automatic -- where a KV head's tiles of 128 (row, head)
 *               vectors number fewer than half the SMs, each tile's blocks
 *               are split over min(8, SMs / tiles) CTAs, else 1;
 *               1 .. 32: that many (a split may get no block).
 *               With more than one, each CTA writes the fp32 partials of its
 *               share of the tile's blocks (and of the candidates at their
 *               positions; a vector sent to the FP32 path publishes an FP32
 *               partial of its share), and the split_combine kernel merges
 *               them with the sink into out and lse (onnxruntime PR 33707,
 *               Summary of Changes §2: the split-K partials and their merge).
 * With workspace NULL, or where the gathering kernel serves the shape, it is
 * dsa_prefill (unsplit; num_splits has no effect on the gathering kernel).
 * The workspace holds nothing the caller needs afterwards.
 * Errors: as dsa_prefill; I8KV_EINVAL if num_splits is outside [0, 32];
 * I8KV_EWORKSPACE if workspace_bytes is too small, or workspace is NULL with
 * num_splits > 1 on the tensor-core path; I8KV_EALIGN if the workspace is not
 * 16-byte aligned.
 */
i8kv_status dsa_prefill_ws(const uint16_t* q, const int8_t* k_cache, const int8_t* v_cache,
                           const float* k_scale, const float* v_scale, int32_t scale_kind,
                           const int32_t* idx, int32_t S, int32_t Hq, int32_t Hkv, int32_t D,
                           int64_t N, int32_t max_sel, float softmax_scale,
                           const float* head_sink, int32_t num_splits, void* workspace,
                           size_t workspace_bytes, uint16_t* out, float* lse, uint32_t* flags,
                           void* stream);

/*
 * paged_decode -- split-KV decode over a paged block-table cache
 * (onnxruntime PR 29912, CUDA kernels: "split-KV, block-table-aware decode
 * with native head-sink ... and on-the-fly cache dequantization").
 *   q            [B, Hq, D] fp16              one query row per sequence
 *   k_cache, v_cache [num_blocks, block_size, Hkv, D] int8, float8 e4m3fn or fp16
 *   cache_dtype  I8KV_CACHE_INT8, I8KV_CACHE_FP8 (both dequantised with the
 *                scales) or I8KV_CACHE_FP16 (scales ignored, may be NULL)
 *   block_table  [B, max_blocks] int32        token t of sequence b is row
 *                block_table[b, t / block_size] * block_size + t % block_size
 *   seq_lens     [B] int32, DEVICE memory     live lengths, clamped to
 *                cap = max_blocks * block_size (I8KV_FLAG_LEN_CLAMPED)
 *   block_size   a multiple of 16
 *   num_splits, chunk  as for dsa_decode over token positions, with cap =
 *                max_blocks*block_size; num_splits = 0: automatic (WAVE rule).
 *                num_splits in [2, 32] with chunk = 0: balanced pieces (not on
 *                the pages; decode_plan's I8KV_GEOM_BALANCED gives the values):
 *                num_splits partial slots per row and ceil(num_splits / 2)
 *                CTAs per (row, KV head), all fixed by the arguments, while
 *                each CTA cuts its piece of a row's live range on the device
 *                from all live lengths, so that the pieces are about equally
 *                long across a ragged batch (about one occupancy wave of
 *                them); the combine merges the used slots, the others are
 *                marked empty.  Needs B <= 128 and slots_out NULL
 *                (I8KV_EUNSUPPORTED otherwise).
 *   slots_out    [B, cap] int32 or NULL       debug output: the gathered row of
 *                every token position, -1 past the live length
 *   other arguments as for dsa_decode.
 */
i8kv_status paged_decode(const uint16_t* q, const void* k_cache, const void* v_cache,
                         int32_t cache_dtype, const float* k_scale, const float* v_scale,
                         int32_t scale_kind, const int32_t* block_table,
                         const int32_t* seq_lens, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                         int32_t block_size, int32_t max_blocks, int64_t num_blocks,
                         float softmax_scale, const float* head_sink, int32_t num_splits,
                         int32_t chunk, void* workspace, size_t workspace_bytes, uint16_t* out,
                         float* lse, int32_t* slots_out, uint32_t* flags, void* stream);

/*
 * paged_decode_ex -- paged_decode with the two score options the same page
 * lists for that kernel (onnxruntime PR 29912, CUDA kernels: "native head-sink,
 * softcap, sliding-window and on-the-fly cache dequantization").  The page
 * names them without a definition; the meanings taken are:
 *   softcap  >= 0, finite.  > 0: each scaled score s becomes
 *            softcap * tanh(s / softcap) before the softmax; 0: off.  The
 *            head-sink logit is not capped.  (Computed as softcap - 2 softcap /
 *            (1 + e^(2 s / softcap)): the error is up to 2^-21 of softcap, not of
 *            s, so a cap far above the scores makes them coarse.)
 *   window   >= -1.  >= 0: the query of sequence b (at position L - 1, L its
 *            clamped live length) attends positions [max(0, L-1-window), L):
 *            itself and the window positions before it; -1: off.
 * With a window the splits count their chunks from the window start rounded
 * down to a multiple of 16, and num_splits * chunk must cover
 * I8KV_WINDOW_SPAN(cap, window) (not cap); num_splits = 0 plans over that span
 * (decode_plan with cap = I8KV_WINDOW_SPAN(cap, window) gives the same
 * geometry).  slots_out then holds -1 outside the window.  Other arguments,
 * errors and work as for paged_decode; softcap < 0, non-finite, or
 * window < -1 -> I8KV_EINVAL.
 */
#define I8KV_WINDOW_SPAN(cap, window)                                              \
  ((window) < 0 || (int64_t)(cap) <= (int64_t)(window) + 16 ? (int64_t)(cap)      \
                                                            : (int64_t)(window) + 16)

/* paged_window_span -- I8KV_WINDOW_SPAN(cap, window) as a function, for
 * bindings that cannot expand the macro: the positions a windowed paged decode's
 * splits cover (cap when window < 0).  Pure host arithmetic, no CUDA call. */
int64_t paged_window_span(int64_t cap, int32_t window);

i8kv_status paged_decode_ex(const uint16_t* q, const void* k_cache, const void* v_cache,
                            int32_t cache_dtype, const float* k_scale, const float* v_scale,
                            int32_t scale_kind, const int32_t* block_table,
                            const int32_t* seq_lens, int32_t B, int32_t Hq, int32_t Hkv,
                            int32_t D, int32_t block_size, int32_t max_blocks, int64_t num_blocks,
                            float softmax_scale, const float* head_sink, float softcap,
                            int32_t window, int32_t num_splits, int32_t chunk, void* workspace,
                            size_t workspace_bytes, uint16_t* out, float* lse,
                            int32_t* slots_out, uint32_t* flags, void* stream);

/*
 * split_combine -- log-sum-exp merge of split partials plus the head sink
 * (onnxruntime PR 33707 §2: the merge kernel; PR 29912: ApplyHeadSink):
 *   M = max_k m_k;  L = sum_k l_k exp(m_k - M);  O = sum_k acc_k exp(m_k - M) / L
 *   lse = M + ln L;  O <- O / (1 + exp(s_h - lse)) if a sink is given.
 * Splits with m_k = -inf are skipped (their acc is not read); all skipped:
 * O = 0, lse = -inf.
 * A split with m_k > -inf and a sum l_k that is NaN (or m_k = +inf or NaN): O
 * and lse are NaN.
 *   acc [units, num_splits, G, D], m, l [units, num_splits, G] fp32 (the
 *   workspace layout of split_workspace_bytes); unit u = row * Hkv + g;
 *   G = Hq / Hkv; out [units*G, D] fp16 (= [rows, Hq, D]); lse [units*G] or
 *   NULL; head_sink [Hq] or NULL, indexed by h = (u % Hkv) * G + j.
 *   num_splits in [1, 32]; D in {64, 128, 256}.
 */
i8kv_status split_combine(const float* acc, const float* m, const float* l, int32_t units,
                          int32_t num_splits, int32_t Hq, int32_t Hkv, int32_t D,
                          const float* head_sink, uint16_t* out, float* lse, void* stream);

/*
 * reshape_and_cache -- quantize-on-write of new key / value rows into a paged
 * INT8 or float8 e4m3fn cache (onnxruntime PR 29912, CUDA kernels:
 * "ReshapeAndCache quantizes on write"; Schema: cache element type int8 or
 * float8e4m3fn).  For every new token n and KV head g, the cache row
 * (slot_mapping[n], g) receives, with q = x[d] / scale:
 *     I8KV_CACHE_INT8: code[d] = clamp(round_half_even(q), -127, 127)
 *     I8KV_CACHE_FP8:  code[d] = the e4m3fn value nearest q (ties to even),
 *                      saturated to +-448
 * with scale = k_scale / v_scale per tensor ([1]) or per channel ([Hkv, D]); q
 * is the IEEE fp32 quotient of the fp16 value widened to fp32 (exactly: the
 * kernel's faster product by the reciprocal falls back to the division
 * wherever the two could round differently); a NaN quotient stores 0.
 *   k_new, v_new   [num_tokens, Hkv, D] fp16, device
 *   slot_mapping   [num_tokens] int32, device: row of the flattened cache
 *                  (block * block_size + offset); < 0: skipped (padding);
 *                  >= num_slots: skipped and I8KV_FLAG_BAD_SLOT raised
 *   k_cache, v_cache [num_slots, Hkv, D] bytes (a paged cache [num_blocks,
 *                  block_size, Hkv, D] with num_slots = num_blocks * block_size)
 *   cache_dtype    I8KV_CACHE_INT8 or I8KV_CACHE_FP8 (others: I8KV_EINVAL)
 *   D a multiple of 8; caches, rows and per-channel scales 16-byte aligned.
 * Scales must be finite and positive (not checked on the device).
 */
i8kv_status reshape_and_cache(const uint16_t* k_new, const uint16_t* v_new,
                              const int32_t* slot_mapping, int32_t num_tokens, int32_t Hkv,
                              int32_t D, void* k_cache, void* v_cache, int64_t num_slots,
                              const float* k_scale, const float* v_scale, int32_t scale_kind,
                              int32_t cache_dtype, uint32_t* flags, void* stream);

/*
 * The MX4 cache -- 4-bit keys and values with a scale for every 16 channels.
 * (Blocks of 16 with an e4m3 scale under an fp32 outer scale.  Microscaling
 * data with blocks of 32 and power-of-two scales is another format and is not
 * taken.)
 *   cache [num_blocks, Hkv, block_size / 16, 18 * D] bytes, 16-byte aligned,
 *   block_size a multiple of 16.  One record of 18 * D bytes holds 16
 *   consecutive tokens of a block for one KV head (one contiguous copy):
 *     [0, 8D)    K codes   [16, D / 2]   e2m1, channel 2j in the low nibble of
 *                                        byte j, channel 2j + 1 in the high one
 *     [8D, 9D)   K scales  [16, D / 16]  float8 e4m3fn, >= 0, one per 16 channels
 *     [9D, 17D)  V codes   [16, D / 2]
 *     [17D, 18D) V scales  [16, D / 16]
 *   K[t, g, d] = k_scale * (block scale * code value), V likewise, with k_scale
 *   and v_scale per tensor ([1]) or per channel ([Hkv, D]) as everywhere here.
 *   The product block scale * code value has 6 significant bits: it is exact in
 *   fp16 and fp32.  9 / 16 of a byte per value.
 *   D: 64, 128 or 256.
 * mx4_cache_bytes -- bytes of such a cache, 0 for sizes it does not take.  Host
 * arithmetic only.
 */
size_t mx4_cache_bytes(int64_t num_blocks, int32_t block_size, int32_t Hkv, int32_t D);

/*
 * rope_and_cache -- append new rows to a paged cache, the position rotation
 * applied on the way: q and k rotated, q written out, k and v written into the
 * cache in its type, all in one launch.  With p = positions[n], R = rot_dim and
 * the pair (a, b) = channels (i, i + R/2) (I8KV_ROPE_HALVES) or (2i, 2i + 1)
 * (I8KV_ROPE_INTERLEAVED), i = 0 .. R/2 - 1:
 *     a' = a cos[p, i] - b sin[p, i]     b' = b cos[p, i] + a sin[p, i]
 * in fp32, each product and the sum rounded on its own (no fused
 * multiply-add: the stored codes follow from the formula bit for bit).
 * Channels >= R are not turned.
 *     q_out = fp16(q')
 *     I8KV_CACHE_FP16: cache row = fp16(k'), v; the scales are not used
 *     I8KV_CACHE_INT8, I8KV_CACHE_FP8: the codes that reshape_and_cache stores of
 *        k' (in fp32, not rounded to fp16 first) and v
 *     I8KV_CACHE_MX4: y = x * fl(1 / scale); per block of 16 channels the scale
 *        s = the e4m3fn value nearest max |y| * fl(1 / 6) (ties to even, at most
 *        448), code = the e2m1 value nearest y * fl(1 / s) (ties to even, at most
 *        +-6); s = 0 stores codes 0.  A NaN stores 0 and does not count in the
 *        maximum.
 *   q, k_new, v_new [num_tokens, H, D] fp16, H = Hq, Hkv, Hkv: the heads of a
 *                  token contiguous, the tokens q_stride / k_stride / v_stride
 *                  elements apart (multiples of 8: the three may be slices of one
 *                  projection's output).  q may be NULL with Hq = 0.
 *   positions      [num_tokens] int32; may be NULL with rot_dim = 0
 *   cos_sin        [max_pos, rot_dim] fp32: rot_dim / 2 cosines, then the sines;
 *                  16-byte aligned; may be NULL with rot_dim = 0
 *   rot_dim        0 .. D, a multiple of 16; with I8KV_ROPE_HALVES and an MX4
 *                  cache a multiple of 32 (I8KV_EUNSUPPORTED otherwise)
 *   slot_mapping   [num_tokens] int32, as for reshape_and_cache: < 0 writes no
 *                  cache row (q is still rotated); >= num_slots: the same, and
 *                  I8KV_FLAG_BAD_SLOT.  A slot named twice ends up with either
 *                  row, or a mixture of the two.
 *   q_out          [num_tokens, Hq, D] fp16, dense; may be q itself where
 *                  q_stride = Hq * D
 *   k_cache, v_cache [num_slots, Hkv, D] of the cache type; with I8KV_CACHE_MX4
 *                  k_cache is the record cache and v_cache is NULL
 *   block_size     of an MX4 cache (num_slots = num_blocks * block_size); not
 *                  looked at otherwise
 *   D a multiple of 16 (64, 128 or 256 for MX4).
 * A token whose position is outside [0, max_pos) is skipped (its q_out and cache
 * rows stay as they were) and raises I8KV_FLAG_BAD_POSITION unless its slot is
 * < 0 (padding).
 */
i8kv_status rope_and_cache(const uint16_t* q, int64_t q_stride, const uint16_t* k_new,
                           int64_t k_stride, const uint16_t* v_new, int64_t v_stride,
                           const int32_t* positions, const float* cos_sin, int64_t max_pos,
                           int32_t rot_dim, int32_t rot_style, const int32_t* slot_mapping,
                           int32_t num_tokens, int32_t Hq, int32_t Hkv, int32_t D,
                           uint16_t* q_out, void* k_cache, void* v_cache, int32_t cache_dtype,
                           int64_t num_slots, int32_t block_size, const float* k_scale,
                           const float* v_scale, int32_t scale_kind, uint32_t* flags,
                           void* stream);

/*
 * norm_rope_and_cache -- rope_and_cache with the heads of queries and keys normed
 * before the rotation, in the same pass.  For every head of D channels, in fp32:
 *     x' = x * r * weight[d],  r = 1 / sqrt(sum_d x^2 / D + eps)
 * then the rotation and the stores as for rope_and_cache.  Values are not normed.
 * The products are rounded each on its own, and r is within 2 units of the last
 * place of 1 / sqrt of the fp32 mean + eps (rsqrtf; the squares of 16 channels are
 * summed in two chains of fused products, the even channels and the odd ones, then
 * over the head by halves).  So a normed head's rows are determined to 24 roundings
 * of 2^-24, not bit for bit as rope_and_cache's are: a code whose value lies that
 * near to a boundary may be either of two.  The same call gives the same bits.
 *   q_weight, k_weight  [D] fp32, 16-byte aligned; NULL: not normed
 *   eps          finite, >= 0
 *   k_out        [num_tokens, Hkv, D] fp16, dense, or NULL: the normed and turned
 *                keys, rounded once, as attention over the new tokens alone wants
 *                them (packed_prefill); written for every token whose position is in
 *                range, also where the slot is not; may be k_new itself where k_stride
 *                = Hkv * D
 *   D 64, 128 or 256 where a weight is given (I8KV_EUNSUPPORTED otherwise).
 *   The other arguments as for rope_and_cache.  A head with a NaN is NaN, one with an
 *   infinity is NaN there and zero elsewhere (before it is turned), a head of zeros
 *   with eps = 0 is NaN; a NaN stores code 0 (an fp16 cache keeps it).
 */
i8kv_status norm_rope_and_cache(const uint16_t* q, int64_t q_stride, const uint16_t* k_new,
                                int64_t k_stride, const uint16_t* v_new, int64_t v_stride,
                                const float* q_weight, const float* k_weight, float eps,
                                const int32_t* positions, const float* cos_sin, int64_t max_pos,
                                int32_t rot_dim, int32_t rot_style, const int32_t* slot_mapping,
                                int32_t num_tokens, int32_t Hq, int32_t Hkv, int32_t D,
                                uint16_t* q_out, uint16_t* k_out, void* k_cache, void* v_cache,
                                int32_t cache_dtype, int64_t num_slots, int32_t block_size,
                                const float* k_scale, const float* v_scale, int32_t scale_kind,
                                uint32_t* flags, void* stream);

/*
 * gather_cache -- cache rows back as fp16 values (the inverse of the append, for
 * a dense prefill over a cached prefix, or to look at what is stored):
 *     out[n, g, :] = fp16(scale * value of the cache row (slot_mapping[n], g)),
 * the fp32 product rounded once; a row of zeros for a slot < 0, and for a slot
 * >= num_slots, which raises I8KV_FLAG_BAD_SLOT.  An fp16 cache is copied.
 *   slot_mapping [num_rows] int32, any order, repeats allowed
 *   k_out, v_out [num_rows, Hkv, D] fp16, 16-byte aligned; either may be NULL
 *   caches, cache_dtype, num_slots, block_size, scales and D as for
 *   rope_and_cache (all four cache types).
 */
i8kv_status gather_cache(const int32_t* slot_mapping, int32_t num_rows, int32_t Hkv, int32_t D,
                         const void* k_cache, const void* v_cache, int32_t cache_dtype,
                         int64_t num_slots, int32_t block_size, const float* k_scale,
                         const float* v_scale, int32_t scale_kind, uint16_t* k_out,
                         uint16_t* v_out, uint32_t* flags, void* stream);

/*
 * paged_decode_mx4 -- paged_decode_ex over an MX4 cache: one new token per
 * sequence, split over the cache's length and joined.
 *   cache        [num_blocks, Hkv, block_size / 16, 18 * D] (see above)
 *   num_splits, chunk  as for paged_decode; num_splits = 0: automatic, the values
 *                of decode_plan(I8KV_PATH_PAGED, I8KV_CACHE_MX4,
 *                I8KV_WINDOW_SPAN(cap, window), ..., I8KV_GEOM_BALANCED).
 *                One split, and balanced pieces (chunk 0) of 2, 4 or 8 slots for
 *                few rows and out given, run as one kernel: a CTA, or a cluster
 *                of num_splits CTAs, per row and KV head, which deals the row's
 *                tiles out in turn and joins in shared memory; the workspace is
 *                not written then.  Other balanced pieces take any batch size:
 *                the live lengths are cut on the device into pieces of about
 *                equal length, about one occupancy wave of them over the batch,
 *                at most num_splits per row, and the combine kernel joins them.
 *   other arguments as for paged_decode_ex, without slots_out; partials in the
 *   workspace have the same layout (a workspace of their size is asked for
 *   whenever num_splits > 1).
 * Numerics: the K and V values of the cache are exact in the fp16 products;
 * Q * k_scale is held as two fp16 numbers with one power of two per head taken
 * out (per channel scales; a scale per tensor is applied to the fp32 scores), so
 * its range is not limited, and I8KV_FLAG_QUERY_RANGE and I8KV_FLAG_FP32_PATH are
 * not raised; the probabilities are rounded to fp16 (by at most a relative
 * 2^-11), the sums are fp32.  A head whose query is not finite gives NaN outputs,
 * the others of its group what they give without it.
 */
i8kv_status paged_decode_mx4(const uint16_t* q, const void* cache, const float* k_scale,
                             const float* v_scale, int32_t scale_kind,
                             const int32_t* block_table, const int32_t* seq_lens, int32_t B,
                             int32_t Hq, int32_t Hkv, int32_t D, int32_t block_size,
                             int32_t max_blocks, int64_t num_blocks, float softmax_scale,
                             const float* head_sink, float softcap, int32_t window,
                             int32_t num_splits, int32_t chunk, void* workspace,
                             size_t workspace_bytes, uint16_t* out, float* lse, uint32_t* flags,
                             void* stream);

/*
 * packed_prefill -- causal attention over whole prompts, packed one after
 * another: what a prompt's own tokens attend before anything of it is cached.
 * Sequence b's tokens are the rows seq_start[b] .. seq_start[b + 1] - 1; its
 * token i attends the tokens [max(0, i - window), i] of the same sequence
 * (window -1: [0, i]), with
 *     s_t = softmax_scale * dot(Q[i, h], K[t, g]), softcap * tanh(s_t / softcap)
 *           where softcap > 0;  O and lse as at the top of this file.
 *   q            [T, Hq, D] fp16, k, v [T, Hkv, D] fp16: the heads of a token
 *                contiguous, the tokens q_stride / k_stride / v_stride elements
 *                apart (multiples of 8: the three may be slices of one
 *                projection's output); strides of a single token are not used
 *   seq_start    [B + 1] int32, device memory, not falling, in [0, T].  Values
 *                outside are clamped (I8KV_FLAG_LEN_CLAMPED); rows before the
 *                first sequence and behind the last stay as they are in out and
 *                lse; a sequence may be empty
 *   head_sink, softcap, window  as for paged_decode_ex (with caps above 128 a
 *                capped score is within 2^-18.9 of itself, however far below it)
 *   out          [T, Hq, D] fp16, dense;  lse [T, Hq] fp32 or NULL
 * Work: one kernel on the tensor cores (tcgen05); its grid depends on T, B and
 * the heads only.  The probabilities are rounded to fp16 (by at most a relative
 * 2^-11), scores and sums are fp32.  A value that is not finite reaches the rows
 * that attend it and no others; a query that is not finite makes its row NaN.
 */
i8kv_status packed_prefill(const uint16_t* q, int64_t q_stride, const uint16_t* k,
                           int64_t k_stride, const uint16_t* v, int64_t v_stride,
                           const int32_t* seq_start, int32_t T, int32_t B, int32_t Hq, int32_t Hkv,
                           int32_t D, float softmax_scale, const float* head_sink, float softcap,
                           int32_t window, uint16_t* out, float* lse, uint32_t* flags,
                           void* stream);

/*
 * paged_prefill -- causal attention of chunks of new tokens over a paged cache
 * that holds them already (rope_and_cache, norm_rope_and_cache,
 * reshape_and_cache): the next chunk of a prompt, proposed tokens that are
 * checked at once, single tokens, and batches that mix them.  Sequence b has
 * n = query_start[b + 1] - query_start[b] new tokens, the last n of its
 * seq_lens[b] cached ones: token i sits at position p = seq_lens[b] - n + i and
 * attends [max(0, p - window), p].  A token at a negative position attends
 * nothing (O = 0, lse = -inf).
 *   q            [T, Hq, D] fp16, tokens q_stride elements apart (as above)
 *   caches, cache_dtype, scales, block_table, block_size, max_blocks, num_blocks
 *                as for paged_decode (I8KV_CACHE_INT8, _FP8, _FP16), or
 *                I8KV_CACHE_MX4 with k_cache the record cache and v_cache NULL
 *   seq_lens     [B] int32, device, clamped to cap = max_blocks * block_size
 *                (I8KV_FLAG_LEN_CLAMPED); query_start [B + 1] as seq_start above
 *   num_splits   1: every (tile of tokens, KV head) is worked on by one CTA.  2 ..
 *                I8KV_MAX_PIECES: the batch's blocks of 128 positions are cut, on the
 *                device, into that many pieces of about equal length, one per CTA,
 *                whose ends fall anywhere in a tile's range; what belongs to one tile
 *                is merged by a second kernel.  0: automatic, by T, B and the heads
 *                (the lengths are not known here) -- as many pieces as the device has
 *                SMs where the whole (tile, KV head)s would leave many of them idle:
 *                with tiles of 128 vectors (sequences below 192 on average, or D =
 *                256) fewer than three to an SM, with tiles of 256 fewer than nine
 *                tenths to an SM (of one sequence: a last round that is not nearly
 *                full, of up to four); and cap > 128.  Unsplit else, and where the
 *                workspace is too small for it
 *   workspace, workspace_bytes  paged_prefill_workspace_bytes(..., num_splits) for
 *                num_splits > 1 (16-byte aligned, else I8KV_EALIGN; too small
 *                I8KV_EWORKSPACE); may be NULL for 0 and 1.  Nothing in it
 *                outlives the call
 *   out, lse, head_sink, softcap, window  as for packed_prefill
 * For a batch of single tokens alone paged_decode (MX4: paged_decode_mx4) is the
 * faster call: it works on the vectors that are there, this one on tiles of 128 (16
 * sequences of 512 to 8192, 32 / 8 heads x 128: int8 50 us against 75, MX4 30
 * against 67, fp16 71 against 78).
 * A block-table entry of an attended position outside [0, num_blocks) is skipped
 * (I8KV_FLAG_BAD_BLOCK); entries of positions that nobody attends are not used.
 * Numerics: the cache's values are exact in the fp16 products, v_scale is applied
 * to the fp32 sums, a k_scale per tensor to the fp32 scores; a k_scale per
 * channel is folded into the query, rounded to fp16 with a power of two taken
 * out (a relative 2^-11 of each term).  Q * k_scale must be finite in fp32.
 * The rest as for packed_prefill.
 */
i8kv_status paged_prefill(const uint16_t* q, int64_t q_stride, const void* k_cache,
                          const void* v_cache, int32_t cache_dtype, const float* k_scale,
                          const float* v_scale, int32_t scale_kind, const int32_t* block_table,
                          const int32_t* seq_lens, const int32_t* query_start, int32_t T,
                          int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t block_size,
                          int32_t max_blocks, int64_t num_blocks, float softmax_scale,
                          const float* head_sink, float softcap, int32_t window,
                          int32_t num_splits, void* workspace, size_t workspace_bytes,
                          uint16_t* out, float* lse, uint32_t* flags, void* stream);

/*
 * paged_prefill_workspace_bytes -- bytes of the workspace of paged_prefill for T
 * new tokens of B sequences with at most cap positions and the given num_splits
 * (0: what the automatic choice takes on the current device): two tiles of 128 or
 * 256 vectors' partials for each piece, splits x 2 x 128 (or 256) x (D + 2) x 4;
 * 0 where it does not split, and for bad sizes.  Host only.
 * This does not grow with T and B: a large batch may run whole and need nothing
 * where a smaller one is split, and the same T in fewer sequences may take the
 * larger tiles.  A workspace for all batches of a serving loop has
 *     pieces x 2 x M x (D + 2) x 4 bytes, M = 256 for D 64 and 128, 128 for D 256
 * (pieces: num_splits, or for 0 the device's SMs; 41 MB for 152 SMs at most), as
 * this function gives for T = 256, B = 1 and num_splits = pieces.
 */
size_t paged_prefill_workspace_bytes(int32_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                     int64_t cap, int32_t num_splits);

/*
 * dsa_decode_static_workspace -- dsa_decode without a caller-supplied
 * workspace, for callers that cannot allocate device memory when they call
 * (an engine's enqueue step that must not allocate, code with no access to the
 * application's allocator, loops that must never enter the allocator).  The
 * pages have no counterpart; this is a convenience of this library.
 *   Arguments and results as for dsa_decode, without workspace and
 *   workspace_bytes, except that out must not be NULL when S > 0 (I8KV_EINVAL:
 *   partials left in the library's private array could not be read by the
 *   caller).  The split partials go to a device array inside the
 *   library of I8KV_STATIC_WORKSPACE_BYTES bytes, allocated when CUDA loads the
 *   library's device code on a device and held on every such device until the
 *   process exits.  Nothing is allocated or freed by the call itself.
 *   - A geometry whose partials need more than I8KV_STATIC_WORKSPACE_BYTES
 *     (split_workspace_bytes(S*Hkv, num_splits, G, D)) returns
 *     I8KV_EWORKSPACE before anything is enqueued.
 *   - The first call on a device looks the array's device address up
 *     (cudaGetSymbolAddress, with that device current) and caches it; make that
 *     first call before any stream capture.  The cached address belongs to the
 *     device's current CUDA context: do not call this entry point again after
 *     cudaDeviceReset (or any other teardown of the primary context) in the
 *     same process.
 *   - All calls on a device share the one array.  Calls whose kernels can run
 *     at the same time on the GPU (different streams without ordering between
 *     them) race on it and give wrong results; calls ordered on one stream are
 *     fine.  Nothing in it needs clearing between calls: each call's decode
 *     kernel writes the (m, l) entry of every (unit, split, head) that its
 *     combine reads, and the combine reads a split's partial vector only when
 *     that split wrote it.
 */
#define I8KV_STATIC_WORKSPACE_BYTES (4u * 1024u * 1024u)
i8kv_status dsa_decode_static_workspace(const uint16_t* q, const int8_t* k_cache,
                                        const int8_t* v_cache, const float* k_scale,
                                        const float* v_scale, int32_t scale_kind,
                                        const int32_t* idx, int32_t S, int32_t Hq, int32_t Hkv,
                                        int32_t D, int64_t N, int32_t max_sel,
                                        float softmax_scale, const float* head_sink,
                                        int32_t num_splits, int32_t chunk, uint16_t* out,
                                        float* lse, uint32_t* flags, void* stream);

/*
 * int8_to_fp16 -- the decode kernels' in-register int8 -> fp16 conversion
 * applied to a buffer (byte permutes into the mantissa of 1024 + 128, then one
 * fp16x2 subtraction of 1152: exact for all 256 codes; onnxruntime PR 29912,
 * "int8->fp16 conversion fast path").  in [n] int8, out [n] fp16, n a multiple
 * of 4, both 16-byte aligned.  For tests of the conversion.
 */
i8kv_status int8_to_fp16(const int8_t* in, uint16_t* out, int64_t n, void* stream);

/*
 * fp8_to_fp16 -- the paged decode kernel's float8 e4m3fn -> fp16 conversion
 * (cvt.rn.f16x2.e4m3x2, exact) over a device buffer of n codes, n a multiple of
 * 4, both buffers 16-byte aligned; out[i] is the value of in[i] (NaN for the
 * two NaN patterns).  Exposed so that the conversion can be checked
 * exhaustively.
 */
i8kv_status fp8_to_fp16(const uint8_t* in, uint16_t* out, int64_t n, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* INT8KV_H_ */
