// Append of new rows to a paged cache with the position rotation applied on the
// way (rope_and_cache), and the read-back of cache rows as fp16 (gather_cache).
//
// Rotation of a pair (a, b) of channels by the angle of its position:
//   a' = a cos - b sin,  b' = b cos + a sin
// in fp32, every product and sum rounded on its own, so that the stored codes
// follow from the formula bit for bit.  Queries leave as fp16; keys and values
// are stored in the cache's type:
//   int8, e4m3fn  the codes of the IEEE quotient x / scale (as the plain
//                 quantize-on-write stores them)
//   fp16          x rounded once
//   MX4           y = x fl(1/scale); block scale s = e4m3(min(max|y| fl(1/6), 448)),
//                 code = e2m1(y fl(1/s))
//
// One thread takes an item: 16 channels of one head of one token, as two pieces
// of 8 (two 16-byte loads).  In the turned part with the halves rotated
// together the pieces are channels 8j .. 8j+7 and their partners rot_dim / 2
// further on; everywhere else they are adjacent.  An MX4 block of 16 channels is
// then either the thread's own two pieces or (halves) one piece of each of two
// adjacent lanes, which exchange their maxima with one shuffle.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/int8kv.h"
#include "codes.cuh"
#include "device.cuh"
#include "internal.h"

namespace i8kv {

namespace {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ void unpack8(uint4 r, float (&x)[8]) {
  const __half2* h = reinterpret_cast<const __half2*>(&r);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(h[j]);
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_h2(x[0], x[1]), pack_h2(x[2], x[3]), pack_h2(x[4], x[5]),
                    pack_h2(x[6], x[7]));
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float ta = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = ta;
}

// Codes of 8 channels for an int8 or e4m3fn cache: s the scales of the channels.
template <bool FP8>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], const float* __restrict__ s,
                                        int s_step) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float q0 = nan_to_zero(__fdiv_rn(x[j], s[j * s_step]));
    const float q1 = nan_to_zero(__fdiv_rn(x[j + 1], s[(j + 1) * s_step]));
    const uint32_t b =
        FP8 ? e4m3x2_of(q0, q1) : int8_byte(int8_code(q0)) | (int8_byte(int8_code(q1)) << 8);
    w[j / 4] |= b << (8 * (j % 4));
  }
  return make_uint2(w[0], w[1]);
}

template <int CACHE>
__global__ void __launch_bounds__(kAppendThreads)
rope_and_cache_kernel(const AppendParams p) {
  grid_dependency_wait();
  const int ipr = p.D >> 4;                  // items per row
  const int ipt = (p.Hq + 2 * p.Hkv) * ipr;  // items per token
  const long long flat = blockIdx.x * (long long)kAppendThreads + threadIdx.x;
  const long long n = flat / ipt;
  if (n >= p.num_tokens) return;
  const int item = (int)(flat - n * ipt);
  const int head = item / ipr, j = item - (item / ipr) * ipr;
  const bool is_q = head < p.Hq, is_v = head >= p.Hq + p.Hkv;
  const int h = is_q ? head : (is_v ? head - p.Hq - p.Hkv : head - p.Hq);
  const int slot = p.slots[n];
  const int half = p.R >> 1;
  const bool turned = !is_v && j < (p.R >> 4);
  const bool split = turned && !p.interleaved;  // the pieces are half apart
  const int c0 = split ? 8 * j : 16 * j;
  const int c1 = split ? c0 + half : c0 + 8;

  const __half* row = is_q ? p.q + n * p.q_stride : is_v ? p.v + n * p.v_stride : p.k + n * p.k_stride;
  row += (long long)h * p.D;
  float a[8], b[8];
  unpack8(*reinterpret_cast<const uint4*>(row + c0), a);
  unpack8(*reinterpret_cast<const uint4*>(row + c1), b);

  if (p.R > 0) {
    const int pos = p.positions[n];
    if (pos < 0 || (long long)pos >= p.max_pos) {
      if (item == 0 && slot >= 0) flag_or(p.flags, I8KV_FLAG_BAD_POSITION);
      return;
    }
    if (turned) {
      const float4* cs = reinterpret_cast<const float4*>(p.cos_sin + (long long)pos * p.R + 8 * j);
      const float4* sn = reinterpret_cast<const float4*>(p.cos_sin + (long long)pos * p.R + half + 8 * j);
      const float4 q0 = cs[0], q1 = cs[1], r0 = sn[0], r1 = sn[1];
      const float c[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
      const float s[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
      if (split) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(a[i], b[i], c[i], s[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          turn(a[2 * i], a[2 * i + 1], c[i], s[i]);
          turn(b[2 * i], b[2 * i + 1], c[4 + i], s[4 + i]);
        }
      }
    }
  }
  if (is_q) {
    __half* o = p.q_out + (n * p.Hq + h) * p.D;
    *reinterpret_cast<uint4*>(o + c0) = pack8(a);
    *reinterpret_cast<uint4*>(o + c1) = pack8(b);
    return;
  }
  if (slot < 0) return;
  if ((long long)slot >= p.num_slots) {
    if (item == p.Hq * ipr) flag_or(p.flags, I8KV_FLAG_BAD_SLOT);
    return;
  }
  const float* sc = is_v ? p.v_scale : p.k_scale;
  const int step = p.per_channel ? 1 : 0;
  const int ch = p.per_channel ? h * p.D : 0;
  if constexpr (CACHE == I8KV_CACHE_FP16) {
    __half* o = static_cast<__half*>(is_v ? p.v_cache : p.k_cache) +
                ((long long)slot * p.Hkv + h) * p.D;
    *reinterpret_cast<uint4*>(o + c0) = pack8(a);
    *reinterpret_cast<uint4*>(o + c1) = pack8(b);
  } else if constexpr (CACHE == I8KV_CACHE_MX4) {
    float ma = 0.f, mb = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = nan_to_zero(__fmul_rn(a[i], __frcp_rn(sc[ch + (c0 + i) * step])));
      b[i] = nan_to_zero(__fmul_rn(b[i], __frcp_rn(sc[ch + (c1 + i) * step])));
      ma = fmaxf(ma, fabsf(a[i]));
      mb = fmaxf(mb, fabsf(b[i]));
    }
    if (split) {
      // adjacent lanes hold the two halves of a block (same token, same row)
      const int lane = threadIdx.x & 31;
      const unsigned pair = 3u << (lane & ~1);
      ma = fmaxf(ma, __shfl_xor_sync(pair, ma, 1));
      mb = fmaxf(mb, __shfl_xor_sync(pair, mb, 1));
    } else {
      ma = mb = fmaxf(ma, mb);
    }
    const uint32_t sb = e4m3x2_of(__fmul_rn(ma, 1.f / 6.f), __fmul_rn(mb, 1.f / 6.f));
    const float sa = e4m3_value(sb & 0xFFu), sbv = e4m3_value(sb >> 8);
    const float ra = sa > 0.f ? __frcp_rn(sa) : 0.f, rb = sbv > 0.f ? __frcp_rn(sbv) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = sa > 0.f ? __fmul_rn(a[i], ra) : 0.f;
      b[i] = sbv > 0.f ? __fmul_rn(b[i], rb) : 0.f;
    }
    int tok;
    uint8_t* rec = static_cast<uint8_t*>(p.k_cache) +
                   mx4_record(slot, h, p.Hkv, p.D, p.bs, p.bs_shift, tok) + (is_v ? 9 * p.D : 0);
    uint8_t* code = rec + tok * (p.D >> 1);
    *reinterpret_cast<uint32_t*>(code + (c0 >> 1)) = e2m1x8_of(a);
    *reinterpret_cast<uint32_t*>(code + (c1 >> 1)) = e2m1x8_of(b);
    uint8_t* scale = rec + 8 * p.D + tok * ipr;
    // one writer per block: the lane that holds the block's first 8 channels
    if ((c0 & 15) == 0) scale[c0 >> 4] = (uint8_t)sb;
    if (split && (c1 & 15) == 0) scale[c1 >> 4] = (uint8_t)(sb >> 8);
  } else {
    constexpr bool FP8 = CACHE == I8KV_CACHE_FP8;
    uint8_t* o = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                 ((long long)slot * p.Hkv + h) * p.D;
    *reinterpret_cast<uint2*>(o + c0) = codes8<FP8>(a, sc + ch + c0 * step, step);
    *reinterpret_cast<uint2*>(o + c1) = codes8<FP8>(b, sc + ch + c1 * step, step);
  }
}

// One thread: 16 channels of one row, K or V.
template <int CACHE>
__global__ void __launch_bounds__(kAppendThreads)
gather_cache_kernel(const AppendParams p, __half* __restrict__ k_out, __half* __restrict__ v_out) {
  grid_dependency_wait();
  const int ipr = p.D >> 4;
  const int ipt = 2 * p.Hkv * ipr;
  const long long flat = blockIdx.x * (long long)kAppendThreads + threadIdx.x;
  const long long n = flat / ipt;
  if (n >= p.num_tokens) return;
  const int item = (int)(flat - n * ipt);
  const int head = item / ipr, j = item - (item / ipr) * ipr;
  const bool is_v = head >= p.Hkv;
  const int h = is_v ? head - p.Hkv : head;
  __half* out = is_v ? v_out : k_out;
  const int slot = p.slots[n];
  if (item == 0 && (long long)slot >= p.num_slots) flag_or(p.flags, I8KV_FLAG_BAD_SLOT);
  if (out == nullptr) return;
  uint4* o = reinterpret_cast<uint4*>(out + (n * p.Hkv + h) * p.D + 16 * j);
  if (slot < 0 || (long long)slot >= p.num_slots) {
    o[0] = o[1] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  if constexpr (CACHE == I8KV_CACHE_FP16) {
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const __half*>(is_v ? p.v_cache : p.k_cache) +
        ((long long)slot * p.Hkv + h) * p.D + 16 * j);
    o[0] = src[0];
    o[1] = src[1];
  } else {
    const float* sc = is_v ? p.v_scale : p.k_scale;
    const int step = p.per_channel ? 1 : 0;
    sc += p.per_channel ? h * p.D + 16 * j : 0;
    float x[16];
    if constexpr (CACHE == I8KV_CACHE_MX4) {
      int tok;
      const uint8_t* rec = static_cast<const uint8_t*>(p.k_cache) +
                           mx4_record(slot, h, p.Hkv, p.D, p.bs, p.bs_shift, tok) +
                           (is_v ? 9 * p.D : 0);
      const uint2 w = *reinterpret_cast<const uint2*>(rec + tok * (p.D >> 1) + 8 * j);
      const float s = e4m3_value(rec[8 * p.D + tok * ipr + j]);
      uint32_t hv[8];
      e2m1x8_to_h2x4(w.x, hv[0], hv[1], hv[2], hv[3]);
      e2m1x8_to_h2x4(w.y, hv[4], hv[5], hv[6], hv[7]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hv[i]));
        x[2 * i] = __fmul_rn(f.x, s);  // exact: 6 significant bits
        x[2 * i + 1] = __fmul_rn(f.y, s);
      }
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(
          static_cast<const uint8_t*>(is_v ? p.v_cache : p.k_cache) +
          ((long long)slot * p.Hkv + h) * p.D + 16 * j);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        if constexpr (CACHE == I8KV_CACHE_FP8) {
          e4m3x4_to_h2x2(ww[i], lo, hi);
        } else {
          const uint32_t f = flip_i8x4(ww[i]);
          lo = i8x2_to_h2(f, 0x4140u);
          hi = i8x2_to_h2(f, 0x4342u);
        }
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        x[4 * i] = f0.x;
        x[4 * i + 1] = f0.y;
        x[4 * i + 2] = f1.x;
        x[4 * i + 3] = f1.y;
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], sc[i * step]);
    o[0] = make_uint4(pack_h2(x[0], x[1]), pack_h2(x[2], x[3]), pack_h2(x[4], x[5]),
                      pack_h2(x[6], x[7]));
    o[1] = make_uint4(pack_h2(x[8], x[9]), pack_h2(x[10], x[11]), pack_h2(x[12], x[13]),
                      pack_h2(x[14], x[15]));
  }
}

cudaLaunchConfig_t config_of(long long threads, cudaLaunchAttribute* attr, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((threads + kAppendThreads - 1) / kAppendThreads));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

cudaError_t launch_rope_and_cache(const AppendParams& p, int cache_dtype, cudaStream_t stream) {
  const long long threads = (long long)p.num_tokens * (p.Hq + 2 * p.Hkv) * (p.D / 16);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config_of(threads, &attr, stream);
  switch (cache_dtype) {
    case I8KV_CACHE_INT8: return cudaLaunchKernelEx(&cfg, rope_and_cache_kernel<I8KV_CACHE_INT8>, p);
    case I8KV_CACHE_FP16: return cudaLaunchKernelEx(&cfg, rope_and_cache_kernel<I8KV_CACHE_FP16>, p);
    case I8KV_CACHE_FP8: return cudaLaunchKernelEx(&cfg, rope_and_cache_kernel<I8KV_CACHE_FP8>, p);
    case I8KV_CACHE_MX4: return cudaLaunchKernelEx(&cfg, rope_and_cache_kernel<I8KV_CACHE_MX4>, p);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_gather_cache(const AppendParams& p, int cache_dtype, void* k_out, void* v_out,
                                cudaStream_t stream) {
  const long long threads = (long long)p.num_tokens * 2 * p.Hkv * (p.D / 16);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config_of(threads, &attr, stream);
  __half* k = static_cast<__half*>(k_out);
  __half* v = static_cast<__half*>(v_out);
  switch (cache_dtype) {
    case I8KV_CACHE_INT8: return cudaLaunchKernelEx(&cfg, gather_cache_kernel<I8KV_CACHE_INT8>, p, k, v);
    case I8KV_CACHE_FP16: return cudaLaunchKernelEx(&cfg, gather_cache_kernel<I8KV_CACHE_FP16>, p, k, v);
    case I8KV_CACHE_FP8: return cudaLaunchKernelEx(&cfg, gather_cache_kernel<I8KV_CACHE_FP8>, p, k, v);
    case I8KV_CACHE_MX4: return cudaLaunchKernelEx(&cfg, gather_cache_kernel<I8KV_CACHE_MX4>, p, k, v);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace i8kv
