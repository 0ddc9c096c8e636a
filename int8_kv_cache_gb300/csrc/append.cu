// Append of new rows to a paged cache with the position rotation applied on the
// way (rope_and_cache), the same with the heads of queries and keys normed first
// (norm_rope_and_cache), and the read-back of cache rows as fp16 (gather_cache).
//
// Rotation of a pair (a, b) of channels by the angle of its position:
//   a' = a cos - b sin,  b' = b cos + a sin
// in fp32, every product and sum rounded on its own, so that the stored codes of heads
// that are not normed follow from the formula bit for bit.  Queries leave as fp16; keys and values
// are stored in the cache's type:
//   int8, e4m3fn  the codes of the IEEE quotient x / scale (as the plain
//                 quantize-on-write stores them)
//   fp16          x rounded once
//   MX4           y = x fl(1/scale); block scale s = e4m3(min(max|y| fl(1/6), 448)),
//                 code = e2m1(y fl(1/s))
//
// The norm of a head: y = x r w with r = 1 / sqrt(mean x^2 + eps) in fp32, the root by rsqrtf (within 2
// units of the last place); the squares of a thread's 16 channels are summed in two chains of fused products,
// the even channels and the odd ones, which are added, then over the D / 16 lanes that hold the head by halves.
//
// Bound: HBM, rows in and rows out once each.  A thread keeps one item -- 16 channels
// of a head as two pieces of 8, so that every access is 16 bytes and neighbouring
// lanes touch neighbouring pieces -- and walks the tokens, so that the reciprocals of
// its 16 scales are formed once and no index is divided in the loop.  In a turned
// range of R channels with the halves rotated together the pieces are channels 8j ..
// 8j + 7 and their partners R / 2 further on; every other range is cut the same way.
// Queries take several heads of a token per thread (they share the sines and
// cosines: 64 of the 192 bytes that a head would load).  An MX4 block of 16 channels is
// one piece of each of two neighbouring lanes, which exchange their maxima.
// Measured on one GB300 (graph of calls): 32768 tokens, 32/8 heads, head_dim 128, all of it
// turned, into MX4: 119 us for 726 MB, 6.1 TB/s, 90 % of the measured copy rate; 16 tokens 2.6 us.
// Keys and values alone are short of the rate (8 heads, MX4: 59 us for 189 MB): what they wait
// for are sines and cosines, at 16 warps per SM; 24 of fewer registers and one token each
// measured no faster (62), nor sines and cosines a step ahead (60).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

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

// Codes of 8 channels for an int8 or e4m3fn cache from the fp32 quotients
// themselves: s the scales of the channels.
template <bool FP8>
__device__ __noinline__ uint2 codes8_exact(float4 lo, float4 hi, const float* __restrict__ s,
                                           int s_step) {
  const float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
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

// max(a, |b|), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// The same codes from the products with the rounded reciprocals r, which are within
// |q| 2^-22 of the rounded quotients: where a product is nearer to a rounding boundary
// than that allows (about one piece in a thousand), or a NaN, the quotients decide.
// (A scale below 2^-128 has no finite reciprocal, and a NaN stands for it.)
template <bool FP8>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], const float (&r)[8],
                                        const float* __restrict__ s, int s_step) {
  uint32_t w[2] = {0u, 0u};
  bool near;
  if constexpr (FP8) {
    // both ends of the product's error interval must have the same code
    float top = 0.f;
    uint32_t differ = 0u;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float q0 = x[j] * r[j], q1 = x[j + 1] * r[j + 1];
      const uint32_t b = e4m3x2_of(q0 * kLoBound, q1 * kLoBound);
      differ |= b ^ e4m3x2_of(q0 * kHiBound, q1 * kHiBound);
      top = max_nan(max_nan(top, q0), q1);
      w[j / 4] |= b << (8 * (j % 4));
    }
    near = differ != 0u || top != top;
  } else {
    // rounding by adding 1.5 * 2^23: the code is the low byte of the sum.  |q| <= 127 here, so
    // a boundary (a half-integer) is nearer than |q| 2^-21 only if |q - code| > 1/2 - 2^-14
    constexpr float kMagic = 12582912.f;
    float far = 0.f;
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float q;
      asm("{\n .reg .f32 t;\n max.NaN.f32 t, %1, 0fC2FE0000;\n min.NaN.f32 %0, t, 0f42FE0000;\n}\n"
          : "=f"(q)
          : "f"(x[j] * r[j]));  // clamped to +-127
      const float t = __fadd_rn(q, kMagic);
      m[j] = __float_as_uint(t);
      far = max_nan(far, __fsub_rn(q, __fsub_rn(t, kMagic)));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = prmt(prmt(m[4 * i], m[4 * i + 1], 0x0040u), prmt(m[4 * i + 2], m[4 * i + 3], 0x0040u), 0x5410u);
    near = !(far <= 0.5f - 0x1p-14f);
  }
  if (near)
    return codes8_exact<FP8>(make_float4(x[0], x[1], x[2], x[3]),
                             make_float4(x[4], x[5], x[6], x[7]), s, s_step);
  return make_uint2(w[0], w[1]);
}

// The two pieces of item j of a row: channels c0 .. c0 + 7 and c1 .. c1 + 7, and whether
// they are turned.
struct Pieces {
  int c0, c1;
  bool turned;
  bool block;  // the two pieces are one MX4 block (else a piece is half of one)
};
__device__ __forceinline__ Pieces pieces_of(const AppendParams& p, int j, bool rotates) {
  Pieces x;
  const int R = rotates ? p.R : 0;
  x.turned = j < (R >> 4);
  const int first = x.turned ? 0 : R, len = x.turned ? R : p.D - R;
  const int i = x.turned ? j : j - (R >> 4);
  // (an interleaved range that is no multiple of 32 keeps its pieces next to each other,
  // so that an MX4 block never straddles two items' lanes unevenly)
  x.block = (p.R & 31) != 0 && p.interleaved;
  x.c0 = first + (x.block ? 16 : 8) * i;
  x.c1 = x.block ? x.c0 + 8 : x.c0 + (len >> 1);
  return x;
}

// Sines and cosines of an item at one position.
struct Angles {
  float4 c[2], s[2];
};
__device__ __forceinline__ Angles angles_of(const AppendParams& p, const Pieces& x, int pos) {
  const float* row = p.cos_sin + (long long)pos * p.R;
  const int half = p.R >> 1;
  // halves: pairs c0 .. c0 + 7; interleaved: pairs c0 / 2 .. + 3 and c1 / 2 .. + 3
  const int t0 = p.interleaved ? x.c0 >> 1 : x.c0, t1 = p.interleaved ? x.c1 >> 1 : x.c0 + 4;
  Angles a;
  a.c[0] = __ldg(reinterpret_cast<const float4*>(row + t0));
  a.c[1] = __ldg(reinterpret_cast<const float4*>(row + t1));
  a.s[0] = __ldg(reinterpret_cast<const float4*>(row + half + t0));
  a.s[1] = __ldg(reinterpret_cast<const float4*>(row + half + t1));
  return a;
}
__device__ __forceinline__ void turn_item(float (&a)[8], float (&b)[8], const Angles& g,
                                          bool interleaved) {
  const float c[8] = {g.c[0].x, g.c[0].y, g.c[0].z, g.c[0].w, g.c[1].x, g.c[1].y, g.c[1].z, g.c[1].w};
  const float s[8] = {g.s[0].x, g.s[0].y, g.s[0].z, g.s[0].w, g.s[1].x, g.s[1].y, g.s[1].z, g.s[1].w};
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn(a[2 * i], a[2 * i + 1], c[i], s[i]);
      turn(b[2 * i], b[2 * i + 1], c[4 + i], s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(a[i], b[i], c[i], s[i]);
  }
}

// Two fp32 operations in one instruction, each rounded by itself.
__device__ __forceinline__ uint64_t two(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ void from_two(uint64_t d, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(x), "=f"(y) : "l"(d));
}
__device__ __forceinline__ uint64_t mul_two(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma_two(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_two(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// turn_item of halves two channels at a time, with the same roundings (a difference is a fused sum with
// -1 times what is taken off).
__device__ __forceinline__ void turn_halves(float (&a)[8], float (&b)[8], const Angles& g) {
  const uint64_t c[4] = {two(g.c[0].x, g.c[0].y), two(g.c[0].z, g.c[0].w), two(g.c[1].x, g.c[1].y), two(g.c[1].z, g.c[1].w)};
  const uint64_t s[4] = {two(g.s[0].x, g.s[0].y), two(g.s[0].z, g.s[0].w), two(g.s[1].x, g.s[1].y), two(g.s[1].z, g.s[1].w)};
  const uint64_t minus = two(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t x = two(a[2 * i], a[2 * i + 1]), y = two(b[2 * i], b[2 * i + 1]);
    from_two(fma_two(mul_two(y, s[i]), minus, mul_two(x, c[i])), a[2 * i], a[2 * i + 1]);
    from_two(add_two(mul_two(y, c[i]), mul_two(x, s[i])), b[2 * i], b[2 * i + 1]);
  }
}

// The norms of N heads, each of which the aligned `ipr` lanes of the warp (a power of two) hold, 16
// channels each, as fp16: r = 1 / sqrt(mean + eps).  All of those lanes are here together: they work
// on the same tokens.  The heads side by side: one after the other, each waits for its sum through the
// lanes, and rsqrtf, which is within 2 units of the last place, for the correctly rounded root, which
// takes some 30 instructions (16384 tokens, 32/8 heads, head_dim 128, half of it turned: 105 us one by
// one; side by side 83 into MX4 and 94 into int8; with rsqrtf 78 and 81; not normed 61 and 63).
template <int N>
__device__ __forceinline__ void norms_of(const uint4 (&a)[N], const uint4 (&b)[N], int ipr, float eps, float (&r)[N]) {
  const int lane = threadIdx.x & 31;
  const unsigned of_head = ((1u << ipr) - 1u) << (lane & ~(ipr - 1));
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float x[8], y[8];
    unpack8(a[i], x);
    unpack8(b[i], y);
    uint64_t sum = 0;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint64_t u = two(x[e], x[e + 1]), v = two(y[e], y[e + 1]);
      sum = fma_two(u, u, sum);
      sum = fma_two(v, v, sum);
    }
    float lo, hi;
    from_two(sum, lo, hi);
    r[i] = lo + hi;
  }
  for (int o = ipr >> 1; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] += __shfl_xor_sync(of_head, r[i], o);
  }
  const float each = 0.0625f / (float)ipr;
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = rsqrtf(fmaf(r[i], each, eps));
}
__device__ __forceinline__ void norm_item(float (&a)[8], float (&b)[8], const float (&wa)[8],
                                          const float (&wb)[8], float r) {
  const uint64_t rr = two(r, r);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    from_two(mul_two(mul_two(two(a[i], a[i + 1]), rr), two(wa[i], wa[i + 1])), a[i], a[i + 1]);
    from_two(mul_two(mul_two(two(b[i], b[i + 1]), rr), two(wb[i], wb[i + 1])), b[i], b[i + 1]);
  }
}
__device__ __forceinline__ void weights8(const float* w, int at, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w + at));
  const float4 b = __ldg(reinterpret_cast<const float4*>(w + at) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// One row's item into the cache.  r0, r1: reciprocals of the scales of the two pieces;
// inv_scale (MX4): the rounded reciprocals of the 127 block scales, by their byte.
template <int CACHE>
__device__ __forceinline__ void store_item(const AppendParams& p, const Pieces& x, int h, bool is_v,
                                           int slot, float (&a)[8], float (&b)[8],
                                           const float (&r0)[8], const float (&r1)[8],
                                           const float* sc, int step, const float* inv_scale) {
  if constexpr (CACHE == I8KV_CACHE_FP16) {
    __half* o = static_cast<__half*>(is_v ? p.v_cache : p.k_cache) +
                ((long long)slot * p.Hkv + h) * p.D;
    *reinterpret_cast<uint4*>(o + x.c0) = pack8(a);
    *reinterpret_cast<uint4*>(o + x.c1) = pack8(b);
  } else if constexpr (CACHE == I8KV_CACHE_MX4) {
    float ma = 0.f, mb = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = __fmul_rn(a[i], r0[i]);
      b[i] = __fmul_rn(b[i], r1[i]);
      ma = max_nan(ma, a[i]);
      mb = max_nan(mb, b[i]);
    }
    if (ma != ma || mb != mb) {  // a NaN counts as a zero
      ma = mb = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = nan_to_zero(a[i]);
        b[i] = nan_to_zero(b[i]);
        ma = fmaxf(ma, fabsf(a[i]));
        mb = fmaxf(mb, fabsf(b[i]));
      }
    }
    const int lane = threadIdx.x & 31;
    if (x.block) {
      ma = mb = fmaxf(ma, mb);
    } else {
      // neighbouring lanes hold the two halves of each block (same token, same row)
      const unsigned pair = 3u << (lane & ~1);
      ma = fmaxf(ma, __shfl_xor_sync(pair, ma, 1));
      mb = fmaxf(mb, __shfl_xor_sync(pair, mb, 1));
    }
    const uint32_t sb = e4m3x2_of(__fmul_rn(ma, 1.f / 6.f), __fmul_rn(mb, 1.f / 6.f));
    const float ra = inv_scale[sb & 0x7Fu], rb = inv_scale[(sb >> 8) & 0x7Fu];  // 0 of a zero
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = __fmul_rn(a[i], ra);
      b[i] = __fmul_rn(b[i], rb);
    }
    int tok;
    uint8_t* rec = static_cast<uint8_t*>(p.k_cache) +
                   mx4_record(slot, h, p.Hkv, p.D, p.bs, p.bs_shift, tok) + (is_v ? 9 * p.D : 0);
    uint8_t* code = rec + tok * (p.D >> 1);
    // (a zero scale stores zeros, not the signs of what vanished)
    *reinterpret_cast<uint32_t*>(code + (x.c0 >> 1)) = ra != 0.f ? e2m1x8_of(a) : 0u;
    *reinterpret_cast<uint32_t*>(code + (x.c1 >> 1)) = rb != 0.f ? e2m1x8_of(b) : 0u;
    uint8_t* scale = rec + 8 * p.D + tok * (p.D >> 4);
    // one writer per block: the lane that holds its first 8 channels
    if ((x.c0 & 15) == 0) {
      scale[x.c0 >> 4] = (uint8_t)sb;
      if (!x.block) scale[x.c1 >> 4] = (uint8_t)(sb >> 8);
    }
  } else {
    constexpr bool FP8 = CACHE == I8KV_CACHE_FP8;
    uint8_t* o = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                 ((long long)slot * p.Hkv + h) * p.D;
    *reinterpret_cast<uint2*>(o + x.c0) = codes8<FP8>(a, r0, sc + x.c0 * step, step);
    *reinterpret_cast<uint2*>(o + x.c1) = codes8<FP8>(b, r1, sc + x.c1 * step, step);
  }
}

// The scales of 8 channels from channel `at` of s (or the one scale, eight times).
template <int CACHE>
__device__ __forceinline__ void scales8(const AppendParams& p, const float* s, int at, float (&sc)[8]) {
  if constexpr (CACHE != I8KV_CACHE_FP16) {
    if (p.per_channel) {
      const float4 a = *reinterpret_cast<const float4*>(s + at);
      const float4 b = *reinterpret_cast<const float4*>(s + at + 4);
      sc[0] = a.x, sc[1] = a.y, sc[2] = a.z, sc[3] = a.w;
      sc[4] = b.x, sc[5] = b.y, sc[6] = b.z, sc[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) sc[i] = s[0];
    }
  }
}

// 1 / s as the codes take it: MX4's are defined by the rounded reciprocal, the others by the quotient,
// of which an infinite reciprocal says nothing.
template <int CACHE>
__device__ __forceinline__ float reciprocal(float s) {
  const float r = __frcp_rn(s);
  return CACHE != I8KV_CACHE_MX4 && isinf(r) ? __int_as_float(0x7fc00000) : r;
}

__host__ __device__ __forceinline__ long long warps_of(long long threads) { return (threads + 31) / 32; }
// floor(w part / all)
__device__ __forceinline__ unsigned share_of(unsigned w, unsigned part, unsigned all) {
  return all < 65536u ? w * part / all : (unsigned)((unsigned long long)w * part / all);
}

__device__ __forceinline__ void copy16(uint4* to, const __half* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
               "l"(from)
               : "memory");
}

// HQ: query heads per thread (1: a few tokens, where threads are short; else 4).
// NORM: queries and keys normed first where their weights are given, keys written out where asked.
template <int CACHE, int HQ, bool NORM>
__global__ void __launch_bounds__(kAppendThreads, 2)
rope_and_cache_kernel(const AppendParams p, long long q_lanes, long long kv_lanes) {
  __shared__ float inv_scale[CACHE == I8KV_CACHE_MX4 ? 128 : 1];
  if constexpr (CACHE == I8KV_CACHE_MX4) {
    if (threadIdx.x < 128) inv_scale[threadIdx.x] = threadIdx.x ? __frcp_rn(e4m3_value(threadIdx.x)) : 0.f;
    __syncthreads();
  }
  __shared__ uint4 ring[CACHE == I8KV_CACHE_FP16 ? 1 : 2][2][2][kAppendThreads];
  grid_dependency_wait();
  const int ipr = p.D >> 4;  // items per row
  // Warps for queries and warps for keys and values (their loops differ, so none does both),
  // spread evenly over the grid: as many as `q_lanes` and `kv_lanes` tokens at a time take.
  // (27242 tokens, 10/2 heads, into MX4: 38 us against 56 with both in a warp.)
  const unsigned q_items = (p.Hq + HQ - 1) / HQ * ipr, kv_items = 2 * p.Hkv * ipr;  // of a token
  const unsigned q_warps = warps_of(q_lanes * q_items), warps = q_warps + warps_of(kv_lanes * kv_items);
  const unsigned w = blockIdx.x * (kAppendThreads / 32) + threadIdx.x / 32;
  const unsigned before = share_of(w, q_warps, warps);  // warps for queries among those before
  const bool queries = share_of(w + 1, q_warps, warps) != before;
  const unsigned flat = (queries ? before : w - before) * 32 + (threadIdx.x & 31);
  const unsigned items = queries ? q_items : kv_items;
  if (w >= warps) return;
  const long long lanes = queries ? q_lanes : kv_lanes;
  const unsigned n0 = flat / items;
  if (n0 >= (unsigned)lanes) return;
  const int item = flat - n0 * items;
  const int unit = item / ipr, j = item - (item / ipr) * ipr;
  const bool il = p.interleaved != 0;

  if (queries) {  // HQ heads of a token
    const Pieces x = pieces_of(p, j, true);
    const int h0 = unit * HQ;
    float w0[8], w1[8];
    const bool normed = NORM && p.q_weight != nullptr;
    if constexpr (NORM) {
      if (normed) {
        weights8(p.q_weight, x.c0, w0);
        weights8(p.q_weight, x.c1, w1);
      }
    }
    int next = p.R > 0 ? __ldg(p.positions + n0) : 0;  // a position ahead of its angles
    for (long long n = n0; n < p.num_tokens; n += lanes) {
      const int pos = next;
      if (p.R > 0 && n + lanes < p.num_tokens) next = __ldg(p.positions + n + lanes);
      const __half* row = p.q + n * p.q_stride + (long long)h0 * p.D;
      uint4 ra[HQ], rb[HQ];
#pragma unroll
      for (int i = 0; i < HQ; ++i) {
        if (NORM) ra[i] = rb[i] = make_uint4(0u, 0u, 0u, 0u);
        if (h0 + i < p.Hq) {
          ra[i] = *reinterpret_cast<const uint4*>(row + i * p.D + x.c0);
          rb[i] = *reinterpret_cast<const uint4*>(row + i * p.D + x.c1);
        }
      }
      Angles g;
      if (p.R > 0) {
        if (pos < 0 || (long long)pos >= p.max_pos) continue;
        if (x.turned) g = angles_of(p, x, pos);
      }
      __half* out = p.q_out + (n * p.Hq + h0) * p.D;
      float r[HQ];
      if constexpr (NORM) {
        if (normed) norms_of(ra, rb, ipr, p.eps, r);
      }
#pragma unroll
      for (int i = 0; i < HQ; ++i)
        if (h0 + i < p.Hq) {
          if (x.turned || normed) {
            float a[8], b[8];
            unpack8(ra[i], a);
            unpack8(rb[i], b);
            if constexpr (NORM) {
              if (normed) norm_item(a, b, w0, w1, r[i]);
            }
            if (NORM && x.turned && !il) turn_halves(a, b, g);
            else if (!NORM || x.turned) turn_item(a, b, g, il);
            ra[i] = pack8(a);
            rb[i] = pack8(b);
          }
          *reinterpret_cast<uint4*>(out + i * p.D + x.c0) = ra[i];
          *reinterpret_cast<uint4*>(out + i * p.D + x.c1) = rb[i];
        }
    }
    return;
  }

  // Keys and values: two tokens at a time, their slots and positions a step ahead, and so are their
  // rows, in shared memory, on the way to codes (32768 tokens, 8 heads, MX4, not turned: 44 us against
  // 57, turned 59 against 62; fp16 rows are stored at once and gain nothing: 128 us against 132 with
  // 32/8 heads).
  const int kv = unit;
  const bool is_v = kv >= p.Hkv;
  const int h = is_v ? kv - p.Hkv : kv;
  const Pieces x = pieces_of(p, j, !is_v);
  const float* sc = is_v ? p.v_scale : p.k_scale;
  const int step = p.per_channel ? 1 : 0;
  if (p.per_channel) sc += h * p.D;
  float r0[8], r1[8];
  if constexpr (CACHE != I8KV_CACHE_FP16) {
    scales8<CACHE>(p, sc, x.c0, r0);
    scales8<CACHE>(p, sc, x.c1, r1);
    if (p.per_channel) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r0[i] = reciprocal<CACHE>(r0[i]);
        r1[i] = reciprocal<CACHE>(r1[i]);
      }
    } else {
      const float r = reciprocal<CACHE>(r0[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) r0[i] = r1[i] = r;
    }
  }
  float w0[8], w1[8];
  const bool normed = NORM && !is_v && p.k_weight != nullptr;
  const bool keys_out = NORM && !is_v && p.k_out != nullptr;
  if constexpr (NORM) {
    if (normed) {
      weights8(p.k_weight, x.c0, w0);
      weights8(p.k_weight, x.c1, w1);
    }
  }
  const __half* src = (is_v ? p.v : p.k) + (long long)h * p.D;
  const long long stride = is_v ? p.v_stride : p.k_stride;
  constexpr int N = 2;
  int slot[N], pos[N];  // of the next tokens
  auto look = [&](long long n) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const long long m = n + i * lanes;
      slot[i] = -1;
      pos[i] = 0;
      if (m < p.num_tokens) {
        slot[i] = __ldg(p.slots + m);
        if (p.R > 0) pos[i] = __ldg(p.positions + m);
      }
    }
  };
  constexpr bool RING = CACHE != I8KV_CACHE_FP16;
  auto fetch = [&](long long n, int st) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const long long m = n + i * lanes;
      if (m < p.num_tokens) {
        copy16(&ring[st][i][0][threadIdx.x], src + m * stride + x.c0);
        copy16(&ring[st][i][1][threadIdx.x], src + m * stride + x.c1);
      }
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  if constexpr (RING) fetch(n0, 0);
  look(n0);
  int st = 0;
  for (long long n = n0; n < p.num_tokens; n += N * lanes, st ^= 1) {
    uint4 raw[N][2] = {};
    if constexpr (RING) {
      fetch(n + N * lanes, st ^ 1);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const long long m = n + i * lanes;
        if (m < p.num_tokens) {
          raw[i][0] = *reinterpret_cast<const uint4*>(src + m * stride + x.c0);
          raw[i][1] = *reinterpret_cast<const uint4*>(src + m * stride + x.c1);
        }
      }
    }
    Angles g[N];
    int at[N];
    bool out[N];  // NORM: the token's keys are written out
#pragma unroll
    for (int i = 0; i < N; ++i) {
      at[i] = slot[i];
      out[i] = keys_out && n + i * lanes < p.num_tokens;
      if (p.R > 0 && (pos[i] < 0 || (long long)pos[i] >= p.max_pos)) {
        // (one key item reports it)
        if (kv == 0 && j == 0 && slot[i] >= 0) flag_or(p.flags, I8KV_FLAG_BAD_POSITION);
        at[i] = -1;
        out[i] = false;
      } else if ((long long)slot[i] >= p.num_slots) {
        if (kv == 0 && j == 0) flag_or(p.flags, I8KV_FLAG_BAD_SLOT);
        at[i] = -1;
      }
      if ((at[i] >= 0 || out[i]) && x.turned) g[i] = angles_of(p, x, pos[i]);
    }
    look(n + N * lanes);
    if constexpr (RING) asm volatile("cp.async.wait_group 1;\n" ::: "memory");
    float r[N];
    if constexpr (NORM) {
      if (normed) {  // (of a token that is left out too, whatever its place holds)
        uint4 ra[N], rb[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          ra[i] = RING ? ring[st][i][0][threadIdx.x] : raw[i][0];
          rb[i] = RING ? ring[st][i][1][threadIdx.x] : raw[i][1];
        }
        norms_of(ra, rb, ipr, p.eps, r);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (at[i] < 0 && !out[i]) continue;
      float a[8], b[8];
      unpack8(RING ? ring[st][i][0][threadIdx.x] : raw[i][0], a);
      unpack8(RING ? ring[st][i][1][threadIdx.x] : raw[i][1], b);
      if constexpr (NORM) {
        if (normed) norm_item(a, b, w0, w1, r[i]);
      }
      if (NORM && x.turned && !il) turn_halves(a, b, g[i]);
      else if (x.turned) turn_item(a, b, g[i], il);
      if constexpr (NORM) {
        if (out[i]) {
          __half* o = p.k_out + ((n + i * lanes) * p.Hkv + h) * p.D;
          *reinterpret_cast<uint4*>(o + x.c0) = pack8(a);
          *reinterpret_cast<uint4*>(o + x.c1) = pack8(b);
        }
        if (at[i] < 0) continue;
      }
      store_item<CACHE>(p, x, h, is_v, at[i], a, b, r0, r1, sc, step, inv_scale);
    }
  }
}

// Read-back: a thread keeps 8 channels of a head, for keys and values alike (one slot,
// one address, two rows), with their scales, and walks the rows a few at a time: the
// slots of the next ones are on their way while these are converted; 16-byte stores.
// Bound: HBM writes.  16384 MX4 rows of 8 heads, head_dim 128: 19.0 us for 19 MB read and
// 67 MB written (a plain fill of 67 MB: 17.1 us); 1 or 4 rows at a time 19.6 and 28 us.
constexpr int kGatherRows = 2;

// fp16 values of 8 channels: codes raw, block scale byte bs, scales sc.
template <int CACHE>
__device__ __forceinline__ uint4 values8(uint4 raw, uint32_t bs, const float (&sc)[8]) {
  if constexpr (CACHE == I8KV_CACHE_FP16) {
    return raw;
  } else {
    uint32_t hv[4];
    if constexpr (CACHE == I8KV_CACHE_MX4) {
      e2m1x8_to_h2x4(raw.x, hv[0], hv[1], hv[2], hv[3]);
      uint32_t s2, unused;
      e4m3x4_to_h2x2(bs * 0x0101u, s2, unused);
#pragma unroll
      for (int k = 0; k < 4; ++k)  // exact: 6 significant bits
        asm("mul.f16x2 %0, %0, %1;\n" : "+r"(hv[k]) : "r"(s2));
    } else if constexpr (CACHE == I8KV_CACHE_FP8) {
      e4m3x4_to_h2x2(raw.x, hv[0], hv[1]);
      e4m3x4_to_h2x2(raw.y, hv[2], hv[3]);
    } else {
      const uint32_t f0 = flip_i8x4(raw.x), f1 = flip_i8x4(raw.y);
      hv[0] = i8x2_to_h2(f0, 0x4140u);
      hv[1] = i8x2_to_h2(f0, 0x4342u);
      hv[2] = i8x2_to_h2(f1, 0x4140u);
      hv[3] = i8x2_to_h2(f1, 0x4342u);
    }
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hv[k]));
      o[k] = pack_h2(__fmul_rn(f.x, sc[2 * k]), __fmul_rn(f.y, sc[2 * k + 1]));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int CACHE>
__global__ void __launch_bounds__(kAppendThreads)
gather_cache_kernel(const AppendParams p, __half* __restrict__ k_out, __half* __restrict__ v_out,
                    int lanes) {
  constexpr bool MX = CACHE == I8KV_CACHE_MX4;
  constexpr int N = kGatherRows;
  grid_dependency_wait();
  const unsigned ipr = p.D >> 3;
  const unsigned ipt = p.Hkv * ipr;
  const unsigned flat = blockIdx.x * kAppendThreads + threadIdx.x;
  const unsigned n0 = flat / ipt;
  if (n0 >= (unsigned)lanes) return;
  const unsigned item = flat - n0 * ipt;
  const int h = item / ipr, c = 8 * (item - h * ipr);
  const int at = h * p.D + c;  // in a row of the outputs (and of a plain cache)
  const long long row = (long long)p.Hkv * p.D;
  float ks[8], vs[8];
  scales8<CACHE>(p, p.k_scale, at, ks);
  scales8<CACHE>(p, p.v_scale, at, vs);
  auto slot_of = [&](long long m) -> int {
    if (m >= p.num_tokens) return -1;
    const int s = __ldg(p.slots + m);
    if ((long long)s < p.num_slots) return s;
    if (item == 0) flag_or(p.flags, I8KV_FLAG_BAD_SLOT);
    return -1;
  };
  int next[N];
#pragma unroll
  for (int i = 0; i < N; ++i) next[i] = slot_of(n0 + (long long)i * lanes);
  for (long long n = n0; n < p.num_tokens; n += (long long)N * lanes) {
    uint4 rk[N], rv[N];
    uint32_t bk[N], bv[N];
    bool some[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      rk[i] = rv[i] = make_uint4(0u, 0u, 0u, 0u);
      bk[i] = bv[i] = 0u;
      some[i] = next[i] >= 0;
      if (!some[i]) continue;
      if constexpr (MX) {
        int tok;
        const uint8_t* rec = static_cast<const uint8_t*>(p.k_cache) +
                             mx4_record(next[i], h, p.Hkv, p.D, p.bs, p.bs_shift, tok);
        const uint8_t* code = rec + tok * (p.D >> 1) + (c >> 1);
        const uint8_t* scale = rec + 8 * p.D + tok * (p.D >> 4) + (c >> 4);
        rk[i].x = *reinterpret_cast<const uint32_t*>(code);
        rv[i].x = *reinterpret_cast<const uint32_t*>(code + 9 * p.D);
        bk[i] = scale[0];
        bv[i] = scale[9 * p.D];
      } else {
        const long long o = next[i] * row + at;
        if constexpr (CACHE == I8KV_CACHE_FP16) {
          rk[i] = *reinterpret_cast<const uint4*>(static_cast<const __half*>(p.k_cache) + o);
          rv[i] = *reinterpret_cast<const uint4*>(static_cast<const __half*>(p.v_cache) + o);
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.k_cache) + o);
          const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.v_cache) + o);
          rk[i].x = a.x, rk[i].y = a.y;
          rv[i].x = b.x, rv[i].y = b.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) next[i] = slot_of(n + (long long)(N + i) * lanes);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const long long m = n + (long long)i * lanes;
      if (m >= p.num_tokens) break;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      if (k_out != nullptr)
        *reinterpret_cast<uint4*>(k_out + m * row + at) = some[i] ? values8<CACHE>(rk[i], bk[i], ks) : zero;
      if (v_out != nullptr)
        *reinterpret_cast<uint4*>(v_out + m * row + at) = some[i] ? values8<CACHE>(rv[i], bv[i], vs) : zero;
    }
  }
}

// Token lanes of a grid: about `ctas` CTAs of threads, at most one lane per token.
long long lanes_of(long long tokens, long long per_token, long long ctas) {
  long long lanes = ctas * kAppendThreads / per_token;
  if (lanes < 1) lanes = 1;
  return lanes < tokens ? lanes : tokens;
}

cudaError_t sm_count(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
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

namespace {

// Tokens of keys and values at a time for one of queries, so that their warps end together (the
// former do two a pass; 32768 tokens, 32/8 heads, head_dim 128, at 0.5 / 0.6 / 0.7 / 0.8: MX4 124 / 118 /
// 121 / 126 us, int8 129 / 122 / 125 / 129, e4m3fn 118 / 120 / 124 / 129, fp16 128 / 130 / 132 / 136;
// 4646 tokens, 128/8, 256, int8: 116 / 106 / 104 / 102).
// With norms, of which queries have more, 0.5 (16384 tokens, 32/8, 128 at 0.4 / 0.5 / 0.55 / 0.65: MX4 91 / 84.5 /
// 88 / 93 us, int8 96 / 90.5 / 95.5 / 97.5).
template <int CACHE, bool NORM>
constexpr double kKvShare = NORM || CACHE == I8KV_CACHE_FP16 ? 0.5 : 0.65;

template <int CACHE, int HQ, bool NORM>
cudaError_t append_with(const AppendParams& p, int sms, cudaStream_t stream) {
  const long long q_items = (p.Hq + HQ - 1LL) / HQ * (p.D / 16), kv_items = 2LL * p.Hkv * (p.D / 16);
  const double per = 2. * sms * kAppendThreads / (q_items + kKvShare<CACHE, NORM> * kv_items);  // the resident CTAs
  const long long q_lanes = std::clamp<long long>((long long)per, 1, p.num_tokens);
  const long long kv_lanes = std::clamp<long long>((long long)(kKvShare<CACHE, NORM> * per), 1, p.num_tokens);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      config_of(32 * (warps_of(q_lanes * q_items) + warps_of(kv_lanes * kv_items)), &attr, stream);
  return cudaLaunchKernelEx(&cfg, rope_and_cache_kernel<CACHE, HQ, NORM>, p, q_lanes, kv_lanes);
}

// Four query heads per thread where one head each would fill the GPU more than once
// over (64 of 192 bytes saved per head); one head each spreads fewer tokens wider.
template <int CACHE, bool NORM>
cudaError_t append_of(const AppendParams& p, cudaStream_t stream) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const long long items = (long long)p.num_tokens * (p.Hq + 2 * p.Hkv) * (p.D / 16);
  return items > 4LL * sms * kAppendThreads ? append_with<CACHE, 4, NORM>(p, sms, stream)
                                            : append_with<CACHE, 1, NORM>(p, sms, stream);
}

template <int CACHE>
cudaError_t gather_of(const AppendParams& p, void* k_out, void* v_out, cudaStream_t stream) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const long long ipt = (long long)p.Hkv * (p.D / 8);
  const long long lanes = lanes_of(p.num_tokens, ipt, 4LL * sms);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config_of(lanes * ipt, &attr, stream);
  return cudaLaunchKernelEx(&cfg, gather_cache_kernel<CACHE>, p, static_cast<__half*>(k_out),
                            static_cast<__half*>(v_out), (int)lanes);
}

}  // namespace

template <bool NORM>
static cudaError_t launch_append(const AppendParams& p, int cache_dtype, cudaStream_t stream) {
  switch (cache_dtype) {
    case I8KV_CACHE_INT8: return append_of<I8KV_CACHE_INT8, NORM>(p, stream);
    case I8KV_CACHE_FP16: return append_of<I8KV_CACHE_FP16, NORM>(p, stream);
    case I8KV_CACHE_FP8: return append_of<I8KV_CACHE_FP8, NORM>(p, stream);
    case I8KV_CACHE_MX4: return append_of<I8KV_CACHE_MX4, NORM>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_rope_and_cache(const AppendParams& p, int cache_dtype, cudaStream_t stream) {
  return p.q_weight != nullptr || p.k_weight != nullptr || p.k_out != nullptr
             ? launch_append<true>(p, cache_dtype, stream)
             : launch_append<false>(p, cache_dtype, stream);
}

cudaError_t launch_gather_cache(const AppendParams& p, int cache_dtype, void* k_out, void* v_out,
                                cudaStream_t stream) {
  switch (cache_dtype) {
    case I8KV_CACHE_INT8: return gather_of<I8KV_CACHE_INT8>(p, k_out, v_out, stream);
    case I8KV_CACHE_FP16: return gather_of<I8KV_CACHE_FP16>(p, k_out, v_out, stream);
    case I8KV_CACHE_FP8: return gather_of<I8KV_CACHE_FP8>(p, k_out, v_out, stream);
    case I8KV_CACHE_MX4: return gather_of<I8KV_CACHE_MX4>(p, k_out, v_out, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace i8kv
