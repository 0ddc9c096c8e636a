// Paged decode over an MX4 cache (4-bit e2m1 codes, an e4m3 scale per 16
// channels): one new token per sequence, split over the cache's length; the
// partials are joined by the combine kernel.
//
//   s_t = sigma * k_scale * sum_d q_d * (block scale * code)_t,d   (softcap, mask)
//   partial of a piece: m = max s_t, l = sum e^(s_t - m), acc = v_scale sum e^(s_t - m) v_t
//
// One warp per query head, lanes over channels, fp32 throughout.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/int8kv.h"
#include "codes.cuh"
#include "device.cuh"
#include "internal.h"

namespace i8kv {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMinTiles = 4;  // tiles of 16 tokens per piece at least

struct Mx4Item {
  int unit, row, g, slot;
  int lo, hi;    // positions of the piece; lo a multiple of 16
  int wlo;       // first attended position (sliding window)
  int pieces;    // pieces of this row (balanced), or 0
  bool valid;
};

// Live range of row r: [wlo, len), cut from base = wlo rounded down to 16.
__device__ __forceinline__ int tiles_of(const DecodeParams& p, int r, int cap, int& len, int& wlo) {
  len = min(max(p.seq_lens[r], 0), cap);
  wlo = p.window >= 0 ? max(0, len - 1 - p.window) : 0;
  return len > 0 ? ((len + 15) >> 4) - (wlo >> 4) : 0;
}

// Balanced pieces.  With t_b the 16-token tiles of row b's live range, S the
// partial slots of a row and W the pieces the batch should have (one occupancy
// wave of CTAs), every row is cut into n_b = clamp(ceil(t_b / L), 1, S) pieces of
// ceil(t_b / n_b) tiles, L = max(kMinTiles, ceil(Hkv sum t_b / max(W - U, W / 2))),
// U = B * Hkv.  The pieces number at most max(W - U, W / 2) + U (and U * S), which
// bounds the grid by the arguments alone; CTAs past the last piece return.  Item c:
// rows in order, a row's pieces in order, the KV heads of a piece next to each
// other.
__device__ Mx4Item balanced_piece(const DecodeParams& p, int c) {
  const int lane = threadIdx.x & 31;
  const int B = p.rows, Hkv = p.Hkv, S = p.num_splits;
  const int cap = p.max_blocks * p.bs;
  int len, wlo;
  long long tot = 0;
  for (int r = lane; r < B; r += 32) tot += tiles_of(p, r, cap, len, wlo);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
  const long long target = p.bal_pieces;
  const long long want = (tot * Hkv + target - 1) / target;
  const int L = want < kMinTiles ? kMinTiles : (int)want;
  long long base = 0;
  for (int r0 = 0; r0 < B; r0 += 32) {
    const int r = r0 + lane;
    int t = 0, n = 0;
    len = wlo = 0;
    if (r < B) {
      t = tiles_of(p, r, cap, len, wlo);
      n = min(max((t + L - 1) / L, 1), S);
    }
    const int per = t > 0 ? (t + n - 1) / n : 0;  // tiles per piece
    if (t > 0) n = (t + per - 1) / per;           // (no empty last pieces)
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const int total = __shfl_sync(0xffffffffu, inc, 31);
    if (c < (base + total) * Hkv) {
      const int q = (int)(c - base * Hkv);  // item among these rows
      const int piece = q / Hkv;
      const unsigned m = __ballot_sync(0xffffffffu, piece < inc);
      const int src = __ffs(m) - 1;
      Mx4Item it;
      const int n_s = __shfl_sync(0xffffffffu, n, src);
      const int inc_s = __shfl_sync(0xffffffffu, inc, src);
      const int per_s = __shfl_sync(0xffffffffu, per, src);
      const int len_s = __shfl_sync(0xffffffffu, len, src);
      it.wlo = __shfl_sync(0xffffffffu, wlo, src);
      it.row = r0 + src;
      it.g = q - piece * Hkv;
      it.slot = piece - (inc_s - n_s);
      it.unit = it.row * Hkv + it.g;
      it.lo = (it.wlo & ~15) + it.slot * per_s * 16;
      it.hi = min(it.lo + per_s * 16, len_s);
      it.pieces = n_s;
      it.valid = true;
      return it;
    }
    base += total;
  }
  Mx4Item none{};
  none.valid = false;
  return none;
}

__device__ Mx4Item item_of(const DecodeParams& p, int c) {
  if (p.balanced) return balanced_piece(p, c);
  const int units = p.rows * p.Hkv;
  const int cap = p.max_blocks * p.bs;
  Mx4Item it;
  it.slot = c / units;
  it.unit = c - it.slot * units;
  it.row = it.unit / p.Hkv;
  it.g = it.unit - it.row * p.Hkv;
  int len;
  tiles_of(p, it.row, cap, len, it.wlo);
  it.lo = (it.wlo & ~15) + it.slot * p.chunk;
  it.hi = min(min(it.lo + p.chunk, cap), len);
  it.pieces = 0;
  it.valid = true;
  return it;
}

template <int D>
__global__ void __launch_bounds__(kThreads) mx4_decode_kernel(const DecodeParams p) {
  constexpr int C = D / 32;  // channels per lane: C * lane ..
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = p.G;
  const Mx4Item it = item_of(p, blockIdx.x);
  if (!it.valid) return;
  const int live = p.seq_lens[it.row];
  if (it.slot == 0 && it.g == 0 && threadIdx.x == 0 && (live < 0 || live > p.max_blocks * p.bs))
    flag_or(p.flags, I8KV_FLAG_LEN_CLAMPED);
  // slots that no piece fills: empty
  if (it.pieces > 0 && it.slot == 0) {
    for (int e = threadIdx.x; e < (p.num_splits - it.pieces) * G; e += kThreads) {
      const long long b = ((long long)it.unit * p.num_splits + it.pieces) * G + e;
      p.ws_m[b] = neg_inf();
      p.ws_l[b] = 0.f;
    }
  }
  const bool direct = p.num_splits == 1;
  const uint8_t* cache = static_cast<const uint8_t*>(p.k);
  for (int h = warp; h < G; h += kWarps) {
    const long long head = (long long)it.row * p.Hq + it.g * G + h;
    const __half* q = static_cast<const __half*>(p.q) + head * D + C * lane;
    float qv[C], acc[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const float ks = p.per_channel ? p.k_scale[it.g * D + C * lane + i] : p.k_scale[0];
      qv[i] = __half2float(q[i]) * ks;
      acc[i] = 0.f;
    }
    float m = neg_inf(), l = 0.f;
    for (int t = max(it.lo, it.wlo); t < it.hi; ++t) {
      const int blk = p.block_table[(long long)it.row * p.max_blocks + t / p.bs];
      if (blk < 0 || (long long)blk >= p.cache_rows) {
        if (lane == 0) flag_or(p.flags, I8KV_FLAG_BAD_BLOCK);
        continue;
      }
      const int off = t % p.bs;
      const uint8_t* rec = cache + (((long long)blk * p.Hkv + it.g) * (p.bs >> 4) + (off >> 4)) * (18LL * D);
      const int tok = off & 15;
      auto values = [&](const uint8_t* base, float (&x)[C]) {
        uint32_t w = 0;
        const uint8_t* src = base + tok * (D / 2) + lane * (C / 2);
        if constexpr (C == 2) w = *src;
        if constexpr (C == 4) w = *reinterpret_cast<const uint16_t*>(src);
        if constexpr (C == 8) w = *reinterpret_cast<const uint32_t*>(src);
        const float s = e4m3_value(base[8 * D + tok * (D / 16) + (C * lane) / 16]);
        uint32_t hv[4];
        e2m1x8_to_h2x4(w, hv[0], hv[1], hv[2], hv[3]);
#pragma unroll
        for (int i = 0; i < C; i += 2) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hv[i / 2]));
          x[i] = f.x * s;
          x[i + 1] = f.y * s;
        }
      };
      float x[C], s = 0.f;
      values(rec, x);
#pragma unroll
      for (int i = 0; i < C; ++i) s = fmaf(qv[i], x[i], s);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= p.sigma;
      if (p.softcap > 0.f) s = p.softcap * tanhf(s / p.softcap);
      const float mn = fmaxf(m, s);
      const float f = mn == neg_inf() ? 1.f : expf(m - mn), w = mn == neg_inf() ? 0.f : expf(s - mn);
      m = mn;
      l = l * f + w;
      values(rec + 9 * D, x);
#pragma unroll
      for (int i = 0; i < C; ++i) acc[i] = fmaf(w, x[i], acc[i] * f);
    }
    float scale = 1.f;
    if (direct) {
      scale = l > 0.f ? 1.f / l : 0.f;
      if (p.sink != nullptr && l > 0.f)
        scale *= 1.f / (1.f + expf(p.sink[it.g * G + h] - (m + logf(l))));
    }
    const long long base = ((long long)it.unit * p.num_splits + it.slot) * G + h;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int d = C * lane + i;
      const float vs = p.per_channel ? p.v_scale[it.g * D + d] : p.v_scale[0];
      const float o = l > 0.f ? acc[i] * scale * vs : 0.f;
      if (direct)
        static_cast<__half*>(p.out)[head * D + d] = __float2half_rn(o);
      else if (l > 0.f)
        p.ws_acc[base * D + d] = o;
    }
    if (lane == 0) {
      if (!direct) {
        p.ws_m[base] = l > 0.f ? m : neg_inf();
        p.ws_l[base] = l;
      } else if (p.lse != nullptr) {
        p.lse[head] = l > 0.f ? m + logf(l) : neg_inf();
      }
    }
  }
}

template <int D>
cudaError_t run_mx4(const DecodeParams& p, cudaStream_t s, KernelInfo* info) {
  auto kern = mx4_decode_kernel<D>;
  if (info != nullptr) {
    info->round = 16 * kWarps;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&info->occupancy, kern, kThreads, 0);
  }
  const long long units = (long long)p.rows * p.Hkv;
  long long ctas = units * p.num_splits;
  if (p.balanced && ctas > p.bal_pieces + units) ctas = p.bal_pieces + units;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_paged_mx4(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                             KernelInfo* info) {
  switch (key.D) {
    case 64: return run_mx4<64>(p, s, info);
    case 128: return run_mx4<128>(p, s, info);
    case 256: return run_mx4<256>(p, s, info);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace i8kv
