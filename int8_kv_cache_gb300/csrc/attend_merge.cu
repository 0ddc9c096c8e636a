// Merge of the partials of attend_kernel's pieces (attend_kernel.cuh): a (tile, KV head) whose
// blocks fell into several CTAs' pieces,
//   M = max_k m_k;  L = sum_k l_k e^(m_k - M);  O = sum_k acc_k e^(m_k - M) / L;
//   lse = M + ln L;  O <- O / (1 + e^(s_h - lse)).
// One CTA per cut between two pieces and 16 of the tile's vectors; it finds the (tile, head) that the
// cut is in from the lengths, as the pieces' CTAs did, and goes on if the cut is the first one in
// it.  A warp takes a vector at a time: its lanes hold 4 channels (2 with head_dim 64) at once, and
// the pieces' partials are loaded a few at a time.  Whole tiles were written by the pieces' CTAs.
#include "attend_launch.cuh"

namespace i8kv {
namespace ap {

constexpr int kMergeThreads = 128, kMergeVectors = 16;

template <int D, int M>
__global__ void __launch_bounds__(kMergeThreads) attend_merge_kernel(const AttendParams p) {
  constexpr int V = D / 32;  // channels of a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The lengths are inputs of attend_kernel, which lets this kernel launch once it may read them itself:
  // the cut is found while its last CTAs still work.
  const int cut = blockIdx.x + 1;
  long long total, x = 0;
  const long long one = piece_length<M>(p, p.pieces, total);
  const long long f = one * cut;
  Item it;
  Length len;
  if (f < total) x = find_place<M>(p, f, it, len);
  // the partials; also where there is nothing to do: the stream goes on when all of this grid has ended,
  // and attend_kernel has to have ended by then
  grid_dependency_wait();
  if (x == 0 || x > one) return;  // the cut is between two tiles, or not the first one in this one
  // pieces cut - 1 (its end), cut, ..., last (their beginnings)
  const int last = (int)((f + (len.of(it.t) - x) - 1) / one);
  const int v0 = it.t * M, nvec = it.q.n * p.G;
  for (int r = blockIdx.y * kMergeVectors + warp; r < (blockIdx.y + 1) * kMergeVectors; r += kMergeThreads / 32) {
    const int v = v0 + r;
    if (v >= nvec) break;
    // slot of piece k: 2 (cut - 1) + 1 + k for the first two, then every second one
    auto slot_of = [&](int k) -> long long { return (long long)(k < cut ? 2 * k + 1 : 2 * k) * M + r; };
    float top = neg_inf();
    for (int k = cut - 1 + lane; k <= last; k += 32) top = fmaxf(top, p.part_m[slot_of(k)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.f;
    bool nan = false;
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    for (int k0 = cut - 1; k0 <= last; k0 += 4) {
      float m[4], l[4], a[4][V];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[j] = neg_inf();
        l[j] = 0.f;
        if (k0 + j <= last) {
          const long long at = slot_of(k0 + j);
          m[j] = p.part_m[at];
          l[j] = p.part_l[at];
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const float2 y = *reinterpret_cast<const float2*>(p.part_acc + at * D + 64 * (e / 2) + 2 * lane);
            a[j][e] = y.x;
            a[j][e + 1] = y.y;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // a piece that attends nothing of this vector has no sums: they are not looked at
        if (m[j] == neg_inf()) continue;
        nan |= l[j] != l[j];
        const float w = fast_exp2((m[j] - top) * kLog2e);
        sum = fmaf(w, l[j], sum);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(w, a[j][e], acc[e]);
      }
    }
    const int tok = v / p.G, h = it.g * p.G + v - tok * p.G;
    float lse = neg_inf(), scale = 0.f;
    if (nan || sum != sum) {
      lse = scale = __int_as_float(0x7fc00000);
    } else if (sum > 0.f) {
      lse = top + logf(sum);
      scale = 1.f / sum;
      if (p.sink != nullptr) scale *= 1.f / (1.f + expf(p.sink[h] - lse));
    }
    const long long row = (it.q.s0 + (long long)tok) * p.Hq + h;
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const uint32_t y = scale == 0.f ? 0u : pack_h2(acc[e] * scale, acc[e + 1] * scale);
      *reinterpret_cast<uint32_t*>(p.out + row * D + 64 * (e / 2) + 2 * lane) = y;
    }
    if (lane == 0 && p.lse != nullptr) p.lse[row] = lse;
  }
}

template <int D, int M>
cudaError_t merge(const AttendParams& p, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.pieces - 1, M / kMergeVectors);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_merge_kernel<D, M>, p);
}

}  // namespace ap

cudaError_t launch_attend_merge(const AttendParams& p, bool two_tiles, cudaStream_t s) {
  switch (p.D) {
    case 64: return two_tiles ? ap::merge<64, 256>(p, s) : ap::merge<64, 128>(p, s);
    case 128: return two_tiles ? ap::merge<128, 256>(p, s) : ap::merge<128, 128>(p, s);
    case 256: return ap::merge<256, 128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace i8kv
