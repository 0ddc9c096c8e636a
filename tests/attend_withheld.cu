// The dense causal attention with copies or arrivals that do not come, for test_gpu_attend_waits.py: a wait for them
// runs out after 20 ms, and the kernel returns.  No access is other than the whole kernel's, and every wait ends: those for
// barriers in memory by their limit or by the word in which one that ran out is told, the named barriers because all of
// their warps come to them whatever became of their waits.
#include <cuda_runtime.h>

namespace {
struct Held {
  int what, item, block;
};
__device__ Held held;
}  // namespace
#define I8KV_ATTEND_WAIT_NS 20000000ull
#define I8KV_ATTEND_WITHHELD(w, i, b) (held.what == (int)(w) && held.item == (int)(i) && held.block == (int)(b))

#include "../int8_kv_cache_gb300/csrc/attend_launch.cuh"

using namespace i8kv;

// One CTA (or `pieces`) of the kernel <D, two ? 2 : 1, src> over fp16 prompts (table NULL) or int8 pages of 16, and
// the device's state behind it.
extern "C" __attribute__((visibility("default"))) int attend_withheld(int what, int item, int block, int src, int two, int pieces, const void* q, const void* k,
                               const void* v, const float* scale, const int32_t* table, const int32_t* lens,
                               const int32_t* starts, int T, int B, int Hq, int Hkv, int D, int max_blocks, int num_blocks,
                               void* out, float* lse, uint32_t* flags, float* part_acc, float* part_m, float* part_l) {
  const Held h{what, item, block};
  cudaError_t e = cudaMemcpyToSymbol(held, &h, sizeof h);
  if (e != cudaSuccess) return e;
  ap::Args a{};
  AttendParams& p = a.p;
  p.q = static_cast<const __half*>(q);
  p.q_stride = static_cast<long long>(Hq) * D;
  p.k = k;
  p.v = v;
  p.k_stride = p.v_stride = static_cast<long long>(Hkv) * D;
  p.k_scale = p.v_scale = scale;
  p.table = table;
  p.lens = lens;
  p.starts = starts;
  p.out = static_cast<__half*>(out);
  p.lse = lse;
  p.flags = flags;
  p.part_acc = part_acc;
  p.part_m = part_m;
  p.part_l = part_l;
  p.pieces = pieces;
  p.T = T;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.D = D;
  p.bs = 16;
  p.bs_log2 = 4;
  p.max_blocks = max_blocks;
  p.cap = max_blocks * 16;
  p.num_blocks = num_blocks;
  p.rows = table != nullptr ? num_blocks * 16 : T;
  p.sigma = 1.f / 16;
  p.window = -1;
  const bool fp16 = src == ap::kF16;
  const int wide = fp16 ? 64 : 128;
  e = ap::map_of(&a.km, k, fp16, D, Hkv, p.k_stride, p.rows, table != nullptr ? 16 : 128, wide);
  if (e == cudaSuccess)
    e = ap::map_of(&a.vm, v, fp16, D, Hkv, p.v_stride, p.rows, table != nullptr ? 16 : D == 256 ? 64 : 128, wide);
  const unsigned ctas = pieces > 0 ? pieces : 1;
  if (e == cudaSuccess) {
    e = cudaErrorInvalidValue;
    if (fp16 && D == 128) e = two ? ap::launch<128, 2, ap::kF16>(a, ctas, nullptr) : ap::launch<128, 1, ap::kF16>(a, ctas, nullptr);
    if (fp16 && D == 256 && !two) e = ap::launch<256, 1, ap::kF16>(a, ctas, nullptr);
    if (src == ap::kI8 && D == 128) e = two ? ap::launch<128, 2, ap::kI8>(a, ctas, nullptr) : ap::launch<128, 1, ap::kI8>(a, ctas, nullptr);
  }
  if (e != cudaSuccess) return e;
  return cudaDeviceSynchronize();
}
