// Launch of attend_kernel.cuh for one kind of source (a translation unit each).
#pragma once

#include <atomic>

#include "attend_kernel.cuh"

namespace i8kv {
namespace ap {

// The tensor map of rows [rows, Hkv, D] (fp16, or bytes) whose tokens are `stride` elements apart: boxes
// of `box` rows of one head by `wide` channels, zeros out of range; fp16 with the 128-byte swizzle.
inline cudaError_t map_of(CUtensorMap* m, const void* base, bool fp16, int D, int Hkv, long long stride, long long rows,
                          int box, int wide) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<Encode> known{nullptr};
  Encode encode = known.load();
  if (encode == nullptr) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || f == nullptr) return cudaErrorNotSupported;
    encode = reinterpret_cast<Encode>(f);
    known.store(encode);
  }
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)rows};
  const int size = fp16 ? 2 : 1;
  const cuuint64_t strides[2] = {(cuuint64_t)D * size, (cuuint64_t)stride * size};
  const cuuint32_t boxes[3] = {(cuuint32_t)wide, 1, (cuuint32_t)box};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r = encode(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, boxes, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE,
                            fp16 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int TILES, int SRC>
cudaError_t launch(const Args& a, unsigned ctas, cudaStream_t s) {
  auto kern = attend_kernel<D, TILES, SRC>;
  constexpr int kSmem = Raw<D, TILES, SRC>::kSmem;
  static std::atomic<unsigned long long> done{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int SRC>
cudaError_t launch_of(const AttendParams& p, bool two_tiles, unsigned ctas, cudaStream_t s) {
  Args a{};
  a.p = p;
  if (SRC != kMx4) {
    const bool paged = p.table != nullptr, fp16 = SRC == kF16;
    const long long row = (long long)p.Hkv * p.D;
    const int wide = fp16 ? 64 : p.D < 128 ? p.D : 128;
    cudaError_t e = map_of(&a.km, p.k, fp16, p.D, p.Hkv, paged ? row : p.k_stride, p.rows, paged ? 16 : 128, wide);
    if (e == cudaSuccess)
      e = map_of(&a.vm, p.v, fp16, p.D, p.Hkv, paged ? row : p.v_stride, p.rows, paged ? 16 : p.D == 256 ? 64 : 128, wide);
    if (e != cudaSuccess) return e;
  }
  switch (p.D) {
    case 64: return two_tiles ? launch<64, 2, SRC>(a, ctas, s) : launch<64, 1, SRC>(a, ctas, s);
    case 128: return two_tiles ? launch<128, 2, SRC>(a, ctas, s) : launch<128, 1, SRC>(a, ctas, s);
    case 256: return launch<256, 1, SRC>(a, ctas, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ap
}  // namespace i8kv
