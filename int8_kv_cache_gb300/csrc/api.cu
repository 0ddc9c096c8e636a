// The extern "C" entry points of libint8kv.so (declared in include/int8kv.h):
// argument validation, split geometry, workspace layout and kernel launches.
// Nothing here allocates device memory or synchronises the host.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>
#include <tuple>

#include "../../include/int8kv.h"
#include "attend.h"
#include "internal.h"

namespace {

using i8kv::DecodeParams;
using i8kv::KernelInfo;
using i8kv::KernelKey;
using i8kv::Mx4Way;
using i8kv::Path;

thread_local int g_last_cuda_error = 0;

i8kv_status cuda_fail(cudaError_t e) {
  g_last_cuda_error = static_cast<int>(e);
  return I8KV_ECUDA;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// log2 of a power of two, -1 of any other number.
int32_t log2_of(int32_t x) {
  for (int32_t sh = 0; sh < 31; ++sh)
    if (x == (1 << sh)) return sh;
  return -1;
}

bool supported_head_dim(int32_t D) { return D == 64 || D == 128 || D == 256; }

// Shape checks shared by the decode / prefill calls.
i8kv_status check_heads(int32_t Hq, int32_t Hkv, int32_t D) {
  if (Hq < 1 || Hkv < 1 || D < 1) return I8KV_EINVAL;
  if (Hq % Hkv != 0) return I8KV_EINVAL;
  if (!supported_head_dim(D)) return I8KV_EUNSUPPORTED;
  if (Hq / Hkv > 16) return I8KV_EUNSUPPORTED;
  return I8KV_OK;
}

i8kv_status check_sigma(float s) {
  if (!std::isfinite(s) || s < 0.f) return I8KV_EINVAL;
  if (s > 1.f) return I8KV_EUNSUPPORTED;  // the FP16 path is bounded for scale <= 1 only
  return I8KV_OK;
}

i8kv_status check_scales(const float* ks, const float* vs, int32_t kind) {
  if (kind != I8KV_SCALE_PER_TENSOR && kind != I8KV_SCALE_PER_CHANNEL) return I8KV_EINVAL;
  if (ks == nullptr || vs == nullptr) return I8KV_EINVAL;
  const uintptr_t a = kind == I8KV_SCALE_PER_CHANNEL ? 16 : 4;
  if (!aligned(ks, a) || !aligned(vs, a)) return I8KV_EALIGN;
  return I8KV_OK;
}

KernelKey make_key(Path path, int32_t D, int32_t G, int32_t cache_dtype, bool p_lo) {
  KernelKey k;
  k.path = path;
  k.D = D;
  k.nt = G <= 8 ? 1 : 2;
  k.fp16_cache = cache_dtype == I8KV_CACHE_FP16;
  k.fp8_cache = cache_dtype == I8KV_CACHE_FP8;
  k.p_lo = p_lo;
  k.mx4_cache = cache_dtype == I8KV_CACHE_MX4;
  return k;
}

cudaError_t launch_key(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                       KernelInfo* info) {
  if (key.path == Path::kDsa) {
    return key.p_lo ? i8kv::launch_dsa_decode(key, p, s, info)
                    : i8kv::launch_dsa_prefill(key, p, s, info);
  }
  if (key.mx4_cache) {
    if (key.way == Mx4Way::kCluster) return i8kv::launch_paged_mx4_cluster(key, p, s, info);
    if (key.way == Mx4Way::kRows)
      return key.wide ? i8kv::launch_paged_mx4_rows_wide(key, p, s, info)
                      : i8kv::launch_paged_mx4_rows(key, p, s, info);
    return key.wide ? i8kv::launch_paged_mx4_wide(key, p, s, info)
                    : i8kv::launch_paged_mx4(key, p, s, info);
  }
  if (key.fp16_cache) return i8kv::launch_paged_fp16(key, p, s, info);
  if (key.fp8_cache) return i8kv::launch_paged_fp8(key, p, s, info);
  return i8kv::launch_paged_int8(key, p, s, info);
}

// One occupancy wave (SM count x resident CTAs per SM) of a kernel on the
// current device and the positions of one round of its CTA, cached per
// (device, kernel).
struct WaveInfo {
  int32_t wave;
  int32_t round;
  int32_t clusters[4] = {0, 0, 0, 0};  // cluster kernels: resident clusters of 2, 4, 8 CTAs, from [1]
};

i8kv_status wave_of(const KernelKey& key, WaveInfo* out) {
  static std::mutex mu;
  static std::map<std::tuple<int, int, int, int, int, int, int, int>, WaveInfo> cache;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  const auto k = std::make_tuple(dev, static_cast<int>(key.path), key.D, key.nt,
                                 static_cast<int>(key.fp16_cache), static_cast<int>(key.fp8_cache),
                                 static_cast<int>(key.p_lo),
                                 key.mx4_cache + 2 * key.wide + 4 * key.per_channel +
                                     8 * static_cast<int>(key.way));
  {
    std::lock_guard<std::mutex> lock(mu);
    auto it = cache.find(k);
    if (it != cache.end()) {
      *out = it->second;
      return I8KV_OK;
    }
  }
  int sms = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e);
  DecodeParams dummy{};
  dummy.per_channel = key.per_channel;
  dummy.G = 8 * key.nt;
  KernelInfo info{};
  e = launch_key(key, dummy, nullptr, &info);
  if (e != cudaSuccess) return cuda_fail(e);
  WaveInfo w{std::max(1, sms * std::max(info.occupancy, 1)), std::max(info.round, 16)};
  std::copy(info.clusters, info.clusters + 4, w.clusters);
  {
    std::lock_guard<std::mutex> lock(mu);
    cache[k] = w;
  }
  *out = w;
  return I8KV_OK;
}

// SMs of the current device (cached per device).
i8kv_status sm_count(int* sms) {
  static std::mutex mu;
  static std::map<int, int> cache;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  {
    std::lock_guard<std::mutex> lock(mu);
    auto it = cache.find(dev);
    if (it != cache.end()) {
      *sms = it->second;
      return I8KV_OK;
    }
  }
  int n = 0;
  e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e);
  std::lock_guard<std::mutex> lock(mu);
  cache[dev] = n;
  *sms = n;
  return I8KV_OK;
}

// The dense prefill's split count: num_splits (1 .. I8KV_MAX_SPLITS), or with 0
// the automatic count on the current device.
i8kv_status prefill_splits(int32_t S, int32_t G, int32_t Hkv, int32_t num_splits, int* ns) {
  if (num_splits > 0) {
    *ns = num_splits;
    return I8KV_OK;
  }
  int sms = 0;
  const i8kv_status st = sm_count(&sms);
  if (st != I8KV_OK) return st;
  *ns = i8kv::prefill_auto_splits(S, G, Hkv, sms);
  return I8KV_OK;
}

// The staged prefill's workspace: the operand images and the rows' bitmasks,
// then (with splits) the partials at the next 256-byte boundary.
size_t prefill_ws_bytes(int32_t S, int32_t Hq, int32_t Hkv, int32_t D, int64_t N, int ns) {
  const size_t stage = i8kv::prefill_stage_bytes(N, Hkv, D, S);
  if (ns <= 1) return stage;
  return (stage + 255) / 256 * 256 + i8kv::prefill_partial_bytes(S, Hq, D, ns);
}

constexpr int32_t kGranuleWave = 16;   // the kernels' 16-position MMA tile
constexpr int32_t kGranuleTiles = 64;  // the pages' 64-candidate tile
constexpr int32_t kMinChunk = 128;     // MIN_CHUNK of the wave rule

// The paged decode kernel deals a split's steps (16 or 32 positions) to its 4
// warps in turn, so a chunk that is not a multiple of one round (warps x step:
// 64 or 128 positions) leaves some warps a step, and an HBM round trip, longer
// than the rest.  The automatic wave-rule chunk ceil(cap / n) therefore goes
// to the multiple of the round nearer to it (the lower one only while it stays
// >= MIN_CHUNK and within MAX_SPLITS), and n follows as ceil(cap / chunk).
// Still a function of cap, units and the kernel only.
void snap_to_round(int64_t cap, int64_t round, int32_t* ns, int32_t* chunk) {
  const int64_t raw = cdiv(cap, *ns);
  const int64_t up = cdiv(raw, round) * round;
  const int64_t dn = raw / round * round;
  int64_t ch = up;
  if (dn >= kMinChunk && raw - dn < up - raw && cdiv(cap, dn) <= I8KV_MAX_SPLITS) ch = dn;
  if (ch > INT32_MAX) return;
  *chunk = static_cast<int32_t>(ch);
  *ns = static_cast<int32_t>(cdiv(cap, ch));
}

i8kv_status plan(const KernelKey& key, int64_t cap, int32_t units, int32_t mode, int32_t ovr,
                 int32_t* ns, int32_t* chunk, int32_t* wave_out) {
  WaveInfo w{0, 0};
  i8kv_status st = wave_of(key, &w);
  if (st != I8KV_OK) return st;
  if (wave_out) *wave_out = w.wave;
  const int32_t granule = mode == I8KV_GEOM_POW2_TILES ? kGranuleTiles : kGranuleWave;
  st = split_geometry(cap, units, w.wave, granule, kMinChunk, I8KV_MAX_SPLITS, mode, ovr, ns,
                      chunk);
  if (st != I8KV_OK) return st;
  if (key.path == Path::kPaged && mode == I8KV_GEOM_WAVE && ovr == 0 && cap > 0 && *ns > 1)
    snap_to_round(cap, w.round, ns, chunk);
  return I8KV_OK;
}

// The kernel of the MX4 decode for one CTA per (row, KV head), `units` of them.  Groups of more
// than 8 query heads run as two units of half of them each (*groups = 2) where those are
// resident at once, on the kernel for at most 8, which takes a tile in about two thirds of the
// time (8 rows x 2 groups of 12 heads, head_dim 256, 2064 tokens: 13.2 us in one unit, 10.3 for half
// of it; the keys and values come from L2 twice).
// CTAs of 8 warps where all of them are resident.  Beyond that 4 warps, whose CTAs come and go
// in smaller steps: for spans of at most 1024 tokens (160 rows x 8 heads of 16: 8.6 us against
// 14.4, of 1024: 41 against 47), and for any where they number 4/3 waves or more (128 rows of 128 to
// 8192: 96 us against 100; 160 x 4 groups of 16 heads of 4096: 106 against 127).  Fewer long
// ones are uneven over the SMs (50 rows x 8 heads of 2048: 40 us, in 8 warps 30).
// The waves are those of the kernels for scales per tensor, which is all that the plan knows of; the
// ones for scales per channel hold as many CTAs but for 4 warps and more than 8 heads at
// head_dim 128 (2 per SM, not 3), so that such groups stay at 8 warps up to 2 waves of theirs (104 rows
// x 4 groups of 16 heads of 4096, 1.4 waves: 85 us, in 4 warps 98; 140 rows, 1.8: 113 and 100).
constexpr int64_t kMx4NarrowSpan = 1024;
i8kv_status mx4_rows(const KernelKey& key, int32_t units, int64_t span, KernelKey* run,
                     int32_t* groups, WaveInfo* w) {
  *run = key;
  run->way = Mx4Way::kRows;
  run->wide = true;
  *groups = 1;
  i8kv_status st;
  if (key.nt == 2) {
    KernelKey half = *run;
    half.nt = 1;
    if ((st = wave_of(half, w)) != I8KV_OK) return st;
    if (2LL * units <= w->wave) {
      *run = half;
      *groups = 2;
      return I8KV_OK;
    }
  }
  if ((st = wave_of(*run, w)) != I8KV_OK) return st;
  if (units <= w->wave) return I8KV_OK;
  KernelKey narrow = *run;
  narrow.wide = false;
  WaveInfo w4{0, 0};
  if ((st = wave_of(narrow, &w4)) != I8KV_OK) return st;
  if (span <= kMx4NarrowSpan || 3LL * units >= 4LL * w4.wave) {
    *run = narrow;
    *w = w4;
  }
  return I8KV_OK;
}

// Whether clusters of c CTAs (a power of two, at most kMx4MaxCluster) per (row, KV head) are all
// resident at once, and their kernel; groups of more than 8 query heads as above.
i8kv_status mx4_clusters(const KernelKey& key, int32_t units, int32_t c, bool* fits, KernelKey* run,
                         int32_t* groups) {
  *run = key;
  run->way = Mx4Way::kCluster;
  run->wide = true;
  *groups = 1;
  *fits = false;
  if (c < 2 || c > i8kv::kMx4MaxCluster || (c & (c - 1)) != 0) return I8KV_OK;
  WaveInfo w{0, 0};
  i8kv_status st;
  if (key.nt == 2) {
    KernelKey half = *run;
    half.nt = 1;
    if ((st = wave_of(half, &w)) != I8KV_OK) return st;
    if (2LL * units <= w.clusters[log2_of(c)]) {
      *run = half;
      *groups = 2;
      *fits = true;
      return I8KV_OK;
    }
  }
  st = wave_of(*run, &w);
  *fits = units <= w.clusters[log2_of(c)];
  return st;
}

// The kernel for balanced pieces of the MX4 decode, and its wave: 8-warp CTAs where the partial
// slots keep the 4-warp ones from filling the GPU and the wider ones put more warps to work (one
// row of 131072 tokens, 8 groups of 4 heads: 35.9 us against 41.3; of 65536, 4 groups of 4 heads at
// head_dim 256: 26.7 against 34.4; two of 65536, 8 groups: 33.3 against 36.5).  Where the GPU
// is full of either, 4 warps wait less for each other (16 x 8192-32768 tokens, 8 groups: 64.5 us
// against 76).
i8kv_status mx4_pieces(KernelKey* key, int32_t units, int32_t num_splits, WaveInfo* w) {
  i8kv_status st = wave_of(*key, w);
  const int64_t slots = static_cast<int64_t>(units) * num_splits;
  if (st != I8KV_OK || slots >= w->wave) return st;
  KernelKey wide = *key;
  wide.wide = true;
  WaveInfo w8{0, 0};
  if ((st = wave_of(wide, &w8)) != I8KV_OK) return st;
  if (std::min<int64_t>(slots, w8.wave) * i8kv::kMx4WideWarps > slots * i8kv::kMx4Warps) {
    *key = wide;
    *w = w8;
  }
  return I8KV_OK;
}

// The automatic geometry of the MX4 decode, from the wave rule's count *ns.  A row and KV head
// is one CTA, or a cluster of 2, 4 or 8 of 8 warps that join without a second kernel: the
// most that are resident at once and leave each warp a tile of 16 tokens while every CTA has an SM of
// its own, 7 tiles where they share (16 rows x 2 heads of 2600: 8.2 us in 4 CTAs, one per SM, 9.0 in
// 8), but for spans that give the warps of one CTA at most 4 tiles (2 at head_dim 256) just that one:
// a cluster's launch and join cost 1.2 us (1 row x 8 heads of 300 tokens: 4.5 us, 4.8 in 4 CTAs;
// of 800 6.5 and 5.3).  This is the way
//   - where it gives a warp of a cluster at most 8 tiles (16 rows x 2 KV heads of 2600 tokens: 8.2 us
//     against 11.7 for pieces; 8 x 2 groups of 12 heads of 4096 at head_dim 256:
//     14.1 against 17.1), 6 at head_dim 256 in clusters of 8 (4 x 2 such groups of 8000: 18.7
//     against 15.7), and of a single CTA 16 (36 rows x 8 heads of 2000: 18.8 us against 26.7; of
//     64 to 4000: 27.8 against 27.1), or
//   - where the rows and heads alone fill the GPU and spans are at most 8192 tokens,
//     so that a long row among short ones is not what is waited for (128 rows x 8 heads
//     of 128 to 4096 tokens: 55 us against 93; 80 rows: 42 against 64).
// Else balanced pieces, twice the wave rule's count as partial slots, and the join
// kernel (about 3 us).
constexpr int64_t kMx4WarpTiles = 8, kMx4WarpTilesWide = 6, kMx4WarpTilesRow = 16;
constexpr int64_t kMx4RowTiles = 512;
constexpr int32_t kMx4SharedTiles = 7, kMx4RowTilesOne = 4, kMx4RowTilesWide = 2;
constexpr int64_t kMx4RankSpan = 1024;
i8kv_status mx4_auto(const KernelKey& key, int64_t span, int32_t units, int32_t* ns,
                     int32_t* chunk) {
  const int64_t tiles = cdiv(span, 16);
  KernelKey run = key;
  run.way = Mx4Way::kRows;
  run.wide = true;
  WaveInfo w{0, 0};
  i8kv_status st = wave_of(run, &w);
  if (st != I8KV_OK) return st;
  const bool fills = units >= w.wave && tiles <= kMx4RowTiles;
  int32_t c = 1, groups = 1;
  if ((st = mx4_rows(key, units, span, &run, &groups, &w)) != I8KV_OK) return st;
  bool fits = false;
  int sms = 0;
  if ((st = sm_count(&sms)) != I8KV_OK) return st;
  while (!fills && c < i8kv::kMx4MaxCluster) {
    int32_t each = 2LL * c * units > sms ? kMx4SharedTiles : 1;
    if (c == 1) each = std::max(each, key.D > 128 ? kMx4RowTilesWide : kMx4RowTilesOne);
    if (c * i8kv::kMx4WideWarps * each >= tiles) break;
    int32_t more = 1;
    if ((st = mx4_clusters(key, units, 2 * c, &fits, &run, &more)) != I8KV_OK) return st;
    // (two units of half the heads in smaller clusters are faster than one in larger ones)
    if (!fits || more < groups) break;
    c *= 2;
  }
  const int64_t most = c == 1                                          ? kMx4WarpTilesRow
                       : key.D > 128 && c == i8kv::kMx4MaxCluster ? kMx4WarpTilesWide
                                                                  : kMx4WarpTiles;
  if (fills || tiles <= most * i8kv::kMx4WideWarps * c) {
    *ns = c;
    *chunk = c > 1 ? 0 : static_cast<int32_t>(std::max<int64_t>(16, tiles * 16));
    return I8KV_OK;
  }
  *ns = std::min<int32_t>(I8KV_MAX_SPLITS, std::max<int32_t>(2, 2 * *ns));
  *chunk = 0;
  return I8KV_OK;
}

// Geometry given by the caller: num_splits in [1, 32], chunk a positive
// multiple of 16 with num_splits * chunk >= cap.
// span: the positions the splits must cover (cap, or the window span);
// base_max: the largest first position of split 0 (0, or cap with a window).
i8kv_status check_geometry(int64_t span, int32_t ns, int32_t chunk, int64_t base_max = 0) {
  if (ns < 1 || ns > I8KV_MAX_SPLITS) return I8KV_EINVAL;
  if (chunk < 16 || chunk % 16 != 0) return I8KV_EINVAL;
  if (static_cast<int64_t>(ns) * chunk < span) return I8KV_EINVAL;
  // positions are 32-bit on the device
  if (base_max + static_cast<int64_t>(ns) * chunk > INT32_MAX) return I8KV_EINVAL;
  return I8KV_OK;
}

i8kv_status set_workspace(DecodeParams& p, void* ws, size_t ws_bytes, int32_t units, int32_t ns,
                          int32_t G, int32_t D) {
  p.ws_acc = p.ws_m = p.ws_l = nullptr;
  if (ns <= 1) return I8KV_OK;
  const size_t need = split_workspace_bytes(units, ns, G, D);
  if (ws == nullptr || ws_bytes < need) return I8KV_EWORKSPACE;
  if (!aligned(ws, 16)) return I8KV_EALIGN;
  float* base = static_cast<float*>(ws);
  const size_t nacc = static_cast<size_t>(units) * ns * G * D;
  const size_t nml = static_cast<size_t>(units) * ns * G;
  p.ws_acc = base;
  p.ws_m = base + nacc;
  p.ws_l = base + nacc + nml;
  return I8KV_OK;
}

i8kv_status run(const KernelKey& key, const DecodeParams& p, cudaStream_t s) {
  cudaError_t e = launch_key(key, p, s, nullptr);
  if (e != cudaSuccess) return cuda_fail(e);
  if (p.num_splits > 1 && p.out != nullptr) {
    e = i8kv::launch_combine(p.ws_acc, p.ws_m, p.ws_l, p.rows * p.Hkv, p.num_splits, p.Hq, p.Hkv,
                             key.D, p.sink, p.out, p.lse, s);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return I8KV_OK;
}

// Common checks of the sparse-candidate calls; fills the shape part of p.
i8kv_status dsa_common(const uint16_t* q, const int8_t* k, const int8_t* v, const float* ks,
                       const float* vs, int32_t kind, const int32_t* idx, int32_t S, int32_t Hq,
                       int32_t Hkv, int32_t D, int64_t N, int32_t max_sel, float sigma,
                       const float* sink, uint16_t* out, float* lse, uint32_t* flags,
                       DecodeParams& p) {
  if (S < 0 || N < 0 || max_sel < 0) return I8KV_EINVAL;
  i8kv_status st = check_heads(Hq, Hkv, D);
  if (st != I8KV_OK) return st;
  if ((st = check_sigma(sigma)) != I8KV_OK) return st;
  if ((st = check_scales(ks, vs, kind)) != I8KV_OK) return st;
  if (S > 0 && (q == nullptr || k == nullptr || v == nullptr)) return I8KV_EINVAL;
  if (S > 0 && max_sel > 0 && idx == nullptr) return I8KV_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k, 16) || !aligned(v, 16)) return I8KV_EALIGN;
  if (!aligned(idx, 4) || !aligned(lse, 4) || !aligned(sink, 4) || !aligned(flags, 4)) return I8KV_EALIGN;
  p = DecodeParams{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.k_scale = ks;
  p.v_scale = vs;
  p.per_channel = kind == I8KV_SCALE_PER_CHANNEL;
  p.idx = idx;
  p.sink = sink;
  p.out = out;
  p.lse = lse;
  p.flags = flags;
  p.cache_rows = N;
  p.rows = S;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.max_sel = max_sel;
  p.sigma = sigma;
  p.softcap = 0.f;
  p.window = -1;
  p.lpt = 0;
  return I8KV_OK;
}

}  // namespace

extern "C" {

const char* i8kv_status_string(int status) {
  switch (status) {
    case I8KV_OK: return "ok";
    case I8KV_EINVAL: return "invalid argument";
    case I8KV_EUNSUPPORTED: return "unsupported shape or option";
    case I8KV_EALIGN: return "misaligned pointer";
    case I8KV_EWORKSPACE: return "workspace missing or too small";
    case I8KV_ECUDA: return "CUDA error";
    default: return "unknown status";
  }
}

int32_t i8kv_version(void) { return 300; }

// The CUDA error code behind the calling thread's last I8KV_ECUDA (0 if none).
int32_t i8kv_last_cuda_error(void) { return g_last_cuda_error; }

int64_t paged_window_span(int64_t cap, int32_t window) { return I8KV_WINDOW_SPAN(cap, window); }

i8kv_status split_geometry(int64_t cap, int32_t units, int32_t wave_ctas, int32_t granule,
                           int32_t min_chunk, int32_t max_splits, int32_t mode,
                           int32_t override_value, int32_t* num_splits, int32_t* chunk) {
  if (num_splits == nullptr || chunk == nullptr) return I8KV_EINVAL;
  if (units < 1 || wave_ctas < 1 || granule < 1 || min_chunk < 1 || max_splits < 1 ||
      override_value < 0)
    return I8KV_EINVAL;
  if (mode != I8KV_GEOM_WAVE && mode != I8KV_GEOM_POW2_TILES) return I8KV_EINVAL;
  if (cap <= 0) {
    *num_splits = 1;
    *chunk = granule;
    return I8KV_OK;
  }
  int64_t n = 0, ch = 0;
  if (mode == I8KV_GEOM_WAVE) {
    if (override_value > 0) {
      n = std::min<int64_t>(cdiv(cap, override_value), max_splits);
    } else {
      const int64_t target = cdiv(wave_ctas, units);
      n = std::min<int64_t>(std::min<int64_t>(target, cdiv(cap, min_chunk)), max_splits);
    }
    n = std::max<int64_t>(n, 1);
    ch = cdiv(cdiv(cap, n), granule) * granule;
    n = cdiv(cap, ch);
  } else {
    const int64_t tiles = cdiv(cap, granule);
    int64_t tps = 1;
    if (override_value > 0) {
      tps = override_value;
    } else {
      while (cdiv(tiles, tps) * units > wave_ctas && tps < tiles) tps *= 2;
    }
    n = std::max<int64_t>(1, std::min<int64_t>(cdiv(tiles, tps), max_splits));
    const int64_t te = cdiv(tiles, n);
    n = cdiv(tiles, te);
    ch = te * granule;
  }
  if (ch > INT32_MAX) return I8KV_EINVAL;
  *num_splits = static_cast<int32_t>(n);
  *chunk = static_cast<int32_t>(ch);
  return I8KV_OK;
}

size_t split_workspace_bytes(int32_t units, int32_t num_splits, int32_t G, int32_t D) {
  if (num_splits <= 1 || units < 1 || G < 1 || D < 1) return 0;
  return static_cast<size_t>(units) * num_splits * G * (static_cast<size_t>(D) + 2) * sizeof(float);
}

i8kv_status decode_plan(int32_t path, int32_t cache_dtype, int64_t cap, int32_t rows, int32_t Hq,
                        int32_t Hkv, int32_t D, int32_t mode, int32_t override_value,
                        int32_t* num_splits, int32_t* chunk, size_t* workspace_bytes,
                        int32_t* wave_ctas) {
  if (num_splits == nullptr || chunk == nullptr || workspace_bytes == nullptr) return I8KV_EINVAL;
  if (path != I8KV_PATH_DSA && path != I8KV_PATH_PAGED) return I8KV_EINVAL;
  if (cache_dtype != I8KV_CACHE_INT8 && cache_dtype != I8KV_CACHE_FP16 &&
      cache_dtype != I8KV_CACHE_FP8 && cache_dtype != I8KV_CACHE_MX4)
    return I8KV_EINVAL;
  if (path == I8KV_PATH_DSA && cache_dtype != I8KV_CACHE_INT8) return I8KV_EUNSUPPORTED;
  if (rows < 0 || cap < 0) return I8KV_EINVAL;
  i8kv_status st = check_heads(Hq, Hkv, D);
  if (st != I8KV_OK) return st;
  const int32_t G = Hq / Hkv;
  const KernelKey key = make_key(path == I8KV_PATH_DSA ? Path::kDsa : Path::kPaged, D, G,
                                 cache_dtype, true);
  const int32_t units = std::max(1, rows * Hkv);
  if (mode == I8KV_GEOM_BALANCED) {
    // balanced pieces: twice the wave rule's splits as partial slots (at most
    // MAX_SPLITS), chunk 0 (the pieces are cut on the device)
    if (path != I8KV_PATH_PAGED) return I8KV_EUNSUPPORTED;
    if ((st = plan(key, cap, units, I8KV_GEOM_WAVE, 0, num_splits, chunk, wave_ctas)) != I8KV_OK)
      return st;
    if (key.mx4_cache) {
      if ((st = mx4_auto(key, cap, units, num_splits, chunk)) != I8KV_OK) return st;
      *workspace_bytes = split_workspace_bytes(rows * Hkv, *num_splits, G, D);
      return I8KV_OK;
    }
    *num_splits = std::min<int32_t>(I8KV_MAX_SPLITS, std::max<int32_t>(2, 2 * *num_splits));
    *chunk = 0;
  } else if ((st = plan(key, cap, units, mode, override_value, num_splits, chunk, wave_ctas)) !=
             I8KV_OK) {
    return st;
  }
  *workspace_bytes = split_workspace_bytes(rows * Hkv, *num_splits, G, D);
  return I8KV_OK;
}

i8kv_status dsa_decode(const uint16_t* q, const int8_t* k_cache, const int8_t* v_cache,
                       const float* k_scale, const float* v_scale, int32_t scale_kind,
                       const int32_t* idx, int32_t S, int32_t Hq, int32_t Hkv, int32_t D,
                       int64_t N, int32_t max_sel, float softmax_scale, const float* head_sink,
                       int32_t num_splits, int32_t chunk, void* workspace,
                       size_t workspace_bytes, uint16_t* out, float* lse, uint32_t* flags,
                       void* stream) {
  DecodeParams p;
  i8kv_status st = dsa_common(q, k_cache, v_cache, k_scale, v_scale, scale_kind, idx, S, Hq, Hkv,
                              D, N, max_sel, softmax_scale, head_sink, out, lse, flags, p);
  if (st != I8KV_OK) return st;
  if (num_splits < 0) return I8KV_EINVAL;
  const KernelKey key = make_key(Path::kDsa, D, p.G, I8KV_CACHE_INT8, true);
  if (num_splits == 0) {
    st = plan(key, max_sel, std::max(1, S * Hkv), I8KV_GEOM_POW2_TILES, 0, &num_splits, &chunk,
              nullptr);
    if (st != I8KV_OK) return st;
  } else if ((st = check_geometry(max_sel, num_splits, chunk)) != I8KV_OK) {
    return st;
  }
  if ((st = set_workspace(p, workspace, workspace_bytes, S * Hkv, num_splits, p.G, D)) != I8KV_OK)
    return st;
  if (out == nullptr && num_splits == 1 && S > 0) return I8KV_EINVAL;  // nowhere to write
  if (S == 0) return I8KV_OK;
  p.num_splits = num_splits;
  p.chunk = chunk;
  return run(key, p, static_cast<cudaStream_t>(stream));
}

i8kv_status dsa_prefill(const uint16_t* q, const int8_t* k_cache, const int8_t* v_cache,
                        const float* k_scale, const float* v_scale, int32_t scale_kind,
                        const int32_t* idx, int32_t S, int32_t Hq, int32_t Hkv, int32_t D,
                        int64_t N, int32_t max_sel, float softmax_scale,
                        const float* head_sink, uint16_t* out, float* lse, uint32_t* flags,
                        void* stream) {
  return dsa_prefill_ws(q, k_cache, v_cache, k_scale, v_scale, scale_kind, idx, S, Hq, Hkv, D, N,
                        max_sel, softmax_scale, head_sink, 0, nullptr, 0, out, lse, flags, stream);
}

int32_t dsa_prefill_auto_splits(int32_t S, int32_t Hq, int32_t Hkv, int32_t sms) {
  if (S < 1 || sms < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return 0;
  return i8kv::prefill_auto_splits(S, Hq / Hkv, Hkv, sms);
}

size_t dsa_prefill_workspace_bytes(int32_t S, int32_t Hq, int32_t Hkv, int32_t D, int64_t N,
                                   int32_t max_sel, int32_t num_splits) {
  if (S < 1 || N < 1 || max_sel < 1 || check_heads(Hq, Hkv, D) != I8KV_OK) return 0;
  if (num_splits < 0 || num_splits > I8KV_MAX_SPLITS) return 0;
  int smem = 0, mask_rows = 0;
  if (!i8kv::prefill_tc_plan(D, Hq / Hkv, S, N, max_sel, &smem, &mask_rows)) return 0;
  int ns = 1;
  if (prefill_splits(S, Hq / Hkv, Hkv, num_splits, &ns) != I8KV_OK) return 0;
  return prefill_ws_bytes(S, Hq, Hkv, D, N, ns);
}

i8kv_status dsa_prefill_ws(const uint16_t* q, const int8_t* k_cache, const int8_t* v_cache,
                           const float* k_scale, const float* v_scale, int32_t scale_kind,
                           const int32_t* idx, int32_t S, int32_t Hq, int32_t Hkv, int32_t D,
                           int64_t N, int32_t max_sel, float softmax_scale,
                           const float* head_sink, int32_t num_splits, void* workspace,
                           size_t workspace_bytes, uint16_t* out, float* lse, uint32_t* flags,
                           void* stream) {
  DecodeParams p;
  i8kv_status st = dsa_common(q, k_cache, v_cache, k_scale, v_scale, scale_kind, idx, S, Hq, Hkv,
                              D, N, max_sel, softmax_scale, head_sink, out, lse, flags, p);
  if (st != I8KV_OK) return st;
  if (S > 0 && out == nullptr) return I8KV_EINVAL;
  if (num_splits < 0 || num_splits > I8KV_MAX_SPLITS) return I8KV_EINVAL;
  if (!aligned(workspace, 16)) return I8KV_EALIGN;
  if (S == 0) return I8KV_OK;
  p.num_splits = 1;
  p.chunk = static_cast<int32_t>(std::max<int64_t>(16, cdiv(max_sel, 16) * 16));
  // dense tensor-core kernel where the rows' lists cover the cache densely
  // enough (a shape rule, so eager and captured calls choose alike), else the
  // gathering mma.sync kernel
  int smem = 0, mask_rows = 0;
  if (i8kv::prefill_tc_plan(D, p.G, S, N, max_sel, &smem, &mask_rows)) {
    // with a workspace: the staged form (fp16 operand images and the rows'
    // bitmasks made once per call, the images copied in by one thread), its
    // tiles' blocks split over several CTAs where the tiles alone leave SMs
    // idle; without: the converting form, unsplit
    void* stage = nullptr;
    int ns = 1;
    float* part = nullptr;
    if (workspace != nullptr) {
      st = prefill_splits(S, p.G, Hkv, num_splits, &ns);
      if (st != I8KV_OK) return st;
      if (workspace_bytes < prefill_ws_bytes(S, Hq, Hkv, D, N, ns)) return I8KV_EWORKSPACE;
      stage = workspace;
      if (ns > 1)
        part = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                        (i8kv::prefill_stage_bytes(N, Hkv, D, S) + 255) / 256 * 256);
    } else if (num_splits > 1) {
      return I8KV_EWORKSPACE;  // the partials need one
    }
    cudaError_t e = i8kv::launch_dsa_prefill_tc(p, D, smem, mask_rows, stage, ns, part,
                                                static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? I8KV_OK : cuda_fail(e);
  }
  return run(make_key(Path::kDsa, D, p.G, I8KV_CACHE_INT8, false), p,
             static_cast<cudaStream_t>(stream));
}

}  // extern "C"

namespace {

i8kv_status paged_common(const uint16_t* q, const void* k_cache, const void* v_cache,
                         int32_t cache_dtype, const float* k_scale, const float* v_scale,
                         int32_t scale_kind, const int32_t* block_table,
                         const int32_t* seq_lens, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                         int32_t block_size, int32_t max_blocks, int64_t num_blocks,
                         float softmax_scale, const float* head_sink, float softcap,
                         int32_t window, int32_t num_splits, int32_t chunk, void* workspace,
                         size_t workspace_bytes, uint16_t* out, float* lse, int32_t* slots_out,
                         uint32_t* flags, void* stream) {
  if (B < 0 || max_blocks < 0 || num_blocks < 0 || block_size < 1 || num_splits < 0)
    return I8KV_EINVAL;
  if (!(softcap >= 0.f) || !std::isfinite(softcap) || window < -1) return I8KV_EINVAL;
  i8kv_status st = check_heads(Hq, Hkv, D);
  if (st != I8KV_OK) return st;
  if (block_size % 16 != 0) return I8KV_EUNSUPPORTED;
  if ((st = check_sigma(softmax_scale)) != I8KV_OK) return st;
  if (cache_dtype != I8KV_CACHE_INT8 && cache_dtype != I8KV_CACHE_FP16 &&
      cache_dtype != I8KV_CACHE_FP8)
    return I8KV_EINVAL;
  const bool fp16c = cache_dtype == I8KV_CACHE_FP16;
  if (!fp16c && (st = check_scales(k_scale, v_scale, scale_kind)) != I8KV_OK) return st;
  if (B > 0 && (q == nullptr || k_cache == nullptr || v_cache == nullptr ||
                seq_lens == nullptr || (max_blocks > 0 && block_table == nullptr)))
    return I8KV_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return I8KV_EALIGN;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) ||
      !aligned(head_sink, 4) || !aligned(slots_out, 4) || !aligned(flags, 4))
    return I8KV_EALIGN;
  const int64_t cap = static_cast<int64_t>(max_blocks) * block_size;
  if (cap > INT32_MAX) return I8KV_EUNSUPPORTED;
  const int32_t G = Hq / Hkv;
  const KernelKey key = make_key(Path::kPaged, D, G, cache_dtype, true);
  const int64_t span = I8KV_WINDOW_SPAN(cap, window);
  if (num_splits == 0) {
    st = plan(key, span, std::max(1, B * Hkv), I8KV_GEOM_WAVE, 0, &num_splits, &chunk, nullptr);
    if (st != I8KV_OK) return st;
  }
  // chunk 0 with num_splits > 1: balanced pieces cut on the device (at most
  // num_splits per row)
  const bool balanced = num_splits > 1 && chunk == 0;
  if (balanced) {
    if (num_splits > I8KV_MAX_SPLITS) return I8KV_EINVAL;
    if (slots_out != nullptr || B > i8kv::kLptMaxRows) return I8KV_EUNSUPPORTED;
  } else if ((st = check_geometry(span, num_splits, chunk, window >= 0 ? cap : 0)) != I8KV_OK) {
    return st;
  }
  DecodeParams p{};
  if ((st = set_workspace(p, workspace, workspace_bytes, B * Hkv, num_splits, G, D)) != I8KV_OK)
    return st;
  if (out == nullptr && num_splits == 1 && B > 0) return I8KV_EINVAL;  // nowhere to write
  if (B == 0) return I8KV_OK;
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.k_scale = fp16c ? nullptr : k_scale;
  p.v_scale = fp16c ? nullptr : v_scale;
  p.per_channel = scale_kind == I8KV_SCALE_PER_CHANNEL;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.sink = head_sink;
  p.out = out;
  p.lse = lse;
  p.slots_out = slots_out;
  p.flags = flags;
  p.cache_rows = num_blocks;
  p.rows = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.bs = block_size;
  p.bs_log2 = -1;
  for (int sh = 4; sh < 31; ++sh)
    if (block_size == (1 << sh)) p.bs_log2 = sh;
  p.max_blocks = max_blocks;
  p.num_splits = num_splits;
  p.chunk = chunk;
  p.sigma = softmax_scale;
  p.softcap = softcap;
  p.window = window;
  // longest-first dispatch: ragged batches of long chunks (a property of the
  // geometry, so eager and captured launches make the same choice)
  p.lpt = !balanced && B <= i8kv::kLptMaxRows && chunk >= i8kv::kLptMinChunk;
  if (balanced) {
    // about one wave of CTAs over the KV heads, at least one piece per row,
    // at most what the grid of ceil(num_splits / 2) CTAs per unit holds
    WaveInfo w{0, 0};
    if ((st = wave_of(key, &w)) != I8KV_OK) return st;
    p.balanced = 1;
    p.bal_round = w.round;
    p.bal_pieces = std::min<int32_t>(std::max<int32_t>(w.wave / Hkv, B),
                                     B * ((num_splits + 1) / 2));
  }
  return run(key, p, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

i8kv_status paged_decode(const uint16_t* q, const void* k_cache, const void* v_cache,
                         int32_t cache_dtype, const float* k_scale, const float* v_scale,
                         int32_t scale_kind, const int32_t* block_table,
                         const int32_t* seq_lens, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                         int32_t block_size, int32_t max_blocks, int64_t num_blocks,
                         float softmax_scale, const float* head_sink, int32_t num_splits,
                         int32_t chunk, void* workspace, size_t workspace_bytes, uint16_t* out,
                         float* lse, int32_t* slots_out, uint32_t* flags, void* stream) {
  return paged_common(q, k_cache, v_cache, cache_dtype, k_scale, v_scale, scale_kind, block_table,
                      seq_lens, B, Hq, Hkv, D, block_size, max_blocks, num_blocks, softmax_scale,
                      head_sink, 0.f, -1, num_splits, chunk, workspace, workspace_bytes, out, lse,
                      slots_out, flags, stream);
}

i8kv_status paged_decode_ex(const uint16_t* q, const void* k_cache, const void* v_cache,
                            int32_t cache_dtype, const float* k_scale, const float* v_scale,
                            int32_t scale_kind, const int32_t* block_table,
                            const int32_t* seq_lens, int32_t B, int32_t Hq, int32_t Hkv,
                            int32_t D, int32_t block_size, int32_t max_blocks, int64_t num_blocks,
                            float softmax_scale, const float* head_sink, float softcap,
                            int32_t window, int32_t num_splits, int32_t chunk, void* workspace,
                            size_t workspace_bytes, uint16_t* out, float* lse,
                            int32_t* slots_out, uint32_t* flags, void* stream) {
  return paged_common(q, k_cache, v_cache, cache_dtype, k_scale, v_scale, scale_kind, block_table,
                      seq_lens, B, Hq, Hkv, D, block_size, max_blocks, num_blocks, softmax_scale,
                      head_sink, softcap, window, num_splits, chunk, workspace, workspace_bytes,
                      out, lse, slots_out, flags, stream);
}

i8kv_status paged_decode_mx4(const uint16_t* q, const void* cache, const float* k_scale,
                             const float* v_scale, int32_t scale_kind,
                             const int32_t* block_table, const int32_t* seq_lens, int32_t B,
                             int32_t Hq, int32_t Hkv, int32_t D, int32_t block_size,
                             int32_t max_blocks, int64_t num_blocks, float softmax_scale,
                             const float* head_sink, float softcap, int32_t window,
                             int32_t num_splits, int32_t chunk, void* workspace,
                             size_t workspace_bytes, uint16_t* out, float* lse, uint32_t* flags,
                             void* stream) {
  if (B < 0 || max_blocks < 0 || num_blocks < 0 || block_size < 1 || num_splits < 0)
    return I8KV_EINVAL;
  if (!(softcap >= 0.f) || !std::isfinite(softcap) || window < -1) return I8KV_EINVAL;
  i8kv_status st = check_heads(Hq, Hkv, D);
  if (st != I8KV_OK) return st;
  if (block_size % 16 != 0) return I8KV_EUNSUPPORTED;
  if ((st = check_sigma(softmax_scale)) != I8KV_OK) return st;
  if ((st = check_scales(k_scale, v_scale, scale_kind)) != I8KV_OK) return st;
  if (B > 0 && (q == nullptr || cache == nullptr || seq_lens == nullptr ||
                (max_blocks > 0 && block_table == nullptr)))
    return I8KV_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache, 16)) return I8KV_EALIGN;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) ||
      !aligned(head_sink, 4) || !aligned(flags, 4))
    return I8KV_EALIGN;
  const int64_t cap = static_cast<int64_t>(max_blocks) * block_size;
  // positions, CTA numbers and the batch's 16-token tiles are 32-bit on the device
  if (cap > INT32_MAX - 16 || static_cast<int64_t>(B) * Hkv * I8KV_MAX_SPLITS > INT32_MAX ||
      static_cast<int64_t>(B) * (cap / 16 + 1) > INT32_MAX - 64)
    return I8KV_EUNSUPPORTED;
  const int32_t units = std::max(1, B * Hkv);
  const KernelKey key = make_key(Path::kPaged, D, Hq / Hkv, I8KV_CACHE_MX4, false);
  const int64_t span = I8KV_WINDOW_SPAN(cap, window);
  if (num_splits == 0) {
    st = plan(key, span, units, I8KV_GEOM_WAVE, 0, &num_splits, &chunk, nullptr);
    if (st != I8KV_OK) return st;
    if ((st = mx4_auto(key, span, units, &num_splits, &chunk)) != I8KV_OK) return st;
  }
  DecodeParams p{};
  p.balanced = num_splits > 1 && chunk == 0;
  if (p.balanced) {
    if (num_splits > I8KV_MAX_SPLITS) return I8KV_EINVAL;
  } else if ((st = check_geometry(span, num_splits, chunk, window >= 0 ? cap : 0)) != I8KV_OK) {
    return st;
  }
  if ((st = set_workspace(p, workspace, workspace_bytes, B * Hkv, num_splits, Hq / Hkv, D)) !=
      I8KV_OK)
    return st;
  if (out == nullptr && num_splits == 1 && B > 0) return I8KV_EINVAL;  // nowhere to write
  if (B == 0) return I8KV_OK;
  p.q = q;
  p.k = cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.per_channel = scale_kind == I8KV_SCALE_PER_CHANNEL;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.sink = head_sink;
  p.out = out;
  p.lse = lse;
  p.flags = flags;
  p.cache_rows = num_blocks;
  p.rows = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.bs = block_size;
  p.bs_log2 = log2_of(block_size);
  p.max_blocks = max_blocks;
  p.num_splits = num_splits;
  p.chunk = chunk;
  p.sigma = softmax_scale;
  p.softcap = softcap;
  p.window = window;
  // one split, and balanced pieces that fit clusters, join inside the kernel
  KernelKey own;
  bool joins = num_splits == 1;
  if (num_splits == 1) {
    WaveInfo w{0, 0};
    if ((st = mx4_rows(key, units, span, &own, &p.head_groups, &w)) != I8KV_OK) return st;
    // More rows and heads than are resident: long rows start first, so that none is what the
    // rest waits for (50 rows x 8 heads of 128 to 4096 tokens: 29 us against 40 in the rows'
    // order, 128 rows: 65 against 75; in all 3 us less now).  Finding the row costs a CTA
    // 0.8 us (128 rows of 2048 tokens each: 67 us against 65), so not for short spans.
    p.longest_first = B <= i8kv::kMx4RankRows && span >= kMx4RankSpan &&
                      static_cast<int64_t>(units) * p.head_groups > w.wave;
  } else if (p.balanced && out != nullptr) {
    if ((st = mx4_clusters(key, units, num_splits, &joins, &own, &p.head_groups)) != I8KV_OK)
      return st;
  }
  if (joins) {
    const cudaError_t e = launch_key(own, p, static_cast<cudaStream_t>(stream), nullptr);
    return e == cudaSuccess ? I8KV_OK : cuda_fail(e);
  }
  own = key;  // (the plan, which does not know the scales, sets the slots only)
  if (p.balanced) {
    own.per_channel = p.per_channel;
    WaveInfo w{0, 0};
    if ((st = mx4_pieces(&own, units, num_splits, &w)) != I8KV_OK) return st;
    // (at least one piece per row and KV head, and one to spare)
    p.bal_pieces = std::max(w.wave, units + std::max(w.wave / 2, Hkv));
  }
  return run(own, p, static_cast<cudaStream_t>(stream));
}

size_t mx4_cache_bytes(int64_t num_blocks, int32_t block_size, int32_t Hkv, int32_t D) {
  if (num_blocks < 1 || block_size < 16 || block_size % 16 != 0 || Hkv < 1 ||
      !supported_head_dim(D))
    return 0;
  return static_cast<size_t>(num_blocks) * Hkv * (block_size / 16) * 18 * D;
}

i8kv_status split_combine(const float* acc, const float* m, const float* l, int32_t units,
                          int32_t num_splits, int32_t Hq, int32_t Hkv, int32_t D,
                          const float* head_sink, uint16_t* out, float* lse, void* stream) {
  if (units < 0 || num_splits < 1 || num_splits > I8KV_MAX_SPLITS) return I8KV_EINVAL;
  i8kv_status st = check_heads(Hq, Hkv, D);
  if (st != I8KV_OK) return st;
  if (units > 0 && (acc == nullptr || m == nullptr || l == nullptr || out == nullptr))
    return I8KV_EINVAL;
  if (!aligned(acc, 16) || !aligned(out, 16) || !aligned(m, 4) || !aligned(l, 4) ||
      !aligned(lse, 4) || !aligned(head_sink, 4))
    return I8KV_EALIGN;
  if (units == 0) return I8KV_OK;
  cudaError_t e = i8kv::launch_combine(acc, m, l, units, num_splits, Hq, Hkv, D, head_sink, out,
                                       lse, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? I8KV_OK : cuda_fail(e);
}

i8kv_status reshape_and_cache(const uint16_t* k_new, const uint16_t* v_new,
                              const int32_t* slot_mapping, int32_t num_tokens, int32_t Hkv,
                              int32_t D, void* k_cache, void* v_cache, int64_t num_slots,
                              const float* k_scale, const float* v_scale, int32_t scale_kind,
                              int32_t cache_dtype, uint32_t* flags, void* stream) {
  if (num_tokens < 0 || Hkv < 1 || D < 8 || num_slots < 0) return I8KV_EINVAL;
  if (cache_dtype != I8KV_CACHE_INT8 && cache_dtype != I8KV_CACHE_FP8) return I8KV_EINVAL;
  if (D % 8 != 0) return I8KV_EUNSUPPORTED;
  i8kv_status st = check_scales(k_scale, v_scale, scale_kind);
  if (st != I8KV_OK) return st;
  if (num_tokens > 0 && (k_new == nullptr || v_new == nullptr || slot_mapping == nullptr ||
                         k_cache == nullptr || v_cache == nullptr))
    return I8KV_EINVAL;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(slot_mapping, 4) || !aligned(flags, 4))
    return I8KV_EALIGN;
  if (num_tokens == 0) return I8KV_OK;
  cudaError_t e = i8kv::launch_reshape_and_cache(
      k_new, v_new, slot_mapping, num_tokens, Hkv, D, k_cache, v_cache, num_slots, k_scale, v_scale,
      scale_kind == I8KV_SCALE_PER_CHANNEL, cache_dtype == I8KV_CACHE_FP8, flags,
      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? I8KV_OK : cuda_fail(e);
}

// Elements of a token's row that 32-bit item numbers take with room to spare.
static constexpr int64_t kMaxRow = 1 << 28;

// What rope_and_cache and gather_cache check alike: the cache and its scales.
static i8kv_status check_cache(const void* k_cache, const void* v_cache, int32_t cache_dtype,
                               int64_t num_slots, int32_t block_size, const float* k_scale,
                               const float* v_scale, int32_t scale_kind, int32_t Hkv, int32_t D,
                               bool used) {
  if (Hkv < 1 || D < 1 || num_slots < 0) return I8KV_EINVAL;
  if (cache_dtype < I8KV_CACHE_INT8 || cache_dtype > I8KV_CACHE_MX4) return I8KV_EINVAL;
  const bool mx4 = cache_dtype == I8KV_CACHE_MX4;
  if (D % 16 != 0 || (mx4 && !supported_head_dim(D))) return I8KV_EUNSUPPORTED;
  if (static_cast<int64_t>(Hkv) * D > kMaxRow) return I8KV_EUNSUPPORTED;
  if (mx4) {
    if (block_size < 1 || v_cache != nullptr) return I8KV_EINVAL;
    if (block_size % 16 != 0) return I8KV_EUNSUPPORTED;
    if (num_slots % block_size != 0) return I8KV_EINVAL;
  }
  if (cache_dtype != I8KV_CACHE_FP16) {
    const i8kv_status st = check_scales(k_scale, v_scale, scale_kind);
    if (st != I8KV_OK) return st;
  }
  if (used && (k_cache == nullptr || (!mx4 && v_cache == nullptr))) return I8KV_EINVAL;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return I8KV_EALIGN;
  return I8KV_OK;
}

static i8kv_status append(const uint16_t* q, int64_t q_stride, const uint16_t* k_new,
                          int64_t k_stride, const uint16_t* v_new, int64_t v_stride,
                          const int32_t* positions, const float* cos_sin, int64_t max_pos,
                          int32_t rot_dim, int32_t rot_style, const int32_t* slot_mapping,
                          int32_t num_tokens, int32_t Hq, int32_t Hkv, int32_t D,
                          uint16_t* q_out, void* k_cache, void* v_cache, int32_t cache_dtype,
                          int64_t num_slots, int32_t block_size, const float* k_scale,
                          const float* v_scale, int32_t scale_kind, const float* q_weight,
                          const float* k_weight, float eps, uint16_t* k_out, uint32_t* flags,
                          void* stream) {
  if (num_tokens < 0 || Hq < 0 || max_pos < 0) return I8KV_EINVAL;
  if (rot_style != I8KV_ROPE_HALVES && rot_style != I8KV_ROPE_INTERLEAVED) return I8KV_EINVAL;
  i8kv_status st = check_cache(k_cache, v_cache, cache_dtype, num_slots, block_size, k_scale,
                               v_scale, scale_kind, Hkv, D, num_tokens > 0);
  if (st != I8KV_OK) return st;
  if (rot_dim < 0 || rot_dim > D) return I8KV_EINVAL;
  if (static_cast<int64_t>(Hq) * D > kMaxRow) return I8KV_EUNSUPPORTED;
  if (rot_dim % 16 != 0 || (cache_dtype == I8KV_CACHE_MX4 && rot_style == I8KV_ROPE_HALVES &&
                            rot_dim % 32 != 0))
    return I8KV_EUNSUPPORTED;
  if (num_tokens > 0) {
    if (k_new == nullptr || v_new == nullptr || slot_mapping == nullptr) return I8KV_EINVAL;
    if (Hq > 0 && (q == nullptr || q_out == nullptr)) return I8KV_EINVAL;
    if (rot_dim > 0 && (positions == nullptr || cos_sin == nullptr)) return I8KV_EINVAL;
  }
  if (num_tokens > 1 && (q_stride < (Hq > 0 ? static_cast<int64_t>(Hq) * D : 0) ||
                         k_stride < static_cast<int64_t>(Hkv) * D ||
                         v_stride < static_cast<int64_t>(Hkv) * D))
    return I8KV_EINVAL;
  if (num_tokens > 1 && ((Hq > 0 && q_stride % 8 != 0) || k_stride % 8 != 0 || v_stride % 8 != 0))
    return I8KV_EALIGN;
  if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(q_out, 16) ||
      !aligned(cos_sin, 16) || !aligned(positions, 4) || !aligned(slot_mapping, 4) ||
      !aligned(flags, 4))
    return I8KV_EALIGN;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(k_out, 16)) return I8KV_EALIGN;
  if (num_tokens == 0) return I8KV_OK;
  i8kv::AppendParams p{};
  p.q = reinterpret_cast<const __half*>(q);
  p.k = reinterpret_cast<const __half*>(k_new);
  p.v = reinterpret_cast<const __half*>(v_new);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.max_pos = max_pos;
  p.R = rot_dim;
  p.interleaved = rot_style == I8KV_ROPE_INTERLEAVED;
  p.slots = slot_mapping;
  p.num_tokens = num_tokens;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.q_out = reinterpret_cast<__half*>(q_out);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.num_slots = num_slots;
  p.bs = block_size;
  p.bs_shift = log2_of(block_size);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.per_channel = scale_kind == I8KV_SCALE_PER_CHANNEL;
  p.flags = flags;
  p.q_weight = Hq > 0 ? q_weight : nullptr;
  p.k_weight = k_weight;
  p.eps = eps;
  p.k_out = reinterpret_cast<__half*>(k_out);
  cudaError_t e = i8kv::launch_rope_and_cache(p, cache_dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? I8KV_OK : cuda_fail(e);
}

i8kv_status rope_and_cache(const uint16_t* q, int64_t q_stride, const uint16_t* k_new,
                           int64_t k_stride, const uint16_t* v_new, int64_t v_stride,
                           const int32_t* positions, const float* cos_sin, int64_t max_pos,
                           int32_t rot_dim, int32_t rot_style, const int32_t* slot_mapping,
                           int32_t num_tokens, int32_t Hq, int32_t Hkv, int32_t D,
                           uint16_t* q_out, void* k_cache, void* v_cache, int32_t cache_dtype,
                           int64_t num_slots, int32_t block_size, const float* k_scale,
                           const float* v_scale, int32_t scale_kind, uint32_t* flags,
                           void* stream) {
  return append(q, q_stride, k_new, k_stride, v_new, v_stride, positions, cos_sin, max_pos, rot_dim,
                rot_style, slot_mapping, num_tokens, Hq, Hkv, D, q_out, k_cache, v_cache,
                cache_dtype, num_slots, block_size, k_scale, v_scale, scale_kind, nullptr, nullptr,
                0.f, nullptr, flags, stream);
}

i8kv_status norm_rope_and_cache(const uint16_t* q, int64_t q_stride, const uint16_t* k_new,
                                int64_t k_stride, const uint16_t* v_new, int64_t v_stride,
                                const float* q_weight, const float* k_weight, float eps,
                                const int32_t* positions, const float* cos_sin, int64_t max_pos,
                                int32_t rot_dim, int32_t rot_style, const int32_t* slot_mapping,
                                int32_t num_tokens, int32_t Hq, int32_t Hkv, int32_t D,
                                uint16_t* q_out, uint16_t* k_out, void* k_cache, void* v_cache,
                                int32_t cache_dtype, int64_t num_slots, int32_t block_size,
                                const float* k_scale, const float* v_scale, int32_t scale_kind,
                                uint32_t* flags, void* stream) {
  if (!(eps >= 0.f) || !std::isfinite(eps)) return I8KV_EINVAL;
  // a head's lanes are a power of two
  if ((q_weight != nullptr || k_weight != nullptr) && Hkv > 0 && D > 0 && !supported_head_dim(D))
    return I8KV_EUNSUPPORTED;
  return append(q, q_stride, k_new, k_stride, v_new, v_stride, positions, cos_sin, max_pos, rot_dim,
                rot_style, slot_mapping, num_tokens, Hq, Hkv, D, q_out, k_cache, v_cache,
                cache_dtype, num_slots, block_size, k_scale, v_scale, scale_kind, q_weight, k_weight,
                eps, k_out, flags, stream);
}

i8kv_status gather_cache(const int32_t* slot_mapping, int32_t num_rows, int32_t Hkv, int32_t D,
                         const void* k_cache, const void* v_cache, int32_t cache_dtype,
                         int64_t num_slots, int32_t block_size, const float* k_scale,
                         const float* v_scale, int32_t scale_kind, uint16_t* k_out,
                         uint16_t* v_out, uint32_t* flags, void* stream) {
  if (num_rows < 0) return I8KV_EINVAL;
  i8kv_status st = check_cache(k_cache, v_cache, cache_dtype, num_slots, block_size, k_scale,
                               v_scale, scale_kind, Hkv, D, num_rows > 0);
  if (st != I8KV_OK) return st;
  if (num_rows > 0 && slot_mapping == nullptr) return I8KV_EINVAL;
  if (!aligned(slot_mapping, 4) || !aligned(k_out, 16) || !aligned(v_out, 16) ||
      !aligned(flags, 4))
    return I8KV_EALIGN;
  if (num_rows == 0 || (k_out == nullptr && v_out == nullptr)) return I8KV_OK;
  i8kv::AppendParams p{};
  p.slots = slot_mapping;
  p.num_tokens = num_rows;
  p.Hkv = Hkv;
  p.D = D;
  p.k_cache = const_cast<void*>(k_cache);
  p.v_cache = const_cast<void*>(v_cache);
  p.num_slots = num_slots;
  p.bs = block_size;
  p.bs_shift = log2_of(block_size);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.per_channel = scale_kind == I8KV_SCALE_PER_CHANNEL;
  p.flags = flags;
  cudaError_t e = i8kv::launch_gather_cache(p, cache_dtype, k_out, v_out,
                                            static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? I8KV_OK : cuda_fail(e);
}

// What packed_prefill and paged_prefill check alike.
static i8kv_status check_attend(const uint16_t* q, int64_t q_stride, const int32_t* starts,
                                int32_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                float softmax_scale, const float* head_sink, float softcap,
                                int32_t window, const uint16_t* out, const float* lse,
                                const uint32_t* flags) {
  if (T < 0 || B < 0) return I8KV_EINVAL;
  if (!(softcap >= 0.f) || !std::isfinite(softcap) || window < -1) return I8KV_EINVAL;
  i8kv_status st = check_heads(Hq, Hkv, D);
  if (st != I8KV_OK) return st;
  if ((st = check_sigma(softmax_scale)) != I8KV_OK) return st;
  if (T > 0 && B > 0 && (q == nullptr || out == nullptr || starts == nullptr)) return I8KV_EINVAL;
  if (T > 1 && q_stride < static_cast<int64_t>(Hq) * D) return I8KV_EINVAL;
  if (T > 1 && q_stride % 8 != 0) return I8KV_EALIGN;
  if (!aligned(q, 16) || !aligned(out, 16)) return I8KV_EALIGN;
  if (!aligned(starts, 4) || !aligned(lse, 4) || !aligned(head_sink, 4) || !aligned(flags, 4))
    return I8KV_EALIGN;
  // a sequence's vectors of a KV head, and the CTAs, are numbered in 32 bits
  if (static_cast<int64_t>(T) * (Hq / Hkv) > INT32_MAX - 512 ||
      (static_cast<int64_t>(T) * (Hq / Hkv) / 128 + std::min(B, T)) * Hkv > INT32_MAX)
    return I8KV_EUNSUPPORTED;
  return I8KV_OK;
}

static i8kv::AttendParams attend_params(const uint16_t* q, int64_t q_stride, const int32_t* starts,
                                        int32_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                        float softmax_scale, const float* head_sink, float softcap,
                                        int32_t window, uint16_t* out, float* lse,
                                        uint32_t* flags) {
  i8kv::AttendParams p{};
  p.q = reinterpret_cast<const __half*>(q);
  p.q_stride = q_stride;
  p.starts = starts;
  p.T = T;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.D = D;
  p.sigma = softmax_scale;
  p.sink = head_sink;
  p.softcap = softcap;
  p.window = window;
  p.out = reinterpret_cast<__half*>(out);
  p.lse = lse;
  p.flags = flags;
  return p;
}

// How a call of packed_prefill or paged_prefill is dealt out: two tiles of 128 vectors per CTA where
// sequences have about that many and, whole, they fill the GPU (one tile at a time spreads wider);
// pieces (see attend_cuts) where whole (tile, KV head)s would leave SMs idle.
struct AttendPlan {
  bool two = false;
  int32_t pieces = 0;   // 0: whole (tile, KV head)s
  unsigned ctas = 0;
  size_t workspace = 0;
};
// Whether the automatic choice cuts the batch into pieces, given how many (tile, KV head)s it has (us, int8,
// 32 / 8 heads x 128 unless said, whole / cut; 152 SMs):
//   one tile per CTA: below three rounds of the SMs (single tokens over 512 to 8192 in 20 sequences 84 / 57, in 48
//     129 / 123, in 64 143 / 148, in 256 213 / 325; 24 / 2 x 256, 200 to 300 over 1000 to 8192 in four 210 / 195)
//   two, one sequence, whose tiles are of about one length: where the last round is not nearly full
//     (1216 tokens over 16384 245 / 280, 1400 453 / 324, 2048 453 / 438, 2432 453 / 500, 4096 826 / 774)
//   two, several: below nine tenths of a round (128 tokens over 1024 to 16384 in four 167 / 120; 512 in eight 244 / 307;
//     1 to 512 in twelve, MX4, 141 / 179; 300 to 1001 over 1001 to 4096 in four, e4m3fn, 16 / 2 x 64, 50 / 70):
//     beyond, the longest first fill the gaps, and the merge costs more (not so where one sequence is far longer:
//     512 over 16384 and over 600 in eleven more 298 / 254, which only the device knows).  288 batches of 3 and 8 sequences
//     of 0.37 to 1.15 rounds, each kind of cache, 32 / 8 x 128 and 16 / 2 x 64, whole's time over cut's (geometric mean):
//     over prefixes of 2000 to 8000 tokens 1.14 below nine tenths (81 of 104 faster cut), 0.90 beyond (35 of 40 faster
//     whole); over prefixes of one to three times the new tokens 0.52 and 0.61.  So the border is where whole tiles begin to
//     win for either; below it the lengths decide, which the host does not know
static bool attend_cuts(int64_t items, bool pairs, int32_t seqs, int sms) {
  if (!pairs) return items < INT64_C(3) * sms;
  if (seqs > 1) return items * 10 < INT64_C(9) * sms;
  const int64_t rounds = (items + sms - 1) / sms;
  return rounds <= 4 && items * 10 < rounds * sms * 9;
}
static AttendPlan attend_plan(int32_t T, int32_t B, int32_t G, int32_t Hkv, int32_t D, int64_t cap,
                              int sms, int32_t num_splits) {
  AttendPlan a;
  const int64_t vec = static_cast<int64_t>(T) * G;
  const int32_t seqs = std::min(B, T);
  const bool pairs = D <= 128 && vec / seqs >= 192;
  const int64_t tiles = std::max<int64_t>(vec / (pairs ? 256 : 128), seqs);
  if (num_splits > 1)
    a.pieces = num_splits;
  else if (num_splits == 0 && cap > 128 && attend_cuts(tiles * Hkv, pairs, seqs, sms))
    a.pieces = sms;
  a.two = pairs && (a.pieces > 0 || tiles * Hkv * 10 >= INT64_C(9) * sms);
  const int32_t M = a.two ? 256 : 128;
  a.ctas = static_cast<unsigned>(a.pieces > 0 ? a.pieces : std::min<int64_t>((vec / M + seqs) * Hkv, sms));
  a.workspace = static_cast<size_t>(a.pieces) * 2 * M * (D + 2) * 4;
  return a;
}

i8kv_status packed_prefill(const uint16_t* q, int64_t q_stride, const uint16_t* k,
                           int64_t k_stride, const uint16_t* v, int64_t v_stride,
                           const int32_t* seq_start, int32_t T, int32_t B, int32_t Hq, int32_t Hkv,
                           int32_t D, float softmax_scale, const float* head_sink, float softcap,
                           int32_t window, uint16_t* out, float* lse, uint32_t* flags,
                           void* stream) {
  i8kv_status st = check_attend(q, q_stride, seq_start, T, B, Hq, Hkv, D, softmax_scale, head_sink,
                                softcap, window, out, lse, flags);
  if (st != I8KV_OK) return st;
  const int64_t row = static_cast<int64_t>(Hkv) * D;
  if (T > 0 && B > 0 && (k == nullptr || v == nullptr)) return I8KV_EINVAL;
  if (T > 1 && (k_stride < row || v_stride < row)) return I8KV_EINVAL;
  if (T > 1 && (k_stride % 8 != 0 || v_stride % 8 != 0)) return I8KV_EALIGN;
  if (!aligned(k, 16) || !aligned(v, 16)) return I8KV_EALIGN;
  // (a copy's token stride has 40 bits of bytes)
  if (T > 1 && (k_stride >= INT64_C(1) << 38 || v_stride >= INT64_C(1) << 38)) return I8KV_EUNSUPPORTED;
  if (T == 0 || B == 0) return I8KV_OK;
  i8kv::AttendParams p = attend_params(q, q_stride, seq_start, T, B, Hq, Hkv, D, softmax_scale,
                                       head_sink, softcap, window, out, lse, flags);
  p.k = k;
  p.v = v;
  p.k_stride = T > 1 ? k_stride : row;
  p.v_stride = T > 1 ? v_stride : row;
  p.rows = T;
  int sms = 0;
  if ((st = sm_count(&sms)) != I8KV_OK) return st;
  const AttendPlan plan = attend_plan(T, B, p.G, Hkv, D, 0, sms, 1);
  const cudaError_t e = i8kv::launch_attend_f16(p, plan.two, plan.ctas, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? I8KV_OK : cuda_fail(e);
}

size_t paged_prefill_workspace_bytes(int32_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                     int64_t cap, int32_t num_splits) {
  if (T < 1 || B < 1 || cap < 0 || num_splits < 0 || num_splits > I8KV_MAX_PIECES ||
      check_heads(Hq, Hkv, D) != I8KV_OK)
    return 0;
  int sms = 0;
  if (num_splits == 0 && sm_count(&sms) != I8KV_OK) return 0;
  return attend_plan(T, B, Hq / Hkv, Hkv, D, cap, sms, num_splits).workspace;
}

i8kv_status paged_prefill(const uint16_t* q, int64_t q_stride, const void* k_cache,
                          const void* v_cache, int32_t cache_dtype, const float* k_scale,
                          const float* v_scale, int32_t scale_kind, const int32_t* block_table,
                          const int32_t* seq_lens, const int32_t* query_start, int32_t T,
                          int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t block_size,
                          int32_t max_blocks, int64_t num_blocks, float softmax_scale,
                          const float* head_sink, float softcap, int32_t window,
                          int32_t num_splits, void* workspace, size_t workspace_bytes,
                          uint16_t* out, float* lse, uint32_t* flags, void* stream) {
  i8kv_status st = check_attend(q, q_stride, query_start, T, B, Hq, Hkv, D, softmax_scale,
                                head_sink, softcap, window, out, lse, flags);
  if (st != I8KV_OK) return st;
  if (max_blocks < 0 || num_blocks < 0 || block_size < 1) return I8KV_EINVAL;
  if (num_splits < 0 || num_splits > I8KV_MAX_PIECES) return I8KV_EINVAL;
  if (cache_dtype < I8KV_CACHE_INT8 || cache_dtype > I8KV_CACHE_MX4) return I8KV_EINVAL;
  if (block_size % 16 != 0) return I8KV_EUNSUPPORTED;
  const bool mx4 = cache_dtype == I8KV_CACHE_MX4, fp16c = cache_dtype == I8KV_CACHE_FP16;
  if (!fp16c && (st = check_scales(k_scale, v_scale, scale_kind)) != I8KV_OK) return st;
  const bool works = T > 0 && B > 0;
  if (works && (k_cache == nullptr || (!mx4 && v_cache == nullptr) || seq_lens == nullptr ||
                (max_blocks > 0 && block_table == nullptr)))
    return I8KV_EINVAL;
  if (mx4 && v_cache != nullptr) return I8KV_EINVAL;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return I8KV_EALIGN;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4)) return I8KV_EALIGN;
  // positions, rows of 16 tokens and a plain cache's rows are 32-bit on the device
  const int64_t cap = static_cast<int64_t>(max_blocks) * block_size;
  if (cap > INT32_MAX - 512 || num_blocks > (INT64_C(1) << 31) ||
      num_blocks * (block_size / 16) > INT32_MAX ||
      (!mx4 && num_blocks * block_size > INT32_MAX))
    return I8KV_EUNSUPPORTED;
  if (!aligned(workspace, 16)) return I8KV_EALIGN;
  int sms = 0;
  if (works && (st = sm_count(&sms)) != I8KV_OK) return st;
  AttendPlan plan;
  if (works) {
    plan = attend_plan(T, B, Hq / Hkv, Hkv, D, cap, sms, num_splits);
    if (plan.pieces > 0 && (workspace == nullptr || workspace_bytes < plan.workspace)) {
      if (num_splits > 1) return I8KV_EWORKSPACE;
      plan = attend_plan(T, B, Hq / Hkv, Hkv, D, cap, sms, 1);
    }
  }
  if (!works) return I8KV_OK;
  i8kv::AttendParams p = attend_params(q, q_stride, query_start, T, B, Hq, Hkv, D, softmax_scale,
                                       head_sink, softcap, window, out, lse, flags);
  p.k = k_cache;
  p.v = v_cache;
  p.k_scale = fp16c ? nullptr : k_scale;
  p.v_scale = fp16c ? nullptr : v_scale;
  p.per_channel = !fp16c && scale_kind == I8KV_SCALE_PER_CHANNEL;
  // (a table without blocks is not read, and a sequence is empty then)
  p.table = block_table != nullptr ? block_table : seq_lens;
  p.lens = seq_lens;
  p.bs = block_size;
  p.bs_log2 = log2_of(block_size);
  p.max_blocks = max_blocks;
  p.cap = static_cast<int32_t>(cap);
  p.num_blocks = num_blocks;
  // (a tensor map has a row at least: without blocks it is not read)
  p.rows = mx4 ? 0 : static_cast<int32_t>(std::max<int64_t>(1, num_blocks * block_size));
  p.pieces = plan.pieces;
  const bool two = plan.two;
  const unsigned ctas = plan.ctas;
  if (plan.pieces > 0) {
    const size_t rows = static_cast<size_t>(plan.pieces) * 2 * (two ? 256 : 128);
    p.part_acc = static_cast<float*>(workspace);
    p.part_m = p.part_acc + rows * D;
    p.part_l = p.part_m + rows;
  }
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  switch (cache_dtype) {
    case I8KV_CACHE_INT8: e = i8kv::launch_attend_int8(p, two, ctas, s); break;
    case I8KV_CACHE_FP8: e = i8kv::launch_attend_fp8(p, two, ctas, s); break;
    case I8KV_CACHE_MX4: e = i8kv::launch_attend_mx4(p, two, ctas, s); break;
    default: e = i8kv::launch_attend_f16(p, two, ctas, s);
  }
  if (e == cudaSuccess && plan.pieces > 1) e = i8kv::launch_attend_merge(p, two, s);
  return e == cudaSuccess ? I8KV_OK : cuda_fail(e);
}

i8kv_status fp8_to_fp16(const uint8_t* in, uint16_t* out, int64_t n, void* stream) {
  if (n < 0 || n % 4 != 0) return I8KV_EINVAL;
  if (n > 0 && (in == nullptr || out == nullptr)) return I8KV_EINVAL;
  if (!aligned(in, 16) || !aligned(out, 16)) return I8KV_EALIGN;
  cudaError_t e = i8kv::launch_fp8_to_fp16(in, out, n, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? I8KV_OK : cuda_fail(e);
}

i8kv_status int8_to_fp16(const int8_t* in, uint16_t* out, int64_t n, void* stream) {
  if (n < 0 || n % 4 != 0) return I8KV_EINVAL;
  if (n > 0 && (in == nullptr || out == nullptr)) return I8KV_EINVAL;
  if (!aligned(in, 16) || !aligned(out, 16)) return I8KV_EALIGN;
  cudaError_t e = i8kv::launch_int8_to_fp16(in, out, n, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? I8KV_OK : cuda_fail(e);
}

}  // extern "C"
