// Paged decode over an MX4 cache (4-bit e2m1 codes, an e4m3 scale per 16 channels): one
// new token per sequence, split over the cache's length and joined.
//
// What it computes, for the G query heads of a KV head over the tokens t of a piece:
//   s_t = sigma * k_scale * sum_d q_d * (block scale * code)_t,d    (softcap, mask)
//   m = reference exponent, l = sum e^(s_t - m), acc = v_scale sum e^(s_t - m) v_t
// and from the pieces of a row O = sum acc e^(m - M) / sum l e^(m - M), the sink, the lse.
//
// Bound: HBM in bytes, the integer pipe in practice.  A record of 16 tokens is 18 D bytes
// (2304 at head_dim 128) and one bulk copy into the ring of the warp that works on it: two
// stages of two records per warp, 16 warps per SM, about 110 KB in flight.  At 6.8 TB/s an SM
// gets a record every 98 cycles; what it issues for one is about 277 instructions (123 of them
// for the integer pipe, which takes one every second cycle: 62 cycles of its four
// schedulers' time), so instructions are what was worked on:
//   - Matrix fragments straight from shared memory.  S = K Q'^T takes tokens as rows and a
//     lane's 32 (head_dim 128) consecutive channels of a token as its part of the contraction:
//     two 16-byte loads, no transposition; the queries are permuted to match.  O^T = V^T P^T
//     takes channels as rows: a lane's 16 channels of four tokens, whose nibbles are paired
//     across tokens with one shift and one select per 8 codes.
//   - Codes to fp16 with one conversion per pair (64 a cycle and SM), times the block scale:
//     code * scale has 6 significant bits, so the fp16 products are exact.
//   - The exponent base of a head moves only when a score exceeds it by 15 bits, so a
//     stage needs no shuffles: 2^8 .. 2^15 is the room that fp16 probabilities leave above
//     the largest so far.  The probabilities are rounded to fp16 (relative 2^-11 at most; the
//     output itself is fp16); their sum and everything accumulated is fp32.
//   - Copy descriptions (address, attended tokens) are formed 32 tiles at a time, a lane each.
// Measured on one GB300 (graph of calls, inputs larger than L2): 16 x 8192-32768 tokens, 32/8
// heads, head_dim 128: 62.5 us, 5.2 TB/s, 77 % of the measured copy rate (integer pipe 53 %
// of its cycles, issue 60 %).  Tried and slower than its 64 to 70 us of then: one record per stage
// (78 us), three stages (73), 8-warp CTAs (76), 5 CTAs per SM (71).  An odd record at a warp's
// end is worked alone (a pair with nothing in its second half costs as much as two).
//
// Ways over the work, chosen by the host from sizes alone (api.cu): balanced pieces of rows (4-warp
// CTAs, 8-warp ones for few long rows) or chunks, joined by the combine kernel; clusters of 8-warp
// CTAs per row and KV head, joined in distributed shared memory; one CTA each, of 4 or 8 warps
// (without the cluster's barriers, which cost such a CTA 1.5 us).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "../../include/int8kv.h"
#include "codes.cuh"
#include "device.cuh"
#include "internal.h"
#include "tc.cuh"

namespace i8kv {

namespace {

struct Mx4Item {
  int unit, row, g, slot;
  int tile0, stride;  // the CTA's warp w takes the 16-token tiles tile0 + w, + stride, ...
  int hi;             // end of the attended positions (of the piece)
  int wlo;            // first attended position (sliding window)
  int pieces;         // pieces of this row (balanced), or 0
  bool valid;
};

// Live range of row r: [wlo, len), cut from base = wlo rounded down to 16.
__device__ __forceinline__ int tiles_of(const DecodeParams& p, int r, int cap, int& len, int& wlo) {
  len = min(max(p.seq_lens[r], 0), cap);
  wlo = p.window >= 0 ? max(0, len - 1 - p.window) : 0;
  return len > 0 ? ((len + 15) >> 4) - (wlo >> 4) : 0;
}

// Balanced pieces.  With t_b the 16-token tiles of row b's live range, S the
// partial slots of a row and P the pieces the grid has room for (one occupancy
// wave of CTAs, or U + half a wave where the U = B * Hkv rows and heads are more
// than that), every row is cut into n_b = clamp(ceil(t_b / L), 1, S) pieces of
// ceil(t_b / n_b) tiles, with the smallest multiple L of W for which the pieces
// number at most P (found by bisection: sum t_b Hkv / P is a lower bound, sum t_b
// Hkv / (P - U) always does).  The grid follows from the arguments alone; CTAs
// past the last piece return.  Item c: rows in order, a row's pieces in order, the
// KV heads of a piece next to each other.
template <int W>
__device__ Mx4Item balanced_piece(const DecodeParams& p, int c) {
  const int lane = threadIdx.x & 31;
  const int B = p.rows, Hkv = p.Hkv, S = p.num_splits;
  const int cap = p.max_blocks * p.bs;
  int len, wlo;
  const int t0 = lane < B ? tiles_of(p, lane, cap, len, wlo) : 0;  // the only rows if B <= 32
  int tot = t0;  // (the host keeps B * cap / 16 within 31 bits)
#pragma unroll 1
  for (int r = 32 + lane; r < B; r += 32) tot += tiles_of(p, r, cap, len, wlo);
  tot = __reduce_add_sync(0xffffffffu, tot);
  const int room = p.bal_pieces / Hkv;  // pieces of one KV head (> B)
  // bisection in units of W tiles (one per warp)
  const int need = (tot + W - 1) / W;
  int lo = max(1, (need + room - 1) / room);
  int up = max(lo, (need + room - B - 1) / (room - B));
  while (lo < up) {
    const int mid = (lo + up) >> 1, len_mid = mid * W;
    int n = lane < B ? min(max((t0 + len_mid - 1) / len_mid, 1), S) : 0;
#pragma unroll 1
    for (int r = 32 + lane; r < B; r += 32)
      n += min(max((tiles_of(p, r, cap, len, wlo) + len_mid - 1) / len_mid, 1), S);
    n = __reduce_add_sync(0xffffffffu, n);
    if (n <= room)
      up = mid;
    else
      lo = mid + 1;
  }
  const int L = lo * W;
  int base = 0;
#pragma unroll 1
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
      const int q = c - base * Hkv;  // item among these rows
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
      it.tile0 = (it.wlo >> 4) + it.slot * per_s;
      it.stride = W;
      // (the last piece's end, rounded up to whole tiles per piece, may be past 2^31 tokens)
      it.hi = it.tile0 + per_s <= len_s >> 4 ? (it.tile0 + per_s) * 16 : len_s;
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

template <int W>
__device__ Mx4Item item_of(const DecodeParams& p, int c) {
  if (p.balanced) return balanced_piece<W>(p, c);
  const int units = p.rows * p.Hkv;
  const int cap = p.max_blocks * p.bs;
  Mx4Item it;
  it.slot = c / units;
  it.unit = c - it.slot * units;
  it.row = it.unit / p.Hkv;
  it.g = it.unit - it.row * p.Hkv;
  int len;
  tiles_of(p, it.row, cap, len, it.wlo);
  const int lo = (it.wlo & ~15) + it.slot * p.chunk;
  it.tile0 = lo >> 4;
  it.stride = W;
  it.hi = min(min(lo + p.chunk, cap), len);
  it.pieces = 0;
  it.valid = true;
  return it;
}

// The row with `rank` rows before it when they are put in the order of falling lengths, to
// about an eighth of the longest (sixteen classes at most; rows of a class by their numbers).  Every
// warp finds it by itself.
__device__ __forceinline__ int row_of_rank(const DecodeParams& p, int rank) {
  constexpr int N = kMx4RankRows / 32;
  const int lane = threadIdx.x & 31, B = p.rows;
  int v[N], top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = lane + 32 * i;
    v[i] = r < B ? min(max(p.seq_lens[r], 0), p.max_blocks * p.bs) : -1;
    top = max(top, v[i]);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const int shift = max(0, 28 - __clz(top));  // the longest is in class 8 to 15
  int cls = 0, before = 0;
#pragma unroll
  for (int bit = 8; bit > 0; bit >>= 1) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += (v[i] >> shift) >= cls + bit;
    n = __reduce_add_sync(0xffffffffu, n);
    if (n > rank)
      cls += bit;
    else
      before = n;
  }
  int k = rank - before, row = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool in = (v[i] >> shift) == cls;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    const unsigned it = __ballot_sync(0xffffffffu, in && __popc(m & ((1u << lane) - 1u)) == k);
    if (it != 0u) row = 32 * i + __ffs(it) - 1;
    k -= __popc(m);
  }
  return row;
}

// Shape of the kernel for head dimension D, NT groups of 8 query heads and W warps.
template <int D, int NT, int W>
struct Mx4Tile {
  static constexpr int kRec = 18 * D;                    // bytes of a 16-token record
  static constexpr int kSub = D <= 128 ? 2 : 1;          // records per stage
  static constexpr int kStages = 2 * (3 - kSub);         // ring depth per warp: 4 records
  static constexpr int kStageBytes = kSub * kRec;
  static constexpr int kRing = kStages * kStageBytes;    // a multiple of 128
  static constexpr int kRow = D + 4;                     // floats of a merged row (padded)
  static constexpr int kMerge = 8 * NT * kRow * 4;       // a warp's rows, in its ring
  static constexpr int kBars = W * kRing;                // mbarriers [warps][stages]
  static constexpr int kMasks = kBars + W * kStages * 8;      // [warps][stages][sub]
  static constexpr int kScal = kMasks + W * kStages * kSub * 4;  // [2][warps][16]
  static constexpr int kQRow = D + 8;                    // halves of a staged query row (padded)
  static constexpr int kQ = kScal + 2 * W * 16 * 4;           // [8 NT][kQRow] fp16
  static constexpr int kQLo = kQ + 8 * NT * kQRow * 2;             // the rest below fp16, likewise
  static constexpr int kInv = kQLo + 8 * NT * kQRow * 2;           // [16] score factors
  static constexpr int kVs = kInv + 16 * 4;              // [D] value scales
  static constexpr int kSink = kVs + D * 4;              // [16] sink logits
  static constexpr int kJoin = kSink + 16 * 4;           // [2][16] base and sum of the CTA (cluster)
  static constexpr int kSmem = kJoin + 2 * 16 * 4;
  // resident CTAs per SM the registers are cut for
  static constexpr int kWarpsPerSm = D * NT >= 512 ? 8 : D * NT >= 256 ? 12 : D * NT >= 128 ? 16 : 20;
  static constexpr int kBlocks = kWarpsPerSm / W;
  static_assert(kMerge <= kRing, "the merge fits the ring");
};

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Both halves of a times one half of b.
__device__ __forceinline__ uint32_t hmul2_half(uint32_t a, uint32_t b, bool high) {
  const __half2 s = *reinterpret_cast<const __half2*>(&b);
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), high ? __high2half2(s) : __low2half2(s));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The values of the two float8 e4m3fn bytes in bits 0 .. 15, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(r) : "r"(w));
  return r;
}

template <int N>  // 4 N bytes
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(w[0]) : "r"(addr));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(addr + 4 * i));
  }
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];\n" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1];\n" : "=r"(v) : "r"(addr));
  return v;
}

constexpr float kUnset = -3.0e38f;  // exponent base of a warp that attended nothing
constexpr float kHead = 15.f;       // log2 of the largest probability the fp16 tile takes
constexpr float kRoom = 8.f;        // log2 of the largest one right after the base is set

// (out of line: block sizes that are no power of two)
static __device__ __noinline__ int quotient(int a, int b) { return a / b; }

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;\n" ::: "memory");
}
// Shared-memory address of `addr` in CTA `rank` of the cluster, and loads from it.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// How the scales come in.  kPlain: one per tensor, applied to the scores.  Per channel they are
// folded into the queries, which then take two fp16 numbers each (22 bits: rounding them to
// one would move the scores by as much as all else together): with at most 4 heads the
// second numbers are the idle columns 4 .. 7 of the product and are added with a shuffle
// (kColumns), else they take products of their own (kProducts).
enum Fold { kPlain = 0, kProducts = 1, kColumns = 2 };

// Resident CTAs per SM the registers are cut for.  The separate products of two head groups
// at head_dim 128 spill at three (16 x 16000 tokens, 64/4 heads: 72 us; 56 at two).
template <int D, int NT, int W, Fold FOLD>
constexpr int mx4_blocks() {
  return FOLD == kProducts && NT == 2 && D == 128 && W == 4 ? 2 : Mx4Tile<D, NT, W>::kBlocks;
}

// W warps.  In a cluster the p.num_splits CTAs share one (row, KV head), its tiles
// dealt to their warps in turn, and join through distributed shared memory.
template <int D, int NT, int W, Mx4Way WAY, Fold FOLD>
__global__ void __launch_bounds__(32 * W, (mx4_blocks<D, NT, W, FOLD>()))
mx4_decode_kernel(const DecodeParams p) {
  using T = Mx4Tile<D, NT, W>;
  constexpr bool ROW = WAY != Mx4Way::kPieces;  // (the length is all that the item follows from)
  constexpr bool CLUSTER = WAY == Mx4Way::kCluster;
  constexpr int kThreads = 32 * W;
  constexpr int KC = D / 16;   // MMA steps of QK^T, and 16-channel tiles of PV
  constexpr int KW = D / 32;   // 32-bit words of a lane's key channels (D / 4 of a token)
  constexpr int VW = D / 64;   // and of its value channels (D / 8 of a token)
  extern __shared__ __align__(128) uint8_t smem[];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = lane >> 2, tig = lane & 3;
  int G = p.G, h0 = 0;  // the query heads h0 .. h0 + G - 1 of the group are this CTA's
  const int rpb = p.bs >> 4;  // records per block
  auto block_of = [&](int tile) { return p.bs_log2 >= 4 ? tile >> (p.bs_log2 - 4) : quotient(tile, rpb); };
  Mx4Item it;
  if constexpr (ROW) {
    const int ctas = CLUSTER ? p.num_splits : 1;  // of a row and head
    it.unit = blockIdx.x / ctas;
    it.slot = blockIdx.x - it.unit * ctas;
    if (p.head_groups == 2) {
      const int half = (p.G + 1) >> 1;
      h0 = it.unit & 1 ? half : 0;
      G = it.unit & 1 ? p.G - half : half;
      it.unit >>= 1;
    }
    it.row = it.unit / p.Hkv;
    it.g = it.unit - it.row * p.Hkv;
    if (!CLUSTER && p.longest_first) {
      it.row = row_of_rank(p, it.row);
      it.unit = it.row * p.Hkv + it.g;
    }
    it.stride = W * ctas;
    it.tile0 = it.slot * W;
    it.pieces = 0;
  } else {
    it = item_of<W>(p, blockIdx.x);
    if (!it.valid) return;
  }
  const int* table = p.block_table + (long long)it.row * p.max_blocks;
  // The table entry of tile j of the warp (tile0 + warp + stride j): within the table, whatever
  // the live length is.
  auto entry = [&](int j) -> int {
    const int b = block_of(it.tile0 + warp + it.stride * j);
    return b < p.max_blocks ? __ldg(table + b) : -1;
  };
  int e0 = -1, e1 = -1;  // entries of the warp's tiles lane and 32 + lane
  const int live = ROW || (it.slot == 0 && it.g == 0) ? p.seq_lens[it.row] : 0;
  if constexpr (ROW) {
    if (p.window < 0) {  // on their way with the length
      e0 = entry(lane);
      e1 = entry(32 + lane);
    }
  }
  // the queries, key and value scales and sinks, on their way too
  constexpr int QN = (D * NT + kThreads - 1) / kThreads;
  uint4 q_raw[QN];
  float4 ks_raw[QN][2];
#pragma unroll
  for (int i = 0; i < QN; ++i) {
    const int e = threadIdx.x + i * kThreads;
    const int h = e / (D / 8), d = 8 * (e % (D / 8));
    q_raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (e < D * NT && h < G)
      q_raw[i] = *reinterpret_cast<const uint4*>(static_cast<const __half*>(p.q) +
                                                 ((long long)it.row * p.Hq + it.g * p.G + h0 + h) * D + d);
    if (FOLD != kPlain && e < D * NT) {
      ks_raw[i][0] = *reinterpret_cast<const float4*>(p.k_scale + it.g * D + d);
      ks_raw[i][1] = *reinterpret_cast<const float4*>(p.k_scale + it.g * D + d + 4);
    }
  }
  float4 vs_raw;
  if (threadIdx.x < D / 4) {
    if constexpr (FOLD != kPlain)
      vs_raw = *reinterpret_cast<const float4*>(p.v_scale + it.g * D + 4 * threadIdx.x);
    else
      vs_raw.x = vs_raw.y = vs_raw.z = vs_raw.w = p.v_scale[0];
  }
  float sink_raw = 0.f;
  if (p.sink != nullptr && threadIdx.x < G) sink_raw = p.sink[it.g * p.G + h0 + threadIdx.x];

  if constexpr (ROW) {
    it.hi = min(max(live, 0), p.max_blocks * p.bs);
    it.wlo = p.window >= 0 ? max(0, it.hi - 1 - p.window) : 0;
    it.tile0 += it.wlo >> 4;
  }
  if (it.slot == 0 && threadIdx.x == 0 && it.g == 0 && (live < 0 || live > p.max_blocks * p.bs))
    flag_or(p.flags, I8KV_FLAG_LEN_CLAMPED);

  // ---- the warp's records: lane j % 32 knows where tile j's is and copies it in ----
  const int first = it.tile0 + warp;
  const int end = (it.hi + 15) >> 4;
  const int mine = end > first ? (end - first + it.stride - 1) / it.stride : 0;
  const int stages = (mine + T::kSub - 1) / T::kSub;
  if (!ROW || p.window >= 0) {
    if (lane < mine) e0 = entry(lane);
    if (32 + lane < mine) e1 = entry(32 + lane);
  }
  const uint8_t* cache = static_cast<const uint8_t*>(p.k);
  // what a lane copies: the record of its tile (nullptr: none) and the attended tokens of it
  const uint8_t* rec_at = nullptr;
  int rec_mask = 0;
  auto place = [&](int j, int blk) {
    rec_at = nullptr;
    rec_mask = 0;
    if (j >= mine) return;
    if (blk < 0 || (long long)blk >= p.cache_rows) {
      flag_or(p.flags, I8KV_FLAG_BAD_BLOCK);
      return;
    }
    const int tile = first + it.stride * j, pos = 16 * tile;
    rec_mask = it.hi - pos >= 16 ? 0xFFFF : (1 << (it.hi - pos)) - 1;
    if (pos < it.wlo) rec_mask &= 0xFFFF << (it.wlo - pos);
    rec_at = cache + (((long long)blk * p.Hkv + it.g) * rpb + (tile - block_of(tile) * rpb)) * T::kRec;
  };
  const uint32_t ring = smem_addr(smem + warp * T::kRing);
  const uint32_t bars = smem_addr(smem + T::kBars) + warp * T::kStages * 8;
  int* masks = reinterpret_cast<int*>(smem + T::kMasks) + warp * T::kStages * T::kSub;
  place(lane, e0);
  auto issue = [&](int k, int st) {  // stage k into slot st of the ring
    const int j0 = k * T::kSub;
    if (j0 > 0 && (j0 & 31) == 0) {
      place(j0 + lane, e1);
      e1 = j0 + 32 + lane < mine ? entry(j0 + 32 + lane) : -1;
    }
    const unsigned s = lane - (j0 & 31);
    if (s < T::kSub) {
      const uint32_t bar = bars + st * 8;
      masks[st * T::kSub + s] = rec_mask;  // (before the arrival that publishes it)
      if (rec_at != nullptr) {
        tc::mbar_arrive_expect_tx(bar, T::kRec);
        tc::bulk_g2s(ring + st * T::kStageBytes + s * T::kRec, rec_at, T::kRec, bar);
      } else {
        tc::mbar_arrive(bar);
      }
    }
  };
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < T::kStages; ++i) tc::mbar_init(bars + 8 * i, T::kSub);
    tc::fence_mbar_init();
  }
  __syncwarp();
#pragma unroll 1
  for (int k = 0; k < min(T::kStages, stages); ++k) issue(k, k);

  // slots that no piece fills: empty
  if (it.pieces > 0 && it.slot == 0) {
#pragma unroll 1
    for (int e = threadIdx.x; e < (p.num_splits - it.pieces) * G; e += kThreads) {
      const long long b = ((long long)it.unit * p.num_splits + it.pieces) * G + e;
      p.ws_m[b] = neg_inf();
      p.ws_l[b] = 0.f;
    }
  }

  // ---- the group's queries, scales folded in, staged in shared memory: 8 channels of a head
  // per thread and pass ----
  __half* sq = reinterpret_cast<__half*>(smem + T::kQ);
  float* sinv = reinterpret_cast<float*>(smem + T::kInv);
  float* svs = reinterpret_cast<float*>(smem + T::kVs);
  float* ssink = reinterpret_cast<float*>(smem + T::kSink);
#pragma unroll
  for (int i = 0; i < QN; ++i) {
    const int e = threadIdx.x + i * kThreads;
    if (e >= D * NT) break;  // (whole warps: D NT is a multiple of 32)
    const int h = e / (D / 8), d = 8 * (e % (D / 8));
    uint4 v = q_raw[i];
    float inv = 1.f;
    if constexpr (FOLD != kPlain) {
      // one power of two per head taken out, so that the largest element is in
      // [2^8, 2^9): nothing overflows fp16, and what the second number loses below fp16's
      // smallest step is less than 2^-32 of the largest
      const float4 k0 = ks_raw[i][0], k1 = ks_raw[i][1];
      const __half2* q2 = reinterpret_cast<const __half2*>(&v);
      const float2 a0 = __half22float2(q2[0]), a1 = __half22float2(q2[1]);
      const float2 a2 = __half22float2(q2[2]), a3 = __half22float2(q2[3]);
      const float x[8] = {a0.x * k0.x, a0.y * k0.y, a1.x * k0.z, a1.y * k0.w,
                          a2.x * k1.x, a2.y * k1.y, a3.x * k1.z, a3.y * k1.w};
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(x[k]));
#pragma unroll
      for (int o = 1; o < D / 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int ex = __float_as_int(amax) >> 23;  // biased exponent (amax >= 0)
      const bool scaled = ex >= 9 && ex < 255;
      const float up = scaled ? __int_as_float((262 - ex) << 23) : 1.f;
      inv = scaled ? __int_as_float((ex - 8) << 23) : 1.f;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float y0 = x[2 * k] * up, y1 = x[2 * k + 1] * up;
        hi[k] = pack_h2(y0, y1);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi[k]));
        lo[k] = pack_h2(y0 - f.x, y1 - f.y);
      }
      v = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      const uint4 rest = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      if constexpr (FOLD == kColumns) {
        if (h >= 4) continue;  // (the first four heads' threads fill these)
        *reinterpret_cast<uint4*>(sq + (h + 4) * T::kQRow + d) = rest;
        if (d == 0) sinv[h + 4] = inv * (p.softcap > 0.f ? p.sigma : p.sigma * kLog2e);
      } else {
        *reinterpret_cast<uint4*>(reinterpret_cast<__half*>(smem + T::kQLo) + h * T::kQRow + d) = rest;
      }
    } else {
      inv = p.k_scale[0];
      // an infinity becomes a NaN (as the second numbers make it above): its scores could all be
      // -inf, which is no sum at all
      __half2* q2 = reinterpret_cast<__half2*>(&v);
#pragma unroll
      for (int k = 0; k < 4; ++k) q2[k] = __hadd2(q2[k], __hsub2(q2[k], q2[k]));
    }
    *reinterpret_cast<uint4*>(sq + h * T::kQRow + d) = v;
    // accumulator -> score in log2 units (natural units with a softcap)
    if (d == 0) sinv[h] = inv * (p.softcap > 0.f ? p.sigma : p.sigma * kLog2e);
  }
  if (threadIdx.x < D / 4) *reinterpret_cast<float4*>(svs + 4 * threadIdx.x) = vs_raw;
  if (threadIdx.x < 16) ssink[threadIdx.x] = sink_raw;
  __syncthreads();
  // B operand of step i: channels 4i, 4i+1 and 4i+2, 4i+3 of the lane's part, which starts
  // at channel tig D/4 of head grp (+ 8); the lane's score columns are heads 2 tig, 2 tig + 1
  uint32_t qf[NT][KC][2];
  float fac[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const uint4* src = reinterpret_cast<const uint4*>(sq + (grp + 8 * nt) * T::kQRow + tig * (D / 4));
#pragma unroll
    for (int i = 0; i < KC / 2; ++i) {
      const uint4 v = src[i];
      qf[nt][2 * i][0] = v.x;
      qf[nt][2 * i][1] = v.y;
      qf[nt][2 * i + 1][0] = v.z;
      qf[nt][2 * i + 1][1] = v.w;
    }
    fac[nt][0] = sinv[8 * nt + 2 * tig];
    fac[nt][1] = sinv[8 * nt + 2 * tig + 1];
  }

  const uint32_t q_lo = smem_addr(smem + T::kQLo) + (grp * T::kQRow + tig * (D / 4)) * 2;

  float acc[KC][NT][4];
  float base[NT][2], lrun[NT][2];
#pragma unroll
  for (int t = 0; t < KC; ++t)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][nt][e] = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      base[nt][j] = 0.f;
      lrun[nt][j] = 0.f;
    }
  // score row r of a tile (0..7; +8 below) is token (r >> 1) + 4 (r & 1), so that a lane's
  // contraction indices 2tig, 2tig+1, 2tig+8, 2tig+9 in PV are tokens tig + 0, 4, 8, 12
  const int tok = (grp >> 1) + 4 * (grp & 1);
  const uint32_t k_off = tok * (D / 2) + tig * (D / 8);
  const uint32_t ks_off = 8 * D + tok * (D / 16) + tig * (D / 64);
  const uint32_t v_off = 9 * D + tig * (D / 2) + grp * (D / 16);
  const uint32_t vs_off = 17 * D + tig * (D / 16) + (grp * D) / 128;
  const float cap_k = 2.f * kLog2e / p.softcap;  // used only when softcap > 0
  bool unset = true;  // no score yet: the bases are not set
  bool timeout = false;

  // The first N records of stage k; false if they did not arrive.
  auto work = [&](auto records, int k) -> bool {
    constexpr int N = decltype(records)::value;
    const int st = k % T::kStages;
    const bool ok = tc::mbar_wait(bars + st * 8, (k / T::kStages) & 1);
    if (!__all_sync(0xffffffffu, ok)) return false;
    const uint32_t rec0 = ring + st * T::kStageBytes;

    // ---- S = K Q'^T, one 16-token tile at a time ----
    float sc[N][NT][4];
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const uint32_t r = rec0 + s * T::kRec;
      float rest[NT][4];  // of the queries' second numbers (a chain of their own, where registers allow)
      uint32_t wa[KW], wb[KW];
      lds<KW>(r + k_off, wa);
      lds<KW>(r + k_off + 8 * (D / 2), wb);
      // block scales of the lane's channels (D / 64 of a token), each as an fp16 pair
      // (two to a register: the products take the half they need of it)
      constexpr int KB = D / 64, KP = (KB + 1) / 2;
      uint32_t fa[KP], fb[KP];
      if constexpr (D == 64) {
        fa[0] = e4m3x2_to_h2(lds_u8(r + ks_off));
        fb[0] = e4m3x2_to_h2(lds_u8(r + ks_off + 8 * (D / 16)));
      } else if constexpr (D == 128) {
        fa[0] = e4m3x2_to_h2(lds_u16(r + ks_off));
        fb[0] = e4m3x2_to_h2(lds_u16(r + ks_off + 8 * (D / 16)));
      } else {
        uint32_t x[1];
        lds<1>(r + ks_off, x);
        e4m3x4_to_h2x2(x[0], fa[0], fa[1]);
        lds<1>(r + ks_off + 8 * (D / 16), x);
        e4m3x4_to_h2x2(x[0], fb[0], fb[1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[s][nt][e] = rest[nt][e] = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {  // 8 channels of a lane: two steps
        uint32_t a[4], b[4];
        e2m1x8_to_h2x4(wa[w], a[0], a[1], a[2], a[3]);
        e2m1x8_to_h2x4(wb[w], b[0], b[1], b[2], b[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = hmul2_half(a[i], fa[w / 4], (w / 2) % 2);
          b[i] = hmul2_half(b[i], fb[w / 4], (w / 2) % 2);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(sc[s][nt], a[0], b[0], a[1], b[1], qf[nt][2 * w][0], qf[nt][2 * w][1]);
          mma16816(sc[s][nt], a[2], b[2], a[3], b[3], qf[nt][2 * w + 1][0], qf[nt][2 * w + 1][1]);
          if constexpr (FOLD == kProducts) {
            uint32_t l[4];
            lds<4>(q_lo + nt * 8 * T::kQRow * 2 + 16 * w, l);
            float(&to)[4] = NT == 1 ? rest[nt] : sc[s][nt];
            mma16816(to, a[0], b[0], a[1], b[1], l[0], l[1]);
            mma16816(to, a[2], b[2], a[3], b[3], l[2], l[3]);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (FOLD == kProducts && NT == 1) sc[s][nt][e] += rest[nt][e];
          // (both columns of a head then hold its score; only the first is read in the end)
          if constexpr (FOLD == kColumns) sc[s][nt][e] += __shfl_xor_sync(0xffffffffu, sc[s][nt][e], 2);
        }
    }

    // ---- online softmax: the exponent base of a head moves only when a score leaves the
    // range that the fp16 probabilities cover ----
    int mask[N], all = 0xFFFF, live_any = 0;
#pragma unroll
    for (int s = 0; s < N; ++s) {
      mask[s] = masks[st * T::kSub + s];
      all &= mask[s];
      live_any |= mask[s];
    }
    const bool partial = all != 0xFFFF, any_live = live_any != 0;  // uniform
    // z: scores less the head's base, in log2 units
    float z[N][NT][4];
    auto scores_less_base = [&]() {
      if (p.softcap > 0.f) {
#pragma unroll
        for (int s = 0; s < N; ++s)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              z[s][nt][e] = fmaf(soft_cap(sc[s][nt][e] * fac[nt][e & 1], p.softcap, cap_k), kLog2e,
                                 -base[nt][e & 1]);
      } else {
#pragma unroll
        for (int s = 0; s < N; ++s)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              z[s][nt][e] = fmaf(sc[s][nt][e], fac[nt][e & 1], -base[nt][e & 1]);
      }
      if (partial) {
#pragma unroll
        for (int s = 0; s < N; ++s) {
          const bool upper = (mask[s] >> tok) & 1, lower = (mask[s] >> (tok + 8)) & 1;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (!upper) z[s][nt][0] = z[s][nt][1] = neg_inf();
            if (!lower) z[s][nt][2] = z[s][nt][3] = neg_inf();
          }
        }
      }
    };
    scores_less_base();
    float top = neg_inf();
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, z[s][nt][e]);
    if (unset || __any_sync(0xffffffffu, top > kHead)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float alpha[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float mx = neg_inf();
#pragma unroll
          for (int s = 0; s < N; ++s) mx = fmaxf(mx, fmaxf(z[s][nt][j], z[s][nt][2 + j]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          // up by what the largest is above the room left; down too on the first scores (a
          // head of NaNs, which has no largest, keeps a finite base and a NaN sum)
          const float up = unset ? (mx > neg_inf() ? mx - kRoom : 0.f) : fmaxf(mx - kRoom, 0.f);
          alpha[j] = unset ? 1.f : fast_exp2(-up);
          base[nt][j] += up;
        }
        lrun[nt][0] *= alpha[0];
        lrun[nt][1] *= alpha[1];
#pragma unroll
        for (int t = 0; t < KC; ++t) {
          acc[t][nt][0] *= alpha[0];
          acc[t][nt][2] *= alpha[0];
          acc[t][nt][1] *= alpha[1];
          acc[t][nt][3] *= alpha[1];
        }
      }
      unset = unset && !any_live;
      scores_less_base();
      // (a score so large that its own rounding exceeds the room still fits fp16)
#pragma unroll
      for (int s = 0; s < N; ++s)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (z[s][nt][e] > kHead) z[s][nt][e] = kHead;
    }
    uint32_t ph[N][NT][2];
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pr[e] = fast_exp2(z[s][nt][e]);
          lrun[nt][e & 1] += pr[e];
        }
        ph[s][nt][0] = movm_t(pack_h2(pr[0], pr[1]));
        ph[s][nt][1] = movm_t(pack_h2(pr[2], pr[3]));
      }

    // ---- O^T += V^T P^T: rows are the channels of group grp, D / 8 from grp D / 8 ----
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const uint32_t r = rec0 + s * T::kRec;
      uint32_t v[4][VW];  // tokens tig, tig + 4, tig + 8, tig + 12
      uint32_t x[4];      // their block scales
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lds<VW>(r + v_off + i * 4 * (D / 2), v[i]);
        if constexpr (D == 256) {
          x[i] = lds_u16(r + vs_off + i * 4 * (D / 16));
        } else {
          x[i] = lds_u8(r + vs_off + i * 4 * (D / 16));
        }
      }
      if (partial) {  // a token that is not attended: nothing of its bytes counts
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((mask[s] >> (tig + 4 * i)) & 1)) x[i] = 0u;
      }
      // scales of token pairs (0, 1) and (2, 3) for each block of the lane's channels
      uint32_t s01[2], s23[2];
      if constexpr (D == 256) {
        e4m3x4_to_h2x2(prmt(x[0], x[1], 0x5140u), s01[0], s01[1]);
        e4m3x4_to_h2x2(prmt(x[2], x[3], 0x5140u), s23[0], s23[1]);
      } else {
        s01[0] = e4m3x2_to_h2(prmt(x[0], x[1], 0x0040u));
        s23[0] = e4m3x2_to_h2(prmt(x[2], x[3], 0x0040u));
      }
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        const int blk = w / 2;
        // nibble pairs (token 0, token 1) of the even and of the odd channels
        uint32_t e01[4], o01[4], e23[4], o23[4];
        e2m1x8_to_h2x4((v[0][w] & 0x0F0F0F0Fu) | ((v[1][w] << 4) & 0xF0F0F0F0u), e01[0], e01[1], e01[2], e01[3]);
        e2m1x8_to_h2x4(((v[0][w] >> 4) & 0x0F0F0F0Fu) | (v[1][w] & 0xF0F0F0F0u), o01[0], o01[1], o01[2], o01[3]);
        e2m1x8_to_h2x4((v[2][w] & 0x0F0F0F0Fu) | ((v[3][w] << 4) & 0xF0F0F0F0u), e23[0], e23[1], e23[2], e23[3]);
        e2m1x8_to_h2x4(((v[2][w] >> 4) & 0x0F0F0F0Fu) | (v[3][w] & 0xF0F0F0F0u), o23[0], o23[1], o23[2], o23[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = hmul2(e01[i], s01[blk]), a1 = hmul2(o01[i], s01[blk]);
          const uint32_t a2 = hmul2(e23[i], s23[blk]), a3 = hmul2(o23[i], s23[blk]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(acc[4 * w + i][nt], a0, a1, a2, a3, ph[s][nt][0], ph[s][nt][1]);
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    if (k + T::kStages < stages) issue(k + T::kStages, st);
    return true;
  };
  const int full = mine / T::kSub;  // stages of kSub records; an odd record at the end is worked alone
  int k = 0;
#pragma unroll 1
  for (; k < full; ++k) {
    if (!work(std::integral_constant<int, T::kSub>{}, k)) {
      timeout = true;
      break;
    }
  }
  if constexpr (T::kSub > 1) {
    if (!timeout && k < stages) timeout = !work(std::integral_constant<int, 1>{}, k);
  }
  if (timeout) {
    // the copies still in flight must not land in memory that others use
    if (lane == 0) flag_or(p.flags, I8KV_FLAG_WAIT_TIMEOUT);
    for (int i = k; i < min(k + T::kStages, stages); ++i)
      tc::mbar_wait(bars + (i % T::kStages) * 8, (i / T::kStages) & 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) lrun[nt][0] = lrun[nt][1] = __int_as_float(0x7fc00000);
  }

  // ---- merge the warps: rows [head][channel] in each warp's ring, then one sum ----
  float* bw = reinterpret_cast<float*>(smem + T::kScal);  // [warps][16] exponent bases
  float* lw = bw + W * 16;                           // [warps][16] sums
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float l = lrun[nt][j];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const int h = nt * 8 + 2 * tig + j;
      if (grp == 0) {
        bw[warp * 16 + h] = unset ? kUnset : base[nt][j];
        lw[warp * 16 + h] = l;
      }
      if (h < G) {
        float* row = reinterpret_cast<float*>(smem + warp * T::kRing) + h * T::kRow + grp * (D / 8);
#pragma unroll
        for (int t = 0; t < KC; t += 2)
          *reinterpret_cast<float4*>(row + 2 * t) =
              make_float4(acc[t][nt][j], acc[t][nt][2 + j], acc[t + 1][nt][j], acc[t + 1][nt][2 + j]);
      }
    }
  // The kernel that follows in the stream (the join, or in the other ways whatever comes next) may be
  // launched now; its CTAs wait for this grid's end before they touch memory.  Graphs of calls,
  // without / with it: one context of 300 tokens 4.47 / 4.32 us, 16 x 2600 8.82 / 8.59,
  // one of 32768 17.1 / 16.7, 16 x 512-8192 24.4 / 24.3.
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  __syncthreads();
  const long long head0 = (long long)it.row * p.Hq + it.g * p.G + h0;
  // the normalised output of 4 channels of head h, or zeros without a score
  auto finish = [&](int h, int d, float4 o, float M, float L) {
    const bool some = !(L <= 0.f);  // (a NaN sum is not an empty one)
    const float m = M * (1.f / kLog2e);
    uint2 v = make_uint2(0u, 0u);
    if (some) {
      float scale = 1.f / L;
      if (p.sink != nullptr) scale *= 1.f / (1.f + expf(ssink[h] - (m + logf(L))));
      const float4 vs = *reinterpret_cast<const float4*>(svs + d);
      v = make_uint2(pack_h2(o.x * scale * vs.x, o.y * scale * vs.y),
                     pack_h2(o.z * scale * vs.z, o.w * scale * vs.w));
    }
    *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + (head0 + h) * D + d) = v;
    if (d == 0 && p.lse != nullptr) p.lse[head0 + h] = some ? m + logf(L) : neg_inf();
  };
  float* jm = reinterpret_cast<float*>(smem + T::kJoin);  // [16] base, [16] sum
#pragma unroll 1
  for (int e = threadIdx.x; e < G * (D / 4); e += kThreads) {
    const int h = e / (D / 4), d = 4 * (e - h * (D / 4));
    float M = bw[h];
#pragma unroll
    for (int w = 1; w < W; ++w) M = fmaxf(M, bw[w * 16 + h]);
    float L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = fast_exp2(bw[w * 16 + h] - M);
      const float4 x = *reinterpret_cast<const float4*>(
          reinterpret_cast<const float*>(smem + w * T::kRing) + h * T::kRow + d);
      L += f * lw[w * 16 + h];
      o.x += f * x.x;
      o.y += f * x.y;
      o.z += f * x.z;
      o.w += f * x.w;
    }
    if constexpr (WAY == Mx4Way::kRows) {
      finish(h, d, o, M, L);
    } else if constexpr (CLUSTER) {
      // the CTA's sum, in the place of its first warp's (which no other thread reads)
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(smem) + h * T::kRow + d) = o;
      if (d == 0) {
        jm[h] = M;
        jm[16 + h] = L;
      }
    } else {
      const bool some = !(L <= 0.f);
      const long long part = ((long long)it.unit * p.num_splits + it.slot) * G + h;
      const float4 vs = *reinterpret_cast<const float4*>(svs + d);
      if (some)
        *reinterpret_cast<float4*>(p.ws_acc + part * D + d) =
            make_float4(o.x * vs.x, o.y * vs.y, o.z * vs.z, o.w * vs.w);
      if (d == 0) {
        p.ws_m[part] = some ? M * (1.f / kLog2e) : neg_inf();
        p.ws_l[part] = some ? L : 0.f;
      }
    }
  }
  if constexpr (CLUSTER) {
    cluster_sync();  // every CTA's sum is there
    const int C = p.num_splits;
    const uint32_t rows = smem_addr(smem), join = smem_addr(smem + T::kJoin);
#pragma unroll 1
    for (int e = it.slot * kThreads + threadIdx.x; e < G * (D / 4); e += C * kThreads) {
      const int h = e / (D / 4), d = 4 * (e - h * (D / 4));
      float m[8], l[8], M = kUnset, L = 0.f;
      float4 x[8], o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r < C) {
          m[r] = ld_cluster(in_cta(join + 4 * h, r));
          l[r] = ld_cluster(in_cta(join + 64 + 4 * h, r));
          x[r] = ld_cluster4(in_cta(rows + 4 * (h * T::kRow + d), r));
        }
      }
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < C) M = fmaxf(M, m[r]);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r < C) {
          const float f = fast_exp2(m[r] - M);
          L += f * l[r];
          o.x += f * x[r].x;
          o.y += f * x[r].y;
          o.z += f * x[r].z;
          o.w += f * x[r].w;
        }
      }
      finish(h, d, o, M, L);
    }
    cluster_sync();  // nobody leaves while others read its sums
  }
}

template <int D, int NT, int W, Mx4Way WAY, Fold FOLD>
cudaError_t run_mx4_with(const DecodeParams& p, cudaStream_t s, KernelInfo* info) {
  using T = Mx4Tile<D, NT, W>;
  auto kern = mx4_decode_kernel<D, NT, W, WAY, FOLD>;
  // the opt-in shared-memory size is a per-function attribute: set it once per device
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(done.load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit);
  }
  if (info != nullptr) {
    info->round = 16 * W;
    if constexpr (WAY == Mx4Way::kCluster) {
      // clusters live inside a part of the GPU: fewer fit than the CTAs alone
      for (int i = 1; i < 4; ++i) {
        cudaLaunchConfig_t c = {};
        c.gridDim = dim3(1024u << i);
        c.blockDim = dim3(32 * W);
        c.dynamicSmemBytes = T::kSmem;
        cudaLaunchAttribute a;
        a.id = cudaLaunchAttributeClusterDimension;
        a.val.clusterDim.x = 1u << i;
        a.val.clusterDim.y = a.val.clusterDim.z = 1;
        c.attrs = &a;
        c.numAttrs = 1;
        if ((e = cudaOccupancyMaxActiveClusters(&info->clusters[i], kern, &c)) != cudaSuccess) return e;
      }
    }
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&info->occupancy, kern, 32 * W, T::kSmem);
  }
  constexpr bool PIECES = WAY == Mx4Way::kPieces;
  const long long units = (long long)p.rows * p.Hkv * (!PIECES && p.head_groups == 2 ? 2 : 1);
  long long ctas = units * (WAY == Mx4Way::kRows ? 1 : p.num_splits);
  if (PIECES && p.balanced && ctas > p.bal_pieces) ctas = p.bal_pieces;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = T::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if constexpr (WAY == Mx4Way::kCluster) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.num_splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int D, int NT, int W, Mx4Way WAY>
cudaError_t run_mx4(const DecodeParams& p, cudaStream_t s, KernelInfo* info) {
  if (!p.per_channel) return run_mx4_with<D, NT, W, WAY, kPlain>(p, s, info);
  if constexpr (NT == 1) {
    if (p.G <= 4)  // (groups that run in halves have 9 heads at least, one half 5)
      return run_mx4_with<D, NT, W, WAY, kColumns>(p, s, info);
  }
  return run_mx4_with<D, NT, W, WAY, kProducts>(p, s, info);
}

template <int W, Mx4Way WAY>
cudaError_t dispatch_mx4(const KernelKey& key, const DecodeParams& p, cudaStream_t s,
                         KernelInfo* info) {
  switch (key.D * 10 + key.nt) {
    case 641: return run_mx4<64, 1, W, WAY>(p, s, info);
    case 642: return run_mx4<64, 2, W, WAY>(p, s, info);
    case 1281: return run_mx4<128, 1, W, WAY>(p, s, info);
    case 1282: return run_mx4<128, 2, W, WAY>(p, s, info);
    case 2561: return run_mx4<256, 1, W, WAY>(p, s, info);
    case 2562: return run_mx4<256, 2, W, WAY>(p, s, info);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

}  // namespace i8kv
