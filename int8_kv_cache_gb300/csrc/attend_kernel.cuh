// Dense causal attention of new tokens on the tensor cores (tcgen05): a packed batch of whole
// prompts (packed_prefill), or chunks of new tokens over a paged cache (paged_prefill).
//
// What it computes, for token i of a sequence's n new ones, at position p = L - n + i of its L
// tokens, and query head h (KV head g = h / G):
//   s_t = sigma dot(Q[i, h], K[t, g]), capped to c tanh(s_t / c) where a cap is given,
//   O[i, h] = sum_t e^(s_t - m) V[t, g] / sum_t e^(s_t - m),  t in [max(0, p - window), p],
// then lse = m + ln sum and the sink.  A row that attends nothing gives 0 and lse = -inf.
//
// Design: a tile is 128 (token, head) vectors of one KV head -- the G heads of a token share its
// keys and values, so a tile spans 128 / G tokens -- and walks its range of the sequence in blocks
// of 128 positions with a running maximum and sum:
//   S[128 x 128] = Q K^T          tcgen05 kind::f16, both operands from shared memory
//   P = 2^(s - base) as fp16, over the scores' columns in tensor memory
//   O[128 x D] += P V             tcgen05 kind::f16, P from tensor memory
// The base of the exponentials follows the running maximum lazily: it moves once the maximum has
// outgrown it by kLazy powers of two, so O is rescaled on few blocks; P carries 2^kShift, so that
// probabilities down to 2^-22 of the base keep the 11 bits of fp16 (they are rounded to it once; sums are fp32).
//
// Two forms.  TILES = 2 (head_dim 64 and 128): a CTA owns two tiles; while the softmax of one
// works, the tensor cores work on the other.  One thread per vector.  TILES = 1 (few vectors, and
// head_dim 256, whose O fills tensor memory): one tile, scores double-buffered, two threads per
// vector (64 positions each), which exchange their maxima through shared memory.
//
// A CTA stays for item after item (an item: a tile's, or two tiles', walk over the blocks of one KV
// head), and every role goes on to the next by itself: its queries are staged and its first scores
// made while the one before is still written out.  152 prompts of 64 tokens, 32 / 8 heads: 59 us.
//
// Warp roles (512 threads, registers dealt out anew with setmaxnreg):
//   warps 0-7    softmax and epilogue
//   warps 8-11   queries into shared memory; then, fp16 sources: look at the V blocks that some row
//                attends in part, where a NaN or infinity that is masked for a row must not reach it
//                through 0 * NaN: such values become 0 and are added back to the rows that do
//                attend them in the epilogue.  int8, e4m3fn, MX4: convert the codes exactly to fp16
//   warp 12      issues the MMAs and owns the tensor memory
//   warp 13      copies: fp16 parts by TMA (a box of a part's rows of a packed prompt, or of 16 rows
//                of a page, by 64 channels, 128-byte swizzle), codes into a ring; rows out of range
//                are zeros
//   warp 15      finds the CTA's next items
// K is K-major, V MN-major, both as 128-byte rows of 64 channels with the 128-byte swizzle.
//
// Scales of a quantised cache: v_scale multiplies the finished sums.  k_scale per tensor joins
// sigma; per channel it is folded into the queries, Q k_scale 2^-e rounded to fp16 (e per vector:
// the largest entry comes to 2^14, so no range is lost; a score's error is at most
// 2^-11 sum |q_d k_d|, what a cache of fp16 keys has).  Relative error against 64 bits (of the outputs'
// norm): 2.1e-4 by their rounding to fp16 alone, 2.9e-4 with P's, 3.8e-4 with the folded queries'.  The
// rest of that rounding as a second product would take half as many tensor-core cycles again; with two tiles of
// head_dim 128, and with head_dim 256, neither memory has room for it beside K and V, and the forms that have it
// (tensor memory with one tile, or head_dim 64) round as those do.
//
// Pieces (few vectors over long caches): the batch's blocks are cut into equal contiguous pieces,
// one per CTA, whose ends fall anywhere in a (tile, KV head)'s range; a CTA writes fp32 partials of
// the two ranges at most that its piece's ends cut, which attend_merge.cu joins.
//
// What bounds it (32 / 8 heads x 128): a prompt of 16384 the tensor cores, at 76 % of their measured
// rate (1510 us), by the chain from a block's scores over its softmax to its product with V, which is longer than
// the products of two tiles; a quantised cache with few new tokens its conversion, 2900 cycles per 128
// positions of K and V of which 1800 are shared memory's (codes in and out, fp16 in, operands out);
// a short call the way from the launch over the first item (2 us), its queries and a block's chain.
//
// Every wait is bounded; a CTA that gives up marks its outputs NaN and raises
// I8KV_FLAG_WAIT_TIMEOUT.  tests/attend_withheld.cu builds the kernel with a shorter limit and copies or arrivals
// that do not come, by the two macros below.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>

#include "../../include/int8kv.h"
#include "attend.h"
#include "codes.cuh"
#include "device.cuh"
#include "tc.cuh"

#ifndef I8KV_ATTEND_WAIT_NS
#define I8KV_ATTEND_WAIT_NS ::i8kv::tc::kWaitNs
#endif
#ifndef I8KV_ATTEND_WITHHELD  // whether what belongs to a block of the CTA's item does not come
#define I8KV_ATTEND_WITHHELD(what, item, block) false
#endif

namespace i8kv {
namespace ap {

constexpr int BM = 128;  // vectors of a tile (tensor-memory lanes)
constexpr int BN = 128;  // positions of a block
constexpr int kProdThreads = 128;
constexpr int kSoftThreads = 256;
constexpr int kThreads = 512;
constexpr int kMmaWarp = 12, kTmaWarp = 13, kLastWarp = 15;
constexpr int kUsers = (kSoftThreads + kProdThreads) / 32 + 2;  // warps that work through the items
constexpr float kLazy = 7.f;   // powers of two that the maximum may outgrow the base
constexpr float kShift = 8.f;  // P holds p 2^kShift: at most 2^15
constexpr int kPoison = 8;     // blocks that a tile's rows can attend in part (6 at most)
constexpr float kLn2 = 0.6931471805599453f;

// What a test keeps from coming: the queries' hand-over, copies of K or V, probabilities (of tile 0 or 1).
enum Hold { kHoldQ, kHoldK, kHoldV, kHoldP };
// What a K or V value is read from.
enum Src { kF16 = 0, kI8 = 1, kE4 = 2, kMx4 = 3 };

template <int D, int TILES>
struct Layout {
  static constexpr int kM = BM * TILES;
  static constexpr int kSlabs = D / 64;
  static constexpr int kSlab = 128 * 128;  // 64 channels of 128 rows
  static constexpr int kQ = 0;
  static constexpr int kQBytes = kM * D * 2;
  // K and V come in parts, each with barriers of its own: a block, or, where shared memory holds one
  // block only (head_dim 256), half of one, so that a half is filled anew while the products of the
  // other are at work: of K half the channels, of V half the positions
  static constexpr int kParts = D == 256 ? 2 : 1;
  static constexpr int kPart = BN * D * 2 / kParts;
  static constexpr int kKSlabs = kSlabs / kParts;
  static constexpr int kVRows = BN / kParts;
  static constexpr int kRing = D == 64 ? 4 : 2;  // places for parts
  static constexpr int kK = kQ + kQBytes;
  static constexpr int kV = kK + kRing * kPart;
  static constexpr int kBars = kV + kRing * kPart;
  static constexpr int kSlots = kBars + 448;
  // two items' worth of what belongs to one: the next is begun while the one before is written out
  static constexpr int kItem = kSlots + 64;
  static constexpr int kPois = kItem + 2 * 128;        // [2][kPoison][4] bits of positions
  static constexpr int kRowScale = kPois + 2 * kPoison * 16;  // [2][kM] 2^e of each vector
  static constexpr int kXchg = kRowScale + 2 * kM * 4;              // TILES == 1: [3][2][BM] floats
  static constexpr int kVote = kXchg + (TILES == 1 ? 6 * BM * 4 : 0);  // TILES == 1: [3][4][2] ints
  static constexpr int kBytes = kVote + (TILES == 1 ? 96 : 0);
  static constexpr int kOCol = 2 * BN;  // O behind the two score buffers
  static_assert(kOCol + TILES * D <= 512, "tensor memory");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// barriers (8 bytes each); the first five by a part's place, the others by tile (or, TILES == 1, by
// score buffer)
// kItemFull, kItemFree, kQFull, kOFree: by the item's parity; kRawFull, kRawFree: by the place in the ring of codes
constexpr int kRawMost = 8;
enum Bar {
  kKFull = 0, kKFree = 4, kVFull = 8, kVFree = 12, kVOk = 16, kSFull = 20, kPFull = 22, kPVDone = 24, kPHalf = 26,
  kItemFull = 28, kItemFree = 30, kQFull = 32, kOFree = 34, kQFree = 36, kDone, kRawFull, kRawFree = kRawFull + kRawMost, kNumBars = kRawFree + kRawMost
};
enum Slot { kTmem, kAbort, kBadPage, kAnyPoison = kBadPage + 2, kNumSlots = kAnyPoison + 2 };  // the last two by parity
static_assert(kNumBars * 8 <= 448 && kNumSlots * 4 <= 64, "misc");

__device__ __forceinline__ void sync_all() { asm volatile("bar.sync 0, 512;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int c, int h, int row,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(map), "r"(c), "r"(h), "r"(row), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// tc::mbar_wait of a converged warp.  All lanes wait: one alone, and the others for it, hears of a phase some 300
// cycles later.
// But every lane's poll takes its turn at the shared memory that the tensor cores read operands
// from, so only the softmax and MMA warps, whose waits are one behind the other, do it ...  A wait in vain is told in
// *abort before the warp does anything else: whoever sees an arrival or a product behind it sees that too.  kFence:
// what follows is issued to the tensor cores, which orders no memory (elsewhere arrivals do; a fence there cost the
// converters 3 %).
template <bool kFence = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  bool ok = tc::mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = tc::global_ns();
#pragma unroll 1
    while (!(ok = tc::mbar_try_wait(bar, parity))) {
      if (*abort != 0 || tc::global_ns() - t0 > I8KV_ATTEND_WAIT_NS) {
        *abort = 1;
        if (kFence) __threadfence_block();
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}
// ... and for an item one lane waits, which sleeps between polls.
__device__ __forceinline__ bool calm_wait(uint32_t bar, uint32_t parity) {
  bool ok = (threadIdx.x & 31) != 0 || tc::mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = tc::global_ns();
    do {
      __nanosleep(100);
      ok = tc::mbar_try_wait(bar, parity);
    } while (!ok && tc::global_ns() - t0 <= I8KV_ATTEND_WAIT_NS);
  }
  ok = __all_sync(0xffffffffu, ok);
  __syncwarp();  // (the vote orders no memory)
  return ok;
}
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}

// The MMA warp works converged, so that descriptors and addresses stay in uniform registers (one
// lane alone took 75 to 130 cycles to form and issue an instruction of 64); the lane that issues is
// elected once (at each group of four instructions: 2665 us against 1520 for a prompt of 16384).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p;
}
// Operands as the low word of their descriptors (start address, and LBO in the upper half); the high
// one is the same for all: 8 rows of 128 bytes per atom (SBO), 128-byte swizzle.
constexpr uint32_t kDescHigh = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo) { return saddr >> 4 | (lbo >> 4) << 16; }
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " mov.b64 a, {%1, %6};\n mov.b64 b, {%2, %6};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(lead), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " mov.b64 b, {%2, %6};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(lead), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(lead)
      : "memory");
}

// Two fp32 values as one operand, and two operations in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(x), "=f"(y) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float sum4(const uint64_t (&p)[2]) {
  float a, b;
  unpair(add2(p[0], p[1]), a, b);
  return a + b;
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// Caps.  soft_cap takes 2 c / (1 + e^(2 y)), y = x / c, from c: up to 2^-21 of c off.  With caps up to kCapExp that is
// 2^-14 at most, an eighth of what a weight's rounding to fp16 is.  A higher cap, which would leave nothing of scores far
// below it, takes the series of c tanh y = x (1 - y^2 / 3 + 2 y^4 / 15 - 17 y^6 / 315 + ...) for |y| < 1/4, within 2^-21
// of the result; beyond, soft_cap is within 2^-18.9 of it.  (For all caps the choice cost 8 to 16 %; now prompts
// of 1000 to 4097 tokens, 32 / 8 heads x 128, take 322 us with a cap of 30, 326 to 349 with one of 300.  Each score's
// choice is its own: what lies beside it, masked perhaps, has no part in it.)
constexpr float kCapExp = 128.f, kSeries = 0.25f;
__device__ __forceinline__ void cap_small(float& x0, float& x1, float inv_c) {
  const uint64_t x = pair(x0, x1), y = mul2(x, pair(inv_c, inv_c)), y2 = mul2(y, y);
  uint64_t t = fma2(y2, pair(-17.f / 315.f, -17.f / 315.f), pair(2.f / 15.f, 2.f / 15.f));
  t = fma2(y2, t, pair(-1.f / 3.f, -1.f / 3.f));
  unpair(fma2(mul2(x, y2), t, x), x0, x1);
}

// Zero the non-finite ones of two fp16 values; returns whether there were any.
__device__ __forceinline__ bool finite_only(uint32_t& x) {
  const bool lo = (x & 0x7C00u) == 0x7C00u, hi = (x & 0x7C000000u) == 0x7C000000u;
  if (lo) x &= 0xFFFF0000u;
  if (hi) x &= 0x0000FFFFu;
  return lo || hi;
}
__device__ __forceinline__ bool finite_only(uint4& v) {
  const bool a = finite_only(v.x), b = finite_only(v.y), c = finite_only(v.z), d = finite_only(v.w);
  return a || b || c || d;
}

// Whether one of 8 fp16 values is not finite: their magnitudes + 2^10 reach the sign's bit.
__device__ __forceinline__ bool not_finite(const uint4& v) {
  auto high = [](uint32_t x) { return (x & 0x7fff7fffu) + 0x04000400u; };
  return ((high(v.x) | high(v.y) | high(v.z) | high(v.w)) & 0x80008000u) != 0u;
}

// Four lanes' 4 x 16 bytes the other way round: lane l of the four gets, at i, the 16 bytes l of lane i.
__device__ __forceinline__ void across(uint32_t (&w)[16], int lane) {
#pragma unroll
  for (int bit = 1; bit < 4; bit *= 2) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & bit) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t &x = w[4 * i + e], &y = w[4 * (i + bit) + e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x : y, bit);
        (up ? x : y) = got;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// the work
// ---------------------------------------------------------------------------

struct Seq {
  int s0, n, len;
};
__device__ __forceinline__ Seq seq_of(const AttendParams& p, int b, bool report = false) {
  const int a0 = __ldg(p.starts + b), a1 = __ldg(p.starts + b + 1);
  Seq s;
  s.s0 = min(max(a0, 0), p.T);
  const int s1 = min(max(a1, s.s0), p.T);
  s.n = s1 - s.s0;
  bool bad = s.s0 != a0 || s1 != a1;
  s.len = s.n;
  if (p.lens != nullptr) {
    const int l = __ldg(p.lens + b);
    s.len = min(max(l, 0), p.cap);
    bad |= s.len != l;
  }
  if (report && bad) flag_or(p.flags, I8KV_FLAG_LEN_CLAMPED);
  return s;
}

// One piece of a (tile, KV head)'s blocks.
struct Item {
  Seq q;
  int b, t, g;
  int first, last;  // tokens of the tile
  int B0, f0, f1;   // its first block; every row attends all of the blocks [f0, f1)
  int blk0, blk1;   // those worked on here
  int slot;         // of the partials; -1: all of the tile's blocks are worked on
  bool has;         // false: there are no more
  __device__ __forceinline__ bool partial(int blk) const { return blk < f0 || blk >= f1; }
  __device__ __forceinline__ int ordinal(int blk) const {
    return min(blk < f0 ? blk - B0 : f0 - B0 + blk - f1, kPoison - 1);
  }
};

template <int M>
__device__ __forceinline__ int tiles_of(const AttendParams& p, int n) {
  return (n * p.G + M - 1) / M;
}

// The length of a sequence's tiles in 64ths of a block, when the batch is cut into pieces of equal
// length: that of tile 0 and what each further one has more.  (A tile's blocks are dealt out in
// proportion, so the lengths need not be exact.)
struct Length {
  long long first;
  int more;
  __device__ __forceinline__ long long of(int t) const { return first + (long long)t * more; }
  __device__ __forceinline__ long long before(int t) const { return t * first + (long long)t * (t - 1) / 2 * more; }
};
template <int M>
__device__ __forceinline__ Length length_of(const AttendParams& p, const Seq& s) {
  const int all = max((s.len + BN - 1) / BN, 1);
  Length l;
  if (p.window >= 0 && p.window < s.len) {
    const long long w = ((long long)p.window + M / p.G) / BN + 1;
    l.first = 64 * (w < all ? w : all);
    l.more = 0;
  } else {
    l.first = 64LL * min(max((s.len - s.n + M / p.G) / BN + 1, 1), all);
    l.more = M / (2 * p.G);
  }
  // What an item costs beside its blocks, in blocks: without it a CTA with 20 short items among its 118 blocks
  // took 424 us, others with 2 and 123 blocks 265.  (With 4 / 10 for two tiles: 512 tokens over 1024 to 16384 in
  // 8 sequences 347 / 305 us; with 2 / 3 for one: single tokens over 512 to 8192 in 64 sequences 154 / 148.)
  l.first += 64 * (M > BM ? 10 : 3);
  return l;
}

// The first position that a token at pos attends (one before the sequence's beginning attends none: the
// difference of a negative one and a wide window would leave the range).
__device__ __forceinline__ int first_seen(const AttendParams& p, int pos) {
  return p.window < 0 ? 0 : max(max(pos, 0) - p.window, 0);
}
// The part [x, y) of w of the tile's blocks.
template <int M>
__device__ __forceinline__ void place(const AttendParams& p, Item& it, long long x, long long y, long long w) {
  const int v0 = it.t * M, v1 = min(it.q.n * p.G, v0 + M);
  it.first = v0 / p.G;
  it.last = (v1 - 1) / p.G;
  const int p0 = it.q.len - it.q.n + it.first, p1 = it.q.len - it.q.n + it.last;
  const int hi_min = max(p0 + 1, 0), hi = max(p1 + 1, 0);
  const int lo = first_seen(p, p0), lo_max = first_seen(p, p1);
  it.B0 = lo / BN;
  const int B1 = (hi + BN - 1) / BN;
  it.f0 = max(it.B0, (lo_max + BN - 1) / BN);
  it.f1 = max(it.f0, hi_min / BN);
  const long long n = max(B1 - it.B0, 0);
  it.blk0 = it.B0 + (int)(x * n / w);
  it.blk1 = it.B0 + (int)(y * n / w);
}

static_assert(sizeof(Item) <= 128, "item");

// The walk over this CTA's items, of the last warp, which hands them out in shared memory.
struct Walk {
  long long f, end, x;  // pieces: where the CTA's next one begins and its last one ends, and the place in the (tile, head)
  Length len;           // of sequence b's tiles
  int round, total, b0, base;
};

__device__ __forceinline__ int scan(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __forceinline__ long long scan(long long x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __forceinline__ Seq of_lane(const Seq& s, int l) {
  return Seq{__shfl_sync(0xffffffffu, s.s0, l), __shfl_sync(0xffffffffu, s.n, l), __shfl_sync(0xffffffffu, s.len, l)};
}

// Unsplit tiles are worked on in the order of falling length where there are few sequences (a count
// of them costs a warp 0.1 us per 32), else sequence after sequence.
constexpr int kSortedSeqs = 128;

// Of a sequence's tiles, those of at least x blocks (without a window): the last ones.
template <int M>
__device__ __forceinline__ int longer_tiles(const AttendParams& p, const Seq& s, int x) {
  const int tiles = tiles_of<M>(p, s.n);
  const int need = (x - 1) * BN - (s.len - s.n);  // the tile's last token must reach this one
  return x <= 0 || need <= 0 ? tiles : need > s.n - 1 ? 0 : tiles - need * p.G / M;
}

// The batch cut into pieces: the length of one (a warp, all lanes alike).
template <int M>
__device__ __forceinline__ long long piece_length(const AttendParams& p, int pieces, long long& total) {
  const int lane = threadIdx.x & 31;
  total = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32)
    if (b0 + lane < p.B) {
      const Seq s = seq_of(p, b0 + lane);
      total += p.Hkv * length_of<M>(p, s).before(tiles_of<M>(p, s.n));
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  return (total + pieces - 1) / pieces;
}
// The (tile, head) at place f < total of the batch: it.b, q, t, g, the lengths, and the place in it.
template <int M>
__device__ __forceinline__ long long find_place(const AttendParams& p, long long f, Item& it, Length& len) {
  const int lane = threadIdx.x & 31;
  long long before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    Seq s{0, 0, 0};
    Length l{0, 0};
    long long x = 0;
    if (b0 + lane < p.B) {
      s = seq_of(p, b0 + lane);
      l = length_of<M>(p, s);
      x = p.Hkv * l.before(tiles_of<M>(p, s.n));
    }
    const long long incl = before + scan(x);
    const unsigned hit = __ballot_sync(0xffffffffu, incl > f);
    if (hit != 0) {
      const int n = __ffs(hit) - 1;
      it.b = b0 + n;
      it.q = of_lane(s, n);
      len.first = __shfl_sync(0xffffffffu, l.first, n);
      len.more = __shfl_sync(0xffffffffu, l.more, n);
      const long long in_seq = f - __shfl_sync(0xffffffffu, incl - x, n);
      int t = 0, end = tiles_of<M>(p, it.q.n);  // the last tile that begins at in_seq or before
      while (end - t > 1) {
        const int mid = (t + end) >> 1;
        if (p.Hkv * len.before(mid) <= in_seq) t = mid; else end = mid;
      }
      it.t = t;
      const long long in_tile = in_seq - p.Hkv * len.before(t);
      it.g = (int)(in_tile / len.of(t));
      return in_tile - it.g * len.of(t);
    }
    before = __shfl_sync(0xffffffffu, incl, 31);
  }
  return 0;
}

template <int M>
__device__ __forceinline__ void start_walk(const AttendParams& p, Item& it, Walk& w) {
  const int lane = threadIdx.x & 31;
  w = Walk{};
  it = Item{};
  if (p.pieces == 0) {
    for (int b0 = 0; b0 < p.B; b0 += 32)
      w.total += __reduce_add_sync(0xffffffffu, b0 + lane < p.B ? tiles_of<M>(p, seq_of(p, b0 + lane).n) : 0);
    w.total *= p.Hkv;
    return;
  }
  long long total;
  const long long one = piece_length<M>(p, p.pieces, total);
  w.f = one * blockIdx.x;
  w.end = min(w.f + one, total);
  if (w.f < w.end) w.x = find_place<M>(p, w.f, it, w.len);
}

// The next item; false: there is none.
template <int M>
__device__ __forceinline__ bool next_item(const AttendParams& p, Item& it, Walk& w) {
  const int lane = threadIdx.x & 31;
  if (p.pieces == 0) {
    it.slot = -1;
    const bool sorted = p.B <= kSortedSeqs;
    // (sorted: back and forth over the CTAs, so that none always has the longer ones)
    const int idx = w.round * gridDim.x + (sorted && (w.round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (idx >= w.total) return false;
    ++w.round;
    int r = idx / p.Hkv;
    it.g = idx - r * p.Hkv;
    int x = 0, next = 0;  // sorted: the tile's blocks, and how many tiles have more
    if (sorted) {
      int hi = (p.lens != nullptr ? p.cap : p.T) / BN + 2;
      while (hi - x > 1) {
        const int mid = (x + hi) >> 1;
        int c = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32)
          if (b0 + lane < p.B) c += longer_tiles<M>(p, seq_of(p, b0 + lane), mid);
        c = __reduce_add_sync(0xffffffffu, c);
        if (c > r) {
          x = mid;
        } else {
          hi = mid;
          next = c;
        }
      }
      r -= next;
      w.base = w.b0 = 0;
    }
    for (;; w.b0 += 32) {
      Seq s{0, 0, 0};
      int c = 0, tiles = 0;
      if (w.b0 + lane < p.B) {
        s = seq_of(p, w.b0 + lane);
        tiles = tiles_of<M>(p, s.n);
        c = sorted ? longer_tiles<M>(p, s, x) : tiles;
      }
      const int mine = sorted ? c - longer_tiles<M>(p, s, x + 1) : c;
      const int incl = w.base + scan(mine);
      const unsigned hit = __ballot_sync(0xffffffffu, incl > r);
      if (hit != 0) {
        const int l = __ffs(hit) - 1;
        it.b = w.b0 + l;
        it.q = of_lane(s, l);
        // (of a sequence the later ones first)
        it.t = __shfl_sync(0xffffffffu, sorted ? tiles - c + (r - (incl - mine)) : tiles - 1 - (r - (incl - mine)), l);
        break;
      }
      w.base = __shfl_sync(0xffffffffu, incl, 31);
      if (w.b0 + 32 >= p.B) return false;
    }
    place<M>(p, it, 0, 1, 1);
    return true;
  }
  if (w.f >= w.end) return false;
  while (w.x == w.len.of(it.t)) {  // the next head, tile or sequence
    w.x = 0;
    if (++it.g < p.Hkv) break;
    it.g = 0;
    if (++it.t < tiles_of<M>(p, it.q.n)) break;
    it.t = 0;
    do {
      if (++it.b >= p.B) return false;
      it.q = seq_of(p, it.b);
    } while (it.q.n == 0);
    w.len = length_of<M>(p, it.q);
    break;
  }
  const long long all = w.len.of(it.t), y = min(all, w.x + (w.end - w.f));
  // a CTA begins inside at most one tile and ends inside at most one
  it.slot = w.x > 0 ? 2 * (int)blockIdx.x : y < all ? 2 * (int)blockIdx.x + 1 : -1;
  place<M>(p, it, w.x, y, all);
  w.f += y - w.x;
  w.x = y;
  return true;
}

// The 16-row group that holds position pos of the item's sequence, as a row number / 16 of the cache; -1
// where the position is not attended by any (past the end) or its page is out of range.  In two parts,
// so that the table can be read well before its entry is needed.
__device__ __forceinline__ int page_of(const AttendParams& p, const Item& it, int pos) {  // as the table has it
  if (pos >= it.q.len) return -1;
  return __ldg(p.table + (long long)it.b * p.max_blocks + (p.bs_log2 >= 0 ? pos >> p.bs_log2 : pos / p.bs));
}
__device__ __forceinline__ int group_in(const AttendParams& p, int page, int pos) {
  if (page < 0 || page >= p.num_blocks) return -1;
  const int off = p.bs_log2 >= 0 ? pos & (p.bs - 1) : pos % p.bs;
  return (int)((long long)page * (p.bs >> 4)) + (off >> 4);
}
__device__ __forceinline__ int group_of(const AttendParams& p, const Item& it, int pos) {
  return group_in(p, page_of(p, it, pos), pos);
}

// V[t, g, d] as stored (without v_scale), for the values that are added back.
template <int D, int SRC>
__device__ __noinline__ float v_value(const AttendParams& p, const Item& it, int t, int d) {
  if (p.table == nullptr)
    return __half2float(reinterpret_cast<const __half*>(p.v)[(it.q.s0 + (long long)t) * p.v_stride +
                                                             (long long)it.g * D + d]);
  const int grp = group_of(p, it, t);
  if (grp < 0) return 0.f;
  const long long row = (long long)grp * 16 + (t & 15);
  if constexpr (SRC == kF16) {
    return __half2float(reinterpret_cast<const __half*>(p.v)[(row * p.Hkv + it.g) * D + d]);
  } else if constexpr (SRC == kE4) {
    return e4m3_value(reinterpret_cast<const uint8_t*>(p.v)[(row * p.Hkv + it.g) * D + d]);
  } else if constexpr (SRC == kMx4) {
    // (only the block scale can be no number)
    const int tiles = p.bs >> 4;
    const uint8_t* rec = reinterpret_cast<const uint8_t*>(p.k) +
                         ((long long)(grp / tiles) * p.Hkv * tiles + (long long)it.g * tiles + grp % tiles) * (18LL * D);
    return e4m3_value(rec[17 * D + (t & 15) * (D / 16) + (d >> 4)]);
  }
  return 0.f;
}

// Adds the non-finite values of the attended positions that were taken out of V to channels d0 .. d1 - 1 of a
// row that its thread has written: fp16 outputs, or fp32 partials.
template <int D, int SRC, typename T>
__device__ __noinline__ void add_poison(const AttendParams& p, const Item& it, const uint32_t* bits,
                                        int lo, int hi, int d0, int d1, T* o) {
  for (int blk = it.blk0; blk < it.blk1; ++blk) {
    if (!it.partial(blk)) continue;
    const uint32_t* w = bits + 4 * it.ordinal(blk);
    for (int j = 0; j < BN; ++j) {
      const int t = blk * BN + j;
      if (!((w[j >> 5] >> (j & 31)) & 1u) || t < lo || t >= hi) continue;
      for (int d = d0; d < d1; ++d) {
        const float x = v_value<D, SRC>(p, it, t, d);
        if (fabsf(x) <= 65504.f) continue;
        const float vs = SRC == kF16 ? 1.f : __ldg(p.v_scale + (p.per_channel ? it.g * D + d : 0));
        o[d] = (T)((float)o[d] + x * vs);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// producers of a quantised cache
// ---------------------------------------------------------------------------

// Codes are copied into a ring in shared memory, unit by unit, some units before they are converted:
// int8, e4m3fn: 8 KB, TMA boxes of 16 rows of a page by 128 bytes (64 with head_dim 64): 64 (128) rows
// to a unit;
// MX4: 64 rows, the K or V half of the records of four 16-row groups (a bulk copy each).
template <int D, int TILES, int SRC>
struct Raw {
  using L = Layout<D, TILES>;
  static constexpr int kWide = D < 128 ? D : 128;  // channels of a unit (MX4: all)
  static constexpr int kRows = SRC == kMx4 ? 64 : 8192 / kWide;
  static constexpr int kBytes = SRC == kMx4 ? 36 * D : 8192;
  static constexpr int kRun = SRC == kMx4 ? 2 : BN * D / 8192;  // units of a block's K or V
  static constexpr int kAt = (L::kBytes + 127) / 128 * 128;
  static constexpr int kRoom = (227 * 1024 - kAt) / kBytes;
  static constexpr int kAhead = SRC == kF16 ? 0 : kRoom < kRawMost ? kRoom : kRawMost;
  static constexpr int kSmem = kAt + kAhead * kBytes;
  static_assert(kAhead == 0 || kAhead >= 3, "units on their way");
  // int8, e4m3fn: where unit u of a part begins in the part
  static __device__ __forceinline__ int first_row(int u, bool is_v) { return D == 256 && is_v ? 0 : u * kRows; }
  static __device__ __forceinline__ int first_slab(int u, bool is_v) { return D == 256 && is_v ? 2 * u : 0; }
};

// A place of the ring and the parity of its turn, one unit after another.
template <int N>
struct Place {
  int place = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void next() {
    if (++place >= N) {
      place = 0;
      turn ^= 1u;
    }
  }
  __device__ __forceinline__ void back(int units) {
    place -= units;
    if (place < 0) {
      place += N;
      turn ^= 1u;
    }
  }
};

// N chunks of 8 fp16 values into a line of a part (64 channels of a row).
template <int N>
__device__ __forceinline__ void store_chunks(const uint4 (&h)[N], uint32_t line, int first, int row_in_part) {
#pragma unroll
  for (int j = 0; j < N; ++j) sts16(line + (((first + j) ^ (row_in_part & 7)) << 4), h[j]);
}

// Zero the e4m3fn NaN codes (all ones but for the sign) among four; returns whether there were any.
__device__ __forceinline__ bool numbers_only(uint32_t& x) {
  const uint32_t nan = ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  x &= ~((nan >> 7) * 255u);
  return nan != 0u;
}
// (bits, any: noted for a row of V where the rows are looked at)
__device__ __forceinline__ void note_row(uint32_t* bits, int row, volatile int* any) {
  atomicOr(bits + (row >> 5), 1u << (row & 31));
  *any = 1;
}

// int8, e4m3fn: U units of a part, from u on, as fp16.  bits: of the block's rows, from row0 on, that have a NaN.
template <int D, int TILES, int SRC, int U>
__device__ __forceinline__ void convert_bytes(int ct, const uint32_t (&at)[U], uint32_t dst, bool is_v, int u,
                                              uint32_t* bits, int row0, volatile int* any) {
  using R = Raw<D, TILES, SRC>;
  const int rows = is_v ? Layout<D, TILES>::kVRows : BN;
  // 8 lanes take 64 bytes of each of two rows, from different halves of them: neither their loads nor
  // their stores meet a bank twice
  const int c = ct & 3;
  auto place = [&](int k, int& row, int& slab) {
    const int q = ct + kProdThreads * k;
    row = q >> 2;
    slab = 0;
    if (D != 64) {
      const int odd = row & 1, pr = q >> 3;
      row = 2 * (pr % (R::kRows / 2)) + odd;
      slab = odd ^ (pr / (R::kRows / 2));
    }
  };
  uint4 code[4 * U];  // (all on their way before the first is used)
#pragma unroll
  for (int k = 0; k < 4 * U; ++k) {
    int row, slab;
    place(k & 3, row, slab);
    code[k] = lds16(at[k >> 2] + row * R::kWide + slab * 64 + c * 16);
  }
  if (SRC == kE4 && bits != nullptr) {
#pragma unroll 1
    for (int k = 0; k < 4 * U; ++k) {
      // (a loop over registers: the chunk in turn is the first, the others move up)
      uint4 x = code[0];
      const bool a = numbers_only(x.x), b = numbers_only(x.y), c1 = numbers_only(x.z), d = numbers_only(x.w);
      if (a || b || c1 || d) {
        int row, slab;
        place(k & 3, row, slab);
        note_row(bits, row0 + row + R::first_row(u + (k >> 2), is_v), any);
      }
#pragma unroll
      for (int e = 1; e < 4 * U; ++e) code[e - 1] = code[e];
      code[4 * U - 1] = x;
    }
  }
#pragma unroll
  for (int k = 0; k < 4 * U; ++k) {
    const uint4 x = code[k];
    int row, slab;
    place(k & 3, row, slab);
    row += R::first_row(u + (k >> 2), is_v);
    slab += R::first_slab(u + (k >> 2), is_v);
    uint4 h[2];
    if constexpr (SRC == kI8) {
      const uint32_t x0 = flip_i8x4(x.x), x1 = flip_i8x4(x.y), x2 = flip_i8x4(x.z), x3 = flip_i8x4(x.w);
      h[0] = make_uint4(i8x2_to_h2(x0, 0x4140u), i8x2_to_h2(x0, 0x4342u), i8x2_to_h2(x1, 0x4140u),
                        i8x2_to_h2(x1, 0x4342u));
      h[1] = make_uint4(i8x2_to_h2(x2, 0x4140u), i8x2_to_h2(x2, 0x4342u), i8x2_to_h2(x3, 0x4140u),
                        i8x2_to_h2(x3, 0x4342u));
    } else {
      e4m3x4_to_h2x2(x.x, h[0].x, h[0].y);
      e4m3x4_to_h2x2(x.y, h[0].z, h[0].w);
      e4m3x4_to_h2x2(x.z, h[1].x, h[1].y);
      e4m3x4_to_h2x2(x.w, h[1].z, h[1].w);
    }
    store_chunks(h, dst + (slab * rows + row) * 128, 2 * c, row);
  }
}

// MX4: N slabs, from slab0, of the 64 rows of a unit, as fp16, to the rows from row_in_part of a part.
template <int D, int N>
__device__ __forceinline__ void convert_mx4(int ct, uint32_t at, uint32_t dst, int rows, int row_in_part, int slab0,
                                            uint32_t* bits, int row0, volatile int* any) {
  const int row = ct >> 1, c = ct & 1;  // 32 channels of each slab
  const uint32_t rec = at + (row >> 4) * (9 * D);
  uint4 code[N];
  uint16_t scale[N];  // two block scales each
#pragma unroll
  for (int k = 0; k < N; ++k) {
    code[k] = lds16(rec + (row & 15) * (D / 2) + (slab0 + k) * 32 + c * 16);
    asm volatile("ld.shared.u16 %0, [%1];\n"
                 : "=h"(scale[k])
                 : "r"(rec + 8 * D + (row & 15) * (D / 16) + (slab0 + k) * 4 + 2 * c)
                 : "memory");
  }
  if (bits != nullptr) {  // (a code is always a number, its scale perhaps not)
    bool bad = false;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      uint32_t x = scale[k];
      bad |= numbers_only(x);
      scale[k] = (uint16_t)x;
    }
    if (bad) note_row(bits, row0 + row, any);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint4 x = code[k];
    const uint16_t both = scale[k];
    uint32_t s0, s1;  // twice each
    e4m3x4_to_h2x2(prmt(both, 0u, 0x1100u), s0, s1);
    uint4 h[4];
    e2m1x8_to_h2x4(x.x, h[0].x, h[0].y, h[0].z, h[0].w);
    e2m1x8_to_h2x4(x.y, h[1].x, h[1].y, h[1].z, h[1].w);
    e2m1x8_to_h2x4(x.z, h[2].x, h[2].y, h[2].z, h[2].w);
    e2m1x8_to_h2x4(x.w, h[3].x, h[3].y, h[3].z, h[3].w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t s = j < 2 ? s0 : s1;
      asm("mul.f16x2 %0, %0, %1;\n" : "+r"(h[j].x) : "r"(s));  // exact: 6 significant bits
      asm("mul.f16x2 %0, %0, %1;\n" : "+r"(h[j].y) : "r"(s));
      asm("mul.f16x2 %0, %0, %1;\n" : "+r"(h[j].z) : "r"(s));
      asm("mul.f16x2 %0, %0, %1;\n" : "+r"(h[j].w) : "r"(s));
    }
    store_chunks(h, dst + (k * rows + row_in_part + row) * 128, 4 * c, row_in_part + row);
  }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------

struct Args {
  // [rows, Hkv, D] of fp16: boxes of 64 channels of a part's rows (packed) or 16 (pages); of int8 or e4m3fn pages: 16 rows of
  // 128 bytes (64 with head_dim 64)
  CUtensorMap km, vm;
  AttendParams p;
};

// Registers of a thread after the deal between the four warpgroups (softmax, twice; producers; the
// rest), which started with 128 each.
template <int TILES, int SRC>
struct Deal {
  static constexpr int kSoft = TILES == 2 ? 176 : 152;
  static constexpr int kProd = TILES == 2 ? 80 : 120;
  static constexpr int kRest = TILES == 2 ? 80 : 88;
  static_assert(2 * kSoft + kProd + kRest == 4 * 128, "what the launch has");
};

template <int D, int TILES, int SRC>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ Args a) {
  using L = Layout<D, TILES>;
  constexpr int M = L::kM, P = L::kParts, N = L::kRing;
  const AttendParams& p = a.p;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_addr(smem);
  auto bar = [&](int k) -> uint32_t { return sbase + L::kBars + 8 * k; };
  volatile int* slot = reinterpret_cast<volatile int*>(smem + L::kSlots);
  uint32_t* poison = reinterpret_cast<uint32_t*>(smem + L::kPois);
  float* rscale = reinterpret_cast<float*>(smem + L::kRowScale);

  if (warp == kMmaWarp) {
    tc::tmem_alloc(sbase + L::kSlots + 4 * kTmem, 512);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < N; ++s) {
      tc::mbar_init(bar(kKFull + s), SRC == kF16 ? 1 : kProdThreads / 32);
      tc::mbar_init(bar(kKFree + s), 1);
      tc::mbar_init(bar(kVFull + s), 1);
      tc::mbar_init(bar(kVFree + s), 1);
      tc::mbar_init(bar(kVOk + s), kProdThreads / 32);
    }
    for (int w = 0; w < 2; ++w) {
      tc::mbar_init(bar(kSFull + w), 1);
      tc::mbar_init(bar(kPFull + w), TILES == 2 ? 4 : 8);
      tc::mbar_init(bar(kPHalf + w), 4);
      tc::mbar_init(bar(kPVDone + w), 1);
      tc::mbar_init(bar(kItemFull + w), 1);
      tc::mbar_init(bar(kItemFree + w), kUsers);
      tc::mbar_init(bar(kQFull + w), kProdThreads / 32);
      tc::mbar_init(bar(kOFree + w), kSoftThreads / 32);
    }
    for (int s = 0; s < kRawMost; ++s) {
      tc::mbar_init(bar(kRawFull + s), 1);
      tc::mbar_init(bar(kRawFree + s), kProdThreads / 32);
    }
    tc::mbar_init(bar(kQFree), 1);
    tc::mbar_init(bar(kDone), 1);
    tc::fence_mbar_init();
    slot[kAbort] = (sbase & 1023u) != 0u;  // the swizzled layouts want 1024-byte alignment
  }
  tc::fence_before_sync();
  sync_all();
  tc::fence_after_sync();
  const uint32_t tbase = static_cast<uint32_t>(slot[kTmem]);
  grid_dependency_wait();  // inputs may come from the previous kernel of the stream
  if (p.pieces > 0) grid_launch_dependents();  // the merge, which waits for all of this kernel before it reads a partial
  // Every role goes through the CTA's items by itself; item `k` is read from shared memory, and given
  // back when the role is done with it.  A role whose wait failed goes on through the items without
  // working, so that the others' waits for it end.
  auto item_of = [&](int k) -> const Item& {
    return *reinterpret_cast<const Item*>(smem + L::kItem + 128 * (k & 1));
  };
  // (items of a very long context take their time: a limit of about two minutes)
  auto wait_item = [&](int b, uint32_t parity) -> bool {
    bool ok = false;
    for (int i = 0; !ok && i < 120; ++i) ok = calm_wait(bar(b), parity);
    if (!ok) slot[kAbort] = 1;
    return ok;
  };
  auto take = [&](int k) -> bool {
    const bool ok = wait_item(kItemFull + (k & 1), (k >> 1) & 1);
    return __all_sync(0xffffffffu, ok && item_of(k).has);
  };
  auto give_back = [&](int k) { warp_arrive(bar(kItemFree + (k & 1))); };
  // part j of the CTA's block nn, of K and V alike: its place, and the parity of its filling (a place
  // is free for it after the filling before: the other parity; the first ones need not wait)
  auto spot = [](int nn, int j) -> int { return (nn * P + j) % N; };
  auto turn = [](int nn, int j) -> uint32_t { return ((nn * P + j) / N) & 1; };

  if (warp < kSoftThreads / 32) {
    // -----------------------------------------------------------------------
    // softmax and epilogue
    // -----------------------------------------------------------------------
    regs_up<Deal<TILES, SRC>::kSoft>();
    constexpr int COLS = TILES == 2 ? 128 : 64;  // positions of a block per thread
    const int half = TILES == 2 ? 0 : warp >> 2, tile = TILES == 2 ? warp >> 2 : 0;
    const int r = 32 * (warp & 3) + lane;  // the vector within its tile
    const uint32_t t_lane = (uint32_t)(32 * (warp & 3)) << 16;
    float* xchg = reinterpret_cast<float*>(smem + L::kXchg);
    volatile int* votes = reinterpret_cast<volatile int*>(smem + L::kVote) + (warp & 3) * 2;
    auto pair_sync = [&]() {
      asm volatile("bar.sync %0, %1;\n" ::"r"(1 + (warp & 3)), "r"(64) : "memory");
    };
    // TILES == 1: the two warps of a lane quarter exchange a float each, and whether their waits succeeded: both
    // go on only if both did.
    auto exchange = [&](int buf, bool ok, float x, float& other) -> bool {
      float* b = xchg + buf * 2 * BM;
      b[half * BM + r] = x;
      if (lane == 0) votes[8 * buf + half] = ok ? 1 : 0;
      pair_sync();
      other = b[(half ^ 1) * BM + r];
      return votes[8 * buf] != 0 && votes[8 * buf + 1] != 0;
    };
    auto wait_all = [&](int b, uint32_t parity) -> bool { return warp_wait(bar(b), parity, slot + kAbort); };
    const float cap_inv = p.softcap > 0.f ? fminf(1.f / p.softcap, 1e38f) : 0.f, cap_k = 2.f * kLog2e * cap_inv;
    const float cap_near = kSeries * p.softcap;
    const bool cap_exp = p.softcap > 0.f && p.softcap <= kCapExp;
    const float ks1 = SRC != kF16 && !p.per_channel ? __ldg(p.k_scale) : 1.f;
    int n = 0;  // blocks done by this CTA
    bool ok = true;
    for (int k = 0; take(k); ++k) {
      const Item& it = item_of(k);
      const int v0 = it.t * M, nvec = it.q.n * p.G;
      ok = ok && wait_all(kQFull + (k & 1), (k >> 1) & 1);
      if constexpr (TILES == 1) {
        float none;
        ok = exchange((n + 1) & 1, ok, 0.f, none);
      }
      const bool enter = ok;
      const int v = v0 + tile * BM + r;
      const bool live = v < nvec;
      const int tok = live ? v / p.G : 0;
      const int h = it.g * p.G + (live ? v - tok * p.G : 0);
      const int pos = it.q.len - it.q.n + tok;
      const int hi = live ? max(pos + 1, 0) : 0;
      const int lo = first_seen(p, pos);
      const bool bad_pages = slot[kBadPage + (k & 1)] != 0;
      // scores to powers of two: s c2 (c2 > 0 keeps an unattended -inf what it is)
      const float rs = rscale[(k & 1) * M + tile * BM + r] * fabsf(ks1);
      const float nat = p.sigma * rs;
      float c2 = p.softcap > 0.f ? kLog2e : nat * kLog2e;
      if (c2 < 1e-30f) c2 = 1e-30f;
      const int nb = it.blk1 - it.blk0;
      const bool warp_live = __any_sync(0xffffffffu, live && hi > lo);
      const int blk0 = it.blk0, f0 = it.f0, f1 = it.f1;
      float m_run = neg_inf(), m_top = neg_inf(), l_run = 0.f;
      // a warp without live rows takes part in the hand-overs only
      for (int i = 0; enter && !warp_live && i < nb; ++i) {
        const int nn = n + i;
        ok = wait_all(kSFull + (TILES == 2 ? tile : nn & 1), TILES == 2 ? nn & 1 : (nn >> 1) & 1) && ok;
        if constexpr (TILES == 1) {
          float none;
          if (!(ok = exchange(nn & 1, ok, 0.f, none))) break;
          ok = i == 0 || wait_all(kPVDone, (nn - 1) & 1);
        } else {
          if (!ok) break;
          warp_arrive(bar(kPHalf + tile));
        }
        warp_arrive(bar(kPFull + tile));
      }
      for (int i = 0; enter && warp_live && i < nb; ++i) {
        const int blk = blk0 + i, nn = n + i;
        const int sb = TILES == 2 ? tile : nn & 1;
        const uint32_t par = TILES == 2 ? nn & 1 : (nn >> 1) & 1;
        ok = wait_all(kSFull + sb, par) && ok;
        if (TILES == 2 && !ok) break;
        tc::fence_after_sync();
        const uint32_t s_col = tbase + t_lane + sb * BN + 64 * half;
        const bool masks = blk < f0 || blk >= f1 || bad_pages;
        if (p.softcap > kCapExp) {  // (by 16: it is seldom used, and the others' code makes way for it)
#pragma unroll 1
          for (int c = 0; c < COLS / 16; ++c) {
            float x[16];
            tc::tmem_ld16(s_col + 16 * c, x);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float y0 = x[j] * nat, y1 = x[j + 1] * nat;
              x[j] = soft_cap(y0, p.softcap, cap_k);
              x[j + 1] = soft_cap(y1, p.softcap, cap_k);
              const bool near0 = fabsf(y0) < cap_near, near1 = fabsf(y1) < cap_near;
              cap_small(y0, y1, cap_inv);
              x[j] = near0 ? y0 : x[j];
              x[j + 1] = near1 ? y1 : x[j + 1];
            }
            tc::tmem_st16(s_col + 16 * c, x);
          }
          tc::tmem_wait_st();
        }
        if (masks || cap_exp) {
          // capped and masked in tensor memory, 32 at a time (less code for a loop that shares its
          // instruction cache with the other roles')
          const int at = blk * BN + 64 * half;
#pragma unroll 1
          for (int c = 0; c < COLS / 32; ++c) {
            float x[32];
            tc::tmem_ld32(s_col + 32 * c, x);
            tc::tmem_wait_ld();
            if (cap_exp) {
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = soft_cap(x[j] * nat, p.softcap, cap_k);
            }
            if (masks) {
              // positions [lo, hi) of these 32
              const int a0 = min(max(lo - (at + 32 * c), 0), 32), a1 = min(max(hi - (at + 32 * c), 0), 32);
              uint32_t w = a1 > a0 ? (0xffffffffu >> (32 - (a1 - a0))) << a0 : 0u;
              if (bad_pages) {
                if (group_of(p, it, at + 32 * c) < 0) w &= 0xffff0000u;
                if (group_of(p, it, at + 32 * c + 16) < 0) w &= 0x0000ffffu;
              }
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = (w >> j) & 1u ? x[j] : neg_inf();
            }
            tc::tmem_st32(s_col + 32 * c, x);
          }
          tc::tmem_wait_st();
        }
        float s[COLS];
#pragma unroll
        for (int c = 0; c < COLS / 32; ++c) tc::tmem_ld32(s_col + 32 * c, *reinterpret_cast<float(*)[32]>(&s[32 * c]));
        tc::tmem_wait_ld();
        float top4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int j = 4; j < COLS; j += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top4[e] = j + 4 < COLS ? max3(top4[e], s[j + e], s[j + 4 + e]) : fmaxf(top4[e], s[j + e]);
        }
        float mx = fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]);
        if constexpr (TILES == 1) {
          float mx2;
          if (!(ok = exchange(nn & 1, ok, mx, mx2))) break;
          mx = fmaxf(mx, mx2);
        }
        m_top = fmaxf(m_top, mx);
        const bool moves = m_top * c2 > m_run * c2 + kLazy;  // (from -inf: any score does)
        const float m_new = moves ? m_top : m_run;
        const float base = m_new == neg_inf() ? 0.f : m_new * c2;
        const float alpha = moves ? fast_exp2(m_run * c2 - base) : 1.f;
        const float off = kShift - base;
        const uint64_t c22 = pair(c2, c2), off2 = pair(off, off);
        uint64_t ps[2] = {0ull, 0ull};
        // probabilities of 64 positions, over the scores' columns
        auto probabilities = [&](int c0) {
#pragma unroll
          for (int c = c0; c < c0 + 2; ++c) {
            uint32_t ph[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float x, y;
              unpair(fma2(pair(s[32 * c + 2 * j], s[32 * c + 2 * j + 1]), c22, off2), x, y);
              x = fast_exp2(x);
              y = fast_exp2(y);
              ps[j & 1] = add2(ps[j & 1], pair(x, y));
              ph[j] = pack_h2(x, y);
            }
            tc::tmem_st16u(s_col + 64 * (c >> 1) + 16 * (c & 1), ph);
          }
        };
        probabilities(0);
        const bool rescale = i > 0 && moves;
        m_run = m_new;
        // O is current: with two tiles QK(i) was issued after PV(i - 1) had completed
        if constexpr (TILES == 1) {
          ok = i == 0 || wait_all(kPVDone, (nn - 1) & 1);
          tc::fence_after_sync();
        }
        if (ok && __any_sync(0xffffffffu, rescale)) {
          constexpr int OC = TILES == 2 ? D : D / 2;  // channels of this thread
#pragma unroll 1
          for (int c = 0; c < OC / 32; ++c) {
            float o[32];
            const uint32_t oc = tbase + t_lane + L::kOCol + tile * D + half * OC + 32 * c;
            tc::tmem_ld32(oc, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= rescale ? alpha : 1.f;
            tc::tmem_st32(oc, o);
          }
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        if constexpr (TILES == 2) {
          // the tensor cores take the first half while the second is made
          warp_arrive(bar(kPHalf + tile));
          probabilities(2);
          tc::tmem_wait_st();
          tc::fence_before_sync();
        }
        l_run = fmaf(l_run, alpha, sum4(ps));
        if (!I8KV_ATTEND_WITHHELD(kHoldP + tile, k, i)) warp_arrive(bar(kPFull + tile));
      }
      n += nb;
      // ---- epilogue ----
      ok = ok && (nb == 0 || wait_all(kPVDone + tile, (n - 1) & 1));
      if constexpr (TILES == 1) {
        float l_other;
        ok = exchange(2, ok, l_run, l_other);
        l_run += l_other;
      }
      tc::fence_after_sync();
      const bool attends = live && max(lo, it.blk0 * BN) < min(hi, it.blk1 * BN);
      const bool some = attends && m_top != neg_inf();
      const bool nan = attends && l_run != l_run;
      const float lsum = l_run * 0.00390625f;  // 2^-kShift
      const float m_nat = m_run * c2 * kLn2;
      constexpr int OC = TILES == 2 ? D : D / 2;  // channels of this thread
      const int c_lo = half * OC;
      const float kNan = __int_as_float(0x7fc00000);
      // The next item's products may go over O.  What was read of it counts if by now nobody has waited in vain: whoever
      // had a part in it, or issued the next item's products without waiting for this, would have told it before.
      auto free_o = [&]() {
        ok = __all_sync(0xffffffffu, ok && slot[kAbort] == 0);
        tc::fence_before_sync();
        warp_arrive(bar(kOFree + (k & 1)));
      };
      const bool fix = slot[kAnyPoison + (k & 1)] != 0;
      const uint32_t* notes = poison + (k & 1) * kPoison * 4;
      if (it.slot >= 0) {
        const long long pvec = (long long)it.slot * M + tile * BM + r;
        float* acc = p.part_acc + pvec * D;
#pragma unroll 1
        for (int c = 0; c < OC / 32; ++c) {
          if (!ok || nb == 0 || !warp_live) break;
          float o[32];
          tc::tmem_ld32(tbase + t_lane + L::kOCol + tile * D + c_lo + 32 * c, o);
          tc::tmem_wait_ld();
          // (lanes whose vectors hold nothing skip the stores, not the turn: all of a warp load together)
          if (some || nan) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int d = c_lo + 32 * c + 4 * e;
              float4 vs = make_float4(1.f, 1.f, 1.f, 1.f);
              if (SRC != kF16) {
                if (p.per_channel) vs = __ldg(reinterpret_cast<const float4*>(p.v_scale + it.g * D + d));
                else vs.x = vs.y = vs.z = vs.w = __ldg(p.v_scale);
              }
              const float f = 0.00390625f;
              *reinterpret_cast<float4*>(acc + d) = make_float4(o[4 * e] * f * vs.x, o[4 * e + 1] * f * vs.y,
                                                                o[4 * e + 2] * f * vs.z, o[4 * e + 3] * f * vs.w);
            }
          }
          __syncwarp();
        }
        free_o();
        if (SRC != kI8 && fix && ok && some) add_poison<D, SRC>(p, it, notes, lo, hi, c_lo, c_lo + OC, acc);
        if (live && half == 0) {
          // a CTA that gave up, and a sum that is no number, make the merged row NaN
          p.part_m[pvec] = !ok || nan ? __int_as_float(0x7f800000) : some ? m_nat : neg_inf();
          p.part_l[pvec] = !ok || nan ? kNan : some ? lsum : 0.f;
        }
      } else {
        float sc = 0.f, lse = neg_inf();
        if (nan) {
          sc = lse = kNan;
        } else if (some) {
          lse = m_nat + logf(lsum);
          sc = 0.00390625f / lsum;
          if (p.sink != nullptr) sc *= 1.f / (1.f + expf(__ldg(p.sink + h) - lse));
        }
        // Four lanes write 64 bytes of one row, not each 16 of its own (a store of 32 rows takes four
        // times the turns at the L1 that one of 8 does)
        const long long mine = live ? (it.q.s0 + (long long)tok) * p.Hq + h : -1;
        __half* out = p.out + mine * D;
        long long rows[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = __shfl_sync(0xffffffffu, mine, (lane & 28) + i);
#pragma unroll 1
        for (int c = 0; c < OC / 32; ++c) {
          float o[32];
          tc::tmem_ld32(tbase + t_lane + L::kOCol + tile * D + c_lo + 32 * c, o);
          tc::tmem_wait_ld();
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int d = c_lo + 32 * c + 4 * e;
            float4 vs = make_float4(1.f, 1.f, 1.f, 1.f);
            if (SRC != kF16) {
              if (p.per_channel) vs = __ldg(reinterpret_cast<const float4*>(p.v_scale + it.g * D + d));
              else vs.x = vs.y = vs.z = vs.w = __ldg(p.v_scale);
            }
            const bool z = sc == 0.f;  // nothing attended: the accumulator may hold anything
            w[2 * e] = z ? 0u : sc != sc ? 0x7e007e00u : pack_h2(o[4 * e] * sc * vs.x, o[4 * e + 1] * sc * vs.y);
            w[2 * e + 1] = z ? 0u : sc != sc ? 0x7e007e00u : pack_h2(o[4 * e + 2] * sc * vs.z, o[4 * e + 3] * sc * vs.w);
          }
          across(w, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (rows[i] >= 0)
              *reinterpret_cast<uint4*>(p.out + rows[i] * D + c_lo + 32 * c + 8 * (lane & 3)) =
                  make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        }
        __syncwarp();
        free_o();
        if (!ok) {
          lse = kNan;
          for (int d = c_lo; live && d < c_lo + OC; d += 8)
            *reinterpret_cast<uint4*>(out + d) = make_uint4(0x7e007e00u, 0x7e007e00u, 0x7e007e00u, 0x7e007e00u);
        }
        if (SRC != kI8 && fix && ok && some) add_poison<D, SRC>(p, it, notes, lo, hi, c_lo, c_lo + OC, out);
        if (live && half == 0 && p.lse != nullptr)
          p.lse[(it.q.s0 + (long long)tok) * p.Hq + h] = lse;
      }
      if (!ok) slot[kAbort] = 1;
      give_back(k);
    }
  } else if (warp < (kSoftThreads + kProdThreads) / 32) {
    // -----------------------------------------------------------------------
    // converters; of fp16 sources: the check of V blocks attended in part
    // -----------------------------------------------------------------------
    regs_down<Deal<TILES, SRC>::kProd>();
    const int ct = tid - kSoftThreads;
    const bool folds = SRC != kF16 && p.per_channel;
    const bool flips = SRC != kF16 && !p.per_channel && __ldg(p.k_scale) < 0.f;
    int n = 0;
    Place<Raw<D, TILES, SRC>::kAhead> ring;
    bool ok = true;
    for (int k = 0; take(k); ++k) {
      const Item& it = item_of(k);
      const int nb = ok ? it.blk1 - it.blk0 : 0;
      uint32_t* notes = poison + (k & 1) * kPoison * 4;
      volatile int* any = slot + kAnyPoison + (k & 1);
      // ---- queries into shared memory, once the item before is done with its own ----
      auto stage_queries = [&]() {
        if (ok && k > 0) ok = warp_wait(bar(kQFree), (k - 1) & 1, slot + kAbort);
        const int v0 = it.t * M, nvec = it.q.n * p.G;
        constexpr int CPR = D / 8;  // 16-byte chunks of a vector
        constexpr int kChunks = M * CPR / kProdThreads;
        // chunk i of a thread: of vector (ct + 128 i) / CPR
        auto at = [&](int i, int& row, int& c) -> uint32_t {
          const int idx = ct + kProdThreads * i;
          row = idx / CPR;
          c = idx % CPR;
          return sbase + L::kQ + ((row >> 7) * L::kSlabs + (c >> 3)) * L::kSlab + (row & 127) * 128 +
                 (((c & 7) ^ (row & 7)) << 4);
        };
        if (ct < kPoison * 4) notes[ct] = 0u;
        if (!folds) {
          for (int i = ct; i < M; i += kProdThreads) rscale[(k & 1) * M + i] = 1.f;
        }
        if (ct == 0) slot[kBadPage + (k & 1)] = *any = 0;
        // token and head of the vector, and its address, go on by sums: with a division for each chunk
        // an item of 256 vectors spent 14 500 cycles here, more than on all else
        constexpr int kStep = kProdThreads / CPR;  // vectors from one chunk of a thread to its next
        const int sub = kStep % p.G;
        const long long step = (long long)(kStep / p.G) * p.q_stride + (long long)sub * D;
        const long long wrap = p.q_stride - (long long)p.G * D;  // from behind a token's last head to the next one's first
        const int v_first = v0 + ct / CPR, tok0 = v_first / p.G;
        int j = v_first - tok0 * p.G;
        const __half* src = p.q + (it.q.s0 + (long long)tok0) * p.q_stride + (long long)(it.g * p.G + j) * D + 8 * (ct % CPR);
#pragma unroll 4
        for (int i = 0; i < kChunks; ++i) {
          int row, c;
          const uint32_t dst = at(i, row, c);
          const bool live = ok && v0 + row < nvec;
          cp_async16(dst, live ? src : p.q, live ? 16 : 0);
          j += sub;
          src += step;
          if (j >= p.G) {
            j -= p.G;
            src += wrap;
          }
        }
        asm volatile("bar.sync 9, 128;\n" ::: "memory");  // the notes are clear, the scales 1
        float4 k0 = make_float4(1.f, 1.f, 1.f, 1.f), k1 = k0;  // (a thread's chunks are all of the same channels)
        if (folds) {
          k0 = __ldg(reinterpret_cast<const float4*>(p.k_scale + it.g * D + 8 * (ct % CPR)));
          k1 = __ldg(reinterpret_cast<const float4*>(p.k_scale + it.g * D + 8 * (ct % CPR)) + 1);
        }
        // pages out of range among those attended (their tokens are skipped)
        if (p.table != nullptr) {
          const int lo = first_seen(p, it.q.len - it.q.n + it.first);
          const int hi = min(it.blk1 * BN, it.q.len - it.q.n + it.last + 1);
          const int step = min(p.bs, BN), from = max(it.blk0 * BN, lo);
          bool bad = false;
          // (unsigned: a thread's next step may lie past 2^31)
          if (hi > from)
            for (unsigned t = (unsigned)from + step * ct; t < (unsigned)hi; t += step * kProdThreads)
              bad |= group_of(p, it, (int)t) < 0;
          if (ct == 0 && hi > from) bad |= group_of(p, it, hi - 1) < 0;
          if (bad) {
            slot[kBadPage + (k & 1)] = 1;
            flag_or(p.flags, I8KV_FLAG_BAD_BLOCK);
          }
        }
        cp_async_wait_all();
        // a query that is not finite makes its row NaN whatever its scores come to
        float* scales = rscale + (k & 1) * M;
        if (!folds) {
          uint32_t odd = 0;  // the thread's chunks that hold such a value
#pragma unroll 8
          for (int i = 0; i < kChunks; ++i) {
            int row, c;
            const uint32_t dst = at(i, row, c);
            const uint4 x = lds16(dst);
            odd |= (uint32_t)not_finite(x) << i;
            if (flips) sts16(dst, make_uint4(x.x ^ 0x80008000u, x.y ^ 0x80008000u, x.z ^ 0x80008000u, x.w ^ 0x80008000u));
          }
          for (; odd != 0; odd &= odd - 1) {
            int row, c;
            at(__ffs(odd) - 1, row, c);
            scales[row] = __int_as_float(0x7fc00000);
          }
        } else {
          // Chunks side by side: one after the other, each waits for its vector's maximum through the lanes.
          // (2048 tokens over 16384 by fours / by twos: int8 436 / 444 us, e4m3fn 420 / 425, MX4 436 / 426.)
          constexpr int kSide = TILES == 2 && SRC == kMx4 ? 2 : 4;
#pragma unroll 1
          for (int i = 0; i < kChunks; i += kSide) {
            float f[kSide][8], top[kSide];
            uint32_t odd = 0;
#pragma unroll
            for (int w = 0; w < kSide; ++w) {
              int row, c;
              const uint4 x = lds16(at(i + w, row, c));
              const __half2* h = reinterpret_cast<const __half2*>(&x);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 z = __half22float2(h[e]);
                f[w][2 * e] = z.x;
                f[w][2 * e + 1] = z.y;
              }
              odd |= (uint32_t)not_finite(x) << w;
              f[w][0] *= k0.x, f[w][1] *= k0.y, f[w][2] *= k0.z, f[w][3] *= k0.w;
              f[w][4] *= k1.x, f[w][5] *= k1.y, f[w][6] *= k1.z, f[w][7] *= k1.w;
              top[w] = 0.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) top[w] = fmaxf(top[w], fabsf(f[w][e]));
            }
#pragma unroll
            for (int o = CPR / 2; o > 0; o >>= 1) {
#pragma unroll
              for (int w = 0; w < kSide; ++w) top[w] = fmaxf(top[w], __shfl_xor_sync(0xffffffffu, top[w], o));
              odd |= __shfl_xor_sync(0xffffffffu, odd, o);
            }
#pragma unroll
            for (int w = 0; w < kSide; ++w) {
              int row, c;
              const uint32_t dst = at(i + w, row, c);
              // 2^e brings the largest entry into [2^14, 2^15): exponent fields, exact
              const int ex = (int)((__float_as_uint(top[w]) >> 23) & 255u);
              const int e = ex == 0 || ex == 255 ? 0 : min(max(ex - 127 - 14, -126), 126);
              const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
              for (int u = 0; u < 8; ++u) f[w][u] *= down;
              sts16(dst, make_uint4(pack_h2(f[w][0], f[w][1]), pack_h2(f[w][2], f[w][3]), pack_h2(f[w][4], f[w][5]),
                                    pack_h2(f[w][6], f[w][7])));
              if (c == 0)
                scales[row] = (odd >> w) & 1u ? __int_as_float(0x7fc00000) : __uint_as_float((uint32_t)(127 + e) << 23);
            }
          }
        }
        tc::fence_smem_to_async();
        if (!I8KV_ATTEND_WITHHELD(kHoldQ, k, 0)) warp_arrive(bar(kQFull + (k & 1)));
      };
      if constexpr (SRC == kF16) {
        stage_queries();
        for (int i = 0; ok && i < nb; ++i) {
          const int nn = n + i, blk = it.blk0 + i;
          const bool partial = it.partial(blk);
          uint32_t* bits = notes + 4 * it.ordinal(blk);
          for (int j = 0; j < P; ++j) {
            const int at = spot(nn, j);
            if (!(ok = warp_wait(bar(kVFull + at), turn(nn, j), slot + kAbort))) break;
            if (partial) {
              const uint32_t v = sbase + L::kV + at * L::kPart;
#pragma unroll 4
              for (int k = 0; k < L::kPart / 16 / kProdThreads; ++k) {
                const int q = ct + kProdThreads * k;
                uint4 x = lds16(v + 16 * q);
                if (finite_only(x)) {
                  sts16(v + 16 * q, x);
                  const int row = j * L::kVRows + (q >> 3) % L::kVRows;
                  atomicOr(bits + (row >> 5), 1u << (row & 31));
                  *any = 1;
                }
              }
              tc::fence_smem_to_async();
            }
            warp_arrive(bar(kVOk + at));
          }
        }
      } else {
        // K runs one block ahead of V: K(0), K(1), V(0), K(2), V(1), ...; a run is one block of one of the two
        using R = Raw<D, TILES, SRC>;
        // units to a turn: two, whose waits and loads then go together (of 3300 cycles for a block of 128
        // positions half were waits), where the registers suffice
        constexpr bool kShares = SRC == kMx4 && P == 2;  // both halves of a K block are in the same two units
        constexpr int U = TILES == 1 && R::kRun / P > 1 ? 2 : 1;
        const int blk0 = it.blk0;
        stage_queries();
#pragma unroll 1
        for (int r = 0; ok && r <= 2 * nb; ++r) {
          const bool is_v = r > 0 && (r & 1) == 0;
          const int i = r == 0 ? 0 : is_v ? r / 2 - 1 : (r + 1) / 2;
          if (nb == 0 || (!is_v && i >= nb)) continue;
          const int nn = n + i, blk = blk0 + i;
          uint32_t* bits = SRC != kI8 && is_v && it.partial(blk) ? notes + 4 * it.ordinal(blk) : nullptr;
#pragma unroll 1
          for (int j = 0; ok && j < P; ++j) {
            const int at = spot(nn, j);
            const uint32_t dst = sbase + (is_v ? L::kV : L::kK) + at * L::kPart;
            const bool shares = kShares && !is_v;
            const int here = shares ? 2 : R::kRun / P;
            if (shares && j > 0) ring.back(2);
#pragma unroll 1
            for (int u = 0; ok && u < here; u += U) {
              // MX4: the lanes wait for the units, one of them for the part's place (113.5 -> 107.5 us for four new
              // tokens over 8192 in 16 sequences); the bytes, whose conversion is shorter, one after the other
              // (together 100 -> 108 us).  A place's first turn, and units had before, are waited for in no time.
              constexpr bool kTogether = SRC == kMx4;
              uint32_t from[U], freed[U];
              uint32_t its_bar = bar((is_v ? kVFree : kKFree) + at), its_turn = turn(nn, j) ^ 1;
#pragma unroll
              for (int w = 0; w < U; ++w) {
                from[w] = sbase + R::kAt + ring.place * R::kBytes;
                freed[w] = bar(kRawFree + ring.place);
                if (kTogether) {
                  if (lane % U == w && (lane != 31 || u > 0)) {
                    its_bar = bar(kRawFull + ring.place);
                    its_turn = ring.turn;
                  }
                } else {
                  if (w == 0 && u == 0) ok = warp_wait(its_bar, its_turn, slot + kAbort);
                  ok = warp_wait(bar(kRawFull + ring.place), ring.turn, slot + kAbort) && ok;
                }
                ring.next();
              }
              if (kTogether) {
                ok = warp_wait(its_bar, its_turn, slot + kAbort);
                __syncwarp();  // (the vote in there orders no memory, and a lane reads what others have waited for)
              }
              if constexpr (SRC == kMx4) {
#pragma unroll
                for (int w = 0; w < U; ++w) {
                  if (shares)
                    convert_mx4<D, L::kKSlabs>(ct, from[w], dst, BN, 64 * (u + w), j * L::kKSlabs, nullptr, 0, nullptr);
                  else
                    convert_mx4<D, L::kSlabs>(ct, from[w], dst, is_v ? L::kVRows : BN, 64 * (u + w), 0, bits,
                                              j * L::kVRows + 64 * (u + w), any);
                }
              } else {
                convert_bytes<D, TILES, SRC, U>(ct, from, dst, is_v, u, bits, j * L::kVRows, any);
              }
              if (!shares || j == P - 1) {
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                  for (int w = 0; w < U; ++w) tc::mbar_arrive(freed[w]);
                }
              }
            }
            tc::fence_smem_to_async();
            warp_arrive(bar((is_v ? kVOk : kKFull) + at));
          }
        }
      }
      n += nb;
      if (!ok) slot[kAbort] = 1;
      give_back(k);
    }
  } else {
    regs_down<Deal<TILES, SRC>::kRest>();
    if (warp == kMmaWarp) {
      // ---------------------------------------------------------------------
      // MMA issue
      // ---------------------------------------------------------------------
      constexpr uint32_t kIdQK = tc::idesc_f16(BM, BN, false, false);
      constexpr uint32_t kIdPV = tc::idesc_f16(BM, D, false, true);
      const uint32_t lead = elect_one(), tm = __shfl_sync(0xffffffffu, tbase, 0);
      int n = 0;
      for (int k = 0; take(k); ++k) {
        const Item& it = item_of(k);
        const int nb = __shfl_sync(0xffffffffu, it.blk1 - it.blk0, 0);
        {
          // Q and K: K-major, 64 channels of a row together (the LBO is not used); V: MN-major, 64-channel
          // slabs of the part's positions at LBO
          const uint32_t qd = desc_low(sbase + L::kQ, 16), kd = desc_low(sbase + L::kK, 16);
          const uint32_t vd = desc_low(sbase + L::kV, L::kVRows * 128);
          // After a wait in vain the loop goes on: what is issued then reads and writes nothing but this CTA's own
          // memory, and the wait told the others before, who look once they have read O: its rows become NaN.
          // (Branches on the outcome made the loop 15 % slower, a predicate of the instructions 13 to 25 %.)
          auto wait = [&](int b, uint32_t par) { warp_wait<true>(bar(b), par, slot + kAbort); };
          // scores of tile w (or into buffer nn & 1); the first tile waits for the parts, the last frees them
          auto qk = [&](int w, int nn) {
            const uint32_t qs = qd + w * (L::kSlabs * L::kSlab >> 4);
            const int buf = TILES == 2 ? w : nn & 1;
#pragma unroll
            for (int j = 0; j < P; ++j) {
              const int at = spot(nn, j);
              if (w == 0) wait(kKFull + at, turn(nn, j));
              tc::fence_after_sync();
              const uint32_t ks = kd + at * (L::kPart >> 4);
#pragma unroll
              for (int kk = 0; kk < 4 * L::kKSlabs; ++kk) {
                const int in_slab = (kk >> 2) * L::kSlab + (kk & 3) * 32;
                mma_ss(lead, tm + buf * BN, qs + ((j * L::kKSlabs * L::kSlab + in_slab) >> 4), ks + (in_slab >> 4), kIdQK,
                       j > 0 || kk > 0);
              }
              // (a commit takes its time: those that the softmax waits for come first)
              if (j == P - 1) commit(lead, bar(kSFull + buf));
              if (w == TILES - 1) commit(lead, bar(kKFree + at));
            }
          };
          // O of tile w; P in two halves with two tiles
          auto pv = [&](int w, int nn, bool first) {
            const int buf = TILES == 2 ? w : nn & 1;
            constexpr int kSteps = 8 / P;  // of 16 positions in a part
#pragma unroll
            for (int j = 0; j < P; ++j) {
              const int at = spot(nn, j);
              const uint32_t vs = vd + at * (L::kPart >> 4);
              if (w == 0) wait(kVOk + at, turn(nn, j));
#pragma unroll
              for (int k = 0; k < kSteps; ++k) {
                const int kk = j * kSteps + k;
                if (kk == 0 || (TILES == 2 && kk == 4)) wait((TILES == 2 && kk == 0 ? kPHalf : kPFull) + w, nn & 1);
                if (k == 0 || (TILES == 2 && kk == 4)) tc::fence_after_sync();
                mma_ts(lead, tm + L::kOCol + w * D, tm + buf * BN + 64 * (kk >> 2) + 8 * (kk & 3),
                       vs + (k * 2048 >> 4), kIdPV, !first || kk > 0);
              }
              if (j == P - 1) commit(lead, bar(kPVDone + w));
              if (w == TILES - 1) commit(lead, bar(kVFree + at));
            }
          };
          wait(kQFull + (k & 1), (k >> 1) & 1);
          tc::fence_after_sync();
          // the first product of an item goes over O: the item before must have been read
          auto o_free = [&]() {
            if (k > 0) wait(kOFree + ((k - 1) & 1), ((k - 1) >> 1) & 1);
          };
          if constexpr (TILES == 2) {
            // (a tile without vectors is worked on too, so that the barriers keep step)
            // Scores go over the probabilities of the block before, of the item before where this one
            // begins: their product must have read them.
            if (nb > 0) {
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                if (n > 0) wait(kPVDone + w, (n - 1) & 1);
                qk(w, n);
              }
              if (nb == 1) commit(lead, bar(kQFree));
              o_free();
            }
#pragma unroll 1
            for (int nn = n; nn < n + nb; ++nn) {
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                pv(w, nn, nn == n);
                if (nn + 1 < n + nb) {
                  wait(kPVDone + w, nn & 1);
                  qk(w, nn + 1);
                }
              }
              if (nn + 2 == n + nb) commit(lead, bar(kQFree));
            }
          } else {
            // QK(0), QK(1), PV(0), QK(2), PV(1), ...; every PVDone is waited for once, and one at most is to come
#pragma unroll 1
            for (int i = 0; i <= nb; ++i) {
              const int nn = n + i;
              // S(i) goes over P(i - 2); an item's first one waits for the last product of the item before
              if (i >= 2) wait(kPVDone, nn & 1);
              else if (i == 0 && nb > 0 && nn > 0) wait(kPVDone, (nn - 1) & 1);
              if (i < nb) {
                qk(0, nn);
                if (i == nb - 1) commit(lead, bar(kQFree));
              }
              if (i == 1) o_free();
              if (i > 0) pv(0, nn - 1, i == 1);
            }
          }
          if (nb == 0) {
            o_free();
            commit(lead, bar(kQFree));
          }
        }
        n += nb;
        give_back(k);
      }
      // everything issued has completed before the tensor memory is given back
      commit(lead, bar(kDone));
      if (!tc::mbar_wait(bar(kDone), 0)) slot[kAbort] = 1;
      __syncwarp();
    } else if (warp == kLastWarp) {
      // ---------------------------------------------------------------------
      // the items
      // ---------------------------------------------------------------------
      Walk walk;
      Item one;
      start_walk<M>(p, one, walk);
      for (int k = 0;; ++k) {
        one.has = next_item<M>(p, one, walk);
        if (k >= 2 && !wait_item(kItemFree + (k & 1), ((k >> 1) & 1) ^ 1)) break;
        if (lane == 0) *reinterpret_cast<Item*>(smem + L::kItem + 128 * (k & 1)) = one;
        warp_arrive(bar(kItemFull + (k & 1)));
        if (!one.has) break;
      }
      if (blockIdx.x == 0)  // lengths and starts that had to be clamped
        for (int b = lane; b < p.B; b += 32) seq_of(p, b, true);
    } else {
      // ---------------------------------------------------------------------
      // copies of fp16 parts, and of units of codes
      // ---------------------------------------------------------------------
      int n = 0;
      bool ok = true;
      int nk = 0, nv = 0;  // parts begun
      int units = 0;       // units begun
      constexpr int kBoxes = SRC == kF16 ? 8 : Raw<D, TILES, SRC>::kRows / 16;  // of a unit of codes
      constexpr int kStep = Raw<D, TILES, SRC>::kAhead >= 6 ? 8 / kBoxes : 1;
      constexpr int kAsk = kBoxes * kStep;  // lanes that ask for data
      const int my_unit = lane / kBoxes % kStep;  // of a step
      Place<Raw<D, TILES, SRC>::kAhead> ring;
      if (my_unit == 1) ring.next();
      for (int k = 0; warp == kTmaWarp && take(k); ++k) {
        const Item& it = item_of(k);
        const int nb = ok ? it.blk1 - it.blk0 : 0;
        if (SRC == kF16) {
          const bool paged = p.table != nullptr;
          // pages: boxes of 16 rows, a lane each (slab-major: group i of the part, slab i / groups); packed rows: a box for
          // each slab of the part
          constexpr int kVGroups = L::kVRows / 16;
          // (the table is read a block before its pages are asked for)
          const int blk0 = it.blk0, blk1 = it.blk1;
          auto pages_of = [&](int blk) -> int { return blk < blk1 ? page_of(p, it, blk * BN + 16 * (lane & 7)) : -1; };
          auto groups_of = [&](int blk, int page) -> int {  // first row of group lane % 8
            const int grp = group_in(p, page, blk * BN + 16 * (lane & 7));
            return grp < 0 ? p.rows : grp * 16;  // (a row past the end is read as zeros)
          };
          auto copy = [&](int i, int j, bool is_v, int groups) -> bool {
            const int nn = n + i, at = spot(nn, j), full = (is_v ? kVFull : kKFull) + at;
            if (nn * P + j >= N && !warp_wait(bar((is_v ? kVFree : kKFree) + at), turn(nn, j) ^ 1, slot + kAbort))
              return false;
            ++(is_v ? nv : nk);
            if (I8KV_ATTEND_WITHHELD(is_v ? kHoldV : kHoldK, k, i)) return true;
            if (lane == 0) tc::mbar_arrive_expect_tx(bar(full), L::kPart);
            int slab, row;
            bool mine;
            uint32_t dst = sbase + (is_v ? L::kV : L::kK) + at * L::kPart;
            if (paged) {
              const int groups_here = is_v ? kVGroups : 8;
              const int grp = lane % groups_here;
              slab = lane / groups_here;
              row = __shfl_sync(0xffffffffu, groups, grp + (is_v ? j * kVGroups : 0));
              mine = slab < (is_v ? L::kSlabs : L::kKSlabs);
              dst += lane * 2048;
            } else {
              row = it.q.s0 + (it.blk0 + i) * BN + (is_v ? j * L::kVRows : 0);
              slab = lane;
              mine = slab < (is_v ? L::kSlabs : L::kKSlabs);
              dst += slab * (is_v ? L::kVRows : BN) * 128;
            }
            if (!is_v) slab += j * L::kKSlabs;
            __syncwarp();
            if (mine) tma_box(dst, is_v ? &a.vm : &a.km, 64 * slab, it.g, row, bar(full));
            return true;
          };
          int g0 = 0, g1 = 0, next = 0;
          if (paged) {
            const int first = pages_of(blk0);
            next = pages_of(blk0 + 1);
            g1 = groups_of(blk0, first);
          }
          for (int i = -1; ok && i < nb; ++i) {  // K runs one block ahead of V
            for (int j = 0; ok && i + 1 < nb && j < P; ++j) ok = copy(i + 1, j, false, g1);
            for (int j = 0; ok && i >= 0 && j < P; ++j) ok = copy(i, j, true, g0);
            if (paged) {
              g0 = g1;
              g1 = groups_of(blk0 + i + 2, next);
              next = pages_of(blk0 + i + 3);
            }
          }
        } else {
          // Up to two units to a step, whose 8 boxes or record halves 8 lanes ask for, each after a look at its own
          // unit's place (one unit at a time took 600 cycles each, and all others waited for the data)
          using R = Raw<D, TILES, SRC>;
          const int blk0 = it.blk0, blk1 = it.blk1;
          auto pages_of = [&](int blk) -> int {  // of group lane % 8 of the block, read a block ahead
            return blk < blk1 ? page_of(p, it, blk * BN + 16 * (lane & 7)) : -1;
          };
          auto groups_of = [&](int blk, int page) -> int { return group_in(p, page, blk * BN + 16 * (lane & 7)); };
          const int first = pages_of(blk0);
          int next = pages_of(blk0 + 1);
          int gk = groups_of(blk0, first), gv = 0;
          for (int r = 0; ok && r <= 2 * nb; ++r) {  // runs as the converters take them
            const bool is_v = r > 0 && (r & 1) == 0;
            if (r & 1) {
              const int blk = blk0 + (r + 1) / 2;
              gv = gk;
              gk = groups_of(blk, next);
              next = pages_of(blk + 1);
            }
            if (nb == 0 || (!is_v && (r + 1) / 2 >= nb)) continue;
            for (int ru = 0; ru < R::kRun; ru += kStep) {
              const int full = bar(kRawFull + ring.place);
              const uint32_t dst = sbase + R::kAt + ring.place * R::kBytes;
              if (!(ok = warp_wait(bar(kRawFree + ring.place), ring.turn ^ 1, slot + kAbort))) break;
              if (I8KV_ATTEND_WITHHELD(is_v ? kHoldV : kHoldK, k, is_v ? r / 2 - 1 : (r + 1) / 2)) {
                r = 2 * nb;
                break;
              }
              units += kStep;
#pragma unroll
              for (int w = 0; w < kStep; ++w) ring.next();
              const int unit = ru + my_unit, box = lane % kBoxes;
              if constexpr (SRC == kMx4) {
                const int grp = __shfl_sync(0xffffffffu, is_v ? gv : gk, 4 * unit + box);
                const uint32_t here = dst + box * 9 * D;
                const bool copies = lane < kAsk && grp >= 0;
                if (copies) {
                  const int tiles = p.bs >> 4;
                  const int page = p.bs_log2 >= 0 ? grp >> (p.bs_log2 - 4) : grp / tiles;
                  tc::bulk_g2s(here, reinterpret_cast<const uint8_t*>(p.k) +
                                         (((long long)page * p.Hkv + it.g) * tiles + (grp - page * tiles)) * (18LL * D) +
                                         (is_v ? 9 * D : 0),
                               9 * D, full);
                } else if (lane < kAsk) {
                  for (int b = 0; b < 9 * D; b += 16) sts16(here + b, make_uint4(0u, 0u, 0u, 0u));
                }
                // (bytes that land before they are announced are counted all the same)
                const unsigned mask = __ballot_sync(0xffffffffu, copies) >> (lane & ~3) & 15u;
                __syncwarp();  // the zeros are there
                if (lane < kAsk && box == 0) tc::mbar_arrive_expect_tx(full, __popc(mask) * 9 * D);
              } else {
                // rows of the block and channels that the unit has
                const int j = unit / (R::kRun / P), u = unit % (R::kRun / P);
                const int row0 = (is_v ? j * L::kVRows : 0) + R::first_row(u, is_v);
                const int c0 = 64 * ((is_v ? 0 : j * L::kKSlabs) + R::first_slab(u, is_v));
                if (lane < kAsk && box == 0) tc::mbar_arrive_expect_tx(full, R::kBytes);
                const int grp = __shfl_sync(0xffffffffu, is_v ? gv : gk, row0 / 16 + box);
                __syncwarp();
                if (lane < kAsk)  // (a row past the end is read as zeros)
                  tma_box(dst + box * 16 * R::kWide, is_v ? &a.vm : &a.km, c0, it.g, grp < 0 ? p.rows : grp * 16, full);
              }
            }
          }
        }
        if (!ok) slot[kAbort] = 1;
        n += nb;
        give_back(k);
      }
      // every copy begun has landed before the CTA ends (the last ones of each place)
      if (lane == 0) {
        auto landed = [&](int b, int turn) {
          if (!tc::mbar_wait(bar(b), turn & 1, nullptr, I8KV_ATTEND_WAIT_NS)) slot[kAbort] = 1;
        };
        constexpr int kAhead = Raw<D, TILES, SRC>::kAhead;
        if constexpr (SRC != kF16)
          for (int k = max(0, units - kAhead); k < units; ++k) landed(kRawFull + k % kAhead, k / kAhead);
        for (int k = max(0, nk - N); k < nk; ++k) landed(kKFull + k % N, k / N);
        for (int k = max(0, nv - N); k < nv; ++k) landed(kVFull + k % N, k / N);
      }
      __syncwarp();
    }
  }
  tc::fence_before_sync();
  sync_all();
  if (tid == 0 && slot[kAbort] != 0) flag_or(p.flags, I8KV_FLAG_WAIT_TIMEOUT);  // whichever role gave up
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, 512);
  }
}

}  // namespace ap
}  // namespace i8kv
