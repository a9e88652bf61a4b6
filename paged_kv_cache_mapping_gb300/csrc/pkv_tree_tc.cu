// pkv_tree_tc.cu -- attention of drafted trees over the paged cache on the
// fifth-generation tensor cores, split along the keys.
//
// What it computes: the q_s nodes of sequence s times the G query heads of a
// KV head are R = q_s * G rows that all read the same keys: every row sees the
// context, and a drafted key is seen by the nodes whose mask has its bit.  A
// verification step has few rows (R of 16 to a few hundred) and many keys, so
// the key axis is the long one; it is put on the MMA's M side:
//     S^T = K Q^T      (M 128 keys, N rows, K = D)
//     O^T += V^T P^T   (M = D, N rows, K 128 keys)
// so that the cost of a tile follows the number of rows (N 16, 32 or 64), not
// a fixed 128, and the softmax works on 128 keys x N rows spread over all
// lanes: a lane is a key, a register a row.  Per-row statistics would need a
// reduction over lanes for each tile; instead a row keeps a reference (its
// largest score when it was last set) and p = 2^(s - ref) may grow to 2^tau
// above it: a tile only votes whether any score passed that bound, and only
// then (and in each item's first tile, and where a mask cuts) the column
// maxima are reduced, the references of the rows that passed it move, and O is
// rescaled in tensor memory.  A row's references depend on its own scores only,
// so its result does not depend on the rows beside it.
//
// Work: an item is (sequence, chunk of keys, KV head, tile of N rows).  The
// chunk length follows from the sequence's own length and node count and the
// call's shapes, not from the other sequences (tree_chunk).  Chunks write normalised partials and log2-sum-exp2, and a second small kernel joins
// them in order.  Items are dealt to the persistent CTAs (one per SM) in
// strides; every CTA finds its items by scanning the lengths, 32 sequences per
// step, so a call needs no plan, keeps nothing between calls, and its
// workspace holds only the partials.
//
// Types: bf16 caches take bf16 MMAs, P as bf16 hi + lo (about 16 bits).  e4m3
// caches take the codes as they are (kind::f8f6f4, no conversion): a query row
// is scaled to a largest element in [128, 256) and split into two e4m3 parts
// (a bf16 element has 8 significant bits, an e4m3 code 4: hi + lo is exact down
// to 2^-18 of the row's largest element), and P = 16 * 2^(s - ref) <= 2^8.5 into
// hi and lo, lo scaled by 16 with an accumulator of its own, so that the
// smallest codes' step is 2^-17 of the row's reference.
//
// CTA: 16 warps.
//   warps 0, 3  copy the K and the V tiles of 128 keys by TMA: boxes of 16 or 8
//               slots that lie in one block, or, for other block sizes, four
//               arbitrary rows at a time (tile::gather4).
//   warp 1      issues the MMAs: S of tile g + 1, then P V of tile g.  The two
//               parts of P are 2 N columns of one operand, so O holds their two
//               products side by side and P V costs one pass of instructions.
//   warp 2      finds the items, publishes them and brings their query rows:
//               bf16 to the swizzled operand layout, or split to e4m3.
//   then 8 or 16 (N = 64) warps of softmax: lane quarter w % 4 = keys, group
//               (w - 4) / 4 = rows.
//   and 4 warps that write O / l of finished items while the next one runs.
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "pkv_kernels.h"

namespace pkv {
namespace {

constexpr int kKeys = 128;  // keys per tile (M of S^T, K of P V)
constexpr int kItemSlots = 6;
constexpr int kInfoSlots = 8;

// ---------------------------------------------------------------- chunking
// Keys per chunk, from the sequence's own length and node count and from how
// many (sequence, KV head, row tile) units the call has: few units are cut
// finely so that every SM has work, many are cut coarsely, since each chunk
// costs its rows' partials (512 bytes per row and head, written and read) and
// an item's start and end.  At least `least` keys, at most `most` chunks, and
// at most kTreePartRows / q_s of them, so that a sequence has at most that many
// partial rows per head.
constexpr int kTreeMaxChunks = 64;
constexpr int kTreePartRows = 1024;
struct Chunking {
  int32_t least, most;
};
inline Chunking tree_chunking(int64_t units) {
  Chunking c;
  c.least = units >= 512 ? 1024 : units >= 128 ? 512 : 256;
  const int64_t m = 2432 / (units < 1 ? 1 : units);  // 16 items per SM
  c.most = static_cast<int32_t>(m < 8 ? 8 : m > kTreeMaxChunks ? kTreeMaxChunks : m);
  return c;
}

__host__ __device__ inline int tree_chunk(int n, int q_s, Chunking k) {
  const int rows = kTreePartRows / q_s;
  const int most = rows < 1 ? 1 : rows < k.most ? rows : k.most;
  const int c = ((n - 1) / most / kKeys + 1) * kKeys;  // ceil(n / most) in whole tiles; n < 2^31 - 128
  return most > 1 && c < k.least ? k.least : c;
}

// ---------------------------------------------------------------- geometry
constexpr int kMiscBytes = 6656;
template <int D, int N, bool F8>
struct Geo {
  static constexpr int kEs = F8 ? 1 : 2;
  static constexpr int kRowB = D * kEs;                       // one K or V row
  static constexpr int kAtomB = kRowB < 128 ? kRowB : 128;    // swizzle width
  static constexpr int kSub = kRowB / kAtomB;                 // sub-tiles along d
  static constexpr int kTileB = kKeys * kRowB;
  static constexpr int kParts = F8 ? 2 : 1;                   // parts of Q
  static constexpr int kQB = N * kRowB * kParts;
  static constexpr int kPRow = 2 * N * kEs;                   // both parts of P of one key
  static constexpr int kPB = kKeys * (kPRow <= 128 ? 128 : 256);  // [1 or 2][128 keys][128 bytes]
  static constexpr int kNK = kTileB == 32768 ? 2 : kTileB == 16384 ? 4 : 6;
  static constexpr int kNV = kTileB == 32768 ? (kPRow == 256 ? 2 : 3) : kTileB == 16384 ? (kPRow == 256 ? 4 : 5) : 6;
  static constexpr int kGroups = N == 64 ? 4 : 2;             // softmax: groups of four warps, each N / kGroups rows
  static constexpr int kSoft = 4 * kGroups;                   // its warps
  static constexpr int kThreads = 32 * (4 + kSoft + 4);
  static constexpr int kNC = N / kGroups;                     // rows (columns of S^T) per softmax warp
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kNK * kTileB;
  static constexpr int kOffP = kOffV + kNV * kTileB;
  static constexpr int kOffQ = kOffP + 2 * kPB;
  static constexpr int kQBufs = kPRow == 256 && kTileB == 32768 ? 1 : 2;  // query tiles: the next item's arrives while this one runs
  static constexpr int kOffMisc = kOffQ + kQBufs * kQB;
  static constexpr int kSmem = kOffMisc + kMiscBytes;
  // tensor memory: S 2 x N columns, then O 2 x (hi N, lo N)
  static constexpr uint32_t kColO = 2 * N;
  static constexpr uint32_t kOCols = 2 * N;
  static constexpr int kKeyStep = F8 ? 32 : 16;               // keys per MMA k step of P V
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kNK + 2 <= kInfoSlots, "tile info ring");
  static_assert(kColO + 2 * kOCols <= 512, "tensor memory");
};

struct alignas(16) Item {
  int s, h, r0;         // sequence, KV head, first row of the tile
  int t0, q_s, n;       // first packed row, nodes, keys
  int k0, k1;           // keys of the chunk
  int c, nchunks;       // its index, chunks of the sequence
  int nt, pad;          // key tiles (0: no more items)
};

// barrier area
enum : int {
  kBKFull = 0, kBKEmpty = 6, kBVFull = 12, kBVEmpty = 18, kBSFull = 24, kBPFull = 26 /* 2 */, kBOFull = 28,
  kBOFree = 30, kBQFull = 32, kBQEmpty = 34, kBQsFull = 36, kBLFull = 40, kBLEmpty = 42, kBItemFull = 44,
  kBItemEmpty = 50, kBODone = 56, kBDrain = 57, kBGroup = 58 /* 4 */, kSTmem = 62, kSAbort = 63, kSPoison = 64 /* [3] ints: 64, 65 */,
  kOffItems = 528, kOffInfo = 816, kOffXch = 944 /* [groups][4][rows] */, kOffSum = 1968 /* [2][4][64] */,
  kOffLref = 4016 /* [2][64] */, kOffRef = 4528 /* [3][64] */, kOffQs = 5296 /* e4m3: [4][64] */,
  kOffUnset = 6320 /* [groups][4] */, kOffFlag = 6384 /* [groups][2] */,
};
static_assert(kOffFlag + 32 <= kMiscBytes, "shared memory");
static_assert(kOffItems + kItemSlots * (int)sizeof(Item) <= kOffInfo, "item ring");

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo, int atom) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFF) << 32) | (1ull << 46) | ((uint64_t)(atom == 128 ? 2 : 4) << 61);
}

// instruction descriptor: fp32 accumulator, A and B bf16 (or e4m3), M 128, N n
__host__ __device__ constexpr uint32_t idesc(int n, bool f8, bool a_mn, bool b_mn) {
  return (1u << 4) | ((f8 ? 0u : 1u) << 7) | ((f8 ? 0u : 1u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}


__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
template <bool F8, int kSteps, int kA, int kB>
__device__ __forceinline__ void mma_steps(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    if constexpr (F8) {
      asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a + k * kA), "l"(b + k * kB), "r"(id), "r"(k ? 1u : acc));
    } else {
      asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a + k * kA), "l"(b + k * kB), "r"(id), "r"(k ? 1u : acc));
    }
  }
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// n (8, 16 or 32) consecutive fp32 columns of this thread's tensor memory lane
__device__ __forceinline__ void tm_ld(uint32_t a, uint32_t (&x)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
               : "r"(a));
}
__device__ __forceinline__ void tm_st(uint32_t a, const uint32_t (&x)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]));
}
#define PKV_O16(x) \
  "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), \
      "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
__device__ __forceinline__ void tm_ld(uint32_t a, uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : PKV_O16(x)
      : "r"(a));
}
__device__ __forceinline__ void tm_ld(uint32_t a, uint32_t (&x)[32]) {
  uint32_t(&lo)[16] = *reinterpret_cast<uint32_t(*)[16]>(&x[0]);
  uint32_t(&hi)[16] = *reinterpret_cast<uint32_t(*)[16]>(&x[16]);
  tm_ld(a, lo);
  tm_ld(a + 16, hi);
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar,
                                        uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(pol)
      : "memory");
}
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int c0, const int (&r)[4],
                                            uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar), "l"(pol)
      : "memory");
}
__device__ __forceinline__ uint64_t l2_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// A bounded wait, and the same by a whole warp: at most 2^18 tries, each of
// which may suspend the warp for up to 20 us (5 s in all).  Without the time
// hint a try comes back after some tens of clocks, and the waiting warps' tries
// took half of the SM's issue slots.  The code is kept short, here and below:
// sixteen and more warps in six roles share the SM's instruction cache, and
// while the roles' code did not fit (105 to 166 KB in all, 42 % of its requests
// missed) it set the pace, not the pipes.
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n"
      "W:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t@p bra D;\n\t"
      "add.u32 n, n, 1;\n\tsetp.lt.u32 q, n, 262144;\n\t@q bra W;\n"
      "D:\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, poll(bar, parity));
}
// A place in a ring of n slots, and the parity of its pass.
struct Ring {
  int at = 0;
  uint32_t pass = 0;
  __device__ __forceinline__ void next(int n) {
    if (++at == n) {
      at = 0;
      pass ^= 1;
    }
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// three-input max: exact, like two fmaxf
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// packed pairs of fp32: one instruction does two lanes' worth of work
__device__ __forceinline__ unsigned long long pk2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void up2(unsigned long long v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long sub2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ void st_s128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void st_s64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// largest of a warp's values, NaN passed over
__device__ __forceinline__ float redux_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint16_t f16x2_to_e4m3x2(__half2 h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&h)));
  return r;
}

// 16-byte chunk c of row r in a swizzled [rows][atom bytes] tile
template <int kAtomB>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return kAtomB == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Adds NC columns up over the 32 lanes by halving: afterwards every lane holds
// column lane / (32 / NC)'s sum.
template <int NC>
__device__ __forceinline__ float col_sum(float (&v)[NC], int lane) {
  int w = NC;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    if (w > 1) {
      w >>= 1;
      const bool up = lane & s;
#pragma unroll
      for (int j = 0; j < NC / 2; ++j) {
        if (j < w) {
          const float send = up ? v[j] : v[j + w], keep = up ? v[j + w] : v[j];
          v[j] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], s);
    }
  }
  return v[0];
}

// Division of 0 <= x < 2^31 by a constant d >= 1 of the call: one multiply-high
// and a shift.  M = floor(2^(32 + s) / d) + 1 with 2^s < d <= 2^(s + 1): M fits
// 32 bits, x M / 2^(32 + s) passes x / d by at most x / 2^(32 + s) < 1 / d, so
// the floor is exact.  d = 1 is x itself.
struct FastDiv {
  uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while (f.s < 31 && (2u << f.s) < d) ++f.s;
  if (d > 1) f.m = static_cast<uint32_t>(((uint64_t)1 << (32 + f.s)) / d + 1);
  return f;
}
__device__ __forceinline__ int quot(int x, const FastDiv& f) {
  return f.d == 1 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), f.m) >> f.s);
}

struct TcArgs {
  TreeParams p;
  FastDiv by_g, by_bs;
  int32_t rows_per_seq;  // partial rows of a sequence
  Chunking chunking;
  int32_t box;           // slots per TMA box, 0: gather4
  int32_t out_bf16;
  float* part_o;         // [B * rows_per_seq, Hq, D] normalised chunk outputs
  float* part_lse;       // [B * rows_per_seq, Hq]
};

// A drafted value (element d of some V row) is not finite: the softmax warps
// took it out of the product, and here it goes to the rows that see its key,
// on top of what this thread has just stored.
template <int D, int N, bool F8>
__device__ __noinline__ void add_poison(const TcArgs& a, const Item& it, int d) {
  const TreeParams& p = a.p;
  const int ctx = it.n - it.q_s, rows = it.q_s * p.G;
  for (int k = max(ctx, it.k0); k < it.k1; ++k) {
    const int lb = k / p.bs, jj = k - ctx;
    const int32_t blk = __ldg(p.bt + (int64_t)it.s * p.bt_stride + lb);
    if ((uint32_t)blk >= (uint64_t)p.num_blocks) continue;
    const int64_t va = (((int64_t)blk * p.bs + (k - lb * p.bs)) * p.Hkv + it.h) * D + d;
    float x;
    if constexpr (F8) {
      const uint32_t hf = e4m3x2_to_f16x2(static_cast<const uint8_t*>(p.v_cache)[va]);
      x = __half2float(__ushort_as_half(static_cast<unsigned short>(hf & 0xffffu)));
    } else {
      x = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_cache)[va]);
    }
    if (fabsf(x) < INFINITY) continue;
    for (int r = it.r0; r < rows && r < it.r0 + N; ++r) {
      const int i = r / p.G, hq = it.h * p.G + r - i * p.G;
      if (!((static_cast<uint32_t>(__ldg(p.mask + (int64_t)(it.t0 + i) * p.mask_stride + (jj >> 5))) >> (jj & 31)) & 1u)) continue;
      if (it.nchunks > 1) {
        a.part_o[(((int64_t)it.s * a.rows_per_seq + (int64_t)i * it.nchunks + it.c) * p.Hq + hq) * D + d] += x;
      } else {
        const int64_t at = (int64_t)(it.t0 + i) * p.o_st + (int64_t)hq * p.o_sh + d;
        if (a.out_bf16) {
          __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.out) + at;
          *y = __float2bfloat16_rn(__bfloat162float(*y) + x);
        } else {
          static_cast<float*>(p.out)[at] += x;
        }
      }
    }
  }
}

template <int D, int N, bool F8>
__global__ void __launch_bounds__(Geo<D, N, F8>::kThreads, 1)
    tree_tc_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v) {
  using G_ = Geo<D, N, F8>;
  constexpr int NC = G_::kNC, NK = G_::kNK, NV = G_::kNV, AT = G_::kAtomB;
  const TreeParams& p = a.p;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* misc = smem + G_::kOffMisc;
  const uint32_t s0 = smem_u32(smem), b0 = smem_u32(misc);
  auto bar = [&](int i) -> uint32_t { return b0 + 8 * i; };
  const uint32_t sK = s0 + G_::kOffK, sV = s0 + G_::kOffV, sP = s0 + G_::kOffP, sQ = s0 + G_::kOffQ;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 8 * kSAbort);
  volatile int* poison = reinterpret_cast<volatile int*>(misc + 8 * kSPoison);  // [3]: item + 1
  uint32_t* tslot = reinterpret_cast<uint32_t*>(misc + 8 * kSTmem);
  Item* items = reinterpret_cast<Item*>(misc + kOffItems);
  uint32_t* info = reinterpret_cast<uint32_t*>(misc + kOffInfo);  // [kInfoSlots][4]: keys without a page
  float* xch = reinterpret_cast<float*>(misc + kOffXch);          // [groups][4 quarters][32]
  float* sums = reinterpret_cast<float*>(misc + kOffSum);         // [2][4 quarters][64]: rows' sums of p
  float* lref = reinterpret_cast<float*>(misc + kOffLref);        // [2][64]: their references, as kept
  float* refs = reinterpret_cast<float*>(misc + kOffRef);         // [3][64]
  volatile uint32_t* unset4 = reinterpret_cast<volatile uint32_t*>(misc + kOffUnset);  // [2 halves][4 quarters]
  float* qscale = reinterpret_cast<float*>(misc + kOffQs);        // e4m3: [4][64]
  // the shuffle tells the compiler that the warp index, and so the branch to a
  // role, is the same for the whole warp: else every warp-wide instruction
  // inside is compiled for a diverged warp
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  auto aborted = [&]() -> bool { return __any_sync(0xffffffffu, *abort_flag != 0); };
  const int G = p.G, Hkv = p.Hkv;

  if (s0 & 1023) {  // the swizzled tiles need their base on 1024 bytes
    if (threadIdx.x == 0) atomicOr(p.err, kErrWaitTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(bar(kBKFull + i), 1);
      mbar_init(bar(kBKEmpty + i), 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(bar(kBVFull + i), 1);
      mbar_init(bar(kBVEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBSFull + i), 2);
      mbar_init(bar(kBOFull + i), 1);
      mbar_init(bar(kBOFree + i), 4);
      mbar_init(bar(kBQFull + i), 1);
      mbar_init(bar(kBQEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBLFull + i), G_::kSoft);
      mbar_init(bar(kBLEmpty + i), 4);
    }
    for (int i = 0; i < 2; ++i) mbar_init(bar(kBPFull + i), G_::kSoft);
    mbar_init(bar(kBODone), 1);
    for (int i = 0; i < G_::kGroups; ++i) mbar_init(bar(kBGroup + i), 4);
    for (int i = 0; i < 4; ++i) mbar_init(bar(kBQsFull + i), 1);
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(bar(kBItemFull + i), 1);
      mbar_init(bar(kBItemEmpty + i), 3 + G_::kSoft + 4);  // every warp but the finder
    }
    mbar_init(bar(kBDrain), 1);
    *abort_flag = 0;
    for (int i = 0; i < 3; ++i) poison[i] = 0;
    for (int i = 0; i < 8; ++i) reinterpret_cast<volatile int*>(misc + kOffFlag)[i] = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane ? &tm_v : &tm_k)) : "memory");
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tslot;
  grid_dep_wait();
  launch_dependents();

  // item j's query buffer, and the parity of its pass
  auto qbuf = [](int j) { return G_::kQBufs == 2 ? j & 1 : 0; };
  auto qpass = [](int j) { return (uint32_t)(G_::kQBufs == 2 ? j >> 1 : j) & 1u; };
  // the next item, as every warp but the finder takes it
  auto take = [&](Ring& r, Item& it) -> bool {
    if (!wait_bar(bar(kBItemFull) + 8 * r.at, r.pass)) return false;
    const int4* q = reinterpret_cast<const int4*>(items + r.at);
    *reinterpret_cast<int4*>(&it) = q[0];
    *(reinterpret_cast<int4*>(&it) + 1) = q[1];
    *(reinterpret_cast<int4*>(&it) + 2) = q[2];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBItemEmpty) + 8 * r.at);
    r.next(kItemSlots);
    return !aborted();
  };

  // ---- copies of K or V tiles: pages, slots, TMA
  const int bx = a.box;
  const int n_box = bx ? kKeys / bx : 32;
  const int key_of = bx ? (lane % n_box) * bx : lane * 4;  // first key of this lane's box (or four keys)
  constexpr int32_t kPast = INT32_MIN;
  // pages of this lane's keys in a tile (one box's, or four keys')
  auto pages = [&](const Item& it, int t, int32_t (&blk)[4]) {
    const int32_t* row = p.bt + (int64_t)it.s * p.bt_stride;
    const int k = it.k0 + t * kKeys + key_of;
    if (bx) {
      blk[0] = k < it.k1 ? __ldg(row + quot(k, a.by_bs)) : kPast;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) blk[e] = k + e < it.k1 ? __ldg(row + quot(k + e, a.by_bs)) : kPast;
    }
  };
  // slots of this lane's keys (-1: none); returns those whose page is out of range
  auto slots = [&](const Item& it, int t, const int32_t (&blk)[4], int (&sl)[4]) -> uint32_t {
    const int k = it.k0 + t * kKeys + key_of;
    auto one = [&](int e) -> uint32_t {
      const bool in = (uint32_t)blk[e] < (uint32_t)p.num_blocks;
      sl[e] = in ? (blk[e] - quot(k + e, a.by_bs)) * p.bs + k + e : -1;
      return !in && blk[e] != kPast ? 1u << e : 0u;
    };
    return bx ? one(0) : one(0) | one(1) | one(2) | one(3);
  };
  // Copies a tile into dst.  The copies are issued by one elected lane, each
  // box's slot handed over by a shuffle: the instruction takes its operands
  // from uniform registers, and lanes that issue one copy each are served one
  // after the other at about 150 clocks (2,450 for a bf16 tile's 16 boxes).
  auto load_tile = [&](int h, const int (&sl)[4], uint32_t dst, const CUtensorMap* map, uint32_t full, uint64_t pol) {
    if (lane == 0) mbar_arrive_expect_tx(full, G_::kTileB);
    __syncwarp();
    if (bx) {
      // past the sequence, or a page out of range: out of bounds, which TMA fills with zeros
      const int mine = sl[0] >= 0 ? sl[0] : (int)(p.num_blocks * p.bs);
#pragma unroll 1
      for (int b = 0; b < n_box; b += 8) {
        int s8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) s8[k] = __shfl_sync(0xffffffffu, mine, b + k);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int u = 0; u < G_::kSub; ++u)
              tma_box(dst + u * kKeys * AT + (b + k) * bx * AT, map, u * (AT / G_::kEs), h, s8[k], full, pol);
        }
        __syncwarp();
      }
    } else {
      int r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = sl[e] >= 0 ? sl[e] * Hkv + h : h;  // any row: the softmax drops it
#pragma unroll 1
      for (int b = 0; b < 32; ++b) {
        int q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = __shfl_sync(0xffffffffu, r[e], b);
        if (elect_one()) {
#pragma unroll
          for (int u = 0; u < G_::kSub; ++u)
            tma_gather4(dst + u * kKeys * AT + b * 4 * AT, map, u * (AT / G_::kEs), q, full, pol);
        }
        __syncwarp();
      }
    }
  };
  // K and V are read once where one tile of rows holds them all
  const uint64_t pol_once = l2_evict_first_policy(), pol_keep = l2_normal_policy();

  if (warp == 0 || warp == 3) {
    // ======================= K tiles, V tiles =======================
    const bool is_v = warp == 3;
    const CUtensorMap* const map = is_v ? &tm_v : &tm_k;
    const uint32_t tiles = is_v ? sV : sK, full = bar(is_v ? kBVFull : kBKFull), empty = bar(is_v ? kBVEmpty : kBKEmpty);
    const int ns = is_v ? NV : NK;
    Ring ir, r;
    int g = 0;
    bool ok = true;
    for (;;) {
      Item it;
      ok = take(ir, it);
      if (!ok || it.nt == 0) break;
      const uint64_t pol = it.q_s * G <= N ? pol_once : pol_keep;
      int32_t blk[4], nb[4];
      pages(it, 0, blk);
      for (int t = 0; t < it.nt; ++t, ++g) {
        pages(it, t + 1, nb);  // past the chunk: none
        ok = wait_bar(empty + 8 * r.at, r.pass ^ 1);
        if (!ok) break;
        int sl[4];
        const uint32_t bad = slots(it, t, blk, sl);
        if (!is_v) {
          // the tile's keys without a page, for the softmax (before the arrival
          // on the tile's barrier, which hands them on)
          uint32_t* w = info + (g % kInfoSlots) * 4;
          if (lane < 4) w[lane] = 0;
          __syncwarp();
          if (__any_sync(0xffffffffu, bad != 0)) {
            if (bad) {
              atomicOr(p.err, kErrBlockRange);
              if (!bx) {
                atomicOr(w + key_of / 32, bad << (key_of & 31));
              } else if (lane < n_box) {
                atomicOr(w + key_of / 32, (bx == 16 ? 0xffffu : 0xffu) << (key_of & 31));
              }
            }
            __syncwarp();
          }
        }
        load_tile(it.h, sl, tiles + r.at * G_::kTileB, map, full + 8 * r.at, pol);
        r.next(ns);
#pragma unroll
        for (int e = 0; e < 4; ++e) blk[e] = nb[e];
      }
      if (!ok) break;
    }
    if (!ok) *abort_flag = 1;
    if (aborted())  // let the copies issued so far land before the CTA exits
      for (int k = 0; k < ns && k < g; ++k) {
        if (r.at-- == 0) {
          r.at = ns - 1;
          r.pass ^= 1;
        }
        wait_bar(full + 8 * r.at, r.pass);
      }
  } else if (warp == 1) {
    // ======================= MMA =======================
    constexpr uint32_t kIdS = idesc(N, F8, false, false), kIdO = idesc(2 * N, F8, true, true);
    Ring ir, kr, vr;
    int j = 0, g = 0, nt = 0;
    // S of tile gg from the next K tile
    auto issue_s = [&](int gg, int qb) -> bool {
      if (!wait_bar(bar(kBKFull) + 8 * kr.at, kr.pass)) return false;
      fence_after();
      const uint64_t dk = sdesc(sK + kr.at * G_::kTileB, 16, 8 * AT, AT);
      const uint64_t dq = sdesc(sQ + qb * G_::kQB, 16, 8 * AT, AT);
      const uint32_t ts = tmem + (gg & 1) * N;
      if (elect_one()) {
#pragma unroll
        for (int part = 0; part < G_::kParts; ++part)
#pragma unroll
          for (int u = 0; u < G_::kSub; ++u)
            mma_steps<F8, AT / 32, 2, 2>(ts, dk + (uint32_t)(u * kKeys * AT >> 4),
                                         dq + (uint32_t)((part * N * G_::kRowB + u * N * AT) >> 4), kIdS, (part | u) != 0);
        commit(bar(kBSFull + (gg & 1)));
        commit(bar(kBKEmpty) + 8 * kr.at);
        // the second arrival hands on what the tile's producer wrote (info)
        mbar_arrive(bar(kBSFull + (gg & 1)));
      }
      __syncwarp();
      kr.next(NK);
      return true;
    };
    bool ok = true;
    for (int t = 0;; ++t, ++g) {  // t: tile of item j - 1, whose S has been issued
      if (t == nt - 1 && elect_one()) commit(bar(kBQEmpty + qbuf(j - 1)));
      int nt2 = nt;
      if (t + 1 >= nt) {  // the tile whose S goes next is the next item's first
        Item it;
        ok = take(ir, it);
        nt2 = it.nt;
        if (!ok || (nt2 == 0 && nt == 0)) break;
        ok = nt2 == 0 || wait_bar(bar(kBQFull + qbuf(j)), qpass(j));
        if (!ok) break;
      }
      const int gs = nt == 0 ? g : g + 1, qb = qbuf(t + 1 >= nt ? j : j - 1);
      if (nt2 > 0 || t + 1 < nt) ok = issue_s(gs, qb);
      if (nt > 0 && ok) {
        const int ob = ~j & 1;
        ok = wait_bar(bar(kBVFull) + 8 * vr.at, vr.pass) && (t > 0 || wait_bar(bar(kBOFree + ob), (((j - 1) >> 1) & 1) ^ 1)) &&
             wait_bar(bar(kBPFull + (g & 1)), (g >> 1) & 1);
        if (!ok) break;
        fence_after();
        // V^T: d contiguous, 8 keys = 8 AT bytes, sub-tiles kKeys AT apart.  With
        // D = 64 the M side's upper 64 rows repeat shifted keys; their lanes
        // are never read.
        constexpr int KS = G_::kKeyStep;
        const uint64_t dv = sdesc(sV + vr.at * G_::kTileB, G_::kSub > 1 ? kKeys * AT : 8 * AT, 8 * AT, AT);
        const uint64_t dp = sdesc(sP + (g & 1) * G_::kPB, kKeys * 128, 1024, 128);
        const uint32_t to = tmem + G_::kColO + ob * G_::kOCols;
        if (elect_one()) {
          mma_steps<F8, 4, KS * AT / 16, KS * 8>(to, dv, dp, kIdO, t > 0);
          if constexpr (!F8) mma_steps<F8, 4, KS * AT / 16, KS * 8>(to, dv + 4 * KS * AT / 16, dp + 4 * KS * 8, kIdO, 1);
          commit(bar(kBODone));
          commit(bar(kBVEmpty) + 8 * vr.at);
          if (t + 1 == nt) commit(bar(kBOFull + ob));
        }
        __syncwarp();
        vr.next(NV);
      }
      if (!ok) break;
      if (t + 1 >= nt) {
        if (nt == 0) --g;  // no tile was finished
        if (nt2 == 0) break;
        nt = nt2;
        t = -1;
        ++j;
      }
    }
    if (!ok) *abort_flag = 1;
    // every MMA issued so far is finished before TMEM is freed
    if (elect_one()) commit(bar(kBDrain));
    __syncwarp();
    wait_bar(bar(kBDrain), 0);
  } else if (warp == 2) {
    // ======================= items, query rows =======================
    int gb = 0;                        // the group of sequences gb .. gb + 31 held by the lanes
    int c0 = 0, q_s = 0, n = 0, chunk = 1, nchunks = 0, rts = 0;
    int cnt = 0, incl = 0, base = 0, total = 0;  // items: this sequence's, prefix in the group; before it; in it
    constexpr int kLanes = D / 8;          // lanes of a row (8 bf16 elements each)
    constexpr int kPer = 32 / kLanes;      // rows per step
    constexpr int kStepsQ = N / kPer;
    const int ch = lane % kLanes, rr = lane / kLanes;
    Ring ir;
    bool ok = true;
    gb = -32;
    for (int j = 0, x = blockIdx.x;; ++j, x += gridDim.x) {
      // item number x of the call
      while (x - base >= total && gb < p.B) {
        base += total;
        gb += 32;
        const int s = gb + lane;
        cnt = 0;
        if (s < p.B) {
          c0 = __ldg(p.cu_q + s);
          const int c1 = __ldg(p.cu_q + s + 1);
          n = __ldg(p.seq_lens + s);
          q_s = c1 - c0;
          const bool bad = c0 < 0 || c1 < c0 || (int64_t)c1 > p.T || q_s > n || (int64_t)n > (int64_t)p.max_blocks * p.bs ||
                           q_s > p.max_nodes;
          if (bad && blockIdx.x == 0) atomicOr(p.err, kErrLengths);
          if (!bad && q_s > 0) {
            chunk = tree_chunk(n, q_s, a.chunking);
            nchunks = (n - 1) / chunk + 1;
            rts = (q_s * G - 1) / N + 1;
            cnt = nchunks * Hkv * rts;
          }
        }
        incl = cnt;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        total = __shfl_sync(0xffffffffu, incl, 31);
      }
      Item it{};
      if (x - base < total) {
        const int o = __ffs(__ballot_sync(0xffffffffu, incl > x - base)) - 1;
        int y = x - base - __shfl_sync(0xffffffffu, incl - cnt, o);
        it.s = gb + o;
        it.t0 = __shfl_sync(0xffffffffu, c0, o);
        it.q_s = __shfl_sync(0xffffffffu, q_s, o);
        it.n = __shfl_sync(0xffffffffu, n, o);
        it.nchunks = __shfl_sync(0xffffffffu, nchunks, o);
        const int rt_n = __shfl_sync(0xffffffffu, rts, o), len = __shfl_sync(0xffffffffu, chunk, o);
        const int z = y / rt_n;
        it.r0 = (y - z * rt_n) * N;
        it.c = z / Hkv;
        it.h = z - it.c * Hkv;
        it.k0 = it.c * len;
        it.k1 = it.n - it.k0 < len ? it.n : it.k0 + len;
        it.nt = (it.k1 - it.k0 + kKeys - 1) / kKeys;
      }
      ok = wait_bar(bar(kBItemEmpty) + 8 * ir.at, ir.pass ^ 1) && !aborted();
      if (!ok) break;
      if (lane == 0) {
        items[ir.at] = it;
        mbar_arrive(bar(kBItemFull) + 8 * ir.at);
      }
      __syncwarp();
      ir.next(kItemSlots);
      if (it.nt == 0) break;
      // its query rows; the buffer is free once the scores of the item that
      // used it last are there
      const int qb = qbuf(j), rows = it.q_s * G;
      const uint32_t dst = sQ + qb * G_::kQB;
      // lane c (and c + 32) finds row c; 0: past the last
      unsigned long long row[(N + 31) / 32];
#pragma unroll
      for (int k = 0; k < (N + 31) / 32; ++k) {
        const int r = it.r0 + lane + 32 * k, i = quot(r, a.by_g);
        const __nv_bfloat16* at = static_cast<const __nv_bfloat16*>(p.q) + (it.t0 + i) * p.q_st + (it.h * G + r - i * G) * p.q_sh;
        row[k] = r < rows ? reinterpret_cast<unsigned long long>(at) : 0;
      }
      ok = wait_bar(bar(kBQEmpty + qb), qpass(j) ^ 1);
      if (!ok) break;
#pragma unroll
      for (int k = 0; k < (N + 31) / 32; ++k)
#pragma unroll 4
        for (int b = 0; b < (N < 32 ? N : 32); b += kPer) {
          const int rt = 32 * k + b + rr;  // row of the tile
          const unsigned long long src = __shfl_sync(0xffffffffu, row[k], b + rr);
          // straight to shared memory; a row past the last is zeros
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (ch * 16 / AT) * N * AT +
                                                                              swz<AT>(rt, ch % (AT / 16))),
                       "l"(src ? src + ch * 16 : reinterpret_cast<unsigned long long>(p.q)), "r"(src ? 16 : 0)
                       : "memory");
        }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      if constexpr (F8) {
        // the bf16 row fills row rt of both parts' tiles; the lanes that hold it
        // replace it by its two e4m3 parts
#pragma unroll 2
        for (int b = 0; b < kStepsQ; ++b) {
          const int rt = b * kPer + rr;
          uint32_t wd[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(wd[0]), "=r"(wd[1]), "=r"(wd[2]), "=r"(wd[3])
                       : "r"(dst + (ch * 16 / AT) * N * AT + swz<AT>(rt, ch % (AT / 16))));
          // the row's largest element, as the bits of its absolute value (infinity and NaN on top)
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(wd[e] & 0x7fffu, (wd[e] >> 16) & 0x7fffu));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          const bool nan = top >= 0x7f80u;
          // 2^e2 <= largest < 2^(e2 + 1); e2 stays where 2^(7 - e2) is a normal number
          const int e2 = max(static_cast<int>(top >> 7) - 127, -100);
          const float up = nan ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + 7 - e2) << 23);
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u0 = bf16_lo(wd[e]) * up, u1 = bf16_hi(wd[e]) * up;
            const uint16_t h2 = f32x2_to_e4m3x2(u0, u1);
            const uint32_t hf = e4m3x2_to_f16x2(h2);
            const float2 hv = __half22float2(*reinterpret_cast<const __half2*>(&hf));
            const uint16_t l2 = f32x2_to_e4m3x2(u0 - hv.x, u1 - hv.y);
            hi[e >> 1] = e & 1 ? hi[e >> 1] | (uint32_t)h2 << 16 : h2;
            lo[e >> 1] = e & 1 ? lo[e >> 1] | (uint32_t)l2 << 16 : l2;
          }
          const uint32_t at = swz<AT>(rt, ch >> 1) + (ch & 1) * 8;
          __syncwarp();
          st_s64(dst + at, hi[0], hi[1]);
          st_s64(dst + N * G_::kRowB + at, lo[0], lo[1]);
          if (ch == 0)
            qscale[(j % 4) * 64 + rt] =
                nan ? __uint_as_float(0x7fffffffu) : __uint_as_float(static_cast<uint32_t>(127 - 7 + e2) << 23) * p.qk_scale_log2;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kBQFull + qb));
        if (F8) mbar_arrive(bar(kBQsFull + j % 4));
      }
    }
    if (!ok) *abort_flag = 1;
  } else if (warp < 4 + G_::kSoft) {
    // ======================= softmax =======================
    const int quarter = warp & 3, grp = (warp - 4) >> 2;
    const int tg = quarter * 32 + lane;  // thread of the group: this lane's key in a tile
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    // p may pass 2^0 (e4m3: 2^kUp, times which p is kept) by 2^kTau before a
    // row's reference moves.  bf16 parts keep their precision over the whole
    // exponent range, so the first reference is 0 unless the row's largest
    // score lies beyond +-kTau; e4m3 parts want the largest p near 2^kUp.
    constexpr float kTau = F8 ? 4.5f : 60.f;
    constexpr float kUp = F8 ? 4.f : 0.f;
    // an e4m3 row's reference is set this far above the largest score seen, so
    // that it rarely has to move again in a chunk
    constexpr float kMargin = F8 ? 2.5f : 0.f;
    float* xh = xch + grp * 4 * NC;
    // A vote of the group's four warps, cast and counted apart so that work can
    // go between: count() tells all four alike whether any of them wanted.
    volatile int* flag = reinterpret_cast<volatile int*>(misc + kOffFlag) + 2 * grp;  // [2]: number of the vote that wants
    int votes = 0;
    auto cast = [&](bool want) {
      if (lane == 0) {
        if (want) flag[votes & 1] = votes + 1;
        mbar_arrive(bar(kBGroup + grp));
      }
    };
    auto count = [&](bool& wanted) -> bool {
      const bool r = wait_bar(bar(kBGroup + grp), votes & 1);
      wanted = flag[votes & 1] == votes + 1;
      ++votes;
      return r;
    };
    auto sync = [&]() -> bool {  // also orders the four warps' shared memory
      bool w;
      __syncwarp();
      cast(false);
      return count(w);
    };
    // this lane's row of P, at the first of the warp's columns in the hi part; a
    // further 16-byte chunk's place, and the lo part's, differ by an exclusive or
    const uint32_t p_at = sP + swz<128>(tg, grp * NC * G_::kEs / 16) + (grp * NC * G_::kEs) % 16;
    if (tg < NC) refs[grp * NC + tg] = kUp;  // item 0's
    Ring ir;
    int g = 0;
    bool ok = sync();
    for (int j = 0; ok; ++j) {
      Item it;
      ok = take(ir, it);
      if (!ok || it.nt == 0) break;
      const int nt = it.nt, rows = it.q_s * G, ctx = it.n - it.q_s;
      const int ra = it.r0 + grp * NC;  // first row of this group
      const float* qs = qscale + (j % 4) * 64 + grp * NC;
      // the rows' references, kept as kUp - reference; the next item's start at
      // reference 0 (three sets: warps of the group may still read the last item's)
      float* rh = refs + (j % 3) * 64 + grp * NC;
      if (tg < NC) refs[((j + 1) % 3) * 64 + grp * NC + tg] = kUp;
      if (F8) {
        ok = wait_bar(bar(kBQsFull + j % 4), (j >> 2) & 1);
        if (!ok) break;
      }
      unsigned long long l2[NC / 2];  // the rows' sums over this lane's keys, in pairs
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) l2[c] = 0ull;
      uint32_t vmask = 0;  // rows of the group without a reference yet (stored as 0), once the first tile has set them
      for (int t = 0; t < nt; ++t, ++g) {
        ok = wait_bar(bar(kBSFull + (g & 1)), (g >> 1) & 1);
        if (!ok) break;
        fence_after();
        const uint32_t ts = tmem + (g & 1) * N + grp * NC + lane_off;  // this tile's q.k of the stored values
        const uint4 bad = *reinterpret_cast<const uint4*>(info + (g % kInfoSlots) * 4);
        const int kt = it.k0 + t * kKeys;  // first key of the tile
        const bool masked = kt + kKeys > ctx || (bad.x | bad.y | bad.z | bad.w) != 0;
        uint32_t see = 0xffffffffu;  // rows that see this lane's key
        if (masked) {
          const int key = kt + tg, jj = key - ctx;
          const uint32_t badw = quarter == 0 ? bad.x : quarter == 1 ? bad.y : quarter == 2 ? bad.z : bad.w;
          if (key >= it.k1 || ((badw >> lane) & 1u)) {
            see = 0;
          } else if (jj >= 0) {
            see = 0;
            const int i = quot(ra, a.by_g);
            int gq = ra - i * G;
            const int32_t* m = p.mask + (int64_t)(it.t0 + i) * p.mask_stride + (jj >> 5);
#pragma unroll 4
            for (int c = 0; c < NC; ++c) {
              if (ra + c < rows) see |= ((static_cast<uint32_t>(__ldg(m)) >> (jj & 31)) & 1u) << c;
              if (++gq == G) {
                gq = 0;
                m += p.mask_stride;
              }
            }
          }
          // V rows that must not reach a row that does not see them: zero what
          // is past the sequence or has no page, and what is not finite among
          // the drafted rows (the rows that see those get it at the end)
          if (!wait_bar(bar(kBVFull + g % NV), (g / NV) & 1)) { ok = false; break; }
          constexpr int kLn = G_::kRowB / 16, kRs = 32 / kLn;
          const int ch = lane % kLn, rr = lane / kLn;
          bool found = false;
#pragma unroll 1
          for (int b = 0; b < kKeys / G_::kSoft; b += kRs) {
            const int kk = (warp - 4) * (kKeys / G_::kSoft) + b + rr, ky = kt + kk;
            const uint32_t bm = kk < 32 ? bad.x : kk < 64 ? bad.y : kk < 96 ? bad.z : bad.w;
            const bool gone = ky >= it.k1 || ((bm >> (kk & 31)) & 1u);
            if (!gone && ky < ctx) continue;
            const uint32_t at = sV + (g % NV) * G_::kTileB + (ch * 16 / AT) * kKeys * AT + swz<AT>(kk, ch % (AT / 16));
            uint32_t w[4] = {0, 0, 0, 0};
            bool hit = gone;
            if (!gone) {
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
              constexpr uint32_t kExp = F8 ? 0x7fu : 0x7f80u, kAll = F8 ? 0xffu : 0xffffu;
              constexpr int kBits = F8 ? 8 : 16;
#pragma unroll 1
              for (int f = 0; f < 32; f += kBits)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (((w[e] >> f) & kExp) == kExp) {
                    w[e] &= ~(kAll << f);
                    hit = true;
                  }
              found = found || hit;
            }
            if (hit) st_s128(at, w[0], w[1], w[2], w[3]);
          }
          if (found) poison[j % 3] = j + 1;
        }
        // y = score in base 2 less the row's reference, plus kUp
        float y[NC];
        uint32_t hi[F8 ? NC / 4 : NC / 2], lo[F8 ? NC / 4 : NC / 2];
        if (F8 && t == 0 && !masked) {
          // the first reference, from the row's largest score among 32 of the
          // tile's keys (each warp takes a quarter of the rows over its own keys)
          uint32_t u[8];
          float m = -INFINITY;
          constexpr int kSample = NC / 4 < 8 ? NC / 4 : 8;
          tm_ld(tmem + (g & 1) * N + lane_off + (grp * NC + quarter * (NC / 4)) / 8 * 8, u);
          wait_ld();
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int cc = c - (grp * NC + quarter * (NC / 4)) % 8;  // row of the quarter
            const float x = redux_max(__uint_as_float(u[c]) * qs[(quarter * (NC / 4)) / 8 * 8 + c]);
            m = lane == cc && cc < kSample ? x : m;
          }
          const bool none = lane < NC / 4 && m == -INFINITY;
          if (lane < NC / 4) rh[quarter * (NC / 4) + lane] = none ? kUp : kUp - kMargin - m;
          const uint32_t unset = __ballot_sync(0xffffffffu, none) << (quarter * (NC / 4));
          if (lane == 0) unset4[grp * 4 + quarter] = unset;
          __syncwarp();
          cast(unset != 0);
          bool some;
          if (!count(some)) { ok = false; break; }
          if (some) vmask = unset4[grp * 4] | unset4[grp * 4 + 1] | unset4[grp * 4 + 2] | unset4[grp * 4 + 3];
        }
        // first try: all of the tile's work against the references there are;
        // careful: new references; last: the work against those
        enum : int { kTry, kCareful, kLast };
        for (int mode = masked || vmask ? kCareful : kTry;;) {
          uint32_t u[NC];
          tm_ld(ts, u);
          wait_ld();
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const float4 r = *reinterpret_cast<const float4*>(rh + c);
            unsigned long long s01, s23;
            if constexpr (F8) {
              const float4 q = *reinterpret_cast<const float4*>(qs + c);
              s01 = pk2(q.x, q.y);
              s23 = pk2(q.z, q.w);
            } else {
              s01 = s23 = pk2(p.qk_scale_log2, p.qk_scale_log2);
            }
            up2(fma2(pk2(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), s01, pk2(r.x, r.y)), y[c], y[c + 1]);
            up2(fma2(pk2(__uint_as_float(u[c + 2]), __uint_as_float(u[c + 3])), s23, pk2(r.z, r.w)), y[c + 2], y[c + 3]);
          }
          if (masked) {
#pragma unroll
            for (int c = 0; c < NC; ++c) y[c] = (see >> c) & 1u ? y[c] : -INFINITY;
          }
          if (mode == kTry) {
            float top = fmaxf(y[0], y[1]);
#pragma unroll
            for (int c = 2; c < NC; c += 2) top = fmax3(top, y[c], y[c + 1]);
            bool want = top > kTau + kUp;
            if (!F8 && t == 0) {
              float low = fminf(y[0], y[1]);
#pragma unroll
              for (int c = 2; c < NC; c += 2) low = fmin3(low, y[c], y[c + 1]);
              want = want || !(low >= -kTau);
            }
            cast(__any_sync(0xffffffffu, want));
          }
          if (mode != kCareful) {
            // P = 2^y in two parts, row = key, hi in columns 0 .. N - 1, lo in N .. 2 N - 1
            // (while the vote is out: if it asks for care, all of this is done again)
#pragma unroll
            for (int c = 0; c < NC; c += 2) {
              const float p0 = ex2(y[c]), p1 = ex2(y[c + 1]);
              const unsigned long long pp = pk2(p0, p1);
              y[c] = p0;
              y[c + 1] = p1;
              if constexpr (F8) {
                // through f16 (11 bits, two values at a time): hi its e4m3 code, lo
                // that of 16 times the exact remainder
                const __half2 h = __floats2half2_rn(p0, p1);
                const uint16_t h2 = f16x2_to_e4m3x2(h);
                const uint32_t hb = e4m3x2_to_f16x2(h2);
                const uint16_t l8 = f16x2_to_e4m3x2(__hmul2(__hsub2(h, *reinterpret_cast<const __half2*>(&hb)), __float2half2_rn(16.f)));
                if (c & 2) {
                  hi[c / 4] |= (uint32_t)h2 << 16;
                  lo[c / 4] |= (uint32_t)l8 << 16;
                } else {
                  hi[c / 4] = h2;
                  lo[c / 4] = l8;
                }
              } else {
                const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
                hi[c / 2] = __byte_perm(u0, u1, 0x7632);
                float r0, r1;  // p - hi exactly: the truncated-away low bits
                up2(sub2(pp, pk2(__uint_as_float(u0 & 0xFFFF0000u), __uint_as_float(u1 & 0xFFFF0000u))), r0, r1);
                lo[c / 2] = __byte_perm(__float_as_uint(r0), __float_as_uint(r1), 0x7632);
              }
            }
            if (mode == kLast) break;
            const bool in = poll(bar(kBGroup + grp), votes & 1), calm = flag[votes & 1] != votes + 1;
            ++votes;
            if (__all_sync(0xffffffffu, in && calm)) break;
            ok = __all_sync(0xffffffffu, in);
            if (!ok) break;
            mode = kCareful;
            continue;
          }
          // ---- the careful path: the rows' largest y over the tile
          float mine = 0.f;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float m = redux_max(y[c]);  // NaN is passed over
            mine = lane == c ? m : mine;
          }
          if (lane < NC) xh[quarter * NC + lane] = mine;
          if (!sync()) { ok = false; break; }
          // lane c: row c's new reference; the stored value is kUp - reference
          float alpha = 1.f, nref = 0.f;
          bool moved = false, none = false;
          if (lane < NC) {
            const float top = fmaxf(fmaxf(xh[lane], xh[NC + lane]), fmaxf(xh[2 * NC + lane], xh[3 * NC + lane]));
            const float old = rh[lane];
            nref = old;
            if ((t == 0 && (!F8 || masked)) || ((vmask >> lane) & 1u)) {  // none yet, 0 stands in
              none = top == -INFINITY;
              if (!none && (F8 || fabsf(top) > kTau)) nref = old + kUp - kMargin - top;
            } else if (top > kTau + kUp) {
              nref = old + kUp - kMargin - top;
              alpha = ex2(kUp - kMargin - top);
              moved = true;
            }
          }
          vmask = __ballot_sync(0xffffffffu, none);
          const bool any = __any_sync(0xffffffffu, moved);
          // every warp has read the references
          if (!sync()) { ok = false; break; }
          if (quarter == 0 && lane < NC) rh[lane] = nref;
          if (any) {  // the same in the group's four warps
#pragma unroll
            for (int c = 0; c < NC; c += 2)
              l2[c / 2] = mul2(l2[c / 2], pk2(__shfl_sync(0xffffffffu, alpha, c), __shfl_sync(0xffffffffu, alpha, c + 1)));
            // t > 0: every P V so far has run after this wait
            if (!wait_bar(bar(kBODone), (g - 1) & 1)) { ok = false; break; }
            fence_after();
            const uint32_t to = tmem + G_::kColO + (j & 1) * G_::kOCols + lane_off + grp * NC;
#pragma unroll 1
            for (int b = 0; b < NC; b += 8) {
              uint32_t o[8], o2[8];
              tm_ld(to + b, o);
              tm_ld(to + N + b, o2);
              wait_ld();
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float f = __shfl_sync(0xffffffffu, alpha, b + c);
                o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                o2[c] = __float_as_uint(__uint_as_float(o2[c]) * f);
              }
              tm_st(to + b, o);
              tm_st(to + N + b, o2);
            }
            wait_st();
          }
          // the references are written
          if (!sync()) { ok = false; break; }
          mode = kLast;
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < NC; c += 2) l2[c / 2] = add2(l2[c / 2], pk2(y[c], y[c + 1]));
        // the P buffer is free: P V of the tile before the last came before this tile's S
        {
          const uint32_t at = p_at + (g & 1) * G_::kPB, at_lo = G_::kPRow == 256 ? at + kKeys * 128 : at ^ (N * G_::kEs);
          if constexpr (NC * G_::kEs == 8) {
            st_s64(at, hi[0], hi[1]);
            st_s64(at_lo, lo[0], lo[1]);
          } else {
#pragma unroll
            for (int q = 0; q < NC * G_::kEs / 16; ++q) {
              st_s128(at ^ (q << 4), hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
              st_s128(at_lo ^ (q << 4), lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
            }
          }
        }
        fence_proxy_async_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBPFull + (g & 1)));
      }
      if (!ok) break;
      // the rows' sums over this warp's keys go to the output warps
      if (!wait_bar(bar(kBLEmpty + (j & 1)), ((j >> 1) & 1) ^ 1)) { ok = false; break; }
      {
        float m[NC];
#pragma unroll
        for (int c = 0; c < NC; c += 2) up2(l2[c / 2], m[c], m[c + 1]);
        const float mine = col_sum<NC>(m, lane);
        const int at = (j & 1) * 64 + grp * NC;
        if (lane % (32 / NC) == 0) sums[(j & 1) * 256 + quarter * 64 + grp * NC + lane / (32 / NC)] = mine;
        if (tg < NC) lref[at + tg] = rh[tg];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBLFull + (j & 1)));
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ======================= O / l: lane = d, register = row =======================
    const int d = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    constexpr float kLo = F8 ? 0.0625f : 1.f;  // the low part's weight
    constexpr int kCols = 16;            // rows at a time
    constexpr int kOff = (N + 31) / 32;  // row offsets held by a lane
    Ring ir;
    bool ok = true;
    for (int j = 0;; ++j) {
      Item it;
      ok = take(ir, it);
      if (!ok || it.nt == 0) break;
      ok = wait_bar(bar(kBLFull + (j & 1)), (j >> 1) & 1);
      if (!ok) break;
      const int rows = it.q_s * G;
      // lane c (and c + 32): 1 / (row c's sum), and its log2-sum-exp2 for the join
      float inv[kOff];
#pragma unroll
      for (int k = 0; k < kOff; ++k) {
        const int c = (lane + 32 * k) & (N - 1), r = it.r0 + c;
        const float* q = sums + (j & 1) * 256 + c;
        const float l = (q[0] + q[64]) + (q[128] + q[192]);
        inv[k] = l == 0.f ? 0.f : p.v_scale / l;
        if (warp == 4 + G_::kSoft && it.nchunks > 1 && r < rows && lane + 32 * k < N) {
          const int i = quot(r, a.by_g);
          a.part_lse[((int64_t)it.s * a.rows_per_seq + i * it.nchunks + it.c) * p.Hq + it.h * G + r - i * G] =
              l == 0.f ? -INFINITY : __log2f(l) - lref[(j & 1) * 64 + (c / NC) * NC + c % NC];  // reference + log2(sum) - kUp
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBLEmpty + (j & 1)));
      ok = wait_bar(bar(kBOFull + (j & 1)), (j >> 1) & 1);
      if (!ok) break;
      fence_after();
      const bool split = it.nchunks > 1, wide = split || !a.out_bf16;  // fp32 elements
      // lane c (and c + 32): where row c's element 0 goes, in bytes from `to_base`; -1: no row
      const int esz = wide ? 4 : 2;
      const int64_t node = split ? (int64_t)it.nchunks * p.Hq * D : p.o_st, head = split ? D : p.o_sh;
      char* const to_base = (split ? reinterpret_cast<char*>(a.part_o + ((int64_t)it.s * a.rows_per_seq + it.c) * p.Hq * D)
                                   : static_cast<char*>(p.out) + it.t0 * p.o_st * esz) + it.h * G * head * esz;
      long long off[kOff];
#pragma unroll
      for (int k = 0; k < kOff; ++k) {
        const int r = it.r0 + lane + 32 * k, i = quot(r, a.by_g);
        off[k] = lane + 32 * k < N && r < rows ? (i * node + (r - i * G) * head) * esz : -1;
      }
      char* const mine = to_base + d * esz;
#pragma unroll 1
      for (int b = 0; b < N; b += kCols) {
        const uint32_t to = tmem + G_::kColO + (j & 1) * G_::kOCols + lane_off + b;
        uint32_t o[kCols], o2[kCols];
        tm_ld(to, o);
        tm_ld(to + N, o2);
        float v[kCols];
        wait_ld();
        if (b + kCols == N) {  // the accumulator has been read
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBOFree + (j & 1)));
        }
        const float si = kOff > 1 && b >= 32 ? inv[kOff - 1] : inv[0];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const float sc = __shfl_sync(0xffffffffu, si, (b & 31) + c);
          const float x = fmaf(__uint_as_float(o2[c]), kLo, __uint_as_float(o[c])) * sc;
          v[c] = sc == 0.f ? 0.f : x;
        }
        long long at[kCols];
        const long long from = kOff > 1 && b >= 32 ? off[kOff - 1] : off[0];
#pragma unroll
        for (int c = 0; c < kCols; ++c) at[c] = __shfl_sync(0xffffffffu, from, (b & 31) + c);
        if (D == 128 || d < D) {
          if (wide) {
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              if (at[c] >= 0) *reinterpret_cast<float*>(mine + at[c]) = v[c];
          } else {
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              if (at[c] >= 0) *reinterpret_cast<__nv_bfloat16*>(mine + at[c]) = __float2bfloat16_rn(v[c]);
          }
        }
      }
      if (poison[j % 3] == j + 1 && (D == 128 || d < D)) add_poison<D, N, F8>(a, it, d);
    }
    if (!ok) *abort_flag = 1;
  }
  // ---- teardown
  fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.err, kErrWaitTimeout);
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

// ---------------------------------------------------------------- join
// o = sum_c 2^(lse_c - M) o_c / sum_c 2^(lse_c - M) over a row's chunks, in
// order.  One warp per (row, query head); lane l holds elements l D/32 ..;
// eight chunks' loads in flight.  grid: (sequences, parts of a sequence's rows).
template <int D, typename OutT>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeParams p, const float* part_o, const float* part_lse,
                                                        int rows_per_seq, Chunking chunking) {
  grid_dep_wait();
  launch_dependents();
  constexpr int E = D / 32;
  const int s = blockIdx.x, lane = threadIdx.x & 31;
  const int c0 = __ldg(p.cu_q + s), c1 = __ldg(p.cu_q + s + 1), n = __ldg(p.seq_lens + s);
  const int q_s = c1 - c0;
  if (c0 < 0 || c1 <= c0 || (int64_t)c1 > p.T || q_s > n || (int64_t)n > (int64_t)p.max_blocks * p.bs || q_s > p.max_nodes)
    return;
  const int chunk = tree_chunk(n, q_s, chunking);
  const int nc = (n - 1) / chunk + 1;
  if (nc == 1) return;
  const int64_t rows = (int64_t)q_s * p.Hq;
  for (int64_t r = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.y * 8) {
    const int i = static_cast<int>(r / p.Hq), hq = static_cast<int>(r - (int64_t)i * p.Hq);
    const int64_t at = ((int64_t)s * rows_per_seq + (int64_t)i * nc) * p.Hq + hq;
    float lv[2], M = -INFINITY;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      lv[k] = lane + 32 * k < nc ? __ldcg(part_lse + at + (int64_t)(lane + 32 * k) * p.Hq) : -INFINITY;
      M = fmaxf(M, lv[k]);  // a NaN stays out of M and comes back through the weights
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ms = M == -INFINITY ? 0.f : M;
    float w[2], L = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      w[k] = lane + 32 * k < nc ? exp2f(lv[k] - ms) : 0.f;
      L += w[k];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float* src = part_o + at * D + lane * E;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int b = 0; b < nc; b += 8) {
      float v[8][E];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (b + k < nc) {
          const float* q = src + (int64_t)(b + k) * p.Hq * D;
          if constexpr (E == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(q));
            v[k][0] = f.x, v[k][1] = f.y, v[k][2] = f.z, v[k][3] = f.w;
          } else {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(q));
            v[k][0] = f.x, v[k][1] = f.y;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float wk = __shfl_sync(0xffffffffu, b < 32 ? w[0] : w[1], (b + k) & 31);
        if (b + k < nc && wk != 0.f) {  // a chunk without weight adds nothing
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(wk, v[k][e], acc[e]);
        }
      }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    OutT* dst = static_cast<OutT*>(p.out) + (int64_t)(c0 + i) * p.o_st + (int64_t)hq * p.o_sh + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) store2(dst + e, acc[e] * inv, acc[e + 1] * inv);
  }
}

// ---------------------------------------------------------------- host
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(f);
  });
  return fn;
}

// Rows of a cache: {d, heads, slots} with a {atom, 1, box} box, or for
// gather4 {d, slots * heads} with a {atom, 1} box.
bool encode_cache(CUtensorMap* m, const void* base, const TreeParams& p, bool f8, int atom_bytes, int box) {
  EncodeTiled fn = encode_fn();
  if (fn == nullptr) return false;
  const uint64_t es = f8 ? 1 : 2, d = p.D, heads = p.Hkv, slots = (uint64_t)p.num_blocks * p.bs;
  const cuuint64_t dims[3] = {d, box ? heads : heads * slots, slots};
  const cuuint64_t strides[2] = {d * es, d * es * heads};
  const cuuint32_t bx[3] = {(cuuint32_t)(atom_bytes / es), 1, (cuuint32_t)box};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, box ? 3 : 2, const_cast<void*>(base),
            dims, strides, bx, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            atom_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int N, bool F8>
cudaError_t launch_t(TcArgs a, int64_t max_items, int num_sms, cudaStream_t st) {
  using G_ = Geo<D, N, F8>;
  a.box = a.p.bs % 16 == 0 ? 16 : a.p.bs % 8 == 0 ? 8 : 0;
  CUtensorMap mk, mv;
  if (!encode_cache(&mk, a.p.k_cache, a.p, F8, G_::kAtomB, a.box) || !encode_cache(&mv, a.p.v_cache, a.p, F8, G_::kAtomB, a.box))
    return cudaErrorInvalidValue;
  auto kern = tree_tc_kernel<D, N, F8>;
  cudaError_t e = set_smem_attr(reinterpret_cast<const void*>(kern), G_::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t grid = std::min<int64_t>(num_sms, max_items);
  return launch_ex(kern, dim3((unsigned)grid), dim3(G_::kThreads), G_::kSmem, st, true, a, mk, mv);
}

}  // namespace

// Rows per MMA tile: the narrowest that holds the largest tree.
static int tree_tile_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
static Chunking call_chunking(int64_t B, int64_t Hkv, int64_t rows) {
  const int64_t N = tree_tile_rows(rows);
  return tree_chunking(B * Hkv * ((rows + N - 1) / N));
}

int64_t tree_tc_rows_per_seq(int64_t B, int64_t Hkv, int64_t G, int64_t max_q, int64_t max_ctx) {
  const Chunking c = call_chunking(B, Hkv, max_q * G);
  const int64_t chunks = std::min<int64_t>(c.most, (max_ctx + c.least - 1) / c.least);
  if (chunks <= 1) return 0;
  return std::min<int64_t>(max_q * chunks, kTreePartRows);
}

cudaError_t launch_tree_tc(const TreeParams& p, bool f8, int out_kind, int64_t max_q, int64_t max_ctx, void* workspace,
                           int num_sms, cudaStream_t st) {
  TcArgs a{};
  a.p = p;
  a.out_bf16 = out_kind;
  a.by_g = fast_div(static_cast<uint32_t>(p.G));
  a.by_bs = fast_div(static_cast<uint32_t>(p.bs));
  const int64_t rps = tree_tc_rows_per_seq(p.B, p.Hkv, p.G, max_q, max_ctx);
  a.rows_per_seq = static_cast<int32_t>(rps);
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = a.part_o + (int64_t)p.B * rps * p.Hq * p.D;
  const int64_t rows = max_q * p.G;
  const int N = tree_tile_rows(rows);
  a.chunking = call_chunking(p.B, p.Hkv, rows);
  const int64_t most = (int64_t)p.B * kTreeMaxChunks * p.Hkv * ((rows + N - 1) / N);
  cudaError_t e;
#define PKV_TC1(D, F8)                                      \
  (N == 16   ? launch_t<D, 16, F8>(a, most, num_sms, st)    \
   : N == 32 ? launch_t<D, 32, F8>(a, most, num_sms, st)    \
             : launch_t<D, 64, F8>(a, most, num_sms, st))
  if (p.D == 128)
    e = f8 ? PKV_TC1(128, true) : PKV_TC1(128, false);
  else
    e = f8 ? PKV_TC1(64, true) : PKV_TC1(64, false);
#undef PKV_TC1
  if (e != cudaSuccess || rps == 0) return e;  // no table holds a second chunk
  const int64_t want = (max_q * p.Hq + 7) / 8;
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(want, (8 * num_sms + p.B - 1) / p.B));
  const dim3 grid((unsigned)p.B, (unsigned)y);
#define PKV_JOIN(D, O) launch_ex(tree_join_kernel<D, O>, grid, dim3(256), 0, st, true, p, (const float*)a.part_o, (const float*)a.part_lse, a.rows_per_seq, a.chunking)
  if (p.D == 128) return out_kind ? PKV_JOIN(128, __nv_bfloat16) : PKV_JOIN(128, float);
  return out_kind ? PKV_JOIN(64, __nv_bfloat16) : PKV_JOIN(64, float);
#undef PKV_JOIN
}

}  // namespace pkv
