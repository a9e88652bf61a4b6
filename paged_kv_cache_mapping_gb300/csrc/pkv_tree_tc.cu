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
// chunk length follows from the sequence's own length and node count, chunks
// write normalised partials and log2-sum-exp2, and a second small kernel joins
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
// CTA: 12 warps.
//   warp 0      items, and TMA copies of the K and V tiles of 128 keys: boxes
//               of 16 or 8 slots that lie in one block, or, for other block
//               sizes, four arbitrary rows at a time (tile::gather4).
//   warp 1      issues the MMAs: S of tile g + 1, then P V of tile g.
//   warps 2, 3  query rows: bf16 to the swizzled operand layout, or split to e4m3.
//   warps 4-11  softmax: lane quarter w % 4 = keys, half (w - 4) / 4 = rows.
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "pkv_kernels.h"

namespace pkv {
namespace {

constexpr int kKeys = 128;  // keys per tile (M of S^T, K of P V)
constexpr int kThreads = 384;
constexpr int kItemSlots = 4;
constexpr int kInfoSlots = 8;

// ---------------------------------------------------------------- chunking
// Keys per chunk: at most 64 chunks, at most 1024 / q_s (so that a sequence
// has at most 1024 partial rows per head), at least 256 keys, whole tiles.  A
// function of the sequence alone.
constexpr int kTreeMaxChunks = 64;
constexpr int kTreePartRows = 1024;
constexpr int kTreeMinChunk = 256;

__host__ __device__ inline int tree_chunk(int n, int q_s) {
  int most = kTreePartRows / q_s;
  most = most < 1 ? 1 : most > kTreeMaxChunks ? kTreeMaxChunks : most;
  long long c = ((long long)n + most - 1) / most;
  c = (c + kKeys - 1) / kKeys * kKeys;
  if (most == 1) return static_cast<int>(c < 0x7fffff80ll ? c : 0x7fffff80ll);
  return static_cast<int>(c < kTreeMinChunk ? kTreeMinChunk : c);
}

// ---------------------------------------------------------------- geometry
template <int D, int N, bool F8>
struct Geo {
  static constexpr int kEs = F8 ? 1 : 2;
  static constexpr int kRowB = D * kEs;                       // one K or V row
  static constexpr int kAtomB = kRowB < 128 ? kRowB : 128;    // swizzle width
  static constexpr int kSub = kRowB / kAtomB;                 // sub-tiles along d
  static constexpr int kTileB = kKeys * kRowB;
  static constexpr int kParts = F8 ? 2 : 1;                   // parts of Q
  static constexpr int kQB = N * kRowB * kParts;
  static constexpr int kPB = kKeys * 128;                     // one part of P: [128 keys][128 bytes]
  static constexpr int kNK = kTileB == 32768 ? 2 : kTileB == 16384 ? 4 : 6;
  static constexpr int kNV = kTileB == 32768 ? 3 : kTileB == 16384 ? 5 : 6;
  static constexpr int kNC = N / 2;                           // rows (columns of S^T) per softmax warp
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kNK * kTileB;
  static constexpr int kOffP = kOffV + kNV * kTileB;
  static constexpr int kOffQ = kOffP + 2 * kPB;
  static constexpr int kOffMisc = kOffQ + 2 * kQB;
  static constexpr int kSmem = kOffMisc + (F8 ? 4096 : 3072);
  // tensor memory: S 2 x N columns, then O: 2 x N (e4m3: hi and lo of each)
  static constexpr uint32_t kColO = 2 * N;
  static constexpr uint32_t kOCols = F8 ? 2 * N : N;
  static constexpr int kSteps = kRowB / 32;                   // MMA k steps of S^T (32 bytes each)
  static constexpr int kKeyStep = F8 ? 32 : 16;               // keys per MMA k step of P V
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kNK + 2 <= kInfoSlots, "tile info ring");
  static_assert(kColO + 2 * kOCols <= 512, "tensor memory");
};

struct Item {
  int s, h, r0, rows;       // sequence, KV head, first row of the tile, rows of the sequence (q_s * G)
  int t0, q_s, n, ctx;      // first packed row, nodes, keys, context keys
  int k0, k1, c, nchunks;   // keys of the chunk, its index, chunks of the sequence
  int live, pad0, pad1, pad2;
};

// barrier area
enum : int {
  kBKFull = 0, kBKEmpty = 6, kBVFull = 12, kBVEmpty = 18, kBSFull = 24, kBPFull = 26, kBODone = 27, kBOFree = 28,
  kBQFull = 30, kBQEmpty = 32, kBQsFull = 34, kBItemFull = 38, kBItemEmpty = 42, kBInfo = 46, kBGroup = 54,
  kBAll = 56, kBDrain = 57, kSTmem = 58, kSAbort = 59, kSVote = 60 /* [2][2] ints: 60, 61 */, kSPoison = 62,
  /* [3] ints: 62, 63 */
  kOffItems = 512, kOffInfo = 768, kOffXch = 896, kOffLinv = 1920, kOffQs = 2688,
};

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

// Issued from one lane of a converged warp (elect.sync), operands uniform.
template <bool F8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  if constexpr (F8) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc));
  } else {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc));
  }
}

__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void st_s128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void st_s64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

// 16-byte chunk c of row r in a swizzled [rows][atom bytes] tile
template <int kAtomB>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return kAtomB == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Reduces NC columns over the 32 lanes by halving: afterwards every lane
// holds column lane / (32 / NC)'s result.
template <int NC, typename Op>
__device__ __forceinline__ float col_reduce(float (&v)[NC], int lane, Op op) {
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
          v[j] = op(keep, __shfl_xor_sync(0xffffffffu, send, s));
        }
      }
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], s));
    }
  }
  return v[0];
}

struct TcArgs {
  TreeParams p;
  int32_t rows_per_seq;  // partial rows of a sequence
  int32_t box;           // slots per TMA box, 0: gather4
  int32_t out_bf16;
  float* part_o;         // [B * rows_per_seq, Hq, D] normalised chunk outputs
  float* part_lse;       // [B * rows_per_seq, Hq]
};

template <int D, int N, bool F8>
__global__ void __launch_bounds__(kThreads, 1)
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
  uint32_t* tslot = reinterpret_cast<uint32_t*>(misc + 8 * kSTmem);
  Item* items = reinterpret_cast<Item*>(misc + kOffItems);
  uint32_t* info = reinterpret_cast<uint32_t*>(misc + kOffInfo);  // [kInfoSlots][4]: keys without a page
  float* xch = reinterpret_cast<float*>(misc + kOffXch);          // [2][4][32]
  float* linv = reinterpret_cast<float*>(misc + kOffLinv);        // [3][64]
  float* qscale = reinterpret_cast<float*>(misc + kOffQs);        // e4m3: [4][64]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
      mbar_init(bar(kBSFull + i), 1);
      mbar_init(bar(kBOFree + i), 8);
      mbar_init(bar(kBQFull + i), 2);
      mbar_init(bar(kBQEmpty + i), 1);
      mbar_init(bar(kBGroup + i), 4);
    }
    mbar_init(bar(kBPFull), 8);
    mbar_init(bar(kBODone), 1);
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(bar(kBQsFull + i), 2);
      mbar_init(bar(kBItemFull + i), 1);
      mbar_init(bar(kBItemEmpty + i), 11);
    }
    for (int i = 0; i < kInfoSlots; ++i) mbar_init(bar(kBInfo + i), 1);
    mbar_init(bar(kBAll), 8);
    mbar_init(bar(kBDrain), 1);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) reinterpret_cast<volatile int*>(misc + 8 * kSVote)[i] = 0;
    for (int i = 0; i < 4; ++i) reinterpret_cast<volatile int*>(misc + 8 * kSPoison)[i] = 0;
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

  // item j as the other warps take it
  auto take = [&](int j, Item& it) -> bool {
    if (!mbar_wait_warp(bar(kBItemFull + j % kItemSlots), (j / kItemSlots) & 1, p.err)) return false;
    it = items[j % kItemSlots];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBItemEmpty + j % kItemSlots));
    return true;
  };
  auto tiles_of = [](const Item& it) { return (it.k1 - it.k0 + kKeys - 1) / kKeys; };

  if (warp == 0) {
    // ======================= items and copies =======================
    const uint64_t pol_once = l2_evict_first_policy(), pol_keep = l2_normal_policy();
    const int64_t n_slots = p.num_blocks * p.bs;
    int gb = 0;                        // the group of sequences gb .. gb + 31 held by the lanes
    int c0 = 0, q_s = 0, n = 0, chunk = 1, nchunks = 0, rts = 0;
    long long cnt = 0, incl = 0, base = 0, total = 0;  // items: this sequence's, prefix in the group; before it; in it
    auto load_group = [&]() {
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
          chunk = tree_chunk(n, q_s);
          nchunks = static_cast<int>(((long long)n + chunk - 1) / chunk);
          rts = static_cast<int>(((int64_t)q_s * G + N - 1) / N);
          cnt = (long long)nchunks * Hkv * rts;
        }
      }
      incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      total = __shfl_sync(0xffffffffu, incl, 31);
    };
    load_group();
    // item number x of the call, or live = 0 past the last
    auto find = [&](long long x) -> Item {
      Item it{};
      while (x >= base + total) {
        base += total;
        gb += 32;
        if (gb >= p.B) return it;
        load_group();
      }
      const int o = __ffs(__ballot_sync(0xffffffffu, base + incl > x)) - 1;
      long long y = x - base - __shfl_sync(0xffffffffu, incl - cnt, o);
      it.s = gb + o;
      it.t0 = __shfl_sync(0xffffffffu, c0, o);
      it.q_s = __shfl_sync(0xffffffffu, q_s, o);
      it.n = __shfl_sync(0xffffffffu, n, o);
      it.nchunks = __shfl_sync(0xffffffffu, nchunks, o);
      const int rt_n = __shfl_sync(0xffffffffu, rts, o), len = __shfl_sync(0xffffffffu, chunk, o);
      it.r0 = static_cast<int>(y % rt_n) * N;
      y /= rt_n;
      it.h = static_cast<int>(y % Hkv);
      it.c = static_cast<int>(y / Hkv);
      it.k0 = static_cast<int>((long long)it.c * len);
      it.k1 = static_cast<int>(min((long long)it.n, (long long)it.k0 + len));
      it.rows = it.q_s * G;
      it.ctx = it.n - it.q_s;
      it.live = 1;
      return it;
    };
    const int bx = a.box;
    const int n_box = bx ? kKeys / bx : 0;
    const int key_of = bx ? (lane % n_box) * bx : lane * 4;  // first key of this lane's box (or four keys)
    const int sub_of = bx ? lane / n_box : 0;                // its sub-tile
    const bool issuer = bx ? sub_of < G_::kSub : true;
    constexpr int32_t kPast = INT32_MIN;
    // pages of this lane's keys in a tile
    auto pages = [&](const Item& it, int t, int32_t (&blk)[4]) {
      const int32_t* row = p.bt + (int64_t)it.s * p.bt_stride;
      const int k = it.k0 + t * kKeys + key_of;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        blk[e] = kPast;
        if ((e == 0 || !bx) && k + e < it.k1) blk[e] = __ldg(row + (p.bs_shift >= 0 ? (k + e) >> p.bs_shift : (k + e) / p.bs));
      }
    };
    // slots of this lane's keys (-1: none), and the tile's keys whose page is
    // out of range as bits in `info`
    auto slots = [&](const Item& it, int t, const int32_t (&blk)[4], int (&sl)[4], int g) {
      const int k = it.k0 + t * kKeys + key_of;
      uint32_t bad = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sl[e] = -1;
        if (e > 0 && bx) break;
        if ((uint32_t)blk[e] < (uint64_t)p.num_blocks) {
          const int lb = p.bs_shift >= 0 ? (k + e) >> p.bs_shift : (k + e) / p.bs;
          sl[e] = blk[e] * p.bs + (k + e - lb * p.bs);
        } else if (blk[e] != kPast) {
          bad |= 1u << e;
        }
      }
      uint32_t* w = info + (g % kInfoSlots) * 4;
      if (lane < 4) w[lane] = 0;
      __syncwarp();
      if (__any_sync(0xffffffffu, bad != 0)) {
        if (bad) {
          atomicOr(p.err, kErrBlockRange);
          if (bx) {
            if (sub_of == 0) atomicOr(w + key_of / 32, (bx == 16 ? 0xffffu : 0xffu) << (key_of & 31));
          } else {
            atomicOr(w + key_of / 32, bad << (key_of & 31));
          }
        }
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(bar(kBInfo + g % kInfoSlots));
    };
    auto load_tile = [&](const Item& it, const int (&sl)[4], uint32_t dst, const CUtensorMap* map, uint32_t full, uint64_t pol) {
      if (lane == 0) mbar_arrive_expect_tx(full, G_::kTileB);
      __syncwarp();
      if (bx) {
        // past the sequence, or a page out of range: out of bounds, which TMA fills with zeros
        if (issuer)
          tma_box(dst + sub_of * kKeys * AT + key_of * AT, map, sub_of * (AT / G_::kEs), it.h,
                  sl[0] >= 0 ? sl[0] : (int)n_slots, full, pol);
      } else {
        int r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = sl[e] >= 0 ? sl[e] * Hkv + it.h : it.h;  // any row: the softmax drops it
#pragma unroll
        for (int u = 0; u < G_::kSub; ++u)
          tma_gather4(dst + u * kKeys * AT + key_of * AT, map, u * (AT / G_::kEs), r, full, pol);
      }
    };
    int j = 0, g = 0;
    bool ok = true;
    Item it = find(blockIdx.x);
    int vs[4] = {-1, -1, -1, -1};  // slots of tile g - 1, whose V follows K of tile g
    int v_h = 0;
    uint64_t v_pol = pol_once;
    auto load_v = [&](int gv) -> bool {
      if (!mbar_wait_warp(bar(kBVEmpty + gv % NV), ((gv / NV) & 1) ^ 1, p.err)) return false;
      Item vi{};
      vi.h = v_h;
      load_tile(vi, vs, sV + (gv % NV) * G_::kTileB, &tm_v, bar(kBVFull + gv % NV), v_pol);
      return true;
    };
    int32_t blk[4];
    if (it.live) pages(it, 0, blk);
    for (;; ++j) {
      ok = ok && mbar_wait_warp(bar(kBItemEmpty + j % kItemSlots), ((j / kItemSlots) & 1) ^ 1, p.err) && !aborted();
      if (!ok) break;
      if (lane == 0) {
        items[j % kItemSlots] = it;
        mbar_arrive(bar(kBItemFull + j % kItemSlots));
      }
      __syncwarp();
      if (!it.live) break;
      const int nt = tiles_of(it);
      const Item next = find(blockIdx.x + (long long)(j + 1) * gridDim.x);
      // K and V are read once where one tile of rows holds them all
      const uint64_t pol = it.rows <= N ? pol_once : pol_keep;
      for (int t = 0; t < nt && ok; ++t, ++g) {
        int32_t nb[4] = {kPast, kPast, kPast, kPast};
        if (t + 1 < nt) {
          pages(it, t + 1, nb);
        } else if (next.live) {
          pages(next, 0, nb);
        }
        ok = mbar_wait_warp(bar(kBKEmpty + g % NK), ((g / NK) & 1) ^ 1, p.err);
        if (!ok) break;
        int sl[4];
        slots(it, t, blk, sl, g);
        load_tile(it, sl, sK + (g % NK) * G_::kTileB, &tm_k, bar(kBKFull + g % NK), pol);
        if (g > 0) ok = load_v(g - 1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          vs[e] = sl[e];
          blk[e] = nb[e];
        }
        v_h = it.h;
        v_pol = pol;
      }
      it = next;
    }
    if (ok && g > 0) ok = load_v(g - 1);
    if (!ok) *abort_flag = 1;
    if (!ok || aborted()) {
      // let the copies issued so far land before the CTA exits
      for (int k = g - 1; k >= 0 && k >= g - NK; --k) mbar_wait_warp(bar(kBKFull + k % NK), (k / NK) & 1, p.err);
      for (int k = g - 1; k >= 0 && k >= g - NV; --k) mbar_wait_warp(bar(kBVFull + k % NV), (k / NV) & 1, p.err);
    }
  } else if (warp == 1) {
    // ======================= MMA =======================
    constexpr uint32_t kIdS = idesc(N, F8, false, false), kIdO = idesc(N, F8, true, true);
    Item it{};
    int j = 0, g = 0;
    auto issue_s = [&](int gg, int qb) -> bool {
      if (!mbar_wait_warp(bar(kBKFull + gg % NK), (gg / NK) & 1, p.err)) return false;
      fence_after();
      const uint64_t dk = sdesc(sK + (gg % NK) * G_::kTileB, 16, 8 * AT, AT);
      const uint64_t dq = sdesc(sQ + qb * G_::kQB, 16, 8 * AT, AT);
      const uint32_t ts = tmem + (gg & 1) * N;
#pragma unroll
      for (int part = 0; part < G_::kParts; ++part)
#pragma unroll
        for (int k = 0; k < G_::kSteps; ++k) {
          constexpr int per = AT / 32;
          const uint32_t ok_ = (uint32_t)((k / per) * kKeys * AT + (k % per) * 32) >> 4;
          const uint32_t oq = (uint32_t)(part * N * G_::kRowB + (k / per) * N * AT + (k % per) * 32) >> 4;
          mma<F8>(ts, dk + ok_, dq + oq, kIdS, (part | k) != 0);
        }
      commit(bar(kBSFull + (gg & 1)));
      commit(bar(kBKEmpty + gg % NK));
      __syncwarp();
      return true;
    };
    auto next_item = [&](int jj) -> bool {
      if (!take(jj, it)) return false;
      return !it.live || mbar_wait_warp(bar(kBQFull + (jj & 1)), (jj >> 1) & 1, p.err);
    };
    bool ok = next_item(0);
    if (ok && it.live) ok = issue_s(0, 0);
    while (ok && it.live && !aborted()) {
      const int nt = tiles_of(it), ob = j & 1;
      for (int t = 0; t < nt && ok; ++t, ++g) {
        if (t + 1 < nt) {
          ok = issue_s(g + 1, j & 1);
        } else {
          commit(bar(kBQEmpty + (j & 1)));
          __syncwarp();
          ok = next_item(j + 1);
          if (ok && it.live) ok = issue_s(g + 1, (j + 1) & 1);
        }
        ok = ok && mbar_wait_warp(bar(kBPFull), g & 1, p.err) &&
             mbar_wait_warp(bar(kBVFull + g % NV), (g / NV) & 1, p.err) &&
             (t > 0 || mbar_wait_warp(bar(kBOFree + ob), ((j >> 1) & 1) ^ 1, p.err));
        if (!ok) break;
        fence_after();
        const uint32_t to = tmem + G_::kColO + ob * G_::kOCols;
        // V^T: d contiguous, 8 keys = 8 AT bytes, sub-tiles kKeys AT apart.  With
        // D = 64 the M side's upper 64 rows repeat shifted keys; their lanes
        // are never read.
        const uint64_t dv = sdesc(sV + (g % NV) * G_::kTileB, G_::kSub * AT / G_::kEs >= 128 && G_::kSub > 1 ? kKeys * AT : 8 * AT,
                                  8 * AT, AT);
        const uint64_t dp = sdesc(sP, G_::kPB, 1024, 128);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int k = 0; k < kKeys / G_::kKeyStep; ++k) {
            const uint32_t ov = (uint32_t)(k * G_::kKeyStep * AT) >> 4;
            const uint32_t op = (uint32_t)(part * G_::kPB + k * G_::kKeyStep * 128) >> 4;
            const uint32_t acc = F8 ? (t > 0 || k > 0) : (t > 0 || k > 0 || part > 0);
            mma<F8>(to + (F8 ? part * N : 0), dv + ov, dp + op, kIdO, acc);
          }
        commit(bar(kBVEmpty + g % NV));
        commit(bar(kBODone));
        __syncwarp();
      }
      ++j;
    }
    if (!ok) *abort_flag = 1;
    // every MMA issued so far is finished before TMEM is freed
    commit(bar(kBDrain));
    __syncwarp();
    mbar_wait_warp(bar(kBDrain), 0, p.err);
  } else if (warp < 4) {
    // ======================= query rows =======================
    constexpr int kLanes = D / 8;            // lanes of a row (8 bf16 elements each)
    constexpr int kPer = 32 / kLanes;        // rows per step of a warp
    constexpr int kStepsQ = N / (2 * kPer);  // steps of a warp
    constexpr int kBatch = kStepsQ < 8 ? kStepsQ : 8;
    const int w = warp - 2, ch = lane % kLanes, rr = lane / kLanes;
    bool ok = true;
    for (int j = 0;; ++j) {
      Item it;
      ok = take(j, it) && !aborted();
      if (!ok || !it.live) break;
      const int qb = j & 1;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
      bool waited = false;
#pragma unroll 1
      for (int b = 0; b < kStepsQ && ok; b += kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int r = it.r0 + ((b + k) * 2 + w) * kPer + rr;
          x[k] = make_uint4(0, 0, 0, 0);
          if (r < it.rows) {
            const int i = r / G;
            x[k] = __ldg(reinterpret_cast<const uint4*>(q + (int64_t)(it.t0 + i) * p.q_st +
                                                        (int64_t)(it.h * G + r - i * G) * p.q_sh) + ch);
          }
        }
        if (!waited) {
          ok = mbar_wait_warp(bar(kBQEmpty + qb), ((j >> 1) & 1) ^ 1, p.err);
          if (!ok) break;
          waited = true;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int r = ((b + k) * 2 + w) * kPer + rr;  // row of the tile
          const uint32_t dst = sQ + qb * G_::kQB;
          if constexpr (!F8) {
            st_s128(dst + (ch * 16 / AT) * N * AT + swz<AT>(r, ch % (AT / 16)), x[k].x, x[k].y, x[k].z, x[k].w);
          } else {
            float f[8];
            const uint32_t wd[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            float mx = 0.f;
            bool fine = true;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[2 * e] = bf16_lo(wd[e]);
              f[2 * e + 1] = bf16_hi(wd[e]);
              mx = fmaxf(mx, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
              fine = fine && fabsf(f[2 * e]) < INFINITY && fabsf(f[2 * e + 1]) < INFINITY;
            }
            int nan = !fine;
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) {
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              nan |= __shfl_xor_sync(0xffffffffu, nan, o);
            }
            // 2^e <= largest < 2^(e + 1); e is kept where 2^(7 - e) is a normal number
            int e2 = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
            e2 = e2 < -100 ? -100 : e2;
            const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - e2) << 23);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - 7 + e2) << 23);
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float u0 = nan ? 0.f : f[2 * e] * up, u1 = nan ? 0.f : f[2 * e + 1] * up;
              const uint16_t h2 = f32x2_to_e4m3x2(u0, u1);
              const uint32_t hf = e4m3x2_to_f16x2(h2);
              const float2 hv = __half22float2(*reinterpret_cast<const __half2*>(&hf));
              const uint16_t l2 = f32x2_to_e4m3x2(u0 - hv.x, u1 - hv.y);
              if (e & 1) {
                hi[e >> 1] |= (uint32_t)h2 << 16;
                lo[e >> 1] |= (uint32_t)l2 << 16;
              } else {
                hi[e >> 1] = h2;
                lo[e >> 1] = l2;
              }
            }
            const uint32_t at = swz<AT>(r, ch >> 1) + (ch & 1) * 8;
            st_s64(dst + at, hi[0], hi[1]);
            st_s64(dst + N * G_::kRowB + at, lo[0], lo[1]);
            if (ch == 0)
              qscale[(j % 4) * 64 + r] = nan ? __uint_as_float(0x7fffffffu) : down * p.qk_scale_log2;
          }
        }
      }
      if (!ok) break;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kBQFull + qb));
        if (F8) mbar_arrive(bar(kBQsFull + j % 4));
      }
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ======================= softmax =======================
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int w8 = warp - 4;
    const int tg = quarter * 32 + lane;  // thread of the half's group; also this lane's key in a tile, and its d of O^T
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    constexpr float kTau = F8 ? 4.5f : 10.f;     // p may pass 2^0 by this much before the reference moves
    constexpr float kUp = F8 ? 4.f : 0.f;        // e4m3: p is kept times 2^4
    volatile int* vote = reinterpret_cast<volatile int*>(misc + 8 * kSVote) + 2 * half;
    volatile int* poison = reinterpret_cast<volatile int*>(misc + 8 * kSPoison);  // [3]
    float* xh = xch + half * 128;
    int gs = 0, as = 0;  // group / whole synchronisations so far
    auto group_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBGroup + half));
      const bool r = mbar_wait_warp(bar(kBGroup + half), gs & 1, p.err);
      ++gs;
      return r;
    };
    auto all_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBAll));
      const bool r = mbar_wait_warp(bar(kBAll), as & 1, p.err);
      ++as;
      return r;
    };
    auto fmax_op = [](float x, float y) { return fmaxf(x, y); };
    auto add_op = [](float x, float y) { return x + y; };
    int g = 0;
    bool ok = true;
    float ref[NC], l[NC];
    // the item whose O is still to be written
    bool pend = false;
    Item pi{};
    int pj = 0;

    // Writes O / l of item pj: lane = d, register = row.
    auto epilogue = [&]() {
      pend = false;
      fence_after();
      const uint32_t to = tmem + G_::kColO + (pj & 1) * G_::kOCols + lane_off + half * NC;
      uint32_t o[NC];
      tm_ld(to, o);
      float v[NC];
      if constexpr (F8) {
        uint32_t o2[NC];
        tm_ld(to + N, o2);
        wait_ld();
#pragma unroll
        for (int c = 0; c < NC; ++c) v[c] = fmaf(__uint_as_float(o2[c]), 0.0625f, __uint_as_float(o[c]));
      } else {
        wait_ld();
#pragma unroll
        for (int c = 0; c < NC; ++c) v[c] = __uint_as_float(o[c]);
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBOFree + (pj & 1)));
      if (tg >= D) return;
      const float* li = linv + (pj % 3) * 64 + half * NC;
      const int ra = pi.r0 + half * NC;  // first row of this half
      if (poison[pj % 3] == pj + 1) {
        // a drafted value is not finite: it was taken out of the product and
        // goes to the rows that see its key
        for (int k = max(pi.ctx, pi.k0); k < pi.k1; ++k) {
          const int lb = k / p.bs;
          const int32_t b = __ldg(p.bt + (int64_t)pi.s * p.bt_stride + lb);
          if ((uint32_t)b >= (uint64_t)p.num_blocks) continue;
          const int64_t at = (((int64_t)b * p.bs + (k - lb * p.bs)) * Hkv + pi.h) * D + tg;
          float x;
          if constexpr (F8) {
            const uint32_t hf = e4m3x2_to_f16x2(static_cast<const uint8_t*>(p.v_cache)[at]);
            x = __half2float(__ushort_as_half(static_cast<unsigned short>(hf & 0xffffu)));
          } else {
            x = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_cache)[at]);
          }
          if (fabsf(x) < INFINITY) continue;
          const int jj = k - pi.ctx;
#pragma unroll 1
          for (int c = 0; c < NC; ++c) {
            const int r = ra + c;
            if (r >= pi.rows) break;
            if ((static_cast<uint32_t>(__ldg(p.mask + (int64_t)(pi.t0 + r / G) * p.mask_stride + (jj >> 5))) >> (jj & 31)) & 1u) {
#pragma unroll
              for (int e = 0; e < NC; ++e)
                if (e == c) v[e] += x;
            }
          }
        }
      }
      if (ra >= pi.rows) return;
      int i = ra / G, gq = ra - i * G;
      if (pi.nchunks == 1) {
        int64_t at = (int64_t)(pi.t0 + i) * p.o_st + (int64_t)(pi.h * G + gq) * p.o_sh + tg;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (ra + c >= pi.rows) break;
          const float s = li[c];
          const float y = s == 0.f ? 0.f : v[c] * s;
          if (a.out_bf16)
            store1(static_cast<__nv_bfloat16*>(p.out) + at, y);
          else
            store1(static_cast<float*>(p.out) + at, y);
          at += p.o_sh;
          if (++gq == G) {
            gq = 0;
            at += p.o_st - (int64_t)G * p.o_sh;
          }
        }
      } else {
        int64_t at = (((int64_t)pi.s * a.rows_per_seq + (int64_t)i * pi.nchunks + pi.c) * p.Hq + pi.h * G + gq) * D + tg;
        const int64_t wrap = ((int64_t)pi.nchunks * p.Hq - G) * D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (ra + c >= pi.rows) break;
          const float s = li[c];
          a.part_o[at] = s == 0.f ? 0.f : v[c] * s;
          at += D;
          if (++gq == G) {
            gq = 0;
            at += wrap;
          }
        }
      }
    };

    for (int j = 0;; ++j) {
      Item it;
      ok = take(j, it) && !aborted();
      if (!ok || !it.live) break;
      const int nt = tiles_of(it);
      const float* qs = qscale + (j % 4) * 64 + half * NC;
      if (F8) {
        ok = mbar_wait_warp(bar(kBQsFull + j % 4), (j >> 2) & 1, p.err);
        if (!ok) break;
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        ref[c] = -INFINITY;
        l[c] = 0.f;
      }
      const int ra = it.r0 + half * NC;
      bool virgin = true;  // some row has not seen a key yet
      for (int t = 0; t < nt; ++t, ++g) {
        ok = mbar_wait_warp(bar(kBSFull + (g & 1)), (g >> 1) & 1, p.err) &&
             mbar_wait_warp(bar(kBInfo + g % kInfoSlots), (g / kInfoSlots) & 1, p.err);
        if (!ok) break;
        fence_after();
        float x[NC];
        {
          uint32_t u[NC];
          tm_ld(tmem + (g & 1) * N + half * NC + lane_off, u);
          const uint32_t* bw = info + (g % kInfoSlots) * 4;
          const uint32_t bad0 = bw[0], bad1 = bw[1], bad2 = bw[2], bad3 = bw[3];
          wait_ld();
#pragma unroll
          for (int c = 0; c < NC; ++c) x[c] = __uint_as_float(u[c]) * (F8 ? qs[c] : p.qk_scale_log2);
          const int kt = it.k0 + t * kKeys;  // first key of the tile
          const bool any_bad = (bad0 | bad1 | bad2 | bad3) != 0;
          const bool masked = kt + kKeys > it.ctx || any_bad;
          bool slow = t == 0 || masked || virgin;
          if (masked) {
            const int key = kt + tg, jj = key - it.ctx;
            const uint32_t badw = quarter == 0 ? bad0 : quarter == 1 ? bad1 : quarter == 2 ? bad2 : bad3;
            const bool in = key < it.k1 && !((badw >> lane) & 1u);
            int i = ra / G, gq = ra - i * G;
            const int32_t* mrow = p.mask + (int64_t)(it.t0 + i) * p.mask_stride + (jj > 0 ? jj >> 5 : 0);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              bool see = in && ra + c < it.rows;
              if (see && jj >= 0) see = (static_cast<uint32_t>(__ldg(mrow)) >> (jj & 31)) & 1u;
              x[c] = see ? x[c] : -INFINITY;
              if (++gq == G) {
                gq = 0;
                mrow += p.mask_stride;
              }
            }
            // V rows that some row of the product must not see: zero what is
            // past the sequence or has no page, and what is not finite among
            // the drafted rows (the epilogue hands that on)
            if (!mbar_wait_warp(bar(kBVFull + g % NV), (g / NV) & 1, p.err)) { ok = false; break; }
            constexpr int kLn = G_::kRowB / 16, kRs = 32 / kLn;
            const int ch = lane % kLn, rr = lane / kLn;
            bool found = false;
            for (int b = 0; b < 16; b += kRs) {
              const int kk = w8 * 16 + b + rr;
              const int ky = kt + kk;
              const uint32_t bm = kk < 32 ? bad0 : kk < 64 ? bad1 : kk < 96 ? bad2 : bad3;
              const bool gone = ky >= it.k1 || ((bm >> (kk & 31)) & 1u);
              if (!gone && ky < it.ctx) continue;
              const uint32_t at = sV + (g % NV) * G_::kTileB + (ch * 16 / AT) * kKeys * AT + swz<AT>(kk, ch % (AT / 16));
              if (gone) {
                st_s128(at, 0, 0, 0, 0);
                continue;
              }
              uint32_t w[4];
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
              bool hit = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if constexpr (F8) {
#pragma unroll
                  for (int f = 0; f < 4; ++f)
                    if (((w[e] >> (8 * f)) & 0x7fu) == 0x7fu) {
                      w[e] &= ~(0xffu << (8 * f));
                      hit = true;
                    }
                } else {
#pragma unroll
                  for (int f = 0; f < 2; ++f)
                    if (((w[e] >> (16 * f)) & 0x7f80u) == 0x7f80u) {
                      w[e] &= ~(0xffffu << (16 * f));
                      hit = true;
                    }
                }
              }
              if (hit) {
                st_s128(at, w[0], w[1], w[2], w[3]);
                found = true;
              }
            }
            if (found) poison[j % 3] = j + 1;
            fence_proxy_async_smem();
            if (!all_sync()) { ok = false; break; }
          }
          if (!slow) {
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < NC; ++c) top = fmaxf(top, x[c] - ref[c]);
            if (__any_sync(0xffffffffu, top > kTau)) vote[gs & 1] = gs + 1;
            const int tag = gs + 1, vb = gs & 1;
            if (!group_sync()) { ok = false; break; }
            slow = vote[vb] == tag;
          }
          if (slow) {
            float m[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) m[c] = x[c] == x[c] ? x[c] : -INFINITY;
            const float mine = col_reduce<NC>(m, lane, fmax_op);
            if (lane % (32 / NC) == 0) xh[quarter * 32 + lane / (32 / NC)] = mine;
            if (!group_sync()) { ok = false; break; }
            // move the references that were passed; O (every P V so far has
            // run after this wait) and the sums follow, eight rows at a time
            if (t > 0) {
              if (!mbar_wait_warp(bar(kBODone), (g - 1) & 1, p.err)) { ok = false; break; }
              fence_after();
            }
            virgin = false;
            const uint32_t to = tmem + G_::kColO + (j & 1) * G_::kOCols + lane_off + half * NC;
#pragma unroll
            for (int b = 0; b < NC; b += 8) {
              float al[8];
              bool moved = false;  // the same in all warps of the half
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float mx = fmaxf(fmaxf(xh[b + c], xh[32 + b + c]), fmaxf(xh[64 + b + c], xh[96 + b + c]));
                float& rf = ref[b + c];
                const bool need = mx > rf + kTau || (rf == -INFINITY && mx > -INFINITY);
                const float nr = need ? mx : rf;
                al[c] = need ? ex2(rf - nr) : 1.f;
                moved = moved || need;
                rf = nr;
                virgin = virgin || nr == -INFINITY;
                l[b + c] *= al[c];
              }
              if (t > 0 && moved) {
#pragma unroll
                for (int part = 0; part < (F8 ? 2 : 1); ++part) {
                  uint32_t o[8];
                  tm_ld(to + part * N + b, o);
                  wait_ld();
#pragma unroll
                  for (int c = 0; c < 8; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * al[c]);
                  tm_st(to + part * N + b, o);
                }
              }
            }
            wait_st();
            // xh is written again only after another synchronisation of the group
            if (!group_sync()) { ok = false; break; }
          }
        }
        // P = 2^(s - ref), in two parts, to shared memory: row = key
        uint32_t hi[F8 ? NC / 4 : NC / 2], lo[F8 ? NC / 4 : NC / 2];
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
          const float r0 = ref[c] == -INFINITY ? 0.f : ref[c], r1 = ref[c + 1] == -INFINITY ? 0.f : ref[c + 1];
          const float p0 = ex2(x[c] - r0 + kUp), p1 = ex2(x[c + 1] - r1 + kUp);
          l[c] += p0;
          l[c + 1] += p1;
          if constexpr (F8) {
            const uint16_t h2 = f32x2_to_e4m3x2(p0, p1);
            const uint32_t hf = e4m3x2_to_f16x2(h2);
            const float2 hv = __half22float2(*reinterpret_cast<const __half2*>(&hf));
            const uint16_t l2 = f32x2_to_e4m3x2((p0 - hv.x) * 16.f, (p1 - hv.y) * 16.f);
            if (c & 2) {
              hi[c / 4] |= (uint32_t)h2 << 16;
              lo[c / 4] |= (uint32_t)l2 << 16;
            } else {
              hi[c / 4] = h2;
              lo[c / 4] = l2;
            }
          } else {
            const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
            hi[c / 2] = __byte_perm(u0, u1, 0x7632);
            lo[c / 2] = __byte_perm(__float_as_uint(p0 - __uint_as_float(u0 & 0xFFFF0000u)),
                                    __float_as_uint(p1 - __uint_as_float(u1 & 0xFFFF0000u)), 0x7632);
          }
        }
        // the buffer is free once P V of the previous tile has run
        if (g > 0 && !mbar_wait_warp(bar(kBODone), (g - 1) & 1, p.err)) { ok = false; break; }
        if constexpr (F8) {
          if constexpr (NC == 8) {
            st_s64(sP + swz<128>(tg, 0) + half * 8, hi[0], hi[1]);
            st_s64(sP + G_::kPB + swz<128>(tg, 0) + half * 8, lo[0], lo[1]);
          } else {
#pragma unroll
            for (int c = 0; c < NC / 16; ++c) {
              const uint32_t at = sP + swz<128>(tg, half * (NC / 16) + c);
              st_s128(at, hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
              st_s128(at + G_::kPB, lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < NC / 8; ++c) {
            const uint32_t at = sP + swz<128>(tg, half * (NC / 8) + c);
            st_s128(at, hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
            st_s128(at + G_::kPB, lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
          }
        }
        fence_proxy_async_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBPFull));
        if (t == 0 && pend) epilogue();  // the previous item's last P V was waited for above
      }
      if (!ok) break;
      // the rows' sums over the lanes and the four warps of the half
      {
        float m[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) m[c] = l[c];
        const float mine = col_reduce<NC>(m, lane, add_op);
        if (lane % (32 / NC) == 0) xh[quarter * 32 + lane / (32 / NC)] = mine;
        if (!group_sync()) { ok = false; break; }
        if (tg < NC) {
          const float s = (xh[tg] + xh[32 + tg]) + (xh[64 + tg] + xh[96 + tg]);
          linv[(j % 3) * 64 + half * NC + tg] = s == 0.f ? 0.f : p.v_scale / s;
          float rf = 0.f;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (c == tg) rf = ref[c];
          const int r = ra + tg;
          if (it.nchunks > 1 && r < it.rows) {
            const int i = r / G;
            a.part_lse[((int64_t)it.s * a.rows_per_seq + (int64_t)i * it.nchunks + it.c) * p.Hq + it.h * G + r - i * G] =
                s == 0.f ? -INFINITY : rf + log2f(s) - kUp;
          }
        }
        if (!group_sync()) { ok = false; break; }
      }
      pend = true;
      pi = it;
      pj = j;
    }
    if (ok && pend) {
      if (mbar_wait_warp(bar(kBODone), (g - 1) & 1, p.err))
        epilogue();
      else
        ok = false;
    }
    if (!ok) *abort_flag = 1;
  }
  // ---- teardown
  fence_before();
  __syncthreads();
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
                                                        int rows_per_seq) {
  grid_dep_wait();
  launch_dependents();
  constexpr int E = D / 32;
  const int s = blockIdx.x, lane = threadIdx.x & 31;
  const int c0 = __ldg(p.cu_q + s), c1 = __ldg(p.cu_q + s + 1), n = __ldg(p.seq_lens + s);
  const int q_s = c1 - c0;
  if (c0 < 0 || c1 <= c0 || (int64_t)c1 > p.T || q_s > n || (int64_t)n > (int64_t)p.max_blocks * p.bs || q_s > p.max_nodes)
    return;
  const int chunk = tree_chunk(n, q_s);
  const int nc = static_cast<int>(((long long)n + chunk - 1) / chunk);
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
  return launch_ex(kern, dim3((unsigned)grid), dim3(kThreads), G_::kSmem, st, true, a, mk, mv);
}

}  // namespace

int64_t tree_tc_rows_per_seq(int64_t max_q, int64_t max_ctx) {
  const int64_t chunks = std::min<int64_t>(kTreeMaxChunks, (max_ctx + kTreeMinChunk - 1) / kTreeMinChunk);
  if (chunks <= 1) return 0;
  return std::min<int64_t>(max_q * chunks, kTreePartRows);
}

cudaError_t launch_tree_tc(const TreeParams& p, bool f8, int out_kind, int64_t max_q, int64_t max_ctx, void* workspace,
                           int num_sms, cudaStream_t st) {
  TcArgs a{};
  a.p = p;
  a.out_bf16 = out_kind;
  const int64_t rps = tree_tc_rows_per_seq(max_q, max_ctx);
  a.rows_per_seq = static_cast<int32_t>(rps);
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = a.part_o + (int64_t)p.B * rps * p.Hq * p.D;
  // rows per MMA tile: the narrowest that holds the largest tree
  const int64_t rows = max_q * p.G;
  const int N = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
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
#define PKV_JOIN(D, O) launch_ex(tree_join_kernel<D, O>, grid, dim3(256), 0, st, true, p, (const float*)a.part_o, (const float*)a.part_lse, a.rows_per_seq)
  if (p.D == 128) return out_kind ? PKV_JOIN(128, __nv_bfloat16) : PKV_JOIN(128, float);
  return out_kind ? PKV_JOIN(64, __nv_bfloat16) : PKV_JOIN(64, float);
#undef PKV_JOIN
}

}  // namespace pkv
