// pkv_tree_narrow.cuh -- attention over the paged cache on the fifth-generation
// tensor cores for up to 64 query rows that read the same keys, split along the
// keys: drafted trees (pkv_tree_tc.cu), and requests that share a prefix
// (pkv_share_tc.cu), whose rows are those of a group or of one request.
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
// call's shapes, not from the other sequences (tree_chunk).  Chunks write
// normalised partials and log2-sum-exp2, and a second small kernel joins them in
// order.  Items are dealt to the persistent CTAs (one per SM) in strides; every
// CTA finds its items by scanning the lengths, 32 sequences per step, so a call
// needs no plan, keeps nothing between calls, and its workspace holds only the
// partials.
//
// Types: bf16 caches take bf16 MMAs, P as bf16 hi + lo (about 16 bits).  e4m3
// caches: S takes K's codes as they are (kind::f8f6f4, no conversion): a query
// row is scaled to a largest element in [128, 256) and split into two e4m3 parts
// (a bf16 element has 8 significant bits, an e4m3 code 4: hi + lo is exact down
// to 2^-18 of the row's largest element).  P V is in f16: the softmax warps
// widen V's codes (exactly), and P = 2^8 * 2^(s - ref) <= 2^15.75 is one f16, as
// in decode: 11 bits, and keys as far as 2^-33 below the reference, which is a
// score that was seen, still weigh something.  (P as two e4m3 codes saved
// the widening and lost what lay 15.5 powers of two below the reference: behind
// one leading key the mass of thousands of small ones went missing, several per
// cent of an output.  With the widening, 8 trees of 16 nodes over 32K to 128K
// keys take 324 us instead of 296, and 64 trees of 4 / 8 / 16 nodes times 4 heads
// over 4,096 to 16,384 (16 nodes: 512 to 4,096) keys, cut alike, 277 / 327 / 147
// instead of 268 / 285 / 137.  With the V codes' loads behind the wait for S, one after the other
// between conversions, the first took 20 us more.)
//
// More than 64 rows (bf16 caches) go to pkv_tree_wide.cuh, whose tiles of 128 rows
// put the rows on the M side: up to 64 rows this kernel is the faster one (64
// trees of 8 / 12 / 16 nodes times 4 heads over 512 to 4,096 keys: 109 / 129 / 132
// us here, 126 / 131 / 135 there), above it the other (16 trees of 64 nodes over
// up to 8,192 keys: 192 and 150 us when it was new, 109 now).
//
// Bound: the memory while there are few rows, then the softmax: with a key per
// lane each warp runs about 290 instructions for 32 keys and 16 rows; with e4m3
// caches also the widening, which waits for V's codes and shares the issue slots.
// Measured, with the join: 64 trees of 8 nodes over 512 to 4,096 keys, bf16: 109
// us (5.5 TB/s of 600 MB, 81 % of a plain copy's rate); 8 trees of 16 nodes over
// 32K to 128K keys, e4m3: 324 us (3.8 TB/s of 1,240 MB); one tree of 8 nodes over
// 2,048 keys: 11.1 us.
//
// CTA: 16 warps, 24 for N = 64.
//   warps 0, 3  copy the K and the V tiles of 128 keys by TMA: boxes of 16, 8 or
//               4 slots that lie in one block, or, for other block sizes, four
//               arbitrary rows at a time (tile::gather4).
//   warp 1      issues the MMAs: S of tile g + 1, then P V of tile g.  The two
//               parts of P are 2 N columns of one operand, so O holds their two
//               products side by side and P V costs one pass of instructions.
//   warp 2      finds the items, publishes them and brings their query rows:
//               bf16 to the swizzled operand layout, or split to e4m3.
//   then 8 or 16 (N = 64) warps of softmax: lane quarter w % 4 = keys, group
//               (w - 4) / 4 = rows.
//   and 4 warps that write O / l of finished items while the next one runs.
#pragma once
#include <type_traits>

#include "pkv_tree_tc.cuh"

namespace pkv {
namespace {

// ---------------------------------------------------------------- geometry
template <int D, int N, bool F8, bool S>
struct Geo {
  static constexpr int kD = D, kN = N;
  static constexpr bool kF8 = F8, kShared = S;
  static constexpr int kEs = F8 ? 1 : 2;                      // of a cache element; those of P V have two bytes
  static constexpr int kRowB = D * kEs;                       // one K or V row
  static constexpr int kAtomB = kRowB < 128 ? kRowB : 128;    // swizzle width
  static constexpr int kSub = kRowB / kAtomB;                 // sub-tiles along d
  static constexpr int kTileB = kKeys * kRowB;
  static constexpr int kParts = F8 ? 2 : 1;                   // parts of Q
  static constexpr int kQB = N * kRowB * kParts;
  static constexpr int kVRowB = 2 * D;                        // a V row in the product (e4m3: widened)
  static constexpr int kVSub = kVRowB / 128;
  static constexpr int kWideB = F8 ? kKeys * kVRowB : 0;      // a widened V tile; there are two, as of P
  static constexpr int kParts2 = F8 ? 1 : 2;                  // parts of P
  static constexpr int kPRow = 2 * N * kParts2;               // P of one key
  static constexpr int kPB = kKeys * (kPRow <= 128 ? 128 : 256);  // [1 or 2][128 keys][128 bytes]
  // tiles of K and of V in flight (of V codes fewer: they are free once they are widened)
  static constexpr int kNK = F8 ? (D == 128 ? (N == 16 ? 4 : 3) : 6) : D == 128 ? 2 : 4;
  static constexpr int kNV = F8 ? (D == 128 ? (N == 64 ? 2 : 3) : 6) : D == 128 ? (kPRow == 256 ? 2 : 3) : (kPRow == 256 ? 4 : 5);
  static constexpr int kGroups = N == 64 ? 4 : 2;             // softmax: groups of four warps, each N / kGroups rows
  static constexpr int kSoft = 4 * kGroups;                   // its warps
  static constexpr int kThreads = 32 * (4 + kSoft + 4);
  static constexpr int kNC = N / kGroups;                     // rows (columns of S^T) per softmax warp
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kNK * kTileB;
  static constexpr int kOffWide = kOffV + kNV * kTileB;
  static constexpr int kOffP = kOffWide + 2 * kWideB;
  static constexpr int kOffQ = kOffP + 2 * kPB;
  static constexpr int kQBufs = kPRow == 256 && kTileB == 32768 ? 1 : 2;  // query tiles: the next item's arrives while this one runs
  // item j's query buffer, and the parity of its pass
  __device__ static int qbuf(int j) { return kQBufs == 2 ? j & 1 : 0; }
  __device__ static uint32_t qpass(int j) { return (uint32_t)(kQBufs == 2 ? j >> 1 : j) & 1u; }
  static constexpr int kOffMisc = kOffQ + kQBufs * kQB;
  static constexpr int kSmem = kOffMisc + kMiscBytes;
  // tensor memory: S 2 x N columns, then O 2 x (hi N, lo N), or 2 x N
  static constexpr uint32_t kColO = 2 * N;
  static constexpr uint32_t kOCols = kParts2 * N;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kNK + 2 <= kInfoSlots, "tile info ring");
  static_assert(kColO + 2 * kOCols <= 512, "tensor memory");
};
enum : int {
  kOffXch = kOffOwn /* [groups][4][rows] */, kOffSum = 1968 /* [2][4][64] */,
  kOffLref = 4016 /* [2][64] */, kOffRef = 4528 /* [3][64] */, kOffQs = 5296 /* e4m3: [4][64] */,
  kOffUnset = 6320 /* [groups][4] */, kOffFlag = 6384 /* [groups][2] */,
};
static_assert(kOffFlag + 32 <= kMiscBytes, "shared memory");

// A drafted value (element d of some V row) is not finite: the softmax warps
// took it out of the product, and here it goes to the rows that see its key,
// on top of what this thread has just stored.
template <int D, int N, bool F8, bool S>
__device__ __noinline__ void add_poison(const TcArgs& a, const Item& it, int d) {
  const TreeParams& p = a.p;
  const int ctx = it.ctx, rows = it.q_s * p.G;
  const Part part = part_of<S>(a, it);
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
      if (!sees<S>(p, it, i, jj)) continue;
      if (part.split) {
        a.part_o[((part.at + i * part.step) * p.Hq + hq) * D + d] += x;
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

// A softmax warp's share of a tile of V codes, widened to f16 for the product.  A
// lane takes 16 codes of a row at a time, 16 bytes in and twice 16 out; the rows
// of eight neighbouring lanes are chosen so that neither side has bank
// conflicts.  load() and store() are apart so that waits go between them.
template <class G_>
struct WidenV {
  static constexpr int AT = G_::kAtomB, kRows = kKeys / G_::kSoft;
  static constexpr int kSteps = kRows / (AT == 128 ? 4 : 8);
  static_assert(kRows % 8 == 0 && G_::kSub == 1, "codes of a row in one swizzle atom");
  int row;            // the lane's row in the first step
  uint32_t from, from_x, to, to_x;  // its place in both tiles: offset, and the swizzled chunk
  uint32_t w[kSteps][4];
  __device__ __forceinline__ WidenV(int w_of, int lane) {
    // D = 128: eight lanes hold four chunks of rows r and r ^ 5; D = 64: all four of rows r and r ^ 1
    const int ch = AT == 128 ? (lane & 3) | (lane & 8) >> 1 : lane & 3;
    const int r = AT == 128 ? (lane >> 4) ^ (lane & 4 ? 5 : 0) : lane >> 2;
    row = w_of * kRows + r;
    from = row * AT;
    from_x = (ch ^ (AT == 128 ? r : r >> 1)) << 4;
    to = (ch >> 2) * (kKeys * 128) + row * 128;
    to_x = (((2 * ch) & 7) ^ r) << 4;
  }
  // rows further down, and the change of the swizzle: D = 128: steps take rows 0,
  // 1, 4, 5 and 2, 3, 6, 7 of eight
  __device__ static constexpr int down(int b) { return AT == 128 ? (b & 1) * 2 + (b >> 1) * 8 : b * 8; }
  __device__ static constexpr uint32_t turn(int b) { return (AT == 128 ? (b & 1) * 2 : 0) << 4; }
  __device__ __forceinline__ void load(uint32_t codes) {
#pragma unroll
    for (int b = 0; b < kSteps; ++b)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[b][0]), "=r"(w[b][1]), "=r"(w[b][2]), "=r"(w[b][3])
                   : "r"(codes + from + down(b) * AT + (from_x ^ turn(b))));
  }
  // what clean_v does to a bf16 tile; true: a drafted value is not finite
  __device__ __forceinline__ bool clean(int kt, int ctx, int k1, const uint4& bad) {
    bool found = false;
    const int first = row & ~31;
    const uint32_t bm = first == 0 ? bad.x : first == 32 ? bad.y : first == 64 ? bad.z : bad.w;  // a warp's rows lie in one word
#pragma unroll
    for (int b = 0; b < kSteps; ++b) {
      const int kk = row + down(b), ky = kt + kk;
      const bool gone = ky >= k1 || ((bm >> (kk & 31)) & 1u);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // NaN, the only code that is not finite: ones all over but for the sign,
        // which carry into the sign's place
        const uint32_t t = ky >= ctx ? ((w[b][e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u : 0u;
        found |= t != 0 && !gone;
        w[b][e] = gone ? 0u : w[b][e] & ~((t >> 7) * 0xffu);
      }
    }
    return found;
  }
  __device__ __forceinline__ void store(uint32_t wide) const {
#pragma unroll
    for (int b = 0; b < kSteps; ++b) {
      uint32_t h[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) e4m3x4_to_f16(w[b][e], h[2 * e], h[2 * e + 1]);
      const uint32_t at = wide + to + down(b) * 128 + (to_x ^ turn(b));
      st_s128(at, h[0], h[1], h[2], h[3]);
      st_s128(at ^ 16, h[4], h[5], h[6], h[7]);
    }
  }
};
struct NoWiden {
  __device__ __forceinline__ NoWiden(int, int) {}
};

template <int D, int N, bool F8, bool S>
__global__ void __launch_bounds__(Geo<D, N, F8, S>::kThreads, 1)
    tree_tc_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v) {
  using G_ = Geo<D, N, F8, S>;
  constexpr int NC = G_::kNC, NK = G_::kNK, NV = G_::kNV, AT = G_::kAtomB;
  const TreeParams& p = a.p;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* misc = smem + G_::kOffMisc;
  const uint32_t s0 = smem_u32(smem), b0 = smem_u32(misc);
  auto bar = [&](int i) -> uint32_t { return b0 + 8 * i; };
  const uint32_t sK = s0 + G_::kOffK, sV = s0 + G_::kOffV, sP = s0 + G_::kOffP, sQ = s0 + G_::kOffQ, sW = s0 + G_::kOffWide;
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
  const int G = p.G;
  const Cta cta{b0, abort_flag, items, info, lane};

  if (s0 & 1023) {  // the swizzled tiles need their base on 1024 bytes
    if (threadIdx.x == 0) atomicOr(p.err, kErrWaitTimeout);
    if (S) grid_dep_wait();
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(bar(kBKFull + i), 1);
      mbar_init(bar(kBKEmpty + i), 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(bar(kBVFull + i), 1);
      mbar_init(bar(kBVEmpty + i), F8 ? G_::kSoft : 1);
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
  begin_phase<S>(a);
  // Trees: no launch_dependents(): the join starts when the last CTAs end.  With its grid
  // pending from here on, the 32K to 128K key case took 385 us in a loop of calls
  // and 343 from a graph, instead of 324; 64 trees of 4 / 8 / 16 nodes, e4m3, 270 /
  // 334 / 146 instead of 263 / 315 / 141; of 8 nodes, bf16, 108.0 and 108.2.

  if (warp == 0 || warp == 3) {
    copy_tiles<G_>(a, cta, warp == 3, warp == 3 ? sV : sK, warp == 3 ? &tm_v : &tm_k);
  } else if (warp == 1) {
    // ======================= MMA =======================
    constexpr uint32_t kIdS = idesc(N, F8, false, false), kIdO = idesc(G_::kParts2 * N, F8, true, true);
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
      if (t == nt - 1 && elect_one()) commit(bar(kBQEmpty + G_::qbuf(j - 1)));
      int nt2 = nt;
      if (t + 1 >= nt) {  // the tile whose S goes next is the next item's first
        Item it;
        ok = cta.take(ir, it);
        nt2 = it.nt;
        if (!ok || (nt2 == 0 && nt == 0)) break;
        ok = nt2 == 0 || wait_bar(bar(kBQFull + G_::qbuf(j)), G_::qpass(j));
        if (!ok) break;
      }
      const int gs = nt == 0 ? g : g + 1, qb = G_::qbuf(t + 1 >= nt ? j : j - 1);
      if (nt2 > 0 || t + 1 < nt) ok = issue_s(gs, qb);
      if (nt > 0 && ok) {
        const int ob = ~j & 1;
        // (e4m3: the arrivals on P's barrier tell of the widened V tile too)
        ok = (F8 || wait_bar(bar(kBVFull) + 8 * vr.at, vr.pass)) && (t > 0 || wait_bar(bar(kBOFree + ob), (((j - 1) >> 1) & 1) ^ 1)) &&
             wait_bar(bar(kBPFull + (g & 1)), (g >> 1) & 1);
        if (!ok) break;
        fence_after();
        // V^T: d contiguous, 8 keys = 1,024 bytes, sub-tiles of d kKeys * 128 apart.
        // With D = 64 the M side's upper 64 rows repeat shifted keys; their lanes
        // are never read.
        const uint32_t v_at = F8 ? sW + (g & 1) * G_::kWideB : sV + vr.at * G_::kTileB;
        const uint64_t dv = sdesc(v_at, G_::kVSub > 1 ? kKeys * 128 : 1024, 1024, 128);
        const uint64_t dp = sdesc(sP + (g & 1) * G_::kPB, kKeys * 128, 1024, 128);
        const uint32_t to = tmem + G_::kColO + ob * G_::kOCols;
        if (elect_one()) {
          mma_steps<false, 8, 128, 128>(to, dv, dp, kIdO, t > 0);  // 16 keys of 128 bytes a step
          commit(bar(kBODone));
          if (!F8) commit(bar(kBVEmpty) + 8 * vr.at);
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
    find_items<G_>(a, cta, sQ, qscale);
  } else if (warp < 4 + G_::kSoft) {
    // ======================= softmax =======================
    const int quarter = warp & 3, grp = (warp - 4) >> 2;
    const int tg = quarter * 32 + lane;  // thread of the group: this lane's key in a tile
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    // p may pass 2^0 (e4m3: 2^kUp, times which p is kept) by 2^kTau before a
    // row's reference moves.  bf16 parts keep their precision over the whole
    // exponent range, so the first reference is 0 unless the row's largest
    // score lies beyond +-kTau.  f16 ends at 2^16 and below 2^-25: half of its
    // range on either side of 2^kUp leaves 33 powers of two downwards, and few
    // rows whose reference has to move again.
    constexpr float kTau = F8 ? 7.75f : 16.f;
    constexpr float kUp = F8 ? 8.f : 0.f;
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
    const uint32_t p_at = sP + swz<128>(tg, grp * NC / 8);
    if (tg < NC) refs[grp * NC + tg] = kUp;  // item 0's
    Ring ir, vr;                // (vr, wv: e4m3)
    typename std::conditional<F8, WidenV<G_>, NoWiden>::type wv(warp - 4, lane);
    int g = 0;
    bool ok = sync();
    for (int j = 0; ok; ++j) {
      Item it;
      ok = cta.take(ir, it);
      if (!ok || it.nt == 0) break;
      const int nt = it.nt, rows = it.q_s * G, ctx = it.ctx;
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
        if constexpr (F8) {
          ok = wait_bar(bar(kBVFull) + 8 * vr.at, vr.pass);
          if (!ok) break;
          wv.load(sV + vr.at * G_::kTileB);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBVEmpty) + 8 * vr.at);
          vr.next(NV);
        }
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
            if constexpr (S) {
              const int from = (jj + 1) * G - ra;  // rows from here on see it
              see = from >= 32 ? 0u : from <= 0 ? 0xffffffffu : 0xffffffffu << from;
            } else {
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
          }
        }
        if constexpr (F8) {
          if (masked && wv.clean(kt, ctx, it.k1, bad)) poison[j % 3] = j + 1;
          // the widened tile before the last has been read: its P V came before this tile's S
          wv.store(sW + (g & 1) * G_::kWideB);
        } else if (masked) {
          if (!wait_bar(bar(kBVFull + g % NV), (g / NV) & 1)) { ok = false; break; }
          if (clean_v<G_>(sV + (g % NV) * G_::kTileB, warp - 4, G_::kSoft, lane, kt, ctx, it.k1, bad)) poison[j % 3] = j + 1;
        }
        // y = score in base 2 less the row's reference, plus kUp
        float y[NC];
        uint32_t hi[NC / 2], lo[NC / 2];  // (lo: bf16)
        if (S && F8 && t == 0 && !masked) {
          // the first reference: the row's largest score in the tile.  (Not that among some
          // keys, as below: a row behind a shared prefix has the same bits wherever its group puts it.)
          uint32_t u[NC];
          tm_ld(ts, u);
          wait_ld();
          float mine = 0.f;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float m = redux_max(__uint_as_float(u[c]) * qs[c]);  // NaN is passed over
            mine = lane == c ? m : mine;
          }
          if (lane < NC) xh[quarter * NC + lane] = mine;
          if (!sync()) { ok = false; break; }
          bool none = false;
          if (lane < NC) {  // the same in the group's four warps
            const float top = fmaxf(fmaxf(xh[lane], xh[NC + lane]), fmaxf(xh[2 * NC + lane], xh[3 * NC + lane]));
            none = top == -INFINITY;
            rh[lane] = none ? kUp : kUp - top;
          }
          vmask = __ballot_sync(0xffffffffu, none);
          // every warp has read the scores before the careful path puts others in their place
          if (vmask != 0 && !sync()) { ok = false; break; }
          __syncwarp();
        } else if (F8 && t == 0 && !masked) {
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
          if (lane < NC / 4) rh[quarter * (NC / 4) + lane] = none ? kUp : kUp - m;
          const uint32_t unset = __ballot_sync(0xffffffffu, none) << (quarter * (NC / 4));
          if (lane == 0) unset4[grp * 4 + quarter] = unset;
          __syncwarp();
          cast(unset != 0);
          bool some;
          if (!count(some)) { ok = false; break; }
          if (some) vmask = unset4[grp * 4] | unset4[grp * 4 + 1] | unset4[grp * 4 + 2] | unset4[grp * 4 + 3];
        }
        // first try: all of the tile's work against the references there are;
        // careful: new references; last: the work against those.  (A tile that a mask
        // cuts is tried like any other once the rows have references: what they do not
        // see is -infinity.)
        enum : int { kTry, kCareful, kLast };
        for (int mode = (masked && t == 0) || vmask ? kCareful : kTry;;) {
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
            // P = 2^y, row = key: one f16, or bf16 hi in columns 0 .. N - 1 and lo in N ..
            // 2 N - 1 (while the vote is out: if it asks for care, all of this is done again)
#pragma unroll
            for (int c = 0; c < NC; c += 2) {
              const float p0 = ex2(y[c]), p1 = ex2(y[c + 1]);
              y[c] = p0;
              y[c + 1] = p1;
              if constexpr (F8) {
                hi[c / 2] = pack_f16(p0, p1);
              } else {
                const unsigned long long pp = pk2(p0, p1);
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
              if (!none && (F8 || fabsf(top) > kTau)) nref = old + kUp - top;
            } else if (top > kTau + kUp) {
              nref = old + kUp - top;
              alpha = ex2(kUp - top);
              moved = true;
            }
          }
          vmask = __ballot_sync(0xffffffffu, none);
          const bool any = __any_sync(0xffffffffu, moved);
          // every warp has read the references
          if (!sync()) { ok = false; break; }
          if (quarter == 0 && lane < NC) rh[lane] = nref;
          // the same in the group's four warps.  In an item's first tile there is
          // nothing to rescale: the sums are zero and the first P V overwrites O,
          // which until kBOFree belongs to the item before the last
          if (any && t > 0) {
#pragma unroll
            for (int c = 0; c < NC; c += 2)
              l2[c / 2] = mul2(l2[c / 2], pk2(__shfl_sync(0xffffffffu, alpha, c), __shfl_sync(0xffffffffu, alpha, c + 1)));
            // every P V so far has run after this wait
            if (!wait_bar(bar(kBODone), (g - 1) & 1)) { ok = false; break; }
            fence_after();
            const uint32_t to = tmem + G_::kColO + (j & 1) * G_::kOCols + lane_off + grp * NC;
#pragma unroll 1
            for (int b = 0; b < NC; b += 8) {
              uint32_t o[8], o2[8];  // (o2: bf16)
              tm_ld(to + b, o);
              if (!F8) tm_ld(to + N + b, o2);
              wait_ld();
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float f = __shfl_sync(0xffffffffu, alpha, b + c);
                o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                if (!F8) o2[c] = __float_as_uint(__uint_as_float(o2[c]) * f);
              }
              tm_st(to + b, o);
              if (!F8) tm_st(to + N + b, o2);
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
          const uint32_t at = p_at + (g & 1) * G_::kPB, at_lo = G_::kPRow == 256 ? at + kKeys * 128 : at ^ (2 * N);
#pragma unroll
          for (int q = 0; q < NC / 8; ++q) {
            st_s128(at ^ (q << 4), hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
            if (!F8) st_s128(at_lo ^ (q << 4), lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
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
    constexpr int kCols = 16;            // rows at a time
    constexpr int kOff = (N + 31) / 32;  // row offsets held by a lane
    Ring ir;
    bool ok = true;
    for (int j = 0;; ++j) {
      Item it;
      ok = cta.take(ir, it);
      if (!ok || it.nt == 0) break;
      ok = wait_bar(bar(kBLFull + (j & 1)), (j >> 1) & 1);
      if (!ok) break;
      // read before kBLEmpty hands the item on: the softmax warps may then run as
      // far as item j + 3, which takes this flag's place
      const bool spoilt = poison[j % 3] == j + 1;
      const int rows = it.q_s * G;
      const Part part = part_of<S>(a, it);
      // lane c (and c + 32): 1 / (row c's sum), and its log2-sum-exp2 for the join
      float inv[kOff];
#pragma unroll
      for (int k = 0; k < kOff; ++k) {
        const int c = (lane + 32 * k) & (N - 1), r = it.r0 + c;
        const float* q = sums + (j & 1) * 256 + c;
        const float l = (q[0] + q[64]) + (q[128] + q[192]);
        inv[k] = l == 0.f ? 0.f : p.v_scale / l;
        if (warp == 4 + G_::kSoft && part.split && r < rows && lane + 32 * k < N) {
          const int i = quot(r, a.by_g);
          a.part_lse[(part.at + i * part.step) * p.Hq + it.h * G + r - i * G] =
              l == 0.f ? -INFINITY : __log2f(l) - lref[(j & 1) * 64 + (c / NC) * NC + c % NC];  // reference + log2(sum) - kUp
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBLEmpty + (j & 1)));
      ok = wait_bar(bar(kBOFull + (j & 1)), (j >> 1) & 1);
      if (!ok) break;
      fence_after();
      const bool split = part.split, wide = split || !a.out_bf16;  // fp32 elements
      // lane c (and c + 32): where row c's element 0 goes, in bytes from `to_base`; -1: no row
      const int esz = wide ? 4 : 2;
      const int64_t node = split ? part.step * p.Hq * D : p.o_st, head = split ? D : p.o_sh;
      char* const to_base = (split ? reinterpret_cast<char*>(a.part_o + part.at * p.Hq * D)
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
        if (!F8) tm_ld(to + N, o2);
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
          const float x = __uint_as_float(o[c]) + (F8 ? 0.f : __uint_as_float(o2[c]));
          v[c] = sc == 0.f ? 0.f : x * sc;
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
      if (spoilt && (D == 128 || d < D)) add_poison<D, N, F8, S>(a, it, d);
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
  end_phase<S>(a);
}

}  // namespace
}  // namespace pkv
