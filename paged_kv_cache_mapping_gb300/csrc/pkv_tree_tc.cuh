// pkv_tree_tc.cuh -- what the tensor-core kernels of tree attention share: the
// cut of a call into items, the barriers of a CTA, the warps that find items and
// bring their query rows, the warps that copy K and V tiles, and the PTX they
// are made of.
#pragma once
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "pkv_kernels.h"

namespace pkv {

constexpr int kKeys = 128;  // keys per tile (M of S^T, K of P V)
constexpr int kItemSlots = 6;
constexpr int kInfoSlots = 8;

// ---------------------------------------------------------------- chunking
// Keys per chunk, from the sequence's own length and node count and from how
// many (sequence, KV head, row tile) units the call has: few units are cut
// finely so that every SM has work, many are cut coarsely, since each chunk
// costs its rows' partials (512 bytes per row and head, written and read) and
// an item's start and end.  A sequence is cut into equal chunks of at most
// `least` keys, but into no more than `most`, and no more than
// kTreePartRows / q_s, so that it has at most that many partial rows per head.
// Measured, us, `least` 256 / 512 / 1024 / 2048 / 4096, 8 KV heads of 4 query heads,
// D 128, contexts uniform up to the number given:
//   units  8: 8 nodes, 2,100 keys  12.0 / 12.7 / 14.7 / 20.2 / 30
//         16: 4 nodes,  8,192      18.3 / 17.9 / 16.0 / 19.8 / 31; 8 nodes, 4,096  14.9 / 13.3 / 15.0 / 20.7 / 31
//         64: 8 nodes,  4,096      24.7 / 22.6 / 25.3 / 25.8 / 37; 64 nodes (wide tiles), 8,192  55 / 56 / 49 / 53 / 54
//        128: 16 nodes, 16,384, e4m3  134 / 134 / 128 / 118 / 124; 64 nodes, 8,192  73 / 70 / 63 / 71 / 80
//        192: 8 nodes,  4,096      56 / 51 / 49 / 60 / 64; 64 nodes, 8,192  104 / 98 / 88 / 93 / 91
//        240, 256: 64 nodes, 8,192  128 / 122 / 112 / 112 / 118 and 140 / 133 / 124 / 114 / 132
//        256: 8 nodes,  4,096      66 / 65 / 61 / 63 / 67; 16 nodes, 8,192  140 / 130 / 125 / 120 / 122
//        512: 8 nodes,  4,096      123 / 120 / 113 / 114 / 113; 64 nodes, 8,192  267 / 257 / 240 / 219 / 231
// `most` with 64 units of 32K to 131K keys: 16 303, 19 (8 items per SM) 288, 24 319,
// 48 337.  (The SMs are counted here, not asked for: a workspace's size is known
// without a device.)
constexpr int kTreeMaxChunks = 64;
constexpr int kTreePartRows = 1024;
constexpr int kTreeItems = 8 * 152;
struct Chunking {
  int32_t least, most;
};
inline Chunking tree_chunking(int64_t units) {
  Chunking c;
  c.least = units >= 256 ? 2048 : units >= 16 ? 1024 : 256;
  const int64_t m = kTreeItems / (units < 1 ? 1 : units);
  c.most = static_cast<int32_t>(m < 8 ? 8 : m > kTreeMaxChunks ? kTreeMaxChunks : m);
  return c;
}

__host__ __device__ inline int tree_chunk(int n, int q_s, Chunking k) {
  const int rows = kTreePartRows / q_s;
  const int most = rows < 1 ? 1 : rows < k.most ? rows : k.most;
  const int tiles = (n - 1) / kKeys + 1, least = k.least / kKeys;
  const int chunks = tiles <= least ? 1 : tiles <= (int64_t)least * most ? (tiles - 1) / least + 1 : most;
  return ((tiles - 1) / chunks + 1) * kKeys;  // n < 2^31 - 128
}

struct alignas(16) Item {
  int s, h, r0;         // sequence, KV head, first row of the tile
  int t0, q_s, n;       // first packed row, nodes, keys
  int k0, k1;           // keys of the chunk
  int c, nchunks;       // its index, chunks of the sequence
  int nt, pad;          // key tiles (0: no more items)
};

constexpr int kMiscBytes = 6656;  // a CTA's control area
// barriers (each kernel's own ones stand with it) and shared places of a CTA's
// control area
enum : int {
  kBKFull = 0, kBKEmpty = 6, kBVFull = 12, kBVEmpty = 18, kBSFull = 24, kBPFull = 26 /* 2 */, kBOFull = 28,
  kBOFree = 30, kBQFull = 32, kBQEmpty = 34, kBQsFull = 36, kBLFull = 40, kBLEmpty = 42, kBItemFull = 44,
  kBItemEmpty = 50, kBODone = 56, kBDrain = 57, kBGroup = 58 /* 4 */, kSTmem = 62, kSAbort = 63, kSPoison = 64 /* [3] ints: 64, 65 */,
  kOffItems = 528, kOffInfo = 816, kOffOwn = 944,
};
static_assert(kOffItems + kItemSlots * (int)sizeof(Item) <= kOffInfo, "item ring");

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo, int atom) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFF) << 32) | (1ull << 46) | ((uint64_t)(atom == 128 ? 2 : 4) << 61);
}

// instruction descriptor: fp32 accumulator, A and B bf16 (f8: e4m3, or in kind::f16
// f16, which have the same code), M 128, N n
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
// which may suspend the warp for up to 20 us (5 s in all).  The code is kept
// short, here and below: sixteen and more warps in six roles share the SM's
// instruction cache, and while the roles' code did not fit (105 to 166 KB in
// all, 42 % of its requests missed) it set the pace, not the pipes.
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

struct TcArgs {
  TreeParams p;
  FastDiv by_g, by_bs;
  int32_t rows_per_seq;  // partial rows of a sequence
  Chunking chunking;
  int32_t box;           // slots per TMA box: 16, 8 or 4, so that a box lies in one block; 0: gather4
  int32_t out_bf16;
  float* part_o;         // [B * rows_per_seq, Hq, D] normalised chunk outputs
  float* part_lse;       // [B * rows_per_seq, Hq]
};

// What every warp of a CTA needs: its barriers and its items.
struct Cta {
  uint32_t b0;
  volatile int* abort_flag;
  Item* items;
  uint32_t* info;  // [kInfoSlots][4]: a tile's keys without a page
  int lane;
  __device__ __forceinline__ uint32_t bar(int i) const { return b0 + 8 * i; }
  __device__ __forceinline__ bool aborted() const { return __any_sync(0xffffffffu, *abort_flag != 0); }
  // the next item, as every warp but the finder takes it
  __device__ __forceinline__ bool take(Ring& r, Item& it) const {
    if (!wait_bar(bar(kBItemFull) + 8 * r.at, r.pass)) return false;
    const int4* q = reinterpret_cast<const int4*>(items + r.at);
    *reinterpret_cast<int4*>(&it) = q[0];
    *(reinterpret_cast<int4*>(&it) + 1) = q[1];
    *(reinterpret_cast<int4*>(&it) + 2) = q[2];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBItemEmpty) + 8 * r.at);
    r.next(kItemSlots);
    return !aborted();
  }
};

// ---------------------------------------------------------------- K tiles, V tiles
// One warp copies the K tiles, one the V tiles: pages, slots, TMA.
template <class G_>
__device__ __forceinline__ void copy_tiles(const TcArgs& a, const Cta& c, bool is_v, uint32_t tiles, const CUtensorMap* map) {
  constexpr int NK = G_::kNK, NV = G_::kNV, AT = G_::kAtomB, N = G_::kN;
  const TreeParams& p = a.p;
  const int lane = c.lane, G = p.G, Hkv = p.Hkv;
  auto bar = [&](int i) -> uint32_t { return c.bar(i); };
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
      // eight at a time: with a shuffle before every copy each took 150 clocks (by
      // twos, fours and eights 123, 104 and 100 us for 7 sequences of up to 40,000
      // keys in pages of one slot)
#pragma unroll 1
      for (int b = 0; b < 32; b += 8) {
        int q[8][4];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int x = 0; x < 4; ++x) q[k][x] = __shfl_sync(0xffffffffu, r[x], b + k);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int u = 0; u < G_::kSub; ++u)
              tma_gather4(dst + u * kKeys * AT + (b + k) * 4 * AT, map, u * (AT / G_::kEs), q[k], full, pol);
        }
        __syncwarp();
      }
    }
  };
  // K and V are read once where one tile of rows holds them all
  const uint64_t pol_once = l2_evict_first_policy(), pol_keep = l2_normal_policy();

  const uint32_t full = bar(is_v ? kBVFull : kBKFull), empty = bar(is_v ? kBVEmpty : kBKEmpty);
  const int ns = is_v ? NV : NK;
  Ring ir, r;
  int g = 0;
  bool ok = true;
  for (;;) {
    Item it;
    ok = c.take(ir, it);
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
        uint32_t* w = c.info + (g % kInfoSlots) * 4;
        if (lane < 4) w[lane] = 0;
        __syncwarp();
        if (__any_sync(0xffffffffu, bad != 0)) {
          if (bad) {
            atomicOr(p.err, kErrBlockRange);
            if (!bx) {
              atomicOr(w + key_of / 32, bad << (key_of & 31));
            } else if (lane < n_box) {
              atomicOr(w + key_of / 32, ((1u << bx) - 1u) << (key_of & 31));
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
  if (!ok) *c.abort_flag = 1;
  if (c.aborted())  // let the copies issued so far land before the CTA exits
    for (int k = 0; k < ns && k < g; ++k) {
      if (r.at-- == 0) {
        r.at = ns - 1;
        r.pass ^= 1;
      }
      wait_bar(full + 8 * r.at, r.pass);
    }
}

// ---------------------------------------------------------------- items, query rows
// One warp finds the CTA's items, publishes them and brings their query rows.
// qscale: e4m3: [4][64], the rows' scales.
template <class G_>
__device__ __forceinline__ void find_items(const TcArgs& a, const Cta& cta, uint32_t sQ, float* qscale) {
  constexpr int D = G_::kD, N = G_::kN, AT = G_::kAtomB;
  constexpr bool F8 = G_::kF8;
  const TreeParams& p = a.p;
  const int lane = cta.lane, G = p.G, Hkv = p.Hkv;
  auto bar = [&](int i) -> uint32_t { return cta.bar(i); };
  int gb = 0;                        // the group of sequences gb .. gb + 31 held by the lanes
  int c0 = 0, q_s = 0, n = 0, chunk = 1, nchunks = 0, rts = 0;
  // items: this sequence's, prefix in the group, in it; before it.  A sequence has
  // at most Hq max(1024, q_s) / 16 + 64 Hkv of them, 2^27 since T Hq <= 2^30, and so
  // a group's fit 32 bits, whatever the lengths are
  int cnt = 0;
  uint32_t incl = 0, total = 0;
  int64_t base = 0;
  constexpr int kLanes = D / 8;          // lanes of a row (8 bf16 elements each)
  constexpr int kPer = 32 / kLanes;      // rows per step
  constexpr int kStepsQ = N / kPer;
  const int ch = lane % kLanes, rr = lane / kLanes;
  Ring ir;
  bool ok = true;
  gb = -32;
  int64_t x = blockIdx.x;
  for (int j = 0;; ++j, x += gridDim.x) {
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
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      total = __shfl_sync(0xffffffffu, incl, 31);
    }
    Item it{};
    if (x - base < total) {
      const uint32_t at = static_cast<uint32_t>(x - base);
      const int o = __ffs(__ballot_sync(0xffffffffu, incl > at)) - 1;
      const int y = static_cast<int>(at - __shfl_sync(0xffffffffu, incl - cnt, o));
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
    ok = wait_bar(bar(kBItemEmpty) + 8 * ir.at, ir.pass ^ 1) && !cta.aborted();
    if (!ok) break;
    if (lane == 0) {
      cta.items[ir.at] = it;
      mbar_arrive(bar(kBItemFull) + 8 * ir.at);
    }
    __syncwarp();
    ir.next(kItemSlots);
    if (it.nt == 0) break;
    // its query rows; the buffer is free once the scores of the item that
    // used it last are there
    const int qb = G_::qbuf(j), rows = it.q_s * G;
    const uint32_t dst = sQ + qb * G_::kQB;
    // lane c (and c + 32) finds row c; 0: past the last
    unsigned long long row[(N + 31) / 32];
#pragma unroll
    for (int k = 0; k < (N + 31) / 32; ++k) {
      const int r = it.r0 + lane + 32 * k, i = quot(r, a.by_g);
      const __nv_bfloat16* at = static_cast<const __nv_bfloat16*>(p.q) + (it.t0 + i) * p.q_st + (it.h * G + r - i * G) * p.q_sh;
      row[k] = r < rows ? reinterpret_cast<unsigned long long>(at) : 0;
    }
    ok = wait_bar(bar(kBQEmpty + qb), G_::qpass(j) ^ 1);
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
  if (!ok) *cta.abort_flag = 1;
}

// V rows that must not reach a row that does not see them: zeroes what is past
// the sequence or has no page, and what is not finite among the drafted rows
// (the rows that see those get it at the end).  Each of a tile's `warps` warps
// takes its share of the rows; true: this lane found a value that is not finite.
template <class G_>
__device__ __forceinline__ bool clean_v(uint32_t tile, int w_of, int warps, int lane, int kt, int ctx, int k1, const uint4& bad) {
  constexpr int AT = G_::kAtomB;
  constexpr bool F8 = G_::kF8;
  constexpr int kLn = G_::kRowB / 16, kRs = 32 / kLn;
  const int ch = lane % kLn, rr = lane / kLn;
  bool found = false;
  // the context's rows stay as they are, unless pages are out of range
  const uint32_t bm = w_of * (kKeys / warps) < 64 ? w_of * (kKeys / warps) < 32 ? bad.x : bad.y
                                                  : w_of * (kKeys / warps) < 96 ? bad.z : bad.w;  // this warp's rows lie in one word
  const int first = w_of * (kKeys / warps), from = bm ? 0 : max(0, ctx - kt - first) / kRs * kRs;
#pragma unroll 2
  for (int b = from; b < kKeys / warps; b += kRs) {
    const int kk = first + b + rr, ky = kt + kk;
    const bool gone = ky >= k1 || ((bm >> (kk & 31)) & 1u);
    if (!gone && ky < ctx) continue;
    const uint32_t at = tile + (ch * 16 / AT) * kKeys * AT + swz<AT>(kk, ch % (AT / 16));
    uint32_t w[4] = {0, 0, 0, 0};
    bool hit = gone;
    if (!gone) {
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
      // an exponent (e4m3: all but the sign) of ones carries into the sign's place
      constexpr uint32_t kExp = F8 ? 0x7f7f7f7fu : 0x7f807f80u, kOne = F8 ? 0x01010101u : 0x00800080u;
      constexpr uint32_t kTop = F8 ? 0x80808080u : 0x80008000u, kAll = F8 ? 0xffu : 0xffffu;
      constexpr int kBits = F8 ? 8 : 16;
      uint32_t any = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) any |= ((w[e] & kExp) + kOne) & kTop;
      if (any) {
        found = hit = true;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll 1
          for (uint32_t t = ((w[e] & kExp) + kOne) & kTop; t; t &= t - 1) w[e] &= ~(kAll << (__ffs(t) - kBits));
      }
    }
    if (hit) st_s128(at, w[0], w[1], w[2], w[3]);
  }
  return found;
}

// ---------------------------------------------------------------- host
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_fn() {
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
inline bool encode_cache(CUtensorMap* m, const void* base, const TreeParams& p, bool f8, int atom_bytes, int box) {
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

// Launches a kernel's persistent CTAs over at most max_items items.
template <class G_, class Kern>
cudaError_t launch_items(Kern kern, TcArgs a, int64_t max_items, int num_sms, cudaStream_t st) {
  a.box = a.p.bs % 16 == 0 ? 16 : a.p.bs % 8 == 0 ? 8 : a.p.bs % 4 == 0 ? 4 : 0;
  CUtensorMap mk, mv;
  if (!encode_cache(&mk, a.p.k_cache, a.p, G_::kF8, G_::kAtomB, a.box) || !encode_cache(&mv, a.p.v_cache, a.p, G_::kF8, G_::kAtomB, a.box))
    return cudaErrorInvalidValue;
  cudaError_t e = set_smem_attr(reinterpret_cast<const void*>(kern), G_::kSmem);
  if (e != cudaSuccess) return e;
  return launch_ex(kern, dim3((unsigned)std::min<int64_t>(num_sms, max_items)), dim3(G_::kThreads), G_::kSmem, st, true, a, mk, mv);
}

// 128 rows a tile, bf16 caches (pkv_tree_wide.cu)
cudaError_t launch_tree_wide(const TcArgs& a, int64_t max_items, int num_sms, cudaStream_t st);

}  // namespace pkv
