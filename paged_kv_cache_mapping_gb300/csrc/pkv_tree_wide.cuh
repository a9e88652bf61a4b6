// pkv_tree_wide.cuh -- attention over bf16 caches for more than 64 query rows of a
// KV head that read the same keys, on the fifth-generation tensor cores: wide
// drafted trees, and requests that share a prefix.
//
// What it computes is what pkv_tree_narrow.cuh computes, over the same items; here a
// tile holds 128 query rows, enough to fill the MMA's M side, and the products
// stand the usual way round:
//     S = Q K^T     (M 128 rows, N 128 keys, K = D)
//     O += P V      (M 128 rows, N = D, K 128 keys; P as bf16 hi + lo)
// P stays in tensor memory, where it replaces S, and K and V tiles serve twice
// the rows that 64-row tiles served.
//
// Softmax: two groups of four warps take the tiles in turn, group g & 1 tile g,
// and a thread owns a row of its tile: its largest score and its share of the
// sum need no other thread.  The reference of a row is shared by the groups: a
// group settles it for tile g (it moves when the tile's largest score passes it
// by 2^kTau; then the row of O is rescaled, which is rare) after the other has
// settled it for tile g - 1, half a tile's time earlier.  So there is one O, two
// of them fit tensor memory, and an item's O is written out while the next item
// runs.  (An O for each group, nothing shared, took all of it: every item's end
// cost 4,900 clocks.)  S is read twice, for the largest score and for P, since
// 128 scores do not fit a thread's registers beside the rest.
//
// Not kept: shared K and V tiles in a CTA pair.  They took 107 us for the 16 trees
// below instead of 110, and gave up more wherever the row tiles are odd (65 nodes
// instead of 64: 139 us instead of 107) or uneven (29 instead of 26 us for the 23
// trees, at the time).
//
// Bound: the K and V tiles, of which each row tile reads all (64 KB for 12.6
// MFLOP), then the tensor cores (55 % active; a tile takes them about 1,540 clocks
// of the 2,300 that it takes in all).  Probes of the 16 trees below, 110 us whole:
// without the softmax 104, without the MMAs 97, without either 93; half of the
// MMAs 107; the softmax's loops rolled or unrolled 110.  The instruction cache
// (see poll()): code in one place instead of unrolled took 3,000 clocks off every
// item's start, but the halves of P V, whose descriptors want to be constants,
// stand twice (124 us in a loop, 116 so, at the time).
// Measured, with the join: 16 trees of 64 nodes times 4 heads (256 rows) over
// 1,024 to 8,192 keys, D 128: 109 us (73 GFLOP of visible pairs, 0.67 PFLOP/s);
// 23 uneven trees of up to 37 nodes times 5 heads, D 64, pages of 12 slots: 28 us.
//
// CTA: 16 warps: K, MMA, items and query rows, V, 2 x 4 of softmax, 4 that write.
#pragma once
#include "pkv_tree_tc.cuh"

namespace pkv {
namespace {

// kBPFull + group: P of a tile's keys 0 .. 63; kBPRest + group: of the rest
enum : int {
  kBPRest = kBGroup, kBMax = kOffOwn / 8 /* [2 groups][4 warps] */,
  kOffRef = kOffOwn + 64 /* [2][128] */, kOffStat = kOffRef + 1024 /* [2][2 groups][128] sum and reference */,
  kOffStage = 6144 /* [4 warps][32 rows][128 bytes] */, kWideMisc = kOffStage + 4 * 4096,
};
static_assert(kOffStat + 2 * 2 * 128 * 8 <= kOffStage, "shared memory");

template <int D, bool S>
struct Wide {
  static constexpr int kD = D, kN = 128;
  static constexpr bool kF8 = false, kShared = S;
  static constexpr int kEs = 2, kRowB = 2 * D, kAtomB = 128;
  static constexpr int kSub = kRowB / kAtomB;
  static constexpr int kTileB = kKeys * kRowB;
  static constexpr int kNK = D == 128 ? 2 : 4, kNV = kNK;
  static constexpr int kQB = kN * kRowB;
  static constexpr int kQBufs = 2;
  __device__ static int qbuf(int j) { return j & 1; }
  __device__ static uint32_t qpass(int j) { return (uint32_t)(j >> 1) & 1u; }
  static constexpr int kSoft = 8;  // softmax warps
  static constexpr int kThreads = 32 * (4 + kSoft + 4);
  static constexpr int kOffK = 0, kOffV = kNK * kTileB, kOffQ = kOffV + kNV * kTileB, kOffMisc = kOffQ + kQBufs * kQB;
  static constexpr int kSmem = kOffMisc + kWideMisc;
  static constexpr uint32_t kColO = 256;  // tensor memory: S and then P of each group's tile; then O, twice
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kColO + 2 * D <= 512, "tensor memory");
  static_assert(kNK + 2 <= kInfoSlots, "tile info ring");
};

// kSteps k steps of 16 keys with A in tensor memory: 8 columns for the hi part,
// and 8 for the lo part 16 columns on
template <int kSteps>
__device__ __forceinline__ void mma_p_steps(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
#pragma unroll
  for (int k = 0; k < kSteps; ++k)
#pragma unroll
    for (int part = 0; part < 2; ++part)
      asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                   "r"(a + (k >> 1) * 32 + (k & 1) * 8 + part * 16), "l"(b + k * 128), "r"(id), "r"(k || part ? 1u : acc));
}

__device__ __forceinline__ void tm_st(uint32_t a, const uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(a),
      "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]),
      "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]));
}

// A drafted key's V value is not finite: the softmax warps took it out of the
// product, and here it goes to the row of this thread if that sees the key, on
// top of what its warp has just stored.
template <int D, bool S>
__device__ __noinline__ void add_poison_row(const TcArgs& a, const Item& it, int r) {
  const TreeParams& p = a.p;
  const Part part = part_of<S>(a, it);
  const int ctx = it.ctx, i = r / p.G, hq = it.h * p.G + r - i * p.G;
  for (int k = max(ctx, it.k0); k < it.k1; ++k) {
    const int lb = k / p.bs, jj = k - ctx;
    const int32_t blk = __ldg(p.bt + (int64_t)it.s * p.bt_stride + lb);
    if ((uint32_t)blk >= (uint64_t)p.num_blocks) continue;
    if (!sees<S>(p, it, i, jj)) continue;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v_cache) + (((int64_t)blk * p.bs + (k - lb * p.bs)) * p.Hkv + it.h) * D;
    for (int d = 0; d < D; ++d) {
      const float x = __bfloat162float(v[d]);
      if (fabsf(x) < INFINITY) continue;
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

template <int D, bool S>
__global__ void __launch_bounds__(Wide<D, S>::kThreads, 1)
    tree_wide_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v) {
  using G_ = Wide<D, S>;
  constexpr int NK = G_::kNK, NV = G_::kNV, AT = G_::kAtomB;
  const TreeParams& p = a.p;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* misc = smem + G_::kOffMisc;
  const uint32_t s0 = smem_u32(smem), b0 = smem_u32(misc);
  auto bar = [&](int i) -> uint32_t { return b0 + 8 * i; };
  const uint32_t sK = s0 + G_::kOffK, sV = s0 + G_::kOffV, sQ = s0 + G_::kOffQ;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 8 * kSAbort);
  volatile int* poison = reinterpret_cast<volatile int*>(misc + 8 * kSPoison);  // [3]: item + 1
  uint32_t* tslot = reinterpret_cast<uint32_t*>(misc + 8 * kSTmem);
  uint32_t* info = reinterpret_cast<uint32_t*>(misc + kOffInfo);
  float* refs = reinterpret_cast<float*>(misc + kOffRef);  // [2][128]: the rows' references
  float2* stat = reinterpret_cast<float2*>(misc + kOffStat);
  // as in the narrow kernel: the warp index, and so a role, is the warp's
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int G = p.G;
  const Cta cta{b0, abort_flag, reinterpret_cast<Item*>(misc + kOffItems), info, lane};

  if (s0 & 1023) {  // the swizzled tiles need their base on 1024 bytes
    if (threadIdx.x == 0) atomicOr(p.err, kErrWaitTimeout);
    if (S) grid_dep_wait();
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(bar(kBKFull + i), 1);
      mbar_init(bar(kBKEmpty + i), 1);
      mbar_init(bar(kBVFull + i), 1);
      mbar_init(bar(kBVEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBSFull + i), 2);
      mbar_init(bar(kBPFull + i), 4);
      mbar_init(bar(kBPRest + i), 4);
      mbar_init(bar(kBOFull + i), 1);
      mbar_init(bar(kBOFree + i), 4);
      mbar_init(bar(kBQFull + i), 1);
      mbar_init(bar(kBQEmpty + i), 1);
      mbar_init(bar(kBLFull + i), G_::kSoft);
      mbar_init(bar(kBLEmpty + i), 4);
    }
    for (int i = 0; i < 8; ++i) mbar_init(bar(kBMax + i), 1);
    mbar_init(bar(kBODone), 1);
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(bar(kBItemFull + i), 1);
      mbar_init(bar(kBItemEmpty + i), 3 + G_::kSoft + 4);  // every warp but the finder
    }
    mbar_init(bar(kBDrain), 1);
    *abort_flag = 0;
    for (int i = 0; i < 3; ++i) poison[i] = 0;
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
  // trees: no launch_dependents(): as in the narrow kernel, a join that is pending while
  // this runs costs (14 of the trees below 121 us instead of 114, 16 of them 111
  // instead of 110)

  if (warp == 0 || warp == 3) {
    copy_tiles<G_>(a, cta, warp == 3, warp == 3 ? sV : sK, warp == 3 ? &tm_v : &tm_k);
  } else if (warp == 1) {
    // ======================= MMA =======================
    constexpr uint32_t kIdS = idesc(128, false, false, false), kIdO = idesc(D, false, false, true);
    // The tensor core takes the MMAs of a tile about as fast as they are issued
    // and holds a few: what has to be waited for is waited for behind MMAs that
    // are still to run, so that S of tile g + 2 follows P V of tile g at once.
    Ring ir, kr, vr;
    int js = -1, ns = 0, is = 0, gs = 0;  // S that goes next: item, its tiles, tile, tile of all
    int n1 = 0, n2 = 0;                   // tiles of the items after the one whose P V runs (S may be two items on)
    int j = 0, nt = 0;                    // P V: item, its tiles
    // finds the tile whose S goes next; its K tile remains to be waited for
    auto find_s = [&](bool& more) -> bool {
      if (is == ns) {
        Item it;
        if (!cta.take(ir, it)) return false;
        ++js;
        is = 0;
        ns = it.nt;
        (js == j ? nt : js == j + 1 ? n1 : n2) = ns;
        more = ns > 0;
        if (!more) return true;
        if (!wait_bar(bar(kBQFull + G_::qbuf(js)), G_::qpass(js))) return false;
      }
      return true;
    };
    // S replaces the P of its group's last tile, whose P V was issued earlier
    auto issue_s = [&]() {
      fence_after();
      const uint64_t dk = sdesc(sK + kr.at * G_::kTileB, 16, 8 * AT, AT);
      const uint64_t dq = sdesc(sQ + G_::qbuf(js) * G_::kQB, 16, 8 * AT, AT);
      const int grp = gs & 1;
      if (elect_one()) {
#pragma unroll
        for (int u = 0; u < G_::kSub; ++u)
          mma_steps<false, 4, 2, 2>(tmem + grp * 128, dq + (uint32_t)(u * 128 * AT >> 4), dk + (uint32_t)(u * kKeys * AT >> 4),
                                    kIdS, u != 0);
        commit(bar(kBSFull + grp));
        commit(bar(kBKEmpty) + 8 * kr.at);
        if (is + 1 == ns) commit(bar(kBQEmpty + G_::qbuf(js)));
        // the second arrival hands on what the tile's producer wrote (info)
        mbar_arrive(bar(kBSFull + grp));
      }
      __syncwarp();
      kr.next(NK);
      ++is;
      ++gs;
    };
    bool more = true, ok = find_s(more) && (!more || wait_bar(bar(kBKFull) + 8 * kr.at, kr.pass));
    for (int g = -1, t = 0; ok && (nt > 0 || more); ++g) {
      if (more) issue_s();  // of tile g + 1
      const int ob = j & 1, grp = g & 1;
      // V: d contiguous, 8 keys = 8 AT bytes, sub-tiles of d kKeys AT apart
      const uint64_t dv = sdesc(sV + vr.at * G_::kTileB, G_::kSub > 1 ? kKeys * AT : 8 * AT, 8 * AT, AT);
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // the halves of P V; before them what they and the next S need
        if (h == 1 && more) ok = find_s(more);
        if (!ok) break;
        const bool k = lane == 3 && h == 1 && more, v = lane == 1, o = lane == 2 && t == 0;
        if (g < 0) {  // no tile yet: the next S alone
          if (h == 1 && more) ok = wait_bar(bar(kBKFull) + 8 * kr.at, kr.pass);
          continue;
        }
        ok = wait_bar(k ? bar(kBKFull) + 8 * kr.at : v ? bar(kBVFull) + 8 * vr.at : o ? bar(kBOFree + ob) : bar((h ? kBPRest : kBPFull) + grp),
                      k ? kr.pass : v ? vr.pass : o ? ((j >> 1) & 1) ^ 1 : (g >> 1) & 1);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          mma_p_steps<4>(tmem + G_::kColO + ob * D, tmem + grp * 128 + h * 64, dv + h * (4 * 128), kIdO, t > 0 || h > 0);
          if (h == 1) {
            commit(bar(kBODone));
            commit(bar(kBVEmpty) + 8 * vr.at);
            if (t + 1 == nt) commit(bar(kBOFull + ob));
          }
        }
        __syncwarp();
      }
      if (!ok || g < 0) continue;
      vr.next(NV);
      if (++t == nt) {
        t = 0;
        ++j;
        nt = n1;
        n1 = n2;
        n2 = 0;
      }
    }
    if (!ok) *abort_flag = 1;
    // every MMA issued so far is finished before TMEM is freed
    if (elect_one()) commit(bar(kBDrain));
    __syncwarp();
    wait_bar(bar(kBDrain), 0);
  } else if (warp == 2) {
    find_items<G_>(a, cta, sQ, nullptr);
  } else if (warp < 4 + G_::kSoft) {
    // ======================= softmax: lane = row =======================
    const int quarter = warp & 3, grp = (warp - 4) >> 2, row = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    const uint32_t ts = tmem + grp * 128 + lane_off;
    // p may pass 1 by 2^kTau before a row's reference moves; bf16 parts keep
    // their precision over the whole exponent range
    constexpr float kTau = 16.f;
    const unsigned long long scale2 = pk2(p.qk_scale_log2, p.qk_scale_log2);
    Ring ir;
    int g = 0;  // first tile of the item
    bool ok = true;
    for (int j = 0;; ++j) {
      Item it;
      ok = cta.take(ir, it);
      if (!ok || it.nt == 0) break;
      const int nt = it.nt, ctx = it.ctx, r = it.r0 + row;
      // the row's reference as this group used it last; -infinity: none yet
      float ref = -INFINITY;
      float* const shared_ref = refs + (j & 1) * 128 + row;
      unsigned long long l2 = 0ull;
      for (int t = (g ^ grp) & 1; t < nt; t += 2) {
        const int gg = g + t;
        const int kt = it.k0 + t * kKeys, jj = kt - ctx;  // first key of the tile, and its place among the drafted
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};  // keys of the tile that this row sees
        if (jj > -kKeys) {
          const int i = quot(r, a.by_g);
          uint32_t w[5];
          if constexpr (!S) {
            const int words = i < it.q_s ? (it.q_s + 31) >> 5 : 0;
            const int32_t* m = p.mask + (int64_t)(it.t0 + i) * p.mask_stride;
#pragma unroll
            for (int c = 0; c < 5; ++c) {
              const int at = (jj >> 5) + c;
              w[c] = at < 0 ? ~0u : at < words ? static_cast<uint32_t>(__ldg(m + at)) : 0u;
            }
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // without masks row i sees the keys before ctx + i
            const int left = (S ? min(it.k1, ctx + min(i, it.n - ctx)) : it.k1) - (kt + 32 * c);
            const uint32_t in = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1u : 0u;
            if constexpr (S)
              see[c] = in;
            else
              see[c] = __funnelshift_r(w[c], w[c + 1], jj & 31) & in;
          }
        }
        ok = wait_bar(bar(kBSFull + grp), (gg >> 1) & 1);
        if (!ok) break;
        fence_after();
        const uint4 bad = *reinterpret_cast<const uint4*>(info + (gg % kInfoSlots) * 4);
        if (jj > -kKeys || (bad.x | bad.y | bad.z | bad.w) != 0) {
          // scores that this row does not see become -inf, in place
          see[0] &= ~bad.x;
          see[1] &= ~bad.y;
          see[2] &= ~bad.z;
          see[3] &= ~bad.w;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            const uint32_t w = (c < 4 ? c < 2 ? see[0] : see[1] : c < 6 ? see[2] : see[3]) >> (c & 1) * 16;
            uint32_t u[16];
            tm_ld(ts + 16 * c, u);
            wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = (w >> e) & 1u ? u[e] : 0xff800000u;
            tm_st(ts + 16 * c, u);
          }
          wait_st();
          const int vs = gg % NV;
          if (!wait_bar(bar(kBVFull + vs), (gg / NV) & 1)) { ok = false; break; }
          if (clean_v<G_>(sV + vs * G_::kTileB, quarter, 4, lane, kt, ctx, it.k1, bad)) poison[j % 3] = j + 1;
          fence_proxy_async_smem();
        }
        uint32_t u[2][32];
        float top = -INFINITY;
        tm_ld(ts, u[0]);
        // (loops of two chunks: the code of all roles shares the instruction cache)
#pragma unroll 1
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            wait_ld();
            tm_ld(ts + (2 * h + c + 1) % 4 * 32, u[c ^ 1]);  // the last: the first again, for P
#pragma unroll
            for (int e = 0; e < 32; e += 2) top = fmax3(top, __uint_as_float(u[c][e]), __uint_as_float(u[c][e + 1]));  // NaN is passed over
          }
        top *= p.qk_scale_log2;
        // the other group has settled the tile before this one
        if (gg > 0 && !wait_bar(bar(kBMax + (grp ^ 1) * 4 + quarter), ((gg - 1) >> 1) & 1)) { ok = false; break; }
        const float old = t == 0 ? -INFINITY : *shared_ref;
        const bool moved = old != -INFINITY && top > old + kTau;
        const float now = old == -INFINITY || moved ? top : old;
        *shared_ref = now;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBMax + grp * 4 + quarter));
        if (__any_sync(0xffffffffu, ref != now)) {  // this group's sum follows
          const float f = ref == -INFINITY || ref == now ? 1.f : ex2(ref - now);
          l2 = mul2(l2, pk2(f, f));
          ref = now;
        }
        if (__any_sync(0xffffffffu, moved)) {
          // and O, which every P V before this tile's has to have reached
          if (!wait_bar(bar(kBODone), (gg - 1) & 1)) { ok = false; break; }
          fence_after();
          wait_ld();
          const float alpha = moved ? ex2(old - now) : 1.f;
          const uint32_t to = tmem + G_::kColO + (j & 1) * D + lane_off;
#pragma unroll 1
          for (int b = 0; b < D; b += 16) {
            uint32_t o[16];
            tm_ld(to + b, o);
            wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
            tm_st(to + b, o);
          }
          wait_st();
        }
        const float neg = ref == -INFINITY ? 0.f : -ref;
        const unsigned long long neg2 = pk2(neg, neg);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t at = ts + h * 64 + c * 32;
            wait_ld();
            if (c == 0 || h == 0) tm_ld(at + 32, u[c ^ 1]);
            uint32_t(&x)[32] = u[c];
            // P = 2^y in two parts: hi by cutting the low bits off, lo exactly what was cut off, then cut itself
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float y0, y1, r0, r1;
              up2(fma2(pk2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), scale2, neg2), y0, y1);
              const float p0 = ex2(y0), p1 = ex2(y1);
              const unsigned long long pp = pk2(p0, p1);
              l2 = add2(l2, pp);
              const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
              hi[e / 2] = __byte_perm(u0, u1, 0x7632);
              up2(sub2(pp, pk2(__uint_as_float(u0 & 0xFFFF0000u), __uint_as_float(u1 & 0xFFFF0000u))), r0, r1);
              lo[e / 2] = __byte_perm(__float_as_uint(r0), __float_as_uint(r1), 0x7632);
            }
            // over the scores of the same keys, which have been read
            tm_st(at, hi);
            tm_st(at + 16, lo);
          }
          wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar((h == 0 ? kBPFull : kBPRest) + grp));
        }
      }
      if (!ok) break;
      g += nt;
      ok = wait_bar(bar(kBLEmpty + (j & 1)), ((j >> 1) & 1) ^ 1);
      if (!ok) break;
      float l0, l1;
      up2(l2, l0, l1);
      stat[((j & 1) * 2 + grp) * 128 + row] = make_float2(l0 + l1, ref);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBLFull + (j & 1)));
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ======================= O / l: lane = row =======================
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t stage = b0 + kOffStage + (warp & 3) * 4096;
    Ring ir;
    bool ok = true;
    for (int j = 0;; ++j) {
      Item it;
      ok = cta.take(ir, it);
      if (!ok || it.nt == 0) break;
      ok = wait_bar(bar(kBLFull + (j & 1)), (j >> 1) & 1);
      if (!ok) break;
      // a group's sum stands against the reference it used last (none: the sum is
      // 0, or NaN), O against the larger one
      const float2 s0 = stat[(j & 1) * 256 + row], s1 = stat[(j & 1) * 256 + 128 + row];
      // read before kBLEmpty hands the item on: the softmax warps may then run as
      // far as item j + 3, which takes this flag's place
      const bool spoilt = poison[j % 3] == j + 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBLEmpty + (j & 1)));
      const float top = fmaxf(s0.y, s1.y), M = top == -INFINITY ? 0.f : top;
      const float l = (s0.y == -INFINITY ? s0.x : s0.x * ex2(s0.y - M)) + (s1.y == -INFINITY ? s1.x : s1.x * ex2(s1.y - M));
      const float inv = l == 0.f ? 0.f : p.v_scale / l;
      const int r = it.r0 + row, i = quot(r, a.by_g), hq = it.h * G + r - i * G;
      const Part part = part_of<S>(a, it);
      const bool here = i < it.q_s, split = part.split, wide = split || !a.out_bf16;  // fp32 elements
      const int64_t prow = (part.at + i * part.step) * p.Hq + hq;
      if (split && here) a.part_lse[prow] = l == 0.f ? -INFINITY : __log2f(l) + M;
      // where this lane's row goes
      const int64_t el = split ? prow * D : (int64_t)(it.t0 + i) * p.o_st + (int64_t)hq * p.o_sh;
      char* const mine = !here ? nullptr : (split ? reinterpret_cast<char*>(a.part_o) : static_cast<char*>(p.out)) + el * (wide ? 4 : 2);
      ok = wait_bar(bar(kBOFull + (j & 1)), (j >> 1) & 1);
      if (!ok) break;
      fence_after();
      const uint32_t to = tmem + G_::kColO + (j & 1) * D + lane_off;
      // 32 columns of the warp's rows at a time turn through shared memory: stored
      // as they are, each lane would touch a line of its own
#pragma unroll 1
      for (int b = 0; b < D; b += 32) {
        uint32_t o[32];
        tm_ld(to + b, o);
        wait_ld();
        if (b + 32 == D) {  // the accumulator has been read
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBOFree + (j & 1)));
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = inv == 0.f ? 0u : __float_as_uint(__uint_as_float(o[c]) * inv);
#pragma unroll
        for (int q = 0; q < 8; ++q) st_s128(stage + swz<128>(lane, q), o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        __syncwarp();
        const int e = b + lane % 8 * 4;
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
          char* const to_row = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), 4 * k + lane / 8));
          float4 x;
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                       : "r"(stage + swz<128>(4 * k + lane / 8, lane % 8)));
          if (to_row != nullptr) {
            if (split) {
              *reinterpret_cast<float4*>(to_row + e * 4) = x;
            } else if (wide) {  // rows lie on 8 bytes
              *reinterpret_cast<float2*>(to_row + e * 4) = make_float2(x.x, x.y);
              *reinterpret_cast<float2*>(to_row + e * 4 + 8) = make_float2(x.z, x.w);
            } else {
              *reinterpret_cast<uint2*>(to_row + e * 2) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
            }
          }
          __syncwarp();
        }
      }
      if (here && spoilt) add_poison_row<D, S>(a, it, r);
      __syncwarp();
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
