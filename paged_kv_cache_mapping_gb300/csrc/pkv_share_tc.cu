// pkv_share_tc.cu -- attention of requests that share prefixes over the paged
// cache, on the fifth-generation tensor cores.
//
// What it computes: causal attention of every request over its own table, where
// the first tokens of neighbouring requests lie in the same blocks.  With p the
// group's prefix, row r of a request has
//     o_r = sum_c 2^(lse_c - M) o_c / sum_c 2^(lse_c - M)
// over chunks c of the keys 0 .. p - 1 and of the keys p .. of its own, each with
// its normalised output o_c and its log2-sum-exp2 lse_c.  The prefix's chunks take
// the rows of all the group's requests as one block of rows that see every key, so
// a prefix tile is read once for 16 to 128 rows (tiles of pkv_tree_narrow.cuh and
// pkv_tree_wide.cuh) instead of once for each request; the own keys are those
// kernels' chunks with a causal bound for a mask.
//
// Three launches: the prefixes, the own keys beside them (their CTAs take the SMs as
// the prefixes' leave them, see begin_phase()), and a join.  Where both take tiles of
// one size, the first two are one launch of which the prefixes are the first items.
// Calls with prompts, or in buffers of many more rows than they have, have a fourth in
// front (see Cut).
//
// Bound: the memory on bf16 caches where requests have many keys of their own, once a kernel
// runs (its start takes about 5 us, of which there are mostly two); on e4m3 caches the
// chain that the softmax warps of a 64-row tile go through together (load, scores, widening, vote, P: 0.44
// warps issued per scheduler and 45 % of the memory's rate behind 65,536 keys), and for short
// requests what an item costs besides its tiles (3 us, e4m3 4, of which a tile or two are
// hidden).  Measured, whole calls, 8 KV heads of 4 query heads, D 128, and pkv_attention
// in the same loop on the same batch: 64 requests of 512 to 2,048 keys behind 2,048, bf16, 71 us
// (4.9 TB/s of the 347 MB that have to be read; 105); 64 in groups of 2 to 12 behind
// 1,024 to 8,192, bf16, 61 us (4.4 TB/s of 268 MB; 128); 16 behind 65,536, e4m3, 68 us
// (3.0 TB/s of 205 MB; 418); 256 of 64 to 1,024 in groups of 16 behind 512 to 2,048, e4m3,
// 112 us (2.9 TB/s of 329 MB; 202); 4 behind 1,024, bf16, 11 us (28); nothing shared, 64
// of 512 to 4,096, bf16, 101 us (111).
#include "pkv_tree_narrow.cuh"

namespace pkv {
namespace {

// How a call's keys are cut.  A chunk costs its rows' partials, an item's start and
// end, and the join's reading; too few leave SMs without work.  `units` are the row
// tiles of all rows, times the KV heads, as if every tile were full.
//
// Prefixes: chunks of `least` keys, but no more of them than give each SM one item of
// one full group, or 8, and no more than leave kPrePartRows partial rows per head in
// all.  Measured, us, `least` 256 / 512 / 1024 / 2048 / 4096 (whole calls):
//     8 units, 4 rows over 1,024 keys    13.9 / 12.8 / 15.6 / 15.6 / 15.6
//    12       , 92 rows, D 64, 12 to 3,001   27.8 / 21.9 / 22.2 / 29.4 / 37.4
//    16       , 64 rows over 2,048       82.3 / 74.8 / 76.2 / 79.8 / 79.8
//    32       , 64 rows in 10 groups, 1,024 to 8,192   74.6 / 64.5 / 62.2 / 67.6 / 69.3
//   128, e4m3 , 256 rows in 16 groups, 512 to 2,048    143 / 127 / 121 / 117 / 117
//   and 8 units, 65,536 keys, e4m3, at most 64 / 19 / 8 / 4 chunks   84 / 70 / 100 / 164
//
// Own keys: the trees' rule, but at most 1,024 keys a chunk, since what is left over
// when CTAs claim their last items is an item (64 requests of 512 to 2,048 keys, 512 /
// 1,024 / 2,048 keys: 71.9 / 71.8 / 74.7; 256 of 64 to 1,024, e4m3: 123 / 117 / 117).
//
// A request whose rows fill a tile and that takes all of its keys alone has chunks of
// 8,192 keys when there are units for all SMs (16 requests of 64 rows times 4 heads behind
// 4,096 keys, 1,024 / 2,048 / 4,096 / 8,192 keys: 119 / 118 / 119 / 103, as two launches).
constexpr int kPrePartRows = 4096;
constexpr int kSms = 152;  // counted here, not asked for: a workspace's size is known without a device
constexpr int kPreLeast = 512;
__host__ __device__ inline int64_t row_units(int64_t rows, int64_t Hkv, int64_t G, int64_t tile) {
  const int64_t units = Hkv * ((rows * G + tile - 1) / tile);
  return units < 1 ? 1 : units;
}
// `rows`: of all the requests, or of those that read a prefix together
__host__ __device__ inline Chunking prefix_cut(int64_t rows, int64_t units) {
  const int64_t sms = kSms / units < 8 ? 8 : kSms / units, part = rows < 1 ? kPrePartRows : kPrePartRows / rows;
  const int64_t most = part < sms ? part : sms;
  return Chunking{units < 32 ? kPreLeast : units < 128 ? 1024 : 2048, most < 1 ? 1 : most > kTreeMaxChunks ? kTreeMaxChunks : (int32_t)most};
}

// With a plan, a small kernel looks through the groups first: where groups may have
// rows for several tiles, and a request for kLong, or for one while the buffers hold one
// for each; or where the buffers hold many more rows than the requests can have.  It
// decides from the rows that are there, request by request, so that neither rows behind
// the last nor a prompt among decodes keeps others from sharing, and it numbers the
// rows that share, so that only those have partials.  Without one every group of two
// and more shares.
constexpr int kLong = 4;
struct Cut {
  int n_pre, n_own;  // rows per MMA tile
  Chunking pre, own;
  int alone_least;
  bool plan;
  int64_t pre_chunks, pre_rows, own_chunks, rows_per_seq;
  int64_t rows;  // partial rows in all
};
Cut shared_cut(int64_t T, int64_t B, int64_t Hkv, int64_t G, int64_t max_q, int64_t max_group, int64_t max_ctx, bool f8) {
  Cut c;
  c.n_pre = tree_tile_rows(max_group * G, f8);
  c.n_own = tree_tile_rows(max_q * G, f8);
  const int64_t all = std::min(T, B * max_q), units = row_units(all, Hkv, G, c.n_pre);
  auto chunks = [&](const Chunking& k) { return std::max<int64_t>(1, std::min<int64_t>(k.most, (max_ctx + k.least - 1) / k.least)); };
  c.pre = prefix_cut(all, units);
  c.pre_chunks = chunks(c.pre);
  c.pre_rows = T * c.pre_chunks;
  const int64_t largest = std::min(max_q, std::max<int64_t>(1, T - B + 1)) * G;  // rows of a request, the others having one at least
  c.plan = (max_group * G > c.n_pre && (largest >= kLong * c.n_pre || (largest >= c.n_pre && T * G >= B * c.n_pre))) ||
           c.pre_rows > std::max<int64_t>(T, kPrePartRows);
  if (c.plan) c.pre_rows = std::min<int64_t>(std::max<int64_t>(T, kPrePartRows), T * kTreeMaxChunks);
  c.own = call_chunking(B, Hkv, max_q * G, f8);
  c.own.least = std::min(c.own.least, 1024);
  c.alone_least = units >= kSms ? 8192 : c.own.least;
  const int64_t most = chunks(c.own);
  c.rows_per_seq = most > 1 ? std::min<int64_t>(max_q * most, kTreePartRows) : 0;
  c.own_chunks = most > 1 && T * most <= B * c.rows_per_seq ? most : 0;
  c.rows = shared_own(T, c.pre_rows) + (c.own_chunks ? T * c.own_chunks : B * c.rows_per_seq);
  return c;
}

// The plan: which requests read their prefix with their group, where the partials of
// their rows are, and how prefixes are cut.
//
// A request with rows for kLong tiles reads all of its keys alone.  The others of a
// group read its prefix together when that takes a fifth (e4m3: a third) fewer tiles
// than one by one.  16 requests behind 4,096 keys, 4 heads, us, together and one by one:
//   bf16, tiles of 128 rows: 33 rows each 75 / 109, 50 rows 98 / 104, 56 rows 99 / 104, 58
//   rows 114 / 104, 64 rows 121 / 104, 100 rows 175 / 189, 128 rows 206 / 190, 1 to 61 rows
//   72 / 93
//   e4m3, tiles of 64: 17 rows 71 / 118, 20 rows 81 / 92, 24 to 28 rows 92 / 92, 30 rows 103
//   / 95, 1 to 61 rows 115 / 106
// A prompt of 2,048 rows and 32 decodes behind 4,096 keys: all together 537, one by one
// 356, so 285; e4m3 668, 458 and 391.
//
// One CTA, bound by latency: 2 to 3 us of a call (16 requests of 64 rows 102.5 -> 104.7 us,
// 52 of 1 to 27 rows 44.5 -> 47.4).  A request that takes no part gets -1, which the kernels
// behind record as they record it without a plan.
constexpr int kPlanThreads = 1024;
struct PlanArgs {
  int32_t* cut;     // [2]
  int32_t* prefix;  // [B]
  int32_t* at;      // [B] (see SharedArgs)
  uint32_t* tiles;  // [B + 1] of the requests before, one by one
  uint32_t* rows;   // [B + 1] of the requests before
  int32_t own_least, f8;
};

// Exclusive sums of two numbers over a block, from `carry` on.  Sums of counts below
// 2^31 stay there, whatever the lengths are (then v + its number is kSat).
constexpr uint32_t kSat = 0x7fffffffu;
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }
__device__ __forceinline__ void warp_sums(uint32_t (&v)[2], int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, v[k], o);
      if (lane >= o) v[k] = sat_add(v[k], x);
    }
  }
}
__device__ __forceinline__ void block_sums(uint32_t (&v)[2], uint32_t (&carry)[2], uint32_t (&warps)[32][2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
  const uint32_t own[2] = {v[0], v[1]};
  warp_sums(v, lane);
  __syncthreads();  // the last sums have been read
  if (lane == 31) {
    warps[warp][0] = v[0];
    warps[warp][1] = v[1];
  }
  __syncthreads();
  uint32_t w[2] = {lane < n ? warps[lane][0] : 0u, lane < n ? warps[lane][1] : 0u};
  warp_sums(w, lane);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t before = __shfl_sync(0xffffffffu, w[k], (warp - 1) & 31), all = __shfl_sync(0xffffffffu, w[k], 31);
    v[k] = sat_add(sat_add(carry[k], warp > 0 ? before : 0u), v[k]) - own[k];
    carry[k] = sat_add(carry[k], all);
  }
}

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const TreeParams p, const SharedArgs h, const PlanArgs out) {
  __shared__ uint32_t warps[32][2];
  launch_dependents();
  grid_dep_wait();
  auto heads_rows = [&](int q) { return (uint32_t)max(min(q, (int)p.T), 0) * (uint32_t)p.G; };  // in range whatever the lengths are
  auto tiles_of = [&](int q) { return (int)((heads_rows(q) + (1u << h.tile_log2) - 1) >> h.tile_log2); };
  auto is_long = [&](int q) { return heads_rows(q) >> h.tile_log2 >= kLong; };
  uint32_t carry[2] = {0, 0};
  for (int base = 0; base < p.B; base += blockDim.x) {
    const int s = base + threadIdx.x;
    uint32_t v[2] = {0, 0};
    if (s < p.B) {
      const int q = __ldg(p.cu_q + s + 1) - __ldg(p.cu_q + s);
      if (!is_long(q)) {
        v[0] = tiles_of(q);
        v[1] = max(q, 0);
      }
    }
    block_sums(v, carry, warps);
    if (s < p.B) {
      out.tiles[s] = v[0];
      out.rows[s] = v[1];
    }
  }
  if (threadIdx.x == 0) {
    out.tiles[p.B] = carry[0];
    out.rows[p.B] = carry[1];
  }
  __syncthreads();
  const uint32_t all = max(min(__ldg(p.cu_q + p.B), (int)p.T), 0);  // rows there are
  const int alone_least = (int64_t)tiles_of(static_cast<int>(all)) * p.Hkv >= kSms ? 8192 : out.own_least;
  uint32_t sums[2] = {0, 0};  // rows that share
  for (int base = 0; base < p.B; base += blockDim.x) {
    const int s = base + threadIdx.x;
    uint32_t v[2] = {0, 0};
    int prefix = 0, q = 0, least = out.own_least;
    if (s < p.B) {
      int c0, n;
      Group of;
      const bool bad = shared_request(p, h, s, c0, q, n, of);
      if (bad) prefix = -1;
      if (!bad && fills_tile(p, h, q)) least = alone_least;
      if (!bad && of.shares() && !is_long(q)) {
        const uint32_t alone = __ldcg(out.tiles + of.end) - __ldcg(out.tiles + of.first), rows = __ldcg(out.rows + of.end) - __ldcg(out.rows + of.first);
        const int part = out.f8 ? 3 : 5;
        if (part * (int64_t)tiles_of(static_cast<int>(rows)) <= (part - 1) * (int64_t)alone) prefix = of.prefix;
      }
      if (prefix > 0) v[0] = q;
    }
    block_sums(v, sums, warps);
    if (s < p.B) {
      // (more rows than there are: lengths that are inconsistent elsewhere)
      out.prefix[s] = prefix > 0 && (int64_t)v[0] + q > p.T ? -1 : prefix;
      out.at[s] = prefix > 0 ? static_cast<int32_t>(v[0]) : least;
    }
  }
  if (threadIdx.x == 0) {
    const int64_t rows = min((int64_t)sums[0], p.T);
    const Chunking c = prefix_cut(rows, max((int64_t)1, (int64_t)tiles_of(static_cast<int>(rows)) * p.Hkv));
    out.cut[0] = c.least;
    out.cut[1] = c.most;
  }
}

// One warp per (row, query head), as in tree_join_kernel: lane l holds elements l
// D / 32 .., four chunks' loads in flight; lane c of the weights holds those of
// chunks c, c + 32, .. (the prefix's, then the request's own).
template <int D, typename OutT>
__global__ void __launch_bounds__(256) shared_join_kernel(const __grid_constant__ TcArgs a) {
  constexpr int E = D / 32, kAt = 4, kW = 2 * kTreeMaxChunks / 32;
  const TreeParams& p = a.p;
  const SharedArgs& h = a.shared;
  const int s = blockIdx.x, lane = threadIdx.x & 31;
  // what does not come from the kernels before is read while they still run
  int c0, q, n, np = 0, own = 1, at = 0, pre_step = 0;
  Group of;
  const bool bad = shared_request(p, h, s, c0, q, n, of) || q == 0;
  if (!bad) {
    Chunking cut = h.own;
    if (of.shares()) {
      const Chunking pre = prefix_chunking(h);
      np = (of.prefix - 1) / tree_chunk(of.prefix, 1, pre) + 1;
      pre_step = prefix_step(h, pre);
      at = h.at ? __ldg(h.at + s) : c0;
    } else {
      of.prefix = 0;
      cut.least = own_least(p, h, s, q);
    }
    own = (n - of.prefix - 1) / tree_chunk(n - of.prefix, q, cut) + 1;
  }
  grid_dep_wait();
  launch_dependents();
  const int nc = np + own;
  if (bad || nc == 1) return;
  const int64_t rows = (int64_t)q * p.Hq;
  int own_step;
  const int64_t own_first = own_part(p, h, a.rows_per_seq, s, c0, own, own_step);
  for (int64_t r = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.y * 8) {
    const int i = static_cast<int>(r / p.Hq), hq = static_cast<int>(r - (int64_t)i * p.Hq);
    const int64_t pre_at = (int64_t)(at + i) * pre_step;
    const int64_t own_at = own == 1 ? shared_single(h.pre_rows, c0 + i) : own_first + (int64_t)i * own_step;
    auto row_of = [&](int c) { return ((c < np ? pre_at + c : own_at + (c - np)) * p.Hq + hq); };
    float v[kAt][E];
    auto load = [&](int b) {
#pragma unroll
      for (int k = 0; k < kAt; ++k) {
        if (b + k < nc) {
          const float* q = a.part_o + row_of(b + k) * D + lane * E;
          if constexpr (E == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(q));
            v[k][0] = f.x, v[k][1] = f.y, v[k][2] = f.z, v[k][3] = f.w;
          } else {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(q));
            v[k][0] = f.x, v[k][1] = f.y;
          }
        }
      }
    };
    float w[kW], M = -INFINITY;
#pragma unroll
    for (int k = 0; k < kW; ++k) w[k] = lane + 32 * k < nc ? __ldcg(a.part_lse + row_of(lane + 32 * k)) : -INFINITY;
    load(0);  // together with the weights
#pragma unroll
    for (int k = 0; k < kW; ++k) M = fmaxf(M, w[k]);  // a NaN stays out of M and comes back through the weights
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ms = M == -INFINITY ? 0.f : M;
    float L = 0.f;
#pragma unroll
    for (int k = 0; k < kW; ++k) {
      w[k] = lane + 32 * k < nc ? exp2f(w[k] - ms) : 0.f;
      L += w[k];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int b = 0;;) {
      float ws = w[0];
#pragma unroll
      for (int k = 1; k < kW; ++k) ws = b >= 32 * k ? w[k] : ws;
#pragma unroll
      for (int k = 0; k < kAt; ++k) {
        const float wk = __shfl_sync(0xffffffffu, ws, (b + k) & 31);
        if (b + k < nc && wk != 0.f) {  // a chunk without weight adds nothing
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(wk, v[k][e], acc[e]);
        }
      }
      b += kAt;
      if (b >= nc) break;
      load(b);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    OutT* dst = static_cast<OutT*>(p.out) + (int64_t)(c0 + i) * p.o_st + (int64_t)hq * p.o_sh + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) store2(dst + e, acc[e] * inv, acc[e + 1] * inv);
  }
}

template <int D, bool F8>
cudaError_t launch_phase(const TcArgs& a, int N, int64_t most, int num_sms, cudaStream_t st) {
  if constexpr (!F8) {
    if (N == 128) return launch_shared_wide(a, most, num_sms, st);
  }
  return N == 16   ? launch_items<Geo<D, 16, F8, true>>(tree_tc_kernel<D, 16, F8, true>, a, most, num_sms, st)
         : N == 32 ? launch_items<Geo<D, 32, F8, true>>(tree_tc_kernel<D, 32, F8, true>, a, most, num_sms, st)
                   : launch_items<Geo<D, 64, F8, true>>(tree_tc_kernel<D, 64, F8, true>, a, most, num_sms, st);
}

}  // namespace

int64_t shared_rows(int64_t T, int64_t B, int64_t Hkv, int64_t G, int64_t max_q, int64_t max_group, int64_t max_ctx, bool f8, int64_t* words) {
  const Cut c = shared_cut(T, B, Hkv, G, max_q, max_group, max_ctx, f8);
  *words = 1 + (c.plan ? 2 + 4 * B + 2 : 0);
  return c.rows;
}

cudaError_t launch_shared_tc(const TreeParams& p, const int32_t* groups, bool f8, int out_kind, int64_t max_q, int64_t max_group,
                             int64_t max_ctx, void* workspace, int num_sms, cudaStream_t st) {
  TcArgs a{};
  a.p = p;
  a.out_bf16 = out_kind;
  a.by_g = fast_div(static_cast<uint32_t>(p.G));
  a.by_bs = fast_div(static_cast<uint32_t>(p.bs));
  const Cut c = shared_cut(p.T, p.B, p.Hkv, p.G, max_q, max_group, max_ctx, f8);
  a.rows_per_seq = static_cast<int32_t>(c.rows_per_seq);
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = a.part_o + c.rows * p.Hq * p.D;
  SharedArgs& h = a.shared;
  h.groups = groups;
  h.by_bs = a.by_bs;
  h.prefix = groups + 2;
  h.prefix_step = 3;
  h.tile_log2 = c.n_pre == 16 ? 4 : c.n_pre == 32 ? 5 : c.n_pre == 64 ? 6 : 7;
  h.max_group = static_cast<int32_t>(max_group);
  h.pre_chunks = static_cast<int32_t>(c.pre_chunks);
  h.pre_rows = c.pre_rows;
  h.own_chunks = static_cast<int32_t>(c.own_chunks);
  h.pre = c.pre;
  h.own = c.own;
  h.alone_least = c.alone_least;
  h.claims = reinterpret_cast<unsigned int*>(a.part_lse + c.rows * p.Hq);
  cudaError_t e;
  if (c.plan) {
    PlanArgs out;
    out.cut = reinterpret_cast<int32_t*>(h.claims + 1);
    out.prefix = out.cut + 2;
    out.at = out.prefix + p.B;
    out.tiles = reinterpret_cast<uint32_t*>(out.at + p.B);
    out.rows = out.tiles + p.B + 1;
    out.own_least = c.own.least;
    out.f8 = f8;
    e = launch_ex(shared_plan_kernel, dim3(1), dim3(std::min(kPlanThreads, (p.B + 31) / 32 * 32)), 0, st, true, p, h, out);
    if (e != cudaSuccess) return e;
    h.plan = out.cut;
    h.prefix = out.prefix;
    h.prefix_step = 1;
    h.at = out.at;
  }
  // the wide kernel masks the products before they are scaled
  const int wide = p.qk_scale_log2 > 0.f ? 128 : 64, n_pre = std::min(c.n_pre, wide), n_own = std::min(c.n_own, wide);
  // One launch of one tile saves a kernel's start; us, two launches and one:
  //   4 requests behind 1,024 keys, 32 heads, bf16                  12.9   11.9
  //   38, groups up to 16 behind 20,611, 4 heads, D 64, e4m3        28.1   21.7
  //   62, groups of 2 behind 2,785, 24 heads, e4m3                  46.8   40.9
  //   16 of 64 rows, each alone (above)                            103.3  102.3
  // and none of 28 calls became slower.  At the larger of two tiles it would depend on
  // where the keys are (16 and 32 rows: 18.3 to 14.3, but also 83 to 94).
  const bool both = n_pre == n_own;
  const int64_t most_pre = std::max<int64_t>(1, (c.plan ? kTreeMaxChunks : c.pre_chunks) * p.Hkv * ((p.T * p.G + n_pre - 1) / n_pre + p.B));
  const int64_t most_own = (int64_t)p.B * kTreeMaxChunks * p.Hkv * ((max_q * p.G + n_own - 1) / n_own);
  auto launch = [&](int phase, int N, int64_t most) {
    h.phase = phase;
    if (p.D == 128) return f8 ? launch_phase<128, true>(a, N, most, num_sms, st) : launch_phase<128, false>(a, N, most, num_sms, st);
    return f8 ? launch_phase<64, true>(a, N, most, num_sms, st) : launch_phase<64, false>(a, N, most, num_sms, st);
  };
  if (both) {
    e = launch(kBoth, n_own, most_pre + most_own);
  } else {
    e = launch(kPrefixes, n_pre, most_pre);
    if (e == cudaSuccess) e = launch(kOwnKeys, n_own, most_own);
  }
  if (e != cudaSuccess) return e;
  const int64_t want = (max_q * p.Hq + 7) / 8;
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(want, (8 * num_sms + p.B - 1) / p.B));
  const dim3 grid((unsigned)p.B, (unsigned)y);
#define PKV_JOIN(D, O) launch_ex(shared_join_kernel<D, O>, grid, dim3(256), 0, st, true, a)
  if (p.D == 128) return out_kind ? PKV_JOIN(128, __nv_bfloat16) : PKV_JOIN(128, float);
  return out_kind ? PKV_JOIN(64, __nv_bfloat16) : PKV_JOIN(64, float);
#undef PKV_JOIN
}

}  // namespace pkv
