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
//
// Bound: the memory on bf16 caches, once a kernel runs (its start takes about 5 us, of
// which there are mostly two); on e4m3 caches the softmax of the prefixes' 64-row
// tiles, and for short requests what an item costs besides its tiles (3 us, e4m3 4, of
// which a tile or two are hidden).  Measured, whole calls, 8 KV heads of 4 query heads, D 128,
// and pkv_attention on the same batch: 64 requests of 512 to 2,048 keys behind 2,048,
// bf16, 70 us (5.0 TB/s of the 347 MB that have to be read; 105); 64 in groups of 2 to
// 12 behind 1,024 to 8,192, bf16, 61 us (4.4 TB/s of 268 MB; 128); 16 behind 65,536,
// e4m3, 70 us (2.9 TB/s of 205 MB; 418); 256 of 64 to 1,024 in groups of 16 behind 512
// to 2,048, e4m3, 116 us (2.8 TB/s of 329 MB; 202); 4 behind 1,024, bf16, 11 us (28);
// nothing shared, 64 of 512 to 4,096, bf16, 92 us (104).
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
// Where a request's own rows fill a tile, on average, a prefix tile would serve no
// more of them, and its partials only cost: every request then takes all of its keys
// alone (16 requests of 64 rows times 4 heads behind 4,096 keys: 119 us instead of
// 125), with chunks of 8,192 keys when there are units for all SMs (1,024 / 2,048 /
// 4,096 / 8,192 keys: 119 / 118 / 119 / 103, as two launches).
constexpr int kPrePartRows = 4096;
constexpr int kSms = 152;  // counted here, not asked for: a workspace's size is known without a device
struct Cut {
  int n_pre, n_own;  // rows per MMA tile
  Chunking pre, own;
  bool alone;
  int64_t pre_chunks, own_chunks, rows_per_seq;
  int64_t rows;  // partial rows in all
};
Cut shared_cut(int64_t T, int64_t B, int64_t Hkv, int64_t G, int64_t max_q, int64_t max_group, int64_t max_ctx, bool f8) {
  Cut c;
  c.n_pre = tree_tile_rows(max_group * G, f8);
  c.n_own = tree_tile_rows(max_q * G, f8);
  c.alone = T * G >= B * c.n_pre;
  const int64_t units = std::max<int64_t>(1, Hkv * ((T * G + c.n_pre - 1) / c.n_pre));
  c.own = call_chunking(B, Hkv, max_q * G, f8);
  c.own.least = c.alone && units >= kSms ? 8192 : std::min(c.own.least, 1024);
  c.pre.least = units < 32 ? 512 : units < 128 ? 1024 : 2048;
  c.pre.most = static_cast<int32_t>(std::min<int64_t>(kTreeMaxChunks, std::max<int64_t>(8, kSms / units)));
  c.pre.most = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(c.pre.most, kPrePartRows / std::max<int64_t>(T, 1))));
  auto chunks = [&](const Chunking& k) { return std::max<int64_t>(1, std::min<int64_t>(k.most, (max_ctx + k.least - 1) / k.least)); };
  c.pre_chunks = c.alone ? 0 : chunks(c.pre);
  const int64_t most = chunks(c.own);
  c.rows_per_seq = most > 1 ? std::min<int64_t>(max_q * most, kTreePartRows) : 0;
  c.own_chunks = most > 1 && T * most <= B * c.rows_per_seq ? most : 0;
  c.rows = shared_own(T, c.pre_chunks) + (c.own_chunks ? T * c.own_chunks : B * c.rows_per_seq);
  return c;
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
  int c0, q, n, prefix;
  const bool bad = shared_request(p, h, s, c0, q, n, prefix) || q == 0;
  int np = 0, own = 1;
  if (!bad) {
    if (prefix > 0) np = (prefix - 1) / tree_chunk(prefix, 1, h.pre) + 1;
    own = (n - prefix - 1) / tree_chunk(n - prefix, q, h.own) + 1;
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
    const int64_t pre_at = (int64_t)(c0 + i) * h.pre_chunks;
    const int64_t own_at = own == 1 ? shared_single(p.T, h.pre_chunks, c0 + i) : own_first + (int64_t)i * own_step;
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

int64_t shared_rows(int64_t T, int64_t B, int64_t Hkv, int64_t G, int64_t max_q, int64_t max_group, int64_t max_ctx, bool f8) {
  return shared_cut(T, B, Hkv, G, max_q, max_group, max_ctx, f8).rows;
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
  h.alone = c.alone;
  h.max_group = static_cast<int32_t>(max_group);
  h.pre_chunks = static_cast<int32_t>(c.pre_chunks);
  h.own_chunks = static_cast<int32_t>(c.own_chunks);
  h.pre = c.pre;
  h.own = c.own;
  h.claims = reinterpret_cast<unsigned int*>(a.part_lse + c.rows * p.Hq);
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
  const int64_t most_pre = std::max<int64_t>(1, c.pre_chunks * p.Hkv * ((p.T * p.G + n_pre - 1) / n_pre + p.B));
  const int64_t most_own = (int64_t)p.B * kTreeMaxChunks * p.Hkv * ((max_q * p.G + n_own - 1) / n_own);
  auto launch = [&](int phase, int N, int64_t most) {
    h.phase = phase;
    if (p.D == 128) return f8 ? launch_phase<128, true>(a, N, most, num_sms, st) : launch_phase<128, false>(a, N, most, num_sms, st);
    return f8 ? launch_phase<64, true>(a, N, most, num_sms, st) : launch_phase<64, false>(a, N, most, num_sms, st);
  };
  cudaError_t e;
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
