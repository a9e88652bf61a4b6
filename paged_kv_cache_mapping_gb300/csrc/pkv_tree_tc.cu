// pkv_tree_tc.cu -- attention of drafted trees over the paged cache: the choice
// among the tensor-core kernels of pkv_tree_narrow.cuh and pkv_tree_wide.cuh, and
// the kernel that joins the chunks of a long sequence.
#include "pkv_tree_narrow.cuh"

namespace pkv {
namespace {

// ---------------------------------------------------------------- join
// o = sum_c 2^(lse_c - M) o_c / sum_c 2^(lse_c - M) over a row's chunks, in
// order.  One warp per (row, query head); lane l holds elements l D/32 ..;
// four chunks' loads in flight, the first with those of the weights.  grid: (sequences, parts of a sequence's rows).
template <int D, typename OutT>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeParams p, const float* part_o, const float* part_lse,
                                                        int rows_per_seq, Chunking chunking) {
  // what does not come from the kernel before is read while its last CTAs still
  // run (they end after that kernel's own predecessors have)
  constexpr int E = D / 32, kAt = 4;  // chunks in flight (eight: 1 % slower in all)
  const int s = blockIdx.x, lane = threadIdx.x & 31;
  const int c0 = __ldg(p.cu_q + s), c1 = __ldg(p.cu_q + s + 1), n = __ldg(p.seq_lens + s);
  const int q_s = c1 - c0;
  const bool bad = c0 < 0 || c1 <= c0 || (int64_t)c1 > p.T || q_s > n || (int64_t)n > (int64_t)p.max_blocks * p.bs || q_s > p.max_nodes;
  const int chunk = bad ? 1 : tree_chunk(n, q_s, chunking);
  const int nc = bad ? 1 : (n - 1) / chunk + 1;
  grid_dep_wait();
  launch_dependents();
  if (nc == 1) return;
  const int64_t rows = (int64_t)q_s * p.Hq;
  for (int64_t r = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.y * 8) {
    const int i = static_cast<int>(r / p.Hq), hq = static_cast<int>(r - (int64_t)i * p.Hq);
    const int64_t at = ((int64_t)s * rows_per_seq + (int64_t)i * nc) * p.Hq + hq;
    const float* src = part_o + at * D + lane * E;
    float v[kAt][E];
    auto load = [&](int b) {
#pragma unroll
      for (int k = 0; k < kAt; ++k) {
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
    };
    float lv[2], M = -INFINITY;
#pragma unroll
    for (int k = 0; k < 2; ++k) lv[k] = lane + 32 * k < nc ? __ldcg(part_lse + at + (int64_t)(lane + 32 * k) * p.Hq) : -INFINITY;
    load(0);  // together with the weights
#pragma unroll
    for (int k = 0; k < 2; ++k) M = fmaxf(M, lv[k]);  // a NaN stays out of M and comes back through the weights
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
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int b = 0;;) {
#pragma unroll
      for (int k = 0; k < kAt; ++k) {
        const float wk = __shfl_sync(0xffffffffu, b < 32 ? w[0] : w[1], (b + k) & 31);
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
// ---------------------------------------------------------------- host
}  // namespace

int64_t tree_tc_rows_per_seq(int64_t B, int64_t Hkv, int64_t G, int64_t max_q, int64_t max_ctx, bool f8) {
  const Chunking c = call_chunking(B, Hkv, max_q * G, f8);
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
  const int64_t rps = tree_tc_rows_per_seq(p.B, p.Hkv, p.G, max_q, max_ctx, f8);
  a.rows_per_seq = static_cast<int32_t>(rps);
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = a.part_o + (int64_t)p.B * rps * p.Hq * p.D;
  const int64_t rows = max_q * p.G;
  // the wide kernel masks the products before they are scaled
  const int most_n = tree_tile_rows(rows, f8), N = p.qk_scale_log2 > 0.f ? most_n : std::min(most_n, 64);
  a.chunking = call_chunking(p.B, p.Hkv, rows, f8);
  const int64_t most = (int64_t)p.B * kTreeMaxChunks * p.Hkv * ((rows + N - 1) / N);
  cudaError_t e;
#define PKV_TC1(D, F8)                                      \
  (N == 16   ? launch_items<Geo<D, 16, F8, false>>(tree_tc_kernel<D, 16, F8, false>, a, most, num_sms, st)    \
   : N == 32 ? launch_items<Geo<D, 32, F8, false>>(tree_tc_kernel<D, 32, F8, false>, a, most, num_sms, st)    \
             : launch_items<Geo<D, 64, F8, false>>(tree_tc_kernel<D, 64, F8, false>, a, most, num_sms, st))
  if (N == 128)
    e = launch_tree_wide(a, most, num_sms, st);
  else if (p.D == 128)
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
