// pkv_tree.cu -- drafted trees: masks and positions from parent links, the
// plain attention kernel of the fp32 path, and the move of an accepted
// path's cache rows.
#include "pkv_kernels.h"
#include "pkv_share.cuh"

namespace pkv {

// ---------------------------------------------------------------- masks
// One CTA per sequence, one thread per node: a node walks its ancestors,
// whose indices descend, so the words of its mask row are finished from the
// last to the first.  Bound by latency (a chain of loads per level); parents
// are staged in shared memory when the tree fits.
constexpr int kMaskThreads = 128;
constexpr int kMaskStage = 2048;

__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const int32_t* __restrict__ parents,
                                                                 const int32_t* __restrict__ cu_q,
                                                                 const int32_t* __restrict__ seq_lens, int64_t T,
                                                                 int32_t* __restrict__ mask, int64_t mask_stride,
                                                                 int32_t words, int32_t* __restrict__ positions,
                                                                 unsigned int* err) {
  __shared__ int32_t stage[kMaskStage];
  launch_dependents();
  grid_dep_wait();
  const int s = blockIdx.x;
  const int64_t c0 = __ldg(cu_q + s), c1 = __ldg(cu_q + s + 1);
  const int64_t n = __ldg(seq_lens + s);
  if (c0 < 0 || c1 < c0 || c1 > T) {  // the rows themselves are not known
    if (threadIdx.x == 0) atomicOr(err, kErrLengths);
    return;
  }
  const int q = static_cast<int>(c1 - c0);
  const bool bad = q > n || (int64_t)q > 32ll * words;
  if (bad) {
    if (threadIdx.x == 0) atomicOr(err, kErrLengths);
    for (int64_t i = threadIdx.x; i < q; i += kMaskThreads) {
      for (int w = 0; w < words; ++w) mask[(c0 + i) * mask_stride + w] = 0;
      positions[c0 + i] = 0;
    }
    return;
  }
  const bool staged = q <= kMaskStage;
  if (staged) {
    for (int i = threadIdx.x; i < q; i += kMaskThreads) {
      const int32_t par = __ldg(parents + c0 + i);
      stage[i] = par;
      if (par < -1 || par >= i) atomicOr(err, kErrLengths);
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < q; i += kMaskThreads) {
    int32_t* row = mask + (c0 + i) * mask_stride;
    int w = i >> 5, depth = 0, at = i;
    for (int k = words - 1; k > w; --k) row[k] = 0;
    uint32_t bits = 1u << (i & 31);
    for (;;) {
      int32_t par = staged ? stage[at] : __ldg(parents + c0 + at);
      if (par < -1 || par >= at) {  // a bad link ends the path
        if (!staged) atomicOr(err, kErrLengths);
        par = -1;
      }
      if (par < 0) break;
      ++depth;
      at = par;
      while ((at >> 5) < w) {
        row[w--] = static_cast<int32_t>(bits);
        bits = 0;
      }
      bits |= 1u << (at & 31);
    }
    for (; w >= 0; --w) {
      row[w] = static_cast<int32_t>(bits);
      bits = 0;
    }
    positions[c0 + i] = static_cast<int32_t>(n - q + depth);
  }
}

cudaError_t launch_tree_mask(const int32_t* parents, const int32_t* cu_q, const int32_t* seq_lens, int32_t B, int64_t T,
                             int32_t* mask, int64_t mask_stride, int32_t words, int32_t* positions, unsigned int* err,
                             cudaStream_t st) {
  if (B == 0 || T == 0) return cudaSuccess;
  return launch_ex(tree_mask_kernel, dim3((unsigned)B), dim3(kMaskThreads), 0, st, true, parents, cu_q, seq_lens, T,
                   mask, mask_stride, words, positions, err);
}

// ---------------------------------------------------------------- commit
// A path ascends, so entry i's destination base + i is at or before its
// source base + a_i, and never the source of a later entry (a_j >= j > i).
// Each thread owns one vector column of the token rows and takes the path's
// entries in order, a batch of loads before the batch's stores: no thread
// needs another's data, and one pass moves everything in place.  Bound by
// latency at a step's sizes (lengths, path, tables, rows: four dependent
// trips).
constexpr int kCommitThreads = 256;
constexpr int kCommitStage = 128;  // path entries whose slots are held at a time
constexpr int kCommitBatch = 8;

template <typename VecT>
__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const CommitParams p) {
  __shared__ int64_t src[kCommitStage], dst[kCommitStage];
  launch_dependents();
  grid_dep_wait();
  const int s = blockIdx.x;
  const int tid = threadIdx.x;
  const int64_t n = __ldg(p.seq_lens + s);
  const int64_t q = (int64_t)__ldg(p.cu_q + s + 1) - __ldg(p.cu_q + s);
  const int64_t len = __ldg(p.accepted_lens + s);
  const int64_t base = n - q;
  const int32_t* path = p.accepted + (int64_t)s * p.accepted_stride;
  const int32_t* bt = p.bt + (int64_t)s * p.bt_stride;
  unsigned int bad = 0;
  if (q < 0 || base < 0 || n > (int64_t)p.max_blocks * p.bs || len < 0 || len > q || len > p.A) bad = kErrLengths;
  auto slot_of = [&](int64_t pos) -> int64_t {
    const int32_t b = __ldg(bt + pos / p.bs);
    return (uint32_t)b < (uint64_t)p.num_blocks ? (int64_t)b * p.bs + pos % p.bs : -1;
  };
  if (!bad) {  // the whole path is checked before any row moves
    for (int64_t i = tid; i < len; i += kCommitThreads) {
      const int64_t a = __ldg(path + i), before = i > 0 ? __ldg(path + i - 1) : -1;
      if (a <= before || a >= q || a < i) {
        bad |= kErrLengths;
      } else if (slot_of(base + i) < 0 || slot_of(base + a) < 0) {
        bad |= kErrBlockRange;
      }
    }
  }
  const int any_len = __syncthreads_or(bad & kErrLengths), any_blk = __syncthreads_or(bad & kErrBlockRange);
  if (any_len || any_blk) {
    if (tid == 0 && blockIdx.y == 0) {
      atomicOr(p.err, (any_len ? kErrLengths : 0u) | (any_blk ? kErrBlockRange : 0u));
      if (p.new_lens) p.new_lens[s] = static_cast<int32_t>(n);
    }
    return;
  }
  if (tid == 0 && blockIdx.y == 0 && p.new_lens) p.new_lens[s] = static_cast<int32_t>(base + len);
  const int64_t cols = p.row_bytes / (int64_t)sizeof(VecT);  // vectors of a row; K's, then V's
  const int64_t c = (int64_t)blockIdx.y * kCommitThreads + tid;
  const bool act = c < 2 * cols;
  char* cache = (c < cols ? p.k_cache : p.v_cache) + (c < cols ? c : c - cols) * (int64_t)sizeof(VecT);
  for (int64_t b0 = 0; b0 < len; b0 += kCommitStage) {
    const int m = static_cast<int>(len - b0 < kCommitStage ? len - b0 : kCommitStage);
    __syncthreads();
    for (int i = tid; i < m; i += kCommitThreads) {
      src[i] = slot_of(base + __ldg(path + b0 + i));
      dst[i] = slot_of(base + b0 + i);
    }
    __syncthreads();
    if (!act) continue;
    for (int i0 = 0; i0 < m; i0 += kCommitBatch) {
      VecT x[kCommitBatch];
#pragma unroll
      for (int k = 0; k < kCommitBatch; ++k)
        if (i0 + k < m && src[i0 + k] != dst[i0 + k])
          x[k] = *reinterpret_cast<const VecT*>(cache + src[i0 + k] * p.row_bytes);
#pragma unroll
      for (int k = 0; k < kCommitBatch; ++k)
        if (i0 + k < m && src[i0 + k] != dst[i0 + k])
          *reinterpret_cast<VecT*>(cache + dst[i0 + k] * p.row_bytes) = x[k];
    }
  }
}

cudaError_t launch_tree_commit(const CommitParams& p, cudaStream_t st) {
  if (p.B == 0) return cudaSuccess;
  const int vec = p.row_bytes % 16 == 0 ? 16 : 8;
  const int64_t cols = 2 * p.row_bytes / vec;
  const dim3 grid((unsigned)p.B, (unsigned)((cols + kCommitThreads - 1) / kCommitThreads));
  if (vec == 16) return launch_ex(tree_commit_kernel<uint4>, grid, dim3(kCommitThreads), 0, st, true, p);
  return launch_ex(tree_commit_kernel<uint2>, grid, dim3(kCommitThreads), 0, st, true, p);
}

// ---------------------------------------------------------------- fp32 attention
// fp32 queries and caches, on the CUDA cores like pkv_attention's fp32 path:
// one CTA per (row, KV head), a warp per query head of the group, lanes over
// D, one key at a time.
// kShared: requests that share prefixes, each over its own table, causal.
template <typename OutT, bool kShared>
__global__ void __launch_bounds__(128) tree_f32_kernel(TreeParams p, SharedArgs h) {
  launch_dependents();
  grid_dep_wait();
  const int64_t t = blockIdx.x;
  const int g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (g == 0) {
    // inconsistent lengths are recorded, those of sequences without a row of their own too
    for (int64_t i = t * blockDim.x + threadIdx.x; i < p.B; i += (int64_t)gridDim.x * blockDim.x) {
      if constexpr (kShared) {
        int a, e, m;
        Group f;
        if (shared_request(p, h, static_cast<int>(i), a, e, m, f)) atomicOr(p.err, kErrLengths);
        continue;
      }
      const int a = __ldg(p.cu_q + i), e = __ldg(p.cu_q + i + 1), m = __ldg(p.seq_lens + i);
      if (a < 0 || e < a || (int64_t)e > p.T || e - a > m || (int64_t)m > (int64_t)p.max_blocks * p.bs || e - a > p.max_nodes)
        atomicOr(p.err, kErrLengths);
    }
  }
  if (t >= __ldg(p.cu_q + p.B)) return;
  const int s = upper_index(p.cu_q, p.B, static_cast<int>(t));
  const int c0 = __ldg(p.cu_q + s);
  const int q_s = __ldg(p.cu_q + s + 1) - c0;
  const int n = __ldg(p.seq_lens + s);
  if (q_s < 0 || q_s > n || (int64_t)n > (int64_t)p.max_blocks * p.bs || t < c0 || t - c0 >= q_s || q_s > p.max_nodes ||
      c0 < 0 || (int64_t)c0 + q_s > p.T) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrLengths);
    return;
  }
  if constexpr (kShared) {
    int a, e, m;
    Group f;
    if (shared_request(p, h, s, a, e, m, f)) return;
  }
  const int ctx = n - q_s;
  const int per = p.D / 32;  // elements per lane, <= 8
  const float* kc = static_cast<const float*>(p.k_cache);
  const float* vc = static_cast<const float*>(p.v_cache);
  const int32_t* bt_row = p.bt + (int64_t)s * p.bt_stride;
  const int32_t* mask = kShared ? nullptr : p.mask + t * p.mask_stride;
  for (int hh = warp; hh < p.G; hh += blockDim.x >> 5) {
    const int h = g * p.G + hh;
    const float* qrow = static_cast<const float*>(p.q) + t * p.q_st + (int64_t)h * p.q_sh;
    float qv[8], o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      qv[k] = k < per ? __ldg(qrow + lane + 32 * k) : 0.f;
      o[k] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
      if (kShared && j > ctx + static_cast<int>(t - c0)) break;
      if (!kShared && j >= ctx && !((static_cast<uint32_t>(__ldg(mask + ((j - ctx) >> 5))) >> ((j - ctx) & 31)) & 1u)) continue;
      const int lb = p.bs_shift >= 0 ? (j >> p.bs_shift) : (j / p.bs);
      const int32_t blk = __ldg(bt_row + lb);
      if (blk < 0 || blk >= p.num_blocks) {
        if (lane == 0) atomicOr(p.err, kErrBlockRange);
        continue;
      }
      const int64_t row = (((int64_t)blk * p.bs + (j - lb * p.bs)) * p.Hkv + g) * p.D;
      float dot = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < per) dot = fmaf(qv[k], __ldg(kc + row + lane + 32 * k), dot);
#pragma unroll
      for (int o2 = 16; o2 > 0; o2 >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o2);
      const float x = dot * p.qk_scale_log2;
      const float mn = fmaxf(m, x);
      const float ms = mn == -INFINITY ? 0.f : mn;  // every score so far is -inf
      const float alpha = exp2f(m - ms), w = exp2f(x - ms);
      l = l * alpha + w;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < per) o[k] = fmaf(w, __ldg(vc + row + lane + 32 * k), o[k] * alpha);
      m = mn;
    }
    OutT* orow = static_cast<OutT*>(p.out) + t * p.o_st + (int64_t)h * p.o_sh;
    const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing is zero
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < per) store1(orow + lane + 32 * k, l == 0.f ? 0.f : o[k] * inv);
  }
}

template <bool kShared>
static cudaError_t launch_f32_rows(const TreeParams& p, const SharedArgs& h, int out_kind, cudaStream_t st) {
  const dim3 grid((unsigned)p.T, (unsigned)p.Hkv), block(128);
  return out_kind ? launch_ex(tree_f32_kernel<__nv_bfloat16, kShared>, grid, block, 0, st, true, p, h)
                  : launch_ex(tree_f32_kernel<float, kShared>, grid, block, 0, st, true, p, h);
}

cudaError_t launch_tree_f32(const TreeParams& p, int out_kind, cudaStream_t st) {
  return launch_f32_rows<false>(p, SharedArgs{}, out_kind, st);
}

cudaError_t launch_shared_f32(const TreeParams& p, const int32_t* groups, int64_t max_group, int out_kind, cudaStream_t st) {
  SharedArgs h{};
  h.groups = groups;
  h.by_bs = fast_div(static_cast<uint32_t>(p.bs));
  h.prefix = groups + 2;
  h.prefix_step = 3;
  h.max_group = static_cast<int32_t>(max_group);
  return launch_f32_rows<true>(p, h, out_kind, st);
}

}  // namespace pkv
