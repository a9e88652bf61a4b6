// pkv_tables.cu -- what a serving step needs around the attention of requests
// that grow, shrink and share prompts: block tables, slots and positions from the
// requests' lengths, and the prefixes that neighbouring block tables share.
#include <algorithm>

#include "pkv_kernels.h"

namespace pkv {

namespace {

constexpr uint32_t kSat = 0x7fffffffu;
// sums of counts below 2^31 that stay there: still associative
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }

// last s with at[s] <= x, for at[0] <= x < at[n] non-decreasing
__device__ __forceinline__ int find(const uint32_t* at, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

}  // namespace

// ---------------------------------------------------------------- tables of a step
// Request s goes from a = seq_lens[s] to b = new_seq_lens[s] tokens.  Its rows, the
// blocks it takes and those it gives back are counted, and three exclusive sums over
// the requests say where each of them lies.  The free list with the blocks given
// back behind it is one stack V of c + r entries; taken block i is V[c + r - 1 - i],
// whoever takes it, so every thread finds its own block without waiting for
// another's: in the list, or in the table that gave it back.  Nothing that is read is
// written: tables are written behind the old lengths of requests that grow, the list
// from entry c on.  Only the count may lie over its old value, and it is written
// when every CTA has read that.
//
// One cluster of up to eight CTAs: each scans all the lengths, and they share the
// rows and blocks.  Bound by latency: lengths, scan, list or table entry, store: 2.4
// us for 64 decodes, 3.9 for 608 rows and 814 blocks of 37 requests, 10.6 for 33,222
// rows of 256.  The cluster is for a count in its old place; where that has a place of
// its own nothing has to be ordered, and independent CTAs on all SMs could share the rows:
// not built.
constexpr int kTableThreads = 1024;

template <typename SlotT, int V>
__global__ void __launch_bounds__(kTableThreads) step_tables_kernel(const StepTablesParams p) {
  extern __shared__ uint32_t smem_u[];
  uint32_t* const row_at = smem_u;                // [B + 1] exclusive sums: rows
  uint32_t* const take_at = row_at + (p.B + 1);   // blocks taken
  uint32_t* const give_at = take_at + (p.B + 1);  // blocks given back
  __shared__ uint32_t warp_sum[32][3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  launch_dependents();
  grid_dep_wait();
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int64_t cap = (int64_t)p.max_blocks * p.bs;
  const int count = __ldcg(p.free_count);
  auto up = [&](int n) { return n == 0 ? 0 : quot(n - 1, p.by_bs) + 1; };

  uint32_t carry[3] = {0, 0, 0};
  for (int base = 0; base < p.B || base == 0; base += blockDim.x) {
    const int s = base + tid;
    uint32_t v[3] = {0, 0, 0}, own[3];
    if (s < p.B) {
      const int a = __ldg(p.seq_lens + s), b = __ldg(p.new_seq_lens + s), sh = p.shared_blocks ? __ldg(p.shared_blocks + s) : 0;
      const bool bad = a < 0 || b < 0 || a > cap || b > cap || sh < 0 || sh > p.max_blocks || (b > a && (int64_t)sh * p.bs > a);
      if (bad) {
        if (rank == 0) atomicOr(p.err, kErrLengths);
      } else {
        v[0] = max(b - a, 0);
        v[1] = max(up(b) - up(a), 0);
        v[2] = max(up(a) - max(up(b), sh), 0);
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) own[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, v[k], o);
        if (lane >= o) v[k] = sat_add(v[k], x);
      }
    }
    if (lane == 31) {
#pragma unroll
      for (int k = 0; k < 3; ++k) warp_sum[warp][k] = v[k];
    }
    __syncthreads();
    if (warp == 0) {
      uint32_t w[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) w[k] = lane < blockDim.x / 32 ? warp_sum[lane][k] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, w[k], o);
          if (lane >= o) w[k] = sat_add(w[k], x);
        }
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) warp_sum[lane][k] = w[k];
    }
    __syncthreads();
    uint32_t* const to[3] = {row_at, take_at, give_at};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t before = sat_add(carry[k], warp > 0 ? warp_sum[warp - 1][k] : 0u);
      // a saturated sum is refused below, so that the exclusive one may be taken by difference
      const uint32_t upto = sat_add(before, v[k]);
      if (s < p.B) to[k][s] = upto - own[k];
      carry[k] = sat_add(carry[k], warp_sum[31][k]);
    }
    __syncthreads();
  }
  if (tid == 0) {
    row_at[p.B] = carry[0];
    take_at[p.B] = carry[1];
    give_at[p.B] = carry[2];
  }
  // every CTA has read the count
  if (ctas > 1) {
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  }
  __syncthreads();
  const int64_t rows = carry[0], taken = carry[1], given = carry[2], top = count + given, left = top - taken;
  unsigned int refuse = 0;
  if (count < 0 || count > p.F || rows == kSat || taken == kSat || given == kSat || rows > p.T)
    refuse = kErrLengths;
  else if (left < 0)
    refuse = kErrOutOfBlocks;
  else if (left > p.F)
    refuse = kErrLengths;
  if (rank == 0 && tid == 0) {
    if (refuse) atomicOr(p.err, refuse);
    *p.new_free_count = refuse ? count : static_cast<int>(left);
  }
  if (rank == 0)
    for (int s = tid; s <= p.B; s += blockDim.x) p.cu_q[s] = refuse ? 0 : static_cast<int>(row_at[s]);
  const int64_t first = (int64_t)rank * blockDim.x + tid, step = (int64_t)ctas * blockDim.x;
  // entry x of the blocks given back; entry i of the blocks taken
  auto back = [&](uint32_t x) -> int {
    const int s = find(give_at, p.B, x);
    const int keep = max(up(__ldg(p.new_seq_lens + s)), p.shared_blocks ? __ldg(p.shared_blocks + s) : 0);
    return __ldcg(p.bt + s * p.bt_stride + keep + static_cast<int>(x - give_at[s]));
  };
  auto took = [&](uint32_t i) -> int {
    const int64_t at = top - 1 - i;
    return at < count ? __ldcg(p.free_blocks + at) : back(static_cast<uint32_t>(at - count));
  };
  SlotT* const slots = static_cast<SlotT*>(p.slots);
  const int64_t n_rows = refuse ? 0 : rows;
  // One numbering of all the work, so that its chains of loads run side by side: the
  // rows, V in turn (which mostly are one request's and lie in one block), the blocks
  // taken, the blocks given back that stay in the list.
  const int64_t row_units = (p.T + V - 1) / V, n_taken = refuse ? 0 : taken, n_back = refuse ? 0 : max(left - count, (int64_t)0);
  for (int64_t u = first; u < row_units + n_taken + n_back; u += step) {
    if (u >= row_units + n_taken) {
      const int64_t x = u - row_units - n_taken;
      p.free_blocks[count + x] = back(static_cast<uint32_t>(x));
      continue;
    }
    if (u >= row_units) {
      const uint32_t i = static_cast<uint32_t>(u - row_units);
      const int s = find(take_at, p.B, i);
      p.bt[s * p.bt_stride + up(__ldg(p.seq_lens + s)) + static_cast<int>(i - take_at[s])] = took(i);
      continue;
    }
    const int64_t t0 = u * V;
    int s = t0 < n_rows ? find(row_at, p.B, static_cast<uint32_t>(t0)) : p.B, held = -1, block = -1;
    SlotT out[V];
    int at[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int64_t t = t0 + k;
      out[k] = -1;
      at[k] = 0;
      if (t >= n_rows) continue;
      while (t >= row_at[s + 1]) {  // (row_at[B] is n_rows)
        ++s;
        held = -1;
      }
      const int a = __ldg(p.seq_lens + s);
      at[k] = a + static_cast<int>(t - row_at[s]);
      const int lb = quot(at[k], p.by_bs);
      if (lb != held) {
        const int had = up(a);
        block = lb < had ? __ldcg(p.bt + s * p.bt_stride + lb) : took(take_at[s] + (lb - had));
        held = lb;
      }
      const int64_t slot = (int64_t)block * p.bs + (at[k] - lb * p.bs);
      if (block < 0 || (sizeof(SlotT) == 4 && slot > INT32_MAX))
        atomicOr(p.err, block < 0 ? kErrBlockRange : kErrSlotRange);
      else
        out[k] = static_cast<SlotT>(slot);
    }
    if (V == 4 && p.vectors && t0 + V <= p.T) {
      if constexpr (sizeof(SlotT) == 4) {
        *reinterpret_cast<int4*>(slots + t0) = make_int4(out[0], out[1 % V], out[2 % V], out[3 % V]);
      } else {
        *reinterpret_cast<longlong2*>(slots + t0) = make_longlong2(out[0], out[1 % V]);
        *reinterpret_cast<longlong2*>(slots + t0 + 2) = make_longlong2(out[2 % V], out[3 % V]);
      }
      if (p.positions) *reinterpret_cast<int4*>(p.positions + t0) = make_int4(at[0], at[1 % V], at[2 % V], at[3 % V]);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if (t0 + k >= p.T) break;
        slots[t0 + k] = out[k];
        if (p.positions) p.positions[t0 + k] = at[k];
      }
    }
  }
}

template <typename SlotT, int V>
static cudaError_t launch_tables(const StepTablesParams& p, unsigned ctas, unsigned threads, cudaStream_t st) {
  const size_t smem = 3 * sizeof(uint32_t) * ((size_t)p.B + 1);
  const auto f = step_tables_kernel<SlotT, V>;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) e = set_smem_attr(reinterpret_cast<const void*>(f), 3 * sizeof(uint32_t) * (kMaxRequests + 1));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;  // a launch with a cluster takes the host longer
  return cudaLaunchKernelEx(&cfg, f, p);
}

cudaError_t launch_step_tables(const StepTablesParams& p, bool slots_i64, cudaStream_t st) {
  StepTablesParams q = p;
  q.vectors = reinterpret_cast<uintptr_t>(p.slots) % 16 == 0 && reinterpret_cast<uintptr_t>(p.positions) % 16 == 0;
  // four rows a thread where there are many (33,222 rows of 256 requests: 10.9 us, one
  // by one 13.0; 4 CTAs 15.2).  One CTA of fewer warps for a few rows and requests
  // meets at its barriers sooner (64 of each: 2.9 us with 256 threads, 3.3 with 1,024;
  // 608 rows and 814 blocks 6.9 and 4.5).
  if (p.T <= kTableThreads) {
    const unsigned threads = p.T <= 256 && p.B <= 256 ? 256 : kTableThreads;
    return slots_i64 ? launch_tables<int64_t, 1>(q, 1, threads, st) : launch_tables<int32_t, 1>(q, 1, threads, st);
  }
  unsigned ctas = 2;
  while (ctas < 8 && (int64_t)ctas * kTableThreads < p.T) ctas *= 2;
  return slots_i64 ? launch_tables<int64_t, 4>(q, ctas, kTableThreads, st) : launch_tables<int32_t, 4>(q, ctas, kTableThreads, st);
}

// ---------------------------------------------------------------- shared prefixes
// common[s]: leading entries of the tables of requests s - 1 and s that are the
// same block, over the blocks that both have full of context.  Request s is linked
// to the one before it when that is at least min_tokens, and at least half of what
// either of them shares with its other neighbour.  A group is a run of links, its prefix
// the least common: a link costs its neighbours half of theirs at most, a chain of
// links more.
//
// A CTA per pair of tables compares 2,048 entries a trip, all loads of a trip in
// flight, and stops at the first difference; then one CTA finds the runs by a scan.
// Bound by latency: lengths, table entries, and the second kernel's trip: 4.0 us for 64
// requests behind 2,048 tokens, 4.9 for 256 with prefixes of up to 65,536.  (Both in one
// cluster of eight CTAs, the counts handed over in shared memory: 4.8 and 4.6.)
constexpr int kPairThreads = 256, kPairLoads = 8;

__global__ void __launch_bounds__(kPairThreads) common_kernel(const PrefixParams p) {
  __shared__ int first_off;
  launch_dependents();
  grid_dep_wait();
  const int s = blockIdx.x, tid = threadIdx.x;
  int full = 0;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {  // this request, then the one before
    if (s < k) {
      full = 0;
      break;
    }
    const int c0 = __ldg(p.cu_q + s - k), c1 = __ldg(p.cu_q + s - k + 1), n = __ldg(p.seq_lens + s - k);
    const bool off = c0 < 0 || c1 < c0 || c1 - c0 > n || (int64_t)n > (int64_t)p.max_blocks * p.bs;
    const int f = off ? 0 : (n - (c1 - c0)) / p.bs;
    full = k == 0 ? f : min(full, f);
    bad |= off && k == 0;
  }
  if (bad && tid == 0) atomicOr(p.err, kErrLengths);
  if (tid == 0) first_off = full;
  const int32_t* mine = p.bt + (int64_t)s * p.bt_stride;
  const int32_t* prev = mine - p.bt_stride;
  __syncthreads();
  for (int base = 0; base < full; base += kPairThreads * kPairLoads) {
    int a[kPairLoads], b[kPairLoads];
#pragma unroll
    for (int k = 0; k < kPairLoads; ++k) {
      const int j = base + k * kPairThreads + tid;
      a[k] = b[k] = 0;
      if (j < full) {
        a[k] = __ldg(mine + j);
        b[k] = __ldg(prev + j);
      }
    }
    int off = full;
#pragma unroll
    for (int k = kPairLoads - 1; k >= 0; --k)
      if (a[k] != b[k] || a[k] < 0) off = min(off, base + k * kPairThreads + tid);
    const bool any = __syncthreads_or(off < full);
    if (any) {
      if (off < full) atomicMin(&first_off, off);
      break;
    }
  }
  __syncthreads();
  if (tid == 0) p.groups[3 * s + 2] = s == 0 ? 0 : first_off;
}

constexpr int kGroupThreads = 1024;

__global__ void __launch_bounds__(kGroupThreads) groups_kernel(const PrefixParams p) {
  extern __shared__ int smem_i[];
  int* const common = smem_i;          // [B + 2]: common[s] at s, 0 behind the last
  int* const first = common + p.B + 2;  // [B]: first request of its group
  int* const least = first + p.B;       // [B], at a group's first request: least common of its links
  int* const end = least + p.B;         // [B], there too: request behind its last
  __shared__ int warp_max[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.B;
  launch_dependents();
  grid_dep_wait();
  for (int s = tid; s < B + 2; s += kGroupThreads) {
    common[s] = s < B ? __ldcg(p.groups + 3 * s + 2) : 0;
    if (s < B) {
      least[s] = INT32_MAX;
      end[s] = 0;
    }
  }
  __syncthreads();
  int carry = 0;
  for (int base = 0; base < B; base += kGroupThreads) {
    const int s = base + tid;
    bool link = false;
    int c = 0;
    if (s < B) {
      c = common[s];
      const int64_t side = max(s > 0 ? common[s - 1] : 0, common[s + 1]);
      link = c > 0 && (int64_t)c * p.bs >= p.min_tokens && 2 * (int64_t)c >= side;
    }
    int f = s < B && !link ? s : 0;  // the largest of these at or before s is its group's first (request 0 has no link)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, f, o);
      if (lane >= o) f = max(f, x);
    }
    if (lane == 31) warp_max[warp] = f;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < warp; ++w) before = max(before, warp_max[w]);
    int all = before;
    for (int w = warp; w < 32; ++w) all = max(all, warp_max[w]);
    carry = all;
    f = max(f, before);
    if (s < B) {
      first[s] = f;
      atomicMax(end + f, s + 1);
      if (link) atomicMin(least + f, c);
    }
    __syncthreads();
  }
  for (int s = tid; s < B; s += kGroupThreads) {
    const int f = first[s], l = least[f];
    p.groups[3 * s] = f;
    p.groups[3 * s + 1] = end[f];
    p.groups[3 * s + 2] = l == INT32_MAX ? 0 : l * p.bs;
  }
}

cudaError_t launch_shared_prefixes(const PrefixParams& p, cudaStream_t st) {
  if (p.B == 0) return cudaSuccess;
  cudaError_t e = launch_ex(common_kernel, dim3((unsigned)p.B), dim3(kPairThreads), 0, st, true, p);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(int) * (4 * (size_t)p.B + 2);
  if (smem > 48 * 1024) {
    e = set_smem_attr(reinterpret_cast<const void*>(groups_kernel), sizeof(int) * (4 * kMaxRequests + 2));
    if (e != cudaSuccess) return e;
  }
  return launch_ex(groups_kernel, dim3(1), dim3(kGroupThreads), smem, st, true, p);
}

}  // namespace pkv
