// pkv_share.cuh -- requests of a step in groups that share a prefix: what the
// kernels of pkv_shared_attention read of them, and how their workspace is laid
// out.
#pragma once

#include "pkv_kernels.h"

namespace pkv {

// What a launch computes: the groups' rows over their prefixes, the requests' rows
// over the rest, or first the one and then the other.
enum : int { kPrefixes = 0, kOwnKeys = 1, kBoth = 2 };

// Keys per chunk of a long axis (see tree_chunking()).
struct Chunking {
  int32_t least, most;
};

struct SharedArgs {
  const int32_t* groups;  // [B, 3]: first request, request behind the last, tokens of the prefix
  int32_t phase;          // kPrefixes, kOwnKeys or kBoth
  int32_t alone;          // requests with rows enough for tiles of their own: none reads a prefix with others
  int32_t max_group;      // rows of a group at most
  int32_t pre_chunks;     // chunks of a prefix at most
  int32_t own_chunks;     // partial rows for each packed row, of own keys; 0: they are counted by request
  Chunking pre, own;      // how prefixes and own keys are cut
  unsigned int* claims;   // items of the own keys that are taken (see next_item())
};

// Partial rows of the workspace: pre_chunks for each packed row, one more for each,
// then those of own keys in several chunks: own_chunks for each packed row, or
// rows_per_seq for each request, whichever is less in all.  (A bound on a request's
// rows says little of a batch with one prompt among decodes, and the number of packed
// rows little where most of them are padding.)
__host__ __device__ inline int64_t shared_single(int64_t T, int64_t pre_chunks, int64_t t) { return T * pre_chunks + t; }
__host__ __device__ inline int64_t shared_own(int64_t T, int64_t pre_chunks) { return T * (pre_chunks + 1); }
// of request s, packed rows from c0 on, nc chunks: its first partial row, and how far a row's are from the last one's
__device__ __forceinline__ int64_t own_part(const TreeParams& p, const SharedArgs& h, int rows_per_seq, int s, int c0, int nc, int& step) {
  step = h.own_chunks ? h.own_chunks : nc;
  return shared_own(p.T, h.pre_chunks) + (h.own_chunks ? (int64_t)c0 * step : (int64_t)s * rows_per_seq);
}

// Request s: packed rows c0 .. c0 + q - 1, n keys, the first `prefix` of them read
// with its group.  Returns whether it takes no part: inconsistent lengths, a prefix that
// is not whole blocks of its context, or a group that its first request does not
// name in the same words or whose rows do not hold the request's.
__device__ __forceinline__ bool shared_request(const TreeParams& p, const SharedArgs& h, int s, int& c0, int& q, int& n, int& prefix) {
  const int32_t* g = h.groups + 3 * (int64_t)s;
  c0 = __ldg(p.cu_q + s);
  const int c1 = __ldg(p.cu_q + s + 1), g0 = __ldg(g), g1 = __ldg(g + 1);
  n = __ldg(p.seq_lens + s);
  prefix = __ldg(g + 2);
  q = c1 - c0;
  if (c0 < 0 || c1 < c0 || (int64_t)c1 > p.T || q > n || (int64_t)n > (int64_t)p.max_blocks * p.bs || q > p.max_nodes) return true;
  if (prefix == 0) return false;
  if (prefix < 0 || prefix > n - q || prefix % p.bs != 0 || g0 < 0 || g0 > s || g1 <= s || g1 > p.B) return true;
  const int32_t* f = h.groups + 3 * (int64_t)g0;
  const int t0 = __ldg(p.cu_q + g0), t1 = __ldg(p.cu_q + g1), same = prefix;
  if (h.alone) prefix = 0;
  return __ldg(f) != g0 || __ldg(f + 1) != g1 || __ldg(f + 2) != same || t0 < 0 || t0 > c0 || t1 < c1 || (int64_t)t1 > p.T ||
         t1 - t0 > h.max_group;
}

// Prefixes are read for runs of neighbours that name the same group in the same
// words, found by a warp for 32 requests (s = from + lane) at a time: whether request s
// is the first of a run, whose packed rows are c0 .. c0 + q - 1, over n keys of the table of
// request `table`.  Mostly a run is its group, but nothing keeps groups that the
// caller made from overlapping, and a partial row must have one writer: its run is the
// only one that a request is in.  What shared_request() takes for a request of the run
// has passed all of this.
//
// (Groups taken at their word: 0.1 to 0.4 us less a call.  What is rare stands apart: a
// call's first item waits until this code is fetched.)
static __device__ __noinline__ int run_end(const SharedArgs& h, int s, int lane, int first, int end, int prefix) {
  for (; s < end; s += 128) {
    uint32_t other[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int32_t* g = h.groups + 3 * (int64_t)min(s + 32 * k + lane, end - 1);
      other[k] = __ldg(g) != first || __ldg(g + 1) != end || __ldg(g + 2) != prefix;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      other[k] = __ballot_sync(0xffffffffu, other[k]);
      if (other[k]) return min(end, s + 32 * k + __ffs(other[k]) - 1);
    }
  }
  return end;
}
static __device__ __noinline__ bool names(const SharedArgs& h, int s, int first, int end, int prefix) {
  const int32_t* g = h.groups + 3 * (int64_t)s;
  return __ldg(g) == first && __ldg(g + 1) == end && __ldg(g + 2) == prefix;
}
__device__ __forceinline__ int load_now(const int32_t* q) {  // where it stands, not where it is needed
  int x;
  asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(x) : "l"(q));
  return x;
}
__device__ __forceinline__ bool shared_run(const TreeParams& p, const SharedArgs& h, int from, int lane, int& c0, int& q, int& n, int& table) {
  if (h.alone) return false;
  const int s = from + lane;
  bool head = s < p.B;
  // this request's numbers, those of the one before, and of the one 32 on, in one trip
  const int32_t* g = h.groups + 3 * (int64_t)min(s, p.B - 1);
  const int32_t* const after = h.groups + 3 * (int64_t)min(s + 32, p.B - 1);
  const int32_t* const before = s > 0 ? g - 3 : g;
  const int end = load_now(g + 1), a0 = load_now(after), a1 = load_now(after + 1), a2 = load_now(after + 2);
  table = __ldg(g);
  n = __ldg(g + 2);
  c0 = __ldg(p.cu_q + min(s, p.B));
  const bool goes_on = head && s > 0 && __ldg(before) == table && __ldg(before + 1) == end && __ldg(before + 2) == n;
  head = head && n > 0 && table >= 0 && (table == s || (table < s && !goes_on)) && end > s && end <= p.B &&
         (int64_t)n <= (int64_t)p.max_blocks * p.bs && n % p.bs == 0;
  const int t1 = head ? __ldg(p.cu_q + end) : 0;
  // behind the run: the next request that names another group
  const uint32_t other = __ballot_sync(0xffffffffu, !goes_on) & ~((2u << lane) - 1u);
  int behind = min(end, other ? from + __ffs(other) - 1 : from + 32);
  // only the last run can go on behind these requests
  if (const uint32_t on = __ballot_sync(0xffffffffu, head && other == 0 && end > from + 32)) {
    const int o = 31 - __clz(on), of = __shfl_sync(0xffffffffu, table, o), l = __shfl_sync(0xffffffffu, end, o), m = __shfl_sync(0xffffffffu, n, o);
    const uint32_t off = __ballot_sync(0xffffffffu, a0 != of || a1 != l || a2 != m);
    int e = min(l, from + 32 + (off ? __ffs(off) - 1 : 32));
    if (off == 0 && l > from + 64) e = run_end(h, from + 64, lane, of, l, m);
    if (lane == o) behind = e;
  }
  if (!head) return false;
  const int upto = behind == end ? t1 : __ldg(p.cu_q + behind);
  int t0 = c0;
  if (table != s) {
    if (!names(h, table, table, end, n)) return false;
    t0 = __ldg(p.cu_q + table);
  }
  q = upto - c0;
  return t0 >= 0 && t0 <= c0 && upto > c0 && upto <= t1 && (int64_t)t1 <= p.T && t1 - t0 <= h.max_group;
}

}  // namespace pkv
