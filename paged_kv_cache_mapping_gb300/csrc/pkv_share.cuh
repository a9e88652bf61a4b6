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

// Whether request s is the first of a group with a prefix of n keys, read through
// its table, for rows c0 .. c0 + q - 1 (those of all its requests).  What
// shared_request() takes for a request of the group has passed all of this.
__device__ __forceinline__ bool shared_prefix(const TreeParams& p, const SharedArgs& h, int s, int& c0, int& q, int& n) {
  if (h.alone) return false;
  const int32_t* g = h.groups + 3 * (int64_t)s;
  const int g0 = __ldg(g), g1 = __ldg(g + 1);
  c0 = __ldg(p.cu_q + s);
  n = __ldg(g + 2);
  if (g0 != s || n <= 0 || g1 <= s || g1 > p.B || (int64_t)n > (int64_t)p.max_blocks * p.bs || n % p.bs != 0) return false;
  const int t1 = __ldg(p.cu_q + g1);
  q = t1 - c0;
  return c0 >= 0 && t1 > c0 && (int64_t)t1 <= p.T && q <= h.max_group;
}

}  // namespace pkv
