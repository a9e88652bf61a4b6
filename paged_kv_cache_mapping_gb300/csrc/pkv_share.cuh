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
  const int32_t* prefix;  // [B], prefix_step apart: tokens that a request reads with its group, as groups or the plan has them
  int32_t prefix_step;
  FastDiv by_bs;          // tokens of a block
  int32_t tile_log2;      // rows of a tile over a prefix
  int32_t max_group;      // rows of a group at most
  int32_t pre_chunks;     // chunks of a prefix at most (without a plan)
  int64_t pre_rows;       // partial rows of prefixes
  int32_t own_chunks;     // partial rows for each packed row, of own keys; 0: they are counted by request
  Chunking pre, own;      // how prefixes and own keys are cut (pre: without a plan)
  int32_t alone_least;    // own.least of requests that fill tiles and read all of their keys (without a plan)
  unsigned int* claims;   // items of the own keys that are taken (see next_item())
  // What shared_plan_kernel wrote, or NULL: {pre.least, pre.most}, and [B]: where the partial
  // rows of a request's prefix begin, in rows (without a plan: at its packed rows), or,
  // of one that reads all of its keys alone, its own.least
  const int32_t* plan;
  const int32_t* at;
};

// Partial rows of the workspace: those of prefixes, so many for each row that reads
// one with others; one for each packed row; then those of own keys in several chunks:
// own_chunks for each packed row, or rows_per_seq for each request, whichever is less
// in all.  (A bound on a request's rows says little of a batch with one prompt among
// decodes, and the number of packed rows little where most of them are padding.)
__host__ __device__ inline int64_t shared_single(int64_t pre_rows, int64_t t) { return pre_rows + t; }
__host__ __device__ inline int64_t shared_own(int64_t T, int64_t pre_rows) { return pre_rows + T; }
// of request s, packed rows from c0 on, nc chunks: its first partial row, and how far a row's are from the last one's
__device__ __forceinline__ int64_t own_part(const TreeParams& p, const SharedArgs& h, int rows_per_seq, int s, int c0, int nc, int& step) {
  step = h.own_chunks ? h.own_chunks : nc;
  return shared_own(p.T, h.pre_rows) + (h.own_chunks ? (int64_t)c0 * step : (int64_t)s * rows_per_seq);
}
// How a call's keys are cut, as its plan has it if there is one.
__device__ __forceinline__ Chunking prefix_chunking(const SharedArgs& h) {
  return h.plan ? Chunking{__ldg(h.plan), __ldg(h.plan + 1)} : Chunking{h.pre.least, h.pre.most};
}
__device__ __forceinline__ int prefix_step(const SharedArgs& h, const Chunking& pre) { return h.plan ? pre.most : h.pre_chunks; }

// A group: its requests, its rows, the tokens of its prefix that are read together (0: none).
struct Group {
  int first, end, rows, prefix;
  __device__ __forceinline__ bool shares() const { return prefix > 0 && end - first > 1; }
};

__device__ __forceinline__ bool whole_blocks(const TreeParams& p, const SharedArgs& h, int n) { return quot(n, h.by_bs) * p.bs == n; }

// Request s: packed rows c0 .. c0 + q - 1, n keys, its group.  Returns whether it
// takes no part: inconsistent lengths, a prefix that is not whole blocks of its
// context, or a group that its first request does not name in the same words or
// whose rows do not hold the request's.
__device__ __forceinline__ bool shared_request(const TreeParams& p, const SharedArgs& h, int s, int& c0, int& q, int& n, Group& of) {
  const int32_t* g = h.groups + 3 * (int64_t)s;
  c0 = __ldg(p.cu_q + s);
  const int c1 = __ldg(p.cu_q + s + 1), g0 = __ldg(g), g1 = __ldg(g + 1);
  n = __ldg(p.seq_lens + s);
  of = Group{g0, g1, 0, __ldg(h.prefix + s * (int64_t)h.prefix_step)};
  q = c1 - c0;
  if (c0 < 0 || c1 < c0 || (int64_t)c1 > p.T || q > n || (int64_t)n > (int64_t)p.max_blocks * p.bs || q > p.max_nodes) return true;
  if (of.prefix == 0) return false;
  if (of.prefix < 0 || of.prefix > n - q || !whole_blocks(p, h, of.prefix) || g0 < 0 || g0 > s || g1 <= s || g1 > p.B) return true;
  const int32_t* f = h.groups + 3 * (int64_t)g0;
  const int t0 = __ldg(p.cu_q + g0), t1 = __ldg(p.cu_q + g1);
  of.rows = t1 - t0;
  return __ldg(f) != g0 || __ldg(f + 1) != g1 || __ldg(f + 2) != of.prefix || t0 < 0 || t0 > c0 || t1 < c1 || (int64_t)t1 > p.T ||
         of.rows > h.max_group;
}
// whether q rows, times the heads, fill a tile over a prefix
__device__ __forceinline__ bool fills_tile(const TreeParams& p, const SharedArgs& h, int q) { return (q * p.G) >> h.tile_log2 != 0; }
// own.least of request s, which has q rows and reads all of its keys alone
__device__ __forceinline__ int own_least(const TreeParams& p, const SharedArgs& h, int s, int q) {
  return h.plan ? __ldg(h.at + s) : fills_tile(p, h, q) ? h.alone_least : h.own.least;
}

// Prefixes are read for runs of neighbours that name the same group in the same
// words, found by a warp for 32 requests (s = from + lane) at a time: whether request s
// is the first of a run, whose packed rows are c0 .. c0 + q - 1, over n keys of the table of
// request `table`.  Mostly a run is its group, but nothing keeps groups that the
// caller made from overlapping, and a partial row must have one writer: its run is the
// only one that a request is in.  What shared_request() takes for a request of the run
// has passed all of this.
//
// (With groups taken at their word small calls took 0.1 to 0.3 us less.  What is rare
// stands apart, and no division stands here: a call's first item waits for this.)
static __device__ __noinline__ int run_end(const SharedArgs& h, int s, int lane, int first, int end, int prefix) {
  for (; s < end; s += 128) {
    uint32_t other[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int32_t* g = h.groups + 3 * (int64_t)min(s + 32 * k + lane, end - 1);
      other[k] = __ldg(g) != first || __ldg(g + 1) != end ||
                 __ldg(h.prefix + (int64_t)min(s + 32 * k + lane, end - 1) * h.prefix_step) != prefix;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      other[k] = __ballot_sync(0xffffffffu, other[k]);
      if (other[k]) return min(end, s + 32 * k + __ffs(other[k]) - 1);
    }
  }
  return end;
}
static __device__ __noinline__ bool named(const SharedArgs& h, int first, int end, int prefix) {
  const int32_t* g = h.groups + 3 * (int64_t)first;
  return __ldg(g) == first && __ldg(g + 1) == end && __ldg(g + 2) == prefix;
}
__device__ __forceinline__ int load_now(const int32_t* q) {  // where it stands, not where it is needed
  int x;
  asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(x) : "l"(q));
  return x;
}
__device__ __forceinline__ bool shared_run(const TreeParams& p, const SharedArgs& h, int from, int lane, int& c0, int& q, int& n, int& table) {
  const int s = from + lane;
  bool head = s < p.B;
  // this request's numbers, those of the one before, and of the one 32 on, in one trip
  const int32_t* g = h.groups + 3 * (int64_t)min(s, p.B - 1);
  const int32_t* const after = h.groups + 3 * (int64_t)min(s + 32, p.B - 1);
  const int32_t* const before = s > 0 ? g - 3 : g;
  const int32_t* const m = h.prefix + (int64_t)min(s, p.B - 1) * h.prefix_step;
  const int end = load_now(g + 1), a0 = load_now(after), a1 = load_now(after + 1), a2 = load_now(h.prefix + (int64_t)min(s + 32, p.B - 1) * h.prefix_step);
  table = __ldg(g);
  n = __ldg(m);
  c0 = __ldg(p.cu_q + min(s, p.B));
  const bool goes_on = head && s > 0 && __ldg(before) == table && __ldg(before + 1) == end && __ldg(m - (s > 0 ? h.prefix_step : 0)) == n;
  head = head && n > 0 && table >= 0 && (table == s || (table < s && !goes_on)) && end > s && end <= p.B && end - table > 1 &&
         (int64_t)n <= (int64_t)p.max_blocks * p.bs && whole_blocks(p, h, n);
  const int t1 = head ? __ldg(p.cu_q + end) : 0;
  // behind the run: the next request that names another group
  const uint32_t other = __ballot_sync(0xffffffffu, !goes_on) & ~((2u << lane) - 1u);
  int behind = min(end, other ? from + __ffs(other) - 1 : from + 32);
  // only the last run can go on behind these requests
  if (const uint32_t on = __ballot_sync(0xffffffffu, head && other == 0 && end > from + 32)) {
    const int o = 31 - __clz(on), of = __shfl_sync(0xffffffffu, table, o), l = __shfl_sync(0xffffffffu, end, o), of_n = __shfl_sync(0xffffffffu, n, o);
    const uint32_t off = __ballot_sync(0xffffffffu, a0 != of || a1 != l || a2 != of_n);
    int e = min(l, from + 32 + (off ? __ffs(off) - 1 : 32));
    if (off == 0 && l > from + 64) e = run_end(h, from + 64, lane, of, l, of_n);
    if (lane == o) behind = e;
  }
  if (!head) return false;
  const int upto = behind == end ? t1 : __ldg(p.cu_q + behind);
  int t0 = c0;
  if (table != s) {
    if (!named(h, table, end, n)) return false;
    t0 = __ldg(p.cu_q + table);
  }
  q = upto - c0;
  return t0 >= 0 && t0 <= c0 && upto > c0 && upto <= t1 && (int64_t)t1 <= p.T && t1 - t0 <= h.max_group;
}

}  // namespace pkv
