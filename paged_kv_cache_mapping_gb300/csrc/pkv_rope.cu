// pkv_rope.cu -- rotary position embedding fused with the slot-mapped cache
// append.
//
// Mathematics: pair i of a head's first rot_dim elements (a, b) turns by the
// angle position * f_i:  (a cos - b sin, a sin + b cos).  Angles are kept as
// fractions of a turn in 64-bit fixed point: turns_i = f_i / (2 pi) * 2^64
// mod 2^64, and the low 64 bits of position * turns_i are the angle modulo
// one turn, exactly, for any integer position (f_i itself has the 53 bits that the
// host worked it out in: a position p turns it by an error of about p 2^-53 f_i);
// the upper 32 of them, as a signed number, lie in [-1/2, 1/2) turn with an error
// of 2^-33 turn, and 24 of them enter sincospif, which never sees a large argument
// and needs no fp64.  The rotation
// itself is fp32, rounded once to the destination's type.
//
// Bound: memory.  Each row of q, k and v is read once and written once; a
// decode step's few rows are bound by latency.  One CTA takes one token (or a
// part of its rows, when there are few tokens, so that the whole GPU works):
// its threads issue their first loads, then compute the token's cos / sin pairs
// into shared memory (shared by all Hq + Hkv heads), and rotate after the
// barrier, so that the sine's latency hides under the loads'.  A thread holds
// one unit at a time: three in flight took 79 registers instead of 39 and left
// six CTAs on an SM, which cost more than the loads' latency saved (8,192 tokens
// of 32 + 8 + 8 heads at D 128: 40 us with three, 34 with one; with 64, 192 and
// 256 threads 36, 39 and 51).
// Measured: those 8,192 bf16 tokens 33.7 us (6.0 TB/s of 201 MB, 88 % of a plain
// copy's rate); a decode step of 64 tokens 2.4 us; 777 drafted tokens of 20 + 5 +
// 5 heads at D 64 into e4m3 caches 3.5 us.
#include <math.h>

#include "pkv_kernels.h"

namespace pkv {

namespace {

template <typename SrcT> struct VecOf;
template <> struct VecOf<float> { static constexpr int n = 4; };
template <> struct VecOf<__nv_bfloat16> { static constexpr int n = 8; };

template <int VE> __device__ __forceinline__ void unpack(const uint4& v, float (&x)[VE]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (VE == 8) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    } else {
      x[i] = __uint_as_float(w[i]);
    }
  }
}

// VE elements to a destination of the source's type
template <int VE> __device__ __forceinline__ uint4 pack_same(const float (&x)[VE]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (VE == 8) {
      w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    } else {
      w[i] = __float_as_uint(x[i]);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int VE> __device__ __forceinline__ void store_codes(uint8_t* dst, const float (&x)[VE], float inv) {
  uint32_t w[VE / 4];
#pragma unroll
  for (int i = 0; i < VE / 4; ++i) {
    const uint32_t a = f32x2_to_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv);
    const uint32_t b = f32x2_to_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv);
    w[i] = a | (b << 16);
  }
  if constexpr (VE == 8) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint32_t*>(dst) = w[0];
  }
}

// cos and sin of pair i at a position, times the amplitude
__device__ __forceinline__ float2 rope_cs(unsigned long long pos, unsigned long long turns, float amp) {
  const unsigned long long x = pos * turns;                        // turns modulo 1, 2^-64 units
  const int32_t half_turns = static_cast<int32_t>(x >> 32);        // [-1/2, 1/2) turn, 2^-32 units
  float s, c;
  sincospif(static_cast<float>(half_turns) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
  return make_float2(c * amp, s * amp);
}

// A unit of a row: two vectors of VE elements.  Rotated part, half layout:
// elements VE c .. and rot/2 + VE c ..; interleaved: 2 VE c .. and
// 2 VE c + VE ..; pass-through part (and v rows): the vectors two by two.
// The second vector of an interleaved or pass-through unit may lie past the
// part's end (e1 < 0).
struct Unit {
  int row;      // 0 .. Hq - 1 q, .. Hq + Hkv - 1 k, .. Hq + 2 Hkv - 1 v
  int e0, e1;   // element offsets of the two vectors
  int rotated;
};

template <int VE>
__device__ __forceinline__ Unit unit_of(int u, const RopeParams& p) {
  Unit r;
  const int per_rot = p.rot_units + p.pass_units;
  const int n_rot = (p.Hq + p.Hkv) * per_rot;
  if (u < n_rot) {
    r.row = quot(u, p.by_row);
    const int c = u - r.row * per_rot;
    r.rotated = c < p.rot_units;
    if (r.rotated) {
      if (p.rope.interleaved) {
        r.e0 = 2 * VE * c;
        r.e1 = r.e0 + VE < p.rope.rot_dim ? r.e0 + VE : -1;
      } else {
        r.e0 = VE * c;
        r.e1 = p.rope.rot_dim / 2 + VE * c;
      }
    } else {
      r.e0 = p.rope.rot_dim + 2 * VE * (c - p.rot_units);
      r.e1 = r.e0 + VE < p.D ? r.e0 + VE : -1;
    }
  } else {
    const int w = u - n_rot;
    const int vr = quot(w, p.by_v);
    r.row = p.Hq + p.Hkv + vr;
    r.e0 = 2 * VE * (w - vr * p.v_units);
    r.e1 = r.e0 + VE < p.D ? r.e0 + VE : -1;
    r.rotated = 0;
  }
  return r;
}

template <typename SrcT>
__device__ __forceinline__ const SrcT* src_row(const RopeParams& p, int64_t t, int row) {
  if (row < p.Hq) return static_cast<const SrcT*>(p.q) + t * p.q_st + (int64_t)row * p.q_sh;
  row -= p.Hq;
  if (row < p.Hkv) return static_cast<const SrcT*>(p.k) + t * p.k_st + (int64_t)row * p.k_sh;
  row -= p.Hkv;
  return static_cast<const SrcT*>(p.v) + t * p.v_st + (int64_t)row * p.v_sh;
}

template <typename SrcT, bool kFp8, int VE>
__device__ __forceinline__ void put(const RopeParams& p, int64_t t, int64_t slot, int row, int e, const float (&x)[VE]) {
  if (row < p.Hq) {
    *reinterpret_cast<uint4*>(static_cast<SrcT*>(p.q_out) + t * p.o_st + (int64_t)row * p.o_sh + e) = pack_same<VE>(x);
    return;
  }
  if (slot < 0) return;
  const bool is_v = row >= p.Hq + p.Hkv;
  const int h = row - p.Hq - (is_v ? p.Hkv : 0);
  const int64_t at = (slot * p.Hkv + h) * p.D + e;
  if constexpr (kFp8) {
    store_codes<VE>(static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + at, x, is_v ? p.v_inv_scale : p.k_inv_scale);
  } else {
    *reinterpret_cast<uint4*>(static_cast<SrcT*>(is_v ? p.v_cache : p.k_cache) + at) = pack_same<VE>(x);
  }
}

constexpr int kRopeThreads = 128;

// Slots and positions are read as their caller's integer type.
template <typename SlotT>
__device__ __forceinline__ long long index_at(const void* a, int64_t t) {
  return static_cast<long long>(static_cast<const SlotT*>(a)[t]);
}

// A token's slot, -1 where nothing is to be written.
__device__ __forceinline__ int64_t token_slot(const RopeParams& p, int64_t t, bool report) {
  int64_t slot = p.slots_i64 ? index_at<int64_t>(p.slots, t) : index_at<int32_t>(p.slots, t);
  if (slot >= p.num_slots) {
    if (report) atomicOr(p.err, kErrSlotRange);
    slot = -1;
  }
  return slot;
}

// Place of pair i in the vector kernel's table: two pairs of padding after every
// eight, so that the threads of a row's units, eight pairs (VE 8) apart, read 16
// bytes each from banks of their own.
__device__ __forceinline__ int place(int i) { return i + (i >> 3) * 2; }

template <bool kPadded>
__device__ __forceinline__ void fill_table(const RopeParams& p, int64_t t, float2* cs) {
  const unsigned long long pos = static_cast<unsigned long long>(
      p.pos_i64 ? index_at<int64_t>(p.positions, t) : index_at<int32_t>(p.positions, t));
  for (int i = threadIdx.x; i < p.rope.rot_dim / 2; i += kRopeThreads)
    cs[kPadded ? place(i) : i] = rope_cs(pos, p.rope.turns[i], p.rope.amplitude);
}

// VE / 2 neighbouring pairs by their table entries (two to 16 bytes)
template <int VE> __device__ __forceinline__ void turn_pairs(float (&x)[VE], const float2* table) {
  const float4* c0 = reinterpret_cast<const float4*>(table);
#pragma unroll
  for (int i = 0; i < VE; i += 4) {
    const float4 c = c0[i / 4];
    const float f0 = x[i], g0 = x[i + 1], f1 = x[i + 2], g1 = x[i + 3];
    x[i] = f0 * c.x - g0 * c.y;
    x[i + 1] = f0 * c.y + g0 * c.x;
    x[i + 2] = f1 * c.z - g1 * c.w;
    x[i + 3] = f1 * c.w + g1 * c.z;
  }
}

// grid: (tokens, parts of a token's units)
template <typename SrcT, bool kFp8>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeParams p) {
  constexpr int VE = VecOf<SrcT>::n;
  __shared__ __align__(16) float2 cs[PKV_ROPE_MAX_PAIRS / 8 * 10];
  launch_dependents();
  grid_dep_wait();
  const int64_t t = blockIdx.x;
  const int u0 = blockIdx.y * p.units_per_part;
  const int u1 = min(u0 + p.units_per_part, p.units);
  bool table = false;
  int64_t slot = -1;
  // the first unit's loads are on their way while the table is made
  for (int u = u0 + threadIdx.x;; u += kRopeThreads) {
    const bool some = u < u1;
    Unit un{};
    uint4 a{}, b{};
    if (some) {
      un = unit_of<VE>(u, p);
      const SrcT* s = src_row<SrcT>(p, t, un.row);
      a = *reinterpret_cast<const uint4*>(s + un.e0);
      if (un.e1 >= 0) b = *reinterpret_cast<const uint4*>(s + un.e1);
    }
    if (!table) {
      slot = token_slot(p, t, threadIdx.x == 0 && blockIdx.y == 0);
      fill_table<true>(p, t, cs);
      __syncthreads();
      table = true;
    }
    if (!some) break;
    float x[VE], y[VE];
    unpack<VE>(a, x);
    unpack<VE>(b, y);
    if (un.rotated) {
      if (p.rope.interleaved) {
        turn_pairs<VE>(x, cs + place(un.e0 / 2));
        if (un.e1 >= 0) turn_pairs<VE>(y, cs + place(un.e1 / 2));
      } else {
        const float4* c0 = reinterpret_cast<const float4*>(cs + place(un.e0));
#pragma unroll
        for (int i = 0; i < VE; i += 2) {
          const float4 c = c0[i / 2];
          const float f0 = x[i], g0 = y[i], f1 = x[i + 1], g1 = y[i + 1];
          x[i] = f0 * c.x - g0 * c.y;
          y[i] = f0 * c.y + g0 * c.x;
          x[i + 1] = f1 * c.z - g1 * c.w;
          y[i + 1] = f1 * c.w + g1 * c.z;
        }
      }
    }
    put<SrcT, kFp8, VE>(p, t, slot, un.row, un.e0, x);
    if (un.e1 >= 0) put<SrcT, kFp8, VE>(p, t, slot, un.row, un.e1, y);
  }
}

template <typename SrcT, bool kFp8>
__device__ __forceinline__ void put1(const RopeParams& p, int64_t t, int64_t slot, int row, int e, float x) {
  if (row < p.Hq) {
    store1(static_cast<SrcT*>(p.q_out) + t * p.o_st + (int64_t)row * p.o_sh + e, x);
    return;
  }
  if (slot < 0) return;
  const bool is_v = row >= p.Hq + p.Hkv;
  const int h = row - p.Hq - (is_v ? p.Hkv : 0);
  const int64_t at = (slot * p.Hkv + h) * p.D + e;
  if constexpr (kFp8) {
    static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache)[at] =
        static_cast<uint8_t>(f32x2_to_e4m3x2(x * (is_v ? p.v_inv_scale : p.k_inv_scale), 0.f));
  } else {
    store1(static_cast<SrcT*>(is_v ? p.v_cache : p.k_cache) + at, x);
  }
}

// Rotated parts that do not fall into whole 16-byte vectors (rot_dim / 2, or
// rot_dim when interleaved, not a multiple of the vector): one pair, or two
// elements of the rest, per thread.
template <typename SrcT, bool kFp8>
__global__ void __launch_bounds__(kRopeThreads) rope_append_pairs_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs[PKV_ROPE_MAX_PAIRS];
  launch_dependents();
  grid_dep_wait();
  const int64_t t = blockIdx.x;
  const int64_t slot = token_slot(p, t, threadIdx.x == 0 && blockIdx.y == 0);
  fill_table<false>(p, t, cs);
  __syncthreads();
  const int half = p.rope.rot_dim / 2, per = p.D / 2;
  const int u1 = min((int)(blockIdx.y + 1) * p.units_per_part, p.units);
  for (int u = blockIdx.y * p.units_per_part + threadIdx.x; u < u1; u += kRopeThreads) {
    const int row = quot(u, p.by_row), i = u - row * per;
    const bool rotated = i < half && row < p.Hq + p.Hkv;
    const int e0 = rotated && !p.rope.interleaved ? i : 2 * i;
    const int e1 = rotated && !p.rope.interleaved ? i + half : 2 * i + 1;
    const SrcT* s = src_row<SrcT>(p, t, row);
    const float a = static_cast<float>(s[e0]), b = static_cast<float>(s[e1]);
    float x = a, y = b;
    if (rotated) {
      const float2 c = cs[i];
      x = a * c.x - b * c.y;
      y = a * c.y + b * c.x;
    }
    put1<SrcT, kFp8>(p, t, slot, row, e0, x);
    put1<SrcT, kFp8>(p, t, slot, row, e1, y);
  }
}

template <typename SrcT, bool kFp8>
cudaError_t launch_t(RopeParams p, int num_sms, cudaStream_t st) {
  constexpr int VE = VecOf<SrcT>::n;
  const int rot = p.rope.rot_dim;
  const bool vec = (p.rope.interleaved ? rot : rot / 2) % VE == 0;
  if (vec) {
    const int half_units = p.rope.interleaved ? (rot / VE + 1) / 2 : rot / 2 / VE;
    p.rot_units = half_units;
    p.pass_units = ((p.D - rot) / VE + 1) / 2;
    p.v_units = (p.D / VE + 1) / 2;
    p.units = (p.Hq + p.Hkv) * (p.rot_units + p.pass_units) + p.Hkv * p.v_units;
    p.by_row = fast_div(p.rot_units + p.pass_units);
    p.by_v = fast_div(p.v_units);
  } else {
    p.units = (p.Hq + 2 * p.Hkv) * (p.D / 2);
    p.by_row = fast_div(p.D / 2);
  }
  // few tokens: cut a token's units into parts of at least one per thread,
  // so that about two CTAs per SM share the rows
  int64_t parts = p.T >= 2 * num_sms ? 1 : (2 * num_sms + p.T - 1) / p.T;
  const int most = (p.units + kRopeThreads - 1) / kRopeThreads;
  if (parts > most) parts = most;
  p.units_per_part = (p.units + (int)parts - 1) / (int)parts;
  parts = (p.units + p.units_per_part - 1) / p.units_per_part;
  const dim3 grid((unsigned)p.T, (unsigned)parts);
  if (vec) return launch_ex(rope_append_kernel<SrcT, kFp8>, grid, dim3(kRopeThreads), 0, st, true, p);
  return launch_ex(rope_append_pairs_kernel<SrcT, kFp8>, grid, dim3(kRopeThreads), 0, st, true, p);
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, int src_kind, bool fp8, int num_sms, cudaStream_t st) {
  if (p.T == 0) return cudaSuccess;
  if (src_kind == 0) return fp8 ? launch_t<float, true>(p, num_sms, st) : launch_t<float, false>(p, num_sms, st);
  return fp8 ? launch_t<__nv_bfloat16, true>(p, num_sms, st) : launch_t<__nv_bfloat16, false>(p, num_sms, st);
}

}  // namespace pkv
