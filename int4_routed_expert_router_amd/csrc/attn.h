// What the attention kernels and their entry points share (see include/moe_attn.h).
#pragma once
#include <hip/hip_runtime.h>

#include "moe_attn.h"
#include "moe_common.h"

namespace moe {

struct AttnArgs {
  const uint16_t *k, *v;        // cache
  const int32_t *table, *length, *off;
  const uint16_t *q, *gate;     // gate or nullptr
  int32_t q_ts, q_hs, g_ts, g_hs;   // token and head strides, elements
  uint16_t* o;
  float scale;
  int B, N, Hq, Hk, page_log, n_pages, max_pages;
};

struct AppendArgs {
  uint16_t *kc, *vc;
  const int32_t *table, *length, *off;   // off nullptr: token t is sequence t's only one
  const uint16_t *k, *v, *q;             // q or nullptr
  int32_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs;
  uint16_t* q_out;
  const float *q_norm, *k_norm;
  const double* freq;
  float eps;
  int rot, B, N, Hq, Hk, page_log, n_pages, max_pages;
};

// Two values rounded to nearest even, the first in the low half.
template <int ACT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (ACT == 2) return __builtin_bit_cast(uint32_t, bf16x2_t{static_cast<__bf16>(a), static_cast<__bf16>(b)});
  else return __builtin_bit_cast(uint32_t, f16x2_t{static_cast<_Float16>(a), static_cast<_Float16>(b)});
}

// 16-bit matrix products with fp32 accumulators.
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
template <int ACT>
__device__ __forceinline__ f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
  if constexpr (ACT == 2)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

template <int ACT>
__device__ __forceinline__ f32x16_t mfma32(uint4 a, uint4 b, f32x16_t c) {
  if constexpr (ACT == 2)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// Maximum and sum over the two lanes l, l ^ 32.
__device__ __forceinline__ float pair_max(float v) {
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_int(v), __float_as_int(v), false, false);
  return fmaxf(__int_as_float(b[0]), __int_as_float(b[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_int(v), __float_as_int(v), false, false);
  return __int_as_float(b[0]) + __int_as_float(b[1]);
}
// Maximum and sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48; identical bits in each.
__device__ __forceinline__ float quad_max(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_int(v), __float_as_int(v), false, false);
  v = fmaxf(__int_as_float(a[0]), __int_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_int(v), __float_as_int(v), false, false);
  return fmaxf(__int_as_float(b[0]), __int_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_int(v), __float_as_int(v), false, false);
  v = __int_as_float(a[0]) + __int_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_int(v), __float_as_int(v), false, false);
  return __int_as_float(b[0]) + __int_as_float(b[1]);
}

constexpr float kLog2e = 1.44269504f;
// Softmax weights in the decode kernel are 2^kShift exp(z - max): fp16 keeps its
// full precision down to 2^-14, so a shift of 7 leaves 2^-21 of the largest weight.
template <int ACT>
constexpr float kShift = ACT == 2 ? 0.0f : 7.0f;
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// tokens of sequence b in the cache, the new ones included
__device__ __forceinline__ int seq_length(const int32_t* length, int b, int max_pages, int page_log) {
  return min(max(length[b], 0), max_pages << page_log);
}

// First element of head h's row of token t.
__device__ __forceinline__ int64_t row_at(int t, int32_t ts, int h, int32_t hs) {
  return static_cast<int64_t>(t) * ts + static_cast<int64_t>(h) * hs;
}

// Four neighbouring normalised values of a row and head with their gates, if
// there are any; a row that sees no position is 0 whatever its gate is.
__device__ __forceinline__ uint2 gates_of(const AttnArgs& a, int t, int h, int d) {
  return a.gate ? *reinterpret_cast<const uint2*>(a.gate + row_at(t, a.g_ts, h, a.g_hs) + d) : make_uint2(0, 0);
}
template <int ACT>
__device__ __forceinline__ void store_row(const AttnArgs& a, int t, int h, int D, int d, f32x4_t v, uint2 g, bool none) {
  if (a.gate) {
    v[0] *= sigmoid(act_to_f32<ACT>(g.x & 0xFFFFu)), v[1] *= sigmoid(act_to_f32<ACT>(g.x >> 16));
    v[2] *= sigmoid(act_to_f32<ACT>(g.y & 0xFFFFu)), v[3] *= sigmoid(act_to_f32<ACT>(g.y >> 16));
    if (none) v = f32x4_t{0, 0, 0, 0};
  }
  *reinterpret_cast<uint2*>(a.o + (static_cast<int64_t>(t) * a.Hq + h) * D + d) =
      make_uint2(pack2<ACT>(v[0], v[1]), pack2<ACT>(v[2], v[3]));
}

// Rows [begin, end) of sequence b, with the offsets forced into [0, N].
__device__ __forceinline__ void seq_rows(const int32_t* off, int b, int N, int& begin, int& end) {
  begin = min(max(off[b], 0), N);
  end = max(min(max(off[b + 1], 0), N), begin);
}

// The sequence that owns row t (wave-uniform; B where none does): a search
// that takes 64 offsets at a time, one to a lane, so that up to 64 sequences
// cost one load and 4096 two.  The answer is checked against the range that it
// names, so offsets in any order only leave rows without an owner.
__device__ __forceinline__ int seq_of_row(const int32_t* off, int B, int N, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = B;   // candidates lo .. lo + n - 1: the last b with off[b] <= t and b < B that owns rows
  while (n > 64) {
    const int step = (n + 63) / 64, i = lo + lane * step;
    const uint64_t le = __ballot(i < lo + n && off[min(i, B)] <= t);
    if (le == 0) return B;
    const int last = 63 - __builtin_clzll(le);
    const int from = lo + last * step;
    n = min(step, lo + n - from);
    lo = from;
  }
  const uint64_t le = __ballot(lane < n && off[min(lo + lane, B)] <= t);
  if (le == 0) return B;
  const int b = lo + 63 - __builtin_clzll(le);
  int begin, end;
  seq_rows(off, b, N, begin, end);
  return t >= begin && t < end ? b : B;
}

hipError_t launch_kv_append(int act, int d, const AppendArgs& a, hipStream_t s);
bool attn_prefill_fits(const moe_attn_desc* d, int N);   // whether a grid holds the call
size_t attn_decode_bytes(const moe_attn_desc* d);
size_t attn_prefill_bytes(const moe_attn_desc* d, int N);
hipError_t launch_attn_decode(int act, int d, const AttnArgs& a, void* ws, hipStream_t s);
hipError_t launch_attn_prefill(int act, int d, const AttnArgs& a, void* ws, hipStream_t s);

}  // namespace moe
