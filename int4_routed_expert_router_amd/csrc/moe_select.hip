// Scored, biased and group-limited expert choice (see include/moe_select.h
// for the definition).
//
// One wave per token.  Lane l holds experts l, l + 64, ... .  Scores and keys
// are fp64, so the order is the true one also where two keys differ by less
// than an fp32 rounding.
#include <hip/hip_runtime.h>

#include <cmath>

#include "moe_common.h"
#include "moe_kernels.h"
#include "moe_select.h"

namespace moe {
moe_status set_error(moe_status code, const char* fmt, ...);

namespace {

constexpr int kSelWaves = 4;   // tokens per workgroup

__device__ __forceinline__ double shfl_xor_f64(double v, int m) { return __shfl_xor(v, m, kWave); }
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += shfl_xor_f64(v, m);
  return v;
}
// larger double, larger key; -0 counts as +0; 0 is left free to mark "off"
__device__ __forceinline__ uint64_t order_key64(double d) {
  const uint64_t u = __builtin_bit_cast(uint64_t, d + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
// sum of the slices of one logit, in order (as the top-K kernel adds them)
__device__ __forceinline__ float logit_at(const SelectArgs& a, int t, int e) {
  const float* p = a.part + static_cast<size_t>(t) * a.ld + e;
  float z = p[0];
  for (int s = 1; s < a.n_part; ++s) z += p[s * a.pstride];
  return z;
}
__device__ __forceinline__ bool is_off(float z) { return !(z > -INFINITY); }   // -inf or NaN

// exp(z - m) of a softmax with maximum m; at an infinite maximum the limit
__device__ __forceinline__ double soft_ex(float z, float m) {
  return z == m ? 1.0 : exp(static_cast<double>(z) - static_cast<double>(m));
}

template <int kJ>
__device__ void select_token(const SelectArgs& a, int t, int lane, double* keys) {
  const double ninf = -INFINITY;
  float z[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) z[j] = lane + 64 * j < a.E ? logit_at(a, t, lane + 64 * j) : -INFINITY;
  if (a.logits != nullptr) {
#pragma unroll
    for (int j = 0; j < kJ; ++j)
      if (lane + 64 * j < a.E) a.logits[static_cast<size_t>(t) * (a.E + 1) + lane + 64 * j] = z[j];
  }
  if (lane == 0 && (a.gamma != nullptr || a.logits != nullptr)) {
    const float zg = logit_at(a, t, a.E);
    if (a.logits != nullptr) a.logits[static_cast<size_t>(t) * (a.E + 1) + a.E] = zg;
    if (a.gamma != nullptr) a.gamma[t] = 1.0f / (1.0f + expf(-zg));
  }
  float m = -INFINITY;
  double total = 1.0;
  if (a.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int j = 0; j < kJ; ++j) m = fmaxf(m, z[j]);
    m = wave_max(m);
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < kJ; ++j) s += is_off(z[j]) ? 0.0 : soft_ex(z[j], m);
    total = wave_sum_f64(s);
  }
  auto score = [&](float zz) {
    return a.score == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-static_cast<double>(zz))) : soft_ex(zz, m) / total;
  };
  uint64_t key[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int e = lane + 64 * j;
    double k = ninf;
    if (e < a.E && !is_off(z[j])) k = score(z[j]) + (a.bias != nullptr ? static_cast<double>(a.bias[e]) : 0.0);
    if (!(k > ninf)) k = ninf;
    if (e < a.E && a.top_groups < a.n_group) keys[e] = k;
    key[j] = k > ninf ? order_key64(k) : 0;
  }
  if (a.top_groups < a.n_group) {
    // lanes g * L .. g * L + L - 1 scan group g for its two largest keys
    const int per = a.E / a.n_group;
    int L = 64;
    while (L > 1 && 64 / L < a.n_group) L >>= 1;
    const int g = lane / L;
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    double b1 = ninf, b2 = ninf;
    if (g < a.n_group) {
      for (int i = lane % L; i < per; i += L) {
        const double k = keys[g * per + i];
        b2 = fmax(b2, fmin(b1, k));
        b1 = fmax(b1, k);
      }
    }
    for (int s = 1; s < L; s <<= 1) {
      const double o1 = shfl_xor_f64(b1, s), o2 = shfl_xor_f64(b2, s);
      b2 = fmax(fmin(b1, o1), fmax(b2, o2));
      b1 = fmax(b1, o1);
    }
    double rank = b1;
    if (a.group_top == 2 && b2 > ninf) rank += b2;
    uint64_t kept = 0;
    for (int c = 0; c < a.n_group; ++c) {   // group c is kept when fewer than top_groups are before it
      const double rc = __shfl(rank, c * L, kWave);
      const bool before = lane % L == 0 && g < a.n_group && (rank > rc || (rank == rc && g < c));
      if (__popcll(__ballot(before)) < a.top_groups) kept |= 1ull << c;
    }
    const float inv = 1.0f / static_cast<float>(per);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int e = lane + 64 * j;
      const int ge = static_cast<int>((static_cast<float>(e) + 0.5f) * inv);   // e / per, exact for e < 1024
      if (e < a.E && !((kept >> ge) & 1ull)) key[j] = 0;
    }
  }
  int my_e = -1;
  for (int k = 0; k < a.K; ++k) {
    uint64_t best = 0;
    int bj = 0;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const bool take = key[j] > best;
      best = take ? key[j] : best;
      bj = take ? j : bj;
    }
    const uint32_t bh = static_cast<uint32_t>(best >> 32), bl = static_cast<uint32_t>(best);
    const uint32_t mh = wave_max_u32_s(bh);
    if (mh == 0) break;   // no live expert is left (a live key's high word is never 0)
    const uint32_t ml = wave_max_u32_s(bh == mh ? bl : 0u);
    const bool cand = bh == mh && bl == ml;
    const int e = static_cast<int>(wave_min_u32_s(cand ? static_cast<uint32_t>(64 * bj + lane) : 0xFFFFFFFFu));
#pragma unroll
    for (int j = 0; j < kJ; ++j)
      if (e == 64 * j + lane) key[j] = 0;
    if (lane == k) my_e = e;
  }
  double sc = my_e >= 0 ? score(logit_at(a, t, my_e)) : 0.0;
  if (a.renorm) {
    const double s = wave_sum_f64(sc);
    sc = s > 0.0 ? sc / s : 0.0;
  }
  if (lane < a.K) {
    a.idx[static_cast<size_t>(t) * a.K + lane] = my_e;
    a.w[static_cast<size_t>(t) * a.K + lane] = static_cast<float>(sc * static_cast<double>(a.scale));
  }
}

template <int kJ>
__global__ __launch_bounds__(64 * kSelWaves) void k_select(SelectArgs a) {
  __shared__ double keys[kSelWaves][64 * kJ];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kSelWaves + wave;
  if (t < a.T) select_token<kJ>(a, t, lane, keys[wave]);
}

}  // namespace

hipError_t launch_select(const SelectArgs& a, hipStream_t s) {
  const dim3 grid((a.T + kSelWaves - 1) / kSelWaves), block(64 * kSelWaves);
  if (a.E <= 64) hipLaunchKernelGGL(k_select<1>, grid, block, 0, s, a);
  else if (a.E <= 128) hipLaunchKernelGGL(k_select<2>, grid, block, 0, s, a);
  else if (a.E <= 256) hipLaunchKernelGGL(k_select<4>, grid, block, 0, s, a);
  else if (a.E <= 512) hipLaunchKernelGGL(k_select<8>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(k_select<16>, grid, block, 0, s, a);
  return hipGetLastError();
}

moe_status check_select(const moe_select_desc* d, SelectArgs* a) {
  if (!d) return set_error(MOE_EINVAL, "select desc is NULL");
  const int E = d->n_experts, K = d->top_k;
  const int ng = d->n_group ? d->n_group : 1, tg = d->top_groups ? d->top_groups : ng;
  const int gt = d->group_top ? d->group_top : 1;
  if (E < 1 || E > kMaxExperts) return set_error(MOE_ESHAPE, "n_experts=%d must be in [1, %d]", E, kMaxExperts);
  if (K < 1 || K > E || K > kMaxTopK)
    return set_error(MOE_ESHAPE, "top_k=%d must be in [1, min(E, %d)]", K, kMaxTopK);
  if (d->score != MOE_SCORE_SOFTMAX && d->score != MOE_SCORE_SIGMOID)
    return set_error(MOE_EINVAL, "score=%d is not a MOE_SCORE_*", d->score);
  if (ng < 1 || ng > 64 || E % ng) return set_error(MOE_ESHAPE, "n_group=%d must be in [1, 64] and divide n_experts=%d", ng, E);
  if (tg < 1 || tg > ng || tg * (E / ng) < K)
    return set_error(MOE_ESHAPE, "top_groups=%d must be in [1, n_group=%d] and hold top_k=%d experts", tg, ng, K);
  if (gt != 1 && gt != 2) return set_error(MOE_EINVAL, "group_top=%d must be 1 or 2", gt);
  if (d->renorm != 0 && d->renorm != 1) return set_error(MOE_EINVAL, "renorm=%d must be 0 or 1", d->renorm);
  if (!std::isfinite(d->scale)) return set_error(MOE_EINVAL, "scale must be finite");
  *a = SelectArgs{};
  a->E = E;
  a->K = K;
  a->score = d->score;
  a->n_group = ng;
  a->top_groups = tg;
  a->group_top = gt;
  a->renorm = d->renorm;
  a->scale = d->scale;
  return MOE_OK;
}

}  // namespace moe

extern "C" moe_status moe_select(const moe_select_desc* d, const float* logits, int64_t stride, const float* bias,
                                 int32_t T, int32_t* topk_idx, float* topk_w, float* shared_gate, moe_stream stream) {
  using moe::set_error;
  moe::SelectArgs a;
  const moe_status st = moe::check_select(d, &a);
  if (st) return st;
  if (T < 0) return set_error(MOE_ESHAPE, "n_tokens=%d < 0", T);
  const int64_t need = shared_gate ? a.E + 1 : a.E;
  if (stride < need) return set_error(MOE_ESHAPE, "logits_stride=%lld < %lld", (long long)stride, (long long)need);
  if (T == 0) return set_error(MOE_OK, "");
  if (!logits || !topk_idx || !topk_w) return set_error(MOE_EINVAL, "logits, topk_idx and topk_w are required");
  a.part = logits;
  a.n_part = 1;
  a.ld = stride;
  a.bias = bias;
  a.T = T;
  a.idx = topk_idx;
  a.w = topk_w;
  a.gamma = shared_gate;
  const hipError_t e = moe::launch_select(a, reinterpret_cast<hipStream_t>(stream));
  if (e != hipSuccess) return set_error(MOE_EHIP, "select kernel launch: %s", hipGetErrorString(e));
  return set_error(MOE_OK, "");
}
