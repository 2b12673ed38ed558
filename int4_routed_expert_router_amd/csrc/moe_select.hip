// Scored, biased and group-limited expert choice (see include/moe_select.h
// for the definition).
//
// One wave per token.  Lane l holds experts l, l + 64, ... .  The order is that
// of fp64 keys, but a wave first takes fp32 keys, whose error is bounded.  Its
// rounds go on past rank K until a key is below the one before by more than the
// bound: what came before holds the first K.  Where two of those candidates
// are nearer than the bound, their fp64 keys (one per lane) put them in order.
// Only where the fp32 keys leave open which groups take part, or where 64
// candidates lie too near each other, does the wave start over in fp64.
//
// One token, 10 of 512: 6.2 us, bound by latency: the launch, the loads, then
// 11 rounds that each take a maximum over the wave, and the fp64 scores of the
// chosen.  64 tokens, 8 of 256 in 4 of 8 groups: 7.8 us.  8191 such tokens: 17.2
// us, 8.9 MB at 0.5 TB/s, bound by the vector instructions of the rounds (four
// tokens to a wave, 16 lanes each, were 19.9 us against 21.7 for this form when
// all keys were fp64, and more than twice as long for few tokens; with the fp32
// keys, or from a token count on, that form has not been tried).  Above 256
// experts some scalar registers are spilled to lanes of vector registers (14 up
// to 512, 70 up to 1024).
#include <hip/hip_runtime.h>

#include <cmath>

#include "moe_common.h"
#include "moe_kernels.h"
#include "moe_select.h"
#include "moe_topk.h"

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

// The two largest of keys g per + i, i = first, first + L, ... < per (-inf for
// g >= n_group); four reads are in flight at a time.
template <class F>
__device__ __forceinline__ void two_largest(const F* keys, int per, int g, int first, int L, int n_group, F& b1, F& b2) {
  const F ninf = -INFINITY;
  b1 = b2 = ninf;
  const F* mine = keys + min(g, n_group - 1) * per;
  for (int i = first; i < per; i += 4 * L) {
    F k[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) k[u] = mine[min(i + u * L, per - 1)];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const F v = g < n_group && i + u * L < per ? k[u] : ninf;
      b2 = fmax(b2, fmin(b1, v));
      b1 = fmax(b1, v);
    }
  }
}
// Groups: lanes g L .. g L + L - 1 scan group g's keys (in LDS) for its two
// largest; every lane of group g returns its rank.
template <class F>
__device__ __forceinline__ F group_rank(const SelectArgs& a, const F* keys, int lane, int L) {
  F b1, b2;
  two_largest(keys, a.E / a.n_group, lane / L, lane % L, L, a.n_group, b1, b2);
  const F ninf = -INFINITY;
  for (int s = 1; s < L; s <<= 1) {
    const F o1 = __shfl_xor(b1, s, kWave), o2 = __shfl_xor(b2, s, kWave);
    b2 = fmax(fmin(b1, o1), fmax(b2, o2));
    b1 = fmax(b1, o1);
  }
  return a.group_top == 2 && b2 > ninf ? b1 + b2 : b1;
}
// Bit c: group c is kept (fewer than top_groups groups come before it).
template <class F>
__device__ __forceinline__ uint64_t kept_groups(const SelectArgs& a, F rank, int lane, int L) {
  const int g = lane / L;
  uint64_t kept = 0;
  for (int c0 = 0; c0 < a.n_group; c0 += 4) {   // four ranks fetched at a time
    F rc[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) rc[u] = __shfl(rank, min(c0 + u, a.n_group - 1) * L, kWave);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u;
      const bool before = lane % L == 0 && g < a.n_group && (rank > rc[u] || (rank == rc[u] && g < c));
      if (c < a.n_group && __popcll(__ballot(before)) < a.top_groups) kept |= 1ull << c;
    }
  }
  return kept;
}
__device__ __forceinline__ int group_of(int e, float inv_per) {   // e / per, exact for e < 1024
  return static_cast<int>((static_cast<float>(e) + 0.5f) * inv_per);
}

struct Softmax {
  float m;        // maximum of the logits
  double total;   // sum of exp(z - m) over the live experts
};
template <int kJ>
__device__ __forceinline__ double total64(const float (&z)[kJ], float m) {
  double s = 0.0;
#pragma unroll
  for (int j = 0; j < kJ; ++j) s += is_off(z[j]) ? 0.0 : soft_ex(z[j], m);
  return wave_sum_f64(s);
}
__device__ __forceinline__ double score64(const SelectArgs& a, float z, const Softmax& sm) {
  return a.score == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-static_cast<double>(z))) : soft_ex(z, sm.m) / sm.total;
}

// The choice in fp64: lane k returns the expert of rank k, or -1.
template <int kJ>
__device__ __forceinline__ int choose64(const SelectArgs& a, const float (&z)[kJ], const Softmax& sm, int lane, int L,
                                        double* keys) {
  const double ninf = -INFINITY;
  const bool grouped = a.top_groups < a.n_group;
  uint64_t key[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int e = lane + 64 * j;
    double k = ninf;
    if (e < a.E && !is_off(z[j])) k = score64(a, z[j], sm) + (a.bias != nullptr ? static_cast<double>(a.bias[e]) : 0.0);
    if (!(k > ninf)) k = ninf;
    if (e < a.E && grouped) keys[e] = k;
    key[j] = k > ninf ? order_key64(k) : 0;
  }
  if (grouped) {
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    const uint64_t kept = kept_groups(a, group_rank(a, keys, lane, L), lane, L);
    const float inv = 1.0f / static_cast<float>(a.E / a.n_group);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int e = lane + 64 * j;
      if (e < a.E && !((kept >> group_of(e, inv)) & 1ull)) key[j] = 0;
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
  return my_e;
}

// Candidates from fp32 keys: lane c < n has the expert of fp32 rank c, and the
// fp64 choice lies among them.  ordered: the first K are its ranks.
struct Candidates {
  int e, n;
  bool open;      // not even that is sure
  bool ordered;
};
// Error of an fp32 key.  exp is the hardware's exp2 (1 ulp) of a product with
// log2 e: z - m (half an ulp), the constant and the product are off by 2.4 x
// 2^-24 of up to 150 (beyond, the score is 0 in fp32 and below 2^-149 in fp64),
// which is a relative error under 2^-15.9 of the exponential; the sum, the
// hardware's reciprocal (1 ulp) and the softmax's sum (16 + 6 additions) add
// 2^-19.  So a score above fp32's subnormals is within 2^-15.7 of itself; a
// sigmoid is within 2^-21.5 and a softmax within 2^-18 of its largest (the
// product's error times |d| e^-|d| < 0.4); adding the bias rounds by 2^-24 of
// the key.  Two keys are in order for sure when they differ by more than twice
// that; two ranks of up to two keys, when by more than four times that at the
// largest key's magnitude.
struct Margin {   // two keys of magnitude up to v are in order when they differ by more than rel v + cap
  float rel, cap;
};
__device__ __forceinline__ Margin margin(const SelectArgs& a, float largest_score) {
  if (a.bias == nullptr) return {0x1p-14f, 0x1p-120f};
  return {0x1p-22f, a.score == MOE_SCORE_SIGMOID ? 0x1p-20f : 0x1p-17f * largest_score};
}
template <int kJ>
__device__ __forceinline__ Candidates choose32(const SelectArgs& a, const float (&z)[kJ], float m, int lane, int L,
                                               float* keys) {
  const float ninf = -INFINITY;
  const bool grouped = a.top_groups < a.n_group, sigmoid = a.score == MOE_SCORE_SIGMOID;
  constexpr float kLog2e = 1.44269504f;
  float s[kJ], total = 0.0f;
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    s[j] = sigmoid ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z[j]))
                   : (z[j] == m ? 1.0f : __builtin_amdgcn_exp2f(kLog2e * (z[j] - m)));
    total += is_off(z[j]) ? 0.0f : s[j];
  }
  const float inv_total = sigmoid ? 1.0f : __builtin_amdgcn_rcpf(wave_sum(total));
  uint32_t hi[kJ], lo[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int e = lane + 64 * j;
    float k = ninf;
    if (e < a.E && !is_off(z[j])) k = s[j] * inv_total + (a.bias != nullptr ? a.bias[e] : 0.0f);
    if (!(k > ninf)) k = ninf;
    if (e < a.E && grouped) keys[e] = k;
    hi[j] = k > ninf ? order_key(k) : 0u;
    lo[j] = kJ - 1 - j;
  }
  const Margin mg = margin(a, inv_total);
  Candidates r = {-1, 0, false, true};
  if (grouped) {
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    float big = 0.0f;
#pragma unroll
    for (int j = 0; j < kJ; ++j) big = hi[j] != 0u ? fmaxf(big, fabsf(key_value(hi[j]))) : big;
    big = wave_max(big);
    const float rank = group_rank(a, keys, lane, L);
    const uint64_t kept = kept_groups(a, rank, lane, L);
    const bool head = lane % L == 0 && lane / L < a.n_group, in = (kept >> (lane / L)) & 1ull;
    const float least = -wave_max(head && in ? -rank : ninf), next = wave_max(head && !in ? rank : ninf);
    // groups without a live expert (-inf) cannot matter, on either side; sums
    // of two keys near fp32's end might overflow
    r.open = next > ninf && !(least - next > 2.0f * fmaf(mg.rel, big, mg.cap));
    r.open = r.open || !(big < 1e38f);
    const float inv = 1.0f / static_cast<float>(a.E / a.n_group);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int e = lane + 64 * j;
      if (e < a.E && !((kept >> group_of(e, inv)) & 1ull)) hi[j] = 0u;
    }
  }
  oddeven_merge_sort<kJ>([&](int x, int y) {
    const bool swap = hi[y] > hi[x] || (hi[y] == hi[x] && lo[y] > lo[x]);
    const uint32_t hx = hi[x], lx = lo[x];
    hi[x] = swap ? hi[y] : hx;
    lo[x] = swap ? lo[y] : lx;
    hi[y] = swap ? hx : hi[y];
    lo[y] = swap ? lx : lo[y];
  });
  TopkList<kJ> list;
  list.lo = list.lo_hi8 = 0;
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    list.hi[j] = hi[j];
    if (j < 8) list.lo |= lo[j] << (4 * j);
    else list.lo_hi8 |= lo[j] << (4 * (j - 8));
  }
  list.head = (kJ - 1 - static_cast<int>(list.lo & 0xFu)) * 64 + lane;
  float prev = 0.0f;
  bool closed = false;
  for (int k = 0; k < kWave && !closed; ++k) {
    uint32_t key;
    const int e = topk_round(list, lane, key);
    const float v = key_value(key);
    // false for inf - inf and next to an infinite key
    const bool apart = k == 0 || prev - v > fmaf(mg.rel, fmaxf(fabsf(prev), fabsf(v)), mg.cap);
    closed = key == 0u || (k >= a.K && apart);   // no live expert is left, or a gap behind rank K
    if (!closed) {
      r.ordered = r.ordered && apart;
      r.n = k + 1;
      r.e = lane == k ? e : r.e;
      prev = v;
    }
  }
  r.open = r.open || !(closed || wave_max_u32_s(list.hi[0]) == 0u);
  return r;
}

// The candidates in the order of their fp64 keys (ties: the lower expert).
__device__ __forceinline__ int reorder64(const SelectArgs& a, int t, const Candidates& c, const Softmax& sm, int lane,
                                         double* scratch) {
  double k = 0.0;
  if (lane < c.n) k = score64(a, logit_at(a, t, c.e), sm) + (a.bias != nullptr ? static_cast<double>(a.bias[c.e]) : 0.0);
  int* to = reinterpret_cast<int*>(scratch);
  int rank = 0;
  for (int i = 0; i < c.n; ++i) {
    const double ki = __shfl(k, i, kWave);
    const int ei = __shfl(c.e, i, kWave);
    rank += (ki > k || (ki == k && ei < c.e)) ? 1 : 0;
  }
  if (lane < c.n) to[rank] = c.e;
  __builtin_amdgcn_wave_barrier();
  __threadfence_block();
  return lane < c.n ? to[lane] : -1;
}

template <int kJ>
__device__ __forceinline__ void load_token(const SelectArgs& a, int t, int lane, float (&z)[kJ]) {
#pragma unroll
  for (int j = 0; j < kJ; ++j) z[j] = lane + 64 * j < a.E ? logit_at(a, t, lane + 64 * j) : -INFINITY;
}
template <int kJ>
__device__ __forceinline__ float logit_max(const float (&z)[kJ]) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kJ; ++j) m = fmaxf(m, z[j]);
  return wave_max(m);
}
__device__ __forceinline__ int lanes_per_group(const SelectArgs& a) {   // a power of two: every group has its own
  int L = 64;
  while (L > 1 && 64 / L < a.n_group) L >>= 1;
  return L;
}
__device__ __forceinline__ void write_choice(const SelectArgs& a, int t, int lane, int my_e, const Softmax& sm) {
  double sc = my_e >= 0 ? score64(a, logit_at(a, t, my_e), sm) : 0.0;
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
__device__ __forceinline__ void select_token(const SelectArgs& a, int t, int lane, double* keys) {
  float z[kJ];
  load_token<kJ>(a, t, lane, z);
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
  Softmax sm = {-INFINITY, 1.0};
  if (a.score == MOE_SCORE_SOFTMAX) sm.m = logit_max(z);
  const int L = lanes_per_group(a);
  const Candidates c = choose32<kJ>(a, z, sm.m, lane, L, reinterpret_cast<float*>(keys));
  // weights that are renormalised do not need the softmax's sum
  if (a.score == MOE_SCORE_SOFTMAX && (c.open || !c.ordered || !a.renorm)) sm.total = total64(z, sm.m);
  int my_e = c.e;
  if (c.open) my_e = choose64<kJ>(a, z, sm, lane, L, keys);
  else if (!c.ordered) my_e = reorder64(a, t, c, sm, lane, keys);
  my_e = lane < a.K ? my_e : -1;
  write_choice(a, t, lane, my_e, sm);
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
  if (T < 0 || T > moe::kMaxSelectTokens)
    return set_error(MOE_ESHAPE, "n_tokens=%d must be in [0, %d]", T, moe::kMaxSelectTokens);
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
