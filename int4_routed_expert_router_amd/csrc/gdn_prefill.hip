// Gated DeltaNet over whole sequences (see include/moe_gdn.h).
#include <hip/hip_runtime.h>

#include "moe_common.h"
#include "moe_gdn.h"

namespace moe {
moe_status set_error(moe_status code, const char* fmt, ...);

namespace {

constexpr int kDK = 128;
constexpr float kEps = 1e-6f;

bool gp_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
__device__ __forceinline__ float row_sum16(float x) { return __uint_as_float(dpp_row_sum(__float_as_uint(x))); }

struct GdnArgs {
  const int32_t* off;   // [B+1]
  const uint16_t *q, *k, *v;
  const float *g, *beta;
  float *state, *o;
  float q_scale;
  int B, N, Hk, Hv, dv;
};

// tokens [begin, end) of sequence b, with the offsets forced into [0, N]
__device__ __forceinline__ void seq_range(const GdnArgs& a, int b, int& begin, int& end) {
  begin = min(max(a.off[b], 0), a.N);
  end = max(min(max(a.off[b + 1], 0), a.N), begin);
}

// Token by token: one workgroup per (16 state rows, value head, sequence); a
// row of 16 lanes owns one state row in registers, lane l16 its columns
// 8 l16 .. 8 l16 + 7.
template <int ACT>
__global__ __launch_bounds__(256) void k_gdn_tokens(GdnArgs a) {
  const int slices = a.dv / 16;
  const int h = blockIdx.x / slices, row = (blockIdx.x % slices) * 16 + (threadIdx.x >> 4);
  const int b = blockIdx.y, hk = h / (a.Hv / a.Hk), c0 = 8 * (threadIdx.x & 15);
  int t0, t1;
  seq_range(a, b, t0, t1);
  if (t0 == t1) return;
  float* srow = a.state + ((static_cast<size_t>(b) * a.Hv + h) * a.dv + row) * kDK + c0;
  float s[8];
  *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(srow);
  *reinterpret_cast<float4*>(s + 4) = *reinterpret_cast<const float4*>(srow + 4);
  uint4 qv, kv;
  uint32_t vv;
  float gv, bv;
  auto load = [&](int t) {
    const size_t qk = (static_cast<size_t>(t) * a.Hk + hk) * kDK + c0, hv = static_cast<size_t>(t) * a.Hv + h;
    qv = *reinterpret_cast<const uint4*>(a.q + qk);
    kv = *reinterpret_cast<const uint4*>(a.k + qk);
    vv = a.v[hv * a.dv + row];
    gv = a.g[hv];
    bv = a.beta[hv];
  };
  load(t0);
  for (int t = t0; t < t1; ++t) {
    const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w}, kw[4] = {kv.x, kv.y, kv.z, kv.w};
    const float alpha = expf(gv), bt = bv, vt = act_to_f32<ACT>(vv);
    load(min(t + 1, t1 - 1));
    float qn[8], kn[8], qq = 0, kk = 0, kq = 0, u = 0, w = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      qn[j] = act_to_f32<ACT>((qw[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
      kn[j] = act_to_f32<ACT>((kw[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
      qq = fmaf(qn[j], qn[j], qq);
      kk = fmaf(kn[j], kn[j], kk);
      kq = fmaf(kn[j], qn[j], kq);
      u = fmaf(s[j], kn[j], u);
      w = fmaf(s[j], qn[j], w);
    }
    qq = row_sum16(qq);
    kk = row_sum16(kk);
    kq = row_sum16(kq);
    u = row_sum16(u);
    w = row_sum16(w);
    const float rq = a.q_scale / sqrtf(qq + kEps), rk = 1.0f / sqrtf(kk + kEps);
    const float d = bt * (vt - alpha * (u * rk)), dk = d * rk;
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = fmaf(dk, kn[j], alpha * s[j]);
    if (c0 == 0) a.o[(static_cast<size_t>(t) * a.Hv + h) * a.dv + row] = fmaf(dk * rq, kq, alpha * (w * rq));
  }
  *reinterpret_cast<float4*>(srow) = *reinterpret_cast<const float4*>(s);
  *reinterpret_cast<float4*>(srow + 4) = *reinterpret_cast<const float4*>(s + 4);
}

moe_status check_prefill(const moe_gdn_desc* d, int32_t N) {
  if (!d) return set_error(MOE_EINVAL, "desc is NULL");
  if (d->batch < 0 || d->batch > 65535) return set_error(MOE_ESHAPE, "batch=%d must be in [0, 65535]", d->batch);
  if (d->head_k_dim != kDK) return set_error(MOE_ESHAPE, "head_k_dim=%d must be %d", d->head_k_dim, kDK);
  if (d->head_v_dim < 16 || d->head_v_dim > 256 || d->head_v_dim % 16)
    return set_error(MOE_ESHAPE, "head_v_dim=%d must be a multiple of 16 in [16, 256]", d->head_v_dim);
  if (d->k_heads < 1 || d->v_heads < d->k_heads || d->v_heads > 1024 || d->v_heads % d->k_heads)
    return set_error(MOE_ESHAPE, "v_heads=%d must be a multiple of k_heads=%d, at most 1024", d->v_heads, d->k_heads);
  if (d->act_dtype != MOE_F16 && d->act_dtype != MOE_BF16)
    return set_error(MOE_EINVAL, "act_dtype=%d is not MOE_F16/MOE_BF16", d->act_dtype);
  if (N < 0 || N > (1 << 30)) return set_error(MOE_ESHAPE, "n_tokens=%d must be in [0, 2^30]", N);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_gdn_prefill_workspace_bytes(const moe_gdn_desc* d, int32_t n_tokens, size_t* bytes) {
  const moe_status st = moe::check_prefill(d, n_tokens);
  if (st) return st;
  if (!bytes) return moe::set_error(MOE_EINVAL, "bytes is NULL");
  *bytes = 256;
  return moe::set_error(MOE_OK, "");
}

extern "C" moe_status moe_gdn_prefill(const moe_gdn_desc* d, const int32_t* seq_off, int32_t n_tokens, const void* q,
                                      const void* k, const void* v, const float* g, const float* beta, float q_scale,
                                      float* state, float* o, void* ws, size_t ws_bytes, moe_stream stream) {
  using moe::gp_aligned;
  using moe::set_error;
  const moe_status st = moe::check_prefill(d, n_tokens);
  if (st) return st;
  if (d->batch == 0 || n_tokens == 0) return set_error(MOE_OK, "");
  if (!seq_off || !q || !k || !v || !g || !beta || !state || !o) return set_error(MOE_EINVAL, "NULL buffer");
  if (!gp_aligned(q, 16) || !gp_aligned(k, 16) || !gp_aligned(v, 2) || !gp_aligned(state, 16))
    return set_error(MOE_EINVAL, "q, k and state must be 16-byte and v 2-byte aligned");
  if (!gp_aligned(seq_off, 4) || !gp_aligned(g, 4) || !gp_aligned(beta, 4) || !gp_aligned(o, 4))
    return set_error(MOE_EINVAL, "seq_off, g, beta and o must be 4-byte aligned");
  size_t need = 0;
  moe_gdn_prefill_workspace_bytes(d, n_tokens, &need);
  if (!ws || !gp_aligned(ws, 256)) return set_error(MOE_EINVAL, "workspace must be a 256-byte aligned device pointer");
  if (ws_bytes < need) return set_error(MOE_EWORKSPACE, "workspace of %zu bytes < required %zu", ws_bytes, need);
  moe::GdnArgs a{seq_off, static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                 static_cast<const uint16_t*>(v), g, beta, state, o, q_scale, d->batch, n_tokens, d->k_heads,
                 d->v_heads, d->head_v_dim};
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid(d->v_heads * (d->head_v_dim / 16), d->batch);
  if (d->act_dtype == MOE_BF16) hipLaunchKernelGGL(moe::k_gdn_tokens<2>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(moe::k_gdn_tokens<1>, grid, dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(MOE_EHIP, "Gated DeltaNet prefill kernel launch: %s", hipGetErrorString(e));
  return set_error(MOE_OK, "");
}
