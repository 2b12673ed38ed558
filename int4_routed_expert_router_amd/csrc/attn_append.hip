// New tokens' keys and values into the paged cache, with the norms and rotary
// positions of queries and keys (see include/moe_attn.h).
//
// D / 8 lanes take a head of a token, 16 bytes each; a lane of the rotated part
// also loads its partner's 16 bytes, so that only the sum of squares crosses
// lanes.  A workgroup takes up to R heads of one token for each of its rows of
// lanes; all their loads leave before the token's sequence, position and page
// are looked up.  The first threads work the angles out, fp64 until they are
// reduced to half a turn.
#include "attn.h"

namespace moe {
namespace {

constexpr int kManyTokens = 1024;

template <int ACT>
__device__ __forceinline__ void unpack8(uint4 w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = act_to_f32<ACT>((u[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
}

template <int ACT, int D, int R>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a) {
  constexpr int kLanes = D / 8, kRows = 256 / kLanes;
  __shared__ float2 turn[128];
  const int t = blockIdx.x, half = a.rot / 2, nq = a.q ? a.Hq : 0, rows = nq + 2 * a.Hk;
  const int row0 = blockIdx.y * kRows * R + threadIdx.x / kLanes, c0 = 8 * (threadIdx.x % kLanes);
  const int pc = c0 < half ? c0 + half : c0 < a.rot ? c0 - half : c0;   // the partner's values
  uint4 xv[R], yv[R];   // rows behind the last read that one
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = min(row0 + i * kRows, rows - 1), h = row - nq;
    const uint16_t* src = row < nq    ? a.q + row_at(t, a.q_ts, row, a.q_hs)
                          : h < a.Hk ? a.k + row_at(t, a.k_ts, h, a.k_hs)
                                     : a.v + row_at(t, a.v_ts, h - a.Hk, a.v_hs);
    xv[i] = *reinterpret_cast<const uint4*>(src + c0);
    yv[i] = xv[i];
    if (c0 < a.rot && h < a.Hk) yv[i] = *reinterpret_cast<const uint4*>(src + pc);
  }
  int b = t, begin = t, end = t + 1;
  if (a.off) {
    b = __builtin_amdgcn_readfirstlane(seq_of_row(a.off, a.B, a.N, t));
    if (b >= a.B) return;
    seq_rows(a.off, b, a.N, begin, end);
  }
  const int pos = seq_length(a.length, b, a.max_pages, a.page_log) - (end - t);
  if (pos < 0) return;
  const int page = a.table[static_cast<size_t>(b) * a.max_pages + (pos >> a.page_log)];
  const int slot = pos & ((1 << a.page_log) - 1);
  const bool paged = page >= 0 && page < a.n_pages;
  if (static_cast<int>(threadIdx.x) < half) {
    // radians to [-pi, pi]: k whole turns taken off in two parts of 2 pi
    const double x = pos * a.freq[threadIdx.x], k = rint(x * 0.15915494309189535);
    const float r = static_cast<float>(fma(-k, 2.4492935982947064e-16, fma(-k, 6.283185307179586, x)));
    float s, c;
    sincosf(r, &s, &c);
    turn[threadIdx.x] = make_float2(c, s);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = row0 + i * kRows, h = row - nq;
    if (row >= rows || (h >= 0 && !paged)) continue;
    uint16_t* dst = a.q_out + (static_cast<size_t>(t) * a.Hq + row) * D + c0;
    if (h >= 0)
      dst = (h < a.Hk ? a.kc : a.vc) +
            (((static_cast<size_t>(page) * a.Hk + (h < a.Hk ? h : h - a.Hk)) << a.page_log) + slot) * D + c0;
    const float* norm = h < 0 ? a.q_norm : a.k_norm;
    uint4 w = xv[i];
    if (h < a.Hk && (norm || c0 < a.rot)) {
      float x[8], y[8];
      unpack8<ACT>(xv[i], x);
      unpack8<ACT>(yv[i], y);
      if (norm) {
        float ss = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) ss += __shfl_xor(ss, m);
        const float r = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] *= r * norm[c0 + j];
          y[j] *= r * norm[pc + j];
        }
      }
      if (c0 < a.rot) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 cs = turn[(c0 < half ? c0 : pc) + j];
          x[j] = c0 < half ? x[j] * cs.x - y[j] * cs.y : x[j] * cs.x + y[j] * cs.y;
        }
      }
      w = make_uint4(pack2<ACT>(x[0], x[1]), pack2<ACT>(x[2], x[3]), pack2<ACT>(x[4], x[5]), pack2<ACT>(x[6], x[7]));
    }
    *reinterpret_cast<uint4*>(dst) = w;
  }
}

template <int ACT, int D>
hipError_t launch(const AppendArgs& a, hipStream_t s) {
  const int rows = (a.q ? a.Hq : 0) + 2 * a.Hk, per = 256 / (D / 8);
  // few tokens, or few heads: every head its own lanes
  if (a.N < kManyTokens || rows <= per)
    hipLaunchKernelGGL((k_kv_append<ACT, D, 1>), dim3(a.N, (rows + per - 1) / per), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_kv_append<ACT, D, 4>), dim3(a.N, (rows + 4 * per - 1) / (4 * per)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(int act, int d, const AppendArgs& a, hipStream_t s) {
  if (act == MOE_BF16) return d == 64 ? launch<2, 64>(a, s) : d == 128 ? launch<2, 128>(a, s) : launch<2, 256>(a, s);
  return d == 64 ? launch<1, 64>(a, s) : d == 128 ? launch<1, 128>(a, s) : launch<1, 256>(a, s);
}

}  // namespace moe
