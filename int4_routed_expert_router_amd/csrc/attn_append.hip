// New tokens' keys and values into the paged cache, with the norms and rotary
// positions of queries and keys (see include/moe_attn.h).
//
// D / 8 lanes take a head of a token, 16 bytes each; a lane of the rotated part
// also loads its partner's 16 bytes, so that only the sum of squares crosses
// lanes.  A workgroup takes up to R heads of one token for each of its rows of
// lanes; all their loads leave before the token's sequence, position and page
// are looked up.
//
// One token, 16 and 2 heads of 256: 2.9 to 3.4 us, latency of the look-up's loads and
// the launch.  8191 tokens of 5 sequences: 50 us, 168 MB at 3.4 TB/s, of which a
// copy without norms and rotation takes 42 (rows of 512 bytes from every other
// 512 bytes of a projection's output, to pages); with every head its own lanes
// (R = 1) 52.  20 rows (16 + 2 + 2) take 20 of a workgroup's 32 places with R = 4:
// the others load the last row and write nothing.  Stores past the caches are 3 us
// faster here, but the attention that follows reads what they wrote.
#include "attn.h"

namespace moe {
namespace {

// From so many tokens on R = 4 (timed for 16 and 2 heads of 256): 300 tokens take 7.0 us with R = 1 against 8.2, 1000 take 10.0
// against 9.9, 8191 52 against 49.5.
constexpr int kManyTokens = 1024;

template <int ACT>
__device__ __forceinline__ void unpack8(uint4 w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = act_to_f32<ACT>((u[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
}

// Sum over a head's 8, 16 or 32 neighbouring lanes, the same in each.
template <int LANES>
__device__ __forceinline__ float head_sum(float v) {
  auto add = [](float a, uint32_t b) { return a + __uint_as_float(b); };
  v = add(v, dpp_u32<0xB1>(__float_as_uint(v)));    // quad_perm [1,0,3,2]
  v = add(v, dpp_u32<0x4E>(__float_as_uint(v)));    // quad_perm [2,3,0,1]
  v = add(v, dpp_u32<0x141>(__float_as_uint(v)));   // row_half_mirror
  if constexpr (LANES >= 16) v = add(v, dpp_u32<0x140>(__float_as_uint(v)));   // row_mirror
  if constexpr (LANES == 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_int(v), __float_as_int(v), false, false);
    v = __int_as_float(a[0]) + __int_as_float(a[1]);
  }
  return v;
}

// Cosine and sine of x radians.  x to [-pi/4, pi/4] in fp64, by quarter turns
// (pi/2 in two parts), then Taylor's series: the first terms left out, x^10 / 10!
// and x^11 / 11!, are below 2^-25.
__device__ __forceinline__ float2 cos_sin(double x) {
  const double k = rint(x * 0.63661977236758134);
  const float r = static_cast<float>(fma(-k, 6.123233995736766e-17, fma(-k, 1.5707963267948966, x))), z = r * r;
  const int n = static_cast<int>(fma(-4.0, floor(0.25 * k), k));   // k mod 4
  const float s = fmaf(r * z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), r);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 40320, -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  const float cc = n & 1 ? s : c, ss = n & 1 ? c : s;
  return make_float2(n == 1 || n == 2 ? -cc : cc, n >= 2 ? -ss : ss);
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
  // the lane's own and its partner's norms, the same for every head of queries (of keys)
  float nx[8], ny[8];
  auto load_norm = [&](const float* norm) {
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      *reinterpret_cast<float4*>(nx + j) = *reinterpret_cast<const float4*>(norm + c0 + j);
      *reinterpret_cast<float4*>(ny + j) = *reinterpret_cast<const float4*>(norm + pc + j);
    }
  };
  const float* loaded = row0 < nq ? a.q_norm : row0 < nq + a.Hk ? a.k_norm : nullptr;
  if (loaded) load_norm(loaded);
  const double freq = static_cast<int>(threadIdx.x) < half ? a.freq[threadIdx.x] : 0.0;
  // the token's sequence and the tokens from it to the sequence's end
  int b = t, left = 1, length;
  if (a.off && a.B <= 64) {   // all sequences at once, one to a lane
    const int lane = threadIdx.x & 63, i = min(lane, a.B - 1);
    int begin, end;
    seq_rows(a.off, i, a.N, begin, end);
    length = seq_length(a.length, i, a.max_pages, a.page_log);
    const uint64_t hit = __ballot(lane < a.B && t >= begin && t < end);
    if (hit == 0) return;
    b = __builtin_ctzll(hit);
    left = __builtin_amdgcn_readlane(end, b) - t;
    length = __builtin_amdgcn_readlane(length, b);
  } else {
    if (a.off) {
      b = __builtin_amdgcn_readfirstlane(seq_of_row(a.off, a.B, a.N, t));
      if (b >= a.B) return;
      int begin, end;
      seq_rows(a.off, b, a.N, begin, end);
      left = end - t;
    }
    length = seq_length(a.length, b, a.max_pages, a.page_log);
  }
  const int pos = length - left;
  if (pos < 0) return;
  const int page = a.table[static_cast<size_t>(b) * a.max_pages + (pos >> a.page_log)];
  const int slot = pos & ((1 << a.page_log) - 1);
  const bool paged = page >= 0 && page < a.n_pages;
  if (static_cast<int>(threadIdx.x) < half) turn[threadIdx.x] = cos_sin(pos * freq);
  __syncthreads();
  float2 cs[8];   // the lane's turns, the same for every head
  if (c0 < a.rot) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cs[j] = turn[(c0 < half ? c0 : pc) + j];
      if (c0 < half) cs[j].y = -cs[j].y;
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = row0 + i * kRows, h = row - nq;
    if (row >= rows || (h >= 0 && !paged)) continue;
    uint16_t* dst = a.q_out + (static_cast<size_t>(t) * a.Hq + row) * D + c0;
    if (h >= 0)
      dst = (h < a.Hk ? a.kc : a.vc) +
            (((static_cast<size_t>(page) * a.Hk + (h < a.Hk ? h : h - a.Hk)) << a.page_log) + slot) * D + c0;
    const float* norm = h < 0 ? a.q_norm : h < a.Hk ? a.k_norm : nullptr;
    if (norm && norm != loaded) load_norm(loaded = norm);
    uint4 w = xv[i];
    if (h < a.Hk && (norm || c0 < a.rot)) {
      float x[8], y[8];
      unpack8<ACT>(xv[i], x);
      unpack8<ACT>(yv[i], y);
      if (norm) {
        auto mean_square = [&](float eps) {
          float ss = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
          return fmaf(head_sum<kLanes>(ss), 1.0f / D, eps);
        };
        float ms = mean_square(a.eps);
        if (__any(ms < 0x1p-80f)) {   // rows whose squares leave fp32's range below, times 2^80
          const float up = ms < 0x1p-80f ? 0x1p80f : 1.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= up, y[j] *= up;
          ms = mean_square(a.eps * up * up);
        }
        const float r = __builtin_amdgcn_rsqf(ms);   // the hardware's, within an ulp
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] *= r * nx[j];
          y[j] *= r * ny[j];
        }
      }
      if (c0 < a.rot) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaf(x[j], cs[j].x, y[j] * cs[j].y);
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
