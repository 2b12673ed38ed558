// Attention over the paged cache (see include/moe_attn.h), key by key: one
// workgroup for each token and key head, its waves take the query heads in
// turn, a wave's lanes the head's dimensions.
#include "attn.h"

namespace moe {
namespace {

template <int ACT, int D>
__global__ __launch_bounds__(256) void k_attn_rows(AttnArgs a) {
  constexpr int kPer = D / 64;
  const int t = blockIdx.x, hk = blockIdx.y, group = a.Hq / a.Hk, lane = threadIdx.x & 63;
  int b = t, begin = t, end = t + 1;
  if (a.off) {
    b = __builtin_amdgcn_readfirstlane(seq_of_row(a.off, a.B, a.N, t));
    if (b >= a.B) return;
    seq_rows(a.off, b, a.N, begin, end);
  }
  const int seen = seq_length(a.length, b, a.max_pages, a.page_log) - (end - 1 - t);
  const int32_t* table = a.table + static_cast<size_t>(b) * a.max_pages;
  for (int g = threadIdx.x >> 6; g < group; g += 4) {
    const int h = hk * group + g;
    float q[kPer], acc[kPer], m = -INFINITY, l = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      q[i] = act_to_f32<ACT>(a.q[t * a.q_ts + h * a.q_hs + lane + 64 * i]);
      acc[i] = 0;
    }
    for (int j = 0; j < seen; ++j) {
      const int page = table[j >> a.page_log];
      if (page < 0 || page >= a.n_pages) continue;
      const size_t at =
          (((static_cast<size_t>(page) * a.Hk + hk) << a.page_log) + (j & ((1 << a.page_log) - 1))) * D + lane;
      float z = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) z = fmaf(q[i], act_to_f32<ACT>(a.k[at + 64 * i]), z);
      z = wave_sum(z) * a.scale;
      const float mn = fmaxf(m, z), base = mn == -INFINITY ? 0.0f : mn, c = expf(m - base), p = expf(z - base);
      m = mn;
      l = fmaf(l, c, p);
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] = fmaf(p, act_to_f32<ACT>(a.v[at + 64 * i]), acc[i] * c);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      float o = l != 0 ? acc[i] / l : 0.0f;
      if (a.gate) o /= 1 + expf(-act_to_f32<ACT>(a.gate[t * a.g_ts + h * a.g_hs + lane + 64 * i]));
      a.o[(static_cast<size_t>(t) * a.Hq + h) * D + lane + 64 * i] = static_cast<uint16_t>(pack2<ACT>(o, 0));
    }
  }
}

hipError_t launch(int act, int d, const AttnArgs& a, hipStream_t s) {
  const auto k = act == MOE_BF16 ? d == 64 ? k_attn_rows<2, 64> : d == 128 ? k_attn_rows<2, 128> : k_attn_rows<2, 256>
                 : d == 64       ? k_attn_rows<1, 64>
                 : d == 128      ? k_attn_rows<1, 128>
                                 : k_attn_rows<1, 256>;
  hipLaunchKernelGGL(k, dim3(a.N, a.Hk), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

size_t attn_prefill_bytes(const moe_attn_desc*, int) { return 256; }
hipError_t launch_attn_prefill(int act, int d, const AttnArgs& a, void*, hipStream_t s) { return launch(act, d, a, s); }

}  // namespace moe
