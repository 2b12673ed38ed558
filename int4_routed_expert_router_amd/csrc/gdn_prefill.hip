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

// ---- token by token ---------------------------------------------------------
// A row of 16 lanes owns NS state rows in registers (row0 + 16 z, those below
// d_v), lane l16 their columns 8 l16 .. 8 l16 + 7.  Runs tokens [t0, t1) of
// one sequence and value head in fp32; the next token's loads are in flight
// meanwhile.  A row's arithmetic does not depend on NS.
template <int ACT, int NS>
__device__ __forceinline__ void run_tokens(const GdnArgs& a, int b, int h, int t0, int t1, int row0) {
  const int hk = h / (a.Hv / a.Hk), c0 = 8 * (threadIdx.x & 15);
  float* srow[NS];
  float s[NS][8];
  int row[NS];
#pragma unroll
  for (int z = 0; z < NS; ++z) {
    row[z] = NS == 1 ? row0 : min(row0 + 16 * z, a.dv - 1);
    srow[z] = a.state + ((static_cast<size_t>(b) * a.Hv + h) * a.dv + row[z]) * kDK + c0;
    *reinterpret_cast<float4*>(s[z]) = *reinterpret_cast<const float4*>(srow[z]);
    *reinterpret_cast<float4*>(s[z] + 4) = *reinterpret_cast<const float4*>(srow[z] + 4);
  }
  uint4 qv, kv;
  uint32_t vv[NS];
  float gv, bv;
  auto load = [&](int t) {
    const size_t qk = (static_cast<size_t>(t) * a.Hk + hk) * kDK + c0, hv = static_cast<size_t>(t) * a.Hv + h;
    qv = *reinterpret_cast<const uint4*>(a.q + qk);
    kv = *reinterpret_cast<const uint4*>(a.k + qk);
#pragma unroll
    for (int z = 0; z < NS; ++z) vv[z] = a.v[hv * a.dv + row[z]];
    gv = a.g[hv];
    bv = a.beta[hv];
  };
  load(t0);
  for (int t = t0; t < t1; ++t) {
    const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w}, kw[4] = {kv.x, kv.y, kv.z, kv.w};
    // the hardware's exp2 and 1/sqrt, each within an ulp; x log2(e) is off by
    // |x| 2^-24 of the decay at most
    const float alpha = __builtin_amdgcn_exp2f(gv * 1.44269504f), bt = bv;
    float vt[NS];
#pragma unroll
    for (int z = 0; z < NS; ++z) vt[z] = act_to_f32<ACT>(vv[z]);
    load(min(t + 1, t1 - 1));
    float qn[8], kn[8], qq = 0, kk = 0, kq = 0;
    // the rows are normalised before they meet each other or the state: a raw
    // product may overflow where the normalised one is finite (or, with a row
    // whose squares overflow, 0)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      qn[j] = act_to_f32<ACT>((qw[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
      kn[j] = act_to_f32<ACT>((kw[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
      qq = fmaf(qn[j], qn[j], qq);
      kk = fmaf(kn[j], kn[j], kk);
    }
    qq = row_sum16(qq);
    kk = row_sum16(kk);
    const float rq = a.q_scale * __builtin_amdgcn_rsqf(qq + kEps), rk = __builtin_amdgcn_rsqf(kk + kEps);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      qn[j] *= rq;
      kn[j] *= rk;
      kq = fmaf(kn[j], qn[j], kq);
    }
    kq = row_sum16(kq);
    float* o = a.o + (static_cast<size_t>(t) * a.Hv + h) * a.dv;
#pragma unroll
    for (int z = 0; z < NS; ++z) {
      float u = 0, w = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u = fmaf(s[z][j], kn[j], u);
        w = fmaf(s[z][j], qn[j], w);
      }
      u = row_sum16(u);
      w = row_sum16(w);
      const float d = bt * fmaf(-alpha, u, vt[z]);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[z][j] = fmaf(d, kn[j], alpha * s[z][j]);
      if (c0 == 0 && (NS == 1 || row0 + 16 * z < a.dv)) o[row[z]] = fmaf(d, kq, alpha * w);
    }
  }
#pragma unroll
  for (int z = 0; z < NS; ++z) {
    if (NS == 1 || row0 + 16 * z < a.dv) {
      *reinterpret_cast<float4*>(srow[z]) = *reinterpret_cast<const float4*>(s[z]);
      *reinterpret_cast<float4*>(srow[z] + 4) = *reinterpret_cast<const float4*>(s[z] + 4);
    }
  }
}

// Sequences up to this length go token by token, longer ones in blocks (32
// value heads of 128; token by token against blocks, us): 20 tokens 11.1
// against 16.4 for one sequence, 35 against 39 for 8, 173 against 243 for 64;
// 24 tokens 12.5 / 16.5, 39.1 / 39.5, 201 / 242; 32 tokens 15.8 / 16.5, 48 / 40,
// 256 / 245.
constexpr int kShort = 24;

// The sequences of at most kShort tokens: one workgroup per (16 NS state rows,
// value head, sequence).  With NS = 1 most of a token's arithmetic is the
// conversion and the norms of its q and k, the same in every row; 4 rows per
// lane share it.  64 sequences of 8 tokens with 32 heads of 128: 97 us, 268 MB
// of state at 2.8 TB/s, bound by the vector arithmetic; 16 tokens of one
// sequence: 9.7 us with its launch, bound by the latency of a token's chain: its
// norms, then its sums with the state.
template <int ACT, int NS>
__global__ __launch_bounds__(256) void k_gdn_tokens(GdnArgs a) {
  const int slices = (a.dv + 16 * NS - 1) / (16 * NS);
  int t0, t1;
  seq_range(a, blockIdx.y, t0, t1);
  if (t0 < t1 && t1 - t0 <= kShort)
    run_tokens<ACT, NS>(a, blockIdx.y, blockIdx.x / slices, t0, t1,
                        (blockIdx.x % slices) * 16 * NS + (threadIdx.x >> 4));
}

// ---- in blocks of 64 tokens -------------------------------------------------
// Within a block, with G_t the running sum of g, S the state before it and
// k^, q^ the normalised rows, the rule is
//   (I + A) D = beta (V - e^G K^ S^T),    A_ij = beta_i e^(G_i - G_j) k^_i.k^_j  (j < i)
//   O = e^G Q^ S^T + P D,                 P_ij = e^(G_i - G_j) q^_i.k^_j         (j <= i)
//   S <- e^(G_last) S + D^T (e^(G_last - G) K^).
// k_gdn_blocks forms, for all blocks at once, what does not depend on S:
// T = (I + A)^-1 diag(beta) and M = P T, so that with R = V - e^G K^ S^T
//   D = T R,  O = e^G Q^ S^T + M R.
// k_gdn_scan then takes one sequence's blocks in order.
//
// State and results are fp32, so fp32 operands enter the matrix cores as an
// fp16 pair hi + lo / 2^11 (22 significant bits) under a power-of-two scale that
// keeps them within fp16's range.  Such a scale holds for a whole block, in
// which numbers differ widely (a state of 10^6 times the values, decays to
// e^-30); with lo scaled up they keep all 22 bits down to 2^-26 of the largest,
// and what lies below 2^-48 of it counts as zero.  (With lo as it is the error
// begins at 2^-15: a state of 10^6 times the values, decayed by e^-0.5 a token,
// ended 10^-3 off.)  Each row of keys and queries is scaled by a power of two of
// its own (the row's norm is applied afterwards): fp16 and bf16 rows are then
// exact in fp16 but for elements below 2^-26 of the row's largest, which are off
// by 2^-37 of it at most.
// An operand pair costs two products against an exact operand and three
// against another pair; fp32 matrix instructions take 8 times as long as
// fp16's for the same product.
constexpr int kBlock = 64;         // tokens of a block
constexpr int kRow = 136;          // LDS row of 128 fp16 values, padded
constexpr int kRowF = 68;          // the same bytes as fp32 values

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Workspace.  A sequence's block c sits in slot begin/64 + b + c: distinct
// for all blocks (a sequence of n tokens takes at most ceil(n/64) <= the
// distance to the next sequence's first slot), below n_tokens/64 + batch.
// Operand tiles ("frags") are stored as the matrix instruction takes them, 16
// bytes per lane.  The summed index of a 32-wide step runs, for lane group q =
// lane/16, over 4q..4q+3 and 16+4q..16+4q+3: the order in which the result
// tiles of two 16-row products hold their rows, so results become operands
// without moving between lanes.
//   per (slot, key head):   K rows [4 tiles][4 steps], Q rows the same, K columns [8 tiles][2 steps]
//   per (slot, value head): T and M rows as [6][hi, lo] (tile rows 0, 1: step 0; 2, 3: steps 0 and 1),
//                           256 floats: e^G rk, e^G, rq per token, then kSc*
// Of a block that goes token by token (see k_gdn_scan) only kScGamma is set, to -1.
constexpr size_t kKeyBytes = 48 * 1024;
constexpr size_t kHeadBytes = 25 * 1024;
constexpr int kScGamma = 192, kScInvT = 193, kScInvM = 194, kScGmax = 195, kScD = 196, kScS = 197;

constexpr size_t kMaxSlots = (1 << 24) - 1;   // a grid dimension holds fewer than 2^32 threads, 256 per slot

__host__ __device__ inline size_t prefill_slots(int B, int N) { return static_cast<size_t>(N) / kBlock + B; }

// offset of the value heads' part, behind the key heads'
__device__ __forceinline__ size_t prefill_ws_heads(const GdnArgs& a) {
  return prefill_slots(a.B, a.N) * a.Hk * kKeyBytes;
}

__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f16x8 as_frag(uint4 v) { return __builtin_bit_cast(f16x8, v); }

// Power of two that brings a magnitude into [2^12, 2^13), and its inverse.
struct Pow2 {
  float up, down;
};
__device__ __forceinline__ Pow2 pow2_scale(float m) {
  const int f = min(266 - static_cast<int>((__float_as_uint(m) >> 23) & 255u), 253);
  return {__uint_as_float(static_cast<uint32_t>(f) << 23), __uint_as_float(static_cast<uint32_t>(254 - f) << 23)};
}
// fp16 pair of v = hi + lo / 2^11: hi = nearest fp16, lo from the exact rest.
// With lo scaled up the pair keeps 22 bits of all v above 2^-14, where the
// scaled operands reach 2^13, and is off by 2^-36 at most below.
constexpr float kLoUp = 0x1p11f, kLoDown = 0x1p-11f;
__device__ __forceinline__ void split16(float v, _Float16& hi, _Float16& lo) {
  hi = static_cast<_Float16>(v);
  lo = static_cast<_Float16>((v - static_cast<float>(hi)) * kLoUp);
}
// max and sum over the four lanes that share a column (lane % 16): swaps of
// rows of 16 lanes and of halves
template <class Op>
__device__ __forceinline__ float col_reduce(float v, Op op) {
  const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = op(__uint_as_float(x[0]), __uint_as_float(x[1]));
  const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return op(__uint_as_float(y[0]), __uint_as_float(y[1]));
}
__device__ __forceinline__ float col_max(float v) {
  return col_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float col_sum(float v) {
  return col_reduce(v, [](float a, float b) { return a + b; });
}
// Inclusive prefix sum over the wave: row shifts within 16 lanes, then the
// totals of the rows before.
template <int kCtrl>
__device__ __forceinline__ double dpp_f64_or0(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = dpp_upd_u32<kCtrl, 0xF>(static_cast<uint32_t>(u), 0u);
  const uint32_t hi = dpp_upd_u32<kCtrl, 0xF>(static_cast<uint32_t>(u >> 32), 0u);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double lane_f64(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double scan_f64(double v, int lane) {
  v += dpp_f64_or0<0x111>(v);   // row_shr 1, 2, 4, 8 (0 where no lane is that far back)
  v += dpp_f64_or0<0x112>(v);
  v += dpp_f64_or0<0x114>(v);
  v += dpp_f64_or0<0x118>(v);
  const double r0 = lane_f64(v, 15), r1 = lane_f64(v, 31), r2 = lane_f64(v, 47);
  if (lane >= 16) v += r0;
  if (lane >= 32) v += r1;
  if (lane >= 48) v += r2;
  return v;
}

// Sequence and block of a slot: the sequence is the last one whose first slot
// (off/64 + b, increasing in b) is not above it.  64 candidates per step.
__device__ __forceinline__ bool find_block(const GdnArgs& a, int slot, int lane, int& b, int& t0, int& len) {
  int lo = 0, hi = a.B;
  while (true) {
    const int step = (hi - lo + 63) / 64, at = lo + lane * step;
    const bool below = at < hi && min(max(a.off[min(at, a.B - 1)], 0), a.N) / kBlock + at <= slot;
    const unsigned long long m = ~__ballot(below);
    const int n = m == 0 ? 64 : __ffsll(m) - 1;   // candidates from the front that are not above the slot
    if (n == 0) return false;
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) break;
  }
  b = lo;
  int begin, end;
  seq_range(a, b, begin, end);
  t0 = begin + (slot - (begin / kBlock + b)) * kBlock;
  len = min(end - t0, kBlock);
  return len > 0 && end - begin > kShort;
}

// 2^x by the hardware's exp2 of x rounded to fp32: off by |x| 2^-24 of the
// result, which is |x| 2^x 2^-24 < 2^-24 of 1
__device__ __forceinline__ float exp2_of(double x) { return __builtin_amdgcn_exp2f(static_cast<float>(x)); }

// 16x16x16 product in fp32: acc += X Y with X rows from LDS (x: lane's row,
// columns 4q .. 4q+3) and Y as a result tile (lane: column lane%16, rows 4q+r)
__device__ __forceinline__ f32x4 mul16(float4 x, f32x4 y, f32x4 acc) {
  acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x.x, y[0], acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x.y, y[1], acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x.z, y[2], acc, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x4f32(x.w, y[3], acc, 0, 0, 0);
}

// One workgroup per (slot, `per` value heads of a key head, one after the
// other); wave w owns tile row w of the 64 x 64 products k.k and q.k, then tile
// column w of T and M.  The inverse is by forward substitution (16 x 16 diagonal
// blocks column by column, then block by block), which stays accurate also
// where powers of A grow.
//
// 8192 tokens, 16 key and 32 value heads: 78 us (10 longer with one value head to
// a workgroup), four workgroups to a compute unit; 205 MB of operands written at
// 2.6 TB/s.  A lone workgroup with one value head takes about 9 us: loads and norms
// a quarter, k.k and q.k with their decays a fifth, the inverse an eighth, T and
// M a fifth, scaling and stores the rest.  81 scalar registers are spilled to
// lanes of vector registers (masks and addresses of the unrolled products).
template <int ACT>
__global__ __launch_bounds__(256, 4) void k_gdn_blocks(GdnArgs a, uint8_t* __restrict__ ws, int per) {
  __shared__ __attribute__((aligned(16))) uint16_t ks[kBlock * kRow];
  __shared__ __attribute__((aligned(16))) uint16_t qs[kBlock * kRow];
  __shared__ double Gs[kBlock];
  __shared__ float bs[kBlock], rks[kBlock], rqs[kBlock], lr[kBlock];   // lr: e^(G_last - G) rk
  __shared__ float wmax[4][2];
  __shared__ int rises;   // some g is above 0, or some beta outside [0, 2]
  float* As = reinterpret_cast<float*>(ks);   // takes the place of the keys once their products are done
  float* Ps = reinterpret_cast<float*>(qs);
  const int tid = threadIdx.x;
  int lane = tid & 63, n = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.x, rep = a.Hv / a.Hk, h0 = blockIdx.y * per, hk = h0 / rep;
  int b, tok0, len;
  if (!find_block(a, slot, lane, b, tok0, len)) return;   // the same for every thread

  {   // rows of K and Q: four lanes per token, 32 columns each
    const int row = tid >> 2, part = tid & 3;
    const bool ok = row < len;
    const size_t at = (static_cast<size_t>(tok0 + min(row, len - 1)) * a.Hk + hk) * kDK + 32 * part;
    uint4 raw[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      raw[0][i] = *reinterpret_cast<const uint4*>(a.k + at + 8 * i);
      raw[1][i] = *reinterpret_cast<const uint4*>(a.q + at + 8 * i);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float f[32], ss = 0.0f, mx = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const uint4& r = raw[m][i >> 3];
        const uint32_t word = (i & 7) < 2 ? r.x : (i & 7) < 4 ? r.y : (i & 7) < 6 ? r.z : r.w;
        f[i] = ok ? act_to_f32<ACT>((word >> (16 * (i & 1))) & 0xFFFFu) : 0.0f;
        ss = fmaf(f[i], f[i], ss);
        mx = fmaxf(mx, fabsf(f[i]));
      }
      ss += __uint_as_float(dpp_u32<0xB1>(__float_as_uint(ss)));
      ss += __uint_as_float(dpp_u32<0x4E>(__float_as_uint(ss)));
      mx = fmaxf(mx, __uint_as_float(dpp_u32<0xB1>(__float_as_uint(mx))));
      mx = fmaxf(mx, __uint_as_float(dpp_u32<0x4E>(__float_as_uint(mx))));
      const Pow2 p = pow2_scale(mx);
      const float norm = (m ? a.q_scale : 1.0f) / sqrtf(ss + kEps);
      if (part == 0) (m ? rqs : rks)[row] = ok ? norm * p.down : 0.0f;
      uint16_t* dst = (m ? qs : ks) + row * kRow + 32 * part;
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        f16x8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = static_cast<_Float16>(f[i + j] * p.up);
        *reinterpret_cast<f16x8*>(dst + i) = v;
      }
    }
  }
  __syncthreads();
  if (h0 % rep == 0) {   // the key head's operands, once
    uint4* out = reinterpret_cast<uint4*>(ws + (static_cast<size_t>(slot) * a.Hk + hk) * kKeyBytes);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint16_t* src = (m ? qs : ks) + (16 * w + n) * kRow + 4 * q;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint2 lo = *reinterpret_cast<const uint2*>(src + 32 * s), hi = *reinterpret_cast<const uint2*>(src + 32 * s + 16);
        out[((m * 4 + w) * 4 + s) * 64 + lane] = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) {   // column tiles 2w, 2w + 1 x two steps of tokens
      const uint16_t* src = ks + 16 * (2 * w + (f >> 1)) + n + (32 * (f & 1) + 4 * q) * kRow;
      uint32_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = (j >> 1) * 16 + 2 * (j & 1);
        v[j] = src[t * kRow] | (static_cast<uint32_t>(src[(t + 1) * kRow]) << 16);
      }
      out[(32 + 4 * w + f) * 64 + lane] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    kk[j] = qk[j] = f32x4{0, 0, 0, 0};
    if (j <= w) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const f16x8 ka = *reinterpret_cast<const f16x8*>(ks + (16 * w + n) * kRow + 32 * s + 8 * q);
        const f16x8 qa = *reinterpret_cast<const f16x8*>(qs + (16 * w + n) * kRow + 32 * s + 8 * q);
        const f16x8 kb = *reinterpret_cast<const f16x8*>(ks + (16 * j + n) * kRow + 32 * s + 8 * q);
        kk[j] = mfma(ka, kb, kk[j]);
        qk[j] = mfma(qa, kb, qk[j]);
      }
    }
  }
  // from here on per value head; the barriers of one head's turn also part its
  // use of the shared arrays from the next one's
  for (int h = h0; h < h0 + per; ++h) {
    // opaque: or the compiler keeps every address and mask of the body in
    // registers across the turns, which leaves room for two workgroups only
    asm volatile("" : "+v"(lane), "+v"(n), "+v"(q));
    float* vec = reinterpret_cast<float*>(ws + prefill_ws_heads(a) + (static_cast<size_t>(slot) * a.Hv + h) * kHeadBytes +
                                          24 * 1024);
    if (w == 0) {
      // log decays are summed in fp64, in units of log 2: differences of sums far
      // from 0 keep their digits (a block of strong decays reaches -1000 and
      // below).  -inf counts as -1000, which clears the state just as well
      // (e^-1000 = 0 in fp32).
      const size_t at = static_cast<size_t>(tok0 + min(lane, len - 1)) * a.Hv + h;
      const bool ok = lane < len;
      float gt = ok ? a.g[at] : 0.0f;
      gt = gt < -1000.0f ? -1000.0f : gt;
      Gs[lane] = scan_f64(static_cast<double>(gt) * 1.4426950408889634, lane);
      const float bt = ok ? a.beta[at] : 0.0f;
      bs[lane] = bt;
      const bool any = __ballot(!(gt <= 0.0f && bt >= 0.0f && bt <= 2.0f)) != 0ull;   // NaN too
      if (lane == 0) rises = any ? 1 : 0;
    }
    __syncthreads();
    if (__builtin_amdgcn_readfirstlane(rises) != 0) {
      if (tid == 0) vec[kScGamma] = -1.0f;
      __syncthreads();   // before the next turn writes `rises`
      continue;
    }
    if (w == 0) lr[lane] = exp2_of(Gs[63] - Gs[lane]) * rks[lane];   // read after the next barrier
    // the lane's rows and columns, read before the products are stored (the
    // compiler would read them again after every store)
    double Gt[4], Gc[4];
    float bt[4], rc[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w + 4 * q + r;
      Gt[r] = Gs[t];
      bt[r] = bs[t] * rks[t];
      Gc[r] = Gs[16 * r + n];
      rc[r] = rks[16 * r + n];
    }
    f32x4 diag = {0, 0, 0, 0};   // A's diagonal block w
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j <= w) {
        const int c = 16 * j + n;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * w + 4 * q + r;
          const float e = exp2_of(Gt[r] - Gc[j]) * rc[j];
          const float av = c < t ? bt[r] * e * kk[j][r] : 0.0f;
          if (j < w) As[t * kRowF + c] = av;
          else diag[r] = av;
          Ps[t * kRowF + c] = c <= t ? e * qk[j][r] : 0.0f;
        }
      }
    }
    // column n of the inverse of I + diagonal block w (the four lane groups
    // alike): x starts as column n of I; then for j = 0, 1, ...: x_i -= A_ij x_j
    // for all i > j at once, A_ij taken from the lane that has it
    f32x4 tcol[4];
    {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = i == n ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < 15; ++j) {
#pragma unroll
        for (int i = j + 1; i < 16; ++i) {
          const float aij = __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(
              static_cast<int>(__float_as_uint(diag[i & 3])), 16 * (i >> 2) + j)));
          x[i] = fmaf(-aij, x[j], x[i]);
        }
        __builtin_amdgcn_sched_barrier(0);   // keeps the column's 15 scalars at most alive
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) tcol[0][r] = q == 0 ? x[r] : q == 1 ? x[4 + r] : q == 2 ? x[8 + r] : x[12 + r];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) As[(16 * w + 4 * q + r) * kRowF + 16 * w + n] = tcol[0][r];
    __syncthreads();
    if (w == 3) {   // the wave with the fewest blocks of T and M: the block's vectors and scalars
      const double G = Gs[lane], last = Gs[63];
      const float bt = bs[lane], eg = exp2_of(G), left = exp2_of(last - G);
      vec[lane] = eg * rks[lane];
      vec[64 + lane] = eg;
      vec[128 + lane] = rqs[lane];
      // bounds on what the block makes of a state row of norm s and values up to
      // v (per state row), for the scales of the pairs: |R| <= v + gmax s,
      // |e^(G_last - G) rk D| <= dd ((1 + sg) v + gamma s), |S'| <= sg v + gamma s.
      // They hold because the factors e^g (I - beta k k^T) have norm 1 at most
      // (g <= 0, beta in [0, 2]) and rk <= 2^-12 (rows are scaled to a largest
      // value of 2^12 or more).  A decay below 2^-126 is 0 here, but not its
      // products in T R: bounds take it as 2^-126.
      const float gmax = wave_max(eg), dd = wave_max(bt) * 0x1p-12f;
      const float sg = wave_sum(bt * fmaxf(left, 0x1p-126f)), gamma = exp2_of(last);
      if (lane == 0) {
        vec[kScGamma] = gamma;
        vec[kScGmax] = gmax;
        vec[kScD] = dd;
        vec[kScS] = sg;
      }
    }
    auto rows = [&](const float* m, int i, int k) {   // operand rows of block (i, k)
      return *reinterpret_cast<const float4*>(m + (16 * i + n) * kRowF + 16 * k + 4 * q);
    };
#pragma unroll
    for (int d = 1; d < 4; ++d) {
      tcol[d] = f32x4{0, 0, 0, 0};
      if (w + d < 4) {
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < d; ++e) acc = mul16(rows(As, w + d, w + e), tcol[e], acc);
        const f32x4 t = mul16(rows(As, w + d, w + d), acc, f32x4{0, 0, 0, 0});
        tcol[d] = -t;
      }
    }
    f32x4 mcol[4];
    float tm = 0.0f, mm = 0.0f;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      mcol[d] = f32x4{0, 0, 0, 0};
      if (w + d < 4) {
#pragma unroll
        for (int e = 0; e <= d; ++e) mcol[d] = mul16(rows(Ps, w + d, w + e), tcol[e], mcol[d]);
      }
    }
    const float bc = bs[16 * w + n];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (w + d < 4) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * (w + d) + 4 * q + r;
          tcol[d][r] *= bc * lr[t];
          mcol[d][r] *= bc;
          // a non-finite query row must not set the scale of the others
          const float at = fabsf(tcol[d][r]), am = fabsf(mcol[d][r]);
          tm = fmaxf(tm, at <= 3e38f ? at : 0.0f);
          mm = fmaxf(mm, am <= 3e38f ? am : 0.0f);
        }
      }
    }
    tm = wave_max(tm);
    mm = wave_max(mm);
    if (lane == 0) {
      wmax[w][0] = tm;
      wmax[w][1] = mm;
    }
    __syncthreads();
    const Pow2 pt = pow2_scale(fmaxf(fmaxf(wmax[0][0], wmax[1][0]), fmaxf(wmax[2][0], wmax[3][0])));
    const Pow2 pm = pow2_scale(fmaxf(fmaxf(wmax[0][1], wmax[1][1]), fmaxf(wmax[2][1], wmax[3][1])));
    if (tid == 0) {
      vec[kScInvT] = pt.down;
      vec[kScInvM] = pm.down;
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (w + d < 4) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = (16 * (w + d) + 4 * q + r) * kRowF + 16 * w + n;
          As[at] = tcol[d][r] * pt.up;
          Ps[at] = mcol[d][r] * pm.up;
        }
      }
    }
    if (w & 1) {   // blocks (0, 1) and (2, 3) lie above the diagonal, inside a stored step
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int at = (16 * (w - 1) + 4 * q + r) * kRowF + 16 * w + n;
        As[at] = 0.0f;
        Ps[at] = 0.0f;
      }
    }
    __syncthreads();
    uint8_t* hd = ws + prefill_ws_heads(a) + (static_cast<size_t>(slot) * a.Hv + h) * kHeadBytes;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s <= (w >> 1)) {
        const int f = w < 2 ? w : 2 * w - 2 + s;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float* src = (m ? Ps : As) + (16 * w + n) * kRowF + 32 * s + 4 * q;
          const float4 x = *reinterpret_cast<const float4*>(src), y = *reinterpret_cast<const float4*>(src + 16);
          const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
          f16x8 hi, lo;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            _Float16 vh, vl;
            split16(v[j], vh, vl);
            hi[j] = vh;
            lo[j] = vl;
          }
          f16x8* out = reinterpret_cast<f16x8*>(hd + m * 12 * 1024 + f * 2048) + lane;
          out[0] = hi;
          out[64] = lo;
        }
      }
    }
  }
}

// One workgroup per (sequence, value head, 16 state rows), its sequence's
// blocks in order.  Wave w holds key columns 32w .. 32w+31 of the state rows
// (result tiles: lane's column = state row) and forms tile row w of R, D and O:
//   S pair -> LDS | K S^T, R pair -> LDS | T R = D pair -> LDS | S += D^T K.
// Each bar is a barrier, and what is not on this chain (Q S^T, M R, bounds,
// stores) stands where the wave would wait for LDS.  A block's operands are
// loaded as soon as the block before is done with theirs; loads return in
// order, so the values, which are needed first, are loaded two blocks ahead.
//
// The scales of the pairs need bounds on R, D and S' before those are known.
// With g <= 0 and beta in [0, 2] (what gates produce) they exist; in a block with
// another g or beta a state may grow by any factor and no scale of a whole block
// fits fp16.  From the first such block of a sequence and value head on, its
// workgroups go token by token in fp32 (33 us for 64 tokens instead of 1.95).
//
// 16 state rows to a workgroup: a tile of the matrix instruction, and the most
// workgroups.  With 32 rows a block's operands do not fit beside two tiles of
// results (8192 tokens, 32 heads of 128: 516 us in all with one wave per SIMD
// against 320, 1270 with spills).
//
// 8192 tokens, 32 value heads of 128: 250 us, 1.95 us a block, 139 TF/s of the
// formula's products.  Bound by the latency of a block's chain: 1.45 us a block
// for one value head alone (an LDS exchange, two to four dependent products and
// the conversions in each of the four parts), and beside that the reads of the
// operands, 73 KB a block and workgroup from L2 at 9.8 TB/s over the chip.  Two
// workgroups on a compute unit overlap: 1.2 us a block each where a batch has
// more than 256.
template <int ACT>
__global__ __launch_bounds__(256, 2) void k_gdn_scan(GdnArgs a, const uint8_t* __restrict__ ws) {
  __shared__ f16x8 sf[4][2][64];
  __shared__ f16x4 rf[2][2][64][2];
  __shared__ f16x4 df[2][2][64][2];
  __shared__ float ssum[4][16];   // per wave and state row: sum of squares of the scaled state
  __shared__ float vmax[4][16];   // per wave and state row: largest value of the next block
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // a sequence's workgroups are dealt to the eight dies in runs, so that the
  // workgroups that read one key head's operands share an L2
  const int slices = a.dv / 16, units = a.Hv * slices, run = (units + 7) / 8;
  const int b = blockIdx.y, i = blockIdx.x;
  const int unit = (i % 8) * run + i / 8;
  if (unit >= units) return;
  const int h = unit / slices, dv0 = (unit % slices) * 16;
  int t0, t1;
  seq_range(a, b, t0, t1);
  if (t0 == t1) return;
  if (t1 - t0 <= kShort && a.B != 1) return;   // k_gdn_tokens' part
  t0 = __builtin_amdgcn_readfirstlane(t0);
  t1 = __builtin_amdgcn_readfirstlane(t1);
  const int nblk = (t1 - t0 + kBlock - 1) / kBlock, slot0 = t0 / kBlock + b, hk = h / (a.Hv / a.Hk);
  const uint8_t* kp = ws + (static_cast<size_t>(slot0) * a.Hk + hk) * kKeyBytes;
  const uint8_t* hp = ws + prefill_ws_heads(a) + (static_cast<size_t>(slot0) * a.Hv + h) * kHeadBytes;
  const size_t kstep = a.Hk * kKeyBytes, hstep = a.Hv * kHeadBytes;
  auto mark = [&](int c) {   // of block c, below 0 where it goes token by token
    return *reinterpret_cast<const float*>(hp + static_cast<size_t>(min(c, nblk - 1)) * hstep + 24 * 1024 + 4 * kScGamma);
  };
  const float first_marks = mark(lane);
  // uniform bases and 32-bit lane offsets: rows 16w + 4q + r of a block
  const uint32_t row_el = static_cast<uint32_t>(a.Hv) * a.dv;
  const uint16_t* vbase = a.v + (static_cast<size_t>(t0 + 16 * w) * a.Hv + h) * a.dv;
  float* obase = a.o + (static_cast<size_t>(t0 + 16 * w) * a.Hv + h) * a.dv;
  const uint32_t el = 4u * q * row_el + dv0 + n;   // element of row 4q, state row of the lane

  float* sp = a.state + ((static_cast<size_t>(b) * a.Hv + h) * a.dv + dv0 + n) * kDK + 32 * w + 4 * q;
  f32x4 S[2] = {*reinterpret_cast<const f32x4*>(sp), *reinterpret_cast<const f32x4*>(sp + 16)};
  uint4 kf[4], qf[4], kt[4], th[2], tl[2], mh[2], ml[2];
  uint16_t va[4], vb[4];   // values of even and odd blocks
  float4 ev, rv;
  struct Scalars {
    float4 a;   // kScGamma .. kScGmax
    float2 b;   // kScD, kScS
    float4 eg;     // e^G rk of the lane's rows
  } sc0, sc1;      // of even and odd blocks
  const uint32_t lane16 = lane * 16;
  // an offset of 0 that the compiler takes for a lane's own: the scalars come
  // by vector loads, since a scalar load in flight makes every LDS wait wait for it
  uint32_t zero = 0;
  asm volatile("" : "+v"(zero));
  auto frag = [&](const uint8_t* p, uint32_t at) { return *reinterpret_cast<const uint4*>(p + (lane16 + at)); };
  auto vec4 = [&](const uint8_t* p, uint32_t at) {
    return *reinterpret_cast<const float4*>(p + (24 * 1024 + 64 * w + 16u * q + at));
  };
  auto load_scalars = [&](const uint8_t* ph, Scalars& sc) {
    sc.a = *reinterpret_cast<const float4*>(ph + (24 * 1024 + 4 * kScGamma + zero));
    sc.b = *reinterpret_cast<const float2*>(ph + (24 * 1024 + 4 * kScD + zero));
    sc.eg = vec4(ph, 0);
  };
  auto load_keys = [&](const uint8_t* pk) {
#pragma unroll
    for (int s = 0; s < 4; ++s) kf[s] = frag(pk + w * 4096, 1024 * s);
  };
  auto load_queries = [&](const uint8_t* pk) {
#pragma unroll
    for (int s = 0; s < 4; ++s) qf[s] = frag(pk + 16384 + w * 4096, 1024 * s);
  };
  auto load_t = [&](const uint8_t* ph) {
    const uint8_t* p = ph + (w < 2 ? w : 2 * w - 2) * 2048;
    th[0] = frag(p, 0);
    tl[0] = frag(p, 1024);
    if (w >= 2) {
      th[1] = frag(p, 2 * 1024);
      tl[1] = frag(p, 3 * 1024);
    }
  };
  auto load_m = [&](const uint8_t* ph) {
    const uint8_t* p = ph + 12288 + (w < 2 ? w : 2 * w - 2) * 2048;
    mh[0] = frag(p, 0);
    ml[0] = frag(p, 1024);
    if (w >= 2) {
      mh[1] = frag(p, 2 * 1024);
      ml[1] = frag(p, 3 * 1024);
    }
    ev = vec4(ph, 256);
    rv = vec4(ph, 512);
  };
  auto load_cols = [&](const uint8_t* pk) {
#pragma unroll
    for (int f = 0; f < 4; ++f) kt[f] = frag(pk + 32768 + w * 4096, 1024 * f);
  };
  auto load_values = [&](int c, uint16_t (&vv)[4]) {
    const uint16_t* p = vbase + static_cast<size_t>(c) * kBlock * row_el;
    if (t0 + (c + 1) * kBlock <= t1) {   // uniform
#pragma unroll
      for (int r = 0; r < 4; ++r) vv[r] = *(p + r * row_el + el);
    } else {   // rows past the end repeat the sequence's last token (masked at use)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = min(t0 + c * kBlock + 16 * w + 4 * q + r, t1 - 1);
        vv[r] = a.v[(static_cast<size_t>(t) * a.Hv + h) * a.dv + dv0 + n];
      }
    }
  };
  // masks the block's values and leaves their largest magnitude in LDS
  auto prepare_values = [&](int c, uint16_t (&vv)[4]) {
    const int left = t1 - (t0 + c * kBlock + 16 * w);   // uniform
    if (left < 16) {
#pragma unroll
      for (int r = 0; r < 4; ++r) vv[r] = 4 * q + r < left ? vv[r] : 0;
    }
    float m = 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(act_to_f32<ACT>(vv[r])));
    vmax[w][n] = col_max(m);   // the same from the four lanes of a column
  };
  load_values(0, va);
  load_scalars(hp, sc0);
  load_keys(kp);
  load_queries(kp);
  load_t(hp);
  load_m(hp);
  load_cols(kp);
  load_values(1, vb);

  // blocks before the first that goes token by token, 64 at a time (a test in
  // the blocks' loop makes it longer: 8192 tokens 358 us instead of 313)
  int end = t1 - t0 <= kShort ? 0 : nblk;
  for (int c = 0; c < end; c += 64) {
    const unsigned long long m = __ballot((c == 0 ? first_marks : mark(c + lane)) < 0.0f);
    if (m != 0) end = min(c + __ffsll(m) - 1, nblk);
  }
  end = __builtin_amdgcn_readfirstlane(end);
  if (end == 0) {
    run_tokens<ACT, 1>(a, b, h, t0, t1, dv0 + (tid >> 4));
    return;
  }
  // the largest values of the state rows
  {
    float m = 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) m = fmaxf(m, fmaxf(fabsf(S[0][r]), fabsf(S[1][r])));
    ssum[w][n] = col_max(m);
  }
  prepare_values(0, va);
  __syncthreads();
  // bound on the norm of the lane's state row; at first from its largest value
  // (128 elements: at most 11.4 times it), then from exact sums
  float bound = 11.4f * fmaxf(fmaxf(ssum[0][n], ssum[1][n]), fmaxf(ssum[2][n], ssum[3][n]));
  __syncthreads();

  auto block = [&](int c, uint16_t (&vv)[4], uint16_t (&vnext)[4], const Scalars& sc, Scalars& scnext) {
    const bool more = c + 1 < end;
    const uint8_t* kn = more ? kp + kstep : kp;
    const uint8_t* hn = more ? hp + hstep : hp;
    load_scalars(hn, scnext);
    const float gamma = sc.a.x, inv_t = sc.a.y, inv_m = sc.a.z, gmax = sc.a.w, dd = sc.b.x, sg = sc.b.y;
    const float gbound = fmaxf(gamma, 0x1p-126f);
    float inv_s, fd, fo, inv_d, vs[4], as[4];
    // S pair
    {
      const Pow2 p = pow2_scale(bound);
      inv_s = p.down;
      f16x8 hi, lo;
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = S[j >> 2][j & 3] * p.up;   // scaled: its square cannot overflow
        _Float16 vh, vl;
        split16(x, vh, vl);
        hi[j] = vh;
        lo[j] = vl;
        ss = fmaf(x, x, ss);
      }
      sf[w][0][lane] = hi;
      sf[w][1][lane] = lo;
      ssum[w][n] = col_sum(ss);
    }
    // scales of R and D from the bounds; V and e^G rk under R's scale
    {
      const float vm = fmaxf(fmaxf(vmax[0][n], vmax[1][n]), fmaxf(vmax[2][n], vmax[3][n]));
      const Pow2 pr = pow2_scale(fmaf(gmax, bound, vm)), pd = pow2_scale(dd * fmaf(gbound, bound, fmaf(sg, vm, vm)));
      fd = inv_t * pd.up * pr.down;   // in this order: nothing on the way leaves fp32's range
      fo = inv_m * pr.down;
      inv_d = pd.down;
      bound = sg * vm;   // the next block's, completed below
      const float at[4] = {sc.eg.x, sc.eg.y, sc.eg.z, sc.eg.w};
      // the two scales' product overflows only where every e^G of the block is
      // below fp32's normal numbers (and v is 0): a finite factor keeps 0 x it 0
      const float sr = fminf(inv_s * pr.up, 0x1.fffffep127f);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        vs[r] = act_to_f32<ACT>(vv[r]) * pr.up;
        as[r] = at[r] * sr;
      }
    }
    __syncthreads();
    // K S^T and the R pair
    f16x8 sh[4], sl[4];
    f32x4 X[2];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      sh[s] = sf[s][0][lane];
      sl[s] = sf[s][1][lane];
    }
    X[0] = X[1] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      X[0] = mfma(as_frag(kf[s]), sh[s], X[0]);
      X[1] = mfma(as_frag(kf[s]), sl[s], X[1]);
    }
    {
      f16x4 rh, rl;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        _Float16 vh, vl;
        split16(fmaf(-as[r], fmaf(kLoDown, X[1][r], X[0][r]), vs[r]), vh, vl);
        rh[r] = vh;
        rl[r] = vl;
      }
      rf[w >> 1][0][lane][w & 1] = rh;
      rf[w >> 1][1][lane][w & 1] = rl;
    }
    load_keys(kn);
    __syncthreads();
    // T R and the D pair; Q S^T meanwhile
    f16x8 rh[2], rl[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s <= (w >> 1)) {
        rh[s] = *reinterpret_cast<const f16x8*>(&rf[s][0][lane][0]);
        rl[s] = *reinterpret_cast<const f16x8*>(&rf[s][1][lane][0]);
      }
    }
    f32x4 Y = {0, 0, 0, 0}, Y1 = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      Y = mfma(as_frag(qf[s]), sh[s], Y);
      Y1 = mfma(as_frag(qf[s]), sl[s], Y1);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) Y[r] = fmaf(kLoDown, Y1[r], Y[r]);
    {
      f32x4 D0 = {0, 0, 0, 0}, D1 = {0, 0, 0, 0};
      D1 = mfma(as_frag(tl[0]), rh[0], D1);
      D0 = mfma(as_frag(th[0]), rh[0], D0);
      D1 = mfma(as_frag(th[0]), rl[0], D1);
      if (w >= 2) {
        D0 = mfma(as_frag(th[1]), rh[1], D0);
        D1 = mfma(as_frag(tl[1]), rh[1], D1);
        D1 = mfma(as_frag(th[1]), rl[1], D1);
      }
      f16x4 dh, dl;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        _Float16 vh, vl;
        split16(fmaf(kLoDown, D1[r], D0[r]) * fd, vh, vl);
        dh[r] = vh;
        dl[r] = vl;
      }
      df[w >> 1][0][lane][w & 1] = dh;
      df[w >> 1][1][lane][w & 1] = dl;
    }
    const float ss = (ssum[0][n] + ssum[1][n]) + (ssum[2][n] + ssum[3][n]);
    bound = fmaf(gbound * inv_s, __builtin_amdgcn_sqrtf(ss), bound);
    load_queries(kn);
    load_t(hn);
    if (more) prepare_values(c + 1, vnext);
    __syncthreads();
    // the new state; M R and the output meanwhile
    f16x8 dh[2], dl[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      dh[s] = *reinterpret_cast<const f16x8*>(&df[s][0][lane][0]);
      dl[s] = *reinterpret_cast<const f16x8*>(&df[s][1][lane][0]);
    }
    f32x4 O1 = mfma(as_frag(ml[0]), rh[0], f32x4{0, 0, 0, 0}), O = mfma(as_frag(mh[0]), rh[0], f32x4{0, 0, 0, 0});
    O1 = mfma(as_frag(mh[0]), rl[0], O1);
    if (w >= 2) {
      O1 = mfma(as_frag(ml[1]), rh[1], O1);
      O = mfma(as_frag(mh[1]), rh[1], O);
      O1 = mfma(as_frag(mh[1]), rl[1], O1);
    }
    f32x4 u[2], u1[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      u[m] = mfma(as_frag(kt[2 * m]), dh[0], f32x4{0, 0, 0, 0});
      u1[m] = mfma(as_frag(kt[2 * m]), dl[0], f32x4{0, 0, 0, 0});
      u[m] = mfma(as_frag(kt[2 * m + 1]), dh[1], u[m]);
      u1[m] = mfma(as_frag(kt[2 * m + 1]), dl[1], u1[m]);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        S[m][r] = fmaf(inv_d, fmaf(kLoDown, u1[m][r], u[m][r]), gamma * S[m][r]);
    const float et[4] = {ev.x, ev.y, ev.z, ev.w}, rt[4] = {rv.x, rv.y, rv.z, rv.w};
    float* op = obase + static_cast<size_t>(c) * kBlock * row_el;
    const int left = t1 - (t0 + c * kBlock + 16 * w);   // uniform
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)   // the row's norm first: its products are some 2^16 times the result
      v[r] = fmaf(rt[r] * Y[r], et[r] * inv_s, rt[r] * fmaf(kLoDown, O1[r], O[r]) * fo);
    if (left >= 16) {
#pragma unroll
      for (int r = 0; r < 4; ++r) *(op + r * row_el + el) = v[r];
    } else {
      uint32_t at = el;
      asm volatile("" : "+v"(at));   // or the compiler keeps the rows' addresses in registers
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (4 * q + r < left) op[r * row_el + at] = v[r];
    }
    load_cols(kn);
    load_m(hn);
    load_values(c + 2, vv);
    kp = kn;
    hp = hn;
  };
  for (int c = 0;;) {
    block(c, va, vb, sc0, sc1);
    if (++c == end) break;
    block(c, vb, va, sc1, sc0);
    if (++c == end) break;
  }
  *reinterpret_cast<f32x4*>(sp) = S[0];
  *reinterpret_cast<f32x4*>(sp + 16) = S[1];
  if (end < nblk) {
    __syncthreads();   // the rows are stored in parts of other lanes
    run_tokens<ACT, 1>(a, b, h, t0 + end * kBlock, t1, dv0 + (tid >> 4));
  }
}

size_t prefill_bytes(const moe_gdn_desc* d, int N) {
  return N <= kShort ? 256
                     : prefill_slots(d->batch, N) * (d->k_heads * kKeyBytes + d->v_heads * kHeadBytes);
}

// Up to so many workgroups of 16 state rows (two for each compute unit) every
// row has its own lanes: the chain of a token is shorter (16 tokens of 2
// sequences with 32 heads of 128: 16.6 us against 19.7 with four rows to a
// lane; of 4 sequences, past the limit: 24.5 against 21.2; of 64: 241 against 148).
constexpr int kFewRows = 512;
// With more blocks of tokens and value heads than the chip holds workgroups of
// k_gdn_blocks (four on each of 256 compute units), a workgroup takes two value
// heads of a key head, which share its loads and products; below, its turns only
// make the one round longer.  us in all, one head against two, 16 key and 32
// value heads of 128: 1024 tokens (512 blocks) 51.6 / 56.1, 2048 (1024) 82.8 /
// 86.4, 8 x 256 (1024) 80.4 / 84.2, 3000 (1500) 117 / 113, 4096 (2048) 152 / 144,
// 8 x 512 (2048) 144.5 / 144.9, 8192 (4096) 322 / 312; 4 and 16 heads: 4096
// (1024) 123 / 128, 8192 (2048) 234 / 230.
constexpr int kChipBlocks = 1024;

template <int ACT>
hipError_t launch_prefill(const GdnArgs& a, uint8_t* ws, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.N <= kShort || a.B > 1) {
    const int rows = a.Hv * (a.dv / 16);
    if (static_cast<int64_t>(rows) * a.B <= kFewRows)
      hipLaunchKernelGGL((k_gdn_tokens<ACT, 1>), dim3(rows, a.B), dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((k_gdn_tokens<ACT, 4>), dim3(a.Hv * ((a.dv + 63) / 64), a.B), dim3(256), 0, s, a);
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.N <= kShort) return e;
  const auto slots = static_cast<uint32_t>(prefill_slots(a.B, a.N));
  const int per = a.Hv / a.Hk % 2 == 0 && static_cast<int64_t>(a.N) / kBlock * a.Hv > kChipBlocks ? 2 : 1;
  hipLaunchKernelGGL(k_gdn_blocks<ACT>, dim3(slots, a.Hv / per), dim3(256), 0, s, a, ws, per);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int units = a.Hv * (a.dv / 16), run = (units + 7) / 8;
  hipLaunchKernelGGL(k_gdn_scan<ACT>, dim3(8 * run, a.B), dim3(256), 0, s, a, ws);
  return hipGetLastError();
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
  if (prefill_slots(d->batch, N) > kMaxSlots)
    return set_error(MOE_ESHAPE, "n_tokens=%d / 64 + batch=%d must be below 2^24", N, d->batch);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_gdn_prefill_workspace_bytes(const moe_gdn_desc* d, int32_t n_tokens, size_t* bytes) {
  const moe_status st = moe::check_prefill(d, n_tokens);
  if (st) return st;
  if (!bytes) return moe::set_error(MOE_EINVAL, "bytes is NULL");
  *bytes = moe::prefill_bytes(d, n_tokens);
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
  const size_t need = moe::prefill_bytes(d, n_tokens);
  if (!ws || !gp_aligned(ws, 256)) return set_error(MOE_EINVAL, "workspace must be a 256-byte aligned device pointer");
  if (ws_bytes < need) return set_error(MOE_EWORKSPACE, "workspace of %zu bytes < required %zu", ws_bytes, need);
  moe::GdnArgs a{seq_off, static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                 static_cast<const uint16_t*>(v), g, beta, state, o, q_scale, d->batch, n_tokens, d->k_heads,
                 d->v_heads, d->head_v_dim};
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const hipError_t e = d->act_dtype == MOE_BF16 ? moe::launch_prefill<MOE_BF16>(a, static_cast<uint8_t*>(ws), s)
                                                : moe::launch_prefill<MOE_F16>(a, static_cast<uint8_t*>(ws), s);
  if (e != hipSuccess) return set_error(MOE_EHIP, "Gated DeltaNet prefill kernel launch: %s", hipGetErrorString(e));
  return set_error(MOE_OK, "");
}
