// Dense products with int4 affine group-quantised weights (see
// include/moe_linear.h for the formula and the packed layout).
//
// On the matrix cores the weight operand is v = 1 + q/16, exact in fp16 and
// bf16 (two logic operations per pair of nibbles), so per group of columns
//   sum q x = 16 sum v x - 16 sum x,
//   y += 16 s (sum v x) + (b - 16 s) (sum x),
// with both sums in fp32; sum x comes from the same matrix instruction with
// an operand of ones.  Tokens are the tile's rows and weight rows its
// columns, so a lane needs the scale and bias of one weight row per tile.
#include <hip/hip_runtime.h>

#include "moe_common.h"
#include "moe_linear.h"

namespace moe {
moe_status set_error(moe_status code, const char* fmt, ...);

namespace {

bool lin_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int ACT>
__device__ __forceinline__ f32x4 mfma32(uint4 a, uint4 b, f32x4 c) {
  if constexpr (ACT == 2)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}
// q_pair of all four pairs of a word: one shift and one and-or each (the
// compiler does not form the and-or from two constants)
template <int ACT>
__device__ __forceinline__ uint4 v_operand(uint32_t w) {
  constexpr uint32_t mask = ACT == 2 ? 0x00780078u : 0x03C003C0u, one = ACT == 2 ? 0x3F803F80u : 0x3C003C00u;
  auto pair = [&](uint32_t t) {
    uint32_t r;
    asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(t), "s"(mask), "v"(one));
    return r;
  };
  if constexpr (ACT == 2) return make_uint4(pair(w << 3), pair(w >> 1), pair(w >> 5), pair(w >> 9));
  else return make_uint4(pair(w << 6), pair(w << 2), pair(w >> 2), pair(w >> 6));
}
template <int ACT>
__device__ __forceinline__ uint4 ones_operand() {
  constexpr uint32_t one = ACT == 2 ? 0x3F803F80u : 0x3C003C00u;
  return make_uint4(one, one, one, one);
}

template <int RES>
__device__ __forceinline__ void store_out(void* y, size_t i, float v) {
  if constexpr (RES == 3) static_cast<float*>(y)[i] = v;
  else static_cast<uint16_t*>(y)[i] = f32_to_act<RES>(v);
}

constexpr int kLinWaves = 8;    // waves of a workgroup, each on every 8th 64-column chunk
constexpr int kLinBatch = 4;    // chunks whose loads a wave issues together

// One workgroup: 32 weight rows (pair-tile blockIdx.x) x 16 TT tokens
// (blockIdx.y).  The waves split the columns; their fp32 partial tiles are
// added in wave order.  A wave issues all loads of its next 4 chunks before it
// uses one: with few tokens nothing else hides their latency.
//
// A vocabulary of 100003 rows, 2048 inputs, one token: 24 us, 115.6 MB at 4.8
// TB/s, bound by reading the weights.  8192 outputs for one token (9.5 MB): 4.1
// us in the kernel, bound by the latency of the launch, two dependent loads and the
// join; 64 tokens of 2048 outputs: 4.7 us.  From about 512 workgroups on it is
// bound by the conversions, which are repeated for every 16 TT tokens.
template <int ACT, int RES, int TT, bool G32>
__global__ __launch_bounds__(64 * kLinWaves) void k_linear(const uint8_t* __restrict__ packed,
                                                           const uint16_t* __restrict__ x, void* __restrict__ y, int T,
                                                           int N, int K, int G, uint64_t scale_off) {
  __shared__ float red[kLinWaves][TT * 8][64];
  const int lane = threadIdx.x & 63, n = lane & 15, kb = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int p = blockIdx.x, nc = K / 64, ng = K / G;
  const uint4* wq = reinterpret_cast<const uint4*>(packed + static_cast<uint64_t>(p) * nc * 1024) + lane;
  const uint8_t* sec = packed + scale_off;
  const uint16_t* xr[TT];
#pragma unroll
  for (int tt = 0; tt < TT; ++tt)   // rows past the last token read the last one; their results are not stored
    xr[tt] = x + static_cast<size_t>(min(static_cast<int>(blockIdx.y) * 16 * TT + 16 * tt + n, T - 1)) * K + 8 * kb;
  f32x4 acc[TT][2];
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) acc[tt][0] = acc[tt][1] = f32x4{0, 0, 0, 0};
  const uint4 ones = ones_operand<ACT>();
  for (int c0 = wave; c0 < nc; c0 += kLinWaves * kLinBatch) {
    uint4 w[kLinBatch], xv[kLinBatch][TT][2];
    ScaleBias sb[kLinBatch][G32 ? 2 : 1];
#pragma unroll
    for (int u = 0; u < kLinBatch; ++u) {
      const int c = min(c0 + u * kLinWaves, nc - 1);
      w[u] = wq[static_cast<size_t>(c) * 64];
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        xv[u][tt][0] = *reinterpret_cast<const uint4*>(xr[tt] + 64 * c);
        xv[u][tt][1] = *reinterpret_cast<const uint4*>(xr[tt] + 64 * c + 32);
      }
      if constexpr (G32) {
        sb[u][0] = load_sb(sec, p, ng, 2 * c, n);
        sb[u][1] = load_sb(sec, p, ng, 2 * c + 1, n);
      } else {
        sb[u][0] = load_sb(sec, p, ng, G == 128 ? c >> 1 : c, n);
      }
    }
#pragma unroll
    for (int u = 0; u < kLinBatch; ++u) {
      const int c = c0 + u * kLinWaves;
      if (c >= nc) break;   // wave-uniform
      const uint32_t ww[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
      f32x4 ga[TT], gb[TT], gx[TT];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const uint4 va = v_operand<ACT>(ww[ks]), vb = v_operand<ACT>(ww[2 + ks]);
        const bool fresh = G32 || ks == 0;
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const f32x4 zero = {0, 0, 0, 0};
          ga[tt] = mfma32<ACT>(xv[u][tt][ks], va, fresh ? zero : ga[tt]);
          gb[tt] = mfma32<ACT>(xv[u][tt][ks], vb, fresh ? zero : gb[tt]);
          gx[tt] = mfma32<ACT>(xv[u][tt][ks], ones, fresh ? zero : gx[tt]);
        }
        if (G32 || ks == 1) {
          const ScaleBias s = sb[u][G32 ? ks : 0];
          const float sa = 16.0f * s.sA, sB = 16.0f * s.sB, ba = s.bA - sa, bB = s.bB - sB;
#pragma unroll
          for (int tt = 0; tt < TT; ++tt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              acc[tt][0][i] = fmaf(sa, ga[tt][i], fmaf(ba, gx[tt][i], acc[tt][0][i]));
              acc[tt][1][i] = fmaf(sB, gb[tt][i], fmaf(bB, gx[tt][i], acc[tt][1][i]));
            }
        }
      }
    }
  }
#pragma unroll
  for (int tt = 0; tt < TT; ++tt)
#pragma unroll
    for (int i = 0; i < 8; ++i) red[wave][tt * 8 + i][lane] = acc[tt][i >> 2][i & 3];
  __syncthreads();
  for (int r = wave; r < TT * 8; r += kLinWaves) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kLinWaves; ++w) v += red[w][r][lane];
    const int t = static_cast<int>(blockIdx.y) * 16 * TT + 16 * (r >> 3) + 4 * kb + (r & 3);
    const int col = 32 * p + 16 * ((r >> 2) & 1) + n;
    if (t < T && col < N) store_out<RES>(y, static_cast<size_t>(t) * N + col, v);
  }
}

// Prompts: one workgroup of 8 waves per 128 tokens x 128 weight rows.  Wave
// (g, p) has pair-tile p of the rows, all 128 tokens (no weight is converted
// twice) and the 64-column chunks 2 i + g; the two halves are added at the end.
// Two waves per SIMD on different chunks let one wave's conversions and
// scalings run beside the other's matrix products.  A chunk's tokens are
// staged in LDS (two buffers, one barrier per pair of chunks; the 16-byte
// pieces of a row are xor-swizzled by the row so that the operand reads spread
// over the banks).  The staging threads also leave each token's sums over
// units of 64 columns (32 with groups of 32) in LDS; every 4 units the
// (b - 16 s) (sum x) term is added by fp32 matrix instructions (4 units deep),
// which costs a quarter of the main products' matrix time and spares 64
// multiply-adds a chunk.
//
// With groups of 32 twice the scales and multiply-adds do not fit: 256 registers
// and 36 spilled, 47 us against 29 (499 tokens, 2048 inputs, 8192 outputs).
//
// 499 tokens, 2048 inputs, 8192 outputs: 32 us, 525 TF/s.  Bound by one
// workgroup's chain per compute unit: conversions, products and scalings of a
// chunk add up where its two waves per SIMD do not overlap; with four waves (one
// per SIMD, every chunk) it took 36 to 39 us.
constexpr int kTileT = 128, kTileN = 128;
// v + v of the lane that the DPP control names (one instruction)
template <int kCtrl>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float(static_cast<uint32_t>(
                 __builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), kCtrl, 0xF, 0xF, true)));
}
template <int ACT, int RES, bool G32>
__global__ __launch_bounds__(512, 2) void k_linear_tile(const uint8_t* __restrict__ packed,
                                                        const uint16_t* __restrict__ x, void* __restrict__ y, int T,
                                                        int N, int K, int G, uint64_t scale_off) {
  constexpr int kUnits = G32 ? 2 : 1;             // units per chunk
  constexpr int kTT = kTileT / 16;
  __shared__ uint4 xs[2][2][kTileT * 8];          // [half][buffer][token][8 pieces of 16 bytes]
  __shared__ float sums[2][2][kTileT][5];         // [half][4 units' buffer][token][unit], padded
  const int tid = threadIdx.x & 255, lane = tid & 63, n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = wave >> 2;
  // The tiles, a row tile's token tiles one after the other, are dealt to the
  // eight dies in runs: each die has the same number of them, and a row tile's
  // lie on one die or a few (16384 tokens, 64 outputs 27 us; with row tile r on
  // die r mod 8 107, and 1152 outputs 137 against 210).
  const int nt = (T + kTileT - 1) / kTileT, tile = (blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8;
  const int r0 = tile / nt * (kTileN / 32), tok0 = tile % nt * kTileT;
  const int np = (N + 31) / 32, nc = K / 64, ng = K / G;
  if (r0 >= np) return;   // the grid is a multiple of 8 tiles
  const int p = r0 + (wave & 3);
  const int pc = min(p, np - 1);   // a wave without rows still stages
  const int nit = (nc + 1) / 2, mine = (nc + 1 - half) / 2;   // steps, and this half's chunks
  const uint8_t* wq = packed + static_cast<uint64_t>(pc) * nc * 1024 + half * 1024;
  const uint8_t* sec = packed + scale_off + static_cast<uint64_t>(pc) * ng * 128;
  // staging: the thread's piece of tokens tid/8 + 32 i
  const int st = tid >> 3, sp = tid & 7;
  const uint16_t* xsrc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    xsrc[i] = x + static_cast<size_t>(min(tok0 + st + 32 * i, T - 1)) * K + 64 * half + 8 * sp;
  // group of this half's unit u (its units run over its own chunks)
  auto group_of = [&](int u) {
    const int c = 2 * (u / kUnits) + half;
    return G32 ? 2 * c + (u & 1) : (G == 128 ? c >> 1 : c);
  };
  struct Loads {
    uint4 x[4], w;
    uint2 s[kUnits];   // [s_A, b_A, s_B, b_B] of the chunk's units
  } even, odd;
  auto load = [&](int i, Loads& l) {   // chunk i of this half (past the last: the last that exists)
    const int cc = max(min(i, mine - 1), 0), back = mine > 0 ? 0 : 1;   // without any chunk: chunk 0
#pragma unroll
    for (int m = 0; m < 4; ++m) l.x[m] = *reinterpret_cast<const uint4*>(xsrc[m] + 128 * cc - 64 * back);
    l.w = *reinterpret_cast<const uint4*>(wq + static_cast<size_t>(cc) * 2048 - 1024 * back + 16 * lane);
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
      l.s[u] = *reinterpret_cast<const uint2*>(sec + min(group_of(cc * kUnits + u), ng - 1) * 128 + 8 * n);
  };
  constexpr uint32_t one = ACT == 2 ? 0x3F803F80u : 0x3C003C00u;
  auto stage = [&](int i, const Loads& l) {   // pieces and unit sums of chunk i
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int t = st + 32 * m;
      xs[half][i & 1][t * 8 + (sp ^ (t & 7))] = l.x[m];
      float v = dot2_acc<ACT>(l.x[m].x, one, 0.0f);
      v = dot2_acc<ACT>(l.x[m].y, one, v);
      v = dot2_acc<ACT>(l.x[m].z, one, v);
      v = dot2_acc<ACT>(l.x[m].w, one, v);
      v = add_dpp<0x4E>(add_dpp<0xB1>(v));
      if constexpr (!G32) v = add_dpp<0x141>(v);
      const int u = i * kUnits + (G32 ? sp >> 2 : 0);
      sums[half][(u >> 2) & 1][t][u & 3] = v;   // the same from every thread of the unit
    }
  };
  f32x4 acc[kTT][2];
#pragma unroll
  for (int tt = 0; tt < kTT; ++tt) acc[tt][0] = acc[tt][1] = f32x4{0, 0, 0, 0};
  // units 4 j .. 4 j + 3 (those below `units`) of the (b - 16 s) (sum x) term;
  // its scales are loaded when unit 4 j begins
  uint2 sq = make_uint2(0, 0);
  auto add_sums = [&](int j, int units) {
    const bool on = 4 * j + q < units;
    const float ba = on ? f16_bits_to_f32(sq.x >> 16) - 16.0f * f16_bits_to_f32(sq.x & 0xFFFFu) : 0.0f;
    const float bb = on ? f16_bits_to_f32(sq.y >> 16) - 16.0f * f16_bits_to_f32(sq.y & 0xFFFFu) : 0.0f;
#pragma unroll
    for (int tt = 0; tt < kTT; ++tt) {
      float v = sums[half][j & 1][16 * tt + n][q];   // not yet written where !on
      v = on ? v : 0.0f;
      acc[tt][0] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, ba, acc[tt][0], 0, 0, 0);
      acc[tt][1] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, bb, acc[tt][1], 0, 0, 0);
    }
  };
  // values and weights are loaded two steps ahead: a step's products take less
  // time than a load from L2
  auto step = [&](int i, Loads& cur, Loads& next) {
    const uint32_t ww[4] = {cur.w.x, cur.w.y, cur.w.z, cur.w.w};
    uint4 va[2], vb[2];
    float sa[kUnits], sB[kUnits];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      va[ks] = v_operand<ACT>(ww[ks]);
      vb[ks] = v_operand<ACT>(ww[2 + ks]);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      sa[u] = 16.0f * f16_bits_to_f32(cur.s[u].x & 0xFFFFu);
      sB[u] = 16.0f * f16_bits_to_f32(cur.s[u].y & 0xFFFFu);
    }
    // This step's registers are free (its tokens lie in LDS).  A use of them
    // that the compiler moved behind the loads would make it load into others
    // and wait for them at the loop's end to copy them: opaque to it.
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      asm volatile("" : "+v"(va[ks].x), "+v"(va[ks].y), "+v"(va[ks].z), "+v"(va[ks].w));
      asm volatile("" : "+v"(vb[ks].x), "+v"(vb[ks].y), "+v"(vb[ks].z), "+v"(vb[ks].w));
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) asm volatile("" : "+v"(sa[u]), "+v"(sB[u]));
    __builtin_amdgcn_sched_barrier(0);
    load(i + 2, cur);
    if (((i * kUnits) & 3) == 0)
      sq = *reinterpret_cast<const uint2*>(sec + min(group_of(i * kUnits + q), ng - 1) * 128 + 8 * n);
    if (i < mine) {   // uniform: the second half may have one chunk less
      const f32x4 zero = {0, 0, 0, 0};
#pragma unroll
      for (int tt = 0; tt < kTT; ++tt) {
        const int t = 16 * tt + n;
        const uint4 x0 = xs[half][i & 1][t * 8 + (q ^ (t & 7))], x1 = xs[half][i & 1][t * 8 + ((4 + q) ^ (t & 7))];
        f32x4 ga = mfma32<ACT>(x0, va[0], zero), gb = mfma32<ACT>(x0, vb[0], zero);
        if constexpr (G32) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            acc[tt][0][r] = fmaf(sa[0], ga[r], acc[tt][0][r]);
            acc[tt][1][r] = fmaf(sB[0], gb[r], acc[tt][1][r]);
          }
          ga = gb = zero;
        }
        ga = mfma32<ACT>(x1, va[1], ga);
        gb = mfma32<ACT>(x1, vb[1], gb);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[tt][0][r] = fmaf(sa[kUnits - 1], ga[r], acc[tt][0][r]);
          acc[tt][1][r] = fmaf(sB[kUnits - 1], gb[r], acc[tt][1][r]);
        }
      }
      const int done = (i + 1) * kUnits;   // units whose sums are staged and visible
      if ((done & 3) == 0 || i + 1 == mine) add_sums((done - 1) >> 2, done);
    }
    if (i + 1 < nit) {
      stage(i + 1, next);
      __syncthreads();
    }
  };
  load(0, even);
  load(1, odd);
  stage(0, even);
  __syncthreads();
  // (a loop with one exit: with a second one in its middle the compiler has
  // every step wait for the loads of the step before)
  for (int i = 0; i + 1 < nit; i += 2) {
    step(i, even, odd);
    step(i + 1, odd, even);
  }
  if (nit & 1) step(nit - 1, even, odd);
  // half g keeps tile g of the pair and hands the other one over
  __syncthreads();
  float* ex = reinterpret_cast<float*>(&xs[0][0][0]) + wave * (kTT * 4 * 64);   // 8 waves x 8 KB
#pragma unroll
  for (int tt = 0; tt < kTT; ++tt)
#pragma unroll
    for (int r = 0; r < 4; ++r) ex[(tt * 4 + r) * 64 + lane] = half ? acc[tt][0][r] : acc[tt][1][r];
  __syncthreads();
  const float* other = reinterpret_cast<const float*>(&xs[0][0][0]) + (wave ^ 4) * (kTT * 4 * 64);
  const int col = 32 * p + 16 * half + n;
  if (p >= np || col >= N) return;
#pragma unroll
  for (int tt = 0; tt < kTT; ++tt)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = tok0 + 16 * tt + 4 * q + r;
      const float o = other[(tt * 4 + r) * 64 + lane];
      const float v = half ? o + acc[tt][1][r] : acc[tt][0][r] + o;   // even chunks' sum first
      if (t < T) store_out<RES>(y, static_cast<size_t>(t) * N + col, v);
    }
}

// One thread per packed word (values), then one per 8-byte scale entry.  Once
// per weight: 115.6 MB in 76 us (3.0 TB/s of reads and writes, 114 us into fresh
// memory; the words of a row are read 4 bytes at a time from 16 rows).  Workgroups in two dimensions: the
// largest weights need more than the 2^32 threads that one holds.
constexpr uint64_t kPackRow = 1 << 20;   // workgroups in the first dimension, at most
__global__ __launch_bounds__(256) void k_linear_pack(const uint32_t* __restrict__ q, const uint16_t* __restrict__ s,
                                                     const uint16_t* __restrict__ b, uint8_t* __restrict__ packed,
                                                     int N, int K, int G, uint64_t n_words, uint64_t n_scales) {
  const uint64_t i = (static_cast<uint64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  if (i < n_words) {
    const int wd = i & 3, lane = (i >> 2) & 63;
    const uint64_t blk = i >> 8;
    const int nc = K / 64, c = static_cast<int>(blk % nc);
    const int64_t row = static_cast<int64_t>(blk / nc) * 32 + 16 * (wd >> 1) + (lane & 15);
    uint32_t out = 0;
    if (row < N) {
      const uint32_t in = q[row * (K / 8) + 8 * c + 4 * (wd & 1) + (lane >> 4)];
#pragma unroll
      for (int j = 0; j < 8; ++j) out |= ((in >> (4 * j)) & 15u) << (4 * ((j >> 1) + 4 * (j & 1)));
    }
    reinterpret_cast<uint32_t*>(packed)[i] = out;
  } else if (i - n_words < n_scales) {
    const uint64_t k = i - n_words;
    const int n = k & 15, ng = K / G;
    const uint64_t pg = k >> 4;
    const int g = static_cast<int>(pg % ng);
    const int64_t ra = static_cast<int64_t>(pg / ng) * 32 + n, rb = ra + 16;
    uint32_t lo = 0, hi = 0;
    if (ra < N) lo = s[ra * ng + g] | (static_cast<uint32_t>(b[ra * ng + g]) << 16);
    if (rb < N) hi = s[rb * ng + g] | (static_cast<uint32_t>(b[rb * ng + g]) << 16);
    reinterpret_cast<uint2*>(packed + 4 * n_words)[k] = make_uint2(lo, hi);
  }
}

constexpr int kLinMaxIn = 65536, kLinMaxOut = 1 << 20, kLinMaxTokens = 1 << 20;
constexpr int kLinMaxTiles = (1 << 23) - 8;   // a grid holds fewer than 2^32 threads, 512 per tile

bool linear_shape_ok(int K, int N, int G) {
  return K >= 64 && K <= kLinMaxIn && K % 64 == 0 && N >= 1 && N <= kLinMaxOut &&
         (G == 32 || G == 64 || G == 128) && K % G == 0;
}
uint64_t padded_rows(int N) { return (static_cast<uint64_t>(N) + 31) / 32 * 32; }

template <int ACT, int RES>
hipError_t launch_linear(const moe_linear_desc* d, const uint8_t* packed, const uint16_t* x, int T, void* y,
                         hipStream_t s) {
  const int K = d->in_dim, N = d->out_dim, G = d->group_size;
  const uint64_t off = padded_rows(N) * K / 2;
  const int np = (N + 31) / 32, nt = (T + kTileT - 1) / kTileT, nr = (N + kTileN - 1) / kTileN;
  // A round of up to 256 tiles (one per compute unit, full or not) takes as long
  // as some 1600 workgroups of k_linear (2560 with groups of 32, where the tile
  // kernel spills), and the kernel that needs less is taken.  us, tiles against
  // k_linear, 2048 inputs:
  //   128 tokens, 8192 outputs (1024 workgroups, 1 round)   26.5 / 18.8, groups of 32 43.8 / 21.3
  //   128 tokens, 12603 outputs (1576, 1)                   26.6 / 31.2
  //   128 tokens, 16384 outputs (2048, 1)                   27.0 / 34.7, groups of 32 44.7 / 37.6
  //   384 tokens, 6684 outputs (2508, 1)                    groups of 32 44.5 / 46.1
  //   4096 tokens, 512 outputs (2048, 1)                    27.6 / 35.0, groups of 32 45.4 / 37.3
  //   48 tokens, 65536 outputs (4096, 2)                    50.5 / 56.7, groups of 32 85.9 / 62.9
  //   32 tokens, 65536 outputs (2048, 2)                    50.1 / 35.0, groups of 32 85.7 / 37.2
  //   64 tokens, 151936 outputs (9496, 5)                   130 / 158, groups of 32 225 / 178
  // and with 8192 inputs, 200 tokens, 8621 outputs (1890, 1) 91.6 / 122; with 512
  // inputs, 160 tokens, 10078 outputs (1575, 1) 10.7 / 11.9.
  const int64_t wgs = static_cast<int64_t>(np) * ((T + 31) / 32), rounds = (static_cast<int64_t>(nt) * nr + 255) / 256;
  if (wgs > rounds * (G == 32 ? 2560 : 1600)) {
    const dim3 grid((nr * nt + 7) / 8 * 8), block(512);
    if (G == 32) hipLaunchKernelGGL((k_linear_tile<ACT, RES, true>), grid, block, 0, s, packed, x, y, T, N, K, G, off);
    else hipLaunchKernelGGL((k_linear_tile<ACT, RES, false>), grid, block, 0, s, packed, x, y, T, N, K, G, off);
    return hipGetLastError();
  }
  const int tiles = (T + 15) / 16;
  // 16 tokens to a workgroup up to two workgroups for each compute unit, then
  // 32, which convert a weight half as often (us, 16 against 32; 2048 inputs):
  // 512 workgroups of 16 tokens 6.6 / 6.8 (128 tokens, 2048 outputs) and 6.4 /
  // 6.6 (32 tokens, 8192), 320 of them 6.4 / 6.5, 256 of them 4.7 / 6.5; 1024
  // of them 11.2 / 10.7 and 10.9 / 10.4.
  const int tt = tiles == 1 || static_cast<int64_t>(np) * tiles <= 512 ? 1 : 2;
  const dim3 grid(np, (tiles + tt - 1) / tt), block(64 * kLinWaves);
#define LIN(TT)                                                                                             \
  do {                                                                                                      \
    if (G == 32) hipLaunchKernelGGL((k_linear<ACT, RES, TT, true>), grid, block, 0, s, packed, x, y, T, N, K, G, off); \
    else hipLaunchKernelGGL((k_linear<ACT, RES, TT, false>), grid, block, 0, s, packed, x, y, T, N, K, G, off);        \
  } while (0)
  if (tt == 1) LIN(1);
  else LIN(2);
#undef LIN
  return hipGetLastError();
}
template <int ACT>
hipError_t launch_linear_res(const moe_linear_desc* d, const uint8_t* packed, const uint16_t* x, int T, void* y,
                             hipStream_t s) {
  switch (d->out_dtype) {
    case MOE_F16: return launch_linear<ACT, MOE_F16>(d, packed, x, T, y, s);
    case MOE_BF16: return launch_linear<ACT, MOE_BF16>(d, packed, x, T, y, s);
    default: return launch_linear<ACT, MOE_F32>(d, packed, x, T, y, s);
  }
}

}  // namespace
}  // namespace moe

extern "C" uint64_t moe_linear_bytes(int32_t K, int32_t N, int32_t G) {
  if (!moe::linear_shape_ok(K, N, G)) return 0;
  const uint64_t rows = moe::padded_rows(N);
  return rows * K / 2 + 4 * rows * (K / G);
}

extern "C" moe_status moe_linear_pack(int32_t K, int32_t N, int32_t G, const uint32_t* q, const uint16_t* scale,
                                      const uint16_t* bias, uint8_t* packed, moe_stream stream) {
  using moe::set_error;
  if (!moe::linear_shape_ok(K, N, G)) return set_error(MOE_ESHAPE, "unsupported linear in=%d out=%d group=%d", K, N, G);
  if (!q || !scale || !bias) return set_error(MOE_EINVAL, "q, scale and bias are required");
  if (!moe::lin_aligned(q, 4) || !packed || !moe::lin_aligned(packed, 256))
    return set_error(MOE_EINVAL, "q must be 4-byte and packed a 256-byte aligned device pointer");
  const uint64_t rows = moe::padded_rows(N), nw = rows * K / 8, ns = rows / 2 * (K / G);
  const uint64_t blocks = (nw + ns + 255) / 256;
  const uint64_t ny = (blocks + moe::kPackRow - 1) / moe::kPackRow;
  const dim3 grid(static_cast<uint32_t>((blocks + ny - 1) / ny), static_cast<uint32_t>(ny));
  hipLaunchKernelGGL(moe::k_linear_pack, grid, dim3(256), 0, reinterpret_cast<hipStream_t>(stream), q, scale, bias,
                     packed, N, K, G, nw, ns);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(MOE_EHIP, "linear pack kernel launch: %s", hipGetErrorString(e));
  return set_error(MOE_OK, "");
}

extern "C" moe_status moe_linear_forward(const moe_linear_desc* d, const uint8_t* packed, const void* x, int32_t T,
                                         void* y, moe_stream stream) {
  using moe::set_error;
  if (!d) return set_error(MOE_EINVAL, "desc is NULL");
  if (!moe::linear_shape_ok(d->in_dim, d->out_dim, d->group_size))
    return set_error(MOE_ESHAPE, "unsupported linear in=%d out=%d group=%d", d->in_dim, d->out_dim, d->group_size);
  if (d->act_dtype != MOE_F16 && d->act_dtype != MOE_BF16)
    return set_error(MOE_EINVAL, "act_dtype=%d is not MOE_F16/MOE_BF16", d->act_dtype);
  if (d->out_dtype != MOE_F16 && d->out_dtype != MOE_BF16 && d->out_dtype != MOE_F32)
    return set_error(MOE_EINVAL, "out_dtype=%d is not MOE_F16/MOE_BF16/MOE_F32", d->out_dtype);
  if (T < 0 || T > moe::kLinMaxTokens) return set_error(MOE_ESHAPE, "n_tokens=%d must be in [0, %d]", T, moe::kLinMaxTokens);
  if (static_cast<int64_t>((T + moe::kTileT - 1) / moe::kTileT) * ((d->out_dim + moe::kTileN - 1) / moe::kTileN) >
      moe::kLinMaxTiles)
    return set_error(MOE_ESHAPE, "n_tokens=%d x out_dim=%d is more than 2^23 - 8 tiles of 128 x 128", T, d->out_dim);
  if (T == 0) return set_error(MOE_OK, "");
  if (!packed || !moe::lin_aligned(packed, 256))
    return set_error(MOE_EINVAL, "packed must be a 256-byte aligned device pointer");
  if (!x || !moe::lin_aligned(x, 16)) return set_error(MOE_EINVAL, "x must be a 16-byte aligned device pointer");
  if (!y || !moe::lin_aligned(y, d->out_dtype == MOE_F32 ? 4 : 2))
    return set_error(MOE_EINVAL, "y must be a device pointer aligned to its type");
  const auto* xb = static_cast<const uint16_t*>(x);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const hipError_t e = d->act_dtype == MOE_BF16 ? moe::launch_linear_res<MOE_BF16>(d, packed, xb, T, y, s)
                                                : moe::launch_linear_res<MOE_F16>(d, packed, xb, T, y, s);
  if (e != hipSuccess) return set_error(MOE_EHIP, "linear kernel launch: %s", hipGetErrorString(e));
  return set_error(MOE_OK, "");
}
