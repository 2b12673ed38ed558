// Attention of one new token per sequence over the paged cache (see
// include/moe_attn.h).
//
// Keys and values are read once, by whom they are used: the queries of a key
// head (up to 16) are one side of a 16-wide matrix product and the keys the
// other, so a wave turns 32 keys from global memory into scores, weights and
// weighted values without LDS or other lanes' help:
//   scores   S^T = K Q^T: a lane's 16 bytes of a key row are the operand as they
//            come; the result leaves lane l with query l % 16 and keys 4 (l / 16) + i
//            of each group of 16, so the running maximum is the lane's own but
//            for two swaps across its four lanes
//   output   O^T = V^T P^T: those weights are the right operand as they are; the
//            left one is V^T, which the lane puts together from 8 values each of
//            its 8 keys (one byte permute for two values).  Column j of those
//            8 goes to product j, which so holds dimensions 8 m + j in row m, and
//            a lane ends with 32 neighbouring dimensions of its query.
// Weights enter as the sum of two 16-bit numbers (16 bits or more of precision):
// the matrix cores are idle for most of the time anyway.
//
// The work of a batch is the list of its tiles (128 keys of one sequence and
// key head, 32 to each of four waves), which the workgroups of one round of the
// chip share evenly, whatever the lengths are: a workgroup takes a run of tiles,
// which may begin and end within a sequence.  What it leaves unfinished goes to
// the workspace, and k_join adds it up.  Lengths are read on the device, so a
// captured call follows them.
//
// Bound by the read of keys and values.  One sequence of 262143 positions, 2 key
// heads of 256 (537 MB): 84 us here and 5 in k_join, 6.0 TB/s in all; a
// plain streaming read of 1 GiB reaches 5.8 to 6.0, and the counters show 537 MB.
// 64 sequences of up to 8192 (568 MB): 92 and 6.
// What carried it from 121 us: no register spills (one wave to a SIMD at 256
// dimensions, 102 to 90), one round of 256 workgroups (117 to 102), loads past
// the caches (121 to 117).  A few positions: 8.6 to 9.0 us, loads that wait for
// each other (length, page, keys).  256 sequences of up to 700: 51 in all, where
// the read takes 37: every unit of a few tiles ends in a merge of the waves with
// nothing under it.  Every workgroup reads all lengths, 64 at a time: 1024
// sequences of up to 100 take 77, 4096 take 291 (the reads 26 and 103).
#include "attn.h"

namespace moe {
namespace {

constexpr int kTileLog = 7, kTile = 1 << kTileLog;   // keys of a tile
constexpr int kChip = 256;                           // compute units

struct Part {   // an unfinished run: unit b * Hk + h (-1: none) and the workgroups that hold its parts
  int32_t unit, first, last, pad;
};
__host__ __device__ constexpr size_t ml_offset(int groups) { return sizeof(Part) * 2 * groups; }
__host__ __device__ constexpr size_t part_offset(int groups) { return ml_offset(groups) + sizeof(float2) * 2 * 16 * groups; }

int groups_of(int64_t batch, int kv_heads, int64_t capacity, int head_dim) {
  const int64_t units = batch * kv_heads, tiles = units * ((capacity + kTile - 1) >> kTileLog);
  // Two workgroups to a compute unit only where its registers hold them and there is a unit for each: 64 sequences of 4000
  // with 8 key heads of 128: 98 us against 104; with fewer units than compute units they only double the parts.
  const int most = head_dim < 256 && units > kChip ? 2 * kChip : kChip;
  return static_cast<int>(tiles < most ? tiles : most);
}

// Sum over the lanes up to this one.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t u = __shfl_up(v, m);
    v += lane >= m ? u : 0u;
  }
  return v;
}

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) >> kTileLog; }
// A unit (a sequence's key head) costs two for each tile and one for its begin
// and end (64 sequences of up to 8192: 98.6 us, without it 107); tiles that lie
// before position v of that.
__device__ __forceinline__ uint32_t cost_of(int len) { return len > 0 ? 2 * tiles_of(len) + 1 : 0; }
__device__ __forceinline__ int tile_at(uint32_t v, int n_tiles) { return min(static_cast<int>(v >> 1), n_tiles); }

// Run of workgroup w of the whole cost: the first `more` are one longer than `per`.
__device__ __forceinline__ uint32_t run_start(uint32_t w, uint32_t per, uint32_t more) { return w * per + min(w, more); }
__device__ __forceinline__ uint32_t run_of(uint32_t t, uint32_t per, uint32_t more) {
  const uint32_t big = more * (per + 1);
  return t < big ? t / (per + 1) : more + (t - big) / per;
}

// Sequences [64 c, 64 c + 64): this lane's length (0 behind the batch).
__device__ __forceinline__ int chunk_length(const AttnArgs& a, int c) {
  const int b = 64 * c + (threadIdx.x & 63);
  return b < a.B ? seq_length(a.length, b, a.max_pages, a.page_log) : 0;
}

// Keys and values are read once a step: they are not to push out of the caches what is read again.  64 sequences of 4000
// positions, 16 and 2 heads of 256: 90 us on pages of their own, 101 through the caches; 16 of 8000: 52 and 50.  Where all
// share their pages the caches would serve: 74 against 53, and 44 against 36; the table does not say so before it is read.
template <class T>
__device__ __forceinline__ T load_once(const uint8_t* p) {
  typedef uint32_t words __attribute__((ext_vector_type(sizeof(T) / 4)));
  return __builtin_bit_cast(T, __builtin_nontemporal_load(reinterpret_cast<const words*>(p)));
}

template <int ACT, int D>
struct Wave {
  static constexpr int kSteps = D / 32, kVec = D >= 128 ? 8 : 4, kBlocks = D / (16 * kVec);
  uint4 q[kSteps], k[2][kSteps];
  uint32_t v[2][4][kBlocks][kVec / 2];
  f32x4_t o[kBlocks][kVec];
  float m, l;

  // at: of each group of 16 keys, uniform; el: the lane's byte in it
  __device__ __forceinline__ void load_keys(const uint8_t* const (&at)[2], uint32_t el) {
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) k[g][s] = load_once<uint4>(at[g] + el + 64 * s);
  }
  __device__ __forceinline__ void load_values(const uint8_t* const (&at)[2], uint32_t el) {
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < kBlocks; ++n) {
          const uint8_t* p = at[g] + el + (2 * i * D + 256 * n);
          if constexpr (kVec == 8) {
            const uint4 w = load_once<uint4>(p);
            v[g][i][n][0] = w.x, v[g][i][n][1] = w.y, v[g][i][n][2] = w.z, v[g][i][n][3] = w.w;
          } else {
            const uint2 w = load_once<uint2>(p);
            v[g][i][n][0] = w.x, v[g][i][n][1] = w.y;
          }
        }
  }
  // scores of the 32 keys, in the exponent of 2; lane's keys 4 (lane / 16) + i of each group
  __device__ __forceinline__ void scores(float c, f32x4_t (&z)[2]) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      z[g] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) z[g] = mfma16<ACT>(k[g][s], q[s], z[g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[g][i] *= c;
    }
  }
  // keys from n[g] on of each group do not take part: what lies there may be anything
  __device__ __forceinline__ void mask(const int (&n)[2], f32x4_t (&z)[2]) {
    const int k0 = (threadIdx.x & 48) >> 2;
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool off = k0 + i >= n[g];
        z[g][i] = off ? -INFINITY : z[g][i];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int j = 0; j < kVec / 2; ++j) v[g][i][b][j] = off ? 0u : v[g][i][b][j];
      }
  }
  __device__ __forceinline__ void softmax(f32x4_t (&z)[2], uint4& hi, uint4& lo) {
    float top = m;
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, z[g][i]);
    top = quad_max(top);
    const float base = top == -INFINITY ? 0.0f : top;   // no key yet: weights of 0
    if (__any(top > m)) {
      const float f = __builtin_amdgcn_exp2f(m - base);
      l *= f;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int j = 0; j < kVec; ++j) o[b][j] *= f;
    }
    m = top;
    uint32_t h[4], r[4];
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float p0 = __builtin_amdgcn_exp2f(z[g][i] - base + kShift<ACT>);
        const float p1 = __builtin_amdgcn_exp2f(z[g][i + 1] - base + kShift<ACT>);
        l += p0 + p1;
        const uint32_t w = pack2<ACT>(p0, p1);
        h[2 * g + i / 2] = w;
        r[2 * g + i / 2] = pack2<ACT>(p0 - act_to_f32<ACT>(w & 0xFFFFu), p1 - act_to_f32<ACT>(w >> 16));
      }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(r[0], r[1], r[2], r[3]);
  }
  __device__ __forceinline__ void add_values(uint4 hi, uint4 lo) {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
        auto two = [&](int g, int i) { return __builtin_amdgcn_perm(v[g][i + 1][b][j >> 1], v[g][i][b][j >> 1], sel); };
        const uint4 t = make_uint4(two(0, 0), two(0, 2), two(1, 0), two(1, 2));
        o[b][j] = mfma16<ACT>(t, hi, o[b][j]);
        o[b][j] = mfma16<ACT>(t, lo, o[b][j]);
      }
  }
};

template <int ACT, int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_attn_decode(AttnArgs a, uint8_t* ws) {
  using W = Wave<ACT, D>;
  __shared__ float sm[4][16], sl[4][16];
  __shared__ __align__(16) float so[4][16][D];
  const int lane = threadIdx.x & 63, n16 = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = blockIdx.x, n_groups = gridDim.x;
  const int group = a.Hq / a.Hk;
  Part* parts = reinterpret_cast<Part*>(ws) + 2 * w;
  float2* part_ml = reinterpret_cast<float2*>(ws + ml_offset(n_groups)) + 2 * 16 * w;
  float* part_o = reinterpret_cast<float*>(ws + part_offset(n_groups)) + static_cast<size_t>(2 * 16 * D) * w;
  if (threadIdx.x < 2) parts[threadIdx.x].unit = -1;

  // this workgroup's run of tiles, and the sequence it begins in
  const int chunks = (a.B + 63) / 64;
  int chunk = 0, len = chunk_length(a, 0);
  uint32_t scan = wave_scan(cost_of(len)), before = 0;   // cost of a key head: up to this lane's sequence; before the chunk
  uint32_t seq_cost = __builtin_amdgcn_readlane(scan, 63);
  for (int c = 1; c < chunks; ++c) seq_cost += __builtin_amdgcn_readlane(wave_scan(cost_of(chunk_length(a, c))), 63);
  // runs of at least two, so that one that lies within a unit has a tile of it
  const uint32_t total = seq_cost * a.Hk, runs = min(static_cast<uint32_t>(n_groups), max(total >> 1, 1u));
  const uint32_t per = total / runs, more = total % runs;
  if (w >= static_cast<int>(runs) || total == 0) return;
  const uint32_t start = run_start(w, per, more), stop = run_start(w + 1, per, more);
  // (searches end with the batch also if lengths change under them)
  while ((before + __builtin_amdgcn_readlane(scan, 63)) * a.Hk <= start) {
    if (chunk + 1 == chunks) return;
    before += __builtin_amdgcn_readlane(scan, 63);
    len = chunk_length(a, ++chunk);
    scan = wave_scan(cost_of(len));
  }
  int at = __builtin_ctzll(__ballot((before + scan) * a.Hk > start));   // lane of the sequence

  // A segment: the run's tiles [t0, t1) of one sequence and key head.
  struct Segment {
    int b, h, length, t0, t1, n_tiles;
    uint32_t unit_start, unit_end, seq_end;
  };
  auto segment_at = [&](uint32_t v) {   // of the sequence in lane `at`
    Segment g;
    g.b = 64 * chunk + at, g.length = __builtin_amdgcn_readlane(len, at);
    g.n_tiles = tiles_of(g.length);
    const uint32_t cost = cost_of(g.length);
    g.seq_end = (before + __builtin_amdgcn_readlane(scan, at)) * a.Hk;
    const uint32_t seq_start = g.seq_end - cost * a.Hk;
    g.h = (v - seq_start) / cost;
    g.unit_start = seq_start + g.h * cost;
    g.unit_end = g.unit_start + cost;
    g.t0 = tile_at(v - g.unit_start, g.n_tiles);
    g.t1 = tile_at(stop - g.unit_start, g.n_tiles);
    return g;
  };
  auto segment_behind = [&](const Segment& g) {
    if (g.unit_end == g.seq_end) {   // on to the next sequence that has tiles
      uint64_t left = __ballot(len > 0) & (at == 63 ? 0ull : ~0ull << (at + 1));
      while (left == 0) {
        if (chunk + 1 == chunks) return Segment{g.b, g.h, 0, 0, 0, 0, stop, stop, stop};
        before += __builtin_amdgcn_readlane(scan, 63);
        len = chunk_length(a, ++chunk);
        scan = wave_scan(cost_of(len));
        left = __ballot(len > 0);
      }
      at = __builtin_ctzll(left);
    }
    return segment_at(g.unit_end);
  };

  const float c = a.scale * kLog2e;
  const uint8_t *kc = reinterpret_cast<const uint8_t*>(a.k), *vc = reinterpret_cast<const uint8_t*>(a.v);
  const uint32_t k_el = 2 * (n16 * D + 8 * quad), v_el = 2 * (4 * quad * D + W::kVec * n16);
  W s;
  Segment cur = segment_at(start);
  auto is_last = [&](const Segment& g) { return stop <= g.unit_end + 1; };   // of the next unit at most the begin
  if (cur.t0 == cur.t1) {   // all tiles of the unit lie before
    if (is_last(cur)) return;
    cur = segment_behind(cur);
    if (cur.t0 == cur.t1) return;
  }
  // Pages of this wave's groups of 16 keys, two a tile, 32 tiles at a time: one to a lane (-1: none).
  int pages = -1, n[2], n_next[2];   // keys of a tile's two groups
  size_t e[2];                       // their first bytes
  auto load_pages = [&](const Segment& g, int t) {
    const int pos = (t + (lane >> 1)) * kTile + 32 * wave + 16 * (lane & 1);
    const int id = pos < g.length ? a.table[static_cast<size_t>(g.b) * a.max_pages + (pos >> a.page_log)] : -1;
    pages = id < a.n_pages ? id : -1;
  };
  auto place = [&](const Segment& g, int t) {
    if (t > g.t0 && ((t - g.t0) & 31) == 0) load_pages(g, t);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int pos = t * kTile + 32 * wave + 16 * i, id = __builtin_amdgcn_readlane(pages, 2 * ((t - g.t0) & 31) + i);
      n_next[i] = id < 0 ? 0 : min(16, g.length - pos);
      e[i] = (((static_cast<size_t>(max(id, 0)) * a.Hk + g.h) << a.page_log) + (pos & ((1 << a.page_log) - 1))) * (2 * D);
    }
  };
  auto load_keys = [&]() {
    const uint8_t* const kp[2] = {kc + e[0], kc + e[1]};
    s.load_keys(kp, k_el);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto begin = [&](const Segment& g) {   // its pages, queries and first keys
    load_pages(g, g.t0);
    const uint16_t* qp = a.q + row_at(g.b, a.q_ts, g.h * group + min(n16, group - 1), a.q_hs) + 8 * quad;
#pragma unroll
    for (int i = 0; i < W::kSteps; ++i) s.q[i] = *reinterpret_cast<const uint4*>(qp + 32 * i);
    place(g, g.t0);
    load_keys();
  };
  begin(cur);
  for (;;) {
    s.m = -INFINITY, s.l = 0;
#pragma unroll
    for (int i = 0; i < W::kBlocks; ++i)
#pragma unroll
      for (int j = 0; j < W::kVec; ++j) s.o[i][j] = f32x4_t{0, 0, 0, 0};
    const bool whole = cur.t0 == 0 && cur.t1 == cur.n_tiles, last = is_last(cur);
    constexpr int kPieces = 16 * D / 1024;   // of four outputs, most that a thread has
    uint2 gates[kPieces];
    if (whole && a.gate) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int x = 4 * threadIdx.x + 1024 * i, row = x / D;
        if (row < group) gates[i] = *reinterpret_cast<const uint2*>(a.gate + row_at(cur.b, a.g_ts, cur.h * group + row, a.g_hs) + x % D);
      }
    }
    for (int t = cur.t0; t < cur.t1; ++t) {
      n[0] = n_next[0], n[1] = n_next[1];
      const uint8_t* const vp[2] = {vc + e[0], vc + e[1]};
      s.load_values(vp, v_el);
      __builtin_amdgcn_sched_barrier(0);   // all of them on their way before the keys are waited for
      f32x4_t z[2];
      s.scores(c, z);
      if (t + 1 < cur.t1) {
        place(cur, t + 1);
        load_keys();
      }
      if (min(n[0], n[1]) < 16) s.mask(n, z);
      uint4 hi, lo;
      s.softmax(z, hi, lo);
      s.add_values(hi, lo);
    }

    // the four waves' results together
    const float l = quad_sum(s.l);
    if (quad == 0) sm[wave][n16] = s.m, sl[wave][n16] = l;
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fmaxf(top, sm[i][n16]);
    const float f = __builtin_amdgcn_exp2f(s.m - (top == -INFINITY ? 0.0f : top));
    if (n16 < group) {
#pragma unroll
      for (int i = 0; i < W::kBlocks; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int j = 0; j < W::kVec; j += 4)
            *reinterpret_cast<float4*>(&so[wave][n16][128 * i + W::kVec * (4 * quad + r) + j]) =
                make_float4(s.o[i][j][r] * f, s.o[i][j + 1][r] * f, s.o[i][j + 2][r] * f, s.o[i][j + 3][r] * f);
    }
    __syncthreads();
    const int slot = cur.t0 > 0 ? 0 : 1;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at4 = 4 * threadIdx.x + 1024 * i, row = at4 / D, d = at4 % D;
      if (row >= group) break;
      float mx = -INFINITY, lsum = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) mx = fmaxf(mx, sm[u][row]);
      const float base = mx == -INFINITY ? 0.0f : mx;
      f32x4_t x = {0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        lsum = fmaf(sl[u][row], __builtin_amdgcn_exp2f(sm[u][row] - base), lsum);
        x += *reinterpret_cast<const f32x4_t*>(&so[u][row][d]);
      }
      if (whole) {
        x *= lsum != 0 ? 1.0f / lsum : 0.0f;
        store_row<ACT>(a, cur.b, cur.h * group + row, D, d, x, gates[i], lsum == 0);
      } else {
        *reinterpret_cast<f32x4_t*>(part_o + (slot * 16 + row) * D + d) = x;
        if (d == 0) part_ml[slot * 16 + row] = make_float2(mx, lsum);
      }
    }
    if (!whole && threadIdx.x == 0) {
      parts[slot] = Part{cur.b * a.Hk + cur.h, static_cast<int>(run_of(cur.unit_start + 1, per, more)),
                         static_cast<int>(run_of(cur.unit_end - 2, per, more)), 0};   // the runs that hold a tile of it
    }
    if (last) return;
    cur = segment_behind(cur);
    if (cur.t0 == cur.t1) return;
    begin(cur);
    __syncthreads();   // sm, sl and so are free again
  }
}

// Adds up the parts of units that several workgroups hold.  The workgroups of a
// unit share its outputs, four neighbouring ones to a piece: P of them take P
// parts each of a P-th of the pieces.  Also writes the zeros of sequences
// without tokens.
template <int ACT, int D>
__global__ __launch_bounds__(256) void k_join(AttnArgs a, const uint8_t* ws) {
  __shared__ float sx[256][6];
  const int w = blockIdx.x, n_groups = gridDim.x, group = a.Hq / a.Hk, tid = threadIdx.x;
  const Part* parts = reinterpret_cast<const Part*>(ws);
  const float2* ml = reinterpret_cast<const float2*>(ws + ml_offset(n_groups));
  const float* po = reinterpret_cast<const float*>(ws + part_offset(n_groups));
  const int pieces = group * D / 4;
  for (int slot = 0; slot < 2; ++slot) {
    const Part p = parts[2 * w + slot];
    if (p.unit < 0) continue;
    const int n = p.last - p.first + 1, i = w - p.first;
    const int from = static_cast<int64_t>(pieces) * i / n, to = static_cast<int64_t>(pieces) * (i + 1) / n;
    const int b = p.unit / a.Hk, h = p.unit % a.Hk;
    // threads of a piece: as many as leave all pieces of the share a place, up to 64
    int lanes = 64;
    while (lanes > 1 && lanes * (to - from) > 256) lanes >>= 1;
    for (int base = from; base < to; base += 256 / lanes) {
      const int piece = base + tid / lanes, row = 4 * piece / D, d = 4 * piece % D;
      float m = -INFINITY, l = 0;
      f32x4_t x = {0, 0, 0, 0};
      if (piece < to) {
        for (int u = p.first + tid % lanes; u <= p.last; u += lanes) {
          const size_t at = (2 * u + (u == p.first)) * 16 + row;
          const float2 v = ml[at];
          const f32x4_t y = *reinterpret_cast<const f32x4_t*>(po + at * D + d);
          const float top = fmaxf(m, v.x), z = top == -INFINITY ? 0.0f : top;
          const float f = __builtin_amdgcn_exp2f(m - z), g = __builtin_amdgcn_exp2f(v.x - z);
          l = l * f + v.y * g;
          x = x * f + y * g;
          m = top;
        }
      }
      sx[tid][0] = m, sx[tid][1] = l;
#pragma unroll
      for (int j = 0; j < 4; ++j) sx[tid][2 + j] = x[j];
      for (int step = 1; step < lanes; step <<= 1) {
        __syncthreads();
        float m2 = -INFINITY, l2 = 0;
        f32x4_t y = {0, 0, 0, 0};
        const bool mine = tid % (2 * step) == 0;
        if (mine) {
          m2 = sx[tid + step][0], l2 = sx[tid + step][1];
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = sx[tid + step][2 + j];
          const float top = fmaxf(m, m2), z = top == -INFINITY ? 0.0f : top;
          const float f = __builtin_amdgcn_exp2f(m - z), g = __builtin_amdgcn_exp2f(m2 - z);
          l = l * f + l2 * g;
          x = x * f + y * g;
          m = top;
          sx[tid][0] = m, sx[tid][1] = l;
#pragma unroll
          for (int j = 0; j < 4; ++j) sx[tid][2 + j] = x[j];
        }
      }
      if (tid % lanes == 0 && piece < to) {
        x *= l != 0 ? 1.0f / l : 0.0f;
        store_row<ACT>(a, b, h * group + row, D, d, x, gates_of(a, b, h * group + row, d), l == 0);
      }
      __syncthreads();
    }
  }
  for (int b = w; b < a.B; b += n_groups)
    if (seq_length(a.length, b, a.max_pages, a.page_log) == 0)
      for (int i = 8 * tid; i < a.Hq * D; i += 2048)
        *reinterpret_cast<uint4*>(a.o + static_cast<size_t>(b) * a.Hq * D + i) = make_uint4(0, 0, 0, 0);
}

template <int ACT, int D>
hipError_t launch(const AttnArgs& a, void* ws, hipStream_t s) {
  const int groups = groups_of(a.B, a.Hk, static_cast<int64_t>(a.max_pages) << a.page_log, D);
  hipLaunchKernelGGL((k_attn_decode<ACT, D>), dim3(groups), dim3(256), 0, s, a, static_cast<uint8_t*>(ws));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_join<ACT, D>), dim3(groups), dim3(256), 0, s, a, static_cast<const uint8_t*>(ws));
  return hipGetLastError();
}

}  // namespace

size_t attn_decode_bytes(const moe_attn_desc* d) {
  const int groups = groups_of(d->batch, d->kv_heads, static_cast<int64_t>(d->max_pages) * d->page_size, d->head_dim);
  return part_offset(groups) + sizeof(float) * 2 * 16 * d->head_dim * groups;
}

hipError_t launch_attn_decode(int act, int d, const AttnArgs& a, void* ws, hipStream_t s) {
  if (act == MOE_BF16)
    return d == 64 ? launch<2, 64>(a, ws, s) : d == 128 ? launch<2, 128>(a, ws, s) : launch<2, 256>(a, ws, s);
  return d == 64 ? launch<1, 64>(a, ws, s) : d == 128 ? launch<1, 128>(a, ws, s) : launch<1, 256>(a, ws, s);
}

}  // namespace moe
