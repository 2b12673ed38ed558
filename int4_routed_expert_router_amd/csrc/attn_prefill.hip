// Causal attention of several new tokens per sequence over the paged cache
// (see include/moe_attn.h).
//
// A unit of work is a key head's queries of a block of neighbouring tokens: its
// 256 rows are (token, query head of the group), so that grouped heads share
// every key that is loaded, and up to 256 rows share a tile of 64 keys in LDS.
// Each wave holds the queries and the accumulators of its rows in registers:
//   scores   S^T = K Q^T by 32 x 32 x 16 products; the result leaves lane l with
//            row l % 32 and 16 of 32 keys, so a row's maximum and sum are the
//            lane's own but for one swap with lane l ^ 32
//   output   O^T = V^T P^T: those weights are the right operand as they lie;
//            V^T comes from LDS by transposing reads
// Weights are rounded to the 16-bit type (half a step each, unbiased; their sum
// is that of the unrounded ones in fp32), as the product's operand has to be.
// Tiles go from global memory straight to LDS, one ahead of the one in use; the
// 16-byte pieces of a row are stored in an order that depends on the key, so
// that the reads of a product fall on different banks.
//
// Units are of very different length (causal blocks, ragged sequences).  Those of
// more than an even share of all tiles are cut into chunks of that size, whose
// parts k_attn_join adds up; where there are enough units none is cut.  Every
// workgroup works out its unit from the lengths and offsets on the device.
#include "attn.h"

namespace moe {
namespace {

constexpr int kRows = 256;                  // rows of a unit
constexpr int kKeys = 64, kKeysLog = 6;     // keys of a tile
constexpr int kShareLog = 8;                // shares of the whole: the compute units
constexpr int kSlots = 2 << kShareLog;      // chunks of cut units: below 2 tiles / share size
constexpr int kMinChunk = 4;                // tiles
constexpr int kMaxUnits = 1 << 22;
constexpr int kAhead = 4;                   // operands in flight from LDS

struct Unit {     // uniform
  int b, h, begin, n, base;   // sequence, key head, first row, tokens, positions before them (may be negative)
  int j, chunk, chunks;       // block, chunk of how many
  int slot;                   // of the chunk's part; -1: not cut
  int size;                   // tiles of a chunk
};
struct Part {
  Unit u;
  int pad[6];
};
struct Header {
  int parts;
  int pad[63];
};

template <int D>
struct Shape {
  // 32-row tiles and waves: registers of accumulators and queries are the bound
  // (192 of the 256 that two waves on a SIMD have)
  static constexpr int kTiles = D == 256 ? 1 : 2, kWaves = kRows / (32 * kTiles);
  static constexpr int kTileBytes = kKeys * D * 2;
};

__host__ __device__ inline int rows_held(int N, int group) {   // rows of a unit's part in the workspace
  const int64_t r = (static_cast<int64_t>(N) * group + 31) / 32 * 32;
  return r < kRows ? static_cast<int>(r) : kRows;
}
__host__ __device__ inline size_t ml_at() { return sizeof(Header) + sizeof(Part) * kSlots; }
__host__ __device__ inline size_t o_at(int rows) { return ml_at() + sizeof(float2) * kSlots * rows; }

// sum over i < n of floor((a i + b) / m); a, b >= 0, a n + b + m < 2^31 after a is reduced
__device__ uint64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  uint64_t r = 0;
  while (n > 0) {
    if (a >= m) {
      r += static_cast<uint64_t>(n) * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      r += static_cast<uint64_t>(n) * (b / m);
      b %= m;
    }
    const uint32_t top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return r;
}

// One lane's sequence: its blocks of tpb tokens and their chunks of m keys.
struct Seq {
  int begin, n, base, first, full, blocks;   // first block that sees a key; blocks of tpb tokens; all blocks
  __device__ __forceinline__ void load(const AttnArgs& a, int b, int tpb) {
    begin = n = base = first = full = blocks = 0;
    if (b >= a.B) return;
    int end;
    seq_rows(a.off, b, a.N, begin, end);
    n = end - begin;
    if (n == 0) return;
    base = seq_length(a.length, b, a.max_pages, a.page_log) - n;
    full = n / tpb;
    blocks = (n + tpb - 1) / tpb;
    first = base < 0 ? min(-base / tpb, blocks) : 0;
  }
  // chunks of blocks [0, j)
  __device__ __forceinline__ uint64_t before(int j, int tpb, uint32_t m) const {
    uint64_t r = floor_sum(max(min(j, full) - first, 0), m, tpb, max(base + (first + 1) * tpb, 0) + m - 1);
    if (j > full && blocks > full) r += (static_cast<uint32_t>(max(base + n, 0)) + m - 1) / m;
    return r;
  }
  // blocks that are one chunk or none
  __device__ __forceinline__ int uncut(int tpb, uint32_t m) const {
    if (base + n <= static_cast<int>(m)) return blocks;
    return max(min(static_cast<int>(static_cast<int>(m) - base) / tpb, full), 0);
  }
};

__device__ __forceinline__ uint64_t wave_scan64(uint64_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint64_t u = __shfl_up(v, m);
    v += lane >= m ? u : 0ull;
  }
  return v;
}
__device__ __forceinline__ uint64_t lane64(uint64_t v, int i) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(v), i);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(v >> 32), i);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// The item-th chunk of the call (wave-uniform; b < 0: there is none): sequences
// in order, in each the last block first (the longest, and the cut ones), its
// chunks, and the key heads innermost, so that neighbours in the order, which
// run on different dies, leave each die its own heads.
__device__ Unit find_unit(const AttnArgs& a, uint32_t item, int tpb, int* n_parts) {
  const int lane = threadIdx.x & 63, chunks = (a.B + 63) / 64;
  Seq s;
  uint64_t tiles = 0;
  for (int c = 0; c < chunks; ++c) {
    s.load(a, 64 * c + lane, tpb);
    tiles += lane64(wave_scan64(s.before(s.blocks, tpb, kKeys)), 63);
  }
  // above an even share, so that cut units' chunks number less than twice the shares
  const uint64_t share = (tiles * a.Hk >> kShareLog) + 1;
  const int size = share < kMinChunk ? kMinChunk : share > (1 << 24) ? 1 << 24 : static_cast<int>(share);
  const uint32_t m = static_cast<uint32_t>(size) << kKeysLog;
  Unit u;
  u.b = -1;
  u.size = size;
  uint64_t items = 0;
  int parts = 0;
  for (int c = 0; c < chunks; ++c) {
    if (chunks > 1) s.load(a, 64 * c + lane, tpb);
    const uint64_t own = s.before(s.blocks, tpb, m);
    const int cut = static_cast<int>(own) - max(s.uncut(tpb, m) - s.first, 0);   // chunks of cut units, a head
    const int own_parts = s.uncut(tpb, m) < s.blocks ? cut : 0;
    const uint64_t upto = wave_scan64(own);
    const int parts_upto = static_cast<int>(wave_scan64(own_parts));
    const uint64_t hit = __ballot((items + upto) * a.Hk > item);
    if (u.b < 0 && hit) {
      const int at = __builtin_ctzll(hit);
      u.b = 64 * c + at;
      u.begin = __builtin_amdgcn_readlane(s.begin, at);
      u.n = __builtin_amdgcn_readlane(s.n, at);
      u.base = __builtin_amdgcn_readlane(s.base, at);
      Seq q;
      q.begin = u.begin, q.n = u.n, q.base = u.base;
      q.first = __builtin_amdgcn_readlane(s.first, at);
      q.full = __builtin_amdgcn_readlane(s.full, at);
      q.blocks = __builtin_amdgcn_readlane(s.blocks, at);
      const uint64_t all = lane64(own, at);
      const uint32_t in_seq = item - static_cast<uint32_t>((items + lane64(upto, at) - all) * a.Hk);
      u.h = in_seq % a.Hk;
      const uint32_t rank = in_seq / a.Hk;
      // the last block j with before(j) < all - rank
      int lo = q.first, n = q.blocks - q.first;
      uint64_t at_lo = 0, next;
      for (;;) {
        const int step = (n + 63) / 64, j = lo + lane * step;
        const uint64_t f = lane * step < n ? q.before(j, tpb, m) : all;
        const int k = 63 - __builtin_clzll(__ballot(lane * step < n && f < all - rank));
        at_lo = lane64(f, k);
        const int from = lo + k * step;
        if (step == 1) {
          next = k == 63 || k + 1 >= n ? q.before(from + 1, tpb, m) : lane64(f, k + 1);
          u.j = from;
          break;
        }
        n = min(step, lo + n - from);
        lo = from;
      }
      u.chunks = static_cast<int>(next - at_lo);
      u.chunk = static_cast<int>(rank - (all - next));
      const int p0 = parts + (__builtin_amdgcn_readlane(parts_upto, at) - __builtin_amdgcn_readlane(own_parts, at)) * a.Hk;
      u.slot = u.chunks > 1 ? p0 + static_cast<int>(in_seq) : -1;
    }
    items += lane64(upto, 63);
    parts += __builtin_amdgcn_readlane(parts_upto, 63) * a.Hk;
  }
  *n_parts = parts;
  return u;
}

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// 16 bytes a lane from base + at to LDS address lds + 16 lane, behind the
// compiler's back: it would wait for every such copy before the next LDS read,
// whichever buffer that reads.  landed() waits for the wave's own.
__device__ __forceinline__ void to_lds16(const void* base, uint32_t at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(at), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)(p)));
}
// Two values of each of 4 rows, transposed: lanes 4 r .. 4 r + 3 of 16 point at row r.
__device__ __forceinline__ uint2 read_transposed(const uint8_t* p) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4_t*)(p)));
}

// whether either 16-bit number of a word is infinite or NaN
template <int ACT>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  constexpr uint32_t e = ACT == 2 ? 0x7F80u : 0x7C00u;
  return (w & e) == e || ((w >> 16) & e) == e;
}

// A row's place and output: v[4] neighbouring values, normalised.
template <int ACT, int D>
__device__ __forceinline__ void store_row(const AttnArgs& a, int t, int hq, int d, f32x4_t v) {
  if (a.gate) {
    const uint2 g = *reinterpret_cast<const uint2*>(a.gate + t * a.g_ts + hq * a.g_hs + d);
    v[0] *= sigmoid(act_to_f32<ACT>(g.x & 0xFFFFu)), v[1] *= sigmoid(act_to_f32<ACT>(g.x >> 16));
    v[2] *= sigmoid(act_to_f32<ACT>(g.y & 0xFFFFu)), v[3] *= sigmoid(act_to_f32<ACT>(g.y >> 16));
  }
  *reinterpret_cast<uint2*>(a.o + (static_cast<size_t>(t) * a.Hq + hq) * D + d) =
      make_uint2(pack2<ACT>(v[0], v[1]), pack2<ACT>(v[2], v[3]));
}

template <int ACT, int D>
__global__ __launch_bounds__(64 * Shape<D>::kWaves, 2) void k_attn_prefill(AttnArgs a, uint8_t* ws) {
  constexpr int kT = Shape<D>::kTiles, kW = Shape<D>::kWaves, kBytes = Shape<D>::kTileBytes;
  constexpr int kSteps = D / 16, kBlocks = D / 32, kPieces = D / 8;   // 16-byte pieces of a row
  constexpr int kLoadKeys = 64 / kPieces, kLoads = kKeys / (kLoadKeys * kW);
  __shared__ __align__(1024) uint8_t tiles[2][2][kBytes];   // buffer, keys and values
  __shared__ int bad_key[2];
  const int lane = threadIdx.x & 63, l32 = lane & 31, hf = lane >> 5, group = a.Hq / a.Hk, tpb = kRows / group;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int n_parts;
  const Unit u = find_unit(a, blockIdx.x, tpb, &n_parts);
  Header* header = reinterpret_cast<Header*>(ws);
  if (blockIdx.x == 0 && threadIdx.x == 0) header->parts = n_parts;
  if (u.b < 0) return;
  if (u.slot >= 0 && threadIdx.x == 0) reinterpret_cast<Part*>(ws + sizeof(Header))[u.slot].u = u;

  const int tok0 = u.j * tpb, n_tok = min(tpb, u.n - tok0), pos0 = u.base + tok0;
  const int t_first = u.chunk * u.size, t_last = min((pos0 + n_tok + kKeys - 1) >> kKeysLog, t_first + u.size);
  const int32_t* table = a.table + static_cast<size_t>(u.b) * a.max_pages;
  const int length = u.base + u.n;

  // this lane's rows: token (the block's last for rows behind it), query head, position
  int tok[kT], head[kT], pos[kT];
  bool real[kT];
  uint4 q[kT][kSteps];
  const uint32_t flip = a.scale < 0 ? 0x80008000u : 0u;
#pragma unroll
  for (int r = 0; r < kT; ++r) {
    const int row = (wave * kT + r) * 32 + l32;
    tok[r] = row / group;
    head[r] = u.h * group + row - tok[r] * group;
    real[r] = tok[r] < n_tok;
    tok[r] = min(tok[r], n_tok - 1);
    pos[r] = pos0 + tok[r];
    const uint16_t* qp = a.q + (u.begin + tok0 + tok[r]) * a.q_ts + head[r] * a.q_hs + 8 * hf;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(qp + 16 * i);
      q[r][i] = make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
    }
  }
  // of the wave's rows; no key at all where none of them is real
  const int low = __builtin_amdgcn_readfirstlane(pos[0]);
  const int high = wave * kT * 32 / group < n_tok ? __builtin_amdgcn_readlane(pos[kT - 1], 31) : -1;

  f32x16_t o[kT][kBlocks];
  float mx[kT], l[kT];
#pragma unroll
  for (int r = 0; r < kT; ++r) {
    mx[r] = -INFINITY, l[r] = 0;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[r][i][j] = 0;
  }
  // scores are non-negative multiples of the products; a scale of 0 counts as 2^-126
  const float c = fmaxf(fabsf(a.scale) * kLog2e, 1.17549435e-38f);

  // pages of 64 groups of 16 keys (16 tiles), one to a lane (-1: none)
  int pages = -1;
  uint64_t live = 0;
  auto load_pages = [&](int t) {
    const int p = ((t & ~15) << kKeysLog) + 16 * lane;
    const int id = p < length ? table[p >> a.page_log] : -1;
    pages = id < a.n_pages ? id : -1;
    live = __ballot(pages >= 0);
  };
  // this lane's 16 bytes of a load: a key's place in its group of 16 is the same in all loads of a wave
  const int load_key = lane / kPieces, in_group = (wave * kLoadKeys & 15) + load_key;
  const int v_swz = D == 64 ? (in_group >> 1) & 1 : in_group & (D / 32 - 1);   // values: 64-byte groups of pieces
  const uint32_t k_at = 2 * (in_group * D + 8 * (lane % kPieces ^ (in_group & 7)));
  const uint32_t v_at = 2 * (in_group * D + 8 * (lane % kPieces ^ v_swz << 2));
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(&tiles[0][0][wave * 1024]));
  auto issue = [&](int t, int buf) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int g = (i * kW + wave) * kLoadKeys >> 4, p = (t << kKeysLog) + 16 * g;
      const int id = max(__builtin_amdgcn_readlane(pages, 4 * (t & 15) + g), 0);
      const size_t at = (((static_cast<size_t>(id) * a.Hk + u.h) << a.page_log) + (p & ((1 << a.page_log) - 1))) * D;
      const uint32_t lds = lds0 + buf * 2 * kBytes + i * kW * 1024;
      to_lds16(a.k + at, k_at, lds);
      to_lds16(a.v + at, v_at, lds + kBytes);
    }
  };
  if (threadIdx.x == 0) bad_key[0] = bad_key[1] = INT_MAX;
  load_pages(t_first);
  issue(t_first, 0);
  int alive = (live >> (4 * (t_first & 15))) & 15;
  for (int t = t_first; t < t_last; ++t) {
    const int buf = (t - t_first) & 1;
    landed();
    __syncthreads();   // tile t has landed, and all are done with tile t - 1
    const int alive_now = alive;
    if (t + 1 < t_last) {
      if (((t + 1) & 15) == 0) load_pages(t + 1);
      alive = (live >> (4 * ((t + 1) & 15))) & 15;
      issue(t + 1, buf ^ 1);
    }
    int bad = INT_MAX;
    if ((t << kKeysLog) + kKeys - 1 > pos0 || alive_now != 15) {
      // Some row does not see some key, whose value may be anything, but 0 times
      // infinity or NaN is not 0: such values become 0, and rows that do see one
      // of them get a NaN by their sum of weights.
      int mine = INT_MAX;
#pragma unroll
      for (int i = 0; i < kBytes / (1024 * kW); ++i) {
        uint4* p = reinterpret_cast<uint4*>(&tiles[buf][1][(i * kW + wave) * 1024 + 16 * lane]);
        uint4 v = *p;
        if (not_finite<ACT>(v.x) || not_finite<ACT>(v.y) || not_finite<ACT>(v.z) || not_finite<ACT>(v.w)) {
          const int key = (i * kW + wave) * kLoadKeys + load_key;
          if (alive_now >> (key >> 4) & 1) mine = min(mine, (t << kKeysLog) + key);
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            constexpr uint32_t e = ACT == 2 ? 0x7F80u : 0x7C00u;
            if ((w[j] & e) == e) w[j] &= 0xFFFF0000u;
            if (((w[j] >> 16) & e) == e) w[j] &= 0xFFFFu;
          }
          *p = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (mine != INT_MAX) atomicMin(&bad_key[t & 1], mine);
      __syncthreads();
      bad = bad_key[t & 1];
    }
    if (threadIdx.x == 0) bad_key[(t + 1) & 1] = INT_MAX;

#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const int key0 = (t << kKeysLog) + 32 * sub;
      if (key0 > high) continue;
      f32x16_t s[kT];
#pragma unroll
      for (int r = 0; r < kT; ++r)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[r][i] = 0;
      // Operands are read kAhead products before they are used.
      const uint8_t* kp = &tiles[buf][0][(32 * sub + l32) * D * 2];
      auto key_part = [&](int i) { return *reinterpret_cast<const uint4*>(kp + (((2 * i + hf) ^ (lane & 7)) << 4)); };
      uint4 kf[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) kf[i] = key_part(i);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
#pragma unroll
        for (int r = 0; r < kT; ++r) s[r] = mfma32<ACT>(kf[i % kAhead], q[r][i], s[r]);
        if (i + kAhead < kSteps) kf[i % kAhead] = key_part(i + kAhead);
      }
      __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
      for (int i = kAhead; i < kSteps; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, kT, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x8, kT * kAhead, 0);
      if (key0 + 31 > low || alive_now != 15) {
#pragma unroll
        for (int r = 0; r < kT; ++r)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int k = 8 * (i >> 2) + 4 * hf + (i & 3);
            const bool see = key0 + k <= pos[r] && (alive_now >> (2 * sub + (i >> 3)) & 1);
            s[r][i] = see ? s[r][i] : -INFINITY;
          }
      }
      uint4 p[kT][2];
#pragma unroll
      for (int r = 0; r < kT; ++r) {
        float top = s[r][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, s[r][i]);
        top = pair_max(top) * c;
        // The reference for the exponents moves only when a weight would pass 2^8:
        // the sums are fp32, and the row's result does not depend on it otherwise.
        const bool grow = top > mx[r] + 8.0f;
        if (__any(grow)) {
          const float next = grow ? top : mx[r], base = next == -INFINITY ? 0.0f : next;
          const float f = __builtin_amdgcn_exp2f(mx[r] - base);
          mx[r] = next;
          const float g = grow ? f : 1.0f;
          l[r] *= g;
#pragma unroll
          for (int i = 0; i < kBlocks; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) o[r][i][j] *= g;
        }
        const float base = (mx[r] == -INFINITY ? 0.0f : mx[r]) - kShift<ACT>;
        float sum = 0;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float p0 = __builtin_amdgcn_exp2f(fmaf(s[r][i], c, -base));
          const float p1 = __builtin_amdgcn_exp2f(fmaf(s[r][i + 1], c, -base));
          sum += p0 + p1;
          w[i / 2] = pack2<ACT>(p0, p1);
        }
        l[r] += pos[r] >= bad ? __builtin_nanf("") : sum;
        p[r][0] = make_uint4(w[0], w[1], w[2], w[3]);
        p[r][1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
      // value rows 32 sub + 16 h + 8 (0 or 1) + 4 hf + (lane / 4) % 4, 8 bytes of a 64-byte group
      const int vk = 4 * hf + ((lane >> 2) & 3);
      const uint8_t* vp = &tiles[buf][1][(32 * sub + vk) * D * 2 + ((lane >> 4) & 1) * 32 + (lane & 3) * 8];
      const int swz = D == 64 ? (vk >> 1) & 1 : vk & (D / 32 - 1);
      auto value_part = [&](int n) {
        const uint8_t* vi = vp + ((n >> 1 ^ swz) << 6) + 16 * (n & 1) * D * 2;
        const uint2 x = read_transposed(vi), y = read_transposed(vi + 8 * D * 2);
        return make_uint4(x.x, x.y, y.x, y.y);
      };
      uint4 vf[kAhead];
#pragma unroll
      for (int n = 0; n < kAhead; ++n) vf[n] = value_part(n);
#pragma unroll
      for (int n = 0; n < 2 * kBlocks; ++n) {
#pragma unroll
        for (int r = 0; r < kT; ++r) o[r][n >> 1] = mfma32<ACT>(vf[n % kAhead], p[r][n & 1], o[r][n >> 1]);
        if (n + kAhead < 2 * kBlocks) vf[n % kAhead] = value_part(n + kAhead);
      }
      __builtin_amdgcn_sched_group_barrier(0x100, 2 * kAhead, 0);
#pragma unroll
      for (int n = kAhead; n < 2 * kBlocks; ++n) {
        __builtin_amdgcn_sched_group_barrier(0x8, kT, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x8, kT * kAhead, 0);
    }
  }

  // dimensions 32 i + 8 j + 4 hf + (0 .. 3) of the lane's row
#pragma unroll
  for (int r = 0; r < kT; ++r) {
    const float sum = pair_sum(l[r]);
    if (u.slot < 0) {
      const float inv = sum != 0 ? 1.0f / sum : 0.0f;
      if (real[r]) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            store_row<ACT, D>(a, u.begin + tok0 + tok[r], head[r], 32 * i + 8 * j + 4 * hf,
                              f32x4_t{o[r][i][4 * j], o[r][i][4 * j + 1], o[r][i][4 * j + 2], o[r][i][4 * j + 3]} * inv);
      }
    } else if (real[r]) {
      const int held = rows_held(a.N, group), row = (wave * kT + r) * 32 + l32;
      const size_t at = static_cast<size_t>(u.slot) * held + row;
      if (hf == 0) reinterpret_cast<float2*>(ws + ml_at())[at] = make_float2(mx[r], sum);
      float* po = reinterpret_cast<float*>(ws + o_at(held)) + at * D + 4 * hf;
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<f32x4_t*>(po + 32 * i + 8 * j) =
              f32x4_t{o[r][i][4 * j], o[r][i][4 * j + 1], o[r][i][4 * j + 2], o[r][i][4 * j + 3]};
    }
  }
}

// Adds up the parts of cut units: the workgroups of a unit's chunks share its
// rows.  Also writes the zeros of rows that have no position.
template <int ACT, int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, const uint8_t* ws) {
  const int group = a.Hq / a.Hk, tpb = kRows / group, held = rows_held(a.N, group);
  if (static_cast<int>(blockIdx.x) < reinterpret_cast<const Header*>(ws)->parts) {
    const Unit u = reinterpret_cast<const Part*>(ws + sizeof(Header))[blockIdx.x].u;
    const int tok0 = u.j * tpb, rows = min(tpb, u.n - tok0) * group;
    const int from = rows * u.chunk / u.chunks, to = rows * (u.chunk + 1) / u.chunks;
    const int first = u.slot - u.chunk * a.Hk;   // chunks of a head are Hk slots apart
    const float2* ml = reinterpret_cast<const float2*>(ws + ml_at());
    const float* po = reinterpret_cast<const float*>(ws + o_at(held));
    for (int i = from * (D / 4) + threadIdx.x; i < to * (D / 4); i += 256) {
      const int row = i / (D / 4), d = 4 * (i % (D / 4));
      float m = -INFINITY, l = 0;
      f32x4_t x = {0, 0, 0, 0};
      for (int k = 0; k < u.chunks; ++k) {
        const size_t at = static_cast<size_t>(first + k * a.Hk) * held + row;
        const float2 v = ml[at];
        const f32x4_t y = *reinterpret_cast<const f32x4_t*>(po + at * D + d);
        const float top = fmaxf(m, v.x), z = top == -INFINITY ? 0.0f : top;
        const float f = __builtin_amdgcn_exp2f(m - z), g = __builtin_amdgcn_exp2f(v.x - z);
        l = l * f + v.y * g;
        x = x * f + y * g;
        m = top;
      }
      const int t = row / group;
      store_row<ACT, D>(a, u.begin + tok0 + t, u.h * group + row - t * group, d, x * (l != 0 ? 1.0f / l : 0.0f));
    }
  }
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    int begin, end;
    seq_rows(a.off, b, a.N, begin, end);
    const int none = min(end - begin - seq_length(a.length, b, a.max_pages, a.page_log), end - begin);
    for (int64_t i = 8 * threadIdx.x; i < static_cast<int64_t>(max(none, 0)) * a.Hq * D; i += 2048)
      *reinterpret_cast<uint4*>(a.o + static_cast<size_t>(begin) * a.Hq * D + i) = make_uint4(0, 0, 0, 0);
  }
}

int64_t units_of(int64_t N, int64_t B, int q_heads, int kv_heads) {
  return kv_heads * (N / (kRows / (q_heads / kv_heads)) + B);
}

template <int ACT, int D>
hipError_t launch(const AttnArgs& a, void* ws, hipStream_t s) {
  const int grid = static_cast<int>(units_of(a.N, a.B < a.N ? a.B : a.N, a.Hq, a.Hk)) + (1 << kShareLog);
  hipLaunchKernelGGL((k_attn_prefill<ACT, D>), dim3(grid), dim3(64 * Shape<D>::kWaves), 0, s, a,
                     static_cast<uint8_t*>(ws));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_attn_join<ACT, D>), dim3(kSlots), dim3(256), 0, s, a, static_cast<const uint8_t*>(ws));
  return hipGetLastError();
}

}  // namespace

bool attn_prefill_fits(const moe_attn_desc* d, int N) {
  return units_of(N, d->batch < N ? d->batch : N, d->q_heads, d->kv_heads) <= kMaxUnits;
}

size_t attn_prefill_bytes(const moe_attn_desc* d, int N) {
  const int held = rows_held(N, d->q_heads / d->kv_heads);
  return o_at(held) + sizeof(float) * kSlots * held * d->head_dim;
}

hipError_t launch_attn_prefill(int act, int d, const AttnArgs& a, void* ws, hipStream_t s) {
  if (act == MOE_BF16)
    return d == 64 ? launch<2, 64>(a, ws, s) : d == 128 ? launch<2, 128>(a, ws, s) : launch<2, 256>(a, ws, s);
  return d == 64 ? launch<1, 64>(a, ws, s) : d == 128 ? launch<1, 128>(a, ws, s) : launch<1, 256>(a, ws, s);
}

}  // namespace moe
