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
// Units are of very different length (causal blocks, ragged sequences).  Where
// they do not fill the chip evenly by themselves, every compute unit takes an
// even run of them, which may begin and end within a unit, and k_attn_join adds
// up the parts.  A unit counts kStart keys more than it has, for its begin and
// end.  Every workgroup works out its run from the lengths and offsets on the
// device, so a captured call follows them.
//
// One prompt of 8192 tokens, 16 query and 2 key heads of 256: 520 to 540 us from
// card to card, 1020 to 1060 TFLOP/s (a library product of 8192^3 reaches 1240 to
// 1250), on a card at work.  After a pause its first 30 runs take 560 to 720, as
// library products then take 840 to 1030 where they settle at 783; after 100 such
// products the kernel is at its steady time from the first run on.  The matrix
// cores are busy 53% and the vector units 48% of the cycles.  Keys and values of 0
// take 442 us with the same products: part of it follows the data, by power as it
// seems.  16 and 4 heads of 128: 329 us, matrix cores 46%, vector units 52%; of
// 64: 210, 32% and 65% (a tile of scores has 16 exponentials to 8 products).
// 12 prompts of 6001 tokens: 121 to 125 us with k_attn_join, which reads up to 134
// MB of parts in 24.  Five drafted tokens over 4096: 19 and 6, latency (40 rows of
// a unit's 256 are theirs).
#include "attn.h"

namespace moe {
namespace {

constexpr int kRows = 256;                  // rows of a unit
constexpr int kKeys = 64, kKeysLog = 6;     // keys of a tile
constexpr int kMaxUnits = 1 << 22;
// A unit's begin and end in keys.  256, 320, 384, 448, 512: 135.7, 131.7, 126.4, 121.9, 122.4 us for 12 prompts of 6001
// tokens; 84.5, 78.5, 80.2, 82.7, 79.9 for 2048 tokens; 39.9, 40.6, 41.4, 40.3, 40.2 for 512; 98.1, 100.3, 101.4, 100.5,
// 103.2 for 2 prompts of 4096 tokens in all, 8 key heads; 143 for 4 turns of 1023 over 12345 with each.  All with heads of
// 256: narrower ones were not swept.
constexpr int kStart = 512;
constexpr int kRunLog = 7;                  // shortest run, in keys

// Two 32-row tiles to a wave where a head is narrow enough: the registers of
// accumulators and queries are the bound (192 of 256).
template <int D_>
struct Shape {
  static constexpr int D = D_, kT = D == 256 ? 1 : 2, kW = kRows / (32 * kT);
  static constexpr int kAhead = 4 / kT;                 // operands in flight from LDS
  static constexpr int kRuns = D == 256 ? 256 : 512;   // workgroups that the chip holds (LDS)
};

struct Unit {     // uniform
  int b, h, begin, n, base;   // sequence, key head, first row, tokens, positions before them (may be negative)
  int j, blocks;              // block of tokens, blocks of the sequence
};
struct Part {     // part of a unit that several runs hold (unit.b < 0: none)
  Unit u;
  int first, last;            // those runs
  int pad[7];
};
struct Header {
  int parts;                  // two for each run (0: no unit is cut)
  int pad[63];
};

__host__ __device__ inline int rows_held(int N, int group) {   // rows of a part in the workspace
  const int64_t r = (static_cast<int64_t>(N) * group + 31) / 32 * 32;
  return r < kRows ? static_cast<int>(r) : kRows;
}
__host__ __device__ inline size_t ml_at(int runs) { return sizeof(Header) + sizeof(Part) * 2 * runs; }
__host__ __device__ inline size_t o_at(int runs, int held) { return ml_at(runs) + sizeof(float2) * 2 * runs * held; }

// A sequence (one to a lane, or uniform): its blocks of tpb tokens.  A unit's
// cost is the keys that its last token sees, and kStart for its begin and end.
struct Seq {
  int begin, n, base, first, blocks;   // first block that sees a key; all blocks
  __device__ __forceinline__ void load(const AttnArgs& a, int b, int tpb) {
    begin = n = base = first = blocks = 0;
    if (b >= a.B) return;
    int end;
    seq_rows(a.off, b, a.N, begin, end);
    n = end - begin;
    base = seq_length(a.length, b, a.max_pages, a.page_log) - n;
    blocks = (n + tpb - 1) / tpb;
    first = base < 0 ? min(-base / tpb, blocks) : 0;
    if (base + n <= 0) first = blocks;
  }
  __device__ __forceinline__ Seq of_lane(int i) const {
    return Seq{__builtin_amdgcn_readlane(begin, i), __builtin_amdgcn_readlane(n, i), __builtin_amdgcn_readlane(base, i),
               __builtin_amdgcn_readlane(first, i), __builtin_amdgcn_readlane(blocks, i)};
  }
  // cost of blocks [first, j) of a head, the last one's taken for whole
  __device__ __forceinline__ int64_t before(int j, int tpb) const {
    const int64_t tri = (static_cast<int64_t>(j) * (j + 1) - static_cast<int64_t>(first) * (first + 1)) / 2;
    return static_cast<int64_t>(j - first) * (base + kStart) + tpb * tri;
  }
  __device__ __forceinline__ int64_t all(int tpb) const {
    return blocks > first ? before(blocks, tpb) - (static_cast<int64_t>(blocks) * tpb - n) : 0;
  }
};

__device__ __forceinline__ int64_t wave_scan64(int64_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int64_t u = __shfl_up(v, m);
    v += lane >= m ? u : 0ll;
  }
  return v;
}
__device__ __forceinline__ int64_t lane64(int64_t v, int i) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(v), i);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(static_cast<uint64_t>(v) >> 32), i);
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ void set_sequence(Unit& u, int b, const Seq& s) {
  u.b = b, u.begin = s.begin, u.n = s.n, u.base = s.base, u.blocks = s.blocks;
}

// Runs of a cut call: the first `more` are one longer than `per`, which is at least kKeys
// (or there is one run): so a run that lies within a unit has a tile of it.
struct Runs {
  int64_t per;
  int more, n;
  __device__ __forceinline__ int64_t start(int r) const { return r * per + min(r, more); }
  __device__ __forceinline__ int of(int64_t x) const {
    const int64_t big = more * (per + 1);
    return static_cast<int>(x < big ? x / (per + 1) : more + (x - big) / per);
  }
};
// Tiles of a unit that lie before its cost position v.
__device__ __forceinline__ int tile_at(int64_t v, int n_tiles) {
  return v <= kStart ? 0 : static_cast<int>(min(static_cast<int64_t>(n_tiles), (v - kStart + kKeys - 1) >> kKeysLog));
}

// Where this workgroup begins (wave-uniform; false: it has nothing to do).
// Cutting costs the parts' way through memory: where no unit is longer than an
// even share, units in falling order fill the chip evenly by themselves, one to
// a workgroup: sequences in order, in each the last block first.  Else each
// workgroup takes an even share of the units in rising order, a run, which may
// begin and end within a unit.  The key heads are innermost either way:
// neighbours in the first order run on different dies, each with its own heads;
// neighbouring runs are dealt to one die.
template <class S>
__device__ bool begin_work(const AttnArgs& a, int tpb, Unit& u, bool& cut, Runs& runs, int& run, int64_t& unit_start) {
  const int lane = threadIdx.x & 63, chunks = (a.B + 63) / 64;
  Seq s;
  int64_t total = 0, upto = 0;
  uint32_t units = 0;
  int longest = 0;
  for (int c = 0; c < chunks; ++c) {
    s.load(a, 64 * c + lane, tpb);
    upto = wave_scan64(s.all(tpb));
    total += lane64(upto, 63);
    int sum = s.blocks - s.first, top = sum > 0 ? s.base + s.n : 0;   // positions of sequences with units
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      top = max(top, __shfl_xor(top, m));
      sum += __shfl_xor(sum, m);
    }
    longest = max(longest, __builtin_amdgcn_readfirstlane(top));
    units += __builtin_amdgcn_readfirstlane(sum);
  }
  total *= a.Hk;
  units *= a.Hk;
  cut = total > 0 && static_cast<int64_t>(longest + kStart) * S::kRuns > total;
  run = blockIdx.x;
  if (!cut) {
    if (blockIdx.x >= units) return false;
    int64_t items = 0;
    for (int c = 0; c < chunks; ++c) {
      if (chunks > 1) s.load(a, 64 * c + lane, tpb);
      const int64_t up = wave_scan64(s.blocks - s.first);
      const uint64_t hit = __ballot((items + up) * a.Hk > blockIdx.x);
      if (hit) {
        const int at = __builtin_ctzll(hit);
        const Seq q = s.of_lane(at);
        set_sequence(u, 64 * c + at, q);
        const uint32_t in_seq = blockIdx.x - static_cast<uint32_t>((items + lane64(up, at) - (q.blocks - q.first)) * a.Hk);
        u.h = in_seq % a.Hk;
        u.j = q.blocks - 1 - static_cast<int>(in_seq / a.Hk);
        return true;
      }
      items += lane64(up, 63);
    }
    return false;
  }
  // (offsets in no order can name more work than the host counted: no more runs than workgroups)
  runs.n = min(static_cast<int>(min(static_cast<int64_t>(S::kRuns), (total >> kRunLog) + 1)), static_cast<int>(gridDim.x) & ~7);
  runs.per = total / runs.n;
  runs.more = static_cast<int>(total - runs.per * runs.n);
  const int die_runs = (runs.n + 7) / 8;
  run = blockIdx.x % 8 * die_runs + blockIdx.x / 8;
  if (static_cast<int>(blockIdx.x / 8) >= die_runs || run >= runs.n) return false;
  const int64_t pos = runs.start(run);
  int64_t sum = 0;
  for (int c = 0; c < chunks; ++c) {
    if (chunks > 1) {
      s.load(a, 64 * c + lane, tpb);
      upto = wave_scan64(s.all(tpb));
    }
    const uint64_t hit = __ballot((sum + upto) * a.Hk > pos);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      const Seq q = s.of_lane(at);
      set_sequence(u, 64 * c + at, q);
      const int64_t seq_start = (sum + lane64(upto, at) - q.all(tpb)) * a.Hk, in_seq = pos - seq_start;
      // the last block j with Hk before(j) <= in_seq
      int lo = q.first, n = q.blocks - q.first;
      for (;;) {
        const int step = (n + 63) / 64, j = lo + lane * step;
        const int64_t f = q.before(j, tpb) * a.Hk;
        const int k = 63 - __builtin_clzll(__ballot(lane * step < n && f <= in_seq));
        const int from = lo + k * step;
        if (step == 1) {
          const int cost = q.base + min((from + 1) * tpb, q.n) + kStart;
          const int64_t rest = in_seq - lane64(f, k);
          u.j = from;
          u.h = static_cast<int>(rest / cost);
          unit_start = seq_start + lane64(f, k) + static_cast<int64_t>(u.h) * cost;
          return true;
        }
        n = min(step, lo + n - from);
        lo = from;
      }
    }
    sum += lane64(upto, 63);
  }
  return false;
}

// The unit behind u in rising order (false: there is none).
__device__ bool next_unit(const AttnArgs& a, int tpb, Unit& u) {
  if (++u.h < a.Hk) return true;
  u.h = 0;
  if (++u.j < u.blocks) return true;
  for (int b = u.b + 1; b < a.B; b += 64) {
    Seq s;
    s.load(a, b + (threadIdx.x & 63), tpb);
    const uint64_t hit = __ballot(s.blocks > s.first);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      const Seq q = s.of_lane(at);
      set_sequence(u, b + at, q);
      u.j = q.first;
      return true;
    }
  }
  return false;
}

// A row's weights are 2^(z - ref), where ref is set to its largest z - kLift and
// moves when a weight would pass 2^(kLift + 8).  fp16: 2^15 at most, and full
// precision down to 2^-21 of the largest weight.  bf16: below 1 (2^-1 and the
// rounding of large scores), so that no sum of weighted values passes that of the
// values' magnitudes; its exponents reach as far as fp32's.
template <int ACT>
constexpr float kLift = ACT == 2 ? -9.0f : 7.0f;

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// 16 bytes a lane from base + at to LDS address lds + 16 lane, behind the
// compiler's back: it would wait for every such copy before the next LDS read,
// whichever buffer that reads.  landed() waits for the wave's own.  A memory
// instruction reads a scalar register five wait states after a vector
// instruction wrote it at the earliest, which the compiler does not look after
// in here: the move and the s_nop before are that many.
__device__ __forceinline__ void to_lds16(const void* base, uint32_t at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(at), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void to_lds16(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds) : "memory", "m0");
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

template <int ACT, class S>
__global__ __launch_bounds__(64 * S::kW, 2) void k_attn_prefill(AttnArgs a, uint8_t* ws) {
  constexpr int D = S::D, kT = S::kT, kW = S::kW, kTileBytes = kKeys * D * 2;
  constexpr int kSteps = D / 16, kBlocks = D / 32, kAhead = S::kAhead, kPieces = D / 8;   // 16-byte pieces of a row
  constexpr int kLoadKeys = 64 / kPieces, kLoads = kKeys / (kLoadKeys * kW);
  constexpr int kKeySwap = D == 64 ? 7 : 15;   // the pieces' order depends on the key: no bank conflicts over 16 keys
  // places that a wave's loads have in their groups of 16 keys
  constexpr int kPlaces = 16 / kLoadKeys > kW ? 16 / kLoadKeys / kW : 1;
  __shared__ __align__(1024) uint8_t tiles[2][2][kTileBytes];   // buffer, keys and values
  __shared__ int bad_key[2];
  const int group = a.Hq / a.Hk, tpb = kRows / group;
  const uint32_t per_group = 65536 / group + 1;   // row / group = row * per_group >> 16 (row < 256, group <= 16)
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int held = rows_held(a.N, group);

  Unit u;
  bool cut;
  Runs runs;
  int run;
  int64_t unit_start = 0;
  const bool work = begin_work<S>(a, tpb, u, cut, runs, run, unit_start);
  if (blockIdx.x == 0 && threadIdx.x == 0) reinterpret_cast<Header*>(ws)->parts = cut ? 2 * runs.n : 0;
  if (!work) return;
  Part* parts = reinterpret_cast<Part*>(ws + sizeof(Header)) + 2 * run;
  if (cut && threadIdx.x < 2) parts[threadIdx.x].u.b = -1;

  // scores are positive multiples of the products; for a scale of 0 the queries are 0
  const uint32_t flip = a.scale < 0 ? 0x80008000u : 0u, keep = a.scale == 0 ? 0u : ~0u;
  const float c = a.scale == 0 ? 1.0f : fabsf(a.scale) * kLog2e;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(&tiles[0][0][wave * 1024]));
  int turn = 0;   // place of the next tile in bad_key
  if (threadIdx.x == 0) bad_key[0] = bad_key[1] = INT_MAX;

  for (;;) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));   // or what follows from it stays in registers from one unit to the next
    const int hf = lane >> 5;
    // this lane's 16 bytes of a load
    uint32_t k_at[kPlaces], v_at[kPlaces];
#pragma unroll
    for (int i = 0; i < kPlaces; ++i) {
      const int key = ((i * kW + wave) * kLoadKeys & 15) + lane / kPieces;
      const int swz = D == 64 ? (key >> 1) & 1 : key & (D / 32 - 1);   // values: 64-byte groups of pieces
      k_at[i] = 2 * (key * D + 8 * (lane % kPieces ^ (key & kKeySwap)));
      v_at[i] = 2 * (key * D + 8 * (lane % kPieces ^ swz << 2));
    }
    const int tok0 = u.j * tpb, n_tok = min(tpb, u.n - tok0), pos0 = u.base + tok0;
    const int n_tiles = (pos0 + n_tok + kKeys - 1) >> kKeysLog;
    int t_first = 0, t_last = n_tiles;
    if (cut) {
      t_first = tile_at(runs.start(run) - unit_start, n_tiles);
      t_last = tile_at(runs.start(run + 1) - unit_start, n_tiles);
    }
    if (t_first < t_last) {
    const bool whole = t_first == 0 && t_last == n_tiles;
    const int32_t* table = a.table + static_cast<size_t>(u.b) * a.max_pages;
    const int length = u.base + u.n;

    // pages of 64 groups of 16 keys (16 tiles), one to a lane (-1: none)
    int pages = -1;
    uint64_t live = 0;
    auto load_pages = [&](int t) {
      const int p = ((t & ~15) << kKeysLog) + 16 * lane;
      const int id = p < length ? table[p >> a.page_log] : -1;
      pages = id < a.n_pages ? id : -1;
      live = __ballot(pages >= 0);
    };
    load_pages(t_first);

    // this lane's rows: token (the block's last for rows behind it), query head
    struct Row {
      int row, tok, head;
      bool real;
    };
    auto row_of = [&](int r, int ln) {
      const int row = (wave * kT + r) * 32 + (ln & 31), tok = row * per_group >> 16;
      return Row{row, min(tok, n_tok - 1), u.h * group + row - tok * group, tok < n_tok};
    };
    int pos[kT];
    uint4 q[kT][kSteps];
#pragma unroll
    for (int r = 0; r < kT; ++r) {
      const Row w = row_of(r, lane);
      pos[r] = pos0 + w.tok;
      const uint16_t* qp = a.q + row_at(u.begin + tok0 + w.tok, a.q_ts, w.head, a.q_hs) + 8 * hf;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(qp + 16 * i);
        q[r][i] = make_uint4((v.x & keep) ^ flip, (v.y & keep) ^ flip, (v.z & keep) ^ flip, (v.w & keep) ^ flip);
      }
    }
    // of the wave's rows; no key at all where none of them is real
    const int low = __builtin_amdgcn_readfirstlane(pos[0]);
    const int high = wave * kT * 32 / group < n_tok ? __builtin_amdgcn_readlane(pos[kT - 1], 31) : -1;

    f32x16_t o[kT][kBlocks];
    float ref[kT], l[kT];
#pragma unroll
    for (int r = 0; r < kT; ++r) {
      ref[r] = -INFINITY, l[r] = 0;
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[r][i][j] = 0;
    }

    auto issue = [&](int t, int buf) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int g = (i * kW + wave) * kLoadKeys >> 4, p = (t << kKeysLog) + 16 * g;
        const int id = max(__builtin_amdgcn_readlane(pages, 4 * (t & 15) + g), 0);
        const size_t at = (((static_cast<size_t>(id) * a.Hk + u.h) << a.page_log) + (p & ((1 << a.page_log) - 1))) * D;
        const uint32_t lds = lds0 + buf * 2 * kTileBytes + i * kW * 1024;
        to_lds16(a.k + at, k_at[i % kPlaces], lds);
        to_lds16(a.v + at, v_at[i % kPlaces], lds + kTileBytes);
      }
    };
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
      } else if (whole && a.gate) {
        // The gates' way from memory is longer than a tile takes: they are brought
        // nearer now, by copies to a free place in LDS that nobody reads.
#pragma unroll 1
        for (int i = 0; i < kRows * kPieces / (64 * kW); ++i) {
          const int at = (i * kW + wave) * 64 + lane, row = at / kPieces, tk = row * per_group >> 16;
          const uint16_t* p = a.gate + row_at(u.begin + tok0 + min(tk, n_tok - 1), a.g_ts, u.h * group + row - tk * group, a.g_hs);
          to_lds16(p + 8 * (at % kPieces), lds0 + (buf ^ 1) * 2 * kTileBytes);
        }
      }
      int bad = INT_MAX;
      if ((t << kKeysLog) + kKeys - 1 > pos0 || alive_now != 15) {
        // Some row does not see some key, whose value may be anything, but 0 times
        // infinity or NaN is not 0: such values become 0, and rows that do see one
        // of them get a NaN by their sum of weights.
        constexpr uint32_t e = ACT == 2 ? 0x7F80u : 0x7C00u, ee = e << 16 | e, one = ACT == 2 ? 0x00800080u : 0x04000400u;
        auto place = [&](int i) { return reinterpret_cast<uint4*>(&tiles[buf][1][(i * kW + wave) * 1024 + 16 * lane]); };
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const uint4 v = *place(i);
          any |= ((v.x & ee) + one) | ((v.y & ee) + one) | ((v.z & ee) + one) | ((v.w & ee) + one);
        }
        int mine = INT_MAX;
        if (any & 0x80008000u) {
#pragma unroll 1
          for (int i = 0; i < kLoads; ++i) {
            const uint4 v = *place(i);
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            bool found = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if ((w[j] & e) == e) w[j] &= 0xFFFF0000u, found = true;
              if ((w[j] >> 16 & e) == e) w[j] &= 0xFFFFu, found = true;
            }
            const int key = (i * kW + wave) * kLoadKeys + lane / kPieces;
            if (found && (alive_now >> (key >> 4) & 1)) mine = min(mine, (t << kKeysLog) + key);
            *place(i) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (mine != INT_MAX) atomicMin(&bad_key[turn], mine);
        __syncthreads();
        bad = bad_key[turn];
      }
      turn ^= 1;
      if (threadIdx.x == 0) bad_key[turn] = INT_MAX;

#pragma unroll 1
      for (int sub = 0; sub < 2; ++sub) {
        const int key0 = (t << kKeysLog) + 32 * sub;
        if (key0 > high) continue;
        int ln = lane;
        asm volatile("" : "+v"(ln));   // or the compiler keeps every address below in a register
        const int hl = ln >> 5;
        f32x16_t s[kT];
#pragma unroll
        for (int r = 0; r < kT; ++r)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[r][i] = 0;
        // Operands are read kAhead products before they are used.
        const uint8_t* kp = &tiles[buf][0][(32 * sub + (ln & 31)) * D * 2];
        auto key_part = [&](int i) { return *reinterpret_cast<const uint4*>(kp + (((2 * i + hl) ^ (ln & kKeySwap)) << 4)); };
        if constexpr (D > 64) __builtin_amdgcn_s_setprio(1);   // the wave in its products first
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
        if constexpr (D > 64) __builtin_amdgcn_s_setprio(0);
        if (key0 + 31 > low || alive_now != 15) {
#pragma unroll
          for (int r = 0; r < kT; ++r)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int k = 8 * (i >> 2) + 4 * hl + (i & 3);
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
          // the sums are fp32, and the row's result does not depend on when ref moves
          bool grow;
          {
#pragma clang fp contract(off)
            top = pair_max(top) * c;
            grow = top - ref[r] > kLift<ACT> + 8.0f;
          }
          float base = ref[r] == -INFINITY ? 0.0f : ref[r];
          // (and what follows them, where a row's reference is far from 0 or not set: looking
          // costs 1%, 528 us to 533 for 8192 tokens)
          if (__any(grow | (fabsf(ref[r]) > 0x1p21f))) {
            const float next = grow ? top - kLift<ACT> : ref[r];
            base = next == -INFINITY ? 0.0f : next;
            const float f = __builtin_amdgcn_exp2f(ref[r] - base);
            ref[r] = next;
            const float g = grow ? f : 1.0f;
            l[r] *= g;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
#pragma unroll
              for (int j = 0; j < 16; ++j) o[r][i][j] *= g;
            if (fabsf(base) > 0x1p21f) {
              // Scores without digits behind the point: a fused s c - base differs from the
              // rounded s c that the reference is one of by up to half a step, which is no
              // part of an exponent any more.  So the rounded ones, as products of c again.
#pragma clang fp contract(off)
              const float per_c = 1.0f / c;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float z = s[r][i] * c, e = z - base;
                s[r][i] = e * per_c;
              }
              base = 0.0f;
            }
          }
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
        const int vk = 4 * hl + ((ln >> 2) & 3);
        const uint8_t* vp = &tiles[buf][1][(32 * sub + vk) * D * 2 + ((ln >> 4) & 1) * 32 + (ln & 3) * 8];
        const int swz = D == 64 ? (vk >> 1) & 1 : vk & (D / 32 - 1);
        auto value_part = [&](int n) {
          const uint8_t* vi = vp + ((n >> 1 ^ swz) << 6) + 16 * (n & 1) * D * 2;
          const uint2 x = read_transposed(vi), y = read_transposed(vi + 8 * D * 2);
          return make_uint4(x.x, x.y, y.x, y.y);
        };
        if constexpr (D > 64) __builtin_amdgcn_s_setprio(1);
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
        if constexpr (D > 64) __builtin_amdgcn_s_setprio(0);
      }
    }

    // Rows leave by LDS, 32 of up to 128 dimensions at a time in each wave's own
    // place, so that a row's values are stored side by side.  The pieces of 4 lie
    // in an order that depends on the row (banks).
    constexpr int kWide = D < 128 ? D : 128, kRowPieces = kWide / 4, kRowsAtOnce = 64 / kRowPieces;
    static_assert(kW * 32 * kWide * 4 <= 4 * kTileBytes, "the rows' places are the tiles'");
    const int slot = 2 * run + (t_first > 0 ? 0 : 1);
    landed();
    __syncthreads();
    {
      int ln = lane;
      asm volatile("" : "+v"(ln));
      f32x4_t* place = reinterpret_cast<f32x4_t*>(&tiles[0][0][0]) + wave * 32 * kRowPieces;
#pragma unroll
      for (int r = 0; r < kT; ++r) {
        const float sum = pair_sum(l[r]), inv = !whole ? 1.0f : sum != 0 ? 1.0f / sum : 0.0f;
        const uint32_t none = static_cast<uint32_t>(__ballot(sum == 0));   // of the 32 rows
        if (!whole && ln < 32 && row_of(r, ln).real)
          reinterpret_cast<float2*>(ws + ml_at(S::kRuns))[static_cast<size_t>(slot) * held + row_of(r, ln).row] = make_float2(ref[r], sum);
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += kWide) {
#pragma unroll
          for (int i = 0; i < kWide / 32; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f32x16_t& x = o[r][d0 / 32 + i];
              place[(ln & 31) * kRowPieces + ((8 * i + 2 * j + (ln >> 5)) ^ (ln & 7))] =
                  f32x4_t{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]} * inv;
            }
          __builtin_amdgcn_wave_barrier();
          constexpr int kBatch = 8;   // loads in flight (2, 4, 8: 142, 132 and 126 us for 12 prompts of 6001 tokens)
          const int piece = ln % kRowPieces, d = d0 + 4 * piece;
#pragma unroll 1
          for (int i = ln / kRowPieces; i < 32; i += kBatch * kRowsAtOnce) {
            f32x4_t x[kBatch];
            uint2 g[kBatch];
            Row w[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
              const int row = i + e * kRowsAtOnce;
              w[e] = row_of(r, row);   // rows that are not real read one that is
              g[e] = make_uint2(0, 0);
              x[e] = place[row * kRowPieces + (piece ^ (row & 7))];
            }
            if (whole) {
              if (a.gate) {
#pragma unroll
                for (int e = 0; e < kBatch; ++e) g[e] = gates_of(a, u.begin + tok0 + w[e].tok, w[e].head, d);
              }
#pragma unroll
              for (int e = 0; e < kBatch; ++e)
                if (w[e].real) store_row<ACT>(a, u.begin + tok0 + w[e].tok, w[e].head, D, d, x[e], g[e],
                                              none >> (i + e * kRowsAtOnce) & 1);
            } else {
#pragma unroll
              for (int e = 0; e < kBatch; ++e)
                if (w[e].real)
                  *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(ws + o_at(S::kRuns, held)) +
                                              (static_cast<int64_t>(slot) * held + w[e].row) * D + d) = x[e];
            }
          }
          __builtin_amdgcn_wave_barrier();
        }
      }
    }
    if (cut && !whole && threadIdx.x == 0) {
      Part p;
      p.u = u;
      p.first = runs.of(unit_start + kStart);   // the runs that hold a tile of it
      p.last = runs.of(unit_start + kStart + (static_cast<int64_t>(n_tiles - 1) << kKeysLog));
      parts[t_first > 0 ? 0 : 1] = p;
    }
    }   // a run's part of a unit may be none of its tiles
    unit_start += pos0 + n_tok + kStart;
    if (!cut || unit_start >= runs.start(run + 1)) return;
    if (!next_unit(a, tpb, u)) return;
    __syncthreads();   // the tiles' places are free again
  }
}

// Adds up the parts of units that several runs hold: the workgroups of a unit's
// runs share its outputs, four neighbouring ones to a piece, kSlices workgroups
// to a part.  Also writes the zeros of the blocks that see no position: they are no units.
constexpr int kSlices = 8;
template <int ACT, class S>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, const uint8_t* ws) {
  constexpr int D = S::D;
  __shared__ float sx[256][6];
  const int group = a.Hq / a.Hk, tpb = kRows / group, held = rows_held(a.N, group);
  const int w = blockIdx.x, tid = threadIdx.x;
  if (w < reinterpret_cast<const Header*>(ws)->parts) {
    const Part p = reinterpret_cast<const Part*>(ws + sizeof(Header))[w];
    if (p.u.b >= 0) {
      const Unit& u = p.u;
      const int tok0 = u.j * tpb, pieces = min(tpb, u.n - tok0) * group * (D / 4), n = p.last - p.first + 1;
      const int shares = n * kSlices, share = (w / 2 - p.first) * kSlices + blockIdx.y;
      const int from = static_cast<int64_t>(pieces) * share / shares, to = static_cast<int64_t>(pieces) * (share + 1) / shares;
      const float2* ml = reinterpret_cast<const float2*>(ws + ml_at(S::kRuns));
      const float* po = reinterpret_cast<const float*>(ws + o_at(S::kRuns, held));
      // threads of a piece: as many as leave all pieces of the share a place
      int lanes = 1;
      while (lanes < 64 && lanes < n && 2 * lanes * (to - from) <= 256) lanes <<= 1;
      for (int base = from; base < to; base += 256 / lanes) {
        const int piece = base + tid / lanes, row = piece / (D / 4), d = 4 * (piece % (D / 4));
        float m = -INFINITY, l = 0;
        f32x4_t x = {0, 0, 0, 0};
        auto add = [&](float m2, float l2, f32x4_t y) {
          const float top = fmaxf(m, m2), z = top == -INFINITY ? 0.0f : top;
          const float f = __builtin_amdgcn_exp2f(m - z), g = __builtin_amdgcn_exp2f(m2 - z);
          l = l * f + l2 * g;
          x = x * f + y * g;
          m = top;
        };
        if (piece < to) {
#pragma unroll 2
          for (int k = p.first + tid % lanes; k <= p.last; k += lanes) {
            const size_t at = static_cast<size_t>(2 * k + (k == p.first)) * held + row;
            const float2 v = ml[at];
            add(v.x, v.y, *reinterpret_cast<const f32x4_t*>(po + at * D + d));
          }
        }
        for (int step = 1; step < lanes; step <<= 1) {
          float* mine = sx[tid];
          mine[0] = m, mine[1] = l, mine[2] = x[0], mine[3] = x[1], mine[4] = x[2], mine[5] = x[3];
          __syncthreads();
          const float* other = sx[tid ^ step];
          const f32x4_t y = {other[2], other[3], other[4], other[5]};
          const float m2 = other[0], l2 = other[1];
          if ((tid & step) == 0) add(m2, l2, y);
          __syncthreads();
        }
        if (tid % lanes == 0 && piece < to) {
          const int t = row / group;
          const int hq = u.h * group + row - t * group;
          store_row<ACT>(a, u.begin + tok0 + t, hq, D, d, x * (l != 0 ? 1.0f / l : 0.0f),
                            gates_of(a, u.begin + tok0 + t, hq, d), l == 0);
        }
      }
    }
  }
  for (int b = w * kSlices + blockIdx.y; b < a.B; b += gridDim.x * kSlices) {
    Seq s;
    s.load(a, b, tpb);
    for (int64_t i = 8 * threadIdx.x; i < static_cast<int64_t>(min(s.first * tpb, s.n)) * a.Hq * D; i += 2048)
      *reinterpret_cast<uint4*>(a.o + static_cast<size_t>(s.begin) * a.Hq * D + i) = make_uint4(0, 0, 0, 0);
  }
}

int64_t units_of(int64_t N, int64_t B, int q_heads, int kv_heads) {
  return kv_heads * (N / (kRows / (q_heads / kv_heads)) + (B < N ? B : N));
}

template <int ACT, int D>
hipError_t launch(const AttnArgs& a, void* ws, hipStream_t s) {
  using S = Shape<D>;
  const int64_t units = units_of(a.N, a.B, a.Hq, a.Hk);
  // the runs that a cut call can have, eight or a multiple
  const int64_t cost = units * ((static_cast<int64_t>(a.max_pages) << a.page_log) + kStart), most = ((cost >> kRunLog) / 8 + 1) * 8;
  const int runs = static_cast<int>(most < S::kRuns ? most : S::kRuns), grid = static_cast<int>(units > runs ? units : runs);
  hipLaunchKernelGGL((k_attn_prefill<ACT, S>), dim3(grid), dim3(64 * S::kW), 0, s, a, static_cast<uint8_t*>(ws));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_attn_join<ACT, S>), dim3(2 * runs, kSlices), dim3(256), 0, s, a,
                     static_cast<const uint8_t*>(ws));
  return hipGetLastError();
}

}  // namespace

bool attn_prefill_fits(const moe_attn_desc* d, int N) {
  return units_of(N, d->batch, d->q_heads, d->kv_heads) <= kMaxUnits;
}

size_t attn_prefill_bytes(const moe_attn_desc* d, int N) {
  const int runs = d->head_dim == 256 ? Shape<256>::kRuns : Shape<128>::kRuns, held = rows_held(N, d->q_heads / d->kv_heads);
  return o_at(runs, held) + sizeof(float) * 2 * runs * held * d->head_dim;
}

hipError_t launch_attn_prefill(int act, int d, const AttnArgs& a, void* ws, hipStream_t s) {
  if (act == MOE_BF16)
    return d == 64 ? launch<2, 64>(a, ws, s) : d == 128 ? launch<2, 128>(a, ws, s) : launch<2, 256>(a, ws, s);
  return d == 64 ? launch<1, 64>(a, ws, s) : d == 128 ? launch<1, 128>(a, ws, s) : launch<1, 256>(a, ws, s);
}

}  // namespace moe
