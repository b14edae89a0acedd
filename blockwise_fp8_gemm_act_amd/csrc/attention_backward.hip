// Attention backward (gfx950).  With P = exp(S - lse), D = rowsum(do o), dS = P
// (do v^T - D):
//   dq = scale dS k,   dk = scale dS^T q,   dv = P^T do
// in two kernels that recompute S: one owns queries and walks the keys (dq, and D
// on the way), one owns keys and walks the queries of their group (dk, dv).  The
// scores are computed twice (7 products instead of 5), but every sum has one owner
// and a fixed order: no atomics, and no fp32 copy of dq in memory.
#include "attention_common.h"

#include <type_traits>

namespace puro {
namespace {

__device__ __forceinline__ void wait_all_and_meet() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ f32x16 splat(float x) {
  f32x16 v;
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = x;
  return v;
}

// ---------------------------------------------------------------- dq
// Three products a pair (S, do v, dS k): bound by the matrix cores, busy 55% of the time
// (counters, 4 x 4096 tokens, 16 and 8 heads of 128: 412 GFLOP and the walks repeated for D
// in 376 us; vector work 46%).  dS is one bf16 in its product with k, as it and P are below:
// relative error of the gradients 0.0024, 0.0017 of it their own rounding; a second bf16 would
// add a product to these three and two to the four below.  Two workgroups a unit at heads of
// 128, whose waves fill each other's gaps; of heads of 64 four.
//
// A workgroup takes `pack` heads of a group by kDqRows / pack queries, as the forward
// kernel does.  Also writes, for the kernel below, stats[0][h][row] = -lse / scale (-infinity
// for a row that sees nothing: its P are then 0) and stats[1][h][row] = -D: the products q k
// and do v start from these, so that exp2(c2 sum) is P and P times the other sum dS.
template <int kHd>
__global__ void __launch_bounds__(64 * kDqWaves, kHd == 64 ? 4 : 2) attn_dq_kernel(AttnArgs a, int slots, int pack) {
  constexpr int kTile = kTileBytes<kHd>(kDqKeys);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][2][kTile];
  __shared__ int again[kDqWaves];
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = (int)(blockIdx.x % a.k_heads);
  const int rest = (int)(blockIdx.x / a.k_heads);
  const int packs = a.group / pack, tall = kDqRows / pack;     // head packs of a group; queries of a block
  const int h = hk * a.group + rest % packs * pack + wave * 32 / tall;
  int slot = slots - 1 - Order(slots, a.sequences, a.window)(rest / packs);
  if (slot < 0) return;
  int sequence;
  const Seq sq = find_seq(a, a.q_start, 1, tall, slot, sequence);
  if ((int64_t)slot * tall >= sq.ql) return;
  const int row0 = slot * tall;
  const int rows = sq.ql - row0 < tall ? sq.ql - row0 : tall;
  const int shift = sq.kl - sq.ql;
  const KeyTiles kt = key_tiles(shift + row0, shift + row0 + rows - 1, a.window, a.sinks, kDqKeys);

  const int wave0 = wave * 32 % tall, mine = wave0 + (lane & 31);
  const int qrow = sq.q0 + row0 + (mine < rows ? mine : rows - 1);
  const int p = shift + row0 + mine;
  const int w_lo = shift + row0 + wave0, w_hi = w_lo + 31;
  const TileCopy<kHd> keys(a.k + (int64_t)sq.k0 * a.ks + (int64_t)hk * kHd, a.ks);
  const TileCopy<kHd> vals(a.v + (int64_t)sq.k0 * a.vs + (int64_t)hk * kHd, a.vs);
  const uint32_t lds0 = lds_addr(lds);
  // This wave's copies of tile i, a part of them at a time between the products (issued
  // together they hold the wave for a quarter of its time).  Past the last tile that one
  // is copied again, to a place that is not read any more.
  constexpr int kParts = kDqKeys / kGroupRows<kHd> / kDqWaves;
  auto copy = [&](int i, int part) {
    const uint32_t at = lds0 + (uint32_t)((i & 1) * 2 * kTile);
    const int t = i < kt.count ? i : kt.count - 1, g = part * kDqWaves + wave;
    keys(kt, t, kDqKeys, g, at);
    vals(kt, t, kDqKeys, g, at + kTile);
  };
  auto copy_all = [&](int i) {
#pragma unroll
    for (int part = 0; part < kParts; ++part) copy(i, part);
  };

  if (kt.count > 0) copy_all(0);
  bf16x8 qf[kHd / 16], df[kHd / 16];
  float dd = 0.0f;
#pragma unroll
  for (int kk = 0; kk < kHd / 16; ++kk) {
    const int64_t at = (int64_t)h * kHd + 16 * kk + 8 * half;
    qf[kk] = load8(a.q + (int64_t)qrow * a.qs + at);
    df[kk] = load8(a.d_o + (int64_t)qrow * a.os + at);
    const bf16x8 of = load8(a.o + (int64_t)qrow * a.os + at);
#pragma unroll
    for (int j = 0; j < 8; ++j) dd = __builtin_fmaf((float)df[kk][j], (float)of[j], dd);
  }
  dd = half_sum(dd);
  const float lse = a.lse[(int64_t)h * a.q_tokens + qrow];
  const float sd = lse == -__builtin_inff() ? lse : -lse / a.scale;
  arrived(qf);
  arrived(df);
  const float c2 = a.scale * kLog2e;
  if (__any(lse == -__builtin_inff())) {      // rows that see nothing have no part, whatever they hold
    const bool sees = lse != -__builtin_inff();
#pragma unroll
    for (int kk = 0; kk < kHd / 16; ++kk) {
      qf[kk] = sees ? qf[kk] : (bf16x8){};
      df[kk] = sees ? df[kk] : (bf16x8){};
    }
    dd = sees ? dd : 0.0f;
  }

  // D = do.o carries the rounding of o to bf16, up to 2^-8 |do| |o|, which no other rounding
  // hides where dS is small against D: rows with a dominating key, values or keys with a mean.
  // With the exact D a row's dS sum to 0, so that their sum is D's error; the stats below always
  // have it put right.  In dq it adds (sum dS) (sum P k), beside roundings of dS that come to
  // 2^-9 of the root of the squared dS times |k|.  Waves with a row whose sum reaches 2^-6 of
  // that root walk their keys again with the D put right.  Mean relative error of dq's rows (the
  // worst row's), 4096 keys, before / so / with the exact D: independent inputs 0.0017 / 0.0017 /
  // 0.0017; keys and values with a mean of three deviations 0.51 (2.3) / 0.006 (0.05) / 0.005
  // (0.02); a key that takes nearly all 1.1 (43) / 0.0016 (0.015) / 0.0015 (0.004).  The sums
  // cost 2% and a walk again in every block 40% of the backward call (4 x 4096 tokens: 842 us
  // without, 861 with the sums, 873 with the few walks of that case, 1176 with all; heads of 64,
  // 4 x 4096 tokens of 16 and 4 heads: 470 / 498 with the sums); a bound of 2^-7 instead takes 918.  Blocks of rows with few keys nearly always need it: they take D
  // from a walk of its own first, two products instead of three.
  bool exact = false;
  if (kt.count > 0 && (shift + row0 < 128 || (a.window > 0 && a.window + a.sinks < 128))) {
    exact = true;
    float off = 0.0f;
    for (int i = 0; i < kt.count; ++i) {
      wait_all_and_meet();
      copy_all(i + 1);
      const uint32_t ktile = lds0 + (uint32_t)((i & 1) * 2 * kTile), vtile = ktile + kTile;
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        f32x16 s = splat(sd), dp = {};
#pragma unroll
        for (int kk = 0; kk < kHd / 16; ++kk) s = mfma(row_frag<kHd>(ktile, 32 * b, kk), qf[kk], s);
#pragma unroll
        for (int kk = 0; kk < kHd / 16; ++kk) dp = mfma(row_frag<kHd>(vtile, 32 * b, kk), df[kk], dp);
        mask_tile(s, kt.key0(i, kDqKeys) + 32 * b, p, a.window, a.sinks);
#pragma unroll
        for (int j = 0; j < 16; ++j) off += __builtin_amdgcn_exp2f(s[j] * c2) * (dp[j] - dd);
      }
    }
    dd += half_sum(off);
    wait_all_and_meet();
    copy_all(0);
  }

  // Starting values kept in registers, where there are enough of them.
  constexpr bool kKept = kHd == 128;
  f32x16 acc[kHd / 32];
#pragma unroll
  for (int d = 0; d < kHd / 32; ++d) acc[d] = (f32x16){};
  // Tiles that this wave's queries see; the others are only copied for the rest.
  const int before = a.window > 0 ? w_lo - a.window + 1 : 0;            // first key in the wave's window
  const bool firsts = kt.first_n > 0 || kt.main0 * kDqKeys < a.sinks;   // the first tiles hold first keys
  int on = firsts || before <= 0 ? 0 : clampi(before / kDqKeys - kt.main0, 0, kt.count);
  int seen = kt.count;
  while (seen > on && kt.key0(seen - 1, kDqKeys) > w_hi) --seen;
  // The walk; with kSums also the sum of its dS and of their squares.
  float off = 0.0f, square = 0.0f;
  auto walk = [&](auto sums) {
    constexpr bool kSums = decltype(sums)::value;
    f32x16 s0, dp0;
    if (kKept) {
      s0 = splat(sd);
      dp0 = splat(-dd);
      asm volatile("" : "+v"(s0), "+v"(dp0));
    }
    if (on < seen) {
#pragma unroll
      for (int d = 0; d < kHd / 32; ++d) acc[d] = (f32x16){};
    }
    int i = 0;
    for (; i < on; ++i) {
      wait_all_and_meet();
      copy_all(i + 1);
    }
    for (; i < seen; ++i) {
      wait_all_and_meet();
      const int key0 = kt.key0(i, kDqKeys);
      const uint32_t ktile = lds0 + (uint32_t)((i & 1) * 2 * kTile), vtile = ktile + kTile;
      const bool all = key0 + kDqKeys - 1 <= w_lo && (a.window == 0 || key0 > w_hi - a.window);
      // Unrolled, heads of 64 would keep LDS addresses in scratch (4 x 2048 tokens: 183 -> 188 us).
#pragma unroll kHd == 64 ? 1 : 2
      for (int b = 0; b < 2; ++b) {
        f32x16 s = {}, dp = {};
        if (kKept) {
          s = s0;
          dp = dp0;
        }
#pragma unroll
        for (int kk = 0; kk < kHd / 16; ++kk) s = mfma(row_frag<kHd>(ktile, 32 * b, kk), qf[kk], s);
        copy(i + 1, b * kParts / 2);
        feed<2, kHd / 16, 0>();
        // Masked here, so that the exponentials run beside do v: 832 -> 826 us (4 x 4096 tokens).
        if (!all) mask_tile(s, key0 + 32 * b, p, a.window, a.sinks);
#pragma unroll
        for (int kk = 0; kk < kHd / 16; ++kk) dp = mfma(row_frag<kHd>(vtile, 32 * b, kk), df[kk], dp);
        if (kParts == 4) copy(i + 1, b * 2 + 1);
#pragma unroll
        for (int j = 0; j < 16; ++j) s[j] = __builtin_amdgcn_exp2f(kKept ? s[j] * c2 : __builtin_fmaf(s[j], c2, sd * c2));
        feed<2, kHd / 16, 0>();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          s[j] *= kKept ? dp[j] : dp[j] - dd;
          if (kSums) {
            off += s[j];
            square = __builtin_fmaf(s[j], s[j], square);
          }
        }
#pragma unroll
        for (int step = 0; step < 2; ++step) {
          const bf16x8 sf = pack_step(s, step);
#pragma unroll
          for (int d = 0; d < kHd / 32; ++d) acc[d] = mfma(col_frag<kHd>(ktile, 32 * b + 16 * step, d), sf, acc[d]);
        }
        feed<2, 0, kHd / 16>();
      }
    }
    for (; i < kt.count; ++i) {
      wait_all_and_meet();
      copy_all(i + 1);
    }
  };
  if (!exact) {
    walk(std::true_type());
    off = half_sum(off);
    square = half_sum(square);
    const bool shows = __any(mine < rows && off != 0.0f && off * off >= 0x1p-12f * square);     // also where both underflow
    if (__builtin_isfinite(off)) dd += off;
    again[wave] = shows;
    wait_all_and_meet();
    exact = __builtin_amdgcn_readfirstlane(again[0] | again[1] | again[2] | again[3]);
    if (exact) copy_all(0);
    if (!shows) on = seen = kt.count;       // this wave only copies for the others
  }
  if (exact) walk(std::false_type());
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // no copy outlives its workgroup's LDS
  if (half == 0 && mine < rows) {
    a.ws[(int64_t)h * a.q_tokens + qrow] = sd;
    a.ws[(int64_t)(a.q_heads + h) * a.q_tokens + qrow] = -dd;
  }
  if (mine < rows) {
    uint16_t *out = a.dq + (int64_t)qrow * a.dqs + (int64_t)h * kHd;
#pragma unroll
    for (int d = 0; d < kHd / 32; ++d) store_block(out + 32 * d, acc[d], a.scale);
  }
}

// ---------------------------------------------------------------- dk, dv
// Four products a pair (S, do v, P^T do, dS^T q).  Keys stand as columns here, so that a
// lane owns a key, and P and dS are again operands in place.  A wave holds 32 keys and
// values (64 registers at heads of 128) and the sums of their gradients (128), which leaves
// two waves a SIMD; the matrix cores are busy 56% of the time (550 GFLOP in 476 to 486 us at 4
// x 4096 tokens, 16 and 8 heads of 128).  What it took, the whole backward call there, us:
// 1492 as first built; masks without branches, reads ahead of the products and long walks
// first 973; copies between the products 903; starting values in the accumulators 823 to 863
// from card to card (847 to 896 with D put right, above).  One wave a SIMD with twice the
// registers: 1150 where this took 979.
//
// DkPlan says what a workgroup's work is.
struct Walk {
  int q_lo, q_hi;     // queries of the sequence
  int tile0, tiles;
};
__device__ __forceinline__ Walk walk_of(const AttnArgs &a, const DkPlan &plan, const Seq &sq, int slot, bool far) {
  const int key0 = slot * kDkRows, shift = sq.kl - sq.ql;
  const int keys = sq.kl - key0 < kDkRows ? sq.kl - key0 : kDkRows;
  Walk w{key0 - shift, sq.ql - 1, 0, 0};
  const bool windowed = a.window > 0 && (key0 >= a.sinks || slot < plan.far_blocks);
  const int near = windowed ? key0 + keys - 1 + a.window - 1 - shift : w.q_hi;   // last query with the block in its window
  if (far) w.q_lo = near + 1 > w.q_lo ? near + 1 : w.q_lo;
  else if (near < w.q_hi) w.q_hi = near;
  if (w.q_lo < 0) w.q_lo = 0;
  w.tile0 = w.q_lo / kDkQueries;
  w.tiles = w.q_lo <= w.q_hi ? w.q_hi / kDkQueries - w.tile0 + 1 : 0;
  return w;
}

// Far parts are numbered over the sequences like query tiles of kFarChunk * 64 / group
// rows; a sequence uses as many of its numbers as its far walk has chunks.
__device__ __forceinline__ int far_first(const AttnArgs &a, int start, int s) {
  return (int)((int64_t)start * a.group / (kFarChunk * kDkQueries)) + s;
}
__device__ __forceinline__ int far_parts(const AttnArgs &a, const DkPlan &plan, const Seq &sq, int s, int slot) {
  const Walk w = walk_of(a, plan, sq, slot, true);
  const int64_t chunks = ((int64_t)w.tiles * a.group + kFarChunk - 1) / kFarChunk;
  const int room = far_first(a, sq.q0 + sq.ql, s + 1) - far_first(a, sq.q0, s);
  return (int)(chunks < room ? chunks : (room > 0 ? room : 0));
}

template <int kHd>
__host__ __device__ constexpr size_t part_floats() {
  return (size_t)2 * kDkRows * kHd;
}

__device__ __forceinline__ void dma4_s(const void *base, uint32_t off, uint32_t lds) {
  uint32_t save;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, %2\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(save)
      : "v"(off), "s"(base), "s"(lds));
}

template <int kHd>
__global__ void __launch_bounds__(64 * kDkWaves, 2) attn_dkdv_kernel(AttnArgs a, DkPlan plan) {
  constexpr int kTile = kTileBytes<kHd>(kDkQueries);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][2][kTile];
  __shared__ __attribute__((aligned(1024))) float stat[2][2][kDkQueries];
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = (int)(blockIdx.x % a.k_heads);
  int rest = (int)(blockIdx.x / a.k_heads);
  const int far_items = plan.far_slots * plan.far_blocks;
  const bool far = rest < far_items;
  int part, parts, slot, s, number = 0;
  Seq sq;
  if (far) {
    slot = rest % plan.far_blocks;
    part = rest / plan.far_blocks;
    sq = find_seq(a, a.q_start, a.group, kFarChunk * kDkQueries, part, s);
    parts = 1;
  } else {
    rest -= far_items;
    part = rest % plan.parts;
    parts = plan.parts;
    slot = Order(plan.slots, a.sequences, a.window)(rest / plan.parts);
    number = slot;
    sq = find_seq(a, a.k_start, 1, kDkRows, slot, s);
  }
  if ((int64_t)slot * kDkRows >= sq.kl) return;
  const int fars = slot < plan.far_blocks ? far_parts(a, plan, sq, s, slot) : 0;
  float *partial = nullptr;
  if (far) {
    if (part >= fars) return;
    parts = fars;
    partial = a.ws + plan.far_at + (size_t)(blockIdx.x) * part_floats<kHd>();
  } else if (parts > 1) {
    partial = a.ws + plan.near_at + ((size_t)(number * a.k_heads + hk) * parts + part) * part_floats<kHd>();
  } else if (fars > 0) {
    partial = a.ws + plan.edge_at + (size_t)((s * plan.far_blocks + slot) * a.k_heads + hk) * part_floats<kHd>();
  }
  const int key0 = slot * kDkRows;
  const int keys = sq.kl - key0 < kDkRows ? sq.kl - key0 : kDkRows;
  const int shift = sq.kl - sq.ql;
  const Walk walk = walk_of(a, plan, sq, slot, far);
  const int tile0 = walk.tile0, tiles = walk.tiles;
  const int64_t work = (int64_t)tiles * a.group;
  const int begin = (int)(work * part / parts), end = (int)(work * (part + 1) / parts);

  const int mine = 32 * wave + (lane & 31);
  const int key = key0 + mine;
  const int w_lo = key0 + 32 * wave, w_hi = w_lo + 31;
  // The positions that see this lane's key in this work: seen_n of them from seen_lo.
  const int first = shift + walk.q_lo, final = shift + walk.q_hi;
  const int seen_lo = key > first ? key : first;
  const int seen_hi = a.window == 0 || key < a.sinks || key + a.window - 1 > final ? final : key + a.window - 1;
  const uint32_t seen_n = (uint32_t)(seen_hi >= seen_lo ? seen_hi - seen_lo + 1 : 0);
  // A key that nothing here sees reads a row that something does (the first of first keys,
  // the last of others), so that what it holds never matters.
  const int krow = sq.k0 + key0 + (mine < keys && seen_n > 0 ? mine : key0 < a.sinks ? 0 : keys - 1);
  const uint32_t lds0 = lds_addr(lds), stat0 = lds_addr(stat);
  int copy_r, copy_c;
  copy_place<kHd>(copy_r, copy_c);
  // Tiles are walked head by head and copied one ahead, a part of the copies at a time
  // between the products: issued together, a tile's copies held each wave for 2200 of the
  // 8000 cycles that it spends on a tile.  Past the last tile that one is copied again, to
  // a place that is not read any more.
  constexpr int kParts = kDkQueries / kGroupRows<kHd> / kDkWaves;
  struct Tile {
    int h, t;
  };
  auto after = [&](Tile x) {
    const bool wrap = x.t + 1 == tiles;
    return Tile{x.h + wrap, wrap ? 0 : x.t + 1};
  };
  struct Source {
    const uint16_t *q, *d;
    int first, last;    // of the tile's rows in the walk: those outside read one of these (they are masked)
  };
  auto source = [&](Tile x) {
    const int q0 = (tile0 + x.t) * kDkQueries;
    return Source{a.q + (int64_t)(sq.q0 + q0) * a.qs + (int64_t)x.h * kHd,
                  a.d_o + (int64_t)(sq.q0 + q0) * a.os + (int64_t)x.h * kHd, walk.q_lo - q0, walk.q_hi - q0};
  };
  auto copy = [&](const Source &from, int buf, int part) {
    const uint32_t at = lds0 + (uint32_t)(buf * 2 * kTile);
    const int g = part * kDkWaves + wave, r = g * kGroupRows<kHd> + copy_r;
    const uint32_t in = (uint32_t)clampi(r, from.first, from.last);
    dma16_s(from.q, __umul24(in, (uint32_t)(a.qs * 2)) + copy_c * 16, at + (uint32_t)(g * kGroupBytes));
    dma16_s(from.d, __umul24(in, (uint32_t)(a.os * 2)) + copy_c * 16, at + kTile + (uint32_t)(g * kGroupBytes));
  };
  auto copy_stat = [&](Tile x, const Source &from, int buf) {      // waves 2 and 3 copy what waves 0 and 1 do
    dma4_s(a.ws + (int64_t)((wave & 1) * a.q_heads + x.h) * a.q_tokens + sq.q0 + (tile0 + x.t) * kDkQueries,
           (uint32_t)(clampi(lane, from.first, from.last) * 4), stat0 + (uint32_t)((buf * 2 + (wave & 1)) * kDkQueries * 4));
  };

  Tile now{};
  if (begin < end) {
    now = Tile{hk * a.group + begin / tiles, begin % tiles};
    const Source from = source(now);
#pragma unroll
    for (int part = 0; part < kParts; ++part) copy(from, 0, part);
    copy_stat(now, from, 0);
  }
  bf16x8 kf[kHd / 16], vf[kHd / 16];
#pragma unroll
  for (int kk = 0; kk < kHd / 16; ++kk) {
    const int64_t at = (int64_t)hk * kHd + 16 * kk + 8 * half;
    kf[kk] = load8(a.k + (int64_t)krow * a.ks + at);
    vf[kk] = load8(a.v + (int64_t)krow * a.vs + at);
  }
  arrived(kf);
  arrived(vf);
  f32x16 dk[kHd / 32], dv[kHd / 32];
#pragma unroll
  for (int d = 0; d < kHd / 32; ++d) dk[d] = dv[d] = (f32x16){};
  const float c2 = a.scale * kLog2e;
  // Tiles that this wave's keys are seen from; the others are only copied for the rest.
  const int from_q = (w_lo > first ? w_lo : first) - shift;
  const int to_q = (a.window == 0 || w_lo < a.sinks || w_hi + a.window - 1 > final ? final : w_hi + a.window - 1) - shift;
  const int seen_from = from_q / kDkQueries - tile0, seen_to = to_q < from_q ? 0 : to_q / kDkQueries - tile0 + 1;

  auto products = [&](int q0, int buf, const Source &from) {
    const uint32_t qtile = lds0 + (uint32_t)(buf * 2 * kTile), dtile = qtile + kTile;
#pragma unroll 1
    for (int b = 0; b < 2; ++b) {
      const int p_lo = shift + q0 + 32 * b, p_hi = p_lo + 31;
      const bool all = p_lo >= first && p_hi <= final && w_hi <= p_lo &&
                       (a.window == 0 || w_lo > p_hi - a.window || w_hi < a.sinks);
      f32x16 s, dp;
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const f32x4 s4 = *reinterpret_cast<const f32x4 *>(&stat[buf][0][32 * b + 2 * j + 4 * half]);
        const f32x4 d4 = *reinterpret_cast<const f32x4 *>(&stat[buf][1][32 * b + 2 * j + 4 * half]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[j + e] = s4[e];
          dp[j + e] = d4[e];
        }
      }
#pragma unroll
      for (int kk = 0; kk < kHd / 16; ++kk) s = mfma(row_frag<kHd>(qtile, 32 * b, kk), kf[kk], s);
      copy(from, buf ^ 1, b * kParts / 2);
      // The mask between the products lets the exponentials run beside the second ones, but
      // takes registers: uneven sequences, heads of 64: 107 -> 105 us; 4 x 4096 tokens, heads
      // of 128: 832 -> 838 us.
      constexpr bool kEarly = kHd == 64;
      auto mask = [&]() {
        if (all) return;
        int since = p_lo + 4 * half - seen_lo;
        asm volatile("" : "+v"(since));      // keeps the comparisons inside this branch
#pragma unroll
        for (int j = 0; j < 16; ++j)
          s[j] = (uint32_t)(since + 8 * (j / 4) + j % 4) < seen_n ? s[j] : -__builtin_inff();
      };
      if (kEarly) {
        feed<2, kHd / 16, 0>();
        mask();
      }
#pragma unroll
      for (int kk = 0; kk < kHd / 16; ++kk) dp = mfma(row_frag<kHd>(dtile, 32 * b, kk), vf[kk], dp);
      if (kParts == 4) copy(from, buf ^ 1, b * 2 + 1);
      feed<2, kEarly ? kHd / 16 : kHd / 8, 0>();
      if (!kEarly) mask();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        s[j] = __builtin_amdgcn_exp2f(s[j] * c2);
        dp[j] *= s[j];
      }
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        const bf16x8 pf = pack_step(s, step), sf = pack_step(dp, step);
#pragma unroll
        for (int d = 0; d < kHd / 32; ++d) {
          dv[d] = mfma(col_frag<kHd>(dtile, 32 * b + 16 * step, d), pf, dv[d]);
          dk[d] = mfma(col_frag<kHd>(qtile, 32 * b + 16 * step, d), sf, dk[d]);
        }
      }
      feed<2, 0, kHd / 8>();
    }
  };

  if (begin < end) {
    int i = begin, buf = 0;
    while (i < end) {
      const int stop = now.t + (end - i) < tiles ? now.t + (end - i) : tiles;     // this head's tiles of the walk
      const int on = clampi(seen_from, now.t, stop), off = clampi(seen_to, on, stop);
      auto turn = [&]() {
        wait_all_and_meet();
        const Tile next = i + 1 < end ? after(now) : now;
        const Source from = source(next);
        copy_stat(next, from, buf ^ 1);
        return from;
      };
      auto done = [&]() {
        now = i + 1 < end ? after(now) : now;
        ++i;
        buf ^= 1;
      };
      for (int t = now.t; t < on; ++t) {
        const Source from = turn();
#pragma unroll
        for (int part = 0; part < kParts; ++part) copy(from, buf ^ 1, part);
        done();
      }
      for (int t = on; t < off; ++t) {
        const Source from = turn();
        products((tile0 + t) * kDkQueries, buf, from);
        done();
      }
      for (int t = off; t < stop; ++t) {
        const Source from = turn();
#pragma unroll
        for (int part = 0; part < kParts; ++part) copy(from, buf ^ 1, part);
        done();
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // no copy outlives its workgroup's LDS
  if (partial) {
    // [dk, dv][key][column]: registers 4g .. 4g+3 are 4 consecutive columns.
    float *pk = partial + mine * kHd, *pv = pk + kDkRows * kHd;
#pragma unroll
    for (int d = 0; d < kHd / 32; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = 32 * d + 8 * g + 4 * half;
        *reinterpret_cast<f32x4 *>(pk + c) = (f32x4){dk[d][4 * g], dk[d][4 * g + 1], dk[d][4 * g + 2], dk[d][4 * g + 3]};
        *reinterpret_cast<f32x4 *>(pv + c) = (f32x4){dv[d][4 * g], dv[d][4 * g + 1], dv[d][4 * g + 2], dv[d][4 * g + 3]};
      }
  } else if (mine < keys) {
    uint16_t *ok = a.dk + (int64_t)(sq.k0 + key) * a.dks + (int64_t)hk * kHd;
    uint16_t *ov = a.dv + (int64_t)(sq.k0 + key) * a.dvs + (int64_t)hk * kHd;
#pragma unroll
    for (int d = 0; d < kHd / 32; ++d) {
      store_block(ok + 32 * d, dk[d], a.scale);
      store_block(ov + 32 * d, dv[d], 1.0f);
    }
  }
}

// Sums the partials of a key block in order: 8 columns a thread, shares of a block in strides.
template <int kHd>
__global__ void __launch_bounds__(256) attn_dkdv_join_kernel(AttnArgs a, DkPlan plan, int shares) {
  constexpr int kThreads = kHd / 8, kRows = 256 / kThreads, kChunks = kDkRows / kRows;
  for (int share = blockIdx.x; share < shares; share += gridDim.x) {
    const int hk = (int)(share % a.k_heads);
    const int rest = (int)(share / a.k_heads);
    const int number = rest / kChunks;
    int slot = number;
    int s;
    const Seq sq = find_seq(a, a.k_start, 1, kDkRows, slot, s);
    const int fars = slot < plan.far_blocks && (int64_t)slot * kDkRows < sq.kl ? far_parts(a, plan, sq, s, slot) : 0;
    if ((int64_t)slot * kDkRows >= sq.kl || (plan.parts == 1 && fars == 0)) continue;
    const int r = (rest % kChunks) * kRows + (int)threadIdx.x / kThreads, c = 8 * ((int)threadIdx.x % kThreads);
    float x[2][8] = {};
    auto add = [&](const float *from) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          const f32x4 v = *reinterpret_cast<const f32x4 *>(from + (w * kDkRows + r) * kHd + c + j);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[w][j + e] += v[e];
        }
    };
    if (plan.parts > 1)
      for (int p = 0; p < plan.parts; ++p)
        add(a.ws + plan.near_at + ((size_t)(number * a.k_heads + hk) * plan.parts + p) * part_floats<kHd>());
    else
      add(a.ws + plan.edge_at + (size_t)((s * plan.far_blocks + slot) * a.k_heads + hk) * part_floats<kHd>());
    if (fars > 0) {
      const int f0 = far_first(a, sq.q0, s);
      for (int p = 0; p < fars; ++p)
        add(a.ws + plan.far_at + (size_t)(((f0 + p) * plan.far_blocks + slot) * a.k_heads + hk) * part_floats<kHd>());
    }
    if (slot * kDkRows + r < sq.kl) {       // a partial has all rows of its block
      const int64_t row = sq.k0 + slot * kDkRows + r;
      u32x4 k, v;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        k[j] = pack_bf16(x[0][2 * j] * a.scale, x[0][2 * j + 1] * a.scale);
        v[j] = pack_bf16(x[1][2 * j], x[1][2 * j + 1]);
      }
      *reinterpret_cast<u32x4 *>(a.dk + row * a.dks + (int64_t)hk * kHd + c) = k;
      *reinterpret_cast<u32x4 *>(a.dv + row * a.dvs + (int64_t)hk * kHd + c) = v;
    }
  }
}

template <int kHd>
hipError_t launch(const AttnArgs &a, hipStream_t stream) {
  const auto grid = [](int64_t blocks) { return dim3((unsigned)blocks); };
  if (a.q_tokens > 0) {
    const int pack = pack_of(a.group), slots = dq_slots(a.q_tokens, a.sequences, pack);
    attn_dq_kernel<kHd><<<grid(dq_blocks(slots, pack, a.q_heads, a.sequences, a.window)), dim3(64 * kDqWaves), 0, stream>>>(
        a, slots, pack);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (a.k_tokens == 0) return hipSuccess;
  const DkPlan plan = plan_dk(a.q_tokens, a.k_tokens, a.sequences, a.q_heads, a.k_heads, kHd, a.window, a.sinks);
  attn_dkdv_kernel<kHd><<<grid(dk_blocks(plan, a.k_heads, a.sequences, a.window)), dim3(64 * kDkWaves), 0, stream>>>(a, plan);
  if (hipError_t e = hipGetLastError()) return e;
  if (plan.parts > 1 || plan.far_blocks > 0) {
    attn_dkdv_join_kernel<kHd><<<grid(dk_join_blocks(plan, a.k_heads, kHd)), dim3(256), 0, stream>>>(
        a, plan, (int)dk_join_shares(plan, a.k_heads, kHd));
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace

size_t attention_backward_ws_bytes(const puro_attention_shape &a) {
  return plan_dk(a.q_tokens, a.k_tokens, a.sequences, a.q_heads, a.k_heads, a.head_dim, a.window, a.sinks).floats * 4;
}

hipError_t run_attention_backward(const AttnArgs &a, int head_dim, hipStream_t stream) {
  return head_dim == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace puro
