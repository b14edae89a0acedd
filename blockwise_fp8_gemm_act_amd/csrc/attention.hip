// Attention forward (gfx950): softmax(scale q k^T + mask) v in one pass over the
// keys with a running maximum and sum.
//
//   attn_kernel        many queries: 256 queries of one head a workgroup, 32 a wave
//   attn_split_kernel  few queries: 32 (query, head) rows a workgroup, the keys
//                      dealt over its waves and over `splits` workgroups
//   attn_join_kernel   joins the splits
#include "attention_common.h"

namespace puro {
namespace {

// Scores of 32 keys x 32 queries from a key tile in LDS and the queries' fragments.
template <int kHd>
__device__ __forceinline__ f32x16 score_tile(uint32_t ktile, int r0, const bf16x8 *qf) {
  f32x16 s = {};
#pragma unroll
  for (int kk = 0; kk < kHd / 16; ++kk) s = mfma(row_frag<kHd>(ktile, r0, kk), qf[kk], s);
  return s;
}

// Softmax state of one query (of a lane and its partner): m is the maximum in use,
// in units of log2, l this lane's share of the sum.
template <int kHd>
struct Row {
  f32x16 o[kHd / 32];
  float m, l;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int d = 0; d < kHd / 32; ++d) o[d] = (f32x16){};
    m = kNoMax;
    l = 0.0f;
  }

  // The maximum in use follows the true one only once that is 2^8 larger: until
  // then exp2(s - m) stays below 2^8, which costs bf16 no precision, and the
  // accumulators need no rescaling.
  __device__ __forceinline__ void raise(float top) {
    if (__any(top > m + 8.0f)) {
      const float next = fmaxf(m, top);
      const float f = __builtin_amdgcn_exp2f(m - next);
      m = next;
      l *= f;
#pragma unroll
      for (int d = 0; d < kHd / 32; ++d) o[d] *= f;
    }
  }
};

__device__ __forceinline__ float tile_max(const f32x16 &s) {
  float t = s[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) t = fmaxf(t, s[i]);
  return t;
}

// ---------------------------------------------------------------- many queries
// Bound by the matrix cores: 4 head_dim operations a visible pair, against 2 bytes of
// keys and values that a block reads for every 256 of its rows.  Beside them an
// exponential and four other vector operations a pair want as long as the products at
// heads of 128, and one wave alone issues them at half rate.
//
// So the two waves of a SIMD take turns: while one multiplies (scores of the next tile,
// values of this one), the other does the softmax of its next tile, with a barrier
// between the turns.  Waves 4-7 run one turn behind waves 0-3.
//
//   turn          2i                 2i+1               2i+2
//   waves 0-3     multiply i         softmax i+1        multiply i+1
//   waves 4-7     softmax i          multiply i         softmax i+1
//
// multiply i reads the keys of tile i+1 and the values of tile i, and between its
// products starts copies of the keys of tile i+3 and the values of tile i+2, each wave
// its part; they are awaited a turn later, at the end of softmax i+1, and needed two
// turns after that.  With three places each for keys and values, the places they take
// were read for the last time two turns before.
//
// What it took, at 4 x 4096 tokens, 16 and 8 heads of 128 (275 GFLOP, us): waves that run
// freely 342; turns 289; copies spread between the products (together they stall their
// wave as long as the softmax) and heads that share keys in one block 278; addresses of
// the copies worked out a turn ahead (a turn's products issue 200 other instructions
// instead of 270) 266; the softmax first in line, and no maximum taken 248 to 262 from card
// to card (1050 to 1110 TFLOP/s; the clock falls to 1.9 GHz under this load).  One wave a
// SIMD with 64 queries: 458.
//
// Read from the shader's clock there, cycles: a turn 1375, of which the products need 1024;
// a workgroup of 33 tiles 109000, of them 11000 to 13000 before its first turn (the first
// tiles' way from memory, with every unit asking), 91000 in turns, the rest after the last
// one; and 124000 from one workgroup of a unit to the next, by the counters.  So the matrix
// cores are busy 74% of the turns and 54% of the kernel.  A window of 1024 at 16381 tokens:
// 18 tiles of 3000, 18000 to 21000 before them, 80000 in all, 93000 to the next workgroup.
//
// Heads of 64 take 128 registers and half the LDS, so that two workgroups share a unit:
// 216 -> 175 us at 4 x 4096 tokens, 16 and 4 heads of 64 (157 with the steps above).
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <int kHd>
__global__ void __launch_bounds__(64 * kFwdWaves, kHd == 64 ? 4 : 2) attn_kernel(AttnArgs a, int slots, int pack) {
  constexpr int kTile = kTileBytes<kHd>(kFwdKeys);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[6 * kTile];     // three places of keys, three of values
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool late = wave >= kFwdWaves / 2;
  // Key heads run fastest over the workgroups, so that with 8 of them each XCD's L2
  // serves one; the last tiles of a sequence, which see most keys, start first.
  const int hk = (int)(blockIdx.x % a.k_heads);
  const int rest = (int)(blockIdx.x / a.k_heads);
  const int packs = a.group / pack, tall = kFwdRows / pack;     // head packs of a group; queries of a block
  const int h = hk * a.group + rest % packs * pack + wave * 32 / tall;
  int slot = slots - 1 - Order(slots, a.sequences, a.window)(rest / packs);
  if (slot < 0) return;
  int sequence;
  const Seq sq = find_seq(a, a.q_start, 1, tall, slot, sequence);
  if ((int64_t)slot * tall >= sq.ql) return;
  const int shift = sq.kl - sq.ql;                              // position of query 0
  typedef TileStream<kHd, kFwdKeys, kFwdWaves> Stream;
  constexpr int kParts = Stream::kParts;
  Stream keys(a.k + (int64_t)sq.k0 * a.ks + (int64_t)hk * kHd, a.ks, wave);
  Stream vals(a.v + (int64_t)sq.k0 * a.vs + (int64_t)hk * kHd, a.vs, wave);
  const uint32_t lds0 = lds_addr(lds);
  const float c2 = a.scale * kLog2e;

  const int row0 = slot * tall;
  const int rows = sq.ql - row0 < tall ? sq.ql - row0 : tall;
  const KeyTiles kt = key_tiles(shift + row0, shift + row0 + rows - 1, a.window, a.sinks, kFwdKeys);
  const int wave0 = wave * 32 % tall, mine = wave0 + (lane & 31);   // the wave's first query in the block, this lane's
  const int qrow = sq.q0 + row0 + (mine < rows ? mine : rows - 1);
  const int p = shift + row0 + mine;
  const int w_lo = shift + row0 + wave0, w_hi = w_lo + 31;  // positions of the wave's queries
  // Tiles past the wave's last query are only copied for the others.
  int seen = kt.count;
  while (seen > 0 && kt.key0(seen - 1, kFwdKeys) > w_hi) --seen;
  bf16x8 qf[kHd / 16];
#pragma unroll
  for (int kk = 0; kk < kHd / 16; ++kk)
    qf[kk] = load8(a.q + (int64_t)qrow * a.qs + (int64_t)h * kHd + 16 * kk + 8 * half);

  // Places of the tiles i, i + 1 and i + 2, those of keys first; turned with i.
  uint32_t place[3] = {lds0, lds0 + kTile, lds0 + 2 * kTile};
  constexpr int kValues = 3 * kTile;
  Row<kHd> st;
  st.clear();
  f32x16 s[2];
  bf16x8 pf[2][2];
  auto score = [&](uint32_t ktile, int b) { s[b] = score_tile<kHd>(ktile, 32 * b, qf); };
  auto values = [&](uint32_t vtile, int b) {
#pragma unroll
    for (int step = 0; step < 2; ++step)
#pragma unroll
      for (int d = 0; d < kHd / 32; ++d)
        st.o[d] = mfma(col_frag<kHd>(vtile, 32 * b + 16 * step, d), pf[b][step], st.o[d]);
  };
  // exp2 of 32 keys' scores: the packed probabilities, and their sum.  P is one bf16 in its
  // product with v, its sum is not rounded: relative error of o 0.0022, 0.0016 of it o's own
  // rounding.  A second bf16, as below for few queries, would add half of all products to a
  // kernel that they bound.
  auto exps = [&](f32x16 x, int b) {
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      x[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[j], c2, -st.m));
      sum[j & 1] += x[j];
    }
    pf[b][0] = pack_step(x, 0);
    pf[b][1] = pack_step(x, 1);
    return sum[0] + sum[1];
  };
  // Mask and exponentials of tile i.  The maximum is looked for only where a sum says that
  // the one in use is too low (as the first is): nothing is lost while exp2(s - m) grows,
  // for bf16 has the exponents of fp32, and where it outgrows them the sum is infinite, the
  // scores are still there, and the tile is done again.  (With every tile's maximum taken
  // first: 266 us against 262 at 4 x 4096 tokens, 16 and 8 heads of 128.  Moving
  // exponentials between the products, one half or all of them, made those turns longer by
  // more: 344 to 426 us against 289.)
  auto softmax = [&](int i) {
    const int key0 = kt.key0(i, kFwdKeys);
    const bool all = key0 + kFwdKeys - 1 <= w_lo && (a.window == 0 || key0 > w_hi - a.window);
    if (!all) {
      mask_tile(s[0], key0, p, a.window, a.sinks);
      mask_tile(s[1], key0 + 32, p, a.window, a.sinks);
    }
    float sum = exps(s[0], 0) + exps(s[1], 1);
    if (__any(sum > 0x1p20f)) {
      st.raise(half_max(fmaxf(tile_max(s[0]), tile_max(s[1]))) * c2);
      sum = exps(s[0], 0) + exps(s[1], 1);
    }
    st.l += sum;
  };

  if (kt.count > 0) {
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      keys.aim(kt, t);
      keys.aim_rows(kt, t);
      vals.aim(kt, t);
      vals.aim_rows(kt, t);
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        keys.copy(part, place[t]);
        if (t < 2) vals.copy(part, place[t] + kValues);
      }
    }
    keys.aim(kt, 3);
    keys.aim_rows(kt, 3);
  }
  arrived(qf);
  landed();
  meet();
  if (seen > 0) {
    score(place[0], 0);
    score(place[0], 1);
    if (!late) softmax(0);
  }
  meet();
  if (late) {
    if (seen > 0) softmax(0);
    meet();
  }
  int i = 0;
  // To the next tile: bases and places, then the rows.
  auto turn = [&]() {
    keys.aim(kt, i + 4);
    vals.aim(kt, i + 3);
    const uint32_t p = place[0];
    place[0] = place[1];
    place[1] = place[2];
    place[2] = p;
  };
  auto turn_rows = [&]() {
    keys.aim_rows(kt, i + 4);
    vals.aim_rows(kt, i + 3);
  };
  for (; i + 1 < seen; ++i) {
    const uint32_t ktile = place[1], vtile = place[0] + kValues;
    score(ktile, 0);
    keys.copy(0, place[0]);
    score(ktile, 1);
    vals.copy(0, place[2] + kValues);
    values(vtile, 0);
    if (kParts > 1) keys.copy(kParts - 1, place[0]);
    values(vtile, 1);
    if (kParts > 1) vals.copy(kParts - 1, place[2] + kValues);
    turn();
    feed<4, kHd / 8, kHd / 8>();
    meet();
    __builtin_amdgcn_s_setprio(3);      // before the products of the SIMD's other wave: 262 -> 259 us
    softmax(i + 1);
    turn_rows();
    __builtin_amdgcn_s_setprio(0);
    landed();
    meet();
  }
  for (; i < kt.count; ++i) {
    if (i + 1 == seen) {
      values(place[0] + kValues, 0);
      values(place[0] + kValues, 1);
    }
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
      keys.copy(part, place[0]);
      vals.copy(part, place[2] + kValues);
    }
    turn();
    turn_rows();
    meet();
    landed();
    meet();
  }
  if (!late) meet();

  const float l = half_sum(st.l);
  if (mine < rows) {
    const float f = l == 0.0f ? 0.0f : 1.0f / l;            // 0: nothing seen; NaN stays NaN
    uint16_t *orow = a.o + (int64_t)qrow * a.os + (int64_t)h * kHd;
#pragma unroll
    for (int d = 0; d < kHd / 32; ++d) store_block(orow + 32 * d, st.o[d], f);
    if (a.lse && half == 0)
      a.lse[(int64_t)h * a.q_tokens + qrow] = l == 0.0f ? -__builtin_inff() : (st.m + __builtin_log2f(l)) * kLn2;
  }
}

// ---------------------------------------------------------------- few queries
// Partials of one (tile, key head, split): kSplitRows rows of kHd values, then m
// and l of each row.
template <int kHd>
__device__ __host__ constexpr size_t split_floats() {
  return (size_t)kSplitRows * (kHd + 2);
}

// Bound by memory with single queries: keys and values are read once, 32 rows share them.
// A row of a tile is (query, head of the group): rows of a sequence are numbered
// query * group + head, so that the heads that share keys share the tile.  Each
// wave keeps its own two places for keys and two for values in LDS and waits for nobody;
// the waves' states are joined at the end.  One query over 131071 keys, 16 and 8 heads of
// 128: 537 MB in 99 us and 6 more for the join (138 us with one tile of read-ahead and one
// load at a time in the join); 64 queries of 64 sequences over up to 8192 keys with a
// window of 4096: 988 MB in 175 us, some of it from the last-level cache.
template <int kHd>
__global__ void __launch_bounds__(64 * kSplitWaves) attn_split_kernel(AttnArgs a, int splits) {
  constexpr int kTile = kTileBytes<kHd>(kSplitKeys);
  constexpr int kCopies = kSplitKeys / kGroupRows<kHd>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kSplitWaves][4 * kTile];
  __shared__ float stat[kSplitWaves][2][kSplitRows];
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = (int)(blockIdx.x % a.k_heads);
  const int rest = (int)(blockIdx.x / a.k_heads);
  const int split = rest % splits, tile = rest / splits;
  int slot = tile;
  int sequence;
  const Seq sq = find_seq(a, a.q_start, a.group, kSplitRows, slot, sequence);
  const int all_rows = sq.ql * a.group;
  if ((int64_t)slot * kSplitRows >= all_rows) return;
  const int row0 = slot * kSplitRows;
  const int rows = all_rows - row0 < kSplitRows ? all_rows - row0 : kSplitRows;
  const int shift = sq.kl - sq.ql;
  const KeyTiles kt = key_tiles(shift + row0 / a.group, shift + (row0 + rows - 1) / a.group, a.window, a.sinks, kSplitKeys);

  const int mine = lane & 31;
  const int r = row0 + (mine < rows ? mine : rows - 1);
  const int qi = r / a.group, h = hk * a.group + r % a.group;
  const int qrow = sq.q0 + qi, p = shift + qi;
  const int p_lo = shift + row0 / a.group, p_hi = shift + (row0 + rows - 1) / a.group;
  bf16x8 qf[kHd / 16];
#pragma unroll
  for (int kk = 0; kk < kHd / 16; ++kk)
    qf[kk] = load8(a.q + (int64_t)qrow * a.qs + (int64_t)h * kHd + 16 * kk + 8 * half);

  const TileCopy<kHd> keys(a.k + (int64_t)sq.k0 * a.ks + (int64_t)hk * kHd, a.ks);
  const TileCopy<kHd> vals(a.v + (int64_t)sq.k0 * a.vs + (int64_t)hk * kHd, a.vs);
  const uint32_t lds0 = lds_addr(lds[wave]);
  // Chunk i's keys at the places 0 and 1 in turn, its values at 2 and 3.
  auto copy_keys = [&](int i, int odd) {
#pragma unroll
    for (int g = 0; g < kCopies; ++g) keys(kt, i, kSplitKeys, g, lds0 + (uint32_t)(odd * kTile));
  };
  auto copy_values = [&](int i, int odd) {
#pragma unroll
    for (int g = 0; g < kCopies; ++g) vals(kt, i, kSplitKeys, g, lds0 + (uint32_t)((2 + odd) * kTile));
  };

  Row<kHd> st;
  st.clear();
  const float c2 = a.scale * kLog2e;
  const int begin = (int)((int64_t)kt.count * split / splits), end = (int)((int64_t)kt.count * (split + 1) / splits);
  // Copies run two chunks ahead, each issued as soon as its place has been read: keys
  // after the scores, values after their products.  Waiting for one tile then leaves
  // the three younger ones under way.
  auto younger = [&](bool three) {
    if (!three) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    else if (kCopies == 8) asm volatile("s_waitcnt vmcnt(24)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(12)" ::: "memory");
  };
  auto read = [&]() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };
  int i = begin + wave;
  if (i < end) {
    copy_keys(i, 0);
    copy_values(i, 0);
  }
  if (i + kSplitWaves < end) {
    copy_keys(i + kSplitWaves, 1);
    copy_values(i + kSplitWaves, 1);
  }
  arrived(qf);                                        // and the copies before: from here on only copies are counted
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  for (int odd = 0; i < end; i += kSplitWaves, odd ^= 1) {
    const bool one = i + kSplitWaves < end, two = i + 2 * kSplitWaves < end;    // chunks that follow
    const int key0 = kt.key0(i, kSplitKeys);
    const uint32_t ktile = lds0 + (uint32_t)(odd * kTile), vtile = ktile + 2 * kTile;
    younger(one);
    f32x16 s = score_tile<kHd>(ktile, 0, qf);
    feed<4, kHd / 16, 0>();
    if (two) {
      read();
      copy_keys(i + 2 * kSplitWaves, odd);
    }
    const bool all = key0 + kSplitKeys - 1 <= p_lo && (a.window == 0 || key0 > p_hi - a.window);
    if (!all) mask_tile(s, key0, p, a.window, a.sinks);
    st.raise(half_max(tile_max(s)) * c2);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      s[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j], c2, -st.m));
      st.l += s[j];
    }
    younger(two);
#pragma unroll
    for (int step = 0; step < 2; ++step) {
      // P in two parts, so that its rounding adds nothing to the output's own (relative error
      // 0.0016 instead of 0.0023).  Where memory is the bound, the matrix cores have time for
      // it (single tokens: unchanged; 1 x 512 queries over 16896 keys: 192 -> 209 us).
      const bf16x8 pf = pack_step(s, step), pr = pack_rest(s, step, pf);
#pragma unroll
      for (int d = 0; d < kHd / 32; ++d) {
        const bf16x8 v = col_frag<kHd>(vtile, 16 * step, d);
        st.o[d] = mfma(v, pf, st.o[d]);
        st.o[d] = mfma(v, pr, st.o[d]);
      }
    }
    feed<4, 0, kHd / 16, 2>();
    if (two) {
      read();
      copy_values(i + 2 * kSplitWaves, odd);
    }
  }

  // Join the waves: each scales its state to the common maximum, wave by wave in
  // order, through LDS (which no copy needs any more).
  const float l = half_sum(st.l);
  if (half == 0) {
    stat[wave][0][mine] = st.m;
    stat[wave][1][mine] = l;
  }
  __syncthreads();
  float m = kNoMax, sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kSplitWaves; ++w) m = fmaxf(m, stat[w][0][mine]);
#pragma unroll
  for (int w = 0; w < kSplitWaves; ++w) sum += stat[w][1][mine] * __builtin_amdgcn_exp2f(stat[w][0][mine] - m);
  const float f = __builtin_amdgcn_exp2f(st.m - m);
  // Each wave's own part holds its scaled accumulators, [d][row]: 32 floats a row of
  // d, one bank row for the 32 queries.
  float *acc = reinterpret_cast<float *>(lds[wave]);
#pragma unroll
  for (int d = 0; d < kHd / 32; ++d)
#pragma unroll
    for (int j = 0; j < 16; ++j)
      acc[(32 * d + 8 * (j / 4) + 4 * half + j % 4) * kSplitRows + mine] = st.o[d][j] * f;
  __syncthreads();
  // Wave w takes columns w * kHd/4 .. of every row: lane = row (both halves split them).
  constexpr int kCols = kHd / kSplitWaves / 2;
  const int d0 = (wave * 2 + half) * kCols;
  float out[kCols];
#pragma unroll
  for (int j = 0; j < kCols; ++j) {
    float x = 0.0f;
#pragma unroll
    for (int w = 0; w < kSplitWaves; ++w)
      x += reinterpret_cast<const float *>(lds[w])[(d0 + j) * kSplitRows + mine];
    out[j] = x;
  }
  if (mine >= rows) return;
  if (splits == 1) {
    const float g = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t *orow = a.o + (int64_t)qrow * a.os + (int64_t)h * kHd + d0;
#pragma unroll
    for (int j = 0; j < kCols; j += 8) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = pack_bf16(out[j + 2 * e] * g, out[j + 2 * e + 1] * g);
      *reinterpret_cast<u32x4 *>(orow + j) = w;
    }
    if (a.lse && wave == 0 && half == 0)
      a.lse[(int64_t)h * a.q_tokens + qrow] = sum == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(sum)) * kLn2;
  } else {
    float *part = a.ws + ((size_t)((size_t)tile * a.k_heads + hk) * splits + split) * split_floats<kHd>();
#pragma unroll
    for (int j = 0; j < kCols; j += 4)
      *reinterpret_cast<f32x4 *>(part + mine * kHd + d0 + j) = (f32x4){out[j], out[j + 1], out[j + 2], out[j + 3]};
    if (wave == 0 && half == 0) {
      part[kSplitRows * kHd + mine] = m;
      part[kSplitRows * kHd + kSplitRows + mine] = sum;
    }
  }
}

// One wave a row: lanes first as splits (the maxima and sums of up to 128 of them),
// then as columns, kHd / 64 each, eight splits' partials in flight.
template <int kHd>
__global__ void __launch_bounds__(256) attn_join_kernel(AttnArgs a, int splits) {
  constexpr int kPer = kHd / 64;
  typedef float cols __attribute__((ext_vector_type(kPer)));
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = (int)(blockIdx.x % a.k_heads);
  const int rest = (int)(blockIdx.x / a.k_heads);
  const int mine = (rest % (kSplitRows / 4)) * 4 + wave, tile = rest / (kSplitRows / 4);
  int slot = tile;
  int sequence;
  const Seq sq = find_seq(a, a.q_start, a.group, kSplitRows, slot, sequence);
  if ((int64_t)slot * kSplitRows + mine >= sq.ql * a.group) return;
  const int r = slot * kSplitRows + mine;
  const int qrow = sq.q0 + r / a.group, h = hk * a.group + r % a.group;
  const float *part = a.ws + (size_t)((size_t)tile * a.k_heads + hk) * splits * split_floats<kHd>();
  float ms[2], ls[2], m = kNoMax, sum = 0.0f;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int s = 64 * w + lane;
    const float *stat = part + (s < splits ? s : 0) * split_floats<kHd>() + kSplitRows * kHd + mine;
    ms[w] = s < splits ? stat[0] : kNoMax;
    ls[w] = s < splits ? stat[kSplitRows] : 0.0f;
  }
  m = wave_max(fmaxf(ms[0], ms[1]));
#pragma unroll
  for (int w = 0; w < 2; ++w) ms[w] = __builtin_amdgcn_exp2f(ms[w] - m);
  for (int s = 0; s < splits; ++s)      // in order, as the columns below
    sum += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s < 64 ? ms[0] * ls[0] : ms[1] * ls[1]), s & 63));
  float x[kPer] = {};
  for (int s0 = 0; s0 < splits; s0 += 8) {
    cols one[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int s = s0 + e < splits ? s0 + e : splits - 1;
      one[e] = *reinterpret_cast<const cols *>(part + s * split_floats<kHd>() + mine * kHd + kPer * lane);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int s = s0 + e;
      const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s < 64 ? ms[0] : ms[1]), s & 63));
      const float f = s < splits ? w : 0.0f;
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[j] += one[e][j] * f;
    }
  }
  const float g = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t *orow = a.o + (int64_t)qrow * a.os + (int64_t)h * kHd;
  if (kPer == 2)
    *reinterpret_cast<uint32_t *>(orow + 2 * lane) = pack_bf16(x[0] * g, x[kPer - 1] * g);
  else
    orow[lane] = (uint16_t)pack_bf16(x[0] * g, 0.0f);
  if (a.lse && lane == 0)
    a.lse[(int64_t)h * a.q_tokens + qrow] = sum == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(sum)) * kLn2;
}

template <int kHd>
hipError_t launch(const AttnArgs &a, const AttnPlan &plan, hipStream_t stream) {
  const auto grid = [](int64_t blocks) { return dim3((unsigned)blocks); };
  if (!plan.split) {
    attn_kernel<kHd><<<grid(fwd_blocks(plan, a.q_heads, a.sequences, a.window)), dim3(64 * kFwdWaves), 0, stream>>>(
        a, plan.slots, plan.pack);
    return hipGetLastError();
  }
  attn_split_kernel<kHd><<<grid(split_blocks(plan, a.k_heads)), dim3(64 * kSplitWaves), 0, stream>>>(a, plan.splits);
  if (hipError_t e = hipGetLastError()) return e;
  if (plan.splits > 1) {
    attn_join_kernel<kHd><<<grid(split_join_blocks(plan, a.k_heads)), dim3(256), 0, stream>>>(a, plan.splits);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace

AttnPlan plan_attention(const puro_attention_shape &a) { return forward_plan(a); }

hipError_t run_attention(const AttnArgs &a, int head_dim, const AttnPlan &plan, hipStream_t stream) {
  return head_dim == 128 ? launch<128>(a, plan, stream) : launch<64>(a, plan, stream);
}

}  // namespace puro
