// How the attention kernels are launched, from sizes alone: tiles, which kernel, splits and
// parts, workspaces, workgroups.  Host code (but for Order), kept apart from the kernels so that
// it can be built and looked at without them.
#pragma once

#include <initializer_list>

#include "launch_attention.h"

namespace puro {

// ---------------------------------------------------------------- tiles
// Many queries: (query, head) rows of a workgroup, 32 a wave; `pack` heads of a group by
// kFwdRows / pack queries.
constexpr int kFwdWaves = 8, kFwdKeys = 64, kFwdRows = 32 * kFwdWaves;
// Few queries.
constexpr int kSplitWaves = 4, kSplitRows = 32, kSplitKeys = 32, kMostSplits = 128;
// Backward: queries of a workgroup of the kernel for dq, keys of one of the kernel for dk and dv.
constexpr int kDqWaves = 4, kDqRows = 32 * kDqWaves, kDqKeys = 64;
constexpr int kDkWaves = 4, kDkRows = 32 * kDkWaves, kDkQueries = 64;

// Heads that share keys and a workgroup.
inline int pack_of(int64_t group) { return group % 4 == 0 ? 4 : group % 2 == 0 ? 2 : 1; }

// Order in which tiles start.  Without a window a tile's work grows along its sequence:
// the x-th numbers of `sequences` equal parts of the number line come before the next of
// any, so that (with sequences alike) those that walk far start first in all of them and
// the short ones fill the end.  A permutation in any case, up to numbers past the end,
// which are no tiles.  4 x 4096 tokens backward: 1094 -> 975 us.  With a window the work
// is even, and neighbours in the sequence share keys: as numbered.
struct Order {
  int slots, parts;
  __device__ __host__ __forceinline__ Order(int slots, int sequences, int window)
      : slots(slots), parts(window > 0 ? 1 : sequences) {}
  __device__ __host__ __forceinline__ int each() const { return (slots + parts - 1) / parts; }
  __device__ __host__ __forceinline__ int count() const { return each() * parts; }
  __device__ __forceinline__ int operator()(int x) const { return x % parts * each() + x / parts; }
};

// ---------------------------------------------------------------- forward
// Both kernels' times are estimated from the average sequence and the smaller wins.  A
// workgroup costs a fixed time and one for each 64 (128) keys it walks, and 256 of them
// run at a time; the constants, in us, are fitted to 42 shapes of heads of 128 and 104 of
// heads of 64, with 1 to 64 sequences, 8 to 4096 queries and up to 16384 earlier keys (on
// average 0.2% slower than the better kernel, 7% at worst).  Examples (many / few queries'
// kernel), 16 and 8 heads of 128: 64 x 8 queries over 2056 keys 145 / 127 us; 16 x 64 over
// 2112 49 / 63; 1 x 256 over 256 14.6 / 8.3; 8 x 512 over 512 23 / 69; 1 x 1500 over 1500
// 37 / 49; 1 x 4096 over 4096 92 / 252; 1 x 512 over 16896 309 / 210.
inline AttnPlan forward_plan(const puro_attention_shape &a) {
  AttnPlan p{};
  const double units = 256.0;
  const int64_t group = a.q_heads / a.k_heads;
  const int64_t few = a.q_tokens * group / kSplitRows + a.sequences;
  const double ql = (double)a.q_tokens / a.sequences;
  double kl = a.max_k > 0 ? (double)a.max_k : (double)a.k_tokens / a.sequences;
  const double far = a.window > 0 ? (double)(a.window + a.sinks) : kl;
  // Keys that a tile of `rows` queries walks, at most and on average.
  auto most = [&](double rows) {
    const double see = far + (rows < ql ? rows : ql);
    return kl < see ? kl : see;
  };
  auto mean = [&](double rows) {
    const double all = kl > ql / 2 ? kl - ql / 2 : 0;
    return all < most(rows) ? all : most(rows);
  };

  // Few queries' kernel: splits fill the units once, empty tiles counted (a 257th
  // workgroup waits for a place: 16 x 16 queries over 2064 keys took 38 us split in two,
  // 30 us whole), and hold at least 4 chunks of keys a wave.
  const double wf = (double)a.sequences * (int64_t)((ql * group + kSplitRows - 1) / kSplitRows) * a.k_heads;
  int64_t splits = 256 / (few * a.k_heads);
  const int64_t longest = (int64_t)(most(1) / (4 * kSplitWaves * kSplitKeys));
  if (splits > longest) splits = longest;
  if (splits > kMostSplits) splits = kMostSplits;
  if (splits < 1) splits = 1;
  const bool wide = a.head_dim == 128;
  const double per_few = wide ? 2.2 : 0.9, per_many = wide ? 1.25 : 1.3, start_few = wide ? 6 : 3, start_many = wide ? 7 : 6;
  const double walk_few = wf < units ? most(1) / splits : mean(1);
  const double t_few = (wf < units ? 1 : wf / units) * (start_few + per_few * walk_few / (kSplitWaves * kSplitKeys));
  // Heads that share keys share a workgroup: lower blocks see fewer keys that only some
  // of their queries see (heads alone / in twos / in fours, us: 287 / 280 / - at 4 x 4096
  // tokens, 194 / 186 / - at 16381 with a window of 1024, 16 and 8 heads of 128; - / 51 /
  // 46 at 8192 with a window of 512, 16 and 4 heads of 64).
  p.pack = pack_of(group);
  const int tall = kFwdRows / p.pack;
  const double wm = (double)a.sequences * (int64_t)((ql + tall - 1) / tall) * (a.q_heads / p.pack);
  const double walk_many = wm < units ? most(tall) : mean(tall);
  const double t_many = (wm < units ? 1 : wm / units) * (start_many + per_many * walk_many / kFwdKeys);

  p.split = t_few < t_many;
  p.splits = 1;
  p.slots = (int)(p.split ? few : a.q_tokens / tall + a.sequences);
  if (p.split && splits > 1) {
    p.splits = (int)splits;
    p.ws_bytes = (size_t)few * (size_t)a.k_heads * (size_t)splits * (size_t)kSplitRows * (size_t)(a.head_dim + 2) * 4;
  }
  return p;
}

// Workgroups of each launch.
inline int64_t fwd_blocks(const AttnPlan &p, int64_t q_heads, int sequences, int window) {
  return (int64_t)Order(p.slots, sequences, window).count() * (q_heads / p.pack);
}
inline int64_t split_blocks(const AttnPlan &p, int64_t k_heads) { return (int64_t)p.slots * k_heads * p.splits; }
inline int64_t split_join_blocks(const AttnPlan &p, int64_t k_heads) {
  return (int64_t)p.slots * k_heads * (kSplitRows / 4);
}

// ---------------------------------------------------------------- backward
inline int dq_slots(int q_tokens, int sequences, int pack) { return q_tokens / (kDqRows / pack) + sequences; }
inline int64_t dq_blocks(int slots, int pack, int64_t q_heads, int sequences, int window) {
  return (int64_t)Order(slots, sequences, window).count() * (q_heads / pack);
}

// Work on one block of 128 keys and one key head: tiles of 64 queries of each head of
// the group.  `near` tiles hold the queries that have the block in their window; for a
// block of first keys `far` tiles hold the later queries, which see the first keys
// only.  Without far work such a block would walk its whole sequence while all others
// walk a window.  Either walk is cut into parts where it is long for the card (many
// heads over few keys; a long sequence past its first keys), which leave fp32 partials
// for the join.
struct DkPlan {
  int slots;          // key blocks, empty ones included
  int parts;          // of each near walk
  int far_blocks;     // key blocks of a sequence that hold first keys; 0: no far work
  int far_slots;      // parts of far walks over all sequences, empty ones included
  size_t near_at, edge_at, far_at, floats;   // partials in the workspace, in floats: of near walks, of near walks over
                                             // first keys that are not cut, of far walks
};
constexpr int kFarChunk = 24;     // tiles of a far part: about a near walk's, whose workgroups run beside it

inline DkPlan plan_dk(int64_t q_tokens, int64_t k_tokens, int64_t sequences, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                      int64_t window, int64_t sinks) {
  DkPlan p{};
  const int64_t floats = 2 * kDkRows * head_dim;
  p.slots = (int)(k_tokens / kDkRows + sequences);
  const int64_t group = q_heads / k_heads;
  const int64_t per_seq = (q_tokens + sequences - 1) / sequences;
  // Near walks are cut into the number of parts with the least estimated time, in us: the
  // longest part alone, or all parts over the places of the card (256 compute units, two
  // workgroups each, three with heads of 64), and the partials' way through memory.  The
  // constants are fitted to 112 shapes of 1 to 64 sequences of 128 to 16384 tokens: 0.8%
  // slower on average than the best number, 9% at worst.  The whole backward call, causal,
  // 1 / 2 / 3 / 4 / 6 / 8 parts, us (dq has since become 7 to 12% slower, for any number):
  // 4096 tokens, 16 and 8 heads of 128: 380 / 302 / 276 / 282 / 309 / 351; 4 x 4096: 860 / 932 /
  // 979 / 1033 / 1138 / 1263; 8 x 2048, 8 heads and 1 of 128: 625 / 384 / 319 / 291 / 267 / 281;
  // 8192, 16 and 4 of 64: 839 / 596 / 528 / 502 / 506 / 505.
  const bool windowed = window > 0 && window + kDkRows < per_seq;
  const int64_t seen = windowed ? window + kDkRows : per_seq;
  const int64_t longest = (seen + kDkQueries - 1) / kDkQueries * group;
  const double average = windowed ? (double)longest : (double)(longest + group) / 2;
  const int64_t keys = (k_tokens + sequences - 1) / sequences;
  const double blocks = (double)sequences * ((keys + kDkRows - 1) / kDkRows) * k_heads;
  double best = 0;
  for (int parts : {1, 2, 3, 4, 6, 8, 12, 16}) {
    if (parts > 1 && longest < 2 * parts) break;
    const double alone = 2.0 * longest / parts + 2;
    const double all = 3.0 * blocks * (average + 2 * parts) / (head_dim == 128 ? 512 : 768);
    const double time = (alone > all ? alone : all) + (parts > 1 ? 4 + 0.08 * blocks * parts * head_dim / 128 : 0);
    if (parts > 1 && time >= best) continue;
    best = time;
    p.parts = parts;
  }
  p.near_at = ((size_t)2 * q_heads * q_tokens + 63) / 64 * 64;
  p.floats = p.near_at + (p.parts > 1 ? (size_t)p.slots * k_heads * p.parts * floats : 0);
  p.edge_at = p.far_at = p.floats;
  // Far work pays where a sequence may be several windows long; many first keys make
  // enough blocks by themselves, and partials for them would be large.
  if (window > 0 && sinks > 0 && sinks <= 2 * kDkRows && q_tokens >= 2 * (window + kDkRows)) {
    p.far_blocks = (int)((sinks + kDkRows - 1) / kDkRows);
    p.far_slots = (int)(q_tokens * group / (kFarChunk * kDkQueries) + sequences);
    p.far_at = p.edge_at + (p.parts == 1 ? (size_t)sequences * p.far_blocks * k_heads * floats : 0);
    p.floats = p.far_at + (size_t)p.far_slots * p.far_blocks * k_heads * floats;
  }
  return p;
}

inline int64_t dk_blocks(const DkPlan &p, int64_t k_heads, int sequences, int window) {
  return ((int64_t)p.far_slots * p.far_blocks + (int64_t)Order(p.slots, sequences, window).count() * p.parts) * k_heads;
}
// The join's share of a workgroup: 256 threads of 8 columns.  Its workgroups stride over the shares, since the runtime takes
// fewer than 2^32 threads.
inline int64_t dk_join_shares(const DkPlan &p, int64_t k_heads, int64_t head_dim) {
  return (int64_t)p.slots * (kDkRows / (256 / (head_dim / 8))) * k_heads;
}
inline int64_t dk_join_blocks(const DkPlan &p, int64_t k_heads, int64_t head_dim) {
  const int64_t shares = dk_join_shares(p, k_heads, head_dim), most = (int64_t(1) << 24) - 1;
  return shares < most ? shares : most;
}

// ---------------------------------------------------------------- rotation
constexpr int kRopeWaves = 4;      // waves of a workgroup

struct RopePlan {
  int parts;          // waves a token
  int64_t tokens;     // of a launch, at most: the runtime takes fewer than 2^32 threads
};

inline RopePlan plan_rope(int64_t tokens, int64_t heads, int64_t head_dim) {
  const int64_t teams = 512 / head_dim, groups = (heads + teams - 1) / teams;       // heads that a wave reads at once
  // Waves a token: one where the tokens alone fill the card, one per group of heads where
  // they are few, so that no wave loops.  Norms of 24 heads of 128, back to back in a graph,
  // 1 / 2 / 3 / 6 waves, us: 32 tokens 4.7 / 3.5 / 3.2 / 3.0; 512 tokens 5.2 / 4.0 / 4.1 /
  // 4.2; 2048 tokens 8.4 / 8.1 / 7.9 / 9.5; 4096 tokens 11.4 / 12.6 / 12.9 / 15.6; 16384
  // tokens 37.1 / 38.6 / 42.7 / 60.5.
  const int64_t parts = tokens >= 4096 ? 1 : tokens >= 512 ? 2 : groups;
  return RopePlan{(int)(parts < groups ? parts : groups), int64_t(1) << 25};
}
inline int64_t rope_blocks(const RopePlan &p, int64_t tokens) { return (tokens * p.parts + kRopeWaves - 1) / kRopeWaves; }

}  // namespace puro
