// Internal launchers behind puro_attention.h (host side).  Arguments are
// already validated by the ABI layer when these run.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "puro_attention.h"

namespace puro {

hipError_t run_rope_table(int64_t positions, int64_t rot, double base, int scaling, double factor, int64_t trained,
                          float *table, hipStream_t stream);

// The rotation and the head norms of one launch: x rows of q_heads + k_heads
// (+ v_heads) heads to q, k (and v).  The plain rotation has all its heads as
// query heads and no weights; the append form has rows.
struct RopeArgs {
  const uint16_t *x;
  int64_t xs, tokens;
  int heads_q, heads_k, heads_v;
  const uint16_t *wq, *wk;
  float eps;
  const float *table;
  int64_t positions;
  int rot;
  const int32_t *pos;
  float sign;            // of the sines: -1 for the inverse
  uint16_t *q, *k, *v;
  int64_t qs, ks, vs;
  const int32_t *rows;
  int64_t cache_rows;
};
hipError_t run_rope(const RopeArgs &a, int head_dim, bool interleaved, hipStream_t stream);

struct RopeBackArgs {
  const uint16_t *dq, *dk, *x;
  int64_t dqs, dks, xs, tokens;
  int heads_q, heads_k;
  const uint16_t *wq, *wk;
  float eps;
  const float *table;
  int64_t positions;
  int rot;
  const int32_t *pos;
  uint16_t *dx;
  int64_t dxs;
  float *dwq, *dwk;
  float *partial;        // [rope_back_blocks][2][head_dim]
};
int rope_back_blocks(int64_t tokens);
hipError_t run_rope_back(const RopeBackArgs &a, int head_dim, bool interleaved, hipStream_t stream);

struct AttnArgs {
  const uint16_t *q, *k, *v;
  uint16_t *o;
  float *lse;                                  // may be NULL in the forward call
  int64_t qs, ks, vs, os;
  int q_tokens, k_tokens, sequences;
  int q_heads, k_heads, group;                 // group = q_heads / k_heads
  const int32_t *q_start, *k_start, *k_len;
  int window, sinks;
  float scale;
  // backward
  const uint16_t *d_o;
  uint16_t *dq, *dk, *dv;
  int64_t dqs, dks, dvs;
  // workspace
  float *ws;
};

// How a forward call is launched (host only, deterministic).
struct AttnPlan {
  bool split;        // the kernel for few queries: 32 (query, head) rows a tile, keys over waves and splits
  int slots;         // query tiles, empty ones included
  int pack;          // heads of a workgroup of the kernel for many queries
  int splits;        // key ranges of a tile
  size_t ws_bytes;   // fp32 partials, when splits > 1
};
AttnPlan plan_attention(const puro_attention_shape &a);
hipError_t run_attention(const AttnArgs &a, int head_dim, const AttnPlan &plan, hipStream_t stream);

size_t attention_backward_ws_bytes(const puro_attention_shape &a);
hipError_t run_attention_backward(const AttnArgs &a, int head_dim, hipStream_t stream);

}  // namespace puro
