// The attention kernels' plans (csrc/attention_plan.h) for tests/attention_plan.py, built for the host.  Tests only.
#include "attention_plan.h"

using namespace puro;

namespace {

AttnArgs args(const puro_attention_shape &s) {
  AttnArgs a{};
  a.q_tokens = (int)s.q_tokens;
  a.k_tokens = (int)s.k_tokens;
  a.sequences = (int)s.sequences;
  a.q_heads = (int)s.q_heads;
  a.k_heads = (int)s.k_heads;
  a.group = (int)(s.q_heads / s.k_heads);
  a.window = (int)s.window;
  a.sinks = (int)s.sinks;
  return a;
}

}  // namespace

// A shape as the launchers get it (its idle window dropped).
// out: few queries' kernel, heads of a workgroup, splits; workgroups of the first launch and its threads, of the join.
extern "C" void forward(const puro_attention_shape *s, int64_t *out) {
  const AttnArgs a = args(*s);
  const AttnPlan p = forward_plan(*s);
  out[0] = p.split;
  out[1] = p.pack;
  out[2] = p.splits;
  out[3] = p.split ? split_blocks(p, a.k_heads) : fwd_blocks(p, a.q_heads, a.sequences, a.window);
  out[4] = 64 * (p.split ? kSplitWaves : kFwdWaves);
  out[5] = p.splits > 1 ? split_join_blocks(p, a.k_heads) : 0;
}

// out: heads of a workgroup of the kernel for dq, parts of near walks, key blocks with far work; workgroups of 256 threads
// of dq, of dk and dv, of their join.
extern "C" void backward(const puro_attention_shape *s, int64_t *out) {
  const AttnArgs a = args(*s);
  const int pack = pack_of(a.group);
  const DkPlan p = plan_dk(a.q_tokens, a.k_tokens, a.sequences, a.q_heads, a.k_heads, s->head_dim, a.window, a.sinks);
  out[0] = pack;
  out[1] = p.parts;
  out[2] = p.far_blocks;
  out[3] = dq_blocks(dq_slots(a.q_tokens, a.sequences, pack), pack, a.q_heads, a.sequences, a.window);
  out[4] = dk_blocks(p, a.k_heads, a.sequences, a.window);
  out[5] = p.parts > 1 || p.far_blocks > 0 ? dk_join_blocks(p, a.k_heads, s->head_dim) : 0;
}

// out: waves a token, launches, workgroups of 256 threads of the largest.
extern "C" void rope(int64_t tokens, int64_t heads, int64_t head_dim, int64_t *out) {
  const RopePlan p = plan_rope(tokens, heads, head_dim);
  out[0] = p.parts;
  out[1] = (tokens + p.tokens - 1) / p.tokens;
  out[2] = rope_blocks(p, tokens < p.tokens ? tokens : p.tokens);
}
