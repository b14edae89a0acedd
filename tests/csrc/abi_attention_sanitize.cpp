// Host-only driver of the attention block's ABI layer (blockwise_fp8_gemm_act_amd/
// csrc/abi_attention.cpp), built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_abi_attention_sanitized.py.  Tests only.
//
// The HIP calls and the launchers behind the layer are stubs that record what they
// are given; no pointer is dereferenced by the layer, so buffers are fake addresses.
// Checked: valid calls reach their launcher with the caller's arguments (the idle
// window dropped, absent weights replaced), error paths reach none, and sizes at the
// limits evaluate without undefined behaviour.  Prints "abi under sanitizers: ok".
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <string>

#include "launch_attention.h"
#include "puro_attention.h"

hipError_t hipGetDevice(int *dev) {
  *dev = 0;
  return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_t *prop, int) {
  std::memset(prop, 0, sizeof(*prop));
  std::strcpy(prop->gcnArchName, "gfx950:sramecc+:xnack-");
  return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }

namespace {
std::string g_name;
int g_calls = 0;
puro::RopeArgs g_rope;
puro::RopeBackArgs g_back;
puro::AttnArgs g_attn;
int g_hd;
bool g_inter;
hipError_t g_result = hipSuccess;

hipError_t record(const char *name) {
  g_name = name;
  ++g_calls;
  return g_result;
}
}  // namespace

namespace puro {
hipError_t run_rope_table(int64_t, int64_t, double, int, double, int64_t, float *, hipStream_t) { return record("table"); }
hipError_t run_rope(const RopeArgs &a, int hd, bool inter, hipStream_t) {
  g_rope = a;
  g_hd = hd;
  g_inter = inter;
  return record("rope");
}
int rope_back_blocks(int64_t tokens) { return (int)(tokens < 1024 ? tokens : 1024); }
hipError_t run_rope_back(const RopeBackArgs &a, int hd, bool inter, hipStream_t) {
  g_back = a;
  g_hd = hd;
  g_inter = inter;
  return record("rope_back");
}
AttnPlan plan_attention(const puro_attention_shape &a) {
  AttnPlan p{};
  p.split = a.q_tokens < 64;
  p.splits = p.split && a.max_k > 4096 ? 4 : 1;
  p.ws_bytes = p.splits > 1 ? (size_t)a.q_tokens * (size_t)a.q_heads * 4 * 4 : 0;
  return p;
}
hipError_t run_attention(const AttnArgs &a, int hd, const AttnPlan &, hipStream_t) {
  g_attn = a;
  g_hd = hd;
  return record("attention");
}
size_t attention_backward_ws_bytes(const puro_attention_shape &a) { return (size_t)a.q_tokens * (size_t)a.q_heads * 8; }
hipError_t run_attention_backward(const AttnArgs &a, int hd, hipStream_t) {
  g_attn = a;
  g_hd = hd;
  return record("attention_backward");
}
}  // namespace puro

namespace {
int g_fail = 0;
#define CHECK(x)                                             \
  do {                                                       \
    if (!(x)) {                                              \
      std::printf("line %d: %s\n", __LINE__, #x);            \
      ++g_fail;                                              \
    }                                                        \
  } while (0)

template <typename T>
T *at(int i) {
  return reinterpret_cast<T *>((uintptr_t(1) << 40) + uintptr_t(i) * (uintptr_t(1) << 43));
}
uint16_t *h(int i) { return at<uint16_t>(i); }

// Status s, and no launcher reached.
#define REFUSED(call, s)             \
  do {                               \
    const int before = g_calls;      \
    CHECK((call) == (s));            \
    CHECK(g_calls == before);        \
  } while (0)
}  // namespace

int main() {
  puro_rotation r{at<float>(0), 4096, 64, PURO_ROPE_INTERLEAVED, at<int32_t>(1)};
  CHECK(puro_rope_table(4096, 64, 1e6, PURO_ROPE_YARN, 8.0, 4096, at<float>(0), nullptr) == PURO_OK && g_name == "table");
  REFUSED(puro_rope_table((int64_t)1 << 62, 64, 1e6, PURO_ROPE_PLAIN, 1.0, 0, at<float>(0), nullptr), PURO_ERR_SHAPE);

  CHECK(puro_rope(&r, 1, h(2), 4096, 100, 16, 128, h(3), 2048, nullptr) == PURO_OK);
  CHECK(g_name == "rope" && g_rope.x == h(2) && g_rope.q == h(3) && g_rope.xs == 4096 && g_rope.qs == 2048 && g_hd == 128 && g_inter);
  CHECK(g_rope.sign == -1.0f && !g_rope.wq && !g_rope.rows && g_rope.heads_q == 16 && g_rope.heads_k == 0 && g_rope.rot == 64);
  REFUSED(puro_rope(&r, 0, h(2), INT64_MAX / 8 * 8, 100, 16, 128, h(3), 2048, nullptr), PURO_ERR_SHAPE);
  REFUSED(puro_rope(&r, 0, h(2), 4096, INT64_MAX, 16, 128, h(3), 2048, nullptr), PURO_ERR_SHAPE);
  REFUSED(puro_rope(&r, 0, h(2), 4096, 100, INT64_MAX, 128, h(3), 2048, nullptr), PURO_ERR_SHAPE);
  REFUSED(puro_rope(&r, 0, h(2), 4096, 100, 16, INT64_MIN, h(3), 2048, nullptr), PURO_ERR_SHAPE);
  REFUSED(puro_rope(&r, 0, h(2), 4096, 100, 16, 128, h(2), 2048, nullptr), PURO_ERR_ALIAS);

  CHECK(puro_qk_norm_rope(&r, h(2), 4096, 100, 0, 8, 128, nullptr, h(4), 1e-6f, nullptr, 0, h(5), 1024, nullptr) == PURO_OK);
  CHECK(g_rope.wq == h(4) && g_rope.wk == h(4) && g_rope.k == h(5) && g_rope.heads_v == 0 && !g_rope.rows);
  CHECK(puro_qk_norm_rope_append(&r, h(2), 4096, 100, 16, 8, 128, h(3), h(4), 1e-6f, h(5), 2048, h(6), 1024, h(7), 1032, at<int32_t>(8),
                                 1 << 20, nullptr) == PURO_OK);
  CHECK(g_rope.heads_v == 8 && g_rope.rows == at<int32_t>(8) && g_rope.cache_rows == 1 << 20 && g_rope.v == h(7) && g_rope.vs == 1032);
  REFUSED(puro_qk_norm_rope_append(&r, h(2), 4096, 100, 16, 8, 128, h(3), h(4), 1e-6f, h(5), 2048, h(6), 1024, h(7), 1032,
                                   at<int32_t>(8), INT64_MAX, nullptr), PURO_ERR_SHAPE);

  const size_t need = puro_qk_norm_rope_backward_workspace_bytes(100, 128);
  CHECK(puro_qk_norm_rope_backward(&r, h(2), 2048, h(3), 1024, h(4), 4096, 100, 16, 8, 128, h(5), h(6), 1e-6f, h(7), 4096, at<float>(8),
                                   at<float>(9), h(10), need, nullptr) == PURO_OK);
  CHECK(g_name == "rope_back" && g_back.dq == h(2) && g_back.dk == h(3) && g_back.dx == h(7) && g_back.dwk == at<float>(9) && g_back.tokens == 100);
  REFUSED(puro_qk_norm_rope_backward(&r, h(2), 2048, h(3), 1024, h(4), 4096, 100, 16, 8, 128, h(5), h(6), 1e-6f, h(7), 4096, at<float>(8),
                                     at<float>(9), h(10), need - 1, nullptr), PURO_ERR_WORKSPACE);
  CHECK(puro_qk_norm_rope_backward_workspace_bytes(INT64_MAX, 128) == 0);

  puro_attention_shape a{};
  a.q_tokens = 100, a.k_tokens = 300, a.sequences = 2, a.q_heads = 16, a.k_heads = 8, a.head_dim = 128;
  a.q_stride = 2048, a.k_stride = 1024, a.v_stride = 4096, a.o_stride = 2048;
  a.dq_stride = 2048, a.dk_stride = 1024, a.dv_stride = 4096;
  a.window = 40, a.sinks = 1000, a.scale = 0.1f;
  auto fwd = [&](uint16_t *o, void *ws, size_t n) {
    return puro_attention(&a, h(0), h(1), h(2), at<int32_t>(3), at<int32_t>(4), at<int32_t>(5), o, at<float>(7), ws, n, nullptr);
  };
  auto back = [&](uint16_t *dv, size_t n) {
    return puro_attention_backward(&a, h(0), h(1), h(2), h(3), h(4), at<float>(5), at<int32_t>(6), at<int32_t>(7), h(8), h(9), dv, h(11), n,
                                   nullptr);
  };
  CHECK(fwd(h(6), nullptr, 0) == PURO_OK && g_name == "attention");
  CHECK(g_attn.window == 40 && g_attn.sinks == 300 && g_attn.group == 2 && g_attn.vs == 4096 && g_attn.k_len == at<int32_t>(5) && g_attn.o == h(6));
  a.window = 300;                                     // reaches every key: dropped, and the first keys with it
  CHECK(fwd(h(6), nullptr, 0) == PURO_OK && g_attn.window == 0 && g_attn.sinks == 0);
  a.window = INT64_MAX;
  a.sinks = INT64_MAX;
  CHECK(fwd(h(6), nullptr, 0) == PURO_OK && g_attn.window == 0 && g_attn.sinks == 0);
  a.window = 7;
  CHECK(back(h(10), 1 << 20) == PURO_OK && g_name == "attention_backward");
  CHECK(g_attn.d_o == h(0) && g_attn.dv == h(10) && g_attn.dvs == 4096 && g_attn.window == 7 && g_attn.sinks == 300 && !g_attn.k_len);
  REFUSED(back(h(9), 1 << 20), PURO_ERR_ALIAS);
  REFUSED(back(h(10), 5), PURO_ERR_WORKSPACE);
  REFUSED(fwd(h(0), nullptr, 0), PURO_ERR_ALIAS);
  for (int64_t *p : {&a.q_tokens, &a.k_tokens, &a.sequences, &a.q_heads, &a.k_heads, &a.head_dim, &a.q_stride, &a.k_stride, &a.v_stride, &a.o_stride}) {
    const int64_t was = *p;
    for (int64_t v : {INT64_MAX, INT64_MIN, INT64_MAX / 8 * 8, (int64_t)-8}) {
      *p = v;
      REFUSED(fwd(h(6), nullptr, 0), PURO_ERR_SHAPE);
      REFUSED(back(h(10), 1 << 20), PURO_ERR_SHAPE);
      CHECK(puro_attention_workspace_bytes(&a) == 0 && puro_attention_backward_workspace_bytes(&a) == 0);
    }
    *p = was;
  }
  // the largest sizes of the contract
  a.q_tokens = a.k_tokens = 1 << 30, a.sequences = 1, a.q_heads = a.k_heads = 1;
  a.q_stride = a.k_stride = a.v_stride = a.o_stride = a.dq_stride = a.dk_stride = a.dv_stride = 512;
  a.max_k = INT64_MAX;
  CHECK(fwd(h(6), nullptr, 0) == PURO_OK);
  g_result = hipErrorInvalidValue;
  CHECK(fwd(h(6), nullptr, 0) == PURO_ERR_LAUNCH);
  if (g_fail) return 1;
  std::printf("abi under sanitizers: ok\n");
  return 0;
}
