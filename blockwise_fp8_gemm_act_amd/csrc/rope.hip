// Rotary positions, and the RMS norms of query and key heads with the rotation
// in the same pass (gfx950).
//
//   n = x r w,  r = 1 / sqrt(mean(x^2) + eps);  (a', b') = (a c - b s, b c + a s)
//
// Everything here is bound by memory, or by its launch: 2 bytes in and 2 out per element
// (4 in, 2 out backward), a handful of operations each.  16384 tokens of 24 heads of 128:
// the norms with the rotation 41 us (5.0 TB/s, the rate of a large copy), their backward
// 56 us and 4 to sum the weights' gradients (5.0 TB/s); the rotation alone of 16381 tokens
// of 16 heads 27 us (5.1 TB/s); one token 2.6 us, 32 tokens into a cache 4.5 us.
//
// A team of head_dim / 8 lanes holds one head, 16 bytes a lane, so that a wave reads 4 (or
// 8) whole heads of one token per load and the norm's sum is three or four DPP adds.  The
// pairs of the half layout lie rot/2 elements apart: the partner's raw 16 bytes come from
// the lane rot/16 away by a lane permute, not by a second read.  A token's cosines and
// sines are loaded once per wave and used for all its heads.
#include "attention_plan.h"
#include "device_common.h"
#include "launch_attention.h"

namespace puro {
namespace {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kWaves = kRopeWaves;

__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){a, b}, v2bf));
}

__device__ __forceinline__ u32x4 load16(const uint16_t *p) { return *reinterpret_cast<const u32x4 *>(p); }

__device__ __forceinline__ void unpack8(u32x4 w, float *f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16lo(w[j]);
    f[2 * j + 1] = bf16hi(w[j]);
  }
}

__device__ __forceinline__ u32x4 pack8(const float *f) {
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = pack2_bf16(f[2 * j], f[2 * j + 1]);
  return w;
}

template <int kCtrl>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, true));
}

// Sum over a team of 8 or 16 consecutive lanes, in every lane of the team.
template <int kLanes>
__device__ __forceinline__ float team_sum(float v) {
  v = dpp_add<0xB1>(v);                     // quad_perm 1,0,3,2
  v = dpp_add<0x4E>(v);                     // quad_perm 2,3,0,1
  v = dpp_add<0x141>(v);                    // row_half_mirror
  if (kLanes == 16) v = dpp_add<0x140>(v);  // row_mirror
  return v;
}

// The rotation of one token as one lane needs it: the lane holds elements 8 c ..
// 8 c + 7 of a head.  Half layout: cs[i], sn[i] belong to element i, and its
// partner is element i of lane `mate`.  Interleaved: cs[j], sn[j], j < 4, belong
// to the pair (2j, 2j + 1).
template <bool kInter>
struct Turn {
  float cs[kInter ? 4 : 8], sn[kInter ? 4 : 8];
  bool on;     // these elements rotate
  int mate;

  __device__ __forceinline__ void load(const float *table, int64_t positions, int rot, const int32_t *pos, int64_t t,
                                       int c, int lane, float sign) {
    on = c < rot / 8;
    const int64_t p = pos ? (int64_t)pos[t] : t;
    const bool known = p >= 0 && p < positions;
    constexpr int kN = kInter ? 4 : 8;
    const int span = rot / 16;
    const bool low = c < span;
    mate = kInter || !on ? lane : (low ? lane + span : lane - span);
    const int first = kInter ? 4 * c : 8 * (low ? c : c - span);
    if (on && known) {
      const float *row = table + p * rot + first;
#pragma unroll
      for (int j = 0; j < kN; j += 4) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(row + j);
        const f32x4 b = *reinterpret_cast<const f32x4 *>(row + rot / 2 + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cs[j + i] = a[i];
          sn[j + i] = b[i] * sign * (kInter ? 1.0f : (low ? -1.0f : 1.0f));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) cs[j] = sn[j] = __builtin_nanf("");   // a position outside the table
    }
  }

  __device__ __forceinline__ u32x4 partner(u32x4 w) const {
    if (kInter) return w;
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = (uint32_t)__shfl((int)w[j], mate);
    return o;
  }

  // v: the lane's elements, m: its partners' (half layout only).
  __device__ __forceinline__ void apply(float *v, const float *m) const {
    if (kInter) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = v[2 * j] * cs[j] - v[2 * j + 1] * sn[j];
        const float b = v[2 * j + 1] * cs[j] + v[2 * j] * sn[j];
        v[2 * j] = on ? a : v[2 * j];
        v[2 * j + 1] = on ? b : v[2 * j + 1];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = on ? v[i] * cs[i] + m[i] * sn[i] : v[i];
    }
  }
};

// ---------------------------------------------------------------- forward
// Tokens from `first` on.  `parts` waves share a token: each takes every parts-th group
// of heads.  kBatch heads a lane are in flight at once.
template <int kHd, bool kInter, bool kNorm, bool kAppend>
__global__ void __launch_bounds__(64 * kWaves) rope_kernel(RopeArgs a, int parts, int64_t first) {
  constexpr int kTeam = kHd / 8, kTeams = 64 / kTeam, kBatch = 3;
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t in = w / parts, t = first + in;
  const int part = (int)(w - in * parts);
  if (t >= a.tokens) return;
  const int c = lane % kTeam, team = lane / kTeam;
  const int normed = a.heads_q + a.heads_k, heads = normed + a.heads_v;
  const int step = parts * kTeams;

  Turn<kInter> turn;
  turn.load(a.table, a.positions, a.rot, a.pos, t, c, lane, a.sign);
  u32x4 wq, wk, wqm, wkm;
  if (kNorm) {
    wq = load16(a.wq + 8 * c);
    wk = load16(a.wk + 8 * c);
    wqm = turn.partner(wq);
    wkm = turn.partner(wk);
  }
  int64_t row = t;
  bool keep = true;
  if (kAppend) {
    row = a.rows[t];
    keep = row >= 0 && row < a.cache_rows;
  }
  const uint16_t *xr = a.x + t * a.xs + 8 * c;

  for (int h0 = part * kTeams + team; h0 - team < heads; h0 += kBatch * step) {
    u32x4 raw[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + u * step;
      raw[u] = h < heads ? load16(xr + (int64_t)h * kHd) : (u32x4){0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + u * step;
      float v[8], m[8];
      unpack8(raw[u], v);
      unpack8(turn.partner(raw[u]), m);
      if (kNorm) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(v[i], v[i], ss);
        ss = team_sum<kTeam>(ss);
        const float r = 1.0f / __builtin_sqrtf(ss * (1.0f / kHd) + a.eps);
        const bool isq = h < a.heads_q;
        float wv[8], wm[8];
        unpack8(isq ? wq : wk, wv);
        unpack8(isq ? wqm : wkm, wm);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = v[i] * r * wv[i];
          m[i] = m[i] * r * wm[i];
        }
      }
      turn.apply(v, m);
      const u32x4 y = pack8(v);
      if (h < a.heads_q) {
        *reinterpret_cast<u32x4 *>(a.q + t * a.qs + (int64_t)h * kHd + 8 * c) = y;
      } else if (h < normed) {
        if (!kAppend || keep) *reinterpret_cast<u32x4 *>(a.k + row * a.ks + (int64_t)(h - a.heads_q) * kHd + 8 * c) = y;
      } else if (kAppend && h < heads && keep) {
        *reinterpret_cast<u32x4 *>(a.v + row * a.vs + (int64_t)(h - normed) * kHd + 8 * c) = raw[u];
      }
    }
  }
}

template <int kHd, bool kInter>
hipError_t launch_rope(const RopeArgs &a, hipStream_t stream) {
  const RopePlan plan = plan_rope(a.tokens, a.heads_q + a.heads_k + a.heads_v, kHd);
  const dim3 block(64 * kWaves);
  for (int64_t first = 0; first < a.tokens; first += plan.tokens) {
    const int64_t left = a.tokens - first, n = left < plan.tokens ? left : plan.tokens;
    const dim3 grid((unsigned)rope_blocks(plan, n));
    if (a.rows)
      rope_kernel<kHd, kInter, true, true><<<grid, block, 0, stream>>>(a, plan.parts, first);
    else if (a.wq)
      rope_kernel<kHd, kInter, true, false><<<grid, block, 0, stream>>>(a, plan.parts, first);
    else
      rope_kernel<kHd, kInter, false, false><<<grid, block, 0, stream>>>(a, plan.parts, first);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

// ---------------------------------------------------------------- backward
// One wave a token at a time, workgroups striding over the tokens, so that the
// weight gradients stay in registers: 8 columns a lane for q and for k, joined
// over the workgroup's teams in LDS and over the workgroups by a second kernel,
// both in a fixed order.
template <int kHd, bool kInter>
__global__ void __launch_bounds__(64 * kWaves) rope_back_kernel(RopeBackArgs a) {
  constexpr int kTeam = kHd / 8, kTeams = 64 / kTeam, kBatch = 3;
  __shared__ float sums[kWaves * kTeams][2][kHd];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane % kTeam, team = lane / kTeam;
  const int heads = a.heads_q + a.heads_k;
  const u32x4 wq = load16(a.wq + 8 * c), wk = load16(a.wk + 8 * c);
  float aq[8], ak[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) aq[i] = ak[i] = 0.0f;

  for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < a.tokens; t += (int64_t)gridDim.x * kWaves) {
    Turn<kInter> turn;
    turn.load(a.table, a.positions, a.rot, a.pos, t, c, lane, -1.0f);
    const uint16_t *xr = a.x + t * a.xs + 8 * c;
    for (int h0 = team; h0 - team < heads; h0 += kBatch * kTeams) {
      u32x4 rx[kBatch], rg[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int h = h0 + u * kTeams;
        rx[u] = rg[u] = (u32x4){0, 0, 0, 0};
        if (h < heads) {
          rx[u] = load16(xr + (int64_t)h * kHd);
          rg[u] = h < a.heads_q ? load16(a.dq + t * a.dqs + (int64_t)h * kHd + 8 * c)
                                : load16(a.dk + t * a.dks + (int64_t)(h - a.heads_q) * kHd + 8 * c);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int h = h0 + u * kTeams;
        const bool isq = h < a.heads_q;
        float x[8], g[8], m[8], wv[8];
        unpack8(rx[u], x);
        unpack8(rg[u], g);
        unpack8(turn.partner(rg[u]), m);
        unpack8(isq ? wq : wk, wv);
        turn.apply(g, m);
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = __builtin_fmaf(x[i], x[i], ss);
          dot = __builtin_fmaf(g[i] * wv[i], x[i], dot);
        }
        ss = team_sum<kTeam>(ss);
        dot = team_sum<kTeam>(dot);
        const float r = 1.0f / __builtin_sqrtf(ss * (1.0f / kHd) + a.eps);
        const float mean = dot * r * (1.0f / kHd);
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = x[i] * r;
          const float gh = g[i] * xh;
          d[i] = r * (wv[i] * g[i] - xh * mean);
          if (h < heads) {                       // a NaN of the rotation stays out of the sums where there is no head
            aq[i] += isq ? gh : 0.0f;
            ak[i] += isq ? 0.0f : gh;
          }
        }
        if (h < heads) *reinterpret_cast<u32x4 *>(a.dx + t * a.dxs + (int64_t)h * kHd + 8 * c) = pack8(d);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sums[wave * kTeams + team][0][8 * c + i] = aq[i];
    sums[wave * kTeams + team][1][8 * c + i] = ak[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * kHd; i += 64 * kWaves) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < kWaves * kTeams; ++j) s += sums[j][i / kHd][i % kHd];
    a.partial[(int64_t)blockIdx.x * 2 * kHd + i] = s;
  }
}

// Column sums of the workgroups' partials: 16 columns a workgroup, 64 interleaved runs
// of at most 16 rows, all of a run's loads in flight, the runs joined in LDS in order.
// (With 16 runs in loops it took 20 us, a quarter of the whole backward call at 16384
// tokens.)
constexpr int kMostBlocks = 1024, kRuns = 64;
__global__ void __launch_bounds__(16 * kRuns) rope_back_sum_kernel(const float *partial, int blocks, int hd, float *dwq,
                                                                    float *dwk) {
  __shared__ float part[kRuns][16];
  const int c = threadIdx.x & 15, col = blockIdx.x * 16 + c, run = threadIdx.x >> 4;
  float v[kMostBlocks / kRuns], s = 0.0f;
#pragma unroll
  for (int j = 0; j < kMostBlocks / kRuns; ++j) {
    const int b = run + kRuns * j;
    v[j] = b < blocks ? partial[(int64_t)b * 2 * hd + col] : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < kMostBlocks / kRuns; ++j) s += v[j];
  part[run][c] = s;
  __syncthreads();
  if (run < 4) {
    float sum = 0.0f;
    for (int j = 0; j < kRuns / 4; ++j) sum += part[run * (kRuns / 4) + j][c];
    part[run * (kRuns / 4)][c] = sum;      // read by this thread alone so far
  }
  __syncthreads();
  if (run == 0) {
    float sum = 0.0f;
    for (int j = 0; j < 4; ++j) sum += part[j * (kRuns / 4)][c];
    (col < hd ? dwq : dwk)[col < hd ? col : col - hd] = sum;
  }
}

// ---------------------------------------------------------------- the table
__global__ void __launch_bounds__(256) rope_table_kernel(int64_t positions, int rot, double base, int scaling,
                                                          double factor, double trained, float *table) {
  const int half = rot / 2;
  const int64_t n = positions * half;
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t p = e / half;
    const int i = (int)(e - p * half);
    double b = base, m = 1.0;
    if (scaling == PURO_ROPE_NTK) b *= pow(factor, (double)rot / (rot - 2));
    double f = pow(b, -2.0 * i / rot);
    if (scaling == PURO_ROPE_LINEAR) f /= factor;
    if (scaling == PURO_ROPE_YARN) {
      const double turns = trained * f / 6.283185307179586476925286766559;
      const double g = fmin(fmax((turns - 1.0) / 31.0, 0.0), 1.0);
      f *= (1.0 - g) / factor + g;
      m = 0.1 * log(factor) + 1.0;
    }
    double sn, cs;
    sincos((double)p * f, &sn, &cs);
    table[p * rot + i] = (float)(m * cs);
    table[p * rot + half + i] = (float)(m * sn);
  }
}

}  // namespace

hipError_t run_rope_table(int64_t positions, int64_t rot, double base, int scaling, double factor, int64_t trained,
                          float *table, hipStream_t stream) {
  const int64_t blocks = (positions * (rot / 2) + 255) / 256;
  rope_table_kernel<<<dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, stream>>>(
      positions, (int)rot, base, scaling, factor, (double)trained, table);
  return hipGetLastError();
}

hipError_t run_rope(const RopeArgs &a, int head_dim, bool interleaved, hipStream_t stream) {
  if (head_dim == 128) return interleaved ? launch_rope<128, true>(a, stream) : launch_rope<128, false>(a, stream);
  return interleaved ? launch_rope<64, true>(a, stream) : launch_rope<64, false>(a, stream);
}

int rope_back_blocks(int64_t tokens) {
  const int64_t b = (tokens + kWaves - 1) / kWaves;
  return (int)(b < kMostBlocks ? b : kMostBlocks);
}

hipError_t run_rope_back(const RopeBackArgs &a, int head_dim, bool interleaved, hipStream_t stream) {
  const int blocks = rope_back_blocks(a.tokens);
  if (blocks > 0) {
    const dim3 grid((unsigned)blocks), block(64 * kWaves);
    if (head_dim == 128) {
      if (interleaved) rope_back_kernel<128, true><<<grid, block, 0, stream>>>(a);
      else rope_back_kernel<128, false><<<grid, block, 0, stream>>>(a);
    } else {
      if (interleaved) rope_back_kernel<64, true><<<grid, block, 0, stream>>>(a);
      else rope_back_kernel<64, false><<<grid, block, 0, stream>>>(a);
    }
    if (hipError_t e = hipGetLastError()) return e;
  }
  rope_back_sum_kernel<<<dim3((unsigned)(2 * head_dim / 16)), dim3(16 * kRuns), 0, stream>>>(a.partial, blocks, head_dim,
                                                                                       a.dwq, a.dwk);
  return hipGetLastError();
}

}  // namespace puro
