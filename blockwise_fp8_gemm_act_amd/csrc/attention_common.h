// Device pieces shared by the attention kernels (gfx950): sequence lookup, the
// mask, LDS tiles and their two reads, the bf16 matrix product.
//
// Every kernel works on transposed score tiles: a 32x32x16 MFMA with 32 keys as
// rows and 32 queries as columns leaves lane l with query l & 31 and 16 of the 32
// keys, register i holding key 8 (i/4) + 4 (l/32) + i%4.  A softmax row is then
// one lane and its partner 32 lanes away, statistics are scalars of the lane, and
// the probabilities are, in place, the B operand of the next product: registers
// 8s .. 8s+7 are the 8 keys a lane feeds to contraction step s, in the order {0-3,
// 8-11} for lanes below 32 and {4-7, 12-15} above, which the A operand's read
// follows.
#pragma once

#include "attention_plan.h"
#include "device_common.h"
#include "launch_attention.h"

namespace puro {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Running maximum of a row that has seen nothing: finite, so that differences of
// maxima never are inf - inf; every score of the contract is far above it.
constexpr float kNoMax = -1e30f;

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ bf16x8 load8(const uint16_t *p) { return *reinterpret_cast<const bf16x8 *>(p); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// Fragments that stay in registers through a loop: waits for their loads here, so that
// the compiler does not wait for them inside the loop, where its wait would also be one
// for the copies under way.
template <int n>
__device__ __forceinline__ void arrived(bf16x8 (&f)[n]) {
#pragma unroll
  for (int i = 0; i < n; ++i) asm volatile("" : "+v"(f[i]));
}

// The other half wave's value: lanes 0-31 and 32-63 exchange.
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// ---------------------------------------------------------------- sequences
struct Seq {
  int q0, ql, k0, kl;    // first rows and lengths
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Tiles of `unit` rows are numbered over all sequences without a prefix sum: sequence
// s owns the numbers from start(s) * mul / unit + s up to that of s + 1, `start` being
// q_start or k_start.  These are never fewer than its tiles; the surplus ones are empty.
// Returns the sequence (and its number) of tile `slot` and subtracts its first number.
//
// Starts and lengths come from device memory: clamped, so that no row outside the
// tensors is ever addressed.  63 sequences at a time, one a lane and the next one's
// start in the lane beside, so that everything is there after one latency.
__device__ __forceinline__ Seq find_seq(const AttnArgs &a, const int32_t *start, int mul, int unit, int &slot, int &s) {
  s = 0;
  if (!start) return Seq{0, a.q_tokens, 0, a.k_len ? clampi(a.k_len[0], 0, a.k_tokens) : a.k_tokens};
  const int lane = threadIdx.x & 63;
  const bool over_q = start == a.q_start;
  int first = 0, q0 = 0, q1 = 0, k0 = 0, k1 = 0, kl = 0;
  for (int b = 0; b < a.sequences; b += 63) {
    const int i = b + lane, in = i < a.sequences ? i : a.sequences;
    const int qs = clampi(a.q_start[in], 0, a.q_tokens), ks = clampi(a.k_start[in], 0, a.k_tokens);
    const int len = a.k_len ? a.k_len[in < a.sequences ? in : a.sequences - 1] : a.k_tokens;
    const int base = i < a.sequences && lane < 63 ? (int)((int64_t)(over_q ? qs : ks) * mul / unit) + i : 0x7fffffff;
    const uint64_t le = __ballot(base <= slot);
    if (!le) break;
    const int n = 63 - __builtin_clzll(le);
    s = b + n;
    first = __builtin_amdgcn_readlane(base, n);
    q0 = __builtin_amdgcn_readlane(qs, n);
    q1 = __builtin_amdgcn_readlane(qs, n + 1);
    k0 = __builtin_amdgcn_readlane(ks, n);
    k1 = __builtin_amdgcn_readlane(ks, n + 1);
    kl = __builtin_amdgcn_readlane(len, n);
  }
  slot -= first;
  const int most = k1 > k0 ? k1 - k0 : 0;
  return Seq{q0, q1 > q0 ? q1 - q0 : 0, k0, clampi(kl, 0, most)};
}

// ---------------------------------------------------------------- mask
// The key tiles that a block of queries at positions p_lo .. p_hi looks at, `unit`
// keys each: those of the visible first keys, then those of the window.  Keys that
// none of these queries sees are read from row `lo` or `hi` instead (they are
// masked), so that what such rows hold never matters.
struct KeyTiles {
  int first_n, main0, count;    // tiles of the first keys; first tile of the window; all
  int lo, hi, sinks;
  __device__ __forceinline__ int key0(int i, int unit) const { return (i < first_n ? i : main0 + i - first_n) * unit; }
};

__device__ __forceinline__ KeyTiles key_tiles(int p_lo, int p_hi, int window, int sinks, int unit) {
  KeyTiles t;
  t.hi = p_hi;
  t.lo = window > 0 && p_lo >= window ? p_lo - window + 1 : 0;
  t.sinks = sinks < t.lo ? sinks : t.lo;
  t.main0 = t.lo / unit;
  t.first_n = (t.sinks + unit - 1) / unit;
  if (t.first_n > t.main0) t.first_n = t.main0;
  t.count = p_hi < 0 ? 0 : t.first_n + p_hi / unit - t.main0 + 1;
  return t;
}

// ---------------------------------------------------------------- LDS tiles
// A tile holds rows of kHd bf16 in groups of 1 KB (4 rows of 128 columns, or 8 of
// 64), each one copy of a wave, 16 bytes between groups.  Inside a group 4 rows by 64
// bytes are contiguous: chunk c (16 bytes) of row r of 4 lies at 256 (c/4) + 64 r + 16
// (c%4); with 64 columns the second 4 rows follow at 512.  Then
//   - a row fragment's phase (16 rows, one chunk) and a transposed fragment's (4 rows
//     by 64 bytes, contiguous) spread over the 64 banks: the hardware counts no
//     conflicts;
//   - every address is one lane-dependent base plus a constant, so that the reads
//     cost no address arithmetic (an xor swizzle took 24 registers or as many
//     instructions a tile).
template <int kHd>
constexpr int kGroupRows = 512 / kHd;
constexpr int kGroupBytes = 1024 + 16;
template <int kHd>
constexpr int kTileBytes(int rows) { return rows / kGroupRows<kHd> * kGroupBytes; }

// Global -> LDS copy of 16 bytes a lane to lds + 16 lane, from a uniform base and a
// 32-bit offset of the lane.  Asm, so that the compiler does not make every later LDS read
// wait for it: completion is awaited explicitly.  Without a memory clobber, so that reads
// of other tiles may be scheduled around it: what it writes is read only after a barrier
// that has one, and what it overwrites was read before one.
__device__ __forceinline__ void dma16_s(const void *base, uint32_t off, uint32_t lds) {
  uint32_t save;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(save)
      : "v"(off), "s"(base), "s"(lds));
}

__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

// The row of a group and the 16-byte chunk of it that this lane copies.
template <int kHd>
__device__ __forceinline__ void copy_place(int &r, int &c) {
  const int lane = threadIdx.x & 63;
  if (kHd == 128) {
    r = (lane >> 2) & 3;
    c = 4 * (lane >> 4) + (lane & 3);
  } else {
    r = ((lane >> 2) & 3) + 4 * (lane >> 5);
    c = 4 * ((lane >> 4) & 1) + (lane & 3);
  }
}

// Copies of key (or value) tiles of `unit` keys, group by group and without branches:
// the base is uniform, a lane's offset inside the tile clamps the rows that no query of
// the block sees (token strides are below 2^23 elements, so 64 rows fit 32 bits).
template <int kHd>
struct TileCopy {
  const uint16_t *base;
  int64_t stride;
  int row;               // this lane's row and chunk of a group
  uint32_t chunk;
  __device__ __forceinline__ TileCopy(const uint16_t *base, int64_t stride) : base(base), stride(stride) {
    int c;
    copy_place<kHd>(row, c);
    chunk = (uint32_t)(c * 16);
  }
  __device__ __forceinline__ void operator()(const KeyTiles &kt, int i, int unit, int g, uint32_t tile) const {
    const int key0 = kt.key0(i, unit);
    const bool first = i < kt.first_n;
    const int key = key0 + g * kGroupRows<kHd> + row;
    const int in = key < kt.sinks ? key : clampi(key, first ? 0 : kt.lo, first ? kt.sinks - 1 : kt.hi);
    dma16_s(base + (int64_t)key0 * stride, __umul24(in - key0, (uint32_t)(stride * 2)) + chunk,
            tile + (uint32_t)(g * kGroupBytes));
  }
};

// The same for a loop whose products must not wait for addresses: the next tile's are
// worked out ahead of its turn, the base beside the products (scalars only) and a lane's
// offsets where there is time; copy() then is one instruction and its LDS address.  Only
// tiles with rows that no query of the block sees need offsets of their own: those of the
// first keys, the first of the window and the last.  A wave copies kParts groups of a tile.
template <int kHd, int kUnit, int kWaves>
struct TileStream {
  static constexpr int kParts = kUnit / kGroupRows<kHd> / kWaves;
  const uint16_t *base, *at;
  uint32_t bytes;        // of a row's stride
  int row, wave;
  uint32_t chunk, off[kParts];
  __device__ __forceinline__ TileStream(const uint16_t *base, int64_t stride, int wave)
      : base(base), bytes((uint32_t)(stride * 2)), wave(wave) {
    int c;
    copy_place<kHd>(row, c);
    chunk = (uint32_t)(c * 16);
    row += wave * kGroupRows<kHd>;
  }
  // Past the last tile: that one again.
  static __device__ __forceinline__ int upto(const KeyTiles &kt, int i) { return i < kt.count ? i : kt.count - 1; }
  __device__ __forceinline__ void aim(const KeyTiles &kt, int i) {
    at = reinterpret_cast<const uint16_t *>(reinterpret_cast<const char *>(base) +
                                            (uint64_t)(uint32_t)kt.key0(upto(kt, i), kUnit) * bytes);
  }
  __device__ __forceinline__ void aim_rows(const KeyTiles &kt, int i) {
    i = upto(kt, i);
#pragma unroll
    for (int part = 0; part < kParts; ++part) off[part] = __umul24(row + part * kWaves * kGroupRows<kHd>, bytes) + chunk;
    if (i <= kt.first_n || i == kt.count - 1) {
      const int key0 = kt.key0(i, kUnit);
      const bool first = i < kt.first_n;
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        const int key = key0 + row + part * kWaves * kGroupRows<kHd>;
        const int in = key < kt.sinks ? key : clampi(key, first ? 0 : kt.lo, first ? kt.sinks - 1 : kt.hi);
        off[part] = __umul24(in - key0, bytes) + chunk;     // 64 rows, below 2^24 bytes each
        asm volatile("" : "+v"(off[part]));      // a branch, not a choice of values
      }
    }
  }
  __device__ __forceinline__ void copy(int part, uint32_t tile) const {
    dma16_s(at, off[part], tile + (uint32_t)((part * kWaves + wave) * kGroupBytes));
  }
};

typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

// Rows r0 .. r0+31 (r0 a multiple of 32), contraction step kk (16 columns): lane l
// gets row r0 + (l & 31), columns 16 kk + 8 (l / 32) .. +7.
template <int kHd>
__device__ __forceinline__ bf16x8 row_frag(uint32_t tile, int r0, int kk) {
  const int lane = threadIdx.x & 63;
  const int r = lane & 31;
  uint32_t base = (uint32_t)(r / kGroupRows<kHd> * kGroupBytes + (r & 3) * 64 + (lane >> 5) * 16);
  if (kHd == 64) base += (uint32_t)(((r >> 2) & 1) * 512);
  return *(lds_bf16x8 *)(uintptr_t)(tile + base + (uint32_t)((kk >> 1) * 256 + (kk & 1) * 32 + kTileBytes<kHd>(r0)));
}

// The transpose's fragment: lane l gets column 32 db + (l & 31) of the 8 rows r0 +
// 4 (l / 32) + {0-3, 8-11}; r0 a multiple of 16.  Each 16 lanes read 4 rows by 16
// columns, 8 bytes a lane, and get them transposed.
template <int kHd>
__device__ __forceinline__ bf16x8 col_frag(uint32_t tile, int r0, int db) {
  const int lane = threadIdx.x & 63;
  const int half = lane >> 5, i = lane & 15;
  const uint32_t base = (uint32_t)((i >> 2) * 64 + (i & 3) * 8 + (lane & 16) * 2 + half * (kHd == 128 ? kGroupBytes : 512));
  bf16x4 v[2];
#pragma unroll
  for (int w = 0; w < 2; ++w)
    v[w] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
        (lds_bf16x4 *)(uintptr_t)(tile + base + (uint32_t)(db * 256 + kTileBytes<kHd>(r0 + 8 * w))));
  return __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
}

// Order of a block of products: the LDS reads of the first `ahead` products go out
// first, then each product is followed by the reads of one further on (one a product
// of row fragments, two of column fragments; `rows` products of the first kind come
// first).  kTimes: products of each fragment.  Left alone, the compiler reads, waits and
// multiplies one by one.
template <int kAhead, int kRowProducts, int kColProducts, int kTimes = 1>
__device__ __forceinline__ void feed() {
  constexpr int n = kRowProducts + kColProducts;
#pragma unroll
  for (int j = 0; j < n + kAhead; ++j) {
    if (j >= kAhead) __builtin_amdgcn_sched_group_barrier(0x008, kTimes, 0);
    if (j < n) {
      if (j < kRowProducts) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      else __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
  }
}

// Registers 8s .. 8s+7 of a score tile as the B operand of step s.
__device__ __forceinline__ bf16x8 pack_step(const f32x16 &p, int s) {
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = pack_bf16(p[8 * s + 2 * j], p[8 * s + 2 * j + 1]);
  return __builtin_bit_cast(bf16x8, w);
}

// And what their rounding left out, in the same place.
__device__ __forceinline__ bf16x8 pack_rest(const f32x16 &p, int s, bf16x8 rounded) {
  const u32x4 r = __builtin_bit_cast(u32x4, rounded);
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = pack_bf16(p[8 * s + 2 * j] - __uint_as_float(r[j] << 16), p[8 * s + 2 * j + 1] - __uint_as_float(r[j] & 0xffff0000u));
  return __builtin_bit_cast(bf16x8, w);
}

// Masks the scores of keys key0 .. key0+31 for the lane's query at p.
__device__ __forceinline__ void mask_tile(f32x16 &s, int key0, int p, int window, int sinks) {
  const int half = (threadIdx.x & 63) >> 5;
  if (key0 < sinks) {                   // first keys that stay visible among them
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int key = key0 + 8 * (i / 4) + 4 * half + i % 4;
      s[i] = (key <= p) & ((window == 0) | (key > p - window) | (key < sinks)) ? s[i] : -__builtin_inff();
    }
    return;
  }
  // p - key is negative for keys after p: causality and the window are one unsigned
  // comparison.
  int before = p - key0 - 4 * half;
  asm volatile("" : "+v"(before));      // keeps the comparisons inside the caller's branch
  const uint32_t reach = window == 0 ? 0x7fffffffu : (uint32_t)window;
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = (uint32_t)(before - (8 * (i / 4) + i % 4)) < reach ? s[i] : -__builtin_inff();
}

// One block of 32 columns of a transposed accumulator (column of the result = lane
// & 31's row, register i = column 8 (i/4) + 4 (lane/32) + i%4) to a bf16 row: the
// half waves exchange so that each lane stores 16 bytes twice.
__device__ __forceinline__ void store_block(uint16_t *row, const f32x16 &x, float f) {
  const int half = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const auto r = __builtin_amdgcn_permlane32_swap(pack_bf16(x[8 * g + 2 * j] * f, x[8 * g + 2 * j + 1] * f),
                                                      pack_bf16(x[8 * g + 4 + 2 * j] * f, x[8 * g + 5 + 2 * j] * f),
                                                      false, false);
      w[j] = r[0];
      w[2 + j] = r[1];
    }
    *reinterpret_cast<u32x4 *>(row + 16 * g + 8 * half) = w;
  }
}

}  // namespace puro
