// What the kernels of the linear layer share, gfx950 (device code; included by linear_rows.h and
// linear_tiles.h):
//   z[m][n] = bias[n] + sum_b d[n][b] sum_{j<32} c[n][32b+j] x[m][32b+j],   y = act(z) mul + residual
//
// Codes meet the rows in the matrix cores, as numbers of the rows' type: a code of any of the formats
// is exact in bf16 and in fp16, and so are products of two such numbers in fp32.  fp32 rows go as three
// bf16 parts that add up to them.  A matrix product covers one block of 32 (or half of one, the other
// half added by the next), so the block's scale, which need not be exact in 16 bits, is applied to its
// sum by one fp32 FMA.  The only roundings are those of fp32 sums, and the last one to y's type.
#pragma once

#include "mma_ops.h"
#include "mxfp4.h"

namespace bqm {
namespace lin {

struct Args {
  const uint8_t* w;
  const uint8_t* x;
  const float* bias;       // or null
  const uint8_t* mul;      // or null
  const uint8_t* res;      // or null
  uint8_t* y;
  const int32_t* offsets;  // [E + 1] first rows of the groups, or null: all rows are one group's
  int64_t N, R, scales_off;
  int64_t xs, ms, rs, ys;  // row strides: x in bytes, the others in elements
  int nb, ks, kg, E, act, y_type;
};

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
using mma::bf16x8;
using mx::f32x4;
using mx::u32x4;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kOob = 0x80000000u;  // an offset past every descriptor: reads 0

__host__ __device__ constexpr int type_size(int type) { return type == BQM_F32 ? 4 : 2; }
constexpr int parts_of(int type) { return type == BQM_F32 ? 3 : 1; }

// The same value in every lane, as the compiler does not always see.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// (Where it does not see that a descriptor is the same in all lanes, the compiler loops over them at each load.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, int64_t bytes) {
  const int64_t most = 0x7FFFFFFF;
  return __builtin_amdgcn_make_buffer_rsrc((void*)uniform((int64_t)p), 0,
                                           __builtin_amdgcn_readfirstlane((int)(bytes < 0 ? 0 : bytes < most ? bytes : most)), 0x00020000);
}

// ---- codes as matrix operands ----
// 1024 + n is an fp16 number with n in its last bits: bytes are put under 0x64 and what is too much is
// taken off again, exactly.
__device__ __forceinline__ uint32_t f16_add(uint32_t v, float by) {
  const f16x2 r = __builtin_bit_cast(f16x2, v) + f16x2{(_Float16)by, (_Float16)by};
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint32_t f16_sixteenth(uint32_t v, float by) {
  const f16x2 r = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, v), f16x2{(_Float16)0.0625f, (_Float16)0.0625f},
                                            f16x2{(_Float16)by, (_Float16)by});
  return __builtin_bit_cast(uint32_t, r);
}
// Four codes of a word, one per byte (low nibbles to lo, high ones to hi), as pairs of 16-bit numbers.
// Q4_0 comes out in units of kUnit, MXFP4 beside bf16 times `by`, a power of two.
template <int FMT, int XT>
constexpr float kUnit = FMT == BQM_Q4_0 && XT != BQM_F16 ? 0.0625f : 1.0f;
template <int FMT, int XT>
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t (&lo)[2], uint32_t (&hi)[2], float by = 1.0f) {
  if constexpr (FMT == BQM_MXFP4) {  // the conversion takes the two nibbles of a byte
    const uint32_t w4 = w >> 4, l = (w & 0x000F000Fu) | (w4 & 0xFFF0FFF0u), h = (w4 & 0x000F000Fu) | ((w >> 8) & 0xFFF0FFF0u);
    if constexpr (XT == BQM_F16) {
      lo[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(l, 1.0f, 0));
      lo[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(l, 1.0f, 2));
      hi[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(h, 1.0f, 0));
      hi[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(h, 1.0f, 2));
    } else {
      lo[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(l, by, 0));
      lo[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(l, by, 2));
      hi[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(h, by, 0));
      hi[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(h, by, 2));
    }
  } else if constexpr (XT == BQM_F16) {
    const uint32_t b01 = __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u), b23 = __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u);
    lo[0] = f16_add(b01 & 0xFF0FFF0Fu, -1032.0f);
    lo[1] = f16_add(b23 & 0xFF0FFF0Fu, -1032.0f);
    hi[0] = f16_sixteenth(b01 & 0xFFF0FFF0u, -72.0f);
    hi[1] = f16_sixteenth(b23 & 0xFFF0FFF0u, -72.0f);
  } else {
    const uint32_t l = ((w << 4) ^ 0x80808080u) & 0xF0F0F0F0u, h = (w ^ 0x80808080u) & 0xF0F0F0F0u;
    lo[0] = mma::bf_pair(mma::sbyte(l, 0), mma::sbyte(l, 1));
    lo[1] = mma::bf_pair(mma::sbyte(l, 2), mma::sbyte(l, 3));
    hi[0] = mma::bf_pair(mma::sbyte(h, 0), mma::sbyte(h, 1));
    hi[1] = mma::bf_pair(mma::sbyte(h, 2), mma::sbyte(h, 3));
  }
}
// Four Q8_0 codes of a word.
template <int XT>
__device__ __forceinline__ void bytes(uint32_t w, uint32_t (&v)[2]) {
  if constexpr (XT == BQM_F16) {
    const uint32_t u = w ^ 0x80808080u;
    v[0] = f16_add(__builtin_amdgcn_perm(0x64646464u, u, 0x04010400u), -1152.0f);
    v[1] = f16_add(__builtin_amdgcn_perm(0x64646464u, u, 0x04030402u), -1152.0f);
  } else {
    v[0] = mma::bf_pair(mma::sbyte(w, 0), mma::sbyte(w, 1));
    v[1] = mma::bf_pair(mma::sbyte(w, 2), mma::sbyte(w, 3));
  }
}

// A block's scale from the bits that were loaded for it, in units of the codes.
template <int FMT, int XT>
__device__ __forceinline__ float scale_from(uint32_t bits) {
  if constexpr (FMT == BQM_MXFP4) return mx::scale_of(bits);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)bits) * kUnit<FMT, XT>;
}

// ---- rows as matrix operands ----
// V numbers (a multiple of two) as bf16 parts, V / 2 words of each: a part is the upper half of what the parts
// before it leave.  Nothing is left of an infinity; what is left of a NaN is one, whose upper half stays one.
template <int V>
__device__ __forceinline__ void three_parts(const float (&x)[V], uint32_t (&part)[3][V / 2]) {
#pragma unroll
  for (int j = 0; j < V; j += 2) {
    uint32_t u[3][2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const float f = x[j + k];
      u[0][k] = __float_as_uint(f);
      const float g = __builtin_isinf(f) ? 0.0f : f - __uint_as_float(u[0][k] & 0xFFFF0000u);
      u[1][k] = __float_as_uint(g);
      u[2][k] = __float_as_uint(g - __uint_as_float(u[1][k] & 0xFFFF0000u));
    }
#pragma unroll
    for (int p = 0; p < 3; p++) part[p][j / 2] = __builtin_amdgcn_perm(u[p][1], u[p][0], 0x07060302u);
  }
}

// ---- what follows the sum ----
__device__ __forceinline__ float load_as(const uint8_t* p, int64_t at, int type) {
  if (type == BQM_F32) return reinterpret_cast<const float*>(p)[at];
  const uint32_t h = reinterpret_cast<const uint16_t*>(p)[at];
  return type == BQM_BF16 ? __uint_as_float(h << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}
__device__ __forceinline__ uint16_t bits16(float v, int type) {
  if (type == BQM_BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
  return __builtin_bit_cast(uint16_t, (_Float16)v);
}
__device__ __forceinline__ void store_as(uint8_t* p, int64_t at, float v, int type) {
  if (type == BQM_F32)
    reinterpret_cast<float*>(p)[at] = v;
  else
    reinterpret_cast<uint16_t*>(p)[at] = bits16(v, type);
}

// z / (1 + 2^u).  The exponential and the reciprocal are the hardware's, each off by a step of fp32 at most, and
// u's rounding counts |u| 2^-24 of the exponential: no more than a step of z where that counts.  (With expf and a
// correctly rounded division the 512-token product of 17408 x 5120 takes 12 us longer.)  The reciprocal is 0 where
// it would be below 2^-126: a far z has the exponential taken 64 powers of two lower, beside which 1 counts nothing.
__device__ __forceinline__ float over_one_plus_exp2(float z, float u, bool far) {
  if (far) return ldexpf(z * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(u - 64.0f)), -64);
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u));
}
// silu, or gelu's tanh form.  FAR: some z may be below -87 or -9.9, from where u is 125.5 or 122.7 and more.
constexpr float kFarSilu = -87.0f, kFarTanh = -9.9f;
template <bool FAR, int V>
__device__ __forceinline__ void sigmoid_times(float (&z)[V], int act) {
  if (act == BQM_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < V; j++) z[j] = over_one_plus_exp2(z[j], z[j] * -1.44269504f, FAR && z[j] < kFarSilu);
  } else {
#pragma unroll
    for (int j = 0; j < V; j++)
      z[j] = over_one_plus_exp2(z[j], -2.30220819f * (z[j] + 0.044715f * z[j] * z[j] * z[j]), FAR && z[j] < kFarTanh);
  }
}
// The two gelus are written with the tail of their distribution, which keeps its digits far below 0.
template <int V>
__device__ __forceinline__ void activate(float (&z)[V], int act) {
  if (act == BQM_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < V; j++) z[j] = z[j] < 0.0f ? 0.0f : z[j];  // a NaN stays
  } else if (act == BQM_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < V; j++) z[j] = 0.5f * z[j] * erfcf(z[j] * -0.70710678f);
  } else if (act != BQM_ACT_NONE) {
    float low = z[0];
#pragma unroll
    for (int j = 1; j < V; j++) low = fminf(low, z[j]);
    if (__builtin_expect(low < (act == BQM_ACT_SILU ? kFarSilu : kFarTanh), 0))
      sigmoid_times<true>(z, act);
    else
      sigmoid_times<false>(z, act);
  }
}
// y of row m (of all rows) and column n, whose group's bias starts at `bias`.
__device__ __forceinline__ float finish(const Args& a, const float* bias, int64_t m, int64_t n, float sum) {
  float z[1] = {bias ? sum + bias[n] : sum};
  activate(z, a.act);
  if (a.mul) z[0] *= load_as(a.mul, m * a.ms + n, a.y_type);
  if (a.res) z[0] += load_as(a.res, m * a.rs + n, a.y_type);
  return z[0];
}
// Four columns from n on in each of R rows (m, m + step, ...; those from `end` on are left out), loaded and
// stored whole where n + 4 <= N and the strides are multiples of four.
template <int R>
__device__ __forceinline__ void finish4(const Args& a, const f32x4& bias, int64_t m, int step, int64_t end, int64_t n, const f32x4 (&sum)[R]) {
  float z[R * 4];
#pragma unroll
  for (int r = 0; r < R; r++)
#pragma unroll
    for (int j = 0; j < 4; j++) z[r * 4 + j] = sum[r][j] + bias[j];
  const int size = a.y_type == BQM_F32 ? 4 : 2;
  auto loaded = [&](const uint8_t* p, int64_t stride, auto&& use) {
    if (size == 4) {
      f32x4 u[R];
#pragma unroll
      for (int r = 0; r < R; r++)
        if (m + r * step < end) u[r] = *reinterpret_cast<const f32x4*>(p + ((m + r * step) * stride + n) * 4);
#pragma unroll
      for (int r = 0; r < R; r++)
#pragma unroll
        for (int j = 0; j < 4; j++) use(z[r * 4 + j], u[r][j]);
      return;
    }
    u32x2 u[R];
#pragma unroll
    for (int r = 0; r < R; r++)
      if (m + r * step < end) u[r] = *reinterpret_cast<const u32x2*>(p + ((m + r * step) * stride + n) * 2);
    if (a.y_type == BQM_BF16) {
#pragma unroll
      for (int r = 0; r < R; r++)
#pragma unroll
        for (int j = 0; j < 4; j++) use(z[r * 4 + j], __uint_as_float(j & 1 ? u[r][j >> 1] & 0xFFFF0000u : u[r][j >> 1] << 16));
    } else {
#pragma unroll
      for (int r = 0; r < R; r++)
#pragma unroll
        for (int j = 0; j < 4; j++) use(z[r * 4 + j], (float)__builtin_bit_cast(_Float16, (uint16_t)(u[r][j >> 1] >> (16 * (j & 1)))));
    }
  };
  activate(z, a.act);
  if (a.mul) loaded(a.mul, a.ms, [](float& v, float u) { v *= u; });
  if (a.res) loaded(a.res, a.rs, [](float& v, float u) { v += u; });
  if (size == 4) {
#pragma unroll
    for (int r = 0; r < R; r++)
      if (m + r * step < end)
        *reinterpret_cast<f32x4*>(a.y + ((m + r * step) * a.ys + n) * 4) = f32x4{z[r * 4], z[r * 4 + 1], z[r * 4 + 2], z[r * 4 + 3]};
    return;
  }
  u32x2 u[R];
  if (a.y_type == BQM_BF16) {
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
      for (int j = 0; j < 2; j++) u[r][j] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)z[r * 4 + 2 * j], (__bf16)z[r * 4 + 2 * j + 1]});
  } else {
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
      for (int j = 0; j < 2; j++) u[r][j] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)z[r * 4 + 2 * j], (_Float16)z[r * 4 + 2 * j + 1]});
  }
#pragma unroll
  for (int r = 0; r < R; r++)
    if (m + r * step < end) *reinterpret_cast<u32x2*>(a.y + ((m + r * step) * a.ys + n) * 2) = u[r];
}
__device__ __forceinline__ bool by_fours(const Args& a) {
  return ((a.ys | (a.mul ? a.ms : 0) | (a.res ? a.rs : 0)) & 3) == 0;
}

// ---- groups of rows ----
struct RowTile {
  int e, rows;   // group; rows of the tile, 0: no such tile
  int64_t m0;    // the first of them
};
// Row tiles of `each` rows: exactly, or with groups at most, the whole ones and an end of each, no more than rows.
inline int64_t most_tiles(bool grouped, int64_t R, int64_t groups, int64_t each) {
  if (!grouped) return (R + each - 1) / each;
  return groups + R / each < R ? groups + R / each : R;
}
inline int64_t most_tiles(const Args& a, int64_t groups, int64_t each) { return most_tiles(a.offsets != nullptr, a.R, groups, each); }

// The row tiles of BM rows, as a workgroup of NT threads counts them (one barrier) and then finds one of them
// (another): first the whole ones, groups ascending, then what is left of each group, so that the longest work
// is given out first.  Offsets are kept within the rows, so that whatever they hold, no row outside is touched.
// `room`: LDS, free again after the next barrier.
template <int NT, int BM>
struct RowTiles {
  static constexpr int kWaves = NT / 64, kRoom = 2 * kWaves + 4;
  const Args& a;
  int (&room)[kRoom];
  int e0, e1, lo0, hi0;    // the groups that this thread looks at; the rows of the first, often the only one
  int whole, parts;        // tiles of the groups before these
  int all_whole, all;

  __device__ __forceinline__ int at(int e) const {
    const int o = a.offsets[e];
    return o < 0 ? 0 : o < a.R ? o : (int)a.R;
  }
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {  // f(group, first row, rows) for those that have any
    int lo = lo0, hi = hi0;
    for (int e = e0; e < e1;) {
      if (hi > lo) f(e, lo, hi - lo);
      lo = hi;
      if (++e < e1) hi = at(e + 1);
    }
  }

  __device__ __forceinline__ RowTiles(const Args& args, int (&lds)[kRoom]) : a(args), room(lds) {
    if (!a.offsets) {
      all = (int)((a.R + BM - 1) / BM);
      return;
    }
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int per = (a.E + NT - 1) / NT;
    e0 = tid * per < a.E ? tid * per : a.E;
    e1 = e0 + per < a.E ? e0 + per : a.E;
    lo0 = hi0 = 0;
    if (e0 < e1) lo0 = at(e0), hi0 = at(e0 + 1);
    int w = 0, p = 0;
    each([&](int, int, int rows) { w += rows / BM, p += rows % BM != 0; });
    whole = w, parts = p;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(whole, o, 64), v = __shfl_up(parts, o, 64);
      if (lane >= o) whole += u, parts += v;
    }
    if (lane == 63) room[wave] = whole, room[kWaves + wave] = parts;
    if (tid == 0) room[2 * kWaves] = -1;
    __syncthreads();
    whole -= w, parts -= p;
    all_whole = all = 0;
#pragma unroll
    for (int k = 0; k < kWaves; k++) {
      const int u = __builtin_amdgcn_readfirstlane(room[k]), v = __builtin_amdgcn_readfirstlane(room[kWaves + k]);
      if (k < wave) whole += u, parts += v;
      all_whole += u, all += u + v;
    }
  }

  __device__ __forceinline__ RowTile find(int tile) {
    if (!a.offsets) {
      const int64_t m0 = (int64_t)tile * BM, left = a.R - m0;
      return {0, (int)(left < BM ? (left > 0 ? left : 0) : BM), m0};
    }
    int w = whole, p = all_whole + parts;
    each([&](int e, int lo, int rows) {
      const int n = rows / BM;
      const bool first = tile >= w && tile < w + n, last = rows % BM != 0 && tile == p;
      if (first || last) {
        room[2 * kWaves] = e;
        room[2 * kWaves + 1] = lo + (first ? tile - w : n) * BM;
        room[2 * kWaves + 2] = first ? BM : rows % BM;
      }
      w += n, p += rows % BM != 0;
    });
    __syncthreads();
    const int e = __builtin_amdgcn_readfirstlane(room[2 * kWaves]);
    if (e < 0) return {0, 0, 0};
    // (offsets that fall and rise again over many rows can have more tiles than an int counts, and two groups the
    // same number: the end of the rows holds for those too)
    const int m0 = __builtin_amdgcn_readfirstlane(room[2 * kWaves + 1]), rows = __builtin_amdgcn_readfirstlane(room[2 * kWaves + 2]);
    return {e, rows < (int)a.R - m0 ? rows : (int)a.R - m0, (int64_t)m0};
  }
};

}  // namespace lin
}  // namespace bqm
