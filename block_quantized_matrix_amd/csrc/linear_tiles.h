// The linear layer for many rows (kernel and launcher; included by qmm.hip).  linear.h has the formula.
//
// The matrix cores and the vector unit bind it together: a block of 32 x 32 outputs takes two
// v_mfma_f32_32x32x16 (64 clocks of a SIMD) and 16 FMAs for the block's scale; the codes' conversion
// comes on top, once for all the row tiles of a wave.  So a wave takes 64 weight rows by 128 rows (the
// conversion of two tiles over eight products), and two waves share a SIMD, one's vector work under the
// other's products.
#pragma once

#include "linear.h"
#include "mxfp4_qmm.h"

namespace bqm {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Four waves side by side along the weight rows (TN tiles of 32 each), all over the same TM tiles of 32 rows.
// K advances by steps of two blocks.  The rows go from memory straight into LDS, four stages, three steps
// ahead; codes and scales straight to the registers of the wave that converts them, D steps ahead.
template <int FMT, int XT, int TN, int TM>
struct LinTile {
  static constexpr int kWaves = 4, kBN = kWaves * TN * 32, kBM = TM * 32;
  static constexpr int kXB = lin::type_size(XT), kRow = 64 * kXB;  // bytes of a row's step
  static constexpr int kStage = kBM * kRow, kPieces = kStage / (kWaves * 1024);
  static constexpr int kLoads = FMT == BQM_Q8_0 ? 2 : 1;           // of 16 bytes a lane, of a weight tile's step
  static_assert(kStage % (kWaves * 1024) == 0, "whole loads");
};

template <int FMT, int XT, int TN, int TM>
__device__ __forceinline__ void lin_core(const lin::Args& a, const lin::RowTile& at, int tn, uint8_t* lds0, uint8_t* lds1, uint8_t* lds2,
                                         uint8_t* lds3) {
  using namespace lin;
  using C = LinTile<FMT, XT, TN, TM>;
  constexpr int P = parts_of(XT), L = C::kLoads, PX = C::kPieces, D = 2;
  constexpr bool MX = FMT == BQM_MXFP4;
  constexpr int CB = FMT == BQM_Q8_0 ? 32 : 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 31, h = lane >> 5;
  const int64_t n0 = (int64_t)tn * C::kBN + wave * TN * 32;
  const int nb = a.nb, steps = (nb + 1) >> 1;

  // weights: rows past the end repeat the last one
  const int64_t first = at.e * a.N + (n0 < a.N ? n0 : a.N - 1), t0 = first >> 4;
  const uint8_t* wc = a.w + (MX ? t0 * a.ks * mx::kOperand : first * nb * CB);
  const uint8_t* wd = a.w + a.scales_off + (MX ? t0 * a.kg * mx::kScaleTile : first * nb * 2);
  const int left = (int)(a.N - n0 < TN * 32 ? a.N - n0 : TN * 32);  // rows of this wave
  const int own = left > 0 ? left : 1;
  const int64_t span = ((first & 15) + own + 15) >> 4;
  const __amdgpu_buffer_rsrc_t rc = rsrc(wc, MX ? span * a.ks * mx::kOperand : (int64_t)own * nb * CB);
  const __amdgpu_buffer_rsrc_t rd = rsrc(wd, MX ? span * a.kg * mx::kScaleTile : (int64_t)own * nb * 2 + 2);  // a word at the last scale
  uint32_t oc[TN], od[TN];
#pragma unroll
  for (int t = 0; t < TN; t++) {
    const int r = t * 32 + i < own ? t * 32 + i : own - 1, mr = (int)(first & 15) + r;
    if (MX)
      oc[t] = (uint32_t)mx::code_at(mr, h, a.ks), od[t] = (uint32_t)((mr >> 4) * a.kg * mx::kScaleTile + h * 64 + (mr & 15) * 4);
    else
      oc[t] = (uint32_t)(r * nb * CB + h * 16), od[t] = (uint32_t)(r * nb * 2);
  }
  // Every step loads, those past the last again what the last one takes (a branch around a load would make
  // the compiler wait for all loads where the paths join).
  u32x4 code[D][TN][L];
  uint32_t scale[D][TN];
  auto load_w = [&](int d, int s) {
    s = s < steps ? s : steps - 1;
#pragma unroll
    for (int t = 0; t < TN; t++) {
#pragma unroll
      for (int l = 0; l < L; l++)
        code[d][t][l] = __builtin_amdgcn_raw_buffer_load_b128(rc, oc[t] + l * 32, MX ? (s >> 1) * mx::kOperand + (s & 1) * 512 : s * 2 * CB, 0);
      if constexpr (MX)  // of one of the two blocks
        scale[d][t] = __builtin_amdgcn_raw_buffer_load_b8(rd, od[t], (s >> 3) * mx::kScaleTile + (s & 1) * 128 + (s >> 1 & 3), 0);
      else  // of both
        scale[d][t] = __builtin_amdgcn_raw_buffer_load_b32(rd, od[t], s * 4, 0);
    }
  };

  // rows: 16-byte slots, that of place p in row m holding slot p ^ (m & 7), so that lanes a row apart read
  // other banks
  const __amdgpu_buffer_rsrc_t rx = rsrc(a.x + at.m0 * a.xs, (int64_t)(at.rows - 1) * a.xs + (int64_t)nb * 32 * C::kXB);
  constexpr int kSlots = C::kRow / 16;
  uint32_t ox[PX];
#pragma unroll
  for (int p = 0; p < PX; p++) {
    const int u = (p * 4 + wave) * 64 + lane, m = u / kSlots, slot = u % kSlots ^ (m & 7);
    ox[p] = (uint32_t)((m < at.rows ? m : at.rows - 1) * (int)a.xs + slot * 16);
  }
  auto load_x = [&](int s, uint8_t* stage) {
    s = s < steps ? s : steps - 1;
#pragma unroll
    for (int p = 0; p < PX; p++)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (LdsPtr)(stage + (p * 4 + wave) * 1024), 16, ox[p], s * C::kRow, 0, 0);
  };
  auto slot_at = [&](const uint8_t* stage, int t, int slot) {
    return *reinterpret_cast<const u32x4*>(stage + (t * 32 + i) * C::kRow + (slot ^ (i & 7)) * 16);
  };

  f32x16 acc[TN][TM] = {};
  auto meet = [&] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto block = [&](int d, int b, const uint8_t* stage) {
    // the codes of block b: of each tile, first half and second half of its k
    u32x4 w[TN][2];
    float f[TN];
#pragma unroll
    for (int t = 0; t < TN; t++) {
      u32x4 v = code[d][t][FMT == BQM_Q8_0 ? b : 0];
      // the halves of a wave loaded a unit each; now each has its half of both
      uint32_t v0 = v[0], v1 = v[1], v2 = v[2], v3 = v[3];
      mma::swap32(v0, v2);
      mma::swap32(v1, v3);
      if constexpr (FMT == BQM_Q8_0) {
        uint32_t u[4][2];
        bytes<XT>(v0, u[0]);
        bytes<XT>(v1, u[1]);
        bytes<XT>(v2, u[2]);
        bytes<XT>(v3, u[3]);
        w[t][0] = u32x4{u[0][0], u[0][1], u[1][0], u[1][1]};
        w[t][1] = u32x4{u[2][0], u[2][1], u[3][0], u[3][1]};
      } else {
        uint32_t lo[2][2], hi[2][2];
        nibbles<FMT, XT>(b ? v2 : v0, lo[0], hi[0]);
        nibbles<FMT, XT>(b ? v3 : v1, lo[1], hi[1]);
        w[t][0] = u32x4{lo[0][0], lo[0][1], lo[1][0], lo[1][1]};
        w[t][1] = u32x4{hi[0][0], hi[0][1], hi[1][0], hi[1][1]};
      }
      uint32_t s0 = scale[d][t], s1 = s0;
      if constexpr (MX)
        mma::swap32(s0, s1);
      else
        s1 >>= 16;
      f[t] = scale_from<FMT, XT>(b ? s1 : s0);
    }
#pragma unroll
    for (int m = 0; m < TM; m++) {
      u32x4 x[2][P];
#pragma unroll
      for (int j = 0; j < 2; j++) {
        if constexpr (P == 1) {
          x[j][0] = slot_at(stage, m, b * 4 + j * 2 + h);
        } else {
          const u32x4 v0 = slot_at(stage, m, b * 8 + j * 4 + h * 2), v1 = slot_at(stage, m, b * 8 + j * 4 + h * 2 + 1);
          float g[8];
#pragma unroll
          for (int k = 0; k < 4; k++) g[k] = __uint_as_float(v0[k]), g[4 + k] = __uint_as_float(v1[k]);
          uint32_t part[3][4];
          three_parts<8>(g, part);
#pragma unroll
          for (int p = 0; p < 3; p++) x[j][p] = u32x4{part[p][0], part[p][1], part[p][2], part[p][3]};
        }
      }
#pragma unroll
      for (int t = 0; t < TN; t++) {
        f32x16 sum{};
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
          for (int p = 0; p < P; p++) {
            if constexpr (XT == BQM_F16)
              sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x[j][p]), __builtin_bit_cast(f16x8, w[t][j]), sum, 0, 0, 0);
            else
              sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x[j][p]), __builtin_bit_cast(bf16x8, w[t][j]), sum, 0, 0, 0);
          }
#pragma unroll
        for (int r = 0; r < 16; r++) acc[t][m][r] = fmaf(f[t], sum[r], acc[t][m][r]);
      }
    }
  };
  auto step = [&](int d, int s, uint8_t* cur, uint8_t* free) {
    // x of step s was issued before the weights of s + D - 1 .. and the rows of s + 1, s + 2
    vm_wait<2 * (PX + TN * (L + 1))>();
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave has read all of the stage that is free now
    meet();
    __builtin_amdgcn_sched_barrier(0);
    load_x(s + 3, free);
    __builtin_amdgcn_sched_barrier(0);
    block(d, 0, cur);
    if (2 * s + 1 < nb) block(d, 1, cur);
    __builtin_amdgcn_sched_barrier(0);
    load_w(d, s + D);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (steps > 0) {
    load_x(0, lds0);
    __builtin_amdgcn_sched_barrier(0);
    load_w(0, 0);
    __builtin_amdgcn_sched_barrier(0);
    load_x(1, lds1);
    __builtin_amdgcn_sched_barrier(0);
    load_w(1, 1);
    __builtin_amdgcn_sched_barrier(0);
    load_x(2, lds2);
    __builtin_amdgcn_sched_barrier(0);
    for (int s = 0;; s += 4) {
      step(0, s, lds0, lds3);
      if (s + 1 >= steps) break;
      step(1, s + 1, lds1, lds0);
      if (s + 2 >= steps) break;
      step(0, s + 2, lds2, lds1);
      if (s + 3 >= steps) break;
      step(1, s + 3, lds3, lds2);
      if (s + 4 >= steps) break;
    }
  }
  vm_wait<0>();  // nothing may be on its way into LDS when it is used again
  __syncthreads();
  // A lane holds column i of a weight tile, rows 8 (r / 4) + 4 h + r % 4 of a row tile.  Each wave turns its row
  // tiles in a stage of its own, so that it stores whole runs of a row of Y.
  constexpr int kCols = TN * 32;
  static_assert(32 * kCols * 4 <= C::kStage, "a row tile's outputs fit a stage");
  float* turn = reinterpret_cast<float*>(wave == 0 ? lds0 : wave == 1 ? lds1 : wave == 2 ? lds2 : lds3);
  const float* bias = a.bias ? a.bias + at.e * a.N : nullptr;
  const bool fours = by_fours(a);
#pragma unroll
  for (int m = 0; m < TM; m++) {
#pragma unroll
    for (int t = 0; t < TN; t++)
#pragma unroll
      for (int r = 0; r < 16; r++) turn[(8 * (r >> 2) + 4 * h + (r & 3)) * kCols + t * 32 + i] = acc[t][m][r];
    mx::wave_turn();
    const int rows = at.rows - m * 32 < 32 ? at.rows - m * 32 : 32;
    if (fours) {
#pragma unroll 1
      for (int o = lane; o < rows * (kCols / 4); o += 64) {
        const int row = o / (kCols / 4), c = o % (kCols / 4) * 4;
        const f32x4 z = *reinterpret_cast<const f32x4*>(turn + row * kCols + c);
        const int64_t y = at.m0 + m * 32 + row, n = n0 + c;
        if (n + 4 <= a.N)
          finish4(a, bias, y, n, z);
        else
#pragma unroll
          for (int j = 0; j < 4; j++)
            if (n + j < a.N) store_as(a.y, y * a.ys + n + j, finish(a, bias, y, n + j, z[j]), a.y_type);
      }
    } else {
#pragma unroll 1
      for (int o = lane; o < rows * kCols; o += 64) {
        const int64_t y = at.m0 + m * 32 + o / kCols, n = n0 + o % kCols;
        if (n < a.N) store_as(a.y, y * a.ys + n, finish(a, bias, y, n, turn[o]), a.y_type);
      }
    }
    mx::wave_turn();
  }
}

template <int FMT, int XT, int TN, int TM, int OCC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(OCC, OCC))) void k_linear_tiles(lin::Args a, int tiles_m, int tiles_n) {
  using namespace lin;
  using C = LinTile<FMT, XT, TN, TM>;
  __shared__ __attribute__((aligned(16))) uint8_t lds0[C::kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[C::kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds2[C::kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds3[C::kStage];
  __shared__ int64_t room[256 / 64 + 2];
  RowTiles<256, C::kBM> groups(a, room);
  int tm, tn;
  if (a.offsets) {  // an XCD (workgroups go round them) takes a run of items, along the weights of a row tile
    const int items = groups.all * tiles_n, xcd = blockIdx.x & 7, more = items & 7, nth = blockIdx.x >> 3;
    if (nth >= (items >> 3) + (xcd < more)) return;  // none left, the whole workgroup
    const int item = xcd * (items >> 3) + (xcd < more ? xcd : more) + nth;
    tm = item / tiles_n, tn = item - tm * tiles_n;
  } else {
    const MxPlace at = mx_place(blockIdx.x, tiles_m, tiles_n);
    tm = at.m, tn = at.n;
  }
  const RowTile at = groups.find(tm);
  if (at.rows <= 0) return;
  lin_core<FMT, XT, TN, TM>(a, at, tn, lds0, lds1, lds2, lds3);
}

template <int FMT, int XT, int TN, int TM, int OCC>
int launch_tiles_as(const lin::Args& a, int64_t groups, hipStream_t s) {
  using C = LinTile<FMT, XT, TN, TM>;
  const int64_t tm = a.offsets ? groups + a.R / C::kBM : (a.R + C::kBM - 1) / C::kBM, tn = (a.N + C::kBN - 1) / C::kBN;
  // with groups, up to seven workgroups more: the items are dealt to the XCDs in eight runs
  const int64_t grid = a.offsets ? (tm * tn + 7) / 8 * 8 : tm * tn;
  if (grid > kMaxGrid) return BQM_E_SHAPE;
  hipLaunchKernelGGL((k_linear_tiles<FMT, XT, TN, TM, OCC>), dim3((unsigned)grid), dim3(256), 0, s, a, (int)tm, (int)tn);
  return launch_status();
}
template <int FMT, int XT>
int launch_tiles_of(const lin::Args& a, int64_t groups, hipStream_t s) {
  return launch_tiles_as<FMT, XT, 2, XT == BQM_F32 ? 2 : 4, 2>(a, groups, s);
}

}  // namespace

int launch_linear_tiles(int fmt, int x_type, const lin::Args& a, int64_t groups, int64_t rows_each, hipStream_t s) {
  (void)rows_each;
#define BQM_TILES(FMT)                                                   \
  return x_type == BQM_F32   ? launch_tiles_of<FMT, BQM_F32>(a, groups, s) \
         : x_type == BQM_F16 ? launch_tiles_of<FMT, BQM_F16>(a, groups, s) \
                             : launch_tiles_of<FMT, BQM_BF16>(a, groups, s)
  if (fmt == BQM_Q4_0) BQM_TILES(BQM_Q4_0);
  if (fmt == BQM_Q8_0) BQM_TILES(BQM_Q8_0);
  BQM_TILES(BQM_MXFP4);
#undef BQM_TILES
}

}  // namespace bqm
