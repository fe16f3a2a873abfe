// The linear layer for few rows: one token, a decode batch, the rows of an expert that few tokens chose
// (kernel and launcher; included by qmv_mma.hip).  linear.h has the formula.
//
// Weights are read once per run of RM rows, which binds the wide formats; Q4_0 is bound by its conversion (105
// vector instructions for 16 x 128 weights, 60 of them conversion).  A workgroup takes a run of weight rows (T
// tiles of 16) and its W waves the steps of 128 k in turn: wave w the steps w, w + W, ...  A wave brings the
// rows' part of a step to the operands' order through LDS of its own, once for all its tiles, and its
// codes from memory straight to registers, D steps ahead; nothing waits for another wave until the end,
// where the waves' sums are added in order.  One row: 4096 x 4096 of Q4_0 6.1 us, 17408 x 5120 18.8, 34816 x 5120 of
// Q8_0 45 (4.2 TB/s, of which some 8 us are its start and end); 5120 x 17408 of MXFP4 by 8 rows 20, from memory all.
#pragma once

#include "linear.h"

namespace bqm {
namespace {

// RM: rows of x that a workgroup takes.
template <int FMT, int XT, int RM, int T, int D, int W, int OCC>
__global__ __launch_bounds__(W * 64) __attribute__((amdgpu_waves_per_eu(OCC, OCC))) void k_linear_rows(lin::Args a, int halves, int span) {
  using namespace lin;
  constexpr int P = parts_of(XT), TM = (RM + 15) / 16;
  constexpr int kXB = type_size(XT);
  constexpr int kPieces = 128 * kXB / 16;               // of 16 bytes: a row's part of a step
  constexpr int R = (RM * kPieces + 63) / 64;           // pieces that a lane brings
  constexpr int kLot = (RM | 1) * 16;                   // bytes of eight k of all rows; odd in 16s: no bank conflicts
  constexpr int kTurn = P * 16 * kLot, kSums = T * RM * 64;
  constexpr int kWave = kTurn > kSums ? kTurn : kSums;
  constexpr int CB = FMT == BQM_Q8_0 ? 32 : 16;         // code bytes of a block
  constexpr int L = FMT == BQM_Q8_0 ? 2 : 1;            // loads of a tile's step
  __shared__ __attribute__((aligned(16))) uint8_t lds[W * kWave];
  __shared__ int room[RowTiles<W * 64, RM>::kRoom];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, q = lane >> 4;
  const int tile = blockIdx.x / span, run = blockIdx.x - tile * span;
  const RowTile at = RowTiles<W * 64, RM>(a, room).find(tile);
  if (at.rows <= 0) return;  // the whole workgroup
  const int64_t r0 = (int64_t)run * halves * 8, r1 = r0 + halves * 8 < a.N ? r0 + halves * 8 : a.N;
  const int64_t w0 = at.e * a.N + r0;  // the first weight row, of all matrices
  const int nb = a.nb, steps = (nb + 3) >> 2;

  // weights: a lane's 16 bytes of a tile's step, and the scale of one of its four blocks
  constexpr bool MX = FMT == BQM_MXFP4;
  const int64_t t0 = w0 >> 4;
  const uint8_t* wc = a.w + (MX ? t0 * a.ks * mx::kOperand : w0 * nb * CB);
  const uint8_t* wd = a.w + a.scales_off + (MX ? t0 * a.kg * mx::kScaleTile : w0 * nb * 2);
  const int64_t wcb = MX ? (int64_t)(T + 1) * a.ks * mx::kOperand : (r1 - r0) * nb * CB;
  const int64_t wdb = MX ? (int64_t)(T + 1) * a.kg * mx::kScaleTile : (r1 - r0) * nb * 2 + 2;  // a word at the last scale
  uint32_t oc[T], od[T];
#pragma unroll
  for (int t = 0; t < T; t++) {
    const int64_t row = r0 + t * 16 + i;
    const int r = (int)(w0 & 15) + t * 16 + i;  // counted from the first row of tile t0
    if (row >= r1)
      oc[t] = od[t] = kOob;
    else if (MX)
      oc[t] = (uint32_t)mx::code_at(r, q, a.ks), od[t] = (uint32_t)((r >> 4) * a.kg * mx::kScaleTile + q * 64 + (r & 15) * 4);
    else
      oc[t] = (uint32_t)((t * 16 + i) * nb * CB + q * 16), od[t] = (uint32_t)(((t * 16 + i) * nb + q) * 2);
  }
  u32x4 code[D][T][L], xv[D][R];
  uint32_t scale[D][T];
  auto load_w = [&](int d, int t, int s) {
    const bool in = s < steps;  // a step past the last finds nothing: its descriptors are empty
    const __amdgpu_buffer_rsrc_t rc = rsrc(wc, in ? wcb : 0), rd = rsrc(wd, in ? wdb : 0);
#pragma unroll
    for (int l = 0; l < L; l++)
      code[d][t][l] = __builtin_amdgcn_raw_buffer_load_b128(rc, oc[t] + l * 64, s * (MX ? mx::kOperand : 4 * CB), 0);
    const uint32_t o = MX || 4 * s + q < nb ? od[t] : kOob;  // a block past the row's end counts nothing: scale 0
    if constexpr (MX)
      scale[d][t] = __builtin_amdgcn_raw_buffer_load_b8(rd, o, (s >> 2) * mx::kScaleTile + (s & 3), 0);
    else
      scale[d][t] = __builtin_amdgcn_raw_buffer_load_b32(rd, o, s * 8, 0);
  };

  // rows
  const uint8_t* x0 = a.x + at.m0 * a.xs;
  const int64_t xb = (int64_t)(at.rows - 1) * a.xs + (int64_t)nb * 32 * kXB;
  uint32_t ox[R];
#pragma unroll
  for (int r = 0; r < R; r++) {
    const int item = r * 64 + lane, m = item / kPieces, p = item % kPieces;
    ox[r] = m < at.rows && m < RM ? (uint32_t)(m * (int)a.xs + p * 16) : kOob;
  }
  const int block = lane % kPieces / (kPieces / 4);  // of the step, the same for all of a lane's pieces
  auto load_x = [&](int d, int s) {
    const __amdgpu_buffer_rsrc_t rx = rsrc(x0, s < steps ? xb : 0);
#pragma unroll
    for (int r = 0; r < R; r++) xv[d][r] = __builtin_amdgcn_raw_buffer_load_b128(rx, 4 * s + block < nb ? ox[r] : kOob, s * 128 * kXB, 0);
  };
  // A lot is what lane group q of the instruction holds of block u: for Q8_0 eight k on end, for nibbles
  // four of the block's first half and four of its second.
  uint8_t* mine = lds + wave * kWave;
  auto put8 = [&](int part, int u, int lot, int m, int half, u32x2 v) {
    *reinterpret_cast<u32x2*>(mine + ((part * 16 + u * 4 + lot) * kLot) + m * 16 + half * 8) = v;
  };
  auto turn = [&](int d) {
#pragma unroll
    for (int r = 0; r < R; r++) {
      const int item = r * 64 + lane, m = item / kPieces;
      const u32x4 v = xv[d][r];
      if constexpr (P == 3) {
        const int c = lane & 7;  // four numbers of block `block`
        const float f[4] = {__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3])};
        uint32_t part[3][2];
        three_parts<4>(f, part);
        if (m < RM)
#pragma unroll
          for (int p = 0; p < 3; p++) {
            const u32x2 w{part[p][0], part[p][1]};
            FMT == BQM_Q8_0 ? put8(p, block, c >> 1, m, c & 1, w) : put8(p, block, c & 3, m, c >> 2, w);
          }
      } else {
        const int c = lane & 3;  // eight numbers
        if (m < RM) {
          if constexpr (FMT == BQM_Q8_0) {
            *reinterpret_cast<u32x4*>(mine + (block * 4 + c) * kLot + m * 16) = v;
          } else {
            put8(0, block, 2 * (c & 1), m, c >> 1, u32x2{v[0], v[1]});
            put8(0, block, 2 * (c & 1) + 1, m, c >> 1, u32x2{v[2], v[3]});
          }
        }
      }
    }
  };

  f32x4 acc[T][TM] = {};
#pragma unroll
  for (int d = 0; d < D; d++) {
    load_x(d, wave + d * W);
    __builtin_amdgcn_sched_barrier(0);  // in the loop's order, by which it waits
#pragma unroll
    for (int t = 0; t < T; t++) {
      load_w(d, t, wave + d * W);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  for (int s0 = wave; s0 < steps; s0 += D * W) {
#pragma unroll
    for (int d = 0; d < D; d++) {
      const int s = s0 + d * W;
      turn(d);
      __builtin_amdgcn_sched_barrier(0);
      load_x(d, s + D * W);
      mx::wave_turn();
      auto operand = [&](int u, int tm, int p) {
        const int m = tm * 16 + i < RM ? tm * 16 + i : RM - 1;
        return *reinterpret_cast<const u32x4*>(mine + ((p * 16 + u * 4 + q) * kLot) + m * 16);
      };
      u32x4 xop[4][TM][P];
#pragma unroll
      for (int u = 0; u < 4; u++)
#pragma unroll
        for (int tm = 0; tm < TM; tm++)
#pragma unroll
          for (int p = 0; p < P; p++) xop[u][tm][p] = operand(u, tm, p);
#pragma unroll
      for (int t = 0; t < T; t++) {
        if (t * 16 < (int)(r1 - r0)) {  // (loads go on: a branch around them would make the compiler wait for all)
          // words (or pairs of them) of the four blocks to the lane groups, and each block's scale to all
          uint32_t wop[4][4];
#pragma unroll
          for (int l = 0; l < L; l++) {
            u32x4 v = code[d][t][l];
            mma::exchange<FMT != BQM_Q8_0>(v);
            if constexpr (FMT == BQM_Q8_0) {
#pragma unroll
              for (int u = 0; u < 2; u++) {
                uint32_t x0w[2], x1w[2];
                bytes<XT>(v[2 * u], x0w);
                bytes<XT>(v[2 * u + 1], x1w);
                wop[2 * l + u][0] = x0w[0], wop[2 * l + u][1] = x0w[1], wop[2 * l + u][2] = x1w[0], wop[2 * l + u][3] = x1w[1];
              }
            } else {
#pragma unroll
              for (int u = 0; u < 4; u++) {
                uint32_t lo[2], hi[2];
                nibbles<FMT, XT>(v[u], lo, hi);
                wop[u][0] = lo[0], wop[u][1] = lo[1], wop[u][2] = hi[0], wop[u][3] = hi[1];
              }
            }
          }
          const uint32_t f = __float_as_uint(scale_from<FMT, XT>(scale[d][t]));
          u32x4 fs{f, f, f, f};
          mma::exchange<true>(fs);
#pragma unroll
          for (int tm = 0; tm < TM; tm++)
            if (TM == 1 || tm * 16 < at.rows) {
#pragma unroll
              for (int u = 0; u < 4; u++) {
                const u32x4 w{wop[u][0], wop[u][1], wop[u][2], wop[u][3]};
                f32x4 sum{};
#pragma unroll
                for (int p = 0; p < P; p++) {
                  const u32x4 x = xop[u][tm][p];
                  if constexpr (XT == BQM_F16)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, w), sum, 0, 0, 0);
                  else
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, w), sum, 0, 0, 0);
                }
#pragma unroll
                for (int r = 0; r < 4; r++) acc[t][tm][r] = fmaf(__uint_as_float(fs[u]), sum[r], acc[t][tm][r]);
              }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        load_w(d, t, s + D * W);
      }
      mx::wave_turn();  // the next step's rows go where these were read
    }
  }
  // a lane holds column i of a tile, rows 4q .. 4q + 3
#pragma unroll
  for (int t = 0; t < T; t++)
#pragma unroll
    for (int tm = 0; tm < TM; tm++)
#pragma unroll
      for (int r = 0; r < 4; r++)
        if (tm * 16 + 4 * q + r < RM) *reinterpret_cast<float*>(mine + ((t * RM + tm * 16 + 4 * q + r) * 16 + i) * 4) = acc[t][tm][r];
  __syncthreads();
  const float* bias = a.bias ? a.bias + at.e * a.N : nullptr;
  for (int o = threadIdx.x; o < T * 16 * at.rows; o += W * 64) {
    const int col = o % (T * 16), m = o / (T * 16);
    const int64_t n = r0 + col;
    if (n >= r1) continue;
    float z = 0;
#pragma unroll
    for (int w = 0; w < W; w++) z += *reinterpret_cast<const float*>(lds + w * kWave + (((col >> 4) * RM + m) * 16 + (col & 15)) * 4);
    store_as(a.y, (at.m0 + m) * a.ys + n, finish(a, bias, at.m0 + m, n, z), a.y_type);
  }
}

// Rows of x that a workgroup takes, weight rows in eights, row tiles, runs of weight rows.
struct RowsPlan {
  int rm, halves;
  int64_t tiles, span;
};
RowsPlan rows_plan(int x_type, bool grouped, int64_t R, int64_t N, int64_t groups) {
  const int64_t each = (R + groups - 1) / groups;
  RowsPlan p;
  p.rm = each <= 4 ? 4 : each <= 16 || x_type == BQM_F32 ? 16 : 64;
  p.tiles = lin::most_tiles(grouped, R, groups, p.rm);
  const int64_t runs = (N + 7) / 8, most = p.rm == 64 ? 4 : 18;
  const int64_t rounds = (runs * p.tiles + 256 * most - 1) / (256 * most);
  p.halves = (int)((runs * p.tiles + 256 * rounds - 1) / (256 * rounds));
  p.halves = p.halves > most ? (int)most : p.halves < runs ? p.halves : (int)runs;
  p.span = (runs + p.halves - 1) / p.halves;
  return p;
}
// Weight tiles of the kernel that takes a plan: the least that hold its run.
constexpr int rows_kernel(int rm, int halves) {
  const int T = (halves + 1) / 2;
  return rm == 64 ? 2 : T <= 3 ? T : T <= 5 ? 5 : 9;
}

template <int FMT, int XT, int RM, int T>
int launch_rows_as(const lin::Args& a, const RowsPlan& p, hipStream_t s) {
  // Sixteen waves where their registers allow: shorter walks of a long K (5120 x 17408 of MXFP4 by 8 rows 19.9 us, by
  // eight waves 20.9); at K = 4096 and 5120 the longer sum at the end costs as much or more (4096 x 4096 of Q4_0 6.0
  // and 5.7, eight experts of 1536 x 4096 11.6 and 10.6).
  constexpr int W = (XT != BQM_F32 && RM <= 16 && T <= 3) || (RM <= 4 && T <= 2) ? 16 : 8;
  constexpr int D = T == 1 ? 2 : 1;
  hipLaunchKernelGGL((k_linear_rows<FMT, XT, RM, T, D, W, W / 4>), dim3((unsigned)(p.tiles * p.span)), dim3(W * 64), 0, s, a, p.halves,
                     (int)p.span);
  return launch_status();
}
template <int FMT, int XT>
int launch_rows_of(const lin::Args& a, const RowsPlan& p, hipStream_t s) {
  const int T = rows_kernel(p.rm, p.halves);
#define BQM_ROWS(RM)                                         \
  return T == 1   ? launch_rows_as<FMT, XT, RM, 1>(a, p, s)  \
         : T == 2 ? launch_rows_as<FMT, XT, RM, 2>(a, p, s)  \
         : T == 3 ? launch_rows_as<FMT, XT, RM, 3>(a, p, s)  \
         : T == 5 ? launch_rows_as<FMT, XT, RM, 5>(a, p, s)  \
                  : launch_rows_as<FMT, XT, RM, 9>(a, p, s)
  if (p.rm == 4) BQM_ROWS(4);
  if constexpr (XT != BQM_F32)
    if (p.rm == 64) return launch_rows_as<FMT, XT, 64, 2>(a, p, s);
  BQM_ROWS(16);
#undef BQM_ROWS
}

}  // namespace

int launch_linear_rows(int fmt, int x_type, const lin::Args& a, int64_t groups, hipStream_t s) {
  const RowsPlan p = rows_plan(x_type, a.offsets != nullptr, a.R, a.N, groups);
  if (p.tiles * p.span > kMaxGrid) return BQM_E_SHAPE;
#define BQM_ROWS(FMT)                                                        \
  return x_type == BQM_F32   ? launch_rows_of<FMT, BQM_F32>(a, p, s)         \
         : x_type == BQM_F16 ? launch_rows_of<FMT, BQM_F16>(a, p, s)         \
                             : launch_rows_of<FMT, BQM_BF16>(a, p, s)
  if (fmt == BQM_Q4_0) BQM_ROWS(BQM_Q4_0);
  if (fmt == BQM_Q8_0) BQM_ROWS(BQM_Q8_0);
  BQM_ROWS(BQM_MXFP4);
#undef BQM_ROWS
}

// Which of the two kernels: 1 for the one above.  Up to 16 rows it wins everywhere (17408 x 5120, Q4_0: 16 rows
// 21.2 us, by tiles 40; 17 rows 43 and 38).  With more it does where its workgroups, which share K out among
// their waves, are one round on 256 units (1024 x 4096: 512 rows 16 us, by tiles 29, 1024 rows 48 and 29;
// 5120 x 17408, 64 rows 53 and 114); fp32 rows, of which it takes 16 at a time, up to four (4096 x 4096: 64 rows
// 19 and 59, 256 rows 55 and 64).  The rule knows neither K nor a group's mean rows: with a long K the kernel above
// would stay ahead for more rows (5120 x 17408, 65 rows 81 us, by tiles as chosen 114; 256 rows 132 and 135), and
// for groups up to three tokens of eight experts in 128 (1536 x 4096, Q4_0: 3 tokens 25 and 30, 8 tokens 43 and 41).
extern "C" int bqm_internal_linear_rows(int x_type, int grouped, int64_t R, int64_t N, int64_t groups) {
  if (R <= 16) return 1;
  const int64_t each = x_type == BQM_F32 ? 16 : 64;
  return lin::most_tiles(grouped, R, groups, each) * ((N + 31) / 32) <= (x_type == BQM_F32 ? 1024 : 256);
}

// The kernel's rows (times 16) and weight tiles, for the tests: they have to run every one.
extern "C" int bqm_internal_linear_rows_kernel(int x_type, int grouped, int64_t R, int64_t N, int64_t groups) {
  const RowsPlan p = rows_plan(x_type, grouped, R, N, groups);
  return p.rm * 16 + rows_kernel(p.rm, p.halves);
}

// Workgroups of a call, whichever the kernel: kMaxGrid at most are launched.
extern "C" int64_t bqm_internal_linear_workgroups(int fmt, int x_type, int grouped, int64_t R, int64_t N, int64_t K, int64_t groups) {
  if (!bqm_internal_linear_rows(x_type, grouped, R, N, groups)) return linear_tiles_grid(fmt, x_type, grouped, R, N, K, groups);
  const RowsPlan p = rows_plan(x_type, grouped, R, N, groups);
  return p.tiles * p.span;
}

int launch_linear(int fmt, const void* w, int E, const int32_t* offsets, int x_type, const void* X, int64_t x_stride,
                  const float* bias, int act, const void* mul, int64_t mul_stride, const void* res, int64_t res_stride,
                  int y_type, void* Y, int64_t y_stride, int64_t R, int64_t N, int64_t K, hipStream_t s) {
  lin::Args a{static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(X), bias, static_cast<const uint8_t*>(mul),
              static_cast<const uint8_t*>(res), static_cast<uint8_t*>(Y), offsets, N, R, 0, x_stride * lin::type_size(x_type),
              mul_stride, res_stride, y_stride, (int)(K / kQK), 0, 0, E, act, y_type};
  if (fmt == BQM_MXFP4) {
    const MxLayout L = mx_layout((int64_t)E * N, K);
    a.scales_off = L.scales_off, a.ks = (int)L.ks, a.kg = (int)L.kg;
  } else {
    Layout L;
    layout_of(fmt, (int64_t)E * N, K, &L);
    a.scales_off = L.scales_off;
  }
  const int64_t groups = offsets ? (E < R ? E : R) : 1;
  if (bqm_internal_linear_rows(x_type, offsets != nullptr, R, N, groups))
    return launch_linear_rows(fmt, x_type, a, groups, s);
  return launch_linear_tiles(fmt, x_type, a, groups, s);
}

}  // namespace bqm
