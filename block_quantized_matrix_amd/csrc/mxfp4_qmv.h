// Decode product with MXFP4 weights (kernel and launcher; included by qmv_mma.hip):
//   Y[m][n] = sum_b 2^(e[n][b] - 127) sum_{j<32} c[n][32b+j] X[m][32b+j],   M <= 8, fp32 X and Y.
//
// HBM binds it (4.25 bits a weight), so the vector work per weight has to stay small.  Codes are
// converted two at a time to bf16 with their block's scale in place, exact, and go to
// v_mfma_f32_16x16x32_bf16 as its rows.  (The fp4 x fp8 instruction would take them as they are, but
// it drops products below 2^-13 of the largest beside them: inputs in fp8 parts lose too much.)  Each
// input is split into three bf16 parts, together exactly x; the parts of up to five inputs are 15 of
// the 16 columns of one instruction, those of six to eight take two.  Products of bf16 are exact in
// fp32, so what is left is the rounding of fp32 sums.
#pragma once

#include "mma_ops.h"
#include "mxfp4.h"

namespace bqm {
namespace {

constexpr uint32_t kMxOob = 0x80000000u;  // an offset past every descriptor: reads 0

struct MxvArgs {
  const uint8_t* w;
  const float* x;
  float* y;
  int64_t scales_off, N, K, tiles;
  int M, ks, kg, halves;
};

// The three bf16 parts of eight inputs, a[j] and b[j] the pair of word j: each part the upper half of
// what the parts before it leave.
template <bool ODD>
__device__ __forceinline__ void mxv_parts(const float (&a)[4], const float (&b)[4], mx::u32x4 (&part)[3]) {
#pragma unroll
  for (int j = 0; j < 4; j++) {
    float f[2] = {a[j], b[j]};
#pragma unroll
    for (int p = 0; p < 3; p++) {
      uint32_t u[2];
#pragma unroll
      for (int k = 0; k < 2; k++) {
        u[k] = __float_as_uint(f[k]);
        if (ODD && f[k] != f[k]) u[k] |= 0x00400000u;  // a payload in the low half must not leave an infinity
        if (p < 2) f[k] -= __uint_as_float(u[k] & 0xFFFF0000u);
        if (ODD && !__builtin_isfinite(f[k])) f[k] = 0;  // nothing is left of an infinity or a NaN
      }
      part[p][j] = __builtin_amdgcn_perm(u[1], u[0], 0x07060302u);
    }
  }
}
__device__ __forceinline__ void mxv_split(const float (&a)[4], const float (&b)[4], mx::u32x4 (&part)[3]) {
  float probe = 0;
#pragma unroll
  for (int j = 0; j < 4; j++) probe = fmaf(a[j], 0.0f, fmaf(b[j], 0.0f, probe));  // NaN if any is not finite
  if (__any(probe != probe))
    mxv_parts<true>(a, b, part);
  else
    mxv_parts<false>(a, b, part);
}

// A step of a tile where scale bytes may be above 252, whose largest weights bf16 does not hold: infinite,
// they would come out as NaN beside those parts of an input that are 0.  A row with such a byte (among the
// step's four, which lanes i, i + 16, ... hold for row i) takes all its weights at a quarter, exact in bf16
// down to the lowest scale, and its sum times four.
template <int CT>
__device__ __forceinline__ void mxv_far_step(const mx::u32x4& code, uint32_t scale, const mma::bf16x8 (&b)[4][CT], int q,
                                             mx::f32x4 (&acc)[CT]) {
  uint64_t rows = __ballot(scale > 252 && scale < 255);
  rows |= rows >> 32;
  rows |= rows >> 16;
  const uint32_t far = (uint32_t)rows & 0xFFFF;
  const float f = mx::scale_of(scale) * (far >> (threadIdx.x & 15) & 1 ? 0.25f : 1.0f);
  mx::f32x4 sum[CT] = {};
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const mx::f32x2 v[4] = {mx::pair_of<0>(code[k], 1.0f), mx::pair_of<1>(code[k], 1.0f), mx::pair_of<2>(code[k], 1.0f),
                            mx::pair_of<3>(code[k], 1.0f)};
    mx::u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; j++) w[j] = __builtin_amdgcn_perm(__float_as_uint(v[j].y * f), __float_as_uint(v[j].x * f), 0x07060302u);
#pragma unroll
    for (int c = 0; c < CT; c++)
      sum[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mma::bf16x8, w), b[k][c], sum[c], 0, 0, 0);
  }
#pragma unroll
  for (int c = 0; c < CT; c++)
#pragma unroll
    for (int r = 0; r < 4; r++) acc[c][r] += sum[c][r] * (far >> (4 * q + r) & 1 ? 4.0f : 1.0f);
}

// A workgroup takes `halves` runs of eight rows (a run is a whole 128-byte line of a step's codes),
// at most T tiles of 16, its W waves the steps of 128 k in turn: wave w the steps w, w + W, ...  A
// wave splits the inputs of its step once (R items of eight a lane), turns them to the
// instruction's columns (CT of 16) through LDS of its own, and multiplies all the workgroup's
// tiles by them; loads run D steps ahead.  No wave waits for another until the end, when the
// waves' sums are added in order.
template <int R, int CT, int T, int D, int W, int OCC>
__global__ __launch_bounds__(W * 64) __attribute__((amdgpu_waves_per_eu(OCC, OCC))) void k_qmv_mxfp4(MxvArgs a) {
  constexpr int kCols = CT * 16;
  constexpr int kTurn = 16 * (CT == 1 ? 15 : 25) * 16;  // bytes: 16 lots of eight inputs, the columns in use
  constexpr int kSums = T * kCols * 16 * 4;              // bytes of a wave's sums: [tile][column][row]
  constexpr int kWave = kTurn > kSums ? kTurn : kSums;
  __shared__ __attribute__((aligned(16))) uint8_t lds[W * kWave];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, q = lane >> 4;
  const int cols = 3 * a.M, lot = (cols | 1) * 16;  // bytes of a lot; an odd count of 16: no bank conflicts
  const int64_t r0 = (int64_t)blockIdx.x * a.halves * 8, t0 = r0 >> 4;
  const int64_t r1 = r0 + a.halves * 8 < a.N ? r0 + a.halves * 8 : a.N;
  const int64_t cb = (a.tiles - t0) * a.ks * mx::kOperand, sb = (a.tiles - t0) * a.kg * mx::kScaleTile, most = 0x7FFFFFFF;
  // a step past the last finds nothing (and moves nothing): its descriptors are empty
  auto within = [&](const void* p, int64_t bytes, int s) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, s < a.ks ? (int)(bytes < most ? bytes : most) : 0, 0x00020000);
  };
  uint32_t oc[T], os[T];
#pragma unroll
  for (int t = 0; t < T; t++) {
    const int64_t row = (t0 + t) * 16 + i;
    const bool in = row >= r0 && row < r1;
    oc[t] = in ? (uint32_t)(t * a.ks * mx::kOperand + lane * 16) : kMxOob;
    os[t] = in ? (uint32_t)(t * a.kg * mx::kScaleTile + lane * 4) : kMxOob;
  }
  const int nb = (int)(a.K / kQK);
  mx::u32x4 code[D][T], xa[D][R], xb[D][R];
  uint32_t scale[D][T];
  uint32_t ox[R];
#pragma unroll
  for (int r = 0; r < R; r++) {
    const int item = r * 64 + lane, m = item >> 4;
    ox[r] = m < a.M ? (uint32_t)(m * (int)a.K + (item >> 2 & 3) * 32 + (item & 3) * 4) * 4 : kMxOob;
  }
  auto load_x = [&](int d, int s) {
    const __amdgpu_buffer_rsrc_t rx = within(a.x, a.M * a.K * 4, s);
#pragma unroll
    for (int r = 0; r < R; r++) {
      const uint32_t at = 4 * s + (lane >> 2 & 3) < nb ? ox[r] : kMxOob;  // a block past the row's end is not read
      xa[d][r] = __builtin_amdgcn_raw_buffer_load_b128(rx, at, s * 512, 0);
      xb[d][r] = __builtin_amdgcn_raw_buffer_load_b128(rx, at + 64, s * 512, 0);
    }
  };
  auto load_w = [&](int d, int t, int s) {
    code[d][t] = __builtin_amdgcn_raw_buffer_load_b128(within(a.w + t0 * a.ks * mx::kOperand, cb, s), oc[t], s * mx::kOperand, 0);
    scale[d][t] = __builtin_amdgcn_raw_buffer_load_b8(within(a.w + a.scales_off + t0 * a.kg * mx::kScaleTile, sb, s), os[t],
                                                      (s >> 2) * mx::kScaleTile + (s & 3), 0);
  };
  uint8_t* mine = lds + wave * kWave;
  mx::f32x4 acc[T][CT] = {};
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
  auto split = [&](int d) {  // the inputs of a step, as parts, to this wave's LDS
#pragma unroll
    for (int r = 0; r < R; r++) {
      const int item = r * 64 + lane, m = item >> 4, at = (item & 3) * 4 + (item >> 2 & 3);
      float fa[4], fb[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        fa[j] = __uint_as_float(xa[d][r][j]);
        fb[j] = __uint_as_float(xb[d][r][j]);
      }
      mx::u32x4 part[3];
      mxv_split(fa, fb, part);
      if (m < a.M)
#pragma unroll
        for (int p = 0; p < 3; p++) *reinterpret_cast<mx::u32x4*>(mine + at * lot + (3 * m + p) * 16) = part[p];
    }
  };
  auto columns = [&](mma::bf16x8 (&b)[4][CT]) {  // and from there
#pragma unroll
    for (int t = 0; t < 4; t++)
#pragma unroll
      for (int c = 0; c < CT; c++) {
        const int col = c * 16 + i < cols ? c * 16 + i : cols - 1;  // columns not in use repeat one that is
        b[t][c] = *reinterpret_cast<const mma::bf16x8*>(mine + (t * 4 + q) * lot + col * 16);
      }
  };
  for (int s0 = wave; s0 < a.ks; s0 += D * W) {
#pragma unroll
    for (int d = 0; d < D; d++) {
      const int s = s0 + d * W;
      split(d);
      __builtin_amdgcn_sched_barrier(0);
      load_x(d, s + D * W);  // loads are issued in the order of their use, each as soon as its registers are free
      mx::wave_turn();
      mma::bf16x8 b[4][CT];
      columns(b);
#pragma unroll
      for (int t = 0; t < T; t++) {
        const float f = __uint_as_float(scale[d][t] << 23);  // the conversion goes by the exponent field alone
#pragma unroll
        for (int k = 0; k < 4; k++) {
          typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
          const uint32_t word = code[d][t][k];
          const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, f, 1),
                       p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, f, 3);
          const mma::bf16x8 w{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
#pragma unroll
          for (int c = 0; c < CT; c++) acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, b[k][c], acc[t][c], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        load_w(d, t, s + D * W);
      }
      mx::wave_turn();  // the next step's inputs go where these were read
    }
  }
  // Sums that are not finite (from such scales, from a NaN scale, from the inputs) are made again with
  // mxv_far_step.  Looking at the sums costs 0.03 to 0.3 us (4096 x 4096, one input: 4.49 -> 4.52, 34816 x
  // 5120: 16.2 -> 16.3, 5120 x 17408 with five: 14.1 -> 14.4); looking at each scale in the loop: 16.7 for
  // the second.
  float probe[4] = {};
#pragma unroll
  for (int t = 0; t < T; t++)
#pragma unroll
    for (int c = 0; c < CT; c++)
#pragma unroll
      for (int r = 0; r < 4; r++) probe[r] += acc[t][c][r];
  if (__builtin_expect(__any(!__builtin_isfinite((probe[0] + probe[1]) + (probe[2] + probe[3]))), 0)) {  // this wave's steps again
#pragma unroll
    for (int t = 0; t < T; t++)
#pragma unroll
      for (int c = 0; c < CT; c++) acc[t][c] = mx::f32x4{};
    for (int s = wave; s < a.ks; s += W) {
      load_x(0, s);
      split(0);
      mx::wave_turn();
      mma::bf16x8 b[4][CT];
      columns(b);
#pragma unroll
      for (int t = 0; t < T; t++) {
        load_w(0, t, s);
        mxv_far_step<CT>(code[0][t], scale[0][t], b, q, acc[t]);
      }
      mx::wave_turn();
    }
  }
#pragma unroll
  for (int t = 0; t < T; t++)
#pragma unroll
    for (int c = 0; c < CT; c++)
      *reinterpret_cast<mx::f32x4*>(mine + ((t * kCols + c * 16 + i) * 16 + 4 * q) * 4) = acc[t][c];
  __syncthreads();
  for (int o = threadIdx.x; o < T * 16 * a.M; o += W * 64) {
    const int row = o % (T * 16), m = o / (T * 16);
    const int64_t n = t0 * 16 + row;
    if (n < r0 || n >= r1) continue;
    float part[3] = {};
#pragma unroll
    for (int w = 0; w < W; w++)
#pragma unroll
      for (int p = 0; p < 3; p++)
        part[p] += *reinterpret_cast<const float*>(lds + w * kWave + (((row >> 4) * kCols + 3 * m + p) * 16 + (row & 15)) * 4);
    a.y[m * a.N + n] = part[0] + (part[1] + part[2]);
  }
}

template <int R, int CT, int T, int D, int W, int OCC>
int launch_mxv_as(const MxvArgs& a, int64_t grid, hipStream_t s) {
  hipLaunchKernelGGL((k_qmv_mxfp4<R, CT, T, D, W, OCC>), dim3((unsigned)grid), dim3(W * 64), 0, s, a);
  return launch_status();
}
template <int R, int CT>
int launch_mxv(const MxvArgs& a, int64_t grid, hipStream_t s) {
  const int T = (a.halves + 1) / 2;
  return T <= 1   ? launch_mxv_as<R, CT, 1, 2, 16, 4>(a, grid, s)
         : T <= 2 ? launch_mxv_as<R, CT, 2, 1, 16, 4>(a, grid, s)
         : T <= 3 ? launch_mxv_as<R, CT, 3, 1, 8, 2>(a, grid, s)
         : T <= 5 ? launch_mxv_as<R, CT, 5, 1, 8, 2>(a, grid, s)
         : T <= 7 ? launch_mxv_as<R, CT, 7, 1, 8, 2>(a, grid, s)
                  : launch_mxv_as<R, CT, 9, 1, 8, 2>(a, grid, s);
}

}  // namespace

// One workgroup per compute unit, or as many rounds of them as nine tiles each make, so that all end
// together: sixteen waves where a unit has up to two tiles of rows, eight with registers for more
// tiles above.  Measured (us, weights from memory but for the first): 4096 x 4096, one input, 4.5 (eight
// waves 5.7; two workgroups a unit 7.5; 4.8 where the loads past the end were branches; from memory 5.4);
// 5120 x 17408 at batch 8 20.9 (eight waves 22.0, two a unit 31.9); 34816 x 5120 with eight waves 19.3,
// 4.9 TB/s (sixteen and two rounds 27.1), at batch 8 22.9 (38.8).  Loads two steps ahead instead of one gained nothing from two tiles on (5120 x 17408
// at batch 8: 23.4), nor did runs of four rows, which give every unit as many (7168 x 5120: 7.2, 5.7
// with eight).
extern "C" int64_t bqm_internal_qmv_mxfp4_runs(int64_t N) {  // of eight rows, of a workgroup
  const int64_t runs = (N + 7) / 8, rounds = (runs + 256 * 17 - 1) / (256 * 17);
  return (runs + 256 * rounds - 1) / (256 * rounds);
}

int launch_qmv_mxfp4(const void* w, const float* X, float* Y, int M, int64_t N, int64_t K, hipStream_t s) {
  const MxLayout L = mx_layout(N, K);
  if (K > BQM_MXFP4_MAX_K || N > ((int64_t)1 << 29)) return BQM_E_SHAPE;  // the grid stays below kMaxGrid
  const int64_t halves = bqm_internal_qmv_mxfp4_runs(N), grid = ((N + 7) / 8 + halves - 1) / halves;
  const MxvArgs a{static_cast<const uint8_t*>(w), X, Y, L.scales_off, N, K, L.rt, M, (int)L.ks, (int)L.kg, (int)halves};
  return M <= 4 ? launch_mxv<1, 1>(a, grid, s) : M == 5 ? launch_mxv<2, 1>(a, grid, s) : launch_mxv<2, 2>(a, grid, s);
}

}  // namespace bqm
