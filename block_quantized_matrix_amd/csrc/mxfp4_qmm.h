// Products of two packed MXFP4 matrices, dense and expert-indexed (kernels and launchers;
// included by qmm.hip):
//   Y[m][n] = sum_k w[n][k] x[m][k]
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies the blocks as they are stored: products of
// codes are exact, block scales only move their exponents, sums are fp32.
#pragma once

#include "mxfp4.h"

namespace bqm {
namespace {

// One wave per 16 x 16 tile of Y; the operands come straight from memory.  Lane l holds row
// l % 16 and block l / 16 of a step of either operand.
__device__ __forceinline__ mx::f32x4 mx_tile(const uint8_t* wc, const uint8_t* ws, const uint8_t* xc, const uint8_t* xs, int64_t ks) {
  mx::f32x4 acc{0, 0, 0, 0};
  for (int64_t k = 0; k < ks; k++) {
    const mx::i32x4 a = *reinterpret_cast<const mx::i32x4*>(wc + k * mx::kOperand);
    const mx::i32x4 b = *reinterpret_cast<const mx::i32x4*>(xc + k * mx::kOperand);
    const int sa = ws[(k >> 2) * mx::kScaleTile + (k & 3)], sb = xs[(k >> 2) * mx::kScaleTile + (k & 3)];
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx::i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                           mx::i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, acc, 4, 4, 0, sa, 0, sb);
  }
  return acc;
}

__global__ __launch_bounds__(64) void k_qmm_mxfp4(const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
                                                  const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
                                                  float* __restrict__ Y, int64_t M, int64_t N, int64_t ks, int64_t kg,
                                                  int64_t tiles_n) {
  const int lane = threadIdx.x, i = lane & 15, q = lane >> 4;
  const int64_t tm = blockIdx.x / tiles_n, tn = blockIdx.x - tm * tiles_n;
  const int at = i * 64 + q * 16, sat = i * 16 + q * 4;
  const mx::f32x4 d = mx_tile(wc + tn * ks * mx::kOperand + at, ws + tn * kg * mx::kScaleTile + sat,
                              xc + tm * ks * mx::kOperand + at, xs + tm * kg * mx::kScaleTile + sat, ks);
  const int64_t m = tm * 16 + i;
  for (int r = 0; r < 4; r++) {
    const int64_t n = tn * 16 + 4 * q + r;
    if (m < M && n < N) Y[m * N + n] = d[r];
  }
}

// One wave per slot and 16 rows of its expert; 15 of the 16 columns repeat the slot's.
__global__ __launch_bounds__(64) void k_qmm_id_mxfp4(const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
                                                     const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
                                                     const int32_t* __restrict__ ids, float* __restrict__ Y, int E, int64_t N,
                                                     int64_t ks, int64_t kg, int top_k, int64_t xtr, int64_t xsr, int64_t tiles_n) {
  const int lane = threadIdx.x, i = lane & 15, q = lane >> 4;
  const int64_t slot = blockIdx.x / tiles_n, n0 = (blockIdx.x - slot * tiles_n) * 16;
  const int e = ids[slot];
  mx::f32x4 d{0, 0, 0, 0};
  if (e >= E) {
    d = mx::f32x4{__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
  } else if (e >= 0) {
    const int64_t t = slot / top_k, x = t * xtr + (slot - t * top_k) * xsr;
    const int64_t w = (int64_t)e * N + (n0 + i < N ? n0 + i : N - 1);
    d = mx_tile(wc + mx::code_at(w, q, ks), ws + mx::scale_at(w, q, kg), xc + mx::code_at(x, q, ks), xs + mx::scale_at(x, q, kg), ks);
  }
  for (int r = 0; r < 4; r++)
    if (i == 0 && n0 + 4 * q + r < N) Y[slot * N + n0 + 4 * q + r] = d[r];
}

}  // namespace

int launch_qmm_mxfp4(const void* w, const void* x, float* Y, int64_t M, int64_t N, int64_t K, hipStream_t s) {
  const MxLayout W = mx_layout(N, K), X = mx_layout(M, K);
  const uint8_t* wc = static_cast<const uint8_t*>(w);
  const uint8_t* xc = static_cast<const uint8_t*>(x);
  if (W.rt * X.rt > kMaxGrid) return BQM_E_SHAPE;
  hipLaunchKernelGGL(k_qmm_mxfp4, dim3((unsigned)(W.rt * X.rt)), dim3(64), 0, s, wc, wc + W.scales_off, xc, xc + X.scales_off, Y, M, N,
                     W.ks, W.kg, W.rt);
  return launch_status();
}

int launch_qmm_id_mxfp4(const void* w, int E, int64_t N, int64_t K, const int32_t* ids, int T, int top_k, const void* x,
                        int64_t x_rows, int64_t x_tok_rows, int64_t x_slot_rows, float* Y, hipStream_t s) {
  const MxLayout W = mx_layout((int64_t)E * N, K), X = mx_layout(x_rows, K);
  const uint8_t* wc = static_cast<const uint8_t*>(w);
  const uint8_t* xc = static_cast<const uint8_t*>(x);
  const int64_t tiles_n = (N + 15) / 16, grid = (int64_t)T * top_k * tiles_n;
  if (grid > kMaxGrid) return BQM_E_SHAPE;
  hipLaunchKernelGGL(k_qmm_id_mxfp4, dim3((unsigned)grid), dim3(64), 0, s, wc, wc + W.scales_off, xc, xc + X.scales_off, ids, Y, E, N,
                     W.ks, W.kg, top_k, x_tok_rows, x_slot_rows, tiles_n);
  return launch_status();
}

}  // namespace bqm
