// Decode product with MXFP4 weights (kernel and launcher; included by qmv_mma.hip):
//   Y[m][n] = sum_b 2^(e[n][b] - 127) sum_{j<32} c[n][32b+j] X[m][32b+j],   M <= 8, fp32 X and Y.
#pragma once

#include "mxfp4.h"

namespace bqm {
namespace {

// One wave per row: lane b takes the blocks b, b + 64, ..., the lanes' sums are added at the end.
__global__ __launch_bounds__(256) void k_qmv_mxfp4(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                   const float* __restrict__ X, float* __restrict__ Y, int M, int64_t N,
                                                   int64_t K, int64_t ks, int64_t kg) {
  const int lane = threadIdx.x & 63;
  const int64_t row = blockIdx.x * (int64_t)4 + (threadIdx.x >> 6);
  if (row >= N) return;
  float acc[BQM_QMV_MAX_M] = {};
  for (int64_t b = lane; b < K / kQK; b += 64) {
    const mx::u32x4 v = *reinterpret_cast<const mx::u32x4*>(codes + mx::code_at(row, b, ks));
    const float s = mx::scale_of(scales[mx::scale_at(row, b, kg)]);
    for (int m = 0; m < BQM_QMV_MAX_M; m++) {
      if (m >= M) break;
      const float* x = X + m * K + b * 32;
      float c = 0;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const mx::f32x2 p[4] = {mx::pair_of<0>(v[j], 1.0f), mx::pair_of<1>(v[j], 1.0f), mx::pair_of<2>(v[j], 1.0f),
                                mx::pair_of<3>(v[j], 1.0f)};
#pragma unroll
        for (int k = 0; k < 4; k++) c = fmaf(p[k].y, x[4 * j + k + 16], fmaf(p[k].x, x[4 * j + k], c));
      }
      acc[m] = fmaf(s, c, acc[m]);
    }
  }
  for (int m = 0; m < BQM_QMV_MAX_M; m++) {
    if (m >= M) break;
    float a = acc[m];
    for (int o = 32; o > 0; o >>= 1) a += __shfl_xor(a, o, 64);
    if (lane == 0) Y[m * N + row] = a;
  }
}

}  // namespace

int launch_qmv_mxfp4(const void* w, const float* X, float* Y, int M, int64_t N, int64_t K, hipStream_t s) {
  const MxLayout L = mx_layout(N, K);
  const uint8_t* codes = static_cast<const uint8_t*>(w);
  const int64_t grid = (N + 3) / 4;
  if (grid > kMaxGrid) return BQM_E_SHAPE;
  hipLaunchKernelGGL(k_qmv_mxfp4, dim3((unsigned)grid), dim3(256), 0, s, codes, codes + L.scales_off, X, Y, M, N, K, L.ks, L.kg);
  return launch_status();
}

}  // namespace bqm
