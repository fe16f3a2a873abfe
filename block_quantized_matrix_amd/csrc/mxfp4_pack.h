// MXFP4 rows: repacking of interchange blocks, quantization and its inverse (kernels and
// launchers; included by repack.hip).
#pragma once

#include "mxfp4.h"

namespace bqm {
namespace {

using namespace mx;

constexpr int kPackThreads = 256;
constexpr int kPackGrid = 1 << 16;  // workgroups of a launch at most; each takes every kPackGrid-th

__global__ __launch_bounds__(kPackThreads) void k_repack_mxfp4(const uint8_t* __restrict__ src, uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales, int64_t rows, int64_t nb,
                                                               int64_t ks, int64_t kg, int64_t total) {
  for (int64_t i = blockIdx.x * (int64_t)kPackThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kPackThreads) {
    const int64_t row = i / (kg * 16), b = i - row * (kg * 16);
    const bool real = row < rows && b < nb;
    const uint8_t* s = src + (row * nb + b) * 17;
    scales[scale_at(row, b, kg)] = real ? s[0] : kOne;
    if (b >= ks * 4) continue;
    u32x4 v{0, 0, 0, 0};
    if (real)
#pragma unroll
      for (int k = 0; k < 4; k++)
        v[k] = (uint32_t)s[1 + 4 * k] | (uint32_t)s[2 + 4 * k] << 8 | (uint32_t)s[3 + 4 * k] << 16 | (uint32_t)s[4 + 4 * k] << 24;
    *reinterpret_cast<u32x4*>(codes + code_at(row, b, ks)) = v;
  }
}

__global__ __launch_bounds__(kPackThreads) void k_unpack_mxfp4(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                               uint8_t* __restrict__ dst, int64_t nb, int64_t ks, int64_t kg,
                                                               int64_t total) {
  for (int64_t i = blockIdx.x * (int64_t)kPackThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kPackThreads) {
    const int64_t row = i / nb, b = i - row * nb;
    uint8_t* d = dst + i * 17;
    d[0] = scales[scale_at(row, b, kg)];
    const uint8_t* c = codes + code_at(row, b, ks);
    for (int k = 0; k < 16; k++) d[1 + k] = c[k];
  }
}

template <int TYPE>
__global__ __launch_bounds__(kPackThreads) void k_quantize_mxfp4(const typename Elem<TYPE>::T* __restrict__ X, int64_t stride,
                                                                 uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                                 int64_t rows, int64_t nb, int64_t ks, int64_t kg, int64_t total) {
  for (int64_t i = blockIdx.x * (int64_t)kPackThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kPackThreads) {
    const int64_t row = i / (kg * 16), b = i - row * (kg * 16);
    uint32_t byte = kOne;
    u32x4 v{0, 0, 0, 0};
    if (row < rows && b < nb) {
      const auto* x = X + row * stride + b * 32;
      float f[32], top = 0;
      bool finite = true;
#pragma unroll
      for (int j = 0; j < 32; j++) {
        f[j] = (float)x[j];
        finite = finite && __builtin_isfinite(f[j]);
        top = fmaxf(top, fabsf(f[j]));
      }
      // floor(log2 top) - 2 + 127 from the exponent field; e8m0 has nothing below 2^-127
      const int field = (int)(__float_as_uint(top) >> 23);
      byte = finite ? (field > 2 ? field - 2 : 0) : kNanScale;
      if (finite) {
        const float s = scale_of(byte);
#pragma unroll
        for (int j = 0; j < 4; j++) {
          uint32_t w = 0;
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4 * j], f[4 * j + 16], s, 0);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4 * j + 1], f[4 * j + 17], s, 1);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4 * j + 2], f[4 * j + 18], s, 2);
          v[j] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4 * j + 3], f[4 * j + 19], s, 3);
        }
      }
    }
    scales[scale_at(row, b, kg)] = (uint8_t)byte;
    if (b < ks * 4) *reinterpret_cast<u32x4*>(codes + code_at(row, b, ks)) = v;
  }
}

template <int TYPE>
__global__ __launch_bounds__(kPackThreads) void k_dequantize_mxfp4(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                                   typename Elem<TYPE>::T* __restrict__ Y, int64_t stride,
                                                                   int64_t nb, int64_t ks, int64_t kg, int64_t total) {
  for (int64_t i = blockIdx.x * (int64_t)kPackThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kPackThreads) {
    const int64_t row = i / nb, b = i - row * nb;
    const float s = scale_of(scales[scale_at(row, b, kg)]);
    const u32x4 v = *reinterpret_cast<const u32x4*>(codes + code_at(row, b, ks));
    auto* y = Y + row * stride + b * 32;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const f32x2 p[4] = {pair_of<0>(v[j], 1.0f), pair_of<1>(v[j], 1.0f), pair_of<2>(v[j], 1.0f), pair_of<3>(v[j], 1.0f)};
#pragma unroll
      for (int k = 0; k < 4; k++) {
        y[4 * j + k] = (typename Elem<TYPE>::T)(p[k].x * s);
        y[4 * j + k + 16] = (typename Elem<TYPE>::T)(p[k].y * s);
      }
    }
  }
}

dim3 pack_grid(int64_t total) {
  const int64_t g = (total + kPackThreads - 1) / kPackThreads;
  return dim3((unsigned)(g < kPackGrid ? g : kPackGrid));
}

}  // namespace

int launch_repack_mxfp4(const void* src, void* dst, int64_t rows, int64_t K, hipStream_t s) {
  const MxLayout L = mx_layout(rows, K);
  uint8_t* codes = static_cast<uint8_t*>(dst);
  const int64_t total = L.rt * kTileRows * L.kg * 16;
  hipLaunchKernelGGL(k_repack_mxfp4, pack_grid(total), dim3(kPackThreads), 0, s, static_cast<const uint8_t*>(src), codes,
                     codes + L.scales_off, rows, K / kQK, L.ks, L.kg, total);
  return launch_status();
}

int launch_unpack_mxfp4(const void* src, void* dst, int64_t rows, int64_t K, hipStream_t s) {
  const MxLayout L = mx_layout(rows, K);
  const uint8_t* codes = static_cast<const uint8_t*>(src);
  const int64_t total = rows * (K / kQK);
  hipLaunchKernelGGL(k_unpack_mxfp4, pack_grid(total), dim3(kPackThreads), 0, s, codes, codes + L.scales_off,
                     static_cast<uint8_t*>(dst), K / kQK, L.ks, L.kg, total);
  return launch_status();
}

template <int TYPE>
static int launch_quantize_as(const void* X, int64_t stride, void* packed, int64_t rows, int64_t K, hipStream_t s) {
  const MxLayout L = mx_layout(rows, K);
  uint8_t* codes = static_cast<uint8_t*>(packed);
  const int64_t total = L.rt * kTileRows * L.kg * 16;
  hipLaunchKernelGGL(k_quantize_mxfp4<TYPE>, pack_grid(total), dim3(kPackThreads), 0, s,
                     static_cast<const typename Elem<TYPE>::T*>(X), stride, codes, codes + L.scales_off, rows, K / kQK, L.ks, L.kg,
                     total);
  return launch_status();
}

int launch_quantize_mxfp4(int type, const void* X, int64_t stride, void* packed, int64_t rows, int64_t K, hipStream_t s) {
  return type == BQM_F32   ? launch_quantize_as<BQM_F32>(X, stride, packed, rows, K, s)
         : type == BQM_F16 ? launch_quantize_as<BQM_F16>(X, stride, packed, rows, K, s)
                           : launch_quantize_as<BQM_BF16>(X, stride, packed, rows, K, s);
}

template <int TYPE>
static int launch_dequantize_as(const void* packed, void* Y, int64_t stride, int64_t rows, int64_t K, hipStream_t s) {
  const MxLayout L = mx_layout(rows, K);
  const uint8_t* codes = static_cast<const uint8_t*>(packed);
  const int64_t total = rows * (K / kQK);
  hipLaunchKernelGGL(k_dequantize_mxfp4<TYPE>, pack_grid(total), dim3(kPackThreads), 0, s, codes, codes + L.scales_off,
                     static_cast<typename Elem<TYPE>::T*>(Y), stride, K / kQK, L.ks, L.kg, total);
  return launch_status();
}

int launch_dequantize_mxfp4(const void* packed, int type, void* Y, int64_t stride, int64_t rows, int64_t K, hipStream_t s) {
  return type == BQM_F32   ? launch_dequantize_as<BQM_F32>(packed, Y, stride, rows, K, s)
         : type == BQM_F16 ? launch_dequantize_as<BQM_F16>(packed, Y, stride, rows, K, s)
                           : launch_dequantize_as<BQM_BF16>(packed, Y, stride, rows, K, s);
}

}  // namespace bqm
