// MXFP4 rows: repacking of interchange blocks, quantization and its inverse (kernels and
// launchers; included by repack.hip).
#pragma once

#include "mxfp4.h"

namespace bqm {
namespace {

using namespace mx;

constexpr int kPackThreads = 256, kPackWaves = kPackThreads / 64;
constexpr int kPackGrid = 1 << 16;  // workgroups of a launch at most; each takes every kPackGrid-th

// One lane per block and padding block.  The 17-byte blocks are read as unaligned words: 17408 x 5120 takes
// 34.8 us (2.7 TB/s read and written), the way back 39.0 (2.4), once as weights are loaded.
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
    if (real) __builtin_memcpy(&v, s + 1, 16);
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
    const u32x4 v = *reinterpret_cast<const u32x4*>(codes + code_at(row, b, ks));
    __builtin_memcpy(d + 1, &v, 16);
  }
}

// Quantizer and its inverse: bound by the bytes that they move.  A quantizer's wave takes S steps (512 of K, or
// 128 where that would leave units idle) of a 16-row tile; the four lanes of a quad hold a block,
// lane u the values 4u .. 4u + 3 and 16 + 4u .. 16 + 4u + 3, which are word u of its codes.  So a
// load of floats covers 64-byte runs of 16 rows, and a store of codes 256 bytes on end.  17408 x 5120:
// 46.8 us in bf16 (4.8 TB/s), 78 in fp32 (5.2).
template <typename T>
__device__ __forceinline__ void load4(const T* p, bool vec, float (&f)[4]) {
  T v[4];
  if (vec) {
    __builtin_memcpy(v, __builtin_assume_aligned(p, 4 * sizeof(T)), 4 * sizeof(T));
  } else {
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = p[j];
  }
#pragma unroll
  for (int j = 0; j < 4; j++) f[j] = (float)v[j];
}
template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
  return x > y ? x : y;
}

template <int TYPE, int S>
__global__ __launch_bounds__(kPackThreads) void k_quantize_mxfp4(const typename Elem<TYPE>::T* __restrict__ X, int64_t stride, int vec,
                                                                 uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                                 int64_t rows, int64_t nb, int64_t ks, int64_t kg, int64_t units) {
  const int lane = threadIdx.x & 63, u = lane & 3, r = lane >> 2;
  const int64_t per = kg * (4 / S);  // units of a row tile
  for (int64_t i = blockIdx.x * (int64_t)kPackWaves + (threadIdx.x >> 6); i < units; i += (int64_t)gridDim.x * kPackWaves) {
    const int64_t tile = i / per, s0 = (i - tile * per) * S, row = tile * 16 + r;
    const auto* x = X + row * stride + 4 * u;
    uint32_t word = 0;  // the scales of block u of each step
#pragma unroll
    for (int s = 0; s < S; s++) {
      float f[4][2][4];
      bool real[4];
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int64_t b = (s0 + s) * 4 + q;
        real[q] = row < rows && b < nb;
#pragma unroll
        for (int h = 0; h < 2; h++) {
          if (real[q]) {
            load4(x + b * 32 + 16 * h, vec, f[q][h]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; j++) f[q][h][j] = 0;
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 4; q++) {
        uint32_t top = 0;  // as bits: infinities above all numbers, NaN above those
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const uint32_t m = __float_as_uint(f[q][h][j]) & 0x7FFFFFFFu;
            top = top > m ? top : m;
          }
        top = quad_max<0xB1>(top);
        top = quad_max<0x4E>(top);
        // floor(log2 top) - 2 + 127 from the exponent field; e8m0 has nothing below 2^-127
        const uint32_t field = top >> 23, byte = !real[q] ? kOne : field == 255 ? kNanScale : field > 2 ? field - 2 : 0;
        uint32_t c = 0;
        if (field != 255) {
          const float scale = scale_of(byte);
          c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[q][0][0], f[q][1][0], scale, 0);
          c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[q][0][1], f[q][1][1], scale, 1);
          c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[q][0][2], f[q][1][2], scale, 2);
          c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[q][0][3], f[q][1][3], scale, 3);
        }
        if (s0 + s < ks) *reinterpret_cast<uint32_t*>(codes + code_at(row, (s0 + s) * 4 + q, ks) + 4 * u) = c;
        if (u == q) word |= byte << (8 * s);
      }
    }
    uint8_t* at = scales + scale_at(row, s0 * 4 + u, kg);
    if constexpr (S == 4)
      *reinterpret_cast<uint32_t*>(at) = word;
    else
      *at = (uint8_t)word;
  }
}

// 32 lanes write a row of a step, four values each, each lane with the word that holds them, past the
// caches: 17408 x 5120 33.5 us in bf16 (6.7 TB/s; 43 by way of the caches), 70 in fp32.  In the
// quantizer's manner, sixteen rows at a time, fp32 took 207: where K is a multiple of 1024 those rows lie
// on the same memory channels.
template <int TYPE>
__global__ __launch_bounds__(kPackThreads) void k_dequantize_mxfp4(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                                   typename Elem<TYPE>::T* __restrict__ Y, int64_t stride, int vec,
                                                                   int64_t rows, int64_t nb, int64_t ks, int64_t kg, int64_t units) {
  typedef typename Elem<TYPE>::T T;
  const int lane = threadIdx.x & 63;
  auto put = [&](T* y, const float (&f)[4]) {
    typedef T T4 __attribute__((ext_vector_type(4)));
    const T4 v{(T)f[0], (T)f[1], (T)f[2], (T)f[3]};
    if (vec) {
      __builtin_nontemporal_store(v, reinterpret_cast<T4*>(y));
    } else {
#pragma unroll
      for (int k = 0; k < 4; k++) y[k] = v[k];
    }
  };
  for (int64_t i = blockIdx.x * (int64_t)kPackWaves + (threadIdx.x >> 6); i < units; i += (int64_t)gridDim.x * kPackWaves) {
    const int64_t tile = i / ks, s = i - tile * ks;
    const int q = lane >> 3 & 3, j = lane * 4 & 31;  // block and first value of the lane, in rows 0, 2, ... or 1, 3, ...
    const int64_t b = s * 4 + q;
    uint32_t word[8], byte[8];  // the padding has codes and scales too: no load depends on a test
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const int64_t row = tile * 16 + 2 * k + (lane >> 5);
      word[k] = *reinterpret_cast<const uint32_t*>(codes + code_at(row, b, ks) + (j & 15));
      byte[k] = scales[scale_at(row, b, kg)];
    }
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const int64_t row = tile * 16 + 2 * k + (lane >> 5);
      const float scale = scale_of(byte[k]);
      const uint32_t w = word[k] >> (j < 16 ? 0 : 4);  // the codes wanted in the low halves
      const float f[4] = {pair_of<0>(w, 1.0f).x * scale, pair_of<1>(w, 1.0f).x * scale, pair_of<2>(w, 1.0f).x * scale,
                          pair_of<3>(w, 1.0f).x * scale};
      if (row < rows && b < nb) put(Y + row * stride + b * 32 + j, f);
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

static dim3 unit_grid(int64_t units) {
  const int64_t g = (units + kPackWaves - 1) / kPackWaves;
  return dim3((unsigned)(g < kPackGrid ? g : kPackGrid));
}

template <int TYPE>
static int launch_quantize_as(const void* X, int64_t stride, void* packed, int64_t rows, int64_t K, hipStream_t s) {
  const MxLayout L = mx_layout(rows, K);
  uint8_t* codes = static_cast<uint8_t*>(packed);
  const auto* x = static_cast<const typename Elem<TYPE>::T*>(X);
  const int vec = stride % 4 == 0;
  const int64_t units = L.rt * L.kg;
  // four steps a wave where that makes eight waves a unit and more (17408 x 5120: 10880 waves)
  if (units >= 2048)
    hipLaunchKernelGGL((k_quantize_mxfp4<TYPE, 4>), unit_grid(units), dim3(kPackThreads), 0, s, x, stride, vec, codes,
                       codes + L.scales_off, rows, K / kQK, L.ks, L.kg, units);
  else
    hipLaunchKernelGGL((k_quantize_mxfp4<TYPE, 1>), unit_grid(4 * units), dim3(kPackThreads), 0, s, x, stride, vec, codes,
                       codes + L.scales_off, rows, K / kQK, L.ks, L.kg, 4 * units);
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
  const int64_t units = L.rt * L.ks;
  hipLaunchKernelGGL(k_dequantize_mxfp4<TYPE>, unit_grid(units), dim3(kPackThreads), 0, s, codes, codes + L.scales_off,
                     static_cast<typename Elem<TYPE>::T*>(Y), stride, (int)(stride * (int)sizeof(typename Elem<TYPE>::T) % 16 == 0),
                     rows, K / kQK, L.ks, L.kg, units);
  return launch_status();
}

int launch_dequantize_mxfp4(const void* packed, int type, void* Y, int64_t stride, int64_t rows, int64_t K, hipStream_t s) {
  return type == BQM_F32   ? launch_dequantize_as<BQM_F32>(packed, Y, stride, rows, K, s)
         : type == BQM_F16 ? launch_dequantize_as<BQM_F16>(packed, Y, stride, rows, K, s)
                           : launch_dequantize_as<BQM_BF16>(packed, Y, stride, rows, K, s);
}

}  // namespace bqm
