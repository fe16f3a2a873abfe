// Rows of a packed table by token id (kernel and launcher; included by repack.hip):
//   Y[t][k] = scale * dequant(W)[ids[t]][k]
//
// Bound by the bytes that it writes.  A wave takes 512 numbers of a row, a lane eight on end: a store of
// theirs covers whole lines, and the four lanes of a block read its scale and codes from one line.
#pragma once

#include "mxfp4.h"

namespace bqm {
namespace {

constexpr int kEmbedWaves = 4, kEmbedRun = 512;

template <int FMT, int TYPE>
__global__ __launch_bounds__(kEmbedWaves * 64) void k_embed(const uint8_t* __restrict__ w, int64_t scales_off, int64_t rows, int64_t K,
                                                            int64_t ks, int64_t kg, const int32_t* __restrict__ ids, int64_t units,
                                                            int per_row, float scale, typename mx::Elem<TYPE>::T* __restrict__ Y,
                                                            int64_t y_stride, int vec) {
  typedef typename mx::Elem<TYPE>::T T;
  const int lane = threadIdx.x & 63;
  for (int64_t unit = (int64_t)blockIdx.x * kEmbedWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); unit < units;
       unit += (int64_t)gridDim.x * kEmbedWaves) {
    const int64_t t = unit / per_row, k = (unit - t * per_row) * kEmbedRun + lane * 8;
    const int64_t id = ids[t];
    if (k >= K) continue;
    float f[8];
    if (id < 0 || id >= rows) {
#pragma unroll
      for (int j = 0; j < 8; j++) f[j] = id < 0 ? 0.0f : __builtin_nanf("");
    } else {
      const int64_t b = k >> 5, at = id * (K >> 5) + b;
      const int c = (int)(k >> 3) & 3;  // the lane's eight of the block
      uint32_t u[2];
      if constexpr (FMT == BQM_Q8_0)
        __builtin_memcpy(u, __builtin_assume_aligned(w + at * 32 + c * 8, 8), 8);
      else if constexpr (FMT == BQM_Q4_0)
        __builtin_memcpy(u, __builtin_assume_aligned(w + at * 16 + (c & 1) * 8, 8), 8);
      else
        __builtin_memcpy(u, __builtin_assume_aligned(w + mx::code_at(id, b, ks) + (c & 1) * 8, 8), 8);
      if constexpr (FMT == BQM_MXFP4) {
        // the scale last: a weight beyond fp32's largest number counts as it is
        const uint32_t e = w[scales_off + mx::scale_at(id, b, kg)];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t v = u[h] >> (c & 2 ? 4 : 0);
          const float g[4] = {mx::pair_of<0>(v, 1.0f).x, mx::pair_of<1>(v, 1.0f).x, mx::pair_of<2>(v, 1.0f).x, mx::pair_of<3>(v, 1.0f).x};
#pragma unroll
          for (int j = 0; j < 4; j++) f[h * 4 + j] = e == mx::kNanScale ? __builtin_nanf("") : ldexpf(g[j] * scale, (int)e - 127);
        }
      } else {
        const float d = (float)reinterpret_cast<const _Float16*>(w + scales_off)[at];
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const uint32_t v = u[j >> 2] >> (8 * (j & 3));
          const int code = FMT == BQM_Q8_0 ? (int)(int8_t)v : (int)(v >> (c & 2 ? 4 : 0) & 15) - 8;
          f[j] = (float)code * d * scale;  // the first product is exact
        }
      }
    }
    T* y = Y + t * y_stride + k;
    if (vec) {
      T o[8];
#pragma unroll
      for (int j = 0; j < 8; j++) o[j] = (T)f[j];
      __builtin_memcpy(__builtin_assume_aligned(y, 16), o, sizeof(o));
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) y[j] = (T)f[j];
    }
  }
}

template <int FMT>
int launch_embed_of(const uint8_t* w, int64_t scales_off, int64_t rows, int64_t K, int64_t ks, int64_t kg, const int32_t* ids,
                    int64_t T, float scale, int type, void* Y, int64_t y_stride, hipStream_t s) {
  const int64_t per_row = (K + kEmbedRun - 1) / kEmbedRun, units = T * per_row, need = (units + kEmbedWaves - 1) / kEmbedWaves;
  const dim3 grid((unsigned)(need < kMaxGrid ? need : kMaxGrid)), block(kEmbedWaves * 64);
  const int vec = y_stride * (type == BQM_F32 ? 4 : 2) % 16 == 0;
#define BQM_EMBED(TYPE)                                                                                                  \
  hipLaunchKernelGGL((k_embed<FMT, TYPE>), grid, block, 0, s, w, scales_off, rows, K, ks, kg, ids, units, (int)per_row, scale, \
                     static_cast<mx::Elem<TYPE>::T*>(Y), y_stride, vec)
  if (type == BQM_F32)
    BQM_EMBED(BQM_F32);
  else if (type == BQM_F16)
    BQM_EMBED(BQM_F16);
  else
    BQM_EMBED(BQM_BF16);
#undef BQM_EMBED
  return launch_status();
}

}  // namespace

int launch_embed(int fmt, const void* w, int64_t rows, int64_t K, const int32_t* ids, int64_t T, float scale, int y_type, void* Y,
                 int64_t y_stride, hipStream_t s) {
  const uint8_t* wc = static_cast<const uint8_t*>(w);
  if (fmt == BQM_MXFP4) {
    const MxLayout L = mx_layout(rows, K);
    return launch_embed_of<BQM_MXFP4>(wc, L.scales_off, rows, K, L.ks, L.kg, ids, T, scale, y_type, Y, y_stride, s);
  }
  Layout L;
  layout_of(fmt, rows, K, &L);
  return fmt == BQM_Q4_0 ? launch_embed_of<BQM_Q4_0>(wc, L.scales_off, rows, K, 0, 0, ids, T, scale, y_type, Y, y_stride, s)
                         : launch_embed_of<BQM_Q8_0>(wc, L.scales_off, rows, K, 0, 0, ids, T, scale, y_type, Y, y_stride, s);
}

}  // namespace bqm
