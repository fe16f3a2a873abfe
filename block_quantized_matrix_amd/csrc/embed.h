// Rows of a packed table by token id (kernel and launcher; included by repack.hip):
//   Y[t][k] = scale * dequant(W)[ids[t]][k]
//
// Bound by the bytes that it writes.  A wave takes runs of 512 numbers of a row, a lane eight on end of each: a
// store of theirs covers whole lines, and the four lanes of a block read its scale and codes from one line.
// The loads of its U runs go out together: each is a trip to memory behind that of the id; and the many rows of
// such calls are stored past the caches, which would hold them at the cost of writing back others (16384 x 5120
// of Q4_0 to bf16, outputs in turn: a run a wave 77 us, four 56, stored past 41; a fill of the output takes 27).
#pragma once

#include "mxfp4.h"

namespace bqm {
namespace {

constexpr int kEmbedWaves = 4, kEmbedRun = 512;

struct EmbedArgs {
  const uint8_t* w;
  const int32_t* ids;
  int64_t scales_off, rows, K, ks, kg, units, y_stride;
  int per_row;  // units of a row
  float scale;  // the call's, times 2^-shift
  int shift;    // 0 but beside MXFP4
  int vec;      // rows of Y start at multiples of 16 bytes
};

template <int FMT, int TYPE, int U>
__global__ __launch_bounds__(kEmbedWaves * 64) void k_embed(EmbedArgs a, typename mx::Elem<TYPE>::T* __restrict__ Y) {
  typedef typename mx::Elem<TYPE>::T T;
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const int lane = threadIdx.x & 63;
  for (int64_t unit = (int64_t)blockIdx.x * kEmbedWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); unit < a.units;
       unit += (int64_t)gridDim.x * kEmbedWaves) {
    const int64_t t = unit / a.per_row, k0 = (unit - t * a.per_row) * (kEmbedRun * U) + lane * 8;
    const int64_t id = a.ids[t];
    const bool inside = id >= 0 && id < a.rows;
    uint32_t code[U][2], bits[U];
#pragma unroll
    for (int r = 0; r < U; r++) {
      const int64_t k = k0 + r * kEmbedRun, b = k >> 5, at = id * (a.K >> 5) + b;
      const int c = (int)(k >> 3) & 3;  // the lane's eight of the block
      if (!inside || k >= a.K) continue;
      if constexpr (FMT == BQM_Q8_0)
        __builtin_memcpy(code[r], __builtin_assume_aligned(a.w + at * 32 + c * 8, 8), 8);
      else if constexpr (FMT == BQM_Q4_0)
        __builtin_memcpy(code[r], __builtin_assume_aligned(a.w + at * 16 + (c & 1) * 8, 8), 8);
      else
        __builtin_memcpy(code[r], __builtin_assume_aligned(a.w + mx::code_at(id, b, a.ks) + (c & 1) * 8, 8), 8);
      bits[r] = FMT == BQM_MXFP4 ? a.w[a.scales_off + mx::scale_at(id, b, a.kg)] : reinterpret_cast<const uint16_t*>(a.w + a.scales_off)[at];
    }
#pragma unroll
    for (int r = 0; r < U; r++) {
      const int64_t k = k0 + r * kEmbedRun;
      const int c = (int)(k >> 3) & 3;
      if (k >= a.K) continue;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; j++) f[j] = id < 0 ? 0.0f : __builtin_nanf("");
      if (inside) {
        if constexpr (FMT == BQM_MXFP4) {
#pragma unroll
          for (int h = 0; h < 2; h++) {
            const uint32_t v = code[r][h] >> (c & 2 ? 4 : 0);
            const float g[4] = {mx::pair_of<0>(v, 1.0f).x, mx::pair_of<1>(v, 1.0f).x, mx::pair_of<2>(v, 1.0f).x, mx::pair_of<3>(v, 1.0f).x};
            // the powers of two last: the product counts as it is where the weight or the scale alone is far from 1
#pragma unroll
            for (int j = 0; j < 4; j++)
              f[h * 4 + j] = bits[r] == mx::kNanScale ? __builtin_nanf("") : ldexpf(g[j] * a.scale, (int)bits[r] - 127 + a.shift);
          }
        } else {
          const float d = (float)__builtin_bit_cast(_Float16, (uint16_t)bits[r]);
#pragma unroll
          for (int j = 0; j < 8; j++) {
            const uint32_t v = code[r][j >> 2] >> (8 * (j & 3));
            const int n = FMT == BQM_Q8_0 ? (int)(int8_t)v : (int)(v >> (c & 2 ? 4 : 0) & 15) - 8;
            f[j] = (float)n * d * a.scale;  // the first product is exact
          }
        }
      }
      T* y = Y + t * a.y_stride + k;
      T o[8];
#pragma unroll
      for (int j = 0; j < 8; j++) o[j] = (T)f[j];
      if (a.vec) {
        u32x4 v[sizeof(o) / 16];
        __builtin_memcpy(v, o, sizeof(o));
#pragma unroll
        for (int q = 0; q < (int)(sizeof(o) / 16); q++) {
          if (U > 1)
            __builtin_nontemporal_store(v[q], reinterpret_cast<u32x4*>(y) + q);
          else
            reinterpret_cast<u32x4*>(y)[q] = v[q];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = o[j];
      }
    }
  }
}

template <int FMT, int TYPE>
int launch_embed_as(EmbedArgs a, int64_t T, void* Y, hipStream_t s) {
  const int64_t runs = (a.K + kEmbedRun - 1) / kEmbedRun;
  const bool many = T * runs >= 16384;  // where the units have waves enough with four runs each
  a.per_row = (int)(many ? (runs + 3) / 4 : runs);
  a.units = T * a.per_row;
  const int64_t need = (a.units + kEmbedWaves - 1) / kEmbedWaves;
  const dim3 grid((unsigned)(need < kMaxGrid ? need : kMaxGrid)), block(kEmbedWaves * 64);
  auto* y = static_cast<typename mx::Elem<TYPE>::T*>(Y);
  if (many)
    hipLaunchKernelGGL((k_embed<FMT, TYPE, 4>), grid, block, 0, s, a, y);
  else
    hipLaunchKernelGGL((k_embed<FMT, TYPE, 1>), grid, block, 0, s, a, y);
  return launch_status();
}
template <int FMT>
int launch_embed_of(const EmbedArgs& a, int64_t T, int type, void* Y, hipStream_t s) {
  return type == BQM_F32   ? launch_embed_as<FMT, BQM_F32>(a, T, Y, s)
         : type == BQM_F16 ? launch_embed_as<FMT, BQM_F16>(a, T, Y, s)
                           : launch_embed_as<FMT, BQM_BF16>(a, T, Y, s);
}

}  // namespace

int launch_embed(int fmt, const void* w, int64_t rows, int64_t K, const int32_t* ids, int64_t T, float scale, int y_type, void* Y,
                 int64_t y_stride, hipStream_t s) {
  EmbedArgs a{static_cast<const uint8_t*>(w), ids, 0, rows, K, 0, 0, 0, y_stride, 0, scale, 0, y_stride * (y_type == BQM_F32 ? 4 : 2) % 16 == 0};
  if (fmt == BQM_MXFP4) {
    const MxLayout L = mx_layout(rows, K);
    a.scales_off = L.scales_off, a.ks = L.ks, a.kg = L.kg;
    if (__builtin_isfinite(scale)) a.scale = frexpf(scale, &a.shift);  // 0.5 to 1 in magnitude, or 0
    return launch_embed_of<BQM_MXFP4>(a, T, y_type, Y, s);
  }
  Layout L;
  layout_of(fmt, rows, K, &L);
  a.scales_off = L.scales_off;
  return fmt == BQM_Q4_0 ? launch_embed_of<BQM_Q4_0>(a, T, y_type, Y, s) : launch_embed_of<BQM_Q8_0>(a, T, y_type, Y, s);
}

}  // namespace bqm
