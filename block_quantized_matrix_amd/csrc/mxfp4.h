// The MXFP4 format on the device, gfx950: packed layout, e8m0 scales, conversions (included by
// the sources that read or write it).
//
// A block is 32 e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) under one e8m0
// scale 2^(byte - 127), byte 255 standing for NaN.  gfx950 multiplies such blocks as they are:
// in v_mfma_scale_f32_16x16x128_f8f6f4 each lane holds the 32 codes of one block (16 bytes;
// lane l: row l % 16, block l / 16 of the four that the instruction covers) and its scale in a
// byte of a register.  The packed layout is made of that instruction's operands:
//
//   codes   [row tile of 16][step of 128 k][block in step][row][16 bytes]: an operand is 1024
//           contiguous bytes in lane order, one load of 16 bytes per lane
//   scales  [row tile of 16][four steps][block in step][row][step]: one 4-byte word per lane
//           holds the scales of four steps, which the instruction picks its byte from
//
// (With a row's four blocks next to each other, 64 bytes, the lanes of a load are 64 bytes apart
// and a wave's 1024 bytes take the address unit four times as long.)
// The order of the codes inside a block is the interchange one (byte j: code j low, code
// j + 16 high); a dot product of two such blocks does not depend on it.  Rows are padded to 16,
// K to 128 in the codes and to 512 in the scales, with codes 0 and scales 1.
#pragma once

#include "bqm_internal.h"

namespace bqm {
namespace mx {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kTileRows = 16;       // rows of an operand
constexpr int kStepK = 128;         // k of an operand
constexpr int kOperand = 1024;      // its code bytes
constexpr int kScaleTile = 256;     // scale bytes of 16 rows and four steps
constexpr uint8_t kOne = 127;       // the scale 1
constexpr uint8_t kNanScale = 255;

__host__ __device__ __forceinline__ int64_t code_at(int64_t row, int64_t b, int64_t ks) {
  return ((row >> 4) * ks + (b >> 2)) * kOperand + (b & 3) * 256 + (row & 15) * 16;
}
__host__ __device__ __forceinline__ int64_t scale_at(int64_t row, int64_t b, int64_t kg) {
  return ((row >> 4) * kg + (b >> 4)) * kScaleTile + (b & 3) * 64 + (row & 15) * 4 + ((b >> 2) & 3);
}

// 2^(byte - 127) as a float (byte 0 is subnormal), NaN for 255
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 255 ? 0x7FC00000u : byte == 0 ? 0x00400000u : byte << 23);
}

// Codes b (low nibble) and b + 16 (high) of word b / 4 of a block, b % 4 = B, times the scale.
template <int B>
__device__ __forceinline__ f32x2 pair_of(uint32_t word, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, scale, B);
}

// Between what a wave writes to LDS and other lanes of it read there, and before the place is
// written again.  (A wave's LDS operations keep their order; this keeps the compiler, which sees one
// lane's addresses, from changing it.)
__device__ __forceinline__ void wave_turn() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Element types of float rows (the codes of bqm_type).
template <int TYPE>
struct Elem;
template <>
struct Elem<BQM_F32> { typedef float T; };
template <>
struct Elem<BQM_F16> { typedef _Float16 T; };
template <>
struct Elem<BQM_BF16> { typedef __bf16 T; };

}  // namespace mx
}  // namespace bqm
