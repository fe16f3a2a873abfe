// The linear layer for many rows (kernel and launcher; included by qmm.hip).  linear.h has the formula.
//
// The matrix cores and the vector unit bind it together: a block of 32 x 32 outputs takes two
// v_mfma_f32_32x32x16 (64 clocks of a SIMD) and 16 FMAs for the block's scale; the codes' conversion
// (15 instructions for eight codes of Q4_0, 12 of Q8_0, 8 of MXFP4 to bf16) comes on top, once for all the row
// tiles of a wave.  A SIMD issues one vector instruction in about 4.3 clocks, a wave alone one in 4.9 and a
// matrix instruction takes some twelve of them, so the widest tile, 64 weight rows by 128 rows a wave, two waves
// a SIMD, cannot pass 60 % of the matrix rate; it reaches 0.86 PFLOP/s (4096 x 17408 x 5120, Q4_0 and Q8_0, 850
// us; fp16 0.92), with MXFP4's scales folded into the conversion 1.3 (562 us).
#pragma once

#include "linear.h"
#include "mxfp4_qmm.h"

namespace bqm {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// NW waves side by side along the weight rows (TN tiles of 32 each), all over the same TM tiles of 32 rows.  K
// advances by steps of two blocks.  The rows go from memory straight into LDS, four stages, some two steps
// ahead; codes straight to the registers of the wave that converts them, one to two steps ahead; scales by way
// of LDS of the wave's own, four steps at a time (asked for at every step they were a third of what L2 delivered).
template <int FMT, int XT, int NW, int TN, int TM>
struct LinTile {
  static constexpr int kWaves = NW, kBN = kWaves * TN * 32, kBM = TM * 32;
  static constexpr int kXB = lin::type_size(XT), kRow = 64 * kXB;  // bytes of a row's step
  static constexpr int kStage = kBM * kRow, kRoom = kStage > NW * TN * 1024 ? kStage : NW * TN * 1024,  // LDS of a stage
                        kPieces = (kStage / 1024 + kWaves - 1) / kWaves;
  static constexpr int kLoads = FMT == BQM_Q8_0 ? 2 : 1;           // of 16 bytes a lane, of a weight tile's step
  static_assert(TN <= 2, "a lane for each of a wave's rows");
  static_assert(kStage % 1024 == 0, "whole loads");
};

// The sums of a workgroup's tile.  FOLD (MXFP4 beside bf16): the block's scale goes into the codes' conversion,
// exact for scales up to 2^125, and products add to the sums at once; else an FMA applies it to a block's sum.
template <bool FOLD, int FMT, int XT, int NW, int TN, int TM>
__device__ __forceinline__ void lin_sums(const lin::Args& a, const lin::RowTile& at, int tn, uint8_t* lds0, uint8_t* lds1, uint8_t* lds2,
                                         uint8_t* lds3, uint8_t* scales, f32x16 (&acc)[TN][TM]) {
  using namespace lin;
  using C = LinTile<FMT, XT, NW, TN, TM>;
  constexpr int P = parts_of(XT), L = C::kLoads, PX = C::kPieces;
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
  const __amdgpu_buffer_rsrc_t rd = rsrc(wd, MX ? span * a.kg * mx::kScaleTile : (int64_t)own * nb * 2 + 14);  // sixteen bytes at the last scale
  // Loads past the last again take what the last one takes (a branch around a load would make the compiler
  // wait for all loads where the paths join).
  uint32_t oc[TN];
#pragma unroll
  for (int t = 0; t < TN; t++) {
    const int r = t * 32 + i < own ? t * 32 + i : own - 1;
    oc[t] = MX ? (uint32_t)mx::code_at((first & 15) + r, h, a.ks) : (uint32_t)(r * nb * CB + h * 16);
  }
  u32x4 code[2][TN];  // of two blocks of Q8_0 each, two steps of the others
  auto load_codes = [&](int d, int u) {
    const int most = L == 2 ? nb - 1 : steps - 1;
    u = u < most ? u : most;
    const int at = MX ? (u >> 1) * mx::kOperand + (u & 1) * 512 : u * 32;
#pragma unroll
    for (int t = 0; t < TN; t++) code[d][t] = __builtin_amdgcn_raw_buffer_load_b128(rc, oc[t], at, 0);
  };
  // Scales: lane l brings those of row l and four steps (16 bytes) to LDS of the wave's own.
  uint32_t od;
  {
    const int r = lane < own ? lane : own - 1, mr = (int)(first & 15) + r;
    od = MX ? (uint32_t)((mr >> 4) * a.kg * mx::kScaleTile + (mr & 15) * 4) : (uint32_t)(r * nb * 2);
  }
  u32x4 fresh;
  auto load_scales = [&](int g) {  // of steps 4 g .. 4 g + 3
    if constexpr (MX) {  // a word: four blocks, four apart
      const int most = (steps - 1) >> 3, at = (g >> 1 < most ? g >> 1 : most) * mx::kScaleTile;
#pragma unroll
      for (int k = 0; k < 4; k++) fresh[k] = __builtin_amdgcn_raw_buffer_load_b32(rd, od + k * 64, at, 0);
    } else {
      const int most = (steps - 1) >> 2;
      fresh = __builtin_amdgcn_raw_buffer_load_b128(rd, od, (g < most ? g : most) * 16, 0);
    }
  };
  uint8_t* sc = scales + wave * 2 * 1024;
  auto keep_scales = [&](int g) { *reinterpret_cast<u32x4*>(sc + (g & 1) * 1024 + lane * 16) = fresh; };
  auto scale_at = [&](int t, int s, int b) {  // of block b of step s
    const uint8_t* p = sc + (s >> 2 & 1) * 1024 + (t * 32 + i) * 16;
    // (as a word: what is read as bytes might be any LDS to the compiler, which then waits for the loads into it)
    if constexpr (MX) return reinterpret_cast<const uint32_t*>(p)[(s & 1) * 2 + b] >> (8 * (s >> 1 & 3)) & 0xFF;
    return (uint32_t)reinterpret_cast<const uint16_t*>(p)[(s & 3) * 2 + b];
  };

  // rows: 16-byte slots, place p of row m holding slot p ^ turned(m): the sixteen lanes that LDS serves
  // at a time, a row apart each, find their slots in all 64 banks
  const __amdgpu_buffer_rsrc_t rx = rsrc(a.x + at.m0 * a.xs, (int64_t)(at.rows - 1) * a.xs + (int64_t)nb * 32 * C::kXB);
  constexpr int kSlots = C::kRow / 16;  // 8, or 16 of fp32
  auto turned = [](int m) { return kSlots == 8 ? m >> 1 & 7 : m & 15; };
  // where the waves do not divide the lots of 1024 bytes, some bring the last one too
  auto lot_of = [&](int p) { return (p + 1) * NW <= C::kStage / 1024 || p * NW + wave < C::kStage / 1024 ? p * NW + wave : C::kStage / 1024 - 1; };
  uint32_t ox[PX];
#pragma unroll
  for (int p = 0; p < PX; p++) {
    const int u = lot_of(p) * 64 + lane, m = u / kSlots, slot = (u % kSlots ^ turned(m)) & (nb > 1 ? kSlots - 1 : kSlots / 2 - 1);
    ox[p] = (uint32_t)((m < at.rows ? m : at.rows - 1) * (int)a.xs + slot * 16);
  }
  // The last step of an odd number of blocks takes the last two (of a single block: that block twice), so that
  // nothing is read past a row.
  auto load_x = [&](int s, uint8_t* stage) {
    s = s < steps ? s : steps - 1;
    const int at = 2 * s + 2 <= nb || nb == 1 ? 2 * s : nb - 2;
#pragma unroll
    for (int p = 0; p < PX; p++)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (LdsPtr)(stage + lot_of(p) * 1024), 16, ox[p], at * (C::kRow / 2), 0, 0);
  };
  auto slot_at = [&](const uint8_t* stage, int t, int slot) {
    return *reinterpret_cast<const u32x4*>(stage + (t * 32 + i) * C::kRow + (slot ^ turned(i)) * 16);
  };

  auto meet = [&] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // Matrix operands of block b of step s from the codes: of each weight tile the two halves of its k.  (The
  // lane halves hold a unit of 16 bytes each.  A unit of Q8_0 is half a block: lanes h take k = 16 h + 8 j ..
  // of half j.  One of nibbles is a block: halves of units are exchanged, then lanes h hold k = 8 h .. of the
  // low nibbles and 16 + 8 h .. of the high ones.)
  auto convert = [&](int b, int d, int t, uint32_t scale, u32x4 (&w)[2], float& f) {
    u32x4& v = code[d][t];
    if constexpr (FMT == BQM_Q8_0) {
#pragma unroll
      for (int j = 0; j < 2; j++) {
        uint32_t u[2][2];
        bytes<XT>(v[2 * j], u[0]);
        bytes<XT>(v[2 * j + 1], u[1]);
        w[j] = u32x4{u[0][0], u[0][1], u[1][0], u[1][1]};
      }
    } else {
      if (b == 0) {
        uint32_t v0 = v[0], v1 = v[1], v2 = v[2], v3 = v[3];
        mma::swap32(v0, v2);
        mma::swap32(v1, v3);
        v = u32x4{v0, v1, v2, v3};
      }
      uint32_t lo[2][2], hi[2][2];
      const float by = FOLD ? __uint_as_float(scale << 23) : 1.0f;  // the conversion goes by the exponent field alone
      nibbles<FMT, XT>(v[2 * b], lo[0], hi[0], by);
      nibbles<FMT, XT>(v[2 * b + 1], lo[1], hi[1], by);
      w[0] = u32x4{lo[0][0], lo[0][1], lo[1][0], lo[1][1]};
      w[1] = u32x4{hi[0][0], hi[0][1], hi[1][0], hi[1][1]};
    }
    f = FOLD ? 1.0f : scale_from<FMT, XT>(scale);
    asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(f));  // here, not where the next block uses them
  };
  auto rows_of = [&](const uint8_t* stage, int m, int b, u32x4 (&x)[2][P]) {
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const int eight = b * 4 + (FMT == BQM_Q8_0 ? h * 2 + j : j * 2 + h);  // of the step's lots of eight k
      if constexpr (P == 1) {
        x[j][0] = slot_at(stage, m, eight);
      } else {
        const u32x4 v0 = slot_at(stage, m, eight * 2), v1 = slot_at(stage, m, eight * 2 + 1);
        float g[8];
#pragma unroll
        for (int e = 0; e < 4; e++) g[e] = __uint_as_float(v0[e]), g[4 + e] = __uint_as_float(v1[e]);
        uint32_t part[3][4];
        three_parts<8>(g, part);
#pragma unroll
        for (int p = 0; p < 3; p++) x[j][p] = u32x4{part[p][0], part[p][1], part[p][2], part[p][3]};
      }
    }
  };
  auto products = [&](const u32x4 (&x)[2][P], const u32x4 (&w)[2], f32x16 sum) {
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int p = 0; p < P; p++) {
        if constexpr (XT == BQM_F16)
          sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x[j][p]), __builtin_bit_cast(f16x8, w[j]), sum, 0, 0, 0);
        else
          sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x[j][p]), __builtin_bit_cast(bf16x8, w[j]), sum, 0, 0, 0);
      }
    return sum;
  };
  auto add_scaled = [&](f32x16& to, const f32x16& sum, float f) {
#pragma unroll
    for (int r = 0; r < 16; r++) to[r] = fmaf(f, sum[r], to[r]);
  };
  // Blocks in a pipeline: beside a pair of tiles' products stand the scaling of the pair before, the reading of
  // the next rows as soon as the last product has taken these, and likewise the conversion of the next block.
  constexpr int K = TM * TN;
  u32x4 w[TN][2], x[2][P];
  float f[TN], f_last;
  f32x16 sum[2];  // in turn, from block 0 to block 1 too
  auto block = [&](auto bc, int s, int next_d, const uint8_t* stage, const uint8_t* next_stage, auto&& between) {
    constexpr int B = decltype(bc)::value;
    float g[TN];
    uint32_t bits[TN];
#pragma unroll
    for (int k = 0; k < K; k++) {
      const int m = k / TN, t = k % TN;
      if (k == (K - 1) / 2) between();
      if constexpr (FOLD)
        acc[t][m] = products(x, w[t], acc[t][m]);
      else
        sum[(k + B * K) & 1] = products(x, w[t], f32x16{});
      if (t == TN - 1) {
        if (m + 1 < TM)
          rows_of(stage, m + 1, B, x);
        else
          rows_of(next_stage, 0, B ^ 1, x);
      }
      if constexpr (!FOLD) {
        if (k > 0)
          add_scaled(acc[(k - 1) % TN][(k - 1) / TN], sum[(k - 1 + B * K) & 1], f[(k - 1) % TN]);
        else if (B == 1)
          add_scaled(acc[TN - 1][TM - 1], sum[(K - 1) & 1], f_last);
      }
      if (m == (TM > 1 ? TM - 2 : 0)) bits[t] = scale_at(t, B ? s + 1 : s, B ^ 1);
      if (m == TM - 1) convert(B ^ 1, next_d, t, bits[t], w[t], g[t]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (B == 1 && !FOLD) add_scaled(acc[TN - 1][TM - 1], sum[(K - 1 + B * K) & 1], f[TN - 1]);
    f_last = f[TN - 1];
#pragma unroll
    for (int t = 0; t < TN; t++) f[t] = g[t];
  };
  // The Q-th step of four; whole steps, both blocks.  TAIL: one of the last, behind the whole fours.
  auto step = [&](auto qc, auto tail, int s, const uint8_t* cur, const uint8_t* nxt, uint8_t* free) {
    constexpr int Q = decltype(qc)::value, d = Q & 1;
    constexpr bool TAIL = decltype(tail)::value;
    // codes: block 0 converts block 1 of this step, block 1 block 0 of the next
    if constexpr (L == 2) {
      load_codes(0, 2 * s + 2);
      __builtin_amdgcn_sched_barrier(0);
    }
    block(std::integral_constant<int, 0>{}, s, L == 2 ? 1 : d, cur, cur, [] {});
    load_codes(L == 2 ? 1 : d, L == 2 ? 2 * s + 3 : s + 2);
    if constexpr (Q == 0 && !TAIL) load_scales((s >> 2) + 1);
    if constexpr (Q == 3) {  // the next step's are asked for in the block that follows
      keep_scales((s >> 2) + 1);
      mx::wave_turn();
    }
    __builtin_amdgcn_sched_barrier(0);
    block(std::integral_constant<int, 1>{}, s, L == 2 ? 0 : d ^ 1, cur, nxt, [&] {
      // The rows of step s + 1 have arrived (after them came those of step s + 2, the codes of two blocks of
      // nibbles or four of bytes, and the scales of every fourth step), and every wave has read all of step s - 1.
      // A tail counts the rows of step s + 2 alone: the compiler leaves out what it loads for steps that never come.
      vm_wait<TAIL ? PX : PX + (L == 2 ? 4 : 2) * TN + (Q <= 1 ? (MX ? 4 : 1) : 0)>();
      meet();
      load_x(s + 3, free);
      __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_sched_barrier(0);
  };
  const int whole = nb >> 1;
  if (steps > 0) {
    load_scales(0);
    load_codes(0, 0);
    load_codes(1, 1);
    __builtin_amdgcn_sched_barrier(0);
    load_x(0, lds0);
    load_x(1, lds1);
    load_x(2, lds2);
    keep_scales(0);
    mx::wave_turn();
    vm_wait<0>();
    meet();
    rows_of(lds0, 0, 0, x);
#pragma unroll
    for (int t = 0; t < TN; t++) convert(0, 0, t, scale_at(t, 0, 0), w[t], f[t]);
    __builtin_amdgcn_sched_barrier(0);
    int s = 0;  // (left in one place only: exits from each step had the sums copied, and spilled)
    for (; s + 4 <= whole; s += 4) {
      step(std::integral_constant<int, 0>{}, std::false_type{}, s, lds0, lds1, lds3);
      step(std::integral_constant<int, 1>{}, std::false_type{}, s + 1, lds1, lds2, lds0);
      step(std::integral_constant<int, 2>{}, std::false_type{}, s + 2, lds2, lds3, lds1);
      step(std::integral_constant<int, 3>{}, std::false_type{}, s + 3, lds3, lds0, lds2);
    }
    if (s < whole) step(std::integral_constant<int, 0>{}, std::true_type{}, s, lds0, lds1, lds3);
    if (s + 1 < whole) step(std::integral_constant<int, 1>{}, std::true_type{}, s + 1, lds1, lds2, lds0);
    if (s + 2 < whole) step(std::integral_constant<int, 2>{}, std::true_type{}, s + 2, lds2, lds3, lds1);
    if (nb & 1) {  // a last block without a partner, its codes already at hand
      const uint8_t* stage = (whole & 3) == 0 ? lds0 : (whole & 3) == 1 ? lds1 : (whole & 3) == 2 ? lds2 : lds3;
#pragma unroll
      for (int m = 0; m < TM; m++) {
        rows_of(stage, m, nb > 1, x);
#pragma unroll
        for (int t = 0; t < TN; t++) {
          if constexpr (FOLD)
            acc[t][m] = products(x, w[t], acc[t][m]);
          else
            add_scaled(acc[t][m], products(x, w[t], f32x16{}), f[t]);
        }
      }
    }
  }
  vm_wait<0>();  // nothing may be on its way into LDS when it is used again
  __syncthreads();
}

template <int FMT, int XT, int NW, int TN, int TM>
__device__ __forceinline__ void lin_core(const lin::Args& a, const lin::RowTile& at, int tn, uint8_t* lds0, uint8_t* lds1, uint8_t* lds2,
                                         uint8_t* lds3, uint8_t* scales) {
  using namespace lin;
  using C = LinTile<FMT, XT, NW, TN, TM>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 31, h = lane >> 5;
  const int64_t n0 = (int64_t)tn * C::kBN + wave * TN * 32;
  constexpr bool FOLD = FMT == BQM_MXFP4 && XT != BQM_F16;
  f32x16 acc[TN][TM] = {};
  lin_sums<FOLD, FMT, XT, NW, TN, TM>(a, at, tn, lds0, lds1, lds2, lds3, scales, acc);
  if constexpr (FOLD) {
    // Scales beyond 2^125, whose largest weights bf16 does not hold, and the scale NaN leave sums that are not
    // numbers, as such inputs do: these tiles are made again with the scales apart.
    float probe = 0;
#pragma unroll
    for (int t = 0; t < TN; t++)
#pragma unroll
      for (int m = 0; m < TM; m++)
#pragma unroll
        for (int r = 0; r < 16; r++) probe = fmaf(acc[t][m][r], 0.0f, probe);  // NaN if any is not finite
    if (__builtin_expect(__syncthreads_or(probe != probe), 0)) {
#pragma unroll
      for (int t = 0; t < TN; t++)
#pragma unroll
        for (int m = 0; m < TM; m++) acc[t][m] = f32x16{};
      lin_sums<false, FMT, XT, NW, TN, TM>(a, at, tn, lds0, lds1, lds2, lds3, scales, acc);
    }
  }
  // A lane holds column i of a weight tile, rows 8 (r / 4) + 4 h + r % 4 of a row tile.  Each wave turns its row
  // tiles in a stage of its own, so that it stores whole runs of a row of Y.
  constexpr int kCols = TN * 32, kTurn = 32 * kCols * 4;
  constexpr int kRoom = C::kRoom / (((NW + 3) / 4) * kTurn), kOnce = kRoom >= TM ? TM : kRoom >= TM / 2 && TM % 2 == 0 ? TM / 2 : 1;  // row tiles turned at a time
  constexpr int kShare = (NW + 3) / 4;  // waves that share a stage
  static_assert(kOnce > 0 && TM % kOnce == 0 && kOnce * kTurn * kShare <= C::kRoom, "the waves' tiles fit the stages");
  uint8_t* stage = wave < kShare ? lds0 : wave < 2 * kShare ? lds1 : wave < 3 * kShare ? lds2 : lds3;
  float* turn = reinterpret_cast<float*>(stage + wave % kShare * kOnce * kTurn);
  const float* bias = a.bias ? a.bias + at.e * a.N : nullptr;
  const bool fours = by_fours(a);
  constexpr int kWide = kCols / 4, kRows = 64 / kWide, R = 4;  // lanes along a row, rows at a time, those of a turn
  const int c = lane % kWide * 4;
  const int64_t n = n0 + c;
  f32x4 b4{};
  if (bias)
#pragma unroll
    for (int j = 0; j < 4; j++) b4[j] = n + j < a.N ? bias[n + j] : 0.0f;
#pragma unroll
  for (int m0 = 0; m0 < TM; m0 += kOnce) {
#pragma unroll
    for (int m = 0; m < kOnce; m++)
#pragma unroll
      for (int t = 0; t < TN; t++)
#pragma unroll
        for (int r = 0; r < 16; r++) turn[(m * 32 + 8 * (r >> 2) + 4 * h + (r & 3)) * kCols + t * 32 + i] = acc[t][m0 + m][r];
    mx::wave_turn();
    const int rows = at.rows - m0 * 32 < kOnce * 32 ? at.rows - m0 * 32 : kOnce * 32;
    const int64_t y0 = at.m0 + m0 * 32;
    if (fours) {
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += R * kRows) {
        f32x4 z[R];
#pragma unroll
        for (int r = 0; r < R; r++) z[r] = *reinterpret_cast<const f32x4*>(turn + (r0 + r * kRows + lane / kWide) * kCols + c);
        if (n + 4 <= a.N) {
          finish4<R>(a, b4, y0 + r0 + lane / kWide, kRows, y0 + rows, n, z);
        } else if (n < a.N) {
#pragma unroll 1
          for (int k = 0; k < R * 4; k++) {
            const int row = r0 + (k >> 2) * kRows + lane / kWide;
            if (row < rows && n + (k & 3) < a.N)
              store_as(a.y, (y0 + row) * a.ys + n + (k & 3), finish(a, bias, y0 + row, n + (k & 3), turn[row * kCols + c + (k & 3)]), a.y_type);
          }
        }
      }
    } else {
#pragma unroll 1
      for (int o = lane; o < rows * kCols; o += 64) {
        const int64_t y = y0 + o / kCols, col = n0 + o % kCols;
        if (col < a.N) store_as(a.y, y * a.ys + col, finish(a, bias, y, col, turn[o]), a.y_type);
      }
    }
    mx::wave_turn();
  }
}

template <int FMT, int XT, int NW, int TN, int TM, int OCC>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(OCC, OCC))) void k_linear_tiles(lin::Args a, int tiles_m, int tiles_n) {
  using namespace lin;
  using C = LinTile<FMT, XT, NW, TN, TM>;
  __shared__ __attribute__((aligned(16))) uint8_t lds0[C::kRoom];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[C::kRoom];
  __shared__ __attribute__((aligned(16))) uint8_t lds2[C::kRoom];
  __shared__ __attribute__((aligned(16))) uint8_t lds3[C::kRoom];
  __shared__ __attribute__((aligned(16))) uint8_t scales[NW * 2 * 1024];  // a wave's, twice
  __shared__ int room[RowTiles<NW * 64, C::kBM>::kRoom];
  RowTiles<NW * 64, C::kBM> groups(a, room);
  int tm, tn;
  if (a.offsets) {  // row tiles go round the XCDs (as workgroups do), each with all its columns: its rows come to one L2 only
    const int nth = blockIdx.x >> 3, turn = nth / tiles_n;
    tm = turn * 8 + (blockIdx.x & 7), tn = nth - turn * tiles_n;
    if (tm >= groups.all) return;  // the whole workgroup
  } else {
    const MxPlace at = mx_place(blockIdx.x, tiles_m, tiles_n);
    tm = at.m, tn = at.n;
  }
  const RowTile at = groups.find(tm);
  if (at.rows <= 0) return;
  // a tile of few rows (the last of a group) as one of a lower height
  if (TM > 1 && at.rows <= 32)
    lin_core<FMT, XT, NW, TN, 1>(a, at, tn, lds0, lds1, lds2, lds3, scales);
  else if (TM > 2 && at.rows <= 64)
    lin_core<FMT, XT, NW, TN, 2>(a, at, tn, lds0, lds1, lds2, lds3, scales);
  else
    lin_core<FMT, XT, NW, TN, TM>(a, at, tn, lds0, lds1, lds2, lds3, scales);
}

// Workgroups of a call by tiles of bn weight rows and bm rows.
int64_t lin_grid(bool grouped, int64_t R, int64_t N, int64_t groups, int64_t bn, int64_t bm) {
  const int64_t tm = lin::most_tiles(grouped, R, groups, bm);
  return (grouped ? (tm + 7) / 8 * 8 : tm) * ((N + bn - 1) / bn);
}
template <int FMT, int XT, int NW, int TN, int TM, int OCC>
int launch_tiles_as(const lin::Args& a, int64_t groups, hipStream_t s) {
  using C = LinTile<FMT, XT, NW, TN, TM>;
  const int64_t tm = lin::most_tiles(a, groups, C::kBM), tn = (a.N + C::kBN - 1) / C::kBN;
  const int64_t grid = lin_grid(a.offsets != nullptr, a.R, a.N, groups, C::kBN, C::kBM);
  if (grid > kMaxGrid) return BQM_E_SHAPE;
  hipLaunchKernelGGL((k_linear_tiles<FMT, XT, NW, TN, TM, OCC>), dim3((unsigned)grid), dim3(NW * 64), 0, s, a, (int)tm, (int)tn);
  return launch_status();
}
// The tiles: weight tiles and row tiles of 32 a wave, workgroups that a unit holds at most, and the time of a
// step (us; 64 of K) where it holds one, two, ... of them, measured with N = 17408 and K = 5120, weights from
// memory.  (fp32 rows take four times the LDS of the others' step, so their tiles are lower.)  Q4_0's serve MXFP4 beside
// fp16, whose scales are not folded, and one table fp32 rows of every format: the tile that they choose is within 8 % of
// the best (17408 x 5120, MXFP4 beside fp16: 128 rows 59 us and 55, 512 rows 144 and 135, 4096 rows 794 and 764; fp32 rows:
// 128 rows of Q8_0 167 and 160, 512 rows of each format the best).
struct LinChoice {
  int tn, tm, resident;
  float step[4];
};
constexpr int kLinTiles = 5, kLinTiles32 = 2;
constexpr LinChoice kLinQ4[kLinTiles] = {{1, 1, 4, {0.46f, 0.61f, 0.85f, 0.95f}}, {1, 2, 3, {0.58f, 0.80f, 1.08f}}, {1, 3, 2, {0.68f, 0.95f}},
                                         {1, 4, 2, {0.81f, 1.17f}}, {2, 4, 2, {1.45f, 2.05f}}};
constexpr LinChoice kLinQ8[kLinTiles] = {{1, 1, 4, {0.68f, 0.98f, 1.28f, 1.32f}}, {1, 2, 3, {0.75f, 1.08f, 1.47f}}, {1, 3, 2, {0.80f, 1.10f}},
                                         {1, 4, 2, {0.87f, 1.36f}}, {2, 4, 2, {1.53f, 2.15f}}};
constexpr LinChoice kLinMx[kLinTiles] = {{1, 1, 4, {0.38f, 0.43f, 0.55f, 0.60f}}, {1, 2, 3, {0.42f, 0.54f, 0.76f}}, {1, 3, 2, {0.50f, 0.67f}},
                                         {1, 4, 2, {0.57f, 0.83f}}, {2, 4, 2, {0.93f, 1.37f}}};
constexpr LinChoice kLin32[kLinTiles32] = {{1, 1, 3, {0.92f, 1.35f, 1.85f}}, {2, 2, 2, {2.03f, 2.90f}}};

const LinChoice* lin_table(int fmt, int x_type) {
  return x_type == BQM_F32 ? kLin32 : fmt == BQM_Q8_0 ? kLinQ8 : fmt == BQM_MXFP4 && x_type == BQM_BF16 ? kLinMx : kLinQ4;
}

template <int FMT, int XT>
int launch_tiles_of(const lin::Args& a, int64_t groups, int choice, hipStream_t s) {
  if constexpr (XT == BQM_F32)
    return choice == 0 ? launch_tiles_as<FMT, XT, 4, 1, 1, 3>(a, groups, s) : launch_tiles_as<FMT, XT, 4, 2, 2, 2>(a, groups, s);
  else
    return choice == 0 ? launch_tiles_as<FMT, XT, 4, 1, 1, 4>(a, groups, s)
           : choice == 1 ? launch_tiles_as<FMT, XT, 4, 1, 2, 3>(a, groups, s)
           : choice == 2 ? launch_tiles_as<FMT, XT, 4, 1, 3, 2>(a, groups, s)
           : choice == 3 ? launch_tiles_as<FMT, XT, 4, 1, 4, 2>(a, groups, s)
                         : launch_tiles_as<FMT, XT, 4, 2, 4, 2>(a, groups, s);
}

}  // namespace

// The index of the tile.  One matrix: the least time by the table, in rounds of workgroups on 256 units and 4 us
// for each.  Groups, of whose lengths the host knows only the mean, are short and long beside each other (their
// short ends run as lower tiles): by the mean, and lower where that leaves units without work.  128 experts of
// 1536 x 4096, skewed, us with the lowest tile, with three row tiles and with the widest:
//     mean    Q4_0             Q8_0             MXFP4
//        4    67,  71,  82     106, 126, 123    44,  55,  49
//       10    108, 93,  101    177, 141, 143    74,  70,  74
//       32    193, 156, 169    303, 215, 202    121, 116, 109
//      256                     -,   782, 683    -,   502, 412
// (The tests ask too: they have to run every tile.)
extern "C" int bqm_internal_linear_choice(int fmt, int x_type, int grouped, int64_t R, int64_t N, int64_t K, int64_t groups) {
  const bool wide = x_type == BQM_F32;
  const LinChoice* table = lin_table(fmt, x_type);
  auto workgroups = [&](int c) {
    const int64_t bm = table[c].tm * 32, bn = table[c].tn * 128;
    return lin::most_tiles(grouped, R, groups, bm) * ((N + bn - 1) / bn);
  };
  if (grouped) {
    const int64_t mean = R / (groups > 0 ? groups : 1);
    int c = wide ? mean > 16 : mean <= 6 ? 0 : mean < 24 ? 2 : 4;
    while (c > 0 && workgroups(c) < 256) c--;
    return c;
  }
  int best = 0;
  double least = 0;
  for (int c = 0; c < (wide ? kLinTiles32 : kLinTiles); c++) {
    const LinChoice& t = table[c];
    const int64_t wgs = workgroups(c), round = 256 * t.resident, full = wgs / round, left = wgs % round;
    // (units that are done early start on the last round before the others end the one before)
    const double step = full * t.step[t.resident - 1] + (left ? t.step[(left - 1) / 256] * (full ? 0.85f : 1.0f) : 0.0f);
    const double time = (double)((K + 63) / 64) * step + 4.0 * (full + (left > 0));
    if (c == 0 || time < least) best = c, least = time;
  }
  return best;
}

int64_t linear_tiles_grid(int fmt, int x_type, bool grouped, int64_t R, int64_t N, int64_t K, int64_t groups) {
  const LinChoice& t = lin_table(fmt, x_type)[bqm_internal_linear_choice(fmt, x_type, grouped, R, N, K, groups)];
  return lin_grid(grouped, R, N, groups, t.tn * 128, t.tm * 32);
}

int launch_linear_tiles(int fmt, int x_type, const lin::Args& a, int64_t groups, hipStream_t s) {
  const int c = bqm_internal_linear_choice(fmt, x_type, a.offsets != nullptr, a.R, a.N, (int64_t)a.nb * kQK, groups);
#define BQM_TILES(FMT)                                                      \
  return x_type == BQM_F32   ? launch_tiles_of<FMT, BQM_F32>(a, groups, c, s) \
         : x_type == BQM_F16 ? launch_tiles_of<FMT, BQM_F16>(a, groups, c, s) \
                             : launch_tiles_of<FMT, BQM_BF16>(a, groups, c, s)
  if (fmt == BQM_Q4_0) BQM_TILES(BQM_Q4_0);
  if (fmt == BQM_Q8_0) BQM_TILES(BQM_Q8_0);
  BQM_TILES(BQM_MXFP4);
#undef BQM_TILES
}

}  // namespace bqm
