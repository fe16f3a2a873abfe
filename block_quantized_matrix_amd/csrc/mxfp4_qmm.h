// Products of two packed MXFP4 matrices, dense and expert-indexed (kernels and launchers;
// included by qmm.hip):
//   Y[m][n] = sum_k w[n][k] x[m][k]
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies the blocks as they are stored: products of
// codes are exact, block scales only move their exponents, sums are fp32.
#pragma once

#include <type_traits>

#include "mxfp4.h"

namespace bqm {
namespace {

typedef mx::f32x4 MxAcc;

template <int J>  // the step of its group of four: the byte of the scale words
__device__ __forceinline__ MxAcc mx_mfma(const mx::i32x4& a, const mx::i32x4& b, MxAcc c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx::i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                          mx::i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, 4, 4, J, sa, J, sb);
}

// ---- tiled product ----
// A workgroup computes (WN TN 16) x (WM TM 16) outputs with KS groups of WN x WM waves, each group
// over its share of K, each wave TN x TM MFMA tiles: weights are the MFMA's rows (n), activations its
// columns (m).
template <int WN, int WM, int TN, int TM, int KS>
struct MxTile {
  static constexpr int kGroup = WN * WM, kThreads = kGroup * KS * 64;
  static constexpr int kRT = WN * TN, kCT = WM * TM;         // operand tiles of a step: weights, activations
  static constexpr int kBN = kRT * 16, kBM = kCT * 16;
  static constexpr int kStage = (kRT + kCT) * mx::kOperand;  // LDS bytes of a group's stage
  static constexpr int kPieces = (kRT + kCT) / kGroup;       // operand tiles that a wave copies per step
  static_assert((kRT + kCT) % kGroup == 0 && kRT % kGroup == 0, "whole operands per wave");
  static_assert(TN % 2 == 0, "a step has two halves");
};

// An operand matrix as a workgroup reads it: buffer descriptors that start at a row tile, so that
// lane offsets fit 32 bits and the step's offset is a scalar.
struct MxOperand {
  __amdgpu_buffer_rsrc_t codes, scales;
};
__device__ __forceinline__ MxOperand mx_operand(const uint8_t* base, int64_t scales_off, int64_t tile, int64_t tiles, int ks, int kg) {
  const int64_t c = (tiles - tile) * ks * mx::kOperand, g = (tiles - tile) * kg * mx::kScaleTile, most = 0xFFFFFFFF;
  return {__builtin_amdgcn_make_buffer_rsrc((void*)(base + tile * ks * mx::kOperand), 0, (int)(uint32_t)(c < most ? c : most), 0x00020000),
          __builtin_amdgcn_make_buffer_rsrc((void*)(base + scales_off + tile * kg * mx::kScaleTile), 0,
                                            (int)(uint32_t)(g < most ? g : most), 0x00020000)};
}

typedef __attribute__((address_space(3))) void* LdsPtr;
template <int N>  // waits until at most N vector memory operations are under way
__device__ __forceinline__ void vm_wait() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// The product of a workgroup's tile.  K advances by one step of 128.  Operands go from memory
// straight into LDS (each wave copies whole operands, 1024 bytes an instruction) in the MFMA's own
// order, so that a lane's 16 bytes lie at lane * 16 and LDS is read without conflicts.  Three
// stages: in the middle of step s, when every wave has read the last of it, its stage takes the
// loads of step s + 3, and the operands of step s + 1 are waited for; their reading goes on under
// the second half of the step's products.  Scales do not pass through LDS: a word per lane and
// operand holds four steps' worth, loaded a group of steps ahead.
//
// wrow(r), xrow(r): the row, counted from the operand's first, of row r of the workgroup's weights
// and activations (any valid row for those past the end); yrow(m): row m of the outputs, or null;
// n0: the first of its columns.
template <int WN, int WM, int TN, int TM, int KS, typename WRow, typename XRow, typename YRow>
__device__ __forceinline__ void mx_core(const MxOperand& W, const MxOperand& X, int ks, int kg, uint8_t* lds0, uint8_t* lds1,
                                        uint8_t* lds2, int64_t n0, int64_t N, WRow&& wrow, XRow&& xrow, YRow&& yrow) {
  using C = MxTile<WN, WM, TN, TM, KS>;
  constexpr int P = C::kPieces, H = TN / 2;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, q = lane >> 4;
  const int part = wave / C::kGroup, member = wave % C::kGroup;  // share of K, wave of its group
  const int wn = member % WN, wm = member / WN;
  // this group's steps: from a multiple of four, so that a step's scale byte is known at compile time
  const int per = (kg + KS - 1) / KS * 4, first = part * per;
  const int mine = ks - first < per ? ks - first : per;  // none where negative or zero
  const int steps = ks < per ? ks : per;                 // that the workgroup runs
  uint32_t src[P];
#pragma unroll
  for (int p = 0; p < P; p++) {
    const int t = p * C::kGroup + member;  // kRT is a multiple of kGroup: p alone says which operand
    src[p] = (uint32_t)mx::code_at(p * C::kGroup < C::kRT ? wrow(t * 16 + i) : xrow((t - C::kRT) * 16 + i), q, ks);
  }
  uint32_t sw[TN], sx[TM];
#pragma unroll
  for (int t = 0; t < TN; t++) sw[t] = (uint32_t)mx::scale_at(wrow((wn * TN + t) * 16 + i), q, kg);
#pragma unroll
  for (int t = 0; t < TM; t++) sx[t] = (uint32_t)mx::scale_at(xrow((wm * TM + t) * 16 + i), q, kg);
  // Every step loads, the last ones again the last step's operands: a branch around a load would
  // make the compiler wait for all loads where the paths join.
  auto fetch = [&](int s, uint8_t* stage) {
    const int at = (first + s < ks ? first + s : ks - 1) * mx::kOperand;
#pragma unroll
    for (int p = 0; p < P; p++)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(p * C::kGroup < C::kRT ? W.codes : X.codes,
                                               (LdsPtr)(stage + part * C::kStage + (p * C::kGroup + member) * mx::kOperand), 16, src[p],
                                               at, 0, 0);
  };
  int fw[TN], fx[TM], fw2[TN], fx2[TM];
  auto scales = [&](int g) {
    const int at = (first / 4 + g < kg ? first / 4 + g : kg - 1) * mx::kScaleTile;
#pragma unroll
    for (int t = 0; t < TN; t++) fw2[t] = __builtin_amdgcn_raw_buffer_load_b32(W.scales, sw[t], at, 0);
#pragma unroll
    for (int t = 0; t < TM; t++) fx2[t] = __builtin_amdgcn_raw_buffer_load_b32(X.scales, sx[t], at, 0);
  };
  auto next = [&] {
#pragma unroll
    for (int t = 0; t < TN; t++) fw[t] = fw2[t];
#pragma unroll
    for (int t = 0; t < TM; t++) fx[t] = fx2[t];
  };
  auto meet = [&] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  MxAcc acc[TN][TM] = {};
  mx::i32x4 a[TN], b[TM], b2[TM];
  auto read_a = [&](uint8_t* stage, int u) {
    a[u] = *reinterpret_cast<const mx::i32x4*>(stage + part * C::kStage + (wn * TN + u) * mx::kOperand + lane * 16);
  };
  auto read_b = [&](uint8_t* stage, int t) {
    b2[t] = *reinterpret_cast<const mx::i32x4*>(stage + part * C::kStage + (C::kRT + wm * TM + t) * mx::kOperand + lane * 16);
  };
  auto step = [&](auto jc, int s, uint8_t* cur, uint8_t* nxt) {
    constexpr int j = decltype(jc)::value;
    const bool live = KS == 1 || s < mine;
#pragma unroll
    for (int u = H; u < TN; u++) read_a(cur, u);
    __builtin_amdgcn_sched_barrier(0);
    if (live) {
#pragma unroll
      for (int u = 0; u < H; u++)
#pragma unroll
        for (int t = 0; t < TM; t++) acc[u][t] = mx_mfma<j>(a[u], b[t], acc[u][t], fw[u], fx[t]);
    }
    __builtin_amdgcn_sched_barrier(0);
    // Loads end in order and the P of step s + 2 are the last issued: with P under way those of
    // step s + 1 have arrived.
    vm_wait<P>();
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave has read the last of stage s
    meet();
    if (j == 1) scales((s >> 2) + 1);
    __builtin_amdgcn_sched_barrier(0);
    fetch(s + 3, cur);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < TM; t++) read_b(nxt, t);
#pragma unroll
    for (int u = 0; u < H; u++) read_a(nxt, u);
    __builtin_amdgcn_sched_barrier(0);
    if (live) {
#pragma unroll
      for (int u = H; u < TN; u++)
#pragma unroll
        for (int t = 0; t < TM; t++) acc[u][t] = mx_mfma<j>(a[u], b[t], acc[u][t], fw[u], fx[t]);
    }
    if (j == 2) {  // a use that keeps the loads of the scales from sinking below it
#pragma unroll
      for (int t = 0; t < TN; t++) asm volatile("" : "+v"(fw2[t]));
#pragma unroll
      for (int t = 0; t < TM; t++) asm volatile("" : "+v"(fx2[t]));
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < TM; t++) b[t] = b2[t];
  };
  scales(0);
  __builtin_amdgcn_sched_barrier(0);  // the counted wait goes by this order
  fetch(0, lds0);
  __builtin_amdgcn_sched_barrier(0);
  fetch(1, lds1);
  fetch(2, lds2);
  __builtin_amdgcn_sched_barrier(0);
  next();
  vm_wait<2 * P>();
  meet();
#pragma unroll
  for (int t = 0; t < TM; t++) read_b(lds0, t);
#pragma unroll
  for (int u = 0; u < H; u++) read_a(lds0, u);
#pragma unroll
  for (int t = 0; t < TM; t++) b[t] = b2[t];
  // twelve steps a turn: the scales come round every four, the stages every three
  for (int s = 0;; s += 12) {
#define BQM_MX_STEP(U, CUR, NXT)                             \
  step(std::integral_constant<int, (U) & 3>{}, s + (U), CUR, NXT); \
  if (s + (U) + 1 >= steps) break;                           \
  if (((U) & 3) == 3) next();
    BQM_MX_STEP(0, lds0, lds1)
    BQM_MX_STEP(1, lds1, lds2)
    BQM_MX_STEP(2, lds2, lds0)
    BQM_MX_STEP(3, lds0, lds1)
    BQM_MX_STEP(4, lds1, lds2)
    BQM_MX_STEP(5, lds2, lds0)
    BQM_MX_STEP(6, lds0, lds1)
    BQM_MX_STEP(7, lds1, lds2)
    BQM_MX_STEP(8, lds2, lds0)
    BQM_MX_STEP(9, lds0, lds1)
    BQM_MX_STEP(10, lds1, lds2)
    BQM_MX_STEP(11, lds2, lds0)
#undef BQM_MX_STEP
  }
  vm_wait<0>();  // nothing may be on its way into LDS when it is used again, or when the workgroup ends
  __syncthreads();
  // Each wave turns its outputs in LDS, 16 columns (rows of Y) at a time, so that a store covers
  // whole runs of a row of Y: straight from the MFMA's layout a store's lanes are rows apart.  The
  // groups' shares of K are added on the way, in order; each group stores a part.
  constexpr int kRow = TN * 16 + 4, kTurn = 16 * kRow;  // floats; four of padding against bank conflicts
  constexpr int kThird = (C::kGroup * KS + 2) / 3;
  static_assert(kThird * kTurn * 4 <= C::kStage * KS, "a third of the waves turn their outputs in one stage");
  auto turn = [&](int w) { return reinterpret_cast<float*>(w < kThird ? lds0 : w < 2 * kThird ? lds1 : lds2) + (w % kThird) * kTurn; };
  float* own = turn(wave);
  const int64_t nw = n0 + wn * TN * 16;
#pragma unroll
  for (int t = 0; t < TM; t++) {
#pragma unroll
    for (int u = 0; u < TN; u++) *reinterpret_cast<MxAcc*>(own + i * kRow + u * 16 + 4 * q) = acc[u][t];
    KS > 1 ? __syncthreads() : mx::wave_turn();
    if ((N & 3) == 0) {
#pragma unroll
      for (int r = 0; r < TN; r++) {
        if (r % KS != part) continue;
        const int at = r * 64 + lane, m = at / (TN * 4), n = at % (TN * 4) * 4;
        MxAcc d = *reinterpret_cast<const MxAcc*>(turn(member) + m * kRow + n);
#pragma unroll
        for (int k = 1; k < KS; k++) {
          const MxAcc e = *reinterpret_cast<const MxAcc*>(turn(k * C::kGroup + member) + m * kRow + n);
          d = MxAcc{d[0] + e[0], d[1] + e[1], d[2] + e[2], d[3] + e[3]};
        }
        float* y = yrow((wm * TM + t) * 16 + m);
        if (y && nw + n < N) *reinterpret_cast<MxAcc*>(y + nw + n) = d;
      }
    } else {
      for (int r = part; r < TN * 4; r += KS) {
        const int at = r * 64 + lane, m = at / (TN * 16), n = at % (TN * 16);
        float d = turn(member)[m * kRow + n];
#pragma unroll
        for (int k = 1; k < KS; k++) d += turn(k * C::kGroup + member)[m * kRow + n];
        float* y = yrow((wm * TM + t) * 16 + m);
        if (y && nw + n < N) y[nw + n] = d;
      }
    }
    KS > 1 ? __syncthreads() : mx::wave_turn();
  }
}

// Tile of a workgroup.  Workgroups are dealt round-robin to the eight XCDs: those of one XCD take
// consecutive tiles, ordered in bands of eight row tiles and along the weights inside a band, so
// that what an XCD computes at a time is about square and its L2 is asked for little.
struct MxPlace {
  int m, n;
};
__device__ __forceinline__ MxPlace mx_place(int bid, int tiles_m, int tiles_n) {
  const int nwg = tiles_m * tiles_n, xcd = bid & 7, more = nwg & 7;
  const int t = xcd * (nwg >> 3) + (xcd < more ? xcd : more) + (bid >> 3);
  const int band = t / (8 * tiles_n), r = t - band * 8 * tiles_n;
  const int high = tiles_m - band * 8 < 8 ? tiles_m - band * 8 : 8;
  return {band * 8 + r % high, r / high};
}

template <int WN, int WM, int TN, int TM, int KS, int OCC>
__global__ __launch_bounds__(WN* WM* KS * 64) __attribute__((amdgpu_waves_per_eu(OCC, OCC))) void k_qmm_mxfp4(
    const uint8_t* __restrict__ w, int64_t w_scales, const uint8_t* __restrict__ x, int64_t x_scales, float* __restrict__ Y, int64_t M,
    int64_t N, int ks, int kg, int tiles_m, int tiles_n) {
  using C = MxTile<WN, WM, TN, TM, KS>;
  const MxPlace at = mx_place(blockIdx.x, tiles_m, tiles_n);
  const int64_t tn = at.n, tm = at.m;
  const int64_t n0 = tn * C::kBN, m0 = tm * C::kBM;
  const int nr = (int)(N - n0 < C::kBN ? N - n0 : C::kBN), mr = (int)(M - m0 < C::kBM ? M - m0 : C::kBM);
  auto wr = [&](int r) { return r < nr ? r : nr - 1; };
  auto xr = [&](int r) { return r < mr ? r : mr - 1; };
  const MxOperand wo = mx_operand(w, w_scales, tn * C::kRT, (N + 15) >> 4, ks, kg);
  const MxOperand xo = mx_operand(x, x_scales, tm * C::kCT, (M + 15) >> 4, ks, kg);
  __shared__ __attribute__((aligned(16))) uint8_t lds0[KS * C::kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[KS * C::kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds2[KS * C::kStage];
  mx_core<WN, WM, TN, TM, KS>(wo, xo, ks, kg, lds0, lds1, lds2, n0, N, wr, xr, [&](int m) { return m < mr ? Y + (m0 + m) * N : nullptr; });
}

// ---- expert-indexed product ----
// Every workgroup counts the slots per expert, cuts each expert's slots (in index order) into row
// tiles of kBM and numbers them, experts ascending; item i is row tile i / span with those weight tiles
// that have tile % span == i % span, one after another: the slots are counted once for all of them.
// Workgroups past the last item only take part in filling the rows that no tile computes.
template <int WN, int WM, int TN, int TM, int KS, int OCC>
__global__ __launch_bounds__(WN* WM* KS * 64) __attribute__((amdgpu_waves_per_eu(OCC, OCC))) void k_qmm_id_mxfp4(
    const uint8_t* __restrict__ w, int64_t w_scales, const uint8_t* __restrict__ x, int64_t x_scales, const int32_t* __restrict__ ids,
    float* __restrict__ Y, int E, int64_t N, int ks, int kg, int TS, int top_k, int64_t xtr, int64_t xsr, int64_t x_tiles, int tiles_n,
    int span, int deal) {
  using C = MxTile<WN, WM, TN, TM, KS>;
  constexpr int NT = C::kThreads;
  __shared__ __attribute__((aligned(16))) uint8_t lds0[KS * C::kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[KS * C::kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds2[KS * C::kStage];
  __shared__ int cnt[BQM_QMV_ID_MAX_E];
  __shared__ int xrow[C::kBM], yrow[C::kBM];
  __shared__ int wsum[NT / 64], tile_e, tile_m0, n_fill;
  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // f(first slot, the ids of four slots; those past the end are -1) for the slots of this wave, a run
  // of them, 256 at a time in index order, four lots of loads in flight; the first four stay in
  // registers for all three passes over the slots
  const int run = (TS + 256 * (NT / 64) - 1) / (256 * (NT / 64)) * 256, r0 = wave * run;
  const __amdgpu_buffer_rsrc_t rI = __builtin_amdgcn_make_buffer_rsrc((void*)ids, 0, TS * 4, 0x00020000);
  auto load_ids = [&](int s, mx::u32x4 (&v)[4]) {
#pragma unroll
    for (int k = 0; k < 4; k++) v[k] = __builtin_amdgcn_raw_buffer_load_b128(rI, (s + k * 256 + lane * 4) * 4, 0, 0);
  };
  mx::u32x4 ids0[4];
  load_ids(r0, ids0);
  auto for_slots = [&](auto&& f) {
    for (int s = r0; s < r0 + run && s < TS; s += 1024) {
      mx::u32x4 v[4] = {ids0[0], ids0[1], ids0[2], ids0[3]};
      if (s > r0) load_ids(s, v);
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const int at = s + k * 256 + lane * 4;
        int id[4];
#pragma unroll
        for (int c = 0; c < 4; c++) id[c] = at + c < TS && s + k * 256 < r0 + run ? (int)v[k][c] : -1;
        f(at, id);
      }
    }
  };
  // Rows that no tile computes, each by one workgroup (slots b, b + grid, ...): a padding slot
  // (negative id) gives zeros, an id >= E NaN.  Most calls have none.
  auto outside = [&](int64_t s) { return s < TS && (unsigned)ids[s] >= (unsigned)E; };
  bool any = false;
  for (int64_t s = (int64_t)tid * gridDim.x + blockIdx.x; s < TS; s += (int64_t)NT * gridDim.x) any = any || outside(s);
  if (__syncthreads_or(any)) {
    for (int64_t s0 = 0; s0 < TS; s0 += (int64_t)NT * gridDim.x) {
      if (tid == 0) n_fill = 0;
      __syncthreads();
      const int64_t s = s0 + (int64_t)tid * gridDim.x + blockIdx.x;
      if (outside(s)) cnt[atomicAdd(&n_fill, 1)] = (int)s;
      __syncthreads();
      for (int k = 0; k < n_fill; k++) {
        const int at = cnt[k];
        const float v = ids[at] < 0 ? 0.0f : __builtin_nanf("");
        for (int64_t n = tid; n < N; n += NT) Y[at * N + n] = v;
      }
      __syncthreads();
    }
  }
  for (int e = tid; e < E; e += NT) cnt[e] = 0;
  for (int r = tid; r < C::kBM; r += NT) yrow[r] = -1;
  __syncthreads();
  for_slots([&](int, const int(&id)[4]) {
#pragma unroll
    for (int c = 0; c < 4; c++)
      if ((unsigned)id[c] < (unsigned)E) atomicAdd(&cnt[id[c]], 1);
  });
  __syncthreads();
  // the expert and the first of its slots that this workgroup's row tile holds: thread t looks at a
  // run of experts, after a sum of the tile counts over the threads before it
  const int per = (E + NT - 1) / NT;
  const int e0 = tid * per < E ? tid * per : E, e1 = e0 + per < E ? e0 + per : E;
  int tiles = 0;
  for (int e = e0; e < e1; e++) tiles += (cnt[e] + C::kBM - 1) / C::kBM;
  int before = tiles;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(before, o, 64);
    if (lane >= o) before += u;
  }
  if (lane == 63) wsum[wave] = before;
  __syncthreads();
  before -= tiles;
  int all_tiles = 0;
#pragma unroll
  for (int k = 0; k < NT / 64; k++) {
    before += k < wave ? wsum[k] : 0;
    all_tiles += wsum[k];
  }
  // item of this workgroup: in order, or dealt so that an XCD (workgroups go round them) has a run of them
  const int items = __builtin_amdgcn_readfirstlane(all_tiles) * span, mask = (1 << deal) - 1;
  const int run_at = blockIdx.x & mask, more = items & mask, nth = blockIdx.x >> deal;
  if (nth >= (items >> deal) + (run_at < more)) return;  // none left, the whole workgroup
  const int item = run_at * (items >> deal) + (run_at < more ? run_at : more) + nth;
  const int tm = item / span;
  if (tm >= before && tm < before + tiles)
    for (int e = e0; e < e1; e++) {
      const int k = (cnt[e] + C::kBM - 1) / C::kBM;
      if (tm < before + k) {
        tile_e = e;
        tile_m0 = (tm - before) * C::kBM;
        break;
      }
      before += k;
    }
  __syncthreads();
  const int e = __builtin_amdgcn_readfirstlane(tile_e), m0 = __builtin_amdgcn_readfirstlane(tile_m0);
  const int rows = cnt[e] - m0 < C::kBM ? cnt[e] - m0 : C::kBM;
  // its slots: those of rank m0 and up among the expert's, the waves before this one counted first
  int found = 0;
  for_slots([&](int, const int(&id)[4]) {
#pragma unroll
    for (int c = 0; c < 4; c++) found += __popcll(__ballot(id[c] == e));
  });
  if (lane == 0) wsum[wave] = found;
  __syncthreads();
  int rank = -m0;
  for (int k = 0; k < wave; k++) rank += wsum[k];
  for_slots([&](int s, const int(&id)[4]) {
    const uint64_t any = __ballot(id[0] == e || id[1] == e || id[2] == e || id[3] == e);
    if (any == 0) return;
    int at = rank;
#pragma unroll
    for (int c = 0; c < 4; c++) {
      const uint64_t b = __ballot(id[c] == e);
      at += __popcll(b & ((1ull << lane) - 1));
      rank += __popcll(b);
    }
#pragma unroll
    for (int c = 0; c < 4; c++) {
      if (id[c] != e) continue;
      if (at >= 0 && at < C::kBM) {
        const int t = (s + c) / top_k;
        xrow[at] = (int)(t * xtr + (s + c - t * top_k) * xsr);
        yrow[at] = s + c;
      }
      at++;
    }
  });
  __syncthreads();
  const MxOperand xo = mx_operand(x, x_scales, 0, x_tiles, ks, kg);
  const int64_t all = ((int64_t)E * N + 15) >> 4;
  for (int tn = item - tm * span; tn < tiles_n; tn += span) {
    const int64_t n0 = (int64_t)tn * C::kBN, at = (int64_t)e * N + n0;
    const int nr = (int)(N - n0 < C::kBN ? N - n0 : C::kBN), off = (int)(at & 15);
    mx_core<WN, WM, TN, TM, KS>(
        mx_operand(w, w_scales, at >> 4, all, ks, kg), xo, ks, kg, lds0, lds1, lds2, n0, N, [&](int r) { return off + (r < nr ? r : nr - 1); },
        [&](int r) { return xrow[r < rows ? r : rows - 1]; },
        [&](int m) { return yrow[m] >= 0 ? Y + (int64_t)yrow[m] * N : nullptr; });
    __syncthreads();  // the next tile's operands go where this one's outputs were turned
  }
}

template <int WN, int WM, int TN, int TM, int KS, int OCC>
int launch_qmm_mx_as(const uint8_t* wc, const uint8_t* xc, float* Y, int64_t M, int64_t N, const MxLayout& W, const MxLayout& X,
                     hipStream_t s) {
  using C = MxTile<WN, WM, TN, TM, KS>;
  const int64_t tm = (M + C::kBM - 1) / C::kBM, tn = (N + C::kBN - 1) / C::kBN;
  hipLaunchKernelGGL((k_qmm_mxfp4<WN, WM, TN, TM, KS, OCC>), dim3((unsigned)(tm * tn)), dim3(C::kThreads), 0, s, wc, W.scales_off, xc,
                     X.scales_off, Y, M, N, (int)W.ks, (int)W.kg, (int)tm, (int)tn);
  return launch_status();
}

template <int WN, int WM, int TN, int TM, int KS, int OCC>
int launch_qmm_id_mx_as(const uint8_t* wc, int E, int64_t N, const MxLayout& W, const int32_t* ids, int TS, int top_k, const uint8_t* xc,
                        const MxLayout& X, int64_t xtr, int64_t xsr, float* Y, int aim, int deal, hipStream_t s) {
  using C = MxTile<WN, WM, TN, TM, KS>;
  const int64_t tn = (N + C::kBN - 1) / C::kBN;
  // row tiles: at most one partial tile per expert that has slots, plus the full ones
  const int64_t tm = (TS < E ? TS : E) + TS / C::kBM > 0 ? (TS < E ? TS : E) + TS / C::kBM : 1;
  // about `aim` workgroups, each with the same number of weight tiles as far as that goes
  int64_t span = (aim + tm / 2) / tm;
  span = span < 1 ? 1 : span < tn ? span : tn;
  const int64_t each = (tn + span - 1) / span;
  span = (tn + each - 1) / each;
  if (tm * span > kMaxGrid || tn > INT32_MAX) return BQM_E_SHAPE;
  hipLaunchKernelGGL((k_qmm_id_mxfp4<WN, WM, TN, TM, KS, OCC>), dim3((unsigned)(tm * span)), dim3(C::kThreads), 0, s, wc, W.scales_off, xc,
                     X.scales_off, ids, Y, E, N, (int)W.ks, (int)W.kg, TS, top_k, xtr, xsr, X.rt, (int)tn, (int)span, deal);
  return launch_status();
}

}  // namespace

// Offsets into an operand are 32 bits wide: a workgroup's 17 row tiles of weights or activations
// (and, where rows are gathered, the activations as a whole) stay below 2 GiB.
static bool mx_fits(const MxLayout& L) { return L.ks <= BQM_MXFP4_MAX_K / mx::kStepK && L.ks * 17 * mx::kOperand < ((int64_t)1 << 31); }

// The dense product's tile, by an estimate of its time on 256 compute units, from two figures for each:
// `one`, the time of a step where a unit holds one workgroup (latency), and `full`, its share of a step
// where it holds several (throughput); 2 us a launch and 1 a round of workgroups are the same for all.
// Both were measured with weights in the last cache, but for the 0.84 of 256 x 256: measured 0.88, and set
// lower because that tile reads weights from memory less often, for which the estimate has no term.  It
// turns products of about 512 tokens its way: with the quantizer and N x K = 17408 x 5120, weights from
// memory, 512 tokens take 46.9 us (128 x 128: 53.2) and 600 take 46.9 (52.7); with weights in the cache
// it loses, 36.5 (35.5) and 41.4 (37.3) without the quantizer.  Other N and K at that length were not
// measured both ways.
// Measured (us, N x K = 17408 x 5120): 4096 tokens 207 with 128 x 128 or 256 x 256, 64: 12.1 with 128 x 64
// in two shares of K (in one: 14.8), 16: 10.5 with 128 x 32 in four (64 x 16 in eight: 14.8); 8192^3: 255
// with 256 x 256 (128 x 128: 290).  N x K = 5120 x 17408: 512 tokens 38.5 with 128 x 128 in two shares (in
// one: 48.6), 64: 15.1 with 64 x 32 in eight, one: 11.3 with 32 x 16 in sixteen.  256 x 128 tiles gained
// nowhere: 4096 tokens 228 with waves of 64 x 64, 243 with waves of 128 x 64, whose registers spill.
struct MxChoice {
  int bn, bm, shares;
  float one, full;
  int (*launch)(const uint8_t*, const uint8_t*, float*, int64_t, int64_t, const MxLayout&, const MxLayout&, hipStream_t);
};
static constexpr MxChoice kMxChoices[] = {
    {256, 256, 1, 0.84f, 0.97f, launch_qmm_mx_as<2, 4, 8, 4, 1, 2>}, {128, 128, 1, 0.35f, 0.27f, launch_qmm_mx_as<2, 2, 4, 4, 1, 3>},
    {128, 128, 2, 0.54f, 0.85f, launch_qmm_mx_as<2, 2, 4, 4, 2, 2>}, {128, 64, 2, 0.40f, 0.44f, launch_qmm_mx_as<2, 2, 4, 2, 2, 4>},
    {128, 32, 4, 0.55f, 0.83f, launch_qmm_mx_as<2, 1, 4, 2, 4, 2>},  {64, 64, 4, 0.50f, 0.77f, launch_qmm_mx_as<1, 1, 4, 4, 4, 1>},
    {64, 32, 8, 0.78f, 1.30f, launch_qmm_mx_as<1, 1, 4, 2, 8, 2>},   {64, 16, 8, 0.73f, 1.06f, launch_qmm_mx_as<1, 1, 4, 1, 8, 2>},
    {32, 16, 16, 1.30f, 1.80f, launch_qmm_mx_as<1, 1, 2, 1, 16, 4>}};

// The index of the tile, -1 where none has room for the outputs.  (The tests ask too: they have to run
// every tile.)
extern "C" int bqm_internal_qmm_mxfp4_choice(int64_t M, int64_t N, int64_t K) {
  const MxLayout W = mx_layout(N, K);
  int best = -1;
  double least = 0;
  for (const MxChoice& c : kMxChoices) {
    const int64_t wgs = ((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn), load = (wgs + 255) / 256;
    if (wgs > kMaxGrid) continue;
    const int64_t steps = (W.kg + c.shares - 1) / c.shares * 4;
    const double t = (double)(steps < W.ks ? steps : W.ks) * (load == 1 ? c.one : load * c.full) + 2.0 + load;
    if (best < 0 || t < least) {
      best = (int)(&c - kMxChoices);
      least = t;
    }
  }
  return best;
}

int launch_qmm_mxfp4(const void* w, const void* x, float* Y, int64_t M, int64_t N, int64_t K, hipStream_t s) {
  const MxLayout W = mx_layout(N, K), X = mx_layout(M, K);
  if (!mx_fits(W)) return BQM_E_SHAPE;
  const int c = bqm_internal_qmm_mxfp4_choice(M, N, K);
  if (c < 0) return BQM_E_SHAPE;
  return kMxChoices[c].launch(static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(x), Y, M, N, W, X, s);
}

// Experts that have slots, at most.
static int mx_used(int E, int TS) { return TS < E ? TS : E > 0 ? E : 1; }

// The tile by the slots of an expert if all were used alike: a wide and tall tile reads gathered rows
// and the weights of busy experts less often, a smaller one spends less on empty rows.  `aim`: with
// more workgroups each counts the slots for less work, with fewer the last ones to end leave units
// idle.  Measured in order (us; 128 experts, top-8, a skewed router, 1536 x 4096 each): 4096 tokens 361
// with 256 x 128 (256 x 64: 379, 128 x 128: 450), 512: 87 with 256 x 64 (128 x 128: 89, 256 x 128:
// 96), 128: 41 with 128 x 64 (256 x 64: 47), 16: 23 with 128 x 32 (128 x 64: 24, 64 x 16 in four
// shares of K: 25), one 7.7 with 64 x 16 (128 x 32: 10.1); aiming at 1536 instead of 1024, 2048
// tokens take 218 and not 190, 128 tokens at 2048 take 46 and not 41, 16 tokens at 1024 26 and not 23.
// Items are dealt to the XCDs in eight runs where experts have few row tiles (16 tokens 21.4, in order
// 23.1; 64: 34 and 36.7; 256: 68 and 71), and taken in order where several row tiles share the weights in
// the last cache (512 tokens 88, dealt 95; 4096: 371 and 403).  All of it is from this one layer: with few
// experts or few outputs the items may be fewer than the units, each over all of K.  A row per slot (4096 x
// 1536 each): one token 8.3, 16 tokens 23.6, 128: 66, 512: 116, 2048: 331, 4096: 703.
extern "C" int bqm_internal_qmm_id_mxfp4_choice(int E, int64_t N, int TS) {
  const int used = mx_used(E, TS);
  if ((int64_t)used * ((N + 63) / 64) <= 768 && TS <= 2 * used) return 0;
  return TS >= 48 * used ? 1 : TS >= 12 * used ? 2 : TS >= 6 * used ? 3 : 4;
}

int launch_qmm_id_mxfp4(const void* w, int E, int64_t N, int64_t K, const int32_t* ids, int T, int top_k, const void* x,
                        int64_t x_rows, int64_t x_tok_rows, int64_t x_slot_rows, float* Y, hipStream_t s) {
  const MxLayout W = mx_layout((int64_t)E * N, K), X = mx_layout(x_rows, K);
  const uint8_t* wc = static_cast<const uint8_t*>(w);
  const uint8_t* xc = static_cast<const uint8_t*>(x);
  if (!mx_fits(W) || X.scales_off >= ((int64_t)1 << 31)) return BQM_E_SHAPE;
  const int TS = T * top_k, used = mx_used(E, TS), deal = TS >= 24 * used ? 0 : 3;
#define BQM_MX_ID(aim, ...) \
  launch_qmm_id_mx_as<__VA_ARGS__>(wc, E, N, W, ids, TS, top_k, xc, X, x_tok_rows, x_slot_rows, Y, aim, deal, s)
  switch (bqm_internal_qmm_id_mxfp4_choice(E, N, TS)) {
    case 0: return BQM_MX_ID(2048, 1, 1, 4, 1, 4, 2);
    case 1: return BQM_MX_ID(1024, 4, 2, 4, 4, 1, 2);
    case 2: return BQM_MX_ID(1536, 4, 1, 4, 4, 1, 2);
    case 3: return BQM_MX_ID(1024, 2, 2, 4, 2, 1, 3);
    default: return BQM_MX_ID(2048, 2, 1, 4, 2, 1, 2);
  }
#undef BQM_MX_ID
}

}  // namespace bqm
