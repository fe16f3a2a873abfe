// Routing to experts (kernel and launcher; included by repack.hip).
//
// A token's E values lie in the registers of G lanes, V neighbouring experts a lane: sixteen lanes a
// token (four tokens a wave) where there are tokens enough to fill the chip, since a reduction over
// sixteen lanes takes four DPP steps and serves four tokens; all 64 lanes otherwise.  Each of the
// top_k rounds takes the largest value and, of equal ones, the lowest index, first over a
// lane's registers, then over its lanes.  Values are 64 bits wide: between neighbours in the order
// of the real numbers an id hangs on the last bits of a score, and fp32 scores would swap them now and
// then.  (exp in 64 bits runs at the rate of fp32 here; what binds the kernel is the selection.)
#pragma once

#include "mxfp4.h"

namespace bqm {
namespace {

struct RouteArgs {
  const void* logits;
  int64_t stride;
  const float* bias;
  int T, E, n_group, topk_group, group_top, top_k, renorm, vec;
  float scale;
  int32_t* ids;
  float* weights;
};

constexpr int kRouteWaves = 4;

// f(value, the value of a lane that holds another part of the token's lanes), until all lanes have
// taken in all: within quads, then mirrored halves and rows (each already alike inside), then
// rows 16 and 32 lanes apart.
template <int CTRL>
__device__ __forceinline__ int dpp(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = dpp<CTRL>((int)(uint32_t)u), hi = dpp<CTRL>((int)(u >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ void best2(double& v, int& i, double u, int j) {
  if (u > v || (u == v && j < i)) {
    v = u;
    i = j;
  }
}
template <int G>
__device__ __forceinline__ void best_of(double& v, int& i) {
  best2(v, i, dpp<0xB1>(v), dpp<0xB1>(i));    // quad_perm 1 0 3 2
  best2(v, i, dpp<0x4E>(v), dpp<0x4E>(i));    // quad_perm 2 3 0 1
  best2(v, i, dpp<0x141>(v), dpp<0x141>(i));  // row_half_mirror
  best2(v, i, dpp<0x140>(v), dpp<0x140>(i));  // row_mirror
  if constexpr (G == 64) {
    best2(v, i, __shfl_xor(v, 16, 64), __shfl_xor(i, 16, 64));
    best2(v, i, __shfl_xor(v, 32, 64), __shfl_xor(i, 32, 64));
  }
}
template <int G, typename F>
__device__ __forceinline__ double reduce(double v, F&& f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  v = f(v, dpp<0x140>(v));
  if constexpr (G == 64) {
    v = f(v, __shfl_xor(v, 16, 64));
    v = f(v, __shfl_xor(v, 32, 64));
  }
  return v;
}

template <int TYPE, bool SIGMOID, int G, int V>
__global__ __launch_bounds__(kRouteWaves * 64) void k_route(RouteArgs a) {
  typedef typename mx::Elem<TYPE>::T Elem;
  constexpr int kTokens = kRouteWaves * 64 / G;  // of a workgroup
  constexpr int kVec = 16 / sizeof(Elem);
  constexpr int kHeld = V * G <= 1024 ? V * G : 1;  // values that fit LDS beside one another
  __shared__ double val_lds[kTokens * (V * G <= 1024 ? kHeld : 1)];
  __shared__ double grp_lds[kTokens][BQM_ROUTE_MAX_GROUPS];
  const int lane = threadIdx.x % G, at = threadIdx.x / G;
  const int64_t t = (int64_t)blockIdx.x * kTokens + at;
  const int64_t row = t < a.T ? t : a.T - 1;  // lanes past the last token repeat it and write nothing
  const Elem* l = static_cast<const Elem*>(a.logits) + row * a.stride;
  const double inf = __builtin_inf();
  const int e0 = lane * V;
  float x[V];
  if (V % kVec == 0 && a.vec) {
#pragma unroll
    for (int c = 0; c < V; c += kVec) {
      Elem v[kVec];
      if (e0 + c < a.E) __builtin_memcpy(v, __builtin_assume_aligned(l + e0 + c, 16), 16);
#pragma unroll
      for (int k = 0; k < (V < kVec ? V : kVec); k++) x[c + k] = e0 + c < a.E ? (float)v[k] : -__builtin_inff();
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; v++) x[v] = e0 + v < a.E ? (float)l[e0 + v] : -__builtin_inff();
  }
  float bias[V];
#pragma unroll
  for (int v = 0; v < V; v++) bias[v] = a.bias && e0 + v < a.E ? a.bias[e0 + v] : 0.0f;
  // the row's maximum and whether anything in it is no number
  double top = -inf, bad = 0;
#pragma unroll
  for (int v = 0; v < V; v++) {
    top = x[v] > top ? (double)x[v] : top;
    if (x[v] != x[v] || bias[v] != bias[v] || (!SIGMOID && x[v] == __builtin_inff())) bad = 1;
  }
  bad = reduce<G>(bad, [](double p, double q) { return p > q ? p : q; });
  const bool sums = a.n_group > 1 && a.group_top == 2, scored = a.bias || sums;
  double total = 1;
  if (!SIGMOID) {
    top = reduce<G>(top, [](double p, double q) { return p > q ? p : q; });
    if (scored || !a.renorm) {
      total = 0;
#pragma unroll
      for (int v = 0; v < V; v++) total += x[v] == -__builtin_inff() ? 0.0 : exp((double)x[v] - top);
      total = reduce<G>(total, [](double p, double q) { return p + q; });
    }
  }
  auto score = [&](float f) { return SIGMOID ? 1.0 / (1.0 + exp(-(double)f)) : exp((double)f - top) / total; };
  double val[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    const double s = scored ? score(x[v]) : (double)x[v];
    val[v] = x[v] == -__builtin_inff() ? -inf : s + (double)bias[v];
  }
  if (a.n_group > 1) {
    const int size = a.E / a.n_group;
    double* held = val_lds + at * kHeld;
    if constexpr (V * G <= 1024) {
#pragma unroll
      for (int v = 0; v < V; v++) held[e0 + v] = val[v];
    }
    __syncthreads();
    for (int g = lane; g < a.n_group; g += G) {
      double v1 = -inf, v2 = -inf;
      for (int e = g * size; e < (g + 1) * size; e++) {
        double v;
        if constexpr (V * G <= 1024) {
          v = held[e];
        } else {
          const float f = (float)l[e];
          v = f == -__builtin_inff() ? -inf : (scored ? score(f) : (double)f) + (a.bias ? (double)a.bias[e] : 0.0);
        }
        v2 = v > v1 ? v1 : v > v2 ? v : v2;
        v1 = v > v1 ? v : v1;
      }
      grp_lds[at][g] = a.group_top == 2 && v2 != -inf ? v1 + v2 : v1;
    }
    __syncthreads();
    // groups that stay open, one bit each
    uint64_t open = 0;
    for (int g = 0; g < a.n_group; g += G) {
      const int h = g + lane;
      int before = 0;
      if (h < a.n_group)
        for (int k = 0; k < a.n_group; k++) {
          const double u = grp_lds[at][k], w = grp_lds[at][h];
          before += u > w || (u == w && k < h);
        }
      const uint64_t b = __ballot(h < a.n_group && before < a.topk_group);
      open |= (G == 64 ? b : b >> (threadIdx.x % 64 / G * G) & ((1ull << (G % 64)) - 1)) << g;
    }
    int g = e0 < a.E ? e0 / size : 0, rest = e0 - g * size;
#pragma unroll
    for (int v = 0; v < V; v++) {
      const double own = a.bias ? val[v] : (double)x[v];  // group sums were of scores, the order is the logits'
      val[v] = open >> (g & 63) & 1 ? own : -inf;
      const bool turn = ++rest == size;
      g += turn;
      rest = turn ? 0 : rest;
    }
  }
  // the rounds; lane s % G keeps slot s
  constexpr int kKept = BQM_QMV_ID_MAX_TOPK / G > 0 ? BQM_QMV_ID_MAX_TOPK / G : 1;
  int kept[kKept];
#pragma unroll
  for (int k = 0; k < kKept; k++) kept[k] = -1;
  for (int s = 0; s < a.top_k; s++) {
    double best = -inf;
    int i = 1 << 30;
#pragma unroll
    for (int v = 0; v < V; v++)
      if (val[v] > best) {
        best = val[v];
        i = e0 + v;
      }
    best_of<G>(best, i);
#pragma unroll
    for (int v = 0; v < V; v++)
      if (e0 + v == i) val[v] = -inf;
#pragma unroll
    for (int k = 0; k < kKept; k++)
      if (s == k * G + lane) kept[k] = best == -inf ? -1 : i;
  }
  double w[kKept], chosen = 0;
#pragma unroll
  for (int k = 0; k < kKept; k++) {
    w[k] = kept[k] >= 0 ? score((float)l[kept[k]]) : 0.0;
    chosen += w[k];
  }
  if (a.renorm) chosen = reduce<G>(chosen, [](double p, double q) { return p + q; });
#pragma unroll
  for (int k = 0; k < kKept; k++) {
    const int s = k * G + lane;
    if (t >= a.T || s >= a.top_k) continue;
    if (a.renorm) w[k] = chosen == 0 ? 0.0 : w[k] / chosen;
    float f = (float)(w[k] * (double)a.scale);
    int id = kept[k];
    if (bad != 0) {
      id = s < a.E ? s : -1;
      f = s < a.E ? __builtin_nanf("") : 0.0f;
    }
    a.ids[t * a.top_k + s] = id;
    a.weights[t * a.top_k + s] = f;
  }
}

template <int TYPE, int G, int V>
int launch_route_as(int score, const RouteArgs& a, hipStream_t s) {
  constexpr int kTokens = kRouteWaves * 64 / G;
  hipLaunchKernelGGL(score == BQM_SIGMOID ? (k_route<TYPE, true, G, V>) : (k_route<TYPE, false, G, V>),
                     dim3((unsigned)((a.T + kTokens - 1) / kTokens)), dim3(kRouteWaves * 64), 0, s, a);
  return launch_status();
}

template <int TYPE>
int launch_route_type(int score, const RouteArgs& a, hipStream_t s) {
  if (a.E <= 256 && a.T >= 1024)
    return a.E <= 64    ? launch_route_as<TYPE, 16, 4>(score, a, s)
           : a.E <= 128 ? launch_route_as<TYPE, 16, 8>(score, a, s)
                        : launch_route_as<TYPE, 16, 16>(score, a, s);
  return a.E <= 64     ? launch_route_as<TYPE, 64, 1>(score, a, s)
         : a.E <= 128  ? launch_route_as<TYPE, 64, 2>(score, a, s)
         : a.E <= 256  ? launch_route_as<TYPE, 64, 4>(score, a, s)
         : a.E <= 1024 ? launch_route_as<TYPE, 64, 16>(score, a, s)
                       : launch_route_as<TYPE, 64, 64>(score, a, s);
}

}  // namespace

int launch_route(int score, int type, const void* logits, int64_t stride, const float* bias, int64_t T, int E, int n_group,
                 int topk_group, int group_top, int top_k, int renorm, float scale, int32_t* ids, float* weights, hipStream_t s) {
  const int bytes = type == BQM_F32 ? 4 : 2;
  const int vec = stride * bytes % 16 == 0 && E * bytes % 16 == 0;
  const RouteArgs a{logits, stride, bias, (int)T, E, n_group, topk_group, group_top, top_k, renorm, vec, scale, ids, weights};
  return type == BQM_F32   ? launch_route_type<BQM_F32>(score, a, s)
         : type == BQM_F16 ? launch_route_type<BQM_F16>(score, a, s)
                           : launch_route_type<BQM_BF16>(score, a, s);
}

}  // namespace bqm
