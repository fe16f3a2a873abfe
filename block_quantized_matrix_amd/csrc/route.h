// Routing to experts (kernel and launcher; included by repack.hip).
#pragma once

#include "mxfp4.h"

namespace bqm {
namespace {

// One wave per token, the ordering values in LDS, everything in 64 bits.
struct RouteArgs {
  const void* logits;
  int64_t stride;
  const float* bias;
  int E, n_group, topk_group, group_top, top_k, renorm;
  float scale;
  int32_t* ids;
  float* weights;
};

__device__ __forceinline__ void best_of(double& v, int& i, int o) {
  const double u = __shfl_xor(v, o, 64);
  const int j = __shfl_xor(i, o, 64);
  if (u > v || (u == v && j < i)) {
    v = u;
    i = j;
  }
}

template <int TYPE, bool SIGMOID>
__global__ __launch_bounds__(64) void k_route(RouteArgs a) {
  __shared__ double val[BQM_QMV_ID_MAX_E];
  __shared__ double grp[BQM_ROUTE_MAX_GROUPS];
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const auto* l = static_cast<const typename mx::Elem<TYPE>::T*>(a.logits) + t * a.stride;
  const double inf = __builtin_inf();
  double top = -inf, sum = 0;
  bool bad = false;
  for (int e = lane; e < a.E; e += 64) {
    const double v = (double)(float)l[e];
    bad = bad || v != v || (!SIGMOID && v == inf) || (a.bias && a.bias[e] != a.bias[e]);
    top = v > top ? v : top;
  }
  for (int o = 32; o > 0; o >>= 1) top = fmax(top, __shfl_xor(top, o, 64));
  bad = __any(bad);
  if (!SIGMOID) {
    for (int e = lane; e < a.E; e += 64) sum += exp((double)(float)l[e] - top);
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  }
  auto score = [&](int e) {
    const double v = (double)(float)l[e];
    return SIGMOID ? 1.0 / (1.0 + exp(-v)) : exp(v - top) / sum;
  };
  if (bad) {
    for (int s = lane; s < a.top_k; s += 64) {
      a.ids[t * a.top_k + s] = s < a.E ? s : -1;
      a.weights[t * a.top_k + s] = s < a.E ? __builtin_nanf("") : 0.0f;
    }
    return;
  }
  const bool sums = a.n_group > 1 && a.group_top == 2;
  for (int e = lane; e < a.E; e += 64) {
    const double v = (double)(float)l[e];
    val[e] = v == -inf ? -inf : a.bias ? score(e) + (double)a.bias[e] : sums ? score(e) : v;
  }
  __syncthreads();
  if (a.n_group > 1) {
    const int size = a.E / a.n_group;
    for (int g = lane; g < a.n_group; g += 64) {
      double v1 = -inf, v2 = -inf;
      for (int e = g * size; e < (g + 1) * size; e++) {
        const double v = val[e];
        if (v > v1) {
          v2 = v1;
          v1 = v;
        } else if (v > v2) {
          v2 = v;
        }
      }
      grp[g] = a.group_top == 2 && v2 != -inf ? v1 + v2 : v1;
    }
    __syncthreads();
    for (int e = lane; e < a.E; e += 64) {
      const int g = e / size;
      int before = 0;
      for (int h = 0; h < a.n_group; h++) before += grp[h] > grp[g] || (grp[h] == grp[g] && h < g);
      if (before >= a.topk_group)
        val[e] = -inf;
      else if (sums && !a.bias)
        val[e] = (double)(float)l[e];
    }
    __syncthreads();
  }
  double w = 0, total = 0;
  for (int s = 0; s < a.top_k; s++) {
    double v = -inf;
    int i = a.E;
    for (int e = lane; e < a.E; e += 64)
      if (val[e] > v) {
        v = val[e];
        i = e;
      }
    for (int o = 32; o > 0; o >>= 1) best_of(v, i, o);
    const bool none = v == -inf;
    const double sc = none ? 0.0 : score(i);
    total += sc;
    if (lane == s) {
      w = sc;
      a.ids[t * a.top_k + s] = none ? -1 : i;
    }
    __syncthreads();
    if (lane == 0 && !none) val[i] = -inf;
    __syncthreads();
  }
  if (lane < a.top_k) {
    if (a.renorm) w = total == 0 ? 0.0 : w / total;
    a.weights[t * a.top_k + lane] = (float)(w * (double)a.scale);
  }
}

template <int TYPE>
int launch_route_as(int score, const RouteArgs& a, int64_t T, hipStream_t s) {
  hipLaunchKernelGGL(score == BQM_SIGMOID ? (k_route<TYPE, true>) : (k_route<TYPE, false>), dim3((unsigned)T), dim3(64), 0, s, a);
  return launch_status();
}

}  // namespace

int launch_route(int score, int type, const void* logits, int64_t stride, const float* bias, int64_t T, int E, int n_group,
                 int topk_group, int group_top, int top_k, int renorm, float scale, int32_t* ids, float* weights, hipStream_t s) {
  const RouteArgs a{logits, stride, bias, E, n_group, topk_group, group_top, top_k, renorm, scale, ids, weights};
  return type == BQM_F32   ? launch_route_as<BQM_F32>(score, a, T, s)
         : type == BQM_F16 ? launch_route_as<BQM_F16>(score, a, T, s)
                           : launch_route_as<BQM_BF16>(score, a, T, s);
}

}  // namespace bqm
