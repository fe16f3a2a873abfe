// Routing to experts (kernel and launcher; included by repack.hip).
//
// A token's E values lie in the registers of G lanes, V neighbouring experts a lane: sixteen lanes a
// token (four tokens a wave) where there are tokens enough to fill the chip, since a reduction over
// sixteen lanes takes four DPP steps and serves four tokens; all 64 lanes otherwise.  Each of the
// top_k rounds takes the largest value and, of equal ones, the lowest index.
//
// Between neighbours in the order of the real numbers an id hangs on the last bits of a score: fp32
// scores would swap them now and then.  So the order is that of 64-bit scores, but up to 256 experts
// the rounds go by fp32 keys, whose last eight bits name the expert, and take two experts more than
// asked for; these few are then put in order by their 64-bit scores, which the weights need anyway.
// What the keys leave open (a third candidate, or a closed group, nearer than the keys are exact; a
// softmax with a bias, whose 64-bit scores need all experts) the wave selects again in 64 bits.  16-bit
// logits without a bias leave the last bits free: their keys are exact.
//
// Vector instructions bind the kernel (sigmoid with a bias: 990 for a wave's four tokens, the vector
// units busy 85 % of the time), so: a round subtracts the last key and takes the largest of
// the differences in 32 bits that wrap round, 24 instructions for a lane's sixteen keys where
// striking out the key taken had 40; groups are compared by DPP rotations; a bias comes by way of
// LDS (from memory, a lane's sixteen apart, 14.7 us).  Measured (16384 tokens, 256 experts, top-8):
// without a bias 5.9 us, sigmoid with a bias 9.3, in groups 11 to 14 (the rare wave that selects again
// ends last; 20 where a bias is -infinity, whose size counts in the groups' margin); with 64 bits
// throughout 10, 22 and 25.  Sorting each lane's keys and merging the
// lanes' sorted lists instead of rounds: 7.8, 14.7, 18.3, where these rounds took 6.4, 15.0, 20.4.
#pragma once

#include <type_traits>

#include "mxfp4.h"

namespace bqm {
namespace {

struct RouteArgs {
  const void* logits;
  int64_t stride;
  const float* bias;
  int T, E, n_group, size, topk_group, group_top, top_k, renorm, vec;  // size: of a group
  float scale;
  int32_t* ids;
  float* weights;
};

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
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, x)));
}
template <int G, typename T, typename F>
__device__ __forceinline__ T reduce(T v, F&& f) {
  v = f(v, dpp<0xB1>(v));   // quad_perm 1 0 3 2
  v = f(v, dpp<0x4E>(v));   // quad_perm 2 3 0 1
  v = f(v, dpp<0x141>(v));  // row_half_mirror
  v = f(v, dpp<0x140>(v));  // row_mirror
  if constexpr (G == 64) {
    v = f(v, __shfl_xor(v, 16, 64));
    v = f(v, __shfl_xor(v, 32, 64));
  }
  return v;
}

template <int N, typename F>  // f(N), ..., f(1) as constants
__device__ __forceinline__ void count_down(F&& f) {
  f(std::integral_constant<int, N>{});
  if constexpr (N > 1) count_down<N - 1>(f);
}

// e^x by x = n ln 2 + r, |r| <= ln 2 / 2, and the Taylor series of e^r to r^13 / 13! (the next term
// is below 2^-57): within two steps of 64 bits, in half the operations of the library's, which the
// scores of 256 experts make felt.  x in [-1000, 1024 ln 2].
__device__ __forceinline__ double exp64(double x) {
  const double n = __builtin_rint(x * 0x1.71547652b82fep0);
  double r = fma(n, -0x1.62e42fefa39efp-1, x);
  r = fma(n, -0x1.abc9e3b39803fp-56, r);
  double p = 1.0 / 6227020800.0;
  constexpr double c[] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0, 1.0 / 5040.0,
                          1.0 / 720.0,       1.0 / 120.0,      1.0 / 24.0,      1.0 / 6.0,      0.5,           1.0,
                          1.0};
#pragma unroll
  for (int k = 0; k < 13; k++) p = fma(p, r, c[k]);
  return __builtin_ldexp(p, (int)n);
}
// 1 / x for x in [1, 2^1024): the hardware's estimate and two Newton steps.
__device__ __forceinline__ double rcp64(double x) {
  double y = __builtin_amdgcn_rcp(x);
  y = fma(fma(-x, y, 1.0), y, y);
  return fma(fma(-x, y, 1.0), y, y);
}
// 1 / (1 + e^-x); where e^-x passes the range of 64 bits (x below -1024 ln 2), 0.
__device__ __forceinline__ double sigmoid64(float x) {
  constexpr double kEnd = 0x1.62e42fefa39efp+9;
  const double l = x;
  const double s = rcp64(1.0 + exp64(fmin(fmax(-l, -kEnd), kEnd)));
  return l < -kEnd ? 0.0 : s;
}

// BIAS: the order is that of scores with their bias, 64 bits; without it that of the logits as they
// are, fp32.
template <int TYPE, bool SIGMOID, bool BIAS, int G, int V, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_route(RouteArgs a) {
  typedef typename mx::Elem<TYPE>::T Elem;
  typedef std::conditional_t<BIAS, double, float> Key;
  constexpr int kTokens = WAVES * 64 / G;  // of a workgroup
  constexpr int kVec = 16 / sizeof(Elem);
  __shared__ double val_lds[kTokens][V * G];  // values, or each lane's two largest
  __shared__ double grp_lds[kTokens][BQM_ROUTE_MAX_GROUPS];  // and the candidates' ids after that
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
  if constexpr (BIAS && G == 16) {  // by way of LDS: straight from memory a load's lanes are 4 V bytes apart
    float* all = reinterpret_cast<float*>(val_lds);
    for (int e = threadIdx.x; e < V * G; e += WAVES * 64) all[e] = e < a.E ? a.bias[e] : 0.0f;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; v++) bias[v] = all[e0 + v];
    __syncthreads();
  } else {
#pragma unroll
    for (int v = 0; v < V; v++) bias[v] = BIAS && e0 + v < a.E ? a.bias[e0 + v] : 0.0f;
  }
  // the row's maximum and whether anything in it is no number
  float top = -__builtin_inff();
  bool odd = false;
#pragma unroll
  for (int v = 0; v < V; v++) {
    top = __builtin_fmaxf(top, x[v]);
    odd = odd || __builtin_isunordered(x[v], BIAS ? bias[v] : x[v ^ (V > 1)]);
  }
  if (!SIGMOID && top == __builtin_inff()) odd = true;
  const int bad = reduce<G>((int)odd, [](int p, int q) { return p | q; });
  const bool sums = a.n_group > 1 && a.group_top == 2, scored = BIAS || sums;
  if (!SIGMOID) top = reduce<G>(top, [](float p, float q) { return __builtin_fmaxf(p, q); });
  // lane s % G keeps slot s, and its place in the order
  constexpr int kKept = (BQM_QMV_ID_MAX_TOPK + 2 + G - 1) / G;
  int kept[kKept], place[kKept];
  double w[kKept];
  auto keep = [&](int s, int id) {
#pragma unroll
    for (int k = 0; k < kKept; k++)
      if (s == k * G + lane) kept[k] = id;
  };
  // The groups that stay open, one bit each, from the lanes' values of type T; near: set where two
  // groups are within `margin` (negative: never).
  const int size = a.size;
  const bool whole = size % V == 0 && V > 1;  // a lane's experts are of one group
  auto open_groups = [&](auto zero, auto&& value, decltype(zero) margin, bool& near) {
    typedef decltype(zero) T;
    T* vals = reinterpret_cast<T*>(val_lds[at]);
    T* sums2 = reinterpret_cast<T*>(grp_lds[at]);
    T v1 = (T)-inf, v2 = (T)-inf;
    auto take = [&](T v) {  // the largest and the second largest so far
      if constexpr (sizeof(T) == 4)
        v2 = __builtin_amdgcn_fmed3f(v1, v2, v);
      else
        v2 = v > v1 ? v1 : v > v2 ? v : v2;
      v1 = v > v1 ? v : v1;
    };
    if (whole) {
#pragma unroll
      for (int v = 0; v < V; v++) take(value(v));
      vals[2 * lane] = v1;
      vals[2 * lane + 1] = v2;
    } else {
#pragma unroll
      for (int v = 0; v < V; v++) vals[e0 + v] = value(v);
    }
    mx::wave_turn();  // a token's lanes are of one wave
    const int each = whole ? size / V * 2 : size;
    for (int g = lane; g < a.n_group; g += G) {
      v1 = v2 = (T)-inf;
      for (int e = g * each; e < (g + 1) * each; e++) take(vals[e]);
      sums2[g] = a.group_top == 2 && v2 != (T)-inf ? v1 + v2 : v1;
    }
    mx::wave_turn();
    uint64_t open = 0;
    bool close = false;
    for (int g = 0; g < a.n_group; g += G) {
      const int h = g + lane;
      int before = 0;
      if (h < a.n_group) {
        const T w = sums2[h];
        for (int k = 0; k < a.n_group; k++) {
          const T u = sums2[k];
          before += u > w || (u == w && k < h);
          close = close || (margin >= 0 && k != h && u != (T)-inf && !(__builtin_fabs((double)u - (double)w) > margin));
        }
      }
      const uint64_t b = __ballot(h < a.n_group && before < a.topk_group);
      open |= (G == 64 ? b : b >> (threadIdx.x % 64 / G * G) & ((1ull << (G % 64)) - 1)) << g;
    }
    mx::wave_turn();  // the next pass writes there again
    near = near || close;
    return open;
  };
  // The same for sixteen lanes a token whose groups are 1, 2, 4, 8 or 16 of them, fp32: whether the
  // group of this lane stays open, without LDS.
  const int lanes = size / V;  // of a group
  const bool rows = G == 16 && whole && lanes > 0 && (lanes & (lanes - 1)) == 0;
  auto own_open = [&](auto&& value, float margin, bool& near) {
    float v1 = -__builtin_inff(), v2 = v1;
#pragma unroll
    for (int v = 0; v < V; v++) {
      v2 = __builtin_amdgcn_fmed3f(v1, v2, value(v));
      v1 = __builtin_fmaxf(v1, value(v));
    }
    auto join = [&](float o1, float o2) {
      v2 = __builtin_fmaxf(__builtin_fminf(v1, o1), __builtin_fmaxf(v2, o2));
      v1 = __builtin_fmaxf(v1, o1);
    };
    if (lanes > 1) join(dpp<0xB1>(v1), dpp<0xB1>(v2));  // as in reduce
    if (lanes > 2) join(dpp<0x4E>(v1), dpp<0x4E>(v2));
    if (lanes > 4) join(dpp<0x141>(v1), dpp<0x141>(v2));
    if (lanes > 8) join(dpp<0x140>(v1), dpp<0x140>(v2));
    const float w = a.group_top == 2 && v2 != -__builtin_inff() ? v1 + v2 : v1;
    const int g = lane >> __builtin_ctz(lanes);
    int before = 0;  // groups before this one
    count_down<15>([&](auto n) {
      constexpr int kTurn = 0x120 + decltype(n)::value;  // row_ror
      if ((decltype(n)::value & (lanes - 1)) != 0) return;
      const float u = dpp<kTurn>(w);
      const int h = dpp<kTurn>(g);  // here, where all lanes are active
      before += u > w || (u == w && h < g);
    });
    // open and closed ones are told apart where the lowest open value is above the highest closed one
    const bool in = before < a.topk_group;
    const float low = reduce<G>(in ? w : __builtin_inff(), [](float p, float q) { return __builtin_fminf(p, q); });
    const float high = reduce<G>(in ? -__builtin_inff() : w, [](float p, float q) { return __builtin_fmaxf(p, q); });
    near = near || (margin >= 0 && high > -__builtin_inff() && !(low - high > margin));
    return in;
  };
  // f(v, whether the group of expert e0 + v is open)
  auto for_open = [&](uint64_t open, auto&& f) {
    int g = e0 < a.E ? e0 / size : 0, rest = e0 - g * size;
    if (whole) {
      const bool in = open >> (g & 63) & 1;
#pragma unroll
      for (int v = 0; v < V; v++) f(v, in);
    } else {
#pragma unroll
      for (int v = 0; v < V; v++) {
        f(v, open >> (g & 63) & 1);
        const bool turn = ++rest == size;
        g += turn;
        rest = turn ? 0 : rest;
      }
    }
  };
  // e^(x - top), 0 where that is below the range
  auto power = [&](float f) {
    const double d = (double)f - (double)top;
    return d < -746.0 ? 0.0 : exp64(fmax(d, -746.0));
  };
  double rtotal = 1;  // 1 / the softmax's sum, where that counts
  auto scores64 = [&](double (&score)[V]) {
    double total = 0;
#pragma unroll
    for (int v = 0; v < V; v++) {
      score[v] = x[v] == -__builtin_inff() ? 0.0 : SIGMOID ? sigmoid64(x[v]) : power(x[v]);
      total += score[v];
    }
    if constexpr (!SIGMOID) {
      total = reduce<G>(total, [](double p, double q) { return p + q; });
      rtotal = total > 0 ? rcp64(total) : 0.0;  // 0 only where every expert is masked
#pragma unroll
      for (int v = 0; v < V; v++) score[v] *= rtotal;
    }
  };
#pragma unroll
  for (int k = 0; k < kKept; k++) {
    kept[k] = -1;
    place[k] = k * G + lane;
  }
  bool again = true, weighed = false;
  if constexpr (V * G <= 256) {
    // The fp32 pass.  A sigmoid is within kOff of the real one: the product x log2 e and v_exp_f32 move
    // e^-x by 1.25 |x| + 2 steps of 2^-24 of it, which s (1 - s) |x| <= 0.23 makes 0.8 steps of 1; the
    // sum, v_rcp_f32 add 3: below 2^-22.  A softmax's terms and its sum of 256 (16 in turn, then a
    // tree) and its reciprocal: 27 steps of 2^-24, below 2^-19.
    constexpr float kOff = SIGMOID ? 0x1p-22f : 0x1p-19f, kLog2e = 0x1.715476p+0f;
    again = false;
    float score[V], total = 0;
    if (scored) {
#pragma unroll
      for (int v = 0; v < V; v++) {
        score[v] = SIGMOID ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x[v] * kLog2e))
                   : x[v] > -__builtin_inff() ? __builtin_amdgcn_exp2f((x[v] - top) * kLog2e)
                                              : 0.0f;
        total += score[v];
      }
      if (!SIGMOID) {
        total = __builtin_amdgcn_rcpf(reduce<G>(total, [](float p, float q) { return p + q; }));
#pragma unroll
        for (int v = 0; v < V; v++) score[v] *= total;
      }
    }
    float val[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
      val[v] = x[v] > -__builtin_inff() ? BIAS ? score[v] + bias[v] : x[v] : -__builtin_inff();
    }
    if (a.n_group > 1) {
      // each of the two values of a sum is kOff off and rounded (2^-24 of up to 1 + most), the sum too
      // (2^-23 of that); twice for two groups.  Logits are exact.
      float most = 0;
#pragma unroll
      for (int v = 0; v < V; v++) most = BIAS ? __builtin_fmaxf(most, __builtin_fabsf(bias[v])) : 0.0f;
      if (BIAS) most = reduce<G>(most, [](float p, float q) { return __builtin_fmaxf(p, q); });
      const float margin = scored ? 4.0f * (kOff + 0x1p-23f * (1 + most)) : -1.0f;
      // Sums of such biases can leave the range of fp32, and an infinite sum says nothing of its place:
      // below, it equals that of a group without an expert.
      bool near = sums && most > 0x1p126f;  // 2 (1 + 2^126) is far inside
      auto value = [&](int v) { return !BIAS && sums && val[v] > -__builtin_inff() ? score[v] : val[v]; };
      uint64_t open = 0;
      bool own = true;
      if (rows)
        own = own_open(value, margin, near);
      else
        open = open_groups(0.0f, value, margin, near);
      const bool again64 = __any(near && bad == 0);  // groups nearer than fp32 tells: by their 64-bit values
      if (again64) {
        double exact[V];
        scores64(exact);
        open = open_groups(0.0, [&](int v) { return val[v] == -__builtin_inff() ? -inf : BIAS ? exact[v] + (double)bias[v] : exact[v]; }, -1.0,
                           near);
      }
      if (rows && !again64) {
#pragma unroll
        for (int v = 0; v < V; v++) val[v] = own ? val[v] : -__builtin_inff();
      } else {
        for_open(open, [&](int v, bool in) { val[v] = in ? val[v] : -__builtin_inff(); });
      }
    }
    // Keys: the value's bits in the order of unsigned numbers, the last eight 255 - e, which orders equal
    // ones and says whose they are.  A 16-bit value leaves those bits free.
    constexpr bool kExact = !BIAS && sizeof(Elem) == 2;
    constexpr uint32_t kLast = 255;
    constexpr uint32_t kNone = 0x007FFFFFu;  // of -infinity
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
      const uint32_t u = __float_as_uint(val[v] + 0.0f);  // -0 is 0
      key[v] = ((u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) & ~kLast) | (kLast - (e0 + v));
    }
    auto none = [&](uint32_t k) { return (k | kLast) <= (kNone | kLast); };
    auto id_of = [&](uint32_t k) {
      const int e = (int)(kLast - (k & kLast));
      return !none(k) && e < a.E ? e : -1;
    };
    const int rounds = a.top_k + (kExact ? 0 : 2);
    // Two keys are as far apart as the real values but for kOff each (with a bias), a rounding each and
    // the last bits, which take less than 256 steps of 2^-23 from either.
    auto apart = [&](uint32_t k, uint32_t l) {
      auto value = [](uint32_t o) {
        o &= ~kLast;
        return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xFFFFFFFFu));
      };
      const float f = value(k), g = value(l), span = __builtin_fabsf(f) > __builtin_fabsf(g) ? __builtin_fabsf(f) : __builtin_fabsf(g);
      return f - g > (BIAS ? 2 * kOff : 0.0f) + span * (257 * 0x1p-23f);
    };
    constexpr bool kRank = !kExact && (SIGMOID || !BIAS);  // 64-bit values of a few experts alone
    // A key less the one taken last, in 32 bits that wrap round: the keys below it come out above the
    // rest, so that the largest difference is the next key's and nothing has to be struck out.
    uint32_t best = 0, last = 0;
#pragma unroll
    for (int k = 0; k < kKept; k++) {
      uint32_t slot = 0;  // the key of this lane's slot
      for (int s = k * G; s < rounds && s < (k + 1) * G; s++) {
        uint32_t mine = key[0] - best;
#pragma unroll
        for (int v = 1; v < V; v++) mine = key[v] - best > mine ? key[v] - best : mine;
        best += (uint32_t)reduce<G>((int)mine, [](int p, int q) { return (uint32_t)p > (uint32_t)q ? p : q; });
        slot = lane == s - k * G ? best : slot;
        if constexpr (kRank) {  // the last candidate has to lie below the last wanted
          if (s == a.top_k - 1) last = best;
        } else if constexpr (!kExact) {  // each below the one before it
          if (s > 0 && s <= a.top_k && !none(best) && !apart(last, best)) again = true;
          last = best;
        }
      }
      kept[k] = kRank || k * G + lane < a.top_k ? id_of(slot) : -1;
    }
    if constexpr (kRank) again = !none(best) && !apart(last, best);
    if constexpr (kRank) {
      weighed = true;
      int* ids = reinterpret_cast<int*>(grp_lds[at]);
      static_assert(sizeof(grp_lds[0]) >= (BQM_QMV_ID_MAX_TOPK + 2) * sizeof(int) && V * G >= BQM_QMV_ID_MAX_TOPK + 2, "room");
      double val[kKept];
#pragma unroll
      for (int k = 0; k < kKept; k++) {
        w[k] = 0;
        val[k] = -inf;
        if (k * G >= rounds) continue;
        const float f = kept[k] >= 0 ? (float)l[kept[k]] : 0.0f;
        w[k] = kept[k] < 0 ? 0.0 : SIGMOID ? sigmoid64(f) : 0.0;
        val[k] = kept[k] < 0 ? -inf : BIAS ? w[k] + (double)a.bias[kept[k]] : (double)f;
        if (place[k] < rounds) {
          val_lds[at][place[k]] = val[k];
          ids[place[k]] = kept[k];
        }
      }
      mx::wave_turn();
#pragma unroll
      for (int k = 0; k < kKept; k++) place[k] = kept[k] < 0 || bad != 0 ? k * G + lane : 0;
      for (int s = 0; s < rounds; s++) {
        const double u = val_lds[at][s];
        const int j = ids[s];
#pragma unroll
        for (int k = 0; k < kKept; k++)
          if (k * G < rounds) place[k] += kept[k] >= 0 && j >= 0 && bad == 0 && (u > val[k] || (u == val[k] && j < kept[k]));
      }
      mx::wave_turn();
    }
    again = __any(again && bad == 0);
  }
  double score[V];
  if ((again && scored) || (!SIGMOID && !a.renorm)) scores64(score);
  if (again) {
    weighed = false;
#pragma unroll
    for (int k = 0; k < kKept; k++) {
      kept[k] = -1;
      place[k] = k * G + lane;
    }
    // no NaN among the keys: it would be neither above nor below the others (its token is `bad`)
    Key key[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
      if constexpr (BIAS) {
        const double k = score[v] + (double)bias[v];
        key[v] = x[v] > -__builtin_inff() && k > -inf ? k : -inf;
      } else {
        key[v] = x[v] > -__builtin_inff() ? x[v] : -__builtin_inff();
      }
    }
    if (a.n_group > 1) {
      bool near = false;
      const uint64_t open = open_groups(
          0.0, [&](int v) { return BIAS ? (double)key[v] : key[v] == (Key)-inf ? -inf : sums ? score[v] : (double)key[v]; }, -1.0, near);
      for_open(open, [&](int v, bool in) { key[v] = in ? key[v] : (Key)-inf; });
    }
    for (int s = 0; s < a.top_k; s++) {
      Key best = key[0];
#pragma unroll
      for (int v = 1; v < V; v++) best = key[v] > best ? key[v] : best;
      best = reduce<G>(best, [](Key p, Key q) { return p > q ? p : q; });
      int i = 1 << 30;
#pragma unroll
      for (int v = V - 1; v >= 0; v--) i = key[v] == best ? e0 + v : i;
      i = reduce<G>(i, [](int p, int q) { return p < q ? p : q; });
#pragma unroll
      for (int v = 0; v < V; v++) key[v] = e0 + v == i ? (Key)-inf : key[v];
      keep(s, best > (Key)-inf && i < a.E ? i : -1);
    }
  }
  double chosen = 0;
#pragma unroll
  for (int k = 0; k < kKept; k++) {
    if (!(weighed && SIGMOID)) {
      w[k] = 0;
      if (k * G >= a.top_k + 2) continue;
      const float f = kept[k] >= 0 ? (float)l[kept[k]] : 0.0f;
      w[k] = kept[k] < 0 ? 0.0 : SIGMOID ? sigmoid64(f) : power(f) * rtotal;
    }
    chosen += place[k] < a.top_k ? w[k] : 0.0;
  }
  if (a.renorm) chosen = reduce<G>(chosen, [](double p, double q) { return p + q; });
#pragma unroll
  for (int k = 0; k < kKept; k++) {
    const int s = place[k];
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
  constexpr int kWaves = G * V > 1024 ? 1 : 4, kTokens = kWaves * 64 / G;
  auto* k = score == BQM_SIGMOID ? (a.bias ? k_route<TYPE, true, true, G, V, kWaves> : k_route<TYPE, true, false, G, V, kWaves>)
                                 : (a.bias ? k_route<TYPE, false, true, G, V, kWaves> : k_route<TYPE, false, false, G, V, kWaves>);
  hipLaunchKernelGGL(k, dim3((unsigned)((a.T + kTokens - 1) / kTokens)), dim3(kWaves * 64), 0, s, a);
  return launch_status();
}

// Sixteen lanes a token from 1024 tokens on (16384 x 128, top-8: 4.6 us), where that fills the chip's
// units; below, 64 lanes a token end sooner (one token of 256 experts with a bias 4.4 us, in groups 6.3; 512 in
// groups 6.9; with 64 bits throughout 5.7, 7.9 and 8.7).  Above 256 experts the keys have no room for the
// expert: 64 bits throughout, and the same instance for 257 as for 1024 (16384 x 384 or x 512: 34 us without
// a bias, 67 with one, 76 in groups; x 1024 with a bias 70).
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
  const RouteArgs a{logits, stride, bias, (int)T, E, n_group, n_group > 1 ? E / n_group : 1, topk_group, group_top, top_k, renorm, vec, scale, ids, weights};
  return type == BQM_F32   ? launch_route_type<BQM_F32>(score, a, s)
         : type == BQM_F16 ? launch_route_type<BQM_F16>(score, a, s)
                           : launch_route_type<BQM_BF16>(score, a, s);
}

}  // namespace bqm
