// route.hip -- scores, choice and weights of tokens' experts, and their gradient
// (include/sgemm_route.h).
//
// One wave has a token: expert e in register e / 64 of lane e % 64.  What the
// choice compares is held in 64 bits, so that the picks are those of the
// formulas and not of an exponential's rounding.
#include "mxfp4.hpp"
#include "route.hpp"

namespace sgemm {

namespace {

constexpr int kTokens = 4;  // tokens (waves) of a work-group

template <bool BF16>
__device__ __forceinline__ float load1(const void *x, long at) {
  if constexpr (BF16)
    return __uint_as_float((unsigned)static_cast<const unsigned short *>(x)[at] << 16);
  else
    return static_cast<const float *>(x)[at];
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ unsigned long long wave_max(unsigned long long v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) {
    const unsigned long long o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}

// The wave's LDS accesses keep their order; this keeps the compiler's.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

constexpr float kMinusInf = -__builtin_inff();

// Unsigned numbers that order as the doubles do, NaNs above them; 0, below all,
// for -infinity, which cannot be picked.
__device__ __forceinline__ unsigned long long order_key(double v) {
  if (v != v) return ~0ull;
  if (v == (double)kMinusInf) return 0;
  const long long b = __double_as_longlong(v + 0.0);  // -0 as 0
  return (unsigned long long)b ^ (b < 0 ? ~0ull : 1ull << 63);
}

template <bool BF16, int EPL>
__global__ void __launch_bounds__(kTokens *kWave) route_kernel(RouteArgs p) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const long t = (long)blockIdx.x * kTokens + wave;
  if (t >= p.tokens) return;  // whole waves: there is no barrier
  __shared__ double group_c[kTokens][EPL * kWave];

  float l[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * kWave + lane;
    l[i] = e < p.experts ? load1<BF16>(p.logits, t * p.ldl + e) : kMinusInf;
  }
  float top = l[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) top = fmaxf(top, l[i]);
  top = wave_max(top);
  const double m = top == kMinusInf ? 0.0 : (double)top;
  double s[EPL], total = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    s[i] = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - m);
    total += s[i];
  }
  total = wave_sum(total);
  if (!p.sigmoid) {
    if (total == 0) total = 1;  // no expert is enabled
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] /= total;
  }
  unsigned long long key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * kWave + lane;
    double c = l[i];
    if (l[i] != kMinusInf && (p.bias || p.groups > 1))
      c = s[i] + (p.bias && e < p.experts ? (double)p.bias[e] : 0.0);
    key[i] = order_key(c);
    group_c[wave][e] = c;
  }

  if (p.groups > 1) {
    wave_fence();
    const int size = p.experts / p.groups;
    unsigned long long score = 0;
    if (lane < p.groups) {
      double first = kMinusInf, second = kMinusInf;
      for (int i = 0; i < size; ++i) {
        const double c = group_c[wave][lane * size + i];
        if (c > first || c != c) {
          second = first;
          first = c;
        } else if (c > second) {
          second = c;
        }
      }
      if (p.group_top > 1 && second != (double)kMinusInf) first += second;
      score = order_key(first);
    }
    int before = 0;  // groups that come before the lane's
    for (int g = 0; g < p.groups; ++g) {
      const unsigned long long o = __shfl(score, g);
      before += o > score || (o == score && g < lane);
    }
    const unsigned long long kept = __ballot(lane < p.groups && before < p.keep);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = i * kWave + lane;
      if (e < p.experts && !(kept >> (e / size) & 1)) key[i] = 0;
    }
  }

  int pick = -1;  // lane j's: the j-th
  float chosen = 0.f;
  for (int j = 0; j < p.topk; ++j) {
    unsigned long long best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < EPL; ++i) {
      at = key[i] > best ? i : at;
      best = key[i] > best ? key[i] : best;
    }
    const unsigned long long all = wave_max(best);
    if (all == 0) break;
    int e = best == all ? at * kWave + lane : 1 << 20;
#pragma unroll
    for (int d = 32; d > 0; d /= 2) e = min(e, __shfl_xor(e, d));
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e == i * kWave + lane) {
        key[i] = 0;
        mine = p.sigmoid || !p.renormalize ? (float)s[i] : l[i];
      }
    mine = __shfl(mine, e % kWave);
    if (lane == j) {
      pick = e;
      chosen = mine;
    }
  }
  float w = chosen;
  if (p.renormalize) {
    if (!p.sigmoid) {  // the softmax of the picks alone: nothing underflows
      const float high = wave_max(pick >= 0 ? chosen : kMinusInf);
      w = pick >= 0 ? expf(chosen - high) : 0.f;
    }
    const float sum = wave_sum(w);
    w = sum == 0.f ? 0.f : w / sum;
  }
  if (total != total) w = __uint_as_float(0x7fc00000u);  // the row has a NaN, or softmax of infinity
  if (lane < p.topk) {
    p.picks[t * p.topk + lane] = pick;
    p.weights[t * p.topk + lane] = w * p.scale;
  }
}

// dl = the gradient of the logits; with g = scale dweights and p = the renormalised
// scores, for the picked
//   softmax                  s (g - sum g s), where g = 0 for others
//   softmax, renormalised    p (g - sum g p), 0 for others
//   sigmoid                  g s (1 - s), 0 for others
//   sigmoid, renormalised    p (g - sum g p) (1 - s), 0 for others.
template <bool BF16, int EPL>
__global__ void __launch_bounds__(kTokens *kWave) route_backward_kernel(RouteBackArgs p) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const long t = (long)blockIdx.x * kTokens + wave;
  if (t >= p.tokens) return;  // whole waves: there is no barrier
  __shared__ float picked_g[kTokens][EPL * kWave];
  float *const row = picked_g[wave];
#pragma unroll
  for (int i = 0; i < EPL; ++i) row[i * kWave + lane] = 0.f;

  const bool whole = !p.sigmoid && !p.renormalize;  // all experts share the gradient
  int pick = lane < p.topk ? p.picks[t * p.topk + lane] : -1;
  if (pick >= p.experts) pick = -1;
  float l = pick >= 0 ? load1<BF16>(p.logits, t * p.ldl + pick) : kMinusInf;
  if (l == kMinusInf) pick = -1;
  const float g = pick >= 0 ? p.dweights[t * p.topk + lane] * p.scale : 0.f;

  float s[EPL], dot = 0.f;
  wave_fence();
  if (whole) {
    float top = kMinusInf;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = i * kWave + lane;
      s[i] = e < p.experts ? load1<BF16>(p.logits, t * p.ldl + e) : kMinusInf;
      top = fmaxf(top, s[i]);
    }
    top = wave_max(top);
    if (top == kMinusInf) top = 0.f;
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) total += s[i] = expf(s[i] - top);
    total = wave_sum(total);
    const float inverse = total > 0.f || total != total ? 1.f / total : 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] *= inverse;
    dot = wave_sum(pick >= 0 ? g * (expf(l - top) * inverse) : 0.f);
    if (pick >= 0) row[pick] = g;
  } else {
    // 1 - s as sigmoid(-l), which keeps its digits where s is close to 1.
    float score = 0.f, d = 0.f;
    if (p.sigmoid) {
      score = pick >= 0 ? 1.f / (1.f + expf(-l)) : 0.f;
    } else {
      const float high = wave_max(l);
      score = pick >= 0 ? expf(l - high) : 0.f;
    }
    const float rest = p.sigmoid ? 1.f / (1.f + expf(l)) : 1.f;
    if (p.renormalize) {
      const float sum = wave_sum(score);
      score = sum == 0.f ? 0.f : score / sum;
      d = score * (g - wave_sum(g * score)) * rest;
    } else {
      d = g * score * rest;
    }
    if (pick >= 0) row[pick] = d;
  }
  wave_fence();
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * kWave + lane;
    if (e >= p.experts) break;
    const float v = whole ? s[i] * (row[e] - dot) : row[e];
    const long at = t * p.ldd + e;
    if constexpr (BF16)
      static_cast<__bf16 *>(p.dlogits)[at] = (__bf16)v;
    else
      static_cast<float *>(p.dlogits)[at] = v;
  }
}

// f with the registers of a lane as a constant, as many as the experts take.
template <class F>
hipError_t with_registers(int experts, F &&f) {
  if (experts <= 64) return f(std::integral_constant<int, 1>());
  if (experts <= 128) return f(std::integral_constant<int, 2>());
  if (experts <= 256) return f(std::integral_constant<int, 4>());
  if (experts <= 512) return f(std::integral_constant<int, 8>());
  return f(std::integral_constant<int, 16>());
}

}  // namespace

hipError_t launch_route(const RouteArgs &p, bool bf16, hipStream_t s) {
  return with_registers(p.experts, [&](auto R) {
    const dim3 grid((unsigned)((p.tokens + kTokens - 1L) / kTokens)), block(kTokens * kWave);
    if (bf16)
      hipLaunchKernelGGL((route_kernel<true, decltype(R)::value>), grid, block, 0, s, p);
    else
      hipLaunchKernelGGL((route_kernel<false, decltype(R)::value>), grid, block, 0, s, p);
    return hipGetLastError();
  });
}

hipError_t launch_route_backward(const RouteBackArgs &p, bool bf16, hipStream_t s) {
  return with_registers(p.experts, [&](auto R) {
    const dim3 grid((unsigned)((p.tokens + kTokens - 1L) / kTokens)), block(kTokens * kWave);
    if (bf16)
      hipLaunchKernelGGL((route_backward_kernel<true, decltype(R)::value>), grid, block, 0, s, p);
    else
      hipLaunchKernelGGL((route_backward_kernel<false, decltype(R)::value>), grid, block, 0, s, p);
    return hipGetLastError();
  });
}

}  // namespace sgemm
