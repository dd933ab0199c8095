// route.hip -- scores, choice and weights of tokens' experts, and their gradient
// (include/sgemm_route.h).
//
// One wave has a token: expert e in register e / 64 of lane e % 64.  The time is that
// of the steps that pick one expert after the other, each a maximum over the wave: in
// registers and by moves between lanes (DPP), six instructions, where an exchange
// through LDS would wait for it six times over.
//
// The picks are those of the formulas in double precision, but nearly always found in
// single precision: scores and sums there are off by a known bound, and picks whose
// values are further apart than twice that, from each other and from the next, are the
// right ones.  Where some are not (one token in some hundreds), picking goes on until
// the next value is apart, and what was picked is put in order in double precision;
// where it is groups that are close, these are chosen again in double precision.
// Without bias and groups the logits are compared, which is exact.
//
// By graph replay, top 8 of 64 experts for one token: 2.9 us; of 256 experts for 8192
// tokens, bfloat16: 7.7 us; sigmoid with a bias 9.9; with 8 groups too 13.2 (28.4 with
// everything in double precision and exchanges through LDS), 662 vector instructions a
// wave, eight waves on every SIMD and 4 cycles an instruction: 8.8 us of issue; reading the
// logits would take 0.9.
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

// A wave's n values, the rest -infinity.  Every lane loads, from the nearest element
// there is: behind a test of its own each 2-byte load would be waited for before the
// next one goes out.
template <bool BF16, int EPL>
__device__ __forceinline__ void load_row(const void *x, long at, int n, float v[EPL]) {
  const int lane = threadIdx.x % kWave;
#pragma unroll
  for (int i = 0; i < EPL; ++i) v[i] = load1<BF16>(x, at + min(i * kWave + lane, n - 1));
#pragma unroll
  for (int i = 0; i < EPL; ++i) v[i] = i * kWave + lane < n ? v[i] : -__builtin_inff();
}

// op over the lanes by moves inside rows of 16 and from row to row; the result in
// every lane.  A lane without a neighbour there combines with `rest`.
template <class Op>
__device__ __forceinline__ int wave_reduce(int v, Op op, int rest) {
  v = op(v, __builtin_amdgcn_update_dpp(rest, v, 0x111, 0xf, 0xf, false));  // 1 lane before
  v = op(v, __builtin_amdgcn_update_dpp(rest, v, 0x112, 0xf, 0xf, false));  // 2
  v = op(v, __builtin_amdgcn_update_dpp(rest, v, 0x114, 0xf, 0xf, false));  // 4
  v = op(v, __builtin_amdgcn_update_dpp(rest, v, 0x118, 0xf, 0xf, false));  // 8
  v = op(v, __builtin_amdgcn_update_dpp(rest, v, 0x142, 0xa, 0xf, false));  // the row before's last
  v = op(v, __builtin_amdgcn_update_dpp(rest, v, 0x143, 0xc, 0xf, false));  // lane 31
  return __builtin_amdgcn_readlane(v, kWave - 1);
}
__device__ __forceinline__ unsigned wave_max(unsigned v) {
  return (unsigned)wave_reduce(
      (int)v, [](int a, int b) { return (int)max((unsigned)a, (unsigned)b); }, 0);
}
__device__ __forceinline__ float wave_max(float v) {
  return __int_as_float(wave_reduce(
      __float_as_int(v),
      [](int a, int b) { return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b))); },
      __float_as_int(-__builtin_inff())));
}
__device__ __forceinline__ float wave_sum(float v) {
  return __int_as_float(wave_reduce(
      __float_as_int(v),
      [](int a, int b) { return __float_as_int(__int_as_float(a) + __int_as_float(b)); }, 0));
}
// Through LDS: for the rare token.
__device__ __forceinline__ double wave_sum(double v) {
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

__device__ __forceinline__ unsigned order_key(float v) {
  if (v != v) return ~0u;
  if (v == kMinusInf) return 0;
  const unsigned b = __float_as_uint(v + 0.f);  // -0 as 0
  return b ^ ((int)b < 0 ? ~0u : 1u << 31);
}
__device__ __forceinline__ float key_value(unsigned k) {
  return __uint_as_float((int)k < 0 ? k ^ (1u << 31) : ~k);
}

// Highest and second highest of a group.
template <class T>
struct Top2 {
  T first, second;
  __device__ __forceinline__ void add(const Top2 &o) {
    second = fmax(fmin(first, o.first), fmax(second, o.second));
    first = fmax(first, o.first);
  }
  __device__ __forceinline__ void add(T v) { add(Top2{v, (T)kMinusInf}); }
  __device__ __forceinline__ T sum(int count) const {
    return count > 1 && second != (T)kMinusInf ? first + second : first;
  }
};
__device__ __forceinline__ float exchanged(float v, int d) { return __shfl_xor(v, d); }
__device__ __forceinline__ double exchanged(double v, int d) { return __shfl_xor(v, d); }
template <int CTRL>
__device__ __forceinline__ Top2<float> moved(const Top2<float> &t) {
  auto move = [](float v) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
  };
  return {move(t.first), move(t.second)};
}

// Top2 of group lane / share among the wave's values in `row`; `share` lanes have a
// group, each every share-th value, and put theirs together.
template <class T>
__device__ __forceinline__ Top2<T> group_top2(const RouteArgs &p, const T *row) {
  const int lane = threadIdx.x % kWave, share = p.group_share, g = lane / share;
  const int size = p.experts / p.groups;
  Top2<T> best{(T)kMinusInf, (T)kMinusInf};
  if (g < p.groups)
    for (int i = lane % share; i < size; i += share) best.add(row[g * size + i]);
  if constexpr (sizeof(T) == 4) {
    // Lanes 1, 2, 4 and 8 away; where quads (eights) agree, the mirrored one will do.
    if (share > 1) best.add(moved<0xb1>(best));
    if (share > 2) best.add(moved<0x4e>(best));
    if (share > 4) best.add(moved<0x141>(best));
    if (share > 8) best.add(moved<0x140>(best));
    for (int d = 16; d < share; d *= 2)
      best.add(Top2<T>{exchanged(best.first, d), exchanged(best.second, d)});
  } else {
    for (int d = 1; d < share; d *= 2)
      best.add(Top2<T>{exchanged(best.first, d), exchanged(best.second, d)});
  }
  return best;
}

__device__ __forceinline__ unsigned long long lane_key(unsigned long long k, int lane) {
  return (unsigned long long)(unsigned)__builtin_amdgcn_readlane((int)(k >> 32), lane) << 32 |
         (unsigned)__builtin_amdgcn_readlane((int)k, lane);
}

// What is compared, in double precision; -infinity for experts that cannot be picked.
// total: the sum of a softmax's exponentials.
template <int EPL>
__device__ __forceinline__ void values_in_double(const RouteArgs &p, const float l[EPL], float top,
                                                 double v[EPL]) {
  const int lane = threadIdx.x % kWave;
  double total = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    v[i] = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - (double)top);
    total += v[i];
  }
  if (!p.sigmoid) {
    total = wave_sum(total);
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] /= total;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * kWave + lane;
    if (p.bias && e < p.experts) v[i] += (double)p.bias[e];
    if (l[i] == kMinusInf) v[i] = kMinusInf;
  }
}

// The lanes of the groups that are kept, in double precision.  row: room for EPL * 64
// values.
template <int EPL>
__device__ __forceinline__ unsigned long long groups_in_double(const RouteArgs &p,
                                                               const float l[EPL], float top,
                                                               double *row) {
  const int lane = threadIdx.x % kWave, share = p.group_share, g = lane / share;
  double v[EPL];
  values_in_double<EPL>(p, l, top, v);
  wave_fence();
#pragma unroll
  for (int i = 0; i < EPL; ++i) row[i * kWave + lane] = v[i];
  wave_fence();
  const Top2<double> best = group_top2(p, row);
  const unsigned long long score = g < p.groups ? order_key(best.sum(p.group_top)) : 0;
  int before = 0;
  for (int o = 0; o < p.groups; ++o) {
    const unsigned long long other = lane_key(score, o * share);
    before += other > score || (other == score && o < g);
  }
  wave_fence();
  return __ballot(g < p.groups && before < p.keep);
}

// The picks in double precision, lane j's the j-th, -1 for none.  lanes: of the groups
// that are kept.
template <int EPL>
__device__ __forceinline__ int picks_in_double(const RouteArgs &p, const float l[EPL], float top,
                                               unsigned long long lanes) {
  const int lane = threadIdx.x % kWave;
  double v[EPL];
  values_in_double<EPL>(p, l, top, v);
  unsigned long long key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * kWave + lane;
    key[i] = order_key(v[i]);
    if (p.groups > 1 && e < p.experts && !(lanes >> (p.by_size(e) * p.group_share) & 1)) key[i] = 0;
  }
  int pick = -1;
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
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e == i * kWave + lane) key[i] = 0;
    if (lane == j) pick = e;
  }
  return pick;
}

template <bool BF16, int EPL>
__global__ void __launch_bounds__(kTokens *kWave) route_kernel(RouteArgs p) {
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const long t = (long)blockIdx.x * kTokens + wave;
  if (t >= p.tokens) return;  // whole waves: there is no barrier
  __shared__ double room[kTokens][EPL * kWave];
  float *const row = reinterpret_cast<float *>(room[wave]);  // logits, or what is compared

  float l[EPL], bias[EPL];
  load_row<BF16, EPL>(p.logits, t * p.ldl, p.experts, l);
#pragma unroll
  for (int i = 0; i < EPL; ++i) bias[i] = 0.f;
  if (p.bias) load_row<false, EPL>(p.bias, 0, p.experts, bias);
  const bool by_logits = !p.bias && p.groups == 1;
  float top = l[0];
  bool odd = false;  // the row has a NaN, or softmax of an infinity
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    top = fmaxf(top, l[i]);
    odd |= l[i] != l[i] || (!p.sigmoid && l[i] == -kMinusInf);
  }
  odd = __ballot(odd) != 0;
  float total = 1.f;
  if (!p.sigmoid) {
    top = wave_max(top);
    if (top == kMinusInf) top = 0.f;
  }
  unsigned key[EPL];
  if (by_logits && (p.sigmoid || p.renormalize)) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = order_key(l[i]);
  } else {
    float s[EPL];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] = p.sigmoid ? __builtin_amdgcn_rcpf(1.f + __expf(-l[i])) : __expf(l[i] - top);
      sum += s[i];
    }
    if (!p.sigmoid) {
      sum = wave_sum(sum);
      total = sum == 0.f ? 1.f : sum;  // 0: no expert is enabled
    }
    const float inverse = 1.f / total;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float c = l[i] == kMinusInf ? kMinusInf : (p.sigmoid ? s[i] : s[i] * inverse) + bias[i];
      key[i] = order_key(by_logits ? l[i] : c);
    }
  }

  // What a score may be off by: a sigmoid s by s (1 - s) (|l| + 2) 2^-24 for the
  // exponential, below 2^-24, and by 3 2^-24 for the sum and the reciprocal; a softmax by
  // 28 roundings in its sum too; and the sum with the bias by 2^-24 of itself, which is
  // counted where values are compared.
  const float off = p.sigmoid ? 0x1p-21f : 0x1p-18f;
  auto apart = [&](float a, float b, float off) {  // a is above b for certain
    return a - b > 2.f * off + 0x1p-22f * (fabsf(a) + fabsf(b));
  };
  unsigned long long lanes = ~0ull;  // of the groups that are kept
  if (p.groups > 1) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      row[i * kWave + lane] = key[i] == 0 ? kMinusInf : key_value(key[i]);
    wave_fence();
    const int share = p.group_share, g = lane / share;
    const Top2<float> best = group_top2(p, row);
    const float sum = best.sum(p.group_top);
    const bool some = g < p.groups && best.first != kMinusInf;  // the group has an expert
    const unsigned score = some ? order_key(sum) : 0;
    int before = 0;  // groups that come before the lane's
    for (int o = 0; o < p.groups; ++o) {
      const unsigned other = (unsigned)__builtin_amdgcn_readlane((int)score, o * share);
      before += other > score || (other == score && o < g);
    }
    const bool mine = g < p.groups && before < p.keep;
    lanes = __ballot(mine);
    // A sum is off by what its two terms are off by, and three roundings that go by the
    // terms' sizes: where the terms cancel, these are not small against the sum.  The
    // lowest of the kept and the highest of the others have to be further apart, and
    // every sum inside single precision's range.
    const float second = p.group_top > 1 && best.second != kMinusInf ? fabsf(best.second) : 0.f;
    const float error = 2.f * off + 0x1p-22f * (fabsf(best.first) + second);
    const unsigned low = ~wave_max(mine && some ? ~order_key(sum - error) : 0u);
    const unsigned high = wave_max(some && !mine ? order_key(sum + error) : 0u);
    if (__ballot(some && !(fabsf(sum) < -kMinusInf)) != 0 || (high != 0 && low <= high))
      lanes = groups_in_double<EPL>(p, l, top, room[wave]);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = i * kWave + lane;
      if (e < p.experts && !(lanes >> (p.by_size(e) * share) & 1)) key[i] = 0;
    }
    wave_fence();
  }

  int pick = -1;  // lane j's: the j-th
  int picked = 0;
  bool close = false;  // some are not apart
  float last = 0.f;
  for (; picked < kWave; ++picked) {
    if (by_logits && picked == p.topk) break;
    unsigned best = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = max(best, key[i]);
    const unsigned all = wave_max(best);
    if (all == 0) break;
    if (!by_logits) {
      const float value = key_value(all);
      const bool near = picked > 0 && !apart(last, value, off);
      if (picked >= p.topk && !near) break;
      close |= near;
      last = value;
    }
    // The lowest index that has it.
    bool found = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (found) continue;
      const unsigned long long have = __ballot(key[i] == all);
      if (have) {
        const int from = __builtin_ctzll(have);
        if (lane == from) key[i] = 0;
        if (lane == picked) pick = i * kWave + from;
        found = true;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) row[i * kWave + lane] = l[i];
  wave_fence();
  if (close && picked < kWave) {
    // The picked in order, in double precision: lane j's place among them.
    double all = 1.0;
    if (!p.sigmoid) {
      all = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) all += exp((double)l[i] - (double)top);
      all = wave_sum(all);
    }
    unsigned long long mine = 0;
    if (pick >= 0) {
      const double v = row[pick];
      mine = order_key((p.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - (double)top) / all) +
                       (p.bias ? (double)p.bias[pick] : 0.0));
    }
    int place = 0;
    for (int j = 0; j < picked; ++j) {
      const unsigned long long other =
          (unsigned long long)(unsigned)__builtin_amdgcn_readlane((int)(mine >> 32), j) << 32 |
          (unsigned)__builtin_amdgcn_readlane((int)mine, j);
      const int e = __builtin_amdgcn_readlane(pick, j);
      place += other > mine || (other == mine && e < pick);
    }
    int *const order = reinterpret_cast<int *>(row + EPL * kWave);
    if (pick >= 0) order[place] = pick;
    wave_fence();
    pick = lane < picked && lane < p.topk ? order[lane] : -1;
  } else if (!by_logits && picked == kWave) {
    pick = picks_in_double<EPL>(p, l, top, lanes);
  }
  if (lane >= p.topk) pick = -1;
  const float x = pick >= 0 ? row[pick] : kMinusInf;
  float w;
  if (p.sigmoid) {
    w = 1.f / (1.f + expf(-x));
  } else {
    // Renormalised: the softmax of the picks alone, in which nothing underflows.
    w = expf(x - (p.renormalize ? wave_max(x) : top));
    if (!p.renormalize) w /= total;
  }
  if (pick < 0) w = 0.f;
  if (p.renormalize) {
    const float sum = wave_sum(w);
    w = sum == 0.f ? 0.f : w / sum;
  }
  w = pick < 0 ? 0.f : w * p.scale;
  if (odd) w = __uint_as_float(0x7fc00000u);
  if (lane < p.topk) {
    p.picks[t * p.topk + lane] = pick;
    p.weights[t * p.topk + lane] = w;
  }
}

// Bound by the launch, then by memory: 8192 x 256, top 8, bfloat16 4.8 us by graph replay
// for 9 MB (1.8 at a large copy's rate).  Only a softmax that is not renormalised reads
// the whole row; otherwise the picked logits are enough.
//
// dl = the gradient of the logits; with g = scale dweights and p = the renormalised
// scores, for the picked
//   softmax                  s (g - sum g s), where g = 0 for others
//   softmax, renormalised    p (g - sum g p), 0 for others
//   sigmoid                  g s (1 - s), 0 for others
//   sigmoid, renormalised    p (g - sum g p) (1 - s), 0 for others.
template <bool BF16, int EPL>
__global__ void __launch_bounds__(kTokens *kWave) route_backward_kernel(RouteBackArgs p) {
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
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
    load_row<BF16, EPL>(p.logits, t * p.ldl, p.experts, s);
#pragma unroll
    for (int i = 0; i < EPL; ++i) top = fmaxf(top, s[i]);
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
