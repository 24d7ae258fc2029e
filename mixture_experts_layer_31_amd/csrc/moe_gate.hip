// Gate: the router's choice by sigmoid or softmax scores with a bias and groups of
// experts, the gradient of its weights into the logits, and the bias's step
// (moe_gate_fwd, moe_gate_bwd, moe_gate_bias in moe.h).
//
// The choice goes by c = fl32(s + bias).  The scores are computed in 64 bits, so that
// the rounding to fp32 decides which of two neighbours comes first and not the error of
// an fp32 exp (a sequence of 16384 tokens has some five rows where that would show).
//
// LPT lanes share a token, each with VPL of its experts in runs of four; with groups, each
// group has LPT / GP of the lanes (GP the power of two from the number of groups).
// A choice is a 64-bit key: fp32's bits in their order, then the expert from the
// highest down, below a fixed exponent, so that the 64-bit floating maximum (one
// instruction) orders keys and breaks ties.  A lane sorts its keys with a merging network
// (a maximum and a minimum a comparator); a group's score is the sum of its lanes'
// two largest; then K times the largest head of a lane is the next expert, and
// its lane moves on by one.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "moe_args.h"
#include "moe_fp8_codec.h"

namespace moe {
namespace {

constexpr int kGateThreads = 256;
constexpr int kGateMaxExperts = 1024, kGateMaxSlots = 64, kGateMaxGroups = 64;

struct GateArgs {
  const void* z;
  const float* bias;
  int64_t ld, ld_d;
  int T, E, K;
  int groups, top_groups, best;  // groups 1: none
  int each, lanes;               // experts a group, lanes a group
  bool softmax, renorm, accumulate;
  float scale;
};

// Float bits -> unsigned key with the same order (for non-NaN values), and back.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t u = __float_as_uint(z);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// A key: the order of c, then the lower of two places; 0 is behind every key.
constexpr int kPlaceBits = 10;
__device__ __forceinline__ double make_key(float c, int place) {
  const uint64_t k = (uint64_t(order_key(c)) << kPlaceBits) | uint64_t(1023 - place);
  return __longlong_as_double((long long)((1ull << 52) | k));
}
__device__ __forceinline__ int key_place(double k) { return 1023 - int(__double_as_longlong(k) & 1023); }
__device__ __forceinline__ float key_value(double k) {
  return order_value(uint32_t((unsigned long long)(__double_as_longlong(k)) >> kPlaceBits));
}

// A lane's value across an aligned group of lanes, one step: 1, 2 (the quads uniform after
// them), 4, 8 by mirrors of uniform quads and halves, 16 and 32 by the crossbar.
template <int STEP>
__device__ __forceinline__ int cross(int v) {
  if constexpr (STEP == 1) return dpp_swap1(v);
  else if constexpr (STEP == 2) return dpp_swap2(v);
  else if constexpr (STEP == 4) return dpp_mirror8(v);
  else if constexpr (STEP == 8) return dpp_mirror16(v);
  else return __shfl_xor(v, STEP, 64);
}
template <int STEP>
__device__ __forceinline__ double cross(double v) {
  const long long b = __double_as_longlong(v);
  const uint32_t lo = uint32_t(cross<STEP>(int(b))), hi = uint32_t(cross<STEP>(int(b >> 32)));
  return __longlong_as_double((long long)((uint64_t(hi) << 32) | lo));
}
template <int STEP>
__device__ __forceinline__ float cross(float v) { return __int_as_float(cross<STEP>(__float_as_int(v))); }

// f(step) for the steps below `lanes`.
template <class F>
__device__ __forceinline__ void each_step(int lanes, F&& f) {
  if (lanes > 1) f(std::integral_constant<int, 1>{});
  if (lanes > 2) f(std::integral_constant<int, 2>{});
  if (lanes > 4) f(std::integral_constant<int, 4>{});
  if (lanes > 8) f(std::integral_constant<int, 8>{});
  if (lanes > 16) f(std::integral_constant<int, 16>{});
  if (lanes > 32) f(std::integral_constant<int, 32>{});
}
template <int LPT, class T>
__device__ __forceinline__ T token_sum(T v) {
  each_step(LPT, [&](auto s) { v += cross<decltype(s)::value>(v); });
  return v;
}
template <int LPT, class T>
__device__ __forceinline__ T token_max(T v) {
  each_step(LPT, [&](auto s) { const T o = cross<decltype(s)::value>(v); v = o > v ? o : v; });
  return v;
}
template <int LPT>
__device__ __forceinline__ double key_max(double v) {
  each_step(LPT, [&](auto s) { v = __builtin_fmax(v, cross<decltype(s)::value>(v)); });
  return v;
}

// Descending, by Batcher's odd-even merging network.
template <int N>
__device__ __forceinline__ void sort_keys(double (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i) {
          const int a = i + j, b = i + j + q;
          if (b < N && a / (2 * p) == b / (2 * p)) {
            const double hi = __builtin_fmax(k[a], k[b]), lo = __builtin_fmin(k[a], k[b]);
            k[a] = hi;
            k[b] = lo;
          }
        }
}

__device__ __forceinline__ float element(const float* p) { return *p; }
__device__ __forceinline__ float element(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
struct __attribute__((packed, aligned(4))) Four32 { float v[4]; };
struct __attribute__((packed, aligned(2))) Four16 { uint32_t v[2]; };
__device__ __forceinline__ void four(const float* p, float (&f)[4]) {
  const Four32 a = *reinterpret_cast<const Four32*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = a.v[i];
}
__device__ __forceinline__ void four(const uint16_t* p, float (&f)[4]) {
  const Four16 a = *reinterpret_cast<const Four16*>(p);
  f[0] = __uint_as_float(a.v[0] << 16); f[1] = __uint_as_float(a.v[0] & 0xffff0000u);
  f[2] = __uint_as_float(a.v[1] << 16); f[3] = __uint_as_float(a.v[1] & 0xffff0000u);
}
__device__ __forceinline__ void put_four(float* p, const float (&f)[4]) {
  *reinterpret_cast<Four32*>(p) = Four32{{f[0], f[1], f[2], f[3]}};
}
__device__ __forceinline__ void put_four(uint16_t* p, const float (&f)[4]) {
  *reinterpret_cast<Four16*>(p) = Four16{{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])}};
}
__device__ __forceinline__ void put_one(float* p, float f) { *p = f; }
__device__ __forceinline__ void put_one(uint16_t* p, float f) { *p = uint16_t(pack_bf16x2(f, 0.f)); }

// LDS traffic of one wave, in order.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ double sigmoid64(float z) { return 1. / (1. + exp(-double(z))); }

template <class Z, int LPT, int VPL>
__global__ void __launch_bounds__(kGateThreads) gate_fwd_kernel(GateArgs a, int32_t* __restrict__ topk_idx,
                                                                float* __restrict__ topk_w) {
  constexpr int TOKENS = kGateThreads / LPT;
  __shared__ double s_group[TOKENS][kGateMaxGroups < LPT ? kGateMaxGroups : LPT];
  const int l = threadIdx.x & (LPT - 1), tok = threadIdx.x / LPT;
  const int64_t t = int64_t(blockIdx.x) * TOKENS + tok;
  const bool there = t < a.T;  // lanes behind the last token go along with it
  const Z* row = static_cast<const Z*>(a.z) + (there ? t : a.T - 1) * a.ld;
  // the lane's experts: g * each + e for e in runs of four
  const int g = l / a.lanes, in = l & (a.lanes - 1);
  const bool mine = g < a.groups;
  const bool fours = (a.each & 3) == 0;
  float z[VPL];
#pragma unroll
  for (int q = 0; q < VPL / 4; ++q) {
    const int e = 4 * (in + a.lanes * q);
    float f[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (mine) {
      if (fours) {
        if (e < a.each) four(row + g * a.each + e, f);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (e + r < a.each) f[r] = element(row + g * a.each + e + r);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) z[4 * q + r] = f[r];
  }
  float m = 0.f;
  double inv = 1.;
  double key[VPL];
  if (a.softmax) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, z[i]);
    m = token_max<LPT>(m);
    double sum = 0.;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      key[i] = z[i] == -INFINITY ? 0. : exp(double(z[i]) - double(m));
      sum += key[i];
    }
    sum = token_sum<LPT>(sum);
    inv = sum == 0. ? 0. : 1. / sum;
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = sigmoid64(z[i]);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 4 * (in + a.lanes * (i >> 2)) + (i & 3), at = g * a.each + e;
    const bool is = mine && e < a.each;
    double s = key[i];
    if (a.bias != nullptr && is) s += double(a.bias[at]);
    const float c = z[i] == -INFINITY ? -FLT_MAX : fmaxf(float(s), -FLT_MAX);
    key[i] = is ? make_key(c, at) : 0.;
  }
  sort_keys(key);
  if (a.top_groups < a.groups) {
    double k0 = key[0], k1 = key[1];
    each_step(a.lanes, [&](auto s) {
      const double o0 = cross<decltype(s)::value>(k0), o1 = cross<decltype(s)::value>(k1);
      k1 = __builtin_fmax(__builtin_fmin(k0, o0), __builtin_fmax(k1, o1));
      k0 = __builtin_fmax(k0, o0);
    });
    float score = key_value(k0);
    if (a.best == 2 && k1 != 0.) score += key_value(k1);
    const double own = mine ? make_key(score, g) : 0.;
    if (in == 0) s_group[tok][g] = own;
    wave_order();
    int ahead = 0;
    for (int j = 0; j < a.groups; ++j) ahead += s_group[tok][j] > own ? 1 : 0;
    if (ahead >= a.top_groups) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = 0.;
    }
  }
  double won = 0.;
  for (int k = 0; k < a.K; ++k) {
    const double top = key_max<LPT>(key[0]);
    if (l == k) won = top;
    const bool next = key[0] == top;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const double behind = i + 1 < VPL ? key[i + 1] : 0.;
      key[i] = next ? behind : key[i];
    }
  }
  double s = 0.;
  int at = 0;
  if (l < a.K) {
    at = key_place(won);
    const float x = element(row + at);
    s = a.softmax ? (x == -INFINITY ? 0. : exp(double(x) - double(m))) * inv : sigmoid64(x);
  }
  if (a.renorm) {
    const double sum = token_sum<LPT>(s);
    s = sum == 0. ? 0. : s / sum;
  }
  if (l < a.K && there) {
    topk_idx[t * a.K + l] = at;
    topk_w[t * a.K + l] = float(s * double(a.scale));
  }
}

// A token's row of the gradient at the chosen experts is put together in LDS, zero between
// tokens, and written whole.  VPL values a lane in runs of four.
template <class Z, int LPT, int VPL>
__global__ void __launch_bounds__(kGateThreads) gate_bwd_kernel(GateArgs a, const int32_t* __restrict__ topk_idx,
                                                                const float* __restrict__ dtopk_w,
                                                                Z* __restrict__ dlogits) {
  constexpr int TOKENS = kGateThreads / LPT, COLS = LPT * VPL;
  __shared__ __attribute__((aligned(16))) float s_row[TOKENS][COLS];
  const int l = threadIdx.x & (LPT - 1), tok = threadIdx.x / LPT;
  const int64_t t = int64_t(blockIdx.x) * TOKENS + tok;
  const bool there = t < a.T;
  const int64_t tt = there ? t : a.T - 1;
  const Z* row = static_cast<const Z*>(a.z) + tt * a.ld;
  int id = -1;
  float x = -INFINITY, up = 0.f;
  if (l < a.K) {
    id = topk_idx[tt * a.K + l];
    up = dtopk_w[tt * a.K + l] * a.scale;
    if (id < 0 || id >= a.E) id = -1;
    else x = element(row + id);
  }
#pragma unroll
  for (int q = 0; q < VPL / 4; ++q)
    *reinterpret_cast<float4*>(&s_row[tok][4 * (l + LPT * q)]) = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool whole = a.softmax && !a.renorm;  // every logit of the token has a gradient
  float z[VPL], dot = 0.f;
  float part = 0.f;  // this slot's gradient
  if (whole) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = 4 * (l + LPT * (i >> 2)) + (i & 3);
      z[i] = e < a.E ? element(row + e) : -INFINITY;
      m = fmaxf(m, z[i]);
    }
    m = token_max<LPT>(m);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      z[i] = z[i] == -INFINITY ? 0.f : expf(z[i] - m);
      sum += z[i];
    }
    sum = token_sum<LPT>(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < VPL; ++i) z[i] *= inv;
    part = id >= 0 ? up : 0.f;
    dot = token_sum<LPT>(id >= 0 && x != -INFINITY ? expf(x - m) * inv * up : 0.f);
  } else {
    double s = 0.;
    float m = 0.f;
    if (a.softmax) {
      m = token_max<LPT>(id >= 0 ? x : -INFINITY);
      s = id >= 0 && x != -INFINITY ? exp(double(x) - double(m)) : 0.;
    } else if (id >= 0) {
      s = sigmoid64(x);
    }
    const double rest = a.softmax ? 1. : 1. / (1. + exp(double(x)));  // 1 - s
    if (a.renorm) {
      const double sum = token_sum<LPT>(s);
      s = sum == 0. ? 0. : s / sum;
      const double mean = token_sum<LPT>(id >= 0 ? s * double(up) : 0.);
      part = id >= 0 ? float(s * rest * (double(up) - mean)) : 0.f;
    } else {
      part = id >= 0 ? float(s * rest * double(up)) : 0.f;
    }
  }
  wave_order();
  if (id >= 0) __hip_atomic_fetch_add(&s_row[tok][id], part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
  wave_order();
  if (!there) return;
  Z* out = dlogits + t * a.ld_d;
#pragma unroll
  for (int q = 0; q < VPL / 4; ++q) {
    const int e = 4 * (l + LPT * q);
    const float4 v = *reinterpret_cast<const float4*>(&s_row[tok][e]);
    float f[4] = {v.x, v.y, v.z, v.w};
    if (whole) {
#pragma unroll
      for (int r = 0; r < 4; ++r) f[r] = z[4 * q + r] == 0.f ? 0.f : z[4 * q + r] * (f[r] - dot);
    }
    if (e + 4 <= a.E) {
      if (a.accumulate) {
        float old[4];
        four(out + e, old);
#pragma unroll
        for (int r = 0; r < 4; ++r) f[r] += old[r];
      }
      put_four(out + e, f);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (e + r < a.E) put_one(out + e + r, a.accumulate ? f[r] + element(out + e + r) : f[r]);
    }
  }
}

__global__ void __launch_bounds__(1024) gate_bias_kernel(int E, const int32_t* __restrict__ counts, float step,
                                                         float* __restrict__ bias) {
  __shared__ long long red[16];
  long long sum = 0;
  for (int64_t e = threadIdx.x; e < E; e += 1024) sum += counts[e];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = 0;
  for (int w = 0; w < 16; ++w) sum += red[w];
  for (int64_t e = threadIdx.x; e < E; e += 1024) {
    const long long own = (long long)counts[e] * E;  // below 2^62
    if (own != sum) bias[e] += own < sum ? step : -step;
  }
}

// f(lanes a token, values a lane) for a lane count's worth of experts (in runs of four).
template <class F>
int with_lanes(int lpt, int vpl, F&& f) {
  using std::integral_constant;
  if (lpt == 16) {
    if (vpl <= 4) return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    if (vpl <= 8) return f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
    return f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  }
  if (vpl <= 4) return f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  if (vpl <= 8) return f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  if (vpl <= 16) return f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
  return f(integral_constant<int, 64>{}, integral_constant<int, 32>{});
}

// Values a lane with `lanes` lanes for `each` experts, in runs of four.
int values_a_lane(int each, int lanes) { return 4 * int(ceil_div(ceil_div(each, 4), lanes)); }

int check_gate(const moe_gate_desc* d) {
  if (d == nullptr) return MOE_EINVAL;
  if (d->T < 0 || d->E < 1 || d->K < 1 || d->groups < 1 || d->E % d->groups != 0 || d->top_groups < 1 ||
      d->top_groups > d->groups || d->group_best < 1 || d->group_best > 2 ||
      d->K > (long long)d->top_groups * (d->E / d->groups) || (long long)d->T * d->K >= (1LL << 31))
    return MOE_EINVAL;
  if (d->score != MOE_SCORE_SIGMOID && d->score != MOE_SCORE_SOFTMAX) return MOE_EINVAL;
  if (d->in_type != MOE_TYPE_F32 && d->in_type != MOE_TYPE_BF16) return MOE_EINVAL;
  if ((d->flags & ~(MOE_GATE_RENORM | MOE_GATE_ACCUMULATE)) != 0 || !std::isfinite(d->scale)) return MOE_EINVAL;
  if ((d->flags & MOE_GATE_ACCUMULATE) && d->in_type != MOE_TYPE_F32) return MOE_EINVAL;
  if (d->ld_logits < d->E || d->ld_dlogits < d->E) return MOE_EINVAL;
  if (d->E > kGateMaxExperts || d->T >= (1 << 26) ||  // 64 lanes a token, below 2^32 threads
      d->K > kGateMaxSlots || d->groups > kGateMaxGroups ||
      d->ld_logits >= (1LL << 40) || d->ld_dlogits >= (1LL << 40))
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

GateArgs gate_args(const moe_gate_desc& d, const void* z, const float* bias) {
  GateArgs a{};
  a.z = z;
  a.bias = bias;
  a.ld = d.ld_logits;
  a.ld_d = d.ld_dlogits;
  a.T = d.T;
  a.E = d.E;
  a.K = d.K;
  a.groups = d.top_groups < d.groups ? d.groups : 1;  // all groups: none
  a.top_groups = d.top_groups < d.groups ? d.top_groups : 1;
  a.best = d.group_best;
  a.each = d.E / a.groups;
  a.softmax = d.score == MOE_SCORE_SOFTMAX;
  a.renorm = (d.flags & MOE_GATE_RENORM) != 0;
  a.accumulate = (d.flags & MOE_GATE_ACCUMULATE) != 0;
  a.scale = d.scale;
  return a;
}

// Bytes from the first row's start to the last row's end.
size_t span(int64_t rows, int64_t cols, int64_t ld, size_t es) {
  return rows > 0 ? (size_t(rows - 1) * size_t(ld) + size_t(cols)) * es : 0;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_gate_fwd(const moe_gate_desc* d, const void* logits, const float* bias, int32_t* topk_idx,
                 float* topk_w, void* stream) {
  if (const int rc = check_gate(d)) return rc;
  if (d->T == 0) return MOE_OK;
  if (logits == nullptr || topk_idx == nullptr || topk_w == nullptr) return MOE_EINVAL;
  if (!aligned_to(logits, type_bytes(d->in_type)) || !aligned_to(bias, 4) || !aligned_to(topk_idx, 4) ||
      !aligned_to(topk_w, 4))
    return MOE_EALIGN;
  GateArgs a = gate_args(*d, logits, bias);
  int gp = 1;
  while (gp < a.groups) gp *= 2;
  // 16 lanes a token (four tokens a wave) where they hold its experts, groups and slots
  const bool few = gp <= 16 && a.K <= 16 && values_a_lane(a.each, 16 / gp) <= 16;
  const int lpt = few ? 16 : 64;
  a.lanes = lpt / gp;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const unsigned grid = unsigned(ceil_div(a.T, kGateThreads / lpt));
  prof_begin("gate_fwd", s);
  with_lanes(lpt, values_a_lane(a.each, a.lanes), [&](auto l, auto v) {
    constexpr int LPT = decltype(l)::value, VPL = decltype(v)::value;
    if (d->in_type == MOE_TYPE_F32) gate_fwd_kernel<float, LPT, VPL><<<grid, kGateThreads, 0, s>>>(a, topk_idx, topk_w);
    else gate_fwd_kernel<uint16_t, LPT, VPL><<<grid, kGateThreads, 0, s>>>(a, topk_idx, topk_w);
    return 0;
  });
  prof_end(s);
  return launched();
}

int moe_gate_bwd(const moe_gate_desc* d, const void* logits, const int32_t* topk_idx, const float* dtopk_w,
                 void* dlogits, void* stream) {
  if (const int rc = check_gate(d)) return rc;
  if (d->T == 0) return MOE_OK;
  if (logits == nullptr || topk_idx == nullptr || dtopk_w == nullptr || dlogits == nullptr) return MOE_EINVAL;
  const size_t es = type_bytes(d->in_type);
  if (!aligned_to(logits, es) || !aligned_to(topk_idx, 4) || !aligned_to(dtopk_w, 4) || !aligned_to(dlogits, es))
    return MOE_EALIGN;
  const size_t out = span(d->T, d->E, d->ld_dlogits, es), pairs = size_t(d->T) * d->K * 4;
  if (overlap(dlogits, out, logits, span(d->T, d->E, d->ld_logits, es)) || overlap(dlogits, out, topk_idx, pairs) ||
      overlap(dlogits, out, dtopk_w, pairs))
    return MOE_EINVAL;
  GateArgs a = gate_args(*d, logits, nullptr);
  const int lpt = a.K <= 16 && a.E <= 256 ? 16 : 64;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const unsigned grid = unsigned(ceil_div(a.T, kGateThreads / lpt));
  prof_begin("gate_bwd", s);
  with_lanes(lpt, values_a_lane(a.E, lpt), [&](auto l, auto v) {
    constexpr int LPT = decltype(l)::value, VPL = decltype(v)::value < 16 ? decltype(v)::value : 16;  // E <= 1024
    if (d->in_type == MOE_TYPE_F32)
      gate_bwd_kernel<float, LPT, VPL><<<grid, kGateThreads, 0, s>>>(a, topk_idx, dtopk_w, static_cast<float*>(dlogits));
    else
      gate_bwd_kernel<uint16_t, LPT, VPL><<<grid, kGateThreads, 0, s>>>(a, topk_idx, dtopk_w, static_cast<uint16_t*>(dlogits));
    return 0;
  });
  prof_end(s);
  return launched();
}

int moe_gate_bias(int32_t E, const int32_t* counts, float step, float* bias, void* stream) {
  if (E < 1 || counts == nullptr || bias == nullptr || !std::isfinite(step)) return MOE_EINVAL;
  if (!aligned_to(counts, 4) || !aligned_to(bias, 4)) return MOE_EALIGN;
  if (overlap(bias, size_t(E) * 4, counts, size_t(E) * 4)) return MOE_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  prof_begin("gate_bias", s);
  gate_bias_kernel<<<1, 1024, 0, s>>>(E, counts, step, bias);
  prof_end(s);
  return launched();
}

}  // extern "C"
