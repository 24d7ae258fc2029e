// One AdamW step over a list of tensors, states in fp32 or in e4m3 with a scale for each
// run of 128 (moe_adamw in moe.h).
//
// Bound by memory: a bf16 parameter with its master, fp32 states and a bf16 gradient
// move 28 bytes an element, a bf16 parameter with e4m3 states 10.  75.5 M elements of the first kind 357 us (5.9 TB/s),
// 604 M of the second 1020 (6.0; 990 to 1050 a call, and 1030 to 1150 in the first twenty after a pause); 200 000 with fp32
// states 6 us (a launch).
//
// The list travels in the kernel arguments (kMaxAdam entries a launch), so nothing is
// copied to the device and a captured graph holds its own list.  A tensor is cut into chunks
// of kChunk elements from its first.  With codes a thread has eight neighbouring elements, so that sixteen
// lanes hold a run: its largest value is four lane moves away.  Loads take 16 bytes at any element's address.  The
// step's coefficients (two powers of the betas in 64 bits) are computed by every thread for itself, some 100 instructions
// beside a chunk's 1000: a launch to compute them once costs more.
#include <algorithm>
#include <cmath>
#include <new>
#include <type_traits>

#include "moe_args.h"
#include "moe_fp8_codec.h"

namespace moe {
namespace {

constexpr int kMaxAdam = 46;  // entries a launch
constexpr int kAdamThreads = 256;
constexpr int kChunk = 8 * kAdamThreads;
constexpr uint32_t kMaxAdamBlocks = (1u << 24) - 1;  // HIP counts a launch's threads in 32 bits
// Lists past this go by with nontemporal loads and stores: 2.1 GB of fp32 states 425 -> 398 us, 6 GB with codes 1464 ->
// 1334 (either alone gains nothing), 300 MB in two launches 111 -> 106; below, the gradients and the parameters may be
// in the memory-side cache (256 MB) for this call and the next forward.
constexpr uint64_t kStreamBytes = 64ull << 20;
// With codes a workgroup takes two chunks of such a list (6 GB: 1054 -> 1016 us; four 1073): its coefficients
// cost a tenth of a chunk's instructions.  With fp32 states one (359 us; two 368), and never a few workgroups that
// step through the list (4096: 1334 and 398 us), which drift apart.

struct AdamList {
  void* param[kMaxAdam];
  float* master[kMaxAdam];
  const void* grad[kMaxAdam];
  void *m[kMaxAdam], *v[kMaxAdam];
  float *ms[kMaxAdam], *vs[kMaxAdam];
  int64_t n[kMaxAdam];
  float decay[kMaxAdam];
  uint32_t first[kMaxAdam + 1];  // chunks before each entry
  uint8_t kind[kMaxAdam];        // bit 0: fp32 param, bit 1: fp32 gradient
  int count;
};

struct AdamStep {
  const float *lr, *norm;
  const int32_t* step;
  double log_b1, log_b2;
  float b1, b2, a1, a2, eps, max_norm;
};
static_assert(sizeof(AdamList) + sizeof(AdamStep) <= 3584, "kernel arguments hold the list");

// The step's numbers, the same in every thread.
struct Coef {
  float c, b1, b2, a1, a2;    // clipping factor, betas and 1 - betas
  float lr, rate, root, eps;  // lr, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  bool none;                  // nothing to do
};
__device__ __forceinline__ Coef coefficients(const AdamStep& s) {
  Coef k;
  const float lr = *s.lr;
  const int t = *s.step;
  k.c = 1.f;
  k.none = t < 1;
  if (s.norm != nullptr) {
    const float nm = *s.norm;
    k.none |= !(fabsf(nm) < INFINITY);
    if (!(nm <= s.max_norm)) k.c = s.max_norm / nm;
  }
  k.b1 = s.b1; k.b2 = s.b2;
  k.a1 = s.a1; k.a2 = s.a2;
  k.lr = lr;
  k.rate = lr / float(1. - exp64(double(t) * s.log_b1));
  k.root = 1.f / sqrtf(float(1. - exp64(double(t) * s.log_b2)));
  k.eps = s.eps;
  return k;
}

// N neighbouring elements (4 or 8) from p, `n` of which are there (zeros behind them).
template <class T, int N>
struct Piece {
  static constexpr int WORDS = N * int(sizeof(T)) / 4;
  uint32_t w[WORDS];
  template <bool STREAM>
  __device__ __forceinline__ void get(const T* p, int n) {
    if (n >= N) {
      if constexpr (WORDS == 2) {
        const uint2 v = fetch8<STREAM>(p);
        w[0] = v.x; w[1] = v.y;
      } else {
#pragma unroll
        for (int k = 0; k < WORDS / 4; ++k) {
          const uint4 v = fetch16<STREAM>(p + k * 16 / sizeof(T));
          w[4 * k] = v.x; w[4 * k + 1] = v.y; w[4 * k + 2] = v.z; w[4 * k + 3] = v.w;
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < WORDS; ++k) w[k] = 0;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) {
          if constexpr (sizeof(T) == 2) w[i / 2] |= uint32_t(p[i]) << (16 * (i & 1));
          else w[i] = __float_as_uint(p[i]);
        }
    }
  }
  __device__ __forceinline__ void values(float (&f)[N]) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < WORDS; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int k = 0; k < WORDS; ++k) f[k] = __uint_as_float(w[k]);
    }
  }
  template <bool STREAM>
  static __device__ __forceinline__ void put(T* p, int n, const float (&f)[N]) {
    uint32_t o[WORDS];
#pragma unroll
    for (int k = 0; k < WORDS; ++k) {
      if constexpr (sizeof(T) == 2) o[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
      else o[k] = __float_as_uint(f[k]);
    }
    if (n >= N) {
      if constexpr (WORDS == 2) {
        keep8<STREAM>(p, make_uint2(o[0], o[1]));
      } else {
#pragma unroll
        for (int k = 0; k < WORDS / 4; ++k)
          keep16<STREAM>(p + k * 16 / sizeof(T), make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) {
          if constexpr (sizeof(T) == 2) p[i] = uint16_t(o[i / 2] >> (16 * (i & 1)));
          else p[i] = f[i];
        }
    }
  }
};
// Eight e4m3 codes.
struct Codes {
  uint2 a;
  template <bool STREAM>
  __device__ __forceinline__ void get(const uint8_t* p, int n) {
    if (n >= 8) {
      a = fetch8<STREAM>(p);
    } else {
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) w[i / 4] |= uint32_t(p[i]) << (8 * (i & 3));
      a = make_uint2(w[0], w[1]);
    }
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int w = int(k ? a.y : a.x);
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
      f[4 * k] = lo[0]; f[4 * k + 1] = lo[1]; f[4 * k + 2] = hi[0]; f[4 * k + 3] = hi[1];
    }
  }
  template <bool STREAM>
  static __device__ __forceinline__ void put(uint8_t* p, int n, const uint2& c) {
    if (n >= 8) {
      keep8<STREAM>(p, c);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = uint8_t((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
  }
};

// The moments, each product and sum rounded to fp32 (no fused multiply-add: the codes of the next
// step are those of these numbers, and a definition that names each rounding can be computed elsewhere).
__device__ __forceinline__ void moments(float g, float& m, float& v, const Coef& k) {
#pragma clang fp contract(off)
  m = k.b1 * m + k.a1 * g;
  v = k.b2 * v + k.a2 * (g * g);
}

// Codes of x[i] / s, the quotient rounded to fp32, of eight values a lane.  Both x rc (1 - d) and x rc (1 + d) are
// coded, with rc an approximation of 1 / s: the conversion is monotone, so where the codes are equal they are the
// quotient's.  Elsewhere (a border between codes lies within some ulps: one wave in a hundred) `exact` gives the
// quotients.  d covers the reciprocal's ulp (2 u), a rounding each of rc (1 +- d), of the product and of the
// quotient, and the error that x itself has (2 u more and a rounding, for a root): 5 u, or 8 u.
template <class F>
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], float s, float d, F&& exact) {
  const float rc = __builtin_amdgcn_rcpf(s), lo = rc * (1.f - d), hi = rc * (1.f + d);
  uint2 c = make_uint2(pack_e4m3x4(x[0] * lo, x[1] * lo, x[2] * lo, x[3] * lo),
                       pack_e4m3x4(x[4] * lo, x[5] * lo, x[6] * lo, x[7] * lo));
  const uint2 h = make_uint2(pack_e4m3x4(x[0] * hi, x[1] * hi, x[2] * hi, x[3] * hi),
                             pack_e4m3x4(x[4] * hi, x[5] * hi, x[6] * hi, x[7] * hi));
  if (((c.x ^ h.x) | (c.y ^ h.y)) != 0 || !(s >= 0x1p-120f)) {  // below, the reciprocal may be infinite
    float y[8];
    // a scale of a few of the smallest numbers is rounded by up to half, and the quotient is then past 448, where the
    // conversion would give NaN
#pragma unroll
    for (int i = 0; i < 8; ++i)
      y[i] = __builtin_elementwise_minimum(__builtin_elementwise_maximum(exact(i), -448.f), 448.f);  // a NaN stays
    c = make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
  }
  return c;
}
// A run's eight values in each of its sixteen lanes; returns the scale.  Of a run that has shrunk to half of 448 of the
// smallest numbers the quotient is 0, and x / 0 would be NaN for its zeros and for all of it in the next step: its scale is 1,
// whose codes are zeros.
__device__ __forceinline__ float code8(const float (&x)[8], uint2& codes) {
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(x[i]));
  am = max16(am);
  const float of = am / 448.f, s = of == 0.f ? 1.f : of;
  codes = codes_of(x, s, 0x1p-21f, [&](int i) { return x[i] / s; });
  return s;
}
// The same of the square roots of v, r their approximations within an ulp (2^-75 at least, so that only 0 has a scale of 0);
// what is positive has a positive code.
__device__ __forceinline__ float code8_root(const float (&v)[8], const float (&r)[8], uint2& codes) {
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) am = fmaxf(am, v[i]);
  am = max16(am);
  const float s = am == 0.f ? 1.f : sqrtf(am) / 448.f;
  codes = codes_of(r, s, 0x1p-20f, [&](int i) { return sqrtf(v[i]) / s; });
  // codes are below 0x80: a byte + 0x7f has its top bit clear where the code is 0
  if ((((codes.x + 0x7f7f7f7fu) & (codes.y + 0x7f7f7f7fu)) & 0x80808080u) != 0x80808080u) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = v[i] > 0.f ? fmaxf(sqrtf(v[i]) / s, 0x1p-9f) : v[i];
    codes = make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
  }
  return s;
}

// This thread's elements of chunk c of entry i: with codes eight neighbouring ones (sixteen lanes a run), with fp32
// states two pieces of four, so that a wave's loads of 16 bytes lie side by side.  WHOLE: the chunk ends inside
// the tensor.
template <bool E4M3, bool STREAM, bool WHOLE, class P, class G>
__device__ __forceinline__ void step_chunk(const AdamList& L, int i, uint32_t c, const Coef& k) {
  constexpr int N = E4M3 ? 8 : 4, PIECES = 8 / N;
  const int64_t base = int64_t(c) * kChunk;
  const G* const grad = static_cast<const G*>(L.grad[i]) + base;
  P* const param = static_cast<P*>(L.param[i]) + base;
  float* const master = L.master[i] == nullptr ? nullptr : L.master[i] + base;
  const bool own = master == nullptr;
  const float shrink = 1.f - k.lr * L.decay[i];
  const int64_t rest = L.n[i] - base;
  const int there = WHOLE || rest > kChunk ? kChunk : int(rest);
  Piece<G, N> g8[PIECES];
  Piece<P, N> p8[PIECES];
  Piece<float, N> w8[PIECES], m8[PIECES], v8[PIECES];
  Codes mc, vc;
  float ms = 0.f, vs = 0.f;
#pragma unroll
  for (int q = 0; q < PIECES; ++q) {
    const uint32_t e = (q * kAdamThreads + threadIdx.x) * N;
    const int n = WHOLE ? N : there - int(e);
    g8[q].template get<STREAM>(grad + e, n);
    if (own) p8[q].template get<STREAM>(param + e, n);
    else w8[q].template get<STREAM>(master + e, n);
    if constexpr (E4M3) {
      mc.get<STREAM>(static_cast<const uint8_t*>(L.m[i]) + base + e, n);
      vc.get<STREAM>(static_cast<const uint8_t*>(L.v[i]) + base + e, n);
      if (n > 0) {
        ms = (L.ms[i] + (base >> 7))[e >> 7];
        vs = (L.vs[i] + (base >> 7))[e >> 7];
      }
    } else {
      m8[q].template get<STREAM>(static_cast<const float*>(L.m[i]) + base + e, n);
      v8[q].template get<STREAM>(static_cast<const float*>(L.v[i]) + base + e, n);
    }
  }
#pragma unroll
  for (int q = 0; q < PIECES; ++q) {
    const uint32_t e = (q * kAdamThreads + threadIdx.x) * N;
    const int n = WHOLE ? N : there - int(e);
    float g[N], p[N], m[N], v[N], r[N];
    g8[q].values(g);
    if (own) p8[q].values(p);
    else w8[q].values(p);
    if constexpr (E4M3) {
      mc.values(m);
      vc.values(v);
    } else {
      m8[q].values(m);
      v8[q].values(v);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if constexpr (E4M3) {
        m[j] *= ms;
        v[j] *= vs;
        v[j] *= v[j];
      }
      moments(g[j] * k.c, m[j], v[j], k);
      r[j] = __builtin_amdgcn_sqrtf(v[j]);  // within an ulp; 0 for what is below the normal numbers
    }
    if (k.eps < 0x1p-30f) {  // where such a root (below 2^-63) would count beside eps
#pragma unroll
      for (int j = 0; j < N; ++j) r[j] = v[j] < 0x1p-126f ? sqrtf(v[j]) : r[j];
    }
    float by[N];
#pragma unroll
    for (int j = 0; j < N; ++j) by[j] = m[j] * __builtin_amdgcn_rcpf(__builtin_fmaf(r[j], k.root, k.eps));
    if (k.eps < 0x1p-126f) {  // where v is 0 so is the denominator to the reciprocal, which would make 0 / eps NaN
#pragma unroll
      for (int j = 0; j < N; ++j) by[j] = m[j] / __builtin_fmaf(r[j], k.root, k.eps);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] = __builtin_fmaf(p[j], shrink, -k.rate * by[j]);
    if (!own) Piece<float, N>::template put<STREAM>(master + e, n, p);
    Piece<P, N>::template put<STREAM>(param + e, n, p);
    if constexpr (E4M3) {
      uint2 codes;
      ms = code8(m, codes);
      Codes::put<STREAM>(static_cast<uint8_t*>(L.m[i]) + base + e, n, codes);
      vs = code8_root(v, r, codes);
      Codes::put<STREAM>(static_cast<uint8_t*>(L.v[i]) + base + e, n, codes);
      if ((threadIdx.x & 15) == 0 && n > 0) {
        (L.ms[i] + (base >> 7))[e >> 7] = ms;
        (L.vs[i] + (base >> 7))[e >> 7] = vs;
      }
    } else {
      Piece<float, N>::template put<STREAM>(static_cast<float*>(L.m[i]) + base + e, n, m);
      Piece<float, N>::template put<STREAM>(static_cast<float*>(L.v[i]) + base + e, n, v);
    }
  }
}

template <bool E4M3, bool STREAM>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(AdamList L, AdamStep s) {
  const Coef k = coefficients(s);
  if (k.none) return;
  const uint32_t total = L.first[L.count];
  int i = 0;
  for (uint32_t c = blockIdx.x; c < total; c += gridDim.x) {
    while (c >= L.first[i + 1]) ++i;
    const uint32_t at = c - L.first[i];
    auto go = [&](auto whole) __attribute__((always_inline)) {
      constexpr bool W = decltype(whole)::value;
      if (L.kind[i] == 3) step_chunk<E4M3, STREAM, W, float, float>(L, i, at, k);
      else if (L.kind[i] == 2) step_chunk<E4M3, STREAM, W, uint16_t, float>(L, i, at, k);
      else if (L.kind[i] == 1) step_chunk<E4M3, STREAM, W, float, uint16_t>(L, i, at, k);
      else step_chunk<E4M3, STREAM, W, uint16_t, uint16_t>(L, i, at, k);
    };
    if (c + 1 < L.first[i + 1]) go(std::true_type{});
    else go(std::false_type{});
  }
}

bool float_type(int32_t t) { return t == MOE_TYPE_F32 || t == MOE_TYPE_BF16; }

int check_params(const moe_adamw_desc& d, const moe_adamw_param* p, int32_t count) {
  const bool e4m3 = d.state_type == MOE_TYPE_E4M3;
  int rc = MOE_OK;
  for (int32_t i = 0; i < count; ++i) {
    const moe_adamw_param& q = p[i];
    if (q.n < 0 || q.reserved != 0 || !float_type(q.param_type) || !float_type(q.grad_type) ||
        !std::isfinite(q.weight_decay) || (q.master != nullptr && q.param_type == MOE_TYPE_F32))
      return MOE_EINVAL;
    if (q.n == 0) continue;
    if (q.n >= (int64_t(1) << 34)) return MOE_EUNSUPPORTED;  // 46 of them stay below 2^31 chunks
    if (q.param == nullptr || q.grad == nullptr || q.m == nullptr || q.v == nullptr ||
        (q.m_scale != nullptr) != e4m3 || (q.v_scale != nullptr) != e4m3)
      return MOE_EINVAL;
    const size_t ss = e4m3 ? 16 : 4;
    if (!aligned_to(q.param, type_bytes(q.param_type)) || !aligned_to(q.grad, type_bytes(q.grad_type)) ||
        !aligned_to(q.master, 4) || !aligned_to(q.m, ss) || !aligned_to(q.v, ss) || !aligned_to(q.m_scale, 4) ||
        !aligned_to(q.v_scale, 4))
      rc = MOE_EALIGN;
  }
  return rc;
}

struct Part {
  uintptr_t a, b;
  bool written;
};

// Whether a buffer that the step writes overlaps another one.
int check_apart(const moe_adamw_param* p, int32_t count, bool e4m3, const void* lr, const void* step, const void* norm) {
  Part* r = new (std::nothrow) Part[size_t(count) * 7 + 3];
  if (r == nullptr) return MOE_EHIP;
  size_t m = 0;
  auto add = [&](const void* q, size_t bytes, bool written) {
    if (q != nullptr) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(q);
      r[m++] = {a, a + bytes, written};
    }
  };
  for (int32_t i = 0; i < count; ++i) {
    const size_t n = size_t(p[i].n), scales = (n + 127) / 128 * 4, state = n * (e4m3 ? 1 : 4);
    if (n == 0) continue;
    add(p[i].param, n * type_bytes(p[i].param_type), true);
    add(p[i].master, n * 4, true);
    add(p[i].grad, n * type_bytes(p[i].grad_type), false);
    add(p[i].m, state, true);
    add(p[i].v, state, true);
    add(p[i].m_scale, scales, true);
    add(p[i].v_scale, scales, true);
  }
  add(lr, 4, false);
  add(step, 4, false);
  add(norm, 4, false);
  std::sort(r, r + m, [](const Part& x, const Part& y) { return x.a < y.a; });
  // by start: a part overlaps an earlier one if that one, or one before it, ends behind its start
  int rc = MOE_OK;
  uintptr_t end = 0, end_written = 0;
  for (size_t k = 0; k < m; ++k) {
    if (r[k].a < end_written || (r[k].written && r[k].a < end)) rc = MOE_EINVAL;
    end = std::max(end, r[k].b);
    if (r[k].written) end_written = std::max(end_written, r[k].b);
  }
  delete[] r;
  return rc;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_adamw(const moe_adamw_desc* d, const moe_adamw_param* p, int32_t count, const float* lr,
                         const int32_t* step, const float* norm, float max_norm, void* stream) {
  if (d == nullptr || count < 0 || (p == nullptr && count > 0) || d->reserved != 0) return MOE_EINVAL;
  if (d->state_type != MOE_TYPE_F32 && d->state_type != MOE_TYPE_E4M3) return MOE_EINVAL;
  if (!(d->beta1 >= 0. && d->beta1 < 1.) || !(d->beta2 >= 0. && d->beta2 < 1.) || !(d->eps >= 0.) ||
      !std::isfinite(float(d->eps)))
    return MOE_EINVAL;
  if (norm != nullptr && (!(max_norm >= 0.f) || std::isinf(max_norm))) return MOE_EINVAL;
  const int rc = check_params(*d, p, count);
  if (rc && rc != MOE_EALIGN) return rc;
  if (lr == nullptr || step == nullptr) return MOE_EINVAL;
  if (rc || !aligned_to(lr, 4) || !aligned_to(step, 4) || !aligned_to(norm, 4)) return MOE_EALIGN;
  const bool e4m3 = d->state_type == MOE_TYPE_E4M3;
  if (const int bad = check_apart(p, count, e4m3, lr, step, norm)) return bad;
  AdamStep st{};
  st.lr = lr; st.norm = norm; st.step = step;
  st.b1 = float(d->beta1); st.b2 = float(d->beta2);
  st.a1 = float(1. - d->beta1); st.a2 = float(1. - d->beta2);
  st.log_b1 = std::log(d->beta1); st.log_b2 = std::log(d->beta2);
  st.eps = float(d->eps); st.max_norm = max_norm;
  hipStream_t s = static_cast<hipStream_t>(stream);
  AdamList L;
  L.count = 0;
  L.first[0] = 0;
  uint64_t bytes = 0;
  auto flush = [&]() {
    if (L.count == 0) return int(MOE_OK);
    const bool stream_it = bytes > kStreamBytes;
    const uint32_t chunks = L.first[L.count];
    const unsigned grid = std::min(e4m3 && stream_it ? (chunks + 1) / 2 : chunks, kMaxAdamBlocks);
    prof_begin("adamw", s);
    if (e4m3) {
      if (stream_it) adamw_kernel<true, true><<<grid, kAdamThreads, 0, s>>>(L, st);
      else adamw_kernel<true, false><<<grid, kAdamThreads, 0, s>>>(L, st);
    } else {
      if (stream_it) adamw_kernel<false, true><<<grid, kAdamThreads, 0, s>>>(L, st);
      else adamw_kernel<false, false><<<grid, kAdamThreads, 0, s>>>(L, st);
    }
    prof_end(s);
    L.count = 0;
    bytes = 0;
    return launched();
  };
  for (int32_t i = 0; i < count; ++i) {
    if (p[i].n == 0) continue;
    if (L.count == kMaxAdam)
      if (const int bad = flush()) return bad;
    const int k = L.count;
    L.param[k] = p[i].param; L.master[k] = p[i].master; L.grad[k] = p[i].grad;
    L.m[k] = p[i].m; L.v[k] = p[i].v; L.ms[k] = p[i].m_scale; L.vs[k] = p[i].v_scale;
    L.n[k] = p[i].n;
    L.decay[k] = p[i].weight_decay;
    L.kind[k] = uint8_t((p[i].param_type == MOE_TYPE_F32 ? 1 : 0) | (p[i].grad_type == MOE_TYPE_F32 ? 2 : 0));
    L.first[k + 1] = L.first[k] + uint32_t(ceil_div(p[i].n, kChunk));
    L.count = k + 1;
    bytes += uint64_t(p[i].n) * (type_bytes(p[i].param_type) + type_bytes(p[i].grad_type) + (p[i].master ? 4 : 0) + (e4m3 ? 2 : 8));
  }
  return flush();
}
