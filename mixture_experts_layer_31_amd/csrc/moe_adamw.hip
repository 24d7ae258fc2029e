// One AdamW step over a list of tensors, states in fp32 or in e4m3 with a scale for each
// run of 128 (moe_adamw in moe.h).
//
// Bound by memory: a bf16 parameter with its master, an fp32 state and a bf16 gradient
// move 28 bytes an element, a bf16 parameter with e4m3 states 10.  The moments are
// computed in 64 bits and rounded once to fp32 (the vector ALU takes 64-bit multiply-adds at
// the rate of 32-bit ones), so that a code next to a border does not depend on an order
// of roundings.
//
// The list travels in the kernel arguments (kMaxAdam entries a launch), so nothing is
// copied to the device and a captured graph holds its own list.  A tensor is cut into chunks
// of kChunk elements from its first, eight neighbouring ones a thread, so that sixteen lanes
// hold a run: its largest value is four lane moves away.  Loads take 16 bytes at any
// element's address.  The step's coefficients are computed by every thread for itself: a launch
// to compute them once costs more.
#include <algorithm>
#include <cmath>
#include <new>

#include "moe_args.h"
#include "moe_fp8_codec.h"

namespace moe {
namespace {

constexpr int kMaxAdam = 46;  // entries a launch
constexpr int kAdamThreads = 256;
constexpr int kChunk = 8 * kAdamThreads;
constexpr int kMaxAdamBlocks = 4096;
constexpr uint64_t kStreamBytes = 256ull << 20;  // what the memory-side cache holds

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
  double b1, b2, log_b1, log_b2;
  float eps, max_norm;
};
static_assert(sizeof(AdamList) + sizeof(AdamStep) <= 3584, "kernel arguments hold the list");

// The step's numbers, the same in every thread.
struct Coef {
  double c, b1, b2, a1, a2;  // clipping factor, betas and 1 - betas
  float lr, rate, root, eps;  // lr, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  bool none;                  // nothing to do
};
__device__ __forceinline__ Coef coefficients(const AdamStep& s) {
  Coef k;
  const float lr = *s.lr;
  const int t = *s.step;
  k.c = 1.;
  k.none = t < 1;
  if (s.norm != nullptr) {
    const float nm = *s.norm;
    k.none |= !(fabsf(nm) < INFINITY);
    if (!(nm <= s.max_norm)) k.c = double(s.max_norm) / double(nm);
  }
  k.b1 = s.b1; k.b2 = s.b2;
  k.a1 = 1. - s.b1; k.a2 = 1. - s.b2;
  k.lr = lr;
  k.rate = float(double(lr) / -expm1(double(t) * s.log_b1));
  k.root = float(1. / sqrt(-expm1(double(t) * s.log_b2)));
  k.eps = s.eps;
  return k;
}

template <bool STREAM>
__device__ __forceinline__ uint4 fetch16(const void* p) {
  typedef uint32_t any_u32x4 __attribute__((ext_vector_type(4), aligned(2)));
  if constexpr (STREAM) {
    const any_u32x4 v = __builtin_nontemporal_load(static_cast<const any_u32x4*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
  } else {
    return load16(p);
  }
}
template <bool STREAM>
__device__ __forceinline__ void keep16(void* p, const uint4& a) {
  typedef uint32_t any_u32x4 __attribute__((ext_vector_type(4), aligned(2)));
  if constexpr (STREAM) {
    const any_u32x4 v = {a.x, a.y, a.z, a.w};
    __builtin_nontemporal_store(v, static_cast<any_u32x4*>(p));
  } else {
    store16(p, a);
  }
}

// Eight elements from p, `n` of which are there (zeros behind them), as they are stored.
template <class T> struct Eight;
template <> struct Eight<float> {
  uint4 a, b;
  template <bool STREAM>
  __device__ __forceinline__ void get(const float* p, int n) {
    if (n >= 8) {
      a = fetch16<STREAM>(p);
      b = fetch16<STREAM>(p + 4);
    } else {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = i < n ? __float_as_uint(p[i]) : 0u;
      a = make_uint4(w[0], w[1], w[2], w[3]);
      b = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
  }
  template <bool STREAM>
  static __device__ __forceinline__ void put(float* p, int n, const float (&f)[8]) {
    if (n >= 8) {
      keep16<STREAM>(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
      keep16<STREAM>(p + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = f[i];
    }
  }
};
template <> struct Eight<uint16_t> {
  uint4 a;
  template <bool STREAM>
  __device__ __forceinline__ void get(const uint16_t* p, int n) {
    if (n >= 8) {
      a = fetch16<STREAM>(p);
    } else {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) w[i / 2] |= uint32_t(p[i]) << (16 * (i & 1));
      a = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  template <bool STREAM>
  static __device__ __forceinline__ void put(uint16_t* p, int n, const float (&f)[8]) {
    if (n >= 8) {
      keep16<STREAM>(p, make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                   pack_bf16x2(f[6], f[7])));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = uint16_t(pack_bf16x2(f[i], 0.f));
    }
  }
};
// Eight e4m3 codes.
struct Codes {
  uint2 a;
  __device__ __forceinline__ void get(const uint8_t* p, int n) {
    if (n >= 8) {
      a = *reinterpret_cast<const uint2*>(p);
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
  static __device__ __forceinline__ void put(uint8_t* p, int n, const uint2& c) {
    if (n >= 8) {
      *reinterpret_cast<uint2*>(p) = c;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = uint8_t((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
  }
};

// Codes of a run's eight values in each of its sixteen lanes; LEAST: what is positive has a
// positive code.  Returns the scale.
template <bool LEAST>
__device__ __forceinline__ float code8(const float (&x)[8], uint2& codes) {
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(x[i]));
  am = max16(am);
  const float s = am == 0.f ? 1.f : am / 448.f;
  float y[8];
  if (s >= 0x1p-120f) {
    block_quotients(x, s, 1.f / s, y);
  } else {  // the reciprocal may be infinite
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] / s;
  }
  if constexpr (LEAST) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] > 0.f ? fmaxf(y[i], 0x1p-9f) : y[i];
  }
  codes.x = pack_e4m3x4(y[0], y[1], y[2], y[3]);
  codes.y = pack_e4m3x4(y[4], y[5], y[6], y[7]);
  return s;
}

// This thread's eight elements of chunk c of entry i.
template <bool E4M3, bool STREAM, class P, class G>
__device__ __forceinline__ void step_chunk(const AdamList& L, int i, uint32_t c, const Coef& k) {
  const int64_t e = int64_t(c) * kChunk + threadIdx.x * 8, left = L.n[i] - e;
  const int n = left > 8 ? 8 : int(left);  // may be negative
  P* param = static_cast<P*>(L.param[i]) + e;
  float* master = L.master[i];
  const bool own = master == nullptr;
  Eight<G> g8;
  Eight<P> p8;
  Eight<float> w8, m8, v8;
  Codes mc, vc;
  float ms = 0.f, vs = 0.f;
  g8.template get<STREAM>(static_cast<const G*>(L.grad[i]) + e, n);
  if (own) p8.template get<STREAM>(param, n);
  else w8.template get<STREAM>(master + e, n);
  if constexpr (E4M3) {
    mc.get(static_cast<const uint8_t*>(L.m[i]) + e, n);
    vc.get(static_cast<const uint8_t*>(L.v[i]) + e, n);
    if (n > 0) {
      ms = L.ms[i][e >> 7];
      vs = L.vs[i][e >> 7];
    }
  } else {
    m8.template get<STREAM>(static_cast<const float*>(L.m[i]) + e, n);
    v8.template get<STREAM>(static_cast<const float*>(L.v[i]) + e, n);
  }
  float g[8], p[8], m[8], v[8];
  g8.values(g);
  if (own) p8.values(p);
  else w8.values(p);
  if constexpr (E4M3) {
    mc.values(m);
    vc.values(v);
  } else {
    m8.values(m);
    v8.values(v);
  }
  const float shrink = 1.f - k.lr * L.decay[i];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const double gd = double(g[j]) * k.c;
    double md = double(m[j]), vd = double(v[j]);
    if constexpr (E4M3) {
      md *= double(ms);
      vd *= double(vs);  // exact
      vd *= vd;
    }
    m[j] = float(__builtin_fma(k.a1, gd, k.b1 * md));
    const float v32 = float(__builtin_fma(k.a2 * gd, gd, k.b2 * vd));
    const float sq = sqrtf(v32);
    p[j] = __builtin_fmaf(p[j], shrink, -k.rate * (m[j] / __builtin_fmaf(sq, k.root, k.eps)));
    v[j] = E4M3 ? sq : v32;
  }
  if (own) {
    Eight<P>::template put<STREAM>(param, n, p);
  } else {
    Eight<float>::template put<STREAM>(master + e, n, p);
    Eight<P>::template put<STREAM>(param, n, p);
  }
  if constexpr (E4M3) {
    uint2 codes;
    ms = code8<false>(m, codes);
    Codes::put(static_cast<uint8_t*>(L.m[i]) + e, n, codes);
    vs = code8<true>(v, codes);
    Codes::put(static_cast<uint8_t*>(L.v[i]) + e, n, codes);
    if ((threadIdx.x & 15) == 0 && n > 0) {
      L.ms[i][e >> 7] = ms;
      L.vs[i][e >> 7] = vs;
    }
  } else {
    Eight<float>::template put<STREAM>(static_cast<float*>(L.m[i]) + e, n, m);
    Eight<float>::template put<STREAM>(static_cast<float*>(L.v[i]) + e, n, v);
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
    if (L.kind[i] == 3) step_chunk<E4M3, STREAM, float, float>(L, i, at, k);
    else if (L.kind[i] == 2) step_chunk<E4M3, STREAM, uint16_t, float>(L, i, at, k);
    else if (L.kind[i] == 1) step_chunk<E4M3, STREAM, float, uint16_t>(L, i, at, k);
    else step_chunk<E4M3, STREAM, uint16_t, uint16_t>(L, i, at, k);
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
  st.b1 = d->beta1; st.b2 = d->beta2;
  st.log_b1 = std::log(d->beta1); st.log_b2 = std::log(d->beta2);
  st.eps = float(d->eps); st.max_norm = max_norm;
  hipStream_t s = static_cast<hipStream_t>(stream);
  AdamList L;
  L.count = 0;
  L.first[0] = 0;
  uint64_t bytes = 0;
  auto flush = [&]() {
    if (L.count == 0) return int(MOE_OK);
    const unsigned grid = std::min<uint32_t>(L.first[L.count], kMaxAdamBlocks);
    const bool stream_it = bytes > kStreamBytes;
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
