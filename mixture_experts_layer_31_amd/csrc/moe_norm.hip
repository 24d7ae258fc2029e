// The residual sum between two blocks with the norms on both of its sides, and its backward
// (moe_norm_fwd, moe_norm_bwd in moe.h).
//
// Both are bound by memory: four arrays of rows forward (b, r in, h, y out), six
// backward (b, h, dy, dh in, db, dr out).  A row stays in the registers of its WAVES waves, eight
// neighbouring values a lane and piece: it is read once, its sums are joined over the
// lanes and, past one wave, through LDS, and what depends on them is computed from the
// registers.  The weights of a lane's columns stay in registers over the rows that a workgroup takes,
// and so do its parts of dw and dw_post, which go to the scratch as one row a workgroup; a second launch
// adds those rows in their order.
//
// Sums.  With e = w dy, q = 1 / rms(h): dh' = q (e - h q^2 mean(e h)), so sum h^2, sum e h and sum b^2 are
// joined together; only sum g w_post b, of the finished gradient g, needs a second join.
// h with a gate or w_post is computed in 64 bits: kept in bf16, a value next to a border
// goes one way or the other, and an fp32 sum of squares decides that for one value in 2^15.
#include <cmath>
#include <type_traits>

#include "moe_args.h"
#include "moe_fp8_codec.h"

namespace moe {
namespace {

constexpr int kNormMaxD = 16384;
constexpr int kNormPartials = 1024;  // workgroups, so rows of the scratch, of a backward

struct NormArgs {
  const void *b, *r, *w_post, *w;
  const float* gate;
  void *h, *y;
  const void *dy, *dh;
  void *db, *dr;
  float *dgate, *part, *part_post;  // part: [workgroups][D]
  int64_t ld_b, ld_r, ld_h, ld_y;
  int T, D;
  float eps, scale;
  bool w_f32;
};

__device__ __forceinline__ float one(const float* p) { return *p; }
__device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ void put_one(float* p, float f) { *p = f; }
__device__ __forceinline__ void put_one(uint16_t* p, float f) { *p = uint16_t(pack_bf16x2(f, 0.f)); }
// A value as its type keeps it.
__device__ __forceinline__ float kept(const float*, float f) { return f; }
__device__ __forceinline__ float kept(const uint16_t*, float f) {
  return __uint_as_float(pack_bf16x2(f, 0.f) << 16);
}

__device__ __forceinline__ void whole8(const float* p, float (&f)[8]) {
  const uint4 a = load16(p), b = load16(p + 4);
  f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
  f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
}
__device__ __forceinline__ void whole8(const uint16_t* p, float (&f)[8]) {
  const uint4 v = load16(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ void put8(float* p, const float (&f)[8]) {
  store16(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
  store16(p + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
}
__device__ __forceinline__ void put8(uint16_t* p, const float (&f)[8]) {
  store16(p, make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                        pack_bf16x2(f[6], f[7])));
}

// Values c .. c + 7 of a row of D (zeros behind its end), and their store.
template <class T>
__device__ __forceinline__ void get(const T* row, int c, int D, float (&f)[8]) {
  if (c + 8 <= D) {
    whole8(row + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < D ? one(row + c + i) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void put(T* row, int c, int D, const float (&f)[8]) {
  if (c + 8 <= D) {
    put8(row + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < D) put_one(row + c + i, f[i]);
  }
}
__device__ __forceinline__ void get_weight(const void* w, bool f32, int c, int D, float (&f)[8]) {
  if (f32) get(static_cast<const float*>(w), c, D, f);
  else get(static_cast<const uint16_t*>(w), c, D, f);
}

template <class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sums over a row's waves.  `red` is used by one join at a time: a join writes one half and
// reads it behind one barrier, the next join of the workgroup uses the other half.
template <int WAVES, int N, class V>
__device__ __forceinline__ void row_sums(V (&v)[N], double (*red)[WAVES][3], int& half) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (WAVES > 1) {
    const int wv = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[half][wv][i] = double(v[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      double s = 0.;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) s += red[half][w][i];
      v[i] = V(s);
    }
    half ^= 1;
  }
}

// What enters the residual: nothing (h = r), scale b, or b with its norm or gate.
enum { BLOCK_NONE = 0, BLOCK_SUM = 1, BLOCK_NORM = 2 };

// Threads of a workgroup whose rows take WAVES waves: one row a workgroup, or four of one wave each.
constexpr int norm_threads(int waves) { return waves == 1 ? 256 : 64 * waves; }

template <class IO, class R, int BLOCK, int WAVES, int NV>
__global__ void __launch_bounds__(norm_threads(WAVES)) norm_fwd_kernel(NormArgs a) {
  constexpr int ROWS = WAVES == 1 ? 4 : 1;
  __shared__ double red[2][WAVES][3];
  int half = 0;
  const int tid = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int D = a.D;
  float w[NV][8], wp[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = 8 * (tid + 64 * WAVES * k);
    if (a.w != nullptr) get_weight(a.w, a.w_f32, c, D, w[k]);
    if (BLOCK == BLOCK_NORM && a.w_post != nullptr) get_weight(a.w_post, a.w_f32, c, D, wp[k]);
  }
  for (int64_t t = int64_t(blockIdx.x) * ROWS + (WAVES == 1 ? threadIdx.x >> 6 : 0); t < a.T;
       t += int64_t(gridDim.x) * ROWS) {
    const IO* b = static_cast<const IO*>(a.b) + t * a.ld_b;
    const R* r = static_cast<const R*>(a.r) + t * a.ld_r;
    float x[NV][8], bv[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (tid + 64 * WAVES * k);
      get(r, c, D, x[k]);
      if (BLOCK != BLOCK_NONE) get(b, c, D, bv[k]);
    }
    if constexpr (BLOCK == BLOCK_SUM) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = __builtin_fmaf(a.scale, bv[k][i], x[k][i]);
    } else if constexpr (BLOCK == BLOCK_NORM) {
      double by = double(a.scale);
      if (a.gate != nullptr) by /= 1. + exp(-double(a.gate[t]));
      if (a.w_post != nullptr) {
        double sum[1] = {0.};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[0] = __builtin_fma(double(bv[k][i]), double(bv[k][i]), sum[0]);
        row_sums<WAVES>(sum, red, half);
        by /= sqrt(sum[0] / D + double(a.eps));
      }
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          double u = double(bv[k][i]);
          if (a.w_post != nullptr) u *= double(wp[k][i]);  // exact
          x[k][i] = float(__builtin_fma(by, u, double(x[k][i])));
        }
    }
    float sum[1] = {0.f};
    R* h = static_cast<R*>(a.h) + t * a.ld_h;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (tid + 64 * WAVES * k);
      if (a.h != nullptr) put(h, c, D, x[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[k][i] = kept(h, x[k][i]);
        sum[0] = __builtin_fmaf(x[k][i], x[k][i], sum[0]);
      }
    }
    if (a.w == nullptr) continue;
    row_sums<WAVES>(sum, red, half);
    const float q = 1.f / sqrtf(sum[0] / float(D) + a.eps);
    IO* y = static_cast<IO*>(a.y) + t * a.ld_y;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = x[k][i] * q * w[k][i];
      put(y, 8 * (tid + 64 * WAVES * k), D, o);
    }
  }
}

// One row a workgroup at a time.
template <class IO, class R, int BLOCK, int WAVES, int NV>
__global__ void __launch_bounds__(64 * WAVES) norm_bwd_kernel(NormArgs a) {
  __shared__ double red[2][WAVES][3];
  int half = 0;
  const int tid = threadIdx.x, D = a.D;
  const bool pre = a.w != nullptr, post = BLOCK == BLOCK_NORM && a.w_post != nullptr;
  float w[NV][8], wp[NV][8];
  double acc[NV][8], acc_post[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = 8 * (tid + 64 * WAVES * k);
    if (pre) get_weight(a.w, a.w_f32, c, D, w[k]);
    if (post) get_weight(a.w_post, a.w_f32, c, D, wp[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      acc[k][i] = acc_post[k][i] = 0.;
      if (!post) wp[k][i] = 1.f;
    }
  }
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const IO* b = static_cast<const IO*>(a.b) + t * a.ld_b;
    const IO* dy = static_cast<const IO*>(a.dy) + t * a.ld_y;
    const R* h = static_cast<const R*>(a.h) + t * a.ld_h;
    const R* dh = static_cast<const R*>(a.dh) + t * a.ld_h;
    float g[NV][8], x[NV][8], e[NV][8], bv[NV][8];
    float sum[3] = {0.f, 0.f, 0.f};  // h^2, e h, b^2
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (tid + 64 * WAVES * k);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[k][i] = x[k][i] = e[k][i] = 0.f;
      if (a.dh != nullptr) get(dh, c, D, g[k]);
      if (pre && a.dy != nullptr) {
        get(h, c, D, x[k]);
        get(dy, c, D, e[k]);
      }
      if (BLOCK == BLOCK_NORM) get(b, c, D, bv[k]);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (pre) {
          sum[0] = __builtin_fmaf(x[k][i], x[k][i], sum[0]);
          sum[1] = __builtin_fmaf(e[k][i] * w[k][i], x[k][i], sum[1]);
        }
        if (post) sum[2] = __builtin_fmaf(bv[k][i], bv[k][i], sum[2]);
      }
    row_sums<WAVES>(sum, red, half);
    if (pre && a.dy != nullptr) {
      const float q = 1.f / sqrtf(sum[0] / float(D) + a.eps);
      const float m = sum[1] / float(D) * q * q;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[k][i] += double(e[k][i] * (x[k][i] * q));
          g[k][i] = __builtin_fmaf(q, __builtin_fmaf(-x[k][i], m, e[k][i] * w[k][i]), g[k][i]);
        }
    }
    R* dr = static_cast<R*>(a.dr) + t * a.ld_r;
    IO* db = static_cast<IO*>(a.db) + t * a.ld_b;
#pragma unroll
    for (int k = 0; k < NV; ++k) put(dr, 8 * (tid + 64 * WAVES * k), D, g[k]);
    if constexpr (BLOCK == BLOCK_SUM) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[k][i] *= a.scale;
        put(db, 8 * (tid + 64 * WAVES * k), D, g[k]);
      }
    } else if constexpr (BLOCK == BLOCK_NORM) {
      float by = a.scale, rest = 0.f;
      if (a.gate != nullptr) {
        const float z = a.gate[t];
        by = a.scale / (1.f + expf(-z));
        rest = 1.f / (1.f + expf(z));
      }
      float dot[1] = {0.f};
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[0] = __builtin_fmaf(g[k][i] * wp[k][i], bv[k][i], dot[0]);
      row_sums<WAVES>(dot, red, half);
      const float p = post ? 1.f / sqrtf(sum[2] / float(D) + a.eps) : 1.f;
      if (a.gate != nullptr && tid == 0) a.dgate[t] = by * rest * (dot[0] * p);
      const float m = post ? dot[0] / float(D) * p * p : 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (post) acc_post[k][i] += double(by * g[k][i] * (bv[k][i] * p));
          o[i] = by * p * __builtin_fmaf(-bv[k][i], m, g[k][i] * wp[k][i]);
        }
        put(db, 8 * (tid + 64 * WAVES * k), D, o);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = 8 * (tid + 64 * WAVES * k);
    float f[8];
    if (pre) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = float(acc[k][i]);
      put(a.part + size_t(blockIdx.x) * D, c, D, f);
    }
    if (post) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = float(acc_post[k][i]);
      put(a.part_post + size_t(blockIdx.x) * D, c, D, f);
    }
  }
}

// The rows of the scratch, 64 columns a workgroup and 16 rows side by side.
__global__ void __launch_bounds__(1024) norm_finish_kernel(const float* __restrict__ part, const float* __restrict__ part_post,
                                                           int rows, int D, float* __restrict__ dw,
                                                           float* __restrict__ dw_post) {
  __shared__ double s[16][64];
  const int l = threadIdx.x & 63, r = threadIdx.x >> 6, c = blockIdx.x * 64 + l;
  const bool second = blockIdx.y == 1 || dw == nullptr;
  const float* in = second ? part_post : part;
  double v = 0.;
  if (c < D) {
#pragma unroll 8
    for (int k = r; k < rows; k += 16) v += double(in[size_t(k) * D + c]);
  }
  s[r][l] = v;
  __syncthreads();
  if (r != 0 || c >= D) return;
#pragma unroll
  for (int k = 1; k < 16; ++k) v += s[k][l];
  (second ? dw_post : dw)[c] = float(v);
}

// f(waves a row, pieces a lane) for a forward and for a backward row.
template <class F>
int with_row_fwd(int D, F&& f) {
  using std::integral_constant;
  if (D <= 512) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (D <= 1024) return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (D <= 2048) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (D <= 4096) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  if (D <= 8192) return f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
}
template <class F>
int with_row_bwd(int D, F&& f) {
  using std::integral_constant;
  if (D <= 512) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (D <= 1024) return f(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  if (D <= 2048) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (D <= 4096) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (D <= 8192) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
}
// f(IO, R) by example.
template <class F>
int with_types(const moe_norm_desc& d, F&& f) {
  const bool io = d.io_type == MOE_TYPE_F32, res = d.res_type == MOE_TYPE_F32;
  if (io) return res ? f(float(), float()) : f(float(), uint16_t());
  return res ? f(uint16_t(), float()) : f(uint16_t(), uint16_t());
}

bool float_type(int32_t t) { return t == MOE_TYPE_F32 || t == MOE_TYPE_BF16; }

int check_norm(const moe_norm_desc* d) {
  if (d == nullptr) return MOE_EINVAL;
  if (d->T < 0 || d->D < 1 || !float_type(d->io_type) || !float_type(d->res_type) || !float_type(d->w_type) ||
      !std::isfinite(d->scale) || !std::isfinite(d->eps) || !(d->eps >= 0.f))
    return MOE_EINVAL;
  if (d->ld_b < d->D || d->ld_r < d->D || d->ld_h < d->D || d->ld_y < d->D) return MOE_EINVAL;
  constexpr int64_t most = int64_t(1) << 40;
  if (d->D > kNormMaxD || d->ld_b >= most || d->ld_r >= most || d->ld_h >= most || d->ld_y >= most)
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

struct Buffer {
  const void* p;
  size_t n, align;
};
Buffer rows_of(const moe_norm_desc& d, const void* p, int64_t ld, int32_t type) {
  const size_t es = type_bytes(type);
  return {p, d.T > 0 ? (size_t(d.T - 1) * size_t(ld) + size_t(d.D)) * es : 0, es};
}
Buffer weight_of(const moe_norm_desc& d, const void* p) {
  const size_t es = type_bytes(d.w_type);
  return {p, size_t(d.D) * es, es};
}

// Alignment of all, and written ones apart from all others but for the pair (same, as).
int check_buffers(const Buffer* in, int n_in, const Buffer* out, int n_out, const void* same, const void* as) {
  for (int i = 0; i < n_in; ++i)
    if (!aligned_to(in[i].p, in[i].align)) return MOE_EALIGN;
  for (int i = 0; i < n_out; ++i)
    if (!aligned_to(out[i].p, out[i].align)) return MOE_EALIGN;
  for (int i = 0; i < n_out; ++i) {
    for (int k = 0; k < n_in; ++k)
      if (overlap(out[i].p, out[i].n, in[k].p, in[k].n) && !(out[i].p == same && in[k].p == as && same == as))
        return MOE_EINVAL;
    for (int k = 0; k < i; ++k)
      if (overlap(out[i].p, out[i].n, out[k].p, out[k].n)) return MOE_EINVAL;
  }
  return MOE_OK;
}

int norm_partials(const moe_norm_desc& d) { return d.T < kNormPartials ? (d.T > 0 ? d.T : 1) : kNormPartials; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_norm_fwd(const moe_norm_desc* d, const void* b, const void* r, const float* gate, const void* w_post,
                 const void* w, void* h, void* y, void* stream) {
  if (const int rc = check_norm(d)) return rc;
  if (d->T == 0) return MOE_OK;
  if (b == nullptr ? gate != nullptr || w_post != nullptr || w == nullptr : h == nullptr) return MOE_EINVAL;
  if ((w == nullptr) != (y == nullptr) || r == nullptr) return MOE_EINVAL;
  const Buffer in[] = {rows_of(*d, b, d->ld_b, d->io_type), rows_of(*d, r, d->ld_r, d->res_type),
                       {gate, size_t(d->T) * 4, 4}, weight_of(*d, w_post), weight_of(*d, w)};
  const Buffer out[] = {rows_of(*d, h, d->ld_h, d->res_type), rows_of(*d, y, d->ld_y, d->io_type)};
  const bool in_place = h == r && d->ld_h == d->ld_r;
  if (const int rc = check_buffers(in, 5, out, 2, in_place ? h : nullptr, in_place ? r : nullptr)) return rc;
  NormArgs a{};
  a.b = b; a.r = r; a.w_post = w_post; a.w = w; a.gate = gate; a.h = h; a.y = y;
  a.ld_b = d->ld_b; a.ld_r = d->ld_r; a.ld_h = d->ld_h; a.ld_y = d->ld_y;
  a.T = d->T; a.D = d->D; a.eps = d->eps; a.scale = d->scale;
  a.w_f32 = d->w_type == MOE_TYPE_F32;
  hipStream_t s = static_cast<hipStream_t>(stream);
  prof_begin("norm_fwd", s);
  with_types(*d, [&](auto io, auto res) {
    return with_row_fwd(d->D, [&](auto waves, auto nv) {
      constexpr int W = decltype(waves)::value, NV = decltype(nv)::value;
      using IO = decltype(io);
      using R = decltype(res);
      const long long want = ceil_div(d->T, W == 1 ? 4 : 1);
      const unsigned grid = unsigned(want < 4096 ? want : 4096);
      if (b == nullptr) norm_fwd_kernel<IO, R, BLOCK_NONE, W, NV><<<grid, norm_threads(W), 0, s>>>(a);
      else if (gate != nullptr || w_post != nullptr) norm_fwd_kernel<IO, R, BLOCK_NORM, W, NV><<<grid, norm_threads(W), 0, s>>>(a);
      else norm_fwd_kernel<IO, R, BLOCK_SUM, W, NV><<<grid, norm_threads(W), 0, s>>>(a);
      return 0;
    });
  });
  prof_end(s);
  return launched();
}

// A row of dw's parts and one of dw_post's for each workgroup.
size_t moe_norm_scratch_bytes(const moe_norm_desc* d) {
  if (check_norm(d) != MOE_OK) return 0;
  return 2 * align256(size_t(norm_partials(*d)) * d->D * 4);
}

int moe_norm_bwd(const moe_norm_desc* d, const void* b, const void* h, const float* gate, const void* w_post,
                 const void* w, const void* dy, const void* dh, void* db, void* dr, float* dgate,
                 float* dw_post, float* dw, void* scratch, size_t scratch_bytes, void* stream) {
  if (const int rc = check_norm(d)) return rc;
  if ((w == nullptr) != (dw == nullptr) || (w_post == nullptr) != (dw_post == nullptr) ||
      (w == nullptr && dy != nullptr) || scratch == nullptr)
    return MOE_EINVAL;
  const bool block = gate != nullptr || w_post != nullptr;
  if (d->T > 0) {
    if (dr == nullptr || (w != nullptr && h == nullptr) || (gate == nullptr) != (dgate == nullptr) ||
        (block && (b == nullptr || db == nullptr)) || (b != nullptr && db == nullptr))
      return MOE_EINVAL;
  }
  const Buffer in[] = {rows_of(*d, b, d->ld_b, d->io_type), rows_of(*d, h, d->ld_h, d->res_type),
                       {gate, size_t(d->T) * 4, 4}, weight_of(*d, w_post), weight_of(*d, w),
                       rows_of(*d, dy, d->ld_y, d->io_type), rows_of(*d, dh, d->ld_h, d->res_type)};
  const size_t need = moe_norm_scratch_bytes(d);
  const Buffer out[] = {rows_of(*d, db, d->ld_b, d->io_type), rows_of(*d, dr, d->ld_r, d->res_type),
                        {dgate, size_t(d->T) * 4, 4}, {dw_post, size_t(d->D) * 4, 4}, {dw, size_t(d->D) * 4, 4},
                        {scratch, need, 16}};
  const bool in_place = dr == dh && d->ld_r == d->ld_h;
  if (const int rc = check_buffers(in, 7, out, 6, in_place ? dr : nullptr, in_place ? dh : nullptr)) return rc;
  if (scratch_bytes < need) return MOE_ESCRATCH;
  NormArgs a{};
  a.b = b; a.w_post = w_post; a.w = w; a.gate = gate; a.h = const_cast<void*>(h);
  a.dy = dy; a.dh = dh; a.db = db; a.dr = dr; a.dgate = dgate;
  a.part = static_cast<float*>(scratch);
  a.part_post = reinterpret_cast<float*>(static_cast<char*>(scratch) + need / 2);
  a.ld_b = d->ld_b; a.ld_r = d->ld_r; a.ld_h = d->ld_h; a.ld_y = d->ld_y;
  a.T = d->T; a.D = d->D; a.eps = d->eps; a.scale = d->scale;
  a.w_f32 = d->w_type == MOE_TYPE_F32;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const unsigned grid = unsigned(norm_partials(*d));
  if (d->T > 0) {
    prof_begin("norm_bwd", s);
    with_types(*d, [&](auto io, auto res) {
      return with_row_bwd(d->D, [&](auto waves, auto nv) {
        constexpr int W = decltype(waves)::value, NV = decltype(nv)::value;
        using IO = decltype(io);
        using R = decltype(res);
        if (db == nullptr) norm_bwd_kernel<IO, R, BLOCK_NONE, W, NV><<<grid, 64 * W, 0, s>>>(a);
        else if (block) norm_bwd_kernel<IO, R, BLOCK_NORM, W, NV><<<grid, 64 * W, 0, s>>>(a);
        else norm_bwd_kernel<IO, R, BLOCK_SUM, W, NV><<<grid, 64 * W, 0, s>>>(a);
        return 0;
      });
    });
    prof_end(s);
    if (const int rc = launched()) return rc;
  }
  if (dw == nullptr && dw_post == nullptr) return MOE_OK;
  prof_begin("norm_finish", s);
  const dim3 blocks(unsigned(ceil_div(d->D, 64)), dw != nullptr && dw_post != nullptr ? 2 : 1);
  norm_finish_kernel<<<blocks, 1024, 0, s>>>(a.part, a.part_post, d->T > 0 ? int(grid) : 0, d->D, dw, dw_post);
  prof_end(s);
  return launched();
}

}  // extern "C"
