// The residual sum between two blocks with the norms on both of its sides, and its backward
// (moe_norm_fwd, moe_norm_bwd in moe.h).
//
// Both are bound by memory: four arrays of rows forward (b, r in, h, y out), six
// backward (b, h, dy, dh in, db, dr out; without gate and w_post no b).  16384 x 2048 bf16: 48 us forward (5.6 TB/s),
// 56 backward (6.0) and 5 for the second launch; 16384 x 4096 with an fp32 residual, gate and both norms 140 (5.8) and
// 218 (5.5); a row by itself 2.3.  A row stays in the registers of its TPR threads (16 of them for up to 128
// values, 512 for 4096), eight or four neighbouring values a thread and piece: it is read once, its sums are joined over
// the lanes and, past one wave, through LDS, and what depends on them is computed from the
// registers.  The weights of a lane's columns stay in registers over the rows that a workgroup takes,
// and so do its parts of dw and dw_post, which go to the scratch as one row a workgroup; a second launch
// adds those rows in their order.  Rows past 8192 columns take 1024 threads, of 128 registers each, and spill with
// w_post (4096 x 16384: 235 us forward and backward, with w_post 733); there no row is loaded ahead (with one 326 and 1153).
//
// Sums.  With e = w dy, q = 1 / rms(h): dh' = q (e - h q^2 mean(e h)), so sum h^2, sum e h and sum b^2 are
// joined together; only sum g w_post b, of the finished gradient g, needs a second join.
// h with a gate or w_post is computed in 64 bits where it is kept in bf16: there a value next to a border goes one
// way or the other, and an fp32 sum of squares would decide that for one value in 2^15.  An fp32 residual is computed in
// fp32: its own rounding is of the size of the sum's, and 64-bit values of a row need twice the registers.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "moe_args.h"
#include "moe_fp8_codec.h"

namespace moe {
namespace {

constexpr int kNormMaxD = 16384;
constexpr int kFold = 16;  // rows

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
  double inv_d;  // 1 / D
  bool w_f32;
};

__device__ __forceinline__ void put_one(float* p, float f) { *p = f; }
__device__ __forceinline__ void put_one(uint16_t* p, float f) { *p = uint16_t(pack_bf16x2(f, 0.f)); }
// A value as its type keeps it.
__device__ __forceinline__ float kept(const float*, float f) { return f; }
__device__ __forceinline__ float kept(const uint16_t*, float f) {
  return __uint_as_float(pack_bf16x2(f, 0.f) << 16);
}

// P values c .. c + P - 1 of a row of D (zeros behind its end) as they are stored, and their store.  Of fp32 rows P is
// 4: pieces of 8 are two loads of 16 bytes that each touch half of every line (1363 x 1001 forward and backward 23.5 us,
// so 22.7); beside bf16 rows, whose loads would have 8 bytes, it is 8 (16384 x 4096: 364 us, with 4 386).
//
// MOVED, for rows of bf16 alone that do not fill their threads: a load that would pass the row's end starts where it ends
// there, with no branch, and `mend` shifts what it got.  With a branch a row's last piece, loaded element by element, waits
// for each of them (16784 x 1999 forward and backward: 233 us, so 146; 13421 x 2500 315, so 181; 524288 x 64, whose lanes
// behind the end only skip their loads, 208, so 149).  Where all pieces are whole the shifts cost registers (16384 x 4096
// with both norms 262 us, with them 276), and fp32 rows, whose elements need not be put together, lose more than
// they gain (1363 x 1001 with both norms: 22 us, so 24).
template <class T, int P, bool MOVED>
struct Piece {
  static constexpr int W = P * int(sizeof(T)) / 4;
  static constexpr int N = 16 / int(sizeof(T));  // elements a load, with MOVED
  uint32_t w[W];
  __device__ __forceinline__ void get(const T* row, int c, int D) {
    if (MOVED && D >= N) {
#pragma unroll
      for (int u = 0; u < P / N; ++u) {
        const uint4 v = load16(row + min(c + u * N, D - N));
        w[4 * u] = v.x; w[4 * u + 1] = v.y; w[4 * u + 2] = v.z; w[4 * u + 3] = v.w;
      }
    } else if (c + P <= D) {
      if constexpr (W == 2) {
        const uint2 v = fetch8<false>(row + c);
        w[0] = v.x; w[1] = v.y;
      } else {
#pragma unroll
        for (int k = 0; k < W / 4; ++k) {
          const uint4 v = load16(row + c + k * 16 / sizeof(T));
          w[4 * k] = v.x; w[4 * k + 1] = v.y; w[4 * k + 2] = v.z; w[4 * k + 3] = v.w;
        }
      }
    } else {
      clear();
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (c + i < D) {
          if constexpr (sizeof(T) == 2) w[i / 2] |= uint32_t(row[c + i]) << (16 * (i & 1));
          else w[i] = __float_as_uint(row[c + i]);
        }
    }
  }
  __device__ __forceinline__ void mend(int c, int D) {
    if constexpr (MOVED) {
      if (D < N || __ballot(c + P > D) == 0) return;
#pragma unroll
      for (int u = 0; u < P / N; ++u) {
        const int past = min(max(c + u * N - (D - N), 0), N), words = past * int(sizeof(T)) / 4;
        uint32_t v[5] = {w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3], 0};
#pragma unroll
        for (int by = 4; by >= 1; by /= 2) {
          const bool go = (words & by) != 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = go ? (k + by < 4 ? v[k + by] : 0u) : v[k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[4 * u + k] = sizeof(T) == 2 ? __builtin_amdgcn_alignbit(v[k + 1], v[k], (past & 1) * 16) : v[k];
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = 0;
  }
  __device__ __forceinline__ void values(float (&f)[P]) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < W; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k) f[k] = __uint_as_float(w[k]);
    }
  }
};
template <bool MOVED, class T, int P>
__device__ __forceinline__ void get(const T* row, int c, int D, float (&f)[P]) {
  Piece<T, P, MOVED> e;
  e.get(row, c, D);
  e.mend(c, D);
  e.values(f);
}
template <class T, int P>
__device__ __forceinline__ void put(T* row, int c, int D, const float (&f)[P]) {
  constexpr int W = P * int(sizeof(T)) / 4;
  if (c + P <= D) {
    uint32_t w[W];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      if constexpr (sizeof(T) == 2) w[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
      else w[k] = __float_as_uint(f[k]);
    }
    if constexpr (W == 2) {
      keep8<false>(row + c, make_uint2(w[0], w[1]));
    } else {
#pragma unroll
      for (int k = 0; k < W / 4; ++k)
        store16(row + c + k * 16 / sizeof(T), make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (c + i < D) put_one(row + c + i, f[i]);
  }
}
template <bool MOVED, int P>
__device__ __forceinline__ void get_weight(const void* w, bool f32, int c, int D, float (&f)[P]) {
  if (f32) get<MOVED>(static_cast<const float*>(w), c, D, f);
  else get<MOVED>(static_cast<const uint16_t*>(w), c, D, f);
}

// Sum over the wave by lane moves of the vector ALU (a shuffle through the LDS crossbar costs ten times as long, and
// a row has two to six of them on its way): within sixteen lanes, then row by row into the last lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v) {
  const long long b = __double_as_longlong(v);
  const uint32_t lo = uint32_t(__builtin_amdgcn_update_dpp(0, int(b), CTRL, ROWS, 0xF, false));
  const uint32_t hi = uint32_t(__builtin_amdgcn_update_dpp(0, int(b >> 32), CTRL, ROWS, 0xF, false));
  return __longlong_as_double((long long)((uint64_t(hi) << 32) | lo));
}
__device__ __forceinline__ float last_lane(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ double last_lane(double v) {
  const long long b = __double_as_longlong(v);
  const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(int(b), 63)), hi = uint32_t(__builtin_amdgcn_readlane(int(b >> 32), 63));
  return __longlong_as_double((long long)((uint64_t(hi) << 32) | lo));
}
template <class V>
__device__ __forceinline__ V wave_sum(V v) {
  v += moved<0xB1, 0xF>(v);   // quad_perm [1,0,3,2]
  v += moved<0x4E, 0xF>(v);   // quad_perm [2,3,0,1]
  v += moved<0x141, 0xF>(v);  // row_half_mirror
  v += moved<0x140, 0xF>(v);  // row_mirror
  v += moved<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  v += moved<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
  return last_lane(v);
}

// Sum over an aligned group of 16 or 32 lanes, in each of them.
template <int LANES, class V>
__device__ __forceinline__ V group_sum(V v) {
  v += moved<0xB1, 0xF>(v);
  v += moved<0x4E, 0xF>(v);
  v += moved<0x141, 0xF>(v);
  v += moved<0x140, 0xF>(v);
  if constexpr (LANES == 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// Rows of a workgroup whose rows take TPR threads: 256 threads at least.
constexpr int norm_rows(int tpr) { return tpr < 256 ? 256 / tpr : 1; }
constexpr int norm_threads(int tpr) { return tpr * norm_rows(tpr); }
constexpr int norm_waves(int tpr) { return tpr > 64 ? tpr / 64 : 1; }

// Sums over a row's threads; `row` is the workgroup's row that this thread belongs to.  A join of several waves writes one
// half of `red` and reads it behind one barrier, the next join of the workgroup uses the other half.
template <int TPR>
using Joins = double[2][norm_rows(TPR)][norm_waves(TPR)][3];
template <int TPR, int N, class V>
__device__ __forceinline__ void row_sums(V (&v)[N], Joins<TPR>& red, int row, int& half) {
  if constexpr (TPR < 64) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = group_sum<TPR>(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  }
  if constexpr (TPR > 64) {
    constexpr int WAVES = TPR / 64;
    const int wv = (threadIdx.x >> 6) % WAVES;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[half][row][wv][i] = double(v[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      double s = 0.;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) s += red[half][row][w][i];
      v[i] = V(s);
    }
    half ^= 1;
  }
}

__device__ __forceinline__ float fma_of(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ __forceinline__ double fma_of(double a, double b, double c) { return __builtin_fma(a, b, c); }
__device__ __forceinline__ float sigmoid_times(float s, float z) { return s * __builtin_amdgcn_rcpf(1.f + expf(-z)); }
__device__ __forceinline__ double sigmoid_times(double s, float z) { return s * sigmoid64(z); }
// The hardware's, within an ulp (a correctly rounded root and quotient take 25 instructions a row, of some 200); it takes
// numbers below the normal ones for 0.
__device__ __forceinline__ float inverse_root(float x) {
  const bool tiny = x < 0x1p-100f;
  const float r = __builtin_amdgcn_rsqf(tiny ? x * 0x1p100f : x);
  return tiny ? r * 0x1p50f : r;
}
// The hardware's 2^-24 and two steps of Newton's: 2^-50.  Of an infinity it is 0, which the steps would make NaN of (0 inf).
__device__ __forceinline__ double inverse_root(double x) {
  const double r0 = __builtin_amdgcn_rsq(x);
  double r = r0 * __builtin_fma(-0.5 * x * r0, r0, 1.5);
  r = r * __builtin_fma(-0.5 * x * r, r, 1.5);
  return x < INFINITY ? r : r0;
}

// What enters the residual: nothing (h = r), scale b, or b with its norm or gate.
enum { BLOCK_NONE = 0, BLOCK_SUM = 1, BLOCK_NORM = 2 };

template <class IO, class R>
constexpr int piece_of() { return sizeof(IO) + sizeof(R) == 8 ? 4 : 8; }

template <class IO, class R, int BLOCK, int TPR, int EIGHTS, bool MOVED>
__global__ void __launch_bounds__(norm_threads(TPR)) norm_fwd_kernel(NormArgs a) {
  constexpr int P = piece_of<IO, R>(), NV = EIGHTS * 8 / P, ROWS = norm_rows(TPR);
  __shared__ Joins<TPR> red;
  int half = 0;
  const int tid = threadIdx.x % TPR, row = threadIdx.x / TPR, D = a.D;
  const float inv_d = float(a.inv_d);
  float w[NV][P], wp[NV][P];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = P * (tid + TPR * k);
    if (a.w != nullptr) get_weight<MOVED>(a.w, a.w_f32, c, D, w[k]);
    if (BLOCK == BLOCK_NORM && a.w_post != nullptr) get_weight<MOVED>(a.w_post, a.w_f32, c, D, wp[k]);
  }
  for (int64_t first = int64_t(blockIdx.x) * ROWS; first < a.T; first += int64_t(gridDim.x) * ROWS) {
    const int64_t t = first + row;
    const bool there = t < a.T;  // a row behind the last one goes along with it
    const R* r = static_cast<const R*>(a.r) + (there ? t : first) * a.ld_r;
    const IO* b = static_cast<const IO*>(a.b) + (there ? t : first) * a.ld_b;
    float x[NV][P], bv[NV][P];
    Piece<R, P, MOVED> rp[NV];
    Piece<IO, P, MOVED> bp[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = P * (tid + TPR * k);
      rp[k].get(r, c, D);
      if (BLOCK != BLOCK_NONE) bp[k].get(b, c, D);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = P * (tid + TPR * k);
      rp[k].mend(c, D);
      rp[k].values(x[k]);
      if (BLOCK != BLOCK_NONE) {
        bp[k].mend(c, D);
        bp[k].values(bv[k]);
      }
    }
    if constexpr (BLOCK == BLOCK_SUM) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) x[k][i] = __builtin_fmaf(a.scale, bv[k][i], x[k][i]);
    } else if constexpr (BLOCK == BLOCK_NORM) {
      using V = std::conditional_t<sizeof(R) == 2, double, float>;  // see above
      V by = V(a.scale);
      if (a.gate != nullptr) by = sigmoid_times(by, a.gate[there ? t : 0]);
      if (a.w_post != nullptr) {
        V sum[1] = {V(0)};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < P; ++i) sum[0] = fma_of(V(bv[k][i]), V(bv[k][i]), sum[0]);
        row_sums<TPR>(sum, red, row, half);
        by *= inverse_root(fma_of(sum[0], V(a.inv_d), V(a.eps)));
      }
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) {
          // converted here again: 64-bit copies of b and w_post kept over the join cost a third of the waves
          asm("" : "+v"(bv[k][i]));
          V u = V(bv[k][i]);
          if (a.w_post != nullptr) {
            asm("" : "+v"(wp[k][i]));
            u *= V(wp[k][i]);  // exact in 64 bits
          }
          x[k][i] = float(fma_of(by, u, V(x[k][i])));
        }
    }
    float sum[1] = {0.f};
    R* h = static_cast<R*>(a.h) + t * a.ld_h;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = P * (tid + TPR * k);
      if (a.h != nullptr && there) put(h, c, D, x[k]);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        x[k][i] = kept(h, x[k][i]);
        sum[0] = __builtin_fmaf(x[k][i], x[k][i], sum[0]);
      }
    }
    if (a.w == nullptr) continue;
    row_sums<TPR>(sum, red, row, half);
    const float q = inverse_root(__builtin_fmaf(sum[0], inv_d, a.eps));
    IO* y = static_cast<IO*>(a.y) + t * a.ld_y;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float o[P];
#pragma unroll
      for (int i = 0; i < P; ++i) o[i] = x[k][i] * q * w[k][i];
      if (there) put(y, P * (tid + TPR * k), D, o);
    }
  }
}

template <class IO, class R, int BLOCK, int TPR, int EIGHTS, bool MOVED>
__global__ void __launch_bounds__(norm_threads(TPR)) norm_bwd_kernel(NormArgs a) {
  constexpr int P = piece_of<IO, R>(), NV = EIGHTS * 8 / P, ROWS = norm_rows(TPR);
  __shared__ Joins<TPR> red;
  int half = 0;
  const int tid = threadIdx.x % TPR, row = threadIdx.x / TPR, D = a.D;
  const float inv_d = float(a.inv_d);
  const bool pre = a.w != nullptr, post = BLOCK == BLOCK_NORM && a.w_post != nullptr;
  float w[NV][P], wp[NV][P];
  // parts of dw and dw_post: 64 bits, or (two eights a thread, where those do not fit the registers) fp32 over kFold rows,
  // folded into 64 bits in LDS
  constexpr bool FOLD = EIGHTS == 2 && TPR == 512;
  using Acc = std::conditional_t<FOLD, float, double>;
  Acc acc[NV][P], acc_post[NV][P];
  __shared__ double kept_sums[FOLD ? 2 : 1][FOLD ? NV : 1][FOLD ? P : 1][FOLD ? TPR : 1];
  auto fold = [&](Acc (&v)[NV][P], int which) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < P; ++i) {
        kept_sums[which][k][i][tid] += double(v[k][i]);
        v[k][i] = 0;
      }
  };
  int since = 0;  // rows since the last fold
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = P * (tid + TPR * k);
    if (pre) get_weight<MOVED>(a.w, a.w_f32, c, D, w[k]);
    if (post) get_weight<MOVED>(a.w_post, a.w_f32, c, D, wp[k]);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      acc[k][i] = acc_post[k][i] = 0;
      if constexpr (FOLD) kept_sums[0][k][i][tid] = kept_sums[1][k][i][tid] = 0.;
      if (!post) wp[k][i] = 1.f;
    }
  }
  // a row ahead; a row behind the last one is a row of zeros
  struct Row {
    Piece<IO, P, MOVED> b[NV], dy[NV];
    Piece<R, P, MOVED> h[NV], dh[NV];
  } next;
  auto fetch = [&](int64_t t) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = P * (tid + TPR * k);
      next.b[k].clear(); next.dy[k].clear(); next.h[k].clear(); next.dh[k].clear();
      if (t >= a.T) continue;
      if (a.dh != nullptr) next.dh[k].get(static_cast<const R*>(a.dh) + t * a.ld_h, c, D);
      if (pre && a.dy != nullptr) {
        next.h[k].get(static_cast<const R*>(a.h) + t * a.ld_h, c, D);
        next.dy[k].get(static_cast<const IO*>(a.dy) + t * a.ld_y, c, D);
      }
      if (BLOCK == BLOCK_NORM) next.b[k].get(static_cast<const IO*>(a.b) + t * a.ld_b, c, D);
    }
  };
  const int64_t step = int64_t(gridDim.x) * ROWS;
  constexpr bool AHEAD = TPR < 1024;
  if (AHEAD) fetch(int64_t(blockIdx.x) * ROWS + row);
  for (int64_t first = int64_t(blockIdx.x) * ROWS; first < a.T; first += step) {
    const int64_t t = first + row;
    const bool there = t < a.T;
    float g[NV][P], x[NV][P], e[NV][P], bv[NV][P];
    float sum[3] = {0.f, 0.f, 0.f};  // h^2, e h, b^2
    if (!AHEAD) fetch(t);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = P * (tid + TPR * k);
      next.dh[k].mend(c, D);
      next.dh[k].values(g[k]);
      next.h[k].mend(c, D);
      next.h[k].values(x[k]);
      next.dy[k].mend(c, D);
      next.dy[k].values(e[k]);
      if (BLOCK == BLOCK_NORM) {
        next.b[k].mend(c, D);
        next.b[k].values(bv[k]);
      }
    }
    if (AHEAD && first + step < a.T) fetch(t + step);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (pre) {
          sum[0] = __builtin_fmaf(x[k][i], x[k][i], sum[0]);
          sum[1] = __builtin_fmaf(e[k][i] * w[k][i], x[k][i], sum[1]);
        }
        if (post) sum[2] = __builtin_fmaf(bv[k][i], bv[k][i], sum[2]);
      }
    row_sums<TPR>(sum, red, row, half);
    if (pre && a.dy != nullptr && there) {
      const float q = inverse_root(__builtin_fmaf(sum[0], inv_d, a.eps));
      const float m = sum[1] * inv_d * q * q;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) {
          acc[k][i] += Acc(e[k][i] * (x[k][i] * q));
          g[k][i] = __builtin_fmaf(q, __builtin_fmaf(-x[k][i], m, e[k][i] * w[k][i]), g[k][i]);
        }
    }
    R* dr = static_cast<R*>(a.dr) + t * a.ld_r;
    IO* db = static_cast<IO*>(a.db) + t * a.ld_b;
    if (there) {
#pragma unroll
      for (int k = 0; k < NV; ++k) put(dr, P * (tid + TPR * k), D, g[k]);
    }
    if constexpr (BLOCK == BLOCK_SUM) {
      if (there) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
          for (int i = 0; i < P; ++i) g[k][i] *= a.scale;
          put(db, P * (tid + TPR * k), D, g[k]);
        }
      }
    } else if constexpr (BLOCK == BLOCK_NORM) {
      float by = a.scale, rest = 0.f;
      if (a.gate != nullptr) {
        const float z = a.gate[there ? t : 0];
        by = sigmoid_times(a.scale, z);
        rest = sigmoid_times(1.f, -z);
      }
      float dot[1] = {0.f};
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) dot[0] = __builtin_fmaf(g[k][i] * wp[k][i], bv[k][i], dot[0]);
      row_sums<TPR>(dot, red, row, half);
      if (there) {
        const float p = post ? inverse_root(__builtin_fmaf(sum[2], inv_d, a.eps)) : 1.f;
        if (a.gate != nullptr && tid == 0) a.dgate[t] = by * rest * (dot[0] * p);
        const float m = post ? dot[0] * inv_d * p * p : 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          float o[P];
#pragma unroll
          for (int i = 0; i < P; ++i) {
            if (post) acc_post[k][i] += Acc(by * g[k][i] * (bv[k][i] * p));
            o[i] = by * p * __builtin_fmaf(-bv[k][i], m, g[k][i] * wp[k][i]);
          }
          put(db, P * (tid + TPR * k), D, o);
        }
      }
    }
    if constexpr (FOLD) {
      if (++since == kFold) {
        if (pre) fold(acc, 0);
        if (post) fold(acc_post, 1);
        since = 0;
      }
    }
  }
  // the workgroup's rows, then its row of the scratch
  auto store = [&](Acc (&v)[NV][P], int which, float* part) __attribute__((always_inline)) {
    if constexpr (FOLD) {
      fold(v, which);
      float f[P];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < P; ++i) f[i] = float(kept_sums[which][k][i][tid]);
        put(part + size_t(blockIdx.x) * D, P * (tid + TPR * k), D, f);
      }
    } else if constexpr (ROWS > 1) {
      __shared__ double s[ROWS - 1][NV][P][TPR];
      __syncthreads();
      if (row > 0) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < P; ++i) s[row - 1][k][i][tid] = v[k][i];
      }
      __syncthreads();
      if (row > 0) return;
      float f[P];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          double sum = v[k][i];
#pragma unroll
          for (int r = 0; r < ROWS - 1; ++r) sum += s[r][k][i][tid];
          f[i] = float(sum);
        }
        put(part + size_t(blockIdx.x) * D, P * (tid + TPR * k), D, f);
      }
    } else {
      float f[P];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < P; ++i) f[i] = float(v[k][i]);
        put(part + size_t(blockIdx.x) * D, P * (tid + TPR * k), D, f);
      }
    }
  };
  if (pre) store(acc, 0, a.part);
  if (post) store(acc_post, 1, a.part_post);
}

// The rows of the scratch, sixteen columns a workgroup: 64 rows side by side, four a wave.
__global__ void __launch_bounds__(1024) norm_finish_kernel(const float* __restrict__ part, const float* __restrict__ part_post,
                                                           int rows, int D, float* __restrict__ dw,
                                                           float* __restrict__ dw_post) {
  __shared__ double s[16][16];
  const int l = threadIdx.x & 15, c = blockIdx.x * 16 + l;
  const bool second = blockIdx.y == 1 || dw == nullptr;
  const float* in = second ? part_post : part;
  double v = 0.;
  if (c < D) {
#pragma unroll 8
    for (int k = threadIdx.x >> 4; k < rows; k += 64) v += double(in[size_t(k) * D + c]);
  }
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  if ((threadIdx.x & 63) < 16) s[threadIdx.x >> 6][l] = v;
  __syncthreads();
  if (threadIdx.x >= 16 || c >= D) return;
#pragma unroll
  for (int k = 1; k < 16; ++k) v += s[k][l];
  (second ? dw_post : dw)[c] = float(v);
}

// f(threads a row, eights of values a thread) for a row of D: one eight as long as a row has no more threads than 512, so
// that short rows keep all lanes busy (65536 x 128 forward and backward 34 us, with 64 threads a row 83; x 256 61, so 110).
template <class F>
int with_row(int D, F&& f) {
  using std::integral_constant;
  if (D <= 128) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if (D <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (D <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  if (D <= 1024) return f(integral_constant<int, 128>{}, integral_constant<int, 1>{});
  if (D <= 2048) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  if (D <= 4096) return f(integral_constant<int, 512>{}, integral_constant<int, 1>{});
  if (D <= 8192) return f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  return f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
}
int rows_a_workgroup(int D) { return D <= 128 ? 16 : D <= 256 ? 8 : D <= 512 ? 4 : D <= 1024 ? 2 : 1; }
// f(IO, R, MOVED) by example.
template <class F>
int with_types(const moe_norm_desc& d, F&& f) {
  const std::true_type yes;
  const std::false_type no;
  const bool io = d.io_type == MOE_TYPE_F32, res = d.res_type == MOE_TYPE_F32;
  if (io) return res ? f(float(), float(), no) : f(float(), uint16_t(), no);
  if (res) return f(uint16_t(), float(), no);
  // rows that fill their threads' pieces (with_row's powers of two), or past those at least whole pieces
  const bool whole = d.D <= 4096 ? d.D >= 128 && (d.D & (d.D - 1)) == 0 : d.D % 8 == 0;
  return whole ? f(uint16_t(), uint16_t(), no) : f(uint16_t(), uint16_t(), yes);
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

// Alignment of all, and written ones apart from all others but for out[mine] over in[theirs], the same
// rows (-1: none).
int check_buffers(const Buffer* in, int n_in, const Buffer* out, int n_out, int mine, int theirs) {
  for (int i = 0; i < n_in; ++i)
    if (!aligned_to(in[i].p, in[i].align)) return MOE_EALIGN;
  for (int i = 0; i < n_out; ++i)
    if (!aligned_to(out[i].p, out[i].align)) return MOE_EALIGN;
  for (int i = 0; i < n_out; ++i) {
    for (int k = 0; k < n_in; ++k)
      if (overlap(out[i].p, out[i].n, in[k].p, in[k].n) && !(i == mine && k == theirs)) return MOE_EINVAL;
    for (int k = 0; k < i; ++k)
      if (overlap(out[i].p, out[i].n, out[k].p, out[k].n)) return MOE_EINVAL;
  }
  return MOE_OK;
}

// Workgroups of a backward, so rows of the scratch: as many as there is room for (8 to 12 waves a CU).  16384 x 2048 forward
// and backward 115 us with 768, 129 with 256; 16384 x 4096 of an fp32 residual 382 with 768, 366 with 256.
int norm_partials(const moe_norm_desc& d) {
  const long long most = d.D <= 2048 ? 768 : 256, want = ceil_div(d.T, rows_a_workgroup(d.D));
  return int(std::max(1ll, std::min(most, want)));
}

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
  if (const int rc = check_buffers(in, 5, out, 2, in_place ? 0 : -1, 1)) return rc;
  NormArgs a{};
  a.b = b; a.r = r; a.w_post = w_post; a.w = w; a.gate = gate; a.h = h; a.y = y;
  a.ld_b = d->ld_b; a.ld_r = d->ld_r; a.ld_h = d->ld_h; a.ld_y = d->ld_y;
  a.T = d->T; a.D = d->D; a.eps = d->eps; a.scale = d->scale;
  a.inv_d = 1. / d->D;
  a.w_f32 = d->w_type == MOE_TYPE_F32;
  hipStream_t s = static_cast<hipStream_t>(stream);
  prof_begin("norm_fwd", s);
  with_types(*d, [&](auto io, auto res, auto moved) {
    return with_row(d->D, [&](auto threads, auto nv) {
      constexpr int W = decltype(threads)::value, NV = decltype(nv)::value;
      using IO = decltype(io);
      using R = decltype(res);
      constexpr bool M = decltype(moved)::value;
      // a workgroup for each row or rows: 1024 that step through 16384 rows of 4096 take 383 us forward and backward, so 366
      const unsigned grid = unsigned(std::min(ceil_div(d->T, norm_rows(W)), (1LL << 32) / norm_threads(W) - 1));
      if (b == nullptr) norm_fwd_kernel<IO, R, BLOCK_NONE, W, NV, M><<<grid, norm_threads(W), 0, s>>>(a);
      else if (gate != nullptr || w_post != nullptr) norm_fwd_kernel<IO, R, BLOCK_NORM, W, NV, M><<<grid, norm_threads(W), 0, s>>>(a);
      else norm_fwd_kernel<IO, R, BLOCK_SUM, W, NV, M><<<grid, norm_threads(W), 0, s>>>(a);
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
  if (const int rc = check_buffers(in, 7, out, 6, in_place ? 1 : -1, 6)) return rc;
  if (scratch_bytes < need) return MOE_ESCRATCH;
  NormArgs a{};
  a.b = b; a.w_post = w_post; a.w = w; a.gate = gate; a.h = const_cast<void*>(h);
  a.dy = dy; a.dh = dh; a.db = db; a.dr = dr; a.dgate = dgate;
  a.part = static_cast<float*>(scratch);
  a.part_post = reinterpret_cast<float*>(static_cast<char*>(scratch) + need / 2);
  a.ld_b = d->ld_b; a.ld_r = d->ld_r; a.ld_h = d->ld_h; a.ld_y = d->ld_y;
  a.T = d->T; a.D = d->D; a.eps = d->eps; a.scale = d->scale;
  a.inv_d = 1. / d->D;
  a.w_f32 = d->w_type == MOE_TYPE_F32;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const unsigned grid = unsigned(norm_partials(*d));
  if (d->T > 0) {
    prof_begin("norm_bwd", s);
    with_types(*d, [&](auto io, auto res, auto moved) {
      return with_row(d->D, [&](auto threads, auto nv) {
        constexpr int W = decltype(threads)::value, NV = decltype(nv)::value;
        using IO = decltype(io);
        using R = decltype(res);
        constexpr bool M = decltype(moved)::value;
        if (db == nullptr) norm_bwd_kernel<IO, R, BLOCK_NONE, W, NV, M><<<grid, norm_threads(W), 0, s>>>(a);
        else if (block) norm_bwd_kernel<IO, R, BLOCK_NORM, W, NV, M><<<grid, norm_threads(W), 0, s>>>(a);
        else norm_bwd_kernel<IO, R, BLOCK_SUM, W, NV, M><<<grid, norm_threads(W), 0, s>>>(a);
        return 0;
      });
    });
    prof_end(s);
    if (const int rc = launched()) return rc;
  }
  if (dw == nullptr && dw_post == nullptr) return MOE_OK;
  prof_begin("norm_finish", s);
  const dim3 blocks(unsigned(ceil_div(d->D, 16)), dw != nullptr && dw_post != nullptr ? 2 : 1);
  norm_finish_kernel<<<blocks, 1024, 0, s>>>(a.part, a.part_post, d->T > 0 ? int(grid) : 0, d->D, dw, dw_post);
  prof_end(s);
  return launched();
}

}  // extern "C"
