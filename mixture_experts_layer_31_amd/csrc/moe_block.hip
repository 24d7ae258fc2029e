// Dense e4m3 operands with one fp32 scale for each block of 128, and their product
// (moe_block_quant, moe_block_mm in moe.h).
//
// Quantiser.  s = amax / 448 over a 1 x 128 run or a 128 x 128 block, code =
// e4m3(x / s) of the fp32 quotient.  The quotient must be the correctly rounded one
// (it decides between two codes when it lies next to their border), without the
// eight-odd instructions of a division: q0 = x r with r = 1 / s, then two steps
// q <- q - r (q s - x), each with an exact residual in one FMA; the first leaves q
// within an ulp, and from there the second rounds correctly (Markstein's theorem:
// r is the correctly rounded reciprocal).  Where x is -0 the residual is +0, so that q stays
// -0 (x - q s would be +0 too, and q + 0 = +0).  Residuals and r stay in range because
// a run with a small amax is first scaled by a power of two, which the quotient does
// not see.
//
// Product.  C[m, n] = sum over runs b of 128 of sA[b, m] sB[b, n] P_b[m, n], P_b =
// sum_{k in b} A[m, k] B[n, k] from the matrix core; each run's P_b is promoted
// into the fp32 result on the vector ALU.  The codes become bf16 (exact) in registers for
// the bf16 matrix instruction, whose products are exact and whose sums are fp32's (5e-9 to 4e-8
// off, relative 2-norm, normal data), at 2.3 PFLOP/s in registers.  The e4m3 matrix instruction has
// twice that rate and is not used: it adds eight products at a time, each cut at 13 bits below
// the largest one's leading bit (beside products of +-2^16 one of 2^3 survives and one of 2^2
// does not), so where large terms cancel the rest of the sum is lost.  Its results are 1.5e-5 off on normal
// data, and 16384 x 4096 x 4096 took 232 us with it against 495.
#include <type_traits>

#include "moe_args.h"
#include "moe_gemm_common.h"

namespace moe {
namespace {

using namespace gemm;

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int64_t kMaxStride = 1 << 22;  // a 256-row tile of codes stays within 2^30 bytes

// ---------------------------------------------------------------------------
// Quantiser.

// The scale of a run with the given amax, and what its quotients are formed with.
struct Quant {
  float scale;     // stored: amax / 448, 1 where that is 0
  float s, r, up;  // quotient of x: (x up) / s with s = scale up, r = 1 / s
  __device__ __forceinline__ explicit Quant(float amax) {
    scale = amax / 448.f;
    if (scale == 0.f) scale = 1.f;
    up = scale < 0x1p-60f ? 0x1p+80f : 1.f;
    s = scale * up;
    r = 1.f / s;
    if (r == 0.f) s = 1.f;  // an infinite scale: 0 of what is finite, NaN of what is not
  }
  __device__ __forceinline__ float quotient(float x) const {
    x *= up;
    float q = x * r;
    q = __builtin_fmaf(-__builtin_fmaf(q, s, -x), r, q);
    return __builtin_fmaf(-__builtin_fmaf(q, s, -x), r, q);
  }
  __device__ __forceinline__ uint32_t codes(float a, float b, float c, float d) const {
    return pack_e4m3x4(quotient(a), quotient(b), quotient(c), quotient(d));
  }
  // Values of type T whose quotients may pass 448, where the conversion would give NaN, as those that saturate: a scale of a
  // few of the smallest numbers is rounded by up to half.  Above 2^9 of them quotients are 448.5 at most, and bf16's
  // smallest number has a scale of 146.
  template <class T, int N>
  __device__ __forceinline__ void saturate(float (&x)[N]) const {
    if (sizeof(T) == 4 && __ballot(scale < 0x1p-140f) != 0) {
      const float top = scale < 0x1p-140f ? 448.f * scale : INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i)  // a NaN stays
        x[i] = __builtin_elementwise_minimum(__builtin_elementwise_maximum(x[i], -top), top);
    }
  }
  template <class T>
  __device__ __forceinline__ uint2 codes8(const float (&v)[8]) const {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i];
    saturate<T>(x);
    return make_uint2(codes(x[0], x[1], x[2], x[3]), codes(x[4], x[5], x[6], x[7]));
  }
};

struct QuantArgs {
  const void* x;
  int64_t ldx, ldq, ldt;
  int rows, cols, ctiles;
  uint8_t* q;    // [rows, ldq] or null
  float* sc;
  uint8_t* qt;   // [cols, ldt] or null
  float* sct;
};

template <class T>
__device__ __forceinline__ void as_floats(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 2) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    } else {
      f[j] = __uint_as_float(w[j]);
    }
  }
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// One workgroup of 256 threads takes a 128 x 128 tile.  Sixteen lanes share a row,
// eight consecutive values each, so a wave's load covers whole row segments, and a
// row's amax is four DPP moves.  For the transpose the tile goes through LDS.  With a
// scale for the block the codes do, since both outputs have the same ones, and a
// thread turns a 16 x 4 piece of them over in registers (4096 x 2048 bf16, both
// outputs: 8.5 us against 10.8 us with the values through LDS and coded twice).  With
// tiles the values do: a thread then holds half a column (64 values, the other half is
// in lane ^ 32), and its codes go back through LDS so that eight lanes store a row's
// 128 bytes.  16384 x 4096 bf16 in tiles: the transpose alone 36 us, 5.6 TB/s; both orientations 62 us,
// 4.3 TB/s, bound by two exact quotients a value.  (Column pairs in 32-bit LDS reads free of bank
// conflicts took the same time.)
template <class T, bool BLOCK>
__global__ void __launch_bounds__(256) block_quant_kernel(QuantArgs p) {
  constexpr int LD = 128 + 16 / sizeof(T);  // values: rows apart in banks, 16-byte aligned
  constexpr int LDC = 33;                   // codes: words
  __shared__ __attribute__((aligned(16))) char smem[BLOCK ? 128 * LDC * 4 : 128 * LD * sizeof(T)];
  __shared__ float red[4];
  const int rt = blockIdx.x / p.ctiles, ct = blockIdx.x - rt * p.ctiles;
  const int64_t r0 = int64_t(rt) * 128;
  const int c0 = ct * 128;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, l16 = lane & 15;
  const int rw = wv * 4 + (lane >> 4);
  T* tile = reinterpret_cast<T*>(smem);
  float v[8][8];
  {
    constexpr int N = 16 / sizeof(T), NP = 8 / N;  // pieces of eight elements
    const T* x = static_cast<const T*>(p.x);
    RowPiece<T> raw[8][NP];
    const bool wide = p.cols >= N, edge = c0 + 128 > p.cols;
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int64_t r = r0 + it * 16 + rw;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (wide) raw[it][i].load(x + r * p.ldx, c0 + 8 * l16 + i * N, p.cols, r < p.rows, x);
        else raw[it][i].load_short(x + r * p.ldx, c0 + 8 * l16 + i * N, p.cols, r < p.rows);
      }
    }
#pragma unroll
    for (int it = 0; it < 8; ++it)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (wide) raw[it][i].mend(edge);
        as_floats<T>(raw[it][i].v, v[it] + i * N);
      }
  }
  float amax = 0.f;
  if constexpr (BLOCK) {
#pragma unroll
    for (int it = 0; it < 8; ++it) amax = fmaxf(amax, amax8(v[it]));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
    if (lane == 0) red[wv] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const int rb = (p.rows + 127) / 128;
    if (tid == 0) {
      const float s = Quant(amax).scale;
      if (p.q) p.sc[int64_t(rt) * p.ctiles + ct] = s;
      if (p.qt) p.sct[int64_t(ct) * rb + rt] = s;
    }
  }
  const int cols16 = (p.cols + 15) & ~15;
  if (BLOCK || p.q != nullptr) {
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int64_t r = r0 + it * 16 + rw;
      const Quant qz(BLOCK ? amax : max16(amax8(v[it])));
      const uint2 w = qz.codes8<T>(v[it]);
      if (p.q != nullptr && r < p.rows && c0 + 8 * l16 < cols16) {
        *reinterpret_cast<uint2*>(p.q + r * p.ldq + c0 + 8 * l16) = w;
        if (!BLOCK && l16 == 0) p.sc[int64_t(ct) * p.rows + r] = qz.scale;
      }
      if constexpr (BLOCK) {
        uint32_t* at = reinterpret_cast<uint32_t*>(smem) + (it * 16 + rw) * LDC + 2 * l16;
        at[0] = w.x;
        at[1] = w.y;
      }
    }
  }
  if (p.qt == nullptr) return;
  const int rows16 = (p.rows + 15) & ~15;
  if constexpr (BLOCK) {
    __syncthreads();
    // columns 4 cg .. + 3, rows 16 rg .. + 15: eight lanes a column's 128 bytes
    const int rg = tid & 7, cg = tid >> 3;
    uint32_t t[4][4];  // [column][four rows]
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = reinterpret_cast<const uint32_t*>(smem)[(16 * rg + 4 * q + i) * LDC + cg];
      // bytes of two rows side by side, then of four
      const uint32_t a0 = __builtin_amdgcn_perm(u[1], u[0], 0x05010400), a1 = __builtin_amdgcn_perm(u[1], u[0], 0x07030602);
      const uint32_t b0 = __builtin_amdgcn_perm(u[3], u[2], 0x05010400), b1 = __builtin_amdgcn_perm(u[3], u[2], 0x07030602);
      t[0][q] = __builtin_amdgcn_perm(b0, a0, 0x05040100);
      t[1][q] = __builtin_amdgcn_perm(b0, a0, 0x07060302);
      t[2][q] = __builtin_amdgcn_perm(b1, a1, 0x05040100);
      t[3][q] = __builtin_amdgcn_perm(b1, a1, 0x07060302);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c0 + 4 * cg + c < p.cols && r0 + 16 * rg < rows16)
        *reinterpret_cast<uint4*>(p.qt + int64_t(c0 + 4 * cg + c) * p.ldt + r0 + 16 * rg) =
            make_uint4(t[c][0], t[c][1], t[c][2], t[c][3]);
    return;
  }
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    uint4* at = reinterpret_cast<uint4*>(tile + (it * 16 + rw) * LD + 8 * l16);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[it][i]);
    if constexpr (sizeof(T) == 2) {
      at[0] = make_uint4((w[0] >> 16) | (w[1] & 0xffff0000u), (w[2] >> 16) | (w[3] & 0xffff0000u),
                         (w[4] >> 16) | (w[5] & 0xffff0000u), (w[6] >> 16) | (w[7] & 0xffff0000u));
    } else {
      at[0] = make_uint4(w[0], w[1], w[2], w[3]);
      at[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
  __syncthreads();
  // column q, rows 64 h .. 64 h + 63
  const int q = wv * 32 + (lane & 31), h = lane >> 5;
  float u[64];
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const T e = tile[(64 * h + i) * LD + q];
    if constexpr (sizeof(T) == 2) u[i] = bf2f(e);
    else u[i] = e;
  }
#pragma unroll
  for (int i = 0; i < 64; ++i) amax = fmaxf(amax, fabsf(u[i]));
  amax = fmaxf(amax, __shfl_xor(amax, 32, 64));
  const Quant qz(amax);
  if (h == 0 && c0 + q < p.cols) p.sct[int64_t(rt) * p.cols + c0 + q] = qz.scale;
  qz.saturate<T>(u);
  uint4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* e = u + 16 * i;
    w[i] = make_uint4(qz.codes(e[0], e[1], e[2], e[3]), qz.codes(e[4], e[5], e[6], e[7]),
                      qz.codes(e[8], e[9], e[10], e[11]), qz.codes(e[12], e[13], e[14], e[15]));
  }
  __syncthreads();  // every wave is done with the tile
  auto at = [&](int row, int ch) { return smem + row * 128 + ((ch ^ (row & 7)) << 4); };
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(at(q, 4 * h + i)) = w[i];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int id = tid + 256 * k, row = id >> 3, ch = id & 7;
    if (c0 + row < p.cols && r0 + 16 * ch < rows16)
      *reinterpret_cast<uint4*>(p.qt + int64_t(c0 + row) * p.ldt + r0 + 16 * ch) =
          *reinterpret_cast<const uint4*>(at(row, ch));
  }
}

// Rows alone, in tiles: IT rows a thread and no LDS.
template <class T, int IT>
__global__ void __launch_bounds__(256) block_quant_rows_kernel(QuantArgs p) {
  constexpr int N = 16 / sizeof(T), NP = 8 / N;
  const int rt = blockIdx.x / p.ctiles, ct = blockIdx.x - rt * p.ctiles;
  const int lane = threadIdx.x & 63, l16 = lane & 15;
  const int64_t r0 = int64_t(rt) * (16 * IT) + (threadIdx.x >> 6) * 4 + (lane >> 4);
  const int c = ct * 128 + 8 * l16;
  const T* x = static_cast<const T*>(p.x);
  RowPiece<T> raw[IT][NP];
  const bool wide = p.cols >= N, edge = ct * 128 + 128 > p.cols;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int64_t r = r0 + it * 16;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (wide) raw[it][i].load(x + r * p.ldx, c + i * N, p.cols, r < p.rows, x);
      else raw[it][i].load_short(x + r * p.ldx, c + i * N, p.cols, r < p.rows);
    }
  }
  const int cols16 = (p.cols + 15) & ~15;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int64_t r = r0 + it * 16;
    float v[8];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (wide) raw[it][i].mend(edge);
      as_floats<T>(raw[it][i].v, v + i * N);
    }
    const Quant qz(max16(amax8(v)));
    const uint2 w = qz.codes8<T>(v);
    if (r < p.rows && c < cols16) {
      *reinterpret_cast<uint2*>(p.q + r * p.ldq + c) = w;
      if (l16 == 0) p.sc[int64_t(ct) * p.rows + r] = qz.scale;
    }
  }
}

template <class T>
void launch_quant_rows(const QuantArgs& a, hipStream_t s) {
  // two rows a thread where there are many (bf16, one against two: 256 x 4096 2.58 us, 2.71; 2048 x 4096
  // 6.43, 6.48; 4096 x 4096 12.1, 11.7; 16384 x 4096 37.2, 33.5 = 6 TB/s read and written; eight: 36.9)
  const long long slabs = ceil_div(a.rows, 16) * a.ctiles;
  if (slabs >= 8192) block_quant_rows_kernel<T, 2><<<unsigned(ceil_div(a.rows, 32) * a.ctiles), 256, 0, s>>>(a);
  else block_quant_rows_kernel<T, 1><<<unsigned(slabs), 256, 0, s>>>(a);
}

int launch_block_quant(const QuantArgs& a, int in_type, bool block, hipStream_t s) {
  const unsigned grid = unsigned(ceil_div(a.rows, 128) * a.ctiles);
  prof_begin("block_quant", s);
  if (a.qt == nullptr && !block) {
    if (in_type == MOE_TYPE_BF16) launch_quant_rows<uint16_t>(a, s);
    else launch_quant_rows<float>(a, s);
  } else if (in_type == MOE_TYPE_BF16) {
    if (block) block_quant_kernel<uint16_t, true><<<grid, 256, 0, s>>>(a);
    else block_quant_kernel<uint16_t, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (block) block_quant_kernel<float, true><<<grid, 256, 0, s>>>(a);
    else block_quant_kernel<float, false><<<grid, 256, 0, s>>>(a);
  }
  prof_end(s);
  return launched();
}

QuantArgs quant_args(const void* x, int rows, int cols, int64_t ldx) {
  QuantArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.rows = rows;
  a.cols = cols;
  a.ctiles = int(ceil_div(cols, 128));
  return a;
}

// ---------------------------------------------------------------------------
// Product.

struct MmArgs {
  int M, N, K, ntm, ntn, ksteps;
  const uint8_t* A;
  const float* SA;  // [ksteps][ldsa]
  int ldsa;
  const uint8_t* B;
  const float* SB;  // TILE: [ksteps][N]; BLOCK: [ceil(N/128)][ksteps]
  int64_t lda, ldb, ldc;
  void* C;
  bool add;         // C +=
  int ldsb;         // BLOCK: entries between rows of SB
  // The contraction in parts of `per` runs, a part a workgroup: the parts' sums go to
  // part [parts][M][ldp] and are added by block_join_kernel (null: one part, to C).
  int per;
  float* part;
  int64_t ldp;
};

// Makes p the arguments of the part that holds workgroup l; returns l's place in it.
template <bool B_TILE>
__device__ __forceinline__ int take_part(MmArgs& p, int l) {
  if (p.part == nullptr) return l;
  const int tiles = p.ntm * p.ntn, s = l / tiles, k0 = s * p.per;
  p.A += int64_t(k0) * 128;
  p.B += int64_t(k0) * 128;
  p.SA += int64_t(k0) * p.ldsa;
  p.SB += B_TILE ? int64_t(k0) * p.N : k0;
  p.part += int64_t(s) * p.M * p.ldp;
  p.K = min(p.K - k0 * 128, p.per * 128);
  p.ksteps = min(p.ksteps - k0, p.per);
  return l - s * tiles;
}

// A scale as m 2^e: the power goes into the operand when its codes are widened, which costs nothing
// (the conversion takes the exponent of `power`), and m stays for the promotion.  The product of two scales
// may lie far outside fp32's range where the result does not.  With 2^e in [2^-50, 2^51] no sum of a
// run's products passes 2^127 or is below 2^-118 unless it is 0.  m is in [1, 2) but for scales past that
// range: below 2^-50 it is smaller, from 2^52 on larger, and then the other scale's power (or the result's
// own range) leaves room for it, so that a run's sum times A's m and then B's m is infinite or subnormal
// only where the run's result is.
struct Scale {
  float power, m;
  __device__ __forceinline__ Scale() = default;
  __device__ __forceinline__ explicit Scale(float s) {
    power = __builtin_amdgcn_fmed3f(fabsf(s), 0x1p-50f, 0x1p51f);
    m = s * __uint_as_float(0x7f000000u - (__float_as_uint(power) & 0x7f800000u));
  }
};

// Both m of a run at once, where B has one for all columns (16384 x 4096 x 4096: 495 us, 539 with a
// multiplication more for each value).  Two finite ones past the range count as its end: a sum of 0 stays 0, another one is
// past the range by its power alone.
__device__ __forceinline__ float both(float a, float b) {
  const float p = a * b, end = copysignf(3.402823466e38f, p);
  return isinf(p) && !isinf(a) && !isinf(b) ? end : p;
}

// Eight of the fragment's codes, times the power of two in `power`, as bf16 (exact): the part s of its 32.
__device__ __forceinline__ bf16x8 widen(const i32x8& f, int s, float power) {
  bf16x8 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * s + i], power, false);
    const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * s + i], power, true);
    r[4 * i] = lo[0]; r[4 * i + 1] = lo[1]; r[4 * i + 2] = hi[0]; r[4 * i + 3] = hi[1];
  }
  return r;
}

// One 4-byte entry a lane into LDS at lds + 4 * lane.
__device__ __forceinline__ void dma4(i32x4 rsrc, uint32_t lds, int voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}

// Large products with bf16 results: 256 x 128 tiles of eight waves, 64 x 64 each, or, where those
// are too few, 128 x 128 (96 x 128) tiles of two groups of four waves, 64 x 64 (48 x 64) each, that
// share the runs and are joined at the end.  Two stages of a run each; a wave goes over its rows of 16 x 16 blocks.
// 16384 x 4096 x 4096: 495 us, 1.11 PFLOP/s, with tile scales 552; 4096 x 4096 x 4096 121 and 140 (a library's
// bf16 product on values 425 and 95).  Bound by the matrix instructions at the clock that the power
// allows: without the widening, or without the promotion, the same product takes as long.  256 x 256
// tiles took 476, and 637 with tile scales: their sums and operands do not fit the registers.
template <int MB_, int WGM_, int WGN_, int KG_>
struct LargeTile {
  static constexpr int MB = MB_, NB = 4, WGM = WGM_, WGN = WGN_, KG = KG_;
  static constexpr int BM = 16 * MB * WGM, BN = 16 * NB * WGN, WAVES = WGM * WGN, THREADS = 64 * WAVES * KG;
};

template <class TL, bool B_TILE>
__global__ void __launch_bounds__(TL::THREADS, 2) block_mm_large_kernel(MmArgs p) {
  constexpr int BM = TL::BM, BN = TL::BN, WAVES = TL::WAVES, MB = TL::MB, NB = TL::NB, KG = TL::KG;
  constexpr int QA = (BM + 63) / 64;  // 64 scales a wave: A's, then B's
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES + (64 * QA + BN) * 4, RING = 2 * STAGE;
  __shared__ __attribute__((aligned(1024))) char lds[KG * RING];
  int l = xcd_remap(blockIdx.x, gridDim.x);
  if constexpr (KG > 1) l = take_part<B_TILE>(p, l);
  int mt, nt;
  wgrad_mn(l, p.ntm, p.ntn, mt, nt);
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = wv / WAVES, wave = wv % WAVES, wm = wave / TL::WGN, wn = wave % TL::WGN;
  const int group_tid = wave * 64 + lane;
  char* smem = lds + kg * RING;
  const int m0 = mt * BM, n0 = nt * BN;
  const int mrows = min(BM, p.M - m0), nrows = min(BN, p.N - n0);
  const int kbytes = (p.K + 15) & ~15;
  KStager<BM, WAVES, 128> sa;
  sa.init(make_rsrc(p.A + int64_t(m0) * p.lda, uint32_t((mrows - 1) * p.lda + kbytes)),
          [&](int r) { return r < mrows ? int(r * p.lda) : -1; }, wave, lane);
  KStager<BN, WAVES, 128> sb;
  sb.init(make_rsrc(p.B + int64_t(n0) * p.ldb, uint32_t((nrows - 1) * p.ldb + kbytes)),
          [&](int r) { return r < nrows ? int(r * p.ldb) : -1; }, wave, lane);
  const uint32_t base = lds_addr(smem);
  const int nblocks = (p.N + 127) / 128;
  // scales, 64 a load; with more waves than loads some come twice
  constexpr int QB = BN / 64;
  static_assert(QA + QB <= WAVES, "a load of scales a wave");
  const int sq = wave % (QA + QB);
  const bool sis_a = sq < QA;
  const i32x4 rs = sis_a ? make_rsrc(p.SA, uint32_t(p.ksteps) * p.ldsa * 4u)
                         : make_rsrc(p.SB, (B_TILE ? uint32_t(p.ksteps) * p.N : uint32_t(nblocks) * p.ldsb) * 4u);
  const int sr = (sis_a ? sq : sq - QA) * 64 + lane;
  const int sstep = sis_a ? p.ldsa * 4 : B_TILE ? p.N * 4 : 4;
  const int soff = sr >= (sis_a ? mrows : nrows) ? int(0x80000000u)
                   : sis_a ? (m0 + sr) * 4 : B_TILE ? (n0 + sr) * 4 : (n0 + sr) / 128 * p.ldsb * 4;
  // Loads of the group's i-th step (run i KG + kg) into stage s, the q-th of NL; past the last
  // run they miss every buffer (no traffic) and bring zeros.
  constexpr int NL = decltype(sa)::NI + decltype(sb)::NI + 1;
  auto issue1 = [&](int s, int i, int q) __attribute__((always_inline)) {
    const uint32_t st = base + s * STAGE;
    const int kt = i * KG + kg;
    const bool there = kt < p.ksteps;
    constexpr int NA = decltype(sa)::NI, NBI = decltype(sb)::NI;
    const int kb = there ? kt * 128 : 0x40000000;
    if (q < NA) dma16(sa.rsrc, st + uint32_t(wave * NA + q) * 1024u, sa.vb[q] + kb);
    else if (q < NA + NBI)
      dma16(sb.rsrc, st + A_BYTES + uint32_t(wave * NBI + q - NA) * 1024u, sb.vb[q - NA] + kb);
    else dma4(rs, st + A_BYTES + B_BYTES + sq * 256, there ? soff + kt * sstep : int(0x80000000u));
  };
  auto issue = [&](int s, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NL; ++q) issue1(s, i, q);
  };
  f32x4 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{};
  // fragments of a stage: chunks g and g + 4 of the lane's row
  const int sw = (l16 >> 1) & 7;
  const char* f0 = smem + l16 * 128 + ((g ^ sw) << 4);
  const char* f1 = smem + l16 * 128 + (((g + 4) ^ sw) << 4);
  auto frag = [&](int at) __attribute__((always_inline)) {
    const i32x4 x = *reinterpret_cast<const i32x4*>(f0 + at);
    const i32x4 y = *reinterpret_cast<const i32x4*>(f1 + at);
    return i32x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
  };
  const char* sap = smem + A_BYTES + B_BYTES + (wm * 16 * MB + l16) * 4;
  const char* sbp = smem + A_BYTES + B_BYTES + QA * 256 + (wn * 16 * NB + (B_TILE ? 4 * g : 0)) * 4;
  auto frag_a = [&](int st, int i) __attribute__((always_inline)) { return frag(st + (wm * MB + i) * 2048); };
  auto frag_b = [&](int st, int j) __attribute__((always_inline)) {
    return frag(st + A_BYTES + (wn * NB + j) * 2048);
  };
  auto scale_a = [&](int st, int i) __attribute__((always_inline)) {
    return *reinterpret_cast<const float*>(sap + st + i * 64);
  };
  constexpr int NS = B_TILE ? NB : 1;
  using SB_ = typename std::conditional<B_TILE, f32x4, float>::type;
  auto scale_b = [&](int st, int j) __attribute__((always_inline)) {
    return *reinterpret_cast<const SB_*>(sbp + st + j * 64);
  };
  // the scale of the lane's row of B in a fragment
  const char* sbr = smem + A_BYTES + B_BYTES + QA * 256 + (wn * 16 * NB + l16) * 4;
  auto row_scale_b = [&](int st, int j) __attribute__((always_inline)) {
    return *reinterpret_cast<const float*>(sbr + st + j * 64);
  };
  // A step goes over its MB blocks of 16 rows of A against the NB blocks of B, two of those at a time.
  // A block's codes are widened while the one before it is multiplied, and a pair's run sums are promoted
  // during the next pair's products: a wave that promotes right behind its own product stalls on it.
  bf16x8 wb[NB][4], wa[4];
  i32x8 rb[2];        // the last pair of B, widened during the step's first products, and its scales
  float rs2[2];
  SB_ sbv[NS] = {};
  float sav = 0.f, sp = 0.f;  // m of the current block of A; of the one promoted last, with block scales times B's
  f32x4 R[2] = {};    // run sums of the last pair
  auto widen_all = [&](const i32x8& f, float scale, bf16x8 (&w)[4]) __attribute__((always_inline)) {
    const Scale s(scale);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = widen(f, e, s.power);
    return s.m;
  };
  auto open = [&](int st) __attribute__((always_inline)) {
    sav = widen_all(frag_a(st, 0), scale_a(st, 0), wa);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      widen_all(frag_b(st, j), row_scale_b(st, j), wb[j]);
      rb[j] = frag_b(st, j + 2);
      rs2[j] = row_scale_b(st, j + 2);
    }
  };
  auto products = [&](int j0, f32x4 (&q)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        q[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j0 + j][e], wa[e], e ? q[j] : f32x4{}, 0, 0, 0);
  };
  auto promote = [&](int i, int j, const f32x4& part, float m) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (B_TILE) acc[i][j][e] = __builtin_fmaf(part[e] * m, sbv[j][e], acc[i][j][e]);
      else acc[i][j][e] = __builtin_fmaf(part[e], m, acc[i][j][e]);
    }
  };
  // Block i of stage st; `next` is what follows: 0 its next block, 1 the first one of stage sn, 2 nothing
  // that can be read yet.  `loads(q)` issues what goes with quarter q of it.
  auto row = [&](auto next, int st, int i, int sn, auto loads) __attribute__((always_inline)) {
    constexpr int NEXT = decltype(next)::value;
    i32x8 an, bn[2];
    float san = 0.f, sbn[2];
    if constexpr (NEXT < 2) {
      an = NEXT ? frag_a(sn, 0) : frag_a(st, i + 1);
      san = NEXT ? scale_a(sn, 0) : scale_a(st, i + 1);
    }
    if constexpr (NEXT == 1) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        bn[j] = frag_b(sn, j);
        sbn[j] = row_scale_b(sn, j);
      }
    }
    f32x4 Q[2];
    loads(0);
    products(0, Q);
    loads(1);
#pragma unroll
    for (int j = 0; j < 2; ++j) promote(i > 0 ? i - 1 : MB - 1, j + 2, R[j], sp);
    if (i == 0) {
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        sbv[j] = scale_b(st, j);
        if constexpr (B_TILE) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sbv[j][e] = Scale(sbv[j][e]).m;
        } else {
          sbv[j] = Scale(sbv[j]).m;
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) widen_all(rb[j], rs2[j], wb[j + 2]);
    }
    if constexpr (NEXT == 1) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        rb[j] = frag_b(sn, j + 2);
        rs2[j] = row_scale_b(sn, j + 2);
      }
    }
    loads(2);
    products(2, R);
    loads(3);
    if constexpr (B_TILE) sp = sav; else sp = both(sav, sbv[0]);
#pragma unroll
    for (int j = 0; j < 2; ++j) promote(i, j, Q[j], sp);
    if constexpr (NEXT < 2) sav = widen_all(an, san, wa);
    if constexpr (NEXT == 1) {
#pragma unroll
      for (int j = 0; j < 2; ++j) widen_all(bn[j], sbn[j], wb[j]);
    }
    if constexpr (NEXT == 0) {
      __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  using same_stage = std::integral_constant<int, 0>;
  using next_stage = std::integral_constant<int, 1>;
  using nothing = std::integral_constant<int, 2>;
  const auto none = [](int) __attribute__((always_inline)) {};
  // the last step's codes behind column K become 0, once its stage has arrived
  const bool tail = p.K % 128 != 0;
  auto mend = [&](int st) __attribute__((always_inline)) {
    if ((p.ksteps - 1) % KG == kg) {
      const int kr = p.K % 128;
      for (int r = group_tid; r < BM + BN; r += 64 * WAVES) {
        char* at = smem + st + r * 128;  // B's rows follow A's
        const int w8 = swz_k(r < BM ? r : r - BM);
        for (int c = kr >> 4; c < 8; ++c) {
          uint32_t* w = reinterpret_cast<uint32_t*>(at + ((c ^ w8) << 4));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int keep = kr - c * 16 - 4 * j;  // bytes of this word that exist
            if (keep <= 0) w[j] = 0;
            else if (keep < 4) w[j] &= (1u << (8 * keep)) - 1;
          }
        }
      }
    }
    __syncthreads();
  };
  const int n = (p.ksteps + KG - 1) / KG;  // steps a group
  // A step's loads are issued over the last products of the step two before it, into the stage that has
  // just been read, a quarter with each eight products (in one burst they hold up the fragment reads).
  issue(0, 0);
  issue(1, 1);
  wait_vmcnt<NL>();
  __builtin_amdgcn_s_barrier();
  if (tail && n == 1) mend(0);
  open(0);
  int kt = 0, st = 0;
  const int straight = n - 1 - (tail ? 1 : 0);  // steps whose successor needs no mending
  for (; kt < straight; ++kt) {
    const int sn = STAGE - st;
#pragma unroll
    for (int i = 0; i < MB - 1; ++i) row(same_stage{}, st, i, sn, none);
    // with the last block of A in registers the stage is read: the next one takes over, its
    // fragments replacing those of B as the last products release them
    wait_lgkm0();
    wait_vmcnt<0>();
    __builtin_amdgcn_s_barrier();
    row(next_stage{}, st, MB - 1, sn, [&](int r) __attribute__((always_inline)) {
#pragma unroll
      for (int q = r * NL / 4; q < (r + 1) * NL / 4; ++q) issue1(st ? 1 : 0, kt + 2, q);
    });
    st = sn;
  }
  const auto last_rows = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MB - 1; ++i) row(same_stage{}, st, i, 0, none);
    row(nothing{}, st, MB - 1, 0, none);
  };
  if (tail && n > 1) {
    last_rows();
    wait_lgkm0();
    wait_vmcnt<0>();
    __builtin_amdgcn_s_barrier();
    st = STAGE - st;
    mend(st);
    open(st);
  }
  last_rows();
#pragma unroll
  for (int j = 0; j < 2; ++j) promote(MB - 1, j + 2, R[j], sp);
  wait_vmcnt<0>();  // the loads that missed still write their zeros
  if constexpr (KG > 1) {  // join the groups' sums
    constexpr int LDR = BN + 4;
    static_assert(RING >= BM * LDR * 4, "the join fits a group's ring");
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        *reinterpret_cast<f32x4*>(smem + (((wm * MB + i) * 16 + l16) * LDR + (wn * NB + j) * 16 + 4 * g) * 4) = acc[i][j];
    __syncthreads();
    uint16_t* c = static_cast<uint16_t*>(p.C) + int64_t(m0) * p.ldc + n0;
#pragma unroll 2
    for (int e = threadIdx.x; e < BM * BN / 8; e += TL::THREADS) {
      const int r = e / (BN / 8), col = e % (BN / 8) * 8;
      if (r >= mrows || col >= nrows) continue;
      f32x4 v[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const char* at = lds + (r * LDR + col + 4 * q) * 4;
        v[q] = *reinterpret_cast<const f32x4*>(at);
#pragma unroll
        for (int x = 1; x < KG; ++x) v[q] += *reinterpret_cast<const f32x4*>(at + x * RING);
      }
      if (p.part != nullptr) {
        float* dst = p.part + int64_t(m0 + r) * p.ldp + n0 + col;
        *reinterpret_cast<f32x4*>(dst) = v[0];
        if (col + 4 < nrows) *reinterpret_cast<f32x4*>(dst + 4) = v[1];
        continue;
      }
      const uint32_t w[4] = {pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]),
                             pack_bf16x2(v[1][0], v[1][1]), pack_bf16x2(v[1][2], v[1][3])};
      uint16_t* dst = c + r * p.ldc + col;
      if (col + 8 <= nrows) {
        store16(dst, make_uint4(w[0], w[1], w[2], w[3]));
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (col + q < nrows) dst[q] = uint16_t(w[q >> 1] >> (16 * (q & 1)));
      }
    }
    return;
  }
  // Epilogue: the whole bf16 tile through LDS, whole rows out
  static_assert(BN / 8 <= 32 && RING >= BM * BN * 2, "the tile fits the ring, its rows have at most 32 chunks");
  __syncthreads();
  BandTile<2> t{smem, BN};
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      *reinterpret_cast<uint2*>(t.at((wm * MB + i) * 16 + l16, (wn * NB + j) * 16 + 4 * g)) =
          pack4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
  __syncthreads();
  uint16_t* c = static_cast<uint16_t*>(p.C) + int64_t(m0) * p.ldc + n0;
#pragma unroll 4
  for (int k = threadIdx.x; k < BM * (BN / 8); k += TL::THREADS) {
    const int r = k / (BN / 8), ch = k % (BN / 8);
    if (r >= mrows || ch * 8 >= nrows) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(smem + r * BN * 2 + ((ch ^ (r & (BN / 8 - 1))) << 4));
    uint16_t* dst = c + r * p.ldc + ch * 8;
    if (ch * 8 + 8 <= nrows) {
      store16(dst, v);
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (ch * 8 + e < nrows) dst[e] = uint16_t(w[e >> 1] >> (16 * (e & 1)));
    }
  }
}

template <class TL>
int launch_mm_large(const MmArgs& a, bool b_tile, hipStream_t s) {
  MmArgs p = a;
  p.ntm = int(ceil_div(p.M, TL::BM));
  p.ntn = int(ceil_div(p.N, TL::BN));
  const long long tiles = (long long)p.ntm * p.ntn * (p.part ? ceil_div(p.ksteps, p.per) : 1);
  const unsigned grid = unsigned(tiles);
  prof_begin("block_mm_large", s);
  if (b_tile) block_mm_large_kernel<TL, true><<<grid, TL::THREADS, 0, s>>>(p);
  else block_mm_large_kernel<TL, false><<<grid, TL::THREADS, 0, s>>>(p);
  prof_end(s);
  return launched();
}

// Products of a medium size, and all but the smallest with fp32 results: BM x BN tiles of WGM x WGN
// waves in 16 x 16 blocks, KG such groups a workgroup that share the runs of the contraction and
// are joined at the end.  Where tiles or steps are few, a step's latency is what it costs: a
// ring of four stages is filled four steps ahead, a step's fragments are read one step before
// their products, and a product's sums are promoted one step behind it (256 x 4096 x 4096 16.7 us, fp32 17).
template <int BM_, int BN_, int WGM_, int WGN_, int KG_>
struct MidTile {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, KG = KG_;
  static constexpr int WAVES = WGM * WGN, THREADS = 64 * WAVES * KG, MB = BM / WGM / 16, NB = BN / WGN / 16;
};

template <class TL, bool B_TILE, bool OUT_F32>
__global__ void __launch_bounds__(TL::THREADS) block_mm_mid_kernel(MmArgs p) {
  constexpr int BM = TL::BM, BN = TL::BN, KG = TL::KG, WAVES = TL::WAVES, MB = TL::MB, NB = TL::NB;
  constexpr int S = 4, A_BYTES = BM * 128, BYTES = (BM + BN) * 128, STAGE = BYTES + (BM + BN) * 4, RING = S * STAGE;
  constexpr int LDR = BN + 4;  // join: rows apart in banks
  static_assert(RING >= BM * LDR * 4, "the join fits a group's ring");
  __shared__ __attribute__((aligned(1024))) char smem[KG * RING];
  const int l = take_part<B_TILE>(p, xcd_remap(blockIdx.x, gridDim.x));
  int mt, nt;
  wgrad_mn(l, p.ntm, p.ntn, mt, nt);
  const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = wv / WAVES, wave = wv % WAVES, wm = wave / TL::WGN, wn = wave % TL::WGN;
  const int m0 = mt * BM, n0 = nt * BN;
  const int mrows = min(BM, p.M - m0), nrows = min(BN, p.N - n0);
  const int kbytes = (p.K + 15) & ~15;
  char* ring = smem + kg * RING;
  KStager<BM, WAVES, 128> sa;
  sa.init(make_rsrc(p.A + int64_t(m0) * p.lda, uint32_t((mrows - 1) * p.lda + kbytes)),
          [&](int r) { return r < mrows ? int(r * p.lda) : -1; }, wave, lane);
  KStager<BN, WAVES, 128> sb;
  sb.init(make_rsrc(p.B + int64_t(n0) * p.ldb, uint32_t((nrows - 1) * p.ldb + kbytes)),
          [&](int r) { return r < nrows ? int(r * p.ldb) : -1; }, wave, lane);
  constexpr int NA = decltype(sa)::NI, NBI = decltype(sb)::NI, NI = NA + NBI + 1;
  const int nblocks = (p.N + 127) / 128;
  // scales, 64 a load; with more waves than loads some come twice
  constexpr int QA = BM / 64, QB = BN / 64;
  static_assert(QA + QB <= WAVES, "a load of scales a wave");
  const int sq = wave % (QA + QB);
  const bool of_a = sq < QA;
  const i32x4 rs = of_a ? make_rsrc(p.SA, uint32_t(p.ksteps) * p.ldsa * 4u)
                        : make_rsrc(p.SB, (B_TILE ? uint32_t(p.ksteps) * p.N : uint32_t(nblocks) * p.ldsb) * 4u);
  const int sr = (of_a ? sq : sq - QA) * 64 + lane;
  const int sstep = of_a ? p.ldsa * 4 : B_TILE ? p.N * 4 : 4;
  const int soff = sr >= (of_a ? mrows : nrows) ? int(0x80000000u)
                   : of_a ? (m0 + sr) * 4 : B_TILE ? (n0 + sr) * 4 : (n0 + sr) / 128 * p.ldsb * 4;
  const uint32_t base = lds_addr(ring);
  // the group's i-th step is run i KG + kg; one past the last misses every buffer and loads zeros
  auto issue = [&](int i) __attribute__((always_inline)) {
    const uint32_t st = base + (i % S) * STAGE;
    const int kt = i * KG + kg;
    const bool there = kt < p.ksteps;
    const int kb = there ? kt * 128 : 0x40000000;
#pragma unroll
    for (int j = 0; j < NA; ++j) dma16(sa.rsrc, st + uint32_t(wave * NA + j) * 1024u, sa.vb[j] + kb);
#pragma unroll
    for (int j = 0; j < NBI; ++j)
      dma16(sb.rsrc, st + A_BYTES + uint32_t(wave * NBI + j) * 1024u, sb.vb[j] + kb);
    dma4(rs, st + BYTES + sq * 256, there ? soff + kt * sstep : int(0x80000000u));
  };
  const int sw = (l16 >> 1) & 7;
  const int f0 = l16 * 128 + ((g4 ^ sw) << 4), f1 = l16 * 128 + (((g4 + 4) ^ sw) << 4);
  using SB_ = typename std::conditional<B_TILE, f32x4, float>::type;
  struct Step {
    i32x8 a[MB], b[NB];
    float sa[MB], sr[NB];  // scales of the lane's rows of A and B
    SB_ sb[NB];            // and of its results' columns
  };
  auto read = [&](int i, Step& x) __attribute__((always_inline)) {
    const char* st = ring + (i % S) * STAGE;
    const float* sc = reinterpret_cast<const float*>(st + BYTES);
    auto frag = [&](const char* rows) __attribute__((always_inline)) {
      const i32x4 u = *reinterpret_cast<const i32x4*>(rows + f0), v = *reinterpret_cast<const i32x4*>(rows + f1);
      return i32x8{u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
    };
#pragma unroll
    for (int q = 0; q < MB; ++q) {
      const int r = (wm * MB + q) * 16;
      x.a[q] = frag(st + r * 128);
      x.sa[q] = sc[r + l16];
    }
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int r = (wn * NB + q) * 16;
      x.b[q] = frag(st + A_BYTES + r * 128);
      x.sr[q] = sc[BM + r + l16];
      x.sb[q] = *reinterpret_cast<const SB_*>(sc + BM + r + (B_TILE ? 4 * g4 : 0));
    }
  };
  f32x4 acc[MB][NB] = {}, P[MB][NB] = {};
  float psa[MB] = {};
  SB_ psb[NB] = {};
  auto promote = [&](int i, int j) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (B_TILE) acc[i][j][e] = __builtin_fmaf(P[i][j][e] * psa[i], psb[j][e], acc[i][j][e]);
      else acc[i][j][e] = __builtin_fmaf(P[i][j][e], psa[i], acc[i][j][e]);
    }
  };
  auto promote_all = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) promote(i, j);
  };
  auto multiply = [&](const Step& x) __attribute__((always_inline)) {
    promote_all();
    Scale ra[MB], rb[NB];
#pragma unroll
    for (int i = 0; i < MB; ++i) ra[i] = Scale(x.sa[i]);
#pragma unroll
    for (int j = 0; j < NB; ++j) rb[j] = Scale(x.sr[j]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bf16x8 wb[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) wb[j] = widen(x.b[j], e, rb[j].power);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const bf16x8 wa = widen(x.a[i], e, ra[i].power);
#pragma unroll
        for (int j = 0; j < NB; ++j)
          P[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], wa, e ? P[i][j] : f32x4{}, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      // the tile is in one block of B
      if constexpr (B_TILE) psa[i] = ra[i].m; else psa[i] = both(ra[i].m, Scale(x.sb[0]).m);
    }
    if constexpr (B_TILE) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) psb[j][e] = Scale(x.sb[j][e]).m;
    }
  };
  const int n = (p.ksteps + KG - 1) / KG;  // steps a group
  const bool tail = p.K % 128 != 0;
  // stage i has arrived for every wave; the last run's codes behind column K become 0
  auto arrive = [&](int i) __attribute__((always_inline)) {
    wait_lgkm0();
    wait_vmcnt<(S - 2) * NI>();
    __builtin_amdgcn_s_barrier();
    if (tail && i == n - 1) {
      if (i * KG + kg == p.ksteps - 1) {
        const int kr = p.K % 128;
        for (int r = wave * 64 + lane; r < BM + BN; r += 64 * WAVES) {  // B's rows follow A's
          char* at = ring + (i % S) * STAGE + r * 128;
          const int w8 = swz_k(r < BM ? r : r - BM);
          for (int c = kr >> 4; c < 8; ++c) {
            uint32_t* w = reinterpret_cast<uint32_t*>(at + ((c ^ w8) << 4));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int keep = kr - c * 16 - 4 * j;  // bytes of this word that exist
              if (keep <= 0) w[j] = 0;
              else if (keep < 4) w[j] &= (1u << (8 * keep)) - 1;
            }
          }
        }
      }
      wait_lgkm0();
      __builtin_amdgcn_s_barrier();
    }
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);
  // here S - 1 stages are on the way; `arrive` lets S - 2 of them be out
  Step x0, x1;
  arrive(0);
  issue(S - 1);
  read(0, x0);
  // step i: the next stage arrives, the one just read takes the loads four steps on
  auto step = [&](int i, const Step& cur, Step& nxt) __attribute__((always_inline)) {
    arrive(i + 1);
    issue(i + S);
    read(i + 1, nxt);
    __builtin_amdgcn_sched_barrier(0);  // the reads ahead of the products that hide them
    multiply(cur);
    // and the promotions here, not sunk into the next step behind its wait
#pragma unroll
    for (int r = 0; r < MB; ++r)
#pragma unroll
      for (int j = 0; j < NB; ++j) asm volatile("" : "+v"(acc[r][j]));
  };
  int i = 0;
  for (; i + 2 < n; i += 2) {
    step(i, x0, x1);
    step(i + 1, x1, x0);
  }
  if (i + 1 < n) {
    step(i, x0, x1);
    multiply(x1);
  } else {
    multiply(x0);
  }
  promote_all();
  wait_vmcnt<0>();  // loads that missed still write their zeros
  __syncthreads();
  float* red = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int r = 0; r < MB; ++r)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      *reinterpret_cast<f32x4*>(red + ((wm * MB + r) * 16 + l16) * LDR + (wn * NB + j) * 16 + 4 * g4) = acc[r][j];
  __syncthreads();
  using T = typename std::conditional<OUT_F32, float, uint16_t>::type;
  constexpr int VE = 16 / sizeof(T);
  T* c = static_cast<T*>(p.C) + int64_t(m0) * p.ldc + n0;
#pragma unroll
  for (int e = threadIdx.x; e < BM * BN / VE; e += TL::THREADS) {
    const int row = e / (BN / VE), col = e % (BN / VE) * VE;
    if (row >= mrows || col >= nrows) continue;
    float v[VE];
#pragma unroll
    for (int q = 0; q < VE; q += 4) {
      f32x4 t = *reinterpret_cast<const f32x4*>(smem + (row * LDR + col + q) * 4);
#pragma unroll
      for (int k = 1; k < KG; ++k) t += *reinterpret_cast<const f32x4*>(smem + k * RING + (row * LDR + col + q) * 4);
      v[q] = t[0]; v[q + 1] = t[1]; v[q + 2] = t[2]; v[q + 3] = t[3];
    }
    if (p.part != nullptr) {
      float* dst = p.part + int64_t(m0 + row) * p.ldp + n0 + col;
#pragma unroll
      for (int q = 0; q < VE; q += 4)
        if (col + q < nrows) *reinterpret_cast<f32x4*>(dst + q) = f32x4{v[q], v[q + 1], v[q + 2], v[q + 3]};
      continue;
    }
    T* dst = c + row * p.ldc + col;
    if (col + VE <= nrows) {
      if constexpr (OUT_F32) {
        if (p.add) {
          float o[4];
          as_floats<float>(load16(dst), o);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] += o[q];
        }
        store16(dst, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                __float_as_uint(v[3])));
      } else {
        store16(dst, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                pack_bf16x2(v[6], v[7])));
      }
    } else {
#pragma unroll
      for (int q = 0; q < VE; ++q)
        if (col + q < nrows) {
          if constexpr (OUT_F32) dst[q] = p.add ? dst[q] + v[q] : v[q];
          else dst[q] = uint16_t(pack_bf16x2(v[q], 0.f));
        }
    }
  }
}

template <class TL, bool BF16 = true>  // BF16: bf16 results take these tiles too
int launch_mm_mid(const MmArgs& a, bool b_tile, bool f32, hipStream_t s) {
  MmArgs p = a;
  p.ntm = int(ceil_div(p.M, TL::BM));
  p.ntn = int(ceil_div(p.N, TL::BN));
  const long long tiles = (long long)p.ntm * p.ntn * (p.part ? ceil_div(p.ksteps, p.per) : 1);
  const unsigned grid = unsigned(tiles);
  prof_begin("block_mm_mid", s);
  if (f32) {
    if (b_tile) block_mm_mid_kernel<TL, true, true><<<grid, TL::THREADS, 0, s>>>(p);
    else block_mm_mid_kernel<TL, false, true><<<grid, TL::THREADS, 0, s>>>(p);
  } else if constexpr (BF16) {
    if (b_tile) block_mm_mid_kernel<TL, true, false><<<grid, TL::THREADS, 0, s>>>(p);
    else block_mm_mid_kernel<TL, false, false><<<grid, TL::THREADS, 0, s>>>(p);
  }
  prof_end(s);
  return launched();
}

// Small products: 16 x 16 tiles of C, `wk` waves on a tile, its runs split over them and their
// sums joined in LDS in wave order.  B goes from memory to registers, a run ahead.  A as codes
// does too; A as values is quantised by the workgroup into LDS first (16 rows, up to kDirectK
// columns), while the first of B is on its way, so that the call is one launch.  Lane l of a
// fragment holds row l & 15 and bytes 32 (l >> 4) .. + 31 of a run, for A and B alike; with B as
// the first operand a lane's results are row l & 15 of C and columns 4 (l >> 4) .. + 3.
// Every workgroup of a row of tiles quantises its A again, which costs less than a second launch
// up to the size in use_direct.  1 x 4096 x 2048 from bf16: 4.8 us in a graph, 8.4 MB of codes, of it 3 a
// launch's; 33 x 1000 x 1363 from fp32: 7.7, of it 2 the quotients.
enum AKind { A_CODES = 0, A_BF16 = 1, A_F32 = 2 };
constexpr int kDirectWaves = 16, kDirectK = 4096;

struct DirectArgs {
  MmArgs m;
  const void* X;  // A as values
  int64_t ldx;
  int wk;         // waves a tile
};

// A quarter of a run of codes of a row on its way, from column k (k % 32 == 0).
struct RunPart {
  i32x4 c[2];
  int left;  // codes that exist from k on
  __device__ __forceinline__ void load(const uint8_t* row, int k, int K, bool ok) {
    left = ok ? K - k : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[i] = i32x4{};
      if (left > 16 * i) c[i] = *reinterpret_cast<const i32x4*>(row + k + 16 * i);
    }
  }
  __device__ __forceinline__ i32x8 codes() const {  // 0 behind column K
    i32x8 r;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int v = c[j >> 2][j & 3], keep = left - 4 * j;
      r[j] = keep >= 4 ? v : keep <= 0 ? 0 : v & int((1u << (8 * keep)) - 1);
    }
    return r;
  }
};

template <int AK, bool B_TILE, bool OUT_F32>
__global__ void __launch_bounds__(64 * kDirectWaves) block_direct_kernel(DirectArgs p) {
  constexpr bool VALUES = AK != A_CODES;
  constexpr int LDR = 20;           // join: rows apart in banks
  constexpr int LDA = kDirectK + 16;  // staged codes: 16 rows on 64 banks
  constexpr int STAGED = VALUES ? 16 * LDA + kDirectK / 128 * 64 : 0, JOIN = kDirectWaves * 16 * LDR * 4;
  __shared__ __attribute__((aligned(16))) char smem[STAGED > JOIN ? STAGED : JOIN];
  const MmArgs& q = p.m;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wt = wave / p.wk, kw = wave - wt * p.wk;  // tile of the workgroup, share of its runs
  const int mt = blockIdx.x % q.ntm, nt = blockIdx.x / q.ntm * int((blockDim.x >> 6) / p.wk) + wt;
  const int m = mt * 16 + l16, n = nt * 16 + l16, nc = nt * 16 + 4 * g;
  const uint8_t* arow = q.A + int64_t(m) * q.lda;
  const uint8_t* brow = q.B + int64_t(n) * q.ldb;
  const int nb = min(nt * 16, q.N - 1) >> 7;
  struct Run {
    RunPart a, b;
    float sa, sr, sb[B_TILE ? 4 : 1];  // scales of the lane's row of A, of B and of its results' columns
  };
  auto load = [&](int kt, Run& r) __attribute__((always_inline)) {
    const int k = kt * 128 + 32 * g;
    const bool run = kt < q.ksteps;
    if constexpr (!VALUES) {
      r.a.load(arow, k, q.K, m < q.M && run);
      r.sa = m < q.M && run ? q.SA[int64_t(kt) * q.ldsa + m] : 0.f;
    }
    r.b.load(brow, k, q.K, n < q.N && run);
    if constexpr (B_TILE) {
#pragma unroll
      for (int e = 0; e < 4; ++e) r.sb[e] = nc + e < q.N && run ? q.SB[int64_t(kt) * q.N + nc + e] : 0.f;
      r.sr = n < q.N && run ? q.SB[int64_t(kt) * q.N + n] : 0.f;
    } else {
      r.sr = r.sb[0] = q.SB[int64_t(nb) * q.ksteps + min(kt, q.ksteps - 1)];
    }
  };
  Run cur;
  load(kw, cur);
  float* scales = reinterpret_cast<float*>(smem + 16 * LDA);  // [run][row]
  if constexpr (VALUES) {
    using T = typename std::conditional<AK == A_BF16, uint16_t, float>::type;
    constexpr int N = 16 / sizeof(T), NP = 8 / N;
    const T* x = static_cast<const T*>(p.X);
    const int rows = min(16, q.M - mt * 16), groups = blockDim.x >> 4;
    const bool wide = q.K >= N;
    // sixteen lanes a run, in pairs of runs so that two loads are on their way
    for (int u = threadIdx.x >> 4; u < rows * q.ksteps; u += 2 * groups) {
      RowPiece<T> raw[2][NP];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int v = u + h * groups, r = v / q.ksteps, c = (v - r * q.ksteps) * 128 + 8 * l16;
        const T* row = x + int64_t(mt * 16 + r) * p.ldx;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          if (wide) raw[h][i].load(row, c + i * N, q.K, r < rows, x);
          else raw[h][i].load_short(row, c + i * N, q.K, r < rows);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int v = u + h * groups, r = v / q.ksteps, kt = v - r * q.ksteps;
        float f[8];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          if (wide) raw[h][i].mend(q.K % 128 != 0);
          as_floats<T>(raw[h][i].v, f + i * N);
        }
        const Quant qz(max16(amax8(f)));
        const uint2 w = qz.codes8<T>(f);
        if (r < rows) {
          *reinterpret_cast<uint2*>(smem + r * LDA + kt * 128 + 8 * l16) = w;
          if (l16 == 0) scales[kt * 16 + r] = qz.scale;
        }
      }
    }
    __syncthreads();
  }
  const int arl = VALUES ? min(l16, q.M - 1 - mt * 16) : 0;  // a row that is staged
  f32x4 acc = {};
  for (int kt = kw; kt < q.ksteps; kt += p.wk) {
    Run next;
    load(kt + p.wk, next);
    i32x8 a;
    float sa;
    if constexpr (VALUES) {
      const i32x4* s = reinterpret_cast<const i32x4*>(smem + arl * LDA + kt * 128 + 32 * g);
      const i32x4 u = s[0], v = s[1];
      a = i32x8{u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
      sa = scales[kt * 16 + arl];
    } else {
      a = cur.a.codes();
      sa = cur.sa;
    }
    const i32x8 b = cur.b.codes();
    const Scale ra(sa), rb(cur.sr);
    f32x4 part = {};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(b, e, rb.power), widen(a, e, ra.power), part, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (B_TILE) acc[e] = __builtin_fmaf(part[e] * ra.m, Scale(cur.sb[e]).m, acc[e]);
      else acc[e] = __builtin_fmaf(part[e], both(ra.m, rb.m), acc[e]);
    }
    cur = next;
  }
  using O = typename std::conditional<OUT_F32, float, uint16_t>::type;
  O* c = static_cast<O*>(q.C);
  auto put = [&](int r, int col, float s) __attribute__((always_inline)) {
    if (r >= q.M || col >= q.N) return;
    O* dst = c + int64_t(r) * q.ldc + col;
    if constexpr (OUT_F32) *dst = q.add ? *dst + s : s;
    else *dst = uint16_t(pack_bf16x2(s, 0.f));
  };
  if (p.wk == 1) {  // a tile a wave: nothing to join
#pragma unroll
    for (int e = 0; e < 4; ++e) put(m, nc + e, acc[e]);
    return;
  }
  if constexpr (VALUES) __syncthreads();  // the join overwrites the staged codes
  float* red = reinterpret_cast<float*>(smem);
  *reinterpret_cast<f32x4*>(red + (wave * 16 + l16) * LDR + 4 * g) = acc;
  __syncthreads();
  for (int e = kw * 64 + lane; e < 256; e += p.wk * 64) {
    const int r = e >> 4, col = e & 15;
    const float* t = red + (wt * p.wk * 16 + r) * LDR + col;
    float s = t[0];
    for (int w = 1; w < p.wk; ++w) s += t[w * 16 * LDR];
    put(mt * 16 + r, nt * 16 + col, s);
  }
}

template <int AK>
int launch_direct(const DirectArgs& a, bool b_tile, bool f32, hipStream_t s) {
  DirectArgs p = a;
  // a power of two of waves on a tile's runs, up to one each; at least eight waves a workgroup, the
  // rest of them on further tiles (a launch of thousands of single waves is slower than its work)
  p.wk = 1;
  while (p.wk < kDirectWaves && p.wk < p.m.ksteps) p.wk *= 2;
  const int waves = p.wk > 8 ? p.wk : 8;
  p.m.ntm = int(ceil_div(p.m.M, 16));
  const unsigned grid = unsigned(p.m.ntm) * unsigned(ceil_div(ceil_div(p.m.N, 16), waves / p.wk));
  prof_begin("block_direct", s);
  if (b_tile) {
    if (f32) block_direct_kernel<AK, true, true><<<grid, 64 * waves, 0, s>>>(p);
    else block_direct_kernel<AK, true, false><<<grid, 64 * waves, 0, s>>>(p);
  } else {
    if (f32) block_direct_kernel<AK, false, true><<<grid, 64 * waves, 0, s>>>(p);
    else block_direct_kernel<AK, false, false><<<grid, 64 * waves, 0, s>>>(p);
  }
  prof_end(s);
  return launched();
}

// C (+)= the sum of the parts, in their order; four columns a thread.
template <class T>
__global__ void __launch_bounds__(256) block_join_kernel(MmArgs p, int parts) {
  const int quads = int(p.ldp / 4);
  const int64_t step = int64_t(p.M) * p.ldp;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < int64_t(p.M) * quads; i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / quads;
    const int col = int(i - r * quads) * 4;
    const float* src = p.part + r * p.ldp + col;
    f32x4 v = *reinterpret_cast<const f32x4*>(src);
#pragma unroll 4
    for (int k = 1; k < parts; ++k) v += *reinterpret_cast<const f32x4*>(src + k * step);
    T* dst = static_cast<T*>(p.C) + r * p.ldc + col;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (col + q < p.N) {
        if constexpr (sizeof(T) == 4) dst[q] = p.add ? dst[q] + v[q] : v[q];
        else dst[q] = uint16_t(pack_bf16x2(v[q], 0.f));
      }
  }
}

// C = 0: a product over nothing.
template <class T>
__global__ void __launch_bounds__(256) block_zero_kernel(T* C, int64_t ldc, int M, int N) {
  for (int64_t r = blockIdx.x; r < M; r += gridDim.x)
    for (int64_t j = threadIdx.x; j < N; j += 256) C[r * ldc + j] = T(0);
}

// Which kernel a product takes.  Measured on an MI355X (256 CUs, one workgroup of 256 x 128 or 128 x
// 128, or two of 64 x 64, a CU), in us a round of workgroups with `steps` runs:
//   256 x 128             5.5 + 1.75 steps  (4096 x 4096 x 4096 121 in two rounds, 8192 x 2048 x 1536 53)
//   128 x 128             6   + 0.92 steps  (2048 x 2048 x 2048 20.8, 2048 x 2048 x 8192 63 to 73)
//   96 x 128              5.3 + 0.76 steps  (1536 x 2048 x 2048 17.1, 1536 x 2048 x 8192 54.5)
//   64 x 64, two a CU     3.9 + 0.73 steps  (2048 x 1024 x 2048 15.4, 2048 x 1024 x 8192 51)
//   64 x 64, two groups   3.9 + 0.36 steps  (1024 x 1024 x 2048 9.6, 1024 x 1024 x 8192 27.6)
// and with fp32 results, which have other 128 x 128 tiles and none larger,
//   128 x 128             2.5 + 1.28 steps  (2048 x 2048 x 2048 24.9)
//   64 x 64, two a CU     2   + 0.8  steps  (2048 x 1024 x 2048 16.1)
//   64 x 64, two groups   3   + 0.45 steps  (1024 x 1024 x 2048 10)
// The sizes' best is the least of these.  Where a few rows past a multiple of 256 cost a further round, they
// go to a launch of 64 x 64 tiles (8197 x 2048 x 1536: 64.4, in one launch 75.9; 4128 x 4096 x 2048: 79.3, 93.4).
// With too few tiles for the chip the contraction is cut into parts, whose sums take a second launch:
// 4 us and their bytes at 3 TB/s, written and read (256 x 256 x 16384 13.0, whole 50; 512 x 512 x 8192 15.2, whole
// 27.3; 64 x 64 x 16384 10.6, whole 50).
enum MmKind { MM_LARGE, MM_128, MM_96, MM_64, MM_64X2 };
struct MmPlan {
  MmKind kind;
  double us;
  int peel;   // rows at the end that take a launch of their own
  int parts, per;  // of the contraction, and runs in each
};
constexpr double kPartBytes = 64 << 20;  // most of the parts' sums

MmPlan mm_plan(long long M, long long N, int steps, bool f32, bool whole = false) {
  constexpr int kCus = 256;
  const auto tiles = [&](long long m, int bm, int bn) { return ceil_div(m, bm) * ceil_div(N, bn); };
  const auto large = [&](long long m) { return ceil_div(tiles(m, 256, 128), kCus) * (5.5 + 1.75 * steps); };
  MmPlan best{MM_64, 1e30, 0, 1, steps};
  const auto consider = [&](MmKind kind, int bm, int bn, int slots, double fix, double each) {
    const long long t = tiles(M, bm, bn);
    for (int parts = 1; parts <= 64; parts = parts < 4 ? parts + 1 : parts < 16 ? parts + 2 : parts * 2) {
      const int per = int(ceil_div(steps, parts));
      const double bytes = 4. * parts * double(M) * double(N);
      if (parts > 1 && (whole || t * parts > 2 * slots || per < 4 || bytes > kPartBytes)) break;
      const double us = ceil_div(t * parts, slots) * (fix + each * per) + (parts > 1 ? 4 + 2 * bytes / 3e6 : 0);
      if (us < best.us) best = {kind, us, 0, int(ceil_div(steps, per)), per};
    }
  };
  consider(MM_64X2, 64, 64, kCus, f32 ? 3 : 3.9, f32 ? 0.448 : 0.36);
  consider(MM_64, 64, 64, 2 * kCus, f32 ? 2 : 3.9, f32 ? 0.8 : 0.73);
  consider(MM_128, 128, 128, kCus, f32 ? 2.5 : 6, f32 ? 1.28 : 0.92);
  if (f32) return best;
  consider(MM_96, 96, 128, kCus, 5.3, 0.76);
  if (large(M) < best.us) best = {MM_LARGE, large(M), 0, 1, steps};
  const int rest = int(M % 256);
  if (M > 256 && rest > 0 && rest <= 64) {
    const double us = large(M - rest) + mm_plan(rest, N, steps, f32, true).us + 1.5;
    if (us < best.us) best = {MM_LARGE, us, rest, 1, steps};
  }
  return best;
}

size_t part_bytes(long long M, long long N, const MmPlan& plan) {
  return plan.parts > 1 ? size_t(plan.parts) * M * (ceil_div(N, 4) * 4) * sizeof(float) : 0;
}

// Where the plan peels rows, their launch's plan does not use parts.
int launch_mm(const MmArgs& a, const MmPlan& plan, bool b_tile, bool f32, float* part, hipStream_t s) {
  MmArgs p = a;
  p.per = plan.per;
  p.ldp = (int64_t(p.N) + 3) / 4 * 4;
  p.part = plan.parts > 1 ? part : nullptr;
  const auto one = [&]() {
    switch (plan.kind) {
      case MM_64X2: return launch_mm_mid<MidTile<64, 64, 2, 2, 2>>(p, b_tile, f32, s);
      case MM_64: return launch_mm_mid<MidTile<64, 64, 2, 2, 1>>(p, b_tile, f32, s);
      case MM_128:
        if (!f32) return launch_mm_large<LargeTile<4, 2, 2, 2>>(p, b_tile, s);
        return launch_mm_mid<MidTile<128, 128, 2, 4, 1>, false>(p, b_tile, true, s);
      case MM_96: return launch_mm_large<LargeTile<3, 2, 2, 2>>(p, b_tile, s);
      case MM_LARGE: break;
    }
    return launch_mm_large<LargeTile<4, 4, 2, 1>>(p, b_tile, s);
  };
  if (plan.peel > 0) {
    MmArgs rest = p;
    p.M -= plan.peel;
    rest.M = plan.peel;
    rest.A += int64_t(p.M) * p.lda;
    rest.SA += p.M;
    rest.C = static_cast<uint16_t*>(p.C) + int64_t(p.M) * p.ldc;
    if (const int rc = one()) return rc;
    return launch_mm(rest, mm_plan(rest.M, rest.N, rest.ksteps, f32, true), b_tile, f32, nullptr, s);
  }
  const int rc = one();
  if (rc || plan.parts == 1) return rc;
  const long long blocks = ceil_div((long long)p.M * (p.ldp / 4), 256);
  const unsigned grid = unsigned(blocks < 4096 ? blocks : 4096);
  prof_begin("block_join", s);
  if (f32) block_join_kernel<float><<<grid, 256, 0, s>>>(p, plan.parts);
  else block_join_kernel<uint16_t><<<grid, 256, 0, s>>>(p, plan.parts);
  prof_end(s);
  return launched();
}

// Whether the one-launch kernel takes the product: for values, up to the work of quantising A again
// in every workgroup (in runs of 128 values: 64 x 1024 x 1024, 32768 runs, takes 6.1 us against 8.9
// in two launches, 128 x 1024 x 1024, 65536, 8.3 against 8.9, 16 x 4096 x 4096, 131072, 14.6 against
// 12.2); for codes, up to 4096 runs of tiles (128 x 1024 x 1024: 4.6 us against 6.5; 256 x
// 1024 x 1024: 7.9 against 6.6), and with one row of tiles up to 16384 (16 x 4096 x 4096: 7.5 against 10.0),
// as long as a wave has four runs at most (16 x 512 x 8192: 10.9 against 9.1 in parts and a launch's
// host time; 16 x 512 x 16384: 18.3 against 10.9).
bool use_direct(long long M, long long N, long long K, bool values) {
  const long long steps = ceil_div(K, 128), tm = ceil_div(M, 16), tn = ceil_div(N, 16);
  if (!values) return steps <= 4 * kDirectWaves && tm * tn * steps <= (M <= 16 ? 16384 : 4096);
  if (K > kDirectK) return false;
  long long wk = 1;
  while (wk < kDirectWaves && wk < steps) wk *= 2;
  const long long groups = ceil_div(tn, wk > 8 ? 1 : 8 / wk);  // workgroups a row of tiles
  return tm * groups * (M < 16 ? M : 16) * steps <= 65536;
}

// ---------------------------------------------------------------------------
// Argument checks.

int check_quant_desc(const moe_block_quant_desc* q) {
  if (q == nullptr || q->rows < 0 || q->cols < 0) return MOE_EINVAL;
  if (q->in_type != MOE_TYPE_F32 && q->in_type != MOE_TYPE_BF16) return MOE_EINVAL;
  if (q->scale != MOE_SCALE_TILE && q->scale != MOE_SCALE_BLOCK) return MOE_EINVAL;
  return MOE_OK;
}

bool quantised_by_call(const moe_block_mm_desc& m) { return m.a_type != MOE_TYPE_E4M3; }
int64_t code_ld(int64_t cols) { return (cols + 15) / 16 * 16; }

int check_mm_desc(const moe_block_mm_desc* m) {
  if (m == nullptr || m->M < 0 || m->N < 0 || m->K < 0) return MOE_EINVAL;
  if (m->a_type != MOE_TYPE_F32 && m->a_type != MOE_TYPE_BF16 && m->a_type != MOE_TYPE_E4M3)
    return MOE_EINVAL;
  if (m->b_scale != MOE_SCALE_TILE && m->b_scale != MOE_SCALE_BLOCK) return MOE_EINVAL;
  if (m->c_type != MOE_TYPE_F32 && m->c_type != MOE_TYPE_BF16) return MOE_EINVAL;
  if ((m->flags & ~MOE_MM_ACCUMULATE) != 0) return MOE_EINVAL;
  if ((m->flags & MOE_MM_ACCUMULATE) && m->c_type != MOE_TYPE_F32) return MOE_EINVAL;
  if (m->lda < m->K || m->ldb < m->K || m->ldc < m->N) return MOE_EINVAL;
  if (m->lda >= kMaxStride || m->ldb >= kMaxStride) return MOE_EUNSUPPORTED;
  // scale entries are counted in 31 bits, offsets into C's rows in 63
  const long long steps = ceil_div(m->K, 128), wide = m->M > m->N ? m->M : m->N;
  if (steps * wide * 4 >= (1LL << 31) || m->ldc >= (1LL << 40)) return MOE_EUNSUPPORTED;
  if (quantised_by_call(*m) && !launchable(ceil_div(m->M, 16) * steps, 256)) return MOE_EUNSUPPORTED;
  if (!launchable(ceil_div(m->M, 64) * ceil_div(m->N, 64), 512)) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

MmPlan plan_of(const moe_block_mm_desc& m) {
  return mm_plan(m.M, m.N, int(ceil_div(m.K, 128)), m.c_type == MOE_TYPE_F32);
}

size_t mm_quant_bytes(const moe_block_mm_desc& m, size_t* scales) {
  if (!quantised_by_call(m)) return *scales = 0;
  const size_t codes = align256(size_t(m.M) * code_ld(m.K));
  *scales = codes;
  return codes + align256(size_t(ceil_div(m.K, 128)) * m.M * 4);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_block_quant(const moe_block_quant_desc* q, const void* x, uint8_t* codes, float* scales,
                    uint8_t* codes_t, float* scales_t, void* stream) {
  const int rc = check_quant_desc(q);
  if (rc) return rc;
  if ((codes != nullptr) != (scales != nullptr) || (codes_t != nullptr) != (scales_t != nullptr))
    return MOE_EINVAL;
  if (q->rows == 0 || q->cols == 0) return MOE_OK;
  if (x == nullptr || (codes == nullptr && codes_t == nullptr)) return MOE_EINVAL;
  if (q->ld_in < q->cols || (codes && q->ld_codes < q->cols) || (codes_t && q->ld_codes_t < q->rows))
    return MOE_EINVAL;
  if (!aligned_to(x, type_bytes(q->in_type)) || !aligned_to(codes, 16) || !aligned_to(codes_t, 16) ||
      !aligned_to(scales, 4) || !aligned_to(scales_t, 4) || (codes && q->ld_codes % 16 != 0) ||
      (codes_t && q->ld_codes_t % 16 != 0))
    return MOE_EALIGN;
  if (q->ld_in >= (1LL << 40) || (codes && q->ld_codes >= kMaxStride) ||
      (codes_t && q->ld_codes_t >= kMaxStride) ||
      !launchable(ceil_div(q->rows, 16) * ceil_div(q->cols, 128), 256))
    return MOE_EUNSUPPORTED;
  QuantArgs a = quant_args(x, q->rows, q->cols, q->ld_in);
  a.q = codes;
  a.ldq = q->ld_codes;
  a.sc = scales;
  a.qt = codes_t;
  a.ldt = q->ld_codes_t;
  a.sct = scales_t;
  return launch_block_quant(a, q->in_type, q->scale == MOE_SCALE_BLOCK, static_cast<hipStream_t>(stream));
}

size_t moe_block_mm_scratch_bytes(const moe_block_mm_desc* m) {
  if (check_mm_desc(m) != MOE_OK) return 0;
  size_t at;
  const size_t codes = mm_quant_bytes(*m, &at);
  if (m->M == 0 || m->N == 0 || m->K == 0 || use_direct(m->M, m->N, m->K, quantised_by_call(*m))) return codes;
  return codes + part_bytes(m->M, m->N, plan_of(*m));
}

int moe_block_mm(const moe_block_mm_desc* m, const void* a, const float* a_scales,
                 const uint8_t* b, const float* b_scales, void* c, void* scratch,
                 size_t scratch_bytes, void* stream) {
  int rc = check_mm_desc(m);
  if (rc) return rc;
  if (m->M == 0 || m->N == 0) return MOE_OK;
  const bool quant = quantised_by_call(*m);
  if (c == nullptr || (quant && a_scales != nullptr)) return MOE_EINVAL;
  if (m->K > 0 && (a == nullptr || b == nullptr || b_scales == nullptr || (!quant && a_scales == nullptr)))
    return MOE_EINVAL;
  if (!aligned_to(a, quant ? type_bytes(m->a_type) : 16) || (!quant && m->lda % 16 != 0) ||
      !aligned_to(b, 16) || m->ldb % 16 != 0 || !aligned_to(a_scales, 4) || !aligned_to(b_scales, 4) ||
      !aligned_to(c, type_bytes(m->c_type)) || !aligned_to(scratch, 16))
    return MOE_EALIGN;
  const size_t need = moe_block_mm_scratch_bytes(m);
  if (need > 0 && scratch == nullptr) return MOE_EINVAL;
  if (scratch_bytes < need) return MOE_ESCRATCH;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool f32 = m->c_type == MOE_TYPE_F32;
  if (m->K == 0) {
    if (m->flags & MOE_MM_ACCUMULATE) return MOE_OK;
    prof_begin("block_zero", s);
    const unsigned grid = unsigned(m->M < 65536 ? m->M : 65536);
    if (f32) block_zero_kernel<<<grid, 256, 0, s>>>(static_cast<float*>(c), m->ldc, m->M, m->N);
    else block_zero_kernel<<<grid, 256, 0, s>>>(static_cast<uint16_t*>(c), m->ldc, m->M, m->N);
    prof_end(s);
    return launched();
  }
  MmArgs p{};
  p.M = m->M;
  p.N = m->N;
  p.K = m->K;
  p.ksteps = int(ceil_div(m->K, 128));
  p.A = static_cast<const uint8_t*>(a);
  p.SA = a_scales;
  p.ldsa = m->M;
  p.lda = m->lda;
  p.B = b;
  p.SB = b_scales;
  p.ldb = m->ldb;
  p.C = c;
  p.ldc = m->ldc;
  p.add = (m->flags & MOE_MM_ACCUMULATE) != 0;
  p.ldsb = p.ksteps;
  const bool bt = m->b_scale == MOE_SCALE_TILE;
  if (use_direct(m->M, m->N, m->K, quant)) {
    const DirectArgs dp{p, a, m->lda, 0};
    if (!quant) return launch_direct<A_CODES>(dp, bt, f32, s);
    if (m->a_type == MOE_TYPE_BF16) return launch_direct<A_BF16>(dp, bt, f32, s);
    return launch_direct<A_F32>(dp, bt, f32, s);
  }
  char* sc = static_cast<char*>(scratch);
  size_t at;
  float* part = reinterpret_cast<float*>(sc + mm_quant_bytes(*m, &at));
  if (quant) {
    QuantArgs q = quant_args(a, m->M, m->K, m->lda);
    q.q = reinterpret_cast<uint8_t*>(sc);
    q.ldq = code_ld(m->K);
    q.sc = reinterpret_cast<float*>(sc + at);
    if ((rc = launch_block_quant(q, m->a_type, false, s))) return rc;
    p.A = q.q;
    p.lda = q.ldq;
    p.SA = q.sc;
  }
  return launch_mm(p, plan_of(*m), bt, f32, part, s);
}

}  // extern "C"
