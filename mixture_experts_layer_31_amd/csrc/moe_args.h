// Argument checks and small device helpers shared by the operators around the
// layer (moe_balance.hip, moe_gate.hip, moe_block.hip, moe_norm.hip, moe_clip.hip,
// moe_adamw.hip).
#pragma once

#include "moe_common.h"

namespace moe {

inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP; }
inline size_t type_bytes(int32_t t) { return t == MOE_TYPE_F32 ? 4 : t == MOE_TYPE_BF16 ? 2 : 1; }
// HIP counts a launch's threads in 32 bits.
inline bool launchable(long long blocks, int threads) { return blocks * threads < (1LL << 32); }
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && x < y + nb && y < x + na;
}
inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Sixteen bytes at any element's address: gfx950 takes global accesses that are not
// aligned to their width, so rows of odd strides need no path of their own.
struct __attribute__((packed, aligned(2))) Bytes16 { uint32_t w[4]; };
__device__ __forceinline__ uint4 load16(const void* p) {
  const Bytes16 v = *static_cast<const Bytes16*>(p);
  return make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}
// Sixteen bytes of a row from element c, zeros where the row (`cols` elements, at least 16
// bytes of them) does not exist, in two halves so that many loads are in flight: `load`
// issues one without a branch (at the row's end from where 16 bytes still fit; with
// nothing to load from `safe`, any readable 16 bytes), and `mend`, once all are issued,
// clears what does not exist and shifts what came from an earlier element.
template <class T>
struct RowPiece {
  static constexpr int N = 16 / sizeof(T);
  uint4 v;
  int past;   // elements that the load starts early
  bool there;
  __device__ __forceinline__ void load(const T* row, int c, int cols, bool ok, const T* safe) {
    there = ok && c < cols;
    past = max(0, c - (cols - N));
    v = load16(there ? row + (c - past) : safe);
  }
  // edge: whether some lane's piece passes its row's end
  __device__ __forceinline__ void mend(bool edge) {
    uint32_t a = there ? v.x : 0, b = there ? v.y : 0, c = there ? v.z : 0, d = there ? v.w : 0;
    if (edge) {  // words by two, by one, then half a word
      const int words = past * int(sizeof(T)) / 4;
      const bool two = (words & 2) != 0, one = (words & 1) != 0;
      a = two ? c : a; b = two ? d : b; c = two ? 0 : c; d = two ? 0 : d;
      a = one ? b : a; b = one ? c : b; c = one ? d : c; d = one ? 0 : d;
      if constexpr (sizeof(T) == 2) {
        const int bits = (past & 1) * 16;
        a = __builtin_amdgcn_alignbit(b, a, bits); b = __builtin_amdgcn_alignbit(c, b, bits);
        c = __builtin_amdgcn_alignbit(d, c, bits); d = __builtin_amdgcn_alignbit(0u, d, bits);
      }
    }
    v = make_uint4(a, b, c, d);
  }
  // rows of less than 16 bytes, element by element
  __device__ __forceinline__ void load_short(const T* row, int c, int cols, bool ok) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (ok && c + i < cols) {
        if constexpr (sizeof(T) == 2) w[i / 2] |= uint32_t(row[c + i]) << (16 * (i & 1));
        else w[i] = __float_as_uint(row[c + i]);
      }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
__device__ __forceinline__ void store16(void* p, const uint4& a) {
  *static_cast<Bytes16*>(p) = Bytes16{{a.x, a.y, a.z, a.w}};
}
// Sixteen and eight bytes at any element's address; STREAM: nontemporal, for data touched once
// per pass that no cache holds until its next use.
typedef uint32_t any_u32x4 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t any_u32x2 __attribute__((ext_vector_type(2), aligned(2)));
template <bool STREAM>
__device__ __forceinline__ uint4 fetch16(const void* p) {
  any_u32x4 v;
  if constexpr (STREAM) v = __builtin_nontemporal_load(static_cast<const any_u32x4*>(p));
  else v = *static_cast<const any_u32x4*>(p);
  return make_uint4(v.x, v.y, v.z, v.w);
}
template <bool STREAM>
__device__ __forceinline__ uint2 fetch8(const void* p) {
  any_u32x2 v;
  if constexpr (STREAM) v = __builtin_nontemporal_load(static_cast<const any_u32x2*>(p));
  else v = *static_cast<const any_u32x2*>(p);
  return make_uint2(v.x, v.y);
}
template <bool STREAM>
__device__ __forceinline__ void keep16(void* p, const uint4& a) {
  const any_u32x4 v = {a.x, a.y, a.z, a.w};
  if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<any_u32x4*>(p));
  else *static_cast<any_u32x4*>(p) = v;
}
template <bool STREAM>
__device__ __forceinline__ void keep8(void* p, const uint2& a) {
  const any_u32x2 v = {a.x, a.y};
  if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<any_u32x2*>(p));
  else *static_cast<any_u32x2*>(p) = v;
}

// A constant of 64 bits in scalar registers where it is used: kept over a loop in vector registers, those of
// exp64 take half of them.
__device__ __forceinline__ double scalar(double c) {
  asm volatile("" : "+s"(c));
  return c;
}
// e^x in 64 bits (2^-45 relative): its Taylor series on half an octave, which ln 2 in two parts leaves.  0 below -745.2, infinite
// above 709.
__device__ __forceinline__ double exp64(double x) {
  const double c = x < -746. ? -746. : x > 746. ? 746. : x;  // a NaN stays
  const double n = __builtin_rint(c * scalar(1.4426950408889634074));
  double r = __builtin_fma(n, scalar(-0.693147180559945286), c);
  r = __builtin_fma(n, scalar(-2.3190468138462996e-17), r);
  double y = scalar(1. / 39916800.);
  y = __builtin_fma(y, r, scalar(1. / 3628800.));
  y = __builtin_fma(y, r, scalar(1. / 362880.));
  y = __builtin_fma(y, r, scalar(1. / 40320.));
  y = __builtin_fma(y, r, scalar(1. / 5040.));
  y = __builtin_fma(y, r, scalar(1. / 720.));
  y = __builtin_fma(y, r, scalar(1. / 120.));
  y = __builtin_fma(y, r, scalar(1. / 24.));
  y = __builtin_fma(y, r, scalar(1. / 6.));
  y = __builtin_fma(y, r, 0.5);
  y = __builtin_fma(y, r, 1.);
  y = __builtin_fma(y, r, 1.);
  return __builtin_ldexp(y, int(n));
}
// 1 / y for y of normal size (2^-50 relative).
__device__ __forceinline__ double inverse64(double y) {
  double r = __builtin_amdgcn_rcp(y);
  r = __builtin_fma(__builtin_fma(-y, r, 1.), r, r);
  return __builtin_fma(__builtin_fma(-y, r, 1.), r, r);
}
__device__ __forceinline__ double sigmoid64(float z) {
  const bool far = z < -600.f;  // there 1 / (1 + e^-z) is e^z, and e^-z may be infinite
  const double e = exp64(far ? double(z) : -double(z));
  return far ? e : inverse64(1. + e);
}

}  // namespace moe
