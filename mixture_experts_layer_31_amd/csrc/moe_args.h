// Argument checks and small device helpers shared by the operators around the
// layer (moe_balance.hip, moe_block.hip, moe_clip.hip).
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

}  // namespace moe
