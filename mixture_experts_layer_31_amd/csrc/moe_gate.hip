// Gate: the router's choice by sigmoid or softmax scores with a bias and groups of
// experts, the gradient of its weights into the logits, and the bias's step
// (moe_gate_fwd, moe_gate_bwd, moe_gate_bias in moe.h).
//
// The choice goes by c = fl32(s + bias) of scores in 64 bits, so that the rounding to fp32 decides which
// of two neighbours comes first and not the error of an fp32 exp.  64-bit scores of every logit cost more than
// the memory does (65536 tokens of 256 experts in groups: 63 us, where the logits take 11), so a wave first chooses by
// fp32 scores in fixed point (31 us) and then looks whether any two choices that matter lie within their error bound of
// each other: the K chosen ones and the next, and the groups at the border.  Only then (a row in a few hundred, rows
// with equal scores, masked groups, scores past the numbers) it chooses again by 64-bit ones.
//
// Forward is bound by the vector ALU: 768 instructions for four tokens of 256 experts in groups, of which the scores are a
// third, the sort and the K + 1 maxima another.  Counted at 65536 tokens (31 us) they take 52000 of the 54000 cycles in which a
// SIMD's waves run, some 25 us; the rest is the launch's start and end (2^20 tokens take 362 us, 22.6 for each 65536).  At
// 16384 x 128 it takes 6.5 us, at one token 2.7 (a launch).  Where every third expert is masked by -inf, in the bias or the
// logits, all rows are chosen again: 79 and 76 us for 65536 x 256.  Backward moves a
// row of zeros for K gathered logits and is bound by memory: 15.4 us for 65536 x 256 fp32 (67 MB written, the gathers touch
// half of the logits' lines), 4.9 for 16384 x 128.
//
// LPT lanes share a token (the rules and both sides measured are at the entry points), each with VPL of its experts in runs of four; with groups, each
// group has LPT / GP of the lanes (GP the power of two from the number of groups).
// * A fixed-point key is c in units of 2^-22 (2^-20 past 256 experts) of the row's largest score or choice, then
//   the expert from the highest down, so that an integer maximum orders keys.  A lane sorts its keys by merging
//   networks (a maximum and a minimum a comparator) and keeps eight; K + 1 times the largest head of a lane is
//   the next expert, and its lane moves on by one.
// * A 64-bit key is fp32's bits of c in their order, then the expert, below a fixed exponent, so that the 64-bit
//   floating maximum (one instruction) orders keys and breaks ties.
#include <algorithm>
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
__device__ __forceinline__ uint32_t cross(uint32_t v) { return uint32_t(cross<STEP>(int(v))); }
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

__device__ __forceinline__ float element(const float* p) { return *p; }
__device__ __forceinline__ float element(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
// Four elements at any element's address, in one access.
typedef float four_f32 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t four_bf16 __attribute__((ext_vector_type(2), aligned(2)));
__device__ __forceinline__ void four(const float* p, float (&f)[4]) {
  const four_f32 a = *reinterpret_cast<const four_f32*>(p);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
}
__device__ __forceinline__ void four(const uint16_t* p, float (&f)[4]) {
  const four_bf16 a = *reinterpret_cast<const four_bf16*>(p);
  f[0] = __uint_as_float(a.x << 16); f[1] = __uint_as_float(a.x & 0xffff0000u);
  f[2] = __uint_as_float(a.y << 16); f[3] = __uint_as_float(a.y & 0xffff0000u);
}
__device__ __forceinline__ void put_four(float* p, const float (&f)[4]) {
  *reinterpret_cast<four_f32*>(p) = four_f32{f[0], f[1], f[2], f[3]};
}
__device__ __forceinline__ void put_four(uint16_t* p, const float (&f)[4]) {
  *reinterpret_cast<four_bf16*>(p) = four_bf16{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
}
__device__ __forceinline__ void put_one(float* p, float f) { *p = f; }
__device__ __forceinline__ void put_one(uint16_t* p, float f) { *p = uint16_t(pack_bf16x2(f, 0.f)); }

// LDS traffic of one wave, in order.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Descending, by Batcher's odd-even merging network.
template <int N>
__device__ __forceinline__ void sort8(uint32_t (&k)[N], int from) {
#pragma unroll
  for (int p = 1; p < 8; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < 8; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i) {
          const int a = i + j, b = i + j + q;
          if (b < 8 && a / (2 * p) == b / (2 * p) && from + b < N) {
            const uint32_t x = k[from + a], y = k[from + b];
            k[from + a] = max(x, y);
            k[from + b] = min(x, y);
          }
        }
}
// The largest eight of a lane's keys, descending in its first eight (all of fewer).
template <int VPL>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[VPL]) {
  constexpr int N = VPL < 8 ? VPL : 8;
#pragma unroll
  for (int f = 0; f < VPL; f += 8) sort8(k, f);
#pragma unroll
  for (int f = 8; f < VPL; f += 8) {
    // the larger of a descending and an ascending row: the eight largest, which rise and then fall
#pragma unroll
    for (int i = 0; i < N; ++i) k[i] = max(k[i], k[f + N - 1 - i]);
#pragma unroll
    for (int q = N / 2; q >= 1; q /= 2)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((i & q) == 0) {
          const uint32_t x = k[i], y = k[i + q];
          k[i] = max(x, y);
          k[i + q] = min(x, y);
        }
  }
}
template <int LPT>
__device__ __forceinline__ uint32_t token_min(uint32_t v) {
  each_step(LPT, [&](auto s) { v = min(v, cross<decltype(s)::value>(v)); });
  return v;
}
// Of the groups of `lanes` lanes in this one's sixteen, those whose v is larger.
template <int N, int STEP>
__device__ __forceinline__ int ahead_from(uint32_t v) {
  const uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x120 + N, 0xF, 0xF, true));  // row_ror:N
  if constexpr (N + STEP < 16) return (o > v ? 1 : 0) + ahead_from<N + STEP, STEP>(v);
  else return o > v ? 1 : 0;
}
__device__ __forceinline__ int groups_ahead(uint32_t v, int lanes) {
  if (lanes == 1) return ahead_from<1, 1>(v);
  if (lanes == 2) return ahead_from<2, 2>(v);
  if (lanes == 4) return ahead_from<4, 4>(v);
  return ahead_from<8, 8>(v);
}

// A token's lanes and the experts of one of them.
template <int LPT>
struct Share {
  int l, g, in;  // lane of the token, its group, its place in the group
  bool mine;
  __device__ __forceinline__ explicit Share(const GateArgs& a)
      : l(threadIdx.x & (LPT - 1)), g(l / a.lanes), in(l & (a.lanes - 1)), mine(g < a.groups) {}
  __device__ __forceinline__ int place(const GateArgs& a, int i) const {  // in its group, of the i-th value
    return 4 * (in + a.lanes * (i >> 2)) + (i & 3);
  }
};
// Its experts' values, -inf where it has fewer than VPL (RAGGED).
template <bool RAGGED, class Z, int LPT, int VPL>
__device__ __forceinline__ void load_logits(const GateArgs& a, const Share<LPT>& s, const Z* row, float (&z)[VPL]) {
  const bool fours = (a.each & 3) == 0;
#pragma unroll
  for (int q = 0; q < VPL / 4; ++q) {
    const int e = s.place(a, 4 * q);
    float f[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if constexpr (!RAGGED) {
      four(row + s.g * a.each + e, f);
    } else if (s.mine) {
      if (fours) {
        if (e < a.each) four(row + s.g * a.each + e, f);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (e + r < a.each) f[r] = element(row + s.g * a.each + e + r);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) z[4 * q + r] = f[r];
  }
}

// Sum by halves: log2 VPL roundings.
template <int N>
__device__ __forceinline__ float half_sum(const float* v) {
  if constexpr (N == 1) return v[0];
  else return half_sum<N / 2>(v) + half_sum<N / 2>(v + N / 2);
}

// What a lane ends up with: the expert `at`, its logit and its slot (K or more: none).
struct Choice {
  int at, slot;
  float x;
};

// The choice by fixed-point keys; false where this wave's tokens have to be chosen by 64-bit keys.  m, inv: the largest
// logit and 1 / sum exp(z - m) for softmax scores (inv only where a weight needs it).  RAGGED: some lane has fewer
// than VPL experts.
//
// Errors, u = 2^-24: of a sigmoid's e^-z 3 u (its exponent is formed in two parts), 1 + e u, the reciprocal 2 u; of a
// softmax's score 2 u + 0.6 u of the row's largest for the exp, 11 u for the sum by halves over VPL values and
// the lanes, 3 u for the reciprocal and the product; 1 u each for the sum with the bias and the product with the unit's
// reciprocal: below 8 u and 20 u of M, the largest score or choice.  A unit of 2^-22 M is 4 u, so that keys
// are off by 2 or 5 units and half a one for their rounding, the fp32 rounding of c a quarter: a difference of 6 or 13
// units is one of c's.  With units of 2^-20 M (16 u) one of 3 or 5 is.  The sums of two of a group twice that and two for an fp32
// rounding.  Of logits in units of 2^-22 of the largest or 1 a difference of 4 (2^-20: 3) is one of 2.5 (1.5) units, more
// than 2^-21 relative in their scores, so that those differ in fp32 as long as they are normal numbers.
template <bool RAGGED, class Z, int LPT, int VPL>
__device__ __forceinline__ bool choose_fixed(const GateArgs& a, const Share<LPT>& sh, const Z* row, Choice& out,
                                             float& m, float& inv) {
  constexpr int PB = LPT == 16 ? 8 : 10, N = VPL < 8 ? VPL : 8;
  // Softmax scores without a bias rise with the logits, one by one or by the best of a group: no score is computed.
  const bool by_logit = a.softmax && a.bias == nullptr && (a.top_groups == a.groups || a.best == 1 || a.each == 1);
  const int gap = by_logit ? (LPT == 16 ? 4 : 3) : LPT == 16 ? (a.softmax ? 13 : 6) : (a.softmax ? 5 : 3);
  constexpr uint32_t PLACES = (1u << PB) - 1;
  constexpr float TOP = LPT == 16 ? 4194304.f : 1048576.f;  // units of M
  constexpr float MAGIC = LPT == 16 ? 12582912.f : 13631488.f;  // 1.5 * 2^23 (+ TOP): an integer's bits are the low ones
  auto is = [&](int i) { return sh.mine && sh.place(a, i) < a.each; };
  // -inf, NaN and +inf, of the bias too, are left to the 64-bit keys
  float z[VPL], c[VPL];
  load_logits<RAGGED>(a, sh, row, z);
#pragma unroll
  for (int i = 0; i < VPL; ++i) c[i] = z[i];
  if constexpr (RAGGED) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = is(i) ? c[i] : 0.f;
  }
  bool hard = !(fabsf(half_sum<VPL>(c)) < INFINITY);
  if (a.softmax) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, z[i]);
    m = fmaxf(token_max<LPT>(m), -FLT_MAX);
    if (!by_logit || !a.renorm) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = __builtin_amdgcn_exp2f((z[i] - m) * 1.44269504f);
      inv = __builtin_amdgcn_rcpf(token_sum<LPT>(half_sum<VPL>(c)));
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] *= inv;
    }
    if (by_logit) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = !RAGGED || is(i) ? z[i] : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float y = __builtin_amdgcn_fmed3f(z[i], -88.f, 88.f);
      const float hi = y * -1.44269504f;
      const float lo = __builtin_fmaf(y, -1.92596299e-8f, __builtin_fmaf(y, -1.44269504f, -hi));
      const float e = __builtin_amdgcn_exp2f(hi);
      c[i] = __builtin_amdgcn_rcpf(1.f + __builtin_fmaf(e, lo * 0.693147181f, e));
    }
  }
  float M = by_logit ? 1.f : 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) M = fmaxf(M, fabsf(c[i]));
  if (a.bias != nullptr) {
    load_logits<RAGGED>(a, sh, a.bias, z);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      c[i] += RAGGED && !is(i) ? 0.f : z[i];
      M = __builtin_elementwise_maximum(M, fabsf(c[i]));  // NaN where one of them is: the bias may hold one
    }
  }
  hard |= !(M < 0x1p100f);  // this lane's: a NaN may not pass the maximum over the token
  M = token_max<LPT>(M);
  hard |= !(M >= 0x1p-60f && M < 0x1p100f);
  const float unit = __builtin_amdgcn_rcpf(M) * (TOP - 2048.f);
  uint32_t key[VPL];
#pragma unroll
  for (int q = 0; q < VPL / 4; ++q) {
    const uint32_t last = PLACES - uint32_t(sh.g * a.each + sh.place(a, 4 * q));
#pragma unroll
    for (int r = 0; r < 4; ++r)
      key[4 * q + r] = (__float_as_uint(__builtin_fmaf(c[4 * q + r], unit, MAGIC)) << PB) + (last - r);
  }
  if constexpr (RAGGED) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = is(i) ? key[i] : 0u;
  }
  sort_keys(key);
  bool full = VPL > 8 && key[N - 1] != 0;  // there may be more than the eight kept
  auto place_of = [&](uint32_t k) { const int e = int(PLACES - (k & PLACES)); return e < a.E ? e : 0; };
  if (a.top_groups < a.groups) {
    uint32_t k0 = key[0], k1 = key[1];
    each_step(a.lanes, [&](auto s) {
      const uint32_t o0 = cross<decltype(s)::value>(k0), o1 = cross<decltype(s)::value>(k1);
      k1 = max(min(k0, o0), max(k1, o1));
      k0 = max(k0, o0);
    });
    // a group's score in units; by its best alone the whole key, whose place orders equal ones
    const bool two = a.best == 2 && a.each > 1;
    const uint32_t score = two ? (k0 >> PB) + (k1 >> PB) : k0;
    int ahead;
    if constexpr (LPT == 16) {
      ahead = groups_ahead(score, a.lanes);
    } else {
      ahead = 0;
      for (int j = 0; j < a.groups; ++j) ahead += uint32_t(__shfl(int(score), j * a.lanes, 64)) > score ? 1 : 0;
    }
    const bool in = ahead < a.top_groups;
    const uint32_t worst = token_min<LPT>(in ? score : 0xffffffffu), next = token_max<LPT>(in ? 0u : score);
    if (two) {
      hard |= worst < next + (2 * gap + 2);  // also where equal ones are all in, which then are too many: worst >= next
      const uint64_t lanes = LPT == 64 ? ~0ull : 0xffffull << (threadIdx.x & 48);
      hard |= __popcll(__ballot(in) & lanes) != a.top_groups * a.lanes;
    } else if (__ballot((worst >> PB) < (next >> PB) + gap) != 0) {
      // equal logits without a bias have equal choices: near the border all have to be
      const int to_border = int(score >> PB) - int(worst >> PB);
      const bool at_border = sh.mine && to_border < gap && to_border > -gap;
      hard |= at_border && !(a.bias == nullptr && element(row + place_of(k0)) == element(row + place_of(worst)));
    }
    if (by_logit) hard |= float((token_max<LPT>(score) >> PB) - (worst >> PB)) > 60.f * unit;  // e^-60: see below
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = in ? key[i] : 0u;
    full &= in;
  }
  uint32_t won = 0, loser = 0;
  auto pop = [&](int k) __attribute__((always_inline)) {
    loser = token_max<LPT>(key[0]);
    if (sh.l == k) won = loser;
    // one bit-field insert a key; a select of two of them becomes a search through the array
    const uint32_t next = key[0] == loser ? ~0u : 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = ((i + 1 < N ? key[i + 1] : 0u) & next) | (key[i] & ~next);
  };
  for (int k = 0; k <= a.K; ++k) pop(k);
  out.at = place_of(won);
  out.x = element(row + out.at);
  out.slot = sh.l;
  // Whether the candidate of a lane below n is near the next one (`loser` behind lane n - 1's); of equal logits without
  // a bias the place decides.
  auto near = [&](int n) {
    uint32_t behind;
    float x_behind;
    if constexpr (LPT == 16) {
      behind = uint32_t(__builtin_amdgcn_update_dpp(0, int(won), 0x101, 0xF, 0xF, true));  // row_shl:1: the next lane's
      x_behind = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(out.x), 0x101, 0xF, 0xF, true));
    } else {
      behind = __shfl_down(won, 1, 64);
      x_behind = __shfl_down(out.x, 1, 64);
    }
    if (sh.l == n - 1) {
      behind = loser;
      if (a.bias == nullptr) x_behind = element(row + place_of(loser));
    }
    return sh.l < n && behind != 0 && (won >> PB) < (behind >> PB) + gap && !(a.bias == nullptr && out.x == x_behind);
  };
  const bool close = near(a.K);
  hard |= full && key[0] == 0;
  hard |= by_logit && sh.l < a.K && m - out.x > 60.f;  // scores that may be below the normal numbers, equal ones then
  if (__ballot(hard) != 0 || (__ballot(close) != 0 && a.softmax)) return false;
  if (__ballot(close) == 0) return true;
  // Sigmoid scores: K and three more candidates, if the next one is clear of them, by 64-bit keys.
  const int n = min(a.K + 3, LPT);
  for (int k = a.K + 1; k <= n; ++k) pop(k);
  out.at = place_of(won);
  out.x = element(row + out.at);
  const bool last = near(n) && sh.l == n - 1;
  if (__ballot(last || (full && key[0] == 0)) != 0) return false;
  double s = sigmoid64(out.x);
  if (a.bias != nullptr) s += double(a.bias[out.at]);
  const double own = sh.l < n && won != 0 ? make_key(float(s), out.at) : 0.;
  out.slot = 0;
  for (int j = 0; j < n; ++j) out.slot += __shfl(own, (int(threadIdx.x) & 63 & ~(LPT - 1)) + j, 64) > own ? 1 : 0;
  if (own == 0.) out.slot = a.K;
  return true;
}

// The choice by 64-bit keys, one maximum over the lane's values a slot.
template <bool RAGGED, class Z, int LPT, int VPL>
__device__ __forceinline__ void choose_exactly(const GateArgs& a, const Share<LPT>& sh, const Z* row, Choice& out, float& m,
                                               float& inv_sum) {
  float z[VPL];
  load_logits<RAGGED>(a, sh, row, z);
  double key[VPL];
  if (a.softmax) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, z[i]);
    m = token_max<LPT>(m);
    double sum = 0.;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      key[i] = z[i] == -INFINITY ? 0. : exp64(double(z[i]) - double(m));
      sum += key[i];
    }
    sum = token_sum<LPT>(sum);
    const double inv = sum == 0. ? 0. : 1. / sum;
    // of weights that are not renormalised choose_fixed's stays: a token's do not depend on its neighbours in the wave.  That
    // sum is fp32, of the hardware's exp: one of 64-bit exps of every logit is what the first choice is there to spare.
    if (a.renorm || !(inv_sum > 0.f && inv_sum < INFINITY)) inv_sum = sum == 0. ? INFINITY : float(inv);
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = sigmoid64(z[i]);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = sh.place(a, i), to = sh.g * a.each + e;
    const bool is = !RAGGED || (sh.mine && e < a.each);
    double s = key[i];
    if (a.bias != nullptr && is) s += double(a.bias[to]);
    const float c = z[i] == -INFINITY ? -FLT_MAX : fmaxf(float(s), -FLT_MAX);
    key[i] = is ? make_key(c, to) : 0.;
  }
  if (a.top_groups < a.groups) {
    double k0 = 0., k1 = 0.;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      k1 = __builtin_fmax(k1, __builtin_fmin(k0, key[i]));
      k0 = __builtin_fmax(k0, key[i]);
    }
    each_step(a.lanes, [&](auto s) {
      const double o0 = cross<decltype(s)::value>(k0), o1 = cross<decltype(s)::value>(k1);
      k1 = __builtin_fmax(__builtin_fmin(k0, o0), __builtin_fmax(k1, o1));
      k0 = __builtin_fmax(k0, o0);
    });
    float score = sh.mine ? key_value(k0) : 0.f;
    if (a.best == 2 && k1 != 0.) score += key_value(k1);
    const double own = sh.mine ? make_key(score, sh.g) : 0.;
    int ahead = 0;
    for (int j = 0; j < a.groups; ++j) {
      const int from = (int(threadIdx.x) & 63 & ~(LPT - 1)) + j * a.lanes;
      ahead += __shfl(own, from, 64) > own ? 1 : 0;
    }
    if (ahead >= a.top_groups) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = 0.;
    }
  }
  double won = 0.;
  for (int k = 0; k < a.K; ++k) {
    double top = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = __builtin_fmax(top, key[i]);
    top = key_max<LPT>(top);
    if (sh.l == k) won = top;
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = key[i] == top ? 0. : key[i];
  }
  out.at = sh.l < a.K ? key_place(won) : 0;
  out.x = element(row + out.at);
  out.slot = sh.l;
}

// The sum of a token's chosen scores s, of logits x (slot: whether this lane has one).  Where it comes to the end of 64-bit
// numbers (a bias can choose experts whose logits lie 700 below the row's largest) the quotients s / sum would be 0 / 0 or
// their sum's reciprocal infinite: there they are those of exp(x - max) over the chosen, whose sum is 1 or more.  So far
// down a sigmoid is exp x; scores of it that are 0 stay 0.
template <int LPT>
__device__ __forceinline__ double slot_sum(bool softmax, bool slot, float x, double& s) {
  double sum = token_sum<LPT>(s);
  if (sum < 1e-280 && (softmax || sum > 0.)) {  // the same in all lanes of a token
    const float m = token_max<LPT>(slot ? x : -INFINITY);
    s = slot && x != -INFINITY ? exp64(double(x) - double(m)) : 0.;
    sum = token_sum<LPT>(s);
  }
  return sum;
}

template <class Z, int LPT, int VPL, bool RAGGED>
__global__ void __launch_bounds__(kGateThreads) gate_fwd_kernel(GateArgs a, int32_t* __restrict__ topk_idx,
                                                                float* __restrict__ topk_w) {
  constexpr int TOKENS = kGateThreads / LPT;
  const Share<LPT> sh(a);
  const int64_t t = int64_t(blockIdx.x) * TOKENS + threadIdx.x / LPT;
  // lanes behind the last token go along with it
  const Z* row = static_cast<const Z*>(a.z) + (t < a.T ? t : a.T - 1) * a.ld;
  Choice ch;
  float m = 0.f, inv = 1.f;
  if (!choose_fixed<RAGGED, Z, LPT, VPL>(a, sh, row, ch, m, inv)) choose_exactly<RAGGED, Z, LPT, VPL>(a, sh, row, ch, m, inv);
  const bool chosen = ch.slot < a.K;
  double s = 0.;
  if (chosen) s = a.softmax ? (ch.x == -INFINITY ? 0. : exp64(double(ch.x) - double(m))) : sigmoid64(ch.x);
  if (a.softmax && (!a.renorm || !(inv < INFINITY))) s *= inv == INFINITY ? 0. : double(inv);  // a row of only -inf, a NaN
  if (a.renorm) {
    const double sum = slot_sum<LPT>(a.softmax, chosen, ch.x, s);
    s = sum == 0. ? 0. : s * inverse64(sum);
  }
  if (chosen && t < a.T) {
    topk_idx[t * a.K + ch.slot] = ch.at;
    topk_w[t * a.K + ch.slot] = float(s * double(a.scale));
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
      s = id >= 0 && x != -INFINITY ? exp64(double(x) - double(m)) : 0.;
    } else if (id >= 0) {
      s = sigmoid64(x);
    }
    const double rest = a.softmax ? 1. : sigmoid64(-x);  // 1 - s
    if (a.renorm) {
      const double sum = slot_sum<LPT>(a.softmax, id >= 0, x, s);
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
  if (d->E > kGateMaxExperts || !launchable(ceil_div(d->T, kGateThreads / 64), kGateThreads) ||  // 64 lanes a token
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
  const size_t in = span(d->T, d->E, d->ld_logits, type_bytes(d->in_type)), out = size_t(d->T) * d->K * 4,
               row = size_t(d->E) * 4;
  if (overlap(topk_idx, out, topk_w, out) || overlap(topk_idx, out, logits, in) || overlap(topk_w, out, logits, in) ||
      overlap(topk_idx, out, bias, row) || overlap(topk_w, out, bias, row))
    return MOE_EINVAL;
  GateArgs a = gate_args(*d, logits, bias);
  int gp = 1;
  while (gp < a.groups) gp *= 2;
  // 16 lanes a token (four tokens a wave) where they hold its experts, groups and slots: a sum or maximum over a token is
  // four lane moves of the vector ALU for four tokens at once, with 64 six for one, two of them through LDS (forward and
  // backward of 16384 x 128: 13 us, with 64 lanes 19; 65536 x 256 in groups 49, with 64 71)
  const bool few = gp <= 16 && a.K <= 16 && values_a_lane(a.each, 16 / gp) <= 16;
  const int lpt = few ? 16 : 64;
  a.lanes = lpt / gp;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const unsigned grid = unsigned(ceil_div(a.T, kGateThreads / lpt));
  prof_begin("gate_fwd", s);
  with_lanes(lpt, values_a_lane(a.each, a.lanes), [&](auto l, auto v) {
    constexpr int LPT = decltype(l)::value, VPL = decltype(v)::value;
    auto go = [&](auto z, auto ragged) {
      gate_fwd_kernel<decltype(z), LPT, VPL, decltype(ragged)::value><<<grid, kGateThreads, 0, s>>>(a, topk_idx, topk_w);
      return 0;
    };
    if (a.each == a.lanes * VPL && gp == a.groups)
      return d->in_type == MOE_TYPE_F32 ? go(float(), std::false_type{}) : go(uint16_t(), std::false_type{});
    return d->in_type == MOE_TYPE_F32 ? go(float(), std::true_type{}) : go(uint16_t(), std::true_type{});
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
  // as forward (with 64 lanes 16384 x 128 16 us for 13, 65536 x 256 58 for 49, forward included)
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
