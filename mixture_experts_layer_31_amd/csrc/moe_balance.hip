// Load-balancing loss, z-loss and per-expert counts of the router, and their
// gradient into the logits (moe_balance_fwd, moe_balance_bwd in moe.h).
//
// With p = softmax(z), f_e = counts_e / (n K) and P_e the mean of p_te over the n
// kept tokens, loss0 = E sum_e f_e P_e has d loss0 / d z_tj =
// (E / n) p_tj (f_j - sum_e f_e p_te), and loss1 = mean lse_t^2 has
// d loss1 / d z_tj = (2 / n) lse_t p_tj.
//
// Both passes read each logit once into registers.  LPT lanes share a token (16 up
// to 256 experts, so a wave holds four tokens and a row reduction is four DPP
// moves; 64 above, where 16 would hold 32 logits a lane), each with VPL logits of it in
// runs of four: 65536 tokens, forward + backward in us (with fp32 sums, one to two less),
// 16 lanes against 64: 64 experts 21.8, 47; 128 experts 29.9, 50; 256 experts 47.4, 52; 512
// experts 112, 82.  The forward
// adds p to per-lane sums over the block's tokens, joined at the end over the
// wave's tokens and the block's waves in a fixed order, and counts the block's ids
// with LDS atomics (integers: their order does not show).  Up to kBalOneBlock tokens
// one block does it all; past that a second launch adds the blocks' partial sums, 64
// experts a block, and its last block the loss.  Every sum over tokens is 64 bits wide: equal
// numbers added in fp32 are rounded the same way each time (2^22 tokens of 3 experts: 11 u off).  A wave's sum
// and a block's are rounded to fp32 where they are handed on, which adds u each.
// Partial sums in global atomics would be one launch fewer and another result with
// each run.  256 tokens of 128 experts take 10.1 us in one launch and 8.4 in two, whose
// second costs the host 4; 128 tokens 7.0 and 8.3.  The limit is on tokens alone and was set there: with
// more experts two launches win earlier (256 tokens of 256 experts 15.1 and 11.7, of 512 29.8 and 14.6, of
// 1024 46.8 and 20.1; 128 tokens of 512 16.6 and 14.6).
//
// Bound by launches up to some 16384 x 128 (10.5 us forward, 6.7 backward).  65536 x 512 (134 MB): forward 36.5,
// 3.7 TB/s read, bound by the loads in flight (a workgroup a CU, a token ahead a wave; 1024 experts,
// with twice the bytes ahead, 56.6 and 4.7); backward 48.5, 5.5 TB/s read and written, by memory.
#include <type_traits>

#include "moe_args.h"
#include "moe_fp8_codec.h"

namespace moe {
namespace {

constexpr int kBalThreads = 1024;  // forward: 16 waves join their sums in LDS
constexpr int kBalBwdThreads = 256;
constexpr int kBalMaxBlocks = 256;     // forward: one a CU
// Backward: the next token's values on their way over several tokens a group (65536 x 128: 15.5 us,
// 21.4 with 4096 blocks and a token or two each).
constexpr int kBalBwdBlocks = 1024;
constexpr int kBalOneBlock = 256;      // tokens
constexpr int kMaxExperts = 1024;

struct BalScratch {
  float* p;      // [blocks][E] sums of p
  int32_t* c;    // [blocks][E] counts
  float* z;      // [blocks] sums of lse^2
  int32_t* n;    // [blocks] kept tokens
  double* dot;   // [E / 64] a finishing block's part of sum f P
  uint32_t* done;  // finishing blocks that are through; cleared by the pass before
  size_t bytes;
};

int bal_blocks(int T) {
  if (T <= kBalOneBlock) return 1;
  const long long b = ceil_div(T, 64);
  return b > kBalMaxBlocks ? kBalMaxBlocks : int(b);
}

BalScratch bal_scratch(const moe_desc& d, char* base) {
  const size_t G = bal_blocks(d.T), E = d.E;
  BalScratch s;
  size_t o = 0;
  auto take = [&](size_t bytes) { char* r = base + o; o = align256(o + bytes); return r; };
  s.p = reinterpret_cast<float*>(take(G * E * 4));
  s.c = reinterpret_cast<int32_t*>(take(G * E * 4));
  s.z = reinterpret_cast<float*>(take(G * 4));
  s.n = reinterpret_cast<int32_t*>(take(G * 4));
  s.dot = reinterpret_cast<double*>(take((E + 63) / 64 * 8));
  s.done = reinterpret_cast<uint32_t*>(take(4));
  s.bytes = o;
  return s;
}

// Sum over aligned groups of LPT lanes, in every lane.
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
  v += __int_as_float(dpp_swap1(__float_as_int(v)));
  v += __int_as_float(dpp_swap2(__float_as_int(v)));
  v += __int_as_float(dpp_mirror8(__float_as_int(v)));
  v += __int_as_float(dpp_mirror16(__float_as_int(v)));
  if constexpr (LPT == 64) {
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
  v = max16(v);
  if constexpr (LPT == 64) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    v = fmaxf(v, __shfl_xor(v, 32, 64));
  }
  return v;
}

// Expert of a lane's i-th value: runs of four, the group's lanes side by side.
template <int LPT>
__device__ __forceinline__ int expert_of(int l, int i) { return 4 * (l + LPT * (i >> 2)) + (i & 3); }

// A token's logits (-inf past E); VEC: E % 4 == 0 and 16-byte rows.
template <int LPT, int VPL, bool VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int l, float (&z)[VPL]) {
#pragma unroll
  for (int q = 0; q < VPL / 4; ++q) {
    const int e = expert_of<LPT>(l, 4 * q);
    if constexpr (VEC) {
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) v = *reinterpret_cast<const float4*>(row + e);
      z[4 * q] = v.x; z[4 * q + 1] = v.y; z[4 * q + 2] = v.z; z[4 * q + 3] = v.w;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) z[4 * q + r] = e + r < E ? row[e + r] : -INFINITY;
    }
  }
}

// Softmax of the row in place; returns its log-sum-exp.
template <int LPT, int VPL>
__device__ __forceinline__ float softmax_row(float (&z)[VPL], int E, int l) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) m = fmaxf(m, z[i]);
  m = group_max<LPT>(m);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    // the padding stays out also where m is not finite
    z[i] = expert_of<LPT>(l, i) < E ? expf(z[i] - m) : 0.f;
    s += z[i];
  }
  s = group_sum<LPT>(s);
  const float r = 1.f / s;
#pragma unroll
  for (int i = 0; i < VPL; ++i) z[i] *= r;
  return m + logf(s);
}

// Sum over the block in a fixed order, valid in thread 0.
__device__ __forceinline__ double block_sum(double v, double (&red)[kBalThreads / 64]) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.;
  if (threadIdx.x == 0)
    for (int w = 0; w < kBalThreads / 64; ++w) s += red[w];
  return s;
}

struct BalOut {
  int32_t* counts;
  float *mean_p, *losses;
};

template <int LPT, int VPL, bool VEC>
__global__ void __launch_bounds__(kBalThreads) balance_fwd_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const uint8_t* __restrict__ valid, int T, int E, int K, BalScratch out, BalOut res) {
  constexpr int GROUPS = kBalThreads / LPT, WAVES = kBalThreads / 64, COLS = LPT * VPL;
  __shared__ int32_t hist[COLS];
  __shared__ float red[WAVES][COLS];
  __shared__ double zred[WAVES];
  __shared__ int32_t nred[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, l = tid & (LPT - 1);
  // token numbers in 64 bits: a step past the last of 2^31 - 1 tokens must not wrap
  const int64_t chunk = (int64_t(T) + gridDim.x - 1) / gridDim.x;
  const int64_t t0 = min(int64_t(T), blockIdx.x * chunk), t1 = min(int64_t(T), t0 + chunk);
  const int pairs = int(t1 - t0) * K;
  float next[VPL];  // the next token's logits: on their way while the ids are counted
  bool keep = false;
  auto fetch = [&](int64_t t) __attribute__((always_inline)) {
    keep = t < t1 && (valid == nullptr || valid[t]);
    if (keep) load_row<LPT, VPL, VEC>(logits + size_t(t) * E, E, l, next);
  };
  fetch(t0 + tid / LPT);
  for (int e = tid; e < COLS; e += kBalThreads) hist[e] = 0;
  __syncthreads();
  // ids, one (token, slot) pair a thread
  for (int64_t i = tid; i < pairs; i += kBalThreads) {
    if (valid == nullptr || valid[t0 + int(i) / K]) {
      const int e = topk_idx[size_t(t0) * K + i];
      if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
    }
  }
  double acc[VPL], zsum = 0.;
  int n = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.;
  for (int64_t t = t0 + tid / LPT; t < t1; t += GROUPS) {
    float p[VPL];
    const bool kept = keep;
#pragma unroll
    for (int i = 0; i < VPL; ++i) p[i] = next[i];
    fetch(t + GROUPS);
    if (!kept) continue;
    const float lse = softmax_row<LPT>(p, E, l);
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] += double(p[i]);
    zsum = __builtin_fma(double(lse), double(lse), zsum);
    n += 1;
  }
  if constexpr (LPT == 16) {  // the wave's four tokens
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      acc[i] += __shfl_xor(acc[i], 16, 64);
      acc[i] += __shfl_xor(acc[i], 32, 64);
    }
    zsum += __shfl_xor(zsum, 16, 64);
    zsum += __shfl_xor(zsum, 32, 64);
    n += __shfl_xor(n, 16, 64);
    n += __shfl_xor(n, 32, 64);
  }
  if (lane < LPT) {
#pragma unroll
    for (int q = 0; q < VPL / 4; ++q)
      *reinterpret_cast<float4*>(&red[wv][expert_of<LPT>(l, 4 * q)]) =
          make_float4(float(acc[4 * q]), float(acc[4 * q + 1]), float(acc[4 * q + 2]), float(acc[4 * q + 3]));
  }
  if (lane == 0) {
    zred[wv] = zsum;
    nred[wv] = n;
  }
  __syncthreads();
  double p = 0., z = 0.;  // thread e: expert e's sum
  int all = 0;
  if (tid < E) {
#pragma unroll
    for (int w = 0; w < WAVES; ++w) p += double(red[w][tid]);
  }
  for (int w = 0; w < WAVES; ++w) {
    z += zred[w];
    all += nred[w];
  }
  if (gridDim.x > 1) {
    if (tid < E) {
      out.p[size_t(blockIdx.x) * E + tid] = float(p);
      out.c[size_t(blockIdx.x) * E + tid] = hist[tid];
    }
    if (tid == 0) {
      out.z[blockIdx.x] = float(z);
      out.n[blockIdx.x] = all;
      if (blockIdx.x == 0) *out.done = 0;
    }
    return;
  }
  double dot = 0.;
  if (tid < E) {
    const double mp = all > 0 ? p / all : 0.;
    res.counts[tid] = hist[tid];
    res.mean_p[tid] = float(mp);
    dot = all > 0 ? mp * (double(hist[tid]) / (double(all) * K)) : 0.;
  }
  __shared__ double dred[WAVES];
  dot = block_sum(dot, dred);
  if (tid == 0) {
    res.counts[E] = all;
    res.losses[0] = float(E * dot);
    res.losses[1] = all > 0 ? float(z / all) : 0.f;
  }
}

// The partial sums of the forward's blocks: COLS experts a block (128 where that makes it one
// block), 1024 / COLS threads an expert.  The last block to be through adds the blocks' parts of
// the loss, in their order.
template <int COLS>
__global__ void __launch_bounds__(kBalThreads) balance_finish_kernel(BalScratch in, int blocks, int E,
                                                                     int K, BalOut res) {
  constexpr int ROWS = kBalThreads / COLS;
  __shared__ double ps[ROWS][COLS], dred[kBalThreads / 64];
  __shared__ int32_t cs[ROWS][COLS], n_all;
  const int tid = threadIdx.x, l = tid % COLS, r = tid / COLS, e = blockIdx.x * COLS + l;
  constexpr int NB = kBalMaxBlocks / 64;
  float zb[NB] = {};
  int nb[NB] = {};
  if (tid < 64) {
#pragma unroll
    for (int q = 0; q < NB; ++q)
      if (l + 64 * q < blocks) {
        zb[q] = in.z[l + 64 * q];
        nb[q] = in.n[l + 64 * q];
      }
  }
  double p = 0.;
  int c = 0;
  if (e < E) {
#pragma unroll 16
    for (int b = r; b < blocks; b += ROWS) {
      p += in.p[size_t(b) * E + e];
      c += in.c[size_t(b) * E + e];
    }
  }
  if (tid < 64) {
    double z = 0.;
    int n = 0;
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      z += zb[q];
      n += nb[q];
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      z += __shfl_xor(z, o, 64);
      n += __shfl_xor(n, o, 64);
    }
    if (l == 0) {
      n_all = n;
      if (blockIdx.x == 0) {
        res.counts[E] = n;
        res.losses[1] = n > 0 ? float(z / n) : 0.f;
      }
    }
  }
  ps[r][l] = p;
  cs[r][l] = c;
  __syncthreads();
  double dot = 0.;
  if (r == 0 && e < E) {
    const int n = n_all;
#pragma unroll
    for (int k = 1; k < ROWS; ++k) {
      p += ps[k][l];
      c += cs[k][l];
    }
    const double mp = n > 0 ? p / n : 0.;
    res.counts[e] = c;
    res.mean_p[e] = float(mp);
    dot = n > 0 ? mp * (double(c) / (double(n) * K)) : 0.;
  }
  dot = block_sum(dot, dred);
  if (tid == 0) {
    bool last = true;
    if (gridDim.x > 1) {
      __hip_atomic_store(&in.dot[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(in.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
      if (last) {
        dot = 0.;
        for (unsigned b = 0; b < gridDim.x; ++b)
          dot += __hip_atomic_load(&in.dot[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (last) res.losses[0] = float(E * dot);
  }
}

template <int LPT, int VPL, bool VEC, bool ROUTER>
__global__ void __launch_bounds__(kBalBwdThreads) balance_bwd_kernel(
    const float* __restrict__ logits, const uint8_t* __restrict__ valid,
    const int32_t* __restrict__ counts, const float* __restrict__ dlosses,
    const int32_t* __restrict__ topk_idx, const float* __restrict__ topk_w,
    const float* __restrict__ dtopk_w, int T, int E, int K, float* __restrict__ dlogits) {
  constexpr int GROUPS = kBalBwdThreads / LPT, COLS = LPT * VPL;
  // a group's row of the router's gradient, zero between tokens
  __shared__ __attribute__((aligned(16))) float s_g[ROUTER ? GROUPS : 1][ROUTER ? COLS : 4];
  const int tid = threadIdx.x, l = tid & (LPT - 1), g = tid / LPT;
  const int64_t step = int64_t(gridDim.x) * GROUPS, first = int64_t(blockIdx.x) * GROUPS + g;
  // a token's logits and slot l of its routing, a token ahead
  struct Token {
    float z[VPL], w = 0.f, dw = 0.f;
    int id = -1;
    bool keep = false;
  } next;
  auto fetch = [&](int64_t t) __attribute__((always_inline)) {
    if (t >= T) return;
    next.keep = valid == nullptr || valid[t];
    if (next.keep) load_row<LPT, VPL, VEC>(logits + size_t(t) * E, E, l, next.z);
    if (ROUTER && l < K) {
      next.id = topk_idx[size_t(t) * K + l];
      next.w = topk_w[size_t(t) * K + l];
      next.dw = dtopk_w[size_t(t) * K + l];
    }
  };
  fetch(first);
  const int n = counts[E];
  const float per = n > 0 ? 1.f / float(n) : 0.f;
  const float a = dlosses[0] * (float(E) * per), b = dlosses[1] * (2.f * per);
  float f[VPL];  // the lane's experts' shares
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = expert_of<LPT>(l, i);
    f[i] = e < E ? float(counts[e]) * (per / float(K)) : 0.f;
  }
  if constexpr (ROUTER) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) s_g[g][expert_of<LPT>(l, i)] = 0.f;
  }
  for (int64_t t = first; t < T; t += step) {
    float p[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) p[i] = next.z[i];
    const float w = next.w, dw = next.dw;
    const int id = next.id;
    const bool keep = next.keep;
    fetch(t + step);
    if (keep) {
      const float lse = softmax_row<LPT>(p, E, l);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) s = __builtin_fmaf(f[i], p[i], s);
      s = group_sum<LPT>(s);
      const float zl = b * lse;
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] *= __builtin_fmaf(a, f[i] - s, zl);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] = 0.f;
    }
    if constexpr (ROUTER) {
      // w_k (dw_k - sum w dw) into the group's row at the selected experts; the group's lanes are in
      // one wave, whose LDS accesses stay in order
      float c = w * dw;
      for (int k = l + LPT; k < K; k += LPT) c += topk_w[size_t(t) * K + k] * dtopk_w[size_t(t) * K + k];
      c = group_sum<LPT>(c);
      auto add = [&](int j, float v) __attribute__((always_inline)) {
        if (j >= 0 && j < E) __hip_atomic_fetch_add(&s_g[g][j], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
      };
      auto order = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      };
      if (l < K) add(id, w * (dw - c));
      for (int k = l + LPT; k < K; k += LPT)
        add(topk_idx[size_t(t) * K + k], topk_w[size_t(t) * K + k] * (dtopk_w[size_t(t) * K + k] - c));
      order();
#pragma unroll
      for (int q = 0; q < VPL / 4; ++q) {
        float4* row = reinterpret_cast<float4*>(&s_g[g][expert_of<LPT>(l, 4 * q)]);
        const float4 v = *row;
        *row = make_float4(0.f, 0.f, 0.f, 0.f);
        p[4 * q] += v.x; p[4 * q + 1] += v.y; p[4 * q + 2] += v.z; p[4 * q + 3] += v.w;
      }
      order();
    }
    float* out = dlogits + size_t(t) * E;
#pragma unroll
    for (int q = 0; q < VPL / 4; ++q) {
      const int e = expert_of<LPT>(l, 4 * q);
      if constexpr (VEC) {
        if (e < E)
          *reinterpret_cast<float4*>(out + e) =
              make_float4(p[4 * q], p[4 * q + 1], p[4 * q + 2], p[4 * q + 3]);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (e + r < E) out[e + r] = p[4 * q + r];
      }
    }
  }
}

template <class F>
int with_shape(int E, bool vec, F&& f) {
  auto go = [&](auto lpt, auto vpl) {
    return vec ? f(lpt, vpl, std::true_type{}) : f(lpt, vpl, std::false_type{});
  };
  using std::integral_constant;
  if (E <= 64) return go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  if (E <= 128) return go(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  if (E <= 256) return go(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  if (E <= 512) return go(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  return go(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

int check_balance_desc(const moe_desc* d) {
  if (d == nullptr) return MOE_EINVAL;
  if (d->T < 0 || d->E <= 0 || d->K <= 0 || d->K > d->E) return MOE_EINVAL;
  if ((long long)d->T * d->K >= (1LL << 31)) return MOE_EINVAL;
  return d->E > kMaxExperts ? MOE_EUNSUPPORTED : MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_balance_scratch_bytes(const moe_desc* d) {
  return check_balance_desc(d) == MOE_OK ? bal_scratch(*d, nullptr).bytes : 0;
}

int moe_balance_fwd(const moe_desc* d, const float* logits, const int32_t* topk_idx,
                    const uint8_t* valid, int32_t* counts, float* mean_p, float* losses,
                    void* scratch, size_t scratch_bytes, void* stream) {
  const int rc = check_balance_desc(d);
  if (rc) return rc;
  if (counts == nullptr || mean_p == nullptr || losses == nullptr || scratch == nullptr ||
      (d->T > 0 && (logits == nullptr || topk_idx == nullptr)))
    return MOE_EINVAL;
  if (!aligned_to(logits, 4) || !aligned_to(topk_idx, 4) || !aligned_to(counts, 4) ||
      !aligned_to(mean_p, 4) || !aligned_to(losses, 4) || !aligned_to(scratch, 16))
    return MOE_EALIGN;
  const BalScratch sc = bal_scratch(*d, static_cast<char*>(scratch));
  if (scratch_bytes < sc.bytes) return MOE_ESCRATCH;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int blocks = bal_blocks(d->T);
  const BalOut out{counts, mean_p, losses};
  const bool vec = d->E % 4 == 0 && aligned_to(logits, 16);
  prof_begin("balance_fwd", s);
  with_shape(d->E, vec, [&](auto lpt, auto vpl, auto v) {
    balance_fwd_kernel<decltype(lpt)::value, decltype(vpl)::value, decltype(v)::value>
        <<<unsigned(blocks), kBalThreads, 0, s>>>(logits, topk_idx, valid, d->T, d->E, d->K, sc, out);
    return 0;
  });
  prof_end(s);
  const int rc1 = launched();
  if (rc1 || blocks == 1) return rc1;
  prof_begin("balance_finish", s);
  if (d->E > 64 && d->E <= 128)
    balance_finish_kernel<128><<<1, kBalThreads, 0, s>>>(sc, blocks, d->E, d->K, out);
  else
    balance_finish_kernel<64><<<unsigned(ceil_div(d->E, 64)), kBalThreads, 0, s>>>(sc, blocks, d->E, d->K, out);
  prof_end(s);
  return launched();
}

int moe_balance_bwd(const moe_desc* d, const float* logits, const uint8_t* valid,
                    const int32_t* counts, const float* dlosses, const int32_t* topk_idx,
                    const float* topk_w, const float* dtopk_w, float* dlogits, void* stream) {
  const int rc = check_balance_desc(d);
  if (rc) return rc;
  const bool router = topk_idx != nullptr;
  if ((topk_w != nullptr) != router || (dtopk_w != nullptr) != router) {
    if (d->T > 0) return MOE_EINVAL;
  }
  if (router && d->K > 64) return MOE_EUNSUPPORTED;
  if (d->T == 0) return MOE_OK;
  if (logits == nullptr || counts == nullptr || dlosses == nullptr || dlogits == nullptr) return MOE_EINVAL;
  if (!aligned_to(logits, 4) || !aligned_to(counts, 4) || !aligned_to(dlosses, 4) ||
      !aligned_to(topk_idx, 4) || !aligned_to(topk_w, 4) || !aligned_to(dtopk_w, 4) ||
      !aligned_to(dlogits, 4))
    return MOE_EALIGN;
  const size_t T = d->T, E = d->E, pairs = T * d->K, out = T * E * 4;
  if (overlap(dlogits, out, logits, out) || overlap(dlogits, out, valid, T) || overlap(dlogits, out, counts, E * 4 + 4) ||
      overlap(dlogits, out, dlosses, 8) || overlap(dlogits, out, topk_idx, pairs * 4) ||
      overlap(dlogits, out, topk_w, pairs * 4) || overlap(dlogits, out, dtopk_w, pairs * 4))
    return MOE_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool vec = d->E % 4 == 0 && aligned_to(logits, 16) && aligned_to(dlogits, 16);
  prof_begin("balance_bwd", s);
  with_shape(d->E, vec, [&](auto lpt, auto vpl, auto v) {
    constexpr int LPT = decltype(lpt)::value, VPL = decltype(vpl)::value;
    constexpr bool VEC = decltype(v)::value;
    const long long want = ceil_div(d->T, kBalBwdThreads / LPT);
    const unsigned grid = unsigned(want < kBalBwdBlocks ? want : kBalBwdBlocks);
    if (router)
      balance_bwd_kernel<LPT, VPL, VEC, true><<<grid, kBalBwdThreads, 0, s>>>(
          logits, valid, counts, dlosses, topk_idx, topk_w, dtopk_w, d->T, d->E, d->K, dlogits);
    else
      balance_bwd_kernel<LPT, VPL, VEC, false><<<grid, kBalBwdThreads, 0, s>>>(
          logits, valid, counts, dlosses, topk_idx, topk_w, dtopk_w, d->T, d->E, d->K, dlogits);
    return 0;
  });
  prof_end(s);
  return launched();
}

}  // extern "C"
