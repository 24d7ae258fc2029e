// Global L2 norm of a list of gradients and their clipping (moe_grad_norm,
// moe_grad_clip in moe.h).
//
// norm = sqrt(sum x^2) over every tensor, then dst = src * min(1, max / norm).  Both
// are bound by memory: 2 (bf16) or 4 bytes read per element, then as many read
// and written.  Squares are summed in 64 bits: an fp32 square overflows past 1.8e19
// and vanishes below 1e-23, and the vector ALU has the rate to spare (one
// conversion and one 64-bit FMA an element against 16 instruction slots an element
// and lane at the rate of the memory).
//
// The list travels in the kernel arguments (kMaxList entries a launch), so nothing
// is copied to the device and a captured graph holds its own list.  A tensor is
// cut into chunks of kChunkBytes counted from the 16-byte line that holds its first
// element; every chunk is whole 16-byte vectors but for the tensor's first and
// last, whose elements are taken one by one (no load leaves the tensor).  The
// workgroups step through the chunks side by side (each in a run of its own: the norm
// of 1.2 GB took 264 us, so 241), and a workgroup's sum goes to its own slot: the
// result does not depend on the order in which they run.
//
// Launches past kStreamChunks (of up to kMaxList tensors each) go by with nontemporal loads and stores (1.2 GB: norm 241 -> 187
// us, 6.5 TB/s; clip 429 -> 417 us, 5.8 TB/s); below, the clip finds part of the list in the
// memory-side cache (256 MB), which they would cost it (104 MB: 58 us for both calls, 64
// nontemporal).  Loading the end of a long list plainly and clipping from there lost
// more than it won (604 -> 655 us).
#include <algorithm>
#include <cmath>
#include <new>

#include "moe_args.h"

namespace moe {
namespace {

constexpr int kMaxList = 96;          // entries a launch: 96 * 28 bytes of arguments
constexpr int kClipThreads = 256;
constexpr int kChunkBytes = 16384;    // four 16-byte vectors a thread
constexpr int kMaxBlocks = 2048;      // workgroups a launch
// Chunks up to which one workgroup takes the norm in one launch: 4 chunks 4.9 us eager and 3.4 in a graph, 8
// 5.7 and 5.2, 16 9.2 and 8.7, against 9.1 and 4.5 in two launches.
constexpr uint32_t kOneBlock = 8;
constexpr uint32_t kStreamChunks = 144 * 64;  // 144 MB

struct GradList {
  const void* src[kMaxList];
  void* dst[kMaxList];
  int64_t n[kMaxList];
  uint32_t first[kMaxList + 1];  // chunks before each entry
  uint32_t f32[kMaxList / 32];   // bit: the entry is fp32
  int count;
};
static_assert(sizeof(GradList) <= 3584, "kernel arguments hold the list");

// Entry of chunk c: the last i with first[i] <= c (entries have at least a chunk each).
__device__ __forceinline__ int entry_of(const GradList& L, uint32_t c) {
  int lo = 0, hi = L.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (L.first[mid] <= c) lo = mid; else hi = mid;
  }
  return lo;
}

template <class T> struct Vec;  // a 16-byte vector's elements as floats
template <> struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ float round(float x) { return x; }
};
template <> struct Vec<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  static __device__ __forceinline__ float load(const uint16_t* p) {
    return __uint_as_float(uint32_t(*p) << 16);
  }
  static __device__ __forceinline__ uint16_t round(float x) { return uint16_t(pack_bf16x2(x, 0.f)); }
};

// The vectors of chunk c of an entry.  Vector v covers elements [v N - off, +N), off
// the elements between the 16-byte line of the first element and that element.
template <class T>
struct Chunk {
  const T* src;
  int64_t n, v0;  // v0: this thread's first vector
  int off;
  __device__ __forceinline__ Chunk(const void* s, int64_t count, uint32_t c)
      : src(static_cast<const T*>(s)), n(count), v0(int64_t(c) * (kChunkBytes / 16) + threadIdx.x % kClipThreads),
        off(int((reinterpret_cast<uintptr_t>(s) & 15) / sizeof(T))) {}
  __device__ __forceinline__ int64_t elem(int k) const {  // first element of this thread's k-th vector
    return (v0 + k * kClipThreads) * Vec<T>::N - off;
  }
  __device__ __forceinline__ bool whole(int64_t e) const { return e >= 0 && e + Vec<T>::N <= n; }
};
constexpr int kPer = kChunkBytes / 16 / kClipThreads;  // vectors a thread and chunk

template <bool STREAM>
__device__ __forceinline__ uint4 load_vec(const void* p) {
  if constexpr (STREAM) return load16_nt(p);
  else return *static_cast<const uint4*>(p);
}

template <bool STREAM, class T>
__device__ __forceinline__ double chunk_squares(const void* src, int64_t n, uint32_t c) {
  const Chunk<T> ch(src, n, c);
  double s = 0.;
  uint4 raw[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    raw[k] = make_uint4(0, 0, 0, 0);
    const int64_t e = ch.elem(k);
    if (ch.whole(e)) raw[k] = load_vec<STREAM>(ch.src + e);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    float f[Vec<T>::N];
    Vec<T>::get(raw[k], f);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) s = __builtin_fma(double(f[i]), double(f[i]), s);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t e = ch.elem(k);
    if (ch.whole(e) || e >= n || e + Vec<T>::N <= 0) continue;
    for (int i = 0; i < Vec<T>::N; ++i)
      if (e + i >= 0 && e + i < n) {
        const double x = Vec<T>::load(ch.src + e + i);
        s = __builtin_fma(x, x, s);
      }
  }
  return s;
}

template <bool STREAM>
__global__ void __launch_bounds__(kClipThreads) grad_squares_kernel(GradList L,
                                                                    double* __restrict__ out) {
  const uint32_t total = L.first[L.count];
  double s = 0.;
  int i = 0;
  if (blockIdx.x < total) i = entry_of(L, blockIdx.x);
  for (uint32_t c = blockIdx.x; c < total; c += gridDim.x) {
    while (c >= L.first[i + 1]) ++i;
    const uint32_t k = c - L.first[i];
    s += (L.f32[i >> 5] >> (i & 31)) & 1 ? chunk_squares<STREAM, float>(L.src[i], L.n[i], k)
                                         : chunk_squares<STREAM, uint16_t>(L.src[i], L.n[i], k);
  }
  __shared__ double red[kClipThreads / 64];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) out[blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// A short list's norm by one workgroup, four chunks at a time.
__global__ void __launch_bounds__(1024) grad_norm_one_kernel(GradList L, float* __restrict__ norm) {
  const uint32_t total = L.first[L.count];
  const uint32_t c0 = threadIdx.x / kClipThreads;
  double s = 0.;
  int i = 0;
  for (uint32_t c = c0; c < total; c += 1024 / kClipThreads) {
    while (c >= L.first[i + 1]) ++i;
    const uint32_t k = c - L.first[i];
    s += (L.f32[i >> 5] >> (i & 31)) & 1 ? chunk_squares<false, float>(L.src[i], L.n[i], k)
                                         : chunk_squares<false, uint16_t>(L.src[i], L.n[i], k);
  }
  __shared__ double red[16];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.;
    for (int w = 0; w < 16; ++w) t += red[w];
    norm[0] = float(sqrt(t));
  }
}

__global__ void __launch_bounds__(1024) grad_norm_kernel(const double* __restrict__ in, int64_t n,
                                                         float* __restrict__ norm) {
  double s = 0.;
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += in[i];
  __shared__ double red[16];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.;
    for (int w = 0; w < 16; ++w) t += red[w];
    norm[0] = float(sqrt(t));
  }
}

template <bool STREAM, class T>
__device__ __forceinline__ void chunk_scale(const void* src, void* dst, int64_t n, uint32_t c,
                                            float by) {
  const Chunk<T> ch(src, n, c);
  T* out = static_cast<T*>(dst);
  const bool lined = ((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
  uint4 raw[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t e = ch.elem(k);
    if (ch.whole(e)) raw[k] = load_vec<STREAM>(ch.src + e);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t e = ch.elem(k);
    if (ch.whole(e)) {
      float f[Vec<T>::N];
      Vec<T>::get(raw[k], f);
#pragma unroll
      for (int i = 0; i < Vec<T>::N; ++i) f[i] *= by;
      const uint4 v = Vec<T>::put(f);
      if (!lined) store16(out + e, v);
      else if (STREAM) store16_nt(out + e, v);
      else *reinterpret_cast<uint4*>(out + e) = v;
    } else if (e < n && e + Vec<T>::N > 0) {
      for (int i = 0; i < Vec<T>::N; ++i)
        if (e + i >= 0 && e + i < n) out[e + i] = Vec<T>::round(Vec<T>::load(ch.src + e + i) * by);
    }
  }
}

template <bool STREAM>
__global__ void __launch_bounds__(kClipThreads) grad_scale_kernel(GradList L,
                                                                  const float* __restrict__ norm,
                                                                  float max_norm) {
  const float nm = norm[0];
  const float by = nm <= max_norm ? 1.f : max_norm / nm;  // NaN for a NaN norm
  const uint32_t total = L.first[L.count];
  if (blockIdx.x >= total) return;
  int i = entry_of(L, blockIdx.x);
  for (uint32_t c = blockIdx.x; c < total; c += gridDim.x) {
    while (c >= L.first[i + 1]) ++i;
    if (by == 1.f && L.src[i] == L.dst[i]) continue;
    const uint32_t k = c - L.first[i];
    if ((L.f32[i >> 5] >> (i & 31)) & 1) chunk_scale<STREAM, float>(L.src[i], L.dst[i], L.n[i], k, by);
    else chunk_scale<STREAM, uint16_t>(L.src[i], L.dst[i], L.n[i], k, by);
  }
}

int check_list(const moe_grad* g, int32_t count, bool dst) {
  if (count < 0 || (g == nullptr && count > 0)) return MOE_EINVAL;
  int rc = MOE_OK;
  for (int32_t i = 0; i < count; ++i) {
    if (g[i].n < 0 || g[i].reserved != 0 ||
        (g[i].type != MOE_TYPE_F32 && g[i].type != MOE_TYPE_BF16))
      return MOE_EINVAL;
    if (g[i].n == 0) continue;
    if (g[i].n >= (int64_t(1) << 34)) return MOE_EUNSUPPORTED;  // 96 of them stay below 2^31 chunks
    if (g[i].src == nullptr || (dst && g[i].dst == nullptr)) return MOE_EINVAL;
    const size_t es = type_bytes(g[i].type);
    if (!aligned_to(g[i].src, es) || (dst && !aligned_to(g[i].dst, es))) rc = MOE_EALIGN;
  }
  return rc;
}

struct Range {
  uintptr_t a, b;
  int32_t entry;
};

// Whether some dst overlaps another dst, a src other than its own whole one, or the norm.
int check_overlaps(const moe_grad* g, int32_t count, const float* norm) {
  if (count == 0) return MOE_OK;
  Range* r = new (std::nothrow) Range[count];
  if (r == nullptr) return MOE_EHIP;
  int m = 0, rc = MOE_OK;
  for (int32_t i = 0; i < count; ++i)
    if (g[i].n > 0) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(g[i].dst);
      r[m++] = {a, a + uintptr_t(g[i].n) * type_bytes(g[i].type), i};
    }
  std::sort(r, r + m, [](const Range& x, const Range& y) { return x.a < y.a; });
  for (int k = 1; k < m; ++k)
    if (r[k].a < r[k - 1].b) rc = MOE_EINVAL;
  for (int32_t i = 0; rc == MOE_OK && i < count; ++i) {
    if (g[i].n == 0) continue;
    if (overlap(g[i].dst, size_t(g[i].n) * type_bytes(g[i].type), norm, 4)) rc = MOE_EINVAL;
    const uintptr_t a = reinterpret_cast<uintptr_t>(g[i].src);
    const uintptr_t b = a + uintptr_t(g[i].n) * type_bytes(g[i].type);
    // the dsts are disjoint and sorted: the first that ends past a
    const Range* q = std::upper_bound(r, r + m, a, [](uintptr_t v, const Range& x) { return v < x.b; });
    for (; q < r + m && q->a < b; ++q)
      if (q->entry != i || q->a != a) rc = MOE_EINVAL;
  }
  delete[] r;
  return rc;
}

uint64_t chunks_of(const moe_grad& g) {
  if (g.n == 0) return 0;
  const uint64_t head = reinterpret_cast<uintptr_t>(g.src) & 15;
  return (head + uint64_t(g.n) * type_bytes(g.type) + kChunkBytes - 1) / kChunkBytes;
}

// Calls f(list) for the list's non-empty entries, kMaxList of them at a time (check_list
// keeps an entry below 2^34 elements, 2^22 chunks, so that a launch counts them in 32 bits).
template <class F>
int for_lists(const moe_grad* g, int32_t count, F&& f) {
  GradList L;
  L.count = 0;
  L.first[0] = 0;
  for (auto& w : L.f32) w = 0;
  auto flush = [&]() {
    const int rc = L.count ? f(L) : MOE_OK;
    L.count = 0;
    for (auto& w : L.f32) w = 0;
    return rc;
  };
  for (int32_t i = 0; i < count; ++i) {
    const uint64_t c = chunks_of(g[i]);
    if (c == 0) continue;
    if (L.count == kMaxList) {
      if (const int rc = flush()) return rc;
    }
    const int k = L.count;
    L.src[k] = g[i].src;
    L.dst[k] = g[i].dst;
    L.n[k] = g[i].n;
    if (g[i].type == MOE_TYPE_F32) L.f32[k >> 5] |= 1u << (k & 31);
    L.first[k + 1] = L.first[k] + uint32_t(c);
    L.count = k + 1;
  }
  return flush();
}

unsigned grid_of(const GradList& L) {
  return std::min<uint32_t>(L.first[L.count], kMaxBlocks);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

// A slot for each workgroup of the launches that the list takes (at least one launch's).
size_t moe_grad_scratch_bytes(int32_t count) {
  if (count < 0) return 0;
  return size_t(count ? ceil_div(count, kMaxList) : 1) * kMaxBlocks * sizeof(double);
}

int moe_grad_norm(const moe_grad* g, int32_t count, float* norm, void* scratch,
                  size_t scratch_bytes, void* stream) {
  int rc = check_list(g, count, false);
  if (rc && rc != MOE_EALIGN) return rc;
  if (norm == nullptr || scratch == nullptr) return MOE_EINVAL;
  if (rc || !aligned_to(norm, 4) || !aligned_to(scratch, 16)) return MOE_EALIGN;
  if (scratch_bytes < moe_grad_scratch_bytes(count)) return MOE_ESCRATCH;
  hipStream_t s = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(scratch);
  int64_t used = 0;
  bool done = false;  // one workgroup took it all
  rc = for_lists(g, count, [&](const GradList& L) {
    const unsigned grid = grid_of(L);
    if (count <= kMaxList && L.first[L.count] <= kOneBlock) {
      done = true;
      prof_begin("grad_norm", s);
      grad_norm_one_kernel<<<1, 1024, 0, s>>>(L, norm);
      prof_end(s);
      return launched();
    }
    prof_begin("grad_squares", s);
    if (L.first[L.count] > kStreamChunks) grad_squares_kernel<true><<<grid, kClipThreads, 0, s>>>(L, part + used);
    else grad_squares_kernel<false><<<grid, kClipThreads, 0, s>>>(L, part + used);
    prof_end(s);
    used += grid;
    return launched();
  });
  if (rc || done) return rc;
  prof_begin("grad_norm", s);
  grad_norm_kernel<<<1, 1024, 0, s>>>(part, used, norm);
  prof_end(s);
  return launched();
}

int moe_grad_clip(const moe_grad* g, int32_t count, const float* norm, float max_norm,
                  void* stream) {
  int rc = check_list(g, count, true);
  if (rc && rc != MOE_EALIGN) return rc;
  if (norm == nullptr || !(max_norm >= 0.f) || std::isinf(max_norm)) return MOE_EINVAL;
  if (rc || !aligned_to(norm, 4)) return MOE_EALIGN;
  if ((rc = check_overlaps(g, count, norm))) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return for_lists(g, count, [&](const GradList& L) {
    prof_begin("grad_scale", s);
    if (L.first[L.count] > kStreamChunks) grad_scale_kernel<true><<<grid_of(L), kClipThreads, 0, s>>>(L, norm, max_norm);
    else grad_scale_kernel<false><<<grid_of(L), kClipThreads, 0, s>>>(L, norm, max_norm);
    prof_end(s);
    return launched();
  });
}

}  // extern "C"
