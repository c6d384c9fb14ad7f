// The global norm over many tensors, and their scaling by it.
//
//   norm = sqrt(sum of all squares), or the largest magnitude
//   out  = x * min(1, max_norm / (norm + 1e-6))
//
// The coefficient is rounded to fp32, the product to fp32, and from there to a 16-bit type:
// off by 2^-23 beside the type's own half step, for one multiplication a value.
//
// Bound by memory: every value is read for the norm and again for the scaling, and
// written once.  The tensors are cut into chunks of 32 KB; a workgroup takes every
// G-th chunk of a launch.  The launch's tensors (address, length, type) travel in the
// kernel's arguments, up to kSet of them, so that a call needs no table on the device
// and takes other addresses every time.  Sums of squares are held in 64 bits from the
// first square on: no gradient over- or underflows them, and 64-bit multiply-adds
// still take a fraction of the loads' time.  Every workgroup of the scaling adds the
// partial sums up by itself, in one fixed order, instead of a launch between the two.  A
// few small tensors take one workgroup and one launch, cut into chunks of 4 KB a wave.
//
// Three fp32 tensors of 88 million values: 615 us, the norm 214 of them at 4.9 TB/s and the
// scaling 401 at 5.3 (a large copy reaches 5.15).  250 bf16 tensors, 54 MB: 46 us in four
// launches.  Six fp32 tensors, 131 KB: 7.5.  Tried and not faster: 252 tensors a launch, the
// chunks before each counted in the kernel (56 us of 47.8).
#include <algorithm>

#include "common.h"
#include "grad_clip.h"

namespace moe {

namespace {

typedef unsigned int u32x4_g __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_g2 __attribute__((ext_vector_type(4), aligned(2)));

constexpr int kSet = 128;           // tensors of a launch: 3 KB of arguments
constexpr int kChunk = 32768;       // bytes (64 KB: 623 us of 615 for 1.06 GB, 47.8 of 46.2 for 54 MB)
constexpr int kThreads = 256;
constexpr int kGroups = 2048;       // workgroups of all launches together, about
constexpr int kLeastGroups = 256;   // ... but of each launch this many
constexpr int kMostPartials = 4096;  // that a scaling workgroup adds up
constexpr int kSmallChunk = 4096;   // bytes, of one wave
constexpr int kSmallSet = 16;       // tensors: arguments of 0.5 KB instead of 3.6, 1 us of a launch
constexpr int kSmallThreads = 1024;
constexpr int kPerWave = 3;
constexpr int kSmallChunks = kPerWave * kSmallThreads / 64;  // of one workgroup, at most

template <int K>
struct SetOf {
  const void *x[K];
  int64_t n[K];          // values; type in the top bits
  int32_t start[K + 1];  // chunks before each tensor
  int32_t count;
};
template <int K>
struct OutsOf {
  void *out[K];
};
typedef SetOf<kSet> Set;
typedef OutsOf<kSet> Outs;
constexpr int kTypeShift = 60;

// A chunk of the set.
struct Chunk {
  const char *x;
  char *out;
  int type, n;  // n: values
};

// Finds chunks of BYTES at most.  The tensors lie in the lanes, up to two each, loaded together: a
// search in the arguments would wait for them once a step (250 tensors in two launches of
// either kernel: 52.4 us with a search, 47.5 so, both in chunks of 64 KB).
template <int BYTES, bool OUT, int K>
struct Chunks {
  static_assert(K <= 128, "two a lane");
  int count, first[2];
  int64_t n[2], x[2], out[2];
  __device__ __forceinline__ Chunks(const SetOf<K> &s, const OutsOf<K> *o) : count(s.count) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int t = min(64 * i + lane, K - 1);
      first[i] = s.start[t];
      n[i] = s.n[t];
      x[i] = (int64_t)s.x[t];
      out[i] = OUT ? (int64_t)o->out[t] : 0;
    }
  }
  __device__ __forceinline__ static int64_t lane64(const int64_t (&v)[2], int t) {
    const int64_t w = t < 64 ? v[0] : v[1];
    return (uint32_t)__builtin_amdgcn_readlane((int)w, t & 63) |
           (int64_t)__builtin_amdgcn_readlane((int)(w >> 32), t & 63) << 32;
  }
  __device__ __forceinline__ Chunk operator()(int c) const {
    const int lane = threadIdx.x & 63;
    const int t = __popcll(__ballot(lane < count && first[0] <= c)) +
                  __popcll(__ballot(64 + lane < count && first[1] <= c)) - 1;
    const int c0 = __builtin_amdgcn_readlane(t < 64 ? first[0] : first[1], t & 63);
    const int64_t typed = lane64(n, t);
    Chunk k;
    k.type = (int)(typed >> kTypeShift);
    const int size = k.type == MOE_ROW_F32 ? 4 : 2;
    const int64_t at = (int64_t)(c - c0) * (BYTES / size);
    k.n = (int)min((int64_t)(BYTES / size), (typed & ((1ll << kTypeShift) - 1)) - at);
    k.x = (const char *)lane64(x, t) + at * size;
    k.out = OUT ? (char *)lane64(out, t) + at * size : nullptr;
    return k;
  }
};

// 16 bytes as values of a type.
template <int TYPE>
struct Vec {
  static constexpr int N = TYPE == MOE_ROW_F32 ? 4 : 8;
  typedef typename std::conditional<TYPE == MOE_ROW_F32, uint32_t, uint16_t>::type Raw;
  static __device__ __forceinline__ float value(const u32x4_g &v, int i) {
    if constexpr (TYPE == MOE_ROW_F32) return __uint_as_float(v[i]);
    else return one((Raw)(v[i >> 1] >> (16 * (i & 1))));
  }
  static __device__ __forceinline__ float one(Raw r) {
    if constexpr (TYPE == MOE_ROW_F32) return __uint_as_float(r);
    else if constexpr (TYPE == MOE_ROW_F16) return (float)__builtin_bit_cast(_Float16, r);
    else return bf16_to_f32(r);
  }
  static __device__ __forceinline__ Raw raw(float f) {
    if constexpr (TYPE == MOE_ROW_F32) return __float_as_uint(f);
    else if constexpr (TYPE == MOE_ROW_F16) return __builtin_bit_cast(uint16_t, (_Float16)f);
    else return __builtin_bit_cast(uint16_t, (__bf16)f);
  }
  static __device__ __forceinline__ u32x4_g2 scaled(const u32x4_g &v, float coef) {
    u32x4_g2 o;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (N == 4) o[i] = raw(value(v, i) * coef);
      else o[i] = raw(value(v, 2 * i) * coef) | (uint32_t)raw(value(v, 2 * i + 1) * coef) << 16;
    }
    return o;
  }
};

// The running result of one thread: a sum of squares, or the bits of the largest
// magnitude (as integers they order as the magnitudes do, NaN above infinity).
template <bool INF>
struct Norm {
  double sum = 0.0;
  uint32_t top = 0;
  __device__ __forceinline__ void add(float v) {
    if constexpr (INF) top = max(top, __float_as_uint(v) & 0x7FFFFFFFu);
    else sum = fma((double)v, (double)v, sum);
  }
  __device__ __forceinline__ double get() const { return INF ? (double)__uint_as_float(top) : sum; }
};
template <bool INF>
__device__ __forceinline__ double joined(double a, double b) {
  if constexpr (INF) return a > b || a != a ? a : b;  // NaN stays
  else return a + b;
}

// Over a workgroup of NT threads, in a fixed order; in every thread.
template <bool INF, int NT>
__device__ __forceinline__ double block_join(double v) {
  __shared__ double part[NT / 64];
#pragma unroll
  for (int o = 32; o; o >>= 1) v = joined<INF>(v, __shfl_xor(v, o, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < NT / 64; w++) v = joined<INF>(v, part[w]);
  return v;
}

// f(values index, 16 bytes) for the whole vectors of a chunk, U of a thread together.
template <int TYPE, class F>
__device__ __forceinline__ void each_vector(const void *x, int n, F &&f) {
  constexpr int N = Vec<TYPE>::N, U = 4;
  const int whole = n / N;
  const auto *p = (const u32x4_g2 *)x;
  for (int i = threadIdx.x; i < whole; i += U * kThreads) {
    u32x4_g v[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const u32x4_g2 q = p[min(i + u * kThreads, whole - 1)];
      v[u] = (u32x4_g){q[0], q[1], q[2], q[3]};
    }
#pragma unroll
    for (int u = 0; u < U; u++)
      if (i + u * kThreads < whole) f(i + u * kThreads, v[u]);
  }
}

template <int TYPE, bool INF>
__device__ __forceinline__ void norm_values(const void *x, int n, Norm<INF> &acc) {
  typedef Vec<TYPE> V;
  each_vector<TYPE>(x, n, [&](int, const u32x4_g &v) {
#pragma unroll
    for (int i = 0; i < V::N; i++) acc.add(V::value(v, i));
  });
  const int r = n / V::N * V::N + threadIdx.x;
  if (r < n) acc.add(V::one(((const typename V::Raw *)x)[r]));
}

template <bool INF>
__device__ __forceinline__ void norm_chunk(const Chunk &k, Norm<INF> &acc) {
  if (k.type == MOE_ROW_F32) norm_values<MOE_ROW_F32, INF>(k.x, k.n, acc);
  else if (k.type == MOE_ROW_F16) norm_values<MOE_ROW_F16, INF>(k.x, k.n, acc);
  else norm_values<MOE_ROW_BF16, INF>(k.x, k.n, acc);
}

template <bool INF>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(Set s, double *__restrict__ partials) {
  Norm<INF> acc;
  const Chunks<kChunk, false, kSet> chunk(s, nullptr);
  for (int c = blockIdx.x; c < s.start[s.count]; c += gridDim.x) {
    norm_chunk<INF>(chunk(c), acc);
  }
  const double v = block_join<INF, kThreads>(acc.get());
  if (threadIdx.x == 0) partials[blockIdx.x] = v;
}

// The partial sums together.
template <bool INF>
__device__ __forceinline__ double total_of(const double *partials, int n) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) v = joined<INF>(v, partials[i]);
  return block_join<INF, kThreads>(v);
}

template <bool INF>
__global__ __launch_bounds__(kThreads) void grad_total_kernel(const double *__restrict__ partials, int n,
                                                              double *total, float *norm) {
  const double v = total_of<INF>(partials, n);
  if (threadIdx.x) return;
  if (total) *total = v;
  if (norm) *norm = (float)(INF ? v : sqrt(v));
}

template <int TYPE>
__device__ __forceinline__ void scale_values(const void *x, void *out, int n, float coef) {
  typedef Vec<TYPE> V;
  auto *dst = (u32x4_g2 *)out;
  each_vector<TYPE>(x, n, [&](int at, const u32x4_g &v) { dst[at] = V::scaled(v, coef); });
  const int r = n / V::N * V::N + threadIdx.x;
  typedef typename V::Raw Raw;
  if (r < n) ((Raw *)out)[r] = V::raw(V::one(((const Raw *)x)[r]) * coef);
}

__device__ __forceinline__ void scale_chunk(const Chunk &k, float coef) {
  if (k.x == k.out && coef == 1.0f) return;
  if (k.type == MOE_ROW_F32) scale_values<MOE_ROW_F32>(k.x, k.out, k.n, coef);
  else if (k.type == MOE_ROW_F16) scale_values<MOE_ROW_F16>(k.x, k.out, k.n, coef);
  else scale_values<MOE_ROW_BF16>(k.x, k.out, k.n, coef);
}

// The coefficient, and the norm that it comes from.
template <bool INF>
__device__ __forceinline__ float coef_of(double total, float max_norm, double *norm) {
  *norm = INF ? total : sqrt(total);
  double c = (double)max_norm / (*norm + 1e-6);
  if (c > 1.0) c = 1.0;  // NaN stays
  return (float)c;
}

// Chunks from the last to the first: what the norm read last is still in the caches.
template <bool INF>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(Set s, Outs o,
                                                              const double *__restrict__ partials,
                                                              int n, float max_norm, float *norm) {
  const Chunks<kChunk, true, kSet> chunk(s, &o);
  double nm;
  const float coef = coef_of<INF>(total_of<INF>(partials, n), max_norm, &nm);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)nm;
  for (int i = s.start[s.count] - 1 - (int)blockIdx.x; i >= 0; i -= gridDim.x)
    scale_chunk(chunk(i), coef);
}

// All of it in one workgroup: a wave holds kPerWave chunks in registers from the one
// reading of them to the scaling.
template <bool INF>
__global__ __launch_bounds__(kSmallThreads) void grad_small_kernel(SetOf<kSmallSet> s,
                                                                   OutsOf<kSmallSet> o,
                                                                   float max_norm, float *norm) {
  constexpr int kWaves = kSmallThreads / 64, V = kSmallChunk / 1024;  // vectors of a lane and chunk
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const Chunks<kSmallChunk, true, kSmallSet> chunk(s, &o);
  const int total = s.start[s.count];
  Chunk k[kPerWave];
  u32x4_g v[kPerWave][V];
  uint32_t tail[kPerWave];
#pragma unroll
  for (int q = 0; q < kPerWave; q++) {
    k[q] = chunk(min(wave + q * kWaves, total - 1));
    if (wave + q * kWaves >= total) k[q].n = 0;
    const int N = k[q].type == MOE_ROW_F32 ? 4 : 8, whole = k[q].n / N;
#pragma unroll
    for (int i = 0; i < V; i++) {
      v[q][i] = (u32x4_g){0, 0, 0, 0};
      if (64 * i + lane < whole) {
        const u32x4_g2 u = ((const u32x4_g2 *)k[q].x)[64 * i + lane];
        v[q][i] = (u32x4_g){u[0], u[1], u[2], u[3]};
      }
    }
    const int r = whole * N + lane;
    tail[q] = 0;
    if (r < k[q].n)
      tail[q] = k[q].type == MOE_ROW_F32 ? ((const uint32_t *)k[q].x)[r] : ((const uint16_t *)k[q].x)[r];
  }
  // f(Vec of the type) for each chunk; what lies past its end is zero, and adds nothing
  auto each_type = [&](int q, auto &&f) {
    if (k[q].type == MOE_ROW_F32) f(Vec<MOE_ROW_F32>{});
    else if (k[q].type == MOE_ROW_F16) f(Vec<MOE_ROW_F16>{});
    else f(Vec<MOE_ROW_BF16>{});
  };
  Norm<INF> acc;
#pragma unroll
  for (int q = 0; q < kPerWave; q++)
    if (k[q].n)
      each_type(q, [&](auto vec) {
        typedef decltype(vec) T;
#pragma unroll
        for (int i = 0; i < V; i++)
#pragma unroll
          for (int e = 0; e < T::N; e++) acc.add(T::value(v[q][i], e));
        acc.add(T::one((typename T::Raw)tail[q]));
      });
  double nm;
  const float coef = coef_of<INF>(block_join<INF, kSmallThreads>(acc.get()), max_norm, &nm);
  if (norm && threadIdx.x == 0) *norm = (float)nm;
#pragma unroll
  for (int q = 0; q < kPerWave; q++)
    if (k[q].n && !(k[q].x == k[q].out && coef == 1.0f))
      each_type(q, [&](auto vec) {
        typedef decltype(vec) T;
        const int whole = k[q].n / T::N, r = whole * T::N + lane;
#pragma unroll
        for (int i = 0; i < V; i++)
          if (64 * i + lane < whole) ((u32x4_g2 *)k[q].out)[64 * i + lane] = T::scaled(v[q][i], coef);
        if (r < k[q].n)
          ((typename T::Raw *)k[q].out)[r] = T::raw(T::one((typename T::Raw)tail[q]) * coef);
      });
}

int64_t chunks_of(const moe_grad_tensor &t, int bytes) {
  const int64_t per = t.type == MOE_ROW_F32 ? bytes / 4 : bytes / 2;
  return (t.numel + per - 1) / per;
}

// The next launch's tensors, from the first one that is not in one yet; those
// without values are left out.
template <int K>
int fill(SetOf<K> *s, OutsOf<K> *o, int at, int count, const moe_grad_tensor *t, int bytes = kChunk) {
  s->count = 0;
  s->start[0] = 0;
  for (; at < count && s->count < K; at++) {
    if (!t[at].numel) continue;
    const int64_t c = s->start[s->count] + chunks_of(t[at], bytes);
    if (c > 0x7FFFFFFF) break;  // (a launch of its own then: one tensor has fewer)
    s->x[s->count] = t[at].x;
    o->out[s->count] = t[at].out;
    s->n[s->count] = t[at].numel | (int64_t)t[at].type << kTypeShift;
    s->start[++s->count] = (int32_t)c;
  }
  return at;
}

int launches(int count) { return std::max(1, (count + kSet - 1) / kSet); }

int groups_of(const Set &s, int nl) {
  return (int)std::min<int64_t>(s.start[s.count], std::max(kLeastGroups, kGroups / nl));
}

// Partial sums of every launch, one behind the other; returns how many.
template <bool INF>
int norm_launches(int count, const moe_grad_tensor *t, double *partials, hipStream_t s) {
  int n = 0;
  const int nl = launches(count);
  for (int at = 0; at < count;) {
    Set set;
    Outs o;
    at = fill(&set, &o, at, count, t);
    if (!set.count) continue;
    const int g = groups_of(set, nl);
    if (partials)
      hipLaunchKernelGGL(grad_norm_kernel<INF>, dim3(g), dim3(kThreads), 0, s, set, partials + n);
    n += g;
  }
  return n;
}

template <bool INF>
void scale_launches(int count, const moe_grad_tensor *t, const double *partials, int n, float max_norm,
                    float *norm, hipStream_t s) {
  const int nl = launches(count);
  bool any = false;
  for (int at = 0; at < count;) {
    Set set;
    Outs o;
    at = fill(&set, &o, at, count, t);
    if (!set.count) continue;
    hipLaunchKernelGGL(grad_scale_kernel<INF>, dim3(groups_of(set, nl)), dim3(kThreads), 0, s, set, o,
                       partials, n, max_norm, any ? nullptr : norm);
    any = true;
  }
  if (!any && norm)
    hipLaunchKernelGGL(grad_total_kernel<INF>, dim3(1), dim3(kThreads), 0, s, partials, n,
                       (double *)nullptr, norm);
}

template <bool INF>
void clip(int count, const moe_grad_tensor *t, double *partials, float max_norm, float *norm,
          hipStream_t s) {
  // Six tensors of 131 KB together: 10.3 us in two launches, 7.5 here.
  int64_t small = 0;
  for (int i = 0; i < count && small <= kSmallChunks; i++) small += chunks_of(t[i], kSmallChunk);
  if (small && small <= kSmallChunks) {
    SetOf<kSmallSet> set{};
    OutsOf<kSmallSet> o{};
    if (fill(&set, &o, 0, count, t, kSmallChunk) == count) {
      hipLaunchKernelGGL(grad_small_kernel<INF>, dim3(1), dim3(kSmallThreads), 0, s, set, o, max_norm,
                         norm);
      return;
    }
  }
  int n = norm_launches<INF>(count, t, partials, s);
  if (n > kMostPartials) {  // one sum of them, behind them
    hipLaunchKernelGGL(grad_total_kernel<INF>, dim3(1), dim3(kThreads), 0, s, partials, n, partials + n,
                       (float *)nullptr);
    partials += n;
    n = 1;
  }
  scale_launches<INF>(count, t, partials, n, max_norm, norm, s);
}

}  // namespace

size_t grad_partials(int count, const moe_grad_tensor *t) {
  return norm_launches<false>(count, t, nullptr, nullptr) + 1;
}

void launch_grad_norm(int count, const moe_grad_tensor *t, bool inf, double *partials, double *total,
                      float *norm, hipStream_t s) {
  auto go = [&](auto is_inf) {
    constexpr bool INF = decltype(is_inf)::value;
    const int n = norm_launches<INF>(count, t, partials, s);
    hipLaunchKernelGGL(grad_total_kernel<INF>, dim3(1), dim3(kThreads), 0, s, partials, n, total, norm);
  };
  inf ? go(std::true_type{}) : go(std::false_type{});
}

void launch_grad_scale(int count, const moe_grad_tensor *t, bool inf, const double *partials, int n,
                       float max_norm, float *norm, hipStream_t s) {
  inf ? scale_launches<true>(count, t, partials, n, max_norm, norm, s)
      : scale_launches<false>(count, t, partials, n, max_norm, norm, s);
}

void launch_grad_clip(int count, const moe_grad_tensor *t, bool inf, double *partials,
                      float max_norm, float *norm, hipStream_t s) {
  inf ? clip<true>(count, t, partials, max_norm, norm, s)
      : clip<false>(count, t, partials, max_norm, norm, s);
}

}  // namespace moe
