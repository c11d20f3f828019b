// Rows of V fp32 values (logits, probabilities): how they are read, and clusters of
// CTAs that share one (see sample.cu, beam.cu).
//
// Rows are read in aligned groups of four values whatever V is: a row that starts
// `mis` values past a 16-byte boundary has groups [4 g - mis, 4 g - mis + 4), of which
// the first and last may be partial.
#pragma once
#include <cmath>
#include <cooperative_groups.h>
#include "common.cuh"

namespace sub {

namespace cg = cooperative_groups;

constexpr int MAX_CLUSTER = 8;        // the portable size
constexpr int64_t MAX_V = 1 << 20;

struct Row {
  int64_t V;
  int mis, n;               // groups
  int inner, n_inner;       // whole ones: n_inner from `inner` on
  __device__ Row(const float* z, int64_t v)
      : V(v), mis((int)((reinterpret_cast<uintptr_t>(z) >> 2) & 3)) {
    n = (int)((V + mis + 3) / 4);
    inner = mis ? 1 : 0;
    n_inner = max(0, n - ((V + mis) % 4 ? 1 : 0) - inner);
  }
  __device__ int64_t first(int g) const { return (int64_t)g * 4 - mis; }   // may be < 0 in group 0
  __device__ bool whole(int g) const { return (unsigned)(g - inner) < (unsigned)n_inner; }
};

// Group g of row z, through L2 (the kernel just before may have written it); `none`
// where the row has no value.
template <bool VEC = true>
__device__ __forceinline__ float4 load_group(const float* z, const Row& r, int g, float none) {
  if (VEC && r.whole(g)) return __ldcg(reinterpret_cast<const float4*>(z - r.mis) + g);
  const int64_t e = r.first(g);
  float4 x;
  x.x = e >= 0 && e < r.V ? __ldcg(z + e) : none;
  x.y = e + 1 >= 0 && e + 1 < r.V ? __ldcg(z + e + 1) : none;
  x.z = e + 2 >= 0 && e + 2 < r.V ? __ldcg(z + e + 2) : none;
  x.w = e + 3 < r.V ? __ldcg(z + e + 3) : none;
  return x;
}

// The CTAs of a cluster write into each other's shared memory once all of them
// run: each says so at its start, and asks before its first write.
__device__ __forceinline__ void cluster_here() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_all_here() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ float exp2_small(float x) {   // as exp2_fast, down to 2^-149
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A CTA's share of a row's groups.
__device__ __forceinline__ void share(int groups, int rank, int size, int& lo, int& hi) {
  const int per = (groups + size - 1) / size;
  lo = min(groups, rank * per);
  hi = min(groups, lo + per);
}

// exp(d / T) = 2^(d c), c = log2(e) / T in two parts: one rounding of d c.  (Both
// are positive, so that d = -infinity gives 0.)
struct Sharpen {
  float hi, lo;
  __device__ __forceinline__ float expo(float d) const { return exp2_fast(fmaf(d, hi, d * lo)); }
  // exponents of x + minus, two at a time
  __device__ __forceinline__ float4 exponents(const float4& x, float minus) const {
    const float2 hi2 = make_float2(hi, hi), lo2 = make_float2(lo, lo), r2 = make_float2(minus, minus);
    const float2 a = add2(make_float2(x.x, x.y), r2), b = add2(make_float2(x.z, x.w), r2);
    const float2 ea = fma2(a, hi2, mul2(a, lo2)), eb = fma2(b, hi2, mul2(b, lo2));
    return make_float4(ea.x, ea.y, eb.x, eb.y);
  }
  // sums relative to their maxima
  __device__ __forceinline__ void merge(float& m, float& s, float m2, float s2) const {
    const float big = fmaxf(m, m2);
    if (m2 == -INFINITY && s2 == 0.f) return;
    s = (m == -INFINITY && s == 0.f ? 0.f : s * expo(m - big)) + s2 * expo(m2 - big);
    m = big;
  }
};
inline Sharpen make_sharpen(float temperature) {
  const double c = 1.4426950408889634074 / (double)temperature;
  float hi = (float)c;
  if ((double)hi >= c) hi = std::nextafterf(hi, 0.f);
  return {hi, (float)(c - (double)hi)};
}

template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), int64_t rows, int size, int threads,
                            size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * size));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// Whether a and b, of that many values of 4 bytes, have any in common (none at NULL).
inline bool overlap(const void* a, __int128 n_a, const void* b, __int128 n_b) {
  const __int128 x = (__int128)reinterpret_cast<uintptr_t>(a), y = (__int128)reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + 4 * n_b && y < x + 4 * n_a;
}
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

}  // namespace sub
