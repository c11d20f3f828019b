// The best continuations of each sequence's beams: a level of a batch's draft trees,
// or a step of a beam search ("SubSpec: Using the Target Model's Own Low-Bit Shadow
// as Its Draft Model", 6.3/6.4).
//
//   score(j, v) = S_j + z_v / T - lse_j,  lse_j = log sum_w exp(z_w / T)
//
// Within a beam the order is that of the logits, so a beam's n_best largest logits are
// all that can be chosen, and only their scores are formed.  Two launches:
//
// scan   one pass over the logits, bound by HBM: per CTA the running maximum and sum
//        of exp, and the largest logit of every block of 128.  512 rows of 128256: 47 us,
//        5.6 TB/s, whatever the loads in flight (2 to 16 per thread) and CTAs per row.
// pick   one cluster per sequence, a CTA per beam (or several): the k largest of the
//        block maxima name k blocks that hold all of the k largest logits (a logit
//        above which there are fewer than k others cannot lie in a block that k others
//        exceed), which are read again, from L2; the beams' lists meet in the
//        cluster's first CTA, where each candidate finds its place by bisection in the
//        others' lists.  Bound by latency: some ten dependent steps, 8 us after the scan
//        of 8 rows.  (16 us before the log of the sum had a warp of its own and the
//        bisections several lanes and whole numbers to compare.)
//
// Rows that a cluster reads in a moment take both in one launch (beam_kernel).
//
// (Every CTA keeping the best of its part while it streams would need no second
// reading, but a sorted list per thread costs the scan its loads in flight.)
//
// Rounding: within a beam the order is that of the logits, exactly.  Between beams it is that of
// scores formed and compared in 64 bits, from sums whose terms and whose parts within a CTA are fp32
// (the CTAs' parts are joined in 64 bits).  A term 2^-e of the largest has an exponent rounded twice,
// 2^-23 e of it, which matters up to e = 20 or so, where 2^20 terms weigh as much as the largest one:
// 2^-19.6 of the sum.  Each exponential adds 2^-22, of a term and of a maximum that has changed, each
// addition 2^-24: below 2^-16 if all point one way, 2^-20 as they come.  Two beams' candidates that
// are closer than that can change places; those of equal rows, too, whose first values lie
// unlike far from a 16-byte boundary, as their terms are added in another order.
#include <algorithm>
#include <atomic>
#include "rows.cuh"

namespace sub {
namespace {

constexpr int SCAN_THREADS = 256, SCAN_WARPS = SCAN_THREADS / 32;
constexpr int SCAN_MLP = 8;            // blocks that a warp has in flight
constexpr int MAX_CHUNKS = 64;         // CTAs per row of the scan
constexpr int PICK_THREADS = 256;
constexpr int BLOCK_GROUPS = 32;       // groups of four: one per lane

struct BeamArgs {
  const float* logits;
  const float* score;
  int64_t V;
  float temp;
  Sharpen sharp;
  int n_beams, n_best, n_chunks, n_blocks;   // n_blocks: stride of a row's block maxima
  const int32_t* state;
  int words, slot;
  int32_t *token, *parent;
  float* score_out;
  int32_t* state_out;
  float2* part;      // [rows][n_chunks] (largest logit, sum of exp relative to it)
  float* top;        // [rows][n_blocks]
};

__device__ __forceinline__ bool alive(float score) { return fabsf(score) < INFINITY; }
// NaN is no logit; -0 and 0 are one value
__device__ __forceinline__ float clean(float z) { return fmaxf(z, -INFINITY) + 0.f; }

// A warp's part of blocks lo .. hi of a row, eight at a time: the largest logit of each to top(block,
// value), and into m, s the largest of all and the sum of exp relative to it.  (A row that is not
// alive is left with its first loads under way.)
template <class F>
__device__ __forceinline__ void scan_blocks(const BeamArgs& a, const float* z, const Row& r, int lo, int hi,
                                            bool live, float& m, float& s, F top) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b0 = lo + warp * SCAN_MLP; b0 < hi; b0 += SCAN_WARPS * SCAN_MLP) {
    float4 x[SCAN_MLP];
#pragma unroll
    for (int k = 0; k < SCAN_MLP; ++k) {
      const int g = (b0 + k) * BLOCK_GROUPS + lane;
      x[k] = b0 + k < hi && g < r.n ? load_group(z, r, g, -INFINITY)
                                    : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
    if (!live) break;   // (the whole CTA)
    float big = m;
    uint32_t mine = 0;
#pragma unroll
    for (int k = 0; k < SCAN_MLP; ++k) {
      x[k] = make_float4(clean(x[k].x), clean(x[k].y), clean(x[k].z), clean(x[k].w));
      const float t = fmaxf(fmaxf(x[k].x, x[k].y), fmaxf(x[k].z, x[k].w));
      big = fmaxf(big, t);
      const uint32_t all = __reduce_max_sync(~0u, float_key(t));
      if (lane == k) mine = all;
    }
    if (lane < SCAN_MLP && b0 + lane < hi) top(b0 + lane, key_float(mine));
    // no logit above -infinity so far: every value is 0 whatever the reference
    const float ref = big == -INFINITY ? 0.f : big;
    s *= a.sharp.expo(m - ref);
    m = big;
#pragma unroll
    for (int k = 0; k < SCAN_MLP; ++k) {
      const float4 e = a.sharp.exponents(x[k], -ref);   // (the sum is at least 1: no term below 2^-126 counts)
      s += (exp2_fast(e.x) + exp2_fast(e.y)) + (exp2_fast(e.z) + exp2_fast(e.w));
    }
  }
  if (!live) return;
#pragma unroll
  for (int o = 16; o; o >>= 1)
    a.sharp.merge(m, s, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, s, o));
}

__global__ void __launch_bounds__(SCAN_THREADS, 4) scan_kernel(const __grid_constant__ BeamArgs a) {
  __shared__ float2 s_warp[SCAN_WARPS];
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const float* const z = a.logits + row * a.V;
  const Row r(z, a.V);
  int lo, hi;
  share((r.n + BLOCK_GROUPS - 1) / BLOCK_GROUPS, blockIdx.y, a.n_chunks, lo, hi);
  const bool live = alive(__ldcg(a.score + row));
  float* const top = a.top + row * a.n_blocks;
  float m = -INFINITY, s = 0.f;
  scan_blocks(a, z, r, lo, hi, live, m, s, [&](int block, float x) { top[block] = x; });
  if (!live) return;
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < SCAN_WARPS; ++w) a.sharp.merge(m, s, s_warp[w].x, s_warp[w].y);
  a.part[row * a.n_chunks + blockIdx.y] = make_float2(m, s);
}

// ------------------------------------------------------------------- pick --
// A selection's threshold comes from the largest keys of 64 parts (n_best up to 16: fewer
// comparisons) or 128; `1 << part_threads` threads form a part.
__host__ __device__ inline int part_threads(int k) { return k <= 16 ? 2 : 1; }
static_assert(SUB_MAX_BEAMS <= PICK_THREADS / 2 && PICK_THREADS == 256, "parts for the largest n_best");

// most keys that select() may have to compare with each other: n keys, the k largest, `per`
// in a thread's hands
__host__ __device__ inline int survivors(int n, int k, int per) {
  const int most = k * (per << part_threads(k));
  return n < most ? n : most;
}
constexpr int PICK_WARPS = PICK_THREADS / 32;
__host__ __device__ inline int per_block_key(int n) { return (n + PICK_THREADS - 1) / PICK_THREADS; }
__host__ __device__ inline int per_logit(int k) { return (k + PICK_WARPS - 1) / PICK_WARPS * 4; }

__device__ __forceinline__ void pick_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool pick_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %1, 0;\n barrier.cta.red.or.pred p, 1, 256, q;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// The k largest of n keys in shared memory (all unlike; 0: none) to out, in falling order,
// zeros behind them; best: the largest of those that the thread wrote there.  The k-th
// largest of the parts' largest keys is a threshold that k keys reach and few others
// pass; those are ranked by counting, eight lanes for each.  By the first PICK_THREADS threads.
__device__ void select(const uint64_t* keys, int n, int k, uint64_t best, uint64_t* out, uint64_t* list,
                       uint64_t* s_top, int* s_count) {
  const int tid = threadIdx.x, lg = part_threads(k), parts = PICK_THREADS >> lg;
  for (int o = 1; o < 1 << lg; o <<= 1)
    best = max(best, (uint64_t)__shfl_xor_sync(~0u, (unsigned long long)best, o));
  if (tid == 0) *s_count = 0;
  if (tid < k) out[tid] = 0;
  const int at = tid & ((1 << lg) - 1), share = parts >> lg;   // of the comparisons
  if (at == 0) s_top[tid >> lg] = best;
  pick_sync();
  int above = 0;   // parts whose largest key is above this one's
#pragma unroll 8
  for (int i = 0; i < share; i += 2) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(s_top + at * share + i);
    above += (x.x > best) + (x.y > best);
  }
  for (int o = 1; o < 1 << lg; o <<= 1) above += __shfl_xor_sync(~0u, above, o);
  // fewer than k parts with a key at all: every key is a candidate
  const bool mine = above == k - 1 && best != 0;
  uint64_t least = 1;
  if (pick_any(mine)) {
    if (mine && at == 0) s_top[0] = best;
    pick_sync();
    least = s_top[0];
  }
  for (int i = tid; i < n; i += PICK_THREADS)
    if (keys[i] >= least) list[atomicAdd(s_count, 1)] = keys[i];
  pick_sync();
  const int found = *s_count;
  for (int i0 = 0; i0 < found; i0 += PICK_THREADS / 8) {
    const int i = i0 + (tid >> 3);
    const uint64_t x = i < found ? list[i] : 0;
    int rank = 0;
    for (int j = tid & 7; j < found; j += 8) rank += list[j] > x;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) rank += __shfl_xor_sync(~0u, rank, o);
    if ((tid & 7) == 0 && i < found && rank < k) out[rank] = x;
  }
  pick_sync();
}

struct PickShared {
  size_t list, cand_key, cand_token, bytes;   // offsets; the keys come first
};
__host__ __device__ inline PickShared pick_shared(int n_blocks, int n_beams, int k) {
  const int n = n_blocks > k * 128 ? n_blocks : k * 128;
  PickShared p;
  p.list = (size_t)n * 8;
  p.cand_key = p.list + (size_t)max(survivors(n_blocks, k, per_block_key(n_blocks)),
                                    survivors(k * 128, k, per_logit(k))) * 8;
  p.cand_token = p.cand_key + (size_t)n_beams * k * 8;
  p.bytes = p.cand_token + (size_t)n_beams * k * 4;
  return p;
}

// Scores in whole numbers that compare as they do (a comparison of doubles takes ten times as
// long), and back.
__device__ __forceinline__ int64_t order_key(double x) {
  const int64_t b = __double_as_longlong(x + 0.);   // (-0 and 0 are one value)
  return b ^ (int64_t)((uint64_t)(b >> 63) >> 1);
}
__device__ __forceinline__ double order_value(int64_t k) {
  return __longlong_as_double(k ^ (int64_t)((uint64_t)(k >> 63) >> 1));
}

struct PickState {   // of a CTA
  __align__(16) uint64_t top[PICK_THREADS / 2];
  uint64_t out[SUB_MAX_BEAMS];
  int found, count[SUB_MAX_BEAMS];   // of the first CTA: candidates of each beam
  int parent[SUB_MAX_BEAMS];
  double lse;
};

// The log of a row's sum, from the parts' maxima and sums that the lanes hold, two each.  By a warp.
__device__ __forceinline__ double log_sum(const BeamArgs& a, const float2 (&p)[2]) {
  const float m = warp_max(fmaxf(p[0].x, p[1].x));
  const bool finite = fabsf(m) < INFINITY;
  const double top = (double)m / (double)a.temp, per = 1. / (double)a.temp;
  double e[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    e[h] = p[h].x == -INFINITY || !finite ? 0. : (double)p[h].y * exp(((double)p[h].x - (double)m) * per);
  double s = e[0] + e[1];
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  return finite ? top + log(s) : (double)INFINITY;   // not finite: no continuations
}

// The k largest logits of a row, in falling order, to st.out, from the keys of its blocks; best: the
// largest that the thread wrote there.  By the first PICK_THREADS threads.
__device__ void best_of_row(const float* z, const Row& r, int blocks, int k, uint64_t best, uint64_t* keys,
                            uint64_t* list, PickState& st) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // ---- the blocks that hold them ----
  select(keys, blocks, k, best, st.out, list, st.top, &st.found);
  // ---- their logits ----
  constexpr int AHEAD = 4;
  best = 0;
  for (int i0 = warp; i0 < k; i0 += PICK_WARPS * AHEAD) {
    float4 x[AHEAD];
    int g[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int i = i0 + u * PICK_WARPS;
      const uint64_t y = i < k ? st.out[i] : 0;
      g[u] = y ? (int)rank_idx(y) * BLOCK_GROUPS + lane : r.n;
      x[u] = g[u] < r.n ? load_group(z, r, g[u], -INFINITY)
                        : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int i = i0 + u * PICK_WARPS;
      if (i >= k) break;
      const float v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {   // (elements before and past the row are -infinity)
        const float c = clean(v[e]);
        const uint64_t y = c == -INFINITY ? 0 : rank_key(c, (uint32_t)(r.first(g[u]) + e));
        keys[i * 128 + e * 32 + lane] = y;
        best = max(best, y);
      }
    }
  }
  pick_sync();   // st.out is read
  select(keys, k * 128, k, best, st.out, list, st.top, &st.found);
}

// A beam's candidates, one per thread (key 0: none), to the cluster's first CTA.  By the whole CTA.
__device__ __forceinline__ void send(const BeamArgs& a, int j, float score, uint64_t key, int64_t* cand_key,
                                     int32_t* cand_token, PickState& st) {
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x;
  if (key && !(st.lse < (double)INFINITY)) key = 0;
  if (key) {
    const double zt = (double)key_float((uint32_t)(key >> 32)) / (double)a.temp;
    *cluster.map_shared_rank(cand_key + j * a.n_best + tid, 0) = order_key(((double)score + zt) - st.lse);
    *cluster.map_shared_rank(cand_token + j * a.n_best + tid, 0) = (int32_t)rank_idx(key);
  }
  const int n_cand = __syncthreads_count(key != 0);   // st.out and st.lse are read
  if (tid == 0) *cluster.map_shared_rank(st.count + j, 0) = n_cand;
}

// The first CTA: every candidate's place among all, by 2^lg lanes for each, and the outputs.
__device__ void place_all(const BeamArgs& a, int64_t b, const int64_t* cand_key, const int32_t* cand_token,
                          PickState& st) {
  const int tid = threadIdx.x, k = a.n_best;
  if (tid < SUB_MAX_BEAMS) st.parent[tid] = -1;
  __syncthreads();
  int lg = 0;
  while (lg < 3 && (a.n_beams * k) << (lg + 1) <= PICK_THREADS) ++lg;
  const int part = tid & ((1 << lg) - 1), total = a.n_beams * k;
  for (int i0 = 0; i0 < total && tid < PICK_THREADS; i0 += PICK_THREADS >> lg) {
    const int i = i0 + (tid >> lg), j = i / k, c = i - j * k;
    const bool there = i < total && c < st.count[min(j, a.n_beams - 1)];
    const int64_t x = there ? cand_key[i] : 0;
    int place = 0;
    if (there)
      for (int o = part; o < a.n_beams && place < k; o += 1 << lg) {
        if (o == j) continue;
        int lo = 0, hi = st.count[o];   // its candidates that come before this one
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          const int64_t y = cand_key[o * k + mid];
          if (y > x || (y == x && o < j)) lo = mid + 1;
          else hi = mid;
        }
        place += lo;
      }
    for (int o = 1; o < 1 << lg; o <<= 1) place += __shfl_xor_sync(~0u, place, o);
    place += c;   // of its own beam's, so many come first
    if (!there || part != 0 || place >= k) continue;
    a.token[b * k + place] = cand_token[i];
    a.parent[b * k + place] = j;
    a.score_out[b * k + place] = (float)order_value(x);
    st.parent[place] = j;
  }
  __syncthreads();
  if (tid < k && st.parent[tid] < 0) {
    a.token[b * k + tid] = -1;
    a.parent[b * k + tid] = -1;
    a.score_out[b * k + tid] = -INFINITY;
  }
  // ---- the parents' states ----
  if (a.state_out)
    for (int64_t i = tid; i < (int64_t)k * a.words; i += PICK_THREADS + 32) {
      const int p = (int)(i / a.words), w = (int)(i - (int64_t)p * a.words), j = st.parent[p];
      int32_t x = j < 0 ? 0 : __ldcg(a.state + (b * a.n_beams + j) * a.words + w);
      if (j >= 0 && a.slot >= 0 && (a.slot + p) >> 5 == w) x |= (int32_t)(1u << ((a.slot + p) & 31));
      a.state_out[b * k * a.words + i] = x;
    }
}

// The first eight warps select; the ninth forms the log of the sum meanwhile, in 64 bits
// (exponentials, a logarithm and a division of doubles: 10000 cycles when it came first).
__global__ void __launch_bounds__(PICK_THREADS + 32) pick_kernel(const __grid_constant__ BeamArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ PickState st;
  cg::cluster_group cluster = cg::this_cluster();
  const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t b = blockIdx.x / size;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.n_best;
  if (size > 1) cluster_here();
  const PickShared at = pick_shared(a.n_blocks, a.n_beams, k);
  uint64_t* const keys = reinterpret_cast<uint64_t*>(smem);
  uint64_t* const list = reinterpret_cast<uint64_t*>(smem + at.list);
  int64_t* const cand_key = reinterpret_cast<int64_t*>(smem + at.cand_key);
  int32_t* const cand_token = reinterpret_cast<int32_t*>(smem + at.cand_token);
  pdl_wait();
  pdl_trigger();
  bool alone = size > 1;   // the others may not run yet (each CTA has a beam at least)
  for (int j = rank; j < a.n_beams; j += size) {
    const int64_t row = b * a.n_beams + j;
    const float* const z = a.logits + row * a.V;
    const Row r(z, a.V);
    const int blocks = (r.n + BLOCK_GROUPS - 1) / BLOCK_GROUPS;
    const float score = __ldcg(a.score + row);
    uint64_t key = 0;    // the thread's candidate
    if (!alive(score)) {
      // no candidates
    } else if (warp == PICK_WARPS) {
      static_assert(MAX_CHUNKS == 64, "two per lane");
      float2 p[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        p[h] = lane + 32 * h < a.n_chunks ? __ldcg(a.part + row * a.n_chunks + lane + 32 * h)
                                          : make_float2(-INFINITY, 0.f);
      const double lse = log_sum(a, p);
      if (lane == 0) st.lse = lse;
    } else {
      uint64_t best = 0;
      for (int i = tid; i < blocks; i += PICK_THREADS) {
        const float x = __ldcg(a.top + row * a.n_blocks + i);
        const uint64_t y = x == -INFINITY ? 0 : rank_key(x, (uint32_t)i);
        keys[i] = y;
        best = max(best, y);
      }
      best_of_row(z, r, blocks, k, best, keys, list, st);
      if (tid < k) key = st.out[tid];
    }
    __syncthreads();   // st.lse is there
    if (alone) cluster_all_here();
    alone = false;
    send(a, j, score, key, cand_key, cand_token, st);
  }
  if (size > 1) cluster.sync();
  else __syncthreads();
  if (rank == 0) place_all(a, b, cand_key, cand_token, st);
}

// Both in one launch, where a cluster has a CTA for each beam, or `team` of them: these share the
// row's scan, and the first of them goes on with what the others left in its shared memory.
__global__ void __launch_bounds__(PICK_THREADS + 32, 3) beam_kernel(const __grid_constant__ BeamArgs a, const int team) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ PickState st;
  __shared__ float2 s_warp[SCAN_WARPS], s_part[2 * MAX_CLUSTER];
  static_assert(SCAN_THREADS == PICK_THREADS && 2 * MAX_CLUSTER <= 32, "the same warps, a part per lane");
  cg::cluster_group cluster = cg::this_cluster();
  const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t b = blockIdx.x / size;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.n_best;
  const int j = rank / team, member = rank - j * team, first = rank - member;   // beam, CTA of its team
  if (size > 1) cluster_here();
  const PickShared at = pick_shared(a.n_blocks, a.n_beams, k);
  uint64_t* const keys = reinterpret_cast<uint64_t*>(smem);
  uint64_t* const list = reinterpret_cast<uint64_t*>(smem + at.list);
  int64_t* const cand_key = reinterpret_cast<int64_t*>(smem + at.cand_key);
  int32_t* const cand_token = reinterpret_cast<int32_t*>(smem + at.cand_token);
  uint64_t* const team_keys = cluster.map_shared_rank(keys, first);
  pdl_wait();
  pdl_trigger();
  const int64_t row = b * a.n_beams + j;
  const float* const z = a.logits + row * a.V;
  const Row r(z, a.V);
  const int blocks = (r.n + BLOCK_GROUPS - 1) / BLOCK_GROUPS;
  const float score = __ldcg(a.score + row);
  const bool live = alive(score);
  if (size > 1) cluster_all_here();   // before the first write to another CTA
  if (warp < PICK_WARPS) {
    int lo, hi;
    share(blocks, member, team, lo, hi);
    float m = -INFINITY, s = 0.f;
    scan_blocks(a, z, r, lo, hi, live, m, s, [&](int block, float x) {
      team_keys[block] = x == -INFINITY ? 0 : rank_key(x, (uint32_t)block);
    });
    if (lane == 0) s_warp[warp] = make_float2(m, s);
    pick_sync();
    if (tid == 0) {
      for (int w = 1; w < SCAN_WARPS; ++w) a.sharp.merge(m, s, s_warp[w].x, s_warp[w].y);
      *cluster.map_shared_rank(s_part + member, first) = make_float2(m, s);
    }
  }
  if (size > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (member != 0) return;   // (nobody reads or writes its shared memory)
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  uint64_t key = 0;   // the thread's candidate
  if (!live) {
    // no candidates
  } else if (warp == PICK_WARPS) {
    const float2 p[2] = {lane < team ? s_part[lane] : make_float2(-INFINITY, 0.f), make_float2(-INFINITY, 0.f)};
    const double lse = log_sum(a, p);
    if (lane == 0) st.lse = lse;
  } else {
    uint64_t best = 0;
    for (int i = tid; i < blocks; i += PICK_THREADS) best = max(best, keys[i]);
    best_of_row(z, r, blocks, k, best, keys, list, st);
    if (tid < k) key = st.out[tid];
  }
  __syncthreads();   // st.lse is there
  send(a, j, score, key, cand_key, cand_token, st);
  if (size > 1) cluster.sync();   // (of the CTAs that are left)
  else __syncthreads();
  if (rank == 0) place_all(a, b, cand_key, cand_token, st);
}

// Blocks of the longest layout of a row, and bytes of a call's workspace.
int block_stride(int64_t V) { return (int)((V + 6 + 127) / 128 + 3) / 4 * 4; }
int64_t beam_bytes(int64_t rows, int64_t V) {
  return cdiv(rows * (MAX_CHUNKS * (int64_t)sizeof(float2) + block_stride(V) * 4), 32) * 32;
}

// Most CTAs of a cluster that the device places: 16, twice the portable size, nearly halve
// what many beams take (31 beams of 128256: 28 us, 40 with 8).
constexpr int PICK_SMEM = 160 * 1024;
int largest_cluster() {
  static std::atomic<int> size[MAX_DEVICES];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MAX_CLUSTER;
  const bool known = dev >= 0 && dev < MAX_DEVICES;
  if (known && (n = size[dev].load(std::memory_order_relaxed)) > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * MAX_CLUSTER);
  cfg.blockDim = dim3(PICK_THREADS + 32);
  cfg.dynamicSmemBytes = PICK_SMEM;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * MAX_CLUSTER;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto allows = [&](auto kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
           cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PICK_SMEM) == cudaSuccess &&
           cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0;
  };
  const bool placed = allows(pick_kernel) && allows(beam_kernel);
  if (!placed) cudaGetLastError();   // (not an error of the call)
  n = placed ? 2 * MAX_CLUSTER : MAX_CLUSTER;
  if (known) size[dev].store(n, std::memory_order_relaxed);
  return n;
}

int32_t check_sizes(int32_t n_seqs, int32_t n_beams, int64_t V) {
  SUB_CHECK_ARG(n_seqs >= 0 && n_seqs <= SUB_MAX_SEQS, "n_seqs must be in [0, SUB_MAX_SEQS]");
  SUB_CHECK_ARG(n_beams >= 1 && n_beams <= SUB_MAX_BEAMS, "n_beams must be in [1, SUB_MAX_BEAMS]");
  SUB_CHECK_ARG(V >= 1 && V <= MAX_V, "V must be in [1, 2^20]");
  return SUB_OK;
}

}  // namespace
}  // namespace sub

using namespace sub;

extern "C" int32_t sub_beam_workspace(int32_t n_seqs, int32_t n_beams, int64_t V, int64_t* bytes) {
  SUB_CHECK_ARG(bytes, "null pointer");
  SUB_TRY(check_sizes(n_seqs, n_beams, V));
  *bytes = beam_bytes((int64_t)n_seqs * n_beams, V);
  return SUB_OK;
}

extern "C" int32_t sub_beam_select(const float* logits, const float* score, int32_t n_seqs, int32_t n_beams,
                                   int64_t V, float temperature, int32_t n_best, const int32_t* state,
                                   int32_t state_words, int32_t slot, int32_t* token, int32_t* parent,
                                   float* score_out, int32_t* state_out, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
  SUB_TRY(check_sizes(n_seqs, n_beams, V));
  SUB_CHECK_ARG(n_best >= 1 && n_best <= SUB_MAX_BEAMS, "n_best must be in [1, SUB_MAX_BEAMS]");
  SUB_CHECK_ARG(temperature >= 1e-6f && temperature <= 1e6f, "temperature must be in [1e-6, 1e6]");
  SUB_CHECK_ARG(!state == !state_out, "state and state_out go together");
  SUB_CHECK_ARG(!state || (state_words >= 1 && state_words <= (1 << 20)), "state_words out of range");
  SUB_CHECK_ARG(slot >= -1 && (slot < 0 || !state || (int64_t)slot + n_best <= 32ll * state_words),
                "the slots do not fit the state's bits");
  if (n_seqs == 0) return SUB_OK;
  SUB_CHECK_ARG(logits && score && token && parent && score_out, "null pointer");
  const int64_t rows = (int64_t)n_seqs * n_beams, picked = (int64_t)n_seqs * n_best;
  struct {
    const void* p;
    int64_t n;
  } const in[3] = {{logits, rows * V}, {score, rows}, {state, state ? rows * state_words : 0}},
          out[4] = {{token, picked}, {parent, picked}, {score_out, picked},
                    {state_out, state ? picked * state_words : 0}};
  for (int i = 0; i < 4; ++i) {
    SUB_CHECK_ARG(aligned4(out[i].p) && (i > 2 || aligned4(in[i].p)), "pointers must be 4-byte aligned");
    for (int j = 0; j < 3; ++j)
      SUB_CHECK_ARG(!overlap(out[i].p, out[i].n, in[j].p, in[j].n), "the outputs must lie apart from the inputs");
    for (int j = 0; j < i; ++j)
      SUB_CHECK_ARG(!overlap(out[i].p, out[i].n, out[j].p, out[j].n), "the outputs must lie apart");
  }
  const cudaStream_t st = as_stream(stream);
  const int64_t need = beam_bytes(rows, V);
  StreamScratch scratch(st);
  if (workspace) {
    SUB_CHECK_ARG((reinterpret_cast<uintptr_t>(workspace) & 31) == 0 && workspace_bytes >= need,
                  "workspace too small or not 32-byte aligned");
  } else {
    SUB_TRY(scratch.alloc((size_t)need));
    workspace = scratch.p;
  }
  BeamArgs a{};
  a.logits = logits;
  a.score = score;
  a.V = V;
  a.temp = temperature;
  a.sharp = make_sharpen(temperature);
  a.n_beams = n_beams;
  a.n_best = n_best;
  a.n_blocks = block_stride(V);
  // Enough CTAs for all SMs, each with a round of its warps' loads at least
  const int64_t round = SCAN_WARPS * SCAN_MLP;
  int64_t chunks = cdiv(a.n_blocks, 2 * round);
  while (rows * chunks < 4 * device_sms() && chunks < cdiv(a.n_blocks, SCAN_WARPS)) chunks *= 2;
  a.n_chunks = (int)(chunks < MAX_CHUNKS ? chunks : MAX_CHUNKS);
  a.state = state;
  a.words = state_words;
  a.slot = slot;
  a.token = token;
  a.parent = parent;
  a.score_out = score_out;
  a.state_out = state_out;
  a.part = reinterpret_cast<float2*>(workspace);
  a.top = reinterpret_cast<float*>(a.part + rows * MAX_CHUNKS);
  SUB_CUDA_TRY(once_per_device([] {
    cudaError_t e = cudaFuncSetAttribute(pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PICK_SMEM);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(beam_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PICK_SMEM);
  }));
  const size_t bytes = pick_shared(a.n_blocks, n_beams, n_best).bytes;
  const int most = largest_cluster();
  // One launch where a CTA of a cluster has 80 blocks at most: 3 us less of the host's time, and as
  // long on the GPU (1 beam of 152064 logits 9.7 us and 9.5; 16 trees of 5 beams of 5000 13.0 and 13.8;
  // but 4 beams of 152064, 297 blocks per CTA, 13.3 and 10.4, and 64 trees of 8 of 128256 87 and 59: a
  // cluster's SMs are few, and wait for 16 to be free at once).  More than 16 sequences that the rule
  // sends here were not timed.
  if (a.n_blocks <= 80 * (most / n_beams)) {
    const int team = (int)std::min<int64_t>(most / n_beams, cdiv(a.n_blocks, round));   // a round of loads each
    SUB_CUDA_TRY(launch_clusters(beam_kernel, n_seqs, team * n_beams, PICK_THREADS + 32, bytes, st, a, team));
    return SUB_OK;
  }
  SUB_CUDA_TRY(launch_k(scan_kernel, dim3((unsigned)rows, a.n_chunks), dim3(SCAN_THREADS), 0, st, a));
  SUB_CUDA_TRY(launch_clusters(pick_kernel, n_seqs, std::min(n_beams, most), PICK_THREADS + 32, bytes, st, a));
  return SUB_OK;
}
