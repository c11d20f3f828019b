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
//        of exp, and the largest logit of every block of 128.
// pick   one cluster per sequence, a CTA per beam (or several): the k largest of the
//        block maxima name k blocks that hold all of the k largest logits (a logit
//        above which there are fewer than k others cannot lie in a block that k others
//        exceed), which are read again, from L2; the beams' lists meet in the
//        cluster's first CTA, where each candidate finds its place by bisection in the
//        others' lists.  Bound by latency: some ten dependent steps.
//
// (Every CTA keeping the best of its part while it streams would need no second
// reading, but a sorted list per thread costs the scan its loads in flight.)
//
// Rounding: terms of the sums of exp are fp32 relative to the largest logit, partial
// sums of a thread and a CTA too; the CTAs' sums are joined, and the scores formed and
// compared, in 64 bits, so that where two beams' candidates meet, only the error of the
// sums (2^-23 or so) can exchange them.
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

__global__ void __launch_bounds__(SCAN_THREADS, 4) scan_kernel(const __grid_constant__ BeamArgs a) {
  __shared__ float2 s_warp[SCAN_WARPS];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const float* const z = a.logits + row * a.V;
  const Row r(z, a.V);
  const int blocks = (r.n + BLOCK_GROUPS - 1) / BLOCK_GROUPS;
  int lo, hi;
  share(blocks, blockIdx.y, a.n_chunks, lo, hi);
  const float live = __ldcg(a.score + row);
  float* const top = a.top + row * a.n_blocks;
  float m = -INFINITY, s = 0.f;
  for (int b0 = lo + warp * SCAN_MLP; b0 < hi; b0 += SCAN_WARPS * SCAN_MLP) {
    float4 x[SCAN_MLP];
#pragma unroll
    for (int k = 0; k < SCAN_MLP; ++k) {
      const int g = (b0 + k) * BLOCK_GROUPS + lane;
      x[k] = b0 + k < hi && g < r.n ? load_group(z, r, g, -INFINITY)
                                    : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
    if (!alive(live)) break;   // (the whole CTA, with its first loads under way)
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
    if (lane < SCAN_MLP && b0 + lane < hi) top[b0 + lane] = key_float(mine);
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
  if (!alive(live)) return;
#pragma unroll
  for (int o = 16; o; o >>= 1)
    a.sharp.merge(m, s, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, s, o));
  if (lane == 0) s_warp[warp] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < SCAN_WARPS; ++w) a.sharp.merge(m, s, s_warp[w].x, s_warp[w].y);
  a.part[row * a.n_chunks + blockIdx.y] = make_float2(m, s);
}

// ------------------------------------------------------------------- pick --
constexpr int PARTS = 128;   // a selection's threshold comes from the largest keys of so many parts
static_assert(SUB_MAX_BEAMS <= PARTS && PICK_THREADS == 2 * PARTS, "two threads per part");

// most keys that select() may have to compare with each other: n keys, the k largest
__host__ __device__ inline int survivors(int n, int k) {
  const int per = 2 * ((n + PICK_THREADS - 1) / PICK_THREADS);
  return n < k * per ? n : k * per;
}

// The k largest of n keys in shared memory (all unlike; 0: none) to out, in falling order,
// zeros behind them.  The k-th largest of 128 parts' largest keys is a threshold that k
// keys reach and few others pass; those are ranked by counting.  By the whole CTA.
__device__ void select(const uint64_t* keys, int n, int k, uint64_t* out, uint64_t* list, uint64_t* s_top,
                       int* s_count) {
  const int tid = threadIdx.x;
  uint64_t best = 0;
  for (int i = tid; i < n; i += PICK_THREADS) best = max(best, keys[i]);
  best = max(best, (uint64_t)__shfl_xor_sync(~0u, (unsigned long long)best, 1));
  if (!(tid & 1)) s_top[tid >> 1] = best;
  if (tid == 0) *s_count = 0;
  if (tid < k) out[tid] = 0;
  __syncthreads();
  int above = 0;   // parts whose largest key is above this one's; the two threads count a half each
#pragma unroll 8
  for (int i = 0; i < PARTS / 2; ++i) above += s_top[2 * i + (tid & 1)] > best;
  above += __shfl_xor_sync(~0u, above, 1);
  // fewer than k parts with a key at all: every key is a candidate
  const bool mine = above == k - 1 && best != 0;
  uint64_t least = 1;
  if (__syncthreads_or(mine)) {
    if (mine && !(tid & 1)) s_top[0] = best;
    __syncthreads();
    least = s_top[0];
  }
  for (int i = tid; i < n; i += PICK_THREADS)
    if (keys[i] >= least) list[atomicAdd(s_count, 1)] = keys[i];
  __syncthreads();
  const int found = *s_count;
  for (int i = tid; i < found; i += PICK_THREADS) {
    const uint64_t x = list[i];
    int rank = 0;
    for (int j = 0; j < found && rank < k; ++j) rank += list[j] > x;
    if (rank < k) out[rank] = x;
  }
  __syncthreads();
}

struct PickShared {
  size_t list, cand_score, cand_token, bytes;   // offsets; the keys come first
};
__host__ __device__ inline PickShared pick_shared(int n_blocks, int n_beams, int k) {
  const int n = n_blocks > k * 128 ? n_blocks : k * 128;
  PickShared p;
  p.list = (size_t)n * 8;
  p.cand_score = p.list + (size_t)max(survivors(n_blocks, k), survivors(k * 128, k)) * 8;
  p.cand_token = p.cand_score + (size_t)n_beams * k * 8;
  p.bytes = p.cand_token + (size_t)n_beams * k * 4;
  return p;
}

__global__ void __launch_bounds__(PICK_THREADS) pick_kernel(const __grid_constant__ BeamArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t s_top[PARTS], s_out[SUB_MAX_BEAMS];
  __shared__ int s_found, s_count[SUB_MAX_BEAMS];   // of the first CTA: candidates of each beam
  __shared__ int s_parent[SUB_MAX_BEAMS];
  __shared__ double s_lse;
  cg::cluster_group cluster = cg::this_cluster();
  const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t b = blockIdx.x / size;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.n_best;
  if (size > 1) cluster_here();
  const PickShared at = pick_shared(a.n_blocks, a.n_beams, k);
  uint64_t* const keys = reinterpret_cast<uint64_t*>(smem);
  uint64_t* const list = reinterpret_cast<uint64_t*>(smem + at.list);
  double* const cand_score = reinterpret_cast<double*>(smem + at.cand_score);
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
    int n_cand = 0;
    if (alive(score)) {
      // ---- the log of the sum, by the first warp ----
      if (warp == 0) {
        float m = -INFINITY;
        for (int c = lane; c < a.n_chunks; c += 32) m = fmaxf(m, __ldcg(a.part + row * a.n_chunks + c).x);
        m = warp_max(m);
        double s = 0.;
        for (int c = lane; c < a.n_chunks; c += 32) {
          const float2 p = __ldcg(a.part + row * a.n_chunks + c);
          if (p.x != -INFINITY) s += (double)p.y * exp(((double)p.x - (double)m) / (double)a.temp);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        if (lane == 0)   // not finite: no continuations
          s_lse = fabsf(m) < INFINITY ? (double)m / (double)a.temp + log(s) : (double)INFINITY;
      }
      // ---- the blocks that hold the k largest logits ----
      for (int i = tid; i < blocks; i += PICK_THREADS) {
        const float x = __ldcg(a.top + row * a.n_blocks + i);
        keys[i] = x == -INFINITY ? 0 : rank_key(x, (uint32_t)i);
      }
      __syncthreads();
      select(keys, blocks, k, s_out, list, s_top, &s_found);
      // ---- their logits ----
      constexpr int AHEAD = 4;
      for (int i0 = warp; i0 < k; i0 += PICK_THREADS / 32 * AHEAD) {
        float4 x[AHEAD];
        int g[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const int i = i0 + u * (PICK_THREADS / 32);
          const uint64_t key = i < k ? s_out[i] : 0;
          g[u] = key ? (int)rank_idx(key) * BLOCK_GROUPS + lane : r.n;
          x[u] = g[u] < r.n ? load_group(z, r, g[u], -INFINITY)
                            : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const int i = i0 + u * (PICK_THREADS / 32);
          if (i >= k) break;
          const float v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {   // (elements before and past the row are -infinity)
            const float c = clean(v[e]);
            keys[i * 128 + e * 32 + lane] = c == -INFINITY ? 0 : rank_key(c, (uint32_t)(r.first(g[u]) + e));
          }
        }
      }
      __syncthreads();
      select(keys, k * 128, k, s_out, list, s_top, &s_found);
      if (s_lse < (double)INFINITY)
        while (n_cand < k && s_out[n_cand]) ++n_cand;
    }
    // ---- scores, to the cluster's first CTA ----
    if (alone) cluster_all_here();
    alone = false;
    if (tid < n_cand) {
      const uint64_t key = s_out[tid];
      const double x = ((double)score + (double)key_float((uint32_t)(key >> 32)) / (double)a.temp) - s_lse;
      *cluster.map_shared_rank(cand_score + j * k + tid, 0) = x;
      *cluster.map_shared_rank(cand_token + j * k + tid, 0) = (int32_t)rank_idx(key);
    }
    if (tid == 0) *cluster.map_shared_rank(s_count + j, 0) = n_cand;
    __syncthreads();   // s_out and s_lse are read
  }
  if (size > 1) cluster.sync();
  if (rank != 0) return;

  // ---- the first CTA: every candidate's place among all ----
  if (tid < SUB_MAX_BEAMS) s_parent[tid] = -1;
  __syncthreads();
  for (int i = tid; i < a.n_beams * k; i += PICK_THREADS) {
    const int j = i / k, c = i - j * k;
    if (c >= s_count[j]) continue;
    const double x = cand_score[i];
    int place = c;   // of its own beam's, so many come first
    for (int o = 0; o < a.n_beams && place < k; ++o) {
      if (o == j) continue;
      int lo = 0, hi = s_count[o];   // its candidates that come before this one
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const double y = cand_score[o * k + mid];
        if (y > x || (y == x && o < j)) lo = mid + 1;
        else hi = mid;
      }
      place += lo;
    }
    if (place >= k) continue;
    a.token[b * k + place] = cand_token[i];
    a.parent[b * k + place] = j;
    a.score_out[b * k + place] = (float)x;
    s_parent[place] = j;
  }
  __syncthreads();
  if (tid < k && s_parent[tid] < 0) {
    a.token[b * k + tid] = -1;
    a.parent[b * k + tid] = -1;
    a.score_out[b * k + tid] = -INFINITY;
  }
  // ---- the parents' states ----
  if (a.state_out)
    for (int64_t i = tid; i < (int64_t)k * a.words; i += PICK_THREADS) {
      const int p = (int)(i / a.words), w = (int)(i - (int64_t)p * a.words), j = s_parent[p];
      int32_t x = j < 0 ? 0 : __ldcg(a.state + (b * a.n_beams + j) * a.words + w);
      if (j >= 0 && a.slot >= 0 && (a.slot + p) >> 5 == w) x |= (int32_t)(1u << ((a.slot + p) & 31));
      a.state_out[b * k * a.words + i] = x;
    }
}

// Blocks of the longest layout of a row, and bytes of a call's workspace.
int block_stride(int64_t V) { return (int)((V + 6 + 127) / 128 + 3) / 4 * 4; }
int64_t beam_bytes(int64_t rows, int64_t V) {
  return cdiv(rows * (MAX_CHUNKS * (int64_t)sizeof(float2) + block_stride(V) * 4), 32) * 32;
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
    return cudaFuncSetAttribute(pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
  }));
  SUB_CUDA_TRY(launch_k(scan_kernel, dim3((unsigned)rows, a.n_chunks), dim3(SCAN_THREADS), 0, st, a));
  const int size = n_beams < MAX_CLUSTER ? n_beams : MAX_CLUSTER;
  SUB_CUDA_TRY(launch_clusters(pick_kernel, n_seqs, size, PICK_THREADS,
                               pick_shared(a.n_blocks, n_beams, n_best).bytes, st, a));
  return SUB_OK;
}
