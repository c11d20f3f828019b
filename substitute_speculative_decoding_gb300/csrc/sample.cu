// Probabilities from logits, and the verification of chains of drafted tokens
// against them ("SubSpec: Using the Target Model's Own Low-Bit Shadow as Its
// Draft Model", 6.2, Leviathan et al.).
//
// Both pass once over rows of V values.  A row belongs to one thread-block
// cluster, so that a single row still streams through several SMs, and the
// CTAs agree on the row's sums through distributed shared memory: one launch,
// no scratch.
#include <cmath>
#include <type_traits>
#include "rows.cuh"

namespace sub {
namespace {

// ------------------------------------------------------------- softmax --
// p = exp((z - m) / T) / sum, with m the largest logit.  Bound by HBM: 4 bytes
// in, 4 out.  The first pass keeps a running maximum and sum per thread, the
// second reads the row again, from L2: a row's CTAs run at the same time, so
// what is between the passes are a few dozen MB.  (Keeping a row in registers between
// the passes left room for two CTAs per SM, and a cluster's copies, sums and
// stores did not overlap enough: 4.1 TB/s on 576 rows of 128256.)  The CTAs exchange maxima
// and sums in one cluster barrier.
template <int THREADS, int MLP>   // MLP: groups a thread loads in one round
__global__ void __launch_bounds__(THREADS, 1280 / THREADS)
probs_kernel(const float* logits, int64_t V, Sharpen sharp, float* probs) {
  constexpr int WARPS = THREADS / 32;
  __shared__ float2 s_warp[WARPS];
  __shared__ float2 s_peer[MAX_CLUSTER];   // each CTA's (largest logit, sum), written by it
  cg::cluster_group cluster = cg::this_cluster();
  const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t row = blockIdx.x / size;
  if (size > 1) cluster_here();
  pdl_wait();
  pdl_trigger();
  const float* z = logits + row * V;
  float* out = probs + row * V;
  const Row r(z, V);
  int lo, hi;
  share(r.n, rank, size, lo, hi);
  auto expo = [&](float d) { return sharp.expo(d); };
  auto exponents = [&](const float4& x, float minus) { return sharp.exponents(x, minus); };
  auto merge = [&](float& m, float& s, float m2, float s2) { sharp.merge(m, s, m2, s2); };
  float m = -INFINITY, s = 0.f;
  float4 x[MLP];
  for (int g0 = lo + threadIdx.x; g0 < hi; g0 += MLP * THREADS) {
#pragma unroll
    for (int k = 0; k < MLP; ++k)
      x[k] = g0 + k * THREADS < hi ? load_group(z, r, g0 + k * THREADS, -INFINITY)
                                   : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    float big = m;
#pragma unroll
    for (int k = 0; k < MLP; ++k)
      big = fmaxf(fmaxf(big, fmaxf(x[k].x, x[k].y)), fmaxf(x[k].z, x[k].w));
    // no logit above -infinity so far: every value is 0 whatever the reference
    const float ref = big == -INFINITY ? 0.f : big;
    s *= expo(m - ref);
    m = big;
#pragma unroll
    for (int k = 0; k < MLP; ++k) {
      const float4 e = exponents(x[k], -ref);   // (the sum is at least 1: no term below 2^-126 counts)
      s += (exp2_fast(e.x) + exp2_fast(e.y)) + (exp2_fast(e.z) + exp2_fast(e.w));
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1)
    merge(m, s, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, s, o));
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = make_float2(m, s);
  __syncthreads();
  m = -INFINITY;
  s = 0.f;
  for (int w = 0; w < WARPS; ++w) merge(m, s, s_warp[w].x, s_warp[w].y);
  if (size > 1) {
    // every CTA writes its own into all of them, so that one barrier is enough:
    // nobody reads the memory of a CTA that may have ended
    cluster_all_here();
    if ((int)threadIdx.x < size) *cluster.map_shared_rank(&s_peer[rank], threadIdx.x) = make_float2(m, s);
    cluster.sync();
    m = -INFINITY;
    s = 0.f;
    for (int i = 0; i < size; ++i) merge(m, s, s_peer[i].x, s_peer[i].y);
  }
  const float ref = m == -INFINITY ? 0.f : m, f = s == 0.f ? 0.f : 1.f / s;
  const bool again = hi - lo > MLP * THREADS;   // a single round is still in registers
  auto store = [&](auto alike) {   // probabilities lie like the logits: stored in fours
    for (int g0 = lo + threadIdx.x; g0 < hi; g0 += MLP * THREADS) {
#pragma unroll
      for (int k = 0; k < MLP; ++k)
        if (again && g0 + k * THREADS < hi) x[k] = load_group(z, r, g0 + k * THREADS, -INFINITY);
#pragma unroll
      for (int k = 0; k < MLP; ++k) {
        const int g = g0 + k * THREADS;
        if (g >= hi) break;
        const float4 e = exponents(x[k], -ref);
        const float w[4] = {exp2_small(e.x) * f, exp2_small(e.y) * f, exp2_small(e.z) * f,
                            exp2_small(e.w) * f};
        if (decltype(alike)::value && r.whole(g)) {
          __stcs(reinterpret_cast<float4*>(out - r.mis) + g, make_float4(w[0], w[1], w[2], w[3]));
        } else {
          const int64_t at = r.first(g);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (at + i >= 0 && at + i < V) out[at + i] = w[i];
        }
      }
    }
  };
  if (((reinterpret_cast<uintptr_t>(z) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0) store(std::true_type{});
  else store(std::false_type{});
}

// ------------------------------------------------- draft verification --
constexpr int VER_THREADS = 256, VER_WARPS = VER_THREADS / 32, VER_MLP = 4;

struct VerifyArgs {
  const float* p;
  const float* q;
  const int32_t* draft;
  const float* u;
  int n_draft;
  int64_t V;
  int32_t* tokens;
  int32_t* n_accepted;
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan64(uint64_t v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// One cluster per sequence.  Every warp repeats the acceptance tests (a few
// numbers each), which name the row to sample from; then the row is read
// once: weights as whole multiples of 2^-43, so that their sums do not depend
// on the order and the sampled token is the same on any split.  (Formed in two
// halves by fp32 additions that leave the whole number in the mantissa's low bits:
// conversions to 64-bit integers run at a small fraction of that rate.)  Each warp sums
// a contiguous part; the sums of all warps of the cluster name the one warp
// whose part holds the number, and that warp alone reads its part again (from
// L2) to find the token.  Bound by the latency of four dependent rounds of
// reads at few sequences, by HBM (one row of p and of q per sequence) at many.
__global__ void __launch_bounds__(VER_THREADS, 4) verify_kernel(VerifyArgs a) {
  __shared__ uint64_t s_sum[MAX_CLUSTER * VER_WARPS];   // every warp of the cluster writes its own
  cg::cluster_group cluster = cg::this_cluster();
  const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t b = blockIdx.x / size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = a.n_draft, me = rank * VER_WARPS + warp;
  if (size > 1) cluster_here();
  pdl_wait();
  pdl_trigger();
  const float uf = __ldcg(a.u + b * (n + 1) + n);

  // ---- the longest accepted prefix ----
  int acc = n;
  bool refused = false;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    bool stop = i < n, bad = false;
    if (i < n) {
      const int x = __ldcg(a.draft + b * n + i);
      if (x >= 0 && x < a.V) {
        const float ui = __ldcg(a.u + b * (n + 1) + i);
        const double pv = __ldcg(a.p + (b * (n + 1) + i) * a.V + x);
        const double qv = a.q ? __ldcg(a.q + (b * n + i) * a.V + x) : 1.f;
        bad = !((double)ui * qv < pv);   // 48-bit product: exact
        stop = bad;
      }
    }
    const unsigned stops = __ballot_sync(~0u, stop);
    if (stops) {
      const int first = __ffs(stops) - 1;
      acc = i0 + first;
      refused = (__ballot_sync(~0u, bad) >> first) & 1u;
      break;
    }
  }
  if (rank == 0) {
    for (int i = threadIdx.x; i <= n; i += VER_THREADS)
      if (i != acc) a.tokens[b * (n + 1) + i] = i < acc ? __ldcg(a.draft + b * n + i) : -1;
    if (threadIdx.x == 0) a.n_accepted[b] = acc;
  }

  const float* p = a.p + (b * (n + 1) + acc) * a.V;
  const float* q = a.q ? a.q + (b * n + acc) * a.V : nullptr;   // read after a rejection only
  const int64_t x = refused ? __ldcg(a.draft + b * n + acc) : -1;
  const Row r(p, a.V);
  const bool q_vec = q && ((reinterpret_cast<uintptr_t>(q) >> 2) & 3) == (unsigned)r.mis;
  int lo, hi;
  share(r.n, me, size * VER_WARPS, lo, hi);
  // rint(x 2^43) = high 2^22 + low for x in [0, 1]: high = rint(x 2^21) in 23 bits over
  // 2^23, low = rint(rest 2^22) in -2^21 .. 2^21 over 3 2^22
  constexpr uint32_t HIGH0 = 0x4B000000u, LOW0 = 0x4B400000u;
  auto halves = [&](float d, uint32_t& high, uint32_t& low) {
    const float x = fminf(fmaxf(d, 0.f), 1.f);   // NaN counts as 0
    const float h = fmaf(x, 0x1p21f, 8388608.f);
    const float rest = fmaf(x, 0x1p21f, -(h - 8388608.f));   // exact
    high = __float_as_uint(h);
    low = __float_as_uint(fmaf(rest, 0x1p22f, 12582912.f));
  };
  auto weights = [&](const float4& pv, const float4& qv, uint64_t (&w)[4]) {
    const float d[4] = {pv.x - qv.x, pv.y - qv.y, pv.z - qv.z, pv.w - qv.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h, l;
      halves(d[i], h, l);
      w[i] = (uint64_t)(((int64_t)(h - HIGH0) << 22) + (int32_t)(l - LOW0));
    }
  };
  auto load_q = [&](int g, bool diff) {
    if (!diff) return make_float4(0.f, 0.f, 0.f, 0.f);
    if (q) return q_vec ? load_group(q, r, g, 0.f) : load_group<false>(q, r, g, 0.f);
    const int64_t e = x - r.first(g);
    return make_float4(e == 0, e == 1, e == 2, e == 3);
  };
  const uint64_t u64 = __float2ull_rz(fminf(fmaxf(uf, 0.f), 0x1.fffffep-1f) * 0x1p64f);

  bool alone = size > 1;   // the others may not run yet
  for (bool diff = refused;; diff = false) {
    // sums of the halves, at most 2^9 values per lane (V <= 2^20): 2^30 of each
    uint32_t high = 0, low = 0, count = 0;
    for (int g0 = lo + lane; g0 < hi; g0 += 32 * VER_MLP) {
      float4 pv[VER_MLP], qv[VER_MLP];
#pragma unroll
      for (int k = 0; k < VER_MLP; ++k) {
        const int g = g0 + 32 * k;
        pv[k] = qv[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (g < hi) {
          pv[k] = load_group(p, r, g, 0.f);
          qv[k] = load_q(g, diff);
        }
      }
#pragma unroll
      for (int k = 0; k < VER_MLP; ++k) {
        const float d[4] = {pv[k].x - qv[k].x, pv[k].y - qv[k].y, pv[k].z - qv[k].z, pv[k].w - qv[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t h, l;
          halves(d[i], h, l);
          high += h;
          low += l;
        }
      }
      count += 4 * VER_MLP;
    }
    // (what the bits lie over goes with the wrapped-around sums)
    const uint64_t mine = warp_sum64((uint64_t)(((int64_t)(high - count * HIGH0) << 22) +
                                                (int32_t)(low - count * LOW0)));
    if (alone) cluster_all_here();
    alone = false;
    if (lane < size) *cluster.map_shared_rank(&s_sum[me], lane) = mine;
    if (size > 1) cluster.sync();
    else __syncthreads();
    uint64_t total = 0, before = 0;
    for (int i = lane; i < size * VER_WARPS; i += 32) {
      const uint64_t t = s_sum[i];
      total += t;
      before += i < me ? t : 0;
    }
    total = warp_sum64(total);
    before = warp_sum64(before);
    if (total == 0) {
      if (diff) {   // nothing left after the rejection: sample p itself
        if (size > 1) cluster.sync();   // everyone has read the sums
        else __syncthreads();
        continue;
      }
      if (me == 0 && lane == 0) a.tokens[b * (n + 1) + acc] = 0;
      return;
    }
    // ---- the value whose running sum first exceeds u * total ----
    const uint64_t target = __umul64hi(total, u64);   // floor: sums are whole numbers
    if (target < before || target - before >= mine) return;
    uint64_t rest = target - before;   // within this warp's part
    for (int g0 = lo; g0 < hi; g0 += 32 * VER_MLP) {
      float4 pv[VER_MLP], qv[VER_MLP];
#pragma unroll
      for (int k = 0; k < VER_MLP; ++k) {
        const int g = g0 + 32 * k + lane;
        pv[k] = qv[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (g < hi) {
          pv[k] = load_group(p, r, g, 0.f);
          qv[k] = load_q(g, diff);
        }
      }
#pragma unroll
      for (int k = 0; k < VER_MLP; ++k) {
        uint64_t w[4];
        weights(pv[k], qv[k], w);
        const uint64_t t = (w[0] + w[1]) + (w[2] + w[3]);
        const uint64_t run = warp_scan64(t, lane);
        const unsigned over = __ballot_sync(~0u, run > rest);
        if (over) {
          if (lane == __ffs(over) - 1) {
            uint64_t at = run - t;
            int i = 0;
            while (i < 3 && (at += w[i]) <= rest) ++i;
            a.tokens[b * (n + 1) + acc] = (int32_t)(r.first(g0 + 32 * k + lane) + i);
          }
          return;
        }
        rest -= __shfl_sync(~0u, run, 31);
      }
    }
    return;
  }
}

}  // namespace
}  // namespace sub

using namespace sub;

extern "C" int32_t sub_probs(const float* logits, int64_t rows, int64_t V, float temperature,
                             float* probs, void* stream) {
  SUB_CHECK_ARG(rows >= 0 && rows <= (1 << 24), "rows out of range");
  SUB_CHECK_ARG(V >= 1 && V <= MAX_V, "V must be in [1, 2^20]");
  SUB_CHECK_ARG(temperature >= 1e-6f && temperature <= 1e6f,
                "temperature must be in [1e-6, 1e6]");
  if (rows == 0) return SUB_OK;
  SUB_CHECK_ARG(logits && probs, "null pointer");
  SUB_CHECK_ARG(aligned4(logits) && aligned4(probs), "logits and probs must be 4-byte aligned");
  SUB_CHECK_ARG(probs == logits || !overlap(logits, rows * V, probs, rows * V),
                "probs must be the logits or lie apart from them");
  const Sharpen sharp = make_sharpen(temperature);
  const cudaStream_t st = as_stream(stream);
  // A round of a CTA's loads takes 16 values per thread.  Rows of one round: one
  // small CTA.  Longer ones: a cluster whose CTAs need two rounds at most, or as many
  // CTAs as there are SMs (448 rows of 5000: 7 us, against 22 as clusters of eight).
  if (V <= 2048) {
    SUB_CUDA_TRY(launch_clusters(probs_kernel<128, 4>, rows, 1, 128, 0, st, logits, V, sharp, probs));
    return SUB_OK;
  }
  int size = 1;
  const int sms = device_sms();
  while (size < MAX_CLUSTER && (V > size * 8192 || (rows * size < sms && V > size * 4096))) size *= 2;
  SUB_CUDA_TRY(launch_clusters(probs_kernel<256, 4>, rows, size, 256, 0, st, logits, V, sharp, probs));
  return SUB_OK;
}

extern "C" int32_t sub_verify_sample(const float* p, const float* q, const int32_t* draft,
                                     const float* u, int32_t n_seqs, int32_t n_draft, int64_t V,
                                     int32_t* tokens, int32_t* n_accepted, void* stream) {
  SUB_CHECK_ARG(n_seqs >= 0 && n_seqs <= (1 << 24), "n_seqs out of range");
  SUB_CHECK_ARG(n_draft >= 0 && n_draft <= (1 << 20), "n_draft out of range");
  SUB_CHECK_ARG(V >= 1 && V <= MAX_V, "V must be in [1, 2^20]");
  if (n_seqs == 0) return SUB_OK;
  SUB_CHECK_ARG(p && u && tokens && n_accepted && (draft || n_draft == 0), "null pointer");
  SUB_CHECK_ARG(aligned4(p) && aligned4(q) && aligned4(draft) && aligned4(u) && aligned4(tokens) &&
                    aligned4(n_accepted),
                "pointers must be 4-byte aligned");
  const __int128 chain = n_draft, seqs = n_seqs;
  for (int i = 0; i < 2; ++i) {
    const void* const out = i ? (const void*)n_accepted : tokens;
    const __int128 n = i ? seqs : seqs * (chain + 1);
    SUB_CHECK_ARG(!overlap(out, n, p, seqs * (chain + 1) * V) && !overlap(out, n, q, seqs * chain * V) &&
                      !overlap(out, n, draft, seqs * chain) && !overlap(out, n, u, seqs * (chain + 1)),
                  "tokens and n_accepted must lie apart from the inputs");
  }
  SUB_CHECK_ARG(!overlap(tokens, seqs * (chain + 1), n_accepted, seqs),
                "tokens and n_accepted must lie apart");
  VerifyArgs a{p, q, draft, u, n_draft, V, tokens, n_accepted};
  // rows one CTA reads in a few rounds need no cluster
  const int size = V <= 8192 ? 1 : MAX_CLUSTER;
  SUB_CUDA_TRY(launch_clusters(verify_kernel, n_seqs, size, VER_THREADS, 0, as_stream(stream), a));
  return SUB_OK;
}
