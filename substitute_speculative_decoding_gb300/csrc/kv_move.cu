// Rows of a paged cache moved within their sequences, in all layers: the commit of
// the accepted paths of a batch's draft trees ("SubSpec: Using the Target Model's Own
// Low-Bit Shadow as Its Draft Model", 4.1 point 2 and 6.3).
//
// Memory bound, or at a few rows bound by the chain count -> position -> page ->
// row of dependent reads, so a CTA takes one layer of a sequence, K and V, and
// looks its rows' places up once for all heads.  In place: a destination may be
// a later row's source, so all rows of a head are in registers before the first
// of them is written (8 chunks of 16 bytes for each of 256 threads hold
// SUB_MAX_MOVE rows of 256 bytes); several heads at a time where the rows are fewer.
// 32 sequences of up to 12 rows through 28 layers of 4 heads of codes: 6.4 us (8.0 with
// a CTA for each side, two waves of them).
#include "batch.cuh"

namespace sub {
namespace {

constexpr int MOVE_THREADS = 256, MOVE_CHUNKS = 8;

struct MoveArgs {
  SeqTable t;               // start, pos: none
  int n_heads_kv, n_max;
  const int32_t *to, *from, *count;
  void* pool[2];
  float* scale[2];
};

// LANES: 16-byte chunks of a row
template <int LANES, bool Q8>
__global__ void __launch_bounds__(MOVE_THREADS) move_kernel(const __grid_constant__ MoveArgs a) {
  static_assert(SUB_MAX_MOVE * LANES <= MOVE_THREADS * MOVE_CHUNKS, "a head's rows fit the registers");
  __shared__ int64_t s_from[SUB_MAX_MOVE], s_to[SUB_MAX_MOVE];   // rows of the pool, of head 0; -1: not moved
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
  const int n = min(max(__ldcg(a.count + b), 0), a.n_max);
  if (n == 0) return;
  if (tid < n) {
    const int64_t x = __ldcg(a.from + (int64_t)b * a.n_max + tid), y = (int64_t)__ldcg(a.to + b) + tid;
    const int px = page_of(a.t, b, x), py = page_of(a.t, b, y);
    const bool ok = px >= 0 && py >= 0;
    const uint32_t ps = a.t.page_size;
    s_from[tid] = ok ? pool_row(a.t, layer, a.n_heads_kv, px, 0, (int)((uint32_t)x % ps)) : -1;
    s_to[tid] = ok ? pool_row(a.t, layer, a.n_heads_kv, py, 0, (int)((uint32_t)y % ps)) : -1;
  }
  __syncthreads();
  const int per_head = n * LANES, ps = a.t.page_size, heads = 2 * a.n_heads_kv;   // K's, V's
  const int together = MOVE_THREADS * MOVE_CHUNKS / per_head;                     // heads
  // i / per_head for i < 2048: (i + 1/2) / per_head is further than 2^-12 from a whole number, and
  // the product off by less
  const float by_head = 1.f / (float)per_head;
  for (int h0 = 0; h0 < heads; h0 += together) {
    const int items = min(together, heads - h0) * per_head;
    uint4 w[MOVE_CHUNKS];
    float sc[MOVE_CHUNKS];
    auto each = [&](auto f) {
#pragma unroll
      for (int k = 0; k < MOVE_CHUNKS; ++k) {
        const int i = k * MOVE_THREADS + tid;
        if (i >= items) break;
        const int h = (int)(((float)i + 0.5f) * by_head), r = (i - h * per_head) / LANES, c = i % LANES;
        const int side = h0 + h >= a.n_heads_kv, head = h0 + h - side * a.n_heads_kv;
        if (s_from[r] >= 0) f(k, r, side, (int64_t)head * ps, c);
      }
    };
    each([&](int k, int r, int side, int64_t head, int c) {
      w[k] = __ldcg(reinterpret_cast<const uint4*>(a.pool[side]) + (s_from[r] + head) * LANES + c);
      if (Q8 && c == 0) sc[k] = __ldcg(a.scale[side] + s_from[r] + head);
    });
    __syncthreads();
    each([&](int k, int r, int side, int64_t head, int c) {
      reinterpret_cast<uint4*>(a.pool[side])[(s_to[r] + head) * LANES + c] = w[k];
      if (Q8 && c == 0) a.scale[side][s_to[r] + head] = sc[k];
    });
  }
}

template <class Cache>
int32_t move(const Cache* kv, int32_t n_seqs, const int32_t* to, const int32_t* from, int32_t n_max,
             const int32_t* count, MoveArgs a, bool q8, void* stream) {
  SUB_CHECK_ARG(kv && kv->k && kv->v && kv->page_table, "null pointer");
  // (no rows of a batch here: start and pos are not read)
  const sub_batch none{kv->page_table, kv->page_table, n_seqs, 0, 0};
  SUB_TRY(make_seq_table(kv, 0, &none, &a.t));
  SUB_CHECK_ARG(kv->n_layers <= 65535, "n_layers out of range");
  SUB_CHECK_ARG(n_max >= 0 && n_max <= SUB_MAX_MOVE, "n_max must be in [0, SUB_MAX_MOVE]");
  if (n_max == 0) return SUB_OK;
  SUB_CHECK_ARG(to && from && count, "null pointer");
  SUB_CHECK_ARG(((reinterpret_cast<uintptr_t>(to) | reinterpret_cast<uintptr_t>(from) |
                  reinterpret_cast<uintptr_t>(count)) & 3) == 0,
                "to, from and count must be 4-byte aligned");
  a.t.start = a.t.pos = nullptr;
  a.n_heads_kv = kv->n_heads_kv;
  a.n_max = n_max;
  a.to = to;
  a.from = from;
  a.count = count;
  a.pool[0] = kv->k;
  a.pool[1] = kv->v;
  auto k = kv->head_dim == 128 ? (q8 ? move_kernel<8, true> : move_kernel<16, false>)
                               : (q8 ? move_kernel<4, true> : move_kernel<8, false>);
  SUB_CUDA_TRY(launch_k(k, dim3(n_seqs, kv->n_layers), dim3(MOVE_THREADS), 0, as_stream(stream), a));
  return SUB_OK;
}

}  // namespace
}  // namespace sub

using namespace sub;

extern "C" int32_t sub_kv_move(const sub_kv_cache* kv, int32_t n_seqs, const int32_t* to, const int32_t* from,
                               int32_t n_max, const int32_t* count, void* stream) {
  return move(kv, n_seqs, to, from, n_max, count, MoveArgs{}, false, stream);
}

extern "C" int32_t sub_kv8_move(const sub_kv8_cache* kv, int32_t n_seqs, const int32_t* to,
                                const int32_t* from, int32_t n_max, const int32_t* count, void* stream) {
  SUB_TRY(check_scales(kv));
  MoveArgs a{};
  a.scale[0] = kv->k_scale;
  a.scale[1] = kv->v_scale;
  return move(kv, n_seqs, to, from, n_max, count, a, true, stream);
}
