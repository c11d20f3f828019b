// New rows of a batch turned to their positions on the way into a paged cache.
//
// Pair (x1, x2) = elements (i, i + D / 2) of a head becomes (x1 cos - x2 sin,
// x2 cos + x1 sin) of the angle at * freqs[i].  Angles of far positions lose their
// fraction of a turn in fp32 (at 10^5 radians a step is 2^-7), so they are formed in
// whole numbers: step[i] is the frequency in turns times 2^64, right in all of its bits, and
// the product's overflow is the whole turns.  One 64-bit multiplication then gives the
// fraction to 2^-32 of a turn and better (2^-65 times a position below 2^31, and half a step
// of the 2^-32 that are kept), and sincospi takes it without another reduction.
//
// Memory bound: q is read and written, K read and written, V copied.  A warp takes
// one token's K, or V, or 16 heads of its q; D / 16 lanes hold a head, each the two
// 16-byte chunks whose elements are pairs, so that nothing is exchanged between lanes but a
// row's largest value (codes) and the angles: each lane forms two of the D / 2 and the
// warp shares them through shared memory.  A lane reads both chunks before it writes
// them, so q may be turned in place.
// Measured: 8403 rows of 32 and 8 heads of 128 into bf16 36.6 us (206 MB, 5.6 TB/s); one row of 4
// and 2 heads 2.6, its dependent reads.
#include <cmath>
#include "kv_rows.cuh"

namespace sub {
namespace {

constexpr int ROPE_WARPS = 4;
constexpr int Q_HEADS = 16;   // heads of q that a warp takes

struct RopeArgs {
  SeqTable t;
  int layer, n_heads_kv, n_heads_q;
  const uint16_t* src[3];   // K, V, Q rows
  int64_t ld[3];
  void* pool[2];            // bf16 or uint8
  float* scale[2];
  uint16_t* q_out;
  int64_t ldo;
  const int32_t* at;
  uint64_t step[64];
};

template <int D, bool Q8>
__global__ void __launch_bounds__(ROPE_WARPS * 32) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int HL = D / 16, PER = 32 / HL;   // lanes of a head, heads per pass
  constexpr int U = Q_HEADS / PER;            // passes whose loads are in flight together
  __shared__ float2 s_turn[ROPE_WARPS][D / 2];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * ROPE_WARPS + warp;
  if (row >= a.t.n_rows) return;
  const int part = min((int)blockIdx.y, 2);   // K, V, Q
  const int first = part < 2 ? 0 : ((int)blockIdx.y - 2) * Q_HEADS;
  const int heads = part < 2 ? a.n_heads_kv : min(a.n_heads_q, first + Q_HEADS);
  const int sub = lane / HL, l = lane % HL;
  const uint16_t* const src = a.src[part] + row * a.ld[part] + l * 8;
  uint4 w[U][2];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * PER + sub;
#pragma unroll
      for (int x = 0; x < 2; ++x)
        w[u][x] = h < heads ? ldg_cg_v4(src + (int64_t)h * D + x * (D / 2)) : make_uint4(0, 0, 0, 0);
    }
  };
  load(first);   // on its way while the row's place is looked up
  const int given = a.at ? a.at[row] : 0;
  const Place p = find_place(a.t, row, lane);
  if (part < 2 ? p.page < 0 : !p.in_seq) return;
  float2 turn[8];   // (cos, sin) of the lane's pairs
  if (part != 1) {
    const uint64_t at = (uint64_t)(a.at ? (int64_t)given : p.pos);
#pragma unroll
    for (int i = lane; i < D / 2; i += 32) {
      // of the nearest whole turn: half turns in [-1, 1)
      const float x = (float)(int32_t)((at * a.step[i] + 0x80000000u) >> 32) * 0x1p-31f;
      float2 cs;
      sincospif(x, &cs.y, &cs.x);
      s_turn[warp][i] = cs;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) turn[i] = s_turn[warp][l * 8 + i];
  }
  for (int h0 = first; h0 < heads; h0 += U * PER) {
    if (h0 > first) load(h0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * PER + sub;
      const bool ok = h < heads;
      float x[2][8];
      unpack8(w[u][0], x[0]);
      unpack8(w[u][1], x[1]);
      if (part != 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x1 = x[0][i], x2 = x[1][i];
          x[0][i] = fmaf(x1, turn[i].x, -(x2 * turn[i].y));
          x[1][i] = fmaf(x2, turn[i].x, x1 * turn[i].y);
        }
      }
      if (!Q8 || part == 2) {
        uint4* to = nullptr;
        if (ok)
          to = part == 2 ? reinterpret_cast<uint4*>(a.q_out + row * a.ldo + (int64_t)h * D)
                         : reinterpret_cast<uint4*>(a.pool[part]) +
                               pool_row(a.t, a.layer, a.n_heads_kv, p.page, h, p.at) * (D / 8);
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (ok)
            to[y * HL + l] = part == 1 ? w[u][y]   // bit for bit, NaN too
                                       : make_uint4(pack_bf16x2(x[y][0], x[y][1]), pack_bf16x2(x[y][2], x[y][3]),
                                                    pack_bf16x2(x[y][4], x[y][5]), pack_bf16x2(x[y][6], x[y][7]));
      } else {
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) big = max_nan(big, max_nan(fabsf(x[0][i]), fabsf(x[1][i])));
#pragma unroll
        for (int o = HL / 2; o; o >>= 1) big = max_nan(big, __shfl_xor_sync(~0u, big, o));
        float s, t;
        row_scale(big, s, t);
        if (ok) {
          const int64_t r = pool_row(a.t, a.layer, a.n_heads_kv, p.page, h, p.at);
          uint2* const to = reinterpret_cast<uint2*>(a.pool[part]) + r * (D / 8) + l;
          to[0] = codes8(x[0], t);
          to[HL] = codes8(x[1], t);
          if (l == 0) a.scale[part][r] = s;
        }
      }
    }
  }
}

// freq / (2 pi) in units of 2^-64, without its whole turns, to the nearest.  (A quotient of
// doubles has 53 bits before the whole turns drop out: of a frequency of 10^6 that is 2^-36 of a turn,
// and 10^5 positions on 2^-20.)  freq, finite and below 2^20, is m 2^e in whole numbers, so its
// whole turns and its fraction lie in m times 1 / (2 pi) to 192 bits, which is below
// 2^-64 of a unit short.
uint64_t turn_step(double freq) {
  constexpr uint64_t INV_2PI[3] = {0x36d8a5664f10e410u, 0x7f09d5f47d4d3770u, 0x28be60db9391054au};   // low word first
  if (freq == 0.) return 0;
  int e;
  const uint64_t m = (uint64_t)std::ldexp(std::frexp(freq, &e), 53);
  uint64_t w[5] = {0, 0, 0, 0, 0};   // m / (2 pi) in units of 2^-192
  unsigned __int128 sum = 0;
  for (int i = 0; i < 3; ++i) {
    sum += (unsigned __int128)m * INV_2PI[i];
    w[i] = (uint64_t)sum;
    sum >>= 64;
  }
  w[3] = (uint64_t)sum;
  const int shift = 128 + 53 - e;   // from there to the result, 161 at least
  if (shift > 256) return 0;
  const int at = shift / 64, by = shift % 64;   // at = 4: by = 0
  const uint64_t x = by ? w[at] >> by | w[at + 1] << (64 - by) : w[at];
  return x + (w[(shift - 1) / 64] >> (shift - 1) % 64 & 1);
}

template <bool Q8, class Cache>
int32_t append_rope(const sub_bf16* Q, int64_t ldq, int32_t n_heads_q, const sub_bf16* K, int64_t ldk,
                    const sub_bf16* V, int64_t ldv, const Cache* kv, int32_t layer, const sub_batch* batch,
                    const sub_rope* rope, const int32_t* at, sub_bf16* Q_out, int64_t ldo, RopeArgs a,
                    void* stream) {
  SUB_TRY(make_seq_table(kv, layer, batch, &a.t));
  SUB_CHECK_ARG(rope, "null pointer");
  SUB_CHECK_ARG(rope->head_dim == kv->head_dim, "the rotation is of another head_dim");
  SUB_CHECK_ARG(n_heads_q >= 0 && n_heads_q <= 65535, "n_heads_q out of range");
  if (a.t.n_rows == 0) return SUB_OK;
  const int64_t width = (int64_t)kv->n_heads_kv * kv->head_dim, q_width = (int64_t)n_heads_q * kv->head_dim;
  SUB_CHECK_ARG(K && V && (n_heads_q == 0 || (Q && Q_out)), "null pointer");
  SUB_CHECK_ARG((reinterpret_cast<uintptr_t>(at) & 3) == 0, "at must be 4-byte aligned");
  SUB_CHECK_ARG(aligned16(K) && aligned16(V) && ldk % 8 == 0 && ldv % 8 == 0, "rows must be 16-byte aligned");
  SUB_CHECK_ARG(ldk >= width && ldv >= width, "row stride below n_heads_kv * head_dim");
  if (n_heads_q) {
    SUB_CHECK_ARG(aligned16(Q) && aligned16(Q_out) && ldq % 8 == 0 && ldo % 8 == 0,
                  "rows must be 16-byte aligned");
    SUB_CHECK_ARG(ldq >= q_width && ldo >= q_width, "row stride below n_heads_q * head_dim");
    SUB_CHECK_ARG(Q != Q_out || ldq == ldo, "Q turned in place has one row stride");
  }
  a.layer = layer;
  a.n_heads_kv = kv->n_heads_kv;
  a.n_heads_q = n_heads_q;
  a.src[0] = K;
  a.src[1] = V;
  a.src[2] = Q;
  a.ld[0] = ldk;
  a.ld[1] = ldv;
  a.ld[2] = ldq;
  a.pool[0] = kv->k;
  a.pool[1] = kv->v;
  a.q_out = Q_out;
  a.ldo = ldo;
  a.at = at;
  memcpy(a.step, rope->step, sizeof(a.step));
  auto k = kv->head_dim == 128 ? rope_append_kernel<128, Q8> : rope_append_kernel<64, Q8>;
  const dim3 grid((unsigned)cdiv(a.t.n_rows, ROPE_WARPS), 2 + (unsigned)cdiv(n_heads_q, Q_HEADS));
  SUB_CUDA_TRY(launch_k(k, grid, dim3(ROPE_WARPS * 32), 0, as_stream(stream), a));
  return SUB_OK;
}

}  // namespace
}  // namespace sub

using namespace sub;

extern "C" int32_t sub_rope_init(int32_t head_dim, double theta, const double* freqs_host, sub_rope* rope) {
  SUB_CHECK_ARG(rope, "null pointer");
  SUB_CHECK_ARG(head_dim == 64 || head_dim == 128, "head_dim must be 64 or 128");
  SUB_CHECK_ARG(freqs_host || (theta >= 1.0 && theta <= 1e12), "theta must be in [1, 1e12]");
  const int n = head_dim / 2;
  for (int i = 0; freqs_host && i < n; ++i)
    SUB_CHECK_ARG(freqs_host[i] >= 0.0 && freqs_host[i] <= 1e6, "freqs must be in [0, 1e6] radians");
  memset(rope, 0, sizeof(*rope));
  rope->head_dim = head_dim;
  for (int i = 0; i < n; ++i)
    rope->step[i] = turn_step(freqs_host ? freqs_host[i] : std::pow(theta, -2.0 * i / head_dim));
  return SUB_OK;
}

extern "C" int32_t sub_kv_append_rope(const sub_bf16* Q, int64_t ldq, int32_t n_heads_q, const sub_bf16* K,
                                      int64_t ldk, const sub_bf16* V, int64_t ldv, const sub_kv_cache* kv,
                                      int32_t layer, const sub_batch* batch, const sub_rope* rope,
                                      const int32_t* at, sub_bf16* Q_out, int64_t ldo, void* stream) {
  return append_rope<false>(Q, ldq, n_heads_q, K, ldk, V, ldv, kv, layer, batch, rope, at, Q_out, ldo,
                            RopeArgs{}, stream);
}

extern "C" int32_t sub_kv8_append_rope(const sub_bf16* Q, int64_t ldq, int32_t n_heads_q, const sub_bf16* K,
                                       int64_t ldk, const sub_bf16* V, int64_t ldv, const sub_kv8_cache* kv,
                                       int32_t layer, const sub_batch* batch, const sub_rope* rope,
                                       const int32_t* at, sub_bf16* Q_out, int64_t ldo, void* stream) {
  SUB_TRY(check_scales(kv));
  RopeArgs a{};
  a.scale[0] = kv->k_scale;
  a.scale[1] = kv->v_scale;
  return append_rope<true>(Q, ldq, n_heads_q, K, ldk, V, ldv, kv, layer, batch, rope, at, Q_out, ldo, a,
                           stream);
}
