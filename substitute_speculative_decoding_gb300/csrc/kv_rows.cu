// Rows of a batch written into a paged cache and read back: bf16 copies, or
// 8-bit codes with one fp32 scale per (position, KV head) row.
//
// code = 128 + rint(x * (127 / a)), a = max |x| of the row, so that the largest
// value sits on code 1 or 255 and a value is off by at most half a step,
// a / 254.  Against 8-bit floats (e4m3: three mantissa bits, 2^-4 of each
// value) the even steps are about four times closer on rows of a normal
// distribution, and whole numbers up to 127 are exact in fp16 and bf16, so the
// attention's matrix products take the codes as they are and apply the scales
// outside of them.
//
// Memory bound: a row of K is read (2 D bytes) and written (D + 4) once.  D / 8
// lanes hold one (row, head), 16 bytes each, so a warp's load covers 512
// contiguous bytes of a token's row, the largest value is a shuffle away, and a
// warp takes one token: its sequence is searched once for all heads.  K and V
// go to different warps (together in one, with half the warps, both calls took 7% longer
// on 8403 rows of 8 heads and 14% on 64).
// Measured: 8403 rows of 8 heads of 128, K and V, written as codes in 14.5 us and read
// back in 10.9 (52 MB each, 3.6 and 4.8 TB/s, the codes' reading from L2), copied as bf16 in
// 12.3 (69 MB, 5.6 TB/s); 64 rows 3.0, 2.4 and 2.1 us, their dependent reads.  What
// is left to the floor (15.4 us for codes both ways) is the lookup of each row's sequence,
// position and page before its stores.
#include <algorithm>
#include "batch.cuh"

namespace sub {
namespace {

constexpr int ROW_WARPS = 4;

struct RowArgs {
  SeqTable t;
  int layer, n_heads_kv;
  const uint16_t* src[2];   // K, V rows (append)
  int64_t ld[2];
  void* pool[2];            // bf16 or uint8
  float* scale[2];
  uint16_t* dst[2];         // rows read back
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Row of this warp, its sequence and the page of its position.
struct Place {
  int row, page, at;
  bool in_seq;
};
__device__ __forceinline__ Place find_place(const SeqTable& t, int row, int lane) {
  Place p{row, -1, 0, false};
  if (row >= t.n_rows) return p;
  const int b = row_seq(t, row, lane);
  if (b < 0) return p;
  p.in_seq = true;
  const int64_t x = (int64_t)t.pos[b] + (row - seq_first(t, b));
  p.page = page_of(t, b, x);
  p.at = p.page < 0 ? 0 : (int)((uint32_t)x % (uint32_t)t.page_size);
  return p;
}

// 8 bf16 values in a uint4 to fp32.
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo(r[i]);
    x[2 * i + 1] = bf16hi(r[i]);
  }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(ROW_WARPS * 32) append_kernel(RowArgs a) {
  constexpr int LANES = D / 8, PER = 32 / LANES;   // lanes of a head, heads per pass
  constexpr int U = 4;                              // passes whose loads are in flight together
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, side = blockIdx.y;
  const int row = blockIdx.x * ROW_WARPS + (threadIdx.x >> 5);
  if (row >= a.t.n_rows) return;
  const int sub = lane / LANES, l = lane % LANES;
  const uint16_t* src = a.src[side] + row * a.ld[side];
  uint4 w[U];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * PER + sub;
      w[u] = h < a.n_heads_kv ? ldg_cg_v4(src + h * D + l * 8) : make_uint4(0, 0, 0, 0);
    }
  };
  load(0);   // on its way while the row's place is looked up
  const Place p = find_place(a.t, row, lane);
  if (p.page < 0) return;
  for (int h0 = 0; h0 < a.n_heads_kv; h0 += U * PER) {
    if (h0) load(h0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * PER + sub;
      const bool ok = h < a.n_heads_kv;
      const int64_t r = pool_row(a.t, a.layer, a.n_heads_kv, p.page, ok ? h : 0, p.at);
      if constexpr (!Q8) {
        if (ok) *(reinterpret_cast<uint4*>(a.pool[side]) + r * LANES + l) = w[u];
      } else {
        float x[8], big = 0.f;
        unpack8(w[u], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) big = max_nan(big, fabsf(x[i]));
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) big = max_nan(big, __shfl_xor_sync(~0u, big, o));
        float s = 1.f, t = 0.f;
        if (!(big < INFINITY)) {
          s = __int_as_float(0x7fc00000);   // NaN or infinity somewhere in the row
        } else if (big >= 0x1p-100f) {
          s = __fdiv_rn(big, 127.f);
          t = __fdiv_rn(127.f, big);
        }
        uint32_t c[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)   // |x t| <= 127 (1 + 2^-22): the code needs no clamp
          c[i >> 2] |= (uint32_t)(t == 0.f ? 128 : 128 + __float2int_rn(__fmul_rn(x[i], t)))
                       << (8 * (i & 3));
        if (ok) {
          *(reinterpret_cast<uint2*>(a.pool[side]) + r * LANES + l) = make_uint2(c[0], c[1]);
          if (l == 0) a.scale[side][r] = s;
        }
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(ROW_WARPS * 32) read_kernel(RowArgs a) {
  constexpr int LANES = D / 8, PER = 32 / LANES, U = 4;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, side = blockIdx.y;
  const Place p = find_place(a.t, blockIdx.x * ROW_WARPS + (threadIdx.x >> 5), lane);
  if (!p.in_seq) return;
  const int sub = lane / LANES, l = lane % LANES;
  uint4* dst = reinterpret_cast<uint4*>(a.dst[side]) + (int64_t)p.row * a.n_heads_kv * LANES;
  const uint8_t* pool = reinterpret_cast<const uint8_t*>(a.pool[side]);
  for (int h0 = 0; h0 < a.n_heads_kv; h0 += U * PER) {
    uint2 w[U];
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * PER + sub;
      w[u] = make_uint2(0x80808080u, 0x80808080u);
      s[u] = 0.f;
      if (p.page >= 0 && h < a.n_heads_kv) {
        const int64_t r = pool_row(a.t, a.layer, a.n_heads_kv, p.page, h, p.at);
        w[u] = __ldcg(reinterpret_cast<const uint2*>(pool) + r * LANES + l);
        s[u] = __ldcg(a.scale[side] + r);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * PER + sub;
      if (h >= a.n_heads_kv) continue;
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t word = (i < 2 ? w[u].x : w[u].y) >> (16 * (i & 1));
        o[i] = pack_bf16x2((float)((int)(word & 255) - 128) * s[u],
                           (float)((int)((word >> 8) & 255) - 128) * s[u]);
      }
      dst[h * LANES + l] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

dim3 row_grid(const SeqTable& t) { return dim3((unsigned)cdiv(t.n_rows, ROW_WARPS), 2); }

template <bool Q8, class Cache>
int32_t append(const sub_bf16* K, int64_t ldk, const sub_bf16* V, int64_t ldv, const Cache* kv,
               int32_t layer, const sub_batch* batch, RowArgs a, void* stream) {
  SUB_TRY(make_seq_table(kv, layer, batch, &a.t));
  if (a.t.n_rows == 0) return SUB_OK;
  const int64_t width = (int64_t)kv->n_heads_kv * kv->head_dim;
  SUB_CHECK_ARG(K && V, "null pointer");
  SUB_CHECK_ARG(aligned16(K) && aligned16(V) && ldk % 8 == 0 && ldv % 8 == 0,
                "rows must be 16-byte aligned");
  SUB_CHECK_ARG(ldk >= width && ldv >= width, "row stride below n_heads_kv * head_dim");
  a.layer = layer;
  a.n_heads_kv = kv->n_heads_kv;
  a.src[0] = K;
  a.src[1] = V;
  a.ld[0] = ldk;
  a.ld[1] = ldv;
  a.pool[0] = kv->k;
  a.pool[1] = kv->v;
  auto k = kv->head_dim == 128 ? append_kernel<128, Q8> : append_kernel<64, Q8>;
  SUB_CUDA_TRY(launch_k(k, row_grid(a.t), dim3(ROW_WARPS * 32), 0, as_stream(stream), a));
  return SUB_OK;
}

}  // namespace
}  // namespace sub

using namespace sub;

extern "C" int32_t sub_kv_append(const sub_bf16* K, int64_t ldk, const sub_bf16* V, int64_t ldv,
                                 const sub_kv_cache* kv, int32_t layer, const sub_batch* batch,
                                 void* stream) {
  return append<false>(K, ldk, V, ldv, kv, layer, batch, RowArgs{}, stream);
}

extern "C" int32_t sub_kv8_append(const sub_bf16* K, int64_t ldk, const sub_bf16* V, int64_t ldv,
                                  const sub_kv8_cache* kv, int32_t layer, const sub_batch* batch,
                                  void* stream) {
  SUB_TRY(check_scales(kv));
  RowArgs a{};
  a.scale[0] = kv->k_scale;
  a.scale[1] = kv->v_scale;
  return append<true>(K, ldk, V, ldv, kv, layer, batch, a, stream);
}

extern "C" int32_t sub_kv8_read(const sub_kv8_cache* kv, int32_t layer, const sub_batch* batch,
                                sub_bf16* K, sub_bf16* V, void* stream) {
  SUB_TRY(check_scales(kv));
  RowArgs a{};
  SUB_TRY(make_seq_table(kv, layer, batch, &a.t));
  if (a.t.n_rows == 0) return SUB_OK;
  SUB_CHECK_ARG(K && V, "null pointer");
  SUB_CHECK_ARG(aligned16(K) && aligned16(V), "rows must be 16-byte aligned");
  a.layer = layer;
  a.n_heads_kv = kv->n_heads_kv;
  a.pool[0] = kv->k;
  a.pool[1] = kv->v;
  a.scale[0] = kv->k_scale;
  a.scale[1] = kv->v_scale;
  a.dst[0] = K;
  a.dst[1] = V;
  auto k = kv->head_dim == 128 ? read_kernel<128> : read_kernel<64>;
  SUB_CUDA_TRY(launch_k(k, row_grid(a.t), dim3(ROW_WARPS * 32), 0, as_stream(stream), a));
  return SUB_OK;
}
