// Rows on their way into a paged cache: places of a batch's rows, and the 8-bit
// cache's quantiser (see kv_rows.cu).
#pragma once
#include "batch.cuh"

namespace sub {

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Row of this warp, its sequence and the page of its position.
struct Place {
  int row, page, at;
  bool in_seq;
  int64_t pos;   // its position, if it belongs to a sequence
};
__device__ __forceinline__ Place find_place(const SeqTable& t, int row, int lane) {
  Place p{row, -1, 0, false, 0};
  if (row >= t.n_rows) return p;
  const int b = row_seq(t, row, lane);
  if (b < 0) return p;
  p.in_seq = true;
  p.pos = (int64_t)t.pos[b] + (row - seq_first(t, b));
  p.page = page_of(t, b, p.pos);
  p.at = p.page < 0 ? 0 : (int)((uint32_t)p.pos % (uint32_t)t.page_size);
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

// Scale of a row whose largest value is big, and what its values are multiplied by.
__device__ __forceinline__ void row_scale(float big, float& s, float& t) {
  s = 1.f;
  t = 0.f;
  if (!(big < INFINITY)) {
    s = __int_as_float(0x7fc00000);   // NaN or infinity somewhere in the row
  } else if (big >= 0x1p-100f) {
    s = __fdiv_rn(big, 127.f);
    t = __fdiv_rn(127.f, big);
  }
}
// |x t| <= 127 (1 + 2^-22): the code needs no clamp
__device__ __forceinline__ uint2 codes8(const float* x, float t) {
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i >> 2] |= (uint32_t)(t == 0.f ? 128 : 128 + __float2int_rn(__fmul_rn(x[i], t))) << (8 * (i & 3));
  return make_uint2(c[0], c[1]);
}

}  // namespace sub
