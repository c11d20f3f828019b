// Attention of a batch's new rows over a paged cache (see chunk_attn.cu).
#pragma once
#include <cuda.h>
#include "batch.cuh"

namespace sub {

// Division by a number that the host knows: n / d for 0 <= n < 2^31 is the high
// word of n * ceil(2^(31 + s) / d), shifted, with 2^s >= d.  (The error of the
// reciprocal, below 2^-(31 + s), stays below 1 / d even times 2^31.)  A division
// instruction sequence costs some 100 cycles, a dozen of them before a CTA's first load.
struct FastDiv {
  uint32_t d, mul, shift;
  __device__ __forceinline__ int quot(int n) const {
    return d == 1 ? n : (int)(__umulhi((uint32_t)n, mul) >> shift);
  }
};
inline FastDiv make_fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  if (d == 1) return {1, 0, 0};
  return {d, (uint32_t)(((1ull << (31 + s)) + d - 1) / d), s - 1};
}

struct ChunkArgs {
  SeqTable t;
  const uint16_t* Q;     // [n_rows, Hq, D] bf16, rows ldq elements apart
  int64_t ldq;
  uint16_t* O;           // [n_rows, Hq, D] bf16
  const void* k;         // pools: bf16, or 8-bit codes
  const void* v;
  const float* ks;       // scales of the codes
  const float* vs;
  int layer, n_layers, n_heads_q, n_heads_kv, group;   // group = Hq / Hkv
  FastDiv by_group, by_page;
  float sl2;             // softmax scale * log2(e): scores in base 2
  // partial results of units cut between CTAs: two per CTA
  float* part_o;         // [2 n_ctas][rows][D], relative to the maxima of
  float2* part_ml;       // [2 n_ctas][rows] (largest score, sum)
  struct ChunkCut* cuts; // [n_ctas]
};

// The unit of work (below) that is cut first at the end of a CTA's part, for the
// kernel that joins its pieces: written by each CTA, pieces 0 where none is.
struct __align__(16) ChunkCut {
  int row0, rows, tile, head;   // as in ChunkUnit
  int pieces, first;            // the first piece's slot; piece i > 0 of CTA x lies in slot 2 (x + i)
  int pad[2];
};

// Whether CTA part's entry names pieces, rows and a head that there are: what the join goes
// by lies in memory that only kernels which ran to their end have written.
__host__ __device__ inline bool cut_stands(const ChunkCut& c, int part, int n_ctas, int n_rows,
                                           int n_heads_kv, int group, int tile_rows) {
  // (a negative value is a large one; rows * group < 2^31, tile_rows is a power of two)
  const uint32_t row0 = c.row0, rows = c.rows, all = n_rows;
  return ((uint32_t)c.pieces - 2u < (uint32_t)(n_ctas - part - 1)) &
         ((uint32_t)c.first - 2u * part < 2u) & (row0 <= all) & (rows - 1u < all - row0) &
         ((uint32_t)c.head < (uint32_t)n_heads_kv) &
         ((uint32_t)c.tile <= (rows * group - 1u) / (uint32_t)tile_rows);
}

// Quotients of line positions, nearly always of 32 bits.  (The compiler's 64-bit
// division takes a few hundred cycles and instructions; this one's rare case is slow
// but small.)
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  uint64_t q = 0, r = 0;
#pragma unroll 1
  for (int i = 62; i >= 0; --i) {
    r = r << 1 | ((uint64_t)a >> i & 1);
    q <<= 1;
    if (r >= (uint64_t)b) {
      r -= b;
      q |= 1;
    }
  }
  return (int64_t)q;
}

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// Codes in two bytes of w as fp16 code - 128.
__device__ __forceinline__ uint32_t codes2(uint32_t w, uint32_t sel) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(w, 0x64646464u, sel)), "r"(0x64806480u));
  return r;
}

// Last key that row q of a sequence reads, of n_keys.  (pos may be anything.)
__device__ __forceinline__ int last_key(int pos, int q, int n_keys) {
  return (int)min((int64_t)pos + q, (int64_t)n_keys - 1);
}

// ---------------------------------------------------------------- work plan --
// A unit of work is one tile of RT rows -- (row, head in group) pairs of one
// KV head of one sequence -- over all the keys its last row reads, in blocks of
// KB keys.  All units' blocks, sequence by sequence, KV head by KV head, tile by
// tile, form one line that the CTAs share evenly, so that any mix of lengths
// fills the GPU; a unit cut between CTAs is joined afterwards from their
// partial results, in order.  Every CTA works its part out by itself from
// the lengths on the device: the place of its first unit from running sums over the
// sequences, the others one after the other.
struct ChunkUnit {
  int b, head, tile;      // sequence, KV head, tile
  int row0, rows, pos;    // the sequence's first row, its rows, position of the first
  int n_keys, n_blocks;   // of this tile
  int64_t begin;          // its first block on the line
};

template <int RT, int KB>
struct ChunkPlan {
  const ChunkArgs& a;
  __device__ explicit ChunkPlan(const ChunkArgs& a_) : a(a_) {}

  // rows of one head-group of a sequence, tiles of them
  __device__ int tiles(int rows) const { return (rows * a.group + RT - 1) / RT; }
  // keys that tile j of a sequence (rows new rows from position pos on) reads
  __device__ int keys(int pos, int rows, int j) const {
    const int last = min(rows, a.by_group.quot(j * RT + RT - 1) + 1);
    return (int)max((int64_t)0, min((int64_t)pos + last, a.t.capacity));
  }
  __device__ int blocks(int pos, int rows, int j) const {
    return max(1, (keys(pos, rows, j) + KB - 1) / KB);   // a tile without keys still writes zeros
  }
  __device__ void load(ChunkUnit& u) const {
    u.row0 = seq_first(a.t, u.b);
    u.rows = seq_rows(a.t, u.b);
    u.pos = a.t.pos[u.b];
  }
  __device__ void measure(ChunkUnit& u) const {
    u.n_keys = keys(u.pos, u.rows, u.tile);
    u.n_blocks = max(1, (u.n_keys + KB - 1) / KB);
  }

  // pre[b] = blocks of all sequences before b (all KV heads), pre[n_seqs] = all; by NT
  // threads.  A warp takes a sequence, its lanes the tiles.
  template <int NT>
  __device__ void scan(int64_t* pre) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = a.t.n_seqs;
    for (int b = warp; b < n; b += NT / 32) {
      const int rows = seq_rows(a.t, b), pos = a.t.pos[b], nt = tiles(rows);
      int64_t s = 0;
      for (int j = lane; j < nt; j += 32) s += blocks(pos, rows, j);
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
      if (lane == 0) pre[b + 1] = s * a.n_heads_kv;
    }
    __syncthreads();
    if (warp == 0) {   // running sums, 32 sequences at a time
      int64_t at = 0;
      if (lane == 0) pre[0] = 0;
      for (int b0 = 0; b0 < n; b0 += 32) {
        int64_t v = b0 + lane < n ? pre[b0 + lane + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t up = __shfl_up_sync(~0u, v, o);
          if (lane >= o) v += up;
        }
        if (b0 + lane < n) pre[b0 + lane + 1] = at + v;
        at += __shfl_sync(~0u, v, 31);
      }
    }
    __syncthreads();
  }

  // the unit that block `at` (< pre[n_seqs]) of the line belongs to; by a whole warp
  __device__ ChunkUnit find(const int64_t* pre, int64_t at) const {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = a.t.n_seqs - 1;   // last sequence that begins at or before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= at) lo = mid;
      else hi = mid - 1;
    }
    ChunkUnit u;
    u.b = lo;
    load(u);
    const int64_t per_head = quot(pre[lo + 1] - pre[lo], a.n_heads_kv);
    u.head = (int)quot(at - pre[lo], per_head);
    u.begin = pre[lo] + u.head * per_head;
    const int nt = tiles(u.rows);
    for (int j0 = 0;; j0 += 32) {   // 32 tiles at a time
      const int v = j0 + lane < nt ? blocks(u.pos, u.rows, j0 + lane) : 0;
      int64_t run = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(~0u, run, o);
        if (lane >= o) run += up;
      }
      const unsigned over = __ballot_sync(~0u, at - u.begin < run);
      if (over || j0 + 32 >= nt) {
        const int l = over ? __ffs(over) - 1 : 0;
        u.tile = j0 + l;
        u.begin += __shfl_sync(~0u, run - v, l);
        break;
      }
      u.begin += __shfl_sync(~0u, run, 31);
    }
    measure(u);
    return u;
  }

  // the unit after u (past the last one: undefined, but harmless)
  __device__ void next(ChunkUnit& u) const {
    u.begin += u.n_blocks;
    if (++u.tile >= tiles(u.rows)) {
      u.tile = 0;
      if (++u.head == a.n_heads_kv) {
        u.head = 0;
        do {
          if (++u.b >= a.t.n_seqs) return;
          load(u);
        } while (u.rows == 0);
      }
    }
    measure(u);
  }
};

// Blocks per CTA of a line of `total`, at least `least`.
__device__ __forceinline__ int64_t blocks_per_cta(int64_t total, int n_ctas, int least) {
  const int64_t per = quot(total + n_ctas - 1, n_ctas);
  return per < least ? least : per;
}
// A CTA's entry in the list of cuts, from its last piece (blocks [.., kb1) of u;
// the CTA's part of the line begins at lo).
__device__ __forceinline__ ChunkCut make_cut(const ChunkUnit& u, int kb1, int64_t lo, int64_t per) {
  ChunkCut c{u.row0, u.rows, u.tile, u.head, 0, 0, {0, 0}};
  if (kb1 < u.n_blocks && u.begin >= lo) {
    c.pieces = (int)(quot(u.begin + u.n_blocks - 1, per) - blockIdx.x) + 1;
    c.first = 2 * blockIdx.x + (u.begin == lo ? 0 : 1);
  }
  return c;
}

// The kernel for many rows per sequence (chunk_attn_tc.cu): its tiles, and the
// fewest blocks a CTA takes.
constexpr int CHUNK_TC_ROWS = 256, CHUNK_TC_KEYS = 128, CHUNK_TC_LEAST = 2;
bool chunk_tc_fits(int64_t pool_rows);   // rows of head_dim values in a pool
int32_t launch_chunk_tc(const ChunkArgs& a, bool q8, int head_dim, int64_t pool_rows, int n_ctas,
                        cudaStream_t st);
int32_t chunk_tc_timeouts(unsigned int* out);
// Waits that ran out in either kernel.
int32_t chunk_attn_timeouts(unsigned int* out);
// Tensor map of a pool by (page and head, place, column), in boxes of 16 places.
bool chunk_page_map(CUtensorMap* m, const void* pool, const SeqTable& t, int64_t heads, int d, bool codes);

}  // namespace sub
