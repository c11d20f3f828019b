// Attention of a batch's new rows over a paged cache (see chunk_attn.cu).
#pragma once
#include "batch.cuh"

namespace sub {

struct ChunkArgs {
  SeqTable t;
  const uint16_t* Q;     // [n_rows, Hq, D] bf16, rows ldq elements apart
  int64_t ldq;
  uint16_t* O;           // [n_rows, Hq, D] bf16
  const void* k;         // pools: bf16, or 8-bit codes
  const void* v;
  const float* ks;       // scales of the codes
  const float* vs;
  int layer, n_heads_q, n_heads_kv, group;   // group = Hq / Hkv
  float sl2;             // softmax scale * log2(e): scores in base 2
  // partial results of key ranges cut between CTAs: two per CTA
  float* part_o;         // [2 n_ctas][rows][D], relative to the maxima of
  float2* part_ml;       // [2 n_ctas][rows] (largest score, sum)
  struct ChunkCut* cuts; // [n_ctas]
};

// The unit of work (below) that is cut first at the end of a CTA's part, for the
// kernel that joins its pieces: written by each CTA, pieces 0 where none is.
struct __align__(16) ChunkCut {
  int row0, rows, tile, head;   // as in ChunkPlan::Unit
  int pieces, first;            // the first piece's slot; piece i > 0 of CTA x lies in slot 2 (x + i)
  int pad[2];
};

// Quotients of line positions, nearly always of 32 bits (a 64-bit division
// takes a few hundred cycles, in every CTA before its first load).
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// ---------------------------------------------------------------- work plan --
// A unit of work is one tile of RT rows -- (row, head in group) pairs of one
// KV head of one sequence -- over all the keys its last row reads, in blocks of
// KB keys.  All units' blocks, sequence by sequence, KV head by KV head, tile by
// tile, form one line that the CTAs share evenly, so that any mix of lengths
// fills the GPU; a unit cut between CTAs is joined afterwards from their
// partial results, in order.  Every CTA works the plan out by itself from
// the lengths on the device.
template <int RT, int KB>
struct ChunkPlan {
  const SeqTable& t;
  int group, heads;
  __device__ ChunkPlan(const SeqTable& t_, int g, int h) : t(t_), group(g), heads(h) {}

  // rows of one head-group of a sequence, tiles of them
  __device__ int tiles(int rows) const { return (rows * group + RT - 1) / RT; }
  // keys that tile j of sequence b (rows new rows from position pos on) reads
  __device__ int keys(int pos, int rows, int j) const {
    const int last = min(rows, (j * RT + RT - 1) / group + 1);
    return (int)max((int64_t)0, min((int64_t)pos + last, t.capacity));
  }
  __device__ int blocks(int pos, int rows, int j) const {
    return max(1, (keys(pos, rows, j) + KB - 1) / KB);   // a tile without keys still writes zeros
  }
  __device__ int64_t seq_blocks(int b) const {   // of one KV head
    const int rows = seq_rows(t, b), pos = t.pos[b], n = tiles(rows);
    int64_t s = 0;
    for (int j = 0; j < n; ++j) s += blocks(pos, rows, j);
    return s;
  }

  // pre[b] = blocks of all sequences before b (all KV heads), pre[n_seqs] = all
  template <int NT>
  __device__ void scan(int64_t* pre, int64_t* warp_sums) const {
    constexpr int PER = (SUB_MAX_SEQS + NT - 1) / NT;
    const int per = (t.n_seqs + NT - 1) / NT, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t mine[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = threadIdx.x * per + i;
      mine[i] = i < per && b < t.n_seqs ? seq_blocks(b) * heads : 0;
      sum += mine[i];
    }
    int64_t run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(~0u, run, o);
      if (lane >= o) run += up;
    }
    if (lane == 31) warp_sums[warp] = run;
    __syncthreads();
    int64_t at = run - sum;
    for (int w = 0; w < warp; ++w) at += warp_sums[w];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = threadIdx.x * per + i;
      if (i < per && b < t.n_seqs) {
        pre[b] = at;
        at += mine[i];
        if (b == t.n_seqs - 1) pre[t.n_seqs] = at;
      }
    }
    __syncthreads();
  }

  struct Unit {
    int b, head, tile;      // sequence, KV head, tile
    int row0, rows, pos;    // the sequence's first row, its rows, position of the first
    int n_keys, n_blocks;   // of this tile
    int64_t begin;          // its first block on the line
  };
  // the unit that block `at` of the line belongs to
  __device__ Unit find(const int64_t* pre, int64_t at) const {
    int lo = 0, hi = t.n_seqs - 1;   // last sequence that begins at or before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= at) lo = mid;
      else hi = mid - 1;
    }
    Unit u;
    u.b = lo;
    u.row0 = seq_first(t, lo);
    u.rows = seq_rows(t, lo);
    u.pos = t.pos[lo];
    const int64_t per_head = quot(pre[lo + 1] - pre[lo], heads);
    u.head = (int)quot(at - pre[lo], per_head);
    u.begin = pre[lo] + u.head * per_head;
    u.tile = 0;
    u.n_blocks = blocks(u.pos, u.rows, 0);
    while (at - u.begin >= u.n_blocks) {
      u.begin += u.n_blocks;
      u.n_blocks = blocks(u.pos, u.rows, ++u.tile);
    }
    u.n_keys = keys(u.pos, u.rows, u.tile);
    return u;
  }
};

// Blocks per CTA of a line of `total`, at least `least`.
__device__ __forceinline__ int64_t blocks_per_cta(int64_t total, int n_ctas, int least) {
  const int64_t per = quot(total + n_ctas - 1, n_ctas);
  return per < least ? least : per;
}
// A CTA's entry in the list of cuts, from its last piece (blocks [.., kb1) of u;
// the CTA's part of the line begins at lo).
template <class Unit>
__device__ __forceinline__ ChunkCut make_cut(const Unit& u, int kb1, int64_t lo, int64_t per) {
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

}  // namespace sub
