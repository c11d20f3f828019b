// Attention of new rows over a paged cache, few rows per sequence: the decode
// step (one row per sequence) and short chunks of drafted tokens.
//
// o_i = sum_j e_ij v_j / sum_j e_ij, e_ij = 2^(s_ij - m_i), s_ij = q_i . k_j *
// scale * log2(e), over the keys at positions 0 .. pos + i, in one pass with a
// running maximum m_i.  The Hq / Hkv query heads of a KV head are rows of the
// same tile, so a key is read once for all of them.
//
// Bound by HBM: a row tile of 16 does 16 flops per byte of a bf16 cache,
// mma.sync covers that many times over, and what counts is bytes in flight.  So
// each of eight warps streams blocks of 16 or 32 keys (8 KB; 4 KB of codes of 64
// columns) on its own, through a private ring of three stages that bulk tensor copies
// fill, one lane per 2 KB box, over all its units of work one after the other.  (The same
// loop with 16-byte cp.async copies, sixteen per lane and block, ran at 5.1 TB/s
// on 32 sequences of up to 16384 keys and left a quarter of the SMs a fifth slower
// than the rest; the copies alone now take 203 us, 6.7 TB/s, and the kernel
// 215.)  No barrier in the loop, no ldmatrix: a dot product may take its terms
// in any order, if Q is laid out the same way, so lane (g, tig) reads, of key g of an
// 8-key group, the 16-byte chunks 2 tig, 2 tig + 1 of each 128 bytes, and of V, for
// its four keys of a 16-key step, the chunk that makes its B fragments for the n tiles of
// eight chunk-wise permuted columns; the boxes' swizzle spreads both over all banks.
//
// At most 8 rows are a tile of their own, with both products turned over (S^T = K Q^T,
// O^T = V^T P^T): half the matrix instructions, exponentials and accumulators of 16
// rows.  The turned weights are already the next product's operand but for an
// 8x8 transposition.
//
// Measured, 40 or 32 query heads of 8 KV heads of 128: 32 sequences of up to 16384 keys
// 215 us (1.37 GB, 6.35 TB/s); codes, 2 of up to 65001 44 us (4.8 TB/s); 128 of up to
// 2000 keys 116 us (5.7 TB/s), codes 96 (3.5); 1 sequence of 512 keys of 2 heads of 64
// 7.5 us, two launches and their dependent reads.  Over codes the conversions and, on
// short caches, the change of units show: the same loads without the products took four
// fifths of the time of the 128 sequences.  (Twelve warps with two stages each gained 4%
// there and cost the short call a quarter; Q read a unit ahead gained nothing.)
//
// 8-bit codes c stand for (c - 128) * scale, and both products take c - 128 in
// fp16, exactly: the bytes 0x64, c are 1024 + c, a byte permute and a subtraction
// for two of them.  The scale of k_j multiplies the score, and the scale of v_j
// goes into e_ij before it is rounded to fp16.
// The running maximum includes log2 of the largest vscale that the row reads, minus 15, so
// that what is rounded reaches 2^15 at most, and fp16's smallest step, 2^-24, is
// 2^-39 of the largest; the sum takes the unscaled e_ij, in fp32, relative to the
// same maximum (log2(vscale) counts as at least -80, which keeps it in range).  Q
// enters in fp16 scaled by a power of two of its row's largest value: bf16 has three
// bits fewer, so only values below 2^-15 of the largest lose any.  With a bf16
// cache P = hi + lo, two bf16 products, keeps it to 2^-17; in fp16 one product keeps
// 2^-12.
//
// A key that a row must not read can still hold anything, and so can a box past the
// last key or of a page that is not there.  Its score is replaced, and where its
// value is infinite or NaN (bf16 only, and only in blocks that not all rows read
// to the end), the block's products with V are formed one by one without the keys of
// weight zero.
#include <algorithm>
#include <type_traits>
#include "chunk_attn.cuh"
#include "tma.cuh"

namespace sub {
namespace {

using namespace tmah;

constexpr int WIDE = 16, NARROW = 8;   // rows of a tile
constexpr int WARPS = 8;
constexpr int NT = WARPS * 32;
constexpr int STAGES = 3;

__device__ unsigned int g_decode_timeouts;   // waits that ran out (never expected)

struct PageMaps {
  CUtensorMap k, v;   // [pages and heads, page_size, D], boxes of 16 keys x 128 (or 64) bytes
};
// bytes: a multiple of 16, both addresses on 16-byte boundaries
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float log2_fast(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <int D, bool Q8>
struct Ring {
  static constexpr int KB = !Q8 && D == 128 ? 16 : 32;   // keys per block of a warp
  static constexpr int SUBS = KB / 16;                   // 16-key steps; a step lies in one page
  static constexpr int ROW = D * (Q8 ? 1 : 2);           // bytes of a row
  static constexpr int LINE = ROW < 128 ? ROW : 128;     // a box is 16 lines: 16 keys' columns
  static constexpr int BOX = 16 * LINE, H = ROW / LINE;  // boxes side by side
  static constexpr int KI = ROW / 64;                    // 16-byte chunks of a key per lane
  static constexpr int K_BYTES = KB * ROW;
  static constexpr int STAGE = 2 * K_BYTES;
  static constexpr int BYTES = STAGES * STAGE;           // of one warp
  static constexpr int SCALES = Q8 ? 2 * KB * 4 : 0;     // of one stage
  static constexpr int OPS = 2 * H + (Q8 ? 2 : 0);       // copies of a 16-key step
};

template <int D, bool Q8>
constexpr int decode_smem() {
  static_assert(Ring<D, Q8>::STAGE >= WIDE * D * 4, "a stage holds a warp's partial result");
  static_assert(Ring<D, Q8>::SUBS * Ring<D, Q8>::OPS <= 32, "a lane per copy");
  return 1024 + WARPS * (Ring<D, Q8>::BYTES + STAGES * Ring<D, Q8>::SCALES);
}

// The 8x8 matrix of 16-bit values whose row g the lanes (g, .) hold, turned over.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A barrier of two warps.
__device__ __forceinline__ void bar_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id) {
  asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory");
}

// ------------------------------------------------------------------ kernel --
template <int D, bool Q8, int RT>
__global__ void __launch_bounds__(NT, 1)
chunk_attn_kernel(const __grid_constant__ PageMaps maps, const __grid_constant__ ChunkArgs a) {
  using R = Ring<D, Q8>;
  constexpr int KS = D / 16, KB = R::KB, SUBS = R::SUBS;
  // Scores in accumulators of 8 keys x 16 rows, or turned over, of 16 keys x 8 rows;
  // results of 8 columns x 16 rows, or 16 columns x 8 rows
  constexpr bool TURNED = RT == NARROW;
  constexpr int TILES = TURNED ? SUBS : KB / 8, ON = TURNED ? D / 16 : D / 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023u);   // as the boxes' swizzle wants it
  __shared__ int64_t s_pre[SUB_MAX_SEQS + 1];
  __shared__ float4 s_ml[WARPS][32];   // maxima and sums of the warps' partial results, by lane
  __shared__ int s_at[WARPS];          // the stages that these lie in
  __shared__ __align__(8) uint64_t s_bar[WARPS][STAGES];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < WARPS * STAGES) mbar_init(smem_u32(&s_bar[0][0] + tid), 1);
  if (tid == 0) {
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  pdl_wait();
  pdl_trigger();
  const int g = lane >> 2, tig = lane & 3;
  const int G = a.group, ps = a.t.page_size;
  const ChunkPlan<RT, KB> plan(a);
  plan.template scan<NT>(s_pre);
  const int64_t total = s_pre[a.t.n_seqs];
  const int64_t per = blocks_per_cta(total, gridDim.x, WARPS);
  const uint8_t* const ring = smem + warp * R::BYTES;
  const float* const scales =
      reinterpret_cast<const float*>(smem + WARPS * R::BYTES + warp * (STAGES * R::SCALES));
  const uint32_t ring_s = smem_u32(ring), scales_s = smem_u32(scales), bar_s = smem_u32(s_bar[warp]);
  // Where a lane's operands lie in a box, 16-byte chunks swizzled by the line: K of key
  // g, its chunks 2 tig, 2 tig + 1 (of four: tig), V of keys 2 tig, 2 tig + 1, its piece g
  int k_at[2], v_at[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = 2 * tig + x;
    k_at[x] = R::LINE == 128 ? g * 128 + ((r ^ g) * 16) : g * 64 + ((tig ^ (g >> 1)) * 16);
    v_at[x] = R::LINE == 128 ? r * 128 + ((g ^ r) * 16)
                             : r * 64 + (((g >> 1) ^ tig) * 16) + (g & 1) * 8;
  }
  const int64_t line_lo = blockIdx.x * per, line_hi = min(total, line_lo + per);
  if (line_lo >= line_hi) {
    if (tid == 0) a.cuts[blockIdx.x].pieces = 0;
    return;
  }
  ChunkUnit u = plan.find(s_pre, line_lo);

  // ---- the loads: the warp's blocks of all its units, one after the other ----
  // unit f, of which the warp reads blocks f0 + mine + i * WARPS, i < fn.  The last warps
  // come first: the first ones join the results, and a remainder of the blocks
  // goes to those that do not.
  const int mine = WARPS - 1 - warp;
  ChunkUnit f = u;
  int f0, fn, fi;
  const int32_t* pages;
  int places, places2;
  // (page, head) of the warp's next 32 16-key steps (-1: no page), one looked up by
  // each lane, and of the 32 after them: a step's place is a shuffle away.
  auto look_up = [&](int step) {
    const int key = (f0 + mine + step / SUBS * WARPS) * KB + step % SUBS * 16;
    if (key >= f.n_keys || step >= fn * SUBS) return -1;
    const int page = pages[a.by_page.quot(key)];
    if ((unsigned)page >= (unsigned)a.t.n_pages) return -1;
    return (a.layer * a.t.n_pages + page) * a.n_heads_kv + f.head;
  };
  auto open = [&](int64_t at) {
    for (;;) {
      f0 = (int)(at - f.begin);
      const int f1 = (int)min((int64_t)f.n_blocks, line_hi - f.begin);
      fn = (f1 - f0 - mine + WARPS - 1) / WARPS;
      fi = 0;
      at = f.begin + f1;
      if (fn > 0 || at >= line_hi) break;
      plan.next(f);
    }
    pages = a.t.pages + (int64_t)f.b * a.t.width;
    places = look_up(lane);
    places2 = look_up(32 + lane);
  };
  uint32_t missing = 0;   // bits SUBS * stage + step: no page there
  uint32_t phase = 0;     // of the stages' barriers
  uint32_t coming = 0;    // stages with copies under way
  bool dead = false;      // a wait ran out: no more copies, no more waits
  const int my_step = min(lane / R::OPS, SUBS - 1), my_op = lane - my_step * R::OPS;   // op >= OPS: none
  auto feed = [&](int stage) {
    if (fi < fn && !dead) {
      if (fi > 0 && fi % (32 / SUBS) == 0) {
        places = places2;
        places2 = look_up(fi * SUBS + 32 + lane);
      }
      const int place = __shfl_sync(~0u, places, (fi * SUBS + my_step) & 31);
      const unsigned have = __ballot_sync(~0u, place >= 0);
      uint32_t gone = 0;
#pragma unroll
      for (int s = 0; s < SUBS; ++s) gone |= (~(have >> (s * R::OPS)) & 1u) << s;
      missing = (missing & ~(((1u << SUBS) - 1u) << (SUBS * stage))) | gone << (SUBS * stage);
      const uint32_t bar = bar_s + stage * 8;
      coming |= 1u << stage;
      if (lane == 0)
        mbar_expect_tx(bar, (SUBS - __popc(gone)) * (32 * R::ROW + (Q8 ? 128 : 0)));
      __syncwarp();
      if (place >= 0 && my_op < R::OPS) {
        const int key = (f0 + mine + fi * WARPS) * KB + my_step * 16;
        const int at = key - a.by_page.quot(key) * ps;
        if (my_op < 2 * R::H) {
          const int side = my_op / R::H, h = my_op % R::H;
          tma_load_3d(ring_s + stage * R::STAGE + side * R::K_BYTES + (my_step * R::H + h) * R::BOX,
                      side ? &maps.v : &maps.k, h * 64, at, place, bar);
        } else {   // 16 scales of K, 16 of V
          const int side = my_op - 2 * R::H;
          bulk_load(scales_s + stage * R::SCALES + (side * KB + my_step * 16) * 4,
                    (side ? a.vs : a.ks) + (int64_t)place * ps + at, 64, bar);
        }
      }
      if (++fi == fn) {
        const int64_t end = f.begin + min((int64_t)f.n_blocks, line_hi - f.begin);
        if (end < line_hi) {
          plan.next(f);
          open(end);
        }
      }
    }
  };
  open(line_lo);
#pragma unroll 1
  for (int i = 0; i < STAGES - 1; ++i) feed(i);

  int stage = 0;          // of the next block
  int owed = 0;           // the barrier after which the last partial result has been read
  for (int64_t at = line_lo; at < line_hi; plan.next(u)) {
    const int kb0 = (int)(at - u.begin);
    const int kb1 = (int)min((int64_t)u.n_blocks, line_hi - u.begin);
    const int n_mine = (kb1 - kb0 - mine + WARPS - 1) / WARPS;   // blocks kb0 + mine + i * WARPS

    // Element i of accumulator t: which of the lane's two rows, which of its two keys
    auto row_of = [](int i) { return TURNED ? i & 1 : i >> 1; };
    auto key_of = [](int i) { return TURNED ? i >> 1 : i & 1; };
    auto tile_row = [&](int h) { return TURNED ? 2 * tig + h : h * 8 + g; };
    auto block_key = [&](int t, int x) { return TURNED ? 16 * t + 8 * x + g : 8 * t + 2 * tig + x; };

    // ---- Q fragments (of rows g, g + 8, or as the other operand, of row g) ----
    uint32_t qf[KS][TURNED ? 2 : 4];
    float qs[2];    // factor of the row's scores
    int lim[2];     // keys 0 .. lim are read
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int q = a.by_group.quot(u.tile * RT + tile_row(h));
      lim[h] = q < u.rows ? last_key(u.pos, q, u.n_keys) : -1;
      qs[h] = a.sl2;
    }
#pragma unroll
    for (int h = 0; h < (TURNED ? 1 : 2); ++h) {
      const int r = u.tile * RT + h * 8 + g;
      const int q = a.by_group.quot(r);
      const bool ok = q < u.rows;
      const uint16_t* src = a.Q + (int64_t)(u.row0 + (ok ? q : 0)) * a.ldq +
                            (int64_t)(u.head * G + r - q * G) * D;
      uint4 w[KS / 2];
#pragma unroll
      for (int c = 0; c < KS / 2; ++c) {
        // the chunk that K's c-th (bf16, 8 values), (c / 2)-th (codes, 16) operands come from
        const int i = Q8 ? c >> 1 : c, chunk = R::KI == 1 ? tig : 8 * (i >> 1) + 2 * tig + (i & 1);
        const int d = Q8 ? chunk * 16 + (c & 1) * 8 : chunk * 8;
        w[c] = ok ? ldg_cg_v4(src + d) : make_uint4(0, 0, 0, 0);
      }
      // registers of row g: 0 and 2 of a row operand, 0 and 1 of a column operand
      if constexpr (!Q8) {
#pragma unroll
        for (int c = 0; c < KS / 2; ++c) {
          constexpr int UP = TURNED ? 1 : 2;
          qf[2 * c][h] = w[c].x;
          qf[2 * c][UP + h] = w[c].y;
          qf[2 * c + 1][h] = w[c].z;
          qf[2 * c + 1][UP + h] = w[c].w;
        }
      } else {
        // the row's largest value to [1, 2): an exponent in [-126, 126]
        float big = 0.f;
#pragma unroll
        for (int c = 0; c < KS / 2; ++c) {
          const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            big = fmaxf(big, fmaxf(fabsf(bf16lo(x[i])), fabsf(bf16hi(x[i]))));
        }
        big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
        big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
        const int e = min(126, max(-126, (int)(__float_as_uint(big) >> 23) - 127));
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        // (not 0: it meets the masked scores' -infinity)
        qs[h] = fmaxf(a.sl2 * __uint_as_float((uint32_t)(127 + e) << 23), 1e-37f);
#pragma unroll
        for (int c = 0; c < KS / 2; ++c) {
          const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            qf[2 * c + (i >> 1)][(i & 1) * (TURNED ? 1 : 2) + h] =
                pack_f16x2(bf16lo(x[i]) * down, bf16hi(x[i]) * down);
        }
      }
    }
    if constexpr (TURNED && Q8) {
      const float mine = qs[0];   // of row g
      qs[0] = __shfl_sync(~0u, mine, 8 * tig);
      qs[1] = __shfl_sync(~0u, mine, 8 * tig + 4);
    }
    const int lim_min = last_key(u.pos, a.by_group.quot(u.tile * RT), u.n_keys);   // of the tile's first row
    // largest value over the lanes that share their rows
    auto row_max = [](float x) {
#pragma unroll
      for (int d = TURNED ? 4 : 1; d < (TURNED ? 32 : 4); d *= 2) x = fmaxf(x, __shfl_xor_sync(~0u, x, d));
      return x;
    };

    float o[ON][4], mx[2], l[2];
    mx[0] = mx[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < ON; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    if (owed) {
      bar_sync(owed);
      fence_async();   // the copies to come follow the stores of the partial result
      __syncwarp();
    }
    owed = 0;
    for (int i = 0; i < n_mine; ++i) {
      feed(stage == 0 ? STAGES - 1 : stage - 1);   // the stage that was read last
      if (!dead) {
        if (__all_sync(~0u, mbar_wait_polls(bar_s + stage * 8, (phase >> stage) & 1u, 1u << 20))) {
          phase ^= 1u << stage;
          coming &= ~(1u << stage);
        } else {
          dead = true;
          if (lane == 0) atomicAdd(&g_decode_timeouts, 1u);
        }
      }
      const int key0 = (kb0 + mine + i * WARPS) * KB;
      const uint8_t* const st = ring + stage * R::STAGE;
      const uint32_t miss = (missing >> (SUBS * stage)) & ((1u << SUBS) - 1u);
      const bool edge = key0 + KB - 1 > lim_min || miss;

      // ---- S = Q K^T, or K Q^T ----
      float s[TILES][4];
#pragma unroll
      for (int t = 0; t < TILES; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
      // w[t]: the lane's chunk of key g of keys 8 t .. + 7
#pragma unroll
      for (int c = 0; c < R::KI; ++c) {   // (the tiles in turn: their sums do not wait for each other)
        uint32_t w[KB / 8][4];
#pragma unroll
        for (int t = 0; t < KB / 8; ++t) {
          const uint4 x = *reinterpret_cast<const uint4*>(
              st + ((t >> 1) * R::H + (c >> 1)) * R::BOX + (t & 1) * 8 * R::LINE + k_at[c & 1]);
          w[t][0] = x.x;
          w[t][1] = x.y;
          w[t][2] = x.z;
          w[t][3] = x.w;
        }
#pragma unroll
        for (int k = 0; k < (Q8 ? 4 : 2); ++k) {
          uint32_t b[KB / 8][2];   // 16 values' two operand registers
#pragma unroll
          for (int t = 0; t < KB / 8; ++t) {
            b[t][0] = Q8 ? codes2(w[t][k], 0x4140u) : w[t][2 * (k & 1)];
            b[t][1] = Q8 ? codes2(w[t][k], 0x4342u) : w[t][2 * (k & 1) + 1];
          }
          const auto& qk = qf[(Q8 ? 4 : 2) * c + k];
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            if constexpr (TURNED) {
              const uint32_t kf[4] = {b[2 * t][0], b[2 * t + 1][0], b[2 * t][1], b[2 * t + 1][1]};
              if constexpr (Q8) mma_f16(s[t], kf, qk[0], qk[1]);
              else mma_bf16_16816(s[t], kf, qk[0], qk[1]);
            } else {
              if constexpr (Q8) mma_f16(s[t], qk, b[t][0], b[t][1]);
              else mma_bf16_16816(s[t], qk, b[t][0], b[t][1]);
            }
          }
        }
      }

      // ---- weights ----
      float vsc[TILES][2], lv[2] = {0.f, 0.f};
      auto shift = [](float vmax) { return fmaxf(log2_fast(vmax), -80.f) - 15.f; };
      if constexpr (Q8) {
        const float* const sc = scales + stage * (R::SCALES / 4);
        float vmax = 0.f;
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          float ksc[2];
          if constexpr (TURNED) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              ksc[x] = sc[block_key(t, x)];
              vsc[t][x] = sc[KB + block_key(t, x)];
            }
          } else {
            const float2 kq = *reinterpret_cast<const float2*>(sc + block_key(t, 0));
            const float2 vq = *reinterpret_cast<const float2*>(sc + KB + block_key(t, 0));
            ksc[0] = kq.x;
            ksc[1] = kq.y;
            vsc[t][0] = vq.x;
            vsc[t][1] = vq.y;
          }
          vmax = fmaxf(vmax, fmaxf(vsc[t][0], vsc[t][1]));
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][e] *= ksc[key_of(e)];
        }
        lv[0] = lv[1] = shift(vmax);
      }
      if (edge) {
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int x = block_key(t, key_of(e));
            const bool gone = (miss >> (TURNED ? t : t >> 1)) & 1u;
            if (gone || key0 + x > lim[row_of(e)]) s[t][e] = -INFINITY;
          }
        if constexpr (Q8) {   // the scales of keys that a row does not read may be anything
          float vmax[2] = {0.f, 0.f};
#pragma unroll
          for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (s[t][e] != -INFINITY) vmax[row_of(e)] = fmaxf(vmax[row_of(e)], vsc[t][key_of(e)]);
          lv[0] = shift(vmax[0]);
          lv[1] = shift(vmax[1]);
        }
      }
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[row_of(e)] = fmaxf(top[row_of(e)], s[t][e]);
      top[0] = fmaf(top[0], qs[0], lv[0]);
      top[1] = fmaf(top[1], qs[1], lv[1]);
      if (__any_sync(~0u, top[0] > mx[0] || top[1] > mx[1])) {
        float corr[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float now = fmaxf(mx[h], row_max(top[h]));
          corr[h] = now == -INFINITY ? 1.f : exp2_fast(mx[h] - now);
          mx[h] = now;
          l[h] *= corr[h];
        }
#pragma unroll
        for (int n = 0; n < ON; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] *= corr[row_of(e)];
      }
      // a row without a key so far keeps -infinity: subtract 0 there
      const float ref[2] = {mx[0] == -INFINITY ? 0.f : mx[0],
                            mx[1] == -INFINITY ? 0.f : mx[1]};
      // P of the 16-key steps as operands (bf16: high and low part), and, turned over, as
      // they are held: [.. + 2 ..]
      uint32_t pf[SUBS][4], pl[SUBS][4];
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = exp2_fast(fmaf(s[t][e], qs[row_of(e)], -ref[row_of(e)]));
          l[row_of(e)] += p[e];
          if constexpr (Q8) {
            // a masked key's scale may be anything
            p[e] = edge && s[t][e] == -INFINITY ? 0.f : p[e] * vsc[t][key_of(e)];
          }
        }
        const int step = TURNED ? t : t >> 1, r0 = TURNED ? 2 : (t & 1) * 2;
        if constexpr (Q8) {
          pf[step][r0] = pack_f16x2(p[0], p[1]);
          pf[step][r0 + 1] = pack_f16x2(p[2], p[3]);
        } else {
          const uint32_t a01 = pack_bf16x2(p[0], p[1]), a23 = pack_bf16x2(p[2], p[3]);
          pf[step][r0] = a01;
          pf[step][r0 + 1] = a23;
          pl[step][r0] = pack_bf16x2(p[0] - bf16lo(a01), p[1] - bf16hi(a01));
          pl[step][r0 + 1] = pack_bf16x2(p[2] - bf16lo(a23), p[3] - bf16hi(a23));
        }
        if constexpr (TURNED) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            pf[step][x] = transposed(pf[step][2 + x]);
            if constexpr (!Q8) pl[step][x] = transposed(pl[step][2 + x]);
          }
        }
      }

      // ---- O += P V, or V^T P^T: n tile n, column g is column d(g, n) of the head ----
      // (turned over, two n tiles are one of 16 columns)
      const uint8_t* const sv = st + R::K_BYTES;
#pragma unroll
      for (int step = 0; step < SUBS; ++step) {
        if constexpr (!Q8) {
#pragma unroll
          for (int c = 0; c < R::H; ++c) {   // d(g, 8 c + j) = 64 c + 8 g + j
            uint32_t w[4][4];
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint4 x = *reinterpret_cast<const uint4*>(
                  sv + (step * R::H + c) * R::BOX + (kk >> 1) * 8 * R::LINE + v_at[kk & 1]);
              w[kk][0] = x.x;
              w[kk][1] = x.y;
              w[kk][2] = x.z;
              w[kk][3] = x.w;
            }
            bool odd = false;
            if (edge) {   // 0 * x is NaN for what is not finite
              uint32_t z = 0;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(z) : "r"(w[kk][j]), "r"(0u));
              odd = __any_sync(~0u, (z & 0x7fff7fffu) != 0);
            }
            if (!odd) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t b0 = __byte_perm(w[0][j], w[1][j], 0x5410u);
                const uint32_t b1 = __byte_perm(w[2][j], w[3][j], 0x5410u);
                const uint32_t d0 = __byte_perm(w[0][j], w[1][j], 0x7632u);
                const uint32_t d1 = __byte_perm(w[2][j], w[3][j], 0x7632u);
                if constexpr (TURNED) {
                  const uint32_t vf[4] = {b0, d0, b1, d1};
                  mma_bf16_16816(o[c * 4 + j], vf, pf[step][0], pf[step][1]);
                  mma_bf16_16816(o[c * 4 + j], vf, pl[step][0], pl[step][1]);
                } else {
                  mma_bf16_16816(o[c * 8 + 2 * j], pf[step], b0, b1);
                  mma_bf16_16816(o[c * 8 + 2 * j + 1], pf[step], d0, d1);
                  mma_bf16_16816(o[c * 8 + 2 * j], pl[step], b0, b1);
                  mma_bf16_16816(o[c * 8 + 2 * j + 1], pl[step], d0, d1);
                }
              }
            } else {   // element by element
#pragma unroll 1
              for (int key = 0; key < 16; ++key) {
                const int kt = (key & 7) >> 1, kk = (key >> 3) * 2 + (key & 1);   // its lanes, its piece
                float pr[2];
                if constexpr (TURNED) {
                  const int from = (key & 7) * 4 + tig;
                  const uint32_t hi = __shfl_sync(~0u, key & 8 ? pf[step][3] : pf[step][2], from);
                  const uint32_t lo = __shfl_sync(~0u, key & 8 ? pl[step][3] : pl[step][2], from);
                  pr[0] = bf16lo(hi) + bf16lo(lo);
                  pr[1] = bf16hi(hi) + bf16hi(lo);
                } else {
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const uint32_t hi =
                        __shfl_sync(~0u, key & 8 ? pf[step][2 + h] : pf[step][h], g * 4 + kt);
                    const uint32_t lo =
                        __shfl_sync(~0u, key & 8 ? pl[step][2 + h] : pl[step][h], g * 4 + kt);
                    pr[h] = key & 1 ? bf16hi(hi) + bf16hi(lo) : bf16lo(hi) + bf16lo(lo);
                  }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const uint32_t mine = kk == 0 ? w[0][j] : kk == 1 ? w[1][j] : kk == 2 ? w[2][j] : w[3][j];
#pragma unroll
                  for (int e = 0; e < (TURNED ? 1 : 2); ++e) {   // column g, or columns 2 tig + e
                    const uint32_t x = __shfl_sync(~0u, mine, (TURNED ? g : 2 * tig + e) * 4 + kt);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                      if (pr[h] == 0.f) continue;
                      if constexpr (TURNED) {
                        o[c * 4 + j][h] += pr[h] * bf16lo(x);
                        o[c * 4 + j][2 + h] += pr[h] * bf16hi(x);
                      } else {
                        o[c * 8 + 2 * j][2 * h + e] += pr[h] * bf16lo(x);
                        o[c * 8 + 2 * j + 1][2 * h + e] += pr[h] * bf16hi(x);
                      }
                    }
                  }
                }
              }
            }
          }
        } else {
          constexpr int WN = D / 32;   // d(g, n) = g * (D / 8) + n
          uint32_t w[4][WN];
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint8_t* const src = sv + step * R::BOX + (kk >> 1) * 8 * R::LINE + v_at[kk & 1];
            if constexpr (WN == 4) {
              const uint4 x = *reinterpret_cast<const uint4*>(src);
              w[kk][0] = x.x;
              w[kk][1] = x.y;
              w[kk][2] = x.z;
              w[kk][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(src);
              w[kk][0] = x.x;
              w[kk][1] = x.y;
            }
          }
#pragma unroll
          for (int j = 0; j < WN; ++j) {
            const uint32_t a0 = __byte_perm(w[0][j], w[1][j], 0x5140u);
            const uint32_t a1 = __byte_perm(w[0][j], w[1][j], 0x7362u);
            const uint32_t c0 = __byte_perm(w[2][j], w[3][j], 0x5140u);
            const uint32_t c1 = __byte_perm(w[2][j], w[3][j], 0x7362u);
            uint32_t b[4][2];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t sel = x & 1 ? 0x4342u : 0x4140u;
              b[x][0] = codes2(x < 2 ? a0 : a1, sel);
              b[x][1] = codes2(x < 2 ? c0 : c1, sel);
            }
            if constexpr (TURNED) {
#pragma unroll
              for (int x = 0; x < 4; x += 2) {
                const uint32_t vf[4] = {b[x][0], b[x + 1][0], b[x][1], b[x + 1][1]};
                mma_f16(o[2 * j + (x >> 1)], vf, pf[step][0], pf[step][1]);
              }
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x) mma_f16(o[4 * j + x], pf[step], b[x][0], b[x][1]);
            }
          }
        }
      }
      __syncwarp();   // the stage was read by other lanes
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }

    // ---- the warps' results, joined pairwise: 4 .. 7 into 0 .. 3, 2, 3 into 0, 1, 1 into 0 ----
    // A result travels through the stage that its warp has read last (or not yet filled),
    // fragments as they are; the loads of the next unit stay on their way meanwhile.
    auto slot_of = [&](int w, int st) {
      return reinterpret_cast<float4*>(smem + w * R::BYTES + st * R::STAGE);
    };
#pragma unroll 1
    for (int r = WARPS / 2; r > 0; r >>= 1) {
      if (warp >= 2 * r) break;
      const int there = warp & (r - 1);                    // the pair (there, there + r)
      const int full = r + there, free = WARPS - 1 + full;   // its barriers, 1 .. 14
      if (warp >= r) {
        if (kb1 - kb0 > 2 * r - 1 - warp) {   // there is one, its own or joined
          float4* const out = slot_of(warp, stage == 0 ? STAGES - 1 : stage - 1) + lane;
#pragma unroll
          for (int n = 0; n < ON; ++n) out[n * 32] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
          s_ml[warp][lane] = make_float4(mx[0], mx[1], l[0], l[1]);
          s_at[warp] = stage == 0 ? STAGES - 1 : stage - 1;
        }
        bar_arrive(full);
        owed = free;
        break;
      }
      bar_sync(full);
      const int w = warp + r;
      if (kb1 - kb0 > 2 * r - 1 - w) {   // it has one
        const float4 ml = s_ml[w][lane];
        const float4* const in = slot_of(w, s_at[w]) + lane;
        const float m[2] = {ml.x, ml.y};
        float c0[2], c1[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float big = fmaxf(mx[h], m[h]);
          c0[h] = big == -INFINITY ? 1.f : exp2_fast(mx[h] - big);
          c1[h] = big == -INFINITY ? 1.f : exp2_fast(m[h] - big);
          mx[h] = big;
          l[h] = l[h] * c0[h] + (h ? ml.w : ml.z) * c1[h];
        }
#pragma unroll
        for (int n = 0; n < ON; ++n) {
          const float4 v = in[n * 32];
          const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] = o[n][e] * c0[row_of(e)] + x[e] * c1[row_of(e)];
        }
      }
      bar_arrive(free);
    }
    if (warp == 0) {
      const bool whole = kb0 == 0 && kb1 == u.n_blocks;
      // a CTA's first piece goes to its slot 0, its last to slot 1
      const int64_t slot = 2 * (int64_t)blockIdx.x + (at == line_lo ? 0 : 1);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int d = TURNED ? 4 : 1; d < (TURNED ? 32 : 4); d *= 2) l[h] += __shfl_xor_sync(~0u, l[h], d);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = tile_row(h), row = u.tile * RT + r, q = a.by_group.quot(row);
        if (q >= u.rows) continue;
        const float inv = mx[h] == -INFINITY ? 0.f : 1.f / l[h];
        uint16_t* const to =
            a.O + ((int64_t)(u.row0 + q) * a.n_heads_q + u.head * G + row - q * G) * D;
        float* const part = a.part_o + (slot * RT + r) * D;
#pragma unroll
        for (int e = 0; e < (TURNED ? 1 : 2); ++e)   // column g, or columns 2 tig + e
#pragma unroll
          for (int n = 0; n < D / 8; n += 8) {   // columns d .. d + 7
            const int gg = TURNED ? g : 2 * tig + e, d = Q8 ? gg * (D / 8) + n : n * 8 + gg * 8;
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              x[k] = TURNED ? o[(n + k) >> 1][(k & 1) * 2 + h] : o[TURNED ? 0 : n + k][2 * h + e];
            if (whole) {
              *reinterpret_cast<uint4*>(to + d) =
                  make_uint4(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv),
                             pack_bf16x2(x[4] * inv, x[5] * inv), pack_bf16x2(x[6] * inv, x[7] * inv));
            } else {
              __stcg(reinterpret_cast<float4*>(part + d), make_float4(x[0], x[1], x[2], x[3]));
              __stcg(reinterpret_cast<float4*>(part + d + 4), make_float4(x[4], x[5], x[6], x[7]));
            }
          }
        if (!whole && (TURNED ? g : tig) == 0)
          __stcg(a.part_ml + slot * RT + r, make_float2(mx[h], l[h]));
      }
    }
    at = u.begin + kb1;
    if (tid == 0 && at >= line_hi) a.cuts[blockIdx.x] = make_cut(u, kb1, line_lo, per);
  }
  if (owed) bar_sync(owed);
  for (int st = 0; dead && st < STAGES; ++st)   // the copies that are still under way
    if ((coming >> st) & 1u) mbar_wait_polls(bar_s + st * 8, (phase >> st) & 1u, 1u << 16);
}

// ------------------------------------------------------------------- joins --
// The rows of a cut unit from their pieces, in order: one warp per row, whose
// lanes hold the pieces' maxima and sums, then four columns each.  A few dependent
// rounds of reads from L2, at the end of every call: what it needs to know
// lies ready in the list of cuts.
constexpr int JOIN_WARPS = 4;   // per CTA
constexpr int join_split(int rt) { return rt <= WIDE ? rt / JOIN_WARPS : 16; }   // CTAs per tile

template <int D, int RT>
__global__ void __launch_bounds__(JOIN_WARPS * 32) chunk_join_kernel(const __grid_constant__ ChunkArgs a) {
  pdl_wait();
  pdl_trigger();
  const int part = blockIdx.x;
  union {
    int4 w[2];
    ChunkCut cut;
  } x;
  x.w[0] = __ldcg(reinterpret_cast<const int4*>(a.cuts + part));
  x.w[1] = __ldcg(reinterpret_cast<const int4*>(a.cuts + part) + 1);
  const ChunkCut c = x.cut;
  if (!cut_stands(c, part, gridDim.x, a.t.n_rows, a.n_heads_kv, a.group, RT)) return;
  constexpr int LANES = D / 4, PER = 32 / LANES;   // lanes per piece, pieces per load
  constexpr int AHEAD = 8;                          // loads in flight
  const int lane = threadIdx.x & 31, n = c.pieces;
  const int d = (lane % LANES) * 4, mine = lane / LANES;
  auto slot = [&](int i) { return (int64_t)(i == 0 ? c.first : 2 * (part + i)); };
  const FastDiv by = a.by_group;
  // (a tile's CTAs in turn: its last rows are often unused)
#pragma unroll 1
  for (int r = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5); r < RT; r += gridDim.y * JOIN_WARPS) {
    const int row = c.tile * RT + r, q = by.quot(row);
    if (q >= c.rows) break;
    // pieces from i0 on, PER at a time: their columns, asked for together
    float4 v[AHEAD];
    auto load = [&](int i0) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int i = i0 + k * PER + mine;
        v[k] = i < n ? __ldcg(reinterpret_cast<const float4*>(a.part_o + (slot(i) * RT + r) * D + d))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    load(0);   // on their way with the maxima
    auto stats = [&](int i) {
      return i < n ? __ldcg(a.part_ml + slot(i) * RT + r) : make_float2(-INFINITY, 0.f);
    };
    const float2 first = stats(lane);
    float big = first.x;
#pragma unroll 1
    for (int i = 32 + lane; i - lane < n; i += 32) big = fmaxf(big, stats(i).x);
    big = warp_max(big);
    auto weight = [&](float m) { return m == -INFINITY ? 0.f : exp2_fast(m - big); };
    float sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int base = 0; base < n; base += 32) {
      const float2 ml = base == 0 ? first : stats(base + lane);
      const float w = weight(ml.x);   // of piece base + lane, 0 if it is not there
      sum = fmaf(w, ml.y, sum);
#pragma unroll 1
      for (int i0 = 0; i0 < 32 && base + i0 < n; i0 += AHEAD * PER) {
        if (base + i0 > 0) load(base + i0);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
          const float f = __shfl_sync(~0u, w, i0 + k * PER + mine);
          x[0] = fmaf(f, v[k].x, x[0]);
          x[1] = fmaf(f, v[k].y, x[1]);
          x[2] = fmaf(f, v[k].z, x[2]);
          x[3] = fmaf(f, v[k].w, x[3]);
        }
      }
    }
    sum = warp_sum(sum);
    if constexpr (PER == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] += __shfl_xor_sync(~0u, x[e], 16);
    }
    const float inv = big == -INFINITY ? 0.f : 1.f / sum;
    if (mine == 0)
      *reinterpret_cast<uint2*>(
          a.O + ((int64_t)(c.row0 + q) * a.n_heads_q + c.head * a.group + row - q * a.group) * D + d) =
          make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
  }
}

// -------------------------------------------------------------------- host --
template <int D, int RT>
int32_t launch_join(const ChunkArgs& a, int n_ctas, cudaStream_t st) {
  SUB_CUDA_TRY(launch_k(chunk_join_kernel<D, RT>, dim3(n_ctas, join_split(RT)),
                        dim3(JOIN_WARPS * 32), 0, st, a));
  return SUB_OK;
}

template <int D, bool Q8, int RT>
int32_t launch_decode(const ChunkArgs& a, int n_ctas, cudaStream_t st) {
  constexpr int SMEM = decode_smem<D, Q8>();
  SUB_CUDA_TRY(once_per_device([] {
    return cudaFuncSetAttribute(chunk_attn_kernel<D, Q8, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                SMEM);
  }));
  PageMaps maps;
  if (!chunk_page_map(&maps.k, a.k, a.t, (int64_t)a.n_layers * a.n_heads_kv, D, Q8) ||
      !chunk_page_map(&maps.v, a.v, a.t, (int64_t)a.n_layers * a.n_heads_kv, D, Q8))
    return fail(SUB_ECUDA, "chunk_attn: the cache's tensor map was refused");
  SUB_CUDA_TRY(launch_k(chunk_attn_kernel<D, Q8, RT>, dim3(n_ctas), dim3(NT), SMEM, st, maps, a));
  return launch_join<D, RT>(a, n_ctas, st);
}

// Rows of a tile, by the rows that a sequence has on average (rows and sequences are
// known here, lengths only on the device) and the most keys that one may have.  The
// warps' kernel reads the keys again for every tile, the tensor-core kernel once for 256
// rows, but it starts later and wants blocks of 128 keys.  bf16: 16 rows, and 32 up to
// 4096 keys (32 rows of 1 sequence over 1000 keys 12 us here, 16 by the tensor cores; of
// 8 over 4000 43 and 41; of 1 over 16000 28 and 28; 20 rows of 8 over 16000 167 and
// 108; 48 of 8 over 4000 60 and 42).  Codes, which the tensor-core kernel has to convert
// first, with a rounding: 64 rows (32 rows of 8 sequences over 4000 keys 37 and 53, 56
// rows of 4 KV heads 36 and 37, 64 rows 62 and 55; 48 rows of 2 over 64000 147 and 150).
int tile_rows(int group, int n_seqs, int n_rows, bool codes, int64_t keys) {
  const int64_t rows = (int64_t)n_rows * group, seqs = n_seqs;
  const int tiles = codes ? 4 : keys <= 4096 ? 2 : 1;
  return rows <= NARROW * seqs ? NARROW : rows <= tiles * WIDE * seqs ? WIDE : CHUNK_TC_ROWS;
}

// Partial results, two per CTA, and the list of cuts.
int64_t part_bytes(int n_ctas, int rows, int d) {
  return (int64_t)n_ctas * (2 * rows * (d + 2) * 4 + (int64_t)sizeof(ChunkCut));
}
// What a call of these sizes may need: the largest tiles that it may get.
int64_t work_bytes(int n_ctas, int group, int d, int n_seqs, int n_rows) {
  return n_rows ? part_bytes(n_ctas, tile_rows(group, n_seqs, n_rows, false, INT64_MAX), d) : 0;
}

template <class Cache>
int32_t chunk_attn(const sub_bf16* Q, int64_t ldq, int32_t n_heads_q, const Cache* kv,
                   const float* ks, const float* vs, int32_t layer, const sub_batch* batch,
                   float softmax_scale, sub_bf16* O, void* workspace, int64_t workspace_bytes,
                   void* stream) {
  constexpr bool Q8 = std::is_same<Cache, sub_kv8_cache>::value;
  ChunkArgs a{};
  SUB_TRY(make_seq_table(kv, layer, batch, &a.t));
  SUB_CHECK_ARG(n_heads_q >= 1 && n_heads_q % kv->n_heads_kv == 0 &&
                    n_heads_q / kv->n_heads_kv <= 64,
                "Hq must be a multiple of Hkv, at most 64 times");
  SUB_CHECK_ARG(softmax_scale >= 0.f && softmax_scale <= 1e6f, "softmax_scale out of range");
  if (a.t.n_rows == 0) return SUB_OK;
  SUB_CHECK_ARG(Q && O, "null pointer");
  SUB_CHECK_ARG(aligned16(Q) && aligned16(O) && ldq % 8 == 0, "rows must be 16-byte aligned");
  SUB_CHECK_ARG(ldq >= (int64_t)n_heads_q * kv->head_dim, "row stride below Hq * head_dim");
  a.Q = Q;
  a.ldq = ldq;
  a.O = O;
  a.k = kv->k;
  a.v = kv->v;
  a.ks = ks;
  a.vs = vs;
  a.layer = layer;
  a.n_layers = kv->n_layers;
  a.n_heads_q = n_heads_q;
  a.n_heads_kv = kv->n_heads_kv;
  a.group = n_heads_q / kv->n_heads_kv;
  a.by_group = make_fast_div(a.group);
  a.by_page = make_fast_div(kv->page_size);
  // (a scale of 0 must not meet the masked scores' -infinity)
  a.sl2 = fmaxf(softmax_scale, 1e-30f) * 1.4426950408889634f;
  const cudaStream_t st = as_stream(stream);
  const int n_ctas = device_sms();
  const int64_t need = work_bytes(n_ctas, a.group, kv->head_dim, a.t.n_seqs, a.t.n_rows);
  StreamScratch scratch(st);
  if (workspace) {
    SUB_CHECK_ARG((reinterpret_cast<uintptr_t>(workspace) & 31) == 0 && workspace_bytes >= need,
                  "workspace too small or not 32-byte aligned");
  } else {
    SUB_TRY(scratch.alloc((size_t)need));
    workspace = scratch.p;
  }
  const int rt = tile_rows(a.group, a.t.n_seqs, a.t.n_rows, Q8,
                           batch->max_keys ? std::min(batch->max_keys, kv->capacity) : kv->capacity);
  const int64_t pool_rows =
      (int64_t)kv->n_layers * kv->n_pages * kv->n_heads_kv * kv->page_size;
  const bool tensor_cores = rt == CHUNK_TC_ROWS && chunk_tc_fits(pool_rows);
  const int part_rows = tensor_cores ? CHUNK_TC_ROWS : std::min(rt, WIDE);
  a.part_o = reinterpret_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (int64_t)n_ctas * 2 * part_rows * kv->head_dim);
  a.cuts = reinterpret_cast<ChunkCut*>(a.part_ml + (int64_t)n_ctas * 2 * part_rows);
  if (tensor_cores) {
    SUB_TRY(launch_chunk_tc(a, Q8, kv->head_dim, pool_rows, n_ctas, st));
    return kv->head_dim == 128 ? launch_join<128, CHUNK_TC_ROWS>(a, n_ctas, st)
                               : launch_join<64, CHUNK_TC_ROWS>(a, n_ctas, st);
  }
  if (rt == NARROW)
    return kv->head_dim == 128 ? launch_decode<128, Q8, NARROW>(a, n_ctas, st)
                               : launch_decode<64, Q8, NARROW>(a, n_ctas, st);
  return kv->head_dim == 128 ? launch_decode<128, Q8, WIDE>(a, n_ctas, st)
                             : launch_decode<64, Q8, WIDE>(a, n_ctas, st);
}

}  // namespace

int32_t chunk_attn_timeouts(unsigned int* out) {
  unsigned int tc = 0;
  SUB_TRY(chunk_tc_timeouts(&tc));
  SUB_CUDA_TRY(cudaMemcpyFromSymbol(out, g_decode_timeouts, sizeof(unsigned int)));
  *out += tc;
  return SUB_OK;
}

}  // namespace sub

using namespace sub;

extern "C" int32_t sub_chunk_attn_workspace(int32_t n_heads_q, int32_t n_heads_kv,
                                            int32_t head_dim, int32_t n_seqs, int32_t n_rows,
                                            int64_t* bytes) {
  SUB_CHECK_ARG(bytes, "null pointer");
  SUB_CHECK_ARG(head_dim == 64 || head_dim == 128, "head_dim must be 64 or 128");
  SUB_CHECK_ARG(n_heads_kv >= 1 && n_heads_q >= 1 && n_heads_q % n_heads_kv == 0,
                "Hq must be a multiple of Hkv");
  SUB_CHECK_ARG(n_seqs >= 1 && n_seqs <= SUB_MAX_SEQS && n_rows >= 0, "bad batch sizes");
  *bytes = work_bytes(device_sms(), n_heads_q / n_heads_kv, head_dim, n_seqs, n_rows);
  return SUB_OK;
}

extern "C" int32_t sub_chunk_attn(const sub_bf16* Q, int64_t ldq, int32_t n_heads_q,
                                  const sub_kv_cache* kv, int32_t layer, const sub_batch* batch,
                                  float softmax_scale, sub_bf16* O, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  return chunk_attn(Q, ldq, n_heads_q, kv, nullptr, nullptr, layer, batch, softmax_scale, O,
                    workspace, workspace_bytes, stream);
}

extern "C" int32_t sub_chunk_attn8(const sub_bf16* Q, int64_t ldq, int32_t n_heads_q,
                                   const sub_kv8_cache* kv, int32_t layer, const sub_batch* batch,
                                   float softmax_scale, sub_bf16* O, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
  SUB_TRY(check_scales(kv));
  return chunk_attn(Q, ldq, n_heads_q, kv, kv->k_scale, kv->v_scale, layer, batch, softmax_scale,
                    O, workspace, workspace_bytes, stream);
}
