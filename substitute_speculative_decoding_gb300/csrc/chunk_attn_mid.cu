// Attention of tree nodes over a paged cache, a few dozen rows per KV head (the nodes of
// a draft tree's level, times the heads of a group), or more over short caches.
//
// Bound by HBM, if the work per key stays small: 32 rows do 32 flops per byte of a bf16
// cache.  The kernel of 16 rows (chunk_attn.cu) would read and, over codes, convert
// every key once per tile of 16; the kernel of 256 rows (chunk_attn_tc.cu) gives each
// row a thread, and 224 of them are idle.  Here both products are turned over, so that
// the keys take the tensor cores' 128 lanes and the N = 32 or 64 rows their columns:
//   S^T = K Q^T   [128 keys x N], a key per thread: its scales and its masks are the thread's own,
//                 and a block costs N exponentials per thread, not 128
//   O^T = V^T P^T [D x N], with P^T written to shared memory as it is formed (bf16: two
//                 halves, hi in the columns of a product and lo beside them; codes: fp16 times V's scale)
// Roles:
//   warps 0-3, 4-7   softmax of the first and the second half of the rows, block by block: the
//                    scores of the next block and the output of the last are formed meanwhile
//   two warps        copies (TMA) of K and of V into rings of blocks of 128 keys, in boxes of as many
//                    keys as a page holds together; the pages of two blocks are looked up ahead
//   one MMA warp
//   warps 8-11, 12-15   codes: K and V into fp16 (code - 128, exactly; two instructions for two of
//                    them), K into tensor memory, a key per lane, V into shared memory.  (Codes
//                    loaded straight into registers, 64 KB of them under way, queue for the 29 KB that
//                    shared memory leaves to L1: 16 sequences of 32 heads, 10000 keys on average,
//                    took 136 us.)
//
// The running maximum of a row lies across the threads, so it is not formed in every
// block: each thread compares its scores with the references of its rows, and only if
// one exceeds its reference by more than 2^8 (codes: 2^3), the group forms the
// maxima and rescales.  Sums are kept per thread and row.
//
// Codes: the weight times V's scale, of which a power of two is part of the score that the
// reference follows and the rest, in [1, 2), a factor: what is rounded to fp16 is 2^11
// at the reference and below 2^15, its smallest step 2^-36 of the reference.  The
// sum takes the weight itself, in fp32.  Rows' scores thus take nothing from keys
// that they do not read, whose scales may be anything.
//
// Measured, heads of 128: 32 rows of each of 16 sequences and 8 KV heads over 10000 keys on average
// 116 us (0.67 GB, 5.8 TB/s), over codes 86 (4.0 TB/s); 56 rows of 32 sequences and 4 KV heads over
// 5100 68 us (5.1 TB/s); 33 nodes of 1 sequence and 8 KV heads over 500 keys 14.  A block of 128 keys
// takes 2200 cycles over codes, of which the issue slots are busy 1240; a bf16 block at HBM's rate 2800.
// All at pages of 64.  Pages of 16, and of 48, come in boxes of 16 keys, 24 copies of K's side of a block of
// codes, which one lane issues in turn: the 86 us are 128 there (bf16, 56 rows: 70 and 69).
//
// V of a block that not all rows read to its end may hold anything where it is not read: values that
// are not finite are taken out by the thread whose key it is, and added at the end to
// the rows that do read them.
#include <cuda_fp16.h>
#include "chunk_tc.cuh"

namespace sub {
namespace {

__device__ unsigned int g_mid_timeouts;   // waits that ran out (never expected)

template <int D, bool Q8, int N>
struct MidCfg {
  static_assert(N == 32 || N == 64, "rows of a tile: a warp's lanes hold one or two each");
  static constexpr int TILE = KB * D * 2;                // K or V of a block, 16-bit values
  static constexpr int SLOTS = !Q8 && D == 64 ? 4 : 2;   // of V, bf16: and of K
  static constexpr int CODES = Q8 ? KB * D : 0;          // K or V of a block, codes
  static constexpr int RAW = Q8 ? D == 64 ? 4 : 3 : 0;   // blocks of codes
  static constexpr int Q_BYTES = N * D * 2;
  static constexpr int H = N / 2;                        // of a group
  // A key's weights: lines of 64 columns.  bf16: N = 32 hi and lo in one, N = 64 one each
  static constexpr int P_LINES = KB * 128, P_COLS = Q8 ? N : 2 * N;
  static constexpr int P_BYTES = P_COLS > 64 ? 2 * P_LINES : P_LINES;   // of a block; two of them
  static constexpr int COPY_WARP = Q8 ? 16 : 8;          // K's; the next is V's
  static constexpr int MMA_WARP = COPY_WARP + 2;
  static constexpr int THREADS = (MMA_WARP + 2) * 32;    // whole groups of four warps
  // codes: registers by group of four warps, out of 65536 / THREADS each at the launch
  static constexpr int REGS_SOFTMAX = 128, REGS_CONV = 80, REGS_MMA = 64;
  static_assert(!Q8 || (2 * REGS_SOFTMAX + 2 * REGS_CONV + REGS_MMA) * 128 <= 65536 / THREADS / 8 * 8 * THREADS,
                "the shares fit what the block is launched with");
  static constexpr float GROWTH = Q8 ? 3.f : 8.f;        // log2 of how far weights may exceed the reference
  static constexpr float SHIFT = Q8 ? 11.f : 0.f;        // log2 of the weight at it
  // Eight blocks' scales of K, of V.  (K's copies run at most RAW + SLOTS blocks ahead of the scores
  // that are formed, and those one ahead of the softmax.)
  static constexpr int SCALES = Q8 ? 8 * 2 * KB * 4 : 0;
  static_assert(RAW + SLOTS + 1 < 8, "scales are read before their place is written again");
  // of the rows: place in O, last key, mask, factor, minus the reference, whether a key was
  // read, factor of what was formed and difference of the reference; [4 warps] maxima or sums
  static constexpr int INFO = N * (8 + 7 * 4 + 4 * 4);
  static constexpr int TAIL = 512;                       // barriers, flags, TMEM address
  static constexpr int RING = (Q8 ? 1 : 2) * SLOTS * TILE + 2 * RAW * CODES;
  // columns: S^T of two blocks, O^T, codes: K of two blocks
  static constexpr int TM_O = 2 * N, TM_K = TM_O + P_COLS, COLS = TM_K + (Q8 ? D : 0);
  static constexpr int TMEM = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static constexpr int SMEM = 1024 + 2 * P_BYTES + Q_BYTES + RING + SCALES + INFO + TAIL;
  static_assert(SMEM <= 227 * 1024, "one CTA's shared memory");
  static_assert(RING >= (SUB_MAX_SEQS + 1) * 8, "the ring holds the running sums first");
};

// Untiled copy: both addresses 16-byte aligned.  (A tiled one would want its place in shared memory
// at 128 bytes, and 16 scales are 64.)
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, int bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 4, 256;" ::: "memory"); }
__device__ __forceinline__ void group_sync(int t) { asm volatile("bar.sync %0, 128;" ::"r"(t + 1) : "memory"); }
// whether any thread of the group says so
__device__ __forceinline__ bool group_any(int t, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %2, 0;\n barrier.cta.red.or.pred p, %1, 128, q;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"(t + 1), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// v[i] of all lanes joined by f, for i = lane (below M).
template <int M, class F>
__device__ __forceinline__ float across(float (&v)[M], int lane, F f) {
  if constexpr (M == 16) {
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] = f(v[i], __shfl_xor_sync(~0u, v[i], 16));
  }
#pragma unroll
  for (int o = M / 2; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float mine = up ? v[i + o] : v[i], other = up ? v[i] : v[i + o];
      v[i] = f(mine, __shfl_xor_sync(~0u, other, o));
    }
  return v[0];
}

// ------------------------------------------------------------------ kernel --
template <int D, bool Q8, int N>
__global__ void __launch_bounds__(MidCfg<D, Q8, N>::THREADS, 1)
chunk_mid_kernel(const __grid_constant__ Maps maps, const __grid_constant__ ChunkArgs a, const int box,
                 const int pool_rows) {
  using C = MidCfg<D, Q8, N>;
  constexpr int SLOTS = C::SLOTS, H = C::H;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const base_p = smem_raw + (base - smem_u32(smem_raw));
  // (V's ring is followed by another: at D = 64 the product reads 64 columns past a block, for lanes
  // that nobody reads)
  const uint32_t p_s = base, q_s = p_s + 2 * C::P_BYTES, v_s = q_s + C::Q_BYTES, k_s = v_s + SLOTS * C::TILE,
                 raw_s = v_s + SLOTS * C::TILE;   // bf16: K's blocks; codes: K's, then V's
  int64_t* const s_pre = reinterpret_cast<int64_t*>(base_p + (v_s - base));   // until the first copies
  uint8_t* at_p = base_p + (v_s - base) + C::RING;
  auto take = [&](int bytes) {
    uint8_t* const p = at_p;
    at_p += bytes;
    return p;
  };
  float* const s_scale = reinterpret_cast<float*>(take(C::SCALES));    // [8][K: KB, V: KB]
  int64_t* const s_place = reinterpret_cast<int64_t*>(take(N * 8));    // of a row in O; -1: none
  float* const s_qs = reinterpret_cast<float*>(take(N * 4));           // codes: factor of a row's scores
  float* const s_nref = reinterpret_cast<float*>(take(N * 4));         // SHIFT - reference
  float* const s_fac = reinterpret_cast<float*>(take(N * 4));
  float* const s_diff = reinterpret_cast<float*>(take(N * 4));
  float* const s_part = reinterpret_cast<float*>(take(4 * N * 4));     // [group][warp][H]
  int* const s_any = reinterpret_cast<int*>(take(N * 4));              // a key has been read
  int* const s_lim = reinterpret_cast<int*>(take(N * 4));              // keys 0 .. lim are read
  int* const s_mask = reinterpret_cast<int*>(take(N * 4));             // row of the masks
  uint8_t* const tail = take(C::TAIL);
  const uint32_t bars = smem_u32(tail);
  constexpr int BARS = 4 * SLOTS + 4 * C::RAW + 7;
  auto ring = [&](int which, uint32_t block) { return bars + 8u * (which * SLOTS + block % SLOTS); };
  auto k_full = [&](uint32_t block) { return ring(0, block); };
  auto k_empty = [&](uint32_t block) { return ring(1, block); };
  auto v_full = [&](uint32_t block) { return ring(2, block); };
  auto v_empty = [&](uint32_t block) { return ring(3, block); };
  auto raw_full = [&](int side, uint32_t block) {   // codes of K, of V
    return bars + 8u * (4 * SLOTS + 2 * side * C::RAW + block % max(C::RAW, 1));
  };
  auto raw_empty = [&](int side, uint32_t block) { return raw_full(side, block) + 8u * C::RAW; };
  auto pair = [&](int which, uint32_t block) { return bars + 8u * (BARS - 7 + 2 * which + (block & 1)); };
  auto s_full = [&](uint32_t block) { return pair(0, block); };
  auto p_full = [&](uint32_t block) { return pair(1, block); };
  auto o_full = [&](uint32_t block) { return pair(2, block); };
  const uint32_t q_full = bars + 8u * (BARS - 1);
  int* const flags = reinterpret_cast<int*>(tail + 8 * BARS);
  volatile int* const s_dead = flags;                // a wait ran out
  volatile int* const s_odd = flags + 1;             // 1 + the last piece that met infinite values or NaN
  volatile int* const s_force = flags + 2;           // [group] a row has read no key yet
  volatile uint32_t* const s_miss = reinterpret_cast<uint32_t*>(flags + 4);   // [8] blocks' missing 16-key parts
  uint32_t* const s_tmem = reinterpret_cast<uint32_t*>(flags + 12);
  static_assert(8 * BARS + 13 * 4 <= C::TAIL, "tail");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(s_tmem)),
                 "r"(C::TMEM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(k_full(i), Q8 ? 4 : 1);   // an arrival for each warp, or the copies'
      mbar_init(v_full(i), Q8 ? 4 : 1);
      mbar_init(k_empty(i), 1);
      mbar_init(v_empty(i), 1);
    }
    for (int i = 0; i < C::RAW; ++i)
      for (int side = 0; side < 2; ++side) {
        mbar_init(raw_full(side, i), 1);
        mbar_init(raw_empty(side, i), 4);
      }
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(p_full(b), 8);   // one arrival for each softmax warp
      mbar_init(o_full(b), 1);
    }
    mbar_init(q_full, 8);
    *s_dead = 0;
    *s_odd = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 64) {
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  pdl_wait();
  pdl_trigger();
  const ChunkPlan<N, KB> plan(a);
  tc_fence_before();
  plan.template scan<C::THREADS>(s_pre);   // ends with a barrier
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int64_t total = s_pre[a.t.n_seqs];
  const int64_t per = blocks_per_cta(total, gridDim.x, plan.least(total, CHUNK_TC_LEAST));
  int64_t line_lo, line_hi;
  ChunkUnit u = plan.template part<true>(s_pre, total, per, line_lo, line_hi);
  fence_async();     // the ring is written by copies from here on
  __syncthreads();
  const Gate gate{s_dead, &g_mid_timeouts};
  const int G = a.group;
  const uint32_t n = (uint32_t)(line_hi > line_lo ? line_hi - line_lo : 0);   // blocks, across the units
  int kb = (int)(line_lo - u.begin);   // the next block to look up, of unit u
  auto step = [&] {
    if (++kb == u.n_blocks) {
      plan.next(u);
      kb = 0;
    }
  };

  if constexpr (Q8) {
    if (warp < 8) more_registers<C::REGS_SOFTMAX>();
    else if (warp < C::COPY_WARP) fewer_registers<C::REGS_CONV>();
    else fewer_registers<C::REGS_MMA>();
  }

  if (warp < 8) {
    // ------------------------------------------------ softmax, Q, results
    const int t = warp >> 2, wq = warp & 3, r = wq * 32 + lane;   // group, the thread's key of a block (or column of O)
    const int c0 = t * H;                                         // the group's rows
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + c0 + lanes, tO = tmem + C::TM_O + c0 + lanes;
    float* const nref = s_nref + c0;
    float* const fac = s_fac + c0;
    uint32_t block = 0;             // of this CTA's part of the line
    constexpr int CH = D / 8, RP = 32 / CH, QP = N / 8 / RP;   // 16-byte chunks of a Q row, rows per pass of a warp, passes
    const int c = lane % CH, q_row = warp * (N / 8) + lane / CH;
    uint4 qw[QP];
    auto q_load = [&] {
#pragma unroll
      for (int i = 0; i < QP; ++i) {
        const int row = u.tile * N + q_row + i * RP, q = a.by_group.quot(row);
        qw[i] = make_uint4(0, 0, 0, 0);
        if (q < u.rows)
          qw[i] = ldg_cg_v4(a.Q + (int64_t)(u.row0 + q) * a.ldq + (int64_t)(u.head * G + row - q * G) * D + c * 8);
      }
    };
    // (also for a CTA that stops early because a wait ran out)
    if (tid == 0) a.cuts[blockIdx.x].pieces = 0;
    if (line_lo < line_hi) q_load();
    int piece = 0;
    for (int64_t at = line_lo; at < line_hi; ++piece) {
      const int kb0 = (int)(at - u.begin), kb1 = (int)min((int64_t)u.n_blocks, line_hi - u.begin), nb = kb1 - kb0;
      const bool first = at == line_lo, whole = kb0 == 0 && kb1 == u.n_blocks;
      at = u.begin + kb1;
      if (tid == 0 && at >= line_hi) a.cuts[blockIdx.x] = make_cut(u, kb1, line_lo, per);
      // ---- the rows, and Q into shared memory: chunk c of a row at c ^ (row % 8) of its
      // 128-byte line (everyone is through with the last piece's) ----
      softmax_sync();
      if (tid < N) {
        const int row = u.tile * N + tid, q = a.by_group.quot(row);
        const bool real = q < u.rows;
        s_place[tid] = !real ? -1
                             : whole ? ((int64_t)(u.row0 + q) * a.n_heads_q + u.head * G + row - q * G) * D
                                     : ((2 * (int64_t)blockIdx.x + (first ? 0 : 1)) * N + tid) * D;
        s_lim[tid] = real ? last_key(u.pos, q, u.n_keys) : -1;
        s_mask[tid] = u.row0 + min(q, u.rows - 1);
        s_nref[tid] = 0.f;
        s_any[tid] = 0;
      }
#pragma unroll
      for (int i = 0; i < QP; ++i) {
        const int rr = q_row + i * RP;
        uint4 w = qw[i];
        if constexpr (Q8) {
          // the row's largest value to [1, 2), for fp16
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
          float big = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) big = fmaxf(big, fmaxf(fabsf(bf16lo(x[k])), fabsf(bf16hi(x[k]))));
#pragma unroll
          for (int o = CH / 2; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
          const int e = min(126, max(-126, (int)(__float_as_uint(big) >> 23) - 127));
          const float down = __uint_as_float((uint32_t)(127 - e) << 23);
          if (c == 0) s_qs[rr] = fmaxf(a.sl2 * __uint_as_float((uint32_t)(127 + e) << 23), 1e-37f);
          w.x = pack_f16x2(bf16lo(x[0]) * down, bf16hi(x[0]) * down);
          w.y = pack_f16x2(bf16lo(x[1]) * down, bf16hi(x[1]) * down);
          w.z = pack_f16x2(bf16lo(x[2]) * down, bf16hi(x[2]) * down);
          w.w = pack_f16x2(bf16lo(x[3]) * down, bf16hi(x[3]) * down);
        }
        st_shared(q_s + (c >> 3) * (N * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), w.x, w.y, w.z, w.w);
      }
      fence_async();
      tc_fence_before();   // O^T of the last piece is read
      softmax_sync();
      if (lane == 0) mbar_arrive(q_full);
      const int lim_all = plan.template common<true>(u);   // last key that every row reads
      const int slot0 = tree_base(a, u.b);
      // 32 keys from `key` on that the row reads, as far as its place and its mask say
      auto reads = [&](int row, int key) {
        const int left = s_lim[row] - key;
        if (left < 0) return 0u;
        return mask_window(a.mask + (int64_t)s_mask[row] * a.words, a.words, key - slot0) &
               (left >= 31 ? ~0u : (2u << left) - 1u);
      };

      bool force = true;   // a row has read no key yet
      float2 l[H / 2];
#pragma unroll
      for (int x = 0; x < H / 2; ++x) l[x] = make_float2(0.f, 0.f);
      // (A wait that runs out stops no warp: all of them meet in barriers.  The waits after it
      // return soon, and the results are not valid.)
#pragma unroll 1
      for (int i = 0; i < nb; ++i, ++block) {
        const int key0 = (kb0 + i) * KB;
        const bool behind = key0 + KB - 1 > lim_all;
        // lane x: the warp's 32 keys, as the group's row x reads them
        uint32_t word = ~0u;
        if (behind && lane < H) word = reads(c0 + lane, key0 + wq * 32);
        gate.wait_warp(s_full(block), (block >> 1) & 1);
        tc_fence_after();
        const uint32_t miss = s_miss[block & 7];
        float s[H];
        if constexpr (H == 32) tc_ld32(tS + (block & 1) * N, s);
        else tc_ld16(tS + (block & 1) * N, s);
        // codes: this key's scales, that of V as a power of two and the rest of it
        float f = a.sl2, lv = 0.f, part = 1.f, back = 1.f;
        if constexpr (Q8) {
          const float* const sc = s_scale + (block & 7) * (2 * KB);
          // a row that reads a key whose scale of V is not finite gets NaN by its score; weight 0
          // times it stays 0
          float vv = sc[KB + r];
          const bool fine = fabsf(vv) < INFINITY;
          vv = fine ? vv : 1.f;
          const int e = min(126, max(-80, (int)((__float_as_uint(vv) >> 23) & 255u) - 127));
          f = fine ? sc[r] : __int_as_float(0x7fc00000);
          lv = (float)e;
          back = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e
          part = vv * back;
        }
        const float2 f2 = make_float2(f, f), lv2 = make_float2(lv, lv);
        wait_ld();
        if constexpr (Q8) {
#pragma unroll
          for (int x = 0; x < H; x += 4) {
            const float4 qs = *reinterpret_cast<const float4*>(s_qs + c0 + x);
            const float2 a0 = fma2(mul2(make_float2(s[x], s[x + 1]), make_float2(qs.x, qs.y)), f2, lv2);
            const float2 a1 = fma2(mul2(make_float2(s[x + 2], s[x + 3]), make_float2(qs.z, qs.w)), f2, lv2);
            s[x] = a0.x;
            s[x + 1] = a0.y;
            s[x + 2] = a1.x;
            s[x + 3] = a1.y;
          }
        }
        if (behind || miss) {
          const uint32_t gone = miss >> (2 * wq);
          word &= ((gone & 1u) ? 0u : 0xffffu) | ((gone & 2u) ? 0u : 0xffff0000u);
#pragma unroll
          for (int x = 0; x < H; ++x)
            if (!((__shfl_sync(~0u, word, x) >> lane) & 1u)) s[x] = -INFINITY;
        }
        // ---- scores relative to the references ----
        float over[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < H; x += 4) {
          const float4 m = *reinterpret_cast<const float4*>(nref + x);
          float2 a0 = make_float2(s[x], s[x + 1]), a1 = make_float2(s[x + 2], s[x + 3]);
          a0 = Q8 ? add2(a0, make_float2(m.x, m.y)) : fma2(a0, f2, make_float2(m.x, m.y));
          a1 = Q8 ? add2(a1, make_float2(m.z, m.w)) : fma2(a1, f2, make_float2(m.z, m.w));
          over[0] = fmaxf(over[0], s[x] = a0.x);
          over[1] = fmaxf(over[1], s[x + 1] = a0.y);
          over[2] = fmaxf(over[2], s[x + 2] = a1.x);
          over[3] = fmaxf(over[3], s[x + 3] = a1.y);
        }
        const bool above = fmaxf(fmaxf(over[0], over[1]), fmaxf(over[2], over[3])) > C::GROWTH + C::SHIFT;
        if (group_any(t, above || force)) {
          // ---- the references, and what was formed with others ----
          {
            float v[H];
#pragma unroll
            for (int x = 0; x < H; ++x) v[x] = s[x];
            const float m = across(v, lane, [](float x, float y) { return fmaxf(x, y); });
            if (lane < H) s_part[(t * 4 + wq) * H + lane] = m;
          }
          group_sync(t);
          if (wq == 0) {
            bool none = false;
            if (lane < H) {
              float m = -INFINITY;   // largest score, relative to the reference
#pragma unroll
              for (int w = 0; w < 4; ++w) m = fmaxf(m, s_part[(t * 4 + w) * H + lane]);
              const bool any = s_any[c0 + lane];
              float diff = 0.f, less = 1.f;
              if (any ? m > C::SHIFT : m > -INFINITY) {
                diff = C::SHIFT - m;
                less = any ? exp2_fast(diff) : 0.f;   // (nothing was formed without a key)
                nref[lane] += diff;
                s_any[c0 + lane] = 1;
              }
              fac[lane] = less;
              s_diff[c0 + lane] = diff;
              none = !any && !(m > -INFINITY) && s_place[c0 + lane] >= 0;
            }
            none = __any_sync(~0u, none);
            if (lane == 0) s_force[t] = none;
          }
          group_sync(t);
          force = s_force[t];
#pragma unroll
          for (int x = 0; x < H; x += 2) {
            const float2 y = *reinterpret_cast<const float2*>(fac + x);
            const float2 z = *reinterpret_cast<const float2*>(s_diff + c0 + x);
            l[x / 2] = mul2(l[x / 2], y);
            s[x] += z.x;
            s[x + 1] += z.y;
          }
          if (i > 0) {
            gate.wait_warp(o_full(block - 1), ((block - 1) >> 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < (Q8 ? H : 2 * H); x += 16) {
              float o[16];
              const int y = x % H;   // its row; bf16: the halves' columns lie N apart
              __syncwarp();
              tc_ld16(tO + y + x / H * N, o);
              wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= fac[y + k];
              tc_st16(tO + y + x / H * N, reinterpret_cast<const uint32_t*>(o));
            }
            wait_st();
          }
        }
        // ---- weights, into shared memory: chunk k of a key's line at k ^ (key % 8) ----
        const float2 back2 = make_float2(back, back), part2 = make_float2(part, part);
        const uint32_t line = p_s + (block & 1) * C::P_BYTES + r * 128;
#pragma unroll
        for (int x = 0; x < H; x += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float2 e = make_float2(exp2_fast(s[x + 2 * k]), exp2_fast(s[x + 2 * k + 1]));
            if constexpr (Q8) {
              l[x / 2 + k] = fma2(e, back2, l[x / 2 + k]);
              e = mul2(e, part2);
              hi[k] = pack_f16x2(e.x, e.y);
            } else {
              l[x / 2 + k] = add2(l[x / 2 + k], e);
              hi[k] = pack_bf16x2(e.x, e.y);
              const float2 rest = add2(e, make_float2(-bf16lo(hi[k]), -bf16hi(hi[k])));
              lo[k] = pack_bf16x2(rest.x, rest.y);
            }
          }
          auto chunk = [&](int col) {
            return line + (col >> 6) * C::P_LINES + (((((uint32_t)col >> 3) & 7u) ^ (r & 7)) << 4);
          };
          st_shared(chunk(c0 + x), hi[0], hi[1], hi[2], hi[3]);
          if constexpr (!Q8) st_shared(chunk(N + c0 + x), lo[0], lo[1], lo[2], lo[3]);
        }
        if (!Q8 && behind) {
          // V of the block: half of its row r is this thread's
          const int k0 = t * (D / 16);
          gate.wait_warp(v_full(block), (block / SLOTS) & 1);
          const uint32_t v0 = v_s + block % SLOTS * C::TILE + r * 128;
          const bool past = key0 + r >= u.n_keys;
          uint32_t z = 0;   // 0 * x is NaN for what is not finite
#pragma unroll 4
          for (int k = k0; k < k0 + D / 16; ++k) {
            const uint32_t at16 = v0 + (k >> 3) * (KB * 128) + (((k ^ r) & 7) << 4);
            if (past) {
              st_shared(at16, 0, 0, 0, 0);
            } else {
              const uint4 v = lds128(at16);
              const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int y = 0; y < 4; ++y)
                asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(z) : "r"(x[y]), "r"(0u));
            }
          }
          if ((z & 0x7fff7fffu) != 0) {   // hardly ever: take them out, add them at the end
#pragma unroll 1
            for (int k = k0; k < k0 + D / 16; ++k) {
              const uint32_t at16 = v0 + (k >> 3) * (KB * 128) + (((k ^ r) & 7) << 4);
              const uint4 v = lds128(at16);
              uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                if ((x[y] & 0x7f80u) == 0x7f80u) x[y] &= 0xffff0000u;
                if ((x[y] & 0x7f800000u) == 0x7f800000u) x[y] &= 0x0000ffffu;
              }
              st_shared(at16, x[0], x[1], x[2], x[3]);
            }
            *s_odd = piece + 1;
          }
        }
        fence_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(block));
      }
      // ---- the results: the next piece's Q comes meanwhile ----
      const ChunkUnit done = u;
      plan.next(u);
      if (at < line_hi) q_load();
      {   // sums over the group's threads, per row
        float v[H];
#pragma unroll
        for (int x = 0; x < H; x += 2) {
          v[x] = l[x / 2].x;
          v[x + 1] = l[x / 2].y;
        }
        const float sum = across(v, lane, [](float x, float y) { return x + y; });
        if (lane < H) s_part[(t * 4 + wq) * H + lane] = sum;
      }
      group_sync(t);
      if (r < H) {
        const int row = c0 + r;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) sum += s_part[(t * 4 + w) * H + r];
        fac[r] = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
        if (!whole && s_place[row] >= 0)   // (codes: the shift is common to all pieces)
          __stcg(a.part_ml + s_place[row] / D, make_float2(s_any[row] ? -nref[r] : -INFINITY, sum));
      }
      gate.wait_warp(o_full(block - 1), ((block - 1) >> 1) & 1);
      tc_fence_after();
      group_sync(t);
      const bool odd = !Q8 && *s_odd == piece + 1;
      // O^T: the thread's column of D (r), the group's rows
#pragma unroll 1
      for (int x0 = 0; x0 < H; x0 += 16) {
        float o[16];
        __syncwarp();
        tc_ld16(tO + x0, o);
        if constexpr (!Q8) {
          float lo[16];
          tc_ld16(tO + N + x0, lo);
          wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] += lo[k];
        } else {
          wait_ld();
        }
        if (odd && r < D) {
          // values that are not finite, of the keys that a row reads in the blocks looked through
          const uint16_t* const vp = reinterpret_cast<const uint16_t*>(a.v);
#pragma unroll 1
          for (int key = max(kb0, max(0, lim_all + 1) / KB) * KB; key < min(done.n_keys, kb1 * KB); ++key) {
            const int page = page_of(a.t, done.b, key);
            if (page < 0) continue;
            const uint16_t x = __ldcg(
                vp + pool_row(a.t, a.layer, a.n_heads_kv, page, done.head,
                              (int)((uint32_t)key % (uint32_t)a.t.page_size)) * D + r);
            if ((x & 0x7f80u) != 0x7f80u) continue;
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (reads(c0 + x0 + k, key) & 1u) o[k] += bf16_bits_to_f32(x);
          }
        }
        if (r < D) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int64_t place = s_place[c0 + x0 + k];
            if (place < 0) continue;
            if (whole) a.O[place + r] = f32_to_bf16_bits(o[k] * fac[x0 + k]);
            else __stcg(a.part_o + place + r, o[k]);
          }
        }
      }
    }
  } else if (warp < C::COPY_WARP) {
    // ------------------------------------------------------ codes into fp16
    // A key per thread.  Chunk c of a row of codes lies at c ^ (row % 8) of its 128-byte line, or of
    // its half of one: eight lanes read all banks.
    if constexpr (Q8) {
      const int side = (warp - 8) >> 2, key = (warp & 3) * 32 + lane;   // K, V
      const uint32_t raw0 = raw_s + side * (C::RAW * C::CODES) + key * D, turn = D == 128 ? key & 7 : (key >> 1) & 3;
      const uint32_t tK = tmem + C::TM_K + ((uint32_t)((warp & 3) * 32) << 16);
      for (uint32_t j = 0; j < n; ++j) {
        if (!gate.wait_warp(raw_full(side, j), (j / C::RAW) & 1)) break;
        if (j >= SLOTS && !gate.wait_warp(side ? v_empty(j) : k_empty(j), ((j / SLOTS) - 1) & 1)) break;
        if (side == 0) tc_fence_after();
        const uint32_t raw = raw0 + j % C::RAW * C::CODES;
        const uint32_t to = v_s + j % SLOTS * C::TILE + key * 128;
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
          uint32_t x[16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 w = lds128(raw + (((c + h) ^ turn) << 4));
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              x[8 * h + 2 * y] = codes2(v[y], 0x4140u);
              x[8 * h + 2 * y + 1] = codes2(v[y], 0x4342u);
            }
          }
          if (side == 0) {
            tc_st16(tK + (j & 1) * (D / 2) + c * 8, x);
          } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) {   // 16-byte chunks 2 c .. 2 c + 3 of the row
              const int f = 2 * c + h;
              st_shared(to + (f >> 3) * (KB * 128) + (((f & 7) ^ (key & 7)) << 4), x[4 * h], x[4 * h + 1],
                        x[4 * h + 2], x[4 * h + 3]);
            }
          }
        }
        if (side == 0) {
          wait_st();
          tc_fence_before();
        } else {
          fence_async();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(raw_empty(side, j));
          mbar_arrive(side ? v_full(j) : k_full(j));
        }
      }
    }
  } else if (warp < C::MMA_WARP) {
    // --------------------------------------------------------------- copies
    const int side = warp - C::COPY_WARP;   // K, V
    constexpr int DEPTH = Q8 ? C::RAW : SLOTS;
    auto full = [&](uint32_t j) { return Q8 ? raw_full(side, j) : side ? v_full(j) : k_full(j); };
    auto empty = [&](uint32_t j) { return Q8 ? raw_empty(side, j) : side ? v_empty(j) : k_empty(j); };
    const int b0 = lane & 7, n_box = KB / box;   // a box of the block
    // Each box's page is asked for two blocks ahead of its copy.
    int page[2], place[2], head[2];   // place -1: past the last key
    auto ask = [&](uint32_t j, int x) {   // called for j = 0, 1, ..
      if (j >= n) return;
      if (j > 0) step();
      const int key = kb * KB + b0 * box, entry = a.by_page.quot(key);
      const bool there = b0 < n_box && key < u.n_keys;
      place[x] = there ? key - entry * a.t.page_size : -1;
      page[x] = there ? a.t.pages[(int64_t)u.b * a.t.width + entry] : 0;
      head[x] = u.head;
    };
    ask(0, 0);
    ask(1, 1);
    bool ok = true;
    uint32_t j = 0;
    while (j < n && ok) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (j >= n) break;
        if (j >= DEPTH) ok = gate.wait_warp(empty(j), ((j / DEPTH) - 1) & 1);
        if (!ok) break;
        const bool past = place[x] < 0, none = !past && (unsigned)page[x] >= (unsigned)a.t.n_pages;
        // past the pool (zeros) where there is no page
        const int row = past || none
                            ? pool_rows
                            : (int)pool_row(a.t, a.layer, a.n_heads_kv, page[x], head[x], place[x]);
        if (side == 0) {   // the block's 16-key parts without a page
          const unsigned gone = __ballot_sync(~0u, none && lane < n_box);
          if (lane == 0) {
            uint32_t miss = 0;
            if (gone)
              for (int b = 0; b < n_box; ++b)
                if ((gone >> b) & 1u) miss |= ((1u << (box / 16)) - 1u) << (b * box / 16);
            s_miss[j & 7] = miss;
          }
        }
        // scales come where there are some; elsewhere what lies there is not used
        const unsigned some = Q8 && side == 0 ? __ballot_sync(~0u, lane < n_box && !past && !none) : 0;
        const uint32_t bar = full(j);
        if (lane == 0) mbar_expect_tx(bar, Q8 ? C::CODES + __popc(some) * (2 * box * 4) : C::TILE);
        __syncwarp();
        // one lane issues them all, with values that are the same in all lanes
        const CUtensorMap* const map = side ? &maps.v : &maps.k;
#pragma unroll 1
        for (int b = 0; b < n_box; ++b) {
          const int y = __shfl_sync(~0u, row, b);
          if (elect_one()) {
            if constexpr (Q8) {
              tma_load_2d(raw_s + (side * C::RAW + j % C::RAW) * C::CODES + b * box * D, map, 0, y, bar);
              if ((some >> b) & 1u) {
                const uint32_t to = smem_u32(s_scale + (j & 7) * (2 * KB) + b * box);
                bulk_load(to, a.ks + y, box * 4, bar);
                bulk_load(to + KB * 4, a.vs + y, box * 4, bar);
              }
            } else {
              const uint32_t to = (side ? v_s : k_s) + j % SLOTS * C::TILE + b * box * 128;
#pragma unroll
              for (int h = 0; h < D / 64; ++h) tma_load_2d(to + h * (KB * 128), map, h * 64, y, bar);
            }
          }
          __syncwarp();
        }
        ++j;
        ask(j + 1, x);
      }
    }
    // the copies issued last: none may be under way when the CTA ends, whatever its consumers did
    for (uint32_t i = j > DEPTH ? j - DEPTH : 0; i < j; ++i) mbar_wait_polls(full(i), (i / DEPTH) & 1, 1u << 20);
  } else if (warp == C::MMA_WARP) {
    // ---------------------------------------------------------- MMA issuer
    // The whole warp walks through this, with values that the compiler can see to be
    // the same in all lanes, and elects the lane that issues (chunk_attn_tc.cu).
    constexpr uint32_t id_s = idesc(N, !Q8, false), id_o = idesc(C::P_COLS, !Q8, true, true);
    const uint32_t tm = __shfl_sync(~0u, tmem, 0);
    uint32_t block = 0, n_q = 0;
    // descriptors of the first step; a step further is a constant in the address field
    const uint64_t q_desc = desc_k(q_s), p_desc = desc_mn(p_s), v_desc = desc_mn(v_s), k_desc = desc_k(k_s);
    static_assert(C::P_LINES == KB * 128, "the next 64 columns lie where desc_mn says");
    auto scores = [&](uint32_t b) {
      if (!gate.wait_warp(k_full(b), (b / SLOTS) & 1)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t to = tm + (b & 1) * N;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t qd = q_desc + (((k >> 2) * (N * 128) + (k & 3) * 32) >> 4);
          if constexpr (Q8)
            mma_ts(to, tm + C::TM_K + (b & 1) * (D / 2) + k * 8, qd, id_s, k > 0);
          else
            mma_ss(to, k_desc + b % SLOTS * (C::TILE >> 4) + (((k >> 2) * (KB * 128) + (k & 3) * 32) >> 4), qd,
                   id_s, k > 0);
        }
        tc_commit(s_full(b));
        tc_commit(k_empty(b));
      }
      __syncwarp();
      return true;
    };
    auto output = [&](uint32_t b, bool add) {
      if (!gate.wait_warp(v_full(b), (b / SLOTS) & 1) || !gate.wait_warp(p_full(b), (b >> 1) & 1)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t vd = v_desc + b % SLOTS * (C::TILE >> 4), pd = p_desc + (b & 1) * (C::P_BYTES >> 4);
#pragma unroll
        for (int k = 0; k < KB / 16; ++k)
          mma_ss(tm + C::TM_O, vd + k * (2048 >> 4), pd + k * (2048 >> 4), id_o, add || k > 0);
        tc_commit(v_empty(b));
        tc_commit(o_full(b));
      }
      __syncwarp();
      return true;
    };
    bool ok = true;
    for (int64_t at = line_lo; at < line_hi && ok; plan.next(u)) {
      const int kb0 = (int)(at - u.begin), kb1 = (int)min((int64_t)u.n_blocks, line_hi - u.begin);
      at = u.begin + kb1;
      const int nb = __shfl_sync(~0u, kb1 - kb0, 0);
      ok = gate.wait_warp(q_full, n_q++ & 1) && scores(block) && (nb == 1 || scores(block + 1));
      for (int i = 0; i < nb && ok; ++i, ++block) ok = output(block, i > 0) && (i + 2 >= nb || scores(block + 2));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM)
                 : "memory");
}

// -------------------------------------------------------------------- host --
// Rows of codes, in boxes of `box` rows.
bool code_map(CUtensorMap* m, const void* pool, int64_t rows, int d, int box) {
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, pool, d, rows, d, d, box, d);
}
template <int D, bool Q8, int N>
int32_t launch(const ChunkArgs& a, int64_t rows, int n_ctas, cudaStream_t st) {
  using C = MidCfg<D, Q8, N>;
  SUB_CUDA_TRY(once_per_device([] {
    return cudaFuncSetAttribute(chunk_mid_kernel<D, Q8, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::SMEM);
  }));
  Maps maps;
  int box = 16;
  while (box < KB && a.t.page_size % (2 * box) == 0) box *= 2;
  bool fine;
  if constexpr (Q8)
    fine = code_map(&maps.k, a.k, rows, D, box) && code_map(&maps.v, a.v, rows, D, box);
  else
    fine = chunk_pool_map(&maps.k, a.k, rows, D, box) && chunk_pool_map(&maps.v, a.v, rows, D, box);
  if (!fine) return fail(SUB_ECUDA, "chunk_tree_attn: the cache's tensor map was refused");
  SUB_CUDA_TRY(launch_k(chunk_mid_kernel<D, Q8, N>, dim3(n_ctas), dim3(C::THREADS), C::SMEM, st, maps, a,
                        box, (int)rows));
  return SUB_OK;
}

}  // namespace

int32_t launch_chunk_mid(const ChunkArgs& a, bool q8, int head_dim, int rows, int64_t pool_rows, int n_ctas,
                         cudaStream_t st) {
  auto k = rows == 32 ? (q8 ? (head_dim == 128 ? launch<128, true, 32> : launch<64, true, 32>)
                            : (head_dim == 128 ? launch<128, false, 32> : launch<64, false, 32>))
                      : (q8 ? (head_dim == 128 ? launch<128, true, 64> : launch<64, true, 64>)
                            : (head_dim == 128 ? launch<128, false, 64> : launch<64, false, 64>));
  return k(a, pool_rows, n_ctas, st);
}

int32_t chunk_mid_timeouts(unsigned int* out) {
  SUB_CUDA_TRY(cudaMemcpyFromSymbol(out, g_mid_timeouts, sizeof(unsigned int)));
  return SUB_OK;
}

}  // namespace sub
