// Attention of new rows over a paged cache, many rows per sequence: chunks of a
// prompt, on the 5th-generation tensor cores.
//
// The same sums as chunk_attn.cu, in tiles of 256 (row, head in group) pairs x
// 128 keys.  Bound by the tensor cores: a block costs six products of 128 x 128 x D
// (codes: four) and 2 * 128 * 128 exponentials.
// Measured: 2048 rows of 32 heads behind 14336 keys 470 to 484 us, 1070 TFLOP/s (0.55 of
// a plain bf16 matrix product of the library) that are counted, 1600 with the
// weights' second halves; over codes three prompts of up to 1537 rows of 28
// heads behind up to 2600 keys 196 us, 645 TFLOP/s, bounded by the converter warps: of a
// block's 4000 cycles 3200 are its conversion.  1024 rows of 32 heads behind 7000 keys:
// 138 us, over codes 146.  (The softmax warps' registers hold a row's 128 scores and
// little else: 370 to 640 bytes per thread are spilled.)
// So two groups of 128 rows alternate: while the tensor cores form one group's
// scores or output, the four warps of the other turn scores into weights.
//   warps 0-3, 4-7   softmax of rows 0-127 and 128-255, one row per thread (a
//                    row's maximum and sum need no exchange between threads),
//                    the Q tile's way into shared memory, and the results
//   a producer       blocks of 128 keys into a ring, V of one beside K of the next
//                    (they are used together): a TMA warp for a bf16 cache (boxes of as many keys
//                    as a page holds together), or eight warps that turn 8-bit
//                    codes into fp16 values on the way
//   two warps        (codes) that look the blocks' keys up and gather their scales ahead
//   one MMA warp     S = Q K^T into tensor memory; then, once the group's weights
//                    are there, O += P V with P read from tensor memory (in
//                    place of S, as two bf16 halves or as fp16) and S of the next block
// O stays in tensor memory.  It is rescaled only when a row's maximum has grown
// by more than 2^8 (codes: 2^4) since the weights' reference was set: until then the
// weights exceed 1 by at most that factor, which costs a floating-point value nothing.
// Over a bf16 cache P = hi + lo, two bf16 products, like in the few rows' kernel (2^-16 of
// a weight): a token's row rounds alike, whether it is decoded, verified or part
// of a prompt.  (One product, P rounded to bf16, took 362 us of the 2048 rows; its error
// against 64 bits was a third more, as much as the result's own rounding.)  Over codes P
// is rounded once, to fp16, three bits finer; the sums take the unrounded weights.
//
// Codes become fp16 values on the way, (code - 128) * scale relative to the power
// of two of the block's largest scale, rounded to half a step of 2^-11 (three bits
// finer than the bf16 values of the other cache): the power of K's scales goes into
// the scores' factor, that of V's into the weights.  (Scales applied to scores and weights,
// column by column, would be exact, but cost every row 2 * 128 reads of shared
// memory per block: the softmax then took 2.7 times as long.)  K's scale enters in two
// fp16 parts, so that its rounding is not common to all terms of a score; V's in one,
// like a rounding of the weight.  Values are up to 2^15, near the end of fp16: a scale
// may be 2^-21 of the block's largest before it loses a bit.
//
// That power of two is a choice for all rows, so it may come from keys that all
// rows read, only.  In a block that not all rows read to its end the operands are the bare
// codes, and each row applies the scales of its own keys, column by column, with the
// largest of those for its power of two: one or two blocks of a tile, which take about
// 6000 cycles more (the prompts 196 us; 179 with one power of two there, too).
//
// V rows past the tile's last key hold anything, and so may keys of the chunk
// that only later rows read.  In blocks that not all rows read to the end the first
// group's warps look through V: rows past the end and values that are not
// finite become 0, and if there were any of these, each row adds those that it does
// read to its result (whatever is added to them, it stays infinite or NaN).
#include <cuda_fp16.h>
#include "chunk_attn.cuh"
#include "gemv.cuh"
#include "tma.cuh"

namespace sub {
namespace {

using namespace tmah;

constexpr int RT = CHUNK_TC_ROWS, KB = CHUNK_TC_KEYS;
static_assert(RT == 256 && KB == 128, "two groups of 128 rows, blocks of 128 keys");
constexpr int GROUP_ROWS = 128;
// log2 of how far weights may exceed 1; fp16 weights times scales of V are 2^11 at
// the reference and 2^15 at most, so that fp16's smallest step is 2^-35 of the former
constexpr float growth(bool q8) { return q8 ? 4.f : 8.f; }
constexpr float Q8_SHIFT = 11.f;
// log2 of what the values formed from codes are relative to the scales' power of two, and
// the least exponents of that of K and of V (V: sums of weights times 2^-(VALUE_MIN -
// VALUE_UP) stay in range)
constexpr int VALUE_UP = 7, KEY_MIN = VALUE_UP - 126, VALUE_MIN = VALUE_UP - 80;

__device__ unsigned int g_chunk_timeouts;   // waits that ran out (never expected)

template <int D, bool Q8>
struct Cfg {
  static constexpr int HALF = KB * D * 2;                // K or V of a block, 16-bit values
  static constexpr int SLOT = 2 * HALF;                  // V of a block, K of the next
  static constexpr int SLOTS = D == 64 ? 3 : 2;
  static constexpr int Q_BYTES = GROUP_ROWS * D * 2;     // of one group
  static constexpr int CONV = Q8 ? 8 : 0;                // converter warps
  static constexpr int MMA_WARP = 8 + (Q8 ? CONV : 1);
  static constexpr int PLAN = Q8 ? 2 : 0;                // then warps that look the keys up
  static constexpr int THREADS = Q8 ? 640 : 384;         // whole groups of four warps
  // registers by group of four warps, out of 65536 / THREADS each at the launch
  // (bf16: the producer and the MMA warp share one)
  static constexpr int REGS_SOFTMAX = Q8 ? 160 : 192;
  static constexpr int REGS_PROD = Q8 ? 56 : 120;
  static constexpr int REGS_MMA = Q8 ? 48 : 120;
  static_assert((2 * REGS_SOFTMAX + (Q8 ? CONV / 4 : 1) * REGS_PROD + (Q8 ? REGS_MMA : 0)) * 128 <=
                    65536 / THREADS / 8 * 8 * THREADS,
                "the shares fit what the block is launched with");
  // eight blocks' scales of K, of V; the largest of K's by warp, whether operands are the
  // bare codes by warp, the largest of V's by warp; for the softmax the power of two of
  // K's and the exponent of V's
  static constexpr int SCALE_SLOT = 2 * KB + 12;
  static constexpr int SCALES = Q8 ? 8 * SCALE_SLOT * 4 : 0;
  static constexpr int QSCALES = Q8 ? RT * 4 : 0;
  static constexpr int ROWS = Q8 ? 4 * KB * 4 : 0;       // pool rows of four blocks' keys
  static constexpr int TAIL = 256;                       // barriers, flags, TMEM address
  static constexpr int SMEM =
      1024 + 2 * Q_BYTES + SLOTS * SLOT + SCALES + QSCALES + ROWS + TAIL;
  static_assert(SMEM <= 227 * 1024, "one CTA's shared memory");
  static_assert(SLOTS * SLOT >= (SUB_MAX_SEQS + 1) * 8, "the ring holds the running sums first");
};

// ---------------------------------------------------------------- tcgen05 --
// Shared-memory descriptors of operands in the 128-byte swizzle.  K-major (Q, K:
// rows of 64 values): stride 1024 between groups of 8 rows.  MN-major (V: a key
// is a row of 64 columns): 1024 between groups of 8 keys, and the next 64 columns a
// whole block of keys further.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)((KB * 128u) >> 4) << 16 |
         (uint64_t)(1024u >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f16, fp32 accumulator, M = 128; both operands bf16 (1) or fp16 (0).
__device__ constexpr uint32_t idesc(int n, bool bf16, bool b_mn) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 columns of the warp's 32 lanes, one lane per thread; wait_ld before use.
__device__ __forceinline__ void tc_ld32(uint32_t t, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t t, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ bool elect_one() {   // by a whole warp: one lane
  uint32_t x;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(x));
  return x != 0;
}

// Bounded wait.  One that runs out is counted and ends the CTA's work: every
// later wait returns at once, nothing more is issued, and the results are not valid.
struct Gate {
  volatile int* dead;
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return true;
    for (uint32_t i = 0; i < (1u << 20); ++i) {
      if (mbar_try_wait(bar, parity)) return true;
      if ((i & 63) == 63 && *dead) return false;
    }
    if (!*dead) {
      *dead = 1;
      atomicAdd(&g_chunk_timeouts, 1u);
    }
    return false;
  }
  // by a whole warp, which goes on or stops together
  __device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) const {
    return __all_sync(~0u, wait(bar, parity));
  }
};

// Bit of a block's 16-key part in its word of missing pages: the TMA warp writes
// the word, the warps that look keys up a byte per 32 keys.
template <bool Q8>
__device__ constexpr int miss_bit(int part) {
  return Q8 ? 8 * (part >> 1) + (part & 1) : part;
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Converters and the warps that look keys up, once per block.
template <int WARPS>
__device__ __forceinline__ void meet_planners() {
  asm volatile("bar.sync 3, %0;" ::"n"(WARPS * 32) : "memory");
}

struct Maps {
  CUtensorMap k, v;   // pool rows [all rows, D] bf16, boxes of 64 columns x box keys
};

__device__ __forceinline__ void st_shared(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
// 32 bytes at once: a row is written by one thread, and this fills whole sectors.
__device__ __forceinline__ void st_global32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// ------------------------------------------------------------------ kernel --
template <int D, bool Q8>
__global__ void __launch_bounds__(Cfg<D, Q8>::THREADS, 1)
chunk_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ ChunkArgs a, const int box,
                const int pool_rows) {
  using C = Cfg<D, Q8>;
  constexpr int SLOTS = C::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const base_p = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t q_s = base, ring_s = base + 2 * C::Q_BYTES;
  int64_t* const s_pre = reinterpret_cast<int64_t*>(base_p + 2 * C::Q_BYTES);   // until the first copies
  uint8_t* const after = base_p + 2 * C::Q_BYTES + SLOTS * C::SLOT;
  float* const s_scale = reinterpret_cast<float*>(after);                   // [8][SCALE_SLOT]
  float* const s_qs = reinterpret_cast<float*>(after + C::SCALES);          // [RT]
  int* const s_rows = reinterpret_cast<int*>(after + C::SCALES + C::QSCALES);   // [4][KB]
  uint8_t* const tail = after + C::SCALES + C::QSCALES + C::ROWS;
  const uint32_t bars = smem_u32(tail);
  auto kv_full = [&](uint32_t block) { return bars + 8u * (block % SLOTS); };
  auto kv_empty = [&](uint32_t block) { return bars + 8u * (SLOTS + block % SLOTS); };
  auto q_full = [&](int t) { return bars + 8u * (2 * SLOTS + t); };
  auto s_full = [&](int t) { return bars + 8u * (2 * SLOTS + 2 + t); };
  auto p_full = [&](int t) { return bars + 8u * (2 * SLOTS + 4 + t); };
  auto o_full = [&](int t) { return bars + 8u * (2 * SLOTS + 6 + t); };
  int* const flags = reinterpret_cast<int*>(tail + 8 * (2 * SLOTS + 8));
  volatile int* const s_dead = flags;            // a wait ran out
  // [group][2] the piece that met infinite values or NaN, for each group by the parity of
  // the pieces that it takes part in: the first group, which finds them, gets two such pieces
  // ahead of the second only after the second is through with the older one
  volatile int* const s_odd = flags + 1;
  volatile uint32_t* const s_miss = reinterpret_cast<uint32_t*>(flags + 5);   // [8] blocks' missing 16-key parts
  uint32_t* const s_tmem = reinterpret_cast<uint32_t*>(flags + 13);
  static_assert(8 * (2 * SLOTS + 8) + 14 * 4 <= C::TAIL, "tail");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(s_tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32) {
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(kv_full(s), Q8 ? C::CONV : 1);
      mbar_init(kv_empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 4);   // one arrival for each warp of the group
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t), 4);
      mbar_init(o_full(t), 1);
    }
    *s_dead = 0;
    for (int i = 0; i < 4; ++i) s_odd[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (!Q8 && tid == 64) {
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  pdl_wait();
  pdl_trigger();
  const ChunkPlan<RT, KB> plan(a);
  tc_fence_before();
  plan.template scan<C::THREADS>(s_pre);   // ends with a barrier
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int64_t total = s_pre[a.t.n_seqs];
  const int64_t per = blocks_per_cta(total, gridDim.x, CHUNK_TC_LEAST);
  const int64_t line_lo = blockIdx.x * per, line_hi = min(total, line_lo + per);
  ChunkUnit u;
  if (line_lo < line_hi) u = plan.find(s_pre, line_lo);
  fence_async();     // the ring is written by copies from here on
  __syncthreads();
  const Gate gate{s_dead};
  const int G = a.group;
  // Slot j of the ring holds V of block j - 1 and K of block j, across the units;
  // the first has no V, the last no K.
  const uint32_t n = (uint32_t)(line_hi > line_lo ? line_hi - line_lo : 0);
  int kb = (int)(line_lo - u.begin);   // the next block to look up, of unit u
  // pool row of key x of that block; -1: past the last key, -2: on no page
  auto row_of = [&](int x) {
    const int key = kb * KB + x;
    if (key >= u.n_keys) return -1;
    const int entry = a.by_page.quot(key), page = a.t.pages[(int64_t)u.b * a.t.width + entry];
    if ((unsigned)page >= (unsigned)a.t.n_pages) return -2;
    return (int)pool_row(a.t, a.layer, a.n_heads_kv, page, u.head, key - entry * a.t.page_size);
  };
  auto step = [&] {
    if (++kb == u.n_blocks) {
      plan.next(u);
      kb = 0;
    }
  };

  if (warp < 8) more_registers<C::REGS_SOFTMAX>();
  else if (!Q8 || warp < 8 + C::CONV) fewer_registers<C::REGS_PROD>();
  else fewer_registers<C::REGS_MMA>();

  if (warp < 8) {
    // ------------------------------------------------ softmax, Q, results
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;   // group, row in it
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + t * 128 + lanes, tO = tmem + 256 + t * 128 + lanes;
    uint32_t n_s = 0, n_o = 0;      // blocks and pieces seen by this group
    uint32_t block = 0;             // of this CTA's part of the line
    constexpr int CH = D / 8, RP = 32 / CH;   // 16-byte chunks of a Q row, rows per pass of a warp
    const int c = lane % CH;

    // Q of a unit's group, first into registers, then into shared memory: chunk c of
    // a row at c ^ (row % 8) of its 128-byte line, each warp its own threads' rows
    auto group_has_rows = [&](const ChunkUnit& x, int g) { return x.tile * RT + g * GROUP_ROWS < x.rows * G; };
    auto has_rows = [&](const ChunkUnit& x) { return group_has_rows(x, t); };
    auto q_load = [&](const ChunkUnit& x, uint4 (&w)[CH]) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int row = x.tile * RT + t * GROUP_ROWS + (warp & 3) * 32 + i * RP + lane / CH;
        const int q = a.by_group.quot(row);
        w[i] = make_uint4(0, 0, 0, 0);
        if (q < x.rows)
          w[i] = ldg_cg_v4(a.Q + (int64_t)(x.row0 + q) * a.ldq + (int64_t)(x.head * G + row - q * G) * D +
                           c * 8);
      }
    };
    auto q_store = [&](uint4 (&w)[CH]) {
      const uint32_t dst0 = q_s + t * C::Q_BYTES + (c >> 3) * (GROUP_ROWS * 128);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int rr = (warp & 3) * 32 + i * RP + lane / CH;
        if constexpr (Q8) {
          // the row's largest value to [1, 2), for fp16
          const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          float big = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            big = fmaxf(big, fmaxf(fabsf(bf16lo(x[k])), fabsf(bf16hi(x[k]))));
#pragma unroll
          for (int o = CH / 2; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
          const int e = min(126, max(-126, (int)(__float_as_uint(big) >> 23) - 127));
          const float down = __uint_as_float((uint32_t)(127 - e) << 23);
          // (not 0: it meets the masked scores' -infinity)
          if (c == 0)
            s_qs[t * GROUP_ROWS + rr] = fmaxf(a.sl2 * __uint_as_float((uint32_t)(127 + e) << 23), 1e-37f);
          w[i].x = pack_f16x2(bf16lo(x[0]) * down, bf16hi(x[0]) * down);
          w[i].y = pack_f16x2(bf16lo(x[1]) * down, bf16hi(x[1]) * down);
          w[i].z = pack_f16x2(bf16lo(x[2]) * down, bf16hi(x[2]) * down);
          w[i].w = pack_f16x2(bf16lo(x[3]) * down, bf16hi(x[3]) * down);
        }
        st_shared(dst0 + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), w[i].x, w[i].y, w[i].z, w[i].w);
      }
      fence_async();
      __syncwarp();   // (s_qs, too)
      if (lane == 0) mbar_arrive(q_full(t));
    };
    // (also for a CTA that stops early because a wait ran out)
    if (tid == 0) a.cuts[blockIdx.x].pieces = 0;
    bool q_there = false;   // this piece's Q is in shared memory already
    int piece = 0;
    int both = 0;   // pieces so far that the second group took part in
    for (int64_t at = line_lo; at < line_hi; ++piece) {
      const int kb0 = (int)(at - u.begin), kb1 = (int)min((int64_t)u.n_blocks, line_hi - u.begin);
      const bool first = at == line_lo;
      at = u.begin + kb1;
      if (tid == 0 && at >= line_hi) a.cuts[blockIdx.x] = make_cut(u, kb1, line_lo, per);
      if (!has_rows(u)) {   // an empty second group
        block += kb1 - kb0;
        plan.next(u);
        continue;
      }
      if (!q_there) {
        uint4 w[CH];
        q_load(u, w);
        q_store(w);
      }
      const int row = u.tile * RT + t * GROUP_ROWS + r, q = a.by_group.quot(row);
      const bool real = q < u.rows;
      const int n_keys = u.n_keys;
      const int lim = real ? last_key(u.pos, q, n_keys) : -1;                         // keys 0 .. lim are read
      const int lim_first = last_key(u.pos, a.by_group.quot(u.tile * RT), n_keys);    // by every row of the tile
      float factor = a.sl2;        // of the row's scores, to base 2
      if constexpr (Q8) factor = s_qs[t * GROUP_ROWS + r];

      float ref = 0.f, l = 0.f;    // weights are 2^(score - ref)
      bool any = false;            // a key has been read
      for (int kb = kb0; kb < kb1; ++kb, ++block) {
        const int key0 = kb * KB;
        if (!gate.wait_warp(s_full(t), n_s & 1)) break;
        ++n_s;
        tc_fence_after();
        const uint32_t miss = s_miss[block & 7];
        const bool behind = key0 + KB - 1 > lim_first;   // the same for all rows of the tile
        const int last = lim - key0;                     // columns past it are not read
        const float* const sc = s_scale + (block & 7) * C::SCALE_SLOT;
        float lv = 0.f;   // log2 of what V's scales add to the weights
        float2 sum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.f, 0.f);
        // the reference, and the output that was formed with another
        auto raise = [&](float top) {
          const bool grow = top > ref + growth(Q8) || (!any && top != -INFINITY);
          if (!__any_sync(~0u, grow)) return;
          const float less = grow && any ? exp2_fast(ref - top) : 1.f;
          if (grow) {
            ref = top;
            any = true;
          }
          l *= less;
          if (kb > kb0 && __any_sync(~0u, less != 1.f)) {
#pragma unroll 1
            for (int x = 0; x < D; x += 16) {
              float o[16];
              __syncwarp();
              tc_ld16(tO + x, o);
              wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= less;
              tc_st16(tO + x, reinterpret_cast<const uint32_t*>(o));
            }
          }
        };
        if (Q8 && behind) {
          // Bare codes: this row's scales, in two walks over the columns.  (As loops: the
          // code of all 128 columns at once, which a tile runs once or twice, was fetched
          // again each time: the prompts took 229 us, against 196.)
          const float f = fmaxf(factor * (1.f / (1 << VALUE_UP)), 1e-37f);
          float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, vmax4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int x0 = 0; x0 < KB; x0 += 32) {
            float s[32];
            __syncwarp();
            tc_ld32(tS + x0, s);
            wait_ld();
            const uint32_t gone = miss >> miss_bit<Q8>(x0 >> 4);
            const int end = last - x0;
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const float4 k4 = *reinterpret_cast<const float4*>(sc + x0 + x);
              const float4 v4 = *reinterpret_cast<const float4*>(sc + KB + x0 + x);
              const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, vv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const bool unread = x + i > end;
                s[x + i] = unread ? -INFINITY : s[x + i] * kk[i];
                vmax4[i] = fmaxf(vmax4[i], unread ? 0.f : vv[i]);   // (0 where there is no page)
              }
            }
            if (gone & 3u) {
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if ((gone >> miss_bit<Q8>(x >> 4)) & 1u) s[x] = -INFINITY;
            }
#pragma unroll
            for (int x = 0; x < 32; ++x) top4[x & 3] = fmaxf(top4[x & 3], s[x]);
            tc_st16(tS + x0, reinterpret_cast<const uint32_t*>(s));
            tc_st16(tS + x0 + 16, reinterpret_cast<const uint32_t*>(s + 16));
          }
          wait_st();
          const float vmax = fmaxf(fmaxf(vmax4[0], vmax4[1]), fmaxf(vmax4[2], vmax4[3]));
          const int e = max(VALUE_MIN, (int)(__float_as_uint(vmax) >> 23) - 127) + 1;   // vmax < 2^e
          const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
          raise(top == -INFINITY ? top : fmaf(top, f, (float)(e - VALUE_UP)));
          const float shift = Q8_SHIFT - (float)VALUE_UP - ref;
          lv = (float)-VALUE_UP;
#pragma unroll 1
          for (int x0 = 0; x0 < KB; x0 += 32) {
            float s[32];
            __syncwarp();
            tc_ld32(tS + x0, s);
            wait_ld();
            uint32_t pw[16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float4 v = *reinterpret_cast<const float4*>(sc + KB + x0 + 2 * i);   // all finite
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float2 w = make_float2(exp2_fast(fmaf(s[2 * (i + k)], f, shift)),
                                             exp2_fast(fmaf(s[2 * (i + k) + 1], f, shift)));
                sum[(i + k) & 3] = add2(sum[(i + k) & 3], w);
                pw[i + k] = pack_f16x2(w.x * (k ? v.z : v.x), w.y * (k ? v.w : v.y));
              }
            }
            tc_st16(tS + x0 / 2, pw);   // over columns that are read already
          }
        } else {
          const bool edge = behind || miss;
          float s[KB];
#pragma unroll
          for (int x = 0; x < KB; x += 32) tc_ld32(tS + x, s + x);
          float f = factor;
          if constexpr (Q8) {   // the block's powers of two (not 0: it meets the masked scores' -infinity)
            const float2 pw = *reinterpret_cast<const float2*>(sc + 2 * KB + 8);
            f = fmaxf(factor * pw.x, 1e-37f);
            lv = pw.y;
          }
          wait_ld();
          if (edge) {
#pragma unroll
            for (int x = 0; x < KB; ++x)
              if (x > last || ((miss >> miss_bit<Q8>(x >> 4)) & 1u)) s[x] = -INFINITY;
          }
          // eight chains: a single one would wait for itself 128 times
          float top8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) top8[i] = fmaxf(s[i], s[i + 8]);
#pragma unroll
          for (int x = 16; x < KB; x += 16)
#pragma unroll
            for (int i = 0; i < 8; ++i) top8[i] = fmaxf(fmaxf(top8[i], s[x + i]), s[x + 8 + i]);
          const float top = fmaxf(fmaxf(fmaxf(top8[0], top8[1]), fmaxf(top8[2], top8[3])),
                                  fmaxf(fmaxf(top8[4], top8[5]), fmaxf(top8[6], top8[7])));
          // what is rounded to fp16 is the weight times the power of two of V's scales
          raise(top == -INFINITY ? top : fmaf(top, f, lv));
          if (!Q8 && behind && t == 0) {
            // V of the block: row r of it is this thread's
            if (!gate.wait_warp(kv_full(block + 1), ((block + 1) / SLOTS) & 1)) break;
            const uint32_t v0 = ring_s + (block + 1) % SLOTS * C::SLOT + r * 128;
            const bool past = key0 + r >= n_keys;
            uint32_t z = 0;   // 0 * x is NaN for what is not finite
#pragma unroll 1
            for (int i = 0; i < D / 8; ++i) {
              const uint32_t at16 = v0 + (i >> 3) * (KB * 128) + (((i ^ r) & 7) << 4);
              if (past) {
                st_shared(at16, 0, 0, 0, 0);
              } else {
                const uint4 v = lds128(at16);
                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(z) : "r"(x[k]), "r"(0u));
              }
            }
            if ((z & 0x7fff7fffu) != 0) {   // hardly ever: take them out, add them at the end
#pragma unroll 1
              for (int i = 0; i < D / 8; ++i) {
                const uint32_t at16 = v0 + (i >> 3) * (KB * 128) + (((i ^ r) & 7) << 4);
                const uint4 v = lds128(at16);
                uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if ((x[k] & 0x7f80u) == 0x7f80u) x[k] &= 0xffff0000u;
                  if ((x[k] & 0x7f800000u) == 0x7f800000u) x[k] &= 0x0000ffffu;
                }
                st_shared(at16, x[0], x[1], x[2], x[3]);
              }
              s_odd[piece & 1] = piece + 1;
              if (group_has_rows(u, 1)) s_odd[2 + (both & 1)] = piece + 1;
            }
            fence_async();
            __syncwarp();
          }
          // ---- weights, in place of the scores' first columns ----
          const float shift = Q8 ? Q8_SHIFT + lv - ref : -ref;
          const float2 f2 = make_float2(f, f), d2 = make_float2(shift, shift);
#pragma unroll
          for (int x0 = 0; x0 < KB; x0 += 32) {
            uint32_t pw[16], rest[16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const int x = x0 + 2 * i;
              float2 e[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                e[k] = fma2(make_float2(s[x + 2 * k], s[x + 2 * k + 1]), f2, d2);
                e[k].x = exp2_fast(e[k].x);
                e[k].y = exp2_fast(e[k].y);
                sum[(i + k) & 3] = add2(sum[(i + k) & 3], e[k]);
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                if constexpr (Q8) {
                  pw[i + k] = pack_f16x2(e[k].x, e[k].y);
                } else {
                  const uint32_t w = pack_bf16x2(e[k].x, e[k].y);
                  pw[i + k] = w;
                  const float2 r = add2(e[k], make_float2(-bf16lo(w), -bf16hi(w)));
                  rest[i + k] = pack_bf16x2(r.x, r.y);
                }
              }
            }
            tc_st16(tS + x0 / 2, pw);
            if constexpr (!Q8) tc_st16(tS + KB / 2 + x0 / 2, rest);
          }
        }
        wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(t));
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l = fmaf(sum[0].x + sum[0].y, Q8 ? exp2_fast(-lv) : 1.f, l);
      }
      // ---- the next piece's Q takes this one's place as soon as the products are
      // through, so that its scores are formed while the result is written ----
      const ChunkUnit done = u;
      plan.next(u);
      q_there = at < line_hi && has_rows(u);
      bool through;
      if (q_there) {
        uint4 w[CH];
        q_load(u, w);
        through = gate.wait_warp(o_full(t), n_o & 1);
        if (through) q_store(w);
      } else {
        through = gate.wait_warp(o_full(t), n_o & 1);
      }
      if (!through) break;
      ++n_o;
      tc_fence_after();
      const bool whole = kb0 == 0 && kb1 == done.n_blocks;
      const bool odd = !Q8 && s_odd[t ? 2 + (both & 1) : piece & 1] == piece + 1;
      both += group_has_rows(done, 1);
      const float mul = whole ? (any ? 1.f / l : 0.f) : 1.f;
      uint16_t* const out = a.O + ((int64_t)(done.row0 + q) * a.n_heads_q + done.head * G + row - q * G) * D;
      const int64_t part_row = (2 * (int64_t)blockIdx.x + (first ? 0 : 1)) * RT + t * GROUP_ROWS + r;
#pragma unroll 1
      for (int x0 = 0; x0 < D; x0 += 32) {
        float o[32];
        __syncwarp();
        tc_ld32(tO + x0, o);
        wait_ld();
        if (odd && real) {
          // values that are not finite, of the keys this row reads in the blocks looked through
          const uint16_t* const vp = reinterpret_cast<const uint16_t*>(a.v);
          const int from = max(kb0, max(0, lim_first + 1) / KB) * KB;
          for (int key = from; key <= min(lim, kb1 * KB - 1); ++key) {
            const int page = page_of(a.t, done.b, key);
            if (page < 0) continue;
            const uint16_t* const x =
                vp + pool_row(a.t, a.layer, a.n_heads_kv, page, done.head,
                              (int)((uint32_t)key % (uint32_t)a.t.page_size)) * D + x0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const uint16_t bits = __ldcg(x + i);
              if ((bits & 0x7f80u) == 0x7f80u) o[i] += bf16_bits_to_f32(bits);
            }
          }
        }
        if (real && whole) {
          uint32_t b[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) b[i] = pack_bf16x2(o[2 * i] * mul, o[2 * i + 1] * mul);
          if ((reinterpret_cast<uintptr_t>(a.O) & 31) == 0) {
            st_global32(out + x0, b);
            st_global32(out + x0 + 16, b + 8);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(out + x0 + 8 * i) =
                  make_uint4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
          }
        } else if (real) {
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            st_global32(a.part_o + part_row * D + x0 + i, reinterpret_cast<const uint32_t*>(o + i));
        }
      }
      if (!whole && real)
        __stcg(a.part_ml + part_row, make_float2(any ? ref : -INFINITY, l));
      __syncwarp();
      tc_fence_before();   // O is read before the next piece's first weights are announced
      if (*s_dead) break;
    }
  } else if (Q8 ? warp >= 8 + C::CONV : warp > 8) {
    if (warp == C::MMA_WARP) {
      // -------------------------------------------------------- MMA issuer
      // The whole warp walks through this, with values that the compiler can see to be
      // the same in all lanes, and elects the lane that issues: descriptors then stay in
      // uniform registers (an issue from a lane of its own choice has to move them
      // there each time, which took longer than the product).
      constexpr uint32_t id_s = idesc(KB, !Q8, false), id_o = idesc(D, !Q8, true);
      const uint32_t tm = __shfl_sync(~0u, tmem, 0);
      uint32_t block = 0, n_q[2] = {0, 0}, n_p[2] = {0, 0};
      // descriptors of the first step; a step further is a constant in the address field
      const uint64_t q_desc = desc_k(q_s), v_desc = desc_mn(ring_s), k_desc = desc_k(ring_s + C::HALF);
      auto full = [&](uint32_t b) { return gate.wait_warp(kv_full(b), (b / SLOTS) & 1); };
      auto scores = [&](int t, uint32_t b) {
        if (elect_one()) {
          const uint64_t qd = q_desc + t * (C::Q_BYTES >> 4), kd = k_desc + b % SLOTS * (C::SLOT >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * (KB * 128) + (k & 3) * 32) >> 4;
            mma_ss(tm + t * 128, qd + off, kd + off, id_s, k > 0);
          }
          tc_commit(s_full(t));
        }
        __syncwarp();
      };
      auto output = [&](int t, uint32_t b, bool add) {   // V of block b lies beside K of the next
        if (elect_one()) {
          const uint64_t vd = v_desc + (b + 1) % SLOTS * (C::SLOT >> 4);
#pragma unroll
          for (int k = 0; k < KB / 16; ++k) {
            mma_ts(tm + 256 + t * 128, tm + t * 128 + k * 8, vd + k * (2048 >> 4), id_o, add || k > 0);
            if constexpr (!Q8)   // the weights' second halves
              mma_ts(tm + 256 + t * 128, tm + t * 128 + KB / 2 + k * 8, vd + k * (2048 >> 4), id_o, true);
          }
        }
        __syncwarp();
      };
      auto commit = [&](uint32_t bar) {
        if (elect_one()) tc_commit(bar);
        __syncwarp();
      };
      bool ok = line_lo < line_hi && full(0);
      for (int64_t at = line_lo; at < line_hi && ok; plan.next(u)) {
        const int kb0 = (int)(at - u.begin), kb1 = (int)min((int64_t)u.n_blocks, line_hi - u.begin);
        at = u.begin + kb1;
        const int n = __shfl_sync(~0u, kb1 - kb0, 0);
        const int groups = __shfl_sync(~0u, u.tile * RT + GROUP_ROWS < u.rows * G ? 2 : 1, 0);
        for (int t = 0; t < groups && ok; ++t) {
          ok = gate.wait_warp(q_full(t), n_q[t]++ & 1);
          if (ok) scores(t, block);
        }
        if (!ok) break;
        commit(kv_empty(block));
        for (int i = 0; i < n && ok; ++i, ++block) {
          ok = full(block + 1);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == groups || !ok) break;
            ok = gate.wait_warp(p_full(t), n_p[t]++ & 1);
            if (!ok) break;
            tc_fence_after();
            output(t, block, i > 0);
            if (i + 1 < n) scores(t, block + 1);
            else commit(o_full(t));
          }
          if (ok && i + 1 < n) commit(kv_empty(block + 1));
        }
      }
    } else if (Q8 && warp <= C::MMA_WARP + C::PLAN) {
      // ------------------------------------- pool rows and scales of the keys
      // Two blocks, and one block, ahead of the conversion.  (By the converters
      // themselves, four of the eight took half as long again for a block as the others.)
      constexpr int KEYS = KB / 64;   // per lane: keys x0, x0 + 32
      static_assert(C::PLAN != 1 && KEYS == 2, "two warps, two keys per lane");
      const int pw = warp - C::MMA_WARP - 1, x0 = pw * 64 + lane;
      float ksc[KEYS], vsc[KEYS];
      unsigned gone[KEYS];            // of 32 keys: which stand on no page
      uint32_t bare = 0;              // bit j % 32: not all rows read block j to its end
      auto look_up = [&](uint32_t j) {   // called for j = 0, 1, ..
        if (j >= n) return;
        if (j > 0) step();
        const bool behind = kb * KB + KB - 1 > last_key(u.pos, a.by_group.quot(u.tile * RT), u.n_keys);
        bare = (bare & ~(1u << (j & 31))) | (uint32_t)behind << (j & 31);
        int row[KEYS];
#pragma unroll
        for (int h = 0; h < KEYS; ++h) row[h] = row_of(x0 + 32 * h);
#pragma unroll
        for (int h = 0; h < KEYS; ++h) s_rows[(j & 3) * KB + x0 + 32 * h] = row[h];
      };
      auto load_scales = [&](uint32_t j) {
        if (j >= n) return;
#pragma unroll
        for (int h = 0; h < KEYS; ++h) {
          const int row = s_rows[(j & 3) * KB + x0 + 32 * h];
          gone[h] = __ballot_sync(~0u, row == -2);
          ksc[h] = row >= 0 ? __ldcg(a.ks + row) : 0.f;
          vsc[h] = row >= 0 ? __ldcg(a.vs + row) : 0.f;
        }
      };
      auto store_scales = [&](uint32_t j) {
        if (j >= n) return;
        float* const sc = s_scale + (j & 7) * C::SCALE_SLOT;
        float kx = 0.f, vx = 0.f;
#pragma unroll
        for (int h = 0; h < KEYS; ++h) {
          // a row that reads a key whose scale of V is not finite gets NaN by its
          // score; weight 0 times it stays 0
          const bool fine = vsc[h] < INFINITY;
          sc[x0 + 32 * h] = fine ? ksc[h] : __int_as_float(0x7fc00000);
          sc[KB + x0 + 32 * h] = fine ? vsc[h] : 1.f;
          kx = fmaxf(kx, ksc[h] < INFINITY ? ksc[h] : 0.f);
          vx = fmaxf(vx, fine ? vsc[h] : 0.f);
        }
        kx = warp_max(kx);
        vx = warp_max(vx);
        if (lane == 0) {
          sc[2 * KB + pw] = kx;
          sc[2 * KB + 2 + pw] = (float)((bare >> (j & 31)) & 1u);
          sc[2 * KB + 4 + pw] = vx;
#pragma unroll
          for (int h = 0; h < KEYS; ++h)   // 16-key parts: bits 0 and 16 of 32 keys
            reinterpret_cast<volatile uint8_t*>(s_miss + (j & 7))[2 * pw + h] =
                (uint8_t)((gone[h] & 1u) | ((gone[h] >> 16) & 1u) << 1);
        }
      };
      look_up(0);
      look_up(1);
      meet_planners<C::CONV + C::PLAN>();
      load_scales(0);
      store_scales(0);
      meet_planners<C::CONV + C::PLAN>();
      for (uint32_t j = 0; j <= n && n > 0; ++j) {
        load_scales(j + 1);
        look_up(j + 2);
        store_scales(j + 1);
        meet_planners<C::CONV + C::PLAN>();
      }
    }
  } else {
    // ------------------------------------------------------------ producers
    bool ok = true;
    if constexpr (!Q8) {
      // lanes 0..15 move K, 16..31 V: 64 columns (lane & 1) of the boxes (lane & 15) / 2, ..
      const int half = lane & 1, side = lane >> 4, b0 = (lane & 15) >> 1;
      const int n_box = KB / box;
      const bool mine = b0 < n_box && half < D / 64;
      int row = n > 0 && b0 < n_box ? row_of(b0 * box) : -1, before = -1;
      uint32_t j = 0;
      for (; j <= n && n > 0; ++j) {
        // 16-key parts without a page (those past the last key count as read past the end)
        const unsigned gone = __ballot_sync(~0u, side == 0 && half == 0 && row == -2);
        // rows of the pool, one per box; past the pool (zeros) where there is no page
        const int y = side ? before : row;
        before = row;
        if (j + 1 < n) {   // a block ahead
          step();
          row = b0 < n_box ? row_of(b0 * box) : -1;
        }
        if (j >= SLOTS) ok = gate.wait_warp(kv_empty(j), ((j / SLOTS) - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          uint32_t miss = 0;
          if (gone)
            for (int b = 0; b < n_box; ++b)
              if ((gone >> (2 * b)) & 1u) miss |= ((1u << (box / 16)) - 1u) << (b * box / 16);
          if (j < n) s_miss[j & 7] = miss;
          mbar_expect_tx(kv_full(j), (j > 0 ? C::HALF : 0) + (j < n ? C::HALF : 0));
        }
        __syncwarp();
        if (mine && (side ? j > 0 : j < n))
          tma_load_2d(ring_s + j % SLOTS * C::SLOT + (side ? 0 : C::HALF) + half * (KB * 128) +
                          b0 * box * 128,
                      side ? &maps.v : &maps.k, half * 64, y < 0 ? pool_rows : y, kv_full(j));
      }
      // the copies issued last: none may be under way when the CTA ends, whatever its consumers did
      for (uint32_t i = j > SLOTS ? j - SLOTS : 0; i < j; ++i)
        mbar_wait_polls(kv_full(i), (i / SLOTS) & 1, 1u << 20);
    } else {
      // Four lanes take 64 codes of a key, a warp's load eight keys, as soon as their
      // registers are free, under the conversion of the other half.
      constexpr int HV = D / 64, KEYS = C::CONV * 8, N = KB / KEYS * HV;   // halves of a row, keys per pass, loads
      const int ptid = tid - 256, c = ptid & 3, k0 = ptid >> 2;
      uint4 wk[N], wv[N];
      auto load = [&](const void* pool, uint4 (&w)[N], uint32_t j) {
        const uint8_t* const p = reinterpret_cast<const uint8_t*>(pool) + c * 16;
#pragma unroll
        for (int i = 0; i < N; i += HV) {
          const int row = s_rows[(j & 3) * KB + i / HV * KEYS + k0];
#pragma unroll
          for (int h = 0; h < HV; ++h)
            w[i + h] = row >= 0 ? ldg_cg_v4(p + (int64_t)row * D + h * 64)
                                : make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
        }
      };
      // exponent of a block's largest scale
      auto exponent = [&](uint32_t j, int side) {
        const float2 m = *reinterpret_cast<const float2*>(s_scale + (j & 7) * C::SCALE_SLOT + 2 * KB + 4 * side);
        const float x = fmaxf(m.x, m.y);
        return min(126, max(side ? VALUE_MIN : KEY_MIN, (int)(__float_as_uint(x) >> 23) - 127));
      };
      // 16 codes are chunks 2 c, 2 c + 1 of a half row's line; eight lanes' stores are
      // those of two neighbouring keys, whose swizzles differ by one chunk: all banks
      const uint32_t line = k0 * 128, x0 = (uint32_t)((2 * c) ^ (k0 & 7)) << 4;
      auto put = [&](const uint4 (&w)[N], uint32_t dst, uint32_t j, int side, int e) {
        const float* const sc = s_scale + (j & 7) * C::SCALE_SLOT;
        const float less = __uint_as_float((uint32_t)(127 + VALUE_UP - e) << 23);
        const bool bare = sc[2 * KB + 2] != 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          // the scale relative to the power of two; bare codes: a power of two
          const float r = bare ? (float)(1 << VALUE_UP) : sc[side * KB + k0 + i / HV * KEYS] * less;
          const __half hi = __float2half_rn(r), lo = __float2half_rn(r - __half2float(hi));
          const __half2 hi2 = __half2half2(hi), lo2 = __half2half2(lo);
          auto value = [&](uint32_t word, uint32_t sel) {
            const uint32_t x = codes2(word, sel);
            const __half2 h = *reinterpret_cast<const __half2*>(&x);
            const __half2 y = side ? __hmul2(h, hi2) : __hfma2(h, hi2, __hmul2(h, lo2));
            return *reinterpret_cast<const uint32_t*>(&y);
          };
          const uint32_t at = dst + (i % HV) * (KB * 128) + i / HV * (KEYS * 128) + line;
          const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int y = 0; y < 2; ++y)
            st_shared(at + (x0 ^ (uint32_t)(y << 4)), value(v[2 * y], 0x4140u),
                      value(v[2 * y], 0x4342u), value(v[2 * y + 1], 0x4140u),
                      value(v[2 * y + 1], 0x4342u));
        }
      };
      meet_planners<C::CONV + C::PLAN>();
      if (n > 0) load(a.k, wk, 0);
      meet_planners<C::CONV + C::PLAN>();
      int ev = 0;   // exponent of the block's scales of V
      // no thread leaves this loop early (they meet in it): after a wait ran out
      // they only go on writing to their own shared memory
      for (uint32_t j = 0; j <= n && n > 0; ++j) {
        if (j >= SLOTS) gate.wait(kv_empty(j), ((j / SLOTS) - 1) & 1);
        const uint32_t slot = ring_s + j % SLOTS * C::SLOT;
        const int ev_before = ev;
        if (j < n) {
          const int ek = exponent(j, 0);
          ev = exponent(j, 1);
          if (ptid == 0)
            *reinterpret_cast<float2*>(s_scale + (j & 7) * C::SCALE_SLOT + 2 * KB + 8) =
                make_float2(__uint_as_float((uint32_t)(127 + ek - VALUE_UP) << 23), (float)(ev - VALUE_UP));
          put(wk, slot + C::HALF, j, 0, ek);
          if (j + 1 < n) load(a.k, wk, j + 1);
        }
        if (j > 0) put(wv, slot, j - 1, 1, ev_before);
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(kv_full(j));
        if (j < n) load(a.v, wv, j);
        meet_planners<C::CONV + C::PLAN>();   // the rows of block j + 2 and the scales of block j + 1 are there
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
}

// -------------------------------------------------------------------- host --
template <int D, bool Q8>
int32_t launch(const ChunkArgs& a, int64_t rows, int n_ctas, cudaStream_t st) {
  using C = Cfg<D, Q8>;
  SUB_CUDA_TRY(once_per_device([] {
    return cudaFuncSetAttribute(chunk_tc_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::SMEM);
  }));
  Maps maps;
  memset(&maps, 0, sizeof(maps));
  int box = 16;
  while (box < KB && a.t.page_size % (2 * box) == 0) box *= 2;
  auto pool_map = [&](CUtensorMap* m, const void* pool) {
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pool, D, rows, D * 2, 64, box, 128);
  };
  if (!Q8 && (!pool_map(&maps.k, a.k) || !pool_map(&maps.v, a.v)))
    return fail(SUB_ECUDA, "chunk_attn: the cache's tensor map was refused");
  SUB_CUDA_TRY(launch_k(chunk_tc_kernel<D, Q8>, dim3(n_ctas), dim3(C::THREADS), C::SMEM, st, maps, a,
                        box, (int)rows));
  return SUB_OK;
}

}  // namespace

bool chunk_page_map(CUtensorMap* m, const void* pool, const SeqTable& t, int64_t heads, int d, bool codes) {
  auto fn = encode_fn();
  if (!fn) return false;
  const int size = codes ? 1 : 2, line = d * size < 128 ? d * size : 128;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)t.page_size, (cuuint64_t)(heads * t.n_pages)};
  const cuuint64_t strides[2] = {(cuuint64_t)d * size, (cuuint64_t)d * size * t.page_size};
  const cuuint32_t boxes[3] = {(cuuint32_t)(line / size), 16, 1}, es[3] = {1, 1, 1};
  return fn(m, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void*>(pool), dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            line == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool chunk_tc_fits(int64_t pool_rows) { return pool_rows < (1ll << 31) - 4096; }

int32_t launch_chunk_tc(const ChunkArgs& a, bool q8, int head_dim, int64_t pool_rows, int n_ctas,
                        cudaStream_t st) {
  if (q8) return head_dim == 128 ? launch<128, true>(a, pool_rows, n_ctas, st)
                                 : launch<64, true>(a, pool_rows, n_ctas, st);
  return head_dim == 128 ? launch<128, false>(a, pool_rows, n_ctas, st)
                         : launch<64, false>(a, pool_rows, n_ctas, st);
}

int32_t chunk_tc_timeouts(unsigned int* out) {
  SUB_CUDA_TRY(cudaMemcpyFromSymbol(out, g_chunk_timeouts, sizeof(unsigned int)));
  return SUB_OK;
}

}  // namespace sub
