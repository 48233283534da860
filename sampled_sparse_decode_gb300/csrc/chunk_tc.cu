// chunk_tc.cu — causal attention of a chunk of new tokens over a paged bf16 cache on the tensor
// cores (tcgen05, accumulators in TMEM).
//
// A KV head's G query heads share its keys, so the rows of a tile are (token, head) pairs,
// token-major: 128 / G tokens make one 128-row tile, and two tiles (A, B) one work item, which
// walks the keys that its last token sees in steps of 128.  Per step and tile:
//   S = Q K^T   (128 x 128 x d, both operands in shared memory)      -> TMEM
//   P = 2^(S scale - m), running maximum m and sum l per row; bf16   -> TMEM, over S
//   O += P V    (128 x d x 128, P from TMEM, V in shared memory)     -> TMEM
// Roles of a block (one per SM, persistent): warps 0-3 softmax of tile A and warps 4-7 of tile B
// (a thread owns a row, so maxima and sums need no exchange), warp 8 issues the products, warp 9
// feeds K and V through a ring of tensor copies (warps 10 and 11 only give up registers).  While
// one tile's softmax runs, the tensor pipe works on the other tile.  O is rescaled only when a
// row's maximum has grown by more than 2^8 since the last time (the stored m is a reference, not
// the maximum; weights stay below 2^8), so most steps touch O by the product alone.
//
// Work split.  The steps of all items, in the order (sequence, KV head, item, step), are one line
// of W units, a few more for each item's opening; block c of N takes the units [W c / N,
// W (c + 1) / N), give or take a few that spare a cut (line_border).  An item that is cut leaves
// partial (m, l, O) rows in the workspace, at most two per block, and a second launch joins them
// in order: every block has the same work to within a few steps, for one long sequence as for
// many short ones, and nothing depends on timing.
//
// Unseen values.  P is 0 for a masked pair, but 0 * V is not 0 for an infinite or NaN V.  Steps
// that hold masked pairs (the causal border and the sequence's end) therefore pass through the
// copying warp after they land: rows of V that no row of the item sees are cleared, and in rows
// that only some see, non-finite elements are cleared and noted; the rows that do see them add
// their product in the epilogue.
//
// Roundings.  Scores, m, l and O are fp32.  P is rounded to bf16 (half a step is 2^-9 of a weight),
// because the product with bf16 V takes no wider operand; l sums the weights before the rounding.
// The error against 64 bits is 2.0e-3 to 2.4e-3 of the results' size; with a second bf16 piece of P
// it is 1.5e-3 to 1.7e-3, the output's own rounding.  That takes twice the products with V, and a
// softmax that spills and stores twice as much: 2048 tokens on 32K 671 -> 1222 us, ragged prompts
// 779 -> 1418, 4 tokens of 16 sequences on 32K (bound by the cache otherwise) 323 -> 513, 4096
// tokens on 4096 with heads of 64 240 -> 410.
//
// Bound by the chain S -> softmax -> P -> product within a tile, which two tiles per block hide
// in part: a step takes 2950 cycles of which the tensor pipe works 2048 (65.7% active over the
// kernel).  Measured on GB300 in a stream of calls on changing inputs: 2048 tokens on 32K, 28 / 4
// heads of 128, 672 us, 1476 TFLOP/s (77% of a measured library product); prompts from empty, 32 / 8
// heads of 128, 512, 1216 and 4096 tokens 19.8, 27.6 and 131 us; 4 tokens of 16 sequences on 32K
// 326 us, 6.6 TB/s; 4096 tokens on 4096, 32 / 8 heads of 64, 245 us, 842 TFLOP/s.
#include <algorithm>

#include "kernels.h"

namespace santa {

namespace {

constexpr int kTcThreads = 384;         // three warpgroups: softmax A, softmax B, the rest
// Registers per thread of a softmax and of the last warpgroup: 2 * 200 + 104 = 3 * 168, what 384
// threads are launched with.  192 / 120 spills in the softmax (2048 tokens on 32K, the same inputs in
// every call: 834 us where 200 / 104 takes 630), 208 / 88 in the issuing warp (660 us).
constexpr int kSoftmaxRegs = 200;
constexpr int kIssueRegs = 104;
constexpr int kStep = 128;              // keys per step
constexpr int kGroups = 16;             // barriers of the copy groups (more than ring stages)
constexpr int kSnap = 6;                // steps a border may move to an item's end
constexpr int kOpen = 4;                // what opening and closing an item costs, in steps
constexpr uint64_t kDrainNs = 1000000;  // longer than any copy in flight takes
constexpr float kSlack = 8.f;           // growth of a row's maximum that triggers a rescale

template <int D>
struct TcCfg {
  static constexpr int kHalves = D / 64;                 // 128-byte wide column blocks
  static constexpr int kTileBytes = 128 * D * 2;         // one Q tile, one K or V step
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr size_t kSmem = 1024 + (2 + kStages) * static_cast<size_t>(kTileBytes);
  static constexpr int kColS = 0, kColO = 256;           // TMEM columns: S_A S_B | O_A O_B
};

struct TcParams {
  ChunkParams c;
  int tpt;                   // tokens per 128-row tile
  float* part_acc;           // [N][2][D / 4][256][4]
  float* part_ml;            // [N][2][256][2]
  int32_t* join;             // [N][8]
  CUtensorMap tmap_q, tmap_k, tmap_v;
};

struct TcShared {
  uint64_t q_full, q_empty, land, drain;
  uint64_t kv_full[kGroups], kv_empty[kGroups];
  uint64_t s_full[2], p_ready[2], o_full[2];
  uint64_t run_open[3], run_done[3];   // by item ring: a run has begun; both tiles finished it
  int group_of[10];          // by ring stage: the group of the tile in it (copying warp only)
  uint32_t tmem;
  volatile int abort;
  int start[4];              // b, h, item, step of the block's first step
  int64_t total, begin, end; // the line's length; the block's part of it
  int blocks, snap;          // blocks with work; see line_border
  uint32_t noted[3][4][4];   // [item ring][step of the last four][token bits]
};

// ---------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
// 32 consecutive columns of this warp's 32 TMEM lanes: one row piece per thread.
__device__ __forceinline__ void tc_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tc_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Ties later uses of loaded registers to the wait before it.
__device__ __forceinline__ void tc_loaded(uint32_t (&r)[32]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
  asm volatile(""
               : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                 "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory operand with the 128-byte swizzle: rows of 128 bytes, 8-row groups of 1 KiB.
// The low word holds the address and `lead`, the distance of the 64-element blocks of an operand
// whose rows run along K (V; not used by operands whose rows hold K: Q, K).  The high word is a
// constant, and an address step is one 32-bit addition (16-byte units; no carry: addresses stay
// below 2^18).
__device__ __forceinline__ uint32_t tc_desc_lo(uint32_t addr, uint32_t lead) {
  return ((addr >> 4) & 0x3fff) | ((lead >> 4) & 0x3fff) << 16;
}
__device__ __forceinline__ uint64_t tc_desc(uint32_t lo) {
  constexpr uint64_t hi = (1024 >> 4) | 1u << 14 | 2u << 29;
  return hi << 32 | lo;
}
// bf16 x bf16 -> fp32, 128 x n; `b_rows_k`: B's rows run along K.
constexpr uint32_t tc_idesc(int n, bool b_rows_k) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_rows_k ? 1u << 16 : 0u) |
         static_cast<uint32_t>(n >> 3) << 17 | 8u << 24;
}

// Waits for a phase; gives up after the limit or once any warp has (the block then drains).
__device__ __forceinline__ bool wait_or_abort(TcShared& s, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t start = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (s.abort) return false;
    if (global_timer_ns() - start > kWaitLimitNs) {
      s.abort = 1;
      return false;
    }
  }
  return true;
}

// The same by all lanes of a warp, with one answer: a lane that left alone would leave the others
// waiting for it in the warp's next common instruction.
__device__ __forceinline__ bool warp_wait(TcShared& s, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_or_abort(s, bar, parity));
}

// Two fp32 values in a register pair, and the instructions that work on both.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 2^(s scale - ref) of 64 scores, as packed bf16 and, returned, their sum by even and odd ones.
__device__ __forceinline__ uint64_t half_weights(uint32_t (&pk)[32], const uint32_t (&s0)[32],
                                                 const uint32_t (&s1)[32], float scale,
                                                 float ref) {
  const uint64_t scale2 = pair(scale, scale), ref2 = pair(-ref, -ref);
  uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const uint32_t(&src)[32] = e < 16 ? s0 : s1;
    const int at = (2 * e) % 32;
    float a, b;
    unpair(fma2(pair(__uint_as_float(src[at]), __uint_as_float(src[at + 1])), scale2, ref2), &a,
           &b);
    a = ex2_approx(a);
    b = ex2_approx(b);
    pk[e] = pack_bf16(a, b);
    sum[e & 1] = add2(sum[e & 1], pair(a, b));
  }
  return add2(sum[0], sum[1]);
}

// ---------------------------------------------------------------- work line

// sum over i < n of floor((a i + b) / m)
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  int64_t sum = 0;
  while (n > 0) {
    sum += static_cast<int64_t>(n) * (n - 1) / 2 * (a / m) + static_cast<int64_t>(n) * (b / m);
    a %= m;
    b %= m;
    const uint32_t top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

struct Seq {
  int first, n, ctx;         // first token row, new tokens, cached tokens before them
};
// Sequence b's chunk; n = 0 if it has none or must be skipped (*bad).
__device__ __forceinline__ Seq load_seq(const ChunkParams& p, int b, bool* bad) {
  const int64_t c0 = p.cu_q[b], c1 = p.cu_q[b + 1], len = p.seq_lens[b];
  Seq s = {0, 0, 0};
  *bad = c0 < 0 || c1 < c0 || c1 > p.num_tokens ||
         (c1 > c0 && (len < c1 - c0 || len > static_cast<int64_t>(p.max_teams) * p.team_size));
  if (!*bad) {
    s.first = static_cast<int>(c0);
    s.n = static_cast<int>(c1 - c0);
    s.ctx = static_cast<int>(len) - s.n;
  }
  return s;
}
// Line length of the items 0 .. i - 1 (all of them with full token counts) of a sequence: the
// steps, and kOpen for each item.
__device__ __forceinline__ int64_t line_before(const Seq& s, int tpi, int i) {
  return floor_sum(i, kStep, tpi, s.ctx + tpi + kStep - 1) + static_cast<int64_t>(i) * kOpen;
}
__device__ __forceinline__ int item_steps(const Seq& s, int tpi, int i) {
  return (s.ctx + min(s.n, (i + 1) * tpi) + kStep - 1) / kStep;
}
__device__ __forceinline__ int64_t seq_line(const Seq& s, int tpi) {
  if (s.n == 0) return 0;
  const int items = (s.n + tpi - 1) / tpi;
  return line_before(s, tpi, items - 1) + kOpen + (s.ctx + s.n + kStep - 1) / kStep;
}

// Where the line's unit `pos` lies, by one warp: sequence, head, item, offset in the item.
__device__ void find_step(const ChunkParams& p, int tpi, int64_t pos, int* out) {
  const int lane = threadIdx.x & 31;
  int64_t before = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    bool bad;
    const Seq s = b0 + lane < p.batch ? load_seq(p, b0 + lane, &bad) : Seq{0, 0, 0};
    const int64_t mine = seq_line(s, tpi) * p.num_kv_heads;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned over = __ballot_sync(0xffffffffu, before + incl > pos);
    if (over) {
      const int at = __ffs(over) - 1;
      const int64_t start = before + __shfl_sync(0xffffffffu, incl - mine, at);
      const int64_t per_head = __shfl_sync(0xffffffffu, mine, at) / p.num_kv_heads;
      Seq q;
      q.first = 0;
      q.n = __shfl_sync(0xffffffffu, s.n, at);
      q.ctx = __shfl_sync(0xffffffffu, s.ctx, at);
      const int h = static_cast<int>((pos - start) / per_head);
      const int64_t rem = (pos - start) - h * per_head;
      // the last item i with line_before(i) <= rem
      int lo = 0, hi = (q.n + tpi - 1) / tpi;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const bool below = lane == 0 || (i < hi && line_before(q, tpi, i) <= rem);
        const unsigned m = __ballot_sync(0xffffffffu, below);
        lo += (31 - __clz(m)) * step;
        hi = min(hi, lo + step);
      }
      out[0] = b0 + at;
      out[1] = h;
      out[2] = lo;
      out[3] = static_cast<int>(rem - line_before(q, tpi, lo));
      return;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  out[0] = p.batch;
  out[1] = out[2] = out[3] = 0;
}

// Border c of the line (where block c starts): total * c / blocks, moved to the item's start or
// end if that is at most `snap` steps away, which saves a join for a little unevenness.  The
// moves keep the borders in order.  By one warp; out = sequence, head, item, step.
__device__ int64_t line_border(const ChunkParams& p, int tpi, int64_t total, int blocks, int snap,
                               int c, int* out) {
  const int64_t pos = total * c / blocks;
  if (pos >= total) return total;
  find_step(p, tpi, pos, out);
  bool bad;
  const Seq q = load_seq(p, out[0], &bad);
  const int off = out[3], step = max(0, off - kOpen), steps = item_steps(q, tpi, out[2]);
  out[3] = step;
  if (step <= snap) {
    out[3] = 0;
    return pos - off;
  }
  if (steps - step > snap) return pos;
  const int64_t next = pos + kOpen + steps - off;  // the next item's start
  if (next < total) find_step(p, tpi, next, out);
  return next;
}

// One run of steps of one item, and the walk from run to run.
struct Run {
  int b, h, item, s0, s1, steps;
  Seq seq;
  int64_t left;
  bool got;
  __device__ __forceinline__ void begin(const TcShared& s, const ChunkParams& p) {
    b = s.start[0];
    h = s.start[1];
    item = s.start[2];
    s0 = s.start[3];
    left = s.end - s.begin;
    got = left > 0;
    bool bad;
    if (got) seq = load_seq(p, b, &bad);
  }
  // Sets s1 and steps; false at the end of the block's range.
  __device__ __forceinline__ bool open(int tpi) {
    if (!got) return false;
    steps = item_steps(seq, tpi, item);
    s1 = static_cast<int>(min(static_cast<int64_t>(steps), s0 + left - (s0 ? 0 : kOpen)));
    return true;
  }
  __device__ __forceinline__ void next(const ChunkParams& p, int tpi) {
    left -= s1 - s0 + (s0 ? 0 : kOpen);
    got = left > 0;
    if (!got) return;
    s0 = 0;                                     // more is left: the item was finished
    if (static_cast<int64_t>(++item) * tpi < seq.n) return;
    item = 0;
    if (++h < p.num_kv_heads) return;
    h = 0;
    bool bad;
    do seq = load_seq(p, ++b, &bad);            // left > 0: a later sequence has steps
    while (seq.n == 0);
  }
};

// ---------------------------------------------------------------- roles

// V rows [hi, 128) of a landed step are cleared; in rows [lo, hi) non-finite elements are
// cleared and their rows noted.  By one warp, so the common path is kept short: x * 0 is NaN
// exactly if x is not finite, so one packed product-and-sum per two elements carries the answer
// for many of them, and the exact search runs only where it says so.
template <int D>
__device__ __forceinline__ void clean_rows(unsigned char* v, int lo, int hi, uint32_t* noted) {
  const int lane = threadIdx.x & 31;
  constexpr int kPieces = D / 8;                   // 16-byte pieces per row
  constexpr int kRowsAt = 32 / kPieces;            // rows the warp covers at once
  const int piece = lane % kPieces;
  unsigned char* at = v + (piece / 8) * 16384 + (piece % 8) * 16;
#pragma unroll 8
  for (int r = hi + lane / kPieces; r < kStep; r += kRowsAt)
    *reinterpret_cast<uint4*>(at + r * 128) = make_uint4(0u, 0u, 0u, 0u);
  uint32_t acc[4] = {0u, 0u, 0u, 0u};
#pragma unroll 8
  for (int r = lo + lane / kPieces; r < hi; r += kRowsAt) {
    const uint4 w = *reinterpret_cast<const uint4*>(at + r * 128);
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[0]) : "r"(w.x), "r"(0u));
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[1]) : "r"(w.y), "r"(0u));
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[2]) : "r"(w.z), "r"(0u));
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[3]) : "r"(w.w), "r"(0u));
  }
  if (!__any_sync(0xffffffffu, ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu) != 0u)) return;
  const uint32_t e = 0x7f807f80u;                  // all exponent bits: infinite or NaN
  for (int r = lo + lane / kPieces; r < hi; r += kRowsAt) {
    uint4* w = reinterpret_cast<uint4*>(at + r * 128);
    const uint4 x = *w;
    const uint32_t bx = __vcmpeq2(x.x & e, e), by = __vcmpeq2(x.y & e, e);
    const uint32_t bz = __vcmpeq2(x.z & e, e), bw = __vcmpeq2(x.w & e, e);
    if (bx | by | bz | bw) {
      *w = make_uint4(x.x & ~bx, x.y & ~by, x.z & ~bz, x.w & ~bw);
      atomicOr(&noted[r / 32], 1u << (r % 32));
    }
  }
}

// Adds to the bytes that a barrier's phase waits for (no arrival).
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

// K and V of a run arrive in groups, {K(s0)}, {V(s0), K(s0 + 1)}, {V(s0 + 1), K(s0 + 2)}, ...,
// {V(s1 - 1)}: what the products between two hand-overs of P use.  A group has one full and one
// empty barrier, so the issuing warp waits and commits once per step; its tiles take the next
// stages of the ring.
template <int D>
__device__ void copy_role(const TcParams& t, TcShared& s, unsigned char* q_smem,
                          unsigned char* ring) {
  using C = TcCfg<D>;
  const ChunkParams& p = t.c;
  const int lane = threadIdx.x & 31, tpi = 2 * t.tpt, G = p.num_q_heads / p.num_kv_heads;
  const int T = p.team_size;
  uint32_t q_parity = 1, land_parity = 0, runs = 0;
  int group = 0, tiles = 0, stage = 0;
  Run r;
  r.begin(s, p);
  bool ok = true;
  // the next ring stage, once the tile in it has been used
  auto claim = [&] {
    if (tiles >= C::kStages) {
      const int g = s.group_of[stage];
      ok = warp_wait(s, &s.kv_empty[g % kGroups], (g / kGroups) & 1);
      __syncwarp();
    }
    if (lane == 0) s.group_of[stage] = group;
    __syncwarp();
    unsigned char* dst = ring + stage * C::kTileBytes;
    ++tiles;
    if (++stage == C::kStages) stage = 0;
    return dst;
  };
  for (int turn = 0; ok && r.open(tpi); r.next(p, tpi), turn = turn == 2 ? 0 : turn + 1) {
    const int tok = r.item * tpi;
    const bool two = tok + t.tpt < r.seq.n;
    ok = warp_wait(s, &s.q_empty, q_parity);
    q_parity ^= 1;
    if (!ok) break;
    // the notes of three runs ago have been read (tile B may lag behind runs that A has alone)
    ok = warp_wait(s, &s.run_done[turn], (runs / 3 + 1) & 1);
    if (!ok) break;
    if (lane == 0) mbar_arrive(&s.run_open[turn]);
    if (lane < 16) s.noted[turn][lane / 4][lane % 4] = 0u;
    if (lane == 0) {
      const uint32_t box = t.tpt * G * 128;      // bytes of one 64-element wide box
      mbar_arrive_expect_tx(&s.q_full, box * C::kHalves * (two ? 2 : 1));
      for (int x = 0; x < (two ? 2 : 1); ++x)
        for (int i = 0; i < C::kHalves; ++i)
          asm volatile(
              "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
              " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                  smem_u32(q_smem + x * C::kTileBytes + i * 16384)),
              "l"(reinterpret_cast<uint64_t>(&t.tmap_q)), "r"(i * 64), "r"(0), "r"(r.h),
              "r"(r.seq.first + tok + x * t.tpt), "r"(smem_u32(&s.q_full))
              : "memory");
    }
    ++runs;
    const int len = r.seq.ctx + r.seq.n;
    const int seen = r.seq.ctx + min(r.seq.n, tok + tpi);   // keys that some row sees
    const int all_see = r.seq.ctx + tok + 1;                // keys that every row sees
    const int teams = (len + T - 1) / T;
    int window = -1, ids = 0;
    int row[2] = {-1, -1};                       // pool rows of the step's 64-key halves
    for (int j = r.s0; ok && j <= r.s1; ++j, ++group) {     // group {V(j - 1), K(j)}
      uint64_t* bar = &s.kv_full[group % kGroups];
      bool check = false;
      unsigned char* v_dst = nullptr;
      auto load = [&](unsigned char* dst, const CUtensorMap* map, uint64_t* on) {
        if (lane == 0) {
          mbar_expect_tx(on, (row[1] >= 0 ? 2 : 1) * 64 * D * 2);
          for (int c = 0; c < 2; ++c)
            if (row[c] >= 0)
              for (int i = 0; i < C::kHalves; ++i)
                tma_load_2d(dst + i * 16384 + c * 8192, map, i * 64, row[c], on);
        }
      };
      if (j > r.s0) {
        v_dst = claim();
        if (!ok) break;
        check = j * kStep > all_see;             // step j - 1 holds masked pairs
        load(v_dst, &t.tmap_v, check ? &s.land : bar);
        if (check && lane == 0) mbar_arrive(&s.land);
      }
      if (j < r.s1) {
        // page ids of 32 teams at a time, one per lane
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int at = j * kStep + c * 64;
          row[c] = -1;
          if (at >= len) continue;
          const int team = at / T;
          if (window < 0 || team >= window + 32) {
            window = team;
            ids = 0;
            if (team + lane < teams) {
              ids = p.page_table[static_cast<int64_t>(r.b) * p.max_teams + team + lane];
              if (ids < 0 || ids >= p.num_pages) {
                set_status(p.status, SANTA_DEV_BAD_PAGE);
                ids = 0;
              }
            }
          }
          const int page = __shfl_sync(0xffffffffu, ids, team - window);
          row[c] = (page * p.num_kv_heads + r.h) * T + at % T;
        }
        unsigned char* k_dst = claim();
        if (!ok) break;
        load(k_dst, &t.tmap_k, bar);
      }
      if (check) {
        ok = warp_wait(s, &s.land, land_parity);
        land_parity ^= 1;
        if (!ok) break;
        // rows [lo, hi) are seen by some rows of the item only, rows from hi on by none
        const int at = (j - 1) * kStep;
        clean_rows<D>(v_dst, max(0, all_see - at), min(kStep, seen - at),
                      s.noted[turn][j - 1 - r.steps + 4]);
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(bar);
    }
  }
  if (lane == 0) {
    // what was issued lands before the block may end (bounded; it has, unless a wait gave up)
    const uint64_t start = global_timer_ns();
    while (runs && !mbar_try_wait(&s.q_full, (runs - 1) & 1) &&
           global_timer_ns() - start < kWaitLimitNs) {
    }
    for (int g = max(0, group - C::kStages); g < group; ++g)
      while (!mbar_try_wait(&s.kv_full[g % kGroups], (g / kGroups) & 1) &&
             global_timer_ns() - start < kWaitLimitNs) {
      }
    // copies of a group that was not completed: nothing signals them, so the time is waited out
    while (!ok && global_timer_ns() - start < kDrainNs) {
    }
  }
}

template <int D>
__device__ void mma_role(const TcParams& t, TcShared& s, uint32_t q_smem, uint32_t ring) {
  using C = TcCfg<D>;
  const ChunkParams& p = t.c;
  const int tpi = 2 * t.tpt;
  constexpr uint32_t kIdS = tc_idesc(kStep, false), kIdO = tc_idesc(D, true);
  const uint32_t tmem = s.tmem;
  uint32_t q_parity = 0, p_parity[2] = {0, 0};
  int group = 0, stage = 0;
  Run r;
  r.begin(s, p);
  const uint32_t q_lo = tc_desc_lo(q_smem, 16), k_lo = tc_desc_lo(ring, 16),
                 v_lo = tc_desc_lo(ring, 16384);
  constexpr uint32_t kTile = C::kTileBytes >> 4;
  auto next_stage = [&] {
    const int at = stage;
    if (++stage == C::kStages) stage = 0;
    return static_cast<uint32_t>(at);
  };
  auto scores = [&](int x, uint32_t k_at) {         // S_x = Q_x K^T
    const uint32_t q_at = q_lo + x * kTile;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      constexpr uint32_t kHalf = 16384 >> 4;
      const uint32_t off = (k / 4) * kHalf + (k % 4) * 2;
      tc_mma_ss(tmem + C::kColS + 128 * x, tc_desc(q_at + off), tc_desc(k_at + off), kIdS, k > 0);
    }
    tc_commit(&s.s_full[x]);
  };
  // A wait or a commit between products leaves a gap in the tensor pipe (each costs about 100
  // cycles), so a step has as few as it can: the group, P of each tile; S of each tile, the group.
  for (; r.open(tpi); r.next(p, tpi)) {
    const bool two = r.item * tpi + t.tpt < r.seq.n;
    if (!wait_or_abort(s, &s.q_full, q_parity)) return;
    q_parity ^= 1;
    for (int j = r.s0; j <= r.s1; ++j, ++group) {     // O += P(j - 1) V(j - 1), S(j) = Q K(j)^T
      if (!wait_or_abort(s, &s.kv_full[group % kGroups], (group / kGroups) & 1)) return;
      tc_fence_after();
      const uint32_t v_at = j > r.s0 ? v_lo + next_stage() * kTile : 0;
      const uint32_t k_at = j < r.s1 ? k_lo + next_stage() * kTile : 0;
      for (int x = 0; x < (two ? 2 : 1); ++x) {
        if (j > r.s0) {
          if (!wait_or_abort(s, &s.p_ready[x], p_parity[x])) return;
          p_parity[x] ^= 1;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kStep / 16; ++k)
            tc_mma_ts(tmem + C::kColO + D * x, tmem + C::kColS + 128 * x + 8 * k,
                      tc_desc(v_at + (2048 >> 4) * k), kIdO, j > r.s0 + 1 || k > 0);
        }
        if (j < r.s1)
          scores(x, k_at);
        else
          tc_commit(&s.o_full[x]);
      }
      tc_commit(&s.kv_empty[group % kGroups]);
      if (j + 1 == r.s1) tc_commit(&s.q_empty);
    }
  }
}

// Products of noted V elements (see the top of the file) that this row sees, added to the row
// where it was just written: the output (bf16, step 2 bytes) or the partial result.  Such an
// element is infinite or NaN, and so is the sum, whatever the order and the divisor.
template <int D>
__device__ __noinline__ void add_noted(const TcParams& t, const Run& r, const uint32_t (*noted)[4],
                                       int sees, int64_t q_row, float m, uint16_t* out,
                                       float* part) {
  const ChunkParams& p = t.c;
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + q_row;
  for (int e = 0; e < 4; ++e)
    for (int w = 0; w < 4; ++w)
      for (uint32_t bits = noted[e][w]; bits; bits &= bits - 1) {
        const int tok = (r.steps - 4 + e) * kStep + w * 32 + __ffs(bits) - 1;
        if (tok >= sees) continue;
        int64_t page = p.page_table[static_cast<int64_t>(r.b) * p.max_teams + tok / p.team_size];
        if (page < 0 || page >= p.num_pages) page = 0;
        const int64_t row =
            ((page * p.num_kv_heads + r.h) * p.team_size + tok % p.team_size) * D;
        const uint16_t* k = static_cast<const uint16_t*>(p.k_pool) + row;
        const uint16_t* v = static_cast<const uint16_t*>(p.v_pool) + row;
        float dot = 0.f;
        for (int i = 0; i < D; ++i) dot = fmaf(bf16_to_f32(q[i]), bf16_to_f32(k[i]), dot);
        const float w32 = ex2_approx(fmaf(dot, p.scale_log2, -m));
        const float weight = bf16_lo_f(pack_bf16(w32, 0.f));
        for (int i = 0; i < D; ++i)
          if ((v[i] & 0x7f80) == 0x7f80) {
            const float x = weight * bf16_to_f32(v[i]);
            if (out)
              out[i] = static_cast<uint16_t>(pack_bf16(bf16_to_f32(out[i]) + x, 0.f));
            else
              part[(i / 4) * 1024 + i % 4] += x;
          }
      }
}

// 16 consecutive fp32 values (32 bytes of bf16) of a row, scaled; `wide`: dst is 32-byte aligned.
__device__ __forceinline__ void store_row16(uint16_t* dst, const uint32_t* o, float inv,
                                            bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e] = pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int D>
__device__ void softmax_role(const TcParams& t, TcShared& s) {
  using C = TcCfg<D>;
  const ChunkParams& p = t.c;
  const int x = threadIdx.x / 128, row = threadIdx.x % 128, warp = (threadIdx.x / 32) % 4;
  const int tpi = 2 * t.tpt, G = p.num_q_heads / p.num_kv_heads;
  const int g = row % G, token_in_tile = row / G;
  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t tm_s = s.tmem + C::kColS + 128 * x + lanes;
  const uint32_t tm_o = s.tmem + C::kColO + D * x + lanes;
  const float scale = p.scale_log2;
  const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
  uint32_t parity = 0;           // bit 0: s_full, bit 1: o_full, bit 2: run_open
  Run r;
  r.begin(s, p);
  for (int turn = 0; r.open(tpi); r.next(p, tpi), turn = turn == 2 ? 0 : turn + 1) {
    const int tok0 = r.item * tpi + x * t.tpt;           // first token of this tile
    if (tok0 >= r.seq.n) {
      // not before the run has begun: an early arrival would count for another run of the ring
      if (!warp_wait(s, &s.run_open[turn], parity >> 2 & 1)) return;
      if ((threadIdx.x & 31) == 0) mbar_arrive(&s.run_done[turn]);
      if (turn == 2) parity ^= 4;
      continue;
    }
    const int tok = tok0 + token_in_tile;
    const bool mine = token_in_tile < t.tpt && tok < r.seq.n;
    const int sees = mine ? r.seq.ctx + tok + 1 : 0;
    const int all_see = r.seq.ctx + tok0 + 1;
    const bool warp_idle = __ballot_sync(0xffffffffu, mine) == 0u;
    float m = -INFINITY, l = 0.f;
    for (int j = r.s0; j < r.s1; ++j) {
      if (!warp_wait(s, &s.s_full[x], parity & 1)) return;
      parity ^= 1;
      if (!warp_idle) {
        tc_fence_after();
        uint32_t sc[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_ld32(sc[c], tm_s + 32 * c);
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_loaded(sc[c]);
        if ((j + 1) * kStep > all_see) {
          const int cut = sees - j * kStep;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c * 32 + e >= cut) sc[c][e] = 0xff800000u;   // -inf
        }
        // weights of the first half by the reference in hand, while the maximum is formed: it
        // seldom grows past the slack, and then they are formed again
        uint32_t pk[32];
        float ref = m == -INFINITY ? 0.f : m;
        uint64_t sum = half_weights(pk, sc[0], sc[1], scale, ref);
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          mx[c] = fmaxf(__uint_as_float(sc[c][0]), __uint_as_float(sc[c][1]));
#pragma unroll
        for (int e = 2; e < 32; e += 2)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            mx[c] = max3(mx[c], __uint_as_float(sc[c][e]), __uint_as_float(sc[c][e + 1]));
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * scale;
        // grown past the slack (or the first finite score): a new reference
        const bool grow = top > m + kSlack || (m == -INFINITY && top > -INFINITY);
        if (__any_sync(0xffffffffu, grow)) {
          const float old = m;
          if (grow) m = ref = top;
          if (j > r.s0) {
            const float keep = grow ? ex2_approx(old - m) : 1.f;
            l *= keep;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tc_ld32(o, tm_o + 32 * c);
              tc_wait_ld();
              tc_loaded(o);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
              tc_st32(tm_o + 32 * c, o);
            }
          }
          sum = half_weights(pk, sc[0], sc[1], scale, ref);
        }
        tc_st32(tm_s, pk);
        sum = add2(sum, half_weights(pk, sc[2], sc[3], scale, ref));
        tc_st32(tm_s + 32, pk);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&s.p_ready[x]);
        float la, lb;
        unpair(sum, &la, &lb);
        l += la + lb;
      } else if ((threadIdx.x & 31) == 0) {
        mbar_arrive(&s.p_ready[x]);
      }
    }
    // ---- epilogue: the row, or its partial result
    if (!warp_wait(s, &s.o_full[x], parity >> 1 & 1)) return;
    parity ^= turn == 2 ? 6 : 2;
    if (warp_idle) {
      if ((threadIdx.x & 31) == 0) mbar_arrive(&s.run_done[turn]);
      continue;
    }
    tc_fence_after();
    const bool whole = r.s0 == 0 && r.s1 == r.steps;
    const int64_t out_row =
        (static_cast<int64_t>(r.seq.first + tok) * p.num_q_heads + r.h * G + g) * D;
    // notes are taken from the keys on that the item's (not the tile's) first token does not see
    bool noted = false;
    if (r.s1 * kStep > all_see - x * t.tpt)
#pragma unroll
      for (int e = 0; e < 16; ++e) noted |= s.noted[turn][e / 4][e % 4] != 0u;
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const int64_t part_block = static_cast<int64_t>(blockIdx.x) * 2 + (r.s0 > 0 ? 0 : 1);
    const int64_t part = part_block * 256 + x * 128 + row;
    float* part_row = t.part_acc + (part_block * (D / 4) * 256 + x * 128 + row) * 4;
    uint16_t* out = static_cast<uint16_t*>(p.out) + out_row;
    if (!whole && mine) {
      t.part_ml[2 * part] = m;
      t.part_ml[2 * part + 1] = l;
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      __syncwarp();
      tc_ld32(o, tm_o + 32 * c);
      tc_wait_ld();
      tc_loaded(o);
      if (mine && whole) {
        store_row16(out + 32 * c, o, inv, wide);
        store_row16(out + 32 * c + 16, o + 16, inv, wide);
      } else if (mine) {
        // column quads outermost: a warp's 32 rows make one 512-byte piece
        uint4* dst = reinterpret_cast<uint4*>(part_row) + 8 * c * 256;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dst[e * 256] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
    }
    if (noted && mine)
      add_noted<D>(t, r, s.noted[turn], sees, out_row, m == -INFINITY ? 0.f : m,
                   whole ? out : nullptr, part_row);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&s.run_done[turn]);
    tc_fence_before();
  }
}

// The copying warp's work, then what the join needs to know of an item that starts in this
// block and ends in a later one.
template <int D>
__device__ void run_copies(const TcParams& t, TcShared& s, unsigned char* q_smem,
                           unsigned char* ring) {
  const ChunkParams& p = t.c;
  const int tpi = 2 * t.tpt;
  copy_role<D>(t, s, q_smem, ring);
  Run r;
  r.begin(s, p);
  int64_t pos = s.begin;
  int parts = 0, first = 0, n = 0, item = 0, h = 0;
  if (!s.abort)
    for (; r.open(tpi); r.next(p, tpi)) {
      if (r.s0 == 0 && r.s1 < r.steps) {
        // borders inside the item that were not moved to its ends
        parts = 1;
        for (int64_t c = blockIdx.x + 1; c < s.blocks; ++c) {
          const int64_t off = s.total * c / s.blocks - pos - kOpen;
          if (r.steps - off <= s.snap) break;
          ++parts;
        }
        first = r.seq.first;
        n = r.seq.n;
        item = r.item;
        h = r.h;
      }
      pos += r.s1 - r.s0 + (r.s0 ? 0 : kOpen);
    }
  if ((threadIdx.x & 31) == 0) {
    int32_t* j = t.join + blockIdx.x * 8;
    j[0] = parts;
    j[1] = first;
    j[2] = n;
    j[3] = item;
    j[4] = h;
  }
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    chunk_tc_kernel(const __grid_constant__ TcParams t) {
  using C = TcCfg<D>;
  extern __shared__ unsigned char raw[];
  __shared__ TcShared s;
  const ChunkParams& p = t.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  unsigned char* base =
      raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);    // operand tiles: 1 KiB aligned
  unsigned char* q_smem = base;
  unsigned char* ring = base + 2 * C::kTileBytes;
  if (threadIdx.x == 0) {
    mbar_init(&s.q_full, 1);
    mbar_init(&s.q_empty, 1);
    mbar_init(&s.land, 1);
    mbar_init(&s.drain, 1);
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&s.kv_full[i], 1);
      mbar_init(&s.kv_empty[i], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s.s_full[x], 1);
      mbar_init(&s.p_ready[x], 4);
      mbar_init(&s.o_full[x], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&s.run_open[i], 1);
      mbar_init(&s.run_done[i], 8);              // the softmax warps
    }
    s.abort = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&s.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (warp == 9 && lane == 0) {
    prefetch_tensormap(&t.tmap_q);
    prefetch_tensormap(&t.tmap_k);
    prefetch_tensormap(&t.tmap_v);
  }
  grid_dependency_wait();
  const int tpi = 2 * t.tpt;
  if (warp < 2) {
    // the length of the line, then the border before this block (warp 0) and after it (warp 1)
    int64_t total = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      bool bad = false;
      const Seq q = b0 + lane < p.batch ? load_seq(p, b0 + lane, &bad) : Seq{0, 0, 0};
      if (bad && blockIdx.x == 0) set_status(p.status, SANTA_DEV_BAD_SEQLEN);
      int64_t v = seq_line(q, tpi) * p.num_kv_heads;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      total += v;
    }
    const int blocks =
        static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x), total)));
    const int snap = static_cast<int>(
        max(static_cast<int64_t>(1), min(static_cast<int64_t>(kSnap), total / (2 * blocks))));
    int start[4] = {p.batch, 0, 0, 0};
    const int border = min(static_cast<int>(blockIdx.x) + warp, blocks);
    const int64_t at = line_border(p, tpi, total, blocks, snap, border, start);
    if (lane == 0 && warp == 0) {
      for (int i = 0; i < 4; ++i) s.start[i] = start[i];
      s.begin = at;
      s.total = total;
      s.blocks = blocks;
      s.snap = snap;
    }
    if (lane == 0 && warp == 1) s.end = at;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    softmax_role<D>(t, s);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 8) {
      if (lane == 0) {
        mma_role<D>(t, s, smem_u32(q_smem), smem_u32(ring));
        tc_commit(&s.drain);                     // no product is in flight when TMEM is freed
        const uint64_t begin = global_timer_ns();
        while (!mbar_try_wait(&s.drain, 0) && global_timer_ns() - begin < kWaitLimitNs) {
        }
      }
      __syncwarp();
    } else if (warp == 9) {
      run_copies<D>(t, s, q_smem, ring);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && s.abort) set_status(p.status, SANTA_DEV_TIMEOUT);
  if (warp == 8) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(s.tmem));
  }
}

// Joins the partial results of the items that several blocks shared: block (c, y) takes 32 rows
// (a lane each) of the item that starts in block c, its parts in the line's order.  Most blocks
// find nothing to join and end at once, so 1536 threads per SM count for more than registers
// (512 tokens from empty 19.9 us, 20.3 with 1024, 21.7 with 512).
template <int D>
__global__ void __launch_bounds__(D * 4, 384 / D)
    chunk_tc_join_kernel(ChunkParams p, int tpt, const float* part_acc, const float* part_ml,
                         const int32_t* join, int num_blocks) {
  grid_dependency_wait();
  const int c0 = blockIdx.x;
  const int32_t* j = join + c0 * 8;
  const int parts = j[0];
  if (parts < 2 || c0 + parts > num_blocks) return;
  const int first = j[1], n = j[2], item = j[3], h = j[4];
  const int G = p.num_q_heads / p.num_kv_heads;
  const int row = blockIdx.y * 32 + (threadIdx.x & 31), in_tile = (row % 128) / G;
  const int tok = item * 2 * tpt + (row / 128) * tpt + in_tile;
  if (in_tile >= tpt || tok >= n) return;
  // part 0 is the second partial of block c0, part i the first one of block c0 + i
  auto at = [&](int i) { return static_cast<int64_t>(c0 + i) * 2 + (i == 0 ? 1 : 0); };
  // plain loads: this kernel may have been resident while the parts were written, so they are no
  // read-only data to it
  const float2* ml = reinterpret_cast<const float2*>(part_ml);
  float m = -INFINITY;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) m = fmaxf(m, ml[at(i) * 256 + row].x);
  const float ref = m == -INFINITY ? 0.f : m;
  // this warp's 8 columns
  const int q0 = (threadIdx.x / 32) * 2;
  const float4* acc = reinterpret_cast<const float4*>(part_acc);
  float l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float2 e = ml[at(i) * 256 + row];
    const float4 a = acc[(at(i) * (D / 4) + q0) * 256 + row];
    const float4 b = acc[(at(i) * (D / 4) + q0 + 1) * 256 + row];
    const float w = ex2_approx(e.x - ref);
    l = fmaf(w, e.y, l);
    o[0] = fmaf(w, a.x, o[0]);
    o[1] = fmaf(w, a.y, o[1]);
    o[2] = fmaf(w, a.z, o[2]);
    o[3] = fmaf(w, a.w, o[3]);
    o[4] = fmaf(w, b.x, o[4]);
    o[5] = fmaf(w, b.y, o[5]);
    o[6] = fmaf(w, b.z, o[6]);
    o[7] = fmaf(w, b.w, o[7]);
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  uint4* dst = reinterpret_cast<uint4*>(
      static_cast<uint16_t*>(p.out) +
      (static_cast<int64_t>(first + tok) * p.num_q_heads + h * G + (row % 128) % G) * D + q0 * 4);
  *dst = make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                    pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
}

// Blocks that the line is shared out to: one per SM, and no more than the longest possible line
// (known from the shape alone) has units.
int tc_blocks(int64_t num_tokens, int batch, int group, int hkv, int64_t max_len, int sms) {
  const int64_t tpi = 2 * (128 / group);
  const int64_t items = (num_tokens + tpi - 1) / tpi + batch;
  const int64_t steps = (max_len + kStep - 1) / kStep;
  const int64_t most = std::max<int64_t>(1, items * hkv * (steps + kOpen));
  return static_cast<int>(std::min<int64_t>(sms, most));
}

struct TcLayout {
  size_t acc, ml, join, bytes;
};
TcLayout tc_layout(int blocks, int d) {
  TcLayout l;
  l.acc = 0;
  l.ml = static_cast<size_t>(blocks) * 512 * d * sizeof(float);
  l.join = l.ml + static_cast<size_t>(blocks) * 512 * 2 * sizeof(float);
  l.bytes = l.join + static_cast<size_t>(blocks) * 8 * sizeof(int32_t);
  return l;
}

template <int D>
cudaError_t launch(const TcParams& t, int blocks, bool split, cudaStream_t stream) {
  using C = TcCfg<D>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = ensure_dynamic_smem(chunk_tc_kernel<D>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, chunk_tc_kernel<D>, t);
  if (e != cudaSuccess || !split) return e;
  cfg.gridDim = dim3(blocks, 8);
  cfg.blockDim = dim3(D * 4);                     // a warp for every 8 columns
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, chunk_tc_join_kernel<D>, t.c, t.tpt,
                            static_cast<const float*>(t.part_acc),
                            static_cast<const float*>(t.part_ml),
                            static_cast<const int32_t*>(t.join), blocks);
}

}  // namespace

size_t chunk_tc_workspace(int64_t num_tokens, int batch, int group, int hkv, int d,
                          int64_t max_len, int sms) {
  return tc_layout(tc_blocks(num_tokens, batch, group, hkv, max_len, sms), d).bytes;
}

int launch_chunk_tc(const ChunkParams& p, int d, void* workspace, int sms, cudaStream_t stream) {
  const int G = p.num_q_heads / p.num_kv_heads;
  const int64_t rows = p.num_pages * p.num_kv_heads * static_cast<int64_t>(p.team_size);
  if (rows > 0x7fffffffll) return SANTA_ERR_UNSUPPORTED;       // 32-bit row coordinates
  TcParams t = {};
  t.c = p;
  t.tpt = 128 / G;
  int rc = pool_tensor_map(&t.tmap_k, p.k_pool, rows, d);
  if (rc || (rc = pool_tensor_map(&t.tmap_v, p.v_pool, rows, d))) return rc;
  // queries [token][KV head][head of the group][d]: a box is one tile's rows, 64 elements wide
  TensorMapEncode encode = tensor_map_encode();
  if (!encode) return SANTA_ERR_CUDA;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(G),
                              static_cast<cuuint64_t>(p.num_kv_heads),
                              static_cast<cuuint64_t>(p.num_tokens)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2,
                                 static_cast<cuuint64_t>(G) * d * 2,
                                 static_cast<cuuint64_t>(p.num_q_heads) * d * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), 1, static_cast<cuuint32_t>(t.tpt)};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  if (encode(&t.tmap_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p.q), dims,
             strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return SANTA_ERR_CUDA;
  const int blocks = tc_blocks(p.num_tokens, p.batch, G, p.num_kv_heads,
                               static_cast<int64_t>(p.max_teams) * p.team_size, sms);
  const TcLayout l = tc_layout(blocks, d);
  unsigned char* base = static_cast<unsigned char*>(workspace);
  t.part_acc = reinterpret_cast<float*>(base + l.acc);
  t.part_ml = reinterpret_cast<float*>(base + l.ml);
  t.join = reinterpret_cast<int32_t*>(base + l.join);
  // An item is cut only where more than one step is left on both sides (line_border), so tables of
  // up to three steps need no join: 33 tokens on 100, 28 / 4 heads of 128, 12.0 us with a table of 2
  // or 3 pages, 13.6 with one of 4 (whose join finds nothing), 14.1 with one of 256.
  const bool split = blocks > 1 && static_cast<int64_t>(p.max_teams) * p.team_size > 3 * kStep;
  const cudaError_t e = d == 128 ? launch<128>(t, blocks, split, stream)
                                 : launch<64>(t, blocks, split, stream);
  return e == cudaSuccess ? SANTA_OK : SANTA_ERR_CUDA;
}

}  // namespace santa
