// q8_attend.cu — attention of one new token over a paged cache of 8-bit rows, the cache's length split
// among blocks and joined.
//
//   s_j = (q . c_j) ks_j / sqrt(d),  optionally  s_j := cap tanh(s_j / cap)
//   out = sum_j w_j e^{s_j} vs_j c'_j / sum_j w_j e^{s_j}
//
// over the tokens j that are seen (below the length, inside the window, in the listed teams), c and c'
// the codes of key and value, ks and vs their rows' scales, and w = 1 / pi of a listed team.  The
// scale of a key multiplies its whole score and the scale of a value its weight, so that no element
// is scaled by itself.
//
// Work.  The tiles (32 tokens) of all units (sequence, KV head) lie on one line, which the warps of
// the grid share evenly, whatever the lengths of the batch are; the lengths are read on the device, and
// opening a unit counts like two tiles.  A warp takes its stretch of the line through a ring of its own in
// shared memory (asynchronous 16-byte copies), without a barrier.  A unit that lies within one
// stretch is finished by its warp; of the others a warp holds a piece.  At its end a block merges its
// warps' pieces; a unit that goes beyond the block leaves a part in the workspace, and a second launch
// joins the parts in the order of the line.
//
// A tile.  Codes become fp16 exactly (int8 by the bits of 1024 + code, e4m3 by conversion) and go to
// the matrix units as the A operand of m16n8k16, tokens x dimensions for the scores and dimensions x
// tokens for the output, so that the group's up to 8 query heads are the n = 8 columns.  Both are read
// by ldmatrix as pairs of bytes: four dimensions of a key, or (transposed) two dimensions of two
// values' tokens, stand in a register, and which dimension stands at which k is free.
//   - q enters as fp16 pieces (one for bf16, two for fp32) over a power of two, by which the head's largest
//     element becomes 2^14 .. 2^15: bf16 elements are exact down to 2^-31 of it.  The second piece is what
//     the first leaves, 2^11 up, with products of its own, so that an fp32 element keeps 2^-22 of itself
//     down to 2^-28 of the largest, and 2^-50 of the largest below.
//   - The weights enter the second product as two fp16 pieces (one would leave 2^-12 of error in an fp32
//     result) of p_j vs_j over a power of two, by which the largest p vs so far becomes 2^7 .. 2^15: the
//     scales of values may lie any powers of two apart.  The second piece is what the first leaves, 2^11 up,
//     with products of its own: fp16 rounds at 2^-25 below 2^-14, and its sums come down again with 2^-11.
//     A weight so keeps 2^-22 of itself down to 2^-21 of the largest, and 2^-43 of the largest below.
//   - The reference of the exponentials is raised only when a score passes it by 8 (powers of two),
//     which is seldom after a few tiles, so a tile has no reduction among lanes.
//   - The matrix units cut what they add.  A score's products (of first pieces) start from zero for every 32
//     dimensions, those of the output for every tile, and are added to the running sums in fp32 with rounding.
//
// Bound by HBM where there is much to read (2 d + 8 bytes for every token and head), by latency
// where there is little: a launch's chain is lengths -> page ids -> tiles -> pieces -> parts, and its code
// is fetched as it is first run, so the code that short calls run is kept short.  The matrix units are a
// fifth busy: with at most 8 columns mma.sync from registers feeds them well enough, and codes have to
// pass through registers anyway.  Measured on GB300 (bf16 queries, 32 / 8 heads of 128, int8, against a
// measured copy): 16 sequences at 32K and below 138 us, 95%; 16 at 32K with groups of 1 and 8 98 and 96%,
// with fp32 queries 87% (twice the score products; e4m3 98%), capped scores 88%, heads of 64 83% (e4m3 89%);
// 4 x 128K e4m3 with capped scores 86 us, 89%; one sequence of 32K 15.4 us; 523 tokens 8.7 us.
// Both sides of the choices, each on the kernel as it was then: one token at a time per warp 2445 us for the 16 sequences; stretches per
// block with a merge for each unit 164, per warp 149; an opening counted as 0, 1, 2 tiles 156, 149, 139;
// twelve warps and two stages 144 against 149 (eight and three), but 523 tokens 12.3 against 10.3; the last
// block to arrive joins the parts 11.7 and 30.5 us (523 tokens, one sequence of 32K) against 10.3 and 16.6
// with the second launch.
#include <algorithm>

#include "kernels.h"
#include "q8.cuh"

namespace santa {

namespace {

constexpr int kTile = 32;                  // tokens of a tile
constexpr int kJoinWarps = 8;
constexpr int kJoinThreads = kJoinWarps * 32;
constexpr int kStages = 3;                 // tiles of a warp's ring
constexpr int kOpen = 2;                   // what opening a unit counts, in tiles
constexpr int kJoinRounds = 8;             // 32 blocks each that a unit may reach over
constexpr int kBeyond = INT32_MAX - 16;    // behind every place of a line
constexpr int64_t kMostPlaces = INT32_MAX - (1 << 16);
constexpr float kNoScore = -1e38f;         // a reference before the first score
constexpr float kSlack = 8.f;              // how far a score may pass the reference (base 2)
constexpr int kQueryBits = 14;             // a head's largest element stands at 2^14 .. 2^15
constexpr int kWeightBits = 7;             // the largest weight starts out at 2^7 .. 2^8
constexpr float kTopWeight = 0x1p15f;      // and may grow to this (fp16 ends at 65504)
constexpr float kUp = 0x1p11f;             // of second pieces

template <int D>
struct Ring {
  // of a block.  Rows of 64 bytes are half the bytes for the same scores: 16 sequences at 32K take 101 us
  // with twelve warps and 121 with eight, a call of a few hundred tiles 9.9 against 8.8.  Rows of 128 leave
  // registers and shared memory for eight.
  static constexpr int kWarps = D == 128 ? 8 : 12;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kCodes = kTile * D;                     // bytes of a tile's keys or values
  static constexpr int kStage = 2 * kCodes + 2 * kTile * 4;    // keys, values, scales
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kBytes = kWarps * kWarp;
  static constexpr int kPieceRow = D + 4;                      // floats of a head in a piece
  static_assert(kMaxGroup * kPieceRow * 4 <= kWarp, "a piece fits its warp's ring");
};

// Byte of 16-byte piece `chunk` of row r in a tile's block of rows: eight consecutive rows' pieces of
// one chunk lie in eight different groups of four banks.
template <int D>
__device__ __forceinline__ int piece_at(int r, int chunk) {
  if constexpr (D == 128) return r * 128 + ((chunk ^ (r & 7)) << 4);
  return (r >> 1) * 128 + (r & 1) * 64 + ((chunk ^ (r >> 1 & 3)) << 4);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_fill(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Adds a matrix product to a running sum, in register pairs or one by one; which of them costs less depends
// on the code around it (16 x 32K tokens, int8: scores of bf16 queries in pairs 166 us, one by one 172; of
// fp32 queries 191 and 188; outputs 170 and 166).
template <bool PAIRS>
__device__ __forceinline__ void add_product(float (&sum)[4], const float (&c)[4]) {
  if constexpr (PAIRS) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float2 r = halves(add_pair(pair(sum[i], sum[i + 1]), pair(c[i], c[i + 1])));
      sum[i] = r.x, sum[i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += c[i];
  }
}

// The two code pairs of a word, bytes (0, 1) and (2, 3), as fp16.  int8: with its sign bit turned
// a code is u = code + 128, 0x6400 | u is 1024 + u, and 1152 less is the code; exact.
template <int C>
__device__ __forceinline__ void pairs_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (C == kCodeI8) {
    const uint32_t u = w ^ 0x80808080u;
    lo = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
    hi = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    lo = e4m3_to_f16x2(static_cast<uint16_t>(w));
    hi = e4m3_to_f16x2(static_cast<uint16_t>(w >> 16));
  }
}
// The same of a register with two dimensions of two tokens, bytes (d, d + 1) of one and of the next:
// each dimension's pair of tokens.
template <int C>
__device__ __forceinline__ void tokens_to_f16(uint32_t w, uint32_t& d0, uint32_t& d1) {
  if constexpr (C == kCodeI8) {
    const uint32_t u = w ^ 0x80808080u;
    d0 = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4240), 0x64806480u);
    d1 = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4341), 0x64806480u);
  } else {
    pairs_to_f16<C>(__byte_perm(w, 0, 0x3120), d0, d1);
  }
}

// ---------------------------------------------------------------- the line of tiles

// A unit's tokens: positions lo .. len - 1 (dense), or `count` listed teams, in `tiles` tiles.
struct Unit {
  int len, lo;         // at most 2^14 pages of 2^7 tokens
  int count;
  int tiles;
};
// From a sequence's length and (listed) a unit's count of teams; what is out of range is judged here and
// told if `tell`.
__device__ __forceinline__ Unit judge_unit(const Q8AttendParams& p, int len, int count, bool tell) {
  Unit u;
  u.len = len;
  u.count = 0;
  if (len < 0 || len > p.max_teams * p.team_size) {
    if (tell) set_status(p.status, SANTA_DEV_BAD_SEQLEN);
    u.len = 0;
  }
  u.lo = p.window > 0 && u.len > p.window ? u.len - p.window : 0;
  if (p.sel_ids) {
    u.count = min(max(count, 0), p.num_draws);
    if (count != u.count && tell) set_status(p.status, SANTA_DEV_BAD_SEL);
    if (u.len == 0) u.count = 0;
    u.tiles = u.count * (p.team_size / kTile);
  } else {
    u.tiles = (u.len + kTile - 1) / kTile - u.lo / kTile;
  }
  return u;
}
__device__ __forceinline__ Unit load_unit(const Q8AttendParams& p, int b, int h, bool tell) {
  return judge_unit(p, p.seq_lens[b],
                    p.sel_ids ? p.sel_count[static_cast<int64_t>(b) * p.num_kv_heads + h] : 0, tell);
}
// A unit's length on the line: its tiles and its opening.
__device__ __forceinline__ int span(const Unit& u) { return u.tiles ? u.tiles + kOpen : 0; }

// A place on the line: unit (b, h), which begins at `base`; its tile k stands at base + kOpen + k.
struct Walk {
  int b, h;
  int base;
  Unit u;
};
__device__ __forceinline__ void next_unit(const Q8AttendParams& p, Walk& w) {
  w.base += span(w.u);
  if (w.b == p.batch - 1 && w.h == p.num_kv_heads - 1) {
    // not reached while lengths and lists stay as they are; if not, the walk ends here
    w.base = kBeyond;
    w.u = Unit{0, 0, 0, 0};
    return;
  }
  const bool wrap = ++w.h == p.num_kv_heads;
  if (wrap) {
    w.h = 0;
    ++w.b;
  }
  if (wrap || p.sel_ids) w.u = load_unit(p, w.b, w.h, false);
}
// To the unit that owns place `at` (at < the line's length).
__device__ __forceinline__ void walk_to(const Q8AttendParams& p, Walk& w, int at) {
  while (w.base + span(w.u) <= at) next_unit(p, w);
}

__device__ __forceinline__ int warp_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}
template <int W>
__device__ __forceinline__ int block_scan(int v, int* warp_sums) {
  const int warp = threadIdx.x >> 5;
  v = warp_scan(v);
  if ((threadIdx.x & 31) == 31) warp_sums[warp] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w)
    if (w < warp) v += warp_sums[w];
  return v;
}

// ---------------------------------------------------------------- the attention

// What a warp knows of its next tiles' pages: 32 consecutive teams of a sequence (dense) or slots of a
// unit's list, one per lane.
struct PageCache {
  int b, h;            // of which sequence (and unit, listed); b = -1: nothing yet
  int first;           // team or slot of lane 0
  int team;            // listed: -1 for one that is left out
  int page;            // -1: out of range
  float bias;          // listed: -log2 pi
};

template <int NQ, int C, int D>
struct Warp {
  static constexpr int kSteps = D / 16;      // 16-dimension pieces: k steps of a score, tiles of out
  uint32_t q[NQ][kSteps][2];
  float acc[kSteps][4];      // dimensions 16 j + 2 g (+ 1) of heads 2t, 2t + 1 (g, t: lane / 4, lane % 4)
  float ref[2];              // of heads 2t and 2t + 1: reference of the exponentials
  float sum[2];              // this lane's share of the sum of weights
  float big[2], inv[2];      // largest |p vs| (at least), and the power of two that scales weights
  float qs[2];               // score of a unit product, base 2 (or over the cap)
};

// Copies tile `k` of a unit into a stage and notes what the consumer must know of it: the range of its
// tokens that are seen and the bias.
template <int D>
__device__ __forceinline__ void issue_tile(const Q8AttendParams& p, const Walk& w, int k_unit,
                                           PageCache& pc, uint8_t* stage, int2* note) {
  const int lane = threadIdx.x & 31;
  const int T = p.team_size, per = T == 128 ? 2 : 1;  // log2 of a page's tiles
  // tile of the unit, or of the sequence (at most 2^16 of them); then slot or team, and row in it
  const int i = k_unit + (p.sel_ids ? 0 : w.u.lo / kTile);
  const int at = i >> per, row = (i & ((1 << per) - 1)) * kTile;
  if (__builtin_expect(pc.b != w.b || (p.sel_ids && pc.h != w.h) || at < pc.first || at >= pc.first + 32, 0)) {
    pc.b = w.b;
    pc.h = w.h;
    pc.first = at;
    const int mine = at + lane;
    pc.bias = 0.f;
    pc.page = -1;
    pc.team = -1;
    if (!p.sel_ids) {
      if (mine * T < w.u.len) pc.team = mine;
    } else if (mine < w.u.count) {
      const int64_t slot = (static_cast<int64_t>(w.b) * p.num_kv_heads + w.h) * p.num_draws + mine;
      const int team = p.sel_ids[slot];
      const float pi = p.pi[slot];
      if (team >= 0 && team < p.max_teams && team * T < w.u.len && pi > 0.f && pi < INFINITY) {
        // a team before the window: its page may have been given back, and is not looked at
        if ((team + 1) * T > w.u.lo) pc.team = team;
        pc.bias = -log2f(pi);
      } else {
        set_status(p.status, SANTA_DEV_BAD_SEL);
      }
    }
    if (pc.team >= 0) {
      pc.page = p.page_table[static_cast<int64_t>(w.b) * p.max_teams + pc.team];
      if (pc.page < 0 || pc.page >= p.num_pages) {
        set_status(p.status, SANTA_DEV_BAD_PAGE);
        pc.page = -1;
      }
    }
  }
  const int from = at - pc.first;
  const int team = __shfl_sync(0xffffffffu, pc.team, from);
  const int page = __shfl_sync(0xffffffffu, pc.page, from);
  const float bias = __shfl_sync(0xffffffffu, pc.bias, from);
  const int t0 = team * T + row;
  int n0 = min(max(w.u.lo - t0, 0), kTile);
  int n1 = min(max(w.u.len - t0, 0), kTile);
  if (page < 0 || n0 >= n1) n0 = n1 = 0;
  if (lane == 0) *note = make_int2(n0 | n1 << 16, __float_as_int(bias));
  if (n1 > 0) {
    constexpr int kCols = D / 16, kRows = 32 / kCols;   // pieces of a row; rows per round
    const int64_t first = (static_cast<int64_t>(page) * p.num_kv_heads + w.h) * T + row;
    const int r0 = lane / kCols, chunk = lane % kCols;
    const uint8_t* k = static_cast<const uint8_t*>(p.k) + first * D + lane * 16;
    const uint8_t* v = static_cast<const uint8_t*>(p.v) + first * D + lane * 16;
    const uint32_t to = smem_u32(stage);
    if (__builtin_expect(n0 == 0 && n1 == kTile, 1)) {
#pragma unroll
      for (int e = 0; e < kTile / kRows; ++e) {
        cp_async16(to + piece_at<D>(e * kRows + r0, chunk), k + e * 512);
        cp_async16(to + kTile * D + piece_at<D>(e * kRows + r0, chunk), v + e * 512);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kTile / kRows; ++e) {
        const int r = e * kRows + r0;
        const bool on = r >= n0 && r < n1;              // rows that are not seen become zeros
        cp_async16_fill(to + piece_at<D>(r, chunk), k + e * 512, on);
        cp_async16_fill(to + kTile * D + piece_at<D>(r, chunk), v + e * 512, on);
      }
    }
    if (lane < 2 * kTile / 4) {
      const float* s = (lane < kTile / 4 ? p.k_scale : p.v_scale) + first + lane % (kTile / 4) * 4;
      cp_async16(to + 2 * kTile * D + lane * 16, s);
    }
  }
}

// A unit's queries as they are in memory: a lane's share of the B operands of its scores.  Step s has
// dimensions 16 s + 4 t + 0 .. 3 of head g, as a key's register has them.
template <int NQ, int D>
struct Queries {
  uint32_t w[D / 16][2 * NQ];
};
template <int NQ, int D>
__device__ __forceinline__ void fetch_queries(const Q8AttendParams& p, int b, int h,
                                              Queries<NQ, D>& raw) {
  const int lane = threadIdx.x & 31, head = lane >> 2, t = lane & 3;
  const int G = p.num_q_heads / p.num_kv_heads;
  const int64_t at = (static_cast<int64_t>(b) * p.num_q_heads + h * G + head) * D + 4 * t;
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    if constexpr (NQ == 1) {
      uint2 v = make_uint2(0, 0);
      if (head < G) v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + at + 16 * s);
      raw.w[s][0] = v.x, raw.w[s][1] = v.y;
    } else {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (head < G) v = *reinterpret_cast<const uint4*>(static_cast<const float*>(p.q) + at + 16 * s);
      raw.w[s][0] = v.x, raw.w[s][1] = v.y, raw.w[s][2 * NQ - 2] = v.z, raw.w[s][2 * NQ - 1] = v.w;
    }
  }
}

// A unit's beginning: its queries as pieces, no score yet.
template <int NQ, int C, int D>
__device__ __forceinline__ void open_unit(const Q8AttendParams& p, const Queries<NQ, D>& raw,
                                          Warp<NQ, C, D>& w) {
  const int t = threadIdx.x & 3;
  float x[D / 4];
  uint32_t top = 0;
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    float* y = x + 4 * s;
    if constexpr (NQ == 1) {
      y[0] = bf16_lo(raw.w[s][0]), y[1] = bf16_hi(raw.w[s][0]);
      y[2] = bf16_lo(raw.w[s][1]), y[3] = bf16_hi(raw.w[s][1]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = __uint_as_float(raw.w[s][i]);
    }
  }
#pragma unroll
  for (int i = 0; i < D / 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // the power of two and its reciprocal as exponent fields; zeros and tiny queries keep a factor inside
  // fp32's range
  const uint32_t e = min(max(top >> 23, 16u), 254u) - kQueryBits;
  const float down = __uint_as_float((254u - e) << 23), up = __uint_as_float(e << 23);
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = x[4 * s + 2 * i] * down, c = x[4 * s + 2 * i + 1] * down;
      w.q[0][s][i] = pack_f16(a, c);
      if constexpr (NQ == 2) {
        const float2 got = f16x2_to_f32(w.q[0][s][i]);
        w.q[NQ - 1][s][i] = pack_f16((a - got.x) * kUp, (c - got.y) * kUp);
      }
    }
  }
  constexpr float kLog2e = 1.4426950408889634f;
  const float f = up * (p.softcap > 0.f ? p.scale / p.softcap : p.scale * kLog2e);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w.qs[i] = __shfl_sync(0xffffffffu, f, (2 * t + i) * 4);
    w.ref[i] = kNoScore;
    w.sum[i] = w.big[i] = 0.f;
    w.inv[i] = 1.f;
  }
#pragma unroll
  for (int j = 0; j < D / 16; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) w.acc[j][i] = 0.f;
}

// Raises the references to this tile's largest score and weight: x[2 k + i] is the score of token
// 8 k + lane / 4 and head 2 t + i, vs[k] the token's value scale.
template <int NQ, int C, int D>
__device__ __forceinline__ void raise(Warp<NQ, C, D>& w, const float (&x)[8], const float (&vs)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float top = fmaxf(fmaxf(x[i], x[2 + i]), fmaxf(x[4 + i], x[6 + i]));
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool up = top > w.ref[i];
    const float keep = up ? ex2_approx(w.ref[i] - top) : 1.f;
    if (up) w.ref[i] = top;
    float big = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) big = fmaxf(big, fabsf(ex2_approx(x[2 * k + i] - w.ref[i]) * vs[k]));
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    big = fmaxf(big, w.big[i] * keep);
    w.big[i] = big;
    float inv = w.inv[i];
    if (big > 0.f) {
      const uint32_t e = min(max(__float_as_uint(big) >> 23, 1u + kWeightBits), 253u);
      inv = __uint_as_float((254u + kWeightBits - e) << 23);
    }
    // inv / w.inv as a power of two inside fp32's range
    const int d = static_cast<int>(__float_as_uint(inv) >> 23) - static_cast<int>(__float_as_uint(w.inv[i]) >> 23);
    const float f = keep * __uint_as_float(static_cast<uint32_t>(min(max(d, -126), 127) + 127) << 23);
    w.inv[i] = inv;
    w.sum[i] *= keep;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      w.acc[j][i] *= f;
      w.acc[j][2 + i] *= f;
    }
  }
}

template <int NQ, int C, int D>
__device__ __forceinline__ void attend_tile(const Q8AttendParams& p, Warp<NQ, C, D>& w,
                                            const uint8_t* stage, int2 note) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  const float* scales = reinterpret_cast<const float*>(stage + 2 * kTile * D);
  const uint32_t at = smem_u32(stage);
  const int n0 = note.x & 0xffff, n1 = note.x >> 16;
  if (n1 == 0) return;
  float x[8], ks[4], vs[4];                          // token 8 k + g; score 2 k + i: head 2 t + i
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float sum[4] = {0.f, 0.f, 0.f, 0.f}, low[4] = {0.f, 0.f, 0.f, 0.f};   // low: of second pieces
#pragma unroll
    for (int s = 0; s < D / 16; s += 2) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
      // rows 16 m + 0 .. 7 and 8 .. 15, pieces s and s + 1: matrix lane / 8's row is given by the lane
      uint32_t a[4];
      ldmatrix_x4(a, at + piece_at<D>(16 * m + (lane & 15), s + (lane >> 4)));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t f[4];
        pairs_to_f16<C>(a[2 * k], f[0], f[2]);
        pairs_to_f16<C>(a[2 * k + 1], f[1], f[3]);
#pragma unroll
        for (int n = 0; n < NQ; ++n) mma_f16_16816(n ? low : c, f, w.q[n][s + k][0], w.q[n][s + k][1]);
      }
      add_product<NQ == 1>(sum, c);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      ks[2 * m + r] = scales[16 * m + 8 * r + g];
      vs[2 * m + r] = scales[kTile + 16 * m + 8 * r + g];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[4 * m + i] = NQ == 1 ? sum[i] : fmaf(low[i], 1.f / kUp, sum[i]);
  }
  const bool part = n0 > 0 || n1 < kTile;
  if (__builtin_expect(part, 0)) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (8 * k + g < n0 || 8 * k + g >= n1) vs[k] = 0.f;
  }
  // differences from the reference, one rounding each
  const float bias = __int_as_float(note.y);
  float y[8], e[8], pw[8];
  auto scores = [&](float r0, float r1) {
    const float off[2] = {bias - r0, bias - r1};
    if (__builtin_expect(p.softcap > 0.f, 0)) {
      const float cap = p.softcap * 1.4426950408889634f;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fmaf(cap, tanhf(x[i] * (ks[i >> 1] * w.qs[i & 1])), off[i & 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], ks[i >> 1] * w.qs[i & 1], off[i & 1]);
    }
    if (__builtin_expect(part, 0)) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * (i >> 1) + g < n0 || 8 * (i >> 1) + g >= n1) y[i] = -INFINITY;
    }
  };
  auto weigh = [&]() {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = ex2_approx(y[i]);
      pw[i] = e[i] * vs[i >> 1] * w.inv[i & 1];
    }
  };
  scores(w.ref[0], w.ref[1]);
  weigh();
  bool over = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) over |= y[i] > kSlack || fabsf(pw[i]) > kTopWeight;
  if (__builtin_expect(__any_sync(0xffffffffu, over), 0)) {
    scores(0.f, 0.f);
    raise(w, y, vs);
    scores(w.ref[0], w.ref[1]);
    weigh();
  }
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w.sum[0] += e[2 * k];
    w.sum[1] += e[2 * k + 1];
    hi[k] = pack_f16(pw[2 * k], pw[2 * k + 1]);
    const float2 got = f16x2_to_f32(hi[k]);          // what it leaves is exact in fp32
    lo[k] = pack_f16((pw[2 * k] - got.x) * kUp, (pw[2 * k + 1] - got.y) * kUp);
    hi[k] = movmatrix_trans(hi[k]);
    lo[k] = movmatrix_trans(lo[k]);
  }
  // values: matrix lane / 8 is token group lane / 8; a register has two dimensions of two tokens
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    uint32_t a[4];
    ldmatrix_x4_trans(a, at + kTile * D + piece_at<D>(lane, j));
    float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint32_t f[4];
      tokens_to_f16<C>(a[2 * m], f[0], f[1]);
      tokens_to_f16<C>(a[2 * m + 1], f[2], f[3]);
      mma_f16_16816(c, f, hi[2 * m], hi[2 * m + 1]);
      mma_f16_16816(c2, f, lo[2 * m], lo[2 * m + 1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = fmaf(c2[i], 1.f / kUp, c[i]);
    add_product<false>(w.acc[j], c);
  }
}

// Of a power of two between 2^-126 and 2^126.
__device__ __forceinline__ float reciprocal(float two_to_k) {
  return __uint_as_float((254u << 23) - __float_as_uint(two_to_k));
}

// The weights' sums of a warp's unit, over the lanes that share its heads.
template <int NQ, int C, int D>
__device__ __forceinline__ void close_sums(Warp<NQ, C, D>& w) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) w.sum[i] += __shfl_xor_sync(0xffffffffu, w.sum[i], o);
}

// Writes a piece: rows of `stride` floats, one for each head of the group, and (reference, sum).
template <int NQ, int C, int D>
__device__ __forceinline__ void store_piece(Warp<NQ, C, D>& w, int G, float* rows, int stride,
                                            float (*ml)[2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  close_sums(w);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (2 * t + i >= G) continue;
    const float back = reciprocal(w.inv[i]);
    float* row = rows + (2 * t + i) * stride + 2 * g;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
      *reinterpret_cast<float2*>(row + 16 * j) =
          make_float2(w.acc[j][i] * back, w.acc[j][2 + i] * back);
    if (g == 0) {
      ml[2 * t + i][0] = w.ref[i];
      ml[2 * t + i][1] = w.sum[i];
    }
  }
}

// Writes a whole unit's rows of out.
template <int NQ, int C, int D>
__device__ __forceinline__ void store_unit(Warp<NQ, C, D>& w, int G, float* out) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  close_sums(w);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (2 * t + i >= G) continue;
    const float back = reciprocal(w.inv[i]), f = w.sum[i] == 0.f ? 0.f : 1.f / w.sum[i];
    float* row = out + (2 * t + i) * D + 2 * g;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
      *reinterpret_cast<float2*>(row + 16 * j) =
          make_float2(w.acc[j][i] * back * f, w.acc[j][2 + i] * back * f);
  }
}

// Adds (x, m, l) to a running (sum, top, z): sums relative to the largest reference.
template <int N>
__device__ __forceinline__ void add_part(float (&sum)[N], float& top, float& z, const float (&x)[N],
                                         float m, float l) {
  const float best = fmaxf(top, m);
  const float keep = ex2_approx(top - best), f = ex2_approx(m - best);
  top = best;
  z = z * keep + l * f;
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = sum[i] * keep + x[i] * f;
}

// Adds a chain of a unit's pieces, in the order of the line, by all threads of the block: a head's four
// dimensions each.  `on_count` pieces lie `on_stride` floats apart from `on` on, `closing` (or null) follows
// them; ml: their (reference, sum) by head.  `whole`: to rows of out; else to a part and its ml.
template <int D>
__device__ __forceinline__ void add_chain(const float* on, int on_stride, int on_count, const float* closing,
                                          const float* ml_on, const float* ml_closing, int G, bool whole,
                                          float* rows, float* ml) {
  const int count = on_count + (closing != nullptr);
  for (int e = threadIdx.x; e < G * (D / 4); e += Ring<D>::kThreads) {
    const int head = e / (D / 4), dim = e % (D / 4) * 4;
    float sum[4] = {}, top = kNoScore, z = 0.f;
    for (int i = 0; i < count; ++i) {
      const float* row = i < on_count ? on + i * on_stride + head * Ring<D>::kPieceRow : closing + head * D;
      const float* at = (i < on_count ? ml_on + i * kMaxGroup * 2 : ml_closing) + head * 2;
      const float4 v = *reinterpret_cast<const float4*>(row + dim);
      const float x[4] = {v.x, v.y, v.z, v.w};
      add_part(sum, top, z, x, at[0], at[1]);
    }
    const float f = !whole ? 1.f : z == 0.f ? 0.f : 1.f / z;
    *reinterpret_cast<float4*>(rows + head * D + dim) =
        make_float4(sum[0] * f, sum[1] * f, sum[2] * f, sum[3] * f);
    if (!whole && dim == 0) *reinterpret_cast<float2*>(ml + head * 2) = make_float2(top, z);
  }
}

template <int NQ, int C, int D>
__global__ void __launch_bounds__(Ring<D>::kThreads, 1) q8_attend_kernel(Q8AttendParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int sums[2][Ring<D>::kWarps];
  __shared__ int total_s, start_s[Ring<D>::kWarps][2];   // element of a warp's start, its place
  __shared__ int2 notes[Ring<D>::kWarps][kStages];
  // each warp's piece that closes a unit which another warp opened (0, in the workspace), and its
  // piece that goes on beyond its stretch (1, in its ring): of which unit (-1: none), whether it has the
  // unit's first tile, and its (reference, sum)
  __shared__ int owner_s[2][Ring<D>::kWarps];
  __shared__ bool first_s[Ring<D>::kWarps];
  __shared__ float ml_s[2][Ring<D>::kWarps][kMaxGroup][2];
  using R = Ring<D>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = p.num_q_heads / p.num_kv_heads;
  grid_dependency_wait();

  // the line's length, and where this warp's stretch of it starts: by sequences (dense) or units
  const int elems = p.batch * (p.sel_ids ? p.num_kv_heads : 1);
  const int heads = p.sel_ids ? 1 : p.num_kv_heads;
  const bool tell = blockIdx.x == 0;
  const unsigned warps = gridDim.x * Ring<D>::kWarps;
  int total, share, c0;
  Walk use;
  use.h = 0;
  if (elems <= 32) {
    // every warp for itself, without a barrier
    int len = 0, count = 0;
    if (lane < elems) {
      len = p.seq_lens[p.sel_ids ? static_cast<unsigned>(lane) / static_cast<unsigned>(p.num_kv_heads) : lane];
      if (p.sel_ids) count = p.sel_count[lane];
    }
    const int mine = span(judge_unit(p, len, count, tell && warp == 0)) * heads;
    const int upto = warp_scan(mine);
    total = __shfl_sync(0xffffffffu, upto, 31);
    share = (static_cast<unsigned>(total) + warps - 1) / warps;
    c0 = (blockIdx.x * Ring<D>::kWarps + warp) * share;
    const int from = max(__ffs(__ballot_sync(0xffffffffu, upto > c0 && upto - mine <= c0)) - 1, 0);
    use.base = __shfl_sync(0xffffffffu, upto - mine, from);
    use.u = judge_unit(p, __shfl_sync(0xffffffffu, len, from), __shfl_sync(0xffffffffu, count, from), false);
    use.b = p.sel_ids ? from / p.num_kv_heads : from;
    if (p.sel_ids) use.h = from - use.b * p.num_kv_heads;
  } else {
    // by the block, a thread each; more elements than threads are read twice, for the length and the starts
    constexpr int kThreads = Ring<D>::kThreads;
    auto span_of = [&](int e, bool say) {
      if (e >= elems) return 0;
      const int b = p.sel_ids ? e / p.num_kv_heads : e;
      return span(load_unit(p, b, p.sel_ids ? e - b * p.num_kv_heads : 0, say)) * heads;
    };
    int mine = 0, upto = 0;
    total = 0;
    for (int e0 = 0; e0 < elems; e0 += kThreads) {
      mine = span_of(e0 + threadIdx.x, tell);
      upto = total + block_scan<Ring<D>::kWarps>(mine, sums[(e0 / kThreads) & 1]);
      if (threadIdx.x == kThreads - 1) total_s = upto;
      __syncthreads();
      total = total_s;
      __syncthreads();
    }
    share = (static_cast<unsigned>(total) + warps - 1) / warps;
    c0 = blockIdx.x * Ring<D>::kWarps * share;       // of the block, first
    int before = 0;
    for (int e0 = 0; e0 < elems && c0 < total; e0 += kThreads) {
      if (elems > kThreads) {
        mine = span_of(e0 + threadIdx.x, false);
        upto = before + block_scan<Ring<D>::kWarps>(mine, sums[(e0 / kThreads) & 1]);
      }
#pragma unroll
      for (int w = 0; w < Ring<D>::kWarps; ++w)
        if (upto > c0 + w * share && upto - mine <= c0 + w * share) {
          start_s[w][0] = e0 + threadIdx.x;
          start_s[w][1] = upto - mine;
        }
      if (__syncthreads_or(upto > c0 + (Ring<D>::kWarps - 1) * share)) break;
      if (threadIdx.x == kThreads - 1) total_s = upto;
      __syncthreads();
      before = total_s;
      __syncthreads();
    }
    c0 += warp * share;
    if (c0 < total) {
      const int elem = start_s[warp][0];
      use.b = p.sel_ids ? elem / p.num_kv_heads : elem;
      if (p.sel_ids) use.h = elem - use.b * p.num_kv_heads;
      use.base = start_s[warp][1];
      use.u = load_unit(p, use.b, use.h, false);
    }
  }
  const int c1 = min(c0 + share, total);

  if (threadIdx.x < 2 * Ring<D>::kWarps) owner_s[threadIdx.x & 1][threadIdx.x >> 1] = -1;
  __syncthreads();
  uint8_t* ring = smem + warp * R::kWarp;
  float* closing = p.piece + (static_cast<int64_t>(blockIdx.x) * Ring<D>::kWarps + warp) * kMaxGroup * D;
  if (c0 < c1) {
    walk_to(p, use, c0);
    Walk ask = use;
    int ask_k = max(c0 - use.base - kOpen, 0);       // next tile of ask's unit
    PageCache pc;
    pc.b = -1;
    bool more = true;
    int put = 0, get = 0;
    Queries<NQ, D> raw;
    fetch_queries<NQ, D>(p, use.b, use.h, raw);
    auto ask_next = [&]() {
      if (more) {
        while (ask_k >= ask.u.tiles) {               // on to the next unit with a tile
          next_unit(p, ask);
          ask_k = 0;
          if (ask.base >= c1) break;
        }
        more = ask.base + kOpen + ask_k < c1;
        if (more) {
          issue_tile<D>(p, ask, ask_k, pc, ring + put * R::kStage, &notes[warp][put]);
          ++ask_k;
        }
      }
      cp_async_commit();
      put = put + 1 == kStages ? 0 : put + 1;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) ask_next();

    Warp<NQ, C, D> w;
    for (;;) {
      const int k0 = max(c0 - use.base - kOpen, 0), k1 = min(c1 - use.base - kOpen, use.u.tiles);
      if (k0 < k1) {
        open_unit(p, raw, w);
        for (int k = k0; k < k1; ++k) {
          cp_async_wait<kStages - 2>();
          __syncwarp();
          ask_next();
          attend_tile(p, w, ring + get * R::kStage, notes[warp][get]);
          get = get + 1 == kStages ? 0 : get + 1;
          __syncwarp();
        }
      }
      // on to the next unit with a tile, whose queries are asked for before this one's results are stored
      const Walk now = use;
      const bool last = now.base + span(now.u) >= c1;
      if (!last) {
        do next_unit(p, use);
        while (use.u.tiles == 0 && use.base < c1);
        fetch_queries<NQ, D>(p, use.b, use.h, raw);
      }
      if (k0 < k1) {
        const int unit = now.b * p.num_kv_heads + now.h;
        if (k1 < now.u.tiles) {
          if (lane == 0) {
            owner_s[1][warp] = unit;
            first_s[warp] = k0 == 0;
          }
          store_piece(w, G, reinterpret_cast<float*>(ring), R::kPieceRow, ml_s[1][warp]);
        } else if (k0 > 0) {
          if (lane == 0) owner_s[0][warp] = unit;
          store_piece(w, G, closing, D, ml_s[0][warp]);
        } else {
          store_unit(w, G, p.out + static_cast<int64_t>(unit) * G * D);
        }
      }
      if (last) break;
    }
  }
  __syncthreads();
  int part_of[2] = {-1, -1};                         // units of the block's parts

  // The block's chains: pieces that go on, up to one that closes the unit or to the block's end; before
  // them a piece at the block's start that only closes (w = -1).
  for (int w = -1; w < Ring<D>::kWarps;) {
    const bool lone = w < 0;
    const int begin = max(w, 0), unit = owner_s[!lone][begin];
    if (unit < 0) {
      ++w;
      continue;
    }
    int end = begin;                                 // pieces begin .. end - 1 go on
    if (!lone)
      do ++end;
      while (end < Ring<D>::kWarps && owner_s[1][end] >= 0 && owner_s[0][end] < 0);
    const bool closed = end < Ring<D>::kWarps && owner_s[0][end] >= 0;
    const int slot = !lone && first_s[begin];
    const bool whole = closed && slot;
    const int64_t part = (blockIdx.x * 2 + slot) * kMaxGroup;
    add_chain<D>(reinterpret_cast<const float*>(smem + begin * R::kWarp), R::kWarp / 4, end - begin,
                 closed ? p.piece + static_cast<int64_t>(blockIdx.x * Ring<D>::kWarps + end) * kMaxGroup * D : nullptr,
                 ml_s[1][begin][0], closed ? ml_s[0][end][0] : nullptr, G, whole,
                 whole ? p.out + static_cast<int64_t>(unit) * G * D : p.part_acc + part * D,
                 p.part_ml + part * 2);
    if (!whole) part_of[slot] = unit;
    w = lone ? 0 : end;
  }
  if (threadIdx.x == 0) {
    p.goes_on[blockIdx.x] = part_of[0];
    p.begins[blockIdx.x] = part_of[1];
  }
  // units that see nothing
  for (int e = blockIdx.x; e < elems; e += gridDim.x) {
    const int b = p.sel_ids ? e / p.num_kv_heads : e;
    if (load_unit(p, b, p.sel_ids ? e - b * p.num_kv_heads : 0, false).tiles) continue;
    float* row = p.out + static_cast<int64_t>(e) * heads * G * D;
    for (int i = threadIdx.x; i < heads * G * D; i += Ring<D>::kThreads) row[i] = 0.f;
  }
}

// One block per (block of the first launch, query head of a group): joins the unit that begins there and
// ends elsewhere, if there is one: a warp takes every eighth part, eight of them at a time.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) q8_join_kernel(Q8AttendParams p) {
  constexpr int W = D / 32;                          // dimensions of a lane
  __shared__ float acc_s[kJoinWarps][D];
  __shared__ float ml_s[kJoinWarps][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = p.num_q_heads / p.num_kv_heads;
  const int block = blockIdx.x / G, head = blockIdx.x % G;
  grid_dependency_wait();
  const int blocks = gridDim.x / G;
  const int unit = p.begins[block];
  // the unit's parts: of this block and of those after it in which it goes on
  int count = 1;
  int after[kJoinRounds];
#pragma unroll
  for (int i = 0; i < kJoinRounds; ++i) {
    const int k = block + 1 + 32 * i + lane;
    after[i] = k < blocks ? p.goes_on[k] : -1;
  }
  if (unit < 0) return;
#pragma unroll
  for (int i = 0; i < kJoinRounds; ++i) {
    const unsigned miss = __ballot_sync(0xffffffffu, after[i] != unit);
    count += miss ? __ffs(miss) - 1 : 32;
    if (miss) break;
  }
  float sum[W] = {}, top = kNoScore, z = 0.f;
  constexpr int kAhead = 8;
  for (int k0 = warp; k0 < count; k0 += kAhead * kJoinWarps) {
    float x[kAhead][W];
    float2 ml[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = k0 + i * kJoinWarps;
      if (k < count) {
        // the first part is the second slot of its block, the others are the first slots of theirs
        const int64_t part = static_cast<int64_t>(2 * (block + k) + (k == 0)) * kMaxGroup + head;
        const float* row = p.part_acc + part * D + lane * W;
        if constexpr (W == 4) {
          const float4 v = *reinterpret_cast<const float4*>(row);
          x[i][0] = v.x, x[i][1] = v.y, x[i][W - 2] = v.z, x[i][W - 1] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(row);
          x[i][0] = v.x, x[i][1] = v.y;
        }
        ml[i] = *reinterpret_cast<const float2*>(p.part_ml + part * 2);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (k0 + i * kJoinWarps < count) add_part(sum, top, z, x[i], ml[i].x, ml[i].y);
  }
#pragma unroll
  for (int e = 0; e < W; ++e) acc_s[warp][lane * W + e] = sum[e];
  if (lane == 0) {
    ml_s[warp][0] = top;
    ml_s[warp][1] = z;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float all[1] = {0.f}, best = kNoScore, l = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) {
      const float x[1] = {acc_s[i][threadIdx.x]};
      add_part(all, best, l, x, ml_s[i][0], ml_s[i][1]);
    }
    p.out[(static_cast<int64_t>(unit) * G + head) * D + threadIdx.x] = l == 0.f ? 0.f : all[0] / l;
  }
}

template <int NQ, int C, int D>
cudaError_t launch_typed(const Q8AttendParams& p, int blocks, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  auto* kernel = q8_attend_kernel<NQ, C, D>;
  cudaError_t e = ensure_dynamic_smem(kernel, Ring<D>::kBytes, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(Ring<D>::kThreads);
  cfg.dynamicSmemBytes = Ring<D>::kBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kernel, p)) != cudaSuccess) return e;
  cfg.gridDim = dim3(blocks * (p.num_q_heads / p.num_kv_heads));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, q8_join_kernel<D>, p);
}

template <int NQ, int C>
cudaError_t launch_code(const Q8AttendParams& p, int d, int blocks, cudaStream_t stream) {
  return d == 128 ? launch_typed<NQ, C, 128>(p, blocks, stream)
                  : launch_typed<NQ, C, 64>(p, blocks, stream);
}

}  // namespace

int q8_attend_warps(int head_dim) { return head_dim == 128 ? Ring<128>::kWarps : Ring<64>::kWarps; }
int q8_attend_most_blocks() { return 32 * kJoinRounds; }

bool q8_attend_fits(int batch, int num_kv_heads, int team_size, int teams) {
  const int64_t unit = static_cast<int64_t>(teams) * (team_size / kTile) + kOpen;
  return static_cast<int64_t>(batch) * num_kv_heads <= kMostPlaces / unit;
}

cudaError_t launch_q8_attend(const Q8AttendParams& p, int head_dim, bool bf16, int code, int sms,
                             cudaStream_t stream) {
  if (code == kCodeI8)
    return bf16 ? launch_code<1, kCodeI8>(p, head_dim, sms, stream)
                : launch_code<2, kCodeI8>(p, head_dim, sms, stream);
  return bf16 ? launch_code<1, kCodeE4M3>(p, head_dim, sms, stream)
              : launch_code<2, kCodeE4M3>(p, head_dim, sms, stream);
}

}  // namespace santa
