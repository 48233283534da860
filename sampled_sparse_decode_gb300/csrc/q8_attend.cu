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
// Work.  The tiles (32 tokens) of all units (sequence, KV head) lie on one line, which the blocks
// share evenly, whatever the lengths of the batch are; the lengths are read on the device.  A block's
// warps take the tiles of its part in turn, each through a ring of its own in shared memory
// (asynchronous 16-byte copies, two tiles ahead of the one in use, no barrier among warps), and merge
// their results at the end of each unit's part.  A unit that lies within one block is finished there;
// the others' partial results are joined by a second launch in the order of the line.
//
// A tile.  Codes become fp16 exactly (int8 by the bits of 1024 + code, e4m3 by conversion) and go to
// the matrix units as the A operand of m16n8k16, tokens x dimensions for the scores and dimensions x
// tokens for the output, so that the group's up to 8 query heads are the n = 8 columns and a warp
// needs no other padding.  Which dimension stands at which k is free as long as both operands agree:
// a lane reads 16 bytes of one row and has the operands of four products.  Rows are placed so that
// both kinds of read are free of bank conflicts.
//   - q enters as fp16 pieces (one for bf16, two for fp32) of q 2^-e, e the exponent of the head's
//     largest element: fp16's range holds everything down to 2^-24 of it.
//   - The weights enter the second product as two fp16 pieces (22 bits; one would leave 2^-12 of
//     error in an fp32 result) of p_j vs_j over a power of two near the largest p vs so far: the scales of
//     values may lie any powers of two apart.
//   - The reference of the exponentials is raised only when a score passes it by 8 (powers of two),
//     which is seldom after a few tiles, so a tile has no reduction among lanes.
//   - The matrix units cut what they add; each tile's products start from zero and are added to the
//     running sums in fp32 with rounding.
#include <algorithm>

#include "kernels.h"
#include "q8.cuh"

namespace santa {

namespace {

constexpr int kTile = 32;                  // tokens of a tile
constexpr int kQ8Warps = 8;
constexpr int kQ8Threads = kQ8Warps * 32;
constexpr int kStages = 3;                 // tiles of a warp's ring
constexpr int kMinShare = kQ8Warps;        // tiles of a block's part: at least one for each warp
constexpr int kScanRounds = 8;             // 32 sequences or units each that a warp reads by itself
constexpr int kMergeDims = 64;             // dimensions that one merging pass takes
constexpr int kMergeRow = kMergeDims + 4;
constexpr float kNoScore = -1e38f;         // a reference before the first score
constexpr float kSlack = 8.f;              // how far a score may pass the reference (base 2)
constexpr float kTopWeight = 256.f;        // the same for a weight

template <int D>
struct Ring {
  static constexpr int kCodes = kTile * D;                     // bytes of a tile's keys or values
  static constexpr int kStage = 2 * kCodes + 2 * kTile * 4;    // keys, values, scales
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kMerge = kQ8Warps * kMaxGroup * kMergeRow * 4;
  static constexpr int kBytes = kQ8Warps * kWarp + kMerge;
};

// Byte of 16-byte piece `chunk` of row r in a tile's block of rows.  Scores are read by 8 lanes from
// pieces c .. c + 3 of rows 2j and 2j + 1, values from pieces 2j and 2j + 1 (d = 128; the halves of a
// piece for d = 64) of four rows two apart: either way the 8 pieces lie in 8 different banks' groups.
template <int D>
__device__ __forceinline__ int piece_at(int r, int chunk) {
  if constexpr (D == 128) {
    return r * 128 + ((chunk ^ (((r >> 2 ^ r) & 1) << 2 | (r & 2))) << 4);
  } else {
    const int half = (r ^ r >> 1) & 1;
    return (r >> 1) * 128 + (half << 6) + ((chunk ^ ((r >> 2 & 1) << 1)) << 4);
  }
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

// The leading 11 bits of x (fp16 holds them from 2^-14 on; below, it rounds at 2^-25).
__device__ __forceinline__ float cut_f16(float x) {
  return __uint_as_float(__float_as_uint(x) & 0xffffe000u);
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

// ---------------------------------------------------------------- the line of tiles

// A unit's tokens: positions lo .. len - 1 (dense), or `count` listed teams; `tiles` on the line.
struct Unit {
  int len, lo;         // at most 2^14 pages of 2^7 tokens
  int count;
  int64_t tiles;
};
// Reads sequence b (dense) or unit (b, h) (listed); what is out of range is judged here and told if
// `tell`.
__device__ __forceinline__ Unit load_unit(const Q8AttendParams& p, int b, int h, bool tell) {
  Unit u;
  u.len = p.seq_lens[b];
  u.count = 0;
  if (u.len < 0 || u.len > p.max_teams * p.team_size) {
    if (tell) set_status(p.status, SANTA_DEV_BAD_SEQLEN);
    u.len = 0;
  }
  u.lo = p.window > 0 && u.len > p.window ? u.len - p.window : 0;
  if (p.sel_ids) {
    const int count = p.sel_count[static_cast<int64_t>(b) * p.num_kv_heads + h];
    u.count = min(max(count, 0), p.num_draws);
    if (count != u.count && tell) set_status(p.status, SANTA_DEV_BAD_SEL);
    if (u.len == 0) u.count = 0;
    u.tiles = static_cast<int64_t>(u.count) * (p.team_size / kTile);
  } else {
    u.tiles = (u.len + kTile - 1) / kTile - u.lo / kTile;
  }
  return u;
}

// A place on the line: unit (b, h), whose tiles start at `base`.
struct Walk {
  int b, h;
  int64_t base;
  Unit u;
};
__device__ __forceinline__ void next_unit(const Q8AttendParams& p, Walk& w) {
  w.base += w.u.tiles;
  if (w.b == p.batch - 1 && w.h == p.num_kv_heads - 1) {
    // not reached while lengths and lists stay as they are; if not, the walk ends here
    w.u = Unit{0, 0, 0, INT64_MAX / 2};
    return;
  }
  const bool wrap = ++w.h == p.num_kv_heads;
  if (wrap) {
    w.h = 0;
    ++w.b;
  }
  if (wrap || p.sel_ids) w.u = load_unit(p, w.b, w.h, false);
}

__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int64_t before = 0;
#pragma unroll
  for (int w = 0; w < kQ8Warps; ++w)
    if (w < warp) before += warp_sums[w];
  return v + before;
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
  static constexpr int kSteps = D / 16;              // k steps of a score
  static constexpr int kOut = D / 16;                // 16-dimension tiles of the output
  uint32_t q[NQ][kSteps][2];
  float acc[kOut][4];
  float ref[2];              // of heads 2t and 2t + 1: reference of the exponentials
  float sum[2];              // this lane's share of the sum of weights
  float big[2], inv[2];      // largest |p vs| (at least), and the power of two that scales weights
  float qs[2];               // score of a unit product, base 2 (or over the cap)
};

// Copies tile `t` of the line into a stage and returns what the consumer must know of it: the range of
// its tokens that are seen and the bias.
template <int D>
__device__ __forceinline__ void issue_tile(const Q8AttendParams& p, const Walk& w, int64_t t,
                                           PageCache& pc, uint8_t* stage, int2* note) {
  const int lane = threadIdx.x & 31;
  const int T = p.team_size, per = T == 128 ? 2 : 1;  // log2 of a page's tiles
  // tile of the unit, or of the sequence (at most 2^16 of them); then slot or team, and row in it
  const int i = static_cast<int>(t - w.base) + (p.sel_ids ? 0 : w.u.lo / kTile);
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
        pc.team = team;
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

// The group's queries as B operands: k index of step (c, w) are bytes 16 (t + 4 c) + 4 w + ... of a
// row, t = lane % 4 (d = 64: c = 0 only).
template <int NQ, int C, int D>
__device__ void load_queries(const Q8AttendParams& p, int b, int h, Warp<NQ, C, D>& w) {
  const int lane = threadIdx.x & 31, head = lane >> 2, t = lane & 3;
  const int G = p.num_q_heads / p.num_kv_heads;
  const int64_t at = (static_cast<int64_t>(b) * p.num_q_heads + h * G + head) * D;
  float x[D / 4];
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int64_t e = at + 16 * (t + 4 * c) + i;
      float* y = x + 16 * c + i;
      if (head >= G) {
        y[0] = y[1] = y[2] = y[3] = 0.f;
      } else if constexpr (NQ == 1) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + e);
        y[0] = bf16_lo(v.x), y[1] = bf16_hi(v.x), y[2] = bf16_lo(v.y), y[3] = bf16_hi(v.y);
      } else {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + e);
        y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < D / 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // 2^-e and 2^e as exponent fields; zeros and queries near fp32's ends keep a factor inside its range
  const uint32_t e = min(max(top >> 23, 16u), 253u);
  const float down = __uint_as_float((254u - e) << 23), up = __uint_as_float(e << 23);
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = x[4 * s + 2 * i] * down, c = x[4 * s + 2 * i + 1] * down;
      w.q[0][s][i] = pack_f16(a, c);
      if constexpr (NQ == 2) {
        const float2 got = f16x2_to_f32(w.q[0][s][i]);
        w.q[NQ - 1][s][i] = pack_f16(a - got.x, c - got.y);
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
    if (big > 0.f) inv = __uint_as_float((254u - min(max(__float_as_uint(big) >> 23, 1u), 253u)) << 23);
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
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const float* scales = reinterpret_cast<const float*>(stage + 2 * kTile * D);
  const int n0 = note.x & 0xffff, n1 = note.x >> 16;
  if (n1 == 0) return;
  float x[8], ks[4], vs[4];                          // token 8 k + g; score 2 k + i: head 2 t + i
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      const uint4 a = *reinterpret_cast<const uint4*>(stage + piece_at<D>(16 * m + g, t + 4 * h));
      const uint4 b = *reinterpret_cast<const uint4*>(stage + piece_at<D>(16 * m + 8 + g, t + 4 * h));
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t f[4];
        pairs_to_f16<C>(aw[k], f[0], f[2]);
        pairs_to_f16<C>(bw[k], f[1], f[3]);
#pragma unroll
        for (int n = 0; n < NQ; ++n) mma_f16_16816(c, f, w.q[n][4 * h + k][0], w.q[n][4 * h + k][1]);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      ks[2 * m + r] = scales[16 * m + 8 * r + g];
      vs[2 * m + r] = scales[kTile + 16 * m + 8 * r + g];
      x[4 * m + 2 * r] = c[2 * r];
      x[4 * m + 2 * r + 1] = c[2 * r + 1];
    }
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
    // the first piece is cut, not rounded: what it leaves out is then exact in fp32 at once
    const float a = cut_f16(pw[2 * k]), b = cut_f16(pw[2 * k + 1]);
    hi[k] = pack_f16(a, b);
    lo[k] = pack_f16(pw[2 * k] - a, pw[2 * k + 1] - b);
    hi[k] = movmatrix_trans(hi[k]);
    lo[k] = movmatrix_trans(lo[k]);
  }
  // values: 16 tokens at a time; a lane has D / 8 dimensions of four tokens
  constexpr int kWords = D / 32;
  uint32_t v[2][4][kWords];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int tok = 16 * m + 8 * (r >> 1) + 2 * t + (r & 1);
      const uint8_t* at = stage + kTile * D;
      if constexpr (D == 128) {
        const uint4 a = *reinterpret_cast<const uint4*>(at + piece_at<D>(tok, g));
        v[m][r][0] = a.x, v[m][r][1] = a.y, v[m][r][kWords - 2] = a.z, v[m][r][kWords - 1] = a.w;
      } else {
        const uint2 a = *reinterpret_cast<const uint2*>(at + piece_at<D>(tok, g >> 1) + (g & 1) * 8);
        v[m][r][0] = a.x, v[m][r][1] = a.y;
      }
    }
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    float c[2][4] = {};
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint32_t f[2][4];                              // dimensions (4k, 4k + 1) and (4k + 2, 4k + 3)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t a = v[m][2 * r][k], b = v[m][2 * r + 1][k];
        pairs_to_f16<C>(__byte_perm(a, b, 0x5140), f[0][2 * r], f[0][2 * r + 1]);
        pairs_to_f16<C>(__byte_perm(a, b, 0x7362), f[1][2 * r], f[1][2 * r + 1]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mma_f16_16816(c[j], f[j], hi[2 * m], hi[2 * m + 1]);
        mma_f16_16816(c[j], f[j], lo[2 * m], lo[2 * m + 1]);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) w.acc[2 * k + j][i] += c[j][i];
  }
}

template <int NQ, int C, int D>
__global__ void __launch_bounds__(kQ8Threads, 1) q8_attend_kernel(Q8AttendParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t sums[2][kQ8Warps];
  __shared__ int64_t start_s[2];                     // element of the line's start, its first tile
  __shared__ int2 notes[kQ8Warps][kStages];
  __shared__ float ml[kQ8Warps][kMaxGroup][2];
  using R = Ring<D>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = p.num_q_heads / p.num_kv_heads;
  grid_dependency_wait();
  grid_launch_dependents();

  // the length of the line, and where this block's part of it starts: by sequences (dense) or units
  const int64_t elems = static_cast<int64_t>(p.batch) * (p.sel_ids ? p.num_kv_heads : 1);
  const int heads = p.sel_ids ? 1 : p.num_kv_heads;
  auto tiles_of = [&](int64_t e, bool tell) -> int64_t {
    if (e >= elems) return 0;
    const int b = static_cast<int>(p.sel_ids ? e / p.num_kv_heads : e);
    return load_unit(p, b, static_cast<int>(e - static_cast<int64_t>(b) * p.num_kv_heads), tell).tiles *
           heads;
  };
  const bool tell = blockIdx.x == 0;
  int64_t total = 0, share, c0, elem = 0, elem_base = 0;
  auto split = [&]() {
    share = max((total + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(kMinShare));
    c0 = blockIdx.x * share;
  };
  if (elems <= 32 * kScanRounds) {
    // every warp for itself, without a barrier
    int64_t v[kScanRounds], upto[kScanRounds];
#pragma unroll
    for (int i = 0; i < kScanRounds; ++i) v[i] = tiles_of(32 * i + lane, tell && warp == 0);
#pragma unroll
    for (int i = 0; i < kScanRounds; ++i) {
      upto[i] = v[i];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, upto[i], o);
        if (lane >= o) upto[i] += up;
      }
      upto[i] += total;
      total = __shfl_sync(0xffffffffu, upto[i], 31);
    }
    split();
#pragma unroll
    for (int i = 0; i < kScanRounds; ++i) {
      const unsigned hit = __ballot_sync(0xffffffffu, upto[i] > c0 && upto[i] - v[i] <= c0);
      if (hit) {
        elem = 32 * i + __ffs(hit) - 1;
        elem_base = __shfl_sync(0xffffffffu, upto[i] - v[i], __ffs(hit) - 1);
      }
    }
  } else {
    for (int64_t e0 = 0; e0 < elems; e0 += kQ8Threads) {
      const int64_t upto =
          total + block_scan(tiles_of(e0 + threadIdx.x, tell), sums[(e0 / kQ8Threads) & 1]);
      if (threadIdx.x == kQ8Threads - 1) start_s[0] = upto;
      __syncthreads();
      total = start_s[0];
      __syncthreads();
    }
    split();
    int64_t before = 0;
    for (int64_t e0 = 0; e0 < elems && c0 < total; e0 += kQ8Threads) {
      const int64_t mine = tiles_of(e0 + threadIdx.x, false);
      const int64_t upto = before + block_scan(mine, sums[(e0 / kQ8Threads) & 1]);
      if (upto > c0 && upto - mine <= c0) {
        start_s[0] = e0 + threadIdx.x;
        start_s[1] = upto - mine;
      }
      if (__syncthreads_or(upto > c0)) break;
      if (threadIdx.x == kQ8Threads - 1) sums[0][0] = upto;
      __syncthreads();
      before = sums[0][0];
      __syncthreads();
    }
    __syncthreads();
    elem = start_s[0];
    elem_base = start_s[1];
  }
  const int64_t c1 = min(c0 + share, total);
  int64_t split_unit = -1;                           // a unit that starts here and ends elsewhere
  int split_parts = 0;
  // units that see nothing
  auto zero_units = [&]() {
    for (int64_t e = blockIdx.x; e < elems; e += gridDim.x) {
      if (tiles_of(e, false)) continue;
      float* row = p.out + e * heads * G * D;
      for (int i = threadIdx.x; i < heads * G * D; i += kQ8Threads) row[i] = 0.f;
    }
  };
  if (c0 >= c1) {
    zero_units();
    if (threadIdx.x == 0) p.split_unit[blockIdx.x] = -1;
    return;
  }
  Walk use;
  use.b = static_cast<int>(p.sel_ids ? elem / p.num_kv_heads : elem);
  use.h = static_cast<int>(p.sel_ids ? elem % p.num_kv_heads : 0);
  use.base = elem_base;
  use.u = load_unit(p, use.b, use.h, false);
  while (use.base + use.u.tiles <= c0) next_unit(p, use);
  Walk ask = use;

  uint8_t* ring = smem + warp * R::kWarp;
  float* merge = reinterpret_cast<float*>(smem + kQ8Warps * R::kWarp);
  PageCache pc;
  pc.b = -1;
  int64_t next = c0 + warp;                          // the next tile to ask for
  int put = 0, get = 0;
  auto ask_next = [&]() {
    if (next < c1) {
      while (ask.base + ask.u.tiles <= next) next_unit(p, ask);
      issue_tile<D>(p, ask, next, pc, ring + put * R::kStage, &notes[warp][put]);
      next += kQ8Warps;
    }
    cp_async_commit();
    put = put + 1 == kStages ? 0 : put + 1;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) ask_next();
  zero_units();

  Warp<NQ, C, D> w;
  int64_t at = c0 + warp;
  for (;;) {
    const int64_t end = min(c1, use.base + use.u.tiles);
    load_queries(p, use.b, use.h, w);
    for (; at < end; at += kQ8Warps) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      ask_next();
      attend_tile(p, w, ring + get * R::kStage, notes[warp][get]);
      get = get + 1 == kStages ? 0 : get + 1;
      __syncwarp();
    }
    // merge the warps' results of this unit
    const bool whole = use.base >= c0 && use.base + use.u.tiles <= c1;
    const int slot = use.base < c0 ? 0 : 1;          // goes on from the block before, or starts here
    if (!whole && slot == 1) {
      split_unit = static_cast<int64_t>(use.b) * p.num_kv_heads + use.h;
      split_parts = static_cast<int>((use.base + use.u.tiles - 1) / share) - blockIdx.x + 1;
    }
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float s = w.sum[i];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (g == 0) {
        ml[warp][2 * t + i][0] = w.ref[i];
        ml[warp][2 * t + i][1] = s;
      }
      const float back = 1.f / w.inv[i];
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        w.acc[j][i] *= back;
        w.acc[j][2 + i] *= back;
      }
    }
    // dimension D/8 g + 2j + r of the lane's D/8; a pass takes kLane of them from every lane
    constexpr int kLane = kMergeDims / 8;
#pragma unroll
    for (int pass = 0; pass < D / kMergeDims; ++pass) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* row = merge + (warp * kMaxGroup + 2 * t + i) * kMergeRow + g * kLane;
#pragma unroll
        for (int j = 0; j < kLane / 4; ++j) {
          const int o = pass * kLane / 2 + 2 * j;
          *reinterpret_cast<float4*>(row + 4 * j) =
              make_float4(w.acc[o][i], w.acc[o][2 + i], w.acc[o + 1][i], w.acc[o + 1][2 + i]);
        }
      }
      __syncthreads();
      for (int e = threadIdx.x; e < G * kMergeDims; e += kQ8Threads) {
        const int head = e / kMergeDims, col = e % kMergeDims;
        const int dim = col / kLane * (D / 8) + kLane * pass + col % kLane;
        float top = -INFINITY, sum = 0.f, z = 0.f;
#pragma unroll
        for (int i = 0; i < kQ8Warps; ++i) top = fmaxf(top, ml[i][head][0]);
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int i = 0; i < kQ8Warps; ++i) {
          const float keep = ex2_approx(ml[i][head][0] - ref);
          sum += merge[(i * kMaxGroup + head) * kMergeRow + col] * keep;
          z += ml[i][head][1] * keep;
        }
        if (whole) {
          p.out[(static_cast<int64_t>(use.b) * p.num_q_heads + use.h * G + head) * D + dim] =
              z == 0.f ? 0.f : sum / z;
        } else {
          const int64_t part = static_cast<int64_t>(blockIdx.x * 2 + slot) * kMaxGroup + head;
          p.part_acc[part * D + dim] = sum;
          if (dim == 0) {
            p.part_ml[part * 2] = top;
            p.part_ml[part * 2 + 1] = z;
          }
        }
      }
      __syncthreads();
    }
    if (end >= c1) break;
    do next_unit(p, use);
    while (use.u.tiles == 0);
  }
  if (threadIdx.x == 0) {
    p.split_unit[blockIdx.x] = split_unit;
    p.split_parts[blockIdx.x] = split_parts;
  }
}

// One block per (block of the first launch, query head of a group): joins the unit that starts there and
// ends elsewhere, if there is one, by adding its partial results in the order of the line, a warp each
// in turn.
template <int D>
__global__ void __launch_bounds__(kQ8Threads) q8_join_kernel(Q8AttendParams p) {
  constexpr int W = D / 32;                          // dimensions of a lane
  __shared__ float acc_s[kQ8Warps][D];
  __shared__ float ml_s[kQ8Warps][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = p.num_q_heads / p.num_kv_heads;
  const int block = blockIdx.x / G, head = blockIdx.x % G;
  grid_dependency_wait();
  const int64_t unit = p.split_unit[block];
  if (unit < 0) return;
  const int count = p.split_parts[block];
  float* out = p.out + (unit * G + head) * D;
  float m = -INFINITY, l = 0.f, acc[W];
#pragma unroll
  for (int e = 0; e < W; ++e) acc[e] = 0.f;
  for (int k = warp; k < count; k += kQ8Warps) {
    // the first part is the second slot of its block, the others the first slots of theirs
    const int64_t part = static_cast<int64_t>(2 * (block + k) + (k == 0)) * kMaxGroup + head;
    const float pm = p.part_ml[part * 2], pl = p.part_ml[part * 2 + 1];
    float x[W];
#pragma unroll
    for (int e = 0; e < W; ++e) x[e] = p.part_acc[part * D + lane * W + e];
    const float top = fmaxf(m, pm), ref = top == -INFINITY ? 0.f : top;
    const float keep = ex2_approx(m - ref), add = ex2_approx(pm - ref);
    m = top;
    l = l * keep + pl * add;
#pragma unroll
    for (int e = 0; e < W; ++e) acc[e] = acc[e] * keep + x[e] * add;
  }
#pragma unroll
  for (int e = 0; e < W; ++e) acc_s[warp][lane * W + e] = acc[e];
  if (lane == 0) {
    ml_s[warp][0] = m;
    ml_s[warp][1] = l;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float top = -INFINITY, sum = 0.f, z = 0.f;
#pragma unroll
    for (int i = 0; i < kQ8Warps; ++i) top = fmaxf(top, ml_s[i][0]);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int i = 0; i < kQ8Warps; ++i) {
      const float keep = ex2_approx(ml_s[i][0] - ref);
      sum += acc_s[i][threadIdx.x] * keep;
      z += ml_s[i][1] * keep;
    }
    out[threadIdx.x] = z == 0.f ? 0.f : sum / z;
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
  cfg.blockDim = dim3(kQ8Threads);
  cfg.dynamicSmemBytes = Ring<D>::kBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kernel, p)) != cudaSuccess) return e;
  cfg.gridDim = dim3(blocks * (p.num_q_heads / p.num_kv_heads));
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, q8_join_kernel<D>, p);
}

template <int NQ, int C>
cudaError_t launch_code(const Q8AttendParams& p, int d, int blocks, cudaStream_t stream) {
  return d == 128 ? launch_typed<NQ, C, 128>(p, blocks, stream)
                  : launch_typed<NQ, C, 64>(p, blocks, stream);
}

}  // namespace

cudaError_t launch_q8_attend(const Q8AttendParams& p, int head_dim, bool bf16, int code, int sms,
                             cudaStream_t stream) {
  if (code == kCodeI8)
    return bf16 ? launch_code<1, kCodeI8>(p, head_dim, sms, stream)
                : launch_code<2, kCodeI8>(p, head_dim, sms, stream);
  return bf16 ? launch_code<1, kCodeE4M3>(p, head_dim, sms, stream)
              : launch_code<2, kCodeE4M3>(p, head_dim, sms, stream);
}

}  // namespace santa
