// append.cuh — what the append kernels share: 16-byte pieces of a row, the pairs of a rotation, and
// the checked geometry of a sequence's chunk.
#pragma once

#include "kernels.h"

namespace santa {

constexpr int kAppendThreads = 256;
constexpr int kHeadsPerUnit = 4;   // query heads that share one load of cosines and sines

template <bool BF16>
struct Piece {
  static constexpr int kVec = BF16 ? 8 : 4;   // elements per 16 bytes
};

template <bool BF16>
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[Piece<BF16>::kVec]) {
  if constexpr (BF16) {
    x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
    x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
  } else {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
}
// The two pieces of a row that pair `pr` (0 .. pieces/2 - 1) stands for.  Rotation by halves:
// pieces j and j + R/2 of the rotated part, then the rest in twos; otherwise neighbours.
template <bool BF16>
__device__ __forceinline__ void pair_pieces(int pr, int rope_dim, bool interleaved, int* a,
                                            int* b) {
  const int half = interleaved ? 0 : rope_dim / (2 * Piece<BF16>::kVec);
  if (pr < half) {
    *a = pr;
    *b = pr + half;
  } else {
    *a = 2 * half + 2 * (pr - half);
    *b = *a + 1;
  }
}

// x c - y s and y c + x s with every product and sum rounded to fp32 (no contraction: the
// stored bits are then those of the formula as any fp32 program evaluates it)
__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
  const float nx = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = nx;
}

// Checked geometry of sequence b's chunk; false (and the status bit) if it must be skipped.
struct Chunk {
  int64_t first;   // its first token row
  int64_t n;       // new tokens
  int64_t len;     // cached tokens before
};
__device__ __forceinline__ bool load_chunk(const AppendChunkParams& p, int b, Chunk* c) {
  const int64_t c0 = p.cu_q[b], c1 = p.cu_q[b + 1];
  c->first = c0;
  c->n = c1 - c0;
  c->len = p.seq_lens[b];
  const int64_t cap = static_cast<int64_t>(p.max_teams) * p.team_size;
  const int64_t top = p.rope_dim && p.rope_positions < cap ? p.rope_positions : cap;
  return c0 >= 0 && c1 >= c0 && c1 <= p.num_tokens && c->len >= 0 &&
         (c->n == 0 ? c->len <= cap : c->len + c->n <= top);
}

// Blocks of page items: slots floor(cu_q[b] / T) + 2 b of every sequence, one per KV head.
inline int64_t append_page_blocks(int64_t num_tokens, int batch, int num_kv_heads, int team_size) {
  return (num_tokens / team_size + 2 * static_cast<int64_t>(batch)) * num_kv_heads;
}

}  // namespace santa
