// chunk_simt.cu — causal attention of a chunk of new tokens over the paged cache in plain fp32
// arithmetic (fp32 caches).
//
// A KV head's G query heads share its keys, so the rows of a tile are (token, head) pairs: row
// r of a sequence's n * G rows is token r / G, head r % G.  A block takes 64 rows and the keys
// they see, with the running maximum and sum of an online softmax (base 2), in one of two ways:
//   many rows  keys in steps of 64 through shared memory (two blocks per SM, one copies while the
//              other computes): S = Q K^T (4 x 4 scores per thread), P = 2^(S - m), O = 2^(m_old -
//              m) O + P V (4 x d/16).  Bound by fp32 FMAs and their operands' shared loads (8 FMAs
//              per 16-byte load in the scores; 8 in the product with V at d = 64, 10.7 at 128).
//   few rows   (8 at a time, so the single token of any group at once): a warp takes 32 keys at a
//              time, one per lane for the scores, all of them by columns for the product with V;
//              the warps' results are joined at the end.  With 64-row tiles 15 of 16 threads
//              would idle.
// The keys of a tile are split over several blocks when there are few tiles (no split below 4
// steps); a second launch joins their partial (m, l, O) in order.  Tiles are found from cu_q
// through slots, as in append_chunk.cu: sequence b owns floor(cu[b] G / 64) + b onward, at least
// ceil(n G / 64).
//
// Masked scores never enter: P is 0 there, and in a step that holds a masked pair (the causal
// border) the product with V is selected away too, because 0 * V is not 0 when V is not finite.
//
// Measured on GB300 in a stream of calls on changing inputs: prompts of 1000 tokens on 4000 and 800
// on 100, 8 heads of 128, 602 us, 33 TFLOP/s; a batch of 1, 513, 64 and 1 tokens, 8 / 2 heads of 64,
// 33 us (74 us before the few-rows way and the splits by length); one token of 8 sequences on 8000,
// 32 / 8 heads of 128, 183 us, 2.9 TB/s.
#include <algorithm>

#include "kernels.h"

namespace santa {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;        // query rows per tile
constexpr int kKeys = 64;        // keys per step (divides both page sizes)
constexpr int kMinSpan = 4;      // steps below which a tile is not split
constexpr int kFew = 8;          // rows that the few-rows way takes at a time
// Tiles of more rows than these go the other way: with two KV heads of 128 on 12505 tokens, 16 rows
// take 49 us here (two passes) and 54 us there, 24 rows 65 and 54 us.
constexpr int kFewMost = 16;
constexpr int kWarps = kThreads / 32;

template <int D>
struct SimtSmem {
  float q[kRows][D + 4];         // +4: rows 16 apart would share banks
  union {
    float k[kKeys][D + 4];
    float p[kRows][kKeys + 4];   // once the scores are formed
  };
  float v[kKeys][D];
};
template <int D>
struct FewSmem {
  float q[kFew][D];
  float p[kWarps][32][kFew];
  float m[kWarps][kFew], l[kWarps][kFew];
  union {
    float k[kWarps][32][D / 2 + 4];      // half of the warp's 32 key rows
    float o[kWarps][kFew][D];            // once the keys are done
  };
};

__device__ __forceinline__ float4 load4(const void* base, int64_t elem) {
  return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
}
__device__ __forceinline__ void store4(void* base, int64_t elem, float4 v) {
  *reinterpret_cast<float4*>(static_cast<float*>(base) + elem) = v;
}

struct Tile {
  int b;
  int64_t first, n, len;   // first token row, new tokens, cached tokens (with the chunk)
  int64_t row0;            // first of the sequence's n * G rows in this tile
  int64_t keys;            // cached tokens that some row of the tile sees
  int64_t steps;           // of 64 keys
  int splits;              // blocks that share them
};

__device__ __forceinline__ bool find_tile(const ChunkParams& p, int64_t slot, int G, int splits,
                                          Tile* t) {
  // s(b) = floor(cu[b] * G / 64) + b: the search multiplies through 64-bit values
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    bool below = lane == 0;
    if (lane > 0 && at < hi) {
      int64_t c = p.cu_q[at];
      c = c < 0 ? 0 : c > p.num_tokens ? p.num_tokens : c;
      below = c * G / kRows + at <= slot;
    }
    const unsigned m = __ballot_sync(0xffffffffu, below);
    lo += (31 - __clz(m)) * step;
    hi = min(hi, lo + step);
  }
  t->b = lo;
  const int64_t c0 = p.cu_q[lo], c1 = p.cu_q[lo + 1];
  t->first = c0;
  t->n = c1 - c0;
  t->len = p.seq_lens[lo];
  if (c0 < 0 || c1 < c0 || c1 > p.num_tokens ||
      (t->n > 0 &&
       (t->len < t->n || t->len > static_cast<int64_t>(p.max_teams) * p.team_size))) {
    if (threadIdx.x == 0) set_status(p.status, SANTA_DEV_BAD_SEQLEN);
    return false;
  }
  const int64_t j = slot - (c0 * G / kRows + lo);
  t->row0 = j * kRows;
  if (j < 0 || t->row0 >= t->n * G) return false;
  const int64_t last = min(t->row0 + kRows, t->n * G) - 1;
  t->keys = t->len - t->n + last / G + 1;
  t->steps = (t->keys + kKeys - 1) / kKeys;
  t->splits = static_cast<int>(
      min(static_cast<int64_t>(splits), (t->steps + kMinSpan - 1) / kMinSpan));
  return true;
}

// A row's result: the output, or the partial one of this split.  `cols` values from column c.
__device__ __forceinline__ void finish4(const ChunkParams& p, const Tile& t, int64_t tile,
                                        int split, int splits, int h, int G, int r, int D, int c,
                                        float4 o, float m, float l, bool first, float* part_acc,
                                        float* part_ml) {
  const int64_t row = t.row0 + r;
  if (t.splits == 1) {
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    store4(p.out, ((t.first + row / G) * p.num_q_heads + h * G + row % G) * D + c,
           make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  } else {
    const int64_t at = (tile * splits + split) * kRows + r;
    if (first) {
      part_ml[2 * at] = m;
      part_ml[2 * at + 1] = l;
    }
    *reinterpret_cast<float4*>(part_acc + at * D + c) = o;
  }
}

// The pool element of key `tok` (0 of its row); a page out of range is reported and read as 0.
__device__ __forceinline__ int64_t key_at(const ChunkParams& p, int b, int h, int64_t tok, int D,
                                          bool report) {
  int64_t page = p.page_table[static_cast<int64_t>(b) * p.max_teams + tok / p.team_size];
  if (page < 0 || page >= p.num_pages) {
    if (report) set_status(p.status, SANTA_DEV_BAD_PAGE);
    page = 0;
  }
  return ((page * p.num_kv_heads + h) * p.team_size + tok % p.team_size) * static_cast<int64_t>(D);
}

template <int D>
__device__ void few_rows(const ChunkParams& p, const Tile& t, FewSmem<D>& s, int G, int h,
                         int64_t tile, int split, int splits, int64_t s0, int64_t s1, int first,
                         float* part_acc, float* part_ml) {
  constexpr int kCols = D / 32;                 // columns of O per lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t row0 = t.row0 + first;          // of the (up to) 8 rows of this pass
  const int rows = static_cast<int>(min(static_cast<int64_t>(kFew), t.n * G - row0));
  for (int i = threadIdx.x; i < kFew * D; i += kThreads) {
    const int r = i / D;
    const int64_t row = row0 + r;
    s.q[r][i % D] =
        r < rows ? static_cast<const float*>(p.q)[((t.first + row / G) * p.num_q_heads + h * G +
                                                   row % G) * D + i % D]
                 : 0.f;
  }
  int64_t sees[kFew];
#pragma unroll
  for (int r = 0; r < kFew; ++r)
    sees[r] = r < rows ? t.len - t.n + (row0 + r) / G + 1 : 0;
  const int64_t all_see = t.len - t.n + row0 / G + 1;
  __syncthreads();
  float m[kFew], l[kFew], o[kFew][kCols];
#pragma unroll
  for (int r = 0; r < kFew; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[r][c] = 0.f;
  }
  const int64_t end = min(s1 * kKeys, t.keys);
  for (int64_t k0 = s0 * kKeys + warp * 32; k0 < end; k0 += kWarps * 32) {
    const int count = static_cast<int>(min(static_cast<int64_t>(32), end - k0));
    const int64_t base = key_at(p, t.b, h, k0, D, lane == 0);      // 32 keys share a page
    // scores: a lane per key.  The rows come through shared memory, half of their width at a time
    // (lanes reading their own rows from global memory touch 32 lines per load: 2.0 TB/s)
    constexpr int kPieces = D / 8;              // 16-byte pieces of half a row
    const float* k = static_cast<const float*>(p.k_pool) + base;
    float a[kFew];
#pragma unroll
    for (int r = 0; r < kFew; ++r) a[r] = 0.f;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int at = i * 32 + lane, row = at / kPieces, c = at % kPieces * 4;
        cp_async16(&s.k[warp][row][c], k + min(row, count - 1) * D + half * (D / 2) + c);
      }
      cp_async_wait_all();
      __syncwarp();
#pragma unroll 4
      for (int e = 0; e < D / 2; e += 4) {
        const float4 kv = *reinterpret_cast<const float4*>(&s.k[warp][lane][e]);
#pragma unroll
        for (int r = 0; r < kFew; ++r) {
          const float4 q = *reinterpret_cast<const float4*>(&s.q[r][half * (D / 2) + e]);
          a[r] = fmaf(q.x, kv.x, fmaf(q.y, kv.y, fmaf(q.z, kv.z, fmaf(q.w, kv.w, a[r]))));
        }
      }
    }
    float w[kFew];
#pragma unroll
    for (int r = 0; r < kFew; ++r) {
      const float x = lane < count && k0 + lane < sees[r] ? a[r] * p.scale_log2 : -INFINITY;
      const float mn = fmaxf(m[r], warp_max(x));
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float keep = exp2f(m[r] - ref);
      w[r] = exp2f(x - ref);
      l[r] = l[r] * keep + w[r];                // this lane's keys; summed over lanes at the end
      m[r] = mn;
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[r][c] *= keep;
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kFew; r += 4)
      *reinterpret_cast<float4*>(&s.p[warp][lane][r]) =
          make_float4(w[r], w[r + 1], w[r + 2], w[r + 3]);
    __syncwarp();
    const float* v = static_cast<const float*>(p.v_pool) + base + lane * kCols;
    const bool border = k0 + 32 > all_see;
#pragma unroll 8
    for (int j = 0; j < count; ++j) {
      float x[kCols];
#pragma unroll
      for (int c = 0; c < kCols; c += 2) {
        const float2 v2 = *reinterpret_cast<const float2*>(v + j * D + c);
        x[c] = v2.x;
        x[c + 1] = v2.y;
      }
#pragma unroll
      for (int r = 0; r < kFew; ++r) {
        const float pw = s.p[warp][j][r];
        if (!border || k0 + j < sees[r])
#pragma unroll
          for (int c = 0; c < kCols; ++c) o[r][c] = fmaf(pw, x[c], o[r][c]);
      }
    }
  }
  // the warps' results, joined in order
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kFew; ++r) {
    l[r] = warp_sum(l[r]);
    if (lane == 0) {
      s.m[warp][r] = m[r];
      s.l[warp][r] = l[r];
    }
#pragma unroll
    for (int c = 0; c < kCols; ++c) s.o[warp][r][lane * kCols + c] = o[r][c];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s.m[w][r]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(s.m[w][r] - ref);
      const float4 x = *reinterpret_cast<const float4*>(&s.o[w][r][c]);
      ll = fmaf(f, s.l[w][r], ll);
      acc.x = fmaf(f, x.x, acc.x);
      acc.y = fmaf(f, x.y, acc.y);
      acc.z = fmaf(f, x.z, acc.z);
      acc.w = fmaf(f, x.w, acc.w);
    }
    finish4(p, t, tile, split, splits, h, G, first + r, D, c, acc, mm, ll, c == 0, part_acc,
            part_ml);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) chunk_simt_kernel(ChunkParams p, int splits,
                                                                 float* part_acc,
                                                                 float* part_ml) {
  extern __shared__ __align__(16) unsigned char raw[];
  SimtSmem<D>& s = *reinterpret_cast<SimtSmem<D>*>(raw);
  constexpr int kCols = D / 64;                 // float4 columns of O per thread
  const int G = p.num_q_heads / p.num_kv_heads;
  const int h = blockIdx.y, split = blockIdx.z;
  grid_dependency_wait();
  if (blockIdx.x == 0 && h == 0 && split == 0)
    check_bounds(p.cu_q, p.batch, p.num_tokens, p.status);
  Tile t;
  if (!find_tile(p, blockIdx.x, G, splits, &t) || split >= t.splits) return;
  const int64_t tile = static_cast<int64_t>(blockIdx.x) * p.num_kv_heads + h;
  const int64_t per = (t.steps + t.splits - 1) / t.splits;
  const int64_t s0 = split * per, s1 = min(t.steps, s0 + per);
  if (t.n * G - t.row0 <= kFewMost) {
    for (int first = 0; first < t.n * G - t.row0; first += kFew) {
      if (first > 0) __syncthreads();
      few_rows<D>(p, t, *reinterpret_cast<FewSmem<D>*>(raw), G, h, tile, split, splits, s0, s1,
                  first, part_acc, part_ml);
    }
    return;
  }
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    const int64_t row = t.row0 + r;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < t.n * G)
      x = load4(p.q, ((t.first + row / G) * p.num_q_heads + h * G + row % G) * D + c);
    *reinterpret_cast<float4*>(&s.q[r][c]) = x;
  }
  // keys that row ty * 4 + i sees, from this split's first key on
  int sees[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = t.row0 + ty * 4 + i;
    const int64_t ahead = t.len - t.n + row / G + 1 - s0 * kKeys;
    sees[i] = row < t.n * G && ahead > 0 ? static_cast<int>(ahead) : 0;
  }
  const int64_t all_see = t.len - t.n + t.row0 / G + 1;   // keys that every row sees

  float o[4][kCols][4], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < kCols; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][c][e] = 0.f;
  }

  for (int64_t step = s0; step < s1; ++step) {
    const int64_t tok0 = step * kKeys;
    const int at = static_cast<int>(tok0 - s0 * kKeys);
    const int64_t base = key_at(p, t.b, h, tok0, D, threadIdx.x == 0);
    const int valid = static_cast<int>(min(static_cast<int64_t>(kKeys), t.keys - tok0));
    __syncthreads();
    // K, then V, each its own group of asynchronous copies; rows that no row sees are zeros
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const float* src = static_cast<const float*>(kv ? p.v_pool : p.k_pool) + base;
      for (int i = threadIdx.x; i < kKeys * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float* dst = kv ? &s.v[r][c] : &s.k[r][c];
        if (r < valid)
          cp_async16(dst, src + r * D + c);
        else
          *reinterpret_cast<float4*>(dst) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    // S = Q K^T: rows ty * 4 + i, keys tx + 16 j
    float a[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) a[i][j] = 0.f;
#pragma unroll 4
    for (int e = 0; e < D; e += 4) {
      float4 qv[4], kv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(&s.q[ty * 4 + i][e]);
#pragma unroll
      for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(&s.k[tx + 16 * j][e]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          a[i][j] = fmaf(qv[i].x, kv[j].x, fmaf(qv[i].y, kv[j].y,
                    fmaf(qv[i].z, kv[j].z, fmaf(qv[i].w, kv[j].w, a[i][j]))));
    }
    const bool border = tok0 + kKeys > all_see;           // some pair of this step is masked
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();                                      // K is read, V is there
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[i][j] = at + tx + 16 * j < sees[i] ? a[i][j] * p.scale_log2 : -INFINITY;
        mx = fmaxf(mx, a[i][j]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;       // all masked so far: weights 0
      const float keep = exp2f(m[i] - ref);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w = exp2f(a[i][j] - ref);
        s.p[ty * 4 + i][tx + 16 * j] = w;
        sum += w;
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = l[i] * keep + sum;
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][c][e] *= keep;
    }
    __syncwarp();                                         // a row's 16 writers share a warp
    // O += P V: rows ty * 4 + i, columns tx * 4 + 64 c
    if (!border) {
#pragma unroll 2
      for (int j = 0; j < kKeys; j += 4) {
        float4 pv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          pv[i] = *reinterpret_cast<const float4*>(&s.p[ty * 4 + i][j]);
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float4 v = *reinterpret_cast<const float4*>(&s.v[j + u][tx * 4 + 64 * c]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float w = u == 0 ? pv[i].x : u == 1 ? pv[i].y : u == 2 ? pv[i].z : pv[i].w;
              o[i][c][0] = fmaf(w, v.x, o[i][c][0]);
              o[i][c][1] = fmaf(w, v.y, o[i][c][1]);
              o[i][c][2] = fmaf(w, v.z, o[i][c][2]);
              o[i][c][3] = fmaf(w, v.w, o[i][c][3]);
            }
          }
      }
    } else {
#pragma unroll 2
      for (int j = 0; j < valid; ++j)
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(&s.v[j][tx * 4 + 64 * c]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = s.p[ty * 4 + i][j];
            if (at + j < sees[i]) {
              o[i][c][0] = fmaf(w, v.x, o[i][c][0]);
              o[i][c][1] = fmaf(w, v.y, o[i][c][1]);
              o[i][c][2] = fmaf(w, v.z, o[i][c][2]);
              o[i][c][3] = fmaf(w, v.w, o[i][c][3]);
            }
          }
        }
    }
  }

#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (t.row0 + ty * 4 + i < t.n * G)
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        finish4(p, t, tile, split, splits, h, G, ty * 4 + i, D, tx * 4 + 64 * c,
                make_float4(o[i][c][0], o[i][c][1], o[i][c][2], o[i][c][3]), m[i], l[i],
                tx == 0 && c == 0, part_acc, part_ml);
}

// Joins a tile's partial results in split order: one warp per row.
template <int D>
__global__ void __launch_bounds__(kThreads) chunk_join_kernel(ChunkParams p, int splits,
                                                              const float* part_acc,
                                                              const float* part_ml) {
  const int G = p.num_q_heads / p.num_kv_heads;
  const int h = blockIdx.y;
  grid_dependency_wait();
  Tile t;
  if (!find_tile(p, blockIdx.x, G, splits, &t) || t.splits == 1) return;
  const int lane = threadIdx.x & 31;
  const int64_t tile = static_cast<int64_t>(blockIdx.x) * p.num_kv_heads + h;
  constexpr int kVals = D / 32;
  for (int r = blockIdx.z * (kThreads / 32) + threadIdx.x / 32; r < kRows;
       r += gridDim.z * (kThreads / 32)) {
    const int64_t row = t.row0 + r;
    if (row >= t.n * G) break;
    // plain loads: the launch before this one wrote the parts (see grid_dependency_wait)
    const float2* ml = reinterpret_cast<const float2*>(part_ml) + tile * splits * kRows + r;
    float m = -INFINITY, l = 0.f, acc[kVals];
#pragma unroll
    for (int e = 0; e < kVals; ++e) acc[e] = 0.f;
    for (int i = lane; i < t.splits; i += 32) m = fmaxf(m, ml[i * kRows].x);
    m = warp_max(m);
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 8
    for (int i = 0; i < t.splits; ++i) {
      const float2 e2 = ml[i * kRows];
      const float* src = part_acc + ((tile * splits + i) * kRows + r) * D + lane;
      const float w = exp2f(e2.x - ref);                  // 0 for a split that saw nothing
      l = fmaf(w, e2.y, l);
#pragma unroll
      for (int e = 0; e < kVals; ++e) acc[e] = fmaf(w, src[e * 32], acc[e]);
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const int64_t out = ((t.first + row / G) * p.num_q_heads + h * G + row % G) * D;
#pragma unroll
    for (int e = 0; e < kVals; ++e) {
      static_cast<float*>(p.out)[out + e * 32 + lane] = acc[e] * inv;
    }
  }
}

template <int D>
cudaError_t launch(const ChunkParams& p, int splits, float* part_acc, float* part_ml,
                   cudaStream_t stream) {
  const int G = p.num_q_heads / p.num_kv_heads;
  const int64_t slots = chunk_simt_tiles(p.num_tokens, p.batch, G, 1);
  static std::atomic<unsigned long long> done{0};
  constexpr size_t kSmem = std::max(sizeof(SimtSmem<D>), sizeof(FewSmem<D>));
  cudaError_t e = ensure_dynamic_smem(chunk_simt_kernel<D>, kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(slots), p.num_kv_heads, splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, chunk_simt_kernel<D>, p, splits, part_acc, part_ml);
  if (e != cudaSuccess || splits == 1) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(slots), p.num_kv_heads, kRows / kWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel<D>, p, splits,
                            static_cast<const float*>(part_acc),
                            static_cast<const float*>(part_ml));
}

}  // namespace

int64_t chunk_simt_tiles(int64_t num_tokens, int batch, int group, int num_kv_heads) {
  return (num_tokens * group / kRows + batch) * num_kv_heads;
}

// Enough blocks to fill the device four times over (two are resident per SM; blocks differ in
// length, and with half as many a 1000-token prompt on 4000 tokens took 718 us instead of 602),
// and no more than the longest possible sequence can use.
int chunk_simt_splits(int64_t tiles, int64_t max_len, int sms) {
  const int64_t want = (8 * static_cast<int64_t>(sms) + tiles - 1) / tiles;
  const int64_t most = (max_len + kMinSpan * kKeys - 1) / (kMinSpan * kKeys);
  const int64_t s = want < most ? want : most;
  return static_cast<int>(s < 1 ? 1 : s > 64 ? 64 : s);
}

cudaError_t launch_chunk_simt(const ChunkParams& p, int head_dim, int splits, float* part_acc,
                              float* part_ml, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(p, splits, part_acc, part_ml, stream)
                         : launch<64>(p, splits, part_acc, part_ml, stream);
}

}  // namespace santa
