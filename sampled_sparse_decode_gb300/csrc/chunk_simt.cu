// chunk_simt.cu — causal attention of a chunk of new tokens over the paged cache in plain fp32
// arithmetic (fp32 caches).
//
// A KV head's G query heads share its keys, so the rows of a tile are (token, head) pairs: row
// r of a sequence's n * G rows is token r / G, head r % G.  One block takes 64 rows and walks the
// keys they see in tiles of 64, with the running maximum and sum of an online softmax (base 2):
//   S = Q K^T (4 x 4 scores per thread), P = 2^(S - m), O = 2^(m_old - m) O + P V (4 x d/16).
// K and V go through shared memory once per tile; fp32 FMA bound (about 9 FMAs per 16-byte
// shared load).  With few tiles the keys of a tile are split over several blocks, whose partial
// (m, l, O) a second launch joins in order.  Tiles are found from cu_q through slots, as in
// append_chunk.cu: sequence b owns floor(cu[b] G / 64) + b onward, at least ceil(n G / 64).
//
// Masked scores never enter: P is 0 there, and in a tile that holds a masked pair (the causal
// border) the product with V is selected away too, because 0 * V is not 0 when V is not finite.
#include "kernels.h"

namespace santa {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;        // query rows per tile
constexpr int kKeys = 64;        // keys per step (divides both page sizes)

template <int D>
struct SimtSmem {
  float q[kRows][D + 4];         // +4: rows 16 apart would share banks
  float k[kKeys][D + 4];
  float v[kKeys][D];
  float p[kRows][kKeys + 4];
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
};

__device__ __forceinline__ bool find_tile(const ChunkParams& p, int64_t slot, int G, Tile* t) {
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
  return true;
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
  if (blockIdx.x == 0 && h == 0 && split == 0) check_bounds(p.cu_q, p.batch, p.num_tokens, p.status);
  Tile t;
  if (!find_tile(p, blockIdx.x, G, &t)) return;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int64_t steps = (t.keys + kKeys - 1) / kKeys;
  const int64_t per = (steps + splits - 1) / splits;
  const int64_t s0 = split * per, s1 = min(steps, s0 + per);

  for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    const int64_t row = t.row0 + r;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < t.n * G)
      x = load4(p.q, ((t.first + row / G) * p.num_q_heads + h * G + row % G) * D + c);
    *reinterpret_cast<float4*>(&s.q[r][c]) = x;
  }
  // keys that row ty * 4 + i sees
  int64_t sees[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = t.row0 + ty * 4 + i;
    sees[i] = row < t.n * G ? t.len - t.n + row / G + 1 : 0;
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
    int64_t page = p.page_table[static_cast<int64_t>(t.b) * p.max_teams + tok0 / p.team_size];
    if (page < 0 || page >= p.num_pages) {
      if (threadIdx.x == 0) set_status(p.status, SANTA_DEV_BAD_PAGE);
      page = 0;
    }
    const int64_t base =
        ((page * p.num_kv_heads + h) * p.team_size + tok0 % p.team_size) * static_cast<int64_t>(D);
    const int valid = static_cast<int>(min(static_cast<int64_t>(kKeys), t.keys - tok0));
    __syncthreads();
    for (int i = threadIdx.x; i < kKeys * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
      if (r < valid) {
        kx = load4(p.k_pool, base + r * D + c);
        vx = load4(p.v_pool, base + r * D + c);
      }
      *reinterpret_cast<float4*>(&s.k[r][c]) = kx;
      *reinterpret_cast<float4*>(&s.v[r][c]) = vx;
    }
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
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[i][j] = tok0 + tx + 16 * j < sees[i] ? a[i][j] * p.scale_log2 : -INFINITY;
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
      for (int j = 0; j < valid; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (tok0 + j < sees[i]) {
            const float w = s.p[ty * 4 + i][j];
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
              const float4 v = *reinterpret_cast<const float4*>(&s.v[j][tx * 4 + 64 * c]);
              o[i][c][0] = fmaf(w, v.x, o[i][c][0]);
              o[i][c][1] = fmaf(w, v.y, o[i][c][1]);
              o[i][c][2] = fmaf(w, v.z, o[i][c][2]);
              o[i][c][3] = fmaf(w, v.w, o[i][c][3]);
            }
          }
    }
  }

  const int64_t tile = static_cast<int64_t>(blockIdx.x) * p.num_kv_heads + h;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = t.row0 + ty * 4 + i;
    if (row >= t.n * G) continue;
    if (splits == 1) {
      const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;
      const int64_t out = ((t.first + row / G) * p.num_q_heads + h * G + row % G) * D;
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        store4(p.out, out + tx * 4 + 64 * c,
                     make_float4(o[i][c][0] * inv, o[i][c][1] * inv, o[i][c][2] * inv,
                                 o[i][c][3] * inv));
    } else {
      const int64_t at = (tile * splits + split) * kRows + ty * 4 + i;
      if (tx == 0) {
        part_ml[2 * at] = m[i];
        part_ml[2 * at + 1] = l[i];
      }
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        *reinterpret_cast<float4*>(part_acc + at * D + tx * 4 + 64 * c) =
            make_float4(o[i][c][0], o[i][c][1], o[i][c][2], o[i][c][3]);
    }
  }
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
  if (!find_tile(p, blockIdx.x, G, &t)) return;
  const int lane = threadIdx.x & 31;
  const int64_t tile = static_cast<int64_t>(blockIdx.x) * p.num_kv_heads + h;
  constexpr int kVals = D / 32;
  for (int r = blockIdx.z * (kThreads / 32) + threadIdx.x / 32; r < kRows;
       r += gridDim.z * (kThreads / 32)) {
    const int64_t row = t.row0 + r;
    if (row >= t.n * G) break;
    float m = -INFINITY, l = 0.f, acc[kVals];
#pragma unroll
    for (int e = 0; e < kVals; ++e) acc[e] = 0.f;
    for (int i = 0; i < splits; ++i)
      m = fmaxf(m, __ldg(part_ml + 2 * ((tile * splits + i) * kRows + r)));
    const float ref = m == -INFINITY ? 0.f : m;
    for (int i = 0; i < splits; ++i) {
      const int64_t at = (tile * splits + i) * kRows + r;
      const float mi = __ldg(part_ml + 2 * at);
      const float w = exp2f(mi - ref);                    // 0 for a split that saw nothing
      l = fmaf(w, __ldg(part_ml + 2 * at + 1), l);
#pragma unroll
      for (int e = 0; e < kVals; ++e)
        acc[e] = fmaf(w, __ldg(part_acc + at * D + e * 32 + lane), acc[e]);
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
  cudaError_t e = ensure_dynamic_smem(chunk_simt_kernel<D>, sizeof(SimtSmem<D>), done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(slots), p.num_kv_heads, splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(SimtSmem<D>);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, chunk_simt_kernel<D>, p, splits, part_acc, part_ml);
  if (e != cudaSuccess || splits == 1) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(slots), p.num_kv_heads, 2);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel<D>, p, splits,
                            static_cast<const float*>(part_acc),
                            static_cast<const float*>(part_ml));
}

}  // namespace

int64_t chunk_simt_tiles(int64_t num_tokens, int batch, int group, int num_kv_heads) {
  return (num_tokens * group / kRows + batch) * num_kv_heads;
}

// Enough blocks to fill the device twice over (two are resident per SM), unless a block would
// be left with fewer than 4 steps of the longest sequence.
int chunk_simt_splits(int64_t tiles, int64_t max_len, int sms) {
  const int64_t want = (4 * static_cast<int64_t>(sms) + tiles - 1) / tiles;
  const int64_t most = (max_len + 4 * kKeys - 1) / (4 * kKeys);
  const int64_t s = want < most ? want : most;
  return static_cast<int>(s < 1 ? 1 : s > 64 ? 64 : s);
}

cudaError_t launch_chunk_simt(const ChunkParams& p, int head_dim, int splits, float* part_acc,
                              float* part_ml, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(p, splits, part_acc, part_ml, stream)
                         : launch<64>(p, splits, part_acc, part_ml, stream);
}

}  // namespace santa
