// append_chunk.cu — a chunk's keys and values into the paged cache, rotated by position on the
// way, with the representatives of the touched pages brought up to date, in one launch.
//
// Work items, one block each:
//   page items  (touched page, KV head): half of the block's threads rotate the page's new keys,
//               store them and sum the page's valid keys; the other half copies the values.
//   query items a run of (token, four query heads) units: rotate and store.
// How many pages a sequence touches is known on the device only, so the page items are indexed
// through slots: sequence b owns the slots [s(b), s(b + 1)), s(b) = floor(cu_q[b] / T) + 2 b.
// A chunk of n tokens touches at most floor((n - 2) / T) + 2 pages and owns at least
// floor(n / T) + 2 slots, and s is found from cu_q alone (a 32-way search per block, one load
// for up to 32 sequences), without a scan over the batch.  At most two slots per sequence stay
// empty; their blocks return at once.
//
// The mean is summed exactly as reps.cu sums it: the rows group, group + G, ... of piece `col`
// in row order, then the groups in order.  There thread (col, group) owns one 16-byte piece;
// here thread (pair, group) owns the two pieces that a rotation by halves pairs up, so a
// cosine and a sine serve both of its elements and the 128 threads cover the same split.
//
// Bound by HBM for prompts and by latency for single tokens.  Measured on GB300: 8 sequences of
// 4096 tokens (32 query and 8 KV heads of 128, bf16) 134 us, 6.1 TB/s of what must move; one token
// for each of 8 sequences 3.9 us.  The page items' key loop takes four rows at a time with all of
// their loads first (single tokens 4.4 -> 4.0 us), and three blocks per SM rather than two or four
// (145, 133, 143 us for the prompts).
#include "append.cuh"

namespace santa {

namespace {

// Four pairs of a rotation: cosines and sines c, s of four consecutive table entries.  By halves
// the pairs are (a_e, b_e) of two bf16 words each; interleaved they are the neighbours in four
// bf16 words.  A pair of pieces takes two such groups (bf16) or one (fp32), and only one group's
// table entries are in registers at a time.
__device__ __forceinline__ void turn_halves(uint32_t& a0, uint32_t& a1, uint32_t& b0, uint32_t& b1,
                                            const float4& c, const float4& s) {
  float x[4] = {bf16_lo(a0), bf16_hi(a0), bf16_lo(a1), bf16_hi(a1)};
  float y[4] = {bf16_lo(b0), bf16_hi(b0), bf16_lo(b1), bf16_hi(b1)};
  turn_pair(x[0], y[0], c.x, s.x);
  turn_pair(x[1], y[1], c.y, s.y);
  turn_pair(x[2], y[2], c.z, s.z);
  turn_pair(x[3], y[3], c.w, s.w);
  a0 = pack_bf16(x[0], x[1]);
  a1 = pack_bf16(x[2], x[3]);
  b0 = pack_bf16(y[0], y[1]);
  b1 = pack_bf16(y[2], y[3]);
}
__device__ __forceinline__ void turn_word(uint32_t& w, float c, float s) {
  float x = bf16_lo(w), y = bf16_hi(w);
  turn_pair(x, y, c, s);
  w = pack_bf16(x, y);
}
__device__ __forceinline__ void turn_neighbours(uint4& w, const float4& c, const float4& s) {
  turn_word(w.x, c.x, s.x);
  turn_word(w.y, c.y, s.y);
  turn_word(w.z, c.z, s.z);
  turn_word(w.w, c.w, s.w);
}
__device__ __forceinline__ void turn_f32(uint32_t& a, uint32_t& b, float c, float s) {
  float x = __uint_as_float(a), y = __uint_as_float(b);
  turn_pair(x, y, c, s);
  a = __float_as_uint(x);
  b = __float_as_uint(y);
}

// Rotates N pairs of pieces that share a position, with the table row's entries from `first` on:
// by halves both pieces of a pair use the same kVec entries; interleaved, piece a uses kVec / 2
// and piece b (the next one) the kVec / 2 after them.
// Its read-only loads ask that no launch that lets the next one start early writes the table:
// santa_rope_table does not.
template <bool BF16, int N>
__device__ __forceinline__ void rotate(uint4 (&a)[N], uint4 (&b)[N], const float* row, int half_dim,
                                       int first, bool interleaved) {
#pragma unroll
  for (int group = 0; group < (BF16 ? 2 : 1); ++group) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + first + 4 * group));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + half_dim + first + 4 * group));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (BF16) {
        if (interleaved)
          turn_neighbours(group == 0 ? a[i] : b[i], c, s);
        else if (group == 0)
          turn_halves(a[i].x, a[i].y, b[i].x, b[i].y, c, s);
        else
          turn_halves(a[i].z, a[i].w, b[i].z, b[i].w, c, s);
      } else if (interleaved) {
        turn_f32(a[i].x, a[i].y, c.x, s.x);
        turn_f32(a[i].z, a[i].w, c.y, s.y);
        turn_f32(b[i].x, b[i].y, c.z, s.z);
        turn_f32(b[i].z, b[i].w, c.w, s.w);
      } else {
        turn_f32(a[i].x, b[i].x, c.x, s.x);
        turn_f32(a[i].y, b[i].y, c.y, s.y);
        turn_f32(a[i].z, b[i].z, c.z, s.z);
        turn_f32(a[i].w, b[i].w, c.w, s.w);
      }
    }
  }
}

template <bool BF16, int D>
__device__ void page_item(const AppendChunkParams& p, int64_t slot, int h, float* part) {
  constexpr int V = Piece<BF16>::kVec;
  constexpr int kCols = D / V;                       // pieces per row
  constexpr int kPairs = kCols / 2;
  constexpr int kGroups = 256 / kCols;               // row groups of the mean (as in reps.cu)
  static_assert(kPairs * kGroups == kAppendThreads / 2, "half of the block covers the split");
  const int T = p.team_size;
  const int b = find_sequence(p.cu_q, p.batch, p.num_tokens, T, 2, slot);
  Chunk c;
  if (!load_chunk(p, b, &c)) {
    if (threadIdx.x == 0) set_status(p.status, SANTA_DEV_BAD_SEQLEN);
    return;
  }
  const int64_t j = slot - (c.first / T + 2 * static_cast<int64_t>(b));
  if (j == 0 && h == 0 && threadIdx.x == 0 && p.seq_lens_next)
    p.seq_lens_next[b] = static_cast<int32_t>(c.len + c.n);
  const int64_t team = c.len / T + j;                // the touched page, by position
  if (c.n == 0 || j < 0 || team * T >= c.len + c.n) return;
  const int64_t page = p.page_table[static_cast<int64_t>(b) * p.max_teams + team];
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) set_status(p.status, SANTA_DEV_BAD_PAGE);
    return;
  }
  const int row0 = static_cast<int>(max(c.len - team * T, static_cast<int64_t>(0)));
  const int row1 = static_cast<int>(min(c.len + c.n - team * T, static_cast<int64_t>(T)));
  const int64_t tok0 = c.first + team * T - c.len;   // token row of page row 0 (may be < first)
  const int64_t blk = (page * p.num_kv_heads + h) * static_cast<int64_t>(T) * kCols;

  if (threadIdx.x < kAppendThreads / 2) {
    const int pr = threadIdx.x % kPairs, group = threadIdx.x / kPairs;
    int ca, cb;
    pair_pieces<BF16>(pr, p.rope_dim, p.interleaved, &ca, &cb);
    const bool turned = ca * V < p.rope_dim;
    const int first = p.interleaved ? ca * V / 2 : ca * V;
    uint4* pool = static_cast<uint4*>(p.k_pool) + blk;
    const uint4* src = static_cast<const uint4*>(p.k_new) + h * kCols;
    const int64_t stride = p.k_stride / V;
    float sa[V], sb[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sa[e] = sb[e] = 0.f;
    // four rows at a time, all of their loads before the first use
    constexpr int kBatch = 4;
    for (int r0 = group; r0 < row1; r0 += kBatch * kGroups) {
      uint4 wa[kBatch], wb[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + i * kGroups;
        if (r < row1) {
          const uint4* row = r < row0 ? pool + r * kCols : src + (tok0 + r) * stride;
          wa[i] = row[ca];
          wb[i] = row[cb];
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + i * kGroups;
        if (r >= row1) break;
        if (r >= row0) {
          if (turned) {
            uint4 a1[1] = {wa[i]}, b1[1] = {wb[i]};
            rotate<BF16>(a1, b1, p.rope + (team * T + r) * p.rope_dim, p.rope_dim / 2, first,
                         p.interleaved);
            wa[i] = a1[0];
            wb[i] = b1[0];
          }
          pool[r * kCols + ca] = wa[i];
          pool[r * kCols + cb] = wb[i];
        }
        float xa[V], xb[V];
        unpack<BF16>(wa[i], xa);
        unpack<BF16>(wb[i], xb);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          sa[e] += xa[e];
          sb[e] += xb[e];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      *reinterpret_cast<float4*>(part + group * D + ca * V + e) =
          make_float4(sa[e], sa[e + 1], sa[e + 2], sa[e + 3]);
      *reinterpret_cast<float4*>(part + group * D + cb * V + e) =
          make_float4(sb[e], sb[e + 1], sb[e + 2], sb[e + 3]);
    }
  } else {
    const int t = threadIdx.x - kAppendThreads / 2;
    uint4* pool = static_cast<uint4*>(p.v_pool) + blk;
    const uint4* src = static_cast<const uint4*>(p.v_new) + h * kCols;
    const int64_t stride = p.v_stride / V;
    // eight pieces at a time, all of their loads first (plain ones: what the launch before this one
    // writes is no read-only data to it)
    constexpr int kBatch = 8, kStep = kAppendThreads / 2;
    for (int i0 = row0 * kCols + t; i0 < row1 * kCols; i0 += kBatch * kStep) {
      uint4 w[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int i = i0 + e * kStep;
        if (i < row1 * kCols) w[e] = src[(tok0 + i / kCols) * stride + i % kCols];
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int i = i0 + e * kStep;
        if (i < row1 * kCols) pool[i] = w[e];
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kAppendThreads) {
    float s = part[e];
#pragma unroll
    for (int g = 1; g < kGroups; ++g) s += part[g * D + e];
    p.reps[(page * p.num_kv_heads + h) * D + e] = s / row1;
  }
}

template <bool BF16, int D>
__device__ void query_item(const AppendChunkParams& p, int64_t item) {
  constexpr int V = Piece<BF16>::kVec;
  constexpr int kCols = D / V;
  constexpr int kPairs = kCols / 2;
  constexpr int kUnits = kAppendThreads / kPairs;    // (token, head group) units per block
  constexpr int kUnitsPerWarp = 32 / kPairs;
  const int chunks = (p.num_q_heads + kHeadsPerUnit - 1) / kHeadsPerUnit;
  const int64_t units = p.num_tokens * chunks;
  const int64_t u0 = item * kUnits + (threadIdx.x / 32) * kUnitsPerWarp;   // of this warp
  if (u0 >= units) return;
  const int64_t u = u0 + (threadIdx.x % 32) / kPairs;
  const int64_t tok = u / chunks;
  // the warp's units cover few tokens: one search for each
  const int64_t last = min(u0 + kUnitsPerWarp, units) - 1;
  int64_t pos = -1;
  for (int64_t t = u0 / chunks; t <= last / chunks; ++t) {
    const int b = find_sequence(p.cu_q, p.batch, p.num_tokens, 1, 0, t);
    Chunk c;
    const bool ok = load_chunk(p, b, &c) && t >= c.first && t < c.first + c.n;
    if (ok && t == tok) pos = c.len + (t - c.first);
  }
  if (u >= units || pos < 0) return;                 // padding, or a skipped sequence
  const int h0 = static_cast<int>(u % chunks) * kHeadsPerUnit;
  int ca, cb;
  pair_pieces<BF16>(threadIdx.x % kPairs, p.rope_dim, p.interleaved, &ca, &cb);
  const uint4* src = static_cast<const uint4*>(p.q) + tok * (p.q_stride / V);
  uint4* dst = static_cast<uint4*>(p.q_out) + tok * p.num_q_heads * kCols;
  uint4 wa[kHeadsPerUnit] = {}, wb[kHeadsPerUnit] = {};
#pragma unroll
  for (int i = 0; i < kHeadsPerUnit; ++i)
    if (h0 + i < p.num_q_heads) {
      wa[i] = src[(h0 + i) * kCols + ca];
      wb[i] = src[(h0 + i) * kCols + cb];
    }
  if (ca * V < p.rope_dim)
    rotate<BF16>(wa, wb, p.rope + pos * p.rope_dim, p.rope_dim / 2,
                 p.interleaved ? ca * V / 2 : ca * V, p.interleaved);
#pragma unroll
  for (int i = 0; i < kHeadsPerUnit; ++i)
    if (h0 + i < p.num_q_heads) {
      dst[(h0 + i) * kCols + ca] = wa[i];
      dst[(h0 + i) * kCols + cb] = wb[i];
    }
}

// Page items first (they are longer), then query items.
template <bool BF16, int D>
__global__ void __launch_bounds__(kAppendThreads, 3) append_chunk_kernel(AppendChunkParams p) {
  __shared__ __align__(16) float part[kAppendThreads / (D / Piece<BF16>::kVec) * D];
  grid_dependency_wait();
  if (blockIdx.x < p.page_items)
    page_item<BF16, D>(p, blockIdx.x / p.num_kv_heads, blockIdx.x % p.num_kv_heads, part);
  else
    query_item<BF16, D>(p, blockIdx.x - p.page_items);
  if (blockIdx.x == 0) check_bounds(p.cu_q, p.batch, p.num_tokens, p.status);
}

// theta^(-2j/R), the angle and its cosine and sine in 64 bits: at position 131072 an fp32
// angle is off by up to 2^-8 radian.  Bound by 64-bit arithmetic; runs once per model.
__global__ void rope_table_kernel(float* table, int64_t positions, int rope_dim, double theta) {
  const int half = rope_dim / 2;
  const int64_t total = positions * half;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t pos = i / half;
    const int j = static_cast<int>(i % half);
    double s, c;
    sincos(static_cast<double>(pos) * pow(theta, -static_cast<double>(j) / half), &s, &c);
    table[pos * rope_dim + j] = static_cast<float>(c);
    table[pos * rope_dim + half + j] = static_cast<float>(s);
  }
}

}  // namespace

int64_t append_chunk_blocks(int64_t num_tokens, int batch, int num_q_heads, int num_kv_heads,
                            int head_dim, int team_size, bool bf16) {
  const int units = kAppendThreads / (head_dim / (bf16 ? 8 : 4) / 2);
  const int64_t chunks = (num_q_heads + kHeadsPerUnit - 1) / kHeadsPerUnit;
  return append_page_blocks(num_tokens, batch, num_kv_heads, team_size) +
         (num_tokens * chunks + units - 1) / units;
}

cudaError_t launch_append_chunk(const AppendChunkParams& params, int head_dim, bool bf16,
                                cudaStream_t stream) {
  AppendChunkParams p = params;
  const int64_t items = append_chunk_blocks(p.num_tokens, p.batch, p.q ? p.num_q_heads : 0,
                                            p.num_kv_heads, head_dim, p.team_size, bf16);
  p.page_items =
      static_cast<uint32_t>(append_page_blocks(p.num_tokens, p.batch, p.num_kv_heads, p.team_size));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (bf16)
    return head_dim == 128 ? cudaLaunchKernelEx(&cfg, append_chunk_kernel<true, 128>, p)
                           : cudaLaunchKernelEx(&cfg, append_chunk_kernel<true, 64>, p);
  return head_dim == 128 ? cudaLaunchKernelEx(&cfg, append_chunk_kernel<false, 128>, p)
                         : cudaLaunchKernelEx(&cfg, append_chunk_kernel<false, 64>, p);
}

cudaError_t launch_rope_table(float* table, int64_t positions, int rope_dim, double theta,
                              cudaStream_t stream) {
  const int64_t total = positions * (rope_dim / 2);
  const int64_t blocks = (total + 255) / 256;
  rope_table_kernel<<<static_cast<unsigned>(blocks < 65536 ? blocks : 65536), 256, 0, stream>>>(
      table, positions, rope_dim, theta);
  return cudaGetLastError();
}

}  // namespace santa
