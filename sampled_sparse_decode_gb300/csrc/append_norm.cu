// append_norm.cu — a chunk's keys and values into the paged cache with the heads' norms, the rotation
// and the rounding to 8 bits on the way, and the representatives of the touched pages, in one launch.
//
//   y = x / sqrt(mean(x^2) + eps) * w          a query or key of one head (w may be absent)
//   pairs of y turned by the table's angle     as in append_chunk.cu
//   stored: y in the activations' type, or as codes and a scale (q8.cuh); values without norm and
//   rotation
//   representative = mean of the page's keys as stored
//
// The work items are those of append_chunk.cu: page items (half of the block for the keys, half for
// the values) and query items, with the same search for a block's sequence.  A row lies in the
// registers of 4 to 16 neighbouring lanes, two 16-byte pieces each, so the norm's sum and the row's
// largest magnitude are shuffles among them, and every element is read once and written once.
// With a cache of the activations' type the mean is summed in the order of reps.cu (its bits are
// santa_build_reps's); with 8 bits in the same order over the values that the codes stand for.
#include "append.cuh"
#include "q8.cuh"

namespace santa {

namespace {

// Where a thread's two pieces of a row stand, and what becomes of them.
struct Lane {
  int ca, cb;        // pieces
  int first;         // of the table row, for rotated pieces
  bool turned;
};

template <bool BF16>
__device__ __forceinline__ Lane lane_of(const AppendChunkParams& p, int pr) {
  constexpr int V = Piece<BF16>::kVec;
  Lane l;
  pair_pieces<BF16>(pr, p.rope_dim, p.interleaved, &l.ca, &l.cb);
  l.first = p.interleaved ? l.ca * V / 2 : l.ca * V;
  l.turned = l.ca * V < p.rope_dim;
  return l;
}

// Sum and largest word over the `kLanes` neighbouring lanes that hold a row (every lane of the warp
// takes part).
template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int kLanes>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <int V>
__device__ __forceinline__ uint32_t magnitude(const float (&a)[V], const float (&b)[V]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < V; ++e)
    m = max(m, max(__float_as_uint(a[e]) & 0x7fffffffu, __float_as_uint(b[e]) & 0x7fffffffu));
  return m;
}

// A thread's part of a norm's weights.
template <int V>
__device__ __forceinline__ void load_weights(const float* w, const Lane& l, float (&wa)[V],
                                             float (&wb)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    wa[e] = w ? w[l.ca * V + e] : 1.f;
    wb[e] = w ? w[l.cb * V + e] : 1.f;
  }
}

template <int V, int kLanes>
__device__ __forceinline__ void norm_row(float (&a)[V], float (&b)[V], const float (&wa)[V],
                                         const float (&wb)[V], int d, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
  const float r = __frsqrt_rn(row_sum<kLanes>(ss) / d + eps);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    a[e] = a[e] * r * wa[e];
    b[e] = b[e] * r * wb[e];
  }
}

// The rotation of a thread's pieces by the table row's entries from `first` on: by halves the pairs
// are (a_e, b_e); interleaved they are neighbours, V / 2 entries for each piece.
template <int V>
__device__ __forceinline__ void turn_row(float (&a)[V], float (&b)[V], const float* row,
                                         int half_dim, int first, bool interleaved) {
#pragma unroll
  for (int g = 0; g < V / 4; ++g) {
    const float4 c4 = *reinterpret_cast<const float4*>(row + first + 4 * g);
    const float4 s4 = *reinterpret_cast<const float4*>(row + half_dim + first + 4 * g);
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!interleaved) {
        turn_pair(a[4 * g + i], b[4 * g + i], c[i], s[i]);
      } else {
        const int e = 2 * (4 * g + i);
        if (e < V)
          turn_pair(a[e], a[e + 1], c[i], s[i]);
        else
          turn_pair(b[e - V], b[e - V + 1], c[i], s[i]);
      }
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack(const float (&x)[Piece<BF16>::kVec]) {
  if constexpr (BF16)
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
  else
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
}

// V codes of a piece: one or two words.
template <int C, int V>
__device__ __forceinline__ void store_codes(uint8_t* at, float (&x)[V], float scale) {
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    float y[4] = {x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    w[i] = q8_encode<C>(y, scale);
    x[4 * i] = y[0], x[4 * i + 1] = y[1], x[4 * i + 2] = y[2], x[4 * i + 3] = y[3];
  }
  if constexpr (V == 8)
    *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(at) = w[0];
}

// Stores a row's pieces at cache row `at` (a row index over all pages and heads); a and b become
// the values as stored.  Every lane of the warp takes part, `on` says which have a row.
template <bool BF16, int C, int D>
__device__ __forceinline__ void store_row(void* pool, float* scales, int64_t at, const Lane& l,
                                          bool on, float (&a)[Piece<BF16>::kVec],
                                          float (&b)[Piece<BF16>::kVec]) {
  constexpr int V = Piece<BF16>::kVec;
  if constexpr (C == kCodeNone) {
    const uint4 wa = pack<BF16>(a), wb = pack<BF16>(b);
    if (on) {
      uint4* row = static_cast<uint4*>(pool) + at * (D / V);
      row[l.ca] = wa;
      row[l.cb] = wb;
    }
    unpack<BF16>(wa, a);
    unpack<BF16>(wb, b);
  } else {
    const float scale = q8_scale<C>(row_max<D / V / 2>(magnitude(a, b)));
    if (!on) return;
    uint8_t* row = static_cast<uint8_t*>(pool) + at * D;
    store_codes<C>(row + l.ca * V, a, scale);
    store_codes<C>(row + l.cb * V, b, scale);
    if (threadIdx.x % (D / V / 2) == 0) scales[at] = scale;
  }
}

// The values of V codes in the first words of `w`.
template <int C, int V>
__device__ __forceinline__ void stored_codes(const uint4& w, float scale, float (&x)[V]) {
  const uint32_t word[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    float y[4];
    q8_decode<C>(word[i], y);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * i + e] = y[e] * scale;
  }
}
template <int V>
__device__ __forceinline__ void load_codes(const uint8_t* at, uint4& w) {
  if constexpr (V == 8) {
    const uint2 c = *reinterpret_cast<const uint2*>(at);
    w.x = c.x;
    w.y = c.y;
  } else {
    w.x = *reinterpret_cast<const uint32_t*>(at);
  }
}

template <bool BF16, int C, int D>
__device__ void norm_page_item(const AppendNormParams& p, int64_t slot, int h, float* part) {
  constexpr int V = Piece<BF16>::kVec;
  constexpr int kCols = D / V;                       // pieces per row
  constexpr int kPairs = kCols / 2;                  // lanes per row
  constexpr int kGroups = 256 / kCols;               // row groups of the mean (as in reps.cu)
  constexpr int kBatch = 4;                          // rows whose loads go out together
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
  const int64_t blk = (page * p.num_kv_heads + h) * static_cast<int64_t>(T);
  const int group = threadIdx.x % (kAppendThreads / 2) / kPairs;

  if (threadIdx.x < kAppendThreads / 2) {
    const Lane l = lane_of<BF16>(p, threadIdx.x % kPairs);
    const uint4* src = static_cast<const uint4*>(p.k_new) + h * kCols;
    const int64_t stride = p.k_stride / V;
    float wa[V], wb[V], sa[V], sb[V];
    load_weights<V>(p.k_norm, l, wa, wb);
#pragma unroll
    for (int e = 0; e < V; ++e) sa[e] = sb[e] = 0.f;
    for (int base = 0; base < row1; base += kBatch * kGroups) {
      uint4 xa[kBatch] = {}, xb[kBatch] = {};
      float old[kBatch] = {};                        // scales of earlier rows
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = base + group + i * kGroups;
        if (r >= row0 && r < row1) {
          xa[i] = src[(tok0 + r) * stride + l.ca];
          xb[i] = src[(tok0 + r) * stride + l.cb];
        } else if (r < row1) {
          if constexpr (C == kCodeNone) {
            const uint4* row = static_cast<const uint4*>(p.k_pool) + (blk + r) * kCols;
            xa[i] = row[l.ca];
            xb[i] = row[l.cb];
          } else {
            const uint8_t* row = static_cast<const uint8_t*>(p.k_pool) + (blk + r) * D;
            load_codes<V>(row + l.ca * V, xa[i]);
            load_codes<V>(row + l.cb * V, xb[i]);
            old[i] = p.k_scale[blk + r];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (base + i * kGroups >= row1) break;       // no lane of the block has such a row
        const int r = base + group + i * kGroups;
        const bool on = r >= row0 && r < row1;
        float a[V], y[V];
        unpack<BF16>(xa[i], a);
        unpack<BF16>(xb[i], y);
        if (base + (i + 1) * kGroups > row0) {       // new rows among the block's
          float na[V], nb[V];
#pragma unroll
          for (int e = 0; e < V; ++e) na[e] = a[e], nb[e] = y[e];
          if (p.k_norm) norm_row<V, kPairs>(na, nb, wa, wb, D, p.eps);
          if (on && l.turned)
            turn_row<V>(na, nb, p.rope + (team * T + r) * p.rope_dim, p.rope_dim / 2, l.first,
                        p.interleaved);
          store_row<BF16, C, D>(p.k_pool, p.k_scale, blk + r, l, on, na, nb);
          if (on) {
#pragma unroll
            for (int e = 0; e < V; ++e) a[e] = na[e], y[e] = nb[e];
          }
        }
        if constexpr (C != kCodeNone) {
          if (r < row0) {
            stored_codes<C, V>(xa[i], old[i], a);
            stored_codes<C, V>(xb[i], old[i], y);
          }
        }
        if (r < row1) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            sa[e] += a[e];
            sb[e] += y[e];
          }
        }
      }
    }
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      *reinterpret_cast<float4*>(part + group * D + l.ca * V + e) =
          make_float4(sa[e], sa[e + 1], sa[e + 2], sa[e + 3]);
      *reinterpret_cast<float4*>(part + group * D + l.cb * V + e) =
          make_float4(sb[e], sb[e + 1], sb[e + 2], sb[e + 3]);
    }
  } else {
    const int pr = threadIdx.x % kPairs;
    const Lane l = {pr, pr + kPairs, 0, false};
    const uint4* src = static_cast<const uint4*>(p.v_new) + h * kCols;
    const int64_t stride = p.v_stride / V;
    for (int base = row0; base < row1; base += kBatch * kGroups) {
      uint4 xa[kBatch] = {}, xb[kBatch] = {};
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = base + group + i * kGroups;
        if (r < row1) {
          xa[i] = src[(tok0 + r) * stride + l.ca];
          xb[i] = src[(tok0 + r) * stride + l.cb];
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (base + i * kGroups >= row1) break;
        const int r = base + group + i * kGroups;
        float a[V], y[V];
        unpack<BF16>(xa[i], a);
        unpack<BF16>(xb[i], y);
        store_row<BF16, C, D>(p.v_pool, p.v_scale, blk + r, l, r < row1, a, y);
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
__device__ void norm_query_item(const AppendNormParams& p, int64_t item) {
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
  const bool on = u < units && pos >= 0;             // not padding, not a skipped sequence
  const int h0 = static_cast<int>(u % chunks) * kHeadsPerUnit;
  const Lane l = lane_of<BF16>(p, threadIdx.x % kPairs);
  const uint4* src = static_cast<const uint4*>(p.q) + tok * (p.q_stride / V);
  uint4* dst = static_cast<uint4*>(p.q_out) + tok * p.num_q_heads * kCols;
  uint4 xa[kHeadsPerUnit] = {}, xb[kHeadsPerUnit] = {};
#pragma unroll
  for (int i = 0; i < kHeadsPerUnit; ++i)
    if (on && h0 + i < p.num_q_heads) {
      xa[i] = src[(h0 + i) * kCols + l.ca];
      xb[i] = src[(h0 + i) * kCols + l.cb];
    }
  float wa[V], wb[V];
  load_weights<V>(p.q_norm, l, wa, wb);
#pragma unroll
  for (int i = 0; i < kHeadsPerUnit; ++i) {
    float a[V], b[V];
    unpack<BF16>(xa[i], a);
    unpack<BF16>(xb[i], b);
    if (p.q_norm) norm_row<V, kPairs>(a, b, wa, wb, D, p.eps);
    if (on && h0 + i < p.num_q_heads) {
      if (l.turned)
        turn_row<V>(a, b, p.rope + pos * p.rope_dim, p.rope_dim / 2, l.first, p.interleaved);
      dst[(h0 + i) * kCols + l.ca] = pack<BF16>(a);
      dst[(h0 + i) * kCols + l.cb] = pack<BF16>(b);
    }
  }
}

// Page items first (they are longer), then query items.
template <bool BF16, int C, int D>
__global__ void __launch_bounds__(kAppendThreads, 2) append_norm_kernel(AppendNormParams p) {
  __shared__ __align__(16) float part[kAppendThreads / (D / Piece<BF16>::kVec) * D];
  grid_dependency_wait();
  if (blockIdx.x < p.page_items)
    norm_page_item<BF16, C, D>(p, blockIdx.x / p.num_kv_heads, blockIdx.x % p.num_kv_heads, part);
  else
    norm_query_item<BF16, D>(p, blockIdx.x - p.page_items);
  if (blockIdx.x == 0) check_bounds(p.cu_q, p.batch, p.num_tokens, p.status);
}

template <bool BF16, int D>
cudaError_t launch_typed(const cudaLaunchConfig_t& cfg, const AppendNormParams& p, int code) {
  switch (code) {
    case kCodeI8: return cudaLaunchKernelEx(&cfg, append_norm_kernel<BF16, kCodeI8, D>, p);
    case kCodeE4M3: return cudaLaunchKernelEx(&cfg, append_norm_kernel<BF16, kCodeE4M3, D>, p);
    default: return cudaLaunchKernelEx(&cfg, append_norm_kernel<BF16, kCodeNone, D>, p);
  }
}

}  // namespace

cudaError_t launch_append_norm(const AppendNormParams& params, int head_dim, bool bf16, int code,
                               cudaStream_t stream) {
  AppendNormParams p = params;
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
    return head_dim == 128 ? launch_typed<true, 128>(cfg, p, code)
                           : launch_typed<true, 64>(cfg, p, code);
  return head_dim == 128 ? launch_typed<false, 128>(cfg, p, code)
                         : launch_typed<false, 64>(cfg, p, code);
}

}  // namespace santa
