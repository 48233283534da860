// append_norm.cu — a chunk's keys and values into the paged cache with the heads' norms, the rotation
// and the rounding to 8 bits on the way, and the representatives of the touched pages, in one launch.
//
//   y = x / sqrt(mean(x^2) + eps) * w          a query or key of one head (w may be absent)
//   pairs of y turned by the table's angle     as in append_chunk.cu
//   stored: y in the activations' type, or as codes and a scale (q8.cuh); values without norm and
//   rotation
//   representative = mean of the page's keys as stored
//
// The work items are those of append_chunk.cu, page items (touched page, KV head) and query items, with
// the same search for a block's sequence.  A row lies in the registers of 8 or 16 neighbouring lanes,
// two quads of elements each: the two that a rotation by halves pairs up, or neighbours.  The norm's sum
// and the row's largest magnitude are shuffles among them; every element is read once and written once.
// Quads rather than 16-byte pieces keep a thread's row, sums and weights in 8 registers each, so that
// three blocks stay on a multiprocessor; values, which need no sums, are taken in 16-byte pieces.
//
// With a cache of the activations' type the mean is summed in the order of reps.cu (its bits are
// santa_build_reps's): rows group, group + kGroups, ... of a quad in row order, then the groups.  bf16 rows
// fill a block with the groups of reps.cu, and the values are blocks of their own; fp32 rows fill half of
// one, and the other half takes the values.
//
// Bound by latency for single tokens, by issue and HBM together for prompts.  Measured on GB300: 8
// sequences of 4096 tokens (32 query and 8 KV heads of 128, bf16, norms, e4m3) 140 us, 5.4 TB/s of what
// must move; one token for each of 8 sequences into an int8 cache 4.2 us.  Both sides: 16-byte pieces, two
// blocks per SM 200 us, quads and three 178 (two 220, four 174 with spills); true divisions 239 against
// 200; register pairs 155 -> 144, kernels with and without norms 144 -> 139; four query heads per search
// 205 against 178 (eight), 16 in two turns 158 against 141; page items spread among the query items 139
// against 141.5, but 2148 tokens 18.5 against 16.8.
#include "append.cuh"
#include "q8.cuh"

namespace santa {

namespace {

constexpr int kQuad = 4;                             // elements

template <bool BF16, int D>
struct Rows {
  static constexpr int kQuads = D / kQuad;           // of a row
  static constexpr int kLanes = kQuads / 2;          // of a row
  static constexpr int kGroups = 256 / (D * (BF16 ? 2 : 4) / 16);   // row groups of reps.cu
  static constexpr int kTeam = kGroups * kLanes;     // threads that share a page's keys or values
  static constexpr bool kApart = kTeam == kAppendThreads;   // keys and values in blocks of their own
  static constexpr int kLoad = BF16 ? 4 : 2;         // rows whose loads go out together
  static constexpr int kHeads = BF16 ? 8 : 4;        // query heads that share cosines and sines
  static_assert(kApart || kTeam == kAppendThreads / 2, "the block is one team or two");
};

// A quad as it is in memory: two words (bf16) or four.
template <bool BF16>
struct Raw {
  uint32_t w[BF16 ? 2 : 4];
};
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_raw(const void* base, int64_t element) {
  Raw<BF16> r;
  if constexpr (BF16) {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + element);
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const float*>(base) + element);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  }
  return r;
}
template <bool BF16>
__device__ __forceinline__ void store_raw(void* base, int64_t element, const Raw<BF16>& r) {
  if constexpr (BF16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + element) = make_uint2(r.w[0], r.w[1]);
  else
    *reinterpret_cast<uint4*>(static_cast<float*>(base) + element) =
        make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
}
// A lane's part of a row: two quads, (x[0], x[1]) and (x[2], x[3]), each x two neighbours in a register
// pair, so that one instruction works on both.
struct Part {
  uint64_t x[4];
};
template <bool BF16>
__device__ __forceinline__ void values_of(const Raw<BF16>& r, uint64_t& lo, uint64_t& hi) {
  if constexpr (BF16) {
    lo = pair(bf16_lo(r.w[0]), bf16_hi(r.w[0]));
    hi = pair(bf16_lo(r.w[1]), bf16_hi(r.w[1]));
  } else {
    lo = pair(__uint_as_float(r.w[0]), __uint_as_float(r.w[1]));
    hi = pair(__uint_as_float(r.w[2]), __uint_as_float(r.w[3]));
  }
}
template <bool BF16>
__device__ __forceinline__ Part values_of(const Raw<BF16>& a, const Raw<BF16>& b) {
  Part r;
  values_of<BF16>(a, r.x[0], r.x[1]);
  values_of<BF16>(b, r.x[2], r.x[3]);
  return r;
}
template <bool BF16>
__device__ __forceinline__ Raw<BF16> round_to(uint64_t lo, uint64_t hi) {
  const float2 a = halves(lo), b = halves(hi);
  Raw<BF16> r;
  if constexpr (BF16) {
    r.w[0] = pack_bf16(a.x, a.y), r.w[1] = pack_bf16(b.x, b.y);
  } else {
    r.w[0] = __float_as_uint(a.x), r.w[1] = __float_as_uint(a.y);
    r.w[2] = __float_as_uint(b.x), r.w[3] = __float_as_uint(b.y);
  }
  return r;
}

// Where a lane's two quads stand in a row (elements), and where its angles start in a table row.
struct Lane {
  int a, b;
  int first;
  bool turned;
};
__device__ __forceinline__ Lane lane_of(const AppendChunkParams& p, int pr) {
  const int half = p.interleaved ? 0 : p.rope_dim / (2 * kQuad);
  Lane l;
  if (pr < half) {
    l.a = kQuad * pr;
    l.b = l.a + kQuad * half;
  } else {
    l.a = 2 * kQuad * pr;                            // neighbours, behind the paired ones
    l.b = l.a + kQuad;
  }
  l.first = p.interleaved ? l.a / 2 : l.a;
  l.turned = l.a < p.rope_dim;
  return l;
}

// Largest magnitudes of N rows over the kLanes neighbouring lanes that hold a row (the whole warp calls).
template <int kLanes, int N>
__device__ __forceinline__ void row_max(float (&v)[N]) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float u = __shfl_xor_sync(0xffffffffu, v[i], o);
      v[i] = max_abs(v[i], u, u);
    }
}
__device__ __forceinline__ float magnitude(const Part& v) {
  const float2 a = halves(v.x[0]), b = halves(v.x[1]), c = halves(v.x[2]), d = halves(v.x[3]);
  return max_abs(max_abs(max_abs(a.x, a.y, b.x), b.y, c.x), max_abs(c.y, d.x, d.y), 0.f);
}

// A lane's part of a norm's weights.
__device__ __forceinline__ Part load_weights(const float* w, const Lane& l) {
  Part r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.x[i] = twice(1.f);
  if (w) {
    const float4 a = *reinterpret_cast<const float4*>(w + l.a);
    const float4 b = *reinterpret_cast<const float4*>(w + l.b);
    r = {{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
  }
  return r;
}
// N rows at a time, so that their chains of shuffles overlap.
template <int kLanes, int D, int N>
__device__ __forceinline__ void norm_rows(Part (&v)[N], const Part& w, float eps) {
  float ss[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint64_t s = mul_pair(v[i].x[0], v[i].x[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) s = fma_pair(v[i].x[e], v[i].x[e], s);
    const float2 h = halves(s);
    ss[i] = h.x + h.y;
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], o);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint64_t r = twice(rsqrtf(ss[i] * (1.f / D) + eps));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i].x[e] = mul_pair(mul_pair(v[i].x[e], r), w.x[e]);
  }
}

// Cosines and sines of a lane's four pairs of elements at one position.
struct Angles {
  float4 c, s;
};
__device__ __forceinline__ Angles load_angles(const float* row, int half_dim) {
  return {*reinterpret_cast<const float4*>(row), *reinterpret_cast<const float4*>(row + half_dim)};
}
// By halves the rotated pairs are (a_e, b_e) of the two quads, interleaved they are neighbours.  EXACT:
// products and sums rounded one by one, as in append_chunk.cu, for calls without norms (one by one also in
// the instructions: a product and a sum of register pairs may be contracted); else the first product in the
// sum's rounding.
template <bool EXACT>
__device__ __forceinline__ void turn_row(Part& v, const Angles& t, bool interleaved) {
  const float c[4] = {t.c.x, t.c.y, t.c.z, t.c.w}, s[4] = {t.s.x, t.s.y, t.s.z, t.s.w};
  if constexpr (EXACT) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = halves(v.x[i]);
      x[2 * i] = h.x, x[2 * i + 1] = h.y;
    }
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) turn_pair(x[2 * i], x[2 * i + 1], c[i], s[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) turn_pair(x[i], x[4 + i], c[i], s[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v.x[i] = pair(x[2 * i], x[2 * i + 1]);
  } else if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = halves(v.x[i]);
      v.x[i] = fma_pair(v.x[i], twice(c[i]), mul_pair(pair(h.y, h.x), pair(-s[i], s[i])));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t x = v.x[i], y = v.x[2 + i], cc = pair(c[2 * i], c[2 * i + 1]);
      v.x[i] = fma_pair(x, cc, mul_pair(y, pair(-s[2 * i], -s[2 * i + 1])));
      v.x[2 + i] = fma_pair(y, cc, mul_pair(x, pair(s[2 * i], s[2 * i + 1])));
    }
  }
}

// A touched page: its rows before row0 are cached already, row0 .. row1 - 1 are new.
struct Page {
  int row0, row1;
  int64_t tok0;        // token row of page row 0 (may be before the chunk's first)
  int64_t at;          // row 0 among the cache's rows
  int64_t pos;         // position of row 0
};

template <bool BF16, int C, int D, bool NORM>
__device__ __forceinline__ void key_rows(const AppendNormParams& p, const Page& pg, int h, int thread,
                                         float* part) {
  using R = Rows<BF16, D>;
  constexpr int kElement = BF16 ? 2 : 4, kCached = C == kCodeNone ? kElement : 1;   // bytes
  const int group = thread / R::kLanes;
  const Lane l = lane_of(p, thread % R::kLanes);
  const Part w = load_weights(NORM ? p.k_norm : nullptr, l);
  // this lane's quads of page row `group` among the new rows (may be before the first) and in the cache
  const char* src =
      static_cast<const char*>(p.k_new) + ((pg.tok0 + group) * p.k_stride + h * D) * kElement;
  const int64_t src_step = R::kGroups * p.k_stride * kElement;
  char* pool = static_cast<char*>(p.k_pool) + (pg.at + group) * D * kCached;
  float* scales = p.k_scale + pg.at + group;
  const float* angles = p.rope + (pg.pos + group) * p.rope_dim + l.first;
  Part sum;
#pragma unroll
  for (int e = 0; e < 4; ++e) sum.x[e] = 0;
  for (int base = group; base - group < pg.row1; base += R::kLoad * R::kGroups) {
    Raw<BF16> xa[R::kLoad] = {}, xb[R::kLoad] = {};
    float old[R::kLoad] = {};                        // scales of earlier rows
#pragma unroll
    for (int i = 0; i < R::kLoad; ++i) {
      const int r = base + i * R::kGroups;
      const char* row = src + i * src_step;
      const char* cached = pool + i * R::kGroups * D * kCached;
      if (r >= pg.row0 && r < pg.row1) {
        xa[i] = load_raw<BF16>(row, l.a);
        xb[i] = load_raw<BF16>(row, l.b);
      } else if (r < pg.row1) {
        if constexpr (C == kCodeNone) {
          xa[i] = load_raw<BF16>(cached, l.a);
          xb[i] = load_raw<BF16>(cached, l.b);
        } else {
          xa[i].w[0] = *reinterpret_cast<const uint32_t*>(cached + l.a);
          xb[i].w[0] = *reinterpret_cast<const uint32_t*>(cached + l.b);
          old[i] = scales[i * R::kGroups];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < R::kLoad; ++i) {
      const int r = base + i * R::kGroups;
      if (r - group >= pg.row1) break;               // no lane of the team has such a row
      const bool on = r >= pg.row0 && r < pg.row1;
      // what is added to the mean: the row as stored, codes' values with their scale
      Part v[1];
      float scale = 1.f;
      if (r - group + R::kGroups > pg.row0) {        // new rows among the team's: all lanes take part
        v[0] = values_of<BF16>(xa[i], xb[i]);
        Angles t = {};
        if (on && l.turned) t = load_angles(angles + i * R::kGroups * p.rope_dim, p.rope_dim / 2);
        if (NORM && p.k_norm) norm_rows<R::kLanes, D>(v, w, p.eps);
        if (l.turned) turn_row<!NORM>(v[0], t, p.interleaved);
        char* cached = pool + i * R::kGroups * D * kCached;
        if constexpr (C == kCodeNone) {
          if (on) {
            const Raw<BF16> a = round_to<BF16>(v[0].x[0], v[0].x[1]), b = round_to<BF16>(v[0].x[2], v[0].x[3]);
            store_raw<BF16>(cached, l.a, a);
            store_raw<BF16>(cached, l.b, b);
            v[0] = values_of<BF16>(a, b);
          }
        } else {
          float amax[1] = {magnitude(v[0])};
          row_max<R::kLanes>(amax);
          if (on) {
            const Scale s = q8_scale<C>(amax[0]);
            uint64_t a[2] = {v[0].x[0], v[0].x[1]}, b[2] = {v[0].x[2], v[0].x[3]};
            *reinterpret_cast<uint32_t*>(cached + l.a) = q8_encode<C>(a, s);
            *reinterpret_cast<uint32_t*>(cached + l.b) = q8_encode<C>(b, s);
            if (l.a == 0) scales[i * R::kGroups] = s.s;
            v[0] = {{a[0], a[1], b[0], b[1]}};
            scale = s.s;
          }
        }
      }
      if (r < pg.row0) {
        if constexpr (C == kCodeNone) {
          v[0] = values_of<BF16>(xa[i], xb[i]);
        } else {
          float a[kQuad], b[kQuad];
          q8_decode<C>(xa[i].w[0], a);
          q8_decode<C>(xb[i].w[0], b);
          v[0] = {{pair(a[0], a[1]), pair(a[2], a[3]), pair(b[0], b[1]), pair(b[2], b[3])}};
          scale = old[i];
        }
      }
      if (r < pg.row1) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sum.x[e] = C == kCodeNone ? add_pair(sum.x[e], v[0].x[e])
                                    : fma_pair(v[0].x[e], twice(scale), sum.x[e]);
      }
    }
    src += R::kLoad * src_step;
    pool += R::kLoad * R::kGroups * D * kCached;
    scales += R::kLoad * R::kGroups;
    angles += static_cast<int64_t>(R::kLoad) * R::kGroups * p.rope_dim;
  }
  const float2 s0 = halves(sum.x[0]), s1 = halves(sum.x[1]), s2 = halves(sum.x[2]), s3 = halves(sum.x[3]);
  *reinterpret_cast<float4*>(part + group * D + l.a) = make_float4(s0.x, s0.y, s1.x, s1.y);
  *reinterpret_cast<float4*>(part + group * D + l.b) = make_float4(s2.x, s2.y, s3.x, s3.y);
}

// Values: a lane has two 16-byte pieces of a row, half a row apart (nothing else is held in registers).
template <bool BF16, int C, int D>
__device__ __forceinline__ void value_rows(const AppendNormParams& p, const Page& pg, int h, int thread) {
  constexpr int V = Piece<BF16>::kVec, kLanes = D / V / 2, kRows = Rows<BF16, D>::kTeam / kLanes;
  constexpr int kElement = BF16 ? 2 : 4, kCached = C == kCodeNone ? kElement : 1;   // bytes
  constexpr int kLoad = 4;
  const int group = thread / kLanes, col = thread % kLanes * V;
  const char* src = static_cast<const char*>(p.v_new) +
                    ((pg.tok0 + pg.row0 + group) * p.v_stride + h * D + col) * kElement;
  const int64_t src_step = kRows * p.v_stride * kElement;
  char* pool = static_cast<char*>(p.v_pool) + ((pg.at + pg.row0 + group) * D + col) * kCached;
  float* scales = p.v_scale + pg.at + pg.row0 + group;
  for (int base = pg.row0 + group; base - group < pg.row1; base += kLoad * kRows) {
    uint4 xa[kLoad] = {}, xb[kLoad] = {};
#pragma unroll
    for (int i = 0; i < kLoad; ++i)
      if (base + i * kRows < pg.row1) {
        xa[i] = *reinterpret_cast<const uint4*>(src + i * src_step);
        xb[i] = *reinterpret_cast<const uint4*>(src + i * src_step + D / 2 * kElement);
      }
#pragma unroll
    for (int i = 0; i < kLoad; ++i) {
      const int r = base + i * kRows;
      if (r - group >= pg.row1) break;
      char* row = pool + i * kRows * D * kCached;
      if constexpr (C == kCodeNone) {
        if (r < pg.row1) {
          *reinterpret_cast<uint4*>(row) = xa[i];
          *reinterpret_cast<uint4*>(row + D / 2 * kElement) = xb[i];
        }
      } else {
        float a[V], b[V], amax[1];
        unpack<BF16>(xa[i], a);
        unpack<BF16>(xb[i], b);
        if constexpr (BF16) {
          const uint32_t m = max_abs_bf16x2(
              max_abs_bf16x2(max_abs_bf16x2(xa[i].x, xa[i].y), max_abs_bf16x2(xa[i].z, xa[i].w)),
              max_abs_bf16x2(max_abs_bf16x2(xb[i].x, xb[i].y), max_abs_bf16x2(xb[i].z, xb[i].w)));
          amax[0] = max_abs(bf16_lo(m), bf16_hi(m), bf16_hi(m));
        } else {
          amax[0] = max_abs(max_abs(max_abs(a[0], a[1], a[2]), a[3], b[0]),
                            max_abs(b[1], b[2], b[3]), 0.f);
        }
        row_max<kLanes>(amax);
        if (r < pg.row1) {
          const Scale s = q8_scale<C>(amax[0]);
#pragma unroll
          for (int piece = 0; piece < 2; ++piece) {
            uint32_t codes[V / 4];
#pragma unroll
            for (int q = 0; q < V / 4; ++q) {
              const float* x = (piece ? b : a) + 4 * q;
              uint64_t y[2] = {pair(x[0], x[1]), pair(x[2], x[3])};
              codes[q] = q8_encode<C>(y, s);
            }
            char* to = row + piece * (D / 2);
            if constexpr (BF16)
              *reinterpret_cast<uint2*>(to) = make_uint2(codes[0], codes[V / 4 - 1]);
            else
              *reinterpret_cast<uint32_t*>(to) = codes[0];
          }
          if (col == 0) scales[i * kRows] = s.s;
        }
      }
    }
    src += kLoad * src_step;
    pool += kLoad * kRows * D * kCached;
    scales += kLoad * kRows;
  }
}

template <bool BF16, int C, int D, bool NORM>
__device__ __forceinline__ void norm_page_item(const AppendNormParams& p, int64_t slot, int h,
                                               bool values, float* part) {
  using R = Rows<BF16, D>;
  const int T = p.team_size;
  const int b = find_sequence(p.cu_q, p.batch, p.num_tokens, T, 2, slot);
  Chunk c;
  if (!load_chunk(p, b, &c)) {
    if (threadIdx.x == 0) set_status(p.status, SANTA_DEV_BAD_SEQLEN);
    return;
  }
  const int64_t j = slot - (c.first / T + 2 * static_cast<int64_t>(b));
  if (j == 0 && h == 0 && !values && threadIdx.x == 0 && p.seq_lens_next)
    p.seq_lens_next[b] = static_cast<int32_t>(c.len + c.n);
  const int64_t team = c.len / T + j;                // the touched page, by position
  if (c.n == 0 || j < 0 || team * T >= c.len + c.n) return;
  const int64_t page = p.page_table[static_cast<int64_t>(b) * p.max_teams + team];
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) set_status(p.status, SANTA_DEV_BAD_PAGE);
    return;
  }
  Page pg;
  pg.row0 = static_cast<int>(max(c.len - team * T, static_cast<int64_t>(0)));
  pg.row1 = static_cast<int>(min(c.len + c.n - team * T, static_cast<int64_t>(T)));
  pg.tok0 = c.first + team * T - c.len;
  pg.at = (page * p.num_kv_heads + h) * static_cast<int64_t>(T);
  pg.pos = team * T;
  if constexpr (R::kApart) {
    if (values) {
      value_rows<BF16, C, D>(p, pg, h, threadIdx.x);
      return;
    }
    key_rows<BF16, C, D, NORM>(p, pg, h, threadIdx.x, part);
  } else if (threadIdx.x < R::kTeam) {
    key_rows<BF16, C, D, NORM>(p, pg, h, threadIdx.x, part);
  } else {
    value_rows<BF16, C, D>(p, pg, h, threadIdx.x - R::kTeam);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kAppendThreads) {
    float s = part[e];
#pragma unroll
    for (int g = 1; g < R::kGroups; ++g) s += part[g * D + e];
    p.reps[(page * p.num_kv_heads + h) * D + e] = s / pg.row1;
  }
}

// The last sequence b < batch with cu[b] <= t (0 if there is none); any cu at all gives some b.  The whole
// warp calls it with the same arguments; 32 candidates per round.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int batch, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool below = lane == 0 || (at < hi && cu[at] <= t);
    lo += (31 - __clz(__ballot_sync(0xffffffffu, below))) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Units of a query item: (token, kHeads heads), one for every kLanes lanes.
template <bool BF16, int D>
__host__ __device__ constexpr int query_units() {
  return kAppendThreads / Rows<BF16, D>::kLanes;
}

template <bool BF16, int D, bool NORM>
__device__ __forceinline__ void norm_query_item(const AppendNormParams& p, unsigned item) {
  using R = Rows<BF16, D>;
  constexpr int kStep = 2;                           // heads that are worked on together
  constexpr int kElement = BF16 ? 2 : 4;             // bytes
  constexpr int kUnits = query_units<BF16, D>();
  constexpr int kUnitsPerWarp = 32 / R::kLanes;
  // unit number = token * chunks + head group: item = chunks * whole + rest, units at + u of a warp, by
  // 32-bit divisions (chunks < 2^14, items < 2^31)
  const unsigned chunks = (p.num_q_heads + R::kHeads - 1) / R::kHeads;
  const unsigned whole = item / chunks, rest = item - whole * chunks;
  const unsigned at = rest * kUnits + (threadIdx.x / 32) * kUnitsPerWarp;
  const unsigned tokens = at / chunks;
  const int64_t t0 = static_cast<int64_t>(whole) * kUnits + tokens;
  if (t0 >= p.num_tokens) return;
  unsigned mine = at - tokens * chunks + (threadIdx.x % 32) / R::kLanes, more = 0;   // head group, token
#pragma unroll
  for (int i = 1; i < kUnitsPerWarp; ++i)
    if (mine >= chunks) {
      mine -= chunks;
      ++more;
    }
  const int64_t tok = t0 + more;
  const int h0 = static_cast<int>(mine) * R::kHeads;
  const Lane l = lane_of(p, threadIdx.x % R::kLanes);
  // the rows before the search, which they do not wait for; what is not there is read as what is
  const int heads = tok < p.num_tokens ? min(p.num_q_heads - h0, R::kHeads) : 0;
  const char* src = static_cast<const char*>(p.q) +
                    (min(tok, p.num_tokens - 1) * p.q_stride + h0 * D) * kElement;
  char* dst = static_cast<char*>(p.q_out) + (tok * p.num_q_heads + h0) * D * kElement;
  const int last_head = p.num_q_heads - 1 - h0;
  Raw<BF16> xa[R::kHeads], xb[R::kHeads];
#pragma unroll
  for (int i = 0; i < R::kHeads; ++i) {
    const char* row = src + min(i, last_head) * D * kElement;
    xa[i] = load_raw<BF16>(row, l.a);
    xb[i] = load_raw<BF16>(row, l.b);
  }
  const Part w = load_weights(NORM ? p.q_norm : nullptr, l);
  // the warp's units cover few tokens: one search for each
  int64_t pos = -1;
#pragma unroll
  for (int i = 0; i < kUnitsPerWarp; ++i) {
    const int64_t t = t0 + i;
    if (t >= p.num_tokens || !__any_sync(0xffffffffu, tok == t)) break;
    const int b = sequence_of(p.cu_q, p.batch, static_cast<int>(t));
    Chunk c;
    const bool ok = load_chunk(p, b, &c) && t >= c.first && t < c.first + c.n;
    if (ok && t == tok) pos = c.len + (t - c.first);
  }
  const bool on = pos >= 0;                          // not padding, not a skipped sequence
  Angles t = {};
  if (on && l.turned) t = load_angles(p.rope + pos * p.rope_dim + l.first, p.rope_dim / 2);
#pragma unroll
  for (int i0 = 0; i0 < R::kHeads; i0 += kStep) {
    Part v[kStep];
#pragma unroll
    for (int i = 0; i < kStep; ++i) v[i] = values_of<BF16>(xa[i0 + i], xb[i0 + i]);
    if (NORM && p.q_norm) norm_rows<R::kLanes, D>(v, w, p.eps);
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      if (!on || i0 + i >= heads) continue;
      if (l.turned) turn_row<!NORM>(v[i], t, p.interleaved);
      char* row = dst + (i0 + i) * D * kElement;
      store_raw<BF16>(row, l.a, round_to<BF16>(v[i].x[0], v[i].x[1]));
      store_raw<BF16>(row, l.b, round_to<BF16>(v[i].x[2], v[i].x[3]));
    }
  }
}

// Page items first (they are longer), then query items.
template <bool BF16, int C, int D, bool NORM>
__global__ void __launch_bounds__(kAppendThreads, 3) append_norm_kernel(AppendNormParams p) {
  __shared__ __align__(16) float part[Rows<BF16, D>::kGroups * D];
  grid_dependency_wait();
  if (blockIdx.x < p.page_items) {
    const unsigned item = Rows<BF16, D>::kApart ? blockIdx.x / 2 : blockIdx.x;
    const bool values = Rows<BF16, D>::kApart && (blockIdx.x & 1);
    norm_page_item<BF16, C, D, NORM>(p, item / p.num_kv_heads, item % p.num_kv_heads, values, part);
  } else {
    norm_query_item<BF16, D, NORM>(p, blockIdx.x - p.page_items);
  }
  if (blockIdx.x == 0) check_bounds(p.cu_q, p.batch, p.num_tokens, p.status);
}

// Blocks of query items of a launch.
template <bool BF16, int D>
int64_t query_blocks(int64_t num_tokens, int num_q_heads) {
  const int64_t chunks = (num_q_heads + Rows<BF16, D>::kHeads - 1) / Rows<BF16, D>::kHeads;
  return (num_tokens * chunks + query_units<BF16, D>() - 1) / query_units<BF16, D>();
}

template <bool BF16, int D>
cudaError_t launch_typed(AppendNormParams p, int code, cudaStream_t stream) {
  p.page_items = static_cast<uint32_t>(
      append_page_blocks(p.num_tokens, p.batch, p.num_kv_heads, p.team_size) *
      (Rows<BF16, D>::kApart ? 2 : 1));
  const int64_t items =
      p.page_items + (p.q ? query_blocks<BF16, D>(p.num_tokens, p.num_q_heads) : 0);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool norm = p.q_norm || p.k_norm;
  switch (code) {
    case kCodeI8:
      return norm ? cudaLaunchKernelEx(&cfg, append_norm_kernel<BF16, kCodeI8, D, true>, p)
                  : cudaLaunchKernelEx(&cfg, append_norm_kernel<BF16, kCodeI8, D, false>, p);
    case kCodeE4M3:
      return norm ? cudaLaunchKernelEx(&cfg, append_norm_kernel<BF16, kCodeE4M3, D, true>, p)
                  : cudaLaunchKernelEx(&cfg, append_norm_kernel<BF16, kCodeE4M3, D, false>, p);
    default:
      return norm ? cudaLaunchKernelEx(&cfg, append_norm_kernel<BF16, kCodeNone, D, true>, p)
                  : cudaLaunchKernelEx(&cfg, append_norm_kernel<BF16, kCodeNone, D, false>, p);
  }
}

}  // namespace

int64_t append_norm_blocks(int64_t num_tokens, int batch, int num_q_heads, int num_kv_heads,
                           int head_dim, int team_size, bool bf16) {
  const int64_t q = bf16 ? (head_dim == 128 ? query_blocks<true, 128>(num_tokens, num_q_heads)
                                            : query_blocks<true, 64>(num_tokens, num_q_heads))
                         : (head_dim == 128 ? query_blocks<false, 128>(num_tokens, num_q_heads)
                                            : query_blocks<false, 64>(num_tokens, num_q_heads));
  return append_page_blocks(num_tokens, batch, num_kv_heads, team_size) * 2 + q;
}

cudaError_t launch_append_norm(const AppendNormParams& p, int head_dim, bool bf16, int code,
                               cudaStream_t stream) {
  if (bf16)
    return head_dim == 128 ? launch_typed<true, 128>(p, code, stream)
                           : launch_typed<true, 64>(p, code, stream);
  return head_dim == 128 ? launch_typed<false, 128>(p, code, stream)
                         : launch_typed<false, 64>(p, code, stream);
}

}  // namespace santa
