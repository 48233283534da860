// q8_read.cu — tokens of an 8-bit cache read back into a paged pool of bf16 or fp32 rows: a code
// times its row's scale, rounded to fp32 and, for bf16, once more.
//
// One block per (page, KV head).  A thread takes the codes of 16 bytes of output (8 or 4), so that a
// warp's stores are whole lines; four pieces of keys and four of values are asked for before the first is
// converted, and page ids are asked for beside the lengths that decide whether they count.  Bound by HBM:
// d + 4 bytes read and d elements written for every row.  Measured on GB300: 8 sequences of up to 8192 tokens
// (8 heads of 128, e4m3 to bf16) 38 us, 6.2 TB/s; 264 tokens of one to fp32 4.2 us.  16 codes per thread and
// two loads at a time took 45.6 and 6.2 us, two pieces ahead 39.4 and 4.9, eight 37.8 and 4.2 (71 registers).
#include <algorithm>

#include "kernels.h"
#include "q8.cuh"

namespace santa {

namespace {

constexpr int kReadThreads = 256;
constexpr int kAhead = 4;                            // pieces of each of keys and values
// Of a grid that is otherwise as wide as the tables: 64 x 128 tokens with tables of 1024 pages take 21 us,
// one block per entry 368, at most 2048 12; full tables 285, 283 and 298, 8 prompts 38.2, 38.3 and 40.9.
constexpr int kMostBlocks = 16384;

template <bool BF16>
struct Codes {
  uint32_t w[BF16 ? 2 : 1];
};
template <bool BF16>
__device__ __forceinline__ Codes<BF16> load_codes(const void* codes, int64_t at) {
  const uint8_t* from = static_cast<const uint8_t*>(codes) + at;
  Codes<BF16> c;
  if constexpr (BF16) {
    const uint2 v = *reinterpret_cast<const uint2*>(from);
    c.w[0] = v.x, c.w[1] = v.y;
  } else {
    c.w[0] = *reinterpret_cast<const uint32_t*>(from);
  }
  return c;
}

template <bool BF16, int C>
__device__ __forceinline__ void write_values(void* out, int64_t at, const Codes<BF16>& c, float scale) {
  float x[4];
  q8_decode<C>(c.w[0], x);
  if constexpr (BF16) {
    float y[4];
    q8_decode<C>(c.w[1], y);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
        make_uint4(pack_bf16(x[0] * scale, x[1] * scale), pack_bf16(x[2] * scale, x[3] * scale),
                   pack_bf16(y[0] * scale, y[1] * scale), pack_bf16(y[2] * scale, y[3] * scale));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) =
        make_float4(x[0] * scale, x[1] * scale, x[2] * scale, x[3] * scale);
  }
}

template <bool BF16, int C, int D>
__device__ __forceinline__ void read_page(const Q8ReadParams& p, int team, int h, int first, int len,
                                          int64_t src, int64_t dst) {
  constexpr int kPiece = BF16 ? 8 : 4, kCols = D / kPiece;
  const int T = p.team_size;
  const int row0 = max(first - team * T, 0), row1 = min(len - team * T, T);
  if (row0 >= row1) return;
  if (src < 0 || src >= p.num_pages || dst < 0 || dst >= p.dst_pages) {
    if (h == 0 && threadIdx.x == 0) set_status(p.status, SANTA_DEV_BAD_PAGE);
    return;
  }
  const int64_t from = (src * p.num_kv_heads + h) * T, to = (dst * p.num_kv_heads + h) * T;
  for (int i0 = row0 * kCols + threadIdx.x; i0 < row1 * kCols; i0 += kAhead * kReadThreads) {
    Codes<BF16> k[kAhead], v[kAhead];
    float ks[kAhead], vs[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int i = i0 + e * kReadThreads;
      if (i < row1 * kCols) {
        k[e] = load_codes<BF16>(p.k, from * D + i * kPiece);
        v[e] = load_codes<BF16>(p.v, from * D + i * kPiece);
        ks[e] = p.k_scale[from + i / kCols];
        vs[e] = p.v_scale[from + i / kCols];
      }
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int i = i0 + e * kReadThreads;
      if (i < row1 * kCols) {
        write_values<BF16, C>(p.k_out, to * D + i * kPiece, k[e], ks[e]);
        write_values<BF16, C>(p.v_out, to * D + i * kPiece, v[e], vs[e]);
      }
    }
  }
}

template <bool BF16, int C, int D>
__global__ void __launch_bounds__(kReadThreads) q8_read_kernel(Q8ReadParams p) {
  grid_dependency_wait();
  const int h = blockIdx.y, b = blockIdx.z, T = p.team_size;
  const int32_t* src_ids = p.page_table + static_cast<int64_t>(b) * p.max_teams;
  const int32_t* dst_ids = p.dst_table + static_cast<int64_t>(b) * p.max_teams;
  const int len = p.seq_lens[b], first = p.first ? p.first[b] : 0;
  // a grid as wide as the table: page ids beside the lengths; else every gridDim.x-th page from the first
  const bool all = gridDim.x == p.max_teams;
  int64_t src = 0, dst = 0;
  if (all) {
    src = src_ids[blockIdx.x];
    dst = dst_ids[blockIdx.x];
  }
  if (first < 0 || len < first || len > p.max_teams * T) {
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) set_status(p.status, SANTA_DEV_BAD_SEQLEN);
    return;
  }
  if (all) {
    read_page<BF16, C, D>(p, blockIdx.x, h, first, len, src, dst);
    return;
  }
  for (int team = first / T + blockIdx.x; team * T < len; team += gridDim.x)
    read_page<BF16, C, D>(p, team, h, first, len, src_ids[team], dst_ids[team]);
}

template <bool BF16, int C>
cudaError_t launch_typed(const cudaLaunchConfig_t& cfg, const Q8ReadParams& p, int d) {
  return d == 128 ? cudaLaunchKernelEx(&cfg, q8_read_kernel<BF16, C, 128>, p)
                  : cudaLaunchKernelEx(&cfg, q8_read_kernel<BF16, C, 64>, p);
}

}  // namespace

cudaError_t launch_q8_read(const Q8ReadParams& p, int head_dim, bool bf16, int code,
                           cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // blocks of pages that are not asked for end at once, but still have to start: a bounded number of them
  const int64_t units = static_cast<int64_t>(p.num_kv_heads) * p.batch;
  const int64_t wide = std::max<int64_t>(1, std::min<int64_t>(p.max_teams, kMostBlocks / units));
  cfg.gridDim = dim3(static_cast<unsigned>(wide), p.num_kv_heads, p.batch);
  cfg.blockDim = dim3(kReadThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (code == kCodeI8)
    return bf16 ? launch_typed<true, kCodeI8>(cfg, p, head_dim)
                : launch_typed<false, kCodeI8>(cfg, p, head_dim);
  return bf16 ? launch_typed<true, kCodeE4M3>(cfg, p, head_dim)
              : launch_typed<false, kCodeE4M3>(cfg, p, head_dim);
}

}  // namespace santa
