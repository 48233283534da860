// q8_read.cu — tokens of an 8-bit cache read back into a paged pool of bf16 or fp32 rows: a code
// times its row's scale, rounded once (fp32 holds an int8 or e4m3 code times an fp32 scale to its last
// bit or half of it).
//
// One block per (page, KV head): a thread takes 16 codes of a row (one 16-byte load) and stores 16
// values.  Bound by HBM: d + 4 bytes read and d elements written for every row.
#include "kernels.h"
#include "q8.cuh"

namespace santa {

namespace {

constexpr int kReadThreads = 256;

template <bool BF16, int C>
__device__ __forceinline__ void write_values(void* out, int64_t at, const uint4& w, float scale) {
  const uint32_t word[4] = {w.x, w.y, w.z, w.w};
  float x[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y[4];
    q8_decode<C>(word[i], y);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * i + e] = y[e] * scale;
  }
  if constexpr (BF16) {
    uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      to[i] = make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                         pack_bf16(x[8 * i + 4], x[8 * i + 5]),
                         pack_bf16(x[8 * i + 6], x[8 * i + 7]));
  } else {
    float4* to = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      to[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
}

template <bool BF16, int C, int D>
__global__ void __launch_bounds__(kReadThreads) q8_read_kernel(Q8ReadParams p) {
  constexpr int kCols = D / 16;
  grid_dependency_wait();
  const int team = blockIdx.x, h = blockIdx.y, b = blockIdx.z, T = p.team_size;
  const int64_t len = p.seq_lens[b], first = p.first ? p.first[b] : 0;
  if (first < 0 || len < first || len > static_cast<int64_t>(p.max_teams) * T) {
    if (team == 0 && h == 0 && threadIdx.x == 0) set_status(p.status, SANTA_DEV_BAD_SEQLEN);
    return;
  }
  const int row0 = static_cast<int>(max(first - static_cast<int64_t>(team) * T, int64_t(0)));
  const int row1 = static_cast<int>(min(len - static_cast<int64_t>(team) * T, int64_t(T)));
  if (row0 >= row1) return;
  const int64_t at = static_cast<int64_t>(b) * p.max_teams + team;
  const int64_t src = p.page_table[at], dst = p.dst_table[at];
  if (src < 0 || src >= p.num_pages || dst < 0 || dst >= p.dst_pages) {
    if (h == 0 && threadIdx.x == 0) set_status(p.status, SANTA_DEV_BAD_PAGE);
    return;
  }
  const int64_t from = (src * p.num_kv_heads + h) * T, to = (dst * p.num_kv_heads + h) * T;
  for (int i = row0 * kCols + threadIdx.x; i < row1 * kCols; i += kReadThreads) {
    const int r = i / kCols, col = i % kCols;
    const uint4 k = static_cast<const uint4*>(p.k)[(from + r) * kCols + col];
    const uint4 v = static_cast<const uint4*>(p.v)[(from + r) * kCols + col];
    write_values<BF16, C>(p.k_out, (to + r) * D + col * 16, k, p.k_scale[from + r]);
    write_values<BF16, C>(p.v_out, (to + r) * D + col * 16, v, p.v_scale[from + r]);
  }
}

template <bool BF16, int C>
cudaError_t launch_typed(const cudaLaunchConfig_t& cfg, const Q8ReadParams& p, int d) {
  return d == 128 ? cudaLaunchKernelEx(&cfg, q8_read_kernel<BF16, C, 128>, p)
                  : cudaLaunchKernelEx(&cfg, q8_read_kernel<BF16, C, 64>, p);
}

}  // namespace

cudaError_t launch_q8_read(const Q8ReadParams& p, int head_dim, bool bf16, int code, int sms,
                           cudaStream_t stream) {
  (void)sms;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.max_teams, p.num_kv_heads, p.batch);
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
