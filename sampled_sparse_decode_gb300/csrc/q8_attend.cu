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
// A warp takes one token at a time; a lane holds d / 32 elements of every query head of the group.
// The second launch adds a unit's partial results in the order of the splits.
#include <algorithm>

#include "kernels.h"
#include "q8.cuh"

namespace santa {

namespace {

constexpr int kQ8Threads = 256;
constexpr int kQ8Warps = kQ8Threads / 32;

// The tokens that a unit may see: positions lo .. len - 1 (dense), or `count` listed teams.
struct Unit {
  int64_t len, lo;
  int count;
};
__device__ __forceinline__ bool load_unit(const Q8AttendParams& p, int b, int h, Unit* u) {
  u->len = p.seq_lens[b];
  if (u->len < 0 || u->len > static_cast<int64_t>(p.max_teams) * p.team_size) return false;
  u->lo = p.window > 0 && u->len > p.window ? u->len - p.window : 0;
  u->count = 0;
  if (p.sel_ids) {
    u->count = p.sel_count[static_cast<int64_t>(b) * p.num_kv_heads + h];
    if (u->count < 0 || u->count > p.num_draws) {
      set_status(p.status, SANTA_DEV_BAD_SEL);
      u->count = u->count < 0 ? 0 : p.num_draws;
    }
  }
  return true;
}

template <int C, int W>
__device__ __forceinline__ void load_row(const void* codes, int64_t row, int lane, float (&x)[W]) {
  const uint8_t* at = static_cast<const uint8_t*>(codes) + row * (32 * W) + lane * W;
  float y[4];
  if constexpr (W == 4) {
    q8_decode<C>(*reinterpret_cast<const uint32_t*>(at), y);
  } else {
    q8_decode<C>(*reinterpret_cast<const uint16_t*>(at), y);
  }
#pragma unroll
  for (int e = 0; e < W; ++e) x[e] = y[e];
}

template <bool BF16, int C, int D>
__global__ void __launch_bounds__(kQ8Threads) q8_attend_kernel(Q8AttendParams p) {
  constexpr int W = D / 32;
  __shared__ float acc_s[kQ8Warps][D];
  __shared__ float ml_s[kQ8Warps][2];
  grid_dependency_wait();
  const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z, T = p.team_size;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int G = p.num_q_heads / p.num_kv_heads;
  const int64_t unit = static_cast<int64_t>(b) * p.num_kv_heads + h;
  float q[kMaxGroup][W], acc[kMaxGroup][W], m[kMaxGroup], l[kMaxGroup];
#pragma unroll
  for (int g = 0; g < kMaxGroup; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < W; ++e) {
      acc[g][e] = q[g][e] = 0.f;
      if (g < G) {
        const int64_t at = (static_cast<int64_t>(b) * p.num_q_heads + h * G + g) * D + lane * W + e;
        q[g][e] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p.q)[at])
                       : static_cast<const float*>(p.q)[at];
      }
    }
  }
  Unit u;
  const bool ok = load_unit(p, b, h, &u);
  if (!ok && threadIdx.x == 0) set_status(p.status, SANTA_DEV_BAD_SEQLEN);
  const int64_t n = !ok ? 0 : p.sel_ids ? static_cast<int64_t>(u.count) * T : u.len - u.lo;
  const int64_t begin = n * split / p.splits, end = n * (split + 1) / p.splits;
  for (int64_t i = begin + warp; i < end; i += kQ8Warps) {
    int64_t t = u.lo + i;
    float bias = 0.f;
    if (p.sel_ids) {
      const int64_t at = unit * p.num_draws + i / T;
      const int64_t team = p.sel_ids[at];
      const float pi = p.pi[at];
      if (team < 0 || team * T >= u.len || !(pi > 0.f) || pi == INFINITY) {
        set_status(p.status, SANTA_DEV_BAD_SEL);
        continue;
      }
      t = team * T + i % T;
      bias = -logf(pi);
      if (t >= u.len || t < u.lo) continue;
    }
    const int64_t page = p.page_table[static_cast<int64_t>(b) * p.max_teams + t / T];
    if (page < 0 || page >= p.num_pages) {
      set_status(p.status, SANTA_DEV_BAD_PAGE);
      continue;
    }
    const int64_t row = (page * p.num_kv_heads + h) * T + t % T;
    float k[W], v[W];
    load_row<C, W>(p.k, row, lane, k);
    load_row<C, W>(p.v, row, lane, v);
    const float ks = p.k_scale[row] * p.scale, vs = p.v_scale[row];
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g) {
      if (g >= G) break;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < W; ++e) s = fmaf(q[g][e], k[e], s);
      s = warp_sum(s) * ks;
      if (p.softcap > 0.f) s = p.softcap * tanhf(s / p.softcap);
      s += bias;
      const float top = fmaxf(m[g], s);
      const float ref = top == -INFINITY ? 0.f : top;
      const float keep = expf(m[g] - ref), w = expf(s - ref);
      m[g] = top;
      l[g] = l[g] * keep + w;
#pragma unroll
      for (int e = 0; e < W; ++e) acc[g][e] = acc[g][e] * keep + w * vs * v[e];
    }
  }
#pragma unroll
  for (int g = 0; g < kMaxGroup; ++g) {
    if (g >= G) break;
#pragma unroll
    for (int e = 0; e < W; ++e) acc_s[warp][lane * W + e] = acc[g][e];
    if (lane == 0) {
      ml_s[warp][0] = m[g];
      ml_s[warp][1] = l[g];
    }
    __syncthreads();
    float* part = p.part + ((unit * p.splits + split) * G + g) * (D + 2);
    if (threadIdx.x < D) {
      float top = -INFINITY, sum = 0.f, z = 0.f;
      for (int w = 0; w < kQ8Warps; ++w) top = fmaxf(top, ml_s[w][0]);
      const float ref = top == -INFINITY ? 0.f : top;
      for (int w = 0; w < kQ8Warps; ++w) {
        const float keep = expf(ml_s[w][0] - ref);
        sum += acc_s[w][threadIdx.x] * keep;
        z += ml_s[w][1] * keep;
      }
      part[threadIdx.x] = sum;
      if (threadIdx.x == 0) {
        part[D] = top;
        part[D + 1] = z;
      }
    }
    __syncthreads();
  }
}

// One block per (unit, query head), a thread per element.
template <int D>
__global__ void q8_join_kernel(Q8AttendParams p) {
  grid_dependency_wait();
  const int G = p.num_q_heads / p.num_kv_heads;
  const int64_t unit = blockIdx.x / G;
  const int g = blockIdx.x % G;
  const float* part = p.part + (unit * p.splits * G + g) * (D + 2);
  const int64_t step = static_cast<int64_t>(G) * (D + 2);
  float top = -INFINITY, sum = 0.f, z = 0.f;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, part[s * step + D]);
  const float ref = top == -INFINITY ? 0.f : top;
  for (int s = 0; s < p.splits; ++s) {
    const float keep = expf(part[s * step + D] - ref);
    sum += part[s * step + threadIdx.x] * keep;
    z += part[s * step + D + 1] * keep;
  }
  const int64_t b = unit / p.num_kv_heads, h = unit % p.num_kv_heads;
  p.out[(b * p.num_q_heads + h * G + g) * D + threadIdx.x] = z == 0.f ? 0.f : sum / z;
}

template <bool BF16, int C, int D>
cudaError_t launch_typed(const Q8AttendParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.splits, p.num_kv_heads, p.batch);
  cfg.blockDim = dim3(kQ8Threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, q8_attend_kernel<BF16, C, D>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch * static_cast<int64_t>(p.num_q_heads)));
  cfg.blockDim = dim3(D);
  return cudaLaunchKernelEx(&cfg, q8_join_kernel<D>, p);
}

template <int C>
cudaError_t launch_code(const Q8AttendParams& p, int d, bool bf16, cudaStream_t stream) {
  if (bf16) return d == 128 ? launch_typed<true, C, 128>(p, stream) : launch_typed<true, C, 64>(p, stream);
  return d == 128 ? launch_typed<false, C, 128>(p, stream) : launch_typed<false, C, 64>(p, stream);
}

}  // namespace

int q8_attend_splits(int64_t units, int64_t max_tokens, int sms) {
  const int64_t want = (4ll * sms + units - 1) / units, most = (max_tokens + 63) / 64;
  return static_cast<int>(std::max<int64_t>(1, std::min(want, most)));
}

cudaError_t launch_q8_attend(const Q8AttendParams& p, int head_dim, bool bf16, int code,
                             cudaStream_t stream) {
  return code == kCodeI8 ? launch_code<kCodeI8>(p, head_dim, bf16, stream)
                         : launch_code<kCodeE4M3>(p, head_dim, bf16, stream);
}

}  // namespace santa
