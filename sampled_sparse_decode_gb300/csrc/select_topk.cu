// select_topk.cu — the M teams of best representative score, for every unit (sequence, KV head).
//
// One cluster per unit.  Each CTA scores a slice of the unit's teams in fp32 (16 lanes per
// team, the group's queries in registers) and stores the scores in the first CTA's shared
// memory; the first CTA then finds the border of the best M and writes S.
//
// Exactness.  S is the set that 64-bit scores give.  An fp32 score of d <= 128 products, 8 per
// lane and 16 lanes joined by a tree, is off by at most E = 16 * 2^-24 * |q||rep|: each product
// goes through at most 8 fused steps (8 roundings) and 4 tree sums, 12 roundings of at most
// 2^-24 of a partial sum that Cauchy-Schwarz bounds by |q||rep|; 16 leaves room for the second
// order, the norms' own rounding and denormals.  So with t the M-th best fp32 score, a team
// above t + 2E is in S, one below t - 2E is not, and the few between are compared in 64 bits.
// Only if they do not all fit is any 64-bit score formed (usually the M-th alone lies there).
#include "kernels.h"

namespace santa {

namespace {

constexpr int kSelThreads = 256;
constexpr int kLanes = 16;                                // lanes per team

// Order-preserving map of fp32 to unsigned; NaN and -inf map to the lowest value.
__device__ __forceinline__ uint32_t score_key(float s) {
  if (!(s > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(s + 0.f);            // -0 and 0 are one score
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_score(uint32_t k) {
  if (k == 0u) return -INFINITY;
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ void store_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}

// Exclusive prefix sum over the block's threads, and the total.
__device__ __forceinline__ int block_scan(int v, int* buf, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const int c = buf[w];
    if (w < warp) before += c;
    all += c;
  }
  *total = all;
  return before + x - v;
}

template <bool BF16>
__device__ __forceinline__ float q_at(const void* q, int64_t i) {
  return BF16 ? bf16_to_f32(static_cast<const uint16_t*>(q)[i]) : static_cast<const float*>(q)[i];
}

// 64-bit score of team `page` by one warp (all lanes get it), as an order-preserving key: the
// largest product over the heads; 0 for NaN and -inf.
template <bool BF16, int D>
__device__ uint64_t exact_key(const SelectParams& p, int64_t page, int b, int h, int G) {
  const int lane = threadIdx.x & 31;
  const float* rep = p.reps + (page * p.num_kv_heads + h) * D;
  double best = -INFINITY;
  bool nan = false;
  for (int g = 0; g < G; ++g) {
    const int64_t qi = (static_cast<int64_t>(b) * p.num_q_heads + h * G + g) * D;
    double s = 0.0;
#pragma unroll
    for (int e = lane; e < D; e += 32)
      s += static_cast<double>(q_at<BF16>(p.q, qi + e)) * static_cast<double>(rep[e]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    nan |= s != s;
    best = s > best ? s : best;
  }
  if (nan || best == -INFINITY) return 0u;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(best + 0.0));
  return u >> 63 ? ~u : u | 1ull << 63;
}

// The *left-th largest of the n keys in shared memory, one byte at a time from the top; *left
// becomes its place among the keys equal to it.  All threads get both.
template <typename Key>
__device__ Key kth_largest(const Key* keys, int n, int* left, uint32_t* hist, uint32_t* pick) {
  Key prefix = 0, mask = 0;
  int want = *left;
  for (int shift = 8 * sizeof(Key) - 8; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kSelThreads)
      if ((keys[i] & mask) == prefix)
        atomicAdd(&hist[static_cast<uint32_t>(keys[i] >> shift) & 255u], 1u);
    __syncthreads();
    if (threadIdx.x < 32) {
      // lane l holds the digits 255 - 8 l .. 248 - 8 l: lanes and digits go down together
      int c[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += c[e] = hist[255 - (threadIdx.x * 8 + e)];
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (static_cast<int>(threadIdx.x) >= o) before += y;
      }
      before -= sum;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (before < want && want <= before + c[e]) {
          pick[0] = 255 - (threadIdx.x * 8 + e);
          pick[1] = want - before;
        }
        before += c[e];
      }
    }
    __syncthreads();
    prefix |= static_cast<Key>(pick[0]) << shift;
    mask |= static_cast<Key>(255u) << shift;
    want = pick[1];
  }
  __syncthreads();
  *left = want;
  return prefix;
}

template <bool BF16, int D>
__global__ void __launch_bounds__(kSelThreads) select_kernel(SelectParams p) {
  extern __shared__ __align__(16) uint32_t keys[];        // fp32 keys, then 64-bit keys (CTA 0)
  __shared__ float q_s[kMaxGroup * D];
  __shared__ int buf[kSelThreads / 32];
  __shared__ uint32_t norm_max;                           // bits of max |rep|^2 (CTA 0)
  __shared__ uint32_t hist[256];
  __shared__ uint32_t pick[2];                            // digit and what is left
  constexpr int kPer = D / kLanes;                        // elements per lane (8 or 4)
  const int G = p.num_q_heads / p.num_kv_heads;
  const int rank = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int CL = gridDim.x;
  const int64_t unit = static_cast<int64_t>(b) * p.num_kv_heads + h;
  if (threadIdx.x == 0) norm_max = 0u;
  grid_dependency_wait();
  const int64_t len = p.seq_lens[b];
  const bool ok = len >= 1 && len <= static_cast<int64_t>(p.max_teams) * p.team_size;
  const int n = ok ? static_cast<int>((len + p.team_size - 1) / p.team_size) : 0;
  // the unit's group of queries, zero beyond it (heads of a group of less than 8)
  for (int i = threadIdx.x; i < kMaxGroup * D; i += kSelThreads) {
    const int g = i / D;
    q_s[i] = g < G ? q_at<BF16>(p.q, (static_cast<int64_t>(b) * p.num_q_heads + h * G) * D + i)
                   : 0.f;
  }
  if (CL > 1) cluster_sync(); else __syncthreads();

  // ---- scores of this CTA's slice of the teams
  {
    const int lane = threadIdx.x % kLanes, team_lane = threadIdx.x / kLanes;
    float q[kMaxGroup][kPer];
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g)
#pragma unroll
      for (int e = 0; e < kPer; e += 4) {
        const float4 v = *reinterpret_cast<const float4*>(
            q_s + g * D + (e / 4) * (4 * kLanes) + lane * 4);
        q[g][e] = v.x; q[g][e + 1] = v.y; q[g][e + 2] = v.z; q[g][e + 3] = v.w;
      }
    const uint32_t keys0 = cluster_addr(smem_u32(keys), 0);
    const int per = (n + CL - 1) / CL;
    const int lo = rank * per, hi = min(n, lo + per);
    uint32_t norm = 0u;
    // whole warps stay together for the shuffles
    for (int base = lo; base < hi; base += kSelThreads / kLanes) {
      const int team = base + team_lane;
      int64_t page = -1;
      if (team < hi) {
        page = p.page_table[static_cast<int64_t>(b) * p.max_teams + team];
        if (page < 0 || page >= p.num_pages) {
          if (lane == 0) set_status(p.status, SANTA_DEV_BAD_PAGE);
          page = -1;
        }
      }
      float s[kMaxGroup], nn = 0.f;
#pragma unroll
      for (int g = 0; g < kMaxGroup; ++g) s[g] = 0.f;
      if (page >= 0) {
        const float4* rep =
            reinterpret_cast<const float4*>(p.reps + (page * p.num_kv_heads + h) * D);
#pragma unroll
        for (int e = 0; e < kPer; e += 4) {
          const float4 r = __ldg(rep + (e / 4) * kLanes + lane);
          nn = fmaf(r.x, r.x, fmaf(r.y, r.y, fmaf(r.z, r.z, fmaf(r.w, r.w, nn))));
#pragma unroll
          for (int g = 0; g < kMaxGroup; ++g)
            s[g] = fmaf(q[g][e], r.x, fmaf(q[g][e + 1], r.y,
                   fmaf(q[g][e + 2], r.z, fmaf(q[g][e + 3], r.w, s[g]))));
        }
      }
      // sums over the 16 lanes: each step halves the heads a lane keeps (8, 4, 2, 1)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const bool up = lane & 8;
        const float other = __shfl_xor_sync(0xffffffffu, up ? s[g] : s[g + 4], 8);
        s[g] = (up ? s[g + 4] : s[g]) + other;
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const bool up = lane & 4;
        const float other = __shfl_xor_sync(0xffffffffu, up ? s[g] : s[g + 2], 4);
        s[g] = (up ? s[g + 2] : s[g]) + other;
      }
      {
        const bool up = lane & 2;
        const float other = __shfl_xor_sync(0xffffffffu, up ? s[0] : s[1], 2);
        s[0] = (up ? s[1] : s[0]) + other;
      }
      s[0] += __shfl_xor_sync(0xffffffffu, s[0], 1);
      // lane holds head (lane & 8 ? 4 : 0) + (lane & 4 ? 2 : 0) + (lane & 2 ? 1 : 0)
      const int head = ((lane >> 3) & 1) * 4 + ((lane >> 2) & 1) * 2 + ((lane >> 1) & 1);
      bool nan = head < G && s[0] != s[0];
      float best = head < G ? s[0] : -INFINITY;
#pragma unroll
      for (int o = 2; o < kLanes; o <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
      const unsigned nans = __ballot_sync(0xffffffffu, nan);
      nan = (nans >> (threadIdx.x & 16)) & 0xffffu;
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) nn += __shfl_xor_sync(0xffffffffu, nn, o);
      if (team < hi && lane == 0)
        store_cluster_u32(keys0 + team * 4, page < 0 || nan ? 0u : score_key(best));
      // bits of non-negative values order like the values; inf and NaN come out on top
      if (page >= 0) norm = max(norm, __float_as_uint(nn) & 0x7fffffffu);
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, norm);
    if ((threadIdx.x & 31) == 0) {
      const uint32_t at = cluster_addr(smem_u32(&norm_max), 0);
      asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(at), "r"(top)
                   : "memory");
    }
  }
  if (CL > 1) cluster_sync(); else __syncthreads();
  if (rank != 0) return;

  // ---- the first CTA: the border of the best `keep`
  const int keep = min(p.keep, n);
  int32_t* ids = p.sel_ids + unit * p.keep;
  float* pi = p.pi + unit * p.keep;
  if (threadIdx.x == 0) {
    p.sel_count[unit] = keep;
    if (!ok) set_status(p.status, SANTA_DEV_BAD_SEQLEN);
  }
  for (int i = keep + threadIdx.x; i < p.keep; i += kSelThreads) {
    ids[i] = -1;
    pi[i] = 0.f;
  }
  if (n <= p.keep) {
    for (int i = threadIdx.x; i < n; i += kSelThreads) {
      ids[i] = i;
      pi[i] = 1.f;
    }
    return;
  }
  int left = keep;
  const uint32_t border = kth_largest<uint32_t>(keys, n, &left, hist, pick);

  // ---- teams too close to the border for fp32 (see the top of the file); the norms are kept
  // away from zero so that products in the denormal range stay inside the bound
  const float t = key_score(border);
  uint32_t qn = 0u;
  for (int g = 0; g < G; ++g) {
    float s = 0.f;
    for (int e = threadIdx.x & 31; e < D; e += 32) s = fmaf(q_s[g * D + e], q_s[g * D + e], s);
    qn = max(qn, __float_as_uint(warp_sum(s)) & 0x7fffffffu);
  }
  const uint32_t tiny = 0x00800000u;                      // the smallest normal fp32
  const float err = 16.f * 0x1p-24f * sqrtf(__uint_as_float(max(qn, tiny))) *
                        sqrtf(__uint_as_float(max(norm_max, tiny))) + 0x1p-140f;
  // an infinite or NaN bound (or a border of -inf) leaves every team to the 64-bit scores
  const bool finite = err < INFINITY && t > -INFINITY;
  const float above = finite ? t + 2.f * err : INFINITY, below = finite ? t - 2.f * err : -INFINITY;
  const int chunk = (n + kSelThreads - 1) / kSelThreads;  // at most 64 (n <= 16384)
  const int i0 = min(n, static_cast<int>(threadIdx.x) * chunk), i1 = min(n, i0 + chunk);
  uint64_t in = 0u, near = 0u;
  for (int i = i0; i < i1; ++i) {
    const float s = key_score(keys[i]);
    if (s > above)
      in |= 1ull << (i - i0);
    else if (s >= below)
      near |= 1ull << (i - i0);
  }
  int sure, near_total;
  block_scan(__popcll(in), buf, &sure);
  const int near_at = block_scan(__popcll(near), buf, &near_total);
  int want = keep - sure;
  if (near_total > want) {
    // the near teams' indices (over the fp32 keys, which are no longer needed) and 64-bit keys
    uint64_t* exact = reinterpret_cast<uint64_t*>(keys + (p.max_teams + 3) / 4 * 4);
    int at = near_at;
    for (uint64_t m = near; m; m &= m - 1) keys[at++] = i0 + __ffsll(m) - 1;
    __syncthreads();
    for (int i = threadIdx.x / 32; i < near_total; i += kSelThreads / 32) {
      const int64_t page = p.page_table[static_cast<int64_t>(b) * p.max_teams + keys[i]];
      const uint64_t k = page < 0 || page >= p.num_pages
                             ? 0u
                             : exact_key<BF16, D>(p, page, b, h, G);
      if ((threadIdx.x & 31) == 0) exact[i] = k;
    }
    __syncthreads();
    // the best `want` of them; `want` becomes how many of those at the border are taken, and
    // the list is in team order, so ties go to the lower index
    const uint64_t last = kth_largest<uint64_t>(exact, near_total, &want, hist, pick);
    int ties = 0, all;
    for (int i = 0, e = near_at; i < __popcll(near); ++i, ++e) ties += exact[e] == last;
    int tie_at = block_scan(ties, buf, &all);
    at = near_at;
    for (uint64_t m = near; m; m &= m - 1, ++at)
      if (exact[at] > last || (exact[at] == last && tie_at++ < want)) in |= m & -m;
  } else {
    in |= near;
  }
  int total;
  int at = block_scan(__popcll(in), buf, &total);
  for (; in; in &= in - 1) {
    ids[at] = i0 + __ffsll(in) - 1;
    pi[at++] = 1.f;
  }
}

template <bool BF16, int D>
cudaError_t launch(const SelectParams& params, int sms, cudaStream_t stream) {
  const SelectParams& p = params;
  const int64_t units = static_cast<int64_t>(p.batch) * p.num_kv_heads;
  // as many CTAs per unit as fill the device twice over, at least 32 teams (two for each
  // 16-lane group of a block) each
  int cl = 1;
  while (cl < 8 && units * cl * 2 <= 2 * sms && p.max_teams > cl * 32) cl *= 2;
  const size_t up = static_cast<size_t>(p.max_teams + 3) / 4 * 4;
  const size_t smem = up * (4 + 8);           // fp32 keys, 64-bit keys of the near teams
  static std::atomic<unsigned long long> done{0};
  constexpr size_t kMost = 16384 * 12;        // max_teams <= 16384
  cudaError_t e = ensure_dynamic_smem(select_kernel<BF16, D>, kMost, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cl, p.num_kv_heads, p.batch);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_kernel<BF16, D>, p);
}

}  // namespace

cudaError_t launch_select_topk(const SelectParams& p, int head_dim, int sms,
                               cudaStream_t stream) {
  if (p.bf16)
    return head_dim == 128 ? launch<true, 128>(p, sms, stream) : launch<true, 64>(p, sms, stream);
  return head_dim == 128 ? launch<false, 128>(p, sms, stream) : launch<false, 64>(p, sms, stream);
}

}  // namespace santa
