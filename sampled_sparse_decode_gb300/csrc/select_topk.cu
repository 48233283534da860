// select_topk.cu — the M teams of best representative score, for every unit (sequence, KV head).
//
// One cluster per unit.  Each CTA scores some of the unit's teams in fp32 (16 lanes per
// team, two teams at a time) and stores the scores in the first CTA's shared memory; the first
// CTA then finds the border of the best M and writes S.
//
// Exactness.  S is the set that 64-bit scores give.  An fp32 score of d <= 128 products, 8 per
// lane and 16 lanes joined by a tree, is off by at most E = 16 * 2^-24 * |q||rep|: each product
// goes through at most 8 fused steps (8 roundings) and 4 tree sums, 12 roundings of at most
// 2^-24 of a partial sum that Cauchy-Schwarz bounds by |q||rep|; 16 leaves room for the second
// order, the norms' own rounding and denormals.  So with t the M-th best fp32 score, a team
// above t + 2E is in S, one below t - 2E is not, and the few between are compared in 64 bits.
// Only if they do not all fit is any 64-bit score formed (usually the M-th alone lies there).
//
// Bound by latency: a launch makes two dependent reads from DRAM or L2 (the length with the
// page ids, then the representatives), two cluster barriers and two counting passes.  Measured
// on GB300 (d = 128): 5.3 us for 4 units of 256 teams, 9.0 us for 128 units of 256 (16.8 MB of
// representatives), 9.8 us for 16 units of 1024.
#include "kernels.h"

namespace santa {

namespace {

constexpr int kSelThreads = 256;
constexpr int kLanes = 16;                                // lanes per team

// Order-preserving map of fp32 to unsigned: NaN maps to 0 (as a bad page does), -inf to the value
// above it that any score has.
__device__ __forceinline__ uint32_t score_key(float s) {
  if (s != s) return 0u;
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
// The two halves of a cluster barrier, by every thread of every CTA of the cluster.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_acquire() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct SelShared {
  unsigned long long low[256], high[256];                 // keys of a digit
  uint32_t hist[256];
  int pick[2];                                            // digit, place within it
  int scan[kSelThreads / 32];
  uint32_t top[kSelThreads / 32];
  uint32_t norm_q, norm_rep;                              // bits of the largest |q|^2, |rep|^2
};

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
// largest product over the heads; 0 for NaN.
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
  if (nan) return 0u;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(best + 0.0));
  return u >> 63 ? ~u : u | 1ull << 63;
}

// One counting pass over the keys in [lo, hi] of the n in shared memory, digit(key) a monotone
// map to 0 .. 255: the digit that holds the *want-th largest of them becomes the new [lo, hi]
// (the smallest and largest key in it), *want the place within it.
template <typename Key, typename Digit>
__device__ __forceinline__ void narrow(const Key* keys, int n, Key& lo, Key& hi, int& want,
                                       SelShared& s, Digit digit) {
  Key* low = reinterpret_cast<Key*>(s.low);
  Key* high = reinterpret_cast<Key*>(s.high);
  for (int i = threadIdx.x; i < 256; i += kSelThreads) {
    s.hist[i] = 0u;
    low[i] = ~static_cast<Key>(0);
    high[i] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kSelThreads) {
    const Key k = keys[i];
    if (k >= lo && k <= hi) {
      const uint32_t d = digit(k);
      atomicAdd(&s.hist[d], 1u);
      atomicMin(&low[d], k);
      atomicMax(&high[d], k);
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    // lane l holds the digits 255 - 8 l .. 248 - 8 l: lanes and digits go down together
    int c[8], sum = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += c[e] = s.hist[255 - (threadIdx.x * 8 + e)];
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
        s.pick[0] = 255 - (threadIdx.x * 8 + e);
        s.pick[1] = want - before;
      }
      before += c[e];
    }
  }
  __syncthreads();
  lo = low[s.pick[0]];
  hi = high[s.pick[0]];
  want = s.pick[1];
  __syncthreads();
}

// The *left-th largest of the n keys; *left becomes its place among the keys equal to it.  All
// threads get both.  The first pass over fp32 scores takes equal parts of their range (leading
// bits would put nearly all scores, which share sign and exponent, into a few counters); the
// passes after it take 8 bits from the highest in which the remaining keys differ, so at most
// sizeof(Key) of them.  Two passes in all for most sets of scores.
template <typename Key>
__device__ Key kth_largest(const Key* keys, int n, int* left, SelShared& s) {
  Key lo = 0, hi = ~static_cast<Key>(0);
  if constexpr (sizeof(Key) == 4) {
    lo = ~static_cast<Key>(0);
    hi = 0;
    for (int i = threadIdx.x; i < n; i += kSelThreads) {
      lo = min(lo, keys[i]);
      hi = max(hi, keys[i]);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if ((threadIdx.x & 31) == 0) {
      s.scan[threadIdx.x / 32] = static_cast<int>(lo);
      s.top[threadIdx.x / 32] = hi;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) {
      lo = min(lo, static_cast<Key>(s.scan[w]));
      hi = max(hi, s.top[w]);
    }
    const float from = key_score(lo), per = 255.f / (key_score(hi) - from);
    // not for infinite scores, nor a range that is empty or overflows
    if (lo < hi && from > -INFINITY && per > 0.f && per < INFINITY)
      narrow(keys, n, lo, hi, *left, s, [&](Key k) {
        return static_cast<uint32_t>(fminf((key_score(k) - from) * per, 255.f));
      });
  }
  while (lo != hi) {
    const int top = 64 - __clzll(static_cast<unsigned long long>(lo ^ hi));
    const int shift = top > 8 ? top - 8 : 0;
    narrow(keys, n, lo, hi, *left, s, [&](Key k) {
      return static_cast<uint32_t>(k >> shift) & ((1u << (top - shift)) - 1u);
    });
  }
  return hi;
}

template <bool BF16, int D>
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(SelectParams p) {
  extern __shared__ __align__(16) uint32_t keys[];        // fp32 keys, then 64-bit keys (CTA 0)
  __shared__ __align__(16) float q_s[kMaxGroup * D];
  __shared__ SelShared s;
  constexpr int kQuads = D / (4 * kLanes);                // float4 pieces per lane (2 or 1)
  constexpr int kTeams = 2;                               // teams per 16 lanes in a round
  constexpr int kRound = kSelThreads / kLanes * kTeams;   // teams per CTA in a round
  const int G = p.num_q_heads / p.num_kv_heads;
  const int rank = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int CL = gridDim.x;
  const int64_t unit = static_cast<int64_t>(b) * p.num_kv_heads + h;
  if (threadIdx.x == 0) s.norm_q = s.norm_rep = 0u;
  cluster_arrive();                                       // waited for before the first store
  grid_dependency_wait();
  grid_launch_dependents();
  // Rounds of 32 teams are dealt out to the CTAs in turn, so which teams a thread scores does not
  // depend on the length, and the first page ids are on their way together with it and the
  // queries (each is a read from DRAM when the cache is larger than L2).
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  // plain loads: the launch before this one may have written the table and the representatives
  // while this one was resident, so they are no read-only data to it
  const int32_t* table = p.page_table + static_cast<int64_t>(b) * p.max_teams;
  auto load_ids = [&](int base, int(&to)[kTeams]) {
#pragma unroll
    for (int u = 0; u < kTeams; ++u) {
      const int team = base + u * (kSelThreads / kLanes) + group;
      to[u] = team < p.max_teams ? table[team] : -1;
    }
  };
  int page[kTeams], page_next[kTeams];
  load_ids(rank * kRound, page);
  load_ids((rank + CL) * kRound, page_next);
  const int64_t len = p.seq_lens[b];
  // the unit's group of queries, zero beyond it
  for (int i = threadIdx.x; i < kMaxGroup * D; i += kSelThreads)
    q_s[i] = i < G * D ? q_at<BF16>(p.q, (static_cast<int64_t>(b) * p.num_q_heads + h * G) * D + i)
                       : 0.f;
  const bool ok = len >= 1 && len <= static_cast<int64_t>(p.max_teams) * p.team_size;
  const int n = ok ? static_cast<int>((len + p.team_size - 1) / p.team_size) : 0;

  // ---- scores of this CTA's teams
  {
    const uint32_t keys0 = cluster_addr(smem_u32(keys), 0);
    uint32_t norm = 0u;
    bool waited = false;
    float4 r[kTeams][kQuads], r_next[kTeams][kQuads];
    // representatives of a round; a team behind the end or with a bad page id scores nothing (the
    // ids are judged first: a status write between the loads would hold the later ones back)
    auto load_reps = [&](int base, int(&from)[kTeams], float4(&to)[kTeams][kQuads]) {
#pragma unroll
      for (int u = 0; u < kTeams; ++u) {
        const int team = base + u * (kSelThreads / kLanes) + group;
        if (team >= n) {
          from[u] = -1;
        } else if (from[u] < 0 || from[u] >= p.num_pages) {
          if (lane == 0) set_status(p.status, SANTA_DEV_BAD_PAGE);
          from[u] = -1;
        }
      }
#pragma unroll
      for (int u = 0; u < kTeams; ++u) {
        const float4* rep = reinterpret_cast<const float4*>(
            p.reps + (static_cast<int64_t>(from[u]) * p.num_kv_heads + h) * D);
#pragma unroll
        for (int e = 0; e < kQuads; ++e)
          to[u][e] = from[u] < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : rep[e * kLanes + lane];
      }
    };
    load_reps(rank * kRound, page, r);
    __syncthreads();
    // meanwhile |q|^2, a warp per head
    for (int g = threadIdx.x / 32; g < G; g += kSelThreads / 32) {
      float x = 0.f;
      for (int e = threadIdx.x & 31; e < D; e += 32) x = fmaf(q_s[g * D + e], q_s[g * D + e], x);
      x = warp_sum(x);
      if ((threadIdx.x & 31) == 0) atomicMax(&s.norm_q, __float_as_uint(x) & 0x7fffffffu);
    }
    // whole warps stay together for the shuffles; representatives are loaded one round ahead,
    // page ids two
#pragma unroll 1
    for (int base = rank * kRound; base < n; base += CL * kRound) {
      load_reps(base + CL * kRound, page_next, r_next);
      int page_after[kTeams];
      load_ids(base + 2 * CL * kRound, page_after);
      float a[kTeams][kMaxGroup], nn[kTeams];
#pragma unroll
      for (int u = 0; u < kTeams; ++u) {
        nn[u] = 0.f;
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) a[u][g] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < kQuads; ++e) {
#pragma unroll
        for (int u = 0; u < kTeams; ++u)
          nn[u] = fmaf(r[u][e].x, r[u][e].x, fmaf(r[u][e].y, r[u][e].y,
                  fmaf(r[u][e].z, r[u][e].z, fmaf(r[u][e].w, r[u][e].w, nn[u]))));
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) {
          const float4 q = *reinterpret_cast<const float4*>(q_s + g * D + (e * kLanes + lane) * 4);
#pragma unroll
          for (int u = 0; u < kTeams; ++u)
            a[u][g] = fmaf(q.x, r[u][e].x, fmaf(q.y, r[u][e].y,
                      fmaf(q.z, r[u][e].z, fmaf(q.w, r[u][e].w, a[u][g]))));
        }
      }
      // 16 sums over the 16 lanes, each step halving what a lane keeps: lane l ends with team
      // (l >> 3) & 1 and head l & 7
      const bool b3 = lane & 8, b2 = lane & 4, b1 = lane & 2, b0 = lane & 1;
      float c[8], d[4], f[2];
#pragma unroll
      for (int g = 0; g < 8; ++g)
        c[g] = (b3 ? a[1][g] : a[0][g]) + __shfl_xor_sync(0xffffffffu, b3 ? a[0][g] : a[1][g], 8);
#pragma unroll
      for (int g = 0; g < 4; ++g)
        d[g] = (b2 ? c[g + 4] : c[g]) + __shfl_xor_sync(0xffffffffu, b2 ? c[g] : c[g + 4], 4);
#pragma unroll
      for (int g = 0; g < 2; ++g)
        f[g] = (b1 ? d[g + 2] : d[g]) + __shfl_xor_sync(0xffffffffu, b1 ? d[g] : d[g + 2], 2);
      const float sum = (b0 ? f[1] : f[0]) + __shfl_xor_sync(0xffffffffu, b0 ? f[0] : f[1], 1);
      float n2 = (b3 ? nn[1] : nn[0]) + __shfl_xor_sync(0xffffffffu, b3 ? nn[0] : nn[1], 8);
      float best = (lane & 7) < G ? sum : -INFINITY;
      // a NaN of any of the team's heads: its 8 lanes' bits of the warp's vote
      const unsigned nans = __ballot_sync(0xffffffffu, (lane & 7) < G && sum != sum);
      const bool nan = (nans >> (threadIdx.x & 24)) & 0xffu;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
        n2 += __shfl_xor_sync(0xffffffffu, n2, o);
      }
      // bits of non-negative values order like the values; inf and NaN come out on top
      norm = max(norm, __float_as_uint(n2) & 0x7fffffffu);
      if (!waited) cluster_wait_acquire();                // the first CTA is running
      waited = true;
      const int u = b3 ? 1 : 0, team = base + u * (kSelThreads / kLanes) + group;
      if (team < n && (lane & 7) == 0)
        store_cluster_u32(keys0 + team * 4,
                          (b3 ? page[1] : page[0]) < 0 || nan ? 0u : score_key(best));
#pragma unroll
      for (int i = 0; i < kTeams; ++i) {
        page[i] = page_next[i];
        page_next[i] = page_after[i];
#pragma unroll
        for (int e = 0; e < kQuads; ++e) r[i][e] = r_next[i][e];
      }
    }
    if (!waited) cluster_wait_acquire();
    const uint32_t top = __reduce_max_sync(0xffffffffu, norm);
    if ((threadIdx.x & 31) == 0) {
      const uint32_t at = cluster_addr(smem_u32(&s.norm_rep), 0);
      asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(at), "r"(top)
                   : "memory");
    }
  }
  cluster_arrive();
  cluster_wait_acquire();
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
  const uint32_t border = kth_largest<uint32_t>(keys, n, &left, s);

  // ---- teams too close to the border for fp32 (see the top of the file); the norms are kept
  // away from zero so that products in the denormal range stay inside the bound
  const float t = key_score(border);
  const uint32_t tiny = 0x00800000u;                      // the smallest normal fp32
  const float err = 16.f * 0x1p-24f * sqrtf(__uint_as_float(max(s.norm_q, tiny))) *
                        sqrtf(__uint_as_float(max(s.norm_rep, tiny))) + 0x1p-140f;
  // an infinite or NaN bound (or a border of -inf) leaves every team to the 64-bit scores
  const bool finite = err < INFINITY && t > -INFINITY;
  const float above = finite ? t + 2.f * err : INFINITY, below = finite ? t - 2.f * err : -INFINITY;
  const int chunk = (n + kSelThreads - 1) / kSelThreads;  // at most 64 (n <= 16384)
  const int i0 = min(n, static_cast<int>(threadIdx.x) * chunk), i1 = min(n, i0 + chunk);
  uint64_t in = 0u, near = 0u;
  for (int i = i0; i < i1; ++i) {
    const float x = key_score(keys[i]);
    if (x > above)
      in |= 1ull << (i - i0);
    else if (x >= below)
      near |= 1ull << (i - i0);
  }
  // both counts in one scan (each at most 16384)
  int total;
  const int before = block_scan(__popcll(in) | __popcll(near) << 16, s.scan, &total);
  const int near_at = before >> 16, near_total = total >> 16;
  int out_at = (before & 0xffff) + near_at;               // as if every near team is taken
  int want = keep - (total & 0xffff);
  if (near_total > want) {
    // the near teams' indices (over the fp32 keys, which are no longer needed) and 64-bit keys
    unsigned long long* exact =
        reinterpret_cast<unsigned long long*>(keys + (p.max_teams + 3) / 4 * 4);
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
    const unsigned long long last = kth_largest<unsigned long long>(exact, near_total, &want, s);
    int ties = 0, all;
    for (int i = 0, e = near_at; i < __popcll(near); ++i, ++e) ties += exact[e] == last;
    int tie_at = block_scan(ties, s.scan, &all);
    at = near_at;
    for (uint64_t m = near; m; m &= m - 1, ++at)
      if (exact[at] > last || (exact[at] == last && tie_at++ < want)) in |= m & -m;
    out_at = block_scan(__popcll(in), s.scan, &all);
  } else {
    in |= near;
  }
  for (; in; in &= in - 1) {
    ids[out_at] = i0 + __ffsll(in) - 1;
    pi[out_at++] = 1.f;
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
