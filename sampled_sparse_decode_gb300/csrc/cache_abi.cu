// cache_abi.cu — the C entry points of the prompt side of the cache and of the deterministic
// sparse step: argument checks, workspace layout and launches.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kernels.h"

namespace {

constexpr int kMaxTeams = 16384;
constexpr int kMaxDraws = 4096;
constexpr int kMaxRopeDim = 128;
constexpr int64_t kMaxTokens = int64_t(1) << 24;    // tokens of one chunk call
constexpr size_t kAlign = 256;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int map_cuda(cudaError_t e) { return e == cudaSuccess ? SANTA_OK : SANTA_ERR_CUDA; }

int check_cache_shape(int dtype, int batch, int hkv, int d, int T, int max_teams) {
  if (dtype != SANTA_F32 && dtype != SANTA_BF16) return SANTA_ERR_UNSUPPORTED;
  if (batch < 1 || hkv < 1 || max_teams < 1) return SANTA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SANTA_ERR_UNSUPPORTED;
  if (T != 64 && T != 128) return SANTA_ERR_UNSUPPORTED;
  if (max_teams > kMaxTeams || batch > 65535 || hkv > 65535) return SANTA_ERR_UNSUPPORTED;
  return SANTA_OK;
}
int check_heads(int hq, int hkv) {
  if (hq < 1 || hq % hkv != 0) return SANTA_ERR_INVALID_ARG;
  return hq / hkv > santa::kMaxGroup ? SANTA_ERR_UNSUPPORTED : SANTA_OK;
}
int check_tokens(int64_t num_tokens) {
  if (num_tokens < 0) return SANTA_ERR_INVALID_ARG;
  return num_tokens > kMaxTokens ? SANTA_ERR_UNSUPPORTED : SANTA_OK;
}
// Whether [a, a + bytes) meets one of the `rows` rows of row_bytes that lie stride_bytes
// (>= row_bytes) apart from b on.
bool meets(const void* a, int64_t bytes, const void* b, int64_t rows, int64_t row_bytes,
           int64_t stride_bytes) {
  if (!a || !b || bytes <= 0 || rows <= 0 || row_bytes <= 0) return false;
  const __int128 lo = reinterpret_cast<uintptr_t>(a), at = reinterpret_cast<uintptr_t>(b);
  // the first row that ends behind lo
  const __int128 r = at + row_bytes > lo ? 0 : (lo - at - row_bytes) / stride_bytes + 1;
  return r < rows && at + r * stride_bytes < lo + bytes;
}

// Workspace of a chunk attention: bf16 has one of its own; fp32 keeps the partial results of
// its split tiles, accumulators, then (m, l).
struct ChunkLayout {
  int splits, sms;
  size_t acc_bytes, bytes;
};
int chunk_layout(int dtype, int batch, int64_t num_tokens, int hq, int hkv, int d, int T,
                 int max_teams, ChunkLayout* l) {
  const int sms = santa::device_sms();
  if (sms <= 0) return SANTA_ERR_CUDA;
  l->sms = sms;
  if (dtype == SANTA_BF16) {
    l->splits = 1;
    l->acc_bytes = 0;
    l->bytes = kAlign + santa::chunk_tc_workspace(num_tokens, batch, hq / hkv, hkv, d,
                                                  static_cast<int64_t>(max_teams) * T, sms);
    return SANTA_OK;
  }
  const int64_t tiles = santa::chunk_simt_tiles(num_tokens, batch, hq / hkv, hkv);
  l->splits = santa::chunk_simt_splits(tiles, static_cast<int64_t>(max_teams) * T, sms);
  const size_t rows = l->splits > 1 ? static_cast<size_t>(tiles) * l->splits * 64 : 0;
  l->acc_bytes = round_up(rows * d * sizeof(float), kAlign);
  l->bytes = kAlign + l->acc_bytes + round_up(rows * 2 * sizeof(float), kAlign);
  return SANTA_OK;
}

int check_chunk_shape(int dtype, int batch, int64_t num_tokens, int hq, int hkv, int d, int T,
                      int max_teams) {
  int rc = check_cache_shape(dtype, batch, hkv, d, T, max_teams);
  if (rc || (rc = check_heads(hq, hkv)) || (rc = check_tokens(num_tokens))) return rc;
  return SANTA_OK;
}

}  // namespace

#pragma GCC visibility push(default)
extern "C" {

int santa_rope_table(float* table, int64_t positions, int rope_dim, double theta,
                     void* stream) {
  if (!table || !aligned(table, 16) || positions < 1) return SANTA_ERR_INVALID_ARG;
  if (!(theta > 1.0) || !std::isfinite(theta)) return SANTA_ERR_INVALID_ARG;
  if (rope_dim < 16 || rope_dim > kMaxRopeDim || rope_dim % 16) return SANTA_ERR_UNSUPPORTED;
  if (positions > 0x7fffffffll) return SANTA_ERR_UNSUPPORTED;
  return map_cuda(santa::launch_rope_table(table, positions, rope_dim, theta,
                                           static_cast<cudaStream_t>(stream)));
}

int santa_append_chunk(const santa_append_chunk_args* a, void* stream) {
  if (!a) return SANTA_ERR_INVALID_ARG;
  int rc = check_cache_shape(a->dtype, a->batch, a->num_kv_heads, a->head_dim, a->team_size,
                             a->max_teams);
  if (rc || (rc = check_tokens(a->num_tokens))) return rc;
  if (a->num_pages < 1 || (!a->q) != (!a->q_out)) return SANTA_ERR_INVALID_ARG;
  if (a->q && a->num_q_heads < 1) return SANTA_ERR_INVALID_ARG;
  if (a->q && a->num_q_heads > 65535) return SANTA_ERR_UNSUPPORTED;
  if (a->rope_dim < 0 || a->rope_dim > a->head_dim || a->rope_dim % 16)
    return SANTA_ERR_UNSUPPORTED;
  if (a->rope_dim && (!a->rope || !aligned(a->rope, 16) || a->rope_positions < 1))
    return SANTA_ERR_INVALID_ARG;
  const bool bf16 = a->dtype == SANTA_BF16;
  const int vec = bf16 ? 8 : 4;                         // elements per 16 bytes
  const int64_t kv_row = static_cast<int64_t>(a->num_kv_heads) * a->head_dim;
  const int64_t q_row = static_cast<int64_t>(a->num_q_heads) * a->head_dim;
  if (a->num_tokens) {
    if (!a->k_new || !a->v_new) return SANTA_ERR_INVALID_ARG;
    if (a->k_stride < kv_row || a->v_stride < kv_row || a->k_stride % vec || a->v_stride % vec)
      return SANTA_ERR_INVALID_ARG;
    if (a->q && (a->q_stride < q_row || a->q_stride % vec)) return SANTA_ERR_INVALID_ARG;
    // in place only row for row
    if (a->q && a->q == a->q_out && a->q_stride != q_row) return SANTA_ERR_INVALID_ARG;
  }
  if (!a->cu_q || !a->page_table || !a->seq_lens || !a->k_pool || !a->v_pool || !a->reps)
    return SANTA_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || !aligned(a->k_new, 16) || !aligned(a->v_new, 16) ||
      !aligned(a->q_out, 16) || !aligned(a->k_pool, 16) || !aligned(a->v_pool, 16) ||
      !aligned(a->reps, 16) || !aligned(a->cu_q, 4) || !aligned(a->page_table, 4) ||
      !aligned(a->seq_lens, 4) || !aligned(a->seq_lens_next, 4) || !aligned(a->device_status, 4))
    return SANTA_ERR_INVALID_ARG;
  if (santa::append_chunk_blocks(a->num_tokens, a->batch, a->q ? a->num_q_heads : 0,
                                 a->num_kv_heads, a->head_dim, a->team_size, bf16) > 0x7fffffffll)
    return SANTA_ERR_UNSUPPORTED;
  // what is written while other blocks still read: rotated queries over the new rows (but for a
  // rotation in place), new lengths over the batch's lengths and bounds
  const int64_t es = bf16 ? 2 : 4, n = a->num_tokens, len_bytes = int64_t(a->batch) * 4;
  const int64_t q_bytes = a->q ? n * q_row * es : 0;
  if ((a->q_out != a->q && meets(a->q_out, q_bytes, a->q, n, q_row * es, a->q_stride * es)) ||
      meets(a->q_out, q_bytes, a->k_new, n, kv_row * es, a->k_stride * es) ||
      meets(a->q_out, q_bytes, a->v_new, n, kv_row * es, a->v_stride * es) ||
      meets(a->seq_lens_next, len_bytes, a->seq_lens, 1, len_bytes, len_bytes) ||
      meets(a->seq_lens_next, len_bytes, a->cu_q, 1, len_bytes + 4, len_bytes + 4))
    return SANTA_ERR_INVALID_ARG;
  santa::AppendChunkParams p = {};
  p.q = a->q;
  p.k_new = a->k_new;
  p.v_new = a->v_new;
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.cu_q = a->cu_q;
  p.page_table = a->page_table;
  p.seq_lens = a->seq_lens;
  p.rope = a->rope;
  p.rope_positions = a->rope_positions;
  p.num_tokens = a->num_tokens;
  p.num_pages = a->num_pages;
  p.batch = a->batch;
  p.num_q_heads = a->num_q_heads;
  p.num_kv_heads = a->num_kv_heads;
  p.team_size = a->team_size;
  p.max_teams = a->max_teams;
  p.rope_dim = a->rope_dim;
  p.interleaved = a->interleaved != 0;
  p.q_out = a->q_out;
  p.k_pool = a->k_pool;
  p.v_pool = a->v_pool;
  p.reps = a->reps;
  p.seq_lens_next = a->seq_lens_next;
  p.status = a->device_status;
  return map_cuda(santa::launch_append_chunk(p, a->head_dim, bf16,
                                             static_cast<cudaStream_t>(stream)));
}

size_t santa_chunk_workspace_bytes(int dtype, int batch, int64_t num_tokens, int num_q_heads,
                                   int num_kv_heads, int head_dim, int team_size,
                                   int max_teams) {
  if (check_chunk_shape(dtype, batch, num_tokens, num_q_heads, num_kv_heads, head_dim,
                        team_size, max_teams))
    return 0;
  ChunkLayout l;
  return chunk_layout(dtype, batch, num_tokens, num_q_heads, num_kv_heads, head_dim, team_size,
                      max_teams, &l)
             ? 0
             : l.bytes;
}

int santa_chunk_attend(const santa_chunk_args* a, void* stream) {
  if (!a) return SANTA_ERR_INVALID_ARG;
  int rc = check_chunk_shape(a->dtype, a->batch, a->num_tokens, a->num_q_heads, a->num_kv_heads,
                             a->head_dim, a->team_size, a->max_teams);
  if (rc) return rc;
  if (a->num_pages < 1 || !a->k_pool || !a->v_pool || !a->page_table || !a->seq_lens || !a->cu_q)
    return SANTA_ERR_INVALID_ARG;
  if (a->num_tokens && (!a->q || !a->out)) return SANTA_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->k_pool, 16) ||
      !aligned(a->v_pool, 16) || !aligned(a->page_table, 4) || !aligned(a->seq_lens, 4) ||
      !aligned(a->cu_q, 4) || !aligned(a->device_status, 4))
    return SANTA_ERR_INVALID_ARG;
  if (a->num_tokens == 0) return SANTA_OK;
  // queries are read again after rows of `out` are written
  const int64_t row = static_cast<int64_t>(a->num_q_heads) * a->head_dim *
                      (a->dtype == SANTA_BF16 ? 2 : 4);
  if (meets(a->out, a->num_tokens * row, a->q, a->num_tokens, row, row))
    return SANTA_ERR_INVALID_ARG;
  ChunkLayout l;
  if ((rc = chunk_layout(a->dtype, a->batch, a->num_tokens, a->num_q_heads, a->num_kv_heads,
                         a->head_dim, a->team_size, a->max_teams, &l)))
    return rc;
  if (!a->workspace || a->workspace_bytes < l.bytes) return SANTA_ERR_INVALID_ARG;
  unsigned char* base = reinterpret_cast<unsigned char*>(
      round_up(reinterpret_cast<uintptr_t>(a->workspace), kAlign));
  santa::ChunkParams p = {};
  p.q = a->q;
  p.k_pool = a->k_pool;
  p.v_pool = a->v_pool;
  p.page_table = a->page_table;
  p.seq_lens = a->seq_lens;
  p.cu_q = a->cu_q;
  p.num_tokens = a->num_tokens;
  p.num_pages = a->num_pages;
  p.batch = a->batch;
  p.num_q_heads = a->num_q_heads;
  p.num_kv_heads = a->num_kv_heads;
  p.team_size = a->team_size;
  p.max_teams = a->max_teams;
  p.scale_log2 =
      static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a->head_dim)));
  p.out = a->out;
  p.status = a->device_status;
  if (a->dtype == SANTA_BF16)
    return santa::launch_chunk_tc(p, a->head_dim, base, l.sms, static_cast<cudaStream_t>(stream));
  return map_cuda(santa::launch_chunk_simt(p, a->head_dim, l.splits,
                                           reinterpret_cast<float*>(base),
                                           reinterpret_cast<float*>(base + l.acc_bytes),
                                           static_cast<cudaStream_t>(stream)));
}

int santa_select_topk(const santa_decode_args* a, void* stream) {
  if (!a) return SANTA_ERR_INVALID_ARG;
  int rc = check_cache_shape(a->dtype, a->batch, a->num_kv_heads, a->head_dim, a->team_size,
                             a->max_teams);
  if (rc || (rc = check_heads(a->num_q_heads, a->num_kv_heads))) return rc;
  if (a->num_draws < 1 || a->num_draws > kMaxDraws) return SANTA_ERR_UNSUPPORTED;
  if (a->num_pages < 1 || !a->q || !a->reps || !a->page_table || !a->seq_lens || !a->sel_ids ||
      !a->sel_count || !a->pi)
    return SANTA_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || !aligned(a->reps, 16) || !aligned(a->page_table, 4) ||
      !aligned(a->seq_lens, 4) || !aligned(a->sel_ids, 4) || !aligned(a->sel_count, 4) ||
      !aligned(a->pi, 4) || !aligned(a->device_status, 4))
    return SANTA_ERR_INVALID_ARG;
  const int sms = santa::device_sms();
  if (sms <= 0) return SANTA_ERR_CUDA;
  santa::SelectParams p = {};
  p.q = a->q;
  p.reps = a->reps;
  p.page_table = a->page_table;
  p.seq_lens = a->seq_lens;
  p.bf16 = a->dtype == SANTA_BF16;
  p.batch = a->batch;
  p.num_q_heads = a->num_q_heads;
  p.num_kv_heads = a->num_kv_heads;
  p.team_size = a->team_size;
  p.max_teams = a->max_teams;
  p.keep = a->num_draws;
  p.num_pages = a->num_pages;
  p.sel_ids = a->sel_ids;
  p.sel_count = a->sel_count;
  p.pi = a->pi;
  p.status = a->device_status;
  return map_cuda(
      santa::launch_select_topk(p, a->head_dim, sms, static_cast<cudaStream_t>(stream)));
}

int santa_topk_decode(const santa_decode_args* a, void* stream) {
  if (!a) return SANTA_ERR_INVALID_ARG;
  // everything the attention refuses is refused before the selection is launched
  santa_decode_args b = *a;
  b.sampler = SANTA_SAMPLER_IID_HT;
  b.mix_alpha = 0.f;
  int rc = santa::check_attend(&b);
  if (rc || (rc = santa_select_topk(&b, stream))) return rc;
  return santa::attend_full_weights(&b, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
#pragma GCC visibility pop
