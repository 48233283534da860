// cache_abi.cu — the C entry points of the prompt side of the cache and of the deterministic
// sparse step: argument checks, workspace layout and launches.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "abi_checks.h"
#include "q8.cuh"

using namespace santa::abi;

namespace {

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

// What santa_append_chunk and santa_append_norm refuse alike.
int check_append(const santa_append_chunk_args* a) {
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
  return SANTA_OK;
}

// Whether what santa_append_norm writes overlaps anything else that it writes or reads (queries rotated in
// place aside).
bool norm_overlaps(const santa_append_norm_args& a, int code) {
  const santa_append_chunk_args& c = a.chunk;
  const int64_t es = c.dtype == SANTA_BF16 ? 2 : 4, n = c.num_tokens, batch = c.batch, d = c.head_dim;
  const int64_t q_row = (c.q ? c.num_q_heads : 0) * d * es, kv_row = c.num_kv_heads * d * es;
  const int64_t teams = c.max_teams, pages = std::min(c.num_pages, kMaxPages);
  const int64_t rows = pages * c.num_kv_heads * c.team_size;
  const int64_t pool = rows * d * (code == santa::kCodeNone ? es : 1);
  const int64_t positions = std::min(c.rope_positions, teams * c.team_size);
  const Span out[] = {{c.q_out, n * q_row}, {c.k_pool, pool}, {c.v_pool, pool}, {a.k_scale, rows * 4},
                      {a.v_scale, rows * 4}, {c.reps, pages * c.num_kv_heads * d * 4},
                      {c.seq_lens_next, batch * 4}};
  const Span in[] = {{c.cu_q, (batch + 1) * 4},  {c.page_table, batch * teams * 4},
                     {c.seq_lens, batch * 4},    {c.rope, positions * c.rope_dim * 4},
                     {a.q_norm, d * 4},          {a.k_norm, d * 4}};
  for (const Span& o : out) {
    if (meets_any(o, in) || meets(o.at, o.bytes, c.k_new, n, kv_row, c.k_stride * es) ||
        meets(o.at, o.bytes, c.v_new, n, kv_row, c.v_stride * es))
      return true;
    if (!(&o == out && c.q_out == c.q) && meets(o.at, o.bytes, c.q, n, q_row, c.q_stride * es))
      return true;
    for (const Span* other = out; other != &o; ++other)
      if (meets(o.at, o.bytes, other->at, 1, other->bytes, other->bytes)) return true;
  }
  return false;
}

void fill_append(const santa_append_chunk_args* a, santa::AppendChunkParams* p) {
  p->q = a->q;
  p->k_new = a->k_new;
  p->v_new = a->v_new;
  p->q_stride = a->q_stride;
  p->k_stride = a->k_stride;
  p->v_stride = a->v_stride;
  p->cu_q = a->cu_q;
  p->page_table = a->page_table;
  p->seq_lens = a->seq_lens;
  p->rope = a->rope;
  p->rope_positions = a->rope_positions;
  p->num_tokens = a->num_tokens;
  p->num_pages = a->num_pages;
  p->batch = a->batch;
  p->num_q_heads = a->num_q_heads;
  p->num_kv_heads = a->num_kv_heads;
  p->team_size = a->team_size;
  p->max_teams = a->max_teams;
  p->rope_dim = a->rope_dim;
  p->interleaved = a->interleaved != 0;
  p->q_out = a->q_out;
  p->k_pool = a->k_pool;
  p->v_pool = a->v_pool;
  p->reps = a->reps;
  p->seq_lens_next = a->seq_lens_next;
  p->status = a->device_status;
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
  const int rc = check_append(a);
  if (rc) return rc;
  santa::AppendChunkParams p = {};
  fill_append(a, &p);
  return map_cuda(santa::launch_append_chunk(p, a->head_dim, a->dtype == SANTA_BF16,
                                             static_cast<cudaStream_t>(stream)));
}

int santa_append_norm(const santa_append_norm_args* a, void* stream) {
  if (!a) return SANTA_ERR_INVALID_ARG;
  const santa_append_chunk_args* c = &a->chunk;
  int rc = check_append(c);
  if (rc) return rc;
  int code = santa::kCodeNone;
  if (a->cache_type != c->dtype && (rc = code_of(a->cache_type, &code))) return rc;
  if (code != santa::kCodeNone && (!a->k_scale || !a->v_scale)) return SANTA_ERR_INVALID_ARG;
  if (code == santa::kCodeNone && (a->k_scale || a->v_scale)) return SANTA_ERR_INVALID_ARG;
  if (!aligned(a->k_scale, 16) || !aligned(a->v_scale, 16) || !aligned(a->q_norm, 16) ||
      !aligned(a->k_norm, 16))
    return SANTA_ERR_INVALID_ARG;
  if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return SANTA_ERR_INVALID_ARG;
  if (santa::append_norm_blocks(c->num_tokens, c->batch, c->q ? c->num_q_heads : 0, c->num_kv_heads,
                                c->head_dim, c->team_size, c->dtype == SANTA_BF16) > 0x7fffffffll)
    return SANTA_ERR_UNSUPPORTED;
  if (norm_overlaps(*a, code)) return SANTA_ERR_INVALID_ARG;
  santa::AppendNormParams p = {};
  fill_append(c, &p);
  p.q_norm = a->q_norm;
  p.k_norm = a->k_norm;
  p.eps = a->eps;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  return map_cuda(santa::launch_append_norm(p, c->head_dim, c->dtype == SANTA_BF16, code,
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
