// q8_abi.cu — the C entry points over 8-bit caches but for the append (cache_abi.cu): argument checks,
// workspace layout and launches.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "abi_checks.h"

using namespace santa::abi;

namespace {

// caps outside these would take the quotient of a score and its cap near the ends of fp32's range
constexpr float kLeastCap = 0x1p-20f, kMostCap = 0x1p20f;

int check_q8_cache(const void* k, const void* v, const float* k_scale, const float* v_scale,
                   int type, int* code) {
  const int rc = code_of(type, code);
  if (rc) return rc;
  if (!k || !v || !k_scale || !v_scale) return SANTA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16))
    return SANTA_ERR_INVALID_ARG;
  return SANTA_OK;
}

int check_q8_shape(int batch, int hq, int hkv, int d, int T, int max_teams) {
  const int rc = check_cache_shape(SANTA_F32, batch, hkv, d, T, max_teams);
  return rc ? rc : check_heads(hq, hkv);
}

// Workspace of an attention (see Q8AttendParams): split units, parts, pieces, behind room for the
// arrival counters that santa_decode keeps at the start of a workspace (zero between calls).
struct Q8Layout {
  int sms;
  size_t counter_bytes, split_bytes, ml_bytes, acc_bytes, bytes;
};
int q8_layout(int batch, int hkv, int d, Q8Layout* l) {
  l->sms = std::min(santa::device_sms(), santa::q8_attend_most_blocks());
  if (l->sms <= 0) return SANTA_ERR_CUDA;
  const size_t rows = static_cast<size_t>(l->sms) * santa::kMaxGroup;
  l->counter_bytes = santa::arrival_counter_bytes(static_cast<int64_t>(batch) * hkv);
  l->split_bytes = round_up(2 * l->sms * sizeof(int32_t), kAlign);
  l->ml_bytes = round_up(2 * rows * 2 * sizeof(float), kAlign);
  l->acc_bytes = 2 * rows * d * sizeof(float);
  l->bytes = kAlign + l->counter_bytes + l->split_bytes + l->ml_bytes + l->acc_bytes +
             santa::q8_attend_warps(d) * rows * d * sizeof(float);
  return SANTA_OK;
}

// Every check of an attention; listed: over sel_ids.
int check_q8_attend(const santa_decode_args* a, const santa_q8_args* c, bool listed, int* code,
                    Q8Layout* l) {
  if (!a || !c) return SANTA_ERR_INVALID_ARG;
  int rc = check_cache_shape(a->dtype, a->batch, a->num_kv_heads, a->head_dim, a->team_size,
                             a->max_teams);
  if (rc || (rc = check_heads(a->num_q_heads, a->num_kv_heads))) return rc;
  if ((rc = check_q8_cache(c->k, c->v, c->k_scale, c->v_scale, c->type, code))) return rc;
  if (a->num_pages < 1 || !a->q || !a->page_table || !a->seq_lens || !a->out)
    return SANTA_ERR_INVALID_ARG;
  if (a->num_pages > kMaxPages) return SANTA_ERR_UNSUPPORTED;
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->page_table, 4) ||
      !aligned(a->seq_lens, 4) || !aligned(a->device_status, 4))
    return SANTA_ERR_INVALID_ARG;
  if (c->softcap != 0.f && !(c->softcap >= kLeastCap && c->softcap <= kMostCap))
    return SANTA_ERR_INVALID_ARG;
  if (c->window < 0) return SANTA_ERR_INVALID_ARG;
  if (listed) {
    if (a->num_draws < 1 || a->num_draws > kMaxDraws) return SANTA_ERR_UNSUPPORTED;
    if (!a->sel_ids || !a->sel_count || !a->pi) return SANTA_ERR_INVALID_ARG;
    if (!aligned(a->sel_ids, 4) || !aligned(a->sel_count, 4) || !aligned(a->pi, 4))
      return SANTA_ERR_INVALID_ARG;
  }
  if (!santa::q8_attend_fits(a->batch, a->num_kv_heads, a->team_size,
                             listed ? a->num_draws : a->max_teams))
    return SANTA_ERR_UNSUPPORTED;
  if ((rc = q8_layout(a->batch, a->num_kv_heads, a->head_dim, l))) return rc;
  if (!a->workspace || a->workspace_bytes < l->bytes) return SANTA_ERR_INVALID_ARG;
  const int64_t rows = a->num_pages * a->num_kv_heads * static_cast<int64_t>(a->team_size);
  const int64_t units = static_cast<int64_t>(a->batch) * a->num_kv_heads;
  const int64_t row = static_cast<int64_t>(a->num_q_heads) * a->head_dim;
  const int64_t list = listed ? units * a->num_draws * 4 : 0;
  const Span in[] = {{a->q, a->batch * row * (a->dtype == SANTA_BF16 ? 2 : 4)},
                     {c->k, rows * a->head_dim},
                     {c->v, rows * a->head_dim},
                     {c->k_scale, rows * 4},
                     {c->v_scale, rows * 4},
                     {a->page_table, static_cast<int64_t>(a->batch) * a->max_teams * 4},
                     {a->seq_lens, static_cast<int64_t>(a->batch) * 4},
                     {a->sel_ids, list},
                     {a->sel_count, listed ? units * 4 : 0},
                     {a->pi, list}};
  const Span out = {a->out, a->batch * row * 4};
  const Span ws = {a->workspace, static_cast<int64_t>(l->bytes)};
  if (meets_any(out, in) || meets_any(ws, in) || meets(out.at, out.bytes, ws.at, 1, ws.bytes, ws.bytes))
    return SANTA_ERR_INVALID_ARG;
  return SANTA_OK;
}

// Every check of the attention behind a choice of teams.  The choice is among all teams of a sequence: those
// of a window may not be among them, so a window is refused.
int check_q8_chosen(const santa_decode_args* a, const santa_q8_args* c) {
  if (c && c->window > 0) return SANTA_ERR_UNSUPPORTED;
  int code = 0;
  Q8Layout l;
  return check_q8_attend(a, c, true, &code, &l);
}

int launch_q8(const santa_decode_args* a, const santa_q8_args* c, bool listed, void* stream) {
  int code = 0;
  Q8Layout l;
  const int rc = check_q8_attend(a, c, listed, &code, &l);
  if (rc) return rc;
  santa::Q8AttendParams p = {};
  p.q = a->q;
  p.k = c->k;
  p.v = c->v;
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.page_table = a->page_table;
  p.seq_lens = a->seq_lens;
  p.sel_ids = listed ? a->sel_ids : nullptr;
  p.sel_count = a->sel_count;
  p.pi = a->pi;
  p.num_pages = a->num_pages;
  p.batch = a->batch;
  p.num_q_heads = a->num_q_heads;
  p.num_kv_heads = a->num_kv_heads;
  p.team_size = a->team_size;
  p.max_teams = a->max_teams;
  p.num_draws = a->num_draws;
  p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(a->head_dim)));
  p.softcap = c->softcap;
  p.window = c->window;
  unsigned char* base = reinterpret_cast<unsigned char*>(
      round_up(reinterpret_cast<uintptr_t>(a->workspace), kAlign) + l.counter_bytes);
  p.goes_on = reinterpret_cast<int32_t*>(base);
  p.begins = p.goes_on + l.sms;
  p.part_ml = reinterpret_cast<float*>(base += l.split_bytes);
  p.part_acc = reinterpret_cast<float*>(base += l.ml_bytes);
  p.piece = reinterpret_cast<float*>(base + l.acc_bytes);
  p.out = a->out;
  p.status = a->device_status;
  return map_cuda(santa::launch_q8_attend(p, a->head_dim, a->dtype == SANTA_BF16, code, l.sms,
                                          static_cast<cudaStream_t>(stream)));
}

}  // namespace

#pragma GCC visibility push(default)
extern "C" {

size_t santa_q8_workspace_bytes(int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                int team_size, int max_teams) {
  Q8Layout l;
  if (check_q8_shape(batch, num_q_heads, num_kv_heads, head_dim, team_size, max_teams) ||
      q8_layout(batch, num_kv_heads, head_dim, &l))
    return 0;
  return l.bytes;
}

int santa_q8_dense_decode(const santa_decode_args* a, const santa_q8_args* c, void* stream) {
  return launch_q8(a, c, false, stream);
}

int santa_q8_attend(const santa_decode_args* a, const santa_q8_args* c, void* stream) {
  return launch_q8(a, c, true, stream);
}

int santa_q8_topk_decode(const santa_decode_args* a, const santa_q8_args* c, void* stream) {
  // everything the attention refuses is refused before the selection is launched
  int rc = check_q8_chosen(a, c);
  if (rc || (rc = santa_select_topk(a, stream))) return rc;
  return launch_q8(a, c, true, stream);
}

int santa_q8_decode(const santa_decode_args* a, const santa_q8_args* c, void* stream) {
  int rc = check_q8_chosen(a, c);
  if (rc) return rc;
  // the sampling reads representatives only; its checks ask for pools all the same
  santa_decode_args b = *a;
  b.k_pool = c->k;
  b.v_pool = c->v;
  if ((rc = santa_sample(&b, stream))) return rc;
  return launch_q8(a, c, true, stream);
}

int santa_q8_read(const santa_q8_read_args* a, void* stream) {
  if (!a) return SANTA_ERR_INVALID_ARG;
  int rc = check_cache_shape(a->out_dtype, a->batch, a->num_kv_heads, a->head_dim, a->team_size,
                             a->max_teams);
  int code = 0;
  if (rc || (rc = check_q8_cache(a->k, a->v, a->k_scale, a->v_scale, a->type, &code))) return rc;
  if (a->num_pages < 1 || a->dst_pages < 1 || !a->page_table || !a->seq_lens || !a->dst_table ||
      !a->k_out || !a->v_out)
    return SANTA_ERR_INVALID_ARG;
  if (a->num_pages > kMaxPages || a->dst_pages > kMaxPages) return SANTA_ERR_UNSUPPORTED;
  if (!aligned(a->k_out, 16) || !aligned(a->v_out, 16) || !aligned(a->page_table, 4) ||
      !aligned(a->seq_lens, 4) || !aligned(a->first, 4) || !aligned(a->dst_table, 4) ||
      !aligned(a->device_status, 4))
    return SANTA_ERR_INVALID_ARG;
  const int64_t page = static_cast<int64_t>(a->num_kv_heads) * a->team_size;
  const int64_t rows = a->num_pages * page, bytes = a->dst_pages * page * a->head_dim *
                                                    (a->out_dtype == SANTA_BF16 ? 2 : 4);
  const int64_t table = static_cast<int64_t>(a->batch) * a->max_teams * 4, lens = a->batch * 4ll;
  const Span in[] = {{a->k, rows * a->head_dim}, {a->v, rows * a->head_dim},
                     {a->k_scale, rows * 4},     {a->v_scale, rows * 4},
                     {a->page_table, table},     {a->dst_table, table},
                     {a->seq_lens, lens},        {a->first, lens}};
  const Span k = {a->k_out, bytes}, v = {a->v_out, bytes};
  if (meets_any(k, in) || meets_any(v, in) || meets(k.at, bytes, v.at, 1, bytes, bytes))
    return SANTA_ERR_INVALID_ARG;
  santa::Q8ReadParams p = {};
  p.k = a->k;
  p.v = a->v;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.page_table = a->page_table;
  p.seq_lens = a->seq_lens;
  p.first = a->first;
  p.dst_table = a->dst_table;
  p.num_pages = a->num_pages;
  p.dst_pages = a->dst_pages;
  p.batch = a->batch;
  p.num_kv_heads = a->num_kv_heads;
  p.team_size = a->team_size;
  p.max_teams = a->max_teams;
  p.k_out = a->k_out;
  p.v_out = a->v_out;
  p.status = a->device_status;
  return map_cuda(santa::launch_q8_read(p, a->head_dim, a->out_dtype == SANTA_BF16, code,
                                        static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
#pragma GCC visibility pop
