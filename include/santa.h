/*
 * santa.h — C ABI of libsanta.so: SANTA++ decode-step attention on one GB300 (sm_103a).
 *
 * Sources of the method (cited by page title and section):
 *   [ABS]  "SANTA++: Sampling Attention through Representative Keys" (arXiv 2609.35629),
 *          abstract, as printed on arxivdaily.com and fugumt.com.
 *   [EXP]  "SANTA++：用代表性 Key 采样把 KV cache 读带宽砍掉 80%" (papers.ananclaw.com
 *          explainer), section 三 (the core method), its five-step pipeline and 3.1.
 *
 * What the library computes, for every sequence b and KV head h (a "unit"):
 *   teams      the n = ceil(seq_len/T) contiguous blocks of T cached tokens; team i is the
 *              KV page page_table[b][i].                                   [ABS; EXP step 1]
 *   reps       rep_i = mean of team i's valid keys (fp32 side buffer).     [ABS; EXP step 2]
 *   probs      s_{g,i} = q_g . rep_i / sqrt(d) for the G = Hq/Hkv query heads g of the group;
 *              p_{g,i} = softmax_i(s_{g,.});  p_i = (1/G) sum_g p_{g,i}.   [ABS; EXP step 2]
 *   sampling   M i.i.d. draws with replacement from p; draw r uses Philox4x32-10 (Salmon et
 *              al., SC'11) with key (lo32(seed), hi32(seed)) and counter (r, h, b, 0); word 0
 *              x gives u = (x + 0.5) 2^-32, and the draw is the smallest i with u*Z < C_i,
 *              C the running sum of p and Z = C_{n-1}.  S = the distinct drawn teams,
 *              ascending; pi_i = 1 - (1 - p_i)^M.                          [ABS; EXP step 3]
 *   attention  for each query head g of the group, the Horvitz-Thompson ratio
 *              out_g = sum_{i in S} (1/pi_i) sum_{j in team i} e^{s_j} v_j
 *                    / sum_{i in S} (1/pi_i) sum_{j in team i} e^{s_j},
 *              s_j = q_g . k_j / sqrt(d).                               [ABS; EXP steps 4-5]
 *
 * Layouts (all row-major, all device memory unless stated):
 *   q          [B][Hq][d]        dtype; query head hq reads KV head hq / G.
 *   k_pool     [P][Hkv][T][d]    dtype; page p, head h is one contiguous T*d block.
 *   v_pool     [P][Hkv][T][d]    dtype.
 *   reps       [P][Hkv][d]       fp32.
 *   page_table [B][max_teams]    int32, physical page of team i of sequence b.
 *   seq_lens   [B]               int32, 1 <= seq_len <= max_teams*T.
 *   out        [B][Hq][d]        fp32.
 *   draw_ids   [B][Hkv][M]       int32, team index of every draw, in draw order.
 *   sel_ids    [B][Hkv][M]       int32, S ascending, padded with -1.
 *   sel_count  [B][Hkv]          int32, |S|.
 *   pi         [B][Hkv][M]       fp32, pi_i aligned with sel_ids, padded with 0.
 *   team_probs [B][Hkv][max_teams] fp32 (optional), p_i, padded with 0.
 *
 * Conventions:
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy default stream)
 *     and runs on the device that is current on the calling thread.
 *   - The caller owns and allocates every buffer.  The library allocates no memory and keeps
 *     no per-call state; calls on different streams with disjoint buffers may overlap.
 *   - Host-side argument errors return SANTA_ERR_INVALID_ARG / SANTA_ERR_UNSUPPORTED and
 *     launch nothing.  A failed launch returns SANTA_ERR_CUDA.
 *   - Errors only visible on the device (an out-of-range page id or seq_len) never trap:
 *     the kernel ORs a SANTA_DEV_* bit into *device_status, skips the offending team or
 *     unit (a skipped unit gets out = 0 and sel_count = 0) and carries on.  The caller
 *     zeroes *device_status, synchronises and reads it; a non-zero word means the outputs
 *     of the affected units are not meaningful (SANTA_ERR_DEVICE_STATUS).
 *   - Supported shapes: dtype f32 or bf16; head_dim 64 or 128; team_size 64 or 128;
 *     1 <= G <= 8; 1 <= M <= 4096; max_teams <= 16384.  All pointers 16-byte aligned.
 */
#ifndef SANTA_H
#define SANTA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SANTA_ABI_VERSION 1

typedef enum santa_status {
  SANTA_OK = 0,
  SANTA_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misaligned pointer, short workspace */
  SANTA_ERR_UNSUPPORTED = 2,   /* a shape outside the supported set above */
  SANTA_ERR_CUDA = 3,          /* a CUDA runtime call or kernel launch failed */
  SANTA_ERR_DEVICE_STATUS = 4, /* reserved for callers: *device_status was non-zero */
  SANTA_ERR_SCRATCH_LIMIT = 5  /* santa_decode_noalloc: the problem needs more scratch than
                                  santa_noalloc_scratch_bytes() */
} santa_status;

typedef enum santa_dtype {
  SANTA_F32 = 0,
  SANTA_BF16 = 1,
  SANTA_I8 = 2,                /* rows of 8-bit caches only (see "The cache in 8 bits") */
  SANTA_E4M3 = 3
} santa_dtype;

/* Bits ORed into *device_status by the kernels. */
#define SANTA_DEV_BAD_PAGE 1u    /* a page id outside [0, num_pages) */
#define SANTA_DEV_BAD_SEQLEN 2u  /* seq_len < 1 or seq_len > max_teams * team_size */
#define SANTA_DEV_BAD_SEL 4u     /* santa_attend given a sel_ids/sel_count/pi entry out of range */
#define SANTA_DEV_TIMEOUT 8u     /* a bounded wait on an asynchronous copy gave up (2 s) */
#define SANTA_DEV_LAYOUT 16u     /* shared memory not 1 KiB-aligned for the swizzled tile copies;
                                   the kernel returned without writing outputs */

/* Returns SANTA_ABI_VERSION of the loaded library. */
int santa_abi_version(void);

/* Static English text for a santa_status value (never NULL). */
const char* santa_status_string(int status);

/*
 * santa_build_reps — the team representative of every (page, KV head): the mean of the
 * page's valid keys.  [ABS, abstract: each team is represented by one key that the query
 * scores; EXP section 三 step 2 lists the mean key as one choice of representative.]
 *
 *   k_pool      [num_pages][num_kv_heads][team_size][head_dim], dtype.
 *   page_fill   [num_pages] int32 valid-token count of each page (0..team_size), or NULL
 *               for "every page full".  A page with fill 0 gets a zero representative.
 *   reps        [num_pages][num_kv_heads][head_dim] fp32, written.
 *   device_status  one int32 (may be NULL); SANTA_DEV_BAD_SEQLEN if a fill is out of range.
 * Run once after prefill; santa_update_reps refreshes single pages during decode.
 */
int santa_build_reps(const void* k_pool, int dtype, int64_t num_pages, int num_kv_heads,
                     int team_size, int head_dim, const int32_t* page_fill, float* reps,
                     int32_t* device_status, void* stream);

/*
 * santa_update_reps — recompute the representative of the listed pages only (for the pages
 * that received new tokens during decode), with the same arithmetic as santa_build_reps.
 *   pages [num_listed] int32 page ids (device); page_fill as in santa_build_reps (device,
 *   indexed by page id, may be NULL for full pages).  A listed id out of range sets
 *   SANTA_DEV_BAD_PAGE and is skipped.
 */
int santa_update_reps(const void* k_pool, int dtype, int64_t num_pages, int num_kv_heads,
                      int team_size, int head_dim, const int32_t* pages, int num_listed,
                      const int32_t* page_fill, float* reps, int32_t* device_status,
                      void* stream);

/*
 * santa_append_kv — one decode step's new token per (sequence, KV head), written into the
 * paged cache, with the representative of its page brought up to date.  This is the step
 * on either side of the decode path: tokens arrive one at a time and the teams they land in
 * must stay described by their mean key.  [ABS, abstract: one representative key per team;
 * EXP section 三 step 2, mean key; section 八 on keeping teams current as the sequence
 * grows.]
 *
 *   k_new, v_new   [batch][num_kv_heads][head_dim], dtype (device).
 *   seq_lens       [batch] current lengths L_b (device); the token goes to position L_b:
 *                  slot L_b % team_size of page page_table[b][L_b / team_size].
 *   k_pool, v_pool the paged cache, written at that slot.
 *   reps           [num_pages][num_kv_heads][head_dim] fp32; the page's entry becomes the
 *                  mean of its L_b % team_size + 1 valid keys, bit-identical to
 *                  santa_build_reps / santa_update_reps on the grown cache (only that page's
 *                  rows are read).
 *   seq_lens_next  [batch] receives L_b + 1 (may be NULL; must not alias seq_lens).
 *   device_status  SANTA_DEV_BAD_SEQLEN (L_b outside [0, max_teams * team_size)) or
 *                  SANTA_DEV_BAD_PAGE; the sequence is then skipped.
 * The page a token lands in must belong to that sequence alone (a shared-prefix page is
 * never appended to).  Asynchronous on `stream`.
 */
int santa_append_kv(const void* k_new, const void* v_new, int dtype, int batch,
                    int num_kv_heads, int team_size, int head_dim, int max_teams,
                    int64_t num_pages, const int32_t* page_table, const int32_t* seq_lens,
                    void* k_pool, void* v_pool, float* reps, int32_t* seq_lens_next,
                    int32_t* device_status, void* stream);

/* All inputs, outputs and scratch of one decode step (see the layouts above). */
typedef struct santa_decode_args {
  /* inputs */
  const void* q;
  const void* k_pool;
  const void* v_pool;
  const float* reps;           /* read by santa_sample / santa_decode */
  const int32_t* page_table;
  const int32_t* seq_lens;
  int dtype;                   /* santa_dtype of q, k_pool and v_pool */
  int batch;                   /* B */
  int num_q_heads;             /* Hq */
  int num_kv_heads;            /* Hkv, Hq % Hkv == 0 */
  int head_dim;                /* d */
  int team_size;               /* T, also the KV page size */
  int max_teams;               /* row length of page_table */
  int num_draws;               /* M */
  int64_t num_pages;           /* P, rows of k_pool / v_pool / reps */
  uint64_t seed;               /* Philox key */
  /* outputs (santa_attend reads sel_ids, sel_count and pi as inputs) */
  float* out;
  int32_t* draw_ids;
  int32_t* sel_ids;
  int32_t* sel_count;
  float* pi;
  float* team_probs;           /* optional, may be NULL */
  /* scratch: caller-owned device memory (see "Workspace" below), zeroed before first use */
  void* workspace;
  size_t workspace_bytes;
  int32_t* device_status;      /* one int32 the kernels OR SANTA_DEV_* bits into */
  /* sampler variants (santa_sample / santa_decode; zero = the plain method) */
  int32_t sampler;             /* santa_sampler */
  float mix_alpha;             /* defensive mixture weight alpha in [0, 1] */
} santa_decode_args;

/*
 * Samplers.  All draw from q_i = (1 - mix_alpha) p_i + mix_alpha / n, the team distribution
 * with a uniform share mixed in: the defensive mixture of [EXP] section 八 (pitfall 4), which
 * keeps every weight bounded.  mix_alpha = 0 is the plain distribution.  The output pi[k]
 * always holds 1 / (weight of team sel_ids[k]), which santa_attend consumes as it is.
 *   SANTA_SAMPLER_IID_HT      M i.i.d. draws; weight 1/pi_i, pi_i = 1 - (1 - q_i)^M
 *                             (Horvitz-Thompson: the method of [ABS]).
 *   SANTA_SAMPLER_SYSTEMATIC  one uniform u (the Philox word of draw 0), the M points
 *                             (r + u) / M on the CDF; weight 1/pi_i with pi_i = min(1, M q_i)
 *                             (the stratified / systematic variants of [SANTA], abstract).
 *   SANTA_SAMPLER_IID_HH      M i.i.d. draws; weight c_i / (M q_i), c_i the draws of team i
 *                             (Hansen-Hurwitz: the per-draw 1/p_i of [EXP] section 三 step 5).
 * Non-default samplers and mix_alpha > 0 need every unit sampled inside one CTA's shared
 * memory: max_teams <= 1024 and (G + 1) * ceil(max_teams / CL) <= 2048 for the plan's
 * cluster size CL; other shapes return SANTA_ERR_UNSUPPORTED.
 */
typedef enum {
  SANTA_SAMPLER_IID_HT = 0,
  SANTA_SAMPLER_SYSTEMATIC = 1,
  SANTA_SAMPLER_IID_HH = 2
} santa_sampler;

/*
 * Workspace.  A unit is served by one thread-block cluster (up to 16 CTAs sharing their
 * partial results on chip) unless it has so much work that several clusters share it;
 * only then do the clusters' partials and an arrival counter per unit go through the
 * workspace.  santa_decode_workspace_bytes returns the size the library's default plan
 * wants on the current device (0 for an unsupported shape); any size down to
 * santa_decode_workspace_min_bytes also works, with fewer clusters per unit.  When the
 * minimum is 256 bytes (every unit fits one cluster), the workspace may be NULL.  The
 * counters must be zero before the first call (they are left at zero by every call).
 * santa_dense_workspace_bytes sizes the workspace of santa_dense_decode the same way.  A
 * workspace is used by one call at a time.
 */
size_t santa_decode_workspace_bytes(int dtype, int batch, int num_q_heads, int num_kv_heads,
                                    int head_dim, int team_size, int max_teams, int num_draws);
size_t santa_decode_workspace_min_bytes(int batch, int num_q_heads, int num_kv_heads,
                                        int head_dim, int team_size, int max_teams,
                                        int num_draws);

/*
 * santa_sample — score the representatives, form the GQA-mixed team distribution, draw M
 * teams, deduplicate and compute the inclusion probabilities.  Writes draw_ids, sel_ids,
 * sel_count, pi and team_probs (if not NULL).
 * [ABS, abstract: the scores of the representatives decide which teams are sampled; EXP
 * section 三 steps 2-3.]  Uses no workspace.
 */
int santa_sample(const santa_decode_args* a, void* stream);

/*
 * santa_attend — exact attention inside the teams listed in sel_ids[0..sel_count) of every
 * unit, each team weighted by 1/pi, combined as the Horvitz-Thompson ratio into out.
 * sel_ids / sel_count / pi may come from santa_sample or from the caller (distinct team
 * indices < n, any order, pi finite and > 0: the inclusion probability for Horvitz-Thompson
 * weights, M q_i / c_i for Hansen-Hurwitz ones); entries out of range set SANTA_DEV_BAD_SEL
 * and are skipped.
 * [ABS, abstract: attention is exact inside the sampled teams, and each team's share is
 * scaled by one over the probability that the team is in the sample; EXP steps 4-5.]
 */
int santa_attend(const santa_decode_args* a, void* stream);

/*
 * santa_decode_plan — the launch the library would use for `a` (whose pointers need not be
 * valid; only shapes and workspace_bytes are read): out[0] = CTAs per thread-block cluster
 * (CL), out[1] = clusters per unit (NC; NC > 1 routes partials through the workspace),
 * out[2] = teams one CTA scores, out[3] = clusters of CL CTAs the device can run at once,
 * out[4] = 1 if the wide variant runs (bf16 steps whose launch fits one CTA per SM: six
 * stages, two warp groups consuming alternate chunks), else 0.  `out` holds 5 entries.
 * `which`: 0 santa_decode, 1 santa_sample, 2 santa_attend, 3 santa_dense_decode.
 */
int santa_decode_plan(const santa_decode_args* a, int which, int32_t* out);

/* santa_decode — santa_sample followed by santa_attend on `stream`. [ABS] */
int santa_decode(const santa_decode_args* a, void* stream);

/*
 * santa_decode_path — which form of the kernel santa_decode(a) runs (a's pointers need not
 * be valid; shapes, sampler, mix_alpha and workspace_bytes are read).  1: the compact form,
 * for bf16 steps with one cluster per unit and at most 1024 teams per sequence, whose
 * sampling prologue is compiled without the general form's branches (the sampler variants
 * and the mixture run separate instantiations of it); 0: the general form; a negative
 * santa_status for a refused shape.  Both forms compute the same step.
 */
int santa_decode_path(const santa_decode_args* a);

/*
 * santa_dense_decode — exact dense softmax attention over all seq_len tokens of every
 * sequence, split-K over the paged cache (the speed reference the sampled path is compared
 * with; [ABS] compares against a dense FlashAttention baseline).  Reads q, k_pool, v_pool,
 * page_table, seq_lens and the shape fields; writes out; uses workspace and device_status.
 * reps, num_draws, seed and the sampling outputs are ignored.
 */
size_t santa_dense_workspace_bytes(int dtype, int batch, int num_q_heads, int num_kv_heads,
                                   int head_dim, int team_size, int max_teams);
int santa_dense_decode(const santa_decode_args* a, void* stream);

/*
 * santa_decode_noalloc — santa_decode for callers that cannot allocate device memory (no
 * counterpart in the paper; it is a property of this library, not of the method).
 *
 * Who needs it: code that runs where cudaMalloc is not available or not allowed, such as
 * a plug-in inside an inference engine that owns all device memory and lends none after
 * start-up, or a loop that must not allocate once it is running.  Such a caller cannot
 * provide santa_decode's workspace.  This entry point ignores a->workspace and
 * a->workspace_bytes and uses instead a scratch array compiled into the library (a
 * file-scope __device__ array of santa_noalloc_scratch_bytes() = 4 MiB, present on every
 * device that loads the library until the process exits).  It calls no allocator.
 *
 *   - Same inputs, outputs and results as santa_decode (the split plan is the default one
 *     cut down to fit the scratch, so the output may differ from santa_decode's in the
 *     last bits only).
 *   - Returns SANTA_ERR_SCRATCH_LIMIT, before any CUDA call, when the shape needs more than
 *     the scratch holds: santa_decode_workspace_min_bytes > santa_noalloc_scratch_bytes(),
 *     or more than (scratch - 256) / 4 (sequence, KV head) units (their arrival counters).
 *     Every other argument error returns santa_decode's status; a refused call leaves the
 *     array untouched.
 *   - The first call on a device looks up the array's device address (cudaGetSymbolAddress)
 *     with that device current and keeps it for the process; make that first call before any
 *     stream capture.  The kept address is void after cudaDeviceReset on that device (the
 *     module is then loaded again, possibly elsewhere): do not call this entry point after
 *     a reset.
 *   - Every call on a device shares the one array, which keeps the previous call's
 *     contents.  When the plan spreads a unit over several clusters, the call first clears
 *     the arrival counters at the array's start (cudaMemsetAsync on the call's stream, no
 *     allocation).  Calls whose work overlaps on the GPU (different streams, or other
 *     threads) race on the array: serialise them.
 */
int santa_decode_noalloc(const santa_decode_args* a, void* stream);

/*
 * santa_decode_host — one decode step whose inputs come from and whose outputs go to host
 * memory (no counterpart in the paper; a convenience of this library).  On `stream` it
 * copies in_bytes from host_in to dev_in, runs santa_decode(a), copies out_bytes from
 * dev_out to host_out and waits for the stream.
 *
 *   - How each copy is made: when the host buffer is page-locked memory that the current
 *     device reaches at the same address (cudaHostAlloc, a pinned torch tensor) and both
 *     pointers and the size are multiples of 16 bytes, a small kernel of this library moves
 *     the bytes (reading or writing the host memory directly), chained to the decode launch
 *     by programmatic dependent launch; otherwise cudaMemcpyAsync does.  The bytes moved are
 *     the same either way.
 *
 *   - The caller lays out the buffers.  a's input pointers (q, page_table, seq_lens) point
 *     into dev_in, and its output pointers (out, draw_ids, sel_ids, sel_count, pi, and
 *     device_status if the caller wants it back in the same copy) into dev_out, so that
 *     one copy moves each side.  The library reads neither layout: it copies bytes.
 *   - host_in and host_out should be page-locked (cudaHostAlloc or a pinned torch tensor).
 *     Pageable memory works, but then the runtime stages the copies synchronously.
 *   - in_bytes or out_bytes may be 0 (that copy is skipped); otherwise both pointers of
 *     that copy must be non-null (SANTA_ERR_INVALID_ARG, nothing enqueued).
 *   - Returns santa_decode's error if the step is refused (the input copy may already be
 *     enqueued), SANTA_ERR_CUDA if a copy or the stream wait fails, else SANTA_OK after the
 *     host outputs are complete.  device_status is not read here; with device_status in
 *     dev_out, the caller reads the host copy.
 */
int santa_decode_host(const santa_decode_args* a, const void* host_in, void* dev_in,
                      size_t in_bytes, void* host_out, const void* dev_out, size_t out_bytes,
                      void* stream);

/*
 * santa_host_copy_route — how santa_decode_host would move `bytes` between the host buffer
 * `host` and the device buffer `dev` (either direction): 1 when its own copy kernel would
 * (`host` page-locked, reached by the current device at the same address, [host, host +
 * bytes) inside one allocation, both pointers and the size multiples of 16), 0 when
 * cudaMemcpyAsync would (also for null pointers or bytes = 0).  Enqueues nothing.
 */
int santa_host_copy_route(const void* host, const void* dev, size_t bytes);

/*
 * santa_attend_vs — santa_attend with value-row sampling inside every listed team, in place
 * of the full P.V product ([SANTA] "Stochastic Sparse Attention for Memory-Bound
 * Inference", abstract: draw value rows from the post-softmax distribution and gather-add
 * them).  The G query heads of a KV head share one set of S rows per team, drawn from the
 * group-mean in-team softmax r_j; head g weighs a drawn row j by exp(s_gj - m_g) / r_j, and
 * the team denominators stay exact, so the numerator is unbiased given the teams.  Row draw
 * k of team i of unit (b, h) uses Philox4x32-10 word 0 of counter (k, h, b, 1 + i) with key
 * `seed`, decided exactly on a 62-bit fixed-point CDF like the team draws.  Reads only the K
 * rows of the listed teams and S value rows of each.
 *   a          as for santa_attend (sel_ids, sel_count, pi in; out written), num_draws = M
 *              (the slot dimension, <= 1024), seed = key of the row draws, workspace of at
 *              least santa_attend_vs_workspace_bytes bytes (per-team partials).
 *   value_rows S, rows drawn per team, 1..256.
 *   value_ids  [B][Hkv][M][S] int32: the drawn rows (token index within the team), or NULL.
 * Two launches on `stream`.
 */
size_t santa_attend_vs_workspace_bytes(int batch, int num_q_heads, int num_kv_heads,
                                       int head_dim, int num_draws);
int santa_attend_vs(const santa_decode_args* a, int value_rows, int32_t* value_ids,
                    void* stream);

/*
 * ---- The prompt side of the cache and the deterministic sparse step ----
 *
 * A "chunk" is the run of new tokens of every sequence in one call, as many as each has (a
 * prompt, a slice of a prompt, drafted tokens, or the single token of a decode step).  The
 * chunks of a batch lie one behind the other in the token dimension of q, k_new and v_new:
 *   cu_q [B + 1] int32 (device): sequence b's tokens are rows cu_q[b] .. cu_q[b+1] - 1, with
 *   0 <= cu_q[0] and cu_q non-decreasing up to at most num_tokens.  Rows outside
 *   [cu_q[0], cu_q[B]) belong to no sequence (padding): they are neither read for a result
 *   nor written.  A sequence may have no new token.
 * A cu_q that is not so sets SANTA_DEV_BAD_SEQLEN; nothing outside the given buffers is then
 * touched, but the results are not meaningful.
 */

/*
 * santa_rope_table — cosines and sines of a rotary position embedding:
 *   table[p][j] = cos(p theta^(-2j / rope_dim)), table[p][rope_dim / 2 + j] = sin(same),
 *   0 <= j < rope_dim / 2, each computed in 64 bits and rounded once to fp32 (an angle of a
 *   far position has no accurate fp32 value).
 * table [positions][rope_dim] fp32 (device, 16-byte aligned); rope_dim a multiple of 16 up to
 * 128; theta > 1.  Made once; santa_append_chunk also takes tables that the caller computes in
 * another way (scaled frequencies).
 */
int santa_rope_table(float* table, int64_t positions, int rope_dim, double theta, void* stream);

/* One chunk append (layouts as above; see santa_append_chunk). */
typedef struct santa_append_chunk_args {
  const void* q;               /* [num_tokens][Hq][d] or NULL */
  const void* k_new;           /* [num_tokens][Hkv][d] */
  const void* v_new;           /* [num_tokens][Hkv][d] */
  int64_t q_stride;            /* elements from one token's row to the next (>= Hq * d) */
  int64_t k_stride;            /* (>= Hkv * d) */
  int64_t v_stride;
  const int32_t* cu_q;         /* [B + 1] */
  const int32_t* page_table;   /* [B][max_teams] */
  const int32_t* seq_lens;     /* [B] cached tokens before the call */
  const float* rope;           /* [rope_positions][rope_dim], or NULL with rope_dim = 0 */
  int64_t rope_positions;
  int64_t num_tokens;
  int64_t num_pages;
  int dtype;                   /* santa_dtype of q, k_new, v_new, the pools and q_out */
  int batch;
  int num_q_heads;             /* Hq (ignored when q is NULL) */
  int num_kv_heads;
  int head_dim;
  int team_size;
  int max_teams;
  int rope_dim;                /* R: 0 (no rotation) or a multiple of 16 up to head_dim */
  int interleaved;             /* 0: pairs (j, j + R/2); 1: pairs (2j, 2j + 1) */
  void* q_out;                 /* [num_tokens][Hq][d] contiguous, rotated queries; may be q
                                  itself when q_stride = Hq * d, and overlaps no row of q,
                                  k_new or v_new otherwise; NULL with q */
  void* k_pool;                /* [P][Hkv][T][d] */
  void* v_pool;
  float* reps;                 /* [P][Hkv][d] */
  int32_t* seq_lens_next;      /* [B] receives the new lengths (may be NULL; does not overlap
                                  seq_lens or cu_q) */
  int32_t* device_status;      /* may be NULL */
} santa_append_chunk_args;

/*
 * santa_append_chunk — a chunk's keys and values into the paged cache, keys (and queries)
 * rotated by position on the way, and the representatives of the touched pages brought up to
 * date.  Token i of sequence b gets position p = seq_lens[b] + i: slot p % T of page
 * page_table[b][p / T].  With (c, s) = (rope[p][j], rope[p][R/2 + j]), pair j becomes
 *   x' = x c - y s,   y' = y c + x s      (products and sum each rounded to fp32),
 * elements from R on pass unchanged, and the result is rounded once to the cache's type.
 * The representative of every touched page becomes the mean of its valid keys, bit-identical
 * to santa_build_reps on the grown cache.  One launch; reads the earlier keys of a page that
 * was already begun, and nothing else of the cache.
 *
 *   - A sequence whose length is out of range (seq_lens[b] < 0, or seq_lens[b] plus its new
 *     tokens above max_teams * T or, with rotation, above rope_positions) sets
 *     SANTA_DEV_BAD_SEQLEN and is skipped: no token, query or length of it is written.
 *   - A page id out of range sets SANTA_DEV_BAD_PAGE; the tokens of that page are not stored.
 *   - Every page that receives a token must belong to that sequence alone.
 *   - num_tokens may be 0 (seq_lens_next is then a copy of the lengths).
 *   - Pointers are 16-byte aligned (int32 arrays 4), strides multiples of 16 bytes.
 */
int santa_append_chunk(const santa_append_chunk_args* a, void* stream);

/* One chunk attention (see santa_chunk_attend). */
typedef struct santa_chunk_args {
  const void* q;               /* [num_tokens][Hq][d] contiguous, dtype */
  const void* k_pool;          /* [P][Hkv][T][d] */
  const void* v_pool;
  const int32_t* page_table;   /* [B][max_teams] */
  const int32_t* seq_lens;     /* [B] cached tokens, the chunk's included */
  const int32_t* cu_q;         /* [B + 1] */
  int64_t num_tokens;
  int64_t num_pages;
  int dtype;
  int batch;
  int num_q_heads;
  int num_kv_heads;
  int head_dim;
  int team_size;
  int max_teams;
  void* out;                   /* [num_tokens][Hq][d] dtype; does not overlap q */
  void* workspace;             /* santa_chunk_workspace_bytes; contents need not be set */
  size_t workspace_bytes;
  int32_t* device_status;      /* may be NULL */
} santa_chunk_args;

/*
 * santa_chunk_attend — exact causal attention of a chunk over the paged cache that already
 * holds it (santa_append_chunk).  Sequence b's new tokens, n_b = cu_q[b+1] - cu_q[b], are the
 * last n_b of its seq_lens[b]: token i sees the cached tokens 0 .. seq_lens[b] - n_b + i, and
 *   out_i = sum_j softmax_j(q_i . k_j / sqrt(d)) v_j  over them.
 * bf16 runs on the tensor cores with fp32 accumulation (the weights are rounded to bf16 before
 * their product with V, the sum of the weights is not); fp32 is fp32 throughout.  A row whose
 * every score is -inf gets zeros.  What a row does not see (later tokens, slots behind the
 * sequence's end, other sequences' pages) has no influence on it, whatever it holds.
 *
 *   - A sequence with new tokens and a length outside [n_b, max_teams * T] sets
 *     SANTA_DEV_BAD_SEQLEN and is skipped: its rows of out are not written.
 *   - A page id out of range sets SANTA_DEV_BAD_PAGE; page 0 is read in its place, and the
 *     rows of that sequence are not meaningful.
 *   - The workspace holds partial results of tiles that several blocks share; it needs no
 *     initialisation and serves one call at a time.  Results do not depend on its contents
 *     or on timing: equal calls give equal bits.
 *   - num_tokens may be 0 (nothing is launched).
 *   - SANTA_DEV_TIMEOUT (bf16): a bounded wait inside the kernel gave up; the call's results are
 *     not meaningful, the context stays usable.
 */
size_t santa_chunk_workspace_bytes(int dtype, int batch, int64_t num_tokens, int num_q_heads,
                                   int num_kv_heads, int head_dim, int team_size,
                                   int max_teams);
int santa_chunk_attend(const santa_chunk_args* a, void* stream);

/*
 * santa_select_topk — the deterministic counterpart of santa_sample: the score of team i for
 * unit (b, h) is s_i = max over the group's heads g of q_g . rep_i, and S is the min(M, n)
 * teams of largest s_i (ties to the lower index).  A team with a NaN score or with a page id out
 * of range ranks below every score, -inf included; a bad page sets SANTA_DEV_BAD_PAGE.
 * M = num_draws.
 * Scores are fp32; teams whose scores lie too close to the border of S for fp32 to order are
 * compared in 64 bits, so S is the set that 64-bit scores give.  Writes sel_ids (ascending,
 * padded with -1), sel_count and pi (1 for each selected team, padded with 0).  Reads q, reps,
 * page_table, seq_lens; k_pool, v_pool, seed, sampler, draw_ids, team_probs and workspace are
 * not used.
 */
int santa_select_topk(const santa_decode_args* a, void* stream);

/*
 * santa_topk_decode — santa_select_topk followed by santa_attend on `stream`: exact attention
 * inside the M teams of best representative score.  (With bf16 caches the weights enter the
 * product with V in full, where santa_attend keeps about 16 bits of them.)  A chunk of several
 * query tokens of one sequence is served as that many rows of the batch, with the same page-table
 * row and growing lengths.  Workspace as for santa_decode.
 */
int santa_topk_decode(const santa_decode_args* a, void* stream);

/*
 * ---- The cache in 8 bits ----
 *
 * A row (the key or the value of one token and KV head) of d elements x is held as d codes c of one
 * byte and one fp32 scale s, and stands for c s:
 *   s = max(max_j |x_j|, 2^-90) / top,   c_j = x_j / s rounded to the nearest code (ties to even),
 * top = 127 for SANTA_I8 (two's complement) and 448 for SANTA_E4M3 (the finite 4-3 format).  A row
 * with an infinity or a NaN gets s = NaN and codes 0.  Codes of a cache filled in another way may be
 * any byte; an e4m3 NaN code makes what sees it NaN.
 *   codes   k, v             [P][Hkv][T][d] bytes, 16-byte aligned
 *   scales  k_scale, v_scale [P][Hkv][T] fp32, 16-byte aligned
 * Page tables, lengths and representatives are those of the other caches: reps are fp32 means of the
 * keys that the rows stand for, so santa_sample and santa_select_topk work unchanged beside it.
 */

/* One append with norms (see santa_append_norm). */
typedef struct santa_append_norm_args {
  santa_append_chunk_args chunk;  /* as for santa_append_chunk; chunk.dtype is the type of q, k_new,
                                     v_new and q_out; k_pool and v_pool hold the codes of an 8-bit
                                     cache */
  int cache_type;                 /* chunk.dtype, SANTA_I8 or SANTA_E4M3 */
  float eps;                      /* of the norms: >= 0 and finite */
  const float* q_norm;            /* [d] fp32 weights, or NULL: queries are not normed */
  const float* k_norm;            /* [d] fp32 weights, or NULL: keys are not normed */
  float* k_scale;                 /* 8-bit caches; NULL otherwise */
  float* v_scale;
} santa_append_norm_args;

/*
 * santa_append_norm — santa_append_chunk with the norms of the heads in the same pass, into a cache
 * of the activations' type or of 8 bits.  A query or key x of one head becomes
 *   y = x / sqrt(mean_j(x_j^2) + eps) * w
 * (q_norm for queries, k_norm for keys), then its pairs are turned as in santa_append_chunk, all in
 * fp32, and the result is rounded once: queries to their type, keys to the cache's.  The squares'
 * sum is held in fp32 too: where mean + eps lies outside 2^-120 .. 2^120, a row may become zeros,
 * infinities or NaN.  Values are neither normed nor turned.  With a cache of the activations' type and no norms the results are
 * santa_append_chunk's, bit for bit.
 *   - The representative of a touched page is the mean of its keys as stored; it does not depend on
 *     how the tokens were divided among calls.
 *   - What the call writes (q_out, pools, scales, reps, seq_lens_next) overlaps nothing else that it
 *     writes or reads, but for q_out = q.
 *   - Everything else (ragged chunks, lengths, refusals, device status, skipped sequences and pages)
 *     is as for santa_append_chunk.  Scales and weights are 16-byte aligned.
 */
int santa_append_norm(const santa_append_norm_args* a, void* stream);

/* The cache of 8 bits that the santa_q8_* attention reads beside santa_decode_args, and the options
 * of its scores. */
typedef struct santa_q8_args {
  const void* k;               /* codes and scales as above */
  const void* v;
  const float* k_scale;
  const float* v_scale;
  int type;                    /* SANTA_I8 or SANTA_E4M3 */
  int window;                  /* 0: none; else a token sees the last `window` cached tokens only */
  float softcap;               /* 0: none; else (2^-20 .. 2^20) scores s become
                                  softcap * tanh(s / softcap) */
} santa_q8_args;

/*
 * santa_q8_dense_decode / santa_q8_attend — attention of one new token per sequence over an 8-bit
 * cache: every cached token, or the teams listed in a->sel_ids[0 .. sel_count) with weight 1/pi
 * (santa_dense_decode and santa_attend over the values that the rows stand for).  With the score
 * s_j = q . k_j / sqrt(d), capped if asked, over the tokens j < seq_len that the window leaves,
 *   out = sum_j w_j e^{s_j} v_j / sum_j w_j e^{s_j}     (w_j = 1, or 1 / pi of j's team).
 * Sums are held in fp32.  q and the weights enter the products as fp16 pieces: elements of bf16
 * queries exact down to 2^-31 of their head's largest, of fp32 ones to 2^-22 of themselves (or 2^-50 of
 * the largest where that is more), weights to 2^-22 of themselves (or 2^-43 of the largest).
 *   a    q, page_table, seq_lens, dtype (of q), shapes, num_pages, out, workspace, device_status;
 *        santa_q8_attend also sel_ids, sel_count, pi and num_draws (1 .. 4096).  k_pool, v_pool, reps
 *        and the other fields are not read.
 *   - A sequence of length 0 and a unit without a seen token get zeros.  A length outside
 *     [0, max_teams * T] sets SANTA_DEV_BAD_SEQLEN and its rows get zeros; a page id out of range
 *     sets SANTA_DEV_BAD_PAGE and its tokens are left out; a listed team out of range, a weight that
 *     is not finite and positive or a count outside [0, num_draws] sets SANTA_DEV_BAD_SEL, and that
 *     team is left out (a count is clamped).  A team listed twice counts twice.
 *   - What is not seen has no influence, whatever its bytes and scales hold; table entries of pages
 *     that hold no seen token may be anything.
 *   - Scores may be as large as 2^25 in magnitude (before the cap: anything); rows with larger ones may
 *     become NaN.
 *   - batch * num_kv_heads * teams * T / 32 (teams = max_teams, or num_draws of santa_q8_attend) must
 *     stay below about 2^31; more is SANTA_ERR_UNSUPPORTED.
 *   - out does not overlap what the call reads or the workspace.  The workspace
 *     (santa_q8_workspace_bytes) needs no initialisation and serves one call at a time.  The arrival
 *     counters that santa_decode and santa_dense_decode keep in a workspace for the same batch and KV
 *     heads, or fewer, are left as they are: one workspace, large enough for both and with its counters
 *     zeroed once, serves layers of either kind in turn.  Equal calls give equal bits.
 */
size_t santa_q8_workspace_bytes(int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                int team_size, int max_teams);
int santa_q8_dense_decode(const santa_decode_args* a, const santa_q8_args* c, void* stream);
int santa_q8_attend(const santa_decode_args* a, const santa_q8_args* c, void* stream);

/*
 * santa_q8_topk_decode / santa_q8_decode — santa_select_topk or santa_sample followed by
 * santa_q8_attend on `stream`: the sparse steps over an 8-bit cache.  a as for santa_topk_decode and
 * santa_decode but for k_pool and v_pool, which are not read, and the workspace, which is
 * santa_q8_attend's.  The selection takes every team of the sequence and plain scores; softcap acts in
 * the attention.  A window is SANTA_ERR_UNSUPPORTED: the chosen teams might all lie before it.
 */
int santa_q8_topk_decode(const santa_decode_args* a, const santa_q8_args* c, void* stream);
int santa_q8_decode(const santa_decode_args* a, const santa_q8_args* c, void* stream);

/* One reading back (see santa_q8_read). */
typedef struct santa_q8_read_args {
  const void* k;               /* codes and scales as above */
  const void* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;   /* [B][max_teams] */
  const int32_t* seq_lens;     /* [B] */
  const int32_t* first;        /* [B] first token to read, or NULL: 0 */
  const int32_t* dst_table;    /* [B][max_teams] pages of the destination */
  int64_t num_pages;
  int64_t dst_pages;
  int type;                    /* SANTA_I8 or SANTA_E4M3 */
  int out_dtype;               /* SANTA_F32 or SANTA_BF16 */
  int batch;
  int num_kv_heads;
  int head_dim;
  int team_size;
  int max_teams;
  void* k_out;                 /* [dst_pages][Hkv][T][d] out_dtype */
  void* v_out;
  int32_t* device_status;      /* may be NULL */
} santa_q8_read_args;

/*
 * santa_q8_read — tokens first[b] .. seq_lens[b] - 1 of every sequence out of an 8-bit cache into the
 * same slots of the pages dst_table names, as bf16 or fp32: c s in fp32, rounded once.  The result is
 * a cache that santa_chunk_attend, santa_build_reps and the other calls read; `first` lets a prompt's
 * next chunk read back only what it added.
 *   - Slots of other tokens are left as they were.
 *   - first[b] < 0, seq_lens[b] < first[b] or a length above max_teams * T sets
 *     SANTA_DEV_BAD_SEQLEN (that sequence is skipped), a page id out of range on either side
 *     SANTA_DEV_BAD_PAGE (that page is skipped).
 *   - No two pages of a call's destinations may be the same; the outputs overlap neither each other
 *     nor what is read.
 */
int santa_q8_read(const santa_q8_read_args* a, void* stream);

/* Size in bytes of the scratch array santa_decode_noalloc uses. */
size_t santa_noalloc_scratch_bytes(void);

#ifdef __cplusplus
}
#endif

#endif /* SANTA_H */
