/*
 * attn.h -- C ABI of the GB300 (sm_103a) fused attention forward library.
 *
 * The library computes scaled-dot-product attention forward,
 *
 *     S = scale * Q K^T  (+ causal mask),   P = softmax(S),   O = P V,
 *     lse = m + ln(l)    (per query row: m = max_j S, l = sum_j exp(S - m)),
 *
 * as defined by the standard attention chain of "GPU 学习日报 Day 24：Operator
 * Fusion" (Operator Fusion, GPU learning diary day 24), §3.4 "Attention Fusion:
 * FlashAttention", computed by the tiled online-softmax recurrence of the same
 * section's second listing (running row max m, running row sum l, rescaled O
 * accumulator, one normalisation at the end), so that the Lq x Lkv score matrix
 * never reaches HBM.  The log-sum-exp output is not on that page; it is the
 * natural-log normaliser built from the m and l that listing carries.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *    never frees or retains them.  Every pointer must be 16-byte aligned.
 *  - Element types: q, k, v, kcache, vcache are bf16 (raw 16-bit words, passed
 *    as void*).  out is bf16 unless an *_ex call asks for fp32.  lse is fp32.
 *  - Arithmetic: fp32 accumulation everywhere; on the tensor-core paths
 *    (prefill, multi-token decode) P is rounded to bf16 before the P V
 *    product, single-token decode keeps P in fp32.
 *  - Causal masking is aligned to the bottom-right corner: key j is visible to
 *    query i iff j <= i + (Lkv - Lq).  For Lq == Lkv this is the lower
 *    triangle.  A query row that sees no key gets O = 0 and lse = -inf.
 *  - Grouped-query attention: Hq must be a multiple of Hkv; query head h reads
 *    key/value head h / (Hq / Hkv) (contiguous groups).
 *  - D (head dimension) must be 64 or 128.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls are
 *    asynchronous with respect to the host: they enqueue kernels and return.
 *  - Errors the host can see (NULL pointer, bad size, misalignment, wrong GPU)
 *    are returned synchronously before anything is enqueued.  A CUDA launch
 *    failure returns ATTN_ERR_CUDA.  Problems only the device can see (a
 *    kv_len outside [0, Lmax], a pipeline wait that timed out) are recorded in
 *    a per-device status word read by attn_get_device_status(); the kernels
 *    never trap.
 *  - There is no CPU fallback: without an sm_103 device every compute call
 *    returns ATTN_ERR_UNSUPPORTED or ATTN_ERR_CUDA.
 */
#ifndef ATTN_GB300_H
#define ATTN_GB300_H

#ifdef __cplusplus
extern "C" {
#endif

typedef enum attn_status {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1,     /* NULL pointer, non-positive size, Hq % Hkv != 0, ... */
  ATTN_ERR_UNSUPPORTED = 2,     /* D not in {64,128}, device is not sm_103, ...        */
  ATTN_ERR_ALIGNMENT = 3,       /* a pointer is not 16-byte aligned                    */
  ATTN_ERR_CUDA = 4,            /* a CUDA runtime call or launch failed                */
  ATTN_ERR_DEVICE_TIMEOUT = 5,  /* device status: a bounded pipeline wait expired      */
  ATTN_ERR_DEVICE_BOUNDS = 6,   /* device status: a length, position, slot or page id was out of range */
  ATTN_ERR_SCRATCH_TOO_SMALL = 7, /* attn_decode_noalloc: partials exceed its fixed buffer; a caller's workspace is too small */
  ATTN_ERR_DEVICE_POOL = 8      /* device status: attn_page_step found too few free pages  */
} attn_status;

typedef enum attn_dtype { ATTN_DTYPE_BF16 = 0, ATTN_DTYPE_F32 = 1 } attn_dtype;

/*
 * attn_rope -- rotary position embedding (RoPE) applied inside the kernels,
 * as "Что такое kernel fusion и как он применяется в LLM serving?" §3.5 and
 * Operator Fusion's exercise 1 (RoPE fused into the attention kernel)
 * describe; the pages give no formula, so the standard rotary embedding is
 * used: pair i of a row at position p, (a, b), becomes
 *     (a * cos[p][i] - b * sin[p][i],  b * cos[p][i] + a * sin[p][i]),
 * the pairs being dims (i, i + D/2) for ATTN_ROPE_HALF and (2i, 2i + 1) for
 * ATTN_ROPE_INTERLEAVED.
 *
 *   cos, sin  DEVICE fp32 [max_pos, D/2] tables (row p: position p), 16-byte
 *             aligned; read-only.
 *   max_pos   rows of both tables.
 *   style     ATTN_ROPE_NONE (or cos == NULL): no rotation.
 *
 * Positions follow the causal alignment.  Prefill: key j of a sequence sits
 * at j and query i at Lkv - Lq + i (a dense call with Lq > Lkv returns
 * ATTN_ERR_INVALID_ARG; a packed sequence with more queries than keys is
 * flagged ATTN_ERR_DEVICE_BOUNDS).  The keys are rotated once per call by a
 * pass of their own into k_out (or the library workspace, grown like the
 * decode workspace and shared with it), the queries by a second pass into the
 * workspace, then the attention kernel streams the rotated copies.  Such a
 * call needs 256 KiB + (k_out ? 0 : rows of k * D * 2) + rows of q * D * 2
 * bytes of workspace; during CUDA graph capture it is never grown (make one
 * uncaptured call with the largest sizes first), and calls that can overlap
 * on the GPU race on it, as decode calls do.  Decode:
 * only the query is rotated, to kv_len - 1 (token t of attn_decode_multi to
 * kv_len - Lq + t); cached keys must be stored already rotated.  Every
 * position must be below max_pos: calls whose Lkv (prefill) or Lmax (decode)
 * exceeds max_pos return ATTN_ERR_INVALID_ARG.
 */
typedef enum attn_rope_style { ATTN_ROPE_NONE = 0, ATTN_ROPE_HALF = 1, ATTN_ROPE_INTERLEAVED = 2 } attn_rope_style;

typedef struct attn_rope {
  const float* cos;
  const float* sin;
  int max_pos;
  int style;
  void* k_out;  /* prefill only, optional: DEVICE bf16 buffer shaped like k (16-byte aligned) that receives the
                   rotated keys -- e.g. to append them to a KV cache; NULL = the library's workspace holds them */
} attn_rope;

/*
 * attn_fwd -- prefill attention over dense [batch, heads, seq_len, head_dim]
 * tensors (the Q/K/V shape of "Что такое kernel fusion и как он применяется в
 * LLM serving?", §2, and the chain of Operator Fusion §3.4).
 *
 *   q    bf16 [B, Hq,  Lq,  D]  contiguous
 *   k    bf16 [B, Hkv, Lkv, D]  contiguous
 *   v    bf16 [B, Hkv, Lkv, D]  contiguous
 *   out  bf16 [B, Hq,  Lq,  D]  written
 *   lse  fp32 [B, Hq,  Lq]      written; may be NULL (then not written)
 *   scale   multiplies the logits (pass 1/sqrt(D) for the standard chain), before
 *           the mask is added; any finite value, zero (uniform weights over the
 *           visible keys) and negative values included (NaN or +-inf:
 *           ATTN_ERR_INVALID_ARG).  Every entry point treats scale this way.
 *   causal  0 = no mask, 1 = bottom-right-aligned causal mask
 *
 * Runs on the tensor cores (tcgen05 MMAs with TMEM accumulators, TMA-fed
 * shared-memory tiles).  Returns an attn_status.
 */
int attn_fwd(const void* q, const void* k, const void* v, void* out, float* lse,
             int B, int Hq, int Hkv, int Lq, int Lkv, int D, float scale, int causal,
             void* stream);

/*
 * attn_fwd_params / attn_fwd_ex -- prefill with every option.
 *
 * Dense layout (cu_seqlens_q == NULL): as attn_fwd; Lq/Lkv are the lengths.
 *
 * Packed variable-length layout (cu_seqlens_q != NULL and cu_seqlens_k != NULL):
 *   q    bf16 [total_q, Hq,  D]   (token-major, heads, head_dim)
 *   k/v  bf16 [total_k, Hkv, D]
 *   out       [total_q, Hq,  D]
 *   lse  fp32 [total_q, Hq]       may be NULL
 *   cu_seqlens_q/k  DEVICE int32 [B + 1], non-decreasing, cu[0] = 0,
 *                   cu_q[B] == total_q, cu_k[B] == total_k; sequence s owns
 *                   rows cu[s] .. cu[s+1]-1 and is an independent problem.
 *   Lq, Lkv   upper bounds of the per-sequence query / key lengths.
 *   B         number of sequences.
 *
 * out_dtype selects bf16 (ATTN_DTYPE_BF16) or fp32 (ATTN_DTYPE_F32) output.
 */
typedef struct attn_fwd_params {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  int B, Hq, Hkv, Lq, Lkv, D;
  float scale;
  int causal;
  int out_dtype;
  const int* cu_seqlens_q;
  const int* cu_seqlens_k;
  int total_q, total_k;
  void* stream;
  attn_rope rope;  /* optional; zero-initialised = no rotation */
} attn_fwd_params;

int attn_fwd_ex(const attn_fwd_params* p);

/*
 * attn_decode -- single-token decode over a KV cache ("Оптимизация Decoder
 * Attention для LLM на GPU", section on the structure of attention in decoding
 * mode: the new token's query against all cached keys, softmax, times V),
 * split along the KV sequence (Flash-Decoding, Operator Fusion FAQ Q4) and
 * merged by a log-sum-exp combine.
 *
 *   q        bf16 [B, Hq, D]
 *   kcache   bf16 [B, Hkv, Lmax, D]
 *   vcache   bf16 [B, Hkv, Lmax, D]
 *   kv_lens  DEVICE int32 [B]; sequence b attends to cache rows 0..kv_lens[b]-1.
 *            A value outside [0, Lmax] is clamped into it and flagged as
 *            ATTN_ERR_DEVICE_BOUNDS in the device status word.  kv_len == 0
 *            gives O = 0, lse = -inf.
 *   out      bf16 [B, Hq, D]
 *   lse      fp32 [B, Hq]  may be NULL
 *
 * Uses a library-owned split-KV workspace on the current device, grown on
 * demand with cudaMalloc (see attn_release_workspace); during CUDA graph
 * capture it is never grown (a call that would need a larger one returns
 * ATTN_ERR_INVALID_ARG: make one uncaptured call with the largest sizes
 * first).  Decode calls on one device share that workspace, so calls that can
 * overlap on the GPU (different streams with no ordering) race on it.
 * One kernel is enqueued: persistent CTAs (three per SM when a CTA serves up
 * to 4 query heads, two with 8) each stream an equal slice of the flattened
 * key space of all rows (every row also charged a fixed cost for its
 * piece-end work), and the CTA that lands a row's last partial merges that
 * row's partials.
 */
int attn_decode(const void* q, const void* kcache, const void* vcache, const int* kv_lens,
                void* out, float* lse, int B, int Hq, int Hkv, int Lmax, int D, float scale,
                void* stream);

/*
 * attn_decode_params / attn_decode_ex -- decode with every option.
 *   out_dtype     ATTN_DTYPE_BF16 or ATTN_DTYPE_F32
 *   chunk         0 = default; otherwise the smallest number of keys one CTA's
 *                 slice of the key space may hold (default 64), in
 *                 [1, 1048576]: smaller values spread short problems over more
 *                 CTAs and split rows into more partials.  The slices never
 *                 number fewer than the rows that have keys (while CTAs
 *                 last), so a short problem still runs a row per CTA.
 * Rows: B * Hkv * (Hq / Hkv / g) must stay at or below 65534, g being the
 * number of query heads one CTA serves (the largest of 8, 4, 2, 1 dividing
 * Hq / Hkv); otherwise ATTN_ERR_UNSUPPORTED.
 */
typedef struct attn_decode_params {
  const void* q;
  const void* kcache;
  const void* vcache;
  const int* kv_lens;
  void* out;
  float* lse;
  int B, Hq, Hkv, Lmax, D;
  float scale;
  int out_dtype;
  int chunk;
  void* stream;
  attn_rope rope;  /* optional; zero-initialised = no rotation */
} attn_decode_params;

int attn_decode_ex(const attn_decode_params* p);

/*
 * attn_decode_paged_params / attn_decode_paged -- decode over a paged KV cache
 * (the serving form of the cache: fixed-size pages from a shared pool, listed
 * per sequence in a block table, as in PagedAttention, which "Что такое kernel
 * fusion и как он применяется в LLM serving?" §6 names).  Same computation
 * and results as attn_decode_ex on the cache the pages describe.
 *
 *   kpages, vpages  bf16 [num_pages, Hkv, page_size, D]: page g of kv head h
 *                   holds page_size consecutive key (value) rows
 *   block_table     DEVICE int32 [B, max_pages]: entry (b, i) is the pool page
 *                   holding keys i*page_size .. (i+1)*page_size-1 of sequence b
 *   kv_lens         DEVICE int32 [B], at most max_pages * page_size (clamped
 *                   and flagged otherwise, as in attn_decode)
 *   page_size       keys per page, 8 .. 65536 (any value, not only powers of 2)
 *   max_pages       columns of block_table; num_pages rows of the pool.  Only
 *                   the entries of pages that hold keys of a sequence (the
 *                   first ceil(kv_len / page_size)) are read; the rest may hold
 *                   anything (e.g. -1 padding).  A page id read outside
 *                   [0, num_pages) is flagged ATTN_ERR_DEVICE_BOUNDS in the
 *                   device status word and page 0 is read instead.
 *   other fields    as attn_decode_params (q, out, lse, B, Hq, Hkv, D, scale,
 *                   out_dtype, chunk, stream); same workspace as attn_decode_ex.
 */
typedef struct attn_decode_paged_params {
  const void* q;
  const void* kpages;
  const void* vpages;
  const int* block_table;
  const int* kv_lens;
  void* out;
  float* lse;
  int B, Hq, Hkv, D;
  int page_size, max_pages, num_pages;
  float scale;
  int out_dtype;
  int chunk;
  void* stream;
  attn_rope rope;  /* optional; zero-initialised = no rotation */
} attn_decode_paged_params;

int attn_decode_paged(const attn_decode_paged_params* p);

/*
 * attn_decode_multi_params / attn_decode_multi -- decode of several new tokens
 * per sequence at once (multi-token or speculative decode), on the tensor
 * cores.  The decoder page ("Оптимизация Decoder Attention для LLM на GPU",
 * "Техника выжимания производительности", item 1: token-level parallelism)
 * processes several query tokens of a step together so that each K/V block is
 * loaded once for all of them and the tensor cores have work.
 *
 *   q        bf16 [B, Hq, Lq, D]   the Lq new tokens of every sequence
 *   kcache   bf16 [B, Hkv, Lmax, D]
 *   vcache   bf16 [B, Hkv, Lmax, D]
 *   kv_lens  DEVICE int32 [B]: the number of cached keys of sequence b,
 *            INCLUDING the Lq new tokens, whose keys and values must already
 *            be in rows kv_len-Lq .. kv_len-1.  New token t (0-based) sits at
 *            position kv_len - Lq + t and attends to keys 0 .. kv_len - Lq + t
 *            (the bottom-right causal mask of attn_fwd with Lkv = kv_len).
 *            Rows at or past kv_len are never read.  A value outside
 *            [0, Lmax] is clamped and flagged ATTN_ERR_DEVICE_BOUNDS; a token
 *            that sees no key (kv_len < Lq) gets O = 0, lse = -inf.
 *   out      [B, Hq, Lq, D]  bf16, or fp32 when out_dtype = ATTN_DTYPE_F32
 *   lse      fp32 [B, Hq, Lq]  may be NULL
 *   Lq       1 .. 128 / (Hq / Hkv): every query row of one kv head (the heads
 *            of its group times the tokens) forms one 128-row MMA tile;
 *            larger products return ATTN_ERR_UNSUPPORTED.
 * B * Hkv must stay at or below 65534 and B * Hq * Lq below 2^31
 * (ATTN_ERR_UNSUPPORTED otherwise).  Uses the split-KV workspace of
 * attn_decode (same growth, capture and concurrency rules).  One kernel is
 * enqueued: persistent CTAs (one per SM) each stream an equal share of all
 * sequences' 128-key tiles, and the CTA that lands an item's last partial
 * merges its partials.
 */
typedef struct attn_decode_multi_params {
  const void* q;
  const void* kcache;
  const void* vcache;
  const int* kv_lens;
  void* out;
  float* lse;
  int B, Hq, Hkv, Lq, Lmax, D;
  float scale;
  int out_dtype;
  void* stream;
  attn_rope rope;  /* optional; zero-initialised = no rotation */
} attn_decode_multi_params;

int attn_decode_multi(const attn_decode_multi_params* p);

/*
 * attn_decode_workspace_bytes -- bytes of split-KV workspace a decode call
 * with these sizes needs (0 on invalid sizes).  It depends on Hq / Hkv, D and
 * the current device's SM count (148 assumed when no device is visible), not
 * on B, Lmax or chunk: 256 KiB of counters plus two partials per CTA.
 */
unsigned long long attn_decode_workspace_bytes(int B, int Hq, int Hkv, int Lmax, int D, int chunk);

/*
 * ---------------------------------------------------------------------------
 * A serving step around a paged cache.  The calls below go together: pages and
 * slots for the step's tokens (attn_page_step), norm and rotation of their q and
 * k (attn_qk_norm_rope), their rows into a cache held in 4 bits
 * (attn_kv_append_q4), then decode over it (attn_decode_q4) or, for prefill over
 * cached keys, the rows read back as bf16 (attn_kv_gather_q4) for attn_fwd_ex.
 * (The source pages name fused RMSNorm + RoPE, "Что такое kernel fusion и как он
 * применяется в LLM serving?" §3.5, and PagedAttention, §6; they give no formulas.)
 * None of them allocates or synchronises, so all can be captured into CUDA graphs
 * (attn_decode_q4 without a workspace of the caller's: see there).  For all of
 * them every host-visible size is checked before anything is enqueued, and a row
 * whose index the device finds out of range is skipped and flagged
 * ATTN_ERR_DEVICE_BOUNDS in the device status word.
 * ---------------------------------------------------------------------------
 */

/*
 * attn_page_step -- block tables and slot maps of a step, from request lengths,
 * on the GPU (no host round trip).
 *
 * Row b holds a = kv_lens[b] keys on the first ceil(a / page_size) pages of its
 * block-table row.  The step keeps the first keep_lens[b] keys and adds
 * new_lens[b] tokens: a decode step adds one, a prompt its length, refused draft
 * tokens are dropped by keeping less, a finished request keeps 0.  Pages past the
 * row's new length are given back, missing ones are taken, kept ones stay.
 *
 *   kv_lens      int32 [B]  in: a; out: keep + new
 *   keep_lens    int32 [B]  0 <= keep <= a; NULL: keep everything
 *   new_lens     int32 [B]  >= 0; NULL: nothing is added
 *   block_table  int32 [B, max_pages]  entries of pages taken are written, those of
 *                pages given back become -1, the others stay as they are
 *   free_pages   int32 [num_pages]  the stack of free pages: entries below
 *                *free_count; pages are taken from its end in row-major order and
 *                given back in reverse, so that taking back a step's tokens restores
 *                it exactly.  Entries at and above the count hold anything.
 *   free_count   int32 [1]  in/out
 *   cu_new       int32 [B + 1]  running sum of new_lens (cu_seqlens_q of the step);
 *                may be NULL
 *   slots        int32 [max_tokens]  token i of the step (rows in order, positions
 *                rising): page * page_size + offset within the page, what
 *                attn_kv_append_q4 takes; -1 past the last token; may be NULL
 *   positions    int32 [max_tokens]  its position, what attn_qk_norm_rope takes; -1
 *                past the last token; may be NULL
 *
 * All or nothing: lengths out of range, a row beyond max_pages pages or more than
 * max_tokens tokens while slots or positions is given (ATTN_ERR_DEVICE_BOUNDS), or
 * too few free pages (ATTN_ERR_DEVICE_POOL; pages given back by the same step
 * count) leave lengths, table and stack as they were; every slot and position is
 * then -1 and cu_new 0.  A page id out of [0, num_pages) met on the way, taken, kept or
 * given back, is flagged ATTN_ERR_DEVICE_BOUNDS, and its tokens' slots are -1.  The
 * buffers must not overlap, except that an input not written may be passed twice; a
 * page stands in one row at most.  B == 0: nothing is done.
 *
 * B at most 8192; num_pages * page_size, B * max_pages and max_pages * page_size
 * below 2^31 (ATTN_ERR_UNSUPPORTED otherwise).  int32 pointers are 4-byte aligned
 * here and in the calls below.
 */
typedef struct attn_page_step_params {
  int* kv_lens;
  const int* keep_lens;
  const int* new_lens;
  int* block_table;
  int* free_pages;
  int* free_count;
  int* cu_new;
  int* slots;
  int* positions;
  int B, page_size, max_pages, num_pages, max_tokens;
  void* stream;
} attn_page_step_params;

int attn_page_step(const attn_page_step_params* p);

/*
 * attn_qk_norm_rope -- RMS norm of every query and key head over its D elements,
 * and the rotation of attn_rope, in one pass:
 *     y = x / sqrt(mean(x^2) + eps) * weight,   then (a, b) -> (a cos - b sin, b cos + a sin),
 * in fp32, rounded to bf16 once.  Rows are addressed by strides, in elements, of
 * sequence, token and head, so q and k may be views of a fused projection's output
 * and either [B, H, L, D] or [B, L, H, D]; a row's D elements are contiguous.
 *
 *   q, k          bf16, B sequences of L tokens with Hq (Hkv) heads; Hkv = 0: no k
 *   q_out, k_out  bf16; either apart from every input, or exactly the rows of q (of k)
 *                 itself (same pointer and strides: in place)
 *   q_weight, k_weight  bf16 [D], or NULL for ones
 *   positions     int32 [B, L]; -1 marks a padded row, which is left as it was.  Any
 *                 other value outside [0, max_pos) is flagged and its row left as it
 *                 was.  May be NULL without rotation.
 *   rope          tables and style (k_out unused); ATTN_ROPE_NONE: norm only
 *   eps           finite, >= 0 (a row of zeros with eps = 0 is 0 * inf = NaN)
 * (In fp32 the squares of elements beyond some 10^18 overflow, and such a row is 0; those
 * of elements below some 10^-19 count as 0, which matters where eps does not cover them.)
 * Pointers are 16-byte aligned, strides multiples of 8 elements (that of an axis of one
 * element may be anything).
 */
typedef struct attn_qk_norm_rope_params {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const void* q_weight;
  const void* k_weight;
  const int* positions;
  int B, L, Hq, Hkv, D;
  float eps;
  long long q_stride[3], k_stride[3], q_out_stride[3], k_out_stride[3];
  attn_rope rope;
  void* stream;
} attn_qk_norm_rope_params;

int attn_qk_norm_rope(const attn_qk_norm_rope_params* p);

/*
 * The 4-bit cache.  A pool of num_pages pages, each Hkv * page_size / 16 tiles of
 * 16 keys of one kv head (18 * D bytes a tile, 4.5 bits an element), G = D / 64:
 *     K codes [G][16 keys][32 bytes], V codes alike, then K's and V's fp16 pairs
 *     (scale, minimum) [16 keys][G][2].
 * Byte j of a code row holds dims 2j (low four bits) and 2j + 1 of its group of 64
 * dims; code u reads back as scale * u + minimum.  page_size is a multiple of 16;
 * slot = page * page_size + offset.  The pool is 128-byte aligned.
 *
 * attn_kv_q4_page_bytes -- bytes of one page (0 on invalid sizes).
 */
unsigned long long attn_kv_q4_page_bytes(int page_size, int Hkv, int D);

/*
 * attn_kv_append_q4 -- quantises T rows of k and v into their slots.  Per group of 64
 * dims: minimum = fp16(min x), scale = fp16((max x - min x) / 15), code =
 * clamp(round((x - minimum) / scale), 0, 15), ties to even (0 where scale is 0).  NaN
 * counts as 0, values beyond +-65504 as that.
 *
 *   k, v   bf16 [T, Hkv, D] with strides of token and head in elements (multiples of
 *          8, unless there is one; D contiguous; 16-byte aligned): views of a
 *          projection's output will do
 *   slots  int32 [T]; -1: the row is not written.  Any other slot outside the pool is
 *          flagged and not written.  The slots of one call must differ: rows of the same
 *          slot would be written over each other in no order.
 * T * Hkv below 2^31 (ATTN_ERR_UNSUPPORTED otherwise).
 */
typedef struct attn_kv_append_q4_params {
  const void* k;
  const void* v;
  void* pool;
  const int* slots;
  int T, Hkv, D, page_size, num_pages;
  long long k_stride[2], v_stride[2];
  void* stream;
} attn_kv_append_q4_params;

int attn_kv_append_q4(const attn_kv_append_q4_params* p);

/*
 * attn_kv_gather_q4 -- reads rows back: key kv_starts[b] + i of sequence b becomes row
 * cu_k[b] + i of the packed k and v (the layout of attn_fwd_ex), rounded to bf16, for
 * i < cu_k[b + 1] - cu_k[b].
 *
 *   block_table  int32 [B, max_pages]; only entries of pages read are looked at
 *   cu_k         int32 [B + 1], non-decreasing, cu_k[0] = 0, cu_k[B] <= total_k
 *   kv_starts    int32 [B], or NULL for zeros
 *   k, v         bf16 [total_k, Hkv, D]; rows at and past cu_k[B] stay as they were, and
 *                so do rows of positions or pages out of range, which are flagged
 * total_k * Hkv below 2^31 (ATTN_ERR_UNSUPPORTED otherwise).
 */
typedef struct attn_kv_gather_q4_params {
  const void* pool;
  const int* block_table;
  const int* cu_k;
  const int* kv_starts;
  void* k;
  void* v;
  int B, Hkv, D, page_size, max_pages, num_pages, total_k;
  void* stream;
} attn_kv_gather_q4_params;

int attn_kv_gather_q4(const attn_kv_gather_q4_params* p);

/*
 * attn_decode_q4 -- decode over the 4-bit cache, one or Lq new tokens a sequence, with
 * the masks and results of attn_decode_multi on the values the cache stands for
 * (Lq = 1: of attn_decode).  q is taken as it is (rotated by attn_qk_norm_rope).
 *
 *   q            bf16 [B, Hq, Lq, D]
 *   pool, block_table, page_size, max_pages, num_pages  as above; kv_lens int32 [B], at
 *                most max_pages * page_size (clamped and flagged otherwise).  Only
 *                entries of pages that hold keys are read; a page id outside the pool
 *                is flagged and page 0 read instead.
 *   out, lse     as attn_decode_multi, apart from every input
 *   chunk        0 = default; otherwise the smallest number of keys of one CTA's slice,
 *                in [1, 1048576]
 *   workspace    NULL: a workspace of the library, its own, apart from attn_decode's: made
 *                by the first call on a device, which must not be one that is captured, and
 *                kept until attn_release_workspace; calls that can overlap on the GPU race
 *                on it.  Otherwise a DEVICE buffer of workspace_bytes (at least
 *                attn_decode_q4_workspace_bytes; ATTN_ERR_SCRATCH_TOO_SMALL if not),
 *                16-byte aligned, all zeros before its first call; the calls leave it so.
 *                Calls that can overlap, and graphs that can be replayed at once, each take
 *                a buffer of their own.  After ATTN_ERR_DEVICE_TIMEOUT the caller zeroes it
 *                again.
 * (Hq / Hkv) * Lq at most 128.  Weights are rounded to fp16 before the second product,
 * whose sums are fp32 with truncated adds; with out_dtype = ATTN_DTYPE_F32 they are carried
 * in two fp16 terms and the adds are rounded.
 * A weight is its softmax numerator times V's scale; it is off by 2^-11 (2^-22) of itself,
 * or by 2^-34 of the largest scale among the keys it is taken with (up to 48 neighbours,
 * both groups of 64 dims), whichever is more.
 */
typedef struct attn_decode_q4_params {
  const void* q;
  const void* pool;
  const int* block_table;
  const int* kv_lens;
  void* out;
  float* lse;
  int B, Hq, Hkv, Lq, D;
  int page_size, max_pages, num_pages;
  float scale;
  int out_dtype;
  int chunk;
  void* workspace;
  unsigned long long workspace_bytes;
  void* stream;
} attn_decode_q4_params;

int attn_decode_q4(const attn_decode_q4_params* p);

/* attn_decode_q4_workspace_bytes -- bytes a workspace of attn_decode_q4 needs on the current device (0 on invalid
 * sizes; 152 SMs assumed when no device is visible).  It depends on D and the device only. */
unsigned long long attn_decode_q4_workspace_bytes(int Hq, int Hkv, int Lq, int D);

/*
 * ---------------------------------------------------------------------------
 * A draft step over a paged bf16 cache (the pools of attn_decode_paged).  Several
 * drafted tokens of every sequence are checked at once; the step's tokens are packed,
 * sequence after sequence, as attn_page_step lists them: attn_page_step (slots and
 * positions, cu_new), attn_kv_append_paged (q and k rotated, k and v written),
 * attn_decode_multi_paged, the model's output head, attn_verify_drafts (which drafts
 * stand, the token that follows), attn_page_step again with its keep_lens.
 * attn_rope_tables makes the rotation's tables.  What the serving step's calls promise
 * holds here: no allocation and no synchronisation (attn_decode_multi_paged without a
 * workspace of the caller's: see there), sizes checked before anything is enqueued, rows
 * of indices out of range skipped and flagged ATTN_ERR_DEVICE_BOUNDS.  (The source pages
 * name RoPE and PagedAttention, "Что такое kernel fusion и как он применяется в LLM
 * serving?" §3.5 and §6, and several query tokens of a step at once, "Оптимизация
 * Decoder Attention для LLM на GPU"; they give no formulas.)
 * ---------------------------------------------------------------------------
 */

/*
 * attn_rope_tables -- rotary tables: row r of cos and sin holds
 *     amplitude * cos((start + r) f_i),  amplitude * sin((start + r) f_i),
 * i < rotary_dim / 2, with f_i = base^(-2i / rotary_dim) radians a position, changed for
 * contexts longer than the model was trained on by
 *     ATTN_ROPE_SCALE_NONE    nothing
 *     ATTN_ROPE_SCALE_LINEAR  f_i / factor
 *     ATTN_ROPE_SCALE_BASE    base * factor^(R / (R - 2)) for base, R = rotary_dim: the slowest
 *                             pair is slowed by factor, the fastest not at all
 *     ATTN_ROPE_SCALE_TURNS   f_i (g + (1 - g) / factor), g = clamp((t - low) / (high - low), 0, 1)
 *                             with t = context f_i / (2 pi), the turns over the trained context
 *     ATTN_ROPE_SCALE_INDEX   the same with g = 1 - clamp((i - a) / max(b - a, 0.001), 0, 1), where
 *                             a = max(0, floor(c(high))) and b = min(R - 1, ceil(c(low))),
 *                             c(t) = (R / 2) ln(context / (2 pi t)) / ln(base): the pair of t turns
 * Angles are kept as fractions of a turn in 64 bits, so that far positions are about as exact
 * as near ones: within 2^-22 + 2^-50 of the angle, times the amplitude.  (On the ramps of TURNS and
 * INDEX g is rounded too, in 64 bits: TURNS' by 2^-49 high / (high - low).)
 *
 *   cos, sin    fp32 [rows, rotary_dim / 2], 16-byte aligned, apart from each other
 *   rotary_dim  16, 32 .. 128: the rotated dims of a head.  Tables of rotary_dim = D are
 *               those of attn_rope; attn_kv_append_paged takes narrower ones too.
 *   start       >= 0, start + rows below 2^31: tables can grow with the longest request
 *   base        > 1 (also once factor has changed it); factor > 0; 0 < low < high and context > 0 where they are used; all
 *               finite, the amplitude too (ATTN_ERR_INVALID_ARG otherwise)
 * rows == 0: nothing is done.
 */
typedef enum attn_rope_scaling {
  ATTN_ROPE_SCALE_NONE = 0,
  ATTN_ROPE_SCALE_LINEAR = 1,
  ATTN_ROPE_SCALE_BASE = 2,
  ATTN_ROPE_SCALE_TURNS = 3,
  ATTN_ROPE_SCALE_INDEX = 4
} attn_rope_scaling;

typedef struct attn_rope_tables_params {
  float* cos;
  float* sin;
  int rows, start, rotary_dim, scaling;
  double base, factor, context, low, high, amplitude;
  void* stream;
} attn_rope_tables_params;

int attn_rope_tables(const attn_rope_tables_params* p);

/*
 * attn_kv_append_paged -- T rows of k, rotated, and of v into their slots of the pages, and
 * the same tokens' q rotated, in one pass.  The first rotary_dim dims of a head turn as in
 * attn_rope, pairs being dims (i, i + rotary_dim / 2) or (2i, 2i + 1), in fp32, rounded to
 * bf16 once; the others, and v, are copied bit for bit.
 *
 *   k, v     bf16 [T, Hkv, D] with strides of token and head in elements (multiples of 8,
 *            unless there is one; D contiguous; 16-byte aligned): views of a projection's
 *            output will do
 *   kpages, vpages  bf16 [num_pages, Hkv, page_size, D], page_size at least 1 here
 *   slots    int32 [T], page * page_size + offset; -1: k and v of this token are not written.
 *            Any other slot outside the pool is flagged and not written.  The slots of one
 *            call must differ: rows of the same slot would be written over each other in no
 *            order.
 *   rope     tables [max_pos, rotary_dim / 2] and style (k_out unused); ATTN_ROPE_NONE:
 *            nothing turns, and rotary_dim is not looked at
 *   positions  int32 [T]; -1 marks a padded token, of which nothing is written.  Any other
 *            value outside [0, max_pos) is flagged and its token left out alike.  May be NULL
 *            without rotation.
 *   q, q_out bf16 [T, Hq, D] with strides, both NULL when there is no q (Hq = 0); they go
 *            with a rotation
 *   k_out    bf16 [T, Hkv, D] with strides, or NULL: the rotated rows as well, for attn_fwd_ex
 *            over a prompt's own keys, whatever the slot; goes with a rotation
 *            q_out and k_out are either apart from every input, or exactly the rows of q (of k)
 *            itself (same pointer and strides).  The pools are apart from everything else.
 * rotary_dim is a multiple of 16, at most D (ATTN_ERR_UNSUPPORTED otherwise); num_pages *
 * page_size below 2^31, Hq + 2 Hkv at most 65535.
 */
typedef struct attn_kv_append_paged_params {
  const void* k;
  const void* v;
  void* kpages;
  void* vpages;
  const int* slots;
  const int* positions;
  const void* q;
  void* q_out;
  void* k_out;
  int T, Hq, Hkv, D, page_size, num_pages, rotary_dim;
  long long k_stride[2], v_stride[2], q_stride[2], q_out_stride[2], k_out_stride[2];
  attn_rope rope;
  void* stream;
} attn_kv_append_paged_params;

int attn_kv_append_paged(const attn_kv_append_paged_params* p);

/*
 * attn_decode_multi_paged -- attn_decode_multi over pages, with as many new tokens of each
 * sequence as it has, packed.  q is taken as it is (rotated by attn_kv_append_paged).
 *
 *   q, out       [T, Hq, D]: bf16, and bf16 or fp32; lse fp32 [T, Hq] may be NULL
 *   cu_new       DEVICE int32 [B + 1]: the tokens of sequence b are rows cu_new[b] ..
 *                cu_new[b + 1] - 1.  A sequence without any is left out (a length of its out of
 *                range is flagged all the same).  Offsets that
 *                fall, leave [0, T] or give a sequence more than max_new tokens are flagged,
 *                and its rows left as they were, as are rows of no sequence.
 *   max_new      the most new tokens of a sequence, 1 .. 128 / (Hq / Hkv)
 *                (ATTN_ERR_UNSUPPORTED above)
 *   kpages, vpages, block_table, max_pages, num_pages  as attn_decode_paged
 *   page_size    a multiple of 8, 8 .. 65536 (ATTN_ERR_UNSUPPORTED for others in that range)
 *   kv_lens      DEVICE int32 [B], at most max_pages * page_size (clamped and flagged
 *                otherwise): the keys of sequence b, its n = cu_new[b + 1] - cu_new[b] new
 *                tokens' own among them.  Token t sits at kv_len - n + t and attends to keys
 *                0 .. kv_len - n + t; one that sees no key gets O = 0, lse = -inf.  Keys at or
 *                past kv_len may hold anything.  (Keys that a token does not see because they
 *                are later tokens' own count with weight 0, so a NaN or an infinity in their
 *                values still reaches it, unless it sees no key at all.)  A NaN among a head's
 *                logits of a token, or one of +infinity, gives NaN in its O and its lse, and in
 *                no other row's.
 *   out          apart from every input.  Weights are rounded to bf16 before they meet V.
 *   workspace    as attn_decode_q4: NULL for one of the library, its own, made by the first
 *                call on a device, which must not be one that is captured; or a DEVICE buffer
 *                of at least attn_decode_multi_paged_workspace_bytes, 16-byte aligned, all
 *                zeros before its first call.  Calls that can overlap, and graphs that can be
 *                replayed at once, each take a buffer of their own.  After
 *                ATTN_ERR_DEVICE_TIMEOUT the caller zeroes it again.
 * B * Hkv at most 65534, num_pages * Hkv and T * Hq below 2^31 (ATTN_ERR_UNSUPPORTED
 * otherwise).
 */
typedef struct attn_decode_multi_paged_params {
  const void* q;
  const void* kpages;
  const void* vpages;
  const int* block_table;
  const int* kv_lens;
  const int* cu_new;
  void* out;
  float* lse;
  int B, T, Hq, Hkv, D, max_new;
  int page_size, max_pages, num_pages;
  float scale;
  int out_dtype;
  void* workspace;
  unsigned long long workspace_bytes;
  void* stream;
} attn_decode_multi_paged_params;

int attn_decode_multi_paged(const attn_decode_multi_paged_params* p);

/* attn_decode_multi_paged_workspace_bytes -- bytes a workspace of attn_decode_multi_paged needs on the current device
 * (0 on invalid sizes; 152 SMs assumed when no device is visible).  A buffer can serve calls of several sizes if it is
 * large enough for each. */
unsigned long long attn_decode_multi_paged_workspace_bytes(int Hq, int Hkv, int max_new, int D);

/*
 * attn_verify_drafts -- which drafted tokens stand, and the token that follows them, so that
 * every token comes out as if drawn from the target's probabilities.  Sequence b has n drafts
 * x_0 .. x_{n-1} drawn from q_0 .. q_{n-1}, and rows p_0 .. p_n of the target.  Draft i stands
 * if those before it do and u_i q_i(x_i) < p_i(x_i) (products and comparison exact).  With r
 * standing drafts the next token has the weights max(p_r - q_r, 0) if r < n, or p_n if all
 * stand, and is the lowest j with w_0 + .. + w_j > u_K (w_0 + .. + w_{V-1}).  Weights that are
 * not positive finite numbers count as 0; where p_r is nowhere above q_r the weights are p_r;
 * where u_K is 1 or more, or NaN, the token is the last one with any weight.
 *
 *   draft_tokens  int32 [B, K]; K may be 0.  A token outside [0, V) does not stand, and is flagged.
 *   target_probs  bf16 or fp32 (dtype) rows of V probabilities, strides in elements.  With
 *                 cu_target: [total, V], rows cu_target[b] .. cu_target[b + 1] - 1 of sequence b
 *                 (n = their number - 1; a sequence without rows gets no token); target_stride[1]
 *                 is a row's.  Without: [B, K + 1, V], strides of sequence and row.
 *   draft_probs   [B, K, V] of the same type, strides of sequence and row; or NULL for drafts
 *                 that were not drawn (looked up, or the drafter's likeliest token): q_i is 1 at x_i
 *   uniforms      fp32 [B, K + 1], random numbers in [0, 1): entry i < K for draft i, entry K for
 *                 the token that follows
 *   cu_target     int32 [B + 1] or NULL.  Offsets that fall, leave [0, total] or give more than
 *                 K + 1 rows are flagged, and the sequence counts as one without rows.
 *   draft_lens    int32 [B], n of every sequence, without cu_target; NULL: K.  A value outside
 *                 [0, K] is clamped and flagged.
 *   tokens        int32 [B, K + 1]: the drafts that stand, the token that follows them, then -1
 *   accepted      int32 [B]: r
 *   kv_lens, keep_lens  int32 [B], both or neither: keep = kv_lens - (n - r), what attn_page_step
 *                 takes to drop the refused drafts' keys (kv_lens as the step that added the n + 1
 *                 tokens left them)
 * A row that holds no weight at all, or weights whose sum passes fp32's range, gives -1 and is
 * flagged.  The sums are exact to 2^-39 of themselves for V up to 2^20, to 2^-34 beyond (sums below
 * 2^-100: to fp32's smallest number), and the same every time.  Outputs are apart from inputs and from each other.  K
 * below 2^20, V below 2^30, B (K + 1) below 2^28 (ATTN_ERR_UNSUPPORTED otherwise).
 */
typedef struct attn_verify_drafts_params {
  const int* draft_tokens;
  const void* target_probs;
  const void* draft_probs;
  const float* uniforms;
  const int* cu_target;
  const int* draft_lens;
  const int* kv_lens;
  int* tokens;
  int* accepted;
  int* keep_lens;
  int B, K, V, total, dtype;
  long long target_stride[2], draft_stride[2];
  void* stream;
} attn_verify_drafts_params;

int attn_verify_drafts(const attn_verify_drafts_params* p);

/*
 * attn_get_device_status -- synchronises `stream`, then returns and clears the
 * current device's status word (ATTN_OK if no kernel flagged a problem since
 * the last read).  Of several problems it holds the first, but
 * ATTN_ERR_DEVICE_TIMEOUT takes the place of any other: a decode that gave up may
 * leave partial results in its workspace, so the outputs of every call since the
 * last read are to be taken as wrong.  Reading it synchronises the device and
 * zeroes the library's workspaces; a caller's own are the caller's to zero.
 * Returns ATTN_ERR_CUDA if the synchronisation fails.
 */
int attn_get_device_status(void* stream);

/* attn_status_string -- static, NUL-terminated name of a status code. */
const char* attn_status_string(int status);

/*
 * attn_release_workspace -- frees the current device's split-KV workspaces.
 * The caller must ensure no decode call using it is still in flight (for
 * example by synchronising the streams it was used on).
 */
void attn_release_workspace(void);

/*
 * attn_decode_noalloc -- attn_decode_ex for callers that must not allocate
 * device memory.  (The source pages have no counterpart: this entry point is
 * an integration aid, not part of the attention method.)
 *
 * Who needs it: code that runs while a CUDA graph is being captured (where a
 * cudaMalloc is not allowed), serving engines that reserve nearly all of HBM
 * up front for KV caches and route every allocation through their own pool,
 * and latency-critical paths that cannot afford the device-wide
 * synchronisation cudaMalloc/cudaFree can cause.  attn_decode_ex may grow its
 * workspace with cudaMalloc on the first call with a larger problem; this
 * call never does.
 *
 * Same arguments, layouts and results as attn_decode_ex.  Its scratch is a
 * fixed 4 MiB buffer compiled into the library (a file-scope __device__
 * array): every GPU on which the library's kernels are loaded holds that
 * buffer until the process exits, whether or not this call is used.  The
 * buffer holds 256 KiB of work counters followed by the split-KV partials,
 * two per CTA of the persistent launch (2.5 MiB at most on a 152-SM GB300).
 * A problem that does not fit -- more than 65534 (b, kv head, head group)
 * rows, or partials beyond the buffer on a device with more SMs -- returns
 * ATTN_ERR_SCRATCH_TOO_SMALL before anything is enqueued.
 *
 * No call allocates: no cudaMalloc, no cudaFree, no allocating library
 * routine.  The first call on a device looks up the buffer's device address
 * (cudaGetSymbolAddress, once per device, with that device current) and
 * zeroes the counter area (cudaMemset, then a device synchronise); make that
 * first call outside any stream capture (a first call on a capturing stream
 * returns ATTN_ERR_INVALID_ARG and leaves the capture untouched).  The kernel leaves the counters at
 * zero after every call, and every partial is written before it is read in
 * the same call.  All calls share the one buffer and it keeps the last call's
 * contents: two calls that can overlap on the GPU (different streams with no
 * ordering between them) race on it and may return wrong results.  Order such
 * calls on one stream.
 */
int attn_decode_noalloc(const attn_decode_params* p);

/*
 * attn_selftest_wait_timeout -- exercises the failure detection every kernel
 * carries, without a GPU fault.  (The pages have no counterpart; it exists so
 * that the device-timeout path can be tested.)  Enqueues a one-thread kernel
 * that waits on an mbarrier nothing arrives on, using the same bounded wait
 * as every pipeline stage but a limit of limit_us microseconds (1 .. 1000000);
 * when it expires the kernel records ATTN_ERR_DEVICE_TIMEOUT in the device
 * status word, exactly as a stalled pipeline would, and returns.  The context
 * stays usable; attn_get_device_status() then reports and clears the status.
 * Returns ATTN_ERR_INVALID_ARG for a limit out of range.
 */
int attn_selftest_wait_timeout(unsigned int limit_us, void* stream);

/* attn_version -- library version as major*10000 + minor*100 + patch. */
int attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_H */
