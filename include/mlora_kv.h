/*
 * mlora_kv.h -- C ABI of libmlora.so: a paged key/value cache held in 8 bits,
 * the operators on it, page tables made on the GPU, and rollouts of the transformer-block model
 * (mlora_tf.h) that call them.  The pages describe rollouts as a service
 * beside training (OpenTinker, "Multi-LoRA rollout") and fix no cache format;
 * everything below is this library's own.
 *
 * The cache.  A page holds the keys and the values of MLORA_KV_PAGE = 64
 * consecutive tokens of one sequence, for every key/value head, as e4m3 bytes
 * (4 exponent bits, 3 mantissa bits, largest value 448, no infinity) with one
 * fp32 scale per (page, head) for the keys and one for the values:
 *     x = scale * e4m3 byte,   scale = 2^e, e >= MLORA_KV_MIN_EXP.
 * A power of two makes the division by the scale exact, so every stored value
 * is the input rounded once to e4m3 (relative error at most 2^-4 for values
 * of at least 2^-6 scale), and a scale that grows moves stored values
 * without rounding them again unless they fall below 2^-6 of the new scale.
 * Sequence s owns the pages page_table[s * max_pages + 0, 1, ..]: position p
 * lies in page p / 64.  Pages may be shared by sequences for reading; a page
 * that a call writes must belong to one sequence of that call.
 *
 * Byte order inside the [64 x head_dim] tile of a (page, head), hd = head_dim:
 *   k: token j, dim c at  j hd + ((c / 16) ^ s) 16 + c % 16,  s = 4 (j % 2) if hd = 128, else 0
 *   v: token j, dim c at  (j / 4) 4 hd + ((c / 4) ^ 2 (j / 4 % 4)) 16 + 4 (c % 4) + j % 4
 * (a thread of the attention kernel finds the bytes of its matrix fragments
 * side by side, and eight threads' 16-byte reads touch distinct banks).
 *
 * Rows.  Every call takes rows of queries, keys or values for a set of
 * sequences.  Sequence s has the n_s rows row_off[s] .. row_off[s+1]-1, or
 * row s alone where row_off is NULL; they are its newest tokens: row i of the
 * n_s sits at position kv_len[s] - n_s + i, kv_len[s] being the sequence's
 * length with these rows counted.  kv_len[s] = 0 marks an empty slot: its
 * rows have no position.  Rows at and behind row_off[n_seqs] are not touched.
 *
 * Conventions are those of mlora.h: return codes, mlora_last_error(), device
 * buffers of the current device owned by the caller and never kept, work
 * queued on the caller's stream.  No call allocates or synchronises, so all
 * can be captured into a CUDA graph.  What only the device sees never traps:
 * a sequence with kv_len < 0 or beyond max_pages * 64 (or beyond max_len), n_s
 * < 0, > max_rows or > kv_len > 0, rows outside 0 .. n_rows-1, or a page id
 * outside 0 .. n_pages-1 raises bit 0 of *status; append and read skip it (a
 * bad page: that page), attention writes NaN to those of its rows that lie in
 * range.  A device wait that exceeds its bound raises bit 1.
 */
#ifndef MLORA_KV_H
#define MLORA_KV_H

#include "mlora_tf.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLORA_KV_PAGE 64
#define MLORA_KV_MIN_EXP (-100)
/* An attention workspace that serves every shape. */
#define MLORA_KV_WORKSPACE_BYTES (32 << 20)

/* A pool of pages (DEVICE buffers).  k, v: n_pages * n_kv_heads * 64 *
 * head_dim bytes, 16-byte aligned; scales: n_pages * n_kv_heads. */
typedef struct {
    uint8_t* k;
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    int32_t* status;       /* DEVICE int32 (may be NULL): bits raised by the kernels (above)  */
    int32_t n_pages;       /* >= 1                                    */
    int32_t n_kv_heads;    /* 1 .. 1024                               */
    int32_t head_dim;      /* 64 or 128                               */
} mlora_kv_cache;

/* The sequences of a call (DEVICE int32 arrays). */
typedef struct {
    const int32_t* page_table;   /* [n_seqs x max_pages]                               */
    const int32_t* kv_len;       /* [n_seqs]                                           */
    const int32_t* row_off;      /* [n_seqs + 1], or NULL: one row a sequence          */
    int64_t n_rows;              /* rows of the row arrays                             */
    int32_t n_seqs;              /* >= 0                                               */
    int32_t max_pages;           /* >= 1                                               */
    int32_t max_rows;            /* upper bound of n_s (1 where row_off is NULL); 0: nothing to do */
} mlora_kv_seqs;

/* Write the rows' keys and values into the cache.  k, v: DEVICE rows of
 * n_kv_heads * head_dim elements of `dtype` (mlora_dtype), k_stride / v_stride
 * elements apart (>= n_kv_heads * head_dim).  Pointers and row distances are
 * multiples of 16 bytes.  For each (page, head) that gets new rows, and for K
 * and V apart:
 *     a = largest finite |x| of the new rows in the page
 *     need = the smallest e >= MLORA_KV_MIN_EXP with a <= 448 * 2^e
 *     e = max(need, the page's exponent) if the page holds older positions of
 *         the sequence, else need
 * older positions' bytes are moved to the new scale (rounded to nearest even
 * where they become subnormal) if it grew; each new x is stored as
 * e4m3(x * 2^-e), to nearest even, infinities and NaN as NaN.  What the page
 * holds behind the sequence's end is unspecified afterwards.  Errors: E_ARG,
 * E_CUDA. */
int mlora_kv_append(const mlora_kv_cache* c, const mlora_kv_seqs* q, int32_t dtype, const void* k,
                    int64_t k_stride, const void* v, int64_t v_stride, void* stream);

/* Read the rows' positions back: k_out, v_out DEVICE [n_rows x n_kv_heads x
 * head_dim] of `dtype`, 16-byte aligned (either may be NULL).  Exact in both
 * types, but for magnitudes below the type's smallest.  Rows of skipped and
 * empty sequences are not written.  Errors: E_ARG, E_CUDA. */
int mlora_kv_read(const mlora_kv_cache* c, const mlora_kv_seqs* q, int32_t dtype, void* k_out, void* v_out,
                  void* stream);

/* Attention of the rows over their sequences' cached positions.  Query head j
 * of row r (position p) reads key/value head j / (n_heads / n_kv_heads):
 *     s_i = scale * q . k_i  for the positions i = 0 .. p;
 *     out = sum_i exp(s_i - lse) v_i,   lse = log sum_i exp(s_i).
 * A row without positions gets out = 0 and lse = -infinity.  q, out: rows of
 * n_heads * head_dim elements of `dtype`, q_stride / out_stride elements apart;
 * pointers and row distances are multiples of 16 bytes; out may be q (with its
 * stride), else no row of out overlaps one of q.  lse: DEVICE fp32
 * [n_rows x n_heads], or NULL.  max_len: upper bound of kv_len (a longer
 * sequence is a range error); it sets how far the work is split.
 * Sums and softmax statistics are fp32.  Scores are formed from the stored bytes
 * and q as fp16 values relative to the power of two above the row's largest
 * |q|: bf16 elements of at least 2^-17 of that are exact, smaller ones off by up
 * to 2^-25 of it; fp32 elements enter as two fp16 parts, to 2^-22 of themselves or
 * 2^-36 of it.  The probabilities enter the second product as fp16 (relative
 * rounding 2^-11, below bf16's own 2^-8), and on fp32 as two fp16 parts (2^-22);
 * a probability below 2^-22 of its row's largest has an absolute error of up to
 * 2^-33 (fp32: 2^-44) of that largest instead.  The dims of a result do not
 * touch one another, whatever the scales of the pages; a page whose value scale
 * is below 2^-64 of the largest in the sequence may count as zero in out (never in
 * lse).  A call repeats bit for bit.
 * workspace: DEVICE, 16-byte aligned, of any content (may be NULL); calls that
 * may overlap need one each.  With MLORA_KV_WORKSPACE_BYTES the work is shared
 * evenly whatever the lengths: long sequences are cut where a block's share
 * ends and their parts joined, so the order of a row's sums depends on the
 * lengths of the batch.  With less than the shape needs (0, say) no sequence is
 * cut, and a row's result is bit for bit the same whatever other sequences a call
 * with the same max_rows holds.
 * Errors: E_ARG, E_CUDA. */
typedef struct {
    const void* q;
    void* out;
    float* lse;
    void* workspace;
    int64_t q_stride, out_stride;
    int64_t workspace_bytes;
    int64_t max_len;
    int32_t dtype;
    int32_t n_heads;       /* a multiple of n_kv_heads                */
    float scale;           /* finite                                  */
} mlora_kv_attn;
int mlora_kv_attention(const mlora_kv_cache* c, const mlora_kv_seqs* q, const mlora_kv_attn* a, void* stream);

/* ------------------------------------------------------------------------
 * Page tables on the GPU.  A pool says which pages are free, so that sequences
 * grow and shrink by lengths that only the device knows (accepted drafted tokens,
 * finished sequences), with no table made on the host.  One pool serves the caches
 * of all layers, as they share their page ids.
 *
 * A row of the page table is a sequence's home: it owns the pages that it took.
 * A page in a row that another row owns (a shared prefix, put there by the caller)
 * is read as any other, never given back by this one, and never written: a sequence
 * does not grow inside a page that is not its own, so a shared prefix ends with a page
 * and its readers are cut back to whole pages of it.  When the owner gives a page
 * back, or is cut back inside it and grows again, entries of other rows stay and name
 * what others, or its new rows, are written to: cut those rows first.
 *
 * The free list is a stack, free_pages[0 .. *n_free).  A new pool of n pages has
 * their ids there in any order, *n_free = n and owner[i] = -1.  What the device
 * finds wrong never traps: it raises bits of *status, bit 0 for what is out of
 * range, bit 2 where pages were too few.  Calls on one pool are serialised by the
 * caller (one stream, or events).
 * ------------------------------------------------------------------------ */
typedef struct {
    int32_t* free_pages;   /* DEVICE [n_pages]                                             */
    int32_t* n_free;       /* DEVICE [1]                                                   */
    int32_t* owner;        /* DEVICE [n_pages]: the page table row that owns it, -1: none  */
    int32_t* status;       /* DEVICE int32 (may be NULL)                                   */
    int32_t n_pages;       /* >= 1                                                         */
} mlora_kv_pool;

/* Grow sequence s by n_new[s] >= 0 tokens: kv_len[s] += n_new[s], and the pages
 * that positions kv_len[s] .. kv_len[s] + n_new[s] - 1 need beyond the first
 * ceil(kv_len[s] / 64) come from the list's top, in the order of the sequences and
 * of their pages, into page_table and owner.  Then, as the calls above take them:
 *   row_off [n_seqs + 1]: the sequences' new rows, one sequence behind the other
 *   positions, seqs, slots [n_rows] (any may be NULL): each new row's position, its
 *     sequence, and its place page * 64 + position % 64 in a pool of pages; -1 for
 *     the rows behind the last.
 * A sequence is left as it is, with no rows, if its numbers are out of range
 * (negative, or together more than max_pages * 64 or 2^31 - 1), if the new rows of the
 * sequences up to it exceed n_rows, if its last page is part-filled and row s does not
 * own it (all bit 0), or if their pages exceed the free ones (bit 2).  Those sums
 * count every sequence in range, so one that is too large refuses those behind it that
 * need pages too.  Give row_off to the calls above even where every sequence was to get
 * one row: without it they take one row of each, the last old one of a sequence that was
 * left as it is.  Errors: E_ARG, E_CUDA. */
typedef struct {
    int32_t* page_table;       /* DEVICE [n_seqs x max_pages], updated       */
    int32_t* kv_len;           /* DEVICE [n_seqs], updated                   */
    const int32_t* n_new;      /* DEVICE [n_seqs]                            */
    int32_t* row_off;          /* DEVICE [n_seqs + 1], written               */
    int32_t* positions;        /* DEVICE, written                            */
    int32_t* seqs;             /* DEVICE, written                            */
    int64_t* slots;            /* DEVICE, written                            */
    int64_t n_rows;            /* 0 .. 2^31 - 1                              */
    int32_t n_seqs;            /* >= 0                                       */
    int32_t max_pages;         /* >= 1                                       */
} mlora_kv_growth;
int mlora_kv_reserve(const mlora_kv_pool* p, const mlora_kv_growth* q, void* stream);

/* Cut sequence s back to its first keep[s] tokens (keep NULL: to none): kv_len[s] =
 * min(kv_len[s], keep[s]), the page table entries behind ceil(keep[s] / 64) become
 * -1, and of those pages the ones that row s owns go back to the pool, last sequence
 * and last page first: the call undoes a mlora_kv_reserve exactly, and a growth by
 * as much takes the same pages again.  A sequence whose kv_len or keep is out of
 * range stays as it is, a page id out of range is dropped (bit 0).  Errors: E_ARG,
 * E_CUDA. */
int mlora_kv_release(const mlora_kv_pool* p, int32_t* page_table, int32_t* kv_len, const int32_t* keep,
                     int32_t n_seqs, int32_t max_pages, void* stream);

/* ------------------------------------------------------------------------
 * Rollouts of the transformer-block model (OpenTinker, "Multi-LoRA rollout":
 * rows of many adapters share the base projections).  The batch holds the new
 * rows of seqs' sequences, each with its own adapter: whole prompts, parts of
 * them, drafted tokens or one token a sequence.  Every layer rotates the rows'
 * keys by their positions, appends keys and values to its own cache and
 * attends over it; all else is mlora_tf_forward.  b->positions is not read
 * (may be NULL): seqs says where the rows stand.  seqs.n_rows = b->n_tokens.
 *
 * Ranges, besides those above: positions must be below the handle's
 * max_tokens (the bound of its rotary table).  A row outside them, with a bad
 * token, target or adapter id, or of a sequence that is out of range gets NaN
 * and raises MLORA_E_RANGE in mlora_tf_check_status; with a bad adapter id its
 * keys and values in the cache are unspecified.  The caches' own status reports
 * sequences out of range too, and alone a bad page id, whose sequence's rows get
 * NaN.  Rows of no sequence or of an empty slot get NaN and raise nothing, so a
 * batch can be padded to a fixed size.  Gradients, weights and step counts are not
 * changed.  No call allocates or synchronises, so a decode step can be captured
 * into a graph
 * (not while mlora_tf_profile_enable is on).
 * ------------------------------------------------------------------------ */
typedef struct {
    const mlora_kv_cache* caches;  /* HOST [n_layers]: the layers' page pools, which do not overlap, n_kv_heads of the model, head_dim 128 */
    mlora_kv_seqs seqs;            /* the same pages of every pool                 */
    void* workspace;               /* as in mlora_kv_attn                          */
    int64_t workspace_bytes;
    int64_t max_len;               /* upper bound of kv_len, 1 .. max_tokens       */
} mlora_tf_context;

/* Target-token logprobs of the rows; logprobs_out DEVICE fp32 [n_tokens], or
 * NULL (a prompt that is only to be cached).  Errors: E_ARG, E_CUDA. */
int mlora_tf_forward_cached(mlora_tf_t* h, const mlora_tf_batch* b, const mlora_tf_context* c, float* logprobs_out,
                            void* stream);

/* The same, and the next token of every sequence from its last row's
 * distribution: the smallest id v with CDF(v) > uniforms[s] (as
 * mlora_sampler_sample; the logits of the 256 ids around v are formed again
 * in fp32).  b->targets is not read (may be NULL).  uniforms: DEVICE fp32
 * [n_seqs] in [0, 1); next_out: DEVICE int32 [n_seqs], -1 for a sequence without
 * a good last row; logprob_out: DEVICE fp32 [n_seqs], NaN there.  n_seqs <=
 * max_tokens.  Errors: E_ARG, E_CUDA. */
int mlora_tf_sample_cached(mlora_tf_t* h, const mlora_tf_batch* b, const mlora_tf_context* c, const float* uniforms,
                           int32_t* next_out, float* logprob_out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MLORA_KV_H */
