/*
 * m3_attn.h -- C ABI of libm3.so, second part: the attention layer of a hybrid
 * stack on AMD MI355X (gfx950). Rotary positions, a paged cache of keys and
 * values held in 8 bits, and attention over it.
 *
 * The pages put one attention layer beside every five recurrent mixers
 * ("Mamba-3架构技术解析：新一代语言建模的范式转移", §4.2: the 5:1 hybrid). These are
 * that layer's operators; its projections are plain matrix products.
 *
 * Conventions, ownership, streams and errors are those of m3.h: caller-owned
 * device buffers, no allocation, every argument checked before any HIP call,
 * asynchronous on `stream`, nothing throws. What lives in device memory (lengths,
 * page numbers) cannot be checked on the host: the kernels hold every access
 * inside the buffers whatever those values are, and treat a position whose page
 * number is outside [0, num_pages) or [0, max_pages) as absent.
 *
 * Rows. Queries, keys and values of a batch are rows of tokens: row t, head h at
 * p + t * token_stride + h * head_stride (elements; the D entries of a head are
 * contiguous), so the parts of one fused projection are used where they lie.
 * Pointers and strides that are multiples of 16 bytes take the wide loads; others
 * work too. Sequences follow one another: sequence i owns rows cu_q[i] ..
 * cu_q[i + 1] - 1, and its last row is the token at position kv_len[i] - 1.
 */
#ifndef M3_ATTN_H
#define M3_ATTN_H

#include "m3.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens that share one scale, per head. */
#define M3_KV_BLOCK 16

/* How a cached value is held: value = code * scale of its block.
 * INT8: whole numbers -127 .. 127. FP8: e4m3 (OCP, finite up to 448). */
typedef enum m3_kv_format { M3_KV_INT8 = 0, M3_KV_FP8 = 1 } m3_kv_format;

/*
 * The cache, num_pages pages of page_size tokens (a power of two, >= 16):
 *   k        [num_pages][heads][page_size / 16][16][headdim]   codes, 8 bits
 *   v        [num_pages][heads][page_size / 16][headdim][16]   codes, 8 bits
 *   k_scale, v_scale [num_pages][heads][page_size / 16]        fp32
 * headdim: a multiple of 16 up to 256. All four are 16-byte aligned; scales are
 * not negative. A sequence
 * holds position j in page pages[i][j / page_size]. The 16 slots of a block are
 * written together when its first token comes, so no slot of a block in use is
 * left undefined.
 */
typedef struct m3_kv_cache {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int64_t num_pages;
    int32_t page_size;
    int32_t heads;
    int32_t headdim;
    int32_t format;       /* m3_kv_format */
} m3_kv_cache;

/*
 * A ragged batch. Device arrays are int32.
 *   cu_q   [batch + 1], cu_q[0] = 0, not decreasing, cu_q[batch] = tokens; or NULL:
 *          one row per sequence (tokens = batch)
 *   kv_len [batch]  tokens held once the batch's new ones are in; 0 marks an idle
 *          slot, whose rows are not stored and attend to nothing
 *   pages  [batch][max_pages]
 * max_q: at least the longest sequence's rows. max_kv: at least the largest
 * kv_len. A sequence's rows beyond the first max_q are left out (not stored, their
 * outputs not written) and keys beyond max_kv not seen; the other rows keep their
 * positions. Both only size the launch. A max_kv that is too large costs a step or a
 * piece of a prompt next to nothing; a prompt that starts a sequence may take a fifth
 * longer (its row tiles are then as large as a piece's). A max_q of all rows costs up to a
 * fifth. One kernel serves a batch, chosen by its rows: single tokens beside a long prompt
 * may be better off in a call of their own.
 */
typedef struct m3_kv_batch {
    int64_t batch;
    int64_t tokens;
    int64_t max_pages;
    int64_t max_q;
    int64_t max_kv;
    const int32_t* cu_q;
    const int32_t* kv_len;
    const int32_t* pages;
} m3_kv_batch;

/* Rows of an input or output (see above). A const buffer is never written. */
typedef struct m3_rows {
    void* p;
    int64_t token_stride;
    int64_t head_stride;
} m3_rows;

/*
 * Rotary positions: pair i < rot / 2 of a head turns by theta = position *
 * inv_freq[i] (formed in 64 bits, so late positions lose nothing),
 *   (a, b) -> (a c - b s, a s + b c),  c = mscale cos theta, s = mscale sin theta,
 * with pairs (2i, 2i + 1) (interleaved) or (i, i + rot / 2); entries rot .. D - 1
 * pass unchanged. inv_freq [rot / 2] fp32 (scaled frequencies and mscale carry the
 * long-context variants).
 */
typedef struct m3_rotary {
    const float* inv_freq;
    int32_t rot;          /* even, 0 < rot <= headdim */
    int32_t interleaved;  /* 0: pairs (i, i + rot / 2) */
    float mscale;         /* finite; 1 without attention scaling */
} m3_rotary;

/*
 * m3_rope -- turn x [tokens][heads] rows of headdim entries into y.
 * positions [tokens] int32. backward != 0: the transposed map, (a, b) ->
 * (a c + b s, b c - a s) and unchanged tails: dL/dx from dL/dy. fp32 arithmetic,
 * one rounding to the io dtype. y may be x itself (same strides); any other
 * overlap is refused. headdim 2 .. 65536, any alignment.
 */
m3_status m3_rope(const m3_rows* x, const m3_rows* y, int64_t tokens, int32_t heads, int32_t headdim,
                  m3_dtype io_dtype, const int32_t* positions, const m3_rotary* rotary, int32_t backward,
                  void* stream);

/*
 * m3_kv_append -- put the batch's new keys and values into the cache, the keys
 * turned on the way; optionally turn the queries in the same launch.
 * k, v: rows of cache->heads heads, io dtype. rotary: NULL leaves keys and queries
 * unturned. q, q_out, q_heads: both rows or both NULL; a query turns by its
 * token's position (q_out may be q itself).
 *
 * Per touched block and head, with "old" its tokens from before the call:
 *   scale' = max(old ? scale : 0, max |new| * (1 / Q))      Q = 127 (INT8), 448 (FP8)
 *   code   = nearest(new * (1 / scale')), nearest(code * (scale * (1 / scale'))) for
 *            the old, ties to even, held to +-Q; 0 in slots after the last token of a
 *            block that begins here; all in fp32, every operation rounded. A scale
 *            below 2^-126 counts as 0 (so do the block's values then)
 * so old codes change only when the scale grows. Positions start at
 * kv_len[i] - (rows of i); a sequence may be cut back by a smaller kv_len and
 * continued. A value that is not finite makes its block's scale NaN: attention
 * over that block then gives NaN, as it would over the value. Sequences of one
 * call must not write into a shared block.
 */
m3_status m3_kv_append(const m3_kv_cache* cache, const m3_kv_batch* batch, const m3_rows* k, const m3_rows* v,
                       const m3_rows* q, const m3_rows* q_out, int32_t q_heads, m3_dtype io_dtype,
                       const m3_rotary* rotary, void* stream);

/*
 * m3_kv_read -- the values that the cache stands for, as dense rows:
 * k_out, v_out [batch][max_count][heads][headdim] io dtype; row j of sequence i is
 * position first[i] + j, zero for j >= count[i] and for absent positions.
 */
m3_status m3_kv_read(const m3_kv_cache* cache, int64_t batch, const int32_t* first, const int32_t* count,
                     const int32_t* pages, int64_t max_pages, int64_t max_count, void* k_out, void* v_out,
                     m3_dtype io_dtype, void* stream);

/*
 * m3_kv_attend -- softmax attention of the batch's queries over the cache.
 *   out[t][h] = sum_j p_j v_j,  p = softmax over the keys that row t sees of
 *   scale * q . k_j; key / value head h / (q_heads / cache->heads)
 * A row at position p sees keys j < kv_len, with causal != 0 only j <= p, and with
 * window > 0 (causal only) only j > p - window. A row that sees none gives 0, and
 * lse = -inf.
 * q: rows of q_heads heads (a multiple of cache->heads). out [tokens][q_heads][headdim]
 * io dtype, dense, not overlapping an input; lse [tokens][q_heads] fp32 (natural
 * logarithm of the softmax's denominator), or NULL. Scores, the softmax and its
 * sums are fp32. With fp32 rows nothing is rounded to fewer bits; with bf16 rows each
 * probability is rounded to fp16 for the product with V: to 2^-11 of itself, or to 2^-32
 * of the largest probability times V scale that the row sees, where that is more (keys
 * more than about 14 nats below a key that takes all keep fewer bits).
 * workspace: at least m3_kv_attend_workspace_size() bytes, 16-byte aligned (NULL
 * when that is 0); holds the parts of rows whose keys are split over workgroups.
 */
m3_status m3_kv_attend(const m3_kv_cache* cache, const m3_kv_batch* batch, const m3_rows* q, void* out, float* lse,
                       int32_t q_heads, m3_dtype io_dtype, float scale, int32_t causal, int64_t window,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes m3_kv_attend needs (0 on invalid sizes). Host only; device arrays are not read. */
size_t m3_kv_attend_workspace_size(const m3_kv_cache* cache, const m3_kv_batch* batch, int32_t q_heads,
                                   m3_dtype io_dtype, int32_t causal, int64_t window);

/*
 * What rows see, beyond causal and window of m3_kv_attend: first tokens that stay visible
 * under a window, and first pages that sequences hold together.
 * sinks: with a window, a row at position p sees the keys j <= p with j > p - window or j <
 * sinks (without one it sees them all the same). Pages that hold none of either are not read: their
 * entries may name anything.
 * groups > 0: sequences group_start[g] .. group_start[g + 1] - 1 hold their first prefix_count[g] pages (whole
 * pages, all full) together; prefix_pages[g] names them, and the sequences' own entries for them
 * are not read. Positions and lengths count the prefix, and batch->max_pages covers it. A
 * sequence of no group shares nothing. group_start NULL: one group (groups 1) of all sequences.
 * Device arrays are int32; group_start does not decrease. A count outside 0 .. max_prefix is
 * taken to the nearer end.
 */
typedef struct m3_kv_view {
    int32_t causal;
    int64_t window;              /* 0: none */
    int64_t sinks;               /* >= 0 */
    int64_t groups;              /* 0: no prefixes */
    int64_t max_prefix;          /* pages of a row of prefix_pages; sizes the launch, as max_kv does */
    const int32_t* group_start;  /* [groups + 1] or NULL */
    const int32_t* prefix_count; /* [groups] */
    const int32_t* prefix_pages; /* [groups][max_prefix] */
} m3_kv_view;

/*
 * m3_kv_attend_view -- m3_kv_attend over such a view. The outputs are those of m3_kv_attend over tables that name
 * the shared pages themselves (up to the order of fp32 sums); the prefix of a group is read once
 * for many of its rows where that pays, without a window and up to 64 (row, head of a group)
 * pairs a sequence (32 for fp32 rows and above headdim 128). Sequences with more rows each read it for their own.
 */
m3_status m3_kv_attend_view(const m3_kv_cache* cache, const m3_kv_batch* batch, const m3_kv_view* view,
                            const m3_rows* q, void* out, float* lse, int32_t q_heads, m3_dtype io_dtype, float scale,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes m3_kv_attend_view needs (0 on invalid sizes). Host only; device arrays are not read. */
size_t m3_kv_attend_view_workspace_size(const m3_kv_cache* cache, const m3_kv_batch* batch, const m3_kv_view* view,
                                        int32_t q_heads, m3_dtype io_dtype);

#ifdef __cplusplus
}
#endif
#endif /* M3_ATTN_H */
