/*
 * wc_attn.h — C ABI of libwc, attention of a serving step: a cache of keys and
 * values in the 4-bit form of wc_fp4.h, attention of a sequence's newest tokens
 * over it, and attention over whole prompts in BF16.
 *
 * A query at position p of its sequence attends to the positions
 *   max(0, p - window + 1) .. p        (window 0: 0 .. p)
 * of its own sequence, with the head of keys and values h / (heads / kv_heads):
 *   s[j] = scale sum_d q[d] K[j][d],   lse = log sum_j exp s[j]
 *   out  = sum_j exp(s[j] - lse) V[j]
 * A query with no position to attend to (p < 0) gets out = 0 and lse = -inf,
 * as does one whose scores are all -inf.  NaN and infinities count where they
 * are attended to and nowhere else.
 *
 * Scores, exponentials and sums are fp32; products of BF16 and 4-bit values are
 * exact.  out is rounded to BF16 once; over a prompt the weights exp(s - lse), not
 * their sum, are too.  The sums' order is fixed by the shape and the lengths: the same
 * call gives the same bits.  Values are summed with weights of up to 2^16 before they are
 * divided: values past 2^111 / tokens may overflow where the output itself would not.
 *
 * The cache is an array of pages, tiles of 32 tokens in each:
 *   uint8 [pages][kv_heads][page_size / 32][34 head_dim]
 * Slot s is token s % page_size of page s / page_size.  A tile holds for each of
 * its tokens a row of keys and one of values, in the form of a matrix row of
 * wc_fp4.h (two codes in a byte, one scale for 32 columns), in the order in which
 * a wave's lanes take them.  Of column c, with G = head_dim / 32, g = c / 32 and
 * token t of the tile:
 *   keys' codes     16 head_dim bytes.  Half t / 4 % 2 (64 G dwords each), quad g / 4
 *                   of groups (256 dwords), part c % 32 / 8, row 4 (t / 8) + t % 4,
 *                   group g % 4 of min(4, G - 4 (g / 4)): a dword of 8 codes
 *   values' codes   16 head_dim bytes.  Pair g / 2 of groups (1024 bytes), t / 8,
 *                   c % 32 / 2, group g % 2 of min(2, G - 2 (g / 2)), t % 8: a byte of 2
 *   keys' scales    32 G bytes, [row][half][g]
 *   values' scales  32 G bytes, [t / 8][g][t % 8]
 *
 * Conventions as in wc.h.  The cache, q, k, v and out are 16-byte aligned and
 * their strides multiples of 8 elements; d_lse, d_table, d_lengths and d_starts
 * 4-byte, d_slots 8-byte, d_work 16-byte.
 */
#ifndef WC_ATTN_H
#define WC_ATTN_H

#include "wc_fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WC_ATTN_MAX_DIM 256u  /* head_dim: a multiple of 32 up to this */
#define WC_ATTN_MAX_NEW 16u   /* new tokens per sequence of wc_fp4_attention */
#define WC_ATTN_MAX_HEADS 1024u

typedef struct wc_fp4_cache {
  uint8_t *d_data;
  uint64_t pages;     /* 1 .. 2^31 - 1; pages * page_size below 2^36 */
  uint32_t page_size; /* tokens, a multiple of 32 up to 2^20 */
  uint32_t kv_heads;  /* 1 .. WC_ATTN_MAX_HEADS */
  uint32_t head_dim;
} wc_fp4_cache;

#define WC_FP4_CACHE_BYTES(pages, page_size, kv_heads, head_dim) \
  ((uint64_t)(pages) * (kv_heads) * ((page_size) / 32u) * 34u * (head_dim))

/*
 * Keys and values of `tokens` tokens, BF16 [kv_heads][head_dim] each, k_stride and
 * v_stride elements from one token to the next, into the slots d_slots[tokens].
 * Rounded as by wc_fp4_encode.  A slot outside 0 .. pages * page_size - 1 leaves
 * its token out (-1 for a place that is not used).  Slots of one call must
 * differ: of a slot that is given twice the bytes may be either token's.  tokens and
 * the strides are below 2^31 (WC_E_SIZE).
 */
int wc_fp4_cache_append(const wc_fp4_cache *cache, const uint16_t *d_k, uint64_t k_stride,
                        const uint16_t *d_v, uint64_t v_stride, const int64_t *d_slots,
                        uint64_t tokens, void *stream);

/* The BF16 values that the cache holds for the slots, into d_k and d_v
 * [tokens][kv_heads][head_dim]; NaN for a slot outside the cache. */
int wc_fp4_cache_read(const wc_fp4_cache *cache, const int64_t *d_slots, uint64_t tokens,
                      uint16_t *d_k, uint16_t *d_v, void *stream);

typedef struct wc_fp4_attention_shape {
  uint64_t q_stride;    /* elements from one token's queries to the next one's */
  uint32_t seqs;        /* sequences */
  uint32_t new_tokens;  /* queries per sequence, 1 .. WC_ATTN_MAX_NEW */
  uint32_t heads;       /* a multiple of kv_heads, up to WC_ATTN_MAX_HEADS */
  uint32_t table_width; /* pages per sequence */
  uint32_t window;      /* 0: none */
  float scale;
} wc_fp4_attention_shape;

/* Device scratch of a call of that shape (0: none is needed, or the call refuses the
 * shape).  Host only; asks the current device for its size. */
size_t wc_fp4_attention_workspace_bytes(const wc_fp4_cache *cache, const wc_fp4_attention_shape *shape);

/*
 * d_q BF16 [seqs * new_tokens][heads][head_dim]; d_table int32 [seqs][table_width],
 * the pages of each sequence in order; d_lengths int32 [seqs], tokens of each
 * sequence in the cache, its new ones included: query i of a sequence of length n is
 * at position n - new_tokens + i.  d_out BF16 [seqs * new_tokens][heads][head_dim],
 * d_lse fp32 [seqs * new_tokens][heads] or NULL.  Entries of the table past a
 * sequence's length, or before its window, are not used.  A query that attends to a
 * token whose page is outside the cache, or past the table, gets NaN.
 *
 * The sizes are those of the table, whatever the lengths.  WC_E_SIZE where
 *   table_width * page_size is past 2^30,
 *   seqs times the tiles of 32 tokens that a sequence may have (of the table, or that
 *   a window may touch) is 2^30 or more,
 *   seqs * new_tokens * heads is 2^24 or more,
 *   kv_heads * ceil(new_tokens * heads / kv_heads / 16) * seqs is near 2^22 or more, or
 *   q_stride is 2^31 or more.
 */
int wc_fp4_attention(const wc_fp4_cache *cache, const wc_fp4_attention_shape *shape,
                     const uint16_t *d_q, const int32_t *d_table, const int32_t *d_lengths,
                     uint16_t *d_out, float *d_lse, void *d_work, size_t work_bytes, void *stream);

typedef struct wc_prompt_shape {
  uint64_t tokens;                       /* of all prompts */
  uint64_t q_stride, k_stride, v_stride; /* elements from one token to the next, below 2^24 (of one
                                            token alone: any multiple of 8) */
  uint32_t seqs;
  uint32_t heads, kv_heads, head_dim;
  uint32_t window; /* 0: none */
  float scale;
} wc_prompt_shape;

/*
 * Prompts one after the other: d_q BF16 [tokens][heads][head_dim], d_k and d_v
 * [tokens][kv_heads][head_dim]; d_starts int32 [seqs + 1], not falling: sequence i
 * is the tokens d_starts[i] .. d_starts[i + 1] - 1, the first of them at position 0.
 * (Entries outside 0 .. tokens count as the nearer end.)  d_out BF16
 * [tokens][heads][head_dim], d_lse fp32 [tokens][heads] or NULL; tokens of no
 * sequence are left as they were.  WC_E_SIZE where tokens or seqs is 2^31 or more, and
 * possibly from (tokens / 128 + seqs) * heads = 2^23 on.
 */
int wc_prompt_attention(const wc_prompt_shape *shape, const uint16_t *d_q, const uint16_t *d_k,
                        const uint16_t *d_v, const int32_t *d_starts, uint16_t *d_out, float *d_lse,
                        void *stream);

#ifdef __cplusplus
}
#endif
#endif /* WC_ATTN_H */
