/*
 * q8_attention.h -- C ABI of the attention half of the quantised transformer path for one NVIDIA GB300
 * (sm_103a): norms and rotation of query and key heads, a paged cache of codes, attention of the newest
 * tokens over that cache and attention over whole prompts. Exported by the same library as q8.h and
 * with the same conventions (statuses, the current device, streams, what a run may do).
 *
 * Heads. A matrix of heads holds, for each token, `heads` rows of head_dim elements; element
 * (token, head, i) lies at token * pitch + head * head_pitch + i, both pitches in elements. Elements
 * between those are neither written nor used.
 *
 * Codes of a row (one token's head): int8 and e4m3 as in q8.h, scale = amax / 127 or 448 (1 if amax
 * is 0), q = 127 or 448 * v / amax rounded to the nearest code, ties to even. 4-bit codes have a scale
 * and a lowest value: v ~ q * scale + lowest with lowest = min v, scale = (max v - min v) / 15 (1 if that
 * is 0), q = 15 * (v - lowest) / (max v - min v) rounded to the nearest of 0 .. 15, ties to even; byte i of
 * a row holds the codes of 2i (low bits) and 2i + 1. The quotients are those of the unrounded scale: rows
 * of 16-bit values lie on ties often. A row that holds a NaN or an infinity, or whose max - min overflows
 * fp32, has the scale NaN (and the lowest value 0) and codes 0.
 *
 * Cache. Pages of page_size tokens (a multiple of 16):
 *   codes [pages][kv_heads][page_size][head_dim or head_dim / 2 bytes], on 16 bytes
 *   scale [pages][kv_heads][page_size] fp32, of 4-bit codes [..][2]: scale, lowest; on 16 bytes
 * without gaps; head_dim 64, 128 or 256. A slot is page * page_size + place in the page.
 */
#ifndef Q8_ATTENTION_H
#define Q8_ATTENTION_H

#include "q8.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { Q8_INT4 = 3 }; /* beside q8_code_type's, in caches only */

typedef struct {
    void *k_codes, *v_codes;
    float *k_scale, *v_scale;
    long long pages;
    int page_size, kv_heads, head_dim, code_type;
} q8_cache;

/* The widest head of heads_q8_run. */
#define Q8_MAX_HEAD_DIM 256
/* The most axes of positions. */
#define Q8_MAX_AXES 4

/*
 * Heads of queries and keys, from a product's output to what attention takes, in one pass:
 *   y = x / sqrt(mean over the head of x^2 + eps) * weight       (where the weight is not NULL)
 *   pairs of y turned by their angles                           (where turns is not NULL)
 * Pair j (j < rot_dim / 2) is (y[2j], y[2j+1]) if `adjacent`, else (y[j], y[j + rot_dim / 2]); elements
 * from rot_dim on stay. (a, b) becomes (a cos - b sin, b cos + a sin) with the angle, in turns,
 *   turns[j] * positions[axis[j]][token] / 2^64, of which the whole turns are dropped exactly
 * (products of 64 bits modulo 2^64): an angle is as exact at position 10^6, or 10^12, as at 1.
 * Everything is in fp32 and rounded once. A sum of squares above 2^100, or below 2^-80 beside an eps below
 * 2^-100, is taken of values scaled by a power of two, so that huge and tiny rows are normed too; a row of
 * zeros stays 0 with an eps of 0.
 *
 * q -> q_out; k -> k_out and, with a cache, the codes of k (of the unrounded values) and of v (which is
 * neither normed nor rotated) at the slot of each token. q, k and v may be NULL, k_out too with a cache;
 * v is there exactly when the cache is, and k then too. A negative slot, or one past the cache, is that of a padding
 * token: nothing is written for it there. No two tokens may have one slot. q_out may be q and k_out k (with the same
 * pitches); apart from that no output may overlap an input or another output.
 *
 * Errors: EINVAL (nothing to do: neither q nor k; an input without its output or the reverse; v or slots without a
 * cache, or a cache without k, v and slots; sizes below 1, tokens < 0, rot_dim above head_dim or odd, axes outside
 * 1 .. Q8_MAX_AXES, positions missing where turns are there or with rows that overlap (but for a pitch of 0), an axis
 * list missing with more than one axis, a pitch or head pitch that makes rows overlap or is not a multiple of 16 bytes,
 * matrices that are not on 16 bytes, vectors that are not aligned to their element, eps negative or not finite, an
 * unknown type, a cache whose kv_heads or head_dim differ, page_size not a multiple of 16; `device` not the current one),
 * EUNSUPPORTED (head_dim not a multiple of 8 or above Q8_MAX_HEAD_DIM; with a cache other than 64, 128 and 256;
 * tokens of 2^31 or more, heads of 2^16 or more, a cache of 2^31 slots or more, a device that is not sm_103), ECUDA.
 * tokens == 0 does nothing. axis[j] >= axes is taken as axis 0.
 */
typedef struct {
    const void *q;              /* [tokens][q_heads][head_dim] value_type, or NULL */
    void *q_out;                /* the same */
    const void *k;              /* [tokens][kv_heads][head_dim] value_type, or NULL */
    void *k_out;                /* the same, or NULL with a cache */
    const void *v;              /* [tokens][kv_heads][head_dim] value_type, with a cache */
    const void *q_weight, *k_weight; /* [head_dim] weight_type, or NULL: no norm */
    const unsigned long long *turns; /* [rot_dim / 2], turns a position times 2^64; NULL: no rotation */
    const unsigned char *axis;  /* [rot_dim / 2], or NULL with one axis */
    const long long *positions; /* [axes][tokens] */
    const long long *slots;     /* [tokens], with a cache */
    const q8_cache *cache;      /* NULL: none. Read by the call, not kept */
    long long q_pitch, q_head_pitch, q_out_pitch, q_out_head_pitch;
    long long k_pitch, k_head_pitch, k_out_pitch, k_out_head_pitch, v_pitch, v_head_pitch;
    long long positions_pitch;  /* between axes; 0: all axes have one row of positions */
    long long tokens;
    void *stream;
    int q_heads, kv_heads, head_dim, rot_dim, axes, adjacent;
    int value_type, weight_type, device;
    float eps;
} heads_q8_args;

conv3d_status heads_q8_run(const heads_q8_args *args);

/*
 * Rows of a cache as values: k[t] and v[t] = the values of slot slots[t], q * scale (+ lowest) in fp32,
 * rounded once. A slot may come several times; the rows of one that is negative or past the cache are
 * left as they were. Errors: as heads_q8_run's, of what is here.
 */
typedef struct {
    const q8_cache *cache;
    const long long *slots;     /* [tokens] */
    void *k, *v;                /* [tokens][kv_heads][head_dim] value_type */
    long long k_pitch, k_head_pitch, v_pitch, v_head_pitch;
    long long tokens;
    void *stream;
    int value_type, device;
} cache_q8_read_args;

conv3d_status cache_q8_read_run(const cache_q8_read_args *args);

/*
 * Attention of each sequence's newest tokens over its part of a cache, in which they are already:
 *   o = sum_s p_s v_s / sum_s p_s,   p_s = exp(scale * q . k_s)
 * over s < lengths[b] - tokens + 1 + t for token t (0 <= t < tokens) of sequence b, whose row is b *
 * tokens + t of q and o; head h of q reads head h / (q_heads / kv_heads) of the cache. A token that
 * sees nothing (a length below tokens - t, scores of -inf) gets 0. The place s of sequence b is page table[b][s /
 * page_size]. A cached row whose scale is NaN makes every output that sees it NaN, and no other; e4m3
 * codes that are NaN, which heads_q8_run does not write, may be in no row below lengths[b].
 *
 * Codes and q are multiplied in f16, where codes are exact and a row of q, scaled by a power of two, is too
 * but for elements below 2^-22 of the row's largest, which err by 2^-33 of that. A weight times v's scale has two parts
 * of f16's 11 bits for f16 outputs; for bf16 outputs it is cut to one, the same for all that is made of it (an output errs by at
 * most 2^-11 of sum p |v - o|). Either way codes of such products below 2^-21 of the largest err by 2^-31 of it, and a
 * key whose product is below 2^-133 of it counts as not seen. Sums, maxima and scales are fp32. Scales of v below 2^-80
 * count as 2^-80, and the scale 1 of a row of v whose codes are all 0 (zeros, or equal values in 4 bits) as 2^-64, or as an
 * eighth of its lowest value's magnitude if that is more: such a row takes no bits from the others, and keeps its own down to
 * 2^-85. Results are the same from run to run.
 *
 * A plan holds the device's workspace: a status word and the partial results of sequences that several blocks share,
 * fixed by q_heads, kv_heads, max_tokens and head_dim, whatever the lengths. All that a run is given lies on its plan's
 * device. At most one run of a plan may be in flight at a time (one plan for each concurrent stream; graphs that were captured
 * with one plan are replayed one after another).
 */
typedef struct attn_q8_plan_s *attn_q8_plan_t; /* opaque, owned by the library */

/* Optional planning knobs of both attentions; none changes what is computed. Zero-initialise. */
typedef struct {
    int wait_timeout_ms; /* 0: 2000 ms; a bounded wait inside a kernel gives up after this long */
    int debug_flags;     /* test-only: bit 0 leaves out the copy of the first sequence's first keys (for prompts: the
                            first block's first copy), so that the waits on it must run out (exercises the error path
                            without faulting anything) */
} attn_options;

/* Errors: EINVAL (a size below 1, q_heads no multiple of kv_heads, an unknown code type), EUNSUPPORTED (a head_dim
 * other than 64, 128 and 256, max_seqs above 65536, max_tokens above 64, q_heads of 4096 or more, a device that is
 * not sm_103), ENOMEM, ECUDA. On error *plan is set to NULL. */
conv3d_status attn_q8_plan(attn_q8_plan_t *plan, long long max_seqs, int max_tokens, int q_heads,
                           int kv_heads, int head_dim, int code_type, int device);
/* With planning knobs (opts may be NULL; EINVAL for a negative timeout). */
conv3d_status attn_q8_plan_ex(attn_q8_plan_t *plan, long long max_seqs, int max_tokens, int q_heads,
                              int kv_heads, int head_dim, int code_type, int device,
                              const attn_options *opts);

/* Errors: EINVAL (a NULL pointer with seqs > 0, seqs < 0 or above max_seqs, tokens outside 1 .. max_tokens, a cache
 * that does not fit the plan, q and o not bf16 or f16 on 16 bytes with pitches of whole 16 bytes, table_pitch below
 * table_width, scale not finite, the wrong current device), ECUDA. A length below 0, or above table_width * page_size,
 * and a page outside the cache are met on the device: that sequence's output is then NaN and attn_q8_check reports
 * EDEVICE. seqs == 0 does nothing. */
typedef struct {
    const q8_cache *cache;
    const void *q;              /* [seqs * tokens][q_heads][head_dim] value_type: bf16 or f16 */
    void *o;                    /* the same; may be q with the same pitches */
    const int *table;           /* [seqs][table_width] */
    const int *lengths;         /* [seqs], the newest tokens included */
    long long q_pitch, q_head_pitch, o_pitch, o_head_pitch;
    long long seqs, table_width, table_pitch;
    void *stream;
    int tokens, q_heads, value_type;
    float scale;
} attn_q8_args;

conv3d_status attn_q8_run(attn_q8_plan_t plan, const attn_q8_args *args);

/* Synchronise the device, then report and clear the plan's device status: OK, or EDEVICE (a bad length or page, or one
 * of a kernel's bounded waits ran out). */
conv3d_status attn_q8_check(attn_q8_plan_t plan);
size_t attn_q8_workspace_size(attn_q8_plan_t plan); /* 0 for NULL */
void attn_q8_destroy(attn_q8_plan_t plan);          /* waits for the device; NULL is allowed */

/*
 * Attention over whole prompts, packed one behind the other: for sequence b, its rows starts[b] ..
 * starts[b+1] - 1 of q and o and key_starts[b] .. key_starts[b+1] - 1 of k and v,
 *   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale * q_i . k_j)
 * over all keys of the sequence, if `causal` over j <= i + (keys - queries) (the last query sees all keys).
 * key_starts may be starts, or others: a chunk of queries whose keys begin earlier. A query that sees no key
 * gets 0 (a score of -inf is that of a key it does not see); rows of o outside all sequences are left as they were. Head
 * h of q reads head h / (q_heads / kv_heads) of k and v. Scores and sums are fp32, p is rounded to the value type before it
 * meets v. What a query does not see does not reach it, infinities and NaN included. All that a run is given lies on its plan's
 * device.
 *
 * Starts are device memory; those that decrease or leave 0 .. rows (q_rows, k_rows) are cut to it; rows of q that
 * several sequences then have are left with any one's output or as they were. A plan holds a status word; its runs may be
 * in flight at once.
 */
typedef struct attn_prompt_plan_s *attn_prompt_plan_t; /* opaque, owned by the library */

/* Errors: EINVAL (`device` not the current one), EUNSUPPORTED (not an sm_103), ENOMEM, ECUDA. */
conv3d_status attn_prompt_plan(attn_prompt_plan_t *plan, int device);
conv3d_status attn_prompt_plan_ex(attn_prompt_plan_t *plan, int device, const attn_options *opts);

/* Errors: EINVAL (a NULL pointer with seqs, q_rows > 0, sizes below 1 or negative, q_heads no multiple of kv_heads,
 * value_type not bf16 or f16, matrices that are not on 16 bytes, pitches that are no whole 16 bytes or make rows
 * overlap, scale not finite, the wrong current device), EUNSUPPORTED (head_dim not a multiple of 8 or above 128, rows of 2^31 or more, seqs above 65536,
 * q_heads of 65536 or more), ECUDA. Nothing is done where seqs or q_rows is 0. o may not overlap an input. */
typedef struct {
    const void *q;              /* [q_rows][q_heads][head_dim] value_type */
    const void *k, *v;          /* [k_rows][kv_heads][head_dim] value_type */
    void *o;                    /* [q_rows][q_heads][head_dim] value_type */
    const int *starts;          /* [seqs + 1] */
    const int *key_starts;      /* [seqs + 1], or NULL: starts */
    long long q_pitch, q_head_pitch, k_pitch, k_head_pitch, v_pitch, v_head_pitch;
    long long o_pitch, o_head_pitch;
    long long q_rows, k_rows, seqs;
    void *stream;
    int q_heads, kv_heads, head_dim, value_type, causal;
    float scale;
} attn_prompt_args;

conv3d_status attn_prompt_run(attn_prompt_plan_t plan, const attn_prompt_args *args);
conv3d_status attn_prompt_check(attn_prompt_plan_t plan); /* as attn_q8_check: OK or EDEVICE */
void attn_prompt_destroy(attn_prompt_plan_t plan);

#ifdef __cplusplus
}
#endif
#endif /* Q8_ATTENTION_H */
