/*
 * dspark_tree.h -- C ABI of the GB300 (sm_103a) operators that follow a draft:
 * the target model's check of drafted tokens over a paged key/value cache.
 *
 * The walk (dspark_walk.h) proposes tokens; a round of the target model then
 *  1. writes the drafted tokens' keys and values into the cache
 *     (dspark_tree_write, 16-bit or quantised to e4m3),
 *  2. lets every drafted token attend to the cached context and to its own
 *     ancestors in the draft (dspark_tree_attend),
 *  3. keeps the accepted path's rows of the cache (dspark_tree_keep).
 * dspark_tree_read gives cached rows back in the model's type.  dspark_tree_place is
 * the first step for a model that norms and rotates its query and key heads: it does that
 * on the way into the cache.  dspark_pages.h has the page tables and slots.
 *
 * The cache is paged: position p of request b is slot p % page_size of page
 * pages[b][p / page_size].  A quantised row (one token, one head) is held as
 * e4m3 codes and one power-of-two scale, stored as its biased exponent byte:
 *
 *     a    = max |x|
 *     e    = the smallest integer with a <= 448 * 2^e, within [-127, 127]
 *     code = e4m3_rne(x * 2^-e),   byte = e + 127,   value = code * 2^e
 *
 * (a = 0: byte 0.  A row that holds a NaN or an infinity: byte 255, codes NaN,
 * and it reads back as NaN.)  A power of two makes x * 2^-e exact, so a code
 * is one rounding of x, and makes every value exact in bf16 (but those past
 * its range).
 *
 * A row in 4 bits is held as e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6, and a sign in
 * the top bit; two a byte, the even element in the low half) and a byte for each
 * 16 elements, bits 14 .. 7 of the block's scale as an f16:
 *
 *     a    = max |x| of the block
 *     s    = the smallest f16 with three mantissa bits with a <= 6 s, at most 10240
 *     code = e2m1_rne(x / s), at most 6 in size,   byte = f16 bits of s >> 7,
 *     value = code * s
 *
 * (a = 0: byte 0.  A block that holds a NaN or an infinity: byte 255, codes 0, and
 * it reads back as NaN.  Bytes 227 to 254 are not written; what a block under one
 * reads as is not specified.)  A value has six significant bits and is exact in f16
 * and in bf16.
 *
 * Attention: node i of request b (row first[b] + i of q) with query head h
 * reads cached head h / (q_heads / kv_heads) at positions 0 .. start[b]-1 (the
 * context: all visible) and start[b] + j, j < T_b (the draft: visible if bit
 * j % 32 of mask word [first[b] + i][j / 32] is set, or, without a mask, if
 * j <= i: a chain):
 *
 *     s   = scale * q.k                        (fp32)
 *     s   = softcap * tanh(s / softcap)        (softcap > 0)
 *     out = sum_j softmax(s)_j v_j,  lse = ln sum_j e^(s_j)
 *
 * A row that sees nothing gets out = 0 and lse = -infinity.  Keys and values
 * at invisible positions do not affect a row, whatever they hold.  Sums, maxima
 * and out are fp32 until out is rounded; the weights e^(s - m) are rounded once to
 * a 16-bit type for their product with v: the handle's, or f16 where the cache is
 * e4m3 or e2m1 and the rows are few (rows of q in bf16 are then brought to f16 by a
 * power of two each, exact for elements down to 2^-32 of the row's largest and to 2^-40
 * of that below).  Any finite scale, and any cap from 0 on.
 *
 * Conventions as in dspark_walk.h: 0 or a negative DSPARK_E* code, nothing
 * traps, calls on one handle are ordered by the caller, `stream` is a
 * cudaStream_t of the handle's device (which need not be the current one),
 * launches are graph-capturable.  Sizes
 * that only the device knows (start, first, pages, path, count) are checked
 * there: a request that fails is left out (its rows and cache stay as they
 * were) and dspark_tree_status then returns DSPARK_EPAGES.  Where only an entry
 * of the page table is no page of the cache, write and read leave out the rows
 * on it, and attend's rows of that request are unspecified; nothing outside
 * the cache is touched.
 */
#ifndef DSPARK_TREE_H
#define DSPARK_TREE_H

#include "dspark_walk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define DSPARK_TYPE_BF16 0
#define DSPARK_TYPE_F16 1
#define DSPARK_TYPE_E4M3 2 /* cache only */
#define DSPARK_TYPE_E2M1 3 /* cache only */

/* Largest sizes of a handle. */
#define DSPARK_TREE_MAX_HEAD_DIM 128
#define DSPARK_TREE_MAX_REQUESTS 1024
#define DSPARK_TREE_MAX_NODES 256
#define DSPARK_TREE_MAX_LENGTH 2147483392 /* cached rows of a request, 2^31 - 256 */

typedef struct dspark_tree dspark_tree;
typedef dspark_tree *dspark_tree_t;

/* The model's side of every call of one handle. */
struct dspark_tree_config {
    int q_heads;      /* query heads, a multiple of kv_heads */
    int kv_heads;     /* cached heads */
    int head_dim;     /* a multiple of 8 (e4m3 cache: 16, e2m1: 32), at most 128 */
    int type;         /* DSPARK_TYPE_BF16 or DSPARK_TYPE_F16: q, k, v, out */
    int max_requests; /* largest B of an attend call, at most 1024 */
    int max_nodes;    /* most nodes of one request in an attend call, at most 256 */
};

/*
 * A paged cache: k and v are [n_pages, page_size, kv_heads, head_dim] of
 * `type` (the handle's type, DSPARK_TYPE_E4M3 or DSPARK_TYPE_E2M1), head_dim
 * contiguous, the other strides free: {page, slot, head} in elements (e2m1: in
 * bytes).  Base addresses and strides are multiples of 16 bytes, those of pages and
 * slots below 2^31 bytes.  k_scale and v_scale: e4m3, bytes [n_pages, page_size,
 * kv_heads] with strides of their own; e2m1, bytes [n_pages, page_size, kv_heads,
 * head_dim / 16], the last contiguous, addresses and the other strides multiples of
 * the largest power of two in head_dim / 16.  NaN codes stand under byte 255 only, as
 * dspark_tree_write leaves them.
 */
struct dspark_tree_cache {
    void *k, *v;
    uint8_t *k_scale, *v_scale;
    int64_t k_stride[3], v_stride[3];
    int64_t k_scale_stride[3], v_scale_stride[3];
    int64_t n_pages;
    int page_size;
    int type;
};

/*
 * The requests of one call, all arrays on the device: pages int32, max_pages
 * entries a request, the requests' rows pages_stride entries apart (max_pages *
 * page_size < 2^31; positions from DSPARK_TREE_MAX_LENGTH on are not used), start
 * int32 [B] (the position of the request's first row), first int32 [B + 1] (the
 * request's rows are first[b] .. first[b+1]-1 of the packed arrays; no two requests
 * have a row in common).  None of them changes while a call runs.  N: rows of the
 * packed arrays.
 */
struct dspark_tree_batch {
    const int32_t *pages;
    const int32_t *start;
    const int32_t *first; /* null for dspark_tree_keep */
    int64_t pages_stride;
    int max_pages;
    int B;
    int N;
};

/*
 * A handle on the current device: workspace and status word.
 * DSPARK_EINVAL: a size outside its range; DSPARK_EUNSUPPORTED: not sm_103.
 */
int dspark_tree_create(const struct dspark_tree_config *config, dspark_tree_t *out);

/*
 * Write rows of k and v ([N, kv_heads, head_dim], strides {row, head} in
 * elements, 16-byte multiples) at positions start[b] + i of the cache.
 */
int dspark_tree_write(dspark_tree_t h, const struct dspark_tree_cache *cache,
                      const struct dspark_tree_batch *batch, const void *k,
                      const int64_t *k_stride, const void *v, const int64_t *v_stride,
                      void *stream);

/*
 * Positions start[b] + i of the cache into rows of out_k and out_v
 * ([N, kv_heads, head_dim] contiguous, 16-byte aligned): code times scale rounded
 * once to the handle's type; values past its range become the largest finite
 * one.
 */
int dspark_tree_read(dspark_tree_t h, const struct dspark_tree_cache *cache,
                     const struct dspark_tree_batch *batch, void *out_k, void *out_v,
                     void *stream);

/*
 * Move position start[b] + path[b][i] of the cache to start[b] + i, i <
 * count[b].  path int32, rows path_stride entries apart, strictly ascending
 * from >= 0 in the first count[b] <= max_path <= 256 entries of a row.  Codes and scales move as they
 * are.  batch->first and batch->N are not read.
 */
int dspark_tree_keep(dspark_tree_t h, const struct dspark_tree_cache *cache,
                     const struct dspark_tree_batch *batch, const int32_t *path,
                     int64_t path_stride, int max_path, const int32_t *count, void *stream);

/*
 * Attention of the drafted rows (see above).  batch->start is the context's
 * length; the draft's own keys and values are already in the cache, at
 * start[b] + i.  q [N, q_heads, head_dim], strides {row, head} in elements
 * (16-byte multiples); mask uint32, mask_words words a row, rows mask_stride
 * words apart, or null (a chain); out [N, q_heads, head_dim] contiguous,
 * 16-byte aligned; lse fp32 [N, q_heads] or null.
 */
int dspark_tree_attend(dspark_tree_t h, const struct dspark_tree_cache *cache,
                       const struct dspark_tree_batch *batch, const void *q,
                       const int64_t *q_stride, const uint32_t *mask, int64_t mask_stride,
                       int mask_words, float scale, float softcap, void *out, float *lse,
                       void *stream);

/*
 * Norms of query and key heads, and the rotation by a token's position.  A row x of
 * head_dim elements (a multiple of 16) becomes, in fp32 with one rounding at the end:
 *
 *     y_d = x_d / sqrt(mean x^2 + eps) * norm_d         (without norm: y = x)
 *     t   = 2 pi position turns_i / 2^64                 pair i = (a, b):
 *     y_a, y_b = y_a cos t - y_b sin t, y_b cos t + y_a sin t
 *
 * for the pairs i < rotary_dim / 2 (rotary_dim a multiple of 16, from 0 to head_dim):
 * elements i and i + rotary_dim / 2, or, interleaved, 2 i and 2 i + 1.  The elements
 * past rotary_dim are not turned.  Rows of any size are normed: one whose squares leave
 * fp32 is multiplied by a power of two first.  Arrays on the device: turns [rotary_dim / 2], the
 * turns of a position as fractions of 2^64 (whole turns do not count), norms fp32
 * [head_dim], 16-byte aligned.
 */
struct dspark_tree_rotation {
    const uint64_t *turns;
    const float *q_norm; /* or null: no norm */
    const float *k_norm; /* or null */
    float eps;
    int rotary_dim;
    int interleaved;
};

/*
 * Rows of q [N, q_heads, head_dim] and k [N, kv_heads, head_dim] (strides {row, head}
 * in elements, 16-byte multiples) to out_q and out_k, contiguous, 16-byte aligned.
 * position int32 [N], of any sign.
 */
int dspark_tree_rotate(dspark_tree_t h, const struct dspark_tree_rotation *rotation,
                       const int32_t *position, int N, const void *q, const int64_t *q_stride,
                       const void *k, const int64_t *k_stride, void *out_q, void *out_k,
                       void *stream);

/*
 * The same with k and v on their way into the cache: rows of k, normed, rotated and
 * rounded, and of v as they are, go to slot[n] of the cache (page slot / page_size, place
 * slot % page_size; int32 [N], no two rows in the same slot), quantised where it is, as
 * dspark_tree_rotate and then dspark_tree_write leave them.  A row whose slot is below 0
 * is left out: out_q and the cache stay as they were there.  So is one past the cache, and
 * dspark_tree_status then returns DSPARK_EPAGES.  n_pages * page_size < 2^31.
 */
int dspark_tree_place(dspark_tree_t h, const struct dspark_tree_cache *cache, const int32_t *slot,
                      const struct dspark_tree_rotation *rotation, const int32_t *position, int N,
                      const void *q, const int64_t *q_stride, const void *k,
                      const int64_t *k_stride, const void *v, const int64_t *v_stride, void *out_q,
                      void *stream);

/* Wait for the stream; return and clear the handle's device status. */
int dspark_tree_status(dspark_tree_t h, void *stream);

int dspark_tree_destroy(dspark_tree_t h);

#ifdef __cplusplus
}
#endif

#endif
