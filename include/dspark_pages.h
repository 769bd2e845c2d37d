/*
 * dspark_pages.h -- C ABI of the page tables of a paged key/value cache (dspark_tree.h),
 * kept on the GPU (GB300, sm_103a): which pages a request holds, pages handed out as
 * requests grow and taken back as they shrink, and the offsets, slots and positions of
 * a round's rows, all from lengths that stay on the device.
 *
 * All state is the caller's memory on the device.  Calls on one set of tables are ordered
 * by the caller; they launch one kernel each on `stream` of the current device, copy
 * nothing to the host and are graph-capturable.  Conventions as in dspark_walk.h.
 *
 * Request r holds the first held[r] entries of its row of the table; the others are -1.
 * free[0 .. n_free-1] are the pages that no request holds, handed out from the end.
 */
#ifndef DSPARK_PAGES_H
#define DSPARK_PAGES_H

#include "dspark_walk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DSPARK_PAGES_MAX_REQUESTS 1024

struct dspark_pages {
    int32_t *table;       /* [requests, max_pages], rows table_stride entries apart */
    int32_t *held;        /* [requests] */
    int32_t *free;        /* [n_pages] */
    int32_t *n_free;      /* [1] */
    int32_t *state;       /* [2]: status word, and 0 between calls */
    int64_t table_stride;
    int n_pages;          /* n_pages * page_size < 2^31 */
    int page_size;
    int requests;         /* 1 .. DSPARK_PAGES_MAX_REQUESTS */
    int max_pages;        /* of a request; max_pages * page_size < 2^31 */
};

/* All pages free, page 0 handed out first; no request holds any. */
int dspark_pages_reset(const struct dspark_pages *p, void *stream);

/*
 * Request r, which has length[r] cached rows, is to have count[r] more: it gets the pages
 * that it lacks for them (requests in order), and of its rows, first[r] + i for i <
 * count[r], N of all requests:
 *
 *     first[r]    = count[0] + .. + count[r-1]             (int32 [requests + 1])
 *     slot[n]     = table[r][pos / page_size] * page_size + pos % page_size,
 *                   pos = length[r] + i                    (int32 [N])
 *     position[n] = pos, or, with a mask, length[r] plus the set bits of row n less one:
 *                   a tree's node by its depth             (int32 [N])
 *
 * mask uint32, mask_words words a row, rows mask_stride words apart, or null.  Rows from
 * first[requests] on get slot and position -1.  A request whose numbers do not fit (below 0,
 * past max_pages) gets no pages, its rows slot and position -1.  Free pages go to the requests
 * in order and to none past its turn: the first request that they do not serve gets none, its
 * rows slot -1, nor does any later one that lacks a page, also where one is left for it; those
 * that lack none get their slots all the same.  Of a request whose rows go past N those below N
 * get slot and position -1.  dspark_pages_status then returns DSPARK_EPAGES.  A count below 0
 * counts as 0 in first.
 */
int dspark_pages_grow(const struct dspark_pages *p, const int32_t *length, const int32_t *count,
                      int N, const uint32_t *mask, int64_t mask_stride, int mask_words,
                      int32_t *first, int32_t *slot, int32_t *position, void *stream);

/*
 * Request r keeps the pages of its first length[r] rows and gives the others back, so that
 * trim after grow with the same lengths leaves everything as it was, where no request held
 * more pages before than its length needs (trim takes those, too).  length[r] = 0: all of
 * them.  A length below 0 or past max_pages changes nothing of its request and is reported
 * as above.  So is an entry of the table on its way back that is no page of the pool: it
 * leaves the table and becomes no free page, so n_free grows by the others alone.
 */
int dspark_pages_trim(const struct dspark_pages *p, const int32_t *length, void *stream);

/* Wait for the stream; return and clear the status word. */
int dspark_pages_status(const struct dspark_pages *p, void *stream);

#ifdef __cplusplus
}
#endif

#endif
