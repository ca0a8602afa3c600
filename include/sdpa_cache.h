/*
 * sdpa_cache.h -- C ABI of the key/value cache on GB300 (sm_103a): attention of
 * a few new tokens over cached keys (single tokens, chains, trees of drafted
 * tokens), appending accepted tokens, weighing keys by the attention they get,
 * and evicting the light ones. It serves what sdpa_fwd.h computes for whole
 * prompts: the same scores, windows, sinks and grouped heads.
 *
 * The cache. Sequence i holds lengths[i] keys in its slots 0 .. lengths[i] - 1.
 * Slot j lies in page page_table[i][j / page_size], row j % page_size. Every
 * kv-head of a sequence holds the same number of keys; after an eviction the
 * heads of a sequence hold different tokens. A key's position is the number of
 * tokens that its sequence had taken in before it: positions[i][g][j], or j
 * itself without the positions array. next_pos[i] is the position of the next
 * token.
 *
 * Conventions (as in sdpa_bwd.h): the caller owns every buffer; calls enqueue
 * on `stream` and return without synchronising (except the status check);
 * arguments are checked on the host before anything is enqueued, with a message
 * in sdpa_bwd_last_error(). Each call can be captured into a CUDA graph and
 * replayed: lengths, counts, masks and tables are read on the device. Two calls
 * that change one cache, or one that changes and one that reads it, must be
 * ordered by the caller (one stream, or events).
 *
 * Problems found on the device are recorded in cache->status, first one wins:
 * SDPA_ERR_BAD_LENGTHS (a length, count or row index out of its range),
 * SDPA_ERR_BOUNDS (a page-table entry outside [0, n_pages)), SDPA_ERR_TIMEOUT
 * (a wait inside a kernel ran out; the call's outputs are not to be used).
 * Nothing outside the buffers is accessed then: each call says below what it
 * leaves out.
 */
#ifndef SDPA_CACHE_H
#define SDPA_CACHE_H

#include "sdpa_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * All strides are in elements; the feature stride is 1, every other stride a
 * non-negative multiple of 8 elements, k and v are 16-byte aligned. Arrays of
 * 4-byte entries are 4-byte aligned and contiguous.
 */
typedef struct sdpa_cache {
    int32_t dtype;              /* SDPA_BF16 | SDPA_F16 for K, V and the calls' tensors */
    int32_t reserved0;
    int64_t b, h_kv, d;         /* sequences, kv-heads (up to 4096), head dimension (64 or 128) */
    int64_t n_pages, page_size; /* pages in k and v, rows of a page (any number >= 1) */
    int64_t max_pages;          /* entries of a page-table row; a sequence has room for
                                   max_pages * page_size keys (its capacity, at most
                                   2^31 - 2^16) */
    void *k, *v;                /* device [n_pages][page_size][h_kv][d] */
    int64_t k_stride[3], v_stride[3]; /* page, row, head */
    const int32_t *page_table;  /* device [b][max_pages]; NULL: page i is sequence i's only one
                                   (max_pages = 1, n_pages >= b). Entries behind a sequence's
                                   keys are not read. A page may be in several places (a common
                                   prefix) as long as no call writes it: append writes the slots
                                   behind a sequence's keys, evict any slot below its length. */
    int32_t *lengths;           /* device [b] */
    int32_t *next_pos;          /* device [b] with positions, else NULL (equal to lengths) */
    int32_t *positions;         /* device [b][h_kv][capacity] or NULL (the slot's number) */
    float *weights;             /* device [b][h_kv][capacity] or NULL: attention weight of each key */
    int32_t *status;            /* device [1], zero at first: the first problem found */
} sdpa_cache;

/* sizeof of the structs as compiled into the library, for binding checks. */
size_t sdpa_cache_bytes(void);
size_t sdpa_cache_fwd_params_bytes(void);
size_t sdpa_cache_append_params_bytes(void);
size_t sdpa_cache_weigh_params_bytes(void);
size_t sdpa_cache_evict_params_bytes(void);

/*
 * Attention of up to 64 new tokens per sequence over the cached keys and over
 * each other. The new tokens' own keys and values are not in the cache yet. More
 * tokens take several calls, each followed by an append; a whole prompt is
 * sdpa_fwd's, whose keys lie in one run.
 *
 * tree[i][r] says which of sequence i's new tokens token r descends from: bit u
 * is set for u = r and for every token on the way from the root to r. Token r's
 * position is next_pos[i] + (number of set bits - 1). A mask without its own bit
 * is an empty row (padding): it admits no key, while its token keeps the position
 * that its bits say for rows that list it. Without masks the tokens are a chain.
 * Token r admits
 *     cached key j    iff  pos_r - pos_j <= window_left  (if window_left >= 0)
 *     new key u       iff  bit u is set and pos_r - pos_u <= window_left
 * and, with s over the admitted keys (scale * q . k),
 *     LSE = log( sum exp(s) + exp(sink_h) )     (sink term only with a sink)
 *     O   = sum exp(s - LSE) v.
 * A row that admits no key gets O = 0 and LSE = -inf, or LSE = sink_h with a
 * sink. A row that admits one and has a NaN in its q gets NaN for both. Rows at
 * or behind seq_q_lens[i] get O = 0, LSE = -inf, and their keys are not admitted
 * by any row; bits at or behind it are ignored.
 * Sums, maxima and O are kept in fp32. For the P V product P is split into a
 * 16-bit value and its 16-bit remainder where a kv-head has up to 8 rows (s_q *
 * h_q / h_kv; d = 64: up to 16), and rounded to the I/O dtype, as sdpa_fwd
 * does, where it has more. In f16 P is held on a grid of 2^-31 of the row's
 * heaviest key, or finer: keys lighter than half of that count in LSE alone.
 * Keys on pages out of range are left out; lengths out of [0, capacity] are
 * taken as the nearer end. Not read, or without effect whatever they hold, are
 * slots behind a sequence's keys, keys that no row's window has, and new tokens
 * that no row admits. The other keys' K and V have to be finite, those too that
 * only some rows admit: a masked V meets a P of 0.
 */
typedef struct sdpa_cache_fwd_params {
    int64_t s_q, h_q;                    /* new tokens per sequence (1..64), q-heads */
    int64_t window_left;                 /* -1: no window */
    float scale;
    int32_t reserved0;
    const void *q;                       /* device [b][s_q][h_q][d] */
    const void *k, *v;                   /* device [b][s_q][h_kv][d] */
    int64_t q_stride[3], k_stride[3], v_stride[3], o_stride[3]; /* batch, token, head */
    const int64_t *tree;                 /* device [b][s_q] or NULL (a chain) */
    const int32_t *seq_q_lens;           /* device [b] or NULL (s_q each) */
    const float *sink;                   /* device [h_q] or NULL */
    void *o;                             /* device [b][s_q][h_q][d] */
    float *lse;                          /* device fp32 [b][h_q][s_q], contiguous */
} sdpa_cache_fwd_params;

/* Workspace of sdpa_cache_fwd in bytes: 0 on invalid arguments (then
 * sdpa_bwd_last_error() names one) and where none is needed (it is empty, and
 * the workspace may be NULL). It needs no initialisation and is 256-byte
 * aligned. Calls that may overlap on the GPU (other streams, two graphs) need a
 * workspace each. */
size_t sdpa_cache_fwd_workspace_bytes(const sdpa_cache *cache, const sdpa_cache_fwd_params *params);
sdpa_status_t sdpa_cache_fwd(const sdpa_cache *cache, const sdpa_cache_fwd_params *params, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * Puts new keys and values behind each sequence's cached ones, in order, at the
 * positions from next_pos on, with weight 0, and moves lengths and next_pos on.
 *  SDPA_BSHD: k, v [b][s][h_kv][d]; counts[i] rows of sequence i (s, or n with
 *    an index, each without counts): rows 0, 1, .. or, with index [b][n], rows
 *    index[i][0], index[i][1], .. (the accepted ones of drafted tokens).
 *  SDPA_THD: k, v [total][h_kv][d], offsets [b+1] with offsets[0] = 0 and
 *    offsets[b] = total; s at least the longest slot. counts[i] as above (the
 *    whole slot without counts); index is not taken.
 * A sequence whose new rows do not fit its capacity, whose count is out of
 * range, or one of whose indexes or pages is, is left as it was and reported.
 */
typedef struct sdpa_cache_append_params {
    int32_t layout;
    int32_t reserved0;
    int64_t s, n, total;          /* rows per sequence, index entries per sequence, THD rows */
    const void *k, *v;
    int64_t k_stride[3], v_stride[3];   /* batch (THD: ignored), token, head */
    const int32_t *index;         /* device [b][n] or NULL */
    const int32_t *counts;        /* device [b] or NULL */
    const int32_t *offsets;       /* device [b+1], THD only */
} sdpa_cache_append_params;
sdpa_status_t sdpa_cache_append(const sdpa_cache *cache, const sdpa_cache_append_params *params, void *stream);

/*
 * Adds to each cached key's weight the attention that it gets from given rows:
 *     weights[i][g][j] += sum over rows r and the q-heads h of group g of
 *                         exp(scale * q_r . k_j - lse_r)
 * over the rows with q_pos >= 0 and a finite LSE that admit the key:
 * pos_j <= q_pos, and q_pos - pos_j <= window_left (if >= 0). Without q_pos the
 * rows are the last s_q tokens: q_pos = next_pos - s_q + r. The sum over a
 * key's rows is formed in fp32 in a fixed order (bitwise repeatable). Keys on
 * pages out of range keep their weight; such a page may be reported although no
 * row's window has a key on it. A key's K has to be finite, and the q of
 * rows that count.
 */
typedef struct sdpa_cache_weigh_params {
    int64_t s_q, h_q;             /* rows per sequence (>= 1), q-heads */
    int64_t window_left;          /* -1: no window */
    float scale;
    int32_t reserved0;
    const void *q;                /* device [b][s_q][h_q][d] */
    int64_t q_stride[3];
    const float *lse;             /* device fp32 [b][h_q][s_q], contiguous */
    const int32_t *q_pos;         /* device [b][s_q] or NULL */
} sdpa_cache_weigh_params;
sdpa_status_t sdpa_cache_weigh(const sdpa_cache *cache, const sdpa_cache_weigh_params *params, void *stream);

/*
 * Brings each sequence that holds more than `keep` keys back to `keep`, for each
 * kv-head on its own. Kept are the keys at positions below `first`, those at
 * positions >= next_pos - recent, and of the others the heaviest (ties: the
 * lowest slot; NaN counts as heavier than every number). Should the protected
 * ones alone be more than `keep`, those in the lowest slots stay. Kept keys in
 * slots below `keep` stay where they are; the others, in slot order, fill the
 * free slots below `keep` in slot order, with their positions and weights.
 * Slots from `keep` on are left as they were. Sequences that hold no more than
 * `keep` keys are not touched. Needs positions and weights. A sequence whose
 * length is out of range is left alone; K and V on pages out of range do not
 * move (their positions and weights do).
 */
typedef struct sdpa_cache_evict_params {
    int64_t keep, first, recent;  /* keep >= first + recent, all >= 0 */
} sdpa_cache_evict_params;
size_t sdpa_cache_evict_workspace_bytes(const sdpa_cache *cache, const sdpa_cache_evict_params *params);
sdpa_status_t sdpa_cache_evict(const sdpa_cache *cache, const sdpa_cache_evict_params *params, void *workspace,
                               size_t workspace_bytes, void *stream);

/*
 * Test-only hook of the bounded waits (defaults: 2 s, no flags). A wait that
 * runs out records SDPA_ERR_TIMEOUT: the kernel sends no more copies, lets
 * those and the products in flight finish, frees its tensor memory and returns.
 * This call changes, for the calling thread's later calls on any cache:
 *   wait_limit_ns  the bound of every device wait (<= 0: the default);
 *   flags          bit 0: forward, weigh and evict leave out copies that a
 *                  wait is for, so that it runs out; 0: normal operation.
 * Returns SDPA_ERR_INVALID_ARG for undefined flag bits. Call it with (0, 0) to
 * restore normal operation.
 */
sdpa_status_t sdpa_cache_test_hook(int64_t wait_limit_ns, int32_t flags);

/* Synchronises `stream`, returns the cache's status word and clears it. */
sdpa_status_t sdpa_cache_check_status(const sdpa_cache *cache, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SDPA_CACHE_H */
