/*
 * spmm_dynamic.h -- C ABI of the products whose sparse matrix a model chooses
 * anew in every call (libspmm.so; spmm.h holds the products with a fixed A).
 *
 *   routes  tokens x slots: tokens sorted by expert, gathered, each expert's rows
 *           times its matrix, and the experts' rows weighted and added back per
 *           token, with every gradient.
 *   blocks  queries x key blocks: each query attends to the key blocks that a
 *           cheap score selects for it; forward, single tokens over a cache,
 *           and backward (through the transpose of the selection).
 *   heads   what comes before the blocks: queries and keys, each head normed and
 *           its pairs of elements turned by the token's position (a block-diagonal
 *           matrix of 2 x 2 rotations), also written into a cache, and the gradient.
 *
 * Conventions are spmm.h's: device pointers of the current device, `stream` a
 * cudaStream_t as void*, argument checks on the host before any CUDA call, no
 * exception and no trap. Besides:
 *   - Every call is asynchronous and allocates nothing. Where one needs
 *     scratch, the caller passes `work` of at least the bytes that the matching
 *     *_workspace function returns (16-byte aligned); the scratch holds nothing
 *     between calls.
 *   - Elements are fp32, bf16 or fp16 (spmm_dtype). Sums, scores, softmax
 *     statistics and the routes' weights are fp32; an output is rounded to its
 *     type once. Attention's weights are rounded to the inputs' type where they
 *     enter a matrix product; dS enters it as two such parts; the gradients'
 *     <dO, O> is formed from the rounded output.
 *   - Results are bitwise reproducible run to run: no floating-point atomics.
 */
#ifndef GB300_SPMM_DYNAMIC_H
#define GB300_SPMM_DYNAMIC_H

#include "spmm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { SPMM_F32 = 0, SPMM_BF16 = 1, SPMM_F16 = 2 } spmm_dtype;

/*
 * spmm_dynamic_sync -- wait for `stream`, then report SPMM_ERR_TIMEOUT if a
 * bounded device-side wait of one of these calls on it gave up since it was last
 * asked (its outputs are then incomplete), or one in a captured graph, whichever
 * stream of the current device replayed it: each stream is told of a graph's once.
 * Synchronous.
 */
spmm_status spmm_dynamic_sync(void *stream);

/*
 * spmm_dynamic_check_wait_timeout -- diagnostic of that path, as
 * spmm_check_wait_timeout is of a plan's: one warp on `stream` waits for an
 * arrival that nobody makes and gives up after limit_us microseconds (1 to 10^7),
 * as a broken wait of these calls would. Asynchronous.
 */
spmm_status spmm_dynamic_check_wait_timeout(int64_t limit_us, void *stream);

/* ------------------------------------------------------------------ routes */

/* Largest number of experts (the sort keeps a counter per warp and expert in
 * shared memory). */
#define SPMM_ROUTES_MAX_EXPERTS 2048

/* Bytes of scratch spmm_routes_sort needs (0 for few pairs or bad arguments). */
int64_t spmm_routes_workspace(int64_t T, int64_t k, int64_t E);

/*
 * spmm_routes_sort -- a stable sort of the pairs (t, j) by expert.
 *   ids     : device, int32 [T, k]: the expert of token t's j-th choice. A value
 *             outside [0, E) drops the pair (over capacity, padding).
 *   slots   : device, int32 [T, k], written: the pair's rank among the kept
 *             pairs in order of (expert, t, j); -1 for a dropped pair.
 *   offsets : device, int32 [E + 1], written: expert e owns the slots
 *             [offsets[e], offsets[e + 1]); offsets[E] pairs are kept.
 * T * k < 2^31 and E <= SPMM_ROUTES_MAX_EXPERTS, else SPMM_ERR_UNSUPPORTED.
 */
spmm_status spmm_routes_sort(const int32_t *ids, int64_t T, int64_t k, int64_t E, int32_t *slots,
                             int32_t *offsets, void *work, int64_t work_bytes, void *stream);

/*
 * spmm_routes_dispatch -- xs[slots[t, j]] = x[t]; rows offsets[E] .. T k - 1 of
 * xs are set to 0.
 *   x  : device, [T, H] of `dtype`, rows `ldx` elements apart (>= 0; 0 is one
 *        row for every token), elements of a row adjacent.
 *   xs : device, [T k, H], contiguous, written.
 * 16-byte accesses when H, ldx and the pointers allow, else element by element.
 */
spmm_status spmm_routes_dispatch(int dtype, const void *x, int64_t ldx, const int32_t *slots,
                                 const int32_t *offsets, int64_t T, int64_t k, int64_t E,
                                 int64_t H, void *xs, void *stream);

/*
 * spmm_routes_combine -- out[t] = sum_j w[t, j] y[slots[t, j]], in the order of
 * j, in fp32. Dropped pairs are skipped; a token whose pairs are all dropped
 * gives 0. With w NULL (every weight 1) it is the gradient of dispatch.
 *   y : device, [T k, H], contiguous. w : device, fp32 [T, k] or NULL.
 *   out : device, [T, H], contiguous, written.
 */
spmm_status spmm_routes_combine(int dtype, const void *y, const float *w, const int32_t *slots,
                                const int32_t *offsets, int64_t T, int64_t k, int64_t E,
                                int64_t H, void *out, void *stream);

/*
 * spmm_routes_combine_backward -- the gradients of combine:
 *   dy[slots[t, j]] = w[t, j] dout[t]  (rows offsets[E] .. are set to 0),
 *   dw[t, j] = <dout[t], y[slots[t, j]]>, 0 for a dropped pair.
 *   dout : device, [T, H], rows `lddout` elements apart (as x above).
 *   dw   : device, fp32 [T, k], written, or NULL to skip it.
 */
spmm_status spmm_routes_combine_backward(int dtype, const void *dout, int64_t lddout,
                                         const void *y, const float *w, const int32_t *slots,
                                         const int32_t *offsets, int64_t T, int64_t k, int64_t E,
                                         int64_t H, void *dy, float *dw, void *stream);

/*
 * spmm_routes_product -- each expert's rows times its matrix:
 *   ys[s, f] = sum_h xs[s, h] w[e, h, f] for the slots s of expert e;
 * rows offsets[E] .. P - 1 of ys are set to 0, those of xs do not matter.
 *   xs : device, [P, H], contiguous (P = T k slots). ys : device, [P, F], contiguous, written.
 *   w  : device, [E, H, F], element strides w_se, w_sh, w_sf. One of w_sh and w_sf
 *        is 1; the other and w_se are multiples of 8 (w_se may be 0: one matrix
 *        for every expert).
 * With w transposed (w_sh and w_sf, H and F exchanged) it is the gradient of xs.
 * dtype is SPMM_BF16 or SPMM_F16, H and F multiples of 8 up to 2^20, E at most
 * SPMM_ROUTES_MAX_EXPERTS, P below 2^31 - 2^16, strides below 2^38 (else
 * SPMM_ERR_UNSUPPORTED); pointers are 16-byte aligned.
 */
spmm_status spmm_routes_product(int dtype, const void *xs, const void *w, int64_t w_se,
                                int64_t w_sh, int64_t w_sf, const int32_t *offsets, int64_t P,
                                int64_t E, int64_t H, int64_t F, void *ys, void *stream);

/*
 * spmm_routes_product_weights -- the gradient of the matrices:
 *   dw[e, h, f] = sum over the slots s of e of xs[s, h] dys[s, f]; 0 without slots.
 *   dw : device, written whole, strides as w's above, no two elements in one place.
 * Scratch: for few experts with many slots, and for more than 2^24 slots, which are then
 * summed in parts.
 */
int64_t spmm_routes_product_weights_workspace(int64_t P, int64_t E, int64_t H, int64_t F);
spmm_status spmm_routes_product_weights(int dtype, const void *xs, const void *dys,
                                        const int32_t *offsets, int64_t P, int64_t E, int64_t H,
                                        int64_t F, void *dw, int64_t dw_se, int64_t dw_sh,
                                        int64_t dw_sf, void *work, int64_t work_bytes,
                                        void *stream);

/* ------------------------------------------------------------------ blocks */

/* A [B, T, heads, D] tensor: element strides of the first three dimensions; the
 * D elements of a row are adjacent. Rows are 16-byte aligned: `data` a multiple
 * of 16 bytes and the strides multiples of 16 bytes. */
typedef struct {
    const void *data;
    int64_t sb, st, sh;
} spmm_rows;

/*
 * What the block calls share. Sequence b holds len_b = lengths[b] keys (clamped
 * to [0, Tk]; lengths NULL: Tk) in blocks of `block`; its Tq queries are its
 * last tokens: query i sits at position len_b - Tq + i. Causal, it sees the keys
 * up to its position (none if that is negative); otherwise all len_b keys.
 * Keys past those are never used, whatever they hold.
 * Head h of Hq reads the keys and the selection of head h / (Hq / Hk).
 * Limits, beyond which a call is SPMM_ERR_UNSUPPORTED: Tq and Tk 2^26, n 2^20,
 * Hq 65535, B Tq Hq < 2^31, B Tk Hk 2^40.
 */
typedef struct {
    int64_t B, Tq, Tk, Hq, Hk, D;
    int64_t block;           /* 16, 32, 64 or 128                                  */
    int64_t n;               /* entries of a query's list                          */
    int32_t dtype;           /* SPMM_BF16 or SPMM_F16 (means and select: also F32) */
    int32_t causal;
    float scale;             /* of q . k                                           */
    const int32_t *lengths;  /* device, int32 [B], or NULL                         */
} spmm_blocks_shape;

/*
 * spmm_blocks_means -- means[b, c, h] = the mean of block c's valid keys, fp32
 * [B, ceil(Tk / block), Hk, D] contiguous; 0 for a block without any.
 *   new_keys : < 0 writes every block; otherwise only the blocks that hold one
 *              of the sequence's last new_keys keys (after appending them).
 * D a multiple of 8, at most 256. Uses B, Tk, Hk, D, block, dtype, lengths.
 */
spmm_status spmm_blocks_means(const spmm_blocks_shape *s, spmm_rows k, int64_t new_keys,
                              float *means, void *stream);

/*
 * spmm_blocks_select -- the list of blocks each query attends to, int32
 * [B, Tq, Hk, n], ascending, filled up with -1.
 *   score(query, c) = (sum of the group's query rows) . means[c], in fp32.
 * Causal: the block of the query's own position, and the n - 1 blocks before it
 * with the largest scores. Otherwise the n largest of all blocks that hold a
 * key. Equal scores go to the lowest block; NaN is below every number.
 * Prompts are taken in strips of queries: the scratch is at most 1 GB or, if that is
 * more, the scores of 64 queries of each sequence (of fewer than 24: of all of them).
 */
int64_t spmm_blocks_select_workspace(const spmm_blocks_shape *s);
spmm_status spmm_blocks_select(const spmm_blocks_shape *s, spmm_rows q, const float *means,
                               int32_t *blocks, void *work, int64_t work_bytes, void *stream);

/*
 * spmm_blocks_select_kept -- the same, and a copy of lengths as the lists were made
 * for them: int32 [B] at `kept` (NULL: none; not written without lengths or queries).
 * A caller that adds to its lengths in place passes the copy to the calls below.
 */
spmm_status spmm_blocks_select_kept(const spmm_blocks_shape *s, spmm_rows q, const float *means,
                                    int32_t *blocks, int32_t *kept, void *work, int64_t work_bytes,
                                    void *stream);

/*
 * spmm_blocks_check -- whether every list is strictly ascending block numbers
 * below ceil(Tk / block), then only -1: writes 0 or 1 (a bad list exists) to
 * the device word *bad. The calls below skip an entry that is out of range or
 * not above the one before it.
 */
spmm_status spmm_blocks_check(const spmm_blocks_shape *s, const int32_t *blocks, int32_t *bad,
                              void *stream);

/*
 * spmm_blocks_attend -- softmax attention of each query over the seen keys of
 * its blocks: out [B, Tq, Hq, D] contiguous of `dtype`, and lse fp32
 * [B, Tq, Hq], the natural logarithm of the sum of exp(scale q . k). A query
 * that sees no key gives 0 and -infinity. D is 64 or 128.
 */
spmm_status spmm_blocks_attend(const spmm_blocks_shape *s, spmm_rows q, spmm_rows k, spmm_rows v,
                               const int32_t *blocks, void *out, float *lse, void *stream);

/*
 * spmm_blocks_backward -- the gradients of out with respect to q, k and v (the
 * selection is a constant): dq [B, Tq, Hq, D], dk and dv [B, Tk, Hk, D], all
 * contiguous and written whole (0 where nothing attends).
 *   out, lse : as attend wrote them. dout : the gradient of out.
 */
int64_t spmm_blocks_backward_workspace(const spmm_blocks_shape *s);
spmm_status spmm_blocks_backward(const spmm_blocks_shape *s, spmm_rows q, spmm_rows k,
                                 spmm_rows v, const int32_t *blocks, const void *out,
                                 const float *lse, spmm_rows dout, void *dq, void *dk, void *dv,
                                 void *work, int64_t work_bytes, void *stream);

/* ------------------------------------------------------------------- heads */

/*
 * What the calls on heads share. A token's heads [H, D] of queries (Hq) and keys
 * (Hk, may be 0) become, with a weight [D] for the tensor, z = x w / sqrt(mean(x^2) + eps),
 * else z = x; then the first R elements are turned in pairs by the angle
 * 2 pi 2^-64 turns[i] p, p the token's position (an integer product mod 2^64:
 * exact at any position):
 *   y1 = magnitude (z1 cos - z2 sin), y2 = magnitude (z2 cos + z1 sin),
 * pairs being (i, i + R / 2) or, interleaved, (2 i, 2 i + 1); elements from R on are z.
 * Token t of sequence b is at positions[b p_sb + t p_st], else, with lengths, at
 * lengths[b] - T + t, else at t. Positions may be negative.
 * Sums and angles are fp32 or better; results are rounded once.
 * D and R are multiples of 16, D at most 256, R at most D; tensors are spmm_rows
 * of fp32, bf16 or fp16. Limits, else SPMM_ERR_UNSUPPORTED: T 2^26, Hq and Hk 65535,
 * B T (Hq + Hk) < 2^31.
 */
typedef struct {
    int64_t B, T, Hq, Hk, D, R;
    int32_t dtype;               /* of the tensors                                   */
    int32_t weight_dtype;        /* of the weights: SPMM_F32 or dtype                */
    int32_t interleaved;
    float eps, magnitude;
    const uint64_t *turns;       /* device, [R / 2], 16-byte aligned                 */
    const int32_t *positions;    /* device, or NULL                                  */
    int64_t p_sb, p_st;
    const int32_t *lengths;      /* device, int32 [B], or NULL                       */
    const void *wq, *wk;         /* device, [D], 16-byte aligned, or NULL            */
} spmm_heads_shape;

/* spmm_heads_rotate -- q_out [B, T, Hq, D] and k_out [B, T, Hk, D], contiguous, written. */
spmm_status spmm_heads_rotate(const spmm_heads_shape *s, spmm_rows q, spmm_rows k, void *q_out,
                              void *k_out, void *stream);

/*
 * spmm_heads_append -- the same, the new keys going into a cache [B, Tk, Hk, D] at
 * their positions and the values v [B, T, Hk, D] as they are into another. Needs
 * lengths (those after the new tokens) and no positions. Keys at positions outside
 * [0, Tk) are not written; every other row of the caches stays as it is.
 * The caches overlap neither each other nor q, k and v.
 */
spmm_status spmm_heads_append(const spmm_heads_shape *s, spmm_rows q, spmm_rows k, spmm_rows v,
                              void *q_out, spmm_rows cache_k, spmm_rows cache_v, int64_t Tk,
                              void *stream);

/*
 * spmm_heads_rotate_backward -- the gradients of q, k and the weights, given those of
 * rotate's results. dq, dk contiguous, dwq, dwk [D] of weight_dtype (NULL where there is no
 * weight), all written. q and k are read for tensors with a weight only.
 */
int64_t spmm_heads_backward_workspace(const spmm_heads_shape *s);
spmm_status spmm_heads_rotate_backward(const spmm_heads_shape *s, spmm_rows grad_q,
                                       spmm_rows grad_k, spmm_rows q, spmm_rows k, void *dq,
                                       void *dk, void *dwq, void *dwk, void *work,
                                       int64_t work_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GB300_SPMM_DYNAMIC_H */
