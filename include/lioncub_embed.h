/*
 * lioncub_embed.h -- C ABI of the input-layer operators: the embedding lookup
 * with scaling, its gradient by sorted tokens, and dropout from a
 * counter-based generator whose mask is never stored.
 *
 * They produce and consume what the compressed Lion step of lioncub.h works
 * on: the lookup reads the fp32 parameters (or a bf16 copy), and its gradient
 * fills the dense rows of the input embedding inside a worker's flat gradient
 * vector -- the tensor whose momentum "Lion Cub: Minimizing Communication
 * Overhead in Distributed Lion" synchronizes, and the one whose rows are exact
 * zeros for every token that a batch does not hold.
 *
 * With i a place of the batch, j a column, e = i * dim + j:
 *   lookup    out[i,j]  = keep(e) ? RN(r * RN(RN(scale * table[t_i,j]) + pos_table[q_i,j])) : 0
 *   gradient  grad[v,j] = base[v,j] + f * sum over i with t_i == v of keep(e) ? dout[i,j] : 0,  f = RN(scale * r)
 *             pos_grad[q,j] = pos_base[q,j] + r * sum over i with q_i == q, t_i a token, of the same
 *   dropout   out[e] = (keep(e) ? RN(r * x[e]) : 0) (+ residual[e], rounded once more)
 * RN is a rounding to fp32; every operation is in fp32 and the result is
 * rounded once to the output's type.  Terms without a base, a position table,
 * or dropout are left out (keep true, r = 1).  A dropped element is 0 whatever
 * its value, an infinity or a NaN included.
 *
 * Places: t_i is a token id.  A negative id marks an empty place: its output
 * row is zeros, and its row of dout is not read.  An id >= vocab is treated
 * like an empty place and sets LIONCUB_EMBED_STATUS_INDEX in the handle's
 * status word.  q_i is positions[i], or first_position + i % seq_len when
 * positions is NULL; an explicit position outside [0, positions) adds no
 * position row, has no position gradient, and sets the same status bit.  The
 * position of an empty place may be anything.
 *
 * Random numbers: SplitMix64 (Steele, Lea and Flood 2014) as a function of
 * (start, k): output number k (from 0) of the generator that starts at
 * `start`.  The key is output number `stream` of `seed`; element e uses the
 * 16-bit field e % 4 (field 0 the lowest) of output number e / 4 of the key,
 * u16, and keep(e) = u16 >= T with T = floor(65536 p + 0.5).  r = RN(65536 /
 * (65536 - T)) (0 when T == 65536), the exact inverse of the share kept, so
 * the expectation is unbiased.  The element number is the logical one (row *
 * columns + column), whatever the strides, so a lookup with dropout equals a
 * lookup followed by dropout with the same seed and stream.  Give each (step,
 * worker, layer) a stream of its own.
 *
 * The sums of the gradient are fp32 in an order that depends on the batch, the
 * width, whether every matrix allows 16-byte moves (see lioncub_rows) and, for
 * positions, whether they are given or run; never on the schedule.  So a call
 * repeats bit for bit, but long sums may differ in their last bits from those of
 * the same values laid out otherwise.
 *
 * Calls only enqueue kernels on `stream`: nothing is allocated or
 * synchronized outside create, and a call can be captured into a CUDA graph
 * (the seed and stream are then frozen in it).  A handle's workspace is used
 * by backward calls only; they must be ordered one after another (one stream,
 * or events between them), on the host too.  Forward calls and dropout share
 * nothing and may be made by several host threads at once.
 * Return codes are those of lioncub.h.
 */
#ifndef LIONCUB_EMBED_H
#define LIONCUB_EMBED_H

#include "lioncub.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct lioncub_embed_s* lioncub_embed_t;

/* Element types of lioncub_rows; the values of LIONCUB_GRAD_*. */
enum { LIONCUB_ROWS_BF16 = 0, LIONCUB_ROWS_F32 = 1 };
enum { LIONCUB_INDEX_I64 = 0, LIONCUB_INDEX_I32 = 1 };

enum {
    LIONCUB_EMBED_MAX_VOCAB = 1 << 20, /* rows of either table          */
    LIONCUB_EMBED_MAX_DIM = 1 << 16,
    LIONCUB_EMBED_MAX_TOKENS = 1 << 30
};

/* Bits of the status word, beside LIONCUB_STATUS_OUT_OF_BOUNDS and
 * LIONCUB_STATUS_GUARD (sticky until destroy). */
enum { LIONCUB_EMBED_STATUS_INDEX = 8 /* a token id or position beyond its table */ };

/* A matrix in device memory: row i starts at data + i * stride elements, its
 * columns are contiguous.  Any element alignment works; rows whose starts are
 * 16-byte aligned and whose width is a multiple of 8 are moved 16 bytes at a
 * time. */
typedef struct {
    void* data;
    int64_t stride; /* elements between rows, >= the row's width */
    int32_t type;   /* LIONCUB_ROWS_* */
    int32_t reserved;
} lioncub_rows;

/* The places of a batch: n token ids, and where they stand. */
typedef struct {
    const void* tokens;     /* n ids, device                                        */
    const void* positions;  /* n positions, device, or NULL: first + i % seq_len    */
    int64_t n;
    int64_t seq_len;        /* >= 1 (read only when positions is NULL)              */
    int64_t first_position; /* >= 0 (read only when positions is NULL)              */
    int32_t index_type;     /* LIONCUB_INDEX_*, of both arrays                      */
    int32_t reserved;
} lioncub_token_batch;

typedef struct {
    uint64_t seed, stream;
    float p; /* probability of dropping, 0..1 (to the nearest 1/65536) */
    uint32_t reserved;
} lioncub_drop;

/*
 * A layer of `vocab` token rows and `positions` position rows (0: none) of
 * `dim` columns, for batches of at most max_tokens places; `scale` multiplies
 * the token rows.  Allocates the workspace of the gradient, which lookups do not
 * use (16 bytes a place and table, 8 a row of either table, about 4 * dim bytes
 * for every 16 to 64 places and table; 23 MB for 65536 places of 2048 columns
 * with positions), on the current device, which must be current in every later
 * call on the handle, and synchronizes the legacy default stream once.  LIONCUB_FAIL_ALLOC and
 * LIONCUB_FAIL_LAUNCH (lioncub.h) apply to the handle's own allocations and
 * kernel launches.  Errors: ERR_ARG, ERR_OOM, ERR_CUDA (*out is NULL then).
 */
LIONCUB_API int lioncub_embed_create(lioncub_embed_t* out, int64_t vocab, int64_t dim, int64_t positions,
                                     int64_t max_tokens, float scale);

/*
 * out (n x dim) from table (vocab x dim) and, unless it is NULL, pos_table
 * (positions x dim, of table's type).  drop may be NULL.  One launch; a single
 * token of a sequence that is being generated is a batch with n == 1 and its
 * place in first_position.  out must not overlap the tables, the tokens or
 * the positions it reads.  Errors:
 * ERR_ARG, ERR_ALIGN (a pointer that is not aligned to its element), ERR_STATE
 * (another device is current), ERR_CUDA.
 */
LIONCUB_API int lioncub_embed_forward(lioncub_embed_t h, const lioncub_token_batch* batch, const lioncub_rows* table,
                                      const lioncub_rows* pos_table, const lioncub_rows* out,
                                      const lioncub_drop* drop, lioncub_stream_t stream);

/*
 * The gradients of both tables from dout (n x dim): every row of grad (vocab x
 * dim) is written, rows without a token with zeros or their row of base.
 * base (NULL: zeros) and grad have one type; base->data == grad->data (then
 * with the same stride) adds in place and touches only the rows of the
 * batch's tokens.  pos_grad (NULL: not wanted) and pos_base likewise, of
 * grad's type.  The two gradients may overlap neither each other, nor dout,
 * the tokens or the positions, nor a base except as above.  drop: as in the forward call.  Errors as the
 * forward call.
 */
LIONCUB_API int lioncub_embed_backward(lioncub_embed_t h, const lioncub_token_batch* batch, const lioncub_rows* dout,
                                       const lioncub_rows* base, const lioncub_rows* grad,
                                       const lioncub_rows* pos_base, const lioncub_rows* pos_grad,
                                       const lioncub_drop* drop, lioncub_stream_t stream);

/* Checks the guard bands around the workspace and copies the status word to
 * dst_dev (one int32 in device memory) on `stream`. */
LIONCUB_API int lioncub_embed_status(lioncub_embed_t h, int32_t* dst_dev, lioncub_stream_t stream);

/* Message of this thread's last failed call on a handle where that was h, else of
 * h's last failed call in any thread ("" if none); valid until this thread's next
 * failed call or message.  h == NULL: of this thread's last failed create or
 * dropout call. */
LIONCUB_API const char* lioncub_embed_last_error(lioncub_embed_t h);

/* Frees the handle and its workspace (NULL is a no-op); synchronizes. */
LIONCUB_API void lioncub_embed_destroy(lioncub_embed_t h);

/*
 * Dropout over a rows x cols matrix.  forward: out = dropout(x) (+ residual,
 * of out's type, NULL for none).  backward: dx = dropout(dout) with the
 * forward call's seed, stream and p.  The result may be the same matrix as an
 * input of its type, but must not overlap one in any other way.  Errors as
 * lioncub_embed_forward (messages via lioncub_embed_last_error(NULL)).
 */
LIONCUB_API int lioncub_dropout_forward(int64_t rows, int64_t cols, const lioncub_rows* x,
                                        const lioncub_rows* residual, const lioncub_rows* out,
                                        const lioncub_drop* drop, lioncub_stream_t stream);
LIONCUB_API int lioncub_dropout_backward(int64_t rows, int64_t cols, const lioncub_rows* dout, const lioncub_rows* dx,
                                         const lioncub_drop* drop, lioncub_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIONCUB_EMBED_H */
