/*
 * lioncub_block.h -- C ABI of the block operators: what stands between the
 * input layer (lioncub_embed.h) and the matrix products of a transformer block.
 * The root-mean-square norm with the residual's addition and its gradient,
 * activation checkpoints in 8 bits, the activation whose backward pass reads
 * them, and rotary positions.
 *
 * With i a row (a token), j a column, RN a rounding to fp32:
 *   norm       h = RN(x + residual) (x itself without a residual),
 *              rstd_i = 1 / sqrt(mean_j h_ij^2 + eps),  out = h * rstd_i * weight_j
 *   gradient   n = h * rstd_i, g = dout * weight_j,
 *              dx = residual_grad + rstd_i * (g - n * mean_j(g * n)),
 *              weight_grad_j = weight_base_j + sum_i dout * n,  again = n * weight_j
 *   activation out = f(x) (* up), f(x) = x * s(z), s(z) = 1 / (1 + exp(-z)),
 *              z = x (SiLU) or 2 sqrt(2 / pi) (x + 0.044715 x^3) (GELU by the hyperbolic tangent,
 *              since 0.5 (1 + tanh(t)) = s(2 t))
 *   gradient   dx = dout (* up) * f'(x),  dup = dout * f(x),  again = f(x) (* up)
 *   rotary     (a, b) -> m * (a cos - b sin, a sin + b cos) for each pair of columns, angle =
 *              position * frequency of the pair; the gradient is the same with the angle negated
 * Every operation is in fp32 (sums of a row and of a column too), and each
 * result is rounded once to its own type; the norm is that of h before it is
 * rounded to the type of `summed`.  Mean squares must lie within fp32's range.
 * The activation's exponential and quotient are the GPU's approximate ones: f is
 * off by at most 16 (1 + (1 - s) |z|) units of 2^-24 of itself, each term of f' by
 * at most 32, and an s below 2^-126 counts as 0.
 *
 * 8 bits (lioncub_packed): the columns of a row are cut into groups (the last
 * may be shorter) that share an fp32 scale.  With a the largest magnitude of a
 * group and top = 127 (whole numbers) or 448 (e4m3):
 *   inv = RN(top / a),  scale = RN(a * RN(1 / top)),
 *   code = RN(x * inv) rounded to a whole number or to e4m3 (to nearest, ties to even),
 * and a code stands for RN(code * scale).  A group whose a is below 2^-100 is
 * held as zeros (scale 0); one that holds an infinity or a NaN has codes of 0
 * and a NaN as its scale, so that all of it stands for NaN.
 *
 * Calls only enqueue kernels on `stream`: nothing is allocated or synchronized
 * outside create, and a call can be captured into a CUDA graph.  Everything but
 * lioncub_rms_norm_backward may be called by several host threads at once, on
 * one handle too.  That call uses its handle's workspace: calls on one handle
 * must be ordered one after another, on the device (one stream, or events
 * between them; graphs that captured calls on one handle count like calls) and
 * on the host.  Results do not depend on the schedule: sums run in an order that
 * depends on the sizes, on whether all matrices allow 16-byte moves and on the
 * number of the GPU's multiprocessors, so a call repeats bit for bit.
 * Return codes are those of lioncub.h.
 *
 * Matrices are lioncub_rows, as in lioncub_embed.h; rows that start on 16-byte
 * boundaries and whose width is a multiple of 8 are moved 16 bytes at a time, if
 * all matrices of a call allow it and rows of codes start on 8-byte boundaries
 * (read by a norm's gradient: 16, and a width that is a multiple of 16).  Heads
 * want 16-byte boundaries and halves of the rotated columns of 8.  Anything else
 * works element by element, at two to four times the cost.
 * A result may be the same lioncub_rows matrix as an input of its type (the same
 * address and stride), each element then being read before it is written, but for
 * what is read later: weight_base may be weight_grad only, and a forward call's
 * weight not summed.  Results may not share bytes with inputs in any other way,
 * nor with one another.
 */
#ifndef LIONCUB_BLOCK_H
#define LIONCUB_BLOCK_H

#include "lioncub_embed.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct lioncub_rms_norm_s* lioncub_rms_norm_t;
typedef struct lioncub_rotary_s* lioncub_rotary_t;

enum {
    LIONCUB_NORM_MAX_DIM = 16384, /* columns of a norm, or of a row that shares one scale */
    LIONCUB_ROTARY_MAX_DIM = 1024 /* columns of a head                                    */
};

enum { LIONCUB_CODES_INT8 = 0, LIONCUB_CODES_E4M3 = 1 };
enum { LIONCUB_ACTIVATION_SILU = 0, LIONCUB_ACTIVATION_GELU = 1 };
enum { LIONCUB_SCALING_NONE = 0, LIONCUB_SCALING_LINEAR = 1, LIONCUB_SCALING_BASE = 2, LIONCUB_SCALING_PARTS = 3 };

/* A matrix in 8 bits, in device memory: row i's codes start at codes + i *
 * stride, its scales at scales + i * scale_stride. */
typedef struct {
    void* codes;
    float* scales;
    int64_t stride;       /* bytes between rows, >= the row's columns                   */
    int64_t scale_stride; /* elements between rows, >= the row's groups                 */
    int32_t group;        /* columns of a group: 32, 64, 128 or 256; 0: the whole row   */
    int32_t format;       /* LIONCUB_CODES_*                                            */
} lioncub_packed;

/* Heads in device memory: head h of place s of sequence b starts at data + b *
 * batch_stride + s * place_stride + h * head_stride elements; its columns are
 * contiguous.  Inputs may have strides of 0. */
typedef struct {
    void* data;
    int64_t batch_stride, place_stride, head_stride;
    int32_t heads;
    int32_t type; /* LIONCUB_ROWS_* */
} lioncub_heads;

/* Where the places stand: positions[b * seq_len + s], or first_position + s when
 * positions is NULL.  Any number counts, a negative one too. */
typedef struct {
    const void* positions; /* batch * seq_len of them, device, or NULL */
    int64_t batch, seq_len;
    int64_t first_position; /* read only when positions is NULL, |first_position| <= 2^40 */
    int32_t index_type;     /* LIONCUB_INDEX_*, of positions */
    int32_t reserved;
} lioncub_sequences;

/* How frequencies are scaled for contexts longer than those trained on. */
typedef struct {
    double factor;    /* >= 1: the new length over the old one                                */
    double length;    /* PARTS: the old length                                                */
    double low, high; /* PARTS: pairs that turn `high` times or more within `length` keep     */
                      /* their frequency, those that turn `low` times or less have it divided */
                      /* by `factor`, those between are interpolated linearly                 */
    int32_t kind;     /* LIONCUB_SCALING_*: LINEAR divides all frequencies by factor; BASE    */
                      /* raises the base by factor^(rotary_dim / (rotary_dim - 2))            */
    int32_t reserved;
} lioncub_rotary_scaling;

/* ---- the norm ------------------------------------------------------------- */

/*
 * A norm over rows of `dim` columns.  Allocates the gradient's workspace (4 *
 * dim bytes for each multiprocessor) on the current device, which must be
 * current in every later call on the handle, and synchronizes the legacy default
 * stream once.  LIONCUB_FAIL_ALLOC and LIONCUB_FAIL_LAUNCH (lioncub.h) apply to
 * the handle's own allocations and kernel launches, LIONCUB_WAIT_POLLS to the first wait of
 * each of a gradient's teams of warps for the copies that bring it rows.  eps must be positive (a row
 * of zeros then gives zeros).  Errors: ERR_ARG, ERR_OOM, ERR_CUDA (*out is NULL then).
 */
LIONCUB_API int lioncub_rms_norm_create(lioncub_rms_norm_t* out, int64_t dim, float eps);

/*
 * out (n x dim), or its codes in packed_out -- exactly one of the two -- from x
 * and, unless they are NULL: residual, added to x; weight (one row of dim; NULL:
 * ones).  Each of these is written unless it is NULL: summed = x + residual (of
 * any type, without a residual a copy of x); saved, the same in 8 bits, for the
 * backward pass; rstd (n fp32).  One launch.  Errors: ERR_ARG, ERR_ALIGN (a pointer that is not aligned to
 * its element), ERR_STATE (another device is current), ERR_CUDA.
 */
LIONCUB_API int lioncub_rms_norm_forward(lioncub_rms_norm_t h, int64_t n, const lioncub_rows* x,
                                         const lioncub_rows* residual, const lioncub_rows* weight,
                                         const lioncub_rows* summed, const lioncub_packed* saved, float* rstd,
                                         const lioncub_rows* out, const lioncub_packed* packed_out,
                                         lioncub_stream_t stream);

/*
 * The gradients from dout (n x dim), with h = x + residual as the forward call
 * left it, in saved or in packed_saved (exactly one of the two), and its rstd.
 * dx is the gradient of x and of residual; residual_grad (NULL: none) is what
 * reaches their sum by another way.  Unless they are NULL: weight_grad (one row)
 * is written, weight_base (of its type, possibly weight_grad itself) added to
 * it; again receives the normed rows once more, for the weight gradient of the
 * product that read them.  weight as in the forward call.  One launch, two with weight_grad.
 * Errors as the forward call.
 */
LIONCUB_API int lioncub_rms_norm_backward(lioncub_rms_norm_t h, int64_t n, const lioncub_rows* dout,
                                          const lioncub_rows* saved, const lioncub_packed* packed_saved,
                                          const float* rstd, const lioncub_rows* weight,
                                          const lioncub_rows* residual_grad, const lioncub_rows* dx,
                                          const lioncub_rows* weight_base, const lioncub_rows* weight_grad,
                                          const lioncub_rows* again, lioncub_stream_t stream);

/* Checks the guard bands around the workspace and copies the status word
 * (LIONCUB_STATUS_* bits, 0: all is well) to dst_dev (one int32 in device
 * memory) on `stream`. */
LIONCUB_API int lioncub_rms_norm_status(lioncub_rms_norm_t h, int32_t* dst_dev, lioncub_stream_t stream);

/* Frees the handle and its workspace (NULL is a no-op); synchronizes. */
LIONCUB_API void lioncub_rms_norm_destroy(lioncub_rms_norm_t h);

/* ---- 8 bits ------------------------------------------------------------------ */

/* The codes and scales of x (rows x cols).  A whole row shares one scale
 * (group 0) only up to LIONCUB_NORM_MAX_DIM columns.  Errors as the norm's. */
LIONCUB_API int lioncub_pack8(int64_t rows, int64_t cols, const lioncub_rows* x, const lioncub_packed* out,
                              lioncub_stream_t stream);

/* What the codes stand for, in out (rows x cols). */
LIONCUB_API int lioncub_unpack8(int64_t rows, int64_t cols, const lioncub_packed* x, const lioncub_rows* out,
                                lioncub_stream_t stream);

/* ---- the activation ------------------------------------------------------------ */

/*
 * out = f(x) (* up unless it is NULL), rows x cols; x, up and out of one type.
 * saved and saved_up (NULL: not wanted) receive x and up in 8 bits, for the
 * backward pass (groups of columns, not whole rows).  Errors as the norm's.
 */
LIONCUB_API int lioncub_activation_forward(int64_t rows, int64_t cols, int kind, const lioncub_rows* x,
                                           const lioncub_rows* up, const lioncub_rows* out, const lioncub_packed* saved,
                                           const lioncub_packed* saved_up, lioncub_stream_t stream);

/*
 * dx and, with up, dup (NULL: not wanted) from dout; x and up as matrices or as
 * packed_x and packed_up, both the same way.  again (NULL: not wanted) receives
 * the forward call's result once more.  All matrices of one type.
 */
LIONCUB_API int lioncub_activation_backward(int64_t rows, int64_t cols, int kind, const lioncub_rows* dout,
                                            const lioncub_rows* x, const lioncub_rows* up,
                                            const lioncub_packed* packed_x, const lioncub_packed* packed_up,
                                            const lioncub_rows* dx, const lioncub_rows* dup, const lioncub_rows* again,
                                            lioncub_stream_t stream);

/* ---- rotary positions ------------------------------------------------------------- */

/* Host function: frequencies[k] = base^(-2 k / rotary_dim) for the rotary_dim / 2
 * pairs, in radians a position, scaled as scaling says (NULL: not). */
LIONCUB_API int lioncub_rotary_frequencies(int64_t rotary_dim, double base, const lioncub_rotary_scaling* scaling,
                                           double* frequencies);

/*
 * Rotation of the first rotary_dim (even, at least 2) columns of heads of
 * head_dim; the others are copied.  Pair k is columns (k, k + rotary_dim / 2),
 * or (2 k, 2 k + 1) when interleaved.  frequencies: rotary_dim / 2 in [0, 65536),
 * read during the call.  magnitude (finite) multiplies the rotated columns.  Keeps 4 * rotary_dim bytes on
 * the current device, which must be current in later calls.  The angle is reduced
 * exactly, as position * frequency / (2 pi) modulo 1 in 64-bit fixed point: it is
 * off by less than 2^-27 + |position| * (2^-52 * frequency + 2^-64) of a turn.  Errors as lioncub_rms_norm_create.
 */
LIONCUB_API int lioncub_rotary_create(lioncub_rotary_t* out, int64_t head_dim, int64_t rotary_dim,
                                      const double* frequencies, float magnitude, int interleaved);

/*
 * Rotates q into q_out and, unless k is NULL, k into k_out (batch, places and
 * head_dim in common; heads of their own; all of one type), by the angle or, if
 * `inverse`, by its negative.  One launch.  q_out may be q, k_out may be k.  Errors as the norm's.
 */
LIONCUB_API int lioncub_rotary_apply(lioncub_rotary_t h, const lioncub_sequences* places, const lioncub_heads* q,
                                     const lioncub_heads* q_out, const lioncub_heads* k, const lioncub_heads* k_out,
                                     int inverse, lioncub_stream_t stream);

/* Frees the handle (NULL is a no-op); synchronizes. */
LIONCUB_API void lioncub_rotary_destroy(lioncub_rotary_t h);

/* Message of this thread's last failed call of this header ("" if none); valid
 * until its next failed call. */
LIONCUB_API const char* lioncub_block_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* LIONCUB_BLOCK_H */
