// embed.cu -- the C ABI of the input-layer operators (include/lioncub_embed.h):
// argument checks, the handle's workspace, launches and errors.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <new>

#include "embed.h"
#include "guard.h"
#include "operands.h"
#include "splitmix64.cuh"

// Layouts the language bindings rely on.
static_assert(sizeof(lioncub_rows) == 24, "lioncub_rows must stay 24 bytes");
static_assert(sizeof(lioncub_token_batch) == 48, "lioncub_token_batch must stay 48 bytes");
static_assert(sizeof(lioncub_drop) == 24, "lioncub_drop must stay 24 bytes");
static_assert(lc::kStatusIndex == LIONCUB_EMBED_STATUS_INDEX, "status bits are part of the ABI");

namespace {
constexpr int kWords = 4;    // single words of the workspace: the status word, the sorts' totals, `begun`
constexpr int kBuffers = 5;
static_assert(kBuffers + 1 <= lc::kMaxGuardBands, "a band before, between and after the buffers");
}  // namespace

struct lioncub_embed_s {
    int device = 0;
    int64_t vocab = 0, dim = 0, positions = 0, max_tokens = 0;
    float scale = 1.0f;

    // device workspace: one allocation, its buffers between guard bands
    void* memory = nullptr;
    lc::GuardList guards{};
    int* status = nullptr;       // kWords words, the first the status word
    int4* order = nullptr;       // for each table: max_tokens entries of the sort
    int2* segment = nullptr;     // vocab + positions ranges of order
    uint64_t* arrived = nullptr;  // arrival counters of the row sums, for each table
    float* partial = nullptr;    // partial_rows x partial_stride sums of pieces, for each table
    int64_t arrived_count = 0, partial_rows = 0, partial_stride = 0;

    // fault injection (environment, read at create; 0 = off)
    int64_t fail_alloc_at = 0, alloc_count = 0;
    int64_t fail_launch_at = 0;
    std::atomic<int64_t> launch_count{0};

    uint32_t calls = 0;  // gradients, numbered 1, 2, ... (see lc::SortArgs::call)

    uint64_t number = 0;  // of the handles, from 1
    std::mutex err_lock;  // lookups may fail in several threads
    char err[256] = "";
};

namespace {

using lc::aligned_rows;
using lc::element_size;
using lc::env_index;
using lc::NvtxRange;
using lc::overlap;
using lc::rows_of;
using lc::same_matrix;

std::atomic<uint64_t> g_handles{0};

// Messages of this thread's last failed call without a handle, and of that on a
// handle, whose number (not its address, which another may get) goes with it.
thread_local char g_err[256] = "";
thread_local char t_err[256] = "";
thread_local uint64_t t_err_of = 0;

int fail(lioncub_embed_t h, int code, const char* fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(h ? t_err : g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    if (h) {
        t_err_of = h->number;
        std::lock_guard<std::mutex> hold(h->err_lock);
        std::memcpy(h->err, t_err, sizeof t_err);
    }
    return code;
}

int cuda_fail(lioncub_embed_t h, cudaError_t e, const char* what)
{
    return fail(h, LIONCUB_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// The workspace: buffers of these sizes, each on a 256-byte boundary with guard
// bands before and after it.
cudaError_t allocate(lioncub_embed_t h, const size_t (&bytes)[kBuffers], void** const (&to)[kBuffers])
{
    static_assert(lc::kGuardBytes % 256 == 0, "guards keep alignment");
    size_t at[kBuffers], total = 0;
    for (int k = 0; k < kBuffers; ++k) {
        at[k] = total + lc::kGuardBytes;
        total = at[k] + (bytes[k] + 255) / 256 * 256;
    }
    if (++h->alloc_count == h->fail_alloc_at)
        return cudaErrorMemoryAllocation;
    cudaError_t e = cudaMalloc(&h->memory, total + lc::kGuardBytes);
    if (e != cudaSuccess) {
        h->memory = nullptr;
        return e;
    }
    char* base = static_cast<char*>(h->memory);
    for (int k = 0; k <= kBuffers && e == cudaSuccess; ++k) {
        char* band = base + (k < kBuffers ? at[k] - lc::kGuardBytes : total);
        h->guards.band[h->guards.n++] = reinterpret_cast<const uint32_t*>(band);
        e = cudaMemsetAsync(band, static_cast<int>(lc::kGuardByte), lc::kGuardBytes, nullptr);
        if (k < kBuffers)
            *to[k] = base + at[k];
    }
    return e;
}

void release(lioncub_embed_t h)
{
    cudaFree(h->memory);
    delete h;
}

template <typename Launch>
cudaError_t launch(lioncub_embed_t h, const char* name, Launch&& go)
{
    NvtxRange range(name);
    if (++h->launch_count == h->fail_launch_at)
        return cudaErrorLaunchOutOfResources;
    return go();
}

// --- arguments ---------------------------------------------------------------------

int check_rows(lioncub_embed_t h, const char* name, const lioncub_rows* m, int64_t rows, int64_t cols)
{
    if (!m || (!m->data && rows > 0 && cols > 0))
        return fail(h, LIONCUB_ERR_ARG, "%s is NULL", name);
    if (m->type != LIONCUB_ROWS_BF16 && m->type != LIONCUB_ROWS_F32)
        return fail(h, LIONCUB_ERR_ARG, "%s: unknown type %d", name, m->type);
    if (m->stride < cols || m->stride > (int64_t(1) << 40))
        return fail(h, LIONCUB_ERR_ARG, "%s: stride %lld for %lld columns", name, (long long)m->stride, (long long)cols);
    if (reinterpret_cast<uintptr_t>(m->data) % element_size(m->type))
        return fail(h, LIONCUB_ERR_ALIGN, "%s is not aligned to its elements", name);
    return LIONCUB_OK;
}

// NULL, p == 0 and a p that rounds to 0 mean no dropout.
int check_drop(lioncub_embed_t h, const lioncub_drop* d, int64_t cols, lc::DropArgs* out, bool* on)
{
    *out = lc::DropArgs{0, 0, 0, 1.0f};
    *on = false;
    if (!d)
        return LIONCUB_OK;
    if (!(d->p >= 0.0f && d->p <= 1.0f))
        return fail(h, LIONCUB_ERR_ARG, "p must be in [0, 1]");
    const uint32_t T = static_cast<uint32_t>(std::floor(static_cast<double>(d->p) * 65536.0 + 0.5));
    if (T == 0)
        return LIONCUB_OK;
    out->first = lc::splitmix64(d->seed, d->stream) + lc::kSplitMix64Step;
    out->row_step = static_cast<uint64_t>(cols / 4) * lc::kSplitMix64Step;
    out->limit = static_cast<uint32_t>((static_cast<uint64_t>(T) << 16) - 1);
    out->rescale = T == 65536 ? 0.0f : static_cast<float>(65536.0 / (65536.0 - T));
    *on = true;
    return LIONCUB_OK;
}

int check_places(lioncub_embed_t h, const lioncub_token_batch* b, bool positions_used, lc::Places* out)
{
    if (!b || b->n < 0 || b->n > h->max_tokens)
        return fail(h, LIONCUB_ERR_ARG, "a batch of 0..%lld places is needed", (long long)h->max_tokens);
    if (b->n > 0 && !b->tokens)
        return fail(h, LIONCUB_ERR_ARG, "tokens is NULL");
    if (b->index_type != LIONCUB_INDEX_I64 && b->index_type != LIONCUB_INDEX_I32)
        return fail(h, LIONCUB_ERR_ARG, "unknown index type %d", b->index_type);
    const uintptr_t size = b->index_type == LIONCUB_INDEX_I64 ? 8 : 4;
    if (reinterpret_cast<uintptr_t>(b->tokens) % size || reinterpret_cast<uintptr_t>(b->positions) % size)
        return fail(h, LIONCUB_ERR_ALIGN, "tokens or positions are not aligned to their elements");
    if (positions_used && h->positions == 0)
        return fail(h, LIONCUB_ERR_ARG, "the layer has no position rows");
    if (positions_used && !b->positions) {
        if (b->seq_len < 1)
            return fail(h, LIONCUB_ERR_ARG, "seq_len must be 1 or more for running positions (got %lld)", (long long)b->seq_len);
        const int64_t span = b->seq_len < b->n ? b->seq_len : b->n;
        if (b->first_position < 0 || b->first_position > h->positions - span)
            return fail(h, LIONCUB_ERR_ARG, "positions %lld..%lld are outside the table's %lld", (long long)b->first_position,
                        (long long)(b->first_position + span - 1), (long long)h->positions);
    }
    out->tokens = b->tokens;
    out->positions = b->positions;
    out->seq_len = b->seq_len < 1 ? 1 : b->seq_len < INT_MAX ? b->seq_len : INT_MAX;
    out->first = b->first_position;
    out->n = static_cast<int32_t>(b->n);
    out->wide = b->index_type == LIONCUB_INDEX_I64;
    out->vocab = static_cast<int32_t>(h->vocab);
    out->npos = static_cast<int32_t>(h->positions);
    return LIONCUB_OK;
}

// A result must not share bytes with the ids that the call reads: they would change
// under it.
int check_apart(lioncub_embed_t h, const char* name, const lioncub_rows& m, int64_t rows, const lioncub_token_batch& b,
                bool positions_used)
{
    if (rows == 0 || b.n == 0)
        return LIONCUB_OK;
    const uintptr_t m0 = reinterpret_cast<uintptr_t>(m.data), step = m.stride * element_size(m.type);
    const uintptr_t width = h->dim * element_size(m.type), m1 = m0 + (rows - 1) * step + width;
    const uintptr_t bytes = b.n * (b.index_type == LIONCUB_INDEX_I64 ? 8 : 4);
    for (const void* ids : {b.tokens, positions_used ? b.positions : nullptr}) {
        const uintptr_t i0 = reinterpret_cast<uintptr_t>(ids);
        if (!ids || i0 >= m1 || i0 + bytes <= m0)
            continue;
        // begins before a row's end, or reaches the next row
        if (i0 < m0 || (i0 - m0) % step < width || (i0 - m0) % step + bytes > step)
            return fail(h, LIONCUB_ERR_ARG, "%s overlaps the tokens or positions", name);
    }
    return LIONCUB_OK;
}

int check_device(lioncub_embed_t h)
{
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(h, e, "cudaGetDevice");
    if (dev != h->device)
        return fail(h, LIONCUB_ERR_STATE, "device %d is current, the handle belongs to %d", dev, h->device);
    return LIONCUB_OK;
}

uint32_t* begun_word(lioncub_embed_t h) { return reinterpret_cast<uint32_t*>(h->status + kWords - 1); }

// One table's part of a backward call.
struct TableGradient {
    lc::KeyKind kind;
    int64_t rows;
    const lioncub_rows *base, *grad;
    float factor;
};

// Positions that run with the place are summed without a sort while a position
// has few places, since a block at most adds those of a slab.  (Whole gradients of
// 768 columns, microseconds without and with a sort: 128 sequences of 16 19.0 and
// 22.2, of 1024 121 and 149; 1024 of 16 43.1 and 42.8, of 64 80.7 and 87.8, of 256
// 258 and 337; 2048 of 16 80 and 57, of 32 137 and 87.)
constexpr int64_t kRunning = 1024;

lc::SortTask sort_task(lioncub_embed_t h, const lc::Places& at, const TableGradient& g)
{
    lc::SortTask t{};
    const int which = g.kind;
    t.at = at;
    t.kind = which;
    t.keys = static_cast<int32_t>(g.rows);
    t.capacity = static_cast<int32_t>(h->max_tokens);
    t.order = h->order + which * h->max_tokens;
    t.segment = h->segment + which * h->vocab;
    t.total = h->status + 1 + which;
    return t;
}

lc::RowSumArgs row_sum_args(lioncub_embed_t h, const lc::Places& at, const TableGradient& g, const lioncub_rows* dout,
                            const lc::DropArgs& drop)
{
    const lc::SortTask t = sort_task(h, at, g);
    lc::RowSumArgs a{};
    a.dout = rows_of(dout);
    a.base = rows_of(g.base);
    a.grad = rows_of(g.grad);
    a.order = t.order;
    a.segment = t.segment;
    a.total = t.total;
    a.partial = h->partial + g.kind * h->partial_rows * h->partial_stride;
    a.partial_stride = h->partial_stride;
    a.partial_rows = h->partial_rows;
    a.arrived = h->arrived + g.kind * h->arrived_count;
    a.drop = drop;
    a.factor = g.factor;
    a.rows = static_cast<int32_t>(g.rows);
    a.dim = static_cast<int32_t>(h->dim);
    a.n = at.n;
    a.begun = begun_word(h);
    a.call = h->calls;
    a.status = h->status;
    return a;
}

// grad with its optional base: types, strides and overlaps.
int check_gradient(lioncub_embed_t h, const char* name, const lioncub_rows* base, const lioncub_rows* grad, int64_t rows,
                   const lioncub_rows* dout, int64_t n)
{
    int rc = check_rows(h, name, grad, rows, h->dim);
    if (rc == LIONCUB_OK && base)
        rc = check_rows(h, "base", base, rows, h->dim);
    if (rc != LIONCUB_OK)
        return rc;
    if (base && base->type != grad->type)
        return fail(h, LIONCUB_ERR_ARG, "%s and its base must have one type", name);
    if (base && !same_matrix(*base, *grad) && overlap(*base, rows, *grad, rows, h->dim))
        return fail(h, LIONCUB_ERR_ARG, "%s overlaps its base without being it", name);
    if (overlap(*dout, n, *grad, rows, h->dim))
        return fail(h, LIONCUB_ERR_ARG, "%s overlaps dout", name);
    return LIONCUB_OK;
}

int run_dropout(const char* in_name, const char* out_name, int64_t rows, int64_t cols, const lioncub_rows* x,
                const lioncub_rows* residual, const lioncub_rows* out, const lioncub_drop* drop, cudaStream_t s)
{
    NvtxRange range("lioncub_dropout");
    g_err[0] = '\0';
    if (rows < 0 || cols < 0 || rows > INT_MAX || cols > (int64_t(1) << 40) || (rows > 0 && cols > (int64_t(1) << 41) / rows))
        return fail(nullptr, LIONCUB_ERR_ARG, "bad sizes: %lld x %lld", (long long)rows, (long long)cols);
    int rc = check_rows(nullptr, in_name, x, rows, cols);
    if (rc == LIONCUB_OK)
        rc = check_rows(nullptr, out_name, out, rows, cols);
    if (rc == LIONCUB_OK && residual)
        rc = check_rows(nullptr, "residual", residual, rows, cols);
    if (rc != LIONCUB_OK)
        return rc;
    if (residual && residual->type != out->type)
        return fail(nullptr, LIONCUB_ERR_ARG, "residual and %s must have one type", out_name);
    for (const lioncub_rows* m : {x, residual})
        if (m && !same_matrix(*m, *out) && overlap(*m, rows, *out, rows, cols))
            return fail(nullptr, LIONCUB_ERR_ARG, "%s overlaps an input without being it", out_name);
    lc::DropoutArgs a{};
    bool on = false;
    rc = check_drop(nullptr, drop, cols, &a.drop, &on);
    if (rc != LIONCUB_OK)
        return rc;
    a.x = rows_of(x);
    a.residual = rows_of(residual);
    a.out = rows_of(out);
    a.rows = rows;
    a.cols = cols;
    const bool starts = reinterpret_cast<uintptr_t>(x->data) % 16 == 0 && reinterpret_cast<uintptr_t>(out->data) % 16 == 0 &&
                        (!residual || reinterpret_cast<uintptr_t>(residual->data) % 16 == 0);
    const bool dense = x->stride == cols && out->stride == cols && (!residual || residual->stride == cols);
    const bool vec = starts && (dense || (aligned_rows(x) && aligned_rows(out) && aligned_rows(residual)));
    if (!(vec && dense) && cols > int64_t(65535) * 256)
        return fail(nullptr, LIONCUB_ERR_ARG, "rows that are apart or unaligned may have 65535 * 256 columns at most");
    const cudaError_t e = lc::launch_dropout(a, x->type, out->type, vec, on, s);
    return e == cudaSuccess ? LIONCUB_OK : cuda_fail(nullptr, e, "dropout launch");
}

}  // namespace

extern "C" {

const char* lioncub_embed_last_error(lioncub_embed_t h)
{
    if (!h)
        return g_err;
    if (t_err_of != h->number) {
        std::lock_guard<std::mutex> hold(h->err_lock);
        std::memcpy(t_err, h->err, sizeof t_err);
        t_err_of = 0;  // read anew next time
    }
    return t_err;
}

int lioncub_embed_create(lioncub_embed_t* out, int64_t vocab, int64_t dim, int64_t positions, int64_t max_tokens,
                         float scale)
{
    g_err[0] = '\0';
    if (!out)
        return fail(nullptr, LIONCUB_ERR_ARG, "out is NULL");
    *out = nullptr;
    if (vocab < 1 || vocab > LIONCUB_EMBED_MAX_VOCAB || positions < 0 || positions > LIONCUB_EMBED_MAX_VOCAB)
        return fail(nullptr, LIONCUB_ERR_ARG, "tables of 1..%d token rows and 0..%d position rows are supported (got %lld, %lld)",
                    LIONCUB_EMBED_MAX_VOCAB, LIONCUB_EMBED_MAX_VOCAB, (long long)vocab, (long long)positions);
    if (dim < 1 || dim > LIONCUB_EMBED_MAX_DIM)
        return fail(nullptr, LIONCUB_ERR_ARG, "dim must be 1..%d (got %lld)", LIONCUB_EMBED_MAX_DIM, (long long)dim);
    if (max_tokens < 0 || max_tokens > LIONCUB_EMBED_MAX_TOKENS)
        return fail(nullptr, LIONCUB_ERR_ARG, "max_tokens must be 0..%d (got %lld)", LIONCUB_EMBED_MAX_TOKENS,
                    (long long)max_tokens);
    if (!std::isfinite(scale))
        return fail(nullptr, LIONCUB_ERR_ARG, "scale must be finite");
    lioncub_embed_t h = new (std::nothrow) lioncub_embed_s();
    if (!h)
        return fail(nullptr, LIONCUB_ERR_OOM, "no host memory for the handle");
    h->number = ++g_handles;
    h->vocab = vocab;
    h->dim = dim;
    h->positions = positions;
    h->max_tokens = max_tokens;
    h->scale = scale;
    const int64_t tables = positions > 0 ? 2 : 1;
    const int64_t slabs = lc::slabs_of(dim, false);  // the most: rows that allow 16-byte moves have fewer
    const int64_t stretches = lc::grad_max_stretches(max_tokens, lc::slabs_of(dim, true));
    h->partial_rows = lc::grad_partial_rows(stretches);
    h->partial_stride = slabs * 256;
    h->arrived_count = h->partial_rows * slabs;
    h->fail_alloc_at = env_index("LIONCUB_FAIL_ALLOC");
    h->fail_launch_at = env_index("LIONCUB_FAIL_LAUNCH");
    cudaError_t e = cudaGetDevice(&h->device);
    if (e == cudaSuccess)
        e = allocate(h, {kWords * sizeof(int), tables * max_tokens * sizeof(int4), (vocab + positions) * sizeof(int2),
                         tables * h->arrived_count * sizeof(uint64_t),
                         tables * h->partial_rows * h->partial_stride * sizeof(float)},
                     {reinterpret_cast<void**>(&h->status), reinterpret_cast<void**>(&h->order),
                      reinterpret_cast<void**>(&h->segment), reinterpret_cast<void**>(&h->arrived),
                      reinterpret_cast<void**>(&h->partial)});
    if (e == cudaSuccess)
        e = cudaMemsetAsync(h->status, 0, kWords * sizeof(int), nullptr);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        release(h);
        cudaGetLastError();  // a failed allocation leaves a non-sticky error behind
        return e == cudaErrorMemoryAllocation ? fail(nullptr, LIONCUB_ERR_OOM, "no device memory for the workspace")
                                              : cuda_fail(nullptr, e, "create");
    }
    *out = h;
    return LIONCUB_OK;
}

int lioncub_embed_forward(lioncub_embed_t h, const lioncub_token_batch* batch, const lioncub_rows* table,
                          const lioncub_rows* pos_table, const lioncub_rows* out, const lioncub_drop* drop,
                          lioncub_stream_t stream)
{
    if (!h)
        return LIONCUB_ERR_ARG;
    NvtxRange range("lioncub_embed_forward");
    lc::LookupArgs a{};
    int rc = check_places(h, batch, pos_table != nullptr, &a.at);
    if (rc == LIONCUB_OK)
        rc = check_rows(h, "table", table, h->vocab, h->dim);
    if (rc == LIONCUB_OK && pos_table)
        rc = check_rows(h, "pos_table", pos_table, h->positions, h->dim);
    if (rc == LIONCUB_OK)
        rc = check_rows(h, "out", out, batch->n, h->dim);
    if (rc != LIONCUB_OK)
        return rc;
    if (pos_table && pos_table->type != table->type)
        return fail(h, LIONCUB_ERR_ARG, "table and pos_table must have one type");
    if (overlap(*out, batch->n, *table, h->vocab, h->dim) ||
        (pos_table && overlap(*out, batch->n, *pos_table, h->positions, h->dim)))
        return fail(h, LIONCUB_ERR_ARG, "out overlaps a table");
    rc = check_apart(h, "out", *out, batch->n, *batch, pos_table != nullptr);
    bool on = false;
    if (rc == LIONCUB_OK)
        rc = check_drop(h, drop, h->dim, &a.drop, &on);
    if (rc == LIONCUB_OK)
        rc = check_device(h);
    if (rc != LIONCUB_OK)
        return rc;
    a.table = rows_of(table);
    a.pos_table = rows_of(pos_table);
    a.out = rows_of(out);
    a.scale = h->scale;
    a.dim = static_cast<int32_t>(h->dim);
    a.status = h->status;
    const bool vec = h->dim % 8 == 0 && aligned_rows(table) && aligned_rows(pos_table) && aligned_rows(out);
    const cudaError_t e =
        launch(h, "embed_lookup", [&] { return lc::launch_lookup(a, table->type, out->type, vec, on, stream); });
    return e == cudaSuccess ? LIONCUB_OK : cuda_fail(h, e, "lookup launch");
}

int lioncub_embed_backward(lioncub_embed_t h, const lioncub_token_batch* batch, const lioncub_rows* dout,
                           const lioncub_rows* base, const lioncub_rows* grad, const lioncub_rows* pos_base,
                           const lioncub_rows* pos_grad, const lioncub_drop* drop, lioncub_stream_t stream)
{
    if (!h)
        return LIONCUB_ERR_ARG;
    NvtxRange range("lioncub_embed_backward");
    lc::Places at{};
    int rc = check_places(h, batch, pos_grad != nullptr, &at);
    if (rc == LIONCUB_OK)
        rc = check_rows(h, "dout", dout, batch->n, h->dim);
    if (rc == LIONCUB_OK)
        rc = check_gradient(h, "grad", base, grad, h->vocab, dout, batch->n);
    if (rc == LIONCUB_OK && pos_base && !pos_grad)
        rc = fail(h, LIONCUB_ERR_ARG, "pos_base without pos_grad");
    if (rc == LIONCUB_OK && pos_grad)
        rc = check_gradient(h, "pos_grad", pos_base, pos_grad, h->positions, dout, batch->n);
    if (rc != LIONCUB_OK)
        return rc;
    if (pos_grad && pos_grad->type != grad->type)
        return fail(h, LIONCUB_ERR_ARG, "grad and pos_grad must have one type");
    if (pos_grad && overlap(*grad, h->vocab, *pos_grad, h->positions, h->dim))
        return fail(h, LIONCUB_ERR_ARG, "grad and pos_grad overlap");
    if ((pos_grad && base && overlap(*base, h->vocab, *pos_grad, h->positions, h->dim)) ||
        (pos_base && overlap(*pos_base, h->positions, *grad, h->vocab, h->dim)))
        return fail(h, LIONCUB_ERR_ARG, "a gradient overlaps the other's base");
    rc = check_apart(h, "grad", *grad, h->vocab, *batch, pos_grad != nullptr);
    if (rc == LIONCUB_OK && pos_grad)
        rc = check_apart(h, "pos_grad", *pos_grad, h->positions, *batch, true);
    lc::DropArgs d;
    bool on = false;
    if (rc == LIONCUB_OK)
        rc = check_drop(h, drop, h->dim, &d, &on);
    if (rc == LIONCUB_OK)
        rc = check_device(h);
    if (rc != LIONCUB_OK)
        return rc;

    TableGradient token = {lc::kKeyToken, h->vocab, base, grad, h->scale * d.rescale};
    TableGradient position = {lc::kKeyPosition, h->positions, pos_base, pos_grad, d.rescale};
    const bool running = pos_grad && !at.positions && (at.n + at.seq_len - 1) / at.seq_len <= kRunning;
    const bool sorted_positions = pos_grad && !running;

    lc::SortArgs so{};
    so.task[so.tasks++] = sort_task(h, at, token);
    if (sorted_positions)
        so.task[so.tasks++] = sort_task(h, at, position);
    const bool vec = h->dim % 8 == 0 && aligned_rows(dout) && aligned_rows(base) && aligned_rows(grad) &&
                     aligned_rows(pos_base) && aligned_rows(pos_grad);
    const int64_t slabs = lc::slabs_of(h->dim, vec);
    so.arrived[0] = h->arrived;
    so.arrived[1] = sorted_positions ? h->arrived + h->arrived_count : h->arrived;
    so.arrived_count = lc::grad_partial_rows(lc::grad_stretches(at.n, lc::grad_piece(at.n, slabs))) * slabs;
    so.status = h->status;
    so.begun = begun_word(h);
    h->calls = h->calls == UINT32_MAX ? 1 : h->calls + 1;
    so.call = h->calls;  // its own: a call whose row sums failed leaves its number in the word
    cudaError_t e = launch(h, "embed_sort", [&] { return lc::launch_sort(so, stream); });
    if (e != cudaSuccess)
        return cuda_fail(h, e, "sort launch");

    const lc::RowSumArgs t = row_sum_args(h, at, token, dout, d), p = row_sum_args(h, at, position, dout, d);
    const lc::PositionKind kind = !pos_grad ? lc::kNoPositions : running ? lc::kRunningPositions : lc::kSortedPositions;
    e = launch(h, "embed_row_sums", [&] {
        return lc::launch_row_sums(t, pos_grad ? &p : nullptr, kind, at, dout->type, grad->type, vec, on, stream);
    });
    return e == cudaSuccess ? LIONCUB_OK : cuda_fail(h, e, "row sum launch");
}

int lioncub_embed_status(lioncub_embed_t h, int32_t* dst_dev, lioncub_stream_t stream)
{
    if (!h)
        return LIONCUB_ERR_ARG;
    if (!dst_dev)
        return fail(h, LIONCUB_ERR_ARG, "dst_dev is NULL");
    int rc = check_device(h);
    if (rc != LIONCUB_OK)
        return rc;
    cudaError_t e = lc::launch_guard_check(h->guards, h->status, stream);
    if (e == cudaSuccess)
        e = cudaMemcpyAsync(dst_dev, h->status, sizeof(int32_t), cudaMemcpyDeviceToDevice, stream);
    return e == cudaSuccess ? LIONCUB_OK : cuda_fail(h, e, "status");
}

void lioncub_embed_destroy(lioncub_embed_t h)
{
    if (h)
        release(h);
}

int lioncub_dropout_forward(int64_t rows, int64_t cols, const lioncub_rows* x, const lioncub_rows* residual,
                            const lioncub_rows* out, const lioncub_drop* drop, lioncub_stream_t stream)
{
    return run_dropout("x", "out", rows, cols, x, residual, out, drop, stream);
}

int lioncub_dropout_backward(int64_t rows, int64_t cols, const lioncub_rows* dout, const lioncub_rows* dx,
                             const lioncub_drop* drop, lioncub_stream_t stream)
{
    return run_dropout("dout", "dx", rows, cols, dout, nullptr, dx, drop, stream);
}

}  // extern "C"
