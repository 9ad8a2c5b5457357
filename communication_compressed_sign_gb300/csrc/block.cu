// block.cu -- the C ABI of the block operators (include/lioncub_block.h):
// argument checks, handles, launches and errors.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>

#include "block.h"
#include "guard.h"
#include "operands.h"

// Layouts the language bindings rely on.
static_assert(sizeof(lioncub_packed) == 40, "lioncub_packed must stay 40 bytes");
static_assert(sizeof(lioncub_heads) == 40, "lioncub_heads must stay 40 bytes");
static_assert(sizeof(lioncub_sequences) == 40, "lioncub_sequences must stay 40 bytes");
static_assert(sizeof(lioncub_rotary_scaling) == 40, "lioncub_rotary_scaling must stay 40 bytes");

struct lioncub_rms_norm_s {
    int device = 0;
    int64_t dim = 0;
    float eps = 0.0f;
    int multiprocessors = 0;

    // device workspace: one allocation, its buffers between guard bands
    void* memory = nullptr;
    lc::GuardList guards{};
    int* status = nullptr;
    float* partial = nullptr;  // a row of dim for each multiprocessor

    // fault injection (environment, read at create; 0 = off)
    int64_t fail_launch_at = 0;
    std::atomic<int64_t> launch_count{0};
    uint32_t first_wait_polls = 0;
};

struct lioncub_rotary_s {
    int device = 0;
    int64_t head_dim = 0, rotary_dim = 0;
    float magnitude = 1.0f;
    bool interleaved = false;
    uint64_t* turns = nullptr;  // rotary_dim / 2
    int64_t fail_launch_at = 0;
    std::atomic<int64_t> launch_count{0};
};

namespace {

using lc::aligned_rows;
using lc::element_size;
using lc::NvtxRange;
using lc::Span;

thread_local char t_error[256] = "";

int fail(int code, const char* fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(t_error, sizeof t_error, fmt, ap);
    va_end(ap);
    return code;
}

int cuda_fail(cudaError_t e, const char* what)
{
    return fail(LIONCUB_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

template <typename Handle, typename Launch>
cudaError_t launch(Handle* h, const char* name, Launch&& go)
{
    NvtxRange range(name);
    if (++h->launch_count == h->fail_launch_at)
        return cudaErrorLaunchOutOfResources;
    return go();
}

template <typename Handle>
int check_device(Handle* h)
{
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaGetDevice");
    if (dev != h->device)
        return fail(LIONCUB_ERR_STATE, "device %d is current, the handle belongs to %d", dev, h->device);
    return LIONCUB_OK;
}

// --- matrices -------------------------------------------------------------------------

constexpr int64_t kMaxStride = int64_t(1) << 40;

int check_size(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 0 || rows > INT_MAX || cols > (int64_t(1) << 38) || (rows > 0 && cols > (int64_t(1) << 41) / rows))
        return fail(LIONCUB_ERR_ARG, "bad sizes: %lld x %lld", (long long)rows, (long long)cols);
    return LIONCUB_OK;
}

// The operands of a call: each is checked as it is added, and in the end the
// results must share no bytes with one another, nor with an input unless both are one
// matrix of elements (neither codes, scales nor a vector) and it has been read by then.  `step` counts the parts of a call that follow one
// another over all its rows: an input's is that of its last reading, a result's that of its writing.
class Operands {
public:
    int code = LIONCUB_OK;  // of the first refusal
    bool vec = true;        // all allow 16-byte moves (but for the width)
    bool dense = true;      // rows follow one another, groups do not cross them

    void input(const char* name, const lioncub_rows* m, int64_t rows, int64_t cols, int step = 0) { add(name, m, rows, cols, false, step); }
    void result(const char* name, const lioncub_rows* m, int64_t rows, int64_t cols, int step = 0) { add(name, m, rows, cols, true, step); }
    void input(const char* name, const lioncub_packed* m, int64_t rows, int64_t cols) { add(name, m, rows, cols, false); }
    void result(const char* name, const lioncub_packed* m, int64_t rows, int64_t cols) { add(name, m, rows, cols, true); }
    void vector(const char* name, const float* v, int64_t n, bool is_result)
    {
        if (code != LIONCUB_OK || !v)
            return;
        if (reinterpret_cast<uintptr_t>(v) % sizeof(float))
            code = fail(LIONCUB_ERR_ALIGN, "%s is not aligned to its elements", name);
        else
            keep(name, {reinterpret_cast<uintptr_t>(v), n * sizeof(float), n * sizeof(float), n ? 1 : 0}, is_result);
    }
    int finish()
    {
        for (int i = 0; i < count_ && code == LIONCUB_OK; ++i)
            for (int j = 0; j < count_ && code == LIONCUB_OK; ++j) {
                const Item &a = items_[i], &b = items_[j];
                if (i == j || !a.result || (b.result && j < i) || !lc::overlap(a.span, b.span))
                    continue;
                const bool same = a.matrix && b.matrix && a.span.at == b.span.at && a.span.step == b.span.step &&
                                  a.span.width == b.span.width && a.span.rows == b.span.rows && b.step <= a.step;
                if (b.result || !same)
                    code = fail(LIONCUB_ERR_ARG, b.result ? "%s overlaps %s" : "%s overlaps %s without being it", a.name, b.name);
            }
        return code;
    }

private:
    struct Item {
        const char* name;
        Span span;
        bool result, matrix;
        int step;
    };
    Item items_[16];
    int count_ = 0;

    void keep(const char* name, const Span& span, bool is_result, bool is_matrix = false, int step = 0)
    {
        items_[count_++] = {name, span, is_result, is_matrix, step};
    }

    void add(const char* name, const lioncub_rows* m, int64_t rows, int64_t cols, bool is_result, int step)
    {
        if (code != LIONCUB_OK || !m)
            return;
        if (!m->data && rows > 0 && cols > 0)
            code = fail(LIONCUB_ERR_ARG, "%s is NULL", name);
        else if (m->type != LIONCUB_ROWS_BF16 && m->type != LIONCUB_ROWS_F32)
            code = fail(LIONCUB_ERR_ARG, "%s: unknown type %d", name, m->type);
        else if (m->stride < cols || m->stride > kMaxStride || (rows > 1 && m->stride > (int64_t(1) << 46) / rows))
            code = fail(LIONCUB_ERR_ARG, "%s: stride %lld for %lld columns", name, (long long)m->stride, (long long)cols);
        else if (reinterpret_cast<uintptr_t>(m->data) % element_size(m->type))
            code = fail(LIONCUB_ERR_ALIGN, "%s is not aligned to its elements", name);
        if (code != LIONCUB_OK)
            return;
        const bool starts = reinterpret_cast<uintptr_t>(m->data) % 16 == 0;
        vec = vec && (rows == 1 || m->stride == cols ? starts : aligned_rows(m));
        dense = dense && (rows == 1 || m->stride == cols);
        keep(name, lc::span_of(*m, rows, cols), is_result, true, step);
    }

    void add(const char* name, const lioncub_packed* m, int64_t rows, int64_t cols, bool is_result)
    {
        if (code != LIONCUB_OK || !m)
            return;
        const bool known = m->group == 0 || m->group == 32 || m->group == 64 || m->group == 128 || m->group == 256;
        const int64_t groups = m->group && known ? (cols + m->group - 1) / m->group : 1;
        if ((!m->codes && rows > 0 && cols > 0) || (!m->scales && rows > 0))
            code = fail(LIONCUB_ERR_ARG, "%s is NULL", name);
        else if (m->format != LIONCUB_CODES_INT8 && m->format != LIONCUB_CODES_E4M3)
            code = fail(LIONCUB_ERR_ARG, "%s: unknown format %d", name, m->format);
        else if (!known)
            code = fail(LIONCUB_ERR_ARG, "%s: a group has 32, 64, 128 or 256 columns, or 0: the whole row (got %d)", name, m->group);
        else if (m->stride < cols || m->stride > kMaxStride || (rows > 1 && m->stride > (int64_t(1) << 46) / rows))
            code = fail(LIONCUB_ERR_ARG, "%s: stride %lld for %lld columns", name, (long long)m->stride, (long long)cols);
        else if (m->scale_stride < groups || m->scale_stride > kMaxStride || (rows > 1 && m->scale_stride > (int64_t(1) << 44) / rows))
            code = fail(LIONCUB_ERR_ARG, "%s: stride %lld for %lld scales", name, (long long)m->scale_stride, (long long)groups);
        else if (reinterpret_cast<uintptr_t>(m->scales) % sizeof(float))
            code = fail(LIONCUB_ERR_ALIGN, "%s: scales are not aligned to their elements", name);
        if (code != LIONCUB_OK)
            return;
        const bool starts = reinterpret_cast<uintptr_t>(m->codes) % 8 == 0;  // 8 codes beside 16 bytes of bf16
        vec = vec && starts && (rows == 1 || m->stride == cols || m->stride % 8 == 0);
        dense = dense && (rows == 1 || (m->stride == cols && m->group && cols % m->group == 0 && m->scale_stride == groups));
        keep(name, {reinterpret_cast<uintptr_t>(m->codes), static_cast<uintptr_t>(m->stride), static_cast<uintptr_t>(cols), rows}, is_result);
        keep(name, {reinterpret_cast<uintptr_t>(m->scales), m->scale_stride * sizeof(float), groups * sizeof(float), rows}, is_result);
    }
};

// As many rows of matrices as a checked build's kernels may touch: fewer than there are by
// LIONCUB_CHECKED_ROWS, to see that the checks find what lies beyond.
[[maybe_unused]] int64_t checked_rows(int64_t rows)
{
    const int64_t most = lc::env_index("LIONCUB_CHECKED_ROWS");
    return most ? std::min(most, rows) : rows;
}

lc::TypedRows typed(const lioncub_rows* m, [[maybe_unused]] int64_t rows, [[maybe_unused]] int64_t cols)
{
    lc::TypedRows t = {};
    t.type = LIONCUB_ROWS_BF16;
    if (!m)
        return t;
    t.data = m->data;
    t.stride = m->stride;
    t.type = m->type;
#ifdef LIONCUB_BOUNDS_CHECK
    t.rows = checked_rows(rows);
    t.cols = cols;
#endif
    return t;
}

lc::PackedRows packed(const lioncub_packed* m, [[maybe_unused]] int64_t rows, int64_t cols)
{
    if (!m)
        return lc::PackedRows{};
    int log_group = lc::kRowGroup;
    for (int k = 5; k <= 8; ++k)
        if (m->group == 1 << k)
            log_group = k;
    lc::PackedRows p = {static_cast<uint8_t*>(m->codes), m->scales, m->stride, m->scale_stride, cols, log_group, m->format == LIONCUB_CODES_E4M3, 1.0f};
#ifdef LIONCUB_BOUNDS_CHECK
    p.rows = checked_rows(rows);
#endif
    return p;
}

// Matrices whose rows follow one another are one long row to the kernels that
// work element by element.  Returns whether 8 elements may be moved at a time.
bool as_one_row(const Operands& o, int64_t& rows, int64_t& cols)
{
    if (o.dense && rows > 1) {
        cols *= rows;
        rows = 1;
    }
    return o.vec && cols % 8 == 0 && (rows == 1 || !o.dense);
}

int check_kind(int kind)
{
    if (kind != LIONCUB_ACTIVATION_SILU && kind != LIONCUB_ACTIVATION_GELU)
        return fail(LIONCUB_ERR_ARG, "unknown activation %d", kind);
    return LIONCUB_OK;
}

int check_type(const char* name, const lioncub_rows* m, const lioncub_rows* like)
{
    if (m && m->type != like->type)
        return fail(LIONCUB_ERR_ARG, "%s: the matrices must be of one type", name);
    return LIONCUB_OK;
}

int finish_launch(cudaError_t e, const char* what) { return e == cudaSuccess ? LIONCUB_OK : cuda_fail(e, what); }

// --- heads ---------------------------------------------------------------------------------

// The places of heads in bytes: rows of `width` at at + b * step[0] + s * step[1] + h * step[2].
struct Box {
    uintptr_t at, width;
    int64_t step[3], count[3];  // a dimension of one has step 0
};

Box box_of(const lioncub_heads& m, const lioncub_sequences& p, int64_t head_dim)
{
    const int64_t size = static_cast<int64_t>(element_size(m.type));
    Box b{reinterpret_cast<uintptr_t>(m.data), static_cast<uintptr_t>(head_dim * size), {}, {p.batch, p.seq_len, m.heads}};
    const int64_t step[3] = {m.batch_stride, m.place_stride, m.head_stride};
    for (int k = 0; k < 3; ++k)
        b.step[k] = b.count[k] > 1 ? step[k] * size : 0;
    return b;
}

bool empty(const Box& b) { return b.count[0] == 0 || b.count[1] == 0 || b.count[2] == 0; }

// Bytes from the first to behind the last, over the dimensions order[from], ...
uintptr_t extent(const Box& b, const int (&order)[3], int from)
{
    uintptr_t n = b.width;
    for (int k = from; k < 3; ++k)
        n += (b.count[order[k]] - 1) * b.step[order[k]];
    return n;
}

constexpr int kAnyOrder[3] = {0, 1, 2};

// The dimensions by falling step, of two boxes where both have one or one has none.
void by_step(const Box& a, const Box& b, int (&order)[3])
{
    std::copy(kAnyOrder, kAnyOrder + 3, order);
    std::sort(order, order + 3, [&](int i, int j) { return std::max(a.step[i], b.step[i]) > std::max(a.step[j], b.step[j]); });
}

// Whether no two rows of a box share bytes, taken in this order: each step
// passes over all that lies within.
bool apart(const Box& b, const int (&order)[3])
{
    for (int k = 0; k < 3; ++k)
        if (b.count[order[k]] > 1 && static_cast<uintptr_t>(b.step[order[k]]) < extent(b, order, k + 1))
            return false;
    return true;
}

// Whether some difference of the indexes of two boxes from the k-th dimension on
// bridges `ahead`, the second's start behind the first's.
bool meet(const Box& a, const Box& b, const int (&order)[3], int k, int64_t ahead)
{
    if (k == 3)
        return ahead < static_cast<int64_t>(a.width) && -ahead < static_cast<int64_t>(b.width);
    const int at = order[k];
    const int64_t step = std::max(a.step[at], b.step[at]);
    if (step == 0)
        return meet(a, b, order, k + 1, ahead);
    const int64_t low = ahead >= 0 ? ahead / step : -((-ahead + step - 1) / step);
    for (int64_t d = low; d <= low + 1; ++d)  // index of a - index of b; any other leaves more than what lies within
        if (d < a.count[at] && -d < b.count[at] && meet(a, b, order, k + 1, ahead - d * step))
            return true;
    return false;
}

bool overlap(const Box& a, const Box& b)
{
    if (empty(a) || empty(b))
        return false;
    if (a.at >= b.at + extent(b, kAnyOrder, 0) || b.at >= a.at + extent(a, kAnyOrder, 0))
        return false;
    for (int k = 0; k < 3; ++k)
        if (a.count[k] > 1 && b.count[k] > 1 && a.step[k] != b.step[k])
            return true;  // other steps: taken to meet
    int order[3];
    by_step(a, b, order);
    for (int k = 0; k < 3; ++k) {  // a step must pass over all that lies within, of either
        const uintptr_t step = std::max(a.step[order[k]], b.step[order[k]]);
        if (step && (step < extent(a, order, k + 1) || step < extent(b, order, k + 1)))
            return true;
    }
    return meet(a, b, order, 0, static_cast<int64_t>(b.at) - static_cast<int64_t>(a.at));
}

// reach: the bits of all addresses and strides in bytes, of which the lowest tells the alignment.
int check_heads(const char* name, const lioncub_heads* m, const lioncub_sequences& p, int64_t head_dim, bool is_result, uintptr_t* reach)
{
    if (m->heads < 0 || m->heads > 1 << 20)
        return fail(LIONCUB_ERR_ARG, "%s: %d heads", name, m->heads);
    if (m->type != LIONCUB_ROWS_BF16 && m->type != LIONCUB_ROWS_F32)
        return fail(LIONCUB_ERR_ARG, "%s: unknown type %d", name, m->type);
    const bool none = p.batch == 0 || p.seq_len == 0 || m->heads == 0;
    if (!none && !m->data)
        return fail(LIONCUB_ERR_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(m->data) % element_size(m->type))
        return fail(LIONCUB_ERR_ALIGN, "%s is not aligned to its elements", name);
    const int64_t stride[3] = {m->batch_stride, m->place_stride, m->head_stride}, count[3] = {p.batch, p.seq_len, m->heads};
    *reach |= reinterpret_cast<uintptr_t>(m->data);
    for (int k = 0; k < 3; ++k) {
        if (count[k] <= 1)
            continue;
        if (stride[k] < 0 || stride[k] > kMaxStride || stride[k] > (int64_t(1) << 46) / count[k])
            return fail(LIONCUB_ERR_ARG, "%s: stride %lld", name, (long long)stride[k]);
        *reach |= stride[k] * element_size(m->type);
    }
    if (is_result && !none) {
        const Box b = box_of(*m, p, head_dim);
        int order[3];
        by_step(b, b, order);
        if (!apart(b, order))
            return fail(LIONCUB_ERR_ARG, "%s: its heads share memory", name);
    }
    return LIONCUB_OK;
}

bool same_heads(const lioncub_heads& a, const lioncub_heads& b, const lioncub_sequences& p)
{
    return a.data == b.data && (p.batch <= 1 || a.batch_stride == b.batch_stride) &&
           (p.seq_len <= 1 || a.place_stride == b.place_stride) && (a.heads <= 1 || a.head_stride == b.head_stride);
}

// The range of the positions, which a result must not share.
int check_positions(const char* name, const lioncub_heads& m, const lioncub_sequences& p, int64_t head_dim)
{
    if (!p.positions)
        return LIONCUB_OK;
    const int64_t n = p.batch * p.seq_len;
    const Box b = box_of(m, p, head_dim);
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.positions), bytes = n * (p.index_type == LIONCUB_INDEX_I64 ? 8 : 4);
    if (!empty(b) && at < b.at + extent(b, kAnyOrder, 0) && b.at < at + bytes)
        return fail(LIONCUB_ERR_ARG, "%s may overlap the positions", name);
    return LIONCUB_OK;
}

lc::HeadsArgs heads_of(const lioncub_heads& in, const lioncub_heads& out, [[maybe_unused]] const lioncub_sequences& p,
                       [[maybe_unused]] int64_t head_dim)
{
    lc::HeadsArgs a = {in.data, out.data, in.batch_stride, in.place_stride, in.head_stride, out.batch_stride, out.place_stride, out.head_stride};
#ifdef LIONCUB_BOUNDS_CHECK
    lioncub_sequences some = p;
    some.seq_len = checked_rows(p.seq_len);
    a.in_end = static_cast<const char*>(in.data) + extent(box_of(in, some, head_dim), kAnyOrder, 0);
    a.out_end = static_cast<const char*>(out.data) + extent(box_of(out, some, head_dim), kAnyOrder, 0);
#endif
    return a;
}

}  // namespace

extern "C" {

const char* lioncub_block_last_error(void) { return t_error; }

#ifdef LIONCUB_BOUNDS_CHECK
// Only in checked builds: what the kernels recorded since the last call; synchronizes.
LIONCUB_API int lioncub_block_checked_word(int32_t* word)
{
    *word = 0;
    for (const auto take : {lc::take_norm_word, lc::take_norm_grad_word, lc::take_activation_word, lc::take_rotary_word}) {
        int one = 0;
        const cudaError_t e = take(&one);
        if (e != cudaSuccess)
            return cuda_fail(e, "checked word");
        *word |= one;
    }
    return LIONCUB_OK;
}
#endif

// ---- the norm ---------------------------------------------------------------------------

int lioncub_rms_norm_create(lioncub_rms_norm_t* out, int64_t dim, float eps)
{
    t_error[0] = '\0';
    if (!out)
        return fail(LIONCUB_ERR_ARG, "out is NULL");
    *out = nullptr;
    if (dim < 1 || dim > LIONCUB_NORM_MAX_DIM)
        return fail(LIONCUB_ERR_ARG, "dim must be 1..%d (got %lld)", LIONCUB_NORM_MAX_DIM, (long long)dim);
    if (!(eps > 0.0f) || !std::isfinite(eps))
        return fail(LIONCUB_ERR_ARG, "eps must be positive and finite");
    lioncub_rms_norm_t h = new (std::nothrow) lioncub_rms_norm_s();
    if (!h)
        return fail(LIONCUB_ERR_OOM, "no host memory for the handle");
    h->dim = dim;
    h->eps = eps;
    h->fail_launch_at = lc::env_index("LIONCUB_FAIL_LAUNCH");
    h->first_wait_polls = static_cast<uint32_t>(std::min<int64_t>(lc::env_index("LIONCUB_WAIT_POLLS"), 1 << 20));
    cudaError_t e = cudaGetDevice(&h->device);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&h->multiprocessors, cudaDevAttrMultiProcessorCount, h->device);
    // the status word and the partial sums, each between guard bands
    const size_t sums = (static_cast<size_t>(h->multiprocessors) * dim * sizeof(float) + 255) / 256 * 256;
    const size_t at[2] = {lc::kGuardBytes, 2 * lc::kGuardBytes + 256}, total = at[1] + sums;
    if (e == cudaSuccess)
        e = lc::env_index("LIONCUB_FAIL_ALLOC") == 1 ? cudaErrorMemoryAllocation : cudaMalloc(&h->memory, total + lc::kGuardBytes);
    if (e != cudaSuccess)
        h->memory = nullptr;
    char* base = static_cast<char*>(h->memory);
    for (size_t band : {at[0] - lc::kGuardBytes, at[1] - lc::kGuardBytes, total})
        if (e == cudaSuccess) {
            h->guards.band[h->guards.n++] = reinterpret_cast<const uint32_t*>(base + band);
            e = cudaMemsetAsync(base + band, static_cast<int>(lc::kGuardByte), lc::kGuardBytes, nullptr);
        }
    if (e == cudaSuccess) {
        h->status = reinterpret_cast<int*>(base + at[0]);
        h->partial = reinterpret_cast<float*>(base + at[1]);
        e = cudaMemsetAsync(h->status, 0, sizeof(int), nullptr);
    }
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        lioncub_rms_norm_destroy(h);
        cudaGetLastError();  // a failed allocation leaves a non-sticky error behind
        return e == cudaErrorMemoryAllocation ? fail(LIONCUB_ERR_OOM, "no device memory for the workspace") : cuda_fail(e, "create");
    }
    *out = h;
    return LIONCUB_OK;
}

void lioncub_rms_norm_destroy(lioncub_rms_norm_t h)
{
    if (!h)
        return;
    cudaFree(h->memory);
    delete h;
}

int lioncub_rms_norm_status(lioncub_rms_norm_t h, int32_t* dst_dev, lioncub_stream_t stream)
{
    if (!h)
        return fail(LIONCUB_ERR_ARG, "the handle is NULL");
    if (!dst_dev)
        return fail(LIONCUB_ERR_ARG, "dst_dev is NULL");
    const int rc = check_device(h);
    if (rc != LIONCUB_OK)
        return rc;
    cudaError_t e = lc::launch_guard_check(h->guards, h->status, stream);
    if (e == cudaSuccess)
        e = cudaMemcpyAsync(dst_dev, h->status, sizeof(int32_t), cudaMemcpyDeviceToDevice, stream);
    return finish_launch(e, "status");
}

int lioncub_rms_norm_forward(lioncub_rms_norm_t h, int64_t n, const lioncub_rows* x, const lioncub_rows* residual,
                             const lioncub_rows* weight, const lioncub_rows* summed, const lioncub_packed* saved, float* rstd,
                             const lioncub_rows* out, const lioncub_packed* packed_out, lioncub_stream_t stream)
{
    if (!h)
        return fail(LIONCUB_ERR_ARG, "the handle is NULL");
    NvtxRange range("lioncub_rms_norm_forward");
    if (!x || !out == !packed_out)
        return fail(LIONCUB_ERR_ARG, x ? "one of out and packed_out is needed" : "x is NULL");
    Operands o;
    o.code = check_size(n, h->dim);
    o.input("x", x, n, h->dim);
    o.input("residual", residual, n, h->dim);
    o.input("weight", weight, 1, h->dim, 1);  // read between the sum's writing and the result's
    o.result("summed", summed, n, h->dim);
    o.result("saved", saved, n, h->dim);
    o.vector("rstd", rstd, n, true);
    o.result("out", out, n, h->dim, 1);
    o.result("packed_out", packed_out, n, h->dim);
    int rc = o.finish();
    if (rc == LIONCUB_OK)
        rc = check_device(h);
    if (rc != LIONCUB_OK)
        return rc;
    lc::NormArgs a{};
    a.x = typed(x, n, h->dim);
    a.residual = typed(residual, n, h->dim);
    a.weight = typed(weight, 1, h->dim);
    a.summed = typed(summed, n, h->dim);
    a.out = typed(out, n, h->dim);
    a.saved = packed(saved, n, h->dim);
    a.packed = packed(packed_out, n, h->dim);
    a.rstd = rstd;
    a.n = n;
    a.dim = static_cast<int32_t>(h->dim);
    a.eps = h->eps;
    const bool vec = o.vec && h->dim % 8 == 0;
    return finish_launch(launch(h, "rms_norm", [&] { return lc::launch_norm(a, vec, stream); }), "norm launch");
}

int lioncub_rms_norm_backward(lioncub_rms_norm_t h, int64_t n, const lioncub_rows* dout, const lioncub_rows* saved,
                              const lioncub_packed* packed_saved, const float* rstd, const lioncub_rows* weight,
                              const lioncub_rows* residual_grad, const lioncub_rows* dx, const lioncub_rows* weight_base,
                              const lioncub_rows* weight_grad, const lioncub_rows* again, lioncub_stream_t stream)
{
    if (!h)
        return fail(LIONCUB_ERR_ARG, "the handle is NULL");
    NvtxRange range("lioncub_rms_norm_backward");
    if (!dout || !dx)
        return fail(LIONCUB_ERR_ARG, "%s is NULL", dout ? "dx" : "dout");
    if (!saved == !packed_saved)
        return fail(LIONCUB_ERR_ARG, "one of saved and packed_saved is needed");
    if (!rstd && n > 0)
        return fail(LIONCUB_ERR_ARG, "rstd is NULL");
    if (weight_base && !weight_grad)
        return fail(LIONCUB_ERR_ARG, "weight_base without weight_grad");
    if (weight_base && weight_base->type != weight_grad->type)
        return fail(LIONCUB_ERR_ARG, "weight_grad and its base must have one type");
    Operands o;
    o.code = check_size(n, h->dim);
    o.input("dout", dout, n, h->dim);
    o.input("saved", saved, n, h->dim);
    o.input("packed_saved", packed_saved, n, h->dim);
    o.vector("rstd", rstd, n, false);
    o.input("weight", weight, 1, h->dim);
    o.input("residual_grad", residual_grad, n, h->dim);
    o.result("dx", dx, n, h->dim);
    o.result("again", again, n, h->dim);
    // Rows are copied by 16 bytes, codes among them.  The weight's gradient is moved element by element.
    const bool vec = o.vec && h->dim % (packed_saved ? 16 : 8) == 0 &&
                     (!packed_saved || (reinterpret_cast<uintptr_t>(packed_saved->codes) | (n > 1 ? packed_saved->stride : 0)) % 16 == 0);
    o.input("weight_base", weight_base, 1, h->dim, 1);  // by the second launch
    o.result("weight_grad", weight_grad, 1, h->dim, 1);
    int rc = o.finish();
    if (rc == LIONCUB_OK)
        rc = check_device(h);
    if (rc != LIONCUB_OK)
        return rc;
    lc::NormGradArgs a{};
    a.dout = typed(dout, n, h->dim);
    a.saved = typed(saved, n, h->dim);
    a.residual_grad = typed(residual_grad, n, h->dim);
    a.dx = typed(dx, n, h->dim);
    a.weight = typed(weight, 1, h->dim);
    a.again = typed(again, n, h->dim);
    a.packed = packed(packed_saved, n, h->dim);
    a.rstd = rstd;
    a.partial = weight_grad ? h->partial : nullptr;
    a.partial_rows = h->multiprocessors;
    a.n = n;
    a.dim = static_cast<int32_t>(h->dim);
    a.first_wait_polls = h->first_wait_polls;
    a.status = h->status;
    const int blocks = lc::norm_grad_blocks(n, a.dim, h->multiprocessors);
    cudaError_t e = launch(h, "rms_norm_grad", [&] { return lc::launch_norm_grad(a, blocks, vec, stream); });
    if (e != cudaSuccess)
        return cuda_fail(e, "norm gradient launch");
    if (!weight_grad)
        return LIONCUB_OK;
    lc::WeightGradArgs w{};
    w.partial = h->partial;
    w.rows = blocks;
    w.base = typed(weight_base, 1, h->dim);
    w.grad = typed(weight_grad, 1, h->dim);
    w.dim = a.dim;
    return finish_launch(launch(h, "rms_norm_weight_grad", [&] { return lc::launch_weight_grad(w, stream); }), "weight gradient launch");
}

// ---- 8 bits --------------------------------------------------------------------------------

int lioncub_pack8(int64_t rows, int64_t cols, const lioncub_rows* x, const lioncub_packed* out, lioncub_stream_t stream)
{
    NvtxRange range("lioncub_pack8");
    if (!x || !out)
        return fail(LIONCUB_ERR_ARG, "%s is NULL", x ? "out" : "x");
    Operands o;
    o.code = check_size(rows, cols);
    o.input("x", x, rows, cols);
    o.result("out", out, rows, cols);
    const int rc = o.finish();
    if (rc != LIONCUB_OK)
        return rc;
    if (out->group == 0 && cols > LIONCUB_NORM_MAX_DIM)
        return fail(LIONCUB_ERR_ARG, "rows of up to %d columns may share one scale (got %lld)", LIONCUB_NORM_MAX_DIM, (long long)cols);
    if (rows == 0 || cols == 0)
        return LIONCUB_OK;
    if (out->group == 0)
        return finish_launch(lc::launch_pack_rows(typed(x, rows, cols), packed(out, rows, cols), rows, static_cast<int>(cols), o.vec && cols % 8 == 0, stream),
                             "pack launch");
    lc::ActivationArgs a{};
    const bool vec = as_one_row(o, rows, cols);
    a.x = typed(x, rows, cols);
    a.saved = packed(out, rows, cols);
    a.rows = rows;
    a.cols = cols;
    return finish_launch(lc::launch_activation(a, lc::kIdentity, vec, stream), "pack launch");
}

int lioncub_unpack8(int64_t rows, int64_t cols, const lioncub_packed* x, const lioncub_rows* out, lioncub_stream_t stream)
{
    NvtxRange range("lioncub_unpack8");
    if (!x || !out)
        return fail(LIONCUB_ERR_ARG, "%s is NULL", x ? "out" : "x");
    Operands o;
    o.code = check_size(rows, cols);
    o.input("x", x, rows, cols);
    o.result("out", out, rows, cols);
    const int rc = o.finish();
    if (rc != LIONCUB_OK)
        return rc;
    const bool vec = as_one_row(o, rows, cols);
    return finish_launch(lc::launch_unpack(packed(x, rows, cols), typed(out, rows, cols), rows, cols, vec, stream), "unpack launch");
}

// ---- the activation --------------------------------------------------------------------------

int lioncub_activation_forward(int64_t rows, int64_t cols, int kind, const lioncub_rows* x, const lioncub_rows* up,
                               const lioncub_rows* out, const lioncub_packed* saved, const lioncub_packed* saved_up,
                               lioncub_stream_t stream)
{
    NvtxRange range("lioncub_activation_forward");
    if (!x || !out)
        return fail(LIONCUB_ERR_ARG, "%s is NULL", x ? "out" : "x");
    if (saved_up && !up)
        return fail(LIONCUB_ERR_ARG, "saved_up without up");
    Operands o;
    o.code = check_kind(kind);
    if (o.code == LIONCUB_OK)
        o.code = check_size(rows, cols);
    o.input("x", x, rows, cols);
    o.input("up", up, rows, cols);
    o.result("out", out, rows, cols);
    o.result("saved", saved, rows, cols);
    o.result("saved_up", saved_up, rows, cols);
    int rc = o.finish();
    if (rc == LIONCUB_OK)
        rc = check_type("up", up, x);
    if (rc == LIONCUB_OK)
        rc = check_type("out", out, x);
    if (rc == LIONCUB_OK && ((saved && !saved->group) || (saved_up && !saved_up->group)))
        rc = fail(LIONCUB_ERR_ARG, "saved matrices need groups of columns, not whole rows");
    if (rc != LIONCUB_OK)
        return rc;
    lc::ActivationArgs a{};
    const bool vec = as_one_row(o, rows, cols);
    a.x = typed(x, rows, cols);
    a.up = typed(up, rows, cols);
    a.out = typed(out, rows, cols);
    a.saved = packed(saved, rows, cols);
    a.saved_up = packed(saved_up, rows, cols);
    a.rows = rows;
    a.cols = cols;
    return finish_launch(lc::launch_activation(a, kind, vec, stream), "activation launch");
}

int lioncub_activation_backward(int64_t rows, int64_t cols, int kind, const lioncub_rows* dout, const lioncub_rows* x,
                                const lioncub_rows* up, const lioncub_packed* packed_x, const lioncub_packed* packed_up,
                                const lioncub_rows* dx, const lioncub_rows* dup, const lioncub_rows* again, lioncub_stream_t stream)
{
    NvtxRange range("lioncub_activation_backward");
    if (!dout || !dx)
        return fail(LIONCUB_ERR_ARG, "%s is NULL", dout ? "dx" : "dout");
    if (!x == !packed_x || (packed_up && !packed_x) || (up && !x))
        return fail(LIONCUB_ERR_ARG, "x and up are needed as matrices or packed, both the same way");
    if (dup && !up && !packed_up)
        return fail(LIONCUB_ERR_ARG, "dup without up");
    Operands o;
    o.code = check_kind(kind);
    if (o.code == LIONCUB_OK)
        o.code = check_size(rows, cols);
    o.input("dout", dout, rows, cols);
    o.input("x", x, rows, cols);
    o.input("up", up, rows, cols);
    o.input("packed_x", packed_x, rows, cols);
    o.input("packed_up", packed_up, rows, cols);
    o.result("dx", dx, rows, cols);
    o.result("dup", dup, rows, cols);
    o.result("again", again, rows, cols);
    int rc = o.finish();
    const struct { const char* name; const lioncub_rows* m; } others[] = {{"x", x}, {"up", up}, {"dx", dx}, {"dup", dup}, {"again", again}};
    for (const auto& m : others)
        if (rc == LIONCUB_OK)
            rc = check_type(m.name, m.m, dout);
    if (rc != LIONCUB_OK)
        return rc;
    lc::ActivationArgs a{};
    const bool vec = as_one_row(o, rows, cols);
    a.dout = typed(dout, rows, cols);
    a.x = typed(x, rows, cols);
    a.up = typed(up, rows, cols);
    a.saved = packed(packed_x, rows, cols);
    a.saved_up = packed(packed_up, rows, cols);
    a.dx = typed(dx, rows, cols);
    a.dup = typed(dup, rows, cols);
    a.again = typed(again, rows, cols);
    a.rows = rows;
    a.cols = cols;
    return finish_launch(lc::launch_activation_grad(a, kind, vec, stream), "activation gradient launch");
}

// ---- rotary positions ---------------------------------------------------------------------------

int lioncub_rotary_frequencies(int64_t rotary_dim, double base, const lioncub_rotary_scaling* scaling, double* frequencies)
{
    t_error[0] = '\0';
    if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > LIONCUB_ROTARY_MAX_DIM)
        return fail(LIONCUB_ERR_ARG, "rotary_dim must be even, 2..%d (got %lld)", LIONCUB_ROTARY_MAX_DIM, (long long)rotary_dim);
    if (!frequencies)
        return fail(LIONCUB_ERR_ARG, "frequencies is NULL");
    if (!(base >= 1.0) || !std::isfinite(base))
        return fail(LIONCUB_ERR_ARG, "base must be 1 or more");
    const int kind = scaling ? scaling->kind : LIONCUB_SCALING_NONE;
    if (kind < LIONCUB_SCALING_NONE || kind > LIONCUB_SCALING_PARTS)
        return fail(LIONCUB_ERR_ARG, "unknown scaling %d", kind);
    const double factor = kind == LIONCUB_SCALING_NONE ? 1.0 : scaling->factor;
    if (!(factor >= 1.0) || !std::isfinite(factor))
        return fail(LIONCUB_ERR_ARG, "factor must be 1 or more");
    if (kind == LIONCUB_SCALING_BASE) {
        if (rotary_dim == 2)
            return fail(LIONCUB_ERR_ARG, "two columns have one frequency, which does not go by the base");
        base *= std::pow(factor, static_cast<double>(rotary_dim) / static_cast<double>(rotary_dim - 2));
    }
    if (kind == LIONCUB_SCALING_PARTS && !(scaling->length > 0.0 && std::isfinite(scaling->length) && scaling->low >= 0.0 &&
                                           scaling->high > scaling->low && std::isfinite(scaling->high)))
        return fail(LIONCUB_ERR_ARG, "length must be positive and low below high");
    constexpr double kTurn = 6.283185307179586476925;
    for (int64_t k = 0; k < rotary_dim / 2; ++k) {
        const double f = std::pow(base, -2.0 * static_cast<double>(k) / static_cast<double>(rotary_dim));
        double share = kind == LIONCUB_SCALING_LINEAR ? 0.0 : 1.0;  // of f itself, the rest of f / factor
        if (kind == LIONCUB_SCALING_PARTS)
            share = std::min(1.0, std::max(0.0, (scaling->length * f / kTurn - scaling->low) / (scaling->high - scaling->low)));
        frequencies[k] = share == 1.0 ? f : f * (share + (1.0 - share) / factor);
    }
    return LIONCUB_OK;
}

int lioncub_rotary_create(lioncub_rotary_t* out, int64_t head_dim, int64_t rotary_dim, const double* frequencies, float magnitude,
                          int interleaved)
{
    t_error[0] = '\0';
    if (!out)
        return fail(LIONCUB_ERR_ARG, "out is NULL");
    *out = nullptr;
    if (head_dim < 2 || head_dim > LIONCUB_ROTARY_MAX_DIM || rotary_dim < 2 || rotary_dim > head_dim || rotary_dim % 2)
        return fail(LIONCUB_ERR_ARG, "head_dim must be 2..%d and rotary_dim even, 2..head_dim (got %lld, %lld)", LIONCUB_ROTARY_MAX_DIM,
                    (long long)head_dim, (long long)rotary_dim);
    if (!frequencies)
        return fail(LIONCUB_ERR_ARG, "frequencies is NULL");
    if (!std::isfinite(magnitude))
        return fail(LIONCUB_ERR_ARG, "magnitude must be finite");
    uint64_t turns[LIONCUB_ROTARY_MAX_DIM / 2];
    for (int64_t k = 0; k < rotary_dim / 2; ++k) {
        if (!(frequencies[k] >= 0.0 && frequencies[k] < 65536.0))
            return fail(LIONCUB_ERR_ARG, "frequency %lld is not in [0, 65536)", (long long)k);
        const double t = frequencies[k] * 0.15915494309189533577;  // 1 / (2 pi)
        turns[k] = static_cast<uint64_t>(std::ldexp(t - std::floor(t), 64) + 0.5);  // below 2^64: the difference has 53 bits and is below 1
    }
    lioncub_rotary_t h = new (std::nothrow) lioncub_rotary_s();
    if (!h)
        return fail(LIONCUB_ERR_OOM, "no host memory for the handle");
    h->head_dim = head_dim;
    h->rotary_dim = rotary_dim;
    h->magnitude = magnitude;
    h->interleaved = interleaved != 0;
    h->fail_launch_at = lc::env_index("LIONCUB_FAIL_LAUNCH");
    const size_t bytes = rotary_dim / 2 * sizeof(uint64_t);
    cudaError_t e = cudaGetDevice(&h->device);
    if (e == cudaSuccess)
        e = lc::env_index("LIONCUB_FAIL_ALLOC") == 1 ? cudaErrorMemoryAllocation
                                                     : cudaMalloc(reinterpret_cast<void**>(&h->turns), bytes);
    if (e != cudaSuccess)
        h->turns = nullptr;
    if (e == cudaSuccess)
        e = cudaMemcpyAsync(h->turns, turns, bytes, cudaMemcpyHostToDevice, nullptr);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        lioncub_rotary_destroy(h);
        cudaGetLastError();
        return e == cudaErrorMemoryAllocation ? fail(LIONCUB_ERR_OOM, "no device memory for the frequencies") : cuda_fail(e, "create");
    }
    *out = h;
    return LIONCUB_OK;
}

int lioncub_rotary_apply(lioncub_rotary_t h, const lioncub_sequences* places, const lioncub_heads* q, const lioncub_heads* q_out,
                         const lioncub_heads* k, const lioncub_heads* k_out, int inverse, lioncub_stream_t stream)
{
    if (!h)
        return fail(LIONCUB_ERR_ARG, "the handle is NULL");
    NvtxRange range("lioncub_rotary_apply");
    if (!places || !q || !q_out || !k != !k_out)
        return fail(LIONCUB_ERR_ARG, "%s is NULL", !places ? "places" : !q ? "q" : !q_out ? "q_out" : k ? "k_out" : "k");
    const lioncub_sequences p = *places;
    if (p.batch < 0 || p.seq_len < 0 || p.batch > INT_MAX || p.seq_len > INT_MAX || (p.seq_len > 0 && p.batch > INT_MAX / p.seq_len))
        return fail(LIONCUB_ERR_ARG, "bad sizes: %lld sequences of %lld places", (long long)p.batch, (long long)p.seq_len);
    if (p.positions) {
        if (p.index_type != LIONCUB_INDEX_I64 && p.index_type != LIONCUB_INDEX_I32)
            return fail(LIONCUB_ERR_ARG, "unknown index type %d", p.index_type);
        if (reinterpret_cast<uintptr_t>(p.positions) % (p.index_type == LIONCUB_INDEX_I64 ? 8 : 4))
            return fail(LIONCUB_ERR_ALIGN, "positions are not aligned to their elements");
    } else if (p.first_position < -(int64_t(1) << 40) || p.first_position > int64_t(1) << 40) {
        return fail(LIONCUB_ERR_ARG, "first_position %lld is beyond 2^40", (long long)p.first_position);
    }
    const lioncub_heads* in[2] = {q, k};
    const lioncub_heads* to[2] = {q_out, k_out};
    static const char* const names[2][2] = {{"q", "q_out"}, {"k", "k_out"}};
    uintptr_t reach = 0;
    bool copy = false;
    for (int i = 0; i < 2 && in[i]; ++i) {
        int rc = check_heads(names[i][0], in[i], p, h->head_dim, false, &reach);
        if (rc == LIONCUB_OK)
            rc = check_heads(names[i][1], to[i], p, h->head_dim, true, &reach);
        if (rc == LIONCUB_OK)
            rc = check_positions(names[i][1], *to[i], p, h->head_dim);
        if (rc != LIONCUB_OK)
            return rc;
        if (in[i]->type != q->type || to[i]->type != q->type)
            return fail(LIONCUB_ERR_ARG, "%s: the heads must be of one type", names[i][to[i]->type != q->type]);
        if (in[i]->heads != to[i]->heads)
            return fail(LIONCUB_ERR_ARG, "%s: %d heads for %d", names[i][1], to[i]->heads, in[i]->heads);
        copy = copy || !same_heads(*in[i], *to[i], p);
    }
    for (int i = 0; i < 2 && to[i]; ++i) {
        const Box mine = box_of(*to[i], p, h->head_dim);
        for (int j = 0; j < 2 && in[j]; ++j) {
            const bool same = i == j && same_heads(*in[j], *to[i], p);
            if (!same && overlap(mine, box_of(*in[j], p, h->head_dim)))
                return fail(LIONCUB_ERR_ARG, "%s may overlap %s without being it", names[i][1], names[j][0]);
        }
        if (i == 1 && overlap(mine, box_of(*to[0], p, h->head_dim)))
            return fail(LIONCUB_ERR_ARG, "k_out may overlap q_out");
    }
    const int rc = check_device(h);
    if (rc != LIONCUB_OK)
        return rc;
    lc::RotaryArgs a{};
    a.side[0] = heads_of(*q, *q_out, p, h->head_dim);
    a.heads[0] = q->heads;
    if (k) {
        a.side[1] = heads_of(*k, *k_out, p, h->head_dim);
        a.heads[1] = k->heads;
    }
    a.turns = h->turns;
    a.positions = p.positions;
    a.wide = p.index_type == LIONCUB_INDEX_I64;
    a.first = p.first_position;
    a.places = p.batch * p.seq_len;
    a.seq = static_cast<int32_t>(p.seq_len);
    a.head_dim = static_cast<int32_t>(h->head_dim);
    a.pairs = static_cast<int32_t>(h->rotary_dim / 2);
    a.copy = copy;
    a.cos_factor = h->magnitude;
    a.sin_factor = inverse ? -h->magnitude : h->magnitude;
    // elements moved at once: halves of the rotated columns (or all of them, where pairs lie side
    // by side), and those behind, are whole moves
    const int64_t widths = h->head_dim | (h->interleaved ? 2 * a.pairs : a.pairs);
    const int64_t size = static_cast<int64_t>(element_size(q->type));
    int move = reach % 16 == 0 && h->head_dim % 8 == 0 && a.pairs % 8 == 0 ? 8 : 4;
    while (move < 8 && move > 1 && (reach % (move * size) || widths % move))
        move /= 2;
    const bool copy_by_four = reach % (4 * size) == 0 && h->head_dim % 4 == 0 && a.pairs % 2 == 0;
    return finish_launch(launch(h, "rotary", [&] { return lc::launch_rotary(a, q->type, h->interleaved, move, copy_by_four, stream); }), "rotary launch");
}

void lioncub_rotary_destroy(lioncub_rotary_t h)
{
    if (!h)
        return;
    cudaFree(h->turns);
    delete h;
}

}  // extern "C"
