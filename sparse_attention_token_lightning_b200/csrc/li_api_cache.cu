// Host side of the rotary, cache and cache-attention entry points of include/li.h: argument
// validation and the launch sequence.
#include <cmath>
#include <initializer_list>

#include "li_cache.cuh"
#include "li_cache_attn.cuh"
#include "li_host.cuh"
#include "li_internal.cuh"
#include "li_rope.cuh"

namespace {

using namespace li::host;
using li::dtype_bytes;

// Strides are element counts; the limit keeps every offset far inside 64 bits.
bool strides_ok(std::initializer_list<int64_t> v) {
    for (int64_t s : v)
        if (s < 0 || s > ((int64_t)1 << 31)) return false;
    return true;
}

// Whether n x m runs of d elements lie apart, at strides ns and ms: the m inside the n or the n inside the m.
bool apart(int64_t n, int64_t ns, int64_t m, int64_t ms, int64_t d) {
    const bool m_in = (m == 1 || ms >= d) && (n == 1 || ns >= (m == 1 ? 0 : (m - 1) * ms) + d);
    const bool n_in = (n == 1 || ns >= d) && (m == 1 || ms >= (n == 1 ? 0 : (n - 1) * ns) + d);
    return m_in || n_in;
}

li_status validate_rope(const li_rope_args *a) {
    if (!a) return fail(LI_ERR_INVALID_ARG, "args is NULL");
    const int e = dtype_bytes(a->dtype);
    if (!e) return fail(LI_ERR_INVALID_ARG, "dtype=%d, must be bf16, fp16 or fp32", a->dtype);
    if (a->rope_dim < 2 || a->rope_dim > 2 * LI_ROPE_MAX_PAIRS || a->rope_dim % 2)
        return fail(LI_ERR_INVALID_ARG, "rope_dim=%d must be even in [2, %d]", a->rope_dim,
                    2 * LI_ROPE_MAX_PAIRS);
    if (a->heads < 1 || a->heads > 1024 || a->head_dim < a->rope_dim || a->head_dim > 4096)
        return fail(LI_ERR_INVALID_ARG, "heads=%d (1..1024), head_dim=%d (rope_dim..4096)", a->heads,
                    a->head_dim);
    if (a->rope_offset < 0 || a->rope_offset > a->head_dim - a->rope_dim)
        return fail(LI_ERR_INVALID_ARG, "rope_offset=%d outside [0, %d]", a->rope_offset,
                    a->head_dim - a->rope_dim);
    if (a->interleaved != 0 && a->interleaved != 1)
        return fail(LI_ERR_INVALID_ARG, "interleaved=%d, must be 0 or 1", a->interleaved);
    if (a->position_bits != 32 && a->position_bits != 64)
        return fail(LI_ERR_INVALID_ARG, "position_bits=%d, must be 32 or 64", a->position_bits);
    if (a->rows < 0) return fail(LI_ERR_INVALID_ARG, "rows=%lld < 0", (long long)a->rows);
    if (a->rows > INT32_MAX)
        return fail(LI_ERR_UNSUPPORTED, "rows=%lld above 2^31-1", (long long)a->rows);
    if (!std::isfinite(a->magnitude))
        return fail(LI_ERR_INVALID_ARG, "magnitude must be finite");
    for (int i = 0; i < a->rope_dim / 2; ++i)
        if (!std::isfinite(a->freq[i]))
            return fail(LI_ERR_INVALID_ARG, "freq[%d] must be finite", i);
    if (!strides_ok({a->x_row_stride, a->x_head_stride, a->y_row_stride, a->y_head_stride}))
        return fail(LI_ERR_INVALID_ARG, "strides must lie in [0, 2^31]");
    if (a->rows == 0) return LI_OK;
    if (!a->x || !a->y || !a->positions)
        return fail(LI_ERR_INVALID_ARG, "x, y and positions are required");
    if (!aligned(a->x, e) || !aligned(a->y, e) || !aligned(a->positions, a->position_bits / 8))
        return fail(LI_ERR_INVALID_ARG, "x, y and positions must be aligned to their elements");
    if (a->x == a->y && (a->x_row_stride != a->y_row_stride || a->x_head_stride != a->y_head_stride))
        return fail(LI_ERR_INVALID_ARG, "in place, x and y must have the same strides");
    if (!apart(a->rows, a->y_row_stride, a->heads, a->y_head_stride, a->head_dim))
        return fail(LI_ERR_INVALID_ARG, "y's strides (%lld, %lld) make its elements overlap",
                    (long long)a->y_row_stride, (long long)a->y_head_stride);
    return LI_OK;
}

li_status run_rope(const li_rope_args *args, bool grad, void *stream) {
    li_status st = validate_rope(args);
    if (st != LI_OK) return st;
    if (args->rows == 0) return ok();
    cudaError_t e = li::launch_rope(*args, grad, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(LI_ERR_CUDA, "rope launch: %s", cudaGetErrorString(e));
    return ok();
}

li_status validate_cache(const li_cache_args *a) {
    if (!a) return fail(LI_ERR_INVALID_ARG, "args is NULL");
    if (a->reserved != 0) return fail(LI_ERR_INVALID_ARG, "reserved field must be 0");
    const int e = dtype_bytes(a->dtype);
    if (!e) return fail(LI_ERR_INVALID_ARG, "dtype=%d, must be bf16, fp16 or fp32", a->dtype);
    if (a->pow2 != 0 && a->pow2 != 1) return fail(LI_ERR_INVALID_ARG, "pow2=%d, must be 0 or 1", a->pow2);
    if (a->dim < 16 || a->dim > 1024 || a->dim % 16)
        return fail(LI_ERR_INVALID_ARG, "dim=%d must be a multiple of 16 in [16, 1024]", a->dim);
    if (a->rope_dim < 0 || a->rope_dim > 256 || a->rope_dim % 8)
        return fail(LI_ERR_INVALID_ARG, "rope_dim=%d must be a multiple of 8 in [0, 256]", a->rope_dim);
    if (a->batch < 0 || a->x_len < 0) return fail(LI_ERR_INVALID_ARG, "batch / x_len must be >= 0");
    if (a->layout_x != LI_LAYOUT_BSND && a->layout_x != LI_LAYOUT_TND)
        return fail(LI_ERR_INVALID_ARG, "layout_x=%d, must be BSND or TND", a->layout_x);
    const bool tnd = a->layout_x == LI_LAYOUT_TND;
    const int64_t rows = tnd ? (a->batch > 0 ? a->x_len : 0) : (int64_t)a->batch * a->x_len;
    if (rows > INT32_MAX) return fail(LI_ERR_UNSUPPORTED, "more than 2^31-1 rows");
    if (tnd != (a->cu_seqlens != nullptr) && rows > 0)
        return fail(LI_ERR_INVALID_ARG, "cu_seqlens goes with layout_x = TND, and only with it");
    if (a->layout_k == LI_LAYOUT_PA_BSND) {
        if (a->block_size < 1 || a->block_size > 1024)
            return fail(LI_ERR_INVALID_ARG, "block_size=%d outside [1, 1024]", a->block_size);
        if (a->num_blocks < 1) return fail(LI_ERR_INVALID_ARG, "num_blocks must be >= 1");
        if ((int64_t)a->num_blocks * a->block_size > INT32_MAX)
            return fail(LI_ERR_UNSUPPORTED, "more than 2^31-1 cache rows");
        if (a->block_table_stride < 1 || a->block_table_stride > INT32_MAX)
            return fail(LI_ERR_INVALID_ARG, "block_table_stride=%lld outside [1, 2^31-1]",
                        (long long)a->block_table_stride);
        if (rows > 0 && (!a->block_table || !a->seqused_k))
            return fail(LI_ERR_INVALID_ARG, "PA_BSND needs block_table and seqused_k");
    } else if (a->layout_k == LI_LAYOUT_BSND) {
        if (a->block_table || a->block_table_stride || a->num_blocks || a->block_size)
            return fail(LI_ERR_INVALID_ARG, "block_table fields are for PA_BSND only");
        if (a->k_len < 0) return fail(LI_ERR_INVALID_ARG, "k_len=%d < 0", a->k_len);
        if ((int64_t)a->batch * a->k_len > INT32_MAX)
            return fail(LI_ERR_UNSUPPORTED, "more than 2^31-1 cache rows");
    } else {
        return fail(LI_ERR_INVALID_ARG, "layout_k=%d must be BSND or PA_BSND", a->layout_k);
    }
    if (!strides_ok({a->x_row_stride, a->rope_row_stride}) || a->x_batch_stride < 0 ||
        a->rope_batch_stride < 0 || a->x_batch_stride > ((int64_t)1 << 40) ||
        a->rope_batch_stride > ((int64_t)1 << 40))
        return fail(LI_ERR_INVALID_ARG, "row strides must lie in [0, 2^31], batch strides in [0, 2^40]");
    if (rows > 0) {
        if (!a->x || !a->codes || !a->descale)
            return fail(LI_ERR_INVALID_ARG, "x, codes and descale are required");
        if ((a->rope_dim > 0) != (a->rope != nullptr) || (a->rope_dim > 0) != (a->rope_cache != nullptr))
            return fail(LI_ERR_INVALID_ARG, "rope and rope_cache go with rope_dim > 0, and only with it");
    }
    if (!aligned(a->x, e) || !aligned(a->rope, e) || !aligned(a->codes, 16) ||
        !aligned(a->rope_cache, 16) || !aligned(a->descale, 4) || !aligned(a->cu_seqlens, 4) ||
        !aligned(a->seqused, 4) || !aligned(a->seqused_k, 4) || !aligned(a->block_table, 4) ||
        !aligned(a->device_status, 4))
        return fail(LI_ERR_INVALID_ARG, "codes and rope_cache must be 16-byte aligned, the others "
                    "to their elements");
    return LI_OK;
}

bool cache_has_rows(const li_cache_args *a) { return a->batch > 0 && a->x_len > 0; }

// Rows that li_cache_read writes must not overlap.
li_status validate_cache_out(const li_cache_args *a) {
    const int64_t n = a->layout_x == LI_LAYOUT_TND ? 1 : a->batch;
    if (!apart(n, a->x_batch_stride, a->x_len, a->x_row_stride, a->dim) ||
        (a->rope_dim > 0 && !apart(n, a->rope_batch_stride, a->x_len, a->rope_row_stride, a->rope_dim)))
        return fail(LI_ERR_INVALID_ARG, "the strides of x or rope make rows overlap");
    return LI_OK;
}

li_status validate_cache_attn(const li_cache_attn_args *a, li::CacheAttnPlan *p) {
    if (!a) return fail(LI_ERR_INVALID_ARG, "args is NULL");
    if (a->reserved != 0) return fail(LI_ERR_INVALID_ARG, "reserved field must be 0");
    if (a->batch < 0 || a->s1 < 0 || a->s2 < 0)
        return fail(LI_ERR_INVALID_ARG, "batch / s1 / s2 must be >= 0");
    if (a->G < 1 || a->G > 128) return fail(LI_ERR_INVALID_ARG, "G=%d outside [1, 128]", a->G);
    if (a->Dm < 128 || a->Dm > 512 || a->Dm % 128)
        return fail(LI_ERR_INVALID_ARG, "Dm=%d must be 128, 256, 384 or 512", a->Dm);
    if (a->Dr != 0 && a->Dr != 64) return fail(LI_ERR_INVALID_ARG, "Dr=%d must be 0 or 64", a->Dr);
    if (a->topk < 1 || a->topk > li::kMaxTopk)
        return fail(LI_ERR_INVALID_ARG, "topk=%d outside [1, 8192]", a->topk);
    if (!(a->scale > 0.0f) || !(a->scale < 3.0e38f))
        return fail(LI_ERR_INVALID_ARG, "scale must be a positive finite number");
    const int64_t rows = (int64_t)a->batch * a->s1;
    if (rows > 0 && a->s2 < 1) return fail(LI_ERR_INVALID_ARG, "S2=0 with query rows");
    if (rows > INT32_MAX / 128 || (int64_t)a->batch * a->s2 > INT32_MAX)
        return fail(LI_ERR_UNSUPPORTED, "more than 2^24-1 query rows or 2^31-1 key rows");
    if (rows > 0 && (!a->q || !a->codes || !a->descale || !a->sparse_indices))
        return fail(LI_ERR_INVALID_ARG, "q, codes, descale and sparse_indices are required");
    if (rows > 0 && ((a->Dr > 0) != (a->q_rope != nullptr) || (a->Dr > 0) != (a->k_rope != nullptr)))
        return fail(LI_ERR_INVALID_ARG, "q_rope and k_rope go with Dr > 0, and only with it");
    if (a->layout_k == LI_LAYOUT_PA_BSND) {
        if (a->block_size < 1 || a->block_size > 1024)
            return fail(LI_ERR_INVALID_ARG, "block_size=%d outside [1, 1024]", a->block_size);
        if (a->num_blocks < 1) return fail(LI_ERR_INVALID_ARG, "num_blocks must be >= 1");
        if ((int64_t)a->num_blocks * a->block_size > INT32_MAX)
            return fail(LI_ERR_UNSUPPORTED, "more than 2^31-1 cache rows");
        const int64_t need = ((int64_t)a->s2 + a->block_size - 1) / a->block_size;
        if (a->block_table_stride < need || a->block_table_stride > INT32_MAX)
            return fail(LI_ERR_INVALID_ARG, "block_table_stride=%lld outside [ceil(S2 / block_size)=%lld, 2^31-1]",
                        (long long)a->block_table_stride, (long long)need);
        if (rows > 0 && !a->block_table)
            return fail(LI_ERR_INVALID_ARG, "PA_BSND needs a block_table");
    } else if (a->layout_k == LI_LAYOUT_BSND) {
        if (a->block_table || a->block_table_stride || a->num_blocks || a->block_size)
            return fail(LI_ERR_INVALID_ARG, "block_table fields are for PA_BSND only");
    } else {
        return fail(LI_ERR_INVALID_ARG, "layout_k=%d must be BSND or PA_BSND", a->layout_k);
    }
    if (!aligned(a->q, 16) || !aligned(a->q_rope, 16) || !aligned(a->codes, 16) || !aligned(a->k_rope, 16) ||
        !aligned(a->descale, 4) || !aligned(a->sparse_indices, 4) || !aligned(a->block_table, 4) ||
        !aligned(a->device_status, 4))
        return fail(LI_ERR_INVALID_ARG, "q, codes and the rope parts must be 16-byte aligned, the "
                    "others 4-byte");
    if (!li::cache_attn_plan(*a, p))
        return fail(LI_ERR_UNSUPPORTED, "G=%d with Dm=%d does not fit the kernel's shared memory", a->G, a->Dm);
    return LI_OK;
}

}  // namespace

extern "C" {

li_status li_rope(const li_rope_args *args, void *stream) {
    NvtxRange range("li_rope");
    return run_rope(args, false, stream);
}

li_status li_rope_grad(const li_rope_args *args, void *stream) {
    NvtxRange range("li_rope_grad");
    return run_rope(args, true, stream);
}

li_status li_rope_frequencies(const li_rope_scaling *s, double *freq, float *magnitude) {
    if (!s || !freq || !magnitude) return fail(LI_ERR_INVALID_ARG, "an argument is NULL");
    if (s->reserved != 0) return fail(LI_ERR_INVALID_ARG, "reserved field must be 0");
    if (s->rope_dim < 2 || s->rope_dim > 2 * LI_ROPE_MAX_PAIRS || s->rope_dim % 2)
        return fail(LI_ERR_INVALID_ARG, "rope_dim=%d must be even in [2, %d]", s->rope_dim,
                    2 * LI_ROPE_MAX_PAIRS);
    if (!(s->base > 1.0) || !std::isfinite(s->base))
        return fail(LI_ERR_INVALID_ARG, "base must be above 1 and finite");
    if (s->mode != LI_ROPE_PLAIN && s->mode != LI_ROPE_LINEAR && s->mode != LI_ROPE_YARN)
        return fail(LI_ERR_INVALID_ARG, "mode=%d, must be 0, 1 or 2", s->mode);
    const bool scaled = s->mode != LI_ROPE_PLAIN;
    if (scaled && (!(s->factor > 0.0) || !std::isfinite(s->factor)))
        return fail(LI_ERR_INVALID_ARG, "factor must be positive and finite");
    const int n = s->rope_dim / 2;
    double low = 0.0, high = 0.0;
    if (s->mode == LI_ROPE_YARN) {
        if (!(s->beta_slow > 0.0) || !(s->beta_fast >= s->beta_slow) || !std::isfinite(s->beta_fast))
            return fail(LI_ERR_INVALID_ARG, "beta_fast >= beta_slow > 0 wanted");
        if (s->original_max < 1) return fail(LI_ERR_INVALID_ARG, "original_max=%d < 1", s->original_max);
        if (!(s->magnitude_coef >= 0.0) || !std::isfinite(s->magnitude_coef))
            return fail(LI_ERR_INVALID_ARG, "magnitude_coef must be >= 0 and finite");
        constexpr double kTwoPi = 6.283185307179586476925286766559;
        auto t = [&](double turns) {
            return s->rope_dim * std::log(s->original_max / (turns * kTwoPi)) / (2.0 * std::log(s->base));
        };
        low = std::fmax(std::floor(t(s->beta_fast)), 0.0);
        high = std::fmin(std::ceil(t(s->beta_slow)), s->rope_dim - 1.0);
    }
    for (int i = 0; i < n; ++i) {
        const double f = std::pow(s->base, -2.0 * i / s->rope_dim);
        if (s->mode == LI_ROPE_PLAIN) freq[i] = f;
        else if (s->mode == LI_ROPE_LINEAR) freq[i] = f / s->factor;
        else {
            const double r = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
            freq[i] = f * (1.0 - r) + f / s->factor * r;
        }
    }
    *magnitude = s->mode == LI_ROPE_YARN && s->factor > 1.0
                     ? (float)(s->magnitude_coef * std::log(s->factor) + 1.0)
                     : 1.0f;
    return ok();
}

li_status li_cache_write(const li_cache_args *args, void *stream) {
    NvtxRange range("li_cache_write");
    li_status st = validate_cache(args);
    if (st != LI_OK) return st;
    if (!cache_has_rows(args)) return ok();
    cudaError_t e = li::launch_cache_write(*args, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(LI_ERR_CUDA, "cache write launch: %s", cudaGetErrorString(e));
    return ok();
}

li_status li_cache_read(const li_cache_args *args, void *stream) {
    NvtxRange range("li_cache_read");
    li_status st = validate_cache(args);
    if (st != LI_OK) return st;
    if (!cache_has_rows(args)) return ok();
    st = validate_cache_out(args);
    if (st != LI_OK) return st;
    cudaError_t e = li::launch_cache_read(*args, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(LI_ERR_CUDA, "cache read launch: %s", cudaGetErrorString(e));
    return ok();
}

li_status li_cache_attention(const li_cache_attn_args *args, void *out, float *softmax_max, float *softmax_sum,
                             void *stream) {
    NvtxRange range("li_cache_attention");
    li::CacheAttnPlan p;
    li_status st = validate_cache_attn(args, &p);
    if (st != LI_OK) return st;
    if (p.units == 0) return ok();
    if (!out || !aligned(out, 16)) return fail(LI_ERR_INVALID_ARG, "out must be a 16-byte aligned device buffer");
    if ((softmax_max == nullptr) != (softmax_sum == nullptr) || !aligned(softmax_max, 4) || !aligned(softmax_sum, 4))
        return fail(LI_ERR_INVALID_ARG, "softmax_max and softmax_sum go together, 4-byte aligned");
    cudaError_t e = li::launch_cache_attention(*args, p, out, softmax_max, softmax_sum, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(LI_ERR_CUDA, "cache attention launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // extern "C"
