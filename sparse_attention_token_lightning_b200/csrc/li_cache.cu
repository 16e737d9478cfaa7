// Quantised key cache (li_cache_write, li_cache_read), sm_100a.
//
// write: s = max(max_d |x_d| / 448, 2^-90) over the row's finite elements (1 for a row of zeros),
// or the smallest power of two that is no less; code_d = E4M3(x_d / s). read: code_d s in fp32,
// rounded once. Row i of batch b is key position L2_b - L1_b + i and goes through the block table.
//
// A row belongs to a group of lanes (a power of two, eight elements a lane and step), so the
// row's maximum is a shuffle reduction and a row is read from memory once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "li_cache.cuh"

namespace li {
namespace {

constexpr int kThreads = 256;
constexpr float kMinScale = 8.077935669463161e-28f;     // 2^-90

struct CacheParams {
    void *x, *rope;
    uint8_t *codes;
    float *descale;
    uint8_t *rope_cache;
    const int32_t *cu_seqlens, *seqused, *seqused_k, *block_table;
    uint32_t *status;
    int64_t x_batch, x_row, r_batch, r_row;     // strides in elements
    int64_t bt_stride;
    int32_t rows, batch, x_len, k_len, num_blocks, block_size;
    int32_t dim, rope_dim;
    int32_t paged, lanes;                       // lanes per row
};

__device__ __forceinline__ void report(const CacheParams &P, uint32_t bits) {
    if (bits && P.status) atomicOr(P.status, bits);
}

// Where row r of the call sits: its batch and position inside it, and its cache row; false when
// the row takes no part (past the rows in use, or data that does not fit, which is reported).
struct Place {
    int64_t x_off, r_off;       // element offsets of the row in x and rope
    int64_t slot;               // cache row
};
__device__ __forceinline__ bool place_row(const CacheParams &P, int32_t r, Place *out) {
    int32_t b, i, L1;
    uint32_t err = 0;
    if (P.cu_seqlens) {
        const int32_t *cu = P.cu_seqlens;
        if (r < cu[0] || r >= cu[P.batch]) return false;
        int32_t lo = 0, hi = P.batch;
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if (cu[mid] <= r) lo = mid; else hi = mid;
        }
        b = lo;
        i = r - cu[b];
        L1 = cu[b + 1] - cu[b];
        if (i < 0 || i >= L1) {                 // only lengths that decrease lead here
            report(P, LI_DEVERR_LENGTHS);
            return false;
        }
        out->x_off = (int64_t)r * P.x_row;
        out->r_off = (int64_t)r * P.r_row;
    } else {
        b = r / P.x_len;
        i = r - b * P.x_len;
        L1 = P.x_len;
        out->x_off = b * P.x_batch + i * P.x_row;
        out->r_off = b * P.r_batch + i * P.r_row;
    }
    if (P.seqused) {
        const int32_t u = P.seqused[b];
        if (u < 0 || u > L1) err |= LI_DEVERR_LENGTHS;
        L1 = min(max(u, 0), L1);
    }
    const int64_t cap = P.paged ? P.bt_stride * P.block_size : P.k_len;
    int64_t L2 = P.k_len;
    if (P.seqused_k) {
        L2 = P.seqused_k[b];
        if (L2 < 0 || L2 > cap) err |= LI_DEVERR_LENGTHS;
    }
    const int64_t pos = L2 - L1 + i;
    bool take = i < L1;
    if (take && (pos < 0 || pos >= cap)) {
        err |= LI_DEVERR_LENGTHS;
        take = false;
    }
    if (take && P.paged) {
        const int32_t q = (int32_t)(pos / P.block_size);
        const int32_t blk = P.block_table[(int64_t)b * P.bt_stride + q];
        if (blk < 0 || blk >= P.num_blocks) {
            err |= LI_DEVERR_TABLE;
            take = false;
        }
        out->slot = (int64_t)blk * P.block_size + (pos - (int64_t)q * P.block_size);
    } else {
        out->slot = (int64_t)b * P.k_len + pos;
    }
    report(P, err);
    return take;
}

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f32(float v) { return v; }

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __int_as_float(0x7f800000); }

// E4M3 code of the exact quotient x / s. The fp32 quotient is rounded to odd first (its last bit
// set when the division leaves a remainder), so the second rounding sees on which side of a
// border between two codes the quotient lies.
__device__ __forceinline__ uint8_t quantise(float x, float s) {
    float q = __fdiv_rn(x, s);
    const float rem = fmaf(-q, s, x);
    if (rem != 0.0f && finite(q)) {
        int bits = __float_as_int(q);
        if ((rem < 0.0f) != (x < 0.0f)) bits -= 1;      // the quotient was rounded away from zero
        q = __int_as_float(bits | 1);
    }
    if (!finite(x)) q = __int_as_float(0x7fc00000);
    return (uint8_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float row_scale(float amax, bool pow2) {
    if (!(amax > 0.0f)) return 1.0f;
    if (!pow2) return fmaxf(__fdiv_rn(amax, 448.0f), kMinScale);
    // 448 = 1.75 x 2^8: the exponent of amax less 8, one more where its mantissa is above 1.75
    const int e = (__float_as_int(amax) + 0x1fffff) >> 23;
    return __int_as_float(max(e - 8, 127 - 90) << 23);
}

template <class T, bool kPow2>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheParams P) {
    const int lane = threadIdx.x % P.lanes;
    const int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / P.lanes;
    Place at;
    const bool take = r < P.rows && place_row(P, (int32_t)r, &at);
    const T *x = static_cast<const T *>(P.x) + (take ? at.x_off : 0);
    float amax = 0.0f;
    if (take)
        for (int d = lane; d < P.dim; d += P.lanes) {
            const float v = to_f32(x[d]);
            if (finite(v)) amax = fmaxf(amax, fabsf(v));
        }
    for (int o = P.lanes / 2; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!take) return;
    const float s = row_scale(amax, kPow2);
    if (lane == 0) P.descale[at.slot] = s;
    for (int d = lane; d < P.dim; d += P.lanes)
        P.codes[at.slot * P.dim + d] = quantise(to_f32(x[d]), s);
    const T *rx = static_cast<const T *>(P.rope) + at.r_off;
    T *rc = reinterpret_cast<T *>(P.rope_cache) + at.slot * P.rope_dim;
    for (int d = lane; d < P.rope_dim; d += P.lanes) rc[d] = rx[d];
}

template <class T>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheParams P) {
    const int lane = threadIdx.x % P.lanes;
    const int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / P.lanes;
    Place at;
    if (r >= P.rows || !place_row(P, (int32_t)r, &at)) return;
    T *x = static_cast<T *>(P.x) + at.x_off;
    const float s = P.descale[at.slot];
    for (int d = lane; d < P.dim; d += P.lanes) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(P.codes[at.slot * P.dim + d], __NV_E4M3);
        x[d] = from_f32<T>(__half2float(__half(h)) * s);
    }
    T *rx = static_cast<T *>(P.rope) + at.r_off;
    const T *rc = reinterpret_cast<const T *>(P.rope_cache) + at.slot * P.rope_dim;
    for (int d = lane; d < P.rope_dim; d += P.lanes) rx[d] = rc[d];
}

CacheParams params(const li_cache_args &a) {
    CacheParams P{};
    P.x = a.x;
    P.rope = a.rope;
    P.codes = static_cast<uint8_t *>(a.codes);
    P.descale = a.descale;
    P.rope_cache = static_cast<uint8_t *>(a.rope_cache);
    P.cu_seqlens = a.layout_x == LI_LAYOUT_TND ? a.cu_seqlens : nullptr;
    P.seqused = a.seqused;
    P.seqused_k = a.seqused_k;
    P.block_table = a.block_table;
    P.status = a.device_status;
    P.x_batch = a.x_batch_stride;
    P.x_row = a.x_row_stride;
    P.r_batch = a.rope_batch_stride;
    P.r_row = a.rope_row_stride;
    P.bt_stride = a.block_table_stride;
    P.rows = P.cu_seqlens ? a.x_len : a.batch * a.x_len;
    P.batch = a.batch;
    P.x_len = a.x_len;
    P.k_len = a.k_len;
    P.num_blocks = a.num_blocks;
    P.block_size = a.block_size;
    P.dim = a.dim;
    P.rope_dim = a.rope_dim;
    P.paged = a.layout_k == LI_LAYOUT_PA_BSND;
    P.lanes = 2;
    while (P.lanes < 32 && P.lanes * 8 < a.dim) P.lanes *= 2;
    return P;
}

unsigned blocks_of(const CacheParams &P) {
    return (unsigned)(((int64_t)P.rows * P.lanes + kThreads - 1) / kThreads);
}

}  // namespace

cudaError_t launch_cache_write(const li_cache_args &a, cudaStream_t st) {
    const CacheParams P = params(a);
    const unsigned n = blocks_of(P);
    auto go = [&](auto kern) { kern<<<n, kThreads, 0, st>>>(P); };
    const bool p2 = a.pow2 != 0;
    switch (a.dtype) {
        case LI_DTYPE_BF16: go(p2 ? cache_write_kernel<__nv_bfloat16, true> : cache_write_kernel<__nv_bfloat16, false>); break;
        case LI_DTYPE_FP16: go(p2 ? cache_write_kernel<__half, true> : cache_write_kernel<__half, false>); break;
        default: go(p2 ? cache_write_kernel<float, true> : cache_write_kernel<float, false>); break;
    }
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const li_cache_args &a, cudaStream_t st) {
    const CacheParams P = params(a);
    const unsigned n = blocks_of(P);
    switch (a.dtype) {
        case LI_DTYPE_BF16: cache_read_kernel<__nv_bfloat16><<<n, kThreads, 0, st>>>(P); break;
        case LI_DTYPE_FP16: cache_read_kernel<__half><<<n, kThreads, 0, st>>>(P); break;
        default: cache_read_kernel<float><<<n, kThreads, 0, st>>>(P); break;
    }
    return cudaGetLastError();
}

}  // namespace li
