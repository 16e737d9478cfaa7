// Quantised key cache (li_cache_write, li_cache_read), sm_100a.
//
// write: s = max(max_d |x_d| / 448, 2^-90) over the row's finite elements (1 for a row of zeros),
// or the smallest power of two that is no less; code_d = E4M3(x_d / s). read: code_d s in fp32,
// rounded once. Row i of batch b is key position L2_b - L1_b + i and goes through the block table.
//
// A row belongs to a group of lanes, eight elements a lane and step, and stays in registers between
// its maximum (a shuffle reduction) and its codes, so it is read from memory once. Bound by memory:
// %FIG%
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
    int32_t paged, lanes, lanes_log2;           // lanes per row
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
        const int32_t q = (int32_t)pos / P.block_size;         // below the int32 L2
        const int32_t blk = P.block_table[(int64_t)b * P.bt_stride + q];
        if (blk < 0 || blk >= P.num_blocks) {
            err |= LI_DEVERR_TABLE;
            take = false;
        }
        out->slot = (int64_t)blk * P.block_size + ((int32_t)pos - q * P.block_size);
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

// E4M3 codes of the exact quotients a / s and b / s; inv = 1 / s. a * inv is within two units in the
// last place of the quotient, which decides the code unless it lies that near to a border between
// two codes. Borders have at most 5 significant bits, so the 19 lowest mantissa bits tell; there
// the quotient is rounded to odd instead (its last bit set when the division leaves a remainder),
// and the second rounding sees on which side it lies. Powers of two divide exactly.
__device__ __noinline__ float odd_quotient(float x, float s) {
    const float q = __fdiv_rn(x, s);
    const float rem = fmaf(-q, s, x);
    if (rem == 0.0f || !finite(q)) return q;
    int bits = __float_as_int(q);
    if ((rem < 0.0f) != (x < 0.0f)) bits -= 1;          // the quotient was rounded away from zero
    return __int_as_float(bits | 1);
}
template <bool kPow2>
__device__ __forceinline__ float quotient(float x, float s, float inv) {
    const float q = x * inv;
    if constexpr (!kPow2) {
        if (((__float_as_int(q) + 4) & 0x7ffff) < 8) return odd_quotient(x, s);
    }
    return q;
}
// NaN stays NaN; an infinity has no code either.
__device__ __forceinline__ float coded(float x, float q) { return finite(x) ? q : __int_as_float(0x7fc00000); }

__device__ __forceinline__ float row_scale(float amax, bool pow2) {
    if (!(amax > 0.0f)) return 1.0f;
    if (!pow2) return fmaxf(__fdiv_rn(amax, 448.0f), kMinScale);
    // 448 = 1.75 x 2^8: the exponent of amax less 8, one more where its mantissa is above 1.75
    const int e = (__float_as_int(amax) + 0x1fffff) >> 23;
    return __int_as_float(max(e - 8, 127 - 90) << 23);
}

// Eight elements of T in one or two 16-byte accesses, or element by element.
template <class T, bool kWide>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    if constexpr (!kWide) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(p[i]);
    } else {
        T t[8];
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            reinterpret_cast<uint4 *>(t)[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(t[i]);
    }
}
template <class T, bool kWide>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    if constexpr (!kWide) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = from_f32<T>(v[i]);
    } else {
        T t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = from_f32<T>(v[i]);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(t)[i];
    }
}
// The rope part of a row: eight elements a lane and step (rope_dim is a multiple of eight).
template <class T, bool kWide>
__device__ __forceinline__ void copy_row(T *to, const T *from, int n, int lane, int lanes) {
    for (int d = 8 * lane; d < n; d += 8 * lanes) {
        float v[8];
        load8<T, kWide>(from + d, v);
        store8<T, kWide>(to + d, v);
    }
}

// kSteps: steps of eight elements that a lane may take (dim <= 8 lanes kSteps).
template <class T, bool kWide, bool kPow2, int kSteps>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheParams P) {
    const int lane = threadIdx.x & (P.lanes - 1);
    const int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> P.lanes_log2;
    Place at;
    const bool take = r < P.rows && place_row(P, (int32_t)r, &at);
    float v[kSteps][8];
    float amax = 0.0f;
    if (take) {
        const T *x = static_cast<const T *>(P.x) + at.x_off;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int d = 8 * (lane + k * P.lanes);
            if (d < P.dim) load8<T, kWide>(x + d, v[k]);
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
            if (8 * (lane + k * P.lanes) < P.dim)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (finite(v[k][i])) amax = fmaxf(amax, fabsf(v[k][i]));
    }
    for (int o = P.lanes / 2; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!take) return;
    const float s = row_scale(amax, kPow2), inv = __frcp_rn(s);
    if (lane == 0) P.descale[at.slot] = s;
    uint8_t *codes = P.codes + at.slot * P.dim;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const int d = 8 * (lane + k * P.lanes);
        if (d >= P.dim) continue;
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = v[k][2 * i], b = v[k][2 * i + 1];
            c[i] = __nv_cvt_float2_to_fp8x2(make_float2(coded(a, quotient<kPow2>(a, s, inv)), coded(b, quotient<kPow2>(b, s, inv))),
                                            __NV_SATFINITE, __NV_E4M3);
        }
        *reinterpret_cast<uint2 *>(codes + d) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    }
    if (P.rope_dim > 0)
        copy_row<T, kWide>(reinterpret_cast<T *>(P.rope_cache) + at.slot * P.rope_dim,
                           static_cast<const T *>(P.rope) + at.r_off, P.rope_dim, lane, P.lanes);
}

template <class T, bool kWide>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheParams P) {
    const int lane = threadIdx.x & (P.lanes - 1);
    const int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> P.lanes_log2;
    Place at;
    if (r >= P.rows || !place_row(P, (int32_t)r, &at)) return;
    T *x = static_cast<T *>(P.x) + at.x_off;
    const uint8_t *codes = P.codes + at.slot * P.dim;
    const float s = P.descale[at.slot];
    for (int d = 8 * lane; d < P.dim; d += 8 * P.lanes) {
        const uint2 c = *reinterpret_cast<const uint2 *>(codes + d);
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = (i < 2 ? c.x : c.y) >> (16 * (i & 1)) & 0xffffu;
            const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3)));
            v[2 * i] = f.x * s;
            v[2 * i + 1] = f.y * s;
        }
        store8<T, kWide>(x + d, v);
    }
    if (P.rope_dim > 0)
        copy_row<T, kWide>(static_cast<T *>(P.rope) + at.r_off,
                           reinterpret_cast<const T *>(P.rope_cache) + at.slot * P.rope_dim, P.rope_dim,
                           lane, P.lanes);
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
    P.lanes_log2 = 1;
    while (P.lanes_log2 < 5 && (8 << P.lanes_log2) < a.dim) ++P.lanes_log2;
    P.lanes = 1 << P.lanes_log2;
    return P;
}

// Rows in 16-byte accesses: x and rope start on 16 bytes and so does every row (the cache always).
bool wide_rows(const li_cache_args &a) {
    const int64_t e = a.dtype == LI_DTYPE_FP32 ? 4 : 2;
    const auto whole = [&](const void *p, int64_t row, int64_t batch) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row * e % 16 == 0 &&
               (a.layout_x == LI_LAYOUT_TND || batch * e % 16 == 0);
    };
    return whole(a.x, a.x_row_stride, a.x_batch_stride) &&
           (a.rope_dim == 0 || whole(a.rope, a.rope_row_stride, a.rope_batch_stride));
}

unsigned blocks_of(const CacheParams &P) {
    return (unsigned)(((int64_t)P.rows * P.lanes + kThreads - 1) / kThreads);
}

}  // namespace

namespace {

template <class T, bool kWide, bool kPow2>
void write_steps(const CacheParams &P, unsigned n, cudaStream_t st) {
    const int steps = (P.dim + 8 * P.lanes - 1) / (8 * P.lanes);
    if (steps == 1) cache_write_kernel<T, kWide, kPow2, 1><<<n, kThreads, 0, st>>>(P);
    else if (steps == 2) cache_write_kernel<T, kWide, kPow2, 2><<<n, kThreads, 0, st>>>(P);
    else cache_write_kernel<T, kWide, kPow2, 4><<<n, kThreads, 0, st>>>(P);
}
template <class T>
void write_type(const CacheParams &P, bool wide, bool pow2, unsigned n, cudaStream_t st) {
    if (wide) pow2 ? write_steps<T, true, true>(P, n, st) : write_steps<T, true, false>(P, n, st);
    else pow2 ? write_steps<T, false, true>(P, n, st) : write_steps<T, false, false>(P, n, st);
}
template <class T>
void read_type(const CacheParams &P, bool wide, unsigned n, cudaStream_t st) {
    if (wide) cache_read_kernel<T, true><<<n, kThreads, 0, st>>>(P);
    else cache_read_kernel<T, false><<<n, kThreads, 0, st>>>(P);
}

}  // namespace

cudaError_t launch_cache_write(const li_cache_args &a, cudaStream_t st) {
    const CacheParams P = params(a);
    const bool wide = wide_rows(a), pow2 = a.pow2 != 0;
    if (a.dtype == LI_DTYPE_BF16) write_type<__nv_bfloat16>(P, wide, pow2, blocks_of(P), st);
    else if (a.dtype == LI_DTYPE_FP16) write_type<__half>(P, wide, pow2, blocks_of(P), st);
    else write_type<float>(P, wide, pow2, blocks_of(P), st);
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const li_cache_args &a, cudaStream_t st) {
    const CacheParams P = params(a);
    const bool wide = wide_rows(a);
    if (a.dtype == LI_DTYPE_BF16) read_type<__nv_bfloat16>(P, wide, blocks_of(P), st);
    else if (a.dtype == LI_DTYPE_FP16) read_type<__half>(P, wide, blocks_of(P), st);
    else read_type<float>(P, wide, blocks_of(P), st);
    return cudaGetLastError();
}

}  // namespace li
