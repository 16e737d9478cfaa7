// Quantised key cache (li_cache_write, li_cache_read), sm_100a.
//
// write: s = max(max_d |x_d| / 448, 2^-90) over the row's finite elements (1 for a row of zeros),
// or the smallest power of two that is no less; code_d = E4M3(x_d / s). read: code_d s in fp32,
// rounded once. Row i of batch b is key position L2_b - L1_b + i and goes through the block table.
//
// A row belongs to a group of lanes, eight elements a lane and step, and stays in registers between
// its maximum (a shuffle reduction) and its codes, so it is read from memory once. Bound by memory:
// 57344 rows of 512 + 64 bf16 values are written in 21.2 us
// (103 MB, 4.9 TB/s; at a copy's 6.5 TB/s 15.7), 53248 read back in 18.4 (96 MB, 5.2 TB/s). 32768 keys of
// 128 are written in 7.2 us (1.9): one wave of blocks, whose time is a row's chain of reads (its
// sequence, lengths, block) and some 10 instructions an element; 1120 rows are read in 3.2, most of
// it the launch.
#include <cuda_fp8.h>

#include "li_cache.cuh"
#include "li_fixed_div.cuh"
#include "li_float.cuh"

namespace li {
namespace {

constexpr int kThreads = 128;
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
    int64_t x_size, r_size, cache_rows;         // elements that x and rope span, rows of the cache
    int32_t rows, batch, x_len, k_len, num_blocks, block_size;
    int32_t dim, rope_dim;
    int32_t paged, lanes, lanes_log2;           // lanes per row
    FixedDiv by_len, by_block;                  // x_len, block_size
};

__device__ __forceinline__ void report(const CacheParams &P, uint32_t bits) {
    if (bits && P.status) atomicOr(P.status, bits);
}

// Packed rows: the last block has none of them and checks the sequences' ends instead, since a row's search
// sees only some of them. True in that block.
__device__ __forceinline__ bool checks_sequences(const CacheParams &P) {
    if (!P.cu_seqlens || blockIdx.x + 1 < gridDim.x) return false;
    uint32_t err = 0;
    for (int32_t b = threadIdx.x; b < P.batch; b += kThreads) {
        const int32_t c0 = __ldg(P.cu_seqlens + b), c1 = __ldg(P.cu_seqlens + b + 1);
        if (c0 < 0 || c1 < c0 || c1 > P.rows) err |= LI_DEVERR_LENGTHS;
    }
    report(P, err);
    return true;
}

// Element offset of row r of the call in x (or rope), by its strides.
__device__ __forceinline__ int64_t row_offset(const CacheParams &P, int32_t r, int64_t batch, int64_t row) {
    if (P.cu_seqlens) return (int64_t)r * row;
    const int32_t b = P.by_len.div(r);
    return b * batch + (r - b * P.x_len) * row;
}

// The packed sequences among which row r lies, [*lo, *hi): one of 32 ranges, found by the warp at once
// (its rows are neighbours, and 32 reads side by side take as long as one step of a search). All lanes
// call; rows outside the call get any. For the read, which waits for its place (1120 rows of 32
// sequences 3.2 us against 3.5); the write has its rows to read meanwhile, and the votes cost it more
// (32768 rows 7.6 against 7.0).
__device__ __forceinline__ void sequences_of(const CacheParams &P, int64_t r, int32_t *lo, int32_t *hi) {
    const int lane = threadIdx.x & 31, step = (P.batch + 31) / 32, at = (lane + 1) * step;
    const int32_t start = at < P.batch ? __ldg(P.cu_seqlens + at) : INT32_MAX;
    uint32_t below = 0;
    for (int k = 0; k < 32; k += P.lanes) {             // a row of the warp
        const int64_t row = __shfl_sync(0xffffffffu, r, k);
        const uint32_t v = __ballot_sync(0xffffffffu, start <= row);
        if (lane / P.lanes == k / P.lanes) below = v;
    }
    *lo = __popc(below) * step;
    *hi = min(*lo + step, P.batch);
}

// Whether row r of the call lies inside x and rope.
__device__ __forceinline__ bool row_ok(const CacheParams &P, int32_t r) {
    return run_ok(row_offset(P, r, P.x_batch, P.x_row), P.dim, P.x_size, P.status) &&
           (P.rope_dim == 0 || run_ok(row_offset(P, r, P.r_batch, P.r_row), P.rope_dim, P.r_size, P.status));
}

// Cache row of row r of the call (packed: of one of the sequences [lo, hi)), -1 where it takes no part:
// past the rows in use, or data that does not fit, which is added to *err.
__device__ __forceinline__ int64_t cache_row(const CacheParams &P, int32_t r, int32_t lo, int32_t hi, uint32_t *err) {
    int32_t b, i, L1;
    if (P.cu_seqlens) {
        const int32_t *cu = P.cu_seqlens;
        if (r < __ldg(cu) || r >= __ldg(cu + P.batch)) return -1;
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if (__ldg(cu + mid) <= r) lo = mid; else hi = mid;
        }
        b = lo;
        const int32_t first = __ldg(cu + b);
        i = r - first;
        L1 = __ldg(cu + b + 1) - first;
        if (i < 0 || i >= L1) {                 // only ends that decrease lead here
            *err |= LI_DEVERR_LENGTHS;
            return -1;
        }
    } else {
        b = P.by_len.div(r);
        i = r - b * P.x_len;
        L1 = P.x_len;
    }
    if (!idx_ok(b, (int64_t)P.batch + kBoundsSlack, P.status)) return -1;
    const int64_t cap = P.paged ? P.bt_stride * P.block_size : P.k_len;
    int64_t L2 = P.seqused_k ? __ldg(P.seqused_k + b) : P.k_len;
    if (L2 < 0 || L2 > cap) *err |= LI_DEVERR_LENGTHS;
    if (P.seqused) {
        const int32_t u = __ldg(P.seqused + b);
        if (u < 0 || u > L1) *err |= LI_DEVERR_LENGTHS;
        L1 = min(max(u, 0), L1);
    }
    const int64_t pos = L2 - L1 + i;
    if (i >= L1) return -1;
    if (pos < 0 || pos >= cap) {
        *err |= LI_DEVERR_LENGTHS;
        return -1;
    }
    if (!P.paged) return (int64_t)b * P.k_len + pos;
    const int32_t q = P.by_block.div((int32_t)pos);         // pos is below the int32 L2
    if (!idx_ok((int64_t)b * P.bt_stride + q, (int64_t)P.batch * P.bt_stride, P.status)) return -1;
    const int32_t blk = __ldg(P.block_table + (int64_t)b * P.bt_stride + q);
    if (blk < 0 || blk >= P.num_blocks) {
        *err |= LI_DEVERR_TABLE;
        return -1;
    }
    return (int64_t)blk * P.block_size + ((int32_t)pos - q * P.block_size);
}

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __int_as_float(0x7f800000); }

// x / s for the conversion to E4M3, which rounds it to nearest, ties to even: x * inv, inv = 1 / s,
// is within two units in the last place of the quotient, and that decides the code unless a border
// between two codes is as near. Of codes above 2^-6 a border has bit 19 of the mantissa as its last
// one; there, and below 2^-6, the quotient is rounded to odd instead (its last bit set when the
// division leaves a remainder), and the second rounding sees on which side it lies. Powers of two
// divide exactly.
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
        if (((__float_as_int(q) + 0x80004) & 0xfffff) < 8 || fabsf(q) < 0.015625f) return odd_quotient(x, s);
    }
    return q;
}

__device__ __forceinline__ float row_scale(float amax, bool pow2) {
    if (!(amax > 0.0f)) return 1.0f;
    if (!pow2) return fmaxf(__fdiv_rn(amax, 448.0f), kMinScale);
    // 448 = 1.75 x 2^8: the exponent of amax less 8, one more where its mantissa is above 1.75
    const int e = (__float_as_int(amax) + 0x1fffff) >> 23;
    return __int_as_float(max(e - 8, 127 - 90) << 23);
}

// Eight elements of T: one or two 16-byte accesses, or element by element.
template <class T> struct alignas(16) Eight { T v[8]; };
template <class T, bool kWide>
__device__ __forceinline__ void load8(Eight<T> &e, const T *p) {
    if constexpr (kWide) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            reinterpret_cast<uint4 *>(e.v)[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) e.v[i] = p[i];
    }
}
template <class T, bool kWide>
__device__ __forceinline__ void store8(T *p, const Eight<T> &e) {
    if constexpr (kWide) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(e.v)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = e.v[i];
    }
}

// max(m, |e|) over the eight elements, NaN left out (two 16-bit elements an instruction).
__device__ __forceinline__ void max8(__nv_bfloat162 &m, const Eight<__nv_bfloat16> &e) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) m = __hmax2(m, __habs2(__nv_bfloat162(e.v[i], e.v[i + 1])));
}
__device__ __forceinline__ void max8(__half2 &m, const Eight<__half> &e) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) m = __hmax2(m, __habs2(__half2(e.v[i], e.v[i + 1])));
}
__device__ __forceinline__ void max8(float &m, const Eight<float> &e) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(e.v[i]));
}
__device__ __forceinline__ float most(__nv_bfloat162 m) { return fmaxf(__low2float(m), __high2float(m)); }
__device__ __forceinline__ float most(__half2 m) { return fmaxf(__low2float(m), __high2float(m)); }
__device__ __forceinline__ float most(float m) { return m; }
template <class T> struct MaxOf { using type = float; };
template <> struct MaxOf<__nv_bfloat16> { using type = __nv_bfloat162; };
template <> struct MaxOf<__half> { using type = __half2; };

__device__ __forceinline__ float group_max(float m, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// A row per group of lanes; kSteps: steps of eight elements that a lane may take (dim <= 8 lanes
// kSteps). The row is read before its place in the cache is looked up.
template <class T, bool kWide, bool kPow2, int kSteps>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheParams P) {
    if (checks_sequences(P)) return;
    const int lane = threadIdx.x & (P.lanes - 1);
    const int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> P.lanes_log2;
    Eight<T> v[kSteps], rp;
    int64_t slot = -1;
    typename MaxOf<T>::type m2{};
    const T *rope = static_cast<const T *>(P.rope);
    if (r < P.rows && row_ok(P, (int32_t)r)) {
        const T *x = static_cast<const T *>(P.x) + row_offset(P, (int32_t)r, P.x_batch, P.x_row) + 8 * lane;
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
            if (8 * (lane + k * P.lanes) < P.dim) load8<T, kWide>(v[k], x + 8 * k * P.lanes);
        if (8 * lane < P.rope_dim) {
            rope += row_offset(P, (int32_t)r, P.r_batch, P.r_row) + 8 * lane;
            load8<T, kWide>(rp, rope);
        }
        uint32_t err = 0;
        slot = cache_row(P, (int32_t)r, 0, P.batch, &err);
        if (slot >= 0 && !idx_ok(slot, P.cache_rows, P.status)) slot = -1;
        report(P, err);
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
            if (8 * (lane + k * P.lanes) < P.dim) max8(m2, v[k]);
    }
    float amax = group_max(most(m2), P.lanes);
    // a row with an infinity: once more without it, and no code for it but NaN's
    const bool inf = !finite(amax);
    if (__any_sync(0xffffffffu, inf)) {
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
            if (inf && 8 * (lane + k * P.lanes) < P.dim)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float t = fabsf(to_f32(v[k].v[i]));
                    if (finite(t)) m = fmaxf(m, t);
                    else v[k].v[i] = from_f32<T>(__int_as_float(0x7fc00000));
                }
        m = group_max(m, P.lanes);
        if (inf) amax = m;
    }
    if (slot < 0) return;
    const float s = row_scale(amax, kPow2), inv = __frcp_rn(s);
    if (lane == 0) P.descale[slot] = s;
    uint8_t *codes = P.codes + slot * P.dim + 8 * lane;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        if (8 * (lane + k * P.lanes) >= P.dim) continue;
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[i] = __nv_cvt_float2_to_fp8x2(make_float2(quotient<kPow2>(to_f32(v[k].v[2 * i]), s, inv),
                                                        quotient<kPow2>(to_f32(v[k].v[2 * i + 1]), s, inv)),
                                            __NV_SATFINITE, __NV_E4M3);
        *reinterpret_cast<uint2 *>(codes + 8 * k * P.lanes) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    }
    if (8 * lane >= P.rope_dim) return;
    T *rc = reinterpret_cast<T *>(P.rope_cache) + slot * P.rope_dim + 8 * lane;
    store8<T, true>(rc, rp);
    for (int d = 8 * P.lanes; d + 8 * lane < P.rope_dim; d += 8 * P.lanes) {
        load8<T, kWide>(rp, rope + d);
        store8<T, true>(rc + d, rp);
    }
}

template <class T, bool kWide, int kSteps>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheParams P) {
    if (checks_sequences(P)) return;
    const int lane = threadIdx.x & (P.lanes - 1);
    const int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> P.lanes_log2;
    int32_t lo = 0, hi = 0;
    if (P.cu_seqlens) sequences_of(P, r, &lo, &hi);
    if (r >= P.rows) return;
    uint32_t err = 0;
    const int64_t slot = cache_row(P, (int32_t)r, lo, hi, &err);
    report(P, err);
    if (slot < 0 || !idx_ok(slot, P.cache_rows, P.status) || !row_ok(P, (int32_t)r)) return;
    const float s = __ldg(P.descale + slot);
    const uint8_t *codes = P.codes + slot * P.dim + 8 * lane;
    const T *rc = reinterpret_cast<const T *>(P.rope_cache) + slot * P.rope_dim + 8 * lane;
    uint2 c[kSteps];
    Eight<T> rp;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
        if (8 * (lane + k * P.lanes) < P.dim) c[k] = __ldcs(reinterpret_cast<const uint2 *>(codes + 8 * k * P.lanes));
    if (8 * lane < P.rope_dim) load8<T, true>(rp, rc);
    T *x = static_cast<T *>(P.x) + row_offset(P, (int32_t)r, P.x_batch, P.x_row) + 8 * lane;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        if (8 * (lane + k * P.lanes) >= P.dim) continue;
        Eight<T> e;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = (i < 2 ? c[k].x : c[k].y) >> (16 * (i & 1)) & 0xffffu;
            const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3)));
            e.v[2 * i] = from_f32<T>(f.x * s);
            e.v[2 * i + 1] = from_f32<T>(f.y * s);
        }
        store8<T, kWide>(x + 8 * k * P.lanes, e);
    }
    if (8 * lane >= P.rope_dim) return;
    T *rope = static_cast<T *>(P.rope) + row_offset(P, (int32_t)r, P.r_batch, P.r_row) + 8 * lane;
    store8<T, kWide>(rope, rp);
    for (int d = 8 * P.lanes; d + 8 * lane < P.rope_dim; d += 8 * P.lanes) {
        load8<T, true>(rp, rc + d);
        store8<T, kWide>(rope + d, rp);
    }
}

// Elements of a lane, at most (dim allowing). A row's address work is shared by them, and the kernels
// are bound by instructions when there are many rows: 32 rather than 16 write 57344 rows of 512 in 21.2 us
// against 27.4, read 53248 in 18.4 against 21.6 and write 32768 of 128 in 7.2 against 7.8. Where the
// elements do not fill the SMs' threads at 8 a thread, more threads hide more latency: 1120 rows of 128
// read in 3.2 us against 3.6, 64 of 512 written in 2.5 against 2.6. (Blocks of 256 threads: 0.1 to 0.2 us more.)
int per_lane(int64_t rows, int dim) { return rows * dim > (int64_t)device_sm_count() * 2048 * 8 ? 32 : 16; }

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
    const int64_t outer = P.cu_seqlens ? 0 : a.batch - 1;
    P.x_size = outer * a.x_batch_stride + (a.x_len - 1) * a.x_row_stride + a.dim;
    P.r_size = outer * a.rope_batch_stride + (a.x_len - 1) * a.rope_row_stride + a.rope_dim;
    P.cache_rows = a.layout_k == LI_LAYOUT_PA_BSND ? (int64_t)a.num_blocks * a.block_size : (int64_t)a.batch * a.k_len;
    P.rows = P.cu_seqlens ? a.x_len : a.batch * a.x_len;
    P.batch = a.batch;
    P.x_len = a.x_len;
    P.k_len = a.k_len;
    P.num_blocks = a.num_blocks;
    P.block_size = a.block_size;
    P.dim = a.dim;
    P.rope_dim = a.rope_dim;
    P.paged = a.layout_k == LI_LAYOUT_PA_BSND;
    P.lanes_log2 = 0;
    while (P.lanes_log2 < 5 && (per_lane(P.rows, a.dim) << P.lanes_log2) < a.dim) ++P.lanes_log2;
    P.lanes = 1 << P.lanes_log2;
    P.by_len = FixedDiv(a.x_len);
    P.by_block = FixedDiv(P.paged ? a.block_size : 1);
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
    return (unsigned)(((int64_t)P.rows * P.lanes + kThreads - 1) / kThreads + (P.cu_seqlens ? 1 : 0));
}

template <class T, bool kWide, bool kPow2>
void write_steps(const CacheParams &P, cudaStream_t st) {
    if (P.dim <= 16 * P.lanes) cache_write_kernel<T, kWide, kPow2, 2><<<blocks_of(P), kThreads, 0, st>>>(P);
    else cache_write_kernel<T, kWide, kPow2, 4><<<blocks_of(P), kThreads, 0, st>>>(P);
}
template <class T>
void write_type(const CacheParams &P, bool wide, bool pow2, cudaStream_t st) {
    if (wide) pow2 ? write_steps<T, true, true>(P, st) : write_steps<T, true, false>(P, st);
    else pow2 ? write_steps<T, false, true>(P, st) : write_steps<T, false, false>(P, st);
}
template <class T, bool kWide>
void read_steps(const CacheParams &P, cudaStream_t st) {
    if (P.dim <= 16 * P.lanes) cache_read_kernel<T, kWide, 2><<<blocks_of(P), kThreads, 0, st>>>(P);
    else cache_read_kernel<T, kWide, 4><<<blocks_of(P), kThreads, 0, st>>>(P);
}
template <class T>
void read_type(const CacheParams &P, bool wide, cudaStream_t st) {
    if (wide) read_steps<T, true>(P, st);
    else read_steps<T, false>(P, st);
}

}  // namespace

cudaError_t launch_cache_write(const li_cache_args &a, cudaStream_t st) {
    const CacheParams P = params(a);
    const bool wide = wide_rows(a), pow2 = a.pow2 != 0;
    if (a.dtype == LI_DTYPE_BF16) write_type<__nv_bfloat16>(P, wide, pow2, st);
    else if (a.dtype == LI_DTYPE_FP16) write_type<__half>(P, wide, pow2, st);
    else write_type<float>(P, wide, pow2, st);
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const li_cache_args &a, cudaStream_t st) {
    const CacheParams P = params(a);
    const bool wide = wide_rows(a);
    if (a.dtype == LI_DTYPE_BF16) read_type<__nv_bfloat16>(P, wide, st);
    else if (a.dtype == LI_DTYPE_FP16) read_type<__half>(P, wide, st);
    else read_type<float>(P, wide, st);
    return cudaGetLastError();
}

}  // namespace li
