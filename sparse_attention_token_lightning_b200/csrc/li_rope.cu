// Rotary positions (li_rope) and their gradient (li_rope_grad), sm_100a.
//
// For a row at position p and pair i of every head, a = p freq[i]:
//     y[u] = m (x[u] cos a - x[v] sin a),    y[v] = m (x[u] sin a + x[v] cos a)
// (the gradient: sin a with the other sign); the head's other elements are copied when y is not x.
//
// A block takes a few rows: its threads first put m cos a and m sin a of every (row, pair) into
// shared memory, then run over the rows' heads. The angle is reduced in double (p freq in turns,
// less its nearest integer) and only the remainder, at most half a turn, goes through fp32, so a
// position of 2^20 is as accurate as position 1; a table per row instead of a table of all
// positions costs no memory traffic and no limit on positions.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "li_rope.cuh"

namespace li {
namespace {

constexpr int kThreads = 256;

struct RopeParams {
    const void *x;
    void *y;
    const void *positions;
    int64_t x_row, x_head, y_row, y_head;
    int32_t rows, heads, head_dim, pairs, offset;
    int32_t rows_per_block;
    int32_t copy;                       // elements outside the rotated part are copied
    int32_t pos64;
    float magnitude, sign;              // sign of sin: -1 for the gradient
    double turns[LI_ROPE_MAX_PAIRS];    // freq / 2 pi
};

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f32(float v) { return v; }

template <class T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams P) {
    extern __shared__ float2 cs[];      // [rows_per_block][pairs]: m cos a, m sin a
    const int32_t row0 = (int32_t)blockIdx.x * P.rows_per_block;
    const int nrow = min(P.rows_per_block, P.rows - row0);
    for (int t = threadIdx.x; t < nrow * P.pairs; t += kThreads) {
        const int r = t / P.pairs, i = t - r * P.pairs;
        const double p = P.pos64 ? (double)static_cast<const int64_t *>(P.positions)[row0 + r]
                                 : (double)static_cast<const int32_t *>(P.positions)[row0 + r];
        const double turns = p * P.turns[i];
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        cs[t] = make_float2(P.magnitude * c, P.magnitude * P.sign * s);
    }
    __syncthreads();
    const T *x = static_cast<const T *>(P.x);
    T *y = static_cast<T *>(P.y);
    const int per_head = P.copy ? P.head_dim - P.pairs : P.pairs;      // pairs, then single copies
    const int64_t items = (int64_t)nrow * P.heads * per_head;
    for (int64_t t = threadIdx.x; t < items; t += kThreads) {
        const int rh = (int)(t / per_head), e = (int)(t - (int64_t)rh * per_head);
        const int r = rh / P.heads, h = rh - r * P.heads;
        const T *xh = x + (row0 + r) * P.x_row + h * P.x_head;
        T *yh = y + (row0 + r) * P.y_row + h * P.y_head;
        if (e < P.pairs) {
            const int u = P.offset + (kInterleaved ? 2 * e : e), v = u + (kInterleaved ? 1 : P.pairs);
            const float2 a = cs[r * P.pairs + e];
            const float xu = to_f32(xh[u]), xv = to_f32(xh[v]);
            yh[u] = from_f32<T>(xu * a.x - xv * a.y);
            yh[v] = from_f32<T>(xu * a.y + xv * a.x);
        } else {
            int d = e - P.pairs;
            if (d >= P.offset) d += 2 * P.pairs;
            yh[d] = xh[d];
        }
    }
}

template <class T>
cudaError_t launch_type(const RopeParams &P, bool interleaved, cudaStream_t st) {
    const int64_t blocks = ((int64_t)P.rows + P.rows_per_block - 1) / P.rows_per_block;
    const size_t smem = (size_t)P.rows_per_block * P.pairs * sizeof(float2);
    auto kern = interleaved ? rope_kernel<T, true> : rope_kernel<T, false>;
    kern<<<(unsigned)blocks, kThreads, smem, st>>>(P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const li_rope_args &a, bool grad, cudaStream_t st) {
    RopeParams P{};
    P.x = a.x;
    P.y = a.y;
    P.positions = a.positions;
    P.x_row = a.x_row_stride;
    P.x_head = a.x_head_stride;
    P.y_row = a.y_row_stride;
    P.y_head = a.y_head_stride;
    P.rows = (int32_t)a.rows;
    P.heads = a.heads;
    P.head_dim = a.head_dim;
    P.pairs = a.rope_dim / 2;
    P.offset = a.rope_offset;
    P.copy = a.x != a.y;
    P.pos64 = a.position_bits == 64;
    P.magnitude = a.magnitude;
    P.sign = grad ? -1.0f : 1.0f;
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    for (int i = 0; i < P.pairs; ++i) P.turns[i] = a.freq[i] / kTwoPi;
    // about 4096 elements a block, at most 32 rows (a table of 32 KB at 128 pairs)
    const int64_t row_elems = (int64_t)a.heads * (P.copy ? a.head_dim : a.rope_dim);
    int r = (int)((4096 + row_elems - 1) / row_elems);
    P.rows_per_block = r < 1 ? 1 : r > 32 ? 32 : r;
    switch (a.dtype) {
        case LI_DTYPE_BF16: return launch_type<__nv_bfloat16>(P, a.interleaved != 0, st);
        case LI_DTYPE_FP16: return launch_type<__half>(P, a.interleaved != 0, st);
        default: return launch_type<float>(P, a.interleaved != 0, st);
    }
}

}  // namespace li
