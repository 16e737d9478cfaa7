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
#include "li_float.cuh"
#include "li_rope.cuh"

namespace li {
namespace {

constexpr int kThreads = 256;

// t / d by one multiplication where every t d < 2^32, by a division elsewhere.
struct FastDiv {
    uint32_t d = 1, m = 0;              // m = ceil(2^32 / d), 0: divide
    __host__ FastDiv() {}
    __host__ FastDiv(uint32_t d_, int64_t most)
        : d(d_), m(d_ > 1 && most * d_ < ((int64_t)1 << 32) ? 0xffffffffu / d_ + 1 : 0) {}
    __device__ __forceinline__ uint32_t div(uint32_t t) const { return m ? __umulhi(t, m) : t / d; }
};

struct RopeParams {
    const void *x;
    void *y;
    const void *positions;
    int64_t x_row, x_head, y_row, y_head;
    int64_t x_size, y_size;             // elements that they span
    int32_t rows, heads, head_dim, pairs, offset;
    int32_t rows_per_block;
    int32_t rotated, copies;            // items of a head
    int32_t u_step, v_step;             // pair items: u = offset + e u_step, v = u + v_step
    FastDiv by_rotated, by_copies, by_heads;
    int32_t pos64;
    float magnitude, sign;              // sign of sin: -1 for the gradient
    double turns[LI_ROPE_MAX_PAIRS];    // freq / 2 pi
};

// kVec elements of T in one access.
template <class T, int kVec> struct alignas(sizeof(T) * kVec) Vec { T v[kVec]; };

// Whether an access of kVec elements at `from` of x and `to` of y lies inside them. There is no status word
// here: the bounds-checked build leaves the access out.
template <int kVec> __device__ __forceinline__ bool access_ok(const RopeParams &P, int64_t from, int64_t to) {
    return run_ok(from, kVec, P.x_size, nullptr) && run_ok(to, kVec, P.y_size, nullptr);
}

// Item t of the block's rows: element offsets of its access in x and y, its row and item in the head.
struct Place {
    int64_t from, to;
    uint32_t r, e;
};
__device__ __forceinline__ Place place(const RopeParams &P, int32_t row0, uint32_t t, const FastDiv &by_items) {
    Place p;
    const uint32_t rh = by_items.div(t);
    p.e = t - rh * by_items.d;
    p.r = P.by_heads.div(rh);
    const uint32_t h = rh - p.r * P.heads;
    const int64_t row = row0 + (int64_t)p.r;
    p.from = row * P.x_row + h * P.x_head;
    p.to = row * P.y_row + h * P.y_head;
    return p;
}

// An item is one access of kVec elements to read and write: a copy, kVec / 2 whole pairs (kPairs
// false: the interleaved layout in wide accesses) or, with kPairs, two accesses that hold the u
// and the v elements of kVec pairs (the half layout, and every layout element by element). Copies
// and rotated items run in loops of their own, so that no warp holds both.
//
// Bound by memory: 4096 x 64 heads of 128 bf16 dims, 64 of them rotated in the half layout, take
// 24.6 us (5.4 TB/s; mixed in one loop 36.8), 2999 x 16 heads of 576 fp32 dims 35.6 us (6.2 TB/s).
// The half layout wants threads rather than accesses in flight: eight blocks an SM with one pair
// item a thread at a time; two or four items, or fewer blocks, take 28 to 58 us.
template <class T, int kVec, bool kPairs>
__global__ void __launch_bounds__(kThreads, kPairs ? 8 : 6) rope_kernel(const __grid_constant__ RopeParams P) {
    constexpr int kItems = kPairs ? 1 : 4;              // rotated items of a thread in flight
    using V = Vec<T, kVec>;
    extern __shared__ __align__(16) float2 cs[];        // [rows_per_block][pairs]: m cos a, m sin a
    const int32_t row0 = (int32_t)blockIdx.x * P.rows_per_block;
    const int nrow = min(P.rows_per_block, P.rows - row0);
    const T *x = static_cast<const T *>(P.x);
    T *y = static_cast<T *>(P.y);
    for (int t = threadIdx.x; t < nrow * P.pairs; t += kThreads) {
        const int r = t / P.pairs, i = t - r * P.pairs;
        const double p = P.pos64 ? (double)static_cast<const int64_t *>(P.positions)[row0 + r]
                                 : (double)static_cast<const int32_t *>(P.positions)[row0 + r];
        const double turns = p * P.turns[i];
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        cs[t] = make_float2(P.magnitude * c, P.magnitude * P.sign * s);
    }
    const uint32_t copies = (uint32_t)nrow * P.heads * P.copies;
    for (uint32_t t0 = threadIdx.x; t0 < copies; t0 += kThreads * 4) {
        V a[4];
        int64_t to[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t t = t0 + k * kThreads;
            if (t >= copies) continue;
            const Place p = place(P, row0, t, P.by_copies);
            int d = p.e * kVec;
            if (d >= P.offset) d += 2 * P.pairs;
            to[k] = p.to + d;
            if (!access_ok<kVec>(P, p.from + d, to[k])) {
                to[k] = -1;
                continue;
            }
            a[k] = *reinterpret_cast<const V *>(x + p.from + d);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (t0 + k * kThreads < copies && (!kDebugBounds || to[k] >= 0)) *reinterpret_cast<V *>(y + to[k]) = a[k];
    }
    __syncthreads();
    const uint32_t items = (uint32_t)nrow * P.heads * P.rotated;
    for (uint32_t t0 = threadIdx.x; t0 < items; t0 += kThreads * kItems) {
        V a[kItems], b[kItems];
        int64_t to[kItems];
        int angle[kItems];                              // first entry in cs
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const uint32_t t = t0 + k * kThreads;
            if (t >= items) continue;
            const Place p = place(P, row0, t, P.by_rotated);
            const int d = P.offset + p.e * P.u_step;
            angle[k] = p.r * P.pairs + p.e * (kPairs ? kVec : kVec / 2);
            to[k] = p.to + d;
            if (!access_ok<kVec>(P, p.from + d, to[k]) ||
                (kPairs && !access_ok<kVec>(P, p.from + d + P.v_step, to[k] + P.v_step)) ||
                !run_ok(angle[k], kPairs ? kVec : kVec / 2, (int64_t)P.rows_per_block * P.pairs + kBoundsSlack, nullptr)) {
                to[k] = -1;
                continue;
            }
            a[k] = *reinterpret_cast<const V *>(x + p.from + d);
            if (kPairs) b[k] = *reinterpret_cast<const V *>(x + p.from + d + P.v_step);
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (t0 + k * kThreads >= items || (kDebugBounds && to[k] < 0)) continue;
            const float2 *ang = cs + angle[k];
            if constexpr (kPairs) {
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float2 w = ang[i];
                    const float u = to_f32(a[k].v[i]), v = to_f32(b[k].v[i]);
                    a[k].v[i] = from_f32<T>(u * w.x - v * w.y);
                    b[k].v[i] = from_f32<T>(u * w.y + v * w.x);
                }
                *reinterpret_cast<V *>(y + to[k] + P.v_step) = b[k];
            } else {
#pragma unroll
                for (int i = 0; i < kVec / 2; ++i) {
                    const float2 w = ang[i];
                    const float u = to_f32(a[k].v[2 * i]), v = to_f32(a[k].v[2 * i + 1]);
                    a[k].v[2 * i] = from_f32<T>(u * w.x - v * w.y);
                    a[k].v[2 * i + 1] = from_f32<T>(u * w.y + v * w.x);
                }
            }
            *reinterpret_cast<V *>(y + to[k]) = a[k];
        }
    }
}

template <class T, int kVec, bool kPairs>
cudaError_t launch(RopeParams &P, bool interleaved, bool in_place, cudaStream_t st) {
    P.rotated = kPairs ? P.pairs / kVec : 2 * P.pairs / kVec;
    P.copies = in_place ? 0 : (P.head_dim - 2 * P.pairs) / kVec;
    P.u_step = kPairs && interleaved ? 2 : kVec;
    P.v_step = interleaved ? 1 : P.pairs;
    // about 2048 accesses a block, so that the angles of a row are shared by its heads and several
    // blocks fit an SM; at most 32 rows (a table of 32 KB at 128 pairs), and fewer where that would
    // leave SMs without a block (64 rows of 16 heads: 2.6 us, 5.7 with 16 rows a block)
    const int64_t row_items = (int64_t)P.heads * (P.rotated * (kPairs ? 2 : 1) + P.copies);
    const int64_t spread = P.rows / device_sm_count();
    int64_t r = 2048 / row_items;
    r = r < spread ? r : spread;
    P.rows_per_block = (int)(r < 1 ? 1 : r > 32 ? 32 : r);
    const int64_t heads = (int64_t)P.rows_per_block * P.heads;
    P.by_rotated = FastDiv(P.rotated, heads * P.rotated);
    P.by_copies = FastDiv(P.copies > 0 ? P.copies : 1, heads * P.copies);
    P.by_heads = FastDiv(P.heads, heads);
    const int64_t blocks = ((int64_t)P.rows + P.rows_per_block - 1) / P.rows_per_block;
    const size_t smem = (size_t)P.rows_per_block * P.pairs * sizeof(float2);
    rope_kernel<T, kVec, kPairs><<<(unsigned)blocks, kThreads, smem, st>>>(P);
    return cudaGetLastError();
}

template <class T>
cudaError_t launch_type(RopeParams &P, bool interleaved, bool in_place, cudaStream_t st) {
    constexpr int kVec = 16 / sizeof(T);
    // 16-byte accesses where every one of them is aligned and whole
    const auto whole = [](int64_t n) { return n % kVec == 0; };
    const bool wide = reinterpret_cast<uintptr_t>(P.x) % 16 == 0 && reinterpret_cast<uintptr_t>(P.y) % 16 == 0 &&
                      whole(P.x_row) && whole(P.x_head) && whole(P.y_row) && whole(P.y_head) &&
                      whole(P.offset) && whole(P.head_dim) && whole(interleaved ? 2 * P.pairs : P.pairs);
    if (!wide) return launch<T, 1, true>(P, interleaved, in_place, st);
    return interleaved ? launch<T, kVec, false>(P, true, in_place, st)
                       : launch<T, kVec, true>(P, false, in_place, st);
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
    P.x_size = (a.rows - 1) * P.x_row + (a.heads - 1) * P.x_head + a.head_dim;
    P.y_size = (a.rows - 1) * P.y_row + (a.heads - 1) * P.y_head + a.head_dim;
    P.rows = (int32_t)a.rows;
    P.heads = a.heads;
    P.head_dim = a.head_dim;
    P.pairs = a.rope_dim / 2;
    P.offset = a.rope_offset;
    P.pos64 = a.position_bits == 64;
    P.magnitude = a.magnitude;
    P.sign = grad ? -1.0f : 1.0f;
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    for (int i = 0; i < P.pairs; ++i) P.turns[i] = a.freq[i] / kTwoPi;
    switch (a.dtype) {
        case LI_DTYPE_BF16: return launch_type<__nv_bfloat16>(P, a.interleaved != 0, a.x == a.y, st);
        case LI_DTYPE_FP16: return launch_type<__half>(P, a.interleaved != 0, a.x == a.y, st);
        default: return launch_type<float>(P, a.interleaved != 0, a.x == a.y, st);
    }
}

}  // namespace li
