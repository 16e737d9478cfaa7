// Attention over the selected rows of an E4M3 key cache (li_cache_attention), sm_100a.
//
// Query row r of batch b, head g, selected cache rows s with codes c_s and scale d_s (k_s = d_s c_s):
//     x[s]   = scale (d_s q.c_s + q_rope.k_rope_s),   o = sum_s e^x[s] d_s c_s / sum_s e^x[s]
//
// The codes go to the tensor cores as they lie in the cache: no key is converted. What multiplies
// them is split into E4M3 parts instead, whose products with the codes and sums in fp32 are exact
// to fp32 rounding:
//   q       times a power of two per head (largest element in [128, 256)) = hi + lo / 16, hi and
//           lo in E4M3: 8 bits in 4 + 4, so every bf16 element down to 2^-13 of the row's largest
//           is held exactly (and none is off by more than 2^-21 of it)
//   weights with y = x log2(e) + log2(d_s), 2^(y - ref) = hi + lo / 16 likewise (9 bits by way of
//           fp16's 11: 1.25 x 2^-9, less than a bf16 weight's 2^-8). The reference follows the
//           largest y, not the largest x, so the scale is inside the exponent and the parts are
//           full where the products are large; the normaliser sums 2^(x log2(e) - ref) in fp32, whose
//           largest terms are normal numbers for every scale in [2^-100, 2^100].
// The products S = K Q^T (keys on M = 128, hi and lo heads on N) and O^T += V^T P^T (dims on M = 128,
// the key tile read MN-major, keys on K) both read the same gathered tile; the rope part is a bf16
// product of its own into other TMEM columns, since its codes have no scale.
//
// One CTA per SM works in turn on units: a row, a block of up to 32 heads, and its tiles of 128 selected
// keys. When there are few rows (decode) a cluster of two, four or eight CTAs shares each unit's tiles,
// and joins its partial outputs through distributed shared memory (cache_attn_plan says when). Warps:
//   softmax   two groups of 4 warps, each with half the heads: a thread owns one key of the tile and
//             8 or 16 heads. The largest weight is set to 2^7 and may grow to 2^8.75 (E4M3 holds 448)
//             before the reference moves; a vote per tile finds that out, and only then are the
//             maxima reduced and O rescaled. Weights below 2^-21 of the largest may round to 0
//   prep      the next unit's q: normalised, split and stored in the MMA layout
//   lookup    each selected key's cache row for the gather and its scale for the softmax warps, a few
//             tiles ahead, and how many tiles a unit has
//   gather    copies codes and rope part with cp.async into 16 KB slots (128 keys x 128 bytes,
//             128-byte swizzle); rows that select nothing are zero-filled
//   qk, pv    one thread each issues the two products
// Measured (576 values a key, 16 heads; graph replay on one B200): 64 sequences x 2048 keys 25.9 to 28.0 us
// by machine (85 MB of selected rows, 3.3 TB/s at best; what memory alone takes is 13.3), one sequence 13.0, causal
// 2048 tokens x 1024 keys 179 us (1.05 GB out of L2, 5.9 TB/s), 21 rows x 777 keys x 128 heads of 256 21
// us, 64 rows x 2048 keys x 128 heads 83.
// A tile then costs a CTA some 3900 cycles, of which no unit is full: the gather alone takes 2140 (38
// bytes a cycle and SM, for 16 SMs as for 148), the operands of the products 150 KB of shared memory
// (1500 cycles), a softmax from scores to weights 2000. More overlap did not help (figures of the builds in
// which it was tried, each against the build before it): with tiles of 64 keys the 2048 tokens took 247 us
// where these took 205, with twice the softmax warps on alternate tiles 209 against 184, with eight gather
// warps 183, with TMA's gather for two of five slots more than either. Shorter code did: the roles' code
// shares the instruction caches, and its loops are kept (226 us at 110 KB of code, 205 at 87, 184 at 79, 172 at
// 71), as did room for more slots (201 against 186).
// Every wait is bounded in time; on expiry the kernel records LI_DEVERR_TIMEOUT and returns. The
// softmax warps of a group agree on giving up (the vote carries it), so none is left at a barrier; a wait for a
// unit's last product, which no vote follows, is told by the warp that made it.
#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "li_cache_attn.cuh"
#include "li_fixed_div.cuh"
#include "li_internal.cuh"
#include "li_sm100.cuh"

namespace li {
namespace {

using namespace sm100;

constexpr int kKeys = 128;                          // selected keys per tile (MMA M)
constexpr uint32_t kSlot = kKeys * 128;             // 128 bytes of 128 keys
constexpr int kMaxCutLog2 = 3, kMaxCuts = 1 << kMaxCutLog2;     // CTAs that share a unit (portable clusters)
constexpr int kMaxSlots = 16, kTileRing = 4, kAhRing = 4;
constexpr int kGatherWarps = 4;
constexpr uint32_t kSmemBytes = 232448;
constexpr uint32_t kTailBytes = 8192;
constexpr uint32_t kTailOff = kSmemBytes - kTailBytes;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A tile's largest weight is set to 2^kShift when the reference moves, and it moves when a weight
// would pass 2^kTop (of the 448 that E4M3 holds). The lo part ends in steps of 2^-13, so a weight is held
// to 2^-(14 + kShift) of the row's largest, and what a sink's tail of n keys may lose in all is n times
// that: 2^-10 of the output at 2048 keys and 2^-8, half a step of bf16, at 8192. More room for fewer
// moves takes accuracy: 2048 tokens took 169 us with a shift of 4 (up to 2^-5 there), 174 with 6, 178 with 7
// and 184 with 8.
constexpr float kShift = 7.0f, kTop = 8.75f;
constexpr uint32_t kNoKey = 0xffc0ffeeu;            // a NaN that marks it
constexpr float kNoRef = -1e30f;                    // reference of a piece without keys
constexpr float kMinDescale = 7.888609052210118e-31f, kMaxDescale = 1.2676506002282294e30f;  // 2^+-100
constexpr uint32_t kDevErrInternal = 0x20u;

template <int N> struct Roles {
    static constexpr int kHeads = N / 2;                // heads of a softmax group (4 warps) and thread
    static constexpr int kSoft = 8;
    static constexpr int kPrep0 = kSoft, kPrep = 4;
    static constexpr int kGather0 = kPrep0 + kPrep;
    static constexpr int kLookup = kGather0 + kGatherWarps, kQk = kLookup + 1;  // then pv
    static constexpr int kThreads = 32 * (kLookup + 3);
};

// What a CTA works on in turn. Every role finds its units by itself (unit_at); only the tiles that
// are left once those behind the last selected entry are dropped come from the lookup warp.
struct Unit {
    int32_t row;            // -1: no more units
    int32_t head0;          // first head
    int32_t tile0, tiles;   // tiles of the row's selection
};

// Barriers and small arrays in the shared-memory tail.
struct Bars {
    uint32_t base;
    __device__ uint32_t at(int i) const { return base + 8 * i; }
    __device__ uint32_t u_full(int i) const { return at(0 + i); }
    __device__ uint32_t u_empty(int i) const { return at(2 + i); }
    __device__ uint32_t q_full() const { return at(4); }
    __device__ uint32_t q_empty() const { return at(5); }
    __device__ uint32_t s_full(int i) const { return at(6 + i); }
    __device__ uint32_t s_empty(int i) const { return at(8 + i); }
    __device__ uint32_t p_full(int i) const { return at(10 + i); }
    __device__ uint32_t p_empty(int i) const { return at(12 + i); }
    __device__ uint32_t o_empty() const { return at(14); }
    __device__ uint32_t rows_full(int i) const { return at(15 + i); }           // a tile's cache rows,
    __device__ uint32_t scales_full(int i) const { return at(15 + kTileRing + i); }     // its scales,
    __device__ uint32_t looked_up(int i) const { return at(15 + 2 * kTileRing + i); }   // both read
    __device__ uint32_t slot_full(int i) const { return at(15 + 3 * kTileRing + i); }
    __device__ uint32_t slot_empty(int i) const { return at(15 + 3 * kTileRing + kMaxSlots + i); }
    __device__ uint32_t drained(int i) const { return at(15 + 3 * kTileRing + 2 * kMaxSlots + i); }
};
constexpr int kNumBars = 17 + 3 * kTileRing + 2 * kMaxSlots;
struct Tail {
    uint64_t bars[kNumBars];
    int32_t tiles[2];                           // the units' tiles left
    uint32_t tmem;
    volatile int abort_flag, no_abort;          // no_abort: always 0
    alignas(16) int vote[2][2][4];              // [group][turn][warp]
    alignas(16) float ah[kAhRing][32];          // scale log2(e) / the head's power of two
    alignas(16) float ref[2][16];               // [group][head]: y of a weight 1
    alignas(16) float coef[2][16];              // what O counts in the output
    alignas(16) float alpha[2][16], moved[2][16];   // root of what O and the sums shrink by; its log2
    int seen[2][16], fresh[2];                  // whether a head's reference is set; any that is not
    alignas(16) float red[2][16][4];            // [group][head][warp]
    alignas(16) float lsum[2][16][4], mx[2][16][4];
    alignas(16) float descale[kTileRing][kKeys];    // kNoKey: the entry selects nothing
    alignas(16) int32_t row[kTileRing][kKeys];  // cache rows, -1: none; key 32 w + s + 4 i at 32 w + 8 s + i
};
static_assert(sizeof(Tail) <= kTailBytes, "shared memory tail");

struct Params {
    const uint16_t *q, *q_rope;
    const uint8_t *codes;
    const float *descale;
    const uint16_t *k_rope;
    const int32_t *indices, *block_table;
    uint32_t *status;
    uint16_t *out;
    float *smax, *ssum;
    int64_t bt_stride, key_rows;
    int64_t units;
    float scale;
    int32_t rows, s1, s2, G, Dm, topk, block_size, num_blocks;
    int32_t has_rope, blocks, head_blocks, tiles, cut_log2;    // CTAs per unit
    int32_t slots;
    uint32_t p_off, slot_off, tmem_cols;
    FixedDiv by_block, by_s1, by_heads;
};

struct Ring {
    int idx = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n, int by) {       // by <= n
        idx += by;
        if (idx >= n) { idx -= n; phase ^= 1u; }
    }
    __device__ __forceinline__ void next(int n) {
        if (++idx == n) { idx = 0; phase ^= 1u; }
    }
};

// Bounded wait of a whole warp, with one answer for all lanes. What follows a first try that fails is
// out of line: the kernel has some thirty waits, and its loops compete for the instruction caches.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    return mbar_wait(bar, parity, abort_flag);
}
// Every lane for itself (the loops that issue copies and products: a vote per wait costs them more
// than the wait); the lanes may differ in their answer, and the caller lets them agree later.
__device__ __forceinline__ bool wait_lane(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    bool ok = mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) ok = __all_sync(0xffffffffu, wait_long(bar, parity, abort_flag));
    return ok;
}
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// One lane of the warp, chosen by the hardware (all lanes call).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// 16-byte copy, `bytes` (0 or 16) of them read and the rest filled with zeros.
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ float exp2_(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// x = hi + lo / 16 with both parts in E4M3, two elements each (4 bits and the next 4, with a sign).
__device__ __forceinline__ void split_e4m3(__half2 x, uint32_t *hi, uint32_t *lo) {
    *hi = __nv_cvt_halfraw2_to_fp8x2((__half2_raw)x, __NV_SATFINITE, __NV_E4M3);
    const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)*hi, __NV_E4M3));
    const __half2 rest = __hfma2(h, __float2half2_rn(-16.0f), __hmul2(x, __float2half2_rn(16.0f)));
    *lo = __nv_cvt_halfraw2_to_fp8x2((__half2_raw)rest, __NV_SATFINITE, __NV_E4M3);
}
// n consecutive fp32 columns of this thread's TMEM lane, without the wait.
__device__ __forceinline__ void tmem_ld_nowait(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16_nowait(taddr, r); }
__device__ __forceinline__ void tmem_ld_nowait(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_nowait(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_nowait(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The weights operand: row = key, 2 N bytes (hi of N heads, then lo), i.e. an MN-major B whose rows
// are one swizzle span: 32 bytes (N = 16) or 64 (N = 32); eight keys form an atom.
template <int N> __device__ __forceinline__ uint64_t weights_desc(uint32_t saddr) {
    constexpr uint64_t kType = N == 16 ? 6 : 4;         // 32- or 64-byte swizzle
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)((16 * N) >> 4) << 32) |
           ((uint64_t)1 << 46) | (kType << 61);
}
// Byte of chunk c (16 heads) in row `key`.
template <int N> __device__ __forceinline__ uint32_t weights_at(int key, int c) {
    const int x = N == 16 ? (key >> 2) & 1 : (key >> 1) & 3;
    return (uint32_t)(key * 2 * N + ((c ^ x) << 4));
}

// Largest of v over the warp (NaN counts as -infinity).
__device__ __forceinline__ float warp_max(float v) {
    int i = __float_as_int(v == v ? v : -__int_as_float(0x7f800000));
    i ^= (i >> 31) & 0x7fffffff;
    i = __reduce_max_sync(0xffffffffu, i);
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}
// Sums (or maxima) of H values over the warp, transposed: lane l returns value l / (32 / H).
template <bool kMax, int H>
__device__ __forceinline__ float transpose_reduce(const float (&v)[H], int lane) {
    float a[H];
#pragma unroll
    for (int i = 0; i < H; ++i) a[i] = v[i];
    int bit = 16;
#pragma unroll
    for (int half = H / 2; half >= 1; half >>= 1, bit >>= 1) {
        const bool up = (lane & bit) != 0;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = up ? a[i + half] : a[i];
            const float send = up ? a[i] : a[i + half];
            const float recv = __shfl_xor_sync(0xffffffffu, send, bit);
            a[i] = kMax ? fmaxf(keep, recv) : keep + recv;
        }
    }
    for (; bit >= 1; bit >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, a[0], bit);
        a[0] = kMax ? fmaxf(a[0], o) : a[0] + o;
    }
    return a[0];
}

// The it-th unit of this CTA, or its share of one.
__device__ __forceinline__ Unit unit_at(const Params &P, int it) {
    Unit u{-1, 0, 0, P.tiles};
    const int64_t i = (blockIdx.x >> P.cut_log2) + (int64_t)it * (gridDim.x >> P.cut_log2);
    if (i >= P.units) return u;                         // below 2^26
    if (P.cut_log2) {
        const int c = (int)blockIdx.x & ((1 << P.cut_log2) - 1);
        u.tile0 = c * P.tiles >> P.cut_log2;
        u.tiles = ((c + 1) * P.tiles >> P.cut_log2) - u.tile0;
    }
    u.row = P.by_heads.div((int32_t)i);
    u.head0 = ((int32_t)i - u.row * P.head_blocks) * 32;
    return u;
}

// ---- clusters ----------------------------------------------------------------------------------------
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four floats at the same place as `addr` in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_peer(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

// ---- lookups -----------------------------------------------------------------------------------------
// 4-byte copy into shared memory, tracked like every cp.async of the thread.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Entry `at` of all rows' selections; the bounds-checked build takes one outside for none.
__device__ __forceinline__ int32_t entry(const Params &P, int64_t at) {
    return idx_ok(at, (int64_t)P.rows * P.topk, P.status) ? __ldg(P.indices + at) : -1;
}
// Block q of batch b's sequence.
__device__ __forceinline__ int32_t block_of(const Params &P, int32_t b, int32_t q) {
    const int64_t at = b * P.bt_stride + q;
    return idx_ok(at, (int64_t)P.by_s1.div(P.rows) * P.bt_stride, P.status) ? __ldg(P.block_table + at) : -1;
}

// One warp: the tiles of each unit (those behind its last selected entry are left out), and for each
// tile the cache rows of its keys, four a lane, with their scales on the way into shared memory.
__device__ void lookup_role(const Params &P, Tail *T, const Bars &bars) {
    const int lane = threadIdx.x & 31;
    Ring tr;
    uint32_t err = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
        const Unit u = unit_at(P, it);
        if (u.row < 0) break;
        const int64_t first = (int64_t)u.row * P.topk;
        const int32_t b = P.by_s1.div(u.row);
        const int32_t *table = P.block_table ? P.block_table + b * P.bt_stride : nullptr;
        const int from = u.tile0 * kKeys, to = min((u.tile0 + u.tiles) * kKeys, P.topk);
        const int32_t tail = entry(P, first + to - 1);
        int32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = from + lane + 32 * i;
            v[i] = p < to ? entry(P, first + p) : -1;
        }
        // the rest of the unit's entries, and the start of its block-table row, on their way to L2
        for (int p = from + kKeys + 32 * lane; p < to; p += 32 * 32) prefetch_l2(P.indices + first + p);
        if (table && 32 * lane < P.bt_stride) prefetch_l2(table + 32 * lane);
        int tiles = u.tiles;
        if (tail < 0) {
            int last = -1;
#pragma unroll 8
            for (int p = from + lane; p < to; p += 32)
                if (entry(P, first + p) >= 0) last = p;
            last = __reduce_max_sync(0xffffffffu, last);
            tiles = last < from ? 0 : (last - from) / kKeys + 1;
        }
        ok = wait_warp(bars.u_empty(it & 1), ((it >> 1) & 1) ^ 1, &T->abort_flag);
        if (!ok) break;
        if (lane == 0) {
            T->tiles[it & 1] = tiles;
            mbar_arrive(bars.u_full(it & 1));
        }
        __syncwarp();
        for (int j = 0; j < tiles; ++j, tr.next(kTileRing)) {
            // positions outside the sequence, blocks outside the cache and negative entries select nothing
            // (dense keys: one block of S2 rows a batch, batch b's is block b)
            int32_t blk[4], off[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool in = (uint32_t)v[i] < (uint32_t)P.s2;
                if (!in && v[i] >= 0) err |= LI_DEVERR_LENGTHS;
                const int32_t q = table && in ? P.by_block.div(v[i]) : 0;
                off[i] = in ? v[i] - q * P.block_size : -1;
                blk[i] = table && in ? block_of(P, b, q) : b;
            }
            // the next tile's entries
            const int next = from + (j + 1) * kKeys + lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = next + 32 * i < to ? entry(P, first + next + 32 * i) : -1;
            ok = wait_warp(bars.looked_up(tr.idx), tr.phase ^ 1u, &T->abort_flag);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                int32_t r = -1;
                if (off[i] >= 0) {
                    if ((uint32_t)blk[i] < (uint32_t)P.num_blocks) r = blk[i] * P.block_size + off[i];
                    else err |= LI_DEVERR_TABLE;
                }
                if (r >= 0 && !idx_ok(r, P.key_rows, P.status)) r = -1;
                T->row[tr.idx][32 * i + 8 * (lane & 3) + (lane >> 2)] = r;
                // the scale goes to the softmax warps, which check it
                float *d = &T->descale[tr.idx][32 * i + lane];
                if (r >= 0) cp_async4(smem_u32(d), P.descale + r);
                else *d = __uint_as_float(kNoKey);
            }
            mbar_arrive(bars.rows_full(tr.idx));
            // the copies arrive by themselves; the marks above are ordinary stores and take an arrival that
            // releases them
            cp_async_arrive(bars.scales_full(tr.idx));
            mbar_arrive(bars.scales_full(tr.idx));
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");    // no copy may outlive the CTA
    if (!ok) T->abort_flag = 1;
    if (err && P.status) atomicOr(P.status, err);
}

// The tiles left of this CTA's it-th unit, for a whole warp; -1 on giving up.
__device__ __forceinline__ int take_tiles(Tail *T, const Bars &bars, int it) {
    if (!wait_warp(bars.u_full(it & 1), (it >> 1) & 1, &T->abort_flag)) return -1;
    const int tiles = T->tiles[it & 1];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bars.u_empty(it & 1));
    return __shfl_sync(0xffffffffu, tiles, 0);
}

// ---- q: normalised and split ---------------------------------------------------------------------
template <int N>
__device__ void prep_role(const Params &P, uint8_t *smem, Tail *T, const Bars &bars) {
    using R = Roles<N>;
    const int wp = (threadIdx.x >> 5) - R::kPrep0, lane = threadIdx.x & 31;
    const float kInf = __int_as_float(0x7f800000);
    int n = 0;                                  // units with tiles so far
    for (int it = 0;; ++it) {
        const Unit u = unit_at(P, it);
        if (u.row < 0) return;
        const int heads = min(P.G - u.head0, N);
        const int64_t row0 = (int64_t)u.row * P.G + u.head0;
        bool some = true;
        for (int h0 = wp; h0 < N && some; h0 += 4 * R::kPrep) {
            // four heads of the warp at once, so that their reads overlap; the first four are read
            // while the unit's tiles and the buffer are not known yet
            uint4 v[4][2], rope = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int h = h0 + t * R::kPrep;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int vec = lane + 32 * i;          // 8 elements
                    v[t][i] = make_uint4(0u, 0u, 0u, 0u);
                    if (h < heads && vec * 8 < P.Dm && idx_ok((row0 + h) * P.Dm + vec * 8, (int64_t)P.rows * P.G * P.Dm, P.status))
                        v[t][i] = __ldg(reinterpret_cast<const uint4 *>(P.q + (row0 + h) * P.Dm) + vec);
                }
            }
            // the rope parts: 8 lanes a head
            const int rh = h0 + (lane >> 3) * R::kPrep, piece = lane & 7;
            if (P.has_rope && rh < heads && idx_ok((row0 + rh) * 64 + piece * 8, (int64_t)P.rows * P.G * 64, P.status))
                rope = __ldg(reinterpret_cast<const uint4 *>(P.q_rope + (row0 + rh) * 64) + piece);
            if (h0 == wp) {
                const int tiles = take_tiles(T, bars, it);
                some = tiles != 0;
                if (!some) break;
                if (tiles < 0 || !wait_warp(bars.q_empty(), (n & 1) ^ 1, &T->abort_flag)) {
                    T->abort_flag = 1;
                    return;
                }
            }
            if (P.has_rope)
                *reinterpret_cast<uint4 *>(smem + P.blocks * (2 * N * 128) + rh * 128 + ((piece ^ (rh & 7)) << 4)) = rope;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int h = h0 + t * R::kPrep;
                __nv_bfloat162 m2 = __float2bfloat162_rn(0.0f);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __nv_bfloat162 *w = reinterpret_cast<const __nv_bfloat162 *>(&v[t][i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) m2 = __hmax2(m2, __habs2(w[j]));
                }
                const float amax = warp_max(fmaxf(__low2float(m2), __high2float(m2)));
                // f = 2^(7 - exponent of amax): the largest element lands in [128, 256). An infinity
                // has no code: f is NaN then, so that the head's result shows it
                const int e = max((int)(__float_as_uint(amax) >> 23), 8);   // biased; 8 keeps f finite
                float f = amax > 0.0f ? __uint_as_float((uint32_t)(127 + 7 + 127 - e) << 23) : 1.0f;
                if (amax == kInf) f = __int_as_float(0x7fc00000);
                if (lane == 0) T->ah[n & (kAhRing - 1)][h] = P.scale * kLog2e / f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int vec = lane + 32 * i;
                    if (vec * 8 >= P.Dm) continue;
                    const uint32_t w[4] = {v[t][i].x, v[t][i].y, v[t][i].z, v[t][i].w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // fp16 holds q f exactly down to 2^-14, and what lies below has no lo part
                        const __half2 x = __floats2half2_rn(bf16_lo(w[j]) * f, bf16_hi(w[j]) * f);
                        split_e4m3(x, &hi[j], &lo[j]);
                    }
                    const int off = (vec * 8) & 127, b = vec >> 4;
                    const uint32_t at = (uint32_t)(b * 2 * N * 128 + (((off >> 4) ^ (h & 7)) << 4) + (off & 8));
                    *reinterpret_cast<uint2 *>(smem + at + h * 128) =
                        make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                    *reinterpret_cast<uint2 *>(smem + at + (N + h) * 128) =
                        make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                }
            }
        }
        if (!some) continue;                    // a unit without tiles
        fence_async_smem();
        mbar_arrive(bars.q_full());
        ++n;
    }
}

// ---- gather ----------------------------------------------------------------------------------------
template <int N>
__device__ void gather_role(const Params &P, uint8_t *smem, Tail *T, const Bars &bars) {
#if defined(LI_TEST_NO_LOADS)
    return;     // test build: no copy and no arrival, so that the first product's wait runs out
#endif
    const int w = (threadIdx.x >> 5) - Roles<N>::kGather0, lane = threadIdx.x & 31;
    const int piece = lane & 7, sub = lane >> 3;        // this lane copies keys 32 w + sub + 4 i
    const uint8_t *codes = P.codes + piece * 16, *ropes = reinterpret_cast<const uint8_t *>(P.k_rope) + piece * 16;
    // 16-byte piece of row key in a swizzled slot; key & 7 is sub + 4 (i & 1)
    const uint32_t dst = smem_u32(smem) + P.slot_off + (32 * w + sub) * 128;
    const uint32_t even = (uint32_t)((piece ^ sub) << 4), odd = (uint32_t)((piece ^ (sub + 4)) << 4);
    Ring sr, tr;
    bool ok = true;
    for (int it = 0; ok; ++it) {
        if (unit_at(P, it).row < 0) break;
        const int tiles = take_tiles(T, bars, it);
        ok = tiles >= 0;
        for (int j = 0; j < tiles && ok; ++j, tr.next(kTileRing)) {
            ok = wait_warp(bars.rows_full(tr.idx), tr.phase, &T->abort_flag);
            if (!ok) break;
            // the eight rows of this lane, and 16 bytes of each piece or none
            int32_t r[8];
            *reinterpret_cast<int4 *>(r) = *reinterpret_cast<const int4 *>(&T->row[tr.idx][32 * w + 8 * sub]);
            *reinterpret_cast<int4 *>(r + 4) = *reinterpret_cast<const int4 *>(&T->row[tr.idx][32 * w + 8 * sub + 4]);
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.looked_up(tr.idx));
            const uint8_t *row[8];
            uint32_t size[8];
            bool there = true;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (r[i] >= 0 && !idx_ok(r[i], P.key_rows, P.status)) r[i] = -1;
                size[i] = r[i] < 0 ? 0u : 16u;
                r[i] = max(r[i], 0);
                row[i] = codes + (uint64_t)(uint32_t)r[i] * (uint32_t)P.Dm;
            }
            if (P.has_rope) {
                there = wait_lane(bars.slot_empty(sr.idx), sr.phase ^ 1u, &T->abort_flag);
                if (there) {
                    const uint32_t to = dst + sr.idx * kSlot;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        cp_async16_zfill(to + i * 512 + (i & 1 ? odd : even), ropes + (uint64_t)(uint32_t)r[i] * 128u, size[i]);
                    cp_async_arrive(bars.slot_full(sr.idx));
                }
                sr.next(P.slots);
            }
#pragma unroll 1
            for (int c = 0; c < P.blocks && there; ++c) {       // a slot that is not free is not written
                there = wait_lane(bars.slot_empty(sr.idx), sr.phase ^ 1u, &T->abort_flag);
                if (!there) break;
                const uint32_t to = dst + sr.idx * kSlot;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    cp_async16_zfill(to + i * 512 + (i & 1 ? odd : even), row[i] + 128 * c, size[i]);
                cp_async_arrive(bars.slot_full(sr.idx));
                sr.next(P.slots);
            }
            ok = __all_sync(0xffffffffu, there);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");    // no copy may outlive the CTA
    if (!ok) T->abort_flag = 1;
}

// A warp that issues products gives up: those under way still read shared memory and write TMEM, so
// it waits for them, with the limit of every wait.
__device__ __noinline__ void drain(Tail *T, uint32_t bar) {
    T->abort_flag = 1;
    if (elect_one()) umma_commit(bar);
    __syncwarp();
    wait_long(bar, 0, &T->no_abort);
    __syncwarp();
}

// ---- products --------------------------------------------------------------------------------------
// TMEM: S of tile parity p at p kSCols: [0, 2N) hi and lo of q.c, [2N, 3N) the rope product;
// O block b at 2 kSCols + 2N b: [0, N) hi, [N, 2N) lo.
template <int N> constexpr uint32_t kSCols = 4 * N;

template <int N>
__device__ void qk_role(const Params &P, uint8_t *smem, Tail *T, const Bars &bars, uint32_t tmem) {
    const uint32_t sbase = smem_u32(smem), slots = sbase + P.slot_off;
    constexpr uint32_t kQBlock = 2 * N * 128;
    constexpr uint32_t idesc8 = (1u << 4) | ((2u * N >> 3) << 17) | (8u << 24);
    constexpr uint32_t idesc16 = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
    Ring sr;
    uint32_t kt = 0, nu = 0;
    for (int it = 0;; ++it) {
        if (unit_at(P, it).row < 0) return;
        const int tiles = take_tiles(T, bars, it);
        if (tiles < 0) break;
        if (tiles == 0) continue;
        if (!wait_warp(bars.q_full(), nu & 1u, &T->abort_flag)) break;
        bool ok = true;
        for (int j = 0; j < tiles && ok; ++j, ++kt) {
            const uint32_t b = kt & 1u, d = tmem + b * kSCols<N>;
            // one lane for the whole tile, its waits included; a slot's part of the product starts when
            // the slot is there, the rope part first
            if (elect_one()) {
                int slot = sr.idx;
                uint32_t phase = sr.phase;
                const auto next = [&] {
                    if (++slot == P.slots) { slot = 0; phase ^= 1u; }
                };
                ok = wait_lane(bars.s_empty(b), ((kt >> 1) & 1u) ^ 1u, &T->abort_flag);
                if (P.has_rope && ok) {
                    ok = wait_lane(bars.slot_full(slot), phase, &T->abort_flag);
                    fence_async_smem();         // the gathered rows, for the async proxy
                    tc_fence_after();
                    const uint64_t a = sw128_desc(slots + slot * kSlot), q = sw128_desc(sbase + P.blocks * kQBlock);
                    if (ok) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) umma_f16(d + 2 * N, a + 2 * k, q + 2 * k, idesc16, k > 0);
                        umma_commit(bars.slot_empty(slot));
                    }
                    next();
                }
#pragma unroll 1
                for (int c = 0; c < P.blocks; ++c) {
                    if (!ok) break;
                    ok = wait_lane(bars.slot_full(slot), phase, &T->abort_flag);
                    if (!ok) break;
                    fence_async_smem();
                    tc_fence_after();
                    const uint64_t a = sw128_desc(slots + slot * kSlot), q = sw128_desc(sbase + c * kQBlock);
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma_f8(d, a + 2 * k, q + 2 * k, idesc8, (c | k) != 0);
                    next();
                }
                if (ok) umma_commit(bars.s_full(b));
            }
            ok = __all_sync(0xffffffffu, ok);
            sr.next(P.slots, P.has_rope + P.blocks);
        }
        if (!ok) break;
        if (elect_one()) umma_commit(bars.q_empty());
        __syncwarp();
        ++nu;
    }
    drain(T, bars.drained(0));
}

template <int N>
__device__ void pv_role(const Params &P, uint8_t *smem, Tail *T, const Bars &bars, uint32_t tmem) {
    const uint32_t sbase = smem_u32(smem), slots = sbase + P.slot_off;
    constexpr uint32_t idesc = (1u << 4) | (1u << 15) | (1u << 16) | ((2u * N >> 3) << 17) | (8u << 24);
    Ring sr;
    uint32_t kt = 0, nu = 0;
    for (int it = 0;; ++it) {
        if (unit_at(P, it).row < 0) return;
        const int tiles = take_tiles(T, bars, it);
        if (tiles < 0) break;
        if (tiles == 0) continue;
        bool ok = true;
        for (int j = 0; j < tiles; ++j, ++kt) {
            // the unit's first product overwrites O: the unit before must have been read out
            ok = (j > 0 || nu == 0 || wait_warp(bars.o_empty(), (nu - 1) & 1u, &T->abort_flag)) &&
                 wait_warp(bars.p_full(kt & 1u), (kt >> 1) & 1u, &T->abort_flag);
            if (!ok) break;
            fence_async_smem();                 // the weights, for the async proxy
            tc_fence_after();
            const uint64_t p = weights_desc<N>(sbase + P.p_off + (kt & 1u) * (2 * N * 128));
            // one elected lane for the whole tile
            if (elect_one()) {
                int slot = sr.idx + P.has_rope;
                if (slot == P.slots) slot = 0;
#pragma unroll 1
                for (int c = 0; c < P.blocks; ++c) {
                    const uint64_t v = sw128_desc_mn(slots + slot * kSlot, kSlot);
                    const uint32_t d = tmem + 2 * kSCols<N> + c * 2 * N;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_f8(d, v + k * (32 * 128 >> 4), p + k * (32 * 2 * N >> 4), idesc, (j | k) != 0);
                    umma_commit(bars.slot_empty(slot));
                    if (++slot == P.slots) slot = 0;
                }
#if defined(LI_TEST_NO_LAST_COMMIT)
                // test build: a unit's last product is not announced, so that the output's wait runs out
                if (j < tiles - 1)
#endif
                    umma_commit(bars.p_empty(kt & 1u));
            }
            __syncwarp();
            sr.next(P.slots, P.has_rope + P.blocks);
        }
        if (!ok) break;
        ++nu;
    }
    drain(T, bars.drained(1));
}

// A share's partial outputs in shared memory, from slot_off on: O [N][Dm] in fp32, then per head its
// reference, sum and maximum (16 bytes).
template <int N> __device__ __forceinline__ uint32_t part_stat(int32_t Dm, int h) { return (uint32_t)(N * Dm + 4 * h) * 4u; }

// ---- softmax and output ------------------------------------------------------------------------------
// Barrier of a softmax group's four warps. Its threads do different things before most of them, and the
// aligned barrier wants a warp together; so do the TMEM reads that follow.
__device__ __forceinline__ void group_bar(int id) {
    __syncwarp();
    named_bar(id, 128);
}
// Four consecutive floats of shared memory.
__device__ __forceinline__ void lds4(const float *p, float (&v)[4]) {
    const float4 t = *reinterpret_cast<const float4 *>(p);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
}

// Maximum and sum of a head from its largest x log2(e), the sum against its reference, and that. Maxima leave
// NaN out and the sum does not: a NaN there is the maximum's too.
__device__ __forceinline__ void store_stats(const Params &P, int64_t at, float m, float sum, float ref) {
    const float kInf = __int_as_float(0x7f800000);
    if (!idx_ok(at, (int64_t)P.rows * P.G, P.status)) return;
    P.smax[at] = sum != sum ? sum : m > -kInf ? m * kLn2 : m;
    P.ssum[at] = m > -kInf ? sum * exp2_(ref - m) : sum;
}

template <int N, bool kStats>
__device__ void softmax_role(const Params &P, uint8_t *smem, Tail *T, const Bars &bars, uint32_t tmem) {
    constexpr int H = Roles<N>::kHeads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = warp >> 2, q = warp & 3;              // group, quarter of the TMEM lanes
    const int key = 32 * q + lane;                      // key of the tile; dim of an O block
    const int col = H * g;                              // the group's first head
    const bool holds = (lane & (32 / H - 1)) == 0;      // the lane has a reduced value, of this head:
    const int held = lane / (32 / H);
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const float kInf = __int_as_float(0x7f800000);
    volatile int *abort_flag = &T->abort_flag;
    const int bar_id = 1 + g;
    const float rs = P.scale * kLog2e;
    uint32_t kt = 0;
    uint32_t turn = 0;                                  // votes of the group
    int nu = 0;
    bool ok = true, bad = false;
    for (int it = 0;; ++it) {
        const Unit u = unit_at(P, it);
        if (u.row < 0) {
            if (bad && P.status) atomicOr(P.status, LI_DEVERR_DESCALE);
            return;
        }
        // the group's warps agree on giving up here and by a vote per tile, so that none is left at a
        // barrier
        ok = wait_warp(bars.u_full(it & 1), (it >> 1) & 1, abort_flag) && ok;
        if (lane == 0) T->vote[g][turn & 1][q] = ok ? 0 : 2;
        if (q == 0 && lane < H) {
            T->ref[g][lane] = 0.0f;
            T->seen[g][lane] = 0;
        }
        group_bar(bar_id);
        {
            const int4 v = *reinterpret_cast<const int4 *>(T->vote[g][turn++ & 1]);
            if ((v.x | v.y | v.z | v.w) & 2) break;
        }
        bool failed = false;
        const int tiles = T->tiles[it & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.u_empty(it & 1));
        float l[H], mx[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            l[i] = 0.0f;
            if (kStats) mx[i] = -kInf;
        }
        bool fresh = true;                              // a head has no reference yet
        const float *ah = T->ah[nu & (kAhRing - 1)] + col;
        const float *ref = T->ref[g];
        for (int j = 0; j < tiles; ++j, ++kt) {
            const uint32_t b = kt & 1u, tr = kt & (kTileRing - 1);
            ok = ok && wait_lane(bars.scales_full(tr), (kt / kTileRing) & 1u, abort_flag);
            // an entry that selects nothing, or whose scale is out of range, has scale 0 and a weight
            // of 2^-inf
            float d = ok ? T->descale[tr][key] : 0.0f;
            if (!(d >= kMinDescale && d <= kMaxDescale)) {
                bad |= ok && __float_as_uint(d) != kNoKey;
                d = 0.0f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.looked_up(tr));
            const float log2d = log2f(d), back = d > 0.0f ? log2d : 0.0f;
            ok = ok && wait_lane(bars.s_full(b), (kt >> 1) & 1u, abort_flag);
            float t[H];                                 // y - ref, the weights' exponents
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < H; h += 8) {
                uint32_t hi[8], lo[8], rp[8];
                const uint32_t s = tmem + lanes + b * kSCols<N> + col + h;
                tmem_ld_nowait(s, hi);
                tmem_ld_nowait(s + N, lo);
                if (P.has_rope) tmem_ld_nowait(s + 2 * N, rp);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    float a4[4];
                    lds4(ah + h + i, a4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float sc = fmaf(__uint_as_float(lo[i + k]), 0.0625f, __uint_as_float(hi[i + k]));
                        t[h + i + k] = fmaf(sc, d * a4[k], P.has_rope ? rs * __uint_as_float(rp[i + k]) : 0.0f);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.s_empty(b));
            float top = -kInf;
#pragma unroll
            for (int i = 0; i < H; i += 4) {
                float r4[4];
                lds4(ref + i, r4);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (kStats && d > 0.0f) mx[i + k] = fmaxf(mx[i + k], t[i + k]);
                    t[i + k] = (t[i + k] + log2d) - r4[k];
                    top = fmaxf(top, t[i + k]);
                }
            }
            const bool any = __any_sync(0xffffffffu, top > kTop || (fresh && d > 0.0f));
            const bool all = __all_sync(0xffffffffu, ok);
            if (lane == 0) T->vote[g][turn & 1][q] = (any ? 1 : 0) | (all ? 0 : 2);
            group_bar(bar_id);
            const int4 v4 = *reinterpret_cast<const int4 *>(T->vote[g][turn++ & 1]);
            const int v = v4.x | v4.y | v4.z | v4.w;
            if (v & 2) {
                failed = true;
                break;
            }
            if (v & 1) {
                // references with a larger weight than 2^kTop move so that it is 2^kShift, and a head's
                // first one so whatever its largest weight is; O and the sums follow
                const float m = transpose_reduce<true>(t, lane);
                if (holds) T->red[g][held][q] = m;
                group_bar(bar_id);
                if (q == 0 && lane < H) {
                    float m4[4];
                    lds4(T->red[g][lane], m4);
                    const float most = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    const bool seen = T->seen[g][lane] != 0;
                    const float up = seen ? fmaxf(most - kShift, 0.0f) : most > -kInf ? most - kShift : 0.0f;
                    T->ref[g][lane] += up;
                    // nothing is summed before the first. The root: 2^-up itself may underflow where a
                    // key with a small scale has its share of the sums
                    T->alpha[g][lane] = seen ? exp2_(-0.5f * up) : 0.0f;
                    T->moved[g][lane] = up;
                    T->seen[g][lane] = seen || most > -kInf;
                    const bool all_seen = __all_sync((1u << H) - 1u, seen || most > -kInf);
                    if (lane == 0) T->fresh[g] = !all_seen;
                }
                group_bar(bar_id);
                fresh = T->fresh[g] != 0;
#pragma unroll
                for (int i = 0; i < H; i += 4) {
                    float a4[4], u4[4];
                    lds4(T->alpha[g] + i, a4);
                    lds4(T->moved[g] + i, u4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        l[i + k] = l[i + k] * a4[k] * a4[k];
                        t[i + k] -= u4[k];
                    }
                }
                if (j > 0) {                            // O holds the tiles before
                    ok = ok && wait_lane(bars.p_empty(b ^ 1u), ((kt - 1) >> 1) & 1u, abort_flag);
                    __syncwarp();
                    tc_fence_after();
                    // two reads in flight where the registers allow (2048 tokens 179 us against 183)
                    constexpr int kB = 16 / H;
#pragma unroll 1
                    for (int c = 0; c < 2 * P.blocks; c += kB) {    // hi and lo of each block
                        const uint32_t o = tmem + lanes + 2 * kSCols<N> + c * N + col;
                        uint32_t x[kB][H];
#pragma unroll
                        for (int b = 0; b < kB; ++b) tmem_ld_nowait(o + b * N, x[b]);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < H; i += 4) {
                            float a4[4];
                            lds4(T->alpha[g] + i, a4);
#pragma unroll
                            for (int b = 0; b < kB; ++b)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    x[b][i + k] = __float_as_uint(__uint_as_float(x[b][i + k]) * (a4[k] * a4[k]));
                        }
#pragma unroll
                        for (int b = 0; b < kB; ++b) tmem_st_nowait(o + b * N, x[b]);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
            }
            // p_empty(i) completes with the value product of every second tile: it frees that tile's
            // weights, and O holds all tiles up to it. A wait for tile t is sound because the wait
            // below for tile t - 2 came before (a parity says nothing of phases further back)
            ok = ok && wait_lane(bars.p_empty(b), ((kt >> 1) & 1u) ^ 1u, abort_flag);
            // weights as hi + lo / 16, by way of fp16 (11 bits); a key's row of the operand
            uint32_t hi[H / 4], lo[H / 4];
#pragma unroll
            for (int i = 0; i < H; i += 2) {
                const float p0 = exp2_(t[i]), p1 = exp2_(t[i + 1]);
                // e^x / 2^ref: an exponential of its own, since 2^(y - ref) may underflow where the scales
                // span more than 2^126 and this does not
                l[i] += exp2_(t[i] - back);
                l[i + 1] += exp2_(t[i + 1] - back);
                uint32_t h8, l8;
                split_e4m3(__floats2half2_rn(p0, p1), &h8, &l8);
                if (i & 2) {
                    hi[i / 4] |= h8 << 16;
                    lo[i / 4] |= l8 << 16;
                } else {
                    hi[i / 4] = h8;
                    lo[i / 4] = l8;
                }
            }
            uint8_t *pb = smem + P.p_off + b * (2 * N * kKeys);
            if constexpr (H == 8) {
                *reinterpret_cast<uint2 *>(pb + weights_at<N>(key, 0) + col) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2 *>(pb + weights_at<N>(key, 1) + col) = make_uint2(lo[0], lo[1]);
            } else {
                *reinterpret_cast<uint4 *>(pb + weights_at<N>(key, g)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(pb + weights_at<N>(key, 2 + g)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_async_smem();
            mbar_arrive(bars.p_full(b));
        }
        if (failed) break;
        // the group's sums and maxima over its keys, and the unit's last value product
        if (tiles > 0) {
            const float ws = transpose_reduce<false>(l, lane);
            float wm = 0.0f;
            if constexpr (kStats) wm = transpose_reduce<true>(mx, lane);
            if (holds) {
                T->lsum[g][held][q] = ws;
                if (kStats) T->mx[g][held][q] = wm;
            }
            const uint32_t last = bars.p_empty((kt - 1) & 1u), parity = ((kt - 1) >> 1) & 1u;
            ok = ok && wait_lane(last, parity, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                // no vote follows the last unit, so the flag is set here and the warp stores nothing. The warp
                // that issued the product may have left: wait once more before what it works on is given back
                *abort_flag = 1;
                wait_long(last, parity, &T->no_abort);
            }
            group_bar(bar_id);
        }
        const int heads = min(P.G - u.head0 - col, H);          // may be <= 0
        const int64_t head_at = (int64_t)u.row * P.G + u.head0 + col;
        const bool row_ok = ok && idx_ok(u.row, P.rows, P.status);
        if (q == 0 && lane < H) {
            float r = kNoRef, s = 0.0f, m = -kInf;
            if (tiles > 0) {
                float s4[4];
                lds4(T->lsum[g][lane], s4);
                s = (s4[0] + s4[1]) + (s4[2] + s4[3]);
                if (T->seen[g][lane]) r = ref[lane];
                if constexpr (kStats) {
                    lds4(T->mx[g][lane], s4);
                    m = fmaxf(fmaxf(s4[0], s4[1]), fmaxf(s4[2], s4[3]));
                }
            }
            T->coef[g][lane] = P.cut_log2 ? 1.0f : s == 0.0f ? 0.0f : 1.0f / s;
            if (P.cut_log2) {
                *reinterpret_cast<float4 *>(smem + P.slot_off + part_stat<N>(P.Dm, col + lane)) = make_float4(r, s, m, 0.0f);
            } else if (kStats && lane < heads && row_ok) {
                store_stats(P, head_at + lane, m, s, r);
            }
        }
        group_bar(bar_id);
        tc_fence_after();
        // O out of TMEM: a share of a unit as it is in fp32 to where its keys were (the CTA has no other
        // unit, and the last product has read them), whole units normalised as bf16
        float *po = reinterpret_cast<float *>(smem + P.slot_off) + col * P.Dm + key;
        // neighbouring lanes exchange halves: an even lane stores two dims of the even heads, an odd
        // lane of the odd heads
        uint16_t *out = P.out + (head_at + (lane & 1)) * P.Dm + (key & ~1);
#pragma unroll (16 / H)
        for (int c = 0; c < P.blocks; ++c, po += 128, out += 128) {
            float o[H];
#pragma unroll
            for (int i = 0; i < H; ++i) o[i] = 0.0f;
            if (tiles > 0) {
                uint32_t hi[H], lo[H];
                __syncwarp();
                const uint32_t at = tmem + lanes + 2 * kSCols<N> + c * 2 * N + col;
                tmem_ld_nowait(at, hi);
                tmem_ld_nowait(at + N, lo);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < H; i += 4) {
                    float f4[4];
                    lds4(T->coef[g] + i, f4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        o[i + k] = f4[k] * fmaf(__uint_as_float(lo[i + k]), 0.0625f, __uint_as_float(hi[i + k]));
                }
                if (c == P.blocks - 1) {                // the next unit's product may start
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bars.o_empty());
                }
            }
            if (P.cut_log2) {
                // a share without keys is told by its sum of 0; nothing else of it is read
#pragma unroll
                for (int i = 0; i < H; ++i)
                    if (tiles > 0) po[i * P.Dm] = o[i];
            } else {
#pragma unroll
                for (int i = 0; i < H; i += 2) {
                    const __nv_bfloat162 ab = __floats2bfloat162_rn(o[i], o[i + 1]);
                    const uint32_t mine = *reinterpret_cast<const uint32_t *>(&ab);
                    const uint32_t theirs = __shfl_xor_sync(0xffffffffu, mine, 1);
                    const uint32_t v = lane & 1 ? __byte_perm(theirs, mine, 0x7632) : __byte_perm(mine, theirs, 0x5410);
                    if (i + (lane & 1) < heads && row_ok) *reinterpret_cast<uint32_t *>(out + (int64_t)i * P.Dm) = v;
                }
            }
        }
        if (tiles > 0) ++nu;
        group_bar(bar_id);          // sums, maxima and references are read before they are reset
    }
    T->abort_flag = 1;
}

// Joins the cluster's partial outputs of its unit: with references r_i, sums l_i and outputs o_i,
// o = sum o_i 2^(r_i - r) / sum l_i 2^(r_i - r), r = max r_i. The CTAs share the outputs, four dims a
// thread and turn; all shares' reads are in flight.
template <int N, bool kStats>
__device__ void join(const Params &P, uint8_t *smem) {
    const int cuts = 1 << P.cut_log2, rank = (int)blockIdx.x & (cuts - 1);
    const Unit u = unit_at(P, 0);
    const uint32_t base = smem_u32(smem) + P.slot_off;
    const float kInf = __int_as_float(0x7f800000);
    if (!idx_ok(u.row, P.rows, P.status)) return;
    const int items = min(P.G - u.head0, N) * (P.Dm / 4);
    for (int t = rank * Roles<N>::kThreads + threadIdx.x; t < items; t += cuts * Roles<N>::kThreads) {
        const int h = t / (P.Dm / 4), d = 4 * t - h * P.Dm;
        float w[kMaxCuts], l[kMaxCuts], most = kNoRef, m = -kInf, sum = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v[kMaxCuts];
#pragma unroll
        for (int i = 0; i < kMaxCuts; ++i) {
            if (i >= cuts) break;
            const float4 st = ld_peer(base + part_stat<N>(P.Dm, h), i);
            v[i] = ld_peer(base + (uint32_t)(h * P.Dm + d) * 4u, i);
            w[i] = st.x;
            l[i] = st.y;
            m = fmaxf(m, st.z);
            most = fmaxf(most, st.x);
        }
#pragma unroll
        for (int i = 0; i < kMaxCuts; ++i) {
            // a share without keys left no outputs: not even a NaN of what lies there may count
            if (i >= cuts) break;
            if (l[i] == 0.0f) continue;
            const float root = exp2_(0.5f * (w[i] - most));     // as where a reference moves
            w[i] = root * root;
            sum = fmaf(l[i] * root, root, sum);
            o.x = fmaf(v[i].x, w[i], o.x);
            o.y = fmaf(v[i].y, w[i], o.y);
            o.z = fmaf(v[i].z, w[i], o.z);
            o.w = fmaf(v[i].w, w[i], o.w);
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        const int64_t at = (int64_t)u.row * P.G + u.head0 + h;
        *reinterpret_cast<uint2 *>(P.out + at * P.Dm + d) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        if (kStats && d == 0) {
            store_stats(P, at, m, sum, most);
        }
    }
}

template <int N, bool kStats>
__global__ void __launch_bounds__(Roles<N>::kThreads, 1) cache_attn_kernel(const __grid_constant__ Params P) {
    using R = Roles<N>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5;
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0 && P.status) atomicOr(P.status, kDevErrInternal);
        return;
    }
    Tail *T = reinterpret_cast<Tail *>(smem + kTailOff);
    Bars bars{smem_u32(smem) + kTailOff};
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars.u_full(i), 1);
            mbar_init(bars.u_empty(i), 2 + R::kSoft + R::kPrep + kGatherWarps);
            mbar_init(bars.s_full(i), 1);
            mbar_init(bars.s_empty(i), R::kSoft);
            mbar_init(bars.p_full(i), 32 * R::kSoft);
            mbar_init(bars.p_empty(i), 1);
            mbar_init(bars.drained(i), 1);
        }
        mbar_init(bars.q_full(), 32 * R::kPrep);
        mbar_init(bars.q_empty(), 1);
        mbar_init(bars.o_empty(), R::kSoft);
        for (int i = 0; i < kTileRing; ++i) {
            mbar_init(bars.rows_full(i), 32);
            mbar_init(bars.scales_full(i), 2 * 32);
            mbar_init(bars.looked_up(i), kGatherWarps + R::kSoft);
        }
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(bars.slot_full(i), 32 * kGatherWarps);
            mbar_init(bars.slot_empty(i), 1);
        }
        T->abort_flag = T->no_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == R::kQk) {
        tmem_alloc(smem_u32(&T->tmem), P.tmem_cols);
        tmem_relinquish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = T->tmem;

    if (warp < R::kSoft) {
        softmax_role<N, kStats>(P, smem, T, bars, tmem);
    } else if (warp < R::kGather0) {
        prep_role<N>(P, smem, T, bars);
    } else if (warp < R::kLookup) {
        gather_role<N>(P, smem, T, bars);
    } else if (warp == R::kLookup) {
        lookup_role(P, T, bars);
    } else if (warp == R::kQk) {
        qk_role<N>(P, smem, T, bars, tmem);
    } else {
        pv_role<N>(P, smem, T, bars, tmem);
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && T->abort_flag && P.status) atomicOr(P.status, LI_DEVERR_TIMEOUT);
    if (warp == R::kQk) {
        tc_fence_after();
        tmem_dealloc(tmem, P.tmem_cols);
    }
    if (P.cut_log2) {               // every CTA of the cluster comes here, whatever became of its unit
        __syncwarp();
        cluster_sync();
        join<N, kStats>(P, smem);
        __syncwarp();
        cluster_sync();             // its shared memory has been read
    }
}

// Lets a kernel use kSmemBytes of shared memory, once per kernel and device.
template <auto kKernel> cudaError_t allow_smem() {
    static std::atomic<uint64_t> done{0};               // bit per device below 64
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1u)) return cudaSuccess;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    return e;
}

template <int N, bool kStats>
cudaError_t launch_main(const Params &P, int grid, cudaStream_t st) {
    cudaError_t e = allow_smem<cache_attn_kernel<N, kStats>>();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = 1u << P.cut_log2;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(Roles<N>::kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = st;
    cfg.attrs = &cluster;
    cfg.numAttrs = P.cut_log2 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, cache_attn_kernel<N, kStats>, P);
}

}  // namespace

bool cache_attn_plan(const li_cache_attn_args &a, CacheAttnPlan *p) {
    const int sms = device_sm_count();
    p->N = a.G <= 16 ? 16 : 32;
    p->head_blocks = (a.G + 31) / 32;
    p->tiles = (a.topk + kKeys - 1) / kKeys;
    p->blocks = a.Dm / 128;
    p->units = (int64_t)a.batch * a.s1 * p->head_blocks;
    // CTAs per unit: as many as leave every unit its SMs at once and every CTA a tile, if that spares
    // a CTA two tiles or more. A cluster lies in one GPC, whose SMs do not divide by it: 74 clusters of
    // two find room on 148 SMs, 33 of four and 15 of eight.
    // Shared against whole, 16 heads of 576, sequences of 16384 keys: 1 row of 2048 entries 12.9 us and 29.0,
    // 14 rows 14.3 and 30.8, 32 rows (four CTAs each) 19.3 and 32.2, 74 rows (two) 27.8 and 34.1; 512
    // entries, 1 row 10.4 and 12.5, 32 rows 12.2 and 13.1, 74 rows 15.1 and 14.6. One row more than finds
    // room costs a second wave: 16 rows with eight CTAs 26.3 (four: 16.4), 36 with four 33.7 (two: 23.4), 75
    // with two 46.0 (whole: 34.3). Where only one tile is spared sharing loses: 192 entries, 74 rows 11.7 and
    // 10.2. Partial outputs through memory and a second kernel cost 5 us more on the host.
    constexpr int kHalfSms[kMaxCutLog2 + 1] = {2, 4, 9, 20};    // half SMs that a cluster takes
    p->cut_log2 = kMaxCutLog2;
    while (p->cut_log2 > 0 && (p->units * kHalfSms[p->cut_log2] > 2 * (int64_t)sms || p->tiles >> p->cut_log2 == 0)) --p->cut_log2;
    if (p->tiles - ((p->tiles + (1 << p->cut_log2) - 1) >> p->cut_log2) < 2) p->cut_log2 = 0;
    // q, the weights of two tiles, and as many slots for keys as there is room for. A second buffer for
    // the next unit's q takes the room of two slots (2048 tokens 201 us against 186)
    const int per_tile = p->blocks + (a.Dr > 0 ? 1 : 0);
    p->p_off = (uint32_t)(p->blocks * 2 * p->N * 128 + (a.Dr > 0 ? p->N * 128 : 0));
    p->slot_off = (p->p_off + 2u * 2u * p->N * 128u + 1023u) / 1024u * 1024u;
    p->slots = p->slot_off < kTailOff ? (int)((kTailOff - p->slot_off) / kSlot) : 0;
    if (p->slots > kMaxSlots) p->slots = kMaxSlots;
    if (p->slots < 2 * per_tile) return false;
    uint32_t cols = 32;
    while (cols < (uint32_t)(8 * p->N + 2 * p->N * p->blocks)) cols <<= 1;
    p->tmem_cols = cols;
    p->grid = (int)(p->units < sms ? p->units << p->cut_log2 : sms);
    return true;
}

cudaError_t launch_cache_attention(const li_cache_attn_args &a, const CacheAttnPlan &p, void *out, float *smax, float *ssum, cudaStream_t st) {
    if (p.units == 0) return cudaSuccess;
    Params P{};
    P.q = static_cast<const uint16_t *>(a.q);
    P.q_rope = static_cast<const uint16_t *>(a.q_rope);
    P.codes = static_cast<const uint8_t *>(a.codes);
    P.descale = a.descale;
    P.k_rope = static_cast<const uint16_t *>(a.k_rope);
    P.indices = a.sparse_indices;
    P.status = a.device_status;
    P.out = static_cast<uint16_t *>(out);
    P.smax = smax;
    P.ssum = ssum;
    if (a.layout_k == LI_LAYOUT_PA_BSND) {
        P.block_table = a.block_table;
        P.bt_stride = a.block_table_stride;
        P.block_size = a.block_size;
        P.by_block = FixedDiv(a.block_size);
        P.num_blocks = a.num_blocks;
        P.key_rows = (int64_t)a.num_blocks * a.block_size;
    } else {
        P.block_size = a.s2;
        P.num_blocks = a.batch;
        P.key_rows = (int64_t)a.batch * a.s2;
    }
    P.units = p.units;
    P.scale = a.scale;
    P.rows = a.batch * a.s1;
    P.s1 = a.s1;
    P.by_s1 = FixedDiv(a.s1);
    P.s2 = a.s2;
    P.G = a.G;
    P.Dm = a.Dm;
    P.topk = a.topk;
    P.has_rope = a.Dr > 0;
    P.blocks = p.blocks;
    P.head_blocks = p.head_blocks;
    P.by_heads = FixedDiv(p.head_blocks);
    P.tiles = p.tiles;
    P.cut_log2 = p.cut_log2;
    P.slots = p.slots;
    P.p_off = p.p_off;
    P.slot_off = p.slot_off;
    P.tmem_cols = p.tmem_cols;
    // the statistics cost a maximum per score: a kernel of their own
    return p.N == 16 ? (smax ? launch_main<16, true>(P, p.grid, st) : launch_main<16, false>(P, p.grid, st))
                     : (smax ? launch_main<32, true>(P, p.grid, st) : launch_main<32, false>(P, p.grid, st));
}

}  // namespace li
