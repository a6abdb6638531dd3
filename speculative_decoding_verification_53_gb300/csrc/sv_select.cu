// sv_select.cu -- which blocks of a long paged cache each query attends to
// (include/spec_sparse.h): summaries of the blocks' keys, and the selection of blocks by a
// cheap score against them.
//
// Summaries are one pass over the keys, bound by memory: a warp (few blocks: all warps of a
// CTA) takes one block and head, a group of lanes a key, eight elements each, and the groups
// meet by shuffles at the end.  8 x up to 8192 positions of 8 heads of 128, pages of 64: bf16 means 16 us (84 MB,
// floor 13), bounds in pages of 16 17; e4m3 bounds 17 (43 MB, floor 7: the codes' way to fp32 bounds it; compared in
// fp32 instead of as pairs of bf16 18.4).
//
// Scores: score(i, j) = max over rows r of s_r . m_j, s_r . m_j = q_r . mean_j, or
// q_r+ . max_j + q_r- . min_j with q+ = max(q, 0), q- = min(q, 0), both matrix products of the
// query rows by the summaries.  Contexts are long and rows few, so the summaries' bytes bound
// it: mma.sync (m16n8k16), whose 16-row tiles waste least, with both operands loaded from
// global memory straight into fragments: a product does not care for the order of its
// elements, so a lane takes 16 contiguous bytes of its row where the fragments want four
// pieces of 4 bytes, for both operands alike.  The products are exact, their sums fp32.
//
// Selection: the order of scores must not depend on roundings, so it is that of the sums in 64
// bits.  An fp32 score is off by at most e = 2^-16 |q|_1 max|m| (below), so with T the k-th largest
// fp32 score whatever is above T + 2 e is in, whatever is below T - 2 e out, and only what
// lies between (one or two blocks as a rule) is summed again in 64 bits.  Where that are many
// (equal summaries), the 64-bit scores are selected among by their upper bits, then the lower ones.
// One GB300: 32 chains of 6 queries, 32 over 8 heads of 128, 256 to 1024 blocks, 64 of them by bounds 46 us, 28 of it
// the scores (floor 13: 84 MB of summaries; a warp's loads one after the other - row, page, summary, query - and
// 16 warps an SM are what it waits for), by means 38; one token over 1562 blocks 16 us; 16 trees of 61 over 128 to
// 512 blocks 91 us, 103 where their queries share a list.
//
// The error of an fp32 score: its (exact) products are summed in chains of four matrix products, each
// of which sums 17 numbers, taken to be off by at most 17 units of 2^-23 of the largest partial sum (how the hardware
// aligns and cuts them is not documented), and up to eight such chains by fp32 additions.  |q|_1 max|m| bounds every partial sum: 4 * 17 * 2^-23 + 8 * 2^-24 < 2^-16.
// fp32's smallest steps are not in that, so scores count only where |q|_1 max|m| is 2^-100 or more (256 products off by
// 2^-126 each are 2^-18 of it); below, as beyond 2^120, all are summed again.
#include <cstdint>

#include "spec_sparse.h"
#include "sv_internal.h"
#include "sv_paged.cuh"
#include "sv_rows.cuh"

namespace {

using sv::neg_inf;
using sv::pos_inf;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxB = 65535;
constexpr int kMaxQ = 65536;
constexpr int kMaxBlocks = 65536;
constexpr int kMaxTop = 4096;

// ---------------------------------------------------------------- summaries

struct SummaryArgs {
    sv::PagedCache c;
    const int32_t* base;
    const int32_t* new_len;
    int N;
    unsigned blocks;  // blocks of a row that a call can touch
    uint16_t* out;
};

// The larger, and the smaller, of two pairs of bf16; NaN stays.
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min_pair(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// What a lane keeps of its eight elements: their sums, or their bounds as pairs of bf16.  (The largest of rounded
// values is the largest one rounded, so e4m3 values are rounded as they come, two an instruction.)
template <bool BOUNDS>
struct Kept {
    uint32_t a[BOUNDS ? 4 : 8], b[BOUNDS ? 4 : 1];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < (BOUNDS ? 4 : 8); ++k) a[k] = BOUNDS ? 0xff80ff80u : 0u;
#pragma unroll
        for (int k = 0; k < (BOUNDS ? 4 : 1); ++k) b[k] = 0x7f807f80u;
    }
    __device__ __forceinline__ void add(const float x[8]) {
        if (BOUNDS) {
#pragma unroll
            for (int k = 0; k < 4; ++k) pair(k, sv::bf16x2(x[2 * k], x[2 * k + 1]));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) a[BOUNDS ? 0 : k] = __float_as_uint(__uint_as_float(a[BOUNDS ? 0 : k]) + x[k]);
        }
    }
    __device__ __forceinline__ void pair(int k, uint32_t w) {
        a[k] = max_pair(a[k], w);
        b[BOUNDS ? k : 0] = min_pair(b[BOUNDS ? k : 0], w);
    }
    __device__ __forceinline__ void join(const Kept& o) {
        if (BOUNDS) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                a[k] = max_pair(a[k], o.a[k]);
                b[BOUNDS ? k : 0] = min_pair(b[BOUNDS ? k : 0], o.b[BOUNDS ? k : 0]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) a[BOUNDS ? 0 : k] = __float_as_uint(__uint_as_float(a[BOUNDS ? 0 : k]) + __uint_as_float(o.a[BOUNDS ? 0 : k]));
        }
    }
    __device__ __forceinline__ Kept from(int mask) const {
        Kept o;
#pragma unroll
        for (int k = 0; k < (BOUNDS ? 4 : 8); ++k) o.a[k] = __shfl_xor_sync(0xffffffffu, a[k], mask);
#pragma unroll
        for (int k = 0; k < (BOUNDS ? 4 : 1); ++k) o.b[k] = BOUNDS ? __shfl_xor_sync(0xffffffffu, b[k], mask) : 0u;
        return o;
    }
};

// Eight bf16 to a summary's row.
__device__ __forceinline__ void store_pairs(uint16_t* row, int e0, int dim, const uint32_t w[4]) {
    if (dim % 8 == 0) {
        if (e0 < dim) *reinterpret_cast<uint4*>(row + e0) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (e0 + k < dim) row[e0 + k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
    }
}

// grid: x over blocks * heads of one batch row, y the batch row.  WPU warps take one of them.
template <int LPR, bool E4M3, bool BOUNDS, bool AL, int WPU>
__global__ void __launch_bounds__(kThreads) block_summary_kernel(const __grid_constant__ SummaryArgs a) {
    constexpr int G = 32 / LPR, FLY = E4M3 || BOUNDS ? 8 : 4;  // keys of a warp at a time, and how many a lane has in flight
    __shared__ Kept<BOUNDS> s_kept[WPU > 1 ? kWarps : 1][LPR];
    sv::pdl_trigger();
    sv::pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % WPU, e0 = 8 * (lane % LPR);
    const unsigned heads = a.c.heads, unit = blockIdx.x * (unsigned)(kWarps / WPU) + warp / WPU;
    int first, n;
    if (!sv::paged_row(a.c, a.base, a.new_len, blockIdx.y, a.N, first, n) || n == 0) return;
    const int block = first / a.c.page_size + (int)(unit / heads), h = (int)(unit % heads);
    const int64_t start = (int64_t)block * a.c.page_size;
    const bool real = unit / heads < a.blocks && start < first + n;
    int page = -1, row = 0, count = 0;
    if (real) {
        page = sv::paged_place(a.c, blockIdx.y, (int)start, row);
        count = min(a.c.page_size, (int)(first + n - start));
    }
    if (page < 0) count = 0;
    const int64_t at = (page < 0 ? 0 : page) * a.c.page_stride + h * a.c.head_stride;
    const int64_t sc = ((int64_t)(page < 0 ? 0 : page) * heads + h) * a.c.page_size;
    Kept<BOUNDS> kept;
    kept.clear();
    for (int r0 = part * G + lane / LPR; r0 < count; r0 += FLY * G * WPU) {
        sv::EightOfCache<E4M3, AL> x[FLY];
        float scale[FLY];
#pragma unroll
        for (int k = 0; k < FLY; ++k) {
            const int r = r0 + k * G * WPU;
            scale[k] = 1.0f;
            if (r < count) {
                x[k].load(a.c.k + at + r * a.c.row_stride, e0, a.c.dim);
                if (E4M3) scale[k] = __ldg(a.c.k_scale + sc + r);
            }
        }
#pragma unroll
        for (int k = 0; k < FLY; ++k) {
            if (r0 + k * G * WPU >= count) break;
            if constexpr (BOUNDS && !E4M3 && AL) {
                const uint4 w = x[k].b.w[0];
                kept.pair(0, w.x);
                kept.pair(1, w.y);
                kept.pair(2, w.z);
                kept.pair(3, w.w);
            } else {
                float f[8];
                x[k].widen(scale[k], f);
                kept.add(f);
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int x = LPR; x < 32; x <<= 1) kept.join(kept.from(x));
    if (WPU > 1) {
        if (lane < LPR) s_kept[WPU > 1 ? warp : 0][lane] = kept;
        __syncthreads();
        if (part) return;
        for (int w = 1; w < WPU; ++w)
            if (lane < LPR) kept.join(s_kept[WPU > 1 ? warp + w : 0][lane]);
    }
    if (page < 0 || lane >= LPR) return;
    const int dim = a.c.dim;
    uint16_t* out = a.out + ((int64_t)page * heads + h) * (BOUNDS ? 2 * dim : dim);
    if (BOUNDS) {
        store_pairs(out, e0, dim, kept.a);
        store_pairs(out + dim, e0, dim, kept.b);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = sv::bf16x2(__uint_as_float(kept.a[BOUNDS ? 0 : 2 * k]) / (float)count, __uint_as_float(kept.a[BOUNDS ? 0 : 2 * k + 1]) / (float)count);
        store_pairs(out, e0, dim, w);
    }
}

template <int LPR, bool E4M3, bool BOUNDS, bool AL>
cudaError_t summary_lpr(const SummaryArgs& a, int B, cudaStream_t s) {
    const int64_t units = (int64_t)a.blocks * a.c.heads;
    // Eight warps a block where that many do not fill the device.
    if (units * B < 152 * 16 && a.c.page_size > 4)
        return sv::launch_serial(block_summary_kernel<LPR, E4M3, BOUNDS, AL, kWarps>, dim3((unsigned)units, (unsigned)B), dim3(kThreads), 0, s, a);
    return sv::launch_serial(block_summary_kernel<LPR, E4M3, BOUNDS, AL, 1>, dim3((unsigned)((units + kWarps - 1) / kWarps), (unsigned)B),
                             dim3(kThreads), 0, s, a);
}

template <bool E4M3, bool BOUNDS>
cudaError_t summary_dim(const SummaryArgs& a, bool al, int B, cudaStream_t s) {
    if (!al) return summary_lpr<32, E4M3, BOUNDS, false>(a, B, s);
    if (a.c.dim <= 64) return summary_lpr<8, E4M3, BOUNDS, true>(a, B, s);
    if (a.c.dim <= 128) return summary_lpr<16, E4M3, BOUNDS, true>(a, B, s);
    return summary_lpr<32, E4M3, BOUNDS, true>(a, B, s);
}

// ------------------------------------------------------------------- scores

struct SelectArgs {
    const uint16_t* q;  // bf16, element strides below
    int64_t q_sb, q_st, q_sh;
    const uint16_t* summary;  // [num_pages][H][D or 2 D]
    const int32_t* table;
    const int32_t* base;
    const int32_t* new_len;
    int num_pages, page_size, max_pages, H, D, Q, g;
    int gp;      // rows of a query: its heads, padded to a power of two, or to a multiple of 8
    int shift;   // log2 of gp where it is 8 or less
    int span;    // tiles of eight rows of a query: 1 where gp is 8 or less
    int lists;   // per batch row and head: Q, or 1 where shared
    int width;   // scores of a list in the workspace
    int top, sink, recent;
    uint32_t* key;  // [B][lists][H][width]: the scores, as key32
    float* norm;    // [B][lists][H]: the largest |q|_1 of the list's rows
    float* biggest; // [B][H][max_pages / 16]: the largest |m| of 16 blocks
    int32_t* out;   // [B][lists][H][top]
};

// Real queries and context blocks of batch row b (no queries where it is left untouched).
__device__ __forceinline__ void select_row(const SelectArgs& a, int b, int& n, int& blocks) {
    const int base = __ldg(a.base + b);
    n = a.new_len ? __ldg(a.new_len + b) : a.Q;
    blocks = 0;
    if (base < 0 || n < 0 || n > a.Q || (int64_t)base + n > (int64_t)a.max_pages * a.page_size) n = 0;
    else blocks = base / a.page_size;
}

// Keys in the order of the numbers, 0 for a block in a hole (no number's key).
__device__ __forceinline__ uint32_t key32(float x) {
    const uint32_t bits = __float_as_uint(x);
    return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
}
__device__ __forceinline__ float from_key32(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key); }
// 1 for NaN: below -infinity.
__device__ __forceinline__ uint64_t key64(double x) {
    if (x != x) return 1;
    const uint64_t bits = (uint64_t)__double_as_longlong(x);
    return bits >> 63 ? ~bits : bits | 0x8000000000000000ull;
}

__device__ __forceinline__ void mma16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The positive parts, or the negative ones, of two bf16 (of NaN anything: such rows are summed again).
__device__ __forceinline__ uint32_t part_of(uint32_t w, bool negative) {
    uint32_t r;
    if (negative) asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0u));
    else asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0u));
    return r;
}

// The larger magnitudes of two pairs of bf16, of any sign; NaN stays.
__device__ __forceinline__ uint32_t larger_magnitudes(uint32_t a, uint32_t w) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(w));
    return r;
}

__device__ __forceinline__ float magnitudes(uint4 w) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) s += fabsf(sv::bf16_lo(x[k])) + fabsf(sv::bf16_hi(x[k]));
    return s;
}

constexpr int kScoreWarps = 4;

// grid: x over the blocks, 16 per warp, y the batch row and cache head.  KC: chunks of 32 elements, whole
// ones where FULL; NQ: tiles of eight query rows multiplied at a time.  Blocks are the products' 16 rows
// and query rows their 8 columns, so that the heads that meet lie in neighbouring lanes.  A warp asks for
// all of its summaries at once and then does not wait for any other.
// (As a ring of copies in shared memory, two steps ahead, the scores of 32 chains of 6 took 53 us.)
template <int KC, bool BOUNDS, bool FULL, int NQ>
__global__ void __launch_bounds__(kScoreWarps * 32, KC * (BOUNDS ? 2 : 1) > 8 ? 2 : FULL ? 4 : 3) block_score_kernel(const __grid_constant__ SelectArgs a) {
    constexpr int MATS = BOUNDS ? 2 : 1;
    sv::pdl_trigger();
    sv::pdl_wait();
    const int lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
    const int y = blockIdx.y, b = y / a.H, h = y - b * a.H, unit = blockIdx.x * kScoreWarps + (threadIdx.x >> 5), j0 = 16 * unit;
    int pages[2];  // asked for beside the row's length
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int j = j0 + 8 * x + g8;
        pages[x] = j < a.max_pages ? __ldg(a.table + (int64_t)b * a.max_pages + j) : -1;
    }
    int n, blocks;
    select_row(a, b, n, blocks);
    // Lists that need no scores: all blocks, or only the first and last ones.
    if (n == 0 || j0 >= blocks || blocks <= a.top || a.sink + a.recent == a.top) return;
    const int D = FULL ? 32 * KC : a.D;
    uint4 m[2][MATS][KC];  // of blocks j0 + g8 and 8 more
    bool hole[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int j = j0 + 8 * x + g8;
        const int page = j < blocks ? pages[x] : -1;
        hole[x] = (unsigned)page >= (unsigned)a.num_pages;
        const uint16_t* row = a.summary + ((int64_t)(hole[x] ? 0 : page) * a.H + h) * (D * MATS) + 8 * t4;
#pragma unroll
        for (int z = 0; z < MATS; ++z)
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                if (FULL) {
                    m[x][z][k] = sv::ld_nc_v4(row + z * D + 32 * k);  // of page 0 in a hole
                } else {
                    m[x][z][k] = make_uint4(0u, 0u, 0u, 0u);
                    if (32 * k + 8 * t4 < D) m[x][z][k] = sv::ld_nc_v4(row + z * D + 32 * k);
                }
            }
    }
    const bool count = j0 == 0;  // one warp per row and head also sums |q|
    const bool shared = a.lists != a.Q || a.Q == 1;
    const int tiles = (n * a.gp + 7) / 8;
    const uint16_t* q0 = a.q + b * a.q_sb + (int64_t)(h * a.g) * a.q_sh + 8 * t4;
    float run[2] = {neg_inf(), neg_inf()}, run_norm = 0.0f;  // of blocks g8 and g8 + 8: over tiles where they meet
    for (int t0 = 0; t0 < tiles; t0 += NQ) {
        // The row of this lane's column in each tile; rows are queries times gp heads, the last head repeated.
        const uint16_t* from[NQ];
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
            const int tile = t0 + t;
            const int i = a.gp <= 8 ? (8 * tile + g8) >> a.shift : tile / a.span;
            const int head = a.gp <= 8 ? g8 & (a.gp - 1) : 8 * (tile - i * a.span) + g8;
            from[t] = q0 + (i < n ? i : 0) * a.q_st + min(head, a.g - 1) * a.q_sh;
        }
        float acc[NQ][4], norm[NQ];
#pragma unroll
        for (int t = 0; t < NQ; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = norm[t] = 0.0f;
#pragma unroll
        for (int k0 = 0; k0 < KC; k0 += 2) {
            uint4 q[NQ][2];
#pragma unroll
            for (int t = 0; t < NQ; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int e = 32 * (k0 + k);
                    if (FULL) {
                        q[t][k] = __ldg(reinterpret_cast<const uint4*>(from[t] + e));
                    } else {
                        q[t][k] = make_uint4(0u, 0u, 0u, 0u);
                        if (e + 8 * t4 < D) q[t][k] = __ldg(reinterpret_cast<const uint4*>(from[t] + e));
                    }
                    if (count) norm[t] += magnitudes(q[t][k]);
                }
#pragma unroll
            for (int z = 0; z < MATS; ++z) {
                float part[NQ][4];  // chains of four products
#pragma unroll
                for (int t = 0; t < NQ; ++t) part[t][0] = part[t][1] = part[t][2] = part[t][3] = 0.0f;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint4 m0 = m[0][z][k0 + k], m1 = m[1][z][k0 + k];
                    auto of = [&](uint32_t w) { return BOUNDS ? part_of(w, z == 1) : w; };
#pragma unroll
                    for (int t = 0; t < NQ; ++t) {
                        mma16816(part[t], m0.x, m1.x, m0.y, m1.y, of(q[t][k].x), of(q[t][k].y));
                        mma16816(part[t], m0.z, m1.z, m0.w, m1.w, of(q[t][k].z), of(q[t][k].w));
                    }
                }
#pragma unroll
                for (int t = 0; t < NQ; ++t)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[t][v] += part[t][v];
            }
        }
        // Columns that meet: gp neighbours, those of several tiles where gp is above 8, or all.
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
            const int tile = t0 + t;
            if (tile >= tiles) break;
            const int i = a.gp <= 8 ? (8 * tile + 2 * t4) >> a.shift : tile / a.span, i1 = a.gp == 1 ? i + 1 : i;
            const bool fresh = !shared && (a.gp <= 8 || tile % a.span == 0);
            const bool last = shared ? tile == tiles - 1 : a.gp <= 8 || tile % a.span == a.span - 1;
            if (count) {
                auto meet = [](float p, float q) { return p > q || !(p == p) ? p : q; };  // NaN stays
                float w = norm[t];
                w += __shfl_xor_sync(0xffffffffu, w, 1);
                w += __shfl_xor_sync(0xffffffffu, w, 2);  // of the row in column g8
                const int own = a.gp <= 8 ? (8 * tile + g8) >> a.shift : i;
                if (own >= n) w = 0.0f;
                run_norm = fresh ? w : meet(w, run_norm);
                w = run_norm;
                if (shared || a.gp >= 2) w = meet(w, __shfl_xor_sync(0xffffffffu, w, 4));
                if (shared || a.gp >= 4) w = meet(w, __shfl_xor_sync(0xffffffffu, w, 8));
                if (shared || a.gp >= 8) w = meet(w, __shfl_xor_sync(0xffffffffu, w, 16));
                if (last && t4 == 0 && own < n && (shared ? g8 == 0 : (g8 & (a.gp - 1) & 7) == 0)) a.norm[((int64_t)b * a.lists + (shared ? 0 : own)) * a.H + h] = w;
            }
            float u0 = i < n ? acc[t][0] : neg_inf(), u1 = i1 < n ? acc[t][1] : neg_inf();
            float v0 = i < n ? acc[t][2] : neg_inf(), v1 = i1 < n ? acc[t][3] : neg_inf();
            if (shared || a.gp >= 2) {
                u0 = fmaxf(u0, u1);
                v0 = fmaxf(v0, v1);
                run[0] = fresh ? u0 : fmaxf(run[0], u0);
                run[1] = fresh ? v0 : fmaxf(run[1], v0);
                if (!last) continue;
                u0 = run[0];
                v0 = run[1];
                if (shared || a.gp >= 4) {
                    u0 = fmaxf(u0, __shfl_xor_sync(0xffffffffu, u0, 1));
                    v0 = fmaxf(v0, __shfl_xor_sync(0xffffffffu, v0, 1));
                }
                if (shared || a.gp >= 8) {
                    u0 = fmaxf(u0, __shfl_xor_sync(0xffffffffu, u0, 2));
                    v0 = fmaxf(v0, __shfl_xor_sync(0xffffffffu, v0, 2));
                }
                if (!shared && a.gp == 4 ? t4 & 1 : (shared || a.gp >= 8) && t4) continue;
            }
            uint32_t* to = a.key + (((int64_t)b * a.lists + (shared ? 0 : i)) * a.H + h) * a.width + j0 + g8;
            auto put = [&](uint32_t* to, float u, float v) {  // + 0: -0 is 0
                if (j0 + g8 < blocks) to[0] = hole[0] ? 0u : key32(u + 0.0f);
                if (j0 + g8 + 8 < blocks) to[8] = hole[1] ? 0u : key32(v + 0.0f);
            };
            if (i < n) put(to, u0, v0);
            if (!shared && a.gp == 1 && i1 < n) put(to + (int64_t)a.H * a.width, u1, v1);
        }
    }
    uint32_t most = 0u;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int z = 0; z < MATS; ++z)
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                if (hole[x]) continue;
                most = larger_magnitudes(larger_magnitudes(most, m[x][z][k].x), m[x][z][k].y);
                most = larger_magnitudes(larger_magnitudes(most, m[x][z][k].z), m[x][z][k].w);
            }
    most = __reduce_max_sync(0xffffffffu, max(most & 0x7fffu, (most >> 16) & 0x7fffu));
    if (lane == 0) a.biggest[(int64_t)y * ((a.max_pages + 15) / 16) + unit] = __uint_as_float(most << 16);
}

// ---------------------------------------------------------------- selection

constexpr int kFew = 64;     // blocks next to the border whose 64-bit scores are compared with one another
constexpr int kAtOnce = 4;   // query rows that a warp has in flight as it sums again (32 chains of 6: 46 us; one 47, eight 52)
constexpr int kKept = 8192;  // blocks whose keys are kept in shared memory

struct SelectShared {
    uint32_t hist[4][256];
    uint32_t in, unsure, few_n, lost;
    int few[kFew];
    uint64_t few_key[kFew];
    uint64_t best[kWarps];
    uint32_t biggest[kWarps], sums[kWarps];
};

// Whether every score is zero.  (Not where the product is: that of 2^-80 and 2^-80 is, in fp32.)
__device__ __forceinline__ bool all_scores_zero(float norm, float biggest) {
    return (norm == 0.0f && biggest < pos_inf()) || (biggest == 0.0f && norm < pos_inf());
}

// What the sums in 64 bits go by: 2^a with |q|_1 max|m| 2^a below 2^30, or 0 where that bound is not finite, or
// so large or small that products may leave fp32's range.
__device__ __forceinline__ float fixed_scale(float reach) {
    return reach >= 0x1p-60f && reach < 0x1p120f ? __uint_as_float((127u + 29u + 127u - (__float_as_uint(reach) >> 23)) << 23) : 0.0f;
}

// The key of score(i, j) in 64 bits over rows r0, r0 + step, ... of the list's (i1 - i0) * g, by one warp, the
// result in all lanes; ~0 where one of them is NaN.  A product has 16 bits and is exact in fp32; it is added
// up in fixed point, 30 bits and 22 more behind them, each in integers of 32 bits: exact in any order, and as a
// sum of doubles would be, as long as no product has bits below those.  One that may, below 2^-37 of |q|_1 max|m|,
// sets `lost` in its lane, and the list is summed again by doubles (scale 0), as where products may leave fp32's
// range.  The SM adds two of them a clock: with them throughout, 1536 lists of up to 1024 blocks took 27 us longer.
template <bool BOUNDS>
__device__ __forceinline__ uint64_t exact_rows(const SelectArgs& a, float scale, int b, int i0, int i1, int h, int j, int r0, int step, bool& lost) {
    const int lane = threadIdx.x & 31;
    const int page = __ldg(a.table + (int64_t)b * a.max_pages + j);
    const uint16_t* m = a.summary + ((int64_t)page * a.H + h) * (a.D * (BOUNDS ? 2 : 1));
    const int rows = (i1 - i0) * a.g;
    auto two = [](const uint16_t* p) { return __ldg(reinterpret_cast<const uint32_t*>(p)); };
    uint32_t hi[4], lo[BOUNDS ? 4 : 1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int d = 2 * lane + 64 * k;
        hi[k] = d < a.D ? two(m + d) : 0u;
        if (BOUNDS) lo[BOUNDS ? k : 0] = d < a.D ? two(m + a.D + d) : 0u;
    }
    uint64_t best = 0;
    bool nan = false;
    for (int r1 = r0; r1 < rows; r1 += kAtOnce * step) {  // rows whose loads are in flight together
        uint32_t rows_x[kAtOnce][4];
#pragma unroll
        for (int f = 0; f < kAtOnce; ++f) {
            const int r = r1 + f * step < rows ? r1 + f * step : r1;  // (a row twice does no harm)
            const uint16_t* q = a.q + b * a.q_sb + (i0 + r / a.g) * a.q_st + (int64_t)(h * a.g + r % a.g) * a.q_sh;
#pragma unroll
            for (int k = 0; k < 4; ++k) rows_x[f][k] = 2 * lane + 64 * k < a.D ? two(q + 2 * lane + 64 * k) : 0u;
        }
#pragma unroll
        for (int f = 0; f < kAtOnce; ++f) {
            const uint32_t (&x)[4] = rows_x[f];
            auto factors = [&](int e, float& u, float& w) {  // q_d and m_d of the lane's element e
                u = e & 1 ? sv::bf16_hi(x[e / 2]) : sv::bf16_lo(x[e / 2]);
                const uint32_t y = BOUNDS && !(u >= 0.0f) ? lo[BOUNDS ? e / 2 : 0] : hi[e / 2];
                w = e & 1 ? sv::bf16_hi(y) : sv::bf16_lo(y);
            };
            uint64_t key;
            if (scale != 0.0f) {
                int upper = 0, lower = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float u, w;
                    factors(e, u, w);
                    const float p = u * w * scale;
                    lost |= fabsf(p) < 0x1p-7f && u != 0.0f && w != 0.0f;
                    const int n = __float2int_rn(p);
                    upper += n;
                    lower += __float2int_rn((p - (float)n) * 0x1p22f);
                }
                upper = __reduce_add_sync(0xffffffffu, upper);
                lower = __reduce_add_sync(0xffffffffu, lower);
                key = (uint64_t)((int64_t)upper * (1 << 22) + lower) ^ 0x8000000000000000ull;
            } else {
                double s = 0.0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float u, w;
                    factors(e, u, w);
                    if (2 * lane + 64 * (e / 2) < a.D) s = fma((double)u, (double)w, s);
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (s != s) nan = true;
                key = key64(s == 0.0 ? 0.0 : s);  // -0 is 0
            }
            if (key > best) best = key;
        }
    }
    return nan ? ~0ull : best;
}

// Over all rows; NaN has key 1.  By one warp, or by all of the CTA's.
template <bool BOUNDS>
__device__ __forceinline__ uint64_t exact_key(const SelectArgs& a, float scale, int b, int i0, int i1, int h, int j, bool& lost) {
    const uint64_t best = exact_rows<BOUNDS>(a, scale, b, i0, i1, h, j, 0, 1, lost);
    return best == ~0ull ? 1 : best;
}
template <bool BOUNDS>
__device__ __forceinline__ uint64_t exact_key_together(const SelectArgs& a, SelectShared& sh, float scale, int b, int i0, int i1, int h, int j, bool& lost) {
    const int warp = threadIdx.x >> 5;
    uint64_t best = exact_rows<BOUNDS>(a, scale, b, i0, i1, h, j, warp, kWarps, lost);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.best[warp] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (sh.best[w] > best) best = sh.best[w];
    return best == ~0ull ? 1 : best;
}

struct Edge {
    uint32_t key, left, equal;  // the want-th largest key, how many of those equal to it are wanted, how many there are
};

// The `want`-th largest key of blocks whose bit is set in `part`, by digits of eight bits.  Every warp
// looks for the digit by itself, so there is one barrier per digit.
template <typename Part>
__device__ __forceinline__ Edge radix_select(SelectShared& sh, const uint32_t* keys, int words, uint32_t want, Part part) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __syncthreads();
    for (int x = tid; x < 4 * 256; x += kThreads) (&sh.hist[0][0])[x] = 0u;
    __syncthreads();
    Edge e{0u, want, 0u};
#pragma unroll
    for (int digit = 0; digit < 4; ++digit) {
        const int shift = 24 - 8 * digit;
        for (int w = warp; w < words; w += kWarps) {
            const bool mine = (part(w) >> lane) & 1u;
            const uint32_t k = mine ? keys[32 * w + lane] : 0u;
            const bool count = mine && (digit == 0 || (k >> (shift + 8)) == (e.key >> (shift + 8)));
            const uint32_t bin = (k >> shift) & 255u;
            if (digit == 0) {  // few different first digits: one addition for all lanes that have the same
                const uint32_t same = __match_any_sync(0xffffffffu, count ? bin : 256u);
                if (count && lane == __ffs(same) - 1) atomicAdd(&sh.hist[digit][bin], (uint32_t)__popc(same));
            } else if (count) {
                atomicAdd(&sh.hist[digit][bin], 1u);
            }
        }
        __syncthreads();
        const int top = 255 - 8 * lane;  // a lane has eight bins, from the top
        uint32_t c[8], own = 0u;
#pragma unroll
        for (int x = 0; x < 8; ++x) own += c[x] = sh.hist[digit][top - x];
        uint32_t sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        uint32_t before = sum - own, at = 0u, equal = c[0];
        const bool here = before < e.left && e.left <= sum;
#pragma unroll
        for (int y = 0; y < 7; ++y)
            if (at == y && before + c[y] < e.left) {
                before += c[y];
                at = y + 1;
                equal = c[y + 1];
            }
        const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        e.key |= __shfl_sync(0xffffffffu, (uint32_t)(top - (int)at), from) << shift;
        e.left -= __shfl_sync(0xffffffffu, before, from);
        e.equal = __shfl_sync(0xffffffffu, equal, from);
    }
    return e;
}

// One CTA per list.  A warp takes 32 blocks at a time, so that what it decides on them is a word of a bitmap.
// (Three CTAs an SM, 80 registers: left to itself the compiler takes 64 for bounds and spills.)
template <bool BOUNDS>
__global__ void __launch_bounds__(kThreads, 3) block_select_kernel(const __grid_constant__ SelectArgs a) {
    extern __shared__ uint32_t s_bits[];  // [words] blocks that are in, [words] not yet decided, then keys
    __shared__ SelectShared sh;
    sv::pdl_trigger();
    sv::pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned list = blockIdx.x;
    const int h = (int)(list % (unsigned)a.H), bi = (int)(list / (unsigned)a.H), i = bi % a.lists, b = bi / a.lists;
    int n, blocks;
    select_row(a, b, n, blocks);
    int32_t* out = a.out + (int64_t)list * a.top;
    if (n == 0 || (a.lists > 1 && i >= n) || blocks <= a.top) {
        const int have = n == 0 || (a.lists > 1 && i >= n) ? 0 : blocks;
        for (int x = tid; x < a.top; x += kThreads) out[x] = x < have ? x : -1;
        return;
    }
    const int words = (blocks + 31) / 32;
    uint32_t* s_in = s_bits;
    uint32_t* s_unsure = s_bits + words;
    const int from = a.sink, to = blocks - a.recent;  // candidates
    // bits of word w that are candidates, and that are blocks at all
    auto below = [](int w, int end) { const int x = end - 32 * w; return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1u; };
    auto candidates = [&](int w) { return below(w, to) & ~below(w, from); };
    uint32_t want = (uint32_t)(a.top - a.sink - a.recent);
    if (want) {
        uint32_t* keys = a.key + (int64_t)list * a.width;
        uint32_t biggest = 0u;  // NaN (of a positive sign) is above all
        for (int x = tid; 16 * x < blocks; x += kThreads) biggest = max(biggest, __float_as_uint(a.biggest[((int64_t)b * a.H + h) * ((a.max_pages + 15) / 16) + x]));
        const float norm = a.norm[list];
        if (blocks <= kKept) {
            uint32_t* s_key = s_bits + 2 * words;
            for (int j = tid; j < blocks; j += kThreads) s_key[j] = keys[j];
            keys = s_key;
        }
        biggest = __reduce_max_sync(0xffffffffu, biggest);
        if (lane == 0) sh.biggest[warp] = biggest;
        if (tid == 0) sh.in = sh.unsure = sh.few_n = sh.lost = 0u;
        Edge edge = radix_select(sh, keys, words, want, candidates);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) biggest = max(biggest, sh.biggest[w]);
        const float reach = norm * __uint_as_float(biggest);  // |q|_1 max|m|
        const bool all_zero = all_scores_zero(norm, __uint_as_float(biggest));
        const float err = reach * 0x1p-16f;
        const float scale = fixed_scale(reach);
        const bool sure = reach >= 0x1p-100f && reach < 0x1p120f;  // else (NaN among them) every score is summed again
        const float t = from_key32(edge.key);
        const float low = __fadd_rd(t, -2.0f * err), high = __fadd_ru(t, 2.0f * err);
        uint32_t in = 0u, unsure = 0u;
        for (int w = warp; w < words; w += kWarps) {
            const uint32_t part = candidates(w);
            const bool mine = (part >> lane) & 1u;
            const uint32_t k = mine ? keys[32 * w + lane] : 0u;
            const float v = from_key32(k);
            bool yes, maybe;
            if (edge.key == 0u) {  // fewer blocks than wanted are in no hole
                yes = k > 0u;
                maybe = mine && k == 0u;
            } else {
                yes = k > 0u && sure && v > high;
                maybe = k > 0u && !yes && (!sure || v >= low);
            }
            const uint32_t y = __ballot_sync(0xffffffffu, yes), m = __ballot_sync(0xffffffffu, maybe);
            in += __popc(y);
            unsure += __popc(m);
            if (lane == 0) {
                s_in[w] = y | (below(w, blocks) & ~part);
                s_unsure[w] = m;
            }
        }
        if (lane == 0 && in) atomicAdd(&sh.in, in);
        if (lane == 0 && unsure) atomicAdd(&sh.unsure, unsure);
        __syncthreads();
        want -= sh.in;
        uint32_t some = sh.unsure;
        const int i0 = a.lists > 1 ? i : 0, i1 = a.lists > 1 ? i + 1 : n;
        auto open = [&](int w) { return s_unsure[w]; };
        const bool again = edge.key != 0u && !all_zero;  // (holes are all alike)
        if (want < some && again && some <= kFew) {
            for (int w = tid; w < words; w += kThreads)
                for (uint32_t bits = s_unsure[w]; bits; bits &= bits - 1u)
                    sh.few[atomicAdd(&sh.few_n, 1u)] = 32 * w + __ffs(bits) - 1;  // in any order: ranked by key and index
            __syncthreads();
            for (float by = scale;; by = 0.0f) {
                bool lost = false;
                if ((i1 - i0) * a.g <= 2 * kWarps) {
                    for (uint32_t x = warp; x < some; x += kWarps) {
                        const uint64_t k = exact_key<BOUNDS>(a, by, b, i0, i1, h, sh.few[x], lost);
                        if (lane == 0) sh.few_key[x] = k;
                    }
                } else {
                    for (uint32_t x = 0; x < some; ++x) {
                        const uint64_t k = exact_key_together<BOUNDS>(a, sh, by, b, i0, i1, h, sh.few[x], lost);
                        if (tid == 0) sh.few_key[x] = k;
                    }
                }
                if (lost) sh.lost = 1u;
                __syncthreads();
                if (by == 0.0f || !sh.lost) break;
            }
            if (tid < (int)some) {
                const uint64_t k = sh.few_key[tid];
                const int j = sh.few[tid];
                uint32_t before = 0u;
                for (uint32_t x = 0; x < some; ++x) before += sh.few_key[x] > k || (sh.few_key[x] == k && sh.few[x] < j);
                if (before < want) atomicOr(&s_in[j >> 5], 1u << (j & 31));
            }
            want = 0u;
        } else if (want < some && again) {
            float by = scale;
            for (int half = 0; half < 2 && want < some; ++half) {
                bool lost = false;
                for (int w = 0; w < words; ++w) {
                    for (uint32_t bits = s_unsure[w]; bits; bits &= bits - 1u) {
                        const int j = 32 * w + __ffs(bits) - 1;
                        if (j % kWarps != warp) continue;
                        const uint64_t k = exact_key<BOUNDS>(a, by, b, i0, i1, h, j, lost);
                        if (lane == 0) keys[j] = half ? (uint32_t)k : (uint32_t)(k >> 32);
                    }
                }
                if (by != 0.0f && half == 0) {
                    if (lost) sh.lost = 1u;
                    __syncthreads();
                    if (sh.lost) {  // from the start, by doubles
                        by = 0.0f;
                        half = -1;
                        continue;
                    }
                }
                edge = radix_select(sh, keys, words, want, open);
                want = edge.left;
                some = edge.equal;
                for (int w = warp; w < words; w += kWarps) {
                    const uint32_t part = s_unsure[w], k = (part >> lane) & 1u ? keys[32 * w + lane] : 0u;
                    const uint32_t above = __ballot_sync(0xffffffffu, k > edge.key), same = __ballot_sync(0xffffffffu, k == edge.key);
                    if (lane == 0) {
                        s_in[w] |= above & part;
                        s_unsure[w] = same & part;
                    }
                }
                __syncthreads();
            }
        }
        __syncthreads();
        if (want && warp == 0) {  // equals, the lowest first: all of them, or the first `want`
            uint32_t left = want;
            for (int w0 = 0; w0 < words && left; w0 += 32) {
                const int w = w0 + lane;
                uint32_t mine = w < words ? s_unsure[w] : 0u;
                uint32_t sum = __popc(mine), before = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                before = sum - before;
                uint32_t keep = 0u;
                for (uint32_t c = before; mine && c < left; ++c) {
                    keep |= mine & (0u - mine);
                    mine &= mine - 1u;
                }
                if (w < words) s_in[w] |= keep;
                const uint32_t all = __shfl_sync(0xffffffffu, sum, 31);
                left = all < left ? left - all : 0u;
            }
        }
    } else {
        for (int w = tid; w < words; w += kThreads) s_in[w] = below(w, blocks) & ~candidates(w);
    }
    __syncthreads();
    // the list, in ascending order: a thread's words follow the threads' before it
    const int each = (words + kThreads - 1) / kThreads, w0 = min(words, tid * each), w1 = min(words, w0 + each);
    uint32_t own = 0u;
    for (int w = w0; w < w1; ++w) own += __popc(s_in[w]);
    uint32_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) sh.sums[warp] = sum;
    __syncthreads();
    uint32_t at = sum - own;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warp) at += sh.sums[w];
    for (int w = w0; w < w1; ++w)
        for (uint32_t bits = s_in[w]; bits; bits &= bits - 1u, ++at)
            if (at < (uint32_t)a.top) out[at] = 32 * w + __ffs(bits) - 1;
}

// One warp per list of up to 32 * KPL blocks: the keys stay in registers, and the want-th largest is found by
// halving the range of keys.  1536 lists of 256 to 1024 blocks take about 20 us.
template <bool BOUNDS, int KPL>
__global__ void __launch_bounds__(128) block_select_warp_kernel(const __grid_constant__ SelectArgs a, const unsigned lists) {
    constexpr int WPL = (KPL + 31) / 32;  // words of a bitmap that a lane keeps: word 32 x + lane
    sv::pdl_trigger();
    sv::pdl_wait();
    const int lane = threadIdx.x & 31;
    const unsigned list = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (list >= lists) return;
    const int h = (int)(list % (unsigned)a.H), bi = (int)(list / (unsigned)a.H), i = bi % a.lists, b = bi / a.lists;
    int n, blocks;
    select_row(a, b, n, blocks);
    int32_t* out = a.out + (int64_t)list * a.top;
    if (n == 0 || (a.lists > 1 && i >= n) || blocks <= a.top) {
        const int have = n == 0 || (a.lists > 1 && i >= n) ? 0 : blocks;
        for (int x = lane; x < a.top; x += 32) out[x] = x < have ? x : -1;
        return;
    }
    const int from = a.sink, to = blocks - a.recent;  // candidates
    int want = a.top - a.sink - a.recent;
    uint32_t in[WPL], maybe[WPL];
#pragma unroll
    for (int x = 0; x < WPL; ++x) {  // the first and last blocks
        const int j = 32 * (32 * x + lane);
        auto below = [&](int end) { const int y = end - j; return y <= 0 ? 0u : y >= 32 ? ~0u : (1u << y) - 1u; };
        in[x] = below(blocks) & ~(below(to) & ~below(from));
        maybe[x] = 0u;
    }
    if (want) {
        uint32_t* keys = a.key + (int64_t)list * a.width;
        // Blocks that are no candidates have key 0 and are left out of the counts by `floor`.
        uint32_t key[KPL];
#pragma unroll
        for (int x = 0; x < KPL; ++x) {
            const int j = 32 * x + lane;
            key[x] = j >= from && j < to ? __ldg(keys + j) : 0u;
        }
        uint32_t biggest = 0u;
        for (int x = lane; 16 * x < blocks; x += 32) biggest = max(biggest, __float_as_uint(a.biggest[((int64_t)b * a.H + h) * ((a.max_pages + 15) / 16) + x]));
        biggest = __reduce_max_sync(0xffffffffu, biggest);
        const float norm = a.norm[list];
        // The want-th largest of the keys above 0; 0 where there are fewer.  The range is cut where the count
        // would lie if the keys' numbers were spread evenly, and in half, in turn.
        auto search = [&](int want, bool numbers) {
            uint32_t hi = 0u, lo = ~0u;
#pragma unroll
            for (int x = 0; x < KPL; ++x) {
                hi = max(hi, key[x]);
                lo = min(lo, key[x] - 1u);  // of keys above 0
            }
            hi = __reduce_max_sync(0xffffffffu, hi);
            lo = __reduce_min_sync(0xffffffffu, lo) + 1u;
            if (hi == 0u) return 0u;
            auto count = [&](uint32_t k) {  // keys of at least k
                int c = 0;
#pragma unroll
                for (int x0 = 0; x0 < KPL; x0 += 8) {
                    if (32 * x0 >= blocks) break;
#pragma unroll
                    for (int x = x0; x < x0 + 8; ++x) c += key[x] >= k;
                }
                return (int)__reduce_add_sync(0xffffffffu, c);
            };
            int at_lo = count(lo), above_hi = 0;  // keys >= lo, keys > hi
            if (at_lo < want) return 0u;
            for (int turn = 0; lo < hi; ++turn) {
                uint32_t mid = lo + (hi - lo) / 2u + 1u;
                if (numbers) {
                    const float u = from_key32(lo), v = from_key32(hi);
                    const float w = u + (v - u) * (turn & 1 ? 0.5f : ((float)(at_lo - want) + 0.5f) / (float)(at_lo - above_hi));
                    if (w > u && w < v) mid = max(key32(w), lo + 1u);  // false for NaN
                }
                const int c = count(mid);
                if (c >= want) {
                    lo = mid;
                    at_lo = c;
                } else {
                    hi = mid - 1u;
                    above_hi = c;
                }
                if (c == want) {  // the smallest of them is it
                    uint32_t least = ~0u;
#pragma unroll
                    for (int x = 0; x < KPL; ++x)
                        if (key[x] >= mid) least = min(least, key[x]);
                    return __reduce_min_sync(0xffffffffu, least);
                }
            }
            return lo;
        };
        // Keys above `high` are in, those from `low` on are open; returns how many are open.
        auto sort_out = [&](uint32_t low, uint32_t high) {
            uint32_t more[WPL];
#pragma unroll
            for (int x = 0; x < WPL; ++x) more[x] = maybe[x] = 0u;
#pragma unroll
            for (int x0 = 0; x0 < KPL; x0 += 8) {
                if (32 * x0 >= blocks) break;
#pragma unroll
                for (int x = x0; x < x0 + 8; ++x) {
                    const uint32_t y = __ballot_sync(0xffffffffu, key[x] > high), m = __ballot_sync(0xffffffffu, key[x] >= low);
                    if (lane == (x & 31)) {
                        more[x >> 5] = y;
                        maybe[x >> 5] = m & ~y;
                    }
                }
            }
            int taken = 0, open = 0;
#pragma unroll
            for (int x = 0; x < WPL; ++x) {
                in[x] |= more[x];
                taken += __popc(more[x]);
                open += __popc(maybe[x]);
            }
            want -= (int)__reduce_add_sync(0xffffffffu, taken);
            return (int)__reduce_add_sync(0xffffffffu, open);
        };
        const uint32_t edge = search(want, true);
        const float reach = norm * __uint_as_float(biggest);  // |q|_1 max|m|
        const bool all_zero = all_scores_zero(norm, __uint_as_float(biggest));
        const float err = reach * 0x1p-16f, t = from_key32(edge);
        const float scale = fixed_scale(reach);
        const bool sure = reach >= 0x1p-100f && reach < 0x1p120f;  // else (NaN among them) every score is summed again
        int some;
        if (edge == 0u) {  // fewer blocks than wanted are in no hole: holes follow, the lowest first
            some = sort_out(1u, 0u);
#pragma unroll
            for (int x = 0; x < WPL; ++x) {
                const int j = 32 * (32 * x + lane);
                auto below = [&](int end) { const int y = end - j; return y <= 0 ? 0u : y >= 32 ? ~0u : (1u << y) - 1u; };
                maybe[x] = below(to) & ~below(from) & ~in[x];
            }
            some = want;
        } else {
            some = sure ? sort_out(key32(__fadd_rd(t, -2.0f * err)), key32(__fadd_ru(t, 2.0f * err))) : sort_out(1u, ~0u);
        }
        const int i0 = a.lists > 1 ? i : 0, i1 = a.lists > 1 ? i + 1 : n;
        if (want < some && !all_zero) {
            if (some <= 32) {
                int mine = -1;  // lane x has the x-th open block
                uint64_t best = 0;
                for (float by = scale;; by = 0.0f) {
                    bool lost = false;
                    int x = 0;
#pragma unroll
                    for (int w = 0; w < WPL; ++w)
                        for (uint32_t left = __ballot_sync(0xffffffffu, maybe[w] != 0u); left; left &= left - 1u) {
                            const int l = __ffs(left) - 1;
                            for (uint32_t bits = __shfl_sync(0xffffffffu, maybe[w], l); bits; bits &= bits - 1u, ++x) {
                                const int j = 32 * (32 * w + l) + __ffs(bits) - 1;
                                const uint64_t k = exact_key<BOUNDS>(a, by, b, i0, i1, h, j, lost);
                                if (lane == x) {
                                    mine = j;
                                    best = k;
                                }
                            }
                        }
                    if (by == 0.0f || !__any_sync(0xffffffffu, lost)) break;
                }
                int before = 0;
                for (int y = 0; y < some; ++y) {
                    const uint64_t k = __shfl_sync(0xffffffffu, best, y);
                    before += k > best || (k == best && y < lane);  // open blocks are in ascending order
                }
                const bool take = lane < some && before < want;
#pragma unroll
                for (int w = 0; w < WPL; ++w) maybe[w] = 0u;
                for (uint32_t left = __ballot_sync(0xffffffffu, take); left; left &= left - 1u) {
                    const int j = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
#pragma unroll
                    for (int w = 0; w < WPL; ++w)
                        if (lane == ((j >> 5) & 31) && w == j >> 10) in[w] |= 1u << (j & 31);
                }
                want = 0;
            } else {
                // by thirds of the 64 bits, each made larger than 0
                float by = scale;
                for (int third = 0; third < 3 && want < some; ++third) {
                    bool lost = false;
#pragma unroll
                    for (int w = 0; w < WPL; ++w)
                        for (uint32_t left = __ballot_sync(0xffffffffu, maybe[w] != 0u); left; left &= left - 1u) {
                            const int l = __ffs(left) - 1;
                            for (uint32_t bits = __shfl_sync(0xffffffffu, maybe[w], l); bits; bits &= bits - 1u) {
                                const int j = 32 * (32 * w + l) + __ffs(bits) - 1;
                                const uint64_t k = exact_key<BOUNDS>(a, by, b, i0, i1, h, j, lost);
                                if (lane == 0) keys[j] = 1u + (third == 0 ? (uint32_t)(k >> 42) : third == 1 ? (uint32_t)(k >> 21) & 0x1fffffu : (uint32_t)k & 0x1fffffu);
                            }
                        }
                    if (third == 0 && by != 0.0f && __any_sync(0xffffffffu, lost)) {  // from the start, by doubles
                        by = 0.0f;
                        third = -1;
                        continue;
                    }
                    __syncwarp();
#pragma unroll
                    for (int x = 0; x < KPL; ++x) {
                        const bool open = (__shfl_sync(0xffffffffu, maybe[x >> 5], x & 31) >> lane) & 1u;
                        key[x] = open ? __ldcg(keys + 32 * x + lane) : 0u;
                    }
                    const uint32_t cut = search(want, false);
                    some = sort_out(cut, cut);
                }
            }
        }
        if (want) {  // equals, the lowest first: all of them, or the first `want`
            int base = 0;
#pragma unroll
            for (int w = 0; w < WPL; ++w) {
                int sum = __popc(maybe[w]);
                const int own = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                uint32_t mine = maybe[w];
                for (int c = base + sum - own; mine && c < want; ++c) {
                    in[w] |= mine & (0u - mine);
                    mine &= mine - 1u;
                }
                base += __shfl_sync(0xffffffffu, sum, 31);
            }
        }
    }
    int base = 0;
#pragma unroll
    for (int w = 0; w < WPL; ++w) {  // the list, in ascending order
        int sum = __popc(in[w]);
        const int own = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        int at = base + sum - own;
        for (uint32_t bits = in[w]; bits; bits &= bits - 1u, ++at)
            if (at < a.top) out[at] = 32 * (32 * w + lane) + __ffs(bits) - 1;
        base += __shfl_sync(0xffffffffu, sum, 31);
    }
}

bool select_sizes_ok(int B, int Q, int Hq, int H, int max_pages) {
    return B >= 0 && B <= kMaxB && Q >= 1 && Q <= kMaxQ && H >= 1 && H <= sv::PAGED_MAX_HEADS && Hq >= H && Hq <= 65536 &&
           Hq % H == 0 && (int64_t)Q * (Hq / H) < ((int64_t)1 << 30) && max_pages >= 1 && max_pages <= kMaxBlocks;
}

// Workspace: keys, norms, largest summaries of 16 blocks, each from a 16-byte boundary.
struct SelectSpace {
    int64_t lists, width, scores, norms, biggest;
};
SelectSpace select_space(int B, int Q, int H, int max_pages, bool shared) {
    SelectSpace s;
    s.lists = (int64_t)B * H * (shared ? 1 : Q);
    s.width = (max_pages + 3) / 4 * 4;
    s.scores = s.lists * s.width;
    s.norms = (s.lists + 3) / 4 * 4;
    s.biggest = (int64_t)B * H * ((max_pages + 15) / 16);
    return s;
}

template <int KC, bool BOUNDS, bool FULL, int NQ>
cudaError_t launch_score_nq(const SelectArgs& a, int B, cudaStream_t s) {
    const dim3 grid((unsigned)((a.max_pages + 16 * kScoreWarps - 1) / (16 * kScoreWarps)), (unsigned)(B * a.H));
    return sv::launch_serial(block_score_kernel<KC, BOUNDS, FULL, NQ>, grid, dim3(kScoreWarps * 32), 0, s, a);
}

template <int KC, bool BOUNDS>
cudaError_t launch_score(const SelectArgs& a, int B, cudaStream_t s) {
    if (a.D != 32 * KC) return launch_score_nq<KC, BOUNDS, false, 4>(a, B, s);
    const int64_t tiles = ((int64_t)a.Q * a.gp + 7) / 8;
    if (tiles == 1) return launch_score_nq<KC, BOUNDS, true, 1>(a, B, s);
    if (tiles == 2) return launch_score_nq<KC, BOUNDS, true, 2>(a, B, s);
    if (tiles == 3) return launch_score_nq<KC, BOUNDS, true, 3>(a, B, s);
    return launch_score_nq<KC, BOUNDS, true, 4>(a, B, s);
}

template <bool BOUNDS>
cudaError_t run_select(SelectArgs& a, int B, int64_t lists, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (a.top < a.max_pages && a.sink + a.recent < a.top) {  // else no list needs scores
        e = a.D <= 64 ? launch_score<2, BOUNDS>(a, B, s) : a.D <= 128 ? launch_score<4, BOUNDS>(a, B, s) : launch_score<8, BOUNDS>(a, B, s);
        if (e != cudaSuccess) return e;
    }
    // A warp per list, all in registers, where its blocks fit there, no list has many rows to sum again, and the
    // lists are more than the SMs: 1536 lists of up to 1024 blocks 46 us (with the scores) against 61 by a
    // CTA each, 8 lists of 1562 17.3 against 16.3.
    if (a.max_pages <= 2048 && lists > 152 && (a.lists > 1 ? 1 : a.Q) * a.g <= 32) {
        const dim3 grid((unsigned)((lists + 3) / 4));
        auto kern = a.max_pages <= 256 ? block_select_warp_kernel<BOUNDS, 8> : a.max_pages <= 512 ? block_select_warp_kernel<BOUNDS, 16>
                    : a.max_pages <= 1024 ? block_select_warp_kernel<BOUNDS, 32> : block_select_warp_kernel<BOUNDS, 64>;
        return sv::launch_serial(kern, grid, dim3(128), 0, s, a, (unsigned)lists);
    }
    const int kept = a.max_pages < kKept ? a.max_pages : kKept;
    const size_t smem = ((size_t)2 * ((a.max_pages + 31) / 32) + kept) * sizeof(uint32_t);
    static sv::KernelLaunchCache cache;
    int max_dyn = 0;
    e = cache.setup((const void*)block_select_kernel<BOUNDS>, &max_dyn);
    if (e != cudaSuccess) return e;
    if (smem > (size_t)max_dyn) return cudaErrorInvalidValue;
    return sv::launch_serial(block_select_kernel<BOUNDS>, dim3((unsigned)lists), dim3(kThreads), smem, s, a);
}

}  // namespace

extern "C" {

sv_status spec_block_summary(const sv_paged_cache* cache, const int32_t* base, const int32_t* new_len, sv_summary kind,
                             int B, int N, void* summary, void* stream) {
    SummaryArgs a{};
    if (!sv::paged_cache_args(cache, a.c) || (kind != SV_SUMMARY_MEAN && kind != SV_SUMMARY_BOUNDS)) return SV_ERR_INVALID_ARG;
    if (B < 0 || B > kMaxB || N < 0 || N > sv::PAGED_MAX_POS) return SV_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return SV_OK;
    if (!cache->page_table || !base || !summary || (uintptr_t)summary % 2) return SV_ERR_INVALID_ARG;
    const int ps = cache->page_size;
    int64_t blocks = ((int64_t)N + ps - 2) / ps + 1;
    if (blocks > cache->max_pages) blocks = cache->max_pages;
    if (blocks * cache->num_heads >= ((int64_t)1 << 31)) return SV_ERR_UNSUPPORTED;
    if (cache->head_dim % 8 == 0 && (uintptr_t)summary % 16) return SV_ERR_UNSUPPORTED;
    a.base = base;
    a.new_len = new_len;
    a.N = N;
    a.blocks = (unsigned)blocks;
    a.out = static_cast<uint16_t*>(summary);
    const bool e4m3 = cache->dtype == SV_CACHE_E4M3;
    const int64_t cs = e4m3 ? 8 : 16;
    const bool al = cache->head_dim % 8 == 0 && (cache->page_stride | cache->head_stride | cache->row_stride) % cs == 0 &&
                    (uintptr_t)cache->k_pages % cs == 0;
    cudaStream_t s = (cudaStream_t)stream;
    const bool bounds = kind == SV_SUMMARY_BOUNDS;
    const cudaError_t e = e4m3 ? (bounds ? summary_dim<true, true>(a, al, B, s) : summary_dim<true, false>(a, al, B, s))
                               : (bounds ? summary_dim<false, true>(a, al, B, s) : summary_dim<false, false>(a, al, B, s));
    return sv::launch_status(e);
}

size_t spec_block_select_workspace_size(int B, int Q, int num_q_heads, int num_heads, int max_pages, int shared) {
    if (!select_sizes_ok(B, Q, num_q_heads, num_heads, max_pages)) return 0;
    const SelectSpace s = select_space(B, Q, num_heads, max_pages, shared != 0);
    return (size_t)(s.scores + s.norms + s.biggest) * sizeof(float);
}

sv_status spec_block_select(const void* q, const int64_t* q_stride, int num_q_heads, const void* summary, sv_summary kind,
                            const int32_t* page_table, int num_pages, int page_size, int max_pages, int num_heads,
                            int head_dim, const int32_t* base, const int32_t* new_len, int shared, int top_k, int sink,
                            int recent, int B, int Q, int32_t* out_blocks, void* workspace, size_t ws_bytes,
                            void* stream) {
    if (!select_sizes_ok(B, Q, num_q_heads, num_heads, max_pages) || (kind != SV_SUMMARY_MEAN && kind != SV_SUMMARY_BOUNDS) ||
        num_pages < 1 || page_size < 1 || page_size > 65536 || (int64_t)max_pages * page_size > sv::PAGED_MAX_POS ||
        head_dim < 1 || head_dim > sv::PAGED_MAX_DIM || top_k < 1 || top_k > kMaxTop || sink < 0 || recent < 0 ||
        (int64_t)sink + recent > top_k)
        return SV_ERR_INVALID_ARG;
    if (B == 0) return SV_OK;
    if (!q || !q_stride || !summary || !page_table || !base || !out_blocks || !workspace) return SV_ERR_INVALID_ARG;
    if (ws_bytes < spec_block_select_workspace_size(B, Q, num_q_heads, num_heads, max_pages, shared) || (uintptr_t)workspace % 16)
        return SV_ERR_INVALID_ARG;
    if (head_dim % 8 || ((uintptr_t)q | (uintptr_t)summary) % 16 || (q_stride[0] | q_stride[1] | q_stride[2]) % 8)
        return SV_ERR_UNSUPPORTED;
    const SelectSpace sp = select_space(B, Q, num_heads, max_pages, shared != 0);
    if (sp.lists >= ((int64_t)1 << 31) || (int64_t)B * num_heads > 65535) return SV_ERR_UNSUPPORTED;
    SelectArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.q_sb = q_stride[0];
    a.q_st = q_stride[1];
    a.q_sh = q_stride[2];
    a.summary = static_cast<const uint16_t*>(summary);
    a.table = page_table;
    a.base = base;
    a.new_len = new_len;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.H = num_heads;
    a.D = head_dim;
    a.Q = Q;
    a.g = num_q_heads / num_heads;
    a.gp = 1;
    while (a.gp < a.g && a.gp < 8) a.gp *= 2;
    if (a.g > 8) a.gp = (a.g + 7) / 8 * 8;
    while (a.shift < 3 && 1 << a.shift < a.gp) ++a.shift;
    a.span = (a.gp + 7) / 8;
    a.lists = shared ? 1 : Q;
    a.width = (int)sp.width;
    a.top = top_k;
    a.sink = sink;
    a.recent = recent;
    a.key = static_cast<uint32_t*>(workspace);
    a.norm = static_cast<float*>(workspace) + sp.scores;
    a.biggest = a.norm + sp.norms;
    a.out = out_blocks;
    cudaStream_t s = (cudaStream_t)stream;
    return sv::launch_status(kind == SV_SUMMARY_BOUNDS ? run_select<true>(a, B, sp.lists, s) : run_select<false>(a, B, sp.lists, s));
}

}  // extern "C"
