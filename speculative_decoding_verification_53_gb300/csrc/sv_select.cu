// sv_select.cu -- which blocks of a long paged cache each query attends to
// (include/spec_sparse.h): summaries of the blocks' keys, and the selection of blocks by a
// cheap score against them.
//
// Summaries are one pass over the keys, bound by memory: a warp (few blocks: all warps of a
// CTA) takes one block and head, a group of lanes a key, eight elements each, and the groups
// meet by shuffles at the end.
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
// bits.  An fp32 score is off by at most e = 2^-13 |q|_1 max|m| (below), so with T the k-th largest
// fp32 score whatever is above T + 2 e is in, whatever is below T - 2 e out, and only what
// lies between (one or two blocks as a rule) is summed again in 64 bits.  Where that are many
// (equal summaries), the 64-bit scores are selected among by their upper, then their lower halves.
//
// The error of an fp32 score: n = 2 * head_dim <= 512 exact products in steps of 16, each step's sum of 17
// numbers off by at most 17 units of 2^-23 of the largest partial sum, which |q|_1 max|m| bounds:
// 32 * 17 * 2^-23 < 2^-13.
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

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// What a lane keeps of its eight elements.
template <bool BOUNDS>
struct Kept {
    float a[8], b[BOUNDS ? 8 : 1];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            a[k] = BOUNDS ? neg_inf() : 0.0f;
            if (BOUNDS) b[BOUNDS ? k : 0] = pos_inf();
        }
    }
    __device__ __forceinline__ void add(const float x[8]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            a[k] = BOUNDS ? max_nan(a[k], x[k]) : a[k] + x[k];
            if (BOUNDS) b[BOUNDS ? k : 0] = min_nan(b[BOUNDS ? k : 0], x[k]);
        }
    }
    __device__ __forceinline__ void join(const Kept& o) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            a[k] = BOUNDS ? max_nan(a[k], o.a[k]) : a[k] + o.a[k];
            if (BOUNDS) b[BOUNDS ? k : 0] = min_nan(b[BOUNDS ? k : 0], o.b[BOUNDS ? k : 0]);
        }
    }
    __device__ __forceinline__ Kept from(int mask) const {
        Kept o;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            o.a[k] = __shfl_xor_sync(0xffffffffu, a[k], mask);
            if (BOUNDS) o.b[BOUNDS ? k : 0] = __shfl_xor_sync(0xffffffffu, b[BOUNDS ? k : 0], mask);
        }
        return o;
    }
};

// grid: x over blocks * heads of one batch row, y the batch row.  WPU warps take one of them.
template <int LPR, bool E4M3, bool BOUNDS, bool AL, int WPU>
__global__ void __launch_bounds__(kThreads) block_summary_kernel(const __grid_constant__ SummaryArgs a) {
    constexpr int G = 32 / LPR, FLY = 8;  // keys of a warp at a time, and how many a lane has in flight
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
            float f[8];
            x[k].widen(scale[k], f);
            kept.add(f);
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
    if (!BOUNDS) {
#pragma unroll
        for (int k = 0; k < 8; ++k) kept.a[k] = kept.a[k] / (float)count;
    }
    if (dim % 8 == 0) sv::store_row8<uint16_t, true>(out, e0, dim, kept.a);
    else sv::store_row8<uint16_t, false>(out, e0, dim, kept.a);
    if (BOUNDS) {
        float low[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) low[k] = kept.b[BOUNDS ? k : 0];
        if (dim % 8 == 0) sv::store_row8<uint16_t, true>(out + dim, e0, dim, low);
        else sv::store_row8<uint16_t, false>(out + dim, e0, dim, low);
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
    int gp;      // rows of a query: its heads, padded to a power of two, or to a multiple of 16
    int lists;   // per batch row and head: Q, or 1 where shared
    int width;   // scores of a list in the workspace
    int chunks;  // CTAs of the scores along the blocks
    int top, sink, recent;
    float* score;   // [B][lists][H][width]
    float* norm;    // [B][lists][H]: the largest |q|_1 of the list's rows
    float* biggest; // [B][H][chunks]: the largest |m| of a CTA's blocks
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

__device__ __forceinline__ void mma16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The positive parts, or the negative ones, of two bf16.
__device__ __forceinline__ uint32_t part_of(uint32_t w, bool negative) {
    const uint32_t signs = w & 0x80008000u, mask = (signs >> 15) * 0xffffu;  // halves that are negative
    return negative ? w & mask : w & ~mask;
}

__device__ __forceinline__ uint32_t larger_magnitudes(uint32_t a, uint32_t w) { return __vmaxu2(a, w & 0x7fff7fffu); }

__device__ __forceinline__ float magnitudes(uint4 w) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) s += fabsf(sv::bf16_lo(x[k])) + fabsf(sv::bf16_hi(x[k]));
    return s;
}

constexpr int kScoreWarps = 4;

template <int KC, bool BOUNDS>
struct Score {
    static constexpr int MATS = BOUNDS ? 2 : 1;
    static constexpr int FIT = 16 / (KC * MATS);
    static constexpr int NT = FIT > 4 ? 4 : FIT < 1 ? 1 : FIT;  // tiles of eight blocks a warp keeps in registers
    static constexpr int CHUNK = kScoreWarps * NT * 8;          // blocks of a CTA
};

// grid: x over chunks of blocks, y the batch row and cache head.  KC: chunks of 32 elements.
template <int KC, bool BOUNDS>
__global__ void __launch_bounds__(kScoreWarps * 32) block_score_kernel(const __grid_constant__ SelectArgs a) {
    using S = Score<KC, BOUNDS>;
    constexpr int NT = S::NT, MATS = S::MATS;
    __shared__ uint32_t s_biggest[kScoreWarps];
    sv::pdl_trigger();
    sv::pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, t4 = lane & 3;
    const int y = blockIdx.y;
    const int b = y / a.H, h = y - b * a.H;
    int n, blocks;
    select_row(a, b, n, blocks);
    const int begin = blockIdx.x * S::CHUNK, j0 = begin + warp * NT * 8;
    // Lists that need no scores: all blocks, or only the first and last ones.
    if (n == 0 || begin >= blocks || blocks <= a.top || a.sink + a.recent == a.top) return;
    uint4 m[NT][MATS][KC];
    bool hole[NT];
    uint32_t most = 0u;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        const int j = j0 + 8 * x + g8;
        const int page = j < blocks ? __ldg(a.table + (int64_t)b * a.max_pages + j) : -1;
        hole[x] = (unsigned)page >= (unsigned)a.num_pages;
        const uint16_t* row = a.summary + ((int64_t)(hole[x] ? 0 : page) * a.H + h) * (a.D * MATS);
#pragma unroll
        for (int z = 0; z < MATS; ++z)
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                const int e = 32 * k + 8 * t4;
                m[x][z][k] = make_uint4(0u, 0u, 0u, 0u);
                if (!hole[x] && e < a.D) m[x][z][k] = sv::ld_nc_v4(row + z * a.D + e);
                most = larger_magnitudes(larger_magnitudes(most, m[x][z][k].x), m[x][z][k].y);
                most = larger_magnitudes(larger_magnitudes(most, m[x][z][k].z), m[x][z][k].w);
            }
    }
    most = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
    if (lane == 0) s_biggest[warp] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 0; w < kScoreWarps; ++w) most = max(most, s_biggest[w]);
        a.biggest[(int64_t)y * a.chunks + blockIdx.x] = __uint_as_float(most << 16);
    }
    const bool norms = begin == 0 && warp == 0;  // one warp per row and head also sums |q|
    const bool shared = a.lists != a.Q || a.Q == 1;
    const int rows = n * a.gp, tiles = (rows + 15) / 16;
    float run[NT][4], run_norm[2] = {0.0f, 0.0f};
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int z = 0; z < 4; ++z) run[x][z] = neg_inf();
    for (int t = 0; t < tiles; ++t) {
        const uint16_t* from[2];
        bool live[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int r = 16 * t + g8 + 8 * z, i = r / a.gp, head = min(r - i * a.gp, a.g - 1);
            live[z] = i < n;
            from[z] = a.q + b * a.q_sb + (live[z] ? i : 0) * a.q_st + (int64_t)(h * a.g + head) * a.q_sh;
        }
        float acc[NT][4];
#pragma unroll
        for (int x = 0; x < NT; ++x) acc[x][0] = acc[x][1] = acc[x][2] = acc[x][3] = 0.0f;
        float norm[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            const int e = 32 * k + 8 * t4;
            uint4 u = make_uint4(0u, 0u, 0u, 0u), v = u;
            if (e < a.D) {
                u = sv::ld_nc_v4(from[0] + e);
                v = sv::ld_nc_v4(from[1] + e);
            }
            if (norms) {
                norm[0] += magnitudes(u);
                norm[1] += magnitudes(v);
            }
#pragma unroll
            for (int z = 0; z < MATS; ++z) {
                auto of = [&](uint32_t w) { return BOUNDS ? part_of(w, z == 1) : w; };
                const uint32_t u0 = of(u.x), u1 = of(u.y), u2 = of(u.z), u3 = of(u.w);
                const uint32_t v0 = of(v.x), v1 = of(v.y), v2 = of(v.z), v3 = of(v.w);
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    mma16816(acc[x], u0, v0, u1, v1, m[x][z][k].x, m[x][z][k].y);
                    mma16816(acc[x], u2, v2, u3, v3, m[x][z][k].z, m[x][z][k].w);
                }
            }
        }
        // rows of a query meet: within the tile, and over tiles where a query (or a list) has several
        const bool fresh = !shared && 16 * t % a.gp == 0;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            norm[z] += __shfl_xor_sync(0xffffffffu, norm[z], 1);
            norm[z] += __shfl_xor_sync(0xffffffffu, norm[z], 2);
            if (!live[z]) norm[z] = 0.0f;
            run_norm[z] = fresh ? norm[z] : norm[z] > run_norm[z] || !(norm[z] == norm[z]) ? norm[z] : run_norm[z];
        }
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const float v = live[z >> 1] ? acc[x][z] : neg_inf();
                run[x][z] = fresh ? v : fmaxf(run[x][z], v);
            }
        const bool last = shared ? t == tiles - 1 : 16 * (t + 1) % a.gp == 0 || a.gp < 16;
        if (!last) continue;
        const int span = shared ? 16 : min(a.gp, 16);  // rows of the tile that meet
        float r0 = run_norm[0], r1 = run_norm[1];
        auto meet = [](float p, float q) { return p > q || !(p == p) ? p : q; };  // NaN stays
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            if (o >= span) continue;
            r0 = meet(r0, __shfl_xor_sync(0xffffffffu, r0, 4 * o));
            r1 = meet(r1, __shfl_xor_sync(0xffffffffu, r1, 4 * o));
        }
        if (span == 16) r0 = meet(r0, r1);
        const int i0 = shared ? 0 : 16 * t / a.gp + g8 / a.gp, i1 = shared ? 0 : (16 * t + 8) / a.gp + g8 / a.gp;
        const bool lead = g8 % min(span, 8) == 0;
        const int64_t list0 = ((int64_t)b * a.lists + i0) * a.H + h, list1 = ((int64_t)b * a.lists + i1) * a.H + h;
        const bool put0 = lead && i0 < n, put1 = lead && span < 16 && i1 < n;
        if (norms && t4 == 0) {
            if (put0) a.norm[list0] = r0;
            if (put1) a.norm[list1] = r1;
        }
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            float v[4] = {run[x][0], run[x][1], run[x][2], run[x][3]};
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                if (o >= span) continue;
#pragma unroll
                for (int z = 0; z < 4; ++z) v[z] = fmaxf(v[z], __shfl_xor_sync(0xffffffffu, v[z], 4 * o));
            }
            if (span == 16) {
                v[0] = fmaxf(v[0], v[2]);
                v[1] = fmaxf(v[1], v[3]);
            }
            const int j = j0 + 8 * x + 2 * t4;
            // blocks in holes have the lowest key of all
            const bool h0 = __shfl_sync(0xffffffffu, (int)hole[x], 8 * t4), h1 = __shfl_sync(0xffffffffu, (int)hole[x], 8 * t4 + 4);
            const float none = __uint_as_float(0xffffffffu);
            if (put0 && j < blocks) *reinterpret_cast<float2*>(a.score + list0 * a.width + j) = make_float2(h0 ? none : v[0], h1 ? none : v[1]);
            if (put1 && j < blocks) *reinterpret_cast<float2*>(a.score + list1 * a.width + j) = make_float2(h0 ? none : v[2], h1 ? none : v[3]);
        }
    }
}

// ---------------------------------------------------------------- selection

// Keys in the order of the numbers; 0: a hole.
__device__ __forceinline__ uint32_t key32(uint32_t bits) { return bits & 0x80000000u ? ~bits : bits | 0x80000000u; }
__device__ __forceinline__ float from_key32(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key); }
__device__ __forceinline__ uint64_t key64(double x) {
    if (x != x) return 1;  // below -infinity
    const uint64_t bits = (uint64_t)__double_as_longlong(x);
    return bits >> 63 ? ~bits : bits | 0x8000000000000000ull;
}

constexpr int kFew = 64;  // blocks next to the border whose 64-bit scores are compared with one another

struct SelectShared {
    uint32_t hist[256];
    uint32_t prefix, left, equal;  // of a radix selection: key so far, how many are wanted of its equals, how many there are
    uint32_t in, unsure;
    int few[kFew];
    uint64_t few_key[kFew];
    uint64_t best[kWarps];
    float bound[kWarps];
    uint32_t sums[kWarps];
};

// The key of score(i, j) in 64 bits; by all threads, the result in all of them.  A warp takes a row
// of the list at a time.
template <bool BOUNDS>
__device__ uint64_t exact_key(const SelectArgs& a, SelectShared& sh, int b, int i0, int i1, int h, int j, bool by_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int page = __ldg(a.table + (int64_t)b * a.max_pages + j);
    const uint16_t* m = a.summary + ((int64_t)page * a.H + h) * (a.D * (BOUNDS ? 2 : 1));
    const int rows = (i1 - i0) * a.g;
    uint64_t best = 0;
    bool nan = false;
    auto wide = [](uint16_t u) { return (double)__uint_as_float((uint32_t)u << 16); };
    for (int r = by_warp ? 0 : warp; r < rows; r += by_warp ? 1 : kWarps) {
        const uint16_t* q = a.q + b * a.q_sb + (i0 + r / a.g) * a.q_st + (int64_t)(h * a.g + r % a.g) * a.q_sh;
        double s = 0.0;
        for (int d = lane; d < a.D; d += 32) {
            const double x = wide(__ldg(q + d));
            const double y = wide(__ldg(m + (BOUNDS && !(x >= 0.0) ? a.D + d : d)));
            s = fma(x, y, s);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (s != s) nan = true;
        const uint64_t k = key64(s == 0.0 ? 0.0 : s);  // -0 is 0
        if (k > best) best = k;
    }
    if (nan) best = ~0ull;  // for now above all, so that it survives the join
    if (!by_warp) {
        __syncthreads();
        if (lane == 0) sh.best[warp] = best;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (sh.best[w] > best) best = sh.best[w];
    }
    return best == ~0ull ? 1 : best;
}

// The `want`-th largest key(j) of the blocks j in [from, to) that take part; sh.prefix is it, sh.left
// how many of those equal to it are wanted, sh.equal how many there are.  By all threads.
template <typename Key, typename Part>
__device__ void radix_select(SelectShared& sh, int from, int to, uint32_t want, Key key, Part part) {
    uint32_t prefix = 0u, mask = 0u;
    for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        for (int x = threadIdx.x; x < 256; x += kThreads) sh.hist[x] = 0u;
        __syncthreads();
        for (int j = from + threadIdx.x; j < to; j += kThreads) {
            if (!part(j)) continue;
            const uint32_t k = key(j);
            if ((k & mask) == prefix) atomicAdd(&sh.hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x < 32) {  // the bin in which the want-th lies, from the top; a lane has eight bins
            const int lane = threadIdx.x, top = 255 - 8 * lane;
            uint32_t c[8], own = 0u;
#pragma unroll
            for (int x = 0; x < 8; ++x) own += c[x] = sh.hist[top - x];
            uint32_t sum = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            uint32_t before = sum - own;
            if (before < want && want <= sum) {
                int x = 0;
#pragma unroll
                for (int y = 0; y < 7; ++y)
                    if (x == y && before + c[y] < want) {
                        before += c[y];
                        x = y + 1;
                    }
                sh.prefix = prefix | (uint32_t)(top - x) << shift;
                sh.left = want - before;
                sh.equal = sh.hist[top - x];
            }
        }
        __syncthreads();
        prefix = sh.prefix;
        want = sh.left;
        mask |= 255u << shift;
    }
}

// One CTA per list.
template <bool BOUNDS>
__global__ void __launch_bounds__(kThreads) block_select_kernel(const __grid_constant__ SelectArgs a) {
    extern __shared__ uint32_t s_bits[];  // [words] blocks that are in, [words] blocks not yet decided
    __shared__ SelectShared sh;
    sv::pdl_trigger();
    sv::pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t list = blockIdx.x;
    const int h = (int)(list % a.H), i = (int)(list / a.H % a.lists), b = (int)(list / a.H / a.lists);
    int n, blocks;
    select_row(a, b, n, blocks);
    int32_t* out = a.out + list * a.top;
    if (n == 0 || (a.lists > 1 && i >= n) || blocks <= a.top) {
        const int have = n == 0 || (a.lists > 1 && i >= n) ? 0 : blocks;
        for (int x = tid; x < a.top; x += kThreads) out[x] = x < have ? x : -1;
        return;
    }
    const int words = (blocks + 31) / 32;
    uint32_t* s_in = s_bits;
    uint32_t* s_unsure = s_bits + words;
    const int from = a.sink, to = blocks - a.recent;  // candidates
    uint32_t want = (uint32_t)(a.top - a.sink - a.recent);
    for (int w = tid; w < words; w += kThreads) {  // first and last blocks
        uint32_t bits = 0u;
        for (int x = 0; x < 32; ++x) {
            const int j = 32 * w + x;
            if (j < blocks && (j < from || j >= to)) bits |= 1u << x;
        }
        s_in[w] = bits;
        s_unsure[w] = 0u;
    }
    if (tid == 0) sh.in = sh.unsure = 0u;
    if (want) {
        float* score = a.score + list * a.width;
        const uint32_t* bits = reinterpret_cast<const uint32_t*>(score);
        // the error's bound
        float most = 0.0f;
        const int per = BOUNDS ? (a.D <= 64 ? Score<2, true>::CHUNK : a.D <= 128 ? Score<4, true>::CHUNK : Score<8, true>::CHUNK)
                               : (a.D <= 64 ? Score<2, false>::CHUNK : a.D <= 128 ? Score<4, false>::CHUNK : Score<8, false>::CHUNK);
        const int chunks = (blocks + per - 1) / per;
        for (int x = tid; x < chunks; x += kThreads) {
            const float v = a.biggest[((int64_t)b * a.H + h) * a.chunks + x];
            most = v > most || v != v ? v : most;
        }
        uint32_t top_bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));  // NaN (of a positive sign) is above all
        if (lane == 0) sh.sums[warp] = top_bits;
        radix_select(sh, from, to, want, [&](int j) { return key32(__ldcg(bits + j)); }, [](int) { return true; });
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top_bits = max(top_bits, sh.sums[w]);
        const float reach = a.norm[list] * __uint_as_float(top_bits);  // |q|_1 max|m|
        const float err = reach * 0x1p-13f;
        const uint32_t edge = sh.prefix;
        const bool sure = reach < 0x1p120f;  // else (NaN among them) every score is summed again
        const float t = from_key32(edge);
        const float low = __fadd_rd(t, -2.0f * err), high = __fadd_ru(t, 2.0f * err);
        uint32_t in = 0u, unsure = 0u;
        for (int j = from + tid; j < to; j += kThreads) {
            const uint32_t u = __ldcg(bits + j), k = key32(u);
            const float v = __uint_as_float(u);
            bool yes, maybe;
            if (edge == 0u) {  // fewer blocks than wanted are in no hole
                yes = k > 0u;
                maybe = k == 0u;
            } else {
                yes = k > 0u && sure && v > high;
                maybe = k > 0u && !yes && (!sure || v >= low);
            }
            if (yes) atomicOr(&s_in[j >> 5], 1u << (j & 31));
            if (maybe) atomicOr(&s_unsure[j >> 5], 1u << (j & 31));
            in += yes;
            unsure += maybe;
        }
        in = __reduce_add_sync(0xffffffffu, in);
        unsure = __reduce_add_sync(0xffffffffu, unsure);
        __syncthreads();
        if (lane == 0) {
            atomicAdd(&sh.in, in);
            atomicAdd(&sh.unsure, unsure);
        }
        __syncthreads();
        want -= sh.in;
        uint32_t some = sh.unsure;
        const int i0 = a.lists > 1 ? i : 0, i1 = a.lists > 1 ? i + 1 : n;
        auto open = [&](int j) { return (s_unsure[j >> 5] >> (j & 31)) & 1u; };
        if (want < some && edge != 0u && some <= kFew) {
            __syncthreads();
            if (tid == 0) sh.unsure = 0u;
            __syncthreads();
            for (int j = from + tid; j < to; j += kThreads)
                if (open(j)) sh.few[atomicAdd(&sh.unsure, 1u)] = j;  // in any order: ranked by key and index
            __syncthreads();
            for (uint32_t x = 0; x < some; ++x) {
                const uint64_t k = exact_key<BOUNDS>(a, sh, b, i0, i1, h, sh.few[x], false);
                if (tid == 0) sh.few_key[x] = k;
            }
            __syncthreads();
            if (tid < (int)some) {
                const uint64_t k = sh.few_key[tid];
                const int j = sh.few[tid];
                uint32_t before = 0u;
                for (uint32_t x = 0; x < some; ++x) before += sh.few_key[x] > k || (sh.few_key[x] == k && sh.few[x] < j);
                if (before < want) atomicOr(&s_in[j >> 5], 1u << (j & 31));
            }
            want = 0u;
        } else if (want < some && edge != 0u) {
            uint32_t* keys = reinterpret_cast<uint32_t*>(score);
            for (int half = 0; half < 2 && want < some; ++half) {
                for (int j = from + warp; j < to; j += kWarps) {
                    if (!open(j)) continue;
                    const uint64_t k = exact_key<BOUNDS>(a, sh, b, i0, i1, h, j, true);
                    if (lane == 0) __stcg(keys + j, half ? (uint32_t)k : (uint32_t)(k >> 32));
                }
                __syncthreads();
                radix_select(sh, from, to, want, [&](int j) { return __ldcg(keys + j); }, open);
                const uint32_t cut = sh.prefix;
                want = sh.left;
                some = sh.equal;
                for (int w = tid; w < words; w += kThreads) {  // a word is one thread's
                    uint32_t rest = s_unsure[w];
                    for (uint32_t todo = rest; todo; todo &= todo - 1u) {
                        const int x = __ffs(todo) - 1;
                        const uint32_t k = __ldcg(keys + 32 * w + x);
                        if (k > cut) s_in[w] |= 1u << x;
                        if (k != cut) rest &= ~(1u << x);
                    }
                    s_unsure[w] = rest;
                }
                __syncthreads();
            }
        }
        __syncthreads();
        if (want) {  // equals, the lowest first: all of them, or the first `want`
            if (warp == 0) {
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
        }
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
    if (lane == 31) sh.hist[warp] = sum;
    __syncthreads();
    uint32_t at = sum - own;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warp) at += sh.hist[w];
    for (int w = w0; w < w1; ++w)
        for (uint32_t bits = s_in[w]; bits; bits &= bits - 1u, ++at)
            if (at < (uint32_t)a.top) out[at] = 32 * w + __ffs(bits) - 1;
}

bool select_sizes_ok(int B, int Q, int Hq, int H, int max_pages) {
    return B >= 0 && B <= kMaxB && Q >= 1 && Q <= kMaxQ && H >= 1 && H <= sv::PAGED_MAX_HEADS && Hq >= H && Hq <= 65536 &&
           Hq % H == 0 && (int64_t)Q * (Hq / H) < ((int64_t)1 << 30) && max_pages >= 1 && max_pages <= kMaxBlocks;
}

// Workspace: scores, norms, largest summaries (one per eight blocks at most), each from a 16-byte boundary.
struct SelectSpace {
    int64_t lists, width, scores, norms, biggest;
};
SelectSpace select_space(int B, int Q, int H, int max_pages, bool shared) {
    SelectSpace s;
    s.lists = (int64_t)B * H * (shared ? 1 : Q);
    s.width = (max_pages + 3) / 4 * 4;
    s.scores = s.lists * s.width;
    s.norms = (s.lists + 3) / 4 * 4;
    s.biggest = (int64_t)B * H * ((max_pages + 31) / 32);
    return s;
}

template <int KC, bool BOUNDS>
cudaError_t launch_score(SelectArgs& a, int B, cudaStream_t s) {
    a.chunks = (a.max_pages + Score<KC, BOUNDS>::CHUNK - 1) / Score<KC, BOUNDS>::CHUNK;
    const int64_t pairs = (int64_t)B * a.H;
    if (pairs > 65535) return cudaErrorInvalidValue;
    return sv::launch_serial(block_score_kernel<KC, BOUNDS>, dim3((unsigned)a.chunks, (unsigned)pairs), dim3(kScoreWarps * 32), 0, s, a);
}

template <bool BOUNDS>
cudaError_t run_select(SelectArgs& a, int B, int64_t lists, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (a.top < a.max_pages && a.sink + a.recent < a.top) {  // else no list needs scores
        e = a.D <= 64 ? launch_score<2, BOUNDS>(a, B, s) : a.D <= 128 ? launch_score<4, BOUNDS>(a, B, s) : launch_score<8, BOUNDS>(a, B, s);
        if (e != cudaSuccess) return e;
    }
    const size_t smem = (size_t)2 * ((a.max_pages + 31) / 32) * sizeof(uint32_t);
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
    while (a.gp < a.g && a.gp < 16) a.gp *= 2;
    if (a.g > 16) a.gp = (a.g + 15) / 16 * 16;
    a.lists = shared ? 1 : Q;
    a.width = (int)sp.width;
    a.top = top_k;
    a.sink = sink;
    a.recent = recent;
    a.score = static_cast<float*>(workspace);
    a.norm = a.score + sp.scores;
    a.biggest = a.norm + sp.norms;
    a.out = out_blocks;
    cudaStream_t s = (cudaStream_t)stream;
    return sv::launch_status(kind == SV_SUMMARY_BOUNDS ? run_select<true>(a, B, sp.lists, s) : run_select<false>(a, B, sp.lists, s));
}

}  // extern "C"
