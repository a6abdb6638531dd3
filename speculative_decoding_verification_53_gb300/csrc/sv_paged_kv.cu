// sv_paged_kv.cu -- new keys and values written into a paged cache, pages read back, and
// the accepted tree nodes' rows moved through the page table (include/spec_paged_kv.h).
//
// Writing and reading are one pass over the data.  A row of one token and head is held by
// a group of lanes, eight elements each (a power of two of lanes, so that the row's
// largest magnitude is log2 shuffles away); a group does the key and the value of its
// token and head, so both loads are in flight together and the page is looked up once.
//   e4m3: scale s = max(a / 448, 2^-126), a the largest finite magnitude; code = e4m3(x / s).
//   The quotient is x i + x j, i = 1 / s rounded and j = (1 - s i) i what it leaves: i + j is 1 / s
//   to 2^-47, x j is off by 2^-47 of the sum, and the fma that adds them rounds once, so the
//   result is x / s rounded from within 2^-46 of itself; two elements an instruction.  x i
//   alone put 5 in 10000 elements of bf16 rows, where x / s often is next to the middle of two codes,
//   on its wrong side.
//
// One GB300: writing 16 x up to 2048 tokens of 8 heads x 128 as e4m3 takes 34 us (3.7 TB/s, bound by
// issue: the largest magnitude, compared as pairs of bf16 bits, the quotient, which cost 4 us over
// x i, and one rounding per pair), as bf16
// 31 us (5.4 TB/s); reading 8 x up to 8192 positions back from e4m3 45 us (5.6 TB/s).
//
// The paged compaction is the kernel of sv_tree_kv.cu with one more indirection: a warp
// turns the path into byte offsets through the table, then every thread moves its piece
// of each row, loading up to eight sources before storing them.
#include <cstdint>

#include "spec_paged_kv.h"
#include "sv_internal.h"
#include "sv_paged.cuh"

namespace {

using sv::PagedCache;
using sv::pdl_trigger;
using sv::pdl_wait;

constexpr int kThreads = 256;
constexpr int kMaxB = 65535;

struct RowsArgs {
    PagedCache c;
    const int32_t* base;
    const int32_t* new_len;
    int N;
    const unsigned char* key;    // append: source; read: destination (written)
    const unsigned char* value;
    int64_t sb, st, sh;          // element strides of key and value
};

// Elements e0 .. e0+7 of a row of `dim` elements as fp32 (zero beyond dim).
template <typename T, bool AL>
__device__ __forceinline__ void load_row8(const T* row, int e0, int dim, float x[8]) {
    if (AL) {
        if (e0 < dim) {
            if (sizeof(T) == 2) {
                const uint4 v = sv::ld_nc_v4(row + e0);
                x[0] = sv::bf16_lo(v.x); x[1] = sv::bf16_hi(v.x); x[2] = sv::bf16_lo(v.y); x[3] = sv::bf16_hi(v.y);
                x[4] = sv::bf16_lo(v.z); x[5] = sv::bf16_hi(v.z); x[6] = sv::bf16_lo(v.w); x[7] = sv::bf16_hi(v.w);
            } else {
                const uint4 a = sv::ld_nc_v4(row + e0), b = sv::ld_nc_v4(row + e0 + 4);
                x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y);
                x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
                x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y);
                x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.0f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = 0.0f;
            if (e0 + j < dim)
                x[j] = sizeof(T) == 2 ? __uint_as_float((uint32_t)__ldg((const unsigned short*)row + e0 + j) << 16)
                                      : __ldg((const float*)row + e0 + j);
        }
    }
}

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < sv::pos_inf() ? a : 0.0f;  // false for NaN and infinity
}

// Eight elements of a row as they lie in memory (AL), or widened one by one.
template <typename T, bool AL>
struct Eight {
    uint4 w[AL ? (sizeof(T) == 2 ? 1 : 2) : 1];
    float f[AL ? 1 : 8];
    __device__ __forceinline__ void load(const T* row, int e0, int dim) {
        if (!AL) {
            load_row8<T, false>(row, e0, dim, f);
        } else if (e0 < dim) {
            w[0] = sv::ld_nc_v4(row + e0);
            if (sizeof(T) == 4) w[sizeof(T) == 4 ? 1 : 0] = sv::ld_nc_v4(row + e0 + 4);
        } else {
            w[0] = w[sizeof(T) == 4 ? 1 : 0] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    // Bits of the largest magnitude; at 0x7f800000 or beyond where one is not finite.
    __device__ __forceinline__ uint32_t largest() const {
        if (AL && sizeof(T) == 2) {  // two bf16 at a time: as integers magnitudes are in order
            const uint32_t a = __vmaxu2(w[0].x & 0x7fff7fffu, w[0].y & 0x7fff7fffu);
            const uint32_t b = __vmaxu2(w[0].z & 0x7fff7fffu, w[0].w & 0x7fff7fffu);
            const uint32_t c = __vmaxu2(a, b);
            return max(c << 16, c & 0xffff0000u);
        }
        float x[8];
        widen(x);
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ void widen(float x[8]) const {
        if (!AL) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = f[AL ? 0 : j];
        } else if (sizeof(T) == 2) {
            x[0] = sv::bf16_lo(w[0].x); x[1] = sv::bf16_hi(w[0].x); x[2] = sv::bf16_lo(w[0].y); x[3] = sv::bf16_hi(w[0].y);
            x[4] = sv::bf16_lo(w[0].z); x[5] = sv::bf16_hi(w[0].z); x[6] = sv::bf16_lo(w[0].w); x[7] = sv::bf16_hi(w[0].w);
        } else {
            const uint4 b = w[sizeof(T) == 4 ? 1 : 0];
            x[0] = __uint_as_float(w[0].x); x[1] = __uint_as_float(w[0].y);
            x[2] = __uint_as_float(w[0].z); x[3] = __uint_as_float(w[0].w);
            x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y);
            x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
        }
    }
};

// Writes eight elements of a cache row (and the row's scale).  LPR lanes hold the row.
template <typename T, int LPR, bool E4M3, bool AL>
__device__ __forceinline__ void store_cache_row(unsigned char* row, float* scale, int e0, int dim, bool live,
                                                const Eight<T, AL>& v) {
    if (E4M3) {
        uint32_t top = v.largest();
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        float a = __uint_as_float(top);
        // Rare rows: not all finite, or (but for zeros) so small or large that j may be subnormal
        // or a product may be: below 2^-80 or from 2^80 on.
        const bool rare = __any_sync(0xffffffffu, top != 0u && (top < 0x17800000u || top >= 0x67800000u));
        if (rare) {  // the largest finite magnitude
            float x[8];
            v.widen(x);
            a = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) a = fmaxf(a, finite_abs(x[j]));
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        }
        const float s = fmaxf(a / sv::E4M3_MAX, 1.17549435e-38f);
        if (!live) return;
        // Rare rows are divided as x 2^90 and s 2^90 (or 2^-90), exact where it matters.
        const float f = !rare || (s > 1.0e-20f && s < 1.0e20f) ? 1.0f : s < 1.0f ? 1.2379400392853803e27f : 8.0779356694631609e-28f;
        const float i = 1.0f / (s * f), j = fmaf(-s * f, i, 1.0f) * i;
        const float2 i2 = make_float2(i, i), j2 = make_float2(j, j);
        float x[8];
        v.widen(x);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float2 e = make_float2(x[2 * k], x[2 * k + 1]);
            if (rare) e = make_float2(e.x * f, e.y * f);
            float2 q = sv::ffma2(e, i2, sv::fmul2(e, j2));
            if (rare) {  // infinity's x j may be of the other sign
                if (sv::not_finite(e.x)) q.x = e.x;
                if (sv::not_finite(e.y)) q.y = e.y;
            }
            w[k] = sv::e4m3x2(q.x, q.y);
        }
        if (e0 == 0) *scale = s;
        if (AL) {
            if (e0 < dim) *reinterpret_cast<uint2*>(row + e0) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e0 + j < dim) row[e0 + j] = (unsigned char)(w[j / 2] >> (8 * (j & 1)));
        }
    } else {
        if (!live) return;
        float x[8];
        v.widen(x);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = sv::bf16x2(x[2 * j], x[2 * j + 1]);
        if (AL) {
            if (e0 < dim) *reinterpret_cast<uint4*>(row + 2 * e0) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e0 + j < dim) reinterpret_cast<unsigned short*>(row)[e0 + j] = (unsigned short)(w[j / 2] >> (16 * (j & 1)));
        }
    }
}

// Rows (of one token and head) that a group of lanes does where there are blocks to spare: all
// their loads are in flight before the first is looked at, as they lie in memory (widened they
// cost the registers of half the resident blocks).  Reading 8 x up to 8192 positions of 8 heads
// x 128 e4m3 with 1, 2 and 4 rows: 57.6, 50.2, 46.5 us; writing 16 x up to 2048 tokens 40.8,
// 37.1, 39.6 us (magnitudes compared as fp32).  A chain's 48 rows want one: 5.2 against 6.3 us.
template <bool READ, typename T, bool AL>
constexpr int kRows = !AL ? 1 : READ && sizeof(T) == 2 ? 4 : 2;

// grid: x over the N * heads rows of one batch row, y the batch row.
template <typename T, int LPR, bool E4M3, bool AL, int ROWS>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ RowsArgs a) {
    pdl_trigger();
    pdl_wait();  // nothing the previous kernel on the stream writes is read before this
    constexpr int RPC = kThreads / LPR;
    const int b = blockIdx.y, lane = threadIdx.x % LPR, e0 = 8 * lane;
    const unsigned heads = a.c.heads, block0 = blockIdx.x * (unsigned)(RPC * ROWS);
    int first, n;
    if (!sv::paged_row(a.c, a.base, a.new_len, b, a.N, first, n)) return;
    if (block0 / heads >= (unsigned)n) return;  // the whole block is behind the row's tokens
    Eight<T, AL> x[ROWS], y[ROWS];
    int page[ROWS], row[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const unsigned r = block0 + threadIdx.x / LPR + k * RPC, i = r / heads, h = r - i * heads;
        page[k] = -1;
        row[k] = 0;
        const bool in = i < (unsigned)n;
        const int64_t off = in ? b * a.sb + i * a.st + h * a.sh : 0;
        x[k].load(reinterpret_cast<const T*>(a.key) + off, in ? e0 : a.c.dim, a.c.dim);
        y[k].load(reinterpret_cast<const T*>(a.value) + off, in ? e0 : a.c.dim, a.c.dim);
        if (in) page[k] = sv::paged_place(a.c, b, first + i, row[k]);
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const unsigned h = (block0 + threadIdx.x / LPR + k * RPC) % heads;
        const int64_t at = page[k] * a.c.page_stride + h * a.c.head_stride + row[k] * a.c.row_stride;
        const int64_t sc = ((int64_t)page[k] * heads + h) * a.c.page_size + row[k];
        store_cache_row<T, LPR, E4M3, AL>(a.c.k + at, a.c.k_scale + sc, e0, a.c.dim, page[k] >= 0, x[k]);
        store_cache_row<T, LPR, E4M3, AL>(a.c.v + at, a.c.v_scale + sc, e0, a.c.dim, page[k] >= 0, y[k]);
    }
}

// Eight elements of a cache row as they lie there, and widened.
template <bool E4M3, bool AL>
struct EightOfCache {
    Eight<uint16_t, AL> b;
    uint2 w;
    __device__ __forceinline__ void load(const unsigned char* row, int e0, int dim) {
        if (!E4M3) {
            b.load(reinterpret_cast<const uint16_t*>(row), e0, dim);
            return;
        }
        w = make_uint2(0u, 0u);
        if (AL) {
            if (e0 < dim) w = __ldg(reinterpret_cast<const uint2*>(row + e0));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e0 + j < dim) (j < 4 ? w.x : w.y) |= (uint32_t)__ldg(row + e0 + j) << (8 * (j & 3));
        }
    }
    __device__ __forceinline__ void widen(float scale, float x[8]) const {
        if (!E4M3) {
            b.widen(x);
            return;
        }
        const float2 p = sv::e4m3x2_to_f32(w.x & 0xffffu), q = sv::e4m3x2_to_f32(w.x >> 16);
        const float2 r = sv::e4m3x2_to_f32(w.y & 0xffffu), t = sv::e4m3x2_to_f32(w.y >> 16);
        x[0] = p.x * scale; x[1] = p.y * scale; x[2] = q.x * scale; x[3] = q.y * scale;
        x[4] = r.x * scale; x[5] = r.y * scale; x[6] = t.x * scale; x[7] = t.y * scale;
    }
};

template <typename T, bool AL>
__device__ __forceinline__ void store_row8(T* row, int e0, int dim, const float x[8]) {
    if (AL) {
        if (e0 >= dim) return;
        if (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(row + e0) = make_uint4(sv::bf16x2(x[0], x[1]), sv::bf16x2(x[2], x[3]),
                                                             sv::bf16x2(x[4], x[5]), sv::bf16x2(x[6], x[7]));
        } else {
            *reinterpret_cast<float4*>(row + e0) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(row + e0 + 4) = make_float4(x[4], x[5], x[6], x[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (e0 + j < dim) {
                if (sizeof(T) == 2) reinterpret_cast<unsigned short*>(row)[e0 + j] = (unsigned short)sv::bf16x2(x[j], 0.0f);
                else reinterpret_cast<float*>(row)[e0 + j] = x[j];
            }
    }
}

template <typename T, int LPR, bool E4M3, bool AL, int ROWS>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ RowsArgs a) {
    pdl_trigger();
    pdl_wait();
    constexpr int RPC = kThreads / LPR;
    const int b = blockIdx.y, lane = threadIdx.x % LPR, e0 = 8 * lane;
    const unsigned heads = a.c.heads, block0 = blockIdx.x * (unsigned)(RPC * ROWS);
    int first, n;
    if (!sv::paged_row(a.c, a.base, a.new_len, b, a.N, first, n)) return;
    if (block0 / heads >= (unsigned)n) return;
    EightOfCache<E4M3, AL> x[ROWS], y[ROWS];
    float ks[ROWS], vs[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const unsigned r = block0 + threadIdx.x / LPR + k * RPC, i = r / heads, h = r - i * heads;
        int row = 0, page = -1;
        if (i < (unsigned)n) page = sv::paged_place(a.c, b, first + i, row);
        const bool in = page >= 0;  // a hole reads as zeros
        const int64_t at = in ? page * a.c.page_stride + h * a.c.head_stride + row * a.c.row_stride : 0;
        const int64_t sc = in ? ((int64_t)page * heads + h) * a.c.page_size + row : 0;
        ks[k] = E4M3 && in ? __ldg(a.c.k_scale + sc) : 0.0f;
        vs[k] = E4M3 && in ? __ldg(a.c.v_scale + sc) : 0.0f;
        x[k].load(a.c.k + at, in ? e0 : a.c.dim, a.c.dim);
        y[k].load(a.c.v + at, in ? e0 : a.c.dim, a.c.dim);
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const unsigned r = block0 + threadIdx.x / LPR + k * RPC, i = r / heads, h = r - i * heads;
        if (i >= (unsigned)n) continue;
        const int64_t off = b * a.sb + i * a.st + h * a.sh;
        float f[8];
        x[k].widen(ks[k], f);
        store_row8<T, AL>(reinterpret_cast<T*>(const_cast<unsigned char*>(a.key)) + off, e0, a.c.dim, f);
        y[k].widen(vs[k], f);
        store_row8<T, AL>(reinterpret_cast<T*>(const_cast<unsigned char*>(a.value)) + off, e0, a.c.dim, f);
    }
}

template <bool READ, typename T, int LPR, bool E4M3, bool AL, int ROWS>
cudaError_t launch_rows_by(const RowsArgs& a, int B, cudaStream_t stream) {
    constexpr int per = kThreads / LPR * ROWS;  // rows of a block
    const dim3 grid((unsigned)(((int64_t)a.N * a.c.heads + per - 1) / per), (unsigned)B);
    if (READ) return sv::launch_serial(kv_read_kernel<T, LPR, E4M3, AL, ROWS>, grid, dim3(kThreads), 0, stream, a);
    return sv::launch_serial(kv_append_kernel<T, LPR, E4M3, AL, ROWS>, grid, dim3(kThreads), 0, stream, a);
}

template <bool READ, typename T, int LPR, bool E4M3, bool AL>
cudaError_t launch_rows(const RowsArgs& a, int B, cudaStream_t stream) {
    constexpr int many = kRows<READ, T, AL>;
    const int64_t blocks = (int64_t)a.N * a.c.heads * B / (kThreads / LPR * many);
    if (many == 1 || blocks < 512) return launch_rows_by<READ, T, LPR, E4M3, AL, 1>(a, B, stream);
    return launch_rows_by<READ, T, LPR, E4M3, AL, many>(a, B, stream);
}

template <bool READ, typename T, bool E4M3, bool AL>
cudaError_t launch_lpr(const RowsArgs& a, int B, cudaStream_t stream) {
    const int lanes = (a.c.dim + 7) / 8;
    if (lanes <= 8) return launch_rows<READ, T, 8, E4M3, AL>(a, B, stream);
    if (lanes <= 16) return launch_rows<READ, T, 16, E4M3, AL>(a, B, stream);
    return launch_rows<READ, T, 32, E4M3, AL>(a, B, stream);
}

template <bool READ>
sv_status run_rows(const RowsArgs& a, bool e4m3, int dt, bool al, int B, cudaStream_t s) {
    cudaError_t e;
    if (dt == SV_BF16) {
        if (e4m3) e = al ? launch_lpr<READ, uint16_t, true, true>(a, B, s) : launch_lpr<READ, uint16_t, true, false>(a, B, s);
        else e = al ? launch_lpr<READ, uint16_t, false, true>(a, B, s) : launch_lpr<READ, uint16_t, false, false>(a, B, s);
    } else {
        if (e4m3) e = al ? launch_lpr<READ, float, true, true>(a, B, s) : launch_lpr<READ, float, true, false>(a, B, s);
        else e = al ? launch_lpr<READ, float, false, true>(a, B, s) : launch_lpr<READ, float, false, false>(a, B, s);
    }
    return sv::launch_status(e);
}

bool rows_sizes_ok(const PagedCache& c, int B, int N) {
    return B >= 0 && B <= kMaxB && N >= 0 && (int64_t)N * c.heads < ((int64_t)1 << 31);
}

// Whether 16-byte (8-byte for codes) accesses of eight elements are aligned everywhere.
bool rows_aligned(const RowsArgs& a, const sv_paged_cache* c, int es) {
    const int64_t cs = c->dtype == SV_CACHE_BF16 ? 16 : 8;
    return c->head_dim % 8 == 0 && (a.sb * es | a.st * es | a.sh * es) % 16 == 0 &&
           ((uintptr_t)a.key | (uintptr_t)a.value) % 16 == 0 &&
           (c->page_stride | c->head_stride | c->row_stride) % cs == 0 &&
           ((uintptr_t)c->k_pages | (uintptr_t)c->v_pages) % cs == 0;
}

// ---------------------------------------------------------------- compaction

constexpr int kKvMaxBuffers = 256;
constexpr int kKvMaxDepth = 64;
constexpr int kKvBatch = 8;  // sources loaded before their stores

struct PagedMoveArgs {
    unsigned char* buf[kKvMaxBuffers];
    int64_t page_stride, plane_stride, row_stride;
    int num_planes, pieces, D;
    int num_pages, page_size, max_pages;
    unsigned total;  // num_buffers * num_planes * pieces
    const int32_t* table;
    const int32_t* path;
    const int32_t* count;
    const int32_t* base;
};

template <int PW> struct Piece;
template <> struct Piece<16> { using T = uint4; };
template <> struct Piece<4> { using T = uint32_t; };
template <> struct Piece<1> { using T = uint8_t; };

// grid: x covers num_buffers * num_planes * pieces, y is the batch row.
template <int PW>
__global__ void __launch_bounds__(kThreads) kv_compact_paged_kernel(const __grid_constant__ PagedMoveArgs a) {
    pdl_trigger();
    pdl_wait();
    using T = typename Piece<PW>::T;
    __shared__ int64_t s_dst[kKvMaxDepth], s_src[kKvMaxDepth];
    __shared__ int s_moves;
    const int b = blockIdx.y;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int cnt = __ldg(a.count + b);
        const int L = cnt - 1;
        const int base = a.base ? __ldg(a.base + b) : 0;
        const int64_t rows = (int64_t)a.max_pages * a.page_size;
        const int32_t* table = a.table + (int64_t)b * a.max_pages;
        bool ok = cnt >= 1 && L <= a.D && base >= 0;
        int moves = 0;
        for (int d0 = 0; d0 < a.D; d0 += 32) {
            const int d = d0 + lane;
            int s = d;
            bool lane_ok = true;
            if (ok && d < L) {
                s = __ldg(a.path + (int64_t)b * a.D + d);
                lane_ok = s >= d && (int64_t)base + s < rows;
            }
            bool move = ok && lane_ok && d < L && s != d;  // a row already in place is not copied
            int64_t src = 0, dst = 0;
            if (move) {
                const int ps = base + s, pd = base + d;  // below rows < 2^31
                const int is = ps / a.page_size, id = pd / a.page_size;
                const int gs = __ldg(table + is), gd = __ldg(table + id);
                lane_ok = (unsigned)gs < (unsigned)a.num_pages && (unsigned)gd < (unsigned)a.num_pages;
                src = gs * a.page_stride + (ps - is * a.page_size) * a.row_stride;
                dst = gd * a.page_stride + (pd - id * a.page_size) * a.row_stride;
            }
            ok = ok && __all_sync(0xffffffffu, lane_ok);
            move = move && ok;
            const unsigned m = __ballot_sync(0xffffffffu, move);
            if (move) {
                const int slot = moves + __popc(m & ((1u << lane) - 1u));
                s_dst[slot] = dst;
                s_src[slot] = src;
            }
            moves += __popc(m);
        }
        if (lane == 0) s_moves = ok ? moves : 0;
    }
    __syncthreads();
    const int moves = s_moves;
    const unsigned f = blockIdx.x * kThreads + threadIdx.x;
    if (moves == 0 || f >= a.total) return;
    const unsigned piece = f % a.pieces, rest = f / a.pieces;
    const unsigned h = rest % a.num_planes, k = rest / a.num_planes;
    unsigned char* p0 = a.buf[k] + (int64_t)h * a.plane_stride + (int64_t)piece * PW;
    for (int m0 = 0; m0 < moves; m0 += kKvBatch) {
        T v[kKvBatch];
#pragma unroll
        for (int j = 0; j < kKvBatch; ++j)
            if (m0 + j < moves) v[j] = *reinterpret_cast<const T*>(p0 + s_src[m0 + j]);
#pragma unroll
        for (int j = 0; j < kKvBatch; ++j)
            if (m0 + j < moves) *reinterpret_cast<T*>(p0 + s_dst[m0 + j]) = v[j];
    }
}

}  // namespace

extern "C" {

sv_status spec_kv_append(const void* key, const void* value, sv_dtype src, const int64_t* src_stride,
                         const sv_paged_cache* cache, const int32_t* base, const int32_t* new_len, int B, int N,
                         void* stream) {
    RowsArgs a{};
    if (src != SV_F32 && src != SV_BF16) return SV_ERR_INVALID_ARG;
    if (!sv::paged_cache_args(cache, a.c) || !rows_sizes_ok(a.c, B, N)) return SV_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return SV_OK;
    const int es = src == SV_BF16 ? 2 : 4;
    if (!cache->page_table || !key || !value || !base || !src_stride || ((uintptr_t)key | (uintptr_t)value) % es) return SV_ERR_INVALID_ARG;
    a.base = base;
    a.new_len = new_len;
    a.N = N;
    a.key = static_cast<const unsigned char*>(key);
    a.value = static_cast<const unsigned char*>(value);
    a.sb = src_stride[0];
    a.st = src_stride[1];
    a.sh = src_stride[2];
    return run_rows<false>(a, cache->dtype == SV_CACHE_E4M3, src, rows_aligned(a, cache, es), B, (cudaStream_t)stream);
}

sv_status spec_kv_read(const sv_paged_cache* cache, const int32_t* base, const int32_t* new_len, int B, int N,
                       void* out_key, void* out_value, sv_dtype dst, void* stream) {
    RowsArgs a{};
    if (dst != SV_F32 && dst != SV_BF16) return SV_ERR_INVALID_ARG;
    if (!sv::paged_cache_args(cache, a.c) || !rows_sizes_ok(a.c, B, N)) return SV_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return SV_OK;
    const int es = dst == SV_BF16 ? 2 : 4;
    if (!cache->page_table || !out_key || !out_value || !base || ((uintptr_t)out_key | (uintptr_t)out_value) % es) return SV_ERR_INVALID_ARG;
    a.base = base;
    a.new_len = new_len;
    a.N = N;
    a.key = static_cast<const unsigned char*>(out_key);
    a.value = static_cast<const unsigned char*>(out_value);
    a.sh = a.c.dim;
    a.st = a.sh * a.c.heads;
    a.sb = a.st * N;
    return run_rows<true>(a, cache->dtype == SV_CACHE_E4M3, dst, rows_aligned(a, cache, es), B, (cudaStream_t)stream);
}

sv_status spec_kv_compact_paged(void* const* kv_buffers, int num_buffers, int64_t page_stride, int64_t plane_stride,
                                int num_planes, int64_t row_stride, int64_t row_bytes, const int32_t* page_table,
                                int num_pages, int page_size, int max_pages, const int32_t* path,
                                const int32_t* count, const int32_t* base, int B, int max_depth, void* stream) {
    if (B < 0 || B > kMaxB || num_buffers < 1 || num_buffers > kKvMaxBuffers || num_planes < 1 || max_depth < 1 ||
        max_depth > kKvMaxDepth || row_bytes < 1 || row_stride < row_bytes || page_stride < 0 || plane_stride < 0 ||
        num_pages < 1 || page_size < 1 || page_size > 65536 || max_pages < 1 ||
        (int64_t)max_pages * page_size > sv::PAGED_MAX_POS)
        return SV_ERR_INVALID_ARG;
    if (B == 0) return SV_OK;
    if (!kv_buffers || !page_table || !path || !count) return SV_ERR_INVALID_ARG;
    PagedMoveArgs a{};
    uint64_t align = (uint64_t)page_stride | (uint64_t)plane_stride | (uint64_t)row_stride | (uint64_t)row_bytes;
    for (int k = 0; k < num_buffers; ++k) {
        if (!kv_buffers[k]) return SV_ERR_INVALID_ARG;
        a.buf[k] = static_cast<unsigned char*>(kv_buffers[k]);
        align |= (uint64_t)(uintptr_t)kv_buffers[k];
    }
    const int pw = (align % 16 == 0) ? 16 : (align % 4 == 0) ? 4 : 1;
    const int64_t pieces = row_bytes / pw;
    const int64_t limit = (int64_t)INT32_MAX - kThreads;
    if (pieces > limit || (int64_t)num_planes > limit / pieces || (int64_t)num_buffers > limit / (pieces * num_planes))
        return SV_ERR_INVALID_ARG;
    const int64_t total = (int64_t)num_buffers * num_planes * pieces;
    a.page_stride = page_stride;
    a.plane_stride = plane_stride;
    a.row_stride = row_stride;
    a.num_planes = num_planes;
    a.pieces = (int)pieces;
    a.D = max_depth;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.total = (unsigned)total;
    a.table = page_table;
    a.path = path;
    a.count = count;
    a.base = base;
    const dim3 grid((unsigned)((total + kThreads - 1) / kThreads), (unsigned)B);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (pw == 16) e = sv::launch_serial(kv_compact_paged_kernel<16>, grid, dim3(kThreads), 0, s, a);
    else if (pw == 4) e = sv::launch_serial(kv_compact_paged_kernel<4>, grid, dim3(kThreads), 0, s, a);
    else e = sv::launch_serial(kv_compact_paged_kernel<1>, grid, dim3(kThreads), 0, s, a);
    return sv::launch_status(e);
}

}  // extern "C"
