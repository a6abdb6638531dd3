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
#include "sv_rows.cuh"

namespace {

using sv::Eight;
using sv::EightOfCache;
using sv::PagedCache;
using sv::pdl_trigger;
using sv::pdl_wait;
using sv::store_cache_row;
using sv::store_row8;

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
