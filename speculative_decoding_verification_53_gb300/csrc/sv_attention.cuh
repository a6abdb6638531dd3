// sv_attention.cuh -- what the paged-attention kernels share: their arguments, which rows
// and positions a CTA works on, what a query sees, and where results go.
//
// A CTA works on one batch row b, one cache head h, one tile of query rows and one stretch
// of positions ("split").  Query rows are the pairs (query i, head of h's group) in the
// order r = i * group + g, so the queries that share a cache head share its loads.
#pragma once

#include <cuda.h>

#include "sv_internal.h"
#include "sv_paged.cuh"

namespace sv {

struct AttnArgs {
    PagedCache c;
    const uint16_t* q;         // bf16, element strides below
    int64_t q_sb, q_st, q_sh;
    const int32_t* base;
    const int32_t* new_len;    // or nullptr
    const uint32_t* tree_mask; // [B][Q-1][mask_words] or nullptr
    float scale_log2;          // scale * log2(e)
    int Q, Hq, group, mask_words;
    int m_tiles;               // tiles of query rows per (batch row, cache head)
    int whole;                 // tiles [0, whole) are not split, the others `splits` ways
    int splits, chunk;         // a row tile has a split per `chunk` positions, `splits` at most
    int per;                   // splits that a CTA takes: 1 or 2, whose results it joins itself
    int part_rows;             // rows of a tile in the partial results
    int equal;                 // splits are of one length
    int sort;                  // > 0: this many batch rows, taken longest splits first
    int stall_row;             // test hook, -1: none (sv_attention.cu)
    uint16_t* out;             // [B][Q][Hq][D] bf16
    float* lse;                // [B][Q][Hq] or nullptr
    float* part_o;             // [split tile][split / per][part_rows][D] fp32
    float* part_lse;           // [split tile][split / per][part_rows], base 2
};

// Tiles are numbered with the last row tiles first: a chain's late queries see most
// positions, so the long tiles start first and the short ones, which are split, end.
struct AttnPlace {
    int b, h, mt;
};
__device__ __forceinline__ AttnPlace attn_place(const AttnArgs& a, int pairs, unsigned tile) {
    AttnPlace p;
    const int pair = (int)(tile % (unsigned)pairs);
    p.mt = a.m_tiles - 1 - (int)(tile / (unsigned)pairs);
    p.h = pair % a.c.heads;
    p.b = pair / a.c.heads;
    return p;
}

struct AttnTile {
    int b, h, mt, split;
    int base, n;       // positions before the chunk, real queries
    int begin, end;    // this CTA's positions
    int end2;          // of a second split behind them, where a CTA takes two (end: it has none)
    int parts;         // CTAs of this row tile that have positions
    int64_t part;      // first row of this CTA's partial results
};

// End of the positions that rows [0, last query of the tile] can see.
__host__ __device__ __forceinline__ int attn_tile_end(int base, int n, int group, int mt, int tile_rows, bool tree) {
    if (tree) return base + n;
    int last = ((mt + 1) * tile_rows - 1) / group;
    if (last > n - 1) last = n - 1;
    return base + last + 1;
}

// Splits of a row tile that have positions.
__device__ __forceinline__ int attn_active(const AttnArgs& a, int end) {
    int n = (end + a.chunk - 1) / a.chunk;
    if (n > a.splits) n = a.splits;
    return (n & (a.per - 1)) && end > 128 * n ? n + 1 : n;  // splits is a multiple of per
}

// CTAs that take n splits.
__device__ __forceinline__ int attn_parts(const AttnArgs& a, int n) { return (n + a.per - 1) / a.per; }

// First position of split s of n over `end` positions.  Splits of a row tile are of one length,
// in units of 128, and with the longest first (below) a batch of unequal contexts ends together:
// 16 trees of 61 rows x 4 heads over 2048 to 8192 positions of 8 heads, e4m3, 172 us with splits of
// `chunk` positions and a rest, 158 of one length, 151 sorted as well; equal contexts lose 1 us to
// the sort and up to 4 % to the rounding.  16-row tiles keep `chunk`: equal contexts took 139 us
// with it against 148 (16 x 8192, e4m3), unequal ones gained 2 %.  One CTA per SM with an even
// share of all positions, cut where it ends, took 175: a piece costs 10 us of its own, not kept.
__device__ __forceinline__ int attn_split_begin(const AttnArgs& a, int end, int s, int n) {
    if (!a.equal) return s * a.chunk;
    return (int)((unsigned)((end + 127) / 128) * (unsigned)s / (unsigned)n) * 128;  // 2^23 units, 256 splits
}

// The batch row whose splits are the r-th longest, of at most 32 rows (more even out by
// themselves); by whole warps.
__device__ __forceinline__ int attn_sorted(const AttnArgs& a, int r) {
    const int lane = threadIdx.x & 31;
    int base, n, size = -1;
    if (lane < a.sort) {
        size = 0;
        if (paged_row(a.c, a.base, a.new_len, lane, a.Q, base, n) && n > 0) size = attn_split_begin(a, base + n, 1, attn_active(a, base + n));
    }
    int before = 0;
    for (int j = 0; j < a.sort; ++j) {
        const int other = __shfl_sync(0xffffffffu, size, j);
        before += other > size || (other == size && j < lane);
    }
    return __ffs(__ballot_sync(0xffffffffu, lane < a.sort && before == r)) - 1;
}

// The work of CTA `id` (pairs: batch rows times cache heads; per: splits that a CTA takes);
// false where it has none.
__device__ __forceinline__ bool attn_tile(const AttnArgs& a, int pairs, unsigned id, int tile_rows, int per, AttnTile& t) {
    const bool whole = id < (unsigned)a.whole;
    const unsigned rest = id - (unsigned)a.whole, each = (unsigned)(a.splits / per);
    unsigned tile = rest / each;  // among the split ones
    AttnPlace p = attn_place(a, pairs, whole ? id : (unsigned)a.whole + tile);
    if (a.sort) {
        const int b = attn_sorted(a, p.b);
        tile += (b - p.b) * a.c.heads;
        p.b = b;
    }
    t.b = p.b;
    t.h = p.h;
    t.mt = p.mt;
    t.split = whole ? 0 : (int)(rest % each) * per;
    t.part = whole ? 0 : ((int64_t)tile * each + rest % each) * a.part_rows;
    if (!paged_row(a.c, a.base, a.new_len, t.b, a.Q, t.base, t.n)) return false;
    if ((int64_t)t.mt * tile_rows >= (int64_t)t.n * a.group) return false;
    const int end = attn_tile_end(t.base, t.n, a.group, t.mt, tile_rows, a.tree_mask != nullptr);
    const int active = whole ? 1 : attn_active(a, end);
    if (t.split >= active) return false;
    t.parts = attn_parts(a, active);
    t.begin = attn_split_begin(a, end, t.split, active);
    t.end = t.split == active - 1 ? end : attn_split_begin(a, end, t.split + 1, active);
    t.end2 = t.split + 1 >= active ? t.end : t.split + 2 == active ? end : attn_split_begin(a, end, t.split + 2, active);
    return true;
}

// Bits of `count` (at most 32) positions from pos0 on that query i sees by the mask alone
// (holes and the end of the sequence are the caller's): the context, and of the chunk
// what the chain or the tree shows.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

__device__ __forceinline__ uint32_t attn_visible(const AttnArgs& a, const AttnTile& t, int i, int pos0) {
    if (!a.tree_mask) return low_bits(t.base + i + 1 - pos0);
    uint32_t bits = low_bits(t.base + 1 - pos0);  // context and root
    const int j0 = pos0 - t.base - 1;             // node of bit 0
    if (i > 0 && j0 > -32) {
        const uint32_t* row = a.tree_mask + ((int64_t)t.b * (a.Q - 1) + (i - 1)) * a.mask_words;
        if (j0 < 0) {
            bits |= __ldg(row) << (-j0);
        } else if ((j0 >> 5) < a.mask_words) {
            const int w = j0 >> 5;
            const uint32_t lo = __ldg(row + w), hi = w + 1 < a.mask_words ? __ldg(row + w + 1) : 0u;
            bits |= __funnelshift_r(lo, hi, j0 & 31);
        }
    }
    return bits;
}

// Element d of the value at a position, from the cache itself (0 in a hole).
template <bool E4M3>
__device__ __forceinline__ float attn_value(const AttnArgs& a, const AttnTile& t, int pos, int d) {
    int row;
    const int page = paged_place(a.c, t.b, pos, row);
    if (page < 0) return 0.0f;
    const unsigned char* p = a.c.v + page * a.c.page_stride + t.h * a.c.head_stride + row * a.c.row_stride;
    if (!E4M3) return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + d) << 16);
    const float s = __ldg(a.c.v_scale + ((int64_t)page * a.c.heads + t.h) * a.c.page_size + row);
    return e4m3x2_to_f32(__ldg(p + d)).x * s;
}

// Index of query row r's (query, head) in [B][Q][Hq].
__device__ __forceinline__ int64_t attn_row(const AttnArgs& a, const AttnTile& t, int r) {
    return ((int64_t)t.b * a.Q + r / a.group) * a.Hq + t.h * a.group + r % a.group;
}

// One box of a page (some elements x rows of one head) by the copy engine; a page
// outside the cache reads as zeros.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int row, int head, int page, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(row), "r"(head), "r"(page), "r"(smem_u32(bar))
                 : "memory");
}

// Takes values that are not finite out of 16 bytes (codes, or bf16); true if there were any.
template <bool E4M3>
__device__ __forceinline__ bool sanitise(uint4& v) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        constexpr uint32_t ones = E4M3 ? 0x7fu : 0x7f80u, all = E4M3 ? 0xffu : 0xffffu;
#pragma unroll
        for (int y = 0; y < 32; y += E4M3 ? 8 : 16)
            if (((w[i] >> y) & ones) == ones) {
                w[i] &= ~(all << y);
                bad = true;
            }
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
    return bad;
}

// cuTensorMapEncodeTiled, found through the runtime (the library does not link the driver).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// A map of pages [page][head][row][element] for boxes of `rows` rows of `width` elements.
inline bool page_map(CUtensorMap* map, const void* pages, const PagedCache& c, bool e4m3, int width, int rows,
                     CUtensorMapSwizzle swizzle) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)c.page_size, (cuuint64_t)c.heads, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.row_stride, (cuuint64_t)c.head_stride, (cuuint64_t)c.page_stride};
    const cuuint32_t box[4] = {(cuuint32_t)width, (cuuint32_t)rows, 1, 1}, ones[4] = {1, 1, 1, 1};
    return f(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pages), dims,
             strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows per box where the copy engine can fill a tile of `tile` positions (pages of 8 rows up
// that divide it, or of a multiple of it: a box lies in one page and starts on a swizzle
// atom), else 0: cp.async then copies row by row.
inline int page_box_rows(const PagedCache& c, int tile) {
    if (c.page_size >= tile) return c.page_size % tile == 0 ? tile : 0;
    return c.page_size >= 8 && tile % c.page_size == 0 ? c.page_size : 0;
}

// The kernel for many query rows per cache head, or wide heads (sv_attention_tc.cu): tile_rows
// 128 or 256, 128 for heads wider than 128; dual (tile_rows 128, heads of up to 128): a CTA
// takes two splits.
cudaError_t launch_attn_tc(const AttnArgs& a, int pairs, bool e4m3, int tile_rows, bool dual, unsigned ctas,
                           cudaStream_t stream);

}  // namespace sv
