// sv_paged.cuh -- what the kernels over a paged key/value cache share: the cache as the
// kernels see it, the place of a position, 8-bit float conversions, and the host checks.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "spec_paged_kv.h"
#include "sv_common.cuh"

namespace sv {

constexpr float E4M3_MAX = 448.0f;
constexpr int PAGED_MAX_DIM = 256;
constexpr int PAGED_MAX_HEADS = 1024;
constexpr int PAGED_MAX_POS = 1 << 30;  // positions of a page table's row: index sums stay within int

struct PagedCache {
    unsigned char* k;
    unsigned char* v;
    float* k_scale;
    float* v_scale;
    const int32_t* table;
    int64_t page_stride, head_stride, row_stride;  // bytes
    int num_pages, page_size, max_pages, heads, dim;
};

// The rows of batch row b: false where the call leaves the batch row untouched.
__device__ __forceinline__ bool paged_row(const PagedCache& c, const int32_t* base, const int32_t* new_len, int b,
                                          int N, int& first, int& n) {
    first = __ldg(base + b);
    n = new_len ? __ldg(new_len + b) : N;
    return first >= 0 && n >= 0 && n <= N && (int64_t)first + n <= (int64_t)c.max_pages * c.page_size;
}

// Page and row of position pos of batch row b (0 <= pos < max_pages * page_size); the page
// is -1 in a hole.
__device__ __forceinline__ int paged_place(const PagedCache& c, int b, int pos, int& row) {
    const int i = pos / c.page_size;
    row = pos - i * c.page_size;
    const int p = __ldg(c.table + (int64_t)b * c.max_pages + i);
    return (unsigned)p < (unsigned)c.num_pages ? p : -1;
}

__device__ __forceinline__ bool not_finite(float x) { return !(fabsf(x) < pos_inf()); }

// Two fp32 values to two e4m3 codes (lo in the low byte): nearest even, saturating at
// +-448, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes (the low half of w) as two fp32 values, exactly.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t w) {
    uint32_t h;
    asm("{.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(w));
    float2 f;
    asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

// Two fp32 values rounded to bf16 (nearest even), lo in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Host checks of a cache description and the kernels' view of it.
inline bool paged_cache_args(const sv_paged_cache* c, PagedCache& out) {
    if (!c) return false;
    if (c->dtype != SV_CACHE_BF16 && c->dtype != SV_CACHE_E4M3) return false;
    if (c->num_pages < 1 || c->page_size < 1 || c->page_size > 65536 || c->max_pages < 1 ||
        (int64_t)c->max_pages * c->page_size > PAGED_MAX_POS || c->num_heads < 1 ||
        c->num_heads > PAGED_MAX_HEADS || c->head_dim < 1 || c->head_dim > PAGED_MAX_DIM)
        return false;
    const int64_t es = c->dtype == SV_CACHE_BF16 ? 2 : 1;
    if (c->page_stride < 0 || c->head_stride < 0 || c->row_stride < es * c->head_dim) return false;
    if ((c->page_stride | c->head_stride | c->row_stride) % es) return false;
    if (!c->k_pages || !c->v_pages) return false;  // the table may be NULL in a call on no rows
    if (((uintptr_t)c->k_pages | (uintptr_t)c->v_pages) % es) return false;
    if (c->dtype == SV_CACHE_E4M3 && (!c->k_scale || !c->v_scale)) return false;
    out = PagedCache{static_cast<unsigned char*>(c->k_pages), static_cast<unsigned char*>(c->v_pages), c->k_scale,
                     c->v_scale, c->page_table, c->page_stride, c->head_stride, c->row_stride, c->num_pages,
                     c->page_size, c->max_pages, c->num_heads, c->head_dim};
    return true;
}

// A launch with programmatic stream serialization (the kernels call pdl_wait first).
template <typename Kern, typename... Args>
cudaError_t launch_serial(Kern kern, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace sv
