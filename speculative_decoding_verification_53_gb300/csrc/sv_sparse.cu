// sv_sparse.cu -- lists of blocks turned into page tables for the attention kernels
// (include/spec_sparse.h).
//
// Attention over listed blocks is attention over a shorter sequence: the listed context blocks,
// which are whole and which every query of the list sees, then the blocks from the chunk's first on
// under the mask.  So each list becomes a row of a page table of its own, with its own number of positions
// before the chunk, and the kernels of spec_paged_attention run over that (sv_attention.cuh).
#include <cstdint>

#include "sv_attention.cuh"

namespace {

constexpr int kThreads = 256;

// One warp per list: blocks that count, in order, then those from base / page_size on.
__global__ void __launch_bounds__(kThreads) block_table_kernel(const __grid_constant__ sv::PagedCache c,
                                                               const int32_t* base, const int32_t* new_len,
                                                               const int32_t* blocks, int num_blocks, int lists, int64_t rows,
                                                               int Q, int32_t* table, int32_t* out_base, int width) {
    sv::pdl_trigger();
    sv::pdl_wait();
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const int b = (int)(row / c.heads / lists);
    int first, n;
    if (!sv::paged_row(c, base, new_len, b, Q, first, n)) {
        if (lane == 0) out_base[row] = -1;  // left untouched
        return;
    }
    const int full = first / c.page_size;
    const int32_t* own = c.table + (int64_t)b * c.max_pages;
    const int32_t* list = blocks + row * num_blocks;
    int32_t* to = table + row * width;
    int count = 0, most = -1;  // taken, and the largest of them
    for (int x0 = 0; x0 < num_blocks; x0 += 32) {
        int e = x0 + lane < num_blocks ? __ldg(list + x0 + lane) : -1;
        if (e >= full) e = -1;
        int up = e;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up = max(up, y);
        }
        int before = __shfl_up_sync(0xffffffffu, up, 1);
        before = lane ? max(before, most) : most;
        const bool take = e >= 0 && e > before;
        const uint32_t mask = __ballot_sync(0xffffffffu, take);
        if (take) to[count + __popc(mask & ((1u << lane) - 1u))] = __ldg(own + e);
        count += __popc(mask);
        most = max(most, __shfl_sync(0xffffffffu, up, 31));
    }
    const int last = n ? (first + n - 1) / c.page_size : full - 1;
    for (int k = lane; full + k <= last; k += 32) to[count + k] = __ldg(own + full + k);
    if (lane == 0) out_base[row] = count * c.page_size + (first - full * c.page_size);
}

}  // namespace

namespace sv {

cudaError_t launch_block_tables(const PagedCache& c, const int32_t* base, const int32_t* new_len, const int32_t* blocks,
                                int num_blocks, int lists, int64_t rows, int Q, int32_t* table, int32_t* out_base,
                                int width, cudaStream_t stream) {
    constexpr int per = kThreads / 32;
    return launch_serial(block_table_kernel, dim3((unsigned)((rows + per - 1) / per)), dim3(kThreads), 0, stream, c, base,
                         new_len, blocks, num_blocks, lists, rows, Q, table, out_base, width);
}

}  // namespace sv
