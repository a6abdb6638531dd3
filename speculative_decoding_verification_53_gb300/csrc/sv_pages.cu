// sv_pages.cu -- page tables kept on the device (include/spec_pages.h): rows grow and
// shrink to their lengths by a stack of free pages, and new tokens get their slots.
//
// There is no arithmetic to speak of: a call reads the rows' lengths, moves the entries
// that change between table and stack, and writes the slots.  What it costs is latency, a
// chain of dependent steps (count what goes back, sum over the rows before, push, take,
// look up), so all of them are in one launch: one cluster, whose CTAs each sum over all rows by
// themselves and meet at the cluster's barrier between the steps.  Nothing is left to the
// order in which threads arrive: the stack's order follows from the rows' order.
// The work is cut into units, a part of a row each, one warp at a time; every CTA keeps what
// every unit pushes and takes, and its prefix sums, in shared memory (12 bytes a unit).
#include <climits>
#include <cstdint>

#include "spec_pages.h"
#include "sv_internal.h"
#include "sv_paged.cuh"

namespace {

constexpr int kMaxRows = 16384;
constexpr int kBad = INT_MIN;              // a unit of a row that is left untouched
constexpr uint32_t kMost = 0x7fffffffu;    // sums saturate
constexpr int kMaxPages = 1 << 30;

struct PagesArgs {
    int32_t* table;
    int32_t* pages;
    const int32_t* length;
    int32_t* stack;
    int32_t* count;
    const int32_t* base;
    int64_t* slots;
    int32_t* ok;
    int num_pages, page_size, max_pages, B, N;
    int parts;  // units of a row
    int shift;  // log2 of page_size, -1 where it is no power of two
};

__device__ __forceinline__ uint32_t sum_sat(uint32_t a, uint32_t b) { return min(a + b, kMost); }

// The entries [lo, hi) of row b's table that part `part` of `parts` moves: taken where grow, given
// back otherwise; false for a row that is left untouched.
__device__ __forceinline__ bool pages_unit(const PagesArgs& a, int b, int part, int& lo, int& hi, bool& grow) {
    const int length = __ldg(a.length + b), have = a.pages[b];
    lo = hi = 0;
    if (length < 0 || (int64_t)length > (int64_t)a.max_pages * a.page_size || have < 0 || have > a.max_pages) return false;
    const int need = (int)(((unsigned)length + (unsigned)a.page_size - 1u) / (unsigned)a.page_size);
    grow = need > have;
    const int from = grow ? have : need, to = grow ? need : have;
    const int each = (to - from + a.parts - 1) / a.parts;
    lo = (int)min((int64_t)to, (int64_t)from + (int64_t)part * each);
    hi = min(to, lo + each);
    return true;
}

__device__ __forceinline__ int64_t slot_of(const PagesArgs& a, int b, int length, int64_t pos) {
    if (pos < 0 || pos >= length) return -1;
    const int i = a.shift >= 0 ? (int)pos >> a.shift : (int)pos / a.page_size;
    const int p = __ldcg(a.table + (int64_t)b * a.max_pages + i);
    return (unsigned)p < (unsigned)a.num_pages ? (int64_t)p * a.page_size + ((int)pos - i * a.page_size) : -1;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) page_resize_kernel(const __grid_constant__ PagesArgs a) {
    extern __shared__ int s_change[];  // of each unit: > 0 taken, < 0 given back
    constexpr int kWarps = kThreads / 32;
    __shared__ uint32_t s_sum[2][kWarps];
    const int units = a.B * a.parts;
    uint32_t* s_take = reinterpret_cast<uint32_t*>(s_change) + units;  // [units + 1]: before each unit
    uint32_t* s_push = s_take + units + 1;                             // [units + 1]
    sv::pdl_trigger();
    sv::pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ranks = (int)sv::cluster_size(), rank = (int)sv::cluster_rank();
    const int first = rank * kWarps + warp, stride = ranks * kWarps;  // this warp's units
    const int start = min(max(a.count[0], 0), a.num_pages);

    // Entries [e0, e0 + 256) of what a unit gives back, eight of a lane in flight.
    int page[8];
    auto fetch = [&](const int32_t* row, int e0, int hi) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int e = e0 + 32 * k + lane;
            page[k] = e < hi ? __ldcg(row + e) : -1;
        }
    };
    const bool one = units <= stride;  // a warp has one unit at most, and keeps the first of its entries

    if (ranks > 1) sv::cluster_sync_all();  // every CTA runs before its shared memory is written
    for (int u = first; u < units; u += stride) {
        const int b = u / a.parts;
        int lo, hi, change;
        bool grow;
        if (!pages_unit(a, b, u - b * a.parts, lo, hi, grow)) {
            change = kBad;
        } else if (grow) {
            change = hi - lo;
        } else {
            const int32_t* row = a.table + (int64_t)b * a.max_pages;
            int held = 0;
#pragma unroll 8
            for (int e = lo + 256 + lane; e < hi; e += 32) held += (unsigned)__ldcg(row + e) < (unsigned)a.num_pages;
            fetch(row, lo, hi);
#pragma unroll
            for (int k = 0; k < 8; ++k) held += (unsigned)page[k] < (unsigned)a.num_pages;
            change = -(int)__reduce_add_sync(0xffffffffu, (unsigned)held);
        }
        if (lane < ranks) {
            const uint32_t to = sv::dsmem_addr(s_change + u, (uint32_t)lane);
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(change) : "memory");
        }
    }
    if (ranks > 1) sv::cluster_sync_all();
    else __syncthreads();

    // prefix sums over the units, in every CTA
    const int per = (units + kThreads - 1) / kThreads;
    const int u0 = min(units, tid * per), u1 = min(units, u0 + per);
    uint32_t take = 0u, push = 0u;
    for (int u = u0; u < u1; ++u) {
        const int c = s_change[u];
        if (c > 0) take = sum_sat(take, (uint32_t)c);
        else if (c != kBad) push = sum_sat(push, (uint32_t)-c);
    }
    uint32_t t = take, p = push;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, t, x), z = __shfl_up_sync(0xffffffffu, p, x);
        if (lane >= x) {
            t = sum_sat(t, y);
            p = sum_sat(p, z);
        }
    }
    if (lane == 31) {
        s_sum[0][warp] = t;
        s_sum[1][warp] = p;
    }
    __syncthreads();
    uint32_t before_t = 0u, before_p = 0u, all_t = 0u, all_p = 0u;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) {
            before_t = all_t;
            before_p = all_p;
        }
        all_t = sum_sat(all_t, s_sum[0][w]);
        all_p = sum_sat(all_p, s_sum[1][w]);
    }
    t = __shfl_up_sync(0xffffffffu, t, 1);
    p = __shfl_up_sync(0xffffffffu, p, 1);
    take = sum_sat(before_t, lane ? t : 0u);
    push = sum_sat(before_p, lane ? p : 0u);
    for (int u = u0; u < u1; ++u) {
        const int c = s_change[u];
        s_take[u] = take;
        s_push[u] = push;
        if (c > 0) take = sum_sat(take, (uint32_t)c);
        else if (c != kBad) push = sum_sat(push, (uint32_t)-c);
    }
    if (tid == 0) {
        s_take[units] = all_t;
        s_push[units] = all_p;
    }
    __syncthreads();
    const uint32_t top = min(sum_sat((uint32_t)start, all_p), (uint32_t)a.num_pages);

    for (int u = first; u < units; u += stride) {  // what goes back
        const int c = s_change[u];
        if (c > 0 || c == kBad) continue;
        const int b = u / a.parts;
        int lo, hi;
        bool grow;
        pages_unit(a, b, u - b * a.parts, lo, hi, grow);
        int32_t* row = a.table + (int64_t)b * a.max_pages;
        uint32_t at = sum_sat((uint32_t)start, s_push[u]);
        for (int e0 = lo; e0 < hi; e0 += 256) {
            if (!one || e0 > lo) fetch(row, e0, hi);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int e = e0 + 32 * k + lane;
                const bool held = (unsigned)page[k] < (unsigned)a.num_pages;
                const uint32_t mask = __ballot_sync(0xffffffffu, held);
                const uint32_t to = sum_sat(at, __popc(mask & ((1u << lane) - 1u)));
                if (held && to < (uint32_t)a.num_pages) a.stack[to] = page[k];
                if (e < hi) row[e] = -1;
                at = sum_sat(at, __popc(mask));
            }
        }
    }
    if (ranks > 1) sv::cluster_sync_all();
    else __syncthreads();

    for (int u = first; u < units; u += stride) {  // what is taken
        const int c = s_change[u];
        if (c <= 0) continue;
        const int b = u / a.parts;
        if (s_take[(b + 1) * a.parts] > top) continue;
        int lo, hi;
        bool grow;
        pages_unit(a, b, u - b * a.parts, lo, hi, grow);
        int32_t* row = a.table + (int64_t)b * a.max_pages;
        const int32_t* from = a.stack + (top - 1u - s_take[u]);
#pragma unroll 8
        for (int e = lane; e < hi - lo; e += 32) row[lo + e] = __ldcg(from - e);
    }
    if (ranks > 1) sv::cluster_sync_all();
    else __syncthreads();

    // Rows' new state; pages and count are read no more.
    auto fine = [&](int b) {
        const int u = b * a.parts;  // (sums may have saturated; the first part of a row that lacks pages takes some)
        return s_change[u] != kBad && (s_change[u] <= 0 || s_take[u + a.parts] <= top);
    };
    const int all = ranks * kThreads;
    uint32_t taken = 0u;  // by the rows that found enough: they come before those that did not
    for (int b = rank * kThreads + tid; b < a.B; b += all) {
        const bool ok = fine(b);
        if (ok) a.pages[b] = (int)(((unsigned)__ldg(a.length + b) + (unsigned)a.page_size - 1u) / (unsigned)a.page_size);
        a.ok[b] = ok;
    }
    if (rank == 0) {
        for (int b = tid; b < a.B; b += kThreads)
            if (s_take[(b + 1) * a.parts] <= top) taken = max(taken, s_take[(b + 1) * a.parts]);
        taken = __reduce_max_sync(0xffffffffu, taken);
        __syncthreads();
        if (lane == 0) s_sum[0][warp] = taken;
        __syncthreads();
        if (tid == 0) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) taken = max(taken, s_sum[0][w]);
            a.count[0] = (int)(top - taken);
        }
    }
    if (a.slots) {
        const unsigned total = (unsigned)a.B * (unsigned)a.N;
        for (unsigned x = rank * kThreads + tid; x < total; x += all) {
            const int b = (int)(x / (unsigned)a.N), i = (int)(x - (unsigned)b * (unsigned)a.N);
            a.slots[x] = fine(b) ? slot_of(a, b, __ldg(a.length + b), (int64_t)__ldg(a.base + b) + i) : -1;
        }
    }
}

// Up to `most` CTAs of one cluster.
template <int kThreads>
cudaError_t launch_resize(PagesArgs& a, int most, cudaStream_t stream) {
    static sv::KernelLaunchCache cache;
    auto kern = page_resize_kernel<kThreads>;
    int max_dyn = 0;
    cudaError_t e = cache.setup((const void*)kern, &max_dyn);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    auto parts_of = [&](int ranks) { return ranks * (kThreads / 32) > a.B ? ranks * (kThreads / 32) / a.B : 1; };
    // in steps of 16 KB: what fits on the device is remembered for each size
    auto smem_of = [&](int ranks) { return (((size_t)3 * a.B * parts_of(ranks) + 2) * sizeof(int) + 16383) / 16384 * 16384; };
    int ranks = 1;
    if (most > 1) e = cache.pick_cluster((const void*)kern, cfg, most, smem_of, &ranks);
    if (e != cudaSuccess) return e;
    if (ranks < 1 || smem_of(ranks) > (size_t)max_dyn) return cudaErrorInvalidValue;
    a.parts = parts_of(ranks);
    cfg.gridDim = dim3((unsigned)ranks);
    cfg.dynamicSmemBytes = smem_of(ranks);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

constexpr int kSlotThreads = 256, kSlotsEach = 8;

// Slots of many tokens, on the whole device; grid: x over a row's tokens, y the row.
__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const __grid_constant__ PagesArgs a) {
    sv::pdl_trigger();
    sv::pdl_wait();
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const bool ok = a.ok[b] != 0;
        const int length = __ldg(a.length + b), base = __ldg(a.base + b);
        int64_t* out = a.slots + (int64_t)b * a.N;
#pragma unroll
        for (int k = 0; k < kSlotsEach; ++k) {
            const int64_t i = (int64_t)blockIdx.x * (kSlotThreads * kSlotsEach) + k * kSlotThreads + threadIdx.x;
            if (i < a.N) out[i] = ok ? slot_of(a, b, length, base + i) : -1;
        }
    }
}

}  // namespace

extern "C" sv_status spec_page_resize(int32_t* page_table, int32_t* pages, const int32_t* length, int32_t* free_pages,
                                      int32_t* free_count, int num_pages, int page_size, int max_pages,
                                      const int32_t* base, int64_t* out_slots, int32_t* out_ok, int B, int N,
                                      void* stream) {
    if (B < 0 || B > kMaxRows || num_pages < 0 || num_pages > kMaxPages || page_size < 1 || page_size > 65536 ||
        max_pages < 1 || (int64_t)max_pages * page_size > sv::PAGED_MAX_POS || N < 0 || N > sv::PAGED_MAX_POS ||
        (int64_t)B * N >= ((int64_t)1 << 40))
        return SV_ERR_INVALID_ARG;
    if (!base != !out_slots) return SV_ERR_INVALID_ARG;
    if (B == 0) return SV_OK;
    if (!page_table || !pages || !length || (num_pages && !free_pages) || !free_count || !out_ok) return SV_ERR_INVALID_ARG;
    PagesArgs a{page_table, pages, length, free_pages, free_count, base, out_slots, out_ok,
                num_pages, page_size, max_pages, B, N, 1, -1};
    if ((page_size & (page_size - 1)) == 0)
        for (a.shift = 0; 1 << a.shift < page_size;) ++a.shift;
    const bool slots = out_slots && N > 0;
    const int64_t tokens = slots ? (int64_t)B * N : 0;
    const bool apart = tokens > 32768;  // slots by a kernel of their own
    if (apart || !slots) a.slots = nullptr;
    // One small CTA where little can move, else the largest cluster.  For a pair of calls, 8 rows of which each gains and
    // loses a page: 8.1 us by 256 threads, 9.1 by 512, 12 by 1024; 128 rows that move 256 to 1250 pages each, with 2^20
    // slots: 28.8 us by 16 CTAs of 1024 threads, 32.7 by 16 of 512, 45 by 8 of 512.
    cudaError_t e = B > 32 || tokens > 16384 ? launch_resize<1024>(a, 16, (cudaStream_t)stream) : launch_resize<256>(a, 1, (cudaStream_t)stream);
    if (e == cudaSuccess && apart) {
        a.slots = out_slots;
        const int per = kSlotThreads * kSlotsEach;
        e = sv::launch_serial(slot_map_kernel, dim3((unsigned)((N + per - 1) / per), (unsigned)B), dim3(kSlotThreads), 0,
                              (cudaStream_t)stream, a);
    }
    return sv::launch_status(e);
}
