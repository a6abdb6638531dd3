// sv_logits.cu -- penalties, biases and grammar masks on the logits of every row of a
// verify call (include/spec_logits.h).
//
// A CTA takes one batch row and a slice of the vocabulary: every S-th block of 256 tokens, so
// that the frequent tokens, which have low numbers in most vocabularies, are spread over the
// slices (with contiguous slices the first one's CTA ran 5 times as long as the others).
// From the row's token lists it
// builds a table of its slice in shared memory, one word per token (the count in the
// output so far, and a flag for "in the prompt") and, where biases are given, the bias,
// and from it the list of the tokens that have anything; both serve all R rows.  Then each
// warp takes rows of the slice in turn:
//   out of place it copies the row's part, 16 bytes per lane, with -inf where the grammar
//   says so (and does not read what the grammar rules out); in place it writes those -inf only;
//   then it goes through the list, one token per lane, and rewrites those elements;
//   last come the row's drafted tokens (the prefix of a chain, the ancestors in a tree), whose
//   counts are the row's own.
// Copy and list are apart because a group of eight tokens with one listed token among a
// warp's 32 groups is the rule: looking the table up in the copy ran the penalties' code for
// every group (205 instructions a group, 250 us for 16 trees of 61 rows of 128256).
// Nothing in shared memory changes while rows are at work, and no result depends on the
// order of atomics (counts are integers; of two biases of one token the later entry holds;
// the list's order does not matter).
#include <cstdint>

#include "spec_logits.h"
#include "sv_common.cuh"
#include "sv_internal.h"
#include "sv_paged.cuh"

namespace {

using sv::neg_inf;
using sv::pdl_trigger;
using sv::pdl_wait;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxB = 65535;
constexpr int kMaxRows = 1025;
constexpr int kMaxV = 1 << 24;
constexpr int kBlock = 256;       // consecutive tokens of a slice
constexpr int kMaxSlice = 16384;  // tokens of a slice
constexpr uint32_t kPrompt = 0x80000000u;  // table flag; the low 31 bits count

struct AdjustArgs {
    const void* logits;
    void* out;
    const int32_t* history;
    const int32_t* history_len;
    const int32_t* prompt_len;
    const int32_t* drafts;
    const uint32_t* tree_mask;
    const float* repetition;
    const float* presence;
    const float* frequency;
    const int32_t* bias_tokens;
    const float* bias_values;
    const uint32_t* allowed;
    int H, M, R, V;
    int slice;      // tokens of a slice, a multiple of kBlock
    int log_slices;  // log2 of their number
};

struct Penalty {
    float rep, pres, freq;
};

// x after the penalties of a token with table word w, before bias and mask.
__device__ __forceinline__ float penalised(float x, uint32_t w, const Penalty& p) {
    if (w == 0u) return x;
    x = x > 0.0f ? x / p.rep : x * p.rep;
    const uint32_t c = w & ~kPrompt;
    if (c) x = x - (float)c * p.freq - p.pres;
    return x;
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* row, int v) {
    if (BF16) return __uint_as_float((uint32_t) static_cast<const unsigned short*>(row)[v] << 16);
    return static_cast<const float*>(row)[v];
}
template <bool BF16>
__device__ __forceinline__ void store_logit(void* row, int v, float x) {
    if (BF16) static_cast<unsigned short*>(row)[v] = (unsigned short)sv::bf16x2(x, 0.0f);
    else static_cast<float*>(row)[v] = x;
}

// The 16 bytes of a group with -inf where `keep` has a 0.
template <bool BF16>
__device__ __forceinline__ uint4 masked(uint4 g, uint32_t keep) {
    uint32_t w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (BF16) {
            const uint32_t m = ((keep >> (2 * k)) & 1u ? 0x0000ffffu : 0u) | ((keep >> (2 * k + 1)) & 1u ? 0xffff0000u : 0u);
            w[k] = (w[k] & m) | (0xff80ff80u & ~m);
        } else if (!((keep >> k) & 1u)) {
            w[k] = 0xff800000u;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements of a row up to the next 16-byte boundary.
template <bool BF16>
__device__ __forceinline__ int to_boundary(const void* p) {
    return (int)(((16 - ((uintptr_t)p & 15)) & 15) / (BF16 ? 2 : 4));
}

template <bool BF16, bool BIAS>
__global__ void __launch_bounds__(kThreads, 4) adjust_logits_kernel(const __grid_constant__ AdjustArgs a) {
    pdl_trigger();
    pdl_wait();
    extern __shared__ __align__(16) uint32_t s_table[];  // [slice] words, [slice] biases, per-warp lists
    const int b = blockIdx.y, me = blockIdx.x, slices = 1 << a.log_slices;
    // token v of this slice is entry `local` of the tables (-1: of another slice, or none)
    auto local = [&](int v) {
        const int blk = v >> 8;
        return (unsigned)v < (unsigned)a.V && (blk & (slices - 1)) == me ? (blk >> a.log_slices) << 8 | (v & 255) : -1;
    };
    auto token = [&](int u) { return (((u >> 8) << a.log_slices) + me) << 8 | (u & 255); };
    float* s_bias = reinterpret_cast<float*>(s_table + a.slice);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int N = a.R - 1;
    const bool in_place = a.out == a.logits;
    constexpr int ES = BF16 ? 2 : 4;

    __shared__ int s_nodes, s_count;  // drafted and listed tokens of this slice
    uint16_t* s_listed = reinterpret_cast<uint16_t*>(s_table + a.slice * (BIAS ? 2 : 1));  // [slice] entries
    uint16_t* s_node = s_listed + a.slice;    // [N] drafted nodes of the slice
    uint16_t* s_tok = s_node + N;             // [N] their entries
    uint16_t* s_list = s_tok + N + warp * N;  // this warp's: indices into both

    // Everything the tables need is asked for at once: the first 2048 tokens of the history and
    // the first 256 biases do not wait for the lengths or for the tables to be cleared.
    constexpr int AHEAD = 8;
    const int32_t* hist = a.history + (int64_t)b * a.H;
    const int32_t* bt = a.bias_tokens + (int64_t)b * a.M;
    const float* bv = a.bias_values + (int64_t)b * a.M;
    int ahead[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) ahead[k] = a.history && tid + k * kThreads < a.H ? __ldg(hist + tid + k * kThreads) : -1;
    int len = a.history ? __ldg(a.history_len + b) : 0;
    const int prompt = a.prompt_len ? __ldg(a.prompt_len + b) : 0;
    int bias_at = -1;
    float bias_is = 0.0f;
    if (BIAS && tid < a.M) {
        bias_at = __ldg(bt + tid);
        bias_is = __ldg(bv + tid);
    }
    Penalty pen;
    pen.rep = a.repetition ? __ldg(a.repetition + b) : 1.0f;
    pen.pres = a.presence ? __ldg(a.presence + b) : 0.0f;
    pen.freq = a.frequency ? __ldg(a.frequency + b) : 0.0f;
    for (int i = 4 * tid; i < a.slice * (BIAS ? 2 : 1); i += 4 * kThreads)
        *reinterpret_cast<uint4*>(s_table + i) = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) s_nodes = s_count = 0;
    __syncthreads();
    len = len < 0 ? 0 : len > a.H ? a.H : len;
    auto count = [&](int i, int v) {
        const int u = i < len ? local(v) : -1;
        if (u >= 0) {
            if (i < prompt) atomicOr(s_table + u, kPrompt);
            else atomicAdd(s_table + u, 1u);
        }
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) count(tid + k * kThreads, ahead[k]);
#pragma unroll 8
    for (int i = tid + AHEAD * kThreads; i < len; i += kThreads) count(i, __ldg(hist + i));
    if (BIAS) {
        // the last entry of a token wins: its number + 1 is the largest, and takes the word
        uint32_t* at = reinterpret_cast<uint32_t*>(s_bias);
        auto number = [&](int i, int v) {
            const int u = local(v);
            if (u >= 0) atomicMax(at + u, (uint32_t)i + 1u);
        };
        if (tid < a.M) number(tid, bias_at);
        for (int i = tid + kThreads; i < a.M; i += kThreads) number(i, __ldg(bt + i));
        __syncthreads();
        // a winner knows itself; nobody else's word is its own, and no bias is taken for a number
        // because every word is read before the barrier and written after it
        constexpr int MOST = 256;  // 65535 entries over 256 threads
        uint32_t won[MOST / 32] = {};
        int k = 0;
        for (int i = tid; i < a.M; i += kThreads, ++k) {
            const int u = local(i == tid ? bias_at : __ldg(bt + i));
            if (u >= 0 && at[u] == (uint32_t)i + 1u) won[k >> 5] |= 1u << (k & 31);
        }
        __syncthreads();
        k = 0;
        for (int i = tid; i < a.M; i += kThreads, ++k)
            if ((won[k >> 5] >> (k & 31)) & 1u) s_bias[local(i == tid ? bias_at : __ldg(bt + i))] = i == tid ? bias_is : __ldg(bv + i);
    }
    // drafted tokens of this slice, in node order (one warp, so that the order is fixed)
    if (a.drafts && warp == 0) {
        int have = 0;
        for (int i0 = 0; i0 < N; i0 += 32) {
            const int i = i0 + lane;
            const int u = i < N ? local(__ldg(a.drafts + (int64_t)b * N + i)) : -1;
            const bool in = u >= 0;
            const unsigned m = __ballot_sync(0xffffffffu, in);
            if (in) {
                const int at = have + __popc(m & ((1u << lane) - 1u));
                s_node[at] = (uint16_t)i;
                s_tok[at] = (uint16_t)u;
            }
            have += __popc(m);
        }
        if (lane == 0) s_nodes = have;
    }
    __syncthreads();
    for (int i = tid; i < a.slice; i += kThreads) {
        const bool in = s_table[i] != 0u || (BIAS && s_bias[i] != 0.0f);
        const unsigned m = __ballot_sync(0xffffffffu, in);
        int at = 0;
        if (lane == 0 && m) at = atomicAdd(&s_count, __popc(m));
        at = __shfl_sync(0xffffffffu, at, 0);
        if (in) s_listed[at + __popc(m & ((1u << lane) - 1u))] = (uint16_t)i;
    }
    __syncthreads();
    const int listed = s_count;
    const int nodes = s_nodes;
    const int W = (a.V + 31) / 32, MW = (N + 31) / 32;

    for (int r = blockIdx.z * kWarps + warp; r < a.R; r += gridDim.z * kWarps) {
        const int64_t row = (int64_t)b * a.R + r;
        const char* src = static_cast<const char*>(a.logits) + row * a.V * ES;
        char* dst = static_cast<char*>(a.out) + row * a.V * ES;
        const uint32_t* ok = a.allowed ? a.allowed + row * W : nullptr;
        auto word_ok = [&](int v) { return !ok || ((__ldg(ok + (v >> 5)) >> (v & 31)) & 1u); };

        // the nodes this row follows
        int mine = 0;
        for (int i0 = 0; i0 < nodes; i0 += 32) {
            const int node = i0 + lane < nodes ? s_node[i0 + lane] : N;
            bool see = node < N && (a.tree_mask ? r > 0 : node < r);
            if (see && a.tree_mask)
                see = (__ldg(a.tree_mask + ((int64_t)b * N + r - 1) * MW + (node >> 5)) >> (node & 31)) & 1u;
            const unsigned m = __ballot_sync(0xffffffffu, see);
            if (see) s_list[mine + __popc(m & ((1u << lane) - 1u))] = (uint16_t)(i0 + lane);
            mine += __popc(m);
        }
        __syncwarp();
        auto draft_at = [&](int i) { return (int)s_tok[s_list[i]]; };
        // lane i's drafted token and its element's new value, if it is the token's first in the list
        auto redo = [&](int i, int& v, float& x) {
            const int u = draft_at(i);
            uint32_t w = s_table[u];
            for (int k = 0; k < mine; ++k)
                if (draft_at(k) == u) {
                    if (k < i) return false;
                    ++w;
                }
            v = token(u);
            x = penalised(load_logit<BF16>(src, v), w, pen);
            if (BIAS) x += s_bias[u];
            if (!word_ok(v)) x = neg_inf();
            return true;
        };
        int v_mine = -1;
        float x_mine = 0.0f;
        if (lane < mine && !redo(lane, v_mine, x_mine)) v_mine = -1;
        // (a list longer than a warp, in deep trees whose tokens repeat, comes at the end; in place
        // its logits are still as they were then)

        // units of 32 groups of 16 bytes; where a row starts off a 16-byte boundary a unit has one
        // group less, and its first and last elements are left over
        constexpr int VEC = 16 / ES, UNIT = 32 * VEC, STEP = 4;
        constexpr uint32_t ALL = (1u << VEC) - 1u;
        const int head = to_boundary<BF16>(dst);
        const bool same = to_boundary<BF16>(src) == head;
        auto one = [&](int v) {
            if (!word_ok(v)) store_logit<BF16>(dst, v, neg_inf());
            else if (!in_place) store_logit<BF16>(dst, v, load_logit<BF16>(src, v));
        };
        // The listed tokens, four a step; in place an element is written once, so those that the
        // row drafted are left to the end.  The first step's logits are read before the copy.
        int lu[STEP];
        uint32_t lx[STEP], lw[STEP];  // as loaded: looking at them here would wait for them
        auto get_listed = [&](int i0) {
#pragma unroll
            for (int y = 0; y < STEP; ++y) {
                lu[y] = i0 + 32 * y < listed ? (int)s_listed[i0 + 32 * y] : -1;
                if (in_place)
                    for (int k = 0; k < mine; ++k)
                        if (lu[y] == draft_at(k)) lu[y] = -1;
                lx[y] = lw[y] = 0u;
                if (lu[y] < 0) continue;
                const int v = token(lu[y]);
                lx[y] = BF16 ? (uint32_t)reinterpret_cast<const unsigned short*>(src)[v] : reinterpret_cast<const uint32_t*>(src)[v];
                if (ok) lw[y] = __ldg(ok + (v >> 5));
            }
        };
        auto put_listed = [&]() {
#pragma unroll
            for (int y = 0; y < STEP; ++y) {
                if (lu[y] < 0) continue;
                const int v = token(lu[y]);
                if (ok && !((lw[y] >> (v & 31)) & 1u)) continue;  // -inf already
                float x = penalised(__uint_as_float(BF16 ? lx[y] << 16 : lx[y]), s_table[lu[y]], pen);
                if (BIAS) x += s_bias[lu[y]];
                store_logit<BF16>(dst, v, x);
            }
        };
        get_listed(lane);
        if (!in_place || ok) {
            // Four units a step: the logits of the groups whose mask keeps anything, and the next
            // step's masks, are on their way together.
            uint32_t keep[STEP], next[STEP];
            auto masks = [&](int u0, uint32_t (&k)[STEP]) {
#pragma unroll
                for (int y = 0; y < STEP; ++y) {
                    const int u = u0 + y * UNIT, at = token(u) + head + lane * VEC;
                    k[y] = ALL;
                    if (ok && u < a.slice && at + VEC <= a.V) {
                        uint32_t w = __ldg(ok + (at >> 5)) >> (at & 31);
                        if ((at & 31) + VEC > 32) w |= __ldg(ok + (at >> 5) + 1) << (32 - (at & 31));
                        k[y] = w & ALL;
                    }
                }
            };
            masks(0, keep);
            for (int u0 = 0; u0 < a.slice; u0 += STEP * UNIT) {
                uint4 io[STEP];
                int v[STEP];  // this lane's group, or -1
#pragma unroll
                for (int y = 0; y < STEP; ++y) {
                    const int u = u0 + y * UNIT, first = token(u);
                    v[y] = u < a.slice && same && first + UNIT <= a.V && !(head && lane == 31) ? first + head + lane * VEC : -1;
                    io[y] = make_uint4(0u, 0u, 0u, 0u);
                    if (!in_place && v[y] >= 0 && keep[y]) io[y] = sv::ld_nc_v4(src + (int64_t)v[y] * ES);
                }
                masks(u0 + STEP * UNIT, next);
                if (!same || head || token(u0) + ((STEP * UNIT << a.log_slices) + kBlock) > a.V) {
#pragma unroll 1
                    for (int y = 0; y < STEP; ++y) {
                        const int u = u0 + y * UNIT, first = token(u);
                        if (u >= a.slice || first >= a.V) continue;
                        if (!same || first + UNIT > a.V) {  // other alignments, and the vocabulary's end
                            for (int e = lane; e < UNIT && first + e < a.V; e += 32) one(first + e);
                        } else if (head && lane < VEC) {
                            one(first + (lane < head ? lane : 31 * VEC + lane));
                        }
                    }
                }
#pragma unroll
                for (int y = 0; y < STEP; ++y) {
                    if (v[y] < 0) continue;
                    if (!in_place) {
                        if (ok) io[y] = masked<BF16>(io[y], keep[y]);
                        *reinterpret_cast<uint4*>(dst + (int64_t)v[y] * ES) = io[y];
                    } else if (keep[y] == 0u) {
                        *reinterpret_cast<uint4*>(dst + (int64_t)v[y] * ES) = masked<BF16>(io[y], 0u);
                    } else if (keep[y] != ALL) {
#pragma unroll
                        for (int j = 0; j < VEC; ++j)
                            if (!((keep[y] >> j) & 1u)) store_logit<BF16>(dst, v[y] + j, neg_inf());
                    }
                }
#pragma unroll
                for (int y = 0; y < STEP; ++y) keep[y] = next[y];
            }
            __syncwarp();
        }
        put_listed();
        for (int i0 = lane + 32 * STEP; i0 < listed; i0 += 32 * STEP) {
            get_listed(i0);
            put_listed();
        }
        __syncwarp();
        if (v_mine >= 0) store_logit<BF16>(dst, v_mine, x_mine);
        for (int i0 = 32; i0 < mine; i0 += 32) {
            int v;
            float x;
            if (i0 + lane < mine && redo(i0 + lane, v, x)) store_logit<BF16>(dst, v, x);
        }
        __syncwarp();  // the list is rewritten for the next row
    }
}

int device_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return sms;
}

// Slices: the fewest (a power of two) that give two CTAs per SM with at most kMaxSlice tokens
// each (shared memory); every slice's CTA reads the whole history, so no more than one per
// eight blocks.
int pick_log_slices(int B, int V, int sms) {
    const int blocks = (V + kBlock - 1) / kBlock;
    int k = 0;
    while ((((int64_t)blocks + (1 << k) - 1) >> k) * kBlock > kMaxSlice ||
           ((long long)B << k < 2LL * sms && (8 << (k + 1)) <= blocks))
        ++k;
    return k;
}

// CTAs that share the rows of a slice, each with tables of its own: where the slices do not fill
// the four places per SM, down to one round of rows (one per warp) each.  61 rows of 128256 with
// penalties, biases, a grammar and 6000 tokens of history, with one and with as many CTAs: 8 trees
// 148 and 92 us, 4 trees 138 and 56 us, one 107 and 28 us; 2 x 129 rows of 32000 263 and 35 us.
int pick_row_groups(int B, int R, int log_slices, int sms) {
    const int64_t have = (int64_t)B << log_slices, fit = 4LL * sms / have, rounds = (R + kWarps - 1) / kWarps;
    return (int)(fit < 1 ? 1 : fit < rounds ? fit : rounds);
}

template <bool BF16, bool BIAS>
cudaError_t launch_adjust(const AdjustArgs& a, int B, int row_groups, cudaStream_t stream) {
    static sv::KernelLaunchCache cache;
    auto kern = adjust_logits_kernel<BF16, BIAS>;
    int max_dyn = 0;
    const cudaError_t e = cache.setup((const void*)kern, &max_dyn);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)a.slice * (BIAS ? 10 : 6) + (size_t)(a.R - 1) * (2 + kWarps) * sizeof(uint16_t);
    if (smem > (size_t)max_dyn) return cudaErrorInvalidValue;
    return sv::launch_serial(kern, dim3(1u << a.log_slices, (unsigned)B, (unsigned)row_groups), dim3(kThreads), smem, stream, a);
}

}  // namespace

extern "C" sv_status spec_adjust_logits(const void* logits, sv_dtype dt, const int32_t* history,
                                        const int32_t* history_len, const int32_t* prompt_len, int H,
                                        const int32_t* draft_tokens, const uint32_t* tree_mask,
                                        const float* repetition, const float* presence, const float* frequency,
                                        const int32_t* bias_tokens, const float* bias_values, int M,
                                        const uint32_t* allowed, int B, int R, int V, void* out, void* stream) {
    if (dt != SV_F32 && dt != SV_BF16) return SV_ERR_INVALID_ARG;
    if (B < 0 || B > kMaxB || R < 1 || R > kMaxRows || V < 1 || V > kMaxV || H < 0 || H == INT32_MAX || M < 0 ||
        M > 65535)
        return SV_ERR_INVALID_ARG;
    if (B == 0) return SV_OK;
    const uintptr_t es = dt == SV_BF16 ? 2 : 4;
    if (!logits || !out || ((uintptr_t)logits | (uintptr_t)out) % es) return SV_ERR_INVALID_ARG;
    if (H > 0 && history && !history_len) return SV_ERR_INVALID_ARG;
    if (M > 0 && (bias_tokens == nullptr) != (bias_values == nullptr)) return SV_ERR_INVALID_ARG;
    const uintptr_t lo = (uintptr_t)logits, ou = (uintptr_t)out, bytes = (uintptr_t)B * R * V * es;
    if (lo != ou && lo < ou + bytes && ou < lo + bytes) return SV_ERR_INVALID_ARG;  // partial overlap
    const int sms = device_sms();
    if (!sms) return sv::launch_status(cudaErrorInvalidDevice);
    AdjustArgs a{logits, out, H > 0 ? history : nullptr, history_len, prompt_len, R > 1 ? draft_tokens : nullptr,
                 R > 1 && draft_tokens ? tree_mask : nullptr, repetition, presence, frequency, bias_tokens, bias_values,
                 allowed, H, M, R, V, 0, 0};
    a.log_slices = pick_log_slices(B, V, sms);
    const int blocks = (V + kBlock - 1) / kBlock;
    a.slice = ((blocks + (1 << a.log_slices) - 1) >> a.log_slices) * kBlock;
    const int groups = pick_row_groups(B, R, a.log_slices, sms);
    const bool bias = M > 0 && bias_tokens;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (dt == SV_BF16) e = bias ? launch_adjust<true, true>(a, B, groups, s) : launch_adjust<true, false>(a, B, groups, s);
    else e = bias ? launch_adjust<false, true>(a, B, groups, s) : launch_adjust<false, false>(a, B, groups, s);
    return sv::launch_status(e);
}
