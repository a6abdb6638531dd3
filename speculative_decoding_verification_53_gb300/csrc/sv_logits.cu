// sv_logits.cu -- penalties, biases and grammar masks on the logits of every row of a
// verify call (include/spec_logits.h).
//
// A CTA takes one batch row and a slice of the vocabulary.  From the row's token lists it
// builds a table of its slice in shared memory, one word per token (the count in the
// output so far, and a flag for "in the prompt") and, where biases are given, the bias;
// the table serves all R rows.  Then each warp takes rows of the slice in turn:
//   out of place: it streams the row's part, 16 bytes per lane, and looks the table up;
//   in place: it visits only the table's entries, and writes -inf where the grammar says so.
// A row's drafted tokens (the prefix of a chain, the ancestors in a tree) are few of the
// slice's tokens: the warp lists them, and rewrites those elements after the stream from
// the logits it kept aside.  So nothing in shared memory changes while rows are at work,
// and no result depends on the order of atomics (counts are integers; of two biases of one
// token the later entry holds).
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
constexpr int kMaxSlice = 16384;
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
    int H, M, R, V, slice, slices;
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

// The 16 bytes of a group as fp32, back, and with -inf where `keep` has a 0.
template <bool BF16>
__device__ __forceinline__ void unpack(uint4 g, float* x) {
    if (BF16) {
        x[0] = sv::bf16_lo(g.x); x[1] = sv::bf16_hi(g.x); x[2] = sv::bf16_lo(g.y); x[3] = sv::bf16_hi(g.y);
        x[4] = sv::bf16_lo(g.z); x[5] = sv::bf16_hi(g.z); x[6] = sv::bf16_lo(g.w); x[7] = sv::bf16_hi(g.w);
    } else {
        x[0] = __uint_as_float(g.x); x[1] = __uint_as_float(g.y);
        x[2] = __uint_as_float(g.z); x[3] = __uint_as_float(g.w);
    }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack(const float* x) {
    if (BF16) return make_uint4(sv::bf16x2(x[0], x[1]), sv::bf16x2(x[2], x[3]), sv::bf16x2(x[4], x[5]), sv::bf16x2(x[6], x[7]));
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
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
__global__ void __launch_bounds__(kThreads) adjust_logits_kernel(const __grid_constant__ AdjustArgs a) {
    pdl_trigger();
    pdl_wait();
    extern __shared__ __align__(16) uint32_t s_table[];  // [slice] words, [slice] biases, per-warp lists
    const int b = blockIdx.y, v0 = blockIdx.x * a.slice;
    const int n = a.V - v0 < a.slice ? a.V - v0 : a.slice;
    float* s_bias = reinterpret_cast<float*>(s_table + a.slice);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int N = a.R - 1;
    const bool in_place = a.out == a.logits;
    constexpr int ES = BF16 ? 2 : 4;

    __shared__ int s_nodes;  // drafted tokens of this slice
    for (int i = tid; i < a.slice * (BIAS ? 2 : 1); i += kThreads) s_table[i] = 0u;
    if (tid == 0) s_nodes = 0;
    __syncthreads();
    uint16_t* s_node = reinterpret_cast<uint16_t*>(s_table + a.slice * (BIAS ? 2 : 1));  // [N] node, then lists
    uint16_t* s_list = s_node + N + warp * N;                                            // this warp's
    int len = a.history ? __ldg(a.history_len + b) : 0;
    len = len < 0 ? 0 : len > a.H ? a.H : len;
    const int prompt = a.prompt_len ? __ldg(a.prompt_len + b) : 0;
    const int32_t* hist = a.history + (int64_t)b * a.H;
#pragma unroll 4
    for (int i = tid; i < len; i += kThreads) {
        const unsigned v = (unsigned)__ldg(hist + i) - (unsigned)v0;
        if (v < (unsigned)n) {
            if (i < prompt) atomicOr(s_table + v, kPrompt);
            else atomicAdd(s_table + v, 1u);
        }
    }
    if (BIAS) {
        // the last entry of a token wins: its number + 1 is the largest
        uint32_t* at = reinterpret_cast<uint32_t*>(s_bias);
        const int32_t* bt = a.bias_tokens + (int64_t)b * a.M;
        for (int i = tid; i < a.M; i += kThreads) {
            const int t = __ldg(bt + i);
            const unsigned v = (unsigned)t - (unsigned)v0;
            if (t >= 0 && v < (unsigned)n) atomicMax(at + v, (uint32_t)i + 1u);
        }
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            const uint32_t m = at[i];
            s_bias[i] = m ? __ldg(a.bias_values + (int64_t)b * a.M + m - 1) : 0.0f;
        }
    }
    // drafted tokens of this slice, in node order (one warp, so that the order is fixed)
    if (a.drafts && warp == 0) {
        int have = 0;
        for (int i0 = 0; i0 < N; i0 += 32) {
            const int i = i0 + lane;
            const bool in = i < N && (unsigned)__ldg(a.drafts + (int64_t)b * N + i) - (unsigned)v0 < (unsigned)n;
            const unsigned m = __ballot_sync(0xffffffffu, in);
            if (in) s_node[have + __popc(m & ((1u << lane) - 1u))] = (uint16_t)i;
            have += __popc(m);
        }
        if (lane == 0) s_nodes = have;
    }
    __syncthreads();
    const int nodes = s_nodes;
    Penalty pen;
    pen.rep = a.repetition ? __ldg(a.repetition + b) : 1.0f;
    pen.pres = a.presence ? __ldg(a.presence + b) : 0.0f;
    pen.freq = a.frequency ? __ldg(a.frequency + b) : 0.0f;
    const int W = (a.V + 31) / 32, MW = (N + 31) / 32;

    for (int r = warp; r < a.R; r += kWarps) {
        const int64_t row = (int64_t)b * a.R + r;
        const char* src = static_cast<const char*>(a.logits) + (row * a.V + v0) * ES;
        char* dst = static_cast<char*>(a.out) + (row * a.V + v0) * ES;
        const uint32_t* ok = a.allowed ? a.allowed + row * W : nullptr;
        auto word_ok = [&](int v) { return !ok || ((__ldg(ok + ((v0 + v) >> 5)) >> ((v0 + v) & 31)) & 1u); };

        // the nodes this row follows
        int mine = 0;
        for (int i0 = 0; i0 < nodes; i0 += 32) {
            const int node = i0 + lane < nodes ? s_node[i0 + lane] : N;
            bool see = node < N && (a.tree_mask ? r > 0 : node < r);
            if (see && a.tree_mask)
                see = (__ldg(a.tree_mask + ((int64_t)b * N + r - 1) * MW + (node >> 5)) >> (node & 31)) & 1u;
            const unsigned m = __ballot_sync(0xffffffffu, see);
            if (see) s_list[mine + __popc(m & ((1u << lane) - 1u))] = (uint16_t)node;
            mine += __popc(m);
        }
        __syncwarp();
        auto draft_at = [&](int i) { return __ldg(a.drafts + (int64_t)b * N + s_list[i]) - v0; };
        // lane i's drafted token: its element's new value, if it is the token's first in the list
        auto redo = [&](int i, int& v, float& x) {
            v = draft_at(i);
            uint32_t w = s_table[v];
            for (int k = 0; k < mine; ++k)
                if (draft_at(k) == v) {
                    if (k < i) return false;
                    ++w;
                }
            x = penalised(load_logit<BF16>(src, v), w, pen);
            if (BIAS) x += s_bias[v];
            if (!word_ok(v)) x = neg_inf();
            return true;
        };
        int v_mine = -1;
        float x_mine = 0.0f;
        if (lane < mine && !redo(lane, v_mine, x_mine)) v_mine = -1;
        // lists longer than a warp (deep trees whose tokens repeat): kept out of the stream
        // below by being in the list; in place their logits are still unread then

        if (!in_place) {
            constexpr int VEC = 16 / ES;
            const int head0 = to_boundary<BF16>(src);
            const bool same = to_boundary<BF16>(dst) == head0;
            const int head = same ? (head0 < n ? head0 : n) : n;  // element by element up to here
            auto one = [&](int v) {
                float x = penalised(load_logit<BF16>(src, v), s_table[v], pen);
                if (BIAS) x += s_bias[v];
                if (!word_ok(v)) x = neg_inf();
                store_logit<BF16>(dst, v, x);
            };
            for (int v = lane; v < head; v += 32) one(v);
            const int groups = (n - head) / VEC;
            const bool wide = (head & 3) == 0;  // the table's words are read 16 bytes at a time
#pragma unroll 4
            for (int g = lane; g < groups; g += 32) {
                const int v = head + g * VEC;
                uint4 io = sv::ld_nc_v4(src + (int64_t)v * ES);
                uint32_t w[VEC], any = 0u;
                float bias[VEC];
                if (wide) {
#pragma unroll
                    for (int j = 0; j < VEC; j += 4) *reinterpret_cast<uint4*>(w + j) = *reinterpret_cast<const uint4*>(s_table + v + j);
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) w[j] = s_table[v + j];
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) any |= w[j];
                if (BIAS) {
                    if (wide) {
#pragma unroll
                        for (int j = 0; j < VEC; j += 4) *reinterpret_cast<float4*>(bias + j) = *reinterpret_cast<const float4*>(s_bias + v + j);
                    } else {
#pragma unroll
                        for (int j = 0; j < VEC; ++j) bias[j] = s_bias[v + j];
                    }
#pragma unroll
                    for (int j = 0; j < VEC; ++j) any |= __float_as_uint(bias[j]);
                }
                if (any) {  // few groups hold a token of the lists
                    float x[VEC];
                    unpack<BF16>(io, x);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        x[j] = penalised(x[j], w[j], pen);
                        if (BIAS) x[j] += bias[j];
                    }
                    io = pack<BF16>(x);
                }
                if (ok) {
                    const int bit = v0 + v;
                    uint32_t keep = __ldg(ok + (bit >> 5)) >> (bit & 31);
                    if ((bit & 31) + VEC > 32) keep |= __ldg(ok + (bit >> 5) + 1) << (32 - (bit & 31));
                    io = masked<BF16>(io, keep);
                }
                *reinterpret_cast<uint4*>(dst + (int64_t)v * ES) = io;
            }
            for (int v = head + groups * VEC + lane; v < n; v += 32) one(v);
            __syncwarp();
            if (v_mine >= 0) store_logit<BF16>(dst, v_mine, x_mine);
            for (int i0 = 32; i0 < mine; i0 += 32) {
                int v;
                float x;
                if (i0 + lane < mine && redo(i0 + lane, v, x)) store_logit<BF16>(dst, v, x);
            }
        } else {
            // Entries of the table, then the row's drafted tokens: an element is written once,
            // by the drafted token where there is one.
            for (int v = lane; v < n; v += 32) {
                const bool good = word_ok(v);
                const uint32_t w = s_table[v];
                const bool change = !good || w != 0u || (BIAS && s_bias[v] != 0.0f);
                if (!change) continue;
                bool drafted = false;
                for (int k = 0; k < mine; ++k) drafted |= draft_at(k) == v;
                if (drafted) continue;
                float x = neg_inf();
                if (good) {
                    x = penalised(load_logit<BF16>(dst, v), w, pen);
                    if (BIAS) x += s_bias[v];
                }
                store_logit<BF16>(dst, v, x);
            }
            if (v_mine >= 0) store_logit<BF16>(dst, v_mine, x_mine);
            for (int i0 = 32; i0 < mine; i0 += 32) {
                int v;
                float x;
                if (i0 + lane < mine && redo(i0 + lane, v, x)) store_logit<BF16>(dst, v, x);
            }
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

// Tokens per slice: the largest power of two that still gives two CTAs per SM, 2048 at
// least (a slice's CTA reads the whole history) and 16384 at most (shared memory).
int pick_slice(int B, int V, int sms) {
    int s = kMaxSlice;
    while (s > 2048 && (long long)B * ((V + s - 1) / s) < 2LL * sms) s >>= 1;
    return s;
}

template <bool BF16, bool BIAS>
cudaError_t launch_adjust(const AdjustArgs& a, int B, cudaStream_t stream) {
    static sv::KernelLaunchCache cache;
    auto kern = adjust_logits_kernel<BF16, BIAS>;
    int max_dyn = 0;
    const cudaError_t e = cache.setup((const void*)kern, &max_dyn);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)a.slice * (BIAS ? 8 : 4) + (size_t)(a.R - 1) * (1 + kWarps) * sizeof(uint16_t);
    if (smem > (size_t)max_dyn) return cudaErrorInvalidValue;
    return sv::launch_serial(kern, dim3((unsigned)a.slices, (unsigned)B), dim3(kThreads), smem, stream, a);
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
    a.slice = pick_slice(B, V, sms);
    a.slices = (V + a.slice - 1) / a.slice;
    const bool bias = M > 0 && bias_tokens;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (dt == SV_BF16) e = bias ? launch_adjust<true, true>(a, B, s) : launch_adjust<true, false>(a, B, s);
    else e = bias ? launch_adjust<false, true>(a, B, s) : launch_adjust<false, false>(a, B, s);
    return sv::launch_status(e);
}
