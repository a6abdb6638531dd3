// sv_rotary.cu -- rotary positions of queries and keys, alone or on the keys' way into a
// paged cache (include/spec_rotary.h).
//
// Every element is read and written once, so memory bounds it; sines and cosines are one per
// token and pair, shared by all heads, and a block computes them once into shared memory for
// its tokens.  A row of one token and head is held by a group of lanes, eight elements each,
// as in the cache's other kernels (sv_rows.cuh); a pair's other element is in the same lane
// (neighbours paired), or num_freq elements away, read with a second 16-byte load that the
// first level cache answers: another lane of the row has the same bytes in flight.
//
// Angles: position * freq in fp32 would be off by whole radians at 10^7 positions.  Counted in
// turns only the fraction matters: f = freq / 2 pi as hi + lo (fp32 each, from its 64 bits), the
// position as a multiple of 4096 plus a rest (both exact), products as hi * p with the part
// that fma leaves (exact), whole turns dropped exactly, and sincospi of the rest: fp32
// throughout, where 64-bit products would take the SM's few 64-bit lanes.
#include <cstdint>

#include "spec_rotary.h"
#include "sv_internal.h"
#include "sv_paged.cuh"
#include "sv_rows.cuh"

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTokens = 8;  // of a block
constexpr int kMaxFreq = 128;
constexpr int kMaxB = 65535;
constexpr int kMaxN = 1 << 20;

enum { DENSE, CACHE_BF16, CACHE_E4M3 };

struct RotaryArgs {
    sv::PagedCache c;
    const void* src[3];  // queries, keys, values
    void* dst[2];        // queries, keys (DENSE)
    int64_t ss[3][3];    // element strides of the sources (batch, token, head)
    int64_t ds[2][3];    // and of the destinations
    int end[3];          // rows of a token: [0, end[0]) queries, then keys, then values
    const double* freq;
    const int32_t* depth;
    const int32_t* base;
    const int32_t* new_len;
    float amplitude;
    int R, interleaved, inverse;
    int B, N, D;
    int tile;   // tokens of a block: 1, 2, 4 or 8
    int chunk;  // rows of a token that a block does
};

// Position of token i of row b; false where the token is not written.
template <int MODE>
__device__ __forceinline__ bool token_position(const RotaryArgs& a, int b, int i, int64_t& pos, int& first) {
    int n;
    if (MODE == DENSE) {
        first = __ldg(a.base + b);
        n = a.new_len ? __ldg(a.new_len + b) : a.N;
        if (first < 0 || first > sv::PAGED_MAX_POS || n < 0 || n > a.N) return false;
    } else if (!sv::paged_row(a.c, a.base, a.new_len, b, a.N, first, n)) {
        return false;
    }
    if (i >= n) return false;
    pos = first;
    if (!a.depth) pos += i;
    else if (i > 0) pos += __ldg(a.depth + (int64_t)b * (a.N - 1) + (i - 1));
    return true;
}

// Cosine and sine of pos * (fh + fl) turns.
__device__ __forceinline__ float2 turn(int64_t pos, float fh, float fl) {
    const float rest = (float)(int)(pos & 4095), big = (float)(pos - (pos & 4095));
    float x = big * fh, y = rest * fh;
    const float small = fmaf(big, fl, rest * fl) + fmaf(big, fh, -x) + fmaf(rest, fh, -y);
    x -= rintf(x);
    y -= rintf(y);
    const float z = x + y, t = z - x;
    const float left = (x - (z - t)) + (y - t);  // what the sum lost
    const float r = (z - rintf(z)) + (left + small);
    float s, c;
    sincospif(2.0f * r, &s, &c);
    return make_float2(c, s);
}

template <typename T, bool AL>
__device__ __forceinline__ void read8(const T* row, int e0, int dim, float x[8]) {
    if (AL) {
        uint4 w[sizeof(T) / 2];
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k)
            w[k] = e0 < dim ? *reinterpret_cast<const uint4*>(row + e0 + 4 * k) : make_uint4(0u, 0u, 0u, 0u);
        if (sizeof(T) == 2) {
            x[0] = sv::bf16_lo(w[0].x); x[1] = sv::bf16_hi(w[0].x); x[2] = sv::bf16_lo(w[0].y); x[3] = sv::bf16_hi(w[0].y);
            x[4] = sv::bf16_lo(w[0].z); x[5] = sv::bf16_hi(w[0].z); x[6] = sv::bf16_lo(w[0].w); x[7] = sv::bf16_hi(w[0].w);
        } else {
            const uint4 b = w[sizeof(T) == 4 ? 1 : 0];
            x[0] = __uint_as_float(w[0].x); x[1] = __uint_as_float(w[0].y);
            x[2] = __uint_as_float(w[0].z); x[3] = __uint_as_float(w[0].w);
            x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y);
            x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[k] = 0.0f;
            if (e0 + k < dim)
                x[k] = sizeof(T) == 2 ? __uint_as_float((uint32_t)reinterpret_cast<const unsigned short*>(row)[e0 + k] << 16)
                                      : reinterpret_cast<const float*>(row)[e0 + k];
        }
    }
}

template <typename T>
__device__ __forceinline__ float read1(const T* row, int e) {
    return sizeof(T) == 2 ? __uint_as_float((uint32_t)reinterpret_cast<const unsigned short*>(row)[e] << 16)
                          : reinterpret_cast<const float*>(row)[e];
}

// grid: x over tiles of tokens, y over chunks of a token's rows.  LPR lanes hold a row.
template <typename T, int LPR, int MODE, bool AL, int ROWS>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
    extern __shared__ float2 s_turn[];  // [tile][R]
    __shared__ float2 s_freq[kMaxFreq];
    __shared__ int64_t s_pos[kMaxTokens];
    __shared__ int s_first[kMaxTokens];  // the row's base; -1: token not written
    constexpr int G = 32 / LPR;
    sv::pdl_trigger();
    sv::pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned total = (unsigned)a.B * (unsigned)a.N;
    if (tid < a.tile) {
        const unsigned x = blockIdx.x * (unsigned)a.tile + tid;
        int first = -1;
        int64_t pos = 0;
        if (x < total && !token_position<MODE>(a, (int)(x / a.N), (int)(x % a.N), pos, first)) first = -1;
        s_pos[tid] = pos;
        s_first[tid] = first;
    }
    for (int j = tid; j < a.R; j += kThreads) {
        const double f = a.freq[j] * 0.15915494309189533577;
        const float hi = (float)f;
        s_freq[j] = make_float2(hi, (float)(f - (double)hi));
    }
    __syncthreads();
    for (int x = tid; x < a.tile * a.R; x += kThreads) {
        const int t = x / a.R;
        const float2 f = s_freq[x - t * a.R], cs = turn(s_pos[t], f.x, f.y);
        s_turn[x] = make_float2(cs.x * a.amplitude, a.inverse ? -(cs.y * a.amplitude) : cs.y * a.amplitude);
    }
    __syncthreads();
    const int each = kWarps / a.tile;  // warps of a token
    const int t = warp / each;
    const int first = s_first[t];
    if (first < 0) return;
    const unsigned x = blockIdx.x * (unsigned)a.tile + t;
    const int b = (int)(x / a.N), i = (int)(x % a.N);
    int page = -1, slot = 0;
    if (MODE != DENSE) page = sv::paged_place(a.c, b, first + i, slot);

    // This lane's elements: own and partner's factors (0 partner: copied).
    const int e0 = 8 * (lane % LPR), R = a.R, turned = 2 * R;
    float c[8], s[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int e = e0 + k;
        c[k] = 1.0f;
        s[k] = 0.0f;
        if (e < turned) {
            const bool second = a.interleaved ? k & 1 : e >= R;
            const float2 cs = s_turn[t * R + (a.interleaved ? e >> 1 : second ? e - R : e)];
            c[k] = cs.x;
            s[k] = second ? cs.y : -cs.y;
        }
    }
    const bool apart = AL && !a.interleaved && R % 8 == 0;  // the partners are eight elements elsewhere
    const int other = e0 < R ? e0 + R : e0 - R;

    const int r0 = blockIdx.y * a.chunk, r1 = min(a.end[2], r0 + a.chunk);
    for (int r = r0 + (warp - t * each) * (G * ROWS); r < r1; r += each * G * ROWS) {
        float v[ROWS][8], p[ROWS][8];
        int kind[ROWS], head[ROWS];
#pragma unroll
        for (int z = 0; z < ROWS; ++z) {
            const int row = r + z * G + lane / LPR;
            kind[z] = row >= r1 ? -1 : row < a.end[0] ? 0 : row < a.end[1] ? 1 : 2;
            head[z] = kind[z] <= 0 ? row : row - a.end[kind[z] - 1];
            const int kz = max(kind[z], 0);
            const T* from = static_cast<const T*>(a.src[kz]) +
                            (kind[z] >= 0 ? b * a.ss[kz][0] + i * a.ss[kz][1] + head[z] * a.ss[kz][2] : 0);
            const int dim = kind[z] >= 0 ? a.D : 0;
            read8<T, AL>(from, e0, dim, v[z]);
            if (apart) {
                read8<T, AL>(from, other, e0 < turned && kind[z] != 2 ? dim : 0, p[z]);
            } else if (a.interleaved) {
#pragma unroll
                for (int k = 0; k < 8; ++k) p[z][k] = v[z][k ^ 1];
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int e = e0 + k;
                    p[z][k] = e < turned && e < dim ? read1(from, e < R ? e + R : e - R) : 0.0f;
                }
            }
        }
        __syncwarp();  // in place: a row's elements are read before any is written
#pragma unroll
        for (int z = 0; z < ROWS; ++z) {
            if (kind[z] != 2) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (e0 + k < turned) v[z][k] = fmaf(v[z][k], c[k], p[z][k] * s[k]);
            }
            const bool dense = MODE == DENSE ? kind[z] >= 0 : kind[z] == 0;
            if (dense) {
                const int kz = MODE == DENSE ? kind[z] : 0;
                T* to = static_cast<T*>(a.dst[kz]) + b * a.ds[kz][0] + i * a.ds[kz][1] + head[z] * a.ds[kz][2];
                sv::store_row8<T, AL>(to, e0, a.D, v[z]);
            }
            if (MODE != DENSE && __any_sync(0xffffffffu, kind[z] > 0)) {
                const bool live = kind[z] > 0 && page >= 0;
                const int h = kind[z] > 0 ? head[z] : 0, at = live ? page : 0;
                const int64_t off = at * a.c.page_stride + h * a.c.head_stride + slot * a.c.row_stride;
                float* scales = kind[z] == 2 ? a.c.v_scale : a.c.k_scale;
                sv::Eight<float, AL> f;
                if (AL) {
                    f.w[0] = make_uint4(__float_as_uint(v[z][0]), __float_as_uint(v[z][1]), __float_as_uint(v[z][2]), __float_as_uint(v[z][3]));
                    f.w[AL ? 1 : 0] = make_uint4(__float_as_uint(v[z][4]), __float_as_uint(v[z][5]), __float_as_uint(v[z][6]), __float_as_uint(v[z][7]));
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) f.f[AL ? 0 : k] = v[z][k];
                }
                sv::store_cache_row<float, LPR, MODE == CACHE_E4M3, AL>(
                    (kind[z] == 2 ? a.c.v : a.c.k) + off, scales + ((int64_t)at * a.c.heads + h) * a.c.page_size + slot, e0, a.D, live, f);
            }
        }
    }
}

template <typename T, int LPR, int MODE, bool AL>
cudaError_t launch_lpr(RotaryArgs& a, cudaStream_t stream) {
    const int64_t tokens = (int64_t)a.B * a.N;
    const int rows = a.end[2];
    int sms = 152;
    // Tokens of a block: as many as leave six blocks per SM, since they share the frequencies;
    // a few tokens are spread over blocks by their rows instead, one pass of a block's warps each.
    a.tile = 1;
    while (a.tile < kMaxTokens && tokens / (2 * a.tile) >= 6 * sms) a.tile *= 2;
    constexpr int pass = kWarps * (32 / LPR);
    a.chunk = tokens >= 2 * sms ? rows : pass;
    if (a.chunk < 1) a.chunk = 1;
    const dim3 grid((unsigned)((tokens + a.tile - 1) / a.tile), (unsigned)((rows + a.chunk - 1) / a.chunk));
    const size_t smem = (size_t)a.tile * a.R * sizeof(float2);
    if (tokens >= 2 * sms) return sv::launch_serial(rotary_kernel<T, LPR, MODE, AL, AL ? 2 : 1>, grid, dim3(kThreads), smem, stream, a);
    return sv::launch_serial(rotary_kernel<T, LPR, MODE, AL, 1>, grid, dim3(kThreads), smem, stream, a);
}

template <typename T, int MODE>
cudaError_t launch_mode(RotaryArgs& a, bool al, cudaStream_t stream) {
    if (!al) return launch_lpr<T, 32, MODE, false>(a, stream);
    if (a.D <= 64) return launch_lpr<T, 8, MODE, true>(a, stream);
    if (a.D <= 128) return launch_lpr<T, 16, MODE, true>(a, stream);
    return launch_lpr<T, 32, MODE, true>(a, stream);
}

cudaError_t launch(RotaryArgs& a, int mode, int dt, bool al, cudaStream_t s) {
    if (dt == SV_BF16) {
        if (mode == DENSE) return launch_mode<uint16_t, DENSE>(a, al, s);
        return mode == CACHE_BF16 ? launch_mode<uint16_t, CACHE_BF16>(a, al, s) : launch_mode<uint16_t, CACHE_E4M3>(a, al, s);
    }
    if (mode == DENSE) return launch_mode<float, DENSE>(a, al, s);
    return mode == CACHE_BF16 ? launch_mode<float, CACHE_BF16>(a, al, s) : launch_mode<float, CACHE_E4M3>(a, al, s);
}

// The parts of the arguments that both entries share; false: invalid.
bool common_args(RotaryArgs& a, const sv_rotary* rotary, int dt, int B, int N, int head_dim) {
    if (dt != SV_F32 && dt != SV_BF16) return false;
    if (B < 0 || B > kMaxB || N < 0 || N > kMaxN || (int64_t)B * N >= ((int64_t)1 << 31) || head_dim < 1 || head_dim > sv::PAGED_MAX_DIM) return false;
    if (!rotary || rotary->num_freq < 0 || rotary->num_freq > kMaxFreq || 2 * rotary->num_freq > head_dim) return false;
    if (rotary->num_freq && !rotary->freq) return false;
    if (!(rotary->amplitude - rotary->amplitude == 0.0f)) return false;  // NaN or infinite
    a.freq = rotary->freq;
    a.depth = N > 1 ? rotary->tree_depth : nullptr;
    a.amplitude = rotary->amplitude;
    a.R = rotary->num_freq;
    a.interleaved = rotary->interleaved != 0;
    a.inverse = rotary->inverse != 0;
    a.B = B;
    a.N = N;
    a.D = head_dim;
    return true;
}

// Strides of one array into `to`; whether eight elements are 16-byte accesses everywhere.
bool take_strides(int64_t to[3], const int64_t* from, const void* p, int es) {
    for (int k = 0; k < 3; ++k) to[k] = from[k];
    return (uintptr_t)p % 16 == 0 && (from[0] * es | from[1] * es | from[2] * es) % 16 == 0;
}

}  // namespace

extern "C" {

sv_status spec_rotary(const void* q, const int64_t* q_stride, int num_q_heads, const void* k, const int64_t* k_stride,
                      int num_k_heads, sv_dtype dt, const sv_rotary* rotary, const int32_t* base,
                      const int32_t* new_len, int B, int N, int head_dim, void* out_q, const int64_t* out_q_stride,
                      void* out_k, const int64_t* out_k_stride, void* stream) {
    RotaryArgs a{};
    if (!common_args(a, rotary, dt, B, N, head_dim) || num_q_heads < 1 || num_q_heads > 65536 || num_k_heads < 0 ||
        num_k_heads > 65536)
        return SV_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return SV_OK;
    if (!q || !q_stride || !out_q || !out_q_stride || !base) return SV_ERR_INVALID_ARG;
    if (num_k_heads && (!k || !k_stride || !out_k || !out_k_stride)) return SV_ERR_INVALID_ARG;
    const int es = dt == SV_BF16 ? 2 : 4;
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)out_q | (uintptr_t)out_k) % es) return SV_ERR_INVALID_ARG;
    bool al = head_dim % 8 == 0;
    a.src[0] = q;
    a.dst[0] = out_q;
    al &= take_strides(a.ss[0], q_stride, q, es);
    al &= take_strides(a.ds[0], out_q_stride, out_q, es);
    a.end[0] = num_q_heads;
    a.end[1] = a.end[2] = num_q_heads + num_k_heads;
    if (num_k_heads) {
        a.src[1] = k;
        a.dst[1] = out_k;
        al &= take_strides(a.ss[1], k_stride, k, es);
        al &= take_strides(a.ds[1], out_k_stride, out_k, es);
    }
    a.base = base;
    a.new_len = new_len;
    return sv::launch_status(launch(a, DENSE, dt, al, (cudaStream_t)stream));
}

sv_status spec_rotary_append(const void* q, const int64_t* q_stride, int num_q_heads, const void* key,
                             const void* value, const int64_t* kv_stride, sv_dtype dt, const sv_rotary* rotary,
                             const sv_paged_cache* cache, const int32_t* base, const int32_t* new_len, int B, int N,
                             void* out_q, const int64_t* out_q_stride, void* stream) {
    RotaryArgs a{};
    if (!sv::paged_cache_args(cache, a.c) || !common_args(a, rotary, dt, B, N, cache->head_dim) || num_q_heads < 0 ||
        num_q_heads > 65536)
        return SV_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return SV_OK;
    if (!key || !value || !kv_stride || !base || !cache->page_table) return SV_ERR_INVALID_ARG;
    if (num_q_heads && (!q || !q_stride || !out_q || !out_q_stride)) return SV_ERR_INVALID_ARG;
    const int es = dt == SV_BF16 ? 2 : 4;
    if (((uintptr_t)q | (uintptr_t)key | (uintptr_t)value | (uintptr_t)out_q) % es) return SV_ERR_INVALID_ARG;
    const int64_t cs = cache->dtype == SV_CACHE_BF16 ? 16 : 8;
    bool al = cache->head_dim % 8 == 0 && (cache->page_stride | cache->head_stride | cache->row_stride) % cs == 0 &&
              ((uintptr_t)cache->k_pages | (uintptr_t)cache->v_pages) % cs == 0;
    if (num_q_heads) {
        a.src[0] = q;
        a.dst[0] = out_q;
        al &= take_strides(a.ss[0], q_stride, q, es);
        al &= take_strides(a.ds[0], out_q_stride, out_q, es);
    }
    a.src[1] = key;
    a.src[2] = value;
    al &= take_strides(a.ss[1], kv_stride, key, es);
    al &= take_strides(a.ss[2], kv_stride, value, es);
    a.end[0] = num_q_heads;
    a.end[1] = num_q_heads + cache->num_heads;
    a.end[2] = a.end[1] + cache->num_heads;
    a.base = base;
    a.new_len = new_len;
    return sv::launch_status(launch(a, cache->dtype == SV_CACHE_BF16 ? CACHE_BF16 : CACHE_E4M3, dt, al, (cudaStream_t)stream));
}

}  // extern "C"
