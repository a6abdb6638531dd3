// sv_rotary.cu -- rotary positions of queries and keys, alone or on the keys' way into a
// paged cache (include/spec_rotary.h).
//
// Every element is read and written once, so memory bounds it; sines and cosines are one per
// token and pair, shared by all heads, and a block computes them once into shared memory for
// its tokens.  A row of one token and head is held by a group of lanes, eight elements each,
// as in the cache's other kernels (sv_rows.cuh); a pair's other element is in the same lane
// (neighbours paired), in another one (num_freq a multiple of 8: by shuffles), or anywhere in the
// row, which lies in shared memory.  Rows in flight go through a ring there, since registers hold too
// few (4 x 6001 tokens, 32 + 8 heads of 128, bf16, a quarter of them in pairs: with two rows ahead in registers 6 us
// more, with none 43).  A warp decides on the kind of a group of rows as one (decided per row: 23 us more).
//
// With the bytes in flight, instructions bound it.  160 a group of rows, most of them for 64-bit addresses and for
// factors picked one by one, took 87 us in those 4 x 6001 tokens; factors read as vectors from planes of cosines
// and sines 82; pointers that move on by their kind's stride, found anew only for another kind, 76 (5.9 TB/s).
// fp32 198 us (5.0 TB/s), num_freq 10 104; 16 x 2048 tokens on their way into a cache of bf16 83 (floor 75), of e4m3 92.
// Tokens of few rows pay for their sines, places and idle lanes, so a warp takes four of them at once (rotary_few_kernel):
// 64 x 2000 tokens of 4 + 1 heads of 64 43 us (80 without; their bytes' time 24), into a cache of bf16 49 (89; 18).
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
constexpr int kEach = 4;       // tokens of a warp, where tokens have few rows
constexpr int kMaxFreq = 128;
constexpr int kMaxB = 65535;
constexpr int kMaxN = 1 << 20;
constexpr int kDepth = 4;  // places of the ring: groups of rows in flight per warp, and the one read

enum { DENSE, CACHE_BF16, CACHE_E4M3 };
template <int K>
struct Int {
    static constexpr int value = K;
};

// Where a pair's other element is: beside it; in another lane (num_freq a multiple of 8); or anywhere.
enum { BESIDE, LANE, ANYWHERE };

struct RotaryArgs {
    sv::PagedCache c;
    const void* src[3];  // queries, keys, values
    void* dst[2];        // queries, keys (DENSE)
    int64_t ss[3][3];    // element strides of the sources (batch, token, head)
    int64_t ds[2][3];    // and of the destinations
    int heads[3];        // of queries, keys, values
    int64_t in_step[3];  // from a group of a warp to its next one: elements,
    int64_t out_step[2]; // bytes (queries, keys and values)
    int magic[3];        // 2^16 / heads, rounded up (kernel for few rows)
    int groups[3];       // groups of rows of a token: [0, groups[0]) queries, then keys, then values
    const double* freq;
    const int32_t* depth;
    const int32_t* base;
    const int32_t* new_len;
    float amplitude;
    int R, interleaved, inverse;
    int B, N, D;
    int tile;   // tokens of a block: 1, 2, 4 or 8
    int chunk;  // groups of a token that a block does
};

// n strides (n >= 0): two instructions, where the product of a signed number takes four.
__device__ __forceinline__ int64_t times(int n, int64_t stride) { return (int64_t)((uint64_t)(uint32_t)n * (uint64_t)stride); }

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

// Cosine and sine of (big + rest) * (fh + fl) turns.
__device__ __forceinline__ float2 turn(float big, float rest, float fh, float fl) {
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

// A token's cosine, negated sine and sine of one frequency, in planes of RP.
__device__ __forceinline__ void put_turn(float* to, int RP, float2 pos, float2 f, float amplitude, int inverse) {
    const float2 cs = turn(pos.x, pos.y, f.x, f.y);
    const float sine = inverse ? -(cs.y * amplitude) : cs.y * amplitude;
    to[0] = cs.x * amplitude;
    to[RP] = -sine;
    to[2 * RP] = sine;
}

// The factors of a lane's elements e0 .. e0 + 7: of their own (c), and of their partners (s).  Those of elements that
// are copied are not used, only read within the block's memory.
template <int PAIR>
__device__ __forceinline__ void row_factors(const float* planes, int RP, int R, int e0, float2 c[4], float2 s[4]) {
    const int turned = 2 * R;
    if (PAIR == BESIDE) {
        const float* at = planes + (e0 < turned ? e0 >> 1 : 0);
        const float4 cs = *reinterpret_cast<const float4*>(at), sn = *reinterpret_cast<const float4*>(at + 2 * RP);
        c[0] = make_float2(cs.x, cs.x);
        c[1] = make_float2(cs.y, cs.y);
        c[2] = make_float2(cs.z, cs.z);
        c[3] = make_float2(cs.w, cs.w);
        s[0] = make_float2(-sn.x, sn.x);
        s[1] = make_float2(-sn.y, sn.y);
        s[2] = make_float2(-sn.z, sn.z);
        s[3] = make_float2(-sn.w, sn.w);
    } else if (PAIR == LANE) {
        const float* at = planes + (e0 < R ? e0 : e0 < turned ? e0 - R : 0);
        const float* from = at + (e0 < R ? RP : 2 * RP);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float4 cs = reinterpret_cast<const float4*>(at)[k], sn = reinterpret_cast<const float4*>(from)[k];
            c[2 * k] = make_float2(cs.x, cs.y);
            c[2 * k + 1] = make_float2(cs.z, cs.w);
            s[2 * k] = make_float2(sn.x, sn.y);
            s[2 * k + 1] = make_float2(sn.z, sn.w);
        }
    } else {
        float cc[8], ss[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int e = e0 + k;
            cc[k] = 1.0f;
            ss[k] = 0.0f;
            if (e < turned) {
                cc[k] = planes[e < R ? e : e - R];
                ss[k] = planes[e < R ? RP + e : 2 * RP + e - R];
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            c[k] = make_float2(cc[2 * k], cc[2 * k + 1]);
            s[k] = make_float2(ss[2 * k], ss[2 * k + 1]);
        }
    }
}

// Eight elements of a row as they lie in memory (AL), or widened one by one; zero where there is no row.
// Plain loads: in place the same kernel writes the row.
template <typename T, bool AL>
struct Raw {
    static constexpr int W = AL ? (int)sizeof(T) * 2 : 8;  // words
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* row, int e0, int dim) {
        if (AL) {
#pragma unroll
            for (int k = 0; k < W / 4; ++k) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (e0 < dim) v = *reinterpret_cast<const uint4*>(row + e0 + k * (16 / (int)sizeof(T)));
                w[4 * k] = v.x;
                w[4 * k + 1] = v.y;
                w[4 * k + 2] = v.z;
                w[4 * k + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) w[AL ? 0 : k] = e0 + k < dim ? __float_as_uint(one(row, e0 + k)) : 0u;
        }
    }
    static __device__ __forceinline__ float one(const T* row, int e) {
        return sizeof(T) == 2 ? __uint_as_float((uint32_t)reinterpret_cast<const unsigned short*>(row)[e] << 16)
                              : reinterpret_cast<const float*>(row)[e];
    }
    __device__ __forceinline__ float at(int k) const {
        if (AL && sizeof(T) == 2) return k & 1 ? sv::bf16_hi(w[AL ? k / 2 : 0]) : sv::bf16_lo(w[AL ? k / 2 : 0]);
        return __uint_as_float(w[k]);
    }
};

// grid: x over tiles of tokens, y over chunks of a token's rows.  LPR lanes hold a row.  A token is one warp's or
// several warps'.
template <typename T, int LPR, int MODE, bool AL, int PAIR>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ RotaryArgs a) {
    extern __shared__ uint4 s_raw[];  // AL: the ring; then of each token RP cosines, sines negated, sines
    const int RP = (a.R + 3) & ~3;
    float* s_turn = reinterpret_cast<float*>(s_raw + (AL ? kDepth * ((int)sizeof(T) / 2) * kThreads : 0));
    __shared__ float2 s_freq[kMaxFreq];
    __shared__ float2 s_pos[kMaxTokens];  // a multiple of 4096, and the rest
    __shared__ int s_first[kMaxTokens];   // the row's base; -1: token not written
    constexpr int G = 32 / LPR;
    sv::pdl_trigger();
    sv::pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const unsigned total = (unsigned)a.B * (unsigned)a.N;
    const int e0 = 8 * (lane % LPR);
    // This warp's token, and the groups of rows that it takes of it (a group is of one kind, so
    // the warp decides on it as one); the first ones are asked for ahead of the angles.
    const int each = kWarps / a.tile, t = warp / each;
    const unsigned token = blockIdx.x * (unsigned)a.tile + t;
    const int b = token < total ? (int)(token / a.N) : 0, i = token < total ? (int)(token % a.N) : 0;
    const int last = min(a.groups[2], (int)(blockIdx.y + 1) * a.chunk);
    int at = blockIdx.y * a.chunk + (warp - t * each);
    // Where a group's rows are read and written: found for its kind, then moved on by its heads.
    const int lane_row = lane / LPR, stride = each * G;
    const int row_or_none = !AL || e0 < a.D ? lane_row : 1 << 20;  // lanes behind the row's end have none
    auto to_kind = [&](int& kind, int& head) {
        if (kind == 0 && head >= a.heads[0]) {
            head -= a.groups[0] * G;
            kind = 1;
        }
        if (MODE != DENSE && kind == 1 && head >= a.heads[1]) {
            head -= (a.groups[1] - a.groups[0]) * G;
            kind = 2;
        }
    };
    int in_kind = 0, in_head = at * G, in_heads = 0;  // of the next group to ask for; in_head of its first row
    const T* in_row = nullptr;
    int64_t in_step = 0;
    auto find_in = [&]() {
        to_kind(in_kind, in_head);
        auto of = [&](auto k) {  // (by constants: their operands need no loads)
            constexpr int K = decltype(k)::value;
            in_heads = a.heads[K];
            in_row = static_cast<const T*>(a.src[K]) + (times(b, a.ss[K][0]) + times(i, a.ss[K][1]) + times(in_head + lane_row, a.ss[K][2]) + (AL ? e0 : 0));
            in_step = a.in_step[K];
        };
        if (in_kind == 0) of(Int<0>{});
        else if (MODE == DENSE || in_kind == 1) of(Int<1>{});
        else of(Int<2>{});
    };
    // Groups in flight go through a ring in shared memory, kDepth deep.
    constexpr int PIECES = (int)sizeof(T) / 2;
    uint4* ring = reinterpret_cast<uint4*>(s_raw) + tid;
    if (AL && e0 >= a.D) {
#pragma unroll
        for (int k = 0; k < kDepth * PIECES; ++k) ring[k * kThreads] = make_uint4(0u, 0u, 0u, 0u);
    }
    int ahead = at;  // the next group to ask for
    auto fetch = [&](int slot) {
        if (!AL) return;
        if (ahead < last) {
            if (in_head >= in_heads) find_in();
            if (in_head + row_or_none < in_heads) {
#pragma unroll
                for (int k = 0; k < PIECES; ++k)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sv::smem_u32(ring + (slot * PIECES + k) * kThreads)),
                                 "l"(in_row + k * 4)
                                 : "memory");
            }
            in_row += in_step;
            in_head += stride;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ahead += each;
    };
#pragma unroll
    for (int k = 0; k < kDepth - 1; ++k) fetch(k);
    if (tid < a.tile) {
        const unsigned x = blockIdx.x * (unsigned)a.tile + tid;
        int first = -1;
        int64_t pos = 0;
        if (x < total && !token_position<MODE>(a, (int)(x / a.N), (int)(x % a.N), pos, first)) first = -1;
        s_pos[tid] = make_float2((float)(pos & ~(int64_t)4095), (float)((int)pos & 4095));
        s_first[tid] = first;
    }
    for (int j = tid; j < a.R; j += kThreads) {
        const double f = a.freq[j] * 0.15915494309189533577;
        const float hi = (float)f;
        s_freq[j] = make_float2(hi, (float)(f - (double)hi));
    }
    __syncthreads();
    float* mine = s_turn + t * 3 * RP;
    const float2 pos = s_pos[t];
    for (int j = tid - t * each * 32; j < a.R; j += each * 32) {  // by the token's warps
        put_turn(mine + j, RP, pos, s_freq[j], a.amplitude, a.inverse);
    }
    if (each == 1) __syncwarp();
    else __syncthreads();
    const int first = s_first[t];
    if (first < 0) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }
    int page = -1, line = 0;
    int64_t place = 0, scale_place = 0;  // of this lane's row of the first heads, in the keys and values
    if (MODE != DENSE) {
        page = sv::paged_place(a.c, b, first + i, line);
        const int pg = max(page, 0);
        place = times(pg, a.c.page_stride) + times(line, a.c.row_stride) + times(lane_row, a.c.head_stride);
        if (MODE == CACHE_E4M3) scale_place = ((int64_t)pg * a.c.heads + lane_row) * a.c.page_size + line;
    }

    const int R = a.R, turned = 2 * R;
    float2 c[4], s[4];
    row_factors<PAIR>(mine, RP, R, e0, c, s);
    const int mate = PAIR == LANE && e0 < turned ? lane + (e0 < R ? R / 8 : -(R / 8)) : lane;
    const int same = e0 >= turned ? 0 : min(turned - e0, 8);  // elements of this lane that are turned

    int kind = 0, head = at * G, heads = 0;
    unsigned char* to = nullptr;
    float* scale = nullptr;
    int64_t step = 0;
    for (int slot = 0; at < last; slot = slot + 1 == kDepth ? 0 : slot + 1) {
        if (head >= heads) {
            to_kind(kind, head);
            auto dense = [&](auto k) {
                constexpr int K = decltype(k)::value;
                heads = a.heads[K];
                to = reinterpret_cast<unsigned char*>(static_cast<T*>(a.dst[K]) + (times(b, a.ds[K][0]) + times(i, a.ds[K][1]) + times(head + lane_row, a.ds[K][2])));
                step = a.out_step[K];
            };
            if (kind == 0) {
                dense(Int<0>{});
            } else if (MODE == DENSE) {
                dense(Int<1>{});
            } else {
                heads = a.heads[1];
                to = (kind == 2 ? a.c.v : a.c.k) + (place + times(head, a.c.head_stride));
                step = a.out_step[1];
                if (MODE == CACHE_E4M3) scale = (kind == 2 ? a.c.v_scale : a.c.k_scale) + (scale_place + head * a.c.page_size);
            }
        }
        const bool in = head + row_or_none < heads;
        const T* row = in_row;  // !AL: read here
        if (!AL) {
            if (in_head >= in_heads) {
                find_in();
                row = in_row;
            }
            in_row += in_step;
            in_head += stride;
        }
        Raw<T, AL> x;
        if (AL) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
            if (PAIR == ANYWHERE) __syncwarp();  // every lane's pieces are there, and the group before is read
#pragma unroll
            for (int k = 0; k < PIECES; ++k) {
                const uint4 w = ring[(slot * PIECES + k) * kThreads];
                x.w[4 * k] = w.x;
                x.w[4 * k + 1] = w.y;
                x.w[4 * k + 2] = w.z;
                x.w[4 * k + 3] = w.w;
            }
        } else {
            x.load(row, e0, in ? a.D : 0);
        }
        fetch(slot ? slot - 1 : kDepth - 1);  // into the place of the group before
        at += each;
        unsigned char* const dst = to;
        float* const dst_scale = scale;
        const int of_kind = kind;
        to += step;
        head += stride;
        if (MODE == CACHE_E4M3) scale += (int64_t)stride * a.c.page_size;
        float v[8];
        if (MODE == DENSE || of_kind != 2) {
            float p[8];
            if (PAIR == BESIDE) {
#pragma unroll
                for (int k = 0; k < 8; ++k) p[k] = x.at(k ^ 1);
            } else if (PAIR == LANE) {
                Raw<T, AL> y;
#pragma unroll
                for (int k = 0; k < Raw<T, AL>::W; ++k) y.w[k] = __shfl_sync(0xffffffffu, x.w[k], mate);
#pragma unroll
                for (int k = 0; k < 8; ++k) p[k] = y.at(k);
            } else {
                // (AL: rows are whole in the ring, fp32 ones in two planes of four elements per lane)
                const T* from = AL ? reinterpret_cast<const T*>(ring + slot * PIECES * kThreads - lane % LPR) : row;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int e = e0 + k, other = e < R ? e + R : e - R;
                    p[k] = 0.0f;
                    if (e < turned && in)
                        p[k] = Raw<T, AL>::one(from, AL && sizeof(T) == 4 ? ((other >> 2) & 1) * (kThreads * 4) + (other >> 3) * 4 + (other & 3) : other);
                }
                if (!AL) __syncwarp();  // in place: a row's elements are read before any is written
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = sv::ffma2(make_float2(x.at(2 * k), x.at(2 * k + 1)), c[k], sv::fmul2(make_float2(p[2 * k], p[2 * k + 1]), s[k]));
                v[2 * k] = f.x;
                v[2 * k + 1] = f.y;
            }
            if (same < 8) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k >= same) v[k] = x.at(k);
            }
            if (MODE == DENSE || of_kind == 0) {
                if (in) sv::store_row8<T, AL>(reinterpret_cast<T*>(dst), e0, a.D, v);
                continue;
            }
        }
        if constexpr (MODE != DENSE) {
            const bool live = in && page >= 0;
            if (of_kind == 2) {  // values as they are
                sv::Eight<T, AL> f;
                if constexpr (AL) {
#pragma unroll
                    for (int k = 0; k < (int)sizeof(T) / 2; ++k) f.w[k] = make_uint4(x.w[4 * k], x.w[4 * k + 1], x.w[4 * k + 2], x.w[4 * k + 3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) f.f[k] = x.at(k);
                }
                sv::store_cache_row<T, LPR, MODE == CACHE_E4M3, AL>(dst, dst_scale, e0, a.D, live, f);
            } else {
                sv::Eight<float, AL> f;
                if constexpr (AL) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        f.w[k] = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3]));
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) f.f[k] = v[k];
                }
                sv::store_cache_row<float, LPR, MODE == CACHE_E4M3, AL>(dst, dst_scale, e0, a.D, live, f);
            }
        }
    }
}

// Tokens of few rows (bf16): a warp takes kEach tokens, and a group of rows may be of several of them, since the rows of
// each kind are taken together, token by token.  What a token costs (its place, a warp's start and the lanes that a
// group leaves idle) is shared; the factors are read for each group.  grid: x over tiles of kWarps * kEach tokens.
template <int LPR, int MODE, int PAIR>
__global__ void __launch_bounds__(kThreads, 4) rotary_few_kernel(const __grid_constant__ RotaryArgs a) {
    extern __shared__ uint4 s_raw[];  // the ring; then of each token RP cosines, sines negated, sines
    const int RP = (a.R + 3) & ~3;
    float* s_turn = reinterpret_cast<float*>(s_raw + kDepth * kThreads);
    constexpr int G = 32 / LPR, TOKENS = kWarps * kEach;
    __shared__ float2 s_freq[kMaxFreq];
    __shared__ float2 s_pos[TOKENS];
    __shared__ int s_state[TOKENS];                            // 2: written, 1: but its page is a hole, 0: not written
    __shared__ int64_t s_in[3][TOKENS], s_out[2][TOKENS];      // offsets of a token's first row
    __shared__ int64_t s_scale[MODE == CACHE_E4M3 ? TOKENS : 1];
    sv::pdl_trigger();
    sv::pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), t0 = warp * kEach;
    const unsigned total = (unsigned)a.B * (unsigned)a.N, token = blockIdx.x * (unsigned)TOKENS + t0 + lane;
    const bool real = lane < kEach && token < total;
    const int b = real ? (int)(token / a.N) : 0, i = real ? (int)(token % a.N) : 0;
    const int e0 = 8 * (lane % LPR), lane_row = lane / LPR;
    if (lane < kEach) {
#pragma unroll
        for (int k = 0; k < (MODE == DENSE ? 2 : 3); ++k) s_in[k][t0 + lane] = times(b, a.ss[k][0]) + times(i, a.ss[k][1]);
#pragma unroll
        for (int k = 0; k < (MODE == DENSE ? 2 : 1); ++k) s_out[k][t0 + lane] = times(b, a.ds[k][0]) + times(i, a.ds[k][1]);
    }
    uint4* ring = s_raw + tid;
    if (e0 >= a.D) {
#pragma unroll
        for (int k = 0; k < kDepth; ++k) ring[k * kThreads] = make_uint4(0u, 0u, 0u, 0u);
    }
    __syncwarp();
    // Group x: its kind, and this lane's token of the warp (kEach: none) and head.
    auto row_of = [&](int x, int& kind, int& tt, int& h) {
        kind = x < a.groups[0] ? 0 : MODE == DENSE || x < a.groups[1] ? 1 : 2;
        const int r = (x - (kind == 0 ? 0 : kind == 1 ? a.groups[0] : a.groups[1])) * G + lane_row;
        const int heads = a.heads[MODE != DENSE && kind == 2 ? 1 : kind];
        tt = (int)((unsigned)r * (unsigned)a.magic[MODE != DENSE && kind == 2 ? 1 : kind] >> 16);
        h = r - tt * heads;
    };
    auto fetch = [&](int x, int slot) {
        if (x < a.groups[2]) {
            int kind, tt, h;
            row_of(x, kind, tt, h);
            if (tt < kEach && e0 < a.D) {
                const uint16_t* from = static_cast<const uint16_t*>(a.src[kind]) + (s_in[kind][t0 + tt] + times(h, a.ss[kind][2]) + e0);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sv::smem_u32(ring + slot * kThreads)), "l"(from) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < kDepth - 1; ++k) fetch(k, k);
    if (lane < kEach) {
        int first = -1, state = 0;
        int64_t pos = 0;
        if (real && token_position<MODE>(a, b, i, pos, first)) {
            state = 2;
            if (MODE != DENSE) {
                int line;
                const int page = sv::paged_place(a.c, b, first + i, line);
                if (page < 0) state = 1;
                else s_out[1][t0 + lane] = times(page, a.c.page_stride) + times(line, a.c.row_stride);
                if (MODE == CACHE_E4M3) s_scale[MODE == CACHE_E4M3 ? t0 + lane : 0] = times(max(page, 0), (int64_t)a.c.heads * a.c.page_size) + line;
            }
        }
        s_pos[t0 + lane] = make_float2((float)(pos & ~(int64_t)4095), (float)((int)pos & 4095));
        s_state[t0 + lane] = state;
    }
    for (int j = tid; j < a.R; j += kThreads) {
        const double f = a.freq[j] * 0.15915494309189533577;
        const float hi = (float)f;
        s_freq[j] = make_float2(hi, (float)(f - (double)hi));
    }
    __syncthreads();
    for (int j = lane; j < a.R; j += 32) {
        const float2 f = s_freq[j];
#pragma unroll
        for (int k = 0; k < kEach; ++k) put_turn(s_turn + (t0 + k) * 3 * RP + j, RP, s_pos[t0 + k], f, a.amplitude, a.inverse);
    }
    __syncwarp();
    const int R = a.R, turned = 2 * R;
    const int mate = PAIR == LANE && e0 < turned ? lane + (e0 < R ? R / 8 : -(R / 8)) : lane;
    const int same = e0 >= turned ? 0 : min(turned - e0, 8);  // elements of this lane that are turned
    for (int x = 0, slot = 0; x < a.groups[2]; ++x, slot = slot + 1 == kDepth ? 0 : slot + 1) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
        Raw<uint16_t, true> w;
        const uint4 raw = ring[slot * kThreads];
        w.w[0] = raw.x;
        w.w[1] = raw.y;
        w.w[2] = raw.z;
        w.w[3] = raw.w;
        fetch(x + kDepth - 1, slot ? slot - 1 : kDepth - 1);  // into the place of the group before
        int kind, tt, h;
        row_of(x, kind, tt, h);
        const int t = t0 + min(tt, kEach - 1), state = tt < kEach ? s_state[t] : 0;
        float v[8];
        if (MODE == DENSE || kind != 2) {
            float2 c[4], s[4];
            row_factors<PAIR>(s_turn + t * 3 * RP, RP, R, e0, c, s);
            Raw<uint16_t, true> y;
#pragma unroll
            for (int k = 0; k < 4; ++k) y.w[k] = PAIR == LANE ? __shfl_sync(0xffffffffu, w.w[k], mate) : __byte_perm(w.w[k], 0u, 0x1032);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = sv::ffma2(make_float2(w.at(2 * k), w.at(2 * k + 1)), c[k], sv::fmul2(make_float2(y.at(2 * k), y.at(2 * k + 1)), s[k]));
                v[2 * k] = f.x;
                v[2 * k + 1] = f.y;
            }
            if (same < 8) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k >= same) v[k] = w.at(k);
            }
            if (MODE == DENSE || kind == 0) {
                const int K = MODE == DENSE ? kind : 0;
                if (state) sv::store_row8<uint16_t, true>(static_cast<uint16_t*>(a.dst[K]) + (s_out[K][t] + times(h, a.ds[K][2])), e0, a.D, v);
                continue;
            }
        }
        if constexpr (MODE != DENSE) {
            unsigned char* to = (kind == 2 ? a.c.v : a.c.k) + (s_out[1][t] + times(h, a.c.head_stride));
            float* scale = MODE == CACHE_E4M3 ? (kind == 2 ? a.c.v_scale : a.c.k_scale) + (s_scale[t] + h * a.c.page_size) : nullptr;
            const bool live = state == 2 && e0 < a.D;
            if (kind == 2) {
                sv::Eight<uint16_t, true> f;
                f.w[0] = raw;
                sv::store_cache_row<uint16_t, LPR, MODE == CACHE_E4M3, true>(to, scale, e0, a.D, live, f);
            } else {
                sv::Eight<float, true> f;
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    f.w[k] = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3]));
                sv::store_cache_row<float, LPR, MODE == CACHE_E4M3, true>(to, scale, e0, a.D, live, f);
            }
        }
    }
}

// Whether that kernel is the faster one: where kEach tokens' rows fill 12 groups or fewer and the tokens a full wave of
// blocks.  In us, this one and the other: 64 x 2000 tokens of 4 + 1 heads of 64 43 and 80, on the way into a cache
// 49 and 89; 1 + 1 heads of 128 into e4m3 65 and 125; 32 x 2000 of 4 + 1 heads of 128 into e4m3 (12 groups) 51 and 66,
// 20 x 1000 of 2 + 2 into bf16 (12) 19.6 and 18.5; but 32 x 2000 of 8 + 2 of 128 (20 groups) 74 and 64, and 8 x 1000 tokens of
// 4 + 1 10.7 and 8.
template <int LPR, int MODE>
bool few_rows(const RotaryArgs& a) {
    constexpr int G = 32 / LPR;
    int n = 0;
    for (int k = 0; k < 3; ++k) n += (kEach * a.heads[k] + G - 1) / G;
    return n <= 12 && (int64_t)a.B * a.N >= 4 * 152 * kWarps * kEach;
}

template <int LPR, int MODE, int PAIR>
cudaError_t launch_few(RotaryArgs& a, cudaStream_t stream) {
    constexpr int G = 32 / LPR, TOKENS = kWarps * kEach;
    for (int k = 0, n = 0; k < 3; ++k) {
        a.groups[k] = n += (kEach * a.heads[k] + G - 1) / G;
        a.magic[k] = a.heads[k] ? (65536 + a.heads[k] - 1) / a.heads[k] : 0;
    }
    const int64_t tokens = (int64_t)a.B * a.N;
    const size_t smem = kDepth * kThreads * sizeof(uint4) + ((size_t)TOKENS * 3 * ((a.R + 3) & ~3) + 8) * sizeof(float);
    static sv::KernelLaunchCache cache;
    auto kern = rotary_few_kernel<LPR, MODE, PAIR>;
    int max_dyn = 0;
    const cudaError_t e = cache.setup((const void*)kern, &max_dyn);
    if (e != cudaSuccess) return e;
    if (smem > (size_t)max_dyn) return cudaErrorInvalidValue;
    return sv::launch_serial(kern, dim3((unsigned)((tokens + TOKENS - 1) / TOKENS)), dim3(kThreads), smem, stream, a);
}

template <typename T, int LPR, int MODE, bool AL, int PAIR>
cudaError_t launch_rows(RotaryArgs& a, cudaStream_t stream) {
    const int64_t tokens = (int64_t)a.B * a.N;
    constexpr int sms = 152, G = 32 / LPR;
    for (int k = 0, n = 0; k < 3; ++k) a.groups[k] = n += (a.heads[k] + G - 1) / G;
    // Tokens of a block: as many as leave six blocks per SM (a wave and a half: four at a time, by registers), since they
    // share the frequencies;
    // a few tokens are spread over blocks by their rows instead, one pass of a block's warps each.
    a.tile = 1;
    while (a.tile < kMaxTokens && tokens / (2 * a.tile) >= 6 * sms) a.tile *= 2;
    const int64_t stride = (kWarps / a.tile) * G;  // heads from a group of a warp to its next
    for (int k = 0; k < 3; ++k) a.in_step[k] = stride * a.ss[k][2];
    a.out_step[0] = stride * a.ds[0][2] * (int64_t)sizeof(T);
    a.out_step[1] = stride * (MODE == DENSE ? a.ds[1][2] * (int64_t)sizeof(T) : a.c.head_stride);
    a.chunk = tokens >= 2 * sms ? a.groups[2] : kWarps;
    const dim3 grid((unsigned)((tokens + a.tile - 1) / a.tile), (unsigned)((a.groups[2] + a.chunk - 1) / a.chunk));
    // Without pairs the factors are read all the same: eight floats behind the first of a plane.
    const size_t smem = ((size_t)a.tile * 3 * ((a.R + 3) & ~3) + 8) * sizeof(float);
    constexpr size_t ring = AL ? kDepth * kThreads * sizeof(T) * 8 : 0;
    static sv::KernelLaunchCache cache;
    auto kern = rotary_kernel<T, LPR, MODE, AL, PAIR>;
    int max_dyn = 0;
    const cudaError_t e = cache.setup((const void*)kern, &max_dyn);
    if (e != cudaSuccess) return e;
    if (ring + smem > (size_t)max_dyn) return cudaErrorInvalidValue;
    return sv::launch_serial(kern, grid, dim3(kThreads), ring + smem, stream, a);
}

template <typename T, int LPR, int MODE, bool AL, int PAIR>
cudaError_t launch_pair(RotaryArgs& a, cudaStream_t stream) {
    if constexpr (AL && PAIR != ANYWHERE && sizeof(T) == 2)
        if (few_rows<LPR, MODE>(a)) return launch_few<LPR, MODE, PAIR>(a, stream);
    return launch_rows<T, LPR, MODE, AL, PAIR>(a, stream);
}

template <typename T, int LPR, int MODE, bool AL>
cudaError_t launch_lpr(RotaryArgs& a, cudaStream_t stream) {
    if (a.interleaved) return launch_pair<T, LPR, MODE, AL, BESIDE>(a, stream);
    if (AL && a.R % 8 == 0) return launch_pair<T, LPR, MODE, AL, AL ? LANE : ANYWHERE>(a, stream);
    return launch_pair<T, LPR, MODE, AL, ANYWHERE>(a, stream);
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
    a.heads[0] = num_q_heads;
    a.heads[1] = num_k_heads;
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
    a.heads[0] = num_q_heads;
    a.heads[1] = a.heads[2] = cache->num_heads;
    a.base = base;
    a.new_len = new_len;
    return sv::launch_status(launch(a, cache->dtype == SV_CACHE_BF16 ? CACHE_BF16 : CACHE_E4M3, dt, al, (cudaStream_t)stream));
}

}  // extern "C"
