// sv_attention.cu -- attention of a chunk of new tokens over a paged cache
// (include/spec_paged_kv.h): the entry point, the kernel for few query rows per cache
// head, and the kernel that joins the splits of a long context.
//
// out = softmax(scale q k^T) v in one pass over the cache: each warp keeps the running
// maximum m and sum l of its rows and rescales its fp32 accumulator when m grows.  Few
// rows (one token times the heads that share a cache head) are bound by the cache's bytes: the kernel's work is to keep loads in flight.  So a CTA
// streams tiles of 64 positions through a ring of shared-memory stages filled by cp.async
// (16 bytes per thread, any page size, holes and rows behind the end filled with zeros),
// its warps take 16 positions each of every tile, and their partial results meet once at
// the end.  The products use mma.sync (m16n8k16): 16-row tiles waste less than the 128
// rows of tcgen05 (sv_attention_tc.cu, the kernel of longer chunks; make_plan chooses).
// 64 contexts of 4096, one query of 32 over 8 heads of 128, one GB300: bf16 208 us
// (5.2 TB/s), e4m3 201 us (2.8 TB/s; bound by the issue of the widening and the softmax).
// Probabilities (e4m3: times the value's scale) are rounded to bf16, the values' type in the second
// product; a second term for what that leaves would double it.
// Filling the stages by the copy engine instead of cp.async: 258 against 213 us, not kept.
//
// e4m3 pages are copied as they are, and each warp widens its fragments to bf16 (exactly);
// a position's key scale multiplies its scores, its value scale its probabilities.  Keys:
// a thread reads 16 contiguous codes of a position, which fixes an order of the head's
// elements within a product; the queries are stored in that order.  Values: ldmatrix
// transposes pairs of codes, so two column tiles hold the even and the odd elements.
// Multiplied as fp16 (two codes an instruction) with units that a row takes from the value
// scales it sees, that call took 195 us: not worth the units' code, not kept.
#include <cstdint>
#include <cstdlib>

#include "spec_paged_kv.h"
#include "sv_attention.cuh"

namespace {

using sv::AttnArgs;
using sv::AttnTile;
using sv::neg_inf;
using sv::pdl_trigger;
using sv::pdl_wait;
using sv::smem_u32;

constexpr int TN = 64;         // positions per tile
constexpr int RING = 8;        // row offsets and hole bits of the tiles in flight
constexpr int KW = 4;          // warps along the positions, 16 each

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t r[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t r[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 codes in the low half of w to a bf16 pair (exact).
__device__ __forceinline__ uint32_t widen(uint32_t w) {
    const float2 f = sv::e4m3x2_to_f32(w);
    return sv::bf16x2(f.x, f.y);
}

template <int DP, bool E4M3>
struct Shape {
    static constexpr int ROWS = 16;
    static constexpr int THREADS = KW * 32;
    static constexpr int ES = E4M3 ? 1 : 2;
    static constexpr int PITCH = DP * ES;          // bytes of a staged row
    static constexpr int CH = PITCH / 16;          // 16-byte pieces of a staged row
    static constexpr int MAT = TN * PITCH;         // a tile of keys, or of values
    static constexpr int STAGE = 2 * MAT + (E4M3 ? 2 * TN * 4 : 0);
    // One CTA of wide heads fills an SM's registers; else two share it.
    static constexpr int BUDGET = DP == 256 ? 160 * 1024 : 97 * 1024;
    static constexpr int FIT = BUDGET / STAGE;
    static constexpr int STAGES = FIT > 6 ? 6 : FIT < 3 ? 3 : FIT;
    static_assert(E4M3 || DP <= 128, "wide heads of bf16 take the tcgen05 kernel");
    static constexpr int QBYTES = ROWS * DP * 2;
    static constexpr int SMEM = STAGES * STAGE + QBYTES;
    static_assert(STAGES + 1 <= RING, "a tile's offsets outlive its stage");
    static_assert(2 * ROWS * DP * 4 <= STAGES * STAGE, "the join of the warps reuses the stages");
    static_assert((STAGES - 1) * TN <= 5 * THREADS, "prologue offsets");
};

// Byte offset of 16-byte piece c of staged row r; neighbouring rows start in other banks.
template <int PITCH>
__device__ __forceinline__ int k_piece(int r, int c) {  // e4m3 keys: pairs of rows are read together
    return r * PITCH + ((PITCH >= 128 ? c ^ ((r & 1) << 2) : c) << 4);
}
template <int PITCH>
__device__ __forceinline__ int v_piece(int r, int c) {  // eight rows are read together
    return r * PITCH + ((PITCH >= 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

template <int DP, bool E4M3>
__global__ void __launch_bounds__(KW * 32, DP == 256 ? 1 : 2)
    paged_attention_kernel(const __grid_constant__ AttnArgs a, const int pairs) {
    using S = Shape<DP, E4M3>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t s_off[RING][TN];  // byte offset of each position's row, -1: nothing there
    __shared__ int64_t s_sc[E4M3 ? RING : 1][E4M3 ? TN : 1];  // index of its scales
    __shared__ uint32_t s_valid[RING][2];
    __shared__ float s_m[KW][S::ROWS], s_l[KW][S::ROWS];
    __shared__ int s_bad;

    pdl_trigger();
    pdl_wait();
    AttnTile t;
    if (!sv::attn_tile(a, pairs, blockIdx.x, S::ROWS, 1, t)) return;
    const int tid = threadIdx.x, lane = tid & 31, wk = tid >> 5;
    const int D = a.c.dim, row_bytes = D * S::ES;
    const int tiles = (t.end - t.begin + TN - 1) / TN;
    const unsigned char* kbase = a.c.k + t.h * a.c.head_stride;
    const unsigned char* vbase = a.c.v + t.h * a.c.head_stride;
    unsigned char* s_q = smem + S::STAGES * S::STAGE;
    const uint32_t smem0 = smem_u32(smem), q0 = smem_u32(s_q);

    auto put_place = [&](int tile, int p, int row, int page) {
        const bool ok = page >= 0;
        s_off[tile % RING][p] = ok ? page * a.c.page_stride + row * a.c.row_stride : -1;
        if (E4M3) s_sc[tile % RING][p] = ((int64_t)page * a.c.heads + t.h) * a.c.page_size + row;
        const uint32_t bits = __ballot_sync(0xffffffffu, ok);
        if (lane == 0) s_valid[tile % RING][p >> 5] = bits;
    };
    auto load_tile = [&](int tile) {
        const uint32_t st = smem0 + (tile % S::STAGES) * S::STAGE;
        const int64_t* off = s_off[tile % RING];
#pragma unroll
        for (int x = 0; x < TN * S::CH / S::THREADS; ++x) {
            const int f = tid + x * S::THREADS, r = f / S::CH, c = f % S::CH;
            const int64_t o = off[r];
            int bytes = row_bytes - 16 * c;
            bytes = o < 0 || bytes < 0 ? 0 : bytes > 16 ? 16 : bytes;
            const int64_t at = bytes ? o + 16 * c : 0;
            cp_async16(st + (E4M3 ? k_piece<S::PITCH>(r, c) : v_piece<S::PITCH>(r, c)), kbase + at, bytes);
            cp_async16(st + S::MAT + v_piece<S::PITCH>(r, c), vbase + at, bytes);
        }
        if (E4M3) {
            if (tid < 2 * TN) {
                const int p = tid & (TN - 1);
                const int64_t i = s_sc[tile % RING][p];
                const bool ok = off[p] >= 0;
                cp_async4(st + 2 * S::MAT + 4 * tid, (tid < TN ? a.c.k_scale : a.c.v_scale) + (ok ? i : 0), ok ? 4 : 0);
            }
        }
    };

    // places of the first tiles; all threads take part in the ballots
    for (int f = tid; f < (S::STAGES - 1) * TN; f += S::THREADS) {
        const int tile = f / TN, p = f % TN, pos = t.begin + f;
        int row = 0, page = -1;
        if (pos < t.end) page = sv::paged_place(a.c, t.b, pos, row);
        put_place(tile, p, row, page);
    }
    if (tid == 0) s_bad = 0;
    // the queries, zero behind the last real one
    for (int f = tid; f < S::ROWS * (DP / 8); f += S::THREADS) {
        const int r = f / (DP / 8), c = f % (DP / 8), R = t.mt * S::ROWS + r;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (R < t.n * a.group && 8 * c < D)
            w = sv::ld_nc_v4(a.q + t.b * a.q_sb + (int64_t)(R / a.group) * a.q_st +
                             (int64_t)(t.h * a.group + R % a.group) * a.q_sh + 8 * c);
        if (!E4M3) {
            *reinterpret_cast<uint4*>(s_q + v_piece<2 * DP>(r, c)) = w;
        } else {
            // element 64 e + 16 u + 4 s + 2 v + z goes to place 16 (4 e + s) + 8 v + 2 u + z
            const int e = c >> 3, u = (c >> 1) & 3, s0 = (c & 1) * 2;
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = 16 * (4 * e + s0 + (j >> 1)) + 8 * (j & 1) + 2 * u;
                *reinterpret_cast<uint32_t*>(s_q + v_piece<2 * DP>(r, col >> 3) + 2 * (col & 7)) = ww[j];
            }
        }
    }
    __syncthreads();
    for (int j = 0; j < S::STAGES - 1; ++j) {
        if (j < tiles) load_tile(j);
        cp_commit();
    }
    // the page of the next tile's position, looked up one tile ahead
    int next_row = 0, next_page = -1;
    if (tid < TN) {
        const int pos = t.begin + (S::STAGES - 1) * TN + tid;
        if (pos < t.end) next_page = sv::paged_place(a.c, t.b, pos, next_row);
        put_place(S::STAGES - 1, tid, next_row, next_page);
        next_page = -1;
        if (pos + TN < t.end) next_page = sv::paged_place(a.c, t.b, pos + TN, next_row);
    }

    constexpr bool QREG = DP <= 128;
    constexpr int KS = DP / 16;
    uint32_t qf[QREG ? KS : 1][4];
    const int q_r = ((lane >> 3) & 1) * 8 + (lane & 7), q_c = lane >> 4;
    if (QREG) {
#pragma unroll
        for (int k = 0; k < KS; ++k) ldsm4(q0 + v_piece<2 * DP>(q_r, 2 * k + q_c), qf[k]);
    }
    float o[DP / 8][4];
    float mx[2], l[2];
    mx[0] = mx[1] = neg_inf();
    l[0] = l[1] = 0.0f;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;

    const int g = lane >> 2, t4 = lane & 3;
    for (int j = 0; j < tiles; ++j) {
        cp_wait<S::STAGES - 2>();
        const int tile0 = t.begin + j * TN;
        const bool tail = tile0 + TN > t.base;  // holds new tokens: some queries see it in part
        unsigned char* stage = smem + (j % S::STAGES) * S::STAGE;
        if (tail) {
            // A value that is not finite must not reach queries that do not see it, and a
            // probability of 0 does not hide it from a product: it is taken out here (by the
            // thread that copied it) and put back at the end for the queries that do.
            bool bad = false;
            for (int x = 0; x < TN * S::CH / S::THREADS; ++x) {
                const int f = tid + x * S::THREADS;
                uint4* p = reinterpret_cast<uint4*>(stage + S::MAT + v_piece<S::PITCH>(f / S::CH, f % S::CH));
                uint4 v = *p;
                if (sv::sanitise<E4M3>(v)) {
                    *p = v;
                    bad = true;
                }
            }
            if (E4M3 && tid >= TN && tid < 2 * TN) {
                float* p = reinterpret_cast<float*>(stage + 2 * S::MAT) + tid;
                if (sv::not_finite(*p)) { *p = 0.0f; bad = true; }
            }
            if (bad) s_bad = 1;
        }
        __syncthreads();  // tile j is whole; tile j - 1 is no longer read
        if (j + S::STAGES - 1 < tiles) load_tile(j + S::STAGES - 1);
        cp_commit();
        if (tid < TN) {
            put_place(j + S::STAGES, tid, next_row, next_page);
            const int pos = t.begin + (j + S::STAGES + 1) * TN + tid;
            next_page = -1;
            if (pos < t.end) next_page = sv::paged_place(a.c, t.b, pos, next_row);
        }
        const uint32_t valid = (s_valid[j % RING][wk >> 1] >> (16 * (wk & 1))) & 0xffffu;
        const uint32_t ks0 = smem_u32(stage), vs0 = ks0 + S::MAT;
        const float* k_sc = reinterpret_cast<const float*>(stage + 2 * S::MAT);

        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
        if (!E4M3) {
            const int kr = wk * 16 + (lane >> 4) * 8 + (lane & 7), kc = (lane >> 3) & 1;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t b[4];
                ldsm4(ks0 + v_piece<S::PITCH>(kr, 2 * k + kc), b);
                mma16816(s[0], qf[QREG ? k : 0], b[0], b[1]);
                mma16816(s[1], qf[QREG ? k : 0], b[2], b[3]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < DP / 64; ++e) {
                uint4 w[2];
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    w[n] = *reinterpret_cast<const uint4*>(stage + k_piece<S::PITCH>(wk * 16 + n * 8 + g, 4 * e + t4));
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int k = 4 * e + u;
                    uint32_t b[4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const uint32_t x = u == 0 ? w[n].x : u == 1 ? w[n].y : u == 2 ? w[n].z : w[n].w;
                        b[2 * n] = widen(x & 0xffffu);
                        b[2 * n + 1] = widen(x >> 16);
                    }
                    uint32_t qa[4];
                    if (!QREG) ldsm4(q0 + v_piece<2 * DP>(q_r, 2 * k + q_c), qa);
                    const uint32_t* q = QREG ? qf[QREG ? k : 0] : qa;
                    mma16816(s[0], q, b[0], b[1]);
                    mma16816(s[1], q, b[2], b[3]);
                }
            }
        }
        float ksc[2][2], vsc[2][2];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int p = wk * 16 + n * 8 + 2 * t4 + z;
                ksc[n][z] = E4M3 ? k_sc[p] * a.scale_log2 : a.scale_log2;
                vsc[n][z] = E4M3 ? k_sc[TN + p] : 1.0f;
            }
        uint32_t pf[4];
        uint32_t see[2] = {valid, valid};
        if (tail) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int R = t.mt * S::ROWS + g + 8 * y;
                see[y] &= R < t.n * a.group ? sv::attn_visible(a, t, R / a.group, tile0 + wk * 16) : 0u;
            }
        }
        float top[2] = {neg_inf(), neg_inf()};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float v = s[n][x] * ksc[n][x & 1];
                if (!((see[x >> 1] >> (n * 8 + 2 * t4 + (x & 1))) & 1u)) v = neg_inf();
                s[n][x] = v;
                top[x >> 1] = fmaxf(top[x >> 1], v);
            }
        float shift[2], fac[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            top[y] = fmaxf(top[y], __shfl_xor_sync(0xffffffffu, top[y], 1));
            top[y] = fmaxf(top[y], __shfl_xor_sync(0xffffffffu, top[y], 2));
            const float now = fmaxf(mx[y], top[y]);
            shift[y] = now == neg_inf() ? 0.0f : now;
            fac[y] = sv::ex2(mx[y] - shift[y]);  // 0 while the row has seen nothing
            mx[y] = now;
        }
        if (__any_sync(0xffffffffu, fac[0] != 1.0f || fac[1] != 1.0f)) {
            l[0] *= fac[0];
            l[1] *= fac[1];
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) {
                o[n][0] *= fac[0];
                o[n][1] *= fac[0];
                o[n][2] *= fac[1];
                o[n][3] *= fac[1];
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float p[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                p[x] = sv::ex2(s[n][x] - shift[x >> 1]);
                l[x >> 1] += p[x];
                if (E4M3) p[x] *= vsc[n][x & 1];
            }
            pf[2 * n] = sv::bf16x2(p[0], p[1]);
            pf[2 * n + 1] = sv::bf16x2(p[2], p[3]);
        }
        if (!E4M3) {
            const int vr = wk * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), vc = lane >> 4;
#pragma unroll
            for (int n = 0; n < DP / 16; ++n) {
                uint32_t b[4];
                ldsm4t(vs0 + v_piece<S::PITCH>(vr, 2 * n + vc), b);
                mma16816(o[2 * n], pf, b[0], b[1]);
                mma16816(o[2 * n + 1], pf, b[2], b[3]);
            }
        } else {
            const int vr = wk * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), vc = lane >> 4;
#pragma unroll
            for (int n = 0; n < DP / 32; ++n) {
                uint32_t b[4];  // positions 0-7 and 8-15 of 16 elements, then of the next 16
                ldsm4t(vs0 + v_piece<S::PITCH>(vr, 2 * n + vc), b);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const uint32_t lo = __byte_perm(b[2 * z], 0u, 0x3120), hi = __byte_perm(b[2 * z + 1], 0u, 0x3120);
                    const uint32_t e0 = widen(lo & 0xffffu), e1 = widen(hi & 0xffffu);
                    const uint32_t f0 = widen(lo >> 16), f1 = widen(hi >> 16);
                    mma16816(o[4 * n + 2 * z], pf, e0, e1);      // even elements
                    mma16816(o[4 * n + 2 * z + 1], pf, f0, f1);  // odd elements
                }
            }
        }
    }

    // ---- the four warps of a row tile join
    cp_wait<0>();
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
        l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
        const int r = g + 8 * y;
        if (t4 == 0) {
            s_m[wk][r] = mx[y];
            s_l[wk][r] = l[y];
        }
    }
    __syncthreads();
    float inv[2], lse2[2];
    bool none[2];  // no weight at all: zero, whatever the values hold
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int r = g + 8 * y;
        float top = s_m[0][r];
#pragma unroll
        for (int w = 1; w < KW; ++w) top = fmaxf(top, s_m[w][r]);
        const float shift = top == neg_inf() ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w) sum += s_l[w][r] * sv::ex2(s_m[w][r] - shift);
        const float fac = sv::ex2(mx[y] - shift);
        inv[y] = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;  // NaN stays
        lse2[y] = sum == 0.0f ? neg_inf() : shift + log2f(sum);
        none[y] = sum == 0.0f && t.parts <= 1;
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) {
            o[n][2 * y] *= fac;
            o[n][2 * y + 1] *= fac;
        }
    }
    float4* join = reinterpret_cast<float4*>(smem) + lane;
#pragma unroll
    for (int half = 2; half >= 1; half >>= 1) {
        if (wk >= half && wk < 2 * half) {
            float4* to = join + (size_t)(wk - half) * (DP / 8) * 32;
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
                to[n * 32] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
        }
        __syncthreads();
        if (wk < half) {
            const float4* from = join + (size_t)wk * (DP / 8) * 32;
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) {
                const float4 v = from[n * 32];
                o[n][0] += v.x;
                o[n][1] += v.y;
                o[n][2] += v.z;
                o[n][3] += v.w;
            }
        }
        __syncthreads();
    }
    if (wk != 0) return;

#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int R = t.mt * S::ROWS + g + 8 * y;
        if (R >= t.n * a.group) continue;
        const int64_t row = sv::attn_row(a, t, R);
        const int64_t part = t.part + R - t.mt * S::ROWS;
        if (t4 == 0) {
            if (t.parts > 1) a.part_lse[part] = lse2[y];
            else if (a.lse) a.lse[row] = lse2[y] * 0.69314718055994531f;
        }
        // a thread's elements of each 16: bf16 pages 2 t4, 2 t4 + 1 and 8 more; e4m3 4 t4 .. 4 t4 + 3
#pragma unroll
        for (int n = 0; n < DP / 16; ++n) {
            float v[4];
            int d[2];
            if (!E4M3) {
                d[0] = 16 * n + 2 * t4;
                d[1] = d[0] + 8;
                v[0] = o[2 * n][2 * y]; v[1] = o[2 * n][2 * y + 1];
                v[2] = o[2 * n + 1][2 * y]; v[3] = o[2 * n + 1][2 * y + 1];
            } else {
                d[0] = 16 * n + 4 * t4;
                d[1] = d[0] + 2;
                v[0] = o[2 * n][2 * y]; v[1] = o[2 * n + 1][2 * y];
                v[2] = o[2 * n][2 * y + 1]; v[3] = o[2 * n + 1][2 * y + 1];
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] = none[y] ? 0.0f : v[x] * inv[y];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                if (d[z] >= D) continue;
                if (s_bad && !none[y]) {
                    const int from = t.begin + (t.base > t.begin ? (t.base - t.begin) / TN * TN : 0);
                    for (int pos = from; pos < t.end; ++pos) {
                        if (!(sv::attn_visible(a, t, R / a.group, pos) & 1u)) continue;
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float w = sv::attn_value<E4M3>(a, t, pos, d[z] + x);
                            if (sv::not_finite(w)) v[2 * z + x] += w;
                        }
                    }
                }
                if (t.parts > 1)
                    *reinterpret_cast<float2*>(a.part_o + part * D + d[z]) = make_float2(v[2 * z], v[2 * z + 1]);
                else
                    *reinterpret_cast<uint32_t*>(a.out + row * D + d[z]) = sv::bf16x2(v[2 * z], v[2 * z + 1]);
            }
        }
    }
}

// Joins the splits of a row: weights 2^(lse_s - max), one warp per row of the split tiles.
__global__ void __launch_bounds__(256) paged_attention_join_kernel(const __grid_constant__ AttnArgs a, int pairs,
                                                                   int tile_rows, int64_t rows) {
    const int part_rows = a.part_rows;
    pdl_trigger();
    pdl_wait();
    const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (at >= rows) return;
    const int rest = (int)(at / part_rows), r = (int)(at - (int64_t)rest * part_rows);
    const sv::AttnPlace p = sv::attn_place(a, pairs, (unsigned)(a.whole + rest));
    int base, n;
    if (!sv::paged_row(a.c, a.base, a.new_len, p.b, a.Q, base, n)) return;
    const int64_t R = (int64_t)p.mt * tile_rows + r;
    if (R >= (int64_t)n * a.group) return;
    const int parts = sv::attn_parts(a, sv::attn_active(a, sv::attn_tile_end(base, n, a.group, p.mt, tile_rows, a.tree_mask != nullptr)));
    if (parts <= 1) return;  // written by the one CTA that had the row
    const int64_t row = ((int64_t)p.b * a.Q + R / a.group) * a.Hq + p.h * a.group + R % a.group;
    const int64_t part = (int64_t)rest * (a.splits / a.per) * part_rows + r;  // the first; the next ones part_rows apart
    const int D = a.c.dim;
    const float* lse = a.part_lse + part;
    float top = neg_inf();
    for (int s = lane; s < parts; s += 32) top = fmaxf(top, lse[(int64_t)s * part_rows]);
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float shift = top == neg_inf() ? 0.0f : top;
    float sum = 0.0f;
    for (int s = lane; s < parts; s += 32) sum += sv::ex2(lse[(int64_t)s * part_rows] - shift);
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    for (int d = 4 * lane; d < D; d += 128) {
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float* from = a.part_o + part * D + d;
#pragma unroll 4
        for (int s = 0; s < parts; ++s) {
            const float w = sv::ex2(lse[(int64_t)s * part_rows] - shift) * inv;
            const float4 v = *reinterpret_cast<const float4*>(from + (int64_t)s * part_rows * D);
            acc.x += w * v.x;
            acc.y += w * v.y;
            acc.z += w * v.z;
            acc.w += w * v.w;
        }
        if (sum == 0.0f) acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // no weight at all, whatever the values hold
        *reinterpret_cast<uint2*>(a.out + row * D + d) =
            make_uint2(sv::bf16x2(acc.x, acc.y), sv::bf16x2(acc.z, acc.w));
    }
    if (a.lse && lane == 0) a.lse[row] = sum == 0.0f ? neg_inf() : (shift + log2f(sum)) * 0.69314718055994531f;
}

template <int DP, bool E4M3>
cudaError_t launch_few(const AttnArgs& a, int pairs, unsigned ctas, cudaStream_t stream) {
    using S = Shape<DP, E4M3>;
    static sv::KernelLaunchCache cache;
    auto kern = paged_attention_kernel<DP, E4M3>;
    int max_dyn = 0;
    const cudaError_t e = cache.setup((const void*)kern, &max_dyn);
    if (e != cudaSuccess) return e;
    if (S::SMEM > max_dyn) return cudaErrorInvalidValue;
    return sv::launch_serial(kern, dim3(ctas), dim3(S::THREADS), S::SMEM, stream, a, pairs);
}

constexpr int kMaxB = 65535;
constexpr int kMaxQ = 65536;

struct Plan {
    int tile_rows, m_tiles, splits, chunk, per, part_rows;
    int64_t tiles, whole, ctas;
    bool dual;  // a CTA takes two splits (per: how many), and joins them
    size_t ws;  // of partial results: none where each row tile is one CTA's
};

// How a call is cut: tiles of query rows, and stretches of positions where there are too
// few tiles to fill the SMs.
Plan make_plan(int B, int Q, int Hq, int H, int D, bool e4m3, int max_len, int num_sms) {
    Plan p{};
    if (max_len > sv::PAGED_MAX_POS) max_len = sv::PAGED_MAX_POS;
    const int64_t rows = (int64_t)Q * (Hq / H);
    // One GB300, 32 over 8 heads, mma.sync against tcgen05, us.  Wide heads (256), 4 and 16 rows:
    //   bf16: 64 contexts of 4096 464 and 381, 746 and 384; one of 8000 79 and 46, 150 and 46; of 700 25 and
    //     31, 49 and 31: tcgen05 throughout, though a short context of 4 rows gives away a fifth;
    //   e4m3: 64 of 4096 450 and 798, 744 and 800; 16 of 4096 169 and 258, 271 and 261; one of 8000 81
    //     and 58, 152 and 59; of 700 27 and 48, 51 and 49: mma.sync up to 16 rows, for the batches of 4
    //     rows; one or two long contexts, and 16 rows of few, would be faster on tcgen05.
    if (D > 128) p.tile_rows = e4m3 && rows <= 16 ? 16 : 128;
    else if (rows > 128) p.tile_rows = 256;
    // Sixteen rows or fewer waste most of a 128-row product, and e4m3 its widening besides; a few long
    // contexts leave the mma.sync kernel's copies too little in flight.  Heads of 128, 4 rows:
    //   bf16: 64 contexts of 4096 206 and 204, 16 of 4096 83 and 86, 8 of 32768 224 and 196, 8 of 8000 79
    //     and 85, 4 of 8000 49 and 61; one of 2000 19 and 23, of 8000 38 and 29, of 131072 128 and 113:
    //     tcgen05 for long contexts of no more cache heads than SMs (two to eight contexts lose up to
    //     a quarter or win up to an eighth by it, one wins a tenth to a quarter, with 16 rows more);
    //   e4m3: 64 of 4096 190 and 292; one of 2000 20 and 29, of 8000 39 and 31, of 32768 54 and 54, of
    //     131072 117 and 129: mma.sync, which loses a fifth at one context of about 8000 only.
    // 17 rows and more: 64 x 300 x 24 rows 105 and 49.
    else if (rows > 16 || (!e4m3 && max_len >= 4096 && (int64_t)B * H <= num_sms)) p.tile_rows = 128;
    else p.tile_rows = 16;
    p.m_tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
    p.tiles = (int64_t)B * H * p.m_tiles;
    const bool large = p.tile_rows >= 128;  // one such CTA fills an SM
    const int tn = large ? 128 : TN;        // positions per tile of the kernel taken
    // Enough CTAs that rows of unequal length even out: four per SM.  Large tiles: three per
    // SM where there are fewer tiles than SMs; else whole waves of tiles, and what is left
    // over split so that it fills the last wave.
    p.dual = p.tile_rows == 128 && D <= 128 && max_len >= 512;
    int64_t splits, least = 128;  // positions worth a split
    if (p.dual) {
        least = 256;
        splits = 2 * ((B == 1 ? 1LL : 3LL) * num_sms / p.tiles);
        if (splits < 2) splits = 2;
    } else if (!large) {
        splits = (4LL * num_sms + p.tiles - 1) / p.tiles;
    } else if (p.tiles < num_sms) {
        least = D > 128 ? 512 : 1024;
        splits = 3LL * num_sms / p.tiles;
    } else {
        least = D > 128 ? 512 : 1024;
        p.whole = p.tiles / num_sms * num_sms;
        splits = p.tiles > p.whole ? num_sms / (p.tiles - p.whole) : 1;
    }
    if (splits > ((int64_t)max_len + least - 1) / least) splits = ((int64_t)max_len + least - 1) / least;
    if (splits > 256) splits = 256;
    if (splits < 1) splits = 1;
    p.chunk = (int)((((int64_t)max_len + splits - 1) / splits + tn - 1) / tn * tn);
    p.splits = (int)(((int64_t)max_len + p.chunk - 1) / p.chunk);
    if (p.dual) p.splits += p.splits & 1;
    if (p.splits <= 1) p.whole = p.tiles;
    p.per = p.dual ? 2 : 1;
    const int64_t parts = (p.tiles - p.whole) * p.splits / p.per;
    p.ctas = p.whole + parts;
    p.part_rows = p.m_tiles == 1 ? (int)rows : p.tile_rows;
    p.ws = p.splits > p.per ? (size_t)parts * p.part_rows * (D + 1) * sizeof(float) : 0;
    return p;
}

bool sizes_ok(int B, int Q, int Hq, int H, int D, int max_len) {
    return B >= 0 && B <= kMaxB && Q >= 1 && Q <= kMaxQ && H >= 1 && H <= sv::PAGED_MAX_HEADS && Hq >= H &&
           Hq <= 65536 && Hq % H == 0 && D >= 1 && D <= sv::PAGED_MAX_DIM && max_len >= 1 &&
           (int64_t)Q * (Hq / H) < ((int64_t)1 << 30);
}

// Test hook for the time-out path (SPEC_VERIFY_TEST_STALL_ATTENTION=<batch row>): the tcgen05
// kernel's CTAs of that row never report one tile's notes, so the waits for it run out and the
// row is written as NaN.  Read once; unset, nothing changes.
int test_stall_row() {
    static const int row = [] {
        const char* s = std::getenv("SPEC_VERIFY_TEST_STALL_ATTENTION");
        return s && *s ? std::atoi(s) : -1;
    }();
    return row;
}

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return sms;
}

}  // namespace

extern "C" {

size_t spec_paged_attention_workspace_size(int B, int Q, int num_q_heads, int num_heads, int head_dim,
                                           sv_cache_dtype dtype, int max_len) {
    if (!sizes_ok(B, Q, num_q_heads, num_heads, head_dim, max_len) || B == 0) return 0;
    if (dtype != SV_CACHE_BF16 && dtype != SV_CACHE_E4M3) return 0;
    const int sms = sm_count();
    return sms ? make_plan(B, Q, num_q_heads, num_heads, head_dim, dtype == SV_CACHE_E4M3, max_len, sms).ws : 0;
}

sv_status spec_paged_attention(const void* q, const int64_t* q_stride, int num_q_heads, const sv_paged_cache* cache,
                               const int32_t* base, const int32_t* new_len, const uint32_t* tree_mask, float scale,
                               int B, int Q, int max_len, void* out, float* out_lse, void* workspace, size_t ws_bytes,
                               void* stream) {
    AttnArgs a{};
    if (!sv::paged_cache_args(cache, a.c) ||
        !sizes_ok(B, Q, num_q_heads, cache->num_heads, cache->head_dim, max_len))
        return SV_ERR_INVALID_ARG;
    if (!(scale - scale == 0.0f)) return SV_ERR_INVALID_ARG;  // NaN or infinite
    if (B == 0) return SV_OK;
    if (!cache->page_table || !q || !q_stride || !base || !out) return SV_ERR_INVALID_ARG;
    const int D = cache->head_dim;
    if (D % 8 || ((uintptr_t)q | (uintptr_t)cache->k_pages | (uintptr_t)cache->v_pages | (uintptr_t)out) % 16 ||
        (cache->page_stride | cache->head_stride | cache->row_stride) % 16 ||
        (q_stride[0] | q_stride[1] | q_stride[2]) % 8)
        return SV_ERR_UNSUPPORTED;
    const int sms = sm_count();
    if (!sms) return sv::launch_status(cudaErrorInvalidDevice);
    Plan p = make_plan(B, Q, num_q_heads, cache->num_heads, D, cache->dtype == SV_CACHE_E4M3, max_len, sms);
    if (p.ws && (!workspace || ws_bytes < p.ws || (uintptr_t)workspace % 16)) {
        p.whole = p.ctas = p.tiles;
        p.splits = 1;
        p.chunk = sv::PAGED_MAX_POS;
        p.dual = false;
        p.per = 1;
        p.ws = 0;
    }
    if (p.ctas >= ((int64_t)1 << 31)) return SV_ERR_UNSUPPORTED;
    a.q = static_cast<const uint16_t*>(q);
    a.q_sb = q_stride[0];
    a.q_st = q_stride[1];
    a.q_sh = q_stride[2];
    a.base = base;
    a.new_len = new_len;
    a.tree_mask = Q > 1 ? tree_mask : nullptr;
    a.scale_log2 = scale * sv::LOG2E;
    a.Q = Q;
    a.Hq = num_q_heads;
    a.group = num_q_heads / cache->num_heads;
    a.mask_words = (Q - 1 + 31) / 32;
    a.m_tiles = p.m_tiles;
    a.whole = (int)p.whole;
    a.splits = p.splits;
    a.per = p.per;
    a.part_rows = p.part_rows;
    a.equal = p.tile_rows >= 128;
    a.sort = a.equal && B > 1 && B <= 32 && p.whole == 0 && p.ctas > sms ? B : 0;
    a.chunk = p.chunk;
    a.stall_row = test_stall_row();
    a.out = static_cast<uint16_t*>(out);
    a.lse = out_lse;
    const int64_t rows = p.ws ? (p.tiles - p.whole) * p.part_rows : 0;  // of the split tiles
    a.part_o = static_cast<float*>(workspace);
    a.part_lse = p.ws ? a.part_o + rows * (p.splits / p.per) * D : nullptr;
    cudaStream_t s = (cudaStream_t)stream;
    const bool e4m3 = cache->dtype == SV_CACHE_E4M3;
    const int pairs = B * cache->num_heads;
    const unsigned ctas = (unsigned)p.ctas;
    cudaError_t e;
    if (p.tile_rows >= 128) e = sv::launch_attn_tc(a, pairs, e4m3, p.tile_rows, p.dual, ctas, s);
    else if (D <= 64) e = e4m3 ? launch_few<64, true>(a, pairs, ctas, s) : launch_few<64, false>(a, pairs, ctas, s);
    else if (D <= 128) e = e4m3 ? launch_few<128, true>(a, pairs, ctas, s) : launch_few<128, false>(a, pairs, ctas, s);
    else e = launch_few<256, true>(a, pairs, ctas, s);
    if (e == cudaSuccess && rows)
        e = sv::launch_serial(paged_attention_join_kernel, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, a, pairs,
                              p.tile_rows, rows);
    return sv::launch_status(e);
}

}  // extern "C"
