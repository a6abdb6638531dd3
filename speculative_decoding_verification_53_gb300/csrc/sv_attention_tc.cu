// sv_attention_tc.cu -- paged attention for many query rows per cache head (trees, chunks
// of prompts) on the 5th-generation tensor cores (include/spec_paged_kv.h).
//
// A CTA holds MQ tiles of 128 query rows and walks the positions in tiles of 128.  Per
// tile and row tile: S = Q K^T into TMEM (tcgen05.mma, Q and K in 128-byte-swizzled shared
// memory), the softmax warps read their rows of S, write the probabilities P as bf16 over
// S, and O += P V accumulates in TMEM with P read from TMEM and V from shared memory in
// its stored order (positions x elements, "MN-major").  Roles:
//   warps 0 .. 4 MQ - 1   softmax, one thread per query row, one warpgroup per row tile
//   the next four warps   producers: keys and values into a ring of NB shared buffers
//   the last four         one thread issues every tcgen05.mma (a whole warpgroup gives its registers up)
// While one row tile's softmax runs, the tensor cores work on the other's products.
// Dependences: full/empty barriers per buffer; s_full (S is in TMEM, and so is the last
// O, since a commit covers every earlier product); p_full (P is written, O rescaled).
//
// The running maximum is moved only when it grows by more than 2^8: probabilities may
// then reach 256 instead of 1, harmless in fp32 sums and bf16's range, and the rescale of
// O in TMEM becomes rare.
//
// Every wait is bounded; a CTA whose wait runs out writes NaN for its rows, which a verify
// reports as invalid data, and frees its TMEM.
#include <cstdint>

#include "spec_paged_kv.h"
#include "sv_attention.cuh"

namespace {

using sv::AttnArgs;
using sv::AttnTile;
using sv::fence_proxy_async;
using sv::ffma2;
using sv::fmul2;
using sv::mbar_init;
using sv::mbar_wait_bounded;
using sv::neg_inf;
using sv::pdl_trigger;
using sv::pdl_wait;
using sv::smem_u32;

constexpr int TN = 128;          // positions per tile
constexpr int BLK = 128 * 128;   // bytes of 128 rows x 64 bf16 elements, 128-byte swizzled
constexpr int META = 4;          // tiles whose hole bits and scales are kept
constexpr float RESCALE = 8.0f;  // log2 of how far the maximum may lag

template <int DP, int MQ, bool E4M3>
struct Tc {
    static constexpr int ROWS = 128 * MQ;
    static constexpr int SOFTMAX = 128 * MQ;
    static constexpr int THREADS = SOFTMAX + 256;  // whole warpgroups, as setmaxnreg wants
    // Registers: the launch gives every thread 65536 / THREADS; softmax threads hold a row of
    // 128 scores and take what the others give back.
    //   MQ = 2: 512 x 128 = 65536 >= 256 x 184 + 128 x 96 + 128 x 40 = 64512
    //   MQ = 1: 384 x 168 = 64512 >= 128 x 216 + 128 x 136 + 128 x 40 = 50176
    static constexpr int R_SOFTMAX = MQ == 2 ? 184 : 216, R_LOAD = MQ == 2 ? 96 : 136, R_MMA = 40;
    static constexpr int MAT = (DP / 64) * BLK;   // a tile of keys, values or queries
    static constexpr int NB = DP == 64 ? 6 : E4M3 ? 3 : 4;   // buffers of the ring
    static constexpr int RAW = E4M3 ? 3 : 0;      // e4m3: items whose codes are in flight
    static constexpr int SMEM = (MQ + NB) * MAT + RAW * MAT / 2 + 1024;  // and room to align
    static constexpr int S_COL = 0, O_COL = 128 * MQ;    // TMEM columns
    static constexpr int COLS = MQ == 2 ? 512 : 256;
};

// ------------------------------------------------------------ tcgen05 wrappers

__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
// One lane of a converged warp, the same one for every call.  The products' warp runs its
// loop with all lanes, so that addresses and descriptors are uniform, and only this lane
// issues: with one lane alone in the loop each product cost 130 cycles to issue instead of 64.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}
__device__ __forceinline__ void tc_commit(uint64_t* bar, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(leader)
        : "memory");
}
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(leader)
        : "memory");
}

#define SV_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define SV_W8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])

// 32 columns of this warp's 32 lanes; the registers hold them after tc_wait_ld().
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t v[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : SV_R8(v, 0), SV_R8(v, 8), SV_R8(v, 16), SV_R8(v, 24)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t v[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : SV_R8(v, 0), SV_R8(v, 8)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t v[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            addr),
        SV_W8(v, 0), SV_W8(v, 8)
        : "memory");
}

// Shared-memory operand: start, leading and stride byte offsets, 128-byte swizzle.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead, uint32_t stride) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// fp32 accumulator, bf16 operands, 128 rows, n columns; b_mn: B is stored along n.
__host__ __device__ constexpr uint32_t instruction(int n, bool b_mn) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 16-byte piece c (of 8 elements) of row r in a tile of 64-element blocks.
__device__ __forceinline__ uint32_t piece(int r, int c) {
    return (uint32_t)((c >> 3) * BLK + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// An arrival on `bar` (counted among its expected ones) once this thread's copies have landed.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Sixteen e4m3 codes to bf16 (exact), as two 16-byte pieces.
__device__ __forceinline__ void widen16(uint4 w, uint4& a, uint4& b) {
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 lo = sv::e4m3x2_to_f32(in[i] & 0xffffu), hi = sv::e4m3x2_to_f32(in[i] >> 16);
        out[2 * i] = sv::bf16x2(lo.x, lo.y);
        out[2 * i + 1] = sv::bf16x2(hi.x, hi.y);
    }
    a = make_uint4(out[0], out[1], out[2], out[3]);
    b = make_uint4(out[4], out[5], out[6], out[7]);
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

// Scores of a row, scaled in place (e4m3: by the keys' scales too), -inf where hidden.
template <bool E4M3, bool MASK>
__device__ __forceinline__ void scale_scores(uint32_t v[TN], const uint32_t see[4], const float* ksc, float sc) {
#pragma unroll
    for (int k = 0; k < TN; k += 4) {
        const float4 w = E4M3 ? *reinterpret_cast<const float4*>(ksc + k) : make_float4(sc, sc, sc, sc);
        float2 f[2] = {make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])),
                       make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]))};
        f[0] = fmul2(f[0], make_float2(w.x, w.y));
        f[1] = fmul2(f[1], make_float2(w.z, w.w));
        const float g[4] = {f[0].x, f[0].y, f[1].x, f[1].y};
#pragma unroll
        for (int z = 0; z < 4; ++z)
            v[k + z] = __float_as_uint(!MASK || ((see[k >> 5] >> ((k & 31) + z)) & 1u) ? g[z] : neg_inf());
    }
}

__device__ __forceinline__ float largest(const uint32_t v[TN]) {
    float t[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
    for (int k = 0; k < TN; ++k) t[k & 3] = fmaxf(t[k & 3], __uint_as_float(v[k]));
    return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

struct __align__(16) Shared {
    uint64_t full[8], empty[8], s_full[2], p_full[2], o_full[2], drain;
    uint32_t tmem;
    int bad, failed;
    uint32_t valid[META][4];       // which of the tile's positions hold something
    __align__(16) float ksc[META][TN];  // e4m3: key scale times the score factor
    __align__(16) float vsc[META][TN];  // value scale
};

template <int DP, int MQ, bool E4M3>
__global__ void __launch_bounds__(MQ * 128 + 256, 1) paged_attention_tc_kernel(const __grid_constant__ AttnArgs a) {
    using S = Tc<DP, MQ, E4M3>;
    extern __shared__ unsigned char raw[];
    __shared__ Shared sh;
    pdl_trigger();
    pdl_wait();
    AttnTile t;
    if (!sv::attn_tile(a, blockIdx.x, S::ROWS, t)) return;
    const uint32_t smem0 = (smem_u32(raw) + 1023u) & ~1023u;  // queries, then the ring
    unsigned char* gen = raw + (smem0 - smem_u32(raw));       // the same place, generic
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = a.c.dim, rows = t.n * a.group;
    const int tiles = (t.end - t.begin + TN - 1) / TN;
    // Positions below this are seen by every query of the CTA.
    const int open = a.tree_mask ? t.base + 1 : t.base + t.mt * S::ROWS / a.group + 1;

    if (warp == 0) tmem_alloc(&sh.tmem, S::COLS);
    if (tid == 0) {
        for (int i = 0; i < S::NB; ++i) {
            mbar_init(&sh.full[i], E4M3 ? 4 : 128);  // warps, or threads, that fill a buffer
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < MQ; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 4);
            mbar_init(&sh.o_full[i], 1);
        }
        mbar_init(&sh.drain, 1);
        sh.bad = 0;
        sh.failed = 0;
        sv::fence_mbar_init();
    }
    // the queries, zero behind the last real one
    for (int f = tid; f < S::ROWS * (DP / 8); f += S::THREADS) {
        const int r = f / (DP / 8), c = f % (DP / 8), R = t.mt * S::ROWS + r;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (R < rows && 8 * c < D)
            w = sv::ld_nc_v4(a.q + t.b * a.q_sb + (int64_t)(R / a.group) * a.q_st +
                             (int64_t)(t.h * a.group + R % a.group) * a.q_sh + 8 * c);
        *reinterpret_cast<uint4*>(gen + (r >> 7) * S::MAT + piece(r & 127, c)) = w;
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const uint32_t ring = smem0 + MQ * S::MAT;
    bool ok = true;

    if (warp < 4 * MQ) {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::R_SOFTMAX));
        const int q = warp >> 2;
        const int R = t.mt * S::ROWS + q * 128 + (warp & 3) * 32 + lane;
        const bool live = R < rows;
        const int i = live ? R / a.group : 0;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 lanes per warp, lane field at bit 16
        const uint32_t s_at = tmem + lanes + S::S_COL + 128 * q, o_at = tmem + lanes + S::O_COL + DP * q;
        const float sc = a.scale_log2;
        float mx = neg_inf(), l = 0.0f;
        for (int j = 0; j < tiles; ++j) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.s_full[q], j & 1));
            if (!ok) break;
            tc_fence_after();
            const int tile0 = t.begin + j * TN, m = j % META;
            uint32_t see[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) see[c] = sh.valid[m][c];
            const bool whole = tile0 + TN <= open && (see[0] & see[1] & see[2] & see[3]) == 0xffffffffu;
            if (tile0 + TN > open) {
#pragma unroll
                for (int c = 0; c < 4; ++c) see[c] &= live ? sv::attn_visible(a, t, i, tile0 + 32 * c) : 0u;
            }
            uint32_t v[TN];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, v + 32 * c);
            tc_wait_ld();
            float top, mul = 1.0f;
            if (!E4M3 && whole && sc >= 0.0f) {
                top = largest(v) * sc;  // the factor joins the exponent's product below
                mul = sc;
            } else {
                if (whole) scale_scores<E4M3, false>(v, see, sh.ksc[m], sc);
                else scale_scores<E4M3, true>(v, see, sh.ksc[m], sc);
                top = largest(v);
            }
            // move the maximum where it grew too far
            float fac = 1.0f;
            if (top > mx + RESCALE || mx == neg_inf()) {
                const float now = fmaxf(top, mx);
                fac = now == neg_inf() ? 1.0f : sv::ex2(mx - now);
                mx = now;
                l *= fac;
            }
            if (j > 0 && __any_sync(0xffffffffu, fac != 1.0f)) {
#pragma unroll 1
                for (int c = 0; c < DP / 16; ++c) {
                    uint32_t o[16];
                    tmem_ld16(o_at + 16 * c, o);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fac);
                    tmem_st16(o_at + 16 * c, o);
                }
            }
            const float shift = mx == neg_inf() ? 0.0f : mx;
            const float2 mul2 = make_float2(mul, mul), sh2 = make_float2(-shift, -shift);
            float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t p[16];
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const uint32_t* x = v + 32 * c + k;
                    float2 e = ffma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), mul2, sh2);
                    float2 f = ffma2(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), mul2, sh2);
                    e = make_float2(sv::ex2(e.x), sv::ex2(e.y));
                    f = make_float2(sv::ex2(f.x), sv::ex2(f.y));
                    sum0 = sv::fadd2(sum0, e);
                    sum1 = sv::fadd2(sum1, f);
                    if (E4M3) {
                        const float4 w = *reinterpret_cast<const float4*>(&sh.vsc[m][32 * c + k]);
                        e = fmul2(e, make_float2(w.x, w.y));
                        f = fmul2(f, make_float2(w.z, w.w));
                    }
                    p[k >> 1] = sv::bf16x2(e.x, e.y);
                    p[(k >> 1) + 1] = sv::bf16x2(f.x, f.y);
                }
                tmem_st16(s_at + 16 * c, p);  // over S, which this warp has read
            }
            sum0 = sv::fadd2(sum0, sum1);
            l += sum0.x + sum0.y;
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[q]);
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.o_full[q], 0));
        if (!ok) sh.failed = 1;
        tc_fence_after();
        const float inv = !ok ? __int_as_float(0x7fffffff) : l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
        const float lse2 = !ok ? inv : l == 0.0f ? neg_inf() : mx + log2f(l);
        const int64_t row = live ? sv::attn_row(a, t, R) : 0, part = row * a.splits + t.split;
        if (live) {
            if (t.active > 1) a.part_lse[part] = lse2;
            else if (a.lse) a.lse[row] = lse2 * 0.69314718055994531f;
        }
        const bool patch = ok && sh.bad != 0;
        for (int c = 0; c < DP / 32; ++c) {
            uint32_t v[32];
            __syncwarp();
            tmem_ld32(o_at + 32 * c, v);
            tc_wait_ld();
            if (live && patch) {
                // values that are not finite, for the queries that see them
                int from = t.begin;
                if (open > t.begin) from += (open - t.begin) / TN * TN;
                for (int pos = from; pos < t.end; ++pos) {
                    if (!(sv::attn_visible(a, t, i, pos) & 1u)) continue;
                    for (int k = 0; k < 32 && 32 * c + k < D; ++k) {
                        const float w = sv::attn_value<E4M3>(a, t, pos, 32 * c + k);
                        if (sv::not_finite(w)) {
#pragma unroll
                            for (int z = 0; z < 32; ++z)
                                if (z == k) v[z] = __float_as_uint(__uint_as_float(v[z]) + w);
                        }
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
                if (!live || 32 * c + k >= D) break;
                float f[8];
#pragma unroll
                for (int z = 0; z < 8; ++z) f[z] = __uint_as_float(v[k + z]) * inv;
                if (t.active > 1) {
                    float4* to = reinterpret_cast<float4*>(a.part_o + part * D + 32 * c + k);
                    to[0] = make_float4(f[0], f[1], f[2], f[3]);
                    to[1] = make_float4(f[4], f[5], f[6], f[7]);
                } else {
                    *reinterpret_cast<uint4*>(a.out + row * D + 32 * c + k) = make_uint4(
                        sv::bf16x2(f[0], f[1]), sv::bf16x2(f[2], f[3]), sv::bf16x2(f[4], f[5]), sv::bf16x2(f[6], f[7]));
                }
            }
        }
    } else if (warp < 4 * MQ + 4) {
        // ---------------------------------------------------------- producers
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::R_LOAD));
        // Warp w copies rows 32 w .. 32 w + 31 of every tile; a lane looks up its row's place.
        const int w = warp - 4 * MQ;
        const unsigned char* mat[2] = {a.c.k + t.h * a.c.head_stride, a.c.v + t.h * a.c.head_stride};
        auto look_up = [&](int tile, int& page, int& row) {
            const int pos = t.begin + tile * TN + 32 * w + lane;
            page = -1;
            row = 0;
            if (tile < tiles && pos < t.end) page = sv::paged_place(a.c, t.b, pos, row);
        };
        auto offset = [&](int page, int row) {
            return page < 0 ? (int64_t)-1 : page * a.c.page_stride + row * a.c.row_stride;
        };
        bool bad = false;
        int page, row, page1, row1;  // of the tile at work and of the next
        look_up(0, page, row);
        look_up(1, page1, row1);
        if constexpr (!E4M3) {
            constexpr int CH = DP / 8, RPI = 32 / CH;  // pieces of a row, rows per instruction
            const int c = lane % CH, r0 = lane / CH;
            const uint32_t place0 = piece(32 * w + r0, c);
            // row r0 + RPI x: 128 bytes further per row, and the swizzle moves with the row
            auto place = [&](int x) { return (place0 ^ (uint32_t)(((RPI * x) & 7) << 4)) + x * RPI * 128; };
            const int most = 2 * D - 16 * c < 0 ? 0 : 2 * D - 16 * c > 16 ? 16 : 2 * D - 16 * c;
            int64_t off = -1;
            for (int n = 0; n < 2 * tiles; ++n) {
                const int tile = n >> 1, buf = n % S::NB;
                if (n >= S::NB) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.empty[buf], (n / S::NB - 1) & 1));
                    if (!ok) break;
                }
                if (!(n & 1)) {
                    off = offset(page, row);
                    const uint32_t bits = __ballot_sync(0xffffffffu, page >= 0);
                    if (lane == 0) sh.valid[tile % META][w] = bits;
                    page = page1;
                    row = row1;
                    look_up(tile + 2, page1, row1);
                }
                const unsigned char* src = mat[n & 1] + (most ? 16 * c : 0);
                const uint32_t dst = ring + buf * S::MAT;
#pragma unroll
                for (int x = 0; x < 32 / RPI; ++x) {
                    const int64_t o = __shfl_sync(0xffffffffu, off, x * RPI + r0);
                    cp_async16(dst + place(x), src + (o < 0 ? 0 : o), o < 0 ? 0 : most);
                }
                if ((n & 1) && t.begin + tile * TN + TN > open) {
                    // some queries see this tile in part: values that are not finite are taken out
                    // (and put back at the end for the queries that see them)
                    cp_wait_all();
                    for (int x = 0; x < 32 / RPI; ++x) {
                        uint4* p = reinterpret_cast<uint4*>(gen + (MQ + buf) * S::MAT + place(x));
                        uint4 v = *p;
                        if (sanitise<false>(v)) {
                            *p = v;
                            bad = true;
                        }
                    }
                    if (bad) sh.bad = 1;
                    fence_proxy_async();
                    mbar_arrive(&sh.full[buf]);
                } else {
                    cp_arrive(&sh.full[buf]);  // when this thread's copies have landed
                }
            }
            cp_wait_all();
        } else {
            constexpr int CH = DP / 16, RPI = 32 / CH, X = 32 / RPI;  // 16 codes a piece
            // A thread copies its pieces of an item to a place of its own, so that only it has to
            // wait for them; RAW items ahead cover the memory's latency.
            unsigned char* mine = gen + (MQ + S::NB) * S::MAT + 16 * (tid - 128 * MQ);
            const uint32_t mine_at = smem_u32(mine);
            const int c = lane % CH, r0 = lane / CH;
            const int most = D - 16 * c < 0 ? 0 : D - 16 * c > 16 ? 16 : D - 16 * c;
            const uint32_t place0 = piece(32 * w + r0, 2 * c);
            // row r0 + RPI x, element 16 c + 8 y; RPI is 4 or 8 rows
            auto place = [&](int x, int y) { return (place0 ^ (uint32_t)(((((RPI * x) & 7) ^ y)) << 4)) + x * RPI * 128; };
            float ks = 0.0f, vs = 0.0f, ks1 = 0.0f, vs1 = 0.0f;
            auto scales = [&](int page, int row, float& k, float& v) {
                k = v = 0.0f;
                if (page >= 0) {
                    const int64_t at = ((int64_t)page * a.c.heads + t.h) * a.c.page_size + row;
                    k = __ldg(a.c.k_scale + at);
                    v = __ldg(a.c.v_scale + at);
                }
            };
            // The copies run ahead of the conversions: tile `ahead` is the next to be copied.
            int ahead = 0, page2 = page, row2 = row, page3 = page1, row3 = row1;
            int64_t off = -1;
            auto copy = [&](int n) {
                if (n < 2 * tiles) {
                    if (!(n & 1)) {
                        off = offset(page2, row2);
                        page2 = page3;
                        row2 = row3;
                        ++ahead;
                        look_up(ahead + 1, page3, row3);
                    }
                    const unsigned char* src = mat[n & 1] + (most ? 16 * c : 0);
                    const uint32_t dst = mine_at + (n % S::RAW) * (S::MAT / 2);
#pragma unroll
                    for (int x = 0; x < X; ++x) {
                        const int64_t o = __shfl_sync(0xffffffffu, off, x * RPI + r0);
                        cp_async16(dst + x * 2048, src + (o < 0 ? 0 : o), o < 0 ? 0 : most);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            copy(0);
            copy(1);
            scales(page, row, ks, vs);
            for (int n = 0; n < 2 * tiles; ++n) {
                const int j = n >> 1, buf = n % S::NB, m = j % META;
                copy(n + 2);
                if (n >= S::NB) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.empty[buf], (n / S::NB - 1) & 1));
                    if (!ok) break;
                }
                const bool clean = (n & 1) && t.begin + j * TN + TN > open;
                if (!(n & 1)) {
                    if (t.begin + j * TN + TN > open && sv::not_finite(vs)) {
                        vs = 0.0f;
                        bad = true;
                    }
                    sh.ksc[m][32 * w + lane] = ks * a.scale_log2;
                    sh.vsc[m][32 * w + lane] = vs;
                    const uint32_t bits = __ballot_sync(0xffffffffu, page >= 0);
                    if (lane == 0) sh.valid[m][w] = bits;
                    scales(page1, row1, ks1, vs1);
                    ks = ks1;
                    vs = vs1;
                    page = page1;
                    row = row1;
                    look_up(j + 2, page1, row1);
                }
                asm volatile("cp.async.wait_group 2;" ::: "memory");
                unsigned char* dst = gen + (MQ + buf) * S::MAT;
                const unsigned char* from = mine + (n % S::RAW) * (S::MAT / 2);
#pragma unroll
                for (int x = 0; x < X; ++x) {
                    uint4 g = *reinterpret_cast<const uint4*>(from + x * 2048);
                    if (clean) bad |= sanitise<true>(g);
                    uint4 p, q;
                    widen16(g, p, q);
                    // lanes of a row's second 64 elements, whose banks are the first's, swap halves
                    const int y = (c >> 2) & 1;
                    *reinterpret_cast<uint4*>(dst + place(x, y)) = y ? q : p;
                    *reinterpret_cast<uint4*>(dst + place(x, y ^ 1)) = y ? p : q;
                }
                if (clean && bad) sh.bad = 1;
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.full[buf]);
            }
            cp_wait_all();
        }
        if (!ok) sh.failed = 1;
    } else {
        // ------------------------------------------------------------ products
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::R_MMA));
        if (warp == 4 * MQ + 4) {
            const uint32_t leader = elect_one();
            // the same in every lane, and known to be
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), sm0 = __shfl_sync(0xffffffffu, smem0, 0);
            const int todo = __shfl_sync(0xffffffffu, tiles, 0);
            const uint32_t ring0 = sm0 + MQ * S::MAT;
            constexpr uint32_t id_s = instruction(TN, false), id_o = instruction(DP, true);
            auto full = [&](int n) {
                const bool there = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.full[n % S::NB], (n / S::NB) & 1));
                fence_proxy_async();  // copies by other threads, seen through the barrier, before the products read them
                return there;
            };
            auto scores = [&](int q, int n) {  // S_q = Q_q K^T, K in item n
                const uint64_t qa = operand(sm0 + q * S::MAT, 16, 1024);
                const uint64_t ka = operand(ring0 + (n % S::NB) * S::MAT, 16, 1024);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const int at = ((k >> 2) * BLK + (k & 3) * 32) >> 4;
                    mma_ss(tm + S::S_COL + 128 * q, qa + at, ka + at, id_s, k > 0, leader);
                }
                tc_commit(&sh.s_full[q], leader);
            };
            ok = full(0);
            tc_fence_after();
            if (ok) {
                #pragma unroll
                for (int q = 0; q < MQ; ++q) scores(q, 0);
                tc_commit(&sh.empty[0], leader);
            }
            for (int j = 0; j < todo && ok; ++j) {
                const int nv = 2 * j + 1, nk = 2 * j + 2;
                ok = full(nv);
                const uint64_t va = operand(ring0 + (nv % S::NB) * S::MAT, BLK, 1024);
                for (int q = 0; q < MQ && ok; ++q) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.p_full[q], j & 1));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < TN / 16; ++k)
                        mma_ts(tm + S::O_COL + DP * q, tm + S::S_COL + 128 * q + 8 * k,
                               va + k * (2048 >> 4), id_o, j > 0 || k > 0, leader);
                    if (j + 1 < todo) {
                        if (q == 0) ok = full(nk);
                        if (ok) scores(q, nk);
                    } else {
                        tc_commit(&sh.o_full[q], leader);
                    }
                }
                if (ok) {
                    tc_commit(&sh.empty[nv % S::NB], leader);
                    if (j + 1 < todo) tc_commit(&sh.empty[nk % S::NB], leader);
                }
            }
            if (!ok) {
                sh.failed = 1;
                tc_commit(&sh.drain, leader);  // whatever was issued ends before the memory is given back
                (void)mbar_wait_bounded(&sh.drain, 0);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_free(tmem, S::COLS);
    }
}

template <int DP, int MQ, bool E4M3>
cudaError_t launch_one(const AttnArgs& a, unsigned ctas, cudaStream_t stream) {
    using S = Tc<DP, MQ, E4M3>;
    static sv::KernelLaunchCache cache;
    auto kern = paged_attention_tc_kernel<DP, MQ, E4M3>;
    int max_dyn = 0;
    const cudaError_t e = cache.setup((const void*)kern, &max_dyn);
    if (e != cudaSuccess) return e;
    if (S::SMEM > max_dyn) return cudaErrorInvalidValue;
    return sv::launch_serial(kern, dim3(ctas), dim3(S::THREADS), S::SMEM, stream, a);
}

template <int DP, bool E4M3>
cudaError_t launch_dim(const AttnArgs& a, int tile_rows, unsigned ctas, cudaStream_t stream) {
    return tile_rows == 256 ? launch_one<DP, 2, E4M3>(a, ctas, stream) : launch_one<DP, 1, E4M3>(a, ctas, stream);
}

}  // namespace

namespace sv {

cudaError_t launch_attn_tc(const AttnArgs& a, bool e4m3, int tile_rows, unsigned ctas, cudaStream_t stream) {
    if (a.c.dim <= 64) return e4m3 ? launch_dim<64, true>(a, tile_rows, ctas, stream) : launch_dim<64, false>(a, tile_rows, ctas, stream);
    return e4m3 ? launch_dim<128, true>(a, tile_rows, ctas, stream) : launch_dim<128, false>(a, tile_rows, ctas, stream);
}

}  // namespace sv
