// sv_attention_tc.cu -- paged attention for many query rows per cache head (trees, chunks
// of prompts) on the 5th-generation tensor cores (include/spec_paged_kv.h).
//
// A CTA holds MQ tiles of 128 query rows and walks the positions in tiles of 128.  Per
// tile and row tile: S = Q K^T into TMEM (tcgen05.mma, Q and K in 128-byte-swizzled shared
// memory), the softmax warps read their rows of S, write the probabilities P as bf16 (e4m3 pages:
// fp16) over S, and O += P V accumulates in TMEM with P read from TMEM and V from shared memory in
// its stored order (positions x elements, "MN-major").  Roles:
//   warps 0 .. 4 MQ - 1   softmax, one thread per query row, one warpgroup per row tile
//   the next four         keys and values into a ring of NB shared buffers, where the copy
//                         engine cannot do it alone (odd page sizes; e4m3 codes, widened to
//                         fp16; values that are not finite taken out where hidden in part)
//   one warp each         the products (one lane issues every tcgen05.mma), the copy engine's
//                         requests, and notes on each tile (holes, scales); a fourth idles to
//                         make the warpgroup whole
// While one row tile's softmax runs, the tensor cores work on the other's products.
// Dependences: full/empty barriers per buffer; s_full (S is in TMEM, and so is the last
// O, since a commit covers every earlier product); p_full (P is written, O rescaled).
//
// DUAL: for 128 query rows or fewer the two warpgroups take the same rows and two stretches of
// positions, whose tiles alternate (tile v belongs to stretch v & 1): one row tile alone leaves
// the tensor cores and the copies waiting for its softmax (3600 cycles a tile of 64 KB; the
// memory brings one in 3000).  The CTA joins its two stretches itself: both O are in the TMEM lanes of
// either stretch's warps, which take half of the columns each.  As two partial results joined by the
// second kernel 512 chains of 6 over 1000 positions took 541 MB of scratch and 640 us, now none
// and 457 us (32 over 8 heads of 128, bf16).
//
// P is rounded to the type of V, since both operands of a product are of one type; what the rounding
// leaves could only enter as a second term, at twice the products of P V and twice the conversions
// of the softmax.  Errors against 64 bits grow from 0.0017 to 0.0023 of the largest output (bf16).
//
// The running maximum is moved only when it grows by more than 2^8: probabilities may
// then reach 256 instead of 1, harmless in fp32 sums and in bf16's and fp16's range, and the rescale of
// O in TMEM becomes rare.
//
// e4m3 pages are multiplied as fp16, which holds every code exactly and converts two in one
// instruction (bf16 takes four).  A position's key scale multiplies its scores, in fp32: rounding
// scaled keys to 11 bits moved lse by 10^-4.  A value's code times its scale, over a power of two
// that keeps the stretch's largest below 2^15, is rounded once to 11 bits, below what rounding the
// scaled probabilities to bf16 cost: code * hi + code * lo with the scale as two fp16 numbers,
// four instructions for two codes.  Queries are brought to [2^14, 2^15) row by row by a power
// of two, exactly to 2^-39 of the row's largest element.  Probabilities enter as fp16 too, 2^7
// times larger, so that fp16's subnormal step is 2^-31 of the largest.  O is held in units of
// the values' power of two and rescaled when it grows.
//
// That power of two follows the scales that every query of the CTA sees, never a token that some do
// not see.  Tiles with new tokens leave room for scales of up to 2^12 above those; values with larger
// ones are left out of the products and put back at the end for the queries that see them, as
// values that are not finite are.  (A unit per row in the softmax loop cost 172 -> 195 us of a tree
// batch in instruction-cache misses.)
//
// Heads wider than 128 take one row tile, 384 columns of TMEM and a ring of two 64 KB buffers; e4m3
// codes then go from the cache through registers.  16 trees of 61 over 4096, 32 over 8 heads of 256,
// bf16: 274 us (480 TFLOP/s), e4m3 460 us.
//
// Measured on one GB300, 32 over 8 heads of 128: 2 x 2048 queries over 6001 positions, bf16, 347-359 us
// (1310-1360 TFLOP/s, tensor pipe 53 %; the exponentials, 32 per SM and clock, take half as long as
// the products); 16 trees of 61 over 2048 to 8192, e4m3, 149-153 us (550 TFLOP/s; a tile takes 5700
// cycles, 2048 of them products, the rest widening and softmax); 8 chains of 6 over 3277 to 32768,
// bf16, 132 us (5.1 TB/s).
//
// Every wait is bounded.  A role whose wait runs out stops, so that the others' waits run out too;
// the softmax's warps then write NaN for their rows, which a verify reports as invalid data, and
// the CTA leaves when its copies have landed and its products have ended, which their warps wait
// for (with the same bound) whoever gave up.
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
constexpr float RAISE = 7.0f;    // e4m3: log2 of the probabilities' factor; 2^(8 + 7) is within fp16

template <int DP, int MQ, bool E4M3, bool DUAL>
struct Tc {
    static constexpr int QM = DUAL ? 1 : MQ;       // query matrices
    static constexpr int ROWS = 128 * QM;
    static constexpr int SOFTMAX = 128 * MQ;
    static constexpr int THREADS = SOFTMAX + 256;  // whole warpgroups, as setmaxnreg wants
    // Registers: the launch gives every thread 65536 / THREADS; softmax threads hold a row of
    // 128 scores and take what the others give back.
    //   MQ = 2: 512 x 128 = 65536 = 256 x 184 + 128 x 80 + 128 x 64 (bf16) = 256 x 176 + 128 x 96 + 128 x 64
    //   MQ = 1: 384 x 168 = 64512 >= 128 x 216 + 128 x 136 + 128 x 64 = 53248
    static constexpr int R_SOFTMAX = MQ == 1 ? 216 : E4M3 ? 176 : 184;
    static constexpr int R_LOAD = MQ == 1 ? 136 : E4M3 ? 96 : 80, R_MMA = 64;
    static_assert(SOFTMAX * R_SOFTMAX + 128 * (R_LOAD + R_MMA) <= (MQ == 2 ? 65536 : 64512), "registers of the launch");
    static constexpr int MAT = (DP / 64) * BLK;   // a tile of keys, values or queries
    static constexpr int NB = DP == 64 ? 6 : DP == 256 ? 2 : (E4M3 ? 3 : 4) + (DUAL ? 1 : 0);  // buffers of the ring
    static constexpr int RAW = E4M3 && DP != 256 ? 3 : 0;  // e4m3: items whose codes are in flight
    static constexpr int SMEM = (QM + NB) * MAT + RAW * MAT / 2 + 1024;  // and room to align
    static constexpr int S_COL = 0, O_COL = 128 * MQ;    // TMEM columns
    static constexpr int COLS = MQ == 2 || DP == 256 ? 512 : 256;
    static_assert(O_COL + DP * MQ <= COLS, "tensor memory");
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
// fp32 accumulator, bf16 or fp16 operands, 128 rows, n columns; b_mn: B is stored along n.
__host__ __device__ constexpr uint32_t instruction(int n, bool b_mn, bool f16) {
    return 1u << 4 | (f16 ? 0u : 1u << 7 | 1u << 10) | (b_mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint2 lds8(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
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

// Eight e4m3 codes in fp16, or times 2^-9 and a scale if asked (x: twice its fp16, y: twice what that
// leaves).  The 2^-9 is exact (codes are multiples of 2^-9, below 2^9) and keeps the scale 2^9
// further from fp16's subnormal numbers, where it would lose bits; by a branch
// for the tiles that need it alone 16 trees of 61 over 2048 to 8192 took 163 instead of 157 us.
template <bool SCALE>
__device__ __forceinline__ uint4 widen8(uint2 w, uint2 scale) {
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        asm("{.reg .b16 t, u;\n\tmov.b32 {t, u}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
            : "=r"(out[2 * i]), "=r"(out[2 * i + 1])
            : "r"(i ? w.y : w.x));
#pragma unroll
    for (int z = 0; SCALE && z < 4; ++z) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(out[z]) : "r"(0x18001800u));
#pragma unroll
    for (int z = 0; SCALE && z < 4; ++z)
        asm("{.reg .b32 t;\n\tmul.rn.f16x2 t, %0, %2;\n\tfma.rn.f16x2 %0, %0, %1, t;\n\t}"
            : "+r"(out[z])
            : "r"(scale.x), "r"(scale.y));
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// Two fp32 values rounded to fp16 (nearest even), lo in the low half.
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 2^e as fp32 (0 or infinity beyond the normal numbers).
__device__ __forceinline__ float power_of_two(int e) {
    return e < -126 ? 0.0f : e > 127 ? sv::pos_inf() : __int_as_float((e + 127) << 23);
}

// Scores of a row, scaled in place (by sc, and each by its own factor where given), -inf where hidden.
template <bool OWN, bool MASK>
__device__ __forceinline__ void scale_scores(uint32_t v[TN], const uint32_t see[4], const float* ksc, float sc) {
#pragma unroll
    for (int k = 0; k < TN; k += 4) {
        const float4 w = OWN ? *reinterpret_cast<const float4*>(ksc + k) : make_float4(sc, sc, sc, sc);
        const float2 f = fmul2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), make_float2(w.x, w.y));
        const float2 h = fmul2(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), make_float2(w.z, w.w));
        const float g[4] = {f.x, f.y, h.x, h.y};
#pragma unroll
        for (int z = 0; z < 4; ++z)
            v[k + z] = __float_as_uint(!MASK || ((see[k >> 5] >> ((k & 31) + z)) & 1u) ? g[z] : neg_inf());
    }
}

__device__ __forceinline__ float largest(const uint32_t v[TN]) {
    float t[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
    for (int k = 0; k < TN; k += 2) {
        float& m = t[(k >> 1) & 3];
        asm("max.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(__uint_as_float(v[k])), "f"(__uint_as_float(v[k + 1])));
    }
    return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

struct __align__(16) Shared {
    uint64_t full[8], empty[8];              // the ring's buffers
    uint64_t q_full, s_full[2], p_full[2][2], o_full[2], drain;
    uint64_t land[8], raw_full[4], raw_empty[4];  // copy engine: values to be looked over; e4m3 codes
    uint64_t note_full[META], note_empty[META];   // the tiles' notes below
    uint32_t tmem;
    int bad;
    int asked;  // copies that the copy engine has been asked for
    uint32_t valid[META][4];       // which of the tile's positions hold something
    __align__(16) float ksc[META][TN];  // e4m3: a position's key scale times the score factor
    __align__(16) uint2 vsc[META][TN];  // its value scale times 2^(9 - vexp), as two fp16 numbers
    int vexp[META];
    float limit[2];  // by stretch: larger value scales of new tokens are left to the end
    float row_factor[128];  // DUAL: what a row's scores are multiplied by
    float row_max[2][128], row_sum[2][128];  // DUAL: the stretches' results, to be joined
    int unit[2];    // DUAL: their vexp
    int gave_up;    // DUAL: a softmax warp whose wait ran out
};

template <int DP, int MQ, bool E4M3, bool DUAL>
__global__ void __launch_bounds__(MQ * 128 + 256, 1) paged_attention_tc_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                              const __grid_constant__ CUtensorMap v_map, const int box_rows, const int pairs) {
    using S = Tc<DP, MQ, E4M3, DUAL>;
    extern __shared__ unsigned char raw[];
    __shared__ Shared sh;
    pdl_trigger();
    pdl_wait();
    AttnTile t;
    if (!sv::attn_tile<false>(a, pairs, blockIdx.x, S::ROWS, DUAL ? 2 : 1, t)) return;
    const uint32_t smem0 = (smem_u32(raw) + 1023u) & ~1023u;  // queries, then the ring
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = a.c.dim, rows = t.n * a.group;
    // DUAL: a second stretch, of as many positions, fewer or none, follows the first
    const int mid = t.end, last_end = DUAL ? t.end2 : t.end;
    const int longest = DUAL && last_end - mid > mid - t.begin ? last_end - mid : mid - t.begin;
    const int tiles = (DUAL ? 2 : 1) * ((longest + TN - 1) / TN);
    // first position of tile v, and the end of its stretch
    auto start = [&](int v) { return DUAL ? (v & 1 ? mid : t.begin) + (v >> 1) * TN : t.begin + v * TN; };
    auto stop = [&](int v) { return DUAL && (v & 1) ? last_end : mid; };
    // Positions below this are seen by every query of the CTA.
    const int open = a.tree_mask ? t.base + 1 : t.base + t.mt * S::ROWS / a.group + 1;

    if (warp == 0) tmem_alloc(&sh.tmem, S::COLS);
    if (tid == 0) {
        for (int i = 0; i < S::NB; ++i) {
            mbar_init(&sh.full[i], E4M3 || box_rows ? 4 : 128);  // warps, or threads, that fill a buffer
            mbar_init(&sh.empty[i], 1);
            mbar_init(&sh.land[i], 1);
        }
        for (int i = 0; i < META; ++i) {
            mbar_init(&sh.note_full[i], 1);
            mbar_init(&sh.note_empty[i], 4 * S::QM + (E4M3 ? 4 : 0));
        }
        for (int i = 0; i < MQ; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i][0], 4);
            mbar_init(&sh.p_full[i][1], 4);
            mbar_init(&sh.o_full[i], 1);
        }
        mbar_init(&sh.q_full, 4 * S::QM);
        mbar_init(&sh.drain, 1);
        for (int i = 0; i < S::RAW; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], 4);
        }
        sh.bad = 0;
        sh.asked = 0;
        sh.gave_up = 0;
        sh.limit[0] = sh.limit[1] = sv::pos_inf();
        sv::fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const uint32_t ring = smem0 + S::QM * S::MAT;
    bool ok = true;

    if (warp < 4 * MQ) {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::R_SOFTMAX));
        const int q = warp >> 2;
        float own = 1.0f;  // e4m3: what the row's scores are multiplied by
        if (!DUAL || q == 0) {  // the queries of this warp's rows, zero behind the last real one
            constexpr int CH = DP / 8, RPI = 32 / CH;
            const int c = lane % CH, R = t.mt * S::ROWS + q * 128 + (warp & 3) * 32 + lane;
            const int y = R / a.group;
            const int64_t here = R < rows ? y * a.q_st + (int64_t)(t.h * a.group + R - y * a.group) * a.q_sh : -1;
            const uint16_t* from = a.q + t.b * a.q_sb;
            const uint32_t to = smem0 + q * S::MAT;
#pragma unroll 1
            for (int x = 0; x < 32; x += RPI) {
                const int64_t o = __shfl_sync(0xffffffffu, here, x + lane / CH);
                const bool there = o >= 0 && 8 * c < D;
                cp_async16(to + piece((warp & 3) * 32 + x + lane / CH, c), from + (there ? o + 8 * c : 0), there ? 16 : 0);
            }
            cp_wait_all();
            if (E4M3) {  // to fp16, a lane its row
                __syncwarp();
                const int r = (warp & 3) * 32 + lane;
                uint32_t top = 0u;  // largest magnitude, as bf16 bits
#pragma unroll 2
                for (int z = 0; z < CH; ++z) {
                    const uint4 v = lds16(to + piece(r, z));
                    const uint32_t m0 = max(max(v.x & 0x7fffu, v.y & 0x7fffu), max(v.z & 0x7fffu, v.w & 0x7fffu));
                    const uint32_t m1 = max(max((v.x >> 16) & 0x7fffu, (v.y >> 16) & 0x7fffu), max((v.z >> 16) & 0x7fffu, (v.w >> 16) & 0x7fffu));
                    top = max(top, max(m0, m1));
                }
                const int e = (int)(top >> 7) - 127;  // its exponent; 128: not finite, -127: 0 or subnormal
                const int up = e == 128 ? 0 : 14 - e > 126 ? 126 : 14 - e;
                const float f = power_of_two(up);
#pragma unroll 2
                for (int z = 0; z < CH; ++z) {
                    const uint32_t at = to + piece(r, z);
                    const uint4 v = lds16(at);
                    sts16(at, make_uint4(f16x2(sv::bf16_lo(v.x) * f, sv::bf16_hi(v.x) * f), f16x2(sv::bf16_lo(v.y) * f, sv::bf16_hi(v.y) * f),
                                         f16x2(sv::bf16_lo(v.z) * f, sv::bf16_hi(v.z) * f), f16x2(sv::bf16_lo(v.w) * f, sv::bf16_hi(v.w) * f)));
                }
                own = power_of_two(-up);
                if (DUAL) sh.row_factor[r] = own;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full);
        } else if (E4M3) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.q_full, 0));
            own = sh.row_factor[(warp & 3) * 32 + lane];
        }
        const int R = t.mt * S::ROWS + (DUAL ? 0 : q * 128) + (warp & 3) * 32 + lane;
        const bool live = R < rows;
        const int i = live ? R / a.group : 0;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 lanes per warp, lane field at bit 16
        const uint32_t s_at = tmem + lanes + S::S_COL + 128 * q, o_at = tmem + lanes + S::O_COL + DP * q;
        const float sc = a.scale_log2;
        float mx = neg_inf(), l = 0.0f;
        int vexp = 0;  // e4m3: O is held times 2^-vexp
        const bool idle = t.mt * S::ROWS + (DUAL ? 0 : q * 128) + (warp & 3) * 32 >= rows;  // no row of this warp is real
        for (int j = 0; j < (DUAL ? tiles / 2 : tiles) && ok; ++j) {
            const int u = DUAL ? 2 * j + q : j;  // the tile
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.s_full[q], j & 1));
            if (!ok) break;
            tc_fence_after();
            if (idle) {  // whatever its rows of P hold stays in its rows of O
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.p_full[q][0]);
                    mbar_arrive(&sh.p_full[q][1]);
                    mbar_arrive(&sh.note_empty[u % META]);
                }
                continue;
            }
            const int tile0 = start(u), m = u % META;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.note_full[m], (u / META) & 1));
            if (!ok) break;
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
            float top, mul = own;
            if (!E4M3 && whole && sc >= 0.0f) {
                top = largest(v) * sc;  // the factor joins the exponent's product below
                mul = sc;
            } else {
                if (E4M3 && whole) scale_scores<E4M3, false>(v, see, sh.ksc[m], sc);
                else scale_scores<E4M3, true>(v, see, sh.ksc[m], sc);
                top = largest(v) * own;
            }
            // move the maximum where it grew too far
            float fac = 1.0f;
            if (top > mx + RESCALE || mx == neg_inf()) {
                const float now = fmaxf(top, mx);
                fac = now == neg_inf() ? 1.0f : sv::ex2(mx - now);
                mx = now;
                l *= fac;
            }
            if (E4M3) {
                const int e = sh.vexp[m];
                if (j > 0) fac *= power_of_two(vexp - e);
                vexp = e;
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
            const float shift = (mx == neg_inf() ? 0.0f : mx) - (E4M3 ? RAISE : 0.0f);
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
                    p[k >> 1] = E4M3 ? f16x2(e.x, e.y) : sv::bf16x2(e.x, e.y);
                    p[(k >> 1) + 1] = E4M3 ? f16x2(f.x, f.y) : sv::bf16x2(f.x, f.y);
                }
                tmem_st16(s_at + 16 * c, p);  // over S, which this warp has read
                if (c & 1) {  // half of the row: its product may start
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.p_full[q][c >> 1]);
                }
            }
            if (lane == 0) mbar_arrive(&sh.note_empty[m]);
            sum0 = sv::fadd2(sum0, sum1);
            l += sum0.x + sum0.y;
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.o_full[q], 0));
        // DUAL: both stretches end before their results meet and leave through their memory
        if (DUAL && ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.o_full[q ^ 1], 0));
        tc_fence_after();
        // What O, or each stretch's O, is multiplied by.  DUAL: a row's maximum and sum meet in shared
        // memory; both O are in the TMEM lanes of either stretch's warp, which does half of the columns.
        float gain0, gain1 = 0.0f, shift = mx == neg_inf() ? 0.0f : mx;
        if (DUAL) {
            const int r = (warp & 3) * 32 + lane;
            sh.row_max[q][r] = mx;
            sh.row_sum[q][r] = l;
            if (!idle) sh.unit[q] = vexp;  // one for all rows
            if (!ok) sh.gave_up = 1;
            asm volatile("bar.sync 1, %0;" ::"n"(S::SOFTMAX) : "memory");
            ok = sh.gave_up == 0;
            const float m0 = sh.row_max[0][r], m1 = sh.row_max[1][r], most = fmaxf(m0, m1);
            shift = most == neg_inf() ? 0.0f : most;
            gain0 = sv::ex2(m0 - shift);
            gain1 = sv::ex2(m1 - shift);
            l = sh.row_sum[0][r] * gain0 + sh.row_sum[1][r] * gain1;
        }
        const float inv = !ok ? __int_as_float(0x7fffffff) : l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
        const float lse2 = !ok ? inv : l == 0.0f ? neg_inf() : shift + log2f(l) - (E4M3 ? RAISE : 0.0f);
        if (DUAL) {
            gain0 *= inv;
            gain1 *= inv;
            if (E4M3 && !idle) {
                gain0 *= power_of_two(sh.unit[0]);
                gain1 *= power_of_two(sh.unit[1]);
            }
        } else {
            gain0 = E4M3 ? inv * power_of_two(vexp) : inv;
        }
        const int64_t row = live ? sv::attn_row(a, t, R) : 0, part = t.part + (R - t.mt * S::ROWS);
        if (live && (!DUAL || q == 0)) {
            if (t.parts > 1) a.part_lse[part] = lse2;
            else if (a.lse) a.lse[row] = lse2 * 0.69314718055994531f;
        }
        const bool patch = sh.bad != 0;
        // no weight at all: zero, whatever the values hold
        const uint32_t keep = l == 0.0f && t.parts <= 1 ? 0u : 0xffffffffu;
        // Rows leave through shared memory (where this row tile's queries were), so that a store
        // covers whole rows: a lane writing its own row touched 32 lines per store and cost
        // 15000 cycles a CTA.  Part of a row at a time, 16-byte pieces swizzled by the row.
        constexpr int PASSES = DP == 256 ? 4 : 2, CW = DP / PASSES, PC = CW / 4;
        if (!ok) {  // nothing of this CTA's memory is sure to be at rest
            if (live && t.parts <= 1 && (!DUAL || q == 0))
                for (int d = 0; d < D; d += 8)
                    *reinterpret_cast<uint4*>(a.out + row * D + d) = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        } else if (!idle) {
            const uint32_t stage = smem0 + q * S::MAT + (warp & 3) * (S::MAT / 4);
            const uint32_t o0_at = tmem + lanes + S::O_COL + (DUAL ? 0 : DP * q);
            static_assert(!DUAL || PASSES == 2, "a pass per stretch's warps");
#pragma unroll 1
            for (int c = DUAL ? q : 0; c < (DUAL ? q + 1 : PASSES); ++c) {
                uint32_t v[CW];
                __syncwarp();
#pragma unroll
                for (int z = 0; z < CW; z += 32) tmem_ld32(o0_at + CW * c + z, v + z);
                tc_wait_ld();
#pragma unroll
                for (int k = 0; k < CW; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * gain0);
                if (DUAL) {
#pragma unroll
                    for (int z = 0; z < CW; z += 32) {
                        uint32_t w[32];
                        tmem_ld32(o0_at + DP + CW * c + z, w);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[z + k] = __float_as_uint(fmaf(__uint_as_float(w[k]), gain1, __uint_as_float(v[z + k])));
                    }
                }
                if (keep && live && patch) {
                    // Values that were left out, for the queries that see them: position by position, which
                    // takes long where there are many.  A prompt's first 2048 queries take 0.7 ms instead
                    // of 76 us where its first value row is zero (32 over 8 heads of 128; 8 over 8: 2.5 ms
                    // instead of 67 us, as a tile then has 256 new tokens; the queries' scattered reads
                    // bound it; element by element 1.7 and 6.6 ms).
                    int from = t.begin;  // stretches start at multiples of TN
                    if (open > t.begin) from += (open - t.begin) / TN * TN;
                    for (int pos = from; pos < last_end; ++pos) {
                        if (!(sv::attn_visible(a, t, i, pos) & 1u)) continue;
                        if (!E4M3) {
#pragma unroll
                            for (int k = 0; k < CW; ++k) {
                                if (CW * c + k >= D) break;
                                const float w = sv::attn_value<E4M3>(a, t, pos, CW * c + k);
                                if (sv::not_finite(w)) v[k] = __float_as_uint(__uint_as_float(v[k]) + w);
                            }
                        } else {
                            int r;
                            const int page = sv::paged_place(a.c, sv::attn_table_row(a, t), pos, r);
                            if (page < 0) continue;
                            const int64_t at = page * a.c.page_stride + t.h * a.c.head_stride + r * a.c.row_stride;
                            const int64_t sc_at = ((int64_t)page * a.c.heads + t.h) * a.c.page_size + r;
                            const float vs = __ldg(a.c.v_scale + sc_at);
                            const bool large = pos >= open && !sv::not_finite(vs) && fabsf(vs) > sh.limit[DUAL && pos >= mid ? 1 : 0];
                            float p = 0.0f;
                            if (large) {  // its probability, from the cache
                                const uint16_t* qr = a.q + t.b * a.q_sb + i * a.q_st + (int64_t)(t.h * a.group + R - i * a.group) * a.q_sh;
#pragma unroll 8
                                for (int d = 0; d < D; d += 8) {
                                    const uint4 x = sv::ld_nc_v4(qr + d);
                                    const uint2 y = __ldg(reinterpret_cast<const uint2*>(a.c.k + at + d));
                                    auto two = [&](uint32_t u, uint32_t w) {
                                        const float2 f = sv::e4m3x2_to_f32(w);
                                        p = fmaf(sv::bf16_hi(u), f.y, fmaf(sv::bf16_lo(u), f.x, p));
                                    };
                                    two(x.x, y.x & 0xffffu);
                                    two(x.y, y.x >> 16);
                                    two(x.z, y.y & 0xffffu);
                                    two(x.w, y.y >> 16);
                                }
                                p = sv::ex2(p * (__ldg(a.c.k_scale + sc_at) * a.scale_log2) - shift + RAISE) * inv;
                            }
#pragma unroll
                            for (int k = 0; k < CW; k += 4) {
                                if (CW * c + k >= D) break;
                                const uint32_t y = __ldg(reinterpret_cast<const uint32_t*>(a.c.v + at + CW * c + k));
#pragma unroll
                                for (int z = 0; z < 4; ++z) {
                                    const float w = sv::e4m3x2_to_f32((y >> 8 * z) & 0xffu).x;
                                    if (large) v[k + z] = __float_as_uint(__uint_as_float(v[k + z]) + p * w * vs);
                                    else if (sv::not_finite(w * vs)) v[k + z] = __float_as_uint(__uint_as_float(v[k + z]) + w * vs);
                                }
                            }
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < PC; ++k)
                    sts16(stage + 16 * (PC * lane + (k ^ (lane & (PC - 1)))), make_uint4(v[4 * k] & keep, v[4 * k + 1] & keep, v[4 * k + 2] & keep, v[4 * k + 3] & keep));
                __syncwarp();
                if (t.parts > 1) {
                    const int k = lane % PC, d = CW * c + 4 * k;
                    for (int x = 0; x < PC; ++x) {
                        const int r = (32 / PC) * x + lane / PC;
                        const int64_t to = __shfl_sync(0xffffffffu, live ? part : (int64_t)-1, r);
                        if (to >= 0 && d < D)
                            *reinterpret_cast<uint4*>(a.part_o + to * D + d) = lds16(stage + 16 * (PC * r + (k ^ (r & (PC - 1)))));
                    }
                } else {
                    const int k = 2 * (lane % (PC / 2)), d = CW * c + 4 * k;
                    for (int x = 0; x < PC / 2; ++x) {
                        const int r = (64 / PC) * x + lane / (PC / 2);
                        const int64_t to = __shfl_sync(0xffffffffu, live ? row : (int64_t)-1, r);
                        if (to >= 0 && d < D) {
                            const uint4 f = lds16(stage + 16 * (PC * r + (k ^ (r & (PC - 1)))));
                            const uint4 g = lds16(stage + 16 * (PC * r + ((k + 1) ^ (r & (PC - 1)))));
                            auto pair = [](uint32_t lo, uint32_t hi) { return sv::bf16x2(__uint_as_float(lo), __uint_as_float(hi)); };
                            *reinterpret_cast<uint4*>(a.out + to * D + d) =
                                make_uint4(pair(f.x, f.y), pair(f.z, f.w), pair(g.x, g.y), pair(g.z, g.w));
                        }
                    }
                }
            }
        }
    } else if (warp < 4 * MQ + 4) {
        // ---------------------------------------------------------- producers
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::R_LOAD));
        // Warp w fills rows 32 w .. 32 w + 31 of every tile.  With the copy engine it only looks
        // bf16 values over where some queries see them in part, or widens e4m3 codes; without,
        // it copies the rows, a lane looking up the place of one.
        const int w = warp - 4 * MQ;
        const unsigned char* mat[2] = {a.c.k + t.h * a.c.head_stride, a.c.v + t.h * a.c.head_stride};
        auto look_up = [&](int tile) {
            const int pos = start(tile) + 32 * w + lane;
            if (box_rows || tile >= tiles || pos >= stop(tile)) return (int64_t)-1;
            int row;
            const int page = sv::paged_place(a.c, sv::attn_table_row(a, t), pos, row);
            return page < 0 ? (int64_t)-1 : page * a.c.page_stride + row * a.c.row_stride;
        };
        bool bad = false;
        int64_t off = look_up(0), off1 = look_up(1);  // rows of the tile to be copied and of the next
        if constexpr (!E4M3) {
            constexpr int CH = DP / 8, RPI = 32 / CH;  // pieces of a row, rows per instruction
            const int c = lane % CH, r0 = lane / CH;
            const uint32_t place0 = piece(32 * w + r0, c);
            // row r0 + RPI x: 128 bytes further per row, and the swizzle moves with the row
            auto place = [&](int x) { return (place0 ^ (uint32_t)(((RPI * x) & 7) << 4)) + x * RPI * 128; };
            // Values that are not finite are taken out (and put back at the end for the queries
            // that see them), and whatever a page holds behind the sequence.
            auto look_over = [&](int tile, int buf) {
                for (int x = 0; x < 32 / RPI; ++x) {
                    const uint32_t at = ring + buf * S::MAT + place(x);
                    uint4 v = lds16(at);
                    if (start(tile) + 32 * w + x * RPI + r0 >= stop(tile)) {
                        sts16(at, make_uint4(0u, 0u, 0u, 0u));
                    } else if (sv::sanitise<false>(v)) {
                        sts16(at, v);
                        bad = true;
                    }
                }
                if (bad) sh.bad = 1;
                fence_proxy_async();
            };
            if (box_rows) {
                uint32_t lands = 0;  // phase of each buffer's barrier
                int asked = -1;      // copies asked for when a wait last ran out
                for (int j = 0; j < tiles; ++j) {
                    if (start(j) + TN <= open) continue;
                    const int buf = (2 * j + 1) % S::NB;
                    // The wait for the first such tile covers all tiles before it, however many: it
                    // starts again while copies go on being asked for.
                    do {
                        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.land[buf], (lands >> buf) & 1));
                        const int now = __shfl_sync(0xffffffffu, *(volatile int*)&sh.asked, 0);
                        if (ok || now == asked) break;
                        asked = now;
                    } while (true);
                    if (!ok) break;
                    lands ^= 1u << buf;
                    look_over(j, buf);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.full[buf]);
                }
            } else {
                const int most = 2 * D - 16 * c < 0 ? 0 : 2 * D - 16 * c > 16 ? 16 : 2 * D - 16 * c;
                for (int n = 0; n < 2 * tiles; ++n) {
                    const int tile = n >> 1, buf = n % S::NB;
                    if (n >= S::NB) {
                        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.empty[buf], (n / S::NB - 1) & 1));
                        if (!ok) break;
                    }
                    const unsigned char* src = mat[n & 1] + (most ? 16 * c : 0);
                    const uint32_t dst = ring + buf * S::MAT;
#pragma unroll
                    for (int x = 0; x < 32 / RPI; ++x) {
                        const int64_t o = __shfl_sync(0xffffffffu, off, x * RPI + r0);
                        cp_async16(dst + place(x), src + (o < 0 ? 0 : o), o < 0 ? 0 : most);
                    }
                    if (n & 1) {
                        off = off1;
                        off1 = look_up(tile + 2);
                    }
                    if ((n & 1) && start(tile) + TN > open) {
                        cp_wait_all();
                        look_over(tile, buf);
                        mbar_arrive(&sh.full[buf]);
                    } else {
                        cp_arrive(&sh.full[buf]);  // when this thread's copies have landed
                    }
                }
                cp_wait_all();
            }
        } else {
            constexpr int CH = DP / 16, RPI = 32 / CH, X = 32 / RPI;  // 16 codes a piece
            constexpr int RAW = S::RAW ? S::RAW : 1;
            // Wide heads leave no room for codes beside the ring: they come straight to registers,
            // PER pieces a lane, asked for while the PER before them are widened.
            constexpr bool DIRECT = S::RAW == 0;
            constexpr int PER = DIRECT ? 8 : 4;
            const int c = lane % CH, r0 = lane / CH;
            const int most = D - 16 * c < 0 ? 0 : D - 16 * c > 16 ? 16 : D - 16 * c;
            // Codes arrive in one of RAW places: by the copy engine as rows of DP codes, else a
            // thread copies its own pieces, so that only it has to wait for them.
            const uint32_t raw0 = ring + S::NB * S::MAT;
            const uint32_t own = 16 * (tid - 128 * MQ);
            const uint32_t mine = raw0 + (box_rows ? (32 * w + r0) * DP + 16 * c : own);
            const int step = box_rows ? RPI * DP : 2048;
            const uint32_t place0 = piece(32 * w + r0, 2 * c);
            // row r0 + RPI x, element 16 c + 8 y; RPI is 2, 4 or 8 rows
            auto place = [&](int x, int y) { return (place0 ^ (uint32_t)(((((RPI * x) & 7) ^ y)) << 4)) + x * RPI * 128; };
            auto copy = [&](int n) {
                if (n < 2 * tiles) {
                    const unsigned char* src = mat[n & 1] + (most ? 16 * c : 0);
                    const uint32_t dst = raw0 + own + (n % RAW) * (S::MAT / 2);
#pragma unroll
                    for (int x = 0; x < X; ++x) {
                        const int64_t o = __shfl_sync(0xffffffffu, off, x * RPI + r0);
                        cp_async16(dst + x * 2048, src + (o < 0 ? 0 : o), o < 0 ? 0 : most);
                    }
                    if (n & 1) {
                        off = off1;
                        off1 = look_up((n >> 1) + 2);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            uint4 now[DIRECT ? PER : 1], next[DIRECT ? PER : 1];
            auto ask = [&](int n, int x0) {  // rows x0 .. x0 + PER - 1 of item n, items in turn
                const unsigned char* src = mat[n & 1] + 16 * c;
#pragma unroll
                for (int x = 0; x < (DIRECT ? PER : 0); ++x) {
                    const int64_t o = __shfl_sync(0xffffffffu, off, (x0 + x) * RPI + r0);
                    next[x] = make_uint4(0u, 0u, 0u, 0u);
                    if (n < 2 * tiles && o >= 0) {
                        if (most == 16) next[x] = sv::ld_nc_v4(src + o);
                        else if (most == 8) *reinterpret_cast<uint2*>(&next[x]) = __ldg(reinterpret_cast<const uint2*>(src + o));
                    }
                }
                if ((n & 1) && x0 + PER == X) {
                    off = off1;
                    off1 = look_up((n >> 1) + 2);
                }
            };
            if (DIRECT) {
                ask(0, 0);
            } else if (!box_rows) {
                copy(0);
                copy(1);
            }
            for (int n = 0; n < 2 * tiles; ++n) {
                const int j = n >> 1, buf = n % S::NB;
                if (!DIRECT && !box_rows) copy(n + 2);
                if (n >= S::NB) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.empty[buf], (n / S::NB - 1) & 1));
                    if (!ok) break;
                }
                if (!DIRECT && box_rows) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.raw_full[n % RAW], (n / RAW) & 1));
                    if (!ok) break;
                } else if (!DIRECT) {
                    asm volatile("cp.async.wait_group 2;" ::: "memory");
                }
                if (!(n & 1)) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.note_full[j % META], (j / META) & 1));
                    if (!ok) break;
                }
                const uint2* scale = sh.vsc[j % META] + 32 * w + r0;
                const bool clean = (n & 1) && start(j) + TN > open;
                const uint32_t dst = ring + buf * S::MAT, from = mine + (n % RAW) * (S::MAT / 2);
                // Lanes of a row's second 64 elements, whose banks are the first's, take their two
                // halves in the other order.
                const int y = (c >> 2) & 1;
                // A short loop: unrolled in full, this and the softmax ran out of the instruction
                // caches (3000 cycles an item instead of 600).
#pragma unroll 1
                for (int x = 0; x < X; x += PER) {
                    uint2 g[2 * PER];
                    if (DIRECT) {
#pragma unroll
                        for (int z = 0; z < (DIRECT ? PER : 0); ++z) now[z] = next[z];
                        ask(x + PER < X ? n : n + 1, x + PER < X ? x + PER : 0);
                    }
#pragma unroll
                    for (int z = 0; z < 2 * PER; ++z) {
                        if (DIRECT) {
                            const uint4 v = now[DIRECT ? z >> 1 : 0];
                            g[z] = (z & 1) ^ y ? make_uint2(v.z, v.w) : make_uint2(v.x, v.y);
                        } else {
                            g[z] = lds8(from + (x + (z >> 1)) * step + 8 * ((z & 1) ^ y));
                        }
                    }
                    if (clean) {
#pragma unroll
                        for (int z = 0; z < 2 * PER; ++z) {
                            uint4 h = make_uint4(g[z].x, g[z].y, 0u, 0u);
                            if (start(j) + 32 * w + (x + (z >> 1)) * RPI + r0 >= stop(j)) h = make_uint4(0u, 0u, 0u, 0u);
                            bad |= sv::sanitise<true>(h);
                            g[z] = make_uint2(h.x, h.y);
                        }
                    }
                    if (n & 1) {
#pragma unroll
                        for (int z = 0; z < 2 * PER; ++z)
                            sts16(dst + place(x + (z >> 1), (z & 1) ^ y), widen8<true>(g[z], scale[(x + (z >> 1)) * RPI]));
                    } else {
#pragma unroll
                        for (int z = 0; z < 2 * PER; ++z)
                            sts16(dst + place(x + (z >> 1), (z & 1) ^ y), widen8<false>(g[z], make_uint2(0u, 0u)));
                    }
                }
                if (!DIRECT && box_rows) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.raw_empty[n % RAW]);
                }
                if (clean && bad) sh.bad = 1;
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.full[buf]);
                    if (n & 1) mbar_arrive(&sh.note_empty[j % META]);
                }
            }
            cp_wait_all();
        }
    } else {
        // ------------------------------------------------------------ products
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::R_MMA));
        if (warp == 4 * MQ + 4) {
            // one lane issues
            const uint32_t leader = elect_one();
            // the same in every lane, and known to be
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), sm0 = __shfl_sync(0xffffffffu, smem0, 0);
            const int todo = __shfl_sync(0xffffffffu, tiles, 0);
            const uint32_t ring0 = sm0 + S::QM * S::MAT;
            constexpr uint32_t id_s = instruction(TN, false, E4M3), id_o = instruction(DP, true, E4M3);
            auto full = [&](int n) {
                const bool there = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.full[n % S::NB], (n / S::NB) & 1));
                fence_proxy_async();  // copies by other threads, seen through the barrier, before the products read them
                return there;
            };
            auto scores = [&](int q, int n) {  // S_q = Q_q K^T, K in item n
                const uint64_t qa = operand(sm0 + (DUAL ? 0 : q * S::MAT), 16, 1024);
                const uint64_t ka = operand(ring0 + (n % S::NB) * S::MAT, 16, 1024);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const int at = ((k >> 2) * BLK + (k & 3) * 32) >> 4;
                    mma_ss(tm + S::S_COL + 128 * q, qa + at, ka + at, id_s, k > 0, leader);
                }
                tc_commit(&sh.s_full[q], leader);
            };
            // O_q += P_q V, V in item n, once the halves of P_q of its j-th tile are there
            auto outputs = [&](int q, int n, int j) {
                const uint64_t va = operand(ring0 + (n % S::NB) * S::MAT, BLK, 1024);
                bool there = true;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    there = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.p_full[q][half], j & 1)) && there;
                    tc_fence_after();
                    if (there) {
#pragma unroll
                        for (int k = 4 * half; k < 4 * half + 4; ++k)
                            mma_ts(tm + S::O_COL + DP * q, tm + S::S_COL + 128 * q + 8 * k, va + k * (2048 >> 4), id_o,
                                   j > 0 || k > 0, leader);
                    }
                }
                return there;
            };
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.q_full, 0));
            if (DUAL) {
                // tile u: keys in item 2 u, values in 2 u + 1, of stretch u & 1
                for (int q = 0; q < 2 && ok; ++q) {
                    ok = full(2 * q);
                    tc_fence_after();
                    if (ok) {
                        scores(q, 2 * q);
                        tc_commit(&sh.empty[2 * q % S::NB], leader);
                    }
                }
                for (int u = 0; u < todo && ok; ++u) {
                    const int q = u & 1, nv = 2 * u + 1, nk = 2 * u + 4;
                    ok = full(nv);
                    ok = outputs(q, nv, u >> 1) && ok;
                    if (!ok) break;
                    tc_commit(&sh.empty[nv % S::NB], leader);
                    if (u + 2 < todo) {
                        ok = full(nk);
                        if (ok) {
                            scores(q, nk);
                            tc_commit(&sh.empty[nk % S::NB], leader);
                        }
                    } else {
                        tc_commit(&sh.o_full[q], leader);
                    }
                }
            } else {
                ok = full(0) && ok;
                tc_fence_after();
                if (ok) {
#pragma unroll
                    for (int q = 0; q < MQ; ++q) scores(q, 0);
                    tc_commit(&sh.empty[0], leader);
                }
                for (int j = 0; j < todo && ok; ++j) {
                    const int nv = 2 * j + 1, nk = 2 * j + 2;
                    ok = full(nv);
                    for (int q = 0; q < MQ && ok; ++q) {
                        ok = outputs(q, nv, j);
                        if (!ok) break;
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
            }
            // whatever was issued ends before the memory is given back, whoever may have given up
            tc_commit(&sh.drain, leader);
            (void)mbar_wait_bounded(&sh.drain, 0);
        } else if (warp == 4 * MQ + 5 && box_rows) {
            // ---------------------------------------------------------- copies
            // Lane l < boxes copies the box of positions l * box_rows .. of a tile, which lie in
            // one page, into the ring, or e4m3 codes into the places before it.  bf16 values that
            // are to be looked over land on a barrier of their own.
            const int boxes = TN / box_rows;
            auto box_page = [&](int tile, int& page, int& row) {
                const int pos = start(tile) + lane * box_rows;
                page = a.c.num_pages;  // a page outside the cache reads as zeros
                row = 0;
                if (lane < boxes && tile < tiles && pos < stop(tile)) {
                    const int p = sv::paged_place(a.c, sv::attn_table_row(a, t), pos, row);
                    if (p >= 0) page = p;
                }
            };
            auto look_over = [&](int item) { return !E4M3 && (item & 1) && start(item >> 1) + TN > open; };
            uint32_t lands = 0;  // phase of each buffer's landing barrier
            int page, row, page1, row1, n = 0;
            box_page(0, page, row);
            box_page(1, page1, row1);
            for (; n < 2 * tiles; ++n) {
                constexpr int PLACES = S::RAW ? S::RAW : S::NB;
                const int slot = n % PLACES;
                if (n >= PLACES) {
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait_bounded(E4M3 ? &sh.raw_empty[slot & 3] : &sh.empty[slot], (n / PLACES - 1) & 1));
                    if (!ok) break;
                }
                const bool tail = look_over(n);
                if (tail) lands ^= 1u << slot;
                uint64_t* bar = E4M3 ? &sh.raw_full[slot & 3] : tail ? &sh.land[slot] : &sh.full[slot];
                if (lane == 0) {
                    sv::mbar_arrive_expect_tx(bar, E4M3 ? S::MAT / 2 : S::MAT);
                    if (!E4M3 && !tail) mbar_arrive_n(bar, 3);
                    *(volatile int*)&sh.asked = n + 1;
                }
                __syncwarp();
                const CUtensorMap* map = n & 1 ? &v_map : &k_map;
                if (lane < boxes) {
                    if (E4M3) {
                        sv::tma_box(smem0 + (S::QM + S::NB) * S::MAT + slot * (S::MAT / 2) + lane * box_rows * DP, map, 0, row, t.h, page, bar);
                    } else {
#pragma unroll
                        for (int z = 0; z < DP / 64; ++z)
                            sv::tma_box(ring + slot * S::MAT + z * BLK + lane * box_rows * 128, map, 64 * z, row, t.h, page, bar);
                    }
                }
                __syncwarp();
                if (n & 1) {
                    page = page1;
                    row = row1;
                    box_page((n >> 1) + 2, page1, row1);
                }
            }
            // The last copy into each place lands before the CTA leaves, whoever may have given up.
            constexpr int PLACES = S::RAW ? S::RAW : S::NB;
            for (int z = n > PLACES ? n - PLACES : 0; z < n; ++z) {
                const int slot = z % PLACES;
                if (E4M3) (void)mbar_wait_bounded(&sh.raw_full[slot & 3], (z / PLACES) & 1);
                else if (look_over(z)) (void)mbar_wait_bounded(&sh.land[slot], (~lands >> slot) & 1);
                else (void)mbar_wait_bounded(&sh.full[slot], (z / PLACES) & 1);
            }
        } else if (warp == 4 * MQ + 6) {
            // ----------------------------------------------------------- notes
            // Which positions of a tile hold something, and e4m3's scales; read ahead, so that
            // nobody else waits for a page table or a scale.
            // The stretches' largest finite value scales so far of positions that every query sees, as
            // bits; `seen` counts the last such position for both stretches.  The unit that values are
            // rounded in comes from these alone, so that no query's roundings hang on what it does
            // not see.  Tiles that hold new tokens keep room for scales of 2^12 times `seen`, which
            // then is at least 2^-7 units: a value is off by at most 3 2^-25 units (the scale's two
            // halves, the product with the lower one, the sum), 2^-25 of 448 seen, beside its 11 bits.
            // Beyond, a new token's value is left to the end, as values that are not finite are.
            uint32_t largest_v = 0u, other_v = 0u, seen = 0u, other_seen = 0u;
            if (E4M3) {
                int row;
                const int page = sv::paged_place(a.c, sv::attn_table_row(a, t), open - 1, row);
                if (page >= 0) {
                    const float s = fabsf(__ldg(a.c.v_scale + ((int64_t)page * a.c.heads + t.h) * a.c.page_size + row));
                    if (!sv::not_finite(s)) seen = other_seen = __float_as_uint(s);
                }
            }
            int64_t at1[4];  // index of the scales of the next tile's positions, -1: nothing there
            float ks[4], vs[4];
            uint32_t bits[4];
            auto look_up = [&](int tile, int64_t (&at)[4]) {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int pos = start(tile) + 32 * z + lane;
                    at[z] = -1;
                    if (tile < tiles && pos < stop(tile)) {
                        int row;
                        const int page = sv::paged_place(a.c, sv::attn_table_row(a, t), pos, row);
                        if (page >= 0) at[z] = ((int64_t)page * a.c.heads + t.h) * a.c.page_size + row;
                    }
                }
            };
            auto fetch = [&]() {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    bits[z] = __ballot_sync(0xffffffffu, at1[z] >= 0);
                    ks[z] = E4M3 && at1[z] >= 0 ? __ldg(a.c.k_scale + at1[z]) : 0.0f;
                    vs[z] = E4M3 && at1[z] >= 0 ? __ldg(a.c.v_scale + at1[z]) : 0.0f;
                }
            };
            look_up(0, at1);
            fetch();
            look_up(1, at1);
            for (int j = 0; j < tiles; ++j) {
                const int m = j % META;
                if (j >= META) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.note_empty[m], (j / META - 1) & 1));
                    if (!ok) break;
                }
                if (lane == 0) {
#pragma unroll
                    for (int z = 0; z < 4; ++z) sh.valid[m][z] = bits[z];
                }
                if (E4M3) {
                    const bool tail = start(j) + TN > open;
                    uint32_t seen_here = 0u;
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        if (start(j) + 32 * z + lane < open && !sv::not_finite(vs[z])) seen_here = max(seen_here, __float_as_uint(fabsf(vs[z])));
                    seen_here = __reduce_max_sync(0xffffffffu, seen_here);
                    largest_v = max(largest_v, seen_here);
                    seen = max(seen, seen_here);
                    if (tail) {
                        const float limit = 4096.0f * __uint_as_float(seen);
                        if (lane == 0) sh.limit[DUAL ? j & 1 : 0] = limit;
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            if (sv::not_finite(vs[z]) || (start(j) + 32 * z + lane >= open && fabsf(vs[z]) > limit)) {
                                vs[z] = 0.0f;  // put back at the end, as the values are
                                sh.bad = 1;
                            }
                    }
                    // scales below 2^6, times codes of at most 448: below 2^15
                    const int e = (int)((tail ? seen : largest_v) >> 23) - 127 + 1 - 6;
                    const int ve = min(max(e, -118) + (tail ? 12 : 0), 126);
                    auto halves = [](float s) {  // as two fp16 numbers, each twice
                        const uint32_t hi = f16x2(s, s);
                        float back;
                        asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(back) : "r"(hi));
                        return make_uint2(hi, f16x2(s - back, s - back));
                    };
                    if (lane == 0) sh.vexp[m] = ve;
                    if (DUAL) {  // the next tile is the other stretch's
                        const uint32_t x = largest_v, y = seen;
                        largest_v = other_v;
                        seen = other_seen;
                        other_v = x;
                        other_seen = y;
                    }
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        sh.ksc[m][32 * z + lane] = ks[z] * a.scale_log2;
                        sh.vsc[m][32 * z + lane] = halves(vs[z] * power_of_two(9 - ve));  // see widen8
                    }
                }
                __syncwarp();
                if (lane == 0 && !(t.b == a.stall_row && j == (tiles > 1))) mbar_arrive(&sh.note_full[m]);
                fetch();
                look_up(j + 2, at1);
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

template <int DP, int MQ, bool E4M3, bool DUAL>
cudaError_t launch_one(const AttnArgs& a, int pairs, unsigned ctas, cudaStream_t stream) {
    using S = Tc<DP, MQ, E4M3, DUAL>;
    static sv::KernelLaunchCache cache;
    auto kern = paged_attention_tc_kernel<DP, MQ, E4M3, DUAL>;
    int max_dyn = 0;
    const cudaError_t e = cache.setup((const void*)kern, &max_dyn);
    if (e != cudaSuccess) return e;
    if (S::SMEM > max_dyn) return cudaErrorInvalidValue;
    int rows = E4M3 && !S::RAW ? 0 : sv::page_box_rows(a.c, TN);
    CUtensorMap k{}, v{};
    const CUtensorMapSwizzle swizzle = E4M3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    if (rows && !(sv::page_map(&k, a.c.k, a.c, E4M3, E4M3 ? DP : 64, rows, swizzle) &&
                  sv::page_map(&v, a.c.v, a.c, E4M3, E4M3 ? DP : 64, rows, swizzle)))
        rows = 0;
    return sv::launch_serial(kern, dim3(ctas), dim3(S::THREADS), S::SMEM, stream, a, k, v, rows, pairs);
}

template <int DP, bool E4M3>
cudaError_t launch_dim(const AttnArgs& a, int pairs, int tile_rows, bool dual, unsigned ctas, cudaStream_t stream) {
    if (dual) return launch_one<DP, 2, E4M3, true>(a, pairs, ctas, stream);
    return tile_rows == 256 ? launch_one<DP, 2, E4M3, false>(a, pairs, ctas, stream)
                            : launch_one<DP, 1, E4M3, false>(a, pairs, ctas, stream);
}

}  // namespace

namespace sv {

cudaError_t launch_attn_tc(const AttnArgs& a, int pairs, bool e4m3, int tile_rows, bool dual, unsigned ctas,
                           cudaStream_t stream) {
    if (a.c.dim > 128) return e4m3 ? launch_one<256, 1, true, false>(a, pairs, ctas, stream) : launch_one<256, 1, false, false>(a, pairs, ctas, stream);
    if (a.c.dim <= 64) return e4m3 ? launch_dim<64, true>(a, pairs, tile_rows, dual, ctas, stream) : launch_dim<64, false>(a, pairs, tile_rows, dual, ctas, stream);
    return e4m3 ? launch_dim<128, true>(a, pairs, tile_rows, dual, ctas, stream) : launch_dim<128, false>(a, pairs, tile_rows, dual, ctas, stream);
}

}  // namespace sv
