// sv_attention_lists.cu -- attention of a few query rows over lists of blocks, a list per query
// (include/spec_sparse.h).
//
// Neighbouring queries select mostly the same blocks.  So a CTA takes the queries of up to 32 rows
// (queries times the heads that share a cache head) and walks the union of their lists, which a first
// kernel builds: pages in ascending order, and for each the queries that listed it, a bit each.  Every block is
// read once for all of them, and a position's bits hide its scores from the others.  (A CTA per
// query, which reads its own list: 8 chains of 6 over 32 of 512 pages of 64, 32 over 8 heads of 128, bf16,
// 77 us, and 43.6 so, with the unions and the join, where three quarters of the lists are in common; all of them 33, half 55,
// nothing 80; e4m3 47, 35, 60 and 88.)
//
// Positions are the products' 16 rows and query rows their columns, 8 at a time: S^T = K Q^T, and
// O^T = V^T P^T, so that tiles of 8 rows waste little, an accumulator of 8 rows takes a quarter of the
// registers of one of 16 x 2, and K and V fragments serve all row tiles.  A warp takes 16 positions
// of each tile of 64 and keeps its own maximum, sum and O; the warps meet at the end.  P leaves S^T's
// fragment layout for O^T's by movmatrix, rounded to bf16 as the values are (half a step, 2^-8 of each; sums of them
// stay fp32), since an fp32 factor would be two products of them.  The maximum is moved only when it grows by more than 2^8:
// until then probabilities are up to 256, harmless in fp32 sums and in bf16's range.
//
// A value that is not finite would reach, by 0 * inf, queries that do not see it.  They are rare, so the
// loop does not look for them: where a result is not finite the CTA starts again and takes them out as
// they arrive, and puts them back at the end for the queries that see them.  Nothing else changes in the
// second walk, so queries that do not see such a value keep every bit.
#include <cstdint>

#include "spec_sparse.h"
#include "sv_attention.cuh"

namespace {

using sv::AttnArgs;
using sv::AttnTile;
using sv::neg_inf;
using sv::smem_u32;

constexpr int TN = 64;       // positions per tile
constexpr int KW = 4;        // warps along the positions, 16 each
constexpr int THREADS = KW * 32;
constexpr float RESCALE = 8.0f;  // log2 of how far the maximum may lag

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t r[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t r[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
// Two e4m3 codes in the low half of w to a bf16 pair (exact).
__device__ __forceinline__ uint32_t widen(uint32_t w) {
    const float2 f = sv::e4m3x2_to_f32(w);
    return sv::bf16x2(f.x, f.y);
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte piece c of row r; the pieces of eight rows lie in different banks (of two rows where
// e4m3 keys are read, two rows at a time).
template <int PITCH>
__device__ __forceinline__ int piece(int r, int c) { return r * PITCH + ((PITCH >= 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4); }
template <int PITCH>
__device__ __forceinline__ int code_piece(int r, int c) { return r * PITCH + ((PITCH >= 128 ? c ^ ((r & 1) << 2) : c) << 4); }

template <int DP, int NQ, bool E4M3>
struct Lists {
    static constexpr int PITCH = (E4M3 ? 1 : 2) * DP, CH = PITCH / 16;
    static constexpr int MAT = TN * PITCH;   // a tile of keys, or of values
    static constexpr int STAGE = 2 * MAT + (E4M3 ? 2 * TN * 4 : 0);
    // Three CTAs an SM; with 3 stages of bf16 two, 8 chains of 6: 55 us against 43.
    static constexpr int STAGES = E4M3 ? 3 : 2;
    static constexpr int RING = 4;           // places and bits of the tiles in flight
    static_assert(STAGES < RING, "a tile's places outlive its copies");
    static constexpr int ROWS = 8 * NQ;
    static constexpr int QBYTES = ROWS * DP * 2;
    static constexpr int OP = DP + 4;        // floats of a row where the warps meet
    static constexpr int JOIN = KW * ROWS * OP * 4;  // which reuses the stages and the queries
    static constexpr int SMEM = STAGES * STAGE + QBYTES > JOIN ? STAGES * STAGE + QBYTES : JOIN;
};

// Which of the tile's queries (bit x: query first + x) see position `pos` of the list's sequence by the
// mask alone.
__device__ __forceinline__ uint32_t who_sees(const AttnArgs& a, const AttnTile& t, const uint32_t* bits, int listed, int pos, int block, int first, int queries) {
    if (pos < listed) return __ldg(bits + block);
    const int j = pos - t.base;  // among the new tokens
    if (j <= 0) return ~0u;      // the context's rest, and a chain's first token or a tree's root
    if (!a.tree_mask) return j - first <= 0 ? ~0u : j - first > 31 ? 0u : ~0u << (j - first);
    uint32_t m = 0u;
    const uint32_t* row = a.tree_mask + ((int64_t)t.b * (a.Q - 1) + first - 1) * a.mask_words + ((j - 1) >> 5);
    for (int x = 0; x < queries; ++x)
        if (first + x > 0) m |= ((__ldg(row + (int64_t)x * a.mask_words) >> ((j - 1) & 31)) & 1u) << x;
    return m;
}

template <int DP, int NQ, bool E4M3>
__global__ void __launch_bounds__(THREADS, NQ == 4 ? 2 : 3)
    list_attention_kernel(const __grid_constant__ AttnArgs a, const int pairs, const uint32_t* bits) {
    using S = Lists<DP, NQ, E4M3>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t s_off[S::RING][TN];   // byte offset of each position's row, -1: nothing there
    __shared__ uint32_t s_see[S::RING][TN];  // queries that see it
    __shared__ int64_t s_sc[E4M3 ? S::RING : 1][E4M3 ? TN : 1];  // index of its scales
    __shared__ float s_m[KW][S::ROWS], s_l[KW][S::ROWS];

    sv::pdl_trigger();
    sv::pdl_wait();
    AttnTile t;
    if (!sv::attn_tile(a, pairs, blockIdx.x, S::ROWS, 1, t)) return;
    const int tid = threadIdx.x, lane = tid & 31, wk = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int D = a.c.dim, row_bytes = (E4M3 ? 1 : 2) * D, rows = t.r1 - t.r0;
    const int tiles = (t.end - t.begin + TN - 1) / TN;
    const unsigned char* kbase = a.c.k + t.h * a.c.head_stride;
    const unsigned char* vbase = a.c.v + t.h * a.c.head_stride;
    const uint32_t smem0 = smem_u32(smem), q0 = smem0 + S::STAGES * S::STAGE;
    const int first = t.r0 / a.group, queries = rows / a.group;
    const int listed = t.base / a.c.page_size * a.c.page_size;  // positions of listed blocks: they come first, whole
    const uint32_t* own_bits = bits + (int64_t)t.row * a.c.max_pages;

    // Place and bits of a position of tile j, looked up a tile ahead of its copies.
    int64_t next_off = -1, next_sc = 0;
    uint32_t next_see = 0u;
    const int ps = a.c.page_size, shift = (ps & (ps - 1)) == 0 ? __ffs(ps) - 1 : -1;
    const int32_t* pages = a.c.table + (int64_t)t.row * a.c.max_pages;
    auto look_up = [&](int j) {
        if (tid >= TN) return;
        const int pos = t.begin + j * TN + tid;
        next_off = -1;
        next_see = 0u;
        if (pos < t.end) {
            const int block = shift >= 0 ? pos >> shift : pos / ps;
            const int page = __ldg(pages + block);
            next_see = who_sees(a, t, own_bits, listed, pos, block, first, queries);
            const int line = pos - block * ps;
            if ((unsigned)page < (unsigned)a.c.num_pages) next_off = page * a.c.page_stride + line * a.c.row_stride;
            else next_see = 0u;
            if (E4M3) next_sc = ((int64_t)page * a.c.heads + t.h) * ps + line;
        }
    };
    auto put_place = [&](int j) {
        if (tid >= TN) return;
        s_off[j % S::RING][tid] = next_off;
        s_see[j % S::RING][tid] = next_see;
        if (E4M3) s_sc[j % S::RING][tid] = next_sc;
    };
    constexpr int RPI = THREADS / S::CH;  // rows per instruction of a copy: a thread keeps to one piece of a row
    static_assert(RPI % 8 == 0, "and to one place in the banks");
    const int my_c = tid % S::CH, my_r = tid / S::CH;
    const int most = row_bytes - 16 * my_c < 16 ? (row_bytes - 16 * my_c < 0 ? 0 : row_bytes - 16 * my_c) : 16;
    const uint32_t my_place = smem0 + (E4M3 ? code_piece<S::PITCH>(my_r, my_c) : piece<S::PITCH>(my_r, my_c));
    const uint32_t my_value = smem0 + S::MAT + piece<S::PITCH>(my_r, my_c);
    const unsigned char* my_k = kbase + (most ? 16 * my_c : 0);
    const int64_t to_v = vbase - kbase;
    auto load_tile = [&](int j) {
        if (j < tiles) {
            const uint32_t st = (j % S::STAGES) * S::STAGE;
            const int64_t* off = s_off[j % S::RING] + my_r;
#pragma unroll
            for (int x = 0; x < TN / RPI; ++x) {
                const int64_t o = off[x * RPI];
                const int bytes = o < 0 ? 0 : most;
                const unsigned char* from = my_k + (o < 0 ? 0 : o);
                cp_async16(my_place + st + x * RPI * S::PITCH, from, bytes);
                cp_async16(my_value + st + x * RPI * S::PITCH, from + to_v, bytes);
            }
            if (E4M3) {  // one scale per thread: keys', then values'
                const int p = tid & (TN - 1);
                const bool there = s_off[j % S::RING][p] >= 0;
                cp_async4(smem0 + st + 2 * S::MAT + 4 * tid, (tid < TN ? a.c.k_scale : a.c.v_scale) + (there ? s_sc[E4M3 ? j % S::RING : 0][E4M3 ? p : 0] : 0), there ? 4 : 0);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // the queries, zero behind the last real row
    for (int f = tid; f < S::ROWS * (DP / 8); f += THREADS) {
        const int r = f / (DP / 8), c = f % (DP / 8), R = t.r0 + r;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows && 8 * c < D)
            w = sv::ld_nc_v4(a.q + t.b * a.q_sb + (int64_t)(R / a.group) * a.q_st + (int64_t)(t.h * a.group + R % a.group) * a.q_sh + 8 * c);
        unsigned char* to = smem + S::STAGES * S::STAGE;
        if (!E4M3) {
            *reinterpret_cast<uint4*>(to + piece<2 * DP>(r, c)) = w;
        } else {
            // A lane takes 16 contiguous codes of a key, which fixes an order of elements within a product:
            // element 64 e + 16 u + 4 s + 2 v + z goes to place 16 (4 e + s) + 8 v + 2 u + z.
            const int e = c >> 3, u = (c >> 1) & 3, s0 = (c & 1) * 2;
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = 16 * (4 * e + s0 + (j >> 1)) + 8 * (j & 1) + 2 * u;
                *reinterpret_cast<uint32_t*>(to + piece<2 * DP>(r, at >> 3) + 2 * (at & 7)) = ww[j];
            }
        }
    }
    // bits of this lane's two columns of each row tile (a row that is not real sees nothing)
    uint32_t col[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int r = 8 * n + 2 * t4 + z;
            col[n][z] = r < rows ? 1u << (r / a.group) : 0u;
        }

    // mx: what is subtracted from a column's scores (0 while it has seen nothing); lim: where it has to move
    float o[DP / 16][NQ][4], mx[NQ][2], lim[NQ][2], l[NQ][2];
    bool clean = false;  // second walk: values that are not finite are taken out
    while (true) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            mx[n][0] = mx[n][1] = 0.0f;
            lim[n][0] = lim[n][1] = neg_inf();
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) o[d][n][0] = o[d][n][1] = o[d][n][2] = o[d][n][3] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < S::STAGES; ++j) {
            look_up(j);
            put_place(j);
        }
        look_up(S::STAGES);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < S::STAGES - 1; ++j) load_tile(j);

        for (int j = 0; j < tiles; ++j) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S::STAGES - 2) : "memory");
            unsigned char* stage = smem + (j % S::STAGES) * S::STAGE;
            if (clean) {  // the pieces that this thread copied
                for (int f = tid; f < TN * S::CH; f += THREADS) {
                    uint4* p = reinterpret_cast<uint4*>(stage + S::MAT + piece<S::PITCH>(f / S::CH, f % S::CH));
                    uint4 v = *p;
                    if (sv::sanitise<E4M3>(v)) *p = v;
                }
                if (E4M3 && tid >= TN) {
                    float* p = reinterpret_cast<float*>(stage + 2 * S::MAT) + tid;
                    if (sv::not_finite(*p)) *p = 0.0f;
                }
            }
            __syncthreads();  // tile j is whole; tile j - 1 is no longer read
            load_tile(j + S::STAGES - 1);
            put_place(j + S::STAGES);
            look_up(j + S::STAGES + 1);

            const uint32_t ks0 = smem_u32(stage), vs0 = ks0 + S::MAT;
            const uint32_t see0 = s_see[j % S::RING][16 * wk + g], see1 = s_see[j % S::RING][16 * wk + 8 + g];
            if (!__any_sync(0xffffffffu, (see0 | see1) != 0u)) continue;
            float s[NQ][4];
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
            const int kr = 16 * wk + (lane & 15), kc = lane >> 4;  // 16 positions by 16 elements
            const int qr = lane & 7, qc = lane >> 3;               // 8 rows by 32 elements
            auto multiply = [&](int k, const uint32_t x[2][4]) {   // 32 elements
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    uint32_t q[4];
                    ldsm4(q0 + piece<2 * DP>(8 * n + qr, 4 * k + qc), q);
                    mma16816(s[n], x[0], q[0], q[1]);
                    mma16816(s[n], x[1], q[2], q[3]);
                }
            };
            if constexpr (!E4M3) {
#pragma unroll
                for (int k = 0; k < DP / 32; ++k) {
                    uint32_t x[2][4];
                    ldsm4(ks0 + piece<S::PITCH>(kr, 4 * k + kc), x[0]);
                    ldsm4(ks0 + piece<S::PITCH>(kr, 4 * k + 2 + kc), x[1]);
                    multiply(k, x);
                }
            } else {
#pragma unroll
                for (int e = 0; e < DP / 64; ++e) {
                    const uint4 w0 = lds16(ks0 + code_piece<S::PITCH>(16 * wk + g, 4 * e + t4));
                    const uint4 w1 = lds16(ks0 + code_piece<S::PITCH>(16 * wk + 8 + g, 4 * e + t4));
                    auto codes = [&](uint32_t u0, uint32_t u1, uint32_t x[4]) {
                        x[0] = widen(u0 & 0xffffu);
                        x[1] = widen(u1 & 0xffffu);
                        x[2] = widen(u0 >> 16);
                        x[3] = widen(u1 >> 16);
                    };
                    uint32_t x[2][4];
                    codes(w0.x, w1.x, x[0]);
                    codes(w0.y, w1.y, x[1]);
                    multiply(2 * e, x);
                    codes(w0.z, w1.z, x[0]);
                    codes(w0.w, w1.w, x[1]);
                    multiply(2 * e + 1, x);
                }
            }
            // scores' factors of positions g and g + 8, and values' scales, which their probabilities take
            float ks[2] = {a.scale_log2, a.scale_log2}, vs[2];
            if (E4M3) {
                const float* sc = reinterpret_cast<const float*>(stage + 2 * S::MAT) + 16 * wk + g;
                ks[0] *= sc[0];
                ks[1] *= sc[8];
                vs[0] = sc[TN];
                vs[1] = sc[TN + 8];
            }
            uint32_t grow = 0u;  // tiles of rows with a column that outgrew its maximum
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const float2 u = sv::fmul2(make_float2(s[n][0], s[n][1]), make_float2(ks[0], ks[0]));
                const float2 w = sv::fmul2(make_float2(s[n][2], s[n][3]), make_float2(ks[1], ks[1]));
                s[n][0] = see0 & col[n][0] ? u.x : neg_inf();
                s[n][1] = see0 & col[n][1] ? u.y : neg_inf();
                s[n][2] = see1 & col[n][0] ? w.x : neg_inf();
                s[n][3] = see1 & col[n][1] ? w.y : neg_inf();
                if (fmaxf(s[n][0], s[n][2]) > lim[n][0] || fmaxf(s[n][1], s[n][3]) > lim[n][1]) grow |= 1u << n;
            }
            // The maximum moves, but only in the columns that outgrew it: what a column does hangs on its own scores
            // alone, so keys that its query does not see move no bit of it.  Tiles of rows without such a column are left
            // out (8 chains of 6, e4m3: 47 us, 52 with all of them; bf16 43.6 and 43.9).
            grow = __reduce_or_sync(0xffffffffu, grow);
            if (grow) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    if (!((grow >> n) & 1u)) continue;
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        float top = fmaxf(s[n][z], s[n][2 + z]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        const bool moves = top > lim[n][z];  // alike in the column's lanes; never to -infinity
                        const float fac = moves && lim[n][z] != neg_inf() ? sv::ex2(mx[n][z] - top) : 1.0f;
                        if (moves) {
                            lim[n][z] = top + RESCALE;
                            mx[n][z] = top;
                        }
                        l[n][z] *= fac;
#pragma unroll
                        for (int d = 0; d < DP / 16; ++d) {
                            o[d][n][z] *= fac;
                            o[d][n][2 + z] *= fac;
                        }
                    }
                }
            }
            uint32_t p[NQ][2];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float e[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    e[x] = sv::ex2(s[n][x] - mx[n][x & 1]);
                    l[n][x & 1] += e[x];
                    if (E4M3) e[x] *= vs[x >> 1];
                }
                p[n][0] = transpose8x8(sv::bf16x2(e[0], e[1]));
                p[n][1] = transpose8x8(sv::bf16x2(e[2], e[3]));
            }
            if constexpr (!E4M3) {
                const int vr = 16 * wk + ((lane >> 4) << 3) + (lane & 7), vc = (lane >> 3) & 1;
#pragma unroll
                for (int d = 0; d < DP / 16; ++d) {
                    uint32_t x[4];
                    ldsm4t(vs0 + piece<S::PITCH>(vr, 2 * d + vc), x);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) mma16816(o[d][n], x, p[n][0], p[n][1]);
                }
            } else {
                // Transposed in pairs of codes: 32 elements are two tiles, of the even and of the odd ones.
                const int vr = 16 * wk + (((lane >> 3) & 1) << 3) + (lane & 7), vc = lane >> 4;
#pragma unroll
                for (int d = 0; d < DP / 32; ++d) {
                    uint32_t y[4], x[2][4];  // positions 0-7 and 8-15 of 16 elements, then of the next 16
                    ldsm4t(vs0 + piece<S::PITCH>(vr, 2 * d + vc), y);
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const uint32_t w = __byte_perm(y[z], 0u, 0x3120);
                        const int to = z == 1 ? 2 : z == 2 ? 1 : z;
                        x[0][to] = widen(w & 0xffffu);
                        x[1][to] = widen(w >> 16);
                    }
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        mma16816(o[2 * d][n], x[0], p[n][0], p[n][1]);
                        mma16816(o[2 * d + 1][n], x[1], p[n][0], p[n][1]);
                    }
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (clean) break;
        float sum = 0.0f;  // not finite where an element is not
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int d = 0; d < DP / 16; ++d)
#pragma unroll
                for (int x = 0; x < 4; ++x) sum += o[d][n][x] * 0.0f;
        if (!__syncthreads_or(sum != 0.0f)) break;
        clean = true;
    }

    // ---- the warps join
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            float w = l[n][z];
            w += __shfl_xor_sync(0xffffffffu, w, 4);
            w += __shfl_xor_sync(0xffffffffu, w, 8);
            w += __shfl_xor_sync(0xffffffffu, w, 16);
            const int r = 8 * n + 2 * t4 + z;
            if (g == 0) {
                s_m[wk][r] = lim[n][z] == neg_inf() ? neg_inf() : mx[n][z];
                s_l[wk][r] = w;
            }
            float* to = reinterpret_cast<float*>(smem) + (wk * S::ROWS + r) * S::OP;
#pragma unroll
            for (int d = 0; d < DP / 16; d += 2) {
                if (!E4M3) {
                    to[16 * d + g] = o[d][n][z];
                    to[16 * d + g + 8] = o[d][n][2 + z];
                    to[16 * d + g + 16] = o[d + 1][n][z];
                    to[16 * d + g + 24] = o[d + 1][n][2 + z];
                } else {
                    *reinterpret_cast<float2*>(to + 16 * d + 2 * g) = make_float2(o[d][n][z], o[d + 1][n][z]);
                    *reinterpret_cast<float2*>(to + 16 * d + 2 * g + 16) = make_float2(o[d][n][2 + z], o[d + 1][n][2 + z]);
                }
            }
        }
    __syncthreads();
    constexpr int TPR = DP / 4;  // threads of a row, four elements each
    for (int r = tid / TPR; r < rows; r += THREADS / TPR) {
        const int d = 4 * (tid % TPR);
        float top = s_m[0][r];
#pragma unroll
        for (int w = 1; w < KW; ++w) top = fmaxf(top, s_m[w][r]);
        const float shift = top == neg_inf() ? 0.0f : top;
        float sum = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            const float fac = sv::ex2(s_m[w][r] - shift);
            const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) + (w * S::ROWS + r) * S::OP + d);
            sum += s_l[w][r] * fac;
            v.x += x.x * fac;
            v.y += x.y * fac;
            v.z += x.z * fac;
            v.w += x.w * fac;
        }
        const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;  // NaN stays
        const float lse2 = sum == 0.0f ? neg_inf() : shift + log2f(sum);
        const bool none = sum == 0.0f;
        float out[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
        const int R = t.r0 + r, i = R / a.group;
        if (none) out[0] = out[1] = out[2] = out[3] = 0.0f;
        if (d >= D) continue;
        if (clean && !(none && t.parts <= 1)) {  // what was taken out, for the queries that see it
            for (int pos = t.begin; pos < t.end; ++pos) {
                if (!((who_sees(a, t, own_bits, listed, pos, pos / ps, first, queries) >> (i - first)) & 1u)) continue;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float w = sv::attn_value<E4M3>(a, t, pos, d + x);
                    if (sv::not_finite(w)) out[x] += w;
                }
            }
        }
        const int64_t row = sv::attn_row(a, t, R), part = t.part + r;
        if (t.parts > 1) {
            *reinterpret_cast<float4*>(a.part_o + part * D + d) = make_float4(out[0], out[1], out[2], out[3]);
            if (d == 0) a.part_lse[part] = lse2;
        } else {
            *reinterpret_cast<uint2*>(a.out + row * D + d) = make_uint2(sv::bf16x2(out[0], out[1]), sv::bf16x2(out[2], out[3]));
            if (d == 0 && a.lse) a.lse[row] = lse2 * 0.69314718055994531f;
        }
    }
}

// ------------------------------------------------------------------ unions

constexpr int kUnionThreads = 256, kUnionWarps = kUnionThreads / 32;

// f(block, query) for every block of every query's list that counts (ascending, of the context); a warp
// takes a list.
template <typename F>
__device__ __forceinline__ void each_taken(const int32_t* list, int64_t stride, int num_blocks, int queries, int full, F f) {
    const int lane = threadIdx.x & 31;
    for (int x = threadIdx.x >> 5; x < queries; x += kUnionWarps) {
        const int32_t* own = list + x * stride;
        int most = -1;  // the last one taken
        for (int e0 = 0; e0 < num_blocks; e0 += 32) {
            int e = e0 + lane < num_blocks ? __ldg(own + e0 + lane) : -1;
            if (e >= full) e = -1;
            int up = e;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up = max(up, y);
            }
            int before = __shfl_up_sync(0xffffffffu, up, 1);
            before = lane ? max(before, most) : most;
            if (e >= 0 && e > before) f(e, x);
            most = max(most, __shfl_sync(0xffffffffu, up, 31));
        }
    }
}

// One CTA per batch row, tile of queries and cache head: the row of the page table (pages of the union, then
// those from base / page_size on), the union's bits, and the positions before the chunk.
__global__ void __launch_bounds__(kUnionThreads) list_union_kernel(const __grid_constant__ sv::PagedCache c, const int32_t* base,
                                                                   const int32_t* new_len, const int32_t* blocks, int num_blocks,
                                                                   int Q, int query_tile, int tiles, int shared, int32_t* table,
                                                                   uint32_t* bits, int32_t* out_base, int width, int most) {
    extern __shared__ uint32_t s_dyn[];  // [most] bits of each block of the union, [words] blocks, [words] how many before
    __shared__ int s_sum[kUnionWarps];
    sv::pdl_trigger();
    sv::pdl_wait();
    const int row = blockIdx.x, h = row % c.heads, mt = row / c.heads % tiles, b = row / c.heads / tiles;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int first, n;
    if (!sv::paged_row(c, base, new_len, b, Q, first, n)) {
        if (tid == 0) out_base[row] = -1;  // left untouched
        return;
    }
    const int full = first / c.page_size, words = (full + 31) / 32;
    // shared: one list for all queries
    const int i0 = shared ? 0 : mt * query_tile, queries = shared ? 1 : max(0, min(query_tile, n - i0));
    uint32_t* s_mask = s_dyn;
    uint32_t* s_in = s_dyn + most;
    uint32_t* s_before = s_in + words;
    for (int w = tid; w < words; w += kUnionThreads) s_in[w] = 0u;
    for (int w = tid; w < most; w += kUnionThreads) s_mask[w] = 0u;
    __syncthreads();
    const int32_t* list = blocks + (((int64_t)b * (shared ? 1 : Q) + i0) * c.heads + h) * num_blocks;
    const int64_t stride = (int64_t)c.heads * num_blocks;
    each_taken(list, stride, num_blocks, queries, full, [&](int e, int) { atomicOr(&s_in[e >> 5], 1u << (e & 31)); });
    __syncthreads();
    const int per = (words + kUnionThreads - 1) / kUnionThreads, w0 = min(words, tid * per), w1 = min(words, w0 + per);
    int own = 0;
    for (int w = w0; w < w1; ++w) own += __popc(s_in[w]);
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) s_sum[warp] = sum;
    __syncthreads();
    int at = sum - own, count = 0;
#pragma unroll
    for (int w = 0; w < kUnionWarps; ++w) {
        if (w < warp) at += s_sum[w];
        count += s_sum[w];
    }
    for (int w = w0; w < w1; ++w) {
        s_before[w] = (uint32_t)at;
        at += __popc(s_in[w]);
    }
    __syncthreads();
    const int32_t* pages = c.table + (int64_t)b * c.max_pages;
    int32_t* to = table + (int64_t)row * width;
    uint32_t* to_bits = bits + (int64_t)row * width;
    each_taken(list, stride, num_blocks, queries, full, [&](int e, int x) {
        const int rank = (int)s_before[e >> 5] + __popc(s_in[e >> 5] & ((1u << (e & 31)) - 1u));
        if (atomicOr(&s_mask[rank], 1u << x) == 0u) to[rank] = __ldg(pages + e);  // the first of them
    });
    __syncthreads();
    for (int x = tid; x < count; x += kUnionThreads) to_bits[x] = shared ? ~0u : s_mask[x];
    const int last = n ? (first + n - 1) / c.page_size : full - 1;
    for (int k = tid; full + k <= last; k += kUnionThreads) to[count + k] = __ldg(pages + full + k);
    if (tid == 0) out_base[row] = count * c.page_size + (first - full * c.page_size);
}

template <int DP, int NQ, bool E4M3>
cudaError_t launch_rows(const AttnArgs& a, int pairs, unsigned ctas, const uint32_t* bits, cudaStream_t stream) {
    using S = Lists<DP, NQ, E4M3>;
    static sv::KernelLaunchCache cache;
    auto kern = list_attention_kernel<DP, NQ, E4M3>;
    int max_dyn = 0;
    const cudaError_t e = cache.setup((const void*)kern, &max_dyn);
    if (e != cudaSuccess) return e;
    if (S::SMEM > max_dyn) return cudaErrorInvalidValue;
    return sv::launch_serial(kern, dim3(ctas), dim3(THREADS), S::SMEM, stream, a, pairs, bits);
}

template <int DP, bool E4M3>
cudaError_t launch_dim(const AttnArgs& a, int pairs, int rows, unsigned ctas, const uint32_t* bits, cudaStream_t stream) {
    if (rows <= 8) return launch_rows<DP, 1, E4M3>(a, pairs, ctas, bits, stream);
    if (rows <= 16) return launch_rows<DP, 2, E4M3>(a, pairs, ctas, bits, stream);
    if (rows <= 24) return launch_rows<DP, 3, E4M3>(a, pairs, ctas, bits, stream);
    return launch_rows<DP, 4, E4M3>(a, pairs, ctas, bits, stream);
}

}  // namespace

namespace sv {

cudaError_t launch_list_attention(const AttnArgs& a, int pairs, bool e4m3, int rows, unsigned ctas, const uint32_t* bits, cudaStream_t stream) {
    if (a.c.dim <= 64) return e4m3 ? launch_dim<64, true>(a, pairs, rows, ctas, bits, stream) : launch_dim<64, false>(a, pairs, rows, ctas, bits, stream);
    return e4m3 ? launch_dim<128, true>(a, pairs, rows, ctas, bits, stream) : launch_dim<128, false>(a, pairs, rows, ctas, bits, stream);
}

cudaError_t launch_list_unions(const PagedCache& c, const int32_t* base, const int32_t* new_len, const int32_t* blocks,
                               int num_blocks, int Q, int query_tile, int tiles, bool shared, int64_t rows, int32_t* table, uint32_t* bits,
                               int32_t* out_base, int width, int most, cudaStream_t stream) {
    const size_t smem = ((size_t)most + 2 * (((size_t)c.max_pages + 31) / 32)) * sizeof(uint32_t);
    static sv::KernelLaunchCache cache;
    int max_dyn = 0;
    const cudaError_t e = cache.setup((const void*)list_union_kernel, &max_dyn);
    if (e != cudaSuccess) return e;
    if (smem > (size_t)max_dyn) return cudaErrorInvalidValue;
    return launch_serial(list_union_kernel, dim3((unsigned)rows), dim3(kUnionThreads), smem, stream, c, base, new_len, blocks,
                         num_blocks, Q, query_tile, tiles, (int)shared, table, bits, out_base, width, most);
}

}  // namespace sv
