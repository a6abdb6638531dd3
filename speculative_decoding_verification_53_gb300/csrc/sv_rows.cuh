// sv_rows.cuh -- rows of one token and head as the kernels that write caches and activations
// hold them: eight elements per lane, loaded as they lie in memory, widened, and stored
// into a cache row (bf16, or e4m3 with its scale) or a dense one.
#pragma once

#include <cstdint>

#include "sv_paged.cuh"

namespace sv {

// Elements e0 .. e0+7 of a row of `dim` elements as fp32 (zero beyond dim).
template <typename T, bool AL>
__device__ __forceinline__ void load_row8(const T* row, int e0, int dim, float x[8]) {
    if (AL) {
        if (e0 < dim) {
            if (sizeof(T) == 2) {
                const uint4 v = ld_nc_v4(row + e0);
                x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
                x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
            } else {
                const uint4 a = ld_nc_v4(row + e0), b = ld_nc_v4(row + e0 + 4);
                x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y);
                x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
                x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y);
                x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.0f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = 0.0f;
            if (e0 + j < dim)
                x[j] = sizeof(T) == 2 ? __uint_as_float((uint32_t)__ldg((const unsigned short*)row + e0 + j) << 16)
                                      : __ldg((const float*)row + e0 + j);
        }
    }
}

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < pos_inf() ? a : 0.0f;  // false for NaN and infinity
}

// Eight elements of a row as they lie in memory (AL), or widened one by one.
template <typename T, bool AL>
struct Eight {
    uint4 w[AL ? (sizeof(T) == 2 ? 1 : 2) : 1];
    float f[AL ? 1 : 8];
    __device__ __forceinline__ void load(const T* row, int e0, int dim) {
        if (!AL) {
            load_row8<T, false>(row, e0, dim, f);
        } else if (e0 < dim) {
            w[0] = ld_nc_v4(row + e0);
            if (sizeof(T) == 4) w[sizeof(T) == 4 ? 1 : 0] = ld_nc_v4(row + e0 + 4);
        } else {
            w[0] = w[sizeof(T) == 4 ? 1 : 0] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    // Bits of the largest magnitude; at 0x7f800000 or beyond where one is not finite.
    __device__ __forceinline__ uint32_t largest() const {
        if (AL && sizeof(T) == 2) {  // two bf16 at a time: as integers magnitudes are in order
            const uint32_t a = __vmaxu2(w[0].x & 0x7fff7fffu, w[0].y & 0x7fff7fffu);
            const uint32_t b = __vmaxu2(w[0].z & 0x7fff7fffu, w[0].w & 0x7fff7fffu);
            const uint32_t c = __vmaxu2(a, b);
            return max(c << 16, c & 0xffff0000u);
        }
        float x[8];
        widen(x);
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ void widen(float x[8]) const {
        if (!AL) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = f[AL ? 0 : j];
        } else if (sizeof(T) == 2) {
            x[0] = bf16_lo(w[0].x); x[1] = bf16_hi(w[0].x); x[2] = bf16_lo(w[0].y); x[3] = bf16_hi(w[0].y);
            x[4] = bf16_lo(w[0].z); x[5] = bf16_hi(w[0].z); x[6] = bf16_lo(w[0].w); x[7] = bf16_hi(w[0].w);
        } else {
            const uint4 b = w[sizeof(T) == 4 ? 1 : 0];
            x[0] = __uint_as_float(w[0].x); x[1] = __uint_as_float(w[0].y);
            x[2] = __uint_as_float(w[0].z); x[3] = __uint_as_float(w[0].w);
            x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y);
            x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
        }
    }
};

// Writes eight elements of a cache row (and the row's scale).  LPR lanes hold the row.
template <typename T, int LPR, bool E4M3, bool AL>
__device__ __forceinline__ void store_cache_row(unsigned char* row, float* scale, int e0, int dim, bool live,
                                                const Eight<T, AL>& v) {
    if (E4M3) {
        uint32_t top = v.largest();
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        float a = __uint_as_float(top);
        // Rare rows: not all finite, or (but for zeros) so small or large that j may be subnormal
        // or a product may be: below 2^-80 or from 2^80 on.
        const bool rare = __any_sync(0xffffffffu, top != 0u && (top < 0x17800000u || top >= 0x67800000u));
        if (rare) {  // the largest finite magnitude
            float x[8];
            v.widen(x);
            a = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) a = fmaxf(a, finite_abs(x[j]));
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        }
        const float s = fmaxf(a / E4M3_MAX, 1.17549435e-38f);
        if (!live) return;
        // Rare rows are divided as x 2^90 and s 2^90 (or 2^-90), exact where it matters.
        const float f = !rare || (s > 1.0e-20f && s < 1.0e20f) ? 1.0f : s < 1.0f ? 1.2379400392853803e27f : 8.0779356694631609e-28f;
        const float i = 1.0f / (s * f), j = fmaf(-s * f, i, 1.0f) * i;
        const float2 i2 = make_float2(i, i), j2 = make_float2(j, j);
        float x[8];
        v.widen(x);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float2 e = make_float2(x[2 * k], x[2 * k + 1]);
            if (rare) e = make_float2(e.x * f, e.y * f);
            float2 q = ffma2(e, i2, fmul2(e, j2));
            if (rare) {  // infinity's x j may be of the other sign
                if (not_finite(e.x)) q.x = e.x;
                if (not_finite(e.y)) q.y = e.y;
            }
            w[k] = e4m3x2(q.x, q.y);
        }
        if (e0 == 0) *scale = s;
        if (AL) {
            if (e0 < dim) *reinterpret_cast<uint2*>(row + e0) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e0 + j < dim) row[e0 + j] = (unsigned char)(w[j / 2] >> (8 * (j & 1)));
        }
    } else {
        if (!live) return;
        float x[8];
        v.widen(x);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = bf16x2(x[2 * j], x[2 * j + 1]);
        if (AL) {
            if (e0 < dim) *reinterpret_cast<uint4*>(row + 2 * e0) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e0 + j < dim) reinterpret_cast<unsigned short*>(row)[e0 + j] = (unsigned short)(w[j / 2] >> (16 * (j & 1)));
        }
    }
}

template <typename T, bool AL>
__device__ __forceinline__ void store_row8(T* row, int e0, int dim, const float x[8]) {
    if (AL) {
        if (e0 >= dim) return;
        if (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(row + e0) = make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]),
                                                             bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
        } else {
            *reinterpret_cast<float4*>(row + e0) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(row + e0 + 4) = make_float4(x[4], x[5], x[6], x[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (e0 + j < dim) {
                if (sizeof(T) == 2) reinterpret_cast<unsigned short*>(row)[e0 + j] = (unsigned short)bf16x2(x[j], 0.0f);
                else reinterpret_cast<float*>(row)[e0 + j] = x[j];
            }
    }
}

// Eight elements of a cache row as they lie there, and widened.
template <bool E4M3, bool AL>
struct EightOfCache {
    Eight<uint16_t, AL> b;
    uint2 w;
    __device__ __forceinline__ void load(const unsigned char* row, int e0, int dim) {
        if (!E4M3) {
            b.load(reinterpret_cast<const uint16_t*>(row), e0, dim);
            return;
        }
        w = make_uint2(0u, 0u);
        if (AL) {
            if (e0 < dim) w = __ldg(reinterpret_cast<const uint2*>(row + e0));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e0 + j < dim) (j < 4 ? w.x : w.y) |= (uint32_t)__ldg(row + e0 + j) << (8 * (j & 3));
        }
    }
    __device__ __forceinline__ void widen(float scale, float x[8]) const {
        if (!E4M3) {
            b.widen(x);
            return;
        }
        const float2 p = e4m3x2_to_f32(w.x & 0xffffu), q = e4m3x2_to_f32(w.x >> 16);
        const float2 r = e4m3x2_to_f32(w.y & 0xffffu), t = e4m3x2_to_f32(w.y >> 16);
        x[0] = p.x * scale; x[1] = p.y * scale; x[2] = q.x * scale; x[3] = q.y * scale;
        x[4] = r.x * scale; x[5] = r.y * scale; x[6] = t.x * scale; x[7] = t.y * scale;
    }
};

}  // namespace sv
