// Arithmetic of one 512-wide row held by a warp, shared by the norm-and-
// rotation kernel (dsa_norm_rope.cu) and the paged append (dsa_append.cu):
//
//   y = x * w / sqrt(mean(x^2) + eps)               (eps < 0: y = x)
//   the last rope_dim columns turned in pairs (a, b) by the row's position:
//     (a, b) -> (a c - b s, b c + a s),  c, s = cos, sin from a float32 table
//
// Lane l holds columns [8 l, 8 l + 8) and [256 + 8 l, 256 + 8 l + 8): every
// load and store of the warp is contiguous (16 bytes a lane in bf16), and a
// pair of neighbouring columns stays in one lane.  All arithmetic is float32.
#pragma once

#include <stdint.h>

#include <cuda_bf16.h>

#include "dsa_internal.h"

namespace dsa {

// First column of slot s (0 or 1) of lane l.
__device__ __forceinline__ int row_col(int s, int lane) { return 256 * s + 8 * lane; }

__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// Row inputs may be the call's outputs (in place): plain loads, not __ldg.
__device__ __forceinline__ void load_row8(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// Eight bf16.
__device__ __forceinline__ void unpack8(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void load_row8(const __nv_bfloat16* p, float* x) { unpack8(*reinterpret_cast<const uint4*>(p), x); }

__device__ __forceinline__ void store_row8(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ void store_row8(__nv_bfloat16* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// x *= w / sqrt(mean(x^2) + eps).  The mean is a float32 sum in a fixed
// order (four chains of four squares, two additions, five across the lanes:
// 11 roundings of 2^-24); with eps, the root, the quotient and two products,
// all correctly rounded, a value is at most 10 * 2^-24 off the 64-bit result.
// A mean that is so small that squares in it may have underflowed is taken
// once more of 2^88 x, with 2^176 eps: the least element's square is then
// normal, and y stays the same.
constexpr float kLeastMean = 0x1p-100f;

__device__ __forceinline__ float row_mean(const float (&x)[2][8], float eps) {
    float part[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        part[i] = x[0][i] * x[0][i];
        part[i] = fmaf(x[0][4 + i], x[0][4 + i], part[i]);
        part[i] = fmaf(x[1][i], x[1][i], part[i]);
        part[i] = fmaf(x[1][4 + i], x[1][4 + i], part[i]);
    }
    float s = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return fmaf(s, 1.0f / kD, eps);
}

__device__ __forceinline__ void row_norm(float (&x)[2][8], const float (&w)[2][8], float eps) {
    float m = row_mean(x, eps);
    if (m < kLeastMean) {       // (the same in every lane)
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[a][i] *= 0x1p88f;
        m = row_mean(x, eps * 0x1p88f * 0x1p88f);
    }
    const float inv = __fdiv_rn(1.0f, __fsqrt_rn(m));
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[a][i] = x[a][i] * inv * w[a][i];
}

// Turns the last rope_dim columns (a multiple of 32) by cs, the position's
// row of the table: rope_dim / 2 pairs (cos, sin).  Neighbouring columns
// (2 i, 2 i + 1) form a pair, or (halves) columns i and i + rope_dim / 2 of
// the rotated part, whose partner is then fetched from its lane.  kBound:
// returns the largest |a c| + |b s| of the lane's turned elements (0 if none is
// turned): each is at most 12 * 2^-24 of that off the 64-bit rotation of the
// 64-bit row.
template <bool kHalves, bool kBound = false>
__device__ __forceinline__ float row_rotate(float (&x)[2][8], const float* cs, int rope_dim, int lane) {
    const int base = kD - rope_dim;
    float bound = 0.0f;
    if (!kHalves) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int c = row_col(a, lane);
            if (c >= base) {                      // base is a multiple of 32: all eight columns or none
                float t[8];
                load8(cs + (c - base), t);        // pair i holds floats 2 i, 2 i + 1
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u = x[a][2 * i], v = x[a][2 * i + 1];
                    if (kBound) {
                        bound = fmaxf(bound, fmaf(fabsf(u), fabsf(t[2 * i]), fabsf(v * t[2 * i + 1])));
                        bound = fmaxf(bound, fmaf(fabsf(v), fabsf(t[2 * i]), fabsf(u * t[2 * i + 1])));
                    }
                    x[a][2 * i] = u * t[2 * i] - v * t[2 * i + 1];
                    x[a][2 * i + 1] = v * t[2 * i] + u * t[2 * i + 1];
                }
            }
        }
    } else {
        const int half = rope_dim / 2;            // a multiple of 16: whole 8-column chunks
        float y[2][8];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int c = row_col(a, lane);
            const bool upper = c >= base + half;
            const int pc = c < base ? c : (upper ? c - half : c + half);    // the partner's column
            const int pl = (pc & 255) >> 3, ps = pc >> 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p0 = __shfl_sync(0xffffffffu, x[0][i], pl);
                const float p1 = __shfl_sync(0xffffffffu, x[1][i], pl);
                y[a][i] = ps ? p1 : p0;
            }
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int c = row_col(a, lane);
            if (c >= base) {
                const bool upper = c >= base + half;
                const float* t = cs + 2 * (c - base - (upper ? half : 0));
                float t0[8], t1[8];
                load8(t, t0);
                load8(t + 8, t1);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float co = i < 4 ? t0[2 * i] : t1[2 * i - 8];
                    const float si = i < 4 ? t0[2 * i + 1] : t1[2 * i - 7];
                    if (kBound) bound = fmaxf(bound, fmaf(fabsf(x[a][i]), fabsf(co), fabsf(y[a][i] * si)));
                    x[a][i] = upper ? x[a][i] * co + y[a][i] * si : x[a][i] * co - y[a][i] * si;
                }
            }
        }
    }
    return bound;
}

}  // namespace dsa
