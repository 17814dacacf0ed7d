// Appending latent rows to a paged 8-bit cache, with the norm and the
// position rotation on the way (see dsa_rows.cuh for that arithmetic).
//
// A block of scale_block tokens shares one scale 2^k, the least with
// amax <= 448 * 2^k over the block's values (e4m3 holds magnitudes up to
// 448), k >= -64.  A power of two, because then moving a stored code to a
// larger scale only changes its exponent: a block that already holds tokens
// keeps max(its scale, what the new tokens need), and when it grows the held
// codes are rescaled in place, exactly except where they become subnormal
// (rounded to nearest even).
//
// The codes and scales are those of the 64-bit result: where a float32 value is
// within its error of the border between two codes (in about one row of a
// hundred), or a maximum of the border between two scales (one of 2^16), the
// value is worked out again in 64 bits.  Float32 alone stored one code of a
// million off by a step; telling them apart takes 5 us of the 22 below.
//
// What bounds it is latency: a CTA's chain of offsets, sequence, page and rows,
// the norm's reductions, the block's maximum, the stores.  16384 rows of bf16 in
// five sequences: 23 to 26 us (29 MB, 1.2 TB/s); 8 or 608 single tokens: 10 us,
// most of it the launch.  (Rows are on their way while the page is looked up: 1 us.)
//
// One CTA runs one group of G = max(8, scale_block) aligned positions of a
// sequence, at most two rows a warp, with the rows' float32 values in registers
// between the maximum and the store: the input is read once.  The grid is known
// on the host without the sequences' lengths: sequence b's groups start at unit
// row_offsets[b] / G + 2 b, and floor(n / G) + 2 is never less than the number
// of groups that n tokens touch, so the units of two sequences never overlap.
#include <math.h>
#include <stdint.h>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "dsa_internal.h"
#include "dsa_ptx.cuh"
#include "dsa_rows.cuh"

namespace dsa {
namespace {

// The least k >= -64 with amax <= 448 * 2^k, for a finite amax >= 0:
// amax = f * 2^e with 1 <= f < 2, and 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int k = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return k < -64 ? -64 : k;
}

__device__ __forceinline__ float exp2_int(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }

// Eight values to e4m3 codes (nearest even, magnitudes above 448 to 448,
// NaN kept).
__device__ __forceinline__ uint2 to_e4m3x8(const float* x) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void from_e4m3x8(uint2 v, float* x) {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// ------------------------------------------------------- rows in 64 bits
// How far a float32 value may be off, relative to its magnitude (10 * 2^-24 of
// the norm, and 2 for the test's own roundings), and a rotated one to its
// bound (10 and 2 of the products and the sum, and 2).
constexpr float kNormError = 12.5f / (1 << 24), kTurnError = 15.0f / (1 << 24);

__device__ __forceinline__ double column_of(const float* row, int c) { return row[c]; }
__device__ __forceinline__ double column_of(const __nv_bfloat16* row, int c) { return __bfloat162float(row[c]); }

// 1 / sqrt(mean(x^2) + eps) of the row (the whole warp takes part).  A square
// is the sum of two floats, and the lane's sum is kept as two: the 64-bit
// pipe is slow.
template <typename T>
__device__ __forceinline__ double exact_inverse(const T* row, float eps, int lane) {
    float hi = 0.0f, lo = 0.0f;
    float x[2][8];
    load_row8(row + row_col(0, lane), x[0]);
    load_row8(row + row_col(1, lane), x[1]);
#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = __fmul_rn(x[a][i], x[a][i]), e = __fmaf_rn(x[a][i], x[a][i], -q);
            const float s = __fadd_rn(hi, q), t = __fsub_rn(s, hi);
            lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(q, t)), e));
            hi = s;
        }
    }
    double sum = static_cast<double>(hi) + static_cast<double>(lo);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const double m = sum * (1.0 / kD) + static_cast<double>(eps);
    const float mf = static_cast<float>(m);
    if (mf < kLeastMean) {
        // squares may have underflowed
        sum = 0.0;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fma(static_cast<double>(x[a][i]), static_cast<double>(x[a][i]), sum);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        return 1.0 / sqrt(sum * (1.0 / kD) + static_cast<double>(eps));
    }
    if (!(mf < 1e38f)) return 1.0 / sqrt(m);
    // r (1 + e / 2 + 3 e^2 / 8) with e = 1 - m r^2 of about 2^-23: 2^-60 off
    const double r = __frsqrt_rn(mf), e = fma(-m * r, r, 1.0);
    return fma(r * e, fma(e, 0.375, 0.5), r);
}

// Column c of the normed and rotated row; cs is the position's row of the table.
template <typename T, bool kHalves>
__device__ __forceinline__ double exact_column(const AppendParams& p, const T* row, const float* cs, double inv, int c) {
    const auto normed = [&](int i) {
        double v = column_of(row, i);
        if (p.eps >= 0.0f) {
            v *= inv;
            if (p.weight) v *= static_cast<double>(__ldg(p.weight + i));
        }
        return v;
    };
    const double v = normed(c);
    const int i = c - (kD - p.rope_dim), half = p.rope_dim / 2;
    if (i < 0) return v;
    const bool second = kHalves ? i >= half : (i & 1) != 0;
    const int pair = kHalves ? (second ? i - half : i) : i >> 1;
    const double u = normed(kHalves ? (second ? c - half : c + half) : c ^ 1);
    const double co = __ldg(cs + 2 * pair), si = __ldg(cs + 2 * pair + 1);
    return second ? v * co + u * si : v * co - u * si;
}

// Whether a maximum (as float bits) is next to 448 * 2^k, the border between two scales.
__device__ __forceinline__ bool next_to_border(uint32_t top) { return (top & 0x7FFFFFu) - (0x600000u - 64u) <= 128u; }

// Whether the row's largest finite magnitude, next to a border, is above it.
template <typename T, bool kHalves>
__device__ __forceinline__ bool exact_above(const AppendParams& p, const T* row, const float* cs, uint32_t top, int lane) {
    const double inv = p.eps >= 0.0f ? exact_inverse(row, p.eps, lane) : 0.0;
    const double border = __uint_as_float((top & 0x7F800000u) | 0x600000u);
    bool above = false;
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
        const double y = fabs(exact_column<T, kHalves>(p, row, cs, inv, row_col(i >> 3, lane) + (i & 7)));
        above |= y > border && y < static_cast<double>(INFINITY);
    }
    return __any_sync(0xffffffffu, above);
}

// The codes of this lane's columns in `which` (bit i: column i % 8 of slot
// i / 8), into the stored row at dst.
template <typename T, bool kHalves>
__device__ __forceinline__ void exact_codes(const AppendParams& p, const T* row, const float* cs, float inv_scale, uint32_t which,
                                            int lane, uint8_t* dst) {
    const double inv = p.eps >= 0.0f ? exact_inverse(row, p.eps, lane) : 0.0;
#pragma unroll 1
    for (; which; which &= which - 1) {
        const int i = __ffs(which) - 1, c = row_col(i >> 3, lane) + (i & 7);
        const double y = exact_column<T, kHalves>(p, row, cs, inv, c) * static_cast<double>(inv_scale);
        // to 24 bits with the last one odd if anything was cut off: rounding
        // that to the code's 4 is rounding y
        float f = __double2float_rz(y);
        if (static_cast<double>(f) != y) f = __uint_as_float(__float_as_uint(f) | 1u);
        dst[c] = __nv_cvt_float_to_fp8(f, __NV_SATFINITE, __NV_E4M3);
    }
}

// Warps of a group, and the groups that an SM has to hold: 64 registers a
// thread.  (16384 rows in groups of 32: 22.0 us, 23.8 with one group an SM and
// no spills; of 64: 24.5 with 32 warps of two rows; 16 of four spill more.)
template <int kG>
__host__ __device__ constexpr int append_warps() { return kG < 16 ? kG : (kG < 64 ? 16 : 32); }
template <int kG>
constexpr int append_groups() { return kG < 16 ? 4 : (kG < 64 ? 2 : 1); }

// Units before sequence b's.
template <int kG>
__device__ __forceinline__ long long unit_base(const int32_t* off, int b) {
    return static_cast<long long>(__ldg(off + b)) / kG + 2LL * b;
}

// The sequence of unit u: the last b in [0, B) with unit_base(b) <= u, by a
// search that probes 32 places at a time (the whole warp takes part).
template <int kG>
__device__ __forceinline__ int find_seq(const int32_t* off, int B, long long u, int lane) {
    int lo = 0, hi = B;                  // the answer is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool le = at < hi && (lane == 0 || unit_base<kG>(off, at) <= u);
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, le));
        lo += last * step;
        hi = lo + step < hi ? lo + step : hi;
    }
    return lo;
}

template <typename T, bool kHalves, int kG>
__global__ void __launch_bounds__(32 * append_warps<kG>(), append_groups<kG>()) dsa_append_kernel(const AppendParams p) {
    constexpr int kWarps = append_warps<kG>();
    constexpr int kRows = kG / kWarps;               // rows a warp
    static_assert(kRows <= 2, "the rows' last pass");
    __shared__ uint32_t amax_s[8];                   // per scale block of the group: bits of the maximum
    __shared__ float held_s[8];                      // the scale that its held tokens were stored with
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < 8) amax_s[threadIdx.x] = 0;
    __syncthreads();
    grid_dependency_wait();
    // the offsets are checked by the launch's first threads, a sequence each
    for (long long b = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; b < p.B;
         b += static_cast<long long>(gridDim.x) * blockDim.x) {
        const int o0 = __ldg(p.row_offsets + b), o1 = __ldg(p.row_offsets + b + 1);
        if (o0 < 0 || o1 < o0 || o1 > p.R) atomicOr(p.err, DSA_DEVERR_SEQ_RANGE);
    }
    const int b = find_seq<kG>(p.row_offsets, p.B, blockIdx.x, lane);
    const int o0 = __ldg(p.row_offsets + b), o1 = __ldg(p.row_offsets + b + 1);
    const int start = __ldg(p.seq_start + b);
    if (o0 < 0 || o1 <= o0 || o1 > p.R) return;      // (uniform over the CTA, as every exit before the barrier)
    const int n = o1 - o0;
    if (start < 0 || static_cast<long long>(start) + n > (static_cast<long long>(p.max_pages) << p.page_shift)) {
        if (threadIdx.x == 0) atomicOr(p.err, DSA_DEVERR_SEQ_RANGE);
        return;
    }
    const int end = start + n;
    const long long local = static_cast<long long>(blockIdx.x) - unit_base<kG>(p.row_offsets, b);
    const long long g0l = (static_cast<long long>(start) / kG + local) * kG;
    if (local < 0 || g0l >= end) return;
    const int g0 = static_cast<int>(g0l);            // the group's first position
    const int page = __ldg(p.page_table + static_cast<size_t>(b) * p.max_pages + (g0 >> p.page_shift));
    // the rows are on their way while the page is looked up
    const bool inexact = p.eps >= 0.0f || p.rope_dim != 0;
    float x[kRows][2][8], turn[kRows] = {};
    const T* kv = static_cast<const T*>(p.kv);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int pos = g0 + warp + r * kWarps;
        if (pos >= start && pos < end) {
            const T* src = kv + static_cast<size_t>(o0 + (pos - start)) * kD;
#pragma unroll
            for (int a = 0; a < 2; ++a) load_row8(src + row_col(a, lane), x[r][a]);
        }
    }
    float w[2][8];
    if (p.eps >= 0.0f) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            if (p.weight) {
                load8(p.weight + row_col(a, lane), w[a]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[a][i] = 1.0f;
            }
        }
    }
    if (page < 0 || page >= p.n_pages) {
        if (threadIdx.x == 0) atomicOr(p.err, DSA_DEVERR_PAGE_RANGE);
        return;
    }
    const size_t pool0 = (static_cast<size_t>(page) << p.page_shift) + (g0 & ((1 << p.page_shift) - 1));
    float* scales = p.cache_scale + (pool0 >> p.block_shift);
    // (read before any is written)
    const float held = threadIdx.x < kG >> p.block_shift ? __ldcg(scales + threadIdx.x) : 0.0f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int j = warp + r * kWarps, pos = g0 + j;
        if (pos >= start && pos < end) {
            if (p.eps >= 0.0f) row_norm(x[r], w, p.eps);
            if (p.rope_dim) {
                if (pos < p.n_positions) {
                    turn[r] = row_rotate<kHalves, true>(x[r], p.table + static_cast<size_t>(pos) * p.rope_dim, p.rope_dim, lane);
                } else {
                    if (lane == 0) atomicOr(p.err, DSA_DEVERR_POS_RANGE);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[r][0][i] = x[r][1][i] = __int_as_float(0x7FC00000);
                }
            }
            uint32_t top = 0;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // an element that is not finite is stored as NaN and does not count
                    const uint32_t m = __float_as_uint(x[r][a][i]) & 0x7FFFFFFFu;
                    if (m >= 0x7F800000u) x[r][a][i] = __int_as_float(0x7FC00000);
                    else top = m > top ? m : top;
                }
            top = __reduce_max_sync(0xffffffffu, top);
            if (inexact && next_to_border(top))
                top = ((top & 0x7F800000u) | 0x600000u) +
                      (exact_above<T, kHalves>(p, kv + static_cast<size_t>(o0 + (pos - start)) * kD,
                                               p.table + static_cast<size_t>(pos) * p.rope_dim, top, lane) ? 1u : 0u);
            if (lane == 0) atomicMax(&amax_s[j >> p.block_shift], top);
        }
    }
    if (threadIdx.x < 8) held_s[threadIdx.x] = held;
    __syncthreads();
    uint32_t which[kRows] = {};                      // columns next to a border
    // the scale of block blk of the group, whose first position is `first`
    const auto scale_of = [&](int blk, int first) {
        const float scale = exp2_int(scale_exponent(__uint_as_float(amax_s[blk])));
        return first < start ? fmaxf(scale, held_s[blk]) : scale;
    };
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int j = warp + r * kWarps, pos = g0 + j;
        const int blk = j >> p.block_shift;
        const int first = g0 + (blk << p.block_shift), last = first + (1 << p.block_shift);
        if (pos >= end || first >= end || last <= start) continue;     // nothing of this block is new, or behind the end
        const float scale = scale_of(blk, first);
        uint8_t* dst = p.cache + (pool0 + j) * kD;
        if (pos >= start) {
            const float inv = 1.0f / scale;                            // a power of two: exact
            uint2 codes[2], other[2];
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                // either side of the value by its error: rotated columns by
                // their slot's, the others by their own
                const bool turned = row_col(a, lane) >= kD - p.rope_dim;
                const float off = turned ? turn[r] * inv * kTurnError : 0.0f;
                const float lo = turned || !inexact ? inv : inv * (1.0f - kNormError), hi = turned || !inexact ? inv : inv * (1.0f + kNormError);
                float below[8], above[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    below[i] = fmaf(x[r][a][i], lo, -off);
                    above[i] = fmaf(x[r][a][i], hi, off > 0.0f ? off : -0.0f);      // (a zero keeps its sign)
                }
                codes[a] = to_e4m3x8(below);
                other[a] = to_e4m3x8(above);
            }
            const uint32_t diff[4] = {codes[0].x ^ other[0].x, codes[0].y ^ other[0].y, codes[1].x ^ other[1].x, codes[1].y ^ other[1].y};
            if ((diff[0] | diff[1] | diff[2] | diff[3]) != 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (diff[i >> 2] >> (8 * (i & 3)) & 0xFFu) which[r] |= 1u << i;
            }
#pragma unroll
            for (int a = 0; a < 2; ++a) *reinterpret_cast<uint2*>(dst + row_col(a, lane)) = codes[a];
        } else if (scale != held_s[blk]) {
            const float ratio = held_s[blk] / scale;
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                float y[8];
                from_e4m3x8(*reinterpret_cast<const uint2*>(dst + row_col(a, lane)), y);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= ratio;
                *reinterpret_cast<uint2*>(dst + row_col(a, lane)) = to_e4m3x8(y);
            }
        }
        if (lane == 0 && pos == (first > start ? first : start)) scales[blk] = scale;
    }
#pragma unroll 1
    for (int r = 0; r < kRows; ++r) {
        const uint32_t mine = r == 0 ? which[0] : which[kRows - 1];
        if (!__any_sync(0xffffffffu, mine != 0)) continue;
        const int j = warp + r * kWarps, pos = g0 + j, blk = j >> p.block_shift;
        exact_codes<T, kHalves>(p, kv + static_cast<size_t>(o0 + (pos - start)) * kD, p.table + static_cast<size_t>(pos) * p.rope_dim,
                                1.0f / scale_of(blk, g0 + (blk << p.block_shift)), mine, lane, p.cache + (pool0 + j) * kD);
    }
}

template <typename T, bool kHalves, int kG>
cudaError_t launch_one(const AppendParams& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.R / kG + 2 * p.B));
    cfg.blockDim = dim3(32 * append_warps<kG>());
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dsa_append_kernel<T, kHalves, kG>, p);
}

template <typename T, bool kHalves>
cudaError_t launch_group(const AppendParams& p, cudaStream_t s) {
    switch (p.scale_block) {
        case 16: return launch_one<T, kHalves, 16>(p, s);
        case 32: return launch_one<T, kHalves, 32>(p, s);
        case 64: return launch_one<T, kHalves, 64>(p, s);
        default: return launch_one<T, kHalves, 8>(p, s);     // 1, 2, 4, 8
    }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, bool bf16, bool halves, cudaStream_t s) {
    if (bf16) return halves ? launch_group<__nv_bfloat16, true>(p, s) : launch_group<__nv_bfloat16, false>(p, s);
    return halves ? launch_group<float, true>(p, s) : launch_group<float, false>(p, s);
}

}  // namespace dsa
