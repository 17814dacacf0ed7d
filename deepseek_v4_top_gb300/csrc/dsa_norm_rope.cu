// Norm of every query head and latent row with the position rotation in the
// same pass (see dsa_rows.cuh for the arithmetic).
//
// Bound: memory.  A bf16 head row is read and written once (2 KB); the
// weights stay in registers for all rows of a warp and the table row (8 bytes
// a pair) is shared by a token's heads through L1.  One warp holds a whole
// row, so the sum of squares is five shuffles and no shared memory.  What
// limits it is how many bytes are on their way: a warp loads its next bf16 row
// before it works on this one (2048 x 64 + 2048 heads of bf16, 273 MB: 50 ->
// 45.9 us, 6.0 TB/s), while a float32 row has twice the bytes and the registers of a
// second one would cost warps (83 us without, 87 with it, for 545 MB).  More
// warps with the weights reloaded for each row took 60 us and more.
#include <math.h>
#include <stdint.h>

#include <mutex>

#include <cuda_bf16.h>

#include "dsa_internal.h"
#include "dsa_ptx.cuh"
#include "dsa_rows.cuh"

namespace dsa {
namespace {

constexpr int kNrThreads = 256;
constexpr int kNrWarps = kNrThreads / 32;

// A bf16 row as it is stored.
__device__ __forceinline__ void load_raw(const void* row, int lane, uint4* v) {
#pragma unroll
    for (int a = 0; a < 2; ++a) v[a] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(row) + row_col(a, lane));
}

template <typename T, bool kHalves>
__global__ void __launch_bounds__(kNrThreads) dsa_norm_rope_kernel(const NormRopeParams p) {
    constexpr bool kAhead = sizeof(T) == 2;
    grid_launch_dependents();
    grid_dependency_wait();
    // the first q_blocks blocks run the query rows, the others the key rows
    const bool is_k = static_cast<int>(blockIdx.x) >= p.q_blocks;
    const T* src = static_cast<const T*>(is_k ? p.k : p.q);
    T* dst = static_cast<T*>(is_k ? p.k_out : p.q_out);
    const float* wt = is_k ? p.k_weight : p.q_weight;
    const int heads = is_k ? p.Hk : p.H;
    const int n = p.R * heads;
    const int block = is_k ? blockIdx.x - p.q_blocks : blockIdx.x;
    const int blocks = is_k ? gridDim.x - p.q_blocks : p.q_blocks;
    const int lane = threadIdx.x & 31;
    float w[2][8];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        if (wt) {
            load8(wt + row_col(a, lane), w[a]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[a][i] = 1.0f;
        }
    }
    const long long step = static_cast<long long>(blocks) * kNrWarps;
    long long row = static_cast<long long>(block) * kNrWarps + (threadIdx.x >> 5);
    uint4 ahead[2] = {};
    if (kAhead && row < n) load_raw(src + row * kD, lane, ahead);
    for (; row < n; row += step) {
        float x[2][8];
        if (kAhead) {
            unpack8(ahead[0], x[0]);
            unpack8(ahead[1], x[1]);
            if (row + step < n) load_raw(src + (row + step) * kD, lane, ahead);
        } else {
#pragma unroll
            for (int a = 0; a < 2; ++a) load_row8(src + row * kD + row_col(a, lane), x[a]);
        }
        int pos = 0;
        if (p.rope_dim) pos = __ldg(p.positions + static_cast<int>(row / heads));
        if (p.eps >= 0.0f) row_norm(x, w, p.eps);
        if (p.rope_dim) {
            if (pos >= 0 && pos < p.n_positions) {
                row_rotate<kHalves>(x, p.table + static_cast<size_t>(pos) * p.rope_dim, p.rope_dim, lane);
            } else {
                if (lane == 0) atomicOr(p.err, DSA_DEVERR_POS_RANGE);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[0][i] = x[1][i] = __int_as_float(0x7FC00000);
            }
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) store_row8(dst + row * kD + row_col(a, lane), x[a]);
    }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& params, bool bf16, bool halves, int sms, cudaStream_t s) {
    NormRopeParams p = params;
    // more rows than these blocks have warps loop (three or four blocks of 256
    // threads with 60 to 80 registers are resident on an SM at a time)
    const long long most = static_cast<long long>(sms) * 8;
    const long long qb = (static_cast<long long>(p.R) * p.H + kNrWarps - 1) / kNrWarps;
    const long long kb = (static_cast<long long>(p.R) * p.Hk + kNrWarps - 1) / kNrWarps;
    p.q_blocks = static_cast<int>(qb < most ? qb : most);
    const int k_blocks = static_cast<int>(kb < most ? kb : most);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.q_blocks + k_blocks));
    cfg.blockDim = dim3(kNrThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (bf16)
        return halves ? cudaLaunchKernelEx(&cfg, dsa_norm_rope_kernel<__nv_bfloat16, true>, p)
                      : cudaLaunchKernelEx(&cfg, dsa_norm_rope_kernel<__nv_bfloat16, false>, p);
    return halves ? cudaLaunchKernelEx(&cfg, dsa_norm_rope_kernel<float, true>, p)
                  : cudaLaunchKernelEx(&cfg, dsa_norm_rope_kernel<float, false>, p);
}

}  // namespace dsa
