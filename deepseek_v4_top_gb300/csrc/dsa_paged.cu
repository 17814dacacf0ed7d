// Attention over a paged 8-bit latent cache on the sm_103a tensor cores.
//
//   s_j = scale * <q_h, c_j> * sigma_j      c_j the e4m3 codes of key j, sigma_j its block's scale
//   out_h = sum_j e^{s_j} sigma_j c_j / (e^{sink_h} + sum_j e^{s_j})
//
// The codes go from the cache to the tensor cores as they are (kind::f8f6f4,
// 32 columns or keys a step): no element is ever converted, and a 128-key tile
// takes 64 KB instead of the 128 KB of bf16, so two of them fit beside Q.
//   * Q (bf16) is split per head into two e4m3 terms, q = 2^e (hi + lo / 32):
//     a bf16 value has 8 significant bits and the terms 4 each, so the split
//     is exact but for elements below 2^-15 of the head's largest (their
//     error is at most 2^-23 of that largest).  hi and lo of the 64 heads are
//     one N = 128 operand.
//   * The scale goes into the exponent: x_j = s_j log2(e) + log2(sigma_j), and
//     W_j = 2^(x_j - m) with m a running reference of the head is the value
//     weight itself; the softmax's denominator adds W_j / sigma_j in float32.
//     Blocks of very different scales need no reference of their own.
//   * W_j enters the value product as e4m3(W) + e5m2(W - e4m3(W)): down to W =
//     2^-6 at most 1.09 * 2^-8 of W off (4 and 3 bits; 2^-9.6 on average, under the
//     bf16 rounding of the output), below that 1.07 * 2^-14.  The second adds up over
//     a long tail of small weights, so the largest weight has to grow with the
//     tiles: a reference makes the first tile's 5, and goes down an octave at
//     tiles 5, 10, 20, 40 and 80 of a unit.  So t tiles never have less than a
//     weight of t beside them, and lose at most 1.07 * 2^-7 of it (every 160th tile,
//     heads whose largest weight there is below 160 go down to that).  A
//     weight that would pass 2^8.75 (e4m3 ends at 448) moves the reference up.  A
//     move rescales O in TMEM.  (With a largest weight of 1 at any length, one key 17
//     octaves above 32767 flat ones lost a sixth of the output, and 2048 rows of 640
//     keys took 256 us against 262 now; a first weight of 32 moves up in three tiles
//     of four, not in one of eight: 302 us with moves down by each tile's maxima.)
//
// Split: the rows' 128-key tiles, row after row, are cut into one equal share
// a CTA (each CTA finds its own share from the lengths on the device), so
// ragged batches balance and only rows cut by a share's border leave partials
// (float32, in the caller's workspace) for dsa_paged_combine_kernel.  A border
// within 1/8 of a share of a row's end moves there: a row more in one share
// costs less than the two halves' partials, second start and merge.
//
// Measured (H = 64, one GB300): 8 rows of 32768 keys 73 us (135 MB, 1.9 TB/s); 608
// rows of up to 640 selected keys 99 us (282 MB with q and out, 2.9 TB/s); 2048
// rows of one sequence with 640 selected keys each 262 us (660 TFLOP/s of the
// formulas' products); 8 rows of 640 keys 20 us with the merge.  What bounds it is
// the chain of a tile, keys landed -> scores -> weights -> value product -> the
// stage's next copy, with two tiles in flight: 5.5 to 6.5 thousand cycles a tile
// against 3.2 of matrix instructions (tensor pipe 25 % busy, issue slots 46 %,
// DRAM under 30 %).  Leaving out all copies of keys, three quarters of the score
// or of the value product, the later splits of Q, the moves or the stores of the
// output shortens the 2048 rows by 2 to 10 % each, so no one of them is the
// bound.  Three stages of 96 keys cost as much a tile as two of 128 (2048 rows:
// 365 us against 283 then), and keys brought to the L2 ahead gained nothing.
// Code size counts: 132, 100 and 90 KB of code took 295, 283 and 277 us, for one
// instruction fetch in ten misses its cache.
//
// The work is laid out for few instructions (pairs of float32 in one, few warps
// with fixed costs of their own), and the MMAs, copies and stores run beside
// it.  Twenty-four warps:
//   * warps 0-7, softmax: warp w reads TMEM lane quadrant w % 4 (32 keys of
//     S^T) and heads 32 (w / 4) .. + 31.
//   * warps 8-15 store a finished unit's output (or partial) while the next
//     one runs, and before that split the next unit's Q into its terms.
//   * warp 16 (one thread) issues the MMAs: S^T[key][hi, lo heads] of the next
//     tile runs while the softmax of the current one does; then
//     O^T[column][head] += V^T W for the current one.
//   * warp 17: key positions -> cache rows, up to four tiles ahead.
//   * warps 20-23 bring the keys' rows into the 128-byte swizzled tiles, a
//     quarter as soon as its last reader is done: of a whole context by TMA
//     boxes of 16 rows (one page holds them), of a selection by 16-byte
//     cp.async (TMA gathers of four rows take as long and more instructions).
//
// Every wait is bounded (see dsa_ptx.cuh); on a timeout the kernel raises an
// error bit, lets its copies land, frees its TMEM and returns.
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dsa_internal.h"
#include "dsa_ptx.cuh"

namespace dsa {
namespace {

constexpr int kPgThreads = 768;
constexpr int kSmWarps = 8;                  // softmax warps 0-7: 32 heads each
constexpr int kOutWarp0 = 8, kOutWarps = 8;
constexpr int kMmaWarp = 16, kIdxWarp = 17;
constexpr int kGatherWarp0 = 20, kGatherWarps = 4;
// Q is split by the output warps, at the start of a share from this head on by
// the softmax warps
constexpr int kOutHeads = 32;
// registers a thread of each warpgroup: the softmax's grow from what the
// launch gives, the others shrink
constexpr uint32_t kRegsLaunch = 80;
constexpr uint32_t kRegsSoftmax = 120;
constexpr uint32_t kRegsOutput = 80;
constexpr uint32_t kRegsOther = 40;          // MMA and index warps; gather warps
static_assert(kRegsSoftmax >= kRegsLaunch && kRegsOutput <= kRegsLaunch && kRegsOther <= kRegsLaunch,
              "setmaxnreg.inc and .dec must not go the other way");
static_assert(2 * kRegsSoftmax + 2 * kRegsOutput + 2 * kRegsOther == 6 * kRegsLaunch && kRegsLaunch * kPgThreads <= 65536,
              "the register split must add up to the launch's");
constexpr int kRing = 4;                     // tiles of key rows and scales in flight

constexpr uint32_t kSegBytes = 128 * 128;    // 128 keys (or Q rows) x 128 columns of one byte
constexpr uint32_t kStageBytes = 4 * kSegBytes;
constexpr uint32_t kPPlane = 128 * 64;       // 128 keys x 64 heads of one byte
constexpr uint32_t kOffKv = 0;
constexpr uint32_t kOffQ = kOffKv + 2 * kStageBytes;
constexpr uint32_t kOffP = kOffQ + kStageBytes;
constexpr uint32_t kOffMisc = kOffP + 2 * kPPlane;

constexpr uint32_t kTmemCols = 512;
__host__ __device__ constexpr uint32_t tmem_s(int buf) { return 128u * static_cast<uint32_t>(buf); }
__host__ __device__ constexpr uint32_t tmem_o(int i) { return 256u + 64u * static_cast<uint32_t>(i); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTop = 8.75f;                // a weight above 2^kTop moves its head's reference,
constexpr float kBase = 2.3219281f;          // which makes the tile's largest weight 5 (a number that the terms hold),
constexpr int kFirstDown = 5, kDowns = 5;    // times two after this tile of a unit and each doubling of it, so often;
                                             // then (every 160 tiles) heads of lower weights go down to that,
constexpr float kDown = 24.0f;               // but not further than this below their highest place

// Flags of a tile: the first and the last of its unit, the last of the share;
// all references go down an octave, those of low weights are renewed; and, from
// bit kLoweredShift on, how often they have gone down in the unit.
// Of a unit: the last of the share, all tiles of its row, a row without a key,
// a part that does not begin at the row's first tile.
constexpr int kFirst = 1, kLast = 2, kEnd = 4, kWhole = 8, kEmpty = 16, kInside = 32, kLower = 64, kRenew = 128;
constexpr int kLoweredShift = 8;
constexpr int kUnits = 8;                    // units of which the index warp may be ahead of the output warps

struct Misc {
    uint64_t kv_full[2];        // gather -> MMA: the stage's tile landed
    uint64_t kv_free[2][4];     // MMA -> gather: the P.V of keys [32 i, 32 i + 32) of the stage is done
    uint64_t s_full[2];         // MMA -> softmax: scores ready (the commit, and an arrive of the issuing
                                // thread, which has seen the unit's q_scale)
    uint64_t s_free[2];         // softmax -> MMA: scores read
    uint64_t p_full;            // softmax -> MMA: weights written (and O rescaled)
    uint64_t pv_done;           // MMA -> softmax: the tile's P.V is done (P and O free)
    uint64_t q_full;            // splitting warps -> MMA: a head of the unit's Q and its q_scale written
    uint64_t q_free;            // MMA -> splitting warps: the unit's last scores are done
    uint64_t o_full;            // MMA -> output warps: the unit's last P.V is done
    uint64_t o_free;            // output warps -> MMA: the unit's O has been read
    uint64_t l_ready;           // softmax -> output warps: red_l, m_ref hold the unit's
    uint64_t l_free;            // output warps -> softmax: they have been read
    uint64_t red_sync;          // softmax warps
    uint64_t ring_full[kRing];  // index warp -> gather, softmax, MMA
    uint64_t ring_free[kRing];
    uint64_t unit_full[kUnits]; // index warp -> output warps
    uint64_t drain;
    alignas(16) int red[3][64];          // by move: each head's largest x of the tile, in ordered_int's order
    // [softmax warp]: minus its heads' references; the factors of the last move; minus the lowest places that the
    // references may take
    alignas(16) float refs[8][96];
    alignas(16) float red_l[4][64];      // a finished unit's sums
    alignas(16) float m_ref[64];
    alignas(16) float fac[8][64];        // [output warp][head]: what the unit's value sums are multiplied by
    // 2^e * scale * log2(e) of each head, by unit: the softmax may still be in the
    // unit before last when the next one's are written
    alignas(16) float q_scale[4][64];
    int unit[kUnits][2];                 // query row and flags of each unit on its way
    alignas(16) int tile[kRing][4];      // valid keys and kFirst.. flags of each tile on its way
    alignas(16) int row[kRing][128];     // cache row of each key; the complement of one: no key, or a bad one
    int move[2];                         // a weight of the tile (by parity) passed 2^kTop
    int seg[4];                          // this CTA's share: first row, tile; last row, tile (exclusive)
    int scan[kPgThreads / 32];
    uint32_t tmem_base;
    int abort_flag;
};
constexpr size_t kSmemBytes = kOffMisc + ((sizeof(Misc) + 15) / 16) * 16;
static_assert(kSmemBytes <= 232448, "shared memory budget");

// mbar_wait in few instructions (the kernel is full of waits, and its code has
// to stay in the instruction cache): the limit counts tries, each of which the
// hardware holds for about 5 us, so it comes after about 2 s too.
constexpr uint32_t kTries = 400000;

__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* err) {
    uint32_t n = 0;
    while (!mbar_try_wait(bar, parity)) {
        if (*abort_flag) return false;
        if (++n > kTries) {
            *abort_flag = 1;
            atomicOr(err, DSA_DEVERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

// ------------------------------------------------------------- 8-bit MMAs
template <uint32_t kAOff, uint32_t kBOff>
__device__ __forceinline__ void umma_f8_at(uint32_t d_tmem, uint64_t a_base, uint64_t b_base, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "add.u64 a, %1, %5;\n\t"
        "add.u64 b, %2, %6;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_base), "l"(b_base), "r"(idesc), "r"(accumulate), "n"(kAOff >> 4), "n"(kBOff >> 4)
        : "memory");
}

// Instruction descriptor of kind::f8f6f4 with a float32 accumulator; A is
// e4m3, B e4m3 or e5m2.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, bool a_mn, bool b_mn, bool b_e5m2) {
    return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Shared-memory descriptor with the 64-byte swizzle.
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (sdesc_sw128(saddr, lbo, sbo) & ~(7ull << 61)) | (4ull << 61);
}

// 16 consecutive columns at two places, one wait for both.
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, float* a, float* b) {
    uint32_t r[16], s[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3]), "=r"(s[4]), "=r"(s[5]), "=r"(s[6]), "=r"(s[7]),
          "=r"(s[8]), "=r"(s[9]), "=r"(s[10]), "=r"(s[11]), "=r"(s[12]), "=r"(s[13]), "=r"(s[14]), "=r"(s[15])
        : "r"(ta), "r"(tb)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        a[i] = __uint_as_float(r[i]);
        b[i] = __uint_as_float(s[i]);
    }
}

// ----------------------------------------------------------- rows and tiles
// Keys of row r, or -1 if its length or selection count is out of range.
template <bool kSparse>
__device__ __forceinline__ int row_keys(const PagedParams& p, int r) {
    const int b = p.T == 1 ? r : r / p.T;
    const int len = __ldg(p.seq_len + b);
    if (len < 0 || static_cast<long long>(len) > (static_cast<long long>(p.max_pages) << p.page_shift)) return -1;
    if (kSparse) {
        const int n = __ldg(p.n_sel + r);
        return n < 0 || n > p.k_max ? -1 : n;
    }
    const int n = len - (p.T - 1 - (r - b * p.T));
    return n < 0 ? 0 : n;
}

// Tiles of a row of n keys; an empty or bad row runs one (masked, NaN) tile.
__device__ __forceinline__ int tiles_of(int n) { return n <= 128 ? 1 : (n + 127) >> 7; }

// The CTA's share of all tiles, by every thread: a scan of the rows' tile
// counts, then the two borders of the share, each found by the thread whose
// rows hold it.  A border is a row and a tile before which it lies.
template <bool kSparse>
__device__ void find_share(const PagedParams& p, Misc& ms) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.R + kPgThreads - 1) / kPgThreads;
    const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
    int sum = 0;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) sum += tiles_of(row_keys<kSparse>(p, r));
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) ms.scan[warp] = incl;
    __syncthreads();
    int before = 0, total = 0;
    // (a lane a warp's sum)
    const int part = lane < kPgThreads / 32 ? ms.scan[lane] : 0;
    total = __reduce_add_sync(0xffffffffu, part);
    before = __reduce_add_sync(0xffffffffu, lane < warp ? part : 0);
    const int first = before + incl - sum, end = first + sum;
    const int ctas = min(static_cast<int>(gridDim.x), total);
    // the borders lie share tiles apart, the first `more` of them one more
    const int share = total / ctas, more = total - share * ctas, slack = share / 8;
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
        const int c = static_cast<int>(blockIdx.x) + e;
        if (c >= ctas) {
            if (tid == 0) {
                ms.seg[2 * e] = p.R;
                ms.seg[2 * e + 1] = 0;
            }
            continue;
        }
        const int x = c * share + min(c, more);
        if (x >= first && x < end) {
            int f = first, r = r0, t = 0;
#pragma unroll 1
            for (; r < r1; ++r) {
                t = tiles_of(row_keys<kSparse>(p, r));
                if (x < f + t) break;
                f += t;
            }
            int at = x - f;
            if (at <= slack && at * 2 <= t) at = 0;
            else if (t - at <= slack) {
                at = 0;
                ++r;
            }
            ms.seg[2 * e] = r;
            ms.seg[2 * e + 1] = at;
        }
    }
}

// ------------------------------------------------------------- index warp
// Positions -> cache rows for the tiles of the share, four keys a lane.
template <bool kSparse>
__device__ void index_role(const PagedParams& p, Misc& ms, int lane) {
    volatile int* ab = &ms.abort_flag;
    const int r_end = ms.seg[2], t_end = ms.seg[3];
    int r = ms.seg[0], t = ms.seg[1], g = 0;
#pragma unroll 1
    for (int nu = 0; r < r_end || (r == r_end && t < t_end); ++nu, ++r, t = 0) {
        const int n = row_keys<kSparse>(p, r), tiles = tiles_of(n);
        const int t1 = r == r_end ? t_end : tiles;
        const bool last_unit = r == r_end || (r + 1 == r_end && t_end == 0);
        const int seq = p.T == 1 ? r : r / p.T;
        const int* table = p.page_table + static_cast<size_t>(seq) * p.max_pages;
        const int len = __ldg(p.seq_len + seq);
        if (lane == 0) {
            ms.unit[nu & (kUnits - 1)][0] = r;
            ms.unit[nu & (kUnits - 1)][1] = (last_unit ? kEnd : 0) | (t == 0 && t1 == tiles ? kWhole : 0) | (n == 0 ? kEmpty : 0) | (t > 0 ? kInside : 0);
            mbar_arrive(smem_addr(&ms.unit_full[nu & (kUnits - 1)]));
            if (n < 0) {
                const bool seq_bad = len < 0 || static_cast<long long>(len) > (static_cast<long long>(p.max_pages) << p.page_shift);
                atomicOr(p.err, seq_bad ? DSA_DEVERR_SEQ_RANGE : DSA_DEVERR_NSEL_RANGE);
            }
        }
        int left = kFirstDown, downs = 0;        // tiles until the references go down next, and how often they have
#pragma unroll 1
        for (int tt = t; tt < t1; ++tt, ++g, --left) {
            // positions (-1: no key, -2: bad; a bad row has one bad key)
            int cur[4], page[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = tt * 128 + lane + 32 * i;
                if (j >= n) cur[i] = n < 0 && j == 0 ? -2 : -1;
                else cur[i] = kSparse ? __ldg(p.idx + static_cast<size_t>(r) * p.k_max + j) : j;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (kSparse && tt * 128 + lane + 32 * i < n && (cur[i] < 0 || cur[i] >= len)) {
                    cur[i] = -2;
                    atomicOr(p.err, DSA_DEVERR_IDX_RANGE);
                }
                page[i] = cur[i] >= 0 ? __ldg(table + (cur[i] >> p.page_shift)) : 0;
            }
            const int slot = g & (kRing - 1);
            if (g >= kRing && !paged_wait(smem_addr(&ms.ring_free[slot]), ((g / kRing) - 1) & 1, ab, p.err)) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (cur[i] >= 0) {
                    if (page[i] >= 0 && page[i] < p.n_pages) {
                        cur[i] = (page[i] << p.page_shift) + (cur[i] & ((1 << p.page_shift) - 1));
                    } else {
                        cur[i] = -2;
                        atomicOr(p.err, DSA_DEVERR_PAGE_RANGE);
                    }
                }
            }
            int go = 0;
            if (left == 0) {
                go = downs < kDowns ? kLower : kRenew;
                left = kFirstDown << downs;
                downs += downs < kDowns ? 1 : 0;
            }
            // a place without a usable key loads the row of the tile's first key (a
            // NaN there is the row's own), marked as its complement
            const int first = max(__shfl_sync(0xffffffffu, cur[0], 0), 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) ms.row[slot][lane + 32 * i] = cur[i] >= 0 ? cur[i] : ~first;
            if (lane == 0)
                *reinterpret_cast<int4*>(ms.tile[slot]) =
                    make_int4(n < 0 ? 1 : min(n - tt * 128, 128),
                              (tt == t ? kFirst : 0) | (tt + 1 == t1 ? kLast | (last_unit ? kEnd : 0) : 0) | go | downs << kLoweredShift,
                              0, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ms.ring_full[slot]));
        }
    }
}

// ----------------------------------------------------------- gather warps
// Four rows of the cache, 128 columns of each, into 512 bytes of a tile.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const void* tmap, int col, int4 rows, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(tmap), "r"(col), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(bar)
        : "memory");
}

// A selection: lane l of warp gw copies 16 bytes of each 128-byte column
// segment of two keys of each quarter of a tile, as soon as the quarter's last
// reader is done.
__device__ void gather_selected(const PagedParams& p, uint8_t* smem, Misc& ms, int gw, int lane) {
    volatile int* ab = &ms.abort_flag;
    const int cc = lane & 7, jr = 4 * gw + (lane >> 3);          // the key in half a quarter
    const uint8_t* src0 = p.cache + cc * 16;
    const uint32_t dst0 = smem_addr(smem + kOffKv) + jr * 128 + ((cc ^ (jr & 7)) << 4);
    for (int g = 0;; ++g) {
        const int slot = g & (kRing - 1), stage = g & 1;
        if (!paged_wait(smem_addr(&ms.ring_full[slot]), (g / kRing) & 1, ab, p.err)) return;
        const int flags = ms.tile[slot][1];
        const uint32_t dst1 = dst0 + stage * kStageBytes;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
            const int r0 = ms.row[slot][32 * q + jr], r1 = ms.row[slot][32 * q + 16 + jr];
            const uint8_t* s0 = src0 + static_cast<size_t>(r0 ^ (r0 >> 31)) * kD;
            const uint8_t* s1 = src0 + static_cast<size_t>(r1 ^ (r1 >> 31)) * kD;
            if (g >= 2 && !paged_wait(smem_addr(&ms.kv_free[stage][q]), ((g >> 1) - 1) & 1, ab, p.err)) return;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                cp_async16(dst1 + q * 4096 + s * kSegBytes, s0 + s * 128, 16u);
                cp_async16(dst1 + q * 4096 + 2048 + s * kSegBytes, s1 + s * 128, 16u);
            }
        }
        cp_async_arrive(smem_addr(&ms.kv_full[stage]));
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ms.ring_free[slot]));
        if (flags & kEnd) return;
    }
}

// A whole context: warp gw brings column segment gw, in boxes of the 16 rows
// that sixteen positions take in their page; where a context ends inside them,
// by gathers of four rows.
__device__ void gather_context(const PagedParams& p, uint8_t* smem, Misc& ms, int gw) {
    volatile int* ab = &ms.abort_flag;
    const uint32_t dst0 = smem_addr(smem + kOffKv) + gw * kSegBytes;
    int g = 0;
    bool ok = true;
    for (;; ++g) {
        const int slot = g & (kRing - 1), stage = g & 1;
        ok = paged_wait(smem_addr(&ms.ring_full[slot]), (g / kRing) & 1, ab, p.err);
        if (!ok) break;
        const int flags = ms.tile[slot][1];
        const uint32_t bar = smem_addr(&ms.kv_full[stage]), dst1 = dst0 + stage * kStageBytes;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const int4* rows = reinterpret_cast<const int4*>(&ms.row[slot][16 * i]);
            const int first = rows[0].x, last = rows[3].w;
            if (g >= 2 && (i & 1) == 0) ok = ok && paged_wait(smem_addr(&ms.kv_free[stage][i >> 1]), ((g >> 1) - 1) & 1, ab, p.err);
            if (!ok) break;
            // (the stage's barrier is in this tile's phase: its last tile has been read)
            if (i == 0) mbar_arrive_expect_tx(bar, kSegBytes);
            if (first >= 0 && last == first + 15) {
                tma_load_2d(dst1 + i * 2048, &p.tmap_box, gw * 128, first, bar);
            } else {
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {
                    int4 r = rows[j];
                    r.x ^= r.x >> 31;
                    r.y ^= r.y >> 31;
                    r.z ^= r.z >> 31;
                    r.w ^= r.w >> 31;
                    tma_gather4(dst1 + i * 2048 + j * 512, &p.tmap, gw * 128, r, bar);
                }
            }
        }
        if (!ok) break;
        mbar_arrive(smem_addr(&ms.ring_free[slot]));
        if (flags & kEnd) break;
    }
    if (ok) ++g;
    // the copies of the tiles issued have landed before the CTA can exit (a
    // tile cut short by an abort has boxes that were never issued: its copies
    // are given the wait limit)
    int dummy = 0;
    if (g > 1) paged_wait(smem_addr(&ms.kv_full[g & 1]), ((g - 2) >> 1) & 1, &dummy, p.err);
    if (g > 0) paged_wait(smem_addr(&ms.kv_full[(g - 1) & 1]), ((g - 1) >> 1) & 1, &dummy, p.err);
    if (!ok) {
        dummy = 0;
        paged_wait(smem_addr(&ms.kv_full[g & 1]), (g >> 1) & 1, &dummy, p.err);
    }
}

// ------------------------------------------------------------------- MMA
// S^T = codes x [q_hi | q_lo], a segment of 128 columns: 4 steps of 32.
__device__ __forceinline__ void score_segment(uint32_t d, uint64_t dK, uint64_t dQ, uint32_t acc) {
    constexpr uint32_t id = idesc_f8(128, 128, false, false, false);
    umma_f8_at<0, 0>(d, dK, dQ, id, acc);
    umma_f8_at<32, 32>(d, dK, dQ, id, 1u);
    umma_f8_at<64, 64>(d, dK, dQ, id, 1u);
    umma_f8_at<96, 96>(d, dK, dQ, id, 1u);
}

// O^T += V^T x W for 32 keys, 128 columns at a time, hi and lo terms into the
// same accumulator.
__device__ __forceinline__ void pv_step(uint32_t tmem, uint64_t dV, uint64_t dHi, uint64_t dLo, uint32_t acc) {
    constexpr uint32_t id4 = idesc_f8(128, 64, true, true, false), id5 = idesc_f8(128, 64, true, true, true);
    umma_f8_at<0 * kSegBytes, 0>(tmem + tmem_o(0), dV, dHi, id4, acc);
    umma_f8_at<0 * kSegBytes, 0>(tmem + tmem_o(0), dV, dLo, id5, 1u);
    umma_f8_at<1 * kSegBytes, 0>(tmem + tmem_o(1), dV, dHi, id4, acc);
    umma_f8_at<1 * kSegBytes, 0>(tmem + tmem_o(1), dV, dLo, id5, 1u);
    umma_f8_at<2 * kSegBytes, 0>(tmem + tmem_o(2), dV, dHi, id4, acc);
    umma_f8_at<2 * kSegBytes, 0>(tmem + tmem_o(2), dV, dLo, id5, 1u);
    umma_f8_at<3 * kSegBytes, 0>(tmem + tmem_o(3), dV, dHi, id4, acc);
    umma_f8_at<3 * kSegBytes, 0>(tmem + tmem_o(3), dV, dLo, id5, 1u);
}

template <bool kSparse>
__device__ void mma_role(const PagedParams& p, uint8_t* smem, Misc& ms, uint32_t tmem) {
    volatile int* ab = &ms.abort_flag;
    const uint32_t sKv = smem_addr(smem + kOffKv), sP = smem_addr(smem + kOffP);
    const uint64_t dQ = sdesc_sw128(smem_addr(smem + kOffQ), 16, 1024);
    const uint64_t dHi = sdesc_sw64(sP, 512, 512), dLo = sdesc_sw64(sP + kPPlane, 512, 512);
    // the scores run up to one tile ahead of the value product: gs tiles (us
    // units) are scored, gp accumulated; fs and fp are the flags of the last tile
    // scored and of the next to accumulate
    int gs = 0, us = 0, gp = 0, nu = 0, fs = 0, fp = 0;
    bool first = true, more = true;
    uint32_t n = 0;
    while (true) {
        // the next tile's scores, as soon as its keys, its unit's Q and a buffer are there
        if (more && gs <= gp + 1) {
            const int slot = gs & (kRing - 1), st = gs & 1;
            if (mbar_try_wait_for(smem_addr(&ms.ring_full[slot]), (gs / kRing) & 1, 20u)) {
                const int f = *reinterpret_cast<volatile int*>(&ms.tile[slot][1]);
                if ((!(f & kFirst) || mbar_try_wait_for(smem_addr(&ms.q_full), us & 1, 20u)) &&
                    (gs < 2 || mbar_try_wait_for(smem_addr(&ms.s_free[st]), ((gs >> 1) - 1) & 1, 20u)) &&
                    mbar_try_wait_for(smem_addr(&ms.kv_full[st]), (gs >> 1) & 1, 20u)) {
                    mbar_arrive(smem_addr(&ms.ring_free[slot]));
                    mbar_arrive(smem_addr(&ms.s_full[st]));
                    if (kSparse) fence_proxy_async();        // (cp.async writes through the generic proxy)
                    tc_fence_after();
                    const uint64_t dK = sdesc_sw128(sKv + st * kStageBytes, 16, 1024);
#pragma unroll 1
                    for (uint32_t e = 0; e < 4; ++e)
                        score_segment(tmem + tmem_s(st), dK + e * (kSegBytes >> 4), dQ + e * (kSegBytes >> 4), e);
                    umma_commit(smem_addr(&ms.s_full[st]));
                    fp = gs == gp ? f : fp;
                    fs = f;
                    ++gs;
                    if (f & kLast) {
                        umma_commit(smem_addr(&ms.q_free));
                        ++us;
                    }
                    more = !(f & kEnd);
                    n = 0;
                }
            }
        }
        // the value product of the tile whose weights are there; a unit's first
        // one overwrites O: the last one has been read
        if (gs > gp && mbar_try_wait_for(smem_addr(&ms.p_full), gp & 1, 20u) &&
            (!first || nu == 0 || mbar_try_wait_for(smem_addr(&ms.o_free), (nu - 1) & 1, 20u))) {
            const int st = gp & 1;
            tc_fence_after();
            const uint64_t dV = sdesc_sw128(sKv + st * kStageBytes, kSegBytes, 1024);
#pragma unroll 1
            for (uint32_t kk = 0; kk < 4; ++kk) {
                pv_step(tmem, dV + kk * (4096 >> 4), dHi + kk * (2048 >> 4), dLo + kk * (2048 >> 4), first && kk == 0 ? 0u : 1u);
                umma_commit(smem_addr(&ms.kv_free[st][kk]));
            }
            umma_commit(smem_addr(&ms.pv_done));
            first = (fp & kLast) != 0;
            if (first) {
                umma_commit(smem_addr(&ms.o_full));
                ++nu;
            }
            if (fp & kEnd) return;
            ++gp;
            fp = fs;
            n = 0;
            continue;
        }
        if (*ab) return;
        // (each round of tries takes a fraction of a microsecond)
        if (++n > 8 * kTries) {
            *ab = 1;
            atomicOr(p.err, DSA_DEVERR_TIMEOUT);
            return;
        }
    }
}

// ------------------------------------------------------- Q in two terms
// Splits a head of Q into the two e4m3 terms.  Lane l holds columns
// [16 l, 16 l + 16): one 16-byte chunk of each term.
__device__ __forceinline__ void split_head(uint8_t* dst, float* q_scale, const uint4& v0, const uint4& v1, int h, int lane,
                                           float scale_log2) {
    uint32_t wd[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint32_t top2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top2 = __vmaxu2(top2, wd[i] & 0x7FFF7FFFu);
    uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 & 0xFFFFu, top2 >> 16));
    if (top >= 0x7F80u) {
        // an element is not finite: it becomes NaN and does not count
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t u0 = wd[i] & 0x7FFFu, u1 = (wd[i] >> 16) & 0x7FFFu;
            top = max(top, max(u0 < 0x7F80u ? u0 : 0u, u1 < 0x7F80u ? u1 : 0u));
            if (u0 >= 0x7F80u) wd[i] = (wd[i] & 0xFFFF0000u) | 0x7FC0u;
            if (u1 >= 0x7F80u) wd[i] = (wd[i] & 0xFFFFu) | 0x7FC00000u;
        }
        top = __reduce_max_sync(0xffffffffu, top);
    }
    // the largest element becomes 2^7 .. 2^8 (e4m3 ends at 448)
    const int e = max(static_cast<int>(top >> 7) - 127, -100);
    const float f = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t hw = 0, lw = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t u = wd[2 * i + k];
            const float a = __uint_as_float(u << 16) * f, b = __uint_as_float(u & 0xFFFF0000u) * f;
            // fp16 holds the 8 bits of these elements down to 2^-21 of the largest
            const __half2 v = __floats2half2_rn(a, b);
            const __nv_fp8x2_storage_t c = __nv_cvt_halfraw2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
            const __half2 r = __hsub2(v, __half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
            const __nv_fp8x2_storage_t d = __nv_cvt_halfraw2_to_fp8x2(__hmul2(r, __half2(__float2half(32.0f), __float2half(32.0f))),
                                                                       __NV_SATFINITE, __NV_E4M3);
            hw |= static_cast<uint32_t>(c) << (16 * k);
            lw |= static_cast<uint32_t>(d) << (16 * k);
        }
        hi[i] = hw;
        lo[i] = lw;
    }
    const uint32_t pc = static_cast<uint32_t>((lane & 7) ^ (h & 7)) << 4;     // h + 64 has the same low bits
    *reinterpret_cast<uint4*>(dst + h * 128 + pc) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(dst + (64 + h) * 128 + pc) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (lane == 0) q_scale[h] = __uint_as_float(static_cast<uint32_t>(127 + e - 7) << 23) * scale_log2;
}

// Splits heads h, h + step, ... below h_end of row r, unit nu's.  The caller
// has seen the last scores of unit nu - 1 complete.
template <int kUnroll>
__device__ __forceinline__ void split_heads(const PagedParams& p, uint8_t* smem, int r, int nu, int h, int step, int h_end) {
    Misc& ms = *reinterpret_cast<Misc*>(smem + kOffMisc);
    const int lane = threadIdx.x & 31;
    uint8_t* dst = smem + kOffQ + (lane >> 3) * kSegBytes;
    const uint4* src = reinterpret_cast<const uint4*>(p.q + static_cast<size_t>(r) * p.H * kD) + 2 * lane;
    const int last = min(h_end, p.H) - 1;
    if (h > last) return;
    // each head's loads are issued two heads ahead
    const uint4* at = src + h * (kD / 8);
    uint4 n0 = __ldg(at), n1 = __ldg(at + 1);
    at = src + min(h + step, last) * (kD / 8);
    uint4 m0 = __ldg(at), m1 = __ldg(at + 1);
#pragma unroll kUnroll
    for (; h <= last; h += step) {
        const uint4 v0 = n0, v1 = n1;
        n0 = m0;
        n1 = m1;
        at = src + min(h + 2 * step, last) * (kD / 8);
        m0 = __ldg(at);
        m1 = __ldg(at + 1);
        split_head(dst, ms.q_scale[nu & 3], v0, v1, h, lane, p.scale * kLog2e);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ms.q_full));
    }
}

// --------------------------------------------------------------- softmax
// Two float32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float2 a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t r) {
    float2 a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
    return a;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pack2(a)), "l"(pack2(b)), "l"(pack2(c)));
    return unpack2(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack2(a)), "l"(pack2(b)));
    return unpack2(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack2(a)), "l"(pack2(b)));
    return unpack2(d);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Sum 32 per-lane values over the warp's lanes: lane l ends with the sum of
// value l.  Fixed order.
__device__ __forceinline__ float transpose_sum32(float* v, int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < o) {
                const float send = up ? v[i] : v[i + o];
                const float keep = up ? v[i + o] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
    }
    return v[0];
}

// The same for maxima (NaN counts as nothing).
__device__ __forceinline__ float transpose_max32(float* v, int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < o) {
                const float send = up ? v[i] : v[i + o];
                const float keep = up ? v[i + o] : v[i];
                v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, o));
            }
        }
    }
    return fmaxf(v[0], -INFINITY);
}

// Floats as integers in the same order, and back (NaN aside).
__device__ __forceinline__ int ordered_int(float f) {
    const int i = __float_as_int(f);
    return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float ordered_float(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF)); }
constexpr int kOrderedNegInf = static_cast<int>(0x807FFFFFu);       // ordered_int(-inf)

__device__ __forceinline__ bool group_sync(Misc& ms, uint32_t& phase, uint32_t* err) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&ms.red_sync));
    const bool ok = paged_wait(smem_addr(&ms.red_sync), phase, &ms.abort_flag, err);
    phase ^= 1u;
    return ok;
}

// x_j - m_h of this thread's key for its 32 heads (in pairs); refs holds -m_h.
__device__ __forceinline__ void load_x(uint32_t ts, const float* qs, const float* refs, float sig, float lsig, float2* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float hi[16], lo[16];
        tmem_ld16x2(ts + 16 * i, ts + 64 + 16 * i, hi, lo);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 f = *reinterpret_cast<const float4*>(qs + 16 * i + 4 * e), r = *reinterpret_cast<const float4*>(refs + 16 * i + 4 * e);
            const float2 fs[2] = {make_float2(f.x, f.y), make_float2(f.z, f.w)}, rs[2] = {make_float2(r.x, r.y), make_float2(r.z, r.w)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = 4 * e + 2 * h;
                const float2 v = mul2(fma2(make_float2(lo[k], lo[k + 1]), both(0.03125f), make_float2(hi[k], hi[k + 1])), fs[h]);
                x[8 * i + 2 * e + h] = fma2(v, both(sig), add2(rs[h], both(lsig)));
            }
        }
    }
}

// Moves the references of the heads whose largest weight over the tile's 128
// keys passes 2^kTop (on a unit's first tile: all), so that it becomes 2^base; on
// a tile where `base` has grown by 1 the others go down by that, on one that
// renews them those whose largest weight is below 2^base go down to it.  The sums
// follow, and behind the first tile rescale_o() has to.  x is used up.  red: this
// move's maxima, which were reset two moves ago.  Lane h works out head h's move;
// the warp reads the factors back four at a time.
__device__ __forceinline__ bool move_refs(const PagedParams& p, Misc& ms, int* red, int* red_reset, int flags, int g,
                                          uint32_t& ph_red, int h0, int lane, float* refs, float2* x, float2* l) {
    const bool is_first = (flags & kFirst) != 0;
    const float base = kBase + (flags >> kLoweredShift), grown = flags & kLower ? 1.0f : 0.0f;
    float v[32];
#pragma unroll
    for (int h = 0; h < 16; ++h) {
        v[2 * h] = x[h].x;
        v[2 * h + 1] = x[h].y;
    }
    atomicMax(red + h0 + lane, ordered_int(transpose_max32(v, lane)));
    if (!group_sync(ms, ph_red, p.err)) return false;
    if (threadIdx.x < 64) red_reset[threadIdx.x] = kOrderedNegInf;
    // (every warp has read the flag)
    if (!is_first && threadIdx.x == 0) *reinterpret_cast<volatile int*>(&ms.move[g & 1]) = 0;
    const float top = ordered_float(red[h0 + lane]);
    // (a tile without a finite score leaves the reference, a first one 0)
    const float was = refs[lane];
    float now = was + grown;
    if (is_first || top + grown > kTop) {
        if (top > -INFINITY) now = was + (base - top);
        refs[64 + lane] = is_first ? now + kDown : fminf(refs[64 + lane], now + kDown);
    } else if ((flags & kRenew) != 0 && top < base && top > -INFINITY) {
        now = fmaxf(was, fminf(was + (base - top), refs[64 + lane]));
    }
    refs[lane] = now;
    refs[32 + lane] = ex2_approx_ftz(now - was);
    __syncwarp();
    if (!is_first) {
#pragma unroll
        for (int h = 0; h < 16; h += 2) {
            const float4 f = *reinterpret_cast<const float4*>(refs + 32 + 2 * h);
            l[h] = mul2(l[h], make_float2(f.x, f.y));
            l[h + 1] = mul2(l[h + 1], make_float2(f.z, f.w));
        }
    }
    return true;
}

// The moved heads' O of the earlier tiles (their value products are done):
// this warp's lanes of it, times the factors.
__device__ __forceinline__ void rescale_o(const float* factors, uint32_t to) {
    tc_fence_after();
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        const uint32_t at = to + tmem_o(i >> 1) + 16 * (i & 1);
        float o[16];
        tmem_ld16(at, o);
#pragma unroll
        for (int h = 0; h < 16; h += 4) {
            const float4 f = *reinterpret_cast<const float4*>(factors + 16 * (i & 1) + h);
            o[h] *= f.x;
            o[h + 1] *= f.y;
            o[h + 2] *= f.z;
            o[h + 3] *= f.w;
        }
        tmem_st16(at, o);
    }
}

// What a softmax thread knows of a tile: its key's scale and what masks it (0,
// -inf for a place without a key, NaN for a bad one), the tile's flags.
struct TileKey {
    float sig, mask;
    int flags;
};

__device__ __forceinline__ bool tile_key(const PagedParams& p, Misc& ms, int g, int key, TileKey& k) {
    const int slot = g & (kRing - 1);
    if (!paged_wait(smem_addr(&ms.ring_full[slot]), (g / kRing) & 1, &ms.abort_flag, p.err)) return false;
    const int2 t = *reinterpret_cast<const int2*>(ms.tile[slot]);
    const int row = ms.row[slot][key];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&ms.ring_free[slot]));
    k.flags = t.y;
    k.sig = row >= 0 ? __ldg(p.cache_scale + (row >> p.block_shift)) : 1.0f;
    k.mask = key >= t.x ? -INFINITY : (row < 0 ? __int_as_float(0x7FC00000) : 0.0f);
    return true;
}

__device__ void softmax_role(const PagedParams& p, uint8_t* smem, Misc& ms, uint32_t tmem) {
    volatile int* ab = &ms.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int qd = warp & 3, h0 = 32 * (warp >> 2), key = 32 * qd + lane;
    const uint32_t ts0 = tmem + (static_cast<uint32_t>(32 * qd) << 16) + h0;
    // this key's row of the weights: 16-byte chunks 2 (warp / 4) and the one after, swizzled
    uint8_t* prow = smem + kOffP + key * 64;
    const int c0 = ((2 * (warp >> 2)) ^ ((key >> 1) & 3)) << 4;
    uint32_t ph_red = 0;
    int nu = 0, red = 2;
    TileKey k;
    // the share's first Q is split by these warps too
    split_heads<1>(p, smem, ms.seg[0], 0, kOutHeads + warp, kSmWarps, kHeadsPad);
    if (!tile_key(p, ms, 0, key, k)) return;
    float* refs = ms.refs[warp];
    float2 l[16];               // sums
    for (int g = 0;; ++g) {
        const int flags = k.flags;
        if (flags & kFirst) {
#pragma unroll
            for (int h = 0; h < 16; ++h) l[h] = make_float2(0.0f, 0.0f);
            refs[lane] = 0.0f;
            __syncwarp();
        }
        const float sig = k.sig, lsig = __log2f(sig) + k.mask;
        // the next tile's scale is on its way meanwhile
        if (!(flags & kEnd) && !tile_key(p, ms, g + 1, key, k)) return;
        const float* qs = &ms.q_scale[nu & 3][h0];
        const uint32_t ts = ts0 + tmem_s(g & 1);
        if (!paged_wait(smem_addr(&ms.s_full[g & 1]), (g >> 1) & 1, ab, p.err)) return;
        tc_fence_after();
        float2 x[16];
        uint32_t hi[8], lo[8];
        // a pass with the references as they are; one for the maxima and
        // another with moved references if a weight passed 2^kTop in any warp (on a
        // unit's first tile, and where references go down, always)
        enum { kTry, kMove, kMoved } pass = flags & (kFirst | kLower | kRenew) ? kMove : kTry;
#pragma unroll 1
        while (true) {
            load_x(ts, qs, refs, sig, lsig, x);
            if (pass == kMove) {
                red = red == 2 ? 0 : red + 1;
                if (!move_refs(p, ms, ms.red[red], ms.red[red == 0 ? 2 : red - 1], flags, g, ph_red, h0, lane, refs, x, l))
                    return;
                pass = kMoved;
                continue;
            }
            if (pass == kTry) {
                float top = fmaxf(x[0].x, x[0].y);
#pragma unroll
                for (int h = 1; h < 16; ++h) top = fmaxf(top, fmaxf(x[h].x, x[h].y));
                const bool passed = __any_sync(0xffffffffu, top > kTop);
                if (lane == 0) {
                    if (passed) *reinterpret_cast<volatile int*>(&ms.move[g & 1]) = 1;
                    mbar_arrive(smem_addr(&ms.red_sync));
                }
            }
            // weights, and their two 8-bit terms, by way of fp16 (11 bits of a
            // weight up to 2^8.75, of which the terms keep 7)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t hw = 0, lw = 0;
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const int h = 2 * e + f;
                    x[h] = make_float2(ex2_approx_ftz(x[h].x), ex2_approx_ftz(x[h].y));
                    const __half2 v = __floats2half2_rn(x[h].x, x[h].y);
                    const __nv_fp8x2_storage_t a = __nv_cvt_halfraw2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
                    const __half2 r = __hsub2(v, __half2(__nv_cvt_fp8x2_to_halfraw2(a, __NV_E4M3)));
                    const __nv_fp8x2_storage_t b = __nv_cvt_halfraw2_to_fp8x2(r, __NV_SATFINITE, __NV_E5M2);
                    hw |= static_cast<uint32_t>(a) << (16 * f);
                    lw |= static_cast<uint32_t>(b) << (16 * f);
                }
                hi[e] = hw;
                lo[e] = lw;
            }
            if (pass == kMoved) break;
            if (!paged_wait(smem_addr(&ms.red_sync), ph_red, ab, p.err)) return;
            ph_red ^= 1u;
            if (!*reinterpret_cast<volatile int*>(&ms.move[g & 1])) break;
            pass = kMove;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ms.s_free[g & 1]));
        const float inv = __fdividef(1.0f, sig);
#pragma unroll
        for (int h = 0; h < 16; ++h) l[h] = fma2(x[h], both(inv), l[h]);
        // the last tile's value product has read P
        if (g > 0 && !paged_wait(smem_addr(&ms.pv_done), (g - 1) & 1, ab, p.err)) return;
        if (pass == kMoved && !(flags & kFirst) && __any_sync(0xffffffffu, refs[32 + lane] != 1.0f))
            rescale_o(refs + 32, ts0);
        *reinterpret_cast<uint4*>(prow + c0) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(prow + (c0 ^ 16)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
        *reinterpret_cast<uint4*>(prow + kPPlane + c0) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4*>(prow + kPPlane + (c0 ^ 16)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ms.p_full));
        if (flags & kLast) {
            // the unit's sums (over this warp's 32 keys) and references, for the output warps
            if (nu > 0 && !paged_wait(smem_addr(&ms.l_free), (nu - 1) & 1, ab, p.err)) return;
            float v[32];
#pragma unroll
            for (int h = 0; h < 16; ++h) {
                v[2 * h] = l[h].x;
                v[2 * h + 1] = l[h].y;
            }
            ms.red_l[qd][h0 + lane] = transpose_sum32(v, lane);
            if (qd == 0) ms.m_ref[h0 + lane] = -refs[lane];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ms.l_ready));
            ++nu;
        }
        if (flags & kEnd) return;
    }
}

// ------------------------------------------------------------ output warps
// 1 / (l + 2^(s2 - m)) of a head: what its value sum (relative to 2^m) is
// multiplied by.  A head without keys and sink gives 0.  Far below the sink the
// value sum may be large enough for a result where the factor is below float32's
// numbers: then -2^64 times the factor is returned, and the value sum takes
// kDeep = -2^-64 first.
constexpr float kDeep = -0x1p-64f;

__device__ __forceinline__ float out_factor(float m, float l, const float* sink, int h) {
    const float s2 = sink ? __ldg(sink + h) * kLog2e : -INFINITY;
    if (s2 == -INFINITY && l == 0.0f) return 0.0f;
    const float ms = isfinite(s2) ? fmaxf(m, s2) : m;
    const float e1 = ex2_approx_ftz(m - ms), e2 = ex2_approx_ftz(s2 - ms);
    return (m - ms < -64.0f ? -ex2_approx_ftz(m - ms + 64.0f) : e1) / fmaf(l, e1, e2);
}

// Value sums of the heads far below their sink (those of negative factors) times
// kDeep, where the output warp will read them: rare, and so apart from its loop.
__device__ __noinline__ void deepen(const float* fac, uint32_t to, int h0, int H) {
#pragma unroll 1
    for (; h0 < H; h0 += 32) {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            float o[16];
            tmem_ld16(to + tmem_o(i) + h0, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] *= fac[h0 + j] < 0.0f ? kDeep : 1.0f;
            tmem_st16(to + tmem_o(i) + h0, o);
        }
    }
}

__device__ void output_role(const PagedParams& p, uint8_t* smem, Misc& ms, uint32_t tmem, int ow, int lane) {
    const int qd = ow & 3;              // TMEM lane quadrant; warps 4-7 take every other 16 heads
    volatile int* ab = &ms.abort_flag;
    const uint32_t lane_off = static_cast<uint32_t>(32 * qd) << 16;
    int row = 0, flags = 0;             // unit nu's
    for (int nu = -1;; ++nu) {
        int row_next = 0, flags_next = 0;
        if (!(flags & kEnd)) {
            // the next unit's Q, as soon as this one's last scores are done
            const int slot = (nu + 1) & (kUnits - 1);
            if (!paged_wait(smem_addr(&ms.unit_full[slot]), ((nu + 1) / kUnits) & 1, ab, p.err)) return;
            row_next = ms.unit[slot][0];
            flags_next = ms.unit[slot][1];
            if (nu >= 0 && !paged_wait(smem_addr(&ms.q_free), nu & 1, ab, p.err)) return;
            split_heads<2>(p, smem, row_next, nu + 1, ow, kOutWarps, nu < 0 ? kOutHeads : kHeadsPad);
            // and the row after it into the L2, 128 bytes a lane and step
            if (!(flags_next & kEnd)) {
                const char* next = reinterpret_cast<const char*>(p.q + static_cast<size_t>(row_next + 1) * p.H * kD);
#pragma unroll 1
                for (int i = (ow * 32 + lane) * 128; i < p.H * kD * 2; i += kOutWarps * 32 * 128)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(next + i));
            }
        }
        if (nu < 0) {
            row = row_next;
            flags = flags_next;
            continue;
        }
        if (!paged_wait(smem_addr(&ms.l_ready), nu & 1, ab, p.err)) return;
        const bool whole = (flags & kWhole) != 0;
        // a row without a key: its one tile holds whatever row the gather took,
        // and nothing of it counts
        const bool empty = (flags & kEmpty) != 0;
        // a share's first unit, if it starts inside its row, is partial 0; the
        // part of a row that the share's end cuts off is partial 1
        float* part = p.part + static_cast<size_t>(2 * blockIdx.x + (flags & kInside ? 0 : 1)) * kPartialFloats;
        bool deep = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = lane + 32 * e;
            const float l = empty ? 0.0f : (ms.red_l[0][h] + ms.red_l[1][h]) + (ms.red_l[2][h] + ms.red_l[3][h]);
            const float m = empty ? 0.0f : ms.m_ref[h];
            if (whole) {
                const float f = h < p.H ? out_factor(m, l, p.sink, h) : 0.0f;
                ms.fac[ow][h] = f;
                deep |= f < 0.0f;
            } else if (ow == 0) {
                part[static_cast<size_t>(kHeadsPad) * kD + h] = m;
                part[static_cast<size_t>(kHeadsPad) * kD + kHeadsPad + h] = l;
            }
        }
        deep = __any_sync(0xffffffffu, deep);
        if (lane == 0) mbar_arrive(smem_addr(&ms.l_free));
        if (!paged_wait(smem_addr(&ms.o_full), nu & 1, ab, p.err)) return;
        tc_fence_after();
        if (deep) deepen(ms.fac[ow], tmem + lane_off, 16 * (ow >> 2), p.H);
        const int d0 = 32 * qd + lane;
        // bf16: neighbouring lanes swap halves of (head j, head j + 1) pairs, so
        // that each stores two neighbouring columns of one head
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (static_cast<size_t>(row) * p.H + (lane & 1)) * kD + (d0 & ~1);
        const uint32_t sel = lane & 1 ? 0x3276u : 0x5410u;
#pragma unroll 1
        for (int h0 = 16 * (ow >> 2); h0 < p.H; h0 += 32) {
            const int hs = p.H - h0;             // heads to store of the 16
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                float o[16];
                tmem_ld16(tmem + lane_off + tmem_o(i) + h0, o);
                if (whole) {
                    __nv_bfloat16* at = dst + h0 * kD + i * 128;
#pragma unroll
                    for (int j4 = 0; j4 < 4; ++j4) {
                        const float4 f = *reinterpret_cast<const float4*>(&ms.fac[ow][h0 + 4 * j4]);
                        const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const int j = 4 * j4 + e;
                            const __nv_bfloat162 v = __floats2bfloat162_rn((empty ? 0.0f : o[j]) * fs[e], (empty ? 0.0f : o[j + 1]) * fs[e + 1]);
                            const uint32_t a = *reinterpret_cast<const uint32_t*>(&v);
                            const uint32_t b = __shfl_xor_sync(0xffffffffu, a, 1);
                            if (j + (lane & 1) < hs) *reinterpret_cast<uint32_t*>(at + j * kD) = __byte_perm(a, b, sel);
                        }
                    }
                } else {
                    float* at = part + h0 * kD + i * 128 + d0;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j < hs) at[j * kD] = o[j];
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ms.o_free));
        if (flags & kEnd) return;
        row = row_next;
        flags = flags_next;
    }
}

// kSparse: the rows' keys are a selection; otherwise their whole context.
template <bool kSparse>
__global__ void __launch_bounds__(kPgThreads, 1) dsa_paged_kernel(const __grid_constant__ PagedParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Misc& ms = *reinterpret_cast<Misc*>(smem + kOffMisc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_launch_dependents();
    if (smem_addr(smem) & 1023u) {   // the swizzle needs 1024-byte alignment
        grid_dependency_wait();
        if (threadIdx.x == 0) atomicOr(p.err, DSA_DEVERR_LAYOUT);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ms.kv_full[i]), kSparse ? 32 * kGatherWarps : kGatherWarps);
            for (int q = 0; q < 4; ++q) mbar_init(smem_addr(&ms.kv_free[i][q]), 1);
            mbar_init(smem_addr(&ms.s_full[i]), 2);
            mbar_init(smem_addr(&ms.s_free[i]), kSmWarps);
            ms.move[i] = 0;
        }
        mbar_init(smem_addr(&ms.p_full), kSmWarps);
        mbar_init(smem_addr(&ms.pv_done), 1);
        mbar_init(smem_addr(&ms.q_full), static_cast<uint32_t>(p.H));
        mbar_init(smem_addr(&ms.q_free), 1);
        mbar_init(smem_addr(&ms.o_full), 1);
        mbar_init(smem_addr(&ms.o_free), kOutWarps);
        mbar_init(smem_addr(&ms.l_ready), kSmWarps);
        mbar_init(smem_addr(&ms.l_free), kOutWarps);
        mbar_init(smem_addr(&ms.red_sync), kSmWarps);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(smem_addr(&ms.ring_full[i]), 1);
            mbar_init(smem_addr(&ms.ring_free[i]), kGatherWarps + kSmWarps + 1);
        }
        for (int i = 0; i < kUnits; ++i) mbar_init(smem_addr(&ms.unit_full[i]), 1);
        mbar_init(smem_addr(&ms.drain), 1);
        ms.abort_flag = 0;
        mbar_fence_init();
        if (!kSparse) prefetch_tmap(&p.tmap_box);
    }
    if (threadIdx.x < 192) ms.red[threadIdx.x >> 6][threadIdx.x & 63] = kOrderedNegInf;
    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(&ms.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    if (p.H < 64) {
        // heads past H: zero rows of both terms, never written again
        for (int e = threadIdx.x; e < (64 - p.H) * 64; e += kPgThreads) {
            const int h = p.H + e / 64, s = (e % 64) / 16, c = e % 8, lo = (e / 8) & 1;
            *reinterpret_cast<uint4*>(smem + kOffQ + s * kSegBytes + (64 * lo + h) * 128 + (c << 4)) = make_uint4(0, 0, 0, 0);
        }
        if (threadIdx.x < 256 && (threadIdx.x & 63) >= p.H) ms.q_scale[threadIdx.x >> 6][threadIdx.x & 63] = 0.0f;
        fence_proxy_async();
    }
    // everything above touched only shared memory and TMEM; the inputs,
    // outputs and workspace may belong to the grid before this one
    grid_dependency_wait();
    find_share<kSparse>(p, ms);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem_base;
    if (threadIdx.x == 0) p.meta[blockIdx.x] = make_int4(ms.seg[0], ms.seg[1], ms.seg[2], ms.seg[3]);

    // (a CTA without a share has nothing to wait for)
    const bool any = ms.seg[0] < ms.seg[2] || (ms.seg[0] == ms.seg[2] && ms.seg[1] < ms.seg[3]);
    if (warp < kSmWarps) {
        regs_inc<kRegsSoftmax>();
        if (any) softmax_role(p, smem, ms, tmem);
        __syncwarp();
    } else if (warp < kOutWarp0 + kOutWarps) {
        regs_dec<kRegsOutput>();
        if (any) output_role(p, smem, ms, tmem, warp - kOutWarp0, lane);
        __syncwarp();
    } else if (warp < kGatherWarp0) {
        regs_dec<kRegsOther>();
        if (warp == kMmaWarp && lane == 0) {
            if (any) mma_role<kSparse>(p, smem, ms, tmem);
            // every MMA this thread issued has completed before TMEM is freed
            umma_commit(smem_addr(&ms.drain));
            int dummy = 0;
            paged_wait(smem_addr(&ms.drain), 0, &dummy, p.err);
        }
        if (warp == kIdxWarp) index_role<kSparse>(p, ms, lane);
        __syncwarp();
    } else {
        regs_dec<kRegsOther>();
        if (kSparse) {
            if (any) gather_selected(p, smem, ms, warp - kGatherWarp0, lane);
            cp_async_wait_all();
        } else if (any && lane == 0) {
            gather_context(p, smem, ms, warp - kGatherWarp0);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Merges the partials of the rows that several CTAs computed.  A row cut by a
// share's border belongs to the share in which it begins; its parts are that
// share's partial 1, then partial 0 of the shares that follow inside it.  A
// work item is such a row and four heads (128 threads each); the blocks find
// the rows from the shares and take items in turn.  One warp a head turns the
// parts' references and sums into weights, then every thread adds its four
// columns over the parts, eight loads in flight.  (One block a share and four
// heads, the references read part by part, took 25 us for 8 rows of 19 parts.)
constexpr int kMergeHeads = 4;
constexpr int kMergeCtas = static_cast<int>(kPagedMaxCtas);

__global__ void __launch_bounds__(128 * kMergeHeads) dsa_paged_combine_kernel(const PagedParams p, int ctas) {
    __shared__ int2 begin_s[kMergeCtas];             // each share's first row and tile
    __shared__ int owner_s[kMergeCtas], count_s[4 * kMergeHeads], owners_s, parts_s;
    __shared__ float w_s[kMergeHeads][kMergeCtas], f_s[kMergeHeads];
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, sub = tid >> 7, col = tid & 127;
    grid_dependency_wait();
    int4 own = make_int4(0, 0, 0, 0);
    if (tid < ctas) {
        own = __ldcg(p.meta + tid);
        begin_s[tid] = make_int2(own.x, own.y);
    }
    // a share that cuts a row which begins in it
    const bool is_owner = tid < ctas && own.w > 0 && !(own.x == own.z && own.y > 0);
    // (every block lists them in the same order)
    const unsigned owners = __ballot_sync(0xffffffffu, is_owner);
    if (lane == 0) count_s[tid >> 5] = __popc(owners);
    __syncthreads();
    if (is_owner) {
        int at = __popc(owners & ((1u << lane) - 1u));
        for (int w = 0; w < (tid >> 5); ++w) at += count_s[w];
        owner_s[at] = tid;
    }
    if (tid == 0) {
        int n = 0;
        for (int w = 0; w < 4 * kMergeHeads; ++w) n += count_s[w];
        owners_s = n;
    }
    __syncthreads();
    const int groups = (p.H + kMergeHeads - 1) / kMergeHeads, items = owners_s * groups;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int c = owner_s[item / groups], h = (item % groups) * kMergeHeads + sub;
        const int row = __ldcg(p.meta + c).z;
        __syncthreads();                             // (the item before is done with w_s, parts_s)
        if (tid < 32) {
            // the run of shares behind c that begin inside the row
            int n = 0;
            for (bool go = true; go; n += 32) {
                const int i = c + 1 + n + lane;
                const unsigned stop = __ballot_sync(0xffffffffu, !(i < ctas && begin_s[i].x == row && begin_s[i].y > 0));
                if (stop) {
                    n += __ffs(stop) - 1 - 32;
                    go = false;
                }
            }
            if (lane == 0) parts_s = 1 + n;
        }
        __syncthreads();
        const int parts = parts_s;
        auto at = [&](int i) { return p.part + static_cast<size_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * kPartialFloats; };
        if ((tid & 127) < 32 && h < p.H) {
            // (a part without a finite score has l = 0: its reference says nothing)
            float M = -INFINITY, l = 0.0f;
            for (int i = lane; i < parts; i += 32) {
                const float m = __ldcg(at(i) + kHeadsPad * kD + h), li = __ldcg(at(i) + kHeadsPad * kD + kHeadsPad + h);
                w_s[sub][i] = li == 0.0f ? -INFINITY : m;
                M = fmaxf(M, w_s[sub][i]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            if (M == -INFINITY) M = 0.0f;
            for (int i = lane; i < parts; i += 32) {
                const float w = exp2f(w_s[sub][i] - M);
                w_s[sub][i] = w;
                l = fmaf(w, __ldcg(at(i) + kHeadsPad * kD + kHeadsPad + h), l);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (lane == 0) f_s[sub] = out_factor(M, l, p.sink, h);
        }
        __syncthreads();
        if (h >= p.H) continue;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < parts; i0 += 8) {
            float4 o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i0 + j < parts) o[j] = __ldcg(reinterpret_cast<const float4*>(at(i0 + j) + static_cast<size_t>(h) * kD) + col);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (i0 + j < parts) {
                    const float w = w_s[sub][i0 + j];
                    acc.x = fmaf(w, o[j].x, acc.x);
                    acc.y = fmaf(w, o[j].y, acc.y);
                    acc.z = fmaf(w, o[j].z, acc.z);
                    acc.w = fmaf(w, o[j].w, acc.w);
                }
            }
        }
        const float f = f_s[sub], pre = f < 0.0f ? kDeep : 1.0f;
        __nv_bfloat162* o2 = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + (static_cast<size_t>(row) * p.H + h) * kD) + 2 * col;
        o2[0] = __floats2bfloat162_rn(acc.x * pre * f, acc.y * pre * f);
        o2[1] = __floats2bfloat162_rn(acc.z * pre * f, acc.w * pre * f);
    }
}

std::mutex g_paged_mu;

PFN_cuTensorMapEncodeTiled_v12000 paged_encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static bool tried = false;
    std::lock_guard<std::mutex> lock(g_paged_mu);
    if (!tried) {
        tried = true;
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    return fn;
}

// The cache as a matrix of rows of 512 bytes, read in boxes of 128 columns and
// box_rows rows (one for the gathers) with the 128-byte swizzle.
bool encode_cache(CUtensorMap* m, const void* base, uint64_t rows, uint32_t box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = paged_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(kD)};
    cuuint32_t box[2] = {128, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_paged(const PagedParams& params, void* workspace, int max_keys, int sms, cudaStream_t s) {
    static bool attr_set[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(g_paged_mu);
        if (!attr_set[dev]) {
            e = cudaFuncSetAttribute(dsa_paged_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
            if (e != cudaSuccess) return e;
            e = cudaFuncSetAttribute(dsa_paged_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
            if (e != cudaSuccess) return e;
            attr_set[dev] = true;
        }
    }
    const int row_tiles = static_cast<int>((static_cast<long long>(max_keys) + 127) / 128);
    const long long tiles = static_cast<long long>(params.R) * row_tiles;
    long long ctas = kPagedMaxCtas < sms ? kPagedMaxCtas : sms;
    if (tiles < ctas) ctas = tiles;
    PagedParams p = params;
    if (!p.idx) {
        // (a selection's rows are not copied by TMA)
        const uint64_t rows = static_cast<uint64_t>(p.n_pages) << p.page_shift;
        if (!encode_cache(&p.tmap, p.cache, rows, 1) || !encode_cache(&p.tmap_box, p.cache, rows, 16))
            return cudaErrorInvalidValue;
    }
    p.meta = static_cast<int4*>(workspace);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ctas * 256);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kPgThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = p.idx ? cudaLaunchKernelEx(&cfg, dsa_paged_kernel<true>, p) : cudaLaunchKernelEx(&cfg, dsa_paged_kernel<false>, p);
    if (e != cudaSuccess || row_tiles == 1) return e;    // rows of one tile are never cut
    // (no more rows are cut than there are rows, or borders between shares)
    const long long items = (params.R < ctas ? params.R : ctas) * static_cast<long long>((p.H + kMergeHeads - 1) / kMergeHeads);
    cfg.gridDim = dim3(static_cast<unsigned>(items < 4LL * sms ? items : 4LL * sms));
    cfg.blockDim = dim3(128 * kMergeHeads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, dsa_paged_combine_kernel, p, static_cast<int>(ctas));
}

}  // namespace dsa
