// Softmax cross entropy of a linear head on sm_103a tensor cores, in pieces of
// the vocabulary, without keeping the logits.
//
//   z[i, j]  = scale * sum_k x[i, k] * w[j, k]             (BF16 products, FP32 sums)
//   lse[i]   = log sum_j exp(z[i, j])
//   loss[i]  = lse[i] - z[i, t_i]                          (0 where t_i is outside [0, v))
//   d[i, j]  = (exp(z[i, j] - lse[i]) - [j = t_i]) * dloss[i]
//   dx       = scale * d w,   dw = scale * d^T x
//
// One GEMM kernel (k_head_gemm) in four modes carries all of it:
//   forward    x w^T with an epilogue that reduces each row's 128 logits to a
//              (maximum, sum of exponentials) pair without the target's term; a
//              small kernel joins the pairs of a row and its target's logit
//   backward, from a copy of x in rows of whole lines (zero without a loss) and
//   each row's d at its target, per piece of the vocabulary (its d is [n x piece]
//   in BF16)
//     1. x w^T again with an epilogue that writes d
//     2. dx += d w: d K-major, w with its N axis (c) contiguous; FP32 slabs
//        in the workspace, one per K split, added to by TMA add-reductions
//     3. dw = d^T x: both operands with their M / N axis contiguous
//   and a last kernel that sums the slabs into BF16 dx.
//
// d is rounded to BF16 once (the tensor core's operand type), scaled by the
// largest |dloss| so that it is O(1) whatever the loss's normalisation, and a
// uniform dloss adds no rounding of its own; sums, softmax statistics, dx
// across pieces and dw stay in FP32 until their one final rounding.  The sums of
// the backward products stay in the tensor core, whose FP32 accumulator
// truncates: within 1e-5 of the sum of magnitudes, where d's rounding is 4e-3 of
// each term.
//
// What bounds it.  Batches: the tensor cores.  Two CTAs of a cluster share a
// 256 x 256 tile (cta_group::2): per 64 columns of K each loads 32 KB for 512
// tensor cycles, where a single CTA's 128 x 256 tile needs 48 KB, more than an
// SM's 64 bytes a cycle from L2.  The tile's FP32 sums are double-buffered in
// TMEM, so the epilogue works under the next tile's products.  4096 tokens x
// 131072 x 4096, back to back: forward 2.58 to 2.67 ms (1.65 to 1.70 PFLOP/s),
// backward 7.6 to 7.9 ms with dw in BF16 (1.69 to 1.73 PFLOP/s, 0.97 to 1.0 of the
// rate cuBLAS sustains under the power cap), 2% more in FP32 and 3 to 5% more where
// it adds into dw.  Few tokens: the weight's stream from HBM (one token x 32000 x
// 4096: 48.5 us for 262 MB).  Widths just past a tile cost the most: 1000 x 50257 x
// 1032 backward takes 280 us (1.11 PFLOP/s), 249 at 1024 columns and 292 at 1280,
// since dx and dw run five tiles of 256 for 4.03; rows of w and dw off the 128-byte
// lines are 4% of it (271 us with both in lines).
//
// The target's term is left out of the sum of exponentials and joined at the
// end: loss = log1p(sum of the others / the target's) where the target leads,
// so a confident token's loss keeps its relative precision.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "head_rows.cuh"
#include "jetq_internal.h"
#include "ptx.cuh"

namespace jetq {

__device__ unsigned g_linear_ce_error;

namespace {

constexpr unsigned kErrTimeout = 1u;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

constexpr int kParts = 2; // the statistics epilogue's column slices of a tile

enum HeadMode : int {
    kStats = 0,    // softmax statistics of the logits
    kGrad = 1,     // d in BF16
    kGradX = 2,    // FP32 slabs of dx
    kGradW16 = 3,  // dw in BF16
    kGradW32 = 4,  // dw in FP32
    kStatsSkip = 5 // kStats without the columns that each row marks
};

__host__ __device__ constexpr bool is_stats(int mode)
{
    return mode == kStats || mode == kStatsSkip;
}

struct HeadParams {
    int mt, nt, splits, num_kb, group; // tiles of M and N, splits and 64-blocks of K, M tiles per raster group
    int64_t M, N;                      // valid rows and columns of the output
    int bn;                            // columns a tile (kStats; else 256)
    int box_a, stages;                 // FEW: rows of A's box, ring stages of box_a rows of A and B's rows
    float k2;                          // scale * log2(e): exponents in base 2
    const int64_t *target;
    bool wait_x;                       // kStatsSkip: x comes from the kernel before
    const uint4 *skip;                 // kStatsSkip: a bit a column, [M][kParts * nt] of 128 columns each
    int fold;                          // kStats: 64-blocks of K summed inside the tensor core, see the epilogue
    int64_t V, col0;                   // whole vocabulary; first vocabulary row of this piece
    float2 *part;                      // [kParts * nt][M] (maximum, sum), base 2
    const GradRow *rows;               // kGrad: [M]
    const float *gmax;
    float scale;
    int add;                           // FP32 output: add to what is there
    unsigned long long limit_ns;
};

// FEW: one tile of at most 128 rows by single CTAs.  A's box then holds those
// rows only (the MMA reads on past them: the rows it makes of that are never
// stored), and the ring has as many stages as fit: one token streams the weight
// with 7 stages of 29 KB instead of 4 of 48.
template <int CG, int MODE, bool FEW>
struct HeadCfg {
    static constexpr int BN = 256, BK = 64;
    static constexpr int kABytes = 128 * 128;
    static constexpr int kBRows = BN / CG; // rows of B in one CTA's shared memory
    static constexpr int kBBytes = kBRows * 128;
    static constexpr int kStage = kABytes + kBBytes;
    // Epilogue: 16 warps of 64 columns a thread for d and the gradients; 8 warps of 128 for the statistics,
    // whose threads hold their columns' sums (4 to 10% faster forward than 16 warps of 64, except at c = 256).
    static constexpr int kEpiWarps = is_stats(MODE) ? 8 : 16;
    static constexpr int kCols = is_stats(MODE) ? 128 : 64;
    static constexpr int kThreads = 128 + 32 * kEpiWarps;
    static constexpr bool kStaging = !is_stats(MODE);
    static constexpr size_t kStagingBytes = kStaging ? kEpiWarps * 4096 : 0; // a 4 KB box a warp
    static constexpr int kStages = FEW ? 12 : (int)((225 * 1024 - kStagingBytes) / kStage); // FEW: at most
    static constexpr size_t kTileBytes = FEW ? 225 * 1024 - kStagingBytes : (size_t)kStages * kStage;
    static constexpr size_t kSmem = 1024 + kTileBytes + kStagingBytes + 256;
    static constexpr bool kAMn = MODE == kGradW16 || MODE == kGradW32; // A's M axis contiguous
    static constexpr bool kBMn = kAMn || MODE == kGradX;               // B's N axis contiguous
    // register split of the statistics: producer warps, epilogue warps
    static constexpr bool kRegSplit = is_stats(MODE);
    static constexpr int kRegProducer = 72, kRegEpilogue = 216;
    static constexpr int kBars = 2 * kStages + 5;
    static_assert(kBars * 8 + 8 <= 256, "barrier area");
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(!FEW || (CG == 1 && !kAMn), "one tile of rows, K-major");
};

// Raster: groups of `group` M tiles; inside a group N tiles in turn, M tiles
// fastest; K splits slowest, so that concurrent tiles read the same K range.
__device__ __forceinline__ void head_coords(const HeadParams &p, int t, int &mi, int &ni, int &ks)
{
    const int mn = p.mt * p.nt;
    ks = t / mn;
    t -= ks * mn;
    const int g = t / (p.group * p.nt);
    t -= g * p.group * p.nt;
    const int gm = min(p.group, p.mt - g * p.group);
    ni = t / gm;
    mi = g * p.group + t - ni * gm;
}

template <int CG, int MODE, bool FEW>
__global__ void __launch_bounds__(HeadCfg<CG, MODE, FEW>::kThreads, 1)
    k_head_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmO, const HeadParams p)
{
    using C = HeadCfg<CG, MODE, FEW>;
    constexpr int kBarS = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *tiles = ptx::align_smem<1024>(smem_raw);
    uint8_t *staging = tiles + C::kTileBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(staging + C::kStagingBytes);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const uint32_t bar0 = ptx::smem_addr(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kBarS + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * kBarS + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (2 * kBarS + 2 + b); };
    const uint32_t done = bar0 + 8u * (2 * kBarS + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? ptx::cluster_ctarank() : 0u;
    const int unit = blockIdx.x / CG, units = gridDim.x / CG;
    unsigned *err = &g_linear_ce_error;
    const int num_tiles = p.mt * p.nt * p.splits;
    const int bn = is_stats(MODE) ? p.bn : C::BN;
    const int S = FEW ? p.stages : C::kStages;
    const uint32_t a_bytes = FEW ? (uint32_t)p.box_a * 128u : (uint32_t)C::kABytes;
    const uint32_t stage_bytes =
        FEW ? a_bytes + (C::kBMn ? (uint32_t)C::kBBytes : (uint32_t)bn * 128u) : (uint32_t)C::kStage;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(acc_full(b), 1);
            ptx::mbar_init(acc_empty(b), C::kEpiWarps * CG);
        }
        ptx::mbar_init(done, 1);
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&tmA);
        ptx::prefetch_tensormap(&tmB);
        if (C::kStaging)
            ptx::prefetch_tensormap(&tmO);
    }
    if (warp == 1)
        ptx::tmem_alloc_cg<CG>(ptx::smem_addr(tmem_slot), 512);
    ptx::tc_fence_before();
    if (CG == 2)
        ptx::cluster_sync(); // the peer's barriers are initialized too
    else
        __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    ptx::grid_dep_launch();
    // kStatsSkip: what the product reads was there before the kernel that marks the columns, which let this one
    // start after its own wait; unless that kernel also copies x, only the epilogue needs its result
    if (MODE != kStatsSkip || warp >= 4 || p.wait_x)
        ptx::grid_dep_wait();
    if constexpr (C::kRegSplit) {
        if (warp < 4)
            ptx::setmaxnreg_dec<C::kRegProducer>();
        else
            ptx::setmaxnreg_inc<C::kRegEpilogue>();
    }

    if (warp < 4) {
        if (warp == 0 && lane == 0) {
            // -------------------------------------------------- TMA producer
            const uint32_t tx =
                FEW ? stage_bytes : (is_stats(MODE) ? (uint32_t)(CG * 128 + bn) * 128u : (uint32_t)(CG * C::kStage));
            int s = 0;
            uint32_t ph = 0; // of the ring's pass
            uint32_t it = 0;
            bool ok = true;
            for (int t = unit; t < num_tiles && ok; t += units) {
                int mi, ni, ks;
                head_coords(p, t, mi, ni, ks);
                const int k0 = (int)((int64_t)p.num_kb * ks / p.splits);
                const int k1 = (int)((int64_t)p.num_kb * (ks + 1) / p.splits);
                const int m0 = mi * 128 * CG + (int)rank * 128;
                const int n0 = ni * bn + (int)rank * (bn / CG);
                for (int kb = k0; kb < k1; ++kb, ++it) {
                    if (!ptx::mbar_wait(empty(s), ph ^ 1u, abort_flag, err, kErrTimeout, p.limit_ns)) {
                        ok = false;
                        break;
                    }
                    // the pair's bytes are counted on the even CTA's barrier, whose thread issues the MMAs
                    if (rank == 0)
                        ptx::mbar_arrive_expect_tx(full(s), tx);
                    const uint32_t bar = CG == 2 ? ptx::map_to_cta(full(s), 0) : full(s);
                    const uint32_t da = ptx::smem_addr(tiles) + (uint32_t)s * stage_bytes, db = da + a_bytes;
                    if (C::kAMn) {
                        ptx::tma_load_2d_cg<CG>(da, &tmA, bar, m0, kb * C::BK);
                        ptx::tma_load_2d_cg<CG>(da + 8192u, &tmA, bar, m0 + 64, kb * C::BK);
                    } else {
                        ptx::tma_load_2d_cg<CG>(da, &tmA, bar, kb * C::BK, m0);
                    }
                    if (C::kBMn) {
#pragma unroll
                        for (int j = 0; j < C::kBRows / 64; ++j)
                            ptx::tma_load_2d_cg<CG>(db + 8192u * j, &tmB, bar, n0 + 64 * j, kb * C::BK);
                    } else {
                        ptx::tma_load_2d_cg<CG>(db, &tmB, bar, kb * C::BK, n0);
                    }
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // no copy may be in flight when the CTA ends (the even CTA's barriers count the pair's)
            if (rank == 0)
                for (int q = 0; q < S; ++q)
                    if (it > (uint32_t)q) {
                        const uint32_t pass = (it - 1u - (uint32_t)q) / (uint32_t)S;
                        ptx::mbar_wait(full(q), pass & 1u, abort_flag, err, kErrTimeout, p.limit_ns, false);
                    }
        } else if (warp == 1 && lane == 0 && rank == 0) {
            // -------------------------------------------------- MMA issuer
            const uint32_t idesc = ptx::idesc_bf16_f32(128 * CG, bn, C::kAMn, C::kBMn);
            constexpr uint32_t a_step = C::kAMn ? 2048u >> 4 : 32u >> 4, b_step = C::kBMn ? 2048u >> 4 : 32u >> 4;
            int s = 0;
            uint32_t ph = 0, tc = 0;
            bool ok = true;
            for (int t = unit; t < num_tiles && ok; t += units) {
                const int ks = t / (p.mt * p.nt);
                const int k0 = (int)((int64_t)p.num_kb * ks / p.splits);
                const int k1 = (int)((int64_t)p.num_kb * (ks + 1) / p.splits);
                if (k0 == k1)
                    continue;
                for (int kb = k0; kb < k1; ++tc) {
                    const uint32_t b = tc & 1u;
                    const int stop = is_stats(MODE) && k1 - kb > p.fold ? kb + p.fold : k1;
                    if (!ptx::mbar_wait<CG == 2>(acc_empty(b), ((tc >> 1) & 1u) ^ 1u, abort_flag, err, kErrTimeout,
                                                 p.limit_ns)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    for (const int start = kb; kb < stop; ++kb) {
                        if (!ptx::mbar_wait<CG == 2>(full(s), ph, abort_flag, err, kErrTimeout, p.limit_ns)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        const uint32_t a = ptx::smem_addr(tiles) + (uint32_t)s * stage_bytes;
                        const uint64_t ad = C::kAMn ? ptx::desc_mnmajor_sw128(a, 8192u) : ptx::desc_kmajor_sw128(a);
                        const uint64_t bd = C::kBMn ? ptx::desc_mnmajor_sw128(a + a_bytes, 8192u)
                                                    : ptx::desc_kmajor_sw128(a + a_bytes);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ptx::mma_bf16<CG>(tmem_base + 256u * b, ad + a_step * k, bd + b_step * k, idesc,
                                              (kb > start || k > 0) ? 1u : 0u);
                        ptx::mma_commit_cg<CG>(empty(s));
                        if (++s == S) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!ok)
                        break;
                    ptx::mma_commit_cg<CG>(acc_full(b));
                }
            }
            ptx::mma_commit_cg<CG>(done);
            ptx::mbar_wait(done, 0u, abort_flag, err, kErrTimeout, p.limit_ns, false);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue: a row and kCols columns a thread
        const int ew = warp - 4, quarter = warp & 3, part = ew >> 2;
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        if constexpr (is_stats(MODE)) {
            uint32_t tc = 0;
            for (int t = unit; t < num_tiles; t += units) {
                int mi, ni, ks;
                head_coords(p, t, mi, ni, ks);
                const int row0 = mi * 128 * CG + (int)rank * 128 + quarter * 32;
                const int64_t row = (int64_t)row0 + lane;
                const int n0 = ni * bn + part * 128;
                int tcol = -1; // the target's column in this thread's 128, or out of range
                uint4 skip = make_uint4(0, 0, 0, 0);
                if (MODE == kStatsSkip) {
                    if (row < p.M)
                        skip = __ldg(p.skip + row * (kParts * p.nt) + kParts * ni + part);
                } else if (row < p.M) {
                    const int64_t tg = __ldg(p.target + row), rel = tg - n0;
                    if (tg >= 0 && tg < p.V && rel >= 0 && rel < min(128, bn - part * 128))
                        tcol = (int)rel;
                }
                auto wait_acc = [&](uint32_t n) {
                    const bool got =
                        ptx::mbar_wait(acc_full(n & 1u), (n >> 1) & 1u, abort_flag, err, kErrTimeout, p.limit_ns);
                    const bool all = __all_sync(0xFFFFFFFFu, got);
                    ptx::tc_fence_after();
                    return all;
                };
                auto acc_addr = [&](uint32_t n) {
                    return tmem_base + 256u * (n & 1u) + lane_addr + (uint32_t)(part * 128);
                };
                auto release = [&](uint32_t n) {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (CG == 2)
                            ptx::mbar_arrive_remote(ptx::map_to_cta(acc_empty(n & 1u), 0));
                        else
                            ptx::mbar_arrive(acc_empty(n & 1u));
                    }
                };
                // The tensor core's FP32 accumulator truncates at each step: over a whole K of 4096 the losses
                // of 4096 tokens are off by 3e-6 (2-norm, against binary64), a single token's by up to 2e-5.
                // So partial tiles of `fold` 64-blocks of K are summed here in round-to-nearest.
                float2 z[64];
#pragma unroll
                for (int j = 0; j < 64; ++j)
                    z[j] = make_float2(0.0f, 0.0f);
                const int folds = (p.num_kb + p.fold - 1) / p.fold;
                bool ok = true;
                for (int f = 0; f < folds && ok; ++f) {
                    const uint32_t n = tc + (uint32_t)f;
                    ok = wait_acc(n);
                    if (!ok)
                        break;
#pragma unroll
                    for (int ch = 0; ch < 2; ++ch) {
                        uint32_t v[64];
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            ptx::tmem_ld_32x32b_x32(acc_addr(n) + 64u * ch + 32u * q,
                                                    *reinterpret_cast<uint32_t(*)[32]>(&v[32 * q]));
                        ptx::tmem_ld_wait_tie(v);
                        if (ch == 1)
                            release(n);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            z[32 * ch + j] = __fadd2_rn(z[32 * ch + j], make_float2(__uint_as_float(v[2 * j]),
                                                                                    __uint_as_float(v[2 * j + 1])));
                    }
                }
                if (!ok)
                    break;
                tc += (uint32_t)folds;
                float v[128];
#pragma unroll
                for (int j = 0; j < 64; ++j) {
                    v[2 * j] = z[j].x;
                    v[2 * j + 1] = z[j].y;
                }
                // this thread's columns inside the tile and the vocabulary
                const int valid = (int)min((int64_t)min(128, bn - part * 128), p.N - n0);
                if (valid < 128) {
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        v[j] = j < valid ? v[j] : -INFINITY;
                }
                float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                for (int j = 4; j < 128; ++j)
                    m4[j & 3] = fmaxf(m4[j & 3], v[j]);
                const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                const float mk = m == -INFINITY ? 0.0f : m * p.k2; // without a number: NaN still reaches the sum
                if constexpr (MODE == kStatsSkip) { // these terms are joined exactly by the last kernel
                    const uint32_t bits[4] = {skip.x, skip.y, skip.z, skip.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (__any_sync(0xFFFFFFFFu, bits[q] != 0u))
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[32 * q + j] = bits[q] >> j & 1u ? -INFINITY : v[32 * q + j];
                } else if (__any_sync(0xFFFFFFFFu, tcol >= 0)) { // the target's term is joined exactly by the last kernel
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        v[j] = j == tcol ? -INFINITY : v[j];
                }
                float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < 128; ++j)
                    s4[j & 3] += ex2(fmaf(v[j], p.k2, -mk));
                if (row < p.M) {
                    // no column, or all of them -inf: an empty sum.  fmaxf passes over NaN, the sum does not: NaN
                    // among numbers or past them (the columns outside are -inf), and where all 128 are NaN
                    const float sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
                    p.part[(int64_t)(kParts * ni + part) * p.M + row] = m == -INFINITY ? make_float2(-INFINITY, sum)
                                                                   : m == m       ? make_float2(mk, sum)
                                                                                  : make_float2(0.0f, m);
                }
            }
        } else {
            const uint32_t stage = ptx::smem_addr(staging) + (uint32_t)ew * 4096u;
            const uint32_t stage_row = stage + (uint32_t)lane * 128u;
            float factor = 1.0f, gmax = 0.0f;
            if (MODE == kGrad)
                gmax = __ldg(p.gmax);
            if (MODE == kGradW16 || MODE == kGradW32)
                factor = __ldg(p.gmax) * p.scale;
            auto tile_row = [&](int mi) { return mi * 128 * CG + (int)rank * 128 + quarter * 32; };
            struct RowIn { // loaded a tile ahead
                int target = -1;
                float lse2 = 0.0f, dloss = 0.0f;
            };
            auto row_in = [&](int t) {
                RowIn r;
                if (MODE == kGrad && t < num_tiles) {
                    int mi, ni, ks;
                    head_coords(p, t, mi, ni, ks);
                    const int64_t row = tile_row(mi) + lane;
                    if (row < p.M) {
                        const int4 q = __ldg(reinterpret_cast<const int4 *>(p.rows + row));
                        r.target = q.x;
                        r.lse2 = __int_as_float(q.y);
                        r.dloss = __int_as_float(q.z);
                    }
                }
                return r;
            };
            auto wait_acc = [&](uint32_t n) {
                const bool got =
                    ptx::mbar_wait(acc_full(n & 1u), (n >> 1) & 1u, abort_flag, err, kErrTimeout, p.limit_ns);
                const bool all = __all_sync(0xFFFFFFFFu, got);
                ptx::tc_fence_after();
                return all;
            };
            auto acc_addr = [&](uint32_t n) {
                return tmem_base + 256u * (n & 1u) + lane_addr + (uint32_t)(part * C::kCols);
            };
            auto release = [&](uint32_t n) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2)
                        ptx::mbar_arrive_remote(ptx::map_to_cta(acc_empty(n & 1u), 0));
                    else
                        ptx::mbar_arrive(acc_empty(n & 1u));
                }
            };
            // writes a box (128 bytes a row, 32 rows) to the staging buffer once its last store has left it
            auto stage_box = [&](const uint32_t *h) {
                if (lane == 0)
                    ptx::bulk_wait_group_read<0>();
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    ptx::st_shared_v4(stage_row + (uint32_t)((j ^ (lane & 7)) << 4), h[4 * j], h[4 * j + 1], h[4 * j + 2],
                                      h[4 * j + 3]);
                ptx::fence_proxy_async_smem();
                __syncwarp();
            };
            uint32_t tc = 0;
            RowIn next = row_in(unit);
            for (int t = unit; t < num_tiles; t += units) {
                int mi, ni, ks;
                head_coords(p, t, mi, ni, ks);
                if (MODE == kGradX &&
                    (int64_t)p.num_kb * ks / p.splits == (int64_t)p.num_kb * (ks + 1) / p.splits)
                    continue;
                const int row0 = tile_row(mi);
                const int64_t row = (int64_t)row0 + lane;
                const int n0 = ni * bn + part * C::kCols;
                const RowIn in = next;
                if constexpr (MODE == kGrad || MODE == kGradW16) { // 64 BF16 columns: one box
                    if (!wait_acc(tc))
                        break;
                    // a row without a loss: logits, lse2 and dloss are zero, and so is d
                    const float lse2 = in.lse2;
                    const float f = MODE == kGradW16 ? factor : (gmax > 0.0f ? __fdiv_rn(in.dloss, gmax) : 0.0f);
                    const int rel = in.target - (int)p.col0 - n0;
                    const int tcol = rel >= 0 && rel < C::kCols ? rel : -1; // the target's column, if here
                    next = row_in(t + units);
                    uint32_t h[32];
#pragma unroll
                    for (int ch = 0; ch < 2; ++ch) {
                        uint32_t v[32];
                        ptx::tmem_ld_32x32b_x32(acc_addr(tc) + 32u * ch, v);
                        ptx::tmem_ld_wait_tie(v);
                        if (ch == 1)
                            release(tc);
                        if constexpr (MODE == kGrad) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = __float_as_uint(ex2(fmaf(__uint_as_float(v[j]), p.k2, -lse2)));
                            if (__any_sync(0xFFFFFFFFu, tcol >> 5 == ch)) {
                                const float dt = tcol >= 0 ? __ldg(&p.rows[row].dt) : 0.0f;
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    v[j] = 32 * ch + j == tcol ? __float_as_uint(dt) : v[j];
                            }
                            if (n0 + 32 * ch + 32 > p.N) { // columns past the piece: zero, part of the dx product's K
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    v[j] = n0 + 32 * ch + j < p.N ? v[j] : 0u;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const __nv_bfloat162 b2 =
                                __floats2bfloat162_rn(__uint_as_float(v[2 * j]) * f, __uint_as_float(v[2 * j + 1]) * f);
                            h[16 * ch + j] = *reinterpret_cast<const uint32_t *>(&b2);
                        }
                    }
                    ++tc;
                    if (row0 >= p.M || (MODE == kGradW16 && n0 >= p.N))
                        continue;
                    stage_box(h);
                    if (lane == 0) {
                        ptx::tma_store_3d(&tmO, stage, n0, row0, 0);
                        ptx::bulk_commit_group();
                    }
                } else {
                    if (!wait_acc(tc))
                        break;
                    const uint32_t acc = acc_addr(tc);
#pragma unroll
                    for (int g = 0; g < 2; ++g) { // 32 FP32 columns a box
                        uint32_t v[32];
                        ptx::tmem_ld_32x32b_x32(acc + 32u * g, v);
                        ptx::tmem_ld_wait_tie(v);
                        if (g == 1)
                            release(tc);
                        const int x0 = n0 + 32 * g;
                        if (x0 >= p.N || row0 >= p.M)
                            continue;
                        if (MODE == kGradW32) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = __float_as_uint(__uint_as_float(v[j]) * factor);
                        }
                        stage_box(v);
                        if (lane == 0) {
                            if (p.add)
                                ptx::tma_add_3d(&tmO, stage, x0, row0, ks);
                            else
                                ptx::tma_store_3d(&tmO, stage, x0, row0, ks);
                            ptx::bulk_commit_group();
                        }
                    }
                    ++tc;
                }
            }
        }
        if (C::kStaging && lane == 0)
            ptx::bulk_wait_group0();
        // the odd CTA's barriers get the even one's commits: the last has arrived before the CTA ends
        if (CG == 2 && rank == 1 && ew == 0 && lane == 0)
            ptx::mbar_wait(done, 0u, abort_flag, err, kErrTimeout, p.limit_ns, false);
        __syncwarp();
    }

    ptx::tc_fence_before();
    if (CG == 2)
        ptx::cluster_sync(); // the peer's MMAs and loads that name this CTA's memory are done
    else
        __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_cg<CG>(tmem_base, 512);
    }
}

// Joins the (maximum, sum) pairs of a row and its target's logit.  blockDim =
// (rows, lanes), powers of two: threadIdx.x walks rows (contiguous in part),
// threadIdx.y parts.  The target's logit is summed here, with compensation: it
// is the largest one of a confident token, whose loss is its distance to the
// others' and whose lse is that logit plus the loss.  With the tensor core's sum
// a single token's loss was off by 2.4e-6 of its value, and lse by 1.4e-5 at 300
// tokens x 2000 x 4096, which the backward pass would meet in exp(z_t - lse) - 1.
__global__ void __launch_bounds__(1024)
    k_ce_join(const float2 *part, const uint16_t *x, int64_t ldx, const uint16_t *w, int64_t ldw, int64_t c,
              const int64_t *target, int64_t n, int64_t v, int parts, float scale, float k2, float *loss, float *lse)
{
    __shared__ float2 red[1024], dots[1024];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t row = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t tg = row < n ? target[row] : -1;
    const bool has = tg >= 0 && tg < v;
    const int at = threadIdx.y * blockDim.x + threadIdx.x;
    float s = 0.0f, comp = 0.0f;
    if (has)
        for (int64_t k = 8 * threadIdx.y; k < c; k += 8 * blockDim.y) // c and the rows are whole vectors
            dot8(s, comp, __ldg(reinterpret_cast<const uint4 *>(x + row * ldx + k)),
                 __ldg(reinterpret_cast<const uint4 *>(w + tg * ldw + k)));
    float2 a = make_float2(-INFINITY, 0.0f);
    if (row < n)
        for (int q = threadIdx.y; q < parts; q += 4 * blockDim.y) { // four loads in flight
            float2 b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[i] = q + i * (int)blockDim.y < parts ? __ldg(part + (int64_t)(q + i * blockDim.y) * n + row)
                                                       : make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                join_pair(a, b[i]);
        }
    red[at] = a;
    dots[at] = make_float2(s, comp);
    for (int o = blockDim.y / 2; o; o >>= 1) {
        __syncthreads();
        if ((int)threadIdx.y < o) {
            join_pair(a, red[at + o * blockDim.x]);
            red[at] = a;
            const float2 d = dots[at + o * blockDim.x];
            two_sum(s, comp, d.x);
            comp += d.y;
            dots[at] = make_float2(s, comp);
        }
    }
    if (threadIdx.y != 0 || row >= n)
        return;
    if (!has) {
        lse[row] = kLn2 * (a.x + log2f(a.y));
        loss[row] = 0.0f;
        return;
    }
    // the target's exponent against the maximum's, rounded once: both products carry errors of lse's size
    const double z = whole_sum(s, comp);
    const float dt = (float)(z * (double)k2 - (double)a.x);
    if (dt >= -1.0f) { // the target leads, or almost
        const float l = log1pf(a.y * exp2f(-dt));
        loss[row] = l;
        lse[row] = (float)(z * (double)scale + (double)l);
    } else {
        const float rest = a.y + exp2f(dt);
        loss[row] = logf(rest) - kLn2 * dt;
        lse[row] = kLn2 * (a.x + log2f(rest));
    }
}

// Rows of x copied to a stride of whole 128-byte lines, a warp a row.  Backward
// (`rows` given): rows without a loss become zero (whatever they hold: the
// products run over every row, and 0 * NaN would reach all of dw), and each
// row's GradRow is written.  A confident token's d at its target is -(1 - p),
// about minus its loss, so the target's logit has to be good to a small part of
// the loss: with the tensor core's truncating sum over K = 4096 a row of dx was
// wrong by half where the loss is 1e-4 to 3e-4 (2000 x 4096 head; 2e-3 now, d's
// rounding).  It is summed here with compensation (BF16 products are exact in
// FP32) and leaves through one rounding of z_t - lse.  The other entries are p
// itself, whose relative error stays that of the exponent, far below d's BF16
// rounding.
// Block 0 has the backward pass's other start: gmax = max |dloss| over the rows
// with a target (1 where that is not finite).
__global__ void __launch_bounds__(256)
    k_ce_start(const uint16_t *x, int64_t n, int64_t c, int64_t ldx, uint16_t *out, int64_t ldo, const uint16_t *w,
               int64_t ldw, const int64_t *target, int64_t v, float scale, const float *lse, const float *dloss,
               GradRow *rows, float *gmax)
{
    __shared__ float red[8];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    if (blockIdx.x > 0) {
        const int lane = threadIdx.x & 31;
        const int64_t step = (int64_t)(gridDim.x - 1) * 8;
        for (int64_t r = (int64_t)(blockIdx.x - 1) * 8 + (threadIdx.x >> 5); r < n; r += step) {
            const int64_t tg = rows ? __ldg(target + r) : 0;
            const bool has = !rows || (tg >= 0 && tg < v);
            float s = 0.0f, comp = 0.0f;
#pragma unroll 4
            for (int64_t k = 8 * lane; k < c; k += 256) { // c and the rows are whole vectors
                uint4 a = make_uint4(0, 0, 0, 0);
                if (has) {
                    a = __ldg(reinterpret_cast<const uint4 *>(x + r * ldx + k));
                    if (rows)
                        dot8(s, comp, a, __ldg(reinterpret_cast<const uint4 *>(w + tg * ldw + k)));
                }
                *reinterpret_cast<uint4 *>(out + r * ldo + k) = a;
            }
            if (!rows)
                continue;
            for (int o = 16; o; o >>= 1) {
                const float s2 = __shfl_xor_sync(0xFFFFFFFFu, s, o), c2 = __shfl_xor_sync(0xFFFFFFFFu, comp, o);
                two_sum(s, comp, s2);
                comp += c2;
            }
            if (lane == 0) {
                GradRow g = {-1, 0.0f, 0.0f, 0.0f};
                if (has) {
                    const double z = whole_sum(s, comp) * (double)scale;
                    g = {(int)tg, lse[r] * kLog2e, dloss[r], expm1f((float)(z - (double)lse[r]))};
                }
                rows[r] = g;
            }
        }
        return;
    }
    if (!gmax)
        return;
    float m = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
        const int64_t tg = target[i];
        if (tg >= 0 && tg < v) {
            const float g = fabsf(dloss[i]);
            m = g < INFINITY ? fmaxf(m, g) : INFINITY; // NaN too: the rows then keep their own values
        }
    }
    for (int o = 16; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i)
            m = fmaxf(m, red[i]);
        *gmax = m < INFINITY ? m : 1.0f;
    }
}

// dx = BF16(scale * gmax * sum of the slabs), four columns a thread.
__global__ void k_ce_dx(const float *slab, int slabs, int64_t n, int64_t c, const float *gmax, float scale,
                        uint16_t *dx, int64_t lddx)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const float f = __ldg(gmax) * scale;
    const int64_t c4 = c / 4, total = n * c4;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const float4 *s = reinterpret_cast<const float4 *>(slab) + i;
        float4 a = *s;
        for (int q = 1; q < slabs; ++q) {
            const float4 b = s[q * total];
            a.x += b.x;
            a.y += b.y;
            a.z += b.z;
            a.w += b.w;
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * f, a.y * f), hi = __floats2bfloat162_rn(a.z * f, a.w * f);
        const int64_t r = i / c4, col = 4 * (i - r * c4);
        *reinterpret_cast<uint2 *>(dx + r * lddx + col) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
}

constexpr int kTileN = 256;

int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

// Tiles in work at a time (1 where no device answers: the size queries run without one).
int units_of(int cg)
{
    const int u = sm_count() / cg;
    return u > 0 ? u : 1;
}

template <int CG, int MODE, bool FEW>
cudaError_t run_tiles(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &o, HeadParams p, cudaStream_t st)
{
    using C = HeadCfg<CG, MODE, FEW>;
    auto kern = k_head_gemm<CG, MODE, FEW>;
    static int configured_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (configured_device != dev) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem)) != cudaSuccess)
            return e;
        if (C::kRegSplit) {
            // setmaxnreg.inc waits until the CTA's registers can serve it: the launch must
            // provide both shares, or the kernel would stall
            cudaFuncAttributes fa;
            if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess)
                return e;
            if (fa.numRegs < C::kRegProducer || fa.numRegs > C::kRegEpilogue ||
                fa.numRegs * C::kThreads < C::kRegProducer * 128 + C::kRegEpilogue * 32 * C::kEpiWarps)
                return cudaErrorInvalidConfiguration;
        }
        configured_device = dev;
    }
    p.limit_ns = kWaitLimitNs;
    if (FEW) {
        // 16 KB stay free: what the MMA reads of the last stage past its box lies inside the allocation
        const int64_t stage = (int64_t)p.box_a * 128 + (C::kBMn ? C::kBBytes : (int64_t)p.bn * 128);
        const int64_t fit = ((int64_t)C::kTileBytes - C::kABytes) / stage;
        p.stages = (int)(fit < C::kStages ? fit : C::kStages);
    }
    const int64_t tiles = (int64_t)p.mt * p.nt * p.splits;
    const int units = (int)(tiles < units_of(CG) ? tiles : units_of(CG));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * CG));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, b, o, p);
}

// cg CTAs a tile; one tile of rows (cg = 1, box_a of them) takes the FEW form.
template <int MODE>
cudaError_t run_head(int cg, const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &o, const HeadParams &p,
                     cudaStream_t st)
{
    if constexpr (!HeadCfg<2, MODE, false>::kAMn) {
        if (cg == 1)
            return p.mt == 1 ? run_tiles<1, MODE, true>(a, b, o, p, st) : run_tiles<1, MODE, false>(a, b, o, p, st);
    }
    return run_tiles<2, MODE, false>(a, b, o, p, st);
}

// Rows of A's box by single CTAs: 128, or one tile's rows.
int box_rows(int64_t n)
{
    return n <= 128 ? (int)(ceil_div(n, 8) * 8) : 128;
}

// CTA pairs (256 x 256 tiles) or single CTAs (128 x 256)?  A 64-block of K is
// 512 tensor cycles for either, but a single CTA loads 48 KB for it, 750 cycles
// at an SM's 64 bytes a cycle from L2, and a CTA of a pair 32 KB: single CTAs
// count 1.2 times as long a tile (back to back at the power cap, where clocks
// fall, d + dx + dw of 4096 tokens x 131072 x 4096 measured 8.72 ms against
// 7.99).  They waste less where the rows do not fill pairs.
int pick_cg(int64_t rows, int64_t tiles_n)
{
    if (rows <= 128)
        return 1;
    const int64_t w1 = ceil_div(ceil_div(rows, 128) * tiles_n, units_of(1));
    const int64_t w2 = ceil_div(ceil_div(rows, 256) * tiles_n, units_of(2));
    return 5 * w2 <= 6 * w1 ? 2 : 1;
}

// CTAs a tile and K splits of the dx product: enough work units to fill the
// machine evenly.  A split costs a slab's traffic, a tile of the whole piece
// about 4.7 ns for every vocabulary row.
void dx_shape(int64_t n, int64_t c, int64_t piece, int &cg, int &splits)
{
    const int64_t most = piece / 64 < 16 ? piece / 64 : 16;
    const double tile_s = 4.7e-9 * (double)piece, slab_s = 0.3 * 8.0 * (double)n * (double)c / 5e12;
    double best = 1e30;
    for (int g = 2; g >= 1; --g) {
        const int64_t tiles = ceil_div(n, 128 * g) * ceil_div(c, kTileN), units = units_of(g);
        for (int64_t s = 1; s <= most; ++s) {
            const double t = (double)ceil_div(tiles * s, units) / (double)s * tile_s * (g == 2 ? 1.0 : 1.2) +
                             (double)s * slab_s;
            if (t < best * 0.999) {
                best = t;
                cg = g;
                splits = (int)s;
            }
        }
    }
}

// Row stride of x's copies: whole 128-byte lines.
int64_t lines_ld(int64_t c)
{
    return ceil_div(c, 64) * 64;
}

size_t lines_bytes(int64_t n, int64_t c)
{
    return ((size_t)n * (size_t)lines_ld(c) * 2 + 1023) / 1024 * 1024;
}

// Forward: a row that does not start on a 128-byte line costs each box row a
// second line.  x is read by every tile of the vocabulary, so for more than one
// tile of rows it is copied first where its width makes rows start off the
// lines (with the copy: 1000 x 50257 x 1032 96 us against 104, 2000 x 50257 x
// 2056 277 against 331; w is read by a few tiles of rows only).
size_t fwd_lines(int64_t n, int64_t c)
{
    return n > 128 && c % 64 != 0 ? lines_bytes(n, c) : 0;
}

// Copies a.x to `at` and makes it the copy; backward: zeroes its rows without a
// loss, and computes their GradRow and gmax.
cudaError_t start(LinearCeArgs &a, void *at, GradRow *rows, float *gmax, cudaStream_t st)
{
    const int64_t blocks = ceil_div(a.n, 8), cap = (int64_t)sm_count() * 8;
    uint16_t *out = static_cast<uint16_t *>(at);
    const cudaError_t e =
        launch_pdl(k_ce_start, dim3((unsigned)(1 + (blocks < cap ? blocks : cap))), dim3(256), 0, st, a.x, a.n, a.c,
                   a.ldx, out, lines_ld(a.c), a.w, a.ldw, a.target, a.v, a.scale, (const float *)a.lse, a.dloss, rows,
                   gmax);
    a.x = out;
    a.ldx = lines_ld(a.c);
    return e;
}

struct BwdPlan {
    int64_t piece; // vocabulary rows a piece (a multiple of 256)
    int dx_cg, splits;
    size_t rows_off, x_off, listed_off, slab_off, d_off, total;
};

// k: listed entries a row (distillation; else 0)
BwdPlan bwd_plan(int64_t n, int64_t v, int64_t c, int64_t k, int64_t piece)
{
    BwdPlan b;
    const int64_t all = ceil_div(v, 256) * 256;
    b.piece = piece < 256 ? 256 : (piece > all ? all : piece / 256 * 256);
    dx_shape(n, c, b.piece, b.dx_cg, b.splits);
    b.rows_off = 1024; // gmax first
    b.x_off = b.rows_off + ((size_t)n * sizeof(GradRow) + 1023) / 1024 * 1024;
    b.listed_off = b.x_off + lines_bytes(n, c);
    b.slab_off = b.listed_off + ((size_t)n * (size_t)k * sizeof(Listed) + 1023) / 1024 * 1024;
    const size_t slabs = (size_t)b.splits * (size_t)n * (size_t)c * 4;
    b.d_off = (b.slab_off + slabs + 1023) / 1024 * 1024;
    b.total = b.d_off + (size_t)n * (size_t)b.piece * 2;
    return b;
}

// A piece's d is about 256 MB: few pieces (each adds to dx once), little memory.
int64_t preferred_piece(int64_t n)
{
    return ((int64_t)1 << 27) / (n > 0 ? n : 1);
}

} // namespace

// Tiles of the forward product's vocabulary axis: 256 columns each, or, for one
// row tile, evenly over the SMs; and a float a row, which the formula has had
// from the start (buffers planned by it stay large enough) and no kernel uses.
size_t linear_ce_fwd_workspace(int64_t n, int64_t v, int64_t c)
{
    int64_t nt = ceil_div(v, kTileN);
    if (n <= 128) // never more than the waves' whole tiles
        nt = ceil_div(nt, units_of(1)) * units_of(1);
    return fwd_lines(n, c) + (size_t)(kParts * nt) * (size_t)n * 8 + (size_t)n * 4;
}

size_t linear_ce_bwd_workspace(int64_t n, int64_t v, int64_t c)
{
    return linear_distill_bwd_workspace(n, v, c, 0);
}

size_t linear_ce_bwd_workspace_min(int64_t n, int64_t v, int64_t c)
{
    return linear_distill_bwd_workspace_min(n, v, c, 0);
}

size_t linear_distill_bwd_workspace(int64_t n, int64_t v, int64_t c, int64_t k)
{
    return bwd_plan(n, v, c, k, preferred_piece(n)).total;
}

size_t linear_distill_bwd_workspace_min(int64_t n, int64_t v, int64_t c, int64_t k)
{
    return bwd_plan(n, v, c, k, 256).total;
}

namespace {

// The forward product's geometry: CTAs a tile, its columns and their number.
struct StatsShape {
    int cg, bn, nt;
};

StatsShape stats_shape(int64_t n, int64_t v)
{
    StatsShape s;
    s.nt = (int)ceil_div(v, kTileN);
    s.cg = pick_cg(n, s.nt);
    s.bn = kTileN;
    if (s.cg == 1 && n <= 128) {
        // One row tile: the weight's stream is what takes time, so its rows are
        // spread evenly over the SMs (a multiple of 16 a tile).
        const int64_t waves = ceil_div(s.nt, units_of(1));
        s.bn = (int)(ceil_div(ceil_div(v, waves * units_of(1)), 16) * 16);
        s.nt = (int)ceil_div(v, s.bn);
    }
    return s;
}

// The statistics of the logits, a.x in the rows that the product reads.
template <int MODE>
cudaError_t run_stats(const LinearCeArgs &a, const StatsShape &shape, float2 *part, const uint4 *skip, bool wait_x,
                      cudaStream_t st)
{
    HeadParams p = {};
    const int cg = shape.cg;
    p.nt = shape.nt;
    p.bn = shape.bn;
    p.box_a = box_rows(a.n);
    cudaError_t e;
    CUtensorMap ta, tb;
    if ((e = make_sw128_map(&ta, a.x, false, a.c, a.n, a.ldx, p.box_a)) != cudaSuccess ||
        (e = make_sw128_map(&tb, a.w, false, a.c, a.v, a.ldw, p.bn / cg)) != cudaSuccess)
        return e;
    p.mt = (int)ceil_div(a.n, 128 * cg);
    p.splits = 1;
    p.num_kb = (int)ceil_div(a.c, 64);
    p.group = p.mt < 64 / cg ? p.mt : 64 / cg; // the group's x stays in L2 while w streams through once
    p.M = a.n;
    p.N = a.v;
    p.k2 = a.scale * kLog2e;
    p.target = a.target;
    p.skip = skip;
    p.wait_x = wait_x;
    // The error of a loss grows with the steps of a partial tile.  Pairs: 8 blocks (1.2e-7 in the 2-norm over
    // 4096 tokens, an FP32 matrix product has 6.7e-7; 4096 x 131072 x 4096 took 2.65 ms with 8, 2.97 with 4 and
    // 4.03 with 2, whose hand-overs between the CTAs stall the tensor core).  Single CTAs: 4 (1e-7; 2 us less than
    // with 2 at 333 tokens x 50257 x 2048, 66 in all, and 3 us less at one token x 1000 x 4096).
    p.fold = cg == 2 ? 8 : 4;
    p.V = a.v;
    p.part = part;
    return run_head<MODE>(cg, ta, tb, ta, p, st);
}

// Whether the forward product reads a copy of x.
bool copies_x(const LinearCeArgs &a)
{
    return fwd_lines(a.n, a.c) > 0 && (a.ldx % 64 != 0 || (reinterpret_cast<uintptr_t>(a.x) & 127u) != 0);
}

} // namespace

cudaError_t launch_linear_ce_fwd(LinearCeArgs a, cudaStream_t st)
{
    cudaError_t e;
    if (copies_x(a) && (e = start(a, a.ws, nullptr, nullptr, st)) != cudaSuccess)
        return e;
    const StatsShape shape = stats_shape(a.n, a.v);
    float2 *part = reinterpret_cast<float2 *>(static_cast<uint8_t *>(a.ws) + fwd_lines(a.n, a.c));
    if ((e = run_stats<kStats>(a, shape, part, nullptr, true, st)) != cudaSuccess)
        return e;
    const int parts = kParts * shape.nt;
    int rx = 1, ry = 1;
    while (rx < 8 && rx < a.n)
        rx *= 2;
    while (rx * ry < 1024 && ry < parts)
        ry *= 2;
    const dim3 grid((unsigned)ceil_div(a.n, rx)), block(rx, ry);
    return launch_pdl(k_ce_join, grid, block, 0, st, (const float2 *)part, a.x, a.ldx, a.w, a.ldw, a.c, a.target, a.n,
                      a.v, parts, a.scale, a.scale * kLog2e, a.loss, a.lse);
}

size_t linear_distill_fwd_workspace(int64_t n, int64_t v, int64_t c, int64_t k)
{
    const size_t parts = linear_ce_fwd_workspace(n, v, c) - fwd_lines(n, c); // the pairs, and 4 bytes a row
    return fwd_lines(n, c) + (parts + 15) / 16 * 16 + 2 * parts + (size_t)n * (size_t)k * sizeof(float2);
}

// Marks and logits of the listed columns, the statistics of all others, and their join.
cudaError_t launch_linear_distill_fwd(LinearCeArgs a, const DistillArgs &t, cudaStream_t st)
{
    const StatsShape shape = stats_shape(a.n, a.v);
    const int parts = kParts * shape.nt;
    uint8_t *ws = static_cast<uint8_t *>(a.ws) + fwd_lines(a.n, a.c);
    float2 *part = reinterpret_cast<float2 *>(ws);
    const size_t pairs = (size_t)parts * (size_t)a.n * sizeof(float2);
    uint4 *skip = reinterpret_cast<uint4 *>(ws + (pairs + 15) / 16 * 16);
    float2 *dots = reinterpret_cast<float2 *>(reinterpret_cast<uint8_t *>(skip) + 2 * pairs);
    uint16_t *copy = copies_x(a) ? static_cast<uint16_t *>(a.ws) : nullptr;
    cudaError_t e = launch_distill_rows(a, t, copy, lines_ld(a.c), shape.bn, parts, skip, dots, st);
    if (e != cudaSuccess)
        return e;
    if (copy) {
        a.x = copy;
        a.ldx = lines_ld(a.c);
    }
    if ((e = run_stats<kStatsSkip>(a, shape, part, skip, copy != nullptr, st)) != cudaSuccess)
        return e;
    return launch_distill_join(a, t, part, parts, dots, st);
}

cudaError_t launch_linear_ce_bwd(LinearCeArgs a, const DistillArgs *t, cudaStream_t st)
{
    // the largest piece that the workspace holds, up to the preferred one
    const int64_t k = t ? t->k : 0;
    BwdPlan plan = bwd_plan(a.n, a.v, a.c, k, preferred_piece(a.n));
    while (plan.total > a.ws_bytes && plan.piece > 256)
        plan = bwd_plan(a.n, a.v, a.c, k, plan.piece / 2);
    if (plan.total > a.ws_bytes)
        return cudaErrorInvalidValue;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    float *gmax = reinterpret_cast<float *>(ws), *slab = reinterpret_cast<float *>(ws + plan.slab_off);
    uint16_t *d = reinterpret_cast<uint16_t *>(ws + plan.d_off);
    GradRow *grad_rows = reinterpret_cast<GradRow *>(ws + plan.rows_off);
    Listed *listed = reinterpret_cast<Listed *>(ws + plan.listed_off);
    cudaError_t e;
    if (t) {
        uint16_t *copy = reinterpret_cast<uint16_t *>(ws + plan.x_off);
        e = launch_distill_start(a, *t, copy, lines_ld(a.c), grad_rows, listed, gmax, st);
        a.x = copy;
        a.ldx = lines_ld(a.c);
    } else {
        e = start(a, ws + plan.x_off, grad_rows, gmax, st);
    }
    if (e != cudaSuccess)
        return e;
    const bool dw16 = a.dw_dtype == JETQ_OUT_BF16;
    for (int64_t v0 = 0; v0 < a.v; v0 += plan.piece) {
        const int64_t rows = a.v - v0 < plan.piece ? a.v - v0 : plan.piece; // vocabulary rows of this piece
        const int64_t cols = ceil_div(rows, 256) * 256;                     // columns of d, zero past rows
        const int cg = pick_cg(a.n, ceil_div(rows, kTileN));
        const uint16_t *w = a.w + v0 * a.ldw;
        void *dwp = static_cast<uint8_t *>(a.dw) + v0 * a.lddw * (dw16 ? 2 : 4);
        const int box = box_rows(a.n);
        CUtensorMap xk, wk, dst, dk, wn, slabs, dm, xn, dw;
        if ((e = make_sw128_map(&xk, a.x, false, a.c, a.n, a.ldx, cg == 1 ? box : 128)) != cudaSuccess ||
            (e = make_sw128_map(&wk, w, false, a.c, rows, a.ldw, kTileN / cg)) != cudaSuccess ||
            (e = make_sw128_map(&dst, d, false, cols, a.n, plan.piece, 32, 1, plan.piece * a.n)) != cudaSuccess ||
            (e = make_sw128_map(&dk, d, false, cols, a.n, plan.piece, plan.dx_cg == 1 ? box : 128)) != cudaSuccess ||
            (e = make_sw128_map(&wn, w, false, a.c, rows, a.ldw, 64)) != cudaSuccess ||
            (e = make_sw128_map(&slabs, slab, true, a.c, a.n, a.c, 32, plan.splits, a.n * a.c)) != cudaSuccess ||
            (e = make_sw128_map(&dm, d, false, cols, a.n, plan.piece, 64)) != cudaSuccess ||
            (e = make_sw128_map(&xn, a.x, false, a.c, a.n, a.ldx, 64)) != cudaSuccess ||
            (e = make_sw128_map(&dw, dwp, !dw16, a.c, rows, a.lddw, 32, 1, rows * a.lddw)) != cudaSuccess)
            return e;
        HeadParams p = {};
        p.bn = kTileN;
        p.box_a = box;
        p.gmax = gmax;
        p.scale = a.scale;
        // d of the piece
        p.mt = (int)ceil_div(a.n, 128 * cg);
        p.nt = (int)ceil_div(rows, kTileN);
        p.splits = 1;
        p.num_kb = (int)ceil_div(a.c, 64);
        p.group = p.mt < 64 / cg ? p.mt : 64 / cg;
        p.M = a.n;
        p.N = rows;
        p.k2 = a.scale * kLog2e;
        p.col0 = v0;
        p.rows = grad_rows;
        if ((e = run_head<kGrad>(cg, xk, wk, dst, p, st)) != cudaSuccess)
            return e;
        // the listed columns' entries, where both of d's terms meet
        if (t && (e = launch_distill_patch(a, *t, listed, gmax, d, plan.piece, v0, rows, st)) != cudaSuccess)
            return e;
        // dx += d w
        p.mt = (int)ceil_div(a.n, 128 * plan.dx_cg);
        p.nt = (int)ceil_div(a.c, kTileN);
        p.splits = plan.splits;
        p.num_kb = (int)(cols / 64);
        p.group = p.mt < 64 / plan.dx_cg ? p.mt : 64 / plan.dx_cg;
        p.N = a.c;
        p.add = v0 > 0;
        if ((e = run_head<kGradX>(plan.dx_cg, dk, wn, slabs, p, st)) != cudaSuccess)
            return e;
        // dw = d^T x: few vocabulary tiles at a time against all of x
        p.mt = (int)ceil_div(rows, 256);
        p.group = p.mt < 4 ? p.mt : 4;
        p.splits = 1;
        p.num_kb = (int)ceil_div(a.n, 64);
        p.M = rows;
        p.add = a.accumulate;
        e = dw16 ? run_head<kGradW16>(2, dm, xn, dw, p, st) : run_head<kGradW32>(2, dm, xn, dw, p, st);
        if (e != cudaSuccess)
            return e;
    }
    if (t)
        return launch_distill_dx(a, *t, listed, slab, plan.splits, gmax, st);
    const int64_t blocks = ceil_div(a.n * (a.c / 4), 256), cap = (int64_t)sm_count() * 8;
    return launch_pdl(k_ce_dx, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, st, (const float *)slab,
                      plan.splits, a.n, a.c, (const float *)gmax, a.scale, a.dx, a.lddx);
}

cudaError_t linear_ce_read_and_clear_error(cudaStream_t st, unsigned *out)
{
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_linear_ce_error, sizeof v, 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(st);
    if (e != cudaSuccess)
        return e;
    *out |= v;
    if (v) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbolAsync(g_linear_ce_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, st);
        if (e == cudaSuccess)
            e = cudaStreamSynchronize(st);
    }
    return e;
}

} // namespace jetq
