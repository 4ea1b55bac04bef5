// Few-token product with NVFP4 weights and BF16 activations (1 to 16 tokens),
// the serving form of the NVFP4 recipe: weights stay in 4 bits, activations
// are not quantized.
//
//   y[i, r] = sg * sum_k e2m1(q[r, k]) * e4m3(sb[r, k / 16]) * x[i, k]
//
// Floor: HBM (9/16 byte a weight).  It runs at three times that, with no pipe
// full at one token: while an SM is active the ALU pipe (masks of the decode,
// permutes of x) is 58% busy and the L1 58%, warps wait for loads most, and a
// third of the time goes at the kernel's two ends.  x is read where it is used,
// again for every 16 rows of the weight: with 8 tokens the L1 is 74% busy, with
// 16 it is 86% and the bound.  A CTA owns 16 rows of the weight, its warps a
// contiguous share of K each, the next batch of the weight's loads in flight
// under a batch's arithmetic.
// The product runs on the tensor cores (mma.m16n8k16, weight rows as M, tokens as
// N): one warp step covers 16 rows x 128 columns, a lane holding 32 consecutive
// values (16 bytes, two scale blocks) of two rows; since both operands permute K
// alike, every lane feeds its own values to the MMA and no data moves between
// lanes.  This is a legacy MMA on purpose: tcgen05 would need the decoded weights
// in shared memory and 128 rows a tile, and the tensor pipe is 13% busy here.
// 12288 x 4096 in a graph (4.2 us of HBM time): 12.1 us for one token, 13.1 for
// eight, 20.7 for nine and 24.6 for sixteen; 4096 x 12288: 11.7, 12.8, 17.4, 20.3.
//
// Decoding is exact (nvfp4_mma.cuh).  FP32 sums, one rounding of the result.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "jetq_internal.h"
#include "nvfp4_mma.cuh"
#include "ptx.cuh"

namespace jetq {

namespace {

constexpr int kRows = 16, kStep = 128; // rows a CTA, columns a warp step
constexpr int kUnroll = 2;             // steps a batch; the next batch's loads are in flight under a batch's arithmetic

struct GemvParams {
    const uint8_t *q, *sb;
    const float *sg;
    const uint16_t *x;
    int64_t n, k, ldx, ldy;
    int m;
    void *y;
    int out_bf16;
};

// MT: tokens in eights; kWarps: shares of K a CTA
template <int MT, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps == 16 ? 1 : (MT == 1 ? 24 : 16) / kWarps)
    k_gemv_nvfp4(const GemvParams p)
{
    __shared__ float red[kWarps][kRows][8 * MT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t row0 = (int64_t)blockIdx.x * kRows;
    const int steps = (int)((p.k + kStep - 1) / kStep);
    const int s0 = steps * warp / kWarps, s1 = steps * (warp + 1) / kWarps;
    const int64_t ra = min(row0 + g, p.n - 1), rb = min(row0 + g + 8, p.n - 1); // rows past n: read, not stored
    // this lane's 32 columns of step 0; a step is 64 bytes of codes, 8 of scales, 256 of x
    const uint8_t *qa = p.q + ra * (p.k / 2) + 16 * t, *qb = p.q + rb * (p.k / 2) + 16 * t;
    const uint8_t *sa = p.sb + ra * (p.k / 16) + 2 * t, *sbb = p.sb + rb * (p.k / 16) + 2 * t;
    const uint16_t *xr[MT]; // lanes past the last token read it too: their sums are not stored
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xr[i] = p.x + min(8 * i + g, p.m - 1) * p.ldx + 32 * t;
    const int left = (int)p.k - 32 * t; // columns from this lane's first one on
    float acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = 0.0f;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();

    struct Batch {
        uint4 ca[kUnroll], cb[kUnroll]; // codes of rows g and g + 8
        uint32_t fa[kUnroll], fb[kUnroll];
    };
    auto load = [&](int s, Batch &b) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            b.ca[u] = b.cb[u] = make_uint4(0, 0, 0, 0);
            b.fa[u] = b.fb[u] = 0;
            if (s + u < s1 && (s + u) * kStep < left) {
                b.ca[u] = __ldcs(reinterpret_cast<const uint4 *>(qa + (s + u) * 64)); // each weight is read once
                b.cb[u] = __ldcs(reinterpret_cast<const uint4 *>(qb + (s + u) * 64));
                b.fa[u] = __ldg(reinterpret_cast<const uint16_t *>(sa + (s + u) * 8));
                b.fb[u] = __ldg(reinterpret_cast<const uint16_t *>(sbb + (s + u) * 8));
            }
        }
    };
    auto multiply = [&](int s, const Batch &b) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (s + u >= s1)
                break;
            uint4 x[MT][4];
            const bool in = (s + u) * kStep < left; // false only in the last, partial step
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[i][j] = in ? __ldg(reinterpret_cast<const uint4 *>(xr[i] + (s + u) * kStep + 8 * j))
                                 : make_uint4(0, 0, 0, 0);
            uint32_t sca[2], scb[2];
            decode_scales(b.fa[u], sca);
            decode_scales(b.fb[u], scb);
            const uint32_t wa[4] = {b.ca[u].x, b.ca[u].y, b.ca[u].z, b.ca[u].w};
            const uint32_t wb[4] = {b.cb[u].x, b.cb[u].y, b.cb[u].z, b.cb[u].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) { // eight values of each row
                uint32_t pa[4], pb[4];
                decode8(wa[j], sca[j >> 1], pa);
                decode8(wb[j], scb[j >> 1], pb);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    // pairs (0, 4), (1, 5), (2, 6), (3, 7), as the weights come
                    const uint4 v = x[i][j];
                    mma_16816(acc[i], pa[0], pb[0], pa[1], pb[1], __byte_perm(v.x, v.z, 0x5410),
                              __byte_perm(v.x, v.z, 0x7632));
                    mma_16816(acc[i], pa[2], pb[2], pa[3], pb[3], __byte_perm(v.y, v.w, 0x5410),
                              __byte_perm(v.y, v.w, 0x7632));
                }
            }
        }
    };
    Batch now, next;
    load(s0, now);
    for (int s = s0; s < s1; s += kUnroll) {
        load(s + kUnroll, next); // past s1: zeros, no load
        multiply(s, now);
        now = next;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        red[warp][g][8 * i + 2 * t] = acc[i][0];
        red[warp][g][8 * i + 2 * t + 1] = acc[i][1];
        red[warp][g + 8][8 * i + 2 * t] = acc[i][2];
        red[warp][g + 8][8 * i + 2 * t + 1] = acc[i][3];
    }
    __syncthreads();
    const float scale = __ldg(p.sg) * 65536.0f;
    for (int i = threadIdx.x; i < kRows * p.m; i += 32 * kWarps) {
        const int r = i % kRows, tok = i / kRows;
        float a = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            a += red[w][r][tok];
        if (row0 + r < p.n) {
            const int64_t at = tok * p.ldy + row0 + r;
            if (p.out_bf16)
                static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(a * scale);
            else
                static_cast<float *>(p.y)[at] = a * scale;
        }
    }
}

} // namespace

cudaError_t launch_gemv_nvfp4(const GemvNvfp4Args &a, cudaStream_t st)
{
    GemvParams p;
    p.q = a.q;
    p.sb = a.sb;
    p.sg = a.sg;
    p.x = a.x;
    p.n = a.n;
    p.k = a.k;
    p.ldx = a.ldx;
    p.ldy = a.ldy;
    p.m = (int)a.m;
    p.y = a.y;
    p.out_bf16 = a.out_dtype == JETQ_OUT_BF16;
    // Shares of K: four warps a CTA where there are CTAs enough for several an
    // SM, twelve (two CTAs an SM) below that (4096 x 12288, eight tokens: 12.7 us
    // against 18.4 with eight), sixteen where there is one CTA an SM at most.
    const int64_t blocks = (a.n + kRows - 1) / kRows;
    const dim3 grid((unsigned)blocks);
    if (blocks >= 3 * (int64_t)sm_count())
        return a.m <= 8 ? launch_pdl(k_gemv_nvfp4<1, 4>, grid, dim3(128), 0, st, p)
                        : launch_pdl(k_gemv_nvfp4<2, 4>, grid, dim3(128), 0, st, p);
    if (blocks > sm_count())
        return a.m <= 8 ? launch_pdl(k_gemv_nvfp4<1, 12>, grid, dim3(384), 0, st, p)
                        : launch_pdl(k_gemv_nvfp4<2, 12>, grid, dim3(384), 0, st, p);
    return a.m <= 8 ? launch_pdl(k_gemv_nvfp4<1, 16>, grid, dim3(512), 0, st, p)
                    : launch_pdl(k_gemv_nvfp4<2, 16>, grid, dim3(512), 0, st, p);
}

} // namespace jetq
