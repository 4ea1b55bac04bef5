// A whole mixture-of-experts layer for 1 to 16 tokens: BF16 router, NVFP4
// expert weights, BF16 activations that are not quantized.
//
//   l[i, e] = sum_k x[i, k] * router[e, k];   the topk largest (the lower index first among equals)
//   p       = exp(l) over their sum (renorm) or over the sum of all experts
//   a       = silu(gate x) * (up x),   y[i] = sum over the chosen of p * down a
//
// Floor: the chosen experts' weights from HBM (9/16 byte each).  Three kernels:
//   1. router logits, a CTA an expert;
//   2. gate and up: a unit is 16 rows of gate and the same 16 of up of one
//      chosen expert, for all tokens that chose it; eight warps share K, the
//      next unit's weights are in flight while one is reduced;
//   3. down: a CTA owns 16 rows of y and runs through all chosen experts, its
//      warps sharing (expert, K) steps, so that y is summed in the CTA's
//      registers and written once, without atomics.
// Kernels 2 and 3 each choose the experts from the logits themselves: it takes
// a warp half a microsecond a token, less than one more kernel, and kernel 3
// does it, and loads its first weights, while kernel 2 is still running
// (kernel 2 lets it start once the logits are there).
//
// Both products run on mma.m16n8k16 (weight rows as M, tokens as N), decoded
// in registers as in the few-token product.  In the down product the
// activations are FP32 values p * sg * a: each goes in as two BF16 numbers (16
// bits; a BF16 y rounds to 8) or, for an FP32 y, three (24 bits), in columns of
// their own that are added at the end, so nothing is rounded between the two
// products beyond that.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "jetq_internal.h"
#include "nvfp4_mma.cuh"
#include "ptx.cuh"

namespace jetq {

namespace {

constexpr int kMaxTokens = 16, kMaxExperts = 256, kMaxTop = 16;
constexpr int kRows = 16, kStep = 128; // rows a unit, columns a warp step

struct MoeParams {
    const uint16_t *x, *router;
    int64_t ldx, ldr;
    int m, h, inter, experts, topk;
    bool renorm;
    const uint8_t *q13, *sb13, *q2, *sb2;
    const float *sg13, *sg2;
    float *logits;        // [m][experts]
    __nv_bfloat16 *act;   // [m * topk][parts][inter]
    int64_t *ids;
    float *weights;
    void *y;
    int64_t ldy;
    int out_bf16;
};

constexpr int kRouterThreads = 128;

// Logits of one expert, eight tokens at a time; the CTA's threads share K.
__global__ void __launch_bounds__(kRouterThreads) k_moe_router(const MoeParams p)
{
    __shared__ float red[kRouterThreads / 32][8];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t *w = p.router + (int64_t)blockIdx.x * p.ldr;
    for (int t0 = 0; t0 < p.m; t0 += 8) {
        float2 acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[i] = make_float2(0.0f, 0.0f);
        for (int k = 8 * threadIdx.x; k < p.h; k += 8 * kRouterThreads) { // h and the rows are whole vectors
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(w + k));
            const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (t0 + i < p.m) {
                    const uint4 b = __ldg(reinterpret_cast<const uint4 *>(p.x + (t0 + i) * p.ldx + k));
                    const uint32_t v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i] = __ffma2_rn(
                            make_float2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u)),
                            make_float2(__uint_as_float(v[e] << 16), __uint_as_float(v[e] & 0xffff0000u)), acc[i]);
                }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t0 + i < p.m) {
                float s = acc[i].x + acc[i].y;
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
                if (lane == 0)
                    red[warp][i] = s;
            }
        __syncthreads();
        if (threadIdx.x < 8 && t0 + threadIdx.x < p.m) {
            float s = 0.0f;
#pragma unroll
            for (int g = 0; g < kRouterThreads / 32; ++g)
                s += red[g][threadIdx.x];
            p.logits[(int64_t)(t0 + threadIdx.x) * p.experts + blockIdx.x] = s;
        }
        __syncthreads();
    }
}

// Which experts the tokens take.  Slots number the experts that some token
// takes, in rising order.
struct Routes {
    int id[kMaxTokens][kMaxTop];
    float p[kMaxTokens][kMaxTop];
    unsigned tokens[kMaxExperts];           // bit i: token i takes the expert
    uint8_t choice[kMaxExperts][kMaxTokens]; // which of the token's choices the expert is
    short expert[kMaxExperts];              // of a slot
    int slots;
};

// An order of all floats as unsigned numbers above 0: NaN largest, -0 as 0.
__device__ __forceinline__ unsigned order_key(float v)
{
    if (isnan(v))
        return 0xFFFFFFFFu;
    const unsigned u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float from_key(unsigned k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// All threads of the CTA; a warp a token.
__device__ __forceinline__ void choose(const MoeParams &p, Routes &r)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x)
        r.tokens[e] = 0;
    __syncthreads();
    for (int t = warp; t < p.m; t += warps) {
        unsigned key[kMaxExperts / 32];
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i) {
            const int e = 32 * i + lane;
            key[i] = e < p.experts ? order_key(__ldcg(p.logits + (int64_t)t * p.experts + e)) : 0u;
        }
        unsigned mine = 0, top = 0;
        int id = 0;
        for (int j = 0; j < p.topk; ++j) {
            unsigned best = 0;
            int at = 0;
#pragma unroll
            for (int i = 0; i < kMaxExperts / 32; ++i)
                if (key[i] > best) { // the first of equals
                    best = key[i];
                    at = 32 * i + lane;
                }
            const unsigned m = __reduce_max_sync(0xFFFFFFFFu, best);
            const int w = (int)__reduce_min_sync(0xFFFFFFFFu, best == m ? (unsigned)at : 0xFFFFu);
            if (j == 0) {
                top = m;
                if (!p.renorm) { // the softmax's sum over all experts
#pragma unroll
                    for (int i = 0; i < kMaxExperts / 32; ++i)
                        all += key[i] ? expf(from_key(key[i]) - from_key(top)) : 0.0f;
#pragma unroll
                    for (int o = 16; o; o >>= 1)
                        all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
                }
            }
#pragma unroll
            for (int i = 0; i < kMaxExperts / 32; ++i)
                if (32 * i + lane == w)
                    key[i] = 0;
            if (lane == j) {
                mine = m;
                id = w;
            }
        }
        const float e = lane < p.topk ? expf(from_key(mine) - from_key(top)) : 0.0f;
        if (p.renorm) {
            all = e;
#pragma unroll
            for (int o = 16; o; o >>= 1)
                all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
        }
        if (lane < p.topk) {
            r.id[t][lane] = id;
            r.p[t][lane] = __fdiv_rn(e, all);
            r.choice[id][t] = (uint8_t)lane;
            atomicOr(&r.tokens[id], 1u << t);
        }
    }
    __syncthreads();
    if (warp == 0) {
        int n = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const bool on = e0 + lane < p.experts && r.tokens[e0 + lane] != 0;
            const unsigned b = __ballot_sync(0xFFFFFFFFu, on);
            if (on)
                r.expert[n + __popc(b & ((1u << lane) - 1u))] = (short)(e0 + lane);
            n += __popc(b);
        }
        if (lane == 0)
            r.slots = n;
    }
    __syncthreads();
}

// The n-th set bit of a mask that has it.
__device__ __forceinline__ int nth_bit(unsigned mask, int n)
{
    while (n-- > 0)
        mask &= mask - 1u;
    return __ffs(mask) - 1;
}

// Codes and scales of two rows (g and g + 8 of 16) of a warp step.
struct Codes {
    uint4 a, b;
    uint32_t fa, fb;
    __device__ __forceinline__ void clear()
    {
        a = b = make_uint4(0, 0, 0, 0);
        fa = fb = 0;
    }
    // q, sb: row g's; K columns a row; the rows are 8 apart
    __device__ __forceinline__ void load(const uint8_t *q, const uint8_t *sb, int K, int step)
    {
        a = __ldcs(reinterpret_cast<const uint4 *>(q + step * 64)); // each weight is read once
        b = __ldcs(reinterpret_cast<const uint4 *>(q + (int64_t)4 * K + step * 64));
        fa = __ldg(reinterpret_cast<const uint16_t *>(sb + step * 8));
        fb = __ldg(reinterpret_cast<const uint16_t *>(sb + K / 2 + step * 8));
    }
    // the pairs that the MMA takes of eight values j of each row
    __device__ __forceinline__ void decode(int j, const uint32_t (&sa)[2], const uint32_t (&sb)[2], uint32_t (&pa)[4],
                                           uint32_t (&pb)[4]) const
    {
        decode8(j == 0 ? a.x : j == 1 ? a.y : j == 2 ? a.z : a.w, sa[j >> 1], pa);
        decode8(j == 0 ? b.x : j == 1 ? b.y : j == 2 ? b.z : b.w, sb[j >> 1], pb);
    }
};

// acc += rows x a column (a lane's eight values x): pairs (0, 4), (1, 5), (2, 6), (3, 7), as the weights come
__device__ __forceinline__ void multiply(float (&acc)[4], const uint32_t (&pa)[4], const uint32_t (&pb)[4],
                                         const uint4 &x)
{
    mma_16816(acc, pa[0], pb[0], pa[1], pb[1], __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632));
    mma_16816(acc, pa[2], pb[2], pa[3], pb[3], __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
}

// a as the sum of BF16 numbers, rounded to nearest each.
template <int PARTS>
__device__ __forceinline__ void split(float a, __nv_bfloat16 (&out)[PARTS])
{
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        out[i] = __float2bfloat16_rn(a);
        const float back = __bfloat162float(out[i]);
        a = fabsf(back) < INFINITY ? a - back : 0.0f; // infinite or no number: in the first part only
    }
}

constexpr int kGateWarps = 8, kGateUnroll = 2;

// MT: tokens of an expert in eights; PARTS: BF16 numbers an activation is stored as
template <int MT, int PARTS>
__global__ void __launch_bounds__(32 * kGateWarps, 2) k_moe_gate_up(const MoeParams p)
{
    __shared__ Routes r;
    __shared__ float red[kGateWarps][2 * kRows][8 * MT + 1];
    __shared__ int list[kMaxTokens]; // the unit's tokens
    ptx::grid_dep_wait();
    ptx::grid_dep_launch(); // after the wait: the next kernel may read the logits at once
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    choose(p, r);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < p.m * p.topk; i += blockDim.x) {
            if (p.ids)
                p.ids[i] = r.id[i / p.topk][i % p.topk];
            if (p.weights)
                p.weights[i] = r.p[i / p.topk][i % p.topk];
        }
    const int blocks = p.inter / kRows, units = r.slots * blocks;
    const int steps = (p.h + kStep - 1) / kStep;
    const int s0 = steps * warp / kGateWarps, s1 = steps * (warp + 1) / kGateWarps;
    const int left = p.h - 32 * t; // columns from this lane's first one on

    struct Batch {
        Codes gate[kGateUnroll], up[kGateUnroll];
    };
    auto load = [&](int unit, int s, Batch &b) {
#pragma unroll
        for (int u = 0; u < kGateUnroll; ++u) {
            b.gate[u].clear();
            b.up[u].clear();
        }
        if (unit >= units)
            return;
        const int64_t row = (int64_t)r.expert[unit / blocks] * 2 * p.inter + unit % blocks * kRows + g;
        const uint8_t *q = p.q13 + row * (p.h / 2) + 16 * t, *sb = p.sb13 + row * (p.h / 16) + 2 * t;
        const int64_t up_q = (int64_t)p.inter * (p.h / 2), up_sb = (int64_t)p.inter * (p.h / 16);
#pragma unroll
        for (int u = 0; u < kGateUnroll; ++u)
            if (s + u < s1 && (s + u) * kStep < left) {
                b.gate[u].load(q, sb, p.h, s + u);
                b.up[u].load(q + up_q, sb + up_sb, p.h, s + u);
            }
    };
    Batch now, next;
    load(blockIdx.x, s0, now);
    for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int e = r.expert[unit / blocks];
        const unsigned tokens = r.tokens[e];
        const int many = __popc(tokens);
        const uint16_t *xr[MT]; // this lane's columns' rows of x
        bool have[MT], on[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            on[i] = 8 * i < many;
            have[i] = 8 * i + g < many;
            const int tok = have[i] ? nth_bit(tokens, 8 * i + g) : 0;
            xr[i] = p.x + tok * p.ldx + 32 * t;
            if (warp == 0 && t == 0 && have[i])
                list[8 * i + g] = tok;
        }
        float ga[MT][4], ua[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ga[i][j] = ua[i][j] = 0.0f;
        for (int s = s0; s < s1; s += kGateUnroll) {
            if (s + kGateUnroll < s1)
                load(unit, s + kGateUnroll, next);
            else
                load(unit + gridDim.x, s0, next);
#pragma unroll
            for (int u = 0; u < kGateUnroll; ++u) {
                if (s + u >= s1)
                    break;
                uint32_t sga[2], sgb[2], sua[2], sub[2];
                decode_scales(now.gate[u].fa, sga);
                decode_scales(now.gate[u].fb, sgb);
                decode_scales(now.up[u].fa, sua);
                decode_scales(now.up[u].fb, sub);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if (!on[i]) // few experts have more than eight tokens: those decode twice
                        break;
                    uint4 x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[j] = have[i] && (s + u) * kStep < left
                                   ? __ldg(reinterpret_cast<const uint4 *>(xr[i] + (s + u) * kStep + 8 * j))
                                   : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t pa[4], pb[4];
                        now.gate[u].decode(j, sga, sgb, pa, pb);
                        multiply(ga[i], pa, pb, x[j]);
                        now.up[u].decode(j, sua, sub, pa, pb);
                        multiply(ua[i], pa, pb, x[j]);
                    }
                }
            }
            now = next;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if (!on[i])
                break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = g + (j >> 1) * 8, col = 8 * i + 2 * t + (j & 1);
                red[warp][row][col] = ga[i][j];
                red[warp][kRows + row][col] = ua[i][j];
            }
        }
        __syncthreads();
        const float scale = __ldg(p.sg13 + e) * 65536.0f, out = __ldg(p.sg2 + e);
        for (int i = threadIdx.x; i < kRows * many; i += 32 * kGateWarps) {
            const int row = i % kRows, n = i / kRows, tok = list[n];
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kGateWarps; ++w) {
                gate += red[w][row][n];
                up += red[w][kRows + row][n];
            }
            gate *= scale;
            up *= scale;
            const int j = r.choice[e][tok];
            const float a = __fdiv_rn(gate, 1.0f + expf(-gate)) * up * (r.p[tok][j] * out);
            __nv_bfloat16 part[PARTS];
            split<PARTS>(a, part);
            __nv_bfloat16 *at =
                p.act + (int64_t)(tok * p.topk + j) * PARTS * p.inter + unit % blocks * kRows + row;
#pragma unroll
            for (int k = 0; k < PARTS; ++k)
                at[(int64_t)k * p.inter] = part[k];
        }
        __syncthreads();
    }
}

constexpr int kDownUnroll = 2;

// NT: tiles of eight columns; a token has COLS columns (PARTS of them in use).
template <int NT, int COLS, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps == 16 ? 1 : 2) k_moe_down(const MoeParams p)
{
    constexpr int kParts = COLS == 4 ? 3 : 2, kTok = 8 / COLS; // tokens a tile
    __shared__ Routes r;
    __shared__ float red[kWarps][kRows][kTok * NT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    choose(p, r); // from the logits, which were there before this kernel could start
    const int steps = (p.inter + kStep - 1) / kStep;
    const int total = r.slots * steps; // (slot, K step) pairs
    const int i0 = (int)((int64_t)total * warp / kWarps), i1 = (int)((int64_t)total * (warp + 1) / kWarps);
    const int64_t row0 = (int64_t)blockIdx.x * kRows;
    const int left = p.inter - 32 * t;

    struct Batch {
        Codes c[kDownUnroll];
    };
    struct Cursor { // a (slot, K step) pair
        int slot, s;
        __device__ __forceinline__ void advance(int steps)
        {
            if (++s == steps) {
                s = 0;
                ++slot;
            }
        }
    };
    Cursor ahead = {i0 / steps, i0 % steps}, here = ahead;
    auto load = [&](int i, Batch &b) {
#pragma unroll
        for (int u = 0; u < kDownUnroll; ++u) {
            b.c[u].clear();
            if (i + u < i1) {
                const int slot = ahead.slot, s = ahead.s;
                ahead.advance(steps);
                if (s * kStep < left) {
                    const int64_t row = (int64_t)r.expert[slot] * p.h + row0 + g;
                    b.c[u].load(p.q2 + row * (p.inter / 2) + 16 * t, p.sb2 + row * (p.inter / 16) + 2 * t, p.inter, s);
                }
            }
        }
    };
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = 0.0f;
    Batch now, next;
    load(i0, now);
    ptx::grid_dep_wait(); // the activations
    ptx::grid_dep_launch();
    for (int i = i0; i < i1; i += kDownUnroll) {
        load(i + kDownUnroll, next);
#pragma unroll
        for (int u = 0; u < kDownUnroll; ++u) {
            if (i + u >= i1)
                break;
            const int s = here.s, e = r.expert[here.slot];
            here.advance(steps);
            const unsigned tokens = r.tokens[e];
            uint32_t sa[2], sb[2], pa[4][4], pb[4][4];
            decode_scales(now.c[u].fa, sa);
            decode_scales(now.c[u].fb, sb);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                now.c[u].decode(j, sa, sb, pa[j], pb[j]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if ((tokens >> (n * kTok) & ((1u << kTok) - 1u)) == 0) // no token of this tile takes the expert
                    continue;
                const int tok = n * kTok + g / COLS, part = g % COLS;
                const bool have = part < kParts && (tokens >> tok & 1u) && s * kStep < left;
                const __nv_bfloat16 *at = p.act;
                if (have)
                    at += ((int64_t)(tok * p.topk + r.choice[e][tok]) * kParts + part) * p.inter + s * kStep + 32 * t;
                uint4 x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[j] = have ? __ldcg(reinterpret_cast<const uint4 *>(at) + j) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    multiply(acc[n], pa[j], pb[j], x[j]);
            }
        }
        now = next;
    }
    // the parts of a token's sum lie in neighbouring columns
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float v = acc[n][2 * half] + acc[n][2 * half + 1];
            if (COLS == 4)
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
            if (COLS == 2 || (t & 1) == 0)
                red[warp][g + 8 * half][n * kTok + (COLS == 2 ? t : t >> 1)] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * p.m; i += 32 * kWarps) {
        const int row = i % kRows, tok = i / kRows;
        float a = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            a += red[w][row][tok];
        a *= 65536.0f; // of the decoding
        const int64_t at = tok * p.ldy + row0 + row;
        if (p.out_bf16)
            static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(a);
        else
            static_cast<float *>(p.y)[at] = a;
    }
}

template <int COLS, int kWarps>
cudaError_t run_down(const MoeParams &p, cudaStream_t st)
{
    const dim3 grid((unsigned)(p.h / kRows)), block(32 * kWarps);
    constexpr int kTok = 8 / COLS;
    if (p.m <= kTok)
        return launch_pdl(k_moe_down<1, COLS, kWarps>, grid, block, 0, st, p);
    if (p.m <= 2 * kTok)
        return launch_pdl(k_moe_down<2, COLS, kWarps>, grid, block, 0, st, p);
    if constexpr (COLS == 4)
        if (p.m > 4 * kTok)
            return launch_pdl(k_moe_down<8, COLS, kWarps>, grid, block, 0, st, p);
    return launch_pdl(k_moe_down<4, COLS, kWarps>, grid, block, 0, st, p);
}

size_t logits_bytes(int64_t m, int64_t experts)
{
    return ((size_t)m * (size_t)experts * 4 + 15) / 16 * 16;
}

} // namespace

size_t moe_nvfp4_workspace(int64_t m, int64_t experts, int64_t inter, int64_t topk)
{
    return logits_bytes(m, experts) + (size_t)m * (size_t)topk * 3 * (size_t)inter * 2;
}

cudaError_t launch_moe_nvfp4(const MoeNvfp4Args &a, cudaStream_t st)
{
    MoeParams p = {};
    p.x = a.x;
    p.router = a.router;
    p.ldx = a.ldx;
    p.ldr = a.ldr;
    p.m = (int)a.m;
    p.h = (int)a.h;
    p.inter = (int)a.inter;
    p.experts = (int)a.experts;
    p.topk = (int)a.topk;
    p.renorm = a.renorm != 0;
    p.q13 = a.q13;
    p.sb13 = a.sb13;
    p.sg13 = a.sg13;
    p.q2 = a.q2;
    p.sb2 = a.sb2;
    p.sg2 = a.sg2;
    p.logits = static_cast<float *>(a.ws);
    p.act = reinterpret_cast<__nv_bfloat16 *>(static_cast<uint8_t *>(a.ws) + logits_bytes(a.m, a.experts));
    p.ids = a.ids;
    p.weights = a.weights;
    p.y = a.y;
    p.ldy = a.ldy;
    p.out_bf16 = a.out_dtype == JETQ_OUT_BF16;
    cudaError_t e = launch_pdl(k_moe_router, dim3((unsigned)a.experts), dim3(kRouterThreads), 0, st, p);
    if (e != cudaSuccess)
        return e;
    // as many CTAs as run at a time, or units at most
    const int64_t used = a.m * a.topk < a.experts ? a.m * a.topk : a.experts, units = used * (a.inter / kRows);
    const int64_t cap = 2 * (int64_t)sm_count();
    const dim3 grid((unsigned)(units < cap ? units : cap)), block(32 * kGateWarps);
    if (p.out_bf16)
        e = a.m <= 8 ? launch_pdl(k_moe_gate_up<1, 2>, grid, block, 0, st, p)
                     : launch_pdl(k_moe_gate_up<2, 2>, grid, block, 0, st, p);
    else
        e = a.m <= 8 ? launch_pdl(k_moe_gate_up<1, 3>, grid, block, 0, st, p)
                     : launch_pdl(k_moe_gate_up<2, 3>, grid, block, 0, st, p);
    if (e != cudaSuccess)
        return e;
    if (a.h / kRows <= sm_count())
        return p.out_bf16 ? run_down<2, 16>(p, st) : run_down<4, 16>(p, st);
    return p.out_bf16 ? run_down<2, 8>(p, st) : run_down<4, 8>(p, st);
}

} // namespace jetq
