// A whole mixture-of-experts layer for 1 to 16 tokens: BF16 router, NVFP4
// expert weights, BF16 activations that are not quantized.
//
//   l[i, e] = sum_k x[i, k] * router[e, k];   the topk largest (the lower index first among equals)
//   p       = exp(l) over their sum (renorm) or over the sum of all experts
//   a       = silu(gate x) * (up x),   y[i] = sum over the chosen of p * down a
//
// Floor: the chosen experts' weights from HBM (9/16 byte each).  Three kernels:
//   1. router logits, a CTA an expert;
//   2. gate and up: a unit is 8 rows of gate and the same 8 of up of one chosen
//      expert, for all tokens that chose it.  Both are contiguous in memory: a
//      producer thread keeps a ring of bulk copies into shared memory ahead of
//      one to four groups of warps, which take a unit each and share its K;
//   3. down: a CTA owns 16 rows of y and runs through all chosen experts in the
//      same way, its 16 warps sharing (expert, K) steps, so that y is summed in
//      the CTA's registers and written once, without atomics.
// Each CTA of kernel 2 chooses the experts from the logits itself (3 to 4 us, in
// place of another kernel), and the first one leaves its choices to kernel 3.
// Measured in a graph, 128 experts of which 8 are taken, 2048/768: one token 23 to 25 us
// (HBM 3.2; the launches, the choice and the kernels' first copies are most of
// it), sixteen tokens (82 experts) 92 us: router 5, choice 4, gate and up 36, down
// 37, HBM 32; the last two use half of the issue slots, most of them to decode.
// Loads issued by the threads themselves, with K shared by eight warps: 145 us.
// Rows copied one by one to a pitch without bank conflicts: 147 us (a bulk copy
// costs about 50 ns, whatever its size).  The down weights of few experts
// prefetched into L2 by kernel 2's idle lanes: one token 24.7 us for 22.7, two
// 32.9 for 30.9, five 55 for 50; they take the bandwidth that gate and up need.
//
// Both products run on mma.m16n8k16 (weight rows as M, tokens as N), decoded
// in registers as in the few-token product.  In the first, rows 0 to 7 of the M
// axis are gate and 8 to 15 up, so that a lane holds both of an activation's
// factors.  In the second the activations are FP32 values p * sg * a: each goes
// in as two BF16 numbers (16 bits; a BF16 y rounds to 8) or, for an FP32 y,
// three (24 bits), in columns of their own that are added at the end, so nothing
// is rounded between the two products beyond that.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "jetq_internal.h"
#include "nvfp4_mma.cuh"
#include "ptx.cuh"

namespace jetq {

__device__ unsigned g_moe_error;

namespace {

constexpr unsigned kErrTimeout = 1u;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

constexpr int kMaxTokens = 16, kMaxExperts = 256, kMaxTop = 16;
constexpr int kStep = 128;             // columns a warp step
constexpr int kConsumers = 16;         // warps that compute; one more copies
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kMaxStages = 28;         // buffers of a ring
constexpr int kRingBytes = 192 * 1024;

struct MoeParams {
    const uint16_t *x, *router;
    int64_t ldx, ldr;
    int m, h, inter, experts, topk;
    bool renorm;
    const uint8_t *q13, *sb13, *q2, *sb2;
    const float *sg13, *sg2;
    float *logits;        // [m][experts]
    __half *x16;          // [m][h]: x times a power of two, and its inverse [m]
    float *unscale;
    struct Routes *routes; // kernel 2's choices, for kernel 3
    __nv_bfloat16 *act;   // [m * topk][parts][inter], eights in the order 0 4 1 5 2 6 3 7: the weights' pairs
    int64_t *ids;
    float *weights;
    void *y;
    int64_t ldy;
    int out_bf16;
    int depth;       // of the kernel's ring: buffers a group (gate and up)
    int buffers;     // in all
    unsigned long long limit_ns;
};

constexpr int kRouterThreads = 256;

// A token's x as FP16 for the first product: times the power of two that puts
// its largest value in [2^14, 2^15), which is exact for all values down to 2^-30
// of the largest (below, FP16's steps of 2^-24 are at most 2^-38 of it).
__device__ __forceinline__ void scale_token(const MoeParams &p, int tok, float *red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t *x = p.x + tok * p.ldx;
    float m = 0.0f;
    for (int k = 8 * threadIdx.x; k < p.h; k += 8 * kRouterThreads) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(x + k));
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) // passes over NaN, which stays one in FP16
            m = fmaxf(m, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xffff0000u))));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (lane == 0)
        red[warp] = m;
    __syncthreads();
    for (int g = 0; g < kRouterThreads / 32; ++g)
        m = fmaxf(m, red[g]);
    // 2^(14 - exponent of m), at most 2^114; 1 for no largest number
    const int e = m > 0.0f && m < INFINITY ? (int)(__float_as_uint(m) >> 23) - 127 : 14;
    const int up = min(14 - e, 114);
    const float f = __uint_as_float((uint32_t)(127 + up) << 23);
    if (threadIdx.x == 0)
        p.unscale[tok] = __uint_as_float((uint32_t)(127 - up) << 23);
    for (int k = 8 * threadIdx.x; k < p.h; k += 8 * kRouterThreads) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(x + k));
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h =
                __floats2half2_rn(__uint_as_float(u[i] << 16) * f, __uint_as_float(u[i] & 0xffff0000u) * f);
            v[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p.x16 + (int64_t)tok * p.h + k) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// Logits of one expert for eight tokens (blockIdx.y); the CTA's threads share K.
// The CTAs past the experts scale a token each.
__global__ void __launch_bounds__(kRouterThreads) k_moe_router(const MoeParams p)
{
    __shared__ float red[kRouterThreads / 32][8];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    if ((int)blockIdx.x >= p.experts) {
        const int tok = (int)blockIdx.x - p.experts + 8 * (int)blockIdx.y;
        if (tok < p.m)
            scale_token(p, tok, &red[0][0]);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t *w = p.router + (int64_t)blockIdx.x * p.ldr;
    const int t0 = 8 * (int)blockIdx.y;
    {
        float2 acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[i] = make_float2(0.0f, 0.0f);
        for (int k = 8 * threadIdx.x; k < p.h; k += 8 * kRouterThreads) { // h and the rows are whole vectors
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(w + k));
            uint4 b[8]; // all in flight; past the last token its row again
#pragma unroll
            for (int i = 0; i < 8; ++i)
                b[i] = __ldg(reinterpret_cast<const uint4 *>(p.x + min(t0 + i, p.m - 1) * p.ldx + k));
            const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t v[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i] = __ffma2_rn(make_float2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u)),
                                        make_float2(__uint_as_float(v[e] << 16), __uint_as_float(v[e] & 0xffff0000u)),
                                        acc[i]);
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
        if (threadIdx.x < 8 && t0 + (int)threadIdx.x < p.m) {
            float s = 0.0f;
#pragma unroll
            for (int g = 0; g < kRouterThreads / 32; ++g)
                s += red[g][threadIdx.x];
            p.logits[(int64_t)(t0 + threadIdx.x) * p.experts + blockIdx.x] = s;
        }
    }
}

// Which experts the tokens take.  Slots number the experts that some token
// takes, in rising order.
struct alignas(16) Routes {
    int id[kMaxTokens][kMaxTop];
    float p[kMaxTokens][kMaxTop];
    unsigned tokens[kMaxExperts];           // bit i: token i takes the expert
    uint8_t choice[kMaxExperts][kMaxTokens]; // which of the token's choices the expert is
    short expert[kMaxExperts];              // of a slot
    uint8_t list[kMaxExperts][kMaxTokens];  // a slot's tokens, in rising order
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
        unsigned key[kMaxExperts / 32], best = 0;
        int at = 0;
        float all = 0.0f;
        auto local_best = [&]() {
            best = 0;
#pragma unroll
            for (int i = 0; i < kMaxExperts / 32; ++i)
                if (key[i] > best) { // the first of equals
                    best = key[i];
                    at = 32 * i + lane;
                }
        };
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i) {
            const int e = 32 * i + lane;
            key[i] = e < p.experts ? order_key(__ldcg(p.logits + (int64_t)t * p.experts + e)) : 0u;
        }
        local_best();
        unsigned mine = 0, top = 0;
        int id = 0;
        for (int j = 0; j < p.topk; ++j) {
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
            if (lane == w % 32) { // the lane that held it looks for its next
#pragma unroll
                for (int i = 0; i < kMaxExperts / 32; ++i)
                    if (32 * i + lane == w)
                        key[i] = 0;
                local_best();
            }
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
    for (int i = threadIdx.x; i < r.slots; i += blockDim.x) {
        unsigned left = r.tokens[r.expert[i]];
        for (int n = 0; left; ++n, left &= left - 1u)
            r.list[i][n] = (uint8_t)(__ffs(left) - 1);
    }
    __syncthreads();
}

__device__ __forceinline__ void mma_16816_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's 32 codes of a weight row with their two scales, as the pairs that the MMA takes.  FP16: pairs of
// neighbours; an E2M1 pair is one conversion, times the block scale exact in FP16 (6 significant bits, 2^-10 to 2688).
__device__ __forceinline__ void decode_half(const uint4 &w, uint32_t scales, uint32_t (&out)[4][4])
{
    uint32_t s2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"((uint16_t)scales));
    const uint32_t s[2] = {__byte_perm(s2, 0, 0x1010), __byte_perm(s2, 0, 0x3232)};
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t v[4];
        asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4; cvt.rn.f16x2.e2m1x2 %0, a; "
            "cvt.rn.f16x2.e2m1x2 %1, b; cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d;}"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
            : "r"(u[j]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 q = __hmul2(*reinterpret_cast<const __half2 *>(&v[i]),
                                      *reinterpret_cast<const __half2 *>(&s[j >> 1]));
            out[j][i] = *reinterpret_cast<const uint32_t *>(&q);
        }
    }
}

// BF16: pairs (0, 4), (1, 5), (2, 6), (3, 7) of each eight, times 2^-16.
__device__ __forceinline__ void decode_bf16(const uint4 &w, uint32_t scales, uint32_t (&out)[4][4])
{
    uint32_t s[2];
    decode_scales(scales, s);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        decode8(u[j], s[j >> 1], out[j]);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t lds16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
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

// The ring: `groups` times `depth` buffers, each filled by the producer thread's
// bulk copies (full) and given back by the warps that read it (empty).  Item i
// is group i % groups' own and goes through that group's buffers in turn, so that
// the same warps follow every phase of a barrier: a wait knows a phase by its
// parity only, and a reader that skipped items of others in a common ring could
// take an older phase for its own.
struct Ring {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int abort_word;
};

__device__ __forceinline__ void init_ring(Ring &ring, int buffers, int readers)
{
    if (threadIdx.x == 0) {
        ring.abort_word = 0;
        for (int s = 0; s < buffers; ++s) {
            ptx::mbar_init(ptx::smem_addr(&ring.full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&ring.empty[s]), readers);
        }
        ptx::fence_barrier_init();
    }
    // the caller's next __syncthreads makes them visible
}

// The producer thread: copy(i, buffer, barrier) issues the `bytes` of item i, for each of `items`.
template <class F>
__device__ __forceinline__ void produce(Ring &ring, int groups, int depth, int items, uint32_t bytes,
                                        unsigned long long limit_ns, F copy)
{
    volatile int *abort_flag = &ring.abort_word;
    int i = 0, g = 0, c = 0; // the item's group and place in its buffers
    uint32_t ph = 0;
    for (; i < items; ++i) {
        const int s = g * depth + c;
        if (!ptx::mbar_wait(ptx::smem_addr(&ring.empty[s]), ph ^ 1u, abort_flag, &g_moe_error, kErrTimeout, limit_ns))
            break;
        const uint32_t bar = ptx::smem_addr(&ring.full[s]);
        ptx::mbar_arrive_expect_tx(bar, bytes);
        copy(i, s, bar);
        if (++g == groups) {
            g = 0;
            if (++c == depth) {
                c = 0;
                ph ^= 1u;
            }
        }
    }
    // no copy may be in flight when the CTA ends: the last one of each buffer
    for (g = 0; g < groups && g < i; ++g) {
        const int mine = (i - 1 - g) / groups + 1; // the group's items
        for (c = 0; c < depth && c < mine; ++c)
            ptx::mbar_wait(ptx::smem_addr(&ring.full[g * depth + c]), (uint32_t)((mine - 1 - c) / depth) & 1u,
                           abort_flag, &g_moe_error, kErrTimeout, limit_ns, false);
    }
}

// A reader's place in its group's buffers, the first of which is `first`.
struct Place {
    int first, c;
    uint32_t ph;
    __device__ __forceinline__ int buffer() const { return first + c; }
    __device__ __forceinline__ void forward(int depth)
    {
        if (++c == depth) {
            c = 0;
            ph ^= 1u;
        }
    }
};

// After a timeout the warps still run through their items and meet their
// barriers, on whatever the buffers hold.
__device__ __forceinline__ void wait_full(Ring &ring, Place at, unsigned long long limit_ns)
{
    ptx::mbar_wait(ptx::smem_addr(&ring.full[at.buffer()]), at.ph, &ring.abort_word, &g_moe_error, kErrTimeout,
                   limit_ns);
    __syncwarp(); // the lanes go on to a warp's instructions
}

__device__ __forceinline__ void give_back(Ring &ring, Place at, int lane)
{
    __syncwarp();
    if (lane == 0)
        ptx::mbar_arrive(ptx::smem_addr(&ring.empty[at.buffer()]));
}

constexpr int kUnitRows = 8; // of gate and of up

// KS: warps that share a unit's K.  PARTS: BF16 numbers an activation is stored as.
template <int KS, int PARTS>
__global__ void __launch_bounds__(kThreads, 1) k_moe_gate_up(const MoeParams p)
{
    constexpr int kGroups = kConsumers / KS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Routes r;
    __shared__ Ring ring;
    __shared__ float red[2][kConsumers][2 * kUnitRows][9];
    uint8_t *buffers = ptx::align_smem<128>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    init_ring(ring, kGroups * p.depth, KS);
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    choose(p, r);
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < (int)(sizeof(Routes) / 16); i += blockDim.x)
            reinterpret_cast<uint4 *>(p.routes)[i] = reinterpret_cast<const uint4 *>(&r)[i];
        for (int i = threadIdx.x; i < p.m * p.topk; i += blockDim.x) {
            if (p.ids)
                p.ids[i] = r.id[i / p.topk][i % p.topk];
            if (p.weights)
                p.weights[i] = r.p[i / p.topk][i % p.topk];
        }
    }
    const int blocks = p.inter / kUnitRows, units = r.slots * blocks;
    const int items = units > (int)blockIdx.x ? (units - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
    // a buffer: gate codes, up codes (4 h bytes each), gate scales, up scales (h / 2 each)
    const uint32_t codes = 4u * p.h, scales = (uint32_t)p.h / 2, bytes = 2 * (codes + scales);

    if (warp == kConsumers) {
        if (lane == 0)
            produce(ring, kGroups, p.depth, items, bytes, p.limit_ns, [&](int i, int s, uint32_t bar) {
                const int unit = (int)blockIdx.x + i * (int)gridDim.x;
                const int64_t row =
                    (int64_t)r.expert[unit / blocks] * 2 * p.inter + (int64_t)(unit % blocks) * kUnitRows;
                const uint32_t dst = ptx::smem_addr(buffers) + (uint32_t)s * bytes;
                const uint8_t *q = p.q13 + row * (p.h / 2), *sb = p.sb13 + row * (p.h / 16);
                ptx::bulk_load(dst, q, codes, bar);
                ptx::bulk_load(dst + codes, q + (int64_t)p.inter * (p.h / 2), codes, bar);
                ptx::bulk_load(dst + 2 * codes, sb, scales, bar);
                ptx::bulk_load(dst + 2 * codes + scales, sb + (int64_t)p.inter * (p.h / 16), scales, bar);
            });
        __syncwarp();
        return;
    }

    const int group = warp / KS, kw = warp % KS;
    const int steps = (p.h + kStep - 1) / kStep;
    const int s0 = steps * kw / KS, s1 = steps * (kw + 1) / KS;
    const int left = p.h - 32 * t; // columns from this lane's first one on
    const int jump = kGroups * (int)gridDim.x, jump_slots = jump / blocks, jump_blocks = jump - jump_slots * blocks;
    int unit = (int)blockIdx.x + group * (int)gridDim.x, slot = unit / blocks, block = unit - slot * blocks;
    int buf = 0;
    Place at = {group * p.depth, 0, 0};
    // eight of a unit's tokens at a time (few experts have more); the values of x are loaded a step ahead
    struct Columns {
        const __half *row; // of this lane's token
        bool have;
    };
    auto columns = [&](int slot, int n0) {
        const bool have = n0 + g < __popc(r.tokens[r.expert[slot]]);
        return Columns{p.x16 + (have ? (int64_t)r.list[slot][n0 + g] * p.h : 0) + 32 * t, have};
    };
    // null: zeros (from a line of zeros in memory they took twice as long as everything else)
    auto source = [&](const Columns &c, int s) { return c.have && s * kStep < left ? c.row + s * kStep : nullptr; };
    auto load = [&](const __half *from, uint4 (&x)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = from ? reinterpret_cast<const uint4 *>(from)[j] : make_uint4(0, 0, 0, 0);
    };
    uint4 x[4], next[4];
    Columns here = unit < units ? columns(slot, 0) : Columns{nullptr, false};
    load(source(here, s0), x);
    for (; unit < units; unit += jump, at.forward(p.depth)) {
        const int e = r.expert[slot], row0 = block * kUnitRows, this_slot = slot;
        const int many = __popc(r.tokens[e]);
        const uint8_t *list = r.list[slot];
        const float scale = __ldg(p.sg13 + e), out = __ldg(p.sg2 + e);
        const uint32_t from = ptx::smem_addr(buffers) + (uint32_t)at.buffer() * bytes;
        const uint32_t row_q = from + (uint32_t)(g * (p.h / 2));
        const uint32_t row_s = from + 2 * codes + (uint32_t)(g * (p.h / 16));
        slot += jump_slots; // the next unit's
        block += jump_blocks;
        if (block >= blocks) {
            block -= blocks;
            ++slot;
        }
        for (int n0 = 0; n0 < many; n0 += 8) {
            const bool last = n0 + 8 >= many;
            Columns then = {nullptr, false};
            if (!last)
                then = columns(this_slot, n0 + 8);
            else if (unit + jump < units)
                then = columns(slot, 0);
            if (n0 == 0)
                wait_full(ring, at, p.limit_ns);
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}; // gate, gate, up, up of row g, tokens 2t and 2t + 1
#pragma unroll 2
            for (int s = s0; s < s1; ++s) {
                load(s + 1 < s1 ? source(here, s + 1) : source(then, s0), next);
                // this lane's 32 columns of the rows; lanes past their end multiply zeros by their start
                const uint32_t k = s * kStep < left ? (uint32_t)(s * (kStep / 32) + t) : 0u;
                uint32_t wa[4][4], wb[4][4];
                decode_half(lds128(row_q + 16u * k), lds16(row_s + 2u * k), wa);
                decode_half(lds128(row_q + codes + 16u * k), lds16(row_s + scales + 2u * k), wb);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mma_16816_f16(acc, wa[j][0], wb[j][0], wa[j][1], wb[j][1], x[j].x, x[j].y);
                    mma_16816_f16(acc, wa[j][2], wb[j][2], wa[j][3], wb[j][3], x[j].z, x[j].w);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[j] = next[j];
            }
            if (s0 >= s1)
                load(source(then, s0), x);
            here = then;
            if (last)
                give_back(ring, at, lane);
            float(&sums)[2 * kUnitRows][9] = red[buf][warp];
            sums[g][2 * t] = acc[0];
            sums[g][2 * t + 1] = acc[1];
            sums[kUnitRows + g][2 * t] = acc[2];
            sums[kUnitRows + g][2 * t + 1] = acc[3];
            ptx::named_bar_sync(1 + group, 32 * KS);
            // the few sums are done by another warp each time
            for (int k = ((kw + unit) % KS) * 32 + lane; k < kUnitRows * min(8, many - n0); k += 32 * KS) {
                const int row = k % kUnitRows, n = k / kUnitRows, tok = list[n0 + n];
                float gate = 0.0f, up = 0.0f;
#pragma unroll
                for (int w = 0; w < KS; ++w) {
                    gate += red[buf][group * KS + w][row][n];
                    up += red[buf][group * KS + w][kUnitRows + row][n];
                }
                const float f = p.unscale[tok] * scale;
                gate *= f;
                up *= f;
                const int j = r.choice[e][tok];
                const float a = __fdiv_rn(gate, 1.0f + expf(-gate)) * up * (r.p[tok][j] * out);
                __nv_bfloat16 part[PARTS];
                split<PARTS>(a, part);
                static_assert(kUnitRows == 8, "an eight of activations");
                __nv_bfloat16 *to = p.act + (int64_t)(tok * p.topk + j) * PARTS * p.inter + row0 +
                                    (row < 4 ? 2 * row : 2 * row - 7);
#pragma unroll
                for (int q = 0; q < PARTS; ++q)
                    to[(int64_t)q * p.inter] = part[q];
            }
            buf ^= 1; // the other half: the next barrier tells that this one has been read
        }
    }
}

constexpr int kDownRows = 16;

// COLS: columns of a token (its activations' parts, and for three of them an
// empty one).  A slot's tokens, 8 / COLS at a time, take the eight columns of a
// tile; its sums are added to the warp's sums of the tokens in shared memory.
template <int COLS>
__global__ void __launch_bounds__(kThreads, 1) k_moe_down(const MoeParams p)
{
    constexpr int kParts = COLS == 4 ? 3 : 2, kTok = 8 / COLS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Routes r;
    __shared__ Ring ring;
    __shared__ float red[kConsumers][kDownRows][kMaxTokens + 1];
    uint8_t *buffers = ptx::align_smem<128>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    ptx::grid_dep_wait(); // the choices and the activations
    ptx::grid_dep_launch();
    for (int i = threadIdx.x; i < (int)(sizeof(Routes) / 16); i += blockDim.x)
        reinterpret_cast<uint4 *>(&r)[i] = __ldcg(reinterpret_cast<const uint4 *>(p.routes) + i);
    __syncthreads();
    const int steps = (p.inter + kStep - 1) / kStep;
    // Warps that share a slot's K, a power of two: what leaves the fewest steps to the busiest warp, where the ring
    // has two buffers for each group that has a slot, or one for every slot.
    int share = kConsumers, depth = p.buffers;
    for (int k = kConsumers, best = 0x7FFFFFFF; k >= 1; k /= 2) {
        const int groups = kConsumers / k, used = min(groups, r.slots);
        const int cost = (r.slots + groups - 1) / groups * ((steps + k - 1) / k);
        if ((used == 1 || 2 * used <= p.buffers || (used == r.slots && used <= p.buffers)) && cost <= best) {
            best = cost;
            share = k;
            depth = p.buffers / used;
        }
    }
    init_ring(ring, p.buffers, share);
    __syncthreads();
    const int64_t row0 = (int64_t)blockIdx.x * kDownRows;
    // a buffer: 16 rows' codes (8 inter bytes), their scales (inter)
    const uint32_t codes = 8u * p.inter, scales = (uint32_t)p.inter, bytes = codes + scales;
    if (warp == kConsumers) {
        if (lane == 0)
            produce(ring, kConsumers / share, depth, r.slots, bytes, p.limit_ns, [&](int i, int s, uint32_t bar) {
                const int64_t row = (int64_t)r.expert[i] * p.h + row0;
                const uint32_t dst = ptx::smem_addr(buffers) + (uint32_t)s * bytes;
                ptx::bulk_load(dst, p.q2 + row * (p.inter / 2), codes, bar);
                ptx::bulk_load(dst + codes, p.sb2 + row * (p.inter / 16), scales, bar);
            });
    } else {
        const int groups = kConsumers / share, group = warp / share, kw = warp % share;
        const int left = p.inter - 32 * t;
        for (int i = lane; i < kDownRows * p.m; i += 32)
            red[warp][i % kDownRows][i / kDownRows] = 0.0f;
        __syncwarp();
        // activations of tile n0 of a slot, loaded a step ahead
        struct Columns {
            const __nv_bfloat16 *row; // this lane's token's part
            bool have;
        };
        auto columns = [&](int slot, int n0) {
            const int e = r.expert[slot], n = n0 + g / COLS, part = g % COLS;
            Columns c = {p.act + 32 * t, n < __popc(r.tokens[e]) && part < kParts};
            if (c.have) {
                const int tok = r.list[slot][n];
                c.row += ((int64_t)(tok * p.topk + r.choice[e][tok]) * kParts + part) * p.inter;
            }
            return c;
        };
        auto source = [&](const Columns &c, int s) { return c.have && s * kStep < left ? c.row + s * kStep : nullptr; };
        auto load = [&](const __nv_bfloat16 *from, uint4 (&x)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = from ? __ldcg(reinterpret_cast<const uint4 *>(from) + j) : make_uint4(0, 0, 0, 0);
        };
        uint4 x[4], next[4];
        Columns here = group < r.slots ? columns(group, 0) : Columns{nullptr, false};
        load(source(here, kw), x);
        Place at = {group * depth, 0, 0};
        for (int i = group; i < r.slots; i += groups, at.forward(depth)) {
            const int many = __popc(r.tokens[r.expert[i]]);
            const uint32_t from = ptx::smem_addr(buffers) + (uint32_t)at.buffer() * bytes;
            const uint32_t row_q = from + (uint32_t)(g * (p.inter / 2));
            const uint32_t row_s = from + codes + (uint32_t)(g * (p.inter / 16));
            for (int n0 = 0; n0 < many; n0 += kTok) {
                const bool last = n0 + kTok >= many;
                Columns then = {nullptr, false};
                if (!last)
                    then = columns(i, n0 + kTok);
                else if (i + groups < r.slots)
                    then = columns(i + groups, 0);
                if (n0 == 0)
                    wait_full(ring, at, p.limit_ns);
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
                for (int s = kw; s < steps; s += share) {
                    load(s + share < steps ? source(here, s + share) : source(then, kw), next);
                    // this lane's 32 columns of the rows; lanes past their end multiply zeros by their start
                    const uint32_t k = s * kStep < left ? (uint32_t)(s * (kStep / 32) + t) : 0u;
                    uint32_t wa[4][4], wb[4][4];
                    decode_bf16(lds128(row_q + 16u * k), lds16(row_s + 2u * k), wa);
                    decode_bf16(lds128(row_q + 4u * p.inter + 16u * k), lds16(row_s + (uint32_t)p.inter / 2 + 2u * k),
                                wb);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        mma_16816(acc, wa[j][0], wb[j][0], wa[j][1], wb[j][1], x[j].x, x[j].y);
                        mma_16816(acc, wa[j][2], wb[j][2], wa[j][3], wb[j][3], x[j].z, x[j].w);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[j] = next[j];
                }
                here = then; // warps without a step have none of any slot
                // the parts of a token's sum lie in neighbouring columns
                float v = acc[0] + acc[1], u = acc[2] + acc[3];
                if (COLS == 4) {
                    v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
                    u += __shfl_xor_sync(0xFFFFFFFFu, u, 1);
                }
                const int n = n0 + (COLS == 2 ? t : t >> 1);
                if (n < many && (COLS == 2 || (t & 1) == 0)) {
                    const int tok = r.list[i][n];
                    red[warp][g][tok] += v;
                    red[warp][g + 8][tok] += u;
                }
            }
            give_back(ring, at, lane);
        }
    }
    __syncthreads();
    if (warp == kConsumers)
        return;
    for (int i = threadIdx.x; i < kDownRows * p.m; i += 32 * kConsumers) {
        const int row = i % kDownRows, tok = i / kDownRows;
        float a = 0.0f;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w)
            a += red[w][row][tok];
        a *= 65536.0f; // of the decoding
        const int64_t to = tok * p.ldy + row0 + row;
        if (p.out_bf16)
            static_cast<__nv_bfloat16 *>(p.y)[to] = __float2bfloat16_rn(a);
        else
            static_cast<float *>(p.y)[to] = a;
    }
}

// Buffers that the ring has room for.
int64_t ring_room(int64_t buffer)
{
    const int64_t room = kRingBytes / buffer;
    return room < kMaxStages ? room : kMaxStages;
}

template <class K>
cudaError_t run_ring(K kern, std::atomic<unsigned long long> &configured, int64_t grid, int64_t buffer, MoeParams p,
                     cudaStream_t st)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !(configured.load(std::memory_order_relaxed) >> dev & 1u)) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes + 128)) !=
            cudaSuccess)
            return e;
        if (dev < 64)
            configured.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    return launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), (size_t)(p.buffers * buffer + 128), st, p);
}

template <int KS, int PARTS>
cudaError_t run_gate_up(MoeParams p, int64_t units, cudaStream_t st)
{
    static std::atomic<unsigned long long> configured{0};
    constexpr int kGroups = kConsumers / KS;
    const int64_t grid = units < sm_count() ? units : sm_count(), buffer = 9 * (int64_t)p.h;
    const int64_t room = ring_room(buffer) / kGroups, items = (units + grid - 1) / grid; // a group's; a CTA's at most
    const int64_t most = (items + kGroups - 1) / kGroups;
    p.depth = (int)(room < most ? room : most);
    p.buffers = p.depth * kGroups;
    return run_ring(k_moe_gate_up<KS, PARTS>, configured, grid, buffer, p, st);
}

// Warps that share a unit: eight where a CTA has few units, so that all of
// them run at a time; four (half the reductions) where it has many; more where
// the ring has no room for two buffers a group.  In a graph, eight and four: 768
// units (5 a CTA) 24.7 us both, 1536 units 35.0 and 32.9, sixteen tokens of 128
// experts (7900) 102.6 and 90.5.
template <int PARTS>
cudaError_t run_gate_up(const MoeParams &p, int64_t units, cudaStream_t st)
{
    const int64_t room = ring_room(9 * (int64_t)p.h);
    if (units > 8 * (int64_t)sm_count() && room >= 8)
        return run_gate_up<4, PARTS>(p, units, st);
    return room >= 4 ? run_gate_up<8, PARTS>(p, units, st) : run_gate_up<16, PARTS>(p, units, st);
}

template <int COLS>
cudaError_t run_down(MoeParams p, int64_t slots, cudaStream_t st)
{
    static std::atomic<unsigned long long> configured{0};
    const int64_t buffer = 9 * (int64_t)p.inter, room = ring_room(buffer);
    p.buffers = (int)(room < slots ? room : slots);
    return run_ring(k_moe_down<COLS>, configured, p.h / kDownRows, buffer, p, st);
}

// The workspace: logits, the tokens' inverse scales, the choices, x in FP16, the activations.
size_t logits_bytes(int64_t m, int64_t experts)
{
    return ((size_t)m * (size_t)experts * 4 + 15) / 16 * 16;
}

constexpr size_t kFixedBytes = kMaxTokens * sizeof(float) + sizeof(Routes);

} // namespace

size_t moe_nvfp4_workspace(int64_t m, int64_t experts, int64_t h, int64_t inter, int64_t topk)
{
    return logits_bytes(m, experts) + kFixedBytes + (size_t)m * (size_t)h * 2 +
           (size_t)m * (size_t)topk * 3 * (size_t)inter * 2;
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
    uint8_t *at = static_cast<uint8_t *>(a.ws) + logits_bytes(a.m, a.experts);
    p.unscale = reinterpret_cast<float *>(at);
    p.routes = reinterpret_cast<Routes *>(at + kMaxTokens * sizeof(float));
    p.x16 = reinterpret_cast<__half *>(at + kFixedBytes);
    p.act = reinterpret_cast<__nv_bfloat16 *>(at + kFixedBytes + (size_t)a.m * (size_t)a.h * 2);
    p.ids = a.ids;
    p.weights = a.weights;
    p.y = a.y;
    p.ldy = a.ldy;
    p.out_bf16 = a.out_dtype == JETQ_OUT_BF16;
    p.limit_ns = kWaitLimitNs;
    const dim3 router((unsigned)(a.experts + (a.m < 8 ? a.m : 8)), (unsigned)((a.m + 7) / 8));
    cudaError_t e = launch_pdl(k_moe_router, router, dim3(kRouterThreads), 0, st, p);
    if (e != cudaSuccess)
        return e;
    // slots at most
    const int64_t slots = a.m * a.topk < a.experts ? a.m * a.topk : a.experts, units = slots * (a.inter / kUnitRows);
    e = p.out_bf16 ? run_gate_up<2>(p, units, st) : run_gate_up<3>(p, units, st);
    if (e != cudaSuccess)
        return e;
    return p.out_bf16 ? run_down<2>(p, slots, st) : run_down<4>(p, slots, st);
}

cudaError_t moe_read_and_clear_error(cudaStream_t st, unsigned *out)
{
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_moe_error, sizeof v, 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(st);
    if (e != cudaSuccess)
        return e;
    *out |= v;
    if (v) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbolAsync(g_moe_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, st);
        if (e == cudaSuccess)
            e = cudaStreamSynchronize(st);
    }
    return e;
}

} // namespace jetq
