// Distillation of a linear head from a teacher that is known by its top
// logits: the steps around the head's products (linear_ce.cu).
//
//   z[i, j] = scale * sum_k x[i, k] * w[j, k],   lse[i] = log sum_j exp(z[i, j])
//   q       = softmax of the listed t (renorm) or exp(t),   Q = sum of q
//   loss[i] = sum over listed of q (log q - (z - lse))
//   d[i, j] = (Q p[i, j] - q[i, j]) * dloss[i],   p = exp(z - lse)
//   dx      = scale * d w,   dw = scale * d^T x
//
// The loss is a small difference of logits where teacher and student agree,
// and the listed columns hold most of a confident token's mass.  So their
// logits are not taken from the product's tensor-core sums: k_distill_rows sums
// them in FP32 with compensated joins and marks their columns, the product's
// statistics leave the marked columns out, and k_distill_join puts the exact
// terms in (losses of 2048 tokens were off by 2e-5 in the 2-norm where an FP32
// product gave the logits).  The backward product writes d = f Q p for every
// column, and k_distill_patch replaces the listed entries, where the two terms
// nearly cancel, by f (Q p - q) from the forward call's log-probabilities.
//
// d is BF16, the tensor cores' operand.  A confident token's d is a few large
// listed entries, whose rounding (2^-8) shows in a gradient: 2.2e-3 to 2.5e-3 in
// the 2-norm, where the rounding of BF16 results alone is 1.7e-3.  For dx, which
// all gradients before the head are made of, what a listed entry's BF16 value
// leaves of it, its rest, is added to the FP32 sums where the slabs are joined
// (k_distill_dx): dx is then at 1.7e-3, as with two BF16 terms for all of d, for
// 2% of the time at 777 tokens x 50257 x 1032 (253 to 258 us) and at 2048 x 131072
// x 4096, 7% at 8192 x 32000 x 512 with 64 entries (613 to 654).  dw takes d in
// BF16, as the cross entropy's does: a second term of d costs a third of the pass,
// and rests added in that product's epilogue cost 5% where the tokens list
// different columns but twice to five times the pass where many list the same
// (one row of dw takes all of their rows of x, in each of its tiles).
//
// Bound by the head's products, but for k_distill_rows, which reads the listed
// rows of w in the order of the tokens: 2048 tokens x 64 entries (half of them
// listed) x 4096 take 130 us at 3.7 TB/s, a tenth of the forward pass over 131072
// rows (1.31 to 1.35 ms for a few passes, 1.41 back to back at the power cap).  A
// single token's 32 entries are read under the product's first tiles (one token x
// 32000 x 4096 55 us in a graph, 38.6 of it HBM's).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "head_rows.cuh"
#include "jetq_internal.h"
#include "ptx.cuh"

namespace jetq {

namespace {

constexpr int kMaxListed = 256; // entries a row
__host__ __device__ constexpr int row_warps(int n) // of a CTA of k_distill_rows<n>
{
    return n == 1 ? 8 : 4;
}

__device__ __forceinline__ float2 unpack2(uint32_t u)
{
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// s + c of all lanes, as a two-sum.
__device__ __forceinline__ void warp_two_sum(float &s, float &c)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float s2 = __shfl_xor_sync(0xFFFFFFFFu, s, o), c2 = __shfl_xor_sync(0xFFFFFFFFu, c, o);
        two_sum(s, c, s2);
        c += c2;
    }
}

struct RowsParams {
    const uint16_t *x, *w;
    int64_t c, ldx, ldw, v;
    const int64_t *ids;
    int64_t ldi;
    int k, bn, parts;
    uint16_t *copy; // x in rows of whole lines, or null
    int64_t ldc;
    uint4 *skip;   // [n][parts]
    float2 *dots;  // [n][k]
};

// A row's CTAs (blockIdx.y): the last one writes its marks and its copy of x,
// the others the products of x with the listed rows of w, N a warp at a time (x
// is unpacked once for them).  Few rows take N = 1 and several CTAs for the
// products, with more loads in flight for each: a single token's 32 entries took
// 17 us by one CTA with N = 4.
template <int N>
__global__ void __launch_bounds__(32 * row_warps(N), N == 1 ? 2 : 6) k_distill_rows(const RowsParams p)
{
    constexpr int kRowWarps = row_warps(N);
    constexpr int kChunk = 1024;             // marks' 128-column parts at a time
    __shared__ __align__(16) uint32_t marks[kChunk * 4]; // read 16 bytes at a time
    __shared__ int64_t ids[kMaxListed];
    // The launch after the wait: the product may start on x and w, whose writers are through.
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int j = threadIdx.x; j < p.k; j += blockDim.x) {
        const int64_t id = __ldg(p.ids + row * p.ldi + j);
        ids[j] = id >= 0 && id < p.v ? id : -1;
    }
    __syncthreads();
    const uint16_t *x = p.x + row * p.ldx;
    const int shares = (int)gridDim.y - 1;
    for (int j0 = N * (warp + kRowWarps * (int)blockIdx.y); (int)blockIdx.y < shares && j0 < p.k;
         j0 += N * kRowWarps * shares) {
        const uint16_t *w[N];
        bool any = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t id = j0 + i < p.k ? ids[j0 + i] : -1;
            any |= id >= 0;
            w[i] = p.w + (id >= 0 ? id : 0) * p.ldw; // row 0 is there: its product is not used
        }
        float2 acc[N][4];
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][e] = make_float2(0.0f, 0.0f);
        if (any) {
#pragma unroll(N == 1 ? 8 : 2)
            for (int64_t k = 8 * lane; k < p.c; k += 256) { // c and the rows are whole vectors
                const uint4 a = __ldg(reinterpret_cast<const uint4 *>(x + k));
                uint4 b[N];
#pragma unroll
                for (int i = 0; i < N; ++i)
                    b[i] = __ldg(reinterpret_cast<const uint4 *>(w[i] + k));
                const float2 f[4] = {unpack2(a.x), unpack2(a.y), unpack2(a.z), unpack2(a.w)};
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const uint32_t u[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][e] = __ffma2_rn(f[e], unpack2(u[e]), acc[i][e]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = acc[i][0].x, c = 0.0f;
            two_sum(s, c, acc[i][0].y);
#pragma unroll
            for (int e = 1; e < 4; ++e) {
                two_sum(s, c, acc[i][e].x);
                two_sum(s, c, acc[i][e].y);
            }
            warp_two_sum(s, c);
            if (lane == 0 && j0 + i < p.k)
                p.dots[row * p.k + j0 + i] = make_float2(s, c);
        }
    }
    if ((int)blockIdx.y < shares)
        return;
    if (p.copy)
        for (int64_t k = 8 * threadIdx.x; k < p.c; k += 8 * blockDim.x)
            *reinterpret_cast<uint4 *>(p.copy + row * p.ldc + k) = __ldg(reinterpret_cast<const uint4 *>(x + k));
    for (int q0 = 0; q0 < p.parts; q0 += kChunk) {
        const int many = min(kChunk, p.parts - q0);
        for (int i = threadIdx.x; i < many * 4; i += blockDim.x)
            marks[i] = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < p.k; j += blockDim.x) {
            const int64_t id = ids[j];
            if (id < 0)
                continue;
            const int tile = (int)(id / p.bn), rel = (int)(id - (int64_t)tile * p.bn);
            const int at = 2 * tile + (rel >> 7) - q0; // two parts a tile
            if (at >= 0 && at < many)
                atomicOr(&marks[at * 4 + ((rel & 127) >> 5)], 1u << (rel & 31));
        }
        __syncthreads();
        for (int i = threadIdx.x; i < many; i += blockDim.x)
            p.skip[row * p.parts + q0 + i] = reinterpret_cast<const uint4 *>(marks)[i];
        __syncthreads();
    }
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

__device__ __forceinline__ float warp_add(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// log2 of a positive number as a whole part and the logarithm of a number in
// [0.75, 1.5), whose rounding is 2^-24 of at most 0.6.
__device__ __forceinline__ float2 split_log2(float s)
{
    if (!(s > 0.0f && s < INFINITY))
        return make_float2(log2f(s), 0.0f);
    int e;
    float f = frexpf(s, &e); // [0.5, 1)
    if (f < 0.75f) {
        f *= 2.0f;
        --e;
    }
    return make_float2((float)e, log2f(f));
}

// The listed entries of a row, entry j in lane j % 32: teacher's logits, their
// maximum and the sum of their exponentials.
struct Teacher {
    float top;   // what is subtracted of t: the maximum (renorm) or 0
    float2 log2; // of the sum of exp(t - top) (renorm), else 0
    float inv;   // 1 / that sum
    bool none;   // renorm, and nothing to normalize: q = 0
    template <class Id>
    __device__ __forceinline__ void load(const float *t, const Id *ids, int k, bool renorm, int lane)
    {
        top = 0.0f;
        log2 = make_float2(0.0f, 0.0f);
        inv = 1.0f;
        none = false;
        if (!renorm)
            return;
        float m = -INFINITY;
        bool nan = false;
        for (int j = lane; j < k; j += 32)
            if (ids[j] >= 0) {
                m = fmaxf(m, __ldg(t + j));
                nan |= isnan(__ldg(t + j));
            }
        m = warp_max(m);
        nan = __any_sync(0xFFFFFFFFu, nan);
        none = m == -INFINITY && !nan;
        top = none ? 0.0f : m;
        float s = 0.0f;
        for (int j = lane; j < k; j += 32)
            s += ids[j] >= 0 ? expf(__ldg(t + j) - top) : 0.0f;
        s = warp_add(s);
        if (none)
            return;
        log2 = split_log2(s);
        inv = __fdiv_rn(1.0f, s);
    }
    __device__ __forceinline__ float q(float t) const { return none ? 0.0f : expf(t - top) * inv; }
    __device__ __forceinline__ double log_q(float t) const
    {
        return ((double)t - (double)top) - (double)kLn2d * ((double)log2.x + (double)log2.y);
    }
    static constexpr double kLn2d = 0.69314718055994530942;
};

// Joins a row's pairs, the exact terms of its listed columns and the teacher:
// loss, lse and the listed log-probabilities.  `cta_rows` rows a CTA (eight, or
// one where there are few), a warp each once the pairs are joined.  Sums of the
// pairs: threadIdx % cta_rows walks rows (contiguous in part).
__global__ void __launch_bounds__(256)
    k_distill_join(int cta_rows, const float2 *part, int parts, const float2 *dots, const int64_t *ids, int64_t ldi,
                   const float *teacher, int64_t ldt, int k, int renorm, int64_t n, int64_t v, float scale, float k2,
                   float *loss, float *lse, float *logp)
{
    __shared__ float2 red[256];
    __shared__ int64_t list[8][kMaxListed];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t row0 = (int64_t)blockIdx.x * cta_rows;
    const int along = 256 / cta_rows; // threads along a row's pairs
    {
        const int rx = threadIdx.x % cta_rows, ry = threadIdx.x / cta_rows;
        const int64_t row = row0 + rx;
        float2 a = make_float2(-INFINITY, 0.0f);
        if (row < n)
            for (int q = ry; q < parts; q += 4 * along) { // four loads in flight
                float2 b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    b[i] = q + along * i < parts ? __ldg(part + (int64_t)(q + along * i) * n + row)
                                                 : make_float2(-INFINITY, 0.0f);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    join_pair(a, b[i]);
            }
        red[rx * along + ry] = a;
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = row0 + warp;
    if (warp >= cta_rows || row >= n)
        return;
    float2 a = red[warp * along + lane];
    for (int i = lane + 32; i < along; i += 32)
        join_pair(a, red[warp * along + i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float2 b = make_float2(__shfl_xor_sync(0xFFFFFFFFu, a.x, o), __shfl_xor_sync(0xFFFFFFFFu, a.y, o));
        join_pair(a, b);
    }
    a = make_float2(__shfl_sync(0xFFFFFFFFu, a.x, 0), __shfl_sync(0xFFFFFFFFu, a.y, 0));
    int64_t *mine = list[warp];
    for (int j = lane; j < k; j += 32) {
        const int64_t id = __ldg(ids + row * ldi + j);
        mine[j] = id >= 0 && id < v ? id : -1;
    }
    __syncwarp();
    // the listed columns' terms, each column's once
    float m = a.x;
    for (int j = lane; j < k; j += 32)
        if (mine[j] >= 0)
            m = fmaxf(m, (float)(whole_sum(dots[row * k + j].x, dots[row * k + j].y) * (double)k2));
    m = warp_max(m);
    const float base = fabsf(m) < INFINITY ? m : 0.0f;
    float s = 0.0f;
    for (int j = lane; j < k; j += 32) {
        bool first = mine[j] >= 0;
        for (int i = 0; first && i < j; ++i)
            first = mine[i] != mine[j];
        if (first) {
            const float2 z = dots[row * k + j];
            s += exp2f((float)(whole_sum(z.x, z.y) * (double)k2 - (double)base));
        }
    }
    s = warp_add(s) + a.y * (a.x == -INFINITY ? 1.0f : exp2f(a.x - base));
    const float2 l = split_log2(s);
    const double lse2 = (double)base + (double)l.x + (double)l.y;
    if (lane == 0)
        lse[row] = (float)(Teacher::kLn2d * lse2);
    Teacher t;
    t.load(teacher + row * ldt, mine, k, renorm != 0, lane);
    float sum = 0.0f;
    for (int j = lane; j < k; j += 32) {
        float lp = 0.0f;
        if (mine[j] >= 0) {
            const float2 z = dots[row * k + j];
            const double d = Teacher::kLn2d * (whole_sum(z.x, z.y) * (double)k2 - lse2);
            lp = (float)d;
            const float tj = __ldg(teacher + row * ldt + j), q = t.q(tj);
            if (q != 0.0f) // 0 log 0 = 0
                sum += q * (float)(t.log_q(tj) - d);
        }
        logp[row * k + j] = lp;
    }
    sum = warp_add(sum);
    if (lane == 0)
        loss[row] = sum;
}

// The start's words in the workspace, zero before it: gmax for the products' kernels first.
struct StartWords {
    float gmax;
    unsigned max_bits, ticket;
};

// Backward: rows of x copied to whole lines (zero for a row without a loss:
// the products run over every row, and 0 * NaN would reach all of dw), each
// row's GradRow and listed entries of d, a warp a row.  The last CTA to finish
// writes gmax = max |dloss| over the rows with a loss (1 where that is not finite).
__global__ void __launch_bounds__(256)
    k_distill_start(const uint16_t *x, int64_t n, int64_t c, int64_t ldx, uint16_t *out, int64_t ldo,
                    const int64_t *ids, int64_t ldi, const float *teacher, int64_t ldt, int k, int renorm, int64_t v,
                    const float *lse, const float *logp, const float *dloss, GradRow *rows, Listed *listed,
                    StartWords *start)
{
    __shared__ int list[8][kMaxListed]; // below 2^31, -1: none
    __shared__ float qs[8][kMaxListed];
    __shared__ float red[8];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int *mine = list[warp];
    float *q = qs[warp];
    // the teacher's probabilities of a row and their sum; whether there is a loss
    auto read_row = [&](int64_t r, float &Q) {
        bool any = false;
        for (int j = lane; j < k; j += 32) {
            const int64_t id = __ldg(ids + r * ldi + j);
            mine[j] = id >= 0 && id < v ? (int)id : -1;
            any |= mine[j] >= 0;
        }
        __syncwarp();
        Teacher t;
        t.load(teacher + r * ldt, mine, k, renorm != 0, lane);
        float s = 0.0f;
        for (int j = lane; j < k; j += 32) {
            q[j] = mine[j] >= 0 ? t.q(__ldg(teacher + r * ldt + j)) : 0.0f;
            s += q[j];
        }
        s = warp_add(s);
        Q = renorm && s > 0.0f ? 1.0f : s;
        __syncwarp();
        return __any_sync(0xFFFFFFFFu, any) && Q != 0.0f;
    };
    const int64_t step = (int64_t)gridDim.x * 8;
    float m = 0.0f; // of this warp's rows
    for (int64_t r = (int64_t)blockIdx.x * 8 + warp; r < n; r += step) {
        float Q;
        const bool has = read_row(r, Q);
        for (int64_t i = 8 * lane; i < c; i += 256) // c and the rows are whole vectors
            *reinterpret_cast<uint4 *>(out + r * ldo + i) =
                has ? __ldg(reinterpret_cast<const uint4 *>(x + r * ldx + i)) : make_uint4(0, 0, 0, 0);
        if (has) {
            const float g = fabsf(__ldg(dloss + r));
            m = g < INFINITY ? fmaxf(m, g) : INFINITY; // NaN too: the rows then keep their own values
        }
        if (lane == 0)
            rows[r] = has ? GradRow{-1, lse[r] * kLog2e, dloss[r] * Q, 0.0f} : GradRow{-1, 0.0f, 0.0f, 0.0f};
        for (int j = lane; j < k; j += 32) {
            Listed e = {-1, 0.0f};
            if (has && mine[j] >= 0) {
                // a column listed twice: its q is the sum, in the first of its entries
                const int own = mine[j];
                int last = -1; // the last entry of the column before this one
                float here = 0.0f, other = 0.0f;
                for (int i = 0; i < j; ++i) {
                    const bool same = mine[i] == own;
                    last = same ? i : last;
                    here += same ? q[i] : 0.0f;
                    other += same ? 0.0f : q[i];
                }
                for (int i = j; i < k; ++i) {
                    const bool same = mine[i] == own;
                    here += same ? q[i] : 0.0f;
                    other += same ? 0.0f : q[i];
                }
                if (last < 0) {
                    // Q p - q; for a confident token as Q (p - 1) + the other q, which keeps its small value
                    const float lp = __ldg(logp + r * k + j);
                    e.id = mine[j];
                    e.d = lp > -0.7f ? fmaf(Q, expm1f(lp), other) : fmaf(Q, expf(lp), -here);
                }
            }
            listed[r * k + j] = e;
        }
        __syncwarp();
    }
    // the largest of all: a maximum does not depend on the order of its atomics
    if (lane == 0)
        red[warp] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i)
            m = fmaxf(m, red[i]);
        atomicMax(&start->max_bits, __float_as_uint(m)); // not negative: ordered as its bits
        __threadfence();
        if (atomicAdd(&start->ticket, 1u) == gridDim.x - 1) {
            __threadfence();
            m = __uint_as_float(atomicMax(&start->max_bits, 0u));
            start->gmax = m < INFINITY ? m : 1.0f;
        }
    }
}

// d at a listed entry, in FP32: d is scaled by the largest |dloss|, f = dloss / gmax.
__device__ __forceinline__ float entry_of(float d, float dloss, float gmax)
{
    return d * (gmax > 0.0f ? __fdiv_rn(dloss, gmax) : 0.0f);
}

// d at the listed columns of a piece [col0, col0 + cols) of the vocabulary.
__global__ void __launch_bounds__(256)
    k_distill_patch(const Listed *listed, int64_t total, int k, const float *dloss, const float *gmax,
                    __nv_bfloat16 *d, int64_t ldd, int64_t col0, int64_t cols)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const float g = __ldg(gmax);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int2 e = __ldg(reinterpret_cast<const int2 *>(listed) + i);
        const int64_t rel = e.x - col0;
        if (e.x < 0 || rel < 0 || rel >= cols)
            continue;
        const int64_t r = i / k;
        d[r * ldd + rel] = __float2bfloat16_rn(entry_of(__int_as_float(e.y), __ldg(dloss + r), g));
    }
}

// dx = BF16(scale * gmax * (sum of the slabs + sum over a row's listed entries of their rest times w's row)), eight
// columns a thread.  The rests' rows of w are what it reads most of: 96 us at 2048 tokens x 64 entries (half of them
// listed) x 4096, 29 without them.  A warp along 256 columns, four that share the entries: 64 or 128 threads along
// wider pieces took 0 to 30% longer than the whole pass does with 32 (64 rows x 256 entries x 4096: 280 and 340 us
// for 261; 777 x 20 x 1032: 260 and 266 for 258).
constexpr int kDxThreads = 128;

__global__ void __launch_bounds__(kDxThreads)
    k_distill_dx(const float *slab, int slabs, int64_t n, int64_t c, const float *gmax, float scale,
                 const float *dloss, const Listed *listed, int k, const uint16_t *w, int64_t ldw, uint16_t *dx,
                 int64_t lddx)
{
    constexpr int kGroups = kDxThreads / 32, kTurns = kMaxListed / kDxThreads;
    __shared__ int64_t from[kMaxListed];
    __shared__ float rest[kMaxListed];
    __shared__ int many[kTurns * kGroups];
    __shared__ float2 sums[kGroups][4][32];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int64_t r = blockIdx.x, col = 8 * ((int64_t)blockIdx.y * 32 + lane);
    const float g = __ldg(gmax), loss = __ldg(dloss + r);
    // the row's entries that leave a rest, in their order
    float v[kTurns];
    int id[kTurns];
    unsigned on[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int j = i * kDxThreads + (int)threadIdx.x;
        int2 e = make_int2(-1, 0);
        if (j < k)
            e = __ldg(reinterpret_cast<const int2 *>(listed) + r * k + j);
        id[i] = e.x;
        v[i] = 0.0f;
        if (e.x >= 0) {
            const float d = entry_of(__int_as_float(e.y), loss, g);
            const float hi = __bfloat162float(__float2bfloat16_rn(d));
            v[i] = fabsf(hi) < INFINITY ? d - hi : 0.0f;
        }
        on[i] = __ballot_sync(0xFFFFFFFFu, v[i] != 0.0f);
        if (lane == 0)
            many[i * kGroups + group] = __popc(on[i]);
    }
    __syncthreads();
    int m = 0;
#pragma unroll
    for (int q = 0; q < kTurns * kGroups; ++q) {
        if (q % kGroups == group && v[q / kGroups] != 0.0f) {
            const int at = m + __popc(on[q / kGroups] & ((1u << lane) - 1u));
            from[at] = (int64_t)id[q / kGroups] * ldw;
            rest[at] = v[q / kGroups];
        }
        m += many[q];
    }
    __syncthreads();
    float2 a[4] = {};
    if (col < c)
        for (int e0 = group; e0 < m; e0 += 8 * kGroups) {
            uint4 b[8]; // in flight together
#pragma unroll
            for (int i = 0; i < 8; ++i)
                b[i] = e0 + i * kGroups < m ? __ldg(reinterpret_cast<const uint4 *>(w + from[e0 + i * kGroups] + col))
                                            : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = e0 + i * kGroups < m ? rest[e0 + i * kGroups] : 0.0f;
                const uint32_t u[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    a[q] = __ffma2_rn(make_float2(f, f), unpack2(u[q]), a[q]);
            }
        }
#pragma unroll
    for (int q = 0; q < 4; ++q)
        sums[group][q][lane] = a[q];
    __syncthreads();
    if (group > 0 || col >= c)
        return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            a[q].x += sums[i][q][lane].x;
            a[q].y += sums[i][q][lane].y;
        }
    const float f = g * scale;
    const float4 *s = reinterpret_cast<const float4 *>(slab + r * c + col);
    float4 lo = s[0], hi = s[1];
    for (int q = 1; q < slabs; ++q) {
        const float4 p = s[q * n * c / 4], t = s[q * n * c / 4 + 1];
        lo = make_float4(lo.x + p.x, lo.y + p.y, lo.z + p.z, lo.w + p.w);
        hi = make_float4(hi.x + t.x, hi.y + t.y, hi.z + t.z, hi.w + t.w);
    }
    alignas(16) const __nv_bfloat162 o[4] = {
        __floats2bfloat162_rn((lo.x + a[0].x) * f, (lo.y + a[0].y) * f),
        __floats2bfloat162_rn((lo.z + a[1].x) * f, (lo.w + a[1].y) * f),
        __floats2bfloat162_rn((hi.x + a[2].x) * f, (hi.y + a[2].y) * f),
        __floats2bfloat162_rn((hi.z + a[3].x) * f, (hi.w + a[3].y) * f)};
    *reinterpret_cast<uint4 *>(dx + r * lddx + col) = *reinterpret_cast<const uint4 *>(o);
}

// Rows that take several CTAs each for their products.  Forward in a graph, with and without: 64 rows x 32000 x 4096,
// 32 entries 58 and 80 us; 384 rows 111 and 126; 384 x 50257 x 1032, 20 entries 74 and 75, 512 rows of it 87 and 84.
constexpr int kFewRows = 384;
// Rows that take a CTA each in the join (above: eight a CTA): 2048 x 32000 x 4096, 32 entries 379 us (384), 2048 x
// 4097 x 128 37 (43); 8192 x 4097 x 128 107 (98), 8192 x 32000 x 256 240 (222).
constexpr int kJoinRows = 2048;

int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

} // namespace

cudaError_t launch_distill_rows(const LinearCeArgs &a, const DistillArgs &t, uint16_t *copy, int64_t ldc, int bn,
                                int parts, uint4 *skip, float2 *dots, cudaStream_t st)
{
    RowsParams p = {a.x, a.w, a.c, a.ldx, a.ldw, a.v, t.ids, t.ldi, t.k, bn, parts, copy, ldc, skip, dots};
    if (a.n > kFewRows)
        return launch_pdl(k_distill_rows<4>, dim3((unsigned)a.n, 2), dim3(32 * row_warps(4)), 0, st, p);
    const dim3 grid((unsigned)a.n, (unsigned)ceil_div(t.k, row_warps(1)) + 1);
    return launch_pdl(k_distill_rows<1>, grid, dim3(32 * row_warps(1)), 0, st, p);
}

cudaError_t launch_distill_join(const LinearCeArgs &a, const DistillArgs &t, const float2 *part, int parts,
                                const float2 *dots, cudaStream_t st)
{
    const int rows = a.n > kJoinRows ? 8 : 1;
    return launch_pdl(k_distill_join, dim3((unsigned)ceil_div(a.n, rows)), dim3(256), 0, st, rows, part, parts, dots,
                      t.ids, t.ldi, t.teacher, t.ldt, t.k, t.renorm, a.n, a.v, a.scale, a.scale * kLog2e, a.loss,
                      a.lse, t.logp);
}

cudaError_t launch_distill_start(const LinearCeArgs &a, const DistillArgs &t, uint16_t *copy, int64_t ldc,
                                 GradRow *rows, Listed *listed, float *gmax, cudaStream_t st)
{
    const int64_t blocks = ceil_div(a.n, 8), cap = (int64_t)sm_count() * 8;
    StartWords *start = reinterpret_cast<StartWords *>(gmax); // the workspace's first kilobyte is gmax's
    const cudaError_t e = cudaMemsetAsync(start, 0, sizeof(StartWords), st);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(k_distill_start, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, st, a.x, a.n,
                      a.c, a.ldx, copy, ldc, t.ids, t.ldi, t.teacher, t.ldt, t.k, t.renorm, a.v,
                      (const float *)a.lse, (const float *)t.logp, a.dloss, rows, listed, start);
}

cudaError_t launch_distill_patch(const LinearCeArgs &a, const DistillArgs &t, const Listed *listed, const float *gmax,
                                 uint16_t *d, int64_t ldd, int64_t col0, int64_t cols, cudaStream_t st)
{
    const int64_t total = a.n * t.k, blocks = ceil_div(total, 256), cap = (int64_t)sm_count() * 8;
    return launch_pdl(k_distill_patch, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, st, listed, total,
                      t.k, a.dloss, gmax, reinterpret_cast<__nv_bfloat16 *>(d), ldd, col0, cols);
}

cudaError_t launch_distill_dx(const LinearCeArgs &a, const DistillArgs &t, const Listed *listed, const float *slab,
                              int slabs, const float *gmax, cudaStream_t st)
{
    return launch_pdl(k_distill_dx, dim3((unsigned)a.n, (unsigned)ceil_div(a.c, 256)), dim3(kDxThreads), 0, st, slab,
                      slabs, a.n, a.c, gmax, a.scale, a.dloss, listed, t.k, a.w, a.ldw, a.dx, a.lddx);
}

} // namespace jetq
