// Layer norm and RMS norm, forward and backward, on rows of BF16 or FP32.
//
//   h = (x - mean) * rstd       (RMS norm: mean = 0)
//   y = h * w + b,   rstd = 1 / sqrt(sum (x - mean)^2 / c + eps)
//   t = dy * w
//   dx = rstd * (t - sum(t) / c - h * sum(t * h) / c)     (RMS norm: without sum(t))
//   dw = sum over rows of dy * h,   db = sum over rows of dy
//
// Every operation is FP32; the variance is summed around the mean (a second
// pass over registers), and each output is rounded once.
//
// Bound: HBM (two rows of traffic a row forward, three backward).  A group of
// G warps owns one row at a time, 16 elements a lane, so a row is read from
// memory once and stays in registers between the statistics and the output.
// The group's next rows are in flight meanwhile: one thread keeps a ring of
// bulk copies into shared memory ahead of the group (loads issued by the
// threads themselves leave too few bytes in flight between a row's two
// reductions).  A lane's columns are the same in every row, so the backward
// pass sums dw and db in registers and writes one partial row a group; a
// second kernel adds the partial rows in a fixed order (no atomics: results
// are bitwise repeatable).  Rows wider than 16 warps hold (8192) take the
// k_norm_*_wide kernels, which read a row more than once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "jetq_internal.h"
#include "ptx.cuh"

namespace jetq {

__device__ unsigned g_norm_error;

namespace {

constexpr unsigned kErrTimeout = 1u;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

struct NormParams {
    const void *x, *dy, *w, *b;
    void *out; // y or dx
    float *mean, *rstd;
    float *pdw, *pdb; // backward: partial rows [groups][cpad], pdb null without a bias
    int64_t n, ldx, lddy, ldo;
    int c, cpad;
    float eps;
    int stages;
    unsigned long long limit_ns;
};

template <class T>
struct Vec; // 16 bytes of T
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void unpack(const uint4 &v, float *f)
    {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    static __device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, float f) { *p = __float2bfloat16_rn(f); }
};
template <>
struct Vec<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void unpack(const uint4 &v, float *f)
    {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float f) { *p = f; }
};

template <class T, int G, int LE>
struct NormCfg {
    static constexpr int E = Vec<T>::E;
    static constexpr int V = LE / E;           // 16-byte vectors a lane
    static constexpr int kWarps = G < 8 ? 8 : G;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kGroups = kWarps / G; // rows in work a CTA
    static constexpr int kLanes = 32 * G;
};

// Sums of a and b over the group; `buf` alternates so that one barrier a call suffices.
template <int G>
__device__ __forceinline__ void group_sum2(float &a, float &b, float2 *red, int group, int wg, int lane, int &buf)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if constexpr (G > 1) {
        float2 *r = red + (buf * 16) + group * G;
        if (lane == 0)
            r[wg] = make_float2(a, b);
        ptx::named_bar_sync(1 + group, 32 * G);
        a = b = 0.0f;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const float2 q = r[i];
            a += q.x;
            b += q.y;
        }
        buf ^= 1;
    } else {
        __syncwarp();
    }
}

template <int G>
__device__ __forceinline__ float group_sum(float a, float2 *red, int group, int wg, int lane, int &buf)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    if constexpr (G > 1) {
        float *r = reinterpret_cast<float *>(red + buf * 16) + group * G;
        if (lane == 0)
            r[wg] = a;
        ptx::named_bar_sync(1 + group, 32 * G);
        a = 0.0f;
#pragma unroll
        for (int i = 0; i < G; ++i)
            a += r[i];
        buf ^= 1;
    } else {
        __syncwarp();
    }
    return a;
}

// The parameters (w, b) of a lane's columns, zero past c; `fallback` without one.
template <class T, int G, int LE>
__device__ __forceinline__ void load_params(const void *p, int c, int lt, float fallback, float (&f)[LE])
{
    using C = NormCfg<T, G, LE>;
#pragma unroll
    for (int k = 0; k < C::V; ++k)
#pragma unroll
        for (int e = 0; e < C::E; ++e) {
            const int col = (k * C::kLanes + lt) * C::E + e;
            f[k * C::E + e] = col < c ? (p ? Vec<T>::get(static_cast<const T *>(p) + col) : fallback) : 0.0f;
        }
}

// A row vector of a lane from the ring (whole vectors) or, where the last
// row's padding cannot be copied, from memory; elements past c are zero.
template <class T>
__device__ __forceinline__ void load_vec(const uint8_t *stage, const T *row, bool last_row, int pos, int c, float *f)
{
    constexpr int E = Vec<T>::E;
    if (pos + E <= c || (pos < c && !last_row)) {
        Vec<T>::unpack(*reinterpret_cast<const uint4 *>(stage + (size_t)pos * sizeof(T)), f);
        if (pos + E > c)
#pragma unroll
            for (int e = 0; e < E; ++e)
                f[e] = pos + e < c ? f[e] : 0.0f;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            f[e] = pos + e < c ? Vec<T>::get(row + pos + e) : 0.0f;
    }
}

template <class T>
__device__ __forceinline__ void store_vec(T *row, int pos, int c, const float *f)
{
    constexpr int E = Vec<T>::E;
    if (pos + E <= c) {
        *reinterpret_cast<uint4 *>(row + pos) = Vec<T>::pack(f);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (pos + e < c)
                Vec<T>::put(row + pos + e, f[e]);
    }
}

// The copies of one row into a ring stage: rows of both tensors, whole 16-byte
// vectors (the padding of a row lies inside the tensor except in its last row).
template <class T>
__device__ __forceinline__ void issue_row(uint32_t bar, uint32_t dst, uint32_t stride, const T *a, const T *b, int c,
                                          bool last_row)
{
    constexpr int E = Vec<T>::E;
    const uint32_t bytes = (uint32_t)(last_row ? c / E : (c + E - 1) / E) * 16u;
    ptx::mbar_arrive_expect_tx(bar, b ? 2u * bytes : bytes);
    if (bytes == 0)
        return;
    ptx::bulk_load(dst, a, bytes, bar);
    if (b)
        ptx::bulk_load(dst + stride, b, bytes, bar);
}

// CTAs an SM that the registers allow.
__host__ __device__ constexpr int norm_ctas(int g, int le, bool bwd)
{
    return g == 16 ? 1 : (bwd || le == 32 ? 2 : 3);
}

template <class T, int G, int LE, bool RMS, bool BWD>
__global__ void __launch_bounds__(NormCfg<T, G, LE>::kThreads, norm_ctas(G, LE, BWD))
    k_norm(const NormParams p)
{
    using C = NormCfg<T, G, LE>;
    constexpr int E = C::E, V = C::V;
    extern __shared__ uint8_t smem_raw[];
    __shared__ float2 red[2 * 16];
    __shared__ uint64_t bars[8 * 8];
    __shared__ int abort_word;
    uint8_t *ring = ptx::align_smem<128>(smem_raw);
    volatile int *abort_flag = &abort_word;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / G, wg = warp - group * G, lt = wg * 32 + lane;
    const uint32_t row_bytes = (uint32_t)(((p.c + E - 1) / E) * 16);
    const uint32_t stage_bytes = BWD ? 2u * row_bytes : row_bytes;
    uint8_t *mine = ring + (size_t)group * p.stages * stage_bytes;
    auto bar = [&](int s) { return ptx::smem_addr(&bars[group * 8 + s]); };

    if (threadIdx.x == 0) {
        abort_word = 0;
        for (int g = 0; g < C::kGroups; ++g)
            for (int s = 0; s < p.stages; ++s)
                ptx::mbar_init(ptx::smem_addr(&bars[g * 8 + s]), 1);
        ptx::fence_barrier_init();
    }
    __syncthreads();
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();

    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
    T *out = static_cast<T *>(p.out);
    const int64_t first = (int64_t)blockIdx.x * C::kGroups + group, step = (int64_t)gridDim.x * C::kGroups;
    auto issue = [&](int64_t row, int s) {
        issue_row<T>(bar(s), ptx::smem_addr(mine + (size_t)s * stage_bytes), row_bytes, x + row * p.ldx,
                     BWD ? dy + row * p.lddy : nullptr, p.c, row == p.n - 1);
    };
    int64_t last_issued = -1; // row, in the issuing thread
    if (lt == 0)
        for (int64_t row = first, i = 0; row < p.n && i < p.stages; row += step, ++i) {
            issue(row, (int)i);
            last_issued = row;
        }

    float w[LE], b[BWD ? 1 : LE];
    load_params<T, G, LE>(p.w, p.c, lt, 1.0f, w);
    if constexpr (!BWD)
        load_params<T, G, LE>(p.b, p.c, lt, 0.0f, b);
    float dw[BWD ? LE : 1], db[BWD && !RMS ? LE : 1];
    if constexpr (BWD) {
#pragma unroll
        for (int i = 0; i < LE; ++i) {
            dw[i] = 0.0f;
            if constexpr (!RMS)
                db[i] = 0.0f;
        }
    }
    bool ok = true;
    int s = 0, buf = 0;
    uint32_t ph = 0;
    auto refill = [&](int64_t row) {
        if (lt == 0 && ok && !*abort_flag && row < p.n) {
            issue(row, s);
            last_issued = row;
        }
    };
    const float inv_c = 1.0f / (float)p.c;
    float next_mean = 0.0f, next_rstd = 0.0f;
    if (BWD && first < p.n) {
        next_mean = RMS ? 0.0f : __ldg(p.mean + first);
        next_rstd = __ldg(p.rstd + first);
    }
    for (int64_t row = first; row < p.n; row += step) {
        // After a timeout every thread still runs through the rows and meets their barriers, without new
        // copies; the issuing thread waits (within its limit) for each copy that it has started.
        if (lt == 0)
            ok = row <= last_issued &&
                 ptx::mbar_wait(bar(s), ph, abort_flag, &g_norm_error, kErrTimeout, p.limit_ns, false);
        else
            ok = ptx::mbar_wait(bar(s), ph, abort_flag, &g_norm_error, kErrTimeout, p.limit_ns);
        const bool last_row = row == p.n - 1;
        const uint8_t *st = mine + (size_t)s * stage_bytes;
        float h[LE];
#pragma unroll
        for (int k = 0; k < V; ++k)
            load_vec<T>(st, x + row * p.ldx, last_row, (k * C::kLanes + lt) * E, p.c, h + k * E);
        if constexpr (!BWD) {
            // pairs: the packed FP32 instructions do two elements an issue slot
            float mean = 0.0f;
            if constexpr (!RMS) {
                float2 a = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < LE; i += 2)
                    a = __fadd2_rn(a, make_float2(h[i], h[i + 1]));
                mean = group_sum<G>(a.x + a.y, red, group, wg, lane, buf) * inv_c;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int pos = (k * C::kLanes + lt) * E;
                    if (pos + E <= p.c) {
#pragma unroll
                        for (int i = k * E; i < (k + 1) * E; i += 2) {
                            const float2 d = __fadd2_rn(make_float2(h[i], h[i + 1]), make_float2(-mean, -mean));
                            h[i] = d.x;
                            h[i + 1] = d.y;
                        }
                    } else { // columns past c do not count
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            h[k * E + e] = pos + e < p.c ? h[k * E + e] - mean : 0.0f;
                    }
                }
            }
            float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < LE; i += 2)
                q = __ffma2_rn(make_float2(h[i], h[i + 1]), make_float2(h[i], h[i + 1]), q);
            float sq = q.x + q.y;
            sq = group_sum<G>(sq, red, group, wg, lane, buf);
            // every lane has its row in registers: the stage takes the next row
            refill(row + (int64_t)p.stages * step);
            const float rstd = __frcp_rn(__fsqrt_rn(fmaf(sq, inv_c, p.eps)));
            if (lt == 0) {
                if (!RMS)
                    p.mean[row] = mean;
                p.rstd[row] = rstd;
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float y[E];
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const int i = k * E + e;
                    const float2 v = __ffma2_rn(
                        __fmul2_rn(make_float2(h[i], h[i + 1]), make_float2(rstd, rstd)),
                        make_float2(w[i], w[i + 1]), make_float2(b[i], b[i + 1]));
                    y[e] = v.x;
                    y[e + 1] = v.y;
                }
                const int pos = (k * C::kLanes + lt) * E;
                if (pos < p.c)
                    store_vec<T>(out + row * p.ldo, pos, p.c, y);
            }
        } else {
            const float mean = next_mean, rstd = next_rstd;
            if (row + step < p.n) {
                next_mean = RMS ? 0.0f : __ldg(p.mean + row + step);
                next_rstd = __ldg(p.rstd + row + step);
            }
            float t[LE];
#pragma unroll
            for (int k = 0; k < V; ++k)
                load_vec<T>(st + row_bytes, dy + row * p.lddy, last_row, (k * C::kLanes + lt) * E, p.c, t + k * E);
            float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int k = 0; k < V; ++k) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i = k * E + e;
                    h[i] = (h[i] - mean) * rstd;
                    dw[i] = fmaf(t[i], h[i], dw[i]); // columns past c: t = 0
                    if constexpr (!RMS)
                        db[i] += t[i];
                    t[i] *= w[i];
                    if constexpr (!RMS)
                        s1 += t[i];
                    s2 = fmaf(t[i], h[i], s2);
                }
            }
            if constexpr (RMS)
                s2 = group_sum<G>(s2, red, group, wg, lane, buf);
            else
                group_sum2<G>(s1, s2, red, group, wg, lane, buf);
            refill(row + (int64_t)p.stages * step);
            s1 = RMS ? 0.0f : s1 * inv_c;
            s2 *= inv_c;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float d[E];
#pragma unroll
                for (int e = 0; e < E; ++e)
                    d[e] = rstd * (t[k * E + e] - s1 - h[k * E + e] * s2);
                const int pos = (k * C::kLanes + lt) * E;
                if (pos < p.c)
                    store_vec<T>(out + row * p.ldo, pos, p.c, d);
            }
        }
        if (++s == p.stages) {
            s = 0;
            ph ^= 1u;
        }
    }
    if constexpr (BWD) {
        if (first < p.n) {
#pragma unroll
            for (int k = 0; k < V; ++k)
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const int col = (k * C::kLanes + lt) * E + e;
                    if (col < p.cpad) { // cpad is a multiple of 8
                        const int i = k * E + e;
                        *reinterpret_cast<float4 *>(p.pdw + first * p.cpad + col) =
                            make_float4(dw[i], dw[i + 1], dw[i + 2], dw[i + 3]);
                        if constexpr (!RMS)
                            if (p.pdb)
                                *reinterpret_cast<float4 *>(p.pdb + first * p.cpad + col) =
                                    make_float4(db[i], db[i + 1], db[i + 2], db[i + 3]);
                    }
                }
        }
    }
}

// dw, db: sums of the partial rows in a fixed order; 32 columns a block, 32 lanes along the rows.
__global__ void __launch_bounds__(1024) k_norm_params(const float *pdw, const float *pdb, int rows, int c, int cpad,
                                                      float *dw, float *db)
{
    __shared__ float red[32][33];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, col = blockIdx.x * 32 + tx;
    const float *src = blockIdx.y == 0 ? pdw : pdb;
    float a = 0.0f;
    if (col < c)
        for (int r = ty; r < rows; r += 32)
            a += src[(int64_t)r * cpad + col];
    red[ty][tx] = a;
    __syncthreads();
    a = red[tx][ty];
#pragma unroll
    for (int o = 16; o; o >>= 1)
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    const int oc = blockIdx.x * 32 + ty;
    if (tx == 0 && oc < c)
        (blockIdx.y == 0 ? dw : db)[oc] = a;
}

// ------------------------------------------------------------- wide rows

__device__ __forceinline__ float2 block_sum2(float a, float b, float2 *red)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    a = b = 0.0f;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) {
        a += red[i].x;
        b += red[i].y;
    }
    return make_float2(a, b);
}

// One CTA a row, the row read again for each step (from L2 after the first).
template <class T, bool RMS, bool BWD>
__global__ void __launch_bounds__(1024) k_norm_wide(const NormParams p)
{
    __shared__ float2 red[32];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const float inv_c = 1.0f / (float)p.c;
    for (int64_t row = blockIdx.x; row < p.n; row += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + row * p.ldx;
        const T *w = static_cast<const T *>(p.w);
        T *out = static_cast<T *>(p.out) + row * p.ldo;
        if constexpr (!BWD) {
            const T *b = static_cast<const T *>(p.b);
            float mean = 0.0f, sq = 0.0f;
            if constexpr (!RMS) {
                for (int i = threadIdx.x; i < p.c; i += blockDim.x)
                    mean += Vec<T>::get(x + i);
                mean = block_sum2(mean, 0.0f, red).x * inv_c;
            }
            for (int i = threadIdx.x; i < p.c; i += blockDim.x) {
                const float v = Vec<T>::get(x + i) - mean;
                sq = fmaf(v, v, sq);
            }
            sq = block_sum2(sq, 0.0f, red).x;
            const float rstd = __frcp_rn(__fsqrt_rn(fmaf(sq, inv_c, p.eps)));
            if (threadIdx.x == 0) {
                if (!RMS)
                    p.mean[row] = mean;
                p.rstd[row] = rstd;
            }
            for (int i = threadIdx.x; i < p.c; i += blockDim.x) {
                const float v = (Vec<T>::get(x + i) - mean) * rstd;
                Vec<T>::put(out + i, fmaf(v, w ? Vec<T>::get(w + i) : 1.0f, b ? Vec<T>::get(b + i) : 0.0f));
            }
        } else {
            const T *dy = static_cast<const T *>(p.dy) + row * p.lddy;
            const float mean = RMS ? 0.0f : p.mean[row], rstd = p.rstd[row];
            float s1 = 0.0f, s2 = 0.0f;
            for (int i = threadIdx.x; i < p.c; i += blockDim.x) {
                const float h = (Vec<T>::get(x + i) - mean) * rstd;
                const float t = Vec<T>::get(dy + i) * (w ? Vec<T>::get(w + i) : 1.0f);
                s1 += t;
                s2 = fmaf(t, h, s2);
            }
            const float2 sum = block_sum2(s1, s2, red);
            const float m1 = RMS ? 0.0f : sum.x * inv_c, m2 = sum.y * inv_c;
            for (int i = threadIdx.x; i < p.c; i += blockDim.x) {
                const float h = (Vec<T>::get(x + i) - mean) * rstd;
                const float t = Vec<T>::get(dy + i) * (w ? Vec<T>::get(w + i) : 1.0f);
                Vec<T>::put(out + i, rstd * (t - m1 - h * m2));
            }
        }
    }
}

// Partial rows of dw and db for wide rows: a thread a column, blockIdx.y a slice of the rows.
template <class T, bool RMS>
__global__ void __launch_bounds__(256) k_norm_wide_params(const NormParams p)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col >= p.c)
        return;
    const int64_t r0 = p.n * blockIdx.y / gridDim.y, r1 = p.n * (blockIdx.y + 1) / gridDim.y;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const float g = Vec<T>::get(static_cast<const T *>(p.dy) + r * p.lddy + col);
        const float v = Vec<T>::get(static_cast<const T *>(p.x) + r * p.ldx + col);
        dw = fmaf(g, (v - (RMS ? 0.0f : p.mean[r])) * p.rstd[r], dw);
        db += g;
    }
    p.pdw[(int64_t)blockIdx.y * p.cpad + col] = dw;
    if (p.pdb)
        p.pdb[(int64_t)blockIdx.y * p.cpad + col] = db;
}

constexpr int kWidest = 8192, kWideSlices = 64, kMaxStages = 4;

// Elements a lane holds.  Forward: 32 (half the reductions and waits of 16 for
// every element; 16384 x 4096 measured in the launcher's comment), 16 where a
// single warp of them holds the row.  Backward: 16 (x, dy and the sums of dw
// and db take four registers an element).
int lane_elems(int64_t c, bool bwd)
{
    return bwd || c <= 512 ? 16 : 32;
}

int warps_of(int64_t c, int le)
{
    int g = 1;
    while (g * 32 * le < c)
        g *= 2;
    return g;
}

struct NormPlan {
    int grid, groups, stages; // groups: partial rows of dw and db
    size_t smem;
};

// Grid and ring of the register kernels.  CTAs an SM: what the registers allow
// (the launch bounds) and the rings' shared memory; a group gets four rows or
// more in the backward pass, so that its partial rows stay a small part of the traffic.
NormPlan norm_plan(int64_t n, int64_t c, int esize, bool bwd)
{
    NormPlan r;
    const int le = lane_elems(c, bwd), g = warps_of(c, le), per_cta = g < 8 ? 8 / g : 1;
    const size_t row = (size_t)((c * esize + 15) / 16 * 16) * (bwd ? 2 : 1);
    r.stages = kMaxStages;
    const int ctas = norm_ctas(g, le, bwd);
    while (r.stages > 2 && ctas * (r.stages * per_cta * row + 2048) > 227 * 1024)
        --r.stages;
    r.smem = r.stages * per_cta * row + 128;
    const int64_t rows_a_group = bwd ? 4 : 1;
    int64_t groups = (n + rows_a_group - 1) / rows_a_group;
    const int64_t most = (int64_t)sm_count() * ctas * per_cta;
    groups = groups < most ? groups : most;
    r.grid = (int)((groups + per_cta - 1) / per_cta);
    // every group that exists and has a row writes its partial row
    const int64_t all = (int64_t)r.grid * per_cta;
    r.groups = (int)(all < n ? all : n);
    return r;
}

template <class T, int G, int LE, bool RMS, bool BWD>
cudaError_t run_norm(const NormParams &p, const NormPlan &plan, cudaStream_t st)
{
    auto kern = k_norm<T, G, LE, RMS, BWD>;
    static int configured_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (configured_device != dev) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024)) != cudaSuccess)
            return e;
        configured_device = dev;
    }
    return launch_pdl(kern, dim3((unsigned)plan.grid), dim3(NormCfg<T, G, LE>::kThreads), plan.smem, st, p);
}

template <class T, bool RMS, bool BWD>
cudaError_t pick_norm(const NormParams &p, const NormPlan &plan, cudaStream_t st)
{
    constexpr int kFull = BWD ? 16 : 32;
    const int le = lane_elems(p.c, BWD);
    if (le != kFull)
        return run_norm<T, 1, 16, RMS, BWD>(p, plan, st);
    switch (warps_of(p.c, le)) {
    case 1: return run_norm<T, 1, kFull, RMS, BWD>(p, plan, st);
    case 2: return run_norm<T, 2, kFull, RMS, BWD>(p, plan, st);
    case 4: return run_norm<T, 4, kFull, RMS, BWD>(p, plan, st);
    case 8: return run_norm<T, 8, kFull, RMS, BWD>(p, plan, st);
    default: break;
    }
    if constexpr (BWD)
        return run_norm<T, 16, 16, RMS, true>(p, plan, st);
    else
        return cudaErrorInvalidValue; // 8 warps of 32 hold every row up to kWidest
}

template <class T, bool RMS>
cudaError_t norm_any(const NormArgs &a, NormParams p, bool bwd, cudaStream_t st)
{
    const bool wide = a.c > kWidest;
    NormPlan plan = {};
    if (!wide)
        plan = norm_plan(a.n, a.c, (int)sizeof(T), bwd);
    if (!bwd) {
        if (!wide)
            return pick_norm<T, RMS, false>(p, plan, st);
        const int64_t cap = (int64_t)sm_count() * 2;
        return launch_pdl(k_norm_wide<T, RMS, false>, dim3((unsigned)(a.n < cap ? a.n : cap)), dim3(1024), 0, st, p);
    }
    cudaError_t e;
    if (!wide) {
        e = pick_norm<T, RMS, true>(p, plan, st);
    } else {
        const int64_t cap = (int64_t)sm_count() * 2;
        plan.groups = (int)(a.n < kWideSlices ? a.n : kWideSlices);
        e = launch_pdl(k_norm_wide<T, RMS, true>, dim3((unsigned)(a.n < cap ? a.n : cap)), dim3(1024), 0, st, p);
        if (e == cudaSuccess)
            e = launch_pdl(k_norm_wide_params<T, RMS>, dim3((unsigned)((a.c + 255) / 256), (unsigned)plan.groups),
                           dim3(256), 0, st, p);
    }
    if (e != cudaSuccess)
        return e;
    return launch_pdl(k_norm_params, dim3((unsigned)((a.c + 31) / 32), a.db ? 2u : 1u), dim3(1024), 0, st,
                      (const float *)p.pdw, (const float *)p.pdb, plan.groups, p.c, p.cpad, a.dw, a.db);
}

cudaError_t launch_norm(const NormArgs &a, bool bwd, cudaStream_t st)
{
    NormParams p = {};
    p.x = a.x;
    p.dy = a.dy;
    p.w = a.w;
    p.b = a.b;
    p.out = a.out;
    p.mean = a.mean;
    p.rstd = a.rstd;
    p.n = a.n;
    p.c = (int)a.c;
    p.cpad = (int)((a.c + 7) / 8 * 8);
    p.ldx = a.ldx;
    p.lddy = a.lddy;
    p.ldo = a.ldo;
    p.eps = a.eps;
    p.limit_ns = kWaitLimitNs;
    if (bwd) {
        const int64_t rows = norm_bwd_partial_rows(a.n, a.c, a.dtype);
        p.pdw = static_cast<float *>(a.ws);
        p.pdb = a.db ? p.pdw + rows * p.cpad : nullptr;
    }
    if (a.c <= kWidest)
        p.stages = norm_plan(a.n, a.c, a.dtype == JETQ_OUT_BF16 ? 2 : 4, bwd).stages;
    const bool rms = a.kind == JETQ_NORM_RMS;
    if (a.dtype == JETQ_OUT_BF16)
        return rms ? norm_any<__nv_bfloat16, true>(a, p, bwd, st) : norm_any<__nv_bfloat16, false>(a, p, bwd, st);
    return rms ? norm_any<float, true>(a, p, bwd, st) : norm_any<float, false>(a, p, bwd, st);
}

} // namespace

int64_t norm_bwd_partial_rows(int64_t n, int64_t c, jetq_out_dtype dtype)
{
    if (c > kWidest)
        return n < kWideSlices ? n : kWideSlices;
    return norm_plan(n, c, dtype == JETQ_OUT_BF16 ? 2 : 4, true).groups;
}

cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t st)
{
    return launch_norm(a, false, st);
}

cudaError_t launch_norm_bwd(const NormArgs &a, cudaStream_t st)
{
    return launch_norm(a, true, st);
}

cudaError_t norm_read_and_clear_error(cudaStream_t st, unsigned *out)
{
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_norm_error, sizeof v, 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(st);
    if (e != cudaSuccess)
        return e;
    *out |= v;
    if (v) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbolAsync(g_norm_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, st);
        if (e == cudaSuccess)
            e = cudaStreamSynchronize(st);
    }
    return e;
}

} // namespace jetq
