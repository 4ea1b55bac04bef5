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
// warps owns one row at a time; its next rows are in flight meanwhile: one
// thread keeps a ring of bulk copies into shared memory ahead of the group
// (loads issued by the threads themselves leave too few bytes in flight
// between a row's two reductions).
//
// Forward: a warp a row (up to 8 KB; 2 or 4 warps above, 8 where there are
// fewer rows than SMs), which runs over the row in shared memory for the mean,
// the spread and the output, two elements an instruction.  16384 x 4096 BF16:
// 45.5 us, 5.9 TB/s, 0.87 of the measured copy rate.  A first version with a
// row in the registers of 8 warps (62 us; 4 warps of 32 elements a lane: 60)
// spent half its instructions on the reductions, waits and addresses of each
// warp's 512 or 1024 elements.
//
// Backward: 2 to 16 warps a row, 16 elements a lane in registers.  A lane's
// columns are the same in every row, so dw and db are summed in registers; each
// group writes one partial row and a second kernel adds the partial rows in a
// fixed order (no atomics: results are bitwise repeatable).  32768 x 2048 BF16
// with that kernel: RMS 68 us, 5.9 TB/s, 0.87 of the copy rate; layer norm with
// its bias 72 to 77 us, 5.2 to 5.6 TB/s (96 us before rows that fill their lanes skipped the
// checks of the row's end).  Rows fill their lanes at 512 * 2^k columns only; at
// others lanes are idle and the checks stay: 16384 x 2560, 5120 and 7168 BF16
// take 86, 160 and 150 us (RMS; 0.43, 0.46 and 0.69 of the copy rate) and 101, 191
// and 177 us (layer norm with its bias) in a graph.
//
// Rows of up to 512 columns take k_norm_short.  Rows wider than 8192 take the
// k_norm_*wide* kernels, which read a row from memory more than once, an element
// at a time: 8192 x 16384 BF16 365 us forward and 566 backward (RMS), 454 and
// 618 (layer norm), about a fifth of the copy rate.
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

constexpr int LE = 16; // elements a lane (backward)

template <class T, int G>
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
template <class T, int G>
__device__ __forceinline__ void load_params(const void *p, int c, int lt, float fallback, float (&f)[LE])
{
    using C = NormCfg<T, G>;
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
__host__ __device__ constexpr int norm_bwd_ctas(int g)
{
    return g == 16 ? 1 : 2;
}

template <class T, int G, bool RMS>
__global__ void __launch_bounds__(NormCfg<T, G>::kThreads, norm_bwd_ctas(G)) k_norm_bwd(const NormParams p)
{
    using C = NormCfg<T, G>;
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
    const uint32_t stage_bytes = 2u * row_bytes;
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
                     dy + row * p.lddy, p.c, row == p.n - 1);
    };
    int64_t last_issued = -1; // row, in the issuing thread
    if (lt == 0)
        for (int64_t row = first, i = 0; row < p.n && i < p.stages; row += step, ++i) {
            issue(row, (int)i);
            last_issued = row;
        }

    float w[LE], dw[LE], db[RMS ? 1 : LE];
    load_params<T, G>(p.w, p.c, lt, 1.0f, w);
#pragma unroll
    for (int i = 0; i < LE; ++i) {
        dw[i] = 0.0f;
        if constexpr (!RMS)
            db[i] = 0.0f;
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
    const bool full = p.c == C::kLanes * LE; // every lane's vectors are whole
    float next_mean = 0.0f, next_rstd = 0.0f;
    if (first < p.n) {
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
        float h[LE], t[LE];
        if (full) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const uint8_t *at = st + (size_t)(k * C::kLanes + lt) * 16;
                Vec<T>::unpack(*reinterpret_cast<const uint4 *>(at), h + k * E);
                Vec<T>::unpack(*reinterpret_cast<const uint4 *>(at + row_bytes), t + k * E);
            }
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int pos = (k * C::kLanes + lt) * E;
                load_vec<T>(st, x + row * p.ldx, last_row, pos, p.c, h + k * E);
                load_vec<T>(st + row_bytes, dy + row * p.lddy, last_row, pos, p.c, t + k * E);
            }
        }
        const float mean = next_mean, rstd = next_rstd;
        if (row + step < p.n) {
            next_mean = RMS ? 0.0f : __ldg(p.mean + row + step);
            next_rstd = __ldg(p.rstd + row + step);
        }
        // pairs: the packed FP32 instructions do two elements an issue slot
        const float2 neg = make_float2(-mean, -mean), r2 = make_float2(rstd, rstd);
        float2 a1 = make_float2(0.0f, 0.0f), a2 = a1;
#pragma unroll
        for (int i = 0; i < LE; i += 2) {
            float2 hv = make_float2(h[i], h[i + 1]), tv = make_float2(t[i], t[i + 1]);
            hv = RMS ? __fmul2_rn(hv, r2) : __fmul2_rn(__fadd2_rn(hv, neg), r2);
            const float2 g = __ffma2_rn(tv, hv, make_float2(dw[i], dw[i + 1])); // columns past c: t = 0
            dw[i] = g.x;
            dw[i + 1] = g.y;
            if constexpr (!RMS) {
                const float2 b = __fadd2_rn(make_float2(db[i], db[i + 1]), tv);
                db[i] = b.x;
                db[i + 1] = b.y;
            }
            tv = __fmul2_rn(tv, make_float2(w[i], w[i + 1]));
            if constexpr (!RMS)
                a1 = __fadd2_rn(a1, tv);
            a2 = __ffma2_rn(tv, hv, a2);
            h[i] = hv.x;
            h[i + 1] = hv.y;
            t[i] = tv.x;
            t[i + 1] = tv.y;
        }
        float s1 = a1.x + a1.y, s2 = a2.x + a2.y;
        if constexpr (RMS)
            s2 = group_sum<G>(s2, red, group, wg, lane, buf);
        else
            group_sum2<G>(s1, s2, red, group, wg, lane, buf);
        refill(row + (int64_t)p.stages * step);
        s1 = RMS ? 0.0f : s1 * inv_c;
        s2 *= inv_c;
        T *o = out + row * p.ldo;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float d[E];
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const int i = k * E + e;
                float2 v = make_float2(t[i], t[i + 1]);
                if constexpr (!RMS)
                    v = __fadd2_rn(v, make_float2(-s1, -s1));
                v = __fmul2_rn(__ffma2_rn(make_float2(h[i], h[i + 1]), make_float2(-s2, -s2), v), r2);
                d[e] = v.x;
                d[e + 1] = v.y;
            }
            const int pos = (k * C::kLanes + lt) * E;
            if (full)
                *reinterpret_cast<uint4 *>(o + pos) = Vec<T>::pack(d);
            else if (pos < p.c)
                store_vec<T>(o, pos, p.c, d);
        }
        if (++s == p.stages) {
            s = 0;
            ph ^= 1u;
        }
    }
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

// Forward.  blockDim = 32 * G * groups; dynamic shared memory: the parameters
// (w, b as they are stored, padded to whole vectors), then a ring a group.
template <class T, int G, bool RMS>
__global__ void __launch_bounds__(512, 2) k_norm_fwd(const NormParams p)
{
    constexpr int E = Vec<T>::E, L = 32 * G;
    extern __shared__ uint8_t smem_raw[];
    __shared__ float2 red[2 * 16];
    __shared__ uint64_t bars[16 * 4];
    __shared__ int abort_word;
    uint8_t *params = ptx::align_smem<128>(smem_raw);
    volatile int *abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, groups = blockDim.x / L;
    const int group = warp / G, wg = warp - group * G, lt = wg * 32 + lane;
    const uint32_t row_bytes = (uint32_t)(((p.c + E - 1) / E) * 16);
    uint8_t *mine = params + (p.b ? 2u : 1u) * row_bytes + (size_t)group * p.stages * row_bytes;
    auto bar = [&](int s) { return ptx::smem_addr(&bars[group * 4 + s]); };

    if (threadIdx.x == 0) {
        abort_word = 0;
        for (int g = 0; g < groups; ++g)
            for (int s = 0; s < p.stages; ++s)
                ptx::mbar_init(ptx::smem_addr(&bars[g * 4 + s]), 1);
        ptx::fence_barrier_init();
    }
    __syncthreads();
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();

    const T *x = static_cast<const T *>(p.x);
    T *out = static_cast<T *>(p.out);
    const int64_t first = (int64_t)blockIdx.x * groups + group, step = (int64_t)gridDim.x * groups;
    auto issue = [&](int64_t row, int s) {
        issue_row<T>(bar(s), ptx::smem_addr(mine + (size_t)s * row_bytes), 0, x + row * p.ldx, (const T *)nullptr, p.c,
                     row == p.n - 1);
    };
    int64_t last_issued = -1; // row, in the issuing thread
    if (lt == 0)
        for (int64_t row = first, i = 0; row < p.n && i < p.stages; row += step, ++i) {
            issue(row, (int)i);
            last_issued = row;
        }
    T *ws = reinterpret_cast<T *>(params), *bs = reinterpret_cast<T *>(params + row_bytes);
    const int whole = p.c / E * E; // columns in whole vectors
    auto copy_param = [&](T *dst, const T *src, float fallback) {
        // whole vectors where the pointer allows them (any element-aligned one is taken)
        const int vec = src && (reinterpret_cast<uintptr_t>(src) & 15u) == 0 ? whole : 0;
        for (int i = threadIdx.x * E; i < vec; i += blockDim.x * E)
            *reinterpret_cast<uint4 *>(dst + i) = __ldg(reinterpret_cast<const uint4 *>(src + i));
        for (int i = vec + threadIdx.x; i < (int)(row_bytes / sizeof(T)); i += blockDim.x)
            Vec<T>::put(dst + i, i < p.c ? (src ? Vec<T>::get(src + i) : fallback) : 0.0f);
    };
    copy_param(ws, static_cast<const T *>(p.w), 1.0f);
    if (p.b)
        copy_param(bs, static_cast<const T *>(p.b), 0.0f);
    __syncthreads();

    const float inv_c = 1.0f / (float)p.c;
    const int tail = whole + lt; // one of the columns past the whole vectors, in the first lanes
    bool ok = true;
    int s = 0, buf = 0;
    uint32_t ph = 0;
    for (int64_t row = first; row < p.n; row += step) {
        // After a timeout every thread still runs through the rows and meets their barriers, without new
        // copies; the issuing thread waits (within its limit) for each copy that it has started.
        if (lt == 0)
            ok = row <= last_issued &&
                 ptx::mbar_wait(bar(s), ph, abort_flag, &g_norm_error, kErrTimeout, p.limit_ns, false);
        else
            ok = ptx::mbar_wait(bar(s), ph, abort_flag, &g_norm_error, kErrTimeout, p.limit_ns);
        const T *st = reinterpret_cast<const T *>(mine + (size_t)s * row_bytes);
        float xt = 0.0f; // the last row's padding was not copied: its tail comes from memory
        if (tail < p.c)
            xt = Vec<T>::get(row == p.n - 1 ? x + row * p.ldx + tail : st + tail);
        float mean = 0.0f;
        if constexpr (!RMS) {
            float2 a = make_float2(xt, 0.0f);
#pragma unroll 4
            for (int pos = lt * E; pos < whole; pos += L * E) {
                float f[E];
                Vec<T>::unpack(*reinterpret_cast<const uint4 *>(st + pos), f);
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    a = __fadd2_rn(a, make_float2(f[e], f[e + 1]));
            }
            mean = group_sum<G>(a.x + a.y, red, group, wg, lane, buf) * inv_c;
        }
        const float2 neg = make_float2(-mean, -mean);
        float2 q = make_float2(tail < p.c ? (xt - mean) * (xt - mean) : 0.0f, 0.0f);
#pragma unroll 4
        for (int pos = lt * E; pos < whole; pos += L * E) {
            float f[E];
            Vec<T>::unpack(*reinterpret_cast<const uint4 *>(st + pos), f);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = __fadd2_rn(make_float2(f[e], f[e + 1]), neg);
                q = __ffma2_rn(v, v, q);
            }
        }
        const float sq = group_sum<G>(q.x + q.y, red, group, wg, lane, buf);
        const float rstd = __frcp_rn(__fsqrt_rn(fmaf(sq, inv_c, p.eps)));
        if (lt == 0) {
            if (!RMS)
                p.mean[row] = mean;
            p.rstd[row] = rstd;
        }
        T *o = out + row * p.ldo;
        const float2 r2 = make_float2(rstd, rstd);
#pragma unroll 2
        for (int pos = lt * E; pos < whole; pos += L * E) {
            float f[E], w[E], b[E];
            Vec<T>::unpack(*reinterpret_cast<const uint4 *>(st + pos), f);
            Vec<T>::unpack(*reinterpret_cast<const uint4 *>(ws + pos), w);
            if (!RMS && p.b)
                Vec<T>::unpack(*reinterpret_cast<const uint4 *>(bs + pos), b);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 h = __fmul2_rn(__fadd2_rn(make_float2(f[e], f[e + 1]), neg), r2);
                const float2 wv = make_float2(w[e], w[e + 1]);
                const float2 y = !RMS && p.b ? __ffma2_rn(h, wv, make_float2(b[e], b[e + 1])) : __fmul2_rn(h, wv);
                f[e] = y.x;
                f[e + 1] = y.y;
            }
            *reinterpret_cast<uint4 *>(o + pos) = Vec<T>::pack(f);
        }
        if (tail < p.c)
            Vec<T>::put(o + tail, fmaf((xt - mean) * rstd, Vec<T>::get(ws + tail),
                                       !RMS && p.b ? Vec<T>::get(bs + tail) : 0.0f));
        // every lane is through with the stage: it takes the next row
        if constexpr (G > 1)
            ptx::named_bar_sync(1 + group, L);
        else
            __syncwarp();
        const int64_t ahead = row + (int64_t)p.stages * step;
        if (lt == 0 && ok && !*abort_flag && ahead < p.n) {
            issue(ahead, s);
            last_issued = ahead;
        }
        if (++s == p.stages) {
            s = 0;
            ph ^= 1u;
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

// ------------------------------------------------------------- short rows

// Rows of up to 512 columns (a head's, for one): L lanes a row, 32 / L rows a
// warp, V vectors a lane, loaded straight from memory for U rows a lane at a
// time.  There are warps enough here to keep the loads in flight, and a ring's
// waits and a warp's reductions would cost a row more than its arithmetic
// (30000 x 128 BF16 through the kernels above: forward 13.5 us, backward 33).
__host__ __device__ constexpr int short_ctas(int elems, bool bwd) // CTAs an SM
{
    return bwd ? 2 : (elems > 8 ? 3 : 4);
}

template <class T, int L, int V, bool RMS, bool BWD>
__global__ void __launch_bounds__(256, short_ctas(Vec<T>::E *V, BWD)) k_norm_short(const NormParams p)
{
    constexpr int E = Vec<T>::E, N = E * V, R = 32 / L, U = N > 8 ? 2 : 4;
    __shared__ float red[BWD ? 8 * L * N : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % L, sub = lane / L;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
    T *out = static_cast<T *>(p.out);
    auto column = [&](int i) { return ((i / E) * L + l) * E + i % E; };
    float w[N], b[BWD ? 1 : N], dw[BWD ? N : 1], db[BWD && !RMS ? N : 1];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int col = column(i);
        w[i] = col < p.c ? (p.w ? Vec<T>::get(static_cast<const T *>(p.w) + col) : 1.0f) : 0.0f;
        if constexpr (!BWD)
            b[i] = !RMS && p.b && col < p.c ? Vec<T>::get(static_cast<const T *>(p.b) + col) : 0.0f;
        if constexpr (BWD)
            dw[i] = 0.0f;
        if constexpr (BWD && !RMS)
            db[i] = 0.0f;
    }
    // a row's vectors as they are stored: rows that wait for their turn take half the registers
    auto load = [&](const T *row, uint4 *raw) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int pos = (v * L + l) * E;
            if (pos + E <= p.c) {
                raw[v] = *reinterpret_cast<const uint4 *>(row + pos);
            } else {
                float f[E];
#pragma unroll
                for (int e = 0; e < E; ++e)
                    f[e] = pos + e < p.c ? Vec<T>::get(row + pos + e) : 0.0f;
                raw[v] = Vec<T>::pack(f);
            }
        }
    };
    auto sum = [&](float a) {
#pragma unroll
        for (int o = L / 2; o; o >>= 1)
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        return a;
    };
    const float inv_c = 1.0f / (float)p.c;
    const int64_t step = (int64_t)gridDim.x * 8 * R * U;
    // rows first .. first + R U of a warp, all of its lanes in every pass (the sums are shuffles)
    for (int64_t first = ((int64_t)blockIdx.x * 8 + warp) * R * U; first < p.n; first += step) {
        uint4 rx[U][V], ry[BWD ? U : 1][V];
        float mean[U], rstd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = first + u * R + sub;
            mean[u] = rstd[u] = 0.0f;
            if (row < p.n) {
                load(x + row * p.ldx, rx[u]);
                if constexpr (BWD) {
                    load(dy + row * p.lddy, ry[u]);
                    mean[u] = RMS ? 0.0f : __ldg(p.mean + row);
                    rstd[u] = __ldg(p.rstd + row);
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    rx[u][v] = make_uint4(0, 0, 0, 0);
                    if constexpr (BWD)
                        ry[u][v] = make_uint4(0, 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = first + u * R + sub;
            float f[N];
#pragma unroll
            for (int v = 0; v < V; ++v)
                Vec<T>::unpack(rx[u][v], f + v * E);
            if constexpr (!BWD) {
                float m = 0.0f;
                if constexpr (!RMS) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        m += f[i];
                    m = sum(m) * inv_c;
                }
                float sq = 0.0f;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if constexpr (!RMS)
                        f[i] = column(i) < p.c ? f[i] - m : 0.0f;
                    sq = fmaf(f[i], f[i], sq);
                }
                const float r = __frcp_rn(__fsqrt_rn(fmaf(sum(sq), inv_c, p.eps)));
                if (l == 0 && row < p.n) {
                    if (!RMS)
                        p.mean[row] = m;
                    p.rstd[row] = r;
                }
#pragma unroll
                for (int i = 0; i < N; ++i)
                    f[i] = fmaf(f[i] * r, w[i], b[i]);
            } else {
                float g[N], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    Vec<T>::unpack(ry[u][v], g + v * E);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    f[i] = (f[i] - mean[u]) * rstd[u];
                    dw[i] = fmaf(g[i], f[i], dw[i]); // columns past c, rows past n: dy = 0
                    if constexpr (!RMS)
                        db[i] += g[i];
                    g[i] *= w[i];
                    s1 += g[i];
                    s2 = fmaf(g[i], f[i], s2);
                }
                s1 = RMS ? 0.0f : sum(s1) * inv_c;
                s2 = sum(s2) * inv_c;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    f[i] = rstd[u] * (g[i] - s1 - f[i] * s2);
            }
            if (row < p.n) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int pos = (v * L + l) * E;
                    if (pos < p.c)
                        store_vec<T>(out + row * p.ldo, pos, p.c, f + v * E);
                }
            }
        }
    }
    if constexpr (BWD) {
        // the CTA's partial row: over a warp's rows by shuffles, over the warps in order
        auto write = [&](float *acc, float *dst) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
#pragma unroll
                for (int o = L; o < 32; o <<= 1)
                    acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], o);
                if (sub == 0)
                    red[warp * L * N + column(i)] = acc[i];
            }
            __syncthreads();
            for (int col = threadIdx.x; col < p.c; col += 256) {
                float a = 0.0f;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    a += red[q * L * N + col];
                dst[(int64_t)blockIdx.x * p.cpad + col] = a;
            }
            __syncthreads();
        };
        write(dw, p.pdw);
        if constexpr (!RMS)
            if (p.pdb)
                write(db, p.pdb);
    }
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

constexpr int kShortest = 512, kWidest = 8192, kWideSlices = 64;
constexpr size_t kSmemMost = 224 * 1024; // dynamic shared memory of the CTAs of one SM

int bwd_warps(int64_t c)
{
    int g = 2; // up to 512 columns: short rows
    while (g * 32 * LE < c)
        g *= 2;
    return g;
}

size_t row_size(int64_t c, int esize)
{
    return (size_t)((c * esize + 15) / 16 * 16);
}

// Short rows: lanes a row, vectors a lane, and the grid (a warp's 32 / lanes
// rows, four or two at a time).
struct ShortPlan {
    int lanes, vecs, grid;
};

ShortPlan short_plan(int64_t n, int64_t c, int esize, bool bwd)
{
    const int64_t vectors = (c * esize + 15) / 16;
    ShortPlan r;
    r.vecs = vectors <= 32 ? 1 : (vectors <= 64 ? 2 : 4);
    r.lanes = vectors <= 8 ? 8 : (vectors <= 16 ? 16 : 32);
    const int elems = 16 / esize * r.vecs, rows = 8 * (32 / r.lanes) * (elems > 8 ? 2 : 4);
    const int64_t need = (n + rows - 1) / rows, most = (int64_t)sm_count() * short_ctas(elems, bwd);
    r.grid = (int)(need < most ? need : most);
    return r;
}

struct NormPlan {
    int warps, threads, grid, stages; // warps a row
    int groups;                       // backward: partial rows of dw and db
    size_t smem;
};

// Backward: what the registers and the rings allow; a group gets four rows or
// more, so that its partial rows stay a small part of the traffic.
NormPlan bwd_plan(int64_t n, int64_t c, int esize)
{
    NormPlan r = {};
    r.warps = bwd_warps(c);
    const int per_cta = r.warps < 8 ? 8 / r.warps : 1, ctas = norm_bwd_ctas(r.warps);
    const size_t row = 2 * row_size(c, esize);
    r.stages = 4;
    while (r.stages > 2 && ctas * (r.stages * per_cta * row + 2048) > kSmemMost)
        --r.stages;
    r.smem = r.stages * per_cta * row + 128;
    r.threads = 32 * r.warps * per_cta;
    int64_t groups = (n + 3) / 4;
    const int64_t most = (int64_t)sm_count() * ctas * per_cta;
    groups = groups < most ? groups : most;
    r.grid = (int)((groups + per_cta - 1) / per_cta);
    // every group that has a row writes its partial row
    const int64_t all = (int64_t)r.grid * per_cta;
    r.groups = (int)(all < n ? all : n);
    return r;
}

// Forward: a warp a row up to 8 KB, more warps above and for few rows; two
// CTAs an SM where half its shared memory holds rings for 8 warps of rows.
NormPlan fwd_plan(int64_t n, int64_t c, int esize, bool bias)
{
    NormPlan r = {};
    const size_t row = row_size(c, esize), params = (bias ? 2 : 1) * row + 128;
    const int sms = sm_count();
    r.warps = 1;
    while (r.warps < 8 && (row > (size_t)8192 * r.warps || (n <= sms && row >= (size_t)1024 * r.warps)))
        r.warps *= 2;
    r.stages = row <= 4096 ? 3 : 2;
    int ctas = 2;
    int64_t groups = ((kSmemMost / 2 - 2048) - params) / (r.stages * row);
    if (kSmemMost / 2 - 2048 < params || groups * r.warps < 8) {
        ctas = 1;
        groups = (kSmemMost - 2048 - params) / (r.stages * row);
    }
    if (groups > 16 / r.warps)
        groups = 16 / r.warps;
    const int64_t want = (n + sms - 1) / sms; // rows an SM: no more groups than that
    if (groups > want)
        groups = want;
    r.threads = (int)(32 * r.warps * groups);
    r.smem = params + (size_t)groups * r.stages * row;
    const int64_t need = (n + groups - 1) / groups, most = (int64_t)sms * ctas;
    r.grid = (int)(need < most ? need : most);
    return r;
}

template <typename K>
cudaError_t run_norm(K kern, int &configured_device, const NormParams &p, const NormPlan &plan, cudaStream_t st)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (configured_device != dev) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMost)) !=
            cudaSuccess)
            return e;
        configured_device = dev;
    }
    return launch_pdl(kern, dim3((unsigned)plan.grid), dim3((unsigned)plan.threads), plan.smem, st, p);
}

template <class T, int G, bool RMS>
cudaError_t run_norm_bwd(const NormParams &p, const NormPlan &plan, cudaStream_t st)
{
    static int configured = -1;
    return run_norm(k_norm_bwd<T, G, RMS>, configured, p, plan, st);
}

template <class T, int G, bool RMS>
cudaError_t run_norm_fwd(const NormParams &p, const NormPlan &plan, cudaStream_t st)
{
    static int configured = -1;
    return run_norm(k_norm_fwd<T, G, RMS>, configured, p, plan, st);
}

template <class T, bool RMS, bool BWD>
cudaError_t run_short(const NormParams &p, const ShortPlan &plan, cudaStream_t st)
{
    const dim3 grid((unsigned)plan.grid), block(256);
    if (plan.vecs == 1) {
        if (plan.lanes == 8)
            return launch_pdl(k_norm_short<T, 8, 1, RMS, BWD>, grid, block, 0, st, p);
        if (plan.lanes == 16)
            return launch_pdl(k_norm_short<T, 16, 1, RMS, BWD>, grid, block, 0, st, p);
        return launch_pdl(k_norm_short<T, 32, 1, RMS, BWD>, grid, block, 0, st, p);
    }
    if (plan.vecs == 2)
        return launch_pdl(k_norm_short<T, 32, 2, RMS, BWD>, grid, block, 0, st, p);
    if constexpr (sizeof(T) == 4 && BWD)
        return launch_pdl(k_norm_short<T, 32, 4, RMS, true>, grid, block, 0, st, p);
    else
        return cudaErrorInvalidValue; // 512 BF16 columns are two vectors a lane
}

template <class T, bool RMS>
cudaError_t pick_norm(const NormParams &p, const NormPlan &plan, bool bwd, cudaStream_t st)
{
    switch (plan.warps) {
    case 1: return run_norm_fwd<T, 1, RMS>(p, plan, st); // the backward pass uses two or more
    case 2: return bwd ? run_norm_bwd<T, 2, RMS>(p, plan, st) : run_norm_fwd<T, 2, RMS>(p, plan, st);
    case 4: return bwd ? run_norm_bwd<T, 4, RMS>(p, plan, st) : run_norm_fwd<T, 4, RMS>(p, plan, st);
    case 8: return bwd ? run_norm_bwd<T, 8, RMS>(p, plan, st) : run_norm_fwd<T, 8, RMS>(p, plan, st);
    default: return run_norm_bwd<T, 16, RMS>(p, plan, st); // the forward pass uses 8 at most
    }
}

template <class T, bool RMS>
cudaError_t norm_any(const NormArgs &a, NormParams p, bool bwd, cudaStream_t st)
{
    // four vectors a lane (FP32 rows of more than 256 columns) pay in the backward pass only: 32768 x 512
    // measured 40.6 us against 46.5, forward 28.1 against 23.4
    const bool wide = a.c > kWidest, narrow = a.c <= kShortest && (bwd || a.c * sizeof(T) <= 1024);
    const ShortPlan sp = narrow ? short_plan(a.n, a.c, (int)sizeof(T), bwd) : ShortPlan{};
    const int64_t cap = (int64_t)sm_count() * 2;
    const dim3 wide_grid((unsigned)(a.n < cap ? a.n : cap));
    if (!bwd) {
        if (narrow)
            return run_short<T, RMS, false>(p, sp, st);
        if (wide)
            return launch_pdl(k_norm_wide<T, RMS, false>, wide_grid, dim3(1024), 0, st, p);
        const NormPlan plan = fwd_plan(a.n, a.c, (int)sizeof(T), a.b != nullptr);
        p.stages = plan.stages;
        return pick_norm<T, RMS>(p, plan, false, st);
    }
    cudaError_t e;
    NormPlan plan = {};
    if (narrow) {
        plan.groups = sp.grid;
        e = run_short<T, RMS, true>(p, sp, st);
    } else if (!wide) {
        plan = bwd_plan(a.n, a.c, (int)sizeof(T));
        p.stages = plan.stages;
        e = pick_norm<T, RMS>(p, plan, true, st);
    } else {
        plan.groups = (int)(a.n < kWideSlices ? a.n : kWideSlices);
        // the sums over dy and x come first: dx, which may be either of them, is written by the second kernel
        e = launch_pdl(k_norm_wide_params<T, RMS>, dim3((unsigned)((a.c + 255) / 256), (unsigned)plan.groups),
                       dim3(256), 0, st, p);
        if (e == cudaSuccess)
            e = launch_pdl(k_norm_wide<T, RMS, true>, wide_grid, dim3(1024), 0, st, p);
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
    const int esize = dtype == JETQ_OUT_BF16 ? 2 : 4;
    return c <= kShortest ? short_plan(n, c, esize, true).grid : bwd_plan(n, c, esize).groups;
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
