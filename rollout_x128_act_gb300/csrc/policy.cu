// Clipped policy-gradient loss of packed sequences with a KL term, and its
// gradient with respect to the token losses (nll = minus log-probability).
//
//   logr = nll_old - nll;   r = exp(logr), or of a segment exp(mean of logr over its counted tokens)
//   L    = -A m;   A >= 0: m = min(r, 1 + high);   A < 0: m = min(max(r, 1 - low), dual)
//   kl   = exp(d) - 1 - d,   d = nll - nll_ref
//   loss = sum over counted tokens of w (L + kl_coef * kl),   w = scale / N, scale / (S n_s) or scale
//   dnll = w (A r [not clipped] + kl_coef * (exp(d) - 1))
//
// Bound: HBM for long batches (17 to 21 bytes a token, read by the forward and
// again by the backward pass, which needs N and S first), launches for short ones.
//
// Work is split along the tokens, not the sequences, whose lengths run from
// one to millions: a warp takes a window of 128 tokens (four a lane, loaded
// together) and walks the sequences that cross it.  The part of sequence s in
// window w is piece w + s of the partial sums: along the staircase of windows
// and sequences each step raises one of the two, so no two pieces share an index
// and none needs a counter or an atomic.  A second kernel joins each sequence's
// pieces in binary64 (few values) in a fixed order: results are repeatable.
//
// Which side of the clip's border a token is on decides whether its gradient
// is there at all, so logr keeps the rounding error of its subtraction and is
// compared with the border's logarithm in two floats.
#include <cuda_runtime.h>

#include <cmath>

#include "jetq_internal.h"
#include "ptx.cuh"

namespace jetq {

namespace {

constexpr int kWindow = 128, kSlots = kWindow / 32; // tokens a warp, tokens a lane
constexpr int kWarps = 8;                           // windows a CTA

struct PolicyParams {
    const float *nll, *old, *ref, *adv;
    const uint8_t *mask;
    const int64_t *seg;
    int64_t n, windows;
    int nseg;
    bool adv_token, by_seg;
    int mean;
    float scale, kl;
    float low, high, dual;             // 1 - low, 1 + high, the bound or infinity
    float2 log_low, log_high, log_dual; // their logarithms, in two floats
    struct Piece *pieces;
    double *part;     // [join CTAs][5]
    unsigned *ticket; // of the join's CTAs
    int segs_cta;     // sequences a CTA of the join
    float *out, *save;
    const float *dloss;
    float *dnll;
};

// Sums over the counted tokens of a sequence in a window.
struct alignas(16) Piece {
    float count, clipped; // clipped: of a segment's ratio the tokens with A < 0
    float a, b, c, kl;    // a: L, or the positive A; b: the negative A; a segment's logr is c + c_rest
    float c_rest, unused;
};

__device__ __forceinline__ bool above(float d, float e, float2 t)
{
    return (d - t.x) + (e - t.y) > 0.0f;
}

__device__ __forceinline__ bool below(float d, float e, float2 t)
{
    return (d - t.x) + (e - t.y) < 0.0f;
}

// a - b and what its rounding lost (Knuth's two-sum); an infinite one has no rest.
__device__ __forceinline__ void two_diff(float a, float b, float &d, float &e)
{
    d = __fsub_rn(a, b);
    const float u = __fsub_rn(d, a);
    e = __fsub_rn(__fsub_rn(a, __fsub_rn(d, u)), __fadd_rn(b, u));
    e = fabsf(d) < INFINITY ? e : 0.0f;
}

__device__ __forceinline__ void add_to(float &s, float &c, float b)
{
    const float t = __fadd_rn(s, b), u = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, u)), __fsub_rn(b, u)));
    s = t;
}

// exp(d) - 1 - d: below 1/2 by its Taylor series (the next term is 1e-8 of the sum).
__device__ __forceinline__ float kl_term(float d)
{
    if (fabsf(d) < 0.5f) {
        float s = 1.0f / 40320.0f;
        s = fmaf(s, d, 1.0f / 5040.0f);
        s = fmaf(s, d, 1.0f / 720.0f);
        s = fmaf(s, d, 1.0f / 120.0f);
        s = fmaf(s, d, 1.0f / 24.0f);
        s = fmaf(s, d, 1.0f / 6.0f);
        return d * d * fmaf(s, d, 0.5f);
    }
    return expm1f(d) - d;
}

// The ratio's bound for advantage A where it is clipped.
__device__ __forceinline__ bool clip(const PolicyParams &p, float A, float d, float e, float &bound)
{
    if (A < 0.0f) {
        bound = p.low;
        if (below(d, e, p.log_low))
            return true;
        bound = p.dual;
        return above(d, e, p.log_dual);
    }
    bound = p.high;
    return above(d, e, p.log_high);
}

// First sequence that ends after token t (nseg: none), searched 32 offsets at a time.
__device__ __forceinline__ int first_segment(const int64_t *seg, int nseg, int64_t t, int lane)
{
    int lo = 0, hi = nseg; // the answer is in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step; // candidates lo, lo + step, ...
        const bool past = at >= hi || __ldg(seg + at + 1) > t;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, past);
        const int f = m ? __ffs(m) - 1 : 32; // the first candidate that ends after t
        if (f == 0)
            return lo;
        const int next = lo + (f - 1) * step + 1;
        hi = min(hi, lo + f * step);
        lo = min(next, hi);
    }
    return lo;
}

// The sequences that cross tokens [t0, t1), in turn: fn(sequence, first token, last token + 1, its advantage).
template <class F>
__device__ __forceinline__ void walk(const PolicyParams &p, int64_t t0, int64_t t1, int lane, F fn)
{
    if (!p.seg) {
        fn(0, t0, t1, p.adv_token ? 0.0f : __ldg(p.adv));
        return;
    }
    int s = first_segment(p.seg, p.nseg, t0, lane);
    while (s < p.nseg) {
        const int mine = min(s + lane, p.nseg - 1); // 32 sequences' offsets in one load
        const int64_t begin = __ldg(p.seg + mine), end = __ldg(p.seg + mine + 1);
        const float adv = p.adv_token ? 0.0f : __ldg(p.adv + mine);
        const int many = min(32, p.nseg - s);
        for (int i = 0; i < many; ++i) {
            const int64_t b = __shfl_sync(0xFFFFFFFFu, begin, i), e = __shfl_sync(0xFFFFFFFFu, end, i);
            const float A = __shfl_sync(0xFFFFFFFFu, adv, i);
            if (b >= t1)
                return;
            const int64_t from = b > t0 ? b : t0, to = e < t1 ? e : t1;
            if (from < to)
                fn(s + i, from, to, A);
        }
        s += many;
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// What a lane loads of its tokens t0 + lane + 32 k.
struct Tokens {
    float d[kSlots], e[kSlots], dref[kSlots], A[kSlots];
    bool on[kSlots];
    __device__ __forceinline__ void load(const PolicyParams &p, int64_t t0, int lane)
    {
        float x[kSlots], y[kSlots], z[kSlots];
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            const int64_t t = t0 + lane + 32 * k;
            on[k] = t < p.n;
            x[k] = y[k] = z[k] = A[k] = 0.0f;
            if (on[k]) {
                x[k] = __ldg(p.nll + t);
                y[k] = __ldg(p.old + t);
                if (p.ref)
                    z[k] = __ldg(p.ref + t);
                if (p.adv_token)
                    A[k] = __ldg(p.adv + t);
                if (p.mask)
                    on[k] = __ldg(p.mask + t) != 0;
            }
        }
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            two_diff(y[k], x[k], d[k], e[k]);
            dref[k] = p.ref ? x[k] - z[k] : 0.0f;
        }
    }
};

template <bool BY_SEG>
__global__ void __launch_bounds__(32 * kWarps) k_policy_pieces(const PolicyParams p)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), t0 = w * kWindow;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *p.ticket = 0;
    if (t0 >= p.n)
        return;
    Tokens tk;
    tk.load(p, t0, lane);
    float r[kSlots], kl[kSlots];
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
        r[k] = 0.0f;
        if (!BY_SEG) {
            r[k] = expf(tk.d[k]);
            if (tk.e[k] != 0.0f)
                r[k] = fmaf(r[k], tk.e[k], r[k]);
        }
        kl[k] = p.ref ? kl_term(tk.dref[k]) : 0.0f;
    }
    const int64_t t1 = min(t0 + kWindow, p.n);
    walk(p, t0, t1, lane, [&](int s, int64_t from, int64_t to, float A_seg) {
        const int lo = (int)(from - t0) - lane, hi = (int)(to - t0) - lane;
        int count = 0, clipped = 0;
        float a = 0.0f, b = 0.0f, c = 0.0f, rest = 0.0f, q = 0.0f;
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            const bool in = tk.on[k] && 32 * k >= lo && 32 * k < hi;
            const float A = p.adv_token ? tk.A[k] : A_seg;
            bool side;
            if (BY_SEG) {
                side = A < 0.0f;
                a += in && !side ? A : 0.0f;
                b += in && side ? A : 0.0f;
                if (in) {
                    add_to(c, rest, tk.d[k]);
                    rest += tk.e[k];
                }
            } else {
                float bound;
                side = clip(p, A, tk.d[k], tk.e[k], bound);
                a += in ? -A * (side ? bound : r[k]) : 0.0f;
            }
            q += in ? kl[k] : 0.0f;
            count += __popc(__ballot_sync(0xFFFFFFFFu, in));
            clipped += __popc(__ballot_sync(0xFFFFFFFFu, in && side));
        }
        a = warp_sum(a);
        if (p.ref)
            q = warp_sum(q);
        if (BY_SEG) {
            b = warp_sum(b);
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const float c2 = __shfl_xor_sync(0xFFFFFFFFu, c, o), r2 = __shfl_xor_sync(0xFFFFFFFFu, rest, o);
                add_to(c, rest, c2);
                rest += r2;
            }
        }
        if (lane == 0) {
            float4 *out = reinterpret_cast<float4 *>(p.pieces + (w + s));
            out[0] = make_float4((float)count, (float)clipped, a, b);
            out[1] = make_float4(c, q, rest, 0.0f);
        }
    });
}

struct SegSums {
    double count, clipped, a, b, c, kl;
    __device__ __forceinline__ void clear() { count = clipped = a = b = c = kl = 0.0; }
    __device__ __forceinline__ void add(const Piece *piece, bool by_seg)
    {
        const float4 u = __ldcg(reinterpret_cast<const float4 *>(piece));
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(piece) + 1);
        count += u.x;
        clipped += u.y;
        a += u.z;
        kl += v.y;
        if (by_seg) {
            b += u.w;
            c += (double)v.x + (fabsf(v.x) < INFINITY ? (double)v.z : 0.0);
        }
    }
    template <class S>
    __device__ __forceinline__ void all(S sum)
    {
        count = sum(count);
        clipped = sum(clipped);
        a = sum(a);
        b = sum(b);
        c = sum(c);
        kl = sum(kl);
    }
};

constexpr int kJoinThreads = 256, kLanesSeg = 4, kLong = 256; // a sequence's lanes; pieces from which the CTA takes it

// Sums of each sequence's pieces; their share of the loss; the last CTA to finish adds the CTAs' shares.
__global__ void __launch_bounds__(kJoinThreads) k_policy_join(const PolicyParams p)
{
    __shared__ double red[kJoinThreads / 32][6];
    __shared__ int longs[kJoinThreads / kLanesSeg], num_longs;
    __shared__ bool last;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = threadIdx.x % kLanesSeg;
    if (threadIdx.x == 0)
        num_longs = 0;
    __syncthreads();
    double tot[5] = {0.0, 0.0, 0.0, 0.0, 0.0}; // surrogate, kl, clipped, tokens, sequences
    auto range = [&](int s, int64_t &w0, int64_t &w1) { // windows of sequence s
        int64_t b = p.seg ? __ldg(p.seg + s) : 0, e = p.seg ? __ldg(p.seg + s + 1) : p.n;
        b = b < 0 ? 0 : b;
        e = e > p.n ? p.n : e;
        w0 = b / kWindow;
        w1 = e > b ? (e - 1) / kWindow + 1 : w0;
    };
    auto finish = [&](int s, const SegSums &x) {
        double surrogate = x.a, clipped = x.clipped;
        float g = 0.0f;
        if (p.by_seg && x.count > 0.0) {
            const double mean = x.c / x.count;
            const float2 l = p.log_low, h = p.log_high, u = p.log_dual;
            const bool hi = mean > (double)h.x + h.y, lo = mean < (double)l.x + l.y, du = mean > (double)u.x + u.y;
            const double ratio = exp(mean);
            // a sum without a token of its sign stays out: 0 * infinity is no number
            const double pos = x.a != 0.0 ? -x.a * (hi ? (double)p.high : ratio) : 0.0;
            const double neg = x.b != 0.0 ? -x.b * (lo ? (double)p.low : du ? (double)p.dual : ratio) : 0.0;
            const double live = (hi ? 0.0 : x.a) + (lo || du ? 0.0 : x.b);
            surrogate = pos + neg;
            clipped = (hi ? x.count - x.clipped : 0.0) + (lo || du ? x.clipped : 0.0);
            g = live != 0.0 ? (float)(live * ratio / x.count) : 0.0f;
        }
        reinterpret_cast<float2 *>(p.save)[s] = make_float2((float)x.count, g);
        if (x.count > 0.0) {
            const double f = p.mean == JETQ_POLICY_MEAN_SEGMENTS ? 1.0 / x.count : 1.0;
            tot[0] += f * surrogate;
            tot[1] += f * x.kl;
            tot[2] += clipped;
            tot[3] += x.count;
            tot[4] += 1.0;
        }
    };
    const int64_t first = (int64_t)blockIdx.x * p.segs_cta;
    const int mine = threadIdx.x / kLanesSeg;
    {
        const int64_t s = first + mine;
        const bool have = mine < p.segs_cta && s < p.nseg;
        int64_t w0 = 0, w1 = 0;
        if (have)
            range((int)s, w0, w1);
        const bool is_long = w1 - w0 > kLong;
        if (is_long && sub == 0)
            longs[atomicAdd(&num_longs, 1)] = (int)s;
        SegSums x;
        x.clear();
        if (!is_long)
            for (int64_t w = w0 + sub; w < w1; w += kLanesSeg)
                x.add(p.pieces + (w + s), p.by_seg);
        x.all([&](double v) {
#pragma unroll
            for (int o = kLanesSeg / 2; o; o >>= 1)
                v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            return v;
        });
        if (have && !is_long && sub == 0)
            finish((int)s, x);
    }
    __syncthreads();
    const int many = num_longs;
    // in the order of the sequences, whatever the order in which they were listed
    int after = -1;
    for (int i = 0; i < many; ++i) {
        int s = 0x7FFFFFFF;
        for (int j = 0; j < many; ++j)
            if (longs[j] > after)
                s = min(s, longs[j]);
        after = s;
        int64_t w0, w1;
        range(s, w0, w1);
        SegSums x;
        x.clear();
#pragma unroll 4
        for (int64_t w = w0 + threadIdx.x; w < w1; w += kJoinThreads)
            x.add(p.pieces + (w + s), p.by_seg);
        auto warp_all = [&](double v) {
#pragma unroll
            for (int o = 16; o; o >>= 1)
                v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            return v;
        };
        x.all(warp_all);
        if (lane == 0) {
            const double v[6] = {x.count, x.clipped, x.a, x.b, x.c, x.kl};
            for (int k = 0; k < 6; ++k)
                red[warp][k] = v[k];
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            double v[6] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
            for (int g = 0; g < kJoinThreads / 32; ++g)
                for (int k = 0; k < 6; ++k)
                    v[k] += red[g][k];
            finish(s, SegSums{v[0], v[1], v[2], v[3], v[4], v[5]});
        }
        __syncthreads();
    }
    // the CTA's share, then all of them
    auto cta_sum = [&](double (&v)[5]) { // to thread 0
        for (int k = 0; k < 5; ++k) {
#pragma unroll
            for (int o = 16; o; o >>= 1)
                v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
            if (lane == 0)
                red[warp][k] = v[k];
        }
        __syncthreads();
        if (threadIdx.x == 0)
            for (int k = 0; k < 5; ++k) {
                v[k] = 0.0;
                for (int g = 0; g < kJoinThreads / 32; ++g)
                    v[k] += red[g][k];
            }
    };
    cta_sum(tot);
    if (gridDim.x > 1) {
        if (threadIdx.x == 0) {
            for (int k = 0; k < 5; ++k)
                p.part[(int64_t)blockIdx.x * 5 + k] = tot[k];
            __threadfence();
            last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
        }
        __syncthreads();
        if (!last)
            return;
        __threadfence();
        for (int k = 0; k < 5; ++k)
            tot[k] = 0.0;
        for (unsigned i = threadIdx.x; i < gridDim.x; i += kJoinThreads)
            for (int k = 0; k < 5; ++k)
                tot[k] += __ldcg(p.part + (int64_t)i * 5 + k);
        cta_sum(tot);
    }
    if (threadIdx.x == 0) {
        double f = p.scale;
        if (p.mean != JETQ_POLICY_SUM) {
            const double by = p.mean == JETQ_POLICY_MEAN_SEGMENTS ? tot[4] : tot[3];
            f = by > 0.0 ? f / by : 0.0;
        }
        p.out[0] = (float)(f * (tot[0] + (p.ref ? (double)p.kl * tot[1] : 0.0)));
        p.out[1] = (float)(f * tot[0]);
        p.out[2] = (float)(f * tot[1]);
        p.out[3] = (float)tot[2];
        p.out[4] = (float)tot[3];
        p.out[5] = (float)tot[4];
    }
}

template <bool BY_SEG>
__global__ void __launch_bounds__(32 * kWarps) k_policy_bwd(const PolicyParams p)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kWindow;
    if (t0 >= p.n)
        return;
    Tokens tk;
    tk.load(p, t0, lane);
    float scale = p.scale;
    if (p.mean == JETQ_POLICY_MEAN_TOKENS)
        scale = __fdiv_rn(scale, __ldg(p.out + 4));
    else if (p.mean == JETQ_POLICY_MEAN_SEGMENTS)
        scale = __fdiv_rn(scale, __ldg(p.out + 5));
    if (p.dloss)
        scale *= __ldg(p.dloss);
    float g[kSlots];
#pragma unroll
    for (int k = 0; k < kSlots; ++k)
        g[k] = 0.0f;
    const int64_t t1 = min(t0 + kWindow, p.n);
    walk(p, t0, t1, lane, [&](int s, int64_t from, int64_t to, float A_seg) {
        const int lo = (int)(from - t0) - lane, hi = (int)(to - t0) - lane;
        const float2 seg = __ldg(reinterpret_cast<const float2 *>(p.save) + s);
        const float f = p.mean == JETQ_POLICY_MEAN_SEGMENTS ? __fdiv_rn(scale, seg.x) : scale;
#pragma unroll
        for (int k = 0; k < kSlots; ++k)
            if (tk.on[k] && 32 * k >= lo && 32 * k < hi) {
                float v = seg.y;
                if (!BY_SEG) {
                    const float A = p.adv_token ? tk.A[k] : A_seg;
                    float bound;
                    v = 0.0f;
                    if (!clip(p, A, tk.d[k], tk.e[k], bound)) {
                        const float r = expf(tk.d[k]);
                        v = A * (tk.e[k] != 0.0f ? fmaf(r, tk.e[k], r) : r);
                    }
                }
                if (p.ref)
                    v = fmaf(p.kl, expm1f(tk.dref[k]), v);
                g[k] = f * v;
            }
    });
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
        const int64_t t = t0 + lane + 32 * k;
        if (t < p.n)
            p.dnll[t] = g[k];
    }
}

int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

float2 two_floats(double v)
{
    const float hi = (float)v;
    return make_float2(hi, std::isfinite(hi) ? (float)(v - (double)hi) : 0.0f);
}

PolicyParams params_of(const PolicyArgs &a)
{
    PolicyParams p = {};
    p.nll = a.nll;
    p.old = a.nll_old;
    p.ref = a.nll_ref;
    p.adv = a.adv;
    p.mask = a.mask;
    p.seg = a.seg;
    p.n = a.n;
    p.windows = ceil_div(a.n, kWindow);
    p.nseg = a.seg ? a.nseg : 1;
    p.adv_token = a.adv_per_token != 0;
    p.by_seg = a.level == JETQ_POLICY_SEGMENT;
    p.mean = a.mean;
    p.scale = a.scale;
    p.kl = a.kl;
    p.low = 1.0f - a.low;
    p.high = 1.0f + a.high;
    p.dual = a.dual > 0.0f ? a.dual : INFINITY;
    p.log_low = two_floats(std::log(1.0 - (double)a.low)); // -infinity at 1
    p.log_high = two_floats(std::log(1.0 + (double)a.high));
    p.log_dual = two_floats(a.dual > 0.0f ? std::log((double)a.dual) : (double)INFINITY);
    p.out = a.out;
    p.save = a.save;
    p.dloss = a.dloss;
    p.dnll = a.dnll;
    return p;
}

// Sequences a CTA of the join: about 512 pieces, in as many CTAs as that makes.
int segs_a_cta(int64_t windows, int64_t nseg)
{
    const int64_t most = kJoinThreads / kLanesSeg, s = 512 * nseg / (windows + nseg);
    return (int)(s < 1 ? 1 : s > most ? most : s);
}

} // namespace

size_t policy_loss_workspace(int64_t n, int64_t nseg)
{
    const int64_t windows = ceil_div(n, kWindow);
    return 16 + (size_t)(windows + nseg) * sizeof(Piece) +
           (size_t)ceil_div(nseg, segs_a_cta(windows, nseg)) * 5 * sizeof(double);
}

cudaError_t launch_policy_fwd(const PolicyArgs &a, cudaStream_t st)
{
    PolicyParams p = params_of(a);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    p.ticket = reinterpret_cast<unsigned *>(ws);
    p.pieces = reinterpret_cast<Piece *>(ws + 16);
    p.part = reinterpret_cast<double *>(ws + 16 + (size_t)(p.windows + p.nseg) * sizeof(Piece));
    p.segs_cta = segs_a_cta(p.windows, p.nseg);
    const dim3 grid((unsigned)ceil_div(p.windows, kWarps)), block(32 * kWarps);
    const cudaError_t e = p.by_seg ? launch_pdl(k_policy_pieces<true>, grid, block, 0, st, p)
                                   : launch_pdl(k_policy_pieces<false>, grid, block, 0, st, p);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(k_policy_join, dim3((unsigned)ceil_div(p.nseg, p.segs_cta)), dim3(kJoinThreads), 0, st, p);
}

cudaError_t launch_policy_bwd(const PolicyArgs &a, cudaStream_t st)
{
    const PolicyParams p = params_of(a);
    const dim3 grid((unsigned)ceil_div(p.windows, kWarps)), block(32 * kWarps);
    return p.by_seg ? launch_pdl(k_policy_bwd<true>, grid, block, 0, st, p)
                    : launch_pdl(k_policy_bwd<false>, grid, block, 0, st, p);
}

} // namespace jetq
