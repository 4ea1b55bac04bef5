// Clipped policy-gradient loss of packed sequences with a KL term, and its
// gradient with respect to the token losses (nll = minus log-probability).
//
//   logr = nll_old - nll;   r = exp(logr), or of a segment exp(mean of logr over its counted tokens)
//   L    = -A m;   A >= 0: m = min(r, 1 + high);   A < 0: m = min(max(r, 1 - low), dual)
//   kl   = exp(d) - 1 - d,   d = nll - nll_ref
//   loss = sum over counted tokens of w (L + kl_coef * kl),   w = scale / N, scale / (S n_s) or scale
//   dnll = w (A r [not clipped] + kl_coef * (exp(d) - 1))
//
// Floor: HBM for long batches (8 to 17 bytes a token, read by the forward and
// again by the backward pass, which needs N and S first and writes 4), launches
// for short ones.  Both directions in a graph: 4194304 tokens in 8192 sequences
// 47 us (issue slots 68% used: some 120 instructions a token and direction; HBM
// would take 10), 1000003 tokens in 24 sequences 29 us (the latencies of three
// kernels; 10 us of it the join), 524288 in 512 21 us, 1531 in 8 15 us.  An
// advantage a token under one ratio a sequence costs 4 us of 51 at 4194304 tokens:
// its two sums are compensated.
//
// Work is split along the tokens, not the sequences, whose lengths run from
// one to millions: a warp takes a chunk of consecutive windows of 128 tokens
// (four a lane, loaded a window ahead) and walks the sequences that cross it.
// The part of sequence s in chunk c is piece c + s of the partial sums: along
// the staircase of chunks and sequences each step raises one of the two, so no
// two pieces share an index and none needs a counter or an atomic.  A lane sums
// its own tokens of a piece, and the lanes are added where the piece ends.  A
// second kernel joins each sequence's pieces in a fixed order, with compensated
// FP32 sums (binary64 is slow here: the join took 25 to 49 us with it): results
// are repeatable.  Up to 4096 tokens in 256 sequences one CTA does both.
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
    bool adv_sums; // both: sums of the advantages of either sign
    int chunk; // consecutive windows a warp
    int mean;
    float scale, kl;
    float low, high, dual;              // 1 - low, 1 + high, the bound or infinity
    float2 log_low, log_high, log_dual; // their logarithms, in two floats
    struct Piece *pieces;
    struct Totals *part; // [join CTAs]
    unsigned *ticket;    // of the join's CTAs
    int segs_cta;        // sequences a CTA of the join
    float *out, *save;
    const float *dloss;
    float *dnll;
};

// Sums over the counted tokens of a sequence in a chunk.
struct alignas(16) Piece {
    // clipped: of a segment's ratio with an advantage a token those with A < 0, and 2^16 times those with A = 0
    int count, clipped;
    float c, c_rest;    // c + c_rest: L, or of a segment's ratio logr
    float kl, unused[3];
    float a, a_rest, b, b_rest; // of a segment's ratio with an advantage a token: the positive A, the negative A
};

// Sums over sequences: surrogate and KL term (with their rests), numbers of clipped tokens, tokens, sequences.
struct alignas(16) Totals {
    float l, l_rest, kl, kl_rest;
    unsigned long long clipped, tokens, segs;
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

// exp(d) - 1 - d: up to |d| = 1 by its Taylor series (the next term is below 2^-26 of the sum).
__device__ __forceinline__ float kl_term(float d)
{
    if (fabsf(d) < 1.0f) {
        float s = 1.0f / 479001600.0f;
        s = fmaf(s, d, 1.0f / 39916800.0f);
        s = fmaf(s, d, 1.0f / 3628800.0f);
        s = fmaf(s, d, 1.0f / 362880.0f);
        s = fmaf(s, d, 1.0f / 40320.0f);
        s = fmaf(s, d, 1.0f / 5040.0f);
        s = fmaf(s, d, 1.0f / 720.0f);
        s = fmaf(s, d, 1.0f / 120.0f);
        s = fmaf(s, d, 1.0f / 24.0f);
        s = fmaf(s, d, 1.0f / 6.0f);
        return d * d * fmaf(s, d, 0.5f);
    }
    return expm1f(d) - d;
}

// exp(d) - 1, from the term above where the two are near.
__device__ __forceinline__ float kl_slope(float d)
{
    return fabsf(d) < 1.0f ? d + kl_term(d) : expm1f(d);
}

// The bound of the ratio, and whether the ratio is beyond it, for advantage A.  With A = 0 the bound changes nothing,
// so such a token is not counted as clipped, unless the ratio is infinite: the bound stands in for 0 * infinity.
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

// The sequences that cross a warp's windows, in turn.
struct Walker {
    int s, base; // the sequence, the first of the 32 that the lanes hold (-1: none yet)
    int64_t begin, end;
    float adv;
    float2 save;
    __device__ __forceinline__ void start(const PolicyParams &p, int64_t t0, int lane)
    {
        s = p.seg ? first_segment(p.seg, p.nseg, t0, lane) : 0;
        base = -1;
    }
    // fn(sequence, first token, last token + 1, advantage, saved pair, whether the sequence's part of the chunk ends
    // here) for tokens [t0, t1), the last ones of the chunk or not; windows follow one another
    template <bool SAVED, class F>
    __device__ __forceinline__ void window(const PolicyParams &p, int64_t t0, int64_t t1, bool last, int lane, F fn)
    {
        while (s < p.nseg) {
            if (base < 0 || s - base >= 32) { // 32 sequences' values in one load
                base = s;
                const int mine = min(s + lane, p.nseg - 1);
                begin = p.seg ? __ldg(p.seg + mine) : 0;
                end = p.seg ? __ldg(p.seg + mine + 1) : p.n;
                adv = p.adv_token ? 0.0f : __ldg(p.adv + mine);
                if (SAVED)
                    save = __ldcg(reinterpret_cast<const float2 *>(p.save) + mine);
            }
            const int i = s - base;
            const int64_t b = __shfl_sync(0xFFFFFFFFu, begin, i), e = __shfl_sync(0xFFFFFFFFu, end, i);
            const float A = __shfl_sync(0xFFFFFFFFu, adv, i);
            float2 sv = make_float2(0.0f, 0.0f);
            if (SAVED)
                sv = make_float2(__shfl_sync(0xFFFFFFFFu, save.x, i), __shfl_sync(0xFFFFFFFFu, save.y, i));
            if (b >= t1)
                return;
            const int64_t from = b > t0 ? b : t0, to = e < t1 ? e : t1;
            if (from < to)
                fn(s, from, to, A, sv, last || e <= t1);
            if (e > t1)
                return;
            ++s;
        }
    }
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// s + c of all lanes, compensated.
__device__ __forceinline__ void warp_sum(float &s, float &c)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float s2 = __shfl_xor_sync(0xFFFFFFFFu, s, o), c2 = __shfl_xor_sync(0xFFFFFFFFu, c, o);
        add_to(s, c, s2);
        c += c2;
    }
}

// What a lane loads of its tokens t0 + lane + 32 k.
struct Tokens {
    float x[kSlots], y[kSlots], z[kSlots], A[kSlots];
    bool on[kSlots];
    __device__ __forceinline__ void load(const PolicyParams &p, int64_t t0, int lane)
    {
        const int64_t at = t0 + lane;
        const int left = (int)min(p.n - t0, (int64_t)kWindow) - lane; // slot k is a token: 32 k < left
        const float *px = p.nll + at, *py = p.old + at;
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            on[k] = 32 * k < left;
            x[k] = on[k] ? __ldg(px + 32 * k) : 0.0f;
            y[k] = on[k] ? __ldg(py + 32 * k) : 0.0f;
            z[k] = A[k] = 0.0f;
        }
        if (p.ref) {
            const float *pz = p.ref + at;
#pragma unroll
            for (int k = 0; k < kSlots; ++k)
                z[k] = on[k] ? __ldg(pz + 32 * k) : 0.0f;
        }
        if (p.adv_token) {
            const float *pa = p.adv + at;
#pragma unroll
            for (int k = 0; k < kSlots; ++k)
                A[k] = on[k] ? __ldg(pa + 32 * k) : 0.0f;
        }
        if (p.mask) {
            const uint8_t *pm = p.mask + at;
#pragma unroll
            for (int k = 0; k < kSlots; ++k)
                on[k] = on[k] && __ldg(pm + 32 * k) != 0;
        }
    }
};

// exp of d + e; an infinite one has no rest (infinity * e + infinity is no number for a negative e)
__device__ __forceinline__ float ratio_of(float d, float e)
{
    const float r = expf(d);
    return e != 0.0f && r < INFINITY ? fmaf(r, e, r) : r;
}

// A chunk's sums of each piece.
template <bool BY_SEG>
__device__ __forceinline__ void sum_pieces(const PolicyParams &p, int64_t chunk, int lane)
{
    const int64_t w0 = chunk * p.chunk, w1 = min(w0 + p.chunk, p.windows);
    Tokens tk, next;
    next.load(p, w0 * kWindow, lane);
    Walker walk;
    walk.start(p, w0 * kWindow, lane);
    // this lane's sums of the piece
    int count = 0, clipped = 0;
    float a = 0.0f, a_rest = 0.0f, b = 0.0f, b_rest = 0.0f, c = 0.0f, rest = 0.0f, q = 0.0f;
    for (int64_t w = w0; w < w1; ++w) {
        tk = next;
        if (w + 1 < w1)
            next.load(p, (w + 1) * kWindow, lane);
        float d[kSlots], e[kSlots], r[kSlots], kl[kSlots];
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            two_diff(tk.y[k], tk.x[k], d[k], e[k]);
            r[k] = BY_SEG ? 0.0f : ratio_of(d[k], e[k]);
            kl[k] = p.ref ? kl_term(tk.x[k] - tk.z[k]) : 0.0f;
        }
        const int64_t t0 = w * kWindow, t1 = min(t0 + kWindow, p.n);
        walk.window<false>(p, t0, t1, w + 1 == w1, lane,
                           [&](int s, int64_t from, int64_t to, float A_seg, float2, bool ends) {
            const int lo = (int)(from - t0) - lane, hi = (int)(to - t0) - lane;
#pragma unroll
            for (int k = 0; k < kSlots; ++k) {
                const bool in = tk.on[k] && 32 * k >= lo && 32 * k < hi;
                const float A = p.adv_token ? tk.A[k] : A_seg;
                bool side;
                // compensated: a policy that is still its sampling policy adds the same -A at each token of a
                // sequence, whose roundings do not average out; and A of either sign nearly cancel
                if (BY_SEG) {
                    side = A < 0.0f;
                    if (p.adv_token && in) {
                        float sum = side ? b : a, lost = side ? b_rest : a_rest;
                        add_to(sum, lost, A);
                        a = side ? a : sum;
                        a_rest = side ? a_rest : lost;
                        b = side ? sum : b;
                        b_rest = side ? lost : b_rest;
                    }
                    if (in) {
                        add_to(c, rest, d[k]);
                        rest += e[k];
                    }
                } else {
                    float bound;
                    side = clip(p, A, d[k], e[k], bound);
                    if (in)
                        add_to(c, rest, -A * (side ? bound : r[k]));
                }
                q += in ? kl[k] : 0.0f;
                count += in;
                if (BY_SEG) // 4096 tokens a piece at most
                    clipped += in && p.adv_token ? side ? 1 : A == 0.0f ? 1 << 16 : 0 : 0;
                else
                    clipped += in && side && (A != 0.0f || !(r[k] < INFINITY));
            }
            if (!ends)
                return;
            count = __reduce_add_sync(0xFFFFFFFFu, count);
            clipped = __reduce_add_sync(0xFFFFFFFFu, clipped);
            if (p.ref)
                q = warp_sum(q);
            warp_sum(c, rest);
            if (BY_SEG && p.adv_token) {
                warp_sum(a, a_rest);
                warp_sum(b, b_rest);
            }
            if (lane == 0) {
                float4 *out = reinterpret_cast<float4 *>(p.pieces + (chunk + s));
                out[0] = make_float4(__int_as_float(count), __int_as_float(clipped), c, rest);
                p.pieces[chunk + s].kl = q;
                if (BY_SEG && p.adv_token)
                    out[2] = make_float4(a, a_rest, b, b_rest);
            }
            count = clipped = 0;
            a = a_rest = b = b_rest = c = rest = q = 0.0f;
        });
    }
}

// Value of a sum and its rest; an infinite one has none.
__device__ __forceinline__ float whole(float s, float rest)
{
    return fabsf(s) < INFINITY ? s + rest : s;
}

struct SegSums {
    unsigned long long count, clipped, zero; // zero: with sums of the advantages, the tokens with A = 0
    float a, a_rest, b, b_rest, c, c_rest, kl, kl_rest;
    __device__ __forceinline__ void clear()
    {
        count = clipped = zero = 0;
        a = a_rest = b = b_rest = c = c_rest = kl = kl_rest = 0.0f;
    }
    __device__ __forceinline__ void add(const Piece *piece, bool adv_sums)
    {
        const float4 u = __ldcg(reinterpret_cast<const float4 *>(piece));
        const unsigned two = (unsigned)__float_as_int(u.y);
        count += (unsigned)__float_as_int(u.x);
        clipped += adv_sums ? two & 0xFFFFu : two;
        add_to(c, c_rest, u.z);
        c_rest += u.w;
        add_to(kl, kl_rest, __ldcg(&piece->kl));
        if (adv_sums) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(piece) + 2);
            zero += two >> 16;
            add_to(a, a_rest, v.x);
            a_rest += v.y;
            add_to(b, b_rest, v.z);
            b_rest += v.w;
        }
    }
    __device__ __forceinline__ void add(const SegSums &o, bool adv_sums)
    {
        count += o.count;
        clipped += o.clipped;
        add_to(c, c_rest, o.c);
        c_rest += o.c_rest;
        add_to(kl, kl_rest, o.kl);
        kl_rest += o.kl_rest;
        if (adv_sums) {
            zero += o.zero;
            add_to(a, a_rest, o.a);
            a_rest += o.a_rest;
            add_to(b, b_rest, o.b);
            b_rest += o.b_rest;
        }
    }
    __device__ __forceinline__ void add_lane(int o, bool adv_sums) // of lane ^ o
    {
        SegSums x;
        x.count = __shfl_xor_sync(0xFFFFFFFFu, count, o);
        x.clipped = __shfl_xor_sync(0xFFFFFFFFu, clipped, o);
        x.c = __shfl_xor_sync(0xFFFFFFFFu, c, o);
        x.c_rest = __shfl_xor_sync(0xFFFFFFFFu, c_rest, o);
        x.kl = __shfl_xor_sync(0xFFFFFFFFu, kl, o);
        x.kl_rest = __shfl_xor_sync(0xFFFFFFFFu, kl_rest, o);
        if (adv_sums) {
            x.zero = __shfl_xor_sync(0xFFFFFFFFu, zero, o);
            x.a = __shfl_xor_sync(0xFFFFFFFFu, a, o);
            x.a_rest = __shfl_xor_sync(0xFFFFFFFFu, a_rest, o);
            x.b = __shfl_xor_sync(0xFFFFFFFFu, b, o);
            x.b_rest = __shfl_xor_sync(0xFFFFFFFFu, b_rest, o);
        }
        add(x, adv_sums);
    }
};

__device__ __forceinline__ void add_totals(Totals &t, const Totals &o)
{
    add_to(t.l, t.l_rest, o.l);
    t.l_rest += o.l_rest;
    add_to(t.kl, t.kl_rest, o.kl);
    t.kl_rest += o.kl_rest;
    t.clipped += o.clipped;
    t.tokens += o.tokens;
    t.segs += o.segs;
}

// Sum over the first `lanes` (a power of two) lanes of a warp.
__device__ __forceinline__ void warp_totals(Totals &t, int lanes)
{
    for (int o = lanes / 2; o; o >>= 1) {
        Totals x;
        x.l = __shfl_xor_sync(0xFFFFFFFFu, t.l, o);
        x.l_rest = __shfl_xor_sync(0xFFFFFFFFu, t.l_rest, o);
        x.kl = __shfl_xor_sync(0xFFFFFFFFu, t.kl, o);
        x.kl_rest = __shfl_xor_sync(0xFFFFFFFFu, t.kl_rest, o);
        x.clipped = __shfl_xor_sync(0xFFFFFFFFu, t.clipped, o);
        x.tokens = __shfl_xor_sync(0xFFFFFFFFu, t.tokens, o);
        x.segs = __shfl_xor_sync(0xFFFFFFFFu, t.segs, o);
        add_totals(t, x);
    }
}

// s + c -= (a + a_rest) f
__device__ __forceinline__ void sub_product(float &s, float &c, float a, float a_rest, float f)
{
    if (a == 0.0f) // a sum without a token of its sign stays out: 0 * infinity is no number
        return;
    const float v = __fmul_rn(-a, f);
    add_to(s, c, v);
    if (fabsf(v) < INFINITY)
        c += fmaf(-a, f, -v) - a_rest * f;
}

// A sequence's saved pair and its share of the totals.
__device__ __forceinline__ void finish(const PolicyParams &p, int s, const SegSums &x, Totals &tot)
{
    const float n = (float)x.count;
    float l = x.c, l_rest = fabsf(x.c) < INFINITY ? x.c_rest : 0.0f, g = 0.0f;
    unsigned long long clipped = x.clipped;
    if (p.by_seg && x.count) {
        float a = x.a, a_rest = fabsf(x.a) < INFINITY ? x.a_rest : 0.0f;
        unsigned long long neg = x.clipped, zero = x.zero;
        float b = x.b, b_rest = fabsf(x.b) < INFINITY ? x.b_rest : 0.0f;
        if (!p.adv_token) { // one advantage: no sum
            const float A = __ldg(p.adv + s), An = A * n, rest = fabsf(An) < INFINITY ? fmaf(A, n, -An) : 0.0f;
            a = A < 0.0f ? 0.0f : An;
            a_rest = A < 0.0f ? 0.0f : rest;
            b = A < 0.0f ? An : 0.0f;
            b_rest = A < 0.0f ? rest : 0.0f;
            neg = A < 0.0f ? x.count : 0ull;
            zero = A == 0.0f ? x.count : 0ull;
        }
        const float c = whole(x.c, x.c_rest);
        // the mean in two floats: it is compared with the borders
        const float mean = __fdiv_rn(c, n);
        float rest = 0.0f;
        if (fabsf(c) < INFINITY) {
            const float lost = __fadd_rn(__fsub_rn(x.c, c), x.c_rest);
            rest = __fdiv_rn(__fadd_rn(fmaf(-mean, n, c), lost), n);
        }
        const bool hi = above(mean, rest, p.log_high), lo = below(mean, rest, p.log_low);
        const bool du = above(mean, rest, p.log_dual);
        const float ratio = ratio_of(mean, rest);
        // What the ratio multiplies, rounded after the two signs have met: their sums grow with n, their
        // difference with its root (each sum rounded first, gradients of 2 million tokens were off by 1e-5).
        float live = hi ? 0.0f : a, live_rest = hi ? 0.0f : a_rest;
        if (!lo && !du) {
            add_to(live, live_rest, b);
            live_rest += b_rest;
        }
        live = whole(live, live_rest);
        l = l_rest = 0.0f;
        sub_product(l, l_rest, live, 0.0f, ratio);
        if (hi)
            sub_product(l, l_rest, a, a_rest, p.high);
        if (lo || du)
            sub_product(l, l_rest, b, b_rest, lo ? p.low : p.dual);
        clipped = (hi ? x.count - neg - (ratio < INFINITY ? zero : 0ull) : 0ull) + (lo || du ? neg : 0ull);
        g = live != 0.0f ? __fdiv_rn(live * ratio, n) : 0.0f;
    }
    reinterpret_cast<float2 *>(p.save)[s] = make_float2(n, g);
    if (x.count) {
        Totals t = {l, l_rest, x.kl, x.kl_rest, clipped, x.count, 1ull};
        if (p.mean == JETQ_POLICY_MEAN_SEGMENTS) {
            t.l = __fdiv_rn(whole(l, l_rest), n);
            t.kl = __fdiv_rn(whole(x.kl, x.kl_rest), n);
            t.l_rest = t.kl_rest = 0.0f;
        }
        add_totals(tot, t);
    }
}

__device__ __forceinline__ void write_out(const PolicyParams &p, const Totals &t)
{
    float f = p.scale;
    if (p.mean != JETQ_POLICY_SUM) {
        const unsigned long long by = p.mean == JETQ_POLICY_MEAN_SEGMENTS ? t.segs : t.tokens;
        f = by ? __fdiv_rn(f, (float)by) : 0.0f;
    }
    const float l = f * whole(t.l, t.l_rest), kl = f * whole(t.kl, t.kl_rest);
    p.out[0] = p.ref ? fmaf(p.kl, kl, l) : l;
    p.out[1] = l;
    p.out[2] = kl;
    p.out[3] = (float)t.clipped;
    p.out[4] = (float)t.tokens;
    p.out[5] = (float)t.segs;
}

// A sequence's lanes in the join; pieces above which the whole CTA takes it.  In a graph, both directions, bounds of
// 16, 64 and 256 pieces: 1000003 tokens in 24 sequences 27, 29 and 41 us, 524288 in 512 25, 23 and 23, 4194304 in 1
// 53 (256 without a bound).
constexpr int kLanesSeg = 4, kLong = 64;

template <int THREADS>
struct JoinShared {
    SegSums seg[THREADS / 32];
    Totals tot[THREADS / 32];
    int longs[THREADS / kLanesSeg], num_longs;
    bool last;
};

// The CTA's sum of `t`, in all lanes of warp 0.
template <int THREADS>
__device__ __forceinline__ void cta_totals(Totals &t, JoinShared<THREADS> &sh)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarpsCta = THREADS / 32;
    warp_totals(t, 32);
    if (lane == 0)
        sh.tot[warp] = t;
    __syncthreads();
    if (warp == 0) {
        t = lane < kWarpsCta ? sh.tot[lane] : Totals{};
        warp_totals(t, 32);
    }
}

// Sequences [first, end) by a CTA: their saved pairs, and the totals in warp 0.
template <int THREADS>
__device__ __forceinline__ Totals join_segments(const PolicyParams &p, int64_t first, int64_t end,
                                                JoinShared<THREADS> &sh)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = threadIdx.x % kLanesSeg;
    Totals tot = {};
    const int64_t span = (int64_t)p.chunk * kWindow;
    auto range = [&](int64_t s, int64_t &w0, int64_t &w1) { // chunks of sequence s
        int64_t b = p.seg ? __ldg(p.seg + s) : 0, e = p.seg ? __ldg(p.seg + s + 1) : p.n;
        b = b < 0 ? 0 : b;
        e = e > p.n ? p.n : e;
        w0 = b / span;
        w1 = e > b ? (e - 1) / span + 1 : w0;
    };
    for (int64_t s0 = first; s0 < end; s0 += THREADS / kLanesSeg) {
        if (threadIdx.x == 0)
            sh.num_longs = 0;
        __syncthreads();
        const int64_t s = s0 + threadIdx.x / kLanesSeg;
        int64_t w0 = 0, w1 = 0;
        if (s < end)
            range(s, w0, w1);
        const bool is_long = w1 - w0 > kLong;
        if (is_long && sub == 0)
            sh.longs[atomicAdd(&sh.num_longs, 1)] = (int)s;
        SegSums x;
        x.clear();
        if (!is_long) {
#pragma unroll 2
            for (int64_t w = w0 + sub; w < w1; w += kLanesSeg)
                x.add(p.pieces + (w + s), p.adv_sums);
        }
#pragma unroll
        for (int o = kLanesSeg / 2; o; o >>= 1)
            x.add_lane(o, p.adv_sums);
        if (s < end && !is_long && sub == 0)
            finish(p, (int)s, x, tot);
        __syncthreads();
        const int many = sh.num_longs;
        // in the order of the sequences, whatever the order in which they were listed
        int after = -1;
        for (int i = 0; i < many; ++i) {
            int which = 0x7FFFFFFF;
            for (int j = 0; j < many; ++j)
                if (sh.longs[j] > after)
                    which = min(which, sh.longs[j]);
            after = which;
            range(which, w0, w1);
            x.clear();
#pragma unroll 4
            for (int64_t w = w0 + threadIdx.x; w < w1; w += THREADS)
                x.add(p.pieces + (w + which), p.adv_sums);
#pragma unroll
            for (int o = 16; o; o >>= 1)
                x.add_lane(o, p.adv_sums);
            if (lane == 0)
                sh.seg[warp] = x;
            __syncthreads();
            if (warp == 0) {
                if (lane < THREADS / 32)
                    x = sh.seg[lane];
                else
                    x.clear();
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    x.add_lane(o, p.adv_sums);
                if (lane == 0)
                    finish(p, which, x, tot);
            }
            __syncthreads();
        }
        __syncthreads();
    }
    cta_totals<THREADS>(tot, sh);
    return tot;
}

constexpr int kSmallThreads = 1024, kJoinThreads = 256;
// Sequences that one CTA joins.  One launch in place of two, which is what a call costs: 1531 tokens in 8 sequences
// 42 us both directions (45 with the two kernels; in a graph 14.5 and 12.5).  Its warps walk the sequences of their
// windows alone: 4096 tokens in 500 sequences are done after 72 us (64), in 4000 after 232 (161).
constexpr int kSmallSegs = 256;

template <bool BY_SEG>
__global__ void __launch_bounds__(32 * kWarps, 3) k_policy_pieces(const PolicyParams p)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t chunk = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *p.ticket = 0;
    if (chunk * p.chunk < p.windows)
        sum_pieces<BY_SEG>(p, chunk, threadIdx.x & 31);
}

// The last CTA to finish adds the CTAs' totals.
__global__ void __launch_bounds__(kJoinThreads) k_policy_join(const PolicyParams p)
{
    __shared__ JoinShared<kJoinThreads> sh;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t first = (int64_t)blockIdx.x * p.segs_cta;
    Totals t = join_segments<kJoinThreads>(p, first, min(first + p.segs_cta, (int64_t)p.nseg), sh);
    if (gridDim.x > 1) {
        if (threadIdx.x == 0) {
            p.part[blockIdx.x] = t;
            __threadfence();
            sh.last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
        }
        __syncthreads();
        if (!sh.last)
            return;
        __threadfence();
        t = Totals{};
        for (unsigned i = threadIdx.x; i < gridDim.x; i += kJoinThreads) {
            Totals o;
            const float4 f = __ldcg(reinterpret_cast<const float4 *>(p.part + i));
            const ulonglong2 u = __ldcg(reinterpret_cast<const ulonglong2 *>(p.part + i) + 1);
            o.l = f.x;
            o.l_rest = f.y;
            o.kl = f.z;
            o.kl_rest = f.w;
            o.clipped = u.x;
            o.tokens = u.y;
            o.segs = __ldcg(&p.part[i].segs);
            add_totals(t, o);
        }
        cta_totals<kJoinThreads>(t, sh);
    }
    if (threadIdx.x == 0)
        write_out(p, t);
}

// Both steps by one CTA, a window a warp.
template <bool BY_SEG>
__global__ void __launch_bounds__(kSmallThreads) k_policy_small(const PolicyParams p)
{
    __shared__ JoinShared<kSmallThreads> sh;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    if ((threadIdx.x >> 5) < p.windows) // chunks of one window
        sum_pieces<BY_SEG>(p, threadIdx.x >> 5, threadIdx.x & 31);
    __syncthreads(); // the pieces are there for the whole CTA
    const Totals t = join_segments<kSmallThreads>(p, 0, p.nseg, sh);
    if (threadIdx.x == 0)
        write_out(p, t);
}

template <bool BY_SEG>
__global__ void __launch_bounds__(32 * kWarps, 3) k_policy_bwd(const PolicyParams p)
{
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t w0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * p.chunk;
    if (w0 >= p.windows)
        return;
    const int64_t w1 = min(w0 + p.chunk, p.windows);
    Tokens tk, next;
    next.load(p, w0 * kWindow, lane);
    float scale = p.scale;
    if (p.mean == JETQ_POLICY_MEAN_TOKENS)
        scale = __fdiv_rn(scale, __ldcg(p.out + 4));
    else if (p.mean == JETQ_POLICY_MEAN_SEGMENTS)
        scale = __fdiv_rn(scale, __ldcg(p.out + 5));
    if (p.dloss)
        scale *= __ldg(p.dloss);
    Walker walk;
    walk.start(p, w0 * kWindow, lane);
    for (int64_t w = w0; w < w1; ++w) {
        tk = next;
        if (w + 1 < w1)
            next.load(p, (w + 1) * kWindow, lane);
        float d[kSlots], e[kSlots], r[kSlots], kl[kSlots], g[kSlots];
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            two_diff(tk.y[k], tk.x[k], d[k], e[k]);
            r[k] = BY_SEG ? 0.0f : ratio_of(d[k], e[k]);
            kl[k] = p.ref ? p.kl * kl_slope(tk.x[k] - tk.z[k]) : 0.0f;
            g[k] = 0.0f;
        }
        const int64_t t0 = w * kWindow, t1 = min(t0 + kWindow, p.n);
        walk.window<true>(p, t0, t1, false, lane, [&](int, int64_t from, int64_t to, float A_seg, float2 seg, bool) {
            const int lo = (int)(from - t0) - lane, hi = (int)(to - t0) - lane;
            const float f = p.mean == JETQ_POLICY_MEAN_SEGMENTS ? __fdiv_rn(scale, seg.x) : scale;
#pragma unroll
            for (int k = 0; k < kSlots; ++k)
                if (tk.on[k] && 32 * k >= lo && 32 * k < hi) {
                    float v = seg.y;
                    if (!BY_SEG) {
                        const float A = p.adv_token ? tk.A[k] : A_seg;
                        float bound;
                        v = clip(p, A, d[k], e[k], bound) ? 0.0f : A * r[k];
                    }
                    g[k] = f * (v + kl[k]);
                }
        });
        float *out = p.dnll + t0 + lane;
        const int left = (int)(t1 - t0) - lane;
#pragma unroll
        for (int k = 0; k < kSlots; ++k)
            if (32 * k < left)
                out[32 * k] = g[k];
    }
}

int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

constexpr int kMaxChunk = 32; // a lane's FP32 sums are of 128 tokens at most
constexpr int kWarpsSm = 24; // warps an SM that share the windows: what its registers hold

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
    p.adv_sums = p.by_seg && p.adv_token;
    const int64_t warps = (int64_t)sm_count() * kWarpsSm;
    const int64_t chunk = ceil_div(p.windows, warps);
    p.chunk = (int)(chunk < kMaxChunk ? chunk : kMaxChunk);
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

// Sequences a CTA of the join: about 128 pieces, in as many CTAs as that makes.
int segs_a_cta(int64_t chunks, int64_t nseg)
{
    const int64_t most = kJoinThreads / kLanesSeg, s = 128 * nseg / (chunks + nseg);
    return (int)(s < 1 ? 1 : s > most ? most : s);
}

} // namespace

// Enough for chunks of one window, whatever the device: a chunk's size only takes pieces away.
size_t policy_loss_workspace(int64_t n, int64_t nseg)
{
    const int64_t windows = ceil_div(n, kWindow);
    return 16 + (size_t)(windows + nseg) * sizeof(Piece) + (size_t)nseg * sizeof(Totals);
}

cudaError_t launch_policy_fwd(const PolicyArgs &a, cudaStream_t st)
{
    PolicyParams p = params_of(a);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    p.ticket = reinterpret_cast<unsigned *>(ws);
    p.pieces = reinterpret_cast<Piece *>(ws + 16);
    const int64_t chunks = ceil_div(p.windows, p.chunk);
    p.part = reinterpret_cast<Totals *>(ws + 16 + (size_t)(chunks + p.nseg) * sizeof(Piece));
    if (p.windows <= kSmallThreads / 32 && p.chunk == 1 && p.nseg <= kSmallSegs)
        return p.by_seg ? launch_pdl(k_policy_small<true>, dim3(1), dim3(kSmallThreads), 0, st, p)
                        : launch_pdl(k_policy_small<false>, dim3(1), dim3(kSmallThreads), 0, st, p);
    p.segs_cta = segs_a_cta(chunks, p.nseg);
    const dim3 grid((unsigned)ceil_div(p.windows, (int64_t)kWarps * p.chunk)), block(32 * kWarps);
    const cudaError_t e = p.by_seg ? launch_pdl(k_policy_pieces<true>, grid, block, 0, st, p)
                                   : launch_pdl(k_policy_pieces<false>, grid, block, 0, st, p);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(k_policy_join, dim3((unsigned)ceil_div(p.nseg, p.segs_cta)), dim3(kJoinThreads), 0, st, p);
}

cudaError_t launch_policy_bwd(const PolicyArgs &a, cudaStream_t st)
{
    const PolicyParams p = params_of(a);
    const dim3 grid((unsigned)ceil_div(p.windows, (int64_t)kWarps * p.chunk)), block(32 * kWarps);
    return p.by_seg ? launch_pdl(k_policy_bwd<true>, grid, block, 0, st, p)
                    : launch_pdl(k_policy_bwd<false>, grid, block, 0, st, p);
}

} // namespace jetq
