// route_fwd.cuh -- the forward kernel of the router: topk experts and their
// gates from a [tokens, experts] score matrix (softmax or sigmoid scores, a
// bias that takes part in the choice only, groups of experts of which the best
// stay open, renormalised and scaled gates, tokens per expert).  One
// translation unit per type of logits instantiates it.
//
// L lanes of a warp share a row (8 up to 256 experts, so that a warp orders
// four rows at once), each with V of its values.  The choice is k rounds of
// a maximum over the lanes; what decides it is an order in which ties go to
// the lower expert, so the result is a function of the row alone.
#pragma once
#include "dd.cuh"
#include "route.cuh"

namespace kosmos {

namespace {

constexpr int ROUTE_WARPS = 8;
constexpr int ROUTE_THREADS = ROUTE_WARPS * 32;
// Blocks per SM that the registers are made to fit: a lane with up to eight
// values runs as well in 64 (40009 x 60: 9.8 us, 11.0 us in 80), one with 16 or
// 32 in 80 (32768 x 256: 32 us, 38 us in 128).
constexpr int route_blocks(int V) { return V <= 8 ? 4 : 3; }
#ifndef SMT
#define SMT 20
#endif
constexpr int SMALL_T = SMT;         // tokens per SM up to which a warp takes one row
constexpr int SLOTS = 16;            // candidates that a row can have

template <int L> constexpr uint32_t row_lanes() { return L == 32 ? FULL : (1u << L) - 1u; }

// The gates of a row's chosen experts, N per lane (logit x, open or not).
// m, z: the row's maximum and sum of exponentials (softmax without renorm).
// Ratios of p are taken relative to the largest chosen one, so that small
// scores keep their precision.
template <int L, int N>
__device__ __forceinline__ void route_gates(const RouteParams &p, const float *x, const bool *open, float m, float z,
                                            float *g) {
    if (!p.renorm) {
#pragma unroll
        for (int h = 0; h < N; ++h)
            g[h] = !open[h] ? 0.f
                            : p.scale * (p.score == KOSMOS_SCORE_SOFTMAX ? expf(x[h] - m) / z : 1.0f / (1.0f + expf(-x[h])));
        return;
    }
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int h = 0; h < N; ++h) top = fmaxf(top, open[h] ? x[h] : -INFINITY);
    top = row_max<L>(top);
    if (p.score == KOSMOS_SCORE_SIGMOID) top = fminf(top, 0.f);
#pragma unroll
    for (int h = 0; h < N; ++h) {
        g[h] = 0.f;
        if (open[h]) {
            if (p.score == KOSMOS_SCORE_SOFTMAX) g[h] = expf(x[h] - top);
            else g[h] = x[h] > 0.f ? 1.0f / (1.0f + expf(-x[h])) : expf(x[h] - top) / (1.0f + expf(x[h]));
        }
        sum += g[h];
    }
    sum = row_sum<L>(sum);
#pragma unroll
    for (int h = 0; h < N; ++h) g[h] = open[h] ? p.scale * (g[h] / sum) : 0.f;
}

// ------------------------------------------------------------ fp32 choice
// How a kernel orders a row's experts: without a bias by their logits, which
// the scores rise with; else by s = p + bias in fp32.  Rows in which two
// neighbours in the order, or the groups either side of the border, are closer
// than the scores' rounding error are chosen again in 64 bits.
enum RouteMode : int { BY_LOGIT = 0, BY_SIGMOID = 1, BY_SOFTMAX = 2 };

// Order-preserving map of floats to unsigned integers (-0 as +0).  Closed
// experts have the key of -inf, and so have the places beyond E, which
// come last of all because ties go to the lower expert.
constexpr uint32_t KEY_NONE = 0u, KEY_CLOSED = 0x007FFFFFu;
__device__ __forceinline__ uint32_t float_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// p in fp32 (rz = 1 / z): x = -inf gives 0.
__device__ __forceinline__ float fast_sigmoid(float x) { return rcp(1.0f + ex2(-LOG2E * x)); }
__device__ __forceinline__ float fast_softmax(float x, float m, float rz) { return ex2(LOG2E * (x - m)) * rz; }

// Bounds on the distance between an fp32 score and the 64-bit one.  Sigmoid:
// the exponential is off by 2 + 1.2 |x| steps of 2^-23 (argument and result),
// which p (1 - p) brings under 6e-8; sum and reciprocal 3e-7 p; the bias'
// addition 6e-8 |s|.  Softmax: e^-y of a term y below the maximum is off by
// (2.5 + 1.7 y) steps, at most 3e-7 of the largest term; the row's sum and its
// reciprocal by 5e-6 (its terms' errors weigh at most ln 1024, and there are
// 37 additions); the bias as above.
__device__ __forceinline__ float score_error(bool softmax, float s, float p, float rz) {
    return (softmax ? 3e-7f * rz + 5e-6f * p : 5e-7f) + 1.2e-7f * fabsf(s);
}

// The same for scores in double words.
__device__ __forceinline__ float score_error_dd(float s) { return 5e-11f + 1e-13f * fabsf(s); }
__device__ __forceinline__ dd score_dd(bool softmax, float x, float b, float m, dd rz) {
    if (!softmax) return dd_add(dd_sigmoid(x), b);
    return dd_add(dd_mul(dd_exp(two_sum(x, -m)), rz), b);
}
__device__ __forceinline__ float difference(dd a, dd b) { return (a.hi - b.hi) + (a.lo - b.lo); }

// A lane's best D keys in order.  A key's low bits hold the expert (as
// MASK - e: the lower expert first), so keys differ and a maximum tells
// whose it is; a value's own low bits are lost, which matters to fp32 values
// only (a bf16 or fp16 value has at least 13 zero bits).  A lane that has given
// its list away makes the next one: of eight choices from eight lanes some lane
// gives four in 13 rows of 100 and five in 2, from 32 lanes two in 60, four
// in 0.2.
template <int L, int V> struct Best {
    static constexpr int D = L == 32 && V > 4 ? 3 : V > 8 ? 5 : 4;
    static constexpr uint32_t MASK = L * V - 1;
    uint32_t k[D];
    // low: MASK - e for a lane's v = 0; the others' differ from it in v's bits alone
    static __device__ __forceinline__ uint32_t key_of(float f, uint32_t low, uint32_t v_bits) {
        return ((float_key(f) & ~MASK) | low) ^ v_bits;
    }
    static __device__ __forceinline__ uint32_t closed(uint32_t key) { return (key & MASK) | (KEY_CLOSED & ~MASK); }
    static __device__ __forceinline__ int expert(uint32_t key) { return static_cast<int>(MASK - (key & MASK)); }
    static __device__ __forceinline__ bool is_open(uint32_t key) { return (key | MASK) > KEY_CLOSED; }
    __device__ __forceinline__ void insert(uint32_t x) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const uint32_t hi = max(k[d], x);
            x = min(k[d], x);
            k[d] = hi;
        }
    }
    __device__ __forceinline__ void fill(const uint32_t *key) {
#pragma unroll
        for (int d = 0; d < D; ++d) k[d] = KEY_NONE;
#pragma unroll
        for (int v = 0; v < V; ++v) insert(key[v]);
    }
    __device__ __forceinline__ void fill_below(const uint32_t *key, uint32_t limit) {
#pragma unroll
        for (int d = 0; d < D; ++d) k[d] = KEY_NONE;
#pragma unroll
        for (int v = 0; v < V; ++v) insert(key[v] < limit ? key[v] : KEY_NONE);
    }
};

// ---------------------------------------------------------- 64-bit choice
// 64-bit keys, ordered like the doubles; NaN and -inf are closed.
constexpr uint64_t KEY64_CLOSED = 0x000FFFFFFFFFFFFFull;
__device__ __forceinline__ uint64_t double_key(double s) {
    if (!(s > -INFINITY)) return KEY64_CLOSED;
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(s + 0.0));
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double key_double(uint64_t k) {
    return __longlong_as_double(static_cast<long long>(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}
__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(FULL, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(FULL, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}

// One row, by the whole warp, whose experts are chosen by their 64-bit selection
// scores, from the logits to the outputs.  fp64 instructions are slow here (two
// lanes a cycle) and the row is waited for, so a score is computed in 64 bits only when
// it comes up: until then its key is an upper bound, the fp32 score and its
// error.  Lane l holds the experts l + 32 v.
template <int VR> struct Row64 {
    uint64_t key[VR];
    float x[VR];
    uint32_t exact = 0;  // one bit per value
    double m = 0.0, z = 1.0;

    __device__ __forceinline__ double score(const RouteParams &p, float xv, int e) const {
        const double d = xv;
        const double q = p.score == KOSMOS_SCORE_SOFTMAX ? exp(d - m) / z : 1.0 / (1.0 + exp(-d));
        return p.bias != nullptr ? q + static_cast<double>(p.bias[e]) : q;
    }
    // every lane makes one of its wanted values exact
    __device__ __forceinline__ void sharpen(const RouteParams &p, int lane, uint32_t want) {
        while (__any_sync(FULL, want != 0u)) {
            const int at = __ffs(want) - 1;
            float xv = 0.f;
#pragma unroll
            for (int v = 0; v < VR; ++v)
                if (v == at) xv = x[v];
            const uint64_t k = at >= 0 ? double_key(score(p, xv, lane + 32 * at)) : 0;
#pragma unroll
            for (int v = 0; v < VR; ++v)
                if (v == at) key[v] = k;
            if (at >= 0) exact |= 1u << at;
            want &= want - 1u;
        }
    }
    // the warp's best key among experts e0 <= e < e1 that are not in skip (one
    // bit per value); its lane gets its place, the others -1
    __device__ __forceinline__ uint64_t best(int lane, int e0, int e1, uint32_t skip, int &at) const {
        uint64_t k = 0;
        at = -1;
#pragma unroll
        for (int v = 0; v < VR; ++v) {
            const int e = lane + 32 * v;
            if (e >= e0 && e < e1 && !((skip >> v) & 1u) && key[v] > k) { k = key[v]; at = v; }
        }
        const uint64_t b = warp_max_key(k);
        // ties: the lowest expert
        const uint32_t e = __reduce_min_sync(FULL, at >= 0 && k == b ? static_cast<uint32_t>(lane + 32 * at) : ~0u);
        if (at < 0 || static_cast<uint32_t>(lane + 32 * at) != e) at = -1;
        return b;
    }
};

template <typename T, int VR>
__device__ __noinline__ void route_row_f64(const RouteParams &p, int64_t t, int lane, int32_t *s_hist) {
    const T *row = static_cast<const T *>(p.logits) + t * p.ld;
    const bool softmax = p.score == KOSMOS_SCORE_SOFTMAX, by_logit = p.bias == nullptr;
    const bool scores = !by_logit || (p.GK < p.G && p.group_top == 2);
    Row64<VR> w;
    bool nan = false;
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < VR; ++v) {
        const int e = lane + 32 * v;
        w.x[v] = e < p.E ? to_f32(row[e]) : -INFINITY;
        nan = nan || w.x[v] != w.x[v] || (softmax && w.x[v] == INFINITY);
        w.x[v] = fmaxf(w.x[v], -INFINITY);  // NaN: closed
        top = fmaxf(top, w.x[v]);
    }
    nan = __any_sync(FULL, nan);
    float rz = 1.f;
    if (softmax && (scores || !p.renorm)) {
        top = row_max<32>(top);
        w.m = top;
        w.z = 0.0;
#pragma unroll
        for (int v = 0; v < VR; ++v)
            if (w.x[v] > -INFINITY) w.z += exp(static_cast<double>(w.x[v]) - w.m);
        w.z = row_sum<32>(w.z);
        rz = static_cast<float>(1.0 / w.z);
    }
#pragma unroll
    for (int v = 0; v < VR; ++v) {
        const int e = lane + 32 * v;
        w.key[v] = KEY64_CLOSED;
        if (w.x[v] > -INFINITY && scores) {
            const float q = softmax ? fast_softmax(w.x[v], top, rz) : fast_sigmoid(w.x[v]);
            const float s = q + (by_logit ? 0.f : p.bias[e]);
            if (s > -INFINITY) w.key[v] = double_key(static_cast<double>(s) + score_error(softmax, s, q, rz));
        } else if (w.x[v] > -INFINITY) {
            w.key[v] = double_key(static_cast<double>(w.x[v]));
        }
        // closed experts, infinite scores and logits are what they are
        if (!scores || w.key[v] == KEY64_CLOSED || w.key[v] == double_key(INFINITY)) w.exact |= 1u << v;
    }
    if (p.GK < p.G) {
        const int gs = p.E / p.G;
        double score = -INFINITY;  // lane g: the score of group g
        bool again = true;
        while (again) {  // until every group's best group_top values are exact
            uint32_t want = 0u;
            for (int g = 0; g < p.G; ++g) {
                int a1, a2 = -1;
                const uint64_t b1 = w.best(lane, g * gs, (g + 1) * gs, 0u, a1);
                double tt = key_double(b1);
                if (p.group_top == 2) {
                    const uint64_t b2 = w.best(lane, g * gs, (g + 1) * gs, a1 >= 0 ? 1u << a1 : 0u, a2);
                    if (b2 > KEY64_CLOSED) tt += key_double(b2);
                }
                if (lane == g) score = tt;
                if (a1 >= 0) want |= 1u << a1;
                if (a2 >= 0) want |= 1u << a2;
            }
            want &= ~w.exact;
            again = __any_sync(FULL, want != 0u);
            w.sharpen(p, lane, want);
        }
        int rank = 0;
        const uint64_t mine = double_key(score);
        for (int g = 0; g < p.G; ++g) {
            const uint64_t o = __shfl_sync(FULL, mine, g);
            rank += (o > mine || (o == mine && g < lane)) ? 1 : 0;
        }
        const uint32_t open = __ballot_sync(FULL, lane < p.G && rank < p.GK);
#pragma unroll
        for (int v = 0; v < VR; ++v) {
            const int e = lane + 32 * v;
            if (e < p.E && !((open >> (e / gs)) & 1u)) {
                w.key[v] = KEY64_CLOSED;
                w.exact |= 1u << v;
            }
        }
    }
    if (by_logit && scores) {  // the scores were the groups'
#pragma unroll
        for (int v = 0; v < VR; ++v)
            if (w.key[v] > KEY64_CLOSED) w.key[v] = double_key(static_cast<double>(w.x[v]));
        w.exact = ~0u;
    }
    int my_e = 0;
    bool my_open = false;
    uint32_t taken = 0u;
    for (int j = 0; j < p.k;) {
        int at;
        const uint64_t b = w.best(lane, 0, p.E, taken, at);
        if (__any_sync(FULL, at >= 0 && !((w.exact >> at) & 1u))) {
            // an upper bound came up: every lane makes the best of its own that is left exact
            uint64_t k = 0;
            uint32_t want = 0u;
#pragma unroll
            for (int v = 0; v < VR; ++v)
                if (!(((taken | w.exact) >> v) & 1u) && w.key[v] > k) { k = w.key[v]; want = 1u << v; }
            w.sharpen(p, lane, want);
            continue;
        }
        const int e = __reduce_max_sync(FULL, at >= 0 ? lane + 32 * at : 0);
        if (at >= 0) taken |= 1u << at;
        if (lane == j) { my_e = e; my_open = b > KEY64_CLOSED; }
        ++j;
    }
    const bool mine = lane < p.k;
    const float my_x = mine ? to_f32(row[my_e]) : 0.f;
    my_open = my_open && mine;
    float g;
    route_gates<SLOTS, 1>(p, &my_x, &my_open, static_cast<float>(w.m), static_cast<float>(w.z), &g);
    if (nan) g = NAN;
    if (mine) {
        p.idx[t * p.k + lane] = my_e;
        p.gate[t * p.k + lane] = g;
        if (p.counts != nullptr) atomicAdd(&s_hist[my_e], 1);
    }
}

// 1 / (sum of the row's exponentials) in double words, by the row's lanes.
template <typename T, int L, int V>
__device__ __noinline__ dd row_inverse_z(const T *row, int E, int l, bool vec, float m) {
    float x[V];
    Layout<T, L, V>::load(row, E, l, vec, x);
    dd z = {0.f, 0.f};
#pragma unroll 1
    for (int v = 0; v < V; ++v) {
        const float xv = x[0];  // shifted down one by one: no indexed registers
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) x[i] = x[i + 1];
        if (xv > -INFINITY) z = dd_add(z, dd_exp(two_sum(xv, -m)));
    }
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) {
        dd o;
        o.hi = __shfl_xor_sync(FULL, z.hi, d);
        o.lo = __shfl_xor_sync(FULL, z.lo, d);
        z = dd_add(z, o);
    }
    return dd_inverse(z);
}

// ------------------------------------------------------------------ groups
// The open groups of a warp's rows as bit masks.  The rows' values s (closed
// experts -inf) pass through shared memory, where a lane takes every L-th group;
// a group's stride there is four times an odd number, so that eight lanes'
// 16-byte loads meet in no bank, and its padding holds -inf.  Where the values'
// errors leave the border open, the groups' best values are looked up and the
// scores taken again in double words; near then tells that those leave it open
// too.
template <typename T, int L, int V, int MODE>
__device__ __forceinline__ uint32_t open_groups(const RouteParams &p, const T *row, const float *s, float *s_row, int l,
                                                int seg, float m, float rz, bool &near) {
    using Lay = Layout<T, L, V>;
    constexpr int NG = 32 / L;  // groups per lane
    const bool fours = p.gs % 4 == 0;
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; v += 4) {
        const int e = Lay::expert(l, v);
        if (fours) {
            if (e < p.E)
                *reinterpret_cast<float4 *>(s_row + e + ((e * p.gmul) >> 20) * (p.gsp - p.gs)) =
                    make_float4(s[v], s[v + 1], s[v + 2], s[v + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (e + i < p.E) s_row[e + i + (((e + i) * p.gmul) >> 20) * (p.gsp - p.gs)] = s[v + i];
        }
    }
    __syncwarp();
    const float err = MODE == BY_SOFTMAX ? 5.3e-6f * rz : 5e-7f;
    float sc[NG], ge[NG];
#pragma unroll
    for (int h = 0; h < NG; ++h) {
        const int g = h * L + l;
        float t1 = -INFINITY, t2 = -INFINITY;
        if (g < p.G)
            for (int i = 0; i < p.gs; i += 4) {
                const float4 q = *reinterpret_cast<const float4 *>(s_row + g * p.gsp + i);
                const float qq[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    t2 = fmaxf(t2, fminf(t1, qq[j]));
                    t1 = fmaxf(t1, qq[j]);
                }
            }
        ge[h] = err + 2.4e-7f * fabsf(t1);  // a score's error and its part of the sum's
        if (p.group_top == 2 && t2 != -INFINITY) {
            ge[h] += err + 2.4e-7f * fabsf(t2);
            t1 += t2;
        }
        sc[h] = t1;
    }
    uint32_t mask = 0u;
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int h = 0; h < NG; ++h) {
        if (h * L >= p.G) break;
        const int g = h * L + l;
        int rank = 0;
#pragma unroll
        for (int ho = 0; ho < NG; ++ho)
            for (int o = 0; o < L && ho * L + o < p.G; ++o) {
                const float v = __shfl_sync(FULL, sc[ho], seg * L + o);
                rank += (v > sc[h] || (v == sc[h] && ho * L + o < g)) ? 1 : 0;
            }
        const bool in = g < p.G && rank < p.GK;
        if (in) lo = fminf(lo, sc[h] - ge[h]);
        else if (g < p.G && sc[h] != -INFINITY) hi = fmaxf(hi, sc[h] + ge[h]);
        mask |= (__ballot_sync(FULL, in) >> (seg * L) & row_lanes<L>()) << (h * L % 32);
    }
    if (MODE == BY_LOGIT) return mask;
    hi = row_max<L>(hi);
    lo = -row_max<L>(-lo);
    const bool open_border = hi != -INFINITY && !(lo > hi);
    if (!__any_sync(FULL, open_border)) return mask;

    const dd drz = MODE == BY_SOFTMAX ? row_inverse_z<T, L, V>(row, p.E, l, p.vec, m) : dd{1.f, 0.f};
    bool bad = false;
    dd d[NG];
#pragma unroll
    for (int h = 0; h < NG; ++h) {
        const int g = h * L + l;
        d[h] = {-INFINITY, 0.f};
        if (g >= p.G) continue;
        float t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
        int e1 = 0, e2 = 0;
        for (int i = 0; i < p.gs; ++i) {
            const float v = s_row[g * p.gsp + i];
            if (v > t1) { t3 = t2; t2 = t1; e2 = e1; t1 = v; e1 = i; }
            else if (v > t2) { t3 = t2; t2 = v; e2 = i; }
            else t3 = fmaxf(t3, v);
        }
        if (t1 == -INFINITY) continue;
        // the values left out have to be below those taken
        const float next = p.group_top == 2 ? t3 : t2, least = p.group_top == 2 ? t2 : t1;
        if (next > -INFINITY && !(least - next > 2.f * (err + 1.2e-7f * fabsf(least)) + 2.4e-7f * fabsf(next))) bad = true;
        if (!(fabsf(t1) < INFINITY)) bad = true;
        e1 += g * p.gs;
        e2 += g * p.gs;
        d[h] = score_dd(MODE == BY_SOFTMAX, to_f32(row[e1]), p.bias != nullptr ? p.bias[e1] : 0.f, m, drz);
        float de = score_error_dd(d[h].hi);
        if (p.group_top == 2 && t2 > -INFINITY) {
            const dd q = score_dd(MODE == BY_SOFTMAX, to_f32(row[e2]), p.bias != nullptr ? p.bias[e2] : 0.f, m, drz);
            de += score_error_dd(q.hi);
            d[h] = dd_add(d[h], q);
        }
        ge[h] = de;
    }
    mask = 0u;
#pragma unroll
    for (int h = 0; h < NG; ++h) {
        if (h * L >= p.G) break;
        const int g = h * L + l;
        int rank = 0;
#pragma unroll
        for (int ho = 0; ho < NG; ++ho)
            for (int o = 0; o < L && ho * L + o < p.G; ++o) {
                const int src = seg * L + o;
                const dd v = {__shfl_sync(FULL, d[ho].hi, src), __shfl_sync(FULL, d[ho].lo, src)};
                const float ve = __shfl_sync(FULL, ge[ho], src);
                const int go = ho * L + o;
                const float by = difference(v, d[h]);  // NaN: neither has an open expert
                rank += (by > 0.f || (!(by < 0.f) && go < g)) ? 1 : 0;
                if (g < p.G && go != g && d[h].hi > -INFINITY && v.hi > -INFINITY && fabsf(by) <= ge[h] + ve) bad = true;
            }
        mask |= (__ballot_sync(FULL, g < p.G && rank < p.GK) >> (seg * L) & row_lanes<L>()) << (h * L % 32);
    }
    const uint32_t bads = __ballot_sync(FULL, bad);  // by every lane: rows differ in open_border
    near = open_border && (bads >> (seg * L) & row_lanes<L>()) != 0u;
    return mask;
}

// A warp takes 32 / L consecutive rows at a time.  A row's lanes hold its
// candidates, the j-th in lane j % L.  Candidates beyond the k-th are taken
// while their keys may hide a better score than the k-th's; the candidates are
// then ranked by their scores in full, and where the fp32 errors leave that
// open, in double words (errors 1e-11).  What those leave open goes to a list
// (LATER rows per warp) and is done at the end by route_row_f64: a call here
// would keep the loop's values out of registers.
constexpr int LATER = 16;

template <typename T, int L, int V, int MODE>
__global__ void __launch_bounds__(ROUTE_THREADS, route_blocks(V)) route_kernel(const __grid_constant__ RouteParams p) {
    constexpr bool EXACT = MODE == BY_LOGIT && sizeof(T) == 2;  // keys hold their values whole
    constexpr int R = 32 / L, N = L < SLOTS ? SLOTS / L : 1;    // rows of a warp, candidates of a lane
    using Lay = Layout<T, L, V>;
    using List = Best<L, V>;
    constexpr uint32_t MASK = List::MASK, ROW = row_lanes<L>();
    extern __shared__ int32_t s_mem[];
    __shared__ int64_t s_later[ROUTE_WARPS][LATER];
    int32_t *s_hist = s_mem;                                           // [E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int seg = lane / L, l = lane % L;
    float *s_row = reinterpret_cast<float *>(s_mem + p.hist_words) + (warp * R + seg) * p.row_words;
    for (int i = threadIdx.x; i < p.hist_words; i += blockDim.x) s_hist[i] = 0;
    if (p.GK < p.G)
        for (int i = l; i < p.row_words; i += L) s_row[i] = -INFINITY;
    __syncthreads();
    pdl_wait();
    const bool softmax = MODE == BY_SOFTMAX || (MODE == BY_LOGIT && p.score == KOSMOS_SCORE_SOFTMAX);
    const bool need_z = MODE == BY_SOFTMAX || (softmax && !p.renorm);
    const T *logits = static_cast<const T *>(p.logits);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * warps * R;
    int64_t t0 = (static_cast<int64_t>(blockIdx.x) * warps + warp) * R;
    while (t0 < p.T) {
        int later = 0;
        for (; t0 < p.T && later <= LATER - R; t0 += stride) {
            const bool live = t0 + seg < p.T;
            const T *row = logits + (live ? t0 + seg : t0) * p.ld;
            float s[V];
            const float odd = Lay::load(row, p.E, l, p.vec, s);
            bool nan = false;
            float m = 0.f, z = 1.f;
            if (__any_sync(FULL, odd != 0.f)) {  // NaN or infinite logits
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    nan = nan || s[v] != s[v] || (softmax && s[v] == INFINITY);
                    s[v] = fmaxf(s[v], -INFINITY);  // NaN: closed
                }
                nan = (__ballot_sync(FULL, nan) >> (seg * L) & ROW) != 0u;
            }
            if (softmax) {
                m = s[0];
#pragma unroll
                for (int v = 1; v < V; ++v) m = fmaxf(m, s[v]);
            }
            // s: what orders the experts and scores the groups; closed experts -inf
            float rz = 1.f;
            if (need_z) {
                m = row_max<L>(m);
                if (m == -INFINITY) m = 0.f;
                z = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float q = ex2(LOG2E * (s[v] - m));
                    z += q;
                    if (MODE == BY_SOFTMAX) s[v] = s[v] > -INFINITY ? q : -INFINITY;
                }
                z = row_sum<L>(z);
                rz = rcp(z);
            }
            uint32_t key[V];
            const uint32_t low = MASK - Lay::expert(l, 0);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = Lay::expert(l, v);
                if (MODE != BY_LOGIT) {
                    const float b = p.bias != nullptr && e < p.E ? __ldg(p.bias + e) : 0.f;
                    const float q = MODE == BY_SOFTMAX ? s[v] * rz : fast_sigmoid(s[v]);
                    s[v] = s[v] > -INFINITY ? fmaxf(q + b, -INFINITY) : -INFINITY;
                }
                key[v] = List::key_of(s[v], low, Lay::expert(0, v));
            }
            bool near = false;
            if (p.GK < p.G) {
                const uint32_t open = open_groups<T, L, V, MODE>(p, row, s, s_row, l, seg, m, rz, near);
                if (p.gs % 4 == 0) {  // four consecutive experts are of one group
#pragma unroll
                    for (int v = 0; v < V; v += 4)
                        if (!((open >> (((Lay::expert(l, v) * p.gmul) >> 20) & 31)) & 1u)) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) key[v + i] = List::closed(key[v + i]);
                        }
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (!((open >> (((Lay::expert(l, v) * p.gmul) >> 20) & 31)) & 1u)) key[v] = List::closed(key[v]);
                }
            }
            List list;
            list.fill(key);
            uint32_t my_key[N], best = KEY_NONE;
#pragma unroll
            for (int h = 0; h < N; ++h) my_key[h] = KEY_NONE;
            auto next = [&](bool take) {  // the row's next key, if it takes one
                const uint32_t b = row_max<L>(list.k[0]);
                if (take) {
                    best = b;
                    if (list.k[0] == b) {
#pragma unroll
                        for (int d = 0; d + 1 < List::D; ++d) list.k[d] = list.k[d + 1];
                        list.k[List::D - 1] = KEY_NONE;
                    }
                }
                if (List::D < V && __any_sync(FULL, list.k[0] == KEY_NONE)) {
                    if (list.k[0] == KEY_NONE) list.fill_below(key, best);  // what is left of a row is below its best
                }
            };
            auto put = [&](int j) {
#pragma unroll
                for (int h = 0; h < N; ++h)
                    if (j == h * L + l) my_key[h] = best;
            };
#pragma unroll 1
            for (int j = 0; j < p.k; ++j) {
                next(true);
                put(j);
            }
            int most = p.k;  // candidates of the longest row
            if (!EXACT && p.k < p.E) {
                // the least key that may hide a score as large as the k-th's (its value is at
                // least its key's): equal but for the expert, or within twice the error
                uint32_t least = best & ~MASK;
                if (MODE != BY_LOGIT) {
                    const float sk = key_float(least);
                    least = float_key(sk - 2.f * score_error(MODE == BY_SOFTMAX, sk, rz, rz)) & ~MASK;
                }
                const bool any_open = List::is_open(best);
                next(true);
                int n = p.k;
                bool more = any_open && best >= least && List::is_open(best);
                while (__any_sync(FULL, more && n < SLOTS && n + 1 < p.E)) {
                    const bool take = more && n < SLOTS && n + 1 < p.E;
                    if (take) put(n++);
                    next(take);
                    more = any_open && best >= least && List::is_open(best);
                }
                near = near || more;
                most = __reduce_max_sync(FULL, n);
            }
            // ---- candidates
            float my_x[N], my_g[N];
            int my_e[N], rank[N];
            bool my_open[N];
#pragma unroll
            for (int h = 0; h < N; ++h) {
                const bool mine = my_key[h] != KEY_NONE;
                my_g[h] = 0.f;
                my_open[h] = mine && List::is_open(my_key[h]);
                my_e[h] = mine ? List::expert(my_key[h]) : 0;
                rank[h] = mine ? h * L + l : p.k;
                my_x[h] = 0.f;
                if (h * L >= most) continue;
                if (EXACT) my_x[h] = key_float((my_key[h] & 0x80000000u) ? my_key[h] & ~MASK : my_key[h] | MASK);
                else my_x[h] = to_f32(row[my_e[h]]);
            }
            if (!EXACT) {
                // ranked by the score in full; equal scores keep the keys' order,
                // which is that of the experts
                float my_s[N], my_b[N], my_err[N];
                bool close = false;
#pragma unroll
                for (int h = 0; h < N; ++h) {
                    my_s[h] = -INFINITY;
                    my_b[h] = my_err[h] = 0.f;
                    if (h * L >= most) continue;
                    my_b[h] = MODE != BY_LOGIT && p.bias != nullptr ? __ldg(p.bias + my_e[h]) : 0.f;
                    const float q = MODE == BY_SOFTMAX ? fast_softmax(my_x[h], m, rz) : fast_sigmoid(my_x[h]);
                    my_s[h] = !my_open[h] ? -INFINITY : MODE == BY_LOGIT ? my_x[h] : q + my_b[h];
                    my_err[h] = MODE == BY_LOGIT || !my_open[h] ? 0.f : score_error(MODE == BY_SOFTMAX, my_s[h], q, rz);
                }
                // in order already, as the keys are, unless some neighbours are not
                // apart: compared with the next slot's score
                bool apart = most <= L;
                if (most <= L) {
                    const float s2 = __shfl_down_sync(FULL, my_s[0], 1);
                    const float err2 = MODE == BY_LOGIT ? 0.f : __shfl_down_sync(FULL, my_err[0], 1);
                    apart = l >= most - 1 || l == L - 1 || s2 == -INFINITY || my_s[0] - s2 > my_err[0] + err2;
                }
                if (!__all_sync(FULL, apart)) {
#pragma unroll
                    for (int h = 0; h < N; ++h)
                        if (my_key[h] != KEY_NONE) rank[h] = 0;
#pragma unroll
                    for (int ho = 0; ho < N; ++ho)
                        for (int o = 0; o < L && ho * L + o < most; ++o) {
                            const float so = __shfl_sync(FULL, my_s[ho], seg * L + o);
#pragma unroll
                            for (int h = 0; h < N; ++h) {
                                const int me = h * L + l, it = ho * L + o;
                                rank[h] += (so > my_s[h] || (so == my_s[h] && it < me)) ? 1 : 0;
                                // a pair within its errors: the wider one's is at least half of their sum
                                if (MODE != BY_LOGIT)
                                    close = close || (it != me && fabsf(so - my_s[h]) <= 2.f * my_err[h]);
                            }
                        }
                }
                if (MODE != BY_LOGIT && __any_sync(FULL, close)) {
                    const dd drz = MODE == BY_SOFTMAX ? row_inverse_z<T, L, V>(row, p.E, l, p.vec, m) : dd{1.f, 0.f};
                    dd my_d[N];
#pragma unroll
                    for (int h = 0; h < N; ++h) {
                        my_d[h] = {-INFINITY, 0.f};
                        if (my_open[h]) {
                            if (fabsf(my_b[h]) < INFINITY) my_d[h] = score_dd(MODE == BY_SOFTMAX, my_x[h], my_b[h], m, drz);
                            else near = true;
                        }
                        if (my_key[h] != KEY_NONE) rank[h] = 0;
                    }
#pragma unroll
                    for (int ho = 0; ho < N; ++ho)
                        for (int o = 0; o < L && ho * L + o < most; ++o) {
                            const int src = seg * L + o;
                            const dd so = {__shfl_sync(FULL, my_d[ho].hi, src), __shfl_sync(FULL, my_d[ho].lo, src)};
                            const float xo = __shfl_sync(FULL, my_x[ho], src), bo = __shfl_sync(FULL, my_b[ho], src);
#pragma unroll
                            for (int h = 0; h < N; ++h) {
                                const int me = h * L + l, it = ho * L + o;
                                const float by = difference(so, my_d[h]);  // NaN: neither is open
                                rank[h] += (by > 0.f || (!(by < 0.f) && it < me)) ? 1 : 0;
                                // the same logit and bias are a tie in 64 bits too
                                if (my_open[h] && so.hi > -INFINITY && fabsf(by) <= 2.f * score_error_dd(my_d[h].hi) &&
                                    !(xo == my_x[h] && bo == my_b[h]))
                                    near = true;
                            }
                        }
                }
                const uint32_t nb = __ballot_sync(FULL, near && live);
                for (int r = 0; nb != 0u && r < R; ++r) {
                    if (((nb >> (r * L)) & ROW) == 0u) continue;
                    if (lane == 0) s_later[warp][later] = t0 + r;
                    ++later;
#pragma unroll
                    for (int h = 0; h < N; ++h)
                        if (seg == r) rank[h] = p.k;  // not now
                }
            }
#pragma unroll
            for (int h = 0; h < N; ++h) my_open[h] = my_open[h] && rank[h] < p.k;
            if (N == 1 || most <= L) route_gates<L, 1>(p, my_x, my_open, m, z, my_g);
            else route_gates<L, N>(p, my_x, my_open, m, z, my_g);
#pragma unroll
            for (int h = 0; h < N; ++h)
                if (live && rank[h] < p.k) {
                    const int64_t at = (t0 + seg) * p.k + rank[h];
                    p.idx[at] = my_e[h];
                    p.gate[at] = nan ? NAN : my_g[h];
                    if (p.counts != nullptr) atomicAdd(&s_hist[my_e[h]], 1);
                }
        }
        __syncwarp();
        for (int i = 0; i < later; ++i) route_row_f64<T, (L * V) / 32>(p, s_later[warp][i], lane, s_hist);
        __syncwarp();
    }
    pdl_trigger();
    if (p.counts == nullptr) return;
    __syncthreads();
    if (gridDim.x == 1) {
        for (int i = threadIdx.x; i < p.E; i += blockDim.x) p.counts[i] = s_hist[i];
        return;
    }
    // blocks add their counts into the workspace (integers: any order gives
    // the same sums); the last one hands them out and leaves zeros
    for (int i = threadIdx.x; i < p.E; i += blockDim.x)
        if (s_hist[i] != 0) atomicAdd(&p.acc[i], s_hist[i]);
    __threadfence();
    __syncthreads();
    __shared__ int s_last;
    if (threadIdx.x == 0) s_last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    for (int i = threadIdx.x; i < p.E; i += blockDim.x) {
        p.counts[i] = __ldcg(&p.acc[i]);
        p.acc[i] = 0;
    }
    if (threadIdx.x == 0) *p.ticket = 0u;
}

template <typename T, int L, int V, int MODE>
kosmos_status launch_route_v(const RouteParams &q, int sms, cudaStream_t stream) {
    RouteParams p = q;
    constexpr int R = 32 / L, run = Layout<T, L, V>::W * sizeof(T);
    p.vec = p.E % Layout<T, L, V>::W == 0 && reinterpret_cast<uintptr_t>(p.logits) % run == 0 &&
            p.ld * static_cast<int64_t>(sizeof(T)) % run == 0;
    p.hist_words = p.counts != nullptr ? static_cast<int>(align_up(p.E, 4)) : 0;
    p.row_words = 0;
    if (p.GK < p.G) {
        p.gs = p.E / p.G;
        p.gmul = ((1 << 20) + p.gs - 1) / p.gs;  // e * gmul >> 20 = e / gs for e < 1024
        p.gsp = static_cast<int>(cdiv(p.gs, 4)) * 4;
        if (p.gsp % 8 == 0) p.gsp += 4;
        p.row_words = p.G * p.gsp;
    }
    // few tokens: small blocks, over as many SMs as there are warps of rows
    int warps = ROUTE_WARPS;
    while (warps > 1 && cdiv(p.T, R * warps) < sms) warps /= 2;
    // shared memory beyond 48 KB is not asked for: fewer warps per block instead
    while (warps > 1 && 4ll * (p.hist_words + warps * R * p.row_words) > 40960) warps /= 2;
    const size_t smem = 4ull * (p.hist_words + warps * R * p.row_words);
    int64_t blocks = cdiv(p.T, R * warps);
    const int64_t most = static_cast<int64_t>(route_blocks(V)) * (ROUTE_WARPS / warps) * sms;
    if (blocks > most) blocks = most;
    return launch_overlapped(&route_kernel<T, L, V, MODE>, static_cast<unsigned>(blocks), warps * 32, smem, stream, p);
}

template <typename T, int MODE> kosmos_status launch_route_m(const RouteParams &p, int sms, cudaStream_t stream) {
    // few tokens: a warp per row, whose latency counts
    if (p.T <= SMALL_T * static_cast<int64_t>(sms) && p.E <= 256)
        return p.E <= 128 ? launch_route_v<T, 32, 4, MODE>(p, sms, stream) : launch_route_v<T, 32, 8, MODE>(p, sms, stream);
    if (p.E <= 32) return launch_route_v<T, 8, 4, MODE>(p, sms, stream);
    if (p.E <= 64) return launch_route_v<T, 8, 8, MODE>(p, sms, stream);
    if (p.E <= 128) return launch_route_v<T, 8, 16, MODE>(p, sms, stream);
    if (p.E <= 256) return launch_route_v<T, 8, 32, MODE>(p, sms, stream);
    if (p.E <= 512) return launch_route_v<T, 16, 32, MODE>(p, sms, stream);
    return launch_route_v<T, 32, 32, MODE>(p, sms, stream);
}

}  // namespace

template <typename T> kosmos_status launch_route_t(const RouteParams &p, int sms, cudaStream_t stream) {
    if (p.bias == nullptr && !(p.GK < p.G && p.group_top == 2)) return launch_route_m<T, BY_LOGIT>(p, sms, stream);
    if (p.score == KOSMOS_SCORE_SIGMOID) return launch_route_m<T, BY_SIGMOID>(p, sms, stream);
    return launch_route_m<T, BY_SOFTMAX>(p, sms, stream);
}

}  // namespace kosmos
