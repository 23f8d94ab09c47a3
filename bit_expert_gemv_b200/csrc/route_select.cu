// Router: scores, selection bias, expert groups, top-K, gates.
//
//   s_e   = exp(l_e - max l) / sum exp(l - max l)   or   1 / (1 + exp(-l_e))
//   key_e = l_e without a bias (s grows with l, and the logit has no rounding),
//           s_e + b_e with one
//   group score = sum of the one or two largest (s_e + b_e) of the group; the
//           best `keep` groups stay
//   picks = the K largest keys of the experts that stay, ties to the lower index
//   gate  = scale * s (/ sum of the picks' s)
//
// A warp per token; lane l holds experts l, l + 32, ...  The order is that of
// the 64-bit values of these formulas.  It is taken in fp32 first, where every
// value is known to within a bound; a comparison that the bound leaves open is
// settled with the candidates' 64-bit values (refine), and where more than a
// few are in question the whole token is done in 64 bits (select_exact).
#include <type_traits>

#include "common.cuh"

namespace gale {
namespace {

struct SelectArgs {
    const void* logits;
    const float* bias;      // or null
    int32_t* ids;
    float* gates;
    int64_t ld;
    int B, E, K;
    int dtype, sigmoid, renorm;
    int groups, gsize, keep, gtop;
    float scale;
    int lanes_log2;         // 2^lanes_log2 lanes read a group's keys: as many as 32 / groups allows
    uint32_t gmagic;        // ceil(2^20 / gsize): e / gsize = e * gmagic >> 20 for e < 1024
};

constexpr float kMinusInf = -INFINITY;
constexpr float kFltMax = 3.402823466e38f;

// The logit as the formulas take it: NaN counts as -inf, +inf as the largest finite number.
__device__ __forceinline__ float clean(float l) {
    return fminf(fmaxf(l, kMinusInf), kFltMax);      // fmaxf drops a NaN
}
__device__ __forceinline__ float logit_at(const SelectArgs& a, int64_t t, int e) {
    return clean(load_as_f32(a.logits, a.dtype, t * a.ld + e));
}
// The logits of experts lane, lane + 32, ...; -inf past the last.
template <int V, bool FULL>
__device__ __forceinline__ void load_logits_of(const SelectArgs& a, int64_t t, int lane, float (&l)[V]) {
    if (a.dtype == GALE_F32) {
        const float* p = static_cast<const float*>(a.logits) + t * a.ld + lane;
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = FULL || lane + 32 * j < a.E ? __ldg(p + 32 * j) : kMinusInf;
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(a.logits) + t * a.ld + lane;
        uint16_t u[V];
#pragma unroll
        for (int j = 0; j < V; ++j) u[j] = FULL || lane + 32 * j < a.E ? __ldg(p + 32 * j) : 0;
        if (a.dtype == GALE_BF16) {
#pragma unroll
            for (int j = 0; j < V; ++j) l[j] = bf16_to_f32(u[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) l[j] = __half2float(__ushort_as_half(u[j]));
        }
        if (!FULL) {
#pragma unroll
            for (int j = 0; j < V; ++j) l[j] = lane + 32 * j < a.E ? l[j] : kMinusInf;
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = clean(l[j]);
}
template <int V>
__device__ __forceinline__ void load_logits(const SelectArgs& a, int64_t t, int lane, float (&l)[V]) {
    if (a.E == 32 * V) load_logits_of<V, true>(a, t, lane, l);
    else load_logits_of<V, false>(a, t, lane, l);
}
// s + b, -inf for a masked expert or a NaN
template <typename T>
__device__ __forceinline__ T with_bias(T s, float b, bool masked) {
    const T k = s + T(b);
    return masked || !(k == k) ? T(-INFINITY) : k;
}

// The float of order bits (the inverse of the function below).
__device__ __forceinline__ float order_value(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
// Unsigned order of a float: larger value, larger integer (-0 as +0); 0 is below every value's.
__device__ __forceinline__ uint32_t order_bits(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
// The warp's largest value, by one integer reduction (no NaN; -0 may come back as +0).
__device__ __forceinline__ float warp_max_f(float v) { return order_value(__reduce_max_sync(0xffffffffu, order_bits(v))); }

template <typename T>
__device__ __forceinline__ T warp_sum_t(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Group scores in 64 bits by warp-wide passes over the groups, four at a time
// (their shuffles overlap): lane g returns group g's.
template <int V>
__device__ __forceinline__ double group_scores(const SelectArgs& a, const double (&sel)[V], int lane) {
    double mine = -INFINITY;
    for (int g0 = 0; g0 < a.groups; g0 += 4) {
        double m1[4], m2[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int lo = (g0 + q) * a.gsize, hi = lo + a.gsize;
            m1[q] = m2[q] = -INFINITY;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = lane + 32 * j;
                const double v = e >= lo && e < hi && e < a.E ? sel[j] : -INFINITY;
                const double low = m1[q] > v ? v : m1[q];
                m1[q] = m1[q] > v ? m1[q] : v;
                m2[q] = m2[q] > low ? m2[q] : low;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const double u1 = __shfl_xor_sync(0xffffffffu, m1[q], o), u2 = __shfl_xor_sync(0xffffffffu, m2[q], o);
                const double low = m1[q] > u1 ? u1 : m1[q];             // the smaller of the two maxima
                m1[q] = m1[q] > u1 ? m1[q] : u1;
                m2[q] = m2[q] > u2 ? m2[q] : u2;
                m2[q] = m2[q] > low ? m2[q] : low;
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const double score = a.gtop == 2 && m2[q] > -INFINITY ? m1[q] + m2[q] : m1[q];
            if (lane == g0 + q) mine = score == score ? score : -INFINITY;
        }
    }
    return mine;
}

// Bit g of the result: group g stays (rank by score, ties to the lower group).
template <typename T>
__device__ __forceinline__ uint32_t kept_groups(const SelectArgs& a, T score, int lane) {
    int rank = 0;
#pragma unroll 4
    for (int g = 0; g < a.groups; ++g) {
        const T o = __shfl_sync(0xffffffffu, score, g);
        rank += o > score || (o == score && g < lane);
    }
    return __ballot_sync(0xffffffffu, lane < a.groups && rank < a.keep);
}

// The two largest keys of every group, from a warp's keys in shared memory (a pad
// word per 32 against bank conflicts): 2^lanes_log2 neighbouring lanes read a
// group; lane g returns group g's (-inf where there is none, or none asked for).
template <typename T>
__device__ __forceinline__ void group_best(const SelectArgs& a, const T* keys, int lane, T& m1, T& m2) {
    const int lg = a.lanes_log2, L = 1 << lg;
    const int g = lane >> lg;
    m1 = m2 = T(-INFINITY);
    if (g < a.groups) {
        for (int i = lane & (L - 1); i < a.gsize; i += L) {
            const int e = g * a.gsize + i;
            const T v = keys[e + (e >> 5)], low = m1 < v ? m1 : v;
            m2 = m2 > low ? m2 : low;
            m1 = m1 > v ? m1 : v;
        }
    }
    for (int o = 1; o < L; o <<= 1) {
        const T u1 = __shfl_xor_sync(0xffffffffu, m1, o), u2 = __shfl_xor_sync(0xffffffffu, m2, o);
        const T low = m1 < u1 ? m1 : u1;
        m2 = m2 > u2 ? m2 : u2;
        m2 = m2 > low ? m2 : low;
        m1 = m1 > u1 ? m1 : u1;
    }
    m1 = __shfl_sync(0xffffffffu, m1, (lane << lg) & 31);
    m2 = __shfl_sync(0xffffffffu, m2, (lane << lg) & 31);
    if (lane >= a.groups) m1 = m2 = T(-INFINITY);
    if (a.gtop == 1) m2 = T(-INFINITY);
}
// Their sum, of those that are there.
template <typename T>
__device__ __forceinline__ T group_sum(T m1, T m2) {
    const T score = m2 > T(-INFINITY) ? m1 + m2 : m1;
    return score == score ? score : T(-INFINITY);
}

// The whole selection in 64 bits; lane k < K returns pick k.
template <int V>
__device__ __noinline__ int select_exact(const SelectArgs& a, int64_t t, int lane) {
    double sel[V];
    float l[V];
    load_logits<V>(a, t, lane, l);
    float lmax = kMinusInf;
#pragma unroll
    for (int j = 0; j < V; ++j) lmax = fmaxf(lmax, l[j]);
    lmax = fmaxf(warp_max_f(lmax), -kFltMax);
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        sel[j] = a.sigmoid ? 1.0 / (1.0 + exp(-double(l[j]))) : exp(double(l[j]) - double(lmax));
        sum += sel[j];
    }
    sum = warp_sum_t(sum);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = lane + 32 * j;
        if (!a.sigmoid) sel[j] = sum > 0.0 ? sel[j] / sum : 0.0;
        sel[j] = with_bias(sel[j], a.bias && e < a.E ? a.bias[e] : 0.f, l[j] == kMinusInf);
    }
    uint32_t kept = 0xFFFFFFFFu;
    if (a.groups > 1) kept = kept_groups(a, group_scores<V>(a, sel, lane), lane);
    uint32_t out = 0u;     // bit j: expert lane + 32 j does not exist, is taken, or its group went
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = lane + 32 * j;
        if (e >= a.E || !((kept >> (a.groups > 1 ? e / a.gsize : 0)) & 1u)) out |= 1u << j;
        if (!a.bias) sel[j] = double(l[j]);
    }
    int mine = 0;
    for (int k = 0; k < a.K; ++k) {
        double bv = -INFINITY;
        int bi = 0x7FFFFFFF;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = lane + 32 * j;
            if (!((out >> j) & 1u) && (sel[j] > bv || (sel[j] == bv && e < bi))) {
                bv = sel[j];
                bi = e;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
            if (ov > bv || (ov == bv && oi < bi)) {
                bv = ov;
                bi = oi;
            }
        }
        if ((bi & 31) == lane) out |= 1u << (bi >> 5);
        if (lane == k) mine = bi;
    }
    return mine;
}

// Whether a >= b is certain to be the order of the 64-bit values when either
// is known to es + 2^-24 |value|.  Infinities are exact.
__device__ __forceinline__ bool certain(float a, float b, float es) {
    return a - b > 2.0f * es + 2.4e-7f * fmaxf(fabsf(a), fabsf(b)) || (a == b && isinf(a)) || b == kMinusInf;
}

// The denominator of the softmax in 64 bits.
template <int V>
__device__ __forceinline__ double softmax_sum64(const float (&l)[V], float lmax) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) sum += exp(double(l[j]) - double(lmax));
    return warp_sum_t(sum);
}
// The score of one logit in fp32 (to within the caller's `es`) and in 64 bits.
__device__ __forceinline__ float score32(const SelectArgs& a, float l, float lmax, float inv) {
    return a.sigmoid ? __frcp_rn(1.0f + expf(-l)) : __expf(l - lmax) * inv;
}
__device__ __forceinline__ double score64(const SelectArgs& a, float l, float lmax, double sum) {
    return a.sigmoid ? 1.0 / (1.0 + exp(-double(l))) : sum > 0.0 ? exp(double(l) - double(lmax)) / sum : 0.0;
}

// The groups that stay with a bias, by 64-bit scores (`keys`: the warp's shared memory).
template <int V>
__device__ __noinline__ uint32_t exact_groups(const SelectArgs& a, int64_t t, int lane, float lmax, double* keys) {
    float l[V];
    load_logits<V>(a, t, lane, l);
    const double sum = a.sigmoid ? 1.0 : softmax_sum64<V>(l, lmax);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = lane + 32 * j;
        keys[lane + 33 * j] = with_bias(score64(a, l[j], lmax, sum), e < a.E ? a.bias[e] : 0.f, l[j] == kMinusInf);
    }
    __syncwarp();
    double m1, m2;
    group_best(a, keys, lane, m1, m2);
    return kept_groups(a, group_sum(m1, m2), lane);
}

// Keys with a bias as fixed point below the token's largest one, `hi`: the
// fraction bits of key * scale + c in [1, 2), c = 1.9999 - hi * scale, over a bit
// that says the expert exists and its index (inverted).  Keys further down have
// the lowest fraction above 0 (kBelow: their order is in doubt), masked ones 0
// (kMasked: theirs is the index's).  scale is 1, or the power of two that brings
// the smallest key into the window where a pick lies below it.  23 bits (22 and 21
// beyond 256 and 512 experts, whose index takes more) resolve what fp32 keys can
// tell, where the leading bits of a float resolved 2^-16 and one token in ten had
// neighbouring picks in doubt.
template <int V>
struct Fixed {
    static constexpr uint32_t kIndex = 32 * V - 1;
    static constexpr int kLow = V <= 8 ? 9 : V == 16 ? 10 : 11;     // index and existence bits
    static constexpr float kUnit = 1.1920929e-7f * (1 << (kLow - 9));   // one step of a fraction
    static constexpr int kMasked = 0, kBelow = 1;
    static __device__ __forceinline__ uint32_t pack(float key, float scale, float c, int e) {
        // (c's rounding may carry the largest keys of a large bias to 2: they tie below it, in doubt)
        const float f = key == kMinusInf ? 1.0f + kMasked * kUnit
                                           : fminf(fmaxf(fmaf(key, scale, c), 1.0f + kBelow * kUnit), 1.9999999f);
        return ((__float_as_uint(f) << 9) & ~((1u << kLow) - 1u)) | (1u << (kLow - 1)) | (kIndex - e);
    }
    static __device__ __forceinline__ int expert(uint32_t m) { return int(kIndex - (m & kIndex)); }
    static __device__ __forceinline__ int fraction(uint32_t m) { return int(m >> kLow); }
};

// The picks with a bias where the order of the fp32 keys is in doubt: lane i holds
// the i-th largest of n packed keys, `m` (0: there were no more); sorts them by
// their 64-bit keys.  False if an expert that is not among them could still
// belong to the picks.
template <int V>
__device__ __noinline__ bool refine(const SelectArgs& a, int64_t t, int lane, int n, float margin, float scale, float c,
                                    float lmax, uint32_t m, int& pick) {
    using F = Fixed<V>;
    const bool live = lane < n && m != 0u;
    const uint32_t last = __shfl_sync(0xffffffffu, m, n - 1);
    const int id = live ? F::expert(m) : -1;
    const float l = live ? logit_at(a, t, id) : kMinusInf;
    const float b = live ? a.bias[id] : 0.f;
    double sum = 1.0;
    if (!a.sigmoid) {
        float all[V];
        load_logits<V>(a, t, lane, all);
        sum = softmax_sum64<V>(all, lmax);
    }
    const double key = with_bias(score64(a, l, lmax, sum), b, l == kMinusInf);
    int rank = live ? 0 : 32;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const double o = __shfl_sync(0xffffffffu, key, i);
        const int oid = __shfl_sync(0xffffffffu, id, i);
        rank += oid >= 0 && (o > key || (o == key && oid < id));
    }
    float kth = 0.f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const int r = __shfl_sync(0xffffffffu, rank, i), oid = __shfl_sync(0xffffffffu, id, i);
        const float o = __shfl_sync(0xffffffffu, float(key), i);
        if (r == lane) pick = oid;
        if (r == a.K - 1) kth = o;
    }
    // a key that is not among the n is at most the last one's
    const float most = 1.0f + float(F::fraction(last) + 1) * F::kUnit - c;      // (in the window's scale)
    return last == 0u || F::fraction(last) == F::kMasked || fmaf(kth, scale, -most) > margin * scale;
}

// The sum over lanes 0 .. K - 1 (zeros from K on), valid in those lanes.
template <typename T>
__device__ __forceinline__ T picks_sum(int K, T v) {
    for (int o = 1; o < K; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Gates of the picks (lane k holds pick k and its logit `l`), written with the ids.  `lmax` and
// `sum`: the softmax's maximum and denominator, read where they are needed.  The fast
// exponential's error grows with its argument, here a pick's distance from the largest logit,
// so expf (no slower: 65,536 tokens 32.8 us with either).  (The denominator's fast
// exponentials weigh with their own size: 8 units of it at most.)  The fast quotients are good
// to 2 units while the divisor is normal and below 2^126, which all of these are; true ones
// took 2 us more.
__device__ __forceinline__ void write_picks(const SelectArgs& a, int64_t t, int lane, int id, float l, float lmax,
                                            float sum) {
    const bool on = lane < a.K;
    if (!on) l = kMinusInf;
    float g, z;
    if (a.sigmoid) {
        // (by the exponential that cannot overflow: scores down to the smallest fp32 keep their digits)
        const float e = expf(-fabsf(l));
        g = __fdividef(l < 0.f ? e : 1.0f, 1.0f + e);      // 0 past the last pick
        if (a.renorm) {
            z = picks_sum(a.K, g);
            if (__any_sync(0xffffffffu, on && g < 1.17549435e-38f && l > kMinusInf && z < 0.25f)) {
                // subnormal scores have lost digits that a small sum brings to light: their ratios in 64 bits
                const double d = l == kMinusInf ? 0.0 : 1.0 / (1.0 + exp(-double(l)));
                const double zd = picks_sum(a.K, d);
                g = zd > 0.0 ? float(d / zd) : 0.f;
            } else {
                g = z > 0.f ? __fdividef(g, z) : 0.f;
            }
        }
    } else if (a.renorm) {
        // relative to the largest pick: the softmax's denominator cancels
        float m = l;
        if (a.bias) m = warp_max_f(l);
        else m = __shfl_sync(0xffffffffu, l, 0);
        g = expf(l - fmaxf(m, -kFltMax));
        z = picks_sum(a.K, g);
        g = z > 0.f ? __fdividef(g, z) : 0.f;
    } else {
        g = sum > 0.f ? __fdividef(expf(l - lmax), sum) : 0.f;
    }
    if (on) {
        const int64_t at = t * a.K + lane;
        a.ids[at] = id;
        a.gates[at] = g * a.scale;
    }
}

// A lane's two largest keys that are not taken, the lower place first on equal keys.
template <int V>
__device__ __forceinline__ void lane_top2(const uint32_t (&key)[V], uint32_t taken, uint32_t& h1, int& j1, uint32_t& h2,
                                          int& j2) {
    h1 = h2 = 0u;
    j1 = j2 = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t k = (taken >> j) & 1u ? 0u : key[j];
        const bool first = k > h1, second = k > h2;
        h2 = first ? h1 : second ? k : h2;
        j2 = first ? j1 : second ? j : j2;
        h1 = first ? k : h1;
        j1 = first ? j : j1;
    }
}

// Picks 0 .. n - 1 by descending key, the lower expert first on equal keys: lane
// k returns pick k's expert.  Every round takes the largest of the lanes' heads; a
// lane that gives its head moves its second up, and looks through its keys again
// only when it gives a third.
template <int V>
__device__ __forceinline__ int take_largest(const uint32_t (&key)[V], int n, int lane) {
    uint32_t taken = 0u, h1, h2;
    int j1, j2, mine = 0;
    bool have2 = true;
    lane_top2<V>(key, taken, h1, j1, h2, j2);
    for (int k = 0; k < n; ++k) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, h1);
        const int e = lane + 32 * j1;
        const uint32_t who = __ballot_sync(0xffffffffu, h1 == m);
        int id;
        if ((who & (who - 1)) == 0) id = __shfl_sync(0xffffffffu, e, __ffs(who) - 1);
        else id = int(__reduce_min_sync(0xffffffffu, h1 == m ? uint32_t(e) : 0xFFFFu));   // equal keys
        if (lane == k) mine = id;
        if (e == id && h1 == m) {
            taken |= 1u << j1;
            if (have2) {
                h1 = h2;
                j1 = j2;
                have2 = false;
            } else {
                lane_top2<V>(key, taken, h1, j1, h2, j2);
                have2 = true;
            }
        }
    }
    return mine;
}

// A lane's three largest packed keys; NEXT: of those below `under`.
template <int V, bool NEXT>
__device__ __forceinline__ void lane_top3(const uint32_t (&pk)[V], uint32_t under, uint32_t& h1, uint32_t& h2,
                                          uint32_t& h3) {
    h1 = h2 = h3 = 0u;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        uint32_t k = !NEXT || pk[j] < under ? pk[j] : 0u, low = min(h1, k);
        h1 = max(h1, k);
        k = min(h2, low);
        h2 = max(h2, low);
        h3 = max(h3, k);
    }
}

// The same picks from packed keys: the leading bits of a key's order over the
// expert's index (inverted: the lower one first), so that one warp-wide maximum
// a round gives both.  Keys of 16-bit logits fit whole; others may tie here,
// which the caller sees from neighbouring picks.  Lane k returns pick k (0:
// none).  A lane that has given its third key looks for its next three.
template <int V>
__device__ __forceinline__ uint32_t take_packed(const uint32_t (&pk)[V], int n, int lane) {
    uint32_t h1, h2, h3, mine = 0u;
    lane_top3<V, false>(pk, 0u, h1, h2, h3);
    auto round = [&](int k, bool third) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, h1);
        mine = lane == k ? m : mine;
        const bool own = h1 == m;
        h1 = own ? h2 : h1;
        h2 = own ? h3 : h2;
        h3 = own ? 0u : h3;
        if (V > 3 && third && __any_sync(0xffffffffu, own && h1 == 0u)) {
            uint32_t g1, g2, g3;
            lane_top3<V, true>(pk, m, g1, g2, g3);
            if (own) {
                h1 = g1;
                h2 = g2;
                h3 = g3;
            }
        }
    };
    // (a lane has given its third key in the third round at the earliest)
    round(0, false);
    if (n > 1) round(1, false);
#pragma unroll 2
    for (int k = 2; k < n; ++k) round(k, true);
    return mine;
}

// CTAs of 8 warps that an SM is to hold.
template <int V, bool SCORED>
constexpr int select_ctas() {
    return V <= 8 ? (SCORED ? 4 : 5) : V == 16 ? (SCORED ? 2 : 3) : (SCORED ? 1 : 2);
}

// SCORED: with a bias or groups; otherwise the keys are the logits.
template <int V, bool SCORED>
__global__ void __launch_bounds__(256, select_ctas<V, SCORED>()) route_select_kernel(const __grid_constant__ SelectArgs a) {
    // (64-bit keys of 1024 experts would not fit: their doubtful groups are left to select_exact)
    using GroupKey = std::conditional_t<V <= 16, double, float>;
    __shared__ GroupKey group_keys[SCORED ? 8 : 1][SCORED ? 33 * V : 1];
    constexpr uint32_t kIndex = 32 * V - 1;      // the bits of a packed key that hold the expert
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (t >= a.B) return;
    float l[V], bias[SCORED ? V : 1];
    if constexpr (SCORED) {      // (asked for before the logits are waited for)
        if (a.bias) {
#pragma unroll
            for (int j = 0; j < V; ++j) bias[j] = lane + 32 * j < a.E ? __ldg(a.bias + lane + 32 * j) : 0.f;
        }
    }
    load_logits<V>(a, t, lane, l);
    float lmax = kMinusInf, sum = 0.f;
    uint32_t pk[V];
    int id = 0;
    if (!a.sigmoid && (SCORED || !a.renorm)) {
#pragma unroll
        for (int j = 0; j < V; ++j) lmax = fmaxf(lmax, l[j]);
        lmax = fmaxf(warp_max_f(lmax), -kFltMax);
    }
    if constexpr (!SCORED) {
        if (!a.sigmoid && !a.renorm) {
#pragma unroll
            for (int j = 0; j < V; ++j) sum += __expf(l[j] - lmax);
            sum = warp_sum(sum);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) pk[j] = (order_bits(l[j]) & ~kIndex) | (kIndex - lane - 32 * j);
        if (a.E < 32 * V) {
#pragma unroll
            for (int j = 0; j < V; ++j) pk[j] = lane + 32 * j < a.E ? pk[j] : 0u;
        }
        // 16-bit logits are packed whole; others with one more than is picked, to see a tie of the last
        const bool whole = a.dtype != GALE_F32;
        const uint32_t m = take_packed<V>(pk, whole ? a.K : a.K + 1, lane);
        id = int(kIndex - (m & kIndex));
        if (whole) {
            // the pick's logit from its key: a negative one's order bits end in ones, and so do those of
            // the largest finite fp32, for which an infinity stands
            const uint32_t o = m & ~kIndex, ones = m | kIndex;
            const bool low = !(o & 0x80000000u) || ones == 0xFF7FFFFFu;
            write_picks(a, t, lane, id, order_value(low ? ones : o), lmax, sum);
            return;
        }
        const uint32_t next = __shfl_down_sync(0xffffffffu, m, 1);
        if (__any_sync(0xffffffffu, lane < a.K && next != 0u && ((m ^ next) & ~kIndex) == 0u)) {
#pragma unroll
            for (int j = 0; j < V; ++j) pk[j] = lane + 32 * j < a.E ? order_bits(l[j]) : 0u;
            id = take_largest<V>(pk, a.K, lane);
        }
    } else {
        // fp32 scores are needed of every expert with a bias, else of the groups' best;
        // es: what one may be off by
        float inv = 0.f, es;
        if (a.sigmoid) {
            // exp good to a unit in the last place (s (1 - s) 2^-23 <= 2^-25 in s), the
            // rounding of 1 + exp (2^-24 s) and of the reciprocal (2^-25): 2^-23.  A faster
            // exponential and quotient would quadruple that and the tokens taken in 64 bits.
            es = 1.2e-7f;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) sum += __expf(l[j] - lmax);
            sum = warp_sum(sum);
            inv = sum > 0.f ? 1.0f / sum : 0.f;
            // the largest score is inv; V + 5 additions, the exponentials (whose argument's
            // rounding times the exponential stays below half a unit of 1), the quotient
            es = inv * float(V + 24) * 1.2e-7f;
        }
        float s[V];         // keys in fp32
        if (!a.bias) {
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = l[j];
        } else {
            if (a.sigmoid) {
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] = __frcp_rn(1.0f + expf(-l[j]));
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] = __expf(l[j] - lmax) * inv;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = with_bias(s[j], bias[j], l[j] == kMinusInf);
        }
        uint32_t kept = 0xFFFFFFFFu;
        bool sure = true;
        if (a.groups > 1 && a.keep < a.groups) {
            float* gk = reinterpret_cast<float*>(group_keys[threadIdx.x >> 5]);
#pragma unroll
            for (int j = 0; j < V; ++j) gk[lane + 33 * j] = s[j];
            __syncwarp();
            float m1, m2;
            group_best(a, gk, lane, m1, m2);
            // what a sum of two is off by: twice es, and the roundings of the keys and of the sum
            const float k1 = a.bias || m1 == kMinusInf ? m1 : score32(a, m1, lmax, inv);
            const float k2 = a.bias || m2 == kMinusInf ? m2 : score32(a, m2, lmax, inv);
            const float f1 = fabsf(k1), f2 = fabsf(k2);
            const float big = warp_max_f(fmaxf(f1 < INFINITY ? f1 : 0.f, f2 < INFINITY ? f2 : 0.f));
            const float score = group_sum(k1, k2);
            kept = kept_groups(a, score, lane);
            const bool in = (kept >> lane) & 1u;
            const float worst = -warp_max_f(in ? -score : kMinusInf);
            const float best = warp_max_f(lane < a.groups && !in ? score : kMinusInf);
            // (a sum of two finite keys that leaves fp32's range, to either side, tells nothing)
            sure = certain(worst, best, 2.0f * es + 4.8e-7f * big) &&
                   !__any_sync(0xffffffffu, isinf(score) && !isinf(k1));
            if (!sure && !a.bias) {
                // the best two of a group are certain (by logit): their scores in 64 bits
                const double all = a.sigmoid ? 1.0 : softmax_sum64<V>(l, lmax);
                const double d1 = m1 == kMinusInf ? double(kMinusInf) : score64(a, m1, lmax, all);
                const double d2 = m2 == kMinusInf ? double(kMinusInf) : score64(a, m2, lmax, all);
                kept = kept_groups(a, group_sum(d1, d2), lane);
                sure = true;
            } else if (!sure && V <= 16) {
                kept = exact_groups<V>(a, t, lane, lmax, reinterpret_cast<double*>(group_keys[threadIdx.x >> 5]));
                sure = true;
            }
        }
        // experts whose group went: 0, below every key
        auto stays = [&](int e) {
            return e < a.E && ((kept >> (a.groups > 1 ? int(uint32_t(e) * a.gmagic >> 20) : 0)) & 1u);
        };
        if (a.bias) {
            using F = Fixed<V>;
            float hi = kMinusInf;
#pragma unroll
            for (int j = 0; j < V; ++j) hi = stays(lane + 32 * j) ? fmaxf(hi, s[j]) : hi;
            hi = warp_max_f(hi);
            sure = sure && hi < INFINITY;
            // what two keys' difference may be off by: the scores, their roundings with the bias and in the window
            const float margin = 2.0f * es + 2.4e-7f * (fabsf(hi) + 2.0f);
            float scale = 1.0f;
#pragma unroll 1
            while (sure) {
                const float c = hi == kMinusInf ? 0.f : fmaf(-hi, scale, 1.9999f);
#pragma unroll
                for (int j = 0; j < V; ++j) pk[j] = stays(lane + 32 * j) ? F::pack(s[j], scale, c, lane + 32 * j) : 0u;
                // one more than is picked: the last pick's lead counts too
                const uint32_t m = take_packed<V>(pk, a.K + 1, lane);
                const uint32_t next = __shfl_down_sync(0xffffffffu, m, 1);
                id = F::expert(m);
                // (margin in the window's scale, and the window's own rounding)
                const float off = fmaf(margin, scale, 2.4e-7f);
                const bool clear = lane >= a.K || next == 0u || F::fraction(next) == F::kMasked ||
                                   float(F::fraction(m) - F::fraction(next) - 1) * F::kUnit > off;
                if (__all_sync(0xffffffffu, clear)) break;
                if (scale == 1.0f && __any_sync(0xffffffffu, lane <= a.K && m != 0u && F::fraction(m) == F::kBelow)) {
                    float lo = INFINITY;
#pragma unroll
                    for (int j = 0; j < V; ++j) lo = stays(lane + 32 * j) && s[j] > kMinusInf ? fminf(lo, s[j]) : lo;
                    lo = -warp_max_f(-lo);
                    if (hi - lo < 1e30f) {
                        scale = exp2f(-ceilf(log2f((hi - lo) * 1.01f)));
                        if (scale < 1.0f) continue;
                    }
                }
                const int n = a.K + 3;
                const uint32_t mn = take_packed<V>(pk, n, lane);
                sure = refine<V>(a, t, lane, n, margin + 2.4e-7f / scale, scale, c, lmax, mn, id);
                break;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = lane + 32 * j;
                pk[j] = stays(e) ? (order_bits(s[j]) & ~kIndex) | (kIndex - e) : 0u;
            }
            const uint32_t m = take_packed<V>(pk, a.K + 1, lane);
            const uint32_t next = __shfl_down_sync(0xffffffffu, m, 1);
            id = int(kIndex - (m & kIndex));
            if (a.dtype == GALE_F32 &&
                __any_sync(0xffffffffu, lane < a.K && next != 0u && ((m ^ next) & ~kIndex) == 0u)) {
#pragma unroll
                for (int j = 0; j < V; ++j) pk[j] = pk[j] != 0u ? order_bits(s[j]) : 0u;
                id = take_largest<V>(pk, a.K, lane);
            }
        }
        if (!sure) id = select_exact<V>(a, t, lane);
    }
    write_picks(a, t, lane, id, lane < a.K ? logit_at(a, t, id) : kMinusInf, lmax, sum);
}

}  // namespace
}  // namespace gale

extern "C" int gale_route_select(const void* logits, int logits_dtype, int64_t ld, const float* bias, int B, int E,
                                 int K, int score, int n_groups, int keep_groups, int group_top, int renorm,
                                 float scale, int32_t* ids, float* gates, void* stream) {
    using namespace gale;
    if (B < 0 || E < 1 || E > 1024 || K < 1 || K > 16 || K > E || ld < E) return GALE_ERR_ARG;
    if (logits_dtype != GALE_F32 && logits_dtype != GALE_BF16 && logits_dtype != GALE_F16) return GALE_ERR_ARG;
    if (score != GALE_SCORE_SOFTMAX && score != GALE_SCORE_SIGMOID) return GALE_ERR_ARG;
    if (n_groups < 1 || n_groups > 32 || E % n_groups || keep_groups < 1 || keep_groups > n_groups)
        return GALE_ERR_ARG;
    const int gsize = E / n_groups;
    if (group_top < 1 || group_top > 2 || int64_t(keep_groups) * gsize < K) return GALE_ERR_ARG;
    if (B == 0) return GALE_OK;
    if (!logits || !ids || !gates) return GALE_ERR_ARG;
    if (!aligned(logits, logits_dtype == GALE_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(gates, 4))
        return GALE_ERR_ALIGN;
    SelectArgs a{logits, bias, ids, gates, ld, B, E, K, logits_dtype, score == GALE_SCORE_SIGMOID, renorm != 0,
                 n_groups, gsize, keep_groups, group_top, scale, 0, 0u};
    while ((2 << a.lanes_log2) * n_groups <= 32) ++a.lanes_log2;
    // exact quotients: e * (gmagic * gsize - 2^20) < 2^20 for e < 1024, gsize <= 1024
    a.gmagic = ((1u << 20) + gsize - 1) / gsize;
    cudaStream_t st = as_stream(stream);
    const unsigned grid = unsigned((int64_t(B) + 7) / 8);
    auto launch = [&](auto v) {
        constexpr int V = decltype(v)::value;
        if (a.bias || a.groups > 1) route_select_kernel<V, true><<<grid, 256, 0, st>>>(a);
        else route_select_kernel<V, false><<<grid, 256, 0, st>>>(a);
    };
    if (E <= 32) launch(std::integral_constant<int, 1>());
    else if (E <= 64) launch(std::integral_constant<int, 2>());
    else if (E <= 128) launch(std::integral_constant<int, 4>());
    else if (E <= 256) launch(std::integral_constant<int, 8>());
    else if (E <= 512) launch(std::integral_constant<int, 16>());
    else launch(std::integral_constant<int, 32>());
    GALE_LAUNCH_CHECK();
    return GALE_OK;
}
