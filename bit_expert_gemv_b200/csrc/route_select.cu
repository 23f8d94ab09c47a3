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
// the 64-bit values of these formulas.  It is taken in fp32 first: every value
// is known to within `err`, and a comparison that the error could turn is
// settled by computing the candidates again in 64 bits (select_exact).
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
    l = l == l ? l : kMinusInf;
    return l > kFltMax ? kFltMax : l;
}
__device__ __forceinline__ float logit_at(const SelectArgs& a, int64_t t, int e) {
    return clean(load_as_f32(a.logits, a.dtype, t * a.ld + e));
}
// s + b, -inf for a masked expert or a NaN
template <typename T>
__device__ __forceinline__ T with_bias(T s, float b, bool masked) {
    const T k = s + T(b);
    return masked || !(k == k) ? T(-INFINITY) : k;
}

template <typename T>
__device__ __forceinline__ T warp_max_t(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const T u = __shfl_xor_sync(0xffffffffu, v, o);
        v = u > v ? u : v;
    }
    return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum_t(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Group scores by warp-wide passes over the groups: lane g returns group g's.
template <typename T, int V>
__device__ __forceinline__ T group_scores(const SelectArgs& a, const T (&sel)[V], int lane) {
    T mine = T(-INFINITY);
    for (int g = 0; g < a.groups; ++g) {
        const int lo = g * a.gsize, hi = lo + a.gsize;
        T m1 = T(-INFINITY), m2 = T(-INFINITY);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = lane + 32 * j;
            if (e >= lo && e < hi) {
                const T v = sel[j];
                if (v > m1) { m2 = m1; m1 = v; }
                else if (v > m2) m2 = v;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const T u1 = __shfl_xor_sync(0xffffffffu, m1, o), u2 = __shfl_xor_sync(0xffffffffu, m2, o);
            const T low = m1 > u1 ? u1 : m1;             // the smaller of the two maxima
            m1 = m1 > u1 ? m1 : u1;
            m2 = m2 > u2 ? m2 : u2;
            m2 = m2 > low ? m2 : low;
        }
        T score = m1;
        if (a.gtop == 2 && m2 > T(-INFINITY)) score = m1 + m2;
        if (lane == g) mine = score == score ? score : T(-INFINITY);
    }
    return mine;
}

// Bit g of the result: group g stays (rank by score, ties to the lower group).
template <typename T>
__device__ __forceinline__ uint32_t kept_groups(const SelectArgs& a, T score, int lane) {
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
        const T o = __shfl_sync(0xffffffffu, score, g);
        rank += o > score || (o == score && g < lane);
    }
    return __ballot_sync(0xffffffffu, lane < a.groups && rank < a.keep);
}

// The whole selection in 64 bits; lane k < K returns pick k.
template <int V>
__device__ __noinline__ int select_exact(const SelectArgs& a, int64_t t, int lane) {
    double sel[V];
    float l[V];
    float lmax = kMinusInf;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = lane + 32 * j;
        l[j] = e < a.E ? logit_at(a, t, e) : kMinusInf;
        lmax = fmaxf(lmax, l[j]);
    }
    lmax = fmaxf(warp_max_t(lmax), -kFltMax);
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
    if (a.groups > 1) kept = kept_groups(a, group_scores<double, V>(a, sel, lane), lane);
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

// Gates of the picks (lane k holds pick k), written with the ids.  `lmax` and
// `sum`: the softmax's maximum and denominator, read where they are needed.
__device__ __forceinline__ void write_picks(const SelectArgs& a, int64_t t, int lane, int id, float lmax, float sum) {
    const bool on = lane < a.K;
    const float l = on ? logit_at(a, t, id) : kMinusInf;
    float g;
    if (a.sigmoid) {
        const float s = 1.0f / (1.0f + expf(-l));
        g = s;
        if (a.renorm) {
            const float z = warp_sum(s);
            g = z > 0.f ? s / z : 0.f;
            if (z < 1e-30f) {       // scores at the end of fp32's range: their ratios in 64 bits
                const double d = l == kMinusInf ? 0.0 : 1.0 / (1.0 + exp(-double(l)));
                const double zd = warp_sum_t(d);
                g = zd > 0.0 ? float(d / zd) : 0.f;
            }
        }
    } else if (a.renorm) {
        // relative to the largest pick: the softmax's denominator cancels
        const float m = fmaxf(warp_max_t(l), -kFltMax);
        const float s = expf(l - m);
        const float z = warp_sum(s);
        g = z > 0.f ? s / z : 0.f;
    } else {
        g = sum > 0.f ? expf(l - lmax) / sum : 0.f;
    }
    if (on) {
        a.ids[t * a.K + lane] = id;
        a.gates[t * a.K + lane] = g * a.scale;
    }
}

// Unsigned order of a float: larger value, larger integer (-0 as +0); 0 is below every value's.
__device__ __forceinline__ uint32_t order_bits(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
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
// k returns pick k's expert and its key (0: there were no more).  Every round
// takes the largest of the lanes' heads; a lane that gives its head moves its
// second up, and looks through its keys again only when it gives a third.
template <int V>
__device__ __forceinline__ int take_largest(const uint32_t (&key)[V], int n, int lane, uint32_t& my_key) {
    uint32_t taken = 0u, h1, h2;
    int j1, j2, mine = 0;
    bool have2 = true;
    lane_top2<V>(key, taken, h1, j1, h2, j2);
    my_key = 0u;
    for (int k = 0; k < n; ++k) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, h1);
        const int e = lane + 32 * j1;
        const int id = int(__reduce_min_sync(0xffffffffu, h1 == m ? uint32_t(e) : 0xFFFFu));
        if (lane == k) {
            mine = id;
            my_key = m;
        }
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

// Whether a >= b is certain to be the order of the 64-bit values when either
// is known to es + 2^-24 |value|.  Infinities are exact.
__device__ __forceinline__ bool certain(float a, float b, float es) {
    return a - b > 2.0f * es + 2.4e-7f * fmaxf(fabsf(a), fabsf(b)) || (a == b && isinf(a)) || b == kMinusInf;
}

template <int V>
__global__ void __launch_bounds__(256) route_select_kernel(SelectArgs a) {
    __shared__ float group_keys[8][33 * V];
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (t >= a.B) return;
    float l[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = lane + 32 * j;
        l[j] = e < a.E ? logit_at(a, t, e) : kMinusInf;
    }
    float lmax = kMinusInf, sum = 0.f;
    uint32_t key[V];
    bool sure = true;
    const bool scored = a.bias || a.groups > 1;
    if (!scored) {
        // no bias, no groups: the keys are the logits
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = lane + 32 * j < a.E ? order_bits(l[j]) : 0u;
        if (!a.sigmoid && !a.renorm) {
#pragma unroll
            for (int j = 0; j < V; ++j) lmax = fmaxf(lmax, l[j]);
            lmax = fmaxf(warp_max_t(lmax), -kFltMax);
#pragma unroll
            for (int j = 0; j < V; ++j) sum += __expf(l[j] - lmax);
            sum = warp_sum(sum);
        }
    } else {
        // fp32 scores and what they may be off by
        float s[V], es;
        if (a.sigmoid) {
            // exp to 2^-22 relatively, 1 + exp and the quotient to two units: below 2^-21 of 1
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = __fdividef(1.0f, 1.0f + __expf(-l[j]));
            es = 4.8e-7f;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) lmax = fmaxf(lmax, l[j]);
            lmax = fmaxf(warp_max_t(lmax), -kFltMax);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[j] = __expf(l[j] - lmax);
                sum += s[j];
            }
            sum = warp_sum(sum);
            const float inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] *= inv;
            // the largest score is inv; V + 5 additions, the exponentials (whose argument's rounding
            // times the exponential stays below half a unit of 1), the quotient
            es = inv * float(V + 24) * 1.2e-7f;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = lane + 32 * j;
            s[j] = with_bias(s[j], a.bias && e < a.E ? __ldg(a.bias + e) : 0.f, l[j] == kMinusInf);
        }
        uint32_t kept = 0xFFFFFFFFu;
        if (a.groups > 1 && a.keep < a.groups) {
            // a group's keys to L neighbouring lanes through shared memory (a pad word per 32 against bank conflicts)
            float* gk = group_keys[threadIdx.x >> 5];
#pragma unroll
            for (int j = 0; j < V; ++j) gk[lane + 33 * j] = s[j];
            __syncwarp();
            const int lg = a.lanes_log2, L = 1 << lg;
            const int g = lane >> lg;
            float m1 = kMinusInf, m2 = kMinusInf;
            if (g < a.groups) {
                for (int i = lane & (L - 1); i < a.gsize; i += L) {
                    const int e = g * a.gsize + i;
                    const float v = gk[e + (e >> 5)];
                    m2 = fmaxf(m2, fminf(m1, v));
                    m1 = fmaxf(m1, v);
                }
            }
            for (int o = 1; o < L; o <<= 1) {
                const float u1 = __shfl_xor_sync(0xffffffffu, m1, o), u2 = __shfl_xor_sync(0xffffffffu, m2, o);
                m2 = fmaxf(fmaxf(m2, u2), fminf(m1, u1));
                m1 = fmaxf(m1, u1);
            }
            float score = a.gtop == 2 && m2 > kMinusInf ? m1 + m2 : m1;
            if (!(score == score)) score = kMinusInf;
            score = __shfl_sync(0xffffffffu, score, (lane << lg) & 31);
            if (lane >= a.groups) score = kMinusInf;
            // what a sum of two is off by: twice es, and the roundings of the keys and of the sum
            const float mag = fmaxf(fabsf(m1), m2 > kMinusInf ? fabsf(m2) : 0.f);
            const float big = warp_max_t(g < a.groups && mag < INFINITY ? mag : 0.f);
            kept = kept_groups(a, score, lane);
            const bool in = (kept >> lane) & 1u;
            const float worst = -warp_max_t(in ? -score : kMinusInf);
            const float best = warp_max_t(lane < a.groups && !in ? score : kMinusInf);
            sure = certain(worst, best, 2.0f * es + 4.8e-7f * big);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = lane + 32 * j;
            const int g = a.groups > 1 ? int(uint32_t(e) * a.gmagic >> 20) : 0;
            const bool live = e < a.E && ((kept >> g) & 1u);
            key[j] = live ? order_bits(a.bias ? s[j] : l[j]) : 0u;
        }
        if (a.bias && sure) {
            // one more than is picked: the last pick's lead counts too
            uint32_t mk;
            const int id = take_largest<V>(key, a.K + 1, lane, mk);
            const uint32_t nk = __shfl_down_sync(0xffffffffu, mk, 1);
            const bool clear = lane >= a.K || nk == 0u || certain(order_value(mk), order_value(nk), es);
            if (__all_sync(0xffffffffu, clear)) {
                write_picks(a, t, lane, id, lmax, sum);
                return;
            }
            sure = false;
        }
    }
    uint32_t mk;
    const int id = sure ? take_largest<V>(key, a.K, lane, mk) : select_exact<V>(a, t, lane);
    write_picks(a, t, lane, id, lmax, sum);
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
    const unsigned grid = unsigned((B + 7) / 8);
    if (E <= 32) route_select_kernel<1><<<grid, 256, 0, st>>>(a);
    else if (E <= 64) route_select_kernel<2><<<grid, 256, 0, st>>>(a);
    else if (E <= 128) route_select_kernel<4><<<grid, 256, 0, st>>>(a);
    else if (E <= 256) route_select_kernel<8><<<grid, 256, 0, st>>>(a);
    else if (E <= 512) route_select_kernel<16><<<grid, 256, 0, st>>>(a);
    else route_select_kernel<32><<<grid, 256, 0, st>>>(a);
    GALE_LAUNCH_CHECK();
    return GALE_OK;
}
