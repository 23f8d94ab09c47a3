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

template <int V>
__global__ void __launch_bounds__(256) route_select_kernel(SelectArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= a.B) return;
    const int id = select_exact<V>(a, t, lane);
    float lmax = kMinusInf, sum = 0.f;
    if (!a.sigmoid && !a.renorm) {
        for (int e = lane; e < a.E; e += 32) lmax = fmaxf(lmax, logit_at(a, t, e));
        lmax = fmaxf(warp_max_t(lmax), -kFltMax);
        for (int e = lane; e < a.E; e += 32) sum += expf(logit_at(a, t, e) - lmax);
        sum = warp_sum(sum);
    }
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
                 n_groups, gsize, keep_groups, group_top, scale};
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
