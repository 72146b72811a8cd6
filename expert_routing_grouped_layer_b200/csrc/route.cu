// route.cu -- expert selection from given router logits, forward and backward.
//
// "DeepSeek V3架构拆解：Kimi-K2-Thinking-NVFP4的MLA注意力与MoE路由实现原理", 三.1-三.3: s = score(l)
// (sigmoid; sqrt(softplus), "DeepSeek-V4-Pro 架构与代码概述" 架构; softmax over the row),
// s' = s + bias, the topk_group best of n_group groups by the sum of their two largest
// s', the k largest s' of those, weights s (divided by their sum) times the routed
// scaling factor. An expert with a logit or bias of -inf is masked: never chosen.
//
// Which expert is chosen is decided exactly. Without bias and groups the order of s' is
// the order of the logits. Otherwise s' is computed in fp32 with a known error bound;
// where two values that the outcome depends on lie closer than twice the bound, they
// are computed in double precision and compared there (then the larger logit, then the
// lower index). That happens for about one token in a thousand, so the fp32 path sets
// the speed.
//
// One warp per token holds the row in registers. The cost is the exponentials and the
// k rounds of a warp-wide maximum (redux.sync on order-preserving integer keys), not the
// bytes: ~1100 instructions a token at 384 experts, top 8, 4 of 8 groups, 15.3 us for 8192
// tokens (2 us of memory time); 45 us for 16384 tokens of 896 experts, top 16. The gradient
// of 16384 x 896 bf16 softmax logits takes 18.5 us (9.3 us of memory time).
#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include "internal.h"
#include "sm100.cuh"
#include "types.cuh"

namespace moe {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr float kInf = INFINITY;

struct RouteParams {
    const void* logits;
    const float* bias;
    int32_t* idx;
    float* w;
    long ld;
    int T, E, k, n_group, topk_group, norm, score_fn;
    float rsf;
};

// fp32 keys ordered as unsigned integers (finite values and infinities).
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ float warp_max(float v) { return value_of(__reduce_max_sync(kFull, key_of(v))); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Scores. m and z: the row's largest logit and sum of exponentials (softmax).
// For the order alone: exponentials and reciprocals of a few units of 2^-24, scaled by the
// argument (|l| s (1 - s) and |l - m| s stay below 0.4), see the bound in the kernel.
template <int FN>
__device__ __forceinline__ float score_fast(float l, float m, float inv_z) {
    if (FN == MOE_SCORE_SIGMOID) return rcp_approx(1.0f + exp_approx(-l));
    if (FN == MOE_SCORE_SQRTSOFTPLUS) return sqrtf(fmaxf(l, 0.0f) + log1pf(expf(-fabsf(l))));
    return exp_approx(l - m) * inv_z;
}
template <typename F>
__device__ __forceinline__ void with_score(int fn, F&& f) {
    if (fn == MOE_SCORE_SIGMOID) f(std::integral_constant<int, MOE_SCORE_SIGMOID>());
    else if (fn == MOE_SCORE_SQRTSOFTPLUS) f(std::integral_constant<int, MOE_SCORE_SQRTSOFTPLUS>());
    else f(std::integral_constant<int, MOE_SCORE_SOFTMAX>());
}

// sqrt(log(1 + e^l)) = e^(l/2) (1 - e^l / 4 + ...): far below zero the first factor alone, since
// e^l leaves the type's range while e^(l/2) is an ordinary number (from l = -88 on in fp32).
__device__ __forceinline__ float score_f(float l, int fn, float m, float inv_z) {
    if (fn == MOE_SCORE_SIGMOID) return 1.0f / (1.0f + expf(-l));
    if (fn == MOE_SCORE_SQRTSOFTPLUS) {
        const float e = expf(-0.5f * fabsf(l));
        return l < -20.0f ? e : sqrtf(fmaxf(l, 0.0f) + log1pf(e * e));  // at -20 the rest is 5e-10 of e
    }
    return expf(l - m) * inv_z;
}
__device__ __forceinline__ double score_d(double l, int fn, double m, double z) {
    if (fn == MOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
    if (fn == MOE_SCORE_SQRTSOFTPLUS)  // at -80 they are below 2^-53
        return l < -80.0 ? exp(0.5 * l) : sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
    return exp(l - m) / z;
}

// The row as the slow paths see it: masked elements are -inf.
template <typename T>
struct Row {
    const T* l;
    const float* bias;
    int E, gsz, fn;
    float m;
    double z;
    uint32_t kept;  // bit g: group g is kept
    __device__ __forceinline__ float logit(int e) const { return to_f32<T>(l[e]) + 0.0f; }
    __device__ __forceinline__ double sel(int e, float le) const {
        const float b = bias ? bias[e] : 0.f;
        if (le == -kInf || b == -kInf) return -(double)kInf;
        return score_d((double)le, fn, (double)m, z) + (double)b;
    }
};

template <typename T>
__device__ __noinline__ double row_z(const T* l, int E, float m) {
    double z = 0.0;
    for (int e = threadIdx.x & 31; e < E; e += 32) {
        const float le = to_f32<T>(l[e]);
        if (le != -kInf) z += exp((double)le - (double)m);
    }
    return warp_sum(z);
}

// The kept groups by their scores in double precision: each group's L = 1 << shift lanes share
// its elements, as in the fp32 path.
template <typename T>
__device__ __noinline__ uint32_t groups_exact(Row<T> r, int n_group, int topk_group, int shift) {
    const int lane = threadIdx.x & 31, g = lane >> shift, L = 1 << shift;
    double b1 = -(double)kInf, b2 = b1;
    if (g < n_group) {
        for (int e = g * r.gsz + (lane & (L - 1)); e < (g + 1) * r.gsz; e += L) {
            const double v = r.sel(e, r.logit(e));
            b2 = fmax(b2, fmin(b1, v));
            b1 = fmax(b1, v);
        }
    }
    for (int o = L >> 1; o > 0; o >>= 1) {
        const double o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
        b2 = fmax(fmin(b1, o1), fmax(b2, o2));
        b1 = fmax(b1, o1);
    }
    const double gs = b2 == -(double)kInf ? b1 : b1 + b2;
    int rank = 0;
    for (int h = 0; h < n_group; ++h) {
        const double o = __shfl_sync(kFull, gs, h << shift);
        rank += (o > gs || (o == gs && h < g)) ? 1 : 0;
    }
    const uint32_t lanes = __ballot_sync(kFull, g < n_group && rank < topk_group);
    uint32_t kept = 0u;
    for (int h = 0; h < n_group; ++h) kept |= ((lanes >> (h << shift)) & 1u) << h;
    return kept;
}

__device__ __forceinline__ bool better_d(double va, float la, int ia, double vb, float lb, int ib) {
    return va > vb || (va == vb && (la > lb || (la == lb && ia < ib)));
}

// Orders up to 32 candidates (one per lane, e < 0: none) by their exact values; the
// expert of rank r lands in lane r (-1 where there is none).
template <typename T>
__device__ __noinline__ int rank_exact(Row<T> r, int e, int count) {
    const int lane = threadIdx.x & 31;
    const float l = e >= 0 ? r.logit(e) : 0.f;
    const double v = e >= 0 ? r.sel(e, l) : -(double)kInf;
    int rank = 0;
    for (int c = 0; c < count; ++c) {
        const double vo = __shfl_sync(kFull, v, c);
        const float lo = __shfl_sync(kFull, l, c);
        const int eo = __shfl_sync(kFull, e, c);
        rank += better_d(vo, lo, eo, v, l, e) ? 1 : 0;
    }
    if (e < 0) rank = 64;
    int mine = -1;
    for (int c = 0; c < count; ++c) {
        const int at = __shfl_sync(kFull, rank, c), eo = __shfl_sync(kFull, e, c);
        if (at == lane) mine = eo;
    }
    return mine;
}

// More than 32 candidates lie within the error bound (rows of nearly equal scores):
// k rounds, each a maximum of the exact values over the experts not yet chosen.
template <typename T>
__device__ __noinline__ int topk_exact(Row<T> r, int k) {
    const int lane = threadIdx.x & 31;
    uint32_t taken = 0;  // bit i: expert lane + 32 i
    int mine = -1;
    for (int round = 0; round < k; ++round) {
        double bv = -(double)kInf;
        float bl = -kInf;
        int be = INT_MAX;
        for (int e = lane, i = 0; e < r.E; e += 32, ++i) {
            if (((taken >> i) & 1u) || !((r.kept >> (e / r.gsz)) & 1u)) continue;
            const float l = r.logit(e);
            const double v = r.sel(e, l);
            if (v != -(double)kInf && better_d(v, l, e, bv, bl, be)) { bv = v; bl = l; be = e; }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(kFull, bv, o);
            const float ol = __shfl_xor_sync(kFull, bl, o);
            const int oe = __shfl_xor_sync(kFull, be, o);
            if (better_d(ov, ol, oe, bv, bl, be)) { bv = ov; bl = ol; be = oe; }
        }
        if (be == INT_MAX) break;
        if ((be & 31) == lane) taken |= 1u << (be >> 5);
        if (round == lane) mine = be;
    }
    return mine;
}

// Lane j's share s_j / sum s of the chosen scores (j < k, valid), and, without
// normalisation, s_j itself. Scores far below the fp32 range (every chosen logit
// around -90 and less) are taken in double precision.
__device__ __forceinline__ float chosen_weight(float l, bool valid, int fn, int norm, float m, float z) {
    float s = valid ? score_f(l, fn, m, 1.0f / z) : 0.f;
    if (!norm) return s;
    if (__any_sync(kFull, valid && s < 1e-30f)) {
        const double sd = valid ? score_d((double)l, fn, (double)m, (double)z) : 0.0;
        const double sum = warp_sum(sd);
        return sum > 0.0 ? (float)(sd / sum) : 0.f;
    }
    const float sum = warp_sum(s);
    return sum > 0.f ? s / sum : 0.f;
}

template <int VEC>
__device__ __forceinline__ void load_bias(float* b, const float* p) {
    if constexpr (VEC % 4 == 0) {  // 16-byte aligned where the logits' vectors are used
#pragma unroll
        for (int v = 0; v < VEC; v += 4) {
            const float4 f = *reinterpret_cast<const float4*>(p + v);
            b[v] = f.x; b[v + 1] = f.y; b[v + 2] = f.z; b[v + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) b[v] = p[v];
    }
}

// Lane (g, sub) of L lanes per group holds the group's elements (sub + L i) VEC + v:
// a group's two largest come from the lanes of that group alone, and without groups
// (L = 32) a load instruction covers consecutive elements.
template <typename T, int VEC, int NI>
__global__ void __launch_bounds__(256, NI * VEC > 32 ? 1 : 3) route_fwd_kernel(RouteParams p, int L) {
    pdl_wait();
    pdl_trigger();
    constexpr int J = NI * VEC;
    typedef unsigned long long u64;
    __shared__ int2 list[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long t = (long)blockIdx.x * (blockDim.x >> 5) + warp;
    if (t >= p.T) return;
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    const int gsz = p.E / p.n_group;
    const int shift = __ffs(L) - 1, g = lane >> shift, sub = lane & (L - 1);
    const int nvec = g < p.n_group ? gsz / VEC : 0;
    const int e0 = g * gsz + sub * VEC;  // element (i, v) is e0 + i L VEC + v

    Pack<T, VEC> raw[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
        if (sub + i * L < nvec) raw[i] = reinterpret_cast<const Pack<T, VEC>*>(row + e0)[i * L];
    const bool by_logit = !p.bias && p.n_group == 1;
    float sel[J];  // logits, then s' (or the logits, by_logit); -inf: masked or no element
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float l = sub + i * L < nvec ? to_f32<T>(raw[i].v[v]) + 0.0f : -kInf;
            bad |= !(l < kInf);
            sel[i * VEC + v] = l;
        }
    }
    // the row's maximum and sum of exponentials (softmax), or the largest score's bound
    float m = 0.f, z = 1.f, scale = 1.f;
    if (p.score_fn != MOE_SCORE_SIGMOID) {
        float lm = sel[0];
#pragma unroll
        for (int j = 1; j < J; ++j) lm = fmaxf(lm, sel[j]);
        const float top = warp_max(bad ? -kInf : lm);
        if (p.score_fn == MOE_SCORE_SOFTMAX) {
            m = top == -kInf ? 0.f : top;
            float zs = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) zs += exp_approx(sel[j] - m);
            z = warp_sum(zs);
        } else {
            scale = fmaxf(1.f, sqrtf(fmaxf(top, 0.f) + 1.f));
        }
    }
    if (!by_logit) {
        const float inv_z = z > 0.f ? 1.0f / z : 0.f;  // 0: every expert is masked
        float bias[J];
#pragma unroll
        for (int j = 0; j < J; ++j) bias[j] = 0.f;
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (sub + i * L < nvec) load_bias<VEC>(bias + i * VEC, p.bias + e0 + i * L * VEC);
        }
        with_score(p.score_fn, [&](auto fn) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float s = score_fast<fn.value>(sel[j], m, inv_z) + bias[j];  // -inf with the bias
                bad |= !(s < kInf);
                sel[j] = sel[j] == -kInf ? -kInf : s;
            }
        });
    }
    if (__any_sync(kFull, bad)) {  // a NaN or +inf among the row's logits or the biases
        if (lane < p.k) {
            p.idx[t * p.k + lane] = -1;
            p.w[t * p.k + lane] = NAN;
        }
        return;
    }
    // |computed s' - s'| <= err + 1.2e-7 |s'|: the last addition's rounding, and an error in
    // proportion to the row's largest score: a few units of 2^-24, for the softmax also its
    // sum's J + 5 additions
    const float err = p.score_fn == MOE_SCORE_SOFTMAX ? (J + 24) * 6.0e-8f * (z > 0.f ? 1.0f / z : 0.f)
                                                      : 4.8e-7f * scale;
    auto bound = [&](float v) { return err + 1.2e-7f * fabsf(v); };

    bool keep = true;  // this lane's group is kept
    if (p.n_group > 1) {
        float b1 = -kInf, b2 = -kInf;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            b2 = fmaxf(b2, fminf(b1, sel[j]));
            b1 = fmaxf(b1, sel[j]);
        }
        for (int o = L >> 1; o > 0; o >>= 1) {
            const float o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
            b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
            b1 = fmaxf(b1, o1);
        }
        // half the sum: two biases of the type's lowest value add up to a number, above "no expert"
        const float gs = 0.5f * b1 + (b2 == -kInf ? 0.f : 0.5f * b2);
        const bool real = g < p.n_group;
        keep = false;
        uint32_t gk = real ? key_of(gs) : 0u, lo_key = 0u;
        for (int r = 0; r < p.topk_group; ++r) {  // the lower group of equal ones
            lo_key = __reduce_max_sync(kFull, gk);
            if (g == (__ffs(__ballot_sync(kFull, gk == lo_key)) - 1) >> shift) {
                keep = true;
                gk = 0u;
            }
        }
        const uint32_t hi_key = __reduce_max_sync(kFull, gk);
        const float lo = value_of(lo_key);                       // smallest kept
        const float hi = hi_key ? value_of(hi_key) : -kInf;      // largest left out
        const float mag = warp_max(real && b1 != -kInf ? fmaxf(fabsf(b1), b2 == -kInf ? 0.f : fabsf(b2)) : 0.f);
        const float tol = 2.5f * bound(mag);  // two halved sums of two values each
        if (hi != -kInf && !(lo - hi > tol)) {
            const double zd = p.score_fn == MOE_SCORE_SOFTMAX ? row_z<T>(row, p.E, m) : 1.0;
            const uint32_t kept = groups_exact<T>(Row<T>{row, p.bias, p.E, gsz, p.score_fn, m, zd, kFull},
                                                  p.n_group, p.topk_group, shift);
            keep = real && ((kept >> g) & 1u);
        }
        if (!keep) {
#pragma unroll
            for (int j = 0; j < J; ++j) sel[j] = -kInf;
        }
    }

    // The k-th largest of the lanes' maxima is a lower bound of the k-th largest of all. What
    // is not below it (less the error bound) is a candidate: usually k to 2 k elements, one
    // to a lane, of which k rounds of a warp maximum take the chosen in order.
    typedef typename std::conditional<(J > 32), u64, uint32_t>::type Bits;
    auto expert = [&](int j) { return e0 + (j / VEC) * L * VEC + j % VEC; };
    float v1 = sel[0];
#pragma unroll
    for (int j = 1; j < J; ++j) v1 = fmaxf(v1, sel[j]);
    uint32_t lane_key = v1 == -kInf ? 0u : key_of(v1), tau = 0u;
    for (int got = 0; got < p.k;) {
        tau = __reduce_max_sync(kFull, lane_key);
        if (tau == 0u) break;  // fewer lanes with elements than k: every element is a candidate
        got += __popc(__ballot_sync(kFull, lane_key == tau));
        if (lane_key == tau) lane_key = 0u;
    }
    float least = -FLT_MAX;
    if (tau != 0u) {
        least = value_of(tau);
        if (!by_logit) least = fmaxf(least - 2.f * bound(least), -FLT_MAX);  // never the masked
    }
    // the elements not below `from`, as bits and (up to 32 of them) in the warp's list
    Bits avail;
    auto collect = [&](float from) {
        avail = 0;
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (sel[j] >= from) avail |= Bits(1) << j;
        const int mine = J > 32 ? __popcll(avail) : __popc((uint32_t)avail);
        int at = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(kFull, at, o);
            if (lane >= o) at += n;
        }
        const int total = __shfl_sync(kFull, at, 31);
        if (total <= 32) {
            at -= mine;
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (avail & (Bits(1) << j)) list[warp][at++] = make_int2(__float_as_int(sel[j]), expert(j));
        }
        __syncwarp();
        return total;
    };
    const int total = collect(least);

    int my_e = -1;
    uint32_t my_key = 0u, last = 0u;
    auto take = [&](int r, uint32_t key, int e) {  // round r: the largest key, the lowest index among equals
        last = __reduce_max_sync(kFull, key);
        const uint32_t who = __ballot_sync(kFull, key == last);
        int win = __shfl_sync(kFull, e, __ffs(who) - 1);
        if (who & (who - 1)) win = __reduce_min_sync(kFull, key == last ? e : INT_MAX);
        if (lane == r) {
            my_e = win;
            my_key = last;
        }
        return win;
    };
    const bool listed = total <= 32;
    uint32_t k1 = 0u;  // largest key of this lane that is not chosen
    int e1 = INT_MAX;
    if (listed) {
        if (lane < total) {
            const int2 c = list[warp][lane];
            k1 = key_of(__int_as_float(c.x));
            e1 = c.y;
        }
        for (int r = 0; r < min(p.k, total); ++r)
            if (take(r, k1, e1) == e1) k1 = 0u;
    } else {
        // rows of equal scores, or few lanes with many elements each: a lane caches its two
        // best and scans again when both are taken. Within a lane the expert grows with j,
        // so the first of equal values is the lower.
        uint32_t k2;
        int e2;
        Bits bit1, bit2;
        auto refill = [&]() {
            float f1 = -kInf, f2 = -kInf;
            e1 = e2 = INT_MAX;
            bit1 = bit2 = 0;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float v = avail & (Bits(1) << j) ? sel[j] : -kInf;
                const bool first = v > f1, second = v > f2;
                f2 = first ? f1 : (second ? v : f2);
                e2 = first ? e1 : (second ? expert(j) : e2);
                bit2 = first ? bit1 : (second ? Bits(1) << j : bit2);
                f1 = first ? v : f1;
                e1 = first ? expert(j) : e1;
                bit1 = first ? Bits(1) << j : bit1;
            }
            k1 = bit1 ? key_of(f1) : 0u;
            k2 = bit2 ? key_of(f2) : 0u;
        };
        refill();
        for (int r = 0; r < p.k; ++r) {  // total > 32 >= k: there is always one left
            if (take(r, k1, e1) == e1) {
                avail &= ~bit1;
                k1 = k2; e1 = e2; bit1 = bit2;
                k2 = 0u; e2 = INT_MAX; bit2 = 0;
                if (k1 == 0u && avail) refill();
            }
        }
    }
    float my_l = my_e >= 0 ? to_f32<T>(row[my_e]) + 0.0f : 0.f;
    if (!by_logit && total > 0) {
        // values that the bound cannot tell apart and that are not the same number: among
        // the chosen one after the other, and of those left out against the last chosen
        const float my_v = value_of(my_key);
        const float my_b = my_e >= 0 && p.bias ? p.bias[my_e] : 0.f;
        const uint32_t next_key = __shfl_down_sync(kFull, my_key, 1);
        const float next_l = __shfl_down_sync(kFull, my_l, 1), next_b = __shfl_down_sync(kFull, my_b, 1);
        bool near = lane + 1 < p.k && next_key != 0u && my_v - value_of(next_key) <= 2.f * bound(my_v) &&
                    !(next_l == my_l && next_b == my_b);
        const int chosen = min(p.k, total);
        const float last_v = value_of(last), cut = fmaxf(last_v - 2.f * bound(last_v), -FLT_MAX);
        const float ll = __shfl_sync(kFull, my_l, chosen - 1), lb = __shfl_sync(kFull, my_b, chosen - 1);
        auto as_last = [&](int e) {
            return to_f32<T>(row[e]) + 0.0f == ll && (p.bias ? p.bias[e] : 0.f) == lb;
        };
        if (k1 != 0u && value_of(k1) >= cut) {
            if (listed) {
                near |= !as_last(e1);
            } else {
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if ((avail & (Bits(1) << j)) && sel[j] >= cut) near |= !as_last(expert(j));
            }
        }
        if (__any_sync(kFull, near)) {
            const double zd = p.score_fn == MOE_SCORE_SOFTMAX ? row_z<T>(row, p.E, m) : 1.0;
            const uint32_t lanes = __ballot_sync(kFull, keep);
            uint32_t kept = 0u;
            for (int h = 0; h < p.n_group; ++h) kept |= ((lanes >> (h << shift)) & 1u) << h;
            const Row<T> r{row, p.bias, p.E, gsz, p.score_fn, m, zd, kept};
            const int close = listed ? total : collect(cut);
            if (close <= 32) {
                my_e = rank_exact<T>(r, lane < close ? list[warp][lane].y : -1, close);
                if (lane >= p.k) my_e = -1;
            } else {
                my_e = topk_exact<T>(r, p.k);
            }
            my_l = my_e >= 0 ? to_f32<T>(row[my_e]) + 0.0f : 0.f;
        }
    }
    const float w = chosen_weight(my_l, my_e >= 0, p.score_fn, p.norm, m, z);
    if (lane < p.k) {
        p.idx[t * p.k + lane] = my_e;
        p.w[t * p.k + lane] = w * p.rsf;
    }
}

struct RouteBwd {
    const void* logits;
    const int32_t* idx;
    const float* dw;
    void* dl;
    long ld, ldd;
    int T, E, k, norm, score_fn;
    float rsf;
};

// d s_j / d l_j over s_j: sigmoid 1 - s, sqrt-softplus sig(l) / (2 softplus(l)) (1/2 far below
// zero, where both go to exp(l)).
__device__ __forceinline__ float log_slope(float l, int fn) {
    if (fn == MOE_SCORE_SIGMOID) return 1.0f / (1.0f + expf(l));
    const float e = expf(-fabsf(l));
    const float sp = fmaxf(l, 0.0f) + log1pf(e);
    if (l < -40.0f) return 0.5f;
    return (l >= 0.0f ? 1.0f : e) / (1.0f + e) * 0.5f / sp;
}

// One warp per token: lane j works out slot j's gradient, the warp writes the row. Only a
// softmax without renormalisation gives the other experts a gradient (-s_e <g s>) and
// reads the whole row; every other row is zeros and the k values.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) route_bwd_kernel(RouteBwd p) {
    pdl_wait();
    pdl_trigger();
    constexpr int NI = 32 / VEC;
    const int lane = threadIdx.x & 31;
    const long t = (long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    T* out = static_cast<T*>(p.dl) + t * p.ldd;
    const int nvec = p.E / VEC;
    const bool dense = p.score_fn == MOE_SCORE_SOFTMAX && !p.norm;

    // the row's loads go out before the slots', whose logits hang on the indices
    Pack<T, VEC> raw[NI];
    if (dense) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (lane + 32 * i < nvec) raw[i] = reinterpret_cast<const Pack<T, VEC>*>(row)[lane + 32 * i];
    }
    int e = lane < p.k ? p.idx[t * p.k + lane] : -1;
    if (e < 0 || e >= p.E) e = -1;
    const bool valid = e >= 0;
    const float l = valid ? to_f32<T>(row[e]) : 0.f;
    const float g = valid ? p.dw[t * p.k + lane] * p.rsf : 0.f;
    const bool any = __any_sync(kFull, valid);

    float s[NI * VEC];
    float m = 0.f, z = 1.f;
    if (p.score_fn == MOE_SCORE_SOFTMAX) {
        if (dense && any) {
            float top = -kInf;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    s[i * VEC + v] = lane + 32 * i < nvec ? to_f32<T>(raw[i].v[v]) : -kInf;
                    top = fmaxf(top, s[i * VEC + v]);
                }
            }
            m = warp_max(top);
            if (m == -kInf) m = 0.f;  // every expert is masked: all scores are zero
            float zs = 0.f;
#pragma unroll
            for (int j = 0; j < NI * VEC; ++j) {
                s[j] = exp_approx(s[j] - m);
                zs += s[j];
            }
            z = warp_sum(zs);
            if (z == 0.f) z = 1.f;
        } else {
            m = warp_max(valid ? l : -kInf);  // renormalised: a softmax over the chosen
            if (m == -kInf) m = 0.f;
        }
    }
    const float w = chosen_weight(l, valid, p.score_fn, p.norm, m, z);
    const float dot = p.norm || dense ? warp_sum(g * w) : 0.f;
    float d = p.norm ? w * (g - dot) : w * g;
    if (p.score_fn != MOE_SCORE_SOFTMAX) d *= log_slope(l, p.score_fn);
    // an expert in several slots gets the slots' sum, added in slot order
    uint32_t same = 0;
    for (int c = 0; c < p.k; ++c) same |= (__shfl_sync(kFull, e, c) == e ? 1u : 0u) << c;
    if (__any_sync(kFull, valid && (same & (same - 1)))) {
        float sum = 0.f;
        for (int c = 0; c < p.k; ++c) {
            const float o = __shfl_sync(kFull, d, c);
            if ((same >> c) & 1u) sum += o;
        }
        d = sum;
    }
    if (dense) d -= w * dot;

    const float back = dense && any ? -dot / z : 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        if (lane + 32 * i >= nvec) continue;
        Pack<T, VEC> o;
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = dense && any ? s[i * VEC + j] * back : 0.f;
        if constexpr (VEC == 8) {
            *reinterpret_cast<uint4*>(&o) = narrow8<T>(v);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) o.v[j] = from_f32<T>(v[j]);
        }
        reinterpret_cast<Pack<T, VEC>*>(out)[lane + 32 * i] = o;
    }
    __syncwarp();
    if (valid) out[e] = from_f32<T>(d);
}

template <typename T, int VEC, int NI>
void fwd(const RouteParams& p, int L, cudaStream_t st) {
    // a few warps per CTA for small batches, so that they spread over the SMs
    const int warps = p.T >= 16 * num_sms() ? 8 : 2;
    launch_pdl(route_fwd_kernel<T, VEC, NI>, (p.T - 1) / warps + 1, warps * 32, 0, st, p, L);
}

template <typename T>
void fwd_type(const RouteParams& p, bool vec, cudaStream_t st) {
    constexpr int V = kFullVec<T>;
    int L = 32;
    while (L * p.n_group > 32) L >>= 1;
    const int gsz = p.E / p.n_group;
    if (vec) {
        const int ni = (gsz / V + L - 1) / L;
        if (ni <= 1) return fwd<T, V, 1>(p, L, st);
        if (ni <= 2) return fwd<T, V, 2>(p, L, st);
        if (V == 4 && ni <= 3) return fwd<T, V, 3>(p, L, st);
        if (ni <= 4) return fwd<T, V, 4>(p, L, st);
        if (ni <= 8) return fwd<T, V, 8>(p, L, st);
        if (V == 4) return fwd<T, V, 64 / V>(p, L, st);
    }
    const int ni = (gsz + L - 1) / L;
    if (ni <= 4) fwd<T, 1, 4>(p, L, st);
    else if (ni <= 16) fwd<T, 1, 16>(p, L, st);
    else if (ni <= 32) fwd<T, 1, 32>(p, L, st);
    else fwd<T, 1, 64>(p, L, st);
}

}  // namespace

cudaError_t launch_route(const moe_config* c, int dtype, const void* logits, long ld, int T,
                         const float* bias, int32_t* idx, float* w, cudaStream_t st) {
    const RouteParams p{logits, bias, idx, w, ld, T, c->n_routed_experts, c->num_experts_per_tok,
                        c->n_group, c->topk_group, c->norm_topk_prob, c->score_fn,
                        c->routed_scaling_factor};
    const int es = esize(dtype);
    const bool vec = (p.E / p.n_group) % (16 / es) == 0 && rows16(logits, ld, es) && rows16(bias, 4, 4);
    if (dtype == MOE_T_BF16) fwd_type<__nv_bfloat16>(p, vec, st);
    else if (dtype == MOE_T_F16) fwd_type<__half>(p, vec, st);
    else fwd_type<float>(p, vec, st);
    return cudaGetLastError();
}

cudaError_t launch_route_backward(const moe_config* c, int dtype, const void* logits, long ld, int T,
                                  const int32_t* idx, const float* dw, void* dl, long ldd,
                                  cudaStream_t st) {
    const RouteBwd p{logits, idx, dw, dl, ld, ldd, T, c->n_routed_experts, c->num_experts_per_tok,
                     c->norm_topk_prob, c->score_fn, c->routed_scaling_factor};
    const int es = esize(dtype);
    const bool vec = p.E % (16 / es) == 0 && rows16(logits, ld, es) && rows16(dl, ldd, es);
    const unsigned grid = (unsigned)((T - 1) / 8 + 1);
    if (dtype == MOE_T_BF16) {
        if (vec) launch_pdl(route_bwd_kernel<__nv_bfloat16, 8>, grid, 256, 0, st, p);
        else launch_pdl(route_bwd_kernel<__nv_bfloat16, 1>, grid, 256, 0, st, p);
    } else if (dtype == MOE_T_F16) {
        if (vec) launch_pdl(route_bwd_kernel<__half, 8>, grid, 256, 0, st, p);
        else launch_pdl(route_bwd_kernel<__half, 1>, grid, 256, 0, st, p);
    } else {
        if (vec) launch_pdl(route_bwd_kernel<float, 4>, grid, 256, 0, st, p);
        else launch_pdl(route_bwd_kernel<float, 1>, grid, 256, 0, st, p);
    }
    return cudaGetLastError();
}

}  // namespace moe
