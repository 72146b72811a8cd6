// norm.cu -- layer norm and RMS norm of rows, forward and backward.
//
//   forward   y_h = (x_h - mean) r w_h + b_h,  r = 1 / sqrt(sum (x - mean)^2 / H + eps)
//             (RMS norm: mean = 0; the norm in front of the router,
//             "DeepSeek V3架构拆解：Kimi-K2-Thinking-NVFP4的MLA注意力与MoE路由实现原理", 三)
//   backward  n = (x - mean) r, g = w dy:
//             dx = r (g - <g> - n <g n>), <.> the mean over h (RMS norm: no <g>),
//             dw = sum_t dy n, db = sum_t dy.
//
// All of it is bound by HBM: one read of every input row and one write of every
// output row, ~10 operations an element. A row lives in the registers of one CTA
// from its load to its store, so the mean, the centred squares (two reductions, no
// cancellation) and the output come from one read.
#include <algorithm>

#include "internal.h"
#include "sm100.cuh"
#include "types.cuh"

namespace moe {

namespace {

// Sum of (a, b) over the CTA, the same bits in every thread: warp butterflies, then
// each warp butterflies the warps' sums. `slot` alternates between two buffers, so
// one barrier a call is enough.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2 (*buf)[32], int& slot) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    const int nw = blockDim.x >> 5;
    if (nw == 1) return make_float2(a, b);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[slot][warp] = make_float2(a, b);
    __syncthreads();
    float2 s = lane < nw ? buf[slot][lane] : make_float2(0.f, 0.f);
    slot ^= 1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    }
    return s;
}

struct NormFwd {
    const void* x;
    void* y;
    const float *w, *b;
    float *mean, *rstd;
    long ldx, ldy;
    int T, H;
    float eps;
};

// One row per CTA; thread i holds the vectors i, i + blockDim, ... of it.
template <typename T, int VEC, int NV, int MAXT, bool LAYER>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(NormFwd p) {
    pdl_wait();
    pdl_trigger();
    __shared__ float2 buf[2][32];
    int slot = 0;
    const int nvec = p.H / VEC;
    const float h = (float)p.H;
    const long t = blockIdx.x;
    const Pack<T, VEC>* x = reinterpret_cast<const Pack<T, VEC>*>(static_cast<const T*>(p.x) + t * p.ldx);
    Pack<T, VEC> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nvec) raw[i] = x[c];
    }
    float v[NV * VEC];
    float sum = 0.f, sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool in = threadIdx.x + i * blockDim.x < nvec;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            v[i * VEC + j] = in ? to_f32<T>(raw[i].v[j]) : 0.f;
            sum += v[i * VEC + j];
        }
    }
    float mean = 0.f;
    if (LAYER) mean = block_sum2(sum, 0.f, buf, slot).x / h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool in = threadIdx.x + i * blockDim.x < nvec;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float d = in ? v[i * VEC + j] - mean : 0.f;
            v[i * VEC + j] = d;
            sq += d * d;
        }
    }
    const float var = block_sum2(sq, 0.f, buf, slot).x / h;
    const float r = 1.0f / sqrtf(var + p.eps);
    if (threadIdx.x == 0) {
        if (LAYER && p.mean) p.mean[t] = mean;
        if (p.rstd) p.rstd[t] = r;
    }
    Pack<T, VEC>* y = reinterpret_cast<Pack<T, VEC>*>(static_cast<T*>(p.y) + t * p.ldy);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
        float w[VEC], b[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            w[j] = p.w ? p.w[c * VEC + j] : 1.f;
            b[j] = p.b ? p.b[c * VEC + j] : 0.f;
        }
        Pack<T, VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) o.v[j] = from_f32<T>(fmaf(v[i * VEC + j] * r, w[j], b[j]));
        y[c] = o;
    }
}

struct NormBwd {
    const void *dy, *x;
    void* dx;
    const float *w, *mean, *rstd;
    float* part;  // [grid][2][H] column sums of this CTA's rows, or null
    long lddy, ldx, lddx;
    int T, H;
};

// Rows blockIdx.x, blockIdx.x + grid, ...: the CTA keeps its columns' weight and the
// two column sums in registers over all its rows, and loads the next row while it
// works on one.
template <typename T, int VEC, int NV, int MAXT, bool LAYER>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(NormBwd p) {
    pdl_wait();
    pdl_trigger();
    __shared__ float2 buf[2][32];
    int slot = 0;
    const int nvec = p.H / VEC;
    const float inv_h = 1.0f / (float)p.H;
    float w[NV * VEC], sw[NV * VEC], sb[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            w[i * VEC + j] = c < nvec ? (p.w ? p.w[c * VEC + j] : 1.f) : 0.f;
            sw[i * VEC + j] = sb[i * VEC + j] = 0.f;
        }
    }
    Pack<T, VEC> rx[NV], rg[NV];
    float mean = 0.f, r = 0.f;
    auto load = [&](long t) {
        const Pack<T, VEC>* x = reinterpret_cast<const Pack<T, VEC>*>(static_cast<const T*>(p.x) + t * p.ldx);
        const Pack<T, VEC>* g = reinterpret_cast<const Pack<T, VEC>*>(static_cast<const T*>(p.dy) + t * p.lddy);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < nvec) {
                rx[i] = x[c];
                rg[i] = g[c];
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) rx[i].v[j] = rg[i].v[j] = from_f32<T>(0.f);
            }
        }
        if (LAYER) mean = p.mean[t];
        r = p.rstd[t];
    };
    if ((long)blockIdx.x < p.T) load(blockIdx.x);
    for (long t = blockIdx.x; t < p.T; t += gridDim.x) {
        float n[NV * VEC], g[NV * VEC];
        float s1 = 0.f, s2 = 0.f;
        const float rt = r;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = threadIdx.x + i * blockDim.x < nvec;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int e = i * VEC + j;
                const float dy = to_f32<T>(rg[i].v[j]);
                n[e] = in ? (to_f32<T>(rx[i].v[j]) - mean) * rt : 0.f;
                sw[e] = fmaf(dy, n[e], sw[e]);
                if (LAYER) sb[e] += dy;
                g[e] = dy * w[e];
                s1 += g[e];
                s2 = fmaf(g[e], n[e], s2);
            }
        }
        if (t + gridDim.x < p.T) load(t + gridDim.x);
        const float2 s = block_sum2(s1, s2, buf, slot);
        const float c1 = LAYER ? s.x * inv_h : 0.f, c2 = s.y * inv_h;
        if (p.dx) {
            Pack<T, VEC>* dx = reinterpret_cast<Pack<T, VEC>*>(static_cast<T*>(p.dx) + t * p.lddx);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c >= nvec) continue;
                Pack<T, VEC> o;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int e = i * VEC + j;
                    o.v[j] = from_f32<T>(rt * (g[e] - c1 - n[e] * c2));
                }
                dx[c] = o;
            }
        }
    }
    if (!p.part) return;
    float* part = p.part + (size_t)blockIdx.x * 2 * p.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            part[c * VEC + j] = sw[i * VEC + j];
            if (LAYER) part[p.H + c * VEC + j] = sb[i * VEC + j];
        }
    }
}

// dw and db from the CTAs' column sums, added in a fixed order: 32 columns per CTA,
// 32 slices of the partial rows, then the slices.
__global__ void __launch_bounds__(1024) norm_param_kernel(const float* __restrict__ part, int n_part,
                                                          int H, float* dw, float* db) {
    pdl_wait();
    pdl_trigger();
    __shared__ float acc[32][33];
    const int which = blockIdx.y;  // 0: dw, 1: db
    float* out = which ? db : dw;
    if (!out) return;
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < H) {
        const float* src = part + (size_t)which * H + c;
#pragma unroll 4
        for (int i = slice; i < n_part; i += 32) s += src[(size_t)i * 2 * H];
    }
    acc[slice][lane] = s;
    __syncthreads();
    // warp `slice` sums column `slice` of the tile over the slices
    float v = acc[lane][slice];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int col = blockIdx.x * 32 + slice;
    if (lane == 0 && col < H) out[col] = v;
}

inline int round32(int v) { return (v + 31) / 32 * 32; }

template <typename T, int VEC, int NV, int MAXT>
void fwd(int layer, const NormFwd& p, cudaStream_t st) {
    const int threads = std::max(32, round32((p.H / VEC + NV - 1) / NV));
    if (layer) launch_pdl(norm_fwd_kernel<T, VEC, NV, MAXT, true>, p.T, threads, 0, st, p);
    else launch_pdl(norm_fwd_kernel<T, VEC, NV, MAXT, false>, p.T, threads, 0, st, p);
}

template <typename T>
void fwd_type(int layer, const NormFwd& p, bool vec, cudaStream_t st) {
    constexpr int V = kFullVec<T>;
    if (!vec) {
        if (p.H <= 4096) fwd<T, 1, 4, 1024>(layer, p, st);
        else fwd<T, 1, 16, 1024>(layer, p, st);
        return;
    }
    const int nvec = p.H / V;
    // few rows: as many threads as a row takes, for the shortest row time; many
    // rows: fewer threads with more loads each
    if (p.T < 2 * num_sms() && nvec <= 1024) fwd<T, V, 1, 1024>(layer, p, st);
    else if constexpr (sizeof(T) == 4) fwd<T, V, 4, 1024>(layer, p, st);
    else fwd<T, V, 4, 512>(layer, p, st);
}

// CTAs that share an SM: about 1024 threads' worth of rows in flight.
int bwd_grid(int T, int threads) {
    const long per_sm = std::min(16, std::max(1, 1024 / threads));
    return (int)std::min<long>(T, per_sm * num_sms());
}
// no variant puts more than 16 elements of a row on a thread
constexpr int kMaxPerThread = 16;

template <typename T, int VEC, int NV, int MAXT>
void bwd(int layer, NormBwd p, float* dw, float* db, cudaStream_t st) {
    static_assert(VEC * NV <= kMaxPerThread, "the workspace's grid bound");
    const int threads = std::max(32, round32((p.H / VEC + NV - 1) / NV));
    const int grid = bwd_grid(p.T, threads);
    if (layer) launch_pdl(norm_bwd_kernel<T, VEC, NV, MAXT, true>, grid, threads, 0, st, p);
    else launch_pdl(norm_bwd_kernel<T, VEC, NV, MAXT, false>, grid, threads, 0, st, p);
    if (p.part)
        launch_pdl(norm_param_kernel, dim3((p.H + 31) / 32, db ? 2 : 1), 1024, 0, st,
                   (const float*)p.part, grid, p.H, dw, db);
}

template <typename T>
void bwd_type(int layer, const NormBwd& p, bool vec, float* dw, float* db, cudaStream_t st) {
    constexpr int V = kFullVec<T>;
    if (!vec) {
        if (p.H <= 4096) bwd<T, 1, 4, 1024>(layer, p, dw, db, st);
        else bwd<T, 1, 16, 1024>(layer, p, dw, db, st);
        return;
    }
    if constexpr (sizeof(T) == 4) bwd<T, V, 4, 1024>(layer, p, dw, db, st);
    else if (p.H <= 8192) bwd<T, V, 2, 512>(layer, p, dw, db, st);
    else bwd<T, V, 2, 1024>(layer, p, dw, db, st);
}

inline bool rows16(const void* p, long ld, int es) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * es) % 16 == 0);
}

}  // namespace

// one pair of column-sum rows per CTA of the widest grid
size_t norm_backward_ws(int T, int H) {
    const int threads = std::max(32, round32((H + kMaxPerThread - 1) / kMaxPerThread));
    return (size_t)bwd_grid(T, threads) * 2 * H * 4;
}

cudaError_t launch_norm_fwd(int kind, int dtype, const void* x, long ldx, int T, int H, const float* w,
                            const float* b, float eps, void* y, long ldy, float* mean, float* rstd,
                            cudaStream_t st) {
    const NormFwd p{x, y, w, b, mean, rstd, ldx, ldy, T, H, eps};
    const int es = esize(dtype), layer = kind == MOE_NORM_LAYER;
    const bool vec = H % (16 / es) == 0 && rows16(x, ldx, es) && rows16(y, ldy, es);
    if (dtype == MOE_T_BF16) fwd_type<__nv_bfloat16>(layer, p, vec, st);
    else if (dtype == MOE_T_F16) fwd_type<__half>(layer, p, vec, st);
    else fwd_type<float>(layer, p, vec, st);
    return cudaGetLastError();
}

cudaError_t launch_norm_bwd(int kind, int dtype, const void* dy, long lddy, const void* x, long ldx,
                            int T, int H, const float* w, const float* mean, const float* rstd,
                            void* dx, long lddx, float* dw, float* db, float* part, cudaStream_t st) {
    if (T == 0) {  // no rows: the sums are zero
        if (dw || db)
            launch_pdl(norm_param_kernel, dim3((H + 31) / 32, 2), 1024, 0, st, (const float*)nullptr, 0, H,
                       dw, db);
        return cudaGetLastError();
    }
    const NormBwd p{dy, x, dx, w, mean, rstd, (dw || db) ? part : nullptr, lddy, ldx, lddx, T, H};
    const int es = esize(dtype), layer = kind == MOE_NORM_LAYER;
    const bool vec = H % (16 / es) == 0 && rows16(x, ldx, es) && rows16(dy, lddy, es) && rows16(dx, lddx, es);
    if (dtype == MOE_T_BF16) bwd_type<__nv_bfloat16>(layer, p, vec, dw, db, st);
    else if (dtype == MOE_T_F16) bwd_type<__half>(layer, p, vec, dw, db, st);
    else bwd_type<float>(layer, p, vec, dw, db, st);
    return cudaGetLastError();
}

}  // namespace moe
