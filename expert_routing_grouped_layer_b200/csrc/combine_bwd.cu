// combine_bwd.cu -- gradient of the weighted combine
// ("DeepSeek V3架构拆解：Kimi-K2-Thinking-NVFP4的MLA注意力与MoE路由实现原理", 三.4):
// out[t] = sum_j w[t][j] y[row(t, j)] + shared, so
//   dy[row(t, j)] = w[t][j] dout[t],   dw[t][j] = <dout[t], y[row(t, j)]>.
//
// Bound by HBM: every expert row is read once and its gradient written once; a token's
// dout is read from HBM once and by its k pairs from L1. One warp per pair (eight pairs a
// CTA), so no barrier stands between a row's loads and stores; with too few pairs to give
// every SM 32 warps, four warps share a pair (96 tokens x 6, H = 7168: 6.3 -> 4.1 us). The
// dot product's order is fixed either way. 4096 tokens x 8, H = 7168: 158 us, 0.97 of
// measured HBM.
#include <cuda_bf16.h>

#include "internal.h"
#include "sm100.cuh"

namespace moe {

namespace {

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ float2 bf2(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// dot += <a, b>, and w * a rounded to bf16
__device__ __forceinline__ uint32_t mul_dot(uint32_t a, uint32_t b, float w, float& dot) {
    const float2 x = bf2(a), y = bf2(b);
    dot = fmaf(x.x, y.x, dot);
    dot = fmaf(x.y, y.y, dot);
    const __nv_bfloat162 r = __floats2bfloat162_rn(w * x.x, w * x.y);
    return *reinterpret_cast<const uint32_t*>(&r);
}

// WPP: warps per pair, 1 or 4; a CTA has 8 / WPP pairs.
template <bool DOT, int WPP>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const uint4* __restrict__ dout,
                                                          const uint4* __restrict__ y,
                                                          const int32_t* __restrict__ row_of,
                                                          const float* __restrict__ w, long N, int k,
                                                          int HV, uint4* __restrict__ dy,
                                                          float* __restrict__ dw) {
    pdl_wait();
    pdl_trigger();
    __shared__ float part[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long pair = (long)blockIdx.x * (8 / WPP) + warp / WPP;
    const bool in = pair < N;
    const long row = in ? row_of[pair] : -1;
    float dot = 0.f;
    if (row >= 0 && row < N) {  // else: a pair without a row
        const float wj = w[pair];
        const uint4* a = dout + (pair / k) * HV;
        const uint4* b = y + row * HV;
        uint4* o = dy + row * HV;
        constexpr int U = 4, STEP = 32 * WPP;
        for (int c0 = (warp % WPP) * 32 + lane; c0 < HV; c0 += STEP * U) {
            uint4 va[U], vb[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int c = c0 + STEP * i;
                if (c < HV) {
                    va[i] = a[c];
                    vb[i] = DOT ? ld_stream(b + c) : make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int c = c0 + STEP * i;
                if (c >= HV) continue;
                float d = 0.f;
                uint4 r;
                r.x = mul_dot(va[i].x, vb[i].x, wj, d);
                r.y = mul_dot(va[i].y, vb[i].y, wj, d);
                r.z = mul_dot(va[i].z, vb[i].z, wj, d);
                r.w = mul_dot(va[i].w, vb[i].w, wj, d);
                dot += d;
                o[c] = r;
            }
        }
    }
    if constexpr (DOT) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        if constexpr (WPP == 1) {
            if (in && lane == 0) dw[pair] = dot;
        } else {
            if (lane == 0) part[warp] = dot;
            __syncthreads();
            if (in && lane == 0 && warp % WPP == 0) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < WPP; ++i) s += part[warp + i];
                dw[pair] = s;
            }
        }
    }
}

template <bool DOT, int WPP>
void launch(const void* dout, const void* y, const int32_t* row_of, const float* w, long N, int k, int H,
            void* dy, float* dw, cudaStream_t st) {
    constexpr int pairs = 8 / WPP;
    launch_pdl(combine_bwd_kernel<DOT, WPP>, (unsigned)((N + pairs - 1) / pairs), 256, 0, st,
               static_cast<const uint4*>(dout), static_cast<const uint4*>(y), row_of, w, N, k, H / 8,
               static_cast<uint4*>(dy), dw);
}

}  // namespace

cudaError_t launch_combine_backward(const void* dout, const void* y, const int32_t* row_of,
                                    const float* w, int T, int k, int H, void* dy, float* dw,
                                    cudaStream_t st) {
    const long N = (long)T * k;
    const bool few = N < 32L * num_sms();
    if (dw) {
        if (few) launch<true, 4>(dout, y, row_of, w, N, k, H, dy, dw, st);
        else launch<true, 1>(dout, y, row_of, w, N, k, H, dy, dw, st);
    } else {
        if (few) launch<false, 4>(dout, y, row_of, w, N, k, H, dy, dw, st);
        else launch<false, 1>(dout, y, row_of, w, N, k, H, dy, dw, st);
    }
    return cudaGetLastError();
}

}  // namespace moe
