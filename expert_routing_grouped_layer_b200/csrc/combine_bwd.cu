// combine_bwd.cu -- gradient of the weighted combine
// ("DeepSeek V3架构拆解：Kimi-K2-Thinking-NVFP4的MLA注意力与MoE路由实现原理", 三.4):
// out[t] = sum_j w[t][j] y[row(t, j)] + shared, so
//   dy[row(t, j)] = w[t][j] dout[t],   dw[t][j] = <dout[t], y[row(t, j)]>.
//
// Bound by HBM: every expert row is read once and its gradient written once; a token's
// dout is read from HBM once and by its k pairs from L1. One warp per pair, so no
// barrier stands between a row's loads and stores, and the dot product's order is fixed.
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

template <bool DOT>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const uint4* __restrict__ dout,
                                                          const uint4* __restrict__ y,
                                                          const int32_t* __restrict__ row_of,
                                                          const float* __restrict__ w, long N, int k,
                                                          int HV, uint4* __restrict__ dy,
                                                          float* __restrict__ dw) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long pair = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (pair >= N) return;
    const long row = row_of[pair];
    if (row < 0 || row >= N) {  // a pair without a row
        if (DOT && lane == 0) dw[pair] = 0.f;
        return;
    }
    const float wj = w[pair];
    const uint4* a = dout + (pair / k) * HV;
    const uint4* b = y + row * HV;
    uint4* o = dy + row * HV;
    float dot = 0.f;
    constexpr int U = 4;
    for (int c0 = lane; c0 < HV; c0 += 32 * U) {
        uint4 va[U], vb[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int c = c0 + 32 * i;
            if (c < HV) {
                va[i] = a[c];
                vb[i] = DOT ? ld_stream(b + c) : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int c = c0 + 32 * i;
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
    if (DOT) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        if (lane == 0) dw[pair] = dot;
    }
}

}  // namespace

cudaError_t launch_combine_backward(const void* dout, const void* y, const int32_t* row_of,
                                    const float* w, int T, int k, int H, void* dy, float* dw,
                                    cudaStream_t st) {
    const long N = (long)T * k;
    const unsigned grid = (unsigned)((N + 7) / 8);
    const auto* a = static_cast<const uint4*>(dout);
    const auto* b = static_cast<const uint4*>(y);
    auto* o = static_cast<uint4*>(dy);
    if (dw) launch_pdl(combine_bwd_kernel<true>, grid, 256, 0, st, a, b, row_of, w, N, k, H / 8, o, dw);
    else launch_pdl(combine_bwd_kernel<false>, grid, 256, 0, st, a, b, row_of, w, N, k, H / 8, o, dw);
    return cudaGetLastError();
}

}  // namespace moe
