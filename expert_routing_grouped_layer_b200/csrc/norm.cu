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
// output row, ~10 operations an element. A row stays in one CTA from its load to its
// store, so the mean, the centred squares (two reductions, no cancellation) and the
// output come from one read. Kernels, by the rows' shape:
//   norm_fwd_kernel         fewer rows than 2 per SM: a row per CTA, straight from registers
//                           (128 x 7168: 2.9 us);
//   norm_*_ring_kernel      many rows on the 16-byte grid: persistent CTAs behind a ring of
//                           rows in shared memory (16384 x 7168 bf16 forward 79 us, 0.90 of
//                           measured HBM; 8192 x 7168 backward 65 us, 0.83, of which 5 us
//                           are the column sums' second kernel);
//   norm_*_ragged_kernel    rows off the grid (8192 x 7166: forward 81 us, backward 150 us;
//                           bound by their instructions).
// The arithmetic runs two elements to an instruction (packed fp32): with single operations
// the forward pass was bound by instruction issue (102 us).
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "internal.h"
#include "row_chunks.h"
#include "sm100.cuh"
#include "types.cuh"

namespace moe {

namespace {

// Sum over the CTA, the same bits in every thread: warp butterflies, then each warp
// butterflies the warps' sums. `slot` alternates between two buffers, so one barrier a
// call is enough.
__device__ __forceinline__ float block_sum(float a, float (*buf)[32], int& slot) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[slot][warp] = a;
    __syncthreads();
    float s = lane < nw ? buf[slot][lane] : 0.f;
    slot ^= 1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// VEC values of a parameter row from element c * VEC on, or `none` without the row.
template <int VEC>
__device__ __forceinline__ void load_param(float* v, const float* row, int c, float none) {
    if (!row) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = none;
    } else if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(row + c * VEC + j);
            v[j] = f.x; v[j + 1] = f.y; v[j + 2] = f.z; v[j + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = row[c * VEC + j];
    }
}

template <int P>
__device__ __forceinline__ void param_pairs(f32x2 (&v)[P], const float* row, int c, float none) {
    float f[2 * P];
    load_param<2 * P>(f, row, c, none);
#pragma unroll
    for (int j = 0; j < P; ++j) v[j] = pack2(f[2 * j], f[2 * j + 1]);
}

// s / H as s times 1 / H, which is held as the sum of two fp32 numbers: nearly always the rounded
// quotient (a constant row's mean is the constant), and infinite for an infinite s, since neither
// part is negative or zero. (Brisebarre and Muller, "Correctly rounded multiplication by arbitrary
// precision constants", 2008. With a division, whose rare path is a call, the forward pass of
// 16384 x 7168 took 98 us.)
struct InvH {
    float hi, lo;
    explicit InvH(int H) {
        const double r = 1.0 / H;
        hi = (float)r;
        if (hi > r) hi = std::nextafterf(hi, 0.0f);
        lo = std::max((float)(r - hi), FLT_MIN);
    }
    __device__ __forceinline__ float of(float s) const { return fmaf(s, hi, s * lo); }
};

struct NormFwd {
    const void* x;
    void* y;
    const float *w, *b;
    float *mean, *rstd;
    long ldx, ldy;
    int T, H;
    float eps;
    InvH over_h;
};

// One row per CTA; thread i holds the vectors i, i + blockDim, ... of it.
template <typename T, int VEC, int NV, int MAXT, bool LAYER>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(NormFwd p) {
    pdl_wait();
    pdl_trigger();
    __shared__ float buf[2][32];
    int slot = 0;
    const int nvec = p.H / VEC;
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
    if (LAYER) mean = p.over_h.of(block_sum(sum, buf, slot));
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
    const float r = rsqrtf(p.over_h.of(block_sum(sq, buf, slot)) + p.eps);
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
        load_param<VEC>(w, p.w, c, 1.f);
        load_param<VEC>(b, p.b, c, 0.f);
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
    InvH over_h;
};

// ------------------------------------------------------------------ rings of rows
// Many rows of 16-byte vectors: persistent CTAs take rows blockIdx.x, + grid, ... and
// copy S - 1 rows ahead into shared memory with cp.async. A thread copies, and later
// reads, its own vectors only, so the ring needs no barrier; the loads of the next rows
// stay in flight during a row's reductions, which registers alone did not allow.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// FULL: every thread holds NV vectors of a row.
template <typename T, int NV, int S, int MAXT, int MINB, bool LAYER, bool FULL>
__global__ void __launch_bounds__(MAXT, MINB) norm_fwd_ring_kernel(NormFwd p) {
    pdl_wait();
    pdl_trigger();
    constexpr int P = kPairs<T>;
    extern __shared__ uint4 ring[];
    __shared__ float buf[2][32];
    int slot = 0;
    const int nvec = p.H / (2 * P), tid = threadIdx.x, nt = blockDim.x;
    f32x2 w[NV][P], b[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * nt;
        if (FULL || c < nvec) {
            param_pairs<P>(w[i], p.w, c, 1.f);
            param_pairs<P>(b[i], p.b, c, 0.f);
        }
    }
    auto copy = [&](long t, uint4* to) {
        if (t < p.T) {
            const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + t * p.ldx) + tid;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (FULL || tid + i * nt < nvec) cp_async16(to + tid + i * nt, x + i * nt);
        }
        cp_async_commit();
    };
    const long step = gridDim.x;
    long t = blockIdx.x;
#pragma unroll
    for (int j = 0; j < S - 1; ++j) copy(t + j * step, ring + j * nvec);
    int st = 0, ahead = S - 1;
    for (; t < p.T; t += step) {
        copy(t + (S - 1) * step, ring + ahead * nvec);
        cp_async_wait<S - 1>();
        f32x2 v[NV][P];
        f32x2 sum = pack2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!FULL && tid + i * nt >= nvec) continue;
            widen<T>(ring[st * nvec + tid + i * nt], v[i]);
            if (LAYER) {
#pragma unroll
                for (int j = 0; j < P; ++j) sum = add2(sum, v[i][j]);
            }
        }
        const float mean = LAYER ? p.over_h.of(block_sum(sum2(sum), buf, slot)) : 0.f;
        const f32x2 minus = pack2(-mean, -mean);
        f32x2 sq = pack2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!FULL && tid + i * nt >= nvec) continue;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if (LAYER) v[i][j] = add2(v[i][j], minus);
                sq = fma2(v[i][j], v[i][j], sq);
            }
        }
        const float r = rsqrtf(p.over_h.of(block_sum(sum2(sq), buf, slot)) + p.eps);
        if (tid == 0) {
            if (LAYER && p.mean) p.mean[t] = mean;
            if (p.rstd) p.rstd[t] = r;
        }
        const f32x2 r2 = pack2(r, r);
        uint4* y = reinterpret_cast<uint4*>(static_cast<T*>(p.y) + t * p.ldy) + tid;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!FULL && tid + i * nt >= nvec) continue;
#pragma unroll
            for (int j = 0; j < P; ++j) v[i][j] = fma2(mul2(v[i][j], r2), w[i][j], b[i][j]);
            y[i * nt] = narrow<T>(v[i]);
        }
        if (++st == S) st = 0;
        if (++ahead == S) ahead = 0;
    }
}

// Sums over the CTA of N values (2 or 4), the same bits in every thread. Within a warp the
// values share the butterfly: log2 N exchanges leave each lane one value's partial sum
// (value lane % N). Then every warp adds the warps' sums, 32 / N lanes per value.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*buf)[N * 32], int& slot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < N; o <<= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < N / 2 / o; ++i) {
            const float keep = up ? v[2 * i + 1] : v[2 * i], give = up ? v[2 * i] : v[2 * i + 1];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    float x = v[0];
#pragma unroll
    for (int o = N; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (nw > 1) {
        if (lane < N) buf[slot][N * warp + lane] = x;
        __syncthreads();
        x = 0.f;
        for (int i = lane; i < N * nw; i += 32) x += buf[slot][i];
        slot ^= 1;
#pragma unroll
        for (int o = N; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, x, i);
}

// R rows at a time, so that one reduction serves them all and its latency is paid once. The
// column sums and the weight stay in registers; x and dy are read from the ring twice, before
// and after the rows' sums are known.
// GROUPED: rows that one warp holds. A CTA's warps (blockDim.y) have rows of their own and add
// their column sums in shared memory, so that fewer partial rows are left for the second kernel
// (16384 x 64 bf16: 17.4 us with a CTA per warp, 10.6 us so).
template <typename T, int NV, int R, int S, int MAXT, bool LAYER, bool FULL, bool GROUPED>
__global__ void __launch_bounds__(MAXT, 1) norm_bwd_ring_kernel(NormBwd p) {
    pdl_wait();
    pdl_trigger();
    constexpr int P = kPairs<T>;
    extern __shared__ uint4 rings[];  // per group of threads [S][R rows][x, dy][nvec]
    __shared__ float buf[2][2 * R * 32];
    int slot = 0;
    const int nvec = p.H / (2 * P), tid = threadIdx.x, nt = blockDim.x;
    const int group = GROUPED ? threadIdx.y : 0, groups = GROUPED ? blockDim.y : 1;
    uint4* ring = GROUPED ? rings + group * (S * R * 2 * nvec) : rings;
    f32x2 w[NV][P], sw[NV][P], sb[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * nt;
        if (FULL || c < nvec) param_pairs<P>(w[i], p.w, c, 1.f);
#pragma unroll
        for (int j = 0; j < P; ++j) sw[i][j] = sb[i][j] = pack2(0.f, 0.f);
    }
    auto copy = [&](long t, uint4* to) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            if (t + q < p.T) {
                const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + (t + q) * p.ldx) + tid;
                const uint4* g = reinterpret_cast<const uint4*>(static_cast<const T*>(p.dy) + (t + q) * p.lddy) + tid;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (!FULL && tid + i * nt >= nvec) continue;
                    cp_async16(to + 2 * q * nvec + tid + i * nt, x + i * nt);
                    cp_async16(to + (2 * q + 1) * nvec + tid + i * nt, g + i * nt);
                }
            }
        }
        cp_async_commit();
    };
    const long step = R * (long)gridDim.x * groups;
    long t = R * ((long)blockIdx.x * groups + group);
#pragma unroll
    for (int j = 0; j < S - 1; ++j) copy(t + j * step, ring + 2 * R * j * nvec);
    int st = 0, ahead = S - 1;
    float mean[R], r[R];
    auto stats = [&](long t) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            if (t + q < p.T) {
                if (LAYER) mean[q] = p.mean[t + q];
                r[q] = p.rstd[t + q];
            } else {
                mean[q] = r[q] = 0.f;
            }
        }
    };
    stats(t);
    for (; t < p.T; t += step) {
        copy(t + (S - 1) * step, ring + 2 * R * ahead * nvec);
        f32x2 minus[R], r2[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            minus[q] = pack2(-mean[q], -mean[q]);
            r2[q] = pack2(r[q], r[q]);
        }
        stats(t + step);
        cp_async_wait<S - 1>();
        const uint4* rows = ring + 2 * R * st * nvec + tid;
        float s[2 * R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            s[2 * q] = s[2 * q + 1] = 0.f;
            if (t + q >= p.T) continue;
            const uint4* rx = rows + 2 * q * nvec;
            f32x2 a1 = pack2(0.f, 0.f), a2 = pack2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!FULL && tid + i * nt >= nvec) continue;
                f32x2 n[P], g[P];
                widen<T>(rx[i * nt], n);
                widen<T>(rx[nvec + i * nt], g);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    n[j] = mul2(LAYER ? add2(n[j], minus[q]) : n[j], r2[q]);
                    sw[i][j] = fma2(g[j], n[j], sw[i][j]);
                    if (LAYER) sb[i][j] = add2(sb[i][j], g[j]);
                    g[j] = mul2(g[j], w[i][j]);
                    if (LAYER) a1 = add2(a1, g[j]);
                    a2 = fma2(g[j], n[j], a2);
                }
            }
            s[2 * q] = sum2(a1);
            s[2 * q + 1] = sum2(a2);
        }
        if (p.dx) {
            block_sums<2 * R>(s, buf, slot);
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (t + q >= p.T) continue;
                const float c1 = -p.over_h.of(s[2 * q]), c2 = -p.over_h.of(s[2 * q + 1]);
                const f32x2 m1 = pack2(c1, c1), m2 = pack2(c2, c2);
                const uint4* rx = rows + 2 * q * nvec;
                uint4* dx = reinterpret_cast<uint4*>(static_cast<T*>(p.dx) + (t + q) * p.lddx) + tid;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (!FULL && tid + i * nt >= nvec) continue;
                    f32x2 n[P], g[P];
                    widen<T>(rx[i * nt], n);
                    widen<T>(rx[nvec + i * nt], g);
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        n[j] = mul2(LAYER ? add2(n[j], minus[q]) : n[j], r2[q]);
                        g[j] = LAYER ? fma2(g[j], w[i][j], m1) : mul2(g[j], w[i][j]);
                        g[j] = mul2(r2[q], fma2(n[j], m2, g[j]));
                    }
                    dx[i * nt] = narrow<T>(g);
                }
            }
        }
        if (++st == S) st = 0;
        if (++ahead == S) ahead = 0;
    }
    if (!p.part) return;
    float* part = p.part + (size_t)blockIdx.x * 2 * p.H;
    // one group writes its sums out; several add theirs, in order, in shared memory first
    float* sums = part;
    if constexpr (GROUPED) {
        cp_async_wait<0>();
        __syncthreads();
        sums = reinterpret_cast<float*>(rings) + group * 2 * p.H;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * nt;
        if (!FULL && c >= nvec) continue;
#pragma unroll
        for (int j = 0; j < P; j += 2) {
            const float2 a = unpack2(sw[i][j]), b = unpack2(sw[i][j + 1]);
            *reinterpret_cast<float4*>(sums + (c * P + j) * 2) = make_float4(a.x, a.y, b.x, b.y);
            if (LAYER) {
                const float2 d = unpack2(sb[i][j]), e = unpack2(sb[i][j + 1]);
                *reinterpret_cast<float4*>(sums + p.H + (c * P + j) * 2) = make_float4(d.x, d.y, e.x, e.y);
            }
        }
    }
    if constexpr (GROUPED) {
        __syncthreads();
        const float* all = reinterpret_cast<const float*>(rings);
        for (int c = group * nt + tid; c < (LAYER ? 2 : 1) * p.H; c += nt * groups) {
            float v = 0.f;
            for (int g = 0; g < groups; ++g) v += all[g * 2 * p.H + c];
            part[c] = v;
        }
    }
}

// ------------------------------------------------------------------ rows off the 16-byte grid
// Rows whose length, stride or base is not a multiple of 16 bytes. Global memory still moves
// in aligned 16-byte chunks (a row's first and last chunk element by element), through shared
// memory, where the row keeps its own offset; threads work on elements tid, tid + threads, ...
// (consecutive lanes on consecutive elements: no bank conflicts at any offset). Element
// accesses straight to global memory ran at a quarter of this kernel's rate.
__host__ __device__ constexpr int slot_bytes(int row_bytes) { return (row_bytes + 15) / 16 * 16 + 16; }

template <typename T>
__device__ __forceinline__ int row_offset(const T* p) { return (int)(reinterpret_cast<uintptr_t>(p) & 15); }

// A matrix whose rows are copied below.
template <typename T>
struct Rows {
    const T* m;
    long ld;
    uintptr_t last;  // one past its last byte
    int H;
    __device__ __forceinline__ Rows(const void* p, long ld, int n_rows, int H)
        : m(static_cast<const T*>(p)), ld(ld), last(reinterpret_cast<uintptr_t>(m + (n_rows - 1) * ld + H)), H(H) {}
    __device__ __forceinline__ const T* row(long t) const { return m + t * ld; }
};

// Copies row t into `slot` at the row's own offset. The chunks at a row's ends bring neighbouring
// bytes along, which nothing reads; chunks that would reach outside the matrix are copied element
// by element.
template <typename T>
__device__ __forceinline__ void copy_row_in(uint8_t* slot, const Rows<T>& a, long t) {
    const T* p = a.row(t);
    const RowChunks r(reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(a.m), a.last, a.H * (int)sizeof(T));
    const uint8_t* base = reinterpret_cast<const uint8_t*>(p) - r.off;
    for (int c = threadIdx.x * 16; c < r.end; c += blockDim.x * 16) {
        if (r.whole(c)) {
            cp_async16(slot + c, base + c);
        } else {
            for (int i = max(c, r.off); i < min(c + 16, r.end); i += (int)sizeof(T))
                *reinterpret_cast<T*>(slot + i) = *reinterpret_cast<const T*>(base + i);
        }
    }
}

// Writes the row that lies in `slot` at offset row_offset(p) to p.
template <typename T>
__device__ __forceinline__ void copy_row_out(T* p, const uint8_t* slot, int H) {
    const int off = row_offset(p), end = off + H * (int)sizeof(T);
    uint8_t* base = reinterpret_cast<uint8_t*>(p) - off;
    for (int c = threadIdx.x * 16; c < end; c += blockDim.x * 16) {
        if (c >= off && c + 16 <= end) {
            *reinterpret_cast<uint4*>(base + c) = *reinterpret_cast<const uint4*>(slot + c);
        } else {
            for (int i = max(c, off); i < min(c + 16, end); i += (int)sizeof(T))
                *reinterpret_cast<T*>(base + i) = *reinterpret_cast<const T*>(slot + i);
        }
    }
}

// Elements tid + i * threads (i < 2 NP) of a row, in pairs. The launch makes sure that all but
// the last of them lie inside the row for every thread, or, with one pair, checks both:
// a test per element cost more instructions than the arithmetic.
template <int NP>
struct Own {
    int c, nt;
    bool first, last;
    __device__ __forceinline__ Own(int H) : c(threadIdx.x), nt(blockDim.x) {
        first = NP > 1 || c < H;
        last = c + (2 * NP - 1) * nt < H;
    }
    __device__ __forceinline__ bool has(int i) const {
        return NP == 1 && i == 0 ? first : (i == 2 * NP - 1 ? last : true);
    }
};
template <typename T, int NP>
__device__ __forceinline__ void read_row(f32x2 (&v)[NP], const uint8_t* row, const Own<NP>& o) {
    const T* r = reinterpret_cast<const T*>(row) + o.c;
#pragma unroll
    for (int i = 0; i < NP; ++i)
        v[i] = pack2(o.has(2 * i) ? to_f32<T>(r[2 * i * o.nt]) : 0.f,
                     o.has(2 * i + 1) ? to_f32<T>(r[(2 * i + 1) * o.nt]) : 0.f);
}
template <typename T, int NP>
__device__ __forceinline__ void write_row(uint8_t* row, const f32x2 (&v)[NP], const Own<NP>& o) {
    T* r = reinterpret_cast<T*>(row) + o.c;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const float2 f = unpack2(v[i]);
        if (o.has(2 * i)) r[2 * i * o.nt] = from_f32<T>(f.x);
        if (o.has(2 * i + 1)) r[(2 * i + 1) * o.nt] = from_f32<T>(f.y);
    }
}
template <int NP>
__device__ __forceinline__ void read_param(f32x2 (&v)[NP], const float* p, const Own<NP>& o, float none) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
        v[i] = pack2(o.has(2 * i) ? (p ? p[o.c + 2 * i * o.nt] : none) : 0.f,
                     o.has(2 * i + 1) ? (p ? p[o.c + (2 * i + 1) * o.nt] : none) : 0.f);
}

// A ring of S rows; the next row's copies start once every thread is done with the slot.
template <typename T, int NP, int S, bool LAYER>
__global__ void __launch_bounds__(1024) norm_fwd_ragged_kernel(NormFwd p) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint4 ring[];
    __shared__ float buf[2][32];
    int which = 0;
    const int H = p.H, SL = slot_bytes(H * (int)sizeof(T));
    uint8_t* slots = reinterpret_cast<uint8_t*>(ring);
    f32x2 w[NP], b[NP];
    const Own<NP> own(H);
    read_param<NP>(w, p.w, own, 1.f);
    read_param<NP>(b, p.b, own, 0.f);
    const Rows<T> x(p.x, p.ldx, p.T, H);
    const long step = gridDim.x;
    long t = blockIdx.x;
#pragma unroll
    for (int j = 0; j < S - 1; ++j) {
        if (t + j * step < p.T) copy_row_in<T>(slots + j * SL, x, t + j * step);
        cp_async_commit();
    }
    int st = 0;
    for (; t < p.T; t += step) {
        cp_async_wait<S - 2>();
        __syncthreads();  // the row is in; every thread has left the slot before it
        const long ahead = t + (S - 1) * step;
        if (ahead < p.T) copy_row_in<T>(slots + (st == 0 ? S - 1 : st - 1) * SL, x, ahead);
        cp_async_commit();
        uint8_t* slot = slots + st * SL;
        f32x2 v[NP];
        read_row<T, NP>(v, slot + row_offset(x.row(t)), own);
        float mean = 0.f;
        if (LAYER) {
            f32x2 sum = v[0];
#pragma unroll
            for (int i = 1; i < NP; ++i) sum = add2(sum, v[i]);
            mean = p.over_h.of(block_sum(sum2(sum), buf, which));
        }
        f32x2 sq = pack2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if (LAYER) v[i] = add2(v[i], pack2(own.has(2 * i) ? -mean : 0.f, own.has(2 * i + 1) ? -mean : 0.f));
            sq = fma2(v[i], v[i], sq);
        }
        const float r = rsqrtf(p.over_h.of(block_sum(sum2(sq), buf, which)) + p.eps);
        if (threadIdx.x == 0) {
            if (LAYER && p.mean) p.mean[t] = mean;
            if (p.rstd) p.rstd[t] = r;
        }
        const f32x2 r2 = pack2(r, r);
#pragma unroll
        for (int i = 0; i < NP; ++i) v[i] = fma2(mul2(v[i], r2), w[i], b[i]);
        T* y = static_cast<T*>(p.y) + t * p.ldy;
        __syncthreads();  // the row has been read by all
        write_row<T, NP>(slot + row_offset(y), v, own);
        __syncthreads();
        copy_row_out<T>(y, slot, H);
        st = st + 1 == S ? 0 : st + 1;
    }
}

template <typename T, int NP, int R, int S, bool LAYER>
__global__ void __launch_bounds__(NP == 8 && S > 1 ? 512 : 1024) norm_bwd_ragged_kernel(NormBwd p) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint4 ring[];  // [S][R rows][x, dy], then [R] rows of dx
    __shared__ float buf[2][2 * R * 32];
    int which = 0;
    const int H = p.H, SL = slot_bytes(H * (int)sizeof(T));
    uint8_t* slots = reinterpret_cast<uint8_t*>(ring);
    uint8_t* outs = slots + S * R * 2 * SL;
    f32x2 w[NP], sw[NP], sb[NP];
    const Own<NP> own(H);
    read_param<NP>(w, p.w, own, 1.f);
#pragma unroll
    for (int i = 0; i < NP; ++i) sw[i] = sb[i] = pack2(0.f, 0.f);
    const Rows<T> x(p.x, p.ldx, p.T, H), dy(p.dy, p.lddy, p.T, H);
    auto copy = [&](long t, uint8_t* to) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            if (t + q < p.T) {
                copy_row_in<T>(to + 2 * q * SL, x, t + q);
                copy_row_in<T>(to + (2 * q + 1) * SL, dy, t + q);
            }
        }
        cp_async_commit();
    };
    const long step = R * (long)gridDim.x;
    long t = R * (long)blockIdx.x;
#pragma unroll
    for (int j = 0; j < S - 1; ++j) copy(t + j * step, slots + j * R * 2 * SL);
    int st = 0;
    for (; t < p.T; t += step) {
        float mean[R], r[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            mean[q] = LAYER && t + q < p.T ? p.mean[t + q] : 0.f;
            r[q] = t + q < p.T ? p.rstd[t + q] : 0.f;
        }
        if constexpr (S == 1) {
            __syncthreads();  // every thread has left the only slot
            copy(t, slots);
            cp_async_wait<0>();
            __syncthreads();
        } else {
            cp_async_wait<(S == 1 ? 0 : S - 2)>();
            __syncthreads();
            copy(t + (S - 1) * step, slots + (st == 0 ? S - 1 : st - 1) * R * 2 * SL);
        }
        const uint8_t* rows = slots + st * R * 2 * SL;
        float s[2 * R];
        // n and the weighted dy of row q; where the row ends they are zero
        auto row = [&](int q, f32x2 (&n)[NP], f32x2 (&g)[NP]) {
            read_row<T, NP>(n, rows + 2 * q * SL + row_offset(x.row(t + q)), own);
            read_row<T, NP>(g, rows + (2 * q + 1) * SL + row_offset(dy.row(t + q)), own);
            const f32x2 minus = pack2(-mean[q], -mean[q]), r2 = pack2(r[q], r[q]);
#pragma unroll
            for (int i = 0; i < NP; ++i) n[i] = mul2(LAYER ? add2(n[i], minus) : n[i], r2);
        };
#pragma unroll
        for (int q = 0; q < R; ++q) {
            s[2 * q] = s[2 * q + 1] = 0.f;
            if (t + q >= p.T) continue;
            f32x2 n[NP], g[NP], a1 = pack2(0.f, 0.f), a2 = pack2(0.f, 0.f);
            row(q, n, g);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                sw[i] = fma2(g[i], n[i], sw[i]);
                if (LAYER) sb[i] = add2(sb[i], g[i]);
                g[i] = mul2(g[i], w[i]);
                if (LAYER) a1 = add2(a1, g[i]);
                a2 = fma2(g[i], n[i], a2);
            }
            s[2 * q] = sum2(a1);
            s[2 * q + 1] = sum2(a2);
        }
        if (p.dx) {
            T* dx = static_cast<T*>(p.dx);
            block_sums<2 * R>(s, buf, which);
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (t + q >= p.T) continue;
                const float c1 = -p.over_h.of(s[2 * q]), c2 = -p.over_h.of(s[2 * q + 1]);
                const f32x2 m1 = pack2(c1, c1), m2 = pack2(c2, c2), r2 = pack2(r[q], r[q]);
                f32x2 n[NP], g[NP];
                row(q, n, g);
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    g[i] = LAYER ? fma2(g[i], w[i], m1) : mul2(g[i], w[i]);
                    g[i] = mul2(r2, fma2(n[i], m2, g[i]));
                }
                write_row<T, NP>(outs + q * SL + row_offset(dx + (t + q) * p.lddx), g, own);
            }
            __syncthreads();
#pragma unroll
            for (int q = 0; q < R; ++q)
                if (t + q < p.T) copy_row_out<T>(dx + (t + q) * p.lddx, outs + q * SL, H);
        }
        st = st + 1 == S ? 0 : st + 1;
    }
    if (!p.part) return;
    float* part = p.part + (size_t)blockIdx.x * 2 * H;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const float2 a = unpack2(sw[i]), b = unpack2(sb[i]);
        float* q = part + own.c + 2 * i * own.nt;
        if (own.has(2 * i)) q[0] = a.x;
        if (own.has(2 * i + 1)) q[own.nt] = a.y;
        if (LAYER) {
            if (own.has(2 * i)) q[H] = b.x;
            if (own.has(2 * i + 1)) q[H + own.nt] = b.y;
        }
    }
}

// dw and db from the CTAs' column sums, added in a fixed order: 32 lanes of VEC columns per
// CTA, 32 slices of the partial rows (16 of a slice's rows loaded at once), then the slices.
template <int VEC>
__global__ void __launch_bounds__(1024) norm_param_kernel(const float* __restrict__ part, int n_part,
                                                          int H, float* dw, float* db) {
    pdl_wait();
    pdl_trigger();
    __shared__ float acc[32][32 * VEC + 1];
    const int which = blockIdx.y;  // 0: dw, 1: db
    float* out = which ? db : dw;
    if (!out) return;
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + lane) * VEC;
    float s[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[j] = 0.f;
    if (c < H) {
        const float* src = part + (size_t)which * H + c;
        constexpr int U = 16 / VEC;
        for (int i0 = slice; i0 < n_part; i0 += 32 * U) {
            Pack<float, VEC> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + 32 * u < n_part)
                    v[u] = *reinterpret_cast<const Pack<float, VEC>*>(src + (size_t)(i0 + 32 * u) * 2 * H);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i0 + 32 * u >= n_part) continue;
#pragma unroll
                for (int j = 0; j < VEC; ++j) s[j] += v[u].v[j];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[slice][lane * VEC + j] = s[j];
    __syncthreads();
    // warp `slice` sums VEC columns of the tile over the slices
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        float v = acc[lane][slice * VEC + j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int col = (blockIdx.x * 32 + slice) * VEC + j;
        if (lane == 0 && col < H) out[col] = v;
    }
}

void launch_param(const float* part, int n_part, int H, float* dw, float* db, cudaStream_t st) {
    if (!dw && !db) return;
    // wide loads for few partial rows; many are spread over four times the CTAs
    if (H % 4 == 0 && n_part <= 256)
        launch_pdl(norm_param_kernel<4>, dim3((H + 127) / 128, db ? 2 : 1), 1024, 0, st, part, n_part, H, dw, db);
    else
        launch_pdl(norm_param_kernel<1>, dim3((H + 31) / 32, db ? 2 : 1), 1024, 0, st, part, n_part, H, dw, db);
}

inline int round32(int v) { return (v + 31) / 32 * 32; }

template <typename T, int VEC, int NV, int MAXT>
void fwd(int layer, const NormFwd& p, cudaStream_t st) {
    const int threads = std::max(32, round32((p.H / VEC + NV - 1) / NV));
    if (layer) launch_pdl(norm_fwd_kernel<T, VEC, NV, MAXT, true>, p.T, threads, 0, st, p);
    else launch_pdl(norm_fwd_kernel<T, VEC, NV, MAXT, false>, p.T, threads, 0, st, p);
}

// CTAs that share an SM, for a persistent grid: what threads and shared memory leave room for.
int ctas_per_sm(int threads, int smem, int most_threads) {
    return std::max(1, std::min({16, most_threads / threads, 227 * 1024 / (smem + 1024)}));
}

template <typename T, int NV, int S, int MAXT, int MINB>
cudaError_t fwd_ring(int layer, const NormFwd& p, cudaStream_t st) {
    const int threads = std::max(32, round32((p.H / kFullVec<T> + NV - 1) / NV));
    const int smem = S * p.H * (int)sizeof(T);
    const bool full = p.H == threads * NV * kFullVec<T>;
    auto kernel = layer ? (full ? norm_fwd_ring_kernel<T, NV, S, MAXT, MINB, true, true>
                                : norm_fwd_ring_kernel<T, NV, S, MAXT, MINB, true, false>)
                        : (full ? norm_fwd_ring_kernel<T, NV, S, MAXT, MINB, false, true>
                                : norm_fwd_ring_kernel<T, NV, S, MAXT, MINB, false, false>);
    if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem)) return e;
    const long grid = std::min<long>(p.T, (long)ctas_per_sm(threads, smem, MAXT * MINB) * num_sms());
    return launch_pdl(kernel, (unsigned)grid, threads, smem, st, p);
}

template <int NP>
int ragged_threads(int H) { return std::max(32, round32((H + 2 * NP - 1) / (2 * NP))); }
// Every thread has all but its last element (at one pair the kernels check both).
template <int NP>
bool ragged_fits(int H) { return NP == 1 || H >= (2 * NP - 1) * ragged_threads<NP>(H); }

template <typename T, int NP, int S>
cudaError_t fwd_ragged(int layer, const NormFwd& p, cudaStream_t st) {
    const int threads = ragged_threads<NP>(p.H);
    const int smem = S * slot_bytes(p.H * (int)sizeof(T));
    auto kernel = layer ? norm_fwd_ragged_kernel<T, NP, S, true> : norm_fwd_ragged_kernel<T, NP, S, false>;
    if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem)) return e;
    const long grid = std::min<long>(p.T, (long)ctas_per_sm(threads, smem, 1024) * num_sms());
    return launch_pdl(kernel, (unsigned)grid, threads, smem, st, p);
}

template <typename T>
cudaError_t fwd_type(int layer, const NormFwd& p, bool vec, cudaStream_t st) {
    constexpr int V = kFullVec<T>;
    if (!vec) {
        // as many elements per thread as divide the row evenly enough (16 above 7680 always)
        if (ragged_fits<8>(p.H))
            return p.H * (int)sizeof(T) <= 32768 ? fwd_ragged<T, 8, 4>(layer, p, st) : fwd_ragged<T, 8, 2>(layer, p, st);
        if (ragged_fits<4>(p.H)) return fwd_ragged<T, 4, 4>(layer, p, st);
        if (ragged_fits<2>(p.H)) return fwd_ragged<T, 2, 4>(layer, p, st);
        return fwd_ragged<T, 1, 4>(layer, p, st);
    }
    const int nvec = p.H / V;
    // few rows: a row per CTA on as many threads as it takes, for the shortest time of a row
    if (p.T < 2 * num_sms()) {
        if (nvec <= 1024) fwd<T, V, 1, 1024>(layer, p, st);
        else fwd<T, V, 4, 1024>(layer, p, st);
        return cudaGetLastError();
    }
    if (nvec <= 1024) return fwd_ring<T, 2, 4, 512, 2>(layer, p, st);
    if constexpr (sizeof(T) == 4)
        if (nvec > 2048) return fwd_ring<T, 4, 3, 1024, 1>(layer, p, st);
    return fwd_ring<T, 2, 4, 1024, 1>(layer, p, st);
}

// CTAs that share an SM: about 1024 threads' worth of rows in flight.
int bwd_grid(int T, int threads) {
    const long per_sm = std::min(16, std::max(1, 1024 / threads));
    return (int)std::min<long>(T, per_sm * num_sms());
}
// no variant puts more than 16 elements of a row on a thread
constexpr int kMaxPerThread = 16;

template <typename T, int NP, int R, int S>
cudaError_t bwd_ragged(int layer, const NormBwd& p, float* dw, float* db, cudaStream_t st) {
    static_assert(2 * NP <= kMaxPerThread, "the workspace's grid bound");
    const int threads = ragged_threads<NP>(p.H);
    const int smem = (S * 2 + 1) * R * slot_bytes(p.H * (int)sizeof(T));
    auto kernel = layer ? norm_bwd_ragged_kernel<T, NP, R, S, true> : norm_bwd_ragged_kernel<T, NP, R, S, false>;
    if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem)) return e;
    const int grid = (int)std::min<long>(bwd_grid((p.T - 1) / R + 1, threads),
                                         (long)ctas_per_sm(threads, smem, NP == 8 ? 512 : 1024) * num_sms());
    if (cudaError_t e = launch_pdl(kernel, grid, threads, smem, st, p)) return e;
    launch_param(p.part, grid, p.H, dw, db, st);
    return cudaGetLastError();
}

template <typename T, int NV, int R, int S, int MAXT, bool LAYER>
void (*pick_bwd_kind(bool full, bool grouped))(NormBwd) {
    if constexpr (MAXT <= 512) {  // wider rows are never one warp's
        if (grouped)
            return full ? norm_bwd_ring_kernel<T, NV, R, S, 256, LAYER, true, true>
                        : norm_bwd_ring_kernel<T, NV, R, S, 256, LAYER, false, true>;
    }
    return full ? norm_bwd_ring_kernel<T, NV, R, S, MAXT, LAYER, true, false>
                : norm_bwd_ring_kernel<T, NV, R, S, MAXT, LAYER, false, false>;
}
template <typename T, int NV, int R, int S, int MAXT>
void (*pick_bwd(bool layer, bool full, bool grouped))(NormBwd) {
    return layer ? pick_bwd_kind<T, NV, R, S, MAXT, true>(full, grouped)
                 : pick_bwd_kind<T, NV, R, S, MAXT, false>(full, grouped);
}

template <typename T, int NV, int R, int S, int MAXT>
cudaError_t bwd_ring(int layer, const NormBwd& p, float* dw, float* db, cudaStream_t st) {
    static_assert(kFullVec<T> * NV <= kMaxPerThread, "the workspace's grid bound");
    const int threads = std::max(32, round32((p.H / kFullVec<T> + NV - 1) / NV));
    const int groups = threads == 32 ? 8 : 1;
    const int smem = groups * S * R * 2 * p.H * (int)sizeof(T);
    const bool full = p.H == threads * NV * kFullVec<T>;
    auto kernel = pick_bwd<T, NV, R, S, MAXT>(layer, full, groups > 1);
    if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem)) return e;
    const int grid = (int)std::min<long>(bwd_grid((p.T - 1) / (R * groups) + 1, threads),
                                         (long)ctas_per_sm(threads * groups, smem, 512) * num_sms());
    if (cudaError_t e = launch_pdl(kernel, grid, dim3(threads, groups), smem, st, p)) return e;
    launch_param(p.part, grid, p.H, dw, db, st);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_type(int layer, const NormBwd& p, bool vec, float* dw, float* db, cudaStream_t st) {
    if (!vec) {
        if (p.H > 8192) return bwd_ragged<T, 8, 1, 1>(layer, p, dw, db, st);
        if (ragged_fits<8>(p.H))
            return sizeof(T) == 4 ? bwd_ragged<T, 8, 1, 2>(layer, p, dw, db, st) : bwd_ragged<T, 8, 2, 2>(layer, p, dw, db, st);
        if (ragged_fits<4>(p.H)) return bwd_ragged<T, 4, 1, 2>(layer, p, dw, db, st);
        if (ragged_fits<2>(p.H)) return bwd_ragged<T, 2, 2, 3>(layer, p, dw, db, st);
        return bwd_ragged<T, 1, 2, 3>(layer, p, dw, db, st);
    }
    // 16 elements of a row on a thread, 512 threads an SM (~100 registers each) and as deep a
    // ring as fits; with less than two pairs of rows per SM the rows go one by one, to more CTAs
    constexpr int NV = kMaxPerThread / kFullVec<T>;
    if (p.H > 8192) return bwd_ring<T, NV, 1, sizeof(T) == 2 ? 3 : 1, 1024>(layer, p, dw, db, st);
    constexpr int S = sizeof(T) == 2 ? 3 : 1;
    if (p.T < 4 * num_sms()) return bwd_ring<T, NV, 1, 2 * S, 512>(layer, p, dw, db, st);
    return bwd_ring<T, NV, 2, S, 512>(layer, p, dw, db, st);
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
    const NormFwd p{x, y, w, b, mean, rstd, ldx, ldy, T, H, eps, InvH(H)};
    const int es = esize(dtype), layer = kind == MOE_NORM_LAYER;
    const bool vec = H % (16 / es) == 0 && rows16(x, ldx, es) && rows16(y, ldy, es) &&
                     rows16(w, 4, 4) && rows16(b, 4, 4);
    if (dtype == MOE_T_BF16) return fwd_type<__nv_bfloat16>(layer, p, vec, st);
    if (dtype == MOE_T_F16) return fwd_type<__half>(layer, p, vec, st);
    return fwd_type<float>(layer, p, vec, st);
}

cudaError_t launch_norm_bwd(int kind, int dtype, const void* dy, long lddy, const void* x, long ldx,
                            int T, int H, const float* w, const float* mean, const float* rstd,
                            void* dx, long lddx, float* dw, float* db, float* part, cudaStream_t st) {
    if (T == 0) {  // no rows: the sums are zero
        launch_param(nullptr, 0, H, dw, db, st);
        return cudaGetLastError();
    }
    const NormBwd p{dy, x, dx, w, mean, rstd, (dw || db) ? part : nullptr, lddy, ldx, lddx, T, H, InvH(H)};
    const int es = esize(dtype), layer = kind == MOE_NORM_LAYER;
    const bool vec = H % (16 / es) == 0 && rows16(x, ldx, es) && rows16(dy, lddy, es) && rows16(dx, lddx, es) &&
                     rows16(w, 4, 4);
    if (dtype == MOE_T_BF16) return bwd_type<__nv_bfloat16>(layer, p, vec, dw, db, st);
    if (dtype == MOE_T_F16) return bwd_type<__half>(layer, p, vec, dw, db, st);
    return bwd_type<float>(layer, p, vec, dw, db, st);
}

}  // namespace moe
