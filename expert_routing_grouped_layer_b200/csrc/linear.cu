// linear.cu -- dense matrix products on the tcgen05 tensor cores with the linear layer's
// epilogue, and the elementwise step of its backward pass.
//
//   forward   z = x W^T + bias,  y = act(z) + residual  (z kept as `pre` where wanted)
//   backward  g = dy act'(z);  dx = g W,  dW = g^T x,  db = sum_m g
//
// All three products are one form: out[r][c] = sum_k R(r, k) C(c, k), where each operand
// lies in memory either with k contiguous (K-major) or with its row index contiguous
// (MN-major: W in dx, and both in dW). Both layouts feed the tensor cores directly: TMA
// writes 128-byte swizzled tiles of 64 k x rows or 64 rows x 64 k, and the shared-memory
// descriptors name the layout, so nothing is transposed in memory. Ragged sizes cost
// nothing extra: TMA fills what lies outside a matrix with zeros and the epilogue
// writes what lies inside.
//
// Two kernels:
//   linear_pair_kernel   many rows: persistent CTA pairs (cta_group::2), a 256 x BN tile
//                        per pair, accumulators double-buffered in tensor memory. Bound by
//                        the tensor cores and the power cap: 8192 x 7168 x 2048 with bias
//                        and residual in 166-180 us (1.34-1.45 PFLOP/s, tensor pipe 91% active at
//                        1.5 GHz; 193-211 us in a long run); a library product of that size
//                        alone took 168-172;
//   linear_split_kernel  few tiles (serving, small gradients): 128 columns x BT rows per
//                        cluster of up to 8 CTAs that share the k range and add their
//                        partial tiles through distributed shared memory in rank order,
//                        so the weights stream through all SMs and equal calls give
//                        equal bits. Bound by the weights' bytes and ~4 us of launch, set-up
//                        and exchange: one token, 2048 x 7168, 8.5-8.7 us.
// Sums are fp32 in tensor memory; y, pre, dx and dW are rounded once to the tensors'
// type, and g once between dy and the products (the tensor cores take 16-bit operands).
#include <type_traits>

#include "gemm_common.cuh"
#include "types.cuh"

namespace moe {

namespace {

using gemm::BK;
using gemm::make_tmap_2d;

constexpr int kSmemMax = 232448;

// ------------------------------------------------------------------ operands
// MN-major tile written by TMA as boxes of 64 elements (128 swizzled bytes) x 64 k:
// 8-k groups are 1024 bytes apart (stride byte offset), 64-element boxes 8192 bytes
// apart (leading byte offset); one MMA's 16 k are 2048 bytes.
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(8192 >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

template <bool MN>
__device__ __forceinline__ uint64_t sdesc(uint32_t base) {
    return MN ? sdesc_mnmajor_sw128(base) : sdesc_kmajor_sw128(base);
}
// Descriptor step (16-byte units, the descriptor's low field) of one MMA's 16 k.
template <bool MN>
constexpr uint64_t kStep = MN ? 2048 / 16 : 32 / 16;

// The MMA loops run on whole warps, and one lane issues: with the loop's state uniform over
// the warp the descriptors stay in uniform registers and advance by additions. (Issued
// from one lane's own loop, which rebuilt them, four MMAs took 540 cycles however narrow
// the tile.)
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}
// mbar_wait by a converged warp, the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// Instruction descriptor, kind::f16: fp32 accumulator, A and B both bf16 or both f16,
// MN-major bits 15 (A) and 16 (B).
template <typename T, bool A_MN, bool B_MN>
__device__ __forceinline__ uint32_t idesc_16(uint32_t M, uint32_t N) {
    const uint32_t fmt = sizeof(T) == 2 && !is_half<T>() ? 1u : 0u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) |
           ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ void mma_pair_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// ------------------------------------------------------------------ epilogue
struct Epilogue {
    const float* bias;  // [cols] or null
    const void* res;    // rows like out, or null
    void* out;
    void* pre;  // or null
    long ld_res, ld_out, ld_pre;
    int cols, act;
    int vec;  // out, res, pre and bias allow 4-element accesses
};

constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kGeluCubic = 0.044715f;

// sigmoid(z) = f^2 r with r = 1 / (1 + e^2), e = exp(-|z| / 2), f = e below zero and 1 above. In two
// factors it keeps its digits down to e^-174, so that z sigmoid(z) is right to where it leaves the
// fp32 range itself (z = -92; 1 / (1 + exp(-z)) is zero from z = -87 on).
__device__ __forceinline__ float times_sigmoid(float a, float z) {
    const float e = exp_approx(-0.5f * fabsf(z)), r = rcp_approx(fmaf(e, e, 1.0f)), f = z < 0.0f ? e : 1.0f;
    return (a * f) * (f * r);
}

// (1 + tanh u) / 2 = sigmoid(2 u) with u = sqrt(2/pi) (z + 0.044715 z^3): no difference of close
// numbers on either side, where 1 + tanh u loses every digit below z = -4.
__device__ __forceinline__ float gelu_tanh_arg(float z) {
    return 2.0f * kSqrt2OverPi * fmaf(kGeluCubic * z * z, z, z);
}

// The normal distribution's Phi(-x) = exp(-x^2 / 2) R(x) for x >= 0, where R goes from 1/2 to
// 1 / (x sqrt(2 pi)) and is fitted as a polynomial in t = 1 / (1 + 0.3 x) that keeps the largest
// relative error over 0 <= x <= 14.5 least (1.7e-7; a linear program over R = erfcx(x / sqrt 2) / 2):
// the tail is right relative to itself, and there is no branch and no more than two
// special-function operations. erff's two ranges diverge within a warp; with it the GELU epilogue
// took 11.6 us a tile.
__device__ __forceinline__ float normal_gauss(float x) { return exp_approx(-0.5f * x * x); }
__device__ __forceinline__ float normal_ratio(float x) {
    const float t = rcp_approx(fmaf(0.3f, x, 1.0f));
    float p = fmaf(t, 0.035431112f, -0.156189101f);
    p = fmaf(t, p, 0.204609411f);
    p = fmaf(t, p, -0.0520822260f);
    p = fmaf(t, p, 0.127717121f);
    p = fmaf(t, p, 0.100168327f);
    p = fmaf(t, p, 0.120713345f);
    p = fmaf(t, p, 0.119631929f);
    return p * t;
}

template <int ACT>
__device__ __forceinline__ float act_f(float z) {
    switch (ACT) {
    case MOE_ACT_RELU: return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    case MOE_ACT_SILU: return times_sigmoid(z, z);
    case MOE_ACT_GELU: {
        const float x = fabsf(z), tail = normal_ratio(x) * normal_gauss(x);
        return z * (z < 0.0f ? tail : 1.0f - tail);
    }
    case MOE_ACT_GELU_TANH: return times_sigmoid(z, gelu_tanh_arg(z));
    }
    return z;
}

// The smaller number, NaN if one is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Each smooth activation is a(z) = z S(z) with S(z) + S(-z) = 1, so a'(z) = 1 - a'(-z): the slope is
// worked out below zero, where it is right relative to itself. Long before |z| = 200 it is 0 and 1 in
// fp32; held there, an infinite z (an f16 `pre` beyond 65504) or a huge one gives that instead of 0
// times infinity.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if (ACT == MOE_ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    if (ACT == MOE_ACT_NONE) return 1.0f;
    const float x = min_nan(fabsf(z), 200.0f);
    float below;  // a'(-x)
    if (ACT == MOE_ACT_GELU) {
        below = normal_gauss(x) * fmaf(x, -kInvSqrt2Pi, normal_ratio(x));
    } else {  // a'(-x) = sigmoid(-v) (1 - x sigmoid(v) v'(x)), the exponential in two factors as above
        const float v = ACT == MOE_ACT_SILU ? x : gelu_tanh_arg(x);
        const float e = exp_approx(-0.5f * v), r = rcp_approx(fmaf(e, e, 1.0f));
        const float xv = ACT == MOE_ACT_SILU ? x : x * fmaf(6.0f * kSqrt2OverPi * kGeluCubic * x, x, 2.0f * kSqrt2OverPi);
        below = (e * fmaf(-xv, r, 1.0f)) * (e * r);
    }
    return z < 0.0f ? below : 1.0f - below;
}

// Calls f with the activation as a compile-time constant: one branch for a group of values.
template <typename F>
__host__ __device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
    case MOE_ACT_RELU: f(std::integral_constant<int, MOE_ACT_RELU>()); break;
    case MOE_ACT_SILU: f(std::integral_constant<int, MOE_ACT_SILU>()); break;
    case MOE_ACT_GELU: f(std::integral_constant<int, MOE_ACT_GELU>()); break;
    case MOE_ACT_GELU_TANH: f(std::integral_constant<int, MOE_ACT_GELU_TANH>()); break;
    default: f(std::integral_constant<int, MOE_ACT_NONE>());
    }
}

// Bias of columns col..col+3 (zero outside).
__device__ __forceinline__ float4 bias4(const Epilogue& e, int col) {
    float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!e.bias) return b;
    if (e.vec && col + 4 <= e.cols) return *reinterpret_cast<const float4*>(e.bias + col);
    if (col < e.cols) b.x = e.bias[col];
    if (col + 1 < e.cols) b.y = e.bias[col + 1];
    if (col + 2 < e.cols) b.z = e.bias[col + 2];
    if (col + 3 < e.cols) b.w = e.bias[col + 3];
    return b;
}

// Whether columns col..col+3 move by one access.
__device__ __forceinline__ bool quad_at(const Epilogue& e, int col) { return e.vec && col + 4 <= e.cols; }

// Residual of four neighbouring elements, raw, loaded ahead of its use where quad_at. (As
// separate 16-bit values the load would be unpacked, and so waited for, on the spot.)
template <typename T>
__device__ __forceinline__ uint2 res4(const Epilogue& e, long row, int col) {
    return *reinterpret_cast<const uint2*>(static_cast<const T*>(e.res) + row * e.ld_res + col);
}

// Four neighbouring results of one row: bias, pre, activation, residual, store. r: the
// residual where quad_at, else it is read here.
template <typename T, int ACT>
__device__ __forceinline__ void store4(const Epilogue& e, float4 acc, float4 b, uint2 r, long row, int col) {
    const float z[4] = {acc.x + b.x, acc.y + b.y, acc.z + b.z, acc.w + b.w};
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = act_f<ACT>(z[j]);
    T* out = static_cast<T*>(e.out) + row * e.ld_out + col;
    T* pre = static_cast<T*>(e.pre) + row * e.ld_pre + col;
    if (quad_at(e, col)) {
        if (e.pre) *reinterpret_cast<uint2*>(pre) = narrow4<T>(z);
        if (e.res) {
            const Pack<T, 4> p = *reinterpret_cast<const Pack<T, 4>*>(&r);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] += to_f32<T>(p.v[j]);
        }
        *reinterpret_cast<uint2*>(out) = narrow4<T>(y);
    } else {
        const T* res = static_cast<const T*>(e.res) + row * e.ld_res + col;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (col + j >= e.cols) break;
            if (e.pre) pre[j] = from_f32<T>(z[j]);
            if (e.res) y[j] += to_f32<T>(res[j]);
            out[j] = from_f32<T>(y[j]);
        }
    }
}

// The first n (1 to 7) of eight 16-bit elements to a 16-byte aligned place.
__device__ __forceinline__ void store_rest(void* out, const void* piece, int n) {
    const uint4 v = *static_cast<const uint4*>(piece);
    char* o = static_cast<char*>(out);
    if (n & 4) *reinterpret_cast<uint2*>(o) = make_uint2(v.x, v.y);
    const uint32_t a = n & 4 ? v.z : v.x, b = n & 4 ? v.w : v.y;
    if (n & 2) *reinterpret_cast<uint32_t*>(o + 2 * (n & 4)) = a;
    if (n & 1) *reinterpret_cast<uint16_t*>(o + 2 * (n & 6)) = (uint16_t)(n & 2 ? b : a);
}

struct GemmDims {
    int R, C, K;  // out rows, out columns, reduction length
    int32_t* status;
};

// ------------------------------------------------------------------ CTA pairs
// 256 rows x BN columns per pair: each SM loads its 128 rows and half of the columns'
// operand, and drains its own 128 accumulator rows.
//   warp 0  TMA, warp 1 MMA (leader), warps 2-9 epilogue: four lane quadrants x two
//   groups that take alternate 32-column chunks.
// Epilogue with outputs on the 16-byte grid (TMA_OUT): a lane finishes one row's 32 columns
// in registers, the warp's 32 x 32 block goes through 2 KB of swizzled shared memory and
// leaves (and the residual comes) by TMA, which also clips it to the matrix. A store clips in
// steps of 16 bytes and would write up to 7 elements behind rows of other widths: the tensor
// maps of out and pre end at the last multiple of 8 columns, and the lanes store the rest. Otherwise a
// chunk goes through shared memory as fp32 and lanes store along rows, element by element
// where need be; with the residual that took 13.8 us a tile against the main loop's 14.5 us
// at K = 2048 and held the tensor cores up.
struct PairCfg {
    static constexpr int A_BYTES = 128 * BK * 2;
    // the ring of stages (six of a 256-column tile, more of a narrower one) and the epilogue's
    // blocks, three a warp with `pre` and two without
    static constexpr int DATA_BYTES = 224 * 1024;
    static constexpr int MAX_STAGES = 9;
    static constexpr int EPI_WARPS = 8;
    static constexpr int epi_warp_bytes(bool pre) { return pre ? 3 * 2048 : 2 * 2048; }
    static constexpr int THREADS = 32 * (2 + EPI_WARPS);
    static constexpr int SMEM_BYTES = 1024 + DATA_BYTES + 8 * (2 * MAX_STAGES + 5 + 2 * EPI_WARPS) + 16;
    static_assert(SMEM_BYTES <= kSmemMax, "shared memory budget");
};

// Tile u of the grid: bands of 8 tile rows, columns inside a band, so that the tiles in
// flight share operands in L2.
__device__ __forceinline__ void tile_of(int u, int mt, int nt, int& tm, int& tn) {
    const int band = 8 * nt;
    const int b = u / band, r = u - b * band;
    const int h = min(8, mt - b * 8);
    tn = r / h;
    tm = b * 8 + (r - tn * h);
}

__device__ __forceinline__ void tma_store_2d(const void* tmap, const void* smem_src, int32_t x, int32_t y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(smem_u32(smem_src)), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Tensor maps of the epilogue's matrices, boxes of 32 x 32 elements, 64-byte swizzle.
struct OutMaps {
    CUtensorMap out, pre, res;
};

template <typename T, bool A_MN, bool B_MN, bool TMA_OUT>
__global__ void __launch_bounds__(PairCfg::THREADS, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ OutMaps tmO, const GemmDims d, const Epilogue epi, const int BN) {
    pdl_wait();
    pdl_trigger();
    using C = PairCfg;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int epi_warp = C::epi_warp_bytes(epi.pre != nullptr);
    const int ring_bytes = C::DATA_BYTES - C::EPI_WARPS * epi_warp;
    uint8_t* stage_out = smem + ring_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::DATA_BYTES);
    uint64_t* empty = full + C::MAX_STAGES;
    uint64_t* tfull = empty + C::MAX_STAGES;
    const int half = BN / 2;
    const int b_boxes = B_MN ? (half + 63) / 64 : 1;
    const int stage_bytes = C::A_BYTES + (B_MN ? b_boxes * 8192 : half * BK * 2);
    const int stages = min(C::MAX_STAGES, ring_bytes / stage_bytes);
    uint64_t* tempty = tfull + 2;
    uint64_t* mma_done = tempty + 2;
    uint64_t* res_full = mma_done + 1;  // two per epilogue warp: a residual block is in
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_full + 2 * C::EPI_WARPS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);   // the leader's expect-tx arrival covers both SMs' copies
            mbar_init(&empty[s], 1);  // the leader's multicast commit
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 2 * C::EPI_WARPS);  // both SMs' epilogue warps (leader's copy used)
        }
        mbar_init(mma_done, 1);
        for (int w = 0; w < 2 * C::EPI_WARPS; ++w) mbar_init(&res_full[w], 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 0) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_barrier();  // both SMs' barriers are initialised before any remote arrival
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int mt = (d.R + 255) / 256, nt = (d.C + BN - 1) / BN, total = mt * nt;
    const int KB = (d.K + BK - 1) / BK;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int issued = 0;
            const uint32_t tx = 2u * (uint32_t)stage_bytes;
            for (int u = pair; u < total && !*abort_flag; u += npairs) {
                int tm, tn;
                tile_of(u, mt, nt, tm, tn);
                const int ra = tm * 256 + (int)rank * 128, rb = tn * BN + (int)rank * half;
                bool ok = true;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
                    uint8_t* st = smem + stage * stage_bytes;
                    const uint32_t lfull = peer_addr(&full[stage], 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], tx);
                    if (A_MN) {
                        tma_load_2d_pair(st, &tmA, ra, kb * BK, lfull);
                        tma_load_2d_pair(st + 8192, &tmA, ra + 64, kb * BK, lfull);
                    } else {
                        tma_load_2d_pair(st, &tmA, kb * BK, ra, lfull);
                    }
                    uint8_t* sb = st + C::A_BYTES;
                    if (B_MN) {
                        for (int i = 0; i < b_boxes; ++i)
                            tma_load_2d_pair(sb + i * 8192, &tmB, rb + 64 * i, kb * BK, lfull);
                    } else {
                        tma_load_2d_pair(sb, &tmB, kb * BK, rb, lfull);
                    }
                    ++issued;
                    if (++stage == stages) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
            }
            if (*abort_flag) {
                // the copies of both SMs complete on the leader's barriers
                if (rank == 0) {
                    volatile int no_abort = 0;
                    int s = stage;
                    uint32_t ph = phase;
                    for (int i = 0; i < min(issued, stages); ++i) {
                        if (--s < 0) { s = stages - 1; ph ^= 1; }
                        mbar_wait(&full[s], ph, &no_abort);
                    }
                }
                status_or(d.status, MOE_DEV_TIMEOUT);
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            const uint32_t idesc = idesc_16<T, A_MN, B_MN>(256, BN);
            const uint64_t da = sdesc<A_MN>(smem_u32(smem)), db = sdesc<B_MN>(smem_u32(smem) + C::A_BYTES);
            for (int u = pair; u < total; u += npairs) {
                if (!warp_wait(&tempty[acc], acc_phase ^ 1, abort_flag)) break;
                tc_fence_after();
                const uint32_t d0 = tmem_base + acc * 256;
                bool ok = true;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!warp_wait(&full[stage], phase, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t off = (uint64_t)((uint32_t)(stage * stage_bytes) >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            mma_pair_f16(d0, da + off + kk * kStep<A_MN>, db + off + kk * kStep<B_MN>, idesc,
                                         (kb | kk) != 0);
                        mma_commit_pair(&empty[stage]);
                    }
                    __syncwarp();
                    if (++stage == stages) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                if (elect_one()) mma_commit_pair(&tfull[acc]);
                __syncwarp();
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1;
            }
            if (elect_one()) {
                mma_commit(mma_done);
                volatile int no_abort = 0;
                mbar_wait(mma_done, 0, &no_abort);
                if (*abort_flag) status_or(d.status, MOE_DEV_TIMEOUT);
            }
            __syncwarp();
        }
    } else {
        const int q = warp & 3, grp = (warp - 2) >> 2;
        if constexpr (TMA_OUT) {
            // Blocks of 2 KB: 0 and 1 alternate for the result, and the next chunk's residual is
            // fetched into the other one while a chunk is worked on; 2 holds pre.
            uint8_t* bufs = stage_out + (warp - 2) * epi_warp;
            uint64_t* res_bar = &res_full[2 * (warp - 2)];  // of buffer 0 and 1
            const bool has_pre = epi.pre != nullptr, has_res = epi.res != nullptr;
            const int y0 = (int)rank * 128 + q * 32;
            int acc = 0, n = 0;  // n: chunks this warp has worked on
            uint32_t acc_phase = 0;
            auto fetch = [&](int u, int c, int to) {  // lane 0: residual of chunk c of tile u
                int tm, tn;
                tile_of(u, mt, nt, tm, tn);
                mbar_arrive_expect_tx(&res_bar[to], 2048);
                tma_load_2d(bufs + to * 2048, &tmO.res, tn * BN + c * 32, tm * 256 + y0, &res_bar[to]);
            };
            auto chunks_of = [&](int u) {
                int tm, tn;
                tile_of(u, mt, nt, tm, tn);
                return (min(BN, d.C - tn * BN) + 31) / 32;
            };
            // the chunk of this warp after chunk c of tile u (u >= total: none)
            auto advance = [&](int& u, int& c) {
                c += 2;
                while (u < total && c >= chunks_of(u)) {
                    u += npairs;
                    c = grp;
                }
            };
            int nu = pair, nc = grp - 2;
            advance(nu, nc);  // the first chunk
            int fetched = 0;
            if (has_res && lane == 0 && nu < total) {
                fetch(nu, nc, 0);
                ++fetched;
            }
            bool ok = true;
            for (int u = pair; u < total && ok; u += npairs) {
                int tm, tn;
                tile_of(u, mt, nt, tm, tn);
                if (!mbar_wait(&tfull[acc], acc_phase, abort_flag)) break;
                tc_fence_after();
                const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * 256;
                const int chunks = chunks_of(u);
                const int row = tm * 256 + y0;
                for (int c = grp; c < chunks; c += 2, ++n) {
                    const int col = tn * BN + c * 32;
                    const int bi = n & 1;
                    uint8_t* buf = bufs + bi * 2048;
                    uint32_t r0[16], r1[16];
                    tmem_ld16(taddr + c * 32, r0);
                    tmem_ld16(taddr + c * 32 + 16, r1);
                    float z[32];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 b = bias4(epi, col + 4 * j);
                        z[4 * j] = b.x; z[4 * j + 1] = b.y; z[4 * j + 2] = b.z; z[4 * j + 3] = b.w;
                    }
                    tmem_ld_wait(r0, r1);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        z[j] += __uint_as_float(r0[j]);
                        z[j + 16] += __uint_as_float(r1[j]);
                    }
                    if (lane == 0) {
                        if (has_res || has_pre) bulk_wait_read<0>();  // the last chunk's blocks have left
                        else bulk_wait_read<1>();                     // this block has
                        if (has_res) {
                            advance(nu, nc);
                            if (nu < total) {
                                fetch(nu, nc, bi ^ 1);
                                ++fetched;
                            }
                        }
                    }
                    __syncwarp();
                    uint8_t* mine = buf + lane * 64;
                    const int swz = (lane >> 1) & 3;
                    const int rest = d.C & 7, edge = d.C - rest;  // columns that the lanes store, from edge on
                    const bool tail = rest != 0 && edge >= col && edge < col + 32 && row + lane < d.R;
                    const int tail_at = (((edge - col) >> 3) ^ swz) << 4;
                    const bool tma = lane == 0 && row < d.R && col < edge;
                    if (has_pre) {
                        uint8_t* mine_pre = bufs + 4096 + lane * 64;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint4*>(mine_pre + ((j ^ swz) << 4)) = narrow8<T>(&z[8 * j]);
                        if (tail)
                            store_rest(static_cast<T*>(epi.pre) + (row + lane) * epi.ld_pre + edge, mine_pre + tail_at, rest);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (tma) tma_store_2d(&tmO.pre, bufs + 4096, col, row);
                    }
                    with_act(epi.act, [&](auto act) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) z[j] = act_f<act.value>(z[j]);
                    });
                    if (has_res) {
                        // every lane waits itself (that makes the block visible to it)
                        const uint32_t parity = (uint32_t)(n >> 1) & 1u;
                        ok = __all_sync(0xffffffffu, mbar_wait(&res_bar[bi], parity, abort_flag));
                        if (!ok) break;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint4 r = *reinterpret_cast<const uint4*>(mine + ((j ^ swz) << 4));
                            f32x2 f[4];
                            widen<T>(r, f);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 g = unpack2(f[i]);
                                z[8 * j + 2 * i] += g.x;
                                z[8 * j + 2 * i + 1] += g.y;
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4*>(mine + ((j ^ swz) << 4)) = narrow8<T>(&z[8 * j]);
                    if (tail)
                        store_rest(static_cast<T*>(epi.out) + (row + lane) * epi.ld_out + edge, mine + tail_at, rest);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (tma) tma_store_2d(&tmO.out, buf, col, row);
                        bulk_commit();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(&tempty[acc]);
                    else mbar_arrive_remote(peer_addr(&tempty[acc], 0));
                }
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1;
            }
            if (lane == 0) {
                // blocks still on their way (only after a wait ran out) land before the CTA exits
                if (*abort_flag) {
                    volatile int no_abort = 0;
                    for (int f = max(0, fetched - 2); f < fetched; ++f)
                        mbar_wait(&res_bar[f & 1], (uint32_t)(f >> 1) & 1u, &no_abort);
                    status_or(d.status, MOE_DEV_TIMEOUT);
                }
                bulk_wait_all();
            }
        } else {
            const int piece = lane & 7, sub = lane >> 3;  // columns 4 piece.., rows sub, sub + 4, ...
            uint8_t* buf = stage_out + (warp - 2) * 4096;
            int acc = 0;
            uint32_t acc_phase = 0;
            for (int u = pair; u < total; u += npairs) {
                int tm, tn;
                tile_of(u, mt, nt, tm, tn);
                const int row0 = tm * 256 + (int)rank * 128 + q * 32;
                const int chunks = (min(BN, d.C - tn * BN) + 31) / 32;
                // bias and residual of a chunk are loaded one chunk ahead, the first before the
                // accumulator is ready: their latency would otherwise stand in every chunk
                uint2 res[8];
                float4 b;
                auto ahead = [&](int c) {
                    const int col = tn * BN + c * 32 + piece * 4;
                    b = bias4(epi, col);
                    if (epi.res && quad_at(epi, col)) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (row0 + i * 4 + sub < d.R) res[i] = res4<T>(epi, row0 + i * 4 + sub, col);
                    }
                };
                ahead(grp);
                if (!mbar_wait(&tfull[acc], acc_phase, abort_flag)) break;
                tc_fence_after();
                const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * 256;
                for (int c = grp; c < chunks; c += 2) {
                    uint32_t r0[16], r1[16];
                    tmem_ld16(taddr + c * 32, r0);
                    tmem_ld16(taddr + c * 32 + 16, r1);
                    tmem_ld_wait(r0, r1);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t* s = j < 4 ? &r0[4 * j] : &r1[4 * (j - 4)];
                        *reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                            make_uint4(s[0], s[1], s[2], s[3]);
                    }
                    __syncwarp();
                    const int col = tn * BN + c * 32 + piece * 4;
                    const float4 bc = b;
                    uint2 rc[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) rc[i] = res[i];
                    if (c + 2 < chunks) ahead(c + 2);
                    if (col < d.C) {
                        with_act(epi.act, [&](auto act) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int r = i * 4 + sub;
                                const float4 v =
                                    *reinterpret_cast<const float4*>(buf + r * 128 + ((piece ^ (r & 7)) << 4));
                                if (row0 + r < d.R) store4<T, act.value>(epi, v, bc, rc[i], row0 + r, col);
                            }
                        });
                    }
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(&tempty[acc]);
                    else mbar_arrive_remote(peer_addr(&tempty[acc], 0));
                }
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_barrier();  // neither SM leaves while the pair may still use its memory
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// ------------------------------------------------------------------ split-K clusters
// One tile per cluster: 128 columns (MMA M, the matrix of the columns) x BT <= 128 rows
// (MMA N). Each of the cluster's CTAs runs its share of the k blocks and leaves its partial
// tile as [row][128] fp32 in its own shared memory; CTA p gathers rows p RP .. of all the
// partial tiles by bulk copies between the SMs, which complete on its barrier, adds them in
// rank order and stores them. (Reading the partial tiles through cluster barriers instead
// cost two release fences, ~1.5 us each, and the loads' latency once per peer.)
constexpr int kSplitThreads = 256;  // warp 0 TMA, warp 1 MMA; all drain, add and store
constexpr int kSplitMaxRows = 128;
constexpr int kSplitMaxStages = 12;
constexpr int kSplitHalf = 110 * 1024;  // shared memory of a CTA that shares its SM with another
constexpr int kSplitFixed = 1024 + 8 * (2 * kSplitMaxStages + 2) + 16;

template <bool MN>
__host__ __device__ constexpr int row_bytes_of(int bt) {  // shared-memory bytes of the row operand
    return MN ? (bt + 63) / 64 * 8192 : bt * BK * 2;
}

__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Bulk copy from this CTA's shared memory into that of cluster CTA `rank`, completing on
// the barrier at the same offset there.
__device__ __forceinline__ void copy_to_peer(void* dst, uint64_t* bar, uint32_t rank, const void* src, uint32_t bytes) {
    asm volatile(
        "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            peer_addr(dst, rank)),
        "r"(smem_u32(src)), "r"(bytes), "r"(peer_addr(bar, rank))
        : "memory");
}

template <typename T, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kSplitThreads)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const GemmDims d, const Epilogue epi, const int BT, const int stages,
                        const int tmem_cols, const int split) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int A_BYTES = 128 * BK * 2;
    const int b_bytes = row_bytes_of<B_MN>(BT);
    const int stage_bytes = A_BYTES + b_bytes;
    const int RP = (BT + split - 1) / split;  // rows a CTA adds and stores
    float* gather = reinterpret_cast<float*>(smem + stages * stage_bytes);  // [split][RP][128]
    uint64_t* full = reinterpret_cast<uint64_t*>(gather + (split > 1 ? split * RP * 128 : 0));
    uint64_t* empty = full + stages;
    uint64_t* tfull = empty + stages;
    uint64_t* gathered = tfull + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gathered + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = split > 1 ? (int)cluster_rank() : 0;
    const int ct = (d.C + 127) / 128;
    const int tile = (int)blockIdx.x / split;
    const int c0 = (tile % ct) * 128, r0 = (tile / ct) * BT;
    const int KB = (d.K + BK - 1) / BK;
    const int kb0 = (int)((long)KB * rank / split), kb1 = (int)((long)KB * (rank + 1) / split);
    const int n_valid = min(BT, d.R - r0);
    const int my_rows = max(0, min(RP, n_valid - rank * RP));

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(tfull, 1);
        mbar_init(gathered, 1);
        *abort_flag = 0;
        fence_barrier_init();
        if (split > 1 && my_rows > 0) mbar_arrive_expect_tx(gathered, (uint32_t)((split - 1) * my_rows * 512));
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    if (split > 1) cluster_arrive_relaxed();  // the barriers are initialised
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int issued = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) break;
                uint8_t* st = smem + stage * stage_bytes;
                mbar_arrive_expect_tx(&full[stage], (uint32_t)stage_bytes);
                if (A_MN) {
                    tma_load_2d(st, &tmA, c0, kb * BK, &full[stage]);
                    tma_load_2d(st + 8192, &tmA, c0 + 64, kb * BK, &full[stage]);
                } else {
                    tma_load_2d(st, &tmA, kb * BK, c0, &full[stage]);
                }
                if (B_MN) {
                    for (int i = 0; i * 64 < BT; ++i)
                        tma_load_2d(st + A_BYTES + i * 8192, &tmB, r0 + 64 * i, kb * BK, &full[stage]);
                } else {
                    tma_load_2d(st + A_BYTES, &tmB, kb * BK, r0, &full[stage]);
                }
                ++issued;
                if (++stage == stages) { stage = 0; phase ^= 1; }
            }
            if (*abort_flag) {  // let every copy land before the CTA exits
                volatile int no_abort = 0;
                int s = stage;
                uint32_t ph = phase;
                for (int i = 0; i < min(issued, stages); ++i) {
                    if (--s < 0) { s = stages - 1; ph ^= 1; }
                    mbar_wait(&full[s], ph, &no_abort);
                }
                status_or(d.status, MOE_DEV_TIMEOUT);
            }
        }
    } else if (warp == 1) {
        int stage = 0;
        uint32_t phase = 0;
        const uint32_t idesc = idesc_16<T, A_MN, B_MN>(128, BT);
        const uint64_t da = sdesc<A_MN>(smem_u32(smem)), db = sdesc<B_MN>(smem_u32(smem) + A_BYTES);
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!warp_wait(&full[stage], phase, abort_flag)) break;
            tc_fence_after();
            const uint64_t off = (uint64_t)((uint32_t)(stage * stage_bytes) >> 4);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk)
                    mma_bf16(tmem_base, da + off + kk * kStep<A_MN>, db + off + kk * kStep<B_MN>, idesc,
                             kb > kb0 || kk > 0);
                mma_commit(&empty[stage]);
            }
            __syncwarp();
            if (++stage == stages) { stage = 0; phase ^= 1; }
        }
        if (elect_one()) {
            mma_commit(tfull);
            volatile int no_abort = 0;
            mbar_wait(tfull, 0, &no_abort);  // every MMA this thread issued has finished
            if (*abort_flag) status_or(d.status, MOE_DEV_TIMEOUT);
        }
        __syncwarp();
    }
    __syncthreads();  // all MMAs are done: the stages are free for the partial tile
    tc_fence_after();
    float* part = reinterpret_cast<float*>(smem);
    {
        const int q = warp & 3;
        for (int c = (warp >> 2) * 16; c < n_valid; c += 32) {
            uint32_t v[16];
            tmem_ld16(tmem_base + ((uint32_t)(q * 32) << 16) + c, v);
            tmem_ld_wait(v);
#pragma unroll
            for (int j = 0; j < 16; ++j) part[(c + j) * 128 + q * 32 + lane] = __uint_as_float(v[j]);
        }
    }
    tc_fence_before();
    const int col = c0 + lane * 4;
    const float4 b = bias4(epi, col);
    bool ok = true;
    if (split > 1) {
        fence_proxy_async_smem();
        __syncthreads();
        cluster_wait();  // the peers' barriers are initialised
        if (warp == 0 && lane < split && lane != rank) {
            const int n = max(0, min(RP, n_valid - lane * RP));
            if (n > 0)
                copy_to_peer(gather + rank * RP * 128, gathered, lane, part + lane * RP * 128, (uint32_t)(n * 512));
        }
        if (my_rows > 0) ok = mbar_wait(gathered, 0, abort_flag);
        if (!ok) status_or(d.status, MOE_DEV_TIMEOUT);
        __syncwarp();
        cluster_arrive_relaxed();  // the peers' copies to this CTA have landed
    } else {
        __syncthreads();
    }
    // one row per warp, four at a time, all their loads before the first use
    constexpr int U = 4;
    for (int r = warp; r < my_rows && ok; r += 8 * U) {
        float4 a[U];
        uint2 res[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int ri = min(r + 8 * i, my_rows - 1);
            if (epi.res && quad_at(epi, col)) res[i] = res4<T>(epi, r0 + rank * RP + ri, col);
            a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int p = 0; p < split; ++p) {  // in rank order, this CTA's own partial tile in its turn
            const float* rows = p == rank ? part + rank * RP * 128 : gather + p * RP * 128;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int ri = min(r + 8 * i, my_rows - 1);
                const float4 v = *reinterpret_cast<const float4*>(rows + ri * 128 + lane * 4);
                a[i].x += v.x; a[i].y += v.y; a[i].z += v.z; a[i].w += v.w;
            }
        }
        if (col < d.C)
            with_act(epi.act, [&](auto act) {
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (r + 8 * i < my_rows)
                        store4<T, act.value>(epi, a[i], b, res[i], r0 + rank * RP + r + 8 * i, col);
            });
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, tmem_cols);
    }
    if (split > 1) cluster_wait();  // every copy out of this CTA has been taken
}

// ------------------------------------------------------------------ backward, elementwise
struct ActBwd {
    const void *dy, *pre;
    void* g;      // dy act'(pre), or null
    float* part;  // [chunks][N] column sums, or null
    long lddy, ldp, ldg;
    int M, N, act, rows;  // rows per CTA
};

// VEC elements of dy and pre into g; their fp32 products are added to sum.
template <typename T, int VEC, int ACT>
__device__ __forceinline__ Pack<T, VEC> act_grad(const Pack<T, VEC>& a, const Pack<T, VEC>& z, float (&sum)[VEC]) {
    Pack<T, VEC> o;
    float v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        v[j] = to_f32<T>(a.v[j]);
        if (ACT != MOE_ACT_NONE) v[j] *= act_slope<ACT>(to_f32<T>(z.v[j]));
        sum[j] += v[j];
    }
    if constexpr (VEC == 8) {
        *reinterpret_cast<uint4*>(&o) = narrow8<T>(v);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) o.v[j] = from_f32<T>(v[j]);
    }
    return o;
}

// CTA (x, y): 32 VEC columns x `rows` rows; warp w takes rows w, w + 8, ..., four at a time
// so that eight loads are in flight (one row at a time: 91 us, four: 70; 8192 x 7168 SiLU).
// The column sums of the unrounded products stay in registers, then cross the warps once.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(256) linear_act_bwd_kernel(ActBwd p) {
    pdl_wait();
    pdl_trigger();
    __shared__ float red[8][32 * VEC];
    using V = Pack<T, VEC>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = (blockIdx.x * 32 + lane) * VEC;
    const long m0 = (long)blockIdx.y * p.rows, m1 = min((long)p.M, m0 + p.rows);
    float sum[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[j] = 0.f;
    const T* dy = static_cast<const T*>(p.dy) + col;
    const T* pre = static_cast<const T*>(p.pre) + col;
    T* g = static_cast<T*>(p.g) + col;
    constexpr int U = 4;
    if (col + VEC <= p.N) {
        for (long m = m0 + warp; m < m1; m += 8 * U) {
            V a[U], z[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const long r = m + 8 * i;
                if (r < m1) {
                    a[i] = *reinterpret_cast<const V*>(dy + r * p.lddy);
                    if (ACT != MOE_ACT_NONE) z[i] = *reinterpret_cast<const V*>(pre + r * p.ldp);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const long r = m + 8 * i;
                if (r >= m1) continue;
                const V o = act_grad<T, VEC, ACT>(a[i], z[i], sum);
                if (p.g) *reinterpret_cast<V*>(g + r * p.ldg) = o;
            }
        }
    } else if (col < p.N) {  // the last, partial vector of a row; the workspace's rows are whole vectors
        for (long m = m0 + warp; m < m1; m += 8) {
            V a, z;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const bool in = col + j < p.N;
                a.v[j] = in ? dy[m * p.lddy + j] : from_f32<T>(0.f);
                z.v[j] = ACT != MOE_ACT_NONE && in ? pre[m * p.ldp + j] : from_f32<T>(0.f);
            }
            const V o = act_grad<T, VEC, ACT>(a, z, sum);
            if (p.g) *reinterpret_cast<V*>(g + m * p.ldg) = o;
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int j = 0; j < VEC; ++j) red[warp][lane * VEC + j] = sum[j];
    __syncthreads();
    for (int c = threadIdx.x; c < 32 * VEC; c += 256) {
        const int n = blockIdx.x * 32 * VEC + c;
        if (n >= p.N) continue;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += red[w][c];
        p.part[(size_t)blockIdx.y * p.N + n] = s;
    }
}

__global__ void __launch_bounds__(256) linear_bias_kernel(const float* __restrict__ part, int chunks, int N,
                                                          float* __restrict__ db) {
    pdl_wait();
    pdl_trigger();
    __shared__ float acc[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int n = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (n < N) {
#pragma unroll 4
        for (int i = w; i < chunks; i += 8) s += part[(size_t)i * N + n];
    }
    acc[w][lane] = s;
    __syncthreads();
    if (w == 0 && n < N) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += acc[i][lane];
        db[n] = s;
    }
}

// ------------------------------------------------------------------ plans and launches
inline int ceil_div(long a, long b) { return (int)((a + b - 1) / b); }

template <typename T>
constexpr CUtensorMapDataType kMapType =
    is_half<T>() ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;

// Tensor map of an operand with `rows` rows of K: K-major boxes of 64 k x box rows, or
// MN-major boxes of 64 rows x 64 k.
template <typename T, bool MN>
bool operand_map(CUtensorMap* tm, const void* p, long ld, long rows, long K, int box) {
    if (MN)
        return make_tmap_2d(tm, kMapType<T>, p, K, rows, ld * 2, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B);
    return make_tmap_2d(tm, kMapType<T>, p, rows, K, ld * 2, BK, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Rows that TMA can address (the stride of a single row counts for nothing).
inline bool on_grid(const void* p, long ld) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0);
}
template <typename T>
bool out_map(CUtensorMap* tm, const void* p, long ld, int rows, int cols) {
    return make_tmap_2d(tm, kMapType<T>, p, rows, cols, ld * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

// Which kernel and tile: the one whose busiest SM is done first, in SM cycles. A k block
// of a tile costs its tensor-core time (8192 FLOP a cycle) or its bytes from L2 (about 64 a
// cycle); a tile costs its epilogue besides.
struct Plan {
    bool pair;
    int bn;                                  // pair: columns per tile
    int bt, split, stages, tmem_cols, smem;  // split
};

// CTAs of `split`-CTA clusters that fit on the device at once, `per_sm` to an SM. Clusters of
// 4 and 8 leave SMs over (a GPC's SMs do not divide evenly): on a 148-SM B200 the driver
// reports 148, 148, 132, 120 CTAs one to an SM, and 296, 296, 284, 264 two to an SM. Constants,
// not a query: how the SMs of one GPU are spread over its GPCs must not decide the split, and with
// it the order of the additions.
int cluster_capacity(int split, int per_sm) {
    static const float share[2][4] = {{1.0f, 1.0f, 132.f / 148, 120.f / 148}, {1.0f, 1.0f, 284.f / 296, 264.f / 296}};
    const int l = split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3;
    return std::max(split, (int)(per_sm * num_sms() * share[per_sm - 1][l] + 0.5f));
}

template <bool B_MN>
Plan plan_gemm(int R, int C, int K) {
    const int sms = num_sms(), KB = ceil_div(K, BK);
    Plan best{};
    double best_t = 1e30;
    for (int bn = 256; bn >= 64; bn -= 32) {
        const long tiles = (long)ceil_div(R, 256) * ceil_div(C, bn);
        const double kb = std::max(2.0 * bn, (16384 + bn * 64) / 64.0);
        const double t = ceil_div(tiles, sms / 2) * (KB * kb + 400) + 45.0 * bn + 8000;
        if (t < best_t) {
            best_t = t;
            best = Plan{true, bn};
        }
    }
    const int passes = ceil_div(R, kSplitMaxRows);
    const int bt = (ceil_div(R, passes) + 15) / 16 * 16;
    const int stage = 128 * BK * 2 + row_bytes_of<B_MN>(bt);
    const long tiles = (long)ceil_div(C, 128) * ceil_div(R, bt);
    for (int split = 1; split <= 8 && split <= KB; split *= 2) {
        const int gather = split > 1 ? split * ceil_div(bt, split) * 512 : 0;
        for (int per_sm = 1; per_sm <= 2; ++per_sm) {
            const int fit = ((per_sm == 2 ? kSplitHalf : kSmemMax) - kSplitFixed - gather) / stage;
            const int stages = std::min(fit, kSplitMaxStages);
            // the partial tile lies in the stages
            if (stages < 3 || stages * stage < bt * 512) continue;
            const long ctas = tiles * split;
            const int waves = ceil_div(ctas, cluster_capacity(split, per_sm));
            const int share = waves == 1 ? std::max(1, ceil_div(ctas, sms)) : per_sm;  // CTAs an SM runs at once
            // the weights come from HBM once, about 25 bytes a cycle into one SM
            const double kb = share * std::max({2.0 * bt, (16384 + bt * 128) / 64.0, 16384 / (25.0 * passes)});
            const double t = waves * (std::max(ceil_div(KB, split) * kb, 1500.0) + 4000 + 8.0 * bt +
                                      30.0 * bt / split + (split > 1 ? 1500 + 4.0 * bt : 0.0)) + 6000;
            if (t < best_t) {
                best_t = t;
                int cols = 32;
                while (cols < bt) cols *= 2;
                best = Plan{false, 0, bt, split, stages, cols, kSplitFixed + gather + stages * stage};
            }
        }
    }
    return best;
}

// out[r][c] = sum_k R(r, k) C(c, k)
template <typename T, bool R_MN, bool C_MN>
cudaError_t product(const void* rp, long ldr, const void* cp, long ldc, const GemmDims& d, const Epilogue& e,
                    cudaStream_t st) {
    const Plan p = plan_gemm<R_MN>(d.R, d.C, d.K);
    CUtensorMap tr, tc;
    if (p.pair) {
        // stores clip in steps of 16 bytes: their maps end at the last multiple of 8 columns
        const int whole = d.C & ~7;
        const bool tma_out = whole > 0 && on_grid(e.out, e.ld_out) && on_grid(e.pre, e.ld_pre) && on_grid(e.res, e.ld_res);
        OutMaps to;
        if (tma_out) {
            if (!out_map<T>(&to.out, e.out, e.ld_out, d.R, whole) ||
                !out_map<T>(&to.pre, e.pre ? e.pre : e.out, e.pre ? e.ld_pre : e.ld_out, d.R, whole) ||
                !out_map<T>(&to.res, e.res ? e.res : e.out, e.res ? e.ld_res : e.ld_out, d.R, d.C))
                return cudaErrorInvalidValue;
        }
        auto kernel = tma_out ? linear_pair_kernel<T, R_MN, C_MN, true> : linear_pair_kernel<T, R_MN, C_MN, false>;
        if (cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(kernel), PairCfg::SMEM_BYTES))
            return err;
        if (!operand_map<T, R_MN>(&tr, rp, ldr, d.R, d.K, 128) ||
            !operand_map<T, C_MN>(&tc, cp, ldc, d.C, d.K, p.bn / 2))
            return cudaErrorInvalidValue;
        const long tiles = (long)ceil_div(d.R, 256) * ceil_div(d.C, p.bn);
        const int pairs = (int)std::min<long>(num_sms() / 2, tiles);
        return launch_cluster(kernel, dim3(2 * pairs), 2, PairCfg::THREADS, PairCfg::SMEM_BYTES, st, tr, tc,
                              to, d, e, p.bn);
    }
    auto kernel = linear_split_kernel<T, C_MN, R_MN>;
    if (cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(kernel), p.smem)) return err;
    if (!operand_map<T, C_MN>(&tc, cp, ldc, d.C, d.K, 128) ||
        !operand_map<T, R_MN>(&tr, rp, ldr, d.R, d.K, p.bt))
        return cudaErrorInvalidValue;
    const long tiles = (long)ceil_div(d.C, 128) * ceil_div(d.R, p.bt);
    return launch_cluster(kernel, dim3((unsigned)(tiles * p.split)), p.split, kSplitThreads, p.smem, st, tc, tr,
                          d, e, p.bt, p.stages, p.tmem_cols, p.split);
}

inline bool quad(const void* p, long ld) {  // 4-element accesses of 16-bit rows
    return !p || ((reinterpret_cast<uintptr_t>(p) & 7) == 0 && ld % 4 == 0);
}

template <typename T>
cudaError_t forward(const LinearArgs& a, cudaStream_t st) {
    const GemmDims d{a.M, a.N, a.K, a.status};
    Epilogue e{a.bias, a.res, a.y, a.pre, a.ldr, a.ldy, a.ldp, a.N, a.act, 0};
    e.vec = quad(a.res, a.ldr) && quad(a.y, a.ldy) && quad(a.pre, a.ldp) &&
            (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0;
    return product<T, false, false>(a.x, a.ldx, a.w, a.ldw, d, e, st);
}

constexpr int kBiasChunks = 64;  // row chunks of the column sums

inline long padded(long n) { return (n + 7) / 8 * 8; }

inline size_t align_up(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// rows per CTA of the elementwise step: enough CTAs to fill the GPU a few times, at most
// kBiasChunks along the rows, whole passes of 8 warps
inline int act_rows(int M, int N, int vec) {
    if (M <= 64) return 64;  // one chunk: its column sums are db already
    const int cx = ceil_div(N, 32 * vec);
    const int want = std::min(kBiasChunks, std::max(1, ceil_div(8L * num_sms(), cx)));
    return (ceil_div(M, want) + 7) / 8 * 8;
}

template <typename T>
cudaError_t backward(const LinearArgs& a, cudaStream_t st) {
    const bool direct = a.act == MOE_ACT_NONE && (reinterpret_cast<uintptr_t>(a.dy) & 15) == 0 && a.lddy % 8 == 0;
    const bool need_g = (a.dx || a.dw) && !direct;
    char* ws = static_cast<char*>(a.ws);
    const void* g = direct ? a.dy : ws;
    const long ldg = direct ? a.lddy : padded(a.N);
    if (need_g || a.db) {
        ActBwd p{a.dy, a.pre, need_g ? ws : nullptr,
                 a.db ? reinterpret_cast<float*>(ws + align_up((size_t)a.M * padded(a.N) * 2)) : nullptr,
                 a.lddy, a.ldp, ldg, a.M, a.N, a.act, 0};
        const bool vec = (reinterpret_cast<uintptr_t>(a.dy) & 15) == 0 && a.lddy % 8 == 0 &&
                         (a.act == MOE_ACT_NONE || ((reinterpret_cast<uintptr_t>(a.pre) & 15) == 0 && a.ldp % 8 == 0));
        p.rows = act_rows(a.M, a.N, vec ? 8 : 1);
        const int chunks = ceil_div(a.M, p.rows);
        if (chunks == 1 && a.db) p.part = a.db;
        const dim3 grid(ceil_div(a.N, vec ? 256 : 32), chunks);
        with_act(a.act, [&](auto act) {
            if (vec) launch_pdl(linear_act_bwd_kernel<T, 8, act.value>, grid, 256, 0, st, p);
            else launch_pdl(linear_act_bwd_kernel<T, 1, act.value>, grid, 256, 0, st, p);
        });
        if (a.db && chunks > 1)
            launch_pdl(linear_bias_kernel, ceil_div(a.N, 32), 256, 0, st, (const float*)p.part, chunks, a.N, a.db);
        if (cudaError_t err = cudaGetLastError()) return err;
    }
    Epilogue e{};
    e.act = MOE_ACT_NONE;
    if (a.dx) {
        e.out = a.dx;
        e.ld_out = a.lddx;
        e.cols = a.K;
        e.vec = quad(a.dx, a.lddx);
        const cudaError_t err =
            product<T, false, true>(g, ldg, a.w, a.ldw, GemmDims{a.M, a.K, a.N, a.status}, e, st);
        if (err != cudaSuccess) return err;
    }
    if (a.dw) {
        e.out = a.dw;
        e.ld_out = a.lddw;
        e.cols = a.K;
        e.vec = quad(a.dw, a.lddw);
        const cudaError_t err =
            product<T, true, true>(g, ldg, a.x, a.ldx, GemmDims{a.N, a.K, a.M, a.status}, e, st);
        if (err != cudaSuccess) return err;
    }
    return cudaGetLastError();
}

}  // namespace

size_t linear_backward_ws(int M, int N) {
    return align_up((size_t)M * padded(N) * 2) + (size_t)kBiasChunks * N * 4;
}

cudaError_t launch_linear(int dtype, const LinearArgs& a, cudaStream_t st) {
    return dtype == MOE_T_BF16 ? forward<__nv_bfloat16>(a, st) : forward<__half>(a, st);
}

cudaError_t launch_linear_backward(int dtype, const LinearArgs& a, cudaStream_t st) {
    return dtype == MOE_T_BF16 ? backward<__nv_bfloat16>(a, st) : backward<__half>(a, st);
}

}  // namespace moe
