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
//                        per pair, accumulators double-buffered in tensor memory;
//   linear_split_kernel  few tiles (serving, small gradients): 128 columns x BT rows per
//                        cluster of up to 8 CTAs that share the k range and add their
//                        partial tiles through distributed shared memory in rank order,
//                        so the weights stream through all SMs and equal calls give
//                        equal bits.
// Sums are fp32 in tensor memory; y, pre, dx and dW are rounded once to the tensors'
// type, and g once between dy and the products (the tensor cores take 16-bit operands).
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
__device__ __forceinline__ uint64_t sdesc(uint32_t base, int kk) {
    return MN ? sdesc_mnmajor_sw128(base + kk * 2048) : sdesc_kmajor_sw128(base + kk * 32);
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
    int rows, cols, act;
    int vec;  // out, res and pre allow 4-element accesses
};

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kGeluCubic = 0.044715f;

__device__ __forceinline__ float sigmoid_f(float z) { return 1.0f / (1.0f + __expf(-z)); }

// tanh through one exponential: accurate to a few units of 2^-24 of 1, saturating cleanly
__device__ __forceinline__ float tanh_f(float u) { return 1.0f - __fdividef(2.0f, 1.0f + __expf(2.0f * u)); }

__device__ __forceinline__ float act_f(float z, int act) {
    switch (act) {
    case MOE_ACT_RELU: return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    case MOE_ACT_SILU: return z * sigmoid_f(z);
    case MOE_ACT_GELU: return 0.5f * z * (1.0f + erff(z * kSqrtHalf));
    case MOE_ACT_GELU_TANH:
        return 0.5f * z * (1.0f + tanh_f(kSqrt2OverPi * (z + kGeluCubic * z * z * z)));
    }
    return z;
}

__device__ __forceinline__ float act_slope(float z, int act) {
    switch (act) {
    case MOE_ACT_RELU: return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    case MOE_ACT_SILU: {
        const float s = sigmoid_f(z);
        return s * (1.0f + z * (1.0f - s));
    }
    case MOE_ACT_GELU:
        return 0.5f * (1.0f + erff(z * kSqrtHalf)) + z * kInvSqrt2Pi * __expf(-0.5f * z * z);
    case MOE_ACT_GELU_TANH: {
        const float t = tanh_f(kSqrt2OverPi * (z + kGeluCubic * z * z * z));
        return 0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * kSqrt2OverPi * (1.0f + 3.0f * kGeluCubic * z * z);
    }
    }
    return 1.0f;
}

// Bias of columns col..col+3 (zero outside).
__device__ __forceinline__ void bias4(const Epilogue& e, int col, float (&b)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = e.bias && col + j < e.cols ? e.bias[col + j] : 0.f;
}

// Four neighbouring results of one row: bias, pre, activation, residual, store.
template <typename T>
__device__ __forceinline__ void store4(const Epilogue& e, const float (&acc)[4], const float (&b)[4],
                                       long row, int col) {
    float z[4], y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = acc[j] + b[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = act_f(z[j], e.act);
    T* out = static_cast<T*>(e.out) + row * e.ld_out + col;
    T* pre = static_cast<T*>(e.pre) + row * e.ld_pre + col;
    const T* res = static_cast<const T*>(e.res) + row * e.ld_res + col;
    if (e.vec && col + 4 <= e.cols) {
        Pack<T, 4> o;
        if (e.pre) {
#pragma unroll
            for (int j = 0; j < 4; ++j) o.v[j] = from_f32<T>(z[j]);
            *reinterpret_cast<Pack<T, 4>*>(pre) = o;
        }
        if (e.res) {
            const Pack<T, 4> r = *reinterpret_cast<const Pack<T, 4>*>(res);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] += to_f32<T>(r.v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[j] = from_f32<T>(y[j]);
        *reinterpret_cast<Pack<T, 4>*>(out) = o;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (col + j >= e.cols) break;
            if (e.pre) pre[j] = from_f32<T>(z[j]);
            if (e.res) y[j] += to_f32<T>(res[j]);
            out[j] = from_f32<T>(y[j]);
        }
    }
}

struct GemmDims {
    int R, C, K;  // out rows, out columns, reduction length
    int32_t* status;
};

// ------------------------------------------------------------------ CTA pairs
// 256 rows x BN columns per pair: each SM loads its 128 rows and half of the columns'
// operand, and drains its own 128 accumulator rows.
//   warp 0  TMA, warp 1 MMA (leader), warps 2-9 epilogue: four lane quadrants x two
//   groups that take alternate 32-column chunks. A chunk goes through the warp's own
//   4 KB of shared memory (16-byte pieces swizzled by row), so that global accesses run
//   along rows: 8 lanes per 64-byte row piece.
struct PairCfg {
    static constexpr int A_BYTES = 128 * BK * 2;
    static constexpr int STAGE_BYTES = 2 * A_BYTES;  // and up to 128 columns of the other
    static constexpr int STAGES = 6;
    static constexpr int EPI_WARPS = 8;
    static constexpr int EPI_BYTES = EPI_WARPS * 4096;
    static constexpr int THREADS = 32 * (2 + EPI_WARPS);
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_BYTES + 8 * (2 * STAGES + 5) + 16;
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

template <typename T, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(PairCfg::THREADS, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const GemmDims d, const Epilogue epi, const int BN) {
    pdl_wait();
    pdl_trigger();
    using C = PairCfg;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* stage_out = smem + C::STAGES * C::STAGE_BYTES;
    uint64_t* full = reinterpret_cast<uint64_t*>(stage_out + C::EPI_BYTES);
    uint64_t* empty = full + C::STAGES;
    uint64_t* tfull = empty + C::STAGES;
    uint64_t* tempty = tfull + 2;
    uint64_t* mma_done = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);   // the leader's expect-tx arrival covers both SMs' copies
            mbar_init(&empty[s], 1);  // the leader's multicast commit
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 2 * C::EPI_WARPS);  // both SMs' epilogue warps (leader's copy used)
        }
        mbar_init(mma_done, 1);
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
    const int half = BN / 2;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int issued = 0;
            const int b_boxes = B_MN ? (half + 63) / 64 : 1;
            const uint32_t tx = 2u * (uint32_t)(C::A_BYTES + (B_MN ? b_boxes * 8192 : half * BK * 2));
            for (int u = pair; u < total && !*abort_flag; u += npairs) {
                int tm, tn;
                tile_of(u, mt, nt, tm, tn);
                const int ra = tm * 256 + (int)rank * 128, rb = tn * BN + (int)rank * half;
                bool ok = true;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
                    uint8_t* st = smem + stage * C::STAGE_BYTES;
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
                    if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
            }
            if (*abort_flag) {
                // the copies of both SMs complete on the leader's barriers
                if (rank == 0) {
                    volatile int no_abort = 0;
                    int s = stage;
                    uint32_t ph = phase;
                    for (int i = 0; i < min(issued, C::STAGES); ++i) {
                        if (--s < 0) { s = C::STAGES - 1; ph ^= 1; }
                        mbar_wait(&full[s], ph, &no_abort);
                    }
                }
                status_or(d.status, MOE_DEV_TIMEOUT);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            const uint32_t idesc = idesc_16<T, A_MN, B_MN>(256, BN);
            for (int u = pair; u < total; u += npairs) {
                if (!mbar_wait(&tempty[acc], acc_phase ^ 1, abort_flag)) break;
                tc_fence_after();
                const uint32_t d0 = tmem_base + acc * 256;
                bool ok = true;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!mbar_wait(&full[stage], phase, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + stage * C::STAGE_BYTES);
                    const uint32_t sb = sa + C::A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk)
                        mma_pair_f16(d0, sdesc<A_MN>(sa, kk), sdesc<B_MN>(sb, kk), idesc, (kb | kk) != 0);
                    mma_commit_pair(&empty[stage]);
                    if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                mma_commit_pair(&tfull[acc]);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1;
            }
            mma_commit(mma_done);
            volatile int no_abort = 0;
            mbar_wait(mma_done, 0, &no_abort);
            if (*abort_flag) status_or(d.status, MOE_DEV_TIMEOUT);
        }
    } else {
        const int q = warp & 3, grp = (warp - 2) >> 2;
        uint8_t* buf = stage_out + (warp - 2) * 4096;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int u = pair; u < total; u += npairs) {
            int tm, tn;
            tile_of(u, mt, nt, tm, tn);
            if (!mbar_wait(&tfull[acc], acc_phase, abort_flag)) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * 256;
            const int row0 = tm * 256 + (int)rank * 128 + q * 32;
            const int chunks = (min(BN, d.C - tn * BN) + 31) / 32;
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
                const int piece = lane & 7, col = tn * BN + c * 32 + piece * 4;
                float b[4];
                bias4(epi, col, b);
                if (col < d.C) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = i * 4 + (lane >> 3);
                        const float4 v = *reinterpret_cast<const float4*>(buf + r * 128 + ((piece ^ (r & 7)) << 4));
                        const float a[4] = {v.x, v.y, v.z, v.w};
                        if (row0 + r < d.R) store4<T>(epi, a, b, row0 + r, col);
                    }
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

    tc_fence_before();
    __syncthreads();
    cluster_barrier();  // neither SM leaves while the pair may still use its memory
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// ------------------------------------------------------------------ split-K clusters
// One tile per cluster: 128 columns (MMA M, the matrix of the columns) x BT rows (MMA N).
// Each of the cluster's CTAs runs its share of the k blocks; the partial tiles, [row][128]
// fp32 in each CTA's shared memory, are added in rank order by the CTA that stores the row.
constexpr int kSplitThreads = 256;  // warp 0 TMA, warp 1 MMA, warps 4-7 drain, all store

constexpr int kSplitFixed = 1024 + 8 * (2 * 16 + 1) + 32;

template <bool MN>
__host__ __device__ constexpr int row_bytes_of(int bt) {  // shared-memory bytes of the row operand
    return MN ? (bt + 63) / 64 * 8192 : bt * BK * 2;
}

__device__ __forceinline__ float4 ld_peer(const void* p, uint32_t rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(peer_addr(p, rank))
                 : "memory");
    return v;
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
    const int data = max(stages * stage_bytes, BT * 512);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + data);
    uint64_t* empty = full + stages;
    uint64_t* tfull = empty + stages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = split > 1 ? (int)cluster_rank() : 0;
    const int ct = (d.C + 127) / 128;
    const int tile = (int)blockIdx.x / split;
    const int c0 = (tile % ct) * 128, r0 = (tile / ct) * BT;
    const int KB = (d.K + BK - 1) / BK;
    const int kb0 = (int)((long)KB * rank / split), kb1 = (int)((long)KB * (rank + 1) / split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(tfull, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
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
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            const uint32_t idesc = idesc_16<T, A_MN, B_MN>(128, BT);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(&full[stage], phase, abort_flag)) break;
                tc_fence_after();
                const uint32_t sa = smem_u32(smem + stage * stage_bytes);
                const uint32_t sb = sa + A_BYTES;
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk)
                    mma_bf16(tmem_base, sdesc<A_MN>(sa, kk), sdesc<B_MN>(sb, kk), idesc, kb > kb0 || kk > 0);
                mma_commit(&empty[stage]);
                if (++stage == stages) { stage = 0; phase ^= 1; }
            }
            mma_commit(tfull);
            volatile int no_abort = 0;
            mbar_wait(tfull, 0, &no_abort);  // every MMA this thread issued has finished
            if (*abort_flag) status_or(d.status, MOE_DEV_TIMEOUT);
        }
    }
    __syncthreads();  // all MMAs are done: the stages are free for the partial tile
    tc_fence_after();
    const int n_valid = min(BT, d.R - r0);
    if (warp >= 4) {
        const int q = warp & 3;
        float* part = reinterpret_cast<float*>(smem) + q * 32 + lane;
        for (int c = 0; c < n_valid; c += 16) {
            uint32_t v[16];
            tmem_ld16(tmem_base + ((uint32_t)(q * 32) << 16) + c, v);
            tmem_ld_wait(v);
#pragma unroll
            for (int j = 0; j < 16; ++j) part[(c + j) * 128] = __uint_as_float(v[j]);
        }
    }
    tc_fence_before();
    if (split > 1) cluster_barrier();
    else __syncthreads();
    const int col = c0 + lane * 4;
    float b[4];
    bias4(epi, col, b);
    for (int r = rank * 8 + warp; r < n_valid; r += split * 8) {
        const float* src = reinterpret_cast<const float*>(smem) + r * 128 + lane * 4;
        float a[4] = {0.f, 0.f, 0.f, 0.f};
        if (split == 1) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            a[0] = v.x; a[1] = v.y; a[2] = v.z; a[3] = v.w;
        } else {
#pragma unroll 8
            for (int p = 0; p < split; ++p) {
                const float4 v = ld_peer(src, p);
                a[0] += v.x; a[1] += v.y; a[2] += v.z; a[3] += v.w;
            }
        }
        if (col < d.C) store4<T>(epi, a, b, r0 + r, col);
    }
    if (split > 1) cluster_barrier();  // no CTA leaves while others read its partial tile
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, tmem_cols);
    }
}

// ------------------------------------------------------------------ backward, elementwise
struct ActBwd {
    const void *dy, *pre;
    void* g;      // dy act'(pre), or null
    float* part;  // [chunks][N] column sums, or null
    long lddy, ldp, ldg;
    int M, N, act, rows;  // rows per CTA
};

// CTA (x, y): 32 VEC columns x `rows` rows; warp w takes rows w, w + 8, ... The column
// sums of the unrounded products stay in registers, then cross the warps once.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) linear_act_bwd_kernel(ActBwd p) {
    pdl_wait();
    pdl_trigger();
    __shared__ float red[8][32 * VEC];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = (blockIdx.x * 32 + lane) * VEC;
    const long m0 = (long)blockIdx.y * p.rows, m1 = min((long)p.M, m0 + p.rows);
    float sum[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[j] = 0.f;
    const bool whole = col + VEC <= p.N;
    if (col < p.N) {
        for (long m = m0 + warp; m < m1; m += 8) {
            const T* dy = static_cast<const T*>(p.dy) + m * p.lddy + col;
            const T* pre = static_cast<const T*>(p.pre) + m * p.ldp + col;
            Pack<T, VEC> a, z, o;
            if (VEC == 1 || whole) {
                a = *reinterpret_cast<const Pack<T, VEC>*>(dy);
                if (p.act != MOE_ACT_NONE) z = *reinterpret_cast<const Pack<T, VEC>*>(pre);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    a.v[j] = col + j < p.N ? dy[j] : from_f32<T>(0.f);
                    z.v[j] = p.act != MOE_ACT_NONE && col + j < p.N ? pre[j] : from_f32<T>(0.f);
                }
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float v = to_f32<T>(a.v[j]);
                if (p.act != MOE_ACT_NONE) v *= act_slope(to_f32<T>(z.v[j]), p.act);
                sum[j] += v;
                o.v[j] = from_f32<T>(v);
            }
            // the workspace's rows are padded to whole vectors
            if (p.g) *reinterpret_cast<Pack<T, VEC>*>(static_cast<T*>(p.g) + m * p.ldg + col) = o;
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

// Which kernel and tile: the one whose busiest SM is done first, in SM cycles. A k block
// of a tile costs its tensor-core time (8192 FLOP a cycle) or its bytes from L2 (about 56 a
// cycle); a tile costs its epilogue besides.
struct Plan {
    bool pair;
    int bn;                                  // pair: columns per tile
    int bt, split, stages, tmem_cols, smem;  // split
};

template <bool B_MN>
Plan plan_gemm(int R, int C, int K) {
    const int sms = num_sms(), KB = ceil_div(K, BK);
    Plan best{};
    double best_t = 1e30;
    for (int bn = 256; bn >= 64; bn -= 32) {
        const long tiles = (long)ceil_div(R, 256) * ceil_div(C, bn);
        const double kb = std::max(2.0 * bn, (16384 + bn * 64) / 56.0);
        const double t = ceil_div(tiles, sms / 2) * (KB * kb + 400) + 12.0 * bn + 4000;
        if (t < best_t) {
            best_t = t;
            best = Plan{true, bn};
        }
    }
    const int passes = ceil_div(R, 256);
    const int bt = (ceil_div(R, passes) + 15) / 16 * 16;
    const int stage = 128 * BK * 2 + row_bytes_of<B_MN>(bt);
    // two CTAs an SM where half the shared memory holds a deep enough ring
    const int per_sm = 4 * stage <= 110 * 1024 ? 2 : 1;
    const int budget = per_sm == 2 ? 110 * 1024 : kSmemMax;
    const int stages = std::min(16, (budget - kSplitFixed) / stage);
    const long tiles = (long)ceil_div(C, 128) * passes;
    int split = 1;
    while (split < 8 && tiles * split * 2 <= (long)per_sm * sms && 2 * split * 2 <= KB) split *= 2;
    const double kb = per_sm * std::max(2.0 * bt, (16384 + bt * 128) / 56.0);
    const double t = ceil_div(tiles * split, per_sm * sms) * (ceil_div(KB, split) * kb + 2000 + 10.0 * bt) +
                     3000 + (split > 1 ? 1500 : 0);
    if (t < best_t) {
        int cols = 32;
        while (cols < bt) cols *= 2;
        const int data = std::max(stages * stage, bt * 512);
        best = Plan{false, 0, bt, split, stages, cols, kSplitFixed + data};
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
        auto kernel = linear_pair_kernel<T, R_MN, C_MN>;
        if (cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(kernel), PairCfg::SMEM_BYTES))
            return err;
        if (!operand_map<T, R_MN>(&tr, rp, ldr, d.R, d.K, 128) ||
            !operand_map<T, C_MN>(&tc, cp, ldc, d.C, d.K, p.bn / 2))
            return cudaErrorInvalidValue;
        const long tiles = (long)ceil_div(d.R, 256) * ceil_div(d.C, p.bn);
        const int pairs = (int)std::min<long>(num_sms() / 2, tiles);
        return launch_cluster(kernel, dim3(2 * pairs), 2, PairCfg::THREADS, PairCfg::SMEM_BYTES, st, tr, tc, d,
                              e, p.bn);
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
    Epilogue e{a.bias, a.res, a.y, a.pre, a.ldr, a.ldy, a.ldp, a.M, a.N, a.act, 0};
    e.vec = quad(a.res, a.ldr) && quad(a.y, a.ldy) && quad(a.pre, a.ldp);
    return product<T, false, false>(a.x, a.ldx, a.w, a.ldw, d, e, st);
}

constexpr int kBiasChunks = 64;  // row chunks of the column sums

inline long padded(long n) { return (n + 7) / 8 * 8; }

inline size_t align_up(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// rows per CTA of the elementwise step: enough CTAs to fill the GPU a few times, at most
// kBiasChunks along the rows, whole passes of 8 warps
inline int act_rows(int M, int N, int vec) {
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
        const dim3 grid(ceil_div(a.N, vec ? 256 : 32), chunks);
        if (vec) launch_pdl(linear_act_bwd_kernel<T, 8>, grid, 256, 0, st, p);
        else launch_pdl(linear_act_bwd_kernel<T, 1>, grid, 256, 0, st, p);
        if (a.db)
            launch_pdl(linear_bias_kernel, ceil_div(a.N, 32), 256, 0, st, (const float*)p.part, chunks, a.N, a.db);
        if (cudaError_t err = cudaGetLastError()) return err;
    }
    Epilogue e{};
    e.act = MOE_ACT_NONE;
    if (a.dx) {
        e.out = a.dx;
        e.ld_out = a.lddx;
        e.rows = a.M;
        e.cols = a.K;
        e.vec = quad(a.dx, a.lddx);
        const cudaError_t err =
            product<T, false, true>(g, ldg, a.w, a.ldw, GemmDims{a.M, a.K, a.N, a.status}, e, st);
        if (err != cudaSuccess) return err;
    }
    if (a.dw) {
        e.out = a.dw;
        e.ld_out = a.lddw;
        e.rows = a.N;
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
