// abi_ops.cu -- the extern "C" entry points of the operators around the routed
// experts (norm, routing of given logits, the combine's gradient, the linear layer):
// argument checks and launches.
#include <cmath>

#include "internal.h"

using namespace moe;

static inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

static inline bool aligned(const void* p, size_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

static inline bool dtype_ok(int d) { return d == MOE_T_BF16 || d == MOE_T_F16 || d == MOE_T_F32; }

// A row operand: present, aligned to its elements, rows that do not overlap.
static inline bool rows_ok(const void* p, int64_t ld, int64_t cols, int dtype) {
    return p && ld >= cols && ld <= (int64_t)1 << 40 && aligned(p, esize(dtype));
}

// A matrix that TMA reads: 16-byte aligned rows; the stride of a single row counts for
// nothing.
static inline bool tma_rows_ok(const void* p, int64_t ld, int rows, int64_t cols, int dtype) {
    return p && aligned(p, 16) && (rows == 1 || (rows_ok(p, ld, cols, dtype) && ld % 8 == 0));
}
static inline int64_t tma_ld(int64_t ld, int rows, int64_t cols) { return rows == 1 ? (cols + 7) / 8 * 8 : ld; }

static moe_status linear_sizes(int dtype, int act, int M, int N, int K) {
    if (!dtype_ok(dtype) || act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH || M < 0 || N < 1 || K < 1)
        return MOE_ERR_INVALID_ARG;
    // sizes round up to whole tiles in 32 bits
    if (M > 0x7fffff00 || N > 0x7fffff00 || K > 0x7fffff00) return MOE_ERR_INVALID_ARG;
    return dtype == MOE_T_F32 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

constexpr int kNormMaxH = 16384;

extern "C" {

moe_status moe_norm(int32_t kind, int32_t dtype, const void* x, int64_t ldx, int32_t T, int32_t H,
                    const float* w, const float* b, float eps, void* y, int64_t ldy, float* mean,
                    float* rstd, void* stream) {
    if (kind != MOE_NORM_LAYER && kind != MOE_NORM_RMS) return MOE_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || T < 0 || H < 1 || !(eps >= 0.0f) || std::isinf(eps)) return MOE_ERR_INVALID_ARG;
    if (H > kNormMaxH) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!rows_ok(x, ldx, H, dtype) || !rows_ok(y, ldy, H, dtype)) return MOE_ERR_INVALID_ARG;
    if (!aligned(w, 4) || !aligned(b, 4) || !aligned(mean, 4) || !aligned(rstd, 4)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_norm_fwd(kind, dtype, x, ldx, T, H, w, b, eps, y, ldy, mean, rstd,
                                       as_stream(stream)));
}

size_t moe_norm_backward_workspace_bytes(int32_t T, int32_t H) {
    if (T < 0 || H < 1 || H > kNormMaxH) return 0;
    return norm_backward_ws(T, H);
}

moe_status moe_norm_backward(int32_t kind, int32_t dtype, const void* dy, int64_t lddy, const void* x,
                             int64_t ldx, int32_t T, int32_t H, const float* w, const float* mean,
                             const float* rstd, void* dx, int64_t lddx, float* dw, float* db, void* ws,
                             size_t ws_bytes, void* stream) {
    if (kind != MOE_NORM_LAYER && kind != MOE_NORM_RMS) return MOE_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || T < 0 || H < 1) return MOE_ERR_INVALID_ARG;
    if (H > kNormMaxH) return MOE_ERR_UNSUPPORTED;
    if (kind == MOE_NORM_RMS) db = nullptr;
    if (!dx && !dw && !db) return MOE_OK;
    if (!aligned(w, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dw, 4) || !aligned(db, 4))
        return MOE_ERR_INVALID_ARG;
    if (T > 0) {
        if (!rows_ok(dy, lddy, H, dtype) || !rows_ok(x, ldx, H, dtype)) return MOE_ERR_INVALID_ARG;
        if (dx && !rows_ok(dx, lddx, H, dtype)) return MOE_ERR_INVALID_ARG;
        if (!rstd || (kind == MOE_NORM_LAYER && !mean)) return MOE_ERR_INVALID_ARG;
        if (dw || db) {
            if (!ws || !aligned(ws, 16)) return MOE_ERR_INVALID_ARG;
            if (ws_bytes < norm_backward_ws(T, H)) return MOE_ERR_WORKSPACE;
        }
    }
    return cuda_status(launch_norm_bwd(kind, dtype, dy, lddy, x, ldx, T, H, w, mean, rstd, dx, lddx, dw,
                                       db, static_cast<float*>(ws), as_stream(stream)));
}

moe_status moe_route(const moe_config* cfg, int32_t dtype, const void* logits, int64_t ld, int32_t T,
                     const float* bias, int32_t* topk_idx, float* topk_w, void* stream) {
    if (!config_valid(cfg) || !dtype_ok(dtype) || T < 0) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!rows_ok(logits, ld, cfg->n_routed_experts, dtype) || !topk_idx || !topk_w) return MOE_ERR_INVALID_ARG;
    if (!aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_route(cfg, dtype, logits, ld, T, bias, topk_idx, topk_w, as_stream(stream)));
}

moe_status moe_route_backward(const moe_config* cfg, int32_t dtype, const void* logits, int64_t ld,
                              int32_t T, const int32_t* topk_idx, const float* dtopk_w, void* dlogits,
                              int64_t ldd, void* stream) {
    if (!config_valid(cfg) || !dtype_ok(dtype) || T < 0) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const int E = cfg->n_routed_experts;
    if (!rows_ok(logits, ld, E, dtype) || !rows_ok(dlogits, ldd, E, dtype)) return MOE_ERR_INVALID_ARG;
    if (!topk_idx || !dtopk_w || !aligned(topk_idx, 4) || !aligned(dtopk_w, 4)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_route_backward(cfg, dtype, logits, ld, T, topk_idx, dtopk_w, dlogits, ldd,
                                             as_stream(stream)));
}

moe_status moe_combine_backward(const moe_config* cfg, const void* dout, const void* y,
                                const int32_t* row_of, const float* topk_w, int32_t T, void* dy,
                                float* dtopk_w, void* stream) {
    if (!config_valid(cfg) || T < 0) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if ((int64_t)T * cfg->num_experts_per_tok > 0x7fffffffLL) return MOE_ERR_INVALID_ARG;
    if (!dout || !row_of || !topk_w || !dy || (dtopk_w && !y)) return MOE_ERR_INVALID_ARG;
    if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16)) return MOE_ERR_INVALID_ARG;
    if (!aligned(row_of, 4) || !aligned(topk_w, 4) || !aligned(dtopk_w, 4)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_combine_backward(dout, y, row_of, topk_w, T, cfg->num_experts_per_tok,
                                               cfg->hidden, dy, dtopk_w, as_stream(stream)));
}

moe_status moe_linear(int32_t dtype, const void* x, int64_t ldx, const void* w, int64_t ldw,
                      const float* bias, const void* residual, int64_t ldr, int32_t act, int32_t M, int32_t N,
                      int32_t K, void* y, int64_t ldy, void* pre, int64_t ldp, int32_t* dev_status,
                      void* stream) {
    const moe_status st = linear_sizes(dtype, act, M, N, K);
    if (st != MOE_OK || M == 0) return st;
    if (!tma_rows_ok(x, ldx, M, K, dtype) || !tma_rows_ok(w, ldw, N, K, dtype)) return MOE_ERR_INVALID_ARG;
    if (!rows_ok(y, ldy, N, dtype)) return MOE_ERR_INVALID_ARG;
    if ((residual && !rows_ok(residual, ldr, N, dtype)) || (pre && !rows_ok(pre, ldp, N, dtype)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(bias, 4) || !aligned(dev_status, 4)) return MOE_ERR_INVALID_ARG;
    LinearArgs a{};
    a.M = M;
    a.N = N;
    a.K = K;
    a.act = act;
    a.x = x;
    a.ldx = tma_ld(ldx, M, K);
    a.w = w;
    a.ldw = tma_ld(ldw, N, K);
    a.bias = bias;
    a.res = residual;
    a.ldr = ldr;
    a.y = y;
    a.ldy = ldy;
    a.pre = pre;
    a.ldp = ldp;
    a.status = dev_status;
    return cuda_status(launch_linear(dtype, a, as_stream(stream)));
}

size_t moe_linear_backward_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t act) {
    if (linear_sizes(MOE_T_BF16, act, M, N, K) != MOE_OK) return 0;
    return linear_backward_ws(M, N);
}

moe_status moe_linear_backward(int32_t dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                               const void* w, int64_t ldw, const void* pre, int64_t ldp, int32_t act, int32_t M,
                               int32_t N, int32_t K, void* dx, int64_t lddx, void* dw, int64_t lddw, float* db,
                               void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
    const moe_status st = linear_sizes(dtype, act, M, N, K);
    if (st != MOE_OK) return st;
    if (!dx && !dw && !db) return MOE_OK;
    if ((dw && !rows_ok(dw, lddw, K, dtype)) || !aligned(db, 4) || !aligned(dev_status, 4)) return MOE_ERR_INVALID_ARG;
    if (M == 0) {  // no rows: the sums are zero
        cudaError_t e = cudaSuccess;
        if (dw) e = cudaMemset2DAsync(dw, (size_t)lddw * 2, 0, (size_t)K * 2, N, as_stream(stream));
        if (db && e == cudaSuccess) e = cudaMemsetAsync(db, 0, (size_t)N * 4, as_stream(stream));
        return cuda_status(e);
    }
    if (!rows_ok(dy, lddy, N, dtype)) return MOE_ERR_INVALID_ARG;
    if (act != MOE_ACT_NONE && !rows_ok(pre, ldp, N, dtype)) return MOE_ERR_INVALID_ARG;
    if (dx && (!rows_ok(dx, lddx, K, dtype) || !tma_rows_ok(w, ldw, N, K, dtype))) return MOE_ERR_INVALID_ARG;
    if (dw && !tma_rows_ok(x, ldx, M, K, dtype)) return MOE_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, 16)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < linear_backward_ws(M, N)) return MOE_ERR_WORKSPACE;
    LinearArgs a{};
    a.M = M;
    a.N = N;
    a.K = K;
    a.act = act;
    a.dy = dy;
    a.lddy = M == 1 ? tma_ld(lddy, M, N) : lddy;
    a.x = x;
    a.ldx = tma_ld(ldx, M, K);
    a.w = w;
    a.ldw = tma_ld(ldw, N, K);
    a.pre = const_cast<void*>(pre);
    a.ldp = ldp;
    a.dx = dx;
    a.lddx = lddx;
    a.dw = dw;
    a.lddw = lddw;
    a.db = db;
    a.ws = ws;
    a.status = dev_status;
    return cuda_status(launch_linear_backward(dtype, a, as_stream(stream)));
}

}  // extern "C"
