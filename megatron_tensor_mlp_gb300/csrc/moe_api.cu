// C-ABI entry points of layer norm, routing, the products grouped by expert and the combination of their rows.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <utility>

#include "api_common.h"
#include "internal.h"

namespace tpmlp {
namespace {

constexpr int kMaxExperts = 1024, kMaxChoice = 32;
constexpr int64_t kMaxNormWidth = 16384;

// A NULL pointer is refused where its tensor has elements (an empty one has no address to pass).
tpmlp_status need(std::initializer_list<std::pair<const void*, bool>> ptrs) {
    int i = 0;
    for (const auto& p : ptrs) {
        if (p.second && p.first == nullptr) {
            set_error("pointer %d must not be NULL", i);
            return TPMLP_ERR_NULL;
        }
        ++i;
    }
    return TPMLP_OK;
}

// rows x cols of at most 2^40 bytes (4 an element); 32-bit indexes run up to a tile past either.
tpmlp_status check_matrix(int64_t rows, int64_t cols, const char* what) {
    if (rows < 0 || cols < 1 || rows > kMaxDim - 1024 || cols > kMaxDim - 1024) {
        set_error("bad shape: %s is %lld x %lld", what, (long long)rows, (long long)cols);
        return TPMLP_ERR_SHAPE;
    }
    if (rows > 0 && cols > ((int64_t(1) << 40) / 4) / rows) {
        set_error("shape too large: %s (%lld x %lld) would exceed 2^40 bytes", what, (long long)rows, (long long)cols);
        return TPMLP_ERR_SHAPE;
    }
    return TPMLP_OK;
}

tpmlp_status check_elements(std::initializer_list<const void*> ptrs, int es) {
    int i = 0;
    for (const void* p : ptrs) {
        if (p && reinterpret_cast<uintptr_t>(p) % es != 0) {
            set_error("pointer argument %d is not aligned to its %d-byte elements", i, es);
            return TPMLP_ERR_ALIGNMENT;
        }
        ++i;
    }
    return TPMLP_OK;
}

tpmlp_status check_norm(int64_t rows, int64_t h, std::initializer_list<int64_t> pitches, tpmlp_dtype dt) {
    if (h > kMaxNormWidth) {
        set_error("rows of %lld elements: at most %lld", (long long)h, (long long)kMaxNormWidth);
        return TPMLP_ERR_SHAPE;
    }
    TP_TRY(check_matrix(rows, h, "X"));
    for (int64_t l : pitches) {
        if (l < h) {
            set_error("row pitch %lld is less than the %lld elements of a row", (long long)l, (long long)h);
            return TPMLP_ERR_SHAPE;
        }
        TP_TRY(check_matrix(rows, l, "a row pitch"));
    }
    return check_dtype(dt);
}
Range pitched(const void* p, int64_t rows, int64_t h, int64_t ld, int es) {
    return {p, rows == 0 ? 0 : ((rows - 1) * ld + h) * es, h * es, ld * es};
}

tpmlp_status check_choice(int64_t tokens, int64_t experts, int k) {
    if (tokens < 0 || experts < 1 || experts > kMaxExperts || k < 1 || k > kMaxChoice || k > experts) {
        set_error("bad shape: tokens=%lld experts=%lld (1..%d) k=%d (1..%d, at most the experts)", (long long)tokens, (long long)experts,
                  kMaxExperts, k, kMaxChoice);
        return TPMLP_ERR_SHAPE;
    }
    if (tokens > kMaxDim / kMaxChoice / 2) {
        set_error("shape too large: %lld tokens", (long long)tokens);
        return TPMLP_ERR_SHAPE;
    }
    return TPMLP_OK;
}

// Rows, tokens and the experts' weights [experts][K][N] of a grouped product.
tpmlp_status check_experts(int64_t tokens, int64_t rows, int64_t experts, int64_t K, int64_t N, bool src) {
    if (experts < 1 || experts > kMaxExperts) {
        set_error("bad shape: %lld experts (1..%d)", (long long)experts, kMaxExperts);
        return TPMLP_ERR_SHAPE;
    }
    TP_TRY(check_matrix(rows, K, "the rows' tensor"));
    TP_TRY(check_matrix(rows, N, "the rows' other tensor"));
    if (src) {
        TP_TRY(check_matrix(tokens, K, "X"));
        if (tokens == 0 && rows > 0) {
            set_error("bad shape: %lld rows of no tokens", (long long)rows);
            return TPMLP_ERR_SHAPE;
        }
    } else if (tokens != rows) {
        set_error("bad shape: without row_token X has the rows themselves (tokens=%lld, rows=%lld)", (long long)tokens, (long long)rows);
        return TPMLP_ERR_SHAPE;
    }
    TP_TRY(check_matrix(experts * K, N, "the weights"));
    // tiles are counted in 32 bits
    const int64_t blocks = ((K + 255) / 256) * ((N + 255) / 256), tiles = (std::max(K, N) / 64 + 1) * (rows / 64 + experts);
    if (blocks > kMaxDim / experts || tiles > kMaxDim) {
        set_error("shape too large: more than 2^31 tiles");
        return TPMLP_ERR_SHAPE;
    }
    return TPMLP_OK;
}

tpmlp_status check_act(tpmlp_act act) {
    if (act != TPMLP_ACT_NONE && act != TPMLP_ACT_SWIGLU && act != TPMLP_ACT_SWIGLU_H32) {
        set_error("activation %d: none or the gated one", (int)act);
        return TPMLP_ERR_SHAPE;
    }
    return TPMLP_OK;
}

tpmlp_status check_gate_width(int64_t packed) {
    if (packed % 256 != 0) {
        set_error("%lld packed gate and up columns: a multiple of 256 is needed", (long long)packed);
        return TPMLP_ERR_DIVISIBILITY;
    }
    return TPMLP_OK;
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;

extern "C" {

tpmlp_status tpmlp_layernorm_fwd(const void* X, const void* gamma, const void* beta, void* Y, void* mean, void* rstd, int64_t rows,
                                 int64_t h, int64_t ldx, int64_t ldy, float eps, tpmlp_dtype dt, void* stream) {
    TP_TRY(need({{X, rows > 0}, {Y, rows > 0}}));
    if (rows > 0 && !mean != !rstd) {
        set_error("mean and rstd come together");
        return TPMLP_ERR_NULL;
    }
    TP_TRY(check_norm(rows, h, {ldx, ldy}, dt));
    if (!(eps >= 0.0f) || std::isinf(eps)) {
        set_error("eps=%g is not a finite number at or above zero", (double)eps);
        return TPMLP_ERR_SHAPE;
    }
    const int es = esize(dt);
    TP_TRY(check_elements({X, gamma, beta, Y}, es));
    TP_TRY(check_elements({mean, rstd}, 4));
    TP_TRY(check_alias({pitched(Y, rows, h, ldy, es), {mean, rows * 4}, {rstd, rows * 4}},
                       {pitched(X, rows, h, ldx, es), {gamma, h * es}, {beta, h * es}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    if (rows == 0) return TPMLP_OK;
    return launch_layernorm_fwd(X, gamma, beta, Y, static_cast<float*>(mean), static_cast<float*>(rstd), rows, h, ldx, ldy, eps,
                                dt == TPMLP_F32, *dev, static_cast<cudaStream_t>(stream));
}

int64_t tpmlp_layernorm_ws_bytes(int64_t rows, int64_t h) {
    return check_norm(rows, h, {}, TPMLP_BF16) == TPMLP_OK ? layernorm_ws_bytes(rows, h) : -1;
}

tpmlp_status tpmlp_layernorm_bwd(const void* X, const void* gamma, const void* mean, const void* rstd, const void* dY, void* dX,
                                 void* dgamma, void* dbeta, void* ws, int64_t rows, int64_t h, int64_t ldx, int64_t lddy, int64_t lddx,
                                 tpmlp_dtype dt, tpmlp_dtype grad_dt, void* stream) {
    const bool some = rows > 0, sums = dgamma || dbeta;
    TP_TRY(need({{X, some}, {mean, some}, {rstd, some}, {dY, some}, {dX, some}, {ws, some && sums}}));
    TP_TRY(check_norm(rows, h, {ldx, lddy, lddx}, dt));
    TP_TRY(check_dtype(grad_dt));
    const int es = esize(dt), gs = esize(grad_dt);
    TP_TRY(check_elements({X, gamma, dY, dX}, es));
    TP_TRY(check_elements({dgamma, dbeta}, gs));
    TP_TRY(check_elements({mean, rstd}, 4));
    TP_TRY(check_aligned({sums ? ws : nullptr}));
    TP_TRY(check_alias({pitched(dX, rows, h, lddx, es), {dgamma, h * gs}, {dbeta, h * gs}, {sums ? ws : nullptr, layernorm_ws_bytes(rows, h)}},
                       {pitched(X, rows, h, ldx, es), {gamma, h * es}, {mean, rows * 4}, {rstd, rows * 4}, pitched(dY, rows, h, lddy, es)}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) {  // sums over nothing
        for (void* d : {dgamma, dbeta})
            if (d) TP_TRY(clear_memory(d, h * gs, st));
        return TPMLP_OK;
    }
    return launch_layernorm_bwd(X, gamma, static_cast<const float*>(mean), static_cast<const float*>(rstd), dY, dX, dgamma, dbeta, ws, rows,
                                h, ldx, lddy, lddx, dt == TPMLP_F32, grad_dt == TPMLP_F32, *dev, st);
}

int64_t tpmlp_moe_route_ws_bytes(int64_t tokens, int64_t experts, int k) {
    return check_choice(tokens, experts, k) == TPMLP_OK ? moe_route_ws_bytes(tokens, static_cast<int>(experts)) : -1;
}

tpmlp_status tpmlp_moe_route(const void* logits, void* ids, void* weights, void* offsets, void* row_token, void* slot_row, void* ws,
                             int64_t tokens, int64_t experts, int k, int chosen, tpmlp_dtype dt, void* stream) {
    const bool some = tokens > 0;
    TP_TRY(need({{logits, some}, {ids, some}, {weights, some}, {offsets, true}, {row_token, some}, {slot_row, some}, {ws, some}}));
    TP_TRY(check_choice(tokens, experts, k));
    TP_TRY(check_dtype(dt));
    const int es = esize(dt);
    TP_TRY(check_elements({logits}, es));
    TP_TRY(check_elements({ids, weights, offsets, row_token, slot_row}, 4));
    TP_TRY(check_aligned({ws}));
    const int64_t slots = tokens * k * 4;
    TP_TRY(check_alias({{ids, slots}, {weights, slots}, {offsets, (experts + 1) * 4}, {row_token, slots}, {slot_row, slots},
                        {ws, moe_route_ws_bytes(tokens, static_cast<int>(experts))}},
                       {{logits, tokens * experts * es}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (tokens == 0) return clear_memory(offsets, (experts + 1) * 4, st);
    return launch_moe_route(logits, static_cast<int*>(ids), static_cast<float*>(weights), static_cast<int*>(offsets),
                            static_cast<int*>(row_token), static_cast<int*>(slot_row), ws, tokens, static_cast<int>(experts), k, chosen != 0,
                            dt == TPMLP_F32, st);
}

tpmlp_status tpmlp_moe_route_bwd(const void* logits, const void* ids, const void* weights, const void* dweights, void* dlogits,
                                 int64_t tokens, int64_t experts, int k, int chosen, tpmlp_dtype dt, void* stream) {
    const bool some = tokens > 0;
    TP_TRY(need({{logits, some}, {ids, some}, {weights, some}, {dweights, some}, {dlogits, some}}));
    TP_TRY(check_choice(tokens, experts, k));
    TP_TRY(check_dtype(dt));
    const int es = esize(dt);
    TP_TRY(check_elements({logits, dlogits}, es));
    TP_TRY(check_elements({ids, weights, dweights}, 4));
    const int64_t slots = tokens * k * 4;
    TP_TRY(check_alias({{dlogits, tokens * experts * es}}, {{logits, tokens * experts * es}, {ids, slots}, {weights, slots}, {dweights, slots}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    if (tokens == 0) return TPMLP_OK;
    return launch_moe_route_bwd(logits, static_cast<const int*>(ids), static_cast<const float*>(weights), static_cast<const float*>(dweights),
                                dlogits, tokens, static_cast<int>(experts), k, chosen != 0, dt == TPMLP_F32, static_cast<cudaStream_t>(stream));
}

tpmlp_status tpmlp_moe_matmul(const void* X, const void* row_token, const void* offsets, const void* W, const void* bias, void* Y, void* H,
                              int64_t tokens, int64_t rows, int64_t experts, int64_t K, int64_t N, tpmlp_act act, tpmlp_dtype out_dt,
                              void* stream) {
    const bool some = rows > 0, h_f32 = act == TPMLP_ACT_SWIGLU_H32, gated = act == TPMLP_ACT_SWIGLU || h_f32;
    const int hs = h_f32 ? 4 : 2;
    TP_TRY(need({{X, some}, {offsets, true}, {W, true}, {Y, some}}));
    TP_TRY(check_experts(tokens, rows, experts, K, N, row_token != nullptr));
    TP_TRY(check_act(act));
    if (!gated && H) {
        set_error("H is for the gated activation only");
        return TPMLP_ERR_SHAPE;
    }
    if (gated) TP_TRY(check_gate_width(N));
    TP_TRY(check_dtype(out_dt));
    if (gated && out_dt != TPMLP_BF16) {
        set_error("the gated activation is stored as bf16");
        return TPMLP_ERR_DTYPE;
    }
    TP_TRY(check_aligned({X, W, bias, Y, H}));
    TP_TRY(check_elements({row_token, offsets}, 4));
    TP_TRY(check_pitch(K, TPMLP_BF16, "K"));
    TP_TRY(check_pitch(N, TPMLP_BF16, "N"));
    TP_TRY(check_alias({{Y, rows * (gated ? N / 2 : N) * esize(out_dt)}, {H, rows * N * hs}},
                       {{X, tokens * K * 2}, {row_token, rows * 4}, {offsets, (experts + 1) * 4}, {W, experts * K * N * 2}, {bias, experts * N * 2}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    if (rows == 0) return TPMLP_OK;
    MoeSpec g{};
    g.rows = rows; g.tokens = tokens; g.K = K; g.N = N; g.experts = static_cast<int>(experts);
    g.offsets = static_cast<const int*>(offsets); g.src = static_cast<const int*>(row_token);
    g.x = X; g.w = W; g.bias = bias; g.out = Y; g.out_f32 = out_dt == TPMLP_F32; g.gated = gated; g.h = H; g.h_f32 = h_f32;
    return launch_moe_matmul(g, *dev, static_cast<cudaStream_t>(stream));
}

tpmlp_status tpmlp_moe_matmul_dx(const void* dY, const void* offsets, const void* W, const void* H, void* dX, int64_t rows, int64_t experts,
                                 int64_t K, int64_t N, tpmlp_act act, tpmlp_dtype dx_dt, void* stream) {
    const bool some = rows > 0, h_f32 = act == TPMLP_ACT_SWIGLU_H32, gated = act == TPMLP_ACT_SWIGLU || h_f32;
    const int hs = h_f32 ? 4 : 2;
    TP_TRY(need({{dY, some}, {offsets, true}, {W, true}, {H, some && gated}, {dX, some}}));
    TP_TRY(check_experts(rows, rows, experts, K, N, false));
    TP_TRY(check_act(act));
    if (!gated && H) {
        set_error("H is for the gated activation only");
        return TPMLP_ERR_SHAPE;
    }
    if (gated) {
        TP_TRY(check_matrix(rows, 2 * K, "H"));
        TP_TRY(check_gate_width(2 * K));
    }
    TP_TRY(check_dtype(dx_dt));
    if (gated && dx_dt != TPMLP_BF16) {
        set_error("the gated activation's gradient is stored as bf16");
        return TPMLP_ERR_DTYPE;
    }
    TP_TRY(check_aligned({dY, W, H, dX}));
    TP_TRY(check_elements({offsets}, 4));
    TP_TRY(check_pitch(K, TPMLP_BF16, "K"));
    TP_TRY(check_pitch(N, TPMLP_BF16, "N"));
    TP_TRY(check_alias({{dX, rows * (gated ? 2 * K : K) * esize(dx_dt)}},
                       {{dY, rows * N * 2}, {offsets, (experts + 1) * 4}, {W, experts * K * N * 2}, {H, gated ? rows * 2 * K * hs : 0}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    if (rows == 0) return TPMLP_OK;
    MoeSpec g{};
    g.rows = rows; g.tokens = rows; g.K = K; g.N = N; g.experts = static_cast<int>(experts);
    g.offsets = static_cast<const int*>(offsets);
    g.x = dY; g.w = W; g.out = dX; g.out_f32 = dx_dt == TPMLP_F32; g.gated = gated; g.h = const_cast<void*>(H); g.h_f32 = h_f32;
    return launch_moe_matmul_dx(g, *dev, static_cast<cudaStream_t>(stream));
}

tpmlp_status tpmlp_moe_matmul_dw(const void* X, const void* row_token, const void* offsets, const void* dY, void* dW, void* dbias,
                                 int64_t tokens, int64_t rows, int64_t experts, int64_t K, int64_t N, tpmlp_dtype grad_dt, void* stream) {
    const bool some = rows > 0;
    TP_TRY(need({{X, some}, {offsets, true}, {dY, some}, {dW, true}}));
    TP_TRY(check_experts(tokens, rows, experts, K, N, row_token != nullptr));
    TP_TRY(check_dtype(grad_dt));
    const int gs = esize(grad_dt);
    TP_TRY(check_aligned({X, dY, dW, dbias}));
    TP_TRY(check_elements({row_token, offsets}, 4));
    TP_TRY(check_pitch(K, TPMLP_BF16, "K"));
    TP_TRY(check_pitch(N, TPMLP_BF16, "N"));
    TP_TRY(check_alias({{dW, experts * K * N * gs}, {dbias, experts * N * gs}},
                       {{X, tokens * K * 2}, {row_token, rows * 4}, {offsets, (experts + 1) * 4}, {dY, rows * N * 2}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) {  // sums over nothing
        TP_TRY(clear_memory(dW, experts * K * N * gs, st));
        return dbias ? clear_memory(dbias, experts * N * gs, st) : TPMLP_OK;
    }
    MoeSpec g{};
    g.rows = rows; g.tokens = tokens; g.K = K; g.N = N; g.experts = static_cast<int>(experts);
    g.offsets = static_cast<const int*>(offsets); g.src = static_cast<const int*>(row_token);
    g.x = X; g.dy = dY; g.out = dW; g.out_f32 = grad_dt == TPMLP_F32; g.dbias = dbias;
    return launch_moe_matmul_dw(g, *dev, st);
}

tpmlp_status tpmlp_moe_combine(const void* O, const void* slot_row, const void* weights, void* Z, int64_t tokens, int64_t rows, int k,
                               int64_t h, void* stream) {
    const bool some = tokens > 0;
    TP_TRY(need({{O, some && rows > 0}, {slot_row, some}, {Z, some}}));
    TP_TRY(check_choice(tokens, kMaxExperts, k));
    TP_TRY(check_matrix(tokens, h, "Z"));
    TP_TRY(check_matrix(rows, h, "O"));
    TP_TRY(check_aligned({O, Z}));
    TP_TRY(check_elements({slot_row, weights}, 4));
    TP_TRY(check_pitch(h, TPMLP_BF16, "h"));
    TP_TRY(check_alias({{Z, tokens * h * 2}}, {{O, rows * h * 2}, {slot_row, tokens * k * 4}, {weights, tokens * k * 4}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    if (tokens == 0) return TPMLP_OK;
    return launch_moe_combine(O, static_cast<const int*>(slot_row), static_cast<const float*>(weights), Z, tokens, rows, k, h,
                              static_cast<cudaStream_t>(stream));
}

tpmlp_status tpmlp_moe_combine_bwd(const void* O, const void* slot_row, const void* weights, const void* dZ, void* dO, void* dweights,
                                   int64_t tokens, int64_t rows, int k, int64_t h, void* stream) {
    const bool some = tokens > 0, any = some && rows > 0;
    TP_TRY(need({{O, any && dweights}, {slot_row, some}, {dZ, some}, {dO, any}}));
    TP_TRY(check_choice(tokens, kMaxExperts, k));
    TP_TRY(check_matrix(tokens, h, "dZ"));
    TP_TRY(check_matrix(rows, h, "O"));
    TP_TRY(check_aligned({O, dZ, dO}));
    TP_TRY(check_elements({slot_row, weights, dweights}, 4));
    TP_TRY(check_pitch(h, TPMLP_BF16, "h"));
    TP_TRY(check_alias({{dO, rows * h * 2}, {dweights, tokens * k * 4}},
                       {{O, rows * h * 2}, {slot_row, tokens * k * 4}, {weights, tokens * k * 4}, {dZ, tokens * h * 2}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    if (tokens == 0) return TPMLP_OK;
    return launch_moe_combine_bwd(O, static_cast<const int*>(slot_row), static_cast<const float*>(weights), dZ, dO, static_cast<float*>(dweights),
                                  tokens, rows, k, h, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
