// C-ABI entry points of the MXFP4 operators: quantisation, the 4-bit product, and the gated block's
// forward and backward on 4-bit operands.
#include <cuda_runtime.h>

#include <cstring>

#include "api_common.h"
#include "internal.h"

namespace tpmlp {
namespace {

int64_t code_bytes(int64_t rows, int64_t k) { return rows * ((k + 31) / 32 * 16); }
int64_t scale_bytes(int64_t rows, int64_t k) { return (rows + 127) / 128 * ((k + 127) / 128) * 512; }

tpmlp_status check_matrix(int64_t rows, int64_t cols, const char* what) {
    if (rows < 0 || cols < 1 || rows > kMaxDim || cols > kMaxDim) {
        set_error("bad shape: %s is %lld x %lld", what, (long long)rows, (long long)cols);
        return TPMLP_ERR_SHAPE;
    }
    if (rows > 0 && cols > ((int64_t(1) << 40) / 4) / rows) {
        set_error("shape too large: %s (%lld x %lld) would exceed 2^40 bytes", what, (long long)rows, (long long)cols);
        return TPMLP_ERR_SHAPE;
    }
    return TPMLP_OK;
}

// Rows and columns of a product: the kernels' 32-bit indexes run up to a tile past them.
tpmlp_status check_product(int64_t m, int64_t n) {
    if (m > kMaxDim - 1024 || n > kMaxDim - 1024) {
        set_error("shape too large: %lld rows, %lld columns", (long long)m, (long long)n);
        return TPMLP_ERR_SHAPE;
    }
    return TPMLP_OK;
}

// An MXFP4 operand inside a workspace.
struct Packed {
    uint8_t* codes;
    uint8_t* scales;
    int64_t rows;
    MxOperand operand() const { return MxOperand{codes, scales, rows, false}; }
    MxOperand blocked() const { return MxOperand{codes, scales, rows, true}; }  // written by a GEMM's epilogue
};

// Carves a workspace into 256-byte aligned pieces; with a null base it only measures.
struct Carver {
    uint8_t* base;
    int64_t at = 0;
    uint8_t* take(int64_t bytes) {
        uint8_t* p = base ? base + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    }
    Packed packed(int64_t rows, int64_t k) {
        Packed o;
        o.rows = rows;
        o.codes = take(code_bytes(rows, k));
        o.scales = take(scale_bytes(rows, k));
        return o;
    }
};

struct FwdWs {
    Packed x, y;
    int64_t bytes;
    FwdWs(void* base, int64_t M, int64_t h, int64_t ffn) {
        Carver c{static_cast<uint8_t*>(base)};
        x = c.packed(M, h);
        y = c.packed(M, ffn);
        bytes = c.at;
    }
};
struct BwdWs {
    Packed dz, dzt, xt, dh, dht, yt;
    float *dh_sums, *dz_sums;  // column sums over blocks of 32 tokens
    int64_t bytes;
    BwdWs(void* base, int64_t M, int64_t h, int64_t ffn) {
        Carver c{static_cast<uint8_t*>(base)};
        dz = c.packed(M, h);
        dzt = c.packed(h, M);
        xt = c.packed(h, M);
        dh = c.packed(M, 2 * ffn);
        dht = c.packed(2 * ffn, M);
        yt = c.packed(ffn, M);
        dh_sums = reinterpret_cast<float*>(c.take((M + 31) / 32 * 2 * ffn * 4));
        dz_sums = reinterpret_cast<float*>(c.take((M + 31) / 32 * h * 4));
        bytes = c.at;
    }
};

MxSpec mx_spec(int64_t M, int64_t N, int64_t K, int epi) {
    MxSpec g;
    std::memset(&g, 0, sizeof(g));
    g.M = M;
    g.N = N;
    g.K = K;
    g.epi = epi;
    return g;
}

// D = A B^T (+ bias): a plain product, its columns in shards of shard_cols (0: not sharded).
MxProduct product(const MxOperand& a, const MxOperand& b, const void* bias, void* D, int64_t K, bool f32, int64_t shard_cols) {
    MxProduct c{a, b, mx_spec(a.rows, b.rows, K, EPI_STORE)};
    c.g.out = D;
    c.g.out_f32 = f32;
    c.g.shard_cols = shard_cols;
    c.g.out_ld = shard_cols > 0 ? shard_cols : b.rows;
    c.g.out_ss = shard_cols > 0 ? a.rows * shard_cols : 0;
    c.g.bias = bias;
    return c;
}
tpmlp_status run(const MxProduct& c, const DeviceInfo& dev, cudaStream_t st) { return launch_mxfp4_gemm(c.a, c.b, c.g, dev, st); }

tpmlp_status check_gated(int64_t s, int64_t b, int64_t h, int64_t ffn, int p) {
    TP_TRY(check_mlp_shape(s, b, h, ffn, p, true));
    // (blocked operands count a row as two 8-byte words, in 32 bits)
    if (ffn > (int64_t(1) << 28) || s * b > (int64_t(1) << 29)) {
        set_error("shape too large: the gated block takes at most 2^29 tokens and 2^28 features");
        return TPMLP_ERR_SHAPE;
    }
    TP_TRY(check_product(h, h));
    if ((ffn / p) % 128 != 0) {
        set_error("the gated block needs ffn/p to be a multiple of 128 (ffn=%lld, p=%d)", (long long)ffn, p);
        return TPMLP_ERR_DIVISIBILITY;
    }
    return TPMLP_OK;
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;

extern "C" {

int64_t tpmlp_mxfp4_code_bytes(int64_t rows, int64_t k) {
    return check_matrix(rows, k, "the operand") == TPMLP_OK ? code_bytes(rows, k) : -1;
}
int64_t tpmlp_mxfp4_scale_bytes(int64_t rows, int64_t k) {
    return check_matrix(rows, k, "the operand") == TPMLP_OK ? scale_bytes(rows, k) : -1;
}
int64_t tpmlp_mxfp4_swiglu_ws_bytes(int64_t s, int64_t b, int64_t h, int64_t ffn, int p, int backward) {
    if (check_gated(s, b, h, ffn, p) != TPMLP_OK) return -1;
    return backward ? BwdWs(nullptr, s * b, h, ffn).bytes : FwdWs(nullptr, s * b, h, ffn).bytes;
}

tpmlp_status tpmlp_mxfp4_quantize(const void* X, void* Q, void* S, void* Qt, void* St, int64_t rows, int64_t cols, int64_t ldx,
                                  int p, tpmlp_dtype dt, void* stream) {
    if (!X || (!Q && !Qt) || (!Q != !S) || (!Qt != !St)) {
        set_error("X and at least one of (Q, S) and (Qt, St) are needed, each pair whole");
        return TPMLP_ERR_NULL;
    }
    TP_TRY(check_matrix(rows, cols, "X"));
    if (p < 1 || ldx < 1 || ldx > kMaxDim) {
        set_error("bad shape: ldx=%lld p=%d", (long long)ldx, p);
        return TPMLP_ERR_SHAPE;
    }
    if (cols % p != 0 || (p > 1 && (cols / p) % 32 != 0)) {
        set_error("cols=%lld must be divisible by p=%d, and column shards be multiples of 32 wide", (long long)cols, p);
        return TPMLP_ERR_DIVISIBILITY;
    }
    if (ldx < cols / p) {
        set_error("row pitch ldx=%lld is less than the %lld columns of a row", (long long)ldx, (long long)(cols / p));
        return TPMLP_ERR_SHAPE;
    }
    if (rows > 0 && ldx > ((int64_t(1) << 40) / 4) / rows / p) {
        set_error("shape too large: X would exceed 2^40 bytes");
        return TPMLP_ERR_SHAPE;
    }
    TP_TRY(check_dtype(dt));
    TP_TRY(check_aligned({X, Q, S, Qt, St}));
    TP_TRY(check_pitch(ldx, dt, "ldx"));
    const int64_t x_bytes = rows == 0 ? 0 : ((p * rows - 1) * ldx + cols / p) * esize(dt);
    TP_TRY(check_alias({{Q, code_bytes(rows, cols)}, {S, scale_bytes(rows, cols)}, {Qt, code_bytes(cols, rows)},
                        {St, scale_bytes(cols, rows)}},
                       {{X, x_bytes}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    if (rows == 0) return TPMLP_OK;
    return launch_mxfp4_quantize(X, ldx, Q, S, Qt, St, rows, cols, p, dt == TPMLP_F32, static_cast<cudaStream_t>(stream));
}

tpmlp_status tpmlp_mxfp4_dequantize(const void* Q, const void* S, void* out, int64_t rows, int64_t k, tpmlp_dtype dt, void* stream) {
    if (!Q || !S || !out) {
        set_error("pointers must not be NULL");
        return TPMLP_ERR_NULL;
    }
    TP_TRY(check_matrix(rows, k, "the operand"));
    TP_TRY(check_dtype(dt));
    TP_TRY(check_aligned({Q, S, out}));
    TP_TRY(check_alias({{out, rows * k * esize(dt)}}, {{Q, code_bytes(rows, k)}, {S, scale_bytes(rows, k)}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    if (rows == 0) return TPMLP_OK;
    return launch_mxfp4_dequantize(Q, S, out, rows, k, dt == TPMLP_F32, *dev, static_cast<cudaStream_t>(stream));
}

tpmlp_status tpmlp_mxfp4_matmul(const void* Aq, const void* As, const void* Bq, const void* Bs, const void* bias, void* D, int64_t m,
                                int64_t n, int64_t k, tpmlp_dtype out_dt, void* stream) {
    if (!Aq || !As || !Bq || !Bs || !D) {
        set_error("only bias may be NULL");
        return TPMLP_ERR_NULL;
    }
    TP_TRY(check_matrix(m, k, "A"));
    TP_TRY(check_matrix(n, k, "B"));
    TP_TRY(check_matrix(m, n, "D"));
    TP_TRY(check_product(m, n));
    TP_TRY(check_dtype(out_dt));
    TP_TRY(check_aligned({Aq, As, Bq, Bs, bias, D}));
    TP_TRY(check_pitch(n, out_dt, "n"));
    TP_TRY(check_alias({{D, m * n * esize(out_dt)}},
                       {{Aq, code_bytes(m, k)}, {As, scale_bytes(m, k)}, {Bq, code_bytes(n, k)}, {Bs, scale_bytes(n, k)}, {bias, n * 2}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    if (m == 0) return TPMLP_OK;
    return run(product({Aq, As, m}, {Bq, Bs, n}, bias, D, k, out_dt == TPMLP_F32, 0), *dev, static_cast<cudaStream_t>(stream));
}

tpmlp_status tpmlp_mxfp4_swiglu_mlp_fwd(const void* X, const void* Wq, const void* Ws, const void* bw_sh, const void* Bq, const void* Bs,
                                        const void* b2, void* Z, void* H, void* ws, int64_t s, int64_t b, int64_t h, int64_t ffn, int p,
                                        tpmlp_dtype z_dt, void* stream) {
    if (!X || !Wq || !Ws || !Bq || !Bs || !Z || !ws) {
        set_error("only bw_sh, b2 and H may be NULL");
        return TPMLP_ERR_NULL;
    }
    TP_TRY(check_gated(s, b, h, ffn, p));
    TP_TRY(check_dtype(z_dt));
    const int64_t M = s * b;
    TP_TRY(check_aligned({X, Wq, Ws, bw_sh, Bq, Bs, b2, Z, H, ws}));
    TP_TRY(check_pitch(h, TPMLP_BF16, "h"));
    const FwdWs w(ws, M, h, ffn);
    TP_TRY(check_alias({{Z, M * h * esize(z_dt)}, {H, 2 * M * ffn * 2}, {ws, w.bytes}},
                       {{X, M * h * 2}, {Wq, code_bytes(2 * ffn, h)}, {Ws, scale_bytes(2 * ffn, h)}, {bw_sh, 2 * ffn * 2},
                        {Bq, code_bytes(h, ffn)}, {Bs, scale_bytes(h, ffn)}, {b2, h * 2}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    if (M == 0) return TPMLP_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    TP_TRY(launch_mxfp4_quantize(X, h, w.x.codes, w.x.scales, nullptr, nullptr, M, h, 1, false, st));
    MxSpec g = mx_spec(M, 2 * ffn, h, EPI_SWIGLU);
    g.bias = bw_sh;
    g.h_out = H;
    g.h_ld = 2 * ffn;
    g.q = w.y.codes;
    g.qs = w.y.scales;
    g.q_cols = ffn;
    g.prefetch_b = true;
    TP_TRY(launch_mxfp4_gemm(w.x.operand(), {Wq, Ws, 2 * ffn}, g, *dev, st));
    MxProduct row = product(w.y.blocked(), {Bq, Bs, h}, b2, Z, ffn, z_dt == TPMLP_F32, 0);
    row.g.prefetch_b = true;
    return run(row, *dev, st);
}

tpmlp_status tpmlp_mxfp4_swiglu_mlp_bwd(const void* X, const void* Wq, const void* Ws, const void* Bq, const void* Bs, const void* H,
                                        const void* dZ, void* dX, void* dW_sh, void* dB_sh, void* dbw_sh, void* db2, void* ws, int64_t s,
                                        int64_t b, int64_t h, int64_t ffn, int p, tpmlp_dtype dx_dt, tpmlp_dtype grad_dt, void* stream) {
    if (!X || !Wq || !Ws || !Bq || !Bs || !H || !dZ || !dX || !dW_sh || !dB_sh || !ws) {
        set_error("only dbw_sh and db2 may be NULL");
        return TPMLP_ERR_NULL;
    }
    TP_TRY(check_gated(s, b, h, ffn, p));
    TP_TRY(check_dtype(dx_dt));
    TP_TRY(check_dtype(grad_dt));
    const int64_t M = s * b, gs = esize(grad_dt);
    TP_TRY(check_aligned({X, Wq, Ws, Bq, Bs, H, dZ, dX, dW_sh, dB_sh, dbw_sh, db2, ws}));
    TP_TRY(check_pitch(h, TPMLP_BF16, "h"));
    const BwdWs w(ws, M, h, ffn);
    TP_TRY(check_alias({{dX, M * h * esize(dx_dt)}, {dW_sh, 2 * h * ffn * gs}, {dB_sh, ffn * h * gs}, {dbw_sh, 2 * ffn * gs},
                        {db2, h * gs}, {ws, w.bytes}},
                       {{X, M * h * 2}, {Wq, code_bytes(h, 2 * ffn)}, {Ws, scale_bytes(h, 2 * ffn)}, {Bq, code_bytes(ffn, h)},
                        {Bs, scale_bytes(ffn, h)}, {H, 2 * M * ffn * 2}, {dZ, M * h * 2}}));
    const DeviceInfo* dev;
    TP_TRY(get_device(&dev));
    if (M == 0) return TPMLP_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool gf32 = grad_dt == TPMLP_F32;
    TP_TRY(launch_mxfp4_quantize_bwd(dZ, w.dz.codes, w.dz.scales, w.dzt.codes, w.dzt.scales, db2 ? w.dz_sums : nullptr, X, w.xt.codes,
                                     w.xt.scales, M, h, st));
    // dY = dZ B^T; its epilogue leaves dH = [dg | du] quantised along both axes and Y along the tokens
    MxSpec g = mx_spec(M, ffn, h, EPI_DSWIGLU);
    g.h_in = H;
    g.h_ld = 2 * ffn;
    g.q = w.dh.codes;
    g.qs = w.dh.scales;
    g.q_cols = 2 * ffn;
    g.ht = w.dht.codes;
    g.hts = w.dht.scales;
    g.yt = w.yt.codes;
    g.yts = w.yt.scales;
    g.colsum = dbw_sh ? w.dh_sums : nullptr;
    TP_TRY(launch_mxfp4_gemm(w.dz.operand(), {Bq, Bs, ffn}, g, *dev, st));
    const MxProduct dB = product(w.yt.blocked(), w.dzt.operand(), nullptr, dB_sh, M, gf32, 0);
    const MxProduct dW = product(w.xt.operand(), w.dht.blocked(), nullptr, dW_sh, M, gf32, p > 1 ? 2 * ffn / p : 0);
    const MxProduct dx = product(w.dh.blocked(), {Wq, Ws, h}, nullptr, dX, 2 * ffn, dx_dt == TPMLP_F32, 0);
    const MxSums sums{{w.dh_sums, w.dz_sums}, {dbw_sh, db2}, {2 * ffn, h}, (M + 31) / 32, gf32};
    return launch_mxfp4_gemms({dB, dW, dx}, sums, *dev, st);
}

tpmlp_status tpmlp_set_mxfp4_mode(int mode) {
    if (mode < 0 || mode > 5) {
        set_error("MXFP4 GEMM mode must be 0 (automatic), 1 (single CTAs), 2 (CTA pairs) or 3, 4, 5 (single CTAs, K split 2, 4, 8 ways)");
        return TPMLP_ERR_SHAPE;
    }
    set_mxfp4_mode(mode);
    return TPMLP_OK;
}
int tpmlp_get_mxfp4_mode(void) { return get_mxfp4_mode(); }

}  // extern "C"
