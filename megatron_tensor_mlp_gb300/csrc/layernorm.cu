// Layer norm over rows, forward and backward.
//
//   y = (x - mean) rstd gamma + beta,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),  g = dy gamma,  xhat = (x - mean) rstd
//   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy
//
// A row is read once and lies in registers: a thread holds NV pieces of VEC elements.  Means are of the values, variances
// of the differences from the mean, both in 32 bits.  The backward's CTAs walk over rows with the same columns on the
// same threads, so the sums of dgamma and dbeta stay in registers until a CTA's last row; the CTAs' sums go to the
// workspace and a second kernel adds them in a fixed order (no atomics: the same bits every time).
//
// Rows whose start is not aligned to 16 bytes (an odd width, pitch or base) are read element by element (VEC 1).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace tpmlp {
namespace {

constexpr int MOST_PARTS = 304;  // CTAs of the backward, two an SM
constexpr int WARP_ROW = 1024;   // elements of a row that one warp takes
// Threads of a CTA at most, by the elements that each holds.
constexpr int most_threads(int elements) { return elements <= 8 ? 1024 : 512; }

template <typename T, int VEC>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 8> {
    using type = uint4;
};
template <>
struct Raw<float, 4> {
    using type = uint4;
};
template <>
struct Raw<__nv_bfloat16, 1> {
    using type = uint16_t;
};
template <>
struct Raw<float, 1> {
    using type = float;
};

template <typename T, int VEC>
__device__ __forceinline__ void widen(const typename Raw<T, VEC>::type& r, float (&f)[VEC]) {
    if constexpr (VEC == 8) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else if constexpr (VEC == 4) {
        f[0] = __uint_as_float(r.x);
        f[1] = __uint_as_float(r.y);
        f[2] = __uint_as_float(r.z);
        f[3] = __uint_as_float(r.w);
    } else if constexpr (sizeof(T) == 2) {
        f[0] = __uint_as_float(static_cast<uint32_t>(r) << 16);
    } else {
        f[0] = r;
    }
}
template <typename T, int VEC>
__device__ __forceinline__ typename Raw<T, VEC>::type narrow(const float (&f)[VEC]) {
    if constexpr (VEC == 8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (VEC == 4) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else if constexpr (sizeof(T) == 2) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
        return f[0];
    }
}

// Sums of N values over a row's threads, the same in each of them: a warp, or the whole CTA (buf: two sets of 32 x N
// floats used in turn, so that one barrier a row is enough).
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* buf, int& turn) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
    if (blockDim.x == 32) return;  // (rows on warps: blockDim is 32 x rows)
    float* b = buf + turn * 32 * N;
    turn ^= 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) b[warp * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = lane < warps ? b[lane * N + i] : 0.0f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
    }
}

struct FwdArgs {
    const void *x, *gamma, *beta;
    void* y;
    float *mean, *rstd;
    long long rows, ldx, ldy;
    int h, vecs;
    float eps;
};

// Row: blockDim.x threads; blockDim.y rows a CTA (more than one only with 32 threads a row).
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(most_threads(VEC * NV)) fwd_kernel(const FwdArgs p) {
    using R = typename Raw<T, VEC>::type;
    __shared__ float buf[2 * 32];
    int turn = 0;
    griddep_wait();
    if (threadIdx.x == 0 && threadIdx.y == 0) griddep_launch_dependents();
    const float inv = 1.0f / static_cast<float>(p.h);
    for (long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y; row < p.rows;
         row += static_cast<long long>(gridDim.x) * blockDim.y) {
        const R* x = reinterpret_cast<const R*>(static_cast<const T*>(p.x) + row * p.ldx);
        float v[NV][VEC], s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c < p.vecs) {
                widen<T, VEC>(x[c], v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[i][j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[0] += v[i][j];
        }
        row_sum<1>(s, buf, turn);
        const float mean = s[0] * inv;
        s[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x) < p.vecs)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float d = v[i][j] - mean;
                    s[0] = fmaf(d, d, s[0]);
                }
        row_sum<1>(s, buf, turn);
        const float rstd = rsqrtf(s[0] * inv + p.eps);
        if (threadIdx.x == 0 && p.mean != nullptr) {
            p.mean[row] = mean;
            p.rstd[row] = rstd;
        }
        R* y = reinterpret_cast<R*>(static_cast<T*>(p.y) + row * p.ldy);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c >= p.vecs) continue;
            float g[VEC], b[VEC], o[VEC];
            if (p.gamma != nullptr) widen<T, VEC>(static_cast<const R*>(p.gamma)[c], g);
            if (p.beta != nullptr) widen<T, VEC>(static_cast<const R*>(p.beta)[c], b);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float n = (v[i][j] - mean) * rstd;
                o[j] = fmaf(n, p.gamma != nullptr ? g[j] : 1.0f, p.beta != nullptr ? b[j] : 0.0f);
            }
            y[c] = narrow<T, VEC>(o);
        }
    }
}

struct BwdArgs {
    const void *x, *gamma, *dy;
    const float *mean, *rstd;
    void* dx;
    float* part;  // [CTAs][2][h], null: no dgamma, dbeta
    long long rows, ldx, lddy, lddx;
    int h, vecs;
};

// x and dy stay in registers as they were read; xhat is computed from them twice, which costs less than holding it.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(most_threads(VEC * NV)) bwd_kernel(const BwdArgs p) {
    using R = typename Raw<T, VEC>::type;
    __shared__ float buf[2 * 32 * 2];
    __shared__ float acc[WARP_ROW];  // rows on warps: their sums, added warp by warp
    int turn = 0;
    griddep_wait();
    if (threadIdx.x == 0 && threadIdx.y == 0) griddep_launch_dependents();
    const float inv = 1.0f / static_cast<float>(p.h);
    const int tx = threadIdx.x, nx = blockDim.x;
    float dgamma[NV][VEC], dbeta[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) dgamma[i][j] = dbeta[i][j] = 0.0f;
    for (long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y; row < p.rows;
         row += static_cast<long long>(gridDim.x) * blockDim.y) {
        const R* x = reinterpret_cast<const R*>(static_cast<const T*>(p.x) + row * p.ldx);
        const R* dy = reinterpret_cast<const R*>(static_cast<const T*>(p.dy) + row * p.lddy);
        const float mean = p.mean[row], rstd = p.rstd[row];
        R xr[NV], dr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * nx + tx;
            if (c < p.vecs) {
                xr[i] = x[c];
                dr[i] = dy[c];
            } else {
                xr[i] = dr[i] = R{};
            }
        }
        float s[2] = {0.0f, 0.0f};
        // calls f(piece, xhat, dy, dy gamma)
        auto each = [&](auto&& f) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = i * nx + tx;
                if (c >= p.vecs) continue;
                float n[VEC], d[VEC], g[VEC];
                widen<T, VEC>(xr[i], n);
                widen<T, VEC>(dr[i], d);
                if (p.gamma != nullptr) widen<T, VEC>(static_cast<const R*>(p.gamma)[c], g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    n[j] = (n[j] - mean) * rstd;
                    g[j] = p.gamma != nullptr ? d[j] * g[j] : d[j];
                }
                f(i, c, n, d, g);
            }
        };
        each([&](int i, int, const float(&n)[VEC], const float(&d)[VEC], const float(&g)[VEC]) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                dgamma[i][j] = fmaf(d[j], n[j], dgamma[i][j]);
                dbeta[i][j] += d[j];
                s[0] += g[j];
                s[1] = fmaf(g[j], n[j], s[1]);
            }
        });
        row_sum<2>(s, buf, turn);
        const float a = s[0] * inv, b = s[1] * inv;
        R* dx = reinterpret_cast<R*>(static_cast<T*>(p.dx) + row * p.lddx);
        each([&](int, int c, const float(&n)[VEC], const float(&)[VEC], const float(&g)[VEC]) {
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] = rstd * (g[j] - a - n[j] * b);
            dx[c] = narrow<T, VEC>(o);
        });
    }
    if (p.part == nullptr) return;
    float* out = p.part + static_cast<long long>(blockIdx.x) * 2 * p.h;
    if (blockDim.y == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * nx + tx;
            if (c >= p.vecs) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                out[c * VEC + j] = dgamma[i][j];
                out[p.h + c * VEC + j] = dbeta[i][j];
            }
        }
    } else if constexpr (32 * NV * VEC <= WARP_ROW) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            for (int w = 0; w < static_cast<int>(blockDim.y); ++w) {
                __syncthreads();
                if (static_cast<int>(threadIdx.y) != w) continue;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = i * nx + tx;
                    if (c >= p.vecs) continue;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float v = which ? dbeta[i][j] : dgamma[i][j];
                        acc[c * VEC + j] = w == 0 ? v : acc[c * VEC + j] + v;
                        if (w == static_cast<int>(blockDim.y) - 1) out[which * p.h + c * VEC + j] = acc[c * VEC + j];
                    }
                }
            }
        }
    }
}

// Sums of the parts' columns: 32 columns a CTA, part i on thread row i % 8, the eight sums added in order.
__global__ void __launch_bounds__(256) parts_kernel(const float* part, int parts, int h, void* dgamma, void* dbeta, int f32) {
    __shared__ float sum[8][33];
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5, which = blockIdx.y;
    void* out = which ? dbeta : dgamma;
    if (out == nullptr) return;
    float s = 0.0f;
    if (col < h)
#pragma unroll 8
        for (int i = r; i < parts; i += 8) s += part[(static_cast<long long>(i) * 2 + which) * h + col];
    sum[r][threadIdx.x & 31] = s;
    __syncthreads();
    if (r == 0 && col < h) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sum[i][threadIdx.x];
        if (f32) static_cast<float*>(out)[col] = s;
        else static_cast<__nv_bfloat16*>(out)[col] = __float2bfloat16_rn(s);
    }
}

template <typename... P, typename... A>
tpmlp_status launch(void (*kern)(P...), dim3 grid, dim3 block, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see griddep_wait
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("layer norm launch: %s", cudaGetErrorString(e));
        return TPMLP_ERR_CUDA;
    }
    count_launch();
    return TPMLP_OK;
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct Shape {
    int nv, x, y;  // pieces a thread, threads a row, rows a CTA
};
// A row of `vecs` pieces: on a warp where its registers hold it, else on a CTA.
Shape shape_of(int vec, int vecs) {
    const int row = vec == 1 ? 4 : 16 / vec;  // pieces of a thread: 4 single elements or 16 elements, 32 for wide rows
    if (vecs <= 32) return {1, 32, 8};
    if (vec > 1 && vecs <= 32 * (32 / vec)) return {32 / vec, 32, 8};
    if (vecs <= most_threads(vec * row) * row) return {row, (vecs + 32 * row - 1) / (32 * row) * 32, 1};
    return {32 / vec, (vecs + 1024 / vec - 1) / (1024 / vec) * 32, 1};
}

template <typename F>
tpmlp_status by_shape(bool f32, bool wide, int nv, F&& f) {
    auto pick = [&](auto t, auto vec) {
        using T = decltype(t);
        constexpr int V = decltype(vec)::value, ROW = V == 1 ? 4 : 16 / V;
        if (nv == 1) return f(t, vec, std::integral_constant<int, 1>{});
        if (nv == ROW) return f(t, vec, std::integral_constant<int, ROW>{});
        return f(t, vec, std::integral_constant<int, 32 / V>{});
    };
    if (f32) return wide ? pick(float{}, std::integral_constant<int, 4>{}) : pick(float{}, std::integral_constant<int, 1>{});
    return wide ? pick(__nv_bfloat16{}, std::integral_constant<int, 8>{}) : pick(__nv_bfloat16{}, std::integral_constant<int, 1>{});
}

// Whether rows of these tensors can be read 16 bytes at a time.
bool wide_rows(int64_t h, int es, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> pitches) {
    bool ok = h * es % 16 == 0;
    for (const void* p : ptrs) ok = ok && aligned(p);
    for (int64_t l : pitches) ok = ok && l * es % 16 == 0;
    return ok;
}

}  // namespace

int64_t layernorm_ws_bytes(int64_t rows, int64_t h) { return std::min<int64_t>(rows, MOST_PARTS) * 2 * h * 4; }

tpmlp_status launch_layernorm_fwd(const void* X, const void* gamma, const void* beta, void* Y, float* mean, float* rstd, int64_t rows,
                                  int64_t h, int64_t ldx, int64_t ldy, float eps, bool f32, const DeviceInfo& dev, cudaStream_t st) {
    const int es = f32 ? 4 : 2;
    const bool wide = wide_rows(h, es, {X, gamma, beta, Y}, {ldx, ldy});
    const int vec = wide ? 16 / es : 1;
    const FwdArgs a{X, gamma, beta, Y, mean, rstd, rows, ldx, ldy, static_cast<int>(h), static_cast<int>(h / vec), eps};
    const Shape s = shape_of(vec, a.vecs);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((rows + s.y - 1) / s.y, int64_t(dev.sm_count) * 64));
    return by_shape(f32, wide, s.nv, [&](auto t, auto v, auto nv) {
        return launch(fwd_kernel<decltype(t), decltype(v)::value, decltype(nv)::value>, dim3(grid), dim3(s.x, s.y), st, a);
    });
}

tpmlp_status launch_layernorm_bwd(const void* X, const void* gamma, const float* mean, const float* rstd, const void* dY, void* dX,
                                  void* dgamma, void* dbeta, void* ws, int64_t rows, int64_t h, int64_t ldx, int64_t lddy, int64_t lddx,
                                  bool f32, bool grad_f32, const DeviceInfo& dev, cudaStream_t st) {
    const int es = f32 ? 4 : 2;
    const bool wide = wide_rows(h, es, {X, gamma, dY, dX}, {ldx, lddy, lddx}), sums = dgamma != nullptr || dbeta != nullptr;
    const int vec = wide ? 16 / es : 1;
    const BwdArgs a{X, gamma, dY, mean, rstd, dX, sums ? static_cast<float*>(ws) : nullptr, rows, ldx, lddy, lddx, static_cast<int>(h),
                    static_cast<int>(h / vec)};
    const Shape s = shape_of(vec, a.vecs);
    const int grid = static_cast<int>(std::min<int64_t>({(rows + s.y - 1) / s.y, 2 * int64_t(dev.sm_count), MOST_PARTS}));
    const tpmlp_status r = by_shape(f32, wide, s.nv, [&](auto t, auto v, auto nv) {
        return launch(bwd_kernel<decltype(t), decltype(v)::value, decltype(nv)::value>, dim3(grid), dim3(s.x, s.y), st, a);
    });
    if (r != TPMLP_OK || !sums) return r;
    return launch(parts_kernel, dim3(static_cast<unsigned>((h + 31) / 32), 2), dim3(256), st, static_cast<const float*>(ws), grid,
                  static_cast<int>(h), dgamma, dbeta, grad_f32 ? 1 : 0);
}

}  // namespace tpmlp
