// Layer norm over rows, forward and backward.
//
//   y = (x - mean) rstd gamma + beta,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),  g = dy gamma,  xhat = (x - mean) rstd
//   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy
//
// A row is read once and lies in registers: a thread holds NV pieces of VEC elements.  Sums are in 32 bits.  The mean of the
// values, m0, is off by a few 2^-24 of their size, which rstd magnifies by up to 1 / sqrt(eps) where the values are large against
// their spread; so the differences from it, d = x - m0, are summed along with their squares: m0 + mean(d) is the mean,
// d - mean(d) the difference that is normalised, mean(d^2) - mean(d)^2 the variance (mean(d) is small against m0: nothing
// cancels).  A constant row's d are multiples of one step, their sum exact, the differences zero and y beta, to the bit.
// (Forward of 8192 x 5120 bf16: 31.1 us, with the mean left as it is 28.6; 8192 x 4096 24.6, 23.4; x 1000 12.0, 11.8.)
//
// The backward's CTAs walk over rows with the same columns on the same threads, so the sums of dgamma and dbeta stay in
// registers until a CTA's last row; the CTAs' sums go to the workspace and a second kernel adds them in a fixed order (no
// atomics: the same bits every time).
//
// Rows whose start is not aligned to 16 bytes (an odd width, pitch or base) are read element by element (VEC 1).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "gemm_tc.cuh"
#include "internal.h"
#include "per_device.h"
#include "ptx.cuh"

namespace tpmlp {
namespace {

// CTAs of the backward at most, whatever the device (the workspace is sized without one): two an SM of a GB300's 152, four where
// rows take few threads.
constexpr int most_parts(long long h) { return h <= 4096 ? 608 : 304; }
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

// Sums of N values over a warp: of one in every lane, of two in half the shuffles, the first's in lanes 0-15 and the second's
// in 16-31 (as v[0]).
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
    static_assert(N == 1 || N == 2);
    if constexpr (N == 2) {
        const bool second = (threadIdx.x & 16) != 0;
        const float mine = second ? v[1] : v[0], other = second ? v[0] : v[1];
        v[0] = mine + __shfl_xor_sync(0xFFFFFFFFu, other, 16);
    }
#pragma unroll
    for (int d = N == 2 ? 8 : 16; d > 0; d >>= 1) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], d);
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

// From the sums of the differences d from m0 and of their squares: the mean of d, by which m0 is off (divided by h, not
// multiplied by a rounded 1 / h: that of a constant row comes out exact), and rstd.  A variance below zero is a rounding; a NaN
// stays one, and squares past the range stay infinite (fma: not infinity less infinity).
__device__ __forceinline__ void spread(float sum, float squares, int h, float inv, float eps, float& off, float& rstd, bool& far) {
    off = sum / static_cast<float>(h);
    float var = fmaf(-sum, off, squares) * inv;
    var = var < 0.0f ? 0.0f : var;
    rstd = rsqrtf(var + eps);
    far = off * off > 0x1p-48f * var;  // m0 is off by more than a rounding of differences of the spread's size
}
// The mean: m0 itself where it is infinite.
__device__ __forceinline__ float corrected(float m0, float off) { return isinf(m0) ? m0 : m0 + off; }

struct FwdArgs {
    const void *x, *gamma, *beta;
    void* y;
    float *mean, *rstd;
    long long rows, ldx, ldy;
    int h, vecs;
    float eps;
};

// Threads of a row.  Where a thread has many pieces each loop over them takes it anew, as far as the compiler can see: it would
// hold the places of all pieces over the whole walk, and spill them (2000 fp32 rows of 8191 elements: 202 us, so 44).
template <int NV>
__device__ __forceinline__ int width() {
    int nx = blockDim.x;
    if constexpr (NV > 8) asm volatile("" : "+r"(nx));
    return nx;
}

// Row: blockDim.x threads; blockDim.y rows a CTA (more than one only with 32 threads a row).  Two CTAs an SM where a thread has
// many pieces (2000 bf16 rows of 8191: 50 us, 58 with one, whose threads have 94 registers).
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(most_threads(VEC * NV), NV > 8 ? 2 : 0) fwd_kernel(const FwdArgs p) {
    using R = typename Raw<T, VEC>::type;
    __shared__ float buf[2 * 32 * 2];  // (one value in turn 0, two in turn 1)
    int turn = 0;
    griddep_wait();
    if (threadIdx.x == 0 && threadIdx.y == 0) griddep_launch_dependents();
    const int tx = threadIdx.x;
    const float inv = 1.0f / static_cast<float>(p.h);
    for (long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y; row < p.rows;
         row += static_cast<long long>(gridDim.x) * blockDim.y) {
        const R* x = reinterpret_cast<const R*>(static_cast<const T*>(p.x) + row * p.ldx);
        float v[NV][VEC], s[1] = {0.0f};
        int nx = width<NV>();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * nx + tx;
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
        const float m0 = s[0] * inv;
        float d[2] = {0.0f, 0.0f};
        nx = width<NV>();
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i * nx + tx < p.vecs)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    v[i][j] -= m0;
                    d[0] += v[i][j];
                    d[1] = fmaf(v[i][j], v[i][j], d[1]);
                }
        row_sum<2>(d, buf, turn);
        float off, rstd;
        bool far;
        spread(d[0], d[1], p.h, inv, p.eps, off, rstd, far);
        if (threadIdx.x == 0 && p.mean != nullptr) {
            p.mean[row] = corrected(m0, off);
            p.rstd[row] = rstd;
        }
        if (far) {  // (the same in all of a row's threads; most rows' are not)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[i][j] -= off;
        }
        R* y = reinterpret_cast<R*>(static_cast<T*>(p.y) + row * p.ldy);
        nx = width<NV>();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * nx + tx;
            if (c >= p.vecs) continue;
            float g[VEC], b[VEC], o[VEC];
            if (p.gamma != nullptr) widen<T, VEC>(static_cast<const R*>(p.gamma)[c], g);
            if (p.beta != nullptr) widen<T, VEC>(static_cast<const R*>(p.beta)[c], b);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float n = v[i][j] * rstd;
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

// (16 bytes at a time: element by element, a lane's 32 bytes from the next one's, 4 rows of 5120 took 9.4 us, so 5.8.)
template <int VEC>
__device__ __forceinline__ void put(float* to, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        *to = v[0];
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) *reinterpret_cast<float4*>(to + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
}

// x and dy stay in registers as they were read; xhat is computed from them twice, which costs less than holding it.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(most_threads(VEC * NV)) bwd_kernel(const BwdArgs p) {
    using R = typename Raw<T, VEC>::type;
    __shared__ float buf[2 * 32 * 2];
    extern __shared__ __align__(16) float warps_sums[];
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
            put<VEC>(out + c * VEC, dgamma[i]);
            put<VEC>(out + p.h + c * VEC, dbeta[i]);
        }
    } else {
        // rows on warps: [warp][2][h], then the warps' sums in order
        float* mine = warps_sums + static_cast<size_t>(threadIdx.y) * 2 * p.h;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * nx + tx;
            if (c >= p.vecs) continue;
            put<VEC>(mine + c * VEC, dgamma[i]);
            put<VEC>(mine + p.h + c * VEC, dbeta[i]);
        }
        __syncthreads();
        for (int c = threadIdx.y * nx + tx; c < 2 * p.h; c += nx * static_cast<int>(blockDim.y)) {
            float v = 0.0f;
            for (int w = 0; w < static_cast<int>(blockDim.y); ++w) v += warps_sums[static_cast<size_t>(w) * 2 * p.h + c];
            out[c] = v;
        }
    }
}

// ---------------------------------------------------------------- many wide rows
// The same for rows on a CTA that are aligned to 16 bytes, where there are more rows than CTAs: a CTA's next rows come by bulk
// copies into a ring of shared memory while it works on one, since what its threads can hold in registers does not keep the
// memory busy.  Sums in pairs of fp32 (add, mul and fma of two values an instruction: the arithmetic alone would take 23 us of
// the backward's 40 at 8192 x 5120 otherwise).
struct Ring {
    uint8_t* at;        // slots of `bytes`
    uint64_t* full;
    uint32_t bytes;
    int slots, slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void init(uint64_t* bars) {
        full = bars;
        if (threadIdx.x == 0) {
            for (int i = 0; i < slots; ++i) mbar_init(full + i, 1);
            fence_mbarrier_init();
            fence_proxy_async_smem();
        }
        __syncthreads();
    }
    // A row that never comes is recorded in the status word; the walk goes on without waiting, so that all threads meet.
    bool live = true;
    __device__ __forceinline__ void wait(uint32_t* status) {
        if (live) live = mbar_wait_bounded(full + slot, phase, status, 2000000000ull, kWhereProducer, false);  // 2 s
    }
    __device__ __forceinline__ void next() {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
};
constexpr int MOST_SLOTS = 8;

// row_sum for a row on a CTA of at most 16 warps: every thread adds the warps' sums, in order, as it reads them (buf: two
// sets of 16 x N floats, used in turn).
template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], float* buf, int& turn) {
    warp_sums<N>(v);
    float* b = buf + turn * 16 * N;
    turn ^= 1;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & (N == 2 ? 15 : 31)) == 0) b[(threadIdx.x & 16) + (threadIdx.x >> 5)] = v[0];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float4* q = reinterpret_cast<const float4*>(b + i * 16);
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // (places past the last warp hold zeros)
            if (j * 4 >= warps) break;
            const float4 w = q[j];
            s += w.x;
            s += w.y;
            s += w.z;
            s += w.w;
        }
        v[i] = s;
    }
}

using f2 = unsigned long long;
__device__ __forceinline__ f2 both(float v) { return tc::f2_pack(v, v); }
// Sum of a pair's halves.
__device__ __forceinline__ float halves_sum(f2 v) {
    float a, b;
    tc::f2_unpack(v, a, b);
    return a + b;
}
// A piece of 16 bytes as pairs.
template <typename T>
__device__ __forceinline__ void pairs(const uint4& r, f2 (&f)[sizeof(T) == 2 ? 4 : 2]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = tc::f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) f[i] = tc::f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
}
template <typename T>
__device__ __forceinline__ uint4 unpair(const f2 (&f)[sizeof(T) == 2 ? 4 : 2]) {
    uint32_t w[4];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            tc::f2_unpack(f[i], a, b);
            w[i] = tc::pack_bf16x2(a, b);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float a, b;
            tc::f2_unpack(f[i], a, b);
            w[2 * i] = __float_as_uint(a);
            w[2 * i + 1] = __float_as_uint(b);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int NV, int THREADS, int PER_SM>
__global__ void __launch_bounds__(THREADS, PER_SM) fwd_ring_kernel(const FwdArgs p, int slots, uint32_t* status) {
    constexpr int P = sizeof(T) == 2 ? 4 : 2;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint64_t bars[MOST_SLOTS];
    __shared__ __align__(16) float buf[2 * 16 * 2];  // (one value in turn 0, two in turn 1)
    if (threadIdx.x < 2 * 16 * 2) buf[threadIdx.x] = 0.0f;
    int turn = 0;
    const uint32_t bytes = static_cast<uint32_t>(p.h) * sizeof(T);
    Ring ring{smem, nullptr, bytes, slots};
    ring.init(bars);
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int tx = threadIdx.x, nx = blockDim.x;
    auto load = [&](long long row, int slot) {
        if (tx == 0 && row < p.rows) {
            mbar_arrive_expect_tx(ring.full + slot, bytes);
            bulk_load(ring.at + static_cast<size_t>(slot) * bytes, static_cast<const T*>(p.x) + row * p.ldx, bytes, ring.full + slot);
        }
    };
    for (int i = 0; i < slots; ++i) load(blockIdx.x + static_cast<long long>(i) * gridDim.x, i);
    const uint32_t one = sizeof(T) == 2 ? 0x3F803F80u : 0x3F800000u;
    uint4 gamma[NV], beta[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * nx + tx;
        gamma[i] = make_uint4(one, one, one, one);
        beta[i] = make_uint4(0, 0, 0, 0);
        if (c < p.vecs && p.gamma != nullptr) gamma[i] = static_cast<const uint4*>(p.gamma)[c];
        if (c < p.vecs && p.beta != nullptr) beta[i] = static_cast<const uint4*>(p.beta)[c];
    }
    const float inv = 1.0f / static_cast<float>(p.h);
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        ring.wait(status);
        const uint4* x = reinterpret_cast<const uint4*>(ring.at + static_cast<size_t>(ring.slot) * bytes);
        f2 v[NV][P], sum = 0;  // (the bits of two zeros)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * nx + tx;
            if (c >= p.vecs) continue;
            pairs<T>(x[c], v[i]);
#pragma unroll
            for (int j = 0; j < P; ++j) sum = tc::f2_add(sum, v[i][j]);
        }
        float s[1] = {halves_sum(sum)};
        cta_sum<1>(s, buf, turn);
        load(row + static_cast<long long>(slots) * gridDim.x, ring.slot);  // (all threads have read the slot)
        ring.next();
        const float m0 = s[0] * inv;
        f2 less = both(-m0), squares = 0;
        sum = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (i * nx + tx >= p.vecs) continue;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                v[i][j] = tc::f2_add(v[i][j], less);
                sum = tc::f2_add(sum, v[i][j]);
                squares = tc::f2_fma(v[i][j], v[i][j], squares);
            }
        }
        float d[2] = {halves_sum(sum), halves_sum(squares)};
        cta_sum<2>(d, buf, turn);
        float off, rstd;
        bool far;
        spread(d[0], d[1], p.h, inv, p.eps, off, rstd, far);
        if (tx == 0 && p.mean != nullptr) {
            p.mean[row] = corrected(m0, off);
            p.rstd[row] = rstd;
        }
        if (far) {  // (the same in all threads; most rows' are not)
            less = both(-off);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j) v[i][j] = tc::f2_add(v[i][j], less);
        }
        const f2 r2 = both(rstd);
        uint4* y = reinterpret_cast<uint4*>(static_cast<T*>(p.y) + row * p.ldy);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * nx + tx;
            if (c >= p.vecs) continue;
            f2 g[P], b[P];
            pairs<T>(gamma[i], g);
            pairs<T>(beta[i], b);
#pragma unroll
            for (int j = 0; j < P; ++j)
                v[i][j] = tc::f2_fma(tc::f2_mul(v[i][j], r2), g[j], b[j]);
            y[c] = unpair<T>(v[i]);
        }
    }
}

template <typename T, int NV, int THREADS, int PER_SM>
__global__ void __launch_bounds__(THREADS, PER_SM) bwd_ring_kernel(const BwdArgs p, int slots, uint32_t* status) {
    constexpr int P = sizeof(T) == 2 ? 4 : 2;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint64_t bars[MOST_SLOTS];
    __shared__ __align__(16) float buf[2 * 16 * 2];
    if (threadIdx.x < 2 * 16 * 2) buf[threadIdx.x] = 0.0f;
    int turn = 0;
    const uint32_t bytes = static_cast<uint32_t>(p.h) * sizeof(T);  // a slot: x, then dy
    Ring ring{smem, nullptr, 2 * bytes, slots};
    ring.init(bars);
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int tx = threadIdx.x, nx = blockDim.x;
    auto load = [&](long long row, int slot) {
        if (tx == 0 && row < p.rows) {
            uint8_t* at = ring.at + static_cast<size_t>(slot) * 2 * bytes;
            mbar_arrive_expect_tx(ring.full + slot, 2 * bytes);
            bulk_load(at, static_cast<const T*>(p.x) + row * p.ldx, bytes, ring.full + slot);
            bulk_load(at + bytes, static_cast<const T*>(p.dy) + row * p.lddy, bytes, ring.full + slot);
        }
    };
    for (int i = 0; i < slots; ++i) load(blockIdx.x + static_cast<long long>(i) * gridDim.x, i);
    const uint32_t one = sizeof(T) == 2 ? 0x3F803F80u : 0x3F800000u;
    uint4 gamma[NV];
    f2 dgamma[NV][P], dbeta[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * nx + tx;
        gamma[i] = make_uint4(one, one, one, one);
        if (c < p.vecs && p.gamma != nullptr) gamma[i] = static_cast<const uint4*>(p.gamma)[c];
#pragma unroll
        for (int j = 0; j < P; ++j) dgamma[i][j] = dbeta[i][j] = 0;
    }
    const float inv = 1.0f / static_cast<float>(p.h);
    // the statistics of this row and the next three: a load takes longer than a row
    constexpr int AHEAD = 4;
    float means[AHEAD], rstds[AHEAD];
    auto stat = [&](int i, long long row) {
        means[i] = row < p.rows ? p.mean[row] : 0.0f;
        rstds[i] = row < p.rows ? p.rstd[row] : 0.0f;
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) stat(i, blockIdx.x + static_cast<long long>(i) * gridDim.x);
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float mean = means[0], rstd = rstds[0];
#pragma unroll
        for (int i = 0; i + 1 < AHEAD; ++i) {
            means[i] = means[i + 1];
            rstds[i] = rstds[i + 1];
        }
        stat(AHEAD - 1, row + static_cast<long long>(AHEAD) * gridDim.x);
        ring.wait(status);
        const uint4* x = reinterpret_cast<const uint4*>(ring.at + static_cast<size_t>(ring.slot) * 2 * bytes);
        const uint4* dy = reinterpret_cast<const uint4*>(ring.at + static_cast<size_t>(ring.slot) * 2 * bytes + bytes);
        const f2 less = both(-mean), r2 = both(rstd);
        f2 s0 = 0, s1 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * nx + tx;
            if (c >= p.vecs) continue;
            f2 n[P], d[P], w[P];
            pairs<T>(x[c], n);
            pairs<T>(dy[c], d);
            pairs<T>(gamma[i], w);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                n[j] = tc::f2_mul(tc::f2_add(n[j], less), r2);
                dgamma[i][j] = tc::f2_fma(d[j], n[j], dgamma[i][j]);
                dbeta[i][j] = tc::f2_add(dbeta[i][j], d[j]);
                d[j] = tc::f2_mul(d[j], w[j]);
                s0 = tc::f2_add(s0, d[j]);
                s1 = tc::f2_fma(d[j], n[j], s1);
            }
        }
        float s[2] = {halves_sum(s0), halves_sum(s1)};
        cta_sum<2>(s, buf, turn);
        // all threads are past the row before: its slot may be filled again
        if (row != blockIdx.x) load(row + static_cast<long long>(slots - 1) * gridDim.x, ring.slot == 0 ? slots - 1 : ring.slot - 1);
        ring.next();
        // rstd (g - a - n b), from the slot once more
        const f2 a = both(-s[0] * inv), b = both(-s[1] * inv);
        uint4* dx = reinterpret_cast<uint4*>(static_cast<T*>(p.dx) + row * p.lddx);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * nx + tx;
            if (c >= p.vecs) continue;
            f2 n[P], d[P], w[P];
            pairs<T>(x[c], n);
            pairs<T>(dy[c], d);
            pairs<T>(gamma[i], w);
#pragma unroll
            for (int j = 0; j < P; ++j)
                d[j] = tc::f2_mul(r2, tc::f2_fma(tc::f2_mul(tc::f2_add(n[j], less), r2), b, tc::f2_fma(d[j], w[j], a)));
            dx[c] = unpair<T>(d);
        }
    }
    if (p.part == nullptr) return;
    float* out = p.part + static_cast<long long>(blockIdx.x) * 2 * p.h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * nx + tx;
        if (c >= p.vecs) continue;
#pragma unroll
        for (int j = 0; j < P; j += 2) {
            reinterpret_cast<ulonglong2*>(out)[(c * P + j) / 2] = make_ulonglong2(dgamma[i][j], dgamma[i][j + 1]);
            reinterpret_cast<ulonglong2*>(out + p.h)[(c * P + j) / 2] = make_ulonglong2(dbeta[i][j], dbeta[i][j + 1]);
        }
    }
}

// Sums of the parts' columns: 32 V columns a CTA, part i on warp i % 16, the warps' sums added in order.  All of a warp's
// loads are on their way at once.
constexpr int PART_WARPS = 16;
template <int V>
__global__ void __launch_bounds__(32 * PART_WARPS) parts_kernel(const float* part, int parts, int h, void* dgamma, void* dbeta, int f32) {
    using R = typename std::conditional<V == 4, float4, typename std::conditional<V == 2, float2, float>::type>::type;
    __shared__ __align__(16) float sum[PART_WARPS][32 * V];
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5, which = blockIdx.y, col = (blockIdx.x * 32 + lane) * V;
    void* out = which ? dbeta : dgamma;
    if (out == nullptr) return;
    float s[V] = {};
    if (col < h) {
        constexpr int BATCH = 19;
        for (int i0 = r; i0 < parts; i0 += BATCH * PART_WARPS) {
            R v[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int at = i0 + i * PART_WARPS;
                v[i] = at < parts ? *reinterpret_cast<const R*>(part + (static_cast<long long>(at) * 2 + which) * h + col) : R{};
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] += reinterpret_cast<const float*>(v + i)[j];
        }
    }
    *reinterpret_cast<R*>(&sum[r][lane * V]) = *reinterpret_cast<R*>(s);
    __syncthreads();
    const int c = blockIdx.x * 32 * V + threadIdx.x;
    if (threadIdx.x < 32 * V && c < h) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < PART_WARPS; ++i) t += sum[i][threadIdx.x];
        if (f32) static_cast<float*>(out)[c] = t;
        else static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(t);
    }
}

template <typename... P, typename... A>
tpmlp_status launch(void (*kern)(P...), dim3 grid, dim3 block, int smem, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
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

// How the ring kernels run: threads of a CTA at most, elements of each, CTAs an SM in the forward and in the backward.  Few
// threads with much to do: what a thread does once a row (waits, the sums across the CTA) is as much work as 10 elements.
// 8192 x 5120 bf16, backward without dgamma, dbeta: 16 elements a thread 52 us, 32 45 (floor 37); forward 36, 29 (25; this and
// the forward's figures below before its mean was corrected, which takes 2 to 9 % of the time).
// Which CTAs fit an SM goes by registers, so each width has its own: 8192 x 4096 with CTAs of 160 threads at most, three and
// two an SM, 25.6 and 43.6 us, of 128, four and three, 23.8 and 40.6; x 2048 with 128 21.2 and 32.7, of 96 17.6 and 30.1.
// 4096 x 16384 47 and 82, by the kernels above 85 and 147.
template <int THREADS, int ELEMENTS, int FWD, int BWD>
struct Conf {
    static constexpr int threads = THREADS, elements = ELEMENTS, fwd = FWD, bwd = BWD;
};
struct RingShape {
    int threads, slots;
};
RingShape ring_shape(int vecs, int nv, int per_sm, int64_t slot_bytes) {
    return {(vecs + 32 * nv - 1) / (32 * nv) * 32,
            static_cast<int>(std::min<int64_t>(MOST_SLOTS, (216 * 1024 / per_sm - 2048) / slot_bytes))};
}

template <typename Kern>
bool allow_smem(Kern kern, const DeviceInfo& dev, int bytes, PerDevice<bool>& done) {
    return done.get(dev.device, [&](bool& ok) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) set_error("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return ok = e == cudaSuccess;
    });
}

template <typename Kern, typename A>
tpmlp_status launch_ring(Kern kern, PerDevice<bool>& done, int grid, const RingShape& r, int64_t slot_bytes, const A& a,
                         const DeviceInfo& dev, cudaStream_t st) {
    if (!allow_smem(kern, dev, 216 * 1024, done)) return TPMLP_ERR_CUDA;
    return launch(kern, dim3(grid), dim3(r.threads), static_cast<int>(r.slots * slot_bytes), st, a, r.slots, dev.status);
}

// Calls f(type, configuration) for rows of `vecs` pieces that the ring kernels take; whether it ran.
template <typename F>
bool with_ring(bool f32, bool wide, int vecs, F&& f) {
    const int h = vecs * (f32 ? 4 : 8);
    if (!wide || h <= WARP_ROW) return false;
    auto pick = [&](auto t) {
        const int threads = (h + 31) / 32;
        if (threads <= 96) return f(t, Conf<96, 32, 5, 4>{});
        if (threads <= 128) return f(t, Conf<128, 32, 4, 3>{});
        if (threads <= 160) return f(t, Conf<160, 32, 3, 2>{});
        if (threads <= 256) return f(t, Conf<256, 32, 2, 2>{});
        if (threads <= 384) return f(t, Conf<384, 32, 1, 1>{});
        return threads <= 512 && f(t, Conf<512, 32, 1, 1>{});
    };
    return f32 ? pick(float{}) : pick(__nv_bfloat16{});
}

}  // namespace

int64_t layernorm_ws_bytes(int64_t rows, int64_t h) { return std::min<int64_t>(rows, most_parts(h)) * 2 * h * 4; }

tpmlp_status launch_layernorm_fwd(const void* X, const void* gamma, const void* beta, void* Y, float* mean, float* rstd, int64_t rows,
                                  int64_t h, int64_t ldx, int64_t ldy, float eps, bool f32, const DeviceInfo& dev, cudaStream_t st) {
    const int es = f32 ? 4 : 2;
    const bool wide = wide_rows(h, es, {X, gamma, beta, Y}, {ldx, ldy});
    const int vec = wide ? 16 / es : 1;
    const FwdArgs a{X, gamma, beta, Y, mean, rstd, rows, ldx, ldy, static_cast<int>(h), static_cast<int>(h / vec), eps};
    tpmlp_status r = TPMLP_OK;
    if (with_ring(f32, wide, a.vecs, [&](auto t, auto conf) {
            using T = decltype(t);
            using C = decltype(conf);
            constexpr int NV = C::elements * static_cast<int>(sizeof(T)) / 16;
            static PerDevice<bool> done;
            const RingShape q = ring_shape(a.vecs, NV, C::fwd, h * es);
            const int grid = C::fwd * dev.sm_count;
            if (q.slots < 2 || rows <= 2 * grid) return false;
            r = launch_ring(fwd_ring_kernel<T, NV, C::threads, C::fwd>, done, grid, q, h * es, a, dev, st);
            return true;
        }))
        return r;
    const Shape s = shape_of(vec, a.vecs);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((rows + s.y - 1) / s.y, int64_t(dev.sm_count) * 64));
    return by_shape(f32, wide, s.nv, [&](auto t, auto v, auto nv) {
        return launch(fwd_kernel<decltype(t), decltype(v)::value, decltype(nv)::value>, dim3(grid), dim3(s.x, s.y), 0, st, a);
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
    tpmlp_status r = TPMLP_OK;
    int grid = 0;
    if (!with_ring(f32, wide, a.vecs, [&](auto t, auto conf) {
            using T = decltype(t);
            using C = decltype(conf);
            constexpr int NV = C::elements * static_cast<int>(sizeof(T)) / 16;
            static PerDevice<bool> done;
            const RingShape q = ring_shape(a.vecs, NV, C::bwd, 2 * h * es);
            grid = std::min(C::bwd * dev.sm_count, most_parts(h));
            if (q.slots < 2 || rows <= 2 * grid) return false;
            r = launch_ring(bwd_ring_kernel<T, NV, C::threads, C::bwd>, done, grid, q, 2 * h * es, a, dev, st);
            return true;
        })) {
        const Shape s = shape_of(vec, a.vecs);
        const int per_sm = s.y == 1 && s.x <= 256 && s.nv * vec <= 8 ? 4 : 2;  // (few registers: more rows at once)
        grid = static_cast<int>(std::min<int64_t>({(rows + s.y - 1) / s.y, int64_t(per_sm) * dev.sm_count, most_parts(h)}));
        const int smem = s.y > 1 && sums ? static_cast<int>(s.y * 2 * h * 4) : 0;
        r = by_shape(f32, wide, s.nv, [&](auto t, auto v, auto nv) {
            auto kern = bwd_kernel<decltype(t), decltype(v)::value, decltype(nv)::value>;
            static PerDevice<bool> done;
            return allow_smem(kern, dev, 8 * 2 * WARP_ROW * 4, done) ? launch(kern, dim3(grid), dim3(s.x, s.y), smem, st, a) : TPMLP_ERR_CUDA;
        });
    }
    if (r != TPMLP_OK || !sums) return r;
    // columns of a thread: more CTAs where rows are short (8192 x 2048: 30.4 us with four, 28.1; x 5120 51.8, 51.9; 64 x 5120 5.7, 5.9)
    const int v = h % 4 == 0 && h > 4096 ? 4 : h % 2 == 0 ? 2 : 1;
    const dim3 cols(static_cast<unsigned>((h + 32 * v - 1) / (32 * v)), 2);
    return launch(v == 4 ? parts_kernel<4> : v == 2 ? parts_kernel<2> : parts_kernel<1>, cols, dim3(32 * PART_WARPS), 0, st,
                  static_cast<const float*>(ws), grid, static_cast<int>(h), dgamma, dbeta, grad_f32 ? 1 : 0);
}

}  // namespace tpmlp
