// MXFP4 quantisation along either axis, or both from one read, and its inverse.
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace {

using mx::abs_bits;

// 16 bytes of a row (8 bf16 or 4 fp32 values) widened to fp32; the first n of them, the rest zero.
template <bool F32>
struct Vec {
    static constexpr int E = F32 ? 4 : 8;
    float v[E];
    uint4 raw;
    __device__ __forceinline__ void load(const void* p, int n) {
        if (n >= E) {
            raw = *static_cast<const uint4*>(p);
        } else {  // a row's ragged end: nothing past it is read
            uint32_t w[4] = {0, 0, 0, 0};
            for (int i = 0; i < n; ++i) {
                if constexpr (F32) {
                    w[i] = static_cast<const uint32_t*>(p)[i];
                } else {
                    w[i >> 1] |= static_cast<uint32_t>(static_cast<const unsigned short*>(p)[i]) << (16 * (i & 1));
                }
            }
            raw = make_uint4(w[0], w[1], w[2], w[3]);
        }
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if constexpr (F32) v[i] = __uint_as_float(w[i]);
            else v[i] = __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
        }
    }
    // Largest |v| over this thread's values and those of the other lanes of its block of 32.
    __device__ __forceinline__ uint32_t block_amax() const {
        uint32_t a = abs_bits(v[0]);
#pragma unroll
        for (int i = 1; i < E; ++i) a = max(a, abs_bits(v[i]));
#pragma unroll
        for (int d = 1; d < 32 / E; d *= 2) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, d));
        return a;
    }
    // This thread's codes (E of them in the low E * 4 bits).
    __device__ __forceinline__ uint32_t codes(uint32_t s) const {
        const float i = mx::inverse_scale(s);
        if (s == 255u) return 0;
        if constexpr (F32) return mx::encode8(v[0] * i, v[1] * i, v[2] * i, v[3] * i, 0.f, 0.f, 0.f, 0.f);
        else
            return mx::encode8(v[0] * i, v[1] * i, v[2] * i, v[3] * i, v[4] * i, v[5] * i, v[6] * i, v[7] * i);
    }
};

struct QuantArgs {
    const uint8_t* x;
    long long ldx, ss;  // row pitch and shard stride in bytes
    int rows, cols, p;  // logical [rows, p * cols]; column c of shard i is i * cols + c
    uint8_t* q;
    uint8_t* s;
    uint8_t* qt;
    uint8_t* st;
};

// Along the columns only.  A group of 16 lanes takes 16 consecutive 16-byte pieces of one row (4
// blocks of bf16 values, 2 of fp32), one piece a lane; a block's maximum takes 2 (bf16) or 3
// (fp32) shuffles, its codes go out 4 (2) bytes a lane, its scales as one word (half word).  Bound
// by memory; for one token by the launch.
template <bool F32>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantArgs a) {
    constexpr int E = Vec<F32>::E, SPAN = 16 * E, ES = F32 ? 4 : 2;
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int lane16 = threadIdx.x & 15;
    const long long total_cols = static_cast<long long>(a.cols) * a.p;
    // spans up to a multiple of 128 columns: the scales of padding blocks are written as zero
    const long long spans = (total_cols + 127) / 128 * (128 / SPAN);
    const long long k_tiles = (total_cols + 127) / 128;
    const long long pitch = (total_cols + 31) / 32 * 16;
    const long long items = spans * a.rows;
    const long long step = static_cast<long long>(gridDim.x) * 16;
    for (long long it = static_cast<long long>(blockIdx.x) * 16 + (threadIdx.x >> 4); __any_sync(0xFFFFFFFFu, it < items);
         it += step) {
        const bool live = it < items;
        const long long row = live ? it / spans : 0;
        const long long c0 = live ? (it - row * spans) * SPAN + lane16 * E : total_cols;
        Vec<F32> v;
        int n = 0;
        const uint8_t* src = a.x;
        if (c0 < total_cols) {
            // shards are at least 32 columns apart in multiples of 32, so a piece lies in one shard
            const long long sh = a.p == 1 ? 0 : c0 / a.cols;
            const long long c = c0 - sh * a.cols;
            n = static_cast<int>(a.cols - c < E ? a.cols - c : E);
            src = a.x + sh * a.ss + row * a.ldx + c * ES;
        }
        v.load(src, n);
        const uint32_t s = mx::scale_of(v.block_amax());
        const uint32_t code = v.codes(s);
        if (c0 / 2 < pitch && live) {
            if constexpr (F32) *reinterpret_cast<uint16_t*>(a.q + row * pitch + c0 / 2) = static_cast<uint16_t>(code);
            else *reinterpret_cast<uint32_t*>(a.q + row * pitch + c0 / 2) = code;
        }
        // the group's scales in one word
        constexpr int LB = 32 / E;  // lanes a block
        const int lane = threadIdx.x & 31;
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 16 / LB; ++j) w |= __shfl_sync(0xFFFFFFFFu, s, (lane & 16) + j * LB) << (8 * j);
        if (lane16 == 0 && live) {
            uint8_t* d = a.s + mx::scale_offset(row, c0 / 32, k_tiles);
            if constexpr (F32) *reinterpret_cast<uint16_t*>(d) = static_cast<uint16_t>(w);
            else *reinterpret_cast<uint32_t*>(d) = w;
        }
    }
}

// Along the rows, and along the columns too where q is given: a CTA takes 128 rows x 256 bytes of
// columns (128 bf16, 64 fp32).  It reads the tile once, 16 lanes to a row, quantises the rows'
// blocks on the way into shared memory, and then the columns' from there (a thread takes 32 rows of
// one word: two bf16 columns or one fp32 column), whose codes it gathers in shared memory so that
// each column leaves as one run of 64 bytes.
template <bool F32>
__global__ void __launch_bounds__(256) quantize_both_kernel(const QuantArgs a) {
    constexpr int E = Vec<F32>::E, ES = F32 ? 4 : 2, TC = 256 / ES, LB = 32 / E;
    __shared__ __align__(16) uint32_t tile[128 * 64];
    __shared__ __align__(16) uint8_t out[TC * 80];  // 64 bytes of codes a column, pitch 80
    __shared__ uint32_t sc[TC];
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int t = threadIdx.x, lane16 = t & 15;
    const long long total_cols = static_cast<long long>(a.cols) * a.p;
    // (up to a multiple of 128 columns: the scales of padding blocks are written as zero)
    const unsigned col_tiles = static_cast<unsigned>((total_cols + 127) / 128 * (128 / TC));
    const int row_tile = static_cast<int>(blockIdx.x / col_tiles);
    const long long c_tile = static_cast<long long>(blockIdx.x - row_tile * col_tiles) * TC;
    const int r_tile = row_tile * 128;
    const long long k_tiles = (total_cols + 127) / 128;
    const long long pitch = (total_cols + 31) / 32 * 16;
    {
        const long long c0 = c_tile + lane16 * E;
        const uint8_t* src = a.x;
        int n = 0;
        if (c0 < total_cols) {
            const long long sh = a.p == 1 ? 0 : c0 / a.cols;
            const long long c = c0 - sh * a.cols;
            n = static_cast<int>(a.cols - c < E ? a.cols - c : E);
            src = a.x + sh * a.ss + c * ES;
        }
        Vec<F32> v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = r_tile + (t >> 4) + i * 16;
            v[i].load(src + row * a.ldx, row < a.rows ? n : 0);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = (t >> 4) + i * 16, row = r_tile + r;
            *reinterpret_cast<uint4*>(tile + r * 64 + lane16 * 4) = v[i].raw;
            if (a.q != nullptr) {
                const uint32_t s = mx::scale_of(v[i].block_amax());
                const uint32_t code = v[i].codes(s);
                uint32_t w = 0;
                const int lane = t & 31;
#pragma unroll
                for (int j = 0; j < 16 / LB; ++j) w |= __shfl_sync(0xFFFFFFFFu, s, (lane & 16) + j * LB) << (8 * j);
                if (row < a.rows) {
                    if (c0 / 2 < pitch) {
                        if constexpr (F32)
                            *reinterpret_cast<uint16_t*>(a.q + row * pitch + c0 / 2) = static_cast<uint16_t>(code);
                        else *reinterpret_cast<uint32_t*>(a.q + row * pitch + c0 / 2) = code;
                    }
                    if (lane16 == 0) {
                        uint8_t* d = a.s + mx::scale_offset(row, c0 / 32, k_tiles);
                        if constexpr (F32) *reinterpret_cast<uint16_t*>(d) = static_cast<uint16_t>(w);
                        else *reinterpret_cast<uint32_t*>(d) = w;
                    }
                }
            }
        }
    }
    __syncthreads();
    {
        const int word = t & 63, rb = t >> 6;
        float lo[32], hi[32];
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            const uint32_t w = tile[(rb * 32 + r) * 64 + word];
            if constexpr (F32) {
                lo[r] = __uint_as_float(w);
            } else {
                lo[r] = __uint_as_float(w << 16);
                hi[r] = __uint_as_float(w & 0xFFFF0000u);
            }
        }
        uint4 codes;
        constexpr int PER = F32 ? 1 : 2;
        uint8_t* sb = reinterpret_cast<uint8_t*>(sc);
        uint32_t s = mx::quantize32(lo, codes);
        *reinterpret_cast<uint4*>(out + word * PER * 80 + rb * 16) = codes;
        sb[word * PER * 4 + rb] = static_cast<uint8_t>(s);
        if constexpr (!F32) {
            s = mx::quantize32(hi, codes);
            *reinterpret_cast<uint4*>(out + (word * 2 + 1) * 80 + rb * 16) = codes;
            sb[(word * 2 + 1) * 4 + rb] = static_cast<uint8_t>(s);
        }
    }
    __syncthreads();
    const long long t_pitch = (static_cast<long long>(a.rows) + 31) / 32 * 16;
    const long long t_tiles = (static_cast<long long>(a.rows) + 127) / 128;
#pragma unroll
    for (int i = 0; i < TC / 64; ++i) {
        const int c = (t >> 2) + i * 64;
        const long long col = c_tile + c, at = r_tile / 2 + (t & 3) * 16;
        if (col < total_cols && at < t_pitch)
            *reinterpret_cast<uint4*>(a.qt + col * t_pitch + at) = *reinterpret_cast<const uint4*>(out + c * 80 + (t & 3) * 16);
    }
    if (t < TC && c_tile + t < total_cols)
        *reinterpret_cast<uint32_t*>(a.st + mx::scale_offset(c_tile + t, row_tile * 4LL, t_tiles)) = sc[t];
}

// Values of an operand: a thread takes 8 codes.
template <bool F32>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, void* out,
                                                         long long rows, long long k) {
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const long long pitch = (k + 31) / 32 * 16, k_tiles = (k + 127) / 128, words = (k + 7) / 8;
    const long long items = rows * words;
    for (long long it = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; it < items;
         it += static_cast<long long>(gridDim.x) * 256) {
        const long long row = it / words, w = it - row * words;
        const uint32_t c = *reinterpret_cast<const uint32_t*>(q + row * pitch + w * 4);
        const float sv = mx::scale_value(s[mx::scale_offset(row, w / 4, k_tiles)]);
        float v[8];
        mx::decode8(c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= sv;
        const long long at = row * k + w * 8;
        if constexpr (F32) {
            float* d = static_cast<float*>(out) + at;
            if (k % 4 == 0 && w * 8 + 8 <= k) {
                *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4*>(d + 4) = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                for (int i = 0; i < 8 && w * 8 + i < k; ++i) d[i] = v[i];
            }
        } else {
            __nv_bfloat16* d = static_cast<__nv_bfloat16*>(out) + at;
            if (k % 8 == 0) {
                __nv_bfloat162 b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(b);
            } else {
                for (int i = 0; i < 8 && w * 8 + i < k; ++i) d[i] = __float2bfloat16_rn(v[i]);
            }
        }
    }
}

template <typename... P, typename... A>
tpmlp_status launch_pdl(const char* what, void (*kern)(P...), dim3 grid, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("%s launch: %s", what, cudaGetErrorString(e));
        return TPMLP_ERR_CUDA;
    }
    count_launch();
    return TPMLP_OK;
}

}  // namespace

tpmlp_status launch_mxfp4_quantize(const void* X, int64_t ldx, void* Q, void* S, void* Qt, void* St, int64_t rows,
                                   int64_t cols, int p, bool f32, const DeviceInfo& dev, cudaStream_t st) {
    const int64_t es = f32 ? 4 : 2;
    QuantArgs a{static_cast<const uint8_t*>(X), ldx * es, rows * ldx * es, static_cast<int>(rows),
                static_cast<int>(cols / p), p, static_cast<uint8_t*>(Q), static_cast<uint8_t*>(S),
                static_cast<uint8_t*>(Qt), static_cast<uint8_t*>(St)};
    if (Qt == nullptr) {
        const int64_t span = f32 ? 64 : 128;
        const int64_t items = (cols + 127) / 128 * (128 / span) * rows;
        const int64_t most = static_cast<int64_t>(dev.sm_count) * 16;
        const dim3 grid(static_cast<unsigned>(std::min<int64_t>((items + 15) / 16, most)));
        return f32 ? launch_pdl("MXFP4 quantisation", quantize_rows_kernel<true>, grid, st, a)
                   : launch_pdl("MXFP4 quantisation", quantize_rows_kernel<false>, grid, st, a);
    }
    const int64_t tc = f32 ? 64 : 128;
    const dim3 grid(static_cast<unsigned>((cols + 127) / 128 * (128 / tc) * ((rows + 127) / 128)));
    return f32 ? launch_pdl("MXFP4 quantisation", quantize_both_kernel<true>, grid, st, a)
               : launch_pdl("MXFP4 quantisation", quantize_both_kernel<false>, grid, st, a);
}

tpmlp_status launch_mxfp4_dequantize(const void* Q, const void* S, void* out, int64_t rows, int64_t k, bool f32,
                                     const DeviceInfo& dev, cudaStream_t st) {
    const int64_t items = rows * ((k + 7) / 8);
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((items + 255) / 256, static_cast<int64_t>(dev.sm_count) * 32)));
    const auto* q = static_cast<const uint8_t*>(Q);
    const auto* s = static_cast<const uint8_t*>(S);
    return f32 ? launch_pdl("MXFP4 dequantisation", dequantize_kernel<true>, grid, st, q, s, out, (long long)rows, (long long)k)
               : launch_pdl("MXFP4 dequantisation", dequantize_kernel<false>, grid, st, q, s, out, (long long)rows, (long long)k);
}

}  // namespace tpmlp
