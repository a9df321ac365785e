// MXFP4 quantisation along either axis, or both from one read, and its inverse.
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace {

// 16 bytes of a row: 8 bf16 or 4 fp32 values.
template <bool F32>
struct Piece {
    static constexpr int E = F32 ? 4 : 8, ES = F32 ? 4 : 2;
    static constexpr int LANES = 32 / E;  // lanes that share a block of 32

    // The first n values at p, zeros behind them; nothing past them is read.
    static __device__ __forceinline__ uint4 load(const uint8_t* p, int n) {
        if (n >= E) return *reinterpret_cast<const uint4*>(p);
        uint32_t w[4] = {0, 0, 0, 0};
        for (int i = 0; i < n; ++i) {
            if constexpr (F32) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
            else w[i >> 1] |= static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(p)[i]) << (16 * (i & 1));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // Scale byte of the block that this lane and its neighbours hold.
    static __device__ __forceinline__ uint32_t scale(const uint4& r) {
        uint32_t a;  // the bits of the largest magnitude as fp32
        if constexpr (F32) {
            a = __float_as_uint(mx::amax3(mx::amax3(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z)),
                                          __uint_as_float(r.w), 0.0f));
        } else {
            const uint32_t m = mx::amax_bf16x2(mx::amax_bf16x2(r.x, r.y), mx::amax_bf16x2(r.z, r.w)) & 0x7FFF7FFFu;
            a = max(m & 0xFFFF0000u, m << 16);
        }
#pragma unroll
        for (int d = 1; d < LANES; d *= 2) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, d));
        return mx::scale_of(a);
    }
    // This lane's codes, E of them in the low E * 4 bits.
    static __device__ __forceinline__ uint32_t codes(const uint4& r, uint32_t s) {
        const float inv = mx::inverse_scale(s);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F32) {
                v[i] = __uint_as_float(w[i]);
                v[4 + i] = 0.0f;
            } else {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
#pragma unroll
        for (int i = 0; i < E; i += 2) mx::mul2(v[i], v[i + 1], inv);
        return s == 255u ? 0u : mx::encode8(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
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
    long long spans;    // row kernel: warp spans a row; both kernel: column tiles
    long long items;    // row kernel: spans of all rows; both kernel: tiles
};

// Address and number of values of the piece at logical column c0 (row 0).
template <bool F32>
__device__ __forceinline__ const uint8_t* piece_at(const QuantArgs& a, long long c0, int& n) {
    n = 0;
    if (c0 >= static_cast<long long>(a.cols) * a.p) return a.x;
    // shards are multiples of 32 columns wide (or there is one), so a piece lies in one shard
    const long long sh = a.p == 1 ? 0 : c0 / a.cols;
    const long long c = c0 - sh * a.cols;
    n = static_cast<int>(a.cols - c < Piece<F32>::E ? a.cols - c : Piece<F32>::E);
    return a.x + sh * a.ss + c * Piece<F32>::ES;
}

// Along the columns only: a warp takes U spans of 512 bytes of a row, a 16-byte piece a lane, all
// loaded before the first is worked on.  A block's maximum takes 2 (bf16) or 3 (fp32) shuffles; its
// codes go out 4 (2) bytes a lane.  Bound by memory; for one token by the launch.
template <bool F32, int U>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantArgs a) {
    using P = Piece<F32>;
    constexpr int SPAN = 32 * P::E;
    const int lane = threadIdx.x & 31;
    const long long total = static_cast<long long>(a.cols) * a.p;
    const long long k_tiles = (total + 127) / 128, pitch = (total + 31) / 32 * 16;
    const long long it0 = (static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * U;
    long long row = it0 / a.spans, span = it0 - row * a.spans;
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    uint4 r[U];
    long long rows[U], c0[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        rows[i] = row;
        c0[i] = span * SPAN + lane * P::E;
        int n;
        const uint8_t* src = piece_at<F32>(a, c0[i], n);
        r[i] = P::load(src + row * a.ldx, row < a.rows ? n : 0);
        if (++span == a.spans) {
            span = 0;
            ++row;
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const uint32_t s = P::scale(r[i]);
        const uint32_t code = P::codes(r[i], s);
        if (rows[i] >= a.rows) continue;
        if (c0[i] / 2 < pitch) {
            uint8_t* d = a.q + rows[i] * pitch + c0[i] / 2;
            if constexpr (F32) *reinterpret_cast<uint16_t*>(d) = static_cast<uint16_t>(code);
            else *reinterpret_cast<uint32_t*>(d) = code;
        }
        // (padding blocks up to a whole scale tile: zero)
        if (lane % P::LANES == 0 && c0[i] < k_tiles * 128)
            a.s[mx::scale_offset(rows[i], c0[i] >> 5, k_tiles)] = static_cast<uint8_t>(s);
    }
}

// Along the rows, and along the columns too where q is given.  A CTA walks tiles of 128 rows x 256
// bytes of columns (128 bf16, 64 fp32) through two shared-memory buffers, the next tile's
// asynchronous copies running behind the work on this one: the tile's values are read from memory
// once and its two quantisations work from shared memory.  Along the columns 16 lanes take a row;
// along the rows a thread takes 32 rows of one word (two bf16 columns or one fp32 column), and the
// codes are gathered in shared memory so that each column leaves as one run of 64 bytes.
template <bool F32>
struct BothSmem {
    uint32_t tile[2][128 * 64];
    uint8_t out[256 / Piece<F32>::ES * 80];  // 64 bytes of codes a column, pitch 80
    uint32_t sc[256 / Piece<F32>::ES];
};

template <bool F32>
__global__ void __launch_bounds__(256) quantize_both_kernel(const QuantArgs a) {
    using P = Piece<F32>;
    constexpr int TC = 256 / P::ES;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    BothSmem<F32>& sm = *reinterpret_cast<BothSmem<F32>*>(smem_raw);
    const int t = threadIdx.x, lane16 = t & 15;
    const long long total = static_cast<long long>(a.cols) * a.p;
    const long long k_tiles = (total + 127) / 128, pitch = (total + 31) / 32 * 16;
    const long long t_pitch = (static_cast<long long>(a.rows) + 31) / 32 * 16, t_tiles = (static_cast<long long>(a.rows) + 127) / 128;
    const unsigned col_tiles = static_cast<unsigned>(a.spans);
    griddep_wait();
    if (t == 0) griddep_launch_dependents();

    auto fetch = [&](unsigned item, uint32_t* dst) {
        const unsigned rt = item / col_tiles;
        const long long c0 = static_cast<long long>(item - rt * col_tiles) * TC + lane16 * P::E;
        int n;
        const uint8_t* src = piece_at<F32>(a, c0, n);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = (t >> 4) + i * 16;
            const long long row = static_cast<long long>(rt) * 128 + r;
            const uint32_t bytes = row < a.rows ? n * P::ES : 0;  // the rest of the 16 are zero-filled, not read
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst + r * 64 + lane16 * 4)),
                         "l"(bytes ? src + row * a.ldx : a.x), "r"(bytes)
                         : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    unsigned item = blockIdx.x;
    const unsigned items = static_cast<unsigned>(a.items);
    int buf = 0;
    if (item < items) fetch(item, sm.tile[0]);
    for (; item < items; item += gridDim.x, buf ^= 1) {
        if (item + gridDim.x < items) {
            fetch(item + gridDim.x, sm.tile[buf ^ 1]);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const uint32_t* tile = sm.tile[buf];
        const unsigned rt = item / col_tiles;
        const long long c_tile = static_cast<long long>(item - rt * col_tiles) * TC, r_tile = static_cast<long long>(rt) * 128;
        if (a.q != nullptr) {
            const long long c0 = c_tile + lane16 * P::E;
            uint8_t* qd = a.q + r_tile * pitch + c0 / 2;
            uint8_t* sd = a.s + mx::scale_offset(r_tile, c0 >> 5, k_tiles);
            const bool put = c0 / 2 < pitch;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = (t >> 4) + i * 16;
                const uint4 v = *reinterpret_cast<const uint4*>(tile + r * 64 + lane16 * 4);
                const uint32_t s = P::scale(v);
                const uint32_t code = P::codes(v, s);
                if (r_tile + r < a.rows) {
                    if (put) {
                        if constexpr (F32) *reinterpret_cast<uint16_t*>(qd + r * pitch) = static_cast<uint16_t>(code);
                        else *reinterpret_cast<uint32_t*>(qd + r * pitch) = code;
                    }
                    // (col_tiles cover whole scale tiles: padding blocks are written as zero)
                    if (lane16 % P::LANES == 0) sd[(r & 31) * 16 + (r >> 5) * 4] = static_cast<uint8_t>(s);
                }
            }
        }
        {
            const int word = t & 63, rb = t >> 6;
            const uint32_t* col = tile + rb * 32 * 64 + word;
            uint8_t* sb = reinterpret_cast<uint8_t*>(sm.sc);
            if constexpr (F32) {
                float v[32];
#pragma unroll
                for (int r = 0; r < 32; ++r) v[r] = __uint_as_float(col[r * 64]);
                uint4 c;
                sb[word * 4 + rb] = static_cast<uint8_t>(mx::quantize32(v, c));
                *reinterpret_cast<uint4*>(sm.out + word * 80 + rb * 16) = c;
            } else {
                uint32_t w[32];
#pragma unroll
                for (int r = 0; r < 32; ++r) w[r] = col[r * 64];
                uint32_t m[4] = {w[0], w[1], w[2], w[3]};
#pragma unroll
                for (int r = 4; r < 32; ++r) m[r & 3] = mx::amax_bf16x2(m[r & 3], w[r]);
                const uint32_t mm = mx::amax_bf16x2(mx::amax_bf16x2(m[0], m[1]), mx::amax_bf16x2(m[2], m[3])) & 0x7FFF7FFFu;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t s = mx::scale_of(half ? (mm & 0xFFFF0000u) : (mm << 16));
                    const float inv = mx::inverse_scale(s);
                    uint32_t c[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            v[i] = __uint_as_float(half ? (w[g * 8 + i] & 0xFFFF0000u) : (w[g * 8 + i] << 16));
#pragma unroll
                        for (int i = 0; i < 8; i += 2) mx::mul2(v[i], v[i + 1], inv);
                        c[g] = s == 255u ? 0u : mx::encode8(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
                    }
                    *reinterpret_cast<uint4*>(sm.out + (word * 2 + half) * 80 + rb * 16) = make_uint4(c[0], c[1], c[2], c[3]);
                    sb[(word * 2 + half) * 4 + rb] = static_cast<uint8_t>(s);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TC / 64; ++i) {
            const int c = (t >> 2) + i * 64;
            const long long col = c_tile + c, at = r_tile / 2 + (t & 3) * 16;
            if (col < total && at < t_pitch)
                *reinterpret_cast<uint4*>(a.qt + col * t_pitch + at) =
                    *reinterpret_cast<const uint4*>(sm.out + c * 80 + (t & 3) * 16);
        }
        if (t < TC && c_tile + t < total)
            *reinterpret_cast<uint32_t*>(a.st + mx::scale_offset(c_tile + t, rt * 4LL, t_tiles)) = sm.sc[t];
        // (the next pass writes out and sc behind its first barrier, and this buffer's copies start there too)
    }
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
tpmlp_status launch_pdl(const char* what, void (*kern)(P...), dim3 grid, int smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
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

template <bool F32>
tpmlp_status quantize(QuantArgs a, int64_t cols, const DeviceInfo& dev, cudaStream_t st) {
    constexpr int E = Piece<F32>::E;
    if (a.qt == nullptr) {
        a.spans = (cols + 32 * E - 1) / (32 * E);
        if constexpr (F32) a.spans = (cols + 127) / 128;  // one span is one scale tile wide
        a.items = a.spans * a.rows;
        // Four spans a warp keep 2 KB of loads in flight; while there are fewer warps than that fills
        // the GPU with, one each.
        const bool many = a.items >= static_cast<int64_t>(dev.sm_count) * 64 * 4;
        const int64_t per = many ? 32 : 8;
        const dim3 grid(static_cast<unsigned>((a.items + per - 1) / per));
        return many ? launch_pdl("MXFP4 quantisation", quantize_rows_kernel<F32, 4>, grid, 0, st, a)
                    : launch_pdl("MXFP4 quantisation", quantize_rows_kernel<F32, 1>, grid, 0, st, a);
    }
    constexpr int TC = 256 / Piece<F32>::ES;
    a.spans = (cols + 127) / 128 * (128 / TC);
    a.items = a.spans * ((a.rows + 127LL) / 128);
    static bool attr_done[64];
    constexpr int smem = sizeof(BothSmem<F32>);
    if (dev.device >= 64 || !attr_done[dev.device]) {
        const cudaError_t e = cudaFuncSetAttribute(quantize_both_kernel<F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) {
            set_error("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
            return TPMLP_ERR_CUDA;
        }
        if (dev.device < 64) attr_done[dev.device] = true;
    }
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.items, dev.sm_count * 2)));
    return launch_pdl("MXFP4 quantisation", quantize_both_kernel<F32>, grid, smem, st, a);
}

}  // namespace

tpmlp_status launch_mxfp4_quantize(const void* X, int64_t ldx, void* Q, void* S, void* Qt, void* St, int64_t rows,
                                   int64_t cols, int p, bool f32, const DeviceInfo& dev, cudaStream_t st) {
    const int64_t es = f32 ? 4 : 2;
    const QuantArgs a{static_cast<const uint8_t*>(X), ldx * es, rows * ldx * es, static_cast<int>(rows),
                      static_cast<int>(cols / p), p, static_cast<uint8_t*>(Q), static_cast<uint8_t*>(S),
                      static_cast<uint8_t*>(Qt), static_cast<uint8_t*>(St), 0, 0};
    return f32 ? quantize<true>(a, cols, dev, st) : quantize<false>(a, cols, dev, st);
}

tpmlp_status launch_mxfp4_dequantize(const void* Q, const void* S, void* out, int64_t rows, int64_t k, bool f32,
                                     const DeviceInfo& dev, cudaStream_t st) {
    const int64_t items = rows * ((k + 7) / 8);
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((items + 255) / 256, static_cast<int64_t>(dev.sm_count) * 32)));
    const auto* q = static_cast<const uint8_t*>(Q);
    const auto* s = static_cast<const uint8_t*>(S);
    return f32 ? launch_pdl("MXFP4 dequantisation", dequantize_kernel<true>, grid, 0, st, q, s, out, (long long)rows, (long long)k)
               : launch_pdl("MXFP4 dequantisation", dequantize_kernel<false>, grid, 0, st, q, s, out, (long long)rows, (long long)k);
}

}  // namespace tpmlp
