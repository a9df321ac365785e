// MXFP4 quantisation along either axis, or both from one read, and its inverse.
#include <cuda_runtime.h>

#include <type_traits>

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
    float* sums;        // sums over blocks of 32 rows [ceil(rows/32)][p * cols]
    long long spans;    // row kernel: warp spans of a row; tile kernel: column tiles
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

// Along the columns of a few rows: a warp takes a span of 512 bytes of a row, a 16-byte piece a lane.  A
// block's maximum takes 2 (bf16) or 3 (fp32) shuffles; its codes go out 4 (2) bytes a lane.  Bound by the
// launch (one token of 5120: 1.2 us in a graph).
template <bool F32>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantArgs a) {
    using P = Piece<F32>;
    constexpr int SPAN = 32 * P::E;
    const int lane = threadIdx.x & 31;
    const long long total = static_cast<long long>(a.cols) * a.p;
    const long long k_tiles = (total + 127) / 128, pitch = (total + 31) / 32 * 16;
    const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const long long row = item / a.spans, c0 = (item - row * a.spans) * SPAN + lane * P::E;
    int n;
    const uint8_t* src = piece_at<F32>(a, c0, n);
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    if (row >= a.rows) return;
    const uint4 v = P::load(src + row * a.ldx, n);
    const uint32_t s = P::scale(v);
    const uint32_t code = P::codes(v, s);
    if (c0 / 2 < pitch) {
        uint8_t* d = a.q + row * pitch + c0 / 2;
        if constexpr (F32) *reinterpret_cast<uint16_t*>(d) = static_cast<uint16_t>(code);
        else *reinterpret_cast<uint32_t*>(d) = code;
    }
    // (padding blocks up to a whole scale tile: zero)
    if (lane % P::LANES == 0 && c0 < k_tiles * 128) a.s[mx::scale_offset(row, c0 >> 5, k_tiles)] = static_cast<uint8_t>(s);
}

// Along the columns, the rows (ACROSS) or both.  A CTA takes a tile of 128 rows x 256 bytes of columns (128
// bf16, 64 fp32), 16 lanes to a row.  ACROSS: asynchronous copies bring it to shared memory, both
// quantisations work from there, and the other four CTAs of the SM cover its latency; along the rows a
// thread takes 32 rows of one word (two bf16 columns or one fp32 column), and the codes are gathered in
// shared memory so that each column leaves as one run of 64 bytes.  The values are read from memory once.
// 8192 x 5120 bf16: along the columns 18.3 us (5.8 TB/s, 85 % of a copy's), along the rows 17.3, both 25.0
// (5.1 TB/s; there issue slots and memory bind about equally).
template <bool F32>
struct BothSmem {
    uint32_t tile[128 * 64];
    uint8_t out[256 / Piece<F32>::ES * 80];  // 64 bytes of codes a column, pitch 80
    uint32_t sc[256 / Piece<F32>::ES];
};

// SUMS (bf16 ACROSS): also a.sums.
template <bool F32, bool ACROSS, bool SUMS>
__device__ __forceinline__ void quantize_tile(const QuantArgs& a, std::conditional_t<ACROSS, BothSmem<F32>, uint4>& sm) {
    using P = Piece<F32>;
    constexpr int TC = 256 / P::ES;
    const int t = threadIdx.x, lane16 = t & 15, r0 = t >> 4;
    const long long total = static_cast<long long>(a.cols) * a.p;
    const unsigned col_tiles = static_cast<unsigned>(a.spans);
    const unsigned rt = blockIdx.x / col_tiles;
    const long long c_tile = static_cast<long long>(blockIdx.x - rt * col_tiles) * TC, r_tile = static_cast<long long>(rt) * 128;
    const long long c0 = c_tile + lane16 * P::E;
    const int rows = static_cast<int>(a.rows - r_tile < 128 ? a.rows - r_tile : 128);  // of this tile
    griddep_wait();
    if (t == 0) griddep_launch_dependents();
    [[maybe_unused]] uint4 piece[8];
    if constexpr (!ACROSS) {
        int n;
        const uint8_t* src = piece_at<F32>(a, c0, n) + (r_tile + r0) * a.ldx;
        if (n == P::E) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                piece[i] = make_uint4(0, 0, 0, 0);
                if (r0 + i * 16 < rows) piece[i] = *reinterpret_cast<const uint4*>(src + i * 16 * a.ldx);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) piece[i] = P::load(src + i * 16 * a.ldx, r0 + i * 16 < rows ? n : 0);
        }
    } else {
        int n;
        const uint8_t* src = piece_at<F32>(a, c0, n) + (r_tile + r0) * a.ldx;
        uint32_t dst = smem_u32(sm.tile + r0 * 64 + lane16 * 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t bytes = r0 + i * 16 < rows ? n * P::ES : 0;  // the rest of the 16 are zero-filled, not read
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * 4096), "l"(bytes ? src : a.x), "r"(bytes)
                         : "memory");
            src += 16 * a.ldx;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
    }
    if (a.q != nullptr) {
        const long long k_tiles = (total + 127) / 128, pitch = (total + 31) / 32 * 16;
        uint8_t* qd = a.q + (r_tile + r0) * pitch + c0 / 2;
        // (r0 < 16: rows r0 + 16 i of a scale tile are constant distances apart)
        uint8_t* sd = a.s + mx::scale_offset(r_tile + r0, c0 >> 5, k_tiles);
        const bool put = c0 / 2 < pitch;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint4 v;
            if constexpr (ACROSS) v = *reinterpret_cast<const uint4*>(sm.tile + (r0 + i * 16) * 64 + lane16 * 4);
            else v = piece[i];
            const uint32_t s = P::scale(v);
            const uint32_t code = P::codes(v, s);
            if (r0 + i * 16 < rows) {
                if (put) {
                    if constexpr (F32) *reinterpret_cast<uint16_t*>(qd) = static_cast<uint16_t>(code);
                    else *reinterpret_cast<uint32_t*>(qd) = code;
                }
            }
            // (whole scale tiles: the scales of padding blocks and rows are written as zero; no product reads those of
            // padding rows but the gated backward's dY, whose epilogue wants them finite)
            if (lane16 % P::LANES == 0) sd[(i & 1) * 256 + (i >> 1) * 4] = static_cast<uint8_t>(s);
            qd += 16 * pitch;
        }
    }
    if constexpr (ACROSS) {
        {
            const int word = t & 63, rb = t >> 6;
            const uint32_t* col = sm.tile + rb * 32 * 64 + word;
            uint8_t* sb = reinterpret_cast<uint8_t*>(sm.sc);
            if constexpr (F32) {
                float v[32];
#pragma unroll
                for (int r = 0; r < 32; ++r) v[r] = __uint_as_float(col[r * 64]);
                uint4 c;
                sb[word * 4 + rb] = static_cast<uint8_t>(mx::quantize32(v, c));
                *reinterpret_cast<uint4*>(sm.out + word * 80 + rb * 16) = c;
            } else {
                // (the values are read twice, so that a CTA's registers leave room for five)
                uint32_t m[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) m[r] = mx::amax_bf16x2(col[r * 64], col[(r + 4) * 64]);
#pragma unroll
                for (int r = 8; r < 32; ++r) m[r & 3] = mx::amax_bf16x2(m[r & 3], col[r * 64]);
                const uint32_t mm = mx::amax_bf16x2(mx::amax_bf16x2(m[0], m[1]), mx::amax_bf16x2(m[2], m[3])) & 0x7FFF7FFFu;
                const uint32_t s0 = mx::scale_of(mm << 16), s1 = mx::scale_of(mm & 0xFFFF0000u);
                const float inv0 = mx::inverse_scale(s0), inv1 = mx::inverse_scale(s1);
                uint32_t c0w[4], c1w[4];
                [[maybe_unused]] float x0 = 0.0f, x1 = 0.0f;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float lo[8], hi[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t w = col[(g * 8 + i) * 64];
                        lo[i] = __uint_as_float(w << 16);
                        hi[i] = __uint_as_float(w & 0xFFFF0000u);
                        if constexpr (SUMS) {
                            x0 += lo[i];
                            x1 += hi[i];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        mx::mul2(lo[i], lo[i + 1], inv0);
                        mx::mul2(hi[i], hi[i + 1], inv1);
                    }
                    c0w[g] = s0 == 255u ? 0u : mx::encode8(lo[0], lo[1], lo[2], lo[3], lo[4], lo[5], lo[6], lo[7]);
                    c1w[g] = s1 == 255u ? 0u : mx::encode8(hi[0], hi[1], hi[2], hi[3], hi[4], hi[5], hi[6], hi[7]);
                }
                uint8_t* o = sm.out + word * 160 + rb * 16;
                *reinterpret_cast<uint4*>(o) = make_uint4(c0w[0], c0w[1], c0w[2], c0w[3]);
                *reinterpret_cast<uint4*>(o + 80) = make_uint4(c1w[0], c1w[1], c1w[2], c1w[3]);
                sb[word * 8 + rb] = static_cast<uint8_t>(s0);
                sb[word * 8 + 4 + rb] = static_cast<uint8_t>(s1);
                if (SUMS && rb * 32 < rows) {
                    float* d = a.sums + (rt * 4LL + rb) * total + c_tile + word * 2;
                    if (c_tile + word * 2 < total) d[0] = x0;
                    if (c_tile + word * 2 + 1 < total) d[1] = x1;
                }
            }
        }
        __syncthreads();
        const long long t_pitch = (static_cast<long long>(a.rows) + 31) / 32 * 16, t_tiles = (static_cast<long long>(a.rows) + 127) / 128;
#pragma unroll
        for (int i = 0; i < TC / 64; ++i) {
            const int c = (t >> 2) + i * 64;
            const long long col = c_tile + c, at = r_tile / 2 + (t & 3) * 16;
            if (col < total && at < t_pitch)
                *reinterpret_cast<uint4*>(a.qt + col * t_pitch + at) = *reinterpret_cast<const uint4*>(sm.out + c * 80 + (t & 3) * 16);
        }
        if (t < TC && c_tile + t < total)
            *reinterpret_cast<uint32_t*>(a.st + mx::scale_offset(c_tile + t, rt * 4LL, t_tiles)) = sm.sc[t];
    }
}

template <bool F32, bool ACROSS>
__global__ void __launch_bounds__(256, ACROSS ? 5 : 4) quantize_tile_kernel(const QuantArgs a) {
    __shared__ __align__(16) std::conditional_t<ACROSS, BothSmem<F32>, uint4> sm;
    quantize_tile<F32, ACROSS, false>(a, sm);
}

// Two bf16 matrices of one shape, along the rows and where wanted the columns, the first with sums where wanted.
struct QuantPair {
    QuantArgs of[2];
};
__global__ void __launch_bounds__(256, 5) quantize_pair_kernel(const __grid_constant__ QuantPair a) {
    __shared__ __align__(16) BothSmem<false> sm;
    const QuantArgs& m = a.of[blockIdx.y];
    if (m.sums != nullptr) quantize_tile<false, true, true>(m, sm);
    else quantize_tile<false, true, false>(m, sm);
}

// The column sums where no kernel of CTA pairs takes them along.
__global__ void __launch_bounds__(256) finish_sums_kernel(const mx::SumsArgs a) {
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int item = static_cast<int>(blockIdx.x * 8 + (threadIdx.x >> 5));
    if (item < a.items) mx::sum_columns(a, item, threadIdx.x & 31);
}

// Values of an operand: a warp takes U spans of 32 words (256 values) of a row, a word of eight codes a
// lane, all loaded before the first is worked on.  Ordinary loads: the quantiser ahead may still be writing q and s when
// this kernel becomes resident, which a non-coherent load does not allow.
template <bool F32, int U>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t* q, const uint8_t* s, void* out, long long rows,
                                                         long long k, long long spans) {
    const int lane = threadIdx.x & 31;
    const long long pitch = (k + 31) / 32 * 16, k_tiles = (k + 127) / 128, words = (k + 7) / 8;
    const long long it0 = (static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * U;
    long long row = it0 / spans, span = it0 - row * spans;
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    uint32_t c[U], sb[U];
    long long rw[U], w[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        rw[i] = row;
        w[i] = row < rows ? span * 32 + lane : words;
        if (w[i] < words) {
            c[i] = reinterpret_cast<const uint32_t*>(q + row * pitch)[w[i]];
            sb[i] = s[mx::scale_offset(row, w[i] >> 2, k_tiles)];
        }
        if (++span == spans) {
            span = 0;
            ++row;
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (w[i] >= words) continue;
        const float sv = mx::scale_value(sb[i]);
        float v[8];
        mx::decode8(c[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= sv;
        const long long at = rw[i] * k + w[i] * 8;
        if constexpr (F32) {
            float* d = static_cast<float*>(out) + at;
            if (k % 4 == 0 && w[i] * 8 + 8 <= k) {
                *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4*>(d + 4) = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                for (int j = 0; j < 8 && w[i] * 8 + j < k; ++j) d[j] = v[j];
            }
        } else {
            __nv_bfloat16* d = static_cast<__nv_bfloat16*>(out) + at;
            if (k % 8 == 0) {
                __nv_bfloat162 b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(b);
            } else {
                for (int j = 0; j < 8 && w[i] * 8 + j < k; ++j) d[j] = __float2bfloat16_rn(v[j]);
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

template <bool F32>
dim3 tile_grid(QuantArgs& a, int64_t cols) {
    constexpr int TC = 256 / Piece<F32>::ES;
    a.spans = (cols + 127) / 128 * (128 / TC);
    return dim3(static_cast<unsigned>(a.spans * ((a.rows + 127LL) / 128)));
}

template <bool F32>
tpmlp_status quantize(QuantArgs a, int64_t cols, cudaStream_t st) {
    const char* what = "MXFP4 quantisation";
    // Along the columns, few values: a span a warp spreads them over more warps than tiles of 128 rows do (bf16, 1 x
    // 5120 1.2 us against 1.6, 128 x 5120 1.6 against 2.2, 2048 x 1024 2.3 both, 8192 x 5120 32 against 18).
    if (a.qt == nullptr && a.rows * cols < (1 << 21)) {
        a.spans = F32 ? (cols + 127) / 128 : (cols + 255) / 256;  // of 512 bytes, whole scale tiles
        return launch_pdl(what, quantize_rows_kernel<F32>, dim3(static_cast<unsigned>((a.spans * a.rows + 7) / 8)), st, a);
    }
    const dim3 grid = tile_grid<F32>(a, cols);
    return a.qt == nullptr ? launch_pdl(what, quantize_tile_kernel<F32, false>, grid, st, a)
                           : launch_pdl(what, quantize_tile_kernel<F32, true>, grid, st, a);
}

QuantArgs quant_args(const void* X, int64_t ldx, void* Q, void* S, void* Qt, void* St, int64_t rows, int64_t cols, int p, int64_t es,
                     float* sums) {
    return {static_cast<const uint8_t*>(X), ldx * es, rows * ldx * es, static_cast<int>(rows), static_cast<int>(cols / p), p,
            static_cast<uint8_t*>(Q), static_cast<uint8_t*>(S), static_cast<uint8_t*>(Qt), static_cast<uint8_t*>(St), sums, 0};
}

}  // namespace

tpmlp_status launch_mxfp4_quantize(const void* X, int64_t ldx, void* Q, void* S, void* Qt, void* St, int64_t rows, int64_t cols,
                                   int p, bool f32, cudaStream_t st) {
    const QuantArgs a = quant_args(X, ldx, Q, S, Qt, St, rows, cols, p, f32 ? 4 : 2, nullptr);
    return f32 ? quantize<true>(a, cols, st) : quantize<false>(a, cols, st);
}

tpmlp_status launch_mxfp4_quantize_bwd(const void* dZ, void* Q, void* S, void* Qt, void* St, float* sums, const void* X, void* Xt,
                                       void* XSt, int64_t rows, int64_t cols, cudaStream_t st) {
    QuantPair a{{quant_args(dZ, cols, Q, S, Qt, St, rows, cols, 1, 2, sums),
                 quant_args(X, cols, nullptr, nullptr, Xt, XSt, rows, cols, 1, 2, nullptr)}};
    dim3 grid = tile_grid<false>(a.of[0], cols);
    a.of[1].spans = a.of[0].spans;
    grid.y = 2;
    return launch_pdl("MXFP4 quantisation", quantize_pair_kernel, grid, st, a);
}

tpmlp_status launch_mxfp4_sums(const mx::SumsArgs& a, cudaStream_t st) {
    return launch_pdl("column sums", finish_sums_kernel, dim3(static_cast<unsigned>((a.items + 7) / 8)), st, a);
}

tpmlp_status launch_mxfp4_dequantize(const void* Q, const void* S, void* out, int64_t rows, int64_t k, bool f32,
                                     const DeviceInfo& dev, cudaStream_t st) {
    const int64_t spans = (k + 255) / 256, items = rows * spans;
    // four spans a warp where every SM then has its 64 warps full
    const bool many = items >= static_cast<int64_t>(dev.sm_count) * 64 * 4;
    const int64_t per = many ? 32 : 8;
    const dim3 grid(static_cast<unsigned>((items + per - 1) / per));
    const auto* q = static_cast<const uint8_t*>(Q);
    const auto* s = static_cast<const uint8_t*>(S);
    const long long r = rows, kk = k, sp = spans;
    const char* what = "MXFP4 dequantisation";
    if (f32)
        return many ? launch_pdl(what, dequantize_kernel<true, 4>, grid, st, q, s, out, r, kk, sp)
                    : launch_pdl(what, dequantize_kernel<true, 1>, grid, st, q, s, out, r, kk, sp);
    return many ? launch_pdl(what, dequantize_kernel<false, 4>, grid, st, q, s, out, r, kk, sp)
                : launch_pdl(what, dequantize_kernel<false, 1>, grid, st, q, s, out, r, kk, sp);
}

}  // namespace tpmlp
