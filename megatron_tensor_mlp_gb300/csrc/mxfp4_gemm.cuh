// D[M,N] = sum_k A[M,k] B[N,k] on MXFP4 operands: block-scaled tcgen05.mma (kind::mxf4, 4-bit
// elements, one E8M0 scale per 32 along k, fp32 accumulators in tensor memory), fed by TMA, with
// the epilogues of the gated feed-forward block fused.
//
// One instruction contracts 64 values of k: 32 bytes of a row, the bytes (and the tensor-core
// cycles) of a 16-deep bf16 instruction, so the pipeline has the shape of the bf16 GEMM's at a
// quarter of the K loop.  A ring stage is 256 values of k: 128-byte rows of codes (K-major,
// 128-byte swizzle) and the scale tiles (128 rows x 4 blocks, 512 bytes) of the same rows, which
// tcgen05.cp copies to tensor memory ahead of the stage's MMAs.  Copies and MMAs of one thread
// execute in issue order, so all stages share one place for their scales.
//
// Two kernels:
//   mx_pair_kernel    CTA pairs (cta_group::2), 256x256 tiles, persistent.  Two 256-column
//                     accumulators and 24 columns of scales do not fit 512 tensor-memory columns,
//                     so the accumulators share 32: [0,256) and [224,480), scales from 480.  Each
//                     epilogue reads the shared columns first and reports them free; the next
//                     tile's MMAs start then, beside the rest of the epilogue.  Several independent
//                     products can share a launch (Problems).
//                     The tensor pipe binds first and, over milliseconds, the power cap: 8192 x 20480 x
//                     5120 takes 218 us (7.9 PFLOP/s) cold and 248 us (6.9) at the cap's 1.6 GHz.  At
//                     4096 x 8192 x 5120 the pipe is busy for 83 % of active cycles, L2 for 47 % and the way
//                     from it to the SMs for 40 % (70 KB a stage and pair in 512 tensor cycles).  The
//                     instruction's 96-deep form, half as fast again, has not been tried: a stage's 256 k
//                     and blocks of 32 do not divide into it, and at the cap it is power that binds.
//   mx_single_kernel  one CTA per 128x128 tile (128 rows of A, 128 of B; for the gated forward 64
//                     gate and 64 up columns), two CTAs an SM, not persistent: for few rows, where
//                     reading B's codes bounds the time, and for GEMMs of few tiles.  Clusters of
//                     up to 8 CTAs split the K loop and add their partial sums through distributed
//                     shared memory in a fixed order.  With at most 64 rows of A only those rows
//                     are copied: the MMA's other rows read whatever lies behind them in shared
//                     memory, and their results are not stored.  1 x 5120 x 20480, weights from
//                     memory: 14 us, of which 8.2 us are its 56 MB at a copy's rate and 5 us a launch's
//                     chain of latencies; 4 x 40960 x 5120 23 us (16.4).
//
// Every wait on an mbarrier is bounded (a status word records a timeout); no TMA load uses
// cluster multicast.
#pragma once
#include "gemm_tc.cuh"
#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace mx {

constexpr int BM = 128;           // rows of A (and of B) in one CTA's stage
constexpr int KC = 256;           // k per ring stage: 128 bytes of codes a row
constexpr int OP_BYTES = BM * 128;
constexpr int SF_TILE = 512;      // scales of 128 rows x 128 k
constexpr int GROUP_M = 16;       // pair kernel: row blocks walked together (4 to 32 within 1 % of one another)

struct Args {
    int M, N;
    int kb;          // ring stages of K: ceil(K / 256)
    int last_steps;  // MMAs (64 k each) of the last one: 1..4
    int m_blocks, n_blocks;  // tiles
    int a_box;       // single kernel: rows of A copied per stage (16, 32, 64 or 128)
    int stages;      // single kernel: ring stages
    int prefetch_b;  // single kernel: B's first stages into L2 while the kernel ahead in the stream ends (B not blocked)
    int a_blocked, b_blocked;  // operand's codes are [k / 32][rows][16 bytes] (written by an epilogue), not [rows][k / 2]
    int out_f32, st32;
    // EPI_STORE: D + bias; column n is at out + (n / shard_cols) * out_ss + m * out_ld + n % shard_cols
    void* out; long long out_ld, out_ss; int shard_cols;
    const __nv_bfloat16* bias;   // EPI_STORE [N], EPI_SWIGLU [N] packed
    // EPI_SWIGLU: h_out (optional) [M][2 ffn]; EPI_DSWIGLU: h_in
    const __nv_bfloat16* h_in; __nv_bfloat16* h_out; long long h_ld;
    // quantised outputs, codes blocked: along the columns EPI_SWIGLU y [M][ffn], EPI_DSWIGLU dH [M][2 ffn]
    uint4* q; uint8_t* qs; long long q_tiles;
    // EPI_DSWIGLU: along the rows (tokens), dH^T [2 ffn][M] and Y^T [ffn][M]
    uint4* ht; uint8_t* hts; uint4* yt; uint8_t* yts; long long t_blocks, t_tiles;
    float* colsum;   // EPI_DSWIGLU, optional: sums of dH over blocks of 32 tokens [ceil(M/32)][2 ffn]
    uint32_t* status;
    unsigned long long timeout_ns;
};

// ---------------------------------------------------------------- tcgen05, block scaled
// Instruction descriptor, kind::mxf4: bits 4-5 B scale id, 7-9 A format (1 = E2M1), 10-12 B
// format, 17-22 N >> 3, 23 scale format (1 = E8M0), 24-28 M >> 4, 29-30 A scale id.  The scale id
// names the byte of the scale columns' 32-bit words that the instruction starts from: 0 for the
// first 64 k of a scale tile, 2 for the second.
__host__ __device__ constexpr uint32_t idesc_mxf4(int m, int n, uint32_t sf_id) {
    return (sf_id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(m >> 4) << 24) | (sf_id << 29);
}
// Shared-memory descriptor of `rows` rows of blocked codes (K-major without swizzle): 8-row groups of 16
// bytes a row 128 bytes apart, the next 16 bytes of k a block of all rows further.
__device__ __forceinline__ uint64_t sdesc_blocked(uint32_t saddr, int rows) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(rows) << 16) |
           (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}
// Shared-memory descriptor of a scale tile for tcgen05.cp: no swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) |
           (static_cast<uint64_t>(1) << 46);
}
template <int CG>
__device__ __forceinline__ void umma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}
// One scale tile (512 bytes) to 4 tensor-memory columns, the same 32 rows for every lane quarter.
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (CG == 2) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// ---------------------------------------------------------------- epilogues
// (Biases are read by ordinary loads: the kernel ahead in the stream may write them while this one is resident, which
// a non-coherent load does not allow.)
// EPI_STORE: 32 consecutive columns of a row.
__device__ __forceinline__ void store_chunk(const Args& p, float (&v)[32], int gm, int gn0) {
    const int nvalid = p.N - gn0;
    if (gm >= p.M || nvalid <= 0) return;
    if (p.bias != nullptr) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const __nv_bfloat16* bp = p.bias + gn0 + g * 8;
            if ((g + 1) * 8 <= nvalid) {
                float b[8];
                tc::unpack_bf16x8(*reinterpret_cast<const uint4*>(bp), b);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[g * 8 + i] += b[i];
            } else if (g * 8 < nvalid) {  // fp32 rows may end on a multiple of 4
#pragma unroll
                for (int i = 0; i < 4; ++i) v[g * 8 + i] += __bfloat162float(bp[i]);
            }
        }
    }
    const int sh = gn0 / p.shard_cols;
    const long long at = sh * p.out_ss + gm * p.out_ld + (gn0 - sh * p.shard_cols);
    if (p.out_f32) tc::store_f32x32(static_cast<float*>(p.out) + at, v, nvalid, p.st32 != 0);
    else tc::store_bf16x32(static_cast<__nv_bfloat16*>(p.out) + at, v, nvalid, p.st32 != 0);
}

// Two fp32 values in one register pair: sums and products of both in one instruction.
using f2 = unsigned long long;
// sigma(x) = 1 / (1 + 2^(-x log2 e)) with the hardware approximations.
__device__ __forceinline__ f2 sigmoid2(f2 x) {
    float a, b;
    tc::f2_unpack(tc::f2_mul(x, tc::f2_pack(-1.4426950408889634f, -1.4426950408889634f)), a, b);
    tc::f2_unpack(tc::f2_add(tc::f2_pack(tc::ex2_approx(a), tc::ex2_approx(b)), tc::f2_pack(1.0f, 1.0f)), a, b);
    return tc::f2_pack(tc::rcp_approx(a), tc::rcp_approx(b));
}

// EPI_SWIGLU: y = silu(g) u for features f0..f0+31 of a row (one block), quantised from fp32.
// Returns the block's scale byte.
__device__ __forceinline__ uint32_t swiglu_chunk(const Args& p, float (&g)[32], float (&u)[32], int gm, int f0) {
    if (gm >= p.M || 2 * f0 >= p.N) return 0;
    const long long pg = (long long)(f0 >> 7) * 256 + (f0 & 127);
    if (p.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float bg[8], bu[8];
            tc::unpack_bf16x8(*reinterpret_cast<const uint4*>(p.bias + pg + j * 8), bg);
            tc::unpack_bf16x8(*reinterpret_cast<const uint4*>(p.bias + pg + 128 + j * 8), bu);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                g[j * 8 + i] += bg[i];
                u[j * 8 + i] += bu[i];
            }
        }
    }
    if (p.h_out != nullptr) {
        __nv_bfloat16* d = p.h_out + gm * p.h_ld + pg;
        tc::store_bf16x32(d, g, 32, p.st32 != 0);
        tc::store_bf16x32(d + 128, u, 32, p.st32 != 0);
    }
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const f2 x = tc::f2_pack(g[j], g[j + 1]);
        tc::f2_unpack(tc::f2_mul(tc::f2_mul(x, sigmoid2(x)), tc::f2_pack(u[j], u[j + 1])), g[j], g[j + 1]);
    }
    uint4 c;
    const uint32_t s = quantize32(g, c);
    p.q[(long long)(f0 >> 5) * p.M + gm] = c;  // a warp's 32 rows: 512 bytes in a row
    return s;
}

// A warp's 32 x 32 values, a row in each lane, turned so that each lane has a column.  buf: 4 KB of
// this warp's; a row's eight 16-byte groups are permuted by the row's low bits, which keeps both passes
// free of bank conflicts without padding.
constexpr int TURN_WORDS = 32 * 32;
__device__ __forceinline__ void turn32(float* buf, const float (&v)[32], float (&w)[32], int lane) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4*>(buf + lane * 32 + 4 * (j ^ (lane & 7))) =
            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    __syncwarp();
#pragma unroll
    for (int t = 0; t < 32; ++t) w[t] = buf[t * 32 + 4 * ((lane >> 2) ^ (t & 7)) + (lane & 3)];
    __syncwarp();
}

// EPI_DSWIGLU, 4096 tokens, h5120, ffn20480: 195 us against 130 for the product alone (before the power cap); the
// epilogue binds, a tile's arithmetic and its shared-memory traffic taking twice the MMAs' time.  Turning the three
// arrays costs 48 us of it, the row-wise blocks 25, the activation 19, the stores 10.  Twelve epilogue warps
// that turn half blocks took 266 us.
//
// EPI_DSWIGLU leaves five quantised arrays.  Their codes go out blocked, a warp's 32 blocks of 16 bytes
// as 512 bytes in a row.  (Row-major codes, 16 bytes a lane into 32 rows, kept the load/store unit busy for
// longer than the arithmetic; as TMA stores of 16 bytes x 32 rows they still cost 25 us of 910 in the
// backward of 4096 tokens, h5120, ffn20480.)  Their scales are gathered in shared memory: the 128 rows x
// 128 features of four warps (a CTA's half of a pair tile) are one scale tile of each array.
enum { SC_Y = 0, SC_G = 1, SC_U = 2, SC_ROW_G = 3, SC_ROW_U = 4, SC_ARRAYS = 5 };
constexpr int SC_BYTES = SC_ARRAYS * SF_TILE;
constexpr int H_BUF = 4096;  // pair kernel: a warp's 32 rows x 32 features of H, gate then up

// Writes the five tiles of a half (128 threads, all its chunks done): features f0..f0+127 of rows row0..row0+127.
// chunks: bit c set where this CTA did features 32 c.. (a split tile's CTAs share them).
__device__ __forceinline__ void put_scales(const Args& p, const uint8_t* sc, int row0, int f0, int thread, uint32_t chunks) {
    const long long k_tile = row0 >> 7, f_tile = f0 >> 7;
    if (f0 >= p.N || k_tile >= p.t_tiles) return;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(sc) + thread;
    // along the tokens: word i of a 16-byte group is features 32 i.., bytes the token blocks
    if (chunks >> (thread & 3) & 1u) {
        uint32_t* y = reinterpret_cast<uint32_t*>(p.yts + (f_tile * p.t_tiles + k_tile) * SF_TILE);
        uint32_t* h = reinterpret_cast<uint32_t*>(p.hts + (2 * f_tile * p.t_tiles + k_tile) * SF_TILE);
        y[thread] = w[SC_Y * 128];
        h[thread] = w[SC_G * 128];
        h[thread + p.t_tiles * 128] = w[SC_U * 128];
    }
    // along the features: word = row, byte c = features 32 c..
    uint32_t* r = reinterpret_cast<uint32_t*>(p.qs + (k_tile * p.q_tiles + 2 * f_tile) * SF_TILE);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        const uint32_t v = w[(SC_ROW_G + part) * 128];
        if (chunks == 15u) {
            r[thread + part * 128] = v;
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (chunks >> c & 1u) reinterpret_cast<uint8_t*>(r + thread + part * 128)[c] = static_cast<uint8_t>(v >> (8 * c));
        }
    }
}

// The saved bf16 pre-activations of features f0..f0+31 of row gm: 16 words of gate, 16 of up pairs;
// zero past the last row.
__device__ __forceinline__ void load_h(const Args& p, int gm, int f0, uint32_t (&h)[32]) {
    if (gm < p.M && f0 < p.N) {
        const __nv_bfloat16* hp = p.h_in + gm * p.h_ld + (long long)(f0 >> 7) * 256 + (f0 & 127);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            if (p.st32) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t w[8];
                    tc::ld_v8(hp + part * 128 + i * 16, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[part * 16 + i * 8 + j] = w[j];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 w = *reinterpret_cast<const uint4*>(hp + part * 128 + i * 8);
                    h[part * 16 + i * 4] = w.x;
                    h[part * 16 + i * 4 + 1] = w.y;
                    h[part * 16 + i * 4 + 2] = w.z;
                    h[part * 16 + i * 4 + 3] = w.w;
                }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) h[j] = 0;
    }
}

// The same from a warp's 32 rows x 32 features of H in shared memory (gate, then up; 64-byte swizzle).
__device__ __forceinline__ void read_h(const uint8_t* hb, int lane, uint32_t (&h)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(hb + (i >> 2) * 2048 + lane * 64 + (((i & 3) ^ ((lane >> 1) & 3)) << 4));
        h[i * 4] = w.x;
        h[i * 4 + 1] = w.y;
        h[i * 4 + 2] = w.z;
        h[i * 4 + 3] = w.w;
    }
}

// EPI_DSWIGLU: v = dY of features f0..f0+31 of this thread's row (token) and, from its pre-activations h,
// dg = dY u silu'(g), du = dY silu(g) and y = silu(g) u, from fp32 quantised along the columns (dg, du) and,
// turned through shared memory, along the tokens (dg, du, y).  tb: the warp's block of 32 tokens.  Rows past
// M are zero: their h is, and their dY is finite (the quantiser writes zero scales for dZ's rows up to a whole
// tile; a NaN there would need a select for every value, which cost 15 us of 770).  buf: turn32's; sc: the five scale tiles.
__device__ __forceinline__ void dswiglu_chunk(const Args& p, float (&v)[32], const uint32_t (&h)[32], int gm, int f0, int tb,
                                              float* buf, uint8_t* sc, int lane) {
    if (f0 >= p.N) return;  // (whole warp; features come in multiples of 128)
    const long long pg = (long long)(f0 >> 7) * 256 + (f0 & 127);
    const bool live = gm < p.M;
    const f2 one = tc::f2_pack(1.0f, 1.0f);
    float g[32], u[32];
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const f2 g2 = tc::f2_pack(__uint_as_float(h[j / 2] << 16), __uint_as_float(h[j / 2] & 0xFFFF0000u));
        const f2 u2 = tc::f2_pack(__uint_as_float(h[16 + j / 2] << 16), __uint_as_float(h[16 + j / 2] & 0xFFFF0000u));
        const f2 dy = tc::f2_pack(v[j], v[j + 1]);
        const f2 sg = sigmoid2(g2), sl = tc::f2_mul(g2, sg);
        const f2 ds = tc::f2_mul(sg, tc::f2_fma(g2, tc::f2_fma(sg, tc::f2_pack(-1.0f, -1.0f), one), one));  // silu'
        tc::f2_unpack(tc::f2_mul(tc::f2_mul(dy, u2), ds), g[j], g[j + 1]);
        tc::f2_unpack(tc::f2_mul(sl, u2), v[j], v[j + 1]);
        tc::f2_unpack(tc::f2_mul(dy, sl), u[j], u[j + 1]);
    }
    const bool blk = tb < p.t_blocks;     // the warp's block of tokens holds a row
    const int c = (f0 >> 5) & 3, q = tb & 3;
    uint8_t* by_token = sc + lane * 16 + c * 4 + q;  // scale of feature f0 + lane, token block q
    uint8_t* by_row = sc + SC_ROW_G * SF_TILE + lane * 16 + q * 4 + c;  // of this row, feature block c
    float w[32];
    uint4 code;
    turn32(buf, v, w, lane);
    by_token[SC_Y * SF_TILE] = static_cast<uint8_t>(quantize32(w, code));
    if (blk) p.yt[(long long)tb * p.N + f0 + lane] = code;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        by_row[part * SF_TILE] = static_cast<uint8_t>(quantize32(part ? u : g, code));
        if (live) p.q[((pg >> 5) + part * 4) * p.M + gm] = code;
        turn32(buf, part ? u : g, w, lane);
        by_token[(SC_G + part) * SF_TILE] = static_cast<uint8_t>(quantize32(w, code));
        const long long col = pg + part * 128 + lane;
        if (blk) p.ht[(long long)tb * (2 * p.N) + col] = code;
        if (p.colsum != nullptr && blk) {
            float s = 0.0f;
#pragma unroll
            for (int t = 0; t < 32; ++t) s += w[t];
            p.colsum[(long long)tb * (2 * p.N) + col] = s;
        }
    }
}

// One stage's codes of an operand, rows from `row`: 128 bytes of k of each (row-major) or 8 blocks of
// all of them (blocked; x counts 8-byte words).
template <bool PAIR>
__device__ __forceinline__ void load_codes(uint8_t* dst, const CUtensorMap* map, uint32_t bar, int it, int row, int blocked) {
    const int x = blocked ? row * 2 : it * 128, y = blocked ? it * 8 : row;
    if constexpr (PAIR) tma_load_3d_pair(dst, map, bar, x, y, 0);
    else tma_load_3d_bar(dst, map, bar, x, y, 0);
}

__device__ __forceinline__ void load_acc32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr, r);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}

// ---------------------------------------------------------------- pair kernel
constexpr int P_BN = 256;
constexpr int P_THREADS = 384;       // warp 0 TMA, warp 1 MMA, warps 4-11 epilogue
constexpr int P_ACC1 = 224;          // second accumulator's first column
constexpr int P_SFA = 480, P_SFB = 488;  // scales: 2 tiles of A (4 columns each), 2 of B (8 each)
constexpr int P_SFA_BYTES = 2 * SF_TILE, P_SFB_BYTES = 4 * SF_TILE;
constexpr int P_STAGE = 2 * OP_BYTES + P_SFA_BYTES + P_SFB_BYTES;
template <int EPI>
struct PairGeom {
    static constexpr int turn = EPI == EPI_DSWIGLU ? 8 * (H_BUF + TURN_WORDS * 4) + 4 * SC_BYTES : 0;
    static constexpr int stages = EPI == EPI_DSWIGLU ? 4 : 6;
    static constexpr int last = 2;  // ring stages at a tile's end that are issued half by half
    static constexpr int smem = 1024 + stages * P_STAGE + turn + 256;
    static_assert(smem <= 227 * 1024, "pair kernel shared memory");
};

__device__ __forceinline__ void decode_tile(const Args& p, int t, int& mb, int& nb) {
    const int per_group = GROUP_M * p.n_blocks;
    const int g = t / per_group;
    const int first_m = g * GROUP_M;
    const int gm = min(p.m_blocks - first_m, GROUP_M);
    const int r = t - g * per_group;
    mb = first_m + r % gm;
    nb = r / gm;
}

// One product: its operands' maps (b2: B in boxes of 64 rows; h: EPI_DSWIGLU's pre-activations) and the rest.
struct Problem {
    CUtensorMap a, b, sa, sb, b2, h;
    Args p;
};
// Up to N independent products in one launch, the longest K loops first.  Every pair takes its share of the long
// tiles; where these do not come out even, the pairs that had one less start on the short ones `skip` tiles
// earlier, which is what a long tile costs.  So no product ends in a wave of its own with most of the GPU idle.
template <int N>
struct Problems {
    Problem of[N];
    int first[N];     // first tile of each product in its class
    int n_long;       // products of the long class
    int long_tiles, short_tiles, skip;
    SumsArgs sums;    // N > 1: the block's bias gradients

    // Tile i of pair `c` of `n`: the product, its tile in t; -1 past the last.
    __device__ __forceinline__ int tile(int c, int n, int i, int& t) const {
        if constexpr (N == 1) {
            t = c + i * n;
            return t < long_tiles ? 0 : -1;
        } else {
            const int r = long_tiles % n, mine = long_tiles / n + (c < r ? 1 : 0);
            int lo = 0, hi = n_long;
            if (i < mine) {
                t = c + i * n;
            } else {
                const int round = i - mine + (c < r ? skip : 0), early = r > 0 ? skip : 0;
                t = round < early ? round * (n - r) + c - r : early * (n - r) + (round - early) * n + c;
                if (t >= short_tiles) return -1;
                lo = n_long;
                hi = N;
            }
            int g = lo;
#pragma unroll
            for (int k = 1; k < N; ++k)
                if (k > lo && k < hi && t >= first[k]) g = k;
            t -= first[g];
            return g;
        }
    }
};

template <int EPI, int N>
__global__ void __launch_bounds__(P_THREADS, 1) mx_pair_kernel(const __grid_constant__ Problems<N> all) {
    uint32_t* const status = all.of[0].p.status;
    const unsigned long long timeout_ns = all.of[0].p.timeout_ns;
    constexpr int LAST = PairGeom<EPI>::last;
    constexpr int STAGES = PairGeom<EPI>::stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + STAGES * OP_BYTES;
    uint8_t* sSA = sB + STAGES * OP_BYTES;
    uint8_t* sSB = sSA + STAGES * P_SFA_BYTES;
    float* turn = reinterpret_cast<float*>(sSB + STAGES * P_SFB_BYTES);
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(turn) + PairGeom<EPI>::turn);
    uint64_t* empty = full + STAGES;
    uint64_t* tfull = empty + STAGES;   // [2] accumulator complete
    uint64_t* tempty = tfull + 2;       // [2] accumulator read
    uint64_t* hfull = tempty + 2;       // [2] the accumulator's half with the shared columns complete
    uint64_t* shared_free = hfull + 2;  // the columns shared with the other accumulator read
    uint64_t* drain = shared_free + 1;
    uint64_t* h_full = drain + 1;       // [8] EPI_DSWIGLU: an epilogue warp's piece of H has landed
    uint64_t* sc_full = h_full + 8;     // [2] EPI_DSWIGLU: the four warps of a half have left a tile's scales
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sc_full + 2);

    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);  // warp-uniform for the compiler
    const int lane = threadIdx.x & 31;
    const uint32_t prank = cluster_ctarank();
    const bool leader = prank == 0;
    const int cluster_id = blockIdx.x / 2;
    const int n_clusters = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull + a, 1);
            mbar_init(tempty + a, 16);  // 8 epilogue warps of either CTA
            mbar_init(hfull + a, 1);
        }
        mbar_init(shared_free, 8);      // the 4 of either CTA that read the shared columns
        mbar_init(drain, 1);
        for (int w = 0; w < 8; ++w) mbar_init(h_full + w, 1);
        for (int w = 0; w < 2; ++w) mbar_init(sc_full + w, 4);
        fence_mbarrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
#pragma unroll
        for (int g = 0; g < N; ++g) {
            tma_prefetch_desc(&all.of[g].a);
            tma_prefetch_desc(&all.of[g].b);
            tma_prefetch_desc(&all.of[g].sa);
            tma_prefetch_desc(&all.of[g].sb);
        }
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();

    if (warp == 0) {
        // ---------------------------------------------------------------- producer (both CTAs)
        int stage = 0;
        uint32_t phase = 0, armed = 0, last_parity = 0;
        bool ok = true;
        const uint32_t full0 = mapa_shared(smem_u32(full), 0);
        for (int i = 0; ok; ++i) {
            int t, mb, nb;
            const int g = all.tile(cluster_id, n_clusters, i, t);
            if (g < 0) break;
            const Problem& pr = all.of[g];
            const Args& p = pr.p;
            decode_tile(p, t, mb, nb);
            const int row_tile = mb * 2 + static_cast<int>(prank);
            const int col0 = nb * P_BN + static_cast<int>(prank) * BM;
            for (int it = 0; it < p.kb; ++it) {
                ok = mbar_wait_bounded_warp(empty + stage, phase ^ 1u, status, timeout_ns, kWhereProducer);
                if (!ok) break;
                if (elect_one()) {
                    if (leader) mbar_arrive_expect_tx(full + stage, 2 * P_STAGE);
                    const uint32_t bar = full0 + stage * 8;
                    load_codes<true>(sA + stage * OP_BYTES, &pr.a, bar, it, row_tile * BM, p.a_blocked);
                    if (it < p.kb - LAST) {
                        load_codes<true>(sB + stage * OP_BYTES, &pr.b, bar, it, col0, p.b_blocked);
                    } else {
                        // each half of the tile's columns as a product of its own: 64 of its columns in each CTA
                        const int c = nb * P_BN + static_cast<int>(prank) * 64;
                        load_codes<true>(sB + stage * OP_BYTES, &pr.b2, bar, it, c, p.b_blocked);
                        load_codes<true>(sB + stage * OP_BYTES + OP_BYTES / 2, &pr.b2, bar, it, c + 128, p.b_blocked);
                    }
                    tma_load_3d_pair(sSA + stage * P_SFA_BYTES, &pr.sa, bar, 0, it * 2, row_tile);
                    tma_load_3d_pair(sSB + stage * P_SFB_BYTES, &pr.sb, bar, 0, it * 2, nb * 2);
                }
                armed |= 1u << stage;
                last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (lane == 0) {
            if (ok) {
                // every stage's last release has arrived before this CTA can exit
                for (int i = 0; i < STAGES; ++i) {
                    if (!mbar_wait_bounded(empty + stage, phase ^ 1u, status, timeout_ns, kWhereDrain)) break;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            } else if (leader) {
                for (int s = 0; s < STAGES; ++s)
                    if (armed & (1u << s))
                        mbar_wait_bounded(full + s, (last_parity >> s) & 1u, status, timeout_ns, kWhereDrain, false);
            } else {
                spin_ns(200000);  // this CTA's last copies, counted on the leader's barriers, land
            }
        }
    } else if (warp == 1) {
        if (leader) {
            // ------------------------------------------------------------ MMA issuer (leader)
            const uint64_t sa0 = sdesc_scales(smem_u32(sSA)), sb0 = sdesc_scales(smem_u32(sSB));
            int stage = 0;
            uint32_t phase = 0;
            int lt = 0;
            bool ok = true;
            for (; ok; ++lt) {
                int t;
                const int g = all.tile(cluster_id, n_clusters, lt, t);
                if (g < 0) break;
                const Args& p = all.of[g].p;
                const uint64_t a0 = p.a_blocked ? sdesc_blocked(smem_u32(sA), BM) : sdesc_sw128(smem_u32(sA), 16, 1024);
                const uint64_t b0 = p.b_blocked ? sdesc_blocked(smem_u32(sB), BM) : sdesc_sw128(smem_u32(sB), 16, 1024);
                // descriptor step of 64 k: 32 bytes of a swizzled row, or two blocks of all rows
                const uint64_t a_step = p.a_blocked ? 2 * BM : 2, b_step = p.b_blocked ? 2 * BM : 2;
                const uint64_t b0h = p.b_blocked ? sdesc_blocked(smem_u32(sB), 64) : b0, bh_step = p.b_blocked ? 128 : 2;
                const int acc = lt & 1;
                ok = mbar_wait_bounded_warp(tempty + acc, ((lt >> 1) & 1) ^ 1u, status, timeout_ns, kWhereMma);
                if (ok && lt > 0) ok = mbar_wait_bounded_warp(shared_free, (lt - 1) & 1, status, timeout_ns, kWhereMma);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem_base + acc * P_ACC1;
                const int it_last = max(p.kb - LAST, 0);
                for (int it = 0; it < it_last; ++it) {
                    ok = mbar_wait_bounded_warp(full + stage, phase, status, timeout_ns, kWhereMma);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t ad = a0 + static_cast<uint64_t>(stage * (OP_BYTES >> 4));
                        const uint64_t bd = b0 + static_cast<uint64_t>(stage * (OP_BYTES >> 4));
                        const uint64_t sad = sa0 + static_cast<uint64_t>(stage * (P_SFA_BYTES >> 4));
                        const uint64_t sbd = sb0 + static_cast<uint64_t>(stage * (P_SFB_BYTES >> 4));
#pragma unroll
                        for (int kt = 0; kt < 2; ++kt) {
                            copy_scales<2>(tmem_base + P_SFA + kt * 4, sad + kt * (SF_TILE >> 4));
                            copy_scales<2>(tmem_base + P_SFB + kt * 8, sbd + kt * (SF_TILE >> 4));
                            copy_scales<2>(tmem_base + P_SFB + kt * 8 + 4, sbd + (2 + kt) * (SF_TILE >> 4));
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_mxf4<2>(d, ad + kk * a_step, bd + kk * b_step, idesc_mxf4(2 * BM, P_BN, (kk & 1) * 2),
                                         tmem_base + P_SFA + (kk >> 1) * 4, tmem_base + P_SFB + (kk >> 1) * 8,
                                         (it | kk) != 0 ? 1u : 0u);
                        umma_commit_pair_mc(empty + stage, 0x3);
                    }
                    __syncwarp();
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                // The last stages half by half: first the 128 columns that hold the shared ones, so that these are read
                // while the other 128 finish and the next tile's MMAs follow on after some 500 idle cycles instead of
                // 1000: 8192 x 20480 x 5120 under the power cap 248 us against 253 (without the cap 218 against 224).
                for (int pass = 0; pass < 2 && ok; ++pass) {
                    const int part = pass == 0 ? 1 - acc : acc;
                    int st = stage;
                    uint32_t ph = phase;
                    for (int it = it_last; it < p.kb; ++it) {
                        if (pass == 0) {
                            ok = mbar_wait_bounded_warp(full + st, ph, status, timeout_ns, kWhereMma);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        if (elect_one()) {
                            const uint64_t ad = a0 + static_cast<uint64_t>(st * (OP_BYTES >> 4));
                            const uint64_t bd = b0h + static_cast<uint64_t>(st * (OP_BYTES >> 4) + part * (OP_BYTES / 2 >> 4));
                            const uint64_t sad = sa0 + static_cast<uint64_t>(st * (P_SFA_BYTES >> 4));
                            const uint64_t sbd = sb0 + static_cast<uint64_t>((st * P_SFB_BYTES + part * 2 * SF_TILE) >> 4);
                            const int steps = it + 1 == p.kb ? p.last_steps : 4;
#pragma unroll
                            for (int kt = 0; kt < 2; ++kt) {
                                if (kt * 2 < steps) {
                                    copy_scales<2>(tmem_base + P_SFA + kt * 4, sad + kt * (SF_TILE >> 4));
                                    copy_scales<2>(tmem_base + P_SFB + kt * 8, sbd + kt * (SF_TILE >> 4));
                                }
                            }
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                if (kk < steps)
                                    umma_mxf4<2>(d + part * 128, ad + kk * a_step, bd + kk * bh_step,
                                                 idesc_mxf4(2 * BM, 128, (kk & 1) * 2), tmem_base + P_SFA + (kk >> 1) * 4,
                                                 tmem_base + P_SFB + (kk >> 1) * 8, (it | kk) != 0 ? 1u : 0u);
                            }
                            if (pass == 1) umma_commit_pair_mc(empty + st, 0x3);
                            if (it + 1 == p.kb) umma_commit_pair_mc((pass == 0 ? hfull : tfull) + acc, 0x3);
                        }
                        __syncwarp();
                        if (++st == STAGES) {
                            st = 0;
                            ph ^= 1u;
                        }
                    }
                    if (pass == 1) {
                        stage = st;
                        phase = ph;
                    }
                }
            }
            if (elect_one()) umma_commit_pair_mc(drain, 0x3);
            __syncwarp();
            // the last releases of the epilogue warps, some from the peer SM, land before this CTA can exit
            if (ok && lt > 0) ok = mbar_wait_bounded_warp(shared_free, (lt - 1) & 1, status, timeout_ns, kWhereDrain);
            for (int i = 0; ok && i < 2; ++i, ++lt)
                ok = mbar_wait_bounded_warp(tempty + (lt & 1), ((lt >> 1) & 1) ^ 1u, status, timeout_ns, kWhereDrain);
        }
        if (lane == 0) mbar_wait_bounded(drain, 0, status, timeout_ns, kWhereDrain, /*watch_status=*/false);
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- epilogue (both CTAs)
        const int q = warp & 3;
        const int half = (warp - 4) >> 2;
        const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0), shared0 = mapa_shared(smem_u32(shared_free), 0);
        [[maybe_unused]] uint8_t* hbuf = reinterpret_cast<uint8_t*>(turn) + (warp - 4) * H_BUF;
        [[maybe_unused]] float* buf = turn + 8 * H_BUF / 4 + (warp - 4) * TURN_WORDS;
        [[maybe_unused]] uint8_t* sc0 = reinterpret_cast<uint8_t*>(turn + 8 * (H_BUF / 4 + TURN_WORDS)) + half * 2 * SC_BYTES;
        constexpr int CH = EPI == EPI_SWIGLU ? 2 : 4;
        const int col0 = half * (CH * 32);
        // EPI_DSWIGLU: each warp copies its next 32 x 32 piece of H while it works on the present one.  (Loads
        // into registers, a row a lane, were most of the epilogue's time.)
        [[maybe_unused]] uint32_t h_phase = 0;
        [[maybe_unused]] bool h_pending = false;
        auto fetch_h = [&](int lt, int i) {
            int t, mb, nb;
            const int g = all.tile(cluster_id, n_clusters, lt, t);
            if (g < 0) return;
            const Problem& pr = all.of[g];
            decode_tile(pr.p, t, mb, nb);
            const int f = nb * P_BN + col0 + ((lt & 1) == 0 ? CH - 1 - i : i) * 32;
            const int row = mb * (2 * BM) + static_cast<int>(prank) * BM + q * 32;
            uint64_t* bar = h_full + (warp - 4);
            if (elect_one()) {
                mbar_arrive_expect_tx(bar, H_BUF);
                const int x = (f >> 7) * 256 + (f & 127);
                tma_load_3d(hbuf, &pr.h, bar, x, row, 0);
                tma_load_3d(hbuf + H_BUF / 2, &pr.h, bar, x + 128, row, 0);
            }
            __syncwarp();
            h_pending = true;
        };
        if constexpr (EPI == EPI_DSWIGLU) {
            fetch_h(0, 0);
        }
        if constexpr (N > 1) {
            // While the first tile's products run, these warps have nothing to do but the column sums, which would
            // otherwise be a launch of their own between the kernels before and after.
            for (int item = static_cast<int>(blockIdx.x) * 8 + warp - 4; item < all.sums.items; item += static_cast<int>(gridDim.x) * 8)
                sum_columns(all.sums, item, lane);
        }
        int lt = 0;
        bool ok = true;
        for (; ok; ++lt) {
            const int acc = lt & 1;
            int t, mb, nb;
            const int g = all.tile(cluster_id, n_clusters, lt, t);
            if (g < 0) break;
            const Args& p = all.of[g].p;
            decode_tile(p, t, mb, nb);  // before the wait: the next tile's MMAs wait for the first columns read here
            const int row0 = mb * (2 * BM) + static_cast<int>(prank) * BM + q * 32;
            // The half with the shared columns: its 128 accumulator columns are complete first.
            const bool first = half == 1 - acc;
            int okw = 0;
            if (lane == 0)
                okw = mbar_wait_bounded((first ? hfull : tfull) + acc, (lt >> 1) & 1, status, timeout_ns, kWhereEpilogue);
            okw = __shfl_sync(0xFFFFFFFFu, okw, 0);
            if (!okw) break;
            tc_fence_after();
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * P_ACC1;
            [[maybe_unused]] uint32_t ys = 0;                         // EPI_SWIGLU: the row's two scale bytes
            [[maybe_unused]] uint8_t* sc = sc0 + acc * SC_BYTES;      // EPI_DSWIGLU: alternating, see below
            // The first accumulator's shared columns are its last, the second's its first: walk the
            // chunks so that they come first.
#pragma unroll 1
            for (int i = 0; i < CH; ++i) {
                const int col = col0 + (acc == 0 ? CH - 1 - i : i) * 32;
                float v[32];
                [[maybe_unused]] float u[32];
                // (EPI_SWIGLU takes gate and up columns, one of them from the other half: the shared chunk, gate of the
                // second accumulator, up of the first, is read alone at first)
                const bool only = EPI == EPI_SWIGLU && i == 0 && first;
                if (!only || acc == 1) load_acc32(t_row + col, v);
                if constexpr (EPI == EPI_SWIGLU) {
                    if (!only || acc == 0) load_acc32(t_row + 128 + col, u);
                }
                if (i == 0 && first) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(shared0);
                    if constexpr (EPI == EPI_SWIGLU) {
                        ok = mbar_wait_bounded_warp(tfull + acc, (lt >> 1) & 1, status, timeout_ns, kWhereEpilogue);
                        if (!ok) break;
                        tc_fence_after();
                        if (acc == 0) load_acc32(t_row + col, v);
                        else load_acc32(t_row + 128 + col, u);
                    }
                }
                if constexpr (EPI == EPI_SWIGLU) ys |= swiglu_chunk(p, v, u, row0 + lane, nb * 128 + col) << (col & 32 ? 8 : 0);
                else if constexpr (EPI == EPI_DSWIGLU) {
                    ok = mbar_wait_bounded_warp(h_full + (warp - 4), h_phase, status, timeout_ns, kWhereEpilogue);
                    if (!ok) break;
                    h_phase ^= 1u;
                    h_pending = false;
                    uint32_t h[32];
                    read_h(hbuf, lane, h);
                    // Every lane's reads are done before the next copy may write here: a warp barrier alone does not
                    // order them before the async proxy's writes (now and then a row came out of the next piece).
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (i + 1 < CH) fetch_h(lt, i + 1);
                    else fetch_h(lt + 1, 0);
                    dswiglu_chunk(p, v, h, row0 + lane, nb * P_BN + col, row0 >> 5, buf, sc, lane);
                } else store_chunk(p, v, row0 + lane, nb * P_BN + col);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + acc * 8);
            if constexpr (EPI == EPI_SWIGLU) {
                const int f0 = nb * 128 + col0;
                if (row0 + lane < p.M && 2 * f0 < p.N)
                    *reinterpret_cast<uint16_t*>(p.qs + scale_offset(row0 + lane, f0 >> 5, p.q_tiles)) = static_cast<uint16_t>(ys);
            }
            if constexpr (EPI == EPI_DSWIGLU) {
                // The half's four warps have written this tile's scales.  The next tile's go to the other buffer,
                // and nobody writes this one again before all have passed the next tile's wait.
                if (lane == 0) mbar_arrive(sc_full + half);
                ok = ok && mbar_wait_bounded_warp(sc_full + half, lt & 1, status, timeout_ns, kWhereEpilogue);
                if (ok) put_scales(p, sc, row0 - q * 32, nb * P_BN + col0, q * 32 + lane, 15u);
            }
        }
        if constexpr (EPI == EPI_DSWIGLU) {
            // (after a wait that gave up) no copy is in flight when this CTA exits
            if (h_pending) mbar_wait_bounded_warp(h_full + (warp - 4), h_phase, status, timeout_ns, kWhereDrain, false);
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // no CTA leaves while its peer may still touch its shared or tensor memory
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// ---------------------------------------------------------------- single kernel
constexpr int S_BN = 128;
constexpr int S_THREADS = 192;       // warp 0 TMA, warp 1 MMA, warps 2-5 epilogue
// Tensor memory: 128 accumulator columns and 32 for the scales, two allocations, so that three CTAs
// fit an SM's 512 columns.
constexpr int S_ACC_COLS = 128, S_SF_COLS = 32;
constexpr int S_SFA = 0, S_SFB = 8;
constexpr int S_MAX_STAGES = 6;
constexpr int S_EPI_BYTES = 4 * TURN_WORDS * 4 + SC_BYTES;  // EPI_DSWIGLU: the end of the ring
template <int EPI, int CTAS>
struct SingleGeom {
    static constexpr int smem = CTAS == 3 ? 75 * 1024 : 113 * 1024;
    static constexpr int ring = smem - 1024 - 256;
    static constexpr int sfb = EPI == EPI_SWIGLU ? 4 * SF_TILE : 2 * SF_TILE;
    static __host__ __device__ constexpr int stage(int a_box) { return a_box * 128 + OP_BYTES + 2 * SF_TILE + sfb; }
    // (the MMA's reads past a narrow A box stay inside the ring: the B stages follow)
    static __host__ __device__ constexpr int stages(int a_box) {
        const int n = ring / stage(a_box);
        return n < S_MAX_STAGES ? n : S_MAX_STAGES;
    }
};
static_assert(SingleGeom<EPI_STORE, 2>::stages(128) >= 3 && SingleGeom<EPI_SWIGLU, 2>::stages(128) >= 3, "ring depth");
static_assert(SingleGeom<EPI_SWIGLU, 3>::stages(32) >= 3, "ring depth");

template <int EPI, int CTAS>
__global__ void __launch_bounds__(S_THREADS, CTAS)
    mx_single_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                     const Args p) {
    constexpr bool GATED = EPI == EPI_SWIGLU;
    constexpr int SFB = SingleGeom<EPI, CTAS>::sfb, S_RING = SingleGeom<EPI, CTAS>::ring;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int a_bytes = p.a_box * 128;
    uint8_t* sA = smem;  // first, so that rows past a narrow box are still in the ring
    uint8_t* sB = sA + p.stages * a_bytes;
    uint8_t* sSA = sB + p.stages * OP_BYTES;
    uint8_t* sSB = sSA + p.stages * 2 * SF_TILE;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S_RING);
    uint64_t* empty = full + S_MAX_STAGES;
    uint64_t* tfull = empty + S_MAX_STAGES;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);  // [2]

    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);  // warp-uniform for the compiler
    const int lane = threadIdx.x & 31;
    uint32_t split, rank;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    rank = cluster_ctarank();
    // all row tiles of a column tile first: B's codes are read from memory once
    const int tile = blockIdx.x / split, nb = tile / p.m_blocks, mb = tile - nb * p.m_blocks;
    const int it0 = static_cast<int>((long long)p.kb * rank / split), it1 = static_cast<int>((long long)p.kb * (rank + 1) / split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(tfull, 1);
        fence_mbarrier_init();
        fence_proxy_async_smem();
    }
    // the tile's columns: gated, 64 gate rows of B and the 64 up rows of the same features
    const int f0 = nb * 64;
    const int gate_row = (f0 >> 7) * 256 + (f0 & 127);
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmSA);
        tma_prefetch_desc(&tmSB);
    }
    if (warp == 2 && lane == 0) {
        // Within the block's forward, the ring's worth of B goes on its way into L2 while the kernel ahead ends:
        // 4 tokens at h5120 f20480 39.3 -> 38.6 us, 100 at h4096 f16384 34.1 -> 33.4.  Twice the ring gained nothing
        // over none and four times lost 4 %.  Products called one after another lose by it (1x20480x5120 12.6 -> 14.0):
        // their kernel ahead still reads memory at full rate.  Nothing is read before the wait, so the order of the
        // stream holds whoever writes B: L2 is where writes arrive.
        if (p.prefetch_b && mb == 0) {
            const int end = min(it0 + p.stages, it1);
            for (int it = it0; it < end; ++it) {
                if constexpr (GATED) {
                    tma_prefetch_3d(&tmB, it * 128, gate_row, 0);
                    tma_prefetch_3d(&tmB, it * 128, gate_row + 128, 0);
                    tma_prefetch_3d(&tmSB, 0, it * 2, (f0 >> 7) * 2);
                } else {
                    tma_prefetch_3d(&tmB, it * 128, nb * S_BN, 0);
                    tma_prefetch_3d(&tmSB, 0, it * 2, nb);
                }
            }
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, S_ACC_COLS);
        tmem_alloc(tmem_slot + 1, S_SF_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = tmem_slot[0], sf_base = tmem_slot[1];
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();

    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        int stage = 0;
        uint32_t phase = 0, armed = 0, last_parity = 0;
        const uint32_t bytes = static_cast<uint32_t>(a_bytes + OP_BYTES + 2 * SF_TILE + SFB);
        for (int it = it0; it < it1; ++it) {
            if (!mbar_wait_bounded_warp(empty + stage, phase ^ 1u, p.status, p.timeout_ns, kWhereProducer)) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(full + stage, bytes);
                uint8_t* b = sB + stage * OP_BYTES;
                const uint32_t bar = smem_u32(full + stage);
                if constexpr (GATED) {
                    tma_load_3d(b, &tmB, full + stage, it * 128, gate_row, 0);
                    tma_load_3d(b + OP_BYTES / 2, &tmB, full + stage, it * 128, gate_row + 128, 0);
                    tma_load_3d(sSB + stage * SFB, &tmSB, full + stage, 0, it * 2, (f0 >> 7) * 2);
                } else {
                    load_codes<false>(b, &tmB, bar, it, nb * S_BN, p.b_blocked);
                    tma_load_3d(sSB + stage * SFB, &tmSB, full + stage, 0, it * 2, nb);
                }
                load_codes<false>(sA + stage * a_bytes, &tmA, bar, it, mb * BM, p.a_blocked);
                tma_load_3d(sSA + stage * 2 * SF_TILE, &tmSA, full + stage, 0, it * 2, mb);
            }
            armed |= 1u << stage;
            last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == p.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        // all copies have landed before this CTA can reuse its ring or exit, also where a wait gave up
        if (lane == 0) {
            for (int s = 0; s < p.stages; ++s)
                if (armed & (1u << s))
                    mbar_wait_bounded(full + s, (last_parity >> s) & 1u, p.status, p.timeout_ns, kWhereDrain, false);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        const uint64_t a0 = p.a_blocked ? sdesc_blocked(smem_u32(sA), p.a_box) : sdesc_sw128(smem_u32(sA), 16, 1024);
        const uint64_t b0 = p.b_blocked ? sdesc_blocked(smem_u32(sB), BM) : sdesc_sw128(smem_u32(sB), 16, 1024);
        const uint64_t a_step = p.a_blocked ? 2 * p.a_box : 2, b_step = p.b_blocked ? 2 * BM : 2;
        const uint64_t sa0 = sdesc_scales(smem_u32(sSA)), sb0 = sdesc_scales(smem_u32(sSB));
        int stage = 0;
        uint32_t phase = 0;
        for (int it = it0; it < it1; ++it) {
            if (!mbar_wait_bounded_warp(full + stage, phase, p.status, p.timeout_ns, kWhereMma)) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t ad = a0 + static_cast<uint64_t>(stage * (a_bytes >> 4));
                const uint64_t bd = b0 + static_cast<uint64_t>(stage * (OP_BYTES >> 4));
                const uint64_t sad = sa0 + static_cast<uint64_t>(stage * (2 * SF_TILE >> 4));
                const uint64_t sbd = sb0 + static_cast<uint64_t>(stage * (SFB >> 4));
                const int steps = it + 1 == p.kb ? p.last_steps : 4;
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) {
                    if (kt * 2 < steps) {
                        copy_scales<1>(sf_base + S_SFA + kt * 4, sad + kt * (SF_TILE >> 4));
                        copy_scales<1>(sf_base + S_SFB + kt * 4, sbd + kt * (SF_TILE >> 4));
                        if constexpr (GATED) copy_scales<1>(sf_base + S_SFB + 8 + kt * 4, sbd + (2 + kt) * (SF_TILE >> 4));
                    }
                }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if (kk < steps) {
                        const uint32_t add = (it != it0 || kk != 0) ? 1u : 0u;
                        const uint32_t sfa = sf_base + S_SFA + (kk >> 1) * 4, sfb = sf_base + S_SFB + (kk >> 1) * 4;
                        if constexpr (GATED) {
                            // 64 rows of a scale tile are two of its four columns
                            const uint32_t id = idesc_mxf4(BM, 64, (kk & 1) * 2), odd = (f0 & 64) ? 2u : 0u;
                            umma_mxf4<1>(tmem_base, ad + kk * a_step, bd + kk * 2, id, sfa, sfb + odd, add);
                            umma_mxf4<1>(tmem_base + 64, ad + kk * a_step, bd + (OP_BYTES / 2 >> 4) + kk * 2, id, sfa, sfb + 8 + odd,
                                         add);
                        } else {
                            umma_mxf4<1>(tmem_base, ad + kk * a_step, bd + kk * b_step, idesc_mxf4(BM, S_BN, (kk & 1) * 2), sfa, sfb, add);
                        }
                    }
                }
                umma_commit(empty + stage);
            }
            __syncwarp();
            if (++stage == p.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (elect_one()) umma_commit(tfull);
    }
    __syncwarp();
    const int q = warp & 3;
    const int row0 = mb * BM + q * 32;
    const bool epi = warp >= 2;
    // Warps whose rows are all past M have nothing to do; the token-wise outputs also want the zeros
    // of a last scale tile's blocks past M.
    const bool work = epi && (EPI == EPI_DSWIGLU || row0 < p.M);
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    // every warp waits: nobody leaves (or lets its shared memory be written by a peer) while copies or
    // MMAs are in flight
    if (lane == 0) mbar_wait_bounded(tfull, 0, p.status, p.timeout_ns, kWhereEpilogue, /*watch_status=*/false);
    __syncwarp();
    tc_fence_after();
    fence_proxy_async_all();  // the ring becomes this kernel's own memory: after the copies' writes and the MMAs' reads
    constexpr int CH = GATED ? 2 : 4;        // 32-column chunks (gated: of features)
    constexpr int PARTS = GATED ? 2 : 1;     // accumulator chunks of one of them
    const int owners = min(static_cast<int>(split), CH);
    const int rows_in = min(BM, ((p.M - mb * BM) + 31) / 32 * 32);  // rows exchanged: whole warps
    const int ethread = q * 32 + lane;       // row of this thread
    uint4* recv = reinterpret_cast<uint4*>(smem);  // over the ring, once all of this CTA's MMAs are done
    if (split > 1) {
        cluster_sync_all();  // every CTA's ring is free
        if (work && row0 - mb * BM < rows_in) {
#pragma unroll 1
            for (int c = 0; c < CH; ++c) {
                const uint32_t owner = static_cast<uint32_t>(c % owners);
                if (owner == rank) continue;
                // slot: [chunk of the owner][sender][part][16-byte piece][row]
                const int sender = static_cast<int>(rank > owner ? rank - 1 : rank);
                const uint32_t slot = ((c / owners) * (split - 1) + sender) * PARTS;
                const uint32_t dst = mapa_shared(smem_u32(recv), owner);
#pragma unroll
                for (int part = 0; part < PARTS; ++part) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(t_row + part * 64 + c * 32, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        st_cluster_v4(dst + (((slot + part) * 8 + j) * rows_in + ethread) * 16, r[4 * j], r[4 * j + 1],
                                      r[4 * j + 2], r[4 * j + 3]);
                }
            }
        }
        cluster_sync_all();  // the partial sums have arrived
    }
    if (work) {
        // (at the ring's end, behind the received partial sums)
        [[maybe_unused]] uint8_t* sc = smem + S_RING - SC_BYTES;
        [[maybe_unused]] float* buf = reinterpret_cast<float*>(sc) - (q + 1) * TURN_WORDS;
        [[maybe_unused]] uint32_t done = 0;
#pragma unroll 1
        for (int c = 0; c < CH; ++c) {
            if (split > 1 && static_cast<uint32_t>(c % owners) != rank) continue;
            float v[32];
            [[maybe_unused]] float u[32];
            load_acc32(t_row + c * 32, v);
            if constexpr (GATED) load_acc32(t_row + 64 + c * 32, u);
            if (split > 1 && row0 - mb * BM < rows_in) {
#pragma unroll 1
                for (uint32_t s = 0; s + 1 < split; ++s) {
                    const uint32_t slot = ((c / owners) * (split - 1) + s) * PARTS;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint4 x = recv[(slot * 8 + j) * rows_in + ethread];
                        v[4 * j] += __uint_as_float(x.x);
                        v[4 * j + 1] += __uint_as_float(x.y);
                        v[4 * j + 2] += __uint_as_float(x.z);
                        v[4 * j + 3] += __uint_as_float(x.w);
                        if constexpr (GATED) {
                            const uint4 y = recv[((slot + 1) * 8 + j) * rows_in + ethread];
                            u[4 * j] += __uint_as_float(y.x);
                            u[4 * j + 1] += __uint_as_float(y.y);
                            u[4 * j + 2] += __uint_as_float(y.z);
                            u[4 * j + 3] += __uint_as_float(y.w);
                        }
                    }
                }
            }
            if constexpr (GATED) {
                const uint32_t s = swiglu_chunk(p, v, u, row0 + lane, f0 + c * 32);
                if (row0 + lane < p.M) p.qs[scale_offset(row0 + lane, (f0 >> 5) + c, p.q_tiles)] = static_cast<uint8_t>(s);
            } else if constexpr (EPI == EPI_DSWIGLU) {
                uint32_t h[32];
                load_h(p, row0 + lane, nb * S_BN + c * 32, h);
                dswiglu_chunk(p, v, h, row0 + lane, nb * S_BN + c * 32, row0 >> 5, buf, sc, lane);
                done |= 1u << c;
            } else store_chunk(p, v, row0 + lane, nb * S_BN + c * 32);
        }
        if constexpr (EPI == EPI_DSWIGLU) {
            asm volatile("bar.sync 1, 128;" ::: "memory");  // the four warps' scales are there
            put_scales(p, sc, mb * BM, nb * S_BN, q * 32 + lane, done);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem_base, S_ACC_COLS);
        tmem_dealloc(sf_base, S_SF_COLS);
    }
}

}  // namespace mx
}  // namespace tpmlp
