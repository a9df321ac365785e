// Products grouped by expert on the bf16 tensor cores (tcgen05, CTA pairs), rows sorted by expert, the
// experts' row ranges read on the device.
//
//   rows kernel   Y[r][n] = sum_k X[src r][k] W[e][k][n]       (W as it is, "forward")
//                 dX[r][k] = sum_n dY[r][n] W[e][k][n]         (W transposed, "dx")
//   dw kernel     dW[e][k][n] = sum over rows r of e of X[src r][k] dY[r][n]
//
// The rows kernel puts the weights' features on the 256 rows of a pair's tile and the tokens on its columns, so a
// tile holds any multiple of 16 tokens up to 256 and an expert with few rows costs the tensor cores, and the way
// from L2, only what it has: the row range of an expert is cut into equal tiles, at most 256 tokens each.  (With
// tokens on the tile's rows every expert would end in a partly empty tile of 256.)  Accumulators come out
// transposed, a feature in each tensor-memory lane; they are read as 8x8 fragments and turned by stmatrix on the
// way to rows in memory.
//
// The gated first layer has 64 gate and the 64 up features of the same indices on a CTA's 128 lanes.  The warps of the up
// features pass their accumulators to those of the gate's through shared memory, 32 x 32 at a time.  (Gate and up as two
// accumulators of 128 tokens on the same lanes need no exchange, but MMAs of 128 columns: their operands take all of the
// shared memory's 128 bytes a cycle, and 16384 rows x 5120 x 8192 took 1011 us in order.)
#pragma once
#include <type_traits>

#include "gemm_tc.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace tpmlp {
namespace moe {

constexpr int MAX_EXPERTS = 1024;
constexpr int BM = 128;  // features of one CTA's half of a tile (rows kernel)
constexpr int BK = 64;   // contraction per ring stage: 128-byte rows
constexpr int CHUNK = BK * 128;        // 64 features x 64 k, or 64 tokens x 64 k
constexpr int THREADS = 384;           // warp 0 TMA, warp 1 MMA, warps 2-3 gathered rows, warps 4-11 epilogue
constexpr int EPI_WARP = 4;
constexpr int EPI_WARPS = 8;
constexpr int GROUP = 16;              // token tiles walked together, so that tiles in flight share weights and tokens
constexpr int TABLE = 2 * (MAX_EXPERTS + 1) * 4 + MAX_EXPERTS * 2;
constexpr int SORTED = 128;            // experts up to which their tiles are walked largest first

enum Mode : int { STORE = 0, SWIGLU = 1, DSWIGLU = 2 };

struct Args {
    const int* offsets;  // [experts + 1]
    const int* src;      // token of each row, may be null
    const __nv_bfloat16* x;  // gathered rows, dw: X [tokens][x_ld]
    int x_ld;
    int rows, tokens, experts;
    int kb;              // rows kernel: blocks of 64 of the contraction
    int chunked;         // W's map is [experts][features / 64][K][64]: a stage's chunks in one copy
    int features;        // rows kernel: features on the tile's rows (SWIGLU, DSWIGLU: gate features); dw: K
    int cols;            // dw: N
    const __nv_bfloat16* dy;  // dw: dY [rows][cols]
    int skip, most;      // dw: each expert's rows past its first `skip`, at most `most` of them
    int add;             // dw: to the (fp32) output
    int m_blocks;        // rows kernel: blocks of 256 features; dw: of K
    int n_blocks;        // dw: blocks of 256 of N
    void* out; long long ld;        // row pitch of out (elements)
    int out_f32;
    const __nv_bfloat16* bias;      // [experts][bias_ld], packed for SWIGLU
    long long bias_ld;
    void* h_out;                    // SWIGLU: packed pre-activations (fp32 with H32), may be null; DSWIGLU reads h_in
    const void* h_in;
    long long h_ld;
    uint32_t* status;
    unsigned long long timeout_ns;
};

// Bounded waits.  They go by their time limit alone: a wait that gave up in another call does not end them.
__device__ __forceinline__ bool wait(const Args& p, uint64_t* bar, uint32_t parity, uint32_t where) {
    return mbar_wait_bounded(bar, parity, p.status, p.timeout_ns, where, false);
}
__device__ __forceinline__ bool wait_warp(const Args& p, uint64_t* bar, uint32_t parity, uint32_t where) {
    return mbar_wait_bounded_warp(bar, parity, p.status, p.timeout_ns, where, false);
}

// A plan that reaches outside of its tensors is cut, and recorded in a word of its own: the first one ends the waits of other
// GEMM kernels, whose calls have nothing to do with it.
__device__ __forceinline__ void record_cut(const Args& p) { atomicExch(p.status + kPlanWord, kStatusDevice); }

// Pieces of shared memory, one behind the other.
struct Carve {
    uint8_t* at;
    template <typename T>
    __device__ __forceinline__ T* take(int n) {
        T* p = reinterpret_cast<T*>(at);
        at += n * sizeof(T);
        return p;
    }
};
constexpr int most_barriers = 5 * 6 + 5;  // of either kernel, and the tensor memory's address

// ---------------------------------------------------------------- the experts' row ranges and tiles
// Row ranges are clamped to the rows that there are; a range that had to be is reported, its product left out or cut.
struct Table {
    int* off;       // [experts + 1] first row
    int* first;     // [experts + 1] first tile of the expert at that place of the order
    uint16_t* at;   // [experts] the order: as they are or, where they are few, by falling tiles
    __device__ __forceinline__ explicit Table(void* smem)
        : off(static_cast<int*>(smem)), first(off + MAX_EXPERTS + 1), at(reinterpret_cast<uint16_t*>(first + MAX_EXPERTS + 1)) {}
    __device__ __forceinline__ int count(int e) const { return max(off[e + 1] - off[e], 0); }
    // All threads.  tiles(n) gives the tiles of an expert of n rows, cost(n) what one of them takes (BY_COST: order by it).
    template <int NTHREADS, bool BY_COST, typename F, typename C>
    __device__ __forceinline__ void build(const Args& p, F&& tiles, C&& cost) {
        bool bad = false;
        for (int i = threadIdx.x; i <= p.experts; i += NTHREADS) {
            const int v = p.offsets[i], c = min(max(v, 0), p.rows);
            bad |= v != c;
            off[i] = c;
            if (i < p.experts) at[i] = static_cast<uint16_t>(i);
        }
        __syncthreads();
        if (BY_COST && p.experts <= SORTED) {
            // each expert's place: the experts with larger tiles, and those ahead of it with equal ones
            const int e = threadIdx.x;
            if (e < p.experts) first[e] = cost(count(e));
            __syncthreads();
            if (e < p.experts) {
                const int mine = first[e];
                int place = 0;
                for (int i = 0; i < p.experts; ++i) place += first[i] > mine || (first[i] == mine && i < e) ? 1 : 0;
                at[place] = static_cast<uint16_t>(e);
            }
            __syncthreads();
        }
        if (threadIdx.x < 32) {
            const int lane = threadIdx.x;
            int carry = 0;
            for (int i0 = 0; i0 < p.experts; i0 += 32) {
                const int i = i0 + lane;
                int v = 0;
                if (i < p.experts) {
                    bad |= off[i + 1] < off[i];
                    v = tiles(count(at[i]));
                }
                int sum = v;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                    if (lane >= d) sum += o;
                }
                if (i < p.experts) first[i] = carry + sum - v;
                carry += __shfl_sync(0xFFFFFFFFu, sum, 31);
            }
            if (lane == 0) first[p.experts] = carry;
        }
        if (bad && blockIdx.x == 0) record_cut(p);
        __syncthreads();
    }
};
// Round i's tile of pair c of n.  BACK: there and back, so that who has a large tile in one round has a small one in the next.
// (Together with the order by cost: weight gradients of 8192 rows on 64 experts, 1024 x 2048, 78 -> 71 us in order, 101 -> 82
// gathered; wide tiles of 2048 rows on 8 experts, 5120 x 8192, 152 -> 140.  Narrow tiles, which overlap their epilogues, gain
// nothing, up to 4 % of their time is lost.)
template <bool BACK>
__device__ __forceinline__ int round_tile(int i, int c, int n) {
    return i * n + (BACK && (i & 1) ? n - 1 - c : c);
}

// Tokens of a tile: an expert's n rows in ceil(n / TN) tiles of equal size, a multiple of 16.  (The last one is
// never empty: with a size below TN there are fewer than TN / 16 tiles.)
template <int TN>
__device__ __forceinline__ int tile_tokens(int n) {
    const int nt = (n + TN - 1) / TN;
    return ((n + nt - 1) / nt + 15) & ~15;
}

struct Tile {
    int e, mb, row0, n;  // expert, feature block, first row, rows (0: past the last tile)
};
// Tile t; i is where the walk over the order stands (tiles come in increasing order).
template <int TN>
__device__ __forceinline__ Tile decode(const Args& p, const Table& tab, int t, int& i) {
    while (i < p.experts && t >= tab.first[i + 1]) ++i;
    if (i >= p.experts) return Tile{0, 0, 0, 0};
    const int e = tab.at[i], n = tab.count(e), nt = (n + TN - 1) / TN, sz = tile_tokens<TN>(n);
    const int l = t - tab.first[i], per_group = GROUP * p.m_blocks;
    const int g = l / per_group, r = l - g * per_group, gt = min(nt - g * GROUP, GROUP);
    const int tb = g * GROUP + r % gt;
    return Tile{e, r / gt, tab.off[e] + tb * sz, min(sz, n - tb * sz)};
}

// ---------------------------------------------------------------- epilogue pieces
// A warp's staging of 32 tokens x 32 features, bf16: rows of 64 bytes, their four 16-byte pieces permuted so that
// the eight rows of an 8x8 matrix lie in different banks.
constexpr int STAGE = 32 * 64;
__device__ __forceinline__ uint32_t stage_at(int token, int piece) {
    return static_cast<uint32_t>(token * 64 + ((piece ^ ((token >> 1) & 3)) << 4));
}
// lo, hi: packed fragments of features 0-15 and 16-31, a word per (8 tokens, 8 features): index 2 i + j.
__device__ __forceinline__ void stage_put(uint32_t buf, const uint32_t (&lo)[8], const uint32_t (&hi)[8], int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        stmatrix_x4_trans(buf + stage_at(i * 8 + (lane & 7), lane >> 3), lo[2 * i], lo[2 * i + 1], hi[2 * i], hi[2 * i + 1]);
}
__device__ __forceinline__ void stage_get(uint32_t buf, uint32_t (&lo)[8], uint32_t (&hi)[8], int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t r[4];
        ldmatrix_x4_trans(buf + stage_at(i * 8 + (lane & 7), lane >> 3), r);
        lo[2 * i] = r[0];
        lo[2 * i + 1] = r[1];
        hi[2 * i] = r[2];
        hi[2 * i + 1] = r[3];
    }
}
// The staged rows to memory: dst is row 0's first feature, n rows, nf features (a multiple of 8) of the 32.
__device__ __forceinline__ void stage_store(const uint8_t* buf, __nv_bfloat16* dst, long long ld, int n, int nf, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = i * 8 + (lane >> 2), c = lane & 3;
        if (t < n && c * 8 < nf) *reinterpret_cast<uint4*>(dst + t * ld + c * 8) = *reinterpret_cast<const uint4*>(buf + stage_at(t, c));
    }
}
__device__ __forceinline__ void stage_load(uint8_t* buf, const uint4 (&v)[4], int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(buf + stage_at(i * 8 + (lane >> 2), lane & 3)) = v[i];
}
__device__ __forceinline__ void rows_load(const __nv_bfloat16* src, long long ld, int n, int nf, int lane, uint4 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = i * 8 + (lane >> 2), c = lane & 3;
        v[i] = t < n && c * 8 < nf ? *reinterpret_cast<const uint4*>(src + t * ld + c * 8) : make_uint4(0, 0, 0, 0);
    }
}
// Packed fragments of 32 tokens x 32 features to their rows in memory.
__device__ __forceinline__ void put_rows(uint8_t* buf, __nv_bfloat16* dst, long long ld, const uint32_t (&lo)[8], const uint32_t (&hi)[8],
                                         int n, int nf, int lane) {
    stage_put(smem_u32(buf), lo, hi, lane);
    __syncwarp();
    stage_store(buf, dst, ld, n, nf, lane);
    __syncwarp();
}
__device__ __forceinline__ void pack_frags(const uint32_t (&a)[16], const uint32_t (&b)[16], uint32_t (&lo)[8], uint32_t (&hi)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = tc::pack_bf16x2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1]));
        hi[i] = tc::pack_bf16x2(__uint_as_float(b[2 * i]), __uint_as_float(b[2 * i + 1]));
    }
}
// silu(gate) up, packed
__device__ __forceinline__ void gate_frags(const uint32_t (&a)[16], const uint32_t (&b)[16], const uint32_t (&ua)[16],
                                           const uint32_t (&ub)[16], uint32_t (&lo)[8], uint32_t (&hi)[8]) {
    auto gated = [](uint32_t g, uint32_t u) {
        const float x = __uint_as_float(g);
        return x * tc::sigmoid_approx(x) * __uint_as_float(u);
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = tc::pack_bf16x2(gated(a[2 * i], ua[2 * i]), gated(a[2 * i + 1], ua[2 * i + 1]));
        hi[i] = tc::pack_bf16x2(gated(b[2 * i], ub[2 * i]), gated(b[2 * i + 1], ub[2 * i + 1]));
    }
}
// dg = dy u silu'(g), du = dy silu(g)
__device__ __forceinline__ void gated_gradient(float dy, float g, float u, float& dg, float& du) {
    const float s = tc::sigmoid_approx(g);
    du = dy * g * s;
    dg = dy * u * (s * (1.0f + g * (1.0f - s)));
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A barrier of two warps.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
// The same, and whether `ok` holds in both.
__device__ __forceinline__ bool pair_and(int id, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(ok ? 1u : 0u), "r"(id)
        : "memory");
    return r != 0;
}
// 32 lanes x 32 columns as fragments: a, lanes 0-15, b, lanes 16-31.
__device__ __forceinline__ void load_frags(uint32_t taddr, uint32_t (&a)[16], uint32_t (&b)[16]) {
    tmem_ld_16x256b_x4(taddr, a);
    tmem_ld_16x256b_x4(taddr + (16u << 16), b);
}
// Bias of this thread's four features (t / 4 + 0, 8, 16, 24) of 32 from f0; zero past nf.
__device__ __forceinline__ void load_bias(const __nv_bfloat16* bias, int nf, int lane, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int f = i * 8 + (lane >> 2);
        v[i] = bias != nullptr && f < nf ? __bfloat162float(bias[f]) : 0.0f;
    }
}

// ---------------------------------------------------------------- rows kernel
// WIDE: two accumulators of 256 tokens, twice the features, for gathered rows: a stage's copies of rows, which bound the
// narrow tile's time, then feed twice the MMAs.  Both take all of tensor memory, so a tile's epilogue and the next tile's
// products do not overlap.
template <int MODE, bool WIDE = false>
struct Geom {
    static constexpr int tn = 256;                      // tokens of a tile at most
    static constexpr int f = (MODE == SWIGLU ? 128 : 256) * (WIDE ? 2 : 1);  // features of a tile (SWIGLU: gate and up of each)
    static constexpr int a_bytes = BM * 128 * (WIDE ? 2 : 1);  // this CTA's features of a stage
    static constexpr int b_bytes = tn / 2 * 128;        // this CTA's half of the tokens
    static constexpr int stage = a_bytes + b_bytes;
    static constexpr int epi = (MODE == DSWIGLU ? 2 : 1) * STAGE;  // staging of an epilogue warp
    static constexpr int pass = MODE == SWIGLU && !WIDE ? 4 * 4096 : 0;  // up accumulators on their way to the gate's warps
    static constexpr int stages = WIDE ? 4 : MODE == STORE ? 6 : 5;
    static constexpr int smem = 1024 + stages * stage + EPI_WARPS * epi + pass + (most_barriers + 1) * 8 + TABLE;
    static_assert(smem <= 227 * 1024, "rows kernel shared memory");
    static_assert(2 * stages + 5 <= most_barriers);
};

// The tokens' maps: boxes of 8, 16 .. 128 rows.  A CTA's half of a tile, any multiple of 8 rows, is copied as the largest
// box that it holds and one more that holds the rest: few copies, at most a third more than is needed.  (A copy costs the
// TMA unit some 75 cycles however small: 15 boxes of 8 rows took twice the MMAs' time.)
struct Boxes {
    CUtensorMap m[5];
};
struct Halves {
    int first, second;  // boxes of 8 << first, 8 << second rows; second -1: none
    __device__ __forceinline__ explicit Halves(int rows) {
        first = 31 - __clz(rows >> 3);
        const int rest = (rows >> 3) - (1 << first);
        second = rest == 0 ? -1 : 32 - __clz(rest - 1);
    }
    __device__ __forceinline__ int rows() const { return (8 << first) + (second < 0 ? 0 : 8 << second); }
};

// Gathered rows come as TMA gathers of four rows, every second one from warp 2 and from warp 3: an elected lane issues
// them in runs without a branch between, the row numbers in its registers.  (With a branch ahead of each, a copy took a
// warp 88 cycles, and the product of 16384 rows x 5120 x 8192 1620 us; without, 910, where rows that lie in order take 780
// as boxes.  Copies by cp.async took 2560: the proxy fence that the tensor cores need behind them waits for all copies
// in flight, also from a warp of its own.)
//
// A token read from src, cut to those that there are.
__device__ __forceinline__ int checked(const Args& p, int v) {
    const int t = min(max(v, 0), p.tokens - 1);
    if (v != t) record_cut(p);
    return t;
}
// Row numbers of a warp's copies: rows row0 + 8 j .. + 3, at most `last`.  (All loads before the first check, which waits.)
template <int PER>
__device__ __forceinline__ void gather_rows(const Args& p, int row0, int last, int copies, int4 (&at)[PER]) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int r = row0 + j * 8;
        at[j] = j < copies ? make_int4(p.src[min(r, last)], p.src[min(r + 1, last)], p.src[min(r + 2, last)], p.src[min(r + 3, last)])
                           : make_int4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) at[j] = make_int4(checked(p, at[j].x), checked(p, at[j].y), checked(p, at[j].z), checked(p, at[j].w));
}
// Copies J .. J + N - 1 of a warp: groups of four rows, every second one of the operand.
template <bool PAIR, int J, int N, int PER>
__device__ __forceinline__ void gather_run(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, const int4 (&at)[PER]) {
#pragma unroll
    for (int j = J; j < J + N; ++j) tma_gather4<PAIR>(dst + j * 1024, map, bar, x, at[j]);
}
// n of at most 2^k copies from J on, by halves.
template <bool PAIR, int J, int MOST, int PER>
__device__ __forceinline__ void gather_some(int n, uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, const int4 (&at)[PER]) {
    if (n == MOST) {
        gather_run<PAIR, J, MOST>(dst, map, bar, x, at);
    } else if constexpr (MOST > 1) {
        if (n >= MOST / 2) {
            gather_run<PAIR, J, MOST / 2>(dst, map, bar, x, at);
            gather_some<PAIR, J + MOST / 2, MOST / 2>(n - MOST / 2, dst, map, bar, x, at);
        } else {
            gather_some<PAIR, J, MOST / 2>(n, dst, map, bar, x, at);
        }
    }
}

// Pre-activations in fp32 (H32): a lane has a feature and goes from token to token, 128 bytes of a warp in each row.  Gate and up
// rounded to bf16 each cost the gradients a rounding of their own (dX through both layers 3.0e-3 off, from fp32 2.3e-3), twice
// the bytes time: 16384 rows on 8 experts, 5120 x 8192 gated and saved 754-774 us, in fp32 793-857; 8192 rows on 64 experts,
// 1024 x 2048 68, 74, gradient of 1024 features 45, 58.
template <bool H32>
using PreAct = typename std::conditional<H32, float, __nv_bfloat16>::type;
__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store_as(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_as(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
// 32 lanes x 32 columns of an accumulator and the lane's bias to n rows.
__device__ __forceinline__ void store_rows_f32(uint32_t taddr, float bias, float* dst, long long ld, int n) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr, r);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j < n) dst[j * ld] = __uint_as_float(r[j]) + bias;
}
// Gate and up of this lane's feature for 16 rows, n of which there are.
__device__ __forceinline__ void load_rows_f32(const float* h, long long ld, int n, float (&g)[16], float (&u)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        g[j] = j < n ? h[j * ld] : 0.0f;
        u[j] = j < n ? h[j * ld + 128] : 0.0f;
    }
}
// Their gradients from 16 columns of the accumulator.
template <int FIRST>
__device__ __forceinline__ void gated_rows(const uint32_t (&d)[32], const float (&g)[16], const float (&u)[16], __nv_bfloat16* dst, long long ld, int n) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float dg, du;
        gated_gradient(__uint_as_float(d[FIRST + j]), g[j], u[j], dg, du);
        if (j < n) {
            dst[j * ld] = __float2bfloat16_rn(dg);
            dst[j * ld + 128] = __float2bfloat16_rn(du);
        }
    }
}

template <bool W_MN, int MODE, bool WIDE = false, bool H32 = false>
__global__ void __launch_bounds__(THREADS, 1)
    rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ Boxes tmX, const Args p) {
    using G = Geom<MODE, WIDE>;
    static_assert(MODE != DSWIGLU || !WIDE);
    static_assert(MODE != STORE || !H32);
    constexpr int S = G::stages, TN = G::tn;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + S * G::a_bytes;
    uint8_t* sE = smem + S * G::stage;
    Carve carve{sE + EPI_WARPS * G::epi + G::pass};
    uint64_t* full = carve.take<uint64_t>(S);
    uint64_t* empty = carve.take<uint64_t>(S);
    uint64_t* tfull = carve.take<uint64_t>(2);
    uint64_t* tempty = carve.take<uint64_t>(2);
    uint64_t* drain = carve.take<uint64_t>(1);
    uint32_t* tmem_slot = carve.take<uint32_t>(2);
    Table tab(carve.take<int>(TABLE / 4));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t prank = cluster_ctarank();
    const bool leader = prank == 0;
    const int cluster_id = blockIdx.x / 2, n_clusters = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull + a, 1);
            mbar_init(tempty + a, 2 * EPI_WARPS);
        }
        mbar_init(drain, 1);
        fence_mbarrier_init();
        fence_proxy_async_smem();
        tma_prefetch_desc(&tmW);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // the peer may signal the leader's barriers from here on
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    griddep_wait();  // no global memory is touched before the kernel ahead has completed
    if (threadIdx.x == 0) griddep_launch_dependents();
    tab.build<THREADS, WIDE>(p, [&](int n) { return (n + TN - 1) / TN * p.m_blocks; }, [](int n) { return n > 0 ? tile_tokens<TN>(n) : 0; });
    const int n_tiles = tab.first[p.experts];

    if (warp == 0) {
        // ---------------------------------------------------------------- producer (both CTAs), a whole warp
        int stage = 0, e = 0;
        uint32_t phase = 0, armed = 0, last_parity = 0;
        bool ok = true;
        const uint32_t full0 = mapa_shared(smem_u32(full), 0);
        for (int i = 0, t; (t = round_tile<WIDE>(i, cluster_id, n_clusters)) < n_tiles && ok; ++i) {
            const Tile c = decode<TN>(p, tab, t, e);
            const int nn = (c.n + 15) & ~15, half = nn / 2;  // columns of the MMA, tokens of this CTA
            const int row0 = c.row0 + static_cast<int>(prank) * half;
            // first column of W of this CTA's (SWIGLU: 64, or 128, gate features of block mb, their up features 128 columns on)
            const int f0 = MODE != SWIGLU ? c.mb * G::f + static_cast<int>(prank) * BM
                           : WIDE         ? (c.mb * 2 + static_cast<int>(prank)) * 256
                                          : c.mb * 256 + static_cast<int>(prank) * 64;
            const Halves box(half);
            const uint32_t bytes = 2 * (G::a_bytes + (p.src == nullptr ? box.rows() : half) * 128);
            for (int it = 0; it < p.kb; ++it) {
                if (!wait_warp(p, empty + stage, phase ^ 1u, kWhereProducer)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = full0 + stage * 8;
                uint8_t* a_dst = sA + stage * G::a_bytes;
                uint8_t* b_dst = sB + stage * G::b_bytes;
                if (lane == 0) {
                    if (leader) {
                        mbar_arrive_expect_tx(full + stage, bytes);
                        armed |= 1u << stage;
                        last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
                    }
                    if constexpr (!W_MN) {
                        tma_load_3d_pair(a_dst, &tmW, bar, it * BK, f0, c.e);
                        if constexpr (WIDE) tma_load_3d_pair(a_dst + BM * 128, &tmW, bar, it * BK, f0 + 256, c.e);
                    } else {
                        // chunks of 64 columns, SWIGLU's narrow tile every second one, STORE's wide tile two and, 256 on, two
                        if (p.chunked) {
                            tma_load_4d_pair(a_dst, &tmW, bar, 0, it * BK, f0 / 64, c.e);
                            if constexpr (MODE == STORE && WIDE) tma_load_4d_pair(a_dst + 2 * CHUNK, &tmW, bar, 0, it * BK, f0 / 64 + 4, c.e);
                        } else {
#pragma unroll
                            for (int j = 0; j < G::a_bytes / CHUNK; ++j)
                                tma_load_3d_pair(a_dst + j * CHUNK, &tmW, bar,
                                                 f0 + (MODE == SWIGLU && !WIDE ? j * 128 : j * 64 + (MODE == STORE ? j / 2 * 128 : 0)),
                                                 it * BK, c.e);
                        }
                    }
                    if (p.src == nullptr) {
                        tma_load_3d_pair(b_dst, &tmX.m[box.first], bar, it * BK, row0, 0);
                        if (box.second >= 0)
                            tma_load_3d_pair(b_dst + (1024 << box.first), &tmX.m[box.second], bar, it * BK, row0 + (8 << box.first), 0);
                    }
                }
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (ok) {
            // every stage's last use released: the commits' arrivals, possibly from the other SM, have landed
            for (int i = 0; i < S; ++i) {
                if (!wait_warp(p, empty + stage, phase ^ 1u, kWhereDrain)) break;
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        } else if (lane == 0) {
            if (leader) {
                for (int s = 0; s < S; ++s)  // the leader's barriers count both CTAs' copies: wait for all of them
                    if (armed & (1u << s))
                        wait(p, full + s, (last_parity >> s) & 1u, kWhereDrain);
            } else {
                spin_ns(200000);  // let this CTA's last copies land before either CTA can exit
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            if (leader) {
                // -------------------------------------------------------- MMA issuer (leader)
                const uint64_t a0 = W_MN ? sdesc_sw128(smem_u32(sA), CHUNK, 1024) : sdesc_sw128(smem_u32(sA), 16, 1024);
                const uint64_t b0 = sdesc_sw128(smem_u32(sB), 16, 1024);
                constexpr uint64_t a_step = W_MN ? (2048 >> 4) : (32 >> 4);
                int stage = 0, lt = 0, e = 0;
                uint32_t phase = 0;
                bool ok = true;
                for (int i = 0, t; (t = round_tile<WIDE>(i, cluster_id, n_clusters)) < n_tiles && ok; ++i, ++lt) {
                    const Tile c = decode<TN>(p, tab, t, e);
                    const uint32_t idesc = idesc_bf16_f32(2 * BM, (c.n + 15) & ~15, W_MN, false);
                    const int acc = WIDE ? 0 : lt & 1;
                    const uint32_t turn = WIDE ? lt & 1 : (lt >> 1) & 1;
                    if (!wait(p, tempty + acc, turn ^ 1u, kWhereMma)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + acc * 256;
                    for (int it = 0; it < p.kb; ++it) {
                        ok = wait(p, full + stage, phase, kWhereMma);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t a = a0 + static_cast<uint64_t>(stage * (G::a_bytes >> 4));
                        const uint64_t b = b0 + static_cast<uint64_t>(stage * (G::b_bytes >> 4));
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk) {
                            umma_f16_pair(d, a + kk * a_step, b + kk * 2, idesc, (it | kk) != 0 ? 1u : 0u);
                            if constexpr (WIDE)
                                umma_f16_pair(d + 256, a + (BM * 128 >> 4) + kk * a_step, b + kk * 2, idesc, (it | kk) != 0 ? 1u : 0u);
                        }
                        umma_commit_pair_mc(empty + stage, 0x3);
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (ok) umma_commit_pair_mc(tfull + acc, 0x3);
                }
                umma_commit_pair_mc(drain, 0x3);
                // the accumulators' last releases land before this CTA can exit
                if (WIDE) ok = ok && wait(p, tempty, (lt & 1) ^ 1u, kWhereDrain);
                for (int i = 0; !WIDE && ok && i < 2; ++i, ++lt)
                    ok = wait(p, tempty + (lt & 1), ((lt >> 1) & 1) ^ 1u, kWhereDrain);
            }
            wait(p, drain, 0, kWhereDrain);
        }
    } else if (warp < EPI_WARP) {
        if (p.src != nullptr) {
            // ------------------------------------------------------------ gathered rows (both CTAs)
            constexpr int PER = TN / 16;  // copies of a warp at most
            int stage = 0, e = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint32_t full0 = mapa_shared(smem_u32(full), 0), dst0 = smem_u32(sB) + (warp - 2) * 512;
            for (int i = 0, t; (t = round_tile<WIDE>(i, cluster_id, n_clusters)) < n_tiles && ok; ++i) {
                const Tile c = decode<TN>(p, tab, t, e);
                const int half = ((c.n + 15) & ~15) / 2, copies = half / 8;  // (half is a multiple of 8)
                const int row0 = c.row0 + static_cast<int>(prank) * half + (warp - 2) * 4;
                int4 at[PER];
                gather_rows(p, row0, c.row0 + c.n - 1, copies, at);
                for (int it = 0; it < p.kb; ++it) {
                    if (!wait_warp(p, empty + stage, phase ^ 1u, kWhereProducer)) {
                        ok = false;
                        break;
                    }
                    if (elect_one())
                        gather_some<true, 0, PER>(copies, dst0 + stage * G::b_bytes, &tmX.m[0], full0 + stage * 8, it * BK, at);
                    __syncwarp();
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) spin_ns(200000);  // let the last copies land before either CTA can exit
        }
    } else {
        // ---------------------------------------------------------------- epilogue (both CTAs)
        const int q = warp & 3, half = (warp - EPI_WARP) >> 2;
        const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
        uint8_t* buf = sE + (warp - EPI_WARP) * G::epi;
        const uint32_t sbuf = smem_u32(buf);
        int lt = 0, e = 0;
        for (int i = 0, t; (t = round_tile<WIDE>(i, cluster_id, n_clusters)) < n_tiles; ++i, ++lt) {
            const Tile c = decode<TN>(p, tab, t, e);
            const int acc = WIDE ? 0 : lt & 1;
            // the saved pre-activations of 32 tokens are loaded a step ahead, the first ones while the products are computed
            [[maybe_unused]] uint4 g4[4], u4[4];
            [[maybe_unused]] float hg[2][16], hu[2][16];
            [[maybe_unused]] auto ahead16 = [&](int c0, float (&g)[16], float (&u)[16]) {  // (H32: of 16 tokens)
                const int f0 = c.mb * 256 + static_cast<int>(prank) * BM + q * 32;
                const bool in = c0 < (half + 1) * (TN / 2) && f0 < p.features;
                load_rows_f32(static_cast<const float*>(p.h_in) + (c.row0 + c0) * p.h_ld + static_cast<long long>(f0 >> 7) * 256 + (f0 & 127) + lane,
                              p.h_ld, in ? c.n - c0 : 0, g, u);
            };
            [[maybe_unused]] auto ahead = [&](int c0) {
                const int f0 = c.mb * 256 + static_cast<int>(prank) * BM + q * 32, n = min(c.n - c0, 32);
                const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(p.h_in) + (c.row0 + c0) * p.h_ld + static_cast<long long>(f0 >> 7) * 256 + (f0 & 127);
                if (c0 < (half + 1) * (TN / 2)) {
                    rows_load(h, p.h_ld, n, p.features - f0, lane, g4);
                    rows_load(h + 128, p.h_ld, n, p.features - f0, lane, u4);
                }
            };
            if constexpr (MODE == DSWIGLU && H32) {
                ahead16(half * (TN / 2), hg[0], hu[0]);
                ahead16(half * (TN / 2) + 16, hg[1], hu[1]);
            } else if constexpr (MODE == DSWIGLU) {
                ahead(half * (TN / 2));
            }
            int okw = 0;
            if (lane == 0) okw = wait(p, tfull + acc, WIDE ? lt & 1 : (lt >> 1) & 1, kWhereEpilogue);
            okw = __shfl_sync(0xFFFFFFFFu, okw, 0);
            if constexpr (MODE == SWIGLU && !WIDE) okw = pair_and(1 + half * 2 + (q & 1), okw);  // both or neither go on to meet
            if (!okw) break;
            tc_fence_after();
          for (int part = 0; part < (WIDE && MODE == STORE ? 2 : 1); ++part) {  // (the wide tile's accumulators)
            // features f0 .. f0 + 31 (SWIGLU: of gate and up; narrow, this warp's the gate where q < 2)
            const int f0 = MODE == SWIGLU && !WIDE ? c.mb * 128 + static_cast<int>(prank) * 64 + (q & 1) * 32
                                                   : c.mb * G::f + part * 256 + static_cast<int>(prank) * BM + q * 32;
            const int nf = min(p.features - f0, 32);
            const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + (acc + part) * 256;
            const long long packed = static_cast<long long>(f0 >> 7) * 256 + (f0 & 127) + (MODE == SWIGLU && !WIDE ? (q >> 1) * 128 : 0);
            [[maybe_unused]] float bias[4], bias_up[4], own = 0.0f, own_up = 0.0f;  // (H32: of this lane's feature)
            if constexpr (MODE != DSWIGLU) {
                const __nv_bfloat16* at = p.bias == nullptr ? nullptr : p.bias + c.e * p.bias_ld + (MODE == SWIGLU ? packed : f0);
                if constexpr (H32)
                    if (at != nullptr && lane < nf) {
                        own = __bfloat162float(at[lane]);
                        if (WIDE) own_up = __bfloat162float(at[128 + lane]);
                    }
                load_bias(at, nf, lane, bias);
                if constexpr (MODE == SWIGLU && WIDE) load_bias(at == nullptr ? nullptr : at + 128, nf, lane, bias_up);
            }
            for (int c0 = half * (TN / 2); c0 < (half + 1) * (TN / 2) && c0 < c.n && nf > 0; c0 += 32) {
                const int n = min(c.n - c0, 32);
                const long long row = c.row0 + c0;
                if constexpr (MODE == STORE) {
                    if (p.out_f32) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(lanes + c0, r);
                        const float b = p.bias != nullptr && lane < nf ? __bfloat162float(p.bias[c.e * p.bias_ld + f0 + lane]) : 0.0f;
                        tmem_ld_wait();
                        float* dst = static_cast<float*>(p.out) + row * p.ld + f0 + lane;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j < n && lane < nf) dst[j * p.ld] = __uint_as_float(r[j]) + b;
                        continue;
                    }
                }
                if constexpr (MODE == SWIGLU && H32) {
                    float* h = static_cast<float*>(p.h_out) + row * p.h_ld + packed + lane;
                    store_rows_f32(lanes + c0, own, h, p.h_ld, n);
                    if constexpr (WIDE) store_rows_f32(lanes + 256 + c0, own_up, h + 128, p.h_ld, n);
                }
                if constexpr (MODE == DSWIGLU && H32) {
                    uint32_t d[32];
                    tmem_ld_32x32b_x32(lanes + c0, d);
                    tmem_ld_wait();
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + row * p.ld + packed + lane;
                    gated_rows<0>(d, hg[0], hu[0], dst, p.ld, n);
                    ahead16(c0 + 32, hg[0], hu[0]);
                    gated_rows<16>(d, hg[1], hu[1], dst + 16 * p.ld, p.ld, n - 16);
                    ahead16(c0 + 48, hg[1], hu[1]);
                    continue;
                }
                uint32_t a[16], b[16], lo[8], hi[8];
                load_frags(lanes + c0, a, b);
                if constexpr (MODE == STORE) {
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float ba = bias[i & 1], bb = bias[2 + (i & 1)];
                        lo[i] = tc::pack_bf16x2(__uint_as_float(a[2 * i]) + ba, __uint_as_float(a[2 * i + 1]) + ba);
                        hi[i] = tc::pack_bf16x2(__uint_as_float(b[2 * i]) + bb, __uint_as_float(b[2 * i + 1]) + bb);
                    }
                    put_rows(buf, static_cast<__nv_bfloat16*>(p.out) + row * p.ld + f0, p.ld, lo, hi, n, nf, lane);
                } else if constexpr (MODE == SWIGLU && WIDE) {
                    uint32_t ua[16], ub[16];
                    load_frags(lanes + 256 + c0, ua, ub);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = (i >> 1) & 1;
                        a[i] = __float_as_uint(__uint_as_float(a[i]) + bias[j]);
                        b[i] = __float_as_uint(__uint_as_float(b[i]) + bias[2 + j]);
                        ua[i] = __float_as_uint(__uint_as_float(ua[i]) + bias_up[j]);
                        ub[i] = __float_as_uint(__uint_as_float(ub[i]) + bias_up[2 + j]);
                    }
                    if (!H32 && p.h_out != nullptr) {
                        __nv_bfloat16* h = static_cast<__nv_bfloat16*>(p.h_out) + row * p.h_ld + packed;
                        pack_frags(a, b, lo, hi);
                        put_rows(buf, h, p.h_ld, lo, hi, n, nf, lane);
                        pack_frags(ua, ub, lo, hi);
                        put_rows(buf, h + 128, p.h_ld, lo, hi, n, nf, lane);
                    }
                    gate_frags(a, b, ua, ub, lo, hi);
                    put_rows(buf, static_cast<__nv_bfloat16*>(p.out) + row * p.ld + f0, p.ld, lo, hi, n, nf, lane);
                } else if constexpr (MODE == SWIGLU) {
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = (i >> 1) & 1;
                        a[i] = __float_as_uint(__uint_as_float(a[i]) + bias[j]);
                        b[i] = __float_as_uint(__uint_as_float(b[i]) + bias[2 + j]);
                    }
                    // the two warps of a pair of (gate, up) lanes and the same tokens: 64 threads
                    const int pair = half * 2 + (q & 1);
                    uint4* pass = reinterpret_cast<uint4*>(sE + EPI_WARPS * G::epi + pair * 4096) + lane;
                    if (q >= 2) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            pass[i * 32] = make_uint4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
                            pass[(4 + i) * 32] = make_uint4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
                        }
                    }
                    pair_sync(1 + pair);
                    uint32_t ua[16], ub[16];
                    if (q < 2) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 u = pass[i * 32], v = pass[(4 + i) * 32];
                            ua[4 * i] = u.x, ua[4 * i + 1] = u.y, ua[4 * i + 2] = u.z, ua[4 * i + 3] = u.w;
                            ub[4 * i] = v.x, ub[4 * i + 1] = v.y, ub[4 * i + 2] = v.z, ub[4 * i + 3] = v.w;
                        }
                    }
                    pair_sync(1 + pair);  // read: the next ones may be written
                    if (!H32 && p.h_out != nullptr) {
                        pack_frags(a, b, lo, hi);
                        put_rows(buf, static_cast<__nv_bfloat16*>(p.h_out) + row * p.h_ld + packed, p.h_ld, lo, hi, n, nf, lane);
                    }
                    if (q < 2) {
                        gate_frags(a, b, ua, ub, lo, hi);
                        put_rows(buf, static_cast<__nv_bfloat16*>(p.out) + row * p.ld + f0, p.ld, lo, hi, n, nf, lane);
                    }
                } else {
                    stage_load(buf, g4, lane);
                    stage_load(buf + STAGE, u4, lane);
                    __syncwarp();
                    ahead(c0 + 32);
                    uint32_t glo[8], ghi[8], ulo[8], uhi[8];
                    stage_get(sbuf, glo, ghi, lane);
                    stage_get(sbuf + STAGE, ulo, uhi, lane);
                    tmem_ld_wait();
                    __syncwarp();
                    auto pair = [&](uint32_t d0, uint32_t d1, uint32_t& g, uint32_t& u) {
                        float g0, g1, u0, u1;
                        gated_gradient(__uint_as_float(d0), lo_f(g), lo_f(u), g0, u0);
                        gated_gradient(__uint_as_float(d1), hi_f(g), hi_f(u), g1, u1);
                        g = tc::pack_bf16x2(g0, g1);
                        u = tc::pack_bf16x2(u0, u1);
                    };
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        pair(a[2 * i], a[2 * i + 1], glo[i], ulo[i]);
                        pair(b[2 * i], b[2 * i + 1], ghi[i], uhi[i]);
                    }
                    stage_put(sbuf, glo, ghi, lane);
                    stage_put(sbuf + STAGE, ulo, uhi, lane);
                    __syncwarp();
                    __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.out) + row * p.ld + packed;
                    stage_store(buf, d, p.ld, n, nf, lane);
                    stage_store(buf + STAGE, d + 128, p.ld, n, nf, lane);
                    __syncwarp();
                }
            }
          }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + acc * 8);
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

// ---------------------------------------------------------------- few rows
// The rows kernel's products for few rows an expert, where reading the weights bounds the time: one CTA per tile of 128 features
// and at most 64 tokens, two CTAs an SM, not persistent, so that many copies are in flight and the SMs even out.  Clusters of
// up to 8 CTAs split the contraction; groups of 8 tokens go to the cluster's CTAs in turn, which add the partial sums through
// distributed shared memory in the order of the ranks.  (4 tokens on 8 of 64 experts, 1024 x 8192: 134 MB of weights, 20 us
// at a copy's rate.)
constexpr int FEW_TN = 64, FEW_STAGES = 4, FEW_THREADS = 256;
constexpr int FEW_A = BM * 128, FEW_B = FEW_TN * 128, FEW_STAGE = FEW_A + FEW_B;
constexpr int FEW_SUMS = 8 * 4096;  // partial sums on their way: 8 (rank, group of 8 tokens) of 128 lanes
constexpr int FEW_SMEM = 1024 + FEW_STAGES * FEW_STAGE + (2 * FEW_STAGES + 2) * 8 + 64;
static_assert(FEW_TN >= 32 && FEW_SUMS <= FEW_STAGES * FEW_STAGE && 2 * (FEW_SMEM + 1024) <= 227 * 1024, "few kernel shared memory");

template <bool W_MN, int MODE, bool H32 = false>
__global__ void __launch_bounds__(FEW_THREADS, 2)
    few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ Boxes tmX, const Args p) {
    constexpr int S = FEW_STAGES;
    constexpr bool GATED = MODE == SWIGLU;
    static_assert(MODE == STORE || W_MN == GATED);
    using HT = PreAct<H32>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + S * FEW_A;
    Carve carve{smem + S * FEW_STAGE};
    uint64_t* full = carve.take<uint64_t>(S);
    uint64_t* empty = carve.take<uint64_t>(S);
    uint64_t* tfull = carve.take<uint64_t>(1);
    uint32_t* tmem_slot = carve.take<uint32_t>(2);
    int* tile = carve.take<int>(4);   // expert, first row, rows, feature block
    int* sums = carve.take<int>(8);   // tiles of each warp's experts

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t ranks;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    const int n_ranks = static_cast<int>(ranks), rank = static_cast<int>(cluster_ctarank());

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(tfull, 1);
        fence_mbarrier_init();
        fence_proxy_async_smem();
        tma_prefetch_desc(&tmW);
        tile[2] = 0;
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, FEW_TN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    // this cluster's tile: feature blocks of an expert's first 64 tokens, of its next ..; threads have four experts each
    {
        const int t = blockIdx.x / n_ranks, e0 = threadIdx.x * 4;
        int off[5], n[4], mine = 0;
#pragma unroll
        for (int i = 0; i < 5; ++i) off[i] = e0 + i <= p.experts ? p.offsets[e0 + i] : 0;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            const int c = min(max(off[i], 0), p.rows);
            bad |= c != off[i];
            off[i] = c;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool there = e0 + i < p.experts;
            bad |= there && off[i + 1] < off[i];
            n[i] = there ? max(off[i + 1] - off[i], 0) : 0;
            mine += (n[i] + FEW_TN - 1) / FEW_TN * p.m_blocks;
        }
        if (bad && blockIdx.x == 0) record_cut(p);
        int sum = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
            if (lane >= d) sum += o;
        }
        if (lane == 31) sums[warp] = sum;
        __syncthreads();
        for (int w = 0; w < warp; ++w) sum += sums[w];
        int first = sum - mine;
        if (t >= first && t < sum) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int nt = (n[i] + FEW_TN - 1) / FEW_TN, tiles = nt * p.m_blocks;
                if (t >= first && t < first + tiles) {
                    const int tb = (t - first) / p.m_blocks, sz = tile_tokens<FEW_TN>(n[i]);
                    tile[0] = e0 + i;
                    tile[1] = off[i] + tb * sz;
                    tile[2] = min(sz, n[i] - tb * sz);
                    tile[3] = (t - first) - tb * p.m_blocks;
                }
                first += tiles;
            }
        }
        __syncthreads();
    }
    const Tile c{tile[0], tile[3], tile[1], tile[2]};
    const int nn = (c.n + 15) & ~15;
    // what this thread stores: column `col` of its rows (GATED: of the gate; the up feature is 128 on), feature f
    const int l = threadIdx.x & 127;
    const int f = GATED ? c.mb * 64 + (l & 63) : c.mb * 128 + l;
    const long long col = GATED ? static_cast<long long>(c.mb >> 1) * 256 + (c.mb & 1) * 64 + (l & 63) : f;
    float bias = 0.0f, bias_up = 0.0f;
    if (c.n > 0 && warp >= EPI_WARP && p.bias != nullptr && f < p.features) {
        bias = __bfloat162float(p.bias[c.e * p.bias_ld + col]);
        if (GATED) bias_up = __bfloat162float(p.bias[c.e * p.bias_ld + col + 128]);
    }
    // DSWIGLU: the pre-activations of eight tokens of a group, the first one's while the products are computed
    [[maybe_unused]] float hg[8], hu[8];
    [[maybe_unused]] const long long packed = static_cast<long long>(f >> 7) * 256 + (f & 127);
    [[maybe_unused]] auto saved = [&](int g) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = g * 8 + j < c.n && f < p.features;
            const HT* h = static_cast<const HT*>(p.h_in) + (c.row0 + g * 8 + j) * p.h_ld + packed;
            hg[j] = in ? as_f32(h[0]) : 0.0f;
            hu[j] = in ? as_f32(h[128]) : 0.0f;
        }
    };
    if constexpr (MODE == DSWIGLU)
        if (warp >= EPI_WARP) saved(rank);
    const int k0 = p.kb * rank / n_ranks, k1 = p.kb * (rank + 1) / n_ranks;
    bool ok = true;

    if (c.n > 0) {
        if (warp == 0) {
            // ------------------------------------------------------------ producer
            const Halves box(nn);
            const uint32_t bytes = FEW_A + (p.src == nullptr ? box.rows() : nn) * 128;
            int stage = 0;
            uint32_t phase = 0;
            for (int it = k0; it < k1; ++it) {
                ok = wait_warp(p, empty + stage, phase ^ 1u, kWhereProducer);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t bar = smem_u32(full + stage);
                    uint8_t *a_dst = sA + stage * FEW_A, *b_dst = sB + stage * FEW_B;
                    mbar_arrive_expect_tx(full + stage, bytes);
                    if constexpr (GATED) {
                        tma_load_3d_bar(a_dst, &tmW, bar, (c.mb >> 1) * 256 + (c.mb & 1) * 64, it * BK, c.e);
                        tma_load_3d_bar(a_dst + CHUNK, &tmW, bar, (c.mb >> 1) * 256 + (c.mb & 1) * 64 + 128, it * BK, c.e);
                    } else if constexpr (!W_MN) {
                        tma_load_3d_bar(a_dst, &tmW, bar, it * BK, c.mb * BM, c.e);
                    } else if (p.chunked) {
                        tma_load_4d(a_dst, &tmW, full + stage, 0, it * BK, c.mb * 2, c.e);
                    } else {
                        tma_load_3d_bar(a_dst, &tmW, bar, c.mb * 128, it * BK, c.e);
                        tma_load_3d_bar(a_dst + CHUNK, &tmW, bar, c.mb * 128 + 64, it * BK, c.e);
                    }
                    if (p.src == nullptr) {
                        tma_load_3d_bar(b_dst, &tmX.m[box.first], bar, it * BK, c.row0, 0);
                        if (box.second >= 0)
                            tma_load_3d_bar(b_dst + (1024 << box.first), &tmX.m[box.second], bar, it * BK, c.row0 + (8 << box.first), 0);
                    }
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            if (lane == 0) {
                const uint64_t a0 = sdesc_sw128(smem_u32(sA), W_MN ? CHUNK : 16, 1024), b0 = sdesc_sw128(smem_u32(sB), 16, 1024);
                const uint32_t idesc = idesc_bf16_f32(BM, nn, W_MN, false);
                int stage = 0;
                uint32_t phase = 0;
                for (int it = k0; it < k1; ++it) {
                    ok = wait(p, full + stage, phase, kWhereMma);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t a = a0 + static_cast<uint64_t>(stage * (FEW_A >> 4)), b = b0 + static_cast<uint64_t>(stage * (FEW_B >> 4));
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk)
                        umma_f16(tmem, a + kk * ((W_MN ? 2048 : 32) >> 4), b + kk * 2, idesc, it > k0 || kk > 0 ? 1u : 0u);
                    umma_commit(empty + stage);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                umma_commit(tfull);
            }
        } else if (warp < EPI_WARP && p.src != nullptr) {
            // ------------------------------------------------------------ gathered rows
            const int copies = nn / 8;
            int4 at[FEW_TN / 8];
            gather_rows(p, c.row0 + (warp - 2) * 4, c.row0 + c.n - 1, copies, at);
            int stage = 0;
            uint32_t phase = 0;
            for (int it = k0; it < k1; ++it) {
                ok = wait_warp(p, empty + stage, phase ^ 1u, kWhereProducer);
                if (!ok) break;
                if (elect_one())
                    gather_some<false, 0, FEW_TN / 8>(copies, smem_u32(sB) + stage * FEW_B + (warp - 2) * 512, &tmX.m[0], smem_u32(full + stage),
                                               it * BK, at);
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        __syncwarp();
        // every warp waits for the products: the ring is then free for the sums
        const bool done = wait_warp(p, tfull, 0, kWhereEpilogue);
        ok = ok && done;
        tc_fence_after();
        fence_proxy_async_all();
    }
    if (n_ranks > 1) cluster_sync_all();  // all of the cluster's rings
    // slot (rank, group / ranks) of the CTA that finishes a group: [token][lane]
    const int groups = (c.n + 7) / 8, per = (groups + n_ranks - 1) / n_ranks;
    float* part = reinterpret_cast<float*>(smem);
    if (c.n > 0 && warp >= EPI_WARP) {
        const int q = warp & 3;
        for (int g0 = 0; g0 < groups; g0 += 4) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + g0 * 8, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int g = g0 + i;
                if (g >= groups) break;
                const uint32_t at = smem_u32(part + ((rank * per + g / n_ranks) * 8) * 128 + q * 32 + lane);
                const uint32_t to = mapa_shared(at, static_cast<uint32_t>(g % n_ranks));
#pragma unroll
                for (int j = 0; j < 8; ++j) st_cluster_u32(to + j * 512, r[i * 8 + j]);
            }
        }
        tc_fence_before();
    }
    if (n_ranks > 1) cluster_sync_all();
    else __syncthreads();
    if (c.n > 0 && warp >= EPI_WARP && __all_sync(0xFFFFFFFFu, ok) && f < p.features) {
        // a thread adds eight tokens of its lane at once (GATED: four, of gate and up), in the order of the ranks
        constexpr int AT_ONCE = GATED ? 4 : 8;
        const int j0 = GATED ? (l >> 6) * 4 : 0, lane0 = GATED ? l & 63 : l;
        for (int g = rank; g < groups; g += n_ranks) {
            float v[AT_ONCE], u[AT_ONCE];
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) v[j] = u[j] = 0.0f;
            if constexpr (MODE == DSWIGLU)
                if (g != rank) saved(g);
            for (int r = 0; r < n_ranks; ++r) {
                const float* at = part + ((r * per + g / n_ranks) * 8 + j0) * 128 + lane0;
#pragma unroll
                for (int j = 0; j < AT_ONCE; ++j) {
                    v[j] += at[j * 128];
                    if (GATED) u[j] += at[j * 128 + 64];
                }
            }
            const int n = c.n - g * 8 - j0;
            const long long row = c.row0 + g * 8 + j0;
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {
                if (j >= n) break;
                const float x = v[j] + bias;
                if constexpr (MODE == DSWIGLU) {
                    __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.out) + (row + j) * p.ld + packed;
                    float dg, du;
                    gated_gradient(x, hg[j], hu[j], dg, du);
                    d[0] = __float2bfloat16_rn(dg);
                    d[128] = __float2bfloat16_rn(du);
                } else if constexpr (GATED) {
                    const float up = u[j] + bias_up;
                    if (p.h_out != nullptr) {
                        HT* h = static_cast<HT*>(p.h_out) + (row + j) * p.h_ld + col;
                        store_as(h, x);
                        store_as(h + 128, up);
                    }
                    static_cast<__nv_bfloat16*>(p.out)[(row + j) * p.ld + f] = __float2bfloat16_rn(x * tc::sigmoid_approx(x) * up);
                } else if (p.out_f32) {
                    static_cast<float*>(p.out)[(row + j) * p.ld + f] = x;
                } else {
                    static_cast<__nv_bfloat16*>(p.out)[(row + j) * p.ld + f] = __float2bfloat16_rn(x);
                }
            }
        }
    }
    if (!ok) spin_ns(200000);  // copies that were not waited for land before this CTA exits
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, FEW_TN);
    }
}

// ---------------------------------------------------------------- dw kernel
// dW[e] = X_e^T dY_e: both operands have the rows as their contraction, 64 to a stage, and come by TMA; gathered rows of X
// from warps 2 and 3, 64 features each.  Where an expert's last block ends inside a stage warps 12 and 13 copy it, both
// operands, by cp.async: the rows behind the last, the next expert's, are zeros in shared memory then (in both operands,
// since a zero times the other's infinity would be a NaN).  Warp 14 waits for these copies, makes them visible to the tensor
// cores and reports to the leader: the proxy fence that it takes holds up a warp that has copied (8192 rows on 64 experts,
// 1024 x 2048 in order: 87 us with the fence in the copying warps, 68 with it in a warp of its own).
//
// A lane's place in a block of rows of 128 bytes, row r0 + 4 j: piece ^ (row % 8) of the row, as the swizzle has it.
struct Lane {
    int piece, r0;
    __device__ __forceinline__ Lane() : piece(threadIdx.x & 7), r0((threadIdx.x >> 3) & 3) {}
    __device__ __forceinline__ uint32_t at(int j) const {
        return static_cast<uint32_t>(j * 512 + r0 * 128 + ((piece ^ (r0 + 4 * (j & 1))) << 4));
    }
};
// WIDE: two accumulators, 512 columns of dY, for gathered rows, as in the rows kernel.
//
// The tensor cores' additions drop what lies below the running sum's last places, always towards zero: an error that grows
// with the steps (700000 rows of terms of one sign: 4.6e-3 of the sum).  fp32 gradients are therefore computed a chunk of each
// expert's rows to a launch (262144, as in the dense weight gradients), the later ones added to the output, rounded to nearest.
constexpr int DW_A = BM * 128;
constexpr int TAIL_WARP = EPI_WARP + EPI_WARPS, TAIL_WARPS = 2;  // and a warp behind them that reports
constexpr int DW_THREADS = THREADS + 32 * (TAIL_WARPS + 1);
template <bool WIDE>
struct DwGeom {
    static constexpr int n = WIDE ? 512 : 256;           // columns of a tile
    static constexpr int parts = WIDE ? 2 : 1;           // accumulators of a tile, of 256 columns
    static constexpr int b_bytes = parts * BM * 128;     // this CTA's half of each
    static constexpr int stage = DW_A + b_bytes;
    static constexpr int stages = WIDE ? 4 : 6;
    static constexpr int smem = 1024 + stages * stage + EPI_WARPS * STAGE + 32 * 16 + (most_barriers + 1) * 8 + TABLE;
    static_assert(smem <= 227 * 1024, "dw kernel shared memory");
    static_assert(5 * stages + 5 <= most_barriers);
};

// 64 bytes of each of a warp's 32 rows through its box of shared memory to the output: a store of its own per lane would
// touch 32 rows an instruction.  (8192 rows on 64 experts, 1024 x 2048, whose contractions are short: 84 us
// so, 80 through the boxes; gathered 129 and 108.)
__device__ __forceinline__ void put_box(uint8_t* box, const CUtensorMap* map, const uint32_t (&w)[32], int x, int y, int z, int lane,
                                        bool add) {
    if (lane == 0) bulk_wait_group_read<0>();  // the box has been read
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(box + stage_at(lane, i)) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (add) tma_add_f32_3d(map, box, x, y, z);
        else tma_store_3d(map, box, x, y, z);
        bulk_commit_group();
    }
}

template <bool WIDE>
__global__ void __launch_bounds__(DW_THREADS, 1)
    dw_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmO,
              const Args p) {
    using G = DwGeom<WIDE>;
    constexpr int S = G::stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + S * DW_A;
    uint8_t* sE = smem + S * G::stage;
    Carve carve{sE + EPI_WARPS * STAGE};
    int4* rows4 = carve.take<int4>(32);             // warps 2 and 3: a block's tokens
    uint64_t* full = carve.take<uint64_t>(S);
    uint64_t* empty = carve.take<uint64_t>(S);
    uint64_t* begin = carve.take<uint64_t>(S);      // the stage is for an expert's last block: to the tail (and gather) warps
    uint64_t* lfull = carve.take<uint64_t>(S);      // it is copied in this CTA: to the warp behind them
    uint64_t* gfull = carve.take<uint64_t>(S);      // leader: in both CTAs
    uint64_t* tfull = carve.take<uint64_t>(2);
    uint64_t* tempty = carve.take<uint64_t>(2);
    uint64_t* drain = carve.take<uint64_t>(1);
    uint32_t* tmem_slot = carve.take<uint32_t>(2);
    Table tab(carve.take<int>(TABLE / 4));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t prank = cluster_ctarank();
    const bool leader = prank == 0;
    const int cluster_id = blockIdx.x / 2, n_clusters = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
            mbar_init(lfull + s, 32 * TAIL_WARPS);
            mbar_init(gfull + s, 2 * (1 + (p.src != nullptr ? 2 : 0)));
            mbar_init(begin + s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull + a, 1);
            mbar_init(tempty + a, 2 * EPI_WARPS);
        }
        mbar_init(drain, 1);
        fence_mbarrier_init();
        fence_proxy_async_smem();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmY);
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
    tab.build<DW_THREADS, true>(p, [&](int) { return p.m_blocks * p.n_blocks; }, [](int n) { return n; });
    const int n_tiles = tab.first[p.experts];  // every expert has its tiles, one without rows to write zeros
    const int per_expert = p.m_blocks * p.n_blocks;
    // an expert's rows of this launch
    auto rows_of = [&](int e) { return min(max(tab.count(e) - p.skip, 0), p.most); };
    auto first_of = [&](int e) { return rows_of(e) > 0 ? tab.off[e] + p.skip : 0; };
    // tile t: expert, block of K, block of N; groups of GROUP blocks of K walked together
    auto place = [&](int t, int& e, int& mb, int& nb) {
        const int i = t / per_expert, l = t - i * per_expert, per_group = GROUP * p.n_blocks;
        e = tab.at[i];
        const int g = l / per_group, r = l - g * per_group, gm = min(p.m_blocks - g * GROUP, GROUP);
        mb = g * GROUP + r % gm;
        nb = r / gm;
    };

    if (warp == 0) {
        // ---------------------------------------------------------------- producer (both CTAs), a whole warp
        int stage = 0;
        uint32_t phase = 0, armed = 0, last_parity = 0;
        bool ok = true;
        const uint32_t full0 = mapa_shared(smem_u32(full), 0);
        for (int i = 0, t; (t = round_tile<true>(i, cluster_id, n_clusters)) < n_tiles && ok; ++i) {
            int e, mb, nb;
            place(t, e, mb, nb);
            const int n = rows_of(e), base = first_of(e), kb = (n + BK - 1) / BK;
            const int a0 = mb * 256 + static_cast<int>(prank) * BM, b0 = nb * G::n + static_cast<int>(prank) * BM;
            for (int it = 0; it < kb; ++it) {
                const bool tail = (it + 1) * BK > n;
                if (!wait_warp(p, empty + stage, phase ^ 1u, kWhereProducer)) {
                    ok = false;
                    break;
                }
                uint8_t* a_dst = sA + stage * DW_A;
                uint8_t* b_dst = sB + stage * G::b_bytes;
                const uint32_t bar = full0 + stage * 8;
                if (lane == 0) {
                    if (leader) {
                        mbar_arrive_expect_tx(full + stage, tail ? 0 : 2 * G::stage);
                        armed |= 1u << stage;
                        last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
                    }
                    if (tail) {
                        mbar_arrive(begin + stage);
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (p.src == nullptr) tma_load_3d_pair(a_dst + j * CHUNK, &tmX, bar, a0 + j * 64, base + it * BK, 0);
#pragma unroll
                        for (int j = 0; j < 2 * G::parts; ++j)
                            tma_load_3d_pair(b_dst + j * CHUNK, &tmY, bar, b0 + j / 2 * 256 + j % 2 * 64, base + it * BK, 0);
                    }
                }
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (ok) {
            for (int i = 0; i < S; ++i) {
                if (!wait_warp(p, empty + stage, phase ^ 1u, kWhereDrain)) break;
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        } else if (lane == 0) {
            for (int s = 0; leader && s < S; ++s)
                if (armed & (1u << s)) wait(p, full + s, (last_parity >> s) & 1u, kWhereDrain);
            if (!leader) spin_ns(200000);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            if (leader) {
                // -------------------------------------------------------- MMA issuer (leader)
                constexpr uint32_t idesc = idesc_bf16_f32(2 * BM, 2 * BM, true, true);
                const uint64_t a0 = sdesc_sw128(smem_u32(sA), CHUNK, 1024), b0 = sdesc_sw128(smem_u32(sB), CHUNK, 1024);
                int stage = 0, lt = 0;
                uint32_t phase = 0, g_parity = 0;  // a stage's next phase of gfull
                bool ok = true;
                for (int i = 0, t; (t = round_tile<true>(i, cluster_id, n_clusters)) < n_tiles && ok; ++i) {
                    int e, mb, nb;
                    place(t, e, mb, nb);
                    const int n = rows_of(e), kb = (n + BK - 1) / BK;
                    if (kb == 0) continue;
                    const int acc = WIDE ? 0 : lt & 1;
                    const uint32_t turn = (WIDE ? lt & 1 : (lt >> 1) & 1) ^ 1u;
                    const uint32_t d = tmem_base + acc * 256;
                    auto arrived = [&](int it) {  // the operands of block it
                        bool in = wait(p, full + stage, phase, kWhereMma);
                        if (in && (it + 1) * BK > n) {
                            in = mbar_wait_bounded_cluster(gfull + stage, (g_parity >> stage) & 1u, p.status, p.timeout_ns, kWhereMma, false);
                            g_parity ^= 1u << stage;
                        }
                        tc_fence_after();
                        return in;
                    };
                    auto multiply = [&](int it, int part) {
                        const uint64_t a = a0 + static_cast<uint64_t>(stage * (DW_A >> 4));
                        const uint64_t b = b0 + static_cast<uint64_t>(stage * (G::b_bytes >> 4) + part * (BM * 128 >> 4));
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            umma_f16_pair(d + part * 256, a + kk * (2048 >> 4), b + kk * (2048 >> 4), idesc, (it | kk) != 0 ? 1u : 0u);
                    };
                    auto next = [&] {
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    };
                    ok = wait(p, tempty + acc, turn, kWhereMma);
                    if (!ok) break;
                    tc_fence_after();
                    int it = 0;
                    if constexpr (WIDE) {
                        // as many blocks as the ring holds into the first accumulator, while the second one is read out
                        const int first = min(kb, S), stage0 = stage;
                        const uint32_t phase0 = phase;
                        for (; it < first && ok; ++it) {
                            ok = arrived(it);
                            if (ok) multiply(it, 0);
                            next();
                        }
                        ok = ok && wait(p, tempty + 1, turn, kWhereMma);
                        if (!ok) break;
                        tc_fence_after();
                        stage = stage0;
                        phase = phase0;
                        for (int j = 0; j < first; ++j) {
                            multiply(j, 1);
                            umma_commit_pair_mc(empty + stage, 0x3);
                            next();
                        }
                    }
                    for (; it < kb; ++it) {
                        ok = arrived(it);
                        if (!ok) break;
#pragma unroll
                        for (int part = 0; part < G::parts; ++part) multiply(it, part);
                        umma_commit_pair_mc(empty + stage, 0x3);
                        next();
                    }
                    if (ok) umma_commit_pair_mc(tfull + acc, 0x3);
                    ++lt;
                }
                umma_commit_pair_mc(drain, 0x3);
                for (int i = 0; ok && i < 2; ++i)
                    ok = WIDE ? wait(p, tempty + i, (lt & 1) ^ 1u, kWhereDrain)
                              : wait(p, tempty + ((lt + i) & 1), (((lt + i) >> 1) & 1) ^ 1u, kWhereDrain);
            }
            wait(p, drain, 0, kWhereDrain);
        }
    } else if (warp < EPI_WARP) {
        if (p.src != nullptr) {
            // ------------------------------------------------------------ gathered rows (both CTAs)
            const uint32_t sa = smem_u32(sA), full0 = mapa_shared(smem_u32(full), 0), gfull0 = mapa_shared(smem_u32(gfull), 0);
            int4* const at = rows4 + (warp - 2) * 16;
            int stage = 0;
            uint32_t phase = 0, b_parity = 0;  // a stage's next phase of `begin`
            bool ok = true;
            for (int i = 0, t; (t = round_tile<true>(i, cluster_id, n_clusters)) < n_tiles && ok; ++i) {
                int e, mb, nb;
                place(t, e, mb, nb);
                const int n = rows_of(e), base = first_of(e), whole = n / BK, a0 = mb * 256 + static_cast<int>(prank) * BM;
                int2 next = make_int2(0, 0);
                auto look = [&](int it) {  // two tokens of block it, ahead of their use (and of their check, which waits for them)
                    if (it < whole) next = make_int2(p.src[base + it * BK + lane * 2], p.src[base + it * BK + lane * 2 + 1]);
                };
                look(0);
                for (int it = 0; it * BK < n; ++it) {
                    int4 rows[16];
                    if (it < whole) {
                        reinterpret_cast<int2*>(at)[lane] = make_int2(checked(p, next.x), checked(p, next.y));
                        look(it + 1);
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 16; ++j) rows[j] = at[j];
                        ok = wait_warp(p, empty + stage, phase ^ 1u, kWhereProducer);
                        if (!ok) break;
                        if (elect_one()) {
                            const uint32_t dst = sa + stage * DW_A + (warp - 2) * CHUNK;
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                tma_gather4<true>(dst + j * 512, &tmX, full0 + stage * 8, a0 + (warp - 2) * 64, rows[j]);
                        }
                        __syncwarp();
                    } else {
                        // A last block is not theirs, but they report it too: no stage passes without them, so that they can
                        // neither run ahead of the ring nor fall behind it (a barrier two phases on looks like the one before).
                        ok = wait_warp(p, begin + stage, (b_parity >> stage) & 1u, kWhereProducer);
                        if (!ok) break;
                        b_parity ^= 1u << stage;
                        if (lane == 0) mbar_arrive_cluster(gfull0 + stage * 8);
                    }
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) spin_ns(200000);  // let the last copies land before either CTA can exit
        }
    } else if (warp >= TAIL_WARP) {
        // ---------------------------------------------------------------- last blocks (both CTAs)
        // A lane has 16 bytes of every fourth row of 32, in each chunk of 64 columns.  The warps walk past the other blocks
        // without a look at `empty`, of which they could miss phases, and are called by the producer, once for each block that
        // cannot pass without them.
        const Lane l;
        const int r0 = (warp - TAIL_WARP) * 32;
        const uint32_t sa = smem_u32(sA), sb = smem_u32(sB), gfull0 = mapa_shared(smem_u32(gfull), 0);
        int stage = 0;
        uint32_t b_parity = 0;  // a stage's next phase of `begin` or `lfull`
        bool ok = true;
        for (int i = 0, t; (t = round_tile<true>(i, cluster_id, n_clusters)) < n_tiles && ok; ++i) {
            int e, mb, nb;
            place(t, e, mb, nb);
            const int n = rows_of(e), base = first_of(e), whole = n / BK;
            stage = (stage + whole) % S;
            if (whole * BK == n) continue;
            if (warp == TAIL_WARP + TAIL_WARPS) {
                ok = wait_warp(p, lfull + stage, (b_parity >> stage) & 1u, kWhereProducer);
                if (!ok) break;
                b_parity ^= 1u << stage;
                fence_proxy_async_smem();
                if (lane == 0) mbar_arrive_cluster(gfull0 + stage * 8);
                if (++stage == S) stage = 0;
                continue;
            }
            int row[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                row[j] = base + min(whole * BK + r0 + j * 4 + l.r0, n - 1);
                if (p.src != nullptr) row[j] = p.src[row[j]];
            }
            if (p.src != nullptr)
#pragma unroll
                for (int j = 0; j < 8; ++j) row[j] = checked(p, row[j]);
            ok = wait_warp(p, begin + stage, (b_parity >> stage) & 1u, kWhereProducer);
            if (!ok) break;
            b_parity ^= 1u << stage;
            const int x0 = mb * 256 + static_cast<int>(prank) * BM + l.piece * 8, y0 = nb * G::n + static_cast<int>(prank) * BM + l.piece * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = whole * BK + r0 + j * 4 + l.r0;
                const uint32_t at = r0 * 128 + l.at(j);
                const __nv_bfloat16* x = p.x + static_cast<long long>(row[j]) * p.x_ld + x0;
                const __nv_bfloat16* y = p.dy + static_cast<long long>(base + min(r, n - 1)) * p.cols + y0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const bool in = r < n && x0 + c * 64 < p.x_ld;
                    cp_async16(sa + stage * DW_A + c * CHUNK + at, in ? x + c * 64 : p.x, in);
                }
#pragma unroll
                for (int c = 0; c < 2 * G::parts; ++c) {
                    const int col = c / 2 * 256 + c % 2 * 64;
                    const bool in = r < n && y0 + col < p.cols;
                    cp_async16(sb + stage * G::b_bytes + c * CHUNK + at, in ? y + col : p.dy, in);
                }
            }
            cp_async_arrive(lfull + stage);
            if (++stage == S) stage = 0;
        }
        cp_async_drain();
    } else if (warp >= EPI_WARP) {
        // ---------------------------------------------------------------- epilogue (both CTAs)
        const int q = warp & 3, half = (warp - EPI_WARP) >> 2;
        const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
        uint8_t* box = sE + (warp - EPI_WARP) * STAGE;  // 32 rows of 64 bytes, 64-byte swizzle
        int lt = 0;
        for (int i = 0, t; (t = round_tile<true>(i, cluster_id, n_clusters)) < n_tiles; ++i) {
            int e, mb, nb;
            place(t, e, mb, nb);
            const bool none = rows_of(e) == 0;
            if (none && p.add) continue;
            const int acc = WIDE ? 0 : lt & 1;
            if (!none) {
                int okw = 0;
                if (lane == 0) okw = wait(p, tfull + acc, WIDE ? lt & 1 : (lt >> 1) & 1, kWhereEpilogue);
                okw = __shfl_sync(0xFFFFFFFFu, okw, 0);
                if (!okw) break;
                tc_fence_after();
            }
            const int k0 = mb * 256 + static_cast<int>(prank) * BM + q * 32;  // this warp's first row of dW
            for (int part = 0; part < G::parts; ++part) {
                const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + (acc + part) * 256;
                for (int c0 = half * 128; c0 < half * 128 + 128; c0 += 32) {
                    const int col = nb * G::n + part * 256 + c0;
                    if (col >= p.cols || k0 >= p.features) break;
                    uint32_t r[32];
                    if (none) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = 0;
                    } else {
                        tmem_ld_32x32b_x32(lanes + c0, r);
                        tmem_ld_wait();
                    }
                    if (p.out_f32) {  // 16 columns at a time
                        put_box(box, &tmO, r, col, k0, e, lane, p.add);
                        if (col + 16 < p.cols) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) r[j] = r[16 + j];
                            put_box(box, &tmO, r, col + 16, k0, e, lane, p.add);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) r[j] = tc::pack_bf16x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                        put_box(box, &tmO, r, col, k0, e, lane, p.add);
                    }
                }
                if (none) continue;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + (acc + part) * 8);
            }
            if (!none) ++lt;
        }
        if (lane == 0) bulk_wait_group_all();  // this warp's stores are complete
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

}  // namespace moe
}  // namespace tpmlp
