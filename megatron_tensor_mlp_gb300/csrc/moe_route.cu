// Routing of tokens to experts and the combination of the experts' rows, each with its backward.
//
// Routing.  A warp takes a token: its logits lie in registers, and k times over the largest that is left is found by a
// maximum over the warp of keys that order as the logits do (NaN above everything, the two zeros alike; a tie goes to
// the lower index).  The plan is a counting sort of the (token, slot) pairs by expert, stable, without atomics whose
// order could show: chunks of tokens are counted, then each chunk sums the counts of those ahead of it and places its
// own pairs by their rank among equal experts (match.any within a warp, counts across warps).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace tpmlp {
namespace {

constexpr int ROUTE_THREADS = 512, ROUTE_WARPS = ROUTE_THREADS / 32;
constexpr int MOST_EXPERTS = 1024;
constexpr uint32_t FULL = 0xFFFFFFFFu;

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 v) {
    return __bfloat162float(v);
}

// Orders as the values do: NaN first, then +inf .. -inf; both zeros alike.  0 is below every value's key.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t KEY_NONE = 0x007FFFFFu;  // of -inf, which is never chosen

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
    return v;
}

struct RouteArgs {
    const void* logits;
    int* ids;
    float* weights;
    int* offsets;
    int* row_token;
    int* slot_row;
    int* hist;  // [chunks][stride]
    int tokens, experts, k, chosen;
    int per_chunk, chunks;  // tokens of a chunk
    int stride;             // experts, rounded up to 4
};

// One token: its k experts and weights, and (lane j) the expert of slot j in the answer (-1: none).
template <typename T, int PER>
__device__ __forceinline__ int route_token(const RouteArgs& p, int t, int lane) {
    const T* row = static_cast<const T*>(p.logits) + static_cast<long long>(t) * p.experts;
    float x[PER];
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        x[i] = e < p.experts ? widen(row[e]) : -INFINITY;
        key[i] = e < p.experts ? key_of(x[i]) : 0u;
    }
    float top = 0.0f, mine = 0.0f, sum = 0.0f;
    int id = -1;
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(FULL, best);
        if (best <= KEY_NONE) break;  // (the same in every lane)
        int at = 0x7FFFFFFF;
        float v = 0.0f;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            if (key[i] == best) {
                at = i * 32 + lane;
                v = x[i];
            }
        const int win = __reduce_min_sync(FULL, at);
        v = __shfl_sync(FULL, v, win & 31);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (win == i * 32 + lane) key[i] = 0;
        if (j == 0) top = v;
        const float ex = expf(v - top);
        sum += ex;
        if (lane == j) {
            id = win;
            mine = ex;
        }
    }
    if (!p.chosen) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) s += expf(x[i] - top);  // (past the last expert: of -inf, 0)
        sum = warp_sum(s);
    }
    if (lane < p.k) {
        const long long slot = static_cast<long long>(t) * p.k + lane;
        p.ids[slot] = id;
        p.weights[slot] = id >= 0 ? mine / sum : 0.0f;
    }
    return id;
}

// Rows of a chunk's slots: count[e] starts as the first row of the chunk's own for expert e.
__device__ __forceinline__ void place_chunk(const RouteArgs& p, int first_slot, int n_slots, int* count, uint8_t (*ahead)[MOST_EXPERTS]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int s0 = 0; s0 < n_slots; s0 += ROUTE_THREADS) {
        for (int i = threadIdx.x; i < ROUTE_WARPS * MOST_EXPERTS / 16; i += ROUTE_THREADS)
            reinterpret_cast<uint4*>(ahead)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        const int s = s0 + threadIdx.x;
        const int e = s < n_slots ? p.ids[first_slot + s] : -1;
        const uint32_t same = __match_any_sync(FULL, e);
        const int rank = __popc(same & ((1u << lane) - 1));
        if (e >= 0 && rank == 0) ahead[warp][e] = static_cast<uint8_t>(__popc(same));
        __syncthreads();
        int row = -1;
        if (e >= 0) {
            row = count[e] + rank;
            for (int w = 0; w < warp; ++w) row += ahead[w][e];
            p.row_token[row] = (first_slot + s) / p.k;
        }
        if (s < n_slots) p.slot_row[first_slot + s] = row;
        __syncthreads();
        if (s0 + ROUTE_THREADS < n_slots) {
            for (int i = threadIdx.x; i < p.experts; i += ROUTE_THREADS) {
                int c = count[i];
                for (int w = 0; w < ROUTE_WARPS; ++w) c += ahead[w][i];
                count[i] = c;
            }
            __syncthreads();
        }
    }
}

// Exclusive sums of total[e] over the experts into base[e], base[experts] the sum of all.  All threads.
__device__ __forceinline__ void scan_experts(const int* total, int* base, int experts, int* warp_sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int carry = 0;
    for (int e0 = 0; e0 < experts; e0 += ROUTE_THREADS) {
        const int e = e0 + threadIdx.x, v = e < experts ? total[e] : 0;
        int sum = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(FULL, sum, d);
            if (lane >= d) sum += o;
        }
        if (lane == 31) warp_sums[warp] = sum;
        __syncthreads();
        int before = carry, all = 0;
        for (int w = 0; w < ROUTE_WARPS; ++w) {
            if (w < warp) before += warp_sums[w];
            all += warp_sums[w];
        }
        if (e < experts) base[e] = before + sum - v;
        carry += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) base[experts] = carry;
    __syncthreads();
}

// Chunk c of the tokens: experts, weights and the chunk's counts; with a single chunk also its plan.
template <typename T, int PER>
__global__ void __launch_bounds__(ROUTE_THREADS) route_kernel(const RouteArgs p) {
    __shared__ int count[MOST_EXPERTS];
    __shared__ int base[MOST_EXPERTS + 1];
    __shared__ int warp_sums[ROUTE_WARPS];
    __shared__ __align__(16) uint8_t ahead[ROUTE_WARPS][MOST_EXPERTS];
    for (int i = threadIdx.x; i < p.stride; i += ROUTE_THREADS) count[i] = 0;
    __syncthreads();
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * p.per_chunk, t1 = min(t0 + p.per_chunk, p.tokens);
    for (int t = t0 + warp; t < t1; t += ROUTE_WARPS) {
        const int id = route_token<T, PER>(p, t, lane);
        if (id >= 0) atomicAdd(count + id, 1);  // (whole numbers: the order does not show)
    }
    __syncthreads();
    if (p.chunks > 1) {
        for (int i = threadIdx.x; i < p.stride; i += ROUTE_THREADS) p.hist[blockIdx.x * p.stride + i] = count[i];
        return;
    }
    scan_experts(count, base, p.experts, warp_sums);
    for (int i = threadIdx.x; i <= p.experts; i += ROUTE_THREADS) p.offsets[i] = base[i];
    const int slots = p.tokens * p.k;
    for (int i = base[p.experts] + threadIdx.x; i < slots; i += ROUTE_THREADS) p.row_token[i] = -1;
    place_chunk(p, 0, slots, base, ahead);
}

// The plan of chunk c from all chunks' counts.
__global__ void __launch_bounds__(ROUTE_THREADS, 4) place_kernel(const RouteArgs p) {
    __shared__ int mine[MOST_EXPERTS];   // counts ahead of this chunk, then its first rows
    __shared__ int total[MOST_EXPERTS];
    __shared__ int base[MOST_EXPERTS + 1];
    __shared__ int warp_sums[ROUTE_WARPS];
    __shared__ __align__(16) uint8_t ahead[ROUTE_WARPS][MOST_EXPERTS];
    for (int i = threadIdx.x; i < p.stride; i += ROUTE_THREADS) mine[i] = total[i] = 0;
    __syncthreads();
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    // a warp's share of the chunks, 128 experts at a time, four a lane
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = lane * 4; e < p.stride; e += 128) {
        int before[4] = {}, all[4] = {};
        for (int c0 = warp; c0 < p.chunks; c0 += ROUTE_WARPS * 4) {
            int4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i * ROUTE_WARPS;
                v[i] = c < p.chunks ? *reinterpret_cast<const int4*>(p.hist + c * p.stride + e) : make_int4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                const bool ahead = c0 + i * ROUTE_WARPS < static_cast<int>(blockIdx.x);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    all[q] += n[q];
                    before[q] += ahead ? n[q] : 0;
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            atomicAdd(total + e + q, all[q]);
            atomicAdd(mine + e + q, before[q]);
        }
    }
    __syncthreads();
    scan_experts(total, base, p.experts, warp_sums);
    for (int i = threadIdx.x; i < p.experts; i += ROUTE_THREADS) mine[i] += base[i];
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i <= p.experts; i += ROUTE_THREADS) p.offsets[i] = base[i];
    const int s0 = blockIdx.x * p.per_chunk * p.k, s1 = min(s0 + p.per_chunk * p.k, p.tokens * p.k);
    for (int i = max(s0, base[p.experts]) + threadIdx.x; i < s1; i += ROUTE_THREADS) p.row_token[i] = -1;
    __syncthreads();
    place_chunk(p, s0, s1 - s0, mine, ahead);
}

// dlogits of a token: p_i ([i chosen] dw_i - sum_j w_j dw_j), over all experts or over the chosen.
template <typename T, int PER>
__global__ void __launch_bounds__(256) route_bwd_kernel(const void* logits, const int* ids, const float* weights, const float* dweights,
                                                        void* dlogits, int tokens, int experts, int k, int chosen) {
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= tokens) return;
    const long long slot = static_cast<long long>(t) * k + lane;
    int id = -1;
    float w = 0.0f, dw = 0.0f;
    if (lane < k) {
        id = ids[slot];
        if (id < 0 || id >= experts) id = -1;
        if (id >= 0) {
            w = weights[slot];
            dw = dweights[slot];
        }
    }
    const float inner = warp_sum(w * dw);
    float d[PER];
    if (!chosen) {
        const T* row = static_cast<const T*>(logits) + static_cast<long long>(t) * experts;
        float m = -INFINITY, s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 32 + lane;
            d[i] = e < experts ? widen(row[e]) : -INFINITY;
            m = fmaxf(m, d[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
        if (m == -INFINITY) m = 0.0f;  // a token of -inf alone: every share is 0
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            d[i] = expf(d[i] - m);
            s += d[i];
        }
        s = warp_sum(s);
        const float scale = s > 0.0f || s != s ? -inner / s : 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) d[i] *= scale;
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) d[i] = 0.0f;
    }
    const float back = chosen ? w * (dw - inner) : w * dw;
    for (int j = 0; j < k; ++j) {
        const int e = __shfl_sync(FULL, id, j);
        const float b = __shfl_sync(FULL, back, j);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e == i * 32 + lane) d[i] += b;
    }
    T* out = static_cast<T*>(dlogits) + static_cast<long long>(t) * experts;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        if (e < experts) {
            if constexpr (sizeof(T) == 4) out[e] = d[i];
            else out[e] = __float2bfloat16_rn(d[i]);
        }
    }
}

// ---------------------------------------------------------------- combination
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint4 u;
    uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return u;
}

struct CombineArgs {
    const __nv_bfloat16* o;
    const int* slot_row;
    const float* weights;  // may be null: 1
    __nv_bfloat16* z;
    const __nv_bfloat16* dz;
    __nv_bfloat16* d_o;
    float* dweights;  // may be null
    int tokens, rows, k, vecs;  // vecs: 16-byte pieces of a row
};

// Z[t] = sum_j w[t][j] O[row(t, j)], slots in order, in 32 bits.  A CTA takes a token, a thread four pieces of 16 bytes at a
// time, of two slots, so that their row numbers are waited for once and eight loads then are on their way.  (16384 rows of 5120
// into 8192 tokens: 41 us, a piece of a slot at a time 47, at a copy's rate 37.  One slot a token: half the registers and
// twice the threads an SM, 28 us, with two slots' 37, at a copy's rate 25.  Where half the pieces do for a row: of 2560, three
// slots, 8192 tokens 34 us with four, 30 with two; of 5120, two slots, 43, 46.)
template <int AT_ONCE, int PIECES>
__global__ void __launch_bounds__(AT_ONCE == 1 ? 512 : 256) combine_kernel(const CombineArgs p) {
    griddep_wait();
    if (threadIdx.x == 0 && threadIdx.y == 0) griddep_launch_dependents();
    const int nx = blockDim.x;
    for (int t = blockIdx.x * blockDim.y + threadIdx.y; t < p.tokens; t += gridDim.x * blockDim.y) {
        const long long s0 = static_cast<long long>(t) * p.k;
        for (int v0 = threadIdx.x; v0 < p.vecs; v0 += PIECES * nx) {
            float sum[PIECES][8] = {};
            for (int j0 = 0; j0 < p.k; j0 += AT_ONCE) {
                uint4 r[AT_ONCE][PIECES];
                float w[AT_ONCE];
                bool there[AT_ONCE];
#pragma unroll
                for (int h = 0; h < AT_ONCE; ++h) {
                    const int row = j0 + h < p.k ? p.slot_row[s0 + j0 + h] : -1;
                    there[h] = row >= 0 && row < p.rows;
                    w[h] = there[h] && p.weights != nullptr ? p.weights[s0 + j0 + h] : 1.0f;
                    const uint4* o = reinterpret_cast<const uint4*>(p.o) + static_cast<long long>(there[h] ? row : 0) * p.vecs;
#pragma unroll
                    for (int i = 0; i < PIECES; ++i)
                        r[h][i] = there[h] && v0 + i * nx < p.vecs ? o[v0 + i * nx] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int h = 0; h < AT_ONCE; ++h) {
                    if (!there[h]) continue;
#pragma unroll
                    for (int i = 0; i < PIECES; ++i) {
                        float x[8];
                        unpack8(r[h][i], x);
#pragma unroll
                        for (int q = 0; q < 8; ++q) sum[i][q] = fmaf(w[h], x[q], sum[i][q]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
                if (v0 + i * nx < p.vecs) reinterpret_cast<uint4*>(p.z)[static_cast<long long>(t) * p.vecs + v0 + i * nx] = pack8(sum[i]);
        }
    }
}

// dO[row] = w dZ[t], dw[t][j] = dZ[t] . O[row]: a warp takes a slot (the slots of a token, next to one another, find dZ in L1).
// (Rows of 512, three slots, 8192 tokens: 11.4 us with four pieces a lane, two of which are empty, 8.7 with two.)
template <int PIECES>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const CombineArgs p) {
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long slots = static_cast<long long>(p.tokens) * p.k;
    for (long long s = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); s < slots; s += static_cast<long long>(gridDim.x) * 8) {
        const int row = p.slot_row[s];
        const bool there = row >= 0 && row < p.rows;
        float dot = 0.0f;
        if (there) {
            const float w = p.weights == nullptr ? 1.0f : p.weights[s];
            const uint4* dz = reinterpret_cast<const uint4*>(p.dz) + s / p.k * p.vecs;
            const uint4* o = reinterpret_cast<const uint4*>(p.o) + static_cast<long long>(row) * p.vecs;
            uint4* d = reinterpret_cast<uint4*>(p.d_o) + static_cast<long long>(row) * p.vecs;
            for (int v0 = lane; v0 < p.vecs; v0 += PIECES * 32) {
                uint4 rz[PIECES], ro[PIECES];
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    const bool in = v0 + i * 32 < p.vecs;
                    rz[i] = in ? dz[v0 + i * 32] : make_uint4(0, 0, 0, 0);
                    ro[i] = in && p.dweights != nullptr ? o[v0 + i * 32] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    float z[8], x[8];
                    unpack8(rz[i], z);
                    unpack8(ro[i], x);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        dot = fmaf(z[q], x[q], dot);
                        z[q] *= w;
                    }
                    if (v0 + i * 32 < p.vecs) d[v0 + i * 32] = pack8(z);
                }
            }
        }
        dot = warp_sum(dot);
        if (p.dweights != nullptr && lane == 0) p.dweights[s] = there ? dot : 0.0f;
    }
}

template <typename... P, typename... A>
tpmlp_status launch(void (*kern)(P...), dim3 grid, dim3 threads, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see griddep_wait
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("routing launch: %s", cudaGetErrorString(e));
        return TPMLP_ERR_CUDA;
    }
    count_launch();
    return TPMLP_OK;
}

// Chunks of tokens: a token a warp while they fit the SMs once, twice where tokens are many; each chunk sums the counts of all
// others, so not more.  (2048 tokens, k 8 of 64 experts: 64 chunks 7.2 us, 128 6.1; 8192, k 8 of 256: 256 chunks 26.8, 152
// 20.5; 65536, k 8 of 64: 152 chunks 52.9, 304 42.1.)  A single one, without the second kernel, for up to two a warp.
// (152 SMs are a GB300's; the workspace is sized without a device.)
int route_chunks(int64_t tokens) {
    if (tokens <= 2 * ROUTE_WARPS) return tokens > 0 ? 1 : 0;
    return static_cast<int>(std::min<int64_t>(tokens < 16384 ? 152 : 304, (tokens + ROUTE_WARPS - 1) / ROUTE_WARPS));
}

// The kernel for that many logits a lane.
template <typename F>
tpmlp_status by_experts(int experts, F&& f) {
    if (experts <= 32) return f(std::integral_constant<int, 1>{});
    if (experts <= 64) return f(std::integral_constant<int, 2>{});
    if (experts <= 128) return f(std::integral_constant<int, 4>{});
    if (experts <= 256) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 32>{});
}

}  // namespace

int64_t moe_route_ws_bytes(int64_t tokens, int experts) { return route_chunks(tokens) * ((int64_t(experts) + 3) / 4 * 4) * 4; }

tpmlp_status launch_moe_route(const void* logits, int* ids, float* weights, int* offsets, int* row_token, int* slot_row, void* ws,
                              int64_t tokens, int experts, int k, bool chosen, bool f32, cudaStream_t st) {
    RouteArgs a{};
    a.logits = logits;
    a.ids = ids;
    a.weights = weights;
    a.offsets = offsets;
    a.row_token = row_token;
    a.slot_row = slot_row;
    a.hist = static_cast<int*>(ws);
    a.tokens = static_cast<int>(tokens);
    a.experts = experts;
    a.stride = (experts + 3) / 4 * 4;
    a.k = k;
    a.chosen = chosen;
    const int chunks = route_chunks(tokens);
    a.per_chunk = static_cast<int>((tokens + chunks - 1) / chunks);
    a.chunks = static_cast<int>((tokens + a.per_chunk - 1) / a.per_chunk);
    const tpmlp_status s = by_experts(experts, [&](auto per) {
        constexpr int PER = decltype(per)::value;
        return f32 ? launch(route_kernel<float, PER>, dim3(a.chunks), ROUTE_THREADS, st, a)
                   : launch(route_kernel<__nv_bfloat16, PER>, dim3(a.chunks), ROUTE_THREADS, st, a);
    });
    if (s != TPMLP_OK || a.chunks == 1) return s;
    return launch(place_kernel, dim3(a.chunks), ROUTE_THREADS, st, a);
}

tpmlp_status launch_moe_route_bwd(const void* logits, const int* ids, const float* weights, const float* dweights, void* dlogits,
                                  int64_t tokens, int experts, int k, bool chosen, bool f32, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((tokens + 7) / 8));
    const int t = static_cast<int>(tokens), c = chosen;
    return by_experts(experts, [&](auto per) {
        constexpr int PER = decltype(per)::value;
        return f32 ? launch(route_bwd_kernel<float, PER>, grid, 256, st, logits, ids, weights, dweights, dlogits, t, experts, k, c)
                   : launch(route_bwd_kernel<__nv_bfloat16, PER>, grid, 256, st, logits, ids, weights, dweights, dlogits, t, experts, k, c);
    });
}

tpmlp_status launch_moe_combine(const void* O, const int* slot_row, const float* weights, void* Z, int64_t tokens, int64_t rows, int k,
                                int64_t h, cudaStream_t st) {
    CombineArgs a{};
    a.o = static_cast<const __nv_bfloat16*>(O);
    a.slot_row = slot_row;
    a.weights = weights;
    a.z = static_cast<__nv_bfloat16*>(Z);
    a.tokens = static_cast<int>(tokens);
    a.rows = static_cast<int>(rows);
    a.k = k;
    a.vecs = static_cast<int>(h / 8);
    const int pieces = k > 1 && a.vecs <= 512 ? 2 : 4;
    const int x = std::min(256, (a.vecs + 32 * pieces - 1) / (32 * pieces) * 32), y = k == 1 ? 256 / x : 1;
    const int64_t ctas = std::min<int64_t>((tokens + y - 1) / y, 1 << 20);
    const auto kern = k == 1 ? combine_kernel<1, 4> : pieces == 2 ? combine_kernel<2, 2> : combine_kernel<2, 4>;
    return launch(kern, dim3(static_cast<unsigned>(ctas)), dim3(x, y), st, a);
}

tpmlp_status launch_moe_combine_bwd(const void* O, const int* slot_row, const float* weights, const void* dZ, void* dO, float* dweights,
                                    int64_t tokens, int64_t rows, int k, int64_t h, cudaStream_t st) {
    CombineArgs a{};
    a.o = static_cast<const __nv_bfloat16*>(O);
    a.slot_row = slot_row;
    a.weights = weights;
    a.dz = static_cast<const __nv_bfloat16*>(dZ);
    a.d_o = static_cast<__nv_bfloat16*>(dO);
    a.dweights = dweights;
    a.tokens = static_cast<int>(tokens);
    a.rows = static_cast<int>(rows);
    a.k = k;
    a.vecs = static_cast<int>(h / 8);
    return launch(a.vecs <= 128 ? combine_bwd_kernel<2> : combine_bwd_kernel<4>, dim3(static_cast<unsigned>(std::min<int64_t>((tokens * k + 7) / 8, 1 << 20))), 256, st, a);
}

}  // namespace tpmlp
