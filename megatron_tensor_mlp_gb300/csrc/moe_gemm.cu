// Host side of the products grouped by expert: tensor maps, launch.  And the bias gradients' sums over an expert's rows.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "moe_choice.h"
#include "moe_gemm.cuh"
#include "per_device.h"

namespace tpmlp {
namespace {

using namespace moe;

static_assert(Geom<STORE>::f == kFeatures && Geom<DSWIGLU>::f == kFeatures && Geom<SWIGLU>::f == kGatedFeatures && BK == kContraction);

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// bf16 [slices][rows][cols], boxes of 64 columns x box_rows; rank 2 (one slice) for tile::gather4, of one row.
bool make_map(CUtensorMap* map, const void* ptr, uint64_t cols, uint64_t rows, uint64_t slices, uint32_t box_rows, uint32_t rank = 3) {
    auto fn = encode_fn();
    if (!fn) {
        set_error("cuTensorMapEncodeTiled is not available from the driver");
        return false;
    }
    const cuuint64_t dims[3] = {cols, rows, slices}, strides[2] = {cols * 2, cols * rows * 2};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(BK), box_rows, 1}, estr[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_error("cuTensorMapEncodeTiled (experts) failed (%d): dims %llu x %llu x %llu", static_cast<int>(r),
                  (unsigned long long)cols, (unsigned long long)rows, (unsigned long long)slices);
        return false;
    }
    return true;
}

// bf16 [slices][rows][cols], cols a multiple of 64, as [slices][cols / 64][rows][64]: boxes of `chunks` 64-column strips x 64 rows.
bool make_chunks(CUtensorMap* map, const void* ptr, uint64_t cols, uint64_t rows, uint64_t slices, uint32_t chunks) {
    auto fn = encode_fn();
    if (!fn) {
        set_error("cuTensorMapEncodeTiled is not available from the driver");
        return false;
    }
    const cuuint64_t dims[4] = {BK, rows, cols / BK, slices}, strides[3] = {cols * 2, BK * 2, cols * rows * 2};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(BK), static_cast<cuuint32_t>(BK), chunks, 1}, estr[4] = {1, 1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_error("cuTensorMapEncodeTiled (experts, chunked) failed (%d)", static_cast<int>(r));
        return false;
    }
    return true;
}
// The output [slices][rows][cols] in boxes of 64 bytes x 32 rows, 64-byte swizzle.
bool make_out_map(CUtensorMap* map, void* ptr, uint64_t cols, uint64_t rows, uint64_t slices, bool f32) {
    auto fn = encode_fn();
    if (!fn) {
        set_error("cuTensorMapEncodeTiled is not available from the driver");
        return false;
    }
    const uint64_t es = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {cols, rows, slices}, strides[2] = {cols * es, cols * rows * es};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(64 / es), 32, 1}, estr[3] = {1, 1, 1};
    const CUresult r = fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ptr, dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_error("cuTensorMapEncodeTiled (experts, output) failed (%d)", static_cast<int>(r));
        return false;
    }
    return true;
}
// The rows' maps of the rows kernel.
bool make_boxes(Boxes* b, const void* ptr, uint64_t cols, uint64_t rows) {
    for (int i = 0; i < 5; ++i)
        if (!make_map(&b->m[i], ptr, cols, rows, 1, 8u << i)) return false;
    return true;
}

template <typename Kern>
bool set_smem(Kern kern, int device, int bytes, PerDevice<bool>& done) {
    return done.get(device, [&](bool& ok) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) set_error("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return ok = e == cudaSuccess;
    });
}

template <typename Kern, typename... A>
tpmlp_status launch(Kern kern, dim3 grid, int threads, int smem, unsigned cluster, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see griddep_wait
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("expert product launch: %s", cudaGetErrorString(e));
        return TPMLP_ERR_CUDA;
    }
    count_launch();
    return TPMLP_OK;
}

template <bool W_MN, int MODE, bool WIDE = false, bool H32 = false>
tpmlp_status launch_rows(const CUtensorMap& w, const Boxes& x, const Args& a, const DeviceInfo& dev, cudaStream_t st) {
    static PerDevice<bool> done;
    using G = Geom<MODE, WIDE>;
    auto kern = rows_kernel<W_MN, MODE, WIDE, H32>;
    if (!set_smem(kern, dev.device, G::smem, done)) return TPMLP_ERR_CUDA;
    const int64_t most = int64_t(a.m_blocks) * (a.rows / G::tn + std::min(a.experts, a.rows));
    const unsigned pairs = static_cast<unsigned>(std::min<int64_t>(most, dev.sm_count / 2));
    return launch(kern, dim3(2 * pairs), THREADS, G::smem, 2, st, w, x, a);
}

template <bool W_MN, int MODE, bool H32 = false>
tpmlp_status launch_few(const CUtensorMap& w, const Boxes& x, const Args& a, const DeviceInfo& dev, cudaStream_t st) {
    static PerDevice<bool> done;
    auto kern = few_kernel<W_MN, MODE, H32>;
    if (!set_smem(kern, dev.device, FEW_SMEM, done)) return TPMLP_ERR_CUDA;
    const int64_t tiles = int64_t(a.m_blocks) * (a.rows / FEW_TN + std::min(a.experts, a.rows));
    // the contraction is split while all CTAs, two an SM, run at once and each has at least four blocks of it
    int ranks = 1;
    while (ranks < 8 && tiles * 2 * ranks <= 2 * dev.sm_count && a.kb >= 8 * ranks) ranks *= 2;
    return launch(kern, dim3(static_cast<unsigned>(tiles * ranks)), FEW_THREADS, FEW_SMEM, ranks, st, w, x, a);
}

template <bool WIDE>
tpmlp_status launch_dw(const CUtensorMap& x, const CUtensorMap& y, const CUtensorMap& o, const Args& a, unsigned pairs, const DeviceInfo& dev, cudaStream_t st) {
    static PerDevice<bool> done;
    auto kern = dw_kernel<WIDE>;
    if (!set_smem(kern, dev.device, DwGeom<WIDE>::smem, done)) return TPMLP_ERR_CUDA;
    return launch(kern, dim3(2 * pairs), DW_THREADS, DwGeom<WIDE>::smem, 2, st, x, y, o, a);
}

// Sums of an expert's rows by column: CTA (64 columns, expert), a warp four rows at a time, 128 a CTA; a lane adds its rows in
// their order, then its warp's four lanes of a column, then the 32 warps.  (3992 x 2048 on 16 experts: 6.6 us, with eight
// warps 12.)
constexpr int SUM_WARPS = 32, SUM_THREADS = 32 * SUM_WARPS;
__global__ void __launch_bounds__(SUM_THREADS) sums_kernel(const __nv_bfloat16* in, const int* offsets, int rows, int cols, void* out,
                                                           int out_f32) {
    __shared__ float part[SUM_WARPS][64];
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.y, c = blockIdx.x * 64 + (lane & 7) * 8, r0 = threadIdx.x >> 3;
    const int a = min(max(offsets[e], 0), rows), b = min(max(offsets[e + 1], 0), rows);
    float s[8] = {};
    if (c < cols) {
        for (int r = a + r0; r < b; r += 4 * 4 * SUM_WARPS) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = r + i * 4 * SUM_WARPS;
                v[i] = at < b ? *reinterpret_cast<const uint4*>(in + static_cast<long long>(at) * cols + c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float f[8];
                tc::unpack_bf16x8(v[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] += f[j];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        s[j] += __shfl_xor_sync(0xFFFFFFFFu, s[j], 8);
        s[j] += __shfl_xor_sync(0xFFFFFFFFu, s[j], 16);
        if (lane < 8) part[warp][lane * 8 + j] = s[j];
    }
    __syncthreads();
    const int col = blockIdx.x * 64 + threadIdx.x;
    if (threadIdx.x < 64 && col < cols) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < SUM_WARPS; ++w) v += part[w][threadIdx.x];
        const long long at = static_cast<long long>(e) * cols + col;
        if (out_f32) static_cast<float*>(out)[at] = v;
        else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
    }
}

Args common(const MoeSpec& g, const DeviceInfo& dev) {
    Args a{};
    a.offsets = g.offsets;
    a.src = g.src;
    a.rows = static_cast<int>(g.rows);
    a.tokens = static_cast<int>(g.tokens);
    a.experts = g.experts;
    a.x = static_cast<const __nv_bfloat16*>(g.x);
    a.x_ld = static_cast<int>(g.K);
    a.status = dev.status;
    a.timeout_ns = 2000000000ull;  // 2 s per wait
    return a;
}

}  // namespace

tpmlp_status launch_moe_matmul(const MoeSpec& g, const DeviceInfo& dev, cudaStream_t st) {
    Args a = common(g, dev);
    a.kb = static_cast<int>((g.K + BK - 1) / BK);
    a.features = static_cast<int>(g.gated ? g.N / 2 : g.N);
    const Kernel kernel = forward_kernel(g.rows, g.experts, g.K, g.N, g.gated, g.src != nullptr, dev.sm_count / 2);
    const bool few = kernel == FEW, wide = kernel == WIDE;
    const int tile = g.gated ? Geom<SWIGLU>::f : Geom<STORE>::f;
    a.m_blocks = static_cast<int>(blocks(a.features, few ? tile / 2 : wide ? tile * 2 : tile));
    a.out = g.out;
    a.ld = a.features;
    a.out_f32 = g.out_f32;
    a.bias = static_cast<const __nv_bfloat16*>(g.bias);
    a.bias_ld = g.N;
    a.h_out = g.h;
    a.h_ld = g.N;
    CUtensorMap w;
    Boxes x{};
    // a CTA's columns of a stage in one copy: two chunks of 64 next to one another, the wide gated tile's four
    const uint32_t chunks = g.gated ? (wide ? 4 : 0) : 2;
    a.chunked = chunks > 0 && g.N % 64 == 0;
    const bool mapped = a.chunked ? make_chunks(&w, g.w, g.N, g.K, g.experts, chunks) : make_map(&w, g.w, g.N, g.K, g.experts, BK);
    if (!mapped || !(g.src ? make_map(&x.m[0], g.x, g.K, g.tokens, 1, 1, 2) : make_boxes(&x, g.x, g.K, g.rows))) return TPMLP_ERR_CUDA;
    if (g.gated && g.h && g.h_f32) {
        if (few) return launch_few<true, SWIGLU, true>(w, x, a, dev, st);
        return wide ? launch_rows<true, SWIGLU, true, true>(w, x, a, dev, st) : launch_rows<true, SWIGLU, false, true>(w, x, a, dev, st);
    }
    if (few) return g.gated ? launch_few<true, SWIGLU>(w, x, a, dev, st) : launch_few<true, STORE>(w, x, a, dev, st);
    if (wide) return g.gated ? launch_rows<true, SWIGLU, true>(w, x, a, dev, st) : launch_rows<true, STORE, true>(w, x, a, dev, st);
    return g.gated ? launch_rows<true, SWIGLU>(w, x, a, dev, st) : launch_rows<true, STORE>(w, x, a, dev, st);
}

tpmlp_status launch_moe_matmul_dx(const MoeSpec& g, const DeviceInfo& dev, cudaStream_t st) {
    Args a = common(g, dev);
    a.kb = static_cast<int>((g.N + BK - 1) / BK);
    a.features = static_cast<int>(g.K);
    const Kernel kernel = dx_kernel(g.rows, g.experts, g.K, g.N, g.gated, dev.sm_count / 2);
    a.m_blocks = static_cast<int>(blocks(a.features, kernel == FEW ? BM : kernel == WIDE ? 512 : 256));
    a.out = g.out;
    a.ld = g.gated ? 2 * g.K : g.K;
    a.out_f32 = g.out_f32;
    a.h_in = g.h;
    a.h_ld = 2 * g.K;
    CUtensorMap w;
    Boxes x;
    if (!make_map(&w, g.w, g.N, g.K, g.experts, BM) || !make_boxes(&x, g.x, g.N, g.rows)) return TPMLP_ERR_CUDA;
    if (g.gated && g.h_f32)
        return kernel == FEW ? launch_few<false, DSWIGLU, true>(w, x, a, dev, st) : launch_rows<false, DSWIGLU, false, true>(w, x, a, dev, st);
    if (kernel == FEW) return g.gated ? launch_few<false, DSWIGLU>(w, x, a, dev, st) : launch_few<false, STORE>(w, x, a, dev, st);
    if (g.gated) return launch_rows<false, DSWIGLU>(w, x, a, dev, st);
    return kernel == WIDE ? launch_rows<false, STORE, true>(w, x, a, dev, st) : launch_rows<false, STORE>(w, x, a, dev, st);
}

tpmlp_status launch_moe_matmul_dw(const MoeSpec& g, const DeviceInfo& dev, cudaStream_t st) {
    Args a = common(g, dev);
    a.features = static_cast<int>(g.K);
    a.cols = static_cast<int>(g.N);
    a.m_blocks = (a.features + 255) / 256;
    const bool wide = dw_kernel(g.rows, g.experts, g.K, g.N, g.src != nullptr, dev.sm_count / 2) == WIDE;
    a.n_blocks = static_cast<int>(blocks(a.cols, wide ? 512 : 256));
    a.out = g.out;
    a.ld = g.N;
    a.out_f32 = g.out_f32;
    a.dy = static_cast<const __nv_bfloat16*>(g.dy);
    CUtensorMap x{}, y, o;
    if (!(g.src ? make_map(&x, g.x, g.K, g.tokens, 1, 1, 2) : make_map(&x, g.x, g.K, g.rows, 1, BK)) || !make_map(&y, g.dy, g.N, g.rows, 1, BK) ||
        !make_out_map(&o, g.out, g.N, g.K, g.experts, g.out_f32))
        return TPMLP_ERR_CUDA;
    const int64_t tiles = int64_t(a.experts) * a.m_blocks * a.n_blocks;
    const unsigned pairs = static_cast<unsigned>(std::min<int64_t>(tiles, dev.sm_count / 2));
    // (an expert may have all rows: as many launches as those take, the later ones short where it has not)
    const int64_t chunk = g.out_f32 ? int64_t(get_k_chunk_blocks()) * BK : g.rows;
    for (int64_t r = 0; r < g.rows; r += chunk) {
        a.skip = static_cast<int>(r);
        a.most = static_cast<int>(std::min(chunk, g.rows - r));
        a.add = r > 0;
        const tpmlp_status s = wide ? launch_dw<true>(x, y, o, a, pairs, dev, st) : launch_dw<false>(x, y, o, a, pairs, dev, st);
        if (s != TPMLP_OK) return s;
    }
    if (g.dbias == nullptr) return TPMLP_OK;
    return launch(sums_kernel, dim3(static_cast<unsigned>((g.N + 63) / 64), static_cast<unsigned>(g.experts)), SUM_THREADS, 0, 1, st,
                  static_cast<const __nv_bfloat16*>(g.dy), g.offsets, a.rows, a.cols, g.dbias, a.out_f32);
}

}  // namespace tpmlp
