// Host side of the MXFP4 GEMM: tensor maps, choice of kernel and split, launch.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "mxfp4_choice.h"
#include "mxfp4_gemm.cuh"
#include "per_device.h"

namespace tpmlp {
namespace {

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

bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* ptr, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
            const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle) {
    auto fn = encode_fn();
    if (!fn) {
        set_error("cuTensorMapEncodeTiled is not available from the driver");
        return false;
    }
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(map, type, 3, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_error("cuTensorMapEncodeTiled (MXFP4) failed (%d): dims %llu x %llu x %llu", static_cast<int>(r),
                  (unsigned long long)dims[0], (unsigned long long)dims[1], (unsigned long long)dims[2]);
        return false;
    }
    return true;
}

// Codes [rows][pitch bytes]: boxes of 128 bytes (256 values of k) x box_rows.
// Blocked codes [ceil(k/32)][rows][16 bytes]: boxes of box_rows rows (two 8-byte words each) x 8 blocks.
bool codes_map(CUtensorMap* map, const MxOperand& o, int64_t k, uint32_t box_rows) {
    if (o.blocked) {
        const uint64_t words = static_cast<uint64_t>(o.rows) * 2, blocks = static_cast<uint64_t>((k + 31) / 32);
        return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, o.codes, {words, blocks, 1}, {words * 8, words * 8 * blocks},
                      {box_rows * 2, 8, 1}, CU_TENSOR_MAP_SWIZZLE_NONE);
    }
    const uint64_t pitch = static_cast<uint64_t>((k + 31) / 32 * 16), rows = static_cast<uint64_t>(o.rows);
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.codes, {pitch, rows, 1}, {pitch, pitch * rows}, {128, box_rows, 1},
                  CU_TENSOR_MAP_SWIZZLE_128B);
}
// Scales [ceil(rows/128)][ceil(k/128)][512 bytes]: boxes of box_tiles row tiles x 2 k tiles.
bool scales_map(CUtensorMap* map, const MxOperand& o, int64_t k, uint32_t box_tiles) {
    const uint64_t kt = static_cast<uint64_t>((k + 127) / 128), rt = static_cast<uint64_t>((o.rows + 127) / 128);
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, o.scales, {128, kt, rt}, {512, 512 * kt}, {128, 2, box_tiles},
                  CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Saved pre-activations [rows][ld] bf16: boxes of 32 features x 32 rows.
bool h_map(CUtensorMap* map, const void* ptr, int64_t ld, int64_t rows) {
    const uint64_t w = static_cast<uint64_t>(ld), r = static_cast<uint64_t>(rows);
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ptr, {w, r, 1}, {w * 2, w * r * 2}, {32, 32, 1}, CU_TENSOR_MAP_SWIZZLE_64B);
}

// 0 auto, 1 single CTAs without a split, 2 CTA pairs, 3 / 4 / 5 single CTAs with the K loop split 2 / 4 / 8 ways
// (where the exchange of that many partial sums fits)
std::atomic<int> g_mode{0};

// Allows the kernel its dynamic shared memory, once per device.
template <typename Kern>
bool set_smem(Kern kern, int device, int bytes, PerDevice<bool>& done) {
    return done.get(device, [&](bool& ok) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) set_error("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return ok = e == cudaSuccess;
    });
}

template <typename Kern, typename... A>
tpmlp_status launch(Kern kern, unsigned grid, int threads, int smem, unsigned cluster, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
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
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("MXFP4 GEMM launch: %s", cudaGetErrorString(e));
        return TPMLP_ERR_CUDA;
    }
    count_launch();
    return TPMLP_OK;
}

template <int EPI, int N = 1>
int pair_capacity(const DeviceInfo& dev) {
    static PerDevice<int> cap;
    static PerDevice<bool> attr_done;
    if (dev.device >= PerDevice<int>::kDevices) return 0;
    return cap.get(dev.device, [&](int& n) {
        auto kern = mx::mx_pair_kernel<EPI, N>;
        if (set_smem(kern, dev.device, mx::PairGeom<EPI>::smem, attr_done)) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2 * (dev.sm_count / 2));
            cfg.blockDim = dim3(mx::P_THREADS);
            cfg.dynamicSmemBytes = mx::PairGeom<EPI>::smem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) n = 0;
            cudaGetLastError();
        }
        return true;
    });
}

template <int EPI, int CTAS>
constexpr mx::Exchange kExchange{EPI == EPI_SWIGLU ? 2 : 4, EPI == EPI_SWIGLU ? 2 : 1,
                                 mx::SingleGeom<EPI, CTAS>::ring - (EPI == EPI_DSWIGLU ? mx::S_EPI_BYTES : 0)};

// The single kernel is allowed more dynamic shared memory than it takes, so that the occupancy of clusters can be asked
// for one CTA an SM.
constexpr int kOneCtaSmem = 120 * 1024;
static_assert(2 * kOneCtaSmem > 227 * 1024 && kOneCtaSmem >= mx::SingleGeom<EPI_STORE, 2>::smem, "one CTA an SM");

template <int EPI>
mx::Machine machine(const DeviceInfo& dev, int pairs) {
    static PerDevice<mx::Machine> kept;
    mx::Machine on = kept.get(dev.device, [&](mx::Machine& m) {
        auto kern = mx::mx_single_kernel<EPI, 2>;
        m.clusters[1] = dev.sm_count;
        bool ok = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kOneCtaSmem) == cudaSuccess;
        for (int s : {2, 3, 4, 8}) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(s * (dev.sm_count / s));
            cfg.blockDim = dim3(mx::S_THREADS);
            cfg.dynamicSmemBytes = kOneCtaSmem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = s;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (!ok || cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) ok = false;
            m.clusters[s] = ok ? n : 0;
        }
        cudaGetLastError();
        return ok;
    });
    on.pairs = pairs;
    return on;
}

template <int EPI, int CTAS>
tpmlp_status launch_single(const MxOperand& a, const MxOperand& b, const MxSpec& g, mx::Args k, int mode, int split, const DeviceInfo& dev,
                           cudaStream_t st) {
    using Geom = mx::SingleGeom<EPI, CTAS>;
    constexpr bool GATED = EPI == EPI_SWIGLU;
    static PerDevice<bool> attr_done;
    auto kern = mx::mx_single_kernel<EPI, CTAS>;
    if (!set_smem(kern, dev.device, CTAS == 2 ? kOneCtaSmem : Geom::smem, attr_done)) return TPMLP_ERR_CUDA;
    k.a_box = g.M <= 16 ? 16 : g.M <= 32 ? 32 : g.M <= 64 ? 64 : 128;
    k.stages = Geom::stages(k.a_box);
    const int64_t n_blocks = GATED ? g.N / 128 : (g.N + 127) / 128, m_blocks = (g.M + 127) / 128;
    const int rows = static_cast<int>(std::min<int64_t>(g.M, mx::BM));
    if (mode >= 3) {
        split = 2 << (mode - 3);
        while (split > 1 && !kExchange<EPI, CTAS>.fits(split, rows, k.kb)) split /= 2;
    }
    k.m_blocks = static_cast<int>(m_blocks);
    CUtensorMap m[4];
    if (!codes_map(&m[0], a, g.K, static_cast<uint32_t>(k.a_box)) || !codes_map(&m[1], b, g.K, GATED ? 64 : 128) ||
        !scales_map(&m[2], a, g.K, 1) || !scales_map(&m[3], b, g.K, GATED ? 2 : 1))
        return TPMLP_ERR_CUDA;
    return launch(kern, static_cast<unsigned>(n_blocks * m_blocks * split), mx::S_THREADS, Geom::smem,
                  static_cast<unsigned>(split), st, m[0], m[1], m[2], m[3], k);
}

template <int EPI>
mx::Choice choose(const MxSpec& g, int kb, int pairs, const DeviceInfo& dev) {
    const int64_t n = EPI == EPI_SWIGLU ? g.N / 128 : (g.N + 127) / 128;
    return mx::choose(machine<EPI>(dev, pairs), kExchange<EPI, 2>,
                      {g.M, n * ((g.M + 127) / 128), ((g.M + 255) / 256) * ((g.N + 255) / 256), kb});
}

// The pair kernel's view of a product.
bool pair_problem(mx::Problem* pr, const MxOperand& a, const MxOperand& b, const MxSpec& g, const mx::Args& k) {
    pr->p = k;
    pr->p.m_blocks = static_cast<int>((g.M + 255) / 256);
    pr->p.n_blocks = static_cast<int>((g.N + 255) / 256);
    return codes_map(&pr->a, a, g.K, mx::BM) && codes_map(&pr->b, b, g.K, mx::BM) && scales_map(&pr->sa, a, g.K, 1) &&
           scales_map(&pr->sb, b, g.K, 2) && codes_map(&pr->b2, b, g.K, mx::BM / 2) &&
           (g.epi != EPI_DSWIGLU || h_map(&pr->h, g.h_in, g.h_ld, g.M));
}
int pair_tiles(const mx::Problem& pr) { return pr.p.m_blocks * pr.p.n_blocks; }

template <int EPI>
tpmlp_status launch_variant(const MxOperand& a, const MxOperand& b, const MxSpec& g, mx::Args k, const DeviceInfo& dev,
                            cudaStream_t st) {
    const int mode = g_mode.load(std::memory_order_relaxed);
    const int cap = pair_capacity<EPI>(dev);
    const mx::Choice choice = mode == 0 ? choose<EPI>(g, k.kb, cap, dev) : mx::Choice{mode == 2 && cap > 0, 1, 0.0};
    if (choice.pair) {
        mx::Problems<1> all{};
        if (!pair_problem(&all.of[0], a, b, g, k)) return TPMLP_ERR_CUDA;
        all.n_long = 1;
        all.long_tiles = pair_tiles(all.of[0]);
        return launch(mx::mx_pair_kernel<EPI, 1>, 2 * std::min(all.long_tiles, cap), mx::P_THREADS, mx::PairGeom<EPI>::smem, 2, st, all);
    }
    if constexpr (EPI != EPI_DSWIGLU) {
        // Three CTAs an SM (three ring stages each, at most 32 rows of A) where two would need another wave for the
        // rest of the tiles: 4 x 40960 x 5120, 320 tiles: 22.8 us against 26.1.  Where two are enough their longer
        // rings are better: 1 x 32768 x 4096, 256 tiles: 14.4 against 15.3.
        const int64_t tiles = EPI == EPI_SWIGLU ? g.N / 128 : (g.N + 127) / 128;
        if (mode == 0 && g.M <= 32 && tiles > 2 * dev.sm_count)
            return launch_single<EPI, 3>(a, b, g, k, mode, 1, dev, st);
    }
    return launch_single<EPI, 2>(a, b, g, k, mode, choice.split, dev, st);
}

mx::Args make_args(const MxOperand& a, const MxOperand& b, const MxSpec& g, const DeviceInfo& dev) {
    mx::Args k{};
    k.M = static_cast<int>(g.M);
    k.N = static_cast<int>(g.N);
    k.kb = static_cast<int>((g.K + mx::KC - 1) / mx::KC);
    k.last_steps = static_cast<int>((g.K - static_cast<int64_t>(k.kb - 1) * mx::KC + 63) / 64);
    k.out_f32 = g.out_f32 ? 1 : 0;
    k.out = g.out;
    k.out_ld = g.out_ld;
    k.out_ss = g.out_ss;
    k.shard_cols = static_cast<int>(g.shard_cols > 0 ? g.shard_cols : g.N);
    k.bias = static_cast<const __nv_bfloat16*>(g.bias);
    k.h_in = static_cast<const __nv_bfloat16*>(g.h_in);
    k.h_out = static_cast<__nv_bfloat16*>(g.h_out);
    k.h_ld = g.h_ld;
    k.a_blocked = a.blocked ? 1 : 0;
    k.b_blocked = b.blocked ? 1 : 0;
    k.q = static_cast<uint4*>(g.q);
    k.qs = static_cast<uint8_t*>(g.qs);
    k.q_tiles = (g.q_cols + 127) / 128;
    k.ht = static_cast<uint4*>(g.ht);
    k.hts = static_cast<uint8_t*>(g.hts);
    k.yt = static_cast<uint4*>(g.yt);
    k.yts = static_cast<uint8_t*>(g.yts);
    k.t_blocks = (g.M + 31) / 32;
    k.t_tiles = (g.M + 127) / 128;
    k.colsum = g.colsum;
    k.prefetch_b = g.prefetch_b ? 1 : 0;
    k.status = dev.status;
    k.timeout_ns = 2000000000ull;  // 2 s per wait
    {
        // 32-byte epilogue accesses: every row that they touch starts on a 32-byte boundary
        auto rows32 = [](const void* ptr, int64_t pitch, int64_t shard) {
            return ptr == nullptr || (reinterpret_cast<uintptr_t>(ptr) % 32 == 0 && pitch % 32 == 0 && shard % 32 == 0);
        };
        const int64_t es = g.out_f32 ? 4 : 2;
        k.st32 = rows32(g.out, g.out_ld * es, g.out_ss * es) && rows32(g.h_in, g.h_ld * 2, 0) && rows32(g.h_out, g.h_ld * 2, 0);
    }
    return k;
}

}  // namespace

void set_mxfp4_mode(int mode) { g_mode.store(mode, std::memory_order_relaxed); }
int get_mxfp4_mode() { return g_mode.load(std::memory_order_relaxed); }

tpmlp_status launch_mxfp4_gemm(const MxOperand& a, const MxOperand& b, const MxSpec& g, const DeviceInfo& dev, cudaStream_t st) {
    const mx::Args k = make_args(a, b, g, dev);
    switch (g.epi) {
        case EPI_STORE: return launch_variant<EPI_STORE>(a, b, g, k, dev, st);
        case EPI_SWIGLU: return launch_variant<EPI_SWIGLU>(a, b, g, k, dev, st);
        case EPI_DSWIGLU: return launch_variant<EPI_DSWIGLU>(a, b, g, k, dev, st);
    }
    set_error("internal: no MXFP4 GEMM for epilogue %d", g.epi);
    return TPMLP_ERR_CUDA;
}

// Independent plain products, in one launch of CTA pairs where that is expected to be faster than one after the
// other: it saves their launches and their last waves.  (s=499 b=4 h1024 ffn4096, the backward's three products: 35 us
// one by one; 4096 tokens, h5120, ffn20480: dX alone ends in a wave of 16 of 76 pairs that lasts 42 us.)
// The column sums go with the pairs' launch (see the kernel) or into one ahead of the products.
tpmlp_status launch_mxfp4_gemms(const MxProduct (&c)[3], const MxSums& sums, const DeviceInfo& dev, cudaStream_t st) {
    mx::SumsArgs sa{};
    sa.rows = static_cast<int>(sums.rows);
    sa.f32 = sums.f32;
    for (int i = 0, n = 0; i < 2; ++i) {
        if (sums.out[i] == nullptr) continue;
        sa.in[n] = sums.in[i];
        sa.out[n] = sums.out[i];
        sa.cols[n++] = static_cast<int>(sums.cols[i]);
        if (n == 1) sa.items0 = static_cast<int>((sums.cols[i] + 7) / 8);
        sa.items += static_cast<int>((sums.cols[i] + 7) / 8);
    }
    const int cap = pair_capacity<EPI_STORE, 3>(dev);
    mx::Args k[3];
    int order[3] = {0, 1, 2};
    double apart = 0.0, together = 0.0;
    for (int i = 0; i < 3; ++i) {
        k[i] = make_args(c[i].a, c[i].b, c[i].g, dev);
        apart += choose<EPI_STORE>(c[i].g, k[i].kb, cap, dev).us;
        together += static_cast<double>((c[i].g.M + 255) / 256 * ((c[i].g.N + 255) / 256)) * mx::pair_tile_us(k[i].kb);
    }
    const int mode = g_mode.load(std::memory_order_relaxed);
    if (cap <= 0 || (mode != 0 && mode != 2) || (mode == 0 && mx::kPairStart + together / cap + mx::pair_tile_us(1) >= apart)) {
        if (sa.items > 0) {
            const tpmlp_status r = launch_mxfp4_sums(sa, st);
            if (r != TPMLP_OK) return r;
        }
        for (const MxProduct& x : c) {
            const tpmlp_status r = launch_mxfp4_gemm(x.a, x.b, x.g, dev, st);
            if (r != TPMLP_OK) return r;
        }
        return TPMLP_OK;
    }
    std::sort(order, order + 3, [&](int x, int y) { return k[x].kb > k[y].kb; });
    mx::Problems<3> all{};
    for (int i = 0; i < 3; ++i) {
        const MxProduct& x = c[order[i]];
        if (!pair_problem(&all.of[i], x.a, x.b, x.g, k[order[i]])) return TPMLP_ERR_CUDA;
        const bool longest = k[order[i]].kb == k[order[0]].kb;
        int& tiles = longest ? all.long_tiles : all.short_tiles;
        all.first[i] = tiles;
        tiles += pair_tiles(all.of[i]);
        if (longest) all.n_long = i + 1;
        else if (all.skip == 0) all.skip = static_cast<int>(mx::pair_tile_us(k[order[0]].kb) / mx::pair_tile_us(k[order[i]].kb) + 0.5);
    }
    all.sums = sa;
    const int clusters = std::min(all.long_tiles + all.short_tiles, cap);
    return launch(mx::mx_pair_kernel<EPI_STORE, 3>, 2 * clusters, mx::P_THREADS, mx::PairGeom<EPI_STORE>::smem, 2, st, all);
}

}  // namespace tpmlp
