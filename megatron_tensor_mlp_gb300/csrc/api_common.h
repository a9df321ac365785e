// Argument checks shared by the entry points (host only, before any CUDA call).
#pragma once
#include <cstdint>
#include <initializer_list>

#include "internal.h"

namespace tpmlp {

inline constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

inline int esize(tpmlp_dtype dt) { return dt == TPMLP_F32 ? 4 : 2; }

struct Range {
    const void* p;
    int64_t bytes;
};

inline bool overlap(const Range& a, const Range& b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    auto a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

// Outputs must not overlap inputs or each other.
inline tpmlp_status check_alias(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    int i = 0;
    for (const Range& o : outs) {
        for (const Range& in : ins)
            if (overlap(o, in)) {
                set_error("output %d overlaps an input", i);
                return TPMLP_ERR_ALIAS;
            }
        int j = 0;
        for (const Range& o2 : outs) {
            if (j > i && overlap(o, o2)) {
                set_error("outputs %d and %d overlap", i, j);
                return TPMLP_ERR_ALIAS;
            }
            ++j;
        }
        ++i;
    }
    return TPMLP_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline tpmlp_status check_aligned(std::initializer_list<const void*> ptrs) {
    int i = 0;
    for (const void* p : ptrs) {
        if (p && !aligned16(p)) {
            set_error("pointer argument %d is not 16-byte aligned", i);
            return TPMLP_ERR_ALIGNMENT;
        }
        ++i;
    }
    return TPMLP_OK;
}

inline tpmlp_status check_pitch(int64_t elems, tpmlp_dtype dt, const char* what) {
    if ((elems * esize(dt)) % 16 != 0) {
        set_error("%s = %lld elements is not a multiple of 16 bytes", what, (long long)elems);
        return TPMLP_ERR_ALIGNMENT;
    }
    return TPMLP_OK;
}

// Common shape checks of the MLP entry points.
inline tpmlp_status check_mlp_shape(int64_t s, int64_t b, int64_t h, int64_t ffn, int p, bool need_h_div) {
    if (s < 0 || b < 0 || h < 1 || ffn < 1 || p < 1) {
        set_error("bad shape: s=%lld b=%lld h=%lld ffn=%lld p=%d", (long long)s, (long long)b, (long long)h,
                  (long long)ffn, p);
        return TPMLP_ERR_SHAPE;
    }
    if (h > kMaxDim || ffn > kMaxDim || (b > 0 && s > kMaxDim / b)) {
        set_error("shape too large: s*b, h and ffn must each be below 2^31");
        return TPMLP_ERR_SHAPE;
    }
    // every tensor of the block (with the 2x SwiGLU and 4-byte gradient widths) below 2^40 bytes
    const int64_t M = s * b, kMaxElems = (int64_t(1) << 40) / 16;
    if ((M > 0 && ffn > kMaxElems / M) || (M > 0 && h > kMaxElems / M) || ffn > kMaxElems / h) {
        set_error("shape too large: a tensor of the block would exceed 2^40 bytes");
        return TPMLP_ERR_SHAPE;
    }
    if (ffn % p != 0) {
        set_error("ffn=%lld is not divisible by p=%d", (long long)ffn, p);
        return TPMLP_ERR_DIVISIBILITY;
    }
    if (need_h_div && h % p != 0) {
        set_error("h=%lld is not divisible by p=%d", (long long)h, p);
        return TPMLP_ERR_DIVISIBILITY;
    }
    return TPMLP_OK;
}

inline tpmlp_status check_dtype(tpmlp_dtype dt) {
    if (dt != TPMLP_BF16 && dt != TPMLP_F32) {
        set_error("unknown dtype %d", (int)dt);
        return TPMLP_ERR_DTYPE;
    }
    return TPMLP_OK;
}

#define TP_TRY(expr)                          \
    do {                                      \
        tpmlp_status _st = (expr);            \
        if (_st != TPMLP_OK) return _st;      \
    } while (0)

inline tpmlp_status get_device(const DeviceInfo** out) {
    const DeviceInfo* d = device_info();
    if (!d) return TPMLP_ERR_CUDA;
    if (d->cc_major != 10 || d->cc_minor != 3) {
        set_error("device %d has compute capability %d.%d; this library is built for sm_103a (10.3) only", d->device,
                  d->cc_major, d->cc_minor);
        return TPMLP_ERR_ARCH;
    }
    *out = d;
    return TPMLP_OK;
}

}  // namespace tpmlp
