// Argument checks that the attention entry points share; all of them run before the first HIP call.
#pragma once

#include <limits.h>
#include <stdint.h>

#include "gdr_internal.h"

namespace gdr {
namespace attn {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int status_of(hipError_t e) {
    if (e == hipSuccess) return GDR_OK;
    // the launchers report a grid beyond 2^32 work-items this way, before any HIP call
    if (e == hipErrorInvalidConfiguration) return GDR_ERR_BAD_SHAPE;
    return GDR_ERR_HIP;
}

// Element type, head sizes and mask, common to every entry point.
inline int common_checks(int dtype, int Hq, int Hkv, int d, int window, int sinks) {
    if (dtype != GDR_DTYPE_F32 && dtype != GDR_DTYPE_BF16) return GDR_ERR_BAD_ENUM;
    if (Hq < 0 || Hkv < 0 || window < 0 || sinks < 0) return GDR_ERR_BAD_SHAPE;
    if (d != 64 && d != 128) return GDR_ERR_UNSUPPORTED;
    if (Hkv == 0 || Hq == 0 ? Hq != Hkv : Hq % Hkv != 0) return GDR_ERR_BAD_SHAPE;
    return GDR_OK;
}

// Rows of one sequence (tokens x heads) stay below 2^29 and heads at 2^15, so
// that offsets inside a tile and row numbers fit 32 bits; no tensor passes
// 2^40 elements.
inline bool sizes_ok(long long B, long long T, long long H, long long d) {
    const long long lim = 1LL << 40;
    if (T >= (1 << 29) || H > (1 << 15) || T * H >= (1 << 29) || B * H > INT_MAX / 8) return false;
    if (T * H > 0 && B > lim / (T * H * d)) return false;
    return true;
}

inline int page_checks(int Hkv, int page_size, int num_pages, int max_pages) {
    if (num_pages < 0 || max_pages < 0) return GDR_ERR_BAD_SHAPE;
    if (page_size < 1 || page_size > 65536 || (page_size & (page_size - 1))) return GDR_ERR_UNSUPPORTED;
    if (static_cast<long long>(max_pages) * page_size > INT_MAX - 4096) return GDR_ERR_BAD_SHAPE;
    // rows of the page tensors are addressed by a 32-bit row number
    const long long rows = static_cast<long long>(num_pages) * page_size;
    if (rows > INT_MAX || (Hkv > 0 && rows > INT_MAX / Hkv)) return GDR_ERR_BAD_SHAPE;
    return GDR_OK;
}

// A window that reaches past the first key hides nothing.
inline int clamp_window(int window, int keys) { return window >= keys ? 0 : window; }
inline int clamp_sinks(int sinks, int window, int keys) { return window == 0 ? 0 : sinks < keys ? sinks : keys; }

}  // namespace attn
}  // namespace gdr
