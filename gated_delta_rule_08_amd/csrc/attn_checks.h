// Argument checks that the attention entry points share; all of them run before the first HIP call.
#pragma once

#include <limits.h>
#include <stdint.h>

#include <initializer_list>

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

// The bytes a call reads or writes of one tensor: `rows` rows of `width` bytes,
// `stride` bytes apart (no less than width).
struct Extent {
    const void* p;
    long long width, stride, rows;
    uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
    uintptr_t end() const { return begin() + static_cast<uintptr_t>((rows - 1) * stride + width); }
    bool empty() const { return !p || width <= 0 || rows <= 0; }
    // whether a row has bytes of [lo, hi)
    bool hits(uintptr_t lo, uintptr_t hi) const {
        const uintptr_t w = static_cast<uintptr_t>(width), s = static_cast<uintptr_t>(stride), b = begin();
        const uintptr_t i = lo < b + w ? 0 : (lo - b - w) / s + 1;  // the first row that ends behind lo
        return i < static_cast<uintptr_t>(rows) && b + i * s < hi;
    }
};
inline Extent dense(const void* p, long long bytes) { return Extent{p, bytes, bytes, 1}; }
// Tokens `stride` elements apart, of `elements` each.
inline Extent tokens_of(const void* p, long long tokens, long long elements, long long stride, int size) {
    return stride == elements || tokens == 1 ? dense(p, tokens * elements * size)
                                             : Extent{p, elements * size, stride * size, tokens};
}
// Whether two tensors share a byte.
inline bool meet(const Extent& a, const Extent& b) {
    if (a.empty() || b.empty() || a.end() <= b.begin() || b.end() <= a.begin()) return false;
    if (a.rows == 1) return b.hits(a.begin(), a.end());
    if (b.rows == 1) return a.hits(b.begin(), b.end());
    if (a.stride == b.stride) {
        // row i of a and row i + n of b share bytes where -b.width < delta + n stride < a.width: the least such n
        const long long delta = static_cast<long long>(b.begin() - a.begin()), s = a.stride, x = -b.width - delta;
        long long n = (x >= 0 ? x / s : -((-x + s - 1) / s)) + 1;
        if (n < 1 - a.rows) n = 1 - a.rows;
        return n < b.rows && delta + n * s < a.width;
    }
    for (long long i = 0; i < a.rows; ++i) {  // views of one buffer that lie differently: not met in earnest
        const uintptr_t at = a.begin() + static_cast<uintptr_t>(i * a.stride);
        if (b.hits(at, at + static_cast<uintptr_t>(a.width))) return true;
    }
    return false;
}
// int32 [rows, width]; larger than any memory where that would leave 64 bits.
inline Extent table_of(const void* p, long long rows, long long width) {
    return dense(p, width && rows > (1LL << 58) / width ? 1LL << 60 : 4 * rows * width);
}
// An output, and which input's place it may take (-1: none's).
struct Written {
    Extent at;
    int own;
};
// Whether an output is another tensor of the call: begins where that does or, with
// `apart`, shares a byte with it.  An output in the place of its own input has to lie
// as that does, which is the caller's to check.
inline bool aliased(bool apart, std::initializer_list<Written> outs, std::initializer_list<Extent> ins) {
    auto same = [&](const Extent& a, const Extent& b) { return apart ? meet(a, b) : !a.empty() && !b.empty() && a.p == b.p; };
    for (const Written* o = outs.begin(); o != outs.end(); ++o) {
        for (const Written* other = outs.begin(); other != o; ++other)
            if (same(o->at, other->at)) return true;
        for (const Extent* in = ins.begin(); in != ins.end(); ++in)
            if (!(in - ins.begin() == o->own && in->p == o->at.p) && same(o->at, *in)) return true;
    }
    return false;
}
// Takes GDR_APART out of an argument.
inline bool take_apart(int& arg) {
    const bool set = arg >= 0 && (arg & GDR_APART);
    if (set) arg &= ~GDR_APART;
    return set;
}

}  // namespace attn
}  // namespace gdr
