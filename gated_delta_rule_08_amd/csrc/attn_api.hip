// C ABI of the attention operators: argument validation and dispatch.  As for
// the mixers, every check runs before the first HIP call.
#include <limits.h>
#include <stdint.h>

#include "attn_backward_plan.h"
#include "gdr_internal.h"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int status_of(hipError_t e) {
    if (e == hipSuccess) return GDR_OK;
    // the launchers report a grid beyond 2^32 work-items this way, before any HIP call
    if (e == hipErrorInvalidConfiguration) return GDR_ERR_BAD_SHAPE;
    return GDR_ERR_HIP;
}

// Element type, head sizes and mask, common to every entry point.
int common_checks(int dtype, int Hq, int Hkv, int d, int window, int sinks) {
    if (dtype != GDR_DTYPE_F32 && dtype != GDR_DTYPE_BF16) return GDR_ERR_BAD_ENUM;
    if (Hq < 0 || Hkv < 0 || window < 0 || sinks < 0) return GDR_ERR_BAD_SHAPE;
    if (d != 64 && d != 128) return GDR_ERR_UNSUPPORTED;
    if (Hkv == 0 || Hq == 0 ? Hq != Hkv : Hq % Hkv != 0) return GDR_ERR_BAD_SHAPE;
    return GDR_OK;
}

// Rows of one sequence (tokens x heads) stay below 2^29 and heads at 2^15, so
// that offsets inside a tile and row numbers fit 32 bits; no tensor passes
// 2^40 elements.
bool sizes_ok(long long B, long long T, long long H, long long d) {
    const long long lim = 1LL << 40;
    if (T >= (1 << 29) || H > (1 << 15) || T * H >= (1 << 29) || B * H > INT_MAX / 8) return false;
    if (T * H > 0 && B > lim / (T * H * d)) return false;
    return true;
}

int page_checks(int Hkv, int page_size, int num_pages, int max_pages) {
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

// The backward's plan for arguments that passed the checks.
gdr::attn::BwdArgs backward_plan(int dtype, int B, int Tq, int Tk, int Hq, int Hkv, int d, int window, int sinks, float scale) {
    window = clamp_window(window, Tk);
    return gdr::attn::make_args(dtype == GDR_DTYPE_F32, B, Tq, Tk, Hq, Hkv, d, window, clamp_sinks(sinks, window, Tk), scale);
}

}  // namespace

extern "C" {

int gdr_attn_prefill(int dtype, int B, int Tq, int Tk, int Hq, int Hkv, int d, int window, int sinks, float scale,
                     const void* q, const void* k, const void* v, void* o, float* lse, void* stream) {
    const int st = common_checks(dtype, Hq, Hkv, d, window, sinks);
    if (st != GDR_OK) return st;
    if (B < 0 || Tq < 0 || Tk < 0 || !sizes_ok(B, Tq, Hq, d) || !sizes_ok(B, Tk, Hkv, d)) return GDR_ERR_BAD_SHAPE;
    if (B == 0 || Tq == 0 || Hq == 0) return GDR_OK;
    if (!q || !o || (Tk > 0 && (!k || !v))) return GDR_ERR_NULL_PTR;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4))
        return GDR_ERR_MISALIGNED;
    window = clamp_window(window, Tk);
    return status_of(gdr::launch_attn_prefill(dtype, B, Tq, Tk, Hq, Hkv, d, window, clamp_sinks(sinks, window, Tk), scale,
                                              q, k, v, o, lse, static_cast<hipStream_t>(stream)));
}

int gdr_attn_prefill_varlen(int dtype, int N, int total_q, int total_k, int max_q, int Hq, int Hkv, int d, int window,
                            int sinks, float scale, const void* q, const void* k, const void* v, const int* cu_q,
                            const int* cu_k, void* o, float* lse, void* stream) {
    const int st = common_checks(dtype, Hq, Hkv, d, window, sinks);
    if (st != GDR_OK) return st;
    if (N < 0 || total_q < 0 || total_k < 0 || max_q < 0) return GDR_ERR_BAD_SHAPE;
    if (max_q > total_q) max_q = total_q;  // a bound may be loose
    if (!sizes_ok(1, total_q, Hq, d) || !sizes_ok(1, total_k, Hkv, d) || !sizes_ok(N, max_q, Hq, 1)) return GDR_ERR_BAD_SHAPE;
    if (N == 0 || max_q == 0 || Hq == 0) return GDR_OK;
    if (!q || !o || !cu_q || !cu_k || (total_k > 0 && (!k || !v))) return GDR_ERR_NULL_PTR;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
        !aligned(cu_q, 4) || !aligned(cu_k, 4))
        return GDR_ERR_MISALIGNED;
    window = clamp_window(window, total_k);
    gdr::AttnPacked pk;
    pk.cu_q = cu_q;
    pk.cu_k = cu_k;
    pk.total_q = total_q;
    pk.total_k = total_k;
    return status_of(gdr::launch_attn_prefill(dtype, N, max_q, 0, Hq, Hkv, d, window, clamp_sinks(sinks, window, total_k),
                                              scale, q, k, v, o, lse, static_cast<hipStream_t>(stream), pk));
}

size_t gdr_attn_backward_workspace_bytes(int dtype, int B, int Tq, int Tk, int Hq, int Hkv, int d, int window,
                                         int sinks) {
    if (common_checks(dtype, Hq, Hkv, d, window, sinks) != GDR_OK || B < 0 || Tq < 0 || Tk < 0 ||
        !sizes_ok(B, Tq, Hq, d) || !sizes_ok(B, Tk, Hkv, d) || B == 0 || Hq == 0 || Tq == 0)
        return 0;
    return gdr::attn::workspace_floats(backward_plan(dtype, B, Tq, Tk, Hq, Hkv, d, window, sinks, 1.f)) * sizeof(float);
}

int gdr_attn_backward(int dtype, int B, int Tq, int Tk, int Hq, int Hkv, int d, int window, int sinks, float scale,
                      const void* q, const void* k, const void* v, const void* o, const float* lse,
                      const void* grad_o, void* grad_q, void* grad_k, void* grad_v, void* workspace,
                      size_t workspace_bytes, void* stream) {
    const int st = common_checks(dtype, Hq, Hkv, d, window, sinks);
    if (st != GDR_OK) return st;
    if (B < 0 || Tq < 0 || Tk < 0 || !sizes_ok(B, Tq, Hq, d) || !sizes_ok(B, Tk, Hkv, d)) return GDR_ERR_BAD_SHAPE;
    if (B == 0 || Hq == 0) return GDR_OK;
    gdr::attn::BwdArgs plan = backward_plan(dtype, B, Tq, Tk, Hq, Hkv, d, window, sinks, scale);
    const size_t need = Tq > 0 ? gdr::attn::workspace_floats(plan) * sizeof(float) : 0;
    if (workspace_bytes < need || (need > 0 && !workspace)) return GDR_ERR_WORKSPACE;
    if (Tq == 0 && Tk == 0) return GDR_OK;
    if (Tq > 0 && (!q || !o || !lse || !grad_o || !grad_q)) return GDR_ERR_NULL_PTR;
    if (Tk > 0 && (!k || !v || !grad_k || !grad_v)) return GDR_ERR_NULL_PTR;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(grad_o, 16) ||
        !aligned(grad_q, 16) || !aligned(grad_k, 16) || !aligned(grad_v, 16) || !aligned(workspace, 16) ||
        !aligned(lse, 4))
        return GDR_ERR_MISALIGNED;
    gdr::attn::set_workspace(plan, static_cast<float*>(workspace));
    return status_of(gdr::launch_attn_backward(dtype, plan, q, k, v, o, lse, grad_o, grad_q, grad_k, grad_v,
                                               static_cast<hipStream_t>(stream)));
}

size_t gdr_attn_decode_workspace_bytes(int dtype, int B, int Hq, int Hkv, int d, int page_size, int max_pages,
                                       int window, int sinks) {
    if (common_checks(dtype, Hq, Hkv, d, window, sinks) != GDR_OK || B < 0 || !sizes_ok(B, 1, Hq, d) ||
        page_checks(Hkv, page_size, 0, max_pages) != GDR_OK || B == 0 || Hq == 0 || max_pages == 0)
        return 0;
    window = clamp_window(window, max_pages * page_size);
    return gdr::attn_decode_workspace_floats(Hq, Hkv, d, page_size, max_pages, window,
                                             clamp_sinks(sinks, window, max_pages * page_size)) *
           sizeof(float);
}

int gdr_attn_decode(int dtype, int B, int Hq, int Hkv, int d, int page_size, int num_pages, int max_pages, int window,
                    int sinks, float scale, const void* q, const void* k, const void* v, void* k_pages, void* v_pages,
                    const int* page_table, const int* lengths, void* o, void* workspace, size_t workspace_bytes,
                    void* stream) {
    int st = common_checks(dtype, Hq, Hkv, d, window, sinks);
    if (st != GDR_OK) return st;
    if (B < 0 || !sizes_ok(B, 1, Hq, d)) return GDR_ERR_BAD_SHAPE;
    if ((st = page_checks(Hkv, page_size, num_pages, max_pages)) != GDR_OK) return st;
    const size_t need = gdr_attn_decode_workspace_bytes(dtype, B, Hq, Hkv, d, page_size, max_pages, window, sinks);
    if (workspace_bytes < need || (need > 0 && !workspace)) return GDR_ERR_WORKSPACE;
    if (B == 0 || Hq == 0 || num_pages == 0 || max_pages == 0) return GDR_OK;
    if (!q || !k || !v || !k_pages || !v_pages || !page_table || !lengths || !o) return GDR_ERR_NULL_PTR;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
        !aligned(o, 16) || !aligned(page_table, 4) || !aligned(lengths, 4) || (need > 0 && !aligned(workspace, 16)))
        return GDR_ERR_MISALIGNED;
    window = clamp_window(window, max_pages * page_size);
    return status_of(gdr::launch_attn_decode(dtype, B, Hq, Hkv, d, page_size, num_pages, max_pages, window,
                                             clamp_sinks(sinks, window, max_pages * page_size), scale, q, k, v, k_pages,
                                             v_pages, page_table, lengths, o, static_cast<float*>(workspace),
                                             static_cast<hipStream_t>(stream)));
}

int gdr_attn_append(int dtype, int N, int total, int Hkv, int d, int page_size, int num_pages, int max_pages,
                    const void* k, const void* v, const int* cu_seqlens, const int* lengths, void* k_pages,
                    void* v_pages, const int* page_table, void* stream) {
    int st = common_checks(dtype, Hkv, Hkv, d, 0, 0);
    if (st != GDR_OK) return st;
    if (N < 0 || total < 0 || !sizes_ok(1, total, Hkv, d)) return GDR_ERR_BAD_SHAPE;
    if ((st = page_checks(Hkv, page_size, num_pages, max_pages)) != GDR_OK) return st;
    if (N == 0 || total == 0 || Hkv == 0 || num_pages == 0 || max_pages == 0) return GDR_OK;
    if (!k || !v || !cu_seqlens || !lengths || !k_pages || !v_pages || !page_table) return GDR_ERR_NULL_PTR;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
        !aligned(cu_seqlens, 4) || !aligned(lengths, 4) || !aligned(page_table, 4))
        return GDR_ERR_MISALIGNED;
    return status_of(gdr::launch_attn_append(dtype, N, total, Hkv, d, page_size, num_pages, max_pages, k, v, cu_seqlens,
                                             lengths, k_pages, v_pages, page_table, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
