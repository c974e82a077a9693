// C ABI of the operators around the attention layers: norm and rotation of queries
// and keys, the page plan, and the 4-bit cache.  Argument validation and dispatch;
// every check runs before the first HIP call.
#include <initializer_list>

#include "attn_checks.h"

using namespace gdr::attn;

namespace {

int rope_checks(int dtype, int flags, int tokens, int Hq, int Hkv, int d, int rot) {
    if (dtype != GDR_DTYPE_F32 && dtype != GDR_DTYPE_BF16) return GDR_ERR_BAD_ENUM;
    if (flags & ~(GDR_ROPE_INTERLEAVED | GDR_ROPE_NO_NORM)) return GDR_ERR_BAD_ENUM;
    if (tokens < 0 || Hq < 0 || Hkv < 0 || rot < 0) return GDR_ERR_BAD_SHAPE;
    if (d != 64 && d != 128) return GDR_ERR_UNSUPPORTED;
    if (rot > d || rot % 16) return GDR_ERR_UNSUPPORTED;
    if (Hq > (1 << 15) || Hkv > (1 << 15) || static_cast<long long>(tokens) * (Hq + Hkv) >= (1 << 29)) return GDR_ERR_BAD_SHAPE;
    return GDR_OK;
}

// Elements from token to token of a [tokens, H, d] tensor whose tokens may lie apart.
int stride_checks(int dtype, int tokens, int H, int d, long long stride) {
    if (H == 0 || tokens == 0) return GDR_OK;
    if (stride < static_cast<long long>(H) * d || stride > (1LL << 40) / tokens) return GDR_ERR_BAD_SHAPE;
    return stride % (dtype == GDR_DTYPE_F32 ? 4 : 8) ? GDR_ERR_MISALIGNED : GDR_OK;
}

// Whether a tensor that is written (and exists) is another of the call's.
bool any_of(const void* out, std::initializer_list<const void*> others) {
    for (const void* p : others)
        if (out && out == p) return true;
    return false;
}

// An output may be its input if it lies the same way.
bool same_way(const void* in, const void* out, long long in_stride, long long out_stride) {
    return in != out || in_stride == out_stride;
}

int mx4_checks(int dtype, int Hkv, int d, int page_size, int num_pages, int max_pages) {
    int st = common_checks(dtype, Hkv, Hkv, d, 0, 0);
    if (st != GDR_OK) return st;
    if (Hkv > (1 << 15)) return GDR_ERR_BAD_SHAPE;
    if ((st = page_checks(Hkv, page_size, num_pages, max_pages)) != GDR_OK) return st;
    return page_size < 32 ? GDR_ERR_UNSUPPORTED : GDR_OK;
}

bool cache_aligned(const void* a, const void* b, const void* c, const void* d) {
    return aligned(a, 16) && aligned(b, 16) && aligned(c, 16) && aligned(d, 16);
}

}  // namespace

extern "C" {

int gdr_attn_norm_rope(int dtype, int flags, int tokens, int Hq, int Hkv, int d, int rot, float eps, long long q_stride,
                       long long k_stride, const void* q, const void* k, const float* w_q, const float* w_k,
                       const int* positions, const float* inv_freq, void* q_out, void* k_out, void* stream) {
    int st = rope_checks(dtype, flags, tokens, Hq, Hkv, d, rot);
    if (st != GDR_OK) return st;
    if ((flags & GDR_ROPE_NO_NORM) && (w_q || w_k)) return GDR_ERR_UNSUPPORTED;
    if (tokens == 0 || Hq + Hkv == 0) return GDR_OK;
    if ((Hq && (!q || !q_out)) || (Hkv && (!k || !k_out)) || (rot && (!positions || !inv_freq))) return GDR_ERR_NULL_PTR;
    if ((st = stride_checks(dtype, tokens, Hq, d, q_stride)) != GDR_OK) return st;
    if ((st = stride_checks(dtype, tokens, Hkv, d, k_stride)) != GDR_OK) return st;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(w_q, 4) ||
        !aligned(w_k, 4) || !aligned(positions, 4) || !aligned(inv_freq, 4))
        return GDR_ERR_MISALIGNED;
    if ((Hq && !same_way(q, q_out, q_stride, static_cast<long long>(Hq) * d)) ||
        (Hkv && !same_way(k, k_out, k_stride, static_cast<long long>(Hkv) * d)))
        return GDR_ERR_ALIAS;
    if (Hq && Hkv && (any_of(q_out, {k, k_out}) || any_of(k_out, {q}))) return GDR_ERR_ALIAS;
    return status_of(gdr::launch_attn_rope(dtype, tokens, Hq, Hkv, d, rot, flags & GDR_ROPE_INTERLEAVED,
                                           !(flags & GDR_ROPE_NO_NORM), eps, q_stride, k_stride, q, k, w_q, w_k, positions,
                                           inv_freq, q_out, k_out, static_cast<hipStream_t>(stream)));
}

size_t gdr_attn_norm_rope_backward_workspace_bytes(int dtype, int tokens, int Hq, int Hkv, int d) {
    if (rope_checks(dtype, 0, tokens, Hq, Hkv, d, 0) != GDR_OK || tokens == 0 || Hq + Hkv == 0) return 0;
    return gdr::attn_rope_backward_workspace_floats(tokens, Hq, Hkv, d) * sizeof(float);
}

int gdr_attn_norm_rope_backward(int dtype, int flags, int tokens, int Hq, int Hkv, int d, int rot, float eps,
                                long long q_stride, long long k_stride, long long grad_q_stride, long long grad_k_stride,
                                const void* q, const void* k, const float* w_q, const float* w_k, const int* positions,
                                const float* inv_freq, const void* grad_q_out, const void* grad_k_out, void* grad_q,
                                void* grad_k, float* grad_w_q, float* grad_w_k, void* workspace, size_t workspace_bytes,
                                void* stream) {
    int st = rope_checks(dtype, flags, tokens, Hq, Hkv, d, rot);
    if (st != GDR_OK) return st;
    const bool norm = !(flags & GDR_ROPE_NO_NORM), weights = grad_w_q || grad_w_k;
    if (!norm && (w_q || w_k || weights)) return GDR_ERR_UNSUPPORTED;
    const bool none = tokens == 0 || Hq + Hkv == 0;
    const size_t need = weights ? gdr_attn_norm_rope_backward_workspace_bytes(dtype, tokens, Hq, Hkv, d) : 0;
    if (workspace_bytes < need || (need && !workspace)) return GDR_ERR_WORKSPACE;
    if (none && !weights) return GDR_OK;
    if (!none) {
        if ((Hq && (!grad_q_out || !grad_q || (norm && !q))) || (Hkv && (!grad_k_out || !grad_k || (norm && !k))) ||
            (rot && (!positions || !inv_freq)))
            return GDR_ERR_NULL_PTR;
        if (norm && ((st = stride_checks(dtype, tokens, Hq, d, q_stride)) != GDR_OK ||
                     (st = stride_checks(dtype, tokens, Hkv, d, k_stride)) != GDR_OK))
            return st;
        if ((st = stride_checks(dtype, tokens, Hq, d, grad_q_stride)) != GDR_OK ||
            (st = stride_checks(dtype, tokens, Hkv, d, grad_k_stride)) != GDR_OK)
            return st;
    }
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(grad_q_out, 16) || !aligned(grad_k_out, 16) || !aligned(grad_q, 16) ||
        !aligned(grad_k, 16) || !aligned(w_q, 4) || !aligned(w_k, 4) || !aligned(positions, 4) || !aligned(inv_freq, 4) ||
        !aligned(grad_w_q, 4) || !aligned(grad_w_k, 4) || (need && !aligned(workspace, 16)))
        return GDR_ERR_MISALIGNED;
    if (!none && ((Hq && !same_way(grad_q_out, grad_q, static_cast<long long>(Hq) * d, grad_q_stride)) ||
                  (Hkv && !same_way(grad_k_out, grad_k, static_cast<long long>(Hkv) * d, grad_k_stride))))
        return GDR_ERR_ALIAS;
    const void *q_read = norm ? q : nullptr, *k_read = norm ? k : nullptr;
    if (any_of(grad_w_q, {grad_w_k}) ||
        (!none && ((Hq && any_of(grad_q, {q_read})) || (Hkv && any_of(grad_k, {k_read})) ||
                   (Hq && Hkv && (any_of(grad_q, {k_read, grad_k_out, grad_k}) || any_of(grad_k, {q_read, grad_q_out}))))))
        return GDR_ERR_ALIAS;
    return status_of(gdr::launch_attn_rope_backward(dtype, none ? 0 : tokens, Hq, Hkv, d, rot, flags & GDR_ROPE_INTERLEAVED, norm, eps,
                                                    q_stride, k_stride, grad_q_stride, grad_k_stride, q, k, w_q, w_k,
                                                    positions, inv_freq, grad_q_out, grad_k_out, grad_q, grad_k, grad_w_q,
                                                    grad_w_k, static_cast<float*>(workspace),
                                                    static_cast<hipStream_t>(stream)));
}

int gdr_attn_plan_pages(int N, int page_size, int max_pages, int n_stack, int max_tokens, const int* lengths, const int* add,
                        const int* free_pages, const int* n_free, int* page_table, int* cu_seqlens, int* added,
                        int* lengths_out, int* slots, int* n_free_out, void* stream) {
    const int st = page_checks(0, page_size, 0, max_pages);
    if (st != GDR_OK) return st;
    if (N < 0 || N == INT_MAX || n_stack < 0 || max_tokens < 0) return GDR_ERR_BAD_SHAPE;
    if (!n_free || !n_free_out || !cu_seqlens || (N && (!lengths || !add || !added || !lengths_out)) ||
        (N && max_pages && !page_table) || (n_stack && !free_pages))
        return GDR_ERR_NULL_PTR;
    const void* all[] = {lengths, add, free_pages, n_free, page_table, cu_seqlens, added, lengths_out, slots, n_free_out};
    for (const void* p : all)
        if (!aligned(p, 4)) return GDR_ERR_MISALIGNED;
    if (N) {
        const void* outs[] = {page_table, cu_seqlens, added, lengths_out, slots, n_free_out};
        const void* own[] = {nullptr, nullptr, add, lengths, nullptr, n_free};  // the input that each may be
        const void* ins[] = {lengths, add, free_pages, n_free};
        for (int i = 0; i < 6; ++i) {
            for (int j = 0; j < i; ++j)
                if (any_of(outs[i], {outs[j]})) return GDR_ERR_ALIAS;
            for (const void* in : ins)
                if (in != own[i] && any_of(outs[i], {in})) return GDR_ERR_ALIAS;
        }
    }
    return status_of(gdr::launch_attn_plan_pages(N, page_size, max_pages, n_stack, max_tokens, lengths, add, free_pages, n_free,
                                                 page_table, cu_seqlens, added, lengths_out, slots, n_free_out,
                                                 static_cast<hipStream_t>(stream)));
}

int gdr_attn_append_mx4(int dtype, int N, int total, int Hkv, int d, int page_size, int num_pages, int max_pages,
                        const void* k, const void* v, const int* cu_seqlens, const int* lengths, void* k_codes, void* k_scales,
                        void* v_codes, void* v_scales, const int* page_table, void* stream) {
    const int st = mx4_checks(dtype, Hkv, d, page_size, num_pages, max_pages);
    if (st != GDR_OK) return st;
    if (N < 0 || total < 0 || !sizes_ok(1, total, Hkv, d)) return GDR_ERR_BAD_SHAPE;
    if (N == 0 || total == 0 || Hkv == 0 || num_pages == 0 || max_pages == 0) return GDR_OK;
    if (!k || !v || !cu_seqlens || !lengths || !k_codes || !k_scales || !v_codes || !v_scales || !page_table)
        return GDR_ERR_NULL_PTR;
    if (!aligned(k, 16) || !aligned(v, 16) || !cache_aligned(k_codes, k_scales, v_codes, v_scales) ||
        !aligned(cu_seqlens, 4) || !aligned(lengths, 4) || !aligned(page_table, 4))
        return GDR_ERR_MISALIGNED;
    if (any_of(k_codes, {v_codes, k, v}) || any_of(v_codes, {k, v}) || any_of(k_scales, {v_scales})) return GDR_ERR_ALIAS;
    return status_of(gdr::launch_attn_append_mx4(dtype, N, total, Hkv, d, page_size, num_pages, max_pages, k, v, cu_seqlens,
                                                 lengths, k_codes, k_scales, v_codes, v_scales, page_table,
                                                 static_cast<hipStream_t>(stream)));
}

int gdr_attn_read_mx4(int dtype, int N, int total, int Hkv, int d, int page_size, int num_pages, int max_pages,
                      const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                      const int* page_table, const int* cu_seqlens, const int* first, void* k, void* v, void* stream) {
    const int st = mx4_checks(dtype, Hkv, d, page_size, num_pages, max_pages);
    if (st != GDR_OK) return st;
    if (N < 0 || total < 0 || !sizes_ok(1, total, Hkv, d)) return GDR_ERR_BAD_SHAPE;
    if (N == 0 || total == 0 || Hkv == 0 || num_pages == 0 || max_pages == 0) return GDR_OK;
    if (!k || !v || !cu_seqlens || !k_codes || !k_scales || !v_codes || !v_scales || !page_table) return GDR_ERR_NULL_PTR;
    if (!aligned(k, 16) || !aligned(v, 16) || !cache_aligned(k_codes, k_scales, v_codes, v_scales) ||
        !aligned(cu_seqlens, 4) || !aligned(first, 4) || !aligned(page_table, 4))
        return GDR_ERR_MISALIGNED;
    if (any_of(k, {v})) return GDR_ERR_ALIAS;
    return status_of(gdr::launch_attn_read_mx4(dtype, N, total, Hkv, d, page_size, num_pages, max_pages, k_codes, k_scales,
                                               v_codes, v_scales, page_table, cu_seqlens, first, k, v,
                                               static_cast<hipStream_t>(stream)));
}

// What the decode step and its workspace query agree on.
static int decode_mx4_checks(int dtype, int B, int Tq, int Hq, int Hkv, int d, int page_size, int num_pages, int max_pages,
                             int window, int sinks) {
    int st = common_checks(dtype, Hq, Hkv, d, window, sinks);
    if (st != GDR_OK) return st;
    if ((st = mx4_checks(dtype, Hkv, d, page_size, num_pages, max_pages)) != GDR_OK) return st;
    if (B < 0 || Tq < 0) return GDR_ERR_BAD_SHAPE;
    if (Tq > 64) return GDR_ERR_UNSUPPORTED;
    return sizes_ok(B, Tq, Hq, d) ? GDR_OK : GDR_ERR_BAD_SHAPE;
}

size_t gdr_attn_decode_mx4_workspace_bytes(int dtype, int B, int Tq, int Hq, int Hkv, int d, int page_size, int max_pages,
                                           int window, int sinks) {
    if (decode_mx4_checks(dtype, B, Tq, Hq, Hkv, d, page_size, 0, max_pages, window, sinks) != GDR_OK || B == 0 || Tq == 0 ||
        Hq == 0 || max_pages == 0)
        return 0;
    window = clamp_window(window, max_pages * page_size);
    return gdr::attn_decode_mx4_workspace_floats(Tq, Hq, Hkv, d, page_size, max_pages, window,
                                                 clamp_sinks(sinks, window, max_pages * page_size)) *
           sizeof(float);
}

int gdr_attn_decode_mx4(int dtype, int B, int Tq, int Hq, int Hkv, int d, int page_size, int num_pages, int max_pages,
                        int window, int sinks, float scale, const void* q, const void* k_codes, const void* k_scales,
                        const void* v_codes, const void* v_scales, const int* page_table, const int* lengths, void* o,
                        void* workspace, size_t workspace_bytes, void* stream) {
    const int st = decode_mx4_checks(dtype, B, Tq, Hq, Hkv, d, page_size, num_pages, max_pages, window, sinks);
    if (st != GDR_OK) return st;
    const size_t need = gdr_attn_decode_mx4_workspace_bytes(dtype, B, Tq, Hq, Hkv, d, page_size, max_pages, window, sinks);
    if (workspace_bytes < need || (need > 0 && !workspace)) return GDR_ERR_WORKSPACE;
    if (B == 0 || Tq == 0 || Hq == 0 || num_pages == 0 || max_pages == 0) return GDR_OK;
    if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !page_table || !lengths || !o) return GDR_ERR_NULL_PTR;
    if (!aligned(q, 16) || !aligned(o, 16) || !cache_aligned(k_codes, k_scales, v_codes, v_scales) ||
        !aligned(page_table, 4) || !aligned(lengths, 4) || (need > 0 && !aligned(workspace, 16)))
        return GDR_ERR_MISALIGNED;
    window = clamp_window(window, max_pages * page_size);
    return status_of(gdr::launch_attn_decode_mx4(dtype, B, Tq, Hq, Hkv, d, page_size, num_pages, max_pages, window,
                                                 clamp_sinks(sinks, window, max_pages * page_size), scale, q, k_codes, k_scales,
                                                 v_codes, v_scales, page_table, lengths, o, static_cast<float*>(workspace),
                                                 static_cast<hipStream_t>(stream)));
}

}  // extern "C"
