// C ABI of the operators around the attention layers: norm and rotation of queries
// and keys, the page plan, and the 4-bit cache.  Argument validation and dispatch;
// every check runs before the first HIP call.
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

int size_of(int dtype) { return dtype == GDR_DTYPE_F32 ? 4 : 2; }

// The 4-bit cache's tensors.
struct CacheExtents {
    Extent k_codes, k_scales, v_codes, v_scales;
};
CacheExtents cache_extents(int Hkv, int d, int page_size, int num_pages, const void* kc, const void* ks, const void* vc,
                           const void* vs) {
    const long long rows = static_cast<long long>(num_pages) * Hkv * page_size;
    return {dense(kc, rows * (d / 2)), dense(ks, rows * (d / 32)), dense(vc, rows * (d / 2)), dense(vs, rows * (d / 32))};
}

bool cache_aligned(const void* a, const void* b, const void* c, const void* d) {
    return aligned(a, 16) && aligned(b, 16) && aligned(c, 16) && aligned(d, 16);
}

}  // namespace

extern "C" {

int gdr_attn_norm_rope(int dtype, int flags, int tokens, int Hq, int Hkv, int d, int rot, float eps, long long q_stride,
                       long long k_stride, const void* q, const void* k, const float* w_q, const float* w_k,
                       const int* positions, const float* inv_freq, void* q_out, void* k_out, void* stream) {
    const bool apart = take_apart(dtype);
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
    const int e = size_of(dtype);
    const long long qe = static_cast<long long>(Hq) * d, ke = static_cast<long long>(Hkv) * d, angles = rot ? tokens : 0;
    if (aliased(apart, {{dense(q_out, tokens * qe * e), 0}, {dense(k_out, tokens * ke * e), 1}},
                {tokens_of(q, tokens, qe, q_stride, e), tokens_of(k, tokens, ke, k_stride, e), dense(w_q, 4 * d), dense(w_k, 4 * d),
                 dense(positions, 4 * angles), dense(inv_freq, 2 * rot)}))
        return GDR_ERR_ALIAS;
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
    const bool apart = take_apart(dtype);
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
    if ((norm && (!aligned(q, 16) || !aligned(k, 16))) || !aligned(grad_q_out, 16) || !aligned(grad_k_out, 16) ||
        !aligned(grad_q, 16) || !aligned(grad_k, 16) || !aligned(w_q, 4) || !aligned(w_k, 4) || !aligned(positions, 4) || !aligned(inv_freq, 4) ||
        !aligned(grad_w_q, 4) || !aligned(grad_w_k, 4) || (need && !aligned(workspace, 16)))
        return GDR_ERR_MISALIGNED;
    if (!none && ((Hq && !same_way(grad_q_out, grad_q, static_cast<long long>(Hq) * d, grad_q_stride)) ||
                  (Hkv && !same_way(grad_k_out, grad_k, static_cast<long long>(Hkv) * d, grad_k_stride))))
        return GDR_ERR_ALIAS;
    const int e = size_of(dtype);
    const long long n = none ? 0 : tokens, qe = static_cast<long long>(Hq) * d, ke = static_cast<long long>(Hkv) * d;
    const long long read = norm ? n : 0, angles = rot ? n : 0;
    if (aliased(apart,
                {{tokens_of(grad_q, n, qe, grad_q_stride, e), 6}, {tokens_of(grad_k, n, ke, grad_k_stride, e), 7},
                 {dense(grad_w_q, 4 * d), -1}, {dense(grad_w_k, 4 * d), -1}, {dense(workspace, static_cast<long long>(need)), -1}},
                {tokens_of(q, read, qe, q_stride, e), tokens_of(k, read, ke, k_stride, e), dense(w_q, n ? 4 * d : 0),
                 dense(w_k, n ? 4 * d : 0), dense(positions, 4 * angles), dense(inv_freq, angles ? 2 * rot : 0),
                 dense(grad_q_out, n * qe * e), dense(grad_k_out, n * ke * e)}))
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
    const bool apart = take_apart(page_size);
    const int st = page_checks(0, page_size, 0, max_pages);
    if (st != GDR_OK) return st;
    if (N < 0 || N == INT_MAX || n_stack < 0 || max_tokens < 0) return GDR_ERR_BAD_SHAPE;
    if (!n_free || !n_free_out || !cu_seqlens || (N && (!lengths || !add || !added || !lengths_out)) ||
        (N && max_pages && !page_table) || (n_stack && !free_pages))
        return GDR_ERR_NULL_PTR;
    const void* all[] = {lengths, add, free_pages, n_free, page_table, cu_seqlens, added, lengths_out, slots, n_free_out};
    for (const void* p : all)
        if (!aligned(p, 4)) return GDR_ERR_MISALIGNED;
    const long long n = 4ll * N;
    if (aliased(apart,
                {{table_of(page_table, N, max_pages), -1}, {dense(cu_seqlens, n + 4), -1}, {dense(added, n), 1},
                 {dense(lengths_out, n), 0}, {dense(slots, N ? 4ll * max_tokens : 0), -1}, {dense(n_free_out, 4), 3}},
                {dense(lengths, n), dense(add, n), dense(free_pages, N ? 4ll * n_stack : 0), dense(n_free, 4)}))
        return GDR_ERR_ALIAS;
    return status_of(gdr::launch_attn_plan_pages(N, page_size, max_pages, n_stack, max_tokens, lengths, add, free_pages, n_free,
                                                 page_table, cu_seqlens, added, lengths_out, slots, n_free_out,
                                                 static_cast<hipStream_t>(stream)));
}

int gdr_attn_append_mx4(int dtype, int N, int total, int Hkv, int d, int page_size, int num_pages, int max_pages,
                        const void* k, const void* v, const int* cu_seqlens, const int* lengths, void* k_codes, void* k_scales,
                        void* v_codes, void* v_scales, const int* page_table, void* stream) {
    const bool apart = take_apart(dtype);
    const int st = mx4_checks(dtype, Hkv, d, page_size, num_pages, max_pages);
    if (st != GDR_OK) return st;
    if (N < 0 || total < 0 || !sizes_ok(1, total, Hkv, d)) return GDR_ERR_BAD_SHAPE;
    if (N == 0 || total == 0 || Hkv == 0 || num_pages == 0 || max_pages == 0) return GDR_OK;
    if (!k || !v || !cu_seqlens || !lengths || !k_codes || !k_scales || !v_codes || !v_scales || !page_table)
        return GDR_ERR_NULL_PTR;
    if (!aligned(k, 16) || !aligned(v, 16) || !cache_aligned(k_codes, k_scales, v_codes, v_scales) ||
        !aligned(cu_seqlens, 4) || !aligned(lengths, 4) || !aligned(page_table, 4))
        return GDR_ERR_MISALIGNED;
    const CacheExtents c = cache_extents(Hkv, d, page_size, num_pages, k_codes, k_scales, v_codes, v_scales);
    const long long bytes = static_cast<long long>(total) * Hkv * d * size_of(dtype), n = 4ll * N;
    if (aliased(apart, {{c.k_codes, -1}, {c.k_scales, -1}, {c.v_codes, -1}, {c.v_scales, -1}},
                {dense(k, bytes), dense(v, bytes), dense(cu_seqlens, n + 4), dense(lengths, n), table_of(page_table, N, max_pages)}))
        return GDR_ERR_ALIAS;
    return status_of(gdr::launch_attn_append_mx4(dtype, N, total, Hkv, d, page_size, num_pages, max_pages, k, v, cu_seqlens,
                                                 lengths, k_codes, k_scales, v_codes, v_scales, page_table,
                                                 static_cast<hipStream_t>(stream)));
}

int gdr_attn_read_mx4(int dtype, int N, int total, int Hkv, int d, int page_size, int num_pages, int max_pages,
                      const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                      const int* page_table, const int* cu_seqlens, const int* first, void* k, void* v, void* stream) {
    const bool apart = take_apart(dtype);
    const int st = mx4_checks(dtype, Hkv, d, page_size, num_pages, max_pages);
    if (st != GDR_OK) return st;
    if (N < 0 || total < 0 || !sizes_ok(1, total, Hkv, d)) return GDR_ERR_BAD_SHAPE;
    if (N == 0 || total == 0 || Hkv == 0 || num_pages == 0 || max_pages == 0) return GDR_OK;
    if (!k || !v || !cu_seqlens || !k_codes || !k_scales || !v_codes || !v_scales || !page_table) return GDR_ERR_NULL_PTR;
    if (!aligned(k, 16) || !aligned(v, 16) || !cache_aligned(k_codes, k_scales, v_codes, v_scales) ||
        !aligned(cu_seqlens, 4) || !aligned(first, 4) || !aligned(page_table, 4))
        return GDR_ERR_MISALIGNED;
    const CacheExtents c = cache_extents(Hkv, d, page_size, num_pages, k_codes, k_scales, v_codes, v_scales);
    const long long bytes = static_cast<long long>(total) * Hkv * d * size_of(dtype), n = 4ll * N;
    if (aliased(apart, {{dense(k, bytes), -1}, {dense(v, bytes), -1}},
                {c.k_codes, c.k_scales, c.v_codes, c.v_scales, dense(cu_seqlens, n + 4), dense(first, n),
                 table_of(page_table, N, max_pages)}))
        return GDR_ERR_ALIAS;
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
    const bool apart = take_apart(dtype);
    const int st = decode_mx4_checks(dtype, B, Tq, Hq, Hkv, d, page_size, num_pages, max_pages, window, sinks);
    if (st != GDR_OK) return st;
    const size_t need = gdr_attn_decode_mx4_workspace_bytes(dtype, B, Tq, Hq, Hkv, d, page_size, max_pages, window, sinks);
    if (workspace_bytes < need || (need > 0 && !workspace)) return GDR_ERR_WORKSPACE;
    if (B == 0 || Tq == 0 || Hq == 0 || num_pages == 0 || max_pages == 0) return GDR_OK;
    if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !page_table || !lengths || !o) return GDR_ERR_NULL_PTR;
    if (!aligned(q, 16) || !aligned(o, 16) || !cache_aligned(k_codes, k_scales, v_codes, v_scales) ||
        !aligned(page_table, 4) || !aligned(lengths, 4) || (need > 0 && !aligned(workspace, 16)))
        return GDR_ERR_MISALIGNED;
    const CacheExtents c = cache_extents(Hkv, d, page_size, num_pages, k_codes, k_scales, v_codes, v_scales);
    const long long bytes = static_cast<long long>(B) * Tq * Hq * d * size_of(dtype);
    if (aliased(apart, {{dense(o, bytes), 0}, {dense(workspace, static_cast<long long>(need)), -1}},
                {dense(q, bytes), c.k_codes, c.k_scales, c.v_codes, c.v_scales, table_of(page_table, B, max_pages),
                 dense(lengths, 4ll * B)}))
        return GDR_ERR_ALIAS;
    window = clamp_window(window, max_pages * page_size);
    return status_of(gdr::launch_attn_decode_mx4(dtype, B, Tq, Hq, Hkv, d, page_size, num_pages, max_pages, window,
                                                 clamp_sinks(sinks, window, max_pages * page_size), scale, q, k_codes, k_scales,
                                                 v_codes, v_scales, page_table, lengths, o, static_cast<float*>(workspace),
                                                 static_cast<hipStream_t>(stream)));
}

}  // extern "C"
