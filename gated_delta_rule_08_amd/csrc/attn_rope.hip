// Norm of queries and keys for each head with the position rotation in the same
// pass, and its backward.
//
// A row is one head's d channels of one token, q's and k's alike.  With
// r = 1 / sqrt(mean x^2 + eps) and weights w, y = x r w; then the pairs of the
// first `rot` channels are turned by the angle position * inv_freq[i]:
// (y_i, y_{i + rot/2}), or (y_2i, y_2i+1) where interleaved.
// Backward, with u the gradient turned back: grad_w = sum over rows of u x r, and
// grad_x = r (u w - x r mean(u w x r)).
//
// Both passes move every row once each way and do little with it: HBM-bound (8192
// tokens of 32 query and 8 key heads, d=128, bf16: forward 168 MB in 34 us, backward
// 252 MB in 48 and 5 for the join).  A lane has two groups of Q = 4 or 8 channels (8
// or 16 bytes) that hold its pairs whole, so a rotation needs no other lane, and a
// row takes d / 2Q lanes; the norm's sum is two to four exchanges inside 16 lanes.
// The angles' cosines and sines belong to a token and are formed once for all its
// heads, in LDS.
#include <type_traits>

#include "attn_common.h"

namespace gdr {
namespace attn {
namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
    int rows, Hq, H;    // all rows, query heads, heads of a token (queries first)
    int chunk;          // rows of a workgroup's chunk
    int rot, norm;
    float eps;
    FastDiv heads;
    long long q_stride, k_stride;    // elements from token to token: of q, k
    long long gq_stride, gk_stride;  // and of the outputs q_out, k_out or grad_q, grad_k
};

// Sum over the L lanes of a row (16, 8 or 4, aligned): each step adds a lane of the
// other half of 2, 4, 8, 16.
template <int CTRL> __device__ __forceinline__ float dpp_add(float x) {
    const int y = __builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true);
    return x + __int_as_float(y);
}
template <int L> __device__ __forceinline__ float row_sum(float x) {
    x = dpp_add<0xB1>(x);                          // 1 0 3 2
    x = dpp_add<0x4E>(x);                          // 2 3 0 1
    if constexpr (L >= 8) x = dpp_add<0x141>(x);   // mirror of 8
    if constexpr (L == 16) x = dpp_add<0x140>(x);  // mirror of 16
    return x;
}

// cos and sin of position * frequency.  The angle is formed and brought into a
// quarter turn in double: far positions keep their angle to fp32's last place.
__device__ __forceinline__ void turn_of(int position, float frequency, float& c, float& s) {
    const double t = static_cast<double>(position) * static_cast<double>(frequency) * 0.63661977236758134308;  // quarter turns
    const double n = rint(t);
    const int quadrant = static_cast<int>(static_cast<long long>(n) & 3);
    float sn, cs;
    sincospif(static_cast<float>(t - n) * 0.5f, &sn, &cs);
    c = quadrant & 1 ? sn : cs;
    s = quadrant & 1 ? cs : sn;
    if (quadrant == 1 || quadrant == 2) c = -c;
    if (quadrant >= 2) s = -s;
}

// What a lane holds of a row: channels a .. a + Q - 1 and b .. b + Q - 1, and its Q
// angles from `angle` on (-1: not rotated).
struct Lane {
    int a, b, angle;
};
template <int Q, bool IL> __device__ __forceinline__ Lane lane_of(int x, int rot) {
    Lane l;
    const bool turns = x < rot / (2 * Q);
    l.angle = turns ? Q * x : -1;
    if (IL || !turns) {
        l.a = 2 * Q * x;
        l.b = 2 * Q * x + Q;
    } else {
        l.a = Q * x;
        l.b = rot / 2 + Q * x;
    }
    return l;
}
template <int Q> __device__ __forceinline__ int channel_of(const Lane& l, int i) { return (i < Q ? l.a : l.b) + i % Q; }

template <int Q> __device__ __forceinline__ void load_group(const float* p, float* x) {
#pragma unroll
    for (int y = 0; y < Q; y += 4) {
        const f32x4 u = *reinterpret_cast<const f32x4*>(p + y);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[y + i] = u[i];
    }
}
template <int Q> __device__ __forceinline__ void load_group(const bf16_t* p, float* x) {
    typedef uint32_t words __attribute__((ext_vector_type(Q / 2)));
    const words u = *reinterpret_cast<const words*>(p);
#pragma unroll
    for (int i = 0; i < Q / 2; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
template <int Q> __device__ __forceinline__ void store_group(float* p, const float* x) {
#pragma unroll
    for (int y = 0; y < Q; y += 4) store4<float>(p + y, x[y], x[y + 1], x[y + 2], x[y + 3]);
}
template <int Q> __device__ __forceinline__ void store_group(bf16_t* p, const float* x) {
    typedef __bf16 group __attribute__((ext_vector_type(Q)));
    group g;
#pragma unroll
    for (int i = 0; i < Q; ++i) g[i] = static_cast<__bf16>(x[i]);
    *reinterpret_cast<group*>(p) = g;
}

// The pairs of x[0 .. Q - 1] (group a) and the rest (group b) turned by the lane's angles.
template <int Q, bool IL> __device__ __forceinline__ void rotate(float (&x)[2 * Q], const float (&c)[Q], const float (&s)[Q]) {
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        float &p = IL ? x[2 * i] : x[i], &q = IL ? x[2 * i + 1] : x[Q + i];
        const float u = p * c[i] - q * s[i], v = q * c[i] + p * s[i];
        p = u;
        q = v;
    }
}

// The angles of tokens t0 .. t1 in LDS: cosines, then sines, rot / 2 of each a token.
__device__ __forceinline__ void fill_turns(float* turns, int t0, int t1, int half, const int* __restrict__ positions,
                                           const float* __restrict__ inv_freq) {
    for (int i = threadIdx.x; i < (t1 - t0 + 1) * half; i += kRopeThreads) {
        const int t = i / half, x = i - t * half;
        float c, s;
        turn_of(positions[t0 + t], inv_freq[x], c, s);
        turns[t * 2 * half + x] = c;
        turns[t * 2 * half + half + x] = s;
    }
}

template <typename T, int D, bool IL, int Q>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a, const T* q, const T* k, const float* __restrict__ w_q,
                                                            const float* __restrict__ w_k,
                                                            const int* __restrict__ positions,
                                                            const float* __restrict__ inv_freq, T* q_out, T* k_out) {
    constexpr int L = D / (2 * Q), N = 2 * Q;
    extern __shared__ __align__(16) float turns[];
    const int half = a.rot / 2;
    const int r0 = blockIdx.x * a.chunk, r1 = min(a.rows, r0 + a.chunk), t0 = a.heads(r0);
    if (half) {
        fill_turns(turns, t0, a.heads(r1 - 1), half, positions, inv_freq);
        __syncthreads();
    }
    const Lane ln = lane_of<Q, IL>(threadIdx.x % L, a.rot);
    float wq[N], wk[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int ch = channel_of<Q>(ln, i);
        wq[i] = a.norm && w_q ? w_q[ch] : 1.f;
        wk[i] = a.norm && w_k ? w_k[ch] : 1.f;
    }
    for (int r = r0 + threadIdx.x / L; r < r1; r += kRopeThreads / L) {  // a row's lanes go together
        const int t = a.heads(r), h = r - t * a.H;
        const bool key = h >= a.Hq;
        const T* p = key ? k + t * a.k_stride + static_cast<long long>(h - a.Hq) * D
                         : q + t * a.q_stride + static_cast<long long>(h) * D;
        T* to = key ? k_out + t * a.gk_stride + static_cast<long long>(h - a.Hq) * D
                    : q_out + t * a.gq_stride + static_cast<long long>(h) * D;
        float x[N];
        load_group<Q>(p + ln.a, x);
        load_group<Q>(p + ln.b, x + Q);
        if (a.norm) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) sum = fmaf(x[i], x[i], sum);
            const float inv = rsqrtf(row_sum<L>(sum) * (1.f / D) + a.eps);
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = x[i] * inv * (key ? wk[i] : wq[i]);
        }
        if (ln.angle >= 0) {
            float c[Q], s[Q];
            load_group<Q>(turns + (t - t0) * 2 * half + ln.angle, c);
            load_group<Q>(turns + (t - t0) * 2 * half + half + ln.angle, s);
            rotate<Q, IL>(x, c, s);
        }
        store_group<Q>(to + ln.a, x);
        store_group<Q>(to + ln.b, x + Q);
    }
}

constexpr int kBackwardGroup = 4;

// Chunks go round the workgroups; each leaves its rows' part of the weights'
// gradients, [2][D], to the join, so that their sums are added in a fixed order.
template <typename T, int D, bool IL>
__global__ __launch_bounds__(kRopeThreads) void rope_backward_kernel(
    RopeArgs a, const T* __restrict__ q, const T* __restrict__ k, const float* __restrict__ w_q,
    const float* __restrict__ w_k, const int* __restrict__ positions, const float* __restrict__ inv_freq, const T* g_q_out,
    const T* g_k_out, T* g_q, T* g_k, float* __restrict__ part) {
    constexpr int Q = kBackwardGroup, L = D / (2 * Q), N = 2 * Q, kGroups = kRopeThreads / L;
    extern __shared__ __align__(16) float turns[];
    const int half = a.rot / 2;
    const Lane ln = lane_of<Q, IL>(threadIdx.x % L, a.rot);
    float wq[N], wk[N], sq[N] = {}, sk[N] = {};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int ch = channel_of<Q>(ln, i);
        wq[i] = a.norm && w_q ? w_q[ch] : 1.f;
        wk[i] = a.norm && w_k ? w_k[ch] : 1.f;
    }
    for (long long first = static_cast<long long>(blockIdx.x) * a.chunk; first < a.rows;
         first += static_cast<long long>(gridDim.x) * a.chunk) {
        const int r0 = static_cast<int>(first), r1 = min(static_cast<long long>(a.rows), first + a.chunk), t0 = a.heads(r0);
        if (half) {
            __syncthreads();
            fill_turns(turns, t0, a.heads(r1 - 1), half, positions, inv_freq);
            __syncthreads();
        }
        for (int r = r0 + threadIdx.x / L; r < r1; r += kGroups) {
            const int t = a.heads(r), h = r - t * a.H;
            const bool key = h >= a.Hq;
            const long long at = key ? static_cast<long long>(h - a.Hq) * D : static_cast<long long>(h) * D;
            const T* g = key ? g_k_out + static_cast<long long>(t) * (a.H - a.Hq) * D + at
                             : g_q_out + static_cast<long long>(t) * a.Hq * D + at;
            T* to = key ? g_k + t * a.gk_stride + at : g_q + t * a.gq_stride + at;
            float u[N], x[N];
            load_group<Q>(g + ln.a, u);
            load_group<Q>(g + ln.b, u + Q);
            if (a.norm) {
                const T* p = key ? k + t * a.k_stride + at : q + t * a.q_stride + at;
                load_group<Q>(p + ln.a, x);
                load_group<Q>(p + ln.b, x + Q);
            }
            if (ln.angle >= 0) {
                float c[Q], s[Q];
                load_group<Q>(turns + (t - t0) * 2 * half + ln.angle, c);
                load_group<Q>(turns + (t - t0) * 2 * half + half + ln.angle, s);
#pragma unroll
                for (int i = 0; i < Q; ++i) s[i] = -s[i];
                rotate<Q, IL>(u, c, s);
            }
            if (a.norm) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < N; ++i) sum = fmaf(x[i], x[i], sum);
                const float inv = rsqrtf(row_sum<L>(sum) * (1.f / D) + a.eps);
                float dot = 0.f;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    x[i] *= inv;
                    const float ux = u[i] * x[i];
                    sq[i] += key ? 0.f : ux;
                    sk[i] += key ? ux : 0.f;
                    u[i] *= key ? wk[i] : wq[i];
                    dot = fmaf(u[i], x[i], dot);
                }
                dot = row_sum<L>(dot) * (1.f / D);
#pragma unroll
                for (int i = 0; i < N; ++i) u[i] = (u[i] - x[i] * dot) * inv;
            }
            store_group<Q>(to + ln.a, u);
            store_group<Q>(to + ln.b, u + Q);
        }
    }
    if (!part) return;
    __syncthreads();
    float* sums = turns;  // [kGroups][2][D]
    float* mine = sums + threadIdx.x / L * (2 * D);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int ch = channel_of<Q>(ln, i);
        mine[ch] = sq[i];
        mine[D + ch] = sk[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kRopeThreads) {
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) s += sums[g * 2 * D + i];
        part[static_cast<size_t>(blockIdx.x) * 2 * D + i] = s;
    }
}

// grad_w: the workgroups' parts, 16 channels to a workgroup, every 64th part to a
// thread, whose sums are added four at a time.
template <int D>
__global__ __launch_bounds__(1024) void rope_join_kernel(int parts, const float* __restrict__ part, float* g_w_q, float* g_w_k) {
    __shared__ float sums[64][16], fewer[16][16];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4, col = blockIdx.x * 16 + x;
    float s = 0.f;
#pragma unroll 16
    for (int p = y; p < parts; p += 64) s += part[static_cast<size_t>(p) * 2 * D + col];
    sums[y][x] = s;
    __syncthreads();
    if (y < 16) fewer[y][x] = (sums[4 * y][x] + sums[4 * y + 1][x]) + (sums[4 * y + 2][x] + sums[4 * y + 3][x]);
    __syncthreads();
    if (y) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += fewer[i][x];
    float* to = col < D ? g_w_q : g_w_k;
    if (to) to[col % D] = s;
}

constexpr int kRopeParts = 1024;  // workgroups of the backward at most

// Rows of a chunk: whole passes of the workgroup, eight where that leaves 1024
// workgroups (four to a CU), and at most 32 tokens, whose angles LDS holds.
int rope_chunk(long long rows, int H, int d, int group) {
    const int pass = kRopeThreads / (d / (2 * group));
    int n = 8;
    while (n > 1 && (rows < 1024ll * n * pass || n * pass > 32 * H)) n >>= 1;
    return n * pass < 32 * H ? n * pass : 32 * H;
}
int chunk_tokens(int chunk, int H) { return (chunk + H - 2) / H + 1; }

RopeArgs rope_args(int tokens, int Hq, int Hkv, int d, int rot, int norm, float eps, int group) {
    RopeArgs a{};
    a.H = Hq + Hkv;
    a.Hq = Hq;
    a.rows = tokens * a.H;
    a.chunk = rope_chunk(a.rows, a.H, d, group);
    a.rot = rot;
    a.norm = norm;
    a.eps = eps;
    a.heads = FastDiv(a.H);
    return a;
}

unsigned rope_parts(const RopeArgs& a) {
    const long long n = (static_cast<long long>(a.rows) + a.chunk - 1) / a.chunk;
    return static_cast<unsigned>(n < kRopeParts ? n : kRopeParts);
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_rope(int dtype, int tokens, int Hq, int Hkv, int d, int rot, int interleaved, int norm, float eps,
                            long long q_stride, long long k_stride, const void* q, const void* k, const float* w_q,
                            const float* w_k, const int* positions, const float* inv_freq, void* q_out, void* k_out,
                            hipStream_t st) {
    // 16 bytes a group; bf16 8 where that leaves the GPU with little to do (2560 rows of
    // d = 128: 3.8 us against 4.7; 327680: 36.3 against 34.7)
    const long long rows = static_cast<long long>(tokens) * (Hq + Hkv);
    const int group = dtype == GDR_DTYPE_F32 || rows < 32768 ? 4 : 8;
    attn::RopeArgs a = attn::rope_args(tokens, Hq, Hkv, d, rot, norm, eps, group);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.gq_stride = static_cast<long long>(Hq) * d;
    a.gk_stride = static_cast<long long>(Hkv) * d;
    const unsigned long long blocks = (static_cast<unsigned long long>(a.rows) + a.chunk - 1) / a.chunk;
    if (!grid_fits(blocks, attn::kRopeThreads)) return hipErrorInvalidConfiguration;
    const size_t lds = static_cast<size_t>(attn::chunk_tokens(a.chunk, a.H)) * rot * sizeof(float);
    auto go = [&](auto t, auto dd, auto g) {
        using T = decltype(t);
        constexpr int D = decltype(dd)::value, Q = decltype(g)::value;
        auto* f = interleaved ? attn::rope_kernel<T, D, true, Q> : attn::rope_kernel<T, D, false, Q>;
        hipLaunchKernelGGL(f, dim3(static_cast<unsigned>(blocks)), dim3(attn::kRopeThreads), lds, st, a,
                           static_cast<const T*>(q), static_cast<const T*>(k), w_q, w_k, positions, inv_freq,
                           static_cast<T*>(q_out), static_cast<T*>(k_out));
        return hipGetLastError();
    };
    using C4 = std::integral_constant<int, 4>;
    using C8 = std::integral_constant<int, 8>;
    using C64 = std::integral_constant<int, 64>;
    using C128 = std::integral_constant<int, 128>;
    if (dtype == GDR_DTYPE_F32) return d == 64 ? go(float(), C64(), C4()) : go(float(), C128(), C4());
    if (group == 4) return d == 64 ? go(bf16_t(), C64(), C4()) : go(bf16_t(), C128(), C4());
    return d == 64 ? go(bf16_t(), C64(), C8()) : go(bf16_t(), C128(), C8());
}

size_t attn_rope_backward_workspace_floats(int tokens, int Hq, int Hkv, int d) {
    return static_cast<size_t>(attn::rope_parts(attn::rope_args(tokens, Hq, Hkv, d, 0, 1, 0.f, attn::kBackwardGroup))) * 2 * d;
}

hipError_t launch_attn_rope_backward(int dtype, int tokens, int Hq, int Hkv, int d, int rot, int interleaved, int norm,
                                     float eps, long long q_stride, long long k_stride, long long gq_stride,
                                     long long gk_stride, const void* q, const void* k, const float* w_q, const float* w_k,
                                     const int* positions, const float* inv_freq, const void* g_q_out, const void* g_k_out,
                                     void* g_q, void* g_k, float* g_w_q, float* g_w_k, float* ws, hipStream_t st) {
    const bool weights = g_w_q || g_w_k;
    auto join = [&](unsigned parts) {
        hipLaunchKernelGGL((d == 64 ? attn::rope_join_kernel<64> : attn::rope_join_kernel<128>), dim3(2 * d / 16), dim3(1024), 0,
                           st, static_cast<int>(parts), ws, g_w_q, g_w_k);
        return hipGetLastError();
    };
    if (tokens == 0) return join(0);  // no rows: the weights' gradients are zero
    attn::RopeArgs a = attn::rope_args(tokens, Hq, Hkv, d, rot, norm, eps, attn::kBackwardGroup);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.gq_stride = gq_stride;
    a.gk_stride = gk_stride;
    const unsigned blocks = attn::rope_parts(a);
    size_t lds = static_cast<size_t>(attn::chunk_tokens(a.chunk, a.H)) * rot * sizeof(float);
    const size_t sums = weights ? static_cast<size_t>(attn::kRopeThreads) * 16 * sizeof(float) : 0;
    if (lds < sums) lds = sums;
    auto go = [&](auto t, auto f) {
        using T = decltype(t);
        hipLaunchKernelGGL(f, dim3(blocks), dim3(attn::kRopeThreads), lds, st, a, static_cast<const T*>(q),
                           static_cast<const T*>(k), w_q, w_k, positions, inv_freq, static_cast<const T*>(g_q_out),
                           static_cast<const T*>(g_k_out), static_cast<T*>(g_q), static_cast<T*>(g_k), weights ? ws : nullptr);
        return hipGetLastError();
    };
    hipError_t e;
    if (dtype == GDR_DTYPE_F32)
        e = d == 64 ? go(float(), interleaved ? attn::rope_backward_kernel<float, 64, true> : attn::rope_backward_kernel<float, 64, false>)
                    : go(float(), interleaved ? attn::rope_backward_kernel<float, 128, true> : attn::rope_backward_kernel<float, 128, false>);
    else
        e = d == 64 ? go(bf16_t(), interleaved ? attn::rope_backward_kernel<bf16_t, 64, true> : attn::rope_backward_kernel<bf16_t, 64, false>)
                    : go(bf16_t(), interleaved ? attn::rope_backward_kernel<bf16_t, 128, true> : attn::rope_backward_kernel<bf16_t, 128, false>);
    return e != hipSuccess || !weights ? e : join(blocks);
}

}  // namespace gdr
