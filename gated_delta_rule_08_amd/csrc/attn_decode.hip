// Attention over a paged key-value cache: the decode step (one new token per
// sequence, appended to its page and attended from) and the append of whole
// prompts.
//
// Pages are [page, key head, slot, channel], so a head's keys of one page are
// one contiguous block.  The step reads every visible key and value once and
// does 4 d flops per query head and key with them: HBM-bound for any group a
// model uses.  It is therefore built for bytes in flight: each wave streams
// its own 32 keys per step, K straight into operand registers, V through
// registers into a wave-private LDS tile (the transposing reads supply the
// second product's operand), the next step's loads issued as soon as the
// registers are free; no barrier until the end.  The group's query heads are
// the 16 columns of S^T = K Q^T, so a key read serves every head of its group.
//
// The visible keys of a sequence are a list (the sinks, then the window) cut
// into equal parts, one workgroup each, where B x Hkv alone would not fill the
// GPU; a second kernel joins the parts' (m, l, O) in order.
#include "attn_common.h"

namespace gdr {
namespace attn {
namespace {

constexpr int kWaves = 4;
constexpr int kStep = 32;                // keys of a wave's step
constexpr int kGrain = kStep * kWaves;   // keys of a workgroup's step
constexpr int kMaxSplits = 64;

struct DecodeArgs {
    int B, Hq, Hkv, G, head_tiles;
    int page_shift, num_pages, max_pages;
    int window, sinks;
    float scale;
    int splits;
};

// What one sequence's step covers, from its device data alone (the same in
// every workgroup and in the join).
struct Span {
    int pos;     // position of the new token; -1: the sequence is skipped
    int w_lo;    // first key of the window
    int sinks;   // keys before it that stay visible
    int count;   // visible keys
    int chunk;   // keys of one part
    int parts;   // parts that hold keys
};

__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b, const int* __restrict__ table,
                                        const int* __restrict__ lengths) {
    Span s;
    const int p = lengths[b];
    s.pos = -1;
    if (p < 0 || (p >> a.page_shift) >= a.max_pages) return s;
    const int page = table[static_cast<size_t>(b) * a.max_pages + (p >> a.page_shift)];
    if (page < 0 || page >= a.num_pages) return s;
    s.pos = p;
    s.w_lo = a.window ? max(0, p - a.window + 1) : 0;
    s.sinks = min(a.sinks, s.w_lo);
    s.count = s.sinks + (p - s.w_lo) + 1;
    const int even = (s.count - 1) / a.splits + 1;
    s.chunk = ((even - 1) / kGrain + 1) * kGrain;
    s.parts = (s.count - 1) / s.chunk + 1;
    return s;
}

template <typename T, int D> struct DecodeCfg {
    static constexpr int kTile = kStep * D * static_cast<int>(sizeof(T));  // a wave's V tile
    static constexpr int kPitch = D + 4;                                   // floats of a joined row
    static constexpr int kJoin = kWaves * 16 * (kPitch + 2) * 4;
    static constexpr int kLds = kWaves * kTile > kJoin ? kWaves * kTile : kJoin;
};

// Column fragment of a 32-row tile for 16x16x32 products: lane (c = lane % 16,
// h = lane / 16) gets column 16 t + c of rows {4h..4h+3, 16+4h..16+4h+3}, the
// rows its registers of two stacked accumulator tiles hold.
template <typename T, int D> struct ColRead16;
template <int D> struct ColRead16<bf16_t, D> {
    using L = Tile<bf16_t, D>;
    __device__ __forceinline__ static int base(int lane) {
        const int h = lane >> 4, lr = lane & 15;
        return (L::at(4 * h + (lr >> 2)) ^ (((lr >> 1) & 1) << 4)) + 8 * (lr & 1);
    }
    __device__ __forceinline__ static bf16x8v get(const unsigned char* lds, int base, int t) {
        typedef __attribute__((address_space(3))) s16x4v lds_s16x4;
        const unsigned char* p = lds + (base ^ (t << 5));
        const s16x4v a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
        const s16x4v b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * L::kRow));
        return __builtin_shufflevector(__builtin_bit_cast(bf16x4v, a), __builtin_bit_cast(bf16x4v, b), 0, 1, 2, 3,
                                       4, 5, 6, 7);
    }
};
template <int D> struct ColRead16<float, D> {
    using L = Tile<float, D>;
    __device__ __forceinline__ static int base(int lane) {
        const int h = lane >> 4, c = lane & 15;
        return (L::at(4 * h) ^ ((c >> 2) << 4)) + 4 * (c & 3);
    }
    __device__ __forceinline__ static f32x8 get(const unsigned char* lds, int base, int t) {
        f32x8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r[i] = *reinterpret_cast<const float*>(lds + (base ^ (t << 6) ^ ((i & 3) << 6)) +
                                                   (16 * (i >> 2) + (i & 3)) * L::kRow);
        return r;
    }
};

// 16-byte loads of the pages: read once, so they need not stay in the caches.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4 stream16(const void* p) {
    return __builtin_nontemporal_load(static_cast<const u32x4*>(p));
}
__device__ __forceinline__ bf16x8v stream8(const bf16_t* p) { return __builtin_bit_cast(bf16x8v, stream16(p)); }
__device__ __forceinline__ f32x8 stream8(const float* p) {
    const f32x4 a = __builtin_bit_cast(f32x4, stream16(p)), b = __builtin_bit_cast(f32x4, stream16(p + 4));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <typename T, int D>
__global__ __launch_bounds__(64 * kWaves) void decode_kernel(
    DecodeArgs a, const T* __restrict__ q, const T* __restrict__ knew, const T* __restrict__ vnew, T* k_pages,
    T* v_pages, const int* __restrict__ table, const int* __restrict__ lengths, T* __restrict__ o,
    float* __restrict__ part_o, float* __restrict__ part_ml) {
    using C = DecodeCfg<T, D>;
    using L = Tile<T, D>;
    constexpr int KS = D / 32, DT = D / 16;
    constexpr int kPer = 1024 / L::kRow, kVLoads = kStep / kPer;  // rows of one V load instruction
    constexpr int kNone = -1, kNew = -2;
    extern __shared__ unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c16 = lane & 15, h4 = lane >> 4;

    int id = blockIdx.x;
    const int split = id % a.splits;
    id /= a.splits;
    const int ht = id % a.head_tiles;
    id /= a.head_tiles;
    const int hk = id % a.Hkv, b = id / a.Hkv;
    const Span sp = span_of(a, b, table, lengths);
    if (sp.pos < 0 || split >= sp.parts) return;

    const int slot_mask = (1 << a.page_shift) - 1;
    const int* trow = table + static_cast<size_t>(b) * a.max_pages;
    const size_t new_row = static_cast<size_t>(b) * a.Hkv + hk;
    if (split == 0 && ht == 0 && threadIdx.x < 2 * L::kUnits) {  // the new token into its page
        const bool val = threadIdx.x >= L::kUnits;
        const int u = threadIdx.x % L::kUnits;
        const int page = trow[sp.pos >> a.page_shift];
        const size_t row = ((static_cast<size_t>(page) * a.Hkv + hk) << a.page_shift) + (sp.pos & slot_mask);
        reinterpret_cast<uint4*>((val ? v_pages : k_pages) + row * D)[u] =
            reinterpret_cast<const uint4*>((val ? vnew : knew) + new_row * D)[u];
    }

    const int head0 = hk * a.G + ht * 16, nheads = min(16, a.G - ht * 16);
    frag_t<T> qf[KS];
    {
        const bool neg = a.scale < 0.f;
        const T* qp = q + (static_cast<size_t>(b) * a.Hq + head0 + min(c16, nheads - 1)) * D + 8 * h4;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            qf[s] = load8(qp + 32 * s);
            if (neg) qf[s] = -qf[s];
        }
    }
    // a scale of 0 as one that no score survives: c -inf of a hidden key stays -inf
    const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-37f);

    // Cache row of list entry i: the new token's own row is taken from the
    // call's k and v (its page is being written); entries past the end and
    // keys of an invalid page are hidden.
    const int first = split * sp.chunk, last = min(sp.count, first + sp.chunk);
    auto row_of = [&](int i) {
        if (i >= last) return kNone;
        const int key = i < sp.sinks ? i : i - sp.sinks + sp.w_lo;
        if (key == sp.pos) return kNew;
        const int page = trow[key >> a.page_shift];
        if (page < 0 || page >= a.num_pages) return kNone;
        return ((page * a.Hkv + hk) << a.page_shift) + (key & slot_mask);
    };
    frag_t<T> kf[2][KS];
    u32x4 vr[kVLoads];
    auto fetch = [&](int rid) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = __shfl(rid, 16 * u + c16);
            const T* p = (r == kNew ? knew + new_row * D : k_pages + static_cast<size_t>(r) * D) + 8 * h4;
#pragma unroll
            for (int s = 0; s < KS; ++s) kf[u][s] = r == kNone ? zero_frag<T>() : stream8(p + 32 * s);
        }
#pragma unroll
        for (int j = 0; j < kVLoads; ++j) {
            const int r = __shfl(rid, kPer * j + lane / L::kUnits);
            const T* p = r == kNew ? vnew + new_row * D : v_pages + static_cast<size_t>(r) * D;
            vr[j] = r == kNone ? u32x4{0u, 0u, 0u, 0u} : stream16(p + (lane % L::kUnits) * (16 / sizeof(T)));
        }
    };

    unsigned char* tile = smem + wave * C::kTile;
    const int vb = ColRead16<T, D>::base(lane);
    f32x4 acc[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;

    int at = first + wave * kStep;
    int rid = row_of(at + (lane & 31));
    if (at < last) fetch(rid);
#pragma unroll 1
    for (; at < last; at += kGrain) {
        const uint32_t shown = static_cast<uint32_t>(__ballot(rid != kNone));
        const int next = row_of(at + kGrain + (lane & 31));
        f32x4 s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            s[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < KS; ++e) s[u] = mma16(kf[u][e], qf[e], s[u]);
        }
#pragma unroll
        for (int j = 0; j < kVLoads; ++j)
            *reinterpret_cast<u32x4*>(tile + (L::at(kPer * j + lane / L::kUnits) ^ ((lane % L::kUnits) << 4))) = vr[j];
        rid = next;
        if (at + kGrain < last) fetch(rid);

        if (shown != 0xffffffffu) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (!((shown >> (16 * u + 4 * h4 + r)) & 1)) s[u][r] = -INFINITY;
        }
        float mx = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                         fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(m, fmaxf(mx, __shfl_xor(mx, 32)));
        const float mc = mx == -INFINITY ? 0.f : mx * c;
        if (__any(mx > m)) {
            const float alpha = m == -INFINITY ? 0.f : ex2(m * c - mc);
            l *= alpha;
#pragma unroll
            for (int t = 0; t < DT; ++t) acc[t] *= alpha;
            m = mx;
        }
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = ex2(fmaf(s[i >> 2][i & 3], c, -mc));
            l += w[i];
        }
        const frag_t<T> pf = pack8<T>(w);
#pragma unroll
        for (int t = 0; t < DT; ++t) acc[t] = mma16(ColRead16<T, D>::get(tile, vb, t), pf, acc[t]);
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // the four waves' parts, joined in LDS in wave order
    __syncthreads();
    float* jo = reinterpret_cast<float*>(smem);
    float* jm = jo + kWaves * 16 * C::kPitch;
    {
        float* dst = jo + (wave * 16 + c16) * C::kPitch + 4 * h4;
#pragma unroll
        for (int t = 0; t < DT; ++t) *reinterpret_cast<f32x4*>(dst + 16 * t) = acc[t];
        if (h4 == 0) {
            jm[(wave * 16 + c16) * 2] = m;
            jm[(wave * 16 + c16) * 2 + 1] = l;
        }
    }
    __syncthreads();
    const int head = threadIdx.x >> 4;
    if (head >= nheads) return;
    float mw[kWaves], M = -INFINITY;
#pragma unroll
    for (int x = 0; x < kWaves; ++x) {
        mw[x] = jm[(x * 16 + head) * 2];
        M = fmaxf(M, mw[x]);
    }
    float lt = 0.f;
#pragma unroll
    for (int x = 0; x < kWaves; ++x) {
        mw[x] = mw[x] == -INFINITY ? 0.f : ex2((mw[x] - M) * c);
        lt = fmaf(jm[(x * 16 + head) * 2 + 1], mw[x], lt);
    }
    const size_t orow = static_cast<size_t>(b) * a.Hq + head0 + head;
    const bool whole = sp.parts == 1;
    const float inv = whole ? (lt == 0.f ? 0.f : 1.f / lt) : 1.f;
    const size_t prow = orow * a.splits + split;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
        const int d = 64 * e + 4 * (threadIdx.x & 15);
        f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < kWaves; ++x)
            if (mw[x] != 0.f) sum += *reinterpret_cast<const f32x4*>(jo + (x * 16 + head) * C::kPitch + d) * mw[x];
        if (whole)
            store4<T>(o + orow * D + d, sum[0] * inv, sum[1] * inv, sum[2] * inv, sum[3] * inv);
        else
            *reinterpret_cast<f32x4*>(part_o + prow * D + d) = sum;
    }
    if (!whole && (threadIdx.x & 15) == 0) {
        part_ml[prow * 2] = M == -INFINITY ? M : M * c;
        part_ml[prow * 2 + 1] = lt;
    }
}

// Joins a sequence's parts, one workgroup per query head: every wave forms the
// parts' weights 2^(m_s - max m) (lane s holds part s) and adds a quarter of
// the parts, the channels over its lanes; the four sums are added in order.
template <typename T, int D>
__global__ __launch_bounds__(256) void join_kernel(DecodeArgs a, const int* __restrict__ table,
                                                   const int* __restrict__ lengths,
                                                   const float* __restrict__ part_o,
                                                   const float* __restrict__ part_ml, T* __restrict__ o) {
    constexpr int N = D / 64, W = 4;
    __shared__ float sums[W - 1][D];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const size_t row = blockIdx.x;
    const Span sp = span_of(a, static_cast<int>(row / a.Hq), table, lengths);
    if (sp.pos < 0 || sp.parts == 1) return;
    const size_t prow = row * a.splits;
    float m = -INFINITY, l = 0.f;
    if (lane < sp.parts) {
        m = part_ml[(prow + lane) * 2];
        l = part_ml[(prow + lane) * 2 + 1];
    }
    const float* p = part_o + prow * D + N * lane;
    float x[kMaxSplits / W][N];
#pragma unroll
    for (int i = 0; i < kMaxSplits / W; ++i)  // all loads before the first use
#pragma unroll
        for (int e = 0; e < N; ++e)
            x[i][e] = W * i + wave < sp.parts ? p[static_cast<size_t>(W * i + wave) * D + e] : 0.f;
    float M = m;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) M = fmaxf(M, __shfl_xor(M, s));
    const float w = m == -INFINITY ? 0.f : ex2(m - M);
    float total = l * w;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) total += __shfl_xor(total, s);
    float acc[N] = {};
#pragma unroll
    for (int i = 0; i < kMaxSplits / W; ++i) {
        const float ws = __shfl(w, W * i + wave);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = fmaf(ws, x[i][e], acc[e]);
    }
    if (wave > 0) {
#pragma unroll
        for (int e = 0; e < N; ++e) sums[wave - 1][N * lane + e] = acc[e];
    }
    __syncthreads();
    if (wave > 0) return;
    const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
    for (int e = 0; e < N; ++e) {
#pragma unroll
        for (int s = 0; s < W - 1; ++s) acc[e] += sums[s][N * lane + e];
        Elem<T>::store(o + row * D + N * lane + e, acc[e] * inv);
    }
}

template <typename T, int D>
hipError_t launch_decode_t(const DecodeArgs& a, const void* q, const void* k, const void* v, void* k_pages,
                           void* v_pages, const int* table, const int* lengths, void* o, float* ws, hipStream_t st) {
    using C = DecodeCfg<T, D>;
    const unsigned long long blocks = static_cast<unsigned long long>(a.B) * a.Hkv * a.head_tiles * a.splits;
    const unsigned long long rows = static_cast<unsigned long long>(a.B) * a.Hq;
    if (!grid_fits(blocks, 64 * kWaves) || !grid_fits(rows, 256)) return hipErrorInvalidConfiguration;
    auto* f = decode_kernel<T, D>;
    if (C::kLds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(f),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, C::kLds);
        if (e != hipSuccess) return e;
    }
    float* part_o = ws;
    float* part_ml = ws ? ws + rows * a.splits * D : nullptr;
    hipLaunchKernelGGL(f, dim3(static_cast<unsigned>(blocks)), dim3(64 * kWaves), C::kLds, st, a,
                       static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v),
                       static_cast<T*>(k_pages), static_cast<T*>(v_pages), table, lengths, static_cast<T*>(o),
                       part_o, part_ml);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    hipLaunchKernelGGL((join_kernel<T, D>), dim3(static_cast<unsigned>(rows)), dim3(256), 0, st, a, table,
                       lengths, part_o, part_ml, static_cast<T*>(o));
    return hipGetLastError();
}

// Append: one 16-byte unit of one key head's new row (K and V) per thread.
__global__ __launch_bounds__(256) void append_kernel(int N, int total, int Hkv, int units, int page_shift,
                                                     int num_pages, int max_pages, const uint4* __restrict__ k,
                                                     const uint4* __restrict__ v, const int* __restrict__ cu,
                                                     const int* __restrict__ lengths, uint4* __restrict__ k_pages,
                                                     uint4* __restrict__ v_pages, const int* __restrict__ table) {
    const int per = Hkv * units;  // units of one token
    const size_t n = static_cast<size_t>(total) * per;
    for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
         i += static_cast<size_t>(gridDim.x) * 256) {
        const int t = static_cast<int>(i / per), x = static_cast<int>(i - static_cast<size_t>(t) * per);
        int lo = 0, hi = N;  // the last sequence that starts at or before t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        const int begin = cu[lo], len = lengths[lo];
        if (begin < 0 || t < begin || t >= cu[lo + 1] || len < 0) continue;
        const long long pos = static_cast<long long>(len) + (t - begin);
        if ((pos >> page_shift) >= max_pages) continue;
        const int page = table[static_cast<size_t>(lo) * max_pages + (pos >> page_shift)];
        if (page < 0 || page >= num_pages) continue;
        const int hk = x / units, u = x - hk * units;
        const size_t row = ((static_cast<size_t>(page) * Hkv + hk) << page_shift) +
                           static_cast<size_t>(pos & ((1 << page_shift) - 1));
        k_pages[row * units + u] = k[i];
        v_pages[row * units + u] = v[i];
    }
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

// Parts per sequence and key head: enough workgroups for several rounds of
// what fits the GPU at a time, no part below 256 keys of the longest sequence
// the page table can hold; up to 512 keys the second launch costs more than
// the parts save.
int decode_splits(int B, int Hkv, int G, int page_size, int max_pages, int window, int sinks) {
    long long keys = static_cast<long long>(max_pages) * page_size;
    if (window && keys > static_cast<long long>(window) + sinks) keys = static_cast<long long>(window) + sinks;
    const long long units = static_cast<long long>(B) * Hkv * ((G + 15) / 16);
    if (units == 0 || keys <= 512) return 1;
    long long s = 2048 / units;
    if (s > (keys + 255) / 256) s = (keys + 255) / 256;
    return static_cast<int>(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
}

}  // namespace
}  // namespace attn

size_t attn_decode_workspace_floats(int B, int Hq, int Hkv, int d, int page_size, int max_pages, int window,
                                    int sinks) {
    const int s = attn::decode_splits(B, Hkv, Hq / Hkv, page_size, max_pages, window, sinks);
    return s == 1 ? 0 : static_cast<size_t>(B) * Hq * s * (d + 2);
}

hipError_t launch_attn_decode(int dtype, int B, int Hq, int Hkv, int d, int page_size, int num_pages, int max_pages,
                              int window, int sinks, float scale, const void* q, const void* k, const void* v,
                              void* k_pages, void* v_pages, const int* table, const int* lengths, void* o, float* ws,
                              hipStream_t st) {
    attn::DecodeArgs a{};
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.head_tiles = (a.G + 15) / 16;
    a.page_shift = attn::log2_of(page_size);
    a.num_pages = num_pages;
    a.max_pages = max_pages;
    a.window = window;
    a.sinks = sinks;
    a.scale = scale;
    a.splits = attn::decode_splits(B, Hkv, a.G, page_size, max_pages, window, sinks);
    auto* f = dtype == GDR_DTYPE_F32 ? (d == 64 ? attn::launch_decode_t<float, 64> : attn::launch_decode_t<float, 128>)
                                     : (d == 64 ? attn::launch_decode_t<bf16_t, 64> : attn::launch_decode_t<bf16_t, 128>);
    return f(a, q, k, v, k_pages, v_pages, table, lengths, o, ws, st);
}

hipError_t launch_attn_append(int dtype, int N, int total, int Hkv, int d, int page_size, int num_pages,
                              int max_pages, const void* k, const void* v, const int* cu, const int* lengths,
                              void* k_pages, void* v_pages, const int* table, hipStream_t st) {
    const int units = d * (dtype == GDR_DTYPE_F32 ? 4 : 2) / 16;
    const unsigned long long n = static_cast<unsigned long long>(total) * Hkv * units;
    const unsigned long long want = (n + 255) / 256;
    const unsigned blocks = static_cast<unsigned>(want < 16384 ? want : 16384);
    hipLaunchKernelGGL(attn::append_kernel, dim3(blocks), dim3(256), 0, st, N, total, Hkv, units,
                       attn::log2_of(page_size), num_pages, max_pages, static_cast<const uint4*>(k),
                       static_cast<const uint4*>(v), cu, lengths, static_cast<uint4*>(k_pages),
                       static_cast<uint4*>(v_pages), table);
    return hipGetLastError();
}

}  // namespace gdr
