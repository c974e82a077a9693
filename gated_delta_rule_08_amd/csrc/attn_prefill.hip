// Windowed attention of a prompt: Tq queries, the last Tq of Tk positions,
// grouped query heads, full causal or sliding window with sink tokens.
//
//   s_ij = scale q_i . k_j,   o_i = sum_j p_ij v_j / l_i,   p_ij = 2^(c s_ij - c m_i),
//
// one pass over the visible keys with the running maximum m and sum l of the
// softmax (fp32; c = scale log2 e, the maximum taken before scaling).
//
// The query heads of one key head are packed into the rows of a tile: row =
// query * G + head of the group.  A workgroup's rows then span few positions
// (few keys outside the mask) and share every key and value tile.  A wave
// holds 32 rows and forms S^T = K Q^T with 32x32 products: a lane owns one
// row (column of S^T) and 16 keys of each tile, so the softmax is in-lane
// apart from one exchange with the lane 32 away, its statistics are one
// register each, and the exponentials are the operand of O^T += V^T P^T as
// they stand (the contracted order is that of the accumulator registers, see
// ColRead).  O stays in registers.
//
// Bound by the matrix cores and the softmax's vector work together: full causal
// T=8192, 32 query on 8 key heads, d=128: 535 us, 1.03 PFLOP/s, matrix cores 51%
// and vector ALUs 48% busy, no LDS bank conflicts; two workgroups per CU (64 KB of
// LDS, 174 registers), whose waves fill each other's gaps.  Eight waves per
// workgroup: 538 us there and 173 against 186 with 32 key heads (T=4096), but 967
// against 951 under a window of 4096 (T=16384) and 336 against 305 at d=64.
#include "attn_common.h"

namespace gdr {
namespace attn {
namespace {

constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;  // query rows of a workgroup

struct PrefillArgs {
    int B, Tq, Tk, Hq, Hkv;  // packed: B sequences, Tq = longest, Tk unused
    FastDiv G;
    int window, sinks;
    float scale;
    int tiles;  // row tiles of a (sequence, key head)
    const int *cu_q, *cu_k;
    int total_q, total_k;
};

template <typename T, int D, bool SPLIT> struct PrefillCfg {
    static constexpr int NS = sizeof(T) == 2 && !SPLIT ? 2 : 1;  // 32-key tiles of a wave's step
    static constexpr int BN = 32 * NS * (SPLIT ? kWaves : 1);    // keys of a workgroup's step
    static constexpr int kTileBytes = BN * D * static_cast<int>(sizeof(T));
    static constexpr int kBufs = 4 * kTileBytes <= 128 * 1024 ? 2 : 1;
    static constexpr int kLds = 2 * kBufs * kTileBytes;  // K and V
};

// The rows of one wave once more with hidden keys left out of every sum: what a
// wave does when a non-finite value has met its sums.  Operands straight from
// global memory, 32 keys and 32 channels at a time, no other wave involved;
// put(t, sums, m, l) takes channels 32 t .. 32 t + 31.
template <typename T, int D, typename P>
__device__ __forceinline__ void seen_rows(Mask mask, int pos, int wp0, int wp1, int Tk, float c, bool neg, const T* q,
                                          const T* k, const T* v, size_t stride, int lane, P put) {
    const int h2 = lane >> 5;
    const KeyList keys(mask.window, mask.sinks, wp0, wp1);
#pragma unroll 1
    for (int t = 0; t < D / 32; ++t) {
        f32x16 acc = zero16();
        float m = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int x0 = 0; x0 < keys.count; x0 += 32) {
            auto row = [&](int r) { return static_cast<size_t>(min(keys.key(x0 + r), Tk - 1)) * stride; };
            const T *kr = k + row(lane & 31) + 8 * h2, *qr = q + 8 * h2;
            f32x16 s = zero16();
#pragma unroll 1
            for (int e = 0; e < D / 16; ++e) s = mma32(load8(kr + 16 * e), neg ? -load8(qr + 16 * e) : load8(qr + 16 * e), s);
            uint32_t seen = 0;
            float mx = m;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (mask.sees(pos, keys.key(x0 + row32(r, h2)))) {
                    seen |= 1u << r;
                    mx = fmaxf(mx, s[r]);
                }
            mx = fmaxf(mx, other_half(mx));
            const float mc = mx == -INFINITY ? 0.f : mx * c, alpha = m == -INFINITY ? 0.f : ex2(m * c - mc);
            m = mx;
            l *= alpha;
            acc *= alpha;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[r] = (seen >> r) & 1 ? ex2(fmaf(s[r], c, -mc)) : 0.f;
                l += s[r];
            }
            mma32_seen<T>(acc, [&](int r) { return v + row(r) + 32 * t; }, s, seen, lane);
        }
        put(t, acc, m, l + other_half(l));
    }
}

// 32 rows per wave, or with SPLIT 32 rows per workgroup, each wave taking a
// quarter of the keys and the four joined at the end.
template <typename T, int D, bool SPLIT>
__global__ __launch_bounds__(64 * kWaves, (PrefillCfg<T, D, SPLIT>::kBufs)) void prefill_kernel(PrefillArgs a, const T* __restrict__ q,
                                                                 const T* __restrict__ k,
                                                                 const T* __restrict__ v, T* __restrict__ o,
                                                                 float* __restrict__ lse) {
    using C = PrefillCfg<T, D, SPLIT>;
    constexpr int BN = C::BN, NS = C::NS, KS = D / 16, DT = D / 32, kGroup = SPLIT ? 32 : kRows;
    extern __shared__ unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h2 = lane >> 5;
    int head, tile;
    place(blockIdx.x, a.B * a.Hkv, a.tiles, head, tile);
    tile = a.tiles - 1 - tile;  // the last rows see the most keys
    const int b = head / a.Hkv, hk = head - b * a.Hkv;
    int Tq = a.Tq, Tk = a.Tk;
    size_t q0 = static_cast<size_t>(b) * a.Tq, k0 = static_cast<size_t>(b) * a.Tk;
    if (a.cu_q) {
        const int qa = a.cu_q[b], qe = a.cu_q[b + 1], ka = a.cu_k[b], ke = a.cu_k[b + 1];
        if (qa < 0 || qe < qa || qe > a.total_q || qe - qa > a.Tq || ka < 0 || ke < ka || ke > a.total_k) return;
        Tq = qe - qa;
        Tk = ke - ka;
        q0 = qa;
        k0 = ka;
    }
    const FastDiv G = a.G;
    const int nrows = Tq * G.d, row0 = tile * kGroup;
    if (row0 >= nrows) return;
    const int off = Tk - Tq;
    const Mask mask{a.window, a.sinks};

    // this wave's and this lane's rows (a wave or lane past the end repeats
    // the last row and stores nothing)
    const int wrow = row0 + (SPLIT ? 0 : 32 * wave);
    const int wr0 = min(wrow, nrows - 1), wr1 = min(wrow + 31, nrows - 1);
    const bool live = wrow + (lane & 31) < nrows, wave_live = wrow < nrows;
    const int row = min(wrow + (lane & 31), nrows - 1);
    const int qi = G(row), g = row - qi * G.d, pos = qi + off;
    const int wp0 = __builtin_amdgcn_readfirstlane(G(wr0) + off);
    const int wp1 = __builtin_amdgcn_readfirstlane(G(wr1) + off);
    const size_t qrow = (q0 + qi) * a.Hq + static_cast<size_t>(hk) * G.d + g;

    const KeyList keys(a.window, a.sinks, G(row0) + off, G(min(row0 + kGroup - 1, nrows - 1)) + off);
    const int n = (keys.count + BN - 1) / BN;

    const size_t kstride = static_cast<size_t>(a.Hkv) * D;
    const T* kbase = k + (k0 * a.Hkv + hk) * D;
    const T* vbase = v + (k0 * a.Hkv + hk) * D;
    const int sub = SPLIT ? 32 * wave : 0;  // this wave's keys of a step
    const TileRange range = TileRange::of<BN, 32 * NS>(keys, a.window, Tk, sub, wp0, wp1);
    const int end = wave_live ? range.end : 0;
    const TileCopy<T, D, BN, kWaves> copy(wave, lane, [&](int r) { return r * static_cast<int>(kstride * sizeof(T)); });
    const T *kp = kbase + keys.jump * kstride, *vp = vbase + keys.jump * kstride;  // the next tile's first rows
    auto fetch = [&](int i) {  // tiles in turn
        const uint32_t buf = lds_addr(smem) + (i & (C::kBufs - 1)) * 2 * C::kTileBytes;
        if (i >= range.full_lo && i < range.full_hi) {
            copy.run(buf, kp);
            copy.run(buf + C::kTileBytes, vp);
        } else {
            auto row = [&](int r) { return static_cast<size_t>(min(keys.key(i * BN + r), Tk - 1)) * kstride; };
            copy.gather(buf, [&](int r) { return kbase + row(r); });
            copy.gather(buf + C::kTileBytes, [&](int r) { return vbase + row(r); });
        }
        kp += BN * kstride;
        vp += BN * kstride;
    };
    if (C::kBufs == 2 && n > 0) fetch(0);

    // Q^T as the B operand.  A negative scale flips the sign of q (exact), so
    // that the largest raw score is the largest scaled one.
    frag_t<T> qf[KS];
    {
        const T* qp = q + qrow * D + 8 * h2;
        const bool neg = a.scale < 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            qf[s] = load8(qp + 16 * s);
            if (neg) qf[s] = -qf[s];
        }
    }
    // a scale of 0 as one that no score survives: c -inf of a hidden key stays -inf
    const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-37f);

    f32x16 acc[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t) acc[t] = zero16();
    float m = -INFINITY, l = 0.f;

    const int kb0 = RowRead<T, D>::base(lane & 31, h2) + sub * Tile<T, D>::kRow;
    const int vb0 = ColRead<T, D>::base(lane) + sub * Tile<T, D>::kRow + C::kTileBytes;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        if (C::kBufs == 1) {
            if (i > 0) tile_barrier();
            fetch(i);
        }
        tile_barrier();
        if (C::kBufs == 2 && i + 1 < n) fetch(i + 1);
        const int buf = (i & (C::kBufs - 1)) * 2 * C::kTileBytes, kb = kb0 + buf, vb = vb0 + buf;
        if (i >= end) continue;

        // The other wave of the SIMD is in another phase: a wave in its products
        // goes first, the exponentials of the other fill the gaps.  With d = 128
        // only in the second product (T=8192, 32/8 heads: 535 us, both products 562,
        // neither 558), with d = 64 in both (305 us, second 314, neither 316; 8/8 heads
        // 121 / 119 / 128).
        if (D == 64) __builtin_amdgcn_s_setprio(1);
        f32x16 s[NS];
#pragma unroll
        for (int u = 0; u < NS; ++u) {
            s[u] = zero16();
#pragma unroll
            for (int e = 0; e < KS; ++e)
                s[u] = mma32(RowRead<T, D>::get(smem, kb, e, 32 * u * Tile<T, D>::kRow), qf[e], s[u]);
        }
        if (D == 64) __builtin_amdgcn_s_setprio(0);
        if (i < range.whole_lo || i >= range.whole_hi) {
            const int x0 = i * BN + sub;
#pragma unroll
            for (int u = 0; u < NS; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (!mask.sees(pos, keys.key(x0 + 32 * u + row32(r, h2)))) s[u][r] = -INFINITY;
        }
        float mx = s[0][0];
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[u][r]);
        mx = fmaxf(m, fmaxf(mx, other_half(mx)));
        // The sums are rescaled only where a row's maximum has grown by more than
        // a factor 2^8 since: weights then reach 2^8, which costs no precision
        // (every rounding is relative), and most tiles leave the sums alone.
        if (__any((mx - m) * c > 8.f)) {
            const float alpha = m == -INFINITY ? 0.f : ex2((m - mx) * c);
            l *= alpha;
#pragma unroll
            for (int t = 0; t < DT; ++t) acc[t] *= alpha;
            m = mx;
        }
        const float mc = m == -INFINITY ? 0.f : m * c;  // a row that has seen no key: weights 0
        frag_t<T> pf[2 * NS];
        float ls = 0.f;
#pragma unroll
        for (int u = 0; u < NS; ++u) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[u][r] = ex2(fmaf(s[u][r], c, -mc));
                ls += s[u][r];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) pf[2 * u + x] = pack_regs<T>(s[u], x);
        }
        l += ls;
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int x = 0; x < 2 * NS; ++x) acc[t] = mma32(ColRead<T, D>::get(smem, vb, t, x), pf[x], acc[t]);
        __builtin_amdgcn_s_setprio(0);
    }

    l += other_half(l);
    if constexpr (SPLIT) {  // the waves' parts, joined by the first in wave order
        constexpr int kBox = (DT * 16 + 2) * 64;  // floats of one wave
        static_assert(C::kLds >= (kWaves - 1) * kBox * 4, "LDS holds the other waves' parts");
        float* box = reinterpret_cast<float*>(smem) + lane;
        tile_barrier();
        if (wave > 0) {
            float* mine = box + (wave - 1) * kBox;
            mine[0] = m;
            mine[64] = l;
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) mine[(t * 16 + r + 2) * 64] = acc[t][r];
        }
        tile_barrier();
        if (wave > 0) return;
#pragma unroll 1
        for (int w = 0; w < kWaves - 1; ++w) {
            const float* its = box + w * kBox;
            const float m1 = its[0], mx = fmaxf(m, m1), mc = mx == -INFINITY ? 0.f : mx * c;
            const float a0 = m == -INFINITY ? 0.f : ex2(m * c - mc), a1 = m1 == -INFINITY ? 0.f : ex2(m1 * c - mc);
            m = mx;
            l = l * a0 + its[64] * a1;
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[t][r] = fmaf(its[(t * 16 + r + 2) * 64], a1, acc[t][r] * a0);
        }
    }

    // A hidden key has weight 0, but 0 times an infinity or NaN in its value
    // row is NaN: a wave whose sums hold a NaN forms its rows again from the
    // visible keys alone.
    bool bad = l != l;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) bad |= acc[t][r] != acc[t][r];
    auto put = [&](int t, const f32x16& x, float m, float l) {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // no visible key: zeros
        if (!live) return;
#pragma unroll
        for (int r = 0; r < 16; r += 4)
            store4<T>(o + qrow * D + 32 * t + row32(r, h2), x[r] * inv, x[r + 1] * inv, x[r + 2] * inv, x[r + 3] * inv);
        if (t == 0 && lse && h2 == 0) lse[qrow] = l == 0.f ? -INFINITY : (m * c + lg2(l)) * kLn2;
    };
#pragma unroll
    for (int t = 0; t < DT; ++t) put(t, acc[t], m, l);
    if (__builtin_expect(__ballot(bad && live) != 0, 0))
        seen_rows<T, D>(mask, pos, wp0, wp1, Tk, c, a.scale < 0.f, q + qrow * D, kbase, vbase, kstride, lane, put);
}

template <typename T, int D, bool SPLIT>
hipError_t launch_tiles(const PrefillArgs& a, const void* q, const void* k, const void* v, void* o, float* lse,
                        hipStream_t st) {
    using C = PrefillCfg<T, D, SPLIT>;
    const unsigned long long blocks = static_cast<unsigned long long>(a.B) * a.Hkv * a.tiles;
    if (!grid_fits(blocks, 64 * kWaves)) return hipErrorInvalidConfiguration;
    auto* f = prefill_kernel<T, D, SPLIT>;
    if (C::kLds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(f),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, C::kLds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(f, dim3(static_cast<unsigned>(blocks)), dim3(64 * kWaves), C::kLds, st, a,
                       static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v),
                       static_cast<T*>(o), lse);
    return hipGetLastError();
}

// Few 128-row workgroups: 32-row workgroups instead, each wave a quarter of the
// keys, which costs four times the copies to LDS.  bf16 below 192 (8 heads:
// T=1024 16 against 29 us, T=2048 39 / 52; 32 query on 8 key heads: T=768, 192
// workgroups, 30 / 24), fp32 up to 256 (T=1000 120 / 146).
template <typename T, int D>
hipError_t launch(PrefillArgs a, const void* q, const void* k, const void* v, void* o, float* lse, hipStream_t st) {
    const long long rows = static_cast<long long>(a.Tq) * a.G.d, heads = static_cast<long long>(a.B) * a.Hkv;
    a.tiles = static_cast<int>((rows + kRows - 1) / kRows);
    if (heads * a.tiles >= (sizeof(T) == 2 ? 192 : 257)) return launch_tiles<T, D, false>(a, q, k, v, o, lse, st);
    a.tiles = static_cast<int>((rows + 31) / 32);
    return launch_tiles<T, D, true>(a, q, k, v, o, lse, st);
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_prefill(int dtype, int B, int Tq, int Tk, int Hq, int Hkv, int d, int window, int sinks,
                               float scale, const void* q, const void* k, const void* v, void* o, float* lse,
                               hipStream_t st, const AttnPacked& pk) {
    attn::PrefillArgs a{};
    a.B = B;
    a.Tq = Tq;
    a.Tk = Tk;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = attn::FastDiv(Hq / Hkv);
    a.window = window;
    a.sinks = sinks;
    a.scale = scale;
    a.cu_q = pk.cu_q;
    a.cu_k = pk.cu_k;
    a.total_q = pk.total_q;
    a.total_k = pk.total_k;
    if (dtype == GDR_DTYPE_F32)
        return d == 64 ? attn::launch<float, 64>(a, q, k, v, o, lse, st) : attn::launch<float, 128>(a, q, k, v, o, lse, st);
    return d == 64 ? attn::launch<bf16_t, 64>(a, q, k, v, o, lse, st) : attn::launch<bf16_t, 128>(a, q, k, v, o, lse, st);
}

}  // namespace gdr
