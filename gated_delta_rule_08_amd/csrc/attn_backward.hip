// Backward of the windowed attention.  With P = 2^(c s - lse log2 e), from the
// forward's log-sum-exp (no softmax pass), and delta_i = grad_o_i . o_i:
//
//   dV_j = sum_i P_ij dO_i             dS_ij = P_ij (dO_i . v_j - delta_i)
//   dQ_i = scale sum_j dS_ij k_j       dK_j = scale sum_i dS_ij q_i
//
// (dK, dV also summed over the query heads of the key head's group).  Sums over
// queries and sums over keys cannot both stay in one workgroup's registers
// without atomics, whose order would change the gradients from run to run, so
// two kernels form S and dP again: dkdv_kernel owns 32 keys per wave and walks
// the rows (queries x heads of the group) that see them; dq_kernel owns 32 rows
// per wave and walks the keys, as the forward does.  Every sum has a fixed
// order.
//
// Sink keys are seen by every later row, a list far longer than any other
// key's: those rows are cut into segments of their own (one wave each), whose
// fp32 partial sums a last kernel adds in order.
#include "attn_common.h"

namespace gdr {
namespace attn {
namespace {

__device__ __forceinline__ void tile_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

constexpr int kWaves = 4;
constexpr int kKeys = 32 * kWaves;  // keys of a dkdv workgroup
constexpr int kRows = 32 * kWaves;  // rows of a dq workgroup
constexpr int kSegRows = 512;       // rows of one sink segment

struct BwdArgs {
    int B, Tq, Tk, Hq, Hkv;
    FastDiv G;
    int window, sinks;
    float scale;
    int rows, pitch;          // rows of a (sequence, key head); pitch of the row statistics
    int key_blocks, row_tiles;
    int sink_tiles, segs;     // 32-key tiles that hold sinks, segments of each (at most)
    float* stats;             // [B Hkv, 2, pitch]: lse log2 e, then delta
    float* part;              // [B Hkv, sink_tiles, 1 + segs, 2, 32, d]
};

// Rows (query * G + head) that see keys [j0, j1] through the window or, with
// no window, causally: [lo, hi).
__device__ __forceinline__ void rows_of(const BwdArgs& a, int j0, int j1, int& lo, int& hi) {
    const int off = a.Tk - a.Tq;
    lo = max(0, j0 - off) * a.G.d;
    const int last = a.window ? min(a.Tq - 1, j1 + a.window - 1 - off) : a.Tq - 1;
    hi = max(lo, (last + 1) * a.G.d);
}

// Row statistics in row order: lse in base 2 and delta, 16 lanes per row.
template <typename T, int D>
__global__ __launch_bounds__(256) void stats_kernel(BwdArgs a, const T* __restrict__ o, const T* __restrict__ go,
                                                    const float* __restrict__ lse) {
    const size_t n = static_cast<size_t>(a.B) * a.Tq * a.Hq;
    const size_t i = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) >> 4;
    if (i >= n) return;
    const int l16 = threadIdx.x & 15;
    constexpr int N = D / 16;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < N; e += 4)
#pragma unroll
        for (int x = 0; x < 4; ++x)
            s = fmaf(Elem<T>::load(o + i * D + N * l16 + e + x), Elem<T>::load(go + i * D + N * l16 + e + x), s);
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) s += __shfl_xor(s, x);
    if (l16) return;
    const size_t tok = i / a.Hq;
    const int head = static_cast<int>(i - tok * a.Hq), b = static_cast<int>(tok / a.Tq);
    const size_t at = (static_cast<size_t>(b) * a.Hkv + a.G(head)) * 2 * a.pitch +
                      (tok - static_cast<size_t>(b) * a.Tq) * a.G.d + (head - a.G(head) * a.G.d);
    a.stats[at] = lse[i] * kLog2e;
    a.stats[at + a.pitch] = s;
}

// What a wave does when a non-finite value met its sums (a hidden pair has
// weight 0, and 0 times an infinity or NaN is NaN): its keys' gradients row by
// row, hidden pairs left out.  A lane holds half of its key's channels.
template <typename T, int D>
__device__ __forceinline__ void exact_keys(const BwdArgs& a, int b, int hk, int key, int off, int lo, int hi, const T* q,
                                        const T* k, const T* v, const T* go, float* dk, float* dv, int h2) {
    constexpr int N = D / 2;
    const Mask mask{a.window, a.sinks};
    const size_t krow = ((static_cast<size_t>(b) * a.Tk + min(key, a.Tk - 1)) * a.Hkv + hk) * D;
    const float c = a.scale * kLog2e;
    const float* stat = a.stats + (static_cast<size_t>(b) * a.Hkv + hk) * 2 * a.pitch;
#pragma unroll 1
    for (int e = 0; e < N; ++e) dk[e] = dv[e] = 0.f;
#pragma unroll 1
    for (int r = lo; r < hi; ++r) {
        const int i = a.G(r);
        const size_t qrow = ((static_cast<size_t>(b) * a.Tq + i) * a.Hq + hk * a.G.d + (r - i * a.G.d)) * D;
        float s = 0.f, dp = 0.f;
#pragma unroll 1
        for (int e = N * h2; e < N * h2 + N; ++e) {
            s = fmaf(Elem<T>::load(q + qrow + e), Elem<T>::load(k + krow + e), s);
            dp = fmaf(Elem<T>::load(go + qrow + e), Elem<T>::load(v + krow + e), dp);
        }
        s += other_half(s);
        dp += other_half(dp);
        if (!mask.sees(i + off, key)) continue;
        const float p = ex2(fmaf(s, c, -stat[r])), ds = p * (dp - stat[a.pitch + r]);
#pragma unroll 1
        for (int e = 0; e < N; ++e) {
            dk[e] = fmaf(ds, Elem<T>::load(q + qrow + N * h2 + e), dk[e]);
            dv[e] = fmaf(p, Elem<T>::load(go + qrow + N * h2 + e), dv[e]);
        }
    }
}

template <typename T, int D, int WAVES> struct DkdvCfg {
    static constexpr int BM = 32;  // rows of a step
    static constexpr int kTile = BM * D * static_cast<int>(sizeof(T));
    static constexpr int kBuf = 2 * kTile;    // Q and dO (addresses are xor-ed: a power of two)
    static constexpr int kStat = 2 * kBuf;    // then lse2 and delta of each buffer, 32 rows by 32 rows
    static constexpr int kStatBuf = 8 * BM;
    static constexpr int kLds = kStat + 2 * kStatBuf;
};

// WAVES = 4: 128 keys of one key head, every row that sees them through the
// window.  WAVES = 1 (sinks): 32 sink keys, one segment of the rows past it.
template <typename T, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, sizeof(T) == 2 && WAVES == 4 ? 2 : 1) void dkdv_kernel(BwdArgs a, const T* __restrict__ q,
                                                             const T* __restrict__ k, const T* __restrict__ v,
                                                             const T* __restrict__ go, T* __restrict__ gk,
                                                             T* __restrict__ gv) {
    using C = DkdvCfg<T, D, WAVES>;
    using L = Tile<T, D>;
    constexpr int KS = D / 16, DT = D / 32, BM = C::BM, NM = BM / 32;
    constexpr bool kSeg = WAVES == 1;
    extern __shared__ unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h2 = lane >> 5;
    const int per = kSeg ? a.sink_tiles * a.segs : a.key_blocks;
    const int heads = a.B * a.Hkv;
    int bid = blockIdx.x, head, x;
    if (heads % 8 == 0) {  // one head's blocks on one XCD
        head = (bid / 8 / per) * 8 + (bid & 7);
        x = (bid / 8) % per;
    } else {
        head = bid % heads;
        x = bid / heads;
    }
    const int b = head / a.Hkv, hk = head - b * a.Hkv;
    const int seg = kSeg ? x % a.segs : 0;
    const int tile = kSeg ? x / a.segs : x * WAVES + wave;  // 32-key tile of this wave
    const int j0 = 32 * tile, j1 = min(j0 + 31, a.Tk - 1), key = j0 + (lane & 31);
    const int off = a.Tk - a.Tq;
    const Mask mask{a.window, a.sinks};

    int lo, hi;
    if (kSeg) {
        const int m0 = j0 / kKeys * kKeys;  // the main workgroup's keys: its rows end at hi
        int end;
        rows_of(a, m0, min(m0 + kKeys, a.Tk) - 1, lo, end);
        lo = end + seg * kSegRows;
        hi = min(a.rows, lo + kSegRows);
    } else {
        rows_of(a, x * kKeys, min(x * kKeys + kKeys, a.Tk) - 1, lo, hi);
    }
    if (kSeg && lo >= hi) return;
    const bool wave_live = j0 < a.Tk;
    // this lane's key is visible to rows [key_lo, key_hi) of [lo, hi)
    const int key_lo = min(a.Tq, max(0, key - off)) * a.G.d;
    const int key_hi = a.window == 0 || key < a.sinks ? hi : min(hi, min(a.Tq, max(0, key + a.window - off)) * a.G.d);

    const size_t kstride = static_cast<size_t>(a.Hkv) * D;
    const size_t k0 = (static_cast<size_t>(b) * a.Tk * a.Hkv + hk) * D;
    frag_t<T> kf[KS], vf[KS];
    {
        const size_t r = k0 + min(key, a.Tk - 1) * kstride + 8 * h2;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            kf[s] = load8(k + r + 16 * s);
            vf[s] = load8(v + r + 16 * s);
        }
    }
    f32x16 dk[DT], dv[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t) dk[t] = dv[t] = zero16();
    const float c = a.scale * kLog2e;
    const float* stat = a.stats + static_cast<size_t>(head) * 2 * a.pitch;
    const size_t q0 = (static_cast<size_t>(b) * a.Tq * a.Hq + static_cast<size_t>(hk) * a.G.d) * D;

    auto fetch = [&](int i) {
        unsigned char* buf = smem + (i & 1) * C::kBuf;
        const int r0 = lo + BM * i, i0 = a.G(r0);
        const size_t base = q0 + static_cast<size_t>(i0) * a.Hq * D;
        copy_rows<T, D, BM, WAVES>(buf, q + base, buf + C::kTile, go + base, wave, lane, [&](int r) {
            const int row = min(r0 + r, a.rows - 1), y = a.G(row);
            return ((y - i0) * a.Hq + (row - y * a.G.d)) * D;
        });
        if (wave < NM) {  // lanes 0..31: lse2, 32..63: delta
            const int r = min(32 * wave + (lane & 31), a.rows - 1 - r0);
            copy_words(smem + C::kStat + (i & 1) * C::kStatBuf + 256 * wave, stat + r0, 4u * (h2 * a.pitch + r));
        }
    };
    const int n = (hi - lo + BM - 1) / BM;
    const int rb0 = RowRead<T, D>::base(lane & 31, h2), cb0 = ColRead<T, D>::base(lane);
    if (n > 0) fetch(0);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        tile_barrier();
        if (i + 1 < n) fetch(i + 1);
        const int buf = (i & 1) * C::kBuf, rb = rb0 + buf, cb = cb0 + buf;
        const int r0 = lo + BM * i;
        const int p0 = a.G(r0) + off, p1 = a.G(min(r0 + BM - 1, hi - 1)) + off;
        if (!wave_live || mask.none(p0, p1, j0, j1)) continue;
        const float* st = reinterpret_cast<const float*>(smem + C::kStat + (i & 1) * C::kStatBuf) + 4 * h2;
        const bool whole = mask.all(p0, p1, j0, j0 + 31) && r0 + BM <= hi;
#pragma unroll
        for (int w = 0; w < NM; ++w) {
            // P: registers of S as they stand are the B operand of dV
            f32x16 s = zero16();
#pragma unroll
            for (int e = 0; e < KS; ++e) {
                s = mma32(RowRead<T, D>::get(smem, rb, e, 32 * w * L::kRow), kf[e], s);
                if (e % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // at most four fragments ahead: no spills
            }
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const f32x4 ls = *reinterpret_cast<const f32x4*>(st + 64 * w + 2 * r);
#pragma unroll
                for (int y = 0; y < 4; ++y) s[r + y] = ex2(fmaf(s[r + y], c, -ls[y]));
            }
            if (!whole) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int row = r0 + 32 * w + row32(r, h2);
                    if (row < key_lo || row >= key_hi) s[r] = 0.f;
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            {
                frag_t<T> pf[2] = {pack_regs<T>(s, 0), pack_regs<T>(s, 1)};
#pragma unroll
                for (int t = 0; t < DT; ++t)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        dv[t] = mma32(ColRead<T, D>::get(smem, cb + C::kTile, t, 2 * w + u), pf[u], dv[t]);
            }
            __builtin_amdgcn_sched_barrier(0);
            f32x16 dp = zero16();
            const int rb2 = again(rb), cb2 = again(cb);
#pragma unroll
            for (int e = 0; e < KS; ++e) {
                dp = mma32(RowRead<T, D>::get(smem, rb2, e, C::kTile + 32 * w * L::kRow), vf[e], dp);
                if (e % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const f32x4 de = *reinterpret_cast<const f32x4*>(st + 64 * w + 32 + 2 * r);
#pragma unroll
                for (int y = 0; y < 4; ++y) dp[r + y] = s[r + y] * (dp[r + y] - de[y]);
            }
            if (!whole) {  // a hidden pair's weight is 0, its dP may be anything
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (s[r] == 0.f) dp[r] = 0.f;
            }
            {
                frag_t<T> df[2] = {pack_regs<T>(dp, 0), pack_regs<T>(dp, 1)};
#pragma unroll
                for (int t = 0; t < DT; ++t)
#pragma unroll
                    for (int u = 0; u < 2; ++u) dk[t] = mma32(ColRead<T, D>::get(smem, cb2, t, 2 * w + u), df[u], dk[t]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (!wave_live) return;

    // the keys' gradients, or this part of a sink tile's
    float* part = nullptr;
    if (tile < a.sink_tiles)
        part = a.part + ((static_cast<size_t>(head) * a.sink_tiles + tile) * (1 + a.segs) + (kSeg ? 1 + seg : 0)) * 64 * D;
    bool bad = false;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) bad |= dk[t][r] != dk[t][r] || dv[t][r] != dv[t][r];
    if (__any(bad && key < a.Tk)) {
        constexpr int N = D / 2;
        float xk[N], xv[N];
        exact_keys<T, D>(a, b, hk, key, off, lo, hi, q, k, v, go, xk, xv, h2);
#pragma unroll 1
        for (int e = 0; e < N; ++e) {
            const int ch = N * h2 + e;
            if (part) {
                part[(lane & 31) * D + ch] = xk[e] * a.scale;
                part[(32 + (lane & 31)) * D + ch] = xv[e];
            } else if (key < a.Tk) {
                Elem<T>::store(gk + k0 + key * kstride + ch, xk[e] * a.scale);
                Elem<T>::store(gv + k0 + key * kstride + ch, xv[e]);
            }
        }
        return;
    }
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const int ch = 32 * t + row32(r, h2);
            const f32x16 g = dk[t] * a.scale;
            if (part) {
                store4<float>(part + (lane & 31) * D + ch, g[r], g[r + 1], g[r + 2], g[r + 3]);
                store4<float>(part + (32 + (lane & 31)) * D + ch, dv[t][r], dv[t][r + 1], dv[t][r + 2], dv[t][r + 3]);
            } else if (key < a.Tk) {
                store4<T>(gk + k0 + key * kstride + ch, g[r], g[r + 1], g[r + 2], g[r + 3]);
                store4<T>(gv + k0 + key * kstride + ch, dv[t][r], dv[t][r + 1], dv[t][r + 2], dv[t][r + 3]);
            }
        }
}

// Adds the parts of one sink tile in order, four elements a thread.
template <typename T, int D>
__global__ __launch_bounds__(256) void sink_join_kernel(BwdArgs a, T* __restrict__ gk, T* __restrict__ gv) {
    const int head = blockIdx.x / a.sink_tiles, tile = blockIdx.x % a.sink_tiles;
    const int b = head / a.Hkv, hk = head - b * a.Hkv;
    const int m0 = 32 * tile / kKeys * kKeys;
    int lo, end;
    rows_of(a, m0, min(m0 + kKeys, a.Tk) - 1, lo, end);
    const int parts = 1 + (a.rows > end ? (a.rows - end - 1) / kSegRows + 1 : 0);
    const float* part = a.part + (static_cast<size_t>(head) * a.sink_tiles + tile) * (1 + a.segs) * 64 * D;
    const int i = blockIdx.y * 256 + threadIdx.x, row = i / (D / 4), ch = 4 * (i % (D / 4)), key = 32 * tile + (row & 31);
    if (key >= a.Tk) return;
    f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int p = 0; p < parts; ++p) s += *reinterpret_cast<const f32x4*>(part + static_cast<size_t>(p) * 64 * D + 4 * i);
    T* dst = (row >= 32 ? gv : gk) + ((static_cast<size_t>(b) * a.Tk + key) * a.Hkv + hk) * D + ch;
    store4<T>(dst, s[0], s[1], s[2], s[3]);
}

// As exact_keys, for one wave's rows of dQ.
template <typename T, int D>
__device__ __forceinline__ void exact_dq(const BwdArgs& a, Mask mask, int pos, bool live, int wp1, float lse2, float delta,
                                      const T* q, const T* go, const T* k, const T* v, size_t stride, T* gq, int h2) {
    constexpr int N = D / 2;
    const float c = a.scale * kLog2e;
    float dq[N];
#pragma unroll 1
    for (int e = 0; e < N; ++e) dq[e] = 0.f;
#pragma unroll 1
    for (int j = 0; j <= wp1; ++j) {
        float s = 0.f, dp = 0.f;
#pragma unroll 1
        for (int e = N * h2; e < N * h2 + N; ++e) {
            s = fmaf(Elem<T>::load(q + e), Elem<T>::load(k + j * stride + e), s);
            dp = fmaf(Elem<T>::load(go + e), Elem<T>::load(v + j * stride + e), dp);
        }
        s += other_half(s);
        dp += other_half(dp);
        if (!mask.sees(pos, j)) continue;
        const float ds = ex2(fmaf(s, c, -lse2)) * (dp - delta);
#pragma unroll 1
        for (int e = 0; e < N; ++e) dq[e] = fmaf(ds, Elem<T>::load(k + j * stride + N * h2 + e), dq[e]);
    }
    if (!live) return;
#pragma unroll 1
    for (int e = 0; e < N; ++e) Elem<T>::store(gq + N * h2 + e, dq[e] * a.scale);
}

template <typename T, int D> struct DqCfg {
    static constexpr int BN = 32;
    static constexpr int kTile = BN * D * static_cast<int>(sizeof(T));
    static constexpr int kLds = 4 * kTile;
};

template <typename T, int D>
__global__ __launch_bounds__(64 * kWaves, sizeof(T) == 2 ? 2 : 1) void dq_kernel(BwdArgs a, const T* __restrict__ q, const T* __restrict__ k,
                                                            const T* __restrict__ v, const T* __restrict__ go,
                                                            T* __restrict__ gq) {
    using C = DqCfg<T, D>;
    constexpr int BN = C::BN, KS = D / 16, DT = D / 32;
    extern __shared__ unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h2 = lane >> 5;
    const int heads = a.B * a.Hkv, bid = blockIdx.x;
    int head, tile;
    if (heads % 8 == 0) {
        head = (bid / 8 / a.row_tiles) * 8 + (bid & 7);
        tile = a.row_tiles - 1 - (bid / 8) % a.row_tiles;
    } else {
        head = bid % heads;
        tile = a.row_tiles - 1 - bid / heads;
    }
    const int b = head / a.Hkv, hk = head - b * a.Hkv;
    const int off = a.Tk - a.Tq, row0 = tile * kRows;
    const Mask mask{a.window, a.sinks};
    const int wr0 = min(row0 + 32 * wave, a.rows - 1), wr1 = min(row0 + 32 * wave + 31, a.rows - 1);
    const bool live = row0 + 32 * wave + (lane & 31) < a.rows, wave_live = row0 + 32 * wave < a.rows;
    const int row = min(row0 + 32 * wave + (lane & 31), a.rows - 1);
    const int qi = a.G(row), pos = qi + off;
    const int wp0 = __builtin_amdgcn_readfirstlane(a.G(wr0) + off);
    const int wp1 = __builtin_amdgcn_readfirstlane(a.G(wr1) + off);
    const size_t qrow = (static_cast<size_t>(b) * a.Tq + qi) * a.Hq + static_cast<size_t>(hk) * a.G.d + (row - qi * a.G.d);
    const int p0 = a.G(row0) + off, p1 = a.G(min(row0 + kRows - 1, a.rows - 1)) + off;
    const int w_lo = a.window ? max(0, p0 - a.window + 1) : 0;
    const int t_lo = w_lo / BN, t_hi = p1 < 0 ? -1 : p1 / BN;
    const int t_sink = a.window ? min((a.sinks + BN - 1) / BN, t_lo) : 0;
    const int n = t_hi < t_lo ? 0 : t_sink + t_hi - t_lo + 1;

    frag_t<T> qf[KS], gf[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        qf[s] = load8(q + qrow * D + 8 * h2 + 16 * s);
        gf[s] = load8(go + qrow * D + 8 * h2 + 16 * s);
    }
    const float lse2 = a.stats[static_cast<size_t>(head) * 2 * a.pitch + row];
    const float delta = a.stats[(static_cast<size_t>(head) * 2 + 1) * a.pitch + row];
    const float c = a.scale * kLog2e;
    f32x16 dq[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t) dq[t] = zero16();
    const size_t kstride = static_cast<size_t>(a.Hkv) * D;
    const T* kbase = k + (static_cast<size_t>(b) * a.Tk * a.Hkv + hk) * D;
    const T* vbase = v + (static_cast<size_t>(b) * a.Tk * a.Hkv + hk) * D;
    auto tile_of = [&](int i) { return i < t_sink ? i : i - t_sink + t_lo; };
    auto fetch = [&](int i) {
        unsigned char* buf = smem + (i & 1) * 2 * C::kTile;
        const int j0 = tile_of(i) * BN;
        copy_rows<T, D, BN, kWaves>(buf, kbase + j0 * kstride, buf + C::kTile, vbase + j0 * kstride, wave, lane,
                                    [&](int r) { return min(r, a.Tk - 1 - j0) * a.Hkv * D; });
    };
    const int rb0 = RowRead<T, D>::base(lane & 31, h2), cb0 = ColRead<T, D>::base(lane);
    if (n > 0) fetch(0);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        tile_barrier();
        if (i + 1 < n) fetch(i + 1);
        const int buf = (i & 1) * 2 * C::kTile, rb = rb0 + buf, cb = cb0 + buf;
        const int j0 = tile_of(i) * BN;
        if (!wave_live || mask.none(wp0, wp1, j0, j0 + BN - 1)) continue;
        f32x16 s = zero16(), dp = zero16();
#pragma unroll
        for (int e = 0; e < KS; ++e) s = mma32(RowRead<T, D>::get(smem, rb, e, 0), qf[e], s);
#pragma unroll
        for (int e = 0; e < KS; ++e) dp = mma32(RowRead<T, D>::get(smem, rb, e, C::kTile), gf[e], dp);
#pragma unroll
        for (int r = 0; r < 16; ++r) dp[r] = ex2(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
        if (!mask.all(wp0, wp1, j0, j0 + BN - 1)) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (!mask.sees(pos, j0 + row32(r, h2))) dp[r] = 0.f;
        }
        frag_t<T> df[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float z[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) z[y] = dp[8 * u + y];
            df[u] = pack8<T>(z);
        }
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) dq[t] = mma32(ColRead<T, D>::get(smem, cb, t, u), df[u], dq[t]);
    }
    bool bad = false;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) bad |= dq[t][r] != dq[t][r];
    if (__any(bad && live)) {
        exact_dq<T, D>(a, mask, pos, live, wp1, lse2, delta, q + qrow * D, go + qrow * D, kbase, vbase, kstride,
                       gq + qrow * D, h2);
        return;
    }
    if (!live) return;
#pragma unroll
    for (int t = 0; t < DT; ++t) {
        const f32x16 g = dq[t] * a.scale;
#pragma unroll
        for (int r = 0; r < 16; r += 4)
            store4<T>(gq + qrow * D + 32 * t + row32(r, h2), g[r], g[r + 1], g[r + 2], g[r + 3]);
    }
}

BwdArgs make_args(int B, int Tq, int Tk, int Hq, int Hkv, int window, int sinks, float scale) {
    BwdArgs a{};
    a.B = B;
    a.Tq = Tq;
    a.Tk = Tk;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = FastDiv(Hq / Hkv);
    a.window = window;
    a.sinks = sinks;
    a.scale = scale;
    a.rows = Tq * a.G.d;
    a.pitch = (a.rows + 3) / 4 * 4;
    a.key_blocks = (Tk + kKeys - 1) / kKeys;
    a.row_tiles = (a.rows + kRows - 1) / kRows;
    a.sink_tiles = window && Tq > 0 ? (sinks + 31) / 32 : 0;
    a.segs = a.sink_tiles ? (a.rows + kSegRows - 1) / kSegRows : 0;
    return a;
}

template <typename K> hipError_t allow_lds(K* f, int bytes) {
    if (bytes <= 64 * 1024) return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, int D>
hipError_t launch(const BwdArgs& a, const void* q_, const void* k_, const void* v_, const void* o_, const float* lse,
                  const void* go_, void* gq, void* gk, void* gv, hipStream_t st) {
    const T *q = static_cast<const T*>(q_), *k = static_cast<const T*>(k_), *v = static_cast<const T*>(v_),
            *o = static_cast<const T*>(o_), *go = static_cast<const T*>(go_);
    const unsigned long long heads = static_cast<unsigned long long>(a.B) * a.Hkv;
    const unsigned long long stat_blocks = (static_cast<unsigned long long>(a.B) * a.Tq * a.Hq + 15) / 16;
    const unsigned long long kv_blocks = heads * a.key_blocks, q_blocks = heads * a.row_tiles;
    const unsigned long long seg_blocks = heads * a.sink_tiles * a.segs, join_blocks = heads * a.sink_tiles;
    if (!grid_fits(stat_blocks, 256) || !grid_fits(kv_blocks, 64 * kWaves) || !grid_fits(q_blocks, 64 * kWaves) ||
        !grid_fits(seg_blocks, 64) || !grid_fits(join_blocks * (D / 16), 256))
        return hipErrorInvalidConfiguration;
    using CK = DkdvCfg<T, D, kWaves>;
    using CQ = DqCfg<T, D>;
    hipError_t e;
    if ((e = allow_lds(dkdv_kernel<T, D, kWaves>, CK::kLds)) != hipSuccess) return e;
    if ((e = allow_lds(dkdv_kernel<T, D, 1>, CK::kLds)) != hipSuccess) return e;
    if ((e = allow_lds(dq_kernel<T, D>, CQ::kLds)) != hipSuccess) return e;
    if (stat_blocks)
        hipLaunchKernelGGL((stats_kernel<T, D>), dim3(static_cast<unsigned>(stat_blocks)), dim3(256), 0, st, a, o, go, lse);
    if (kv_blocks)
        hipLaunchKernelGGL((dkdv_kernel<T, D, kWaves>), dim3(static_cast<unsigned>(kv_blocks)), dim3(64 * kWaves),
                           CK::kLds, st, a, q, k, v, go, static_cast<T*>(gk), static_cast<T*>(gv));
    if (join_blocks) {
        if (seg_blocks)
            hipLaunchKernelGGL((dkdv_kernel<T, D, 1>), dim3(static_cast<unsigned>(seg_blocks)), dim3(64), CK::kLds, st, a,
                               q, k, v, go, static_cast<T*>(gk), static_cast<T*>(gv));
        hipLaunchKernelGGL((sink_join_kernel<T, D>), dim3(static_cast<unsigned>(join_blocks), 64 * D / 4 / 256), dim3(256), 0, st, a,
                           static_cast<T*>(gk), static_cast<T*>(gv));
    }
    if (q_blocks)
        hipLaunchKernelGGL((dq_kernel<T, D>), dim3(static_cast<unsigned>(q_blocks)), dim3(64 * kWaves), CQ::kLds, st, a,
                           q, k, v, go, static_cast<T*>(gq));
    return hipGetLastError();
}

}  // namespace
}  // namespace attn

size_t attn_backward_workspace_floats(int B, int Tq, int Tk, int Hq, int Hkv, int d, int window, int sinks) {
    const attn::BwdArgs a = attn::make_args(B, Tq, Tk, Hq, Hkv, window, sinks, 1.f);
    const size_t heads = static_cast<size_t>(B) * Hkv;
    return heads * (2 * static_cast<size_t>(a.pitch) + static_cast<size_t>(a.sink_tiles) * (1 + a.segs) * 64 * d);
}

hipError_t launch_attn_backward(int dtype, int B, int Tq, int Tk, int Hq, int Hkv, int d, int window, int sinks,
                                float scale, const void* q, const void* k, const void* v, const void* o,
                                const float* lse, const void* go, void* gq, void* gk, void* gv, float* ws,
                                hipStream_t st) {
    attn::BwdArgs a = attn::make_args(B, Tq, Tk, Hq, Hkv, window, sinks, scale);
    const size_t heads = static_cast<size_t>(B) * Hkv;
    a.stats = ws;
    a.part = ws + heads * 2 * a.pitch;
    auto* f = dtype == GDR_DTYPE_F32 ? (d == 64 ? attn::launch<float, 64> : attn::launch<float, 128>)
                                     : (d == 64 ? attn::launch<bf16_t, 64> : attn::launch<bf16_t, 128>);
    return f(a, q, k, v, o, lse, go, gq, gk, gv, st);
}

}  // namespace gdr
