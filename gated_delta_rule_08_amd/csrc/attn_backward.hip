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
// The first of them, dq_kernel, also forms delta (from o, or where few keys are
// visible as sum_j P_ij dP_ij) and writes the row statistics the second one reads.
//
// Sink keys are seen by every later row, a list far longer than any other
// key's: those rows are cut into segments of their own (one wave each), whose
// fp32 partial sums a last kernel adds in order.  Small problems, whose keys
// alone would leave compute units without work, cut every key's rows in the
// same way, and the rows of dq_kernel give each wave a quarter of the keys.
//
// Bound by the products and the vector work between them at two waves per SIMD
// (dK and dV of 32 keys are 128 accumulators of a lane at d=128): T=8192, window
// 1024, 4 sinks, 32 query on 8 key heads: dq 228 us (40% matrix cores busy, 6 d
// flops per pair), dkdv 298 (41%, 8 d), segments 29, join 5.  fp32 with d=128 runs
// one wave per SIMD, and its sink segments (WAVES = 1) keep 18 registers in scratch.
#include "attn_backward_plan.h"
#include "attn_common.h"

namespace gdr {
namespace attn {
namespace {

template <typename T, int D, int WAVES> struct DkdvCfg {
    static constexpr int BM = 32;  // rows of a step
    static constexpr int kTile = BM * D * static_cast<int>(sizeof(T));
    static constexpr int kBuf = 2 * kTile;    // Q and dO (addresses are xor-ed: a power of two)
    static constexpr int kStat = 2 * kBuf;    // then lse2 and delta of each buffer, 32 rows by 32 rows
    static constexpr int kStatBuf = 8 * BM;
    static constexpr int kLds = kStat + 2 * kStatBuf;
};

// 32 channels of a key's gradients, or of this part of them (fp32, dk's 32 rows
// before dv's).
template <typename T, int D>
__device__ __forceinline__ void put_key(float* part, T* gk, T* gv, int t, const f32x16& dk, const f32x16& dv, float scale,
                                        int h2) {
    const f32x16 g = dk * scale;
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
        const int ch = 32 * t + row32(r, h2);
        if (part) {
            store4<float>(part + ch, g[r], g[r + 1], g[r + 2], g[r + 3]);
            store4<float>(part + 32 * D + ch, dv[r], dv[r + 1], dv[r + 2], dv[r + 3]);
        } else {
            store4<T>(gk + ch, g[r], g[r + 1], g[r + 2], g[r + 3]);
            store4<T>(gv + ch, dv[r], dv[r + 1], dv[r + 2], dv[r + 3]);
        }
    }
}

// What a wave does when a non-finite value has met its sums (a hidden pair has
// weight 0, and 0 times an infinity or NaN is NaN): its keys' gradients once
// more, hidden pairs left out.  Operands straight from global memory, 32 rows and
// 32 channels at a time, no other wave involved.
template <typename T, int D>
__device__ __forceinline__ void seen_keys(Mask mask, FastDiv G, int Hq, int rows, int pitch, float scale, int off, int key,
                                          int lo, int hi, const float* stat, const T* q, const T* go, const T* k, const T* v,
                                          float* part, T* gk, T* gv, bool store, int lane) {
    const int h2 = lane >> 5;
    const float c = scale * kLog2e;
#pragma unroll 1
    for (int t = 0; t < D / 32; ++t) {
        f32x16 dk = zero16(), dv = zero16();
#pragma unroll 1
        for (int r0 = lo; r0 < hi; r0 += 32) {
            auto row = [&](int r) {
                r = min(r0 + r, rows - 1);
                const int y = G(r);
                return (static_cast<size_t>(y) * Hq + (r - y * G.d)) * D;
            };
            uint32_t seen = 0;
#pragma unroll 1
            for (int r = 0; r < 16; ++r) {
                const int at = r0 + row32(r, h2);
                if (at < hi && mask.sees(G(at) + off, key)) seen |= 1u << r;
            }
            if (__ballot(seen != 0) == 0) continue;
            f32x16 s = zero16(), dp = zero16();
            const size_t mine = row(lane & 31) + 8 * h2;
#pragma unroll 1
            for (int e = 0; e < D / 16; ++e) {
                s = mma32(load8(q + mine + 16 * e), load8(k + 8 * h2 + 16 * e), s);
                dp = mma32(load8(go + mine + 16 * e), load8(v + 8 * h2 + 16 * e), dp);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int in = min(r0 + row32(r, h2), rows - 1);
                s[r] = ex2(fmaf(s[r], c, -stat[in]));
                dp[r] = s[r] * (dp[r] - stat[pitch + in]);
            }
            mma32_seen<T>(dv, [&](int r) { return go + row(r) + 32 * t; }, s, seen, lane);
            mma32_seen<T>(dk, [&](int r) { return q + row(r) + 32 * t; }, dp, seen, lane);
        }
        if (store) put_key<T, D>(part, gk, gv, t, dk, dv, scale, h2);
    }
}

// WAVES = 4: 128 keys of one key head, every row that sees them through the
// window.  WAVES = 1 (sinks): 32 sink keys, one segment of the rows past it.
template <typename T, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, sizeof(T) == 2 && WAVES == 4 ? 2 : 1) void dkdv_kernel(BwdArgs a, const T* __restrict__ q,
                                                             const T* __restrict__ k, const T* __restrict__ v,
                                                             const T* __restrict__ go, T* __restrict__ gk,
                                                             T* __restrict__ gv) {
    using C = DkdvCfg<T, D, WAVES>;
    constexpr int KS = D / 16, DT = D / 32, BM = C::BM;
    constexpr bool kSeg = WAVES == 1;
    extern __shared__ unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h2 = lane >> 5;
    const Piece pc = piece_of<WAVES>(a, blockIdx.x, wave);
    const int head = pc.head, b = pc.b, hk = pc.hk, lo = pc.lo, hi = pc.hi;
    if (!kSeg && pc.cut > 0 && lo >= hi) return;
    const int j0 = pc.j0, j1 = min(j0 + 31, a.Tk - 1), key = j0 + (lane & 31);
    const int off = a.Tk - a.Tq;
    if (kSeg && lo >= hi) return;
    const bool wave_live = j0 < a.Tk;
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

    // Where the group size divides 32 the rows of a step lie the same way from
    // its first one, and steps the same way apart.
    const bool even = 32 % a.G.d == 0;
    const size_t qstep = static_cast<size_t>(BM / a.G.d) * a.Hq * D;
    const TileCopy<T, D, BM, WAVES> copy(wave, lane, [&](int r) {
        const int y = a.G(r);
        return (y * a.Hq + (r - y * a.G.d)) * D * static_cast<int>(sizeof(T));
    });
    // Steps run backwards from the end of the rows or, under a window, from where
    // the workgroups of overlapping lists are at the same rows at the same time and
    // read them from L2 (window 1024, T=8192, 32 on 8 heads: 1.15 -> 0.18 GB from
    // memory, 1% of the step).
    const int n = (hi - lo + BM - 1) / BM;
    const int from = n > 0 && a.window ? n - 1 - (lo / BM + n - 1) % n : n - 1;
    const size_t low = q0 + static_cast<size_t>(a.G(lo)) * a.Hq * D;
    int next = from;  // step to fetch
    const T *qp = q + low + from * qstep, *gp = go + low + from * qstep;
    auto fetch = [&](int i) {
        const uint32_t buf = lds_addr(smem) + (i & 1) * C::kBuf;
        const uint32_t st = lds_addr(smem) + C::kStat + (i & 1) * C::kStatBuf;
        const int r0 = lo + BM * next;
        if (even && r0 + BM <= a.rows) {
            copy.run(buf, qp);
            copy.run(buf + C::kTile, gp);
            if (wave == 0) copy_words(st, stat + r0, (again(lane) < 32 ? 0u : 4u * a.pitch) + 4u * (again(lane) & 31));  // lanes 0..31: lse2, 32..63: delta
        } else {
            auto row = [&](int r) {
                r = min(r0 + r, a.rows - 1);
                const int y = a.G(r);
                return q0 + (static_cast<size_t>(y) * a.Hq + (r - y * a.G.d)) * D;
            };
            copy.gather(buf, [&](int r) { return q + row(r); });
            copy.gather(buf + C::kTile, [&](int r) { return go + row(r); });
            if (wave == 0) copy_words(st, stat + r0, 4u * (h2 * a.pitch + min(lane & 31, a.rows - 1 - r0)));
        }
        qp -= qstep;
        gp -= qstep;
        if (--next < 0) {
            next += n;
            qp += n * qstep;
            gp += n * qstep;
        }
    };
    // rows [whole_lo, whole_hi) see all of the wave's keys, rows outside [any_lo, any_hi) none
    auto rows_to = [&](int j) { return min(a.Tq, max(0, j - off)) * a.G.d; };
    const int any_lo = wave_live ? rows_to(j0) : hi, whole_lo = min(a.Tq + 1, max(0, j0 + 31 - off)) * a.G.d;
    const int any_hi = a.window == 0 || j0 < a.sinks ? hi : min(hi, rows_to(j1 + a.window));
    const int whole_hi = a.window == 0 || j0 + 31 < a.sinks ? hi : min(hi, rows_to(j0 + a.window));
    int step = from;
    const int rb0 = RowRead<T, D>::base(lane & 31, h2), cb0 = ColRead<T, D>::base(lane);
    if (n > 0) fetch(0);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        tile_barrier();
        if (i + 1 < n) fetch(i + 1);
        const int buf = (i & 1) * C::kBuf, rb = rb0 + buf, cb = cb0 + buf;
        const int r0 = lo + BM * step;
        step = step > 0 ? step - 1 : n - 1;
        if (r0 + BM <= any_lo || r0 >= any_hi) continue;
        const float* st = reinterpret_cast<const float*>(smem + C::kStat + (i & 1) * C::kStatBuf) + 4 * h2;
        const bool whole = r0 >= whole_lo && r0 + BM <= whole_hi;
        // P: registers of S as they stand are the B operand of dV
        f32x16 s = zero16();
#pragma unroll
        for (int e = 0; e < KS; ++e) {
            s = mma32(RowRead<T, D>::get(smem, rb, e, 0), kf[e], s);
            if (e % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // at most four fragments ahead: no spills
        }
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const f32x4 ls = *reinterpret_cast<const f32x4*>(st + 2 * r);
#pragma unroll
            for (int y = 0; y < 4; ++y) s[r + y] = ex2(fmaf(s[r + y], c, -ls[y]));
        }
        if (!whole) {  // the lane's key is visible to rows [key_lo, key_hi)
            const int mine = again(lane), at = j0 + (mine & 31);
            const int key_lo = rows_to(at), key_hi = a.window == 0 || at < a.sinks ? hi : min(hi, rows_to(at + a.window));
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = r0 + row32(r, mine >> 5);
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
                    dv[t] = mma32(ColRead<T, D>::get(smem, cb + C::kTile, t, u), pf[u], dv[t]);
        }
        __builtin_amdgcn_sched_barrier(0);
        f32x16 dp = zero16();
        const int rb2 = again(rb), cb2 = again(cb);
#pragma unroll
        for (int e = 0; e < KS; ++e) {
            dp = mma32(RowRead<T, D>::get(smem, rb2, e, C::kTile), vf[e], dp);
            if (e % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
        // dS is 0 where P is, unless dP - delta is not finite: then, as for dV, the
        // sums become NaN and seen_keys tells hidden pairs from visible ones whose
        // weight underflowed.
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const f32x4 de = *reinterpret_cast<const f32x4*>(st + 32 + 2 * r);
#pragma unroll
            for (int y = 0; y < 4; ++y) dp[r + y] = s[r + y] * (dp[r + y] - de[y]);
        }
        {
            frag_t<T> df[2] = {pack_regs<T>(dp, 0), pack_regs<T>(dp, 1)};
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u) dk[t] = mma32(ColRead<T, D>::get(smem, cb2, t, u), df[u], dk[t]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    if (!wave_live) return;

    bool bad = false;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) bad |= dk[t][r] != dk[t][r] || dv[t][r] != dv[t][r];

    // The keys' gradients, or this part of them.  Where they go is found again:
    // nothing of it takes registers in the loop.
    const Piece to = piece_of<WAVES>(a, __builtin_amdgcn_readfirstlane(again(blockIdx.x)), wave);
    const int me = to.j0 + (again(lane) & 31);
    const size_t at = ((static_cast<size_t>(to.b) * a.Tk + me) * a.Hkv + to.hk) * D;
    float* part = nullptr;
    if (to.parts || to.tile < a.sink_tiles)
        part = a.part_of(to.head, to.tile, kSeg ? 1 + to.cut : to.cut, D) + (me & 31) * D;
    const bool store = part ? !kSeg || me < a.sinks : me < a.Tk;  // a segment's other keys are not read by the join
    if (store) {
#pragma unroll
        for (int t = 0; t < DT; ++t) put_key<T, D>(part, gk + at, gv + at, t, dk[t], dv[t], a.scale, again(lane) >> 5);
    }
    if (__builtin_expect(__ballot(bad && store) != 0, 0)) {
        const size_t kr = ((static_cast<size_t>(to.b) * a.Tk + min(me, a.Tk - 1)) * a.Hkv + to.hk) * D;
        const size_t q0 = (static_cast<size_t>(to.b) * a.Tq * a.Hq + static_cast<size_t>(to.hk) * a.G.d) * D;
        seen_keys<T, D>(Mask{a.window, a.sinks}, a.G, a.Hq, a.rows, a.pitch, a.scale, a.Tk - a.Tq, me, to.lo, to.hi,
                        a.stats + static_cast<size_t>(to.head) * 2 * a.pitch, q + q0, go + q0, k + kr, v + kr, part, gk + at,
                        gv + at, store, again(lane));
    }
}

// Adds the parts of one key tile, every thread four elements: PER threads share
// them, each every PER-th part in order, and their sums are added in order.
template <typename T, int D, int PER>
__global__ __launch_bounds__(256) void join_kernel(BwdArgs a, T* __restrict__ gk, T* __restrict__ gv) {
    constexpr int kFours = 256 / PER;  // groups of four elements of a workgroup
    __shared__ f32x4 sums[PER][PER > 1 ? kFours : 1];
    const int head = blockIdx.x / a.part_tiles, tile = blockIdx.x % a.part_tiles;
    const int b = head / a.Hkv, hk = head - b * a.Hkv;
    const int m0 = 32 * tile / kKeys * kKeys;
    int lo, end, parts = 1;
    rows_of(a, m0, min(m0 + kKeys, a.Tk) - 1, lo, end);
    if (a.sliced) {
        const int size = slice_of(a, end - lo);
        if (end - lo <= size) return;  // written whole
        parts = (end - lo - 1) / size + 1;
    }
    const int segs = a.segs && a.rows > end ? (a.rows - end - 1) / a.seg_rows + 1 : 0;
    const float* part = a.part_of(head, tile, 0, D);
    const size_t apart = static_cast<size_t>(a.part_step) * 64 * D;
    const int x = threadIdx.x % kFours, first = threadIdx.x / kFours;
    const int i = blockIdx.y * kFours + x, row = i / (D / 4), ch = 4 * (i % (D / 4)), key = 32 * tile + (row & 31);
    if (key < a.sinks) parts += segs;  // the others have none
    f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int p = first; p < parts; p += PER)
        s += *reinterpret_cast<const f32x4*>(part + p * apart + 4 * i);
    if constexpr (PER > 1) {
        sums[first][x] = s;
        __syncthreads();
        if (first > 0) return;
#pragma unroll
        for (int p = 1; p < PER; ++p) s += sums[p][x];
    }
    if (key >= a.Tk) return;
    T* dst = (row >= 32 ? gv : gk) + ((static_cast<size_t>(b) * a.Tk + key) * a.Hkv + hk) * D + ch;
    store4<T>(dst, s[0], s[1], s[2], s[3]);
}

// As seen_keys, for one wave's rows of dQ.
template <typename T, int D, typename P>
__device__ __forceinline__ void seen_dq(const BwdArgs& a, Mask mask, int pos, int wp0, int wp1, float lse2, float delta,
                                        const T* q, const T* go, const T* k, const T* v, size_t stride, int lane, P put) {
    const int h2 = lane >> 5;
    const float c = a.scale * kLog2e;
    const KeyList keys(mask.window, mask.sinks, wp0, wp1);
#pragma unroll 1
    for (int t = 0; t < D / 32; ++t) {
        f32x16 dq = zero16();
#pragma unroll 1
        for (int x0 = 0; x0 < keys.count; x0 += 32) {
            auto row = [&](int r) { return static_cast<size_t>(min(keys.key(x0 + r), a.Tk - 1)) * stride; };
            f32x16 s = zero16(), dp = zero16();
            const size_t mine = row(lane & 31) + 8 * h2;
#pragma unroll 1
            for (int e = 0; e < D / 16; ++e) {
                s = mma32(load8(k + mine + 16 * e), load8(q + 8 * h2 + 16 * e), s);
                dp = mma32(load8(v + mine + 16 * e), load8(go + 8 * h2 + 16 * e), dp);
            }
            uint32_t seen = 0;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                if (mask.sees(pos, keys.key(x0 + row32(r, h2)))) seen |= 1u << r;
                dp[r] = ex2(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
            }
            mma32_seen<T>(dq, [&](int r) { return k + row(r) + 32 * t; }, dp, seen, lane);
        }
        put(t, dq);
    }
}

// delta = dO . o carries the rounding of o to the element type, which the
// difference dP - delta does not shrink with: with n visible keys a share of about
// 1 / n of a row's error (all of it for one key, where dS is 0).  Workgroups of bf16
// rows that see at most this many keys form delta = sum_j P_ij dP_ij in fp32
// instead, in a pass of its own (T=18, 4 heads: error of grad_q against float64
// 1.78 -> 1.40 times that of fp32 arithmetic rounded once; T=642: 1.54 -> 1.43; 4 x
// 155 tokens of 32 heads 40 -> 45 us, T=8192 the same); the others would not gain.
constexpr int kFew = 256;

template <typename T, int D, bool SPLIT> struct DqCfg {
    static constexpr int BN = SPLIT ? 32 * kWaves : 32;  // keys of a step
    static constexpr int kTile = BN * D * static_cast<int>(sizeof(T));
    static constexpr int kBufs = 4 * kTile <= 128 * 1024 ? 2 : 1;
    static constexpr int kLds = 2 * kBufs * kTile;
};

// 32 rows per wave, or with SPLIT 32 rows per workgroup, each wave a quarter
// of the keys.
template <typename T, int D, bool SPLIT>
__global__ __launch_bounds__(64 * kWaves, sizeof(T) == 2 ? 2 : 1) void dq_kernel(
    BwdArgs a, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ o,
    const T* __restrict__ go, const float* __restrict__ lse, T* __restrict__ gq) {
    using C = DqCfg<T, D, SPLIT>;
    constexpr int BN = C::BN, KS = D / 16, DT = D / 32, kGroup = SPLIT ? 32 : kRows;
    extern __shared__ unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h2 = lane >> 5;
    int head, tile;
    place(blockIdx.x, a.B * a.Hkv, a.row_tiles, head, tile);
    tile = a.row_tiles - 1 - tile;  // the last rows see the most keys
    const int b = head / a.Hkv, hk = head - b * a.Hkv;
    const int off = a.Tk - a.Tq, row0 = tile * kGroup, wrow = row0 + (SPLIT ? 0 : 32 * wave);
    const Mask mask{a.window, a.sinks};
    const int wr0 = min(wrow, a.rows - 1), wr1 = min(wrow + 31, a.rows - 1);
    const bool live = wrow + (lane & 31) < a.rows, wave_live = wrow < a.rows;
    const int row = min(wrow + (lane & 31), a.rows - 1);
    const int qi = a.G(row), pos = qi + off;
    const int wp0 = __builtin_amdgcn_readfirstlane(a.G(wr0) + off);
    const int wp1 = __builtin_amdgcn_readfirstlane(a.G(wr1) + off);
    const size_t qrow = (static_cast<size_t>(b) * a.Tq + qi) * a.Hq + static_cast<size_t>(hk) * a.G.d + (row - qi * a.G.d);
    const KeyList keys(a.window, a.sinks, a.G(row0) + off, a.G(min(row0 + kGroup - 1, a.rows - 1)) + off);
    const int n = (keys.count + BN - 1) / BN;

    const size_t kstride = static_cast<size_t>(a.Hkv) * D;
    const T* kbase = k + (static_cast<size_t>(b) * a.Tk * a.Hkv + hk) * D;
    const T* vbase = v + (static_cast<size_t>(b) * a.Tk * a.Hkv + hk) * D;
    const int sub = SPLIT ? 32 * wave : 0;  // this wave's keys of a step
    const TileRange range = TileRange::of<BN, 32>(keys, a.window, a.Tk, sub, wp0, wp1);
    const int end_tile = wave_live ? range.end : 0;
    const TileCopy<T, D, BN, kWaves> copy(wave, lane, [&](int r) { return r * static_cast<int>(kstride * sizeof(T)); });
    const T *const kp0 = kbase + keys.jump * kstride, *const vp0 = vbase + keys.jump * kstride;
    const T *kp = kp0, *vp = vp0;  // the next tile's first rows
    auto fetch = [&](int i) {      // tiles in turn
        const uint32_t buf = lds_addr(smem) + (i & (C::kBufs - 1)) * 2 * C::kTile;
        if (i >= range.full_lo && i < range.full_hi) {
            copy.run(buf, kp);
            copy.run(buf + C::kTile, vp);
        } else {
            auto key = [&](int r) { return static_cast<size_t>(min(keys.key(i * BN + r), a.Tk - 1)) * kstride; };
            copy.gather(buf, [&](int r) { return kbase + key(r); });
            copy.gather(buf + C::kTile, [&](int r) { return vbase + key(r); });
        }
        kp += BN * kstride;
        vp += BN * kstride;
    };
    if (C::kBufs == 2 && n > 0) fetch(0);

    frag_t<T> qf[KS], gf[KS];
    float delta = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        qf[s] = load8(q + qrow * D + 8 * h2 + 16 * s);
        gf[s] = load8(go + qrow * D + 8 * h2 + 16 * s);
        const frag_t<T> of = load8(o + qrow * D + 8 * h2 + 16 * s);
#pragma unroll
        for (int x = 0; x < 8; ++x) delta = fmaf(static_cast<float>(of[x]), static_cast<float>(gf[s][x]), delta);
    }
    delta += other_half(delta);
    // a row without weight (no visible key, or none with a score above -infinity): P = 0, not 2^(.. + infinity)
    const float lse2 = lse[qrow] == -INFINITY ? INFINITY : lse[qrow] * kLog2e;
    const float c = a.scale * kLog2e;
    const int rb0 = RowRead<T, D>::base(lane & 31, h2) + sub * Tile<T, D>::kRow;
    if (sizeof(T) == 2 && n > 0 && keys.count <= kFew) {  // delta as a sum over the keys
        float sum = 0.f;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            tile_barrier();
            if (i + 1 < n) fetch(i + 1);
            const int rb = rb0 + (i & 1) * 2 * C::kTile;
            if (i >= end_tile) continue;
            f32x16 s = zero16(), dp = zero16();
#pragma unroll
            for (int e = 0; e < KS; ++e) s = mma32(RowRead<T, D>::get(smem, rb, e, 0), qf[e], s);
#pragma unroll
            for (int e = 0; e < KS; ++e) dp = mma32(RowRead<T, D>::get(smem, rb, e, C::kTile), gf[e], dp);
            const int x0 = i * BN + sub;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                sum += mask.sees(pos, keys.key(x0 + row32(r, h2))) ? ex2(fmaf(s[r], c, -lse2)) * dp[r] : 0.f;
        }
        sum += other_half(sum);
        tile_barrier();
        if constexpr (SPLIT) {  // the waves' sums, in wave order
            float* box = reinterpret_cast<float*>(smem);
            box[64 * wave + lane] = sum;
            tile_barrier();
            sum = box[lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) sum += box[64 * w + lane];
            tile_barrier();
        }
        delta = sum;
        kp = kp0;
        vp = vp0;
        fetch(0);
    }
    if (a.sliced && blockIdx.x == 0)
        for (int j = threadIdx.x; j < a.part_blocks; j += 64 * kWaves) a.slots[j] = a.slots_before(j);
    if (live && (!SPLIT || wave == 0))
        a.stats[(static_cast<size_t>(head) * 2 + h2) * a.pitch + row] = h2 ? delta : lse2;
    f32x16 dq[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t) dq[t] = zero16();
    const int cb0 = ColRead<T, D>::base(lane) + sub * Tile<T, D>::kRow;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        if (C::kBufs == 1) {
            if (i > 0) tile_barrier();
            fetch(i);
        }
        tile_barrier();
        if (C::kBufs == 2 && i + 1 < n) fetch(i + 1);
        const int buf = (i & (C::kBufs - 1)) * 2 * C::kTile, rb = rb0 + buf, cb = cb0 + buf;
        if (i >= end_tile) continue;
        f32x16 s = zero16(), dp = zero16();
#pragma unroll
        for (int e = 0; e < KS; ++e) s = mma32(RowRead<T, D>::get(smem, rb, e, 0), qf[e], s);
#pragma unroll
        for (int e = 0; e < KS; ++e) dp = mma32(RowRead<T, D>::get(smem, rb, e, C::kTile), gf[e], dp);
#pragma unroll
        for (int r = 0; r < 16; ++r) dp[r] = ex2(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
        if (i < range.whole_lo || i >= range.whole_hi) {
            const int x0 = i * BN + sub;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (!mask.sees(pos, keys.key(x0 + row32(r, h2)))) dp[r] = 0.f;
        }
        const frag_t<T> df[2] = {pack_regs<T>(dp, 0), pack_regs<T>(dp, 1)};
        if (D == 128) __builtin_amdgcn_s_setprio(1);  // as in the forward (full T=4096: 1.0% of the training step)
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) dq[t] = mma32(ColRead<T, D>::get(smem, cb, t, u), df[u], dq[t]);
        if (D == 128) __builtin_amdgcn_s_setprio(0);
    }
    if constexpr (SPLIT) {  // the waves' sums, added in wave order by the first
        static_assert(C::kLds >= (kWaves - 1) * 64 * DT * 64, "LDS holds the other waves' sums");
        tile_barrier();
        float* box = reinterpret_cast<float*>(smem);
        if (wave > 0) {
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) box[(((wave - 1) * DT + t) * 16 + r) * 64 + lane] = dq[t][r];
        }
        tile_barrier();
        if (wave > 0) return;
#pragma unroll
        for (int w = 0; w < kWaves - 1; ++w)
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) dq[t][r] += box[((w * DT + t) * 16 + r) * 64 + lane];
    }
    bool bad = false;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) bad |= dq[t][r] != dq[t][r];
    auto put = [&](int t, const f32x16& x) {
        const f32x16 g = x * a.scale;
        if (!live) return;
#pragma unroll
        for (int r = 0; r < 16; r += 4)
            store4<T>(gq + qrow * D + 32 * t + row32(r, h2), g[r], g[r + 1], g[r + 2], g[r + 3]);
    };
#pragma unroll
    for (int t = 0; t < DT; ++t) put(t, dq[t]);
    if (__builtin_expect(__ballot(bad && live) != 0, 0))
        seen_dq<T, D>(a, mask, pos, wp0, wp1, lse2, delta, q + qrow * D, go + qrow * D, kbase, vbase, kstride, lane, put);
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
    const unsigned long long kv_blocks = heads * a.cuts(), q_blocks = heads * a.row_tiles;
    const unsigned long long seg_blocks = heads * a.sink_tiles * a.segs, join_blocks = heads * a.part_tiles;
    if (!grid_fits(kv_blocks, 64 * kWaves) || !grid_fits(q_blocks, 64 * kWaves) ||
        !grid_fits(seg_blocks, 64) || !grid_fits(join_blocks * (D / 2), 256))
        return hipErrorInvalidConfiguration;
    using CK = DkdvCfg<T, D, kWaves>;
    auto* dq = a.split ? dq_kernel<T, D, true> : dq_kernel<T, D, false>;
    const int dq_lds = a.split ? DqCfg<T, D, true>::kLds : DqCfg<T, D, false>::kLds;
    hipError_t e;
    if ((e = allow_lds(dkdv_kernel<T, D, kWaves>, CK::kLds)) != hipSuccess) return e;
    if ((e = allow_lds(dkdv_kernel<T, D, 1>, CK::kLds)) != hipSuccess) return e;
    if ((e = allow_lds(dq, dq_lds)) != hipSuccess) return e;
    if (q_blocks)
        hipLaunchKernelGGL(dq, dim3(static_cast<unsigned>(q_blocks)), dim3(64 * kWaves), dq_lds, st, a, q, k, v, o, go, lse,
                           static_cast<T*>(gq));
    if (kv_blocks)
        hipLaunchKernelGGL((dkdv_kernel<T, D, kWaves>), dim3(static_cast<unsigned>(kv_blocks)), dim3(64 * kWaves),
                           CK::kLds, st, a, q, k, v, go, static_cast<T*>(gk), static_cast<T*>(gv));
    if (seg_blocks)
        hipLaunchKernelGGL((dkdv_kernel<T, D, 1>), dim3(static_cast<unsigned>(seg_blocks)), dim3(64), CK::kLds, st, a, q, k,
                           v, go, static_cast<T*>(gk), static_cast<T*>(gv));
    if (join_blocks) {
        // Eight threads to four elements where parts are many or the work is small; else one, as workgroups then cost
        // more than loads in turn (4 heads, T=2504, 5 parts each: 20000 workgroups 23.6 us, an eighth of them 7.9).
        const bool many = (a.sliced ? max(a.slices, a.long_slices) : 1 + a.segs) > 16 || join_blocks * (D / 2) <= 4096;
        auto* join = many ? join_kernel<T, D, 8> : join_kernel<T, D, 1>;
        hipLaunchKernelGGL(join, dim3(static_cast<unsigned>(join_blocks), 64 * D / 4 / (many ? 32 : 256)), dim3(256), 0, st, a,
                           static_cast<T*>(gk), static_cast<T*>(gv));
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_backward(int dtype, const attn::BwdArgs& a, const void* q, const void* k, const void* v, const void* o,
                                const float* lse, const void* go, void* gq, void* gk, void* gv, hipStream_t st) {
    auto* f = dtype == GDR_DTYPE_F32 ? (a.d == 64 ? attn::launch<float, 64> : attn::launch<float, 128>)
                                     : (a.d == 64 ? attn::launch<bf16_t, 64> : attn::launch<bf16_t, 128>);
    return f(a, q, k, v, o, lse, go, gq, gk, gv, st);
}

}  // namespace gdr
