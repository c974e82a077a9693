// Attention over a key-value cache held in 4 bits: the append of new tokens, their
// way back to dense tensors, and the decode step.
//
// The format of a block is attn_mx4.h's.  Keys lie row by row, a position's d / 2
// bytes together; values lie in blocks of 32 positions, the 16 bytes of a channel
// together, so that the operands of both products of the decode step come from
// memory to the registers of the lanes that need them: a lane of the score product
// wants consecutive channels of a key, a lane of the output product consecutive
// positions of a channel.  No LDS, no transposition, and wide loads throughout.
// Scales lie position by position.
#include <type_traits>

#include "attn_deal.h"
#include "attn_mx4.h"

namespace gdr {
namespace attn {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- decode

constexpr int kMxWaves = 4;
constexpr int kQuad = 4 * kMxRows;  // positions of a wave's step: 4 blocks of 32

// At query position p a key j is visible if j <= p and (window == 0 or j > p - window or j < sinks).
struct Mx4Args {
    int B, Tq, Hq, Hkv, G, head_tiles;
    int page_shift, num_pages, max_pages;
    int window, sinks;
    float scale;
    int shares;  // workgroups the blocks are dealt to; 0: one workgroup per unit
    int heads;   // rows of a unit: min(16, Tq * G)

    __host__ __device__ __forceinline__ int per() const { return Hkv * head_tiles; }
    __device__ __forceinline__ int blocks(int len) const;
    __device__ __forceinline__ bool skipped(int, int, const int*) const { return false; }
    __device__ __forceinline__ JoinRow row(int r) const {  // output row: [b, query, head]
        const int hq = r % Hq, bi = r / Hq, i = bi % Tq, hk = hq / G, c = i * G + hq - hk * G;
        return JoinRow{bi / Tq, hk * head_tiles + c / 16, c & 15};
    }
};

// The blocks of 32 positions that the queries of a sequence of n positions may
// see: those of the sinks, then those from the first query's window on.
struct MxSpan {
    int p0, p1;         // positions of the first and the last query
    int sinks, jump;    // blocks 0 .. sinks-1 come first; entry x >= sinks is block x + jump
    int entries, steps; // steps of four entries; 0: the length is out of range
};
__device__ __forceinline__ MxSpan mx_span(const Mx4Args& a, int n) {
    MxSpan s;
    s.p1 = n - 1;
    s.p0 = n - a.Tq;
    const int lo = a.window ? max(0, s.p0 - a.window + 1) : 0;
    s.sinks = min((min(a.sinks, lo) + kMxRows - 1) / kMxRows, lo / kMxRows);
    s.jump = lo / kMxRows - s.sinks;
    s.entries = n > 0 ? s.p1 / kMxRows - s.jump + 1 : 0;
    const bool fits = n >= 0 && (s.p1 >> a.page_shift) < a.max_pages;
    s.steps = fits ? max(1, (s.entries + 3) / 4) : 0;  // without keys one step, which writes the zeros
    return s;
}
__device__ __forceinline__ int Mx4Args::blocks(int len) const { return mx_span(*this, len).steps; }

// A row of 8 fp32 values as NP bf16 pieces, the first rounded, the next the rest.
template <typename T> struct Pieces;
template <> struct Pieces<bf16_t> { static constexpr int n = 1; };
template <> struct Pieces<float> { static constexpr int n = 3; };
template <int NP> __device__ __forceinline__ void split8(const float (&x)[8], bf16x8v (&to)[NP]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float rest = x[i];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const __bf16 h = static_cast<__bf16>(rest);
            to[p][i] = h;
            rest -= static_cast<float>(h);
        }
    }
}

// One decode step.  A wave takes 128 positions at a time: block h of the four goes
// with the lanes 16 h .. 16 h + 15.
//
//  S^T = K Q^T, eight tiles of 16 keys, tile t holding positions 4 t .. 4 t + 3 of
//  each block: the accumulator of lane (c, h) is then positions 4 t + r of block h
//  for query row c, 32 positions in all, in order.
//  O^T = V^T P^T: the lane's 8 weights of positions 8 i .. 8 i + 7 are the operand as
//  they stand, and the other is word i of a channel's 16 bytes.
//
// The keys' scales are applied by the conversion to bf16, which is exact.  The
// values' scales differ along the summed axis and are multiplied into the weights:
// one set of weights for every 32 channels.  bf16: the weights are rounded to bf16
// before the power of two, or after it, which is the same.  fp32: queries and
// weights go in as three bf16 pieces, 24 bits, and no bit of the codes is lost.
template <typename T, int D>
__global__ __launch_bounds__(64 * kMxWaves, 2) void mx4_decode_kernel(
    Mx4Args a, const T* __restrict__ q, const uint8_t* __restrict__ k_codes, const uint8_t* __restrict__ k_scales,
    const uint8_t* __restrict__ v_codes, const uint8_t* __restrict__ v_scales, const int* __restrict__ table,
    const int* __restrict__ lengths, T* __restrict__ o, float* __restrict__ part_o, float* __restrict__ part_ml) {
    constexpr int NP = Pieces<T>::n, KS = D / 32, DT = D / 16, CB = D / 32;
    constexpr int kLane = D / 8;      // bytes of a key in one lane
    constexpr int kPitch = D + 4;     // floats of a joined row
    constexpr int kWords = CB * 8;    // words of a block's 32 x CB scales
    __shared__ __align__(16) float jo[kMxWaves * 16 * kPitch];
    __shared__ float jm[kMxWaves * 16 * 2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c16 = lane & 15, h4 = lane >> 4;
    const int per = a.per(), slot_mask = (1 << a.page_shift) - 1;
    // a scale of 0 as one that no score survives: c -inf of a hidden key stays -inf
    const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-37f);

    Share share;
    if (!find_share(a, lengths, lane, blockIdx.x, share)) return;
    int b = share.b, unit = share.unit, at_block = share.at_block, left = share.left;
    MxSpan sp = mx_span(a, lengths[b]);

#pragma unroll 1
    while (left > 0) {
        if (unit >= per || sp.steps == 0) {  // the next sequence that is not skipped
            if (++b >= a.B) return;
            unit = 0;
            sp = mx_span(a, lengths[b]);
            continue;
        }
        const int take = min(left, sp.steps - at_block);
        const int hk = unit / a.head_tiles, ht = unit - hk * a.head_tiles;
        const int* trow = table + static_cast<size_t>(b) * a.max_pages;

        // this lane's query row: query i, head g of the group
        const int rows = min(16, a.Tq * a.G - ht * 16);
        const int mine = ht * 16 + min(c16, rows - 1), qi = mine / a.G;
        const int pos = sp.p0 + qi;
        const size_t orow = (static_cast<size_t>(b) * a.Tq + qi) * a.Hq + hk * a.G + mine - qi * a.G;
        bf16x8v qf[KS][NP];
        {
            const T* qp = q + orow * D + (D / 4) * h4;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = Elem<T>::load(qp + 8 * s + i);
                if (a.scale < 0.f) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = -x[i];
                }
                split8<NP>(x, qf[s]);
            }
        }

        // Entry e of the list: the row of its first position in the page tensors, or
        // -1 where there is none (past the list, or on a page outside the pool).
        auto row_of = [&](int e) {
            if (e >= sp.entries) return -1;
            const int first = (e < sp.sinks ? e : e + sp.jump) * kMxRows;
            const int page = trow[first >> a.page_shift];
            if (page < 0 || page >= a.num_pages) return -1;
            return ((page * a.Hkv + hk) << a.page_shift) + (first & slot_mask);
        };

        f32x4 acc[DT];
#pragma unroll
        for (int t = 0; t < DT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, l = 0.f;

#pragma unroll 1
        for (int step = at_block + wave; step < at_block + take; step += kMxWaves) {
            const int krow = row_of(4 * step + (c16 >> 2)), vrow = row_of(4 * step + h4);
            // keys: lane (c, h) has channels D/4 h .. of position 4 t + c % 4 of block c / 4
            uint32_t kf[8][KS];
            uint32_t ks[8];
            {
                const size_t first = static_cast<size_t>(max(krow, 0)) + (c16 & 3);
                const uint8_t* p = k_codes + first * (D / 2) + kLane * h4;
                const uint8_t* s = k_scales + first * CB + (h4 * CB) / 4;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    if constexpr (D == 128) {
                        const u32x4 x = *reinterpret_cast<const u32x4*>(p + t * 4 * (D / 2));
#pragma unroll
                        for (int i = 0; i < 4; ++i) kf[t][i] = x[i];
                    } else {
                        const u32x2 x = *reinterpret_cast<const u32x2*>(p + t * 4 * (D / 2));
#pragma unroll
                        for (int i = 0; i < 2; ++i) kf[t][i] = x[i];
                    }
                    ks[t] = s[t * 4 * CB];
                }
            }
            // values: lane (c, h) has channel 16 t + c of block h; scales: all of block h
            u32x4 vf[DT];
            uint32_t vs[kWords];
            {
                const size_t first = max(vrow, 0);
                const uint8_t* p = v_codes + first * (D / 2) + 16 * c16;
                const u32x4* s = reinterpret_cast<const u32x4*>(v_scales + first * CB);
#pragma unroll
                for (int t = 0; t < DT; ++t) vf[t] = *reinterpret_cast<const u32x4*>(p + t * 256);
#pragma unroll
                for (int t = 0; t < kWords / 4; ++t) {
                    const u32x4 x = s[t];
#pragma unroll
                    for (int i = 0; i < 4; ++i) vs[4 * t + i] = x[i];
                }
            }

            f32x4 s[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
                // the byte 255 gives an infinite scale, which no code but 0 comes with: the scores are NaN
                const float scale = mx_float(ks[t]);
#pragma unroll
                for (int e = 0; e < KS; ++e) {
                    const bf16x8v x = mx_bf16(kf[t][e], scale);
#pragma unroll
                    for (int p = 0; p < NP; ++p) s[t] = mma16(x, qf[e][p], s[t]);
                }
            }

            // Which of its 32 positions the lane's query sees.  A hidden position's weight is
            // 0, and so is its scale: what it holds has no influence whatever it is.
            const int e0 = 4 * step + h4, first = (e0 < sp.sinks ? e0 : e0 + sp.jump) * kMxRows;
            const bool whole = vrow >= 0 && first + kMxRows - 1 <= sp.p0 &&
                               (a.window == 0 || first > sp.p1 - a.window || first + kMxRows <= a.sinks);
            if (!__all(whole)) {
                uint32_t seen = 0;
                if (vrow >= 0) {
                    const int before = min(max(pos + 1 - first, 0), 32);  // j <= pos
                    seen = before == 32 ? 0xffffffffu : (1u << before) - 1;
                    if (a.window) {
                        const int out = min(max(pos - a.window + 1 - first, 0), 32), sink = min(max(a.sinks - first, 0), 32);
                        seen &= (out == 32 ? 0u : 0xffffffffu << out) | (sink == 32 ? 0xffffffffu : (1u << sink) - 1);
                    }
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const bool see = (seen >> j) & 1;
                    if (!see) s[j >> 2][j & 3] = -INFINITY;
                    if constexpr (D == 128) {
                        if (!see) vs[j] = 0;
                    } else {
                        if (!see) vs[j >> 1] &= j & 1 ? 0xffffu : 0xffff0000u;
                    }
                }
            }

            float mx = s[0][0];
#pragma unroll
            for (int j = 1; j < 32; ++j) mx = fmaxf(mx, s[j >> 2][j & 3]);
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
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float w[8];
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    w[y] = ex2(fmaf(s[2 * i + (y >> 2)][y & 3], c, -mc));
                    l += w[y];
                }
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    float x[8];
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const int byte = (8 * i + y) * CB + cb;
                        x[y] = w[y] * mx_float((vs[byte >> 2] >> (8 * (byte & 3))) & 255u);
                    }
                    bf16x8v pf[NP];
                    split8<NP>(x, pf);
#pragma unroll
                    for (int t = 2 * cb; t < 2 * cb + 2; ++t) {
                        const bf16x8v v = mx_bf16(vf[t][i], 1.f);
#pragma unroll
                        for (int p = 0; p < NP; ++p) acc[t] = mma16(v, pf[p], acc[t]);
                    }
                }
            }
        }
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);

        // the four waves' parts, joined in LDS in wave order
        __syncthreads();
        {
            float* dst = jo + (wave * 16 + c16) * kPitch + 4 * h4;
#pragma unroll
            for (int t = 0; t < DT; ++t) *reinterpret_cast<f32x4*>(dst + 16 * t) = acc[t];
            if (h4 == 0) {
                jm[(wave * 16 + c16) * 2] = m;
                jm[(wave * 16 + c16) * 2 + 1] = l;
            }
        }
        __syncthreads();
        const int row = threadIdx.x >> 4;
        const bool whole = take == sp.steps;
        if (row < rows) {
            float mw[kMxWaves], M = -INFINITY;
#pragma unroll
            for (int x = 0; x < kMxWaves; ++x) {
                mw[x] = jm[(x * 16 + row) * 2];
                M = fmaxf(M, mw[x]);
            }
            float lt = 0.f;
#pragma unroll
            for (int x = 0; x < kMxWaves; ++x) {
                mw[x] = mw[x] == -INFINITY ? 0.f : ex2((mw[x] - M) * c);
                lt = fmaf(jm[(x * 16 + row) * 2 + 1], mw[x], lt);
            }
            const int r = ht * 16 + row, i = r / a.G;
            const size_t out = (static_cast<size_t>(b) * a.Tq + i) * a.Hq + hk * a.G + r - i * a.G;
            const float inv = lt == 0.f ? 0.f : 1.f / lt;
            // a shared unit's part: slot 1 holds its beginning, slot 0 what does not begin here
            const size_t prow = (static_cast<size_t>(blockIdx.x) * 2 + (at_block == 0)) * a.heads + row;
#pragma unroll
            for (int e = 0; e < D / 64; ++e) {
                const int d = 64 * e + 4 * (threadIdx.x & 15);
                f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int x = 0; x < kMxWaves; ++x)  // a wave without keys holds zeros; one whose weight underflows may hold a NaN
                    sum += *reinterpret_cast<const f32x4*>(jo + (x * 16 + row) * kPitch + d) * mw[x];
                if (whole)
                    store4<T>(o + out * D + d, sum[0] * inv, sum[1] * inv, sum[2] * inv, sum[3] * inv);
                else
                    *reinterpret_cast<f32x4*>(part_o + prow * D + d) = sum;
            }
            if (!whole && (threadIdx.x & 15) == 0) {
                part_ml[prow * 2] = M == -INFINITY ? M : M * c;
                part_ml[prow * 2 + 1] = lt;
            }
        }
        left -= take;
        at_block = 0;
        ++unit;
        if (left > 0) __syncthreads();  // LDS is free for the next unit
    }
}

// ---------------------------------------------------------------- append and read

// Where the tokens of a packed batch lie in the cache: token t of sequence n
// (cu[n] <= t < cu[n + 1]) is at position first[n] + t - cu[n].
struct MxPlace {
    int N, total, Hkv;
    int page_shift, num_pages, max_pages;
    int range;  // tokens that a wave looks at (at most 64)
    const int* cu;
    const int* first;  // NULL: 0 for every sequence
    const int* table;
};

// A run of tokens in one block of 32 positions of one sequence.
struct MxRun {
    int token, count, slot;  // first token, tokens, position in the block
    size_t row;              // the block's first row in the page tensors, without the head
};

// Calls f for every run that begins in this wave's range of tokens: the first
// token of a sequence, or one at the start of a block.  So no block is written
// from two places, except where sequences share a page.
template <typename F> __device__ __forceinline__ void for_runs(const MxPlace& pl, int wave_range, int lane, F f) {
    const int t = wave_range * pl.range + lane;
    bool lead = false;
    int count = 0, slot = 0;
    int row = 0;
    if (lane < pl.range && t < pl.total) {
        int s = 0;  // the last sequence that starts at or before t
        for (int hi = pl.N; hi - s > 1;) {
            const int mid = (s + hi) >> 1;
            if (pl.cu[mid] <= t)
                s = mid;
            else
                hi = mid;
        }
        const int begin = pl.cu[s], end = min(pl.cu[s + 1], pl.total), from = pl.first ? pl.first[s] : 0;
        const long long pos = static_cast<long long>(from) + (static_cast<long long>(t) - begin);
        slot = static_cast<int>(pos & (kMxRows - 1));
        if (begin >= 0 && t >= begin && t < end && from >= 0 && (pos >> pl.page_shift) < pl.max_pages &&
            (t == begin || slot == 0)) {
            const int page = pl.table[static_cast<size_t>(s) * pl.max_pages + static_cast<size_t>(pos >> pl.page_shift)];
            lead = page >= 0 && page < pl.num_pages;
            count = min(kMxRows - slot, end - t);
            row = static_cast<int>(pos & ((1 << pl.page_shift) - 1)) - slot;
            // page * Hkv rows of page_size positions; below 2^31
            row += (page * pl.Hkv) << pl.page_shift;
        }
    }
    for (uint64_t todo = __ballot(lead); todo; todo &= todo - 1) {
        const int from = __builtin_ctzll(todo);
        MxRun r;
        r.token = wave_range * pl.range + from;
        r.count = __builtin_amdgcn_readlane(count, from);
        r.slot = __builtin_amdgcn_readlane(slot, from);
        r.row = static_cast<size_t>(__builtin_amdgcn_readlane(row, from));
        f(r);
    }
}

// The largest magnitude's bits over the lanes that share a block: 32 / N lanes of N channels each.
template <int N> __device__ __forceinline__ uint32_t block_max(uint32_t x) {
#pragma unroll
    for (int s = 1; s < kMxBlock / N; s <<= 1) x = max(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), s)));
    return x;
}

// N consecutive elements as fp32.
template <int N> __device__ __forceinline__ void load_f32(const bf16_t* p, float (&x)[N]) {
    if constexpr (N == 2) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
        x[0] = __uint_as_float(u << 16);
        x[1] = __uint_as_float(u & 0xffff0000u);
    } else {
        x[0] = bf16_to_f32(*p);
    }
}
template <int N> __device__ __forceinline__ void load_f32(const float* p, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = p[i];
}

// 32 elements as fp32 (16-byte aligned).
__device__ __forceinline__ void load32(const bf16_t* p, float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const u32x4 u = *reinterpret_cast<const u32x4*>(p + 8 * i);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            x[8 * i + 2 * y] = __uint_as_float(u[y] << 16);
            x[8 * i + 2 * y + 1] = __uint_as_float(u[y] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ void load32(const float* p, float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const f32x4 u = *reinterpret_cast<const f32x4*>(p + 4 * i);
#pragma unroll
        for (int y = 0; y < 4; ++y) x[4 * i + y] = u[y];
    }
}

// Append: a wave per (range of tokens, head).  Keys: a lane quantises 32 channels
// of a position by itself.  Values: a lane has 1 or 2 channels and goes through
// the positions, so that it ends with the 16 bytes of its channels; a block that
// the run covers in part keeps its other positions.
template <typename T, int D>
__global__ __launch_bounds__(256) void mx4_append_kernel(MxPlace pl, FastDiv heads, int waves, const T* __restrict__ k,
                                                         const T* __restrict__ v, uint8_t* __restrict__ k_codes,
                                                         uint8_t* __restrict__ k_scales, uint8_t* __restrict__ v_codes,
                                                         uint8_t* __restrict__ v_scales) {
    constexpr int CB = D / 32, N = D / 64;
    const int lane = threadIdx.x & 63, id = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    if (id >= waves) return;
    const int range = heads(id), hk = id - range * heads.d;
    for_runs(pl, range, lane, [&](const MxRun& r) {
        const size_t row = r.row + (static_cast<size_t>(hk) << pl.page_shift);
        const size_t stride = static_cast<size_t>(pl.Hkv) * D;
        const size_t from = static_cast<size_t>(r.token) * stride + static_cast<size_t>(hk) * D;
        // keys
#pragma unroll 1
        for (int j = lane / CB; j < r.count; j += 64 / CB) {
            const int cb = lane % CB;
            float x[32];
            load32(k + from + j * stride + 32 * cb, x);
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) top = max(top, magnitude(x[i]));
            const uint32_t e = mx_scale(top);
            const float inv = mx_inverse(e);
            u32x4 w = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = mx_put<0>(w[i], x[8 * i] * inv, x[8 * i + 1] * inv);
                w[i] = mx_put<1>(w[i], x[8 * i + 2] * inv, x[8 * i + 3] * inv);
                w[i] = mx_put<2>(w[i], x[8 * i + 4] * inv, x[8 * i + 5] * inv);
                w[i] = mx_put<3>(w[i], x[8 * i + 6] * inv, x[8 * i + 7] * inv);
                if (e == kMxNan) w[i] = 0;
            }
            const size_t to = row + r.slot + j;
            *reinterpret_cast<u32x4*>(k_codes + to * (D / 2) + 16 * cb) = w;
            k_scales[to * CB + cb] = static_cast<uint8_t>(e);
        }
        // values
        u32x4* at = reinterpret_cast<u32x4*>(v_codes + row * (D / 2) + static_cast<size_t>(lane) * N * 16);
        u32x4 w[N];
#pragma unroll
        for (int n = 0; n < N; ++n) w[n] = r.count < kMxRows ? at[n] : u32x4{0, 0, 0, 0};
        const int sub = lane % (kMxBlock / N);  // of the lanes of a block of channels
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[8][N];
#pragma unroll
            for (int y = 0; y < 8; ++y) {  // positions outside the run repeat its first or last
                const int j = min(max(8 * i + y - r.slot, 0), r.count - 1);
                load_f32<N>(v + from + j * stride + lane * N, x[y]);
            }
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const int j = 8 * i + y;
                uint32_t top = magnitude(x[y][0]);
                if constexpr (N == 2) top = max(top, magnitude(x[y][1]));
                const uint32_t e = mx_scale(block_max<N>(top));
                const float inv = mx_inverse(e);
                uint32_t code = mx_put<0>(0, x[y][0] * inv, x[y][N - 1] * inv);  // a channel a half
                if (e == kMxNan) code = 0;
                if (j >= r.slot && j < r.slot + r.count) {
                    const uint32_t keep = ~(15u << (4 * y));
                    w[0][i] = (w[0][i] & keep) | ((code & 15u) << (4 * y));
                    if constexpr (N == 2) w[1][i] = (w[1][i] & keep) | ((code >> 4) << (4 * y));
                    if (sub == j % (kMxBlock / N)) v_scales[(row + j) * CB + lane * N / kMxBlock] = static_cast<uint8_t>(e);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n) at[n] = w[n];
    });
}

__device__ __forceinline__ void store_f32(bf16_t* p, float a, float b) {
    *reinterpret_cast<uint32_t*>(p) = f32_to_bf16(a) | static_cast<uint32_t>(f32_to_bf16(b)) << 16;
}
__device__ __forceinline__ void store_f32(float* p, float a, float b) {
    p[0] = a;
    p[1] = b;
}

// Code c (4 bits) times the scale of byte b; NaN where b is 255.
__device__ __forceinline__ float mx_value(uint32_t c, uint32_t b) {
    typedef float f32x2v __attribute__((ext_vector_type(2)));
    const f32x2v x = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 0);
    return b == kMxNan ? NAN : x[0] * mx_float(b);
}

// Read: the same runs, the other way.  Every value is exact in both types.
template <typename T, int D>
__global__ __launch_bounds__(256) void mx4_read_kernel(MxPlace pl, FastDiv heads, int waves,
                                                       const uint8_t* __restrict__ k_codes,
                                                       const uint8_t* __restrict__ k_scales,
                                                       const uint8_t* __restrict__ v_codes,
                                                       const uint8_t* __restrict__ v_scales, T* __restrict__ k,
                                                       T* __restrict__ v) {
    constexpr int CB = D / 32, N = D / 64;
    const int lane = threadIdx.x & 63, id = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    if (id >= waves) return;
    const int range = heads(id), hk = id - range * heads.d;
    for_runs(pl, range, lane, [&](const MxRun& r) {
        const size_t row = r.row + (static_cast<size_t>(hk) << pl.page_shift);
        const size_t stride = static_cast<size_t>(pl.Hkv) * D;
        const size_t to = static_cast<size_t>(r.token) * stride + static_cast<size_t>(hk) * D;
        // keys
#pragma unroll 1
        for (int j = lane / CB; j < r.count; j += 64 / CB) {
            const int cb = lane % CB;
            const size_t from = row + r.slot + j;
            const u32x4 w = *reinterpret_cast<const u32x4*>(k_codes + from * (D / 2) + 16 * cb);
            const uint32_t e = k_scales[from * CB + cb];
            T* p = k + to + j * stride + 32 * cb;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float x[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) x[y] = mx_value((w[i >> 1] >> (16 * (i & 1) + 4 * y)) & 15u, e);
                store4<T>(p + 4 * i, x[0], x[1], x[2], x[3]);
            }
        }
        // values
        const u32x4* at = reinterpret_cast<const u32x4*>(v_codes + row * (D / 2) + static_cast<size_t>(lane) * N * 16);
        u32x4 w[N];
#pragma unroll
        for (int n = 0; n < N; ++n) w[n] = at[n];
#pragma unroll
        for (int j = 0; j < kMxRows; ++j) {
            if (j < r.slot || j >= r.slot + r.count) continue;
            const uint32_t e = v_scales[(row + j) * CB + lane * N / kMxBlock];
            const float a = mx_value((w[0][j >> 3] >> (4 * (j & 7))) & 15u, e);
            T* p = v + to + (j - r.slot) * stride + lane * N;
            if constexpr (N == 2)
                store_f32(p, a, mx_value((w[1][j >> 3] >> (4 * (j & 7))) & 15u, e));
            else
                Elem<T>::store(p, a);
        }
    });
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

MxPlace place_of(int N, int total, int Hkv, int page_size, int num_pages, int max_pages, const int* cu, const int* first,
                 const int* table, unsigned long long& waves) {
    MxPlace pl{N, total, Hkv, log2_of(page_size), num_pages, max_pages, 32, cu, first, table};
    waves = (static_cast<unsigned long long>(total) + pl.range - 1) / pl.range * Hkv;
    return pl;
}

int mx4_shares(int page_size, int max_pages, int window, int sinks, int Tq) {
    long long keys = static_cast<long long>(max_pages) * page_size;
    if (window && keys > static_cast<long long>(window) + Tq + sinks) keys = static_cast<long long>(window) + Tq + sinks;
    return keys <= 512 ? 0 : 512;
}

Mx4Args mx4_args(int B, int Tq, int Hq, int Hkv, int page_size, int num_pages, int max_pages, int window, int sinks,
                 float scale) {
    Mx4Args a{};
    a.B = B;
    a.Tq = Tq;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.head_tiles = (Tq * a.G + 15) / 16;
    a.page_shift = log2_of(page_size);
    a.num_pages = num_pages;
    a.max_pages = max_pages;
    a.window = window;
    a.sinks = sinks;
    a.scale = scale;
    a.shares = mx4_shares(page_size, max_pages, window, sinks, Tq);
    a.heads = Tq * a.G < 16 ? Tq * a.G : 16;
    return a;
}

template <typename T, int D>
hipError_t launch_mx4_decode_t(const Mx4Args& a, const void* q, const void* k_codes, const void* k_scales,
                               const void* v_codes, const void* v_scales, const int* table, const int* lengths, void* o,
                               float* ws, hipStream_t st) {
    const unsigned long long rows = static_cast<unsigned long long>(a.B) * a.Tq * a.Hq;
    const unsigned long long most = (static_cast<unsigned long long>(a.max_pages) << a.page_shift) / kQuad + 2;
    return launch_dealt<T, D>(a, rows, most, 64 * kMxWaves, table, lengths, o, ws, st,
                              [&](unsigned blocks, float* part_o, float* part_ml) {
                                  hipLaunchKernelGGL((mx4_decode_kernel<T, D>), dim3(blocks), dim3(64 * kMxWaves), 0, st, a,
                                                     static_cast<const T*>(q), static_cast<const uint8_t*>(k_codes),
                                                     static_cast<const uint8_t*>(k_scales),
                                                     static_cast<const uint8_t*>(v_codes),
                                                     static_cast<const uint8_t*>(v_scales), table, lengths,
                                                     static_cast<T*>(o), part_o, part_ml);
                                  return hipGetLastError();
                              });
}

}  // namespace
}  // namespace attn

size_t attn_decode_mx4_workspace_floats(int Tq, int Hq, int Hkv, int d, int page_size, int max_pages, int window, int sinks) {
    return attn::part_floats(attn::mx4_args(1, Tq, Hq, Hkv, page_size, 0, max_pages, window, sinks, 1.f), d);
}

hipError_t launch_attn_decode_mx4(int dtype, int B, int Tq, int Hq, int Hkv, int d, int page_size, int num_pages,
                                  int max_pages, int window, int sinks, float scale, const void* q, const void* k_codes,
                                  const void* k_scales, const void* v_codes, const void* v_scales, const int* table,
                                  const int* lengths, void* o, float* ws, hipStream_t st) {
    const attn::Mx4Args a = attn::mx4_args(B, Tq, Hq, Hkv, page_size, num_pages, max_pages, window, sinks, scale);
    auto* f = dtype == GDR_DTYPE_F32
                  ? (d == 64 ? attn::launch_mx4_decode_t<float, 64> : attn::launch_mx4_decode_t<float, 128>)
                  : (d == 64 ? attn::launch_mx4_decode_t<bf16_t, 64> : attn::launch_mx4_decode_t<bf16_t, 128>);
    return f(a, q, k_codes, k_scales, v_codes, v_scales, table, lengths, o, ws, st);
}

hipError_t launch_attn_append_mx4(int dtype, int N, int total, int Hkv, int d, int page_size, int num_pages, int max_pages,
                                  const void* k, const void* v, const int* cu, const int* lengths, void* k_codes,
                                  void* k_scales, void* v_codes, void* v_scales, const int* table, hipStream_t st) {
    unsigned long long waves;
    const attn::MxPlace pl = attn::place_of(N, total, Hkv, page_size, num_pages, max_pages, cu, lengths, table, waves);
    const unsigned long long blocks = (waves + 3) / 4;
    if (!grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
    auto go = [&](auto t, auto dd) {
        using T = decltype(t);
        hipLaunchKernelGGL((attn::mx4_append_kernel<T, decltype(dd)::value>), dim3(static_cast<unsigned>(blocks)), dim3(256),
                           0, st, pl, attn::FastDiv(Hkv), static_cast<int>(waves), static_cast<const T*>(k),
                           static_cast<const T*>(v), static_cast<uint8_t*>(k_codes), static_cast<uint8_t*>(k_scales),
                           static_cast<uint8_t*>(v_codes), static_cast<uint8_t*>(v_scales));
        return hipGetLastError();
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    return dtype == GDR_DTYPE_F32 ? (d == 64 ? go(float(), D64()) : go(float(), D128()))
                                  : (d == 64 ? go(bf16_t(), D64()) : go(bf16_t(), D128()));
}

hipError_t launch_attn_read_mx4(int dtype, int N, int total, int Hkv, int d, int page_size, int num_pages, int max_pages,
                                const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                                const int* table, const int* cu, const int* first, void* k, void* v, hipStream_t st) {
    unsigned long long waves;
    const attn::MxPlace pl = attn::place_of(N, total, Hkv, page_size, num_pages, max_pages, cu, first, table, waves);
    const unsigned long long blocks = (waves + 3) / 4;
    if (!grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
    auto go = [&](auto t, auto dd) {
        using T = decltype(t);
        hipLaunchKernelGGL((attn::mx4_read_kernel<T, decltype(dd)::value>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                           st, pl, attn::FastDiv(Hkv), static_cast<int>(waves), static_cast<const uint8_t*>(k_codes),
                           static_cast<const uint8_t*>(k_scales), static_cast<const uint8_t*>(v_codes),
                           static_cast<const uint8_t*>(v_scales), static_cast<T*>(k), static_cast<T*>(v));
        return hipGetLastError();
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    return dtype == GDR_DTYPE_F32 ? (d == 64 ? go(float(), D64()) : go(float(), D128()))
                                  : (d == 64 ? go(bf16_t(), D64()) : go(bf16_t(), D128()));
}

}  // namespace gdr
