// Attention over a key-value cache held in 4 bits: the append of new tokens, their
// way back to dense tensors, and the decode step.
//
// The format of a block is attn_mx4.h's.  Keys lie row by row, a position's d / 2
// bytes together; values lie in blocks of 32 positions, the 16 bytes of a channel
// together, so that both products of the decode step find their operands' bytes as
// they want them: a lane of the score product takes consecutive channels of a key,
// a lane of the output product consecutive positions of a channel.  The values are
// transposed once, by the append.  Scales lie position by position.
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
// A unit's steps are dealt out as if it had four more at its beginning: its first
// loads wait for one another (length, page, keys) for as long as four waves take for
// a step each.  64 sequences of 16 .. 8000 tokens, whose shortest come in dozens to a
// workgroup: 83 us without, 61 with (2: 67, 6 and 8: 61 and 62).
constexpr int kUnitCost = 4;

// At query position p a key j is visible if j <= p and (window == 0 or j > p - window or j < sinks).
struct Mx4Args {
    int B, Tq, Hq, Hkv, G, head_tiles;
    int page_shift, num_pages, max_pages;
    int window, sinks;
    float scale;
    int shares;  // workgroups the blocks are dealt to; 0: units that are not shared
    bool alone;  // a wave for each unit, else a workgroup (shares == 0)
    int heads;   // rows of a unit: min(16, Tq * G)
    FastDiv by_group, by_tiles;  // by G and by head_tiles

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
    int entries, steps; // steps of four entries and kUnitCost; 0: the length is out of range
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
    s.steps = fits ? (s.entries + 3) / 4 + kUnitCost : 0;
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

// 8 elements of a query as operands, with the sign turned.  An infinity goes in as NaN (the
// pieces of one are): where the keys are negative its scores would all be -inf, as hidden keys'
// are.
__device__ __forceinline__ void query8(const f32x8& q, bool turned, bf16x8v (&to)[3]) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = turned ? -q[i] : q[i];
    split8<3>(f, to);
}
__device__ __forceinline__ void query8(const bf16x8v& q, bool turned, bf16x8v (&to)[1]) {
    u32x4 w = __builtin_bit_cast(u32x4, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // an exponent of ones gets a mantissa
        w[i] |= ((w[i] & 0x7fff7fffu) + 0x00800080u) >> 15 & 0x00010001u;
        w[i] ^= turned ? 0x80008000u : 0u;
    }
    to[0] = __builtin_bit_cast(bf16x8v, w);
}

// LDS of the decode step: for each wave the keys, values and scales of one step.
// Keys are read 16 (d = 64: 8) bytes a lane, four positions of each of the four
// blocks at a time.  d = 128: odd blocks have their 16-byte units swapped in
// pairs; d = 64: these too, and the blocks 2 and 3 lie 128 bytes further.  Either
// way the lanes that share a cycle read different banks.
template <int D> struct Mx4Lds {
    static constexpr int kBlock = kMxRows * D / 2;  // bytes of a block's codes
    static constexpr int kScales = kMxRows * D / 32;
    static constexpr int kGap = D == 64 ? 128 : 0;
    static constexpr int kValues = 4 * kBlock + kGap, kKeyScales = kValues + 4 * kBlock;
    static constexpr int kValueScales = kKeyScales + 4 * kScales;
    static constexpr int kWave = kValueScales + 4 * kScales;
    static constexpr int kPitch = D + 4;  // floats of a joined row
    static constexpr int kJoin = kMxWaves * 16 * (kPitch + 2) * 4;
    static constexpr int kBytes = kMxWaves * kWave > kJoin ? kMxWaves * kWave : kJoin;
    static constexpr int kKeyCopies = 4 * kBlock / 1024, kScaleCopies = 4 * kScales / 256;
    __device__ __forceinline__ static int keys(int block) { return block * kBlock + (block >> 1) * kGap; }
};

// At most n of this wave's latest loads and copies are still on their way.
template <int N> __device__ __forceinline__ void mx4_wait() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
}
// This wave's LDS reads have returned: what they read may be overwritten.
__device__ __forceinline__ void mx4_wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);
    asm volatile("" ::: "memory");
}
// Copies to LDS, base + off in memory: 16 bytes a lane, not to be kept in the
// caches, or 4.
__device__ __forceinline__ void mx4_copy16(uint32_t lds, const void* base, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(lds), "v"(off), "s"(base)
                 : "memory");
}

// v in the lanes where `mine` holds, else zero.
__device__ __forceinline__ bf16x8v of_copy(const bf16x8v& v, bool mine) {
    const u32x4 u = __builtin_bit_cast(u32x4, v);
    return __builtin_bit_cast(bf16x8v, u32x4{mine ? u[0] : 0u, mine ? u[1] : 0u, mine ? u[2] : 0u, mine ? u[3] : 0u});
}
// v as a value the compiler knows nothing about: it is kept, not formed again.
__device__ __forceinline__ bf16x8v kept(const bf16x8v& v) {
    u32x4 u = __builtin_bit_cast(u32x4, v);
    asm volatile("" : "+v"(u));
    return __builtin_bit_cast(bf16x8v, u);
}
// The sum or maximum over the X copies of a row (16 / X lanes apart in its 16), and
// over the four blocks (the lanes 16 and 32 apart), in every lane.
template <int N> __device__ __forceinline__ float rotated(float v) {  // of the lane N further in its 16
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xf, 0xf, true));
}
template <int X, typename F> __device__ __forceinline__ float over_copies(float v, F f) {
    if constexpr (X == 4) v = f(v, rotated<4>(v));
    if constexpr (X >= 2) v = f(v, rotated<8>(v));
    return v;
}
template <typename F> __device__ __forceinline__ float over_blocks(float v, F f) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
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
// A unit of few rows leaves most of the 16 columns idle, and with them most of the
// lanes' softmax.  So there are X = 4 copies of up to 4 rows, or 2 of up to 8: copy x
// takes positions 32 x / X .. of each block.  Of the keys' tiles each meets the query
// in its own copy's columns only, zero in the others, so that X tiles share an
// accumulator, and a lane has 32 / X positions; of the weights each product takes
// one copy's, and the copies' sums are added at the end.  (The code of a step as
// compiled for d = 128, masks and the path of NaN bytes among it: 967 vector
// instructions with X = 1, 896 with 2, 687 with 4; fp32 1671.)
//
// The keys' scales are applied by the conversion to bf16, which is exact.  The
// values' scales differ along the summed axis and are multiplied into the weights:
// one set of weights for every 32 channels.  bf16: the weights are rounded to bf16
// after the power of two, which is the same as before it.  (A second piece of them
// would bring the output's error from 2.0e-3 to 1.65e-3, that of exact weights, and
// take 62 us instead of 59 for 64 sequences of 16 .. 8000, 53 instead of 42 with 16
// rows of 16 .. 4000; the codes themselves stand for values within 11%.)  fp32: queries and
// weights go in as three bf16 pieces, 24 bits, and no bit of the codes is lost.
// Either holds while a weight times the power of two, or its last piece, stays above
// 2^-126; what falls below is an absolute error of that size (values of 2^-100 and
// more show nothing of it).
//
// A unit's steps go to the four waves of a workgroup in turn, joined in LDS, or all
// to one wave (see mx4_args).
//
// Bound by HBM: 64 sequences of 16 .. 8000 tokens, 32 heads over 8, d = 128 (280 MB)
// 54 us and 5 for the join, 5.2 TB/s; one of 32768 14.7 + 4.3.  The vector ALUs are
// busy for 30% of it, the matrix cores for 10% (fp32: 98 us, 52% and 22%).  Everything that is read
// goes through LDS, straight from memory in whole lines: fetched into the registers
// of the lanes that need it, each line of the keys and scales is asked for by
// several of them while it is on its way, and the L1 cache stalls on that (89 us
// with the loads a step ahead in registers, where this took 63).  Keys are refilled
// as soon as the scores are formed, values as soon as they are in registers, no
// barrier until the end.
template <typename T, int D, int X, bool kAlone>
__global__ __launch_bounds__(64 * kMxWaves, 2) void mx4_decode_kernel(
    Mx4Args a, const T* __restrict__ q, const uint8_t* __restrict__ k_codes, const uint8_t* __restrict__ k_scales,
    const uint8_t* __restrict__ v_codes, const uint8_t* __restrict__ v_scales, const int* __restrict__ table,
    const int* __restrict__ lengths, T* __restrict__ o, float* __restrict__ part_o, float* __restrict__ part_ml) {
    using C = Mx4Lds<D>;
    constexpr int NP = Pieces<T>::n, KS = D / 32, DT = D / 16, CB = D / 32, kPitch = C::kPitch;
    constexpr int kCopies = C::kKeyCopies + C::kScaleCopies;  // of a step's keys, and of its values
    constexpr int kRows = 16 / X, kMine = 32 / X;              // rows of a unit; positions of a lane in each block
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c16 = lane & 15, h4 = lane >> 4, x = c16 / kRows;
    const int per = a.per(), slot_mask = (1 << a.page_shift) - 1;
    // a scale of 0 as one that no score survives: c -inf of a hidden key stays -inf
    const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-37f);
    unsigned char* mine_lds = smem + wave * C::kWave;
    const uint32_t lds_at = lds_addr(mine_lds);
    // where this lane reads its keys, their scales, its values and theirs
    const unsigned char* kp = mine_lds + C::keys(c16 >> 2) + (c16 & 3) * (D / 2) +
                              (D == 128 ? 16 * (h4 ^ ((c16 >> 2) & 1)) : 8 * (h4 ^ (((c16 >> 2) & 1) << 1)));
    const unsigned char* ksp = mine_lds + C::kKeyScales + (c16 >> 2) * C::kScales + (c16 & 3) * CB + (h4 * CB) / 4;
    const unsigned char* vp = mine_lds + C::kValues + h4 * C::kBlock + 16 * c16;
    const unsigned char* vsp = mine_lds + C::kValueScales + h4 * C::kScales + x * kMine * CB;
    // and the unit it copies, from the start of 1024 bytes of keys: even and odd blocks
    const uint32_t unit = 16 * lane, swapped = 16 * (lane ^ 1);

    constexpr int kStride = kAlone ? 1 : kMxWaves;
    const int id = kAlone ? blockIdx.x * kMxWaves + wave : blockIdx.x;
    if (kAlone && id >= a.B * per) return;
    Share share;
    if (!find_share(a, lengths, lane, id, share)) return;
    int b = share.b, unit_at = share.unit, at_block = share.at_block, left = share.left;
    MxSpan sp = mx_span(a, share.len);

#pragma unroll 1
    while (left > 0) {
        if (unit_at >= per || sp.steps == 0) {  // the next sequence that is not skipped
            if (++b >= a.B) return;
            unit_at = 0;
            sp = mx_span(a, __builtin_amdgcn_readfirstlane(lengths[b]));
            continue;
        }
        const int take = min(left, sp.steps - at_block);
        const int hk = __builtin_amdgcn_readfirstlane(a.by_tiles(unit_at)), ht = unit_at - hk * a.head_tiles;
        // the table does not change under the call: scalar loads, counted apart from the copies
        typedef const int __attribute__((address_space(4))) * ConstInts;
        const ConstInts trow = (ConstInts)(table + static_cast<size_t>(b) * a.max_pages);

        // this lane's query row: query i, head g of the group
        const int rows = min(16, a.Tq * a.G - ht * 16);
        const int mine = ht * 16 + min(c16 % kRows, rows - 1), qi = a.by_group(mine);
        const int pos = sp.p0 + qi;
        const size_t orow = (static_cast<size_t>(b) * a.Tq + qi) * a.Hq + hk * a.G + mine - qi * a.G;

        // Entry e of the list: its first position; and from the page there the row of its
        // first position in the page tensors, or -1 where there is none (past the list, or
        // on a page outside the pool).
        auto start_of = [&](int e) { return (e < sp.sinks ? e : e + sp.jump) * kMxRows; };
        auto page_of = [&](int e) { return trow[start_of(max(min(e, sp.entries - 1), 0)) >> a.page_shift]; };
        auto row_of = [&](int e, int page) {
            if (e >= sp.entries || page < 0 || page >= a.num_pages) return -1;
            return ((page * a.Hkv + hk) << a.page_shift) + (start_of(e) & slot_mask);
        };
        auto copy_scales = [&](uint32_t lds, const uint8_t* scales, const int (&row)[4]) {  // 256 bytes at a time
            constexpr int kEach = 256 / C::kScales;  // blocks of a copy
#pragma unroll
            for (int j = 0; j < C::kScaleCopies; ++j) {
                int r = row[kEach * j];
#pragma unroll
                for (int x = 1; x < kEach; ++x)
                    if (lane >= x * (64 / kEach)) r = row[kEach * j + x];
                const size_t from = static_cast<size_t>(max(r, 0)) * CB + 4 * (lane & (64 / kEach - 1));
                gather_words(lds + 256 * j, scales + from);
            }
        };
        auto copy_keys = [&](const int (&row)[4]) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint8_t* p = k_codes + static_cast<size_t>(max(row[x], 0)) * (D / 2);
#pragma unroll
                for (int j = 0; j < C::kBlock / 1024; ++j)
                    mx4_copy16(lds_at + C::keys(x) + 1024 * j, p + 1024 * j, x & 1 ? swapped : unit);
            }
            copy_scales(lds_at + C::kKeyScales, k_scales, row);
        };
        auto copy_values = [&](const int (&row)[4]) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint8_t* p = v_codes + static_cast<size_t>(max(row[x], 0)) * (D / 2);
#pragma unroll
                for (int j = 0; j < C::kBlock / 1024; ++j)
                    mx4_copy16(lds_at + C::kValues + C::kBlock * x + 1024 * j, p + 1024 * j, unit);
            }
            copy_scales(lds_at + C::kValueScales, v_scales, row);
        };

        // The query and the pages of two steps come together, then the first copies.
        const int end = max(0, at_block + take - kUnitCost);
        int step = max(0, at_block - kUnitCost) + (kAlone ? 0 : wave), row[4], page[4], next[4];
        bf16x8v qf[X][KS][NP];  // copy by copy: the others' columns are zero
        {
            const T* qp = q + orow * D + (D / 4) * h4;
            frag_t<T> raw[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) raw[s] = load8(qp + 8 * s);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                page[x] = page_of(4 * step + x);
                next[x] = page_of(4 * (step + kStride) + x);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                row[x] = row_of(4 * step + x, page[x]);
                page[x] = next[x];
            }
            if (step < end) {
                copy_keys(row);
                copy_values(row);
            }
            // (waiting for the query, the compiler waits for the copies too, once a unit)
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                bf16x8v f[NP];
                query8(raw[s], a.scale < 0.f, f);
#pragma unroll
                for (int y = 0; y < X; ++y) {
#pragma unroll
                    for (int p = 0; p < NP; ++p) qf[y][s][p] = X > 1 ? kept(of_copy(f[p], x == y)) : f[p];
                }
            }
        }

        f32x4 acc[DT];
#pragma unroll
        for (int t = 0; t < DT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, l = 0.f;

#pragma unroll 1
        for (; step < end; step += kStride) {
            const bool more = step + kStride < end;
            int shown = 0;  // blocks that exist
#pragma unroll
            for (int x = 0; x < 4; ++x) shown |= (row[x] >= 0) << x;
            mx4_wait<kCopies>();  // the keys; the values may still come
            // The byte 255 gives an infinite scale, which no code but 0 comes with: the scores are
            // NaN.  253 and 254, which nothing but an unwritten slot holds, times a code leave the
            // range of bf16.  Where tiles share an accumulator such a key would reach the other
            // copies' scores too, as infinity times their zeros: it goes in with a finite scale,
            // and its own score is set afterwards, to NaN unless the position is hidden.
            uint32_t kb[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) kb[t] = ksp[t * 4 * CB];
            bool odd = false;
            if constexpr (X > 1) {
                uint32_t top = 0;
#pragma unroll
                for (int t = 0; t < 8; ++t) top = max(top, kb[t]);
                odd = __any(top > kMxMost);
                if (odd) {
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        if (kb[t] > kMxMost) kb[t] = 1;
                }
            }
            f32x4 s[8 / X];
#pragma unroll
            for (int j = 0; j < 8 / X; ++j) {
                s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int y = 0; y < X; ++y) {
                    const int t = y * (8 / X) + j;
                    uint32_t k[KS];
                    if constexpr (D == 128) {
                        const u32x4 u = *reinterpret_cast<const u32x4*>(kp + t * 4 * (D / 2));
#pragma unroll
                        for (int i = 0; i < 4; ++i) k[i] = u[i];
                    } else {
                        const u32x2 u = *reinterpret_cast<const u32x2*>(kp + t * 4 * (D / 2));
#pragma unroll
                        for (int i = 0; i < 2; ++i) k[i] = u[i];
                    }
                    const float scale = mx_float(kb[t]);
#pragma unroll
                    for (int e = 0; e < KS; ++e) {
                        const bf16x8v kv = mx_bf16(k[e], scale);
#pragma unroll
                        for (int p = 0; p < NP; ++p) s[j] = mma16(kv, qf[y][e][p], s[j]);
                    }
                }
            }
            if (odd) {
                const unsigned char* own = mine_lds + C::kKeyScales + h4 * C::kScales + x * kMine * CB;
#pragma unroll
                for (int j = 0; j < kMine; ++j) {
                    bool nan = false;
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) nan |= own[j * CB + cb] > kMxMost;
                    if (nan) s[j >> 2][j & 3] = NAN;
                }
            }
            if (more) {
#pragma unroll
                for (int x = 0; x < 4; ++x) row[x] = row_of(4 * (step + kStride) + x, page[x]);
#pragma unroll
                for (int x = 0; x < 4; ++x) page[x] = page_of(4 * (step + 2 * kStride) + x);
                mx4_wait_lds();
                copy_keys(row);
            }

            // Which of its 32 positions the lane's query sees.  A hidden position's weight is
            // 0, and so is its scale: what it holds has no influence whatever it is.
            const int first = start_of(4 * step + h4);
            const bool exists = (shown >> h4) & 1;
            const bool whole = exists && first + kMxRows - 1 <= sp.p0 &&
                               (a.window == 0 || first > sp.p1 - a.window || first + kMxRows <= a.sinks);
            const bool all = __all(whole);
            uint32_t seen = 0xffffffffu;
            if (!all) {
                const int before = min(max(pos + 1 - first, 0), 32);  // j <= pos
                seen = before == 32 ? 0xffffffffu : (1u << before) - 1;
                if (a.window) {
                    const int out = min(max(pos - a.window + 1 - first, 0), 32), sink = min(max(a.sinks - first, 0), 32);
                    seen &= (out == 32 ? 0u : 0xffffffffu << out) | (sink == 32 ? 0xffffffffu : (1u << sink) - 1);
                }
                if (!exists) seen = 0;
                seen >>= x * kMine;
#pragma unroll
                for (int j = 0; j < kMine; ++j)
                    if (!((seen >> j) & 1)) s[j >> 2][j & 3] = -INFINITY;
            }

            float mx = s[0][0];
#pragma unroll
            for (int j = 1; j < kMine; ++j) mx = fmaxf(mx, s[j >> 2][j & 3]);
            auto larger = [](float u, float v) { return fmaxf(u, v); };
            mx = fmaxf(m, over_blocks(over_copies<X>(mx, larger), larger));
            const float mc = mx == -INFINITY ? 0.f : mx * c;
            if (__any(mx > m)) {
                const float alpha = m == -INFINITY ? 0.f : ex2(m * c - mc);
                l *= alpha;
#pragma unroll
                for (int t = 0; t < DT; ++t) acc[t] *= alpha;
                m = mx;
            }
            if (more)
                mx4_wait<kCopies>();  // the values; the next keys may still come
            else
                mx4_wait<0>();
            u32x4 vf[DT], vs[kMine * CB / 16];
#pragma unroll
            for (int t = 0; t < kMine * CB / 16; ++t) vs[t] = *reinterpret_cast<const u32x4*>(vsp + 16 * t);
#pragma unroll
            for (int t = 0; t < DT; ++t) vf[t] = *reinterpret_cast<const u32x4*>(vp + 256 * t);
            if (!all) {
#pragma unroll
                for (int j = 0; j < kMine; ++j) {  // 4 positions to 16 bytes (d = 64: 8)
                    if (!((seen >> j) & 1)) vs[j * CB >> 4][(j * CB >> 2) & 3] &= D == 128 ? 0u : j & 1 ? 0xffffu : 0xffff0000u;
                }
            }
            if (more) {
                mx4_wait_lds();
                copy_values(row);
            }
#pragma unroll
            for (int i = 0; i < 4 / X; ++i) {  // 8 of this lane's positions
                __builtin_amdgcn_sched_barrier(0);
                float w[8];
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    w[y] = ex2(fmaf(s[2 * i + (y >> 2)][y & 3], c, -mc));
                    l += w[y];
                }
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    float f[8];
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const int byte = (8 * i + y) * CB + cb;
                        f[y] = w[y] * mx_float(vs[byte >> 4][(byte >> 2) & 3], byte & 3);
                    }
                    bf16x8v pf[NP];
                    split8<NP>(f, pf);
#pragma unroll
                    for (int y = 0; y < X; ++y) {
                        bf16x8v py[NP];
#pragma unroll
                        for (int p = 0; p < NP; ++p) py[p] = X > 1 ? of_copy(pf[p], x == y) : pf[p];
#pragma unroll
                        for (int t = 2 * cb; t < 2 * cb + 2; ++t) {
                            const bf16x8v v = mx_bf16(vf[t][y * (4 / X) + i], 1.f);
#pragma unroll
                            for (int p = 0; p < NP; ++p) acc[t] = mma16(v, py[p], acc[t]);
                        }
                    }
                }
            }
        }
        auto plus = [](float u, float v) { return u + v; };
        l = over_blocks(over_copies<X>(l, plus), plus);
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[t][r] = over_copies<X>(acc[t][r], plus);

        if constexpr (kAlone) {  // the wave's only unit
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (c16 < rows) {  // one of the copies, which are alike now
#pragma unroll
                for (int t = 0; t < DT; ++t)
                    store4<T>(o + orow * D + 16 * t + 4 * h4, acc[t][0] * inv, acc[t][1] * inv, acc[t][2] * inv, acc[t][3] * inv);
            }
            return;
        }

        // the four waves' parts, joined in LDS in wave order
        __syncthreads();
        float* jo = reinterpret_cast<float*>(smem);
        float* jm = jo + kMxWaves * 16 * kPitch;
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
        const int mr = threadIdx.x >> 4;
        const bool whole = take == sp.steps;
        if (mr < rows) {
            float mw[kMxWaves], M = -INFINITY;
#pragma unroll
            for (int x = 0; x < kMxWaves; ++x) {
                mw[x] = jm[(x * 16 + mr) * 2];
                M = fmaxf(M, mw[x]);
            }
            float lt = 0.f;
#pragma unroll
            for (int x = 0; x < kMxWaves; ++x) {
                mw[x] = mw[x] == -INFINITY ? 0.f : ex2((mw[x] - M) * c);
                lt = fmaf(jm[(x * 16 + mr) * 2 + 1], mw[x], lt);
            }
            const int r = ht * 16 + mr, i = a.by_group(r);
            const size_t out = (static_cast<size_t>(b) * a.Tq + i) * a.Hq + hk * a.G + r - i * a.G;
            const float inv = lt == 0.f ? 0.f : 1.f / lt;
            // a shared unit's part: slot 1 holds its beginning, slot 0 what does not begin here
            const size_t prow = (static_cast<size_t>(blockIdx.x) * 2 + (at_block == 0)) * a.heads + mr;
#pragma unroll
            for (int e = 0; e < D / 64; ++e) {
                const int d = 64 * e + 4 * (threadIdx.x & 15);
                f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int x = 0; x < kMxWaves; ++x)  // a wave without keys holds zeros; one whose weight underflows may hold a NaN
                    sum += *reinterpret_cast<const f32x4*>(jo + (x * 16 + mr) * kPitch + d) * mw[x];
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
        ++unit_at;
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
    const int t0 = wave_range * pl.range, t = t0 + lane;
    bool lead = false;
    int count = 0, slot = 0;
    int row = 0;
    // The last sequence that starts at or before t0: 64 of the offsets at a time, then
    // what is left between two of them.
    int s0 = 0;
    for (int n = pl.N; n > 0;) {
        const int step = (n - 1) / 64 + 1, at = lane * step;
        const uint64_t upto = __ballot(at < n && pl.cu[s0 + min(at, n - 1)] <= t0);
        const int k = max((upto == ~0ull ? 64 : __builtin_ctzll(~upto)) - 1, 0);
        s0 += k * step;
        n = step == 1 ? 0 : min(step, n - k * step);
    }
    if (lane < pl.range && t < pl.total) {
        // few sequences begin within a range, but many without tokens may lie between two that have some
        int s = s0;
        for (int near = 0; s + 1 < pl.N && pl.cu[s + 1] <= t; ++near) {
            ++s;
            if (near < 4) continue;
            for (int hi = pl.N; hi - s > 1;) {
                const int mid = s + ((hi - s) >> 1);
                if (pl.cu[mid] <= t)
                    s = mid;
                else
                    hi = mid;
            }
            break;
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

// How the append and the read go through a run: lane (u, r), u = lane % 16, has 8
// channels of the positions 8 r .. 8 r + 7 of the block, 128 channels in all: one
// head's, or with d = 64 two heads'.  Rows of the dense tensors are then read and
// written 16 bytes (fp32: 32) a lane, whole lines together.  Keys are 4 bytes a
// lane and position as they lie in the cache.  Values have the lane's 8 x 8 codes
// transposed, and 8 words of a channel each exchanged between the four r, so that
// each has all 16 bytes of two of the 8 channels.

// w[i] nibble k <-> w[k] nibble i.
__device__ __forceinline__ void transpose8(uint32_t (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = w[i], b = w[i + 4];
        w[i] = __builtin_amdgcn_perm(b, a, 0x05040100);
        w[i + 4] = __builtin_amdgcn_perm(b, a, 0x07060302);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = (j & 1) | (j & 2) << 1;
        const uint32_t a = w[i], b = w[i + 2];
        w[i] = __builtin_amdgcn_perm(b, a, 0x06020400);
        w[i + 2] = __builtin_amdgcn_perm(b, a, 0x07030501);
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint32_t a = w[i], b = w[i + 1];
        w[i] = (a & 0x0f0f0f0fu) | (b & 0x0f0f0f0fu) << 4;
        w[i + 1] = (a >> 4 & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
    }
}
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {  // a's upper half lanes with b's lower
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {  // a's odd 16 lanes with b's even
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
// The words of 8 channels for this lane's 8 positions, to and from all 32 positions
// of channels 2 r and 2 r + 1.
__device__ __forceinline__ void gather_channels(uint32_t (&w)[8], u32x4 (&c)[2]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) swap32(w[k], w[k + 4]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        swap16(w[k], w[k + 2]);
        swap16(w[k + 4], w[k + 6]);
        c[k] = u32x4{w[k], w[k + 2], w[k + 4], w[k + 6]};
    }
}
__device__ __forceinline__ void spread_channels(const u32x4 (&c)[2], uint32_t (&w)[8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        w[k] = c[k][0];
        w[k + 2] = c[k][1];
        w[k + 4] = c[k][2];
        w[k + 6] = c[k][3];
        swap16(w[k], w[k + 2]);
        swap16(w[k + 4], w[k + 6]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) swap32(w[k], w[k + 4]);
}

// The 8 codes of x, and the scale of the block of 32 that it shares with the three
// lanes beside it.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], uint32_t& scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, magnitude(x[i]));
    top = max(top, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(top), 0xB1, 0xf, 0xf, true)));
    top = max(top, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(top), 0x4E, 0xf, 0xf, true)));
    scale = mx_scale(top);
    const float inv = mx_inverse(scale);
    uint32_t w = 0;
    w = mx_put<0>(w, x[0] * inv, x[1] * inv);
    w = mx_put<1>(w, x[2] * inv, x[3] * inv);
    w = mx_put<2>(w, x[4] * inv, x[5] * inv);
    w = mx_put<3>(w, x[6] * inv, x[7] * inv);
    return scale == kMxNan ? 0 : w;
}

// A lane's place in a run.
template <int D> struct MxLane {
    static constexpr int kHeads = 128 / D;  // of a wave
    int u, r;
    bool live;    // its head exists
    int head;     // its head (one that exists)
    int channel;  // its first channel in the head
    __device__ __forceinline__ MxLane(int lane, int group, int Hkv) {
        u = lane & 15;
        r = lane >> 4;
        const int h = group * kHeads + u / (D / 8);
        live = h < Hkv;
        head = min(h, Hkv - 1);
        channel = 8 * (u % (D / 8));
    }
};

// Append: a wave per (range of tokens, 128 channels).  A block that the run covers
// in part keeps its other positions.  The values are loaded once the keys' registers
// are free, which leaves room for four waves a SIMD (both at once: 142 registers
// and 2 us more).  Bound by HBM: 8 prompts of 1000 .. 4096 tokens, 8 heads of 128,
// 105 MB, 26 us; the read of the same and 100 tokens more each, 109 MB, 23 us.
template <typename T, int D>
__global__ __launch_bounds__(256) void mx4_append_kernel(MxPlace pl, FastDiv groups, int waves, const T* __restrict__ k,
                                                         const T* __restrict__ v, uint8_t* __restrict__ k_codes,
                                                         uint8_t* __restrict__ k_scales, uint8_t* __restrict__ v_codes,
                                                         uint8_t* __restrict__ v_scales) {
    constexpr int CB = D / 32;
    const int lane = threadIdx.x & 63, id = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    if (id >= waves) return;
    const int range = groups(id);
    const MxLane<D> ln(lane, id - range * groups.d, pl.Hkv);
    for_runs(pl, range, lane, [&](const MxRun& r) {
        const size_t row = r.row + (static_cast<size_t>(ln.head) << pl.page_shift);
        // the run's tokens: 32-bit offsets from its first
        const uint32_t stride = static_cast<uint32_t>(pl.Hkv) * D, mine = static_cast<uint32_t>(ln.head) * D + ln.channel;
        const T *kt = k + static_cast<size_t>(r.token) * stride, *vt = v + static_cast<size_t>(r.token) * stride;
        const bool all = r.count == kMxRows;
        auto token = [&](int i) { return min(max(8 * ln.r + i - r.slot, 0), r.count - 1); };  // outside the run: its first or last
        auto within = [&](int i) { return ln.live && 8 * ln.r + i >= r.slot && 8 * ln.r + i < r.slot + r.count; };
        frag_t<T> x[2][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[0][i] = load8(kt + (token(i) * stride + mine));
        u32x4* at = reinterpret_cast<u32x4*>(v_codes + row * (D / 2) + static_cast<size_t>(ln.channel + 2 * ln.r) * 16);
        u32x4 old[2] = {};
        if (!all) {
            old[0] = at[0];
            old[1] = at[1];
        }
        uint32_t w[8], e[8];
        auto quantise = [&](const frag_t<T> (&x)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float f[8];
#pragma unroll
                for (int y = 0; y < 8; ++y) f[y] = static_cast<float>(x[i][y]);
                w[i] = quantise8(f, e[i]);
            }
        };
        // a head's scales of a position in one word (d = 64: half), from the lanes that have its blocks
        auto put_scales = [&](uint8_t* scales) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t s = e[i];
                s |= static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(e[i]), 0x104, 0xf, 0xf, true)) << 8;
                if constexpr (CB == 4) {
                    s |= static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(s), 0x108, 0xf, 0xf, true)) << 16;
                }
                e[i] = s;
            }
            if (ln.channel != 0 || !ln.live) return;
            uint8_t* p = scales + (row + 8 * ln.r) * CB;
            if (all) {
                if constexpr (CB == 4) {
                    reinterpret_cast<u32x4*>(p)[0] = u32x4{e[0], e[1], e[2], e[3]};
                    reinterpret_cast<u32x4*>(p)[1] = u32x4{e[4], e[5], e[6], e[7]};
                } else {
                    u32x4 t;
#pragma unroll
                    for (int i = 0; i < 4; ++i) t[i] = (e[2 * i] & 0xffffu) | e[2 * i + 1] << 16;
                    reinterpret_cast<u32x4*>(p)[0] = t;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (!within(i)) continue;
                    if constexpr (CB == 4)
                        reinterpret_cast<uint32_t*>(p)[i] = e[i];
                    else
                        reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(e[i]);
                }
            }
        };
        quantise(x[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (within(i)) *reinterpret_cast<uint32_t*>(k_codes + (row + 8 * ln.r + i) * (D / 2) + ln.channel / 2) = w[i];
        put_scales(k_scales);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[1][i] = load8(vt + (token(i) * stride + mine));
        quantise(x[1]);
        put_scales(v_scales);
        transpose8(w);
        u32x4 c[2];
        gather_channels(w, c);
        if (!all) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // 8 positions a word
                const int lo = min(max(r.slot - 8 * i, 0), 8), hi = min(max(r.slot + r.count - 8 * i, 0), 8);
                const uint32_t mask = (hi == 8 ? 0xffffffffu : (1u << 4 * hi) - 1) & ~(lo == 8 ? 0xffffffffu : (1u << 4 * lo) - 1);
#pragma unroll
                for (int n = 0; n < 2; ++n) c[n][i] = (c[n][i] & mask) | (old[n][i] & ~mask);
            }
        }
        if (ln.live) {
            at[0] = c[0];
            at[1] = c[1];
        }
    });
}

// The 8 codes of a word times the scale of byte b, exactly, 16 bytes aligned.
__device__ __forceinline__ void store8(bf16_t* p, uint32_t w, uint32_t b) {
    u32x4 x = __builtin_bit_cast(u32x4, mx_bf16(w, mx_float(b)));
    if (b == kMxNan) x = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
    *reinterpret_cast<u32x4*>(p) = x;
}
__device__ __forceinline__ void store8(float* p, uint32_t w, uint32_t b) {
    const bf16x8v x = mx_bf16(w, 1.f);
    const float f = b == kMxNan ? NAN : mx_float(b);
    f32x4 lo, hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo[i] = static_cast<float>(x[i]) * f;
        hi[i] = static_cast<float>(x[4 + i]) * f;
    }
    reinterpret_cast<f32x4*>(p)[0] = lo;
    reinterpret_cast<f32x4*>(p)[1] = hi;
}

// Read: the same runs, the other way.
template <typename T, int D>
__global__ __launch_bounds__(256) void mx4_read_kernel(MxPlace pl, FastDiv groups, int waves,
                                                       const uint8_t* __restrict__ k_codes,
                                                       const uint8_t* __restrict__ k_scales,
                                                       const uint8_t* __restrict__ v_codes,
                                                       const uint8_t* __restrict__ v_scales, T* __restrict__ k,
                                                       T* __restrict__ v) {
    constexpr int CB = D / 32;
    const int lane = threadIdx.x & 63, id = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    if (id >= waves) return;
    const int range = groups(id);
    const MxLane<D> ln(lane, id - range * groups.d, pl.Hkv);
    for_runs(pl, range, lane, [&](const MxRun& r) {
        const size_t row = r.row + (static_cast<size_t>(ln.head) << pl.page_shift) + 8 * ln.r;
        const uint32_t stride = static_cast<uint32_t>(pl.Hkv) * D, mine = static_cast<uint32_t>(ln.head) * D + ln.channel;
        T *kt = k + static_cast<size_t>(r.token) * stride, *vt = v + static_cast<size_t>(r.token) * stride;
        auto within = [&](int i) { return ln.live && 8 * ln.r + i >= r.slot && 8 * ln.r + i < r.slot + r.count; };
        uint32_t w[2][8], e[2][8];
        u32x4 c[2];
        const u32x4* at = reinterpret_cast<const u32x4*>(v_codes + (row - 8 * ln.r) * (D / 2) +
                                                         static_cast<size_t>(ln.channel + 2 * ln.r) * 16);
        c[0] = at[0];
        c[1] = at[1];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[0][i] = *reinterpret_cast<const uint32_t*>(k_codes + (row + i) * (D / 2) + ln.channel / 2);
            e[0][i] = k_scales[(row + i) * CB + ln.channel / 32];
            e[1][i] = v_scales[(row + i) * CB + ln.channel / 32];
        }
        spread_channels(c, w[1]);
        transpose8(w[1]);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (within(i)) store8((n ? vt : kt) + (static_cast<uint32_t>(8 * ln.r + i - r.slot) * stride + mine), w[n][i], e[n][i]);
    });
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

MxPlace place_of(int N, int total, int Hkv, int page_size, int num_pages, int max_pages, const int* cu, const int* first,
                 const int* table, int d, int& groups, unsigned long long& waves) {
    // A wave goes through its runs one after another: a range holds about as many
    // tokens as a run does, and fewer where that leaves the GPU with little to do.
    // Append and read in us, with ranges of 32 and of 8: 5 prompts to 77 tokens, one
    // group, 16.1 and 10.9; eight groups: 8 to 100 16.6, 13.4; 8 to 400 (1604 tokens)
    // 19.8, 17.1; 8 to 1000 (4007) 22.5, 22.2; 32 to 300 (4831) 22.6, 24.0.  One prompt:
    // eight groups 500 tokens 12.6, 10.8, but 1000 13.3, 14.3 and 2000 15.6, 17.5 (its
    // runs lie evenly, and three of four shorter ranges have none); one group 1000
    // 11.7, 9.3, 16000 14.6, 12.6.
    const int mean = total / N;
    groups = d == 64 ? (Hkv + 1) / 2 : Hkv;
    const bool few = static_cast<long long>(total) * groups <= 16384;
    const int range = mean >= 32 && !few ? 32 : mean >= 8 ? 8 : 2;
    MxPlace pl{N, total, Hkv, log2_of(page_size), num_pages, max_pages, range, cu, first, table};
    waves = (static_cast<unsigned long long>(total) + range - 1) / range * groups;
    return pl;
}

// The most keys that a sequence of the batch can have in sight.
long long mx4_keys(int page_size, int max_pages, int window, int sinks, int Tq) {
    const long long keys = static_cast<long long>(max_pages) * page_size, seen = static_cast<long long>(window) + Tq + sinks;
    return window && keys > seen ? seen : keys;
}
constexpr int kMxShares = 512;  // two workgroups to a CU

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
    // A dealt batch pays for its join and for the shares' search, a unit of its own for
    // the longest sequence's steps one after another.  The lengths are device data: the
    // rule goes by what the table has room for, and short sequences behind a wide table
    // are dealt out too (128 of 50 .. 100 tokens, 32 heads over 32: 17.6 us in a table of
    // 128 keys, 47.2 in one of 32768; over 8: 8.3 and 17.5).  Measured with 32 heads over 8 and
    // over 32, graph times in us:
    //  units  keys   a wave  a workgroup  dealt
    //     64   500     14.1      7.4
    //    512   500     14.8     11.3
    //   1024   500     17.1     20.5
    //   2048   100     11.8     26.2
    //   2048  1000     50.3     56.2      63.6
    //   1024  2000     50.0     52.6      54.1   (16 .. 2000: 42.6, 38.6, 45.4)
    //      8  1000     22.0      9.0      11.3
    //      8  2000     40.2     14.6      11.7
    //    256  4000     76.2     28.9      37.0   (16 .. 4000: 75.1, 24.8, 27.3)
    //    256  5000     94.3     35.2      41.3   (16 .. 5000: 29.5 against 27.9, one alone 27.9 against 16.8)
    //     64  4000     75.6     24.0      18.9
    const long long keys = mx4_keys(page_size, max_pages, window, sinks, Tq), units = static_cast<long long>(B) * a.per();
    const long long own = 16 * units < 1024 ? 1024 : 16 * units < 4096 ? 16 * units : 4096;
    a.alone = keys <= (units >= 1024 ? 1024 : kQuad);
    a.shares = a.alone || keys <= own ? 0 : kMxShares;
    a.heads = Tq * a.G < 16 ? Tq * a.G : 16;
    a.by_group = FastDiv(a.G);
    a.by_tiles = FastDiv(a.head_tiles);
    return a;
}

template <typename T, int D, int X>
hipError_t launch_mx4_decode_t(const Mx4Args& a, const void* q, const void* k_codes, const void* k_scales,
                               const void* v_codes, const void* v_scales, const int* table, const int* lengths, void* o,
                               float* ws, hipStream_t st) {
    const unsigned long long rows = static_cast<unsigned long long>(a.B) * a.Tq * a.Hq;
    const unsigned long long most = (static_cast<unsigned long long>(a.max_pages) << a.page_shift) / kQuad + 2 + kUnitCost;
    const unsigned long long units = static_cast<unsigned long long>(a.B) * a.per();
    const unsigned long long blocks = a.shares ? a.shares : a.alone ? (units + kMxWaves - 1) / kMxWaves : units;
    return launch_dealt<T, D>(a, blocks, rows, most, 64 * kMxWaves, table, lengths, o, ws, st,
                              [&](unsigned blocks, float* part_o, float* part_ml) {
                                  auto* f = a.alone ? mx4_decode_kernel<T, D, X, true> : mx4_decode_kernel<T, D, X, false>;
                                  constexpr int lds = Mx4Lds<D>::kBytes;
                                  if (lds > 64 * 1024) {
                                      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(f),
                                                                               hipFuncAttributeMaxDynamicSharedMemorySize, lds);
                                      if (e != hipSuccess) return e;
                                  }
                                  hipLaunchKernelGGL(f, dim3(blocks), dim3(64 * kMxWaves), lds, st, a,
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
    // by the keys alone, from 513 of them: which batches are dealt out is free to change
    attn::Mx4Args a = attn::mx4_args(1, Tq, Hq, Hkv, page_size, 0, max_pages, window, sinks, 1.f);
    a.shares = attn::mx4_keys(page_size, max_pages, window, sinks, Tq) <= 512 ? 0 : attn::kMxShares;
    return attn::part_floats(a, d);
}

hipError_t launch_attn_decode_mx4(int dtype, int B, int Tq, int Hq, int Hkv, int d, int page_size, int num_pages,
                                  int max_pages, int window, int sinks, float scale, const void* q, const void* k_codes,
                                  const void* k_scales, const void* v_codes, const void* v_scales, const int* table,
                                  const int* lengths, void* o, float* ws, hipStream_t st) {
    const attn::Mx4Args a = attn::mx4_args(B, Tq, Hq, Hkv, page_size, num_pages, max_pages, window, sinks, scale);
    auto* f = d == 64 ? attn::launch_mx4_decode_t<float, 64, 1> : attn::launch_mx4_decode_t<float, 128, 1>;
    if (dtype == GDR_DTYPE_BF16) {
        if (a.heads <= 4)
            f = d == 64 ? attn::launch_mx4_decode_t<bf16_t, 64, 4> : attn::launch_mx4_decode_t<bf16_t, 128, 4>;
        else if (a.heads <= 8)
            f = d == 64 ? attn::launch_mx4_decode_t<bf16_t, 64, 2> : attn::launch_mx4_decode_t<bf16_t, 128, 2>;
        else
            f = d == 64 ? attn::launch_mx4_decode_t<bf16_t, 64, 1> : attn::launch_mx4_decode_t<bf16_t, 128, 1>;
    }
    return f(a, q, k_codes, k_scales, v_codes, v_scales, table, lengths, o, ws, st);
}

hipError_t launch_attn_append_mx4(int dtype, int N, int total, int Hkv, int d, int page_size, int num_pages, int max_pages,
                                  const void* k, const void* v, const int* cu, const int* lengths, void* k_codes,
                                  void* k_scales, void* v_codes, void* v_scales, const int* table, hipStream_t st) {
    unsigned long long waves;
    int groups;
    const attn::MxPlace pl = attn::place_of(N, total, Hkv, page_size, num_pages, max_pages, cu, lengths, table, d, groups, waves);
    const unsigned long long blocks = (waves + 3) / 4;
    if (!grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
    auto go = [&](auto t, auto dd) {
        using T = decltype(t);
        hipLaunchKernelGGL((attn::mx4_append_kernel<T, decltype(dd)::value>), dim3(static_cast<unsigned>(blocks)), dim3(256),
                           0, st, pl, attn::FastDiv(groups), static_cast<int>(waves), static_cast<const T*>(k),
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
    int groups;
    const attn::MxPlace pl = attn::place_of(N, total, Hkv, page_size, num_pages, max_pages, cu, first, table, d, groups, waves);
    const unsigned long long blocks = (waves + 3) / 4;
    if (!grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
    auto go = [&](auto t, auto dd) {
        using T = decltype(t);
        hipLaunchKernelGGL((attn::mx4_read_kernel<T, decltype(dd)::value>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                           st, pl, attn::FastDiv(groups), static_cast<int>(waves), static_cast<const uint8_t*>(k_codes),
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
