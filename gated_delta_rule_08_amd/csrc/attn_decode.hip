// Attention over a paged key-value cache: the decode step (one new token per
// sequence, appended to its page and attended from) and the append of whole
// prompts.
//
// Pages are [page, key head, slot, channel], so a head's keys of one page are
// one contiguous block.  The step reads every visible key and value once and
// does 4 d flops per query head and key with them: HBM-bound for any group a
// model uses.  It is therefore built for bytes in flight: each wave streams
// its own 32 keys per step into LDS tiles of its own, straight from memory, the
// next step's keys requested as soon as this step's are read, the values
// likewise; no registers hold them, and no barrier until the end.  The group's
// query heads are the 16 columns of S^T = K Q^T, so a key read serves every head
// of its group.  64 sequences of 16 .. 8000 tokens, 8 key heads, d=128 (1.05 GB):
// 163 us and 6 for the join, 6.0 TB/s of the whole call; one of 32768: 24 + 5 us.
//
// The visible keys of a sequence are a list (the sinks, then the window) in
// blocks of 128.  Sequences differ in length, so it is not they that are dealt
// out but the blocks: the blocks of all (sequence, key head) units in a row are
// cut into equal shares, one per workgroup, whatever the lengths are.  A
// workgroup finds its share from the lengths alone (a scan over the batch),
// writes the units it holds whole, and leaves (m, l, O) of the at most two it
// shares with others to a second kernel, which joins them in order.  Lengths
// of at most 512 keys take one workgroup per unit and no join.
#include "attn_common.h"

namespace gdr {
namespace attn {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kStep = 32;                // keys of a wave's step
constexpr int kBlock = kStep * kWaves;   // keys of a workgroup's step

struct DecodeArgs {
    int B, Hq, Hkv, G, head_tiles;
    int page_shift, num_pages, max_pages;
    int window, sinks;
    float scale;
    int shares;  // workgroups the blocks are dealt to; 0: one workgroup per unit
    int heads;   // query heads of a unit: min(16, G)
};

// What one sequence's step covers, from its length alone (the same in every
// workgroup and in the join).
struct Span {
    int pos;     // position of the new token
    int w_lo;    // first key of the window
    int sinks;   // keys before it that stay visible
    int count;   // visible keys
    int blocks;  // 0: the length is out of range
};
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int p) {
    Span s;
    s.pos = p;
    s.w_lo = a.window ? max(0, p - a.window + 1) : 0;
    s.sinks = min(a.sinks, s.w_lo);
    s.count = s.sinks + (p - s.w_lo) + 1;
    s.blocks = p < 0 || (p >> a.page_shift) >= a.max_pages ? 0 : (s.count - 1) / kBlock + 1;
    return s;
}
// A sequence whose new position has no page is skipped (its blocks count all
// the same).
__device__ __forceinline__ bool has_page(const DecodeArgs& a, int b, int p, const int* __restrict__ table) {
    const int page = table[static_cast<size_t>(b) * a.max_pages + (p >> a.page_shift)];
    return page >= 0 && page < a.num_pages;
}

// The blocks of the batch in a row: sequence by sequence, within one unit by
// unit (key head, 16 query heads), `per` units each.  A wave sums them 256
// sequences at a time, four to a lane, so that their lengths come together.
__device__ __forceinline__ int scan64(int x, int lane) {  // inclusive
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const int y = __shfl_up(x, s);
        if (lane >= s) x += y;
    }
    return x;
}
struct Blocks4 {
    int each[4], upto;  // of sequences at + 4 lane .. + 3; blocks of at .. and these
};
__device__ __forceinline__ Blocks4 blocks_of(const DecodeArgs& a, int at, const int* __restrict__ lengths, int lane) {
    Blocks4 r;
    int sum = 0, len[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) len[x] = at + 4 * lane + x < a.B ? lengths[at + 4 * lane + x] : -1;
#pragma unroll
    for (int x = 0; x < 4; ++x) sum += r.each[x] = span_of(a, len[x]).blocks;
    r.upto = scan64(sum, lane);
    return r;
}
// Blocks of one unit per sequence: of the whole batch, and of the sequences before b.
__device__ __forceinline__ long long all_blocks(const DecodeArgs& a, const int* lengths, int lane, int b, long long& before) {
    long long sum = 0;
    before = 0;
    for (int at = 0; at < a.B; at += 256) {
        const Blocks4 r = blocks_of(a, at, lengths, lane);
        if (b >= at && b < at + 256) {
            const int x = b - at, rest = x & 3;
            int mine = r.upto;  // up to and with this lane's four, less those not before b
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (y >= rest) mine -= r.each[y];
            before = sum + __shfl(mine, x >> 2);
        }
        sum += __shfl(r.upto, 63);
    }
    return sum;
}

// Shares in use: no share is empty, so a unit's parts are consecutive shares.
__device__ __forceinline__ int shares_of(const DecodeArgs& a, long long n) {
    return static_cast<int>(n < a.shares ? n : a.shares);
}
// The share that holds block g of n, share w being blocks [w n / W, (w+1) n / W).
__device__ __forceinline__ int owner(long long g, long long n, int W) {
    return static_cast<int>(((g + 1) * W - 1) / n);
}

template <typename T, int D> struct DecodeCfg {
    static constexpr int kTile = kStep * D * static_cast<int>(sizeof(T));  // a wave's K or V tile
    static constexpr int kTable = 512;                                     // and its table entries, two steps
    static constexpr int kWave = 2 * kTile + kTable;
    static constexpr int kPitch = D + 4;  // floats of a joined row
    static constexpr int kJoin = kWaves * 16 * (kPitch + 2) * 4;
    static constexpr int kLds = kWaves * kWave > kJoin ? kWaves * kWave : kJoin;
};

// Row fragment for 16x16x32 products: lane (c = lane % 16, h = lane / 16) gets
// elements 32 e + 8 h .. + 7 of row c.
template <typename T, int D> struct RowRead16;
template <int D> struct RowRead16<bf16_t, D> {
    __device__ __forceinline__ static int base(int lane) { return Tile<bf16_t, D>::at(lane & 15) ^ ((lane >> 4) << 4); }
    __device__ __forceinline__ static bf16x8v get(const unsigned char* lds, int base, int e) {
        return __builtin_bit_cast(bf16x8v, *reinterpret_cast<const uint4*>(lds + (base ^ (e << 6))));
    }
};
template <int D> struct RowRead16<float, D> {
    __device__ __forceinline__ static int base(int lane) { return Tile<float, D>::at(lane & 15) ^ ((lane >> 4) << 5); }
    __device__ __forceinline__ static f32x8 get(const unsigned char* lds, int base, int e) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(lds + (base ^ (e << 7)));
        const f32x4 b = *reinterpret_cast<const f32x4*>(lds + (base ^ (e << 7) ^ 16));
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
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

// At most n of this wave's latest loads and copies are still on their way.
template <int N> __device__ __forceinline__ void wait_loads() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
}
// This wave's LDS reads have returned: what they read may be overwritten.
__device__ __forceinline__ void wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);
    asm volatile("" ::: "memory");
}

template <typename T, int D>
__global__ __launch_bounds__(64 * kWaves, sizeof(T) * D <= 256 ? 2 : 1) void decode_kernel(
    DecodeArgs a, const T* __restrict__ q, const T* __restrict__ knew, const T* __restrict__ vnew, T* k_pages,
    T* v_pages, const int* __restrict__ table, const int* __restrict__ lengths, T* __restrict__ o,
    float* __restrict__ part_o, float* __restrict__ part_ml) {
    using C = DecodeCfg<T, D>;
    using L = Tile<T, D>;
    constexpr int KS = D / 32, DT = D / 16;
    constexpr int kPer = 1024 / L::kRow, kCopies = kStep / kPer;  // rows of one copy, copies of a tile
    constexpr int kNone = -1, kNew = -2;
    extern __shared__ unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c16 = lane & 15, h4 = lane >> 4;

    const int slot_mask = (1 << a.page_shift) - 1, per = a.Hkv * a.head_tiles;
    // a scale of 0 as one that no score survives: c -inf of a hidden key stays -inf
    const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-37f);
    unsigned char *kt = smem + wave * C::kWave, *vt = kt + C::kTile, *tt = vt + C::kTile;
    const uint32_t kt_at = lds_addr(kt), vt_at = lds_addr(vt), tt_at = lds_addr(tt);
    const int kb = RowRead16<T, D>::base(lane), vb = ColRead16<T, D>::base(lane);

    // this workgroup's blocks: [at_block, at_block + left) of unit `unit` of sequence b and on
    int b, unit, at_block, left;
    Span sp;
    if (a.shares == 0) {
        b = blockIdx.x / per;
        unit = blockIdx.x - b * per;
        sp = span_of(a, lengths[b]);
        at_block = 0;
        left = sp.blocks;
    } else {
        long long before;
        const long long n = per * all_blocks(a, lengths, lane, -1, before);
        const int W = shares_of(a, n);
        if (static_cast<int>(blockIdx.x) >= W) return;
        const long long lo = n * blockIdx.x / W, hi = n * (blockIdx.x + 1) / W;
        left = __builtin_amdgcn_readfirstlane(static_cast<int>(hi - lo));
        before = 0;  // per unit
        for (b = 0; b < a.B; b += 256) {  // the first sequence that ends after lo
            const Blocks4 r = blocks_of(a, b, lengths, lane);
            const uint64_t past = __ballot((before + r.upto) * per > lo);
            if (past) {
                int x = 0, upto = r.upto - r.each[0] - r.each[1] - r.each[2] - r.each[3];
#pragma unroll
                for (int y = 0; y < 3; ++y)
                    if (x == y && (before + upto + r.each[y]) * per <= lo) {
                        upto += r.each[y];
                        ++x;
                    }
                const int from = __builtin_ctzll(past);
                before += __shfl(upto, from);
                b += 4 * from + __shfl(x, from);
                break;
            }
            before += __shfl(r.upto, 63);
        }
        b = __builtin_amdgcn_readfirstlane(b);
        if (b >= a.B) return;  // not reached unless the lengths change under the call
        sp = span_of(a, lengths[b]);
        const long long in = lo - before * per;
        unit = __builtin_amdgcn_readfirstlane(static_cast<int>(in / max(1, sp.blocks)));
        at_block = __builtin_amdgcn_readfirstlane(static_cast<int>(in - static_cast<long long>(unit) * sp.blocks));
    }

#pragma unroll 1
    while (left > 0) {
        if (unit >= per || sp.blocks == 0) {  // the next sequence that is not skipped
            if (++b >= a.B) return;
            unit = 0;
            sp = span_of(a, lengths[b]);
            continue;
        }
        const int take = min(left, sp.blocks - at_block);
        if (!has_page(a, b, sp.pos, table)) {
            left -= take;
            at_block = 0;
            ++unit;
            continue;
        }
        const int hk = unit / a.head_tiles, ht = unit - hk * a.head_tiles;
        const int* trow = table + static_cast<size_t>(b) * a.max_pages;
        const size_t new_row = static_cast<size_t>(b) * a.Hkv + hk;
        if (at_block == 0 && ht == 0 && threadIdx.x < 2 * L::kUnits) {  // the new token into its page
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

        // List entry i (entries past the end repeat the last one and are hidden):
        // its key, and its row in the page tensors.  kNew: the new token's own
        // row is taken from the call's k and v, as its page is being written.
        const int first = at_block * kBlock, last = min(sp.count, first + take * kBlock);
        auto key_of = [&](int i) {
            i = min(i, last - 1);
            return i < sp.sinks ? i : i - sp.sinks + sp.w_lo;
        };
        auto row_of = [&](int i, int page) {
            const int key = key_of(i);
            if (i >= last) return kNone;
            if (key == sp.pos) return kNew;
            if (page < 0 || page >= a.num_pages) return kNone;
            return ((page * a.Hkv + hk) << a.page_shift) + (key & slot_mask);
        };
        // Copies on their way to LDS: the table entries of a step, its keys, its
        // values (unit by unit, each lane fetching what belongs at its place;
        // hidden rows read row 0).
        auto fetch_table = [&](int i, int slot) {
            gather_words(tt_at + 256 * slot, trow + (key_of(i) >> a.page_shift));
        };
        int row[kCopies];  // of the units this lane fetches
        auto rows_to_lanes = [&](int rid) {
#pragma unroll
            for (int j = 0; j < kCopies; ++j) row[j] = __shfl(rid, kPer * j + lane / L::kUnits);
        };
        auto fetch = [&](uint32_t lds, const T* pages, const T* fresh) {
#pragma unroll
            for (int j = 0; j < kCopies; ++j) {
                const int u = (lane % L::kUnits) ^ L::swz(kPer * j + lane / L::kUnits);
                const T* p = row[j] == kNew ? fresh + new_row * D : pages + static_cast<size_t>(max(row[j], 0)) * D;
                stream_1k(lds + 1024 * j, p + u * (16 / sizeof(T)));
            }
        };

        f32x4 acc[DT];
#pragma unroll
        for (int t = 0; t < DT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, l = 0.f;

        // A wave's step: 32 keys.  Its table entries were fetched two steps
        // before, its keys once the step before had read its own, its values once
        // that step was done.
        int at = first + wave * kStep, slot = 0, rid = kNone;
        const int mine = lane & 31;
        if (at < last) {
            fetch_table(at + mine, 0);
            fetch_table(at + kBlock + mine, 1);
            wait_loads<0>();
            rid = row_of(at + mine, *reinterpret_cast<const int*>(tt + 4 * mine));
            rows_to_lanes(rid);
            fetch(kt_at, k_pages, knew);
            fetch(vt_at, v_pages, vnew);
        }
#pragma unroll 1
        for (; at < last; at += kBlock, slot ^= 1) {
            const uint32_t shown = static_cast<uint32_t>(__ballot(rid != kNone));
            const bool more = at + kBlock < last;
            wait_loads<kCopies>();  // the keys; the values may still come
            f32x4 s[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                s[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < KS; ++e)
                    s[u] = mma16(RowRead16<T, D>::get(kt + 16 * u * L::kRow, kb, e), qf[e], s[u]);
            }
            if (more) {
                rid = row_of(at + kBlock + mine, *reinterpret_cast<const int*>(tt + 256 * (slot ^ 1) + 4 * mine));
                rows_to_lanes(rid);
                wait_lds();
                fetch_table(at + 2 * kBlock + mine, slot);
                fetch(kt_at, k_pages, knew);
            }
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
            for (int y = 0; y < 8; ++y) {
                w[y] = ex2(fmaf(s[y >> 2][y & 3], c, -mc));
                l += w[y];
            }
            const frag_t<T> pf = pack8<T>(w);
            if (more)
                wait_loads<kCopies + 1>();  // the values; the next keys and table entries may still come
            else
                wait_loads<0>();
            if (shown != 0xffffffffu) {  // a weight of 0 needs a value that is finite
#pragma unroll
                for (int j = 0; j < kCopies; ++j)
                    if (!((shown >> (kPer * j + lane / L::kUnits)) & 1))
                        *reinterpret_cast<uint4*>(vt + 1024 * j + 16 * lane) = make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int t = 0; t < DT; ++t) acc[t] = mma16(ColRead16<T, D>::get(vt, vb, t), pf, acc[t]);
            if (more) {
                wait_lds();
                fetch(vt_at, v_pages, vnew);
            }
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
        const bool whole = take == sp.blocks;
        if (head < nheads) {
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
            const float inv = lt == 0.f ? 0.f : 1.f / lt;
            // a shared unit's part: slot 1 holds its beginning, slot 0 what does not begin here
            const size_t prow = (static_cast<size_t>(blockIdx.x) * 2 + (at_block == 0)) * a.heads + head;
#pragma unroll
            for (int e = 0; e < D / 64; ++e) {
                const int d = 64 * e + 4 * (threadIdx.x & 15);
                f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int x = 0; x < kWaves; ++x)  // a wave without keys holds zeros; one whose weight underflows may hold a NaN
                    sum += *reinterpret_cast<const f32x4*>(jo + (x * 16 + head) * C::kPitch + d) * mw[x];
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
        left -= take;
        at_block = 0;
        ++unit;
        if (left > 0) __syncthreads();  // LDS is free for the next unit
    }
}

// Joins the parts of a shared unit, W waves per query head: part 0 is slot 1 of
// the unit's first share, the others slot 0 of the shares after it.  16 W parts
// at a time, lane s holding part s's weight 2^(m_s - max m); a wave adds every
// W-th part, the channels over its lanes, and the waves' sums are added in order.
template <typename T, int D, int W>
__global__ __launch_bounds__(256) void join_kernel(DecodeArgs a, const int* __restrict__ table,
                                                   const int* __restrict__ lengths,
                                                   const float* __restrict__ part_o,
                                                   const float* __restrict__ part_ml, T* __restrict__ o) {
    constexpr int N = D / 64, kEach = 16;
    __shared__ float sums[W > 1 ? W - 1 : 1][D];
    const int lane = threadIdx.x & 63, every = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = every % W;
    const int at = blockIdx.x * (4 / W) + every / W, b = at / a.Hq, hq = at - b * a.Hq;
    if (b >= a.B) return;
    const Span sp = span_of(a, lengths[b]);
    if (sp.blocks == 0 || !has_page(a, b, sp.pos, table)) return;
    const int per = a.Hkv * a.head_tiles, hk = hq / a.G, g = hq - hk * a.G;
    long long before;
    const long long n = per * all_blocks(a, lengths, lane, b, before);
    const long long lo = per * before + static_cast<long long>(hk * a.head_tiles + g / 16) * sp.blocks;
    const int used = shares_of(a, n), w0 = owner(lo, n, used), parts = owner(lo + sp.blocks - 1, n, used) - w0 + 1;
    if (parts == 1) return;  // written whole
    auto slot = [&](int s) { return (static_cast<size_t>(w0 + s) * 2 + (s == 0)) * a.heads + (g & 15); };
    float M = -INFINITY, total = 0.f, acc[N] = {};
    for (int s0 = 0; s0 < parts; s0 += kEach * W) {
        float m = -INFINITY, l = 0.f;
        if (lane < kEach * W && s0 + lane < parts) {
            m = part_ml[slot(s0 + lane) * 2];
            l = part_ml[slot(s0 + lane) * 2 + 1];
        }
        float x[kEach][N];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {  // all loads before the first use
            const int s = s0 + W * i + wave;
#pragma unroll
            for (int e = 0; e < N; ++e) x[i][e] = s < parts ? part_o[slot(s) * D + N * lane + e] : 0.f;
        }
        float mx = m;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) mx = fmaxf(mx, __shfl_xor(mx, s));
        mx = fmaxf(M, mx);
        const float old = M == -INFINITY ? 0.f : ex2(M - mx), w = m == -INFINITY ? 0.f : ex2(m - mx);
        M = mx;
        float add = l * w;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) add += __shfl_xor(add, s);
        total = total * old + add;
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] *= old;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const float ws = __shfl(w, W * i + wave);
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] = fmaf(ws, x[i][e], acc[e]);
        }
    }
    if constexpr (W > 1) {
        if (wave > 0) {
#pragma unroll
            for (int e = 0; e < N; ++e) sums[wave - 1][N * lane + e] = acc[e];
        }
        __syncthreads();
        if (wave > 0) return;
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const size_t row = static_cast<size_t>(b) * a.Hq + hq;
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
    const unsigned long long blocks =
        a.shares ? a.shares : static_cast<unsigned long long>(a.B) * a.Hkv * a.head_tiles;
    const unsigned long long rows = static_cast<unsigned long long>(a.B) * a.Hq;
    // a share's blocks have to fit an int, and so have those of one scan's sequences
    const unsigned long long most = (static_cast<unsigned long long>(a.max_pages) << a.page_shift) / kBlock + 1;
    if (a.shares && (static_cast<unsigned long long>(a.B) * a.Hkv * a.head_tiles * most / a.shares > 0x7fffffffull ||
                     (a.B < 256 ? a.B : 256) * most > 0x7fffffffull))
        return hipErrorInvalidConfiguration;
    if (!grid_fits(blocks, 64 * kWaves) || !grid_fits(rows, 256)) return hipErrorInvalidConfiguration;
    auto* f = decode_kernel<T, D>;
    if (C::kLds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(f),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, C::kLds);
        if (e != hipSuccess) return e;
    }
    float* part_o = ws;
    float* part_ml = ws ? ws + static_cast<size_t>(a.shares) * 2 * a.heads * D : nullptr;
    hipLaunchKernelGGL(f, dim3(static_cast<unsigned>(blocks)), dim3(64 * kWaves), C::kLds, st, a,
                       static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v),
                       static_cast<T*>(k_pages), static_cast<T*>(v_pages), table, lengths, static_cast<T*>(o),
                       part_o, part_ml);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.shares == 0) return e;
    // Many heads have few parts each and take a wave (64 sequences of 32: 5.7 against 10.9 us), few heads four.
    const bool many = rows >= 1024;
    auto* join = many ? join_kernel<T, D, 1> : join_kernel<T, D, 4>;
    hipLaunchKernelGGL(join, dim3(static_cast<unsigned>(many ? (rows + 3) / 4 : rows)), dim3(256), 0, st, a, table, lengths,
                       part_o, part_ml, static_cast<T*>(o));
    return hipGetLastError();
}

// Append: a workgroup copies 1024 consecutive 16-byte units of the new keys and
// the same of the values, four of each per thread.  The first unit's sequence is
// searched for once; the others start from it.  HBM-bound: 8 prompts of 1000 ..
// 4096 tokens (167 MB read and written) 35 us, 4.7 TB/s; stores that pass the
// caches by, 37.8 otherwise.
constexpr int kAppendUnits = 4;

__global__ __launch_bounds__(256) void append_kernel(int N, unsigned long long n, FastDiv per, FastDiv units,
                                                     int page_shift, int num_pages, int max_pages, int Hkv,
                                                     const u32x4* __restrict__ k, const u32x4* __restrict__ v,
                                                     const int* __restrict__ cu, const int* __restrict__ lengths,
                                                     u32x4* __restrict__ k_pages, u32x4* __restrict__ v_pages,
                                                     const int* __restrict__ table) {
    const unsigned long long first = static_cast<unsigned long long>(blockIdx.x) * (256 * kAppendUnits);
    const int t0 = static_cast<int>(first / per.d), x0 = static_cast<int>(first - static_cast<unsigned long long>(t0) * per.d);
    int seq = 0;  // the last sequence that starts at or before token t0
    for (int hi = N; hi - seq > 1;) {
        const int mid = (seq + hi) >> 1;
        if (cu[mid] <= t0)
            seq = mid;
        else
            hi = mid;
    }
    const int mask = (1 << page_shift) - 1;
    u32x4 a[kAppendUnits], b[kAppendUnits];
    size_t to[kAppendUnits];
    bool ok[kAppendUnits];
#pragma unroll
    for (int j = 0; j < kAppendUnits; ++j) {
        const int i = threadIdx.x + 256 * j;
        ok[j] = first + i < n;
        if (!ok[j]) continue;
        a[j] = __builtin_nontemporal_load(k + first + i);
        b[j] = __builtin_nontemporal_load(v + first + i);
    }
#pragma unroll
    for (int j = 0; j < kAppendUnits; ++j) {
        if (!ok[j]) continue;
        const int i = x0 + threadIdx.x + 256 * j, y = per(i), t = t0 + y, x = i - y * per.d;
        int s = seq;
        while (s + 1 < N && cu[s + 1] <= t) ++s;
        const int begin = cu[s], len = lengths[s];
        const long long pos = static_cast<long long>(len) + (t - begin);
        ok[j] = begin >= 0 && t >= begin && t < cu[s + 1] && len >= 0 && (pos >> page_shift) < max_pages;
        if (!ok[j]) continue;
        const int page = table[static_cast<size_t>(s) * max_pages + (pos >> page_shift)];
        ok[j] = page >= 0 && page < num_pages;
        const int hk = units(x), u = x - hk * units.d;
        const size_t row = ((static_cast<size_t>(page) * Hkv + hk) << page_shift) + static_cast<size_t>(pos & mask);
        to[j] = row * units.d + u;
    }
#pragma unroll
    for (int j = 0; j < kAppendUnits; ++j)
        if (ok[j]) {
            __builtin_nontemporal_store(a[j], k_pages + to[j]);
            __builtin_nontemporal_store(b[j], v_pages + to[j]);
        }
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

// Shares of the blocks: 512, two workgroups per CU, which registers and LDS allow
// at a time, so that all start and end together; none (one workgroup per unit)
// where no sequence can show more than 512 keys.  fp32 with d=128 (133 KB of LDS)
// fits one to a CU and runs its shares in two rounds, which evens out a large batch
// and costs a small one its start (32 query on 8 key heads, 512 against 256 shares:
// 64 sequences of 16..8000 tokens 348 / 363 us, 8 of 100..2000 42 / 33, one of
// 32768 64 / 55).
int decode_shares(int page_size, int max_pages, int window, int sinks) {
    long long keys = static_cast<long long>(max_pages) * page_size;
    if (window && keys > static_cast<long long>(window) + sinks) keys = static_cast<long long>(window) + sinks;
    return keys <= 512 ? 0 : 512;
}

}  // namespace
}  // namespace attn

size_t attn_decode_workspace_floats(int Hq, int Hkv, int d, int page_size, int max_pages, int window, int sinks) {
    const int G = Hq / Hkv;
    return static_cast<size_t>(attn::decode_shares(page_size, max_pages, window, sinks)) * 2 * (G < 16 ? G : 16) * (d + 2);
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
    a.shares = attn::decode_shares(page_size, max_pages, window, sinks);
    a.heads = a.G < 16 ? a.G : 16;
    auto* f = dtype == GDR_DTYPE_F32 ? (d == 64 ? attn::launch_decode_t<float, 64> : attn::launch_decode_t<float, 128>)
                                     : (d == 64 ? attn::launch_decode_t<bf16_t, 64> : attn::launch_decode_t<bf16_t, 128>);
    return f(a, q, k, v, k_pages, v_pages, table, lengths, o, ws, st);
}

hipError_t launch_attn_append(int dtype, int N, int total, int Hkv, int d, int page_size, int num_pages,
                              int max_pages, const void* k, const void* v, const int* cu, const int* lengths,
                              void* k_pages, void* v_pages, const int* table, hipStream_t st) {
    const int units = d * (dtype == GDR_DTYPE_F32 ? 4 : 2) / 16;
    const unsigned long long n = static_cast<unsigned long long>(total) * Hkv * units;
    const unsigned long long blocks = (n + 256 * attn::kAppendUnits - 1) / (256 * attn::kAppendUnits);
    if (!grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(attn::append_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, N, n,
                       attn::FastDiv(Hkv * units), attn::FastDiv(units), attn::log2_of(page_size), num_pages, max_pages, Hkv,
                       static_cast<const attn::u32x4*>(k), static_cast<const attn::u32x4*>(v), cu, lengths,
                       static_cast<attn::u32x4*>(k_pages), static_cast<attn::u32x4*>(v_pages), table);
    return hipGetLastError();
}

}  // namespace gdr
