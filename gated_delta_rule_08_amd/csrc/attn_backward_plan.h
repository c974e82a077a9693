// How the work of the attention backward is dealt out: which rows and keys a
// workgroup takes, into which parts a key's rows are cut and where the parts are
// kept.  Arithmetic on sizes alone, the same on the host and in the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "attn_plan.h"

namespace gdr {
namespace attn {

constexpr int kWaves = 4;
constexpr int kKeys = 32 * kWaves;  // keys of a dkdv workgroup
constexpr int kRows = 32 * kWaves;  // rows of a dq workgroup

struct BwdArgs {
    int B, Tq, Tk, Hq, Hkv, d;
    FastDiv G;
    int window, sinks;
    float scale;
    int rows, pitch;          // rows of a (sequence, key head); pitch of the row statistics
    int key_blocks, row_tiles;
    bool split;               // dq: 32 rows per workgroup, a quarter of the keys per wave
    bool sliced;              // key blocks cut their lists of rows, slice_rows to a workgroup,
    int slice_rows;
    int long_blocks;          // the first (those with sinks under a window) into at most long_slices,
    int long_slices, slices;  // the others into at most slices
    int sink_tiles, segs;     // not sliced: 32-key tiles that hold sinks, segments of each (at most)
    int seg_rows;
    // Key tiles whose gradients may come in parts.  Not sliced: the sinks' tiles, 1 +
    // segs parts each, slot by slot.  Sliced: those of the first part_blocks blocks,
    // block by block with room for what its list needs, then slot by slot.
    int part_tiles, part_blocks;
    int part_step;            // parts from one of a tile to its next
    int head_parts;           // parts of a head
    // The workspace: the row statistics, the slots, the parts.
    float* stats;             // [B Hkv, 2, pitch]: lse log2 e, then delta
    int* slots;               // sliced: [512], slots_before each block
    float* part;              // [B Hkv, parts of a head, 2, 32, d]
    __host__ __device__ __forceinline__ int cuts() const { return long_blocks * long_slices + (key_blocks - long_blocks) * slices; }
    __host__ __device__ __forceinline__ long long rows_before(int block) const;
    // Slots before a block's: a block of n rows has (rows before it + n) / slice_rows -
    // (rows before it) / slice_rows + 1 of them, at least n / slice_rows rounded up.
    // dq_kernel, which runs first, leaves them in `slots`: formed by every workgroup of
    // the join, the division takes as long as the join itself.
    __host__ __device__ __forceinline__ int slots_before(int block) const {
        return static_cast<int>(rows_before(block) / slice_rows) + block;
    }
    __device__ __forceinline__ float* part_of(int head, int tile, int slot, int d) const {
        const int at = (sliced ? 4 * slots[tile >> 2] : tile & ~3) + slot * part_step + (tile & 3);
        return part + (static_cast<size_t>(head) * head_parts + at) * 64 * d;
    }
};

// Rows in the lists of the key blocks before `block`, or a little more (sliced
// only).  In queries, key block i is seen by at most clamp(Tk - 128 i, 0, most) of
// them: by those from its first key on, under a window by no more than window + 127.
__host__ __device__ __forceinline__ long long rows_before(const BwdArgs& a, int block, int most) {
    const long long n = block, k = a.Tk < most ? 0 : min(block, (a.Tk - most) / kKeys + 1);  // the first k blocks have `most`
    return k * most + (n - k) * a.Tk - kKeys * ((n * (n - 1) - k * (k - 1)) / 2);
}
__host__ __device__ __forceinline__ long long BwdArgs::rows_before(int block) const {
    if (window == 0) return attn::rows_before(*this, block, Tq) * G.d;
    const int longs = min(block, long_blocks), most = min(Tq, window + kKeys - 1);
    // blocks whose last key's window ends before the first query
    const int past = Tk - Tq - window + 1, none = min(block, max(longs, past > 0 ? past / kKeys : 0));
    return (attn::rows_before(*this, longs, Tq) + attn::rows_before(*this, block, most) - attn::rows_before(*this, none, most)) * G.d;
}

// Rows (query * G + head) that see keys [j0, j1] through the window or, with
// no window, causally: [lo, hi).  Counted in queries that exist before the
// product with G: keys far before the first query's window would pass 32 bits.
__host__ __device__ __forceinline__ void rows_of(const BwdArgs& a, int j0, int j1, int& lo, int& hi) {
    const int off = a.Tk - a.Tq;
    lo = (j0 > off ? j0 - off : 0) * a.G.d;
    int end = a.Tq;
    if (a.window) end = max(0, min(end, j1 + a.window - off));
    hi = max(end * a.G.d, lo);
    if (a.sliced && a.window && j0 < a.sinks) hi = a.rows;  // no segments: the sinks' rows are sliced with the rest
}

// Rows of a slice of a list: as few slices of at most slice_rows as there can
// be, about equally long.
__host__ __device__ __forceinline__ int slice_of(const BwdArgs& a, int list) {
    if (!a.sliced || list <= a.slice_rows) return list;
    const int n = (list - 1) / a.slice_rows + 1;
    return ((list - 1) / n + 32) / 32 * 32;
}

// What one wave of dkdv_kernel has to do.
struct Piece {
    int head, b, hk;
    int tile, j0;     // its 32 keys
    int cut, lo, hi;  // the workgroup's rows
    bool parts;       // the keys' rows are not all here
};
template <int WAVES> __host__ __device__ __forceinline__ Piece piece_of(const BwdArgs& a, int bid, int wave) {
    constexpr bool kSeg = WAVES == 1;
    const int per = kSeg ? a.sink_tiles * a.segs : a.cuts();
    int head, x, lo, hi;
    place(bid, a.B * a.Hkv, per, head, x);  // the first keys are seen by the most rows
    // The last slice of every block that has so many, then the last but one: blocks
    // with short lists come at the end, and slices that do not exist are spread over
    // the XCDs.
    const int first = a.long_blocks * a.long_slices;  // pieces of the long blocks
    const bool in = !kSeg && x < first;
    const int b = head / a.Hkv, blocks = kSeg ? a.sink_tiles : in ? a.long_blocks : a.key_blocks - a.long_blocks;
    const int z = kSeg || in ? x : x - first, turn = z / blocks, y = z - turn * blocks + (kSeg || in ? 0 : a.long_blocks);
    const int cut = (kSeg ? a.segs : in ? a.long_slices : a.slices) - 1 - turn;
    const int tile = kSeg ? y : y * WAVES + wave;
    const int m0 = kSeg ? 32 * tile / kKeys * kKeys : y * kKeys;  // the keys of a main workgroup
    rows_of(a, m0, min(m0 + kKeys, a.Tk) - 1, lo, hi);
    const int size = kSeg ? a.seg_rows : slice_of(a, hi - lo);
    const bool parts = kSeg || hi - lo > size;
    lo = kSeg ? hi + cut * size : lo + cut * size;  // a segment's are past what the main workgroup takes
    hi = min(kSeg ? a.rows : hi, lo + size);
    return {head, b, head - b * a.Hkv, tile, 32 * tile, cut, lo, hi, parts};
}

// Most bytes that the parts of slices may take.  Shorter slices balance the compute
// units better, but leave a part of 128 keys each; lists are sliced below 512 key
// blocks only, whose gradients take at most 64 MiB in fp32.  By the estimate below
// the bound costs 0.07% on average over 4000 random training steps and 7% at most
// (8% at T=65408 with 32 query heads on one, for 256 MiB instead of 1.6 GB).
// Measured at T=16384, 32 query on 2 key heads, d=128: 229 MB of parts 10.0 ms,
// without the bound 415 MB and 9.6 ms.
constexpr size_t kPartBytes = 256 << 20;

constexpr int kSliced = 512;  // key blocks of all heads from which on none is sliced

inline BwdArgs make_args(bool f32, int B, int Tq, int Tk, int Hq, int Hkv, int d, int window, int sinks, float scale) {
    BwdArgs a{};
    a.B = B;
    a.Tq = Tq;
    a.Tk = Tk;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.G = FastDiv(Hq / Hkv);
    a.window = window;
    a.sinks = sinks;
    a.scale = scale;
    a.rows = Tq * a.G.d;
    a.pitch = (a.rows + 3) / 4 * 4;
    a.key_blocks = (Tk + kKeys - 1) / kKeys;
    const long long heads = static_cast<long long>(B) * Hkv, groups = heads * a.key_blocks;
    a.split = heads * ((a.rows + kRows - 1) / kRows) < (f32 ? 257 : 192);  // as the forward does
    a.row_tiles = a.split ? (a.rows + 31) / 32 : (a.rows + kRows - 1) / kRows;
    // The rows of a key block are cut into slices where that is faster by this
    // estimate (us): `row`, one CU's time for a row and 128 keys, times the rows of
    // a CU (an equal share and half of the longest piece, or the longest alone; fp32
    // pieces take a CU each, so that few enough to find one, 224, take as long as the
    // longest; 96 rows' time goes to each piece's start and end); `part` for each part
    // written and read, 4 for the kernel that joins them.  Without slices, sinks go
    // to segments.  Of 20 training steps of different sizes, each timed with every
    // length of slice (profiles/attention_slices.md), the one taken here is 1.5% from
    // the fastest on average and 11% at most.
    a.slices = a.long_slices = 1;
    a.slice_rows = a.rows;
    const int tiles = (Tk + 31) / 32;
    if (groups > 0 && groups < kSliced && a.rows > 0) {
        const double row = (f32 ? 0.40 : 0.040) * d / 128, part = 0.06 * d / 128;
        const bool sunk = window && sinks > 0;
        auto list = [&](int j) {
            int lo, hi;
            rows_of(a, j * kKeys, (j + 1) * kKeys < Tk ? (j + 1) * kKeys - 1 : Tk - 1, lo, hi);
            return hi - lo;
        };
        // The lists that slices are cut from, as groups of neighbouring blocks each as
        // long as its middle one's: at most 64 with sinks and 64 without, so that the
        // search takes a few microseconds whatever the length (60000 keys under a window
        // of 256: 3 us of the host, 18 block by block).
        int len[128], of[128], groups_n = 0, longest[2] = {0, 0};  // longest: without and with sinks
        auto time_of = [&](long long total, long long pieces, long long parts, int most_rows, int cut) {
            const double most = cut && cut < most_rows ? cut : most_rows, even = static_cast<double>(total) * heads / 256 + most / 2;
            const double ends = cut ? 96.0 * pieces * heads / 256 : 96.0;
            const bool once = f32 && cut && pieces * heads <= 224;
            return row * ((most > even || once ? most : even) + ends) + (parts ? 4 + part * parts * heads : 0);
        };
        long long total = 0;
        for (int j = 0; j < a.key_blocks; ++j) {
            const int n = list(j);
            total += n;
            if (n > longest[0]) longest[0] = n;
        }
        int best = 0;
        double least = time_of(total, 0, 0, longest[0], 0);
        if (sunk) {  // the segments' kernel and join
            const double even = static_cast<double>(heads) * ((sinks + 31) / 32) * a.rows / 1024;
            least += 8 + 0.13 * (even > 128 ? even : 128) * (f32 ? 5 : 1);
        }
        a.sliced = true;
        if (window) a.long_blocks = (sinks + kKeys - 1) / kKeys;
        total = longest[0] = 0;
        for (int sunken = 1; sunken >= 0; --sunken) {
            const int from = sunken ? 0 : a.long_blocks, end = sunken ? a.long_blocks : a.key_blocks, step = (end - from + 63) / 64;
            for (int j = from; j < end; j += step) {
                const int here = step < end - j ? step : end - j, n = list(j + here / 2);
                len[groups_n] = n;
                of[groups_n++] = here;
                total += static_cast<long long>(n) * here;
            }
            for (int j = from; j < end; ++j)
                if (list(j) > longest[sunken]) longest[sunken] = list(j);
        }
        const int most_rows = longest[0] > longest[1] ? longest[0] : longest[1];
        auto estimate = [&](int cut) {
            long long pieces = 0, parts = 0;
            for (int i = 0; i < groups_n; ++i) {
                const int here = len[i] > cut ? (len[i] - 1) / cut + 1 : 1;
                pieces += here * of[i];
                if (here > 1) parts += here * of[i];
            }
            return time_of(total, pieces, parts, most_rows, cut);
        };
        auto set = [&](int cut) {
            a.slice_rows = cut;
            a.slices = longest[0] > cut ? (longest[0] - 1) / cut + 1 : 1;
            a.long_slices = longest[1] > cut ? (longest[1] - 1) / cut + 1 : 1;
            a.part_blocks = a.slices > 1 ? a.key_blocks : a.long_slices > 1 ? a.long_blocks : 0;
            const long long parts = 4 * (a.rows_before(a.part_blocks) / cut + a.part_blocks);
            a.head_parts = static_cast<int>(parts < 0x7fffffff ? parts : 0x7fffffff);  // beyond kPartBytes
        };
        for (int cut = 32; cut < most_rows; cut = (cut + cut / 4 + 31) / 32 * 32) {
            set(cut);
            if (static_cast<size_t>(heads) * a.head_parts * 64 * d * sizeof(float) > kPartBytes) continue;
            const double t = estimate(cut);
            if (t < least) {
                least = t;
                best = cut;
            }
        }
        a.sliced = best > 0;
        if (a.sliced) {
            set(best);
            a.part_tiles = 4 * a.part_blocks < tiles ? 4 * a.part_blocks : tiles;
            a.part_step = 4;
        } else {
            set(a.rows);
            a.long_blocks = a.part_blocks = 0;
            a.head_parts = 0;
        }
    }
    // Sink segments: one wave per SIMD, no segment under 128 rows.
    if (!a.sliced && window && Tq > 0) a.sink_tiles = (sinks + 31) / 32;
    if (a.sink_tiles) {
        const long long even = heads * a.sink_tiles * a.rows / 1024;
        a.seg_rows = static_cast<int>(even < 128 ? 128 : even > a.rows ? a.rows : (even + 31) / 32 * 32);
        a.segs = (a.rows + a.seg_rows - 1) / a.seg_rows;
        a.part_tiles = a.sink_tiles;
        a.part_step = a.part_tiles;
        a.head_parts = a.part_tiles * (1 + a.segs);
    }
    return a;
}

// Floats of the workspace, and where its pieces are in one that begins at ws.
inline size_t workspace_floats(const BwdArgs& a) {
    const size_t heads = static_cast<size_t>(a.B) * a.Hkv;
    return heads * 2 * a.pitch + (a.sliced ? kSliced : 0) + heads * a.head_parts * 64 * a.d;
}
inline void set_workspace(BwdArgs& a, float* ws) {
    a.stats = ws;
    ws += static_cast<size_t>(a.B) * a.Hkv * 2 * a.pitch;
    a.slots = reinterpret_cast<int*>(ws);
    a.part = ws + (a.sliced ? kSliced : 0);
}

}  // namespace attn
}  // namespace gdr
