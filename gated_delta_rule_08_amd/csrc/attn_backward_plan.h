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
    int B, Tq, Tk, Hq, Hkv;
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
    // Key tiles whose gradients come in parts: the first long_tiles have room for
    // long_slots parts each, the others for slots.
    int part_tiles, long_tiles, long_slots, slots;
    float* stats;             // [B Hkv, 2, pitch]: lse log2 e, then delta
    float* part;              // [B Hkv, parts of a head, 2, 32, d]
    __host__ __device__ __forceinline__ int cuts() const { return long_blocks * long_slices + (key_blocks - long_blocks) * slices; }
    __host__ __device__ __forceinline__ size_t parts_before(int tile) const {  // within a head
        return static_cast<size_t>(tile < long_tiles ? tile : long_tiles) * long_slots +
               static_cast<size_t>(tile < long_tiles ? 0 : tile - long_tiles) * slots;
    }
    __host__ __device__ __forceinline__ float* part_of(int head, int tile, int slot, int d) const {
        return part + (static_cast<size_t>(head) * parts_before(part_tiles) + parts_before(tile) + slot) * 64 * d;
    }
};

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

inline BwdArgs make_args(bool f32, int B, int Tq, int Tk, int Hq, int Hkv, int d, int window, int sinks, float scale) {
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
    // length of slice, the one taken here is 2.0% from the fastest on average and 14%
    // at most.
    a.slices = a.long_slices = 1;
    a.slice_rows = a.rows;
    const int tiles = (Tk + 31) / 32;
    if (groups > 0 && groups < 512 && a.rows > 0) {
        const double row = (f32 ? 0.40 : 0.040) * d / 128, part = 0.06 * d / 128;
        const bool sunk = window && sinks > 0;
        auto list = [&](int j) {
            int lo, hi;
            rows_of(a, j * kKeys, (j + 1) * kKeys < Tk ? (j + 1) * kKeys - 1 : Tk - 1, lo, hi);
            return hi - lo;
        };
        auto estimate = [&](int cut, int& longest) {  // cut 0: no slices
            long long total = 0, pieces = 0, parts = 0;
            longest = 0;
            for (int j = 0; j < a.key_blocks; ++j) {
                const int n = list(j), here = cut && n > cut ? (n - 1) / cut + 1 : 1;
                total += n;
                pieces += here;
                if (here > 1) parts += here;
                if (n > longest) longest = n;
            }
            const double most = cut && cut < longest ? cut : longest, even = static_cast<double>(total) * heads / 256 + most / 2;
            const double ends = cut ? 96.0 * pieces * heads / 256 : 96.0;
            const bool once = f32 && cut && pieces * heads <= 224;
            return row * ((most > even || once ? most : even) + ends) + (parts ? 4 + part * parts * heads : 0);
        };
        int longest, best = 0;
        double least = estimate(0, longest);
        if (sunk) {  // the segments' kernel and join
            const double even = static_cast<double>(heads) * ((sinks + 31) / 32) * a.rows / 1024;
            least += 8 + 0.13 * (even > 128 ? even : 128) * (f32 ? 5 : 1);
        }
        a.sliced = true;
        estimate(0, longest);
        for (int cut = 32; cut < longest; cut = (cut + cut / 4 + 31) / 32 * 32) {
            int unused;
            const double t = estimate(cut, unused);
            if (t < least) {
                least = t;
                best = cut;
            }
        }
        a.sliced = best > 0;
        if (a.sliced) {
            a.slice_rows = best;
            if (window) a.long_blocks = (sinks + kKeys - 1) / kKeys;
            int most[2] = {1, 1};
            for (int j = 0; j < a.key_blocks; ++j) {
                const int cuts = list(j) > 0 ? (list(j) - 1) / best + 1 : 1;
                if (cuts > most[j < a.long_blocks]) most[j < a.long_blocks] = cuts;
            }
            a.slices = most[0];
            a.long_slices = most[1];
            a.slots = a.slices > 1 ? a.slices : 0;
            a.long_slots = a.long_slices > 1 ? a.long_slices : 0;
            a.long_tiles = 4 * a.long_blocks < tiles ? 4 * a.long_blocks : tiles;
            a.part_tiles = a.slots ? tiles : a.long_slots ? a.long_tiles : 0;
        }
    }
    // Sink segments: one wave per SIMD, no segment under 128 rows.
    if (!a.sliced && window && Tq > 0) a.sink_tiles = (sinks + 31) / 32;
    if (a.sink_tiles) {
        const long long even = heads * a.sink_tiles * a.rows / 1024;
        a.seg_rows = static_cast<int>(even < 128 ? 128 : even > a.rows ? a.rows : (even + 31) / 32 * 32);
        a.segs = (a.rows + a.seg_rows - 1) / a.seg_rows;
        a.part_tiles = a.long_tiles = a.sink_tiles;
        a.long_slots = 1 + a.segs;
    }
    return a;
}

}  // namespace attn
}  // namespace gdr
