/*
 * The plan of the attention backward against its definition, on the host: which
 * rows every wave takes, for many sizes.  Built host-only with
 * UndefinedBehaviorSanitizer, so that an overflow ends the program too.
 * Prints "all checks passed" and returns 0, or names what failed and returns 1.
 */
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <utility>
#include <vector>

#include "attn_backward_plan.h"

using namespace gdr::attn;

namespace {

struct Case {
    int f32, B, Tq, Tk, Hq, Hkv, d, window, sinks;
};

int failures = 0;
void fail(const Case& c, const char* what, long long x = 0, long long y = 0) {
    if (++failures <= 20)
        fprintf(stderr, "%s (%lld, %lld): f32 %d B %d Tq %d Tk %d heads %d/%d d %d window %d sinks %d\n", what, x, y, c.f32,
                c.B, c.Tq, c.Tk, c.Hq, c.Hkv, c.d, c.window, c.sinks);
}

BwdArgs plan(Case& c) {  // as the library calls it: a window that hides nothing is none
    if (c.window >= c.Tk) c.window = 0;
    c.sinks = c.window == 0 ? 0 : std::min(c.sinks, c.Tk);
    return make_args(c.f32, c.B, c.Tq, c.Tk, c.Hq, c.Hkv, c.d, c.window, c.sinks, 1.f);
}

// Queries that see one of the keys j0 .. j1 through the window (not as sinks), as [lo, hi) rows, in 64 bits.
void rows_exact(const BwdArgs& a, long long j0, long long j1, long long& lo, long long& hi) {
    const long long off = static_cast<long long>(a.Tk) - a.Tq;
    long long first = std::max(0LL, j0 - off), last = a.Tq - 1LL;
    if (a.window) last = std::min(last, j1 + a.window - 1 - off);
    lo = first * a.G.d;
    hi = std::max(lo, (last + 1) * a.G.d);
    if (a.sliced && a.window && j0 < a.sinks) hi = a.rows;
}

void check_lists(Case c) {
    const BwdArgs a = plan(c);
    for (int j = 0; j < a.key_blocks; j += j < 600 || j + 700 > a.key_blocks ? 1 : 997) {
        const int j0 = j * kKeys, j1 = std::min(j0 + kKeys, a.Tk) - 1;
        int lo, hi;
        long long l, h;
        rows_of(a, j0, j1, lo, hi);
        rows_exact(a, j0, j1, l, h);
        if (lo < 0 || hi > std::max(a.rows, lo)) fail(c, "rows out of range", lo, hi);
        if (std::min<long long>(h, a.rows) - l > 0 ? lo != l || hi != h : hi > lo) fail(c, "rows of a key block", j, hi);
    }
}

// Every visible (row, key) pair is in exactly one piece of its key's tile.
template <int WAVES> void gather(const BwdArgs& a, int blocks, std::vector<std::vector<std::pair<int, int>>>& got, const Case& c) {
    for (int bid = 0; bid < blocks; ++bid)
        for (int wave = 0; wave < WAVES; ++wave) {
            const Piece p = piece_of<WAVES>(a, bid, wave);
            if (p.j0 >= a.Tk || p.lo >= p.hi) continue;
            if (p.head < 0 || p.head >= a.B * a.Hkv || p.tile < 0 || p.lo < 0 || p.hi > a.rows) {
                fail(c, "piece out of range", p.lo, p.hi);
                continue;
            }
            got[static_cast<size_t>(p.head) * ((a.Tk + 31) / 32) + p.tile].push_back({p.lo, p.hi});
        }
}

void check_cover(Case c) {
    const BwdArgs a = plan(c);
    const int heads = c.B * c.Hkv, tiles = (c.Tk + 31) / 32;
    std::vector<std::vector<std::pair<int, int>>> main(static_cast<size_t>(heads) * tiles), segs(main.size());
    gather<kWaves>(a, heads * a.cuts(), main, c);
    gather<1>(a, heads * a.sink_tiles * a.segs, segs, c);
    for (int head = 0; head < heads; ++head)
        for (int tile = 0; tile < tiles; ++tile) {
            auto &m = main[static_cast<size_t>(head) * tiles + tile], &s = segs[static_cast<size_t>(head) * tiles + tile];
            std::vector<std::pair<int, int>> all(m);
            all.insert(all.end(), s.begin(), s.end());
            std::sort(all.begin(), all.end());
            std::sort(m.begin(), m.end());
            for (size_t i = 1; i < all.size(); ++i)
                if (all[i].first < all[i - 1].second) fail(c, "two pieces with the same rows", head, tile);
            for (int key = 32 * tile; key < std::min(c.Tk, 32 * tile + 32); ++key) {
                const long long off = static_cast<long long>(c.Tk) - c.Tq, first = std::max(0LL, key - off) * a.G.d;
                long long last = a.rows;
                if (a.window && key >= a.sinks) last = std::min(last, (key + a.window - off) * a.G.d);
                long long at = first;
                for (const auto& p : key < a.sinks ? all : m)  // the segments' other keys are not read
                    if (p.first <= at && p.second > at) at = p.second;
                if (at < last) fail(c, "rows of a key in no piece", key, at);
            }
        }
}

// The parts of the key tiles that have any lie apart from each other and inside the workspace, which is bounded.
void check_parts(Case c) {
    const BwdArgs a = plan(c);
    const long long heads = static_cast<long long>(c.B) * c.Hkv;
    const double bytes = static_cast<double>(heads) * a.head_parts * 64 * c.d * 4;
    const double sinks = 2.0 * heads * ((c.sinks + 31) / 32) * 64 * c.d * 4 + (32 << 20);
    if (bytes > std::max(256.0 * (1 << 20), sinks)) fail(c, "workspace of the parts", static_cast<long long>(bytes));
    if (c.Tq > 3000 || c.Tk > 5000) return;
    std::vector<long long> used(heads * a.head_parts, -1);
    if (a.sliced && a.part_blocks > kSliced) fail(c, "slots of too many blocks");
    auto at_of = [&](int head, int tile, int slot) {  // as part_of has it
        return static_cast<long long>(head) * a.head_parts + (a.sliced ? 4 * a.slots_before(tile >> 2) : tile & ~3) +
               static_cast<long long>(slot) * a.part_step + (tile & 3);
    };
    auto take = [&](int head, int tile, int slot, bool read) {
        const long long at = at_of(head, tile, slot);
        if (tile >= a.part_tiles || at < 0 || at >= static_cast<long long>(used.size())) return fail(c, "part out of range", tile, slot);
        const long long me = (static_cast<long long>(head) * a.part_tiles + tile) * 100000 + slot;
        if (read ? used[at] != me : used[at] >= 0) fail(c, "part of another", tile, slot);
        used[at] = me;
        if (at - at_of(head, tile, 0) != static_cast<long long>(slot) * a.part_step) fail(c, "distance of parts", tile, slot);
    };
    for (int bid = 0; bid < heads * a.cuts(); ++bid)
        for (int wave = 0; wave < kWaves; ++wave) {
            const Piece p = piece_of<kWaves>(a, bid, wave);
            if (p.j0 < a.Tk && (p.cut == 0 || p.lo < p.hi) && (p.parts || p.tile < a.sink_tiles)) take(p.head, p.tile, p.cut, false);
        }
    for (int bid = 0; bid < heads * a.sink_tiles * a.segs; ++bid) {
        const Piece p = piece_of<1>(a, bid, 0);
        if (p.lo < p.hi) take(p.head, p.tile, 1 + p.cut, false);
    }
    // what the join reads: as many parts as a tile's list has slices, from the first
    for (int head = 0; head < heads; ++head)
        for (int tile = 0; tile < a.part_tiles; ++tile) {
            const int m0 = 32 * tile / kKeys * kKeys;
            int lo, hi, n = 1;
            rows_of(a, m0, std::min(m0 + kKeys, a.Tk) - 1, lo, hi);
            if (a.sliced) {
                const int size = slice_of(a, hi - lo);
                n = hi - lo <= size ? 0 : (hi - lo - 1) / size + 1;
            } else if (a.segs && a.rows > hi) {
                n += (a.rows - hi - 1) / a.seg_rows + 1;
            }
            for (int slot = 0; slot < n; ++slot) take(head, tile, slot, true);
        }
}

unsigned long long state = 1;
int pick(int n) {
    state = state * 6364136223846793005ULL + 1442695040888963407ULL;
    return static_cast<int>((state >> 33) % static_cast<unsigned>(n));
}

}  // namespace

int main() {
    // sizes at the documented limits: 2^15 heads, fewer than 2^29 rows in a sequence
    const Case large[] = {
        {0, 1, 1, 1 << 28, 1 << 15, 1, 64, 1, 0},          {0, 1, 1, (1 << 29) - 1, 1 << 15, 1, 64, 100, 3},
        {0, 1, 1000, 1 << 24, 128, 1, 128, 64, 0},         {1, 1, 16383, 1 << 28, 1 << 15, 1, 64, 4096, 9},
        {0, 1, (1 << 14) - 1, 65000, 1 << 15, 1, 64, 5, 0}, {0, 1, (1 << 14) - 1, 65000, 1 << 15, 1, 64, 0, 0},
        {0, 1, (1 << 29) - 1, 300, 1, 1, 64, 0, 0},        {0, 1, (1 << 29) - 1, 70000, 1, 1, 64, 1000, 900},
        {0, 1, (1 << 29) - 1, (1 << 29) - 1, 1, 1, 128, 7, 1 << 28},
        {0, 1, 1 << 16, 1 << 26, 1 << 12, 4, 64, 1 << 20, 77},
    };
    for (const Case& c : large) {
        check_lists(c);
        check_parts(c);
    }
    // few heads and long sequences, where lists are sliced, up to and past the 512 key blocks
    for (int T : {300, 4096, 16384, 65408, 65536})
        for (int g : {1, 8, 32, 128})
            for (int hkv : {1, 2, 8})
                for (int window : {0, 64, 4096})
                    for (int sinks : {0, 4, 5000}) check_parts({g == 8, 1, T, T, g * hkv, hkv, 128, window, sinks});
    const int group[] = {1, 1, 2, 3, 4, 5, 8, 16, 40};
    for (int i = 0; i < 700; ++i) {
        Case c{};
        c.f32 = pick(2);
        c.B = 1 + pick(i % 3 == 0 ? 40 : 2);
        c.Hkv = 1 + pick(i % 5 == 0 ? 16 : 3);
        c.Hq = c.Hkv * group[pick(9)];
        c.d = 64 << pick(2);
        c.Tq = pick(i % 4 == 0 ? 3000 : 300);
        c.Tk = pick(3) == 0 ? pick(1200) : c.Tq + pick(2) * pick(700);
        c.window = pick(2) * (1 + pick(1 + c.Tk));
        c.sinks = pick(3) == 0 ? pick(1 + c.Tk) : pick(6);
        check_lists(c);
        check_cover(c);
        check_parts(c);
    }
    if (failures) {
        fprintf(stderr, "%d checks failed\n", failures);
        return 1;
    }
    printf("all checks passed\n");
    return 0;
}
