// How a batch of sequences of any lengths is dealt out evenly to the workgroups of
// a decode step, and how the parts of shared units are joined.
//
// The visible keys of a sequence are cut into blocks.  The blocks of all
// (sequence, unit) pairs in a row (unit: key head and up to 16 query rows) are cut
// into equal shares, one per workgroup, found from the lengths alone.  A workgroup
// writes the units it holds whole, and leaves (m, l, O) of the at most two it
// shares with others to join_kernel, which joins them in order.
//
// A describes the step: B sequences, `shares` workgroups (0: units that are not
// shared, and no join), `heads` rows of a part, and
//   int per()                    units of a sequence
//   int blocks(int len)          blocks of a unit, 0 where the sequence is skipped by its length
//   bool skipped(b, len, table)  skipped for another reason (its blocks count all the same)
//   JoinRow row(int r)           output row r
#pragma once

#include "attn_common.h"

namespace gdr {
namespace attn {

struct JoinRow {
    int b, unit, slot;  // the sequence, its unit and the row of the unit
};

// The blocks of the batch in a row: sequence by sequence, within one unit by
// unit, per() units each.  A wave sums them 256 sequences at a time, four to a
// lane, so that their lengths come together.  The sums are formed in registers
// (shifts inside 16 lanes, then the sums of the 16 and 32 lanes before).
__device__ __forceinline__ int scan64(int x) {  // inclusive
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
    return x;
}
struct Blocks4 {
    int len[4], each[4], upto;  // of sequences at + 4 lane .. + 3; blocks of at .. and these
};
template <typename A>
__device__ __forceinline__ Blocks4 blocks_of(const A& a, int at, const int* __restrict__ lengths, int lane) {
    Blocks4 r;
    int sum = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) r.len[x] = at + 4 * lane + x < a.B ? lengths[at + 4 * lane + x] : -1;
#pragma unroll
    for (int x = 0; x < 4; ++x) sum += r.each[x] = a.blocks(r.len[x]);
    r.upto = scan64(sum);
    return r;
}
__device__ __forceinline__ int of4(const int (&v)[4], int x) { return x == 0 ? v[0] : x == 1 ? v[1] : x == 2 ? v[2] : v[3]; }
// Blocks of one unit per sequence: of the whole batch; of the sequences before b, of b itself, and b's length.
template <typename A>
__device__ __forceinline__ long long all_blocks(const A& a, const int* lengths, int lane, int b, long long& before, int& mine,
                                                int& len) {
    long long sum = 0;
    for (int at = 0; at < a.B; at += 256) {
        const Blocks4 r = blocks_of(a, at, lengths, lane);
        if (b >= at && b < at + 256) {
            const int x = b - at, rest = x & 3;
            int upto = r.upto;  // up to and with this lane's four, less those not before b
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (y >= rest) upto -= r.each[y];
            before = sum + __builtin_amdgcn_readlane(upto, x >> 2);
            mine = __builtin_amdgcn_readlane(of4(r.each, rest), x >> 2);
            len = __builtin_amdgcn_readlane(of4(r.len, rest), x >> 2);
        }
        sum += __builtin_amdgcn_readlane(r.upto, 63);
    }
    return sum;
}

// Shares in use: no share is empty, so a unit's parts are consecutive shares.
template <typename A> __device__ __forceinline__ int shares_of(const A& a, long long n) {
    return static_cast<int>(n < a.shares ? n : a.shares);
}
// a / b of non-negative numbers, in 32 bits where both fit (a fifth of the instructions).
__device__ __forceinline__ long long divide(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}
// The share that holds block g of n, share w being blocks [w n / W, (w+1) n / W).
__device__ __forceinline__ int owner(long long g, long long n, int W) {
    return static_cast<int>(divide((g + 1) * W - 1, n));
}

// A workgroup's blocks: [at_block, at_block + left) of unit `unit` of sequence b (of length len) and on.
struct Share {
    int b, len, unit, at_block, left;
};
// The share of workgroup `bid` (shares == 0: the unit `bid`); false: it has none.
template <typename A>
__device__ __forceinline__ bool find_share(const A& a, const int* __restrict__ lengths, int lane, int bid, Share& s) {
    const int per = a.per();
    if (a.shares == 0) {
        s.b = bid / per;
        s.len = __builtin_amdgcn_readfirstlane(lengths[s.b]);
        s.unit = bid - s.b * per;
        s.at_block = 0;
        s.left = a.blocks(s.len);
        return true;
    }
    long long n = 0;
    Blocks4 r;
    for (int at = 0; at < a.B; at += 256) {
        r = blocks_of(a, at, lengths, lane);
        n += __builtin_amdgcn_readlane(r.upto, 63);
    }
    n *= per;
    const int W = shares_of(a, n);
    if (bid >= W) return false;
    const long long lo = divide(n * bid, W), hi = divide(n * (bid + 1), W);
    s.left = static_cast<int>(hi - lo);
    long long before = 0;  // per unit
    for (int b = 0; b < a.B; b += 256) {  // the first sequence that ends after lo
        if (a.B > 256) r = blocks_of(a, b, lengths, lane);
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
            before += __builtin_amdgcn_readlane(upto, from);
            s.b = b + 4 * from + __builtin_amdgcn_readlane(x, from);
            s.len = __builtin_amdgcn_readlane(of4(r.len, x), from);
            const int blocks = __builtin_amdgcn_readlane(of4(r.each, x), from);
            const long long in = lo - before * per;
            s.unit = static_cast<int>(divide(in, max(1, blocks)));
            s.at_block = static_cast<int>(in - static_cast<long long>(s.unit) * blocks);
            return true;
        }
        before += __builtin_amdgcn_readlane(r.upto, 63);
    }
    return false;  // not reached unless the lengths change under the call
}

// Joins the parts of a shared unit, W waves per query head: part 0 is slot 1 of
// the unit's first share, the others slot 0 of the shares after it.  16 W parts
// at a time, lane s holding part s's weight 2^(m_s - max m); a wave adds every
// W-th part, the channels over its lanes, and the waves' sums are added in order.
template <typename T, int D, int W, typename A>
__global__ __launch_bounds__(256) void join_kernel(A a, int rows, const int* __restrict__ table,
                                                   const int* __restrict__ lengths,
                                                   const float* __restrict__ part_o,
                                                   const float* __restrict__ part_ml, T* __restrict__ o) {
    constexpr int N = D / 64, kEach = 16;
    __shared__ float sums[W > 1 ? W - 1 : 1][D];
    const int lane = threadIdx.x & 63, every = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = every % W;
    const int at = blockIdx.x * (4 / W) + every / W;
    if (at >= rows) return;
    const JoinRow jr = a.row(at);
    const int per = a.per();
    long long before = 0;
    int blocks = 0, len = -1;
    const long long n = per * all_blocks(a, lengths, lane, jr.b, before, blocks, len);
    if (blocks == 0 || a.skipped(jr.b, len, table)) return;
    const long long lo = per * before + static_cast<long long>(jr.unit) * blocks;
    const int used = shares_of(a, n), w0 = owner(lo, n, used), parts = owner(lo + blocks - 1, n, used) - w0 + 1;
    if (parts == 1) return;  // written whole
    auto slot = [&](int s) { return (static_cast<size_t>(w0 + s) * 2 + (s == 0)) * a.heads + jr.slot; };
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
    const size_t row = at;
#pragma unroll
    for (int e = 0; e < N; ++e) {
#pragma unroll
        for (int s = 0; s < W - 1; ++s) acc[e] += sums[s][N * lane + e];
        Elem<T>::store(o + row * D + N * lane + e, acc[e] * inv);
    }
}

// Parts in the workspace: O of every share's two slots, then (m, l).
template <typename A> size_t part_floats(const A& a, int d) { return static_cast<size_t>(a.shares) * 2 * a.heads * (d + 2); }

// The launch of `step` (a decode kernel of `blocks` workgroups) and of the join behind it.
// `rows` output rows; `most` blocks that a unit can have at most.
template <typename T, int D, typename A, typename F>
hipError_t launch_dealt(const A& a, unsigned long long blocks, unsigned long long rows, unsigned long long most, int threads,
                        const int* table, const int* lengths, void* o, float* ws, hipStream_t st, F step) {
    const unsigned long long units = static_cast<unsigned long long>(a.B) * a.per();
    // a share's blocks have to fit an int, and so have those of one scan's sequences
    if (a.shares && (units * most / a.shares > 0x7fffffffull || (a.B < 256 ? a.B : 256) * most > 0x7fffffffull))
        return hipErrorInvalidConfiguration;
    if (!grid_fits(blocks, threads) || !grid_fits(rows, 256)) return hipErrorInvalidConfiguration;
    float* part_o = ws;
    float* part_ml = ws ? ws + static_cast<size_t>(a.shares) * 2 * a.heads * D : nullptr;
    const hipError_t e = step(static_cast<unsigned>(blocks), part_o, part_ml);
    if (e != hipSuccess || a.shares == 0) return e;
    // Many rows have few parts each and take a wave (64 sequences of 32: 5.7 against 10.9 us), few rows four.
    const bool many = rows >= 1024;
    auto* join = many ? join_kernel<T, D, 1, A> : join_kernel<T, D, 4, A>;
    hipLaunchKernelGGL(join, dim3(static_cast<unsigned>(many ? (rows + 3) / 4 : rows)), dim3(256), 0, st, a,
                       static_cast<int>(rows), table, lengths, part_o, part_ml, static_cast<T*>(o));
    return hipGetLastError();
}

}  // namespace attn
}  // namespace gdr
