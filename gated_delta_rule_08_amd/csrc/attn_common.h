// Device code shared by the attention kernels (prefill, backward, paged decode).
//
// Every product is a matrix-core tile whose operand fragment is 8 consecutive
// elements of the contracted axis per lane.  For bf16 that is one
// instruction (32x32x16 or 16x16x32); for fp32 the same fragment goes through
// eight fp32 instructions (32x32x2 or 16x16x4), each taking element i of
// every lane: the contracted axis is only summed over, so the two operands
// agreeing on its order is all that is needed, and one kernel body serves
// both types.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_plan.h"
#include "gdr_internal.h"

namespace gdr {
namespace attn {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef short s16x4v __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T> struct Frag;
template <> struct Frag<bf16_t> { typedef bf16x8v type; typedef __bf16 elem; };
template <> struct Frag<float> { typedef f32x8 type; typedef float elem; };
template <typename T> using frag_t = typename Frag<T>::type;

__device__ __forceinline__ f32x16 zero16() {
    return f32x16{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
}

// D[row][col] += sum over 16 elements of A[row][.] B[col][.].  A: row = lane
// % 32; B: col = lane % 32; lane / 32 picks the half of the contracted axis.
// D: col = lane % 32, register r is row (r / 4) * 8 + (lane / 32) * 4 + r % 4.
__device__ __forceinline__ f32x16 mma32(const bf16x8v& a, const bf16x8v& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma32(const f32x8& a, const f32x8& b, f32x16 c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ constexpr int row32(int r, int h) { return (r >> 2) * 8 + h * 4 + (r & 3); }

// D[row][col] += sum over 32 elements (8 per quarter lane / 16).  A: row =
// lane % 16; B: col = lane % 16.  D: col = lane % 16, register r is row
// (lane / 16) * 4 + r.
__device__ __forceinline__ f32x4 mma16(const bf16x8v& a, const bf16x8v& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma16(const f32x8& a, const f32x8& b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
}

template <typename T> __device__ __forceinline__ frag_t<T> zero_frag();
template <> __device__ __forceinline__ bf16x8v zero_frag<bf16_t>() {
    return __builtin_bit_cast(bf16x8v, make_uint4(0u, 0u, 0u, 0u));
}
template <> __device__ __forceinline__ f32x8 zero_frag<float>() {
    return f32x8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
}

// 8 consecutive elements from global memory (16-byte aligned).
__device__ __forceinline__ bf16x8v load8(const bf16_t* p) {
    return __builtin_bit_cast(bf16x8v, *reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ f32x8 load8(const float* p) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// fp32 values as an operand fragment (bf16: rounded to nearest even; a
// probability or a score gradient then carries a relative error of at most
// 2^-8, the size of the rounding of the inputs and of the output).
template <typename T> __device__ __forceinline__ frag_t<T> pack8(const float (&x)[8]);
template <> __device__ __forceinline__ bf16x8v pack8<bf16_t>(const float (&x)[8]) {
    bf16x8v r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = static_cast<__bf16>(x[i]);
    return r;
}
template <> __device__ __forceinline__ f32x8 pack8<float>(const float (&x)[8]) {
    f32x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
    return r;
}

// Registers 8u .. 8u+7 of an accumulator tile as an operand fragment.
template <typename T> __device__ __forceinline__ frag_t<T> pack_regs(const f32x16& s, int u) {
    float x[8];
#pragma unroll
    for (int y = 0; y < 8; ++y) x[y] = s[8 * u + y];
    return pack8<T>(x);
}

template <typename T> __device__ __forceinline__ void store4(T* p, float a, float b, float c, float d);
template <> __device__ __forceinline__ void store4<float>(float* p, float a, float b, float c, float d) {
    *reinterpret_cast<f32x4*>(p) = f32x4{a, b, c, d};
}
template <> __device__ __forceinline__ void store4<bf16_t>(bf16_t* p, float a, float b, float c, float d) {
    const bf16x4v r = {static_cast<__bf16>(a), static_cast<__bf16>(b), static_cast<__bf16>(c),
                       static_cast<__bf16>(d)};
    *reinterpret_cast<uint2*>(p) = __builtin_bit_cast(uint2, r);
}

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float lg2(float x) { return __builtin_amdgcn_logf(x); }

// acc += A B over 32 elements as two mma32 would, summing the pairs whose bit in
// `seen` is set and no others: a hidden pair's weight is 0, but 0 times an
// infinity or NaN would be NaN.  B: the lane's 16 weights w (an accumulator
// tile); A: column lane % 32 of the rows row(0) .. row(31), in global memory.
// Infinities and NaN of A are counted, by products of their signs with those of
// the weights, and added afterwards as the sum over the visible pairs has them.
template <typename T, typename F>
__device__ __forceinline__ void mma32_seen(f32x16& acc, F row, const f32x16& w, uint32_t seen, int lane) {
    typedef typename Frag<T>::elem elem;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        __builtin_amdgcn_sched_barrier(0);  // one half's registers at a time
        frag_t<T> fin, sign, mag, nan;
        float wv[8], ws[8], wm[8], w0[8], vis[8];
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const elem a = __builtin_bit_cast(elem, row(16 * x + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3))[lane & 31]);
            const float af = static_cast<float>(a);
            const bool see = (seen >> (8 * x + i)) & 1, is_nan = af != af, is_inf = fabsf(af) == INFINITY;
            const float s = is_inf ? (af > 0.f ? 1.f : -1.f) : 0.f;
            odd |= is_nan || is_inf;
            fin[i] = is_nan || is_inf ? static_cast<elem>(s) : a;
            sign[i] = static_cast<elem>(s);
            mag[i] = static_cast<elem>(fabsf(s));
            nan[i] = static_cast<elem>(is_nan ? 1.f : 0.f);
            wv[i] = see ? w[8 * x + i] : 0.f;
            ws[i] = wv[i] > 0.f ? 1.f : wv[i] < 0.f ? -1.f : 0.f;
            wm[i] = fabsf(ws[i]);
            vis[i] = see ? 1.f : 0.f;
            w0[i] = see && wv[i] == 0.f ? 1.f : 0.f;
        }
        acc = mma32(fin, pack8<T>(wv), acc);
        if (!__any(odd)) continue;
        const f32x16 z1 = mma32(sign, pack8<T>(ws), zero16()), z2 = mma32(mag, pack8<T>(wm), zero16());
        const f32x16 z3 = mma32(mag, pack8<T>(w0), mma32(nan, pack8<T>(vis), zero16()));
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            if (z2[r] > 0.f) acc[r] += z1[r] == z2[r] ? INFINITY : z1[r] == -z2[r] ? -INFINITY : NAN;
            if (z3[r] > 0.f) acc[r] = NAN;
        }
    }
}

// x of the lane 32 away.
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

// x as a value the compiler knows nothing about: addresses formed from it are
// formed again instead of being kept in registers from their last use.
__device__ __forceinline__ int again(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// ---------------------------------------------------------------- LDS tiles
//
// A tile holds rows of D elements in 16-byte units; unit u of row r sits at
// unit position u ^ swz(r).  Two reads have to be free of bank conflicts:
//  - row fragments: 32 lanes read the same unit of 32 rows, the upper 32
//    lanes the next unit; lanes 8b.. and 8(b ^ 7).. share a cycle;
//  - transposing reads (bf16): 4 lane groups of 16 read 8-byte pieces of 4
//    rows each, 64 bytes wide.
// Rows 0..3 therefore differ in the 64-byte block (bits 2..3 of the unit for
// 256-byte rows, bit 2 for pairs of 128-byte rows) and rows 4..15 in the unit
// inside it.  swz depends on row % 16 only and a row's units are a power of
// two, so an address is (lane's base) ^ constant + constant: a lane keeps one
// base per kind of read.
template <typename T, int D> struct Tile {
    static constexpr int kRow = D * static_cast<int>(sizeof(T));  // bytes
    static constexpr int kUnits = kRow / 16;
    __device__ __forceinline__ static constexpr int swz(int row) {
        return kUnits == 8 ? (((row >> 1) & 1) << 2) | ((row >> 2) & 3) : ((row & 3) << 2) | ((row >> 2) & 3);
    }
    // byte offset of unit 0 of row r; unit u is at this ^ (u << 4)
    __device__ __forceinline__ static int at(int row) { return row * kRow + (swz(row) << 4); }
};

// Row fragment: the 8 elements 8g .. 8g+7 of a row, base = Tile::at(row) (+ a
// multiple of 2^k >= a row: the tile's place in LDS), imm = a constant number of 16-row steps in bytes.
template <typename T, int D> struct RowRead;
template <int D> struct RowRead<bf16_t, D> {
    __device__ __forceinline__ static int base(int row, int h) { return Tile<bf16_t, D>::at(row) ^ (h << 4); }
    // element group 2 e + h
    __device__ __forceinline__ static bf16x8v get(const unsigned char* lds, int base, int e, int imm) {
        return __builtin_bit_cast(bf16x8v, *reinterpret_cast<const uint4*>(lds + (base ^ (e << 5)) + imm));
    }
};
template <int D> struct RowRead<float, D> {
    __device__ __forceinline__ static int base(int row, int h) { return Tile<float, D>::at(row) ^ (h << 5); }
    __device__ __forceinline__ static f32x8 get(const unsigned char* lds, int base, int e, int imm) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(lds + (base ^ (e << 6)) + imm);
        const f32x4 b = *reinterpret_cast<const f32x4*>(lds + (base ^ (e << 6) ^ 16) + imm);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// Column fragment: lane (c = lane % 32, h = lane / 32) gets column 32 t + c of
// the 8 rows {4h..4h+3, 8+4h..8+4h+3} of 16-row step x: the order in which the
// registers of an accumulator tile hold its rows, so that those registers are
// the other operand as they stand.
//
// bf16: transposing reads.  The 16 lanes of a group address 4 rows (lr / 4) at
// 4 column quads (lr % 4); lane lr receives column lr of the 4 rows.
template <typename T, int D> struct ColRead;
template <int D> struct ColRead<bf16_t, D> {
    using L = Tile<bf16_t, D>;
    __device__ __forceinline__ static int base(int lane) {
        const int h = lane >> 5, g = (lane >> 4) & 1, lr = lane & 15;
        return (L::at(4 * h + (lr >> 2)) ^ ((2 * g + ((lr >> 1) & 1)) << 4)) + 8 * (lr & 1);
    }
    __device__ __forceinline__ static bf16x8v get(const unsigned char* lds, int base, int t, int x) {
        typedef __attribute__((address_space(3))) s16x4v lds_s16x4;
        const unsigned char* lo = lds + (base ^ (t << 6)) + 16 * x * L::kRow;
        const unsigned char* hi = lds + (base ^ (t << 6) ^ 32) + (16 * x + 8) * L::kRow;
        const s16x4v a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lo));
        const s16x4v b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(hi));
        return __builtin_shufflevector(__builtin_bit_cast(bf16x4v, a), __builtin_bit_cast(bf16x4v, b), 0, 1, 2, 3,
                                       4, 5, 6, 7);
    }
};
template <int D> struct ColRead<float, D> {
    using L = Tile<float, D>;
    __device__ __forceinline__ static int base(int lane) {
        const int h = lane >> 5, c = lane & 31;
        return (L::at(4 * h) ^ ((c >> 2) << 4)) + 4 * (c & 3);
    }
    __device__ __forceinline__ static f32x8 get(const unsigned char* lds, int base, int t, int x) {
        f32x8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i)  // row 8 (i / 4) + 4 h + i % 4
            r[i] = *reinterpret_cast<const float*>(lds + (base ^ (t << 7) ^ ((i & 3) << 6) ^ ((i >> 2) << 5)) +
                                                   (16 * x + 8 * (i >> 2) + (i & 3)) * L::kRow);
        return r;
    }
};

// Copies straight from global memory to LDS, one instruction of a wave: lane
// by lane, 16 bytes each into 1024 consecutive bytes (4 bytes each into 256).
// They are written as assembly because the compiler would wait for a copy
// before any later LDS read that it cannot tell apart from it, which is every
// read of the other buffer: the kernels wait themselves (vmcnt, before the
// barrier or the read that needs the copy).  They return nothing in registers.
// M0, the destination, is a reserved register that the compiler takes no clobber
// for; nothing else in these kernels uses it (tests/test_attn_m0.py reads the
// compiled code).
// lds: wave-uniform byte address in LDS (lds_addr).
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}
__device__ __forceinline__ void copy_1k_from(uint32_t lds, const void* p) {  // an address per lane
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void copy_words(uint32_t lds, const void* base, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(off), "s"(base)
                 : "memory");
}
__device__ __forceinline__ void stream_1k(uint32_t lds, const void* p) {  // the same, not to be kept in the caches
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" ::"s"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void gather_words(uint32_t lds, const void* p) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory");
}

// This wave's copies and loads have landed, its LDS accesses are done, and every
// wave has come this far: buffers filled before may be read, buffers read
// before may be refilled.
__device__ __forceinline__ void tile_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A wave's copies of a tile of ROWS rows: an instruction fills 1024 / row bytes
// rows, each lane fetching the unit that belongs at its place.  The lanes'
// offsets from the tile's first row are formed once; where a tile's rows exist
// and follow one another, a step costs no address arithmetic but the base's.
// The kernels wait for the copies (vmcnt) and pass a barrier before reading.
template <typename T, int D, int ROWS, int WAVES> struct TileCopy {
    using L = Tile<T, D>;
    static constexpr int kPer = 1024 / L::kRow, kCopies = ROWS / kPer / WAVES;
    static_assert(1024 % L::kRow == 0 && kPer * kCopies * WAVES == ROWS, "whole rows, the same number for every wave");
    // copies a multiple of 16 rows apart have the same swizzle and share an offset
    static constexpr bool kShared = kPer * WAVES % 16 == 0;
    static constexpr int kOffsets = kShared ? 1 : kCopies;
    uint32_t off[kOffsets], apart;
    int wave, lane;
    // offset(r): bytes from the tile's first row to row r; rows kPer * WAVES
    // apart are the same number of bytes apart everywhere
    template <typename F> __device__ __forceinline__ TileCopy(int wave_, int lane_, F offset) : wave(wave_), lane(lane_) {
#pragma unroll
        for (int j = 0; j < kOffsets; ++j) off[j] = static_cast<uint32_t>(offset(row(j))) + unit(j);
        apart = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(offset(kPer * WAVES)));
    }
    __device__ __forceinline__ int row(int j) const { return (wave + j * WAVES) * kPer + lane / L::kUnits; }
    __device__ __forceinline__ uint32_t unit(int j) const { return ((lane % L::kUnits) ^ L::swz(row(j))) << 4; }
    __device__ __forceinline__ void run(uint32_t tile, const void* base) const {
        const uint32_t at = tile + wave * 1024;
#pragma unroll
        for (int j = 0; j < kCopies; ++j) {
            const void* from = kShared ? static_cast<const unsigned char*>(base) + j * apart : base;
            asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at),
                         "v"(off[kShared ? 0 : j]), "s"(from), "n"(j * WAVES * 1024)
                         : "memory", "scc");
        }
    }
    // any other tile: address(r) is row r's
    template <typename F> __device__ __forceinline__ void gather(uint32_t tile, F address) const {
#pragma unroll
        for (int j = 0; j < kCopies; ++j)
            copy_1k_from(tile + (wave + j * WAVES) * 1024, reinterpret_cast<const unsigned char*>(address(row(j))) + unit(j));
    }
};

// The keys that the rows of a workgroup may see, as one list: the sinks before
// the window of its first row, then everything from there to its last row's
// position.  Tiles are cut from the list, so neither the sinks nor a window that
// starts anywhere cost a tile of their own.
struct KeyList {
    int sinks;  // keys 0 .. sinks-1 come first
    int jump;   // entry x >= sinks is key x + jump
    int count;
    // rows at positions p0 .. p1 (p1 < 0: no keys)
    __device__ __forceinline__ KeyList(int window, int sink_keys, int p0, int p1) {
        const int lo = window ? max(0, p0 - window + 1) : 0;
        sinks = min(sink_keys, lo);
        jump = lo - sinks;
        count = p1 < 0 ? 0 : p1 - jump + 1;
    }
    __device__ __forceinline__ int key(int x) const { return x < sinks ? x : x + jump; }
};

// Tiles of BN entries of a list, as a wave looks at them (its 32 NS keys of a
// tile begin at entry `sub`, its rows are at positions p0 .. p1).
struct TileRange {
    int full_lo, full_hi;    // tiles whose keys follow one another and exist
    int whole_lo, whole_hi;  // tiles that every row sees all of
    int end;                 // tiles from here on no row sees
    template <int BN, int SPAN>
    static __device__ __forceinline__ TileRange of(const KeyList& keys, int window, int Tk, int sub, int p0, int p1) {
        static_assert((BN & (BN - 1)) == 0, "shifts floor, also below zero");
        constexpr int lg = __builtin_ctz(BN);
        TileRange t;
        t.full_lo = (keys.sinks + BN - 1) >> lg;
        t.full_hi = (Tk - keys.jump) >> lg;
        t.whole_lo = (keys.sinks - sub + BN - 1) >> lg;
        if (window) t.whole_lo = max(t.whole_lo, (p1 - window + 1 - keys.jump - sub + BN - 1) >> lg);
        t.whole_hi = ((p0 + 1 - SPAN - keys.jump - sub) >> lg) + 1;
        t.end = ((p1 - keys.jump - sub) >> lg) + 1;
        return t;
    }
};

// Keys and queries of one sequence.  Query i is at position i + off; key j is
// visible to position p if j <= p and (window == 0 or j > p - window or j <
// sinks).  window is at most the number of keys, so p + window cannot wrap.
struct Mask {
    int window, sinks;
    __device__ __forceinline__ bool sees(int p, int j) const {
        return j <= p && (window == 0 || j > p - window || j < sinks);
    }
};

}  // namespace attn
}  // namespace gdr
