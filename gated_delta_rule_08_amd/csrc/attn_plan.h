// How workgroups are numbered, for the attention kernels and for the host.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {
namespace attn {

// n / d for 0 <= n < 2^31 by one multiplication: with 2^s >= d the smallest
// such power and m = ceil(2^(31+s) / d), n m / 2^(31+s) exceeds n / d by less
// than n / 2^31 / d < 1 / d, so its floor is exact.
struct FastDiv {
    uint32_t mul, shift;
    int d;
    __host__ FastDiv(int div = 1) : d(div) {
        int s = 0;
        while ((1ll << s) < div) ++s;
        mul = static_cast<uint32_t>(((1ull << (31 + s)) + div - 1) / div);
        shift = 31 + s;
    }
    __host__ __device__ __forceinline__ int operator()(int n) const {
        return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
    }
};

// Which of `tiles` pieces of work (rank 0 the longest) of which head workgroup
// bid takes.  Workgroups go round the 8 XCDs: a head's pieces stay on one, whose
// L2 then holds what they share, the longest first.  Where all fit at once, two
// to a CU (32 CUs to an XCD, filled in turn), the second round goes backwards,
// so that a long piece shares its CU with a short one.
__host__ __device__ __forceinline__ void place(int bid, int heads, int tiles, int& head, int& rank) {
    if (heads % 8 == 0) {
        const int y = bid >> 3, here = heads >> 3, all = here * tiles;
        if (all > 32 && all <= 64) {
            const int r = y < 32 ? y : all - 1 - (y - 32);
            rank = r / here;
            head = (r - rank * here) * 8 + (bid & 7);
        } else {
            head = (y / tiles) * 8 + (bid & 7);
            rank = y % tiles;
        }
    } else {
        const int all = heads * tiles, r = all > 256 && all <= 512 && bid >= 256 ? all - 1 - (bid - 256) : bid;
        head = r % heads;
        rank = r / heads;
    }
}

}  // namespace attn
}  // namespace gdr
