// The page plan of a serving step: page table rows, token offsets and slots of a
// batch of requests, from their lengths and the tokens each is to add.
//
// A request of len tokens that adds n needs ceil((len + n) / page) - ceil(len / page)
// pages.  They are taken from the top of a stack, request by request, until the
// first that the stack or the step's tokens do not suffice for.  Two prefix sums
// over the requests say who is served, where its tokens lie in the packed batch
// and which pages are its own: one workgroup, as the sums are short and the rest
// waits for them.  The slots, one for each token, are found by the same workgroup
// where a step has few, else in a second launch.  Bound by the latency of the loads
// and of the sums: 256 requests of one token each 5.3 us (two launches: 6.8), 64 of up
// to 4096 tokens 7.8.
#include "gdr_internal.h"

namespace gdr {
namespace attn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFewTokens = 4096;  // of a step at most, for slots without a second launch

struct PlanArgs {
    int N, page_shift, max_pages, n_stack, max_tokens;
};

// Inclusive sums of two values over the workgroup.
__device__ __forceinline__ void scan2(long long& x, long long& y, long long (*part)[2]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const long long u = __shfl_up(x, s), v = __shfl_up(y, s);
        if (lane >= s) {
            x += u;
            y += v;
        }
    }
    if (lane == 63) {
        part[wave][0] = x;
        part[wave][1] = y;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        x += part[w][0];
        y += part[w][1];
    }
}

// The last i < kPlanThreads with from[i] <= e (from[0] is).
__device__ __forceinline__ int last_from(const int* from, int e) {
    int i = 0;
#pragma unroll
    for (int s = kPlanThreads / 2; s; s >>= 1)
        if (from[i + s] <= e) i += s;
    return i;
}
__device__ __forceinline__ int slot_of(int page, int pos, int page_shift) {
    // no page, or one whose slots an int does not hold
    return page < 0 || page > (0x7fffffff >> page_shift) ? -1 : (page << page_shift) + (pos & ((1 << page_shift) - 1));
}

// slots: NULL, or where the step's tokens go (few of them).
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs a, const int* lengths, const int* add,
                                                            const int* __restrict__ free_pages, const int* n_free,
                                                            int* __restrict__ table, int* __restrict__ cu, int* added,
                                                            int* lengths_out, int* __restrict__ slots, int* n_free_out) {
    __shared__ long long part[kPlanThreads / 64][2];
    __shared__ int first[kPlanThreads], held[kPlanThreads], begin[kPlanThreads], length[kPlanThreads];
    __shared__ long long all[2], given[2];  // sums up to here: of every request, and of those served
    const int tid = threadIdx.x;
    const int stack = min(max(*n_free, 0), a.n_stack), page = 1 << a.page_shift;
    const long long room = static_cast<long long>(a.max_pages) << a.page_shift;
    if (tid == 0) {
        all[0] = all[1] = given[0] = given[1] = 0;
        cu[0] = 0;
    }
    __syncthreads();
    for (long long at = 0; at < a.N; at += kPlanThreads) {  // up to 2^31 - 2 requests: at passes an int behind the last
        const long long n = at + tid;
        const long long len = n < a.N ? lengths[n] : -1, want = n < a.N ? add[n] : 0;
        const bool fine = len >= 0 && want >= 0 && len + want <= room;
        const long long have = fine ? (len + page - 1) >> a.page_shift : 0;
        const long long need = fine ? ((len + want + page - 1) >> a.page_shift) - have : 0;
        const long long tokens = fine ? want : 0;
        long long p = need, t = tokens;
        scan2(p, t, part);
        const long long taken = given[0], before = given[1];
        p += all[0];
        t += all[1];
        const bool fits = p <= stack && t <= a.max_tokens;  // once false it stays so
        __syncthreads();
        if (tid == kPlanThreads - 1) {
            all[0] = p;
            all[1] = t;
        }
        // the last request that fits has the sums of all that are served
        const int served = __syncthreads_count(fits);
        if (fits && tid == served - 1) {
            given[0] = p;
            given[1] = t;
        }
        __syncthreads();
        const long long total = given[0];
        first[tid] = static_cast<int>((fits ? p - need : total) - taken);
        held[tid] = static_cast<int>(have);
        begin[tid] = static_cast<int>((fits ? t - tokens : given[1]) - before);
        length[tid] = static_cast<int>(len);
        if (n < a.N) {
            cu[n + 1] = static_cast<int>(fits ? t : given[1]);
            added[n] = fits ? static_cast<int>(tokens) : 0;
            lengths_out[n] = static_cast<int>(len) + (fits ? static_cast<int>(tokens) : 0);
        }
        __syncthreads();
        for (int e = tid; e < static_cast<int>(total - taken); e += kPlanThreads) {  // page by page
            const int i = last_from(first, e);
            const size_t to = static_cast<size_t>(at + i) * a.max_pages + held[i] + (e - first[i]);
            table[to] = free_pages[stack - 1 - static_cast<int>(taken) - e];
        }
        if (slots) {
            for (int e = tid; e < static_cast<int>(given[1] - before); e += kPlanThreads) {  // token by token
                const int i = last_from(begin, e), pos = length[i] + e - begin[i], x = pos >> a.page_shift;
                const int page = x >= held[i] ? free_pages[stack - 1 - static_cast<int>(taken) - first[i] - (x - held[i])]
                                              : table[static_cast<size_t>(at + i) * a.max_pages + x];
                slots[before + e] = slot_of(page, pos, a.page_shift);
            }
        }
        __syncthreads();
    }
    if (tid == 0) *n_free_out = stack - static_cast<int>(given[0]);
}

__global__ __launch_bounds__(256) void slots_kernel(PlanArgs a, const int* __restrict__ table, const int* __restrict__ cu,
                                                    const int* __restrict__ lengths, int* __restrict__ slots) {
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t >= cu[a.N]) return;
    int s = 0;  // the request of token t
    for (int hi = a.N; hi - s > 1;) {
        const int mid = s + ((hi - s) >> 1);
        if (cu[mid] <= t)
            s = mid;
        else
            hi = mid;
    }
    const int pos = lengths[s] - (cu[s + 1] - t);  // lengths are those after the step
    const int page = table[static_cast<size_t>(s) * a.max_pages + (pos >> a.page_shift)];
    slots[t] = slot_of(page, pos, a.page_shift);
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_plan_pages(int N, int page_size, int max_pages, int n_stack, int max_tokens, const int* lengths,
                                  const int* add, const int* free_pages, const int* n_free, int* table, int* cu, int* added,
                                  int* lengths_out, int* slots, int* n_free_out, hipStream_t st) {
    attn::PlanArgs a{N, 0, max_pages, n_stack, max_tokens};
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    const unsigned long long blocks = (static_cast<unsigned long long>(max_tokens) + 255) / 256;
    if (!grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
    const bool few = max_tokens <= attn::kFewTokens;
    hipLaunchKernelGGL(attn::plan_kernel, dim3(1), dim3(attn::kPlanThreads), 0, st, a, lengths, add, free_pages, n_free, table,
                       cu, added, lengths_out, few ? slots : nullptr, n_free_out);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || few || !slots || N == 0) return e;
    hipLaunchKernelGGL(attn::slots_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, a, table, cu, lengths_out,
                       slots);
    return hipGetLastError();
}

}  // namespace gdr
