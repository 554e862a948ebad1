// kv_plan.hip -- block table, cache slots and positions of one step.
//
// With want(n) = ceil(n / page_size), request b needs want(after) -
// want(before) pages from entry used + (sum of the needs before b) of the free
// list on, and its token i goes to slot table[b][n / page_size] * page_size +
// n % page_size, n = before + i.
//
// What it must move is small (8 bytes per request, 12 per token), so the
// launch bounds it: there is only one.  Every workgroup scans the requests
// for itself in LDS instead of waiting for another that did, then takes its
// share of the table entries and tokens, finding each one's request by
// bisection.  A token whose page is new computes it like the table's writer
// does; it does not read the entry.
#include "ring_internal.h"
#include "tp_attention.h"

#include <hip/hip_runtime.h>

namespace ringc {
namespace {

constexpr int kThreads = 256;

struct PlanArgs {
    const int *lengths, *new_tokens, *free_pages, *used;
    int *table, *after, *cu, *positions;
    long long* slots;
    int* used_after;
    int B, n_free, stride, shift, capacity, prefix;
};

__device__ __forceinline__ int at_least_0(int x) { return x < 0 ? 0 : x; }

// Running sums over the workgroup of two values; returns the exclusive ones
// and leaves the totals in both totals.
__device__ __forceinline__ void scan2(long long& x, long long& y, long long& tx, long long& ty, long long (*part)[2], int lane,
                                      int wave) {
    const long long x0 = x, y0 = y;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const long long u = __shfl_up(x, d), w = __shfl_up(y, d);
        if (lane >= d) {
            x += u;
            y += w;
        }
    }
    if (lane == 63) {
        part[wave][0] = x;
        part[wave][1] = y;
    }
    __syncthreads();
    tx = ty = 0;
    for (int w = 0; w < kThreads / 64; ++w) {
        if (w < wave) {
            x += part[w][0];
            y += part[w][1];
        }
        tx += part[w][0];
        ty += part[w][1];
    }
    __syncthreads();
    x -= x0;
    y -= y0;
}

__global__ __launch_bounds__(kThreads) void kv_plan_kernel(PlanArgs a) {
    extern __shared__ int lds[];                 // [B + 1] sums of new tokens, [B + 1] of new pages, [B] lengths
    __shared__ long long part[kThreads / 64][2];
    int *cu = lds, *pg = lds + a.B + 1, *len = lds + 2 * (a.B + 1);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int used = *a.used;
    const int page = 1 << a.shift;
    constexpr int kMax = 0x7fffffff;
    auto sat = [](long long x) { return (int)(x < kMax ? x : kMax); };
    auto pages = [&](long long n) { return (n + page - 1) >> a.shift; };
    // each thread sums a run of requests, one scan of the threads' sums places
    // the run, and a second look at its requests writes the running sums
    const int run = (a.B + kThreads - 1) / kThreads;
    const int r0 = tid * run < a.B ? tid * run : a.B, r1 = r0 + run < a.B ? r0 + run : a.B;
    long long n = 0, p = 0, tn, tp;
#pragma unroll 8
    for (int b = r0; b < r1; ++b) {
        const int before = at_least_0(a.lengths[b]), add = at_least_0(a.new_tokens[b]);
        n += add;
        p += pages((long long)before + add) - pages(before);
    }
    scan2(n, p, tn, tp, part, lane, wave);
#pragma unroll 8
    for (int b = r0; b < r1; ++b) {
        const int before = at_least_0(a.lengths[b]), add = at_least_0(a.new_tokens[b]);
        cu[b] = sat(n);
        pg[b] = sat(p);
        len[b] = before;
        if (blockIdx.x == 0) {
            a.cu[b] = sat(n);
            a.after[b] = sat((long long)before + add);
        }
        n += add;
        p += pages((long long)before + add) - pages(before);
    }
    if (tid == 0) {
        cu[a.B] = sat(tn);
        pg[a.B] = sat(tp);
        if (blockIdx.x == 0) a.cu[a.B] = cu[a.B];
    }
    __syncthreads();
    const int total = cu[a.B], need = pg[a.B];
    auto request = [&](const int* sums, int x) {   // the last b with sums[b] <= x
        int lo = 0, hi = a.B;                      // sums[lo] <= x < sums[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (sums[mid] <= x) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    auto free_page = [&](long long i) {            // entry used + i of the free list
        const long long e = (long long)used + i;
        return e >= 0 && e < a.n_free ? a.free_pages[e] : -1;
    };
    const int step = gridDim.x * kThreads, first = blockIdx.x * kThreads + tid;
    for (long long i = first; i < need; i += step) {
        const int b = request(pg, (int)i);
        const long long j = pages(len[b]) + i - pg[b];
        if (j < a.stride) a.table[(long long)b * a.stride + j] = free_page(i);
    }
    for (long long t = first; t < a.capacity; t += step) {
        int pos = 0;
        long long slot = -1;
        if (t < total) {
            const int b = request(cu, (int)t);
            const long long n = (long long)len[b] + t - cu[b], j = n >> a.shift, have = pages(len[b]);
            pos = sat(n + a.prefix);
            if (j < a.stride) {
                const int p = j >= have ? free_page(pg[b] + j - have) : a.table[(long long)b * a.stride + j];
                if (p >= 0) slot = (long long)p * page + (n & (page - 1));
            }
        }
        a.positions[t] = pos;
        a.slots[t] = slot;
    }
    // not in place: workgroups that start later still read *used
    if (blockIdx.x == 0 && tid == 0) *a.used_after = sat((long long)used + need);
}

}  // namespace
}  // namespace ringc

using namespace ringc;

extern "C" int kv_plan(const int* lengths, const int* new_tokens, const int* free_pages, const int* used,
                       int* block_table, int* lengths_after, int* cu_new, int* positions, long long* slots,
                       int* used_after, int B, int n_free, int table_stride, int page_size, int capacity,
                       int prefix_len, void* stream) {
    if (B < 0 || n_free < 0 || table_stride < 0 || capacity < 0 || prefix_len < 0) return RING_EINVAL;
    if (page_size < 1 || (page_size & (page_size - 1)) || page_size > (1 << 20)) return RING_EINVAL;
    if (B == 0) return RING_OK;
    if (B > KV_PLAN_MAX_REQUESTS) return RING_EUNSUPPORTED;
    if (!lengths || !new_tokens || !used || !lengths_after || !cu_new || !used_after || (n_free && !free_pages) ||
        (table_stride && !block_table) || (capacity && (!positions || !slots)))
        return RING_EINVAL;
    if ((((uintptr_t)lengths | (uintptr_t)new_tokens | (uintptr_t)free_pages | (uintptr_t)used |
          (uintptr_t)block_table | (uintptr_t)lengths_after | (uintptr_t)cu_new | (uintptr_t)positions |
          (uintptr_t)used_after) & 3) || ((uintptr_t)slots & 7))
        return RING_EINVAL;
    if (used_after == used || lengths_after == lengths || lengths_after == new_tokens) return RING_EINVAL;
    int shift = 0;
    while ((1 << shift) < page_size) ++shift;
    const PlanArgs a{lengths, new_tokens, free_pages, used, block_table, lengths_after, cu_new, positions, slots,
                     used_after, B, n_free, table_stride, shift, capacity, prefix_len};
    const int work = capacity > B ? capacity : B;
    int blocks = (work + kThreads - 1) / kThreads;
    if (blocks > 2 * dev_info().cus) blocks = 2 * dev_info().cus;
    hipLaunchKernelGGL(kv_plan_kernel, dim3((unsigned)blocks), dim3(kThreads), (3 * (size_t)B + 2) * sizeof(int),
                       (hipStream_t)stream, a);
    return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
}
