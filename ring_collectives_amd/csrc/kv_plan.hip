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
// does; it does not read the entry.  Above 256 requests a thread has several, and
// loads runs shorter than eight one request after the other: six trips to memory
// for 1500.
//
// 24 requests of one token 2.5 us in the kernel, 4.2 to 5.3 a call; 200001 tokens of
// 1500 requests 7.
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

// Sums saturate: of non-negative counts in 32 bits, whatever the order, the
// result is the sum or the largest value.
__device__ __forceinline__ unsigned add_sat(unsigned x, unsigned y) { return __builtin_elementwise_add_sat(x, y); }
__device__ __forceinline__ int as_int(unsigned x) { return x < 0x7fffffffu ? (int)x : 0x7fffffff; }

// Inclusive running sum over the wave's lanes, on the VALU.
__device__ __forceinline__ unsigned scan_sat(unsigned x) {
    x = add_sat(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xf, 0xf, false));
    x = add_sat(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xf, 0xf, false));
    x = add_sat(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xf, 0xf, false));
    x = add_sat(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xf, 0xf, false));
    x = add_sat(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xa, 0xf, false));
    return add_sat(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xc, 0xf, false));
}

__global__ __launch_bounds__(kThreads) void kv_plan_kernel(PlanArgs a) {
    extern __shared__ int lds[];                 // [B + 1] sums of new tokens, [B + 1] of new pages, [B] lengths
    __shared__ unsigned part[kThreads / 64][2];
    int *cu = lds, *pg = lds + a.B + 1, *len = lds + 2 * (a.B + 1);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int used = *a.used;
    const int page = 1 << a.shift;
    auto pages = [&](long long n) { return (n + page - 1) >> a.shift; };
    // each thread sums a run of requests, one scan of the threads' sums places
    // the run, and the run's own sums follow from there
    const int run = (a.B + kThreads - 1) / kThreads;
    const int r0 = tid * run < a.B ? tid * run : a.B, r1 = r0 + run < a.B ? r0 + run : a.B;
    unsigned n = 0, p = 0;
#pragma unroll 8
    for (int b = r0; b < r1; ++b) {
        const int before = at_least_0(a.lengths[b]), add = at_least_0(a.new_tokens[b]);
        len[b] = before;
        cu[b] = add;
        n = add_sat(n, (unsigned)add);
        p = add_sat(p, (unsigned)(pages((long long)before + add) - pages(before)));
    }
    const unsigned n1 = scan_sat(n), p1 = scan_sat(p);
    if (lane == 63) {
        part[wave][0] = n1;
        part[wave][1] = p1;
    }
    __syncthreads();
    // what lies before this thread's run: the lanes below it and the waves
    // below its own (saturated, they say at least that the run lies past 2^31)
    unsigned tn = 0, tp = 0, n0 = (unsigned)__shfl_up((int)n1, 1), p0 = (unsigned)__shfl_up((int)p1, 1);
    if (lane == 0) n0 = p0 = 0;
    for (int w = 0; w < kThreads / 64; ++w) {
        if (w < wave) {
            n0 = add_sat(n0, part[w][0]);
            p0 = add_sat(p0, part[w][1]);
        }
        tn = add_sat(tn, part[w][0]);
        tp = add_sat(tp, part[w][1]);
    }
    for (int b = r0; b < r1; ++b) {
        const int before = len[b], add = cu[b];
        cu[b] = as_int(n0);
        pg[b] = as_int(p0);
        if (blockIdx.x == 0) {
            a.cu[b] = as_int(n0);
            a.after[b] = as_int((unsigned)before + (unsigned)add);
        }
        n0 = add_sat(n0, (unsigned)add);
        p0 = add_sat(p0, (unsigned)(pages((long long)before + add) - pages(before)));
    }
    if (tid == 0) {
        cu[a.B] = as_int(tn);
        pg[a.B] = as_int(tp);
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
            pos = n + a.prefix < 0x7fffffff ? (int)(n + a.prefix) : 0x7fffffff;
            if (j < a.stride) {
                const int p = j >= have ? free_page(pg[b] + j - have) : a.table[(long long)b * a.stride + j];
                if (p >= 0) slot = (long long)p * page + (n & (page - 1));
            }
        }
        a.positions[t] = pos;
        a.slots[t] = slot;
    }
    // not in place: workgroups that start later still read *used
    if (blockIdx.x == 0 && tid == 0) *a.used_after = (long long)used + need < 0x7fffffff ? used + need : 0x7fffffff;
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
