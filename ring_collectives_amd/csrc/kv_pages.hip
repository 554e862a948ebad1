// kv_pages.hip -- the pages of a paged cache: forked with the rows of a block
// table, freed, compacted and copied.
//
// Which pages are in use follows from the block table alone, so no counts of
// holders have to be kept in step with it.  With bit sets over the pages,
//   freed = held before & ~held after,
//   moved = in use & at or above n,  holes = free & below n   (n pages in use),
// in order of their numbers by running sums of the sets' words.
//
// What has to move is small next to the latencies, so the launches and the
// trips to memory bound it.  Few rows and pages are one workgroup's, with its
// sets in LDS.  Else one launch makes the sets, a wave a row, and its last
// workgroup to finish does what needs them whole (rewriting the table of
// kv_compact, which needs all workgroups again, is a launch of its own).  Marks
// are device-scope atomics, which that workgroup reads at device scope; it
// leaves them zero.  A row marks what the row above it does not hold at the
// same place: beams of one prompt hold mostly the same pages.  1024 rows of 250
// pages out of 198000 take 22 us: 10 until the 62000 marks are made, 12 for the
// last workgroup, 5 of them trips to the sets, 4 handing out 22000 freed pages.
// 200 rows of 80 pages out of 48000, compacted, take 12 and 5 us.  The finishing
// workgroup reads and clears the whole pool's sets: 4 rows of 44 pages out of 2^20
// take 28 us, the 1024 rows there 46.
#include "attn_internal.h"
#include "tp_search.h"

#include <hip/hip_runtime.h>

namespace ringc {
namespace {

constexpr int kThreads = 1024, kRowWaves = kThreads / 64;
constexpr int kMaxBlocks = 512;

// Sets and counts lie in the workspace for all workgroups, or in the one
// workgroup's LDS.
template <bool LDS = false> __device__ __forceinline__ void mark(unsigned* set, int i) {
    __hip_atomic_fetch_or(set + (i >> 5), 1u << (i & 31), __ATOMIC_RELAXED,
                          LDS ? __HIP_MEMORY_SCOPE_WORKGROUP : __HIP_MEMORY_SCOPE_AGENT);
}
template <bool LDS = false, class T> __device__ __forceinline__ T seen(const T* p) {
    return LDS ? *p : __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <bool LDS = false> __device__ __forceinline__ void raise_to(int* p, int x) {
    __hip_atomic_fetch_max(p, x, __ATOMIC_RELAXED, LDS ? __HIP_MEMORY_SCOPE_WORKGROUP : __HIP_MEMORY_SCOPE_AGENT);
}

// True in the launch's last workgroup to get here, once what all of them did at
// device scope is done.
__device__ __forceinline__ bool last_block(int* counter) {
    __shared__ int last;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
    __syncthreads();
    return last;
}

// The sum of x over the workgroup's lower threads, and over all of them.
__device__ __forceinline__ int block_scan(int x, int& total) {
    __shared__ int part[kRowWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, s = wave_scan(x);
    __syncthreads();
    if (lane == 63) part[wave] = s;
    __syncthreads();
    int below = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) {
        if (w < wave) below += part[w];
        total += part[w];
    }
    return below + s - x;
}

// kWords words of a set a thread, kThreads apart, so that neighbours' bits are
// spread over the lanes; and, of each, the bits of all words before it.
constexpr int kWords = 8;
template <int W = kWords> struct Words {
    unsigned w[W];
};
__device__ __forceinline__ void word_scan(const Words<1>& x, int, int (&before)[1], int& total) {
    before[0] = block_scan(__builtin_popcount(x.w[0]), total);
}
__device__ __forceinline__ void word_scan(const Words<>& x, int words, int (&before)[kWords], int& total) {
    __shared__ int part[kWords * kRowWaves + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kWords; ++v) {
        int n = 0, s = 0;
        if (v * kThreads < words) {
            n = __builtin_popcount(x.w[v]);
            s = wave_scan(n);
        }
        before[v] = s - n;
        if (lane == 63) part[v * kRowWaves + wave] = s;
    }
    __syncthreads();
    if (wave == 0) {
        static_assert(kWords * kRowWaves == 128, "two sums a lane");
        const int a = part[2 * lane], b = part[2 * lane + 1], s = wave_scan(a + b);
        part[2 * lane] = s - a - b;
        part[2 * lane + 1] = s - b;
        if (lane == 63) part[128] = s;
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kWords; ++v) before[v] += part[v * kRowWaves + wave];
    total = part[128];
}

struct ForkArgs {
    const int *table, *lengths, *parents, *keep, *used;
    int *free_pages, *table_after, *lengths_after, *copies, *n_copies, *shared, *used_after;
    int B, B2, group, n_free, width, shift, pages, words, new_blocks;
    Status* status;
    WsSpan zero;
    int *counter, *owner, *apart;        // owner[page]: B2 - its first row, apart[group]: the room less the shared tokens
    unsigned *old, *full, *part;         // pages the old rows held, those the new ones have full, and partly filled
    unsigned long long* last;            // per new row: its partly filled page + 1 (0: none), and its place above
};

struct ForkRow {
    int parent, tokens, held, full;      // held: pages, full: of them without a free place
};
__device__ __forceinline__ int row_tokens(int n, int width, int shift) {
    const long long room = (long long)width << shift;
    return n < 0 ? 0 : n < room ? n : (int)room;
}
__device__ __forceinline__ ForkRow fork_row(const ForkArgs& a, int i) {
    ForkRow r;
    r.parent = a.parents[i];
    const bool any = r.parent >= 0 && r.parent < a.B;
    if (!any) r.parent = 0;
    int n = any ? row_tokens(a.lengths[r.parent], a.width, a.shift) : 0;
    if (any && a.keep) {
        const int k = a.keep[i];
        n = k < 0 ? 0 : k < n ? k : n;
    }
    r.tokens = n;
    r.full = n >> a.shift;
    r.held = (int)(((long long)n + (1 << a.shift) - 1) >> a.shift);
    return r;
}
__device__ __forceinline__ bool is_page(int e, int pages) { return e >= 0 && e < pages; }

// What a wave takes of a row, so that few long rows are many waves' work: 4 rows
// of 3981 entries fork in 9.6 us so, in 14.9 by pieces of 1024; one row of 5855
// is compacted in 14 and 19, whole in 45.
constexpr int kPiece = 256;
__host__ __device__ __forceinline__ int pieces_of(int width) { return width > kPiece ? (width + kPiece - 1) / kPiece : 1; }
struct RowPiece {
    int row, begin, end;
    __device__ __forceinline__ RowPiece(int x, int pieces, int width) {
        row = pieces == 1 ? x : x / pieces;
        begin = (x - row * pieces) * kPiece;
        end = begin + kPiece < width ? begin + kPiece : width;
    }
};

// A new row's piece, by a wave: its entries, and the marks of its pages.
__device__ __forceinline__ void new_row(const ForkArgs& a, const RowPiece& piece, int lane) {
    const int i = piece.row;
    const int near = lane < i ? a.parents[i - 1 - lane] : -1;
    const ForkRow r = fork_row(a, i);
    ForkRow up = {0, 0, 0, 0};
    if (i) up = fork_row(a, i - 1);
    // one of the 64 rows above has the same pages, and marks them
    const bool again = !a.keep && __any(near == r.parent);
    const int *row = a.table + (long long)r.parent * a.width, *above = a.table + (long long)up.parent * a.width;
    int* to = a.table_after + (long long)i * a.width;
    const bool grouped = a.shared && a.group > 1;
    int common = r.tokens;               // tokens that the row above holds on the same pages
    const int j0 = piece.begin;
    int e[4], x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int j = j0 + 64 * u + lane;
        e[u] = j < r.held ? row[j] : -1;
        x[u] = j < up.held ? above[j] : -1;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int j = j0 + 64 * u + lane;
        // (the finishing workgroup writes the entry of a partly filled page)
        if (j < a.width && (j >= r.held || j < r.full)) to[j] = e[u];
        if (j < r.held && is_page(e[u], a.pages)) {
            if (j >= r.full) {
                mark(a.part, e[u]);
                raise_to(a.owner + e[u], a.B2 - i);
                __hip_atomic_store(a.last + i, (unsigned long long)(unsigned)j << 32 | (unsigned)(e[u] + 1), __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            } else if (!again && !(j < up.full && e[u] == x[u])) {
                mark(a.full, e[u]);
            }
        }
        const unsigned long long other = __ballot(j < r.held && j < up.held && e[u] != x[u]);
        if (other) {
            const long long n = (long long)(j0 + 64 * u + __builtin_ctzll(other)) << a.shift;
            if (n < common) common = (int)n;
        }
    }
    if (lane) return;
    if (!piece.begin) {
        a.lengths_after[i] = r.tokens;
        // a partly filled entry that is no page is passed on
        if (r.held > r.full && !is_page(row[r.full], a.pages)) to[r.full] = row[r.full];
    }
    if (!grouped) return;
    const int room = (int)((long long)a.width << a.shift);
    raise_to(a.apart + i / a.group, room - (i % a.group ? common : r.tokens));
}

// The workgroup that finishes: copies are counted in row order, freed pages by
// number, and the one handed to the other.
template <bool LDS> __device__ __forceinline__ void finish_fork(const ForkArgs& a, int used_before, int* lds) {
    // (what exceeds n_free stands for table entries that got no page)
    const int used = used_before < a.n_free ? used_before : a.n_free;
    int *page = lds, *at = lds + a.B2, *rank = lds + 2 * a.B2, *taken = lds + 3 * a.B2;      // per row: as in last, and its copy; per copy: a freed page
    const int tid = threadIdx.x;
    const bool grouped = a.shared && a.group > 1;
    constexpr int W = LDS ? 1 : kWords, kChunk = kThreads * W;       // in LDS there are no more words than threads
    auto freed = [&](int w0) {
        Words<W> r;
#pragma unroll
        for (int v = 0; v < W; ++v) {
            const int w = w0 + v * kThreads + tid;
            r.w[v] = 0;
            if (w < a.words) r.w[v] = seen<LDS>(a.old + w) & ~seen<LDS>(a.full + w) & ~seen<LDS>(a.part + w);
        }
        return r;
    };
    const Words<W> gone = freed(0);
    int before[W], n_copies = 0, n_freed, all;
    for (int i0 = 0; i0 < a.B2; i0 += kThreads) {
        const int i = i0 + tid;
        int copy = 0;
        if (i < a.B2) {
            const unsigned long long l = seen<LDS>(a.last + i);
            const int e = (int)(unsigned)l - 1;
            page[i] = e;
            at[i] = (int)(l >> 32);
            if (e >= 0) copy = (seen<LDS>(a.full + (e >> 5)) >> (e & 31) & 1) || seen<LDS>(a.owner + e) != a.B2 - i;
            if (copy && grouped) raise_to<LDS>(a.apart + i / a.group, (a.width - at[i]) << a.shift);
        }
        const int k = block_scan(copy, all);
        if (i < a.B2) rank[i] = copy ? n_copies + k : -1;
        n_copies += all;
    }
    if (!LDS) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");        // what raise_to did is done behind the scan's barriers
    word_scan(gone, a.words, before, n_freed);
    const int chunk0 = n_freed;
    for (int w0 = kChunk; w0 < a.words; w0 += kChunk) {
        int some[W];
        word_scan(freed(w0), a.words - w0, some, all);
        n_freed += all;
    }
    auto hand_out = [&](const Words<W>& x, int w0, int base) {
#pragma unroll
        for (int v = 0; v < W; ++v) {
            int k = base + before[v];
            const int p = (w0 + v * kThreads + tid) * 32, entry = used - n_freed + k;
            if (k >= n_copies && entry >= 0 && entry <= a.n_free - 32) {      // all of the word's pages go back
                for (unsigned bits = x.w[v], i = entry; bits; bits &= bits - 1, ++i) a.free_pages[i] = p + __builtin_ctz(bits);
            } else {
                for (unsigned bits = x.w[v]; bits; bits &= bits - 1, ++k) {
                    const int q = p + __builtin_ctz(bits), i = used - n_freed + k;
                    if (k < n_copies) taken[k] = q;
                    else if (i >= 0 && i < a.n_free) a.free_pages[i] = q;
                }
            }
        }
    };
    hand_out(gone, 0, 0);
    for (int w0 = kChunk, base = chunk0; w0 < a.words; w0 += kChunk) {
        const Words<W> x = freed(w0);
        word_scan(x, a.words - w0, before, all);
        hand_out(x, w0, base);
        base += all;
    }
    __syncthreads();
    for (int i = tid; i < a.B2; i += kThreads) {
        const int k = rank[i];
        int e = page[i];
        if (e >= 0) {
            if (!LDS) a.owner[e] = 0;
            if (k >= 0) {
                const long long entry = (long long)used + k - n_freed;
                const int to = k < n_freed ? taken[k] : entry >= 0 && entry < a.n_free ? a.free_pages[entry] : -1;
                a.copies[2 * k] = e;
                a.copies[2 * k + 1] = to;
                e = to;
            }
            a.table_after[(long long)i * a.width + at[i]] = e;
        }
        if (i >= n_copies) a.copies[2 * i] = a.copies[2 * i + 1] = -1;
        if (!LDS) a.last[i] = 0;
    }
    if (a.shared) {
        const int room = (int)((long long)a.width << a.shift);
        for (int g = tid; g < a.B2 / a.group; g += kThreads) {
            if (grouped) {
                a.shared[g] = room - seen<LDS>(a.apart + g);
                if (!LDS) a.apart[g] = 0;
            } else {
                a.shared[g] = fork_row(a, g).tokens;
            }
        }
    }
    if (!LDS)
        for (int w = tid; w < a.words; w += kThreads) a.old[w] = a.full[w] = a.part[w] = 0;
    if (tid == 0) {
        const long long after = (long long)used + n_copies - n_freed;
        *a.used_after = after > 0x7fffffff ? 0x7fffffff : (int)after;
        *a.n_copies = n_copies;
        if (!LDS) *a.counter = 0;
    }
}

// Where tables and pages are few, one workgroup does it all with its sets in
// LDS: two trips to memory (lengths, then entries, all in flight together) and
// none to the sets.  The call takes 5.1 us instead of the 8.0 of the kernel below
// for 4 rows of 7 entries, 6.0 and 9.4 for 32 of 46, 7.6 and 9.4 for 16 of 252,
// and as long as it, 10.4 and 11, at the limits (96 of 77, 240 of 34).
constexpr int kSmallRows = 256, kSmallEntries = 8192, kSmallPages = 8192;

// x / y of numbers up to kSmallEntries: the quotient of x + 1/2 is 1 / 2y or more
// from a whole number, and the fp32 product off by less than a hundredth of that.
struct SmallDiv {
    float inv;
    __device__ __forceinline__ explicit SmallDiv(int n) : inv(1.0f / (float)n) {}
    __device__ __forceinline__ int operator()(int x) const { return (int)(((float)x + 0.5f) * inv); }
};
__global__ __launch_bounds__(kThreads) void kv_fork_small_kernel(ForkArgs a) {
    __shared__ int rows[4 * kSmallRows], entry[kSmallEntries], owner[kSmallPages];
    __shared__ int parent[kSmallRows], tokens[kSmallRows], lengths[kSmallRows], apart[kSmallRows];
    __shared__ unsigned sets[3][kSmallPages / 32];
    __shared__ unsigned long long last[kSmallRows];
    const int tid = threadIdx.x, page = 1 << a.shift;
    const int used = *a.used;
    int p0 = -1, keep0 = 0x7fffffff;
    if (tid < a.B2) {
        p0 = a.parents[tid];
        if (a.keep) keep0 = a.keep[tid];
    }
    if (tid < a.B) lengths[tid] = row_tokens(a.lengths[tid], a.width, a.shift);
    for (int i = tid; i < a.pages; i += kThreads) owner[i] = 0;
    if (tid < a.words) sets[0][tid] = sets[1][tid] = sets[2][tid] = 0;
    if (tid < kSmallRows) {
        apart[tid] = 0;
        last[tid] = 0;
    }
    __syncthreads();
    const int room = a.width << a.shift;
    if (tid < a.B2) {
        const bool any = p0 >= 0 && p0 < a.B;
        int n = any ? lengths[p0] : 0;
        n = keep0 < 0 ? 0 : keep0 < n ? keep0 : n;
        parent[tid] = any ? p0 : 0;
        tokens[tid] = n;
        a.lengths_after[tid] = n;
        if (a.shared && a.group > 1) raise_to<true>(apart + tid / a.group, room - n);
    }
    __syncthreads();
    auto held = [&](int n) { return (n + page - 1) >> a.shift; };
    // the entries of new rows and of old ones, one after the other over the
    // threads (a wave a row took 23 us for 240 rows of 34)
    static_assert(kSmallPages / 32 <= kThreads, "a word of a set a thread");
    constexpr int U = 4;
    const SmallDiv by_width(a.width), by_group(a.group);
    const int fresh = a.B2 * a.width, old = a.B * a.width, both = fresh > old ? fresh : old;
    for (int x0 = tid; x0 < both; x0 += U * kThreads) {
        int e[U], f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = x0 + u * kThreads, i = by_width(x), j = x - i * a.width;
            e[u] = x < fresh && j < held(tokens[i]) ? a.table[parent[i] * a.width + j] : -1;
            f[u] = x < old && j < held(lengths[i]) ? a.table[x] : -1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = x0 + u * kThreads, i = by_width(x), j = x - i * a.width;
            if (is_page(f[u], a.pages)) mark<true>(sets[0], f[u]);
            if (x >= fresh) continue;
            const bool valid = is_page(e[u], a.pages), part = j == tokens[i] >> a.shift && j < held(tokens[i]);
            entry[x] = e[u];
            if (!part || !valid) a.table_after[x] = e[u];
            if (valid) mark<true>(sets[part ? 2 : 1], e[u]);
            if (valid && part) {
                raise_to<true>(owner + e[u], a.B2 - i);
                last[i] = (unsigned long long)(unsigned)j << 32 | (unsigned)(e[u] + 1);
            }
        }
    }
    __syncthreads();
    if (a.shared && a.group > 1)
        for (int x = tid; x < fresh; x += kThreads) {
            const int i = by_width(x), j = x - i * a.width, g = by_group(i);
            if (i == g * a.group || j >= held(tokens[i] < tokens[i - 1] ? tokens[i] : tokens[i - 1])) continue;
            // where this row is another than the one above, for the first time or again
            if (entry[x] != entry[x - a.width] && (!j || entry[x - 1] == entry[x - 1 - a.width]))
                raise_to<true>(apart + g, room - (j << a.shift));
        }
    __syncthreads();
    a.old = sets[0];
    a.full = sets[1];
    a.part = sets[2];
    a.owner = owner;
    a.apart = apart;
    a.last = last;
    finish_fork<true>(a, used, rows);
}

__global__ __launch_bounds__(kThreads) void kv_fork_kernel(ForkArgs a) {
    extern __shared__ int lds[];
    __shared__ unsigned whole[KV_FORK_MAX_ROWS / 32];     // old rows that some new row keeps all tokens of
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pieces = pieces_of(a.width);
    const WsRecord rec = ws_record(a.status);
    if ((int)blockIdx.x < a.new_blocks) {
        if (!ws_ok(a.status, rec, a.zero, lane)) return;
        for (int x = blockIdx.x * kRowWaves + wave; x < a.B2 * pieces; x += a.new_blocks * kRowWaves)
            new_row(a, RowPiece(x, pieces, a.width), lane);
    } else {
        for (int w = tid; w < (a.B + 31) / 32; w += kThreads) whole[w] = 0;
        __syncthreads();
        for (int i = tid; i < a.B2; i += kThreads) {
            const int p = a.parents[i];
            if (p >= 0 && p < a.B && (!a.keep || a.keep[i] >= a.lengths[p]))
                __hip_atomic_fetch_or(whole + (p >> 5), 1u << (p & 31), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
        __syncthreads();
        if (!ws_ok(a.status, rec, a.zero, lane)) return;
        const int blocks = (int)gridDim.x - a.new_blocks;
        for (int y = ((int)blockIdx.x - a.new_blocks) * kRowWaves + wave; y < a.B * pieces; y += blocks * kRowWaves) {
            const RowPiece piece(y, pieces, a.width);
            const int b = piece.row;
            if (whole[b >> 5] >> (b & 31) & 1) continue;
            auto pages = [&](int n) { return (int)(((long long)row_tokens(n, a.width, a.shift) + (1 << a.shift) - 1) >> a.shift); };
            const int held = pages(a.lengths[b]), up_held = b ? pages(a.lengths[b - 1]) : 0;
            const int* row = a.table + (long long)b * a.width;
            const int j0 = piece.begin;
            int e[4], x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = j0 + 64 * u + lane;
                e[u] = j < held ? row[j] : -1;
                x[u] = j < up_held ? row[j - a.width] : -1;
            }
            // what the row above holds too it marks, or a new row keeps
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (is_page(e[u], a.pages) && e[u] != x[u]) mark(a.old, e[u]);
        }
    }
    if (last_block(a.counter)) finish_fork<false>(a, *a.used, lds);
}

// ---------------------------------------------------------------- compaction
struct CompactArgs {
    const int *table, *lengths;
    int *table_after, *free_pages, *copies, *n_copies, *used_after;
    int B, n, width, shift, first, words;
    Status* status;
    WsSpan zero, data;
    int* counter;
    unsigned* live;                      // marks of the pool's pages in use
    unsigned* in_use;                    // a copy of them for the second launch
    int* before;                         // per word: pages in use below it, and last the ones below page n
};

__device__ __forceinline__ int held_pages(const CompactArgs& a, int b) {
    return (int)(((long long)row_tokens(a.lengths[b], a.width, a.shift) + (1 << a.shift) - 1) >> a.shift);
}

__device__ __forceinline__ void finish_compact(const CompactArgs& a) {
    const int tid = threadIdx.x;
    __shared__ int below;
    constexpr int kChunk = kThreads * kWords;
    auto used = [&](int w0) {
        Words<> r;
#pragma unroll
        for (int v = 0; v < kWords; ++v) {
            const int w = w0 + v * kThreads + tid;
            r.w[v] = 0;
            if (w < a.words) r.w[v] = seen(a.live + w);
        }
        return r;
    };
    const Words<> chunk0 = used(0);
    int before[kWords], n, n0, all;
    word_scan(chunk0, a.words, before, n0);
    n = n0;
    for (int w0 = kChunk; w0 < a.words; w0 += kChunk) {
        int some[kWords];
        word_scan(used(w0), a.words - w0, some, all);
        n += all;
    }
    // the pages in use below number n stay: in the word of page n, or all of them
    auto find = [&](const Words<>& x, int w0, int base) {
#pragma unroll
        for (int v = 0; v < kWords; ++v)
            if (w0 + v * kThreads + tid == n >> 5)
                below = base + before[v] + __builtin_popcount(x.w[v] & ((1u << (n & 31)) - 1));
    };
    auto move = [&](const Words<>& x, int w0, int base, int stay) {
#pragma unroll
        for (int v = 0; v < kWords; ++v) {
            const int w = w0 + v * kThreads + tid, k = base + before[v], p = w * 32;
            if (w >= a.words) continue;
            const unsigned under = n - p >= 32 ? ~0u : n > p ? (1u << (n - p)) - 1 : 0u;
            int h = p - k, m = k + __builtin_popcount(x.w[v] & under) - stay;
            for (unsigned y = ~x.w[v] & under; y; y &= y - 1, ++h) a.copies[2 * h + 1] = a.first + p + __builtin_ctz(y);
            for (unsigned y = x.w[v] & ~under; y; y &= y - 1, ++m) a.copies[2 * m] = a.first + p + __builtin_ctz(y);
            a.before[w] = k;
            a.in_use[w] = x.w[v];
            a.live[w] = 0;
        }
    };
    if (tid == 0 && n >> 5 >= a.words) below = n;
    find(chunk0, 0, 0);
    for (int w0 = kChunk, base = n0; w0 < a.words; w0 += kChunk) {
        const Words<> x = used(w0);
        word_scan(x, a.words - w0, before, all);
        find(x, w0, base);
        base += all;
    }
    __syncthreads();
    const int stay = below;
    if (a.words > kChunk) word_scan(chunk0, a.words, before, all);
    move(chunk0, 0, 0, stay);
    for (int w0 = kChunk, base = n0; w0 < a.words; w0 += kChunk) {
        const Words<> x = used(w0);
        word_scan(x, a.words - w0, before, all);
        move(x, w0, base, stay);
        base += all;
    }
    if (tid == 0) {
        a.before[a.words] = stay;
        *a.used_after = n;
        *a.n_copies = n - stay;
        *a.counter = 0;
        ws_add_data(a.status, a.data);
    }
}

__global__ __launch_bounds__(kThreads) void kv_compact_kernel(CompactArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (!ws_ok(a.status, ws_record(a.status), a.zero, lane)) return;
    const int pieces = pieces_of(a.width);
    for (int y = blockIdx.x * kRowWaves + wave; y < a.B * pieces; y += gridDim.x * kRowWaves) {
        const RowPiece piece(y, pieces, a.width);
        const int b = piece.row, held = held_pages(a, b), up = b ? held_pages(a, b - 1) : 0;
        const int* row = a.table + (long long)b * a.width;
        const int j0 = piece.begin;
        int e[4], x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + 64 * u + lane;
            e[u] = j < held ? row[j] : -1;
            x[u] = j < up ? row[j - a.width] : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long long i = (long long)e[u] - a.first;
            if (i >= 0 && i < a.n && e[u] != x[u]) mark(a.live, (int)i);
        }
    }
    if (last_block(a.counter)) finish_compact(a);
}

__global__ __launch_bounds__(256) void kv_renumber_kernel(CompactArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // (its own data lies past the counters: the record says what it said to the first launch)
    if (!ws_ok(a.status, ws_record(a.status), a.zero, lane)) return;
    const int n = *a.used_after, stay = a.before[a.words], moves = n - stay;
    const int step = gridDim.x * 256, first = blockIdx.x * 256 + threadIdx.x;
    for (int i = first; i < a.n; i += step) a.free_pages[i] = a.first + i;
    for (int i = first; i < a.n / 2; i += step)
        if (i >= moves) a.copies[2 * i] = a.copies[2 * i + 1] = -1;
    const int pieces = pieces_of(a.width);
    for (int y = blockIdx.x * 4 + wave; y < a.B * pieces; y += gridDim.x * 4) {
        const RowPiece piece(y, pieces, a.width);
        const int held = held_pages(a, piece.row);
        const long long row = (long long)piece.row * a.width;
        int e[kPiece / 64];
#pragma unroll
        for (int u = 0; u < kPiece / 64; ++u) {
            const int j = piece.begin + 64 * u + lane;
            e[u] = j < held && j < piece.end ? a.table[row + j] : -1;
        }
#pragma unroll
        for (int u = 0; u < kPiece / 64; ++u) {
            const int j = piece.begin + 64 * u + lane;
            const long long i = (long long)e[u] - a.first;
            if (i >= n && i < a.n) {
                const int w = (int)i >> 5;
                e[u] = a.copies[2 * (a.before[w] + __builtin_popcount(a.in_use[w] & ((1u << (i & 31)) - 1)) - stay) + 1];
            }
            if (j < piece.end) a.table_after[row + j] = e[u];
        }
    }
}

// Where tables and pools are few, one workgroup does it all, sets, moves and
// table in LDS: the call takes 5.0 us instead of 9.9 for 9 rows of 32 entries and
// a pool of 300, 7.7 and 12.7 for 256 of 29 and a pool of 8000.
__global__ __launch_bounds__(kThreads) void kv_compact_small_kernel(CompactArgs a) {
    __shared__ int to[kSmallPages / 2], lengths[kSmallRows], before[kSmallPages / 32], below;
    __shared__ unsigned live[kSmallPages / 32];
    const int tid = threadIdx.x;
    if (tid < a.B) lengths[tid] = held_pages(a, tid);
    if (tid < a.words) live[tid] = 0;
    __syncthreads();
    constexpr int U = kSmallEntries / kThreads;
    const SmallDiv by_width(a.width);
    int e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int x = tid + u * kThreads, b = by_width(x);
        e[u] = x < a.B * a.width && x - b * a.width < lengths[b] ? a.table[x] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int x = tid + u * kThreads, b = by_width(x);
        const long long i = (long long)e[u] - a.first;
        if (x < a.B * a.width && x - b * a.width < lengths[b] && i >= 0 && i < a.n) mark<true>(live, (int)i);
    }
    __syncthreads();
    const unsigned bits = tid < a.words ? live[tid] : 0u;
    int n;
    const int k = block_scan(__builtin_popcount(bits), n), p = tid * 32;
    const unsigned under = n - p >= 32 ? ~0u : n > p ? (1u << (n - p)) - 1 : 0u;      // the word's pages below number n
    if (tid < a.words) before[tid] = k;
    if (tid == n >> 5 && tid < a.words) below = k + __builtin_popcount(bits & under);
    if (tid == 0 && n >> 5 >= a.words) below = n;
    __syncthreads();
    const int stay = below, moves = n - stay;
    if (tid < a.words) {
        int h = p - k, m = k + __builtin_popcount(bits & under) - stay;
        for (unsigned y = ~bits & under; y; y &= y - 1, ++h) a.copies[2 * h + 1] = to[h] = a.first + p + __builtin_ctz(y);
        for (unsigned y = bits & ~under; y; y &= y - 1, ++m) a.copies[2 * m] = a.first + p + __builtin_ctz(y);
    }
    __syncthreads();
    for (int i = tid; i < a.n; i += kThreads) a.free_pages[i] = a.first + i;
    for (int i = moves + tid; i < a.n / 2; i += kThreads) a.copies[2 * i] = a.copies[2 * i + 1] = -1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int x = tid + u * kThreads;
        if (x >= a.B * a.width) break;
        const long long i = (long long)e[u] - a.first;
        // (what is no row's is -1 here, and before the pool)
        if (i >= n && i < a.n) e[u] = to[before[i >> 5] + __builtin_popcount(live[i >> 5] & ((1u << (i & 31)) - 1)) - stay];
        a.table_after[x] = e[u];
    }
    if (tid == 0) {
        *a.used_after = n;
        *a.n_copies = moves;
    }
}

// ---------------------------------------------------------------- copies
struct CopyArgs {
    char* cache[2 * RING_MAX_RANKS];
    const int *copies, *n_copies;
    int n_caches, capacity, pages, chunks, vecs, per;    // of a page: chunks of `per` 16-byte vectors, vecs in all
};

// A wave copies a chunk of a page, four 16-byte vectors a lane in flight, past
// the caches: 12000 pages of 4 ranks, 471 MB read and written, 92 us, 5.1 TB/s
// (117 in all with the caches, 106 so).
__global__ __launch_bounds__(256) void kv_copy_kernel(CopyArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int n = *a.n_copies;
    if (n > a.capacity) n = a.capacity;
    const unsigned each = (unsigned)(a.n_caches * a.chunks);
    const long long items = (long long)(n < 0 ? 0 : n) * each;
    for (long long it = blockIdx.x * 4 + wave; it < items; it += (long long)gridDim.x * 4) {
        const int i = (int)(it / each), rest = (int)(it % each), c = rest / a.chunks, k = rest % a.chunks;
        const int from = a.copies[2 * i], to = a.copies[2 * i + 1];
        if (!is_page(from, a.pages) || !is_page(to, a.pages) || from == to) continue;
        const u32x4* src = (const u32x4*)a.cache[c] + (long long)from * a.vecs;
        u32x4* dst = (u32x4*)a.cache[c] + (long long)to * a.vecs;
        const int v0 = k * a.per, v1 = v0 + a.per < a.vecs ? v0 + a.per : a.vecs;
        for (int v = v0 + lane; v < v1; v += 256) {
            u32x4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (v + 64 * u < v1) x[u] = __builtin_nontemporal_load(src + v + 64 * u);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (v + 64 * u < v1) __builtin_nontemporal_store(x[u], dst + v + 64 * u);
        }
    }
}

int shift_of(int page_size) {
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}
bool page_size_ok(int page_size) { return page_size >= 1 && !(page_size & (page_size - 1)) && page_size <= (1 << 20); }
// Places of a row and pages: below 2^31 by more than any loop's step.
constexpr long long kMaxCount = (1LL << 31) - (1 << 20);
bool misaligned4(const void* p) { return (uintptr_t)p & 3; }

size_t fork_words(int pages) { return ((size_t)pages + 31) / 32; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

int row_blocks(int rows, int width) {
    const long long n = ((long long)rows * pieces_of(width) + kRowWaves - 1) / kRowWaves;
    return n < 1 ? 1 : n < kMaxBlocks ? (int)n : kMaxBlocks;
}

}  // namespace
}  // namespace ringc

using namespace ringc;

extern "C" size_t kv_fork_workspace_bytes(int B_after, int pages) {
    if (B_after < 0 || B_after > KV_FORK_MAX_ROWS || pages < 0) return 0;
    return kStatusBytes + up256((64 + 2 * (size_t)B_after + 3 * fork_words(pages) + (size_t)pages + (size_t)B_after) * 4);
}

extern "C" int kv_fork(const int* block_table, const int* lengths, const int* parents, const int* keep, int* free_pages,
                       const int* used, int* table_after, int* lengths_after, int* copies, int* n_copies, int* shared,
                       int* used_after, int B, int B_after, int group, int n_free, int table_stride, int page_size, int pages,
                       void* ws, size_t ws_bytes, void* stream) {
    if (B < 0 || B_after < 0 || n_free < 0 || table_stride < 0 || pages < 0 || group < 1 || B_after % group) return RING_EINVAL;
    if (!page_size_ok(page_size)) return RING_EINVAL;
    if (B > KV_FORK_MAX_ROWS || B_after > KV_FORK_MAX_ROWS || (long long)table_stride * page_size >= kMaxCount || pages >= kMaxCount)
        return RING_EUNSUPPORTED;
    if (!used || !used_after || !n_copies || (B && !lengths) || (B && table_stride && !block_table) || (n_free && !free_pages) ||
        (B_after && (!parents || !lengths_after || !copies)) || (B_after && table_stride && !table_after))
        return RING_EINVAL;
    for (const void* p : {(const void*)block_table, (const void*)lengths, (const void*)parents, (const void*)keep,
                          (const void*)free_pages, (const void*)used, (const void*)table_after, (const void*)lengths_after,
                          (const void*)copies, (const void*)n_copies, (const void*)shared, (const void*)used_after})
        if (misaligned4(p)) return RING_EINVAL;
    if (used_after == used || (B_after && (lengths_after == lengths || (table_stride && table_after == block_table))))
        return RING_EINVAL;
    const size_t need = kv_fork_workspace_bytes(B_after, pages);
    if (!ws || ((uintptr_t)ws & 255) || ws_bytes < need) return RING_EWORKSPACE;
    ForkArgs a;
    a.table = block_table;
    a.lengths = lengths;
    a.parents = parents;
    a.keep = keep;
    a.used = used;
    a.free_pages = free_pages;
    a.table_after = table_after;
    a.lengths_after = lengths_after;
    a.copies = copies;
    a.n_copies = n_copies;
    a.shared = shared;
    a.used_after = used_after;
    a.B = B;
    a.B2 = B_after;
    a.group = group;
    a.n_free = n_free;
    a.width = table_stride;
    a.shift = shift_of(page_size);
    a.pages = pages;
    a.words = (int)fork_words(pages);
    a.status = (Status*)ws;
    a.zero = WsSpan{kStatusBytes, need};
    a.counter = (int*)((char*)ws + kStatusBytes);
    a.last = (unsigned long long*)(a.counter + 64);
    a.old = (unsigned*)(a.last + B_after);
    a.full = a.old + a.words;
    a.part = a.full + a.words;
    a.owner = (int*)a.part + a.words;
    a.apart = a.owner + pages;
    const long long entries = (long long)(B > B_after ? B : B_after) * table_stride;
    if (B <= kSmallRows && B_after <= kSmallRows && entries <= kSmallEntries && pages <= kSmallPages) {
        hipLaunchKernelGGL(kv_fork_small_kernel, dim3(1), dim3(kThreads), 0, (hipStream_t)stream, a);
        return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
    }
    a.new_blocks = row_blocks(B_after, table_stride);
    hipLaunchKernelGGL(kv_fork_kernel, dim3((unsigned)(a.new_blocks + row_blocks(B, table_stride))), dim3(kThreads),
                       4 * (size_t)B_after * sizeof(int), (hipStream_t)stream, a);
    return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
}

extern "C" size_t kv_compact_workspace_bytes(int n_free) {
    if (n_free < 0) return 0;
    const size_t words = fork_words(n_free);
    return kStatusBytes + up256((64 + words) * 4) + up256((2 * words + 1) * 4);
}

extern "C" int kv_compact(const int* block_table, const int* lengths, int* table_after, int* free_pages, int* copies,
                          int* n_copies, int* used_after, int B, int n_free, int table_stride, int page_size, int first_page,
                          void* ws, size_t ws_bytes, void* stream) {
    if (B < 0 || n_free < 0 || table_stride < 0 || first_page < 0 || !page_size_ok(page_size)) return RING_EINVAL;
    if (B > KV_FORK_MAX_ROWS || (long long)table_stride * page_size >= kMaxCount || n_free >= kMaxCount ||
        (long long)first_page + n_free >= (1LL << 31))
        return RING_EUNSUPPORTED;
    if (!used_after || !n_copies || (B && !lengths) || (B && table_stride && (!block_table || !table_after)) ||
        (n_free && !free_pages) || (n_free > 1 && !copies))
        return RING_EINVAL;
    for (const void* p : {(const void*)block_table, (const void*)lengths, (const void*)table_after, (const void*)free_pages,
                          (const void*)copies, (const void*)n_copies, (const void*)used_after})
        if (misaligned4(p)) return RING_EINVAL;
    if (B && table_stride && table_after == block_table) return RING_EINVAL;
    const size_t need = kv_compact_workspace_bytes(n_free);
    if (!ws || ((uintptr_t)ws & 255) || ws_bytes < need) return RING_EWORKSPACE;
    CompactArgs a;
    a.table = block_table;
    a.lengths = lengths;
    a.table_after = table_after;
    a.free_pages = free_pages;
    a.copies = copies;
    a.n_copies = n_copies;
    a.used_after = used_after;
    a.B = B;
    a.n = n_free;
    a.width = table_stride;
    a.shift = shift_of(page_size);
    a.first = first_page;
    a.words = (int)fork_words(n_free);
    a.status = (Status*)ws;
    const size_t data = kStatusBytes + up256((64 + (size_t)a.words) * 4);
    a.zero = WsSpan{kStatusBytes, data};
    a.data = WsSpan{data, need};
    a.counter = (int*)((char*)ws + kStatusBytes);
    a.live = (unsigned*)a.counter + 64;
    a.in_use = (unsigned*)((char*)ws + data);
    a.before = (int*)a.in_use + a.words;
    if (B <= kSmallRows && (long long)B * table_stride <= kSmallEntries && n_free <= kSmallPages) {
        hipLaunchKernelGGL(kv_compact_small_kernel, dim3(1), dim3(kThreads), 0, (hipStream_t)stream, a);
        return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
    }
    hipLaunchKernelGGL(kv_compact_kernel, dim3((unsigned)row_blocks(B, table_stride)), dim3(kThreads), 0, (hipStream_t)stream, a);
    if (hipGetLastError() != hipSuccess) return RING_EHIP;
    const long long by_page = (n_free + 255LL) / 256, by_row = ((long long)B * pieces_of(table_stride) + 3) / 4;
    const long long work = by_page > by_row ? by_page : by_row, blocks = work < 1 ? 1 : work < 4 * kMaxBlocks ? work : 4 * kMaxBlocks;
    hipLaunchKernelGGL(kv_renumber_kernel, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, a);
    return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
}

extern "C" int kv_copy_pages(void* const* caches, const int* copies, const int* n_copies, int n_caches, int capacity,
                             int pages, long long page_bytes, void* stream) {
    if (n_caches < 1 || n_caches > 2 * RING_MAX_RANKS || capacity < 0 || pages < 0 || page_bytes < 0 || page_bytes % 16)
        return RING_EINVAL;
    if (page_bytes >= (1LL << 31)) return RING_EUNSUPPORTED;
    if (!caches || !n_copies || misaligned4(n_copies) || (capacity && !copies) || misaligned4(copies)) return RING_EINVAL;
    if (!capacity || !pages || !page_bytes) return RING_OK;
    CopyArgs a;
    for (int c = 0; c < n_caches; ++c) {
        if (!caches[c] || ((uintptr_t)caches[c] & 15)) return RING_EINVAL;
        a.cache[c] = (char*)caches[c];
    }
    a.copies = copies;
    a.n_copies = n_copies;
    a.n_caches = n_caches;
    a.capacity = capacity;
    a.pages = pages;
    a.vecs = (int)(page_bytes / 16);
    a.chunks = (a.vecs + 255) / 256;
    a.per = ((a.vecs + a.chunks - 1) / a.chunks + 63) / 64 * 64;
    a.chunks = (a.vecs + a.per - 1) / a.per;
    if ((long long)n_caches * a.chunks >= (1LL << 31)) return RING_EUNSUPPORTED;
    const long long items = ((long long)capacity * n_caches * a.chunks + 3) / 4;
    // eight workgroups a compute unit: 48000 pages compacted 94.3 us (89.4 with four,
    // 92.9 with sixteen), 9000 of two bf16 caches a rank 223 (218, 222)
    const long long most = 8LL * dev_info().cus;
    hipLaunchKernelGGL(kv_copy_kernel, dim3((unsigned)(items < most ? items : most)), dim3(256), 0, (hipStream_t)stream, a);
    return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
}
