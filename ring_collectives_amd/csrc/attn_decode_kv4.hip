// attn_decode_kv4.hip -- attention of one query token per row over the 4-bit
// paged cache, keys that a group of rows shares read once.
//
// Over any split of a row's keys,
//   m = max of the parts' m,  l = sum l_i 2^(m_i - m),  o = sum o_i 2^(m_i - m) / l
// gives the whole from parts that hold (m_i, l_i, o_i = sum of weighted values).
//
// Work is cut by the lengths, which lie in device memory: an item is a group's
// shared keys against up to 16 NT of its rows (row, head of the group that
// shares a key head), or a row's own keys against up to 16 of its heads, in
// tiles of 32 keys.  Every (rank, key head) has the same items; its workgroups
// each take the same number of consecutive tiles, found from the sums of the
// items' tiles that every workgroup makes for itself in LDS, and a workgroup's
// four waves split each item it meets.  A part that is all of its row's keys is
// the result; others are joined by a second launch.
//
// A wave's tile goes from memory to registers (two 16-byte loads a lane each
// for key and value codes at width 128, a byte each for their scales), one tile
// ahead.  A lane holds whole scale blocks of one key, so the conversion to bf16,
// two codes an instruction, leaves the A operand of S^T = K Q^T as it is: the
// order of the sum over the head's values is that of the lanes' bytes, for K
// and Q alike.  Values go to LDS as bf16 and are read transposed for
// O^T += V^T P^T, whose B operand are S^T's accumulators rounded to bf16.  No
// wave waits for another until its part is done.
//
// The cache read bounds it: 4.25 bits a value.
#include "kv4_core.h"

#include <hip/hip_runtime.h>

namespace ringc {
namespace {

constexpr int kWaves = 4;
constexpr int kKeys = 32;              // of a tile
constexpr int kMinTiles = 8;           // of a workgroup, if there are as many
constexpr int kPerCu = 3;              // workgroups to aim for

struct Kv4DecodeArgs {
    const unsigned short* q[RING_MAX_RANKS];
    const char* cache[RING_MAX_RANKS];
    unsigned short* o[RING_MAX_RANKS];
    const int *table, *lengths, *shared;
    long long q_stride, o_stride;
    int P, B, group, Hq, Hkv, width, shift, pages;
    int blocks;                        // workgroups of a (rank, key head)
    int shared_rbs, own_rbs, own_rows; // row blocks of a group, of a row; rows of an own part
    float c;
    float *shared_o, *own_o;           // [P Hkv][part][rows][D]
    float2 *shared_ml, *own_ml;        // [P Hkv][part][rows]
    int* start;                        // [items + 2] tiles before each item, in all, and of a workgroup
    Status* status;
    WsSpan data;
};

struct Items {
    int groups, shared, own;           // items: groups * shared_rbs, B * own_rbs
};
__device__ __forceinline__ Items items_of(const Kv4DecodeArgs& a) {
    Items n;
    n.groups = a.shared ? a.B / a.group : 0;
    n.shared = n.groups * a.shared_rbs;
    n.own = a.B * a.own_rbs;
    return n;
}
__device__ __forceinline__ int clamp_len(int n, int width, int shift) {
    const long long room = (long long)width << shift;
    return n < 0 ? 0 : n < room ? n : (int)room;
}

// The running state of 16 rows, one a lane of 16: a lane has every fourth
// block of four of the values, and its own quarter of the sum.
template <int D> struct State {
    f32x4 o[D / 16];
    float mc, l;
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int db = 0; db < D / 16; ++db) o[db] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        mc = -INFINITY;
        l = 0.0f;
    }
};
__device__ __forceinline__ float max_quarters(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float sum_quarters(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// One tile of a wave, as loaded: half h holds keys 16 h + lane % 16.
template <int D> struct Tile {
    typedef unsigned word __attribute__((ext_vector_type(D / 32)));
    word k[2], v[2];
    unsigned ks[2], vs[2];
    bool has[2];                       // the halves' pages are pages
};

// Where a row's keys are looked up: 64 pages of its table row at a time.
struct Pages {
    const int* row;
    int ids, base;                     // lane i: page base + i
    int limit, shift, pages;           // table entries that hold keys
    __device__ __forceinline__ void init(const int* r, int n, int sh, int pg) {
        row = r;
        limit = n;
        shift = sh;
        pages = pg;
        base = -64;
        ids = -1;
    }
    // the page of key `key` (uniform), -1 if it is none
    __device__ __forceinline__ int of(int key, int lane) {
        const int j = key >> shift;
        if (j - base >= 64 || j < base) {
            base = j;
            ids = j + lane < limit ? row[j + lane] : -1;
        }
        const int p = __builtin_amdgcn_readlane(ids, j - base);
        return j < limit && p >= 0 && p < pages ? p : -1;
    }
};

template <int D>
__device__ __forceinline__ void load_tile(Tile<D>& t, const char* cache, Kv4Page<D> page, int Hkv, int head, Pages& pg, int key,
                                          int lane) {
    const int i = lane & 15, quarter = lane >> 4, mask = (1 << page.shift) - 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int p = pg.of(key + 16 * h, lane), row = ((key + 16 * h) & mask) + i;
        t.has[h] = p >= 0;
        const char* base = cache + ((long long)(p < 0 ? 0 : p) * Hkv + head) * page.bytes();
        t.k[h] = *(const typename Tile<D>::word*)(base + page.codes(0, row) + quarter * (D / 8));
        t.v[h] = *(const typename Tile<D>::word*)(base + page.codes(1, row) + quarter * (D / 8));
        t.ks[h] = (unsigned char)base[page.scales(0, row) + quarter * D / 128];
        t.vs[h] = (unsigned char)base[page.scales(1, row) + quarter * D / 128];
    }
}

// A wave's tiles [j0, j1) of one item for NT times 16 rows.  Keys from `end` on
// are no keys of a row (end: this lane's rows', all_end: the least of them).
template <int D, int NT>
__device__ __forceinline__ void run_tiles(State<D> (&st)[NT], const bf16x8 (&q)[NT][D / 32], const char* cache, Kv4Page<D> page,
                                          int Hkv, int head, Pages pg, int j0, int j1, int end, float c, unsigned short* lds,
                                          int at, int lane) {
    typedef Rows<D> R;
    const int i = lane & 15, quarter = lane >> 4;
    Tile<D> t;
    if (j0 < j1) load_tile<D>(t, cache, page, Hkv, head, pg, j0 * kKeys, lane);
    for (int j = j0; j < j1; ++j) {
        Tile<D> now = t;
        if (j + 1 < j1) load_tile<D>(t, cache, page, Hkv, head, pg, (j + 1) * kKeys, lane);
        const int key = j * kKeys;
        const bool whole = now.has[0] && now.has[1] && key + kKeys <= end;
        f32x4 s[NT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float f = kv4_scale(now.ks[h]);
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < D / 32; ++m) {
                const bf16x8 k = kv4_values(now.k[h][m], f);
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[n][m], s[n][h], 0, 0, 0);
            }
        }
        if (!whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (!now.has[h] || key + 16 * h + 4 * quarter + v >= end)
#pragma unroll
                        for (int n = 0; n < NT; ++n) s[n][h][v] = -INFINITY;
                // what is no key may hold anything: its weight of zero has to meet zeros
                const bool out = !now.has[h] || key + 16 * h + i >= end;
#pragma unroll
                for (int m = 0; m < D / 32; ++m) now.v[h][m] = out ? 0u : now.v[h][m];
                now.vs[h] = out ? 127u : now.vs[h];
            }
        }
        // values to LDS: row 16 h + i, this lane's D / 4 of it
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float f = kv4_scale(now.vs[h]);
            const int r = 16 * h + i;
#pragma unroll
            for (int m = 0; m < D / 32; ++m)
                *(bf16x8*)((char*)lds + at + r * R::RB + (((quarter * (D / 32) + m) ^ R::swz(r)) * 16)) = kv4_values(now.v[h][m], f);
        }
        bf16x8 p[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float mx = s[n][0][0];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int v = 0; v < 4; ++v) mx = fmaxf(mx, s[n][h][v]);
            mx *= c;
            if (__any(mx > st[n].mc + 8.0f)) {
                const float mn = fmaxf(st[n].mc, max_quarters(mx));
                const float alpha = mn == -INFINITY ? 1.0f : exp2_hw(st[n].mc - mn);
                st[n].mc = mn;
                st[n].l *= alpha;
#pragma unroll
                for (int db = 0; db < D / 16; ++db)
#pragma unroll
                    for (int v = 0; v < 4; ++v) st[n].o[db][v] *= alpha;
            }
            const float sub = st[n].mc == -INFINITY ? 0.0f : st[n].mc;
            typedef float f32x8 __attribute__((ext_vector_type(8)));
            f32x8 w;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    w[4 * h + v] = exp2_hw(__builtin_fmaf(s[n][h][v], c, -sub));
                    st[n].l += w[4 * h + v];
                }
            p[n] = __builtin_convertvector(w, bf16x8);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int db = 0; db < D / 16; ++db) {
            typedef short s16x8 __attribute__((ext_vector_type(8)));
            s16x4 x[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = 16 * h + 4 * quarter + (i >> 2);
                x[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)lds_at(
                    lds, (unsigned)(at + r * R::RB + (((2 * db + ((i & 3) >> 1)) ^ R::swz(r)) * 16) + (i & 1) * 8)));
            }
            const s16x8 v = {x[0][0], x[0][1], x[0][2], x[0][3], x[1][0], x[1][1], x[1][2], x[1][3]};
#pragma unroll
            for (int n = 0; n < NT; ++n)
                st[n].o[db] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v), p[n], st[n].o[db], 0, 0, 0);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// What a workgroup does with one item.
struct Piece {
    int rank, head, j0, j1, part;      // tiles, and the part's number within its (rank, key head)
    bool direct;                       // the part is all there is: o is the result
};

template <int D, int NT, bool SHARED>
__device__ __forceinline__ void run_piece(const Kv4DecodeArgs& a, const Piece& w, int first_row, int rb, int end, unsigned short* lds,
                                          float (*wave_ml)[16][2]) {
    typedef Rows<D> R;
    constexpr int kTile = kKeys * R::RB;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, quarter = lane >> 4, G = a.Hq / a.Hkv;
    const int rows = SHARED ? a.group * G : G;                  // of the item's group or row
    auto row_of = [&](int r, int& b, int& head) {               // request and query head of the item's r-th row
        b = first_row + (SHARED ? r / G : 0);
        head = w.head * G + (SHARED ? r % G : r);
    };
    State<D> st[NT];
    bf16x8 q[NT][D / 32];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        st[n].init();
        const int r = (rb * NT + n) * 16 + i;
        int b, head;
        row_of(r < rows ? r : rows - 1, b, head);
        const unsigned short* p = a.q[w.rank] + b * a.q_stride + (long long)head * D + quarter * (D / 4);
#pragma unroll
        for (int m = 0; m < D / 32; ++m) q[n][m] = *(const bf16x8*)(p + 8 * m);
    }
    Pages pg;
    pg.init(a.table + (long long)first_row * a.width, (int)(((long long)end + (1 << a.shift) - 1) >> a.shift), a.shift, a.pages);
    const int n = w.j1 - w.j0, j0 = w.j0 + n * wave / kWaves, j1 = w.j0 + n * (wave + 1) / kWaves;
    const int at = wave * kTile;
    run_tiles<D, NT>(st, q, a.cache[w.rank], Kv4Page<D>{a.shift}, a.Hkv, w.head, pg, j0, j1, end, a.c, lds, at, lane);
    // the four waves' results, 16 rows at a time: [row][D] floats in each wave's
    // own tile, a row's 16-byte chunks placed by its number
    static_assert(16 * D * 4 <= kTile, "a wave's output fits its tile");
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float l = sum_quarters(st[nt].l);
        if (quarter == 0) {
            wave_ml[wave][i][0] = st[nt].mc;
            wave_ml[wave][i][1] = l;
        }
#pragma unroll
        for (int db = 0; db < D / 16; ++db)
            *(f32x4*)((char*)lds + at + i * D * 4 + (((4 * db + quarter) ^ i) * 16)) = st[nt].o[db];
        __syncthreads();
        const int t = threadIdx.x, r = t >> 4, row = (rb * NT + nt) * 16 + r;
        float mx = -INFINITY, sum = 0.0f, f[kWaves];
#pragma unroll
        for (int v = 0; v < kWaves; ++v) mx = fmaxf(mx, wave_ml[v][r][0]);
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            f[v] = mx == -INFINITY ? 0.0f : exp2_hw(wave_ml[v][r][0] - mx);
            sum += f[v] * wave_ml[v][r][1];
        }
        if (row < rows) {
            int b, head;
            row_of(row, b, head);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const int part_rows = SHARED ? NT * 16 : a.own_rows, part_row = SHARED ? nt * 16 + r : r;
            const long long slot = (long long)w.part * part_rows + part_row;
            float* po = (SHARED ? a.shared_o : a.own_o) + slot * D;
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                const int ch = (t & 15) + 16 * u;
                f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int v = 0; v < kWaves; ++v) {
                    const f32x4 y = *(const f32x4*)((const char*)lds + v * kTile + r * D * 4 + ((ch ^ r) * 16));
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] += f[v] * y[e];
                }
                if (w.direct) {
                    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] *= inv;
                    *(bf16x4*)(a.o[w.rank] + b * a.o_stride + (long long)head * D + 4 * ch) = __builtin_convertvector(x, bf16x4);
                } else {
                    *(f32x4*)(po + 4 * ch) = x;
                }
            }
            if (!w.direct && (t & 15) == 0) (SHARED ? a.shared_ml : a.own_ml)[slot] = float2{mx, sum};
        }
        __syncthreads();
    }
}

template <int D, int NT> __global__ __launch_bounds__(256, NT == 4 ? 1 : 2) void kv4_decode_kernel(Kv4DecodeArgs a) {
    extern __shared__ int lens[];                          // [B] lengths, [groups] shared tiles
    __shared__ __align__(4096) unsigned short lds[kWaves * kKeys * Rows<D>::RB / 2];
    __shared__ float wave_ml[kWaves][16][2];
    __shared__ int part_sum[kWaves], found[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int units = a.P * a.Hkv, unit = blockIdx.x % units, blk = blockIdx.x / units;
    const Items n = items_of(a);
    int* few = lens + a.B;                                 // per group: the shared keys' tiles
    if (blockIdx.x == 0 && tid == 0) ws_add_data(a.status, a.data);
    for (int g = tid; g < n.groups; g += 256) few[g] = a.pages ? clamp_len(a.shared[g], a.width, a.shift) : 0;
    __syncthreads();
    for (int b = tid; b < a.B; b += 256) {
        const int len = a.pages ? clamp_len(a.lengths[b], a.width, a.shift) : 0;
        lens[b] = len;
        if (n.groups) __hip_atomic_fetch_min(few + b / a.group, len, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
    for (int g = tid; g < n.groups; g += 256) few[g] /= kKeys;       // whole tiles; the rest is every row's own
    __syncthreads();
    // tiles of item it: its first one is the row's own or shared first one
    auto first_tile = [&](int b) { return n.groups ? few[b / a.group] : 0; };
    auto tiles = [&](int it) {
        if (it < n.shared) return few[it / a.shared_rbs];
        const int b = (it - n.shared) / a.own_rbs;
        return (lens[b] + kKeys - 1) / kKeys - first_tile(b);
    };
    // a run of items a thread, and one scan
    const int all = n.shared + n.own, run = (all + 255) / 256;
    const int i0 = tid * run < all ? tid * run : all, i1 = i0 + run < all ? i0 + run : all;
    int mine = 0;
    for (int it = i0; it < i1; ++it) mine += tiles(it);
    const int s = wave_scan(mine);
    if (lane == 63) part_sum[wave] = s;
    __syncthreads();
    int before = s - mine, total = 0;
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += part_sum[w];
        total += part_sum[w];
    }
    int quota = (total + a.blocks - 1) / a.blocks;
    if (quota < kMinTiles) quota = kMinTiles;
    if (blockIdx.x == 0) {                                 // for the launch that joins
        int at = before;
        for (int it = i0; it < i1; ++it) {
            a.start[it] = at;
            at += tiles(it);
        }
        if (tid == 0) {
            a.start[all] = total;
            a.start[all + 1] = quota;
        }
    }
    const long long t0 = (long long)blk * quota, t1 = t0 + quota < total ? t0 + quota : total;
    if (t0 >= t1) return;                                  // the workgroup as one
    if (t0 >= before && t0 < before + mine) {
        int it = i0, at = before;
        while (t0 >= at + tiles(it)) at += tiles(it++);
        found[0] = it;
        found[1] = at;
    }
    __syncthreads();
    int it = __builtin_amdgcn_readfirstlane(found[0]), at = __builtin_amdgcn_readfirstlane(found[1]);
    Piece w;
    w.rank = unit / a.Hkv;
    w.head = unit % a.Hkv;
    for (; at < t1; ++it) {
        const int m = __builtin_amdgcn_readfirstlane(tiles(it));
        const int lo = t0 > at ? (int)(t0 - at) : 0, hi = t1 < at + m ? (int)(t1 - at) : m;
        at += m;
        if (lo >= hi) continue;
        if (it < n.shared) {
            const int g = it / a.shared_rbs;
            w.j0 = lo;
            w.j1 = hi;
            w.part = unit * (n.shared + a.blocks) + it + blk;
            w.direct = false;
            run_piece<D, NT, true>(a, w, g * a.group, it % a.shared_rbs, m * kKeys, lds, wave_ml);
        } else {
            const int b = (it - n.shared) / a.own_rbs, f = __builtin_amdgcn_readfirstlane(first_tile(b));
            w.j0 = f + lo;
            w.j1 = f + hi;
            w.part = unit * (n.own + a.blocks) + it - n.shared + blk;
            w.direct = f == 0 && lo == 0 && hi == m;
            run_piece<D, 1, false>(a, w, b, (it - n.shared) % a.own_rbs, __builtin_amdgcn_readfirstlane(lens[b]), lds, wave_ml);
        }
    }
}

// The parts of every row, joined: D / 4 lanes a row.
template <int D, int NT> __global__ __launch_bounds__(256) void kv4_join_kernel(Kv4DecodeArgs a) {
    constexpr int L = D / 4, kRows = 256 / L;
    const int i = threadIdx.x % L;
    const long long all = (long long)a.P * a.B * a.Hq, m = (long long)blockIdx.x * kRows + threadIdx.x / L;
    if (m >= all) return;
    const int G = a.Hq / a.Hkv;
    const int head = (int)(m % a.Hq), b = (int)(m / a.Hq % a.B), rank = (int)(m / a.Hq / a.B);
    const int unit = rank * a.Hkv + head / G, r = head % G;
    const Items n = items_of(a);
    const int quota = a.start[n.shared + n.own + 1];
    // an item's parts: those of the workgroups its tiles go to; workgroup w has part item + w
    auto parts_of = [&](int it, int& w0) {
        const int lo = a.start[it], hi = a.start[it + 1];
        if (lo == hi) return 0;
        w0 = lo / quota;
        return (hi - 1) / quota - w0 + 1;
    };
    int w0 = 0, parts_s = 0;
    long long first_s = 0;
    if (n.groups) {
        const int row = (b % a.group) * G + r, it = b / a.group * a.shared_rbs + row / (16 * NT);
        parts_s = parts_of(it, w0);
        first_s = ((long long)unit * (n.shared + a.blocks) + it + w0) * (16 * NT) + row % (16 * NT);
    }
    const int own_it = b * a.own_rbs + r / 16, parts_o = parts_of(n.shared + own_it, w0);
    if (parts_o == 1 && !parts_s) return;                    // its one part is the result
    const long long first_o = ((long long)unit * (n.own + a.blocks) + own_it + w0) * a.own_rows + r % 16;
    float mx = -INFINITY, l = 0.0f;
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    auto join = [&](const float* o, const float2* ml, long long first, int parts, int rows) {
        float top = mx;
        for (int p = 0; p < parts; ++p) top = fmaxf(top, ml[first + (long long)p * rows].x);
        const float f0 = top == -INFINITY ? 0.0f : exp2_hw(mx - top);
        l *= f0;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= f0;
#pragma unroll 4
        for (int p = 0; p < parts; ++p) {
            const long long s = first + (long long)p * rows;
            const float2 y = ml[s];
            const f32x4 z = *(const f32x4*)(o + s * D + 4 * i);
            const float f = top == -INFINITY ? 0.0f : exp2_hw(y.x - top);
            l += f * y.y;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] += f * z[e];
        }
        mx = top;
    };
    join(a.shared_o, a.shared_ml, first_s, parts_s, 16 * NT);
    join(a.own_o, a.own_ml, first_o, parts_o, a.own_rows);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= inv;
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    *(bf16x4*)(a.o[rank] + b * a.o_stride + (long long)head * D + 4 * i) = __builtin_convertvector(x, bf16x4);
}

struct Kv4Cut {
    int nt, blocks, shared_rbs, own_rbs, own_rows;
    size_t shared_parts, own_parts, items;                   // parts over all (rank, key head)
};
Kv4Cut kv4_cut(int P, int B, int group, bool shared, int Hq, int Hkv, int cus) {
    Kv4Cut c;
    const int G = Hq / Hkv;
    const long long units = (long long)P * Hkv, rows = (long long)group * G;
    c.nt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    c.shared_rbs = (int)((rows + 16 * c.nt - 1) / (16 * c.nt));
    c.own_rbs = (G + 15) / 16;
    c.own_rows = G < 16 ? G : 16;
    c.blocks = (int)((kPerCu * (long long)cus + units - 1) / units);
    const size_t ns = shared ? (size_t)(B / group) * c.shared_rbs : 0, no = (size_t)B * c.own_rbs;
    c.items = ns + no;
    c.shared_parts = shared ? (ns + c.blocks) * (size_t)units : 0;
    c.own_parts = (no + c.blocks) * (size_t)units;
    return c;
}
size_t kv4_ws(const Kv4Cut& c, int D) {
    const size_t n = c.shared_parts * 16 * c.nt + c.own_parts * c.own_rows;
    return kStatusBytes + (n * (D + 2) * 4 + (c.items + 2) * 4 + 255) / 256 * 256;
}
bool kv4_decode_shape(int P, int B, int group, int Hq, int Hkv, int D) {
    return P >= 1 && P <= RING_MAX_RANKS && B >= 0 && B <= KV_FORK_MAX_ROWS && group >= 1 && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 &&
           (D == 64 || D == 128) && (long long)Hq * D < kMaxRow;
}

}  // namespace
}  // namespace ringc

using namespace ringc;

extern "C" size_t tp_attention_decode_kv4_workspace_bytes(int P, int B, int group, int Hq, int Hkv, int D) {
    if (!kv4_decode_shape(P, B, group, Hq, Hkv, D) || B % group) return 0;
    return kv4_ws(kv4_cut(P, B, group, true, Hq, Hkv, dev_info().cus), D);
}

extern "C" int tp_attention_decode_kv4(const void* const* q, const void* const* cache, void* const* o, const int* block_table,
                                       const int* lengths, const int* shared, int P, int B, int group, int Hq, int Hkv, int D,
                                       int table_stride, int page_size, int pages, long long q_stride, long long o_stride,
                                       float scale, void* ws, size_t ws_bytes, void* stream) {
    if (P < 1 || P > RING_MAX_RANKS || B < 0 || group < 1 || Hq < 1 || Hkv < 1 || table_stride < 0 || pages < 0 || B % group)
        return RING_EINVAL;
    if (!scale_ok(scale)) return RING_EINVAL;
    if (!kv4_decode_shape(P, B, group, Hq, Hkv, D) || !kv4_page_ok(page_size) || (long long)pages * page_size >= (1LL << 31) ||
        (long long)table_stride * page_size >= (1LL << 31) - 64)
        return RING_EUNSUPPORTED;
    if (!row_stride_ok(q_stride, Hq, D) || !row_stride_ok(o_stride, Hq, D)) return RING_EINVAL;
    if (B == 0) return RING_OK;
    if (!q || !cache || !o || !lengths || ((uintptr_t)lengths & 3) || (table_stride && !block_table) || ((uintptr_t)block_table & 3) ||
        ((uintptr_t)shared & 3))
        return RING_EINVAL;
    Kv4DecodeArgs a;
    for (int r = 0; r < P; ++r) {
        if (!q[r] || !o[r] || (pages && !cache[r])) return RING_EINVAL;
        if (((uintptr_t)q[r] | (uintptr_t)o[r] | (uintptr_t)cache[r]) & 15) return RING_EINVAL;
        a.q[r] = (const unsigned short*)q[r];
        a.cache[r] = (const char*)cache[r];
        a.o[r] = (unsigned short*)o[r];
    }
    if (group == 1) shared = nullptr;                        // a row's shared keys are its own
    const Kv4Cut c = kv4_cut(P, B, group, shared != nullptr, Hq, Hkv, dev_info().cus);
    const size_t need = kv4_ws(c, D);
    if (!ws || ((uintptr_t)ws & 255) || ws_bytes < need) return RING_EWORKSPACE;
    // a workgroup's tiles are counted in 32 bits
    if ((long long)(B / group * c.shared_rbs + B * c.own_rbs) * ((long long)table_stride * page_size / kKeys + 1) >= (1LL << 31) ||
        (long long)P * B * Hq >= (1LL << 31) || (c.shared_parts * 16 * c.nt + c.own_parts * c.own_rows) >= (1ull << 31))
        return RING_EUNSUPPORTED;
    a.table = block_table;
    a.lengths = lengths;
    a.shared = shared;
    a.q_stride = q_stride;
    a.o_stride = o_stride;
    a.P = P;
    a.B = B;
    a.group = group;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.width = table_stride;
    a.shift = 0;
    while ((1 << a.shift) < page_size) ++a.shift;
    a.pages = pages;
    a.blocks = c.blocks;
    a.shared_rbs = c.shared_rbs;
    a.own_rbs = c.own_rbs;
    a.own_rows = c.own_rows;
    a.c = scale * kLog2e;
    a.shared_o = (float*)((char*)ws + kStatusBytes);
    a.own_o = a.shared_o + c.shared_parts * 16 * c.nt * D;
    a.shared_ml = (float2*)(a.own_o + c.own_parts * c.own_rows * D);
    a.own_ml = a.shared_ml + c.shared_parts * 16 * c.nt;
    a.start = (int*)(a.own_ml + c.own_parts * c.own_rows);
    a.status = (Status*)ws;
    a.data = WsSpan{kStatusBytes, need};
    hipStream_t s = (hipStream_t)stream;
    const int units = P * Hkv;
    const dim3 grid((unsigned)(units * c.blocks));
    const size_t dyn = ((size_t)B + (shared ? B / group : 0)) * sizeof(int);
    const long long rows = (long long)P * B * Hq;
    const dim3 jg((unsigned)((rows + 1024 / D - 1) / (1024 / D)));
    auto go = [&](auto d, auto nt) -> int {
        constexpr int kD = decltype(d)::value, kNT = decltype(nt)::value;
        hipLaunchKernelGGL((kv4_decode_kernel<kD, kNT>), grid, dim3(256), dyn, s, a);
        if (hipGetLastError() != hipSuccess) return RING_EHIP;
        hipLaunchKernelGGL((kv4_join_kernel<kD, kNT>), jg, dim3(256), 0, s, a);
        return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
    };
    auto with_nt = [&](auto d) -> int {
        if (!shared || c.nt == 1) return go(d, std::integral_constant<int, 1>());
        if (c.nt == 2) return go(d, std::integral_constant<int, 2>());
        return go(d, std::integral_constant<int, 4>());
    };
    return D == 128 ? with_nt(std::integral_constant<int, 128>()) : with_nt(std::integral_constant<int, 64>());
}
