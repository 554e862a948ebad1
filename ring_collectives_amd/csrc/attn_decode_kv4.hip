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
// tiles of 32 keys.  Every (rank, key head) has the same items; its waves each
// take consecutive tiles of the same cost in all, found from the sums of the
// items' costs that every workgroup makes for itself in LDS.  Four waves that
// are all within one item join their results in LDS, so that long items make
// few parts; others go through their items by themselves, without a barrier.
// A part that is all of its row's keys is the result; a second launch joins the
// rest.  Where the table's rows hold 2048 keys at most and nothing is shared,
// every row is one workgroup's and there is neither scan nor second launch.
//
// A wave's tile goes from memory to registers (two 16-byte loads a lane each
// for key and value codes at width 128, a byte each for their scales), one tile
// ahead.  A lane holds whole scale blocks of one key, so the conversion to bf16,
// two codes an instruction, leaves the A operand of S^T = K Q^T as it is: the
// order of the sum over the head's values is that of the lanes' bytes, for K
// and Q alike.  Values go to LDS as bf16 and are read transposed for
// O^T += V^T P^T, whose B operand are S^T's accumulators rounded to bf16.
//
// The cache read bounds it, 4.25 bits a value: 4 rows of 120000 keys of 2 heads
// on 4 ranks, 382 MB, take 62 us, 6.2 TB/s, what reads alone reach here.  24
// groups of 4 beams of 3000 keys, 2700 of them shared, take 24 us for 89 MB read
// and 12 MB of parts written: 2.5 before the first load (lengths, costs and the
// search), 14 at 6.3 TB/s, then 4 until the last wave, whose pieces and pages
// the costs do not foresee.  The launches that join take 5 to 6.
#include "kv4_core.h"

#include <hip/hip_runtime.h>

namespace ringc {
namespace {

constexpr int kWaves = 4;
constexpr int kKeys = 32;              // of a tile
constexpr int kOwnCost = 2;            // of a tile of own keys
// Of an item besides its tiles: its look-ups, and storing its part.  60 groups
// of 4 rows of 1000 keys on 8 ranks 43.7 us, with half of it 44.9; 6 groups of 16
// of 3000 27.6 and 28.6; 2 groups of 4 of 300 12.0 and 13.0; 8 groups of 8 of
// 3000 24.0 and 23.9.
constexpr int kItemCost = 8;
// Rows of at most as many tiles are a workgroup's each.  3 requests of up to 600 /
// 1100 keys on 2 ranks of 2 key heads 7.6 / 9.2 us so, shared out 12; 64 on 4
// ranks 12.7 / 17.5, shared out 17.9 / 21.7, of 2200 27.7 and 29.7; but the only
// long row of a batch is one workgroup's too, and at 2048 keys that takes as
// long as sharing out and joining.
constexpr int kWholeTiles = 64;
// Of a wave, if there is as much (and no less than a tile's).  3 requests of 200 /
// 600 keys in a table of 8192 10.3 / 11.9 us, one of 10000 12.5; with 2 10.3 / 11.3
// and 12.3, with 8 11.3 / 12.5 and 13.3, with 16 11.2 / 14.5 and 15.5; calls of many
// keys alike.
constexpr int kMinCost = 4;

// An item's parts: a wave's each, those before the first and after the last
// workgroup that is within the item, and one each for the workgroups between.
struct alignas(16) ItemParts {
    int w0, inner, outer, n;           // first wave; the first wave of the workgroups within, and past them; parts
    __device__ __forceinline__ int wave(int p) const {
        const int head = inner - w0, mid = (outer - inner) / kWaves;
        return p < head ? w0 + p : p < head + mid ? inner + (p - head) * kWaves : outer + (p - head - mid);
    }
};
// Of an item of cost [lo, hi) of `total`, kItemCost and its tiles' c each, and
// waves of cost quota.
__device__ __forceinline__ ItemParts item_parts(unsigned lo, unsigned hi, unsigned c, unsigned total, unsigned quota) {
    if (lo == hi) return ItemParts{0, 0, 0, 0};
    const unsigned quad = kWaves * quota;
    unsigned w0 = (lo + kItemCost) / quota;                // that the first tile begins in
    const unsigned w1 = (hi - c) / quota + 1;              // past the one that the last tile begins in
    unsigned b0 = w0 / kWaves, b1 = hi == total ? (hi + quad - 1) / quad : hi / quad;
    if (b0 * quad < lo) ++b0;
    if (b1 * kWaves > w1) b1 = (w1 + kWaves - 1) / kWaves; // a last workgroup without a tile, or with few waves' share
    const unsigned inner = b0 < b1 ? b0 * kWaves : w1, outer = b0 < b1 ? b1 * kWaves : w1;
    if (w0 > inner) w0 = inner;                            // a first workgroup that is within the item
    return ItemParts{(int)w0, (int)inner, (int)outer, (int)(inner - w0 + (outer - inner) / kWaves + (outer < w1 ? w1 - outer : 0))};
}

struct Kv4DecodeArgs {
    const unsigned short* q[RING_MAX_RANKS];
    const char* cache[RING_MAX_RANKS];
    unsigned short* o[RING_MAX_RANKS];
    const int *table, *lengths, *shared;
    long long q_stride, o_stride;
    int P, B, group, Hq, Hkv, width, shift, pages;
    int blocks, waves;                 // workgroups and waves of a (rank, key head)
    int planners;                      // workgroups that write the items' parts
    int shared_cost;                   // of a tile of shared keys
    int whole;                         // every row's keys are one workgroup's
    int shared_rbs, own_rbs, own_rows; // row blocks of a group, of a row; rows of an own part
    float c;
    float *shared_o, *own_o;           // [P Hkv][part][rows][D]
    float2 *shared_ml, *own_ml;        // [P Hkv][part][rows]
    struct ItemParts* parts;           // [items]
    Status* status;
    WsSpan data;
};

// A rank's pointers and the sizes that the loops use, read in one trip to
// argument memory at the start (see read_sizes in attn_core.h).
struct Fixed {
    Global<const char> cache;
    Global<const unsigned short> q;
    Global<unsigned short> o;
    Global<const int> table;
    long long q_stride, o_stride;
    int group, G, Hkv, width, shift, pages;
    float c;
};
__device__ __forceinline__ Fixed read_fixed(const Kv4DecodeArgs& a, int rank) {
    Fixed f = {(Global<const char>)a.cache[rank], (Global<const unsigned short>)a.q[rank], (Global<unsigned short>)a.o[rank],
               (Global<const int>)a.table, a.q_stride, a.o_stride, a.group, a.Hq / a.Hkv, a.Hkv, a.width, a.shift, a.pages, a.c};
    asm volatile("" : "+s"(f.cache), "+s"(f.q), "+s"(f.o), "+s"(f.table), "+s"(f.q_stride), "+s"(f.o_stride), "+s"(f.group),
                      "+s"(f.Hkv), "+s"(f.width), "+s"(f.shift), "+s"(f.pages), "+s"(f.c));
    return f;
}

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
// block of four of the values, and the sum of the weights four times (of which
// only the first is kept up when the maximum rises).
template <int D> struct State {
    f32x4 o[D / 16], l;
    float mc;
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int db = 0; db < D / 16; ++db) o[db] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        mc = -INFINITY;
        l = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
};
__device__ __forceinline__ float max_quarters(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}

// One tile of a wave, as loaded: half h holds keys 16 h + lane % 16.
template <int D> struct Tile {
    typedef unsigned word __attribute__((ext_vector_type(D / 32)));
    word k[2], v[2];
    unsigned ks[2], vs[2];
};

// A value tile in LDS: rows of D bf16 values with 16 bytes between them, so
// that the 16 rows that a transposed read touches lie on distinct banks.
template <int D> constexpr int kRowBytes = 2 * D + 16;
template <int D> constexpr int kTileBytes = kKeys * kRowBytes<D>;

// A wave's tiles [j0, j1) of one item for NT times 16 rows.  Keys from `end` on
// are no keys of a row; the page of key k is row[k >> shift].
template <int D, int NT>
__device__ __forceinline__ void run_tiles(State<D> (&st)[NT], const bf16x8 (&q)[NT][D / 32], const Fixed& f, int kv_head,
                                          Global<const int> row, int j0, int j1, int end, unsigned short* lds, int at, int lane) {
    const int i = lane & 15, quarter = lane >> 4;
    const Kv4Page<D> page{f.shift};
    // this lane's bytes of a tile's first half, from its keys' codes and scales on
    const unsigned kc = i * (D / 2) + quarter * (D / 8), vc = kc + page.codes(1, 0);
    const unsigned ksc = page.scales(0, i) + quarter * D / 128, vsc = ksc + page.scales(1, 0) - page.scales(0, 0);
    const unsigned long long bytes = (unsigned)page.bytes(), stride = (unsigned)f.Hkv * bytes;       // a page of all heads may pass 4 GiB
    Global<const char> head = f.cache + (unsigned)kv_head * bytes;
    const unsigned mask = (1u << f.shift) - 1;
    const int write = at + i * kRowBytes<D> + quarter * (D / 2);
    const int read = at + (4 * quarter + (i >> 2)) * kRowBytes<D> + (i & 3) * 8;
    bf16x8 ones;
#pragma unroll
    for (int e = 0; e < 8; ++e) ones[e] = (__bf16)1.0f;
    // 64 pages are looked up at a time; loads within them wait for no look-up
    for (int jc = j0; jc < j1;) {
        const int first = (int)((unsigned)jc * kKeys >> f.shift);
        const unsigned past = ((unsigned)(first + 64) << f.shift) / kKeys;
        const int jn = past < (unsigned)j1 ? (int)past : j1;
        int ids = first + lane <= (end - 1) >> f.shift ? row[first + lane] : -1;
        if (ids >= f.pages) ids = -1;
        Tile<D> t;
        bool has[2];                                   // the halves' pages are pages
        Global<const char> codes[2], scales[2];
        auto look = [&](int j) __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const unsigned key = (unsigned)j * kKeys + 16 * h;
                const int p = __builtin_amdgcn_readlane(ids, (key >> f.shift) - first);
                has[h] = p >= 0;
                Global<const char> base = head + (p < 0 ? 0u : (unsigned)p) * stride;
                codes[h] = base + (key & mask) * (D / 2);
                scales[h] = base + (key & mask) * (D / 32);
            }
        };
        auto load_keys = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                t.k[h] = __builtin_nontemporal_load((Global<const typename Tile<D>::word>)(codes[h] + kc));
                t.ks[h] = *(Global<const unsigned char>)(scales[h] + ksc);
            }
        };
        auto load_values = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                t.v[h] = __builtin_nontemporal_load((Global<const typename Tile<D>::word>)(codes[h] + vc));
                t.vs[h] = *(Global<const unsigned char>)(scales[h] + vsc);
            }
        };
        look(jc);
        load_keys();
        load_values();
        for (int j = jc; j < jn; ++j) {
            const int key = j * kKeys;
            const bool had[2] = {has[0], has[1]};
            f32x4 s[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) s[n][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < D / 32; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bf16x8 k = kv4_values(t.k[h][m], kv4_scale(t.ks[h]));
#pragma unroll
                    for (int n = 0; n < NT; ++n) s[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[n][m], s[n][h], 0, 0, 0);
                }
            // the next tile (the last one again, past it: a load that only some
            // steps make would have every step wait for all)
            look(j + 1 < jn ? j + 1 : j);
            load_keys();
            if (!had[0] || !had[1] || key + kKeys > end) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (!had[h] || key + 16 * h + 4 * quarter + v >= end)
#pragma unroll
                            for (int n = 0; n < NT; ++n) s[n][h][v] = -INFINITY;
                    // what is no key may hold anything: its weight of zero has to meet zeros
                    const bool out = !had[h] || key + 16 * h + i >= end;
#pragma unroll
                    for (int m = 0; m < D / 32; ++m) t.v[h][m] = out ? 0u : t.v[h][m];
                    t.vs[h] = out ? 127u : t.vs[h];
                }
            }
            // values to LDS: row 16 h + i, this lane's D / 4 of it
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float scale = kv4_scale(t.vs[h]);
#pragma unroll
                for (int m = 0; m < D / 32; ++m)
                    *(bf16x8*)((char*)lds + write + 16 * h * kRowBytes<D> + 16 * m) = kv4_values(t.v[h][m], scale);
            }
            load_values();
            bf16x8 p[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float mx = s[n][0][0];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int v = 0; v < 4; ++v) mx = fmaxf(mx, s[n][h][v]);
                mx *= f.c;
                if (__any(mx > st[n].mc + 8.0f)) {
                    const float mn = fmaxf(st[n].mc, max_quarters(mx));
                    const float alpha = mn == -INFINITY ? 1.0f : exp2_hw(st[n].mc - mn);
                    st[n].mc = mn;
                    st[n].l[0] *= alpha;
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
                    for (int v = 0; v < 4; ++v) w[4 * h + v] = exp2_hw(__builtin_fmaf(s[n][h][v], f.c, -sub));
                p[n] = __builtin_convertvector(w, bf16x8);
                // the sum is of the weights as rounded, so that where few keys have
                // most of the weight its rounding cancels (over five inputs 24 groups of
                // 4 rows of 3000 keys are off by 2.05e-3 to 2.10e-3 so, 2.15e-3 to
                // 2.21e-3 with the sum of unrounded ones; 3 rows of 200 by 1.75e-3 to
                // 1.84e-3 both ways), and a product with ones (66.5 us for 4 rows of
                // 120000 keys, 67.5 with additions)
                st[n].l = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, p[n], st[n].l, 0, 0, 0);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (int db = 0; db < D / 16; ++db) {
                typedef short s16x8 __attribute__((ext_vector_type(8)));
                s16x4 x[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    x[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)lds_at(lds, (unsigned)(read + 16 * h * kRowBytes<D> + 32 * db)));
                const s16x8 v = {x[0][0], x[0][1], x[0][2], x[0][3], x[1][0], x[1][1], x[1][2], x[1][3]};
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    st[n].o[db] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v), p[n], st[n].o[db], 0, 0, 0);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        jc = jn;
    }
}

// What a wave, or the four of a workgroup together, do with one item.
struct Piece {
    int head, j0, j1, part;            // tiles, and the part's number
    bool joint;                        // the workgroup's
    bool direct;                       // the part is all there is: o is the result
};

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store4(Global<unsigned short> p, f32x4 x, float f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= f;
    *(Global<bf16x4>)p = __builtin_convertvector(x, bf16x4);
}

template <int D, int NT, bool SHARED>
__device__ __forceinline__ void run_piece(const Kv4DecodeArgs& a, const Fixed& f, const Piece& w, int first_row, int rb, int end, unsigned short* lds,
                                          float (*wave_ml)[16][2]) {
    constexpr int kTile = kTileBytes<D>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, quarter = lane >> 4, G = f.G;
    const int rows = SHARED ? f.group * G : G;                  // of the item's group or row
    auto row_of = [&](int r, int& b, int& head) {               // request and query head of the item's r-th row
        b = first_row + (SHARED ? r / G : 0);
        head = w.head * G + (SHARED ? r % G : r);
    };
    auto result = [&](int row) {
        int b, head;
        row_of(row, b, head);
        return f.o + b * f.o_stride + (long long)head * D;
    };
    State<D> st[NT];
    bf16x8 q[NT][D / 32];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        st[n].init();
        const int r = (rb * NT + n) * 16 + i;
        int b, head;
        row_of(r < rows ? r : rows - 1, b, head);
        Global<const unsigned short> p = f.q + b * f.q_stride + (long long)head * D + quarter * (D / 4);
#pragma unroll
        for (int m = 0; m < D / 32; ++m) q[n][m] = *(Global<const bf16x8>)(p + 8 * m);
    }
    const int n = w.j1 - w.j0, j0 = w.joint ? w.j0 + n * wave / kWaves : w.j0, j1 = w.joint ? w.j0 + n * (wave + 1) / kWaves : w.j1;
    const int at = wave * kTile;
    run_tiles<D, NT>(st, q, f, w.head, f.table + (long long)first_row * f.width, j0, j1, end, lds, at, lane);
    const int part_rows = SHARED ? NT * 16 : a.own_rows;
    float* po = (SHARED ? a.shared_o : a.own_o) + (long long)w.part * part_rows * D;
    float2* pml = (SHARED ? a.shared_ml : a.own_ml) + (long long)w.part * part_rows;
    if (!w.joint) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = (rb * NT + nt) * 16 + i, at_row = nt * 16 + i;
            const float l = st[nt].l[0];
            if (row >= rows) continue;
            if (w.direct) {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                Global<unsigned short> o = result(row);
#pragma unroll
                for (int db = 0; db < D / 16; ++db) store4(o + 16 * db + 4 * quarter, st[nt].o[db], inv);
            } else {
#pragma unroll
                for (int db = 0; db < D / 16; ++db) *(f32x4*)(po + at_row * D + 16 * db + 4 * quarter) = st[nt].o[db];
                if (quarter == 0) pml[at_row] = float2{st[nt].mc, l};
            }
        }
        return;
    }
    // the four waves' results, 16 rows at a time: [row][D] floats in each wave's
    // own tile, a row's 16-byte chunks placed by its number
    static_assert(16 * D * 4 <= kTile, "a wave's output fits its tile");
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float l = st[nt].l[0];
        if (quarter == 0) {
            wave_ml[wave][i][0] = st[nt].mc;
            wave_ml[wave][i][1] = l;
        }
#pragma unroll
        for (int db = 0; db < D / 16; ++db)
            *(f32x4*)((char*)lds + at + i * D * 4 + (((4 * db + quarter) ^ i) * 16)) = st[nt].o[db];
        __syncthreads();
        const int t = threadIdx.x, r = t >> 4, row = (rb * NT + nt) * 16 + r;
        float mx = -INFINITY, sum = 0.0f, part[kWaves];
#pragma unroll
        for (int v = 0; v < kWaves; ++v) mx = fmaxf(mx, wave_ml[v][r][0]);
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            part[v] = mx == -INFINITY ? 0.0f : exp2_hw(wave_ml[v][r][0] - mx);
            sum += part[v] * wave_ml[v][r][1];
        }
        if (row < rows) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                const int ch = (t & 15) + 16 * u;
                f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int v = 0; v < kWaves; ++v) {
                    const f32x4 y = *(const f32x4*)((const char*)lds + v * kTile + r * D * 4 + ((ch ^ r) * 16));
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] += part[v] * y[e];
                }
                if (w.direct) store4(result(row) + 4 * ch, x, inv);
                else *(f32x4*)(po + (nt * 16 + r) * D + 4 * ch) = x;
            }
            if (!w.direct && (t & 15) == 0) pml[nt * 16 + r] = float2{mx, sum};
        }
        __syncthreads();
    }
}

template <int D, int NT> __global__ __launch_bounds__(256, NT == 1 ? 3 : 2) void kv4_decode_kernel(Kv4DecodeArgs a) {
    extern __shared__ int lens[];                          // [B] lengths, [B] own tiles, [groups] shared tiles
    __shared__ __align__(4096) unsigned short lds[kWaves * kTileBytes<D> / 2];
    __shared__ float wave_ml[kWaves][16][2];
    __shared__ int part_sum[kWaves], found[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int units = a.P * a.Hkv, unit = blockIdx.x % units, blk = blockIdx.x / units;
    const int planner = (int)blockIdx.x - units * a.blocks;
    const Items n = items_of(a);
    int *own = lens + a.B, *few = own + a.B;
    if (blockIdx.x == 0 && tid == 0) ws_add_data(a.status, a.data);
    const int len0 = tid < a.B ? a.lengths[tid] : 0, few0 = tid < n.groups ? a.shared[tid] : 0;     // in one trip, where few
    const Fixed f = read_fixed(a, unit / a.Hkv);
    auto tokens = [&](int x) { return f.pages ? clamp_len(x, f.width, f.shift) : 0; };
    if (a.whole) {
        if (tid == 0) {
            const int b = blk / a.own_rbs, len = tokens(a.lengths[b]);
            lens[b] = len;
            own[b] = (len + kKeys - 1) / kKeys;
        }
    } else {
        for (int b = tid; b < a.B; b += 256) lens[b] = tokens(b < 256 ? len0 : a.lengths[b]);
        for (int g = tid; g < n.groups; g += 256) few[g] = tokens(g < 256 ? few0 : a.shared[g]);
        __syncthreads();
        if (n.groups) {
            for (int b = tid; b < a.B; b += 256)
                __hip_atomic_fetch_min(few + b / f.group, lens[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            __syncthreads();
        }
        // whole tiles are shared; the rest is every row's own
        for (int b = tid; b < a.B; b += 256) own[b] = (lens[b] + kKeys - 1) / kKeys - (n.groups ? few[b / f.group] / kKeys : 0);
    }
    __syncthreads();
    auto per = [](int x, int y) { return y == 1 ? x : x / y; };
    auto tiles = [&](int it) { return it < n.shared ? few[per(it, a.shared_rbs)] / kKeys : own[per(it - n.shared, a.own_rbs)]; };
    auto tile_cost = [&](int it) { return it < n.shared ? a.shared_cost : kOwnCost; };
    auto cost = [&](int it) {
        const int m = tiles(it);
        return m ? m * tile_cost(it) + kItemCost : 0;
    };
    Piece w;
    w.head = unit % f.Hkv;
    int it = blk, at = 0, worker = 0;
    long long t0 = 0, t1 = 0;
    w.joint = true;
    if (!a.whole) {
        // a run of items a thread, and one scan
        const int all = n.shared + n.own, run = (all + 255) / 256;
        const int i0 = tid * run < all ? tid * run : all, i1 = i0 + run < all ? i0 + run : all;
        int mine = 0;
        for (int i = i0; i < i1; ++i) mine += cost(i);
        const int s = wave_scan(mine);
        if (lane == 63) part_sum[wave] = s;
        __syncthreads();
        int before = s - mine, total = 0;
        for (int v = 0; v < kWaves; ++v) {
            if (v < wave) before += part_sum[v];
            total += part_sum[v];
        }
        int quota = (total + a.waves - 1) / a.waves;       // of a wave
        if (quota < kMinCost) quota = kMinCost;
        if (quota < a.shared_cost) quota = a.shared_cost;
        if (planner >= 0) {                                // for the launch that joins
            int x = before;
            for (int i = i0; i < i1; ++i) {
                const int c = cost(i);
                if (i % a.planners == planner) a.parts[i] = item_parts(x, x + c, tile_cost(i), total, quota);
                x += c;
            }
            return;
        }
        // a tile is the wave's in whose share its cost begins
        const long long block0 = (long long)blk * kWaves * quota;
        if (block0 >= total) return;                       // the workgroup as one
        if (block0 >= before && block0 < before + mine) {
            int i = i0, x = before;
            while (block0 >= x + cost(i)) x += cost(i++);
            found[0] = i;
            found[1] = x;
        }
        __syncthreads();
        it = __builtin_amdgcn_readfirstlane(found[0]);
        at = __builtin_amdgcn_readfirstlane(found[1]);
        const long long block1 = block0 + kWaves * quota < total ? block0 + kWaves * quota : total;
        w.joint = block1 <= at + __builtin_amdgcn_readfirstlane(cost(it));
        worker = blk * kWaves + (w.joint ? 0 : wave);
        t0 = w.joint ? block0 : block0 + wave * quota;
        t1 = w.joint ? block1 : t0 + quota < total ? t0 + quota : total;
    }
    for (bool more = a.whole || at < t1; more; ++it) {
        const int m = __builtin_amdgcn_readfirstlane(tiles(it)), c = tile_cost(it);
        const int begin = at + kItemCost;                  // of its tiles
        const int lo = t0 > begin ? (int)((t0 - begin + c - 1) / c) : 0;
        const int hi = a.whole || t1 >= begin + (long long)m * c ? m : t1 > begin ? (int)((t1 - begin + c - 1) / c) : 0;
        if (m) at = begin + m * c;
        more = !a.whole && at < t1;
        if (lo >= hi && !a.whole) continue;
        if (it < n.shared) {
            w.j0 = lo;
            w.j1 = hi;
            w.part = unit * (n.shared + a.waves) + it + worker;
            w.direct = false;
            const int g = per(it, a.shared_rbs);
            run_piece<D, NT, true>(a, f, w, g * f.group, it - g * a.shared_rbs, m * kKeys, lds, wave_ml);
        } else {
            const int b = per(it - n.shared, a.own_rbs), len = __builtin_amdgcn_readfirstlane(lens[b]), first = (len + kKeys - 1) / kKeys - m;
            w.j0 = first + lo;
            w.j1 = first + hi;
            w.part = unit * (n.own + a.waves) + it - n.shared + worker;
            w.direct = first == 0 && lo == 0 && hi == m;
            run_piece<D, 1, false>(a, f, w, b, it - n.shared - b * a.own_rbs, len, lds, wave_ml);
        }
    }
}

// The parts of every row, joined: T lanes a row, D / 4 of them a part at a time,
// each with 16 bytes of it.
template <int D, int NT, int T> __global__ __launch_bounds__(256) void kv4_join_kernel(Kv4DecodeArgs a) {
    constexpr int L = D / 4, kGroups = T / L, kBatch = 4;
    __shared__ f32x4 sum[256 / T][kGroups][L];
    __shared__ float2 stat[256 / T][kGroups];
    const int t = threadIdx.x % T, i = t % L, g = t / L, slot = threadIdx.x / T;
    const int slots = (a.Hq + 256 / T - 1) / (256 / T);      // workgroups of a row's heads
    const int rank = blockIdx.y, b = blockIdx.x / slots;
    const int head0 = __builtin_amdgcn_readfirstlane(blockIdx.x % slots * (256 / T) + slot), head = head0 < a.Hq ? head0 : a.Hq - 1;
    const int G = a.Hq / a.Hkv, r = head % G, unit = rank * a.Hkv + head / G;
    const Items n = items_of(a);
    ItemParts ps = {0, 0, 0, 0};
    int it_s = 0, row_s = 0;
    if (n.groups) {
        row_s = b % a.group * G + r;
        it_s = b / a.group * a.shared_rbs + row_s / (16 * NT);
        ps = a.parts[it_s];
    }
    const int it_o = b * a.own_rbs + r / 16;
    const ItemParts po = a.parts[n.shared + it_o];
    const bool whole = !ps.n && po.n == 1;                   // the one part is the result
    float mx = -INFINITY, l = 0.0f;
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    auto join = [&](const float* o, const float2* ml, const ItemParts& p, long long first, int rows) {
        for (int k = g; k < p.n; k += kBatch * kGroups) {
            float2 y[kBatch];
            f32x4 z[kBatch];
            float top = mx;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const bool there = k + u * kGroups < p.n;
                const long long at = first + (long long)p.wave(there ? k + u * kGroups : 0) * rows;
                y[u] = ml[at];
                z[u] = *(const f32x4*)(o + at * D + 4 * i);
                if (!there) {
                    y[u] = float2{-INFINITY, 0.0f};
                    z[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) top = fmaxf(top, y[u].x);
            const float sub = top == -INFINITY ? 0.0f : top, f0 = exp2_hw(mx - sub);
            l *= f0;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] *= f0;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const float f = exp2_hw(y[u].x - sub);
                l += f * y[u].y;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] += f * z[u][e];
            }
            mx = top;
        }
    };
    if (!whole) {
        join(a.shared_o, a.shared_ml, ps, ((long long)unit * (n.shared + a.waves) + it_s) * (16 * NT) + row_s % (16 * NT), 16 * NT);
        join(a.own_o, a.own_ml, po, ((long long)unit * (n.own + a.waves) + it_o) * a.own_rows + r % 16, a.own_rows);
    }
    sum[slot][g][i] = x;
    if (i == 0) stat[slot][g] = float2{mx, l};
    __syncthreads();
    if (g || whole || head0 >= a.Hq) return;
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kGroups; ++u) top = fmaxf(top, stat[slot][u].x);
    const float sub = top == -INFINITY ? 0.0f : top;
    x = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    l = 0.0f;
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
        const float f = exp2_hw(stat[slot][u].x - sub);
        l += f * stat[slot][u].y;
        const f32x4 y = sum[slot][u][i];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += f * y[e];
    }
    store4((Global<unsigned short>)a.o[rank] + b * a.o_stride + (long long)head * D + 4 * i, x, l == 0.0f ? 0.0f : 1.0f / l);
}

struct Kv4Cut {
    int nt, blocks, waves, shared_rbs, own_rbs, own_rows;
    size_t shared_parts, own_parts, items;                   // parts over all (rank, key head)
};
// Shared keys are taken against 32 rows at a time where there are more than 16:
// groups of 8 / 16 / 64 beams of 4 heads 24.1 / 28.9 / 33.9 us so, against 16
// 24.9 / 28.6 / 34.4, against 64, whose registers leave one wave a SIMD for the
// rows' own keys too, 24.0 / 41.3 / 46.1.
Kv4Cut kv4_cut(int P, int B, int group, bool shared, int Hq, int Hkv, int cus) {
    Kv4Cut c;
    const int G = Hq / Hkv;
    const long long units = (long long)P * Hkv, rows = (long long)group * G;
    c.nt = rows <= 16 ? 1 : 2;
    c.shared_rbs = (int)((rows + 16 * c.nt - 1) / (16 * c.nt));
    c.own_rbs = (G + 15) / 16;
    c.own_rows = G < 16 ? G : 16;
    // as many workgroups as run at once: by registers three a compute unit, two with two row tiles
    c.blocks = (int)(((c.nt == 2 && shared ? 2 : 3) * (long long)cus + units - 1) / units);
    c.waves = c.blocks * kWaves;
    const size_t ns = shared ? (size_t)(B / group) * c.shared_rbs : 0, no = (size_t)B * c.own_rbs;
    c.items = ns + no;
    c.shared_parts = shared ? (ns + c.waves) * (size_t)units : 0;
    c.own_parts = (no + c.waves) * (size_t)units;
    return c;
}
size_t kv4_ws(const Kv4Cut& c, int D) {
    const size_t n = c.shared_parts * 16 * c.nt + c.own_parts * c.own_rows;
    return kStatusBytes + (n * (D + 2) * 4 + 16 + c.items * 16 + 255) / 256 * 256;
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
    const size_t with = kv4_ws(kv4_cut(P, B, group, true, Hq, Hkv, dev_info().cus), D);
    const size_t without = kv4_ws(kv4_cut(P, B, group, false, Hq, Hkv, dev_info().cus), D);
    return with > without ? with : without;
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
    // rows that no workgroup shares need no scan, no parts and no second launch
    a.whole = !shared && (long long)table_stride * page_size <= kWholeTiles * kKeys;
    const size_t need = a.whole ? kStatusBytes : kv4_ws(c, D);
    if (!ws || ((uintptr_t)ws & 255) || ws_bytes < need) return RING_EWORKSPACE;
    // costs and rows of parts are counted in 32 bits
    if ((long long)(B / group * c.shared_rbs + B * c.own_rbs) * ((long long)table_stride * page_size / kKeys + 2) * 8 >= (1LL << 31) ||
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
    a.waves = c.waves;
    a.shared_cost = kOwnCost * (c.nt + 1) / 2;
    a.shared_rbs = c.shared_rbs;
    a.own_rbs = c.own_rbs;
    a.own_rows = c.own_rows;
    a.c = scale * kLog2e;
    a.shared_o = (float*)((char*)ws + kStatusBytes);
    a.own_o = a.shared_o + c.shared_parts * 16 * c.nt * D;
    a.shared_ml = (float2*)(a.own_o + c.own_parts * c.own_rows * D);
    a.own_ml = a.shared_ml + c.shared_parts * 16 * c.nt;
    a.parts = (ItemParts*)(((uintptr_t)(a.own_ml + c.own_parts * c.own_rows) + 15) & ~(uintptr_t)15);
    a.status = (Status*)ws;
    a.data = WsSpan{kStatusBytes, need};
    hipStream_t s = (hipStream_t)stream;
    const int units = P * Hkv;
    if (a.whole) a.blocks = B * c.own_rbs;
    // (workgroups of their own, the last to start: within others' time 0.7 us of theirs)
    a.planners = a.whole ? 0 : (int)((c.items + 255) / 256);
    if ((long long)units * a.blocks + a.planners >= (1LL << 31)) return RING_EUNSUPPORTED;
    const dim3 grid((unsigned)(units * a.blocks + a.planners));
    const size_t dyn = (2 * (size_t)B + (shared ? B / group : 0)) * sizeof(int);
    const long long rows = (long long)P * B * Hq;
    // 256 lanes a row, else 64: 8 rows of 60000 keys 17.3 us so, 31.4 with 64; 512 of
    // 5000 22.3 and 22.7; 2048 of 5000 52.3 with 256, 51.2 so; 768 behind shared keys
    // 32.6 and 29.7
    const bool few = rows <= 2LL * dev_info().cus;
    const dim3 jg((unsigned)(few ? B * Hq : B * ((Hq + 3) / 4)), (unsigned)P);
    auto go = [&](auto d, auto nt) -> int {
        constexpr int kD = decltype(d)::value, kNT = decltype(nt)::value;
        hipLaunchKernelGGL((kv4_decode_kernel<kD, kNT>), grid, dim3(256), dyn, s, a);
        if (hipGetLastError() != hipSuccess) return RING_EHIP;
        if (a.whole) return RING_OK;
        if (few) hipLaunchKernelGGL((kv4_join_kernel<kD, kNT, 256>), jg, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((kv4_join_kernel<kD, kNT, 64>), jg, dim3(256), 0, s, a);
        return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
    };
    auto with_nt = [&](auto d) -> int {
        if (!shared || c.nt == 1) return go(d, std::integral_constant<int, 1>());
        return go(d, std::integral_constant<int, 2>());
    };
    return D == 128 ? with_nt(std::integral_constant<int, 128>()) : with_nt(std::integral_constant<int, 64>());
}
