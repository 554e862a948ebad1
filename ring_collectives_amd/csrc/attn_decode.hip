// attn_decode.hip -- attention of one query token per request over a paged
// cache, with a prefix that every request shares.
//
// A request's keys are the prefix's and its own; over any split of them,
//   m = max of the parts' m,  l = sum l_i 2^(m_i - m),  o = sum o_i 2^(m_i - m) / l
// gives the whole from parts that hold (m_i, l_i, o_i = sum of weighted
// values).  One launch makes the parts, a second joins them:
//   - prefix workgroups: 128 rows (request, head of the group) of one (rank,
//     key head) against a range of the prefix, whose tiles all rows share, so
//     the prefix is read once per 128 rows instead of once per request;
//   - own-key workgroups: one request and (rank, key head), up to 32 heads of
//     the group, against a range of its own keys; each of the four waves takes
//     a part of the range through LDS of its own, key and value tiles of 32
//     rows in turn, and the four results join in LDS.
// The cache rows read bound it.  The ranges are cut for two workgroups a compute
// unit, whose loads overlap with each other's products, by the shapes alone, so
// that the grid of a captured call holds for any lengths:
//   - every request gets as many parts, whatever its length.  64 requests on 4
//     ranks of 8 heads of 128 on 2, 375 MB of keys and values: of 1430 keys each
//     70 us, one of 60000 among 63 of 500 733 us, since that one is read by one
//     workgroup a unit.  A table wider than the lengths makes empty parts: 4 of
//     700 keys under one of 704 and of 131072 tokens 11 us both.
//   - at most kMaxParts workgroups go to a request of one (rank, key head), so
//     one request on less than 4 of them has less than one a compute unit (60000
//     keys of one key head 20 us, 1.6 TB/s).
// Within a wave little overlaps: before a tile's first row fragments the
// compiler waits for every load in flight, which are the prefix's next tile and
// the own keys' values of the same one.  What stays in flight is the next tile's
// keys of a request, while this tile's weights and second product are made.
//
// 4 ranks of 8 heads of 128 on 2: 4 requests of up to 60000 keys 153 us, 5.35
// TB/s; 64 requests of up to 700 behind 8192 shared ones 53 us, 3.1 TB/s, the
// join 6 of them.
#include "attn_core.h"
#include "attn_internal.h"

#include <hip/hip_runtime.h>

namespace ringc {
namespace {

constexpr int kWaves = 4;
constexpr int kPreRows = 128, kPreKeys = 64;   // prefix: rows of a workgroup, keys of a tile
constexpr int kOwnKeys = 32;                   // own keys: keys of a wave's tile
constexpr int kIds = 512;                      // cache rows looked up at a time by a wave
constexpr int kMaxParts = 64;                  // of each kind

struct DecodeArgs {
    const unsigned short *q[RING_MAX_RANKS], *kc[RING_MAX_RANKS], *vc[RING_MAX_RANKS];
    unsigned short* o[RING_MAX_RANKS];
    const int *table, *lengths, *prefix_pages;
    long long q_stride, o_stride, kv_stride;
    int P, B, Hq, Hkv, width, shift, pages, prefix;
    int pre_parts, own_parts, pre_blocks, row_tiles;   // row_tiles: tiles of 32 heads of the group
    float c;
    float* part_o;             // [P Hkv][parts][B G][D]
    float* part_ml;            // [P Hkv][parts][B G][2]
    Status* status;
    WsSpan data;
};

// The running state of a wave's 32 columns.
template <int D> struct Soft {
    f32x16 o[Rows<D>::DB];
    float mc, l;               // maximum times c, this half's share of the sum
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int db = 0; db < Rows<D>::DB; ++db)
#pragma unroll
            for (int v = 0; v < 16; ++v) o[db][v] = 0.0f;
        mc = -INFINITY;
        l = 0.0f;
    }
    // NB blocks of 32 scores (masked ones -inf) become weights.
    template <int NB> __device__ __forceinline__ void weigh(f32x16 (&s)[NB], float c) {
        float mx = s[0][0];
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
#pragma unroll
            for (int v = 0; v < 16; ++v) mx = fmaxf(mx, s[kb][v]);
        mx = max_halves(mx) * c;
        if (__any(mx > mc + 8.0f)) {
            const float mn = fmaxf(mc, mx);
            const float alpha = mn == -INFINITY ? 1.0f : exp2_hw(mc - mn);
            mc = mn;
            l *= alpha;
#pragma unroll
            for (int db = 0; db < Rows<D>::DB; ++db)
#pragma unroll
                for (int v = 0; v < 16; ++v) o[db][v] *= alpha;
        }
        const float sub = mc == -INFINITY ? 0.0f : mc;
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                s[kb][v] = exp2_hw(__builtin_fmaf(s[kb][v], c, -sub));
                l += s[kb][v];
            }
    }
};

// One instruction's rows of a gathered tile: the lane's row r is cache row id.
// Rows without a key (id < 0) load cache row 0, and blank() makes zeros of
// what landed.  Both by selects: with a branch per lane around a load, the
// compiler is free to run the lanes on either side of it apart from each other
// through the loop that follows, whose steps are the whole wave's.
template <int D>
__device__ __forceinline__ void gather(const unsigned short* base, long long stride, int id, int r, int lane,
                                       unsigned short* lds, int at) {
    const unsigned short* p = base + (id < 0 ? 0 : id) * stride + ((lane % Rows<D>::C) ^ Rows<D>::swz(r)) * 8;
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p, lds_at(lds, (unsigned)at), 16, 0, 0);
}
__device__ __forceinline__ void blank(unsigned short* lds, int at, int id, int lane) {
    u32x4* p = (u32x4*)((char*)lds + at + lane * 16);
    u32x4 x = *p;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = id < 0 ? 0u : x[e];
    *p = x;
}

__device__ __forceinline__ void lds_settled() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <int D>
__global__ __launch_bounds__(256, 2) void attn_decode_kernel(DecodeArgs a) {
    typedef Rows<D> R;
    constexpr int kPreBytes = kPreKeys * R::RB, kOwnBytes = kOwnKeys * R::RB;
    static_assert(4 * kPreBytes == 2 * kWaves * kOwnBytes, "one LDS size for both kinds");
    __shared__ __align__(4096) unsigned short lds[4 * kPreBytes / 2];
    __shared__ int ids[kWaves][kIds];
    __shared__ float wave_ml[kWaves][32][2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, col = lane & 31;
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.part_o) ws_add_data(a.status, a.data);
    const int units = a.P * a.Hkv, G = a.Hq / a.Hkv;
    const int parts = a.pre_parts + a.own_parts;
    const bool pre = (int)blockIdx.x < a.pre_blocks;
    const int blk = pre ? blockIdx.x : blockIdx.x - a.pre_blocks;
    const int unit = blk % units, rest = blk / units, rank = unit / a.Hkv, kvh = unit % a.Hkv;
    const unsigned short* kbase = a.kc[rank] + (long long)kvh * D;
    const unsigned short* vbase = a.vc[rank] + (long long)kvh * D;
    const long long all = (long long)a.B * G;
    Frags<D> fr;
    fr.init(lane);
    Soft<D> st;
    st.init();
    bf16x8 qf[R::KK];
    long long m;               // this lane's row (request, head of the group)
    bool live;
    int part;
    auto load_q = [&](long long row) {
        const int b = (int)((unsigned)row / (unsigned)G), head = kvh * G + (int)((unsigned)row % (unsigned)G);
        const unsigned short* qp = a.q[rank] + b * a.q_stride + (long long)head * D + 8 * half;
#pragma unroll
        for (int kk = 0; kk < R::KK; ++kk) qf[kk] = *(const bf16x8*)(qp + 16 * kk);
    };
    // the cache row of key `key` of n (n > 0), -1 past them or if its page is not one
    auto page_row = [&](const int* pages, long long key, int n) {
        const int k = key < n ? (int)key : n - 1, p = pages[k >> a.shift];
        const int row = (int)(((long long)p << a.shift) + (k & ((1 << a.shift) - 1)));
        return key < n && p >= 0 && p < a.pages ? row : -1;
    };

    if (pre) {
        part = rest % a.pre_parts;
        const int tile = rest / a.pre_parts;
        const long long m0 = (long long)tile * kPreRows + wave * 32 + col;
        live = m0 < all;
        m = live ? m0 : all - 1;
        load_q(m);
        const int n = a.pages ? (a.prefix + kPreKeys - 1) / kPreKeys : 0;
        const int j0 = (int)((long long)n * part / a.pre_parts), j1 = (int)((long long)n * (part + 1) / a.pre_parts);
        constexpr int J = kPreKeys / R::RPI / kWaves;
        // the rows this lane loads of the tile being loaded, and which keys
        // that tile has; the same of the next one, looked up a tile ahead
        int id[J], id_next[J];
        unsigned long long seen = 0, seen_next = 0;
        auto look_up = [&](int j) {
            const long long k0 = (long long)j * kPreKeys;
#pragma unroll
            for (int i = 0; i < J; ++i)
                id_next[i] = page_row(a.prefix_pages, k0 + (wave * J + i) * R::RPI + lane / R::C, a.prefix);
            seen_next = __ballot(page_row(a.prefix_pages, k0 + lane, a.prefix) >= 0);
        };
        // restrict for the effect told at the prompts' pass: no wait for the
        // loads in flight before a tile's transposed reads (the compiler puts
        // one before its row reads all the same)
        auto pass = [&](const unsigned short* __restrict__ kc, const unsigned short* __restrict__ vc) __attribute__((always_inline)) {
            auto load = [&](int buf) {
#pragma unroll
                for (int i = 0; i < J; ++i) {
                    const int at = buf * kPreBytes + (wave * J + i) * 1024, r = (wave * J + i) * R::RPI + lane / R::C;
                    id[i] = id_next[i];
                    gather<D>(kc, a.kv_stride, id[i], r, lane, lds, at);
                    gather<D>(vc, a.kv_stride, id[i], r, lane, lds, at + 2 * kPreBytes);
                }
            };
            if (j0 < j1) {
                look_up(j0);
                load(0);
                seen = seen_next;
            }
            for (int j = j0; j < j1; ++j) {
                const int buf = (j - j0) & 1;
                const unsigned long long has = seen;
                if (j + 1 < j1) look_up(j + 1);
                wait_vm(0);
                if (~has) {
#pragma unroll
                    for (int i = 0; i < J; ++i) {
                        blank(lds, buf * kPreBytes + (wave * J + i) * 1024, id[i], lane);
                        blank(lds, (2 + buf) * kPreBytes + (wave * J + i) * 1024, id[i], lane);
                    }
                }
                lds_barrier();
                if (j + 1 < j1) {
                    load(buf ^ 1);
                    seen = seen_next;
                }
                f32x16 s[2];
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
                    for (int v = 0; v < 16; ++v) s[kb][v] = 0.0f;
#pragma unroll
                    for (int kk = 0; kk < R::KK; ++kk)
                        s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.rows(lds, buf * kPreBytes, kb, kk), qf[kk], s[kb], 0, 0, 0);
                }
                if (~has) {
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            if (!((has >> (kb * 32 + acc_row(v, half))) & 1)) s[kb][v] = -INFINITY;
                }
                st.weigh(s, a.c);
#pragma unroll
                for (int ks = 0; ks < kPreKeys / 16; ++ks) {
                    const bf16x8 pf = round8(s[ks / 2], ks % 2);
#pragma unroll
                    for (int db = 0; db < R::DB; ++db)
                        st.o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.cols(lds, (2 + buf) * kPreBytes, db, ks), pf, st.o[db], 0, 0, 0);
                }
            }
        };
        pass(kbase, vbase);
        st.l = sum_halves(st.l);
    } else {
        part = a.pre_parts + rest % a.own_parts;
        const int rt = rest / a.own_parts % a.row_tiles, b = rest / a.own_parts / a.row_tiles;
        live = rt * 32 + col < G;
        m = (long long)b * G + (live ? rt * 32 + col : G - 1);
        load_q(m);
        const long long room = (long long)a.width << a.shift;
        const int len0 = a.lengths[b], len = len0 < 0 ? 0 : len0 < room ? len0 : (int)room;
        const int* pages = a.table + (long long)b * a.width;
        const int n = a.pages ? (len + kOwnKeys - 1) / kOwnKeys : 0, cuts = a.own_parts * kWaves;
        const int cut = (part - a.pre_parts) * kWaves + wave;
        const int j0 = __builtin_amdgcn_readfirstlane((int)((long long)n * cut / cuts));
        const int j1 = __builtin_amdgcn_readfirstlane((int)((long long)n * (cut + 1) / cuts));
        const int ka = wave * 2 * kOwnBytes, va = ka + kOwnBytes;
        constexpr int J = kOwnKeys / R::RPI, kTiles = kIds / kOwnKeys;
        auto look_up = [&](int j) {                       // the cache rows of tiles j .. j + kTiles - 1
#pragma unroll
            for (int i = 0; i < kIds / 64; ++i)
                ids[wave][i * 64 + lane] = page_row(pages, (long long)j * kOwnKeys + i * 64 + lane, len);
            lds_settled();
        };
        // the rows this lane loads of tile j, and which keys there are
        auto rows_of = [&](int j, int (&id)[J]) {
            const int* tid = ids[wave] + (j - j0) % kTiles * kOwnKeys;
#pragma unroll
            for (int i = 0; i < J; ++i) id[i] = tid[i * R::RPI + lane / R::C];
            return __builtin_amdgcn_readfirstlane((unsigned)__ballot(tid[col] >= 0));
        };
        // restrict as above: no wait for the next keys before a tile's
        // transposed reads
        auto pass = [&](const unsigned short* __restrict__ kc, const unsigned short* __restrict__ vc) __attribute__((always_inline)) {
            auto load = [&](const unsigned short* base, const int (&id)[J], int at) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < J; ++i) gather<D>(base, a.kv_stride, id[i], i * R::RPI + lane / R::C, lane, lds, at + i * 1024);
            };
            auto blank_rows = [&](const int (&id)[J], int at) {
#pragma unroll
                for (int i = 0; i < J; ++i) blank(lds, at + i * 1024, id[i], lane);
                lds_settled();
            };
            int id[J];
            for (int c0 = j0; c0 < j1; c0 += kTiles) {
                const int c1 = c0 + kTiles < j1 ? c0 + kTiles : j1;
                look_up(c0);
                unsigned seen = rows_of(c0, id);
                load(kc, id, ka);
                load(vc, id, va);
                for (int j = c0; j < c1; ++j) {
                    const unsigned has = seen;
                    int was[J];
#pragma unroll
                    for (int i = 0; i < J; ++i) was[i] = id[i];
                    wait_vm(J);                           // the keys of tile j have landed (and, by the compiler's wait, its values)
                    if (~has) blank_rows(was, ka);
                    f32x16 s[1];
#pragma unroll
                    for (int v = 0; v < 16; ++v) s[0][v] = 0.0f;
#pragma unroll
                    for (int kk = 0; kk < R::KK; ++kk)
                        s[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.rows(lds, ka, 0, kk), qf[kk], s[0], 0, 0, 0);
                    lds_settled();
                    if (j + 1 < c1) {
                        seen = rows_of(j + 1, id);
                        load(kc, id, ka);
                    }
                    if (~has) {
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            if (!((has >> acc_row(v, half)) & 1)) s[0][v] = -INFINITY;
                    }
                    st.weigh(s, a.c);
                    wait_vm(j + 1 < c1 ? J : 0);          // its values have; the next keys may be in flight
                    if (~has) blank_rows(was, va);
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
                        const bf16x8 pf = round8(s[0], ks);
#pragma unroll
                        for (int db = 0; db < R::DB; ++db)
                            st.o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.cols(lds, va, db, ks), pf, st.o[db], 0, 0, 0);
                    }
                    lds_settled();
                    if (j + 1 < c1) load(vc, id, va);
                }
            }
        };
        pass(kbase, vbase);
        // the four waves' results, as [d][column] floats in each wave's own tiles
        st.l = sum_halves(st.l);
        if (half == 0) {
            wave_ml[wave][col][0] = st.mc;
            wave_ml[wave][col][1] = st.l;
        }
        float* mine = (float*)((char*)lds + ka);
        static_assert(D * 32 * 4 <= 2 * kOwnBytes, "a wave's output fits its tiles");
#pragma unroll
        for (int db = 0; db < R::DB; ++db)
#pragma unroll
            for (int v = 0; v < 16; ++v) mine[(32 * db + acc_row(v, half)) * 32 + col] = st.o[db][v];
        __syncthreads();
        if (wave >= R::DB) return;
        float mx = -INFINITY, l = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) mx = fmaxf(mx, wave_ml[w][col][0]);
        float f[kWaves];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            f[w] = mx == -INFINITY ? 0.0f : exp2_hw(wave_ml[w][col][0] - mx);
            l += f[w] * wave_ml[w][col][1];
        }
        st.mc = mx;
        st.l = l;
        // wave db joins block db of the values, in st.o[0]
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            float x = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                x += f[w] * ((const float*)((const char*)lds + w * 2 * kOwnBytes))[(32 * wave + acc_row(v, half)) * 32 + col];
            st.o[0][v] = x;
        }
    }

    // a prefix wave holds all blocks of its rows, an own-key wave block `wave`
    const int db0 = pre ? 0 : wave;
    if (!a.part_o) {                                      // one part in all: the result itself
        const int b = (int)((unsigned)m / (unsigned)G), head = kvh * G + (int)((unsigned)m % (unsigned)G);
        unsigned short* op = a.o[rank] + b * a.o_stride + (long long)head * D + 32 * db0;
        const float inv = st.l == 0.0f ? 0.0f : 1.0f / st.l;
#pragma unroll
        for (int i = 0; i < R::DB; ++i)
            if (pre || i == 0) store_block(op + 32 * i, st.o[i], inv, half, live);
        return;
    }
    if (!live) return;
    const long long at = ((long long)unit * parts + part) * all + m;
    float* po = a.part_o + at * D + 32 * db0 + 4 * half;
#pragma unroll
    for (int i = 0; i < R::DB; ++i)
        if (pre || i == 0)
#pragma unroll
            for (int v = 0; v < 16; v += 4)
                *(f32x4*)(po + 32 * i + 2 * v) = f32x4{st.o[i][v], st.o[i][v + 1], st.o[i][v + 2], st.o[i][v + 3]};
    if (half == 0 && db0 == 0) {
        a.part_ml[2 * at] = st.mc;
        a.part_ml[2 * at + 1] = st.l;
    }
}

// The parts of every row, joined.  A workgroup holds a row: its parts' weights
// go to LDS, then D / 4 lanes each with 16-byte loads sum every 1024 / D-th
// part, so a row's loads are in flight together, and those sums join in LDS.
// (One row per D / 4 lanes, the parts one after the other, took 26 us for the
// 33 parts of 2048 rows of 128; this takes a quarter.)
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(DecodeArgs a) {
    constexpr int L = D / 4, kGroups = 256 / L;
    __shared__ float ml[2 * kMaxParts][2];
    __shared__ f32x4 sum[kGroups][L];
    const int parts = a.pre_parts + a.own_parts, G = a.Hq / a.Hkv;
    const long long all = (long long)a.B * G;
    const int unit = (int)(blockIdx.x / (unsigned)all);
    const long long m = blockIdx.x % (unsigned)all, first = (long long)unit * parts * all + m;
    const int t = threadIdx.x, i = t % L, g = t / L;
    if (t < 2 * parts) ml[t / 2][t % 2] = a.part_ml[2 * (first + t / 2 * all) + t % 2];
    __syncthreads();
    float mx = -INFINITY, l = 0.0f;
    for (int p = 0; p < parts; ++p) mx = fmaxf(mx, ml[p][0]);
    const float sub = mx == -INFINITY ? 0.0f : mx;         // no part has a key: every weight is 0
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int p = g; p < parts; p += kGroups) {
        const float w = exp2_hw(ml[p][0] - sub);
        const f32x4 y = *(const f32x4*)(a.part_o + (first + p * all) * D + 4 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += w * y[e];
    }
    sum[g][i] = x;
    __syncthreads();
    if (g) return;
    for (int p = 0; p < parts; ++p) l += exp2_hw(ml[p][0] - sub) * ml[p][1];
#pragma unroll
    for (int u = 1; u < kGroups; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += sum[u][i][e];
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= inv;
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    const int rank = unit / a.Hkv, head = unit % a.Hkv * G + (int)((unsigned)m % (unsigned)G);
    *(bf16x4*)(a.o[rank] + (unsigned)m / (unsigned)G * a.o_stride + (long long)head * D + 4 * i) = __builtin_convertvector(x, bf16x4);
}
static_assert(4 * kMaxParts <= 256, "a row's statistics are one load of the workgroup");

struct Cuts {
    int pre, own, row_tiles;
    long long pre_tiles;
};

// Parts of the prefix and of the own keys, the same for every request.  Two
// workgroups run on a compute unit.  The prefix is cut until it alone would give each one workgroup, as far
// as every part keeps four tiles; the own keys until they would fill the other
// one (both, without a prefix), as far as every wave keeps a tile.  Own keys
// that a workgroup's waves see in less than four tiles each stay whole: parts
// cost a second launch.  Measured on 4 ranks of 8 heads of 128 on 2: 64
// requests of up to 700 behind 8192, prefix in 8 / 16 / 32 parts 56 / 53 / 62
// us; 4 requests of up to 60000 in 8 / 16 / 32 parts 169 / 156 / 156 us; one
// request of 200 whole 9, cut 12 us.
Cuts decode_cuts(int P, int B, int Hq, int Hkv, int width, int page, int prefix, int cus) {
    Cuts c;
    const long long units = (long long)P * Hkv, G = Hq / Hkv;
    c.row_tiles = (int)((G + 31) / 32);
    c.pre_tiles = (B * G + kPreRows - 1) / kPreRows;
    auto cut = [&](long long per_cu, long long blocks, long long most) {
        long long n = (per_cu * cus + blocks - 1) / blocks;
        if (n > most) n = most;
        if (n > kMaxParts) n = kMaxParts;
        return (int)(n < 1 ? 1 : n);
    };
    const long long own_tiles = ((long long)width * page + kOwnKeys - 1) / kOwnKeys;
    c.pre = prefix ? cut(1, units * c.pre_tiles, (prefix + kPreKeys - 1) / kPreKeys / 4) : 0;
    c.own = cut(prefix ? 1 : 2, units * B * c.row_tiles, own_tiles < 4 * kWaves ? 1 : own_tiles / kWaves);
    return c;
}

size_t decode_ws(int P, int B, int Hq, int Hkv, int D, const Cuts& c) {
    const size_t parts = (size_t)c.pre + c.own;
    if (parts < 2) return kStatusBytes;
    return kStatusBytes + (parts * P * B * Hq * (D + 2) * sizeof(float) + 255) / 256 * 256;
}

// The most that a batch of B requests or fewer needs, so that a workspace kept
// from call to call holds a batch that shrinks: fewer requests are cut into
// more parts.  Own keys are in one part from 2 cus requests on, and batches of
// the same number of 128-row tiles have their prefix in the same parts, so the
// largest of each number and the small batches are all there is to look at.
size_t decode_ws_upto(int P, int B, int Hq, int Hkv, int D, int width, int page, int prefix, int cus) {
    size_t most = kStatusBytes;
    auto look = [&](long long b) {
        const int n = (int)(b < 1 ? 1 : b < B ? b : B);
        const size_t w = decode_ws(P, n, Hq, Hkv, D, decode_cuts(P, n, Hq, Hkv, width, page, prefix, cus));
        if (w > most) most = w;
    };
    if (!B) return most;
    for (int b = 1; b < B && b <= 2 * cus; ++b) look(b);
    for (int t = 1; prefix && t <= cus && (long long)kPreRows * t / (Hq / Hkv) < B; ++t) look((long long)kPreRows * t / (Hq / Hkv));
    look(B);
    return most;
}

bool decode_shape(int P, int B, int Hq, int Hkv, int D, int width, int page, int prefix) {
    return P >= 1 && P <= RING_MAX_RANKS && B >= 0 && Hq >= 1 && Hkv >= 1 && width >= 0 && prefix >= 0 && page >= 1 &&
           !(page & (page - 1)) && page <= (1 << 20) && Hq % Hkv == 0 && (D == 64 || D == 128) &&
           (long long)Hq * D < kMaxRow && (long long)width * page < (1LL << 31) && B <= (1 << 20) &&
           (long long)B * Hq < (1LL << 31);
}

}  // namespace
}  // namespace ringc

using namespace ringc;

extern "C" size_t tp_attention_decode_workspace_bytes(int P, int B, int Hq, int Hkv, int D, int table_stride,
                                                      int page_size, int prefix_len) {
    if (!decode_shape(P, B, Hq, Hkv, D, table_stride, page_size, prefix_len)) return 0;
    return decode_ws_upto(P, B, Hq, Hkv, D, table_stride, page_size, prefix_len, dev_info().cus);
}

extern "C" int tp_attention_decode(const void* const* q, const void* const* k_cache, const void* const* v_cache,
                                   void* const* o, const int* block_table, const int* lengths, const int* prefix_pages,
                                   int P, int B, int Hq, int Hkv, int D, int table_stride, int page_size, int pages,
                                   int prefix_len, long long q_stride, long long o_stride, float scale, void* ws,
                                   size_t ws_bytes, void* stream) {
    if (P < 1 || P > RING_MAX_RANKS || B < 0 || Hq < 1 || Hkv < 1 || table_stride < 0 || pages < 0 || prefix_len < 0)
        return RING_EINVAL;
    if (page_size < 1 || (page_size & (page_size - 1)) || page_size > (1 << 20)) return RING_EINVAL;
    if (!scale_ok(scale)) return RING_EINVAL;
    if (!decode_shape(P, B, Hq, Hkv, D, table_stride, page_size, prefix_len) || (long long)pages * page_size >= (1LL << 31))
        return RING_EUNSUPPORTED;
    if (!row_stride_ok(q_stride, Hq, D) || !row_stride_ok(o_stride, Hq, D)) return RING_EINVAL;
    if (B == 0) return RING_OK;
    if (!q || !k_cache || !v_cache || !o || !lengths || ((uintptr_t)lengths & 3) || (table_stride && !block_table) ||
        ((uintptr_t)block_table & 3) || (prefix_len && !prefix_pages) || ((uintptr_t)prefix_pages & 3))
        return RING_EINVAL;
    DecodeArgs a;
    for (int r = 0; r < P; ++r) {
        if (!q[r] || !o[r] || (pages && (!k_cache[r] || !v_cache[r]))) return RING_EINVAL;
        if (((uintptr_t)q[r] | (uintptr_t)o[r] | (uintptr_t)k_cache[r] | (uintptr_t)v_cache[r]) & 15) return RING_EINVAL;
        a.q[r] = (const unsigned short*)q[r];
        a.kc[r] = (const unsigned short*)k_cache[r];
        a.vc[r] = (const unsigned short*)v_cache[r];
        a.o[r] = (unsigned short*)o[r];
    }
    const Cuts c = decode_cuts(P, B, Hq, Hkv, table_stride, page_size, prefix_len, dev_info().cus);
    const size_t need = decode_ws(P, B, Hq, Hkv, D, c);
    if (!ws || ((uintptr_t)ws & 255) || ws_bytes < need) return RING_EWORKSPACE;
    const int units = P * Hkv;
    const long long pre = c.pre_tiles * c.pre * units, own = (long long)B * c.row_tiles * c.own * units;
    if (pre + own >= (1LL << 31) || (long long)P * B * Hq >= (1LL << 31)) return RING_EUNSUPPORTED;
    a.table = block_table;
    a.lengths = lengths;
    a.prefix_pages = prefix_pages;
    a.q_stride = q_stride;
    a.o_stride = o_stride;
    a.kv_stride = (long long)Hkv * D;
    a.P = P;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.width = table_stride;
    a.shift = 0;
    while ((1 << a.shift) < page_size) ++a.shift;
    a.pages = pages;
    a.prefix = prefix_len;
    a.pre_parts = c.pre;
    a.own_parts = c.own;
    a.pre_blocks = (int)pre;
    a.row_tiles = c.row_tiles;
    a.c = scale * kLog2e;
    const bool join = c.pre + c.own > 1;
    a.part_o = join ? (float*)((char*)ws + kStatusBytes) : nullptr;
    a.part_ml = join ? a.part_o + (size_t)(c.pre + c.own) * P * B * Hq * D : nullptr;
    a.status = (Status*)ws;
    a.data = WsSpan{kStatusBytes, need};
    hipStream_t s = (hipStream_t)stream;
    const dim3 grid((unsigned)(pre + own));
    if (D == 128) hipLaunchKernelGGL(attn_decode_kernel<128>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(attn_decode_kernel<64>, grid, dim3(256), 0, s, a);
    if (hipGetLastError() != hipSuccess) return RING_EHIP;
    if (join) {
        const dim3 jg((unsigned)((long long)P * B * Hq));
        if (D == 128) hipLaunchKernelGGL(attn_join_kernel<128>, jg, dim3(256), 0, s, a);
        else hipLaunchKernelGGL(attn_join_kernel<64>, jg, dim3(256), 0, s, a);
        if (hipGetLastError() != hipSuccess) return RING_EHIP;
    }
    return RING_OK;
}
