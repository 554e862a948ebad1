// attn_grad.hip -- gradient of the packed-prompt attention.
//
//   P = exp(S - lse),  delta = sum(dO O),  dP = dO V^T,  dS = P (dP - delta),
//   dQ = scale dS K,   dK = scale dS^T Q,  dV = P^T dO.
//
// Two passes, each summing its results in registers in a fixed order: one per
// 128 query rows over the keys (dQ; it also leaves lse and delta of its rows
// in the workspace; in shares of the keys as the forward pass), one per 128
// keys over the queries of every head of the group (dK, dV).  S and dP are
// computed in both, seven products in all where five would do, but no result
// is added up through memory: no atomics, whose order would change the
// results, and no fp32 copy of dQ.
//
// delta is summed in fp32 from O as it was rounded to bf16, which costs dQ and
// dK 2.9e-3 of relative error in prompts of two tokens, 1.9e-3 in ones of 8,
// 1.2e-3 in ones of 60 and 0.6 to 1e-3 in ones of hundreds, beside the 1.6e-3 each
// of their own rounding and of dS's.  From sum(P dP) it would be known only after the pass that uses it.
//
// 8192 tokens on 4 ranks of 8 heads of 128 on 2: dQ 724 us, its matrix cores 62%
// busy at 1.8 GHz, the card's power limit; dK and dV 1230 us, 40% at 2.15 GHz,
// one wave per SIMD (128 registers of sums and 64 of K and V in each), whose
// products wait for its own weights.
#include "attn_core.h"
#include "attn_internal.h"

#include <hip/hip_runtime.h>

namespace ringc {
namespace {

constexpr int kRowsWG = 128;   // query rows, or keys, of a workgroup
constexpr int kStep = 64;      // keys, or queries, of a tile
constexpr int kWaves = 4;
constexpr int kAhead = 4;       // row fragments asked for ahead of their MFMA

struct GradArgs {
    PromptArgs p;
    const unsigned short *o[RING_MAX_RANKS], *go[RING_MAX_RANKS];
    const float* lse[RING_MAX_RANKS];
    unsigned short *dq[RING_MAX_RANKS], *dk[RING_MAX_RANKS], *dv[RING_MAX_RANKS];
    long long o_stride, go_stride, dq_stride, dk_stride, dv_stride;
    float* lse2;               // [P][Hq][Tq] lse log2(e), +inf for a row that sees no key
    float* delta;              // [P][Hq][Tq]
    Status* status;
    WsSpan data;
    float scale;
    int slots;
};

template <int D, int kShares>
__global__ __launch_bounds__(256 * kShares, 2) void attn_dq_kernel(GradArgs a) {
    typedef Rows<D> R;
    constexpr int kTileBytes = kStep * R::RB;
    __shared__ __align__(4096) unsigned short lds[kShares * 4 * kTileBytes / 2];   // of each share: K 0, K 1, V 0, V 1
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % kWaves;
    const int share = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / kWaves;
    const int half = lane >> 5;
    if (blockIdx.x == 0 && threadIdx.x == 0) ws_add_data(a.status, a.data);
    int unit, slot;
    const PromptSizes sz = read_sizes(a.p, a.slots);
    unit_slot(sz.P * sz.Hkv, sz.slots, blockIdx.x, unit, slot);
    const int G = sz.Hq / sz.Hkv, rank = unit / sz.Hkv, kvh = unit % sz.Hkv;
    auto gq = (Global<const unsigned short>)a.p.q[rank], gk = (Global<const unsigned short>)a.p.k[rank];
    auto gv = (Global<const unsigned short>)a.p.v[rank], gout = (Global<const unsigned short>)a.o[rank];
    auto ggo = (Global<const unsigned short>)a.go[rank];
    auto glse = (Global<const float>)a.lse[rank];
    auto gdq = (Global<unsigned short>)a.dq[rank];
    auto glse2 = (Global<float>)a.lse2, gdelta = (Global<float>)a.delta;
    asm volatile("" : "+s"(gq), "+s"(gk), "+s"(gv), "+s"(gout), "+s"(ggo), "+s"(glse), "+s"(gdq), "+s"(glse2), "+s"(gdelta));
    PromptTile pt;
    if (!find_tile(sz.cu_q, sz.cu_k, sz.B, sz.Tq, sz.Tk, G, kRowsWG, slot, lane, pt)) return;
    const int tile = pt.tiles - 1 - pt.tile;                 // the longest first
    const int q0 = pt.lo, nq = pt.n, k0 = pt.lo2, nk = pt.n2;
    // this lane's row; rows past the end repeat the last one and are not stored
    const unsigned rows = (unsigned)nq * (unsigned)G, m0 = (unsigned)(tile * kRowsWG + wave * 32);
    const bool live = m0 + (lane & 31) < rows;
    const unsigned m = live ? m0 + (lane & 31) : rows - 1;
    const int qi = (int)(m / (unsigned)G), head = kvh * G + (int)(m % (unsigned)G);

    // keys [0, seen) are visible to this lane's query, [0, every) to every row
    // of the wave, [0, some) to one of them at least, [0, most) to one of the
    // workgroup's
    const int off = nk - nq;
    int seen = nk, every = nk, some = nk, most = nk;
    if (sz.causal) {
        auto upto = [&](unsigned row) {
            const int s = (int)((row < rows ? row : rows - 1) / (unsigned)G) + off + 1;
            return s < 0 ? 0 : s < nk ? s : nk;
        };
        seen = upto(m);
        every = upto(m0);
        some = upto(m0 + 31);
        most = upto((unsigned)(tile * kRowsWG + kRowsWG - 1));
    }

    bf16x8 qf[R::KK], gf[R::KK];
    float delta = 0.0f;
    {
        const long long t = q0 + (long long)qi;
        const unsigned short* qp = (const unsigned short*)gq + t * sz.q_stride + (long long)head * D + 8 * half;
        const unsigned short* op = (const unsigned short*)gout + t * a.o_stride + (long long)head * D + 8 * half;
        const unsigned short* gp = (const unsigned short*)ggo + t * a.go_stride + (long long)head * D + 8 * half;
#pragma unroll
        for (int kk = 0; kk < R::KK; ++kk) {
            qf[kk] = *(const bf16x8*)(qp + 16 * kk);
            gf[kk] = *(const bf16x8*)(gp + 16 * kk);
            const bf16x8 of = *(const bf16x8*)(op + 16 * kk);
#pragma unroll
            for (int e = 0; e < 8; ++e) delta = __builtin_fmaf((float)gf[kk][e], (float)of[e], delta);
        }
        delta = sum_halves(delta);
    }
    const long long at = ((long long)rank * sz.Hq + head) * sz.Tq + q0 + qi;
    float lse2 = glse[(long long)head * sz.Tq + q0 + qi] * kLog2e;
    if (lse2 == -INFINITY) lse2 = INFINITY;              // no key seen: every weight is 0
    if (half == 0 && live && share == 0) {
        glse2[at] = lse2;
        gdelta[at] = delta;
    }

    const unsigned krow = (unsigned)(sz.k_stride * 2), vrow = (unsigned)(sz.v_stride * 2);
    const unsigned short* kbase = (const unsigned short*)gk + (long long)k0 * sz.k_stride + (long long)kvh * D;
    const unsigned short* vbase = (const unsigned short*)gv + (long long)k0 * sz.v_stride + (long long)kvh * D;
    TileLoad<D, kStep, kWaves> kl, vl;
    kl.init(lane, wave, krow);
    vl.init(lane, wave, vrow);
    Frags<D> fr;
    fr.init(lane);
    f32x16 dq[R::DB];
#pragma unroll
    for (int db = 0; db < R::DB; ++db)
#pragma unroll
        for (int v = 0; v < 16; ++v) dq[db][v] = 0.0f;
    const float c = sz.c;
    // restrict for the effect told at the forward pass: no wait for the next
    // tile's loads before a tile's transposed reads
    auto pass = [&](const unsigned short* __restrict__ kp, const unsigned short* __restrict__ vp) __attribute__((always_inline)) {
        auto load = [&](int j, int buf) {
            const int at = (share * 4 + buf) * kTileBytes;
            kl.issue(kp + (long long)j * kStep * sz.k_stride, nk - (long long)j * kStep, krow, lds, at);
            vl.issue(vp + (long long)j * kStep * sz.v_stride, nk - (long long)j * kStep, vrow, lds, at + 2 * kTileBytes);
        };
        const int tiles = (most + kStep - 1) / kStep;
        if (share < tiles) load(share, 0);
        for (int i = 0; i * kShares < tiles; ++i) {
            const int j = i * kShares + share, buf = i & 1;
            wait_vm(0);
            lds_barrier();
            if (j + kShares < tiles) load(j + kShares, buf ^ 1);
            if (j * kStep >= some) continue;
            const int ka = (share * 4 + buf) * kTileBytes, va = ka + 2 * kTileBytes;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                f32x16 s, dp;
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int v = 0; v < 16; ++v) s[v] = dp[v] = 0.0f;
#pragma unroll
                for (int kk = 0; kk < R::KK; ++kk) {
                    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.rows(lds, ka, kb, kk), qf[kk], s, 0, 0, 0);
                    dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.rows(lds, va, kb, kk), gf[kk], dp, 0, 0, 0);
                }
                __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
                for (int i = 0; i < 2 * R::KK - kAhead; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                }
                __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const float p = exp2_hw(__builtin_fmaf(s[v], c, -lse2));
                    s[v] = p * (dp[v] - delta);
                }
                if ((j + 1) * kStep > every) {
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        if (j * kStep + kb * 32 + acc_row(v, half) >= seen) s[v] = 0.0f;
                }
                // dS is rounded to bf16 for the matrix cores, as P is going forward
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const bf16x8 sf = round8(s, ks);
#pragma unroll
                    for (int db = 0; db < R::DB; ++db)
                        dq[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.cols(lds, ka, db, 2 * kb + ks), sf, dq[db], 0, 0, 0);
                }
            }
        }
    };
    pass(kbase, vbase);
    // the shares' sums, added in their order
    if constexpr (kShares > 1) {
        constexpr int kRegs = 16 * R::DB;
        static_assert(kRegs * 4 * 64 * kWaves <= (int)sizeof(lds), "one share's sums");
        float* x = (float*)lds + wave * kRegs * 64 + lane;
#pragma unroll
        for (int u = 1; u < kShares; ++u) {
            lds_barrier();                    // the tiles, or the share before, have been read
            if (share == u) {
#pragma unroll
                for (int db = 0; db < R::DB; ++db)
#pragma unroll
                    for (int v = 0; v < 16; ++v) x[(db * 16 + v) * 64] = dq[db][v];
            }
            lds_barrier();
            if (share == 0) {
#pragma unroll
                for (int db = 0; db < R::DB; ++db)
#pragma unroll
                    for (int v = 0; v < 16; ++v) dq[db][v] += x[(db * 16 + v) * 64];
            }
        }
        if (share) return;
    }
    store_column<D>((unsigned short*)gdq + (q0 + (long long)qi) * a.dq_stride + (long long)head * D, dq, a.scale, half, live);
}

template <int D>
__global__ __launch_bounds__(256, D == 64 ? 2 : 1) void attn_dkv_kernel(GradArgs a) {
    typedef Rows<D> R;
    constexpr int kTileBytes = kStep * R::RB;
    // Q 0, Q 1, dO 0, dO 1, then lse and delta of each buffer's rows
    __shared__ __align__(4096) unsigned short lds[(4 * kTileBytes + 4 * kStep * 4) / 2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5;
    int unit, slot;
    const PromptSizes sz = read_sizes(a.p, a.slots);
    unit_slot(sz.P * sz.Hkv, sz.slots, blockIdx.x, unit, slot);
    const int G = sz.Hq / sz.Hkv, rank = unit / sz.Hkv, kvh = unit % sz.Hkv;
    auto gq = (Global<const unsigned short>)a.p.q[rank], gk = (Global<const unsigned short>)a.p.k[rank];
    auto gv = (Global<const unsigned short>)a.p.v[rank], ggo = (Global<const unsigned short>)a.go[rank];
    auto gdk = (Global<unsigned short>)a.dk[rank], gdv = (Global<unsigned short>)a.dv[rank];
    asm volatile("" : "+s"(gq), "+s"(gk), "+s"(gv), "+s"(ggo), "+s"(gdk), "+s"(gdv));
    PromptTile pt;
    if (!find_tile(sz.cu_k, sz.cu_q, sz.B, sz.Tk, sz.Tq, 1, kRowsWG, slot, lane, pt)) return;
    const int tile = pt.tile;                             // the first keys are seen by the most queries
    const int k0 = pt.lo, nk = pt.n, q0 = pt.lo2, nq = pt.n2, off = nk - nq;
    const int key0 = tile * kRowsWG + wave * 32;          // this wave's first key
    const int key = key0 + (lane & 31), keyc = key < nk ? key : nk - 1;

    bf16x8 kf[R::KK], vf[R::KK];
    {
        const unsigned short* kp = (const unsigned short*)gk + (k0 + (long long)keyc) * sz.k_stride + (long long)kvh * D + 8 * half;
        const unsigned short* vp = (const unsigned short*)gv + (k0 + (long long)keyc) * sz.v_stride + (long long)kvh * D + 8 * half;
#pragma unroll
        for (int kk = 0; kk < R::KK; ++kk) {
            kf[kk] = *(const bf16x8*)(kp + 16 * kk);
            vf[kk] = *(const bf16x8*)(vp + 16 * kk);
        }
    }
    // query i sees key j when i >= j - off
    const int first = sz.causal ? tile * kRowsWG - off : 0;          // first query that sees a key of the workgroup
    const int t0 = first > 0 ? first / kStep : 0, t1 = (nq + kStep - 1) / kStep;
    const int per = t1 > t0 ? t1 - t0 : 0, total = per * G;            // tiles of a head, of the group
    const unsigned qrow = (unsigned)(sz.q_stride * 2), grow = (unsigned)(a.go_stride * 2);
    TileLoad<D, kStep, kWaves> ql, gl;
    ql.init(lane, wave, qrow);
    gl.init(lane, wave, grow);
    Frags<D> fr;
    fr.init(lane);
    f32x16 dk[R::DB], dv[R::DB];
#pragma unroll
    for (int db = 0; db < R::DB; ++db)
#pragma unroll
        for (int v = 0; v < 16; ++v) dk[db][v] = dv[db][v] = 0.0f;
    const float c = sz.c;
    // restrict for the effect told at the forward pass: no wait for the next
    // tile's loads before a tile's transposed reads
    auto pass = [&](const unsigned short* __restrict__ qp, const unsigned short* __restrict__ gp) __attribute__((always_inline)) {
        int lg = 0, lt = t0;                                               // the next tile to load: head of the group, tile
        auto load = [&](int buf) {
            const int head = kvh * G + lg;
            const long long t = q0 + (long long)lt * kStep;
            const long long left = nq - (long long)lt * kStep;
            ql.issue(qp + t * sz.q_stride + (long long)head * D, left, qrow, lds, buf * kTileBytes);
            gl.issue(gp + t * a.go_stride + (long long)head * D, left, grow, lds, (2 + buf) * kTileBytes);
            if (wave < 2) {                                                // wave 0: lse, wave 1: delta, one value per lane
                const float* st = (wave ? a.delta : a.lse2) + ((long long)rank * sz.Hq + head) * sz.Tq + t;
                load_floats(st, left < kStep ? (int)left : kStep, lds, 4 * kTileBytes + (2 * buf + wave) * kStep * 4, lane);
            }
            if (++lt == t1) {
                lt = t0;
                ++lg;
            }
        };
        if (total) load(0);
        int ct = t0;                                                       // the tile being computed
        for (int it = 0; it < total; ++it) {
            const int buf = it & 1;
            wait_vm(0);
            lds_barrier();
            if (it + 1 < total) load(buf ^ 1);
            const int q = ct * kStep;
            if (++ct == t1) ct = t0;
            const int qa = buf * kTileBytes, ga = (2 + buf) * kTileBytes;
            const float* stat = (const float*)((const char*)lds + 4 * kTileBytes + 2 * buf * kStep * 4);
#pragma unroll
            for (int qb = 0; qb < kStep / 32; ++qb) {
                const int qr = q + qb * 32;
                if (sz.causal && qr + 31 + off < key0) continue;          // none of these queries sees a key of the wave
                f32x16 s, dp;
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int v = 0; v < 16; ++v) s[v] = dp[v] = 0.0f;
#pragma unroll
                for (int kk = 0; kk < R::KK; ++kk) {
                    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.rows(lds, qa, qb, kk), kf[kk], s, 0, 0, 0);
                    dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.rows(lds, ga, qb, kk), vf[kk], dp, 0, 0, 0);
                }
                __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
                for (int i = 0; i < 2 * R::KK - kAhead; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                }
                __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int r = qb * 32 + acc_row(v, half);
                    s[v] = exp2_hw(__builtin_fmaf(s[v], c, -stat[r]));
                    dp[v] = s[v] * (dp[v] - stat[kStep + r]);
                }
                if (sz.causal && qr + off < key0 + 31) {
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        if (qr + acc_row(v, half) + off < key) s[v] = dp[v] = 0.0f;
                }
                // columns of dO and Q in turn, kAhead ahead of their MFMA
                bf16x8 col[kAhead];
                auto column = [&](int i) {
                    col[i % kAhead] = fr.cols(lds, i % 2 ? qa : ga, i / 2 % R::DB, 2 * qb + i / (2 * R::DB));
                };
#pragma unroll
                for (int i = 0; i < kAhead; ++i) column(i);
                const bf16x8 pf[2] = {round8(s, 0), round8(s, 1)}, sf[2] = {round8(dp, 0), round8(dp, 1)};
#pragma unroll
                for (int i = 0; i < 4 * R::DB; ++i) {
                    const bf16x8 x = col[i % kAhead];
                    if (i + kAhead < 4 * R::DB) column(i + kAhead);
                    f32x16& acc = i % 2 ? dk[i / 2 % R::DB] : dv[i / 2 % R::DB];
                    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, i % 2 ? sf[i / (2 * R::DB)] : pf[i / (2 * R::DB)], acc, 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    };
    pass((const unsigned short*)gq, (const unsigned short*)ggo);
    store_column<D>((unsigned short*)gdk + (k0 + (long long)keyc) * a.dk_stride + (long long)kvh * D, dk, a.scale, half, key < nk);
    store_column<D>((unsigned short*)gdv + (k0 + (long long)keyc) * a.dv_stride + (long long)kvh * D, dv, 1.0f, half, key < nk);
}

// dK and dV where there are few keys for the device's compute units: a
// workgroup takes 32 keys, and its waves each a quarter of the (head of the
// group, 32 queries) items, every wave with LDS of its own and no barrier
// before the end, where the four sums are added in LDS, in the waves' order.
// Four times the workgroups, and a quarter of the steps one after the other,
// for four times the loads of Q and dO.
template <int D>
__global__ __launch_bounds__(256, D == 64 ? 2 : 1) void attn_dkv_few_kernel(GradArgs a) {
    typedef Rows<D> R;
    constexpr int kRows = 32, kPart = kRows * R::RB;     // queries of an item, bytes of its Q (or dO) tile
    constexpr int kStat = 64 * 4;                        // a load instruction of floats fills 64, the upper 32 with zeros
    // per wave: stages of Q and dO; then, per wave and stage, lse and delta
    __shared__ __align__(4096) unsigned short lds[kWaves * (4 * kPart + 4 * kStat) / 2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, col = lane & 31;
    int unit, slot;
    const PromptSizes sz = read_sizes(a.p, a.slots);
    unit_slot(sz.P * sz.Hkv, sz.slots, blockIdx.x, unit, slot);
    const int G = sz.Hq / sz.Hkv, rank = unit / sz.Hkv, kvh = unit % sz.Hkv;
    auto gq = (Global<const unsigned short>)a.p.q[rank], gk = (Global<const unsigned short>)a.p.k[rank];
    auto gv = (Global<const unsigned short>)a.p.v[rank], ggo = (Global<const unsigned short>)a.go[rank];
    auto gdk = (Global<unsigned short>)a.dk[rank], gdv = (Global<unsigned short>)a.dv[rank];
    asm volatile("" : "+s"(gq), "+s"(gk), "+s"(gv), "+s"(ggo), "+s"(gdk), "+s"(gdv));
    PromptTile pt;
    if (!find_tile(sz.cu_k, sz.cu_q, sz.B, sz.Tk, sz.Tq, 1, kRows, slot, lane, pt)) return;
    const int k0 = pt.lo, nk = pt.n, q0 = pt.lo2, nq = pt.n2, off = nk - nq;
    const int key0 = pt.tile * kRows, key = key0 + col, keyc = key < nk ? key : nk - 1;
    bf16x8 kf[R::KK], vf[R::KK];
    {
        const unsigned short* kp = (const unsigned short*)gk + (k0 + (long long)keyc) * sz.k_stride + (long long)kvh * D + 8 * half;
        const unsigned short* vp = (const unsigned short*)gv + (k0 + (long long)keyc) * sz.v_stride + (long long)kvh * D + 8 * half;
#pragma unroll
        for (int kk = 0; kk < R::KK; ++kk) {
            kf[kk] = *(const bf16x8*)(kp + 16 * kk);
            vf[kk] = *(const bf16x8*)(vp + 16 * kk);
        }
    }
    const int first = sz.causal ? key0 - off : 0;
    const int t0 = first > 0 ? first / kRows : 0, t1 = (nq + kRows - 1) / kRows;
    const int per = t1 > t0 ? t1 - t0 : 0, total = per * G;
    const unsigned qrow = (unsigned)(sz.q_stride * 2), grow = (unsigned)(a.go_stride * 2);
    TileLoad<D, kRows, 1> ql, gl;
    ql.init(lane, 0, qrow);
    gl.init(lane, 0, grow);
    Frags<D> fr;
    fr.init(lane);
    f32x16 dk[R::DB], dv[R::DB];
#pragma unroll
    for (int db = 0; db < R::DB; ++db)
#pragma unroll
        for (int v = 0; v < 16; ++v) dk[db][v] = dv[db][v] = 0.0f;
    const float c = sz.c;
    const int base = wave * 4 * kPart, stats = kWaves * 4 * kPart + wave * 4 * kStat;
    constexpr int kLoads = 2 * decltype(ql)::J + 2;
    // restrict for the effect told at the forward pass
    auto pass = [&](const unsigned short* __restrict__ qp, const unsigned short* __restrict__ gp) __attribute__((always_inline)) {
        auto load = [&](int it, int buf) {
            const int head = kvh * G + it / per, t = t0 + it % per;
            const long long row = q0 + (long long)t * kRows, left = nq - (long long)t * kRows;
            ql.issue(qp + row * sz.q_stride + (long long)head * D, left, qrow, lds, base + 2 * buf * kPart);
            gl.issue(gp + row * a.go_stride + (long long)head * D, left, grow, lds, base + (2 * buf + 1) * kPart);
            const long long st = ((long long)rank * sz.Hq + head) * sz.Tq + row;
            const int n = left < kRows ? (int)left : kRows;
            load_floats(a.lse2 + st, n, lds, stats + 2 * buf * kStat, lane);
            load_floats(a.delta + st, n, lds, stats + (2 * buf + 1) * kStat, lane);
        };
        if (wave < total) load(wave, 0);
        int buf = 0;
        for (int it = wave; it < total; it += kWaves, buf ^= 1) {
            const bool more = it + kWaves < total;
            if (more) load(it + kWaves, buf ^ 1);
            wait_vm(more ? kLoads : 0);                   // this item has landed (D = 128, 18 loads: and two of the next)
            const int qa = base + 2 * buf * kPart, ga = qa + kPart, q = (t0 + it % per) * kRows;
            const float* stat = (const float*)((const char*)lds + stats + 2 * buf * kStat);
            f32x16 s, dp;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int v = 0; v < 16; ++v) s[v] = dp[v] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < R::KK; ++kk) {
                s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.rows(lds, qa, 0, kk), kf[kk], s, 0, 0, 0);
                dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.rows(lds, ga, 0, kk), vf[kk], dp, 0, 0, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
            for (int i = 0; i < 2 * R::KK - kAhead; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int r = acc_row(v, half);
                s[v] = exp2_hw(__builtin_fmaf(s[v], c, -stat[r]));
                dp[v] = s[v] * (dp[v] - stat[kStat / 4 + r]);
            }
            if (sz.causal && q + off < key0 + 31) {
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    if (q + acc_row(v, half) + off < key) s[v] = dp[v] = 0.0f;
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const bf16x8 pf = round8(s, ks), sf = round8(dp, ks);
#pragma unroll
                for (int db = 0; db < R::DB; ++db) {
                    dv[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.cols(lds, ga, db, ks), pf, dv[db], 0, 0, 0);
                    dk[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.cols(lds, qa, db, ks), sf, dk[db], 0, 0, 0);
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // this stage's reads are done before it loads again
        }
    };
    pass((const unsigned short*)gq, (const unsigned short*)ggo);

    // the waves' sums: blocks of 32 x 32 floats, dK's then dV's, in each wave's tiles
    static_assert(2 * R::DB * 4096 <= 4 * kPart, "a wave's sums fit its tiles");
    float* mine = (float*)((char*)lds + base);
#pragma unroll
    for (int b = 0; b < 2 * R::DB; ++b)
#pragma unroll
        for (int v = 0; v < 16; ++v) mine[b * 1024 + acc_row(v, half) * 32 + col] = b < R::DB ? dk[b][v] : dv[b - R::DB][v];
    __syncthreads();
    const long long row = k0 + (long long)keyc;
#pragma unroll
    for (int i = 0; i < 2 * R::DB / kWaves; ++i) {
        const int b = i * kWaves + wave, db = b % R::DB;
        f32x16 x;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            x[v] = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                x[v] += ((const float*)((const char*)lds + w * 4 * kPart))[b * 1024 + acc_row(v, half) * 32 + col];
        }
        unsigned short* p = b < R::DB ? (unsigned short*)gdk + row * a.dk_stride : (unsigned short*)gdv + row * a.dv_stride;
        store_block(p + (long long)kvh * D + 32 * db, x, b < R::DB ? a.scale : 1.0f, half, key < nk);
    }
}

}  // namespace
}  // namespace ringc

using namespace ringc;

extern "C" size_t tp_attention_grad_workspace_bytes(int P, int Tq, int Hq) {
    if (P < 1 || P > RING_MAX_RANKS || Tq < 0 || Hq < 1) return 0;
    return kStatusBytes + ((size_t)P * Hq * Tq * 2 * sizeof(float) + 255) / 256 * 256;
}

extern "C" int tp_attention_grad(const void* const* dout, const void* const* q, const void* const* k, const void* const* v,
                                 const void* const* o, const float* const* lse, void* const* dq, void* const* dk,
                                 void* const* dv, const int* cu_q, const int* cu_k, int P, int B, int Tq, int Tk, int Hq,
                                 int Hkv, int D, long long q_stride, long long k_stride, long long v_stride,
                                 long long o_stride, long long dout_stride, long long dq_stride, long long dk_stride,
                                 long long dv_stride, int causal, float scale, void* ws, size_t ws_bytes, void* stream) {
    int rc = prompt_shape(P, B, Tq, Tk, Hq, Hkv, D, scale);
    if (rc != RING_OK) return rc;
    if (!dout || !q || !k || !v || !o || !lse || !dq || !dk || !dv) return RING_EINVAL;
    if (!row_stride_ok(q_stride, Hq, D) || !row_stride_ok(k_stride, Hkv, D) || !row_stride_ok(v_stride, Hkv, D) ||
        !row_stride_ok(o_stride, Hq, D) || !row_stride_ok(dout_stride, Hq, D) || !row_stride_ok(dq_stride, Hq, D) ||
        !row_stride_ok(dk_stride, Hkv, D) || !row_stride_ok(dv_stride, Hkv, D))
        return RING_EINVAL;
    if (B == 0 || (Tq == 0 && Tk == 0)) return RING_OK;
    if (!cu_q || !cu_k || (((uintptr_t)cu_q | (uintptr_t)cu_k) & 3)) return RING_EINVAL;
    GradArgs a;
    if (!fill_prompt_args(a.p, q, k, v, cu_q, cu_k, P, B, Tq, Tk, Hq, Hkv, D, q_stride, k_stride, v_stride,
                          causal ? 1 : 0, scale))
        return RING_EINVAL;
    for (int r = 0; r < P; ++r) {
        if (Tq && (!o[r] || !dout[r] || !lse[r] || !dq[r])) return RING_EINVAL;
        if (Tk && (!dk[r] || !dv[r])) return RING_EINVAL;
        if ((((uintptr_t)o[r] | (uintptr_t)dout[r] | (uintptr_t)dq[r] | (uintptr_t)dk[r] | (uintptr_t)dv[r]) & 15) ||
            ((uintptr_t)lse[r] & 3))
            return RING_EINVAL;
        a.o[r] = (const unsigned short*)o[r];
        a.go[r] = (const unsigned short*)dout[r];
        a.lse[r] = lse[r];
        a.dq[r] = (unsigned short*)dq[r];
        a.dk[r] = (unsigned short*)dk[r];
        a.dv[r] = (unsigned short*)dv[r];
    }
    const size_t need = tp_attention_grad_workspace_bytes(P, Tq, Hq);
    if (!ws || ((uintptr_t)ws & 255) || ws_bytes < need) return RING_EWORKSPACE;
    a.o_stride = o_stride;
    a.go_stride = dout_stride;
    a.dq_stride = dq_stride;
    a.dk_stride = dk_stride;
    a.dv_stride = dv_stride;
    a.lse2 = (float*)((char*)ws + kStatusBytes);
    a.delta = a.lse2 + (size_t)P * Hq * Tq;
    a.status = (Status*)ws;
    a.data = WsSpan{kStatusBytes, need};
    a.scale = scale;
    const int units = P * Hkv;
    hipStream_t s = (hipStream_t)stream;
    if (Tq) {
        a.slots = prompt_slots(B, Tq, Hq / Hkv, kRowsWG, units);
        if (!a.slots || (Tk && !prompt_slots(B, Tk, 1, kRowsWG, units))) return RING_EUNSUPPORTED;
        const dim3 grid((unsigned)a.slots * (unsigned)units);
        // Two shares where long prompts make few workgroups (keys a prompt on
        // average).  Both passes, one share / two: one prompt of 1000 / 2000 /
        // 6000 on a rank of 8 heads of 128 on 2 79 / 142 / 410 us and 76 / 134 /
        // 378, on 2 ranks of 4 heads of 64 on 2 39 / 69 / 204 and 36 / 61 / 176;
        // three of 1000 on 4 ranks 187 and 197; nine of 333 33 and 36.
        const bool shares = Tk / B >= 768 && 2LL * a.slots * units <= 3LL * dev_info().cus;
        if (shares && D == 128) hipLaunchKernelGGL((attn_dq_kernel<128, 2>), grid, dim3(512), 0, s, a);
        else if (shares) hipLaunchKernelGGL((attn_dq_kernel<64, 2>), grid, dim3(512), 0, s, a);
        else if (D == 128) hipLaunchKernelGGL((attn_dq_kernel<128, 1>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((attn_dq_kernel<64, 1>), grid, dim3(256), 0, s, a);
        if (hipGetLastError() != hipSuccess) return RING_EHIP;
    }
    if (Tk) {
        a.slots = prompt_slots(B, Tk, 1, kRowsWG, units);
        if (!a.slots) return RING_EUNSUPPORTED;
        // Few keys: at most one workgroup of 128 keys for every second compute
        // unit, or, in long prompts, whose first keys' workgroups run longest,
        // for every one.  4 ranks of 8 heads of 128 on 2, dQ (in one share)
        // included, 128 and 32 keys a workgroup: one prompt of 1024 / 2048 /
        // 4096 / 8192 tokens 160 / 315 / 691 / 1821 us and 82 / 172 / 572 / 2134;
        // 5 prompts of 80, 31 and 21; 8 of 512, 121 and 138.
        const long long groups = (long long)a.slots * units, cus = dev_info().cus;
        const bool few = 2 * groups <= cus || (groups <= cus + units && Tk / B >= 1024);
        if (few) a.slots = prompt_slots(B, Tk, 1, 32, units);
        if (!a.slots) return RING_EUNSUPPORTED;
        const dim3 grid((unsigned)a.slots * (unsigned)units);
        if (few && D == 128) hipLaunchKernelGGL(attn_dkv_few_kernel<128>, grid, dim3(256), 0, s, a);
        else if (few) hipLaunchKernelGGL(attn_dkv_few_kernel<64>, grid, dim3(256), 0, s, a);
        else if (D == 128) hipLaunchKernelGGL(attn_dkv_kernel<128>, grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL(attn_dkv_kernel<64>, grid, dim3(256), 0, s, a);
        if (hipGetLastError() != hipSuccess) return RING_EHIP;
    }
    return RING_OK;
}
