// attn_prompt.hip -- attention over packed prompts with grouped heads.
//
//   S = scale Q K^T over the keys a query sees, m = max S, P = exp(S - m),
//   l = sum P, O = P V / l, lse = m + log l.
//
// One pass over the keys with the running maximum and sum.  A workgroup of
// four waves takes 128 rows of one (rank, key head): row i G + g is query i of
// the prompt and query head g of the G that share the key head, so the group
// reads every key tile once.  Each wave keeps 32 of the rows (its Q fragments
// and the accumulators of O^T) in registers; key and value tiles go through two
// LDS buffers each, the next tile loading while one is computed.
//
// Tiles of 64 keys and two workgroups on a compute unit, one computing its
// weights while the other multiplies; for D = 128, where many short prompts
// make many workgroups that spend much of their time in their first loads and
// last stores, tiles of 32 keys and three (kShort).
//
// One prompt of 16384 tokens on 4 ranks of 4 heads of 128 on 1: 1000 to 1080
// us, 1.02 to 1.1 PFLOP/s, at the card's power limit (matrix cores 56% busy at 1.7
// GHz).  D = 64 has half the products per weight, so its vector instructions
// count for more (the VALU is active 79% of the time, nearly a third of that in
// exponentials, the matrix cores 50%, at 1.7 GHz): 16384 tokens on 4 ranks of 4
// heads of 64 on 1, 610 to 680 us.  12 prompts of 8192 tokens in all, 4 ranks of
// 8 heads of 128 on 2: 93 us, where reading Q and writing O alone would take 35;
// the waves wait 40% of their cycles.
#include "attn_core.h"
#include "attn_internal.h"

#include <hip/hip_runtime.h>

namespace ringc {
namespace {

constexpr int kTileRows = 128;     // rows (query, head of the group) of a workgroup
constexpr int kWaves = 4;
// D = 128 takes tiles of 32 keys below this many keys a prompt on average, with
// more than four workgroups a compute unit: 8192 tokens on 4 ranks of 8 heads
// on 2 in prompts of 64 / 256 / 683 / 2048 keys take 33 / 47 / 73 / 166 us with
// 32 and 42 / 50 / 77 / 164 us with 64; one prompt of 1000, 31 and 24 us.
constexpr int kShort = 1024;
// Long prompts that make few workgroups are bound by the tiles that one goes
// through after another: their workgroups have two or four shares of four
// waves, each with its own buffers and every second or fourth tile, whose sums
// are joined in LDS.  D = 64, one share / two / four: one prompt of 1000 on 4
// ranks of 4 heads 18 / 15 / 15 us, 2000 32 / 25 / 23, 6000 on 2 ranks 85 / 66 /
// 57; nine of 333 12.4 / 12.9 / 19.  D = 128, one / two: one prompt of 1000 on a
// rank of 8 heads on 2 22 / 20, 3000 54 / 45, 6000 113 / 94; ten of 600 23 / 26.
constexpr int kAhead = 4;        // row fragments asked for ahead of their MFMA

struct FwdArgs {
    PromptArgs p;
    unsigned short* o[RING_MAX_RANKS];
    float* lse[RING_MAX_RANKS];               // may be null
    long long o_stride;
    int slots;
};

template <int D, int kTileKeys, int kShares>
__global__ __launch_bounds__(256 * kShares, kTileKeys == 32 ? 3 : 2) void attn_fwd_kernel(FwdArgs a) {
    typedef Rows<D> R;
    constexpr int kTileBytes = kTileKeys * R::RB;
    __shared__ __align__(4096) unsigned short lds[kShares * 4 * kTileBytes / 2];   // of each share: K 0, K 1, V 0, V 1
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % kWaves;
    const int share = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / kWaves;
    const int half = lane >> 5;
    int unit, slot;
    const PromptSizes sz = read_sizes(a.p, a.slots);
    unit_slot(sz.P * sz.Hkv, sz.slots, blockIdx.x, unit, slot);
    const int G = sz.Hq / sz.Hkv, rank = unit / sz.Hkv, kvh = unit % sz.Hkv;
    auto gq = (Global<const unsigned short>)a.p.q[rank], gk = (Global<const unsigned short>)a.p.k[rank];
    auto gv = (Global<const unsigned short>)a.p.v[rank];
    auto go = (Global<unsigned short>)a.o[rank];
    auto glse = (Global<float>)a.lse[rank];
    long long o_stride = a.o_stride;
    asm volatile("" : "+s"(gq), "+s"(gk), "+s"(gv), "+s"(go), "+s"(glse), "+s"(o_stride));     // the rank's, in one trip
    PromptTile pt;
    if (!find_tile(sz.cu_q, sz.cu_k, sz.B, sz.Tq, sz.Tk, G, kTileRows, slot, lane, pt)) return;
    const int tile = pt.tiles - 1 - pt.tile;                 // the longest first
    const int q0 = pt.lo, nq = pt.n, k0 = pt.lo2, nk = pt.n2;
    // this lane's row; rows past the end repeat the last one and are not stored
    const unsigned rows = (unsigned)nq * (unsigned)G, m0 = (unsigned)(tile * kTileRows + wave * 32);
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
        most = upto((unsigned)(tile * kTileRows + kTileRows - 1));
    }

    bf16x8 qf[R::KK];
    {
        const unsigned short* qp = (const unsigned short*)gq + (q0 + (long long)qi) * sz.q_stride + (long long)head * D + 8 * half;
#pragma unroll
        for (int kk = 0; kk < R::KK; ++kk) qf[kk] = *(const bf16x8*)(qp + 16 * kk);
    }
    const unsigned krow = (unsigned)(sz.k_stride * 2), vrow = (unsigned)(sz.v_stride * 2);
    const unsigned short* kbase = (const unsigned short*)gk + (long long)k0 * sz.k_stride + (long long)kvh * D;
    const unsigned short* vbase = (const unsigned short*)gv + (long long)k0 * sz.v_stride + (long long)kvh * D;
    TileLoad<D, kTileKeys, kWaves> kl, vl;
    kl.init(lane, wave, krow);
    vl.init(lane, wave, vrow);
    Frags<D> fr;
    fr.init(lane);
    f32x16 o[R::DB];
#pragma unroll
    for (int db = 0; db < R::DB; ++db)
#pragma unroll
        for (int v = 0; v < 16; ++v) o[db][v] = 0.0f;
    float mc = -INFINITY;                 // running maximum times c (of both halves of the column)
    float lp[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // this half's share of the sum, in four parts
    const float c = sz.c;

    // The pass is a function of restrict pointers for one effect: its LDS reads
    // are then known not to alias what it loads from, and the compiler leaves
    // out the wait for every load in flight, the next tile's, that it otherwise
    // puts before each tile's first transposed read.
    auto pass = [&](const unsigned short* __restrict__ kp, const unsigned short* __restrict__ vp) __attribute__((always_inline)) {
        auto load = [&](int j, int buf) {
            const int at = (share * 4 + buf) * kTileBytes;
            kl.issue(kp + (long long)j * kTileKeys * sz.k_stride, nk - (long long)j * kTileKeys, krow, lds, at);
            vl.issue(vp + (long long)j * kTileKeys * sz.v_stride, nk - (long long)j * kTileKeys, vrow, lds, at + 2 * kTileBytes);
        };
        const int tiles = (most + kTileKeys - 1) / kTileKeys;
        if (share < tiles) load(share, 0);
        for (int i = 0; i * kShares < tiles; ++i) {
            const int j = i * kShares + share, buf = i & 1;
            wait_vm(0);                       // tile j has landed
            lds_barrier();                    // everyone's has; the buffers of the turn before are free
            if (j + kShares < tiles) load(j + kShares, buf ^ 1);
            if (j * kTileKeys >= some) continue;    // nothing here for this wave's rows
            const int ka = (share * 4 + buf) * kTileBytes, va = ka + 2 * kTileBytes;
            f32x16 s[kTileKeys / 32];
            // row reads kAhead MFMAs early; left alone, the compiler puts each
            // next to its use and waits out the LDS latency every time
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kb = 0; kb < kTileKeys / 32; ++kb)
#pragma unroll
                for (int v = 0; v < 16; ++v) s[kb][v] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < R::KK; ++kk)
#pragma unroll
                for (int kb = 0; kb < kTileKeys / 32; ++kb)
                    s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.rows(lds, ka, kb, kk), qf[kk], s[kb], 0, 0, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
            for (int i = 0; i < kTileKeys / 32 * R::KK - kAhead; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
            __builtin_amdgcn_sched_barrier(0);
            if ((j + 1) * kTileKeys > every) {
#pragma unroll
                for (int kb = 0; kb < kTileKeys / 32; ++kb)
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        if (j * kTileKeys + kb * 32 + acc_row(v, half) >= seen) s[kb][v] = -INFINITY;
            }
            float mx = s[0][0];
#pragma unroll
            for (int kb = 0; kb < kTileKeys / 32; ++kb)
#pragma unroll
                for (int v = 0; v < 16; ++v) mx = fmaxf(mx, s[kb][v]);
            mx = max_halves(mx) * c;
            // The maximum only keeps the exponents in range: it moves when some
            // row's grows by more than 2^8, which P in bf16 and its fp32 sums hold
            // as exactly as values up to 1.
            if (__any(mx > mc + 8.0f)) {
                const float mn = fmaxf(mc, mx);
                const float alpha = mn == -INFINITY ? 1.0f : exp2_hw(mc - mn);
                mc = mn;
#pragma unroll
                for (int i = 0; i < 4; ++i) lp[i] *= alpha;
#pragma unroll
                for (int db = 0; db < R::DB; ++db)
#pragma unroll
                    for (int v = 0; v < 16; ++v) o[db][v] *= alpha;
            }
            const float sub = mc == -INFINITY ? 0.0f : mc;
#pragma unroll
            for (int kb = 0; kb < kTileKeys / 32; ++kb)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    s[kb][v] = exp2_hw(__builtin_fmaf(s[kb][v], c, -sub));
                    lp[v % 4] += s[kb][v];
                }
            // P is rounded to bf16 for the matrix cores (relative error up to
            // 2^-8 of each weight; l sums the unrounded ones in fp32).
#pragma unroll
            for (int ks = 0; ks < kTileKeys / 16; ++ks) {
                const bf16x8 pf = round8(s[ks / 2], ks % 2);
#pragma unroll
                for (int db = 0; db < R::DB; ++db)
                    o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr.cols(lds, va, db, ks), pf, o[db], 0, 0, 0);
            }
        }
    };
    pass(kbase, vbase);
    float l = sum_halves((lp[0] + lp[1]) + (lp[2] + lp[3]));

    // the shares' sums, brought to one maximum, to the first share
    if constexpr (kShares > 1) {
        constexpr int kRegs = 16 * R::DB + 2;
        static_assert(kRegs * 4 * 64 * kWaves <= (int)sizeof(lds), "one share's sums");
        float* x = (float*)lds + wave * kRegs * 64 + lane;
#pragma unroll
        for (int u = 1; u < kShares; ++u) {
            lds_barrier();                    // the tiles, or the share before, have been read
            if (share == u) {
#pragma unroll
                for (int db = 0; db < R::DB; ++db)
#pragma unroll
                    for (int v = 0; v < 16; ++v) x[(db * 16 + v) * 64] = o[db][v];
                x[(kRegs - 2) * 64] = l;
                x[(kRegs - 1) * 64] = mc;
            }
            lds_barrier();
            if (share == 0) {
                const float lu = x[(kRegs - 2) * 64], mu = x[(kRegs - 1) * 64], mn = fmaxf(mc, mu);
                const float f = mc == mn ? 1.0f : exp2_hw(mc - mn), fu = mu == mn ? 1.0f : exp2_hw(mu - mn);
                mc = mn;
                l = l * f + lu * fu;
#pragma unroll
                for (int db = 0; db < R::DB; ++db)
#pragma unroll
                    for (int v = 0; v < 16; ++v) o[db][v] = __builtin_fmaf(x[(db * 16 + v) * 64], fu, o[db][v] * f);
            }
        }
        if (share) return;
    }

    // The product of a weight that the mask made 0 with a value that is not
    // finite is NaN, in rows that do not see the value.  So where a result of a
    // causal call is not finite the wave makes its rows again, key by key, each
    // key added only to the rows that see it.  That is one trip to memory per key,
    // some 2 us: 16384 tokens on 4 ranks of 4 heads of 128 take 34 ms with one NaN
    // in the last query and 76 ms where no row is finite, instead of 1.1; 12
    // prompts of 8192 tokens in all 2.4 and 3.9 ms instead of 0.08.  It also makes
    // the 32-key kernel spill 109 registers, in this part alone.
    if (sz.causal) {
        float z = 0.0f * l;
#pragma unroll
        for (int db = 0; db < R::DB; ++db)
#pragma unroll
            for (int v = 0; v < 16; ++v) z = __builtin_fmaf(o[db][v], 0.0f, z);
        if (__any(z != 0.0f)) {
            mc = -INFINITY;
            l = 0.0f;
#pragma unroll
            for (int db = 0; db < R::DB; ++db)
#pragma unroll
                for (int v = 0; v < 16; ++v) o[db][v] = 0.0f;
            for (int key = 0; key < some; ++key) {
                const unsigned short* kr = kbase + (long long)key * sz.k_stride + 8 * half;
                const unsigned short* vr = vbase + (long long)key * sz.v_stride + 4 * half;
                float s = 0.0f;
#pragma unroll
                for (int kk = 0; kk < R::KK; ++kk) {
                    const bf16x8 x = *(const bf16x8*)(kr + 16 * kk);
                    bf16x8 y = qf[kk];
                    asm volatile("" : "+v"(y));          // converted here, not once for all keys
#pragma unroll
                    for (int e = 0; e < 8; ++e) s = __builtin_fmaf((float)y[e], (float)x[e], s);
                    __builtin_amdgcn_sched_barrier(0);   // few registers, not speed
                }
                const bool sees = key < seen;
                s = sees ? sum_halves(s) * c : -INFINITY;
                const float mn = fmaxf(mc, s), sub = mn == -INFINITY ? 0.0f : mn;
                const float alpha = mn == mc ? 1.0f : exp2_hw(mc - mn), w = exp2_hw(s - sub);
                mc = mn;
                l = l * alpha + w;
#pragma unroll
                for (int db = 0; db < R::DB; ++db)
#pragma unroll
                    for (int v = 0; v < 16; v += 4) {
                        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                        const bf16x4 x = *(const bf16x4*)(vr + 32 * db + 2 * v);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[db][v + e] = sees ? __builtin_fmaf(w, (float)x[e], o[db][v + e] * alpha) : o[db][v + e];
                        __builtin_amdgcn_sched_barrier(0);
                    }
            }
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;          // a row that sees no key gives zeros
    // D = 128 stores whole rows through the tiles' LDS (128 prompts of 64 on 4
    // ranks of 8 heads 34 to 32.5 us, nine of 333 27 to 25); D = 64, whose rows
    // are half a line wide and whose registers the rows' places would cost a
    // wave, does not (18 to 20 us)
    if constexpr (D == 128) {
        lds_barrier();                                       // every wave has read the tiles
        unsigned row = m;
        asm volatile("" : "+v"(row));                        // its place is computed here, not before the pass
        const unsigned first = m0 / (unsigned)G;
        const unsigned at = (row / (unsigned)G - first) * (unsigned)o_stride + row % (unsigned)G * (unsigned)D;
        const int n = rows > m0 ? (rows - m0 < 32 ? (int)(rows - m0) : 32) : 0;
        store_rows<D>((unsigned short*)go + (q0 + (long long)first) * o_stride + (long long)kvh * G * D, o, inv, at, n, lds,
                      wave * 32 * R::RB, lane);
    } else {
        store_column<D>((unsigned short*)go + (q0 + (long long)qi) * o_stride + (long long)head * D, o, inv, half, live);
    }
    if (glse && live && half == 0)
        glse[(long long)head * sz.Tq + q0 + qi] = l == 0.0f ? -INFINITY : (mc + __log2f(l)) * kLn2;
}

}  // namespace

bool fill_prompt_args(PromptArgs& p, const void* const* q, const void* const* k, const void* const* v, const int* cu_q,
                      const int* cu_k, int P, int B, int Tq, int Tk, int Hq, int Hkv, int D, long long q_stride,
                      long long k_stride, long long v_stride, int causal, float scale) {
    for (int r = 0; r < P; ++r) {
        p.q[r] = (const unsigned short*)q[r];
        p.k[r] = (const unsigned short*)k[r];
        p.v[r] = (const unsigned short*)v[r];
        if ((Tq && !q[r]) || (Tk && (!k[r] || !v[r]))) return false;     // what has no element may have no address
        if (((uintptr_t)q[r] | (uintptr_t)k[r] | (uintptr_t)v[r]) & 15) return false;
    }
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.B = B;
    p.Tq = Tq;
    p.Tk = Tk;
    p.P = P;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.causal = causal;
    p.c = scale * kLog2e;
    return true;
}

// What every packed-prompt call checks of its sizes.  Row strides are whole
// 16-byte chunks, so that every head row is 16-byte aligned, and below 2^21
// elements, so that a tile's view stays below 2 GiB.
int prompt_shape(int P, int B, int Tq, int Tk, int Hq, int Hkv, int D, float scale) {
    if (P < 1 || P > RING_MAX_RANKS || B < 0 || Tq < 0 || Tk < 0 || Hq < 1 || Hkv < 1) return RING_EINVAL;
    if (!scale_ok(scale)) return RING_EINVAL;
    if (Hq % Hkv || (D != 64 && D != 128) || (long long)Hq * D >= kMaxRow || (long long)Hkv * D >= kMaxRow)
        return RING_EUNSUPPORTED;
    return RING_OK;
}
bool row_stride_ok(long long stride, int heads, int D) {
    return stride >= (long long)heads * D && stride < kMaxRow && stride % 8 == 0;
}
// Tiles of `rows` rows that prompts of `total` tokens, `per` rows each, can
// make: 0 if there are too many for a launch or for 32-bit row numbers.
int prompt_slots(int B, int total, int per, int rows, int units) {
    if ((long long)total * per >= (1LL << 31) - rows) return 0;
    const long long n = (long long)total * per / rows + (B < total ? B : total);
    return n * (units > 8 ? units : 8) < (1LL << 31) ? (int)n : 0;
}

}  // namespace ringc

using namespace ringc;

extern "C" int tp_attention(const void* const* q, const void* const* k, const void* const* v, void* const* o,
                            float* const* lse, const int* cu_q, const int* cu_k, int P, int B, int Tq, int Tk, int Hq,
                            int Hkv, int D, long long q_stride, long long k_stride, long long v_stride,
                            long long o_stride, int causal, float scale, void* stream) {
    int rc = prompt_shape(P, B, Tq, Tk, Hq, Hkv, D, scale);
    if (rc != RING_OK) return rc;
    if (!q || !k || !v || !o) return RING_EINVAL;
    if (!row_stride_ok(q_stride, Hq, D) || !row_stride_ok(k_stride, Hkv, D) || !row_stride_ok(v_stride, Hkv, D) ||
        !row_stride_ok(o_stride, Hq, D))
        return RING_EINVAL;
    if (Tq == 0 || B == 0) return RING_OK;
    if (!cu_q || !cu_k || (((uintptr_t)cu_q | (uintptr_t)cu_k) & 3)) return RING_EINVAL;
    FwdArgs a;
    if (!fill_prompt_args(a.p, q, k, v, cu_q, cu_k, P, B, Tq, Tk, Hq, Hkv, D, q_stride, k_stride, v_stride,
                          causal ? 1 : 0, scale))
        return RING_EINVAL;
    for (int r = 0; r < P; ++r) {
        if (!o[r] || ((uintptr_t)o[r] & 15) || (lse && (!lse[r] || ((uintptr_t)lse[r] & 3)))) return RING_EINVAL;
        a.o[r] = (unsigned short*)o[r];
        a.lse[r] = lse ? lse[r] : nullptr;
    }
    a.o_stride = o_stride;
    const int units = P * Hkv;
    a.slots = prompt_slots(B, Tq, Hq / Hkv, kTileRows, units);
    if (!a.slots) return RING_EUNSUPPORTED;
    const dim3 grid((unsigned)a.slots * (unsigned)units);
    hipStream_t st = (hipStream_t)stream;
    const long long groups = (long long)a.slots * units, cus = dev_info().cus, keys = Tk / B;
    if (D == 64) {
        if (keys >= 2048 && 2 * groups <= 3 * cus)
            hipLaunchKernelGGL((attn_fwd_kernel<64, 64, 4>), grid, dim3(1024), 0, st, a);
        else if (keys >= 256 && groups * 256 <= cus * (keys < 1024 ? keys : 1024))
            hipLaunchKernelGGL((attn_fwd_kernel<64, 64, 2>), grid, dim3(512), 0, st, a);
        else
            hipLaunchKernelGGL((attn_fwd_kernel<64, 64, 1>), grid, dim3(256), 0, st, a);
    } else if (keys >= 512 && 2 * groups <= 3 * cus) {
        hipLaunchKernelGGL((attn_fwd_kernel<128, 64, 2>), grid, dim3(512), 0, st, a);
    } else if (keys < kShort && groups > 4 * cus) {
        hipLaunchKernelGGL((attn_fwd_kernel<128, 32, 1>), grid, dim3(256), 0, st, a);
    } else {
        hipLaunchKernelGGL((attn_fwd_kernel<128, 64, 1>), grid, dim3(256), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
}
