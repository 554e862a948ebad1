// beam_select.hip -- the best continuations of every group of beams.
//
// With m = max x and s = sum 2^((x - m) log2 e) over a row's logits,
//   lp = x - (m + ln s),
// and within a row lp orders as x does.  One pass over the logits gives m, s and
// where a row's largest logits lie:
//   - a wave takes a part of a row's columns of one rank, 1024 a step; every
//     lane keeps a running maximum and sum of its own, and the wave a list of
//     its `keep` largest lane maxima of a step, the i-th in lane i: the part's
//     `keep` largest logits are among the 16 values each that those are the
//     maxima of.  After the first steps few maxima exceed the list's last.
//   - a second launch, a workgroup a group, joins each row's parts to ln s in
//     64 bits, takes the group's `keep` best maxima off the heads of the parts'
//     lists, reads their values again (some 64 bytes each), and puts those that
//     are no worse than the last maximum in order.
// (Lists of values instead of maxima took a wave 144 operations where one is
// put in, 25 so: of 512 rows of 100003 logits two thirds of all operations.)
// The logits read bound it, and an exponential a logit, at a quarter of the
// rate of a plain operation: the 184 MB of 460 such rows take 37 us, 4.9 TB/s
// with the VALU 65% busy, and their join 8.5.  Four rows of 8000 take 5 and 6 us:
// launches and five trips to memory one after another.  A join by a group's
// last workgroup to finish instead of a launch was no faster (44 us for the
// large case in all, 43 so; 11.2 for the small one, 10.5 so): what it reads
// then has to pass the caches.
//
// The sum is of fp32 exponentials (the exponent's product with log2 e in two
// parts, so that its error is the rounding of x - m alone), added 16 at a time
// in pairs.  All sums of those, their logarithm and the scores are 64-bit
// numbers, since beams whose scores differ by less than fp32 shows are told
// apart by them: a running fp32 sum rounds once a step, which next to one large
// logit or on a slow ascent put the scores of 200000 tokens off by up to 4.7e-6,
// where they are off by 1.2e-7 so, of like logits by 1e-8 (1 us of the 37).
#include "attn_internal.h"
#include "tp_search.h"

#include <hip/hip_runtime.h>

namespace ringc {
namespace {

constexpr int kChunk = 1024;           // columns of a wave's step, 16 a lane
constexpr int kLists = 64;             // of a group, that a wave joins at once
constexpr int kMaxLists = BEAM_SELECT_MAX * RING_MAX_RANKS;
// Of a group, kept in LDS, and so that a row's parts are no more: 96 KB beside the
// kernel's own 30 of the 160.  16 beams into 16 of 200000 tokens take 41 us, 54 with
// 2048, 39 with 8000; 2 groups of 16 into 32 of 100000 on 4 ranks 61, 70, 61; 8 of 8
// into 16 of 100000 on 8 ranks 40, 39, 40.
constexpr int kLdsEntries = 6144, kLdsLists = 1024;

// A part's largest logit m, and the sum of exp(x - m).
struct alignas(16) MaxSum {
    double s;
    float m;
};

struct BeamArgs {
    const void* logits[RING_MAX_RANKS];
    const float* scores;
    const unsigned char* done;
    int *parents, *tokens;
    float* after;
    unsigned char* done_after;
    long long stride;
    int P, N, W, K, width, vocab, end, parts, part_cols;       // parts of a row of one rank, of part_cols columns
    Status* status;
    WsSpan data;
    MaxSum* ms;                        // [row][rank][part]
    float2* list;                      // [row][rank][part][K] maximum and (bits of) its step and lane
};

// (by value: of a vector's element itself, __builtin_bit_cast takes element 0)
__device__ __forceinline__ float f32_bits(unsigned x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ float bf16_bits(unsigned x) { return f32_bits(x << 16); }
// Logits that are not finite take no part.
__device__ __forceinline__ float only_finite(float x) { return __builtin_fabsf(x) < INFINITY ? x : -INFINITY; }
__device__ __forceinline__ float exp2_of(float d) {            // 2^(d log2 e)
    constexpr float hi = kLog2e, lo = 1.92596299e-8f;          // log2 e - hi
    return exp2_hw(__builtin_fmaf(d, hi, d * lo));
}

// e^(m - top) for m <= top, off by less than 2^-35 of it (so that what many rises
// of a maximum make of a sum adds up to nothing), 1 where they are equal and 0
// where m is -inf: 2^n e^r with |r| <= ln 2 / 2, e^r by its series up to r^9.
__device__ __forceinline__ double exp_below(float m, float top) {
    const double x = fmax((double)m - (double)top, -1000.0), n = __builtin_rint(x * 1.4426950408889634);     // (NaN gives -1000)
    const double r = __builtin_fma(n, -0.6931471805599453, x);
    double p = 1.0 / 362880;
    p = __builtin_fma(p, r, 1.0 / 40320);
    p = __builtin_fma(p, r, 1.0 / 5040);
    p = __builtin_fma(p, r, 1.0 / 720);
    p = __builtin_fma(p, r, 1.0 / 120);
    p = __builtin_fma(p, r, 1.0 / 24);
    p = __builtin_fma(p, r, 1.0 / 6);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}

// A wave's maximum, and its least number, in every lane: four steps within rows
// of 16 lanes and two across them on the VALU, then the last lane's.  (Through
// LDS, six exchanges, a value put into a list took 0.9 us.)
template <class Op> __device__ __forceinline__ int wave_reduce(int x, Op op) {
    x = op(x, __builtin_amdgcn_update_dpp(x, x, 0x111, 0xf, 0xf, false));
    x = op(x, __builtin_amdgcn_update_dpp(x, x, 0x112, 0xf, 0xf, false));
    x = op(x, __builtin_amdgcn_update_dpp(x, x, 0x114, 0xf, 0xf, false));
    x = op(x, __builtin_amdgcn_update_dpp(x, x, 0x118, 0xf, 0xf, false));
    x = op(x, __builtin_amdgcn_update_dpp(x, x, 0x142, 0xa, 0xf, false));
    x = op(x, __builtin_amdgcn_update_dpp(x, x, 0x143, 0xc, 0xf, false));
    return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ float as_float(int x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ int as_bits(float x) { return __builtin_bit_cast(int, x); }
__device__ __forceinline__ float wave_max(float x) {
    return as_float(wave_reduce(as_bits(x), [](int a, int b) { return as_bits(fmaxf(as_float(a), as_float(b))); }));
}
__device__ __forceinline__ int wave_min(int x) {
    return wave_reduce(x, [](int a, int b) { return a < b ? a : b; });
}
__device__ __forceinline__ unsigned wave_umax(unsigned x) {
    return (unsigned)wave_reduce((int)x, [](int a, int b) { return (unsigned)a > (unsigned)b ? a : b; });
}
// The value one lane below (lane 0 keeps its own).
__device__ __forceinline__ int lane_below(int x) { return __builtin_amdgcn_update_dpp(x, x, 0x138, 0xf, 0xf, false); }

// Where in a wave's step a value lies: column of lane and element, and the lane of a column.
template <bool F32> struct Step {
    static constexpr int V = F32 ? 4 : 8;                  // values of a 16-byte vector
    static __device__ __forceinline__ int column(int lane, int e) { return (e / V * 64 + lane) * V + e % V; }
    static __device__ __forceinline__ int lane(int column) { return column / V % 64; }
};

template <bool F32> __global__ __launch_bounds__(256) void beam_scan_kernel(BeamArgs a, unsigned works) {
    typedef Step<F32> At;
    __shared__ float reached[4];               // the last value of each wave's list
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (lane == 0) reached[wave] = -INFINITY;
    __syncthreads();
    const unsigned w = blockIdx.x * 4 + wave;
    if (blockIdx.x == 0 && threadIdx.x == 0) ws_add_data(a.status, a.data);
    if (w >= works) return;
    const int part = (int)(w % (unsigned)a.parts), rank = (int)(w / (unsigned)a.parts % (unsigned)a.P);
    const int row = (int)(w / (unsigned)a.parts / (unsigned)a.P);
    if ((a.done && a.done[row]) || !(__builtin_fabsf(a.scores[row]) < INFINITY)) return;
    const long long left = (long long)a.vocab - (long long)rank * a.width;
    const int cols = left < 0 ? 0 : left < a.width ? (int)left : a.width;       // of this rank
    const int c0 = part * a.part_cols, c1 = c0 + a.part_cols < cols ? c0 + a.part_cols : cols;
    constexpr int E = F32 ? 4 : 2;
    const char* base = (const char*)a.logits[rank] + (long long)row * a.stride * E;
    // a view holds whole words: the last of an odd number of bf16 values is loaded by itself
    const bool odd = !F32 && (cols & 1);
    const rsrc_t view = tile_view(base, (long long)(odd ? cols - 1 : cols) * E);
    const float tail = odd ? bf16_bits(((const unsigned short*)base)[cols - 1]) : 0.0f;
    // the workgroup's waves that have the same row
    const unsigned each = (unsigned)a.parts * a.P;
    const int v0 = (int)(blockIdx.x * 4 >= row * each ? 0 : row * each - blockIdx.x * 4);
    const int v1 = (int)((row + 1) * each - blockIdx.x * 4 < 4 ? (row + 1) * each - blockIdx.x * 4 : 4);
    float m = -INFINITY;                       // this lane's
    double s = 0.0;
    float best = -INFINITY, last = -INFINITY;  // the list: lane i's maximum, and the K-th
    int at = -1;                               // the step and lane it is the maximum of
    auto load = [&](int c, u32x4 (&r)[E]) {
#pragma unroll
        for (int v = 0; v < E; ++v) r[v] = ld16<POL_NT>(view, (unsigned)(c * E + (v * 64 + lane) * 16));
    };
    u32x4 raw[E];
    if (c0 < c1) load(c0, raw);
    for (int c = c0; c < c1; c += kChunk) {
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            if (F32) x[e] = f32_bits(raw[e / 4][e % 4]);
            else x[e] = bf16_bits(e % 2 ? raw[(e / 8) % E][e % 8 / 2] >> 16 : raw[(e / 8) % E][e % 8 / 2] & 0xffffu);
        }
        if (c + kChunk < c1) load(c + kChunk, raw);
        if (c + kChunk > c1) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int col = c + At::column(lane, e);
                if (col >= c1) x[e] = -INFINITY;
                else if (odd && col == cols - 1) x[e] = tail;
            }
        }
        float top, mn, sum;
        auto weigh = [&]() __attribute__((always_inline)) {
            top = x[0];
#pragma unroll
            for (int e = 1; e < 16; ++e) top = fmaxf(top, x[e]);
            mn = fmaxf(m, top);
            const float sub = mn == -INFINITY ? 0.0f : mn;
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = exp2_of(x[e] - sub);
#pragma unroll
            for (int d = 8; d; d /= 2)
#pragma unroll
                for (int e = 0; e < d; ++e) y[e] += y[e + d];
            sum = y[0];
        };
        weigh();
        // NaN and infinity make NaN of the sum: once more without them
        if (__any(!(sum < INFINITY))) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = only_finite(x[e]);
            weigh();
        }
        if (__any(mn > m)) s *= exp_below(m, mn);
        s += sum;
        m = mn;
        float others = -INFINITY;
        for (int v = v0; v < v1; ++v) others = fmaxf(others, ((volatile float*)reached)[v]);
        bool put = false;
        while (__any(top > last && top >= others)) {
            // (what the row's other waves have K of can only tie)
            const float v = wave_max(top);
            const unsigned long long has = __ballot(top == v);
            int owner = __builtin_ctzll(has);
            if (has & (has - 1)) {                         // several lanes: the lowest column
                int col = 0x7fffffff;
#pragma unroll
                for (int e = 15; e >= 0; --e)
                    if (x[e] == v) col = At::column(lane, e);
                owner = At::lane(wave_min(top == v ? col : 0x7fffffff));
            }
            const int pos = __builtin_popcountll(__ballot(lane < a.K && at >= 0 && best >= v));
            const float b1 = as_float(lane_below(as_bits(best)));
            const int a1 = lane_below(at);
            if (lane > pos) {
                best = b1;
                at = a1;
            }
            if (lane == pos) {
                best = v;
                at = c / kChunk * 64 + owner;
            }
            last = as_float(__builtin_amdgcn_readlane(as_bits(best), a.K - 1));
            put = true;
            if (lane == owner) top = -INFINITY;
        }
        if (put && lane == 0) ((volatile float*)reached)[wave] = last;
    }
    const float mw = wave_max(m);
    double sw = m > -INFINITY ? s * exp_below(m, mw) : 0.0;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sw += __shfl_xor(sw, d);
    if (lane == 0) a.ms[w] = MaxSum{sw, mw};
    if (lane < a.K) a.list[(long long)w * a.K + lane] = float2{best, __builtin_bit_cast(float, at)};
}

// Scores as numbers that order as they do; 0: none.
__device__ __forceinline__ unsigned long long order_of(double x) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
    return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double score_of(unsigned long long u) {
    return __builtin_bit_cast(double, u >> 63 ? u & ~(1ull << 63) : ~u);
}
// A candidate: of equal scores the lowest beam goes first, then the largest
// logit, whose bits in order, turned round, are the lower half of `after`.
struct Cand {
    unsigned long long score, after;
    int token;
};
__device__ __forceinline__ unsigned long long after_of(int beam, float logit) {
    const unsigned u = __builtin_bit_cast(unsigned, logit + 0.0f);       // (-0 is 0)
    return (unsigned long long)beam << 32 | (u >> 31 ? u : ~(u | 1u << 31));
}

template <bool F32> __global__ __launch_bounds__(1024) void beam_join_kernel(BeamArgs a, int in_lds) {
    typedef Step<F32> At;
    constexpr int E = F32 ? 4 : 2, V = At::V;
    extern __shared__ unsigned long long keys[];           // [lists][K] scores, where they fit, and the lists
    __shared__ double lse[BEAM_SELECT_MAX], score[BEAM_SELECT_MAX];
    __shared__ unsigned char head[kMaxLists], ended[BEAM_SELECT_MAX];      // entries of a list that are taken; done
    __shared__ int2 group[BEAM_SELECT_MAX];                // the best maxima: list and entry
    __shared__ union {
        Cand cand[16 * BEAM_SELECT_MAX];
        struct {                                           // before them: the best of each wave's lists
            unsigned long long score[16][BEAM_SELECT_MAX];
            int2 group[16][BEAM_SELECT_MAX];
        } of_wave;
    } both;
    Cand* cand = both.cand;
    __shared__ unsigned long long least;                   // the last of the best maxima
    __shared__ int count;
    const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int per = a.P * a.parts, lists = a.W * per, waves = blockDim.x / 64;
    const float2* from = a.list + (long long)n * lists * a.K;
    // the first loads of each kind in one trip
    const int row0 = n * a.W + (wave < a.W ? wave : 0);
    const float sc0 = a.scores[row0];
    const bool done0 = a.done && a.done[row0];
    const MaxSum first = lane < per ? a.ms[(long long)row0 * per + lane] : MaxSum{0.0, -INFINITY};
    float2* entries = (float2*)(keys + lists * a.K);
    constexpr int kEarly = 4;
    float2 early[kEarly];
#pragma unroll
    for (int u = 0; u < kEarly; ++u)
        if (in_lds && tid + u * (int)blockDim.x < lists * a.K) early[u] = from[tid + u * blockDim.x];
    for (int i = tid; i < lists; i += blockDim.x) head[i] = 0;
    for (int i = tid; i < a.K; i += blockDim.x) group[i] = int2{-1, 0};
    if (tid == 0) count = 0;
    for (int w = wave; w < a.W; w += waves) {
        const int row = n * a.W + w;
        const float sc = w == wave ? sc0 : a.scores[row];
        const MaxSum* p = a.ms + (long long)row * per;
        const MaxSum p0 = w == wave ? first : lane < per ? p[lane] : MaxSum{0.0, -INFINITY};
        const bool live = __builtin_fabsf(sc) < INFINITY, done = w == wave ? done0 : a.done && a.done[row];
        double l = 0.0;
        if (live && !done) {
            float m = p0.m;
            for (int i = lane + 64; i < per; i += 64) m = fmaxf(m, p[i].m);
            m = wave_max(m);
            double s = p0.m > -INFINITY ? p0.s * exp_below(p0.m, m) : 0.0;
            for (int i = lane + 64; i < per; i += 64)
                if (p[i].m > -INFINITY) s += p[i].s * exp_below(p[i].m, m);
            for (int d = 1; d < per && d < 64; d *= 2) s += __shfl_xor(s, d);
            l = (double)m + log(s);
        }
        if (lane == 0) {
            lse[w] = l;
            score[w] = live ? (double)sc : -INFINITY;
            ended[w] = done;
        }
    }
    __syncthreads();
    // the score of list i's entry e (its h-th), 0 where there is none
    auto key = [&](int i, int h, float2 e) -> unsigned long long {
        const int w = (int)((unsigned)i / (unsigned)per);
        if (!(score[w] > -INFINITY)) return 0;
        if (ended[w]) return i == w * per && !h ? order_of(score[w]) : 0;
        return as_bits(e.y) < 0 ? 0 : order_of(score[w] + ((double)e.x - lse[w]));
    };
    if (in_lds) {
#pragma unroll
        for (int u = 0; u < kEarly; ++u) {
            const int j = tid + u * blockDim.x;
            if (j < lists * a.K) {
                keys[j] = key(j / a.K, j % a.K, early[u]);
                entries[j] = early[u];
            }
        }
        for (int j = tid + kEarly * blockDim.x; j < lists * a.K; j += blockDim.x) {
            const float2 e = from[j];
            keys[j] = key(j / a.K, j % a.K, e);
            entries[j] = e;
        }
        __syncthreads();
    }
    // The wave's best of one score a lane, by its halves.  Of equals the first
    // beam's, of its (a large score takes the difference away) the largest logit,
    // of equals the first list's: lists are in the order of beams and columns.
    auto best = [&](unsigned long long top, int list, int h, int& owner) {
        const unsigned hi = wave_umax((unsigned)(top >> 32));
        const unsigned lo = wave_umax((unsigned)(top >> 32) == hi ? (unsigned)top : 0u);
        const unsigned long long u = (unsigned long long)hi << 32 | lo, tie = __ballot(top == u);
        owner = __builtin_ctzll(tie);
        if (!u || !(tie & (tie - 1))) return u;
        const int w = (int)((unsigned)list / (unsigned)per), w0 = wave_min(top == u ? w : 0x7fffffff);
        const bool mine = top == u && w == w0;
        const float x = !mine || ended[w0] ? -INFINITY : in_lds ? entries[list * a.K + h].x : from[list * a.K + h].x;
        const float most = wave_max(x);
        const int first = wave_min(mine && x == most ? list : 0x7fffffff);
        owner = __builtin_ctzll(__ballot(mine && list == first));
        return u;
    };
    const int joins = (lists + kLists - 1) / kLists;       // waves that join a list a lane
    if (in_lds && wave < joins) {
        // its next score at hand (a look at LDS in every round took it from 350
        // to 1300 cycles)
        const int list = wave * kLists + lane;
        const unsigned long long* mine = keys + (list < lists ? list : 0) * a.K;
        int h = 0, owner;
        unsigned long long top = list < lists ? mine[0] : 0, next = list < lists && a.K > 1 ? mine[1] : 0, u = 0;
        for (int k = 0; k < a.K; ++k) {
            u = best(top, list, h, owner);
            if (lane == owner) {
                if (joins == 1) {
                    if (u) group[k] = int2{list, h};
                } else {
                    both.of_wave.group[wave][k] = int2{list, h};
                    both.of_wave.score[wave][k] = u;
                }
                top = next;
                ++h;
                next = h + 1 < a.K ? mine[h + 1] : 0;
            }
            if (!u && joins == 1) break;
        }
        if (joins == 1 && lane == 0) least = u;
    }
    if (in_lds && joins > 1) {
        __syncthreads();
        if (wave == 0) {
            int h = 0, owner;
            unsigned long long top = lane < joins ? both.of_wave.score[lane][0] : 0, u = 0;
            int2 g = lane < joins ? both.of_wave.group[lane][0] : int2{0, 0};
            for (int k = 0; k < a.K; ++k) {
                u = best(top, g.x, g.y, owner);
                if (!u) break;
                if (lane == owner) {
                    group[k] = g;
                    if (++h < a.K) g = both.of_wave.group[lane][h];
                    top = h < a.K ? both.of_wave.score[lane][h] : 0;
                }
            }
            if (lane == 0) least = u;
        }
    }
    if (!in_lds && wave == 0) {
        unsigned long long top = 0, u = 0;
        int list = 0, owner;
        auto look = [&]() {
            top = 0;
            list = 0;
            for (int i = lane; i < lists; i += 64) {
                const int h = head[i];
                if (h >= a.K) continue;
                const unsigned long long x = key(i, h, from[i * a.K + h]);
                if (x > top) {
                    top = x;
                    list = i;
                }
            }
        };
        look();
        for (int k = 0; k < a.K; ++k) {
            u = best(top, list, head[list], owner);
            if (!u) break;
            if (lane == owner) {
                group[k] = int2{list, head[list]++};
                look();
            }
        }
        if (lane == 0) least = u;
    }
    __syncthreads();
    // the values that those are the maxima of, as far as they can be among the best
    auto put = [&](unsigned long long u, int w, int token, float x) {
        const int i = __hip_atomic_fetch_add(&count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        cand[i] = Cand{u, after_of(w, x), token};
    };
    for (int t = tid; t < a.K * E; t += blockDim.x) {
        int2 g = group[t / E];
        if (g.x < 0) continue;
        g.y = as_bits((in_lds ? entries[g.x * a.K + g.y] : from[g.x * a.K + g.y]).y);
        const int w = (int)((unsigned)g.x / (unsigned)per), row = n * a.W + w;
        if (ended[w]) {
            if (t % E == 0) put(order_of(score[w]), w, a.end, 0.0f);
            continue;
        }
        const int rank = (int)((unsigned)(g.x - w * per) / (unsigned)a.parts), c = g.y / 64 * kChunk + At::column(g.y % 64, t % E * V);
        const long long left = (long long)a.vocab - (long long)rank * a.width;
        const int cols = left < a.width ? (int)left : a.width;
        const char* p = (const char*)a.logits[rank] + ((long long)row * a.stride + c) * (F32 ? 4 : 2);
        unsigned x[4] = {0, 0, 0, 0};
        if (c + V <= cols) {
            const u32x4 y = *(const u32x4*)p;
#pragma unroll
            for (int v = 0; v < 4; ++v) x[v] = y[v];
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (c + e < cols) {
                    if (F32) x[e % 4] = *(const unsigned*)(p + 4 * e);
                    else x[e / 2 % 4] |= (unsigned)*(const unsigned short*)(p + 2 * e) << (e % 2 * 16);
                }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float f = F32 ? f32_bits(x[e % 4]) : bf16_bits(e % 2 ? x[e / 2 % 4] >> 16 : x[e / 2 % 4] & 0xffffu);
            if (c + e >= cols || !(__builtin_fabsf(f) < INFINITY)) continue;
            const unsigned long long u = order_of(score[w] + ((double)f - lse[w]));
            if (u >= least) put(u, w, rank * a.width + c + e, f);
        }
    }
    __syncthreads();
    // each one's place is the number of those that beat it
    const int all = count;
    for (int i = tid; i < all; i += blockDim.x) {
        const Cand c = cand[i];
        int k = 0;
#pragma unroll 4
        for (int j = 0; j < all; ++j) {
            const Cand o = cand[j];
            k += o.score > c.score || (o.score == c.score && (o.after < c.after || (o.after == c.after && o.token < c.token)));
        }
        if (k < a.K) {
            const long long o = (long long)n * a.K + k;
            const int beam = (int)(c.after >> 32);
            a.parents[o] = n * a.W + beam;
            a.tokens[o] = c.token;
            a.after[o] = (float)score_of(c.score);
            if (a.done_after) a.done_after[o] = ended[beam] || c.token == a.end;
        }
    }
    for (int k = tid; k < a.K; k += blockDim.x)
        if (k >= all) {
            const long long o = (long long)n * a.K + k;
            a.parents[o] = a.tokens[o] = -1;
            a.after[o] = -INFINITY;
            if (a.done_after) a.done_after[o] = 0;
        }
}

// Parts of a row of one rank: as many as give every SIMD four waves (eight, each
// with a list of its own to fill, took 71 us where four took 58), as far as there
// are steps; up to 64 lists a group, more only where a part has four steps, as the
// join then takes two turns.  One group of 16 beams into 16 of 200000 tokens
// takes 41 us with 352 lists, 70 with 64; of 8 into 8 of 150000 to 200000 23 to 24.
struct BeamCut {
    int parts, cols;
};
BeamCut beam_cut(int P, int N, int beams, int keep, int width, int cus) {
    const long long rows = (long long)N * beams * P, steps = ((long long)width + kChunk - 1) / kChunk;
    const int each = beams * P, most = kLdsEntries / keep < kLdsLists ? kLdsEntries / keep : kLdsLists;
    long long n = rows ? (16LL * cus + rows - 1) / rows : 1;
    if (n > steps) n = steps;
    if (n > kLists / each && n > steps / 4) n = kLists / each > steps / 4 ? kLists / each : steps / 4;
    if (n > most / each && n > kLists / each) n = most / each > kLists / each ? most / each : kLists / each;
    if (n < 1) n = 1;
    const long long cols = (steps + n - 1) / n * kChunk;
    BeamCut c;
    c.cols = (int)(cols < 0x7fffffff - kChunk ? cols : 0x7fffffff / kChunk * kChunk);
    c.parts = (int)(steps ? (width + cols - 1) / cols : 1);
    return c;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    return a && b && (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

bool beam_shape(int P, int N, int beams, int keep, int width) {
    return P >= 1 && P <= RING_MAX_RANKS && N >= 0 && beams >= 1 && beams <= BEAM_SELECT_MAX && keep >= 1 && keep <= BEAM_SELECT_MAX &&
           width >= 1 && width <= (1 << 28) && (long long)P * width < (1LL << 31) && (long long)N * beams * P < (1LL << 24);
}

}  // namespace
}  // namespace ringc

using namespace ringc;

extern "C" size_t beam_select_workspace_bytes(int P, int N, int beams, int keep, int width) {
    if (!beam_shape(P, N, beams, keep, width)) return 0;
    const BeamCut c = beam_cut(P, N, beams, keep, width, dev_info().cus);
    const size_t lists = (size_t)P * N * beams * c.parts;
    return kStatusBytes + (lists * (keep * sizeof(float2) + sizeof(MaxSum)) + 255) / 256 * 256;
}

extern "C" int beam_select(const void* const* logits, const float* scores, const unsigned char* done, int* parents,
                           int* tokens, float* scores_after, unsigned char* done_after, int P, int N, int beams, int keep,
                           int width, int vocab, long long stride, int end_token, int dtype, void* ws, size_t ws_bytes,
                           void* stream) {
    if (P < 1 || P > RING_MAX_RANKS || N < 0 || beams < 1 || keep < 1 || width < 1 || vocab < 1) return RING_EINVAL;
    if (dtype != RING_F32 && dtype != RING_BF16) return RING_EUNSUPPORTED;
    if (!beam_shape(P, N, beams, keep, width)) return RING_EUNSUPPORTED;
    if (vocab > (long long)P * width || stride < width || stride % 8 || stride >= (1LL << 31)) return RING_EINVAL;
    if (end_token < -1 || end_token >= vocab || (done && end_token < 0) || !done != !done_after) return RING_EINVAL;
    if (N == 0) return RING_OK;
    if (!logits || !scores || !parents || !tokens || !scores_after) return RING_EINVAL;
    if (((uintptr_t)scores | (uintptr_t)parents | (uintptr_t)tokens | (uintptr_t)scores_after) & 3) return RING_EINVAL;
    // a group may write before another reads
    const size_t in = (size_t)N * beams, out = (size_t)N * keep;
    for (const void* p : {(const void*)parents, (const void*)tokens, (const void*)scores_after})
        if (overlap(p, 4 * out, scores, 4 * in) || overlap(p, 4 * out, done, in)) return RING_EINVAL;
    if (overlap(done_after, out, scores, 4 * in) || overlap(done_after, out, done, in)) return RING_EINVAL;
    const size_t need = beam_select_workspace_bytes(P, N, beams, keep, width);
    if (!ws || ((uintptr_t)ws & 255) || ws_bytes < need) return RING_EWORKSPACE;
    BeamArgs a;
    for (int r = 0; r < P; ++r) {
        if (!logits[r] || ((uintptr_t)logits[r] & 15)) return RING_EINVAL;
        a.logits[r] = logits[r];
    }
    const BeamCut c = beam_cut(P, N, beams, keep, width, dev_info().cus);
    a.scores = scores;
    a.done = done;
    a.parents = parents;
    a.tokens = tokens;
    a.after = scores_after;
    a.done_after = done_after;
    a.stride = stride;
    a.P = P;
    a.N = N;
    a.W = beams;
    a.K = keep;
    a.width = width;
    a.vocab = vocab;
    a.end = end_token;
    a.parts = c.parts;
    a.part_cols = c.cols;
    a.status = (Status*)ws;
    a.data = WsSpan{kStatusBytes, need};
    const size_t lists = (size_t)P * N * beams * c.parts;
    a.ms = (MaxSum*)((char*)ws + kStatusBytes);
    a.list = (float2*)(a.ms + lists);
    if (lists >= (1ull << 31)) return RING_EUNSUPPORTED;
    const dim3 grid((unsigned)((lists + 3) / 4));
    hipStream_t s = (hipStream_t)stream;
    if (dtype == RING_F32) hipLaunchKernelGGL(beam_scan_kernel<true>, grid, dim3(256), 0, s, a, (unsigned)lists);
    else hipLaunchKernelGGL(beam_scan_kernel<false>, grid, dim3(256), 0, s, a, (unsigned)lists);
    if (hipGetLastError() != hipSuccess) return RING_EHIP;
    const int group_lists = beams * P * c.parts, entries = group_lists * keep, in_lds = entries <= kLdsEntries && group_lists <= kLdsLists;
    const int joins = in_lds ? (group_lists + kLists - 1) / kLists : 1, rows = beams < 4 ? 4 : beams < 16 ? beams : 16;
    const dim3 block(64u * (joins > rows ? joins : rows));
    const size_t dyn = in_lds ? entries * 16 : 0;
    if (dtype == RING_F32) hipLaunchKernelGGL(beam_join_kernel<true>, dim3((unsigned)N), block, dyn, s, a, in_lds);
    else hipLaunchKernelGGL(beam_join_kernel<false>, dim3((unsigned)N), block, dyn, s, a, in_lds);
    return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
}
