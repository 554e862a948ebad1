// beam_select.hip -- the best continuations of every group of beams.
//
// With m = max x and s = sum 2^((x - m) log2 e) over a row's logits,
//   lp = x - (m + ln s),
// and a group's best are among each row's `keep` largest logits: within a row
// lp orders as x does.  One pass over the logits gives m, s and those:
//   - a wave takes a part of a row's columns of one rank; every lane keeps a
//     running maximum and sum of its own, and the wave a list of its largest
//     values, the i-th in lane i.  A value that exceeds the list's last is put
//     in; after the first few hundred columns few do.
//   - a second launch, a workgroup a group, joins each row's parts to ln s in
//     64 bits and takes the group's best off the heads of the parts' lists, one
//     after the other.
// The logits read bound it: an exponential is a sixteenth of the rate of a
// plain operation, four exponentials a cycle and SIMD.
//
// The sum is of fp32 exponentials (the exponent's product with log2 e in two
// parts, so that its error is the rounding of x - m alone), added 16 at a time
// in pairs; its logarithm and the scores are 64-bit numbers, since beams whose
// scores differ by less than fp32 shows are told apart by them.
#include "attn_internal.h"
#include "tp_search.h"

#include <hip/hip_runtime.h>

namespace ringc {
namespace {

constexpr int kChunk = 1024;           // columns of a wave's step, 16 a lane
constexpr int kMaxLists = 4096;        // of a group

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
    float2* ms;                        // [row][rank][part] m, s
    float2* list;                      // [row][rank][part][K] value and (bits of) column
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

// The wave's maximum; its least integer.
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x = fmaxf(x, __shfl_xor(x, d));
    return x;
}
__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_xor(x, d);
        x = x < y ? x : y;
    }
    return x;
}

template <bool F32> __global__ __launch_bounds__(256) void beam_scan_kernel(BeamArgs a, unsigned works) {
    const unsigned w = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (blockIdx.x == 0 && threadIdx.x == 0) ws_add_data(a.status, a.data);
    if (w >= works) return;
    const int lane = threadIdx.x & 63;
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
    const float tail = odd ? only_finite(bf16_bits(((const unsigned short*)base)[cols - 1])) : 0.0f;
    float m = -INFINITY, s = 0.0f;             // this lane's
    float best = -INFINITY, last = -INFINITY;  // the list: lane i's value, and the K-th
    int at = -1;                               // its column
    auto column = [&](int e) { return F32 ? (e / 4 * 64 + lane) * 4 + e % 4 : (e / 8 * 64 + lane) * 8 + e % 8; };
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
            x[e] = only_finite(x[e]);
        }
        if (c + kChunk < c1) load(c + kChunk, raw);
        if (c + kChunk > c1) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (c + column(e) >= c1) x[e] = -INFINITY;
                else if (odd && c + column(e) == cols - 1) x[e] = tail;
        }
        float top = x[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = fmaxf(top, x[e]);
        const float mn = fmaxf(m, top);
        if (mn > -INFINITY) {
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = exp2_of(x[e] - mn);
#pragma unroll
            for (int d = 8; d; d /= 2)
#pragma unroll
                for (int e = 0; e < d; ++e) y[e] += y[e + d];
            s = s * exp2_of(m - mn) + y[0];
            m = mn;
        }
        while (__any(top > last)) {
            const float v = wave_max(top);
            int col = 0x7fffffff;
#pragma unroll
            for (int e = 15; e >= 0; --e)
                if (x[e] == v) col = c + column(e);
            const int first = wave_min(col);
            const int pos = __builtin_popcountll(__ballot(lane < a.K && at >= 0 && best >= v));
            const float b1 = __shfl_up(best, 1);
            const int a1 = __shfl_up(at, 1);
            if (lane > pos) {
                best = b1;
                at = a1;
            }
            if (lane == pos) {
                best = v;
                at = first;
            }
            last = __shfl(best, a.K - 1);
            top = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if (c + column(e) == first) x[e] = -INFINITY;
                top = fmaxf(top, x[e]);
            }
        }
    }
    const float mw = wave_max(m);
    float sw = m > -INFINITY ? s * exp2_of(m - mw) : 0.0f;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sw += __shfl_xor(sw, d);
    if (lane == 0) a.ms[w] = float2{mw, sw};
    if (lane < a.K) a.list[(long long)w * a.K + lane] = float2{best, __builtin_bit_cast(float, at)};
}

// A candidate: its score, and its place among equals.
struct Cand {
    double score;
    long long place;                   // beam * vocab + token; none: score -inf
    __device__ __forceinline__ bool beats(const Cand& o) const { return score > o.score || (score == o.score && place < o.place); }
};
__device__ __forceinline__ Cand wave_best(Cand c) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        Cand o;
        o.score = __shfl_xor(c.score, d);
        o.place = __shfl_xor(c.place, d);
        if (o.beats(c)) c = o;
    }
    return c;
}

__global__ __launch_bounds__(256) void beam_join_kernel(BeamArgs a) {
    __shared__ double lse[BEAM_SELECT_MAX], score[BEAM_SELECT_MAX];
    __shared__ unsigned char head[kMaxLists];              // entries of a list that are taken
    const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int per = a.P * a.parts, lists = a.W * per;
    for (int i = tid; i < lists; i += 256) head[i] = 0;
    for (int w = wave; w < a.W; w += 4) {
        const int row = n * a.W + w;
        const float sc = a.scores[row];
        const bool live = __builtin_fabsf(sc) < INFINITY, done = a.done && a.done[row];
        double l = 0.0;
        if (live && !done) {
            const float2* p = a.ms + (long long)row * per;
            float m = -INFINITY;
            for (int i = lane; i < per; i += 64) m = fmaxf(m, p[i].x);
            m = wave_max(m);
            double s = 0.0;
            for (int i = lane; i < per; i += 64)
                if (p[i].x > -INFINITY) s += (double)p[i].y * exp((double)p[i].x - (double)m);
#pragma unroll
            for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
            l = (double)m + log(s);
        }
        if (lane == 0) {
            lse[w] = l;
            score[w] = live ? (double)sc : -INFINITY;
        }
    }
    __syncthreads();
    if (wave) return;
    // the best head of this lane's lists
    auto look = [&]() {
        Cand c = {-INFINITY, 0x7fffffffffffffffLL};
        for (int i = lane; i < lists; i += 64) {
            const int w = i / per, row = n * a.W + w;
            if (!(score[w] > -INFINITY)) continue;
            Cand x = {-INFINITY, 0x7fffffffffffffffLL};
            if (a.done && a.done[row]) {
                if (i % per == 0 && !head[i]) x = Cand{score[w], (long long)w * a.vocab + a.end};
            } else if (head[i] < a.K) {
                const float2 e = a.list[((long long)row * per + i % per) * a.K + head[i]];
                const int at = __builtin_bit_cast(int, e.y);
                if (at >= 0) x = Cand{score[w] + ((double)e.x - lse[w]), (long long)w * a.vocab + i % per / a.parts * a.width + at};
            }
            if (x.beats(c)) c = x;
        }
        return c;
    };
    auto list_of = [&](long long place) {                  // the list a candidate came from
        const int w = (int)(place / a.vocab), t = (int)(place % a.vocab);
        if (a.done && a.done[n * a.W + w]) return w * per;
        return w * per + t / a.width * a.parts + t % a.width / a.part_cols;
    };
    Cand mine = look();
    for (int k = 0; k < a.K; ++k) {
        const Cand c = wave_best(mine);
        const bool any = c.score > -INFINITY;
        const int w = any ? (int)(c.place / a.vocab) : 0, t = any ? (int)(c.place % a.vocab) : -1;
        if (lane == 0) {
            const long long o = (long long)n * a.K + k;
            a.parents[o] = any ? n * a.W + w : -1;
            a.tokens[o] = t;
            a.after[o] = any ? (float)c.score : -INFINITY;
            if (a.done_after) a.done_after[o] = any && (a.done[n * a.W + w] || t == a.end);
        }
        if (any && mine.place == c.place) {
            ++head[list_of(c.place)];
            mine = look();
        }
    }
}

// Parts of a row of one rank: as many as give every SIMD four waves, as far as
// a part keeps two steps and a group's lists are few enough.
struct BeamCut {
    int parts, cols;
};
BeamCut beam_cut(int P, int N, int beams, int width, int cus) {
    const long long rows = (long long)N * beams * P, steps = ((long long)width + kChunk - 1) / kChunk;
    long long n = rows ? (16LL * cus + rows - 1) / rows : 1;
    if (n > steps / 2) n = steps / 2;
    if (n > kMaxLists / (beams * P)) n = kMaxLists / (beams * P);
    if (n < 1) n = 1;
    const long long cols = (steps + n - 1) / n * kChunk;
    BeamCut c;
    c.cols = (int)(cols < 0x7fffffff - kChunk ? cols : 0x7fffffff / kChunk * kChunk);
    c.parts = (int)(steps ? (width + cols - 1) / cols : 1);
    return c;
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
    const BeamCut c = beam_cut(P, N, beams, width, dev_info().cus);
    const size_t lists = (size_t)P * N * beams * c.parts;
    return kStatusBytes + (lists * (keep + 1) * sizeof(float2) + 255) / 256 * 256;
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
    const size_t need = beam_select_workspace_bytes(P, N, beams, keep, width);
    if (!ws || ((uintptr_t)ws & 255) || ws_bytes < need) return RING_EWORKSPACE;
    BeamArgs a;
    for (int r = 0; r < P; ++r) {
        if (!logits[r] || ((uintptr_t)logits[r] & 15)) return RING_EINVAL;
        a.logits[r] = logits[r];
    }
    const BeamCut c = beam_cut(P, N, beams, width, dev_info().cus);
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
    a.ms = (float2*)((char*)ws + kStatusBytes);
    a.list = a.ms + lists;
    if (lists >= (1ull << 31)) return RING_EUNSUPPORTED;
    const dim3 grid((unsigned)((lists + 3) / 4));
    hipStream_t s = (hipStream_t)stream;
    if (dtype == RING_F32) hipLaunchKernelGGL(beam_scan_kernel<true>, grid, dim3(256), 0, s, a, (unsigned)lists);
    else hipLaunchKernelGGL(beam_scan_kernel<false>, grid, dim3(256), 0, s, a, (unsigned)lists);
    if (hipGetLastError() != hipSuccess) return RING_EHIP;
    hipLaunchKernelGGL(beam_join_kernel, dim3((unsigned)N), dim3(256), 0, s, a);
    return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
}
