// qk_rope.hip -- per-head RMS norm of queries and keys with the position
// rotation and the cache write in one pass, and its gradient.
//
//   n = x / sqrt(mean(x^2) + eps),  y = n gain,
//   z_i = y_i cos - y_{i+h} sin,  z_{i+h} = y_{i+h} cos + y_i sin   (i < h = rot / 2)
// and back, with u = dy gain, dy the gradient turned the other way:
//   dx = (u - n mean(n u)) / sqrt(mean(x^2) + eps),   dgain = sum dy n.
//
// Memory bounds both: every value is read and written once.  D / 8 lanes hold
// one head row, 8 values each, so a wave covers 512 / D head rows of one token
// with 16-byte accesses; the row's mean is a reduction over those lanes and
// the rotation's partner values come from the lane rot / 16 further on.  Going
// forward a wave has one such group of rows, so a step of few tokens runs wide
// (a wave per token, its rows one group after the other, took 6.8 us for 32
// tokens of 12 heads on 4 ranks; this 3.7); going back it keeps one group of
// rows for many tokens, since it sums the gains' gradients in registers.
//
// 8192 tokens of 12 heads of 128 on 4 ranks, fp32 rows, with the cache write:
// 61.5 us, 5.5 TB/s.  Back, 4097 tokens of 24 heads of 64 in bf16 on 4 ranks:
// 26 us, 5.2 TB/s, and 4.9 for the sum of the gains' parts in a second launch.
#include "global_ptr.h"
#include "ring_device.h"
#include "tp_attention.h"

#include <hip/hip_runtime.h>

namespace ringc {
namespace {

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct RopeArgs {
    const void* qkv[RING_MAX_RANKS];
    const float *gq[RING_MAX_RANKS], *gk[RING_MAX_RANKS];
    unsigned short *q[RING_MAX_RANKS], *k[RING_MAX_RANKS], *v[RING_MAX_RANKS];      // the gradients, going back
    unsigned short *kc[RING_MAX_RANKS], *vc[RING_MAX_RANKS];
    const float* cs;
    const int* pos;
    const long long* slots;
    long long table_rows, cache_rows, stride;
    int P, T, Hq, Hkv, rot;
    float eps;
};

__device__ __forceinline__ f32x8 load8(const float* p) {
    const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ f32x8 load8(const unsigned short* p) {
    return __builtin_convertvector(*(const bf16x8*)p, f32x8);
}
// Nontemporal: the lines leave the L2s as they fill, not in one flush at the
// kernel's end (the gradient of 4097 tokens of 24 heads of 64 on 4 ranks 38.4
// us without, 34.4 so; 8192 tokens forward 62.7 and 61.5).
__device__ __forceinline__ void store8(float* p, const f32x8& x) {
    __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, (f32x4*)p);
    __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, (f32x4*)(p + 4));
}
__device__ __forceinline__ void store8(unsigned short* p, const f32x8& x) {
    __builtin_nontemporal_store(__builtin_convertvector(x, bf16x8), (bf16x8*)p);
}

// Sum over the W lanes that share a head row.
template <int W> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int d = 1; d < W; d *= 2) x += __shfl_xor(x, d);
    return x;
}

// This lane's cos and sin (its 8 values' pairs), as x -> a x + b partner(x).
struct Turn {
    f32x8 a, b;
    int partner;        // lane that holds the other values of the pairs
    bool turns;
};
template <int D>
__device__ __forceinline__ Turn make_turn(const float* cs, long long p, long long table_rows, int rot, int lane) {
    Turn r;
    const int i = lane % (D / 8), w = rot / 16;          // lanes [0, w) hold the pairs' first values, [w, 2 w) the second
    r.turns = i < 2 * w;
    r.partner = lane + (r.turns ? (i < w ? w : -w) : 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        r.a[e] = 1.0f;
        r.b[e] = 0.0f;
    }
    if (p < 0 || p >= table_rows) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r.a[e] = __builtin_nanf("");
    } else if (r.turns) {
        const float* c = cs + p * rot + (i < w ? i : i - w) * 8;
        r.a = load8(c);
        r.b = load8(c + rot / 2);
        if (i < w)
#pragma unroll
            for (int e = 0; e < 8; ++e) r.b[e] = -r.b[e];
    }
    return r;
}
__device__ __forceinline__ f32x8 turn(const Turn& r, const f32x8& y) {
    f32x8 z;
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = r.a[e] * y[e] + r.b[e] * __shfl(y[e], r.partner);
    return z;
}

template <int D, class X>
__global__ __launch_bounds__(256) void qk_rope_kernel(RopeArgs a, int groups) {
    constexpr int W = D / 8, HW = 64 / W;          // lanes of a head row, head rows of a wave
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane % W, rank = blockIdx.y;
    // All the arguments in one trip to the kernel's argument memory: left
    // alone, the compiler reads each where it is first used, one after the
    // other (8192 tokens of 12 heads on 4 ranks took 71 us so, and take 63).
    auto gx = (Global<const X>)a.qkv[rank];
    auto ggq = (Global<const float>)a.gq[rank], ggk = (Global<const float>)a.gk[rank], gcs = (Global<const float>)a.cs;
    auto gqo = (Global<unsigned short>)a.q[rank], gko = (Global<unsigned short>)a.k[rank], gvo = (Global<unsigned short>)a.v[rank];
    auto gkc = (Global<unsigned short>)a.kc[rank], gvc = (Global<unsigned short>)a.vc[rank];
    auto gpos = (Global<const int>)a.pos;
    auto gslots = (Global<const long long>)a.slots;
    long long stride = a.stride, table_rows = a.table_rows, cache_rows = a.cache_rows;
    int T = a.T, Hq = a.Hq, Hkv = a.Hkv, rot = a.rot;
    float eps = a.eps;
    asm volatile("" : "+s"(gx), "+s"(ggq), "+s"(ggk), "+s"(gcs), "+s"(gqo), "+s"(gko), "+s"(gvo), "+s"(gkc), "+s"(gvc),
                      "+s"(gpos), "+s"(gslots), "+s"(stride), "+s"(table_rows), "+s"(cache_rows), "+s"(T), "+s"(Hq),
                      "+s"(Hkv), "+s"(rot), "+s"(eps), "+s"(groups));
    const X* x = (const X*)gx;
    const float *gq = (const float*)ggq, *gk = (const float*)ggk, *cs = (const float*)gcs;
    unsigned short *qo = (unsigned short*)gqo, *ko = (unsigned short*)gko, *vo = (unsigned short*)gvo;
    unsigned short *kc = (unsigned short*)gkc, *vc = (unsigned short*)gvc;
    const int* pos = (const int*)gpos;
    const long long* slots = (const long long*)gslots;
    // item of the rank: token, then group of HW head rows
    const unsigned it = blockIdx.x * 4 + wave;
    const int t = (int)(it / (unsigned)groups), h = (int)(it % (unsigned)groups) * HW + lane / W;
    const int H = Hq + 2 * Hkv;
    if (t >= T) return;
    const bool is_q = h < Hq, is_k = !is_q && h < Hq + Hkv, is_v = !is_q && !is_k && h < H;
    // the position first, which the table's row waits for; a lane past the
    // heads reads the last one
    const int p = pos[t];
    const long long slot = slots ? slots[t] : -1;
    const bool cached = slot >= 0 && slot < cache_rows;
    const f32x8 y = load8(x + t * stride + (h < H ? h : H - 1) * D + 8 * i);
    f32x8 g = y;
    if (gq) g = load8((is_q ? gq : gk) + 8 * i);
    const Turn r = make_turn<D>(cs, p, table_rows, rot, lane);
    f32x8 z = y;
    if (gq) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s += y[e] * y[e];
        const float inv = 1.0f / sqrtf(row_sum<W>(s) * (1.0f / D) + eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = y[e] * inv * g[e];
    }
    z = turn(r, z);
    if (is_q) {
        store8(qo + ((long long)t * Hq + h) * D + 8 * i, z);
    } else if (is_k) {
        const int g = h - Hq;
        if (ko) store8(ko + ((long long)t * Hkv + g) * D + 8 * i, z);
        if (cached) store8(kc + (slot * Hkv + g) * D + 8 * i, z);
    } else if (is_v) {
        const int g = h - Hq - Hkv;
        if (vo) store8(vo + ((long long)t * Hkv + g) * D + 8 * i, y);
        if (cached) store8(vc + (slot * Hkv + g) * D + 8 * i, y);
    }
}

// Workgroups a compute unit, as many as fit by registers: each has one token's
// loads in flight, so it takes them all (4097 tokens of 24 heads of 64 on 4
// ranks, with 2 / 3 / 4 / 5 / 6: 55 / 46 / 43 / 40 / 39 us; with 8, whose last
// two wait, 47).
constexpr int kGradPerCu = 6;
constexpr int kGradLeast = 1024;       // and room for as many parts per rank, which every group of head rows may need
int grad_blocks_most(int P) {
    const int n = (kGradPerCu * dev_info().cus + P - 1) / P;
    return n > kGradLeast ? n : kGradLeast;
}

struct RopeGradArgs {
    RopeArgs f;                        // q, k, v: the gradients read; kc, vc: unused
    void* dx[RING_MAX_RANKS];
    float* part;                       // [P][blocks][2][D]
    Status* status;
    WsSpan data;
    int blocks, groups;
};

template <int D, class X>
__global__ __launch_bounds__(256, kGradPerCu) void qk_rope_grad_kernel(RopeGradArgs g) {
    constexpr int W = D / 8, HW = 64 / W;
    __shared__ float sum[4][HW][2][D];
    const RopeArgs& a = g.f;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = lane / W, i = lane % W;
    const int H = a.Hq + 2 * a.Hkv, rank = blockIdx.y;
    if (blockIdx.x == 0 && rank == 0 && threadIdx.x == 0) ws_add_data(g.status, g.data);
    const bool norm = a.gq[rank] != nullptr;
    // a wave keeps to one group of head rows, of every step-th token, so a lane
    // sums one gain's gradient
    const int w = blockIdx.x * 4 + wave, step = g.blocks * 4 / g.groups;
    const int h = w % g.groups * HW + sub, t0 = w / g.groups < step ? w / g.groups : a.T;
    const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hkv, there = h < H;
    const int hh = there ? h : H - 1;
    const unsigned short* dz0 = is_q ? a.q[rank] + (long long)h * D
                              : is_k ? a.k[rank] + (long long)(h - a.Hq) * D
                                     : a.v[rank] + (long long)(hh - a.Hq - a.Hkv) * D;
    const int heads = is_q ? a.Hq : a.Hkv;
    f32x8 gain, s8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        s8[e] = 0.0f;
        gain[e] = 1.0f;
    }
    if (norm && (is_q || is_k)) gain = load8((is_q ? a.gq : a.gk)[rank] + 8 * i);
    for (int t = t0; t < a.T; t += step) {
        const f32x8 dz = load8(dz0 + (long long)t * heads * D + 8 * i);
        f32x8 y;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = 0.0f;
        if (norm && (is_q || is_k)) y = load8((const X*)a.qkv[rank] + t * a.stride + h * D + 8 * i);
        const int p = a.pos[t];
        Turn r = make_turn<D>(a.cs, p, a.table_rows, a.rot, lane);
#pragma unroll
        for (int e = 0; e < 8; ++e) r.b[e] = -r.b[e];          // the other way
        f32x8 d = turn(r, dz);
        if (norm) {
            const bool known = p >= 0 && p < a.table_rows;
            float s = 0.0f, c = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += y[e] * y[e];
            const float inv = 1.0f / sqrtf(row_sum<W>(s) * (1.0f / D) + a.eps);
            f32x8 n;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                n[e] = y[e] * inv;
                s8[e] += known ? d[e] * n[e] : 0.0f;
                d[e] *= gain[e];
                c += d[e] * n[e];
            }
            c = row_sum<W>(c) * (1.0f / D);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = (d[e] - n[e] * c) * inv;
        }
        if (there) store8((X*)g.dx[rank] + ((long long)t * H + h) * D + 8 * i, is_q || is_k ? d : dz);
    }
    if (!norm) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        sum[wave][sub][0][8 * i + e] = is_q ? s8[e] : 0.0f;
        sum[wave][sub][1][8 * i + e] = is_k ? s8[e] : 0.0f;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * D; j += 256) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int u = 0; u < HW; ++u) s += sum[w][u][j / D][j % D];
        g.part[(((long long)rank * g.blocks + blockIdx.x) * 2 + j / D) * D + j % D] = s;
    }
}

struct GainArgs {
    const float* part;
    float *dgq[RING_MAX_RANKS], *dgk[RING_MAX_RANKS];
    int blocks;
};

// dgain = the workgroups' partial sums, added in a fixed order: D / 4 lanes
// hold a gain, 4096 / D such groups sum every 4096 / D-th workgroup's part and
// their sums are added one after the other.
template <int D>
__global__ __launch_bounds__(1024) void gain_sum_kernel(GainArgs g) {
    constexpr int L = D / 4, kGroups = 1024 / L;
    __shared__ f32x4 sum[kGroups][L];
    const int rank = blockIdx.x, which = blockIdx.y, i = threadIdx.x % L, u = threadIdx.x / L;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int b = u; b < g.blocks; b += kGroups)
        s += *(const f32x4*)(g.part + (((long long)rank * g.blocks + b) * 2 + which) * D + 4 * i);
    sum[u][i] = s;
    __syncthreads();
    if (u) return;
#pragma unroll 8
    for (int w = 1; w < kGroups; ++w) s += sum[w][i];
    *(f32x4*)((which ? g.dgk : g.dgq)[rank] + 4 * i) = s;
}

int rope_shape(int P, int T, int Hq, int Hkv, int D, int rot, long long table_rows, long long cache_rows,
               long long stride, float eps, int dtype) {
    if (P < 1 || P > RING_MAX_RANKS || T < 0 || Hq < 1 || Hkv < 1 || table_rows < 0 || cache_rows < 0) return RING_EINVAL;
    if (!(eps >= 0.0f) || !(eps <= 3.0e38f)) return RING_EINVAL;
    if (dtype != RING_F32 && dtype != RING_BF16) return RING_EUNSUPPORTED;
    if ((D != 64 && D != 128) || Hq % Hkv) return RING_EUNSUPPORTED;
    if (rot < 0 || rot > D || rot % 16) return RING_EINVAL;
    const long long H = Hq + 2 * (long long)Hkv;
    if (H * D >= (1LL << 21)) return RING_EUNSUPPORTED;
    if (stride < H * D || stride >= (1LL << 21) || stride % 8) return RING_EINVAL;
    return RING_OK;
}

bool all16(const void* const* p, int P) {
    for (int r = 0; r < P; ++r)
        if (!p[r] || ((uintptr_t)p[r] & 15)) return false;
    return true;
}

int rope_inputs(RopeArgs& a, const void* const* qkv, const float* const* gain_q, const float* const* gain_k,
                const float* cos_sin, const int* pos, int P, int rot, long long table_rows) {
    if (!qkv || !all16(qkv, P) || !gain_q != !gain_k || !pos || ((uintptr_t)pos & 3)) return RING_EINVAL;
    if (gain_q && (!all16((const void* const*)gain_q, P) || !all16((const void* const*)gain_k, P))) return RING_EINVAL;
    if ((rot && table_rows && !cos_sin) || ((uintptr_t)cos_sin & 15)) return RING_EINVAL;
    for (int r = 0; r < P; ++r) {
        a.qkv[r] = qkv[r];
        a.gq[r] = gain_q ? gain_q[r] : nullptr;
        a.gk[r] = gain_k ? gain_k[r] : nullptr;
    }
    a.cs = cos_sin;
    a.pos = pos;
    a.P = P;
    a.rot = rot;
    return RING_OK;
}

}  // namespace
}  // namespace ringc

using namespace ringc;

extern "C" int tp_qk_norm_rope(const void* const* qkv, const float* const* gain_q, const float* const* gain_k,
                               const float* cos_sin, const int* pos, void* const* q, void* const* k, void* const* v,
                               void* const* k_cache, void* const* v_cache, const long long* slots, int P, int T, int Hq,
                               int Hkv, int D, int rot, long long table_rows, long long cache_rows, long long qkv_stride,
                               float eps, int dtype, void* stream) {
    int rc = rope_shape(P, T, Hq, Hkv, D, rot, table_rows, cache_rows, qkv_stride, eps, dtype);
    if (rc != RING_OK) return rc;
    // what has no element may have no address: slots of no token, a cache of no row
    if (!k != !v || !k_cache != !v_cache || (T && !k_cache != !slots) || ((uintptr_t)slots & 7)) return RING_EINVAL;
    if (T == 0) return RING_OK;
    RopeArgs a;
    rc = rope_inputs(a, qkv, gain_q, gain_k, cos_sin, pos, P, rot, table_rows);
    if (rc != RING_OK) return rc;
    if (!q || !all16(q, P) || (k && (!all16(k, P) || !all16(v, P))) ||
        (k_cache && cache_rows && (!all16(k_cache, P) || !all16(v_cache, P))))
        return RING_EINVAL;
    for (int r = 0; r < P; ++r) {
        a.q[r] = (unsigned short*)q[r];
        a.k[r] = k ? (unsigned short*)k[r] : nullptr;
        a.v[r] = v ? (unsigned short*)v[r] : nullptr;
        a.kc[r] = k_cache ? (unsigned short*)k_cache[r] : nullptr;
        a.vc[r] = v_cache ? (unsigned short*)v_cache[r] : nullptr;
    }
    a.slots = slots;
    a.table_rows = table_rows;
    a.cache_rows = cache_rows;
    a.stride = qkv_stride;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.eps = eps;
    const int groups = (Hq + 2 * Hkv + 512 / D - 1) / (512 / D);
    const long long items = (long long)T * groups;
    if (items >= (1LL << 31)) return RING_EUNSUPPORTED;
    const dim3 grid((unsigned)((items + 3) / 4), (unsigned)P);
    hipStream_t s = (hipStream_t)stream;
    if (dtype == RING_F32) {
        if (D == 128) hipLaunchKernelGGL((qk_rope_kernel<128, float>), grid, dim3(256), 0, s, a, groups);
        else hipLaunchKernelGGL((qk_rope_kernel<64, float>), grid, dim3(256), 0, s, a, groups);
    } else {
        if (D == 128) hipLaunchKernelGGL((qk_rope_kernel<128, unsigned short>), grid, dim3(256), 0, s, a, groups);
        else hipLaunchKernelGGL((qk_rope_kernel<64, unsigned short>), grid, dim3(256), 0, s, a, groups);
    }
    return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
}

extern "C" size_t tp_qk_norm_rope_grad_workspace_bytes(int P, int D) {
    if (P < 1 || P > RING_MAX_RANKS || (D != 64 && D != 128)) return 0;
    return kStatusBytes + (size_t)P * grad_blocks_most(P) * 2 * D * sizeof(float);
}

extern "C" int tp_qk_norm_rope_grad(const void* const* dq, const void* const* dk, const void* const* dv,
                                    const void* const* qkv, const float* const* gain_q, const float* const* gain_k,
                                    const float* cos_sin, const int* pos, void* const* dqkv, float* const* dgain_q,
                                    float* const* dgain_k, int P, int T, int Hq, int Hkv, int D, int rot,
                                    long long table_rows, long long qkv_stride, float eps, int dtype, void* ws,
                                    size_t ws_bytes, void* stream) {
    int rc = rope_shape(P, T, Hq, Hkv, D, rot, table_rows, 0, qkv_stride, eps, dtype);
    if (rc != RING_OK) return rc;
    if (gain_q && (!dgain_q || !dgain_k)) return RING_EINVAL;
    RopeGradArgs g;
    if (T) {
        rc = rope_inputs(g.f, qkv, gain_q, gain_k, cos_sin, pos, P, rot, table_rows);
        if (rc != RING_OK) return rc;
        if (!dq || !dk || !dv || !dqkv || !all16(dq, P) || !all16(dk, P) || !all16(dv, P) || !all16(dqkv, P))
            return RING_EINVAL;
    } else if (!gain_q) {
        return RING_OK;
    }
    if (gain_q && (!all16((const void* const*)dgain_q, P) || !all16((const void* const*)dgain_k, P))) return RING_EINVAL;
    if (!ws || ((uintptr_t)ws & 255) || ws_bytes < tp_qk_norm_rope_grad_workspace_bytes(P, D)) return RING_EWORKSPACE;
    hipStream_t s = (hipStream_t)stream;
    // kGradPerCu workgroups a compute unit in all, every group of head rows at
    // least one wave: at most 2^21 / 512 = 4096 groups, so kGradLeast do.
    g.groups = (Hq + 2 * Hkv + 512 / D - 1) / (512 / D);
    const long long items = (long long)T * g.groups;
    long long blocks = (kGradPerCu * dev_info().cus + P - 1) / P;
    if (blocks > (items + 3) / 4) blocks = (items + 3) / 4;
    if (blocks < (g.groups + 3) / 4) blocks = (g.groups + 3) / 4;
    if (blocks > grad_blocks_most(P)) blocks = grad_blocks_most(P);
    if (!T) blocks = 0;
    g.part = (float*)((char*)ws + kStatusBytes);
    g.status = (Status*)ws;
    g.data = WsSpan{kStatusBytes, kStatusBytes + (unsigned long long)P * blocks * 2 * D * sizeof(float)};
    g.blocks = (int)blocks;
    if (T) {
        for (int r = 0; r < P; ++r) {
            g.f.q[r] = (unsigned short*)const_cast<void*>(dq[r]);
            g.f.k[r] = (unsigned short*)const_cast<void*>(dk[r]);
            g.f.v[r] = (unsigned short*)const_cast<void*>(dv[r]);
            g.dx[r] = dqkv[r];
        }
        g.f.table_rows = table_rows;
        g.f.stride = qkv_stride;
        g.f.T = T;
        g.f.Hq = Hq;
        g.f.Hkv = Hkv;
        g.f.eps = eps;
        const dim3 grid((unsigned)blocks, (unsigned)P);
        if (dtype == RING_F32) {
            if (D == 128) hipLaunchKernelGGL((qk_rope_grad_kernel<128, float>), grid, dim3(256), 0, s, g);
            else hipLaunchKernelGGL((qk_rope_grad_kernel<64, float>), grid, dim3(256), 0, s, g);
        } else {
            if (D == 128) hipLaunchKernelGGL((qk_rope_grad_kernel<128, unsigned short>), grid, dim3(256), 0, s, g);
            else hipLaunchKernelGGL((qk_rope_grad_kernel<64, unsigned short>), grid, dim3(256), 0, s, g);
        }
        if (hipGetLastError() != hipSuccess) return RING_EHIP;
    }
    if (gain_q) {
        GainArgs w;
        w.part = g.part;
        w.blocks = (int)blocks;
        for (int r = 0; r < P; ++r) {
            w.dgq[r] = dgain_q[r];
            w.dgk[r] = dgain_k[r];
        }
        const dim3 grid((unsigned)P, 2);
        if (D == 128) hipLaunchKernelGGL(gain_sum_kernel<128>, grid, dim3(1024), 0, s, w);
        else hipLaunchKernelGGL(gain_sum_kernel<64>, grid, dim3(1024), 0, s, w);
        if (hipGetLastError() != hipSuccess) return RING_EHIP;
    }
    return RING_OK;
}
