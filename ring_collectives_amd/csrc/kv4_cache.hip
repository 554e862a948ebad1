// kv4_cache.hip -- keys and values to the 4-bit cache, and back.
//
// A block of 32 values x with the largest magnitude m has the scale 2^e, e the
// least with m <= 7 * 2^e: m's exponent less 2, one more where m's mantissa is
// above 1.75, both read off m's bits, and 125 at most (bf16 ends below 6 * 2^126).
// Codes are the nearest of the format's numbers to x / 2^e.
//
// Memory bounds both.  Four lanes hold a block, 16 bytes of bf16 each, which
// are four bytes of codes; a wave takes one head of kTokens tokens, keys or
// values, so what it writes lies together where the tokens' slots do, and its
// loads are in flight together.  16381 tokens of 4 heads of 64 on 4 ranks, 67 MB
// of bf16 and 18 of cache: written in 20 us, read in 15, 4.2 and 5.7 TB/s with
// the bf16 rows past the caches (both 41 us with them, 35 so).  32 tokens take 4
// us each, an empty launch and three trips to memory.
#include "kv4_core.h"

#include <hip/hip_runtime.h>

namespace ringc {
namespace {

constexpr int kTokens = 16;            // of a wave

struct Kv4Args {
    const unsigned short* in[2][RING_MAX_RANKS];       // rows of keys, of values
    unsigned short* out[2][RING_MAX_RANKS];
    char* cache[RING_MAX_RANKS];
    const long long* slots;
    long long stride[2];
    int T, Hkv, shift, pages, tiles;                   // tiles of kTokens tokens
};

// Where a wave's work lies: rank, keys or values, head and tile.
struct Kv4Work {
    int tile, head, kv, rank;
    __device__ __forceinline__ Kv4Work(const Kv4Args& a, unsigned i) {
        tile = (int)(i % (unsigned)a.tiles);
        i /= (unsigned)a.tiles;
        head = (int)(i % (unsigned)a.Hkv);
        i /= (unsigned)a.Hkv;
        kv = (int)(i & 1);
        rank = (int)(i >> 1);
    }
};

// The scale byte of a block whose largest magnitude has the bits m.
__device__ __forceinline__ unsigned scale_byte(unsigned m) {
    const int e = (int)((m + 0x1f) >> 7) - 2;
    return m >= 0x7f80u ? 255u : e < 1 ? 1u : e > 252 ? 252u : (unsigned)e;
}

// (by value: of a vector's element itself, __builtin_bit_cast takes element 0)
__device__ __forceinline__ bf16x2 bf16_pair(unsigned x) { return __builtin_bit_cast(bf16x2, x); }

template <int D, bool WRITE> __global__ __launch_bounds__(256) void kv4_kernel(Kv4Args a, unsigned works) {
    constexpr int L = D / 8, kRows = 64 / L, kSteps = kTokens / kRows;      // lanes of a row, rows of a step
    const unsigned w = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (w >= works) return;
    const Kv4Work k(a, __builtin_amdgcn_readfirstlane(w));
    const int lane = threadIdx.x & 63, i = lane % L;
    const Kv4Page<D> page{a.shift};
    long long at[kSteps];              // this lane's rows in the cache, -1: none
    int row[kSteps];
    const long long end = (long long)a.pages << a.shift;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int t = k.tile * kTokens + s * kRows + lane / L;
        const long long slot = t < a.T ? a.slots[t] : -1;
        row[s] = (int)(slot & ((1 << a.shift) - 1));
        at[s] = slot >= 0 && slot < end ? ((slot >> a.shift) * a.Hkv + k.head) * page.bytes() : -1;
    }
    char* cache = a.cache[k.rank];
    const long long stride = a.stride[k.kv];
    if (WRITE) {
        const unsigned short* in = a.in[k.kv][k.rank] + (long long)k.head * D + i * 8;
        u32x4 x[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int t = k.tile * kTokens + s * kRows + lane / L;
            x[s] = __builtin_nontemporal_load((const u32x4*)(in + (t < a.T ? t : 0) * stride));
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            unsigned m = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const unsigned y = x[s][e] & 0x7fff7fffu, lo = y & 0xffffu, hi = y >> 16;
                m = m > lo ? m : lo;
                m = m > hi ? m : hi;
            }
            const unsigned n = (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, false);     // lanes 1 0 3 2
            m = m > n ? m : n;
            const unsigned o = (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x4e, 0xf, 0xf, false);     // lanes 2 3 0 1
            m = m > o ? m : o;
            const unsigned byte = scale_byte(m);
            const float f = kv4_scale(byte == 255 ? 127u : byte);
            unsigned c = 0;
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair(x[s][0]), f, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair(x[s][1]), f, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair(x[s][2]), f, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair(x[s][3]), f, 3);
            if (at[s] >= 0) {
                *(unsigned*)(cache + at[s] + page.codes(k.kv, row[s]) + 4 * i) = c;
                if (i % 4 == 0) cache[at[s] + page.scales(k.kv, row[s]) + i / 4] = (char)byte;
            }
        }
    } else {
        unsigned c[kSteps], f[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            c[s] = f[s] = 0;
            if (at[s] >= 0) {
                c[s] = *(const unsigned*)(cache + at[s] + page.codes(k.kv, row[s]) + 4 * i);
                f[s] = (unsigned char)cache[at[s] + page.scales(k.kv, row[s]) + i / 4];
            }
        }
        unsigned short* out = a.out[k.kv][k.rank] + (long long)k.head * D + i * 8;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int t = k.tile * kTokens + s * kRows + lane / L;
            if (t < a.T) __builtin_nontemporal_store(kv4_values(c[s], kv4_scale(f[s])), (bf16x8*)(out + t * stride));
        }
    }
}

// Shared checks and launch; in and out as the call has them.
int kv4_run(bool write, const void* const* k, const void* const* v, const void* const* cache, const long long* slots, int P,
            int T, int Hkv, int D, int page_size, int pages, long long k_stride, long long v_stride, void* stream) {
    if (P < 1 || P > RING_MAX_RANKS || T < 0 || Hkv < 1 || pages < 0) return RING_EINVAL;
    if (!kv4_page_ok(page_size) || (D != 64 && D != 128) || (long long)Hkv * D >= kMaxRow || (long long)pages * page_size >= (1LL << 31))
        return RING_EUNSUPPORTED;
    if (!row_stride_ok(k_stride, Hkv, D) || !row_stride_ok(v_stride, Hkv, D)) return RING_EINVAL;
    if (T == 0) return RING_OK;
    if (!k || !v || !cache || !slots || ((uintptr_t)slots & 7)) return RING_EINVAL;
    Kv4Args a;
    for (int r = 0; r < P; ++r) {
        if (!k[r] || !v[r] || (pages && !cache[r])) return RING_EINVAL;
        if (((uintptr_t)k[r] | (uintptr_t)v[r] | (uintptr_t)cache[r]) & 15) return RING_EINVAL;
        a.in[0][r] = (const unsigned short*)k[r];
        a.in[1][r] = (const unsigned short*)v[r];
        a.out[0][r] = (unsigned short*)const_cast<void*>(k[r]);
        a.out[1][r] = (unsigned short*)const_cast<void*>(v[r]);
        a.cache[r] = (char*)const_cast<void*>(cache[r]);
    }
    a.slots = slots;
    a.stride[0] = k_stride;
    a.stride[1] = v_stride;
    a.T = T;
    a.Hkv = Hkv;
    a.shift = 0;
    while ((1 << a.shift) < page_size) ++a.shift;
    a.pages = pages;
    a.tiles = (T + kTokens - 1) / kTokens;
    const long long works = 2LL * P * Hkv * a.tiles;
    if (works >= (1LL << 31)) return RING_EUNSUPPORTED;
    const dim3 grid((unsigned)((works + 3) / 4)), block(256);
    hipStream_t s = (hipStream_t)stream;
    if (write) {
        if (D == 128) hipLaunchKernelGGL((kv4_kernel<128, true>), grid, block, 0, s, a, (unsigned)works);
        else hipLaunchKernelGGL((kv4_kernel<64, true>), grid, block, 0, s, a, (unsigned)works);
    } else {
        if (D == 128) hipLaunchKernelGGL((kv4_kernel<128, false>), grid, block, 0, s, a, (unsigned)works);
        else hipLaunchKernelGGL((kv4_kernel<64, false>), grid, block, 0, s, a, (unsigned)works);
    }
    return hipGetLastError() == hipSuccess ? RING_OK : RING_EHIP;
}

}  // namespace
}  // namespace ringc

using namespace ringc;

extern "C" size_t kv4_page_bytes(int Hkv, int D, int page_size) {
    if (Hkv < 1 || (D != 64 && D != 128) || (long long)Hkv * D >= kMaxRow || !kv4_page_ok(page_size)) return 0;
    return (size_t)Hkv * page_size * (D + D / 16);
}

extern "C" int tp_kv4_write(const void* const* k, const void* const* v, void* const* cache, const long long* slots, int P,
                            int T, int Hkv, int D, int page_size, int pages, long long k_stride, long long v_stride,
                            void* stream) {
    return kv4_run(true, k, v, (const void* const*)cache, slots, P, T, Hkv, D, page_size, pages, k_stride, v_stride, stream);
}

extern "C" int tp_kv4_read(const void* const* cache, const long long* slots, void* const* k, void* const* v, int P, int T,
                           int Hkv, int D, int page_size, int pages, long long k_stride, long long v_stride, void* stream) {
    return kv4_run(false, (const void* const*)k, (const void* const*)v, cache, slots, P, T, Hkv, D, page_size, pages, k_stride,
                   v_stride, stream);
}
