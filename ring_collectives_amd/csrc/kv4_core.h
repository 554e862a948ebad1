// kv4_core.h -- what the kernels of the 4-bit cache share: where things lie in
// a page, and the conversions.
//
// gfx950 converts between bf16 and e2m1 codes two at a time under a power-of-two
// scale, rounding to the nearest code (halfway: the even one) and saturating,
// exactly as the format says for every scale byte: the scale operand is the
// fp32 number with the byte as its exponent field, and 255 there makes NaN of
// every code.
#pragma once

#include "attn_internal.h"
#include "tp_search.h"

namespace ringc {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// A page of one head: key codes, value codes, key scales, value scales.
template <int D> struct Kv4Page {
    static constexpr int kRow = D / 2, kScales = D / 32;       // bytes of a row's codes and scales
    int shift;                                                 // of the page size
    __device__ __forceinline__ int bytes() const { return (2 * (kRow + kScales)) << shift; }
    __device__ __forceinline__ int codes(int kv, int i) const { return (kv << shift) * kRow + i * kRow; }
    __device__ __forceinline__ int scales(int kv, int i) const { return (2 * kRow << shift) + (kv << shift) * kScales + i * kScales; }
};

__device__ __forceinline__ float kv4_scale(unsigned byte) { return __builtin_bit_cast(float, byte << 23); }

// Eight codes of a word as bf16.
__device__ __forceinline__ bf16x8 kv4_values(unsigned codes, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

inline bool kv4_page_ok(int page_size) { return page_size >= 16 && !(page_size & (page_size - 1)) && page_size <= (1 << 16); }

}  // namespace ringc
