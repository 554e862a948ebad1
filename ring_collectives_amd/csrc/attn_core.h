// attn_core.h -- what the attention kernels share: the LDS placement of a tile
// of rows, the direct global->LDS loads that fill it, the two kinds of MFMA
// fragment reads from it, and the search of a tile's prompt.
//
// Every product runs on v_mfma_f32_32x32x16_bf16 with the streamed operand (a
// tile of key, value, query or gradient rows in LDS) as A and the stationary
// one (32 rows per wave, in registers) as B:
//   S^T = K Q^T       A = the rows of K as they lie, B = rows of Q
//   O^T += V^T P^T    A = V read transposed,        B = P^T, the accumulators
//                     of S^T themselves, rounded to bf16
// Lane l of a wave owns column n = l % 32 of every product (one query, or one
// key in the pass over dK and dV), so softmax statistics are one value per
// lane and the row operations never leave the lane but for one exchange with
// lane l ^ 32, which holds the other half of the column's rows.
#pragma once

#include "gemm_core.h"
#include "global_ptr.h"

namespace ringc {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Geometry of rows of D bf16 values in LDS: 2 D bytes each, unpadded, in C
// chunks of 16 bytes.  Chunk c of row r is stored at chunk c ^ swz(r).  With
// these swizzles the 16 rows that a row-fragment read touches in one LDS cycle
// and the 4 rows x 32 columns of a transposed read fall on distinct banks.
template <int D> struct Rows {
    static_assert(D == 64 || D == 128, "head width");
    static constexpr int RB = 2 * D;             // bytes of a row
    static constexpr int C = D / 8;              // 16-byte chunks of a row
    static constexpr int RPI = 64 / C;           // rows filled by one load instruction (1 KiB)
    static constexpr int KK = D / 16;            // MFMA k-steps over a row
    static constexpr int DB = D / 32;            // 32-wide blocks of a row
    static __device__ __forceinline__ int swz(int r) {
        return D == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : ((r & 2) << 1) | ((r >> 2) & 3);
    }
};

// A view of `rows` rows of D values that start `row_bytes` apart (none for
// rows <= 0, at most `most`): it ends with the last row's last value.
template <int D>
__device__ __forceinline__ rsrc_t rows_view(const unsigned short* base, long long rows, int most, unsigned row_bytes) {
    const long long n = rows < 0 ? 0 : rows < most ? rows : most;
    return tile_view(base, n ? (n - 1) * (long long)row_bytes + Rows<D>::RB : 0);
}

// The direct loads of one wave into tiles of ROWS rows shared by NW waves:
// wave w issues instructions w J .. w J + J - 1, each filling RPI rows.  Rows
// past the view's end are filled with zeros by the hardware's bounds check.
template <int D, int ROWS, int NW> struct TileLoad {
    static constexpr int J = ROWS / Rows<D>::RPI / NW;
    static_assert(J * NW * Rows<D>::RPI == ROWS, "load split");
    unsigned voff[J];       // byte offset of this lane's chunk in instruction j, without the tile's start
    int first;              // LDS byte of this wave's first instruction within the tile
    __device__ __forceinline__ void init(int lane, int wave, unsigned row_bytes) {
        first = wave * J * 1024;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int r = (wave * J + j) * Rows<D>::RPI + lane / Rows<D>::C;
            voff[j] = (unsigned)r * row_bytes + (unsigned)(((lane % Rows<D>::C) ^ Rows<D>::swz(r)) * 16);
        }
    }
    // The tile at LDS byte `at` from `rows` rows (at most ROWS of them) on from
    // base.  For the device pass alone: buffer views have no host type, and the
    // host pass silently leaves out all but one of the kernel templates that
    // instantiate a member naming one.
    __device__ __forceinline__ void issue(const unsigned short* base, long long rows, unsigned row_bytes,
                                          unsigned short* lds, int at) const {
#ifdef __HIP_DEVICE_COMPILE__
        const rsrc_t view = rows_view<D>(base, rows, ROWS, row_bytes);
#pragma unroll
        for (int j = 0; j < J; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(view, lds_at(lds, (unsigned)(at + first + j * 1024)), 16, voff[j],
                                                     0, 0, POL_PLAIN);
#endif
    }
};

// `n` floats (at most 64) straight into LDS at byte `at`, one per lane, zeros
// past them.
__device__ __forceinline__ void load_floats(const float* p, int n, unsigned short* lds, int at, int lane) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(tile_view(p, n * 4), lds_at(lds, (unsigned)at), 4, (unsigned)lane * 4, 0, 0,
                                             POL_PLAIN);
}

// Fragment reads from a tile at byte `at` of LDS (a multiple of 4096).
template <int D> struct Frags {
    unsigned row0;          // row fragment: row l % 32, chunk l / 32
    unsigned tr[2];         // transposed: rows 4 (l / 32) + .., and the same 8 rows further down
    __device__ __forceinline__ void init(int lane) {
        typedef Rows<D> R;
        row0 = (unsigned)((lane & 31) * R::RB + (((lane >> 5) ^ R::swz(lane & 31)) * 16));
        const int g = lane >> 4, i = lane & 15;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int r = 8 * t + 4 * (g >> 1) + (i >> 2);
            tr[t] = (unsigned)(r * R::RB + (((2 * (g & 1) + ((i & 3) >> 1)) ^ R::swz(r)) * 16) + (i & 1) * 8);
        }
    }
    // A[m = row 32 b + l % 32][k = 16 kk + 8 (l / 32) + t]
    __device__ __forceinline__ bf16x8 rows(const unsigned short* lds, int at, int b, int kk) const {
        return *(const bf16x8*)((const char*)lds + at + (row0 ^ (unsigned)(kk * 32)) + b * 32 * Rows<D>::RB);
    }
    // A[m = column 32 db + l % 32][k]: rows 16 ks + 4 (l / 32) + {0 .. 3} for
    // t = 0 .. 3 and 8 rows further for t = 4 .. 7, the order in which the
    // accumulators of a product hold its rows.
    __device__ __forceinline__ bf16x8 cols(unsigned short* lds, int at, int db, int ks) const {
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const unsigned o = (unsigned)(at + ks * 16 * Rows<D>::RB);
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)lds_at(lds, (tr[0] ^ (unsigned)(db * 64)) + o));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)lds_at(lds, (tr[1] ^ (unsigned)(db * 64)) + o));
        const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        return __builtin_bit_cast(bf16x8, v);
    }
};

// Accumulators 8 ks .. 8 ks + 7 of a 32 x 32 block, rounded to bf16 (nearest
// even), as the B operand of k-step ks of the next product.
__device__ __forceinline__ bf16x8 round8(const f32x16& x, int ks) {
    typedef float f32x8 __attribute__((ext_vector_type(8)));
    const f32x8 y = {x[8 * ks], x[8 * ks + 1], x[8 * ks + 2], x[8 * ks + 3],
                     x[8 * ks + 4], x[8 * ks + 5], x[8 * ks + 6], x[8 * ks + 7]};
    return __builtin_convertvector(y, bf16x8);
}

// Row of accumulator v of lane half h within its 32 x 32 block.
__device__ __forceinline__ int acc_row(int v, int h) { return 8 * (v / 4) + 4 * h + v % 4; }

// The lower and the upper half's value of x, in both halves.  The two operands
// of the swap have to differ for the compiler: it takes the results of
// swapping a register with itself for equal.
struct Halves {
    float lo, hi;
};
__device__ __forceinline__ Halves both_halves(float x) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    unsigned w = u;
    asm("" : "+v"(w));
    const auto r = __builtin_amdgcn_permlane32_swap(u, w, false, false);
    return Halves{__builtin_bit_cast(float, (unsigned)r[0]), __builtin_bit_cast(float, (unsigned)r[1])};
}
__device__ __forceinline__ float max_halves(float x) {
    const Halves h = both_halves(x);
    return fmaxf(h.lo, h.hi);
}
__device__ __forceinline__ float sum_halves(float x) {
    const Halves h = both_halves(x);
    return h.lo + h.hi;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Inclusive running sum over the wave's lanes (VALU only: four shifts within
// rows of 16 lanes, then the last lane of rows 0 and 2, and of row 1, added on).
__device__ __forceinline__ int wave_scan(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
    return x;
}

// The prompt and tile of work slot `slot`, where prompt b has
// ceil(len_b * per / rows) tiles, len_b = cu[b + 1] - cu[b] clamped to the
// `total` rows there are, and the prompt's range of the other tensor's rows
// likewise (lengths at least 0).  Every lane looks at one prompt, so 64 of
// them cost one trip to memory.  Returns false past the last tile.
struct PromptTile {
    int tile, tiles;        // of the prompt
    int lo, n, lo2, n2;     // its rows, and the other tensor's
};
__device__ __forceinline__ int clamp_cu(int x, int total) { return x < 0 ? 0 : x > total ? total : x; }
__device__ __forceinline__ bool find_tile(const int* cu, const int* cu2, int B, int total, int total2, int per, int rows,
                                          int slot, int lane, PromptTile& t) {
    int before = 0;
    for (int b0 = 0; b0 < B; b0 += 64) {
        int lo = 0, len = 0, lo2 = 0, len2 = 0;
        if (b0 + lane < B) {
            const int x0 = cu[b0 + lane], x1 = cu[b0 + lane + 1], y0 = cu2[b0 + lane], y1 = cu2[b0 + lane + 1];
            lo = clamp_cu(x0, total);
            len = clamp_cu(x1, total) - lo;
            lo2 = clamp_cu(y0, total2);
            len2 = clamp_cu(y1, total2) - lo2;
        }
        if (len < 0) len = 0;
        const int n = (int)(((unsigned)len * (unsigned)per + (unsigned)(rows - 1)) / (unsigned)rows);
        const int sum = wave_scan(n);
        const unsigned long long past = __ballot(before + sum > slot);
        if (past) {
            const int at = __builtin_ctzll(past);
            t.tiles = __builtin_amdgcn_readlane(n, at);
            t.tile = slot - (before + __builtin_amdgcn_readlane(sum, at) - t.tiles);
            t.lo = __builtin_amdgcn_readlane(lo, at);
            t.n = __builtin_amdgcn_readlane(len, at);
            t.lo2 = __builtin_amdgcn_readlane(lo2, at);
            const int n2 = __builtin_amdgcn_readlane(len2, at);
            t.n2 = n2 < 0 ? 0 : n2;
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// Accumulators 4 j .. 4 j + 7 (j even) of the lane's column of a 32 x 32 block,
// times f, as bf16: the two halves of the wave trade, so that each lane has 8
// contiguous values, 8 (j + half) and on.
__device__ __forceinline__ u32x4 round_chunk(const f32x16& x, int j, float f) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    u32x4 y;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        // values 8 j + 4 half + 2 e, + 1 and the same of j + 1: of the pair
        // the lower half keeps j's and gets the upper's, the upper half
        // j + 1's
        const f32x2 lo = {x[4 * j + 2 * e] * f, x[4 * j + 2 * e + 1] * f};
        const f32x2 hi = {x[4 * j + 4 + 2 * e] * f, x[4 * j + 5 + 2 * e] * f};
        const auto r = __builtin_amdgcn_permlane32_swap(
            __builtin_bit_cast(unsigned, __builtin_convertvector(lo, bf16x2)),
            __builtin_bit_cast(unsigned, __builtin_convertvector(hi, bf16x2)), false, false);
        y[e] = r[0];
        y[2 + e] = r[1];
    }
    return y;
}

// Store the lane's column of a 32 x 32 block of accumulators, times f, as bf16
// to p on, 16 bytes a lane.
__device__ __forceinline__ void store_block(unsigned short* p, const f32x16& x, float f, int half, bool live) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        const u32x4 y = round_chunk(x, j, f);
        if (live) *(u32x4*)(p + 8 * (j + half)) = y;
    }
}
template <int D, class Acc>
__device__ __forceinline__ void store_column(unsigned short* p, const Acc& x, float f, int half, bool live) {
#pragma unroll
    for (int db = 0; db < Rows<D>::DB; ++db) store_block(p + 32 * db, x[db], f, half, live);
}

// The same by whole rows: the wave's 32 columns go through its own 32 rows of
// LDS at byte `at`, and each store instruction writes full rows of memory,
// where store_column's writes 32 bytes of each of 32 rows.  Full lines need not
// wait in the L2s to be filled, so they are stored nontemporally.  off: the
// element offset from p of this lane's column's row, n: the rows there are.
template <int D, class Acc>
__device__ __forceinline__ void store_rows(unsigned short* p, const Acc& x, float f, unsigned off, int n, unsigned short* lds,
                                           int at, int lane) {
    typedef Rows<D> R;
    const int half = lane >> 5, r = lane & 31;
    char* w = (char*)lds + at;
#pragma unroll
    for (int db = 0; db < R::DB; ++db)
#pragma unroll
        for (int j = 0; j < 4; j += 2)
            *(u32x4*)(w + r * R::RB + (((4 * db + j + half) ^ R::swz(r)) * 16)) = round_chunk(x[db], j, f);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32 / R::RPI; ++i) {
        const int t = i * R::RPI + lane / R::C, c = lane % R::C;
        const u32x4 y = *(const u32x4*)(w + t * R::RB + ((c ^ R::swz(t)) * 16));
        const unsigned to = (unsigned)__shfl((int)off, t);
        if (t < n) __builtin_nontemporal_store(y, (u32x4*)(p + to + 8 * c));
    }
}

// Arguments of the packed-prompt kernels (per-rank pointers by value).
struct PromptArgs {
    const unsigned short *q[RING_MAX_RANKS], *k[RING_MAX_RANKS], *v[RING_MAX_RANKS];
    const int *cu_q, *cu_k;
    long long q_stride, k_stride, v_stride;   // elements from a token's row to the next
    int B, Tq, Tk, P, Hq, Hkv, causal;
    float c;                                   // scale * log2(e)
};

// A kernel's scalar arguments, read in one trip to its argument memory (its
// rank's pointers are another): left alone, the compiler reads each where it
// is first used, five or six trips one after the other before the first load
// of data (5 prompts of 80 tokens 6.6 us so, 6.2 in two trips).
struct PromptSizes {
    const int *cu_q, *cu_k;
    long long q_stride, k_stride, v_stride;
    int B, Tq, Tk, P, Hq, Hkv, causal, slots;
    float c;
};
__device__ __forceinline__ PromptSizes read_sizes(const PromptArgs& p, int slots) {
    auto cq = (Global<const int>)p.cu_q, ck = (Global<const int>)p.cu_k;
    PromptSizes z = {nullptr, nullptr, p.q_stride, p.k_stride, p.v_stride, p.B, p.Tq, p.Tk, p.P, p.Hq, p.Hkv, p.causal, slots, p.c};
    asm volatile("" : "+s"(cq), "+s"(ck), "+s"(z.B), "+s"(z.Tq), "+s"(z.Tk), "+s"(z.P), "+s"(z.Hq), "+s"(z.Hkv), "+s"(z.causal),
                      "+s"(z.slots));
    z.cu_q = (const int*)cq;
    z.cu_k = (const int*)ck;
    return z;
}

// Work units (rank, key head) vary fastest over the launch, eight at a time:
// workgroups go to the eight XCDs in turn, so one unit's keys and values stay
// with one XCD's L2 and the tiles of one unit run there together.
__device__ __forceinline__ void unit_slot(int units, int slots, int block, int& unit, int& slot) {
    const int full = units / 8 * 8;
    const int g = block / (8 * slots);                     // group of eight units
    if (g * 8 < full) {
        const int i = block - g * 8 * slots;
        unit = g * 8 + i % 8;
        slot = i / 8;
    } else {
        const int i = block - full * slots, n = units - full;
        unit = full + i % n;
        slot = i / n;
    }
}

}  // namespace ringc
