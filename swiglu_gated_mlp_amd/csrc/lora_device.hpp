// Low-rank adapters inside the product kernels: what a row's adapter adds to the
// fp32 sums before the epilogue.
//
// Row m has adapter i = ids[m] (outside 0 .. adapters - 1: none).  With
// t = s_i (A[m] La_i), r numbers a row, its sums get  + t Lb_i.  The factor t is
// computed first (lora_kernels.hpp), into memory as T; here it is multiplied with
// Lb_i's columns of the output tile and added to the accumulators, so the adapted
// sums exist only in registers, like the sums themselves.
//
// T and Lb are laid out in chunks of 16 of the r numbers (the depth of one
// v_mfma_f32_32x32x16_bf16), ranks padded with zeros; `groups` is 2 for the gated
// product (Gate and Up have adapters of their own) and 1 for a plain projection:
//   T   [M][chunk][group][hi, lo][16] bf16, t = hi + lo: the matrix cores take
//       bf16, and two of them hold t to 2^-17, so the adapter's part is as exact
//       as the fp32 sums it joins rather than off by bf16's 2^-8
//   Lb  [adapter][chunk][32-column tile][group][lane][8] bf16: lane l of a tile
//       holds column l % 32, numbers 8 (l / 32) + 0..7 of the chunk, so one wave
//       load is one contiguous 1 KiB operand fragment
#pragma once

#include "device_common.hpp"

namespace swk {

struct LoraArgs {
    const uint16_t* T;
    const uint16_t* B;      // Lb's packed part
    const int* ids;         // [M]
    int adapters;
    int chunks;             // 16-number chunks of the padded rank
    int ntiles;             // 32-column tiles of the packed Lb
};

__device__ __forceinline__ const uint16_t* lora_b(const LoraArgs& la, int groups, int id, int c, int nt, int g) {
    return la.B + ((((size_t)id * la.chunks + c) * la.ntiles + nt) * groups + g) * 512;
}

__device__ __forceinline__ int lora_id(const LoraArgs& la, int m) {
    const int id = la.ids[m];
    return id >= 0 && id < la.adapters ? id : -1;
}

// t Lb of row m (adapter id >= 0), group g, columns n .. n + 3 (n a multiple of
// 4): 16 multiply-adds a column and chunk on the vector units, for the schedules
// whose lanes hold few rows (decode, the reduction of splits).
template <int GROUPS>
__device__ __forceinline__ f32x4 lora_delta4(const LoraArgs& la, int m, int id, int g, int n) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < la.chunks; ++c) {
        const uint16_t* tp = la.T + (((size_t)m * la.chunks + c) * GROUPS + g) * 32;
        const uint16_t* bp = lora_b(la, GROUPS, id, c, n >> 5, g) + (n & 31) * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 hi = ld16(tp + 8 * h), lo = ld16(tp + 16 + 8 * h);
            float t[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                t[2 * q] = __builtin_bit_cast(float, hi[q] << 16) + __builtin_bit_cast(float, lo[q] << 16);
                t[2 * q + 1] =
                    __builtin_bit_cast(float, hi[q] & 0xFFFF0000u) + __builtin_bit_cast(float, lo[q] & 0xFFFF0000u);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const u32x4 b = ld16(bp + 256 * h + 8 * e);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    d[e] += t[2 * q] * __builtin_bit_cast(float, b[q] << 16);
                    d[e] += t[2 * q + 1] * __builtin_bit_cast(float, b[q] & 0xFFFF0000u);
                }
            }
        }
    }
    return d;
}

// What the adapters add to one 32-row block of a wave's sums: d[h] is t Lb for
// output columns of 32-column tile nt[h] (first MFMA operand) and row m of each
// lane (lane & 31 of the block; rid its adapter, -1: none or no row).  The
// block's adapters are taken one after another; the other rows' factors are zero
// then, and where an adapter's weights hold an infinity or NaN (zero times which
// is NaN) its own rows alone take the result: one request's broken adapter cannot
// reach another request's rows.  The sums the block's accumulators hold are not
// touched here: a loop around the matrix instructions that carried them would
// move all of them through VGPRs.
template <int NH, int GROUPS>
__device__ __forceinline__ void lora_block(f32x16 (&d)[NH], const LoraArgs& la, int rid, int m, const int (&nt)[NH],
                                           int lane) {
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int r = 0; r < 16; ++r) d[h][r] = 0.0f;
    unsigned long long pend = __ballot(rid >= 0);
    while (pend) {
        const int e = __builtin_amdgcn_readlane(rid, __builtin_ctzll(pend));
        const bool mine = rid == e;
        pend &= ~__ballot(mine);
        for (int c = 0; c < la.chunks; ++c) {
            const uint16_t* tp = la.T + ((size_t)m * la.chunks + c) * (GROUPS * 32) + 8 * (lane >> 5);
            u32x4 w[NH], hi[NH], lo[NH];
            bool odd = false;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const int g = GROUPS == 2 ? h : 0;
                w[h] = ld16(lora_b(la, GROUPS, e, c, nt[h], g) + lane * 8);
                hi[h] = lo[h] = u32x4{0u, 0u, 0u, 0u};
                if (mine) {
                    hi[h] = ld16(tp + g * 32);
                    lo[h] = ld16(tp + g * 32 + 16);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)   // exponent bits all set
                    odd = odd || (w[h][q] & 0x7F80u) == 0x7F80u || (w[h][q] & 0x7F800000u) == 0x7F800000u;
            }
            const bool select = __ballot(odd) != 0;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                f32x16 v = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    __builtin_bit_cast(bf16x8, w[h]), __builtin_bit_cast(bf16x8, hi[h]), d[h], 0, 0, 0);
                v = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w[h]),
                                                            __builtin_bit_cast(bf16x8, lo[h]), v, 0, 0, 0);
                if (select) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) d[h][r] = mine ? v[r] : d[h][r];
                } else {
                    d[h] = v;
                }
            }
        }
    }
}

}  // namespace swk
