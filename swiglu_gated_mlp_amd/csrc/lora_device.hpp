// Low-rank adapters inside the product kernels: what a row's adapter adds to the
// fp32 sums before the epilogue.
//
// Row m has adapter i = ids[m] (outside 0 .. adapters - 1: none).  With
// t = s_i (A[m] La_i), r numbers a row, its sums get  + t Lb_i.  t is computed
// first (lora_shrink_kernel), into memory as T; the sums' part t Lb_i is formed
//   - up to 16 rows, on the decode schedules with narrow groups: by the lanes that
//     hold the sums (lora_delta4; many workgroups a CU, whose other loads cover it),
//   - up to 256 rows otherwise: by a kernel of its own (lora_expand_kernel), one
//     thread per row and four columns, whatever adapters the rows have, and read
//     back in the epilogue.  In the epilogue itself a batch of decode requests,
//     each with its own adapter, is a chain of loads (7B width, 64 rows of 64
//     adapters: 130 us so, 82 us this way, 52 us without adapters),
//   - above: on the matrix units after the tile's K loop, straight into its sums, one
//     adapter of the tile's list after another (LoraTile): T's rows and Lb's columns are
//     loaded as operand fragments, zeros for rows of other adapters.
//     Tiles of more than LORA_PLACES adapters, and such with an infinity or NaN in
//     one's weights (zero times which is NaN: one request's broken adapter must not
//     reach another request's rows), add them in the epilogue, 32 rows at a time
//     (lora_block).
//
// T and Lb are laid out in chunks of 16 of the r numbers (the depth of one
// v_mfma_f32_32x32x16_bf16), ranks padded with zeros; `groups` is 2 for the gated
// product (Gate and Up have adapters of their own) and 1 for a plain projection:
//   T   up to 256 rows: [part][M][chunk][group][16] fp32, summed over the parts
//       (of the contraction).  Above: bf16 pairs t = hi + lo -- the matrix cores
//       take bf16, and two of them hold t to 2^-17, so the adapter's part is as
//       exact as the fp32 sums it joins rather than off by bf16's 2^-8 -- as
//       [block of 32 rows][chunk][group][hi, lo][lane][8]: lane l holds row l % 32,
//       numbers 8 (l / 32) + 0..7, an operand fragment as Lb's below (from rows of
//       16 numbers a fragment was 32 pieces of 32 bytes)
//   Lb  [adapter][chunk][32-column tile][group][lane][8] bf16: lane l of a tile
//       holds column l % 32, numbers 8 (l / 32) + 0..7 of the chunk, so one wave
//       load is one contiguous 1 KiB operand fragment
#pragma once

#include "device_common.hpp"

namespace swk {

// Longest adapter list of a tile (7B width, rank 32: 2100 rows of 20 requests 574 us
// with 4, 516 us with 7; rank 64, 4096 rows of 64 requests 1298 and 1328 us).
constexpr int LORA_PLACES = 7;
struct LoraNone {
    template <class... X>
    __device__ __forceinline__ LoraNone(const X&...) {}
};
constexpr int LORA_LIST = 8;     // ints of a tile's list: length, adapters

struct LoraArgs {
    const uint16_t* T;      // hi, lo
    const int* lists;       // with it, per tile of `unit` rows: length (-1: none formed), adapters
    const float* Tf;        // or the fp32 parts
    const float* delta;     // or t Lb itself, [M][groups * N]
    const uint16_t* B;      // Lb's packed part
    const int* ids;         // [M]
    int adapters;
    int chunks;             // 16-number chunks of the padded rank
    int ntiles;             // 32-column tiles of the packed Lb
    int parts;              // of Tf
    int M, N;               // rows of Tf; columns of delta
    int unit;
};

__device__ __forceinline__ const uint16_t* lora_b(const LoraArgs& la, int groups, int id, int c, int nt, int g) {
    return la.B + ((((size_t)id * la.chunks + c) * la.ntiles + nt) * groups + g) * 512;
}

__device__ __forceinline__ int lora_id(const LoraArgs& la, int m) {
    const int id = la.ids[m];
    return id >= 0 && id < la.adapters ? id : -1;
}

// t Lb of row m (adapter id >= 0), group g, columns n .. n + 3 (n a multiple of
// 4): 16 multiply-adds a column and chunk on the vector units.
template <int GROUPS>
__device__ __forceinline__ f32x4 lora_delta4(const LoraArgs& la, int m, int id, int g, int n) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < la.chunks; ++c) {
        const uint16_t* bp = lora_b(la, GROUPS, id, c, n >> 5, g) + (n & 31) * 8;
        u32x4 b[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) b[h][e] = ld16(bp + 256 * h + 8 * e);
        f32x4 t[4] = {};
        for (int s = 0; s < la.parts; ++s) {
            const f32x4* tp =
                reinterpret_cast<const f32x4*>(la.Tf + ((((size_t)s * la.M + m) * la.chunks + c) * GROUPS + g) * 16);
#pragma unroll
            for (int q = 0; q < 4; ++q) t[q] += tp[q];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    d[e] += t[2 * h + (q >> 1)][2 * (q & 1)] * __builtin_bit_cast(float, b[h][e][q] << 16);
                    d[e] += t[2 * h + (q >> 1)][2 * (q & 1) + 1] * __builtin_bit_cast(float, b[h][e][q] & 0xFFFF0000u);
                }
    }
    return d;
}

// t Lb as lora_expand_kernel left it: four columns of group g (zero past the
// matrix and for rows without adapter).
__device__ __forceinline__ f32x4 lora_read4(const LoraArgs& la, int groups, int m, int g, int n) {
    if (m >= la.M || n >= la.N) return f32x4{0.f, 0.f, 0.f, 0.f};
    return *reinterpret_cast<const f32x4*>(la.delta + ((size_t)m * groups + g) * la.N + n);
}
// The same for a wave's 32 x 32 block: rows m of each lane, the 16 columns its
// accumulators hold of the 32 from n on.
__device__ __forceinline__ void lora_read_block(f32x16& d, const LoraArgs& la, int groups, int m, int g, int n,
                                                int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const f32x4 v = lora_read4(la, groups, m, g, n + 8 * q + 4 * (lane >> 5));
#pragma unroll
        for (int e = 0; e < 4; ++e) d[4 * q + e] = v[e];
    }
}

// Adds the adapters to one 32-row block of a wave's sums: d[h] gets t Lb for output
// columns of 32-column tile nt[h] (first MFMA operand) and row m of each
// lane (lane & 31 of the block; rid its adapter, -1: none or no row).  The block's
// adapters are taken one after another; the other rows' factors are zero then, and
// where an adapter's weights hold an infinity or NaN its own rows alone take the
// result.  The order of the sums is LoraTile's, so a row's result does not depend on
// which of the two its neighbours' adapters lead to.
template <int NH, int GROUPS>
__device__ __forceinline__ void lora_block(f32x16 (&d)[NH], const LoraArgs& la, int rid, int m, const int (&nt)[NH],
                                           int lane) {
    unsigned long long pend = __ballot(rid >= 0);
    while (pend) {
        const int e = __builtin_amdgcn_readlane(rid, __builtin_ctzll(pend));
        const bool mine = rid == e;
        pend &= ~__ballot(mine);
        for (int c = 0; c < la.chunks; ++c) {
            const uint16_t* tp = la.T + ((size_t)(m >> 5) * la.chunks + c) * (GROUPS * 1024) + lane * 8;
            u32x4 w[NH], hi[NH], lo[NH];
            bool odd = false;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const int g = GROUPS == 2 ? h : 0;
                w[h] = ld16(lora_b(la, GROUPS, e, c, nt[h], g) + lane * 8);
                hi[h] = lo[h] = u32x4{0u, 0u, 0u, 0u};
                if (mine) {
                    hi[h] = ld16(tp + g * 1024);
                    lo[h] = ld16(tp + g * 1024 + 512);
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

// Adds the adapters of the row tile at m0 (its list) to a wave's sums: acc[h][i]
// holds output columns of 32-column tile nt[h] and rows 32 i .. of the tile, rid[i]
// the lane's row's adapter.  One pass per adapter and chunk: the next pass's weights
// and, across passes, the next three blocks' rows of T are in flight; rows of other
// adapters are read past the descriptor's end, which gives zeros.  Bound by the
// latency of T's and Lb's loads from the L2: 7B width, 2100 rows of one adapter of
// rank 32 496 us, 474 us with no row adapted (5 to 6 tiles of two passes a CU: 2 us a
// pass; 2.9 us with one block in flight, 3.4 us with each pass's loads started in
// it).
template <int TM, int GROUPS>
struct LoraTile {
    static constexpr int D = 4;
    static_assert(TM % D == 0, "the ring of blocks runs on across passes");
    const LoraArgs& la;
    const __attribute__((address_space(4))) int* list;   // scalar loads: an earlier launch wrote it
    __amdgpu_buffer_rsrc_t t;
    int rid[TM], nt[2], len, pitch, lane;
    int d, c, id;                 // the pass whose loads are issued next
    bf16x8 w[2], wn[2];
    u32x4 x[D][GROUPS][2];        // hi, lo

    // raw ids of the lane's rows (before the last stages: they arrive meanwhile)
    __device__ __forceinline__ LoraTile(const LoraArgs* a, int m0, int l) : la(*a), lane(l) {
        list = (const __attribute__((address_space(4))) int*)(uintptr_t)(la.lists + m0 / la.unit * LORA_LIST);
#pragma unroll
        for (int i = 0; i < TM; ++i) rid[i] = la.ids[min(m0 + 32 * i + (lane & 31), la.M - 1)];
    }
    __device__ __forceinline__ void load_block(int i) {
        const uint32_t off =
            rid[i % TM] == id ? (uint32_t)(lane * 16 + (i % TM) * pitch + c * (GROUPS * 2048)) : 0xFFFF0000u;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                x[i % D][g][q] = __builtin_amdgcn_raw_buffer_load_b128(t, off + 2048 * g + 1024 * q, 0, 0);
    }
    __device__ __forceinline__ void load_weights() {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            wn[h] = __builtin_bit_cast(bf16x8, ld16(lora_b(la, GROUPS, id, c, nt[h], GROUPS == 2 ? h : 0) + lane * 8));
    }
    // the tile's length (-1: blocks are added in the epilogue) and the first pass's loads
    __device__ __forceinline__ void begin(int m0, int nt0, int nt1) {
        nt[0] = nt0;
        nt[1] = nt1;
        len = list[0];
        if (len <= 0) return;
        // rows past the matrix repeat the last one's adapter: their T is never
        // written, nor are their outputs
        pitch = la.chunks * (GROUPS * 2048);   // bytes of a block's T
        t = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(la.T + (size_t)(m0 >> 5) * (pitch / 2)), 0,
                                              min((la.M - m0 + 31) >> 5, TM) * pitch, 0x00020000);
        d = c = 0;
        id = list[1];
        load_weights();
#pragma unroll
        for (int i = 0; i < D - 1; ++i) load_block(i);
    }
    __device__ __forceinline__ void run(f32x16 (&acc)[2][TM][1]) {
        if (len <= 0) return;
        for (bool more = true; more;) {
            w[0] = wn[0];
            w[1] = wn[1];
            int nd = d, nc = c + 1;
            if (nc == la.chunks) {
                nc = 0;
                ++nd;
            }
            more = nd < len;
            const int nid = more ? list[1 + nd] : 0;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                if (i == TM - D + 1) {   // from here on the next pass's loads (past the last: nothing)
                    d = nd;
                    c = more ? nc : 0;
                    id = nid;
                    load_weights();
                }
                load_block(i + D - 1);
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        acc[h][i][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            w[h], __builtin_bit_cast(bf16x8, x[i % D][GROUPS == 2 ? h : 0][q]), acc[h][i][0], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
};

}  // namespace swk
