// Int8 products of up to some thousand rows: small row tiles, the contraction split over
// workgroups, and as many loads in flight as registers and LDS hold.
//
// Of few rows a product is bound by reading its weights once (7B width, 128 rows: 136 MB
// against 35 GOP, which the matrix cores do in a third of the time), and a CU reaches
// its share of HBM's rate only with some 50 KB in flight.  So
//  - a workgroup takes BM rows and WAVES x WT blocks of 32 packed weight rows, and a
//    part of the contraction, such that all CUs have about as much to do;
//  - the activations go through a ring of NBUF stages (128 k) in LDS, the weights
//    straight to registers (each is needed by one wave), both NBUF - 1 stages ahead;
//  - parts leave their int32 sums in the lanes' own order (1 KiB runs), and a second
//    launch adds them: whole numbers, so in any order the same.
// Of many rows and a short contraction it is bound by what follows the products (scales,
// SiLU, stores): there two or three workgroups share a CU, and one's end overlaps the
// next's loads and products (see NarrowTile).
// WT 2: a wave has the Gate and the Up block of the same 32 columns (or, GEMM, columns
// 128 apart of one weight).  WT 1: one block; the fused product's holds the Gate and Up
// rows of 16 columns, so that a lane has both sums of a column.
// ONCE: weights that no or few other row tiles read are loaded non-temporally: they
// then displace nothing from the caches, and where these hold another kernel's outputs
// nothing waits for those to be written back.  us after 1 GB was written / after the
// same kernel on other weights: fused at 7B width 33 rows 49 -> 27 / 27 -> 24, 128 rows
// 52 -> 35 / 31 -> 30, at 72B width 131 -> 81 / 93 -> 79, one weight of 7B width, 512
// rows in four tiles 56 -> 50 / 44 -> 44; but five tiles of 64 rows (one weight, K=4096
// N=11008) 37 -> 34 / 28 -> 30, and a product whose 9 MB of weights stay in the
// last-level cache (0.5B width, 256 rows) 12.0 -> 11.7 / 6.9 -> 8.4.
#pragma once

#include "fused_kernels.hpp"

#include <utility>

namespace swq {

using namespace swk;

struct NarrowArgs {
    const uint8_t* A;      // [M,K] int8
    const uint8_t* W;      // packed
    uint16_t* Y;           // [M,N]
    const float *sa, *s1, *s2;
    int* part;             // splits > 1: the parts' sums, [split][tile][block][quad][lane][4]
    int M, K, N;
    int KB;                // ceil(K / 128)
    int units;             // waves' shares of the columns: 32, WT 2 GEMM 2 x 32, PAIR 16
    int tiles_m, groups;   // row tiles, groups of WAVES units
    int splits, kb_per_split;
};

template <int BM_, int WAVES_, int WT_, int NBUF_, bool GEMM_, bool ONCE_>
struct Narrow {
    static constexpr int BM = BM_, WAVES = WAVES_, WT = WT_, NBUF = NBUF_;
    static constexpr bool GEMM = GEMM_, ONCE = ONCE_;
    static constexpr int TM = BM / 32;
    static constexpr int BLOCKS = WAVES * WT * TM;   // 32 x 32 blocks of a tile
    static constexpr bool PAIR = !GEMM && WT == 1;   // Gate and Up rows of 16 columns in a block
};

template <int... Q, class F>
__device__ __forceinline__ void each(std::integer_sequence<int, Q...>, F&& f) {
    (f(std::integral_constant<int, Q>{}), ...);
}
template <int N>
using Upto = std::make_integer_sequence<int, N>;

// First column of block t of unit u.
template <class P>
__device__ __forceinline__ int narrow_column(int u, int t) {
    if constexpr (P::GEMM && P::WT == 2) return (u >> 2) * PACK_ROWS + (u & 3) * 32 + PACK_BN * t;
    else return (P::PAIR ? 16 : 32) * u;
}

// The columns' scales of a block, as its sums lie in the lanes (PAIR: of W1 for q = 0,
// 1, of W2 for 2, 3).
template <class P>
__device__ __forceinline__ void narrow_scales(const NarrowArgs& p, int u, int t, int lane, f32x4 (&c)[4]) {
    const int n = narrow_column<P>(u, t) + 4 * (lane >> 5);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (P::PAIR) c[q] = scales4(q < 2 ? p.s1 : p.s2, n + 8 * (q & 1), p.N);
        else c[q] = scales4(P::GEMM || t == 0 ? p.s1 : p.s2, n + 8 * q, p.N);
    }
}

// Block at rows m0 + .., columns n + .. : scaled, finished, stored.
__device__ __forceinline__ void narrow_store(uint16_t* Y, int M, int N, int m0, int n, int lane, const float (&v)[16]) {
    unsigned d[4][2];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int w = 0; w < 2; ++w) d[q][w] = pack2(v[4 * q + 2 * w], v[4 * q + 2 * w + 1]);
    u32x4 out[2];
    block_to_rows(d, out);
    const int col = n + 8 * (2 * ((lane >> 4) & 1) + (lane >> 5));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = m0 + 16 * h + (lane & 15);
        if (row < M && col < N) *reinterpret_cast<u32x4*>(Y + (size_t)row * N + col) = out[h];
    }
}
template <class P>
__device__ __forceinline__ void narrow_finish(const NarrowArgs& p, int u, int t, int m0, int lane, const i32x16& x,
                                              const i32x16& y, const f32x4 (&cx)[4], const f32x4 (&cy)[4],
                                              float row) {
    if constexpr (P::PAIR) {
        unsigned d[2][2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float v[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 4 * q + 2 * w + e;
                    v[e] = silu_f(scaled(x[i], cx[q][2 * w + e], row)) * scaled(x[i + 8], cx[q + 2][2 * w + e], row);
                }
                d[q][w] = pack2(v[0], v[1]);
            }
        // columns 4 (l >> 5) + 0 .. 3 and the same + 8 to 8 (l >> 5) + 0 .. 7
        swap32(d[0][0], d[1][0]);
        swap32(d[0][1], d[1][1]);
        const int m = m0 + (lane & 31), n = narrow_column<P>(u, 0) + 8 * (lane >> 5);
        if (m < p.M && n < p.N)
            *reinterpret_cast<u32x4*>(p.Y + (size_t)m * p.N + n) = u32x4{d[0][0], d[0][1], d[1][0], d[1][1]};
        return;
    }
    float v[16];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[4 * q + e] = scaled(x[4 * q + e], cx[q][e], row);
            if constexpr (!P::GEMM) v[4 * q + e] = silu_f(v[4 * q + e]) * scaled(y[4 * q + e], cy[q][e], row);
        }
    narrow_store(p.Y, p.M, p.N, m0, narrow_column<P>(u, t), lane, v);
}

template <class P>
__global__ __launch_bounds__(64 * P::WAVES) void narrow_kernel(NarrowArgs p) {
    constexpr int BM = P::BM, WAVES = P::WAVES, WT = P::WT, NBUF = P::NBUF, TM = P::TM;
    constexpr int A_ALL = BM / 8;                  // 1 KiB loads of activations a stage,
    constexpr int A_INS = (A_ALL + WAVES - 1) / WAVES;   // of them a wave's (past the last: into a spare slot)
    constexpr int LOADS = A_INS + 4 * WT;          // loads per wave and stage
    constexpr int LPS = (LOADS + 3) / 4;           // of them per sub-step
    constexpr int LATE = LOADS < 3 * LPS ? LOADS : 3 * LPS;   // in the first three sub-steps
    constexpr int ASTAGE = BM * 128;               // bytes
    constexpr bool SPARE = A_ALL % WAVES != 0;
    static_assert(BM % 32 == 0, "tile");
    static_assert(NBUF >= 3 && NBUF * ASTAGE <= 163840, "LDS");
    static_assert((NBUF - 3) * LOADS + LATE <= 63 && (NBUF - 2) * LOADS <= 63, "vmcnt range");
    __shared__ __attribute__((aligned(16))) uint8_t smem[NBUF * ASTAGE + (SPARE ? 1024 : 0)];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // row tiles of a column group next to each other (they read the same weights), then
    // the groups of a part of the contraction (they read the same activations)
    const int logical = xcd_remap(blockIdx.x, gridDim.x);
    const int tm = logical % p.tiles_m, rest = logical / p.tiles_m;
    const int split = rest / p.groups, grp = rest - split * p.groups;
    const int m0 = tm * BM;
    const int kb0 = split * p.kb_per_split;
    const int ns = min(p.KB, kb0 + p.kb_per_split) - kb0;
    const int u_own = grp * WAVES + wave;
    const int u = min(u_own, p.units - 1);         // a wave without a unit repeats the last one

    // lane l of activation load i: row (wave A_INS + i) 8 + l / 8, 16-byte chunk
    // (l % 8) ^ swz(row), so that LDS holds rows of 128 bytes with swizzled chunks
    uint32_t a_off[A_INS];
    int a_k[A_INS];
#pragma unroll
    for (int i = 0; i < A_INS; ++i) {
        const int r = min(wave * A_INS + i, A_ALL - 1) * 8 + (lane >> 3);
        a_k[i] = 16 * ((lane & 7) ^ swz(r));
        a_off[i] = (uint32_t)((size_t)min(m0 + r, p.M - 1) * p.K);
    }
    // weights: fragment (t, kk) of a block of 128 k; see packed_off
    // (two adjacent groups of 16 packed rows a block; PAIR: a Gate group and its Up group)
    const uint32_t w_lane =
        (uint32_t)(((lane >> 4) & 1) * (P::PAIR ? 16384 : 2048) + (lane >> 5) * 256 + (lane & 15) * 16);
    constexpr int EACH = WT == 1 ? 8 : 4;          // units of a packed tile
    const char* w_base = reinterpret_cast<const char*>(p.W) + ((size_t)(u / EACH) * p.KB + kb0) * 32768 +
                         (u % EACH) * (P::PAIR ? 2048 : 4096);

    bf16x8 wf[NBUF][WT][4];
#pragma unroll
    for (int q = 0; q < NBUF; ++q)
#pragma unroll
        for (int t = 0; t < WT; ++t)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) wf[q][t][kk] = bf16x8{};
    // load j of stage ls (weights first) into slot and set SET.  Past the last stage
    // every lane reads the same 16 zeros, so that every stage has the same loads.
    auto issue = [&](int j, int ls, auto setc) __attribute__((always_inline)) {
        constexpr int SET = decltype(setc)::value;
        const bool valid = ls < ns;
        const uint32_t mask = valid ? 0xFFFFFFFFu : 0u;
        const char* const zero = reinterpret_cast<const char*>(g_zero_chunk);
        if (j < 4 * WT) {
            const int t = j >> 2, kk = j & 3;
            const char* b = valid ? w_base + (size_t)ls * 32768 + t * 16384 + (kk >> 1) * 1024 + (kk & 1) * 512 : zero;
            const bf16x8* src = reinterpret_cast<const bf16x8*>(b + (w_lane & mask));
            if constexpr (P::ONCE) wf[SET][t][kk] = __builtin_nontemporal_load(src);
            else wf[SET][t][kk] = *src;
        } else {
            const int i = j - 4 * WT;
            // k past the end: any byte will do, its weights are zero
            const char* b = valid ? reinterpret_cast<const char*>(p.A) : zero;
            const uint32_t k = (uint32_t)min((kb0 + ls) * 128 + a_k[i], p.K - 16);
            const int to = SPARE && wave * A_INS + i >= A_ALL ? NBUF * ASTAGE : SET * ASTAGE + (wave * A_INS + i) * 1024;
            dma16(reinterpret_cast<const uint16_t*>(b + ((a_off[i] + k) & mask)),
                  reinterpret_cast<uint16_t*>(smem + to));
        }
    };
    // fragment reads: row 32 i + (l & 31), chunk 2 kk + (l >> 5), swizzled
    uint32_t rd[4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
        rd[x] = (uint32_t)((lane & 31) * 128 + ((((lane >> 5) ^ swz(lane & 31)) ^ (2 * x)) << 4));
    bf16x8 fa[2][TM];
    auto read_a = [&](int slot, int kk, int i, int set) __attribute__((always_inline)) {
        fa[set][i] = *reinterpret_cast<const bf16x8*>(smem + slot * ASTAGE + i * 4096 + rd[kk ^ (2 * (i & 1))]);
    };

    i32x16 acc[WT][TM];
#pragma unroll
    for (int t = 0; t < WT; ++t)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[t][i][r] = 0;

    // One sub-step: its matrix instructions, the next one's fragments, a share of
    // the loads of stage ls.
    auto substep = [&](auto pc, int kk, int cur, int rslot, int rkk, int ls, auto lsetc, int lq)
                       __attribute__((always_inline)) {
        constexpr int S = decltype(pc)::value;
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int t = 0; t < WT; ++t) acc[t][i] = mma32<true>(wf[S][t][kk], fa[cur][i], acc[t][i]);
            read_a(rslot, rkk, i, cur ^ 1);
#pragma unroll
            for (int j = 0; j < LPS; ++j)
                if (j % TM == i && lq * LPS + j < LOADS) issue(lq * LPS + j, ls, lsetc);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto stage = [&](auto pc, int s) __attribute__((always_inline)) {
        constexpr int S = decltype(pc)::value;
        constexpr int SN = (S + 1) % NBUF;
        using SL = std::integral_constant<int, (S + NBUF - 1) % NBUF>;
        const int ls = s + NBUF - 1;
        __builtin_amdgcn_sched_barrier(0);
        substep(pc, 0, 0, S, 1, ls, SL{}, 0);
        substep(pc, 1, 1, S, 2, ls, SL{}, 1);
        substep(pc, 2, 0, S, 3, ls, SL{}, 2);
        // stage s + 1 has landed; after the barrier no wave reads slot s
        __builtin_amdgcn_s_waitcnt(waitcnt_imm((NBUF - 3) * LOADS + LATE, 0));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        substep(pc, 3, 1, SN, 0, ls, SL{}, 3);
        __builtin_amdgcn_sched_barrier(0);
    };

    // the scales, first of all loads (parts need none)
    f32x4 cs[WT][4];
    float rs[TM];
#pragma unroll
    for (int t = 0; t < WT; ++t) narrow_scales<P>(p, u, t, lane, cs[t]);
#pragma unroll
    for (int i = 0; i < TM; ++i) rs[i] = p.sa[min(m0 + 32 * i + (lane & 31), p.M - 1)];
    __builtin_amdgcn_sched_barrier(0);
    // each stage's loads stay behind the one's before: the wait leaves as many in flight
    // as the later stages have, whichever they are
    each(Upto<NBUF - 1>{}, [&](auto qc) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < LOADS; ++j) issue(j, decltype(qc)::value, qc);
        __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_s_waitcnt(waitcnt_imm((NBUF - 2) * LOADS, 0));
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int t = 0; t < WT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) asm volatile("" : "+v"(cs[t][q]));
#pragma unroll
    for (int i = 0; i < TM; ++i) asm volatile("" : "+v"(rs[i]));
#pragma unroll
    for (int i = 0; i < TM; ++i) read_a(0, 0, i, 0);

    int s = 0;
    for (; s + NBUF <= ns; s += NBUF)
        each(Upto<NBUF>{}, [&](auto qc) __attribute__((always_inline)) { stage(qc, s + decltype(qc)::value); });
    each(Upto<NBUF - 1>{}, [&](auto qc) __attribute__((always_inline)) {
        if (decltype(qc)::value < ns - s) stage(qc, s + decltype(qc)::value);
    });
    // the loads past the end are in flight; their registers are consumed here, without
    // instructions, so that they are not dropped
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
#pragma unroll
    for (int q = 0; q < NBUF; ++q)
#pragma unroll
        for (int t = 0; t < WT; ++t)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) asm volatile("" ::"v"(wf[q][t][kk]));

    if (p.splits > 1) {
        // tile (grp, tm) of this part
        int* d = p.part + (((size_t)split * p.groups + grp) * p.tiles_m + tm) * (P::BLOCKS * 1024) + lane * 4;
#pragma unroll
        for (int t = 0; t < WT; ++t)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<i32x4*>(d + ((wave * WT + t) * TM + i) * 1024 + q * 256) =
                        i32x4{acc[t][i][4 * q], acc[t][i][4 * q + 1], acc[t][i][4 * q + 2], acc[t][i][4 * q + 3]};
        return;
    }
    if (u_own >= p.units) return;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        if constexpr (P::GEMM) {
#pragma unroll
            for (int t = 0; t < WT; ++t)
                narrow_finish<P>(p, u, t, m0 + 32 * i, lane, acc[t][i], acc[t][i], cs[t], cs[t], rs[i]);
        } else {
            narrow_finish<P>(p, u, 0, m0 + 32 * i, lane, acc[0][i], acc[WT - 1][i], cs[0], cs[WT - 1], rs[i]);
        }
    }
}

// The parts' sums, one wave a 32 x 32 block (fused: pair of blocks).
template <class P>
__global__ __launch_bounds__(256) void narrow_reduce_kernel(NarrowArgs p) {
    constexpr int TM = P::TM, JB = P::GEMM ? P::WT : 1;
    constexpr int JOBS = P::WAVES * JB * TM;       // of a tile
    constexpr bool TWO = !P::GEMM && P::WT == 2;   // a Gate block, and its Up block behind the unit's others
    const int lane = threadIdx.x & 63;
    const int id = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile = id / JOBS, job = id - tile * JOBS;
    const int tiles = p.groups * p.tiles_m;
    if (tile >= tiles) return;
    const int grp = tile / p.tiles_m, tm = tile - grp * p.tiles_m;
    const int wave = job / (JB * TM), t = job / TM % JB, i = job % TM;
    const int u = grp * P::WAVES + wave, m0 = tm * P::BM + 32 * i;
    if (u >= p.units || m0 >= p.M) return;
    f32x4 cx[4], cy[4];
    narrow_scales<P>(p, u, t, lane, cx);
    if constexpr (TWO) narrow_scales<P>(p, u, 1, lane, cy);
    const float row = p.sa[min(m0 + (lane & 31), p.M - 1)];
    i32x16 x, y;
#pragma unroll
    for (int r = 0; r < 16; ++r) x[r] = y[r] = 0;
    const int* src = p.part + (size_t)tile * (P::BLOCKS * 1024) + ((wave * P::WT + t) * TM + i) * 1024 + lane * 4;
    const size_t stride = (size_t)tiles * (P::BLOCKS * 1024);
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s, src += stride) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const i32x4 v = *reinterpret_cast<const i32x4*>(src + q * 256);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * q + e] += v[e];
            if constexpr (TWO) {
                const i32x4 w = *reinterpret_cast<const i32x4*>(src + TM * 1024 + q * 256);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[4 * q + e] += w[e];
            }
        }
    }
    narrow_finish<P>(p, u, t, m0, lane, x, y, cx, TWO ? cy : cx, row);
}

}  // namespace swq
