// Device kernels of the gated MLP's training entry points (swiglu_train_*,
// swiglu_mlp_train_backward).
//
// With G = A W1, U = A W2, s = 1 / (1 + e^-G), h = G s and Y = h U, a gradient dY
// gives
//     dU = dY h,   dG = dY U s (1 + G (1 - s)),
//     dA = dG W1^T + dU W2^T,   dW1 = A^T dG,   dW2 = A^T dU,
// and for the whole block Z = Y W3:  dY = dZ W3^T,  dW3 = Y^T dZ.
//
// All of them are products C[i][j] = sum_k a(i, k) b(j, k) on one tile kernel
// (gemm_item): each operand lies in memory either with k contiguous
// (OP_KC: element (i, k) at i * ld + k) or with k strided (OP_KS: at k * ld + i),
// and no operand is transposed through memory: a k-contiguous tile is read from
// LDS as it is, a k-strided one with the transposing LDS read.
//
//   product          i (rows)   j (columns)     k          a    b
//   G, U             token      W1 | W2 column  K          KC   KS, dual
//   dA               token      K               N, then N  KC   KC, two segments
//   dW1 | dW2        K          [dG | dU] col.  token      KS   KS
//   dY -> dG, dU     token      N               K          KC   KC
//   dW3              N          K               token      KS   KS
//
// D = [dG | dU] ([M][2N]) is the one intermediate in memory.  It is rounded to
// bf16 because the matrix cores take bf16 (D as two of them would double the
// gradients' products): each element is then off by at most 2^-8 of itself,
// independently, and the sums over N or M terms that consume it are formed in
// fp32.  That moves dA and the weight gradients about as far as their own rounding
// to bf16 does: in the root mean square they are 0.0023 off the fp64 values,
// relatively, where the rounding of the outputs alone leaves 0.0017.  dY (block)
// and the recomputed G and U stay in fp32 from their sums to dG and dU.
#pragma once

#include "device_common.hpp"

#include <type_traits>

namespace swt {

using namespace swk;

enum Operand : int { OP_KC = 0, OP_KS = 1 };

// What becomes of the sums x (dual products: x the G sums and y the U sums of
// the same columns).
enum Epilogue : int {
    EP_STORE = 0,   // C0 (columns < n0_cols) or C1, bf16
    EP_KEEP = 1,    // dual: Y = SiLU(x) y, G = x, U = y
    EP_DUAL_D = 2,  // dual: D from dY and the recomputed G = x, U = y
    EP_DY_D = 3     // x = dY: D from it and the kept G and U
};

struct GemmArgs {
    const uint16_t* A0;    // operand a; segment 1 from A1
    const uint16_t* A1;
    const uint16_t* B0;    // operand b; segment 1, or the dual product's second half, from B1
    const uint16_t* B1;
    long long lda, ldb;    // leading dimensions (elements)
    int rows, cols;        // output rows and columns (dual: columns of each half)
    int kseg;              // contraction length of one segment
    int segs;              // 1 or 2
    int kb_seg;            // ceil(kseg / 64)
    int tiles_m, tiles_n;
    // work items, one workgroup each: tiles 0 .. whole - 1, then the others (rest
    // of them) in `splits` parts of kb_per_split contraction blocks
    int whole, rest, splits, kb_per_split;
    float* part;           // the parts' sums, [split][rest tile]
    // epilogue operands
    uint16_t* C0;          // STORE: columns below n0_cols (row length ldc); KEEP: Y; D kinds: D
    uint16_t* C1;          // STORE: the other columns; KEEP: G
    uint16_t* C2;          // KEEP: U
    const uint16_t* E0;    // DUAL_D: dY; DY_D: G
    const uint16_t* E1;    // DY_D: U
    int n0_cols, ldc;
};

// dG and dU of one element.  s (1 + g (1 - s)) is SiLU's derivative; at large
// negative g, s is 0 and g (1 - s) finite, so the product is 0 as it should be.
__device__ __forceinline__ void silu_grad(float dy, float g, float u, float& dg, float& du) {
    const float e = __builtin_amdgcn_exp2f(-g * LOG2E);
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    du = dy * (g * s);
    dg = dy * u * (s * (1.0f + g * (1.0f - s)));
}

__device__ __forceinline__ void unpack8(u32x4 v, float (&f)[8]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        f[2 * d] = __builtin_bit_cast(float, v[d] << 16);
        f[2 * d + 1] = __builtin_bit_cast(float, v[d] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
    return u32x4{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
}

__device__ __forceinline__ void st16(uint16_t* p, u32x4 v) { *reinterpret_cast<u32x4*>(p) = v; }

// ---------------------------------------------------------------------------
// Direct global -> LDS loads, 16 bytes a lane: LDS byte address lds (uniform)
// + 16 * lane receives the bytes at the descriptor's base + off.  A lane whose
// offset lies past the descriptor's end gets zeros: that is how k past the end of
// the contraction, and whole stages past it, become zeros in both operands, at
// the price of one compare and select a load (addressing such lanes at a chunk of
// zeros in memory took 64-bit addresses in every lane and 35 % more time).
//   The load is not tracked by the compiler: with the tracked builtin every
// transposing LDS read waits for all loads in flight (vmcnt(0)), as it cannot
// know that they fill other slots.  There is no register to write early; the
// kernels wait with explicit counts, and the compiler's own waits for loads it
// does track only wait for more than they must.  m0 holds the LDS address and is named
// as overwritten, so that no pass of the compiler carries a value of its own in it past
// a load.  (Its warning for a reserved register is off here: it says that the value in m0
// is not kept over the statement, which is what is meant.)
// ---------------------------------------------------------------------------
constexpr int RSRC_END = 0x7FFFFFF0;          // every offset of a valid lane is below
constexpr uint32_t OFF_NONE = 0xFFFFFFF0u;    // past every descriptor's end
__device__ __forceinline__ i32x4 stage_rsrc(const uint16_t* base, bool valid) {
    const uint64_t p = (uint64_t)base;
    return i32x4{(int)(uint32_t)p, (int)(uint32_t)(p >> 32) & 0xFFFF, valid ? RSRC_END : 0, 0x00020000};
}
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16_buffer(i32x4 rsrc, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off),
                 "s"(rsrc)
                 : "m0", "memory");
}
#pragma clang diagnostic pop

// ---------------------------------------------------------------------------
// The epilogue of one 32 x 32 MFMA block without LDS.  A lane holds 16 sums of
// row l & 31: v[4q + e] is column 8q + 4 (l >> 5) + e.  Two exchanges between
// lanes (v_permlane32_swap, v_permlane16_swap) turn the block, packed to bf16,
// into 16 bytes a lane with four lanes on 64 adjacent bytes of a row:
//   out[h]: row 16h + (l & 15), columns 8c .. 8c + 7, c = 2 ((l >> 4) & 1) + (l >> 5).
// They are their own inverse, so operands of the epilogue (dY, G, U) are loaded
// that way too and brought into the lanes that hold the matching sums.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void swap32(unsigned& a, unsigned& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(unsigned& a, unsigned& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// d[q][w]: packed columns 8q + 4 (l >> 5) + 2w, + 1
__device__ __forceinline__ void block_to_rows(unsigned (&d)[4][2], u32x4 (&out)[2]) {
#pragma unroll
    for (int q = 0; q < 4; q += 2)
#pragma unroll
        for (int w = 0; w < 2; ++w) swap32(d[q][w], d[q + 1][w]);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int w = 0; w < 2; ++w) swap16(d[q][w], d[q + 2][w]);
    out[0] = u32x4{d[0][0], d[0][1], d[1][0], d[1][1]};
    out[1] = u32x4{d[2][0], d[2][1], d[3][0], d[3][1]};
}
__device__ __forceinline__ void rows_to_block(const u32x4 (&in)[2], float (&v)[16]) {
    unsigned d[4][2] = {{in[0][0], in[0][1]}, {in[0][2], in[0][3]}, {in[1][0], in[1][1]}, {in[1][2], in[1][3]}};
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int w = 0; w < 2; ++w) swap16(d[q][w], d[q + 2][w]);
#pragma unroll
    for (int q = 0; q < 4; q += 2)
#pragma unroll
        for (int w = 0; w < 2; ++w) swap32(d[q][w], d[q + 1][w]);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            v[4 * q + 2 * w] = __builtin_bit_cast(float, d[q][w] << 16);
            v[4 * q + 2 * w + 1] = __builtin_bit_cast(float, d[q][w] & 0xFFFF0000u);
        }
}

// A matrix seen from a tile's corner, for the block epilogue: accesses of lanes
// past its rows or columns have offsets past the descriptor's end, where loads
// give 0 and stores are dropped, so the epilogue has no branches (with branches
// the compiler moved all sums of a wave out of the accumulation registers at
// once and spilled).
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc corner(const uint16_t* c, long long ld, int m0, int n0) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(c + (size_t)m0 * ld + n0), 0, RSRC_END, 0x00020000);
}
// The lane's two 16-byte pieces of a block: rows r, r + 16 and column n of the
// tile at (m0, n0); inside: whether they lie in the matrix.
struct BlockAt {
    int r, n;
    bool ok[2];
    __device__ __forceinline__ uint32_t at(int h, long long ld) const {
        return ok[h] ? (uint32_t)((r + 16 * h) * (int)ld + n) * 2 : OFF_NONE;
    }
};
__device__ __forceinline__ BlockAt block_at(const GemmArgs& p, int m0, int n0, int r0, int c0, int lane) {
    BlockAt b;
    b.r = r0 + (lane & 15);
    b.n = c0 + 8 * (2 * ((lane >> 4) & 1) + (lane >> 5));
    const bool in = n0 + b.n < p.cols;
    b.ok[0] = in && m0 + b.r < p.rows;
    b.ok[1] = in && m0 + b.r + 16 < p.rows;
    return b;
}
__device__ __forceinline__ void block_store(const BlockAt& b, Rsrc c, long long ld, const float (&v)[16]) {
    unsigned d[4][2];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int w = 0; w < 2; ++w) d[q][w] = pack2(v[4 * q + 2 * w], v[4 * q + 2 * w + 1]);
    u32x4 out[2];
    block_to_rows(d, out);
#pragma unroll
    for (int h = 0; h < 2; ++h) __builtin_amdgcn_raw_buffer_store_b128(out[h], c, b.at(h, ld), 0, 0);
}
__device__ __forceinline__ void block_load(const BlockAt& b, Rsrc c, long long ld, float (&v)[16]) {
    u32x4 in[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) in[h] = __builtin_amdgcn_raw_buffer_load_b128(c, b.at(h, ld), 0, 0);
    rows_to_block(in, v);
}

// The epilogue of the block at row r0, column c0 of the tile at (m0, n0) (x;
// dual: and y).
template <int EPI>
__device__ __forceinline__ void finish_block(const GemmArgs& p, int m0, int n0, int r0, int c0, int lane,
                                             const f32x16& x, const f32x16& y) {
    const BlockAt b = block_at(p, m0, n0, r0, c0, lane);
    float v[16], w[16];
    if constexpr (EPI == EP_STORE) {
        // columns from n0_cols on belong to C1 (a 16-byte piece never straddles)
        BlockAt b0 = b, b1 = b;
        const bool second = n0 + b.n >= p.n0_cols;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            b0.ok[h] = b.ok[h] && !second;
            b1.ok[h] = b.ok[h] && second;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = x[r];
        // the tile's corner within C1 may lie before its first column: the
        // descriptor starts at the row, the column offset is not negative then
        if (n0 < p.n0_cols) block_store(b0, corner(p.C0, p.ldc, m0, n0), p.ldc, v);
        if (n0 + 256 > p.n0_cols) {
            b1.n += n0 - p.n0_cols;
            block_store(b1, corner(p.C1, p.ldc, m0, 0), p.ldc, v);
        }
    } else if constexpr (EPI == EP_KEEP) {
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = silu_f(x[r]) * y[r];
        block_store(b, corner(p.C0, p.cols, m0, n0), p.cols, v);
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = x[r];
        block_store(b, corner(p.C1, p.cols, m0, n0), p.cols, v);
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = y[r];
        block_store(b, corner(p.C2, p.cols, m0, n0), p.cols, v);
    } else {
        float dg[16], du[16];
        block_load(b, corner(p.E0, p.cols, m0, n0), p.cols, v);
        if constexpr (EPI == EP_DUAL_D) {
#pragma unroll
            for (int r = 0; r < 16; ++r) silu_grad(v[r], x[r], y[r], dg[r], du[r]);
        } else {
            block_load(b, corner(p.E1, p.cols, m0, n0), p.cols, w);
#pragma unroll
            for (int r = 0; r < 16; ++r) silu_grad(x[r], v[r], w[r], dg[r], du[r]);
        }
        const Rsrc d = corner(p.C0, 2 * (long long)p.cols, m0, n0);
        block_store(b, d, 2 * (long long)p.cols, dg);
        BlockAt bu = b;
        bu.n += p.cols;
        block_store(bu, d, 2 * (long long)p.cols, du);
    }
}

// ---------------------------------------------------------------------------
// Work items.  A launch holds the items of one product, or of two that do not
// depend on each other (dA and the weight gradients; dY and dW3), and the
// dispatcher hands them to CUs as these fall free (an item's LDS fills a CU), so a
// product of few tiles runs beside the other's, and no CU idles through a last
// round of one product's tiles (7B width, M=8192: 448 and 2072 tiles on 256 CUs).
// Where the items would be too few, tiles are split over the contraction.
// ---------------------------------------------------------------------------
struct ItemAt {
    int m0, n0, s0, s1;   // corner of the tile, stages [s0, s1)
    int slot;             // -1: whole tile; else the part's place in `part`
};
// The corner of a tile of the grid: down eight row tiles before the next column.
template <int BM, int BN>
__device__ __forceinline__ void tile_corner(const GemmArgs& p, int tile, int& m0, int& n0) {
    constexpr int GROUP_M = 8;
    const int per_group = GROUP_M * p.tiles_n;
    const int group = tile / per_group;
    const int first_m = group * GROUP_M;
    const int gsize = min(p.tiles_m - first_m, GROUP_M);
    const int in_group = tile - group * per_group;
    m0 = (first_m + in_group % gsize) * BM;
    n0 = in_group / gsize * BN;
}
// whole tiles: an XCD holds a contiguous run; parts: all tiles of a split before the next, so an XCD holds a range of
// the contraction and fetches its piece of both operands once
template <int BM, int BN>
__device__ __forceinline__ ItemAt item_at(const GemmArgs& p, int b) {
    const int KB = p.segs * p.kb_seg;
    ItemAt it;
    int tile;
    if (b < p.whole) {
        tile = xcd_remap(b, p.whole);
        it.s0 = 0;
        it.s1 = KB;
        it.slot = -1;
    } else {
        it.slot = xcd_remap(b - p.whole, p.rest * p.splits);
        const int split = it.slot / p.rest;
        tile = p.whole + it.slot - split * p.rest;
        it.s0 = split * p.kb_per_split;
        it.s1 = min(KB, it.s0 + p.kb_per_split);   // the host makes no empty part
    }
    tile_corner<BM, BN>(p, tile, it.m0, it.n0);
    // the same in every lane: kept in scalar registers
    it.m0 = __builtin_amdgcn_readfirstlane(it.m0);
    it.n0 = __builtin_amdgcn_readfirstlane(it.n0);
    it.s0 = __builtin_amdgcn_readfirstlane(it.s0);
    it.s1 = __builtin_amdgcn_readfirstlane(it.s1);
    it.slot = __builtin_amdgcn_readfirstlane(it.slot);
    return it;
}

// A 32 x 32 block of sums as it lies in the lanes: [quad][lane][4].
__device__ __forceinline__ void store_sums(float* d, const f32x16& a) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4*>(d + q * 256) = f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
}
__device__ __forceinline__ void add_sums(const float* s, f32x16& a) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(s + q * 256);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[4 * q + e] += v[e];
    }
}

// ---------------------------------------------------------------------------
// A BM x BN item, four waves (2 x 2) of BM/2 x BN/2 sums each (DUAL: BN / 2
// columns of each half, each wave BN/4 of either).
//   256 x 256 (all 256 accumulation registers of a wave): 64 KiB go into a CU per
// 64-deep stage of 2048 matrix-core cycles, and what bounds it is having them in
// flight early enough.  Two whole stages are 128 of the 160 KiB of LDS, so the
// ring is made of five 32 KiB half stages (one operand's 256 x 64 each): stage s's
// b goes out as soon as stage s - 2 has been read, a whole stage before it is
// needed, and its a another three sub-steps earlier, into the fifth slot.
//   Smaller tiles, for few rows: there a product is a chain of load latencies (a
// 128 x 128 stage has 512 matrix-core cycles, its loads take four times as long),
// so the ring holds five or six whole stages, all but one of them in flight.
//   In both, each 16-deep sub-step is a fixed (fenced) sequence of matrix
// instructions with the next sub-step's fragment reads and a share of the loads
// between them; the waits are explicit: fragments at the start of the sub-step
// that uses them, loads before the stage's one barrier, where only those not
// needed by the next stage may be in flight.  Every stage issues the same loads
// (past the end they give zeros), so the counts hold.
//   Rows or columns past the edge repeat the last ones; their sums are not stored.
//   LDS tiles: k-contiguous [rows][64], chunks swizzled by row (lds_off);
// k-strided [64][columns], chunks swizzled by k (rm_off; DUAL: one [64][BN / 2]
// tile for each half).
//   Measured: at 7B width dA and both weight gradients of 8192 tokens 3.51 ms (1.27
// PFLOP/s, matrix cores busy 69 % of the cycles at 1.74 GHz: the chip's power sets
// the clock), the forward product of 4096 tokens with its three outputs 0.99 ms (1.13
// PFLOP/s), of 64 tokens at 0.5B width 10.9 us (a chain of 14 stages' loads).
// ---------------------------------------------------------------------------
template <int BM_, int BN_, int AOP_, int BOP_, bool DUAL_, int EPI_>
struct Product {
    static constexpr int BM = BM_, BN = BN_, AOP = AOP_, BOP = BOP_, EPI = EPI_;
    static constexpr bool DUAL = DUAL_;
    static constexpr int TM = BM / 64, TN = BN / 64;   // a wave's blocks
    static constexpr int COLS = DUAL ? BN / 2 : BN;    // output columns of a tile
    static_assert(!DUAL || TN % 2 == 0, "a wave holds both halves of its columns");
};
constexpr int LDS_BYTES = 163840;

// element offset in a k-strided LDS tile of COLS columns (rm_off; rows of 64
// columns are 128 bytes, where the lowest bit of k alone is free to swizzle with)
template <int COLS>
__device__ __forceinline__ int ks_off(int k, int col) {
    return COLS >= 128 ? rm_off<COLS>(k, col) : k * COLS + (((col >> 3) ^ ((k & 1) << 2)) << 3) + (col & 7);
}

template <class P>
__device__ __forceinline__ void gemm_item(const GemmArgs& p, uint16_t* smem, int b) {
    constexpr int BM = P::BM, BN = P::BN, AOP = P::AOP, BOP = P::BOP, TM = P::TM, TN = P::TN;
    constexpr bool DUAL = P::DUAL;
    constexpr bool HALVES = BM == 256 && BN == 256;   // the ring of half stages
    constexpr int A_INS = BM / 32, B_INS = BN / 32;   // 1 KiB loads per wave and stage
    constexpr int A_ELEMS = BM * BK, B_ELEMS = BN * BK;
    constexpr int NS = HALVES ? 2 : (LDS_BYTES / 2 / (A_ELEMS + B_ELEMS) < 6 ? LDS_BYTES / 2 / (A_ELEMS + B_ELEMS) : 6);
    constexpr int BCOL = DUAL ? BN / 2 : BN;          // columns of a k-strided b tile in LDS
    static_assert(AOP == OP_KC || BM >= 128, "a k-strided tile has rows of at least 128 elements");
    static_assert(BOP == OP_KC || BCOL >= 64, "a k-strided tile has rows of at least 64 elements");
    static_assert(HALVES || (NS - 2) * (A_INS + B_INS) <= 63, "vmcnt range");

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int hi5 = lane >> 5;
    const ItemAt it = item_at<BM, P::COLS>(p, b);
    const int m0 = it.m0, n0 = it.n0;

    // Byte offsets of a lane's 16 bytes in load i from the stage's base, constant
    // over the stages, and the lane's (first) k within the stage.  k-contiguous:
    // 8 rows x 128 bytes a load; k-strided: whole k rows of the tile's columns.
    uint32_t a_off[A_INS], b_off[B_INS];
    auto kc_k = [&](int q) { return 8 * ((lane & 7) ^ swz(q * 8 + (lane >> 3))); };
    auto ks_k = [&](int q, int cols) { return q * (512 / cols) + lane / (cols / 8); };
    auto ks_c = [&](int q, int cols) {   // logical column of the lane's chunk
        const int k = ks_k(q, cols);
        return 8 * ((lane % (cols / 8)) ^ (cols >= 128 ? (k & 3) << 2 : (k & 1) << 2));
    };
#pragma unroll
    for (int i = 0; i < A_INS; ++i) {
        const int q = wave * A_INS + i;
        a_off[i] = AOP == OP_KC ? (uint32_t)((min(m0 + q * 8 + (lane >> 3), p.rows - 1) - m0) * p.lda + kc_k(q)) * 2
                                : (uint32_t)(ks_k(q, BM) * p.lda + min(m0 + ks_c(q, BM), p.rows - 8) - m0) * 2;
    }
    // dual: waves 0, 1 load the first half, waves 2, 3 the second
    auto b_q = [&](int i) { return DUAL ? (wave & 1) * B_INS + i : wave * B_INS + i; };
#pragma unroll
    for (int i = 0; i < B_INS; ++i) {
        const int q = b_q(i);
        b_off[i] = BOP == OP_KC ? (uint32_t)((min(n0 + q * 8 + (lane >> 3), p.cols - 1) - n0) * p.ldb + kc_k(q)) * 2
                                : (uint32_t)(ks_k(q, BCOL) * p.ldb + min(n0 + ks_c(q, BCOL), p.cols - 8) - n0) * 2;
    }

    // descriptor of an operand's stage s
    auto rsrc_of = [&](bool isb, int s) __attribute__((always_inline)) {
        const int seg = s >= p.kb_seg ? 1 : 0;
        const int k0 = (s - seg * p.kb_seg) * BK;
        const int op = isb ? BOP : AOP;
        const long long ld = isb ? p.ldb : p.lda;
        const int r0 = isb ? n0 : m0;
        const uint16_t* m = isb ? ((DUAL ? wave >= 2 : seg) ? p.B1 : p.B0) : (seg ? p.A1 : p.A0);
        return stage_rsrc(m + (op == OP_KC ? (size_t)r0 * ld + k0 : (size_t)k0 * ld + r0), s < it.s1);
    };
    auto left_of = [&](int s) { return p.kseg - (s >= p.kb_seg ? s - p.kb_seg : s) * BK; };
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void_ptr)smem;
    // load i of an operand's stage (its descriptor, k left in it) to LDS element dst
    auto load_a = [&](i32x4 rsrc, int left, int i, int dst) __attribute__((always_inline)) {
        const int q = wave * A_INS + i;
        const int k = AOP == OP_KC ? kc_k(q) : ks_k(q, BM);
        dma16_buffer(rsrc, k < left ? a_off[i] : OFF_NONE, lds0 + (uint32_t)(dst + q * 512) * 2);
    };
    auto load_b = [&](i32x4 rsrc, int left, int i, int dst) __attribute__((always_inline)) {
        const int q = b_q(i);
        const int k = BOP == OP_KC ? kc_k(q) : ks_k(q, BCOL);
        dma16_buffer(rsrc, k < left ? b_off[i] : OFF_NONE,
                     lds0 + (uint32_t)(dst + (DUAL && wave >= 2 ? B_ELEMS / 2 : 0) + q * 512) * 2);
    };

    // Fragment addresses: a few lane offsets and constants.  k-contiguous: rows
    // w + 32i + (l & 31), chunk (2kk + (l >> 5)) ^ swz(row), and
    // swz(32i + r) = swz(r) ^ 4 (i & 1): four bases x = kk ^ 2 (i & 1).
    // k-strided: k row 16kk + 8 (l >> 5) + (l & 15) / 4, whose low bits fix the
    // swizzle for the lane: one base per block.
    uint32_t a_base[4], b_base[4];
    const int tr_k = 8 * hi5 + ((lane & 15) >> 2), tr_c = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    auto kc_base = [&](int x, int row0) {
        const int r = lane & 31;
        return (uint32_t)(row0 * 128 + r * 128 + (((hi5 ^ swz(row0 + r)) ^ (2 * x)) << 4));
    };
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        a_base[x] = AOP == OP_KC ? kc_base(x, wm * (BM / 2))
                                 : (uint32_t)rm_off<BM>(tr_k, wm * (BM / 2) + (x < TM ? x : 0) * 32 + tr_c) * 2;
        if constexpr (BOP == OP_KC) {
            b_base[x] = kc_base(x, wn * (BN / 2));
        } else {
            const int j = x < TN ? x : 0;
            const int half = DUAL ? j / (TN / 2 > 0 ? TN / 2 : 1) : 0;
            const int col = DUAL ? wn * (BN / 4) + j % (TN / 2 > 0 ? TN / 2 : 1) * 32 : wn * (BN / 2) + j * 32;
            b_base[x] = (uint32_t)(half * (B_ELEMS / 2) + ks_off<BCOL>(tr_k, col + tr_c)) * 2;
        }
    }
    auto read_frag = [&](auto opc, auto colsc, const uint32_t (&base)[4], uint32_t so, int kk, int i) -> bf16x8 {
        constexpr int OP = decltype(opc)::value;
        constexpr int COLS = decltype(colsc)::value;
        const char* sm = reinterpret_cast<const char*>(smem) + so;
        if constexpr (OP == OP_KC) {
            return *reinterpret_cast<const bf16x8*>(sm + i * 4096 + base[kk ^ (2 * (i & 1))]);
        } else {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(sm + kk * (16 * COLS * 2) + base[i]);
            const s16x4 both[2] = {ds_read_tr16(q), ds_read_tr16(q + 4 * COLS)};
            return __builtin_bit_cast(bf16x8, both);
        }
    };
    bf16x8 fa[2][TM], fb[2][TN];
    auto read_a = [&](uint32_t so, int kk, int i, int set) {
        fa[set][i] = read_frag(std::integral_constant<int, AOP>{}, std::integral_constant<int, BM>{}, a_base, so, kk, i);
    };
    auto read_b = [&](uint32_t so, int kk, int j, int set) {
        fb[set][j] =
            read_frag(std::integral_constant<int, BOP>{}, std::integral_constant<int, BCOL>{}, b_base, so, kk, j);
    };
    // a byte offset in LDS, opaque so that addresses are formed from the lane bases
    // instead of being kept for every slot
    auto opaque = [](int elems) {
        uint32_t so = (uint32_t)elems * 2;
        asm volatile("" : "+s"(so));
        return so;
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    using Set0 = std::integral_constant<int, 0>;
    using Set1 = std::integral_constant<int, 1>;

    if constexpr (HALVES) {
        constexpr int SLOT = 256 * BK;   // elements of a half stage
        // one 16-deep sub-step on fragment set CUR: 16 matrix instructions, the
        // next sub-step's reads (rkk of the slots at aso, bso) in its first half,
        // and NLD loads a quarter from load l0 on
        auto substep = [&](auto curc, uint32_t aso, uint32_t bso, int rkk, auto ldbc, auto nldc, i32x4 rsrc, int left,
                           int dst, int l0) __attribute__((always_inline)) {
            constexpr int CUR = decltype(curc)::value;
            constexpr bool LDB = decltype(ldbc)::value;
            constexpr int NLD = decltype(nldc)::value;
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[CUR][j], fa[CUR][i], acc[i][j], 0, 0, 0);
                if (i < 2) {
#pragma unroll
                    for (int t = 2 * i; t < 2 * i + 2; ++t) {
                        read_a(aso, rkk, t, CUR ^ 1);
                        read_b(bso, rkk, t, CUR ^ 1);
                    }
                }
#pragma unroll
                for (int t = 0; t < NLD; ++t) {
                    if constexpr (LDB) load_b(rsrc, left, l0 + i * NLD + t, dst);
                    else load_a(rsrc, left, l0 + i * NLD + t, dst);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        using N0 = std::integral_constant<int, 0>;
        using N1 = std::integral_constant<int, 1>;
        using N2 = std::integral_constant<int, 2>;
        using LA = std::false_type;
        using LB = std::true_type;
        auto wrap = [](int x) { return x >= 5 ? x - 5 : x; };
        // stage s sits in slots sa (a) and sa + 1 (b), modulo 5
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const i32x4 ra = rsrc_of(false, it.s0 + t), rb = rsrc_of(true, it.s0 + t);
            const int left = left_of(it.s0 + t);
#pragma unroll
            for (int i = 0; i < 8; ++i) load_a(ra, left, i, 2 * t * SLOT);
#pragma unroll
            for (int i = 0; i < 8; ++i) load_b(rb, left, i, (2 * t + 1) * SLOT);
        }
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(16, 0));
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            read_a(0u, 0, t, 0);
            read_b(SLOT * 2, 0, t, 0);
        }
        int sa = 0;
        for (int s = it.s0; s < it.s1; ++s) {
            const uint32_t ao = opaque(sa * SLOT), bo = opaque(wrap(sa + 1) * SLOT);
            const i32x4 ra = rsrc_of(false, s + 2), rb = rsrc_of(true, s + 2);
            const int left = left_of(s + 2), as = wrap(sa + 4) * SLOT;
            __builtin_amdgcn_sched_barrier(0);
            substep(Set0{}, ao, bo, 1, LA{}, N1{}, ra, left, as, 0);
            substep(Set1{}, ao, bo, 2, LA{}, N1{}, ra, left, as, 4);
            substep(Set0{}, ao, bo, 3, LA{}, N0{}, ra, left, as, 0);
            // stage s + 1 has landed (only stage s + 2's a loads may be in
            // flight), and this wave has read stage s (its last reads fill the
            // next sub-step's fragments)
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(8, 0));
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            const int sn = wrap(sa + 2);
            substep(Set1{}, opaque(sn * SLOT), opaque(wrap(sn + 1) * SLOT), 0, LB{}, N2{}, rb, left, sa * SLOT, 0);
            __builtin_amdgcn_sched_barrier(0);
            sa = sn;
        }
    } else {
        constexpr int SLOT = A_ELEMS + B_ELEMS;
        constexpr int LOADS = A_INS + B_INS;
        auto load_stage = [&](int s, int slot) __attribute__((always_inline)) {
            const i32x4 ra = rsrc_of(false, s), rb = rsrc_of(true, s);
            const int left = left_of(s);
#pragma unroll
            for (int i = 0; i < A_INS; ++i) load_a(ra, left, i, slot * SLOT);
#pragma unroll
            for (int i = 0; i < B_INS; ++i) load_b(rb, left, i, slot * SLOT + A_ELEMS);
        };
        auto substep = [&](auto curc, uint32_t so, int rkk) __attribute__((always_inline)) {
            constexpr int CUR = decltype(curc)::value;
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
#pragma unroll
            for (int i = 0; i < TM; ++i) read_a(so, rkk, i, CUR ^ 1);
#pragma unroll
            for (int j = 0; j < TN; ++j) read_b(so + A_ELEMS * 2, rkk, j, CUR ^ 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[CUR][j], fa[CUR][i], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int t = 0; t < NS; ++t) load_stage(it.s0 + t, t);
        __builtin_amdgcn_s_waitcnt(waitcnt_imm((NS - 1) * LOADS <= 63 ? (NS - 1) * LOADS : 63, 0));
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int i = 0; i < TM; ++i) read_a(0u, 0, i, 0);
#pragma unroll
        for (int j = 0; j < TN; ++j) read_b(A_ELEMS * 2, 0, j, 0);
        int slot = 0;
        for (int s = it.s0; s < it.s1; ++s) {
            const int next = slot + 1 == NS ? 0 : slot + 1;
            const uint32_t so = opaque(slot * SLOT);
            __builtin_amdgcn_sched_barrier(0);
            substep(Set0{}, so, 1);
            substep(Set1{}, so, 2);
            substep(Set0{}, so, 3);
            // stage s + 1 has landed (stages s + 2 .. s + NS - 1 may be in flight),
            // and this wave has read stage s
            __builtin_amdgcn_s_waitcnt(waitcnt_imm((NS - 2) * LOADS, 0));
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            load_stage(s + NS, slot);
            substep(Set1{}, opaque(next * SLOT), 0);
            slot = next;
        }
    }
    // the sums stay in accumulation registers here and leave them block by block
    // (left to itself the compiler copies all of them out at the loop's end, and
    // spills)
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) asm volatile("" : "+a"(acc[i][j]));
    // the loads past the end
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));

    if (it.slot >= 0) {
        float* d = p.part + ((size_t)it.slot * 4 + wave) * (TM * TN * 1024) + lane * 4;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                asm volatile("" : "+a"(acc[i][j]));
                store_sums(d + (i * TN + j) * 1024, acc[i][j]);
                __builtin_amdgcn_sched_barrier(0);
            }
        return;
    }
    constexpr int JB = DUAL ? TN / 2 : TN;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            // an opaque copy of the lane index: the block's addresses are formed
            // here, not kept in registers through the loop
            int el = lane;
            if constexpr (DUAL) asm volatile("" : "+v"(el), "+a"(acc[i][j]), "+a"(acc[i][j + JB]));
            else asm volatile("" : "+v"(el), "+a"(acc[i][j]));
            finish_block<P::EPI>(p, m0, n0, wm * (BM / 2) + i * 32, wn * (P::COLS / 2) + j * 32, el, acc[i][j],
                                 acc[i][DUAL ? j + JB : j]);
            __builtin_amdgcn_sched_barrier(0);
        }
}

struct NoProduct {};

// Items of product A and (unless NoProduct) product B, the one with the longer
// items first.
template <class A, class B>
__global__ __launch_bounds__(256) void gemm_kernel(GemmArgs a, GemmArgs b, int items_a, int items_b, int b_first) {
    __shared__ __attribute__((aligned(16))) uint16_t smem[LDS_BYTES / 2];
    const int blk = blockIdx.x;
    if constexpr (std::is_same_v<B, NoProduct>) {
        gemm_item<A>(a, smem, blk);
    } else {
        const bool is_b = b_first ? blk < items_b : blk >= items_a;
        if (!is_b) gemm_item<A>(a, smem, b_first ? blk - items_b : blk);
        else gemm_item<B>(b, smem, b_first ? blk : blk - items_a);
    }
}

// The parts' sums of one 32 x 32 block (dual: pair) of a split tile, added in
// order of the contraction (whatever workgroup finished first), then the epilogue.
template <class P>
__device__ __forceinline__ void reduce_item(const GemmArgs& p, int id, int lane) {
    constexpr int TM = P::TM, TN = P::TN, JB = P::DUAL ? TN / 2 : TN;
    constexpr int BLOCKS = 4 * TM * JB;
    const int t = id / BLOCKS, blk = id % BLOCKS;
    if (t >= p.rest) return;
    const int wv = blk / (TM * JB), i = blk / JB % TM, j = blk % JB;
    constexpr size_t TILE = (size_t)4 * TM * TN * 1024;
    f32x16 x, y;
#pragma unroll
    for (int r = 0; r < 16; ++r) x[r] = y[r] = 0.0f;
    const float* src = p.part + t * TILE + (size_t)(wv * TM * TN + i * TN + j) * 1024 + lane * 4;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s, src += p.rest * TILE) {
        add_sums(src, x);
        if constexpr (P::DUAL) add_sums(src + JB * 1024, y);
    }
    int m0, n0;
    tile_corner<P::BM, P::COLS>(p, p.whole + t, m0, n0);
    finish_block<P::EPI>(p, m0, n0, (wv & 1) * (P::BM / 2) + i * 32, (wv >> 1) * (P::COLS / 2) + j * 32, lane,
                         x, y);
}
template <class A, class B>
__global__ __launch_bounds__(256) void gemm_reduce_kernel(GemmArgs a, GemmArgs b, int blocks_a) {
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (std::is_same_v<B, NoProduct>) {
        reduce_item<A>(a, blockIdx.x * 4 + w, lane);
    } else {
        if ((int)blockIdx.x < blocks_a) reduce_item<A>(a, blockIdx.x * 4 + w, lane);
        else reduce_item<B>(b, (blockIdx.x - blocks_a) * 4 + w, lane);
    }
}

// D = [dG | dU] from dY and the kept G and U, 8 elements a thread: bound by HBM (7B
// width, 8192 tokens: 1.55 GB in 272 us, 5.7 TB/s).
__global__ __launch_bounds__(256) void dgate_kernel(const uint16_t* __restrict__ dY, const uint16_t* __restrict__ G,
                                                    const uint16_t* __restrict__ U, uint16_t* __restrict__ D, int N,
                                                    long long groups) {
    const int per_row = N / 8;
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < groups; t += (long long)gridDim.x * 256) {
        const long long m = t / per_row;
        const int n = (int)(t - m * per_row) * 8;
        float dy[8], g[8], u[8], dg[8], du[8];
        unpack8(ld16(dY + t * 8), dy);
        unpack8(ld16(G + t * 8), g);
        unpack8(ld16(U + t * 8), u);
#pragma unroll
        for (int e = 0; e < 8; ++e) silu_grad(dy[e], g[e], u[e], dg[e], du[e]);
        uint16_t* d = D + (size_t)m * 2 * N + n;
        st16(d, pack8(dg));
        st16(d + N, pack8(du));
    }
}

// Zeros (weight gradients of an empty batch); count in 16-byte pieces.
__global__ __launch_bounds__(256) void zero_kernel(uint16_t* __restrict__ p, long long count) {
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < count; t += (long long)gridDim.x * 256)
        st16(p + t * 8, u32x4{0u, 0u, 0u, 0u});
}

}  // namespace swt
