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
// (tile_gemm_kernel): each operand lies in memory either with k contiguous
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
// bf16 because the matrix cores take bf16: each element is then off by at most
// 2^-8 of itself, independently, and the sums over N or M terms that consume it
// are formed in fp32, so dA and the weight gradients move by less than their own
// rounding to bf16 does.  dY (block) and the recomputed G and U stay in fp32
// from their sums to dG and dU.
#pragma once

#include "device_common.hpp"

#include <type_traits>

namespace swt {

using namespace swk;

// 16 zero bytes that lanes past the end of a contraction read
__device__ __attribute__((aligned(16))) uint16_t g_zeros[8];

enum Operand : int { OP_KC = 0, OP_KS = 1 };

// What becomes of the sums of 8 adjacent columns (x; dual products: x the G
// sums and y the U sums of the same columns).
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
    int splits, kb_per_split;   // contraction blocks (over both segments) per split
    int full;              // 256-row tiles computed whole (wide_gemm_kernel)
    float* part;           // split sums [split][rows][part_cols], or pieces' sums
    int part_cols;         // cols, or 2 cols for a dual product
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

// The epilogue of columns n .. n + 7 of row m (both in range; n a multiple of 8,
// and every width too, so 8 columns never straddle a matrix's edge).
template <int EPI>
__device__ __forceinline__ void finish8(const GemmArgs& p, int m, int n, const float (&x)[8], const float (&y)[8]) {
    if constexpr (EPI == EP_STORE) {
        uint16_t* c = n < p.n0_cols ? p.C0 + (size_t)m * p.ldc + n : p.C1 + (size_t)m * p.ldc + (n - p.n0_cols);
        st16(c, pack8(x));
    } else if constexpr (EPI == EP_KEEP) {
        const size_t at = (size_t)m * p.cols + n;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = silu_f(x[e]) * y[e];
        st16(p.C0 + at, pack8(v));
        st16(p.C1 + at, pack8(x));
        st16(p.C2 + at, pack8(y));
    } else {
        const size_t at = (size_t)m * p.cols + n;
        float e0[8], dg[8], du[8];
        unpack8(ld16(p.E0 + at), e0);
        if constexpr (EPI == EP_DUAL_D) {
#pragma unroll
            for (int e = 0; e < 8; ++e) silu_grad(e0[e], x[e], y[e], dg[e], du[e]);
        } else {
            float e1[8];
            unpack8(ld16(p.E1 + at), e1);
#pragma unroll
            for (int e = 0; e < 8; ++e) silu_grad(x[e], e0[e], e1[e], dg[e], du[e]);
        }
        uint16_t* d = p.C0 + (size_t)m * 2 * p.cols + n;
        st16(d, pack8(dg));
        st16(d + p.cols, pack8(du));
    }
}

__device__ __forceinline__ void load8(const float* s, float (&x)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(s + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * h + e] = v[e];
    }
}

__device__ __forceinline__ void store8(float* d, const float (&x)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        *reinterpret_cast<f32x4*>(d + 4 * h) = f32x4{x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]};
}

// 8 columns of a finished tile: to the split's sums, or through the epilogue.
template <bool DUAL, int EPI>
__device__ __forceinline__ void finish_or_part(const GemmArgs& p, int split, int m, int n, const float (&x)[8],
                                               const float (&y)[8]) {
    if (p.splits > 1) {
        float* d = p.part + ((size_t)split * p.rows + m) * p.part_cols + n;
        store8(d, x);
        if constexpr (DUAL) store8(d + p.cols, y);
    } else {
        finish8<EPI>(p, m, n, x, y);
    }
}

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
constexpr int RSRC_END = 0x7FFFFFF0;
__device__ __forceinline__ Rsrc corner(const uint16_t* c, long long ld, int m0, int n0) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(c + (size_t)m0 * ld + n0), 0, RSRC_END, 0x00020000);
}
// The lane's two 16-byte pieces of a block: rows r, r + 16 and column n of the
// tile at (m0, n0); inside: whether they lie in the matrix.
struct BlockAt {
    int r, n;
    bool ok[2];
    __device__ __forceinline__ uint32_t at(int h, long long ld) const {
        return ok[h] ? (uint32_t)((r + 16 * h) * (int)ld + n) * 2 : 0xFFFFFFF0u;
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
// One BM x BN tile of sums per workgroup of WM x WN waves (DUAL: BN / 2 columns
// of each half).  Each wave owns BM/WM x BN/WN of it as 32 x 32 MFMA blocks.
//   Stages of 64 k, both operands direct to LDS, two stages: the next stage's
//   loads go out at the start of a stage and have three of its four 16-deep
//   sub-steps to land; the one barrier per stage sits before the last sub-step,
//   whose fragments are in registers by then.
//   Rows or columns past the edge repeat the last ones (their sums are not
//   stored); k past the end reads the zero chunk in both operands, so nothing
//   behind a row's end is ever multiplied (RAGGED; only compiled in when the
//   contraction is not a multiple of 64).
//   The sums leave through LDS in fp32, so the epilogue works on 8 adjacent
//   columns a lane: its reads (dY, G, U) and its stores are 16 bytes a lane over
//   whole row segments.
// ---------------------------------------------------------------------------
template <int BM, int BN, int WM, int WN>
constexpr int tile_smem_bytes() {
    constexpr int stages = 2 * (BM + BN) * BK * 2;
    constexpr int rpp = BM / WM >= 64 ? 64 : BM / WM;
    constexpr int stage_f = WM * WN * rpp * (BN / WN + 4) * 4;
    return stages > stage_f ? stages : stage_f;
}

template <int BM, int BN, int WM, int WN, int AOP, int BOP, bool DUAL, int EPI, bool RAGGED>
__global__ __launch_bounds__(64 * WM * WN) void tile_gemm_kernel(GemmArgs p) {
    constexpr int NW = WM * WN;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
    constexpr int A_INS = BM / 8 / NW, B_INS = BN / 8 / NW;   // 1 KiB direct loads per wave per stage
    constexpr int STAGE = (BM + BN) * BK;
    constexpr int GROUP_M = 8;
    static_assert(TM >= 1 && TN >= 1 && (!DUAL || TN % 2 == 0), "wave tile");
    static_assert(AOP == OP_KC || BM >= 128, "a k-strided tile has rows of at least 128 elements");
    static_assert(BOP == OP_KC || BN >= 128, "a k-strided tile has rows of at least 128 elements");
    __shared__ __attribute__((aligned(16))) unsigned char smem_raw[tile_smem_bytes<BM, BN, WM, WN>()];
    uint16_t* const smem = reinterpret_cast<uint16_t*>(smem_raw);

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;

    // logical id -> (tile, split); a tile's splits are consecutive, so they stay
    // on one XCD, and tiles go down GROUP_M row tiles before the next column
    const int logical = xcd_remap(blockIdx.x, gridDim.x);
    const int tile = logical / p.splits;
    const int split = logical - tile * p.splits;
    int tm, tn;
    {
        const int per_group = GROUP_M * p.tiles_n;
        const int group = tile / per_group;
        const int first_m = group * GROUP_M;
        const int gsize = min(p.tiles_m - first_m, GROUP_M);
        const int in_group = tile - group * per_group;
        tm = first_m + in_group % gsize;
        tn = in_group / gsize;
    }
    const int m0 = tm * BM;
    const int n0 = tn * (DUAL ? BN / 2 : BN);
    const int s_first = split * p.kb_per_split;
    const int s_end = min(p.segs * p.kb_seg, s_first + p.kb_per_split);   // the host makes no empty split

    // per-lane byte offsets from the stage's base, constant over the stages:
    // k-contiguous operand: 8 rows x 128 bytes a load, chunks swizzled by row;
    // k-strided: whole k rows of the tile's columns, chunks swizzled by k
    uint32_t a_off[A_INS], b_off[B_INS];
    int a_k[A_INS], b_k[B_INS];   // RAGGED: the load's (first) k within the stage
#pragma unroll
    for (int i = 0; i < A_INS; ++i) {
        const int q = wave * A_INS + i;
        if constexpr (AOP == OP_KC) {
            const int r = q * 8 + (lane >> 3), c = (lane & 7) ^ swz(r);
            a_off[i] = (uint32_t)((min(m0 + r, p.rows - 1) - m0) * p.lda + 8 * c) * 2;
            a_k[i] = 8 * c;
        } else {
            constexpr int CPR = BM / 8, RPI = 64 / CPR;
            const int r = q * RPI + lane / CPR, c = 8 * ((lane % CPR) ^ ((r & 3) << 2));
            a_off[i] = (uint32_t)(r * p.lda + min(m0 + c, p.rows - 8) - m0) * 2;
            a_k[i] = r;
        }
    }
    const uint16_t* b_half[B_INS];   // dual: which half's matrix a load reads
#pragma unroll
    for (int i = 0; i < B_INS; ++i) {
        const int q = wave * B_INS + i;
        b_half[i] = p.B0;
        if constexpr (BOP == OP_KC) {
            const int r = q * 8 + (lane >> 3), c = (lane & 7) ^ swz(r);
            b_off[i] = (uint32_t)((min(n0 + r, p.cols - 1) - n0) * p.ldb + 8 * c) * 2;
            b_k[i] = 8 * c;
        } else {
            constexpr int CPR = BN / 8, RPI = 64 / CPR;
            const int r = q * RPI + lane / CPR, c = 8 * ((lane % CPR) ^ ((r & 3) << 2));
            const bool up = DUAL && c >= BN / 2;
            const int cc = up ? c - BN / 2 : c;
            b_off[i] = (uint32_t)(r * p.ldb + min(n0 + cc, p.cols - 8) - n0) * 2;
            b_k[i] = r;
            if (up) b_half[i] = p.B1;
        }
    }

    auto issue = [&](int s, int buf) {
        uint16_t* sA = smem + buf * STAGE;
        uint16_t* sB = sA + BM * BK;
        const int seg = s >= p.kb_seg ? 1 : 0;
        const int k0 = (s - seg * p.kb_seg) * BK;
        const int left = p.kseg - k0;   // k left in the segment, > 0
        const char* a_base = reinterpret_cast<const char*>(
            (seg ? p.A1 : p.A0) + (AOP == OP_KC ? (size_t)m0 * p.lda + k0 : (size_t)k0 * p.lda + m0));
        const size_t b_at = BOP == OP_KC ? (size_t)n0 * p.ldb + k0 : (size_t)k0 * p.ldb + n0;
#pragma unroll
        for (int i = 0; i < A_INS; ++i) {
            const uint16_t* src = reinterpret_cast<const uint16_t*>(a_base + a_off[i]);
            if constexpr (RAGGED) {
                if (a_k[i] >= left) src = g_zeros;
            }
            dma16(src, sA + (wave * A_INS + i) * 512);
        }
#pragma unroll
        for (int i = 0; i < B_INS; ++i) {
            const uint16_t* base = DUAL ? b_half[i] : (seg ? p.B1 : p.B0);
            const uint16_t* src =
                reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(base + b_at) + b_off[i]);
            if constexpr (RAGGED) {
                if (b_k[i] >= left) src = g_zeros;
            }
            dma16(src, sB + (wave * B_INS + i) * 512);
        }
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    // fragments: lane l holds row (l & 31) of the block and the 8 k from
    // 16kk + 8(l >> 5); the transposing read takes two reads of 4 k each
    bf16x8 fa[2][TM], fb[2][TN];
    const int tr_k = 8 * (lane >> 5) + ((lane & 15) >> 2);
    const int tr_c = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    auto frag = [&](auto opc, auto widthc, const uint16_t* s, int row, int kk) -> bf16x8 {
        constexpr int OP = decltype(opc)::value;
        constexpr int W = decltype(widthc)::value;
        if constexpr (OP == OP_KC) {
            return *reinterpret_cast<const bf16x8*>(s + lds_off(row + (lane & 31), 2 * kk + (lane >> 5)));
        } else {
            const s16x4 both[2] = {ds_read_tr16(s + rm_off<W>(16 * kk + tr_k, row + tr_c)),
                                   ds_read_tr16(s + rm_off<W>(16 * kk + tr_k + 4, row + tr_c))};
            return __builtin_bit_cast(bf16x8, both);
        }
    };
    auto read_frags = [&](int buf, int kk, int set) {
        const uint16_t* sA = smem + buf * STAGE;
        const uint16_t* sB = sA + BM * BK;
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa[set][i] = frag(std::integral_constant<int, AOP>{}, std::integral_constant<int, BM>{}, sA,
                              wm * (BM / WM) + i * 32, kk);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int col = DUAL ? (j >= TN / 2 ? BN / 2 : 0) + wn * (BN / WN / 2) + (j % (TN / 2 > 0 ? TN / 2 : 1)) * 32
                                 : wn * (BN / WN) + j * 32;
            fb[set][j] =
                frag(std::integral_constant<int, BOP>{}, std::integral_constant<int, BN>{}, sB, col, kk);
        }
    };
    auto mfmas = [&](int set) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[set][j], fa[set][i], acc[i][j], 0, 0, 0);
    };

    issue(s_first, 0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    read_frags(0, 0, 0);
    for (int s = s_first; s < s_end; ++s) {
        const int buf = (s - s_first) & 1;
        const bool more = s + 1 < s_end;
        if (more) issue(s + 1, buf ^ 1);
        read_frags(buf, 1, 1);
        mfmas(0);
        read_frags(buf, 2, 0);
        mfmas(1);
        read_frags(buf, 3, 1);
        mfmas(0);
        // the next stage has landed and every wave has read this one
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (more) read_frags(buf ^ 1, 0, 0);
        mfmas(1);
    }

    // ---- the sums through LDS (fp32), 8 adjacent columns a lane ------------------
    constexpr int CW = BN / WN;                         // staged columns per wave (dual: G half, then U half)
    constexpr int PW = CW + 4;                          // pitch: 16 bytes of padding per row
    constexpr int RPP = BM / WM >= 64 ? 64 : BM / WM;   // rows per pass
    constexpr int OW = DUAL ? CW / 2 : CW;              // output columns per wave
    constexpr int LPR = OW / 8;                         // lanes per row
    constexpr int RPI = 64 / LPR;                       // rows per wave step
    float* const st = reinterpret_cast<float*>(smem_raw) + wave * RPP * PW;
    const int row_base = m0 + wm * (BM / WM);
    const int col_base = n0 + wn * OW;
#pragma unroll
    for (int ps = 0; ps < BM / WM / RPP; ++ps) {
        __syncthreads();
#pragma unroll
        for (int ii = 0; ii < RPP / 32; ++ii)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x16& a = acc[ps * (RPP / 32) + ii][j];
                    *reinterpret_cast<f32x4*>(st + (ii * 32 + (lane & 31)) * PW + j * 32 + 8 * q + 4 * (lane >> 5)) =
                        f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
                }
        __syncthreads();
        for (int t = 0; t < RPP / RPI; ++t) {
            const int r = t * RPI + lane / LPR, c = 8 * (lane % LPR);
            const int m = row_base + ps * RPP + r, n = col_base + c;
            float x[8], y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            load8(st + r * PW + c, x);
            if constexpr (DUAL) load8(st + r * PW + OW + c, y);
            if (m < p.rows && n < p.cols) finish_or_part<DUAL, EPI>(p, split, m, n, x, y);
        }
    }
}

// ---------------------------------------------------------------------------
// The same product on 256 x 256 tiles (dual: 128 columns of each half), for
// outputs large enough to fill the CUs with them.  4 waves, 2 x 2, own 128 x 128
// sums each, all 256 accumulation registers of a wave.
//   A tile moves 64 KiB into a CU per 64-deep stage for 2048 matrix-core cycles;
//   what bounds it is having those loads in flight early enough.  Two whole
//   stages are 128 of the 160 KiB of LDS, so the ring is made of five 32 KiB half
//   stages (one operand's 256 x 64 each): stage s's b goes out as soon as stage
//   s - 2 has been read, a whole stage before it is needed, and its a another
//   three sub-steps earlier, into the fifth slot.
//   Each 16-deep sub-step is a fixed sequence (fenced, four matrix instructions
//   at a time) with the next sub-step's fragment reads and a share of the loads
//   between them; the waits are explicit: fragments at the start of the sub-step
//   that uses them, loads before the stage's one barrier, where only the a loads
//   of the stage after next may still be in flight.  Stages past the end load
//   the zero chunk, so every stage issues the same loads and the counts hold.
// ---------------------------------------------------------------------------
constexpr int WIDE_SLOT = 256 * BK;   // elements of a half stage

// Direct global -> LDS load of 16 bytes a lane that the compiler does not track:
// LDS byte address lds (uniform) + 16 * lane receives the lane's bytes.  With the
// tracked builtin, every transposing LDS read waits for all loads in flight
// (vmcnt(0)): it cannot know that they fill other slots.  There is no register to
// write early; the kernel waits with explicit counts, and the compiler's own
// waits for loads it does track only wait for more than they must.  (m0, which
// holds the LDS address, has no other use in the kernel.)
__device__ __forceinline__ void dma16_uniform(const uint16_t* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
                 : "memory");
}
__device__ __forceinline__ void dma16_lane(const uint16_t* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src)
                 : "memory");
}

// Work of one launch: the first workgroups, one per CU, compute tiles 0 .. full - 1
// whole, tile after tile, and start the next tile's loads before the epilogue of
// the last.  The R stages of the remaining tiles, fewer than there are CUs, are
// dealt out evenly to W further workgroups, which start as CUs fall free: worker w
// takes stages [w R / W, (w + 1) R / W) in order, at most two pieces, each the sums
// of part of one tile, which go to memory and are added by wide_reduce_kernel.  So
// no CU idles through a last round of whole tiles (448 tiles on 256 CUs), and
// outputs of a few tiles fill the CUs too.
struct WideRest {
    int pieces, tile, s0, s_first, s_second, slot;
};
__device__ __forceinline__ WideRest wide_rest(const GemmArgs& p, int KB, int W, int w) {
    const long long R = (long long)(p.tiles_m * p.tiles_n - p.full) * KB;
    const long long r0 = R * w / W, r1 = R * (w + 1) / W;
    WideRest r;
    r.tile = (int)(r0 / KB);
    r.s0 = (int)(r0 - (long long)r.tile * KB);
    const int len = (int)(r1 - r0);   // <= KB
    r.s_first = min(KB, r.s0 + len);
    r.s_second = r.s0 + len - KB;
    r.pieces = len == 0 ? 0 : (r.s_second > 0 ? 2 : 1);
    r.slot = 2 * w;
    return r;
}

// Whole tiles first, first + stride, ... < total (PIECES: the pieces of worker
// first of stride workers), one after another in one workgroup.
template <int AOP, int BOP, bool DUAL, int EPI, bool RAGGED, bool PIECES>
__device__ __forceinline__ void wide_tiles(const GemmArgs& p, uint16_t* smem, int first, int stride, int total) {
    constexpr int INS = 8;   // 1 KiB direct loads per wave and half stage
    constexpr int GROUP_M = 8;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;

    const int KB = p.segs * p.kb_seg;
    WideRest rest{};
    if constexpr (PIECES) rest = wide_rest(p, KB, stride, xcd_remap(first, stride));
    const int nitems = PIECES ? rest.pieces : (total - first + stride - 1) / stride;
    if (nitems <= 0) return;
    struct Item {
        int m0, n0, s0, s1;   // stages [s0, s1)
    };
    auto item_of = [&](int k) __attribute__((always_inline)) {
        Item it;
        int tile;
        if constexpr (PIECES) {
            tile = p.full + rest.tile + k;
            it.s0 = k ? 0 : rest.s0;
            it.s1 = k ? rest.s_second : rest.s_first;
        } else {
            tile = xcd_remap(first + k * stride, total);
            it.s0 = 0;
            it.s1 = KB;
        }
        const int per_group = GROUP_M * p.tiles_n;
        const int group = tile / per_group;
        const int first_m = group * GROUP_M;
        const int gsize = min(p.tiles_m - first_m, GROUP_M);
        const int in_group = tile - group * per_group;
        it.m0 = (first_m + in_group % gsize) * 256;
        it.n0 = (in_group / gsize) * (DUAL ? 128 : 256);
        return it;
    };

    // Byte offsets of a lane's 16 bytes in load i from the stage's base.
    // k-contiguous: load q = 8 wave + i brings rows 8q .. 8q + 7, lane l's chunk
    // is (l & 7) ^ (l >> 3) ^ (q & 7) (lds_off's swizzle); k-strided: k rows 2q
    // and 2q + 1, columns 8 ((l & 31) ^ 4 (k & 3)) (rm_off's).
    uint32_t a_off[INS], b_off[INS];
    int m0 = 0, n0 = 0, s_end = 0;   // of the item that the loads fetch
    const int hi5 = lane >> 5;
    auto ks_chunk = [&](int i) { return (lane & 31) ^ ((2 * (i & 1) + hi5) << 2); };
    // valid: false past the last item, whose loads then all read the zero chunk
    auto load_item = [&](const Item& it, bool valid) __attribute__((always_inline)) {
        m0 = it.m0;
        n0 = it.n0;
        s_end = valid ? it.s1 : 0;
#pragma unroll
    for (int i = 0; i < INS; ++i) {
        const int q = wave * INS + i;
        const int kc = 8 * ((lane & 7) ^ (lane >> 3) ^ i);
        if constexpr (AOP == OP_KC)
            a_off[i] = (uint32_t)((min(m0 + q * 8 + (lane >> 3), p.rows - 1) - m0) * p.lda + kc) * 2;
        else
            a_off[i] = (uint32_t)((2 * q + hi5) * p.lda + min(m0 + 8 * ks_chunk(i), p.rows - 8) - m0) * 2;
        if constexpr (BOP == OP_KC)
            b_off[i] = (uint32_t)((min(n0 + q * 8 + (lane >> 3), p.cols - 1) - n0) * p.ldb + kc) * 2;
        else
            b_off[i] = (uint32_t)((2 * q + hi5) * p.ldb +
                                  min(n0 + 8 * (ks_chunk(i) & (DUAL ? 15 : 31)), p.cols - 8) - n0) * 2;
    }
    };
    // dual: the lanes of a load's second half read the other matrix
    const uint16_t* const b_lane = (DUAL && (lane & 16)) ? p.B1 : p.B0;
    // the first k of a lane's chunk within the stage (RAGGED)
    const int kc_x = 8 * ((lane & 7) ^ (lane >> 3));
    auto lane_k = [&](int op, int i) { return op == OP_KC ? kc_x ^ (8 * i) : 2 * (wave * INS + i) + hi5; };

    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void_ptr)smem;
    // load i of operand a (or b) of stage s into ring slot `slot`
    auto issue = [&](auto bc, int s, int slot, int i) __attribute__((always_inline)) {
        constexpr bool ISB = decltype(bc)::value;
        constexpr int OP = ISB ? BOP : AOP;
        const bool valid = s < s_end;
        const int seg = s >= p.kb_seg ? 1 : 0;
        const int k0 = (s - seg * p.kb_seg) * BK;
        const long long ld = ISB ? p.ldb : p.lda;
        const int r0 = ISB ? n0 : m0;
        const uint32_t off = ISB ? b_off[i] : a_off[i];
        const size_t at = OP == OP_KC ? (size_t)r0 * ld + k0 : (size_t)k0 * ld + r0;
        const uint32_t dst = lds0 + (uint32_t)(slot * WIDE_SLOT + (wave * INS + i) * 512) * 2;
        if constexpr (!RAGGED && !(ISB && DUAL)) {
            const uint16_t* m = ISB ? (seg ? p.B1 : p.B0) : (seg ? p.A1 : p.A0);
            dma16_uniform(valid ? m + at : g_zeros, off & (valid ? 0xffffffffu : 0u), dst);
        } else {
            const uint16_t* m = ISB ? (DUAL ? b_lane : (seg ? p.B1 : p.B0)) : (seg ? p.A1 : p.A0);
            const uint16_t* src =
                reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(m + at) + off);
            if (!valid || (RAGGED && k0 + lane_k(OP, i) >= p.kseg)) src = g_zeros;
            dma16_lane(src, dst);
        }
    };
    using A_ = std::false_type;
    using B_ = std::true_type;

    // Fragment addresses: a few lane offsets and constants.  k-contiguous: rows
    // w*128 + 32i + (l & 31), chunk (2kk + (l >> 5)) ^ swz(row), and
    // swz(32i + r) = swz(r) ^ 4 (i & 1): four bases x = kk ^ 2 (i & 1).
    // k-strided: k row 16kk + 8 (l >> 5) + (l & 15) / 4, whose low bits fix the
    // swizzle for the lane, columns w*128 + 32i + ...: four bases, one per i.
    auto frag_bases = [&](int op, int w, bool dual, uint32_t (&base)[4]) {
        if (op == OP_KC) {
            const int r = lane & 31, hs = hi5 ^ swz(r);
#pragma unroll
            for (int x = 0; x < 4; ++x) base[x] = (uint32_t)(w * 128 * 128 + r * 128 + ((hs ^ (2 * x)) << 4));
        } else {
            const int k = 8 * hi5 + ((lane & 15) >> 2);
            const int c = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = dual ? (i >> 1) * 128 + w * 64 + (i & 1) * 32 : w * 128 + i * 32;
                base[i] = (uint32_t)rm_off<256>(k, col + c) * 2;
            }
        }
    };
    uint32_t a_base[4], b_base[4];
    frag_bases(AOP, wm, false, a_base);
    frag_bases(BOP, wn, DUAL, b_base);
    bf16x8 fa[2][4], fb[2][4];
    auto read_one = [&](int op, const uint32_t (&base)[4], uint32_t so, int kk, int i) -> bf16x8 {
        const char* sm = reinterpret_cast<const char*>(smem) + so;
        if (op == OP_KC)
            return *reinterpret_cast<const bf16x8*>(sm + i * 4096 + base[kk ^ (2 * (i & 1))]);
        const uint16_t* q = reinterpret_cast<const uint16_t*>(sm + kk * 8192 + base[i]);
        const s16x4 both[2] = {ds_read_tr16(q), ds_read_tr16(q + 1024)};
        return __builtin_bit_cast(bf16x8, both);
    };
    // byte offset of a ring slot, opaque so that addresses are formed from the
    // lane bases instead of being kept for every slot
    auto slot_off = [&](int slot) {
        uint32_t so = (uint32_t)slot * (WIDE_SLOT * 2);
        asm volatile("" : "+s"(so));
        return so;
    };

    f32x16 acc[4][4];
    auto zero_acc = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    };

    // one 16-deep sub-step on fragment set CUR: 16 matrix instructions, the next
    // sub-step's reads (sub-step rkk of the slots at aso, bso) in its first half,
    // and NLD loads per quarter of operand LB from load l0 on
    auto substep = [&](auto curc, uint32_t aso, uint32_t bso, int rkk, auto bc, auto nldc, int ls, int lslot, int l0) {
        constexpr int CUR = decltype(curc)::value;
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
                    fa[CUR ^ 1][t] = read_one(AOP, a_base, aso, rkk, t);
                    fb[CUR ^ 1][t] = read_one(BOP, b_base, bso, rkk, t);
                }
            }
#pragma unroll
            for (int t = 0; t < NLD; ++t) issue(bc, ls, lslot, l0 + i * NLD + t);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using C0 = std::integral_constant<int, 0>;
    using C1 = std::integral_constant<int, 1>;
    using C2 = std::integral_constant<int, 2>;

    // stage s in slots sa (a) and sa + 1 (b), modulo 5
    auto wrap = [](int x) { return x >= 5 ? x - 5 : x; };
    auto issue_first = [&](int s0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < INS; ++i) issue(A_{}, s0, 0, i);
#pragma unroll
        for (int i = 0; i < INS; ++i) issue(B_{}, s0, 1, i);
#pragma unroll
        for (int i = 0; i < INS; ++i) issue(A_{}, s0 + 1, 2, i);
#pragma unroll
        for (int i = 0; i < INS; ++i) issue(B_{}, s0 + 1, 3, i);
    };
    Item cur = item_of(0);
    load_item(cur, true);
    issue_first(cur.s0);
    for (int k = 0;;) {
        zero_acc();
        // stage s0 has landed once at most stage s0 + 1's loads are in flight
        // (the last item's stores are in the count too; loads complete in order
        // among themselves)
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * INS, 0));
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            fa[0][t] = read_one(AOP, a_base, 0u, 0, t);
            fb[0][t] = read_one(BOP, b_base, WIDE_SLOT * 2, 0, t);
        }
        int sa = 0;
        for (int s = cur.s0; s < cur.s1; ++s) {
            const uint32_t ao = slot_off(sa), bo = slot_off(wrap(sa + 1));
            __builtin_amdgcn_sched_barrier(0);
            substep(C0{}, ao, bo, 1, A_{}, C1{}, s + 2, wrap(sa + 4), 0);
            substep(C1{}, ao, bo, 2, A_{}, C1{}, s + 2, wrap(sa + 4), 4);
            substep(C0{}, ao, bo, 3, A_{}, C0{}, 0, 0, 0);
            // stage s + 1 has landed (only stage s + 2's a loads may be in
            // flight), and this wave has read stage s (its last reads fill the
            // next sub-step's fragments)
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(INS, 0));
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            const int sn = wrap(sa + 2);
            substep(C1{}, slot_off(sn), slot_off(wrap(sn + 1)), 0, B_{}, C2{}, s + 2, sa, 0);
            __builtin_amdgcn_sched_barrier(0);
            sa = sn;
        }
        // the sums stay in accumulation registers here (left to itself the
        // compiler copies all of them out at the loop's end, and spills)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[i][j]));
        // the zero-chunk loads past the end; then no wave reads the ring any more
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
        __builtin_amdgcn_s_barrier();
        // the next item's first stages stream in during this one's epilogue
        const bool more = k + 1 < nitems;
        const Item nxt = item_of(more ? k + 1 : k);
        load_item(nxt, more);
        issue_first(nxt.s0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (PIECES) {
            // a piece's sums as they lie in the lanes: [wave][i][j][q][lane][4]
            float* d = p.part + (size_t)(rest.slot + k) * 65536 + wave * 16384 + lane * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<f32x4*>(d + ((i * 4 + j) * 4 + q) * 256) =
                            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < (DUAL ? 2 : 4); ++j) {
                    // an opaque copy of the lane index: the block's addresses
                    // are formed here, not kept in registers across the item
                    int el = lane;
                    if constexpr (DUAL) asm volatile("" : "+v"(el), "+a"(acc[i][j]), "+a"(acc[i][j + 2]));
                    else asm volatile("" : "+v"(el), "+a"(acc[i][j]));
                    finish_block<EPI>(p, cur.m0, cur.n0, wm * 128 + i * 32, wn * (DUAL ? 64 : 128) + j * 32, el,
                                      acc[i][j], acc[i][DUAL ? j + 2 : j]);
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
        if (!more) break;
        cur = nxt;
        ++k;
    }
    // the loads past the last item
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
}

template <int AOP, int BOP, bool DUAL, int EPI, bool RAGGED>
__global__ __launch_bounds__(256) void wide_gemm_kernel(GemmArgs p, int whole, int workers) {
    __shared__ __attribute__((aligned(16))) uint16_t smem[5 * WIDE_SLOT];
    const int b = blockIdx.x;
    if (b < whole) wide_tiles<AOP, BOP, DUAL, EPI, RAGGED, false>(p, smem, b, whole, p.full);
    else wide_tiles<AOP, BOP, DUAL, EPI, RAGGED, true>(p, smem, b - whole, workers, workers);
}

// The pieces of the tiles past p.full, added in the order of the contraction
// (whatever workgroup finished first), then the epilogue: one wave per 32 x 32
// block (dual: pair of blocks), 4 to a workgroup.  workers: the product kernel's
// workgroups.
template <bool DUAL, int EPI>
__global__ __launch_bounds__(256) void wide_reduce_kernel(GemmArgs p, int workers) {
    constexpr int GROUP_M = 8;
    constexpr int BLOCKS = DUAL ? 32 : 64;   // per tile
    const int lane = threadIdx.x & 63;
    const int id = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rtile = id / BLOCKS, blk = id % BLOCKS;
    const int wv = blk / (BLOCKS / 4), i = blk / (BLOCKS / 16) % 4, j = blk % (BLOCKS / 16);
    const int KB = p.segs * p.kb_seg;
    const long long total = (long long)(p.tiles_m * p.tiles_n - p.full) * KB;
    // workers [w0, w1] hold the tile's stages
    const long long first = (long long)rtile * KB;
    int w = (int)(first * workers / total);
    while (total * (w + 1) / workers <= first) ++w;
    f32x16 x, y;
#pragma unroll
    for (int r = 0; r < 16; ++r) x[r] = y[r] = 0.0f;
    for (; w < workers && total * w / workers < first + KB; ++w) {
        if (total * w / workers == total * (w + 1) / workers) continue;
        const WideRest rest = wide_rest(p, KB, workers, w);
        const float* src = p.part + (size_t)(rest.slot + (rest.tile == rtile ? 0 : 1)) * 65536 + wv * 16384 + lane * 4;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(src + ((i * 4 + j) * 4 + q) * 256);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * q + e] += a[e];
            if constexpr (DUAL) {
                const f32x4 b = *reinterpret_cast<const f32x4*>(src + ((i * 4 + j + 2) * 4 + q) * 256);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[4 * q + e] += b[e];
            }
        }
    }
    const int tile = p.full + rtile;
    const int per_group = GROUP_M * p.tiles_n;
    const int group = tile / per_group;
    const int first_m = group * GROUP_M;
    const int gsize = min(p.tiles_m - first_m, GROUP_M);
    const int in_group = tile - group * per_group;
    finish_block<EPI>(p, (first_m + in_group % gsize) * 256, (in_group / gsize) * (DUAL ? 128 : 256),
                      (wv & 1) * 128 + i * 32, (wv >> 1) * (DUAL ? 64 : 128) + j * 32, lane, x, y);
}

// The splits' sums of 8 adjacent columns, added in split order 0 .. splits - 1
// (the same result whatever workgroup finished first), then the epilogue.
template <bool DUAL, int EPI>
__global__ __launch_bounds__(256) void tile_reduce_kernel(GemmArgs p) {
    const long long groups = (long long)p.rows * (p.cols / 8);
    const size_t stride = (size_t)p.rows * p.part_cols;
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < groups; t += (long long)gridDim.x * 256) {
        const int m = (int)(t / (p.cols / 8)), n = (int)(t % (p.cols / 8)) * 8;
        const float* src = p.part + (size_t)m * p.part_cols + n;
        float x[8] = {}, y[8] = {};
        for (int s = 0; s < p.splits; ++s, src += stride) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(src + 4 * h);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * h + e] += v[e];
                if constexpr (DUAL) {
                    const f32x4 w = *reinterpret_cast<const f32x4*>(src + p.cols + 4 * h);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[4 * h + e] += w[e];
                }
            }
        }
        finish8<EPI>(p, m, n, x, y);
    }
}

// D = [dG | dU] from dY and the kept G and U, 8 elements a thread.
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
