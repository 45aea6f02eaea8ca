// Kernels of the products that are no templates: the reductions of split-K sums, the
// FP8 weights' pack and the element-wise SwiGLU.  Only swiglu_api.hip launches them,
// and includes them.
#pragma once

#include "fused_kernels.hpp"

namespace swk {

// Y[m, n..n+3] = bf16(SiLU(sum_s G_s) * sum_s U_s), splits added in order
// 0..S-1 (so the result does not depend on which workgroup finished first).
// One thread per 4 outputs, grid-stride.
__global__ __launch_bounds__(256) void splitk_reduce_kernel(const float* __restrict__ part,
                                                            uint16_t* __restrict__ Y, int M, int N,
                                                            int S) {
    const long long groups = (long long)M * (N / 4);
    const size_t split_stride = (size_t)M * 2 * (size_t)N;
    for (long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x; t < groups;
         t += (long long)gridDim.x * blockDim.x) {
        const int m = (int)(t / (N / 4));
        const int n = (int)(t % (N / 4)) * 4;
        const float* src = part + (size_t)m * 2 * (size_t)N + n;
        f32x4 g = *reinterpret_cast<const f32x4*>(src);
        f32x4 u = *reinterpret_cast<const f32x4*>(src + N);
        for (int s2 = 1; s2 < S; ++s2) {
            g += *reinterpret_cast<const f32x4*>(src + s2 * split_stride);
            u += *reinterpret_cast<const f32x4*>(src + s2 * split_stride + N);
        }
        u32x2 out;
        out[0] = pack2(silu_f(g[0]) * u[0], silu_f(g[1]) * u[1]);
        out[1] = pack2(silu_f(g[2]) * u[2], silu_f(g[3]) * u[3]);
        *reinterpret_cast<u32x2*>(Y + (size_t)m * N + n) = out;
    }
}

// The single-weight GEMM's split-K reduction: partials [split][M][2*NT] over
// the NT tiled columns of the pack (the "Gate" sum of tiled column n is output
// column (n / 128) * 256 + n % 128, the "Up" sum that column + 128), added in
// split order 0..S-1 and stored as bf16; output columns >= N are skipped.
__global__ __launch_bounds__(256) void splitk_gemm_reduce_kernel(const float* __restrict__ part,
                                                                 uint16_t* __restrict__ C, int M, int N, int NT,
                                                                 int S) {
    const long long groups = (long long)M * (NT / 4);
    const size_t split_stride = (size_t)M * 2 * (size_t)NT;
    for (long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x; t < groups;
         t += (long long)gridDim.x * blockDim.x) {
        const int m = (int)(t / (NT / 4));
        const int n = (int)(t % (NT / 4)) * 4;
        const float* src = part + (size_t)m * 2 * (size_t)NT + n;
        f32x4 g = *reinterpret_cast<const f32x4*>(src);
        f32x4 u = *reinterpret_cast<const f32x4*>(src + NT);
        for (int s2 = 1; s2 < S; ++s2) {
            g += *reinterpret_cast<const f32x4*>(src + s2 * split_stride);
            u += *reinterpret_cast<const f32x4*>(src + s2 * split_stride + NT);
        }
        const int col = (n / PACK_BN) * PACK_ROWS + n % PACK_BN;
        if (col < N) {
            u32x2 out;
            out[0] = pack2(g[0], g[1]);
            out[1] = pack2(g[2], g[3]);
            *reinterpret_cast<u32x2*>(C + (size_t)m * N + col) = out;
        }
        if (col + PACK_BN < N) {
            u32x2 out;
            out[0] = pack2(u[0], u[1]);
            out[1] = pack2(u[2], u[3]);
            *reinterpret_cast<u32x2*>(C + (size_t)m * N + col + PACK_BN) = out;
        }
    }
}

// ---------------------------------------------------------------------------
// FP8 weight pack: per (128-column tile jt, 128-k block kb) one 32 KiB block
// [32-row block rb][64-k step ks][half h][lane][16 bytes], holding packed row
// rb*32 + (lane & 31) (rows 0-127: W1 column jt*128 + row, 128-255: W2 column
// jt*128 + row - 128) at k = kb*128 + ks*64 + 32*(lane >> 5) + 16*h + 0..15:
// the lane order of a v_mfma_f32_32x32x64_f8f6f4 operand, each half of a
// lane's 32 bytes in its own 1 KiB run so that one wave load reads 1 KiB
// contiguous.  Padding is zero.  One thread per 16-byte piece (piece index =
// byte offset / 16).
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void pack_fp8_kernel(const uint8_t* __restrict__ W1,
                                                       const uint8_t* __restrict__ W2,
                                                       uint8_t* __restrict__ Wp, int K, int N, int KB,
                                                       long long npieces) {
    const long long q = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (q >= npieces) return;
    const long long blk = q >> 11;
    const int within = (int)(q & 2047);
    const int rb = within >> 8, ks = (within >> 7) & 1, half = (within >> 6) & 1, lane = within & 63;
    const int kb = (int)(blk % KB), jt = (int)(blk / KB);
    const int prow = rb * 32 + (lane & 31);
    const bool up = prow >= PACK_BN;
    const int n = jt * PACK_BN + (up ? prow - PACK_BN : prow);
    const int k0 = kb * 128 + ks * 64 + 32 * (lane >> 5) + 16 * half;
    const uint8_t* W = up ? W2 : W1;
    u32x4 out = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const unsigned v = (n < N && k0 + i < K) ? W[(size_t)(k0 + i) * N + n] : 0u;
        out[i >> 2] |= v << (8 * (i & 3));
    }
    *reinterpret_cast<u32x4*>(Wp + q * 16) = out;
}

// ---------------------------------------------------------------------------
// Element-wise SwiGLU of the unfused pipeline: Y = bf16(SiLU(G) * U), fp32 math.
// 8 elements (16 bytes) per thread per step, grid-stride; scalar tail.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void silu_mul_kernel(const uint16_t* __restrict__ G,
                                                       const uint16_t* __restrict__ U,
                                                       uint16_t* __restrict__ Y, long long count) {
    const long long nvec = count / 8;
    const long long stride = (long long)gridDim.x * blockDim.x;
    for (long long v = (long long)blockIdx.x * blockDim.x + threadIdx.x; v < nvec; v += stride) {
        const u32x4 g = *reinterpret_cast<const u32x4*>(G + v * 8);
        const u32x4 u = *reinterpret_cast<const u32x4*>(U + v * 8);
        u32x4 y;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const float g0 = __builtin_bit_cast(float, g[d] << 16);
            const float g1 = __builtin_bit_cast(float, g[d] & 0xFFFF0000u);
            const float u0 = __builtin_bit_cast(float, u[d] << 16);
            const float u1 = __builtin_bit_cast(float, u[d] & 0xFFFF0000u);
            y[d] = pack2(silu_f(g0) * u0, silu_f(g1) * u1);
        }
        *reinterpret_cast<u32x4*>(Y + v * 8) = y;
    }
    const long long t = nvec * 8 + (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (t < count && blockIdx.x == 0 && (long long)threadIdx.x < count - nvec * 8) {
        const float g0 = __builtin_bit_cast(float, (unsigned)G[t] << 16);
        const float u0 = __builtin_bit_cast(float, (unsigned)U[t] << 16);
        Y[t] = (uint16_t)bf16_bits(silu_f(g0) * u0);
    }
}

}  // namespace swk
