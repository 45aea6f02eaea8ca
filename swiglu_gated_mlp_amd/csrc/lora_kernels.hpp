// Kernels of the low-rank adapters: the pack, the factor t = s_i (A La_i), the
// reduction of splits with adapters, and the adapted forms of the streaming and
// decode kernels (their adapter step is lora_device.hpp).
#pragma once

#include "fused_kernels.hpp"
#include "lora_device.hpp"

namespace swk {

// ---------------------------------------------------------------------------
// Pack.  Adapters' factors La [L][K][r] and Lb [L][r][N] (two pairs for the gated
// product) become
//   part A  [adapter][tile][64-deep k block][32-deep half][lane][8], tile
//           t = group * chunks + chunk: lane l holds the tile's number l % 16
//           (of 16) and the 8 k from 8 (l / 16) of its half: one wave load is
//           one 1 KiB operand fragment of v_mfma_f32_16x16x32_bf16
//   part B  Lb as in lora_device.hpp
// one thread per 16 bytes, padding zero.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void lora_pack_kernel(const uint16_t* __restrict__ La1,
                                                        const uint16_t* __restrict__ La2,
                                                        const uint16_t* __restrict__ Lb1,
                                                        const uint16_t* __restrict__ Lb2, uint16_t* __restrict__ out,
                                                        int groups, int K, int N, int r, int chunks, int KB,
                                                        int ntiles, long long pieces_a, long long pieces) {
    for (long long q = (long long)blockIdx.x * 256 + threadIdx.x; q < pieces; q += (long long)gridDim.x * 256) {
        unsigned short v[8];
        if (q < pieces_a) {
            const int lane = (int)(q & 63), half = (int)((q >> 6) & 1);
            long long x = q >> 7;
            const int kb = (int)(x % KB);
            x /= KB;
            const int t = (int)(x % (groups * chunks));
            const long long l = x / (groups * chunks);
            const int j = (t % chunks) * 16 + (lane & 15);
            const int k0 = kb * 64 + half * 32 + 8 * (lane >> 4);
            const uint16_t* src = (t / chunks ? La2 : La1) + (size_t)l * K * r;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = (j < r && k0 + e < K) ? src[(size_t)(k0 + e) * r + j] : (unsigned short)0;
        } else {
            long long x = q - pieces_a;
            const int lane = (int)(x & 63);
            x >>= 6;
            const int g = (int)(x % groups);
            x /= groups;
            const int nt = (int)(x % ntiles);
            x /= ntiles;
            const int c = (int)(x % chunks);
            const long long l = x / chunks;
            const int n = nt * 32 + (lane & 31), j0 = c * 16 + 8 * (lane >> 5);
            const uint16_t* src = (g ? Lb2 : Lb1) + (size_t)l * r * N;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (n < N && j0 + e < r) ? src[(size_t)(j0 + e) * N + n] : (unsigned short)0;
        }
        u32x4 o;
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = (unsigned)v[2 * d] | ((unsigned)v[2 * d + 1] << 16);
        *reinterpret_cast<u32x4*>(out + q * 8) = o;
    }
}

// ---------------------------------------------------------------------------
// T: t = s_i (A[m] La_i) as hi + lo.  A workgroup takes 16 rows and TT tiles of
// 16 of the r numbers; its WAVES waves share the k blocks round-robin and add
// their fp32 sums in LDS in wave order.  The rows' adapters are taken one after
// another (gridDim.z workgroups share them), each as the first operand of
// v_mfma_f32_16x16x32_bf16 against all 16 rows; a row keeps its own adapter's.
// The kernel reads A and the used adapters' La once: it is bound by those loads
// (and, for a few rows, by their latency, hence many waves on one row block).
// ---------------------------------------------------------------------------
struct LoraShrinkArgs {
    const uint16_t* A;      // [M][K]
    const uint16_t* P;      // part A of the pack
    const int* ids;
    const float* scales;
    uint16_t* T;
    int M, K, KB, adapters, groups, chunks, rank;
};

template <int WAVES, int TT>
__global__ __launch_bounds__(64 * WAVES) void lora_shrink_kernel(LoraShrinkArgs p) {
    __shared__ f32x4 red[WAVES][TT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = lane & 15, kq = lane >> 4;
    const int m = blockIdx.x * 16 + row;
    const int tiles = p.groups * p.chunks;
    const int t0 = blockIdx.y * TT;
    int id = -1;
    if (m < p.M) {
        id = p.ids[m];
        if (id < 0 || id >= p.adapters) id = -1;
    }
    const uint16_t* arow = p.A + (size_t)min(m, p.M - 1) * p.K + 8 * kq;
    unsigned long long pend = __ballot(id >= 0);
    for (int d = 0; pend; ++d) {
        const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(pend));
        pend &= ~__ballot(id == e);
        if (d % (int)gridDim.z != (int)blockIdx.z) continue;
        f32x4 acc[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int kb = wave; kb < p.KB; kb += WAVES) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = kb * 64 + 32 * h;
                u32x4 av = {0u, 0u, 0u, 0u};
                if (k + 8 * kq < p.K) av = ld16(arow + k);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const int tt = min(t0 + t, tiles - 1);
                    const u32x4 w =
                        ld16(p.P + ((((size_t)e * tiles + tt) * p.KB + kb) * 2 + h) * 512 + lane * 8);
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w),
                                                                     __builtin_bit_cast(bf16x8, av), acc[t], 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) red[wave][t][lane] = acc[t];
        __syncthreads();
        for (int t = wave; t < TT; t += WAVES) {
            const int tt = t0 + t;
            f32x4 v = red[0][t][lane];
            for (int w = 1; w < WAVES; ++w) v += red[w][t][lane];
            if (id == e && tt < tiles) {
                const int g = tt / p.chunks, c = tt % p.chunks, j0 = 4 * kq;
                float hi[4], lo[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    // padding stays zero even where A holds infinities
                    const float t1 = c * 16 + j0 + q < p.rank ? v[q] * p.scales[e] : 0.0f;
                    hi[q] = __builtin_bit_cast(float, bf16_bits(t1) << 16);
                    // an infinite t has no remainder
                    lo[q] = __builtin_fabsf(hi[q]) < __builtin_inff() ? t1 - hi[q] : 0.0f;
                }
                uint16_t* dst = p.T + (((size_t)m * p.chunks + c) * p.groups + g) * 32 + j0;
                *reinterpret_cast<u32x2*>(dst) = u32x2{pack2(hi[0], hi[1]), pack2(hi[2], hi[3])};
                *reinterpret_cast<u32x2*>(dst + 16) = u32x2{pack2(lo[0], lo[1]), pack2(lo[2], lo[3])};
            }
        }
        __syncthreads();   // the sums are read before the next adapter's are written
    }
}

// ---------------------------------------------------------------------------
// The splits' sums, added in split order, then the adapter's part, then the
// epilogue: gated (NT = N: the Gate sum of column n at n, the Up sum at N + n) or,
// GEMM, the single-weight pack's tiled columns (n: output column
// (n / 128) 256 + n % 128, and that + 128 at NT + n).
// ---------------------------------------------------------------------------
template <bool GEMM>
__global__ __launch_bounds__(256) void lora_reduce_kernel(const float* __restrict__ part, uint16_t* __restrict__ Y,
                                                          LoraArgs la, int M, int N, int NT, int S) {
    const long long groups = (long long)M * (NT / 4);
    const size_t split_stride = (size_t)M * 2 * (size_t)NT;
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < groups; t += (long long)gridDim.x * 256) {
        const int m = (int)(t / (NT / 4)), n = (int)(t % (NT / 4)) * 4;
        const float* src = part + (size_t)m * 2 * (size_t)NT + n;
        f32x4 g = *reinterpret_cast<const f32x4*>(src), u = *reinterpret_cast<const f32x4*>(src + NT);
        for (int s = 1; s < S; ++s) {
            g += *reinterpret_cast<const f32x4*>(src + s * split_stride);
            u += *reinterpret_cast<const f32x4*>(src + s * split_stride + NT);
        }
        const int id = lora_id(la, m);
        if constexpr (GEMM) {
            const int col = (n / PACK_BN) * PACK_ROWS + n % PACK_BN;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int cn = col + half * PACK_BN;
                if (cn >= N) continue;
                f32x4 v = half ? u : g;
                if (id >= 0) v += lora_delta4<1>(la, m, id, 0, cn);
                *reinterpret_cast<u32x2*>(Y + (size_t)m * N + cn) = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
            }
        } else {
            if (id >= 0) {
                g += lora_delta4<2>(la, m, id, 0, n);
                u += lora_delta4<2>(la, m, id, 1, n);
            }
            *reinterpret_cast<u32x2*>(Y + (size_t)m * N + n) =
                u32x2{pack2(silu_f(g[0]) * u[0], silu_f(g[1]) * u[1]), pack2(silu_f(g[2]) * u[2], silu_f(g[3]) * u[3])};
        }
    }
}

// ---------------------------------------------------------------------------
// The streaming kernels with adapters (the decode kernel takes LoraArgs itself).
// ---------------------------------------------------------------------------
template <int BM, bool RAGGED, bool PANELS, bool GEMM>
__global__ __launch_bounds__(256) void stream_lora_kernel(FusedArgs p, LoraArgs la, int total) {
    __shared__ __attribute__((aligned(16))) uint16_t smem[stream_smem_elems<BM>()];
    stream_prefill_tiles<BM, false, RAGGED, PANELS, false, false, false, GEMM, true>(p, smem, blockIdx.x, gridDim.x,
                                                                                    total, &la);
}

template <bool RAGGED, bool GEMM>
__global__ __launch_bounds__(256) void stream_lora_mixed_kernel(FusedArgs big, FusedArgs tail, LoraArgs la, int n_pers,
                                                                int n_big) {
    __shared__ __attribute__((aligned(16))) uint16_t smem[stream_smem_elems<256>()];
    const int b = blockIdx.x;
    if (b < n_pers) {
        stream_prefill_tiles<256, false, RAGGED, false, false, false, false, GEMM, true>(big, smem, b, n_pers, n_big,
                                                                                        &la);
    } else {
        const int n_tail = gridDim.x - n_pers;
        stream_prefill_tiles<128, false, RAGGED, false, false, false, false, GEMM, true>(tail, smem, b - n_pers, n_tail,
                                                                                        n_tail, &la);
    }
}

}  // namespace swk
