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
//   flags   [adapter] int32: 1 where the adapter's Lb holds an infinity or NaN
// one thread per 16 bytes, padding zero; the flags, zero before, by a second launch.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void lora_pack_kernel(const uint16_t* __restrict__ La1,
                                                        const uint16_t* __restrict__ La2,
                                                        const uint16_t* __restrict__ Lb1,
                                                        const uint16_t* __restrict__ Lb2, uint16_t* __restrict__ out,
                                                        int groups, int K, int N, int r, int chunks, int KB,
                                                        int ntiles, long long pieces_a, long long pieces_b,
                                                        long long pieces) {
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
        } else if (q >= pieces_a + pieces_b) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0;   // flags
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

// pieces: 16-byte pieces of an adapter's Lb; `share` workgroups an adapter, and all
// that find one store the same 1.
__global__ __launch_bounds__(256) void lora_flag_kernel(const uint16_t* __restrict__ B, int* __restrict__ flags,
                                                        long long pieces, int share, int adapters) {
    for (int l = blockIdx.x / share; l < adapters; l += gridDim.x / share) {
        const u32x4* b = reinterpret_cast<const u32x4*>(B) + l * pieces;
        bool odd = false;
        for (long long i = (long long)(blockIdx.x % share) * 256 + threadIdx.x; i < pieces; i += (long long)share * 256) {
            const u32x4 v = b[i];
#pragma unroll
            for (int q = 0; q < 4; ++q)   // exponent bits all set
                odd = odd || (v[q] & 0x7F80u) == 0x7F80u || (v[q] & 0x7F800000u) == 0x7F800000u;
        }
        if (odd) flags[l] = 1;
    }
}

// ---------------------------------------------------------------------------
// T: t = s_i (A[m] La_i).  A workgroup takes 16 rows and TT tiles of 16 of the r
// numbers, over part blockIdx.z % parts of the contraction; its 16 waves share the
// k blocks round-robin, two in flight each, and add their fp32 sums in LDS in wave
// order.  The rows' adapters are taken one after another (the gridDim.z / parts
// workgroups of a block share them), each as the first operand of
// v_mfma_f32_16x16x32_bf16 against all 16 rows; a row keeps its own adapter's.
// A workgroup reads its rows of A and the used adapters' La: with few rows it is
// bound by how much one CU loads (a K = 18944 adapter of rank 16 and 16 rows are
// 1.2 MB: 24 us in one workgroup, 7.5 us in 8 parts), hence the parts, which the
// readers of T add up; with many, by latency and La from the L2, hence many waves a
// row block (7B width, 2100 rows, rank 32: 33 us with 4 waves, 16 us with 16).
// PARTS: fp32 parts of T (parts = 1 otherwise).  Else hi and lo, and the row tile's
// adapter list, formed by the tile's first workgroup from its ids: at most
// LORA_PLACES adapters, none flagged.
// ---------------------------------------------------------------------------
struct LoraShrinkArgs {
    const uint16_t* A;      // [M][K]
    const uint16_t* P;      // part A of the pack
    const int* ids;
    const float* scales;
    const int* flags;       // of the pack
    uint16_t* T;
    int* lists;
    float* Tf;
    int M, K, KB, adapters, groups, chunks, rank, parts;
    int unit;
};

template <int TT, bool PARTS>
__global__ __launch_bounds__(1024) void lora_shrink_kernel(LoraShrinkArgs p) {
    constexpr int WAVES = 16, UNROLL = 2;
    __shared__ f32x4 red[WAVES][TT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = lane & 15, kq = lane >> 4;
    const int m = blockIdx.x * 16 + row;
    const int tiles = p.groups * p.chunks;
    const int t0 = blockIdx.y * TT;
    const int part = PARTS ? (int)blockIdx.z % p.parts : 0;
    const int first_d = PARTS ? (int)blockIdx.z / p.parts : (int)blockIdx.z;
    const int step_d = PARTS ? (int)gridDim.z / p.parts : (int)gridDim.z;
    const int kb0 = PARTS ? (int)((long long)p.KB * part / p.parts) : 0;
    const int kb1 = PARTS ? (int)((long long)p.KB * (part + 1) / p.parts) : p.KB;
    int id = -1;
    if (m < p.M) {
        id = p.ids[m];
        if (id < 0 || id >= p.adapters) id = -1;
    }
    const uint16_t* arow = p.A + (size_t)min(m, p.M - 1) * p.K + 8 * kq;
    if constexpr (!PARTS) {
        const int tile = blockIdx.x * 16 / p.unit, r0 = tile * p.unit;
        if ((int)blockIdx.x * 16 == r0 && blockIdx.y == 0 && blockIdx.z == 0 && wave == 0) {
            int ids[4], list[LORA_PLACES], len = 0;
            unsigned long long left[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = r0 + 64 * q + lane;
                ids[q] = 64 * q < p.unit && r < p.M ? p.ids[r] : -1;
                if (ids[q] >= p.adapters) ids[q] = -1;
                left[q] = __ballot(ids[q] >= 0);
            }
#pragma unroll
            for (int j = 0; j <= LORA_PLACES; ++j) {
                int e = -1;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (e < 0 && left[q]) e = __builtin_amdgcn_readlane(ids[q], __builtin_ctzll(left[q]));
                if (j < LORA_PLACES) list[j < LORA_PLACES ? j : 0] = e;
                if (e >= 0 && len >= 0) len = j == LORA_PLACES || p.flags[e] ? -1 : len + 1;
#pragma unroll
                for (int q = 0; q < 4; ++q) left[q] &= ~__ballot(ids[q] == e);
            }
            if (lane == 0) {
                p.lists[tile * LORA_LIST] = len;
#pragma unroll
                for (int j = 0; j < LORA_PLACES; ++j) p.lists[tile * LORA_LIST + 1 + j] = list[j];
            }
        }
    }
    unsigned long long pend = __ballot(id >= 0);
    for (int d = 0; pend; ++d) {
        const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(pend));
        pend &= ~__ballot(id == e);
        if (d % step_d != first_d) continue;
        f32x4 acc[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int kw = kb0 + wave; kw < kb1; kw += WAVES * UNROLL) {
            u32x4 av[UNROLL][2], wv[UNROLL][2][TT];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int kb = kw + u * WAVES;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = kb * 64 + 32 * h;
                    av[u][h] = u32x4{0u, 0u, 0u, 0u};
                    if (kb < kb1 && k + 8 * kq < p.K) av[u][h] = ld16(arow + k);
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        const int tt = min(t0 + t, tiles - 1);
                        // past the part's end: a block that is not used below
                        wv[u][h][t] = ld16(
                            p.P + ((((size_t)e * tiles + tt) * p.KB + (kb < kb1 ? kb : kw)) * 2 + h) * 512 + lane * 8);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                if (kw + u * WAVES < kb1) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int t = 0; t < TT; ++t)
                            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv[u][h][t]),
                                                                             __builtin_bit_cast(bf16x8, av[u][h]),
                                                                             acc[t], 0, 0, 0);
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
                float t1[4], hi[4], lo[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    // padding stays zero even where A holds infinities
                    t1[q] = c * 16 + j0 + q < p.rank ? v[q] * p.scales[e] : 0.0f;
                    hi[q] = __builtin_bit_cast(float, bf16_bits(t1[q]) << 16);
                    // an infinite t has no remainder
                    lo[q] = __builtin_fabsf(hi[q]) < __builtin_inff() ? t1[q] - hi[q] : 0.0f;
                }
                if constexpr (PARTS) {
                    *reinterpret_cast<f32x4*>(
                        p.Tf + ((((size_t)part * p.M + m) * p.chunks + c) * p.groups + g) * 16 + j0) =
                        f32x4{t1[0], t1[1], t1[2], t1[3]};
                } else {
                    uint16_t* dst = p.T + (((size_t)(m >> 5) * p.chunks + c) * p.groups + g) * 1024 +
                                    ((m & 31) + 32 * (j0 >> 3)) * 8 + (j0 & 7);
                    *reinterpret_cast<u32x2*>(dst) = u32x2{pack2(hi[0], hi[1]), pack2(hi[2], hi[3])};
                    *reinterpret_cast<u32x2*>(dst + 512) = u32x2{pack2(lo[0], lo[1]), pack2(lo[2], lo[3])};
                }
            }
        }
        __syncthreads();   // the sums are read before the next adapter's are written
    }
}

// ---------------------------------------------------------------------------
// delta = t Lb, [M][groups N] fp32, zero for rows without adapter: one thread per
// row and four columns of a group; eight threads read 512 contiguous bytes of an
// adapter's Lb, eight rows a wave, so rows of any adapters load side by side.
// 7B width, 32 rows of 32 requests, rank 16: 9 us for 34 MB of Lb and 4.8 MB of
// delta, 4.3 TB/s.
// ---------------------------------------------------------------------------
template <int GROUPS>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs la, float* __restrict__ delta) {
    const int q = blockIdx.x * 8 + (threadIdx.x & 7);          // column quad over both groups
    const int m = blockIdx.y * 32 + (threadIdx.x >> 3);
    const int quads = la.N / 4;
    if (m >= la.M || q >= GROUPS * quads) return;
    const int g = q / quads, n = (q - g * quads) * 4;
    const int id = lora_id(la, m);
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    if (id >= 0) d = lora_delta4<GROUPS>(la, m, id, g, n);
    *reinterpret_cast<f32x4*>(delta + ((size_t)m * GROUPS + g) * la.N + n) = d;
}

// ---------------------------------------------------------------------------
// The splits' sums, added in split order, then the adapter's part, then the
// epilogue: gated (NT = N: the Gate sum of column n at n, the Up sum at N + n) or,
// GEMM, the single-weight pack's tiled columns (n: output column
// (n / 128) 256 + n % 128, and that + 128 at NT + n).  One wave per 32 x 32 block:
// lora_block forms the adapters' part in a matrix instruction's lanes, LDS turns it
// into rows, and the sums are read and the outputs stored along rows (eight lanes
// to 128 bytes of sums: in the other order, 32 rows a load at a stride of a whole
// row, the kernel took 45 us for 2000 x 896 outputs of rank 64, this way 20; with
// the adapters' part on the vector units 30).
// ---------------------------------------------------------------------------
template <bool GEMM>
__global__ __launch_bounds__(256) void lora_reduce_kernel(const float* __restrict__ part, uint16_t* __restrict__ Y,
                                                          LoraArgs la, int M, int N, int NT, int S) {
    constexpr int P = 36;   // pitch of a block's row in LDS
    __shared__ float rows[4][2][32 * P];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int w = blockIdx.x * 4 + wave;
    const int ctiles = (NT + 31) / 32;
    const int i = w / ctiles, n0 = (w - i * ctiles) * 32;
    const bool work = i * 32 < M;
    // the block's sums: row 8 t + lane / 8, four columns
    const size_t stride = (size_t)M * 2 * (size_t)NT;
    const int n = n0 + 4 * (lane & 7);
    f32x4 g[4], u[4];
    // the columns' adapters: gated, both groups of one tile; GEMM, two tiles
    const int col = GEMM ? (n0 / PACK_BN) * PACK_ROWS + n0 % PACK_BN : n0;
    if (work && !la.delta) {
        const int m = i * 32 + (lane & 31);
        const int nt[2] = {col / 32, (GEMM ? col + PACK_BN : col) / 32};
        f32x16 x[2] = {};
        lora_block<2, GEMM ? 1 : 2>(x, la, m < M ? lora_id(la, m) : -1, m, nt, lane);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4*>(&rows[wave][h][(lane & 31) * P + 8 * q + 4 * (lane >> 5)]) =
                    f32x4{x[h][4 * q], x[h][4 * q + 1], x[h][4 * q + 2], x[h][4 * q + 3]};
    }
    __syncthreads();
    if (!work || n >= NT) return;
    const float* src = part + (size_t)(i * 32 + (lane >> 3)) * 2 * (size_t)NT + n;
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float* q = src + s * stride + t * (size_t)16 * NT;
            f32x4 x[2] = {};
            if (i * 32 + 8 * t + (lane >> 3) < M) {
                x[0] = *reinterpret_cast<const f32x4*>(q);
                x[1] = *reinterpret_cast<const f32x4*>(q + NT);
            }
            g[t] = s == 0 ? x[0] : g[t] + x[0];
            u[t] = s == 0 ? x[1] : u[t] + x[1];
        }
    const int oc = GEMM ? (n / PACK_BN) * PACK_ROWS + n % PACK_BN : n;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int r = 8 * t + (lane >> 3), m = i * 32 + r;
        if (m >= M) continue;
        if (la.delta) {
            g[t] += lora_read4(la, GEMM ? 1 : 2, m, 0, oc);
            u[t] += lora_read4(la, GEMM ? 1 : 2, m, GEMM ? 0 : 1, GEMM ? oc + PACK_BN : oc);
        } else {
            g[t] += *reinterpret_cast<const f32x4*>(&rows[wave][0][r * P + 4 * (lane & 7)]);
            u[t] += *reinterpret_cast<const f32x4*>(&rows[wave][1][r * P + 4 * (lane & 7)]);
        }
        if constexpr (GEMM) {
            if (oc < N)
                *reinterpret_cast<u32x2*>(Y + (size_t)m * N + oc) = u32x2{pack2(g[t][0], g[t][1]), pack2(g[t][2], g[t][3])};
            if (oc + PACK_BN < N)
                *reinterpret_cast<u32x2*>(Y + (size_t)m * N + oc + PACK_BN) =
                    u32x2{pack2(u[t][0], u[t][1]), pack2(u[t][2], u[t][3])};
        } else {
            *reinterpret_cast<u32x2*>(Y + (size_t)m * N + n) =
                u32x2{pack2(silu_f(g[t][0]) * u[t][0], silu_f(g[t][1]) * u[t][1]),
                      pack2(silu_f(g[t][2]) * u[t][2], silu_f(g[t][3]) * u[t][3])};
        }
    }
}

// ---------------------------------------------------------------------------
// The streaming kernels with adapters (the decode kernel takes LoraArgs itself).
// ---------------------------------------------------------------------------
template <int BM, bool RAGGED, bool PANELS, bool GEMM, int LORA>
__global__ __launch_bounds__(256) void stream_lora_kernel(FusedArgs p, LoraArgs la, int total) {
    __shared__ __attribute__((aligned(16))) uint16_t smem[stream_smem_elems<BM>()];
    stream_prefill_tiles<BM, false, RAGGED, PANELS, false, false, false, GEMM, LORA>(p, smem, blockIdx.x, gridDim.x,
                                                                                    total, &la);
}

template <bool RAGGED, bool GEMM>
__global__ __launch_bounds__(256) void stream_lora_mixed_kernel(FusedArgs big, FusedArgs tail, LoraArgs la, int n_pers,
                                                                int n_big) {
    __shared__ __attribute__((aligned(16))) uint16_t smem[stream_smem_elems<256>()];
    const int b = blockIdx.x;
    if (b < n_pers) {
        stream_prefill_tiles<256, false, RAGGED, false, false, false, false, GEMM, 1>(big, smem, b, n_pers, n_big,
                                                                                        &la);
    } else {
        const int n_tail = gridDim.x - n_pers;
        stream_prefill_tiles<128, false, RAGGED, false, false, false, false, GEMM, 1>(tail, smem, b - n_pers, n_tail,
                                                                                        n_tail, &la);
    }
}

}  // namespace swk
