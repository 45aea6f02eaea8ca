// Device kernels of the int8 calls besides the products (swiglu_*_int8): quantizing
// rows and columns, and the weight packs.  The products run on the packed kernels of
// fused_kernels.hpp with I8 and on narrow_kernel (int8_narrow.hpp).
//
// Symmetric quantization: x = s q, q whole in -127 .. 127, one s for a row of
// activations (token) or a column of a weight (channel).  Then
//     sum_k a(m, k) w(k, n) = sa(m) sw(n) sum_k qa(m, k) qw(k, n),
// and the sum of products is a whole number below 2^31, exact in int32 up to
// k = 131056 (16 * 8191; |qa qw| <= 2^14 where the caller's codes hold -128).
#pragma once

#include "fused_kernels.hpp"

namespace swq {

using namespace swk;

// The least maximum that a scale is made from: 127 / 2^-96 is finite, and rows
// below it are zeros next to any other's.
constexpr float TOP_MIN = 0x1p-96f;
constexpr unsigned BF16_INF = 0x7F80u;

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// the larger magnitude of both halves; infinities above all numbers, NaN above them
__device__ __forceinline__ unsigned max_abs2(unsigned m, unsigned w) {
    return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                  __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu)));
}
__device__ __forceinline__ unsigned max_abs16(unsigned m, u32x4 v) {
#pragma unroll
    for (int d = 0; d < 4; ++d) m = max_abs2(m, v[d]);
    return m;
}

// From the largest magnitude's bf16 bits: the scale, and what a value is
// multiplied by.  A row that holds an infinity or NaN has the scale NaN (and zeros
// for codes): its outputs are NaN, nobody else's.
struct Scale {
    float s, inv;
};
__device__ __forceinline__ Scale scale_of(unsigned top_bits) {
    if (top_bits >= BF16_INF) return Scale{__builtin_nanf(""), 0.0f};
    const float top = fmaxf(__builtin_bit_cast(float, top_bits << 16), TOP_MIN);
    return Scale{top / 127.0f, 127.0f / top};
}

// Two bf16 to codes in the low bytes of a and b.  The product is rounded before
// its nearest whole number is taken (the definition's two steps): no fma here.
__device__ __forceinline__ void code2(unsigned w, float inv, unsigned& a, unsigned& b) {
#pragma clang fp contract(off)
    const float x = __builtin_bit_cast(float, w << 16) * inv;
    const float y = __builtin_bit_cast(float, w & 0xFFFF0000u) * inv;
    a = __builtin_bit_cast(unsigned, x + ROUND_BITS);
    b = __builtin_bit_cast(unsigned, y + ROUND_BITS);
}
__device__ __forceinline__ u32x2 codes8(u32x4 v, Scale s) {
    unsigned b[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) code2(v[d], s.inv, b[2 * d], b[2 * d + 1]);
    u32x2 out{low_bytes(b[0], b[1], b[2], b[3]), low_bytes(b[4], b[5], b[6], b[7])};
    if (s.inv == 0.0f) out = u32x2{0u, 0u};   // infinity or NaN times 0
    return out;
}

// ---------------------------------------------------------------------------
// Rows: A [M,K] bf16 to codes Q [M,K] and scales [M].  T threads hold a row in
// registers (C chunks of 8 each), so it is read once: 3 bytes an element of HBM
// traffic is what bounds it, and for a few rows the latency of one load, one
// reduction and one store.
// ---------------------------------------------------------------------------
template <int T, int C>
__global__ __launch_bounds__(T < 256 ? 256 : T) void quantize_rows_kernel(const uint16_t* __restrict__ A,
                                                                          uint8_t* __restrict__ Q,
                                                                          float* __restrict__ scales, int M, int K) {
    constexpr int ROWS = T < 256 ? 256 / T : 1;   // rows of a workgroup
    const int t = threadIdx.x % T;
    const int m = blockIdx.x * ROWS + threadIdx.x / T;
    const int chunks = K / 8;
    const bool live = m < M;
    const uint16_t* a = A + (size_t)(live ? m : M - 1) * K;
    u32x4 v[C];
    unsigned top2 = 0u;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = c * T + t;
        v[c] = at < chunks ? ld16(a + (size_t)at * 8) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int c = 0; c < C; ++c) top2 = max_abs16(top2, v[c]);
    unsigned top = max(top2 & 0xFFFFu, top2 >> 16);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = max(top, (unsigned)__shfl_xor((int)top, o));
    if constexpr (T > 64) {
        __shared__ unsigned tops[T / 64];
        if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < T / 64; ++w) top = max(top, tops[w]);
    }
    if (!live) return;
    const Scale s = scale_of(top);
    if (t == 0) scales[m] = s.s;
    uint8_t* q = Q + (size_t)m * K;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = c * T + t;
        if (at < chunks) *reinterpret_cast<u32x2*>(q + (size_t)at * 8) = codes8(v[c], s);
    }
}

// ---------------------------------------------------------------------------
// Columns: W [K,N] bf16 to codes Q [K,N] and scales [N], once, when weights are
// loaded.  A workgroup has 64 columns (8 threads side by side, 32 rows apart) and
// goes over them twice, the second time mostly out of the caches.  Few columns are few
// workgroups, whose loads' latency then bounds it: 3584 x 18944 88 us (2.3 TB/s of 3
// bytes an element), 18944 x 3584, on 56 CUs, 206.
// ---------------------------------------------------------------------------
static __global__ __launch_bounds__(256) void quantize_columns_kernel(const uint16_t* __restrict__ W,
                                                                      uint8_t* __restrict__ Q,
                                                                      float* __restrict__ scales, int K, int N) {
    __shared__ u32x4 tops[32][8];
    const int g = threadIdx.x & 7, r = threadIdx.x >> 3;
    const int n = blockIdx.x * 64 + g * 8;
    const bool live = n < N;
    const uint16_t* w = W + (live ? n : 0);
    u32x4 top = {0u, 0u, 0u, 0u};
#pragma unroll 4
    for (int k = r; k < K; k += 32) {
        const u32x4 v = ld16(w + (size_t)k * N);
#pragma unroll
        for (int d = 0; d < 4; ++d) top[d] = max_abs2(top[d], v[d]);
    }
    tops[r][g] = top;
    __syncthreads();
    for (int i = 0; i < 32; ++i) {
        const u32x4 v = tops[i][g];
#pragma unroll
        for (int d = 0; d < 4; ++d) top[d] = max_abs2(top[d], v[d]);
    }
    if (!live) return;
    Scale s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = scale_of((top[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
    if (r == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) scales[n + e] = s[e].s;
    }
#pragma unroll 4
    for (int k = r; k < K; k += 32) {
        const u32x4 v = ld16(w + (size_t)k * N);
        unsigned b[8], skip;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e & 1) code2(v[e >> 1], s[e].inv, skip, b[e]);
            else code2(v[e >> 1], s[e].inv, b[e], skip);
            if (s[e].inv == 0.0f) b[e] = 0u;
        }
        *reinterpret_cast<u32x2*>(Q + (size_t)k * N + n) =
            u32x2{low_bytes(b[0], b[1], b[2], b[3]), low_bytes(b[4], b[5], b[6], b[7])};
    }
}

// ---------------------------------------------------------------------------
// Weight packs: the bf16 packs' layouts in bytes, 16 int8 for 8 bf16.  A 32 KiB
// block holds 256 packed rows (columns of the weight) and 128 k; a thread turns 16
// k of 4 columns (16 words of adjacent bytes) into four 16-byte pieces.  Bound by HBM:
// a pair of 3584 x 18944 64 us (4.3 TB/s read and written), one 33.
// SINGLE: one weight (W1), 256 columns a tile; else 128 of W1, then 128 of W2.
// ---------------------------------------------------------------------------
template <bool SINGLE>
__global__ __launch_bounds__(256) void pack_int8_kernel(const uint8_t* __restrict__ W1,
                                                        const uint8_t* __restrict__ W2, uint8_t* __restrict__ Wp,
                                                        int K, int N, int KB, long long units) {
    for (long long u = (long long)blockIdx.x * 256 + threadIdx.x; u < units; u += (long long)gridDim.x * 256) {
        const long long blk = u >> 9;
        const int quad = (int)(u & 63), kc = (int)(u >> 6) & 7;   // columns 4 quad, k from 16 kc
        const int kb = (int)(blk % KB), jt = (int)(blk / KB);
        const int row = 4 * quad;
        const bool up = !SINGLE && row >= PACK_BN;
        const int n = SINGLE ? jt * PACK_ROWS + row : jt * PACK_BN + (up ? row - PACK_BN : row);
        const int k0 = kb * 128 + kc * 16;
        const uint8_t* W = up ? W2 : W1;
        unsigned w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            w[i] = (n < N && k0 + i < K) ? *reinterpret_cast<const unsigned*>(W + (size_t)(k0 + i) * N + n) : 0u;
        uint8_t* out = Wp + blk * 32768;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            u32x4 p;
#pragma unroll
            for (int d = 0; d < 4; ++d)
                p[d] = low_bytes(w[4 * d] >> (8 * c), w[4 * d + 1] >> (8 * c), w[4 * d + 2] >> (8 * c),
                                 w[4 * d + 3] >> (8 * c));
            *reinterpret_cast<u32x4*>(out + 2 * packed_off(row + c, kc * 8)) = p;
        }
    }
}

}  // namespace swq
