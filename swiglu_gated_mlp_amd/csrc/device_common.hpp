// Device types and helpers that the library's kernels share: vector types, LDS
// tile addressing, direct global->LDS loads, the transposing LDS read, bf16
// conversion and the XCD-aware order of workgroups.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace swk {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int BK = 64;             // K depth of one LDS stage (one 128-byte row)

constexpr int NUM_XCD = 8;
constexpr float LOG2E = 1.4426950408889634f;

// ---------------------------------------------------------------------------
// LDS tiles, loads, conversions
// ---------------------------------------------------------------------------
// XOR swizzle of the 16-byte chunks of row r of a [rows][64] bf16 LDS tile
__device__ __forceinline__ int swz(int r) { return (r ^ (r >> 3)) & 7; }

// element offset of 16-byte chunk c (0..7) of row r in an LDS tile [rows][64]
__device__ __forceinline__ int lds_off(int r, int c) { return r * BK + ((c ^ swz(r)) << 3); }

__device__ __forceinline__ u32x4 ld16(const uint16_t* p) {
    return *reinterpret_cast<const u32x4*>(p);
}

// SiLU(g) = g * sigmoid(g) = g / (1 + 2^(-g log2 e)); v_exp_f32 and v_rcp_f32.
// g -> -inf: the exponential overflows to +inf, rcp gives 0, result -0.
// g >= 17: the exponential is below 2^-24, 1 + e rounds to 1, result g.
__device__ __forceinline__ float silu_f(float g) {
    const float e = __builtin_amdgcn_exp2f(-g * LOG2E);
    return g * __builtin_amdgcn_rcpf(1.0f + e);
}

__device__ __forceinline__ unsigned bf16_bits(float x) {
    __bf16 h = (__bf16)x;   // v_cvt_pk_bf16_f32: round to nearest even
    return (unsigned)__builtin_bit_cast(unsigned short, h);
}

// Two floats to two bf16 (round to nearest even) in one v_cvt_pk_bf16_f32;
// `lo` lands in the low half.
__device__ __forceinline__ unsigned pack2(float lo, float hi) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 h2 __attribute__((ext_vector_type(2)));
    const h2 h = __builtin_convertvector((f2){lo, hi}, h2);
    return __builtin_bit_cast(unsigned, h);
}

// Map the hardware workgroup id to a logical id such that XCD x (which gets
// ids x, x+8, x+16, ...) owns one contiguous range of logical ids.
__device__ __forceinline__ int xcd_remap(int bid, int total) {
    const int q = total / NUM_XCD, r = total % NUM_XCD;
    const int x = bid % NUM_XCD, j = bid / NUM_XCD;
    return x * q + (x < r ? x : r) + j;
}

typedef __attribute__((address_space(3))) void* lds_void_ptr;

__device__ __forceinline__ void dma16(const uint16_t* gsrc, uint16_t* lds_dst) {
    __builtin_amdgcn_global_load_lds(reinterpret_cast<const void*>(gsrc),
                                     (lds_void_ptr)(lds_dst), 16, 0, 0);
}

// Row-major weight stage in LDS: 64 K-rows of NB columns (N-contiguous); the
// 16-byte chunks of row k are XOR-swizzled by (k & 3) << 2, which keeps the
// transposing fragment reads below free of bank conflicts (each 16-lane group
// reads 4 consecutive rows x 32 bytes, two groups read 16 columns apart).
template <int NB>
__device__ __forceinline__ int rm_off(int k, int col) {
    return k * NB + ((((col >> 3) ^ ((k & 3) << 2))) << 3) + (col & 7);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_ptr;

// ds_read_b64_tr_b16: within each group of 16 lanes, lane i receives element
// (i & 3) of the 8-byte pieces addressed by lanes 4e + (i >> 2), e = 0..3.
__device__ __forceinline__ s16x4 ds_read_tr16(const uint16_t* lds) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4_ptr)((__attribute__((address_space(3))) uint16_t*)(lds)));
}

// s_waitcnt immediate: vector-memory count vm, LDS/scalar count lgkm (no
// export wait)
constexpr int waitcnt_imm(int vm, int lgkm) {
    return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | ((lgkm & 15) << 8);
}

}  // namespace swk
