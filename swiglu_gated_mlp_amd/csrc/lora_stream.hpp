// The streaming kernels with low-rank adapters (the decode kernel takes LoraArgs
// itself; the adapter step is lora_device.hpp).
#pragma once

#include "fused_kernels.hpp"
#include "lora_device.hpp"

namespace swk {

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
