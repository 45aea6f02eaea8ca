// Host side of the products' schedules, shared by the library's translation
// units: the choice of tiles, splits and kernels for a shape (plans), and the
// launches of the packed products' kernels.
#pragma once

#include "swiglu.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fused_kernels.hpp"
#include "host_common.hpp"
#include "lora_stream.hpp"

namespace swl {

using namespace swh;

// The streaming kernel keeps each activation address as a 32-bit byte offset
// from the stage base (row * K * bytes).  Calls whose activation slice would
// reach 2 GiB are split into row chunks of at most this many rows (a multiple
// of 256), each with A and Y advanced to its first row.
inline int64_t stream_rows_limit(int64_t K, int elem_bytes) {
    const int64_t rows = (((int64_t)1 << 31) / (K * elem_bytes)) / 256 * 256;
    return rows >= 256 ? rows : 256;
}

// Equal chunks (multiples of 256 rows) of at most `limit` rows covering M.
inline int64_t balanced_chunk(int64_t M, int64_t limit) {
    const int64_t n = (M + limit - 1) / limit;
    const int64_t per = (M + n - 1) / n;
    return std::min(limit, (per + 255) / 256 * 256);
}

inline int64_t packed_elems(int64_t K, int64_t N) {
    return ceil_div(N, swk::PACK_BN) * ceil_div(K, swk::PACK_BK) * swk::PACK_ROWS * swk::PACK_BK;
}

// Single-weight pack of W [K,N] for the plain GEMM: 256 columns per packed
// tile (the dual kernels' Gate and Up halves), so ceil(N/256) tiles whose
// 128-column "output" width n_tiled the dual schedules are planned on.
inline int64_t gemm_packed_elems(int64_t K, int64_t N) {
    return ceil_div(N, swk::PACK_ROWS) * ceil_div(K, swk::PACK_BK) * swk::PACK_ROWS * swk::PACK_BK;
}
inline int64_t gemm_tiled_cols(int64_t N) { return ceil_div(N, swk::PACK_ROWS) * swk::PACK_BN; }

// ---------------------------------------------------------------------------
// kernel configurations
// ---------------------------------------------------------------------------
// Output tile for a token count and schedule.  M <= 64 (forced data-parallel
// or split-K; AUTO uses the decode kernel there): 32/64-row register-path
// tiles.  Split-K above that: 128 x 64 tiles (two workgroups fit a CU, and a
// narrow tile gives more tiles to split).  Data-parallel: 128 x 128 up to
// 2048 tokens, then 256 x 128 (each wave 128 rows x 64 columns of Gate and Up).
struct TileCfg {
    int BM, BN;
};

// Split-K keeps small row tiles for small M; the data-parallel schedule is
// the streaming kernel at every M (one row of 128-row tiles for M <= 128, on
// the panel schedule when its column tiles leave CUs idle).
// Data-parallel tiles: 256 x 128 (persistent, with the 128-row tail of the
// mixed launch) above 512 rows, and from 385 rows when the last row tile is
// at least three quarters full and the 256-row grid fills the CUs; else
// 128 x 128 (measured against 128-row tiles everywhere up to 2048 rows:
// 7B width M=512 152 -> 141 us, M=768 201 -> 178 us, M=2048 479 -> 422 us,
// 72B width M=1024 865 -> 751 us; 0.5B width M=1024 29.4 -> 25.0 us).
inline TileCfg packed_tile_for(int64_t M, int variant, int64_t N, int cus) {
    if (variant == SWIGLU_VARIANT_SPLIT_K) {
        if (M <= 32) return {32, 128};
        if (M <= 64) return {64, 128};
        return {128, 128};
    }
    if (M <= 512) {
        if (M > 384 && (M % 256 == 0 || M % 256 >= 192) && ceil_div(M, 256) * ceil_div(N, 128) >= cus)
            return {256, 128};
        return {128, 128};
    }
    return {256, 128};
}

// workgroups per CU the split count aims for
constexpr int kSplitWavesPerCu = 2;

// Split-K above this many output tiles is pointless (the tiles alone fill
// the device many times over).
constexpr int kMaxSplitTiles = 16384;

struct Plan {
    TileCfg t;
    int tiles_m, tiles_n, tiles;
    int tail_ntiles;   // data-parallel 256-row tiles: last column tiles run as 128x128 tiles
    int panels;        // data-parallel, one 128-row tile: 32-column panels spread over the CUs
    int splits, kb_per_split, KB;
    int variant;   // resolved: DATA_PARALLEL, SPLIT_K or DECODE
    int decode_mt; // DECODE: 16-token tiles per workgroup
    int cus;       // compute units the plan was made for
};

constexpr int kDecodeMaxM = 64;
inline bool variant_known(int v) { return v >= SWIGLU_VARIANT_AUTO && v <= SWIGLU_VARIANT_SEQUENTIAL; }

// Wave quantisation of the 256 x 128 schedule: when the last round of
// tiles would leave most CUs idle, the column tiles that make up that round
// run afterwards as 128 x 128 tiles (twice as many, half the work each).
inline int tail_tiles(int tiles_m, int tiles_n, int cus) {
    const int tiles = tiles_m * tiles_n;
    const int rem = tiles > cus ? tiles % cus : 0;
    if (rem == 0 || rem * 10 > cus * 6) return 0;
    const int nt = (int)ceil_div(rem, tiles_m);
    return nt < tiles_n ? nt : 0;
}

inline Plan make_plan(int64_t M, int64_t K, int64_t N, int variant, int cus) {
    Plan p{};
    if (cus <= 0) cus = 256;
    p.cus = cus;
    p.KB = (int)ceil_div(K, swk::BK);
    int v = variant;
    int auto_split_cap = 0;   // AUTO's split-K: most splits worth their partial-sum traffic
    if (v == SWIGLU_VARIANT_AUTO) {
        // Decode up to 32 rows; from 33 to 64 rows only while the weight
        // panels cannot fill the CUs (a small product, where the decode
        // kernel's single pass wins), otherwise the panel schedule streams
        // the weights faster (measured: 7B M=64 57 us against 76 us).
        const int64_t panels = 4 * ceil_div(N, swk::PACK_BN);
        if (M <= 32 || (M <= kDecodeMaxM && panels < cus)) {
            v = SWIGLU_VARIANT_DECODE;
        } else if (M <= kDecodeMaxM) {
            v = SWIGLU_VARIANT_DATA_PARALLEL;
        } else {
            // Split-K writes and re-reads S fp32 partial sums of Gate and Up,
            // 16*S*M*N bytes against the 4*K*N bytes of weights: worth it only
            // while the data-parallel tiles leave most CUs idle, and with at
            // most K / (16 M) splits (extra traffic <= a quarter of the
            // weights).  A data-parallel grid that fills half the CUs streams
            // the weights faster than split-K does.
            const TileCfg dp = packed_tile_for(M, SWIGLU_VARIANT_DATA_PARALLEL, N, cus);
            const int64_t dp_tiles = ceil_div(M, dp.BM) * ceil_div(N, dp.BN);
            auto_split_cap = (int)std::min<int64_t>(K / (16 * M), 1 << 20);
            v = (2 * dp_tiles >= cus || p.KB < 4 || auto_split_cap < 2) ? SWIGLU_VARIANT_DATA_PARALLEL
                                                                         : SWIGLU_VARIANT_SPLIT_K;
        }
    }
    p.variant = v;
    p.decode_mt = M <= 16 ? 1 : (M <= 32 ? 2 : 4);
    // the sequential order runs on the data-parallel tiles (no panel schedule)
    const bool dp_tiles = v == SWIGLU_VARIANT_DATA_PARALLEL || v == SWIGLU_VARIANT_SEQUENTIAL;
    p.t = packed_tile_for(M, dp_tiles ? SWIGLU_VARIANT_DATA_PARALLEL : v, N, cus);
    p.tiles_m = (int)ceil_div(M, p.t.BM);
    p.tiles_n = (int)ceil_div(N, p.t.BN);
    p.tiles = p.tiles_m * p.tiles_n;
    p.tail_ntiles = dp_tiles && p.t.BM == 256 ? tail_tiles(p.tiles_m, p.tiles_n, cus) : 0;
    // One row of 128-row tiles that leaves CUs idle: the 32-column weight
    // panels (four per tile) are spread evenly over the CUs instead, so every
    // CU streams weights.
    p.panels = 0;
    if (v == SWIGLU_VARIANT_DATA_PARALLEL && p.t.BM == 128 && p.tiles_m == 1 && p.tiles_n < cus)
        p.panels = 4 * p.tiles_n;
    if (v == SWIGLU_VARIANT_SPLIT_K && p.tiles <= kMaxSplitTiles) {
        // about kSplitWavesPerCu workgroups per CU, at least two K blocks per split
        int s = (int)ceil_div((int64_t)kSplitWavesPerCu * cus, p.tiles);
        if (auto_split_cap > 0) s = std::min(s, auto_split_cap);
        s = std::max(1, std::min(s, p.KB / 2 > 0 ? p.KB / 2 : 1));
        p.kb_per_split = (int)ceil_div(p.KB, s);
        p.splits = (int)ceil_div(p.KB, p.kb_per_split);
    } else {
        p.splits = 1;
        p.kb_per_split = p.KB;
    }
    return p;
}

// Split-K workspace: fp32 Gate and Up partial sums, [split][M][2N].
inline size_t split_workspace_bytes(const Plan& p, int64_t M, int64_t N) {
    if (p.variant != SWIGLU_VARIANT_SPLIT_K || p.splits <= 1) return 0;
    return (size_t)p.splits * (size_t)M * 2 * (size_t)N * sizeof(float);
}

// `total` work items (tiles, or tile x K split) on `grid` <= total workgroups;
// each workgroup takes items b, b + grid, ...
template <int BM, bool SPLIT, bool PANELS = false, bool IL = false, bool F8 = false, bool SEQ = false,
          bool GEMM = false, bool I8 = false>
hipError_t launch_stream(const swk::FusedArgs& a, int total, int grid, hipStream_t s,
                         const swk::LoraArgs* la = nullptr) {
    const bool ragged = (a.K % (F8 ? 128 : swk::BK)) != 0;
    if constexpr (!SPLIT && !IL && !F8 && !SEQ && !I8) {
        if (la) {
            // up to 256 rows (every panel schedule) the adapters' part is in memory
            const void* fn =
                ragged ? reinterpret_cast<const void*>(&swk::stream_lora_kernel<BM, true, PANELS, GEMM, PANELS ? 2 : 1>)
                       : reinterpret_cast<const void*>(&swk::stream_lora_kernel<BM, false, PANELS, GEMM, PANELS ? 2 : 1>);
            if constexpr (BM == 128 && !PANELS) {
                if (la->delta)
                    fn = ragged ? reinterpret_cast<const void*>(&swk::stream_lora_kernel<128, true, false, GEMM, 2>)
                                : reinterpret_cast<const void*>(&swk::stream_lora_kernel<128, false, false, GEMM, 2>);
            }
            swk::FusedArgs args = a;
            swk::LoraArgs lora = *la;
            void* kargs[] = {&args, &lora, &total};
            return hipLaunchKernel(fn, dim3(grid), dim3(256), kargs, 0, s);
        }
    }
    const void* fn =
        ragged ? reinterpret_cast<const void*>(&swk::stream_prefill_kernel<BM, SPLIT, true, PANELS, IL, F8, SEQ, GEMM, I8>)
               : reinterpret_cast<const void*>(&swk::stream_prefill_kernel<BM, SPLIT, false, PANELS, IL, F8, SEQ, GEMM, I8>);
    swk::FusedArgs args = a;
    void* kargs[] = {&args, &total};
    return hipLaunchKernel(fn, dim3(grid), dim3(256), kargs, 0, s);
}

// The data-parallel streaming schedules (128- or 256-row tiles, the panel
// schedule, the mixed 256/128-row launch) on either weight layout; SEQ: the
// sequential Gate-then-Up order (per-tile layout, no panel schedule).
template <bool IL, bool F8 = false, bool SEQ = false, bool GEMM = false, bool I8 = false>
hipError_t launch_stream_dp(const swk::FusedArgs& a, const Plan& p, hipStream_t s,
                            const swk::LoraArgs* la = nullptr) {
    const int grid = p.tiles;
    if constexpr (!I8) if (p.t.BM == 128) {   // int8: 256-row tiles only
        if constexpr (SEQ) return launch_stream<128, false, false, false, false, true>(a, grid, grid, s);
        if constexpr (!GEMM && !IL) {
            // two rows of 128-row tiles that leave CUs idle on a wide product:
            // one row of 256-row tiles on the panel schedule instead, the
            // weights streamed once (7B width M=192 98.6 -> 84.2 us, 72B width
            // M=256 259 -> 226 us; FP8 72B width M=192 144 -> 127 us; the 0.5B
            // width's few short panels lose, 13.5 against 24 us, and keep the
            // 128-row tiles, as does the interleaved layout, 95 against 107 us
            // at the 7B width)
            if (p.tiles_m == 2 && a.M <= 256 && p.tiles_n < p.cus && 2 * p.tiles_n >= p.cus) {
                swk::FusedArgs pa = a;
                pa.tiles_m = 1;
                pa.panels = 4 * p.tiles_n;
                const int g = std::min(pa.panels, p.cus);
                return launch_stream<256, false, true, IL, F8, false, false>(pa, g, g, s, la);
            }
        }
        if (p.panels > 0) {
            // the single-weight GEMM's units are half-panels (one weight half
            // each), as long as no workgroup gets more than its 4 waves
            swk::FusedArgs pa = a;
            pa.panels = GEMM ? 2 * p.panels : p.panels;
            if (pa.panels <= 4 * p.cus) {
                const int g = std::min(pa.panels, p.cus);
                return launch_stream<128, false, true, IL, F8, false, GEMM>(pa, g, g, s, la);
            }
        }
        return launch_stream<128, false, false, IL, F8, false, GEMM>(a, grid, grid, s, la);
    }
    // one workgroup per CU works through the 256-row tiles
    if (p.tail_ntiles == 0)
        return launch_stream<256, false, false, IL, F8, SEQ, GEMM, I8>(a, grid, std::min(grid, p.cus), s, la);
    // one launch: the 256-row tiles of the first column tiles, then
    // the last tail_ntiles column tiles as 128-row tiles
    swk::FusedArgs big = a, tail = a;
    big.tiles_n = p.tiles_n - p.tail_ntiles;
    tail.tiles_m = (int)ceil_div(a.M, 128);
    tail.tiles_n = p.tail_ntiles;
    tail.n_tile0 = big.tiles_n;
    int n_big = big.tiles_m * big.tiles_n;
    int n_pers = std::min(n_big, p.cus);
    const int grid_all = n_pers + tail.tiles_m * tail.tiles_n;
    const bool ragged = (a.K % (F8 ? 128 : swk::BK)) != 0;
    if constexpr (!IL && !F8 && !SEQ && !I8) {
        if (la) {
            const void* lfn = ragged ? reinterpret_cast<const void*>(&swk::stream_lora_mixed_kernel<true, GEMM>)
                                     : reinterpret_cast<const void*>(&swk::stream_lora_mixed_kernel<false, GEMM>);
            swk::LoraArgs lora = *la;
            void* largs[] = {&big, &tail, &lora, &n_pers, &n_big};
            return hipLaunchKernel(lfn, dim3(grid_all), dim3(256), largs, 0, s);
        }
    }
    const void* fn = ragged
                         ? reinterpret_cast<const void*>(&swk::stream_prefill_mixed_kernel<true, IL, F8, SEQ, GEMM, I8>)
                         : reinterpret_cast<const void*>(&swk::stream_prefill_mixed_kernel<false, IL, F8, SEQ, GEMM, I8>);
    void* kargs[] = {&big, &tail, &n_pers, &n_big};
    return hipLaunchKernel(fn, dim3(grid_all), dim3(256), kargs, 0, s);
}

// The data-parallel streaming plan (any M).
inline Plan stream_dp_plan(int64_t M, int64_t K, int64_t N, int cus) {
    return make_plan(M, K, N, SWIGLU_VARIANT_DATA_PARALLEL, cus);
}

}  // namespace swl
