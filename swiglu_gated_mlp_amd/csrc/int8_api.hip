// Host side of the int8 products (swiglu_*_int8; include/swiglu.h): argument
// checks, plans and launches.  Every check runs before the first HIP call.
#include "swiglu.h"
#include "swiglu_probe.h"

#include "int8_kernels.hpp"
#include "int8_narrow.hpp"
#include "launch.hpp"

#include <cmath>

using namespace swh;
using namespace swl;

namespace {

// sums of 2^14 (the caller's codes may hold -128) stay below 2^31
constexpr int64_t kMaxK8 = 131056;

swiglu_status check_shape_int8(int64_t M, int64_t K, int64_t N) {
    const swiglu_status st = check_shape(M, K, N);
    if (st != SWIGLU_OK) return st;
    return (K % 16 != 0 || K > kMaxK8) ? SWIGLU_ERR_UNSUPPORTED_SHAPE : SWIGLU_OK;
}
// the block contracts over K and over N
swiglu_status check_mlp_int8(int64_t M, int64_t K, int64_t N) {
    const swiglu_status st = check_shape_int8(M, K, N);
    return st != SWIGLU_OK ? st : check_shape_int8(M, N, K);
}

// A call's buffers: matrices 16-byte aligned, fp32 vectors 4; inputs may overlap
// each other, an output nothing.
struct Buffers {
    struct Item {
        const void* p;
        int64_t bytes;
        bool out;
        uintptr_t align;
    };
    Item item[12];
    int n = 0;
    void in(const void* p, int64_t bytes, uintptr_t align = 16) { item[n++] = Item{p, bytes, false, align}; }
    void out(const void* p, int64_t bytes, uintptr_t align = 16) { item[n++] = Item{p, bytes, true, align}; }
    swiglu_status check() const {
        for (int i = 0; i < n; ++i)
            if (!item[i].p) return SWIGLU_ERR_NULL_POINTER;
        for (int i = 0; i < n; ++i)
            if ((uintptr_t)item[i].p % item[i].align != 0) return SWIGLU_ERR_MISALIGNED;
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if ((item[i].out || item[j].out) &&
                    overlap(range_of(item[i].p, item[i].bytes), range_of(item[j].p, item[j].bytes)))
                    return SWIGLU_ERR_ALIASING;
        return SWIGLU_OK;
    }
};

// The packs are those of bf16 weights of K / 2 rows, and so are the streaming plans.
int64_t packed_bytes_int8(int64_t K, int64_t N) { return 2 * packed_elems(K / 2, N); }
int64_t gemm_packed_bytes_int8(int64_t K, int64_t N) { return 2 * gemm_packed_elems(K / 2, N); }

// Products whose activations reach 2 GiB run as row chunks, data-parallel.
bool in_chunks(int64_t M, int64_t K) { return M > stream_rows_limit(K, 1); }

// ---------------------------------------------------------------------------
// Plans.  The weight-streaming decode kernel (up to 64 rows), the tiles and parts of
// narrow_kernel, or the streaming kernel of many rows, whichever an estimate says is
// fastest.
//   The estimates are microseconds of a launch on an idle device with the weights in
// HBM and the caches full of something else's outputs, and only their order matters.
// Their constants are this chip's (256 CUs), fitted over some 390 shapes with every tile
// and up to 12 parts.  On 160 other shapes, drawn at random (1 .. 4096 rows, K and N 128
// .. 29568), they are off by 13 % in the root mean square, those of few rows all alike,
// and the chosen plan takes 1.3 % longer than the fastest measured one on average (144
// shapes within 5 %, 18 % at worst).
// ---------------------------------------------------------------------------
struct Plan8 {
    enum How { DECODE, NARROW, STREAM } how;
    int cus;
    Plan stream;            // STREAM: 256-row tiles, or (panels > 0) one row of them on panels
    int tile;               // NARROW: index into kNarrow
    bool once;              // weights loaded non-temporally
    int units, tiles_m, groups, splits, kb_per_split;
    size_t part_bytes;
};

// Tiles: rows, waves and 32-row weight blocks a wave.  One block a wave leaves registers
// for two workgroups a CU (three of 64 rows), so that one's last stores overlap the
// next's products: 2048 rows, K=896 N=4864, fused <128,4,2> 29, <128,4,1> 25 us; two
// reuse the activations' fragments: 7B width, 256 rows, one weight 32 and 39 us.  Counts
// of waves that divide no power of two fill the CUs where the others leave a round
// nearly empty: 7B width, 128 rows, fused <128,4,2> 33, <128,6,1> 30, 64 rows <64,4,1>
// 30, <64,5,1> 25 us.  Leaving out one tile costs 0.5 (<64,5,1>) to 3 % on average.
// 32 rows: batches of up to 32, against the decode kernel (see decode_us), and small
// products of up to 256 (0.5B width, 64 rows, fused <64,3,1> 6.0 us, <32,3,1> 5.5).
struct NarrowTile {
    int bm, waves, wt;
    bool gemm;
    // microseconds outside the items, a stage (128 k) of an item and of each of its
    // blocks, and a block's sums when they are finished
    double once, stage, block, finish;
};
constexpr NarrowTile kNarrow[] = {
    {128, 4, 2, true, 5.9, 0.172, 0.043, 0.68},  {128, 4, 1, true, 7.5, 0.177, 0.046, 0.46},
    {128, 6, 1, false, 7.5, 0.177, 0.046, 0.46}, {64, 4, 1, true, 7.8, 0.138, 0.031, 0.30},
    {64, 3, 1, true, 7.8, 0.138, 0.031, 0.30},   {64, 5, 1, false, 7.8, 0.138, 0.031, 0.30},
    {32, 4, 1, true, 8.2, 0.091, 0.042, 0.07},   {32, 3, 1, true, 8.2, 0.091, 0.042, 0.07},
    {32, 5, 1, false, 8.2, 0.091, 0.042, 0.07}};

// A CU's stages, the weights from HBM and the matrix cores overlap in part.
double overlapped(double cu, double hbm, double mfma) { return std::sqrt(cu * cu + hbm * hbm + mfma * mfma); }

// work items on the CUs: in rounds, which run into each other from three on
double rounds_of(int64_t items, int cus) {
    return items > 3 * (int64_t)cus ? (double)items / cus + 0.3 : (double)ceil_div(items, cus);
}

double narrow_us(const Plan8& p, int64_t K, int64_t M) {
    const NarrowTile& t = kNarrow[p.tile];
    const int64_t items = (int64_t)p.tiles_m * p.groups * p.splits;
    const double rows = (double)p.groups * t.waves * t.wt * 32;   // packed
    // where CUs have several items, the SIMD with the most waves sets the pace
    const int64_t waves = items > 2 * (int64_t)p.cus ? ceil_div(t.waves, 4) * 4 : t.waves;
    const double blocks = (double)waves * t.wt;
    return t.once +
           overlapped(rounds_of(items, p.cus) * (p.kb_per_split * (t.stage + t.block * blocks) + t.finish * blocks),
                      (rows + M) * K / 6.7e6, 2.0 * p.tiles_m * t.bm * rows * K / 2.44e9) +
           (p.splits > 1 ? 2.6 + 0.13 * p.splits + p.part_bytes / 4.0e6 : 0.0);
}

double stream_us(const Plan& p, int64_t M, int64_t K) {
    const double rows = p.tiles_n * 256.0;
    // panels: four to a column tile, a wave each
    if (p.panels > 0)
        return 9.0 + overlapped(ceil_div(p.panels, p.cus) * (p.KB * 0.36 + 7.5), (rows + M) * K / 12.0e6, 0.0);
    const int rest = p.tiles % p.cus;
    const double rounds = p.tiles / p.cus + (rest == 0 ? 0.0 : p.tail_ntiles ? (double)rest / p.cus + 0.25 : 1.0);
    return 4.3 + overlapped(rounds * (p.KB * 0.93 + 12.7), (rows + M) * K / 6.0e6,
                            2.0 * p.tiles_m * 256 * rows * K / 3.3e9);
}

// The fused product on eight column groups a workgroup, one weight on two (see run_decode)
bool decode_wide(bool gemm, int64_t nt, int cus) {
    return gemm ? ceil_div(nt, 16) >= cus : 4 * ceil_div(nt, 128) >= 3 * (int64_t)cus;
}

// The decode kernel as run_decode launches it, up to 32 rows (one weight: 64).  Its workgroups read all
// activations, so that long contractions with few columns are narrow_kernel's, whose
// parts read theirs (one weight K=24352 N=848: 28 rows 24.7 and 13.0 us, 1 row 10.7 and
// 12.5), and those that fill a round and a little (K=16384 N=5120, 8 rows 21.8 and 18.7).
double decode_us(bool gemm, int64_t M, int64_t K, int64_t nt, int cus) {
    const int64_t KB = ceil_div(K, 128), groups = ceil_div(nt, 16);
    if (M > 32) return 7.8 + (0.115 + 0.0005 * M) * KB * ceil_div(2 * groups, cus);
    const bool wide = decode_wide(gemm, nt, cus);
    if (!gemm && wide) return 5.6 + 2.0 * nt * K / 6.85e6;
    const bool pairs = gemm && wide && M > 8 && M <= 16;   // two groups a workgroup
    // a workgroup's 128 k
    const double block = gemm ? (M <= 4 ? 0.038 : M <= 16 ? (0.042 + 0.0016 * M) * (pairs ? 1.7 : 1.0) : 0.093)
                              : (M <= 8 ? 0.086 : M <= 16 ? 0.098 : 0.142);
    return 7.9 + overlapped(block * KB * ceil_div(gemm && !pairs ? 2 * groups : groups, cus), 2.0 * nt * K / 8.0e6, 0.0);
}

// The streaming kernel at any M, without a workspace.
Plan8 stream_plan(bool gemm, int64_t M, int64_t K, int64_t N) {
    Plan8 p{};
    p.how = Plan8::STREAM;
    p.cus = cu_count_now();
    if (p.cus <= 0) p.cus = 256;
    Plan& s = p.stream;
    s.t = TileCfg{256, 128};
    s.cus = p.cus;
    s.KB = (int)ceil_div(K, 128);
    s.tiles_m = (int)ceil_div(M, 256);
    s.tiles_n = (int)ceil_div(gemm ? gemm_tiled_cols(N) : N, swk::PACK_BN);
    s.tiles = s.tiles_m * s.tiles_n;
    s.tail_ntiles = tail_tiles(s.tiles_m, s.tiles_n, p.cus);
    s.splits = 1;
    s.kb_per_split = s.KB;
    // one row of tiles that leaves CUs idle on a wide product: its panels over all CUs
    if (!gemm && s.tiles_m == 1 && s.tiles_n < p.cus && 2 * s.tiles_n >= p.cus) s.panels = 4 * s.tiles_n;
    return p;
}

Plan8 plan_int8(bool gemm, int64_t M, int64_t K, int64_t N) {
    Plan8 best = stream_plan(gemm, M, K, N);
    if (in_chunks(M, K)) return best;
    const int64_t KB = ceil_div(K, 128);
    double best_us = stream_us(best.stream, M, K);
    if (M <= (gemm ? 64 : 32)) {
        best.how = Plan8::DECODE;
        best_us = decode_us(gemm, M, K, gemm ? gemm_tiled_cols(N) : N, best.cus);
    }
    static const int kSplits[] = {1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 12, 16};
    for (const NarrowTile& t : kNarrow) {
        if ((gemm && !t.gemm) || (t.bm == 32 ? M > 256 : M <= 32)) continue;
        Plan8 p = best;
        p.how = Plan8::NARROW;
        p.tile = (int)(&t - kNarrow);
        // a wave's share of the columns (see Narrow)
        p.units = (int)(gemm && t.wt == 2 ? 4 * ceil_div(N, swk::PACK_ROWS) : ceil_div(N, gemm || t.wt == 2 ? 32 : 16));
        p.tiles_m = (int)ceil_div(M, t.bm);
        p.groups = (int)ceil_div(p.units, t.waves);
        // weights that fit the last-level cache beside others stay there; see Narrow::ONCE
        p.once = (int64_t)p.groups * t.waves * t.wt * 32 * KB * 128 > ((int64_t)32 << 20) &&
                 p.tiles_m <= (t.bm == 128 ? 4 : 2);
        for (int s : kSplits) {
            if (s > 1 && 3 * s > KB) break;
            p.kb_per_split = (int)ceil_div(KB, s);
            p.splits = (int)ceil_div(KB, p.kb_per_split);
            // a launch's threads are counted in 32 bits
            if ((int64_t)p.tiles_m * p.groups * p.splits * t.waves * 64 > INT32_MAX) break;
            p.part_bytes = p.splits > 1 ? (size_t)p.splits * p.groups * p.tiles_m * t.waves * t.wt * t.bm * 128
                                        : 0;
            const double us = narrow_us(p, K, M);
            if (us < best_us) {
                best_us = us;
                best = p;
            }
        }
    }
    return best;
}

// One product on the packed kernels; GEMM: N columns of one weight, else of a pair.
struct Product8 {
    const uint8_t* A;
    const float* sa;
    const uint8_t* W;
    const float *s1, *s2;
    uint16_t* Y;
    int64_t M, K, N;
    void* part;
};

template <int MT, int CG, int UNROLL, bool GEMM, bool HALF, bool LDSA, int WAVES>
hipError_t launch_decode8(const swk::DecodeArgs& a, int64_t n_tiled, hipStream_t s) {
    void (*fn)(swk::DecodeArgs) = &swk::decode_kernel<MT, CG, UNROLL, GEMM, HALF, LDSA, true, WAVES>;
    swk::DecodeArgs args = a;
    void* kargs[] = {&args};
    return hipLaunchKernel(reinterpret_cast<const void*>(fn),
                           dim3((unsigned)(ceil_div(n_tiled, 16 * CG) * (HALF ? 2 : 1))), dim3(64 * WAVES), kargs, 0, s);
}

// The decode kernel's configuration (MT 16-row tiles, CG groups of 16 columns a
// workgroup, UNROLL blocks in flight a wave, L: activations through LDS, waves), as
// measured (us, inputs rotated past the last-level cache).  Fused:
//   K=3584 N=18944  M=1 / 8: <1,1,8> 23.3 / 23.4, <1,8,2> 25.4, <1,2,4> 24.2
//                   M=16: <1,1,4,L,8 waves> 24.2, <1,1,8> 25.2, <1,1,8,L> 25.5
//                   M=32: <2,1,4,L> 27.4, <2,8,1> 28.1, <2,2,2> 28.5
//   K=8192 N=29568  M=1 / 16 / 32: <2,8,1> 71.8 / 71.3 / 72.4, <1,1,8> 83.0 / 83.5, <2,1,4,L> 88.3
//   K=896 N=4864    M=1 / 16 / 32: <1,1,8> 4.1 / 4.6, <1,1,4,L,8 waves> 4.4 (16), <2,1,4,L> 5.0 (32)
// wide groups where they still give most CUs a workgroup, else narrow ones, with
// activations through LDS from 9 rows on.  One weight, each half of a tile's columns a
// workgroup of its own (8 waves: the contraction is long, the columns few):
//   K=18944 N=3584  M=1: <1,1,4> 12.8, <1,1,4,L> 13.3, 4 waves <1,1,14> 13.7
//                   M=16: <1,1,4,L> 15.0, <1,1,4> 17.2, 4 waves <1,1,8,L> 15.9
//                   M=32: <2,1,2,L> 18.6, 4 waves <2,2,2> 29.4
//   K=29568 N=8192  M=1 / 16: <1,2,4> 38.4 / 40.3, <1,1,4> 37.3 / 49.2, <1,1,4,L> 38.7 / 42.9
//                   M=32: 4 waves <2,2,2> 49.0, <2,1,2,L> 55.2
//   K=4864 N=896    M=1 / 16 / 32: <1,1,4> 4.3, <1,1,4,L> 5.2 (16), <2,1,2,L> 6.5 (32)
// 33 to 64 rows of one weight, where narrow_kernel needs parts to fill the CUs:
//   K=4864 N=896    M=40 / 64: <4,1,1,L> 8.0 / 8.6, 4 waves 10.4 (narrow_kernel 8.8 / 9.0)
//   K=1024 N=3584   M=40 / 64: <4,1,1,L> 4.2 / 4.5 (narrow_kernel 5.2 / 5.2)
// (the fused product: K=896 N=4864 6.2 / 6.4, narrow_kernel 5.3 / 5.5)
template <bool GEMM>
hipError_t run_decode(const swk::DecodeArgs& d, int64_t nt, int cus, hipStream_t s) {
    const bool wide = decode_wide(GEMM, nt, cus);
    if constexpr (GEMM) {
        if (d.M > 32) return launch_decode8<4, 1, 1, true, true, true, 8>(d, nt, s);
        if (d.M > 16)
            return wide ? launch_decode8<2, 2, 2, true, true, false, 4>(d, nt, s)
                        : launch_decode8<2, 1, 2, true, true, true, 8>(d, nt, s);
        if (wide && d.M > 8) return launch_decode8<1, 2, 4, true, true, false, 8>(d, nt, s);
        return d.M > 4 ? launch_decode8<1, 1, 4, true, true, true, 8>(d, nt, s)
                       : launch_decode8<1, 1, 4, true, true, false, 8>(d, nt, s);
    } else {
        if (wide) return launch_decode8<2, 8, 1, false, false, false, 4>(d, nt, s);
        if (d.M <= 8) return launch_decode8<1, 1, 8, false, false, false, 4>(d, nt, s);
        return d.M <= 16 ? launch_decode8<1, 1, 4, false, false, true, 8>(d, nt, s)
                         : launch_decode8<2, 1, 4, false, false, true, 4>(d, nt, s);
    }
}

template <int BM, int WAVES, int WT, bool GEMM, bool ONCE>
hipError_t launch_narrow_as(const swq::NarrowArgs& a, hipStream_t s) {
    using P = swq::Narrow<BM, WAVES, WT, 4, GEMM, ONCE>;
    if (a.splits > 1 && !a.part) return hipErrorInvalidValue;
    swq::NarrowArgs args = a;
    void* kargs[] = {&args};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&swq::narrow_kernel<P>),
                                         dim3((unsigned)(a.tiles_m * a.groups * a.splits)), dim3(64 * WAVES), kargs, 0, s);
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t jobs = (int64_t)a.tiles_m * a.groups * WAVES * (GEMM ? WT : 1) * P::TM;
    using R = swq::Narrow<BM, WAVES, WT, 4, GEMM, false>;
    return hipLaunchKernel(reinterpret_cast<const void*>(&swq::narrow_reduce_kernel<R>),
                           dim3((unsigned)ceil_div(jobs, 4)), dim3(256), kargs, 0, s);
}

template <int BM, int WAVES, int WT, bool GEMM>
hipError_t launch_narrow(const swq::NarrowArgs& a, bool once, hipStream_t s) {
    return once ? launch_narrow_as<BM, WAVES, WT, GEMM, true>(a, s) : launch_narrow_as<BM, WAVES, WT, GEMM, false>(a, s);
}

template <bool GEMM>
hipError_t run_rows(const Product8& q, const Plan8& p, hipStream_t s) {
    if (p.how == Plan8::NARROW) {
        swq::NarrowArgs a{};
        a.A = q.A; a.W = q.W; a.Y = q.Y;
        a.sa = q.sa; a.s1 = q.s1; a.s2 = q.s2;
        a.part = reinterpret_cast<int*>(q.part);
        a.M = (int)q.M; a.K = (int)q.K; a.N = (int)q.N; a.KB = (int)ceil_div(q.K, 128);
        a.units = p.units; a.tiles_m = p.tiles_m; a.groups = p.groups;
        a.splits = p.splits; a.kb_per_split = p.kb_per_split;
        const NarrowTile& t = kNarrow[p.tile];
        if (t.bm == 128) {
            if (t.wt == 2) return launch_narrow<128, 4, 2, GEMM>(a, p.once, s);
            if (t.waves == 4) return launch_narrow<128, 4, 1, GEMM>(a, p.once, s);
            if constexpr (!GEMM) return launch_narrow<128, 6, 1, false>(a, p.once, s);
        } else if (t.bm == 32) {
            if (t.waves == 4) return launch_narrow<32, 4, 1, GEMM>(a, p.once, s);
            if (t.waves == 3) return launch_narrow<32, 3, 1, GEMM>(a, p.once, s);
            if constexpr (!GEMM) return launch_narrow<32, 5, 1, false>(a, p.once, s);
        } else {
            if (t.waves == 4) return launch_narrow<64, 4, 1, GEMM>(a, p.once, s);
            if (t.waves == 3) return launch_narrow<64, 3, 1, GEMM>(a, p.once, s);
            if constexpr (!GEMM) return launch_narrow<64, 5, 1, false>(a, p.once, s);
        }
        return hipErrorInvalidValue;
    }
    const uint16_t* A = reinterpret_cast<const uint16_t*>(q.A);
    const uint16_t* W = reinterpret_cast<const uint16_t*>(q.W);
    if (p.how == Plan8::DECODE) {
        swk::DecodeArgs d{};
        d.A = A; d.Wp = W; d.Y = q.Y;
        d.M = (int)q.M; d.K = (int)(q.K / 2); d.N = (int)q.N; d.KB = (int)ceil_div(q.K, 128);
        d.sa = q.sa; d.s1 = q.s1; d.s2 = q.s2;
        return run_decode<GEMM>(d, GEMM ? gemm_tiled_cols(q.N) : q.N, p.cus, s);
    }
    swk::FusedArgs a{};
    a.A = A; a.W1 = W; a.Y = q.Y;
    a.M = (int)q.M; a.K = (int)(q.K / 2); a.N = (int)q.N;
    a.tiles_m = p.stream.tiles_m; a.tiles_n = p.stream.tiles_n;
    a.splits = 1; a.kb_per_split = a.KB = p.stream.KB;
    a.sa = q.sa; a.s1 = q.s1; a.s2 = q.s2;
    if constexpr (!GEMM) {
        if (p.stream.panels > 0) {
            a.panels = p.stream.panels;
            const int g = std::min(a.panels, p.cus);
            return launch_stream<256, false, true, false, false, false, false, true>(a, g, g, s);
        }
    }
    return launch_stream_dp<false, false, false, GEMM, true>(a, p.stream, s);
}

template <bool GEMM>
hipError_t run_product(const Product8& q, const Plan8& p, hipStream_t s) {
    if (!in_chunks(q.M, q.K)) return run_rows<GEMM>(q, p, s);
    const int64_t rows = balanced_chunk(q.M, stream_rows_limit(q.K, 1));
    for (int64_t m0 = 0; m0 < q.M; m0 += rows) {
        Product8 c = q;
        c.M = std::min(rows, q.M - m0);
        c.A += m0 * q.K;
        c.sa += m0;
        c.Y += m0 * q.N;
        // not plan_int8: the call's workspace holds no sums of a chunk's parts
        const hipError_t e = run_rows<GEMM>(c, stream_plan(GEMM, c.M, q.K, q.N), s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int T, int C>
hipError_t launch_rows(const uint16_t* A, uint8_t* Q, float* scales, int64_t M, int64_t K, hipStream_t s) {
    constexpr int kRows = T < 256 ? 256 / T : 1;
    // a launch's threads are counted in 32 bits
    constexpr int64_t kMost = (int64_t)1 << 20;
    for (int64_t m0 = 0; m0 < M; m0 += kMost) {
        const uint16_t* a = A + m0 * K;
        uint8_t* q = Q + m0 * K;
        float* sc = scales + m0;
        int m = (int)std::min(kMost, M - m0), k = (int)K;
        void* args[] = {(void*)&a, (void*)&q, (void*)&sc, &m, &k};
        const hipError_t e =
            hipLaunchKernel(reinterpret_cast<const void*>(&swq::quantize_rows_kernel<T, C>),
                            dim3((unsigned)ceil_div(m, kRows)), dim3(T < 256 ? 256 : T), args, 0, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Threads for a row: a wave where a row is short, else so many that each loads a few pieces.
hipError_t run_quantize_rows(const uint16_t* A, uint8_t* Q, float* scales, int64_t M, int64_t K, hipStream_t s) {
    const int64_t chunks = K / 8;
    if (chunks <= 64 * 2) return launch_rows<64, 2>(A, Q, scales, M, K, s);
    if (chunks <= 256 * 2) return launch_rows<256, 2>(A, Q, scales, M, K, s);
    if (chunks <= 256 * 4) return launch_rows<256, 4>(A, Q, scales, M, K, s);
    if (chunks <= 1024 * 4) return launch_rows<1024, 4>(A, Q, scales, M, K, s);
    return launch_rows<1024, 16>(A, Q, scales, M, K, s);
}

int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

// The block's workspace: codes and scales of A, then of Y, then the splits' sums
// (of one product, then of the other).
struct MlpSpace {
    int64_t a8, sa, y8, sy, part, bytes;
};
MlpSpace mlp_space(int64_t M, int64_t K, int64_t N, const Plan8& up, const Plan8& down) {
    MlpSpace w{};
    w.sa = align256(M * K);
    w.y8 = w.sa + align256(4 * M);
    w.sy = w.y8 + align256(M * N);
    w.part = w.sy + align256(4 * M);
    w.bytes = w.part + (int64_t)std::max(up.part_bytes, down.part_bytes);
    return w;
}

template <bool SINGLE>
swiglu_status pack_impl_int8(const int8_t* W1, const int8_t* W2, int8_t* Wp, int64_t K, int64_t N, void* stream) {
    const swiglu_status st = check_shape_int8(0, K, N);
    if (st != SWIGLU_OK) return st;
    const int64_t bytes = SINGLE ? gemm_packed_bytes_int8(K, N) : packed_bytes_int8(K, N);
    Buffers b;
    b.in(W1, K * N); b.in(W2, K * N);
    b.out(Wp, bytes);
    const swiglu_status bad = b.check();
    if (bad != SWIGLU_OK) return bad;
    long long units = bytes / 64;
    int Ki = (int)K, Ni = (int)N, KB = (int)ceil_div(K, 128);
    void* args[] = {(void*)&W1, (void*)&W2, (void*)&Wp, &Ki, &Ni, &KB, &units};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&swq::pack_int8_kernel<SINGLE>),
                                         dim3((unsigned)std::min<int64_t>(ceil_div(units, 256), 1 << 20)), dim3(256),
                                         args, 0, (hipStream_t)stream);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

}  // namespace

extern "C" {

swiglu_status swiglu_quantize_rows_int8(const swiglu_bf16* A, int8_t* Q, float* scales, int64_t M, int64_t K,
                                        void* stream) {
    swiglu_status st = check_shape(M, K, 8);
    if (st != SWIGLU_OK) return st;
    if (K > kMaxK8) return SWIGLU_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return SWIGLU_OK;
    Buffers b;
    b.in(A, 2 * M * K);
    b.out(Q, M * K); b.out(scales, 4 * M, 4);
    if ((st = b.check()) != SWIGLU_OK) return st;
    const hipError_t e = run_quantize_rows(A, reinterpret_cast<uint8_t*>(Q), scales, M, K, (hipStream_t)stream);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

swiglu_status swiglu_quantize_columns_int8(const swiglu_bf16* W, int8_t* Q, float* scales, int64_t K, int64_t N,
                                           void* stream) {
    swiglu_status st = check_shape(0, K, N);
    if (st != SWIGLU_OK) return st;
    Buffers b;
    b.in(W, 2 * K * N);
    b.out(Q, K * N); b.out(scales, 4 * N, 4);
    if ((st = b.check()) != SWIGLU_OK) return st;
    int Ki = (int)K, Ni = (int)N;
    void* args[] = {(void*)&W, (void*)&Q, (void*)&scales, &Ki, &Ni};
    const hipError_t e =
        hipLaunchKernel(reinterpret_cast<const void*>(&swq::quantize_columns_kernel),
                        dim3((unsigned)ceil_div(N, 64)), dim3(256), args, 0, (hipStream_t)stream);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

size_t swiglu_packed_bytes_int8(int64_t K, int64_t N) {
    return check_shape_int8(0, K, N) == SWIGLU_OK ? (size_t)packed_bytes_int8(K, N) : 0;
}

size_t swiglu_gemm_packed_bytes_int8(int64_t K, int64_t N) {
    return check_shape_int8(0, K, N) == SWIGLU_OK ? (size_t)gemm_packed_bytes_int8(K, N) : 0;
}

swiglu_status swiglu_pack_weights_int8(const int8_t* W1, const int8_t* W2, int8_t* Wp, int64_t K, int64_t N,
                                       void* stream) {
    return pack_impl_int8<false>(W1, W2, Wp, K, N, stream);
}

swiglu_status swiglu_gemm_pack_weight_int8(const int8_t* W, int8_t* Wg, int64_t K, int64_t N, void* stream) {
    return pack_impl_int8<true>(W, W, Wg, K, N, stream);
}

size_t swiglu_workspace_bytes_int8(int64_t M, int64_t K, int64_t N) {
    if (check_shape_int8(M, K, N) != SWIGLU_OK || M == 0) return 0;
    return plan_int8(false, M, K, N).part_bytes;
}

size_t swiglu_gemm_workspace_bytes_int8(int64_t M, int64_t K, int64_t N) {
    if (check_shape_int8(M, K, N) != SWIGLU_OK || M == 0) return 0;
    return plan_int8(true, M, K, N).part_bytes;
}

size_t swiglu_mlp_workspace_bytes_int8(int64_t M, int64_t K, int64_t N) {
    if (check_mlp_int8(M, K, N) != SWIGLU_OK || M == 0) return 0;
    return (size_t)mlp_space(M, K, N, plan_int8(false, M, K, N), plan_int8(true, M, N, K)).bytes;
}

swiglu_status swiglu_fused_packed_int8(const int8_t* A, const float* sa, const int8_t* Wp, const float* s1,
                                       const float* s2, swiglu_bf16* Y, int64_t M, int64_t K, int64_t N,
                                       void* workspace, size_t workspace_bytes, void* stream) {
    swiglu_status st = check_shape_int8(M, K, N);
    if (st != SWIGLU_OK) return st;
    if (M == 0) return SWIGLU_OK;
    if (!workspace) workspace_bytes = 0;
    Buffers b;
    b.in(A, M * K); b.in(sa, 4 * M, 4); b.in(Wp, packed_bytes_int8(K, N)); b.in(s1, 4 * N, 4); b.in(s2, 4 * N, 4);
    b.out(Y, 2 * M * N);
    if (workspace) b.out(workspace, (int64_t)workspace_bytes);
    if ((st = b.check()) != SWIGLU_OK) return st;
    const Plan8 p = plan_int8(false, M, K, N);
    if (workspace_bytes < p.part_bytes) return SWIGLU_ERR_WORKSPACE;
    const Product8 q{(const uint8_t*)A, sa, (const uint8_t*)Wp, s1, s2, Y, M, K, N, workspace};
    const hipError_t e = run_product<false>(q, p, (hipStream_t)stream);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

swiglu_status swiglu_gemm_packed_int8(const int8_t* A, const float* sa, const int8_t* Wg, const float* sw,
                                      swiglu_bf16* C, int64_t M, int64_t K, int64_t N, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    swiglu_status st = check_shape_int8(M, K, N);
    if (st != SWIGLU_OK) return st;
    if (M == 0) return SWIGLU_OK;
    if (!workspace) workspace_bytes = 0;
    Buffers b;
    b.in(A, M * K); b.in(sa, 4 * M, 4); b.in(Wg, gemm_packed_bytes_int8(K, N)); b.in(sw, 4 * N, 4);
    b.out(C, 2 * M * N);
    if (workspace) b.out(workspace, (int64_t)workspace_bytes);
    if ((st = b.check()) != SWIGLU_OK) return st;
    const Plan8 p = plan_int8(true, M, K, N);
    if (workspace_bytes < p.part_bytes) return SWIGLU_ERR_WORKSPACE;
    const Product8 q{(const uint8_t*)A, sa, (const uint8_t*)Wg, sw, sw, C, M, K, N, workspace};
    const hipError_t e = run_product<true>(q, p, (hipStream_t)stream);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

swiglu_status swiglu_mlp_packed_int8(const swiglu_bf16* A, const int8_t* Wp, const float* s1, const float* s2,
                                     const int8_t* W3g, const float* s3, swiglu_bf16* Y, swiglu_bf16* Z, int64_t M,
                                     int64_t K, int64_t N, void* workspace, size_t workspace_bytes, void* stream) {
    swiglu_status st = check_mlp_int8(M, K, N);
    if (st != SWIGLU_OK) return st;
    if (M == 0) return SWIGLU_OK;
    if (!workspace) workspace_bytes = 0;
    Buffers b;
    b.in(A, 2 * M * K); b.in(Wp, packed_bytes_int8(K, N)); b.in(s1, 4 * N, 4); b.in(s2, 4 * N, 4);
    b.in(W3g, gemm_packed_bytes_int8(N, K)); b.in(s3, 4 * K, 4);
    b.out(Y, 2 * M * N); b.out(Z, 2 * M * K);
    if (workspace) b.out(workspace, (int64_t)workspace_bytes);
    if ((st = b.check()) != SWIGLU_OK) return st;
    const Plan8 up = plan_int8(false, M, K, N), down = plan_int8(true, M, N, K);
    const MlpSpace w = mlp_space(M, K, N, up, down);
    if (workspace_bytes < (size_t)w.bytes) return SWIGLU_ERR_WORKSPACE;
    char* const base = (char*)workspace;
    uint8_t* const a8 = (uint8_t*)base;
    uint8_t* const y8 = (uint8_t*)(base + w.y8);
    float* const sa = (float*)(base + w.sa);
    float* const sy = (float*)(base + w.sy);
    hipStream_t s = (hipStream_t)stream;
    hipError_t e = run_quantize_rows(A, a8, sa, M, K, s);
    if (e == hipSuccess)
        e = run_product<false>(Product8{a8, sa, (const uint8_t*)Wp, s1, s2, Y, M, K, N, base + w.part}, up, s);
    if (e == hipSuccess) e = run_quantize_rows(Y, y8, sy, M, N, s);
    if (e == hipSuccess)
        e = run_product<true>(Product8{y8, sy, (const uint8_t*)W3g, s3, s3, Z, M, N, K, base + w.part}, down, s);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

int swiglu_probe_int8_plan(int gemm, int64_t M, int64_t K, int64_t N, int32_t* plan) {
    if (check_shape_int8(M, K, N) != SWIGLU_OK || M == 0 || !plan) return 0;
    const Plan8 p = plan_int8(gemm != 0, M, K, N);
    const bool narrow = p.how == Plan8::NARROW;
    const int rows = p.how == Plan8::DECODE ? (M <= 16 ? 16 : M <= 32 ? 32 : 64) : narrow ? kNarrow[p.tile].bm : 256;
    const int cols = narrow ? 32 * kNarrow[p.tile].waves * kNarrow[p.tile].wt
                            : p.how == Plan8::STREAM && p.stream.panels > 0 ? 64 : 256;
    const int32_t v[5] = {p.how, rows, cols, narrow ? p.splits : 1, narrow && p.once};
    std::copy(v, v + 5, plan);
    return 1;
}

int swiglu_probe_int8_form(int gemm, int64_t M, int64_t K, int64_t N, int32_t* form) {
    if (check_shape_int8(M, K, N) != SWIGLU_OK || M == 0 || !form) return 0;
    const Plan8 p = in_chunks(M, K) ? stream_plan(gemm != 0, balanced_chunk(M, stream_rows_limit(K, 1)), K, N)
                                    : plan_int8(gemm != 0, M, K, N);
    const bool stream = p.how == Plan8::STREAM;
    const int panels = stream ? p.stream.panels : 0;
    const int32_t v[4] = {stream && panels == 0 ? p.stream.tail_ntiles : 0, panels,
                          p.how == Plan8::DECODE && decode_wide(gemm != 0, gemm ? gemm_tiled_cols(N) : N, p.cus),
                          K % 128 != 0};
    std::copy(v, v + 4, form);
    return 1;
}

}  // extern "C"
