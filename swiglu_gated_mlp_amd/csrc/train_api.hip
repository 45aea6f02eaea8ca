// Host side of the gated MLP's training entry points (swiglu_train_*,
// swiglu_mlp_train_backward; include/swiglu.h): argument checks, the choice of
// tiles and splits, and the launches.  Every check runs before the first HIP
// call.
#include "swiglu.h"

#include "host_common.hpp"
#include "train_kernels.hpp"

using namespace swh;

namespace {

// Within a tile an operand is addressed by 32-bit byte offsets from the tile's
// corner: up to 256 rows of 2 N elements, so widths stop at 2^20.
constexpr int64_t kMaxTrainDim = (int64_t)1 << 20;

swiglu_status check_train_shape(int64_t M, int64_t K, int64_t N) {
    const swiglu_status st = check_shape(M, K, N);
    if (st != SWIGLU_OK) return st;
    return (K > kMaxTrainDim || N > kMaxTrainDim) ? SWIGLU_ERR_UNSUPPORTED_SHAPE : SWIGLU_OK;
}

// A call's buffers: inputs may overlap each other, an output nothing.
struct Buffers {
    struct Item {
        const void* p;
        int64_t bytes;
        bool out;
    };
    Item item[16];
    int n = 0;
    void in(const void* p, int64_t elems) { item[n++] = Item{p, elems * 2, false}; }
    void out(const void* p, int64_t elems) { item[n++] = Item{p, elems * 2, true}; }
    swiglu_status check() const {
        for (int i = 0; i < n; ++i)
            if (!item[i].p) return SWIGLU_ERR_NULL_POINTER;
        for (int i = 0; i < n; ++i)
            if (!aligned16(item[i].p)) return SWIGLU_ERR_MISALIGNED;
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if ((item[i].out || item[j].out) &&
                    overlap(range_of(item[i].p, item[i].bytes), range_of(item[j].p, item[j].bytes)))
                    return SWIGLU_ERR_ALIASING;
        return SWIGLU_OK;
    }
};

// ---------------------------------------------------------------------------
// tiles and splits of one product
// ---------------------------------------------------------------------------
struct TilePlan {
    int bm, bn;            // tile (dual: bn / 2 columns of each half)
    int tiles_m, tiles_n;
    int splits, kb_per_split;
    int workers, full;     // 256 x 256 tiles: workgroups, and tiles computed whole
};

constexpr int64_t kPieceBytes = 256 * 256 * 4;   // the sums of a piece of a 256 x 256 tile

// rows x cols sums (dual: cols of each half) over kb blocks of 64.  small_ok:
// operand a is k-contiguous, so 64-row tiles exist.
TilePlan plan_tiles(int64_t rows, int64_t cols, bool dual, int64_t kb, bool small_ok, int cus) {
    if (cus <= 0) cus = 256;
    TilePlan t{};
    const int half = dual ? 2 : 1;
    const int64_t big = ceil_div(rows, 256) * ceil_div(cols, 256 / half);
    if (rows > 128 && big * kb >= 12 * cus) {
        t.bm = t.bn = 256;
        t.tiles_m = (int)ceil_div(rows, 256);
        t.tiles_n = (int)ceil_div(cols, 256 / half);
        t.splits = 1;
        t.kb_per_split = (int)kb;
        t.workers = cus;
        t.full = (int)(big / cus * cus);
        // a last round that is nearly full costs less than its pieces' sums
        if (10 * (big - t.full) >= 9 * cus) t.full = (int)big;
        return t;
    }
    t.bm = (rows <= 64 && small_ok) ? 64 : 128;
    t.bn = 128;
    t.tiles_m = (int)ceil_div(rows, t.bm);
    t.tiles_n = (int)ceil_div(cols, t.bn / half);
    const int64_t tiles = (int64_t)t.tiles_m * t.tiles_n;
    int64_t s = 1;
    if (2 * tiles < 3 * cus) s = std::min<int64_t>(ceil_div(3 * cus, 2 * tiles), kb / 8);
    s = std::max<int64_t>(s, 1);
    t.kb_per_split = (int)ceil_div(kb, s);
    t.splits = (int)ceil_div(kb, t.kb_per_split);
    return t;
}

int64_t part_bytes(const TilePlan& t, int64_t rows, int64_t cols, bool dual) {
    if (t.bm == 256) return t.full < t.tiles_m * t.tiles_n ? 2 * t.workers * kPieceBytes : 0;
    return t.splits > 1 ? (int64_t)t.splits * rows * cols * (dual ? 2 : 1) * 4 : 0;
}

int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

// The products of the training entry points, their sizes and tiles.
enum Product { P_FORWARD, P_DUAL_D, P_DA, P_DW, P_DY, P_DW3 };

struct ProductShape {
    int64_t rows, cols, kb;
    bool dual, small_ok;
};

ProductShape shape_of(Product p, int64_t M, int64_t K, int64_t N) {
    switch (p) {
        case P_DA: return {M, K, 2 * ceil_div(N, 64), false, true};
        case P_DW: return {K, 2 * N, ceil_div(M, 64), false, false};
        case P_DY: return {M, N, ceil_div(K, 64), false, true};
        case P_DW3: return {N, K, ceil_div(M, 64), false, false};
        default: return {M, N, ceil_div(K, 64), true, true};   // P_FORWARD, P_DUAL_D
    }
}

TilePlan plan_of(Product p, int64_t M, int64_t K, int64_t N, int cus) {
    const ProductShape s = shape_of(p, M, K, N);
    return plan_tiles(s.rows, s.cols, s.dual, s.kb, s.small_ok, cus);
}

int64_t product_part_bytes(Product p, int64_t M, int64_t K, int64_t N, int cus) {
    const ProductShape s = shape_of(p, M, K, N);
    return part_bytes(plan_of(p, M, K, N, cus), s.rows, s.cols, s.dual);
}

int64_t d_bytes(int64_t M, int64_t N) { return align256(M * 2 * N * 2); }

int64_t train_workspace(int64_t M, int64_t K, int64_t N, int cus) {
    int64_t part = 0;
    for (Product p : {P_FORWARD, P_DUAL_D, P_DA, P_DW, P_DY, P_DW3})
        part = std::max(part, product_part_bytes(p, M, K, N, cus));
    return d_bytes(M, N) + part;
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
template <int BM, int BN, int WM, int WN, int AOP, int BOP, bool DUAL, int EPI>
hipError_t launch_gemm_tile(const swt::GemmArgs& a, hipStream_t s) {
    const void* fn =
        a.kseg % 64 ? reinterpret_cast<const void*>(&swt::tile_gemm_kernel<BM, BN, WM, WN, AOP, BOP, DUAL, EPI, true>)
                    : reinterpret_cast<const void*>(&swt::tile_gemm_kernel<BM, BN, WM, WN, AOP, BOP, DUAL, EPI, false>);
    swt::GemmArgs args = a;
    void* kargs[] = {&args};
    const unsigned grid = (unsigned)((int64_t)a.tiles_m * a.tiles_n * a.splits);
    return hipLaunchKernel(fn, dim3(grid), dim3(64 * WM * WN), kargs, 0, s);
}

template <int AOP, int BOP, bool DUAL, int EPI>
hipError_t launch_wide(const swt::GemmArgs& a, int workers, hipStream_t s) {
    const void* fn = a.kseg % 64 ? reinterpret_cast<const void*>(&swt::wide_gemm_kernel<AOP, BOP, DUAL, EPI, true>)
                                 : reinterpret_cast<const void*>(&swt::wide_gemm_kernel<AOP, BOP, DUAL, EPI, false>);
    swt::GemmArgs args = a;
    const int rest = a.tiles_m * a.tiles_n - a.full;
    int whole = std::min(a.full, workers);
    void* kargs[] = {&args, &whole, &workers};
    hipError_t e = hipLaunchKernel(fn, dim3((unsigned)(whole + (rest ? workers : 0))), dim3(256), kargs, 0, s);
    if (e != hipSuccess || rest == 0) return e;
    void* rargs[] = {&args, &workers};
    return hipLaunchKernel(reinterpret_cast<const void*>(&swt::wide_reduce_kernel<DUAL, EPI>),
                           dim3((unsigned)(rest * (DUAL ? 8 : 16))), dim3(256), rargs, 0, s);
}

template <int AOP, int BOP, bool DUAL, int EPI>
hipError_t launch_product(swt::GemmArgs a, const TilePlan& t, hipStream_t s) {
    a.tiles_m = t.tiles_m;
    a.tiles_n = t.tiles_n;
    a.splits = t.splits;
    a.kb_per_split = t.kb_per_split;
    a.part_cols = a.cols * (DUAL ? 2 : 1);
    a.kb_seg = (int)ceil_div(a.kseg, 64);
    hipError_t e;
    a.full = t.full;
    if (t.bm == 256) return launch_wide<AOP, BOP, DUAL, EPI>(a, t.workers, s);
    if (t.bm == 128) e = launch_gemm_tile<128, 128, 2, 2, AOP, BOP, DUAL, EPI>(a, s);
    else if constexpr (AOP == swt::OP_KC) e = launch_gemm_tile<64, 128, 2, 2, AOP, BOP, DUAL, EPI>(a, s);
    else e = hipErrorInvalidValue;
    if (e != hipSuccess || t.splits == 1) return e;
    void* kargs[] = {&a};
    const int64_t groups = (int64_t)a.rows * (a.cols / 8);
    return hipLaunchKernel(reinterpret_cast<const void*>(&swt::tile_reduce_kernel<DUAL, EPI>),
                           dim3((unsigned)std::min<int64_t>(ceil_div(groups, 256), 8192)), dim3(256), kargs, 0, s);
}

struct Call {
    int64_t M, K, N;
    int cus;
    hipStream_t s;
    float* part;
};

// G, U (dual product) of A and the weights; EPI: EP_KEEP or EP_DUAL_D
swt::GemmArgs dual_args(const Call& c, const uint16_t* A, const uint16_t* W1, const uint16_t* W2) {
    swt::GemmArgs a{};
    a.A0 = A; a.lda = c.K;
    a.B0 = W1; a.B1 = W2; a.ldb = c.N;
    a.rows = (int)c.M; a.cols = (int)c.N;
    a.kseg = (int)c.K; a.segs = 1;
    a.part = c.part;
    return a;
}

// dA = dG W1^T + dU W2^T
hipError_t run_da(const Call& c, const uint16_t* D, const uint16_t* W1, const uint16_t* W2, uint16_t* dA) {
    swt::GemmArgs a{};
    a.A0 = D; a.A1 = D + c.N; a.lda = 2 * c.N;
    a.B0 = W1; a.B1 = W2; a.ldb = c.N;
    a.rows = (int)c.M; a.cols = (int)c.K;
    a.kseg = (int)c.N; a.segs = 2;
    a.part = c.part;
    a.C0 = dA; a.n0_cols = a.ldc = (int)c.K;
    return launch_product<swt::OP_KC, swt::OP_KC, false, swt::EP_STORE>(a, plan_of(P_DA, c.M, c.K, c.N, c.cus), c.s);
}

// X^T Z of two token-major matrices: dW1 | dW2 = A^T D, dW3 = Y^T dZ
hipError_t run_dw(const Call& c, Product p, const uint16_t* X, const uint16_t* Z, uint16_t* C0, uint16_t* C1) {
    const ProductShape sh = shape_of(p, c.M, c.K, c.N);
    swt::GemmArgs a{};
    a.A0 = X; a.lda = sh.rows;
    a.B0 = Z; a.ldb = sh.cols;
    a.rows = (int)sh.rows; a.cols = (int)sh.cols;
    a.kseg = (int)c.M; a.segs = 1;
    a.part = c.part;
    a.C0 = C0; a.C1 = C1;
    a.n0_cols = a.ldc = (int)(p == P_DW ? c.N : c.K);
    return launch_product<swt::OP_KS, swt::OP_KS, false, swt::EP_STORE>(a, plan_of(p, c.M, c.K, c.N, c.cus), c.s);
}

hipError_t run_zero(uint16_t* p, int64_t elems, hipStream_t s) {
    long long pieces = elems / 8;
    void* kargs[] = {&p, &pieces};
    return hipLaunchKernel(reinterpret_cast<const void*>(&swt::zero_kernel),
                           dim3((unsigned)std::min<int64_t>(ceil_div(pieces, 256), 8192)), dim3(256), kargs, 0, s);
}

hipError_t run_dgate(const Call& c, const uint16_t* dY, const uint16_t* G, const uint16_t* U, uint16_t* D) {
    long long groups = c.M * (c.N / 8);
    int N = (int)c.N;
    void* kargs[] = {(void*)&dY, (void*)&G, (void*)&U, (void*)&D, &N, &groups};
    return hipLaunchKernel(reinterpret_cast<const void*>(&swt::dgate_kernel),
                           dim3((unsigned)std::min<int64_t>(ceil_div(groups, 256), 16384)), dim3(256), kargs, 0, c.s);
}

// the weight gradients of an empty batch are zero
swiglu_status empty_batch(uint16_t* const* dW, const int64_t* elems, int n, hipStream_t s) {
    for (int i = 0; i < n; ++i) {
        if (!dW[i]) continue;
        if (!aligned16(dW[i])) return SWIGLU_ERR_MISALIGNED;
    }
    for (int i = 0; i < n; ++i) {
        if (!dW[i]) continue;
        const hipError_t e = run_zero(dW[i], elems[i], s);
        if (e != hipSuccess) return hip_fail(e);
    }
    return SWIGLU_OK;
}

}  // namespace

extern "C" {

size_t swiglu_train_workspace_bytes(int64_t M, int64_t K, int64_t N) {
    if (check_train_shape(M, K, N) != SWIGLU_OK || M == 0) return 0;
    return (size_t)train_workspace(M, K, N, cu_count_now());
}

size_t swiglu_train_forward_workspace_bytes(int64_t M, int64_t K, int64_t N) {
    if (check_train_shape(M, K, N) != SWIGLU_OK || M == 0) return 0;
    return (size_t)product_part_bytes(P_FORWARD, M, K, N, cu_count_now());
}

swiglu_status swiglu_train_forward(const swiglu_bf16* A, const swiglu_bf16* W1, const swiglu_bf16* W2, swiglu_bf16* Y,
                                   swiglu_bf16* G, swiglu_bf16* U, int64_t M, int64_t K, int64_t N, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    swiglu_status st = check_train_shape(M, K, N);
    if (st != SWIGLU_OK) return st;
    if (M == 0) return SWIGLU_OK;
    Buffers b;
    b.in(A, M * K); b.in(W1, K * N); b.in(W2, K * N);
    b.out(Y, M * N); b.out(G, M * N); b.out(U, M * N);
    if (workspace) b.out(workspace, (int64_t)(workspace_bytes / 2));
    if ((st = b.check()) != SWIGLU_OK) return st;
    const int cus = cu_count_now();
    if (!workspace) workspace_bytes = 0;
    if (workspace_bytes < (size_t)product_part_bytes(P_FORWARD, M, K, N, cus)) return SWIGLU_ERR_WORKSPACE;
    const Call c{M, K, N, cus, (hipStream_t)stream, (float*)workspace};
    swt::GemmArgs a = dual_args(c, A, W1, W2);
    a.C0 = Y; a.C1 = G; a.C2 = U;
    const hipError_t e = launch_product<swt::OP_KC, swt::OP_KS, true, swt::EP_KEEP>(a, plan_of(P_FORWARD, M, K, N, cus),
                                                                                   c.s);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

swiglu_status swiglu_train_backward(const swiglu_bf16* dY, const swiglu_bf16* A, const swiglu_bf16* W1,
                                    const swiglu_bf16* W2, const swiglu_bf16* G, const swiglu_bf16* U, swiglu_bf16* dA,
                                    swiglu_bf16* dW1, swiglu_bf16* dW2, int64_t M, int64_t K, int64_t N,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    swiglu_status st = check_train_shape(M, K, N);
    if (st != SWIGLU_OK) return st;
    if (!dW1 != !dW2) return SWIGLU_ERR_NULL_POINTER;   // both weight gradients, or none
    if (M == 0) {
        uint16_t* dW[2] = {dW1, dW2};
        const int64_t elems[2] = {K * N, K * N};
        if (dW1 && overlap(range_of(dW1, 2 * K * N), range_of(dW2, 2 * K * N))) return SWIGLU_ERR_ALIASING;
        return empty_batch(dW, elems, 2, (hipStream_t)stream);
    }
    if (!G != !U) return SWIGLU_ERR_NULL_POINTER;       // both kept, or both recomputed
    Buffers b;
    b.in(dY, M * N); b.in(A, M * K); b.in(W1, K * N); b.in(W2, K * N);
    if (G) { b.in(G, M * N); b.in(U, M * N); }
    if (dA) b.out(dA, M * K);
    if (dW1) { b.out(dW1, K * N); b.out(dW2, K * N); }
    if (workspace) b.out(workspace, (int64_t)(workspace_bytes / 2));
    if ((st = b.check()) != SWIGLU_OK) return st;
    const int cus = cu_count_now();
    if (!workspace || workspace_bytes < (size_t)train_workspace(M, K, N, cus)) return SWIGLU_ERR_WORKSPACE;
    uint16_t* const D = (uint16_t*)workspace;
    const Call c{M, K, N, cus, (hipStream_t)stream, (float*)((char*)workspace + d_bytes(M, N))};
    hipError_t e;
    if (G) {
        e = run_dgate(c, dY, G, U, D);
    } else {
        swt::GemmArgs a = dual_args(c, A, W1, W2);
        a.C0 = D; a.E0 = dY;
        e = launch_product<swt::OP_KC, swt::OP_KS, true, swt::EP_DUAL_D>(a, plan_of(P_DUAL_D, M, K, N, cus), c.s);
    }
    if (e == hipSuccess && dA) e = run_da(c, D, W1, W2, dA);
    if (e == hipSuccess && dW1) e = run_dw(c, P_DW, A, D, dW1, dW2);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

swiglu_status swiglu_mlp_train_backward(const swiglu_bf16* dZ, const swiglu_bf16* A, const swiglu_bf16* W1,
                                        const swiglu_bf16* W2, const swiglu_bf16* W3, const swiglu_bf16* G,
                                        const swiglu_bf16* U, const swiglu_bf16* Y, swiglu_bf16* dA, swiglu_bf16* dW1,
                                        swiglu_bf16* dW2, swiglu_bf16* dW3, int64_t M, int64_t K, int64_t N,
                                        void* workspace, size_t workspace_bytes, void* stream) {
    swiglu_status st = check_train_shape(M, K, N);
    if (st != SWIGLU_OK) return st;
    if (!dW1 != !dW2 || !dW1 != !dW3) return SWIGLU_ERR_NULL_POINTER;   // the three weight gradients, or none
    if (M == 0) {
        uint16_t* dW[3] = {dW1, dW2, dW3};
        const int64_t elems[3] = {K * N, K * N, K * N};
        for (int i = 0; dW1 && i < 3; ++i)
            for (int j = 0; j < i; ++j)
                if (overlap(range_of(dW[i], 2 * K * N), range_of(dW[j], 2 * K * N))) return SWIGLU_ERR_ALIASING;
        return empty_batch(dW, elems, 3, (hipStream_t)stream);
    }
    Buffers b;
    b.in(dZ, M * K); b.in(A, M * K); b.in(W1, K * N); b.in(W2, K * N); b.in(W3, K * N);
    b.in(G, M * N); b.in(U, M * N);
    if (dW1) b.in(Y, M * N);   // only dW3 needs Y
    if (dA) b.out(dA, M * K);
    if (dW1) { b.out(dW1, K * N); b.out(dW2, K * N); b.out(dW3, K * N); }
    if (workspace) b.out(workspace, (int64_t)(workspace_bytes / 2));
    if ((st = b.check()) != SWIGLU_OK) return st;
    const int cus = cu_count_now();
    if (!workspace || workspace_bytes < (size_t)train_workspace(M, K, N, cus)) return SWIGLU_ERR_WORKSPACE;
    uint16_t* const D = (uint16_t*)workspace;
    const Call c{M, K, N, cus, (hipStream_t)stream, (float*)((char*)workspace + d_bytes(M, N))};
    swt::GemmArgs a{};
    a.A0 = dZ; a.lda = K;
    a.B0 = W3; a.ldb = K;
    a.rows = (int)M; a.cols = (int)N;
    a.kseg = (int)K; a.segs = 1;
    a.part = c.part;
    a.C0 = D; a.E0 = G; a.E1 = U;
    hipError_t e = launch_product<swt::OP_KC, swt::OP_KC, false, swt::EP_DY_D>(a, plan_of(P_DY, M, K, N, cus), c.s);
    if (e == hipSuccess && dA) e = run_da(c, D, W1, W2, dA);
    if (e == hipSuccess && dW1) e = run_dw(c, P_DW, A, D, dW1, dW2);
    if (e == hipSuccess && dW3) e = run_dw(c, P_DW3, Y, dZ, dW3, dW3);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

}  // extern "C"
