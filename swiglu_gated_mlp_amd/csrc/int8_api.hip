// Host side of the int8 products (swiglu_*_int8; include/swiglu.h): argument
// checks, plans and launches.  Every check runs before the first HIP call.
#include "swiglu.h"

#include "int8_kernels.hpp"
#include "launch.hpp"

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

// The packs are those of bf16 weights of K / 2 rows, and so are the plans.
int64_t packed_bytes_int8(int64_t K, int64_t N) { return 2 * packed_elems(K / 2, N); }
int64_t gemm_packed_bytes_int8(int64_t K, int64_t N) { return 2 * gemm_packed_elems(K / 2, N); }

// Products whose activations reach 2 GiB run as row chunks, data-parallel.
bool in_chunks(int64_t M, int64_t K) { return M > stream_rows_limit(K, 1); }

Plan fused_plan_int8(int64_t M, int64_t K, int64_t N) {
    return make_plan(M, K / 2, N, in_chunks(M, K) ? SWIGLU_VARIANT_DATA_PARALLEL : SWIGLU_VARIANT_AUTO,
                     cu_count_now());
}
Plan gemm_plan_int8(int64_t M, int64_t K, int64_t N) {
    return in_chunks(M, K) ? make_plan(M, K / 2, gemm_tiled_cols(N), SWIGLU_VARIANT_DATA_PARALLEL, cu_count_now())
                           : gemm_plan(M, K / 2, N);
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

template <bool GEMM>
hipError_t run_rows(const Product8& q, const Plan& p, hipStream_t s) {
    const int64_t nt = GEMM ? gemm_tiled_cols(q.N) : q.N;
    if (p.variant == SWIGLU_VARIANT_DECODE) {
        swk::DecodeArgs d{};
        d.A = reinterpret_cast<const uint16_t*>(q.A);
        d.Wp = reinterpret_cast<const uint16_t*>(q.W);
        d.Y = q.Y;
        d.M = (int)q.M; d.K = (int)(q.K / 2); d.N = (int)q.N; d.KB = p.KB;
        d.sa = q.sa; d.s1 = q.s1; d.s2 = q.s2;
        if constexpr (GEMM) return launch_decode_gemm<true>(d, nt, p, s);
        else return launch_decode_cfg<true>(d, nt, p, s);
    }
    swk::FusedArgs a{};
    a.A = reinterpret_cast<const uint16_t*>(q.A);
    a.W1 = reinterpret_cast<const uint16_t*>(q.W);
    a.Y = q.Y;
    a.M = (int)q.M; a.K = (int)(q.K / 2); a.N = (int)q.N;
    a.tiles_m = p.tiles_m; a.tiles_n = p.tiles_n;
    a.splits = p.splits; a.kb_per_split = p.kb_per_split; a.KB = p.KB;
    a.sa = q.sa; a.s1 = q.s1; a.s2 = q.s2;
    if (p.splits <= 1) return launch_stream_dp<false, false, false, GEMM, true>(a, p, s);
    a.part = reinterpret_cast<float*>(q.part);
    const int grid = p.tiles * p.splits;
    const hipError_t e = launch_stream<128, true, false, false, false, false, GEMM, true>(a, grid, grid, s);
    if (e != hipSuccess) return e;
    const long long groups = (long long)q.M * (nt / 4);
    const int rgrid = (int)std::max<long long>(1, std::min<long long>(ceil_div(groups, 256), (long long)p.cus * 8));
    const int* part = reinterpret_cast<const int*>(q.part);
    int M = (int)q.M, N = (int)q.N, NT = (int)nt, S = p.splits;
    void* args[] = {(void*)&part, (void*)&q.Y, (void*)&q.sa, (void*)&q.s1, (void*)&q.s2, &M, &N, &NT, &S};
    return hipLaunchKernel(reinterpret_cast<const void*>(&swq::splitk_reduce_int8_kernel<GEMM>), dim3(rgrid),
                           dim3(256), args, 0, s);
}

template <bool GEMM>
hipError_t run_product(const Product8& q, const Plan& p, hipStream_t s) {
    if (!in_chunks(q.M, q.K)) return run_rows<GEMM>(q, p, s);
    const int64_t rows = balanced_chunk(q.M, stream_rows_limit(q.K, 1));
    const int64_t nt = GEMM ? gemm_tiled_cols(q.N) : q.N;
    for (int64_t m0 = 0; m0 < q.M; m0 += rows) {
        Product8 c = q;
        c.M = std::min(rows, q.M - m0);
        c.A += m0 * q.K;
        c.sa += m0;
        c.Y += m0 * q.N;
        const Plan cp = make_plan(c.M, q.K / 2, nt, SWIGLU_VARIANT_DATA_PARALLEL, p.cus);
        const hipError_t e = run_rows<GEMM>(c, cp, s);
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
MlpSpace mlp_space(int64_t M, int64_t K, int64_t N, const Plan& up, const Plan& down) {
    MlpSpace w{};
    w.sa = align256(M * K);
    w.y8 = w.sa + align256(4 * M);
    w.sy = w.y8 + align256(M * N);
    w.part = w.sy + align256(4 * M);
    w.bytes = w.part + (int64_t)std::max(split_workspace_bytes(up, M, N), gemm_split_bytes(down, M, K));
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
    return split_workspace_bytes(fused_plan_int8(M, K, N), M, N);
}

size_t swiglu_gemm_workspace_bytes_int8(int64_t M, int64_t K, int64_t N) {
    if (check_shape_int8(M, K, N) != SWIGLU_OK || M == 0) return 0;
    return gemm_split_bytes(gemm_plan_int8(M, K, N), M, N);
}

size_t swiglu_mlp_workspace_bytes_int8(int64_t M, int64_t K, int64_t N) {
    if (check_mlp_int8(M, K, N) != SWIGLU_OK || M == 0) return 0;
    return (size_t)mlp_space(M, K, N, fused_plan_int8(M, K, N), gemm_plan_int8(M, N, K)).bytes;
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
    const Plan p = fused_plan_int8(M, K, N);
    if (workspace_bytes < split_workspace_bytes(p, M, N)) return SWIGLU_ERR_WORKSPACE;
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
    const Plan p = gemm_plan_int8(M, K, N);
    if (workspace_bytes < gemm_split_bytes(p, M, N)) return SWIGLU_ERR_WORKSPACE;
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
    const Plan up = fused_plan_int8(M, K, N), down = gemm_plan_int8(M, N, K);
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

}  // extern "C"
