// Host side of the gated MLP's training entry points (swiglu_train_*,
// swiglu_mlp_train_backward; include/swiglu.h): argument checks, the choice of
// tiles and splits, and the launches.  Every check runs before the first HIP
// call.
#include "swiglu.h"
#include "swiglu_probe.h"

#include "host_common.hpp"
#include "train_kernels.hpp"

#include <algorithm>
#include <mutex>

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
    void kept(const void* codes, const void* scales, int64_t M, int64_t N, bool out) {
        const int64_t groups = ceil_div(N, swt::GROUP);
        item[n++] = Item{codes, M * groups * 2 * swt::GROUP, out};
        item[n++] = Item{scales, M * groups * 4, out};
    }
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
// Products, and their tiles and parts in a launch
// ---------------------------------------------------------------------------
// F_: the forward product; then the products of a backward pass in its two phases,
// D (recomputed, or from dZ; with dW3 beside it), then dA and dW1 | dW2.
// F_KEEP8, D_DY8: with Gate and Up kept as int8.
enum Kind { F_KEEP, D_DUAL, D_DY, G_DA, G_DW, G_DW3, F_KEEP8, D_DY8 };

struct Shape {
    int64_t rows, cols, kb;   // output (dual: columns of each half), contraction blocks
    bool dual, strided;       // strided: both operands k-strided (no 64-row tiles)
};

Shape shape_of(Kind p, int64_t M, int64_t K, int64_t N) {
    switch (p) {
        case G_DA: return {M, K, 2 * ceil_div(N, 64), false, false};
        case G_DW: return {K, 2 * N, ceil_div(M, 64), false, true};
        case D_DY: case D_DY8: return {M, N, ceil_div(K, 64), false, false};
        case G_DW3: return {N, K, ceil_div(M, 64), false, true};
        default: return {M, N, ceil_div(K, 64), true, false};   // F_KEEP, F_KEEP8, D_DUAL
    }
}

// One product's items: tiles of bm x bn, the first `whole` as they are, the rest
// in `splits` parts of kb_per_split blocks.
struct Tiles {
    int bm, bn;
    int tiles_m, tiles_n;
    int whole, rest, splits, kb_per_split;
    int items() const { return whole + rest * splits; }
    int64_t part_bytes() const { return (int64_t)rest * splits * bm * bn * 4; }
};

Tiles make_tiles(const Shape& s, int bm) {
    Tiles t{};
    t.bm = bm;
    t.bn = bm == 256 ? 256 : 128;
    t.tiles_m = (int)ceil_div(s.rows, t.bm);
    t.tiles_n = (int)ceil_div(s.cols, t.bn / (s.dual ? 2 : 1));
    t.whole = t.tiles_m * t.tiles_n;
    t.splits = 1;
    t.kb_per_split = (int)s.kb;
    return t;
}

// The same with the tiles past `whole` in about `splits` parts.
Tiles split_tiles(Tiles t, int64_t kb, int whole, int splits) {
    t.kb_per_split = (int)ceil_div(kb, splits);
    t.splits = (int)ceil_div(kb, t.kb_per_split);
    t.rest = t.splits > 1 ? t.tiles_m * t.tiles_n - whole : 0;
    t.whole = t.tiles_m * t.tiles_n - t.rest;
    if (t.rest == 0) {
        t.splits = 1;
        t.kb_per_split = (int)kb;
    }
    return t;
}

// Microseconds of an item of `kb` contraction blocks, to choose by: so many around the
// 64-deep stages (first loads, epilogue) and so many a stage.  Measured on this chip, a
// launch of 256 items of 1 / 3 / 8 / 16 / 32 / 76 stages (dA, even numbers alone: 2 / 8 /
// 16 / 32 / 76):
//   256 x 256  dW       15.8 / 18.7 / 26.0 / 38.9 / 64.0 / 133 us   dA  16.2 / 25.6 / 38.6 / 61.0 / 127
//              forward  20.2 / 26.3 / 34.9 / 41.2 / 71.6 / 137 (three outputs a tile)
//   128 x 128  dW        6.4 /  8.1 / 11.4 / 16.5 / 26.8 /  57      dA   7.7 / 11.7 / 16.0 / 25.8 /  52
//              forward   7.5 /  8.7 / 12.0 / 17.6 / 26.9 /  52
//    64 x 128  forward   5.8 /  6.7 /  9.9 / 16.2 / 26.2 /  67      dA   5.4 /  8.5 / 14.1 / 23.3 /  58
// The last of these tiles is up to a fifth slower than counted here at 16 and 32 stages, and
// a third to a half at 76, where 256 such items read 320 MB of weights (4.8 to 5.5 TB/s).
double item_us(int bm, int64_t kb) {
    return bm == 256 ? 10.0 + 1.55 * kb : (bm == 128 ? 7.0 + 0.6 * kb : 6.0 + 0.5 * kb);
}
// parts' sums: a launch, and 4 bytes a sum written and read at 5 TB/s.  Measured: 8 MB of
// parts 4.8 us; 67 MB 14.3 us and 3.6 us more in the items that write them, so that large
// parts cost about half of what is counted here.
constexpr double kReduceUs = 6.0, kPartUs = 2.0 / 5.0e6;

// When the last of a launch's items ends, each handed to the CU that falls free
// first: CUs are kept in groups that fall free at the same time.
struct Dispatch {
    double at[64];
    int cus[64];
    int n = 1;
    explicit Dispatch(int total) { at[0] = 0.0; cus[0] = total; }
    void run(int count, double us) {
        while (count > 0) {
            int g = 0;
            for (int i = 1; i < n; ++i)
                if (at[i] < at[g]) g = i;
            // whole rounds of a single group at once
            int m = std::min(count, cus[g]);
            const double end = at[g] + us * (n == 1 && count > cus[g] ? count / cus[g] : 1);
            if (n == 1 && count > cus[g]) {
                count -= count / cus[g] * cus[g];
                at[g] = end;
                continue;
            }
            count -= m;
            int h = 0;
            while (h < n && !(h != g && at[h] > end - 0.5 && at[h] < end + 0.5)) ++h;
            if (m == cus[g]) {
                at[g] = end;
            } else if (h < n || n == 64) {
                cus[h < n ? h : g] += h < n ? m : 0;
                cus[g] -= h < n ? m : 0;
            } else {
                at[n] = end;
                cus[n++] = m;
                cus[g] -= m;
            }
        }
    }
    double end() const { return *std::max_element(at, at + n); }
};

// A launch of one product, or of two at once.
struct Launch {
    int jobs;
    Kind kind[2];
    Tiles t[2];
    bool second_first;   // the second product's items have the longer run
    int64_t part_bytes() const { return t[0].part_bytes() + (jobs == 2 ? t[1].part_bytes() : 0); }
};

// A product's tiles with what they cost: the items' time in all and of the longest.
struct Candidate {
    Tiles t;
    double whole_us, part_us;   // of an item
    double total() const { return t.whole * whole_us + (double)t.rest * t.splits * part_us; }
    double longest() const { return std::max(t.whole ? whole_us : 0.0, t.rest ? part_us : 0.0); }
};

// The fastest of the candidate tiles and splits.
Launch search_launch(int jobs, const Kind* kind, int64_t M, int64_t K, int64_t N, int cus) {
    if (cus <= 0) cus = 256;
    static const int kSplits[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32};
    Candidate cand[2][40];
    int n[2] = {0, 0};
    for (int i = 0; i < jobs; ++i) {
        const Shape s = shape_of(kind[i], M, K, N);
        auto add = [&](const Tiles& t) {
            cand[i][n[i]++] = Candidate{t, item_us(t.bm, s.kb), item_us(t.bm, t.kb_per_split)};
        };
        const int sizes[2] = {256, s.rows <= 64 && !s.strided ? 64 : 128};
        for (int bm : sizes) {
            const Tiles t = make_tiles(s, bm);
            const int64_t all = (int64_t)t.tiles_m * t.tiles_n;
            for (int p : kSplits) {
                if (p > 1 && (p > s.kb / 3 || all * p > 4 * (int64_t)cus)) break;
                add(split_tiles(t, s.kb, 0, p));
            }
            // whole rounds, and the rest of the tiles split to fill one
            const int64_t rest = all % cus;
            if (bm == 256 && all > cus && rest > 0 && s.kb >= 6)
                add(split_tiles(t, s.kb, (int)(all - rest),
                                (int)std::max<int64_t>(2, std::min<int64_t>(cus / rest, s.kb / 3))));
        }
    }
    Launch best{};
    double best_us = 1e30;
    for (int i = 0; i < n[0]; ++i)
        for (int j = 0; j < (jobs == 2 ? n[1] : 1); ++j) {
            const Candidate* c[2] = {&cand[0][i], jobs == 2 ? &cand[1][j] : nullptr};
            if (c[1] && c[0]->t.bm == 256 && c[1]->t.bm != 256) continue;   // no kernel for it
            Launch l{};
            l.jobs = jobs;
            for (int q = 0; q < jobs; ++q) {
                l.kind[q] = kind[q];
                l.t[q] = c[q]->t;
            }
            const double reduce_us = l.part_bytes() ? kReduceUs + l.part_bytes() * kPartUs : 0.0;
            // no dispatch beats an even share of the work, or its longest item
            const double total = c[0]->total() + (c[1] ? c[1]->total() : 0.0);
            const double longest = std::max(c[0]->longest(), c[1] ? c[1]->longest() : 0.0);
            if (std::max(total / cus, longest) + reduce_us >= best_us) continue;
            l.second_first = c[1] && c[1]->longest() > c[0]->longest();
            Dispatch d(cus);
            for (int q = 0; q < jobs; ++q) {
                const Candidate& x = *c[l.second_first ? 1 - q : q];
                d.run(x.t.whole, x.whole_us);
                d.run(x.t.rest * x.t.splits, x.part_us);
            }
            const double us = d.end() + reduce_us;
            if (us < best_us) {
                best_us = us;
                best = l;
            }
        }
    return best;
}

// search_launch, remembered by shape (the choice depends on nothing else), in a table
// of fixed size: nothing is allocated, so nothing can throw across the C interface.  A
// shape has four places to lie in; with all of them taken the next one replaces one.
Launch plan_launch(int jobs, const Kind* kind, int64_t M, int64_t K, int64_t N, int cus) {
    struct Entry {
        int64_t key[5];
        Launch l;
    };
    constexpr int kEntries = 2048, kPlaces = 4;
    static Entry seen[kEntries];
    static std::mutex mu;
    // M > 0: an entry of zeros is a free one
    const int64_t key[5] = {jobs == 2 ? 16 * (kind[1] + 1) + kind[0] : kind[0], M, K, N, cus};
    uint64_t h = 0;
    for (const int64_t x : key) h = (h ^ (uint64_t)x) * 0x9E3779B97F4A7C15u;   // 2^64 / golden ratio
    Entry* const at = seen + (h >> 32) % (kEntries / kPlaces) * kPlaces;
    {
        std::lock_guard<std::mutex> lock(mu);
        for (int i = 0; i < kPlaces; ++i)
            if (std::equal(key, key + 5, at[i].key)) return at[i].l;
    }
    const Launch l = search_launch(jobs, kind, M, K, N, cus);
    std::lock_guard<std::mutex> lock(mu);
    int to = (int)(h >> 62);   // two bits that the place in the table does not depend on
    for (int i = kPlaces - 1; i >= 0; --i)
        if (at[i].key[1] == 0) to = i;
    std::copy(key, key + 5, at[to].key);
    at[to].l = l;
    return l;
}

int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }
int64_t d_bytes(int64_t M, int64_t N) { return align256(M * 2 * N * 2); }
int64_t y_bytes(int64_t M, int64_t N) { return align256(M * N * 2); }

// The launches of a backward pass: D, then the gradients.
struct Passes {
    int n = 0;
    Launch l[3];
    int64_t part_bytes() const {
        int64_t b = 0;
        for (int i = 0; i < n; ++i) b = std::max(b, l[i].part_bytes());
        return b;
    }
};
// d: D_DUAL, D_DY, D_DY8, or -1 (kept Gate and Up: an element-wise kernel)
Passes plan_backward(int d, bool da, bool dw, int64_t M, int64_t K, int64_t N, int cus) {
    Passes p;
    if ((d == D_DY || d == D_DY8) && dw) {
        const Kind k[2] = {(Kind)d, G_DW3};
        p.l[p.n++] = plan_launch(2, k, M, K, N, cus);
    } else if (d >= 0) {
        const Kind k[1] = {(Kind)d};
        p.l[p.n++] = plan_launch(1, k, M, K, N, cus);
    }
    const Kind k[2] = {da ? G_DA : G_DW, G_DW};
    if (da || dw) p.l[p.n++] = plan_launch(da && dw ? 2 : 1, k, M, K, N, cus);
    return p;
}

int64_t train_workspace(int64_t M, int64_t K, int64_t N, int cus) {
    int64_t part = 0;
    for (int d : {(int)D_DUAL, (int)D_DY})
        for (int g = 1; g < 4; ++g) part = std::max(part, plan_backward(d, g & 1, g & 2, M, K, N, cus).part_bytes());
    const Kind f[1] = {F_KEEP};
    return d_bytes(M, N) + std::max(part, plan_launch(1, f, M, K, N, cus).part_bytes());
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
using swt::OP_KC;
using swt::OP_KS;
template <int BM, int EPI>
using PDual = swt::Product<BM, BM == 256 ? 256 : 128, OP_KC, OP_KS, true, EPI>;
template <int BM, int EPI>
using PRows = swt::Product<BM, BM == 256 ? 256 : 128, OP_KC, OP_KC, false, EPI>;    // dA, dY
template <int BM>
using PGrad = swt::Product<BM, BM == 256 ? 256 : 128, OP_KS, OP_KS, false, swt::EP_STORE>;   // weight gradients

template <class A, class B>
hipError_t launch_pair(const Launch& l, swt::GemmArgs a, swt::GemmArgs b, hipStream_t s) {
    int items[2] = {l.t[0].items(), l.jobs == 2 ? l.t[1].items() : 0};
    int b_first = l.second_first;
    void* kargs[] = {&a, &b, &items[0], &items[1], &b_first};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&swt::gemm_kernel<A, B>),
                                         dim3((unsigned)(items[0] + items[1])), dim3(256), kargs, 0, s);
    if (e != hipSuccess || l.part_bytes() == 0) return e;
    auto blocks = [](const Tiles& t, bool dual) {   // four waves a workgroup, one a block (pair)
        return t.rest * (t.bm / 32) * (t.bn / 32) / (dual ? 2 : 1) / 4;
    };
    int na = blocks(l.t[0], A::DUAL);
    const int nb = l.jobs == 2 ? blocks(l.t[1], false) : 0;
    void* rargs[] = {&a, &b, &na};
    return hipLaunchKernel(reinterpret_cast<const void*>(&swt::gemm_reduce_kernel<A, B>), dim3((unsigned)(na + nb)),
                           dim3(256), rargs, 0, s);
}

template <class A>
hipError_t launch_with(const Launch& l, const swt::GemmArgs& a, const swt::GemmArgs& b, hipStream_t s) {
    if (l.jobs == 1) return launch_pair<A, swt::NoProduct>(l, a, b, s);
    if constexpr (A::EPI == swt::EP_STORE || A::EPI == swt::EP_DY_D || A::EPI == swt::EP_DY_D8) {
        if constexpr (A::BM == 256) return launch_pair<A, PGrad<256>>(l, a, b, s);
        else return l.t[1].bm == 256 ? launch_pair<A, PGrad<256>>(l, a, b, s) : launch_pair<A, PGrad<128>>(l, a, b, s);
    }
    return hipErrorInvalidValue;
}

template <template <int, int> class P, int EPI>
hipError_t launch_rows(const Launch& l, const swt::GemmArgs& a, const swt::GemmArgs& b, hipStream_t s) {
    switch (l.t[0].bm) {
        case 256: return launch_with<P<256, EPI>>(l, a, b, s);
        case 128: return launch_with<P<128, EPI>>(l, a, b, s);
        default: return launch_with<P<64, EPI>>(l, a, b, s);
    }
}

hipError_t run_launch(const Launch& l, swt::GemmArgs a, swt::GemmArgs b, float* part, hipStream_t s) {
    swt::GemmArgs* args[2] = {&a, &b};
    for (int i = 0; i < l.jobs; ++i) {
        const Tiles& t = l.t[i];
        args[i]->tiles_m = t.tiles_m;
        args[i]->tiles_n = t.tiles_n;
        args[i]->whole = t.whole;
        args[i]->rest = t.rest;
        args[i]->splits = t.splits;
        args[i]->kb_per_split = t.kb_per_split;
        args[i]->kb_seg = (int)ceil_div(args[i]->kseg, 64);
        args[i]->part = part;
        part += t.part_bytes() / 4;
    }
    switch (l.kind[0]) {
        case F_KEEP: return launch_rows<PDual, swt::EP_KEEP>(l, a, b, s);
        case D_DUAL: return launch_rows<PDual, swt::EP_DUAL_D>(l, a, b, s);
        case D_DY: return launch_rows<PRows, swt::EP_DY_D>(l, a, b, s);
        case F_KEEP8: return launch_rows<PDual, swt::EP_KEEP8>(l, a, b, s);
        case D_DY8: return launch_rows<PRows, swt::EP_DY_D8>(l, a, b, s);
        case G_DA: return launch_rows<PRows, swt::EP_STORE>(l, a, b, s);
        default:
            return l.t[0].bm == 256 ? launch_pair<PGrad<256>, swt::NoProduct>(l, a, b, s)
                                    : launch_pair<PGrad<128>, swt::NoProduct>(l, a, b, s);
    }
}

struct Call {
    int64_t M, K, N;
    hipStream_t s;
    uint16_t* D;
    float* part;
};

// G, U (dual product) of A and the weights
swt::GemmArgs dual_args(const Call& c, const uint16_t* A, const uint16_t* W1, const uint16_t* W2) {
    swt::GemmArgs a{};
    a.A0 = A; a.lda = c.K;
    a.B0 = W1; a.B1 = W2; a.ldb = c.N;
    a.rows = (int)c.M; a.cols = (int)c.N;
    a.kseg = (int)c.K; a.segs = 1;
    return a;
}

// dA = dG W1^T + dU W2^T
swt::GemmArgs da_args(const Call& c, const uint16_t* W1, const uint16_t* W2, uint16_t* dA) {
    swt::GemmArgs a{};
    a.A0 = c.D; a.A1 = c.D + c.N; a.lda = 2 * c.N;
    a.B0 = W1; a.B1 = W2; a.ldb = c.N;
    a.rows = (int)c.M; a.cols = (int)c.K;
    a.kseg = (int)c.N; a.segs = 2;
    a.C0 = dA; a.n0_cols = a.ldc = (int)c.K;
    return a;
}

// X^T Z of two token-major matrices of `rows` and `cols` columns: dW1 | dW2 = A^T D
// (columns from n0_cols on to C1), dW3 = Y^T dZ
swt::GemmArgs dw_args(const Call& c, const uint16_t* X, int64_t rows, const uint16_t* Z, int64_t cols, int64_t n0_cols,
                      uint16_t* C0, uint16_t* C1) {
    swt::GemmArgs a{};
    a.A0 = X; a.lda = rows;
    a.B0 = Z; a.ldb = cols;
    a.rows = (int)rows; a.cols = (int)cols;
    a.kseg = (int)c.M; a.segs = 1;
    a.C0 = C0; a.C1 = C1;
    a.n0_cols = a.ldc = (int)n0_cols;
    return a;
}

// dA and dW1, dW2 from D (the last launch of a plan)
hipError_t run_gradients(const Call& c, const Launch& l, const uint16_t* A, const uint16_t* W1, const uint16_t* W2,
                         uint16_t* dA, uint16_t* dW1, uint16_t* dW2) {
    const swt::GemmArgs da = da_args(c, W1, W2, dA);
    const swt::GemmArgs dw = dw_args(c, A, c.K, c.D, 2 * c.N, c.N, dW1, dW2);
    return run_launch(l, dA ? da : dw, dw, c.part, c.s);
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

// Elements from Gate and Up kept as int8 (swt::KeptUse): four rows a thread once that
// leaves every CU its threads, one row before.
template <int USE, int ROWS>
hipError_t run_kept_rows(const int8_t* codes, const swiglu_bf16* scales, const uint16_t* dY, uint16_t* C0, uint16_t* C1,
                         int64_t M, int64_t N, hipStream_t s) {
    long long units = ceil_div(M, ROWS) * (N / 8);
    int Mi = (int)M, Ni = (int)N;
    void* kargs[] = {(void*)&codes, (void*)&scales, (void*)&dY, (void*)&C0, (void*)&C1, &Mi, &Ni, &units};
    return hipLaunchKernel(reinterpret_cast<const void*>(&swt::kept_kernel<USE, ROWS>),
                           dim3((unsigned)std::min<int64_t>(ceil_div(units, 256), 65536)), dim3(256), kargs, 0, s);
}
template <int USE>
hipError_t run_kept(const int8_t* codes, const swiglu_bf16* scales, const uint16_t* dY, uint16_t* C0, uint16_t* C1,
                    int64_t M, int64_t N, hipStream_t s) {
    return M * N >= (int64_t)1 << 24 ? run_kept_rows<USE, 4>(codes, scales, dY, C0, C1, M, N, s)
                                     : run_kept_rows<USE, 1>(codes, scales, dY, C0, C1, M, N, s);
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
    const Kind f[1] = {F_KEEP};
    return (size_t)plan_launch(1, f, M, K, N, cu_count_now()).part_bytes();
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
    const Kind f[1] = {F_KEEP};
    const Launch l = plan_launch(1, f, M, K, N, cu_count_now());
    if (!workspace) workspace_bytes = 0;
    if (workspace_bytes < (size_t)l.part_bytes()) return SWIGLU_ERR_WORKSPACE;
    const Call c{M, K, N, (hipStream_t)stream, nullptr, (float*)workspace};
    swt::GemmArgs a = dual_args(c, A, W1, W2);
    a.C0 = Y; a.C1 = G; a.C2 = U;
    const hipError_t e = run_launch(l, a, a, c.part, c.s);
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
    const Passes p = plan_backward(G ? -1 : (int)D_DUAL, dA, dW1, M, K, N, cu_count_now());
    if (!workspace || workspace_bytes < (size_t)(d_bytes(M, N) + p.part_bytes())) return SWIGLU_ERR_WORKSPACE;
    const Call c{M, K, N, (hipStream_t)stream, (uint16_t*)workspace, (float*)((char*)workspace + d_bytes(M, N))};
    hipError_t e;
    if (G) {
        e = run_dgate(c, dY, G, U, c.D);
    } else {
        swt::GemmArgs a = dual_args(c, A, W1, W2);
        a.C0 = c.D; a.E0 = dY;
        e = run_launch(p.l[0], a, a, c.part, c.s);
    }
    if (e == hipSuccess && (dA || dW1)) e = run_gradients(c, p.l[p.n - 1], A, W1, W2, dA, dW1, dW2);
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
    const Passes p = plan_backward(D_DY, dA, dW1, M, K, N, cu_count_now());
    if (!workspace || workspace_bytes < (size_t)(d_bytes(M, N) + p.part_bytes())) return SWIGLU_ERR_WORKSPACE;
    const Call c{M, K, N, (hipStream_t)stream, (uint16_t*)workspace, (float*)((char*)workspace + d_bytes(M, N))};
    swt::GemmArgs a{};
    a.A0 = dZ; a.lda = K;
    a.B0 = W3; a.ldb = K;
    a.rows = (int)M; a.cols = (int)N;
    a.kseg = (int)K; a.segs = 1;
    a.C0 = c.D; a.E0 = G; a.E1 = U;
    const swt::GemmArgs dw3 = dw_args(c, Y, N, dZ, K, K, dW3, dW3);
    hipError_t e = run_launch(p.l[0], a, dw3, c.part, c.s);
    if (e == hipSuccess && (dA || dW1)) e = run_gradients(c, p.l[p.n - 1], A, W1, W2, dA, dW1, dW2);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

size_t swiglu_train_workspace_bytes_int8(int64_t M, int64_t K, int64_t N) {
    if (check_train_shape(M, K, N) != SWIGLU_OK || M == 0) return 0;
    return (size_t)(train_workspace(M, K, N, cu_count_now()) + y_bytes(M, N));
}

swiglu_status swiglu_train_forward_int8(const swiglu_bf16* A, const swiglu_bf16* W1, const swiglu_bf16* W2,
                                        swiglu_bf16* Y, int8_t* codes, swiglu_bf16* scales, int64_t M, int64_t K,
                                        int64_t N, void* workspace, size_t workspace_bytes, void* stream) {
    swiglu_status st = check_train_shape(M, K, N);
    if (st != SWIGLU_OK) return st;
    if (M == 0) return SWIGLU_OK;
    Buffers b;
    b.in(A, M * K); b.in(W1, K * N); b.in(W2, K * N);
    b.out(Y, M * N); b.kept(codes, scales, M, N, true);
    if (workspace) b.out(workspace, (int64_t)(workspace_bytes / 2));
    if ((st = b.check()) != SWIGLU_OK) return st;
    const Kind f[1] = {F_KEEP8};
    const Launch l = plan_launch(1, f, M, K, N, cu_count_now());
    if (!workspace) workspace_bytes = 0;
    if (workspace_bytes < (size_t)l.part_bytes()) return SWIGLU_ERR_WORKSPACE;
    const Call c{M, K, N, (hipStream_t)stream, nullptr, (float*)workspace};
    swt::GemmArgs a = dual_args(c, A, W1, W2);
    a.C0 = Y; a.C1 = (uint16_t*)codes; a.C2 = scales;
    const hipError_t e = run_launch(l, a, a, c.part, c.s);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

swiglu_status swiglu_dequantize_kept_int8(const int8_t* codes, const swiglu_bf16* scales, swiglu_bf16* G,
                                          swiglu_bf16* U, int64_t M, int64_t N, void* stream) {
    swiglu_status st = check_train_shape(M, 8, N);
    if (st != SWIGLU_OK) return st;
    if (M == 0) return SWIGLU_OK;
    Buffers b;
    b.kept(codes, scales, M, N, false);
    b.out(G, M * N); b.out(U, M * N);
    if ((st = b.check()) != SWIGLU_OK) return st;
    const hipError_t e = run_kept<swt::KEPT_GU>(codes, scales, nullptr, G, U, M, N, (hipStream_t)stream);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

swiglu_status swiglu_train_backward_int8(const swiglu_bf16* dY, const swiglu_bf16* A, const swiglu_bf16* W1,
                                         const swiglu_bf16* W2, const int8_t* codes, const swiglu_bf16* scales,
                                         swiglu_bf16* dA, swiglu_bf16* dW1, swiglu_bf16* dW2, int64_t M, int64_t K,
                                         int64_t N, void* workspace, size_t workspace_bytes, void* stream) {
    swiglu_status st = check_train_shape(M, K, N);
    if (st != SWIGLU_OK) return st;
    if (!dW1 != !dW2) return SWIGLU_ERR_NULL_POINTER;   // both weight gradients, or none
    if (M == 0) {
        uint16_t* dW[2] = {dW1, dW2};
        const int64_t elems[2] = {K * N, K * N};
        if (dW1 && overlap(range_of(dW1, 2 * K * N), range_of(dW2, 2 * K * N))) return SWIGLU_ERR_ALIASING;
        return empty_batch(dW, elems, 2, (hipStream_t)stream);
    }
    Buffers b;
    b.in(dY, M * N); b.in(A, M * K); b.in(W1, K * N); b.in(W2, K * N);
    b.kept(codes, scales, M, N, false);
    if (dA) b.out(dA, M * K);
    if (dW1) { b.out(dW1, K * N); b.out(dW2, K * N); }
    if (workspace) b.out(workspace, (int64_t)(workspace_bytes / 2));
    if ((st = b.check()) != SWIGLU_OK) return st;
    const Passes p = plan_backward(-1, dA, dW1, M, K, N, cu_count_now());
    if (!workspace || workspace_bytes < (size_t)(d_bytes(M, N) + p.part_bytes())) return SWIGLU_ERR_WORKSPACE;
    const Call c{M, K, N, (hipStream_t)stream, (uint16_t*)workspace, (float*)((char*)workspace + d_bytes(M, N))};
    hipError_t e = run_kept<swt::KEPT_D>(codes, scales, dY, c.D, nullptr, M, N, c.s);
    if (e == hipSuccess && (dA || dW1)) e = run_gradients(c, p.l[p.n - 1], A, W1, W2, dA, dW1, dW2);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

swiglu_status swiglu_mlp_train_backward_int8(const swiglu_bf16* dZ, const swiglu_bf16* A, const swiglu_bf16* W1,
                                             const swiglu_bf16* W2, const swiglu_bf16* W3, const int8_t* codes,
                                             const swiglu_bf16* scales, swiglu_bf16* dA, swiglu_bf16* dW1,
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
    b.kept(codes, scales, M, N, false);
    if (dA) b.out(dA, M * K);
    if (dW1) { b.out(dW1, K * N); b.out(dW2, K * N); b.out(dW3, K * N); }
    if (workspace) b.out(workspace, (int64_t)(workspace_bytes / 2));
    if ((st = b.check()) != SWIGLU_OK) return st;
    const Passes p = plan_backward(D_DY8, dA, dW1, M, K, N, cu_count_now());
    const int64_t before = d_bytes(M, N) + (dW1 ? y_bytes(M, N) : 0);
    if (!workspace || workspace_bytes < (size_t)(before + p.part_bytes())) return SWIGLU_ERR_WORKSPACE;
    const Call c{M, K, N, (hipStream_t)stream, (uint16_t*)workspace, (float*)((char*)workspace + before)};
    uint16_t* const Y = (uint16_t*)((char*)workspace + d_bytes(M, N));
    swt::GemmArgs a{};
    a.A0 = dZ; a.lda = K;
    a.B0 = W3; a.ldb = K;
    a.rows = (int)M; a.cols = (int)N;
    a.kseg = (int)K; a.segs = 1;
    a.C0 = c.D; a.E0 = (const uint16_t*)codes; a.E1 = scales;
    const swt::GemmArgs dw3 = dw_args(c, Y, N, dZ, K, K, dW3, dW3);
    // dW3's operand, before the launch that it shares with dY
    hipError_t e = dW1 ? run_kept<swt::KEPT_Y>(codes, scales, nullptr, Y, nullptr, M, N, c.s) : hipSuccess;
    if (e == hipSuccess) e = run_launch(p.l[0], a, dw3, c.part, c.s);
    if (e == hipSuccess && (dA || dW1)) e = run_gradients(c, p.l[p.n - 1], A, W1, W2, dA, dW1, dW2);
    return e == hipSuccess ? SWIGLU_OK : hip_fail(e);
}

int swiglu_probe_train_plan(int launch, int64_t M, int64_t K, int64_t N, int32_t* plan) {
    static const Kind kinds[SWIGLU_TRAIN_LAUNCHES][2] = {{F_KEEP}, {D_DUAL}, {D_DY},      {D_DY, G_DW3},
                                                         {G_DA},   {G_DW},   {G_DA, G_DW}};
    if (check_train_shape(M, K, N) != SWIGLU_OK || M == 0 || launch < 0 || launch >= SWIGLU_TRAIN_LAUNCHES || !plan)
        return 0;
    const int jobs = launch == SWIGLU_TRAIN_DY_DW3 || launch == SWIGLU_TRAIN_DA_DW ? 2 : 1;
    const Launch l = plan_launch(jobs, kinds[launch], M, K, N, cu_count_now());
    for (int i = 0; i < jobs; ++i) {
        const Tiles& t = l.t[i];
        const int32_t v[6] = {t.bm, t.bn, t.whole, t.rest, t.splits, t.kb_per_split};
        std::copy(v, v + 6, plan + 6 * i);
    }
    return jobs;
}

}  // extern "C"
