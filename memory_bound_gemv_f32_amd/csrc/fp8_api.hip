// libgemv C ABI, the e4m3 operators with a scale for each block of 128:
// argument checks, mapping selection and launch.
#include <hip/hip_runtime.h>

#include "../../include/gemv.h"
#include "fp8_kernels.hpp"
#include "gemv_launch.hpp"

namespace {

using fp8dev::TBF16;
using fp8dev::TF16;
using fp8dev::TF32;
using gemvapi::finish;

static_assert(GEMV_FP8_BLOCK == fp8dev::kScaleBlock, "the header states the block");

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool aligned(const void* p, int n) { return (uintptr_t)p % n == 0; }

gemv_status_t launch(const void* fn, dim3 grid, int threads, int lds_bytes, void** argv,
                     hipStream_t stream) {
    if ((uint64_t)grid.x * threads > 0xffffffffu) return GEMV_ERROR_INVALID_VALUE;  // more than a launch holds
    return finish(hipLaunchKernel(fn, grid, dim3((unsigned)threads), argv, (size_t)lds_bytes, stream));
}

// ---- the product's mapping ---------------------------------------------------

using fp8dev::Split;
using Large = fp8dev::Tile<128, 128, 64, 32, 2, 8>;
using Medium = fp8dev::Tile<128, 64, 32, 32, 4, 8>;
using Split64 = Split<64, 64, 2>;
using Split32 = Split<64, 32, 3>;
using Split16 = Split<64, 16, 3>;

constexpr int kFewTokens = 16, kFewRows = 8192, kFewWaves = 16, kFewBlocks = 2;
constexpr int kExactTokens = 32;  // up to so many, every result takes the exact steps
constexpr int64_t kUnits = 256, kEnoughTiles = 192;
// Of one launch, whose threads a 32-bit number counts: rows of W and tokens of
// the product, wavefronts of the quantiser, columns of its 128 x 128 blocks.
constexpr int kMostRows = 1 << 20, kMostTokens = 1 << 16, kMostUnits = 1 << 25, kMostColumns = 1 << 29;

// A kernel and what its launch needs.
struct Tiled {
    const void* fn;
    int block_m, block_n, threads, lds_bytes;
};

template <class C>
Tiled tiled(const void* fn) {
    return Tiled{fn, C::BM, C::BN, C::kWaves * 64, C::kLds};
}

template <class O, class C>
Tiled tile_kernel(bool direct) {
    // fp32 results take the exact steps: the e4m3 ones' 2^-15 would show
    constexpr bool kExact = O::bytes == 4;
    return tiled<C>(direct ? (const void*)&fp8dev::fp8_tile_kernel<O, C, kExact, true>
                           : (const void*)&fp8dev::fp8_tile_kernel<O, C, kExact, false>);
}

template <class O, class C>
Tiled split_kernel(bool direct, bool exact) {
    if constexpr (O::bytes == 2)
        if (!exact)
            return tiled<C>(direct ? (const void*)&fp8dev::fp8_split_kernel<O, C, false, true>
                                   : (const void*)&fp8dev::fp8_split_kernel<O, C, false, false>);
    return tiled<C>(direct ? (const void*)&fp8dev::fp8_split_kernel<O, C, true, true>
                           : (const void*)&fp8dev::fp8_split_kernel<O, C, true, false>);
}

template <class C>
int64_t tiles_of(int M, int nvec) {
    return ceil_div(M, C::BM) * ceil_div(nvec, C::BN);
}

// Which tile, for everything but few tokens of few rows.  The split kernels, with
// the narrowest token tile that keeps a workgroup to each compute unit at most,
// win wherever they fit; past that the larger tile, which moves fewer bytes,
// where it fills three quarters of the units.  Measured, us at
// tokens x rows x K, bf16 (Split16 | Split32 | Split64 | Medium | Large):
//   16 x 14336 x 4096      12.1 |   13.4 |   15.9 |   18.0 |   25.0
//   64 x 4096 x 4096       10.0 |   10.1 |   12.5 |   17.1 |   23.3
//   128 x 4096 x 4096      15.8 |   10.3 |   12.7 |   17.4 |   24.1
//   192 x 4096 x 4096      22.5 |   18.2 |   13.5 |   18.1 |   24.6
//   250 x 4096 x 11008     61.5 |   38.1 |   29.6 |   40.7 |   61.6
//   300 x 4096 x 4096      34.3 |   24.3 |   22.7 |   17.9 |   24.7
//   512 x 4096 x 4096      55.6 |   32.1 |   24.0 |   18.8 |   24.8
//   768 x 4096 x 4096      78.7 |   46.3 |   35.7 |   33.1 |   25.6
//   1024 x 4096 x 4096    108.4 |   65.0 |   48.7 |   34.6 |   27.1
//   4096 x 14336 x 4096  1528.2 |  936.3 |  801.9 |  442.0 |  276.1
template <class O>
Tiled tiled_kernel(int M, int nvec, bool direct) {
    const bool exact = nvec <= kExactTokens;
    if (nvec <= kFewTokens || tiles_of<Split16>(M, nvec) <= kUnits)
        return split_kernel<O, Split16>(direct, exact);
    if (nvec <= 32 || tiles_of<Split32>(M, nvec) <= kUnits) return split_kernel<O, Split32>(direct, exact);
    if (tiles_of<Split64>(M, nvec) <= kUnits) return split_kernel<O, Split64>(direct, O::bytes == 4);
    if (tiles_of<Large>(M, nvec) >= kEnoughTiles) return tile_kernel<O, Large>(direct);
    return tile_kernel<O, Medium>(direct);
}

template <class D>
gemv_status_t quantise(const typename D::storage* X, int ldx, uint8_t* Q, int ldq, float* scale,
                       int lds, int rows, int K, int block_rows, hipStream_t stream) {
    if (rows < 0 || K < 0 || ldx < K || ldq < K ||
        (block_rows != 1 && block_rows != GEMV_FP8_BLOCK) || lds < ceil_div(K, GEMV_FP8_BLOCK))
        return GEMV_ERROR_INVALID_VALUE;
    if (rows == 0 || K == 0) return GEMV_SUCCESS;
    if (X == nullptr || Q == nullptr || scale == nullptr || !aligned(X, D::bytes) || !aligned(scale, 4))
        return GEMV_ERROR_INVALID_VALUE;
    int64_t ldx64 = ldx, ldq64 = ldq, lds64 = lds;
    if (block_rows == 1) {
        int per_row = (int)ceil_div(K, 512);
        int64_t units = 0;
        void* argv[] = {&X, &ldx64, &Q, &ldq64, &scale, &lds64, &units, &per_row, &K};
        const int most = kMostUnits / per_row;  // rows of a launch
        for (int r = 0, n; r < rows; r += n) {
            n = rows - r < most ? rows - r : most;
            units = (int64_t)n * per_row;
            const gemv_status_t st =
                launch((const void*)&fp8dev::fp8_quantise_rows_kernel<D>,
                       dim3((unsigned)ceil_div(units, fp8dev::kQuantWaves)), fp8dev::kQuantWaves * 64, 0, argv, stream);
            if (st != GEMV_SUCCESS) return st;
            X += n * ldx64;
            Q += n * ldq64;
            scale += n * lds64;
        }
        return GEMV_SUCCESS;
    }
    const int64_t lines = ceil_div(rows, GEMV_FP8_BLOCK);
    if (lines > 65535) return GEMV_ERROR_INVALID_VALUE;
    int columns = 0;
    void* argv[] = {&X, &ldx64, &Q, &ldq64, &scale, &lds64, &rows, &columns};
    for (int k = 0; k < K; k += columns) {
        columns = K - k < kMostColumns ? K - k : kMostColumns;
        const dim3 grid((unsigned)ceil_div(columns, GEMV_FP8_BLOCK), (unsigned)lines);
        const gemv_status_t st = launch((const void*)&fp8dev::fp8_quantise_tile_kernel<D>, grid,
                                        fp8dev::kTileWaves * 64, 0, argv, stream);
        if (st != GEMV_SUCCESS) return st;
        X += columns;
        Q += columns;
        scale += columns / GEMV_FP8_BLOCK;  // (whole blocks but for the last launch)
    }
    return GEMV_SUCCESS;
}

template <class O>
gemv_status_t product(const uint8_t* W, int ldw, const float* w_scale, int ldws, const uint8_t* X,
                      int ldx, const float* x_scale, int ldxs, const float* bias,
                      typename O::storage* Y, int ldy, int M, int K, int nvec, hipStream_t stream) {
    const int64_t blocks = ceil_div(K, GEMV_FP8_BLOCK);
    if (M < 0 || K < 0 || nvec < 0 || ldw < K || ldx < K || ldy < M || ldws < blocks ||
        ldxs < blocks)
        return GEMV_ERROR_INVALID_VALUE;
    if (M == 0 || nvec == 0) return GEMV_SUCCESS;
    if (Y == nullptr || !aligned(Y, O::bytes) || !aligned(bias, 4) || !aligned(w_scale, 4) ||
        !aligned(x_scale, 4))
        return GEMV_ERROR_INVALID_VALUE;
    if (K > 0 && (W == nullptr || X == nullptr || w_scale == nullptr || x_scale == nullptr))
        return GEMV_ERROR_INVALID_VALUE;
    int64_t ldw64 = ldw, ldws64 = ldws, ldx64 = ldx, ldxs64 = ldxs, ldy64 = ldy;
    // whole, aligned 16-byte pieces may be loaded straight into LDS (with
    // 32-bit offsets within 8 rows)
    const bool direct = K % 16 == 0 && ldw % 16 == 0 && ldx % 16 == 0 && aligned(W, 16) &&
                        aligned(X, 16) && ldw < (1 << 28) && ldx < (1 << 28);
    // few tokens of few rows: a workgroup for each 16 rows reads W straight into
    // registers (16 x 4096 x 4096: 7.6 us against 7.9 in LDS; 16 x 8192 x 4096: 13.2
    // against 12.0), and so wherever each of these, with 16 tokens, has a compute
    // unit (32 x 512 x 8192: 12.1 against 14.3; 30 x 1024 x 11008: 14.7 against
    // 17.9; 64 x 1024 x 4096: 9.1 against 9.4).  Also the empty sum, and scales too
    // far apart for the tiles' 32-bit offsets.
    const bool few = (nvec <= kFewTokens && M < kFewRows) || ceil_div(M, 16) * ceil_div(nvec, 16) <= kUnits ||
                     K == 0 || ldws >= (1 << 26) || ldxs >= (1 << 26);
    for (int m = 0, rows; m < M; m += rows) {
        rows = M - m < kMostRows ? M - m : kMostRows;
        for (int t = 0, tokens; t < nvec; t += tokens) {
            tokens = nvec - t < kMostTokens ? nvec - t : kMostTokens;
            const uint8_t *w = W, *x = X;
            const float *ws = w_scale, *xs = x_scale, *add = bias;
            if (K > 0) {
                w += m * ldw64;
                ws += m / GEMV_FP8_BLOCK * ldws64;
                x += t * ldx64;
                xs += t * ldxs64;
            }
            if (bias != nullptr) add += m;
            typename O::storage* y = Y + t * ldy64 + m;
            int row_tiles = 0;
            void* argv[] = {&w,   &ldw64, &ws,    &ldws64, &x, &ldx64,  &xs,       &ldxs64,
                            &add, &y,     &ldy64, &rows,   &K, &tokens, &row_tiles};
            gemv_status_t st;
            if (few) {
                const dim3 grid((unsigned)ceil_div(rows, 16), (unsigned)ceil_div(tokens, 16));
                st = launch((const void*)&fp8dev::fp8_few_kernel<O, kFewWaves, kFewBlocks>, grid, kFewWaves * 64, 0,
                            argv, stream);
            } else {
                const Tiled k = tiled_kernel<O>(rows, tokens, direct);
                row_tiles = (int)ceil_div(rows, k.block_m);
                st = launch(k.fn, dim3((unsigned)(row_tiles * ceil_div(tokens, k.block_n))), k.threads, k.lds_bytes,
                            argv, stream);
            }
            if (st != GEMV_SUCCESS) return st;
        }
    }
    return GEMV_SUCCESS;
}

}  // namespace

#define GEMV_FP8_QUANTISE(NAME, D, T)                                                            \
    extern "C" gemv_status_t gemv_fp8_quantise_##NAME(const T* X, int ldx, uint8_t* Q, int ldq,  \
                                                      float* scale, int lds, int rows, int K,    \
                                                      int block_rows, hipStream_t stream) {      \
        return quantise<D>(X, ldx, Q, ldq, scale, lds, rows, K, block_rows, stream);             \
    }
GEMV_FP8_QUANTISE(f32, TF32, float)
GEMV_FP8_QUANTISE(f16, TF16, uint16_t)
GEMV_FP8_QUANTISE(bf16, TBF16, uint16_t)

#define GEMV_FP8(NAME, O, T)                                                                     \
    extern "C" gemv_status_t gemv_fp8_##NAME(                                                    \
        const uint8_t* W, int ldw, const float* w_scale, int ldws, const uint8_t* X, int ldx,    \
        const float* x_scale, int ldxs, const float* bias, T* Y, int ldy, int M, int K,          \
        int nvec, hipStream_t stream) {                                                          \
        return product<O>(W, ldw, w_scale, ldws, X, ldx, x_scale, ldxs, bias, Y, ldy, M, K,      \
                          nvec, stream);                                                         \
    }
GEMV_FP8(f32, TF32, float)
GEMV_FP8(f16, TF16, uint16_t)
GEMV_FP8(bf16, TBF16, uint16_t)
