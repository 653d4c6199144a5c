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
    return finish(hipLaunchKernel(fn, grid, dim3((unsigned)threads), argv, (size_t)lds_bytes, stream));
}

// ---- the product's mapping ---------------------------------------------------

// Up to so many tokens a workgroup takes 16 rows of W with all the tokens.
constexpr int kFewTokens = 32;
constexpr int kFewWaves = 8;

// 128 x 128 tiles move the fewest bytes, 128 x 64 and 64 x 64 give more
// workgroups, the split gives more wavefronts to a workgroup.  The largest
// that fills three quarters of the compute units is taken; measured, us at
// 1024 x 4096 x 4096 (tokens x rows x K): 33 | 32 | 40 | 58; 512 x 4096 x 4096:
// 31 | 19 | 22 | 28; 250 x 4096 x 11008: 82 | 45 | 35 | 38; 128 x 4096 x 4096:
// 26 | 18 | 15 | 12.
using Large = fp8dev::Tile<128, 128, 64, 32, 2, 8>;
using Medium = fp8dev::Tile<128, 64, 32, 32, 4, 8>;
using Small = fp8dev::Tile<64, 64, 32, 16, 4, 8>;
constexpr int64_t kEnoughTiles = 192;

template <class O, class C, bool EXACT>
const void* tile_fn(bool direct) {
    return direct ? (const void*)&fp8dev::fp8_tile_kernel<O, C, EXACT, true>
                  : (const void*)&fp8dev::fp8_tile_kernel<O, C, EXACT, false>;
}

template <class O>
const void* tiled_kernel(int M, int nvec, bool direct, int* block_m, int* block_n, int* threads,
                         int* lds_bytes) {
    // fp32 results take the exact steps: the e4m3 ones' 2^-15 would show
    constexpr bool kExact = O::bytes == 4;
    const auto use = [&](auto c, const void* fn) {
        using C = decltype(c);
        *block_m = C::BM;
        *block_n = C::BN;
        *threads = C::kWaves * 64;
        *lds_bytes = C::kLds;
        return fn;
    };
    const auto tiles = [&](auto c) {
        using C = decltype(c);
        return ceil_div(M, C::BM) * ceil_div(nvec, C::BN);
    };
    if (tiles(Large{}) >= kEnoughTiles) return use(Large{}, tile_fn<O, Large, kExact>(direct));
    if (tiles(Medium{}) >= kEnoughTiles) return use(Medium{}, tile_fn<O, Medium, kExact>(direct));
    if (tiles(Small{}) >= kEnoughTiles) return use(Small{}, tile_fn<O, Small, kExact>(direct));
    return use(fp8dev::Split{}, direct ? (const void*)&fp8dev::fp8_split_kernel<O, kExact, true>
                                       : (const void*)&fp8dev::fp8_split_kernel<O, kExact, false>);
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
        int64_t units = (int64_t)rows * per_row;
        const int64_t grid = ceil_div(units, fp8dev::kQuantWaves);
        if (grid > 0x7fffffff) return GEMV_ERROR_INVALID_VALUE;
        void* argv[] = {&X, &ldx64, &Q, &ldq64, &scale, &lds64, &units, &per_row, &K};
        return launch((const void*)&fp8dev::fp8_quantise_rows_kernel<D>, dim3((unsigned)grid),
                      fp8dev::kQuantWaves * 64, 0, argv, stream);
    }
    const dim3 grid((unsigned)ceil_div(K, GEMV_FP8_BLOCK), (unsigned)ceil_div(rows, GEMV_FP8_BLOCK));
    if (grid.y > 65535) return GEMV_ERROR_INVALID_VALUE;
    void* argv[] = {&X, &ldx64, &Q, &ldq64, &scale, &lds64, &rows, &K};
    return launch((const void*)&fp8dev::fp8_quantise_tile_kernel<D>, grid,
                  fp8dev::kTileWaves * 64, 0, argv, stream);
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
    // pieces of 16 bytes that may be loaded straight into LDS (with 32-bit
    // offsets within 8 rows)
    int whole_pieces = ldw % 16 == 0 && ldx % 16 == 0 && aligned(W, 16) && aligned(X, 16) &&
                       ldw < (1 << 28) && ldx < (1 << 28);
    int row_tiles = 0, tokens = nvec;
    void* argv[] = {&W,     &ldw64, &w_scale, &ldws64, &X, &ldx64,  &x_scale,   &ldxs64,
                    &bias,  &Y,     &ldy64,   &M,      &K, &tokens, &row_tiles, &whole_pieces};
    // also the empty sum, and scales too far apart for the tiles' 32-bit offsets
    if (nvec <= kFewTokens || K == 0 || ldws >= (1 << 26) || ldxs >= (1 << 26)) {
        const int nt = nvec <= 16 ? 1 : 2;
        const void* fn = nt == 1 ? (const void*)&fp8dev::fp8_few_kernel<O, 1, 1, kFewWaves, 4>
                                 : (const void*)&fp8dev::fp8_few_kernel<O, 2, 1, kFewWaves, 2>;
        constexpr int kMostTokens = 65535 * 32;  // of one launch
        for (int t = 0; t < nvec; t += tokens) {
            tokens = nvec - t < kMostTokens ? nvec - t : kMostTokens;
            const dim3 grid((unsigned)ceil_div(M, 16), (unsigned)ceil_div(tokens, 16 * nt));
            const gemv_status_t st = launch(fn, grid, kFewWaves * 64, 0, argv, stream);
            if (st != GEMV_SUCCESS) return st;
            if (K > 0) {
                X += tokens * ldx64;
                x_scale += tokens * ldxs64;
            }
            Y += tokens * ldy64;
        }
        return GEMV_SUCCESS;
    }
    const bool direct = whole_pieces && K % GEMV_FP8_BLOCK == 0;
    int block_m, block_n, threads, lds_bytes;
    const void* fn = tiled_kernel<O>(M, nvec, direct, &block_m, &block_n, &threads, &lds_bytes);
    row_tiles = (int)ceil_div(M, block_m);
    const int64_t grid = row_tiles * ceil_div(nvec, block_n);
    if (grid > 0x7fffffff) return GEMV_ERROR_INVALID_VALUE;
    return launch(fn, dim3((unsigned)grid), threads, lds_bytes, argv, stream);
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
