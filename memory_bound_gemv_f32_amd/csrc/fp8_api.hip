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

gemv_status_t launch(const void* fn, dim3 grid, int threads, void** argv, hipStream_t stream) {
    return finish(hipLaunchKernel(fn, grid, dim3((unsigned)threads), argv, 0, stream));
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
                      fp8dev::kQuantWaves * 64, argv, stream);
    }
    const dim3 grid((unsigned)ceil_div(K, GEMV_FP8_BLOCK), (unsigned)ceil_div(rows, GEMV_FP8_BLOCK));
    if (grid.y > 65535) return GEMV_ERROR_INVALID_VALUE;
    void* argv[] = {&X, &ldx64, &Q, &ldq64, &scale, &lds64, &rows, &K};
    return launch((const void*)&fp8dev::fp8_quantise_tile_kernel<D>, grid,
                  fp8dev::kTileWaves * 64, argv, stream);
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
    void* argv[] = {&W,       &ldw64,  &w_scale, &ldws64, &X, &ldx64, &x_scale,
                    &ldxs64, &bias, &Y, &ldy64, &M, &K, &nvec};
    constexpr int W8 = 8;
    const int nt = nvec <= 16 ? 1 : nvec <= 32 ? 2 : 4;
    const dim3 grid((unsigned)ceil_div(M, 16), (unsigned)ceil_div(nvec, 16 * nt));
    if (grid.y > 65535) return GEMV_ERROR_INVALID_VALUE;
    const void* fn = nt == 1   ? (const void*)&fp8dev::fp8_few_kernel<O, 1, W8>
                     : nt == 2 ? (const void*)&fp8dev::fp8_few_kernel<O, 2, W8>
                               : (const void*)&fp8dev::fp8_few_kernel<O, 4, W8>;
    return launch(fn, grid, W8 * 64, argv, stream);
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
