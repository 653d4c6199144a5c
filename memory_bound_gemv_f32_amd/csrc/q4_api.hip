// libgemv C ABI, the products with 4-bit weights and group scales: argument
// checks, mapping selection and launch.
#include <hip/hip_runtime.h>

#include "../../include/gemv.h"
#include "gemv_launch.hpp"
#include "q4_kernels.hpp"

namespace {

using gemvapi::finish;
using q4dev::Product;
using q4dev::TBF16;
using q4dev::TF16;
using q4dev::TF32;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool aligned(const void* p, int n) { return (uintptr_t)p % n == 0; }

int bytes_of(gemv_dtype_t t) { return t == GEMV_DTYPE_F32 ? 4 : 2; }

gemv_status_t launch(const void* fn, dim3 grid, int threads, int lds_bytes, void** argv, hipStream_t stream) {
    if ((uint64_t)grid.x * threads > 0xffffffffu) return GEMV_ERROR_INVALID_VALUE;  // more than a launch holds
    return finish(hipLaunchKernel(fn, grid, dim3((unsigned)threads), argv, (size_t)lds_bytes, stream));
}

// Of one launch: rows and vectors.
constexpr int kMostRows = 1 << 20, kMostTokens = 1 << 16;

template <class T, int RT, int NT, int W>
gemv_status_t few(Product& p, hipStream_t stream) {
    void* argv[] = {&p};
    const dim3 grid((unsigned)ceil_div(p.M, 16 * RT), (unsigned)ceil_div(p.T, 16 * NT));
    return launch((const void*)&q4dev::q4_few_kernel<T, RT, NT, W>, grid, W * 64, 0, argv, stream);
}

template <class T>
gemv_status_t product(const uint8_t* Q, int ldq, const typename T::storage* scale, int lds, const uint8_t* zero,
                      int ldz, int group, const typename T::storage* X, int ldx, const float* bias, void* Y,
                      gemv_dtype_t y_dtype, int ldy, int M, int K, int nvec, hipStream_t stream) {
    if (M < 0 || K < 0 || nvec < 0 || (group != 32 && group != 64 && group != 128) ||
        (y_dtype != GEMV_DTYPE_F32 && y_dtype != GEMV_DTYPE_F16 && y_dtype != GEMV_DTYPE_BF16))
        return GEMV_ERROR_INVALID_VALUE;
    const int64_t groups = ceil_div(K, group);
    if (ldq < ceil_div(K, 2) || lds < groups || (zero != nullptr && ldz < groups) || ldx < K || ldy < M)
        return GEMV_ERROR_INVALID_VALUE;
    if (M == 0 || nvec == 0) return GEMV_SUCCESS;
    if (Y == nullptr || !aligned(Y, bytes_of(y_dtype)) || !aligned(bias, 4) || !aligned(scale, T::bytes) ||
        !aligned(X, T::bytes))
        return GEMV_ERROR_INVALID_VALUE;
    if (K > 0 && (Q == nullptr || scale == nullptr || X == nullptr)) return GEMV_ERROR_INVALID_VALUE;
    for (int m = 0, rows; m < M; m += rows) {
        rows = M - m < kMostRows ? M - m : kMostRows;
        for (int t = 0, tokens; t < nvec; t += tokens) {
            tokens = nvec - t < kMostTokens ? nvec - t : kMostTokens;
            Product p{};
            p.Q = Q;
            p.ldq = ldq;
            p.scale = scale;
            p.lds = lds;
            p.zero = K > 0 ? zero : nullptr;
            p.ldz = ldz;
            p.X = X;
            p.ldx = ldx;
            if (K > 0) {
                p.Q += m * p.ldq;
                p.scale = scale + m * p.lds;
                if (zero != nullptr) p.zero += m * p.ldz;
                p.X = X + t * p.ldx;
            }
            p.bias = bias != nullptr ? bias + m : nullptr;
            p.Y = static_cast<uint8_t*>(Y) + (t * (int64_t)ldy + m) * bytes_of(y_dtype);
            p.ldy = ldy;
            p.y_type = y_dtype;
            p.M = rows;
            p.K = K;
            p.T = tokens;
            p.group_log2 = group == 32 ? 0 : group == 64 ? 1 : 2;
            const gemv_status_t st = few<T, 1, 1, 16>(p, stream);
            if (st != GEMV_SUCCESS) return st;
        }
    }
    return GEMV_SUCCESS;
}

}  // namespace

#define GEMV_Q4(NAME, D, T)                                                                      \
    extern "C" gemv_status_t gemv_q4_##NAME(                                                     \
        const uint8_t* Q, int ldq, const T* scale, int lds, const uint8_t* zero, int ldz,        \
        int group, const T* X, int ldx, const float* bias, void* Y, gemv_dtype_t y_dtype,        \
        int ldy, int M, int K, int nvec, hipStream_t stream) {                                   \
        return product<D>(Q, ldq, scale, lds, zero, ldz, group, X, ldx, bias, Y, y_dtype, ldy,   \
                          M, K, nvec, stream);                                                   \
    }
GEMV_Q4(f32, TF32, float)
GEMV_Q4(f16, TF16, uint16_t)
GEMV_Q4(bf16, TBF16, uint16_t)
