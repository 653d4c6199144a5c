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

using q4plan::ceil_div;

bool aligned(const void* p, int n) { return (uintptr_t)p % n == 0; }

int bytes_of(gemv_dtype_t t) { return t == GEMV_DTYPE_F32 ? 4 : 2; }

gemv_status_t launch(const void* fn, dim3 grid, int threads, int lds_bytes, void** argv, hipStream_t stream) {
    if ((uint64_t)grid.x * threads > 0xffffffffu) return GEMV_ERROR_INVALID_VALUE;  // more than a launch holds
    return finish(hipLaunchKernel(fn, grid, dim3((unsigned)threads), argv, (size_t)lds_bytes, stream));
}

using q4plan::kMostRows;
using q4plan::kMostTokens;

template <class T, int RT, int NT, int W, int U, bool STAGED>
gemv_status_t few(Product& p, int group, hipStream_t stream) {
    void* argv[] = {&p};
    const dim3 grid((unsigned)ceil_div(p.M, 16 * RT), (unsigned)ceil_div(p.T, 16 * NT));
    const int64_t staged = STAGED ? q4plan::staged_bytes(q4dev::Operand<T>::parts, p.K, p.T) : 0, sums = RT * NT * W * 64 * 16;
    const void* fn = nullptr;
    if constexpr (RT * U <= 8)  // (groups of 32 with more than that would not fit the registers)
        if (group == 32) fn = (const void*)&q4dev::q4_few_kernel<T, 0, RT, NT, W, U, STAGED>;
    if (fn == nullptr)
        fn = group == 64 ? (const void*)&q4dev::q4_few_kernel<T, 1, RT, NT, W, U, STAGED>
                         : (const void*)&q4dev::q4_few_kernel<T, 2, RT, NT, W, U, STAGED>;
    return launch(fn, grid, W * 64, (int)(staged > sums ? staged : sums), argv, stream);
}

template <class T, int RT, int NT, int W>
gemv_status_t tile(Product& p, int group, hipStream_t stream) {
    int row_tiles = (int)ceil_div(p.M, 16 * RT * W);
    void* argv[] = {&p, &row_tiles};
    const dim3 grid((unsigned)(row_tiles * ceil_div(p.T, 16 * NT)));
    const int lds = 2 * 16 * NT * 256 * q4dev::Operand<T>::parts;
    const void* fn = group == 32   ? (const void*)&q4dev::q4_tile_kernel<T, 0, RT, NT, W>
                     : group == 64 ? (const void*)&q4dev::q4_tile_kernel<T, 1, RT, NT, W>
                                   : (const void*)&q4dev::q4_tile_kernel<T, 2, RT, NT, W>;
    return launch(fn, grid, W * 64, lds, argv, stream);
}

template <class T, int RT, int NT, int W>
gemv_status_t wide(Product& p, int group, hipStream_t stream) {
    int row_tiles = (int)ceil_div(p.M, 16 * RT * W);
    void* argv[] = {&p, &row_tiles};
    const dim3 grid((unsigned)(row_tiles * ceil_div(p.T, 16 * NT)));
    const int lds = 2 * 16 * NT * 256 + 16 * RT * W * 64;
    const void* fn = group == 32   ? (const void*)&q4dev::q4_wide_kernel<T, 0, RT, NT, W>
                     : group == 64 ? (const void*)&q4dev::q4_wide_kernel<T, 1, RT, NT, W>
                                   : (const void*)&q4dev::q4_wide_kernel<T, 2, RT, NT, W>;
    return launch(fn, grid, W * 64, lds, argv, stream);
}

// The kernel that q4plan::family_of names.
template <class T>
gemv_status_t mapped(Product& p, int group, hipStream_t stream) {
    constexpr bool kParts = q4dev::Operand<T>::parts > 1;
    const int64_t pitches[] = {p.ldq, p.lds, p.ldz, p.ldx};
    bool far = false;
    for (const int64_t pitch : pitches) far = far || pitch >= q4plan::kMostOffset;
    const bool whole = p.K % q4dev::kChunk == 0 && aligned(p.Q, 16) && p.ldq % 16 == 0 && aligned(p.X, 16) && p.ldx % 8 == 0;
    const q4plan::Family family = q4plan::family_of(q4dev::Operand<T>::parts, p.M, p.K, p.T, far, whole);
    if (family == q4plan::kShort) {
        void* argv[] = {&p};
        const dim3 grid((unsigned)ceil_div(p.M, 256), (unsigned)p.T);
        return launch((const void*)&q4dev::q4_short_kernel<T>, grid, 256, 0, argv, stream);
    }
    if (family == q4plan::kFew16) return few<T, 1, 1, 8, kParts ? 1 : 4, false>(p, group, stream);
    if (family == q4plan::kFew32) return few<T, 2, 1, 8, kParts ? 1 : 4, false>(p, group, stream);
    if (family == q4plan::kTile64) return tile<T, 1, 4, 4>(p, group, stream);
    if constexpr (kParts) {
        if (family == q4plan::kStaged) return few<T, 1, 1, 16, 2, true>(p, group, stream);
        if (family == q4plan::kFew64) return few<T, 4, 1, 8, 1, false>(p, group, stream);
        return tile<T, 3, 4, 4>(p, group, stream);
    } else {
        // (more chunks at once than one would not fit the registers with groups of 32)
        if (family == q4plan::kFew64)
            return group == 32 ? few<T, 4, 1, 8, 1, false>(p, group, stream) : few<T, 4, 1, 8, 4, false>(p, group, stream);
        if (family == q4plan::kTile128) return tile<T, 2, 8, 4>(p, group, stream);
        if (family == q4plan::kWide64) return wide<T, 4, 4, 4>(p, group, stream);
        if (family == q4plan::kWide112) return wide<T, 4, 7, 4>(p, group, stream);
        return wide<T, 4, 8, 4>(p, group, stream);
    }
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
            // (without zeros the kernels load bytes of the scales, and use none)
            p.zero = zero != nullptr ? zero : reinterpret_cast<const uint8_t*>(scale);
            p.ldz = zero != nullptr ? ldz : lds * (int64_t)T::bytes;
            p.zero_mask = zero != nullptr ? 0xffffffffu : 0u;
            p.no_zero = zero != nullptr ? 0u : q4dev::kNoZero * 0x01010101u;
            p.X = X;
            p.ldx = ldx;
            if (K > 0) {
                p.Q += m * p.ldq;
                p.scale = scale + m * p.lds;
                p.zero += m * p.ldz;
                p.X = X + t * p.ldx;
            }
            p.bias = bias != nullptr ? bias + m : nullptr;
            p.Y = static_cast<uint8_t*>(Y) + (t * (int64_t)ldy + m) * bytes_of(y_dtype);
            p.ldy = ldy;
            p.y_type = y_dtype;
            p.M = rows;
            p.K = K;
            p.T = tokens;
            const gemv_status_t st = mapped<T>(p, group, stream);
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
