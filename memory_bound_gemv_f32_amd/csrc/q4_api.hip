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
constexpr int kMostRows = 1 << 20, kMostTokens = 1 << 15;

// LDS that the vectors (or their parts) of a call take.
template <class T>
int64_t staged_bytes(const Product& p) {
    return q4dev::Operand<T>::parts * (int64_t)p.T * (ceil_div(p.K, q4dev::kChunk) * q4dev::kChunk * 2 + 16);
}

template <class T, int RT, int NT, int W, int U, bool STAGED>
gemv_status_t few(Product& p, int group, hipStream_t stream) {
    void* argv[] = {&p};
    const dim3 grid((unsigned)ceil_div(p.M, 16 * RT), (unsigned)ceil_div(p.T, 16 * NT));
    const int64_t staged = STAGED ? staged_bytes<T>(p) : 0, sums = RT * NT * W * 64 * 16;
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

// Which kernel.  Few vectors read W straight into registers, in as many rows to a
// workgroup as leave two of them to a compute unit at most (X, which each
// of them reads whole, is what wider row tiles save: of more than 8 vectors they are wide as soon as
// most units have one); past that the tiles, whose X goes
// through LDS.  Measured, us at vectors x rows x K, bf16, groups of 128 (16 rows | 32
// rows | 64 rows | tile of 64 x 64):
//   1 x 4096 x 4096        5.7 |  7.2 | 11.6 | 29.8
//   1 x 14336 x 4096      13.3 | 11.5 | 12.1
//   8 x 14336 x 4096      17.4 | 12.9 | 12.6
//   16 x 4096 x 4096       7.8 |  9.0 | 12.5 | 30.1
//   16 x 14336 x 4096     22.5 | 15.4 | 13.0 | 30.2
//   24 x 14336 x 4096          | 25.6 | 23.6 | 30.6
//   64 x 14336 x 4096          | 47.2 | 45.9 | 32.1
//   128 x 4096 x 4096          | 28.3 | 24.5 | 31.2
//   256 x 4096 x 4096          | 52.9 | 45.7 | 31.4
// and of tiles 64 x 64 | 128 x 128 through registers | 256 x 64 | 256 x 112 | 256 x
// 128 straight into LDS, where every unit's first tile takes some 18 us, and each
// 5.5 us for 16 vectors and 25 besides:
//   512 x 4096 x 4096     42.5 |  86.9 |  60.1 |  81.0 |  88.5
//   1024 x 4096 x 4096    82.1 |  92.7 |  66.4 |  84.3 |  90.1
//   2000 x 4096 x 4096   163.2 | 113.7 | 102.7 | 126.4 |  95.9
//   512 x 14336 x 4096   132.0 | 111.6 |  99.5 | 125.6 |  94.4
//   1024 x 14336 x 4096  246.6 | 206.8 | 180.4 | 192.3 | 143.4
//   2000 x 14336 x 4096  503.1 | 388.1 | 314.0 | 267.3 | 276.6
constexpr int64_t kUnits = 256, kEnoughTiles = 384;
constexpr int64_t kMostStaged = 150 * 1024;  // bytes of LDS for vectors
constexpr int kMostOffset = 1 << 22;         // pitch with which a tile's rows are 32-bit offsets apart

template <class T>
gemv_status_t mapped(Product& p, int group, hipStream_t stream) {
    constexpr bool kParts = q4dev::Operand<T>::parts > 1;
    if (p.K < q4dev::kLeastColumns) {
        void* argv[] = {&p};
        const dim3 grid((unsigned)ceil_div(p.M, 256), (unsigned)p.T);
        return launch((const void*)&q4dev::q4_short_kernel<T>, grid, 256, 0, argv, stream);
    }
    if constexpr (kParts)
        // (1 x 4096 x 11008: 11.1 us; with the parts cut by every wavefront for itself 17)
        if (3 * p.T <= 16 && staged_bytes<T>(p) <= kMostStaged) return few<T, 1, 1, 16, 2, true>(p, group, stream);
    const int64_t tokens = ceil_div(p.T, 16);
    const bool far = p.ldq >= kMostOffset || p.lds >= kMostOffset || p.ldz >= kMostOffset || p.ldx >= kMostOffset;
    if (ceil_div(p.M, 16) * tokens <= kUnits) return few<T, 1, 1, 8, kParts ? 1 : 4, false>(p, group, stream);
    const bool wide_rows = !kParts && p.T > 8 && 4 * ceil_div(p.M, 64) * tokens >= 3 * kUnits;
    if (!wide_rows && ceil_div(p.M, 32) * tokens < 2 * kUnits) return few<T, 2, 1, 8, kParts ? 1 : 4, false>(p, group, stream);
    if (far || ceil_div(p.M, 64) * tokens <= 2 * kUnits) {
        if constexpr (!kParts)
            if (group != 32) return few<T, 4, 1, 8, 4, false>(p, group, stream);
        return few<T, 4, 1, 8, 1, false>(p, group, stream);  // (more would not fit the registers)
    }
    if constexpr (kParts) {
        if (ceil_div(p.M, 128) * ceil_div(p.T, 128) < kEnoughTiles) return tile<T, 1, 4, 4>(p, group, stream);
        return tile<T, 3, 4, 4>(p, group, stream);
    } else {
        if (ceil_div(p.M, 64) * ceil_div(p.T, 64) <= 2 * kUnits) return tile<T, 1, 4, 4>(p, group, stream);
        // (straight into LDS: whole chunks and aligned pieces)
        if (p.K % q4dev::kChunk == 0 && aligned(p.Q, 16) && p.ldq % 16 == 0 && aligned(p.X, 16) && p.ldx % 8 == 0) {
            // a compute unit's tiles, and what one of them takes
            const auto cost = [&](int nt) { return ceil_div(ceil_div(p.M, 256) * ceil_div(p.T, 16 * nt), kUnits) * (2 * nt + 9); };
            if (cost(8) <= cost(7) && cost(8) <= cost(4)) return wide<T, 4, 8, 4>(p, group, stream);
            if (cost(7) <= cost(4)) return wide<T, 4, 7, 4>(p, group, stream);
            return wide<T, 4, 4, 4>(p, group, stream);
        }
        if (ceil_div(p.M, 128) * ceil_div(p.T, 128) < kEnoughTiles) return tile<T, 1, 4, 4>(p, group, stream);
        return tile<T, 2, 8, 4>(p, group, stream);
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
