// Kernels of the e4m3 operators with a scale for each block of 128: the
// quantiser and the matrix product.
#pragma once

#include "fp8_device.hpp"

namespace fp8dev {

constexpr int kScaleBlock = 128;  // columns (and weight rows) that share a scale

// ---------------------------------------------------------------------------
// quantiser
//
//   scale = max(amax / 448, 2^-126),   q = e4m3(x · (1/scale))
//
// The division and the reciprocal are IEEE fp32, so the values are the same
// whatever computes the formula; the product is rounded to fp32 and then to
// e4m3.  A block that holds an infinity or NaN gets that as its scale.
// ---------------------------------------------------------------------------

// Eight consecutive elements of a row, widened to fp32; those from `n` on
// read as zero and are not touched.
template <class D>
__device__ __forceinline__ void load8(const typename D::storage* p, int n, float (&v)[8]) {
    if (n >= 8) {
        if constexpr (D::bytes == 4) {
            const quad a = *reinterpret_cast<const quad_any*>(p);
            const quad b = *reinterpret_cast<const quad_any*>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = gemvdev::f32_of(a[i]);
                v[4 + i] = gemvdev::f32_of(b[i]);
            }
        } else {
            const quad a = *reinterpret_cast<const quad_any*>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = widen(D{}, (uint16_t)(a[i] & 0xffffu));
                v[2 * i + 1] = widen(D{}, (uint16_t)(a[i] >> 16));
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? widen(D{}, p[i]) : 0.0f;
}

__device__ __forceinline__ void store8(uint8_t* p, int n, u32x2 w) {
    if (n >= 8) {
        *reinterpret_cast<u32x2_any*>(p) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
}

__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
    const float s = __builtin_bit_cast(float, amax_bits) / kE4m3Max;
    return s < kSmallestScale ? kSmallestScale : s;  // NaN stays
}

// One scale per row and 128 columns.  16 lanes hold a block, 8 elements
// each, so a wavefront takes 512 consecutive columns of a row.
constexpr int kQuantWaves = 4;
template <class D>
__global__ __launch_bounds__(kQuantWaves * 64) void fp8_quantise_rows_kernel(
    const typename D::storage* X, int64_t ldx, uint8_t* Q, int64_t ldq, float* scale, int64_t lds,
    int64_t units, int units_per_row, int K) {
    const int64_t unit = (int64_t)blockIdx.x * kQuantWaves + (threadIdx.x >> 6);
    if (unit >= units) return;
    const int lane = threadIdx.x & 63;
    const int64_t row = unit / units_per_row;
    const int64_t col = (unit - row * units_per_row) * 512 + lane * 8;
    const int n = (int)(K - col);
    float v[8];
    load8<D>(X + row * ldx + col, n, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_u32(m, magnitude(v[i]));
    const float s = scale_of(row_max16(m));
    const float inv = 1.0f / s;
    u32x2 w;
    w[0] = to_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    w[1] = to_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    if (n > 0) {
        store8(Q + row * ldq + col, n, w);
        if ((lane & 15) == 0) scale[row * lds + col / kScaleBlock] = s;
    }
}

// One scale per 128 rows and 128 columns: a workgroup holds the block in
// registers, 16 lanes a row, and reduces its maximum through LDS.
constexpr int kTileWaves = 8;
template <class D>
__global__ __launch_bounds__(kTileWaves * 64) void fp8_quantise_tile_kernel(
    const typename D::storage* X, int64_t ldx, uint8_t* Q, int64_t ldq, float* scale, int64_t lds,
    int rows, int K) {
    constexpr int kPerLane = kScaleBlock / (kTileWaves * 4);
    __shared__ uint32_t part[kTileWaves];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int col = (int)blockIdx.x * kScaleBlock + (lane & 15) * 8;
    const int row0 = (int)blockIdx.y * kScaleBlock + wave * 4 + (lane >> 4);
    const int n = K - col;
    float v[kPerLane][8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
        const int row = row0 + j * kTileWaves * 4;
        load8<D>(X + (int64_t)row * ldx + col, row < rows ? n : 0, v[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_u32(m, magnitude(v[j][i]));
    }
    m = wave_max(m);
    if (lane == 0) part[wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTileWaves; ++w) m = max_u32(m, part[w]);
    const float s = scale_of(m);
    const float inv = 1.0f / s;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
        const int row = row0 + j * kTileWaves * 4;
        u32x2 w;
        w[0] = to_e4m3x4(v[j][0] * inv, v[j][1] * inv, v[j][2] * inv, v[j][3] * inv);
        w[1] = to_e4m3x4(v[j][4] * inv, v[j][5] * inv, v[j][6] * inv, v[j][7] * inv);
        if (row < rows && n > 0) store8(Q + (int64_t)row * ldq + col, n, w);
    }
    if (threadIdx.x == 0) scale[(int64_t)blockIdx.y * lds + blockIdx.x] = s;
}

// ---------------------------------------------------------------------------
// product   Y[t,m] = Σ_b sx[t,b]·sw[m/128,b]·Σ_{k in block b} W[m,k]·X[t,k] + bias[m]
//
// The 128 products of a block are taken by 16×16×32 fp16 matrix-core steps on
// exactly widened values: A is 16 rows of W, B 16 tokens of X.  Measured, a
// block's sum is then within 4e-8 of Σ|products|; the e4m3 steps (16×16×32
// and 16×16×128 alike) align their products to fewer bits and reach 2e-5.
// The order of the products is free as long as A and B agree, so lane l takes
// row (or token) l % 16 and the bytes 16·(l/16) .. +15 and 64 + 16·(l/16) ..
// +15 of the block: one load instruction then covers 64 consecutive bytes of
// each row.  The block's sum starts from zero; it is scaled and added in fp32.
// ---------------------------------------------------------------------------

// 8 e4m3 bytes as fp16, exactly.
__device__ __forceinline__ quad widen8(int lo, int hi) {
    return quad{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true))};
}

struct Wide {
    quad step[4];
};
__device__ __forceinline__ Wide widen32(i32x8 v) {
    Wide w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w.step[i] = widen8(v[2 * i], v[2 * i + 1]);
    return w;
}
__device__ __forceinline__ f32x4 mma_block(const Wide& a, const Wide& b) {
    f32x4 d{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = gemvdev::mma_16x16x32(TF16{}, a.step[i], b.step[i], d);
    return d;
}

__device__ __forceinline__ i32x8 join(quad lo, quad hi) {
    i32x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = (int)lo[i];
        r[4 + i] = (int)hi[i];
    }
    return r;
}

// The lane's 32 bytes of a block that starts at column k of the row at p.
__device__ __forceinline__ i32x8 load_block(const uint8_t* p, int k, int group, int K) {
    const uint8_t* at = p + k + 16 * group;
    const int n = K - k - 16 * group;
    if (K - k >= kScaleBlock)
        return join(*reinterpret_cast<const quad_any*>(at),
                    *reinterpret_cast<const quad_any*>(at + 64));
    return join(load_bytes(at, n), load_bytes(at + 64, n - 64));
}

template <class O>
__device__ __forceinline__ void store_y(void* Y, int64_t i, float v) {
    static_cast<typename O::storage*>(Y)[i] = narrow(O{}, v);
}

// 16 rows of W by 16·NT tokens to a workgroup; its wavefronts take the scale
// blocks in turn and add their sums in LDS, in a fixed order.
template <class O, int NT, int W>
__global__ __launch_bounds__(W * 64) void fp8_few_kernel(
    const uint8_t* A, int64_t lda, const float* as, int64_t ldas, const uint8_t* X, int64_t ldx,
    const float* xs, int64_t ldxs, const float* bias, void* Y, int64_t ldy, int M, int K, int T) {
    __shared__ f32x4 part[W][NT][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int r = lane & 15, group = lane >> 4;
    const int row0 = (int)blockIdx.x * 16;
    const int t0 = (int)blockIdx.y * 16 * NT;
    const int blocks = K / kScaleBlock + (K % kScaleBlock != 0);
    // rows and tokens past the end repeat the last one; their results are not stored
    const int row = row0 + r < M ? row0 + r : M - 1;
    const uint8_t* a = A + (int64_t)row * lda;
    const float* asr = as + (int64_t)(row0 / kScaleBlock) * ldas;
    const uint8_t* x[NT];
    const float* xsr[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int t = t0 + 16 * i + r < T ? t0 + 16 * i + r : T - 1;
        x[i] = X + (int64_t)t * ldx;
        xsr[i] = xs + (int64_t)t * ldxs;
    }
    f32x4 acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = wave; b < blocks; b += W) {
        const Wide af = widen32(load_block(a, b * kScaleBlock, group, K));
        const float s = asr[b];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const Wide xf = widen32(load_block(x[i], b * kScaleBlock, group, K));
            const float st = s * xsr[i][b];
            const f32x4 d = mma_block(af, xf);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_fmaf(d[j], st, acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    for (int e = threadIdx.x; e < NT * 64; e += W * 64) {
        const int i = e >> 6, l = e & 63;
        f32x4 v = part[0][i][l];
#pragma unroll
        for (int w = 1; w < W; ++w) v += part[w][i][l];
        const int t = t0 + 16 * i + (l & 15);
        if (t < T)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = row0 + 4 * (l >> 4) + j;
                if (m < M) store_y<O>(Y, (int64_t)t * ldy + m, bias ? v[j] + bias[m] : v[j]);
            }
    }
}

}  // namespace fp8dev
