// Kernels of the products with 4-bit weights and group scales.
//
//   Y[t,m] = Σ_g scale[m,g]·Σ_{k in g} (q[m,k] - zero[m,g])·X[t,k] + bias[m]
//
// q - zero is a whole number of at most 8 bits, so fp16 and bf16 hold it, and
// the matrix cores' products with X are exact; a group's products are summed
// in fp32 and its sum is scaled and added in fp32.  fp32 vectors go to the
// matrix cores as three bf16 parts that add up to them exactly.
#pragma once

#include "fp8_device.hpp"

namespace q4dev {

using fp8dev::bf16x2;
using fp8dev::f16x2;
using fp8dev::f32x4;
using fp8dev::quad;
using fp8dev::quad_any;
using fp8dev::TBF16;
using fp8dev::TF16;
using fp8dev::TF32;
using fp8dev::u32x2;
using fp8dev::widen;

constexpr int kChunk = 128;      // columns of a step: 16 bytes to a lane
constexpr int kBlock = 32;       // columns of a matrix-core step
constexpr int kNoZero = 8;       // the zero of weights without zeros

struct Product {
    const uint8_t* Q;
    int64_t ldq;
    const void* scale;
    int64_t lds;
    const uint8_t* zero;         // NULL: kNoZero everywhere
    int64_t ldz;
    const void* X;
    int64_t ldx;
    const float* bias;           // or NULL
    void* Y;
    int64_t ldy;
    int y_type;                  // gemv_dtype_t
    int M, K, T;
    int group_log2;              // columns of a group over kBlock, as a power of two: 0, 1 or 2
};

// The type that X meets the weights in, and in how many parts.
template <class T>
struct Operand {
    using type = T;
    static constexpr int parts = 1;
};
template <>
struct Operand<TF32> {
    using type = TBF16;
    static constexpr int parts = 3;
};

// ---------------------------------------------------------------------------
// weights
//
// A word holds eight columns, the first in its lowest four bits.  Shifted right
// by 4·i its two halves' lowest bits are columns i and i + 4, so the eight
// values come out as the pairs (0,4), (1,5), (2,6), (3,7); X is taken in the same
// order.  With 1024's exponent around them the four bits are the fp16 number
// 1024 + q, from which 1024 + zero is taken exactly.
// ---------------------------------------------------------------------------

// 1024 + zero, twice.
__device__ __forceinline__ uint32_t offset_of(uint32_t zero) { return zero * 0x10001u | 0x64006400u; }

__device__ __forceinline__ uint32_t pair_of(uint32_t w, int i) {
    return ((w >> (4 * i)) & 0x000f000fu) | 0x64006400u;
}
__device__ __forceinline__ quad values8(TF16, uint32_t w, uint32_t offset) {
    quad v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, pair_of(w, i)) - __builtin_bit_cast(f16x2, offset));
    return v;
}
__device__ __forceinline__ quad values8(TBF16, uint32_t w, uint32_t offset) {
    const float zero = gemvdev::lo_f16(offset);
    quad v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = pair_of(w, i);
        const uint32_t a = __builtin_bit_cast(uint32_t, gemvdev::lo_f16(p) - zero);
        const uint32_t b = __builtin_bit_cast(uint32_t, gemvdev::hi_f16(p) - zero);
        v[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);  // their upper halves: whole numbers of 8 bits
    }
    return v;
}

// A lane's 16 bytes of a row are columns 32·g .. 32·g+31 of the chunk (g =
// lane / 16); the matrix cores want columns 32·j + 8·g .. +7 at step j, so the
// four words are transposed among the four groups of lanes.
__device__ __forceinline__ quad transposed(quad w) {
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return quad{c[0], c[1], d[0], d[1]};
}

// ---------------------------------------------------------------------------
// vectors
// ---------------------------------------------------------------------------

template <class T>
struct Vec8 {  // eight columns of a vector, as the matrix cores take them
    quad part[Operand<T>::parts];
};

// Pairs (0,4), (1,5), (2,6), (3,7) of eight 16-bit values in order.
__device__ __forceinline__ quad in_order(quad v) {
    return quad{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
}
template <class T>
__device__ __forceinline__ Vec8<T> operand_of(T, quad v) {
    return Vec8<T>{{in_order(v)}};
}
// An fp32 value is the sum of its first 8 bits, the next 8 and the last 8: cut
// off, not rounded, so each part is exact and none overflows.  An infinity or
// NaN is its first part alone.
__device__ __forceinline__ Vec8<TF32> operand_of(TF32, quad lo, quad hi) {
    uint32_t p[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t bits = i < 4 ? lo[i] : hi[i - 4];
        const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
        // (a NaN may have all its bits in the lower half)
        const uint32_t first = finite ? bits : bits | ((bits & 0xffffu) ? 0x10000u : 0u);
        const float rest = finite ? gemvdev::f32_of(bits) - gemvdev::f32_of(bits & 0xffff0000u) : 0.0f;
        const uint32_t second = __builtin_bit_cast(uint32_t, rest);
        const float last = rest - gemvdev::f32_of(second & 0xffff0000u);
        p[0][i] = first;
        p[1][i] = second;
        p[2][i] = __builtin_bit_cast(uint32_t, last);
    }
    Vec8<TF32> v;
#pragma unroll
    for (int n = 0; n < 3; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) v.part[n][i] = __builtin_amdgcn_perm(p[n][i + 4], p[n][i], 0x07060302u);
    return v;
}

// What a lane loads of a vector for one matrix-core step: columns k .. k+7;
// those from K on read as zero and are not touched.
template <class T>
struct Raw8 {
    quad v[T::bytes / 2];
};
template <class T>
__device__ __forceinline__ Raw8<T> load_vec(const typename T::storage* x, int64_t k, bool whole, int K) {
    Raw8<T> r;
    if (whole) {
#pragma unroll
        for (int i = 0; i < T::bytes / 2; ++i)
            r.v[i] = *reinterpret_cast<const quad_any*>(x + k + i * (16 / T::bytes));
        return r;
    }
#pragma unroll
    for (int i = 0; i < T::bytes / 2; ++i) {
        r.v[i] = quad{0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 16 / T::bytes; ++e) {
            const int64_t at = k + i * (16 / T::bytes) + e;
            if (at >= K) continue;
            if constexpr (T::bytes == 4)
                r.v[i][e] = __builtin_bit_cast(uint32_t, x[at]);
            else
                r.v[i][e >> 1] |= (uint32_t)x[at] << (16 * (e & 1));
        }
    }
    return r;
}
template <class T>
__device__ __forceinline__ Vec8<T> operand_of(const Raw8<T>& r) {
    if constexpr (T::bytes == 4)
        return operand_of(T{}, r.v[0], r.v[1]);
    else
        return operand_of(T{}, r.v[0]);
}

// Scale and zero of the four steps of a chunk (their group's, so two or four
// of them may be alike); of steps behind the row's last column, 0.
struct Scales {
    float scale[4];
    uint32_t offset[4];
};
template <class T>
__device__ __forceinline__ Scales load_scales(const Product& p, int m, int chunk) {
    const typename T::storage* s = static_cast<const typename T::storage*>(p.scale) + m * p.lds;
    const uint8_t* z = p.zero ? p.zero + m * p.ldz : nullptr;
    Scales out;
    const int blocks = (p.K + kBlock - 1) / kBlock;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int block = 4 * chunk + j, g = block >> p.group_log2;
        const bool there = block < blocks;
        out.scale[j] = there ? widen(T{}, s[g]) : 0.0f;
        out.offset[j] = offset_of(z && there ? z[g] : kNoZero);
    }
    return out;
}

template <class O>
__device__ __forceinline__ void put(const Product& p, int64_t at, float v) {
    static_cast<typename O::storage*>(p.Y)[at] = fp8dev::narrow(O{}, v);
}
__device__ __forceinline__ void store(const Product& p, int t, int m, float v) {
    const int64_t at = t * p.ldy + m;
    if (p.y_type == 0)
        put<TF32>(p, at, v);
    else if (p.y_type == 1)
        put<TF16>(p, at, v);
    else
        put<TBF16>(p, at, v);
}

// Few vectors: a workgroup takes 16·RT rows by 16·NT vectors; its W wavefronts
// take the chunks of 128 columns in turn and add their sums in LDS, in a fixed
// order.  A lane has row (and vector) lane % 16.
template <class T, int RT, int NT, int W>
__global__ __launch_bounds__(W * 64) void q4_few_kernel(Product p) {
    using MT = typename Operand<T>::type;
    __shared__ f32x4 part[W][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    const int row0 = (int)blockIdx.x * 16 * RT, t0 = (int)blockIdx.y * 16 * NT;
    const int chunks = p.K / kChunk + (p.K % kChunk != 0);
    const int row_bytes = p.K / 2 + (p.K & 1);
    // rows and vectors past the end repeat the last one; their results are not stored
    int m[RT];
    const typename T::storage* x[NT];
#pragma unroll
    for (int i = 0; i < RT; ++i) m[i] = row0 + 16 * i + r < p.M ? row0 + 16 * i + r : p.M - 1;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = t0 + 16 * n + r;
        x[n] = static_cast<const typename T::storage*>(p.X) + (t < p.T ? t : p.T - 1) * p.ldx;
    }
    f32x4 acc[RT][NT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[i][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = wave; c < chunks; c += W) {
        const int64_t k = (int64_t)c * kChunk;
        const bool whole = p.K - k >= kChunk;
        quad w[RT];
        Scales s[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const uint8_t* at = p.Q + m[i] * p.ldq;
            w[i] = whole ? *reinterpret_cast<const quad_any*>(at + k / 2 + 16 * g)
                         : fp8dev::load_end(at, k / 2 + 16 * g, row_bytes);
            s[i] = load_scales<T>(p, m[i], c);
        }
        Raw8<T> raw[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) raw[n][j] = load_vec<T>(x[n], k + 32 * j + 8 * g, whole, p.K);
#pragma unroll
        for (int i = 0; i < RT; ++i) w[i] = transposed(w[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Vec8<T> v[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) v[n] = operand_of(raw[n][j]);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const quad b = values8(MT{}, w[i][j], s[i].offset[j]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    f32x4 d{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int e = 0; e < Operand<T>::parts; ++e) d = gemvdev::mma_16x16x32(MT{}, v[n].part[e], b, d);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][n][e] = __builtin_fmaf(d[e], s[i].scale[j], acc[i][n][e]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (i + n > 0) __syncthreads();
            part[wave][lane] = acc[i][n];
            __syncthreads();
            // of the tile's 256 sums a thread takes one: vector e / 16, row e % 16
            for (int e = threadIdx.x; e < 256; e += W * 64) {
                const int tt = e >> 4, rr = e & 15;
                const int t = t0 + 16 * n + tt, row = row0 + 16 * i + rr;
                if (t >= p.T || row >= p.M) continue;
                float v = part[0][(tt >> 2) * 16 + rr][tt & 3];
#pragma unroll
                for (int q = 1; q < W; ++q) v += part[q][(tt >> 2) * 16 + rr][tt & 3];
                if (p.bias) v += p.bias[row];
                store(p, t, row, v);
            }
        }
}

}  // namespace q4dev
