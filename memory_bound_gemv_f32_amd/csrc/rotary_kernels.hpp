// Kernel of the norms and rotary positions of query and key heads.
//
//   n = x·(mean(x²) + eps)^(-1/2)·weight        (n = x without a weight)
//   (a, b) -> (a·cos - b·sin, b·cos + a·sin)·magnitude,  angle = position·frequency[i]
//
// for the pairs (a, b) = (n[i], n[i + F]) or (n[2i], n[2i + 1]), i < F, of a
// head's first 2·F values; the others are n.  fp32 throughout, rounded once.
#pragma once

#include "kv_kernels.hpp"

namespace rotarydev {

using fp8dev::quad;
using fp8dev::quad_any;
using fp8dev::TBF16;
using fp8dev::TF16;
using fp8dev::TF32;
using fp8dev::widen;

constexpr int kMostParts = 4, kMostDim = 512;

struct Part {
    const void* x;
    int64_t ldx;
    void* y;
    int64_t ldy;
    const float* weight;  // or NULL
    int heads;
    int y_type;           // gemv_dtype_t
};
struct Rotary {
    Part part[kMostParts];
    int parts, heads;     // heads of all parts
    int dim, pairs;       // pairs: F
    bool interleaved;
    const float* frequency;
    float magnitude, eps;
    kvdev::Batch batch;
    int steps;            // head groups that a wavefront takes
};

// The angle of a position in half turns, in [-1, 1].  frequency/π and its
// product with the position are each held as a sum of two 64-bit numbers (whole
// turns may take 30 of a number's 53 bits), so at every position what is lost is the rounding
// to fp32 at the end.
__device__ __forceinline__ float half_turns(int position, float frequency) {
    constexpr double kInvPi = 0.31830988618379067, kInvPiRest = -1.9678676675182486e-17;  // 1/π
    const double f = frequency, n = position;
    const double by = f * kInvPi, by_rest = __builtin_fma(f, kInvPi, -by) + f * kInvPiRest;
    const double a = n * by, a_rest = __builtin_fma(n, by, -a) + n * by_rest;
    return (float)(a - 2.0 * __builtin_rint(0.5 * a) + a_rest);
}

template <class D, int N>
__device__ __forceinline__ void load_run(const void* base, int64_t at, float (&v)[N]) {
    kvdev::load_run<D, N>(static_cast<const typename D::storage*>(base) + at, v);
}
template <class D, int N>
__device__ __forceinline__ void store_run(void* base, int64_t at, const float (&v)[N]) {
    using S = typename D::storage;
    struct __attribute__((packed, aligned(D::bytes))) Run {
        S v[N];
    } r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = fp8dev::narrow(D{}, v[i]);
    *reinterpret_cast<Run*>(static_cast<S*>(base) + at) = r;
}
template <int N>
__device__ __forceinline__ void store_run(int type, void* base, int64_t at, const float (&v)[N]) {
    if (type == 0)
        store_run<TF32>(base, at, v);
    else if (type == 1)
        store_run<TF16>(base, at, v);
    else
        store_run<TBF16>(base, at, v);
}

// A wavefront takes one row; L lanes share a head, each V of its pairs at N
// places, so 64 / L heads at a time.  A pair is also taken where nothing is
// rotated: pairs from F on are the values 2s and 2s + 1.  The sines and cosines
// are worked out once and serve all of a wavefront's heads.
template <class D, int V, int L, int N>
__global__ __launch_bounds__(64) void rotary_kernel(Rotary p) {
    constexpr int kHeads = 64 / L;
    const int lane = threadIdx.x, in = lane % L;
    const int row = (int)blockIdx.x;
    int b;
    if (p.batch.starts == nullptr)
        b = row;
    else
        b = kvdev::sequence_of(p.batch, row, 1, 1, 0);
    const int start = kvdev::start_of(p.batch, b), stop = kvdev::start_of(p.batch, b + 1);
    if (row < start || row >= stop) return;  // padding
    const int position = p.batch.lens[b] - (stop - row);
    const int half = p.dim / 2;
    int slot[N];
    float c[N][V], s[N][V];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        slot[n] = (in + L * n) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[n][i] = 1.0f;
            s[n][i] = 0.0f;
            if (slot[n] + i < p.pairs) {
                sincospif(half_turns(position, p.frequency[slot[n] + i]), &s[n][i], &c[n][i]);
                c[n][i] *= p.magnitude;
                s[n][i] *= p.magnitude;
            }
        }
    }
    for (int step = 0; step < p.steps; ++step) {
        const int head = ((int)blockIdx.y * p.steps + step) * kHeads + lane / L;
        const bool there = head < p.heads;
        // the part that the head is of (a lane without one takes the first, and stores nothing)
        int at = 0, h = there ? head : 0;
        while (at + 1 < p.parts && h >= p.part[at].heads) h -= p.part[at++].heads;
        const Part& part = p.part[at];
        const int64_t from = row * part.ldx + (int64_t)h * p.dim, to = row * part.ldy + (int64_t)h * p.dim;
        float x[N][2 * V];
        float squares = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) x[n][i] = 0.0f;
            if (slot[n] >= half) continue;
            if (p.interleaved || slot[n] >= p.pairs) {
                load_run<D, 2 * V>(part.x, from + 2 * slot[n], x[n]);
            } else {
                float lo[V], hi[V];
                load_run<D, V>(part.x, from + slot[n], lo);
                load_run<D, V>(part.x, from + slot[n] + p.pairs, hi);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    x[n][2 * i] = lo[i];
                    x[n][2 * i + 1] = hi[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) squares = __builtin_fmaf(x[n][i], x[n][i], squares);
        }
        squares = gemvdev::segment_sum<L>(squares);
        if (!there) continue;
        const float by = part.weight ? 1.0f / sqrtf(squares / (float)p.dim + p.eps) : 1.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (slot[n] >= half) continue;
            const bool together = p.interleaved || slot[n] >= p.pairs;
            float y[2 * V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float u = x[n][2 * i], v = x[n][2 * i + 1];
                if (part.weight) {
                    const int j = slot[n] + i;
                    u *= by * part.weight[together ? 2 * j : j];
                    v *= by * part.weight[together ? 2 * j + 1 : j + p.pairs];
                }
                y[2 * i] = __builtin_fmaf(u, c[n][i], -(v * s[n][i]));
                y[2 * i + 1] = __builtin_fmaf(v, c[n][i], u * s[n][i]);
            }
            if (together) {
                store_run<2 * V>(part.y_type, part.y, to + 2 * slot[n], y);
            } else {
                float lo[V], hi[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    lo[i] = y[2 * i];
                    hi[i] = y[2 * i + 1];
                }
                store_run<V>(part.y_type, part.y, to + slot[n], lo);
                store_run<V>(part.y_type, part.y, to + slot[n] + p.pairs, hi);
            }
        }
    }
}

}  // namespace rotarydev
