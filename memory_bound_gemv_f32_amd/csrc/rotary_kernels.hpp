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
constexpr int kWaves = 4;  // rows of a workgroup

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
    int parts, steps;     // steps: of all parts, each of one part's heads
    int dim, pairs;       // pairs: F
    bool interleaved;
    const float* frequency;
    float magnitude, eps;
    kvdev::Batch batch;
    int each;             // steps of a wavefront
};

// The place of a position's angle in its turn, in half turns, in [-1, 1]: as an fp32
// number, and in radians what that leaves out.  Whole turns of the frequency change nothing, as
// positions are whole numbers, so they are taken out before the product with the position.
// 1/π is a sum of three 64-bit numbers and every product keeps what it rounds off, so the
// place has more than fp32's bits at every position, of frequencies up to 2^70.
struct Place {
    float at, rest;
};
// (Products that are taken apart below must be rounded, not passed on unrounded into a
// multiply-add.)
__device__ __forceinline__ double less_turns(double v) {
#pragma clang fp contract(off)
    return v - 2.0 * __builtin_rint(0.5 * v);
}
// a + b rounded, and what that rounds off.
__device__ __forceinline__ double sum_of(double a, double b, double& off) {
#pragma clang fp contract(off)
    const double s = a + b, t = s - a;
    off = (a - (s - t)) + (b - t);
    return s;
}
__device__ __forceinline__ Place place_of(int position, float frequency) {
#pragma clang fp contract(off)
    constexpr double kInvPi = 0.31830988618379067, kSecond = -1.9678676675182486e-17, kThird = -1.0721436282893004e-33;
    const double f = frequency, n = position;
    const double first = f * kInvPi, second = f * kSecond;
    double off1, off2;
    double by = sum_of(less_turns(first), less_turns(__builtin_fma(f, kInvPi, -first)), off1);
    by = sum_of(by, less_turns(second), off2);
    const double by_rest = off1 + off2 + (__builtin_fma(f, kSecond, -second) + f * kThird);
    const double a = n * by, a_rest = __builtin_fma(n, by, -a) + n * by_rest;
    const double place = less_turns(less_turns(a) + a_rest);
    const float at = (float)place;
    return Place{at, (float)(place - at) * 3.14159265f};
}

// N values of a type: as loaded, widened, and stored.
template <class D, int N>
struct __attribute__((packed, aligned(D::bytes))) Run {
    typename D::storage v[N];
};
template <class D, int N>
__device__ __forceinline__ Run<D, N> load_run(const void* base, int64_t at) {
    return *reinterpret_cast<const Run<D, N>*>(static_cast<const typename D::storage*>(base) + at);
}
template <class D, int N>
__device__ __forceinline__ void store_as(void* base, int64_t at, const float (&v)[N]) {
    Run<D, N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = fp8dev::narrow(D{}, v[i]);
    *reinterpret_cast<Run<D, N>*>(static_cast<typename D::storage*>(base) + at) = r;
}
template <int N>
__device__ __forceinline__ void store_run(int type, void* base, int64_t at, const float (&v)[N]) {
    if (type == 0)
        store_as<TF32>(base, at, v);
    else if (type == 1)
        store_as<TF16>(base, at, v);
    else
        store_as<TBF16>(base, at, v);
}

// The first and second values of V pairs that lie in two runs: as they are, or one pair
// behind the other.
template <class D, int V>
__device__ __forceinline__ void pairs_of(const Run<D, V>& lo, const Run<D, V>& hi, bool together, float (&u)[V],
                                         float (&v)[V]) {
    float x[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x[i] = widen(D{}, lo.v[i]);
        x[V + i] = widen(D{}, hi.v[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        u[i] = together ? x[2 * i] : x[i];
        v[i] = together ? x[2 * i + 1] : x[V + i];
    }
}

// A wavefront takes a row, 64 / L heads of one part at a time; L lanes share a
// head, each V of its pairs at N places.  A pair is also taken where nothing is
// rotated: pairs from F on are the values 2s and 2s + 1.  A lane works out the
// angles of every 64th pair, and LDS hands their sines and cosines to the lanes
// that want them, for all of the row's heads; the next heads' values are loaded
// meanwhile.
template <class D, int V, int L, int N>
__global__ __launch_bounds__(kWaves * 64) void rotary_kernel(Rotary p) {
    constexpr int kHeads = 64 / L;
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    __shared__ f32x2 turns[kWaves][kMostDim / 2];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, in = lane % L;
    const int row = (int)blockIdx.x * kWaves + wave;
    if (row >= p.batch.total) return;
    if (p.batch.starts != nullptr && row >= kvdev::start_of(p.batch, p.batch.count)) return;  // padding, which is not read
    const int half = p.dim / 2;
    int slot[N];
#pragma unroll
    for (int n = 0; n < N; ++n) slot[n] = (in + L * n) * V;
    // a lane's values at its places: pairs' first values, then their second ones, or
    // the pairs one behind the other
    struct Raw {
        Run<D, V> lo[N], hi[N];
    };
    const int from = (int)blockIdx.y * p.each;
    const int until = from + p.each < p.steps ? from + p.each : p.steps;
    // the part and the first head of a step
    const auto place = [&](int step, int& at, int& head) {
        at = 0;
        head = step;
        while (at + 1 < p.parts) {
            const int steps = (p.part[at].heads + kHeads - 1) / kHeads;
            if (head < steps) break;
            head -= steps;
            ++at;
        }
        head = head * kHeads + lane / L;
    };
    const auto load = [&](int step, Raw& to) {
        int at, head;
        place(step, at, head);
        const Part& part = p.part[at];
        head = head < part.heads ? head : part.heads - 1;  // (spare lanes repeat the last, and store nothing)
        const int64_t base = row * part.ldx + (int64_t)head * p.dim;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int at_slot = slot[n] < half ? slot[n] : half - V;  // (likewise)
            const bool together = p.interleaved || at_slot >= p.pairs;
            to.lo[n] = load_run<D, V>(part.x, base + (together ? 2 * at_slot : at_slot));
            to.hi[n] = load_run<D, V>(part.x, base + (together ? 2 * at_slot + V : at_slot + p.pairs));
        }
    };
    Raw raw;
    load(from, raw);
    int b;
    if (p.batch.starts == nullptr)
        b = row;
    else
        b = kvdev::sequence_of(p.batch, row, 1, 1, 0);
    const int start = kvdev::start_of(p.batch, b), stop = kvdev::start_of(p.batch, b + 1);
    if (row < start || row >= stop) return;
    const int position = p.batch.lens[b] - (stop - row);
    for (int i = lane; i < p.pairs; i += 64) {
        const Place place = place_of(position, p.frequency[i]);
        float s, c;
        sincospif(place.at, &s, &c);
        // (turned on by the little that is left: its square is below fp32's bits)
        const float cosine = __builtin_fmaf(-s, place.rest, c), sine = __builtin_fmaf(c, place.rest, s);
        turns[wave][i] = f32x2{cosine * p.magnitude, sine * p.magnitude};
    }
    // (a wavefront's own: its LDS accesses are in order)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float c[N][V], s[N][V];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool turned = slot[n] + i < p.pairs;
            const f32x2 t = turns[wave][turned ? slot[n] + i : 0];  // (else unused)
            c[n][i] = t[0];
            s[n][i] = t[1];
        }
    // a part's weights stay in registers while its heads last
    float wu[N][V], wv[N][V];
    int weighted = -1;
    for (int step = from; step < until; ++step) {
        int at, head;
        place(step, at, head);
        const Part& part = p.part[at];
        if (part.weight && weighted != at) {
            weighted = at;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int at_slot = slot[n] < half ? slot[n] : half - V;
                const bool together = p.interleaved || at_slot >= p.pairs;
                const Run<TF32, V> lo = load_run<TF32, V>(part.weight, together ? 2 * at_slot : at_slot);
                const Run<TF32, V> hi = load_run<TF32, V>(part.weight, together ? 2 * at_slot + V : at_slot + p.pairs);
                pairs_of<TF32>(lo, hi, together, wu[n], wv[n]);
            }
        }
        float u[N][V], v[N][V];
        float squares = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const bool together = p.interleaved || slot[n] >= p.pairs;
            pairs_of<D>(raw.lo[n], raw.hi[n], together, u[n], v[n]);
            if (slot[n] < half)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    squares = __builtin_fmaf(u[n][i], u[n][i], __builtin_fmaf(v[n][i], v[n][i], squares));
        }
        if (step + 1 < until) load(step + 1, raw);
        if (part.weight) {
            squares = gemvdev::segment_sum<L>(squares);
            const float by = 1.0f / sqrtf(squares / (float)p.dim + p.eps);
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    u[n][i] *= by * wu[n][i];
                    v[n][i] *= by * wv[n][i];
                }
        }
        if (head >= part.heads) continue;
        const int64_t base = row * part.ldy + (int64_t)head * p.dim;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (slot[n] >= half) continue;
            float lo[V], hi[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // (a pair that is not turned is kept, not multiplied by 1 and 0: an infinity
                // or NaN would reach its neighbour)
                const bool turned = slot[n] + i < p.pairs;
                const float a = __builtin_fmaf(u[n][i], c[n][i], -(v[n][i] * s[n][i]));
                const float b = __builtin_fmaf(v[n][i], c[n][i], u[n][i] * s[n][i]);
                lo[i] = turned ? a : u[n][i];
                hi[i] = turned ? b : v[n][i];
            }
            if (p.interleaved || slot[n] >= p.pairs) {
                float y[2 * V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    y[2 * i] = lo[i];
                    y[2 * i + 1] = hi[i];
                }
                store_run(part.y_type, part.y, base + 2 * slot[n], y);
            } else {
                store_run(part.y_type, part.y, base + slot[n], lo);
                store_run(part.y_type, part.y, base + slot[n] + p.pairs, hi);
            }
        }
    }
}

}  // namespace rotarydev
