// libgemv C ABI, the norms and rotary positions of query and key heads:
// argument checks, mapping selection and launch.
#include <hip/hip_runtime.h>

#include "../../include/gemv.h"
#include "gemv_launch.hpp"
#include "rotary_kernels.hpp"

namespace {

using gemvapi::finish;
using rotarydev::Rotary;
using rotarydev::TBF16;
using rotarydev::TF16;
using rotarydev::TF32;

static_assert(GEMV_ROTARY_MAX_PARTS == rotarydev::kMostParts && GEMV_ROTARY_MAX_DIM == rotarydev::kMostDim,
              "the header states the limits");

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kMostRows = 1 << 25;  // of one launch

bool aligned(const void* p, int n) { return (uintptr_t)p % n == 0; }

// A kernel and the heads of one of its steps.
struct Kernel {
    const void* fn;
    int heads;
};

template <class D>
Kernel kernel_of(int dim, int pairs) {
    // as many pairs to a lane as one 16-byte load of each half holds, or four, where no
    // run of them straddles the rotated ones' end; else one
    if constexpr (D::bytes == 2)
        if (dim % 16 == 0 && pairs % 8 == 0) {
            const int lanes = dim / 16;
            if (lanes <= 4) return {(const void*)&rotarydev::rotary_kernel<D, 8, 4, 1>, 16};
            if (lanes <= 8) return {(const void*)&rotarydev::rotary_kernel<D, 8, 8, 1>, 8};
            if (lanes <= 16) return {(const void*)&rotarydev::rotary_kernel<D, 8, 16, 1>, 4};
            return {(const void*)&rotarydev::rotary_kernel<D, 8, 32, 1>, 2};
        }
    if (dim % 8 == 0 && pairs % 4 == 0) {
        const int lanes = dim / 8;
        if (lanes <= 8) return {(const void*)&rotarydev::rotary_kernel<D, 4, 8, 1>, 8};
        if (lanes <= 16) return {(const void*)&rotarydev::rotary_kernel<D, 4, 16, 1>, 4};
        if (lanes <= 32) return {(const void*)&rotarydev::rotary_kernel<D, 4, 32, 1>, 2};
        return {(const void*)&rotarydev::rotary_kernel<D, 4, 64, 1>, 1};
    }
    return {(const void*)&rotarydev::rotary_kernel<D, 1, 64, rotarydev::kMostDim / 128>, 1};
}

// Wavefronts that fill the GPU several times over: a row's heads go to as many
// wavefronts as there are fewer rows than that.
constexpr int64_t kEnoughWaves = 8192;

bool known(int dtype) { return dtype == GEMV_DTYPE_F32 || dtype == GEMV_DTYPE_F16 || dtype == GEMV_DTYPE_BF16; }

template <class D>
gemv_status_t rotary(const gemv_rotary_part_t* parts, int count, int dim, int rows, const float* frequency,
                     int pairs, int interleaved, float magnitude, float eps, const gemv_kv_batch_t* batch,
                     hipStream_t stream) {
    if (parts == nullptr || count < 1 || count > GEMV_ROTARY_MAX_PARTS || dim < 2 || dim % 2 != 0 ||
        dim > GEMV_ROTARY_MAX_DIM || rows < 0 || pairs < 0 || pairs > dim / 2 || (interleaved != 0 && interleaved != 1) ||
        !(magnitude - magnitude == 0.0f) || !(eps - eps == 0.0f) || eps < 0.0f || batch == nullptr ||
        batch->sequences < 0 || (batch->starts == nullptr && rows != batch->sequences))
        return GEMV_ERROR_INVALID_VALUE;
    const bool any = rows > 0 && batch->sequences > 0;
    if (any && ((pairs > 0 && frequency == nullptr) || !aligned(frequency, 4) || batch->seq_lens == nullptr ||
                !aligned(batch->seq_lens, 4) || !aligned(batch->starts, 4)))
        return GEMV_ERROR_INVALID_VALUE;
    Rotary p{};
    for (int i = 0; i < count; ++i) {
        const gemv_rotary_part_t& a = parts[i];
        if (a.heads < 0 || !known(a.y_dtype) || a.ldx < (int64_t)a.heads * dim || a.ldy < (int64_t)a.heads * dim)
            return GEMV_ERROR_INVALID_VALUE;
        if (a.heads == 0) continue;
        if (any && (a.x == nullptr || a.y == nullptr || !aligned(a.x, D::bytes) ||
                    !aligned(a.y, a.y_dtype == GEMV_DTYPE_F32 ? 4 : 2) || !aligned(a.weight, 4)))
            return GEMV_ERROR_INVALID_VALUE;
        p.part[p.parts++] = rotarydev::Part{a.x, a.ldx, a.y, a.ldy, a.weight, a.heads, a.y_dtype};
    }
    if (!any || p.parts == 0) return GEMV_SUCCESS;
    const Kernel k = kernel_of<D>(dim, pairs);
    int64_t steps = 0;
    for (int i = 0; i < p.parts; ++i) steps += ceil_div(p.part[i].heads, k.heads);
    if (steps > 0x7fffffff || rows > kMostRows) return GEMV_ERROR_INVALID_VALUE;
    int64_t across = ceil_div(kEnoughWaves, rows);
    across = across < steps ? across : steps;
    p.steps = (int)steps;
    p.each = (int)ceil_div(steps, across);
    p.dim = dim;
    p.pairs = pairs;
    p.interleaved = interleaved != 0;
    p.frequency = frequency;
    p.magnitude = magnitude;
    p.eps = eps;
    p.batch = kvdev::Batch{nullptr, 0, 0, batch->seq_lens, batch->starts, batch->sequences, rows};
    void* argv[] = {&p};
    const dim3 grid((unsigned)ceil_div(rows, rotarydev::kWaves), (unsigned)ceil_div(steps, p.each));
    return finish(hipLaunchKernel(k.fn, grid, dim3(rotarydev::kWaves * 64), argv, 0, stream));
}

}  // namespace

#define GEMV_ROTARY(NAME, D)                                                                     \
    extern "C" gemv_status_t gemv_rotary_##NAME(                                                 \
        const gemv_rotary_part_t* parts, int count, int dim, int rows, const float* frequency,   \
        int pairs, int interleaved, float magnitude, float eps, const gemv_kv_batch_t* batch,    \
        hipStream_t stream) {                                                                    \
        return rotary<D>(parts, count, dim, rows, frequency, pairs, interleaved, magnitude, eps, \
                         batch, stream);                                                         \
    }
GEMV_ROTARY(f32, TF32)
GEMV_ROTARY(f16, TF16)
GEMV_ROTARY(bf16, TBF16)
