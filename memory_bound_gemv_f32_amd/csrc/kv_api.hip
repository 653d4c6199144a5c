// libgemv C ABI, the paged 8-bit key/value cache: argument checks, mapping
// selection and launch.
#include <hip/hip_runtime.h>

#include "../../include/gemv.h"
#include "gemv_launch.hpp"
#include "kv_kernels.hpp"

namespace {

using gemvapi::finish;
using kvdev::Attend;
using kvdev::E4m3;
using kvdev::Int8;
using kvdev::TBF16;
using kvdev::TF16;
using kvdev::TF32;
using kvplan::capacity_of;
using kvplan::map_attend;
using kvplan::map_call;
using kvplan::Mapping;
using kvplan::SharedMapping;
using kvplan::workspace_of;

static_assert(GEMV_KV_BLOCK == kvdev::kBlock, "the header states the block");

bool aligned(const void* p, int n) { return (uintptr_t)p % n == 0; }

gemv_status_t launch(const void* fn, dim3 grid, int threads, void** argv, hipStream_t stream) {
    if ((uint64_t)grid.x * threads > 0xffffffffu) return GEMV_ERROR_INVALID_VALUE;  // more than a launch holds
    return finish(hipLaunchKernel(fn, grid, dim3((unsigned)threads), argv, 0, stream));
}

// The head dims and page sizes that there are kernels for.
bool known_dim(int dim) { return dim == 64 || dim == 128 || dim == 256; }

bool known_page(int page_size) {
    return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128 || page_size == 256;
}
constexpr int kMostHeads = 65535;

bool make_cache(const gemv_kv_cache_t* in, kvdev::Cache* out) {
    if (in == nullptr || (in->format != GEMV_KV_INT8 && in->format != GEMV_KV_E4M3) ||
        in->pages < 1 || in->heads < 1 || in->heads > kMostHeads || !known_dim(in->dim) ||
        !known_page(in->page_size))
        return false;
    int log2 = 0;
    while ((GEMV_KV_BLOCK << log2) != in->page_size) ++log2;
    if (in->k == nullptr || in->v == nullptr || in->k_scale == nullptr || in->v_scale == nullptr ||
        !aligned(in->k, 16) || !aligned(in->v, 16) || !aligned(in->k_scale, 4) || !aligned(in->v_scale, 4))
        return false;
    *out = kvdev::Cache{static_cast<uint8_t*>(in->k), static_cast<uint8_t*>(in->v), in->k_scale,
                        in->v_scale, in->heads, in->pages, log2};
    return true;
}

bool make_batch(const gemv_kv_batch_t* in, int rows, kvdev::Batch* out) {
    if (in == nullptr || in->sequences < 0 || in->table_width < 0 || in->table_pitch < in->table_width ||
        rows < 0 || (in->starts == nullptr && rows != in->sequences))
        return false;
    if (in->sequences > 0 && rows > 0 &&
        (in->seq_lens == nullptr || (in->table == nullptr && in->table_width > 0) ||
         !aligned(in->table, 4) || !aligned(in->seq_lens, 4) || !aligned(in->starts, 4)))
        return false;
    *out = kvdev::Batch{in->table, in->table_pitch, in->table_width, in->seq_lens, in->starts,
                        in->sequences, rows};
    return true;
}

template <class D, class F>
gemv_status_t append(int dim, const kvdev::Cache& c, const kvdev::Batch& q, const void* K, int64_t ldk,
                     const void* V, int64_t ldv, hipStream_t stream) {
    // a token each is one block each
    const int64_t places = q.starts == nullptr ? q.count : q.total / GEMV_KV_BLOCK + 2 * (int64_t)q.count;
    if (places > 0x7fffffff) return GEMV_ERROR_INVALID_VALUE;
    void* argv[] = {(void*)&c, (void*)&q, (void*)&K, (void*)&ldk, (void*)&V, (void*)&ldv};
    const void* fn = dim == 64    ? (const void*)&kvdev::kv_append_kernel<D, F, 64>
                     : dim == 128 ? (const void*)&kvdev::kv_append_kernel<D, F, 128>
                                  : (const void*)&kvdev::kv_append_kernel<D, F, 256>;
    return launch(fn, dim3((unsigned)places, (unsigned)c.heads, 2), 64, argv, stream);
}

// Joins p's splits; with s, also those over the shared tokens.
template <class T, int DIM, bool SHARED>
gemv_status_t join(const Mapping& m, Attend& p, Attend& s, int64_t shared_places, hipStream_t stream) {
    int64_t places = m.places;
    void* argv[] = {&p, &places, &s, &shared_places};
    constexpr int kTwo = DIM <= 128 ? 2 : 1;
    const void* fn;
    int rows = m.place_rows;
    if constexpr (SHARED) {
        if (p.splits + s.splits <= kvdev::kFewSplits) {
            fn = m.waves_share == 1
                     ? (const void*)&kvdev::kv_join_rows_kernel<T, DIM, 16 * kvdev::kOwnWaves * kTwo, 16 * kTwo>
                 : m.row_tiles == 2 ? (const void*)&kvdev::kv_join_rows_kernel<T, DIM, 16 * kTwo, 16 * kTwo>
                                    : (const void*)&kvdev::kv_join_rows_kernel<T, DIM, 16, 16>;
            constexpr int kEach = kvdev::kShareWaves * kvdev::kJoinRows;  // rows of a workgroup
            rows = (rows + kEach - 1) / kEach;
            return launch(fn, dim3((unsigned)(places * p.cache.heads), (unsigned)rows), kvdev::kShareWaves * 64, argv,
                          stream);
        }
    }
    fn = m.waves_share == 1
             ? (const void*)&kvdev::kv_join_kernel<T, DIM, 16 * kvdev::kOwnWaves * kTwo, 16 * kTwo, SHARED>
         : m.row_tiles == 2 ? (const void*)&kvdev::kv_join_kernel<T, DIM, 16 * kTwo, 16 * kTwo, SHARED>
                            : (const void*)&kvdev::kv_join_kernel<T, DIM, 16, 16, SHARED>;
    return launch(fn, dim3((unsigned)(places * p.cache.heads), (unsigned)rows), kvdev::kShareWaves * 64, argv, stream);
}

template <class T, class F, int DIM>
gemv_status_t walk(const Mapping& m, Attend& p, hipStream_t stream) {
    int64_t places = m.places;
    const int64_t grid = places * p.cache.heads * p.splits;
    void* argv[] = {&p, &places};
    constexpr int kTwo = DIM <= 128 ? 2 : 1;
    constexpr int kSmall = DIM <= 128 ? DIM : 128;  // (dim 256 has no eight, see cut)
    const void* fn = m.waves_share == 1 ? (const void*)&kvdev::kv_attend_kernel<T, F, DIM, kTwo, 1>
                     : m.row_tiles == 2 ? (const void*)&kvdev::kv_attend_kernel<T, F, DIM, kTwo, 4>
                     : m.waves_share == 8 ? (const void*)&kvdev::kv_attend_kernel<T, F, kSmall, 1, 8>
                                          : (const void*)&kvdev::kv_attend_kernel<T, F, DIM, 1, 4>;
    return launch(fn, dim3((unsigned)grid), 64 * kvplan::waves_of(m), argv, stream);
}

// The shared tokens, and each sequence's own in the same launch where their row
// tiles are of 16 (with two of 32 the workgroup would take a compute unit's LDS alone).
template <class T, class F, int DIM>
gemv_status_t walk_shared(const SharedMapping& m, Attend& s, Attend& p, hipStream_t stream) {
    constexpr int kTwo = DIM <= 128 ? 2 : 1;
    const bool together = kvplan::together(m);
    int64_t shared_places = m.shared.places, own_places = together ? m.own.places : 0;
    const int64_t grid = shared_places * s.cache.heads * s.splits + own_places * p.cache.heads * p.splits;
    void* argv[] = {&s, &shared_places, &p, &own_places};
    const void* fn = m.shared.row_tiles == 2 ? (const void*)&kvdev::kv_attend_shared_kernel<T, F, DIM, kTwo>
                                             : (const void*)&kvdev::kv_attend_shared_kernel<T, F, DIM, 1>;
    const gemv_status_t st = launch(fn, dim3((unsigned)grid), 64 * kvdev::kShareWaves, argv, stream);
    return st != GEMV_SUCCESS || together ? st : walk<T, F, DIM>(m.own, p, stream);
}

template <class T, class F, int DIM>
gemv_status_t attend(const SharedMapping& m, Attend& p, hipStream_t stream) {
    Attend s = p;
    if (m.chunks > 0) {
        s.splits = m.shared.splits;
        s.split_chunks = m.shared.split_chunks;
        s.rows = m.shared.place_rows;
        s.capacity = m.chunks * kvplan::kChunk;
        s.shared = 0;
        s.slack = m.own.waves_share == 1 ? kvdev::kPromptSlack : 0.0f;
        s.partial = p.partial + kvplan::partials_of(m.own, p.cache.heads, DIM) / sizeof(float);
        const gemv_status_t st = walk_shared<T, F, DIM>(m, s, p, stream);
        return st != GEMV_SUCCESS ? st : join<T, DIM, true>(m.own, p, s, m.shared.places, stream);
    }
    const gemv_status_t st = walk<T, F, DIM>(m.own, p, stream);
    return st != GEMV_SUCCESS || p.splits == 1 ? st : join<T, DIM, false>(m.own, p, s, 0, stream);
}

template <class T, class F>
gemv_status_t attend_dim(int dim, const SharedMapping& m, Attend& p, hipStream_t stream) {
    switch (dim) {
    case 64: return attend<T, F, 64>(m, p, stream);
    case 128: return attend<T, F, 128>(m, p, stream);
    default: return attend<T, F, 256>(m, p, stream);
    }
}

template <class D>
gemv_status_t append(const gemv_kv_cache_t* cache, const void* K, int ldk, const void* V, int ldv,
                     int rows, const gemv_kv_batch_t* batch, hipStream_t stream) {
    kvdev::Cache c;
    kvdev::Batch q;
    if (!make_cache(cache, &c) || !make_batch(batch, rows, &q) ||
        (int64_t)ldk < (int64_t)c.heads * cache->dim || (int64_t)ldv < (int64_t)c.heads * cache->dim)
        return GEMV_ERROR_INVALID_VALUE;
    if (rows == 0 || q.count == 0) return GEMV_SUCCESS;
    if (K == nullptr || V == nullptr || !aligned(K, D::bytes) || !aligned(V, D::bytes))
        return GEMV_ERROR_INVALID_VALUE;
    return cache->format == GEMV_KV_E4M3 ? append<D, E4m3>(cache->dim, c, q, K, ldk, V, ldv, stream)
                                         : append<D, Int8>(cache->dim, c, q, K, ldk, V, ldv, stream);
}

template <class T>
gemv_status_t attend(const gemv_kv_cache_t* cache, const uint16_t* Q, int ldq, uint16_t* O, int ldo,
                     int q_heads, int rows, const gemv_kv_batch_t* batch, float scale, int window,
                     int sinks, int shared, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    Attend p;
    if (!make_cache(cache, &p.cache) ||
        !make_batch(batch, rows, &p.batch) || q_heads < 1 || q_heads % p.cache.heads != 0 ||
        (int64_t)ldq < (int64_t)q_heads * cache->dim || (int64_t)ldo < (int64_t)q_heads * cache->dim ||
        (int64_t)rows * q_heads > 0x7fffffff || window < 0 || sinks < 0 || shared < 0 || !(scale - scale == 0.0f))
        return GEMV_ERROR_INVALID_VALUE;
    if (rows == 0 || p.batch.count == 0) return GEMV_SUCCESS;
    if (Q == nullptr || O == nullptr || !aligned(Q, 2) || !aligned(O, 2)) return GEMV_ERROR_INVALID_VALUE;
    const int64_t capacity = capacity_of(batch->table_width, cache->page_size);
    const SharedMapping m = map_call(q_heads, p.cache.heads, cache->dim, rows, p.batch.count,
                                     batch->starts == nullptr, capacity, window, sinks, shared);
    if (!kvplan::launchable(m, p.cache.heads)) return GEMV_ERROR_INVALID_VALUE;
    const size_t need = workspace_of(m, p.cache.heads, cache->dim);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
        return GEMV_ERROR_INVALID_VALUE;
    p.Q = Q;
    p.ldq = ldq;
    p.O = O;
    p.ldo = ldo;
    p.group = q_heads / p.cache.heads;
    p.scale = (scale < 0.0f ? -scale : scale) * 1.44269504088896341f;
    p.q_sign = scale < 0.0f ? 0x80008000u : 0u;
    p.window = window;
    p.sinks = sinks;
    p.capacity = (int)capacity;
    p.splits = m.own.splits;
    p.split_chunks = m.own.split_chunks;
    p.rows = m.own.place_rows;
    p.shared = m.chunks;
    p.slack = 0.0f;
    p.partial = static_cast<float*>(workspace);
    return cache->format == GEMV_KV_E4M3 ? attend_dim<T, E4m3>(cache->dim, m, p, stream)
                                         : attend_dim<T, Int8>(cache->dim, m, p, stream);
}

}  // namespace

extern "C" gemv_status_t gemv_kv_attend_shared_workspace_size(int q_heads, int heads, int dim, int rows,
                                                              int sequences, int one_each, int table_width,
                                                              int page_size, int window, int sinks, int shared,
                                                              size_t* bytes) {
    if (bytes == nullptr || heads < 1 || heads > kMostHeads || q_heads < 1 || q_heads % heads != 0 ||
        !known_dim(dim) || rows < 0 || sequences < 0 || (one_each && rows != sequences) || table_width < 0 ||
        !known_page(page_size) || (int64_t)rows * q_heads > 0x7fffffff || window < 0 || sinks < 0 || shared < 0)
        return GEMV_ERROR_INVALID_VALUE;
    size_t need = 0;
    if (rows > 0 && sequences > 0) {
        const SharedMapping m = map_call(q_heads, heads, dim, rows, sequences, one_each != 0,
                                         capacity_of(table_width, page_size), window, sinks, shared);
        if (!kvplan::launchable(m, heads)) return GEMV_ERROR_INVALID_VALUE;
        need = workspace_of(m, heads, dim);
    }
    *bytes = need;
    return GEMV_SUCCESS;
}

extern "C" gemv_status_t gemv_kv_attend_workspace_size(int q_heads, int heads, int dim, int rows,
                                                       int sequences, int one_each, int table_width,
                                                       int page_size, int window, int sinks, size_t* bytes) {
    return gemv_kv_attend_shared_workspace_size(q_heads, heads, dim, rows, sequences, one_each, table_width,
                                                page_size, window, sinks, 0, bytes);
}

#define GEMV_KV_APPEND(NAME, D, T)                                                             \
    extern "C" gemv_status_t gemv_kv_append_##NAME(const gemv_kv_cache_t* cache, const T* K,     \
                                                   int ldk, const T* V, int ldv, int rows,       \
                                                   const gemv_kv_batch_t* batch,                 \
                                                   hipStream_t stream) {                         \
        return append<D>(cache, K, ldk, V, ldv, rows, batch, stream);                            \
    }
GEMV_KV_APPEND(f32, TF32, float)
GEMV_KV_APPEND(f16, TF16, uint16_t)
GEMV_KV_APPEND(bf16, TBF16, uint16_t)

#define GEMV_KV_ATTEND(NAME, T)                                                                  \
    extern "C" gemv_status_t gemv_kv_attend_##NAME(                                              \
        const gemv_kv_cache_t* cache, const uint16_t* Q, int ldq, uint16_t* O, int ldo,          \
        int q_heads, int rows, const gemv_kv_batch_t* batch, float scale, int window, int sinks, \
        void* workspace, size_t workspace_bytes, hipStream_t stream) {                           \
        return attend<T>(cache, Q, ldq, O, ldo, q_heads, rows, batch, scale, window, sinks, 0,   \
                         workspace, workspace_bytes, stream);                                    \
    }                                                                                            \
    extern "C" gemv_status_t gemv_kv_attend_shared_##NAME(                                       \
        const gemv_kv_cache_t* cache, const uint16_t* Q, int ldq, uint16_t* O, int ldo,          \
        int q_heads, int rows, const gemv_kv_batch_t* batch, float scale, int window, int sinks, \
        int shared, void* workspace, size_t workspace_bytes, hipStream_t stream) {               \
        return attend<T>(cache, Q, ldq, O, ldo, q_heads, rows, batch, scale, window, sinks,      \
                         shared, workspace, workspace_bytes, stream);                            \
    }
GEMV_KV_ATTEND(f16, TF16)
GEMV_KV_ATTEND(bf16, TBF16)
