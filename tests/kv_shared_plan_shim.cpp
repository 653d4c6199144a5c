// Host build of the mapping of the attention behind shared tokens for the CPU
// tests: the functions that the launcher and the kernels use, compiled by the host
// compiler.
#include <initializer_list>

#include "../memory_bound_gemv_f32_amd/csrc/kv_plan.hpp"

extern "C" {

// first, low, high, skip
void shim_span_from(int window, int sinks, int capacity, int min_pos, int max_pos, int len, int from, int* out) {
    const kvplan::Span s = kvplan::span_of(window, sinks, capacity, min_pos, max_pos, len, from);
    out[0] = s.first;
    out[1] = s.low;
    out[2] = s.high;
    out[3] = s.skip;
}
int shim_chunk_from(int first, int low, int high, int skip, int i) {
    return kvplan::Span{first, low, high, skip}.chunk(i);
}
int shim_count_from(int first, int low, int high, int skip) { return kvplan::Span{first, low, high, skip}.count(); }

// chunks; of the shared tokens and of the own ones: row_tiles, waves_share, group_rows, place_rows, splits,
// split_chunks, places; together, launchable, workspace bytes, those of the shared part
void shim_map_both(int q_heads, int heads, int dim, int rows, int sequences, int one_each, long long capacity,
                   int window, int sinks, int shared, long long* out) {
    const kvplan::SharedMapping s =
        kvplan::map_both(q_heads, heads, dim, rows, sequences, one_each != 0, capacity, window, sinks, shared);
    *out++ = s.chunks;
    for (const kvplan::Mapping* m : {&s.shared, &s.own}) {
        const long long all[] = {m->row_tiles, m->waves_share, m->group_rows, m->place_rows,
                                 m->splits,    m->split_chunks, m->places};
        for (long long v : all) *out++ = v;
    }
    *out++ = s.chunks > 0 && kvplan::together(s);
    *out++ = kvplan::launchable(s, heads);
    *out++ = (long long)kvplan::workspace_of(s, heads, dim);
    *out++ = s.chunks > 0 ? (long long)kvplan::partials_of(s.shared, heads, dim) : 0;
}

}  // extern "C"
