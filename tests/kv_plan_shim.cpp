// Host build of the attention's mapping for the CPU tests: the kernels walk the
// tokens with kvplan::span_of, the launcher sizes the grid with
// kvplan::map_attend; the tests call the same functions here, compiled by the
// host compiler.
#include "../memory_bound_gemv_f32_amd/csrc/kv_plan.hpp"

extern "C" {

void shim_span(int window, int sinks, int capacity, int min_pos, int max_pos, int len, int* out) {
    const kvplan::Span s = kvplan::span_of(window, sinks, capacity, min_pos, max_pos, len);
    out[0] = s.first;
    out[1] = s.low;
    out[2] = s.high;
}

int shim_chunk(int first, int low, int high, int i) { return kvplan::Span{first, low, high}.chunk(i); }

// row_tiles, waves_share, group_rows, place_rows, splits, split_chunks, places
void shim_map(int q_heads, int heads, int dim, int rows, int sequences, int one_each, long long capacity,
              int window, int sinks, long long* out) {
    const kvplan::Mapping m =
        kvplan::map_attend(q_heads, heads, dim, rows, sequences, one_each != 0, capacity, window, sinks);
    const long long all[] = {m.row_tiles, m.waves_share, m.group_rows, m.place_rows, m.splits, m.split_chunks, m.places};
    for (int i = 0; i < 7; ++i) out[i] = all[i];
}

// floats before the first partial row, workspace bytes
void shim_workspace(int q_heads, int heads, int dim, int rows, int sequences, int one_each, long long capacity,
                    int window, int sinks, long long* out) {
    const kvplan::Mapping m =
        kvplan::map_attend(q_heads, heads, dim, rows, sequences, one_each != 0, capacity, window, sinks);
    out[0] = kvplan::stats_floats(m.places * heads * m.splits * m.place_rows);
    out[1] = (long long)kvplan::workspace_of(m, heads, dim);
}

}  // extern "C"
