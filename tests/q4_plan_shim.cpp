// Host build of the sizes of the products with 4-bit weights, and of the rule for their
// kernels, for the CPU tests.
#include "../memory_bound_gemv_f32_amd/csrc/q4_plan.hpp"

extern "C" {

int shim_groups_of(int K, int log2) { return q4plan::groups_of(K, log2); }
int shim_family(int parts, int M, int K, int T, int far, int whole) {
    return q4plan::family_of(parts, M, K, T, far != 0, whole != 0);
}
long long shim_staged_bytes(int parts, int K, int T) { return q4plan::staged_bytes(parts, K, T); }

}  // extern "C"
