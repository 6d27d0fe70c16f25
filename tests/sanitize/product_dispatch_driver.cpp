// Test driver for a sanitizer build of the rules that choose the tiles and splits of the
// matrix products (bit_activation_compression_amd/csrc/fc_product_dispatch.h, the code
// the launchers compile). Reads lines "R M N K large", prints the plan of each for a
// device of 256 compute units: two parts, the split of K, and the weight gradient's
// plan of T = K, H = M, K = N. Test infrastructure only.
#include <stdio.h>

#include "fc_product_dispatch.h"

int main() {
    int R, M, N, K, large;
    while (scanf("%d %d %d %d %d", &R, &M, &N, &K, &large) == 5) {
        const fc::ProductPlan p = fc::product_plan(R, M, N, 256, large != 0);
        for (const auto &q : p.part) printf("%d %d %d %d %d ", q.tile, q.from_m, q.to_m, q.from_n, q.to_n);
        const fc::SplitPlan s = fc::linear_plan(R, M, N, K);
        const fc::WeightGradPlan w = fc::weight_grad_plan(R, K, N, M);
        printf("%d %d %d %d %d %d\n", s.split, s.split_k, w.value_bytes != 0, w.part_bytes != 0, w.split.split, w.split.split_k);
    }
    return 0;
}
