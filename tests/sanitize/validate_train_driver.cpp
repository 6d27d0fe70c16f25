// Test driver for a sanitizer build of the argument checks of the training
// operators (bit_activation_compression_amd/csrc/fc_validate_train.h, the same code
// fc_train_api.hip compiles). Prints the answers over grids of arguments; the Python
// test compares them with what libfc.so returns. Test infrastructure only.
#include <stdio.h>

#include "fc_validate_train.h"

int main() {
    using namespace fc::validate;
    const int Rs[] = {-1, 0, 1, 3, 1 << 20, 2147483647};
    const int Ts[] = {-1, 0, 1, 17, 1 << 20, 2147483647};
    const int sizes[] = {0, 1, 15, 17, 4096, 1 << 22, (1 << 22) + 1, 2147483647};
    for (int R : Rs)
        for (int T : Ts)
            for (int K : sizes)
                for (int H : sizes) printf("product %d %d %d %d : %d\n", R, T, K, H, (int)check_product(R, T, K, H));
    const int groups[] = {-8, 0, 4, 8, 12, 24, 4096, 2147483640};
    for (int H : sizes)
        for (int g : groups) printf("group %d %d : %d\n", H, g, H > 0 && payload_group_ok(H, g) ? 1 : 0);
    for (int R : Rs)
        for (int T : Ts)
            for (int H : sizes)
                if (R > 0 && T > 0 && H > 0) printf("elems %d %d %d : %d\n", R, T, H, elems_ok(R, T, H) ? 1 : 0);
    return 0;
}
