// Test driver for a sanitizer build of the argument checks of the
// transformer-block operators (bit_activation_compression_amd/csrc/
// fc_validate_layer.h, the same code fc_api.hip compiles). Prints the status of
// every argument set of two grids; the Python test compares those that refuse
// with what libfc.so returns. Test infrastructure only.
#include <math.h>
#include <stdio.h>

#include "fc_validate_layer.h"

int main() {
    using namespace fc::validate;
    const int Ts[] = {-1, 0, 1, 7, 1 << 20};
    const int Hs[] = {0, 1, 8, 4096, 65536, 65537};
    const int tokens[] = {0, 1, 100};
    const float values[] = {0.0f, 1.0f, -2.0f, 1e-39f, 1e30f, HUGE_VALF, -HUGE_VALF, (float)NAN};
    // regions of 64 MiB of their own, never touched
    auto at = [](int i, int off) { return reinterpret_cast<void *>((uintptr_t)0x10000000 + ((uintptr_t)i << 26) + off); };
    for (int T : Ts)
        for (int H : Hs)
            for (int gt : tokens)
                for (int v = 0; v < 8; ++v)
                    for (int bad = 0; bad < 6; ++bad) {
                        const size_t n = (size_t)(T > 0 ? T : 0) * (size_t)H * 2;
                        void *x = bad == 1 ? nullptr : at(0, 0), *h = bad == 2 ? x : at(5, bad == 3 ? 8 : 0);
                        void *y = bad == 4 ? nullptr : at(6, 0), *res = bad == 5 ? h : at(1, 0);
                        const fc_status st = check_norm(T, H, FC_BF16, {{x, n}}, res, at(2, 0), at(3, 0), gt,
                                                        at(4, 0), 1.0f, values[v], 1e-5f, h, y);
                        const fc_status se = check_norm(T, H, FC_BF16, {{x, n}}, res, at(2, 0), at(3, 0), gt,
                                                        at(4, 0), 1.0f, 1.0f, values[v], h, y);
                        printf("norm %d %d %d %d %d : %d %d\n", T, H, gt, v, bad, (int)st, (int)se);
                    }
    const int Rs[] = {0, 1, 4, 1 << 20};
    const int Ks[] = {0, 1, 127, 128, 129, 1 << 22, (1 << 22) + 1};
    const int Hp[] = {0, 1, 100, 1 << 24, (1 << 24) + 1};
    for (int R : Rs)
        for (int T : Ts)
            for (int K : Ks)
                for (int H : Hp)
                    printf("mx %d %d %d %d : %d %d %zu %zu\n", R, T, K, H, (int)check_mx(R, T, K),
                           (int)check_mx_product(R, T, K, H), mx_padded(K), mx_code_bytes(1, 1, K));
    return 0;
}
