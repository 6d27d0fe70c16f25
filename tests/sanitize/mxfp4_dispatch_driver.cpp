// Test driver for a sanitizer build of the rules that choose the MXFP4
// product's kernel (bit_activation_compression_amd/csrc/fc_mxfp4_dispatch.h, the
// same code the launchers compile). Reads "R T K H" per line and prints what
// the product of coded operands takes, what that of 16-bit activations takes,
// and the tokens' tiles of 256, 128 and 64. Test infrastructure only.
#include <stdio.h>

#include "fc_mxfp4_dispatch.h"

int main() {
    using namespace fc;
    const int cus = 256;
    int R, T, K, H;
    while (scanf("%d %d %d %d", &R, &T, &K, &H) == 4) {
        const int Kp = (K + 127) / 128 * 128, steps = Kp / 128;
        const int rounds = mxfp4_split_rounds(R, H, steps, cus);
        const char *const tile[] = {"256", "128", "64"};
        char product[32], linear[32];
        if (mxfp4_few_tokens(R, T, steps, H, cus)) snprintf(product, sizeof product, "split%d", rounds);
        else snprintf(product, sizeof product, "%s", tile[(int)mxfp4_tile(R, T, H, cus)]);
        if (mxfp4_quantizes_in_place(T, Kp)) snprintf(linear, sizeof linear, "quantize%d", rounds);
        else snprintf(linear, sizeof linear, "%s", product);
        printf("%s %s %d %d %d\n", product, linear, mxfp4_tiles(T, 256), mxfp4_tiles(T, 128), mxfp4_tiles(T, 64));
    }
    return 0;
}
