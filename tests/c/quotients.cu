/* The quotients that the token moves' kernels take by a product, on the host:
 * every divisor of the stated range with the numbers on both sides of each of its
 * multiples.  Prints ok, or the first wrong one. */
#define BMMC_CHK_FILE 99
#include "bounds.cuh"
#include "token_words.cuh"

#include <cstdio>

int main() {
    for (int d = 1; d <= 8192; ++d) {
        const uint64_t magic = bmmc::wide_magic_of(d);
        for (int x = 0; x < 1 << 24; x += d) {
            const int last = x + d - 1 < (1 << 24) - 1 ? x + d - 1 : (1 << 24) - 1;
            if (bmmc::wide_quotient(x, magic) != x / d || bmmc::wide_quotient(last, magic) != last / d) {
                std::printf("%d or %d by %d\n", x, last, d);
                return 1;
            }
        }
    }
    std::printf("ok\n");
    return 0;
}
