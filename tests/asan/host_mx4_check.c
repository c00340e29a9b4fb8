/* Host side of the MX4 entry points under AddressSanitizer and
 * UndefinedBehaviorSanitizer: size queries, packers on heap buffers of
 * exactly the documented sizes, and argument validation. */
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "w2a8_mx4.h"

#define CHECK(c)                                                              \
    do {                                                                      \
        if (!(c)) {                                                           \
            fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #c);           \
            abort();                                                          \
        }                                                                     \
    } while (0)

static void round_trip(int64_t N, int64_t K) {
    const int64_t row = (K + 1) / 2, blocks = (K + 31) / 32, nb = mx4_packed_bytes(N, K);
    uint8_t *c = malloc((size_t)(N * row)), *s = malloc((size_t)(N * blocks));
    uint8_t *c2 = malloc((size_t)(N * row)), *s2 = malloc((size_t)(N * blocks));
    uint8_t *p = malloc((size_t)nb);
    for (int64_t i = 0; i < N * row; ++i) c[i] = (uint8_t)(i * 37 + 11);
    if (K & 1)
        for (int64_t n = 0; n < N; ++n) c[n * row + row - 1] &= 15;
    for (int64_t i = 0; i < N * blocks; ++i) s[i] = (uint8_t)(i * 29 + 3);
    CHECK(pack_mx4(c, s, N, K, p, nb) == W2A8_OK);
    CHECK(unpack_mx4(p, nb, N, K, c2, s2) == W2A8_OK);
    CHECK(memcmp(c, c2, (size_t)(N * row)) == 0 && memcmp(s, s2, (size_t)(N * blocks)) == 0);
    CHECK(pack_mx4(c, s, N, K, p, nb - 1) == W2A8_ERR_BUFSIZE);
    free(c);
    free(s);
    free(c2);
    free(s2);
    free(p);
}

int main(void) {
    const int64_t ns[] = {1, 15, 16, 17, 33}, ks[] = {1, 2, 31, 32, 33, 127, 128, 129, 512, 513, 1000};
    for (size_t i = 0; i < sizeof ns / sizeof *ns; ++i)
        for (size_t j = 0; j < sizeof ks / sizeof *ks; ++j) round_trip(ns[i], ks[j]);
    CHECK(mx4_act_bytes(0, 1) == -1 && mx4_scale_bytes(1, 0) == -1);
    CHECK(mx4_packed_bytes((int64_t)1 << 30, W2A8_MAX_K) > 0);
    CHECK(mx4_act_bytes((int64_t)1 << 62, 1) == -1 && mx4_packed_bytes(1, (int64_t)1 << 62) == -1);
    uint8_t *fake = (uint8_t *)0x10000;
    CHECK(quant_act_mx4(NULL, 0, 1, 1, fake, fake, NULL) == W2A8_ERR_NULL);
    CHECK(quant_act_mx4(fake, 9, 1, 1, fake, fake, NULL) == W2A8_ERR_VALUE);
    CHECK(w4mx4_gemm(fake, fake, fake, 1, 1, -5, (float *)fake, NULL, NULL) == W2A8_ERR_SHAPE);
    CHECK(w2mx4_linear_gemv(fake, fake, 1, 1, 1, 1.0f, NULL, NULL, NULL) == W2A8_ERR_NULL);
    printf("host MX4 checks passed\n");
    return 0;
}
