/* Host side of the entry points of w2a8_block.h under AddressSanitizer and
 * UndefinedBehaviorSanitizer: size queries, packers on heap buffers of
 * exactly the documented sizes, and argument validation. */
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "w2a8_block.h"

#define CHECK(c)                                                              \
    do {                                                                      \
        if (!(c)) {                                                           \
            fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #c);           \
            abort();                                                          \
        }                                                                     \
    } while (0)

static void round_trip(int64_t N, int64_t K, int64_t group, int zeros) {
    const int64_t row = (K + 1) / 2, groups = (K + group - 1) / group;
    const int64_t nb = w4a8_packed_bytes(N, K, group, zeros), ng = N * groups;
    uint8_t *c = malloc((size_t)(N * row)), *c2 = malloc((size_t)(N * row));
    uint16_t *s = malloc((size_t)ng * 2), *s2 = malloc((size_t)ng * 2);
    uint8_t *z = zeros ? malloc((size_t)ng) : NULL, *z2 = zeros ? malloc((size_t)ng) : NULL;
    uint8_t *p = malloc((size_t)nb);
    for (int64_t i = 0; i < N * row; ++i) c[i] = (uint8_t)(i * 37 + 11);
    if (K & 1)
        for (int64_t n = 0; n < N; ++n) c[n * row + row - 1] &= 15;
    for (int64_t i = 0; i < ng; ++i) s[i] = (uint16_t)(i * 2903 + 3);
    for (int64_t i = 0; zeros && i < ng; ++i) z[i] = (uint8_t)(i % 16);
    CHECK(pack_w4a8(c, s, z, N, K, group, p, nb) == W2A8_OK);
    CHECK(unpack_w4a8(p, nb, N, K, group, c2, s2, z2) == W2A8_OK);
    CHECK(memcmp(c, c2, (size_t)(N * row)) == 0 && memcmp(s, s2, (size_t)ng * 2) == 0);
    CHECK(!zeros || memcmp(z, z2, (size_t)ng) == 0);
    CHECK(pack_w4a8(c, s, z, N, K, group, p, nb - 1) == W2A8_ERR_BUFSIZE);
    free(c);
    free(c2);
    free(s);
    free(s2);
    free(z);
    free(z2);
    free(p);
}

int main(void) {
    const int64_t ns[] = {1, 15, 16, 17, 33}, ks[] = {1, 2, 31, 32, 33, 127, 128, 129, 512, 513, 1000};
    for (size_t i = 0; i < sizeof ns / sizeof *ns; ++i)
        for (size_t j = 0; j < sizeof ks / sizeof *ks; ++j)
            for (int64_t g = 32; g <= 128; g *= 2)
                for (int z = 0; z < 2; ++z) round_trip(ns[i], ks[j], g, z);
    CHECK(w4a8_packed_bytes((int64_t)1 << 30, W2A8_MAX_K, 32, 1) > 0);
    CHECK(w4a8_packed_bytes((int64_t)1 << 62, 1, 32, 0) == -1 && w4a8_packed_bytes(1, 1, 0, 0) == -1);
    CHECK(w4a8_workspace_bytes(64, (int64_t)1 << 30, W2A8_MAX_K) > 0);
    CHECK(w4a8_workspace_bytes((int64_t)1 << 62, 1, 1) == -1);
    CHECK(w2a8_moe_workspace_bytes(64, W2A8_MAX_K, W2A8_MAX_K, 256, 16) > 0);
    CHECK(w2a8_moe_workspace_bytes(64, (int64_t)1 << 62, 1, 1, 1) == -1);
    uint8_t *fake = (uint8_t *)0x10000;
    float *f = (float *)fake;
    CHECK(rmsnorm_quant_int8(NULL, NULL, NULL, 1, 1, 1, 0.0f, NULL, (int8_t *)fake, f, NULL) == W2A8_ERR_NULL);
    CHECK(rmsnorm_quant_int8(fake, NULL, NULL, 9, 1, 1, 0.0f, NULL, (int8_t *)fake, f, NULL) == W2A8_ERR_VALUE);
    CHECK(w4a8_gemm(fake, (int8_t *)fake, f, 1, 1, -5, 32, 2, 0, f, NULL, NULL, 0, NULL) == W2A8_ERR_SHAPE);
    CHECK(w2a8_moe((int8_t *)fake, f, fake, 0, fake, fake, fake, f, f, f, 1, 1, 1, 1, 2, 0, 1, f, NULL, fake, 1 << 30,
                   NULL) == W2A8_ERR_SHAPE);
    printf("host block checks passed\n");
    return 0;
}
