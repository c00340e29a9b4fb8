/* Refusals of the device entry points of w2a8_block.h, each argument wrong by
 * itself: stand-in buffers lie far apart, and the call without the mistake gets
 * as far as the device, of which there is none. */
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "w2a8_block.h"

#define CHECK(c)                                                              \
    do {                                                                      \
        if (!(c)) {                                                           \
            fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #c);           \
            abort();                                                          \
        }                                                                     \
    } while (0)

/* Stand-in buffer i, 4 GiB after the one before. */
static void *at(int i) { return (void *)((uintptr_t)0x100000000 * (uintptr_t)(i + 1)); }

static int norm(int type, float eps, void *residual, void *h, void *x_q, void *s_a) {
    return rmsnorm_quant_int8(at(0), residual, at(2), type, 3, 40, eps, h, x_q, s_a, NULL);
}
static int product(int64_t group, int scale_type, void *y_f32, void *y_bf16) {
    return w4a8_gemm(at(0), at(1), at(2), 3, 40, 200, group, scale_type, 1, y_f32, y_bf16, NULL, 0, NULL);
}
static int mixture(int logit_type, int activation, void *y_f32, void *y_bf16, void *workspace) {
    return w2a8_moe(at(0), at(1), at(2), logit_type, at(3), at(4), at(5), at(6), at(7), at(8), 3, 200, 100, 6, 2,
                    activation, 1, y_f32, y_bf16, workspace, w2a8_moe_workspace_bytes(3, 200, 100, 6, 2), NULL);
}

int main(void) {
    CHECK(norm(W2A8_BF16, 1e-5f, at(1), at(3), at(4), at(5)) == W2A8_ERR_NODEVICE);
    CHECK(norm(W2A8_BF16, 0.0f, NULL, NULL, at(4), at(5)) == W2A8_ERR_NODEVICE);
    CHECK(norm(9, 1e-5f, at(1), at(3), at(4), at(5)) == W2A8_ERR_VALUE);
    CHECK(norm(-1, 1e-5f, at(1), at(3), at(4), at(5)) == W2A8_ERR_VALUE);
    CHECK(norm(W2A8_BF16, -1e-5f, at(1), at(3), at(4), at(5)) == W2A8_ERR_VALUE);
    CHECK(norm(W2A8_BF16, NAN, at(1), at(3), at(4), at(5)) == W2A8_ERR_VALUE);
    CHECK(norm(W2A8_BF16, INFINITY, at(1), at(3), at(4), at(5)) == W2A8_ERR_VALUE);
    CHECK(norm(W2A8_BF16, 1e-5f, NULL, at(3), at(4), at(5)) == W2A8_ERR_VALUE);
    for (int i = 0; i < 4; ++i) {
        CHECK(norm(W2A8_BF16, 1e-5f, at(1), at(3), at(i), at(5)) == W2A8_ERR_VALUE);
        CHECK(norm(W2A8_BF16, 1e-5f, at(1), at(3), at(4), at(i)) == W2A8_ERR_VALUE);
    }
    CHECK(norm(W2A8_BF16, 1e-5f, at(1), at(2), at(4), at(5)) == W2A8_ERR_VALUE);
    CHECK(norm(W2A8_BF16, 1e-5f, at(1), at(0), at(4), at(5)) == W2A8_ERR_NODEVICE);   /* in place */
    CHECK(norm(W2A8_BF16, 1e-5f, at(1), at(1), at(4), at(5)) == W2A8_ERR_NODEVICE);

    CHECK(product(64, W2A8_F16, at(3), at(4)) == W2A8_ERR_NODEVICE);
    CHECK(product(48, W2A8_F16, at(3), at(4)) == W2A8_ERR_VALUE);
    CHECK(product(64, W2A8_F32, at(3), at(4)) == W2A8_ERR_VALUE);
    CHECK(product(64, 9, at(3), at(4)) == W2A8_ERR_VALUE);
    for (int i = 0; i < 3; ++i) {
        CHECK(product(64, W2A8_F16, at(i), NULL) == W2A8_ERR_VALUE);
        CHECK(product(64, W2A8_F16, NULL, at(i)) == W2A8_ERR_VALUE);
    }
    CHECK(product(64, W2A8_F16, at(3), at(3)) == W2A8_ERR_VALUE);

    CHECK(mixture(W2A8_F32, W2A8_ACT_SILU, at(9), at(10), at(11)) == W2A8_ERR_NODEVICE);
    CHECK(mixture(9, W2A8_ACT_SILU, at(9), at(10), at(11)) == W2A8_ERR_VALUE);
    CHECK(mixture(W2A8_F32, 2, at(9), at(10), at(11)) == W2A8_ERR_VALUE);
    for (int i = 0; i < 9; ++i) {
        CHECK(mixture(W2A8_F32, W2A8_ACT_RELU2, at(i), NULL, at(11)) == W2A8_ERR_VALUE);
        CHECK(mixture(W2A8_F32, W2A8_ACT_RELU2, NULL, at(i), at(11)) == W2A8_ERR_VALUE);
        CHECK(mixture(W2A8_F32, W2A8_ACT_RELU2, at(9), at(10), at(i)) == W2A8_ERR_VALUE);
    }
    CHECK(mixture(W2A8_F32, W2A8_ACT_RELU2, at(9), at(9), at(11)) == W2A8_ERR_VALUE);
    CHECK(mixture(W2A8_F32, W2A8_ACT_RELU2, at(9), at(10), at(10)) == W2A8_ERR_VALUE);
    printf("host block refusals passed\n");
    return 0;
}
