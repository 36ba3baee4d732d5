/*
 * c_abi_heads_client.c -- the rotary and output-layer entry points from plain C (C99).
 *
 *   ./c_abi_heads_client        layouts of the structs, argument checks, a frequency table
 *   ./c_abi_heads_client gpu    also a rotation and a loss on the GPU, against closed forms
 *
 * Test infrastructure: built and run by tests/test_c_abi_heads.py.
 */
#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "tb.h"

#define CHECK(cond)                                                              \
    do {                                                                         \
        if (!(cond)) {                                                           \
            fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
            return 1;                                                            \
        }                                                                        \
    } while (0)

static int cpu_checks(void) {
    uint64_t freqs[4];
    float magnitude = 0.f;
    size_t bytes = 7;
    tb_heads q = {(void*)0x1000, 64, 16, 8, 2}, out = {(void*)0x9000, 64, 16, 8, 2};
    tb_rope_angles angles = {NULL, NULL, 0, 0, 8, TB_ROPE_HALF, 1.f};
    tb_rope_scaling linear = {TB_ROPE_SCALE_LINEAR, 2.0, 0, 0, 0};
    /* what other languages' bindings lay out by hand */
    CHECK(sizeof(tb_heads) == 40 && offsetof(tb_heads, stride_batch) == 8 && offsetof(tb_heads, heads) == 32);
    CHECK(sizeof(tb_rope_angles) == 48 && offsetof(tb_rope_angles, offset) == 24);
    CHECK(offsetof(tb_rope_angles, rotary_dim) == 32 && offsetof(tb_rope_angles, magnitude) == 40);
    CHECK(tb_rope_freqs(8, 16.0, NULL, freqs, &magnitude) == TB_OK && magnitude == 1.f);
    /* 16^(-2i/8): each frequency is half of the one before */
    CHECK(fabs((double)freqs[0] / 18446744073709551616.0 - 0.15915494309189535) < 1e-15);
    CHECK(freqs[1] / 2 >= freqs[2] - 2 && freqs[1] / 2 <= freqs[2] + 2);
    CHECK(tb_rope_freqs(8, 16.0, &linear, freqs, &magnitude) == TB_OK);
    CHECK(fabs((double)freqs[0] / 18446744073709551616.0 - 0.07957747154594767) < 1e-15);
    CHECK(tb_rope_freqs(7, 16.0, NULL, freqs, &magnitude) == TB_ERR_INVALID_VALUE);
    CHECK(tb_rope(&q, NULL, &out, NULL, 1, 1, 8, &angles, TB_F32, NULL) == TB_ERR_INVALID_VALUE); /* no freqs */
    CHECK(tb_rope(&q, NULL, &out, NULL, 1, 1, 8, NULL, TB_F32, NULL) == TB_ERR_INVALID_VALUE);
    angles.rotary_dim = 0;
    CHECK(tb_rope(&q, NULL, &out, &out, 1, 1, 8, &angles, TB_F32, NULL) == TB_ERR_INVALID_VALUE);
    out.data = (void*)0x1004;
    CHECK(tb_rope(&q, NULL, &out, NULL, 1, 2, 8, &angles, TB_F32, NULL) == TB_ERR_ALIAS);
    CHECK(tb_rope(&q, NULL, &out, NULL, 0, 2, 8, &angles, TB_F32, NULL) == TB_OK);
    CHECK(tb_qk_norm_rope_bwd_workspace_size(0, 2, 4, 2, 64, TB_F32, &bytes) == TB_OK && bytes == 0);
    CHECK(tb_linear_xent_workspace_size(0, 8, 8, TB_BF16, &bytes) == TB_OK && bytes == 0);
    CHECK(tb_linear_xent_bwd_workspace_size(1, 8, 8, TB_F32, &bytes) == TB_ERR_UNSUPPORTED_DTYPE);
    CHECK(tb_linear_xent((void*)0x1000, (void*)0x2000, NULL, NULL, NULL, 1, 8, 8, -100, TB_BF16, NULL, 0, NULL) ==
          TB_ERR_INVALID_VALUE);
    CHECK(tb_linear_xent_selftest_timeout(5, NULL, NULL) == TB_ERR_INVALID_VALUE);
    return 0;
}

#ifdef WITH_CUDA
#include <cuda_runtime_api.h>

static int rope_check(void) {
    /* two tokens of one head of four elements, at positions 0 and 3, frequencies 1 and 1/4 a radian */
    const float x[8] = {1, 2, 3, 4, 1, 2, 3, 4};
    float y[8], magnitude;
    int64_t positions[2] = {0, 3};
    uint64_t freqs[2];
    void *gx = NULL, *gp = NULL, *gf = NULL;
    tb_heads heads = {NULL, 8, 4, 4, 1};
    tb_rope_angles angles = {NULL, NULL, 0, 0, 4, TB_ROPE_HALF, 1.f};
    int i;
    CHECK(tb_rope_freqs(4, 16.0, NULL, freqs, &magnitude) == TB_OK);
    CHECK(cudaMalloc(&gx, sizeof x) == cudaSuccess && cudaMalloc(&gp, sizeof positions) == cudaSuccess);
    CHECK(cudaMalloc(&gf, sizeof freqs) == cudaSuccess);
    CHECK(cudaMemcpy(gx, x, sizeof x, cudaMemcpyHostToDevice) == cudaSuccess);
    CHECK(cudaMemcpy(gp, positions, sizeof positions, cudaMemcpyHostToDevice) == cudaSuccess);
    CHECK(cudaMemcpy(gf, freqs, sizeof freqs, cudaMemcpyHostToDevice) == cudaSuccess);
    heads.data = gx;
    angles.freqs = gf;
    angles.positions = gp;
    CHECK(tb_rope(&heads, NULL, &heads, NULL, 1, 2, 4, &angles, TB_F32, NULL) == TB_OK); /* in place */
    CHECK(cudaMemcpy(y, gx, sizeof y, cudaMemcpyDeviceToHost) == cudaSuccess);
    for (i = 0; i < 4; ++i) CHECK(y[i] == x[i]);
    for (i = 0; i < 2; ++i) {
        const double t = 3.0 * (i ? 0.25 : 1.0);
        CHECK(fabs(y[4 + i] - (x[i] * cos(t) - x[i + 2] * sin(t))) <= 4e-6);
        CHECK(fabs(y[6 + i] - (x[i] * sin(t) + x[i + 2] * cos(t))) <= 4e-6);
    }
    cudaFree(gx), cudaFree(gp), cudaFree(gf);
    printf("rotation through the C ABI: ok\n");
    return 0;
}

static int loss_check(void) {
    /* weights of zero: lse = log(vocab), G = 1/vocab - onehot, dW of a row = dloss * sum of H * G */
    const int64_t rows = 3, D = 16, vocab = 32;
    uint16_t H[48], dW[512];
    int64_t targets[3] = {5, 31, -100};
    float loss[3], lse[3], dloss[3] = {1, 1, 1};
    void *gH = NULL, *gW = NULL, *gt = NULL, *gl = NULL, *gs = NULL, *gd = NULL, *gdW = NULL, *ws = NULL;
    size_t a = 0, b = 0;
    int i;
    for (i = 0; i < 48; ++i) H[i] = 0x3F80; /* 1.0 in bfloat16 */
    CHECK(tb_linear_xent_workspace_size(rows, D, vocab, TB_BF16, &a) == TB_OK);
    CHECK(tb_linear_xent_bwd_workspace_size(rows, D, vocab, TB_BF16, &b) == TB_OK);
    if (a < b) a = b;
    CHECK(cudaMalloc(&gH, sizeof H) == cudaSuccess && cudaMalloc(&gW, sizeof dW) == cudaSuccess);
    CHECK(cudaMalloc(&gdW, sizeof dW) == cudaSuccess && cudaMalloc(&gt, sizeof targets) == cudaSuccess);
    CHECK(cudaMalloc(&gl, 12) == cudaSuccess && cudaMalloc(&gs, 12) == cudaSuccess && cudaMalloc(&gd, 12) == cudaSuccess);
    CHECK(cudaMalloc(&ws, a) == cudaSuccess && cudaMemset(gW, 0, sizeof dW) == cudaSuccess);
    CHECK(cudaMemcpy(gH, H, sizeof H, cudaMemcpyHostToDevice) == cudaSuccess);
    CHECK(cudaMemcpy(gt, targets, sizeof targets, cudaMemcpyHostToDevice) == cudaSuccess);
    CHECK(cudaMemcpy(gd, dloss, sizeof dloss, cudaMemcpyHostToDevice) == cudaSuccess);
    CHECK(tb_linear_xent(gH, gW, gt, gl, gs, rows, D, vocab, -100, TB_BF16, ws, a, NULL) == TB_OK);
    CHECK(tb_linear_xent_bwd(gd, gH, gW, gt, gs, NULL, gdW, rows, D, vocab, -100, TB_BF16, ws, a, NULL) == TB_OK);
    CHECK(cudaMemcpy(loss, gl, 12, cudaMemcpyDeviceToHost) == cudaSuccess);
    CHECK(cudaMemcpy(lse, gs, 12, cudaMemcpyDeviceToHost) == cudaSuccess);
    CHECK(cudaMemcpy(dW, gdW, sizeof dW, cudaMemcpyDeviceToHost) == cudaSuccess);
    for (i = 0; i < 3; ++i) CHECK(fabs(lse[i] - log(32.0)) <= 1e-6);
    CHECK(fabs(loss[0] - log(32.0)) <= 1e-6 && loss[2] == 0.f);
    for (i = 0; i < 512; ++i) { /* 2/32, or 2/32 - 1 in the targets' rows */
        const uint32_t bits = (uint32_t)dW[i] << 16;
        const double want = 2.0 / 32 - (i / 16 == 5 || i / 16 == 31);
        float got;
        memcpy(&got, &bits, 4);
        CHECK(fabs(got - want) <= 3 * 0.00390625 * fabs(want) + 1e-6);
    }
    cudaFree(gH), cudaFree(gW), cudaFree(gdW), cudaFree(gt), cudaFree(gl), cudaFree(gs), cudaFree(gd), cudaFree(ws);
    printf("output layer's loss through the C ABI: ok\n");
    return 0;
}
#endif

int main(int argc, char** argv) {
    int rc = cpu_checks();
    if (rc == 0) printf("argument checks through the C ABI: ok\n");
#ifdef WITH_CUDA
    if (rc == 0 && argc > 1 && strcmp(argv[1], "gpu") == 0) {
        int code = -1;
        rc = rope_check();
        if (rc == 0) rc = loss_check();
        if (rc == 0 && (tb_device_error(&code, 1) != TB_OK || code != 0)) rc = 1;
    }
#else
    (void)argc;
    (void)argv;
#endif
    return rc;
}
