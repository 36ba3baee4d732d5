/*
 * c_abi_blocks_client.c -- attention and the gated projections from plain C (C99).
 *
 *   ./c_abi_blocks_client        constants, argument checks
 *   ./c_abi_blocks_client gpu    also one call of each on the GPU, against closed forms
 *
 * Test infrastructure: built and run by tests/test_c_abi_blocks.py.
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
    size_t bytes = 7;
    const tb_heads q = {(void*)0x10000, 0, 16, 8, 2}, k = {(void*)0x20000, 0, 8, 8, 1}, v = {(void*)0x30000, 0, 8, 8, 1};
    tb_heads out = {(void*)0x40000, 0, 16, 8, 2};
    CHECK(TB_ACT_SILU == 0 && TB_ACT_GELU == 1 && TB_ACT_GELU_TANH == 2);
    CHECK(tb_attention(&q, &k, &v, &out, NULL, 0, 4, 8, NULL, 0, 1.f, TB_BF16, NULL) == TB_OK);
    CHECK(tb_attention(&q, &k, &v, &out, NULL, 1, 4, 8, NULL, 0, 0.f, TB_BF16, NULL) == TB_ERR_INVALID_VALUE);
    CHECK(tb_attention(&q, &k, &v, NULL, NULL, 1, 4, 8, NULL, 0, 1.f, TB_BF16, NULL) == TB_ERR_INVALID_VALUE);
    CHECK(tb_attention(&q, &k, &v, &out, NULL, 1, 4, 8, NULL, 0, 1.f, TB_F32, NULL) == TB_ERR_UNSUPPORTED_DTYPE);
    out.data = (void*)0x10010;
    CHECK(tb_attention(&q, &k, &v, &out, NULL, 1, 4, 8, NULL, 0, 1.f, TB_BF16, NULL) == TB_ERR_ALIAS);
    out.data = (void*)0x40008;
    CHECK(tb_attention(&q, &k, &v, &out, NULL, 1, 4, 8, NULL, 0, 1.f, TB_BF16, NULL) == TB_ERR_MISALIGNED);
    CHECK(tb_attention_bwd_workspace_size(1, 4, 2, 1, 8, TB_BF16, &bytes) == TB_OK && bytes >= 4 * 2 * 8);
    CHECK(tb_attention_bwd_workspace_size(1, 4, 2, 1, 12, TB_BF16, &bytes) == TB_ERR_INVALID_VALUE);
    CHECK(tb_gated_linear_workspace_size(0, 8, 8, TB_F16, &bytes) == TB_OK && bytes == 0);
    CHECK(tb_gated_linear_bwd_workspace_size(4, 8, 9, TB_F16, &bytes) == TB_ERR_INVALID_VALUE);
    CHECK(tb_gated_linear((void*)0x10000, (void*)0x20000, (void*)0x30000, (void*)0x40000, (void*)0x50000, NULL, 4, 8, 8, TB_ACT_SILU,
                          TB_BF16, NULL, 0, NULL) == TB_ERR_INVALID_VALUE);
    CHECK(tb_attention_selftest_timeout(5, NULL, NULL) == TB_ERR_INVALID_VALUE);
    CHECK(tb_gated_linear_selftest_timeout(5, NULL, NULL) == TB_ERR_INVALID_VALUE);
    return 0;
}

#ifdef WITH_CUDA
#include <cuda_runtime_api.h>

static float of_bf16(uint16_t x) {
    const uint32_t bits = (uint32_t)x << 16;
    float f;
    memcpy(&f, &bits, 4);
    return f;
}

static int attention_check(void) {
    /* queries of zero: every token's result is the mean of the values up to it, 0, 1, .. of their tokens, and its log
     * sum log(tokens up to it); the second sequence begins at token 3 */
    enum { kTokens = 8, kDim = 8 };
    uint16_t v[kTokens * kDim], out[kTokens * kDim];
    float lse[kTokens];
    const int64_t offsets[3] = {0, 3, 8};
    void *gq = NULL, *gv = NULL, *go = NULL, *gl = NULL, *gf = NULL;
    tb_heads q, h, o;
    int i, j;
    for (i = 0; i < kTokens * kDim; ++i) {
        const float f = (float)(i / kDim);
        uint32_t bits;
        memcpy(&bits, &f, 4);
        v[i] = (uint16_t)(bits >> 16);
    }
    CHECK(cudaMalloc(&gq, sizeof v) == cudaSuccess && cudaMalloc(&gv, sizeof v) == cudaSuccess);
    CHECK(cudaMalloc(&go, sizeof v) == cudaSuccess && cudaMalloc(&gl, sizeof lse) == cudaSuccess);
    CHECK(cudaMalloc(&gf, sizeof offsets) == cudaSuccess && cudaMemset(gq, 0, sizeof v) == cudaSuccess);
    CHECK(cudaMemcpy(gv, v, sizeof v, cudaMemcpyHostToDevice) == cudaSuccess);
    CHECK(cudaMemcpy(gf, offsets, sizeof offsets, cudaMemcpyHostToDevice) == cudaSuccess);
    q.data = gq, q.stride_batch = 0, q.stride_seq = kDim, q.stride_head = kDim, q.heads = 1;
    h = o = q;
    h.data = gv, o.data = go;
    CHECK(tb_attention(&q, &h, &h, &o, gl, 1, kTokens, kDim, gf, 2, 0.5f, TB_BF16, NULL) == TB_OK);
    CHECK(cudaMemcpy(out, go, sizeof out, cudaMemcpyDeviceToHost) == cudaSuccess);
    CHECK(cudaMemcpy(lse, gl, sizeof lse, cudaMemcpyDeviceToHost) == cudaSuccess);
    for (i = 0; i < kTokens; ++i) {
        const int first = i < 3 ? 0 : 3;
        const double mean = (first + i) / 2.0;
        CHECK(fabs(lse[i] - log(i - first + 1.0)) <= 1e-6);
        for (j = 0; j < kDim; ++j) CHECK(fabs(of_bf16(out[i * kDim + j]) - mean) <= mean / 256);
    }
    cudaFree(gq), cudaFree(gv), cudaFree(go), cudaFree(gl), cudaFree(gf);
    printf("attention through the C ABI: ok\n");
    return 0;
}

static int gated_check(void) {
    /* ones everywhere, 8 contracted elements: G = U = 8, H = 64 / (1 + exp(-8)) */
    enum { kRows = 3, kD = 8, kF = 16 };
    uint16_t ones[kF * kD], H[kRows * kF], G[kRows * kF];
    void *gX = NULL, *gW = NULL, *gH = NULL, *gG = NULL, *gU = NULL, *ws = NULL;
    size_t bytes = 0;
    int i;
    for (i = 0; i < kF * kD; ++i) ones[i] = 0x3F80; /* 1.0 in bfloat16 */
    CHECK(tb_gated_linear_workspace_size(kRows, kD, kF, TB_BF16, &bytes) == TB_OK);
    CHECK(cudaMalloc(&gX, sizeof ones) == cudaSuccess && cudaMalloc(&gW, sizeof ones) == cudaSuccess);
    CHECK(cudaMalloc(&gH, sizeof H) == cudaSuccess && cudaMalloc(&gG, sizeof H) == cudaSuccess && cudaMalloc(&gU, sizeof H) == cudaSuccess);
    CHECK(cudaMalloc(&ws, bytes + 256) == cudaSuccess);
    CHECK(cudaMemcpy(gX, ones, sizeof ones, cudaMemcpyHostToDevice) == cudaSuccess);
    CHECK(cudaMemcpy(gW, ones, sizeof ones, cudaMemcpyHostToDevice) == cudaSuccess);
    CHECK(tb_gated_linear(gX, gW, gW, gH, gG, gU, kRows, kD, kF, TB_ACT_SILU, TB_BF16, ws, bytes, NULL) == TB_OK);
    CHECK(cudaMemcpy(H, gH, sizeof H, cudaMemcpyDeviceToHost) == cudaSuccess);
    CHECK(cudaMemcpy(G, gG, sizeof G, cudaMemcpyDeviceToHost) == cudaSuccess);
    for (i = 0; i < kRows * kF; ++i) {
        const double want = 64.0 / (1.0 + exp(-8.0));
        CHECK(of_bf16(G[i]) == 8.f && fabs(of_bf16(H[i]) - want) <= want / 256 + 1e-4);
    }
    cudaFree(gX), cudaFree(gW), cudaFree(gH), cudaFree(gG), cudaFree(gU), cudaFree(ws);
    printf("gated projections through the C ABI: ok\n");
    return 0;
}
#endif

int main(int argc, char** argv) {
    int rc = cpu_checks();
    if (rc == 0) printf("argument checks through the C ABI: ok\n");
#ifdef WITH_CUDA
    if (rc == 0 && argc > 1 && strcmp(argv[1], "gpu") == 0) {
        int code = -1;
        rc = attention_check();
        if (rc == 0) rc = gated_check();
        if (rc == 0 && (tb_device_error(&code, 1) != TB_OK || code != 0)) rc = 1;
    }
#else
    (void)argc;
    (void)argv;
#endif
    return rc;
}
