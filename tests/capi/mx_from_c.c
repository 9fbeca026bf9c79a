/*
 * The microscaled formats from plain C: a weight quantised to 4 bits and an
 * activation kept in 8, the linear layer and both of its gradients, on whole
 * numbers that both formats hold, so that every result is exact.  Exit status 0
 * and "microscaled: exact" on success.
 */
#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "zs.h"

#define CHECK_HIP(x)                                                                  \
    do {                                                                              \
        hipError_t e_ = (x);                                                          \
        if (e_ != hipSuccess) {                                                       \
            fprintf(stderr, "%s failed: %s\n", #x, hipGetErrorString(e_));            \
            return 1;                                                                 \
        }                                                                             \
    } while (0)
#define CHECK_ZS(x)                                                                   \
    do {                                                                              \
        int r_ = (x);                                                                 \
        if (r_ != ZS_OK) {                                                            \
            fprintf(stderr, "%s failed: %s\n", #x, zs_status_string(r_));             \
            return 1;                                                                 \
        }                                                                             \
    } while (0)

enum { M = 19, N = 45, K = 100 };

static uint32_t st_ = 12345u;
static int rnd(int below) {
    st_ = st_ * 1664525u + 1013904223u;
    return (int)((st_ >> 16) % (uint32_t)below);
}

static uint16_t bf16(float f) {
    uint32_t u;
    memcpy(&u, &f, 4);
    return (uint16_t)(u >> 16);
}

int main(void) {
    static float x[M][K], w[N][K], dy[M][N], y[M][N], dx[M][K], dw[N][K];
    static uint16_t xb[M][K], dyb[M][N];
    const float four[4] = {0.0f, 1.0f, 2.0f, 4.0f};
    for (int i = 0; i < M; ++i)
        for (int k = 0; k < K; ++k) {
            x[i][k] = (float)(rnd(15) - 7);
            xb[i][k] = bf16(x[i][k]);
        }
    for (int j = 0; j < N; ++j)
        for (int k = 0; k < K; ++k) w[j][k] = four[rnd(4)] * (rnd(2) ? 1.0f : -1.0f);
    for (int i = 0; i < M; ++i)
        for (int j = 0; j < N; ++j) {
            dy[i][j] = (float)(rnd(9) - 4);
            dyb[i][j] = bf16(dy[i][j]);
        }

    CHECK_ZS(zs_init(0));
    hipStream_t s;
    CHECK_HIP(hipStreamCreate(&s));
    void *d[7], *ws;
    const size_t size[7] = {sizeof xb, sizeof w, sizeof dyb, sizeof y, sizeof dx, sizeof dw, 0};
    for (int i = 0; i < 6; ++i) CHECK_HIP(hipMalloc(&d[i], size[i]));
    CHECK_HIP(hipMalloc(&ws, ZS_MX_WORKSPACE_BYTES));
    CHECK_HIP(hipMemset(ws, 0, ZS_MX_WORKSPACE_BYTES));
    CHECK_HIP(hipMemcpy(d[0], xb, sizeof xb, hipMemcpyHostToDevice));
    CHECK_HIP(hipMemcpy(d[1], w, sizeof w, hipMemcpyHostToDevice));
    CHECK_HIP(hipMemcpy(d[2], dyb, sizeof dyb, hipMemcpyHostToDevice));
    zs_mx wq = {NULL, NULL, N, K, ZS_MX_FP4, 0}, xq = {NULL, NULL, M, K, ZS_MX_FP8, 0};
    CHECK_HIP(hipMalloc((void **)&wq.codes, (size_t)(N * ZS_MX_ROW_BYTES(ZS_MX_FP4, K))));
    CHECK_HIP(hipMalloc((void **)&wq.scales, (size_t)(N * ((K + 31) / 32))));
    CHECK_HIP(hipMalloc((void **)&xq.codes, (size_t)(M * ZS_MX_ROW_BYTES(ZS_MX_FP8, K))));
    CHECK_HIP(hipMalloc((void **)&xq.scales, (size_t)(M * ((K + 31) / 32))));
    CHECK_HIP(hipDeviceSynchronize());

    const zs_matrix mx = {d[0], M, K, K, ZS_DTYPE_BF16, 0}, mw = {d[1], N, K, K, ZS_DTYPE_FP32, 0};
    const zs_matrix mdy = {d[2], M, N, N, ZS_DTYPE_BF16, 0};
    const zs_matrix my = {d[3], M, N, N, ZS_DTYPE_FP32, 0};
    const zs_matrix mdx = {d[4], M, K, K, ZS_DTYPE_FP32, 0};
    const zs_matrix mdw = {d[5], N, K, K, ZS_DTYPE_FP32, 0};
    CHECK_ZS(zs_mx_quantize(&mw, &wq, s));
    CHECK_ZS(zs_mx_quantize(&mx, &xq, s));
    CHECK_ZS(zs_mx_linear(&mx, &wq, &my, ws, s));
    CHECK_ZS(zs_mx_linear_dgrad(&mdy, &wq, &mdx, ws, s));
    CHECK_ZS(zs_mx_linear_wgrad(&mdy, &xq, &mdw, 0, ws, s));
    CHECK_ZS(zs_mx_linear_wgrad(&mdy, &xq, &mdw, 1, NULL, s));
    CHECK_HIP(hipStreamSynchronize(s));
    CHECK_HIP(hipMemcpy(y, d[3], sizeof y, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(dx, d[4], sizeof dx, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(dw, d[5], sizeof dw, hipMemcpyDeviceToHost));
    for (int i = 0; i < M; ++i)
        for (int j = 0; j < N; ++j) {
            float want = 0.0f;
            for (int k = 0; k < K; ++k) want += x[i][k] * w[j][k];
            if (y[i][j] != want) return fprintf(stderr, "y[%d][%d]\n", i, j), 1;
        }
    for (int i = 0; i < M; ++i)
        for (int k = 0; k < K; ++k) {
            float want = 0.0f;
            for (int j = 0; j < N; ++j) want += dy[i][j] * w[j][k];
            if (dx[i][k] != want) return fprintf(stderr, "dx[%d][%d]\n", i, k), 1;
        }
    for (int j = 0; j < N; ++j)
        for (int k = 0; k < K; ++k) {
            float want = 0.0f;
            for (int i = 0; i < M; ++i) want += 2.0f * dy[i][j] * x[i][k];
            if (dw[j][k] != want) return fprintf(stderr, "dw[%d][%d]\n", j, k), 1;
        }
    /* dequantised again: the same numbers */
    const zs_matrix back = {d[5], N, K, K, ZS_DTYPE_FP32, 0};
    CHECK_ZS(zs_mx_dequantize(&wq, &back, s));
    CHECK_HIP(hipStreamSynchronize(s));
    CHECK_HIP(hipMemcpy(dw, d[5], sizeof dw, hipMemcpyDeviceToHost));
    if (memcmp(dw, w, sizeof w)) {
        for (int j = 0; j < N; ++j)
            for (int k = 0; k < K; ++k)
                if (dw[j][k] != w[j][k]) return fprintf(stderr, "w[%d][%d]\n", j, k), 1;
    }
    puts("microscaled: exact");
    return 0;
}
