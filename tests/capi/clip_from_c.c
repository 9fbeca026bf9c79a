/*
 * The norm and clipping calls from plain C: a shard's partials and two tensors
 * outside it, their sums of squares, the coefficient of the total, the clipped
 * shard step against the C oracle's step with the same coefficient, and the
 * tensors scaled.  Exit status 0 and "clipping: equal to the oracle" on success.
 */
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "zs.h"

/* the oracle's own declaration (it has no header; same field layout) */
int zs_oracle_shard_step(float *, float *, float *, uint16_t *, const uint16_t *const *, int,
                         int64_t, const zs_segment *, int32_t, const zs_hparams *, int64_t);

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

enum { N = 300007, K = 3, T0 = 4099, T1 = 777 };

static uint64_t st_ = 0x853C49E6748FEA9Bull;
static float rndf(float s) {
    st_ ^= st_ << 13;
    st_ ^= st_ >> 7;
    st_ ^= st_ << 17;
    return ((float)((uint32_t)(st_ >> 11) % 20001) - 10000.0f) * s * 1e-4f;
}

static float widen(uint16_t b) {
    uint32_t u = (uint32_t)b << 16;
    float f;
    memcpy(&f, &u, 4);
    return f;
}

int main(void) {
    zs_segment segs[3] = {{0, 1, 0}, {1000, 0, 0}, {1001, 1, 0}};
    zs_hparams hp = {1e-3f, 0.9f, 0.95f, 1e-8f, 0.1f, 0.5f};
    zs_clip_rule rule = {0.75f, 1e-6f, 0, 0};
    float *w = malloc(4 * N), *m = calloc(N, 4), *v = calloc(N, 4), *x = malloc(4 * T0);
    uint16_t *p = calloc(N, 2), *g[K];
    float *got = malloc(4 * N);
    double total = 0.0;

    CHECK_ZS(zs_init(0));
    hipStream_t s;
    CHECK_HIP(hipStreamCreate(&s));
    float *dw, *dm, *dv, *dx;
    uint16_t *dp, *dg[K];
    zs_segment *dsegs;
    zs_clip *rec;
    double *sums;
    void *ws[2];
    zs_piece *dpieces;
    CHECK_HIP(hipMalloc((void **)&dw, 4 * N));
    CHECK_HIP(hipMalloc((void **)&dm, 4 * N));
    CHECK_HIP(hipMalloc((void **)&dv, 4 * N));
    CHECK_HIP(hipMalloc((void **)&dp, 2 * N));
    CHECK_HIP(hipMalloc((void **)&dsegs, sizeof segs));
    CHECK_HIP(hipMalloc((void **)&rec, 2 * sizeof(zs_clip)));
    CHECK_HIP(hipMalloc((void **)&sums, 2 * sizeof(double)));
    CHECK_HIP(hipMalloc((void **)&dx, 4 * T0 + 2 * T1));
    for (int j = 0; j < 2; ++j) {
        CHECK_HIP(hipMalloc(&ws[j], ZS_NORM_WORKSPACE_BYTES));
        CHECK_HIP(hipMemset(ws[j], 0, ZS_NORM_WORKSPACE_BYTES));
    }
    for (int i = 0; i < N; ++i) w[i] = rndf(0.02f);
    CHECK_HIP(hipMemcpy(dw, w, 4 * N, hipMemcpyHostToDevice));
    CHECK_HIP(hipMemset(dm, 0, 4 * N));
    CHECK_HIP(hipMemset(dv, 0, 4 * N));
    CHECK_HIP(hipMemcpy(dsegs, segs, sizeof segs, hipMemcpyHostToDevice));
    for (int j = 0; j < K; ++j) {
        g[j] = malloc(2 * N);
        for (int i = 0; i < N; ++i) {
            float f = rndf(0.01f);
            uint32_t u;
            memcpy(&u, &f, 4);
            g[j][i] = (uint16_t)(u >> 16);
        }
        CHECK_HIP(hipMalloc((void **)&dg[j], 2 * N));
        CHECK_HIP(hipMemcpy(dg[j], g[j], 2 * N, hipMemcpyHostToDevice));
    }
    for (int i = 0; i < N; ++i) {
        float f = widen(g[0][i]);
        for (int j = 1; j < K; ++j) f = f + widen(g[j][i]);
        f = f * hp.grad_scale;
        total += (double)f * (double)f;
    }
    /* two tensors outside the shard: fp32 and, right behind it, bf16 */
    for (int i = 0; i < T0; ++i) {
        x[i] = rndf(0.01f);
        total += (double)x[i] * (double)x[i];
    }
    CHECK_HIP(hipMemcpy(dx, x, 4 * T0, hipMemcpyHostToDevice));
    CHECK_HIP(hipMemcpy(dx + T0, g[0], 2 * T1, hipMemcpyHostToDevice));
    for (int i = 0; i < T1; ++i) total += (double)widen(g[0][i]) * (double)widen(g[0][i]);
    zs_tensor list[2] = {{dx, T0, ZS_DTYPE_FP32, 0}, {dx + T0, T1, ZS_DTYPE_BF16, 0}};
    int64_t np = 0;
    CHECK_ZS(zs_tensor_pieces(list, 2, NULL, 0, &np));
    zs_piece *pieces = malloc(np * sizeof(zs_piece));
    CHECK_ZS(zs_tensor_pieces(list, 2, pieces, np, &np));
    CHECK_HIP(hipMalloc((void **)&dpieces, np * sizeof(zs_piece)));
    CHECK_HIP(hipMemcpy(dpieces, pieces, np * sizeof(zs_piece), hipMemcpyHostToDevice));
    zs_tensor_table tensors = {dpieces, np};

    const uint16_t *const dgs[K] = {dg[0], dg[1], dg[2]};
    const uint16_t *const hgs[K] = {g[0], g[1], g[2]};
    zs_seg_table table = {dsegs, 3, 0};
    zs_step_buffers b = {dw, dm, dv, dp, NULL, NULL, dgs, NULL, NULL};
    CHECK_ZS(zs_grad_norm(dgs, K, N, hp.grad_scale, NULL, &rec[0], ws[0], s));
    CHECK_ZS(zs_tensors_norm(&tensors, NULL, &rec[1], ws[1], s));
    for (int j = 0; j < 2; ++j)
        CHECK_HIP(hipMemcpyAsync(sums + j, &rec[j].sumsq, 8, hipMemcpyDeviceToDevice, s));
    CHECK_ZS(zs_clip_combine(sums, 2, &rule, &rec[0], s));
    CHECK_ZS(zs_shard_step_clipped(ZS_VARIANT_BASE, &b, K, N, &table, &hp, 7, 0, &rec[0], s));
    CHECK_ZS(zs_tensors_clip(&tensors, &rec[0], s));
    CHECK_HIP(hipStreamSynchronize(s));

    zs_clip r;
    CHECK_HIP(hipMemcpy(&r, &rec[0], sizeof r, hipMemcpyDeviceToHost));
    const double norm = sqrt(total), coef = (double)rule.max_norm / (norm + (double)rule.eps);
    int bad = 0;
    /* one rounding to binary32, and the order of a binary64 sum */
    if (!(fabs(r.norm - norm) <= (0x1p-24 + 0x1p-34) * norm)) bad |= 1;
    if (!(fabs(r.coef - coef) <= (0x1p-24 + 0x1p-34) * coef) || !(coef < 1.0)) bad |= 1;
    hp.grad_scale = hp.grad_scale * r.coef;
    if (zs_oracle_shard_step(w, m, v, p, hgs, K, N, segs, 3, &hp, 7) != 0) bad |= 2;
    CHECK_HIP(hipMemcpy(got, dw, 4 * N, hipMemcpyDeviceToHost));
    if (memcmp(got, w, 4 * N)) bad |= 4;
    CHECK_HIP(hipMemcpy(got, dm, 4 * N, hipMemcpyDeviceToHost));
    if (memcmp(got, m, 4 * N)) bad |= 4;
    CHECK_HIP(hipMemcpy(got, dv, 4 * N, hipMemcpyDeviceToHost));
    if (memcmp(got, v, 4 * N)) bad |= 4;
    CHECK_HIP(hipMemcpy(got, dp, 2 * N, hipMemcpyDeviceToHost));
    if (memcmp(got, p, 2 * N)) bad |= 4;
    CHECK_HIP(hipMemcpy(got, dx, 4 * T0, hipMemcpyDeviceToHost));
    for (int i = 0; i < T0; ++i)
        if (got[i] != x[i] * r.coef) bad |= 8;
    CHECK_ZS(zs_fini());
    if (bad) {
        fprintf(stderr, "clipping: wrong (%d): norm %.9g of %.9g, coef %.9g of %.9g\n", bad, r.norm,
                norm, r.coef, coef);
        return 1;
    }
    printf("clipping: equal to the oracle (coef %.6f)\n", r.coef);
    return 0;
}
