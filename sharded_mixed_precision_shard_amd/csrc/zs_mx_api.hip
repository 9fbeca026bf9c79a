// zs_mx_api.hip -- the C ABI of the microscaled formats (include/zs.h):
// argument checks and launches.  Errors are found on the host before anything
// is enqueued; the library allocates nothing and keeps no pointer.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "zs.h"
#include "zs_mx.h"

namespace {

using namespace zs_detail;

constexpr int64_t kMaxDim = int64_t(1) << 28;      // of a product
constexpr int64_t kMaxOut = int64_t(1) << 36;      // elements a product writes
constexpr int64_t kMaxBlocksCast = (int64_t(1) << 32) - 1;  // blocks one call casts

struct Range {
    uintptr_t a, b;
};

bool meet(const Range &x, const Range &y) { return x.a < y.b && y.a < x.b; }

// Bytes [a, b) that a matrix spans; false where its arguments are no matrix.
bool matrix_range(const zs_matrix *x, bool fp16, int *status, Range *out) {
    *status = ZS_ERR_INVALID_ARGUMENT;
    if (!x || x->reserved != 0 || x->rows < 0 || x->cols < 0 || x->ld < x->cols) return false;
    if (x->dtype != ZS_DTYPE_BF16 && x->dtype != ZS_DTYPE_FP32 &&
        !(fp16 && x->dtype == ZS_DTYPE_FP16))
        return false;
    *out = {0, 0};
    if (x->rows == 0 || x->cols == 0) return true;
    if (!x->data) return false;
    const int64_t size = x->dtype == ZS_DTYPE_FP32 ? 4 : 2;
    if (x->ld > (INT64_MAX / 16 - x->cols) / x->rows) return false;
    const uint64_t bytes = (uint64_t)((x->rows - 1) * x->ld + x->cols) * (uint64_t)size;
    const uintptr_t at = (uintptr_t)x->data;
    if (at > UINTPTR_MAX - bytes) return false;
    if (at % (uintptr_t)size) {
        *status = ZS_ERR_MISALIGNED;
        return false;
    }
    *out = {at, at + (uintptr_t)bytes};
    return true;
}

bool held_range(const zs_mx *x, int *status, Range *codes, Range *scales) {
    *status = ZS_ERR_INVALID_ARGUMENT;
    if (!x || x->reserved != 0 || x->rows < 0 || x->cols < 0) return false;
    if (x->format != ZS_MX_FP4 && x->format != ZS_MX_FP8) return false;
    *codes = *scales = {0, 0};
    if (x->rows == 0 || x->cols == 0) return true;
    if (!x->codes || !x->scales) return false;
    if (x->cols > INT64_MAX / 64) return false;
    const int64_t nb = mx_blocks(x->cols);
    if (nb > INT64_MAX / 64 / x->rows) return false;
    const uint64_t blocks = (uint64_t)(nb * x->rows);
    const uint64_t bytes = blocks * (uint64_t)mx_block_bytes(x->format);
    const uintptr_t c = (uintptr_t)x->codes, s = (uintptr_t)x->scales;
    if (c > UINTPTR_MAX - bytes || s > UINTPTR_MAX - blocks) return false;
    if (c % 16) {
        *status = ZS_ERR_MISALIGNED;
        return false;
    }
    *codes = {c, c + (uintptr_t)bytes};
    *scales = {s, s + (uintptr_t)blocks};
    return true;
}

// Arguments of a cast either way; sets `blocks` to 0 where there is nothing to do.
int cast_args(const zs_matrix *x, const zs_mx *q, bool out_codes, MxCastArgs *a) {
    int st;
    Range m, c, s;
    if (!matrix_range(x, true, &st, &m) || !held_range(q, &st, &c, &s)) return st;
    if (x->rows != q->rows || x->cols != q->cols) return ZS_ERR_INVALID_ARGUMENT;
    if (meet(m, c) || meet(m, s) || (out_codes && meet(c, s))) return ZS_ERR_ALIASING;
    a->x = x->data;
    a->codes = q->codes;
    a->scales = q->scales;
    a->cols = x->cols;
    a->ld = x->ld;
    a->nb = mx_blocks(x->cols);
    a->blocks = x->rows > 0 ? a->nb * x->rows : 0;
    if (a->blocks > kMaxBlocksCast) return ZS_ERR_INVALID_ARGUMENT;
    if (x->ld == x->cols && x->cols % kMxBlock == 0) {  // one long row
        a->cols = x->cols * x->rows;
        a->nb = a->blocks;
    }
    return ZS_OK;
}

// One product: P either a bf16 matrix or in blocks, Q in blocks.
int product(MxLeft left, const zs_matrix *p, const zs_mx *px, const zs_mx *q, bool q_cols,
            const zs_matrix *out, int add, void *workspace, void *stream) {
    int st;
    Range rp = {0, 0}, rps = {0, 0}, rq, rqs, ro;
    if (px ? !held_range(px, &st, &rp, &rps) : !matrix_range(p, false, &st, &rp)) return st;
    if (!px && p->dtype != ZS_DTYPE_BF16) return ZS_ERR_INVALID_ARGUMENT;
    if (!held_range(q, &st, &rq, &rqs) || !matrix_range(out, false, &st, &ro)) return st;
    const int64_t p_rows = px ? px->rows : p->rows, p_cols = px ? px->cols : p->cols;
    const int64_t I = left == kLeftCols ? p_cols : p_rows;
    const int64_t C = left == kLeftCols ? p_rows : p_cols;
    const int64_t J = q_cols ? q->cols : q->rows;
    if ((q_cols ? q->rows : q->cols) != C || out->rows != I || out->cols != J)
        return ZS_ERR_INVALID_ARGUMENT;
    if (I > kMaxDim || J > kMaxDim || C > kMaxDim) return ZS_ERR_INVALID_ARGUMENT;
    if (I > 0 && J > kMaxOut / I) return ZS_ERR_INVALID_ARGUMENT;
    if (add != 0 && add != 1) return ZS_ERR_INVALID_ARGUMENT;
    if (add && out->dtype != ZS_DTYPE_FP32) return ZS_ERR_INVALID_ARGUMENT;
    if (meet(ro, rp) || meet(ro, rps) || meet(ro, rq) || meet(ro, rqs)) return ZS_ERR_ALIASING;
    if (workspace) {
        const uintptr_t w = (uintptr_t)workspace;
        if (w % 16) return ZS_ERR_MISALIGNED;
        if (w > UINTPTR_MAX - ZS_MX_WORKSPACE_BYTES) return ZS_ERR_INVALID_ARGUMENT;
        const Range rw = {w, w + ZS_MX_WORKSPACE_BYTES};
        if (meet(rw, ro) || meet(rw, rp) || meet(rw, rps) || meet(rw, rq) || meet(rw, rqs))
            return ZS_ERR_ALIASING;
    }
    MxDevice dev;
    st = mx_device(&dev);
    if (st != ZS_OK) return st;
    if (I == 0 || J == 0 || (add && C == 0)) return ZS_OK;
    MxProductArgs a = {};
    if (px) {
        a.px = {px->codes, px->scales, mx_blocks(px->cols)};
    } else {
        a.p = (const uint16_t *)p->data;
        a.ldp = p->ld;
    }
    a.q = {q->codes, q->scales, mx_blocks(q->cols)};
    a.out = out->data;
    a.ldo = out->ld;
    a.I = (int32_t)I;
    a.J = (int32_t)J;
    a.C = (int32_t)C;
    a.out_f32 = out->dtype == ZS_DTYPE_FP32;
    a.add = add;
    const int right = (q->format == ZS_MX_FP8 ? kRightFp8 : kRightFp4) | (q_cols ? kRightCols : 0);
    return mx_launched(launch_mx_product(left, right, a, workspace, dev, (hipStream_t)stream));
}

}  // namespace

extern "C" {

int zs_mx_quantize(const zs_matrix *x, const zs_mx *out, void *stream) {
    MxCastArgs a;
    int st = cast_args(x, out, true, &a);
    if (st != ZS_OK) return st;
    MxDevice dev;
    st = mx_device(&dev);
    if (st != ZS_OK || a.blocks == 0) return st;
    return mx_launched(launch_mx_quantize(out->format, x->dtype, a, (hipStream_t)stream));
}

int zs_mx_dequantize(const zs_mx *x, const zs_matrix *out, void *stream) {
    MxCastArgs a;
    int st = cast_args(out, x, false, &a);
    if (st != ZS_OK) return st;
    MxDevice dev;
    st = mx_device(&dev);
    if (st != ZS_OK || a.blocks == 0) return st;
    return mx_launched(launch_mx_dequantize(x->format, out->dtype, a, (hipStream_t)stream));
}

int zs_mx_linear(const zs_matrix *x, const zs_mx *w, const zs_matrix *y, void *workspace,
                 void *stream) {
    return product(kLeftRows, x, nullptr, w, false, y, 0, workspace, stream);
}

int zs_mx_product(const zs_mx *x, const zs_mx *w, const zs_matrix *y, void *workspace,
                  void *stream) {
    if (!x) return ZS_ERR_INVALID_ARGUMENT;
    return product(x->format == ZS_MX_FP8 ? kLeftFp8 : kLeftFp4, nullptr, x, w, false, y, 0,
                   workspace, stream);
}

int zs_mx_linear_dgrad(const zs_matrix *dy, const zs_mx *w, const zs_matrix *dx, void *workspace,
                       void *stream) {
    return product(kLeftRows, dy, nullptr, w, true, dx, 0, workspace, stream);
}

int zs_mx_linear_wgrad(const zs_matrix *dy, const zs_mx *x, const zs_matrix *dw, int add,
                       void *workspace, void *stream) {
    return product(kLeftCols, dy, nullptr, x, true, dw, add, workspace, stream);
}

}  // extern "C"
