// zs_norm.h -- what the C ABI layer (zs_api.hip) and the norm and scaling
// kernels (zs_norm.hip) share.  Private to the library.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "zs.h"
#include "zs_kernels.h"

namespace zs_detail {

// A piece is at most kPieceBytes of one tensor, between two multiples of
// kPieceBytes in memory: only a tensor's first piece can start unaligned and
// only its last can be short.
constexpr int64_t kPieceBytes = 8192;
constexpr int64_t kMaxSums = ZS_NORM_WORKSPACE_BYTES / 8;  // workgroups of a norm call

__host__ __device__ constexpr int dtype_size(uint32_t dtype) {
    return dtype == ZS_DTYPE_FP32 ? 4 : 2;
}

// The clipping rule as the kernels take it.
struct Rule {
    float max_norm, eps;
    int32_t skip_nonfinite;
};

struct NormArgs {
    const uint16_t *grads[ZS_MAX_K];
    const int8_t *qgrads[ZS_MAX_K];
    const float *qscales[ZS_MAX_K];
    int64_t n;
    float gscale;
    double *sums;  // one per workgroup
};

// Each launches on `stream`; `blocks` workgroups of kThreads.
hipError_t launch_grad_norm(int k, bool q8, const NormArgs &a, int blocks, hipStream_t stream);
hipError_t launch_tensors_norm(const zs_piece *pieces, int64_t count, double *sums, int blocks,
                               hipStream_t stream);
hipError_t launch_tensors_clip(const zs_piece *pieces, int64_t count, const zs_clip *clip,
                               int blocks, hipStream_t stream);
// S = sums[0] + ... + sums[count - 1] and the record of it: one workgroup.
hipError_t launch_finish(const double *sums, int count, const Rule &rule, zs_clip *clip,
                         hipStream_t stream);

}  // namespace zs_detail
