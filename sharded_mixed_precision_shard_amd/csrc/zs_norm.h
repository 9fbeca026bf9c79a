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

// The workspace: 1 + kCounters arrival counters a cache line apart (0 between
// calls), then one sum per workgroup.
constexpr uint32_t kCounters = 32;
constexpr uint32_t kOneCounter = 64;     // workgroups that use the first counter alone
constexpr uint32_t kCounterStride = 32;  // of 4 bytes
constexpr int64_t kCounterBytes = (1 + kCounters) * kCounterStride * 4;
constexpr int64_t kMaxSums = (ZS_NORM_WORKSPACE_BYTES - kCounterBytes) / 8;
static_assert(kOneCounter >= kCounters, "every counter has an arrival");

constexpr int kGroup = kThreads / kWave;  // pieces a norm workgroup takes at a time

__host__ __device__ constexpr int dtype_size(uint32_t dtype) {
    return dtype == ZS_DTYPE_FP32 ? 4 : 2;
}

// The clipping rule as the kernels take it.
struct Rule {
    float max_norm, eps;
    int32_t skip_nonfinite;
};

// How a norm call ends.
struct FinishArgs {
    double *sums;  // one per workgroup
    uint32_t *counters;
    zs_clip *clip;
    Rule rule;
};

struct NormArgs {
    const uint16_t *grads[ZS_MAX_K];
    const int8_t *qgrads[ZS_MAX_K];
    const float *qscales[ZS_MAX_K];
    int64_t n;
    float gscale;
    int32_t xcds;  // XCDs that get a contiguous run each; 1 = linear order
    int64_t kept;  // tiles at the beginning of each run that are read with ordinary loads
    FinishArgs fin;
};

// Elements of a workgroup's tile in the norm kernel of k partials: 256 lanes
// with about eight 16-byte loads in flight each.
constexpr int norm_unroll(int k) { return k >= 8 ? 1 : 8 / k; }
constexpr int64_t norm_tile(int k, bool q8) {
    return (int64_t)kThreads * norm_unroll(k) * (q8 ? 16 : 8);
}

// Each launches on `stream`; `blocks` workgroups of kThreads, at most kMaxSums.
hipError_t launch_grad_norm(int k, bool q8, const NormArgs &a, int blocks, hipStream_t stream);
hipError_t launch_tensors_norm(const zs_piece *pieces, int64_t count, int64_t kept,
                               const FinishArgs &fin, int blocks, hipStream_t stream);
// One workgroup per piece, at most kMaxBlocks; `lds` bytes of LDS reserved by
// each cap how many a compute unit holds.
hipError_t launch_tensors_clip(const zs_piece *pieces, int64_t count, const zs_clip *clip,
                               int64_t blocks, size_t lds, hipStream_t stream);
// S = sums[0] + ... + sums[count - 1] and the record of it: one workgroup.
hipError_t launch_finish(const double *sums, int count, const Rule &rule, zs_clip *clip,
                         hipStream_t stream);

}  // namespace zs_detail
