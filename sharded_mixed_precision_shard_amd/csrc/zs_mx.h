// zs_mx.h -- what the C ABI layer (zs_mx_api.hip) and the kernels (zs_mx.hip)
// of the microscaled formats share.  Private to the library.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "zs.h"
#include "zs_kernels.h"

namespace zs_detail {

// The device the library runs on: zs_api.hip checks that it is prepared.
struct MxDevice {
    int cus;
};
int mx_device(MxDevice *out);
int mx_launched(hipError_t e);  // ZS_OK, or ZS_ERR_DEVICE with the error recorded

constexpr int kMxBlock = ZS_MX_BLOCK;

constexpr int64_t mx_blocks(int64_t cols) { return (cols + kMxBlock - 1) / kMxBlock; }
constexpr int64_t mx_block_bytes(int format) { return format == ZS_MX_FP4 ? 16 : 32; }

// Quantisation and dequantisation: `blocks` blocks, nb of them to a row of
// cols elements, rows ld elements apart.
struct MxCastArgs {
    void *x;
    uint8_t *codes;
    uint8_t *scales;
    int64_t blocks, nb, cols, ld;
};

// A product out[I, J] = sum over c < C of P[i, c] Q[j, c].
struct MxHeld {
    const uint8_t *codes;
    const uint8_t *scales;
    int64_t nb;  // blocks of a stored row
};
enum MxLeft { kLeftRows, kLeftCols, kLeftFp4, kLeftFp8 };  // bf16 P[i][c], bf16 P[c][i], blocks
enum MxRight { kRightFp4 = 0, kRightFp8 = 1, kRightCols = 2 };  // Q[j][c], + kRightCols: Q[c][j]

struct MxProductArgs {
    const uint16_t *p;
    int64_t ldp;
    MxHeld px, q;
    void *out;
    int64_t ldo;
    int32_t I, J, C;
    int32_t out_f32, add;
    int32_t tiles_i, tiles_j;
    int32_t splits, split_steps;  // a split takes split_steps steps over c
    float *parts;                 // [tile][split][BI * BJ]
    uint32_t *counters;           // one per tile, 0 between calls
};

// Whether 32-bit offsets below 2^31 reach `rows` rows that lie ld bf16 elements apart.  ld may
// be anything up to 2^59, as that of a single row.
constexpr int64_t kMxReach = int64_t(1) << 31;
constexpr bool mx_rows_reach(int64_t ld, int64_t rows) { return ld < kMxReach / (2 * rows); }

constexpr int64_t kMxCounterBytes = 65536;
constexpr int64_t kMxCounters = kMxCounterBytes / 4;
constexpr int64_t kMxPartBytes = ZS_MX_WORKSPACE_BYTES - kMxCounterBytes;

hipError_t launch_mx_quantize(int format, int dtype, const MxCastArgs &a, hipStream_t stream);
hipError_t launch_mx_dequantize(int format, int dtype, const MxCastArgs &a, hipStream_t stream);
// Chooses the kernel and its tile; `workspace` may be null.
hipError_t launch_mx_product(MxLeft left, int right, MxProductArgs a, void *workspace,
                             const MxDevice &dev, hipStream_t stream);

}  // namespace zs_detail
