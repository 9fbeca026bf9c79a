// zs_norm.hip -- the global gradient norm and the scaling by its coefficient
// (include/zs.h, "Global gradient norm and clipping") for gfx950.
//
// S is a sum of squares over up to 10^10 elements, read once: bound by HBM.
// Every element is squared and added in binary64.  The square of any fp32
// value is a normal binary64 number, so no scaling is needed, and a sum of
// 10^10 terms keeps about 6 decimal digits more than the fp32 result shows.
// Each lane keeps one sum, a workgroup adds its lanes' in a fixed tree and
// writes one value, and a second launch of one workgroup adds those: no
// atomics, so the order is fixed.

#include "zs_norm.h"

namespace zs_detail {
namespace {

__device__ __forceinline__ float widen_bf16(uint16_t x) {
    return __uint_as_float((uint32_t)x << 16);
}

__device__ __forceinline__ float widen_fp16(uint16_t x) {
    return (float)__builtin_bit_cast(_Float16, x);
}

// fp32 to bf16, to nearest even: every NaN becomes 0x7FC0.
__device__ __forceinline__ uint16_t round_bf16(float x) {
    const uint32_t u = __float_as_uint(x);
    const uint32_t r = (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
    return (uint16_t)(((u & 0x7fffffffu) > 0x7f800000u) ? 0x7fc0u : r);
}

// Sum over a workgroup, in thread 0: a tree over each wavefront's lanes, then
// the wavefronts in order.
__device__ double workgroup_sum(double x) {
    __shared__ double s_wave[kThreads / kWave];
    for (int off = kWave / 2; off >= 1; off >>= 1) x += __shfl_xor(x, off, kWave);
    if (threadIdx.x % kWave == 0) s_wave[threadIdx.x / kWave] = x;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kThreads / kWave; ++w) t += s_wave[w];
    return t;
}

// The reduced gradient of element i, as the step forms it.
template <int K, bool Q8>
__device__ __forceinline__ float reduced(const NormArgs &a, int64_t i) {
#pragma clang fp contract(off)
    float g;
    if constexpr (Q8) {
        const int64_t blk = i / kQ8Block;
        g = (float)a.qgrads[0][i] * a.qscales[0][blk];
#pragma unroll
        for (int j = 1; j < K; ++j) g = g + (float)a.qgrads[j][i] * a.qscales[j][blk];
    } else {
        g = widen_bf16(a.grads[0][i]);
#pragma unroll
        for (int j = 1; j < K; ++j) g = g + widen_bf16(a.grads[j][i]);
    }
    return g * a.gscale;
}

template <int K, bool Q8>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const NormArgs a) {
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    double s = 0.0;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < a.n; i += stride) {
        const double g = (double)reduced<K, Q8>(a, i);
        s += g * g;
    }
    s = workgroup_sum(s);
    if (threadIdx.x == 0) a.sums[blockIdx.x] = s;
}

__device__ __forceinline__ float piece_value(const zs_piece &p, uint32_t i) {
    if (p.dtype == ZS_DTYPE_FP32) return reinterpret_cast<const float *>(p.addr)[i];
    const uint16_t x = reinterpret_cast<const uint16_t *>(p.addr)[i];
    return p.dtype == ZS_DTYPE_BF16 ? widen_bf16(x) : widen_fp16(x);
}

// A wavefront takes every (waves in the grid)-th piece.
__global__ __launch_bounds__(kThreads) void tensors_norm_kernel(const zs_piece *pieces,
                                                                int64_t count, double *sums) {
    const int64_t waves = (int64_t)gridDim.x * (kThreads / kWave);
    double s = 0.0;
    for (int64_t b = (int64_t)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave; b < count;
         b += waves) {
        const zs_piece p = pieces[b];
        for (uint32_t i = threadIdx.x % kWave; i < p.n; i += kWave) {
            const double x = (double)piece_value(p, i);
            s += x * x;
        }
    }
    s = workgroup_sum(s);
    if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void tensors_clip_kernel(const zs_piece *pieces,
                                                                int64_t count,
                                                                const zs_clip *clip) {
    const float coef = clip->coef;
    if (!clip->apply || coef == 1.0f) return;
    const int64_t waves = (int64_t)gridDim.x * (kThreads / kWave);
    for (int64_t b = (int64_t)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave; b < count;
         b += waves) {
        const zs_piece p = pieces[b];
        for (uint32_t i = threadIdx.x % kWave; i < p.n; i += kWave) {
            const float x = piece_value(p, i) * coef;
            if (p.dtype == ZS_DTYPE_FP32) {
                reinterpret_cast<float *>(p.addr)[i] = x;
            } else {
                reinterpret_cast<uint16_t *>(p.addr)[i] =
                    p.dtype == ZS_DTYPE_BF16 ? round_bf16(x)
                                             : __builtin_bit_cast(uint16_t, (_Float16)x);
            }
        }
    }
}

// The record of the sum S (one thread).
__device__ void write_record(double s, const Rule &r, zs_clip *clip) {
#pragma clang fp contract(off)
    const double norm = sqrt(s);
    const double d = norm + (double)r.eps;
    const float f = (float)norm;
    clip->sumsq = s;
    clip->norm = f;
    clip->coef = d <= (double)r.max_norm ? 1.0f : (float)((double)r.max_norm / d);
    clip->apply = (r.skip_nonfinite && !__builtin_isfinite(f)) ? 0 : 1;
    clip->reserved = 0;
}

__global__ __launch_bounds__(kThreads) void finish_kernel(const double *sums, int count, Rule rule,
                                                          zs_clip *clip) {
    double s = 0.0;
    for (int i = threadIdx.x; i < count; i += kThreads) s += sums[i];
    s = workgroup_sum(s);  // its barrier also puts every read of sums before the record
    if (threadIdx.x == 0) write_record(s, rule, clip);
}

}  // namespace

template <int K>
static const void *norm_kernel(bool q8) {
    return q8 ? (const void *)grad_norm_kernel<K, true> : (const void *)grad_norm_kernel<K, false>;
}

hipError_t launch_grad_norm(int k, bool q8, const NormArgs &a, int blocks, hipStream_t stream) {
    const void *fn = nullptr;
    switch (k) {
        case 1: fn = norm_kernel<1>(q8); break;
        case 2: fn = norm_kernel<2>(q8); break;
        case 3: fn = norm_kernel<3>(q8); break;
        case 4: fn = norm_kernel<4>(q8); break;
        case 5: fn = norm_kernel<5>(q8); break;
        case 6: fn = norm_kernel<6>(q8); break;
        case 7: fn = norm_kernel<7>(q8); break;
        case 8: fn = norm_kernel<8>(q8); break;
        case 9: fn = norm_kernel<9>(q8); break;
        case 10: fn = norm_kernel<10>(q8); break;
        case 11: fn = norm_kernel<11>(q8); break;
        case 12: fn = norm_kernel<12>(q8); break;
        case 13: fn = norm_kernel<13>(q8); break;
        case 14: fn = norm_kernel<14>(q8); break;
        case 15: fn = norm_kernel<15>(q8); break;
        case 16: fn = norm_kernel<16>(q8); break;
        default: return hipErrorInvalidValue;
    }
    NormArgs args = a;
    void *argv[] = {&args};
    return hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(kThreads), argv, 0, stream);
}

hipError_t launch_tensors_norm(const zs_piece *pieces, int64_t count, double *sums, int blocks,
                               hipStream_t stream) {
    void *argv[] = {&pieces, &count, &sums};
    return hipLaunchKernel((const void *)tensors_norm_kernel, dim3((unsigned)blocks),
                           dim3(kThreads), argv, 0, stream);
}

hipError_t launch_tensors_clip(const zs_piece *pieces, int64_t count, const zs_clip *clip,
                               int blocks, hipStream_t stream) {
    void *argv[] = {&pieces, &count, &clip};
    return hipLaunchKernel((const void *)tensors_clip_kernel, dim3((unsigned)blocks),
                           dim3(kThreads), argv, 0, stream);
}

hipError_t launch_finish(const double *sums, int count, const Rule &rule, zs_clip *clip,
                         hipStream_t stream) {
    Rule r = rule;
    void *argv[] = {&sums, &count, &r, &clip};
    return hipLaunchKernel((const void *)finish_kernel, dim3(1), dim3(kThreads), argv, 0, stream);
}

}  // namespace zs_detail
