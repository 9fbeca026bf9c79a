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

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float widen_bf16(uint16_t x) {
    return __uint_as_float((uint32_t)x << 16);
}

__device__ __forceinline__ float widen_fp16(uint16_t x) {
    return (float)__builtin_bit_cast(_Float16, x);
}

// fp32 to fp16, to nearest even, of a product already rounded to fp32.  Left to
// itself the compiler folds a product and this conversion into v_fma_mixlo_f16
// with an addend of +0, which turns a product of -0 into +0 (and rounds once
// where the definition rounds twice); the empty statement keeps them apart.
__device__ __forceinline__ uint16_t round_fp16(float x) {
    asm("" : "+v"(x));
    return __builtin_bit_cast(uint16_t, (_Float16)x);
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

__device__ __forceinline__ float lo16(uint32_t d) { return __uint_as_float(d << 16); }
__device__ __forceinline__ float hi16(uint32_t d) { return __uint_as_float(d & 0xffff0000u); }

__device__ __forceinline__ float i8_at(uint32_t word, int byte) {
    return (float)(int32_t)(int8_t)(uint8_t)(word >> (8 * byte));
}

template <typename T>
__device__ __forceinline__ T load_once(const T *p) {
    return __builtin_nontemporal_load(p);
}

// Four chains of additions per lane, so that they overlap.
constexpr int kChains = 4;

__device__ __forceinline__ void add_square(double &s, float x) {
    const double d = (double)x;
    s = __builtin_fma(d, d, s);
}

// One 16-byte vector of each partial: 8 bf16 or 16 int8 elements.
template <int K, bool Q8>
struct PartialVectors {
    static constexpr int kElems = Q8 ? 16 : 8;
    u32x4 d[K];
    float scale[Q8 ? K : 1];

    __device__ __forceinline__ void load_from(const NormArgs &a, int64_t v) {
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if constexpr (Q8) {
                d[j] = load_once(reinterpret_cast<const u32x4 *>(a.qgrads[j]) + v);
                scale[j] = a.qscales[j][v * kElems / kQ8Block];
            } else {
                d[j] = load_once(reinterpret_cast<const u32x4 *>(a.grads[j]) + v);
            }
        }
    }
    __device__ __forceinline__ float value(int j, int e) const {
        if constexpr (Q8) return i8_at(d[j][e / 4], e % 4) * scale[j];
        else return (e & 1) ? hi16(d[j][e / 2]) : lo16(d[j][e / 2]);
    }
    // Left fold over the partials, then the scale, as the step forms it.
    __device__ __forceinline__ void add_squares(double (&s)[kChains], float gscale) const {
#pragma clang fp contract(off)
#pragma unroll
        for (int e = 0; e < kElems; ++e) {
            float g = value(0, e);
#pragma unroll
            for (int j = 1; j < K; ++j) g = g + value(j, e);
            add_square(s[e % kChains], g * gscale);
        }
    }
};

// The same for one element.
template <int K, bool Q8>
__device__ __forceinline__ float reduced(const NormArgs &a, int64_t i) {
#pragma clang fp contract(off)
    float g = 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        float x;
        if constexpr (Q8) x = (float)a.qgrads[j][i] * a.qscales[j][i / kQ8Block];
        else x = widen_bf16(a.grads[j][i]);
        g = j == 0 ? x : g + x;
    }
    return g * a.gscale;
}

// Vectors a lane has in flight: about eight 16-byte loads.
template <int K>
constexpr int unroll_for() {
    return K >= 8 ? 1 : 8 / K;
}

template <int K, bool Q8>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const NormArgs a) {
    typedef PartialVectors<K, Q8> Vec;
    constexpr int U = unroll_for<K>();
    const int64_t nv = a.n / Vec::kElems;  // whole vectors
    const int64_t step = (int64_t)gridDim.x * kThreads * U;
    double s[kChains] = {};
    for (int64_t v0 = (int64_t)blockIdx.x * kThreads * U; v0 < nv; v0 += step) {
        const int64_t v = v0 + threadIdx.x;
        Vec x[U];
        if (v0 + kThreads * U <= nv) {
#pragma unroll
            for (int u = 0; u < U; ++u) x[u].load_from(a, v + u * kThreads);
#pragma unroll
            for (int u = 0; u < U; ++u) x[u].add_squares(s, a.gscale);
        } else {
            for (int u = 0; u < U; ++u)
                if (v + u * kThreads < nv) {
                    x[0].load_from(a, v + u * kThreads);
                    x[0].add_squares(s, a.gscale);
                }
        }
    }
    // the elements past the last whole vector
    const int64_t i = nv * Vec::kElems + threadIdx.x;
    if (blockIdx.x == 0 && i < a.n) add_square(s[0], reduced<K, Q8>(a, i));
    const double sum = workgroup_sum((s[0] + s[1]) + (s[2] + s[3]));
    if (threadIdx.x == 0) a.sums[blockIdx.x] = sum;
}

// --------------------------------------------------------------- tensor lists

constexpr int kPieceVectors = kPieceBytes / 16;        // 16-byte vectors of a whole piece
constexpr int kLaneVectors = kPieceVectors / kWave;    // of one lane
static_assert(kLaneVectors == 8, "eight loads in flight per lane");

// The pieces are read as constant memory with a wave-uniform index: scalar loads.
typedef const __attribute__((address_space(4))) zs_piece ConstPiece;

__device__ __forceinline__ zs_piece piece_at(const zs_piece *pieces, int64_t b) {
    ConstPiece *c = (ConstPiece *)pieces + b;
    return {c->addr, c->n, c->dtype};
}

__device__ __forceinline__ float piece_value(const zs_piece &p, uint32_t i) {
    if (p.dtype == ZS_DTYPE_FP32) return reinterpret_cast<const float *>(p.addr)[i];
    const uint16_t x = reinterpret_cast<const uint16_t *>(p.addr)[i];
    return p.dtype == ZS_DTYPE_BF16 ? widen_bf16(x) : widen_fp16(x);
}

__device__ __forceinline__ void piece_store(const zs_piece &p, uint32_t i, float x) {
    if (p.dtype == ZS_DTYPE_FP32) {
        reinterpret_cast<float *>(p.addr)[i] = x;
        return;
    }
    reinterpret_cast<uint16_t *>(p.addr)[i] =
        p.dtype == ZS_DTYPE_BF16 ? round_bf16(x) : round_fp16(x);
}

// A 16-byte vector of a type: elements, widening, and rounding back.
template <uint32_t D>
struct Vec16 {
    static constexpr int kElems = 16 / dtype_size(D);
    __device__ __forceinline__ static float get(const u32x4 &d, int e) {
        if constexpr (D == ZS_DTYPE_FP32) return __uint_as_float(d[e]);
        else if constexpr (D == ZS_DTYPE_BF16) return (e & 1) ? hi16(d[e / 2]) : lo16(d[e / 2]);
        else return widen_fp16((uint16_t)(d[e / 2] >> (16 * (e & 1))));
    }
    __device__ __forceinline__ static void add_squares(double (&s)[kChains], const u32x4 &d) {
#pragma unroll
        for (int e = 0; e < kElems; ++e) add_square(s[e % kChains], get(d, e));
    }
    __device__ __forceinline__ static u32x4 scaled(const u32x4 &d, float c) {
        u32x4 r;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (D == ZS_DTYPE_FP32) {
                r[q] = __float_as_uint(__uint_as_float(d[q]) * c);
            } else if constexpr (D == ZS_DTYPE_BF16) {
                r[q] = (uint32_t)round_bf16(lo16(d[q]) * c) |
                       ((uint32_t)round_bf16(hi16(d[q]) * c) << 16);
            } else {
                r[q] = (uint32_t)round_fp16(get(d, 2 * q) * c) |
                       ((uint32_t)round_fp16(get(d, 2 * q + 1) * c) << 16);
            }
        }
        return r;
    }
};

// Where a piece's 16-byte vectors are: `head` elements before the first of
// them (a tensor may start anywhere), `vectors` of them, then the elements
// from `tail` on.
struct Split {
    uint32_t head, vectors, tail;
};

__device__ __forceinline__ Split split_of(const zs_piece &p) {
    const uint32_t size = dtype_size(p.dtype);
    uint32_t head = (uint32_t)((16 - (p.addr & 15)) & 15) / size;
    head = head < p.n ? head : p.n;
    const uint32_t vectors = (p.n - head) * size / 16;
    return {head, vectors, head + vectors * (16 / size)};
}

__device__ __forceinline__ bool whole(const zs_piece &p) {
    return p.n * dtype_size(p.dtype) == kPieceBytes;  // starts at a multiple of kPieceBytes, too
}

template <uint32_t D>
__device__ __forceinline__ void norm_piece(const zs_piece &p, int lane, double (&s)[kChains]) {
    if (whole(p)) {
        const u32x4 *const v = reinterpret_cast<const u32x4 *>(p.addr) + lane;
        u32x4 d[kLaneVectors];
#pragma unroll
        for (int u = 0; u < kLaneVectors; ++u) d[u] = load_once(v + u * kWave);
#pragma unroll
        for (int u = 0; u < kLaneVectors; ++u) Vec16<D>::add_squares(s, d[u]);
        return;
    }
    const Split sp = split_of(p);
    const u32x4 *const v = reinterpret_cast<const u32x4 *>(p.addr + sp.head * dtype_size(D));
    for (uint32_t u = lane; u < sp.vectors; u += kWave) Vec16<D>::add_squares(s, load_once(v + u));
    if ((uint32_t)lane < sp.head) add_square(s[0], piece_value(p, lane));
    if (sp.tail + lane < p.n) add_square(s[0], piece_value(p, sp.tail + lane));
}

// A wavefront takes every (waves in the grid)-th piece; the next one's
// descriptor is loaded while this one's data is on its way.
template <typename F>
__device__ __forceinline__ void each_piece(const zs_piece *pieces, int64_t count, F f) {
    const int64_t waves = (int64_t)gridDim.x * (kThreads / kWave);
    int64_t b = (int64_t)blockIdx.x * (kThreads / kWave) +
                __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (b >= count) return;
    zs_piece p = piece_at(pieces, b);
    while (true) {
        const int64_t next = b + waves;
        const zs_piece q = piece_at(pieces, next < count ? next : b);
        f(p);
        if (next >= count) return;
        b = next;
        p = q;
    }
}

__global__ __launch_bounds__(kThreads) void tensors_norm_kernel(const zs_piece *pieces,
                                                                int64_t count, double *sums) {
    const int lane = threadIdx.x % kWave;
    double s[kChains] = {};
    each_piece(pieces, count, [&](const zs_piece &p) {
        if (p.dtype == ZS_DTYPE_BF16) norm_piece<ZS_DTYPE_BF16>(p, lane, s);
        else if (p.dtype == ZS_DTYPE_FP16) norm_piece<ZS_DTYPE_FP16>(p, lane, s);
        else norm_piece<ZS_DTYPE_FP32>(p, lane, s);
    });
    const double sum = workgroup_sum((s[0] + s[1]) + (s[2] + s[3]));
    if (threadIdx.x == 0) sums[blockIdx.x] = sum;
}

template <uint32_t D>
__device__ __forceinline__ void clip_piece(const zs_piece &p, int lane, float coef) {
    if (whole(p)) {
        u32x4 *const v = reinterpret_cast<u32x4 *>(p.addr) + lane;
        u32x4 d[kLaneVectors];
#pragma unroll
        for (int u = 0; u < kLaneVectors; ++u) d[u] = load_once(v + u * kWave);
#pragma unroll
        for (int u = 0; u < kLaneVectors; ++u)
            __builtin_nontemporal_store(Vec16<D>::scaled(d[u], coef), v + u * kWave);
        return;
    }
    const Split sp = split_of(p);
    u32x4 *const v = reinterpret_cast<u32x4 *>(p.addr + sp.head * dtype_size(D));
    for (uint32_t u = lane; u < sp.vectors; u += kWave) v[u] = Vec16<D>::scaled(v[u], coef);
    if ((uint32_t)lane < sp.head) piece_store(p, lane, piece_value(p, lane) * coef);
    if (sp.tail + lane < p.n)
        piece_store(p, sp.tail + lane, piece_value(p, sp.tail + lane) * coef);
}

__global__ __launch_bounds__(kThreads) void tensors_clip_kernel(const zs_piece *pieces,
                                                                int64_t count,
                                                                const zs_clip *clip) {
    const float coef = clip->coef;
    if (!clip->apply || coef == 1.0f) return;
    const int lane = threadIdx.x % kWave;
    each_piece(pieces, count, [&](const zs_piece &p) {
        if (p.dtype == ZS_DTYPE_BF16) clip_piece<ZS_DTYPE_BF16>(p, lane, coef);
        else if (p.dtype == ZS_DTYPE_FP16) clip_piece<ZS_DTYPE_FP16>(p, lane, coef);
        else clip_piece<ZS_DTYPE_FP32>(p, lane, coef);
    });
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
