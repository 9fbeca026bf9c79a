// zs_norm.hip -- the global gradient norm and the scaling by its coefficient
// (include/zs.h, "Global gradient norm and clipping") for gfx950.
//
// S is a sum of squares over up to 10^10 elements, read once: bound by HBM.
// Every element is squared and added in binary64.  The square of any fp32
// value is a normal binary64 number, so no scaling is needed, and a sum of
// 10^10 terms keeps about 6 decimal digits more than the fp32 result shows.
// Each lane keeps a few sums, a workgroup adds its lanes' in a fixed tree and
// writes one value, and the workgroup that finishes last adds those in the
// order of their indices: one launch, and an order that does not depend on
// which workgroup is last.

#include <type_traits>

#include "zs_norm.h"

namespace zs_detail {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float widen_bf16(uint16_t x) { return bf16_lo(x); }

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
    __syncthreads();  // s_wave may be written again
    return t;
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

// One more arrival at a counter of `size`: whether it is the last, which sets
// the counter back to 0.
__device__ __forceinline__ bool last_of(uint32_t *counter, uint32_t size) {
    const uint32_t before =
        __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (before != size - 1) return false;
    __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

// A norm call's end, for every workgroup: its sum goes to the workspace, and
// the workgroup that arrives last adds all of them and writes the record.  No
// workgroup waits for another.
//
// The workgroups sit on XCDs whose L2 caches do not see each other's writes,
// so the sums are written and read by agent-scope atomics, which go past those
// caches, and a workgroup arrives only when its own has been acknowledged (the
// wait).  Acquire and release on the arrivals would say the same at the price
// of an L2 write-back and an invalidation per workgroup, which no other data
// here needs: an empty kernel of 1024 workgroups with one counter took 24.7 us
// that way and 14.8 this way (2048: 52 and 27).  The rest is the arrivals' taking
// turns at one address, about 12 ns each, so a large grid arrives at kCounters
// counters and their last arrivals at one more: 4.3 us (2048: 5.6), where the
// empty kernel alone takes 1.7 and a second launch would add about 3.5 (and 2.5 us
// on the host).  Up to kOneCounter workgroups one counter is faster (64: 3.0
// against 3.2 us).
__device__ void finish(double s, const FinishArgs &f) {
    __shared__ int s_last;
    s = workgroup_sum(s);
    if (gridDim.x == 1) {
        if (threadIdx.x == 0) write_record(s, f.rule, f.clip);
        return;
    }
    if (threadIdx.x == 0) {
        __hip_atomic_store(f.sums + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const uint32_t n = gridDim.x, g = blockIdx.x % kCounters;
        if (n <= kOneCounter)
            s_last = last_of(f.counters, n);
        else
            s_last = last_of(f.counters + (1 + g) * kCounterStride,
                             n / kCounters + (g < n % kCounters ? 1 : 0)) &&
                     last_of(f.counters, kCounters);
    }
    __syncthreads();
    if (!s_last) return;
    double t = 0.0;
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += kThreads)
        t += __hip_atomic_load(f.sums + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    t = workgroup_sum(t);
    if (threadIdx.x == 0) write_record(t, f.rule, f.clip);
}

// Keep: an ordinary load, which leaves the line in the last-level cache;
// otherwise a streaming one, which does not displace what is there.
template <bool Keep, typename P>
__device__ __forceinline__ u32x4 load(P p) {
    if constexpr (Keep) return *p;
    else return __builtin_nontemporal_load(p);
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

    template <bool Keep>
    __device__ __forceinline__ void load_from(const NormArgs &a, int64_t v) {
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if constexpr (Q8) {
                d[j] = load<Keep>(reinterpret_cast<const u32x4 *>(a.qgrads[j]) + v);
                scale[j] = a.qscales[j][v * kElems / kQ8Block];
            } else {
                d[j] = load<Keep>(reinterpret_cast<const u32x4 *>(a.grads[j]) + v);
            }
        }
    }
    __device__ __forceinline__ float value(int j, int e) const {
        if constexpr (Q8) return i8_at(d[j][e / 4], e % 4) * scale[j];
        else return (e & 1) ? bf16_hi(d[j][e / 2]) : bf16_lo(d[j][e / 2]);
    }
    // Left fold over the partials, then the scale, as the step forms it.
    template <bool Scaled>
    __device__ __forceinline__ void add_squares(double (&s)[kChains], float gscale) const {
#pragma clang fp contract(off)
#pragma unroll
        for (int e = 0; e < kElems; ++e) {
            float g = value(0, e);
#pragma unroll
            for (int j = 1; j < K; ++j) g = g + value(j, e);
            add_square(s[e % kChains], Scaled ? g * gscale : g);
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

// The units begin + y, begin + y + stride, ... below `end` that this workgroup
// takes of `count`.  One XCD: every (grid size)-th unit.  More: the dispatcher
// deals workgroup b to XCD b % xcds, and each XCD is given one contiguous run
// of the units, which its workgroups take in turn, so that each L2 reads a
// stream of its own.
struct Share {
    int64_t begin, end, stride, y;
};

__device__ __forceinline__ Share share_of(int64_t count, int xcds) {
    if (xcds <= 1) return {0, count, (int64_t)gridDim.x, (int64_t)blockIdx.x};
    const int64_t x = blockIdx.x % xcds, y = blockIdx.x / xcds;
    const int64_t q = count / xcds, r = count % xcds;
    const int64_t begin = x * q + (x < r ? x : r);
    const int64_t groups = gridDim.x / xcds + (x < gridDim.x % xcds ? 1 : 0);
    return {begin, begin + q + (x < r ? 1 : 0), groups, y};
}

// f(unit, keep) for the units of a share from the last to the first, keep being
// true_type for the last `kept` of them to be read, those at the run's beginning.
// What reads the data next (the step, the scaling) starts there and finds them
// in the last-level cache.
template <typename F>
__device__ __forceinline__ void each_backwards(const Share &s, int64_t kept, F f) {
    const int64_t mid = s.begin + kept < s.end ? s.begin + kept : s.end;
    int64_t t = s.end - 1 - s.y;
    for (; t >= mid; t -= s.stride) f(t, std::false_type());
    for (; t >= s.begin; t -= s.stride) f(t, std::true_type());
}

// Scaled: with the product by grad_scale; g * 1 = g, so it may be left out where
// that is 1.  The int8 kernels have a form without it: with few partials they are
// as near the VALU's limit as HBM's, and the product is one of five operations per
// element.  2.4 GB, without and with it: one partial 393 and 443 us, two 371 and
// 381, three to seven 0.4-1.5 % apart, eight and more 0.1-0.6 %.  The bf16 kernels
// always multiply: at every k from 1 to 16 both took the same time (2.4 GB: 342-353
// us, 0.4 % apart at most and either way; 200 MB: 32-34 us).
template <int K, bool Q8, bool Scaled>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const NormArgs a) {
    typedef PartialVectors<K, Q8> Vec;
    constexpr int U = norm_unroll(K);
    constexpr int kTileVectors = kThreads * U;
    static_assert(kTileVectors * Vec::kElems == norm_tile(K, Q8), "the grid counts these tiles");
    const int64_t nv = a.n / Vec::kElems;  // whole vectors
    const Share share = share_of((nv + kTileVectors - 1) / kTileVectors, a.xcds);
    double s[kChains] = {};
    each_backwards(share, a.kept, [&](int64_t t, auto keep) {
        constexpr bool kKeep = decltype(keep)::value;
        const int64_t v = t * kTileVectors + threadIdx.x;
        Vec x[U];
        if ((t + 1) * kTileVectors <= nv) {
#pragma unroll
            for (int u = 0; u < U; ++u) x[u].template load_from<kKeep>(a, v + u * kThreads);
#pragma unroll
            for (int u = 0; u < U; ++u) x[u].template add_squares<Scaled>(s, a.gscale);
        } else {
            for (int u = 0; u < U; ++u)
                if (v + u * kThreads < nv) {
                    x[0].template load_from<kKeep>(a, v + u * kThreads);
                    x[0].template add_squares<Scaled>(s, a.gscale);
                }
        }
    });
    // the elements past the last whole vector
    const int64_t i = nv * Vec::kElems + threadIdx.x;
    if (blockIdx.x == 0 && i < a.n) add_square(s[0], reduced<K, Q8>(a, i));
    finish((s[0] + s[1]) + (s[2] + s[3]), a.fin);
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

// An address from a descriptor as a pointer to global memory: the compiler
// cannot tell by itself and would take flat loads and stores.
template <typename T>
using Global = __attribute__((address_space(1))) T;

template <typename T>
__device__ __forceinline__ Global<T> *global_at(uint64_t addr) {
    return reinterpret_cast<Global<T> *>(addr);
}

__device__ __forceinline__ float piece_value(const zs_piece &p, uint32_t i) {
    if (p.dtype == ZS_DTYPE_FP32) return global_at<const float>(p.addr)[i];
    const uint16_t x = global_at<const uint16_t>(p.addr)[i];
    return p.dtype == ZS_DTYPE_BF16 ? widen_bf16(x) : widen_fp16(x);
}

__device__ __forceinline__ void piece_store(const zs_piece &p, uint32_t i, float x) {
    if (p.dtype == ZS_DTYPE_FP32) {
        global_at<float>(p.addr)[i] = x;
        return;
    }
    global_at<uint16_t>(p.addr)[i] =
        p.dtype == ZS_DTYPE_BF16 ? (uint16_t)to_bf16(x) : round_fp16(x);
}

// A 16-byte vector of a type: elements, widening, and rounding back.
template <uint32_t D>
struct Vec16 {
    static constexpr int kElems = 16 / dtype_size(D);
    __device__ __forceinline__ static float get(const u32x4 &d, int e) {
        if constexpr (D == ZS_DTYPE_FP32) return __uint_as_float(d[e]);
        else if constexpr (D == ZS_DTYPE_BF16) return (e & 1) ? bf16_hi(d[e / 2]) : bf16_lo(d[e / 2]);
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
                r[q] = pack_bf16x2(bf16_lo(d[q]) * c, bf16_hi(d[q]) * c);
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

template <uint32_t D, bool Keep>
__device__ __forceinline__ void norm_piece(const zs_piece &p, int lane, double (&s)[kChains]) {
    if (whole(p)) {
        const Global<u32x4> *const v = global_at<u32x4>(p.addr) + lane;
        u32x4 d[kLaneVectors];
#pragma unroll
        for (int u = 0; u < kLaneVectors; ++u) d[u] = load<Keep>(v + u * kWave);
#pragma unroll
        for (int u = 0; u < kLaneVectors; ++u) Vec16<D>::add_squares(s, d[u]);
        return;
    }
    const Split sp = split_of(p);
    const Global<u32x4> *const v = global_at<u32x4>(p.addr + sp.head * dtype_size(D));
    for (uint32_t u = lane; u < sp.vectors; u += kWave) Vec16<D>::add_squares(s, load<true>(v + u));
    if ((uint32_t)lane < sp.head) add_square(s[0], piece_value(p, lane));
    if (sp.tail + lane < p.n) add_square(s[0], piece_value(p, sp.tail + lane));
}

// A workgroup's share is of groups of kGroup consecutive pieces, one piece for
// each of its wavefronts.
__global__ __launch_bounds__(kThreads) void tensors_norm_kernel(const zs_piece *pieces,
                                                                int64_t count, int64_t kept,
                                                                FinishArgs fin) {
    const int lane = threadIdx.x % kWave;
    double s[kChains] = {};
    each_backwards(share_of((count + kGroup - 1) / kGroup, 1), kept, [&](int64_t t, auto keep) {
        constexpr bool kKeep = decltype(keep)::value;
        const int64_t b = t * kGroup + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        if (b >= count) return;
        const zs_piece p = piece_at(pieces, b);
        if (p.dtype == ZS_DTYPE_BF16) norm_piece<ZS_DTYPE_BF16, kKeep>(p, lane, s);
        else if (p.dtype == ZS_DTYPE_FP16) norm_piece<ZS_DTYPE_FP16, kKeep>(p, lane, s);
        else norm_piece<ZS_DTYPE_FP32, kKeep>(p, lane, s);
    });
    finish((s[0] + s[1]) + (s[2] + s[3]), fin);
}

// One piece, by a whole workgroup: two vectors per lane.
template <uint32_t D>
__device__ __forceinline__ void clip_piece(const zs_piece &p, float coef) {
    const uint32_t tid = threadIdx.x;
    if (whole(p)) {
        Global<u32x4> *const v = global_at<u32x4>(p.addr) + tid;
        constexpr int kEach = kPieceVectors / kThreads;
        u32x4 d[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) d[u] = load<false>(v + u * kThreads);
#pragma unroll
        for (int u = 0; u < kEach; ++u)
            __builtin_nontemporal_store(Vec16<D>::scaled(d[u], coef), v + u * kThreads);
        return;
    }
    const Split sp = split_of(p);
    Global<u32x4> *const v = global_at<u32x4>(p.addr + sp.head * dtype_size(D));
    for (uint32_t u = tid; u < sp.vectors; u += kThreads) v[u] = Vec16<D>::scaled(load<true>(v + u), coef);
    if (tid < sp.head) piece_store(p, tid, piece_value(p, tid) * coef);
    if (sp.tail + tid < p.n) piece_store(p, sp.tail + tid, piece_value(p, sp.tail + tid) * coef);
}

// A workgroup takes one piece (more only where the grid cannot describe them
// all).
__global__ __launch_bounds__(kThreads) void tensors_clip_kernel(const zs_piece *pieces,
                                                                int64_t count,
                                                                const zs_clip *clip) {
    const ConstClip *const c = (const ConstClip *)clip;
    const float coef = c->coef;
    if (!c->apply || coef == 1.0f) return;
    for (int64_t b = blockIdx.x; b < count; b += gridDim.x) {
        const zs_piece p = piece_at(pieces, b);
        if (p.dtype == ZS_DTYPE_BF16) clip_piece<ZS_DTYPE_BF16>(p, coef);
        else if (p.dtype == ZS_DTYPE_FP16) clip_piece<ZS_DTYPE_FP16>(p, coef);
        else clip_piece<ZS_DTYPE_FP32>(p, coef);
    }
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
static const void *norm_kernel(bool q8, bool scaled) {
    if (!q8) return (const void *)grad_norm_kernel<K, false, true>;
    return scaled ? (const void *)grad_norm_kernel<K, true, true>
                  : (const void *)grad_norm_kernel<K, true, false>;
}

hipError_t launch_grad_norm(int k, bool q8, const NormArgs &a, int blocks, hipStream_t stream) {
    const bool scaled = a.gscale != 1.0f;
    const void *fn = nullptr;
    switch (k) {
        case 1: fn = norm_kernel<1>(q8, scaled); break;
        case 2: fn = norm_kernel<2>(q8, scaled); break;
        case 3: fn = norm_kernel<3>(q8, scaled); break;
        case 4: fn = norm_kernel<4>(q8, scaled); break;
        case 5: fn = norm_kernel<5>(q8, scaled); break;
        case 6: fn = norm_kernel<6>(q8, scaled); break;
        case 7: fn = norm_kernel<7>(q8, scaled); break;
        case 8: fn = norm_kernel<8>(q8, scaled); break;
        case 9: fn = norm_kernel<9>(q8, scaled); break;
        case 10: fn = norm_kernel<10>(q8, scaled); break;
        case 11: fn = norm_kernel<11>(q8, scaled); break;
        case 12: fn = norm_kernel<12>(q8, scaled); break;
        case 13: fn = norm_kernel<13>(q8, scaled); break;
        case 14: fn = norm_kernel<14>(q8, scaled); break;
        case 15: fn = norm_kernel<15>(q8, scaled); break;
        case 16: fn = norm_kernel<16>(q8, scaled); break;
        default: return hipErrorInvalidValue;
    }
    NormArgs args = a;
    void *argv[] = {&args};
    return hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(kThreads), argv, 0, stream);
}

hipError_t launch_tensors_norm(const zs_piece *pieces, int64_t count, int64_t kept,
                               const FinishArgs &fin, int blocks, hipStream_t stream) {
    FinishArgs f = fin;
    void *argv[] = {&pieces, &count, &kept, &f};
    return hipLaunchKernel((const void *)tensors_norm_kernel, dim3((unsigned)blocks),
                           dim3(kThreads), argv, 0, stream);
}

hipError_t launch_tensors_clip(const zs_piece *pieces, int64_t count, const zs_clip *clip,
                               int64_t blocks, size_t lds, hipStream_t stream) {
    void *argv[] = {&pieces, &count, &clip};
    return hipLaunchKernel((const void *)tensors_clip_kernel, dim3((unsigned)blocks),
                           dim3(kThreads), argv, lds, stream);
}

hipError_t launch_finish(const double *sums, int count, const Rule &rule, zs_clip *clip,
                         hipStream_t stream) {
    Rule r = rule;
    void *argv[] = {&sums, &count, &r, &clip};
    return hipLaunchKernel((const void *)finish_kernel, dim3(1), dim3(kThreads), argv, 0, stream);
}

}  // namespace zs_detail
