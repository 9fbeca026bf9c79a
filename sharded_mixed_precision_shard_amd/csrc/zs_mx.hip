// zs_mx.hip -- kernels of the microscaled formats: quantisation, dequantisation
// and the products of a linear layer on them.
//
// A block is 32 elements along a row with one power of two 2^(b - 127).  Its
// elements are E2M1 (fp4) or E4M3 (fp8) numbers, both exact in bf16, and so is
// their product by the power of two (down to bf16's smallest denormal): the
// products below feed bf16 matrix instructions without any rounding of the
// stored operand, and sum in fp32.

#include <type_traits>

#include "zs_mx.h"

namespace zs_detail {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// Vectors at any address that suits their elements.
struct __attribute__((packed, aligned(2))) Any16 { u32x4 v; };
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Ordinary, or streaming: what is read or written once and does not fit the caches.
template <bool NT>
__device__ __forceinline__ u32x4 get16(const void *p) {
    if constexpr (NT) return __builtin_nontemporal_load((const u32x4_any *)p);
    return ((const Any16 *)p)->v;
}
template <bool NT>
__device__ __forceinline__ void set16(void *p, u32x4 v) {
    if constexpr (NT)
        __builtin_nontemporal_store(v, (u32x4_any *)p);
    else
        ((Any16 *)p)->v = v;
}

__device__ __forceinline__ float scale_of(uint32_t b) { return __uint_as_float(b << 23); }

__device__ __forceinline__ uint32_t bits(bf16x2 v) { return __builtin_bit_cast(uint32_t, v); }

// 8 codes as bf16 times the scale: fp4 in one word, fp8 in two.
__device__ __forceinline__ u32x4 widen_fp4(uint32_t w, float s) {
    return u32x4{bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                 bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                 bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                 bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
}
__device__ __forceinline__ u32x4 widen_fp8(uint32_t w0, uint32_t w1, float s) {
    return u32x4{bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false)),
                 bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true)),
                 bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false)),
                 bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true))};
}

// 32 fp4 codes as an operand of the scaled matrix instruction, which reads four words.
__device__ __forceinline__ i32x8 codes4(u32x4 v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// ------------------------------------------------ quantisation, dequantisation

// Four lanes take a block, 8 elements each; a workgroup takes kCastUnroll times
// 64 blocks.  Bound by memory: bf16 to fp8 moves 3.03 bytes per element, to fp4
// 2.53, against about 3 vector instructions per element.  6.7e7 bf16 elements to fp8 33 us
// (6.1 TB/s), 8.1e8 to fp4 and back 651 us (6.3 TB/s).  Four blocks a thread: two take 34 and
// 666, one 36 and 744.
constexpr int kCastUnroll = 4;
constexpr int kCastBlocks = kCastUnroll * kThreads / 4;
// A grid's dimension holds fewer than 2^32 threads, and 2^32 - 1 blocks take as many: workgroups
// are numbered along x in rows of 2^31 threads.
constexpr int64_t kCastRow = (int64_t(1) << 31) / kThreads;
__device__ __forceinline__ int64_t cast_block() {
    return (blockIdx.y * kCastRow + blockIdx.x) * kCastBlocks + threadIdx.x / 4;
}

template <int DT, bool NT>
__device__ __forceinline__ void load8(const void *x, int64_t at, int64_t left, float v[8]) {
    if constexpr (DT == ZS_DTYPE_FP32) {
        const float *p = (const float *)x + at;
        if (left >= 8) {
            const u32x4 a = get16<NT>(p), b = get16<NT>(p + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = __uint_as_float(a[e]);
                v[e + 4] = __uint_as_float(b[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < left ? p[e] : 0.0f;
        }
    } else {
        const uint16_t *p = (const uint16_t *)x + at;
        u32x4 a = {0, 0, 0, 0};
        if (left >= 8) {
            a = get16<NT>(p);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) a[e / 2] |= (uint32_t)p[e] << (16 * (e % 2));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t h = (a[e / 2] >> (16 * (e % 2))) & 0xffffu;
            if constexpr (DT == ZS_DTYPE_BF16)
                v[e] = __uint_as_float(h << 16);
            else
                v[e] = (float)__builtin_bit_cast(_Float16, (uint16_t)h);
        }
    }
}

// Largest of the four lanes that share a block.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
    const uint32_t a = (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xf, 0xf, true);
    m = m > a ? m : a;
    const uint32_t b = (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xf, 0xf, true);
    return m > b ? m : b;
}

template <int FMT, int DT, int STREAM>
__global__ __launch_bounds__(kThreads) void mx_quantize(MxCastArgs a) {
    const int part = threadIdx.x % 4;
    const int64_t first = cast_block();
    float v[kCastUnroll][8];
#pragma unroll
    for (int u = 0; u < kCastUnroll; ++u) {
        const int64_t block = first + u * (kThreads / 4);
        const int64_t row = a.nb < a.blocks ? (uint32_t)block / (uint32_t)a.nb : 0;
        const int64_t col = (block - row * a.nb) * kMxBlock + part * 8;
        load8<DT, (STREAM > 0)>(a.x, row * a.ld + col, block < a.blocks ? a.cols - col : 0, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kCastUnroll; ++u) {
        const int64_t block = first + u * (kThreads / 4);
        // magnitudes order as their bits do, infinity and NaN above every number
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t b = __float_as_uint(v[u][e]) & 0x7fffffffu;
            m = m > b ? m : b;
        }
        m = block_max(m);
        const bool finite = m < 0x7f800000u;
        constexpr int top = FMT == ZS_MX_FP4 ? 2 : 8;
        const int e = (int)(m >> 23) - top;
        const uint32_t b = e > 0 ? (uint32_t)e : 0u;  // the biased exponent of the scale
        const float inv = finite ? __uint_as_float((254u - b) << 23) : 0.0f;
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            q[i] = finite ? v[u][i] * inv : 0.0f;
            // E4M3 has no infinity to saturate at: 448 is its largest value
            if constexpr (FMT == ZS_MX_FP8) q[i] = __builtin_amdgcn_fmed3f(q[i], -448.0f, 448.0f);
        }
        if (block < a.blocks) {
            if constexpr (FMT == ZS_MX_FP4) {
                uint32_t w = 0;
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[0], q[1], 1.0f, 0);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[2], q[3], 1.0f, 1);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[4], q[5], 1.0f, 2);
                w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[6], q[7], 1.0f, 3);
                uint32_t *to = (uint32_t *)a.codes + block * 4 + part;
                if constexpr (STREAM > 1)
                    __builtin_nontemporal_store(w, to);
                else
                    *to = w;
            } else {
                s16x2 lo = {0, 0}, hi = {0, 0};
                lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, q[0], q[1], 1.0f, false);
                lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, q[2], q[3], 1.0f, true);
                hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, q[4], q[5], 1.0f, false);
                hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, q[6], q[7], 1.0f, true);
                uint64_t *to = (uint64_t *)a.codes + block * 4 + part;
                const uint64_t w = (uint64_t)__builtin_bit_cast(uint32_t, hi) << 32 |
                                   __builtin_bit_cast(uint32_t, lo);
                if constexpr (STREAM > 1)
                    __builtin_nontemporal_store(w, to);
                else
                    *to = w;
            }
            if (part == 0) a.scales[block] = finite ? (uint8_t)b : 255;
        }
    }
}

template <int DT, bool NT>
__device__ __forceinline__ void store8(void *x, int64_t at, int64_t left, const float v[8]) {
    if constexpr (DT == ZS_DTYPE_FP32) {
        float *p = (float *)x + at;
        if (left >= 8) {
            set16<NT>(p, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                               __float_as_uint(v[2]), __float_as_uint(v[3])});
            set16<NT>(p + 4, u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]),
                                   __float_as_uint(v[6]), __float_as_uint(v[7])});
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) p[e] = v[e];
        }
    } else {
        uint16_t *p = (uint16_t *)x + at;
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (DT == ZS_DTYPE_BF16)
                h[e] = __builtin_bit_cast(uint16_t, (__bf16)v[e]);
            else
                h[e] = __builtin_bit_cast(uint16_t, (_Float16)v[e]);
        }
        if (left >= 8) {
            set16<NT>(p, u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16,
                               h[6] | h[7] << 16});
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) p[e] = (uint16_t)h[e];
        }
    }
}

template <int FMT, int DT, bool NT>
__global__ __launch_bounds__(kThreads) void mx_dequantize(MxCastArgs a) {
    const int part = threadIdx.x % 4;
    const int64_t first = cast_block();
    uint2 code[kCastUnroll];
    uint32_t scale[kCastUnroll];
#pragma unroll
    for (int u = 0; u < kCastUnroll; ++u) {
        const int64_t block = first + u * (kThreads / 4);
        code[u] = uint2{0, 0};
        scale[u] = 0;
        if (block < a.blocks) {
            if constexpr (FMT == ZS_MX_FP4)
                code[u].x = ((const uint32_t *)a.codes)[block * 4 + part];
            else
                code[u] = ((const uint2 *)a.codes)[block * 4 + part];
            scale[u] = a.scales[block];
        }
    }
#pragma unroll
    for (int u = 0; u < kCastUnroll; ++u) {
        const int64_t block = first + u * (kThreads / 4);
        const int64_t row = a.nb < a.blocks ? (uint32_t)block / (uint32_t)a.nb : 0;
        const int64_t col = (block - row * a.nb) * kMxBlock + part * 8;
        const float s = scale_of(scale[u]);
        f32x2 w[4];
        if constexpr (FMT == ZS_MX_FP4) {
            w[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[u].x, s, 0);
            w[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[u].x, s, 1);
            w[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[u].x, s, 2);
            w[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[u].x, s, 3);
        } else {
            w[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code[u].x, s, false);
            w[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code[u].x, s, true);
            w[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code[u].y, s, false);
            w[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code[u].y, s, true);
        }
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = w[e / 2][e % 2];
        if (block < a.blocks) store8<DT, NT>(a.x, row * a.ld + col, a.cols - col, v);
    }
}

// ------------------------------------------------------------------ products

constexpr int kStep = 64;  // c's per step: two blocks of a stored row

// A tile in LDS holds bf16, kStep c's of B rows.  Row-major (c along a row):
// 128 bytes a row, half of the banks, its eight 16-byte chunks in an order that the row's
// number permutes: any 16 neighbouring rows have a chunk in each of the 16 places, so the
// reads of a fragment find no bank busy (permuted by row & 7 half of the LDS cycles of the 7B
// products were conflicts).
// Column-major (c a row of B elements): the 64-byte chunks of a row are permuted by c, and
// the 16 bytes inside each, too.  Four rows' 64 bytes, which a transposing read takes, then lie
// in different banks, and so do the pieces that lanes of four rows and blocks write together.
__device__ __forceinline__ int at_rows(int row, int chunk) {
    return row * 128 + ((chunk ^ (row >> 1 & 7)) << 4);
}
template <int B>
__device__ __forceinline__ int at_cols(int c, int byte) {
    if constexpr (B >= 256)
        return c * (B * 2) + (byte ^ ((c & 7) << 6) ^ ((c & 3) << 4));
    else if constexpr (B == 128)
        return c * (B * 2) + (byte ^ ((c & 3) << 6) ^ ((c & 3) << 4));
    else
        return c * (B * 2) + (byte ^ ((c >> 1 & 1) << 6) ^ ((c >> 1 & 3) << 4));
}

// The 8 c's of a 32x32x16 fragment that a lane holds: c = 16 s + 8 (lane / 32) ..
// of row base + lane % 32.
__device__ __forceinline__ bf16x8 frag_rows(const char *lds, int base, int s, int lane) {
    const int row = base + lane % 32;
    return *(const bf16x8 *)(lds + at_rows(row, 2 * s + lane / 32));
}
// The same from a column-major tile: of 16 lanes each reads 8 bytes of row
// (lane % 16) / 4, and the transposing read hands lane i the elements i of four rows.
template <int B>
__device__ __forceinline__ bf16x8 frag_cols(const char *lds, int base, int s, int lane) {
    typedef s16x4 __attribute__((address_space(3))) * lds_s16x4;
    const int t = lane % 16;
    const int c = 16 * s + 8 * (lane / 32) + t / 4;
    const int byte = (base + (lane / 16) % 2 * 16 + (t % 4) * 4) * 2;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4)(lds + at_cols<B>(c, byte)));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4)(lds + at_cols<B>(c + 4, byte)));
    const short v __attribute__((ext_vector_type(8))) = {lo[0], lo[1], lo[2], lo[3],
                                                         hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, v);
}

// What a thread carries of a bf16 operand from memory to LDS.  COLS: c is the row.
template <int B, int NT, bool COLS>
struct PlainStage {
    static constexpr int kChunks = B * kStep / 8;
    static constexpr int kEach = kChunks / NT;
    u32x4 r[kEach];

    __device__ __forceinline__ void load(const uint16_t *p, int64_t ld, int first, int rows, int c0,
                                         int C, int tid) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int q = k * NT + tid;
            int64_t row, col;
            int left;
            if constexpr (COLS) {
                const int c = c0 + q / (B / 8), i = first + q % (B / 8) * 8;
                row = c;
                col = i;
                left = c < C ? rows - i : 0;
            } else {
                const int i = first + q / 8, c = c0 + q % 8 * 8;
                row = i;
                col = c;
                left = i < rows ? C - c : 0;
            }
            const uint16_t *x = p + row * ld + col;
            u32x4 v = {0, 0, 0, 0};
            if (left >= 8) {
                v = ((const Any16 *)x)->v;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < left) v[e / 2] |= (uint32_t)x[e] << (16 * (e % 2));
            }
            r[k] = v;
        }
    }
    // The same where every c of the step and the one after it is inside, and rows >= 8: what
    // lies past the rows is read from inside the matrix, as part of sums that nobody keeps.
    __device__ __forceinline__ void load_inside(const uint16_t *p, int64_t ld, int first, int rows,
                                                int c0, int tid) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int q = k * NT + tid;
            int64_t at;
            if constexpr (COLS)
                at = (int64_t)(c0 + q / (B / 8)) * ld + min(first + q % (B / 8) * 8, rows - 1);
            else
                at = (int64_t)min(first + q / 8, rows - 1) * ld + c0 + q % 8 * 8;
            r[k] = ((const Any16 *)(p + at))->v;
        }
    }
    // Zeros go to LDS where `in` is false.
    __device__ __forceinline__ void store(char *lds, int tid, bool in = true) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int q = k * NT + tid;
            const int at = COLS ? at_cols<B>(q / (B / 8), q % (B / 8) * 16) : at_rows(q / 8, q % 8);
            *(u32x4 *)(lds + at) = in ? r[k] : u32x4{0, 0, 0, 0};
        }
    }
};

// The same of an operand in blocks: a unit is one block, widened to bf16 on its way.
template <int B, int NT, bool COLS, bool F8>
struct HeldStage {
    static constexpr int kUnits = B * kStep / kMxBlock;
    static constexpr int kEach = (kUnits + NT - 1) / NT;
    u32x4 r[kEach][F8 ? 2 : 1];
    uint32_t scale[kEach];

    __device__ __forceinline__ void load(const MxHeld &x, int first, int rows, int c0, int C,
                                         int tid) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int q = k * NT + tid;
            int64_t row, block;
            bool in;
            if constexpr (COLS) {
                row = c0 + q / (B / kMxBlock);
                block = first / kMxBlock + q % (B / kMxBlock);
                in = row < C;
            } else {
                row = first + q / 2;
                block = c0 / kMxBlock + q % 2;
                in = row < rows;
            }
            r[k][0] = u32x4{0, 0, 0, 0};
            if constexpr (F8) r[k][1] = u32x4{0, 0, 0, 0};
            scale[k] = 127;
            if (in && block < x.nb && q < kUnits) {
                const int64_t at = row * x.nb + block;
                const u32x4 *codes = (const u32x4 *)x.codes + at * (F8 ? 2 : 1);
                r[k][0] = codes[0];
                if constexpr (F8) r[k][1] = codes[1];
                scale[k] = x.scales[at];
            }
        }
    }
    __device__ __forceinline__ void load_inside(const MxHeld &x, int first, int rows, int c0,
                                                int tid) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int q = min(k * NT + tid, kUnits - 1);
            int64_t at;
            if constexpr (COLS)
                at = (int64_t)(c0 + q / (B / kMxBlock)) * x.nb +
                     min((int64_t)(first / kMxBlock + q % (B / kMxBlock)), x.nb - 1);
            else
                at = (int64_t)min(first + q / 2, rows - 1) * x.nb + c0 / kMxBlock + q % 2;
            const u32x4 *codes = (const u32x4 *)x.codes + at * (F8 ? 2 : 1);
            r[k][0] = codes[0];
            if constexpr (F8) r[k][1] = codes[1];
            scale[k] = x.scales[at];
        }
    }
    // Where `in` is false the numbers go to LDS times 2^-127.  A bf16 operand's are 0 there, and
    // two stored operands' products, below 2^-235, are 0 in fp32 (a NaN among them is one of the
    // row's, which the row's sum has all the same).
    __device__ __forceinline__ void store(char *lds, int tid, bool in = true) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int q = k * NT + tid;
            if (kUnits % NT != 0 && q >= kUnits) continue;
            const float s = scale_of(in ? scale[k] : 0u);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                u32x4 v;
                if constexpr (F8)
                    v = widen_fp8(r[k][w / 2][w % 2 * 2], r[k][w / 2][w % 2 * 2 + 1], s);
                else
                    v = widen_fp4(r[k][0][w], s);
                const int at = COLS ? at_cols<B>(q / (B / kMxBlock),
                                                 q % (B / kMxBlock) * 64 + w * 16)
                                    : at_rows(q / 2, q % 2 * 4 + w);
                *(u32x4 *)(lds + at) = v;
            }
        }
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return bits(v);
}

// 16 bytes of out from [i, j] on, as far as there are.
__device__ __forceinline__ void put16(const MxProductArgs &a, int i, int j, u32x4 v) {
    if (i >= a.I || j >= a.J) return;
    const int64_t at = (int64_t)i * a.ldo + j;
    if (a.out_f32) {
        uint32_t *o = (uint32_t *)a.out + at;
        if (j + 4 <= a.J) {
            ((Any16 *)o)->v = v;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < a.J) o[e] = v[e];
        }
    } else {
        uint16_t *o = (uint16_t *)a.out + at;
        if (j + 8 <= a.J) {
            ((Any16 *)o)->v = v;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (j + e < a.J) o[e] = (uint16_t)(v[e / 2] >> (16 * (e % 2)));
        }
    }
}
// The fp32 values there, zeros past the end.
__device__ __forceinline__ u32x4 there(const MxProductArgs &a, int i, int j) {
    u32x4 v = {0, 0, 0, 0};
    if (i >= a.I || j >= a.J) return v;
    const uint32_t *o = (const uint32_t *)a.out + (int64_t)i * a.ldo + j;
    if (j + 4 <= a.J) return ((const Any16 *)o)->v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (j + e < a.J) v[e] = o[e];
    return v;
}

// One value of out.
__device__ __forceinline__ void put1(const MxProductArgs &a, int i, int j, float v) {
    if (i >= a.I || j >= a.J) return;
    const int64_t at = (int64_t)i * a.ldo + j;
    if (a.out_f32)
        ((float *)a.out)[at] = v;
    else
        ((__bf16 *)a.out)[at] = (__bf16)v;
}

// Memory of fewer than 2^31 bytes that instructions address by 32-bit offsets: reads past
// its end give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)bytes, 0x00027000);
}

// Sums on their way to the split that joins them.  The workgroups sit on XCDs whose L2
// caches do not see each other's writes, so they are written and read past those caches
// (sc1, as agent-scope atomics are, but 16 bytes at a time); a workgroup arrives when its own
// have been acknowledged.
constexpr int kPastL2 = 16;
__device__ __forceinline__ void put_part(float *parts, uint32_t at, f32x4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v),
                                           buffer_of(parts, (uint32_t)kMxPartBytes), at * 4u, 0,
                                           kPastL2);
}
__device__ __forceinline__ f32x4 get_part(const float *parts, uint32_t at) {
    return __builtin_bit_cast(
        f32x4, __builtin_amdgcn_raw_buffer_load_b128(buffer_of(parts, (uint32_t)kMxPartBytes),
                                                     at * 4u, 0, kPastL2));
}

// Whether another workgroup has arrived at a counter, for all threads.
__device__ __forceinline__ bool arrived(uint32_t *counter, uint32_t *shared) {
    __syncthreads();
    if (threadIdx.x == 0)
        *shared = __hip_atomic_load(counter, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const bool yes = *shared != 0;
    __syncthreads();
    return yes;
}

// Whether this of a tile's splits arrives last: the others' sums are then in memory.  All
// threads call it after they have put theirs; the counter is left at 0.
__device__ __forceinline__ bool last_split(uint32_t *counter, int splits, uint32_t *shared) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t before =
            __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const bool last = before == (uint32_t)splits - 1u;
        if (last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *shared = last;
    }
    __syncthreads();
    return *shared != 0;
}

// Which tile a workgroup makes.  Workgroups are dealt to the XCDs in turn: each XCD
// gets a run of neighbouring tiles, and walks it in bands of kBand tiles of i, so that
// the rows its compute units read at a time are few enough for its L2.
constexpr int kXcds = 8;
constexpr int kBand = 8;
__device__ __forceinline__ void tile_of(int64_t block, int tiles_i, int tiles_j, int *i, int *j) {
    const int64_t tiles = (int64_t)tiles_i * tiles_j;
    const int64_t each = tiles / kXcds, more = tiles % kXcds, x = block % kXcds;
    const int64_t id = x * each + (x < more ? x : more) + block / kXcds;
    const int64_t band = id / ((int64_t)kBand * tiles_j);
    const int rows = min(kBand, tiles_i - (int)band * kBand);
    const int64_t in = id - band * kBand * tiles_j;
    *i = (int)band * kBand + (int)(in % rows);
    *j = (int)(in / rows);
}

// The wave groups of a workgroup, each with a part of c: all but the first leave their sums
// in LDS, wave by wave at scratch(group, wave), and the first adds them in order.  True for
// the first; the others end, and the barriers behind this wait for its waves alone.
template <int KG, int FJ, int FI, class S>
__device__ __forceinline__ bool join_groups(f32x16 (&acc)[FJ][FI], const S &scratch, int group,
                                            int wave, int lane) {
    if constexpr (KG == 1) return true;
    if (group > 0) {
        f32x4 *to = (f32x4 *)scratch(group, wave) + lane;
#pragma unroll
        for (int j = 0; j < FJ; ++j)
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    to[((j * FI + i) * 4 + r) * kWave] =
                        f32x4{acc[j][i][4 * r], acc[j][i][4 * r + 1], acc[j][i][4 * r + 2],
                              acc[j][i][4 * r + 3]};
    }
    __syncthreads();
    if (group > 0) return false;
#pragma unroll
    for (int g = 1; g < KG; ++g) {
        const f32x4 *from = (const f32x4 *)scratch(g, wave) + lane;
#pragma unroll
        for (int j = 0; j < FJ; ++j)
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const f32x4 v = from[((j * FI + i) * 4 + r) * kWave];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][i][4 * r + e] += v[e];
                }
    }
    return true;
}

// Bytes of LDS that a wave's scratch holds: its sums, or 4 KB to turn them in.
constexpr int scratch_bytes(int groups, int frags) { return groups > 1 ? frags * 4096 : 4096; }

// The end of a tile: its sums go out, or to the workspace, where another split finds them.
// `mine` is 4 KB of LDS of the wave's own.
template <int BI, int BJ, int WI, int WJ>
__device__ __forceinline__ void finish_tile(const MxProductArgs &a,
                                            f32x16 (&acc)[BJ / WJ / 32][BI / WI / 32],
                                            int tile, int split, int i0, int j0, int wi, int wj,
                                            int wave, int lane, uint32_t *shared, char *mine) {
    constexpr int FI = BI / WI / 32, FJ = BJ / WJ / 32;
    // Splits are joined two by two: of splits [s, s + n) and [s + n, s + 2 n) the one that is
    // done first leaves its sums and ends, the other adds them to its own and goes on with
    // both.  The tree is the same every time and an addition's two sides may change places,
    // so the order in which splits end does not show.  (Tiles of 256 x 256 are never split, see
    // plan; left out of them, this made the compiler issue the fp4 kernel's transfers in another
    // order, 70B product 1062 us instead of 1034.)
    const uint32_t here = (uint32_t)wave * (FJ * FI * 1024) + (uint32_t)lane * 4;
    const uint32_t slots = (uint32_t)tile * (uint32_t)a.splits;
    for (int n = 1; n < a.splits; n *= 2) {
        const int s = split & ~(2 * n - 1), other = split & n ? s : s + n;
        if (other >= a.splits) continue;
        uint32_t *counter = a.counters + (int64_t)tile * a.splits + s + n;
        if (!arrived(counter, shared)) {
            const uint32_t to = (slots + (uint32_t)(split & ~(n - 1))) * (BI * BJ) + here;
#pragma unroll
            for (int j = 0; j < FJ; ++j)
#pragma unroll
                for (int i = 0; i < FI; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        put_part(a.parts, to + ((j * FI + i) * 4 + r) * 256,
                                 f32x4{acc[j][i][4 * r], acc[j][i][4 * r + 1],
                                       acc[j][i][4 * r + 2], acc[j][i][4 * r + 3]});
            if (!last_split(counter, 2, shared)) return;
        } else if (threadIdx.x == 0) {
            __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        const uint32_t theirs = (slots + (uint32_t)other) * (BI * BJ) + here;
#pragma unroll
        for (int j = 0; j < FJ; ++j)
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const f32x4 v = get_part(a.parts, theirs + ((j * FI + i) * 4 + r) * 256);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][i][4 * r + e] += v[e];
                }
        __syncthreads();  // `shared` is free again
    }
    // A lane holds four neighbours of one row of out.  Through LDS a wave's 32 rows leave in
    // stretches of 64 or 128 bytes (bf16; 128 in fp32), 16 bytes a lane.
    const int i = lane % 32, half = lane / 32, row = lane / 8, chunk = lane % 8;
    constexpr int PAIR = FJ % 2 == 0 ? 2 : 1;  // fragments side by side in a row of bf16
#pragma unroll
    for (int f = 0; f < FI; ++f) {
        if (a.out_f32) {
            // what is there already, all of it on its way at a time (4096^3 151 us one after the
            // other, 142 so)
            u32x4 old[FJ][4];
#pragma unroll
            for (int j = 0; j < FJ; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    old[j][k] = u32x4{0, 0, 0, 0};
                    if (a.add)
                        old[j][k] = there(a, i0 + wi + 32 * f + 8 * k + row,
                                          j0 + wj + 32 * j + 4 * chunk);
                }
#pragma unroll
            for (int j = 0; j < FJ; ++j) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *(f32x4 *)(mine + at_rows(i, 2 * r + half)) =
                        f32x4{acc[j][f][4 * r], acc[j][f][4 * r + 1], acc[j][f][4 * r + 2],
                              acc[j][f][4 * r + 3]};
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    u32x4 v = *(const u32x4 *)(mine + at_rows(8 * k + row, chunk));
                    if (a.add) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = __float_as_uint(__uint_as_float(old[j][k][e]) +
                                                   __uint_as_float(v[e]));
                    }
                    put16(a, i0 + wi + 32 * f + 8 * k + row, j0 + wj + 32 * j + 4 * chunk, v);
                }
                __builtin_amdgcn_wave_barrier();
            }
        } else {
#pragma unroll
            for (int j = 0; j < FJ; j += PAIR) {
#pragma unroll
                for (int e = 0; e < PAIR; ++e)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        *(uint2 *)(mine + at_rows(i, 4 * e + r) + 8 * half) =
                            uint2{pack_bf16(acc[j + e][f][4 * r], acc[j + e][f][4 * r + 1]),
                                  pack_bf16(acc[j + e][f][4 * r + 2], acc[j + e][f][4 * r + 3])};
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (PAIR == 2 || chunk < 4)
                        put16(a, i0 + wi + 32 * f + 8 * k + row, j0 + wj + 32 * j + 8 * chunk,
                              *(const u32x4 *)(mine + at_rows(8 * k + row, chunk)));
                __builtin_amdgcn_wave_barrier();
            }
        }
    }
}

// The steps that each wave group of a split takes; past the last c all reads as 0.
template <int KG>
__device__ __forceinline__ int group_steps(const MxProductArgs &a, int depth, int split) {
    return min((a.C + depth - 1) / depth - split * KG * a.split_steps, a.split_steps);
}

// A workgroup makes a BI x BJ tile of out (of one split of c, in KG wave groups).  The matrix
// instruction takes Q's rows as its rows and P's as its columns: a lane then
// holds four neighbouring j's of one i, and stores them together.
//
// This one takes any strides and depths: both operands go through registers, a step ahead, with
// loads of 16 bytes at addresses of 2.  Bound by what those registers leave to be in flight:
// 4096^3 132 us on odd rows (1.04 PFLOP/s; 109 in the kernels below), 118 for fp8 by fp4, which
// has no other.
template <int BI, int BJ, int WI, int WJ, int KG, int LEFT, int RIGHT>
__global__ __launch_bounds__(WI *WJ *KG *kWave, 2) void mx_tile(MxProductArgs a) {
    constexpr int NT = WI * WJ * kWave;
    constexpr int FI = BI / WI / 32, FJ = BJ / WJ / 32;
    constexpr bool PC = LEFT == kLeftCols, QC = (RIGHT & kRightCols) != 0;
    constexpr bool P_HELD = LEFT == kLeftFp4 || LEFT == kLeftFp8;
    constexpr int P_BYTES = BI * kStep * 2, Q_BYTES = BJ * kStep * 2;
    __shared__ __attribute__((aligned(128))) char all[KG][2 * (P_BYTES + Q_BYTES)];

    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
    const int tid = threadIdx.x % NT, lane = tid % kWave, wave = tid / kWave;
    char *lds = all[group];
    const int split = blockIdx.x % a.splits;
    int ti, tj;
    tile_of(blockIdx.x / a.splits, a.tiles_i, a.tiles_j, &ti, &tj);
    const int tile = tj * a.tiles_i + ti, i0 = ti * BI, j0 = tj * BJ;
    const int wi = wave % WI * (BI / WI), wj = wave / WI * (BJ / WJ);
    // The last step, whole or not, is taken first and element by element; the others have all
    // of their c's inside, and no branches.
    const int full = a.C > 0 ? (a.C - 1) / kStep : 0;
    const int first = (split * KG + group) * a.split_steps;
    const int steps = min(full - split * KG * a.split_steps, a.split_steps);

    f32x16 acc[FJ][FI];
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
        for (int i = 0; i < FI; ++i) acc[j][i] = f32x16{};
    auto multiply = [&](const char *p, const char *q) {
#pragma unroll
        for (int s = 0; s < kStep / 16; ++s) {
            bf16x8 pf[FI], qf[FJ];
#pragma unroll
            for (int i = 0; i < FI; ++i)
                pf[i] = PC ? frag_cols<BI>(p, wi + 32 * i, s, lane)
                           : frag_rows(p, wi + 32 * i, s, lane);
#pragma unroll
            for (int j = 0; j < FJ; ++j)
                qf[j] = QC ? frag_cols<BJ>(q, wj + 32 * j, s, lane)
                           : frag_rows(q, wj + 32 * j, s, lane);
#pragma unroll
            for (int j = 0; j < FJ; ++j)
#pragma unroll
                for (int i = 0; i < FI; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qf[j], pf[i], acc[j][i], 0,
                                                                        0, 0);
        }
    };

    std::conditional_t<P_HELD, HeldStage<BI, NT, false, LEFT == kLeftFp8>,
                       PlainStage<BI, NT, PC>> ps;
    HeldStage<BJ, NT, QC, (RIGHT & kRightFp8) != 0> qs;
    if (split == 0 && a.C > 0) {
        const int c0 = group == 0 ? full * kStep : a.C;  // the other groups add zeros
        if constexpr (P_HELD)
            ps.load(a.px, i0, group == 0 ? a.I : 0, c0, a.C, tid);
        else
            ps.load(a.p, a.ldp, i0, a.I, c0, a.C, tid);
        qs.load(a.q, j0, group == 0 ? a.J : 0, c0, a.C, tid);
        ps.store(lds, tid);
        qs.store(lds + P_BYTES, tid);
        __syncthreads();
        multiply(lds, lds + P_BYTES);
        __syncthreads();
    }
    auto load = [&](int step) {
        const int c0 = min(first + step, full - 1) * kStep;
        if constexpr (P_HELD)
            ps.load_inside(a.px, i0, a.I, c0, tid);
        else if (PC && a.I < 8)
            ps.load(a.p, a.ldp, i0, a.I, c0, a.C, tid);
        else
            ps.load_inside(a.p, a.ldp, i0, a.I, c0, tid);
        qs.load_inside(a.q, j0, a.J, c0, tid);
    };
    auto store = [&](int step) {
        char *p = lds + step % 2 * (P_BYTES + Q_BYTES);
        const bool in = KG == 1 || first + step < full;
        ps.store(p, tid, in);
        qs.store(p + P_BYTES, tid, in);
    };
    if (steps > 0) {
        load(0);
        store(0);
    }
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
        load(step + 1);  // past the last step this reads the last one again
        __syncthreads();
        const char *p = lds + step % 2 * (P_BYTES + Q_BYTES);
        multiply(p, p + P_BYTES);
        store(step + 1);
    }

    __shared__ uint32_t shared;
    __syncthreads();
    constexpr int EACH = 2 * (P_BYTES + Q_BYTES) / (WI * WJ);
    static_assert(EACH >= scratch_bytes(KG, FI * FJ), "scratch");
    auto scratch = [&](int g, int w) { return all[g] + w * EACH; };
    if (join_groups<KG>(acc, scratch, group, wave, lane))
        finish_tile<BI, BJ, WI, WJ>(a, acc, tile, split, i0, j0, wi, wj, wave, lane, &shared,
                                    scratch(0, wave));
}

// ---------------------------------------------- products of two fp4 operands

// Rows of a tile through LDS as they are stored: kStep4 codes (128 bytes, eight
// blocks) of each row per step, the chunks of a row permuted by the row's number as
// at_rows does, and its eight scales beside them.
constexpr int kStep4 = 256;
constexpr int kStep4Blocks = kStep4 / kMxBlock;

typedef __attribute__((address_space(3))) void lds_void;
struct __attribute__((packed, aligned(1))) Bytes8 { uint64_t v; };

// From memory to LDS past the registers: lane l's 16 bytes go to lds + 16 l.  kNowhere, and
// what is added to it, is past every buffer's size.
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t from, char *lds, uint32_t offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void *)lds, 16, (int)offset, 0, 0, 0);
}
// A workgroup's stage is ready: at most N of each wave's memory operations are still on
// their way (they end in order), and nothing of the stage before is still being read.
template <int N>
__device__ __forceinline__ void stage_ready() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Memory operations before this are issued before those behind it.  A wait for all but the N
// newest operations is one for a transfer only as long as N others follow it.
__device__ __forceinline__ void in_order() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Eight scales of a row from `block` on, inside the row, shifted where they reach back: what
// is past the row's end becomes 0 or 1, scales that stand for numbers.  No branch: in the
// loops below one would cost registers that the sums need.
struct Scales8 {
    uint64_t raw;
    int shift;
    __device__ __forceinline__ void load(const uint8_t *row, int block, int nb) {
        const int from = min(block, nb - 8);
        raw = ((const Bytes8 *)(row + from))->v;
        shift = min(8 * (block - from), 63);
    }
    __device__ __forceinline__ uint64_t value() const { return raw >> shift; }
};

// Both operands' codes go into the scaled matrix instruction as they are: 64 products
// of a row and a column per instruction, at four times the rate of bf16.  A lane holds
// a block of 32, so its scale is one byte, taken from a word of four by number.
//
// 8192 x 28672 of depth 8192 1.04 ms (3.7 PFLOP/s, through bf16 instructions 4.5 ms), 4096^3 47
// us.  The matrix pipe is busy 48 % of the time: of the 1.04 ms the transfers take 0.16, the
// scales' way through LDS 0.07, the output 0.07, and each stage ends with both waves of a SIMD
// at its barrier.  Two waves of 128 x 64 per SIMD, since one of 128 x 128 was given copies of all
// its sums every turn.
template <int BI, int BJ, int WI, int WJ, int KG>
__global__ __launch_bounds__(WI *WJ *KG *kWave, 2) void mx_tile_fp4(MxProductArgs a) {
    constexpr int NT = WI * WJ * kWave;
    constexpr int FI = BI / WI / 32, FJ = BJ / WJ / 32;
    constexpr int P_BYTES = BI * 128, Q_BYTES = BJ * 128;
    constexpr int EACH_P = BI * 8 / NT, EACH_Q = BJ * 8 / NT;
    // two stages, each an array of its own: the compiler sees that the codes read of one do not
    // wait for what is on its way into the other (the reads of scales do: it cannot tell them
    // from what the transfers write)
    __shared__ __attribute__((aligned(128))) char all0[KG][P_BYTES + Q_BYTES];
    __shared__ __attribute__((aligned(128))) char all1[KG][P_BYTES + Q_BYTES];
    static_assert(BI + BJ <= NT, "a thread takes the scales of one row at most");
    __shared__ uint64_t all_scales0[KG][NT];
    __shared__ uint64_t all_scales1[KG][NT];

    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
    const int tid = threadIdx.x % NT, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    char *lds0 = all0[group], *lds1 = all1[group];
    uint64_t *scales0 = all_scales0[group], *scales1 = all_scales1[group];
    const int split = blockIdx.x % a.splits;
    int ti, tj;
    tile_of(blockIdx.x / a.splits, a.tiles_i, a.tiles_j, &ti, &tj);
    const int tile = tj * a.tiles_i + ti, i0 = ti * BI, j0 = tj * BJ;
    const int wi = wave % WI * (BI / WI), wj = wave / WI * (BJ / WJ);
    const int nb = (int)a.q.nb;
    const uint32_t row_bytes = (uint32_t)nb * 16u;
    const int first = (split * KG + group) * a.split_steps;
    const int steps = group_steps<KG>(a, kStep4, split);

    const auto p_buf = buffer_of(a.px.codes + (int64_t)i0 * row_bytes,
                                 (uint32_t)min(a.I - i0, BI) * row_bytes);
    const auto q_buf = buffer_of(a.q.codes + (int64_t)j0 * row_bytes,
                                 (uint32_t)min(a.J - j0, BJ) * row_bytes);
    // a wave's chunk k: eight rows, lane / 8 the row, lane % 8 the place in it
    const int row = wave * 8 + lane / 8, chunk = (lane % 8) ^ (row >> 1 & 7);
    const uint32_t p_off = (uint32_t)row * row_bytes + (uint32_t)chunk * 16u;
    const uint8_t *my_scales = tid < BI ? a.px.scales + (int64_t)min(i0 + tid, a.I - 1) * nb
                                        : a.q.scales + (int64_t)min(j0 + tid - BI, a.J - 1) * nb;

    // tiles begin at different steps: the rows of wide operands lie a power of two apart, and
    // workgroups that read the same columns at a time would meet on few of the L2's channels
    const int turns = (steps + 1) / 2 * 2, skew = turns > 0 ? (ti + tj) % 16 * 2 % turns : 0;
    auto block_of = [&](int step) {
        step += skew;
        return (first + (step >= turns ? step - turns : step)) * kStep4Blocks;
    };
    auto fetch = [&](char *lds, int step) {
        const int block = block_of(step);
        // blocks past the row's end read as zero codes (all of the address is in the lane's
        // offset, which is what the size is compared with)
        const uint32_t off = block + chunk < nb ? p_off + (uint32_t)block * 16u : kNowhere;
#pragma unroll
        for (int k = 0; k < EACH_P; ++k)
            dma16(p_buf, lds + (k * (NT / 8) + wave * 8) * 128,
                  off + (uint32_t)(k * (NT / 8)) * row_bytes);
#pragma unroll
        for (int k = 0; k < EACH_Q; ++k)
            dma16(q_buf, lds + P_BYTES + (k * (NT / 8) + wave * 8) * 128,
                  off + (uint32_t)(k * (NT / 8)) * row_bytes);
    };
    auto fetch_scales = [&](int step) {
        Scales8 s;
        s.load(my_scales, block_of(step), nb);
        return s;
    };

    f32x16 acc[FJ][FI];
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
        for (int i = 0; i < FI; ++i) acc[j][i] = f32x16{};

    const int r = lane % 32, h = lane / 32;
    auto multiply = [&](const char *lds, const uint64_t *scales) {
        const char *p = lds + (wi + r) * 128, *q = lds + P_BYTES + (wj + r) * 128;
        uint32_t ps[FI], qs[FJ];
#pragma unroll
        for (int i = 0; i < FI; ++i) ps[i] = ((const uint32_t *)(scales + wi + 32 * i + r))[h];
#pragma unroll
        for (int j = 0; j < FJ; ++j) qs[j] = ((const uint32_t *)(scales + BI + wj + 32 * j + r))[h];
        // the four blocks of a lane's half row; the number of the scale is part of the
        // instruction
#define ZS_MX_QUARTER(S)                                                                       \
    {                                                                                          \
        const int at = ((4 * h + S) ^ (r >> 1 & 7)) << 4;                                      \
        i32x8 pf[FI], qf[FJ];                                                                  \
        _Pragma("unroll") for (int i = 0; i < FI; ++i) pf[i] =                                 \
            codes4(*(const u32x4 *)(p + i * 4096 + at));                                       \
        _Pragma("unroll") for (int j = 0; j < FJ; ++j) qf[j] =                                 \
            codes4(*(const u32x4 *)(q + j * 4096 + at));                                       \
        _Pragma("unroll") for (int j = 0; j < FJ; ++j) _Pragma("unroll") for (int i = 0; i < FI; \
                                                                              ++i) acc[j][i] = \
            __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(qf[j], pf[i], acc[j][i], 4, 4, S,  \
                                                            (int)qs[j], S, (int)ps[i]);        \
    }
        ZS_MX_QUARTER(0)
        ZS_MX_QUARTER(1)
        ZS_MX_QUARTER(2)
        ZS_MX_QUARTER(3)
#undef ZS_MX_QUARTER
    };

    if (steps > 0) {
        fetch(lds0, 0);
        scales0[tid] = fetch_scales(0).value();
    }
    // two steps a turn: a split ends with a whole turn, or with the row, past which all is 0
#pragma unroll 1
    for (int step = 0; step < steps; step += 2) {
        stage_ready<0>();
        fetch(lds1, step + 1);
        Scales8 s = fetch_scales(step + 1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(lds0, scales0);
        scales1[tid] = s.value();
        stage_ready<0>();
        fetch(lds0, step + 2);
        s = fetch_scales(step + 2);
        __builtin_amdgcn_sched_barrier(0);
        multiply(lds1, scales1);
        scales0[tid] = s.value();
    }
    stage_ready<0>();
    constexpr int HALF = WI * WJ / 2, SCRATCH = (P_BYTES + Q_BYTES) / HALF;
    static_assert(SCRATCH >= scratch_bytes(KG, FI * FJ), "scratch");
    auto scratch = [&](int g, int w) {
        return (w < HALF ? all0[g] : all1[g]) + w % HALF * SCRATCH;
    };
    if (join_groups<KG>(acc, scratch, group, wave, lane))
        finish_tile<BI, BJ, WI, WJ>(a, acc, tile, split, i0, j0, wi, wj, wave, lane,
                                    (uint32_t *)all_scales0, scratch(0, wave));
}

// ------------------------------------- bf16 against blocks, rows in full chunks

// A bf16 operand that DMA can take to LDS: rows a multiple of 16 bytes apart, and the
// rows of a tile (or of a step) inside the reach of a 32-bit offset.

// y = x w^T.  x goes through LDS by DMA, four steps deep.  w's codes stay packed: a lane
// loads the block that it multiplies straight into registers, three steps ahead, and
// widens it there, so LDS carries only x.  Half a wave (32 rows of w) takes one of a
// step's two blocks, and the four instructions of a step its four words.
//
// 8192 x 11008 of depth 4096 0.60 ms (1.23 PFLOP/s; codes widened on their way into LDS 0.97),
// the matrix pipe busy 73 % of the time and LDS 20 %, at a clock that the load holds at 1.6 GHz.
// Fragments read an instruction ahead by hand (0.66), raised wave priority around the matrix
// instructions (0.62) and staggered steps (0.65) were no faster.
template <int BI, int BJ, int WI, int WJ, int KG, bool F8>
__global__ __launch_bounds__(WI *WJ *KG *kWave, 2) void mx_tile_rows(MxProductArgs a) {
    constexpr int NT = WI * WJ * kWave;
    constexpr int FI = BI / WI / 32, FJ = BJ / WJ / 32;
    constexpr int EACH = BI * 8 / NT;
    constexpr int W = F8 ? 2 : 1;
    __shared__ __attribute__((aligned(128))) char all0[KG][BI * 128];
    __shared__ __attribute__((aligned(128))) char all1[KG][BI * 128];
    __shared__ __attribute__((aligned(128))) char all2[KG][BI * 128];
    __shared__ __attribute__((aligned(128))) char all3[KG][BI * 128];

    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
    const int tid = threadIdx.x % NT, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    char *lds0 = all0[group], *lds1 = all1[group], *lds2 = all2[group], *lds3 = all3[group];
    const int split = blockIdx.x % a.splits;
    int ti, tj;
    tile_of(blockIdx.x / a.splits, a.tiles_i, a.tiles_j, &ti, &tj);
    const int tile = tj * a.tiles_i + ti, i0 = ti * BI, j0 = tj * BJ;
    const int wi = wave % WI * (BI / WI), wj = wave / WI * (BJ / WJ);
    const int nb = (int)a.q.nb;
    const int first = (split * KG + group) * a.split_steps;
    const int steps = group_steps<KG>(a, kStep, split);
    const int r = lane % 32, h = lane / 32;

    const uint32_t row_bytes = (uint32_t)a.ldp * 2u;
    const auto p_buf =
        buffer_of(a.p + (int64_t)i0 * a.ldp, (uint32_t)min(a.I - i0, BI) * row_bytes);
    const int row = wave * 8 + lane / 8, chunk = (lane % 8) ^ (row >> 1 & 7);
    const uint32_t p_off = (uint32_t)row * row_bytes + (uint32_t)chunk * 16u;
    const uint8_t *codes[FJ];
    const uint8_t *scales[FJ];
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
        const int64_t at = (int64_t)min(j0 + wj + 32 * j + r, a.J - 1) * nb;
        codes[j] = a.q.codes + at * (16 * W);
        scales[j] = a.q.scales + at;
    }

    auto fetch = [&](char *lds, int step) {
        const int c = (first + step) * kStep;
        // whole chunks only: the rest of a row is added at the end
        const uint32_t off = c + chunk * 8 + 8 <= a.C ? p_off + (uint32_t)c * 2u : kNowhere;
#pragma unroll
        for (int k = 0; k < EACH; ++k)
            dma16(p_buf, lds + (k * (NT / 8) + wave * 8) * 128,
                  off + (uint32_t)(k * (NT / 8)) * row_bytes);
    };
    struct Codes {
        u32x4 v[FJ][W];
    };
    auto fetch_codes = [&](int step) {
        Codes q;
        const int block = min((first + step) * 2 + h, nb - 1);
#pragma unroll
        for (int j = 0; j < FJ; ++j)
#pragma unroll
            for (int w = 0; w < W; ++w) q.v[j][w] = ((const u32x4 *)codes[j])[block * W + w];
        return q;
    };

    f32x16 acc[FJ][FI];
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
        for (int i = 0; i < FI; ++i) acc[j][i] = f32x16{};

    auto multiply = [&](const char *lds, const Codes &q, const float (&s)[FJ]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            bf16x8 pf[FI], qf[FJ];
#pragma unroll
            for (int i = 0; i < FI; ++i)
                pf[i] = *(const bf16x8 *)(lds + at_rows(wi + 32 * i + r, 4 * h + k));
#pragma unroll
            for (int j = 0; j < FJ; ++j) {
                if constexpr (F8)
                    qf[j] = __builtin_bit_cast(
                        bf16x8, widen_fp8(q.v[j][k / 2][k % 2 * 2], q.v[j][k / 2][k % 2 * 2 + 1],
                                          s[j]));
                else
                    qf[j] = __builtin_bit_cast(bf16x8, widen_fp4(q.v[j][0][k], s[j]));
            }
#pragma unroll
            for (int j = 0; j < FJ; ++j)
#pragma unroll
                for (int i = 0; i < FI; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qf[j], pf[i], acc[j][i], 0,
                                                                        0, 0);
        }
    };
    // what a row holds past its last whole chunk, fewer than 8 elements
    const int whole = a.C & ~7;
    if (whole < a.C && split == 0 && group == 0) {
        const int at = whole % kMxBlock / 8;
#pragma unroll
        for (int j = 0; j < FJ; ++j) {
            const float s = scale_of(scales[j][whole / kMxBlock]);
            const uint32_t *w =
                (const uint32_t *)(codes[j] + (int64_t)(whole / kMxBlock) * (16 * W)) + at * W;
            u32x4 qf = {0, 0, 0, 0};
            if (h == 0) {
                if constexpr (F8)
                    qf = widen_fp8(w[0], w[1], s);
                else
                    qf = widen_fp4(w[0], s);
            }
#pragma unroll
            for (int i = 0; i < FI; ++i) {
                u32x4 pf = {0, 0, 0, 0};
                const uint16_t *x =
                    a.p + (int64_t)min(i0 + wi + 32 * i + r, a.I - 1) * a.ldp + whole;
                if (h == 0)
                    for (int e = 0; e < a.C - whole; ++e)
                        pf[e / 2] |= (uint32_t)x[e] << (16 * (e % 2));
                acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    __builtin_bit_cast(bf16x8, qf), __builtin_bit_cast(bf16x8, pf), acc[j][i], 0,
                    0, 0);
            }
        }
    }

    // the scales of a turn of four steps, and the next
    uint64_t now[FJ];
    Scales8 next[FJ];
#pragma unroll
    for (int j = 0; j < FJ; ++j) {
        next[j].load(scales[j], first * 2, nb);
        now[j] = next[j].value();
    }
    // fp8 codes take twice the registers, and are loaded a step later
    constexpr int FAR = F8 ? 2 : 3;
    Codes q0, q1, q2, q3;
    // the transfers first: the waits below count on what follows them
    fetch(lds0, 0);
    fetch(lds1, 1);
    fetch(lds2, 2);
    in_order();
    q0 = fetch_codes(0);
    q1 = fetch_codes(1);
    if constexpr (FAR > 2) q2 = fetch_codes(2);
    in_order();
    // Each step issues EACH transfers to LDS and FJ * W loads of codes; those of two steps may
    // be on their way while one is multiplied, and before the loop at least as many operations
    // follow a step's transfers.
    constexpr int AHEAD = 2 * EACH + (F8 ? 1 : 2) * FJ * W;
#define ZS_MX_STEP(T, HERE, Q, NEXT, QN)                                    \
    {                                                                       \
        stage_ready<AHEAD>();                                               \
        fetch(NEXT, step + T + 3);                                          \
        QN = fetch_codes(step + T + FAR);                                   \
        __builtin_amdgcn_sched_barrier(0);                                  \
        float s[FJ];                                                        \
        _Pragma("unroll") for (int j = 0; j < FJ; ++j) s[j] =               \
            scale_of((uint32_t)(now[j] >> (16 * T)) >> (8 * h) & 255u);     \
        multiply(HERE, Q, s);                                               \
    }
#pragma unroll 1
    for (int step = 0; step < steps; step += 4) {
#pragma unroll
        for (int j = 0; j < FJ; ++j) next[j].load(scales[j], (first + step) * 2 + 8, nb);
        if constexpr (F8) {
            ZS_MX_STEP(0, lds0, q0, lds3, q2)
            ZS_MX_STEP(1, lds1, q1, lds0, q3)
            ZS_MX_STEP(2, lds2, q2, lds1, q0)
            ZS_MX_STEP(3, lds3, q3, lds2, q1)
        } else {
            ZS_MX_STEP(0, lds0, q0, lds3, q3)
            ZS_MX_STEP(1, lds1, q1, lds0, q0)
            ZS_MX_STEP(2, lds2, q2, lds1, q1)
            ZS_MX_STEP(3, lds3, q3, lds2, q2)
        }
#pragma unroll
        for (int j = 0; j < FJ; ++j) now[j] = next[j].value();
    }
#undef ZS_MX_STEP
    stage_ready<0>();
    __shared__ uint32_t shared;
    constexpr int QUARTER = WI * WJ / 4, SCRATCH = BI * 128 / QUARTER;
    static_assert(SCRATCH >= scratch_bytes(KG, FI * FJ), "scratch");
    auto scratch = [&](int g, int w) {
        char *p = w / QUARTER == 0   ? all0[g]
                  : w / QUARTER == 1 ? all1[g]
                  : w / QUARTER == 2 ? all2[g]
                                     : all3[g];
        return p + w % QUARTER * SCRATCH;
    };
    if (join_groups<KG>(acc, scratch, group, wave, lane))
        finish_tile<BI, BJ, WI, WJ>(a, acc, tile, split, i0, j0, wi, wj, wave, lane, &shared,
                                    scratch(0, wave));
}

// dx = dy w and dw = dy^T x: the stored operand's rows run along the output, so a fragment
// needs it transposed.  A thread loads a block two steps ahead, widens it and puts it into
// LDS column-major, where the transposing reads take it from; dy goes there by DMA.  Both
// operands' addresses move with c, so a 32-bit offset never passes a step; rows past the
// last read as zeros.
//
// dgrad, 8192 x 4096 of depth 11008 0.58 ms (1.27 PFLOP/s, the matrix pipe busy 66 % of the time,
// LDS 42 %); wgrad, 4096 x 11008 of depth 8192 in fp8 0.68 (1.08; 55-59 % and 37 %).  LDS carries
// both operands and their writes here, and is what bounds the small tiles: 64 x 64 takes three
// times as long per product.  The compiler computes the size of a block's buffer in a vector
// register and wraps each of its loads in a loop over lanes, of one turn.
template <int BI, int BJ, int WI, int WJ, int KG, bool PC, bool F8>
__global__ __launch_bounds__(WI *WJ *KG *kWave, 2) void mx_tile_cols(MxProductArgs a) {
    constexpr int NT = WI * WJ * kWave;
    constexpr int FI = BI / WI / 32, FJ = BJ / WJ / 32;
    constexpr int EACH = BI * 8 / NT;
    constexpr int W = F8 ? 2 : 1;
    constexpr int ROW = BJ / kMxBlock;  // blocks of a tile's row
    static_assert(ROW * kStep <= NT, "a thread for each block of a step");
    __shared__ __attribute__((aligned(128))) char all_p0[KG][BI * 128];
    __shared__ __attribute__((aligned(128))) char all_p1[KG][BI * 128];
    __shared__ __attribute__((aligned(128))) char all_q0[KG][BJ * 128];
    __shared__ __attribute__((aligned(128))) char all_q1[KG][BJ * 128];

    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
    const int tid = threadIdx.x % NT, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    char *p0 = all_p0[group], *p1 = all_p1[group], *q0 = all_q0[group], *q1 = all_q1[group];
    const int split = blockIdx.x % a.splits;
    int ti, tj;
    tile_of(blockIdx.x / a.splits, a.tiles_i, a.tiles_j, &ti, &tj);
    const int tile = tj * a.tiles_i + ti, i0 = ti * BI, j0 = tj * BJ;
    const int wi = wave % WI * (BI / WI), wj = wave / WI * (BJ / WJ);
    const int first = (split * KG + group) * a.split_steps;
    const int steps = group_steps<KG>(a, kStep, split);

    // dy: rows of c (PC) or of i
    const uint32_t p_row = (uint32_t)a.ldp * 2u;
    const int64_t p_at = PC ? (int64_t)i0 * 2 : (int64_t)i0 * p_row;
    uint32_t p_off;
    int chunk = 0;
    if constexpr (PC) {
        // a wave's transfer k: whole rows of the tile, the 64-byte chunks permuted by c
        constexpr int LANES = BI / 8, ROWS = kWave / LANES;
        static_assert(ROWS >= 1, "a transfer holds whole rows");
        const int c = wave * ROWS + lane / LANES;
        // the permutation of a row is the same for every k: rows are NT / LANES apart
        const int byte = at_cols<BI>(c, lane % LANES * 16) - c * (BI * 2);
        p_off = (uint32_t)c * p_row + (uint32_t)byte;
    } else {
        const int row = wave * 8 + lane / 8;
        chunk = (lane % 8) ^ (row >> 1 & 7);
        p_off = (uint32_t)row * p_row + (uint32_t)chunk * 16u;
    }
    auto fetch = [&](char *lds, int step) {
        const int c0 = (first + step) * kStep;
        if constexpr (PC) {
            const int left = min(max(a.C - c0, 0), kStep);
            const auto buf =
                buffer_of((const char *)a.p + (int64_t)min(c0, a.C) * p_row + p_at,
                          left > 0 ? (uint32_t)(left - 1) * p_row + (uint32_t)(a.I - i0) * 2u : 0u);
#pragma unroll
            for (int k = 0; k < EACH; ++k)
                dma16(buf, lds + (k * NT + wave * kWave) * 16,
                      p_off + (uint32_t)(k * (NT / (BI / 8))) * p_row);
        } else {
            const auto buf =
                buffer_of((const char *)a.p + p_at, (uint32_t)min(a.I - i0, BI) * p_row);
            // whole chunks only: the rest of a row is a step of its own
            const uint32_t off = c0 + chunk * 8 + 8 <= a.C ? p_off + (uint32_t)c0 * 2u : kNowhere;
#pragma unroll
            for (int k = 0; k < EACH; ++k)
                dma16(buf, lds + (k * (NT / 8) + wave * 8) * 128,
                      off + (uint32_t)(k * (NT / 8)) * p_row);
        }
    };

    const uint32_t q_row = (uint32_t)a.q.nb;
    // the thread's block of a step: neighbours take up to four of a row
    constexpr int SIDE = ROW < 4 ? ROW : 4;
    const int qc = tid / SIDE % kStep, qb = tid % SIDE + tid / (SIDE * kStep) * SIDE;
    struct Block {
        u32x4 v[W];
        uint32_t scale;
    };
    auto fetch_block = [&](int c0) {
        const int left = min(max(a.C - c0, 0), kStep);
        const int64_t at = (int64_t)min(c0, a.C) * q_row;
        const int jb = j0 / kMxBlock;
        const auto codes = buffer_of(a.q.codes + (at + jb) * (16 * W),
                                     left > 0 ? ((uint32_t)left * q_row - jb) * (16u * W) : 0u);
        const auto scales =
            buffer_of(a.q.scales + at + jb, left > 0 ? (uint32_t)left * q_row - jb : 0u);
        const uint32_t off = (uint32_t)qc * q_row + (uint32_t)qb;
        Block b;
#pragma unroll
        for (int w = 0; w < W; ++w)
            b.v[w] = __builtin_amdgcn_raw_buffer_load_b128(codes, off * (16 * W) + 16 * w, 0, 0);
        b.scale = __builtin_amdgcn_raw_buffer_load_b8(scales, off, 0, 0);
        return b;
    };
    auto put_block = [&](char *lds, const Block &b) {
        if (ROW * kStep < NT && qb >= ROW) return;
        const float s = scale_of(b.scale);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            u32x4 v;
            if constexpr (F8)
                v = widen_fp8(b.v[w / 2][w % 2 * 2], b.v[w / 2][w % 2 * 2 + 1], s);
            else
                v = widen_fp4(b.v[0][w], s);
            *(u32x4 *)(lds + at_cols<BJ>(qc, qb * 64 + w * 16)) = v;
        }
    };

    f32x16 acc[FJ][FI];
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
        for (int i = 0; i < FI; ++i) acc[j][i] = f32x16{};
    auto multiply = [&](const char *p, const char *q) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            bf16x8 pf[FI], qf[FJ];
#pragma unroll
            for (int j = 0; j < FJ; ++j) qf[j] = frag_cols<BJ>(q, wj + 32 * j, s, lane);
#pragma unroll
            for (int i = 0; i < FI; ++i)
                pf[i] = PC ? frag_cols<BI>(p, wi + 32 * i, s, lane)
                           : frag_rows(p, wi + 32 * i, s, lane);
#pragma unroll
            for (int j = 0; j < FJ; ++j)
#pragma unroll
                for (int i = 0; i < FI; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qf[j], pf[i], acc[j][i], 0,
                                                                        0, 0);
            // the reads of a quarter stay in it: hoisted, they would take the registers of the
            // block two steps ahead (seven spilled, 7B wgrad 851 us instead of 675)
            if (F8) __builtin_amdgcn_sched_barrier(0);
        }
    };

    const int whole = a.C & ~7;
    if (!PC && whole < a.C && split == 0) {  // fewer than 8 c's past the last whole chunk
        const int c0 = group == 0 ? whole : a.C;  // the other groups add zeros
        PlainStage<BI, NT, false> rest;
        rest.load(a.p, a.ldp, i0, a.I, c0, a.C, tid);
        rest.store(p0, tid);
        put_block(q0, fetch_block(c0));
        __syncthreads();
        multiply(p0, q0);
        __syncthreads();
    }

    // A stage is ready when its transfers have ended; the loads of a block, W + 1 of them, are
    // issued after those, which the scheduling barriers keep so, and may go on.
    Block b0, b1;
    fetch(p0, 0);
    b0 = fetch_block(first * kStep);
    put_block(q0, b0);
    __builtin_amdgcn_sched_barrier(0);
    b1 = fetch_block((first + 1) * kStep);
    // two steps a turn: a split ends with a whole turn, or with c, past which all is 0
#pragma unroll 1
    for (int step = 0; step < steps; step += 2) {
        stage_ready<W + 1>();
        fetch(p1, step + 1);
        __builtin_amdgcn_sched_barrier(0);
        b0 = fetch_block((first + step + 2) * kStep);
        __builtin_amdgcn_sched_barrier(0);
        multiply(p0, q0);
        put_block(q1, b1);
        stage_ready<W + 1>();
        fetch(p0, step + 2);
        __builtin_amdgcn_sched_barrier(0);
        b1 = fetch_block((first + step + 3) * kStep);
        __builtin_amdgcn_sched_barrier(0);
        multiply(p1, q1);
        put_block(q0, b0);
    }
    stage_ready<0>();
    __shared__ uint32_t shared;
    constexpr int QUARTER = WI * WJ / 4, SCRATCH = (BI < BJ ? BI : BJ) * 128 / QUARTER;
    static_assert(SCRATCH >= scratch_bytes(KG, FI * FJ), "scratch");
    auto scratch = [&](int g, int w) {
        char *p = w / QUARTER == 0   ? all_p0[g]
                  : w / QUARTER == 1 ? all_p1[g]
                  : w / QUARTER == 2 ? all_q0[g]
                                     : all_q1[g];
        return p + w % QUARTER * SCRATCH;
    };
    if (join_groups<KG>(acc, scratch, group, wave, lane))
        finish_tile<BI, BJ, WI, WJ>(a, acc, tile, split, i0, j0, wi, wj, wave, lane, &shared,
                                    scratch(0, wave));
}

// ------------------------------------------------------- products of few rows

// Up to 16 MF rows of x: bound by the bytes of w, which every wave takes 16 NF rows of,
// 16 blocks (kTurn) at a time, the waves of a workgroup in turn along the row.  Of a turn
// the lanes of quarter g load the blocks 4 u + g, u = 0 .. 3: 64 neighbouring bytes of a row
// at a time.  The sums of the waves are joined in LDS, those of the workgroups that share
// a strip in the workspace.  One row, N = 11008, K = 4096 9.0 us (24 MB, 2.6 TB/s, the caches
// holding w); 8 rows of fp4, N = 28672, K = 8192 32 us (125 MB, 3.9 TB/s, from memory).
constexpr int kTurn = 16;

struct __attribute__((packed, aligned(1))) Bytes16 { u32x4 v; };

template <int LEFT, bool F8, int MF, int NF, int WAVES>
__global__ __launch_bounds__(WAVES *kWave) void mx_few(MxProductArgs a) {
    constexpr bool PLAIN = LEFT == kLeftRows, P8 = LEFT == kLeftFp8;
    constexpr bool SCALED = LEFT == kLeftFp4 && !F8;
    constexpr int WQ = F8 ? 2 : 1, WP = P8 ? 2 : 1;
    constexpr int OUT = NF * 16 * MF * 16;
    __shared__ float sums[WAVES][OUT];
    __shared__ uint32_t shared;

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int strip = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
    const int j0 = strip * (NF * 16);
    const int r = lane % 16, g = lane / 16;
    const int nb = (int)a.q.nb;
    const int turns = min((nb + kTurn - 1) / kTurn, (split + 1) * a.split_steps);

    const uint8_t *q_codes[NF], *q_scales[NF];
#pragma unroll
    for (int n = 0; n < NF; ++n) {
        const int64_t at = (int64_t)min(j0 + 16 * n + r, a.J - 1) * nb;
        q_codes[n] = a.q.codes + at * (16 * WQ);
        q_scales[n] = a.q.scales + at;
    }
    const uint16_t *p_rows[MF];
    const uint8_t *p_codes[MF], *p_scales[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
        const int64_t row = min(16 * m + r, a.I - 1);
        p_rows[m] = a.p + row * a.ldp;
        p_codes[m] = a.px.codes + row * nb * (16 * WP);
        p_scales[m] = a.px.scales + row * nb;
    }

    f32x4 acc[NF][MF];
#pragma unroll
    for (int n = 0; n < NF; ++n)
#pragma unroll
        for (int m = 0; m < MF; ++m) acc[n][m] = f32x4{};

    struct Blocks {
        u32x4 code[NF][4][WQ];
        u32x4 scale[NF];
    };
    // the blocks of a turn that lies inside the row
    auto fetch = [&](int turn) {
        Blocks b;
#pragma unroll
        for (int n = 0; n < NF; ++n) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int w = 0; w < WQ; ++w)
                    b.code[n][u][w] =
                        ((const u32x4 *)q_codes[n])[(turn * kTurn + 4 * u + g) * WQ + w];
            b.scale[n] = ((const Bytes16 *)(q_scales[n] + turn * kTurn))->v;
        }
        return b;
    };
    // one block of every row: q's codes, and the block of x, whose scale is ps
    auto multiply = [&](const u32x4 (&code)[NF][WQ], const uint32_t (&qs)[NF],
                        const u32x4 (&pv)[MF][PLAIN ? 4 : WP], const uint32_t (&ps)[MF]) {
        if constexpr (SCALED) {
#pragma unroll
            for (int n = 0; n < NF; ++n)
#pragma unroll
                for (int m = 0; m < MF; ++m)
                    acc[n][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        codes4(code[n][0]), codes4(pv[m][0]), acc[n][m], 4, 4, 0, (int)qs[n], 0,
                        (int)ps[m]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                bf16x8 qf[NF], pf[MF];
#pragma unroll
                for (int n = 0; n < NF; ++n) {
                    const float s = scale_of(qs[n]);
                    if constexpr (F8)
                        qf[n] = __builtin_bit_cast(
                            bf16x8, widen_fp8(code[n][k / 2][k % 2 * 2],
                                              code[n][k / 2][k % 2 * 2 + 1], s));
                    else
                        qf[n] = __builtin_bit_cast(bf16x8, widen_fp4(code[n][0][k], s));
                }
#pragma unroll
                for (int m = 0; m < MF; ++m) {
                    const float s = scale_of(ps[m]);
                    if constexpr (PLAIN)
                        pf[m] = __builtin_bit_cast(bf16x8, pv[m][k]);
                    else if constexpr (P8)
                        pf[m] = __builtin_bit_cast(
                            bf16x8,
                            widen_fp8(pv[m][k / 2][k % 2 * 2], pv[m][k / 2][k % 2 * 2 + 1], s));
                    else
                        pf[m] = __builtin_bit_cast(bf16x8, widen_fp4(pv[m][0][k], s));
                }
#pragma unroll
                for (int n = 0; n < NF; ++n)
#pragma unroll
                    for (int m = 0; m < MF; ++m)
                        acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf[n], pf[m],
                                                                            acc[n][m], 0, 0, 0);
            }
        }
    };

    // turns inside the row, the next one's blocks on their way while one is multiplied
    const int inside = min(turns, (PLAIN ? a.C / kMxBlock : nb) / kTurn);
    int turn = split * a.split_steps + wave;
    if (turn < inside) {
        Blocks now = fetch(turn);
        while (true) {
            const bool more = turn + WAVES < inside;
            Blocks next;
            if (more) next = fetch(turn + WAVES);
            u32x4 xs[MF];
            if constexpr (!PLAIN) {
#pragma unroll
                for (int m = 0; m < MF; ++m)
                    xs[m] = ((const Bytes16 *)(p_scales[m] + turn * kTurn))->v;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int block = turn * kTurn + 4 * u + g;
                u32x4 pv[MF][PLAIN ? 4 : WP], code[NF][WQ];
                uint32_t qs[NF], ps[MF];
#pragma unroll
                for (int m = 0; m < MF; ++m) {
                    ps[m] = 127;
                    if constexpr (PLAIN) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            pv[m][k] =
                                ((const Any16 *)(p_rows[m] + (int64_t)block * kMxBlock))[k].v;
                    } else {
#pragma unroll
                        for (int w = 0; w < WP; ++w)
                            pv[m][w] = ((const u32x4 *)p_codes[m])[block * WP + w];
                        ps[m] = xs[m][u] >> (8 * g) & 255u;
                    }
                }
#pragma unroll
                for (int n = 0; n < NF; ++n) {
#pragma unroll
                    for (int w = 0; w < WQ; ++w) code[n][w] = now.code[n][u][w];
                    qs[n] = now.scale[n][u] >> (8 * g) & 255u;
                }
                multiply(code, qs, pv, ps);
            }
            if (!more) break;
            turn += WAVES;
            now = next;
        }
        turn += WAVES;
    }
    // turns that the row ends in, block by block and element by element
    for (; turn < turns; turn += WAVES)
        for (int u = 0; u < 4 && turn * kTurn + 4 * u < nb; ++u) {
            const int block = turn * kTurn + 4 * u + g;
            const bool in = block < nb;
            u32x4 pv[MF][PLAIN ? 4 : WP], code[NF][WQ];
            uint32_t qs[NF], ps[MF];
#pragma unroll
            for (int m = 0; m < MF; ++m) {
                ps[m] = 127;
                if constexpr (PLAIN) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = block * kMxBlock + 8 * k;
                        pv[m][k] = u32x4{0, 0, 0, 0};
                        if (c + 8 <= a.C)
                            pv[m][k] = ((const Any16 *)(p_rows[m] + c))->v;
                        else
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (c + e < a.C)
                                    pv[m][k][e / 2] |= (uint32_t)p_rows[m][c + e] << (16 * (e % 2));
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < WP; ++w)
                        pv[m][w] = in ? ((const u32x4 *)p_codes[m])[block * WP + w]
                                      : u32x4{0, 0, 0, 0};
                    if (in) ps[m] = p_scales[m][block];
                }
            }
#pragma unroll
            for (int n = 0; n < NF; ++n) {
#pragma unroll
                for (int w = 0; w < WQ; ++w)
                    code[n][w] = in ? ((const u32x4 *)q_codes[n])[block * WQ + w]
                                    : u32x4{0, 0, 0, 0};
                qs[n] = in ? q_scales[n][block] : 127;
            }
            multiply(code, qs, pv, ps);
        }

    // lane: i = lane % 16, four j's from 4 (lane / 16)
#pragma unroll
    for (int n = 0; n < NF; ++n)
#pragma unroll
        for (int m = 0; m < MF; ++m)
            *(f32x4 *)&sums[wave][(m * 16 + r) * (NF * 16) + n * 16 + 4 * g] = acc[n][m];
    __syncthreads();
    float *mine = a.parts + ((int64_t)strip * a.splits + split) * OUT;
    const int rows = min(a.I, MF * 16);
    for (int o = tid; o < rows * NF * 16; o += WAVES * kWave) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v += sums[w][o];
        if (a.splits > 1)
            __hip_atomic_store(mine + o, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        else
            put1(a, o / (NF * 16), j0 + o % (NF * 16), v);
    }
    if (a.splits == 1 || !last_split(a.counters + strip, a.splits, &shared)) return;
    const float *parts = a.parts + (int64_t)strip * a.splits * OUT;
    for (int o = tid; o < rows * NF * 16; o += WAVES * kWave) {
        float v = 0.0f;
        for (int k = 0; k < a.splits; ++k)  // always in this order
            v += __hip_atomic_load(parts + (int64_t)k * OUT + o, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        put1(a, o / (NF * 16), j0 + o % (NF * 16), v);
    }
}

// Tiles of out and splits of c for a kernel of bi x bj tiles whose steps take `depth` c's
// and whose splits are `groups` parts of whole turns of `turn` steps each, `least` steps at
// least for a part: below that the join costs more than the shorter part saves. Eight, but
// four for the fp4 kernel, whose steps are deeper. Measured with eight and with four: fp4
// product 64 x 4096 of depth 8192 19.8 and 14.4 us (depth 4096 10.7 both); linear 32 x 4096
// of depth 4096 11.6 and 13.4; dgrad 64 x 4096 of depth 4096 18.7 and 21.4, though 128 x 768
// of depth 2048 12.2 and 10.7.
void plan(MxProductArgs *a, int bi, int bj, int groups, int depth, int turn, int least,
          void *workspace, const MxDevice &dev) {
    a->tiles_i = (a->I + bi - 1) / bi;
    a->tiles_j = (a->J + bj - 1) / bj;
    const int64_t tiles = (int64_t)a->tiles_i * a->tiles_j;
    const int steps = (a->C + depth - 1) / depth;
    int64_t splits = 1;
    // a workgroup per compute unit, two where they are small
    const int64_t most = groups == 1 && bi * bj <= 64 * 128 ? 2 * dev.cus : dev.cus;
    if (workspace && tiles < most && most <= kMxCounters) {
        splits = most / tiles;
        splits = splits < steps / (least * groups) ? splits : steps / (least * groups);
        const int64_t room = kMxPartBytes / (tiles * bi * bj * 4);
        splits = splits < room ? splits : room;
        splits = splits > 1 ? splits : 1;
    }
    const int64_t parts = splits * groups;
    a->split_steps = steps > 0 ? (int)((steps + parts - 1) / parts + turn - 1) / turn * turn : 0;
    const int64_t each = (int64_t)a->split_steps * groups;
    a->splits = steps > 0 ? (int)((steps + each - 1) / each) : 1;
    a->counters = (uint32_t *)workspace;
    a->parts = (float *)((char *)workspace + kMxCounterBytes);
}

// The size of the tiles, by the elements of out (cus of 256 in the figures below; in us, each
// with the next smaller or larger choice).  Tiles of 256 x 256 from a tile per compute unit
// on: bf16 by fp4, K = 4096, 4096 x 4096 107 against 138 in tiles of 128, 2048 x 4096 81 and 71;
// dgrad 111 and 137, 91 and 72; fp4 48 and 60, 38 and 33; any strides 130 and 167, 115 and 89.
// The elements alone count, though an output of few rows or columns leaves part of such a tile
// empty: 64 rows, N = 262144 340, N = 261888 (in tiles of 64 x 128) 212.
constexpr int64_t kTile256 = 256 * 256;
// Tiles of 128 x 128, more than a compute unit each, in one wave group; up to that many in two,
// since a wave per SIMD hides little: dgrad 2048 x 4096 (512 tiles) 72 in one, 79 in two groups,
// 1024 x 4096 (256) 45 and 41; fp4 33 and 36, 22 and 20; any strides 89 and 101, 56 and 52, and
// 2001 x 3001 (384) 23 and 30.
bool many_tiles(const MxProductArgs &a, const MxDevice &dev) {
    return (int64_t)((a.I + 127) / 128) * ((a.J + 127) / 128) > dev.cus;
}
// Below that, tiles of 64 x 64 in several wave groups leave fewer sums to be joined through
// memory: fp4 512 x 4096 16 in tiles of 128, 23 so, 256 x 4096 14 and 12; any strides 33 and 51, 27
// and 26.
constexpr int64_t kTile64 = 6 * 1024;
// Long sums are worth large tiles all the same: any strides, 256 x 2048 of depth 16384 40 in
// tiles of 128, 45 in tiles of 64, 256 x 4096 of depth 4096 27 and 26.
constexpr int kLong = 8192;
// Rows of w from which up to 64 rows of x take tiles of 128 of them instead of 64: 64 rows,
// N = 28672 53 and 68 (fp4 38 and 45), N = 16384 24 and 21 (16 and 15).
constexpr int64_t kWideRows = 96;

// Tiles of 256 x 256 are 2^21 at most, and where smaller ones are taken there are fewer.
dim3 grid_of(const MxProductArgs &a) {
    return dim3((uint32_t)((int64_t)a.tiles_i * a.tiles_j * a.splits));
}

template <int BI, int BJ, int WI, int WJ, int KG, int LEFT, int RIGHT>
hipError_t run_tile(MxProductArgs a, void *workspace, const MxDevice &dev, hipStream_t stream) {
    plan(&a, BI, BJ, KG, kStep, 1, 8, workspace, dev);
    mx_tile<BI, BJ, WI, WJ, KG, LEFT, RIGHT>
        <<<grid_of(a), dim3(WI * WJ * KG * kWave), 0, stream>>>(a);
    return hipGetLastError();
}

template <int BI, int BJ, int WI, int WJ, int KG>
hipError_t run_fp4(MxProductArgs a, void *workspace, const MxDevice &dev, hipStream_t stream) {
    plan(&a, BI, BJ, KG, kStep4, 2, 4, workspace, dev);
    mx_tile_fp4<BI, BJ, WI, WJ, KG>
        <<<grid_of(a), dim3(WI * WJ * KG * kWave), 0, stream>>>(a);
    return hipGetLastError();
}

template <int BI, int BJ, int WI, int WJ, int KG, bool F8>
hipError_t run_rows(MxProductArgs a, void *workspace, const MxDevice &dev, hipStream_t stream) {
    plan(&a, BI, BJ, KG, kStep, 4, 8, workspace, dev);
    mx_tile_rows<BI, BJ, WI, WJ, KG, F8>
        <<<grid_of(a), dim3(WI * WJ * KG * kWave), 0, stream>>>(a);
    return hipGetLastError();
}

// Whether DMA can take the bf16 operand: 16-byte chunks of its rows at 16-byte addresses,
// `rows` of them within a 32-bit offset.
bool dma_takes(const MxProductArgs &a, int64_t rows) {
    return (uintptr_t)a.p % 16 == 0 && a.ldp % 8 == 0 && mx_rows_reach(a.ldp, rows);
}

// Rows of x up to which the kernel of few rows is taken: where a tiled kernel takes the
// operands, too, it is faster from there on (K = 8192, N = 28672, bf16 x: 8 rows 38 us here and 46
// in tiles of 32, 16 rows 42 and 47, 32 rows 129 and 48; fp4 x: 16 rows 35 and 40, 32 rows 50
// and 41).  Where only the tiles through registers take them the border that suits depends on the
// size of w, and 64 suits small ones (64 rows here and in those tiles: bf16 x at odd strides,
// N = 1003, K = 2001 12.4 and 12.6, N = 4096, K = 4096 52 and 16, N = 28672, K = 8192 414 and 101;
// fp8 x, the latter two 12.6 and 15.9, 149 and 91).
constexpr int kFewRows = 64, kFewTiled = 16;

template <int LEFT, bool F8, int MF, int NF, int WAVES>
hipError_t run_few(MxProductArgs a, void *workspace, const MxDevice &dev, hipStream_t stream) {
    const int64_t strips = (a.J + NF * 16 - 1) / (NF * 16);
    const int turns = (int)((a.q.nb + kTurn - 1) / kTurn);
    int64_t splits = 1;
    // strips that leave compute units idle are split, two turns of each wave at least
    if (workspace && strips <= kMxCounters && strips < dev.cus) {
        splits = dev.cus / strips;
        splits = splits < turns / (2 * WAVES) ? splits : turns / (2 * WAVES);
        splits = splits > 1 ? splits : 1;
    }
    a.split_steps = (int)((turns + splits - 1) / splits);
    a.splits = a.split_steps > 0 ? (turns + a.split_steps - 1) / a.split_steps : 1;
    a.counters = (uint32_t *)workspace;
    a.parts = (float *)((char *)workspace + kMxCounterBytes);
    mx_few<LEFT, F8, MF, NF, WAVES>
        <<<dim3((uint32_t)(strips * a.splits)), dim3(WAVES * kWave), 0, stream>>>(a);
    return hipGetLastError();
}

// Strips of 64 columns read x a quarter as often as strips of 16, and leave a quarter of the
// workgroups: bf16 x, K = 8192, N = 28672, 16 rows 42 us against 72, one row 36 and 38; K = 4096,
// N = 11008, 16 rows 11.2 and 16.4, one row 10.3 and 9.2; N = 4096, 10.9 and 6.8.  With fp8 w, in
// the same order, 67 and 84, 63 and 60; 14.9 and 19.7, 14.0 and 13.8; 14.7 and 8.5.  An x in blocks
// is short: strips of 16 are as fast or faster, up to the 2^23 of 512 threads each that are more
// than a grid's dimension holds.
constexpr int64_t kMostStrips = (int64_t(1) << 23) - 1;

template <int LEFT, bool F8>
hipError_t choose_few(const MxProductArgs &a, void *workspace, const MxDevice &dev,
                      hipStream_t stream) {
    const int64_t wide = LEFT != kLeftRows ? 16 * kMostStrips + 1 : (a.I > 4 ? 32 : 64) * dev.cus;
    if constexpr (LEFT == kLeftRows)
        if (a.J >= wide && a.I <= 16)
            return run_few<LEFT, F8, 1, 4, 4>(a, workspace, dev, stream);
    if (a.J >= wide && a.I <= 32)
        return run_few<LEFT, F8, 2, 2, 4>(a, workspace, dev, stream);
    if (a.J >= wide) return run_few<LEFT, F8, 4, 2, 4>(a, workspace, dev, stream);
    if (a.I <= 16) return run_few<LEFT, F8, 1, 1, 8>(a, workspace, dev, stream);
    if (a.I <= 32) return run_few<LEFT, F8, 2, 1, 8>(a, workspace, dev, stream);
    return run_few<LEFT, F8, 4, 1, 8>(a, workspace, dev, stream);
}

// Here one wave group is as good as two in tiles of 128 (512 x 4096 26 and 29, 1024 x 4096 39 and
// 41): the codes' way through registers hides more.
template <bool F8>
hipError_t choose_rows(const MxProductArgs &a, void *workspace, const MxDevice &dev,
                       hipStream_t stream) {
    const int64_t out = (int64_t)a.I * a.J;
    if (out >= kTile256 * dev.cus)
        return run_rows<256, 256, 2, 4, 1, F8>(a, workspace, dev, stream);
    if (a.I <= 32) return run_rows<32, 128, 1, 4, 2, F8>(a, workspace, dev, stream);
    if (a.I <= 64 && a.J >= kWideRows * dev.cus)
        return run_rows<64, 128, 1, 4, 1, F8>(a, workspace, dev, stream);
    if (out >= kTile64 * dev.cus || (a.I > 64 && a.C >= kLong))
        return run_rows<128, 128, 2, 2, 1, F8>(a, workspace, dev, stream);
    return run_rows<64, 64, 2, 2, 2, F8>(a, workspace, dev, stream);
}

template <int BI, int BJ, int WI, int WJ, int KG, bool PC, bool F8>
hipError_t run_cols(MxProductArgs a, void *workspace, const MxDevice &dev, hipStream_t stream) {
    plan(&a, BI, BJ, KG, kStep, 2, 8, workspace, dev);
    mx_tile_cols<BI, BJ, WI, WJ, KG, PC, F8>
        <<<grid_of(a), dim3(WI * WJ * KG * kWave), 0, stream>>>(a);
    return hipGetLastError();
}

// The transposing reads make small tiles dear: 64 x 64 is for small and shallow outputs only
// (dgrad 1024 x 768 of depth 768 9.6, in tiles of 128 10.6; wgrad 768 x 768 of depth 2048 17.5
// and 17.7, of depth 8192 53 and 28; 1024 x 1024 of depth 4096 28 and 26).
constexpr int64_t kTile64Cols = 4 * 1024;
constexpr int kLongCols = 4096;

template <bool PC, bool F8>
hipError_t choose_cols(const MxProductArgs &a, void *workspace, const MxDevice &dev,
                       hipStream_t stream) {
    const int64_t out = (int64_t)a.I * a.J;
    if (out >= kTile256 * dev.cus)
        return run_cols<256, 256, 2, 4, 1, PC, F8>(a, workspace, dev, stream);
    if (many_tiles(a, dev))
        return run_cols<128, 128, 2, 2, 1, PC, F8>(a, workspace, dev, stream);
    if (out >= kTile64Cols * dev.cus || a.C >= kLongCols)
        return run_cols<128, 128, 2, 2, 2, PC, F8>(a, workspace, dev, stream);
    return run_cols<64, 64, 2, 2, 4, PC, F8>(a, workspace, dev, stream);
}

hipError_t choose_fp4(const MxProductArgs &a, void *workspace, const MxDevice &dev,
                      hipStream_t stream) {
    const int64_t out = (int64_t)a.I * a.J;
    if (out >= kTile256 * dev.cus)
        return run_fp4<256, 256, 2, 4, 1>(a, workspace, dev, stream);
    if (a.I <= 32) return run_fp4<32, 128, 1, 4, 1>(a, workspace, dev, stream);
    if (a.I <= 64 && a.J >= kWideRows * dev.cus)
        return run_fp4<64, 128, 1, 4, 1>(a, workspace, dev, stream);
    if (many_tiles(a, dev))
        return run_fp4<128, 128, 2, 2, 1>(a, workspace, dev, stream);
    if (out >= kTile64 * dev.cus)
        return run_fp4<128, 128, 2, 2, 2>(a, workspace, dev, stream);
    return run_fp4<64, 64, 2, 2, 4>(a, workspace, dev, stream);
}

template <int LEFT, int RIGHT>
hipError_t choose_tile(const MxProductArgs &a, void *workspace, const MxDevice &dev,
                       hipStream_t stream) {
    const int64_t out = (int64_t)a.I * a.J;
    if (out >= kTile256 * dev.cus)
        return run_tile<256, 256, 2, 4, 1, LEFT, RIGHT>(a, workspace, dev, stream);
    if (many_tiles(a, dev))
        return run_tile<128, 128, 2, 2, 1, LEFT, RIGHT>(a, workspace, dev, stream);
    if (out >= kTile64 * dev.cus || (a.I > 64 && a.C >= kLong))
        return run_tile<128, 128, 2, 2, 2, LEFT, RIGHT>(a, workspace, dev, stream);
    return run_tile<64, 64, 2, 2, 4, LEFT, RIGHT>(a, workspace, dev, stream);
}

// Matrices from the size of the L2 caches on are streamed: 6.7e7 bf16 elements to fp8 33 us
// against 37, and read back 30 and 40; 8.4e6 elements 9.9 either way.  The codes are, too, where
// the last-level cache cannot hold both: to fp4 and back 8.1e8 bf16 elements 651 and 678 us,
// 6.7e7 fp32 elements to fp8 and back 138 and 171, but 6.7e7 bf16 elements 69 and 63.
constexpr int64_t kStreamBytes = int64_t(1) << 25;
constexpr int64_t kStreamBoth = int64_t(1) << 28;

constexpr int64_t dtype_bytes(int dtype) { return dtype == ZS_DTYPE_FP32 ? 4 : 2; }

dim3 cast_grid(int64_t blocks) {
    const int64_t groups = (blocks + kCastBlocks - 1) / kCastBlocks;
    return dim3((uint32_t)(groups < kCastRow ? groups : kCastRow),
                (uint32_t)((groups + kCastRow - 1) / kCastRow));
}

template <int FMT, int DT>
hipError_t run_quantize(const MxCastArgs &a, hipStream_t stream) {
    const dim3 grid = cast_grid(a.blocks);
    const int64_t bytes = a.blocks * kMxBlock * dtype_bytes(DT);
    if (bytes + a.blocks * mx_block_bytes(FMT) >= kStreamBoth)
        mx_quantize<FMT, DT, 2><<<grid, dim3(kThreads), 0, stream>>>(a);
    else if (bytes >= kStreamBytes)
        mx_quantize<FMT, DT, 1><<<grid, dim3(kThreads), 0, stream>>>(a);
    else
        mx_quantize<FMT, DT, 0><<<grid, dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

template <int FMT, int DT>
hipError_t run_dequantize(const MxCastArgs &a, hipStream_t stream) {
    const dim3 grid = cast_grid(a.blocks);
    if (a.blocks * kMxBlock * dtype_bytes(DT) >= kStreamBytes)
        mx_dequantize<FMT, DT, true><<<grid, dim3(kThreads), 0, stream>>>(a);
    else
        mx_dequantize<FMT, DT, false><<<grid, dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(int format, int dtype, const MxCastArgs &a, hipStream_t stream) {
    switch (format * 3 + dtype) {
        case 0: return run_quantize<ZS_MX_FP4, ZS_DTYPE_BF16>(a, stream);
        case 1: return run_quantize<ZS_MX_FP4, ZS_DTYPE_FP16>(a, stream);
        case 2: return run_quantize<ZS_MX_FP4, ZS_DTYPE_FP32>(a, stream);
        case 3: return run_quantize<ZS_MX_FP8, ZS_DTYPE_BF16>(a, stream);
        case 4: return run_quantize<ZS_MX_FP8, ZS_DTYPE_FP16>(a, stream);
        default: return run_quantize<ZS_MX_FP8, ZS_DTYPE_FP32>(a, stream);
    }
}

hipError_t launch_mx_dequantize(int format, int dtype, const MxCastArgs &a, hipStream_t stream) {
    switch (format * 3 + dtype) {
        case 0: return run_dequantize<ZS_MX_FP4, ZS_DTYPE_BF16>(a, stream);
        case 1: return run_dequantize<ZS_MX_FP4, ZS_DTYPE_FP16>(a, stream);
        case 2: return run_dequantize<ZS_MX_FP4, ZS_DTYPE_FP32>(a, stream);
        case 3: return run_dequantize<ZS_MX_FP8, ZS_DTYPE_BF16>(a, stream);
        case 4: return run_dequantize<ZS_MX_FP8, ZS_DTYPE_FP16>(a, stream);
        default: return run_dequantize<ZS_MX_FP8, ZS_DTYPE_FP32>(a, stream);
    }
}

hipError_t launch_mx_product(MxLeft left, int right, MxProductArgs a, void *workspace,
                             const MxDevice &dev, hipStream_t stream) {
    constexpr int c4 = kRightFp4 | kRightCols, c8 = kRightFp8 | kRightCols;
    // what the kernels on whole chunks take
    const bool rows = left == kLeftRows && a.q.nb >= 8 && dma_takes(a, 256);
    const bool fp4 = left == kLeftFp4 && right == kRightFp4 && a.q.nb >= kStep4Blocks &&
                     a.q.nb * 16 * 256 < kMxReach;
    // dy^T's chunks lie along i, where a last one that is not whole could reach past the matrix
    const bool cols = right >= kRightCols && dma_takes(a, 256) &&
                      (left == kLeftRows || a.I % 8 == 0) && a.q.nb * 32 * kStep < kMxReach;
    if (right < kRightCols && a.I <= (rows || fp4 ? kFewTiled : kFewRows))
        switch (left * 4 + right) {
            case kLeftRows * 4 + kRightFp4:
                return choose_few<kLeftRows, false>(a, workspace, dev, stream);
            case kLeftRows * 4 + kRightFp8:
                return choose_few<kLeftRows, true>(a, workspace, dev, stream);
            case kLeftFp4 * 4 + kRightFp4:
                return choose_few<kLeftFp4, false>(a, workspace, dev, stream);
            case kLeftFp4 * 4 + kRightFp8:
                return choose_few<kLeftFp4, true>(a, workspace, dev, stream);
            case kLeftFp8 * 4 + kRightFp4:
                return choose_few<kLeftFp8, false>(a, workspace, dev, stream);
            default: return choose_few<kLeftFp8, true>(a, workspace, dev, stream);
        }
    switch (left * 4 + right) {
        case kLeftRows * 4 + kRightFp4:
            if (rows) return choose_rows<false>(a, workspace, dev, stream);
            return choose_tile<kLeftRows, kRightFp4>(a, workspace, dev, stream);
        case kLeftRows * 4 + kRightFp8:
            if (rows) return choose_rows<true>(a, workspace, dev, stream);
            return choose_tile<kLeftRows, kRightFp8>(a, workspace, dev, stream);
        case kLeftRows * 4 + c4:
            if (cols) return choose_cols<false, false>(a, workspace, dev, stream);
            return choose_tile<kLeftRows, c4>(a, workspace, dev, stream);
        case kLeftRows * 4 + c8:
            if (cols) return choose_cols<false, true>(a, workspace, dev, stream);
            return choose_tile<kLeftRows, c8>(a, workspace, dev, stream);
        case kLeftCols * 4 + c4:
            if (cols) return choose_cols<true, false>(a, workspace, dev, stream);
            return choose_tile<kLeftCols, c4>(a, workspace, dev, stream);
        case kLeftCols * 4 + c8:
            if (cols) return choose_cols<true, true>(a, workspace, dev, stream);
            return choose_tile<kLeftCols, c8>(a, workspace, dev, stream);
        case kLeftFp4 * 4 + kRightFp4:
            if (fp4) return choose_fp4(a, workspace, dev, stream);
            return choose_tile<kLeftFp4, kRightFp4>(a, workspace, dev, stream);
        case kLeftFp4 * 4 + kRightFp8:
            return choose_tile<kLeftFp4, kRightFp8>(a, workspace, dev, stream);
        case kLeftFp8 * 4 + kRightFp4:
            return choose_tile<kLeftFp8, kRightFp4>(a, workspace, dev, stream);
        case kLeftFp8 * 4 + kRightFp8:
            return choose_tile<kLeftFp8, kRightFp8>(a, workspace, dev, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace zs_detail
