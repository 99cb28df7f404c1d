// bf16 matrix products of fp32 values cut into bf16 parts (gfx950).
//
// An fp32 value is the exact sum of three bf16 values (its 24 bits cut in three).
// Products of bf16 values are exact in the fp32 accumulator, so a product of a bf16
// value and an fp32 value is three matrix instructions, one of two fp32 values six
// (the other three of the nine are left out: at most 2^-21 of it, 2^-24.7 on average).
#pragma once

#include "lq_internal.h"

namespace lq {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ bool finite_f32(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// x, as a value the compiler must form here: offsets derived from it are computed where
// they are used instead of held in registers across a loop.
__device__ __forceinline__ uint32_t fresh(uint32_t x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Token rows of a chunk as a buffer of `bytes` bytes from base (both wave-uniform): loads
// past its end give zeros and stores past it are dropped, by the hardware's range check,
// so the rows of a partial chunk need no masks, and an address is one 32-bit register.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rows(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00020000);
}
__device__ __forceinline__ uint32_t row_ld(rsrc_t r, uint32_t off) { return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0); }
__device__ __forceinline__ u32x4 row_ld4(rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
// Streaming store (non-temporal).
__device__ __forceinline__ void row_st(rsrc_t r, uint32_t off, uint32_t x) {
    __builtin_amdgcn_raw_buffer_store_b32(x, r, off, 0, 2);
}

// Operand rows in LDS, R rows of pieces of 16 bytes (8 bf16), piece after piece: the rows'
// pieces p are contiguous, so a matrix operand's 16-byte reads (16 rows, four pieces over
// the lane groups) are free of bank conflicts: one serves lanes of the pieces 2 i and 2 i + 1
// together, rows 0-3 and 12-15 of one, 4-11 of the other.  16 bytes of padding after every
// second piece spread the writes of a row.  (Row after row with 16 bytes of padding, the
// chunk kernels spent 40% of their LDS time in conflicts.)  Every address is a constant
// away from the lane's.
template <int R>
__device__ __forceinline__ constexpr int pm(int row, int piece) { return 8 * (piece * R + (piece >> 1) + row); }
template <int R>
constexpr int pm_shorts(int pieces) { return 8 * (pieces * R + (pieces + 1) / 2); }

// Two fp32 values to packed bf16 (nearest even), low half first.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ float lo_f32(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f32(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// Upper halves of (a, b) as packed bf16: truncation to 8 bits.
__device__ __forceinline__ uint32_t top_halves(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float top_f32(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// Whether either bf16 of x is infinite or NaN.
__device__ __forceinline__ uint32_t odd_bf16(uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

__device__ __forceinline__ v4f mfma_bf16(u32x4 a, u32x4 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(__attribute__((ext_vector_type(8))) __bf16, a),
                                                   __builtin_bit_cast(__attribute__((ext_vector_type(8))) __bf16, b), c,
                                                   0, 0, 0);
}

// Transposed LDS read (every lane of a group of 16: 8 bytes, four columns of row lane / 4): lane i
// receives column i of the group's four rows.
__device__ __forceinline__ u32x2 lds_tr(const uint16_t* p) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)const_cast<uint16_t*>(p)));
}

// N values in three bf16 parts, packed.
template <int N>
__device__ __forceinline__ void split3(const float (&x)[N], uint32_t (&p)[3][N / 2]) {
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
        const float a = x[2 * e], b = x[2 * e + 1];
        const float a1 = a - top_f32(a), b1 = b - top_f32(b);
        p[0][e] = top_halves(a, b);
        p[1][e] = top_halves(a1, b1);
        p[2][e] = top_halves(a1 - top_f32(a1), b1 - top_f32(b1));
    }
}

// c += a b, a and b in three parts each; small products first.
__device__ __forceinline__ v4f mfma_split(const u32x4 (&a)[3], const u32x4 (&b)[3], v4f c) {
    c = mfma_bf16(a[2], b[0], c);
    c = mfma_bf16(a[0], b[2], c);
    c = mfma_bf16(a[1], b[1], c);
    c = mfma_bf16(a[1], b[0], c);
    c = mfma_bf16(a[0], b[1], c);
    return mfma_bf16(a[0], b[0], c);
}

// A token value as loaded, widened; four consecutive ones.
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return bf16_to_f32(x); }
template <typename TI> struct Row4;
template <> struct Row4<float> {
    v4f x;
    __device__ __forceinline__ void load(const void* p, size_t at) { x = *reinterpret_cast<const v4f*>(static_cast<const float*>(p) + at); }
    __device__ __forceinline__ void widen4(float (&y)[4]) const { y[0] = x[0], y[1] = x[1], y[2] = x[2], y[3] = x[3]; }
};
template <> struct Row4<uint16_t> {
    u32x2 x;
    __device__ __forceinline__ void load(const void* p, size_t at) { x = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + at); }
    __device__ __forceinline__ void widen4(float (&y)[4]) const { y[0] = lo_f32(x[0]), y[1] = hi_f32(x[0]), y[2] = lo_f32(x[1]), y[3] = hi_f32(x[1]); }
};

// Inclusive prefix sum over the 64 lanes: lane shifts within 16 lanes, then the last lane
// of a row to the rows above it (data-parallel moves, no LDS).
template <int CTRL, int ROWS>
__device__ __forceinline__ double scan_step(double x) {
    const uint64_t u = __double_as_longlong(x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return x + __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double wave_scan(double x) {
    x = scan_step<0x111, 0xf>(x);      // row_shr 1, 2, 4, 8
    x = scan_step<0x112, 0xf>(x);
    x = scan_step<0x114, 0xf>(x);
    x = scan_step<0x118, 0xf>(x);
    x = scan_step<0x142, 0xa>(x);      // row_bcast 15 into rows 1, 3
    return scan_step<0x143, 0xc>(x);   // row_bcast 31 into rows 2, 3
}

__device__ __forceinline__ v4f mfma4(float a, float b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// M = (I + A)^{-1} R for a block of 16 rows and CT column tiles, A strictly lower, in place: four
// rows at a time, lane group p solves its rows; row swaps bring its row 4 p + i to lane group i, the
// B operand of one k = 4 step with -A's columns 4 p .. 4 p + 3 (rows below them).
// own[i] = -A[4 lg + 1 + i][4 lg ..], below[p] = -A[li][4 p + lg].
template <int CT>
__device__ __forceinline__ void block_solve(const v4f (&own)[3], const float (&below)[3], int lg, v4f (&R)[CT]) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        if (lg == p)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                R[ct][1] += own[0][0] * R[ct][0];
                R[ct][2] += own[1][0] * R[ct][0] + own[1][1] * R[ct][1];
                R[ct][3] += own[2][0] * R[ct][0] + own[2][1] * R[ct][1] + own[2][2] * R[ct][2];
            }
        if (p < 3)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const bool on = lg == p;
                const float x = rows_sum4(on ? R[ct][0] : 0.0f, on ? R[ct][1] : 0.0f, on ? R[ct][2] : 0.0f, on ? R[ct][3] : 0.0f);
                R[ct] = mfma4(below[p], x, R[ct]);
            }
    }
}

}  // namespace lq
