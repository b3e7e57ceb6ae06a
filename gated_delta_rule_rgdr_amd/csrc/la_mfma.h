// la_mfma.h -- matrix-core helpers of the linear-attention kernels: operands from LDS, bf16 splits.
// Not part of the C ABI.
//
// v_mfma_f32_32x32x16_bf16: operand A's lane l holds row l % 32, B's column l % 32, both the 8
// products 8 (l / 32) .. + 7; register r of the result's lane l is row 8 (r / 4) + 4 (l / 32) +
// r % 4 of column l % 32.
// v_mfma_f32_16x16x32_bf16: rows and columns l % 16, products 8 (l / 16) .. + 7; the result's
// register r is row 4 (l / 16) + r of column l % 16.
#pragma once

#include "la_common.h"

namespace rgdr {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// 16-byte pieces of LDS rows of PIECES such pieces. A spare piece behind each row (where rows are
// 128 bytes or more) puts the same piece of 16 rows on different banks, and every address is a lane's base
// plus a constant. (Permuting the pieces in each row instead cost the prompt kernel a tenth of its
// vector instructions for addresses; it serves the short rows.) The reads that transpose take
// four rows of 64 bytes at once: three spare pieces (kTrPad) leave two of the four on the same banks,
// one leaves all four.
constexpr int kTrPad = 48;
template <int PIECES, int PAD = 16>
__device__ __forceinline__ constexpr int lds_row_bytes() {
    return PIECES >= 8 ? PIECES * 16 + PAD : PIECES * 16;
}
template <int PIECES, int PAD = 16>
__device__ __forceinline__ int lds_at(int row, int piece) {
    if constexpr (PIECES == 2)
        piece ^= (row >> 3) & 1;
    else if constexpr (PIECES == 4)
        piece ^= (row >> 2) & 3;
    return row * lds_row_bytes<PIECES, PAD>() + piece * 16;
}

__device__ __forceinline__ bf16x8 lds_read(const char *p) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(p));
}

// Eight rows (tokens) of one column for each lane: lane l gets column map32(l % 32) of its
// 32-column group, rows 8 * (l / 32) .. + 7 of the 16 at `row0`. The hardware transposes 4 rows
// by 16 columns for each 16 lanes, which read them as 4-column pieces; lane l's piece is
// chosen so that consecutive accumulator registers hold consecutive rows (see map32).
template <int PIECES, int PAD = 16>
__device__ __forceinline__ bf16x8 lds_read_tr(char *m, int row0, int group, int lane) {
    const int n = lane & 15, row = ((lane >> 5) << 3) + (n >> 2);
    const int piece = ((lane >> 4) & 1) * 2 + (n & 1), half = (n & 2) << 2;
    typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
    s16x4 lo, hi;
    if constexpr (PIECES >= 8) {
        char *const p = m + lds_at<PIECES, PAD>(row, piece) + half + lds_at<PIECES, PAD>(row0, group * 4);
        lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p);
        hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * lds_row_bytes<PIECES, PAD>()));
    } else {
        lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_ptr)(m + lds_at<PIECES>(row0 + row, group * 4 + piece) + half));
        hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_ptr)(m + lds_at<PIECES>(row0 + row + 4, group * 4 + piece) + half));
    }
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The column (or row) that position n of a 32-wide matrix operand read by lds_read_tr stands for:
// groups of four in the order 0, 2, 1, 3. An accumulator lane holds positions 8 m + 4 (l / 32) + 0..3
// in registers 4 m + 0..3, which are then the 8 consecutive rows 16 (m / 2) + 8 (l / 32) + 0..7
// in registers 8 (m / 2) + 0..7: what a matrix operand's lane holds, and 16 bytes of output.
__device__ __forceinline__ int map32(int n) {
    return (n & 16) | ((n & 4) << 1) | ((n & 8) >> 1) | (n & 3);
}

// What bf16 rounding left of x0 and x1: x - hi, exactly. (v_dot2_f32_bf16 with a pair (-1, 0) does
// widening and subtraction in one instruction, exactly too, and was no faster: B=16, T=1024, H=32,
// D=128 141.4 us against 139.4 when operands were split into two numbers.)
__device__ __forceinline__ void bf16_rest(uint32_t hi, float &x0, float &x1) {
    x0 -= bf16_lo(hi);
    x1 -= bf16_hi(hi);
}

// x = hi + lo (+ rest) in bf16, for eight values; x becomes the rest.
__device__ __forceinline__ void split2(float (&x)[8], u32x4 &hi, u32x4 &lo) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        hi[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
        bf16_rest(hi[i], x[2 * i], x[2 * i + 1]);
        lo[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    }
}
__device__ __forceinline__ u32x4 split_rest(float (&x)[8], const u32x4 &lo) {
    u32x4 lo2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bf16_rest(lo[i], x[2 * i], x[2 * i + 1]);
        lo2[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    }
    return lo2;
}

// Between a wave's writes into its own part of LDS and its reads of them across the lanes: LDS serves
// a wave's accesses in order, and the compiler is kept from reordering them.
__device__ __forceinline__ void wave_in_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 mfma(u32x4 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), b, c, 0, 0, 0);
}

// Inclusive sum over the wave's lanes, by register moves between lanes (within rows of 16, then
// from each row's last lane to the rows behind it).
template <int CTRL, int ROWS>
__device__ __forceinline__ double scan_step(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
    return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_scan(double x) {
    x = scan_step<0x111, 0xF>(x);
    x = scan_step<0x112, 0xF>(x);
    x = scan_step<0x114, 0xF>(x);
    x = scan_step<0x118, 0xF>(x);
    x = scan_step<0x142, 0xA>(x);  // lane 15 to row 1, lane 47 to row 3
    return scan_step<0x143, 0xC>(x);  // lane 31 to rows 2 and 3
}
__device__ __forceinline__ double wave_last(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

}  // namespace rgdr
