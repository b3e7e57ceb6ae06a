// la_common.h -- what the linear-attention kernels (la_decode.hip, la_prefill.hip), the 8-bit
// state pools (la_state.hip) and the gated norm (la_norm_gate.hip) share: argument blocks, host
// checks, and the 8-bit block format. Not part of the C ABI.
#pragma once

#include "rgdr_common.h"
#include "rgdr_device.h"

namespace rgdr {

// ---- the 8-bit state format ---------------------------------------------------------------
//
// A block of 32 columns of one state row shares a byte e; a value is code * 2^(e - 127) with
// code in [-127, 127]. A power of two makes scaling exact in both directions, so the only
// rounding is the one to a whole code: at most 2^(e - 128), which is 1/127 to 1/254 of the
// block's largest value. A byte of 255 marks a block that held a NaN, an infinity or a value
// above 127 * 2^121, where the next code, 64 * 2^122, would be 2^128, past fp32's range.

constexpr int kMxBlock = 32;

// The byte for a block whose largest magnitude has these fp32 bits: the smallest e with
// top <= 127 * 2^(e-127). 127 = 1.984375 * 2^6 has the mantissa 0x7E0000; adding 0x1FFFF
// carries into the exponent exactly when top's mantissa is larger.
__host__ __device__ __forceinline__ uint32_t mx_exponent(uint32_t top_bits) {
    const uint32_t eb = (top_bits + 0x1FFFFu) >> 23;
    const uint32_t e = eb < 6 ? 0u : eb - 6u;
    return eb >= 255u ? 255u : e;
}
// 2^(127 - e): e <= 248 for every other block, so this is a normal number.
__device__ __forceinline__ float mx_inverse(uint32_t e) {
    return __uint_as_float((254u - (e == 255u ? 127u : e)) << 23);
}
// 2^(e - 127); e = 0 is a subnormal fp32, 255 is NaN.
__device__ __forceinline__ float mx_scale(uint32_t e) {
    const uint32_t bits = e ? e << 23 : 0x00400000u;
    return __uint_as_float(e == 255u ? 0x7FC00000u : bits);
}
// The code of x: adding 1.5 * 2^23 leaves the nearest whole number (ties to even) in the low
// bits, in two's complement; |x| * inv <= 127.
__device__ __forceinline__ uint32_t mx_code_bits(float x, float inv) {
    return __float_as_uint(__builtin_fmaf(x, inv, 12582912.0f));
}
// The low bytes of four such words, the first in the lowest byte.
__device__ __forceinline__ uint32_t mx_pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
    return lo | hi;
}
// Code i of a word of four (one instruction: the conversion selects the byte).
__device__ __forceinline__ float mx_code(uint32_t w, int i) {
    return static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
}
// The larger magnitude, or NaN if either is (three-operand instruction: two values each).
__device__ __forceinline__ float mx_larger(float top, float x) {
    return __builtin_elementwise_maximum(top, __builtin_fabsf(x));
}
__device__ __forceinline__ uint32_t mx_top_bits(float top) { return __float_as_uint(top) & 0x7FFFFFFFu; }

// ---- linear attention: arguments ------------------------------------------------------------

struct LaStrides {
    long long b, h, t;
};

struct LaArgs {
    const uint16_t *q, *k, *v;
    const float *g;
    const void *pool;
    const uint8_t *scales;
    uint16_t *out;
    void *pool_out;
    uint8_t *scales_out;
    const int32_t *lens, *idx, *nacc;  // each may be null
    LaStrides sq, sk, sv, sg, so;
    float scale;
    int B, Hq, Hv, T, Dv, N_slots, group;
    bool in_place;  // a state that no token changes need not be written
};

constexpr long long kMaxTokenStride = 1 << 24;  // elements from one token's row to the next's

struct LaEntry {
    int L, n, slot;
    bool state;  // the slot is in range: its state is read and committed
};

__device__ __forceinline__ LaEntry la_entry(const LaArgs &a, int b) {
    LaEntry e;
    e.slot = a.idx ? a.idx[b] : b;
    e.state = e.slot >= 0 && e.slot < a.N_slots;
    const int L = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    e.L = e.state ? L : 0;
    e.n = a.nacc ? min(max(a.nacc[b], 0), e.L) : e.L;
    return e;
}

// Log decays below this act as this: exp of it is zero even in fp64, and sums of them stay far
// from the range's end, so differences of such sums are never infinity minus infinity. NaN passes.
constexpr float kMinLogDecay = -1024.0f;
__device__ __forceinline__ float la_log_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }

// ---- host checks ------------------------------------------------------------------------------

constexpr long long kMaxGroups = 0xFFFFFF;  // workgroups of 256 in a launch, whose threads fit 32 bits

inline LaStrides la_strides_or(const la_strides *s, long long b, long long h, long long t) {
    if (s) return {s->b, s->h, s->t};
    return {b, h, t};
}
inline bool la_strides_ok(const LaStrides &s) { return s.b >= 0 && s.h >= 0 && s.t >= 0; }
// Strides of axes of one element move nothing and are free.
inline bool la_strides_aligned(const LaStrides &s, int B, int H, int T) {
    return (B == 1 || s.b % 8 == 0) && (H == 1 || s.h % 8 == 0) && (T == 1 || s.t % 8 == 0);
}
// Rows of D elements at these strides do not overlap. (Sufficient: sorted by stride, each axis
// steps over the whole extent of the ones inside it.)
inline bool la_rows_distinct(const LaStrides &s, int B, int H, int T, int D) {
    struct Axis {
        long long stride, n;
    } ax[3] = {{s.b, B}, {s.h, H}, {s.t, T}};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (ax[j].stride > ax[j + 1].stride) {
                const Axis x = ax[j];
                ax[j] = ax[j + 1];
                ax[j + 1] = x;
            }
    __int128 extent = D;
    for (const Axis &x : ax) {
        if (x.n <= 1) continue;
        if (x.stride < extent) return false;
        extent += (__int128)x.stride * (x.n - 1);
    }
    return extent < ((__int128)1 << 62);
}
// Every offset of the operand fits a 64-bit count of bytes.
inline bool la_extent_ok(const LaStrides &s, int B, int H, int T, int D) {
    const __int128 e = (__int128)s.b * (B - 1) + (__int128)s.h * (H - 1) + (__int128)s.t * (T - 1) + D;
    return e < ((__int128)1 << 60);
}

// The argument checks of la_decode and la_prefill (T up to max_t), and the kernels' argument
// block. B = 0 is RGDR_OK with nothing to launch.
rgdr_status la_check(LaArgs &a, int max_t, const void *query, const la_strides *query_strides,
                     const void *key, const la_strides *key_strides, const void *value,
                     const la_strides *value_strides, const float *g, const la_strides *g_strides,
                     const void *state_pool, const uint8_t *state_scales, int state_dtype,
                     const int32_t *lens, const int32_t *idx, const int32_t *nacc, float scale,
                     int32_t B, int32_t H_q, int32_t H_v, int32_t T, int32_t D_k, int32_t D_v,
                     int32_t N_slots, void *out, const la_strides *out_strides, void *state_out,
                     uint8_t *state_scales_out);
rgdr_status la_check_sizes(int max_t, int32_t B, int32_t H_v, int32_t T, int32_t D_k, int32_t D_v);

}  // namespace rgdr
