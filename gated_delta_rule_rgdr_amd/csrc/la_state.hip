// la_state.hip -- states into and out of 8-bit pools.
//
// Per block of 32 columns: e = the smallest power of two with max|x| <= 127 * 2^e, code =
// x / 2^e rounded to the nearest whole number (ties to even), value = code * 2^e. Scaling by a
// power of two is exact, so the code is the only rounding.
#include "la_common.h"

namespace rgdr {

struct StateMove {
    const void *in;
    const uint8_t *scales_in;
    void *out;
    uint8_t *scales_out;
    const int32_t *src, *dst;  // each may be null
    int N_src, N_dst;
    long long blocks;  // blocks of 32 columns in one slot
    unsigned parts;    // workgroups for each entry
};

// The slots of entry i, resolved; false: nothing to do.
__device__ __forceinline__ bool move_slots(const StateMove &m, int i, int &s, int &d) {
    s = m.src ? m.src[i] : i;
    d = m.dst ? m.dst[i] : i;
    return d >= 0 && d < m.N_dst;
}

// A lane holds 16 bytes of the wide pool, so both pools are read and written in whole lines: 4
// columns in fp32 (8 lanes for a block), 8 in bf16 (4 lanes). U such units are in flight. Bound: the
// bytes. 96 slots of H_v = 32, D = 128: fp32 into 8 bits 49.1 us (5.2 TB/s), back 38.5 us (6.6);
// bf16 27.3 us (5.6) and 24.3 us (6.3); one slot 2.2 us each (the launch).
template <bool BF16>
struct Unit {
    static constexpr int N = BF16 ? 8 : 4;            // columns
    static constexpr int LANES = kMxBlock / N;        // lanes of a block
    static constexpr int W = N / 4;                   // words of codes
};

// The largest of the magnitudes' bits over a block's lanes.
template <int LANES>
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, false));  // lane ^ 1
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, false));  // lane ^ 2
    if constexpr (LANES == 8)
        x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, false));  // other quad of 8
    return x;
}

template <bool BF16, int U>
__global__ __launch_bounds__(256) void la_quantize_kernel(const StateMove m) {
    using T = Unit<BF16>;
    int s, d;
    if (!move_slots(m, blockIdx.x / m.parts, s, d)) return;
    const bool have = s >= 0 && s < m.N_src;
    const long long units = m.blocks * T::LANES;
    const long long j0 = (long long)(blockIdx.x % m.parts) * (256 * U) + threadIdx.x;
    const u32x4 *in = reinterpret_cast<const u32x4 *>(m.in) + (have ? s : 0) * units;
    uint32_t *out = reinterpret_cast<uint32_t *>(m.out) + d * units * T::W;
    uint8_t *scales = m.scales_out + d * m.blocks;
    u32x4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long j = j0 + u * 256;
        w[u] = u32x4{0, 0, 0, 0};
        if (have && j < units) w[u] = __builtin_nontemporal_load(in + j);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long j = j0 + u * 256;
        float x[T::N], top = 0.f;
#pragma unroll
        for (int c = 0; c < T::N; ++c) {
            x[c] = !BF16 ? __uint_as_float(w[u][c]) : c & 1 ? bf16_hi(w[u][c / 2]) : bf16_lo(w[u][c / 2]);
            top = mx_larger(top, x[c]);
        }
        const uint32_t eb = mx_exponent(block_max<T::LANES>(mx_top_bits(top)));
        const float inv = mx_inverse(eb);
        if (j < units) {  // the units are whole blocks
#pragma unroll
            for (int c = 0; c < T::W; ++c)
                out[j * T::W + c] = mx_pack4(mx_code_bits(x[4 * c], inv), mx_code_bits(x[4 * c + 1], inv),
                                             mx_code_bits(x[4 * c + 2], inv), mx_code_bits(x[4 * c + 3], inv));
            if (threadIdx.x % T::LANES == 0) scales[j / T::LANES] = (uint8_t)eb;
        }
    }
}

template <bool BF16, int U>
__global__ __launch_bounds__(256) void la_dequantize_kernel(const StateMove m) {
    using T = Unit<BF16>;
    int s, d;
    if (!move_slots(m, blockIdx.x / m.parts, s, d)) return;
    const bool have = s >= 0 && s < m.N_src;
    const long long units = m.blocks * T::LANES;
    const long long j0 = (long long)(blockIdx.x % m.parts) * (256 * U) + threadIdx.x;
    const uint32_t *in = reinterpret_cast<const uint32_t *>(m.in) + (have ? s : 0) * units * T::W;
    const uint8_t *scales = m.scales_in + (have ? s : 0) * m.blocks;
    u32x4 *out = reinterpret_cast<u32x4 *>(m.out) + d * units;
    uint32_t w[U][T::W] = {}, eb[U] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long j = j0 + u * 256;
        if (have && j < units) {
#pragma unroll
            for (int c = 0; c < T::W; ++c) w[u][c] = in[j * T::W + c];
            eb[u] = scales[j / T::LANES];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long j = j0 + u * 256;
        const float sc = mx_scale(eb[u]);
        float x[T::N];
#pragma unroll
        for (int c = 0; c < T::N; ++c) x[c] = mx_code(w[u][c / 4], c % 4) * sc;
        u32x4 y;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            y[c] = BF16 ? pack_bf16x2(x[2 * c % T::N], x[(2 * c + 1) % T::N]) : __float_as_uint(x[c]);
        if (j < units) __builtin_nontemporal_store(y, out + j);
    }
}

// Checks shared by both directions. `wide` is the fp32 or bf16 pool, `codes` the 8-bit one.
static rgdr_status move_check(const void *wide, int state_dtype, const void *codes,
                              const uint8_t *scales, int32_t N_src, const int32_t *src,
                              int32_t N_dst, const int32_t *dst, int32_t n, int32_t H_v,
                              int32_t D_k, int32_t D_v, StateMove &m) {
    if (n < 0 || H_v <= 0 || D_k <= 0 || D_v <= 0 || N_src <= 0 || N_dst <= 0) return RGDR_ERR_SHAPE;
    if (D_v % kMxBlock != 0) return RGDR_ERR_UNSUPPORTED;
    if (state_dtype != RGDR_F32 && state_dtype != RGDR_BF16) return RGDR_ERR_DTYPE;
    const __int128 blocks = (__int128)H_v * D_k * (D_v / kMxBlock);
    const int slots = N_src > N_dst ? N_src : N_dst;
    if (blocks * slots > ((__int128)1 << 54)) return RGDR_ERR_SHAPE;
    if (n == 0) return RGDR_OK;
    if (!wide || !codes || !scales) return RGDR_ERR_NULL;
    if ((!src && n > N_src) || (!dst && n > N_dst)) return RGDR_ERR_SHAPE;
    if (!aligned(wide, 16) || !aligned(codes, 16) || !aligned(scales, 16) ||
        (src && !aligned(src, 4)) || (dst && !aligned(dst, 4)))
        return RGDR_ERR_ALIGN;
    m.src = src;
    m.dst = dst;
    m.N_src = N_src;
    m.N_dst = N_dst;
    m.blocks = (long long)blocks;
    return RGDR_OK;
}

// Four units for each thread where that still gives every compute unit several workgroups, else one.
template <bool BF16, bool BACK>
static rgdr_status launch_move(StateMove &m, int n, hipStream_t stream) {
    const long long groups = (m.blocks * Unit<BF16>::LANES + 255) / 256;
    const bool four = groups / 4 * n >= 1024;
    const long long parts = four ? (groups + 3) / 4 : groups;
    if ((__int128)parts * n > kMaxGroups) return RGDR_ERR_SHAPE;
    m.parts = (unsigned)parts;
    const dim3 grid((unsigned)(parts * n)), block(256);
    if (four)
        hipLaunchKernelGGL((BACK ? la_dequantize_kernel<BF16, 4> : la_quantize_kernel<BF16, 4>), grid, block, 0, stream, m);
    else
        hipLaunchKernelGGL((BACK ? la_dequantize_kernel<BF16, 1> : la_quantize_kernel<BF16, 1>), grid, block, 0, stream, m);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}

}  // namespace rgdr

extern "C" rgdr_status la_state_quantize(const void *state, rgdr_dtype state_dtype, int32_t N_src,
                                         const int32_t *src_slots, void *codes, uint8_t *scales,
                                         int32_t N_dst, const int32_t *dst_slots, int32_t n,
                                         int32_t H_v, int32_t D_k, int32_t D_v,
                                         hipStream_t stream) {
    using namespace rgdr;
    StateMove m = {};
    if (const rgdr_status st = move_check(state, state_dtype, codes, scales, N_src, src_slots,
                                          N_dst, dst_slots, n, H_v, D_k, D_v, m))
        return st;
    if (n == 0) return RGDR_OK;
    m.in = state;
    m.out = codes;
    m.scales_out = scales;
    return state_dtype == RGDR_BF16 ? launch_move<true, false>(m, n, stream)
                                    : launch_move<false, false>(m, n, stream);
}

extern "C" rgdr_status la_state_dequantize(const void *codes, const uint8_t *scales,
                                           int32_t N_src, const int32_t *src_slots, void *state,
                                           rgdr_dtype state_dtype, int32_t N_dst,
                                           const int32_t *dst_slots, int32_t n, int32_t H_v,
                                           int32_t D_k, int32_t D_v, hipStream_t stream) {
    using namespace rgdr;
    StateMove m = {};
    if (const rgdr_status st = move_check(state, state_dtype, codes, scales, N_src, src_slots,
                                          N_dst, dst_slots, n, H_v, D_k, D_v, m))
        return st;
    if (n == 0) return RGDR_OK;
    m.in = codes;
    m.scales_in = scales;
    m.out = state;
    return state_dtype == RGDR_BF16 ? launch_move<true, true>(m, n, stream)
                                    : launch_move<false, true>(m, n, stream);
}
