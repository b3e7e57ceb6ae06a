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

// One thread for each block of 32 columns.
template <bool BF16>
__global__ __launch_bounds__(256) void la_quantize_kernel(const StateMove m) {
    const int i = blockIdx.x / m.parts;
    int s, d;
    if (!move_slots(m, i, s, d)) return;
    const bool have = s >= 0 && s < m.N_src;
    for (long long j = (long long)(blockIdx.x % m.parts) * 256 + threadIdx.x; j < m.blocks;
         j += (long long)m.parts * 256) {
        float x[kMxBlock];
        const long long e = ((long long)s * m.blocks + j) * kMxBlock;
#pragma unroll
        for (int c = 0; c < kMxBlock; ++c)
            x[c] = !have  ? 0.f
                   : BF16 ? bf16_to_f32(static_cast<const uint16_t *>(m.in)[e + c])
                          : static_cast<const float *>(m.in)[e + c];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < kMxBlock; ++c) top = max(top, __float_as_uint(x[c]) & 0x7FFFFFFFu);
        const uint32_t eb = mx_exponent(top);
        const float inv = mx_inverse(eb);
        uint32_t w[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            w[c] = mx_pack4(mx_code_bits(x[4 * c], inv), mx_code_bits(x[4 * c + 1], inv),
                            mx_code_bits(x[4 * c + 2], inv), mx_code_bits(x[4 * c + 3], inv));
        u32x4 *o = reinterpret_cast<u32x4 *>(static_cast<char *>(m.out) +
                                             ((long long)d * m.blocks + j) * kMxBlock);
        o[0] = u32x4{w[0], w[1], w[2], w[3]};
        o[1] = u32x4{w[4], w[5], w[6], w[7]};
        m.scales_out[(long long)d * m.blocks + j] = (uint8_t)eb;
    }
}

template <bool BF16>
__global__ __launch_bounds__(256) void la_dequantize_kernel(const StateMove m) {
    const int i = blockIdx.x / m.parts;
    int s, d;
    if (!move_slots(m, i, s, d)) return;
    const bool have = s >= 0 && s < m.N_src;
    for (long long j = (long long)(blockIdx.x % m.parts) * 256 + threadIdx.x; j < m.blocks;
         j += (long long)m.parts * 256) {
        const long long e = (long long)s * m.blocks + j;
        u32x4 w[2] = {};
        float sc = 0.f;
        if (have) {
            const u32x4 *p = reinterpret_cast<const u32x4 *>(static_cast<const char *>(m.in) +
                                                             e * kMxBlock);
            w[0] = p[0];
            w[1] = p[1];
            sc = mx_scale(m.scales_in[e]);
        }
        const long long o = ((long long)d * m.blocks + j) * kMxBlock;
#pragma unroll
        for (int c = 0; c < kMxBlock; ++c) {
            const float x = mx_code(w[c / 16][c / 4 % 4], c % 4) * sc;
            if (BF16)
                static_cast<uint16_t *>(m.out)[o + c] = f32_to_bf16(x);
            else
                static_cast<float *>(m.out)[o + c] = x;
        }
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
    const long long full = (m.blocks + 255) / 256;
    const long long most = 0x7FFFFFFFLL / n;  // the grid is counted in an int
    m.parts = (unsigned)(full < most ? full : most);
    return RGDR_OK;
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
    const dim3 grid((unsigned)n * m.parts), block(256);
    if (state_dtype == RGDR_BF16)
        hipLaunchKernelGGL(la_quantize_kernel<true>, grid, block, 0, stream, m);
    else
        hipLaunchKernelGGL(la_quantize_kernel<false>, grid, block, 0, stream, m);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
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
    const dim3 grid((unsigned)n * m.parts), block(256);
    if (state_dtype == RGDR_BF16)
        hipLaunchKernelGGL(la_dequantize_kernel<true>, grid, block, 0, stream, m);
    else
        hipLaunchKernelGGL(la_dequantize_kernel<false>, grid, block, 0, stream, m);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}
