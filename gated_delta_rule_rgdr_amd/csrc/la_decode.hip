// la_decode.hip -- linear attention with a decay for each head, a few tokens at a time.
//
// Per (entry, value head) and valid token, on S (D_k x D_v, fp32 while the call works on it):
//     S = exp(g) S + k v^T,     o = S^T (scale q).
#include "la_common.h"

namespace rgdr {

// Loads and stores of one state element at column c of a row, by 32 lanes (c = lane % 32).
template <int ST>
__device__ __forceinline__ float la_load1(const void *pool, const uint8_t *scales, long long e) {
    if constexpr (ST == RGDR_F32)
        return static_cast<const float *>(pool)[e];
    else if constexpr (ST == RGDR_BF16)
        return bf16_to_f32(static_cast<const uint16_t *>(pool)[e]);
    else
        return static_cast<float>(static_cast<const int8_t *>(pool)[e]) *
               mx_scale(scales[e / kMxBlock]);
}
template <int ST>
__device__ __forceinline__ void la_store1(void *pool, uint8_t *scales, long long e, float x) {
    if constexpr (ST == RGDR_F32) {
        static_cast<float *>(pool)[e] = x;
    } else if constexpr (ST == RGDR_BF16) {
        static_cast<uint16_t *>(pool)[e] = f32_to_bf16(x);
    } else {
        uint32_t top = __float_as_uint(x) & 0x7FFFFFFFu;  // as whole numbers NaN is the largest
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
        const uint32_t eb = mx_exponent(top);
        static_cast<uint8_t *>(pool)[e] = (uint8_t)mx_code_bits(x, mx_inverse(eb));
        if (e % kMxBlock == 0) scales[e / kMxBlock] = (uint8_t)eb;
    }
}

// The plainest form: thread (c, r) holds rows r, r + 8, ... of column c.
template <int ST, int DK>
__global__ __launch_bounds__(256) void la_recurrent_kernel(const LaArgs a, int tiles) {
    constexpr int R = DK / 8;
    __shared__ float ks[DK], qs[DK], red[8][32];
    const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
    const int h = bh % a.Hv, b = bh / a.Hv, hq = h / a.group;
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
    const LaEntry en = la_entry(a, b);
    const long long base = ((long long)en.slot * a.Hv + h) * DK * a.Dv + tile * 32 + c;
    float S[R];
    if (en.state)
#pragma unroll
        for (int m = 0; m < R; ++m)
            S[m] = la_load1<ST>(a.pool, a.scales, base + (long long)(r + 8 * m) * a.Dv);
    auto commit = [&]() {
#pragma unroll
        for (int m = 0; m < R; ++m)
            la_store1<ST>(a.pool_out, a.scales_out, base + (long long)(r + 8 * m) * a.Dv, S[m]);
    };
    if (en.state && en.n == 0) commit();
    const uint16_t *q = a.q + b * a.sq.b + hq * a.sq.h;
    const uint16_t *k = a.k + b * a.sk.b + hq * a.sk.h;
    const uint16_t *v = a.v + b * a.sv.b + h * a.sv.h + tile * 32 + c;
    const float *g = a.g + b * a.sg.b + h * a.sg.h;
    uint16_t *o = a.out + b * a.so.b + h * a.so.h + tile * 32 + c;
    for (int t = 0; t < en.L; ++t) {
        if (threadIdx.x < DK) {
            ks[threadIdx.x] = bf16_to_f32(k[t * a.sk.t + threadIdx.x]);
            qs[threadIdx.x] = bf16_to_f32(q[t * a.sq.t + threadIdx.x]) * a.scale;
        }
        const float vt = bf16_to_f32(v[t * a.sv.t]);
        const float d = expf(la_log_decay(g[t * a.sg.t]));
        __syncthreads();
        float o_part = 0.f;
#pragma unroll
        for (int m = 0; m < R; ++m) {
            S[m] = d * S[m] + ks[r + 8 * m] * vt;
            o_part += qs[r + 8 * m] * S[m];
        }
        red[r][c] = o_part;
        __syncthreads();
        if (r == 0) {
            float x = 0.f;
            for (int m = 0; m < 8; ++m) x += red[m][c];
            o[t * a.so.t] = f32_to_bf16(x);
        }
        if (t + 1 == en.n) commit();
    }
    if (r == 0)
        for (int t = en.L; t < a.T; ++t) o[t * a.so.t] = 0;
}

template <int ST>
static rgdr_status launch_recurrent_st(const LaArgs &a, int D_k, hipStream_t stream) {
    const int tiles = a.Dv / 32;
    const dim3 grid((unsigned)((long long)a.B * a.Hv * tiles)), block(256);
    if (D_k == 64)
        hipLaunchKernelGGL((la_recurrent_kernel<ST, 64>), grid, block, 0, stream, a, tiles);
    else if (D_k == 128)
        hipLaunchKernelGGL((la_recurrent_kernel<ST, 128>), grid, block, 0, stream, a, tiles);
    else
        hipLaunchKernelGGL((la_recurrent_kernel<ST, 256>), grid, block, 0, stream, a, tiles);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}

rgdr_status la_launch_recurrent(const LaArgs &a, int state_dtype, int D_k, hipStream_t stream) {
    if (state_dtype == RGDR_F32) return launch_recurrent_st<RGDR_F32>(a, D_k, stream);
    if (state_dtype == RGDR_BF16) return launch_recurrent_st<RGDR_BF16>(a, D_k, stream);
    return launch_recurrent_st<RGDR_MXI8>(a, D_k, stream);
}

rgdr_status la_check_sizes(int max_t, int32_t B, int32_t H_v, int32_t T, int32_t D_k, int32_t D_v) {
    if (B < 0 || H_v <= 0 || T <= 0 || T > max_t || D_k <= 0 || D_v <= 0) return RGDR_ERR_SHAPE;
    if (D_k != 64 && D_k != 128 && D_k != 256) return RGDR_ERR_UNSUPPORTED;
    if (D_v % 32 != 0 || D_v > 4096) return RGDR_ERR_UNSUPPORTED;
    // the grids are counted in ints
    if ((__int128)B * H_v * (D_v / 32) > 0x7FFFFFFF) return RGDR_ERR_SHAPE;
    return RGDR_OK;
}

rgdr_status la_check(LaArgs &a, int max_t, const void *query, const la_strides *query_strides,
                     const void *key, const la_strides *key_strides, const void *value,
                     const la_strides *value_strides, const float *g, const la_strides *g_strides,
                     const void *state_pool, const uint8_t *state_scales, int state_dtype,
                     const int32_t *lens, const int32_t *idx, const int32_t *nacc, float scale,
                     int32_t B, int32_t H_q, int32_t H_v, int32_t T, int32_t D_k, int32_t D_v,
                     int32_t N_slots, void *out, const la_strides *out_strides, void *state_out,
                     uint8_t *state_scales_out) {
    if (const rgdr_status st = la_check_sizes(max_t, B, H_v, T, D_k, D_v)) return st;
    if (H_q <= 0 || H_v % H_q != 0 || N_slots <= 0) return RGDR_ERR_SHAPE;
    if (state_dtype != RGDR_F32 && state_dtype != RGDR_BF16 && state_dtype != RGDR_MXI8)
        return RGDR_ERR_DTYPE;
    if (B == 0) return RGDR_OK;
    const bool mx = state_dtype == RGDR_MXI8;
    if (!query || !key || !value || !g || !state_pool || !out || !state_out) return RGDR_ERR_NULL;
    if (mx && (!state_scales || !state_scales_out)) return RGDR_ERR_NULL;
    if (!idx && N_slots < B) return RGDR_ERR_SHAPE;
    a.sq = la_strides_or(query_strides, (long long)H_q * T * D_k, (long long)T * D_k, D_k);
    a.sk = la_strides_or(key_strides, (long long)H_q * T * D_k, (long long)T * D_k, D_k);
    a.sv = la_strides_or(value_strides, (long long)H_v * T * D_v, (long long)T * D_v, D_v);
    a.sg = la_strides_or(g_strides, (long long)H_v * T, T, 1);
    a.so = la_strides_or(out_strides, (long long)H_v * T * D_v, (long long)T * D_v, D_v);
    if (!la_strides_ok(a.sq) || !la_strides_ok(a.sk) || !la_strides_ok(a.sv) ||
        !la_strides_ok(a.sg) || !la_strides_ok(a.so))
        return RGDR_ERR_SHAPE;
    if (!la_extent_ok(a.sq, B, H_q, T, D_k) || !la_extent_ok(a.sk, B, H_q, T, D_k) ||
        !la_extent_ok(a.sv, B, H_v, T, D_v) || !la_extent_ok(a.sg, B, H_v, T, 1) ||
        !la_rows_distinct(a.so, B, H_v, T, D_v))
        return RGDR_ERR_SHAPE;
    // offsets within a chunk of tokens are counted in 32 bits
    if (T > 1 && (a.sq.t > kMaxTokenStride || a.sk.t > kMaxTokenStride || a.sv.t > kMaxTokenStride))
        return RGDR_ERR_SHAPE;
    if (!la_strides_aligned(a.sq, B, H_q, T) || !la_strides_aligned(a.sk, B, H_q, T) ||
        !la_strides_aligned(a.sv, B, H_v, T) || !la_strides_aligned(a.so, B, H_v, T))
        return RGDR_ERR_ALIGN;
    if (!aligned(query, 16) || !aligned(key, 16) || !aligned(value, 16) || !aligned(g, 4) ||
        !aligned(state_pool, 16) || !aligned(state_out, 16) || !aligned(out, 16))
        return RGDR_ERR_ALIGN;
    if (mx && (!aligned(state_scales, 16) || !aligned(state_scales_out, 16))) return RGDR_ERR_ALIGN;
    if ((lens && !aligned(lens, 4)) || (idx && !aligned(idx, 4)) || (nacc && !aligned(nacc, 4)))
        return RGDR_ERR_ALIGN;
    if (T == 1) a.sq.t = a.sk.t = a.sv.t = a.sg.t = a.so.t = 0;
    a.q = static_cast<const uint16_t *>(query);
    a.k = static_cast<const uint16_t *>(key);
    a.v = static_cast<const uint16_t *>(value);
    a.g = g;
    a.pool = state_pool;
    a.scales = state_scales;
    a.out = static_cast<uint16_t *>(out);
    a.pool_out = state_out;
    a.scales_out = state_scales_out;
    a.lens = lens;
    a.idx = idx;
    a.nacc = nacc;
    a.scale = scale;
    a.B = B;
    a.Hq = H_q;
    a.Hv = H_v;
    a.T = T;
    a.Dv = D_v;
    a.N_slots = N_slots;
    a.group = H_v / H_q;
    return RGDR_OK;
}

}  // namespace rgdr

extern "C" rgdr_status la_decode(const void *query, const la_strides *query_strides,
                                 const void *key, const la_strides *key_strides,
                                 const void *value, const la_strides *value_strides,
                                 const float *g, const la_strides *g_strides,
                                 const void *state_pool, const uint8_t *state_scales,
                                 rgdr_dtype state_dtype, const int32_t *actual_seq_lengths,
                                 const int32_t *ssm_state_indices,
                                 const int32_t *num_accepted_tokens, float scale, int32_t B,
                                 int32_t H_q, int32_t H_v, int32_t T, int32_t D_k, int32_t D_v,
                                 int32_t N_slots, void *out, const la_strides *out_strides,
                                 void *state_out, uint8_t *state_scales_out, hipStream_t stream) {
    using namespace rgdr;
    LaArgs a;
    if (const rgdr_status st = la_check(
            a, kMaxT, query, query_strides, key, key_strides, value, value_strides, g, g_strides,
            state_pool, state_scales, state_dtype, actual_seq_lengths, ssm_state_indices,
            num_accepted_tokens, scale, B, H_q, H_v, T, D_k, D_v, N_slots, out, out_strides,
            state_out, state_scales_out))
        return st;
    if (B == 0) return RGDR_OK;
    return la_launch_recurrent(a, state_dtype, D_k, stream);
}
