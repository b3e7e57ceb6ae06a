// la_conv.hip -- the short causal convolution between an input projection and a recurrence: for each
// channel
//     y[t] = f(bias + sum_j weight[j] line[t - (W - 1) + j]),
// on the line that the slot's last W - 1 inputs and the call's tokens make up; the slot then holds
// the last W - 1 inputs after the accepted tokens.
#include "la_common.h"

namespace rgdr {

struct ConvArgs {
    const void *x, *pool;
    const float *weight, *bias;
    void *out, *pool_out;
    const int32_t *lens, *idx, *nacc;  // each may be null
    LaStrides sx, so;
    int B, T, C, N_slots, silu;
};

constexpr int kConvChannels = 4;  // of a thread

// A thread has four channels and TT tokens in a row, whose inputs (with the W - 1 before them) it holds in
// registers: W - 1 + TT loads in flight at once. TT >= W - 1 or T = 1, so the slot's inputs are read by the
// thread of the first tokens alone, which also writes the slot: the pool can be updated in place. Bound:
// the bytes. B=16, T=1024 ragged, C=8192, W=4, bf16: 85.8 us (5.1 TB/s); with 8 tokens for each thread 93.7,
// which reads more rows twice, and with eight channels for each (more registers, fewer waves) 95.3; with
// loads that pass the caches by 101. One sequence of 8192 tokens 52.0.
template <typename E, int W, int TT>
__global__ __launch_bounds__(256) void la_conv_kernel(const ConvArgs a, int cl_log, int c_blocks, int t_blocks) {
    constexpr int N = kConvChannels, H = W - 1;
    using V = Row<E, N>;
    const int cb = blockIdx.x % c_blocks, tb = blockIdx.x / c_blocks % t_blocks;
    const int b = blockIdx.x / c_blocks / t_blocks;
    const int c = ((cb << cl_log) + (threadIdx.x & ((1 << cl_log) - 1))) * N;
    const long long t0 = ((long long)tb * (256 >> cl_log) + (threadIdx.x >> cl_log)) * TT;
    if (c >= a.C || t0 >= a.T) return;
    const int slot = a.idx ? a.idx[b] : b;
    const bool state = slot >= 0 && slot < a.N_slots;
    const int L = !state ? 0 : a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const int n = a.nacc ? min(max(a.nacc[b], 0), L) : L;
    const E *x = static_cast<const E *>(a.x) + b * a.sx.b + c;
    E *out = static_cast<E *>(a.out) + b * a.so.b + c;
    const size_t at = (size_t)(state ? slot : 0) * H * a.C + c;
    const E *pool = static_cast<const E *>(a.pool) + at;

    V line[H + TT];
#pragma unroll
    for (int i = 0; i < H + TT; ++i) {
        const long long t = t0 + i - H;
        line[i].zero();
        if (t >= 0 && t < L)
            line[i].load(x + t * a.sx.t);
        else if (i < H && t0 == 0 && state)
            line[i].load(pool + (size_t)i * a.C);
    }
    // The slot's new inputs, read with the others. (One whose entry accepts no token keeps its bytes when the
    // pool is updated in place.)
    const bool commit = t0 == 0 && state && (n > 0 || a.pool_out != a.pool);
    V keep[H];
    if (commit && TT > 1) {
#pragma unroll
        for (int j = 0; j < H; ++j) keep[j].load(n + j < H ? pool + (size_t)(n + j) * a.C : x + (n + j - H) * a.sx.t);
    }
    float w[N * W], bias[N];
#pragma unroll
    for (int i = 0; i < N * W / 4; ++i)
        *reinterpret_cast<f32x4 *>(w + 4 * i) = *reinterpret_cast<const f32x4 *>(a.weight + (size_t)c * W + 4 * i);
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        *reinterpret_cast<f32x4 *>(bias + 4 * i) =
            a.bias ? *reinterpret_cast<const f32x4 *>(a.bias + c + 4 * i) : f32x4{0, 0, 0, 0};
    if (commit) {
        E *to = static_cast<E *>(a.pool_out) + at;
#pragma unroll
        for (int j = 0; j < H; ++j) {
            if (TT == 1) keep[j] = n ? line[j + 1] : line[j];
            keep[j].store(to + (size_t)j * a.C);
        }
    }
#pragma unroll
    for (int u = 0; u < TT; ++u) {
        const long long t = t0 + u;
        if (t >= a.T) return;
        float y[N];
#pragma unroll
        for (int k = 0; k < N; ++k) y[k] = bias[k];
#pragma unroll
        for (int j = 0; j < W; ++j) {
#pragma unroll
            for (int k = 0; k < N; ++k) y[k] = __builtin_fmaf(w[k * W + j], line[u + j].get(k), y[k]);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (a.silu) y[k] *= sigmoid_fast(y[k]);
            y[k] = t < L ? y[k] : 0.f;
        }
        V o;
        o.set(y);
        o.template store<true>(out + t * a.so.t);
    }
}

template <typename E, int W, int TT>
static rgdr_status launch_conv_rows(const ConvArgs &a, hipStream_t stream) {
    const int pieces = a.C / kConvChannels;
    int cl_log = 0;
    while (cl_log < 8 && (1 << cl_log) < pieces) ++cl_log;
    const long long c_blocks = ((long long)pieces + (1 << cl_log) - 1) >> cl_log;
    const long long tu = (long long)(256 >> cl_log) * TT, t_blocks = (a.T + tu - 1) / tu;
    if ((__int128)c_blocks * t_blocks * a.B > kMaxGroups) return RGDR_ERR_SHAPE;
    const dim3 grid((unsigned)(c_blocks * t_blocks * a.B)), block(256);
    hipLaunchKernelGGL((la_conv_kernel<E, W, TT>), grid, block, 0, stream, a, cl_log, (int)c_blocks, (int)t_blocks);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}

template <typename E, int W>
static rgdr_status launch_conv_taps(const ConvArgs &a, hipStream_t stream) {
    if (a.T == 1) return launch_conv_rows<E, W, 1>(a, stream);
    // 16 tokens for each thread where that still gives every compute unit two workgroups;
    // us against 8: B=16, T=1024 ragged, C=8192 85.7/93.6; B=3, T=100, C=512 5.8/4.2; B=1, T=8 4.6/4.4.
    const bool many = (__int128)a.B * a.T * a.C >= 512LL * 256 * kConvChannels * 16;
    if (a.T > 8 && many) return launch_conv_rows<E, W, 16>(a, stream);
    return launch_conv_rows<E, W, 8>(a, stream);
}

template <typename E>
static rgdr_status launch_conv(const ConvArgs &a, int W, hipStream_t stream) {
    if (W == 2) return launch_conv_taps<E, 2>(a, stream);
    if (W == 3) return launch_conv_taps<E, 3>(a, stream);
    return launch_conv_taps<E, 4>(a, stream);
}

}  // namespace rgdr

extern "C" rgdr_status la_conv(const void *x, const la_strides *x_strides, const float *weight,
                               const float *bias, rgdr_dtype dtype, const void *state_pool,
                               const int32_t *actual_seq_lengths, const int32_t *ssm_state_indices,
                               const int32_t *num_accepted_tokens, uint32_t flags, int32_t B, int32_t T,
                               int32_t C, int32_t W, int32_t N_slots, void *out,
                               const la_strides *out_strides, void *state_out, hipStream_t stream) {
    using namespace rgdr;
    if (B < 0 || T < 1 || T > 65536 || C < 1 || W < 1 || N_slots < 1) return RGDR_ERR_SHAPE;
    if (C % 8 != 0 || W < 2 || W > 4 || (flags & ~(uint32_t)LA_CONV_SILU)) return RGDR_ERR_UNSUPPORTED;
    if (dtype != RGDR_F32 && dtype != RGDR_F16 && dtype != RGDR_BF16) return RGDR_ERR_DTYPE;
    if (B == 0) return RGDR_OK;
    if (!x || !weight || !state_pool || !out || !state_out) return RGDR_ERR_NULL;
    ConvArgs a;
    a.sx = la_strides_or(x_strides, (long long)T * C, 0, C);
    a.so = la_strides_or(out_strides, (long long)T * C, 0, C);
    if (!la_strides_ok(a.sx) || !la_strides_ok(a.so) || !la_extent_ok(a.sx, B, 1, T, C) ||
        !la_rows_distinct(a.so, B, 1, T, C) || out == x || (!ssm_state_indices && N_slots < B))
        return RGDR_ERR_SHAPE;
    if (!la_strides_aligned(a.sx, B, 1, T) || !la_strides_aligned(a.so, B, 1, T)) return RGDR_ERR_ALIGN;
    if (!aligned(x, 16) || !aligned(weight, 16) || (bias && !aligned(bias, 16)) || !aligned(state_pool, 16) ||
        !aligned(out, 16) || !aligned(state_out, 16) || !la_index_aligned(actual_seq_lengths, ssm_state_indices, num_accepted_tokens))
        return RGDR_ERR_ALIGN;
    a.x = x;
    a.pool = state_pool;
    a.weight = weight;
    a.bias = bias;
    a.out = out;
    a.pool_out = state_out;
    a.lens = actual_seq_lengths;
    a.idx = ssm_state_indices;
    a.nacc = num_accepted_tokens;
    a.B = B;
    a.T = T;
    a.C = C;
    a.N_slots = N_slots;
    a.silu = (flags & LA_CONV_SILU) != 0;
    if (dtype == RGDR_F32) return launch_conv<float>(a, W, stream);
    if (dtype == RGDR_F16) return launch_conv<_Float16>(a, W, stream);
    return launch_conv<uint16_t>(a, W, stream);
}
