// ssm_decode.hip -- the selective state space scan over a few tokens (T <= 8): each state crosses the
// memory once each way, whatever T.
#include "ssm_common.h"

namespace rgdr {

template <bool F32>
struct StateType;
template <>
struct StateType<true> {
    using E = float;
};
template <>
struct StateType<false> {
    using E = uint16_t;
};

// A sum over aligned groups of LPC lanes, in each of them.
template <int LPC>
__device__ __forceinline__ float lanes_sum(float x) {
    if constexpr (LPC >= 2)
        x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0xB1, 0xF, 0xF, false));  // lane ^ 1
    if constexpr (LPC >= 4)
        x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x4E, 0xF, 0xF, false));  // lane ^ 2
    if constexpr (LPC >= 8)
        x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x141, 0xF, 0xF, false));  // other quad
    return x;
}

// What one token brings to a lane.
template <typename E, int P>
struct Token {
    E x, dt, z;
    Row<E, P> B, C;
};

// 16 bytes of state for each lane, so that a wave reads and writes 1 KB in a row: P = 4 or 8 states of a
// channel, LPC = N / P lanes for each channel. A workgroup has 256 / LPC channels of U entries: the
// channels' decays and biases are read once for all of them.
template <typename E, int N, bool F32, int TMAX, int U>
__global__ __launch_bounds__(256) void ssm_decode_kernel(const SsmArgs a, int c_blocks) {
    using S = typename StateType<F32>::E;
    constexpr int P = 16 / sizeof(S), LPC = N / P;
    const int c = blockIdx.x % c_blocks * (256 / LPC) + threadIdx.x / LPC, n0 = threadIdx.x % LPC * P;
    const int b0 = blockIdx.x / c_blocks * U;
    if (c >= a.C) return;
    const int g = c / (a.C / a.G);

    LaEntry e[U];
    Row<S, P> h0[U];
    Token<E, P> tok[U][TMAX];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int b = b0 + u;
        if (b >= a.B) {
            e[u] = LaEntry{0, 0, 0, false};
            continue;
        }
        e[u] = ssm_entry(a, b);
        if (e[u].state)
            h0[u].load(static_cast<const S *>(a.pool) + ((size_t)e[u].slot * a.C + c) * N + n0);
#pragma unroll
        for (int t = 0; t < TMAX; ++t) {
            if (t < e[u].L) {
                tok[u][t].x = *(static_cast<const E *>(a.x) + b * a.sx.b + t * a.sx.t + c);
                tok[u][t].dt = *(static_cast<const E *>(a.dt) + b * a.sdt.b + t * a.sdt.t + c);
                if (a.z) tok[u][t].z = *(static_cast<const E *>(a.z) + b * a.sz.b + t * a.sz.t + c);
                tok[u][t].B.load(static_cast<const E *>(a.Bm) + b * a.sB.b + t * a.sB.t + g * a.sB.h + n0);
                tok[u][t].C.load(static_cast<const E *>(a.Cm) + b * a.sC.b + t * a.sC.t + g * a.sC.h + n0);
            }
        }
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, D = a.D ? a.D[c] : 0.f;
    Row<float, P> Ar;
    Ar.load(a.A + (size_t)c * N + n0);
    float A[P];
#pragma unroll
    for (int i = 0; i < P; ++i) A[i] = ssm_log2_decay(Ar.get(i));

#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int b = b0 + u;
        if (b >= a.B) return;
        const LaEntry en = e[u];
        E *out = static_cast<E *>(a.out) + b * a.so.b + c;
        S *to = static_cast<S *>(a.pool_out) + ((size_t)(en.state ? en.slot : 0) * a.C + c) * N + n0;
        float h[P];
#pragma unroll
        for (int i = 0; i < P; ++i) h[i] = en.state ? h0[u].get(i) : 0.f;
        if (en.state && en.n == 0 && !a.in_place) row_put(to, h);
#pragma unroll
        for (int t = 0; t < TMAX; ++t) {
            if (t >= a.T) break;
            float y = 0.f;
            if (t < en.L) {
                const Token<E, P> &k = tok[u][t];
                const float x = row_value(k.x), d = ssm_step(row_value(k.dt), bias, a.softplus);
                const float dx = d * x;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * A[i]), h[i], dx * k.B.get(i));
                    y = __builtin_fmaf(k.C.get(i), h[i], y);
                }
                y = lanes_sum<LPC>(y);
                y = ssm_out(y, D, x, a.z != nullptr, a.z ? row_value(k.z) : 0.f);
                if (t + 1 == en.n) row_put(to, h);
            }
            if (n0 == 0) out[t * a.so.t] = t < en.L ? row_store<E>(y) : E(0);
        }
    }
}

// Several tokens and groups of at least CH channels: a workgroup has up to CH channels of one entry and
// group. Its threads load the tokens' x, dt and z in pieces of 16 bytes of one token, compute each d and d x once,
// and pass them on in LDS, with B and C; the sums over the states come back the same way. (Without it
// each lane loads two bytes of them for each token, five loads in all, and computes the same d in LPC lanes.)
template <typename E, int N, bool F32>
__global__ __launch_bounds__(256) void ssm_decode_tokens_kernel(const SsmArgs a, int c_blocks) {
    using S = typename StateType<F32>::E;
    constexpr int P = 16 / sizeof(S), LPC = N / P, CH = 256 / LPC, PIECES = CH / 8;
    __shared__ __align__(16) float sd[kMaxT][CH], su[kMaxT][CH], sB[kMaxT][N], sC[kMaxT][N];
    const int b = blockIdx.x / c_blocks, cb = blockIdx.x % c_blocks;
    const int Cg = a.C / a.G, per = (Cg - 1) / CH + 1, g = cb / per;
    const int c0 = g * Cg + cb % per * CH, channels = min(CH, Cg - cb % per * CH);
    const LaEntry e = ssm_entry(a, b);

    const int c = threadIdx.x / LPC, n0 = threadIdx.x % LPC * P;
    const bool mine = e.state && c < channels;
    const size_t at = ((size_t)(e.state ? e.slot : 0) * a.C + c0 + c) * N + n0;
    Row<S, P> h0;
    Row<float, P> Ar;
    h0.zero();
    Ar.zero();
    if (mine) {
        h0.load(static_cast<const S *>(a.pool) + at);
        Ar.load(a.A + (size_t)(c0 + c) * N + n0);
    }
    // pieces of tokens: PIECES threads for each, 256 / PIECES tokens at once
    constexpr int AT_ONCE = 256 / PIECES, SETS = (kMaxT + AT_ONCE - 1) / AT_ONCE;
    const int pc = threadIdx.x % PIECES * 8, pt = threadIdx.x / PIECES;
    const bool p_ok = pc < channels;
    Row<E, 8> x[SETS], dt[SETS], z[SETS];
    Row<float, 8> bias, D;
    bias.zero();
    D.zero();
    if (p_ok && a.dt_bias) bias.load(a.dt_bias + c0 + pc);
    if (p_ok && a.D) D.load(a.D + c0 + pc);
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
        const int t = pt + s * AT_ONCE;
        x[s].zero();
        dt[s].zero();
        z[s].zero();
        if (t < e.L && p_ok) {
            x[s].load(static_cast<const E *>(a.x) + b * a.sx.b + t * a.sx.t + c0 + pc);
            dt[s].load(static_cast<const E *>(a.dt) + b * a.sdt.b + t * a.sdt.t + c0 + pc);
            if (a.z) z[s].load(static_cast<const E *>(a.z) + b * a.sz.b + t * a.sz.t + c0 + pc);
        }
    }
    constexpr int BC = kMaxT * 2 * N / 8;  // pieces of 8 values of B and C
    static_assert(BC <= 256, "one for each thread");
    if (threadIdx.x < BC) {
        const int t = threadIdx.x / (2 * N / 8), i = threadIdx.x % (2 * N / 8) * 8;
        if (t < e.L) {
            Row<E, 8> r;
            if (i < N)
                r.load(static_cast<const E *>(a.Bm) + b * a.sB.b + t * a.sB.t + g * a.sB.h + i);
            else
                r.load(static_cast<const E *>(a.Cm) + b * a.sC.b + t * a.sC.t + g * a.sC.h + i - N);
            float *to = i < N ? &sB[t][i] : &sC[t][i - N];
#pragma unroll
            for (int k = 0; k < 8; ++k) to[k] = r.get(k);
        }
    }
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
        const int t = pt + s * AT_ONCE;
        if (t >= e.L) continue;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float d = ssm_step(dt[s].get(k), bias.get(k), a.softplus);
            sd[t][pc + k] = d;
            su[t][pc + k] = d * x[s].get(k);
        }
    }
    __syncthreads();
    float h[P], A[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        h[i] = h0.get(i);
        A[i] = ssm_log2_decay(Ar.get(i));
    }
    S *to = static_cast<S *>(a.pool_out) + at;
    if (mine && e.n == 0 && !a.in_place) row_put(to, h);
#pragma unroll
    for (int t = 0; t < kMaxT; ++t) {
        if (t >= e.L) break;
        const float d = sd[t][c], u = su[t][c];
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * A[i]), h[i], u * sB[t][n0 + i]);
            y = __builtin_fmaf(sC[t][n0 + i], h[i], y);
        }
        y = lanes_sum<LPC>(y);
        if (n0 == 0) su[t][c] = y;
        if (t + 1 == e.n && mine) row_put(to, h);
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
        const int t = pt + s * AT_ONCE;
        if (t >= a.T || !p_ok) continue;
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            y[k] = t < e.L ? ssm_out(su[t][pc + k], D.get(k), x[s].get(k), a.z != nullptr, z[s].get(k)) : 0.f;
        row_put(static_cast<E *>(a.out) + b * a.so.b + t * a.so.t + c0 + pc, y);
    }
}

// One token: two entries for each workgroup, which read the channels' A, D and biases once (B=256, C=4096,
// N=16, fp32 states: 25.7 us, 5.6 TB/s, against 28.7 with one and 25.7 with four; B=64 9.0, 10.3 and 9.5).
// Several tokens by way of LDS where that saves more than its barriers cost: from 5 tokens, or 3 in large
// calls. us, by way of LDS against each lane's own loads, C=4096, N=16, fp32 states: 8 tokens B=1 5.4/5.5, B=8
// 5.8/7.0, B=32 10.5/16.1; 4 tokens B=1 4.8/4.1, B=16 6.4/6.3; 3 tokens B=16 6.1/5.5, B=128 23.2/27.6; 2
// tokens B=32 8.1/7.4, B=256 40.6/41.7. B=32, up to 8 tokens, bf16 states, G=8: 8.8/10.4.
template <typename E, int N, bool F32>
static rgdr_status launch_ssm_tokens(const SsmArgs &a, hipStream_t stream) {
    constexpr int CH = 256 / (N * (F32 ? 4 : 2) / 16);
    const int Cg = a.C / a.G;
    const bool large = (long long)a.B * a.G * (Cg / CH) >= 2048;
    const bool tokens = Cg >= CH && (a.T >= 5 || (a.T >= 3 && large));
    const long long c_blocks = tokens ? (long long)a.G * ((Cg - 1) / CH + 1) : ((long long)a.C + CH - 1) / CH;
    const long long b_blocks = a.T > 1 ? a.B : ((long long)a.B + 1) / 2;
    if ((__int128)c_blocks * b_blocks > kMaxGroups) return RGDR_ERR_SHAPE;
    const dim3 grid((unsigned)(c_blocks * b_blocks)), block(256);
    if (tokens)
        hipLaunchKernelGGL((ssm_decode_tokens_kernel<E, N, F32>), grid, block, 0, stream, a, (int)c_blocks);
    else if (a.T > 1)
        hipLaunchKernelGGL((ssm_decode_kernel<E, N, F32, kMaxT, 1>), grid, block, 0, stream, a, (int)c_blocks);
    else
        hipLaunchKernelGGL((ssm_decode_kernel<E, N, F32, 1, 2>), grid, block, 0, stream, a, (int)c_blocks);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}

template <typename E>
static rgdr_status launch_ssm_states(const SsmArgs &a, int N, bool f32, hipStream_t stream) {
    if (N == 8) return f32 ? launch_ssm_tokens<E, 8, true>(a, stream) : launch_ssm_tokens<E, 8, false>(a, stream);
    if (N == 16) return f32 ? launch_ssm_tokens<E, 16, true>(a, stream) : launch_ssm_tokens<E, 16, false>(a, stream);
    return f32 ? launch_ssm_tokens<E, 32, true>(a, stream) : launch_ssm_tokens<E, 32, false>(a, stream);
}

rgdr_status ssm_check_sizes(int max_t, int32_t B, int32_t T, int32_t C, int32_t N, int32_t G) {
    if (B < 0 || T < 1 || T > max_t || C < 1 || N < 1 || G < 1 || C % G != 0) return RGDR_ERR_SHAPE;
    if (C / G % 8 != 0 || (N != 8 && N != 16 && N != 32)) return RGDR_ERR_UNSUPPORTED;
    return RGDR_OK;
}

// The argument checks of both entries, and the kernels' argument block. B = 0 is RGDR_OK with nothing
// to launch.
rgdr_status ssm_check(SsmArgs &a, int max_t, const void *x, const la_strides *x_strides, const void *dt,
                             const la_strides *dt_strides, const float *A, const void *Bm,
                             const la_strides *Bm_strides, const void *Cm, const la_strides *Cm_strides,
                             const float *D, const void *z, const la_strides *z_strides, const float *dt_bias,
                             int dtype, const void *state_pool, int state_dtype, const int32_t *lens,
                             const int32_t *idx, const int32_t *nacc, uint32_t flags, int32_t B, int32_t T,
                             int32_t C, int32_t N, int32_t G, int32_t N_slots, void *out,
                             const la_strides *out_strides, void *state_out) {
    const rgdr_status rc = ssm_check_sizes(max_t, B, T, C, N, G);
    if (rc != RGDR_OK) return rc;
    if (N_slots < 1) return RGDR_ERR_SHAPE;
    if (flags & ~(uint32_t)SSM_DT_SOFTPLUS) return RGDR_ERR_UNSUPPORTED;
    if (dtype != RGDR_F32 && dtype != RGDR_F16 && dtype != RGDR_BF16) return RGDR_ERR_DTYPE;
    if (state_dtype != RGDR_F32 && state_dtype != RGDR_BF16) return RGDR_ERR_DTYPE;
    a.B = B;
    if (B == 0) return RGDR_OK;
    if (!x || !dt || !A || !Bm || !Cm || !state_pool || !out || !state_out) return RGDR_ERR_NULL;
    a.sx = la_strides_or(x_strides, (long long)T * C, 0, C);
    a.sdt = la_strides_or(dt_strides, (long long)T * C, 0, C);
    a.sz = la_strides_or(z ? z_strides : nullptr, (long long)T * C, 0, C);
    a.so = la_strides_or(out_strides, (long long)T * C, 0, C);
    a.sB = la_strides_or(Bm_strides, (long long)T * G * N, N, (long long)G * N);
    a.sC = la_strides_or(Cm_strides, (long long)T * G * N, N, (long long)G * N);
    const long long max_stride = dtype == RGDR_F32 ? kMaxTokenStride / 2 : kMaxTokenStride;
    for (const LaStrides *s : {&a.sx, &a.sdt, &a.sz, &a.so})
        if (!la_strides_ok(*s) || (T > 1 && s->t > max_stride) || !la_extent_ok(*s, B, 1, T, C)) return RGDR_ERR_SHAPE;
    for (const LaStrides *s : {&a.sB, &a.sC})
        if (!la_strides_ok(*s) || (T > 1 && s->t > max_stride) || !la_extent_ok(*s, B, G, T, N)) return RGDR_ERR_SHAPE;
    if (!la_rows_distinct(a.so, B, 1, T, C) || (!idx && N_slots < B)) return RGDR_ERR_SHAPE;
    for (const LaStrides *s : {&a.sx, &a.sdt, &a.so})
        if (!la_strides_aligned(*s, B, 1, T)) return RGDR_ERR_ALIGN;
    if ((z && !la_strides_aligned(a.sz, B, 1, T)) || !la_strides_aligned(a.sB, B, G, T) ||
        !la_strides_aligned(a.sC, B, G, T))
        return RGDR_ERR_ALIGN;
    for (const void *p : {x, dt, (const void *)A, Bm, Cm, (const void *)D, z, (const void *)dt_bias, state_pool,
                          (const void *)out, (const void *)state_out})
        if (!aligned(p, 16)) return RGDR_ERR_ALIGN;
    if (!la_index_aligned(lens, idx, nacc)) return RGDR_ERR_ALIGN;
    a.x = x;
    a.dt = dt;
    a.z = z;
    a.Bm = Bm;
    a.Cm = Cm;
    a.pool = state_pool;
    a.A = A;
    a.D = D;
    a.dt_bias = dt_bias;
    a.out = out;
    a.pool_out = state_out;
    a.lens = lens;
    a.idx = idx;
    a.nacc = nacc;
    a.T = T;
    a.C = C;
    a.G = G;
    a.N_slots = N_slots;
    a.softplus = (flags & SSM_DT_SOFTPLUS) != 0;
    a.in_place = state_out == state_pool;
    return RGDR_OK;
}

}  // namespace rgdr

extern "C" rgdr_status ssm_decode(const void *x, const la_strides *x_strides, const void *dt,
                                  const la_strides *dt_strides, const float *A, const void *Bm,
                                  const la_strides *Bm_strides, const void *Cm, const la_strides *Cm_strides,
                                  const float *D, const void *z, const la_strides *z_strides,
                                  const float *dt_bias, rgdr_dtype dtype, const void *state_pool,
                                  rgdr_dtype state_dtype, const int32_t *actual_seq_lengths,
                                  const int32_t *ssm_state_indices, const int32_t *num_accepted_tokens,
                                  uint32_t flags, int32_t B, int32_t T, int32_t C, int32_t N, int32_t G,
                                  int32_t N_slots, void *out, const la_strides *out_strides, void *state_out,
                                  hipStream_t stream) {
    using namespace rgdr;
    SsmArgs a;
    const rgdr_status rc =
        ssm_check(a, kMaxT, x, x_strides, dt, dt_strides, A, Bm, Bm_strides, Cm, Cm_strides, D, z, z_strides, dt_bias,
                  dtype, state_pool, state_dtype, actual_seq_lengths, ssm_state_indices, num_accepted_tokens, flags,
                  B, T, C, N, G, N_slots, out, out_strides, state_out);
    if (rc != RGDR_OK || B == 0) return rc;
    const bool f32 = state_dtype == RGDR_F32;
    if (dtype == RGDR_F32) return launch_ssm_states<float>(a, N, f32, stream);
    if (dtype == RGDR_F16) return launch_ssm_states<_Float16>(a, N, f32, stream);
    return launch_ssm_states<uint16_t>(a, N, f32, stream);
}
