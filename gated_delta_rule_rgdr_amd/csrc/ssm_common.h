// ssm_common.h -- what the selective state space scan's kernels for few tokens (ssm_decode.hip) and for
// prompts (ssm_prefill.hip) share: the argument block, its checks, and the arithmetic of a token. Not
// part of the C ABI.
//
// On the N states h of each channel, token by token:
//     d = softplus(dt + dt_bias),  h[n] = exp(d A[n]) h[n] + d x B[n],
//     y = (sum_n C[n] h[n] + D x) silu(z).
// exp(d A) is exp2(d (A log2 e)), with A log2 e rounded once: the hardware's exponential is to base 2.
#pragma once

#include "la_common.h"

namespace rgdr {

struct SsmArgs {
    const void *x, *dt, *z, *Bm, *Cm, *pool;
    const float *A, *D, *dt_bias;  // z, D, dt_bias may be null
    void *out, *pool_out;
    const int32_t *lens, *idx, *nacc;  // each may be null
    LaStrides sx, sdt, sz, sB, sC, so;
    int B, T, C, G, N_slots;
    bool softplus, in_place;
};

__device__ __forceinline__ LaEntry ssm_entry(const SsmArgs &a, int b) {
    LaEntry e;
    e.slot = a.idx ? a.idx[b] : b;
    e.state = e.slot >= 0 && e.slot < a.N_slots;
    const int L = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    e.L = e.state ? L : 0;
    e.n = a.nacc ? min(max(a.nacc[b], 0), e.L) : e.L;
    return e;
}

// A log2 e; minus infinity acts as a large negative number, so that a step of 0 keeps the state.
__device__ __forceinline__ float ssm_log2_decay(float A) {
    const float l = A * 1.44269504088896340736f;
    return l < -3e38f ? -3e38f : l;
}
// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|). u = 1 + e rounded loses w = e - (u - 1), at most
// 2^-24: log1p(e) = log(u) + log(1 + w / u), and w instead of the last term is off by w (1 - 1 / u) at
// most, below 2^-24 of the sum. u is in [1, 2], so the hardware's logarithm needs no scaling. NaN and
// infinities pass.
__device__ __forceinline__ float ssm_softplus(float x) {
    const float e = __builtin_amdgcn_exp2f(-1.44269504088896340736f * __builtin_fabsf(x));
    const float u = 1.0f + e, w = e - (u - 1.0f);
    return __builtin_fmaf(__builtin_amdgcn_logf(u), 0.693147180559945309417f, __builtin_fmaxf(x, 0.f)) + w;
}
__device__ __forceinline__ float ssm_step(float dt, float bias, bool softplus) {
    const float s = dt + bias;
    return softplus ? ssm_softplus(s) : s;
}
// (sum + D x) silu(z)
__device__ __forceinline__ float ssm_out(float sum, float D, float x, bool gated, float z) {
    const float y = __builtin_fmaf(D, x, sum);
    if (!gated) return y;
    return y * (z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * z)));
}

// The argument checks of ssm_decode and ssm_prefill (T up to max_t), and the kernels' argument block.
// B = 0 is RGDR_OK with nothing to launch.
rgdr_status ssm_check_sizes(int max_t, int32_t B, int32_t T, int32_t C, int32_t N, int32_t G);
rgdr_status ssm_check(SsmArgs &a, int max_t, const void *x, const la_strides *x_strides, const void *dt,
                      const la_strides *dt_strides, const float *A, const void *Bm, const la_strides *Bm_strides,
                      const void *Cm, const la_strides *Cm_strides, const float *D, const void *z,
                      const la_strides *z_strides, const float *dt_bias, int dtype, const void *state_pool,
                      int state_dtype, const int32_t *lens, const int32_t *idx, const int32_t *nacc, uint32_t flags,
                      int32_t B, int32_t T, int32_t C, int32_t N, int32_t G, int32_t N_slots, void *out,
                      const la_strides *out_strides, void *state_out);

}  // namespace rgdr
