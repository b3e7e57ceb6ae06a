// ssm_scan.hip -- the selective state space scan (ssm_decode, ssm_prefill): on the N states h of each
// channel, token by token,
//     d = softplus(dt + dt_bias),  h[n] = exp(d A[n]) h[n] + d x B[n],
//     y = (sum_n C[n] h[n] + D x) silu(z).
#include "la_common.h"

namespace rgdr {

struct SsmArgs {
    const void *x, *dt, *z, *Bm, *Cm, *pool;
    const float *A, *D, *dt_bias;  // D, z, dt_bias may be null
    void *out, *pool_out;
    const int32_t *lens, *idx, *nacc;  // each may be null
    LaStrides sx, sdt, sz, sB, sC, so;
    int B, T, C, G, N_slots, softplus;
    bool state_f32, in_place;
};

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ LaEntry ssm_entry(const SsmArgs &a, int b) {
    LaEntry e;
    e.slot = a.idx ? a.idx[b] : b;
    e.state = e.slot >= 0 && e.slot < a.N_slots;
    const int L = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    e.L = e.state ? L : 0;
    e.n = a.nacc ? min(max(a.nacc[b], 0), e.L) : e.L;
    return e;
}

template <bool F32>
__device__ __forceinline__ float state_get(const void *pool, size_t i) {
    if constexpr (F32) return static_cast<const float *>(pool)[i];
    return bf16_to_f32(static_cast<const uint16_t *>(pool)[i]);
}
template <bool F32>
__device__ __forceinline__ void state_put(void *pool, size_t i, float v) {
    if constexpr (F32)
        static_cast<float *>(pool)[i] = v;
    else
        static_cast<uint16_t *>(pool)[i] = f32_to_bf16(v);
}

// A thread for each channel, its states in registers, the tokens in order.
template <typename E, int N, bool F32>
__global__ __launch_bounds__(64) void ssm_scan_kernel(const SsmArgs a, int c_blocks) {
    const int b = blockIdx.x / c_blocks;
    const int c = blockIdx.x % c_blocks * 64 + threadIdx.x;
    if (c >= a.C) return;
    const LaEntry e = ssm_entry(a, b);
    const int g = c / (a.C / a.G);
    const E *x = static_cast<const E *>(a.x) + b * a.sx.b + c;
    const E *dt = static_cast<const E *>(a.dt) + b * a.sdt.b + c;
    const E *z = static_cast<const E *>(a.z) + b * a.sz.b + c;
    const E *Bm = static_cast<const E *>(a.Bm) + b * a.sB.b + g * a.sB.h;
    const E *Cm = static_cast<const E *>(a.Cm) + b * a.sC.b + g * a.sC.h;
    E *out = static_cast<E *>(a.out) + b * a.so.b + c;
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, D = a.D ? a.D[c] : 0.f;
    const size_t at = ((size_t)(e.state ? e.slot : 0) * a.C + c) * N;
    float h[N], A[N];
    for (int n = 0; n < N; ++n) {
        h[n] = e.state ? state_get<F32>(a.pool, at + n) : 0.f;
        A[n] = a.A[(size_t)c * N + n] * kLog2e;
    }
    const bool commit = e.state && (e.n > 0 || !a.in_place);
    for (int t = 0; t <= e.L; ++t) {
        if (t == e.n && commit)
            for (int n = 0; n < N; ++n) state_put<F32>(a.pool_out, at + n, h[n]);
        if (t == e.L) break;
        const float xv = row_value(x[t * a.sx.t]);
        float d = row_value(dt[t * a.sdt.t]) + bias;
        if (a.softplus) d = softplus_fast(d);
        const float u = d * xv;
        float y = 0.f;
        for (int n = 0; n < N; ++n) {
            h[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * A[n]), h[n], u * row_value(Bm[t * a.sB.t + n]));
            y = __builtin_fmaf(row_value(Cm[t * a.sC.t + n]), h[n], y);
        }
        if (a.D) y = __builtin_fmaf(D, xv, y);
        if (a.z) {
            const float zv = row_value(z[t * a.sz.t]);
            y *= zv * sigmoid_fast(zv);
        }
        out[t * a.so.t] = row_store<E>(y);
    }
    for (int t = e.L; t < a.T; ++t) out[t * a.so.t] = E(0);
}

template <typename E, int N, bool F32>
static rgdr_status launch_ssm(const SsmArgs &a, hipStream_t stream) {
    const long long c_blocks = ((long long)a.C + 63) / 64;
    if ((__int128)c_blocks * a.B > kMaxGroups) return RGDR_ERR_SHAPE;
    hipLaunchKernelGGL((ssm_scan_kernel<E, N, F32>), dim3((unsigned)(c_blocks * a.B)), dim3(64), 0, stream, a,
                       (int)c_blocks);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}

template <typename E>
static rgdr_status launch_ssm_states(const SsmArgs &a, int N, hipStream_t stream) {
    if (N == 8) return a.state_f32 ? launch_ssm<E, 8, true>(a, stream) : launch_ssm<E, 8, false>(a, stream);
    if (N == 16) return a.state_f32 ? launch_ssm<E, 16, true>(a, stream) : launch_ssm<E, 16, false>(a, stream);
    return a.state_f32 ? launch_ssm<E, 32, true>(a, stream) : launch_ssm<E, 32, false>(a, stream);
}

static rgdr_status ssm_check_sizes(int max_t, int32_t B, int32_t T, int32_t C, int32_t N, int32_t G) {
    if (B < 0 || T < 1 || T > max_t || C < 1 || N < 1 || G < 1 || C % G != 0) return RGDR_ERR_SHAPE;
    if (C % 8 != 0 || (N != 8 && N != 16 && N != 32)) return RGDR_ERR_UNSUPPORTED;
    return RGDR_OK;
}

// The argument checks of both entries, and the kernels' argument block. B = 0 is RGDR_OK with nothing
// to launch.
static rgdr_status ssm_check(SsmArgs &a, int max_t, const void *x, const la_strides *x_strides, const void *dt,
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
    a.sz = la_strides_or(z_strides, (long long)T * C, 0, C);
    a.so = la_strides_or(out_strides, (long long)T * C, 0, C);
    a.sB = la_strides_or(Bm_strides, (long long)T * G * N, N, (long long)G * N);
    a.sC = la_strides_or(Cm_strides, (long long)T * G * N, N, (long long)G * N);
    for (const LaStrides *s : {&a.sx, &a.sdt, &a.sz, &a.so})
        if (!la_strides_ok(*s) || !la_extent_ok(*s, B, 1, T, C)) return RGDR_ERR_SHAPE;
    for (const LaStrides *s : {&a.sB, &a.sC})
        if (!la_strides_ok(*s) || !la_extent_ok(*s, B, G, T, N)) return RGDR_ERR_SHAPE;
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
    a.state_f32 = state_dtype == RGDR_F32;
    a.in_place = state_out == state_pool;
    return RGDR_OK;
}

static rgdr_status launch_ssm_types(const SsmArgs &a, int dtype, int N, hipStream_t stream) {
    if (dtype == RGDR_F32) return launch_ssm_states<float>(a, N, stream);
    if (dtype == RGDR_F16) return launch_ssm_states<_Float16>(a, N, stream);
    return launch_ssm_states<uint16_t>(a, N, stream);
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
    return launch_ssm_types(a, dtype, N, stream);
}

extern "C" rgdr_status ssm_prefill_workspace_size(int32_t B, int32_t T, int32_t C, int32_t N, int32_t G,
                                                  size_t *bytes) {
    using namespace rgdr;
    if (!bytes) return RGDR_ERR_NULL;
    const rgdr_status rc = ssm_check_sizes(65536, B, T, C, N, G);
    if (rc != RGDR_OK) return rc;
    *bytes = 0;
    return RGDR_OK;
}

extern "C" rgdr_status ssm_prefill(const void *x, const la_strides *x_strides, const void *dt,
                                   const la_strides *dt_strides, const float *A, const void *Bm,
                                   const la_strides *Bm_strides, const void *Cm, const la_strides *Cm_strides,
                                   const float *D, const void *z, const la_strides *z_strides,
                                   const float *dt_bias, rgdr_dtype dtype, const void *state_pool,
                                   rgdr_dtype state_dtype, const int32_t *actual_seq_lengths,
                                   const int32_t *ssm_state_indices, const int32_t *num_accepted_tokens,
                                   uint32_t flags, int32_t B, int32_t T, int32_t C, int32_t N, int32_t G,
                                   int32_t N_slots, void *out, const la_strides *out_strides, void *state_out,
                                   void *workspace, size_t workspace_bytes, hipStream_t stream) {
    using namespace rgdr;
    SsmArgs a;
    const rgdr_status rc =
        ssm_check(a, 65536, x, x_strides, dt, dt_strides, A, Bm, Bm_strides, Cm, Cm_strides, D, z, z_strides, dt_bias,
                  dtype, state_pool, state_dtype, actual_seq_lengths, ssm_state_indices, num_accepted_tokens, flags,
                  B, T, C, N, G, N_slots, out, out_strides, state_out);
    if (rc != RGDR_OK || B == 0) return rc;
    if (workspace && !aligned(workspace, 256)) return RGDR_ERR_ALIGN;
    (void)workspace_bytes;
    return launch_ssm_types(a, dtype, N, stream);
}
