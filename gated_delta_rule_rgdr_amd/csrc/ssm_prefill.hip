// ssm_prefill.hip -- the selective state space scan over whole prompts.
#include "ssm_common.h"

namespace rgdr {

constexpr int kTC = 32;  // tokens of a chunk
constexpr int kCH = 64;  // channels of a workgroup
constexpr int kRow = kTC + 4;                           // floats of a channel's row in LDS: d, or d x and then y
constexpr int kRows = kCH * kRow + (kCH / 8 - 1) * 4;   // rows of eight channels start 4 floats further
__device__ __forceinline__ int ssm_at(int c, int t) { return c * kRow + (c >> 3) * 4 + t; }

struct SsmPlan {
    int c_blocks, groups;  // groups of B and C that a workgroup's channels may belong to
    int segs, seg_len;
    float *ends;  // [B][segs][C][N]: a segment's end state from zero, then its incoming state
    float *sums;  // [B][segs][C]: its sum of d
};

enum SsmPass { kSsmWhole, kSsmEnds, kSsmSegment };

// A workgroup has 64 channels of one entry and works through chunks of 32 tokens (of the entry, or of one
// of its segments). What is done once for each token and channel (softplus, d x, the gate) and all memory
// access goes by (token, 8 channels) for each thread, whole 16-byte pieces; the states go by channel:
// four lanes, 16 apart, hold a channel's N states, so that a lane has N / 4 of them in registers for
// all tokens. d, d x and the sums over the states pass between the two through LDS, as do B and C in fp32.
// The four lanes' sums of four tokens meet in three register swaps, which leave each lane with one
// token's.
template <typename E, int N, int PASS>
__global__ __launch_bounds__(256) void ssm_prefill_kernel(const SsmArgs a, const SsmPlan p, const bool state_f32) {
    constexpr int NP = N / 4;
    extern __shared__ __align__(16) float lds[];
    float *sd = lds, *su = lds + kRows, *sB = su + kRows, *sC = sB + p.groups * kTC * N;
    const int cb = blockIdx.x % p.c_blocks, s = blockIdx.x / p.c_blocks % p.segs;
    const int b = blockIdx.x / p.c_blocks / p.segs;
    const int c0 = cb * kCH, Cg = a.C / a.G;
    const LaEntry e = ssm_entry(a, b);
    const int t_begin = s * p.seg_len, t_end = min(e.L, t_begin + p.seg_len);
    if (PASS == kSsmEnds && t_begin + p.seg_len >= e.L) return;

    // by token and 8 channels
    const int st = threadIdx.x / 8, sc = threadIdx.x % 8 * 8, cs = c0 + sc;
    const bool c_ok = cs < a.C;
    const E *px = static_cast<const E *>(a.x) + b * a.sx.b + cs;
    const E *pdt = static_cast<const E *>(a.dt) + b * a.sdt.b + cs;
    const E *pz = static_cast<const E *>(a.z) + b * a.sz.b + cs;
    E *pout = static_cast<E *>(a.out) + b * a.so.b + cs;
    if (PASS != kSsmEnds && c_ok) {
        const float none[8] = {};
        for (int t = max(e.L, t_begin) + st; t < min(a.T, t_begin + p.seg_len); t += kTC)
            row_put(pout + (long long)t * a.so.t, none);
    }

    // by channel and a quarter of its states
    const int q = threadIdx.x / 16 % 4, c = threadIdx.x / 64 * 16 + threadIdx.x % 16, cc = c0 + c;
    const int g0 = c0 / Cg, gl = min(cc, a.C - 1) / Cg - g0;
    const size_t slot_at = ((size_t)(e.state ? e.slot : 0) * a.C + cc) * N + q * NP;
    const size_t seg_at = ((size_t)(b * p.segs + s) * a.C + cc) * N + q * NP;
    const auto commit = [&](const float (&h)[NP]) {
        if (cc >= a.C) return;
        if (state_f32) {
            float *to = static_cast<float *>(a.pool_out) + slot_at;
#pragma unroll
            for (int i = 0; i < NP; ++i) to[i] = h[i];
        } else {
            uint16_t *to = static_cast<uint16_t *>(a.pool_out) + slot_at;
#pragma unroll
            for (int i = 0; i < NP; ++i) to[i] = f32_to_bf16(h[i]);
        }
    };
    float h[NP], A[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        h[i] = A[i] = 0.f;
        if (cc >= a.C || !e.state) continue;
        A[i] = ssm_log2_decay(a.A[(size_t)cc * N + q * NP + i]);
        if (PASS == kSsmWhole)
            h[i] = state_f32 ? static_cast<const float *>(a.pool)[slot_at + i]
                             : bf16_to_f32(static_cast<const uint16_t *>(a.pool)[slot_at + i]);
        if (PASS == kSsmSegment && t_begin < max(e.L, 1)) h[i] = p.ends[seg_at + i];
    }
    if (PASS != kSsmEnds && s == 0 && e.state && e.n == 0 && !a.in_place) commit(h);

    float bias[8], D[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bias[i] = c_ok && a.dt_bias ? a.dt_bias[cs + i] : 0.f;
        D[i] = c_ok && a.D ? a.D[cs + i] : 0.f;
    }
    Row<E, 8> x, dt, z, nx, ndt, nz;
    Row<E, NP> bc, nbc;
    const bool is_C = threadIdx.x % 8 >= 4;
    const int col = threadIdx.x % 4 * NP;
    const auto bc_row = [&](int t, int g) {
        return is_C ? static_cast<const E *>(a.Cm) + b * a.sC.b + (long long)t * a.sC.t + g * a.sC.h + col
                    : static_cast<const E *>(a.Bm) + b * a.sB.b + (long long)t * a.sB.t + g * a.sB.h + col;
    };
    const auto load = [&](int t0, Row<E, 8> &x, Row<E, 8> &dt, Row<E, 8> &z, Row<E, NP> &bc) {
        x.zero();
        dt.zero();
        z.zero();
        bc.zero();
        const int t = t0 + st;
        if (t >= t_end) return;
        if (c_ok) {
            x.load(px + (long long)t * a.sx.t);
            dt.load(pdt + (long long)t * a.sdt.t);
            if (PASS != kSsmEnds && a.z) z.load(pz + (long long)t * a.sz.t);
        }
        if (PASS != kSsmEnds || !is_C) bc.load(bc_row(t, g0));
    };
    load(t_begin, x, dt, z, bc);

    float sum = 0.f;
    for (int t0 = t_begin; t0 < t_end;) {
        // (the accepted tokens end a chunk, so that the state after them is the one at its end)
        int t1 = min(t0 + kTC, t_end);
        if (t0 < e.n) t1 = min(t1, e.n);
        const bool live = t0 + st < t1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = live ? ssm_step(dt.get(i), bias[i], a.softplus) : 0.f;
            sd[ssm_at(sc + i, st)] = d;
            su[ssm_at(sc + i, st)] = live ? d * x.get(i) : 0.f;
        }
        for (int g = 0; g < p.groups; ++g) {
            if (g > 0) {
                bc.zero();
                if (live && g0 + g < a.G) bc.load(bc_row(t0 + st, g0 + g));
            }
            float *to = (is_C ? sC : sB) + (g * kTC + st) * N + col;
#pragma unroll
            for (int i = 0; i < NP; ++i) to[i] = live ? bc.get(i) : 0.f;
        }
        __syncthreads();
        load(t1, nx, ndt, nz, nbc);
        const float *tB = sB + gl * kTC * N + q * NP, *tC = sC + gl * kTC * N + q * NP;
        const int groups4 = (t1 - t0 + 3) / 4;
        for (int k = 0; k < groups4; ++k) {
            const f32x4 d4 = *reinterpret_cast<const f32x4 *>(sd + ssm_at(c, 4 * k));
            const f32x4 u4 = *reinterpret_cast<const f32x4 *>(su + ssm_at(c, 4 * k));
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float *rB = tB + (4 * k + j) * N, *rC = tC + (4 * k + j) * N;
                y[j] = 0.f;
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(d4[j] * A[i]), h[i], u4[j] * rB[i]);
                    if (PASS != kSsmEnds) y[j] = __builtin_fmaf(rC[i], h[i], y[j]);
                }
            }
            if (PASS == kSsmEnds) {
                sum += (d4[0] + d4[1]) + (d4[2] + d4[3]);
            } else {
                // lanes 32 on take tokens 2 and 3, then odd rows of 16 lanes the odd tokens
                const auto r0 = __builtin_amdgcn_permlane32_swap(__float_as_uint(y[0]), __float_as_uint(y[2]), false, false);
                const auto r1 = __builtin_amdgcn_permlane32_swap(__float_as_uint(y[1]), __float_as_uint(y[3]), false, false);
                const float s0 = __uint_as_float(r0[0]) + __uint_as_float(r0[1]);
                const float s1 = __uint_as_float(r1[0]) + __uint_as_float(r1[1]);
                const auto r2 = __builtin_amdgcn_permlane16_swap(__float_as_uint(s0), __float_as_uint(s1), false, false);
                su[ssm_at(c, 4 * k + q)] = __uint_as_float(r2[0]) + __uint_as_float(r2[1]);
            }
        }
        if (PASS != kSsmEnds && t1 == e.n) commit(h);
        __syncthreads();
        if (PASS != kSsmEnds && live && c_ok) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = ssm_out(su[ssm_at(sc + i, st)], D[i], x.get(i), a.z != nullptr, z.get(i));
            row_put(pout + (long long)(t0 + st) * a.so.t, y);
        }
        x = nx;
        dt = ndt;
        z = nz;
        bc = nbc;
        t0 = t1;
    }
    if (PASS == kSsmEnds && cc < a.C) {
#pragma unroll
        for (int i = 0; i < NP; ++i) p.ends[seg_at + i] = h[i];
        if (q == 0) p.sums[(size_t)(b * p.segs + s) * a.C + cc] = sum;
    }
}

// The segments' incoming states, one after the other: a segment takes h to exp(A sum of d) h + its end
// state from zero. A thread for each four states.
__global__ __launch_bounds__(256) void ssm_ends_kernel(const SsmArgs a, const SsmPlan p, const int N,
                                                       const bool state_f32) {
    const int quads = N / 4;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int per_b = a.C * quads;
    const int b = (int)(i / per_b), r = (int)(i % per_b), c = r / quads, n0 = r % quads * 4;
    if (b >= a.B) return;
    const LaEntry e = ssm_entry(a, b);
    if (!e.state) return;
    const int segs = max(1, (e.L + p.seg_len - 1) / p.seg_len);
    const size_t slot_at = ((size_t)e.slot * a.C + c) * N + n0;
    float h[4], A[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[k] = state_f32 ? static_cast<const float *>(a.pool)[slot_at + k]
                         : bf16_to_f32(static_cast<const uint16_t *>(a.pool)[slot_at + k]);
        A[k] = ssm_log2_decay(a.A[(size_t)c * N + n0 + k]);
    }
    float *ends = p.ends + ((size_t)b * p.segs * a.C + c) * N + n0;
    const float *sums = p.sums + (size_t)b * p.segs * a.C + c;
    const size_t step = (size_t)a.C * N;
    for (int s = 0; s < segs; ++s) {
        f32x4 *at = reinterpret_cast<f32x4 *>(ends + s * step);
        f32x4 end = {0, 0, 0, 0};
        float sum = 0.f;
        if (s + 1 < segs) {
            end = *at;
            sum = sums[(size_t)s * a.C];
        }
        *at = f32x4{h[0], h[1], h[2], h[3]};
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = __builtin_fmaf(__builtin_amdgcn_exp2f(sum * A[k]), h[k], end[k]);
    }
}

static int ssm_groups(int C, int G) {
    const int Cg = C / G;
    const int most = Cg % kCH == 0 ? 1 : kCH % Cg == 0 ? kCH / Cg : (kCH - 2) / Cg + 2;
    return most < G ? most : G;
}

template <typename E, int N, int PASS>
static rgdr_status launch_ssm_pass(const SsmArgs &a, const SsmPlan &p, bool f32, hipStream_t stream) {
    const size_t lds = sizeof(float) * (2 * kRows + 2 * p.groups * kTC * N);
    if ((__int128)p.c_blocks * p.segs * a.B > kMaxGroups) return RGDR_ERR_SHAPE;
    hipLaunchKernelGGL((ssm_prefill_kernel<E, N, PASS>), dim3((unsigned)((long long)p.c_blocks * p.segs * a.B)),
                       dim3(256), lds, stream, a, p, f32);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}

template <typename E, int N>
static rgdr_status launch_ssm_prefill(const SsmArgs &a, const SsmPlan &p, bool f32, hipStream_t stream) {
    if (p.segs == 1) return launch_ssm_pass<E, N, kSsmWhole>(a, p, f32, stream);
    const long long threads = (long long)a.B * a.C * (N / 4), blocks = (threads + 255) / 256;
    if (blocks > kMaxGroups) return RGDR_ERR_SHAPE;
    rgdr_status rc = launch_ssm_pass<E, N, kSsmEnds>(a, p, f32, stream);
    if (rc != RGDR_OK) return rc;
    hipLaunchKernelGGL(ssm_ends_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a, p, N, f32);
    if (hipGetLastError() != hipSuccess) return RGDR_ERR_HIP;
    return launch_ssm_pass<E, N, kSsmSegment>(a, p, f32, stream);
}

template <typename E>
static rgdr_status launch_ssm_states(const SsmArgs &a, const SsmPlan &p, int N, bool f32, hipStream_t stream) {
    if (N == 8) return launch_ssm_prefill<E, 8>(a, p, f32, stream);
    if (N == 16) return launch_ssm_prefill<E, 16>(a, p, f32, stream);
    return launch_ssm_prefill<E, 32>(a, p, f32, stream);
}

// How many segments.
static SsmPlan ssm_plan(int B, int T, int C, int N, int G, bool whole) {
    SsmPlan p;
    p.c_blocks = (C + kCH - 1) / kCH;
    p.groups = ssm_groups(C, G);
    p.segs = 1;
    p.seg_len = T;
    p.ends = p.sums = nullptr;
    if (whole) return p;
    const long long items = (long long)p.c_blocks * B;
    if (items >= 512) return p;
    const long long want = (1024 + items - 1) / items;
    long long len = (T + want - 1) / want;
    len = (len + kTC - 1) / kTC * kTC;
    if (len < 2 * kTC) len = 2 * kTC;
    if (len * 2 > T) return p;
    p.seg_len = (int)len;
    p.segs = (int)((T + len - 1) / len);
    return p;
}
static size_t ssm_workspace(const SsmPlan &p, int B, int C, int N) {
    if (p.segs == 1) return 0;
    return sizeof(float) * (size_t)B * p.segs * C * (N + 1);
}

}  // namespace rgdr

extern "C" rgdr_status ssm_prefill_workspace_size(int32_t B, int32_t T, int32_t C, int32_t N, int32_t G,
                                                  size_t *bytes) {
    using namespace rgdr;
    if (!bytes) return RGDR_ERR_NULL;
    const rgdr_status rc = ssm_check_sizes(65536, B, T, C, N, G);
    if (rc != RGDR_OK) return rc;
    *bytes = B == 0 ? 0 : ssm_workspace(ssm_plan(B, T, C, N, G, false), B, C, N);
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
    SsmPlan p = ssm_plan(B, T, C, N, G, false);
    if (!workspace || workspace_bytes < ssm_workspace(p, B, C, N)) p = ssm_plan(B, T, C, N, G, true);
    if (p.segs > 1) {
        p.ends = static_cast<float *>(workspace);
        p.sums = p.ends + (size_t)B * p.segs * C * N;
    }
    const bool f32 = state_dtype == RGDR_F32;
    if (dtype == RGDR_F32) return launch_ssm_states<float>(a, p, N, f32, stream);
    if (dtype == RGDR_F16) return launch_ssm_states<_Float16>(a, p, N, f32, stream);
    return launch_ssm_states<uint16_t>(a, p, N, f32, stream);
}
