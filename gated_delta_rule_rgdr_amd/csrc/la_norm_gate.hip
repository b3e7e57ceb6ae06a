// la_norm_gate.hip -- the norm and gate behind the attention: for each row of D values
//     y = weight * x / sqrt(mean(x^2) + eps) * silu(gate),
// from the attention's [B, H, T, D] to the [B, T, H, D] that the output projection reads.
#include "la_common.h"

namespace rgdr {

struct NormArgs {
    const void *x, *gate;
    const float *weight;
    void *out;
    const int32_t *lens;
    LaStrides sx, sg, so;
    long long sw;
    float eps;
    int B, H, T, D, sigmoid;
};

// Sum over aligned groups of LPR lanes, in each of them.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
    if constexpr (LPR != 32) {
        return group_sum<LPR>(x);
    } else {
        x = group_sum<16>(x);
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
}

// LPR lanes for each row, NV pieces of 16 bytes in each lane: the row stays in registers between the
// sum and the product, so x and the gate are read once. A workgroup's 256 / LPR groups of lanes
// take HR heads (2^hr_log) times TR = 256 / LPR / HR tokens, and U such sets of tokens one after
// the other with all their loads in flight: runs of several rows on both sides of the transposition
// (x keeps a head's tokens together, out a token's heads). Bound: the bytes. B=16, T=1024, H=32,
// D=128, bf16, ragged: 55.5 us (5.5 TB/s); B=64, T=1: 2.7 us (the launch); D=4096: 20.5 us for
// 4096 rows (4.9 TB/s).
template <typename E, int LPR, int NV, int U, bool GATED>
__global__ __launch_bounds__(256) void la_norm_gate_kernel(const NormArgs a, int hr_log, int h_blocks, int t_blocks) {
    using V = RowVec<E>;
    const int hb = blockIdx.x % h_blocks, tb = blockIdx.x / h_blocks % t_blocks;
    const int b = blockIdx.x / h_blocks / t_blocks;
    const int group = threadIdx.x / LPR, tr = (256 / LPR) >> hr_log;
    const int h = (hb << hr_log) + (group & ((1 << hr_log) - 1));
    const int t0 = tb * tr * U + (group >> hr_log);
    if (h >= a.H) return;
    const int L = a.lens ? min(a.lens[b], a.T) : a.T;
    const int c0 = threadIdx.x % LPR * V::N;
    const E *x = static_cast<const E *>(a.x) + b * a.sx.b + h * a.sx.h;
    const E *z = static_cast<const E *>(a.gate) + b * a.sg.b + h * a.sg.h;
    E *out = static_cast<E *>(a.out) + b * a.so.b + h * a.so.h;
    const float *w = a.weight + h * a.sw;
    u32x4 wx[U][NV], wz[U][GATED ? NV : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int t = t0 + u * tr;
#pragma unroll
        for (int m = 0; m < NV; ++m) wx[u][m] = wz[u][GATED ? m : 0] = u32x4{0, 0, 0, 0};
        if (t < L && c0 < a.D) {
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                // a lane whose further pieces lie past the row's end reads its last piece, and
                // leaves it out below
                const int c = m ? min(c0 + m * LPR * V::N, a.D - V::N) : c0;
                wx[u][m] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(x + t * a.sx.t + c));
                if (GATED) wz[u][m] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(z + t * a.sg.t + c));
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int t = t0 + u * tr;
        float ss = 0.f;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            float v[V::N], s1 = 0.f;
            V::get(v, wx[u][m]);
#pragma unroll
            for (int c = 0; c < V::N; ++c) s1 = __builtin_fmaf(v[c], v[c], s1);
            ss += m == 0 || c0 + m * LPR * V::N < a.D ? s1 : 0.f;
        }
        ss = row_sum<LPR>(ss);
        const float r = __builtin_amdgcn_rsqf(ss / (float)a.D + a.eps);
        if (t >= a.T) continue;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int c = c0 + m * LPR * V::N;
            if (c >= a.D) continue;
            float v[V::N], g[V::N];
            V::get(v, wx[u][m]);
            V::get(g, wz[u][GATED ? m : 0]);
#pragma unroll
            for (int j = 0; j < V::N / 4; ++j) {
                const f32x4 w4 = *reinterpret_cast<const f32x4 *>(w + c + j * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float &y = v[j * 4 + i];
                    const float z1 = g[j * 4 + i];
                    y *= r * w4[i];
                    if (GATED) y *= (a.sigmoid ? 1.f : z1) * sigmoid_fast(z1);
                    y = t < L ? y : 0.f;
                }
            }
            __builtin_nontemporal_store(V::put(v), reinterpret_cast<u32x4 *>(out + t * a.so.t + c));
        }
    }
}

template <typename E, int LPR, int NV, int U>
static rgdr_status launch_norm_rows(const NormArgs &a, hipStream_t stream) {
    constexpr int ROWS = 256 / LPR;
    // the split of a workgroup's rows into heads and tokens that leaves the fewest idle; of equal
    // ones the most heads
    int hr_log = 0;
    double best = 0;
    for (int k = 0; (1 << k) <= ROWS; ++k) {
        const int hr = 1 << k, tu = ROWS / hr * U;
        const double use = (double)a.H / ((a.H + (long long)hr - 1) / hr * hr) * a.T /
                           ((a.T + (long long)tu - 1) / tu * tu);
        if (use >= best) {
            best = use;
            hr_log = k;
        }
    }
    const int tu = (ROWS >> hr_log) * U;
    const long long h_blocks = ((long long)a.H + (1 << hr_log) - 1) >> hr_log;
    const long long t_blocks = ((long long)a.T + tu - 1) / tu;
    if ((__int128)h_blocks * t_blocks * a.B > kMaxGroups) return RGDR_ERR_SHAPE;
    const dim3 grid((unsigned)(h_blocks * t_blocks * a.B)), block(256);
    if (a.gate)
        hipLaunchKernelGGL((la_norm_gate_kernel<E, LPR, NV, U, true>), grid, block, 0, stream, a, hr_log,
                           (int)h_blocks, (int)t_blocks);
    else
        hipLaunchKernelGGL((la_norm_gate_kernel<E, LPR, NV, U, false>), grid, block, 0, stream, a, hr_log,
                           (int)h_blocks, (int)t_blocks);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}

// Two rows for each group of lanes where that still gives every compute unit four workgroups (B=16,
// T=1024, H=32, D=128, bf16, against one and four: 55.7 us, 59.8, 58.4).
template <typename E, int LPR>
static rgdr_status launch_norm_lanes(const NormArgs &a, hipStream_t stream) {
    if (a.T >= 2 && (__int128)a.B * a.T * a.H >= 2 * 1024 * (256 / LPR)) return launch_norm_rows<E, LPR, 1, 2>(a, stream);
    return launch_norm_rows<E, LPR, 1, 1>(a, stream);
}

// The fewest lanes that hold a row in one piece each; of long rows a wave holds several.
template <typename E>
static rgdr_status launch_norm(const NormArgs &a, hipStream_t stream) {
    const int pieces = a.D / RowVec<E>::N;
    if (pieces <= 8) return launch_norm_lanes<E, 8>(a, stream);
    if (pieces <= 16) return launch_norm_lanes<E, 16>(a, stream);
    if (pieces <= 32) return launch_norm_lanes<E, 32>(a, stream);
    if (pieces <= 64) return launch_norm_lanes<E, 64>(a, stream);
    if (pieces <= 128) return launch_norm_rows<E, 64, 2, 1>(a, stream);
    if (pieces <= 256) return launch_norm_rows<E, 64, 4, 1>(a, stream);
    if (pieces <= 512) return launch_norm_rows<E, 64, 8, 1>(a, stream);
    if constexpr (sizeof(E) == 4)
        if (pieces > 1024) return launch_norm_rows<E, 64, 32, 1>(a, stream);
    return launch_norm_rows<E, 64, 16, 1>(a, stream);
}

}  // namespace rgdr

extern "C" rgdr_status la_norm_gate(const void *x, const la_strides *x_strides, const void *gate,
                                    const la_strides *gate_strides, const float *weight,
                                    int64_t weight_h_stride, rgdr_dtype dtype,
                                    const int32_t *actual_seq_lengths, float eps, uint32_t flags,
                                    int32_t B, int32_t H, int32_t T, int32_t D, void *out,
                                    const la_strides *out_strides, hipStream_t stream) {
    using namespace rgdr;
    if (B < 0 || H < 0 || T < 0 || D < 0 || !(eps >= 0.f)) return RGDR_ERR_SHAPE;
    if (D % 8 != 0 || D > 8192 || (flags & ~(uint32_t)LA_GATE_SIGMOID)) return RGDR_ERR_UNSUPPORTED;
    if (dtype != RGDR_F32 && dtype != RGDR_F16 && dtype != RGDR_BF16) return RGDR_ERR_DTYPE;
    if (B == 0 || H == 0 || T == 0 || D == 0) return RGDR_OK;
    if (!x || !weight || !out) return RGDR_ERR_NULL;
    NormArgs a;
    a.sx = la_strides_or(x_strides, (long long)H * T * D, (long long)T * D, D);
    a.sg = la_strides_or(gate_strides, (long long)T * H * D, D, (long long)H * D);
    a.so = la_strides_or(out_strides, (long long)T * H * D, D, (long long)H * D);
    if (!la_strides_ok(a.sx) || !la_strides_ok(a.sg) || !la_strides_ok(a.so) ||
        weight_h_stride < 0 || weight_h_stride > ((int64_t)1 << 31) ||
        !la_extent_ok(a.sx, B, H, T, D) || !la_extent_ok(a.sg, B, H, T, D) ||
        !la_rows_distinct(a.so, B, H, T, D))
        return RGDR_ERR_SHAPE;
    if (!la_strides_aligned(a.sx, B, H, T) || (gate && !la_strides_aligned(a.sg, B, H, T)) ||
        !la_strides_aligned(a.so, B, H, T) || (H > 1 && weight_h_stride % 4 != 0))
        return RGDR_ERR_ALIGN;
    if (!aligned(x, 16) || (gate && !aligned(gate, 16)) || !aligned(out, 16) ||
        !aligned(weight, 16) || (actual_seq_lengths && !aligned(actual_seq_lengths, 4)))
        return RGDR_ERR_ALIGN;
    a.x = x;
    a.gate = gate;
    a.weight = weight;
    a.out = out;
    a.lens = actual_seq_lengths;
    a.sw = H > 1 ? weight_h_stride : 0;
    a.eps = eps;
    a.B = B;
    a.H = H;
    a.T = T;
    a.D = D;
    a.sigmoid = (flags & LA_GATE_SIGMOID) != 0;
    if (dtype == RGDR_F32) return launch_norm<float>(a, stream);
    if (dtype == RGDR_F16) return launch_norm<_Float16>(a, stream);
    return launch_norm<uint16_t>(a, stream);
}
