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

// 16 bytes of a row as fp32 values, and back.
template <typename E>
struct NormVec {
    static constexpr int N = 16 / sizeof(E);
    static __device__ __forceinline__ void get(float (&x)[N], const u32x4 &w) {
#pragma unroll
        for (int c = 0; c < N; ++c) {
            if constexpr (sizeof(E) == 4)
                x[c] = __uint_as_float(w[c]);
            else if constexpr (__is_same(E, _Float16))
                x[c] = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w[c / 2] >> (c % 2 * 16))));
            else
                x[c] = c & 1 ? bf16_hi(w[c / 2]) : bf16_lo(w[c / 2]);
        }
    }
    static __device__ __forceinline__ u32x4 put(const float (&x)[N]) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(E) == 4)
                w[i] = __float_as_uint(x[i]);
            else if constexpr (__is_same(E, _Float16))
                w[i] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(x[2 * i])) |
                       (uint32_t)__builtin_bit_cast(uint16_t, static_cast<_Float16>(x[2 * i + 1])) << 16;
            else
                w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
        }
        return w;
    }
};

// LPR lanes for each row, NV pieces of 16 bytes in each lane: the row stays in registers between the
// sum and the product, so x and the gate are read once. Rows are taken in out's order (heads
// fastest). Bound: the bytes.
template <typename E, int LPR, int NV>
__global__ __launch_bounds__(256) void la_norm_gate_kernel(const NormArgs a) {
    using V = NormVec<E>;
    constexpr int ROWS = 256 / LPR;
    const long long r0 = (long long)blockIdx.x * ROWS, bt0 = r0 / a.H;
    const uint32_t hh = (uint32_t)(r0 - bt0 * a.H) + threadIdx.x / LPR, dt = hh / (uint32_t)a.H;
    const int h = (int)(hh - dt * a.H);
    const int b0 = (int)(bt0 / a.T);
    const uint32_t tt = (uint32_t)(bt0 - (long long)b0 * a.T) + dt, db = tt / (uint32_t)a.T;
    const int t = (int)(tt - db * a.T), b = b0 + (int)db;
    if (b >= a.B) return;
    const int c0 = threadIdx.x % LPR * V::N;
    E *out = static_cast<E *>(a.out) + b * a.so.b + h * a.so.h + t * a.so.t;
    if (a.lens && t >= a.lens[b]) {
#pragma unroll
        for (int m = 0; m < NV; ++m)
            if (c0 + m * LPR * V::N < a.D)
                *reinterpret_cast<u32x4 *>(out + c0 + m * LPR * V::N) = u32x4{0, 0, 0, 0};
        return;
    }
    const E *x = static_cast<const E *>(a.x) + b * a.sx.b + h * a.sx.h + t * a.sx.t;
    const E *z = static_cast<const E *>(a.gate) + b * a.sg.b + h * a.sg.h + t * a.sg.t;
    const float *w = a.weight + h * a.sw;
    u32x4 wx[NV], wz[NV];
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int c = c0 + m * LPR * V::N;
        wx[m] = wz[m] = u32x4{0, 0, 0, 0};
        if (c < a.D) {
            wx[m] = *reinterpret_cast<const u32x4 *>(x + c);
            if (a.gate) wz[m] = *reinterpret_cast<const u32x4 *>(z + c);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        float v[V::N];
        V::get(v, wx[m]);
#pragma unroll
        for (int c = 0; c < V::N; ++c) ss = __builtin_fmaf(v[c], v[c], ss);
    }
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor(ss, m);
    const float r = __builtin_amdgcn_rsqf(ss / (float)a.D + a.eps);
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int c = c0 + m * LPR * V::N;
        if (c >= a.D) continue;
        float v[V::N], g[V::N];
        V::get(v, wx[m]);
        V::get(g, wz[m]);
#pragma unroll
        for (int i = 0; i < V::N; ++i) {
            v[i] *= r * w[c + i];
            if (a.gate) v[i] *= a.sigmoid ? sigmoid_fast(g[i]) : g[i] * sigmoid_fast(g[i]);
        }
        *reinterpret_cast<u32x4 *>(out + c) = V::put(v);
    }
}

template <typename E, int LPR, int NV>
static void launch_norm_lanes(const NormArgs &a, unsigned grid, hipStream_t stream) {
    hipLaunchKernelGGL((la_norm_gate_kernel<E, LPR, NV>), dim3(grid), dim3(256), 0, stream, a);
}

// The fewest lanes that hold a row in one piece each; of long rows a wave holds several.
template <typename E>
static rgdr_status launch_norm(const NormArgs &a, hipStream_t stream) {
    const int pieces = a.D / NormVec<E>::N;
    const int lanes = pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : 64;
    const __int128 rows = (__int128)a.B * a.T * a.H, want = (rows + 256 / lanes - 1) / (256 / lanes);
    if (want > 0x7FFFFFFF) return RGDR_ERR_SHAPE;  // the grid is counted in an int
    const unsigned grid = (unsigned)want;
    if (pieces <= 8)
        launch_norm_lanes<E, 8, 1>(a, grid, stream);
    else if (pieces <= 16)
        launch_norm_lanes<E, 16, 1>(a, grid, stream);
    else if (pieces <= 32)
        launch_norm_lanes<E, 32, 1>(a, grid, stream);
    else if (pieces <= 64)
        launch_norm_lanes<E, 64, 1>(a, grid, stream);
    else if (pieces <= 128)
        launch_norm_lanes<E, 64, 2>(a, grid, stream);
    else if (pieces <= 256)
        launch_norm_lanes<E, 64, 4>(a, grid, stream);
    else if (pieces <= 512)
        launch_norm_lanes<E, 64, 8>(a, grid, stream);
    else if (pieces <= 1024)
        launch_norm_lanes<E, 64, 16>(a, grid, stream);
    else
        launch_norm_lanes<E, 64, 32>(a, grid, stream);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
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
