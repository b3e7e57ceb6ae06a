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

template <typename E>
__device__ __forceinline__ float norm_load(const void *p, long long e) {
    if constexpr (sizeof(E) == 2 && !__is_same(E, _Float16))
        return bf16_to_f32(static_cast<const uint16_t *>(p)[e]);
    else
        return static_cast<float>(static_cast<const E *>(p)[e]);
}
template <typename E>
__device__ __forceinline__ void norm_store(void *p, long long e, float x) {
    if constexpr (sizeof(E) == 2 && !__is_same(E, _Float16))
        static_cast<uint16_t *>(p)[e] = f32_to_bf16(x);
    else
        static_cast<E *>(p)[e] = static_cast<E>(x);
}

// One wave for each row.
template <typename E>
__global__ __launch_bounds__(256) void la_norm_gate_kernel(const NormArgs a) {
    const long long rows = (long long)a.B * a.T * a.H;
    const long long stride = (long long)gridDim.x * 4;
    const int lane = threadIdx.x & 63;
    for (long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); r < rows; r += stride) {
        const int h = (int)(r % a.H);
        const long long bt = r / a.H;
        const int t = (int)(bt % a.T), b = (int)(bt / a.T);
        const long long eo = b * a.so.b + h * a.so.h + t * a.so.t;
        if (a.lens && t >= a.lens[b]) {
            for (int d = lane; d < a.D; d += 64) norm_store<E>(a.out, eo + d, 0.f);
            continue;
        }
        const long long ex = b * a.sx.b + h * a.sx.h + t * a.sx.t;
        const long long eg = b * a.sg.b + h * a.sg.h + t * a.sg.t;
        float ss = 0.f;
        for (int d = lane; d < a.D; d += 64) {
            const float x = norm_load<E>(a.x, ex + d);
            ss += x * x;
        }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) ss += __shfl_xor(ss, m);
        const float r_rms = 1.0f / sqrtf(ss / (float)a.D + a.eps);
        for (int d = lane; d < a.D; d += 64) {
            float y = norm_load<E>(a.x, ex + d) * r_rms * a.weight[h * a.sw + d];
            if (a.gate) {
                const float z = norm_load<E>(a.gate, eg + d);
                y *= a.sigmoid ? sigmoid_f32(z) : z * sigmoid_f32(z);
            }
            norm_store<E>(a.out, eo + d, y);
        }
    }
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
    const __int128 rows = (__int128)B * T * H, want = (rows + 3) / 4;
    const dim3 grid((unsigned)(want < 65536 ? want : 65536)), block(256);
    if (dtype == RGDR_F32)
        hipLaunchKernelGGL(la_norm_gate_kernel<float>, grid, block, 0, stream, a);
    else if (dtype == RGDR_F16)
        hipLaunchKernelGGL(la_norm_gate_kernel<_Float16>, grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL(la_norm_gate_kernel<uint16_t>, grid, block, 0, stream, a);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}
