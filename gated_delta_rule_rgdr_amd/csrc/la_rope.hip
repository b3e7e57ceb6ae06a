// la_rope.hip -- rotary positions of queries and keys: pair i of a row's first R columns is turned by
// position * inv_freq[i], the other columns are copied.
#include "la_common.h"

namespace rgdr {

struct RopeArgs {
    const void *q, *k;
    const float *freq;
    const int32_t *pos, *lens;  // may be null
    void *q_out, *k_out;
    LaStrides sq, sk, sqo, sko;
    float factor;
    int B, Hq, H, T, D, R;  // H: query and key heads
    int each;               // a position for each token
};

// Cosine and sine of pos * freq, times the factor. The angle in turns is a 64-bit product, of which
// the whole turns are dropped before it becomes 32 bits: what is left is off by 2^-26 of a turn
// at any position.
__device__ __forceinline__ float2 rope_turn(double pos, float freq, float factor) {
    const double turns = pos * ((double)freq * 0.15915494309189533577);
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    return float2{c * factor, s * factor};
}

enum RopeLayout { kRopeHalves, kRopePairs, kRopeAny };

// A workgroup has 2^tb_log tokens of one entry, and hb of the H heads. It computes the tokens'
// cosines and sines once, into LDS, for all heads. A row is split into units over 2^ul_log threads:
//   kRopeHalves: 16 bytes of the first half with their partners in the second (R / 2 whole pieces
//                of 16 bytes), and 16 bytes of the columns past R;
//   kRopePairs:  interleaved pairs, 16 bytes;
//   kRopeAny:    halves of any length: one pair, or one column past R.
// A thread writes the columns that it reads and no other thread reads, so it can be done in place.
template <typename E, int LAYOUT>
__global__ __launch_bounds__(256) void la_rope_kernel(const RopeArgs a, int tb_log, int hb, int ul_log, int units,
                                                      int h_blocks, int t_blocks) {
    using V = RowVec<E>;
    constexpr int N = V::N;
    extern __shared__ float2 turn[];  // [2^tb_log][R / 2]
    const int hblk = blockIdx.x % h_blocks, tblk = blockIdx.x / h_blocks % t_blocks;
    const int b = blockIdx.x / h_blocks / t_blocks;
    const int half = a.R / 2, tb = 1 << tb_log, t0 = tblk << tb_log;
    const int L = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    for (int i = threadIdx.x; i < tb * half; i += 256) {
        const int u = i / half, t = t0 + u;
        if (t >= L) break;
        const double pos = !a.pos ? (double)t : a.each ? (double)a.pos[(size_t)b * a.T + t] : (double)a.pos[b] + t;
        turn[i] = rope_turn(pos, a.freq[i - u * half], a.factor);
    }
    __syncthreads();
    const int unit0 = threadIdx.x & ((1 << ul_log) - 1), rows = 256 >> ul_log;
    const int h0 = hblk * hb, nh = min(hb, a.H - h0);
    for (int r = threadIdx.x >> ul_log; r < nh << tb_log; r += rows) {
        const int u = r & (tb - 1), t = t0 + u, h = h0 + (r >> tb_log);
        if (t >= a.T) continue;
        const bool key = h >= a.Hq;
        const LaStrides &si = key ? a.sk : a.sq, &so = key ? a.sko : a.sqo;
        const int hh = key ? h - a.Hq : h;
        const E *x = static_cast<const E *>(key ? a.k : a.q) + b * si.b + hh * si.h + t * si.t;
        E *out = static_cast<E *>(key ? a.k_out : a.q_out) + b * so.b + hh * so.h + t * so.t;
        const float2 *cs = turn + u * half;
        const bool live = t < L;
        for (int unit = unit0; unit < units; unit += 1 << ul_log) {
            if constexpr (LAYOUT == kRopeAny) {
                if (unit < half) {
                    float p = 0.f, q = 0.f;
                    if (live) {
                        const float y = row_value(x[unit]), z = row_value(x[unit + half]);
                        p = y * cs[unit].x - z * cs[unit].y;
                        q = y * cs[unit].y + z * cs[unit].x;
                    }
                    out[unit] = row_store<E>(p);
                    out[unit + half] = row_store<E>(q);
                } else {
                    out[unit + half] = live ? x[unit + half] : E(0);
                }
            } else if constexpr (LAYOUT == kRopePairs) {
                u32x4 w = {0, 0, 0, 0};
                if (live) {
                    w = *reinterpret_cast<const u32x4 *>(x + unit * N);
                    float y[N];
                    V::get(y, w);
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        const int pair = unit * (N / 2) + i;
                        if (pair < half) {
                            const float2 c = cs[pair];
                            const float p = y[2 * i], q = y[2 * i + 1];
                            y[2 * i] = p * c.x - q * c.y;
                            y[2 * i + 1] = p * c.y + q * c.x;
                        }
                    }
                    w = V::put(y);
                }
                *reinterpret_cast<u32x4 *>(out + unit * N) = w;
            } else {
                const bool pair = unit * N < half;
                const int c0 = pair ? unit * N : unit * N + half;
                u32x4 w = {0, 0, 0, 0}, w2 = {0, 0, 0, 0};
                if (live) {
                    w = *reinterpret_cast<const u32x4 *>(x + c0);
                    if (pair) {
                        w2 = *reinterpret_cast<const u32x4 *>(x + c0 + half);
                        float y[N], z[N];
                        V::get(y, w);
                        V::get(z, w2);
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            const float2 c = cs[c0 + i];
                            const float p = y[i], q = z[i];
                            y[i] = p * c.x - q * c.y;
                            z[i] = p * c.y + q * c.x;
                        }
                        w = V::put(y);
                        w2 = V::put(z);
                    }
                }
                *reinterpret_cast<u32x4 *>(out + c0) = w;
                if (pair) *reinterpret_cast<u32x4 *>(out + c0 + half) = w2;
            }
        }
    }
}

template <typename E, int LAYOUT>
static rgdr_status launch_rope(const RopeArgs &a, hipStream_t stream) {
    const int units = LAYOUT == kRopeAny ? a.D - a.R / 2
                      : LAYOUT == kRopePairs ? a.D / RowVec<E>::N
                                             : (a.D - a.R / 2) / RowVec<E>::N;
    int ul_log = 0;
    while (ul_log < 8 && (1 << ul_log) < units) ++ul_log;
    int tb_log = 0;
    while (tb_log < 2 && (1 << tb_log) < a.T) ++tb_log;
    const long long t_blocks = (a.T + (1 << tb_log) - 1) >> tb_log;
    const int hb = a.H < 64 ? a.H : 64;
    const long long h_blocks = (a.H + hb - 1) / hb;
    if ((__int128)h_blocks * t_blocks * a.B > kMaxGroups) return RGDR_ERR_SHAPE;
    const dim3 grid((unsigned)(h_blocks * t_blocks * a.B)), block(256);
    const size_t lds = sizeof(float2) * (a.R / 2) << tb_log;
    hipLaunchKernelGGL((la_rope_kernel<E, LAYOUT>), grid, block, lds, stream, a, tb_log, hb, ul_log, units,
                       (int)h_blocks, (int)t_blocks);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}

template <typename E>
static rgdr_status launch_rope_layout(const RopeArgs &a, bool interleaved, hipStream_t stream) {
    if (interleaved) return launch_rope<E, kRopePairs>(a, stream);
    if (a.R / 2 % RowVec<E>::N == 0) return launch_rope<E, kRopeHalves>(a, stream);
    return launch_rope<E, kRopeAny>(a, stream);
}

static bool rope_in_place(const LaStrides &s, const LaStrides &o, int B, int H, int T) {
    return (B == 1 || s.b == o.b) && (H == 1 || s.h == o.h) && (T == 1 || s.t == o.t);
}

}  // namespace rgdr

extern "C" rgdr_status la_rope(const void *query, const la_strides *query_strides, const void *key,
                               const la_strides *key_strides, const float *inv_freq,
                               const int32_t *positions, rgdr_dtype dtype,
                               const int32_t *actual_seq_lengths, float factor, uint32_t flags, int32_t B,
                               int32_t H_q, int32_t H_k, int32_t T, int32_t D, int32_t R, void *query_out,
                               const la_strides *query_out_strides, void *key_out,
                               const la_strides *key_out_strides, hipStream_t stream) {
    using namespace rgdr;
    if (B < 0 || H_q < 0 || H_k < 0 || T < 0 || D < 0 || R < 0 || H_q > INT32_MAX - H_k) return RGDR_ERR_SHAPE;
    if (D % 8 != 0 || D > 1024 || R % 2 != 0 || R > D || (flags & ~(uint32_t)(LA_ROPE_INTERLEAVED | LA_ROPE_EACH_POSITION)))
        return RGDR_ERR_UNSUPPORTED;
    if (dtype != RGDR_F32 && dtype != RGDR_F16 && dtype != RGDR_BF16) return RGDR_ERR_DTYPE;
    if (B == 0 || H_q + H_k == 0 || T == 0 || D == 0) return RGDR_OK;
    if ((H_q && (!query || !query_out)) || (H_k && (!key || !key_out)) || (R && !inv_freq)) return RGDR_ERR_NULL;
    RopeArgs a;
    const int heads[2] = {H_q, H_k};
    const la_strides *in[2] = {query_strides, key_strides}, *to[2] = {query_out_strides, key_out_strides};
    const void *from[2] = {query, key};
    void *out[2] = {query_out, key_out};
    LaStrides *sin[2] = {&a.sq, &a.sk}, *sout[2] = {&a.sqo, &a.sko};
    for (int i = 0; i < 2; ++i) {
        const int H = heads[i];
        *sin[i] = la_strides_or(in[i], (long long)H * T * D, (long long)T * D, D);
        *sout[i] = la_strides_or(to[i], (long long)H * T * D, (long long)T * D, D);
        if (H == 0) continue;
        if (!la_strides_ok(*sin[i]) || !la_strides_ok(*sout[i]) || !la_extent_ok(*sin[i], B, H, T, D) ||
            !la_rows_distinct(*sout[i], B, H, T, D) ||
            (out[i] == from[i] && !rope_in_place(*sin[i], *sout[i], B, H, T)))
            return RGDR_ERR_SHAPE;
        if (!la_strides_aligned(*sin[i], B, H, T) || !la_strides_aligned(*sout[i], B, H, T) ||
            !aligned(from[i], 16) || !aligned(out[i], 16))
            return RGDR_ERR_ALIGN;
    }
    if (!aligned(inv_freq, 4) || !la_index_aligned(positions, actual_seq_lengths, nullptr)) return RGDR_ERR_ALIGN;
    a.q = query;
    a.k = key;
    a.freq = inv_freq;
    a.pos = positions;
    a.lens = actual_seq_lengths;
    a.q_out = query_out;
    a.k_out = key_out;
    a.factor = factor;
    a.B = B;
    a.Hq = H_q;
    a.H = H_q + H_k;
    a.T = T;
    a.D = D;
    a.R = R;
    a.each = (flags & LA_ROPE_EACH_POSITION) != 0;
    const bool interleaved = (flags & LA_ROPE_INTERLEAVED) != 0;
    if (dtype == RGDR_F32) return launch_rope_layout<float>(a, interleaved, stream);
    if (dtype == RGDR_F16) return launch_rope_layout<_Float16>(a, interleaved, stream);
    return launch_rope_layout<uint16_t>(a, interleaved, stream);
}
