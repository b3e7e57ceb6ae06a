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

// Cosine and sine of pos * freq, times the factor. The angle in turns is a 64-bit product, off by at most
// 3/2 2^-52 of its value (1 / 2 pi, and two products, each rounded), of which the whole turns are dropped before
// it becomes 32 bits, off by 2^-26 of a turn: 2^-26 up to some 10^7 turns, 2^-23 at position 2^31 with freq = 1.
__device__ __forceinline__ float2 rope_turn(double pos, float freq, float factor) {
    const double turns = pos * ((double)freq * 0.15915494309189533577);
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    return float2{c * factor, s * factor};
}

enum RopeLayout { kRopeHalves, kRopePairs, kRopeAny };

// The place of a thread's row and unit.
template <typename E>
struct RopeRow {
    const E *x;
    E *out;
    int u;            // its token, of the workgroup's
    bool here, live;  // there is such a row; its token is valid
};
template <typename E>
__device__ __forceinline__ RopeRow<E> rope_row(const RopeArgs &a, int b, int t0, int h0, int r, int rows, int tb_log,
                                               int L) {
    RopeRow<E> w;
    w.u = r & ((1 << tb_log) - 1);
    const int t = t0 + w.u, h = h0 + (r >> tb_log);
    w.here = r < rows && t < a.T;
    w.live = w.here && t < L;
    const bool key = h >= a.Hq;
    const LaStrides &si = key ? a.sk : a.sq, &so = key ? a.sko : a.sqo;
    const int hh = key ? h - a.Hq : h;
    w.x = static_cast<const E *>(key ? a.k : a.q) + b * si.b + hh * si.h + t * si.t;
    w.out = static_cast<E *>(key ? a.k_out : a.q_out) + b * so.b + hh * so.h + t * so.t;
    return w;
}

// A workgroup has 2^tb_log tokens of one entry, and hb of the H heads. It computes the tokens'
// cosines and sines once, into LDS, for all heads, while its first rows are on their way. A row is split
// into units, one for each of 2^ul_log threads:
//   kRopeHalves: N columns of the first half with their partners in the second, and N of the columns past
//                R; N is the most that makes pieces of up to 16 bytes and divides R / 2;
//   kRopePairs:  interleaved pairs, 16 bytes;
//   kRopeAny:    halves of an odd number of 16-bit values: one pair, or one column past R (several units for
//                each thread where there are more than 256).
// A thread writes the columns that it reads and no other thread reads, so it can be done in place.
// Bound: the bytes. B=16, T=1024 ragged, 16 + 16 heads of 128, bf16: 40.5 us (5.4
// TB/s; with stores that stay in the caches 45.5); T=8192, 32 + 8 heads, 64 of 128 interleaved, fp16: 35.7 (4.7).
template <typename E, int LAYOUT, int N>
__global__ __launch_bounds__(256) void la_rope_kernel(const RopeArgs a, int tb_log, int hb, int ul_log, int units,
                                                      int h_blocks, int t_blocks) {
    constexpr int AHEAD = 4;          // rows of a thread in flight
    extern __shared__ float2 turn[];  // [2^tb_log][R / 2]
    const int hblk = blockIdx.x % h_blocks, tblk = blockIdx.x / h_blocks % t_blocks;
    const int b = blockIdx.x / h_blocks / t_blocks;
    const int half = a.R / 2, tb = 1 << tb_log, t0 = tblk << tb_log;
    const int L = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const int unit0 = threadIdx.x & ((1 << ul_log) - 1), at_once = 256 >> ul_log;
    const int h0 = hblk * hb, rows = min(hb, a.H - h0) << tb_log;
    const auto turns = [&] {
        for (int i = threadIdx.x; i < tb * half; i += 256) {
            const int u = i / half, t = t0 + u;
            if (t >= L) break;
            const double pos = !a.pos ? (double)t : a.each ? (double)a.pos[(size_t)b * a.T + t] : (double)a.pos[b] + t;
            turn[i] = rope_turn(pos, a.freq[i - u * half], a.factor);
        }
        __syncthreads();
    };
    if constexpr (LAYOUT == kRopeAny) {
        turns();
        for (int r = threadIdx.x >> ul_log; r < rows; r += at_once) {
            const RopeRow<E> w = rope_row<E>(a, b, t0, h0, r, rows, tb_log, L);
            if (!w.here) continue;
            const float2 *cs = turn + w.u * half;
            for (int unit = unit0; unit < units; unit += 1 << ul_log) {
                if (unit < half) {
                    float p = 0.f, q = 0.f;
                    if (w.live) {
                        const float y = row_value(w.x[unit]), z = row_value(w.x[unit + half]);
                        p = y * cs[unit].x - z * cs[unit].y;
                        q = y * cs[unit].y + z * cs[unit].x;
                    }
                    w.out[unit] = row_store<E>(p);
                    w.out[unit + half] = row_store<E>(q);
                } else {
                    w.out[unit + half] = w.live ? w.x[unit + half] : E(0);
                }
            }
        }
    } else {
        const bool pair = LAYOUT == kRopePairs || unit0 * N < half;
        const int c0 = pair ? unit0 * N : unit0 * N + half;  // the unit's first column
        const bool in_row = unit0 < units;
        for (int r0 = 0; r0 < rows; r0 += AHEAD * at_once) {
            RopeRow<E> w[AHEAD];
            Row<E, N> y[AHEAD], z[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                w[k] = rope_row<E>(a, b, t0, h0, r0 + k * at_once + (threadIdx.x >> ul_log), rows, tb_log, L);
                y[k].zero();
                z[k].zero();
                if (w[k].live && in_row) {
                    y[k].load(w[k].x + c0);
                    if (LAYOUT == kRopeHalves && pair) z[k].load(w[k].x + c0 + half);
                }
            }
            if (r0 == 0) turns();
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (!w[k].here || !in_row) continue;
                if (pair && w[k].live) {
                    const float2 *cs = turn + w[k].u * half;
                    float p[N], q[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        p[i] = y[k].get(i);
                        q[i] = z[k].get(i);
                    }
                    if constexpr (LAYOUT == kRopePairs) {
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) {
                            const int n = c0 / 2 + i;
                            if (n >= half) continue;
                            const float2 c = cs[n];
                            const float u = p[2 * i], v = p[2 * i + 1];
                            p[2 * i] = u * c.x - v * c.y;
                            p[2 * i + 1] = u * c.y + v * c.x;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            const float2 c = cs[c0 + i];
                            const float u = p[i], v = q[i];
                            p[i] = u * c.x - v * c.y;
                            q[i] = u * c.y + v * c.x;
                        }
                        z[k].set(q);
                    }
                    y[k].set(p);
                }
                y[k].template store<true>(w[k].out + c0);
                if (LAYOUT == kRopeHalves && pair) z[k].template store<true>(w[k].out + c0 + half);
            }
        }
    }
}

static int rope_units(int layout, int N, int D, int R) {
    return layout == kRopeAny ? D - R / 2 : layout == kRopePairs ? D / N : (D - R / 2) / N;
}

template <typename E, int LAYOUT, int N>
static rgdr_status launch_rope(const RopeArgs &a, hipStream_t stream) {
    const int units = rope_units(LAYOUT, N, a.D, a.R);
    int ul_log = 0;
    while (ul_log < 8 && (1 << ul_log) < units) ++ul_log;
    int tb_log = 0;
    while (tb_log < 2 && (1 << tb_log) < a.T) ++tb_log;
    const long long t_blocks = ((long long)a.T + (1 << tb_log) - 1) >> tb_log;
    const long long h_blocks = ((long long)a.H + 63) / 64;
    const int hb = (int)((a.H + h_blocks - 1) / h_blocks);
    if ((__int128)h_blocks * t_blocks * a.B > kMaxGroups) return RGDR_ERR_SHAPE;
    const dim3 grid((unsigned)(h_blocks * t_blocks * a.B)), block(256);
    const size_t lds = sizeof(float2) * (a.R / 2) << tb_log;
    hipLaunchKernelGGL((la_rope_kernel<E, LAYOUT, N>), grid, block, lds, stream, a, tb_log, hb, ul_log, units,
                       (int)h_blocks, (int)t_blocks);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}

// Halves in pieces of up to 16 bytes. (R = 24 of 96 columns, bf16, 2000 tokens of 16 heads: 7.9 us in pieces
// of 8 bytes, 30 column by column.)
template <typename E>
static rgdr_status launch_rope_layout(const RopeArgs &a, bool interleaved, hipStream_t stream) {
    constexpr int MOST = 16 / sizeof(E);
    const int half = a.R / 2;
    const auto fits = [&](int N) { return half % N == 0 && rope_units(kRopeHalves, N, a.D, a.R) <= 256; };
    if (interleaved) return launch_rope<E, kRopePairs, MOST>(a, stream);
    if (fits(MOST)) return launch_rope<E, kRopeHalves, MOST>(a, stream);
    if (fits(MOST / 2)) return launch_rope<E, kRopeHalves, MOST / 2>(a, stream);
    if (fits(MOST / 4)) return launch_rope<E, kRopeHalves, MOST / 4>(a, stream);
    return launch_rope<E, kRopeAny, 1>(a, stream);
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
