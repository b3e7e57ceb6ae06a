// la_decode.hip -- linear attention with a decay for each head, a few tokens at a time.
//
// Per (entry, value head) and valid token, on S (D_k x D_v):  S = exp(g) S + k v^T,
// o = S^T (scale q). With G_t the running sum of the log decays and S0 the stored state, that is
//     o_t = S0^T (scale e^{G_t} q_t) + sum_{s <= t} scale e^{G_t - G_s} (q_t . k_s) v_s
//     S_n = e^{G_n} S0 + sum_{s < n} (e^{G_n - G_s} k_s) v_s^T
// so every state element is read once, multiplied by T query rows and T key rows, and written once,
// with nothing carried from token to token. Bound: the state's bytes (2 T + 1 multiply-adds for
// each of its elements, 2 to 8 bytes).
#include "la_mfma.h"

namespace rgdr {

// How one lane holds a piece of a state row: 16 bytes of it.
template <int ST>
struct Piece {
    static constexpr int N = ST == RGDR_F32 ? 4 : ST == RGDR_BF16 ? 8 : 16;  // columns
    // Value c; of an 8-bit state its code.
    static __device__ __forceinline__ float get(const u32x4 &w, int c) {
        if constexpr (ST == RGDR_F32)
            return __uint_as_float(w[c]);
        else if constexpr (ST == RGDR_BF16)
            return c & 1 ? bf16_hi(w[c / 2]) : bf16_lo(w[c / 2]);
        else
            return mx_code(w[c / 4], c % 4);
    }
};

// Rounds a lane's piece of a row. Two neighbouring lanes hold an 8-bit block; every lane of the
// wave calls this.
template <int ST>
__device__ __forceinline__ u32x4 round_piece(const float (&x)[Piece<ST>::N], uint32_t &eb) {
    u32x4 w;
    if constexpr (ST == RGDR_F32) {
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = __float_as_uint(x[c]);
    } else if constexpr (ST == RGDR_BF16) {
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = pack_bf16x2(x[2 * c], x[2 * c + 1]);
    } else {
        float most = 0.f;
#pragma unroll
        for (int c = 0; c < 16; ++c) most = mx_larger(most, x[c]);
        uint32_t top = mx_top_bits(most);  // as whole numbers NaN is the largest
        top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, false));  // lane ^ 1
        eb = mx_exponent(top);
        const float inv = mx_inverse(eb);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            w[c] = mx_pack4(mx_code_bits(x[4 * c], inv), mx_code_bits(x[4 * c + 1], inv),
                            mx_code_bits(x[4 * c + 2], inv), mx_code_bits(x[4 * c + 3], inv));
    }
    return w;
}

template <int ST, int DK, int TV>
struct StepShape {
    static constexpr int CPL = Piece<ST>::N;                       // columns of a lane
    static constexpr int LPR = TV / CPL;                           // lanes across a row of the tile
    static constexpr int NT = DK * LPR < 256 ? DK * LPR : 256;     // threads
    static constexpr int RPP = NT / LPR;                           // rows in one pass of them
    static constexpr int R = DK / RPP;                             // rows of a thread
    static constexpr int NW = NT / 64;
    static_assert(NT % 64 == 0 && NT >= DK && 64 % LPR == 0 && DK % RPP == 0, "tile shape");
};

// Sum over the lanes of the wave that hold the same columns, LPR apart; every lane gets it. Rotations
// within rows of 16 lanes, then exchanges between rows: register moves, no LDS.
template <int CTRL>
__device__ __forceinline__ float add_rotated(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
}
template <int LPR>
__device__ __forceinline__ float row_lanes_sum(float x) {
    static_assert(LPR >= 2 && LPR <= 32, "lanes across a row");
    if constexpr (LPR <= 8) x = add_rotated<0x128>(x);
    if constexpr (LPR <= 4) x = add_rotated<0x124>(x);
    if constexpr (LPR <= 2) x = add_rotated<0x122>(x);
    if constexpr (LPR <= 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// N bf16 values of a row, in fp32; p is aligned to their 2 N bytes or to 16.
template <int N>
__device__ __forceinline__ void load_bf16(float (&x)[N], const uint16_t *p) {
    if constexpr (N == 4) {
        const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            x[2 * e] = bf16_lo(v[e]);
            x[2 * e + 1] = bf16_hi(v[e]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N / 8; ++j) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(p + j * 8);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[j * 8 + 2 * e] = bf16_lo(v[e]);
                x[j * 8 + 2 * e + 1] = bf16_hi(v[e]);
            }
        }
    }
}

// One token: one workgroup for each (entry, value head, TV columns). A lane holds 16 bytes of each
// of its rows, so the state moves in whole lines. The operands' loads go out before the state's,
// whose answers are waited for last. Bound: the state's bytes, in and out. H_v = 32, D = 128: bf16
// B=1 3.4 us (launch and latency), B=256 96.9 us (5.6 TB/s; a large copy reaches 5.3); fp32 B=128
// 95.2 us (5.7); 8 bits B=128 28.9 us (4.9), where widening, the block maximum and packing take
// about 7 vector instructions an element. Held to more waves with fewer registers, the loads go out in
// smaller sets: bf16 B=256 107 us at 6 waves for each SIMD, 151 at 8.
template <int ST, int DK, int TV>
__global__ __launch_bounds__(256) void la_step_kernel(const LaArgs a, int tiles) {
    using Sh = StepShape<ST, DK, TV>;
    constexpr int CPL = Sh::CPL, LPR = Sh::LPR, R = Sh::R, NT = Sh::NT, NW = Sh::NW;
    __shared__ f32x2_t qk[DK];
    __shared__ float red[NW][TV];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int item = xcd_item(blockIdx.x, gridDim.x);
    const int tile = item % tiles;
    item /= tiles;
    const int h = item % a.Hv, b = item / a.Hv, hq = h / a.group;
    const LaEntry en = la_entry(a, b);
    uint16_t *go = a.out + b * a.so.b + h * a.so.h + tile * TV;
    if (!en.state || (en.L == 0 && a.in_place)) {  // nothing to read, nothing new to write
        for (int c = tid; c < TV; c += NT) go[c] = 0;
        return;
    }

    // this thread's columns, and its first row
    const int c0 = tid % LPR * CPL, r0 = tid / LPR;
    const long long first = (((long long)en.slot * a.Hv + h) * DK + r0) * a.Dv + tile * TV + c0;
    constexpr int kSize = 16 / CPL;
    const long long row_bytes = (long long)Sh::RPP * a.Dv * kSize;
    const char *in = static_cast<const char *>(a.pool) + first * kSize;
    const uint8_t *sin = ST == RGDR_MXI8 ? a.scales + first / kMxBlock : nullptr;
    const int srow = Sh::RPP * (a.Dv / kMxBlock);

    float q0 = 0.f, k0 = 0.f, g0 = 0.f, vt[CPL] = {};
    if (en.L) {
        if (tid < DK) {
            q0 = bf16_to_f32(a.q[b * a.sq.b + hq * a.sq.h + tid]) * a.scale;
            k0 = bf16_to_f32(a.k[b * a.sk.b + hq * a.sk.h + tid]);
        }
        load_bf16<CPL>(vt, a.v + b * a.sv.b + h * a.sv.h + tile * TV + c0);
        g0 = a.g[b * a.sg.b + h * a.sg.h];
    }
    u32x4 w[R];
    uint32_t eb[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        w[r] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(in + r * row_bytes));
        if constexpr (ST == RGDR_MXI8) eb[r] = sin[r * srow];
    }
    if (tid < DK) qk[tid] = f32x2_t{q0, k0};
    const float keep = en.L ? expf(la_log_decay(g0)) : 1.f;
    __syncthreads();

    char *const o_state = static_cast<char *>(a.pool_out) + first * kSize;
    uint8_t *const o_scale = ST == RGDR_MXI8 ? a.scales_out + first / kMxBlock : nullptr;
    float acc[CPL] = {};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const f32x2_t op = qk[r0 + r * Sh::RPP];
        const float sc = ST == RGDR_MXI8 ? mx_scale(eb[r]) * keep : keep;  // a power of two: exact
        float x[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            x[c] = __builtin_fmaf(op[1], vt[c], sc * Piece<ST>::get(w[r], c));
            acc[c] = __builtin_fmaf(op[0], x[c], acc[c]);
        }
        if (en.n) w[r] = round_piece<ST>(x, eb[r]);  // else the token is rejected: the bytes as they were
        __builtin_nontemporal_store(w[r], reinterpret_cast<u32x4 *>(o_state + r * row_bytes));
        if constexpr (ST == RGDR_MXI8)
            if ((lane & 1) == 0) o_scale[r * srow] = (uint8_t)eb[r];
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        const float x = row_lanes_sum<LPR>(acc[c]);
        if (lane < LPR) red[wave][c0 + c] = x;
    }
    __syncthreads();
    for (int c = tid; c < TV; c += NT) {
        float x = 0.f;
#pragma unroll
        for (int m = 0; m < NW; ++m) x += red[m][c];
        go[c] = en.L ? f32_to_bf16(x) : 0;  // of no token: 0, also where the state is not finite
    }
}

// Neither of the two is NaN or an infinity.
__device__ __forceinline__ bool finite_bf16x2(uint32_t w) {
    return (w & 0x7F80u) != 0x7F80u && (w & 0x7F800000u) != 0x7F800000u;
}

// 2 to 8 tokens, on the matrix cores: one workgroup for each (entry, value head, 128 columns), CB
// blocks of 32 columns for each wave. A wave moves 32 rows at a time, in whole lines (16 bytes for
// each lane, up to 128 for each row), through LDS into the layout of the products' results,
// transposed (lanes: rows i, registers: columns j), and back; as bf16 they become an operand of
// S^T q on the way. What fp32 holds (fp32 states, scores, weighted values) enters the products as the
// sum of three bf16 numbers, 24 bits; two for the states and scores were no faster. The tokens are a
// quarter of the products' 32 columns; the products are far from bounding the call all the same (31 to
// 47 of them, under 0.7 us, for 4096 elements, whose bytes take a compute unit 0.4 to 1.6 us). H_v = 32,
// D = 128, B = 32, T = 8: fp32 30 us (4.7 TB/s), bf16 16.5 to 18 us (4.1 to 4.4), 8 bits 16 us (2.5: two trips
// of each value through LDS, and vector work as above). Read and written straight in the products'
// layout, 32 rows apart from lane to lane, the same took 46, 29 and 28 us; on the vector units
// alone 60, 82 and 52.
template <int ST, int DK, int CB>
__global__ __launch_bounds__(256 / CB) void la_tokens_kernel(const LaArgs a, int tiles) {
    constexpr int KP = DK / 8;                          // 16-byte pieces of a q or k row
    constexpr int NI = DK / 32;                         // tiles of 32 rows
    constexpr int NT = 256 / CB, NW = 4 / CB;
    constexpr int PL = ST == RGDR_F32 ? 3 : 1;          // bf16 and 8-bit states are whole bf16 numbers
    constexpr int kSize = ST == RGDR_F32 ? 4 : ST == RGDR_BF16 ? 2 : 1;
    constexpr int WP = 2 * kSize;                       // words of 8 columns
    constexpr int PC = CB * 2 * kSize;                  // 16-byte pieces of the wave's part of a row
    constexpr int NM = 32 * PC / 64;                    // of a tile, in each lane's hands
    static_assert(PC <= 8 && NM >= 1, "a wave moves up to 128 bytes of a row");
    __shared__ __align__(256) char lq[kMaxT * lds_row_bytes<KP>()], lk[kMaxT * lds_row_bytes<KP>()];
    __shared__ __align__(256) char lv[kMaxT * lds_row_bytes<16>()];
    __shared__ __align__(256) char ls[NW][PL][32 * 64], lw[NW][32 * lds_row_bytes<PC>()];

    const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, hf = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int item = xcd_item(blockIdx.x, gridDim.x);
    const int tile = item % tiles;
    item /= tiles;
    const int h = item % a.Hv, b = item / a.Hv, hq = h / a.group;
    const LaEntry en = la_entry(a, b);
    const int L = en.L, n = en.n;
    const int col0 = tile * 128 + wave * CB * 32;  // the wave's first column
    const bool mine = col0 < a.Dv;                 // CB divides D_v / 32
    const int vpieces = min(16, (a.Dv - tile * 128) / 8);
    uint16_t *const go = a.out + b * a.so.b + h * a.so.h + tile * 128;
    for (int j = tid; j < (a.T - L) * vpieces; j += NT)
        *reinterpret_cast<u32x4 *>(go + (L + j / vpieces) * a.so.t + j % vpieces * 8) = u32x4{0, 0, 0, 0};
    if (!en.state || (L == 0 && a.in_place)) return;

    // operands: eight rows of q, k and v (the last token's again behind it: those have no weight)
    constexpr int QN = (DK + NT - 1) / NT, VN = (kMaxT * 16 + NT - 1) / NT;
    u32x4 rq[QN] = {}, rk[QN] = {}, rv[VN] = {};
    double G = 0.0;
    const int tg = lane & 7;
    if (L) {
#pragma unroll
        for (int m = 0; m < QN; ++m) {
            const int j = m * NT + tid, t = min(j / KP, L - 1), c = j % KP * 8;
            if (j < DK) {
                rq[m] = *reinterpret_cast<const u32x4 *>(a.q + b * a.sq.b + hq * a.sq.h + t * a.sq.t + c);
                rk[m] = *reinterpret_cast<const u32x4 *>(a.k + b * a.sk.b + hq * a.sk.h + t * a.sk.t + c);
            }
        }
#pragma unroll
        for (int m = 0; m < VN; ++m) {
            const int j = m * NT + tid, t = min(j / 16, L - 1), c = min(j % 16, vpieces - 1) * 8;
            if (j < kMaxT * 16)
                rv[m] = *reinterpret_cast<const u32x4 *>(a.v + b * a.sv.b + h * a.sv.h + t * a.sv.t + tile * 128 + c);
        }
        if (tg < L) G = (double)la_log_decay(a.g[b * a.sg.b + h * a.sg.h + tg * a.sg.t]);
    }
    // the state: lane by lane along its rows' pieces
    const long long head = ((long long)en.slot * a.Hv + h) * DK * a.Dv + col0;
    const int row_l = lane / PC, piece_l = lane % PC;
    const long long lane_off = (long long)row_l * a.Dv * kSize + piece_l * 16;
    const long long move = (long long)(64 / PC) * a.Dv * kSize;  // rows of one instruction
    u32x4 w[NI][NM];
    uint32_t eb[NI];  // CB scale bytes of row 32 it + map32(lane % 32)
    const long long se = (head + (long long)map32(col) * a.Dv) / kMxBlock;
    if (mine)
#pragma unroll
        for (int it = 0; it < NI; ++it) {
            const char *p = static_cast<const char *>(a.pool) + (head + (long long)it * 32 * a.Dv) * kSize + lane_off;
#pragma unroll
            for (int m = 0; m < NM; ++m)
                w[it][m] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + m * move));
            if constexpr (ST == RGDR_MXI8) {
                const uint8_t *sp = a.scales + se + (long long)it * 32 * (a.Dv / kMxBlock);
                eb[it] = CB == 1 ? *sp : *reinterpret_cast<const uint16_t *>(sp);
            }
        }
#pragma unroll
    for (int m = 0; m < QN; ++m) {
        const int j = m * NT + tid;
        if (j < DK) {
            *reinterpret_cast<u32x4 *>(lq + lds_at<KP>(j / KP, j % KP)) = rq[m];
            *reinterpret_cast<u32x4 *>(lk + lds_at<KP>(j / KP, j % KP)) = rk[m];
        }
    }
#pragma unroll
    for (int m = 0; m < VN; ++m) {
        const int j = m * NT + tid;
        if (j < kMaxT * 16) *reinterpret_cast<u32x4 *>(lv + lds_at<16>(j / 16, j % 16)) = rv[m];
    }
    // decay sums in fp64 (a token that forgets all leaves a large sum under the later ones'
    // differences), the same in every group of eight lanes
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) {
        const double y = __shfl_up(G, m);
        if (tg >= m) G += y;
    }
    const double G_n = n ? __shfl(G, n - 1) : 0.0, G_t = __shfl(G, col & 7);
    const float keep = expf((float)G_n);
    const float wk1 = tg < n ? expf((float)(G_n - G)) : 0.f;  // what S_n keeps of token tg
    const float carry = expf((float)G_t) * a.scale;
    float gap[4];  // decay from token s = 4 hf + r to token t = lane % 32
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const double d = G_t - __shfl(G, hf * 4 + r);
        gap[r] = hf * 4 + r <= col && col < L ? expf((float)d) * a.scale : 0.f;
    }
    __syncthreads();
    if (!mine) return;

    // scores: lanes t, registers s = 4 hf + 0..3; then s = 0..7 in the lower lanes
    f32x16 x = {};
#pragma unroll
    for (int c = 0; c < DK / 16; ++c)
        x = mfma(__builtin_bit_cast(u32x4, lds_read(lk + lds_at<KP>(col & 7, c * 2 + hf))),
                 lds_read(lq + lds_at<KP>(col & 7, c * 2 + hf)), x);
    float y[8];
    u32x4 p_hi, p_lo, p_lo2;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const uint32_t z = __float_as_uint(gap[r] != 0.f ? x[r] * gap[r] : 0.f);
        const auto sw = __builtin_amdgcn_permlane32_swap(z, z, false, false);
        y[r] = hf ? 0.f : __uint_as_float(sw[0]);
        y[r + 4] = hf ? 0.f : __uint_as_float(sw[1]);
    }
    split2(y, p_hi, p_lo);
    p_lo2 = split_rest(y, p_lo);
    // values: lanes j, eight tokens in each lane (the upper lanes' have no weight), and the same
    // weighted for the state
    u32x4 vf[CB], v_hi[CB], v_lo[CB], v_lo2[CB];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        vf[cb] = __builtin_bit_cast(u32x4, lds_read_tr<16>(lv, 0, wave * CB + cb, col));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float wk = __shfl(wk1, e);
            y[e] = hf || e >= n ? 0.f : (e & 1 ? bf16_hi(vf[cb][e / 2]) : bf16_lo(vf[cb][e / 2])) * wk;
        }
        split2(y, v_hi[cb], v_lo[cb]);
        v_lo2[cb] = split_rest(y, v_lo[cb]);
    }
    // A value that is not finite would meet the zero scores of the tokens before its own: it is a 0 in the
    // product, and is added behind it.
    bool odd = false;
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
        for (int e = 0; e < 4; ++e) odd |= !finite_bf16x2(vf[cb][e]);
    odd = __any(odd);
    if (odd)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                vf[cb][e] = (finite_bf16x2(vf[cb][e] & 0xFFFFu) ? vf[cb][e] & 0xFFFFu : 0u) |
                            (finite_bf16x2(vf[cb][e] & 0xFFFF0000u) ? vf[cb][e] & 0xFFFF0000u : 0u);

    f32x16 o[CB] = {};
    const bool store = n || !a.in_place;
    char *const raw = lw[wave];
#pragma unroll
    for (int it = 0; it < NI; ++it) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
            *reinterpret_cast<u32x4 *>(raw + lds_at<PC>(m * (64 / PC) + row_l, piece_l)) = w[it][m];
        wave_in_order();
        // keys of the accepted tokens: a rejected one's may be anything
        u32x4 kw = __builtin_bit_cast(u32x4, lds_read_tr<KP>(lk, 0, it, col));
#pragma unroll
        for (int e = 0; e < 4; ++e) kw[e] &= n > 2 * e + 1 ? 0xFFFFFFFFu : n > 2 * e ? 0xFFFFu : 0u;
        const bf16x8 k = __builtin_bit_cast(bf16x8, kw);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            // row map32(lane % 32) of the tile, columns 32 cb + 16 kb + 8 hf .. + 7
            float s[2][8];
            const float sc = ST == RGDR_MXI8 ? mx_scale((eb[it] >> (8 * cb)) & 255) : 1.f;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const int at = (cb * 32 + kb * 16 + hf * 8) * kSize;  // bytes into the row
                u32x4 hi, lo;
                uint32_t u[WP];
                if constexpr (ST == RGDR_MXI8) {
                    const u32x2 z = *reinterpret_cast<const u32x2 *>(raw + lds_at<PC>(map32(col), at / 16) + at % 16);
                    u[0] = z[0];
                    u[1] = z[1];
                } else {
#pragma unroll
                    for (int m = 0; m < WP / 4; ++m) {
                        const u32x4 z = *reinterpret_cast<const u32x4 *>(raw + lds_at<PC>(map32(col), at / 16 + m));
#pragma unroll
                        for (int e = 0; e < 4; ++e) u[m * 4 + e] = z[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (ST == RGDR_F32)
                        s[kb][e] = __uint_as_float(u[e]);
                    else if constexpr (ST == RGDR_BF16)
                        s[kb][e] = e & 1 ? bf16_hi(u[e / 2]) : bf16_lo(u[e / 2]);
                    else
                        s[kb][e] = mx_code(u[e / 4], e % 4) * sc;
                }
                const int pa = lds_at<4>(map32(col), kb * 2 + hf);
                if constexpr (ST == RGDR_F32) {
                    float rest[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) rest[e] = s[kb][e];
                    split2(rest, hi, lo);
                    *reinterpret_cast<u32x4 *>(ls[wave][PL - 2] + pa) = lo;
                    *reinterpret_cast<u32x4 *>(ls[wave][PL - 1] + pa) = split_rest(rest, lo);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        hi[e] = ST == RGDR_BF16 ? u[e % WP] : pack_bf16x2(s[kb][2 * e], s[kb][2 * e + 1]);
                }
                *reinterpret_cast<u32x4 *>(ls[wave][0] + pa) = hi;
            }
            wave_in_order();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const bf16x8 q = lds_read(lq + lds_at<KP>(col & 7, (it * 2 + c) * 2 + hf));
#pragma unroll
                for (int pl = PL - 1; pl >= 0; --pl)
                    o[cb] = mfma(__builtin_bit_cast(u32x4, lds_read_tr<4>(ls[wave][pl], c * 16, 0, lane)), q, o[cb]);
            }
            wave_in_order();
            if (!n) continue;
            f32x16 z;
#pragma unroll
            for (int r = 0; r < 16; ++r) z[r] = s[r / 8][r % 8] * keep;
            z = mfma(v_lo2[cb], k, z);
            z = mfma(v_lo[cb], k, z);
            z = mfma(v_hi[cb], k, z);
            float inv = 0.f;
            if constexpr (ST == RGDR_MXI8) {
                float most = 0.f;
#pragma unroll
                for (int r = 0; r < 16; ++r) most = mx_larger(most, z[r]);
                const uint32_t top = mx_top_bits(most);  // as whole numbers NaN is the largest
                const auto sw = __builtin_amdgcn_permlane32_swap(top, top, false, false);
                const uint32_t e = mx_exponent(max(sw[0], sw[1]));
                inv = mx_inverse(e);
                eb[it] = (eb[it] & ~(255u << (8 * cb))) | e << (8 * cb);
            }
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const int at = (cb * 32 + kb * 16 + hf * 8) * kSize;
                if constexpr (ST == RGDR_MXI8) {
                    u32x2 u;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        u[m] = mx_pack4(mx_code_bits(z[kb * 8 + m * 4], inv), mx_code_bits(z[kb * 8 + m * 4 + 1], inv),
                                        mx_code_bits(z[kb * 8 + m * 4 + 2], inv), mx_code_bits(z[kb * 8 + m * 4 + 3], inv));
                    *reinterpret_cast<u32x2 *>(raw + lds_at<PC>(map32(col), at / 16) + at % 16) = u;
                } else {
#pragma unroll
                    for (int m = 0; m < WP / 4; ++m) {
                        u32x4 u;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            u[e] = ST == RGDR_F32 ? __float_as_uint(z[kb * 8 + m * 4 + e])
                                                  : pack_bf16x2(z[kb * 8 + 2 * e], z[kb * 8 + 2 * e + 1]);
                        *reinterpret_cast<u32x4 *>(raw + lds_at<PC>(map32(col), at / 16 + m)) = u;
                    }
                }
            }
        }
        wave_in_order();
        if (store) {
            char *p = static_cast<char *>(a.pool_out) + (head + (long long)it * 32 * a.Dv) * kSize + lane_off;
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const u32x4 u = *reinterpret_cast<const u32x4 *>(raw + lds_at<PC>(m * (64 / PC) + row_l, piece_l));
                __builtin_nontemporal_store(u, reinterpret_cast<u32x4 *>(p + m * move));
            }
            if constexpr (ST == RGDR_MXI8)
                if (hf == 0) {
                    uint8_t *sp = a.scales_out + se + (long long)it * 32 * (a.Dv / kMxBlock);
                    if constexpr (CB == 1)
                        *sp = (uint8_t)eb[it];
                    else
                        *reinterpret_cast<uint16_t *>(sp) = (uint16_t)eb[it];
                }
        }
        wave_in_order();
    }
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
#pragma unroll
        for (int r = 0; r < 16; ++r) o[cb][r] *= carry;
        o[cb] = mfma(vf[cb], __builtin_bit_cast(bf16x8, p_lo2), o[cb]);
        o[cb] = mfma(vf[cb], __builtin_bit_cast(bf16x8, p_lo), o[cb]);
        o[cb] = mfma(vf[cb], __builtin_bit_cast(bf16x8, p_hi), o[cb]);
        if (odd)
            for (int s = 0; s < L; ++s) {
                // of token t = lane % 32; the rest of it changes no infinity
                const uint32_t hi = s < 2 ? p_hi[0] : s < 4 ? p_hi[1] : s < 6 ? p_hi[2] : p_hi[3];
                const float score = __shfl(s & 1 ? bf16_hi(hi) : bf16_lo(hi), col);
                if (s > col) continue;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(
                        lv + lds_at<16>(s, (wave * CB + cb) * 4 + m * 2 + hf));
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float x = e & 1 ? bf16_hi(v[e / 2]) : bf16_lo(v[e / 2]);
                        if (!__builtin_isfinite(x)) o[cb][m * 8 + e] += score * x;
                    }
                }
            }
        if (col < L) {
            uint16_t *row = go + col * a.so.t + (wave * CB + cb) * 32 + hf * 8;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                u32x4 z;
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = pack_bf16x2(o[cb][m * 8 + 2 * e], o[cb][m * 8 + 2 * e + 1]);
                *reinterpret_cast<u32x4 *>(row + m * 16) = z;
            }
        }
    }
}

template <int ST, int DK, int CB>
static void launch_tokens(const LaArgs &a, hipStream_t stream) {
    const int tiles = (a.Dv + 127) / 128;
    const dim3 grid((unsigned)((long long)a.B * a.Hv * tiles));
    hipLaunchKernelGGL((la_tokens_kernel<ST, DK, CB>), grid, dim3(256 / CB), 0, stream, a, tiles);
}

template <int ST, int DK, int TV>
static void launch_step_tv(const LaArgs &a, hipStream_t stream) {
    const int tiles = a.Dv / TV;
    const dim3 grid((unsigned)((long long)a.B * a.Hv * tiles)), block(StepShape<ST, DK, TV>::NT);
    hipLaunchKernelGGL((la_step_kernel<ST, DK, TV>), grid, block, 0, stream, a, tiles);
}

template <int ST, int DK>
static void launch_dk(const LaArgs &a, hipStream_t stream) {
    if (a.T > 1) {
        // Two blocks of 32 columns for each wave move 16-bit and 8-bit states in longer runs, once
        // that leaves every SIMD two waves (T = 4, H_v = 32, D = 128; two blocks against one: bf16
        // B = 16 11.8 against 10.8 us, B = 32 15.8 against 20.5; 8 bits 12.6 against 10.3 and 15.5
        // against 19.3).
        if constexpr (ST != RGDR_F32) {
            if (a.Dv % 64 == 0 && (long long)a.B * a.Hv * (a.Dv / 64) >= 2048)
                return launch_tokens<ST, DK, 2>(a, stream);
        }
        launch_tokens<ST, DK, 1>(a, stream);
    } else if (a.Dv % 128 == 0 && (long long)a.B * a.Hv * (a.Dv / 128) >= 512) {
        launch_step_tv<ST, DK, 128>(a, stream);
    } else if (a.Dv % 64 == 0) {
        launch_step_tv<ST, DK, 64>(a, stream);
    } else {
        launch_step_tv<ST, DK, 32>(a, stream);
    }
}

template <int ST>
static rgdr_status launch_decode(const LaArgs &a, int D_k, hipStream_t stream) {
    if (D_k == 64)
        launch_dk<ST, 64>(a, stream);
    else if (D_k == 128)
        launch_dk<ST, 128>(a, stream);
    else
        launch_dk<ST, 256>(a, stream);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}

rgdr_status la_check_sizes(int max_t, int32_t B, int32_t H_v, int32_t T, int32_t D_k, int32_t D_v) {
    if (B < 0 || H_v <= 0 || T <= 0 || T > max_t || D_k <= 0 || D_v <= 0) return RGDR_ERR_SHAPE;
    if (D_k != 64 && D_k != 128 && D_k != 256) return RGDR_ERR_UNSUPPORTED;
    if (D_v % 32 != 0 || D_v > 4096) return RGDR_ERR_UNSUPPORTED;
    if ((__int128)B * H_v * (D_v % 128 ? D_v / 32 : D_v / 128) > kMaxGroups) return RGDR_ERR_SHAPE;
    return RGDR_OK;
}

rgdr_status la_check(LaArgs &a, int max_t, const void *query, const la_strides *query_strides,
                     const void *key, const la_strides *key_strides, const void *value,
                     const la_strides *value_strides, const float *g, const la_strides *g_strides,
                     const void *state_pool, const uint8_t *state_scales, int state_dtype,
                     const int32_t *lens, const int32_t *idx, const int32_t *nacc, float scale,
                     int32_t B, int32_t H_q, int32_t H_v, int32_t T, int32_t D_k, int32_t D_v,
                     int32_t N_slots, void *out, const la_strides *out_strides, void *state_out,
                     uint8_t *state_scales_out) {
    if (const rgdr_status st = la_check_sizes(max_t, B, H_v, T, D_k, D_v)) return st;
    if (H_q <= 0 || H_v % H_q != 0 || N_slots <= 0) return RGDR_ERR_SHAPE;
    if (state_dtype != RGDR_F32 && state_dtype != RGDR_BF16 && state_dtype != RGDR_MXI8)
        return RGDR_ERR_DTYPE;
    if (B == 0) return RGDR_OK;
    const bool mx = state_dtype == RGDR_MXI8;
    if (!query || !key || !value || !g || !state_pool || !out || !state_out) return RGDR_ERR_NULL;
    if (mx && (!state_scales || !state_scales_out)) return RGDR_ERR_NULL;
    if (!idx && N_slots < B) return RGDR_ERR_SHAPE;
    a.sq = la_strides_or(query_strides, (long long)H_q * T * D_k, (long long)T * D_k, D_k);
    a.sk = la_strides_or(key_strides, (long long)H_q * T * D_k, (long long)T * D_k, D_k);
    a.sv = la_strides_or(value_strides, (long long)H_v * T * D_v, (long long)T * D_v, D_v);
    a.sg = la_strides_or(g_strides, (long long)H_v * T, T, 1);
    a.so = la_strides_or(out_strides, (long long)H_v * T * D_v, (long long)T * D_v, D_v);
    if (!la_strides_ok(a.sq) || !la_strides_ok(a.sk) || !la_strides_ok(a.sv) ||
        !la_strides_ok(a.sg) || !la_strides_ok(a.so))
        return RGDR_ERR_SHAPE;
    if (!la_extent_ok(a.sq, B, H_q, T, D_k) || !la_extent_ok(a.sk, B, H_q, T, D_k) ||
        !la_extent_ok(a.sv, B, H_v, T, D_v) || !la_extent_ok(a.sg, B, H_v, T, 1) ||
        !la_rows_distinct(a.so, B, H_v, T, D_v))
        return RGDR_ERR_SHAPE;
    // offsets within a chunk of tokens are counted in 32 bits
    if (T > 1 && (a.sq.t > kMaxTokenStride || a.sk.t > kMaxTokenStride || a.sv.t > kMaxTokenStride ||
                  a.sg.t > kMaxTokenStride || a.so.t > kMaxTokenStride))
        return RGDR_ERR_SHAPE;
    if (!la_strides_aligned(a.sq, B, H_q, T) || !la_strides_aligned(a.sk, B, H_q, T) ||
        !la_strides_aligned(a.sv, B, H_v, T) || !la_strides_aligned(a.so, B, H_v, T))
        return RGDR_ERR_ALIGN;
    if (!aligned(query, 16) || !aligned(key, 16) || !aligned(value, 16) || !aligned(g, 4) ||
        !aligned(state_pool, 16) || !aligned(state_out, 16) || !aligned(out, 16))
        return RGDR_ERR_ALIGN;
    if (mx && (!aligned(state_scales, 16) || !aligned(state_scales_out, 16))) return RGDR_ERR_ALIGN;
    if ((lens && !aligned(lens, 4)) || (idx && !aligned(idx, 4)) || (nacc && !aligned(nacc, 4)))
        return RGDR_ERR_ALIGN;
    if (T == 1) a.sq.t = a.sk.t = a.sv.t = a.sg.t = a.so.t = 0;
    a.q = static_cast<const uint16_t *>(query);
    a.k = static_cast<const uint16_t *>(key);
    a.v = static_cast<const uint16_t *>(value);
    a.g = g;
    a.pool = state_pool;
    a.scales = state_scales;
    a.out = static_cast<uint16_t *>(out);
    a.pool_out = state_out;
    a.scales_out = state_scales_out;
    a.in_place = state_pool == state_out && (!mx || state_scales == state_scales_out);
    a.lens = lens;
    a.idx = idx;
    a.nacc = nacc;
    a.scale = scale;
    a.B = B;
    a.Hq = H_q;
    a.Hv = H_v;
    a.T = T;
    a.Dv = D_v;
    a.N_slots = N_slots;
    a.group = H_v / H_q;
    return RGDR_OK;
}

}  // namespace rgdr

extern "C" rgdr_status la_decode(const void *query, const la_strides *query_strides,
                                 const void *key, const la_strides *key_strides,
                                 const void *value, const la_strides *value_strides,
                                 const float *g, const la_strides *g_strides,
                                 const void *state_pool, const uint8_t *state_scales,
                                 rgdr_dtype state_dtype, const int32_t *actual_seq_lengths,
                                 const int32_t *ssm_state_indices,
                                 const int32_t *num_accepted_tokens, float scale, int32_t B,
                                 int32_t H_q, int32_t H_v, int32_t T, int32_t D_k, int32_t D_v,
                                 int32_t N_slots, void *out, const la_strides *out_strides,
                                 void *state_out, uint8_t *state_scales_out, hipStream_t stream) {
    using namespace rgdr;
    LaArgs a;
    if (const rgdr_status st = la_check(
            a, kMaxT, query, query_strides, key, key_strides, value, value_strides, g, g_strides,
            state_pool, state_scales, state_dtype, actual_seq_lengths, ssm_state_indices,
            num_accepted_tokens, scale, B, H_q, H_v, T, D_k, D_v, N_slots, out, out_strides,
            state_out, state_scales_out))
        return st;
    if (B == 0) return RGDR_OK;
    if (state_dtype == RGDR_F32) return launch_decode<RGDR_F32>(a, D_k, stream);
    if (state_dtype == RGDR_BF16) return launch_decode<RGDR_BF16>(a, D_k, stream);
    return launch_decode<RGDR_MXI8>(a, D_k, stream);
}
