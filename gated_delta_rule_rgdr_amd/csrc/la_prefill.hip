// la_prefill.hip -- linear attention with a decay for each head, over whole prompts.
//
// For tokens 0..C-1 of a chunk with the incoming state S, G_t the running sum of the log decays
// and G the chunk's whole sum:
//     o_t = scale e^{G_t} S^T q_t + sum_{s <= t} scale e^{G_t - G_s} (q_t . k_s) v_s
//     S'  = e^G S + sum_s k_s (e^{G - G_s} v_s)^T
// which is the recurrence, regrouped into four dense products for the matrix cores. Exponents are
// differences of sums held in fp64, so a chunk may decay by any amount.
//
// Precision: q, k and v are bf16 and enter the products as they are. What is computed (the state, the
// scores, the weighted v of the state's update) enters as the sum of three bf16 numbers, which hold
// fp32's 24 bits, so that outputs and states are good to fp32 also where large terms cancel. (With two
// numbers, 16 bits, in all three places B=16, T=1024, H=16/32, D=128 took 128 us against 155 for a bf16
// state; the comparisons of parts below were timed in that form.) The state is kept in fp32 over the
// whole prompt.
#include "la_mfma.h"

namespace rgdr {

constexpr int kLaMaxPrompt = 65536;
constexpr int kChunk = 64;    // tokens
constexpr int kXcds = 8;      // of the device, each with its own L2
constexpr int kCols = 128;    // columns of one workgroup: 32 for each of its 4 waves

struct LaPlan {
    int state_dtype, tiles, seg_len, nseg;
    int per;           // workgroups of a unit, which run on one XCD
    float *seg_state;  // [nseg][B*H_v][D_v/32][D_k/32][4][64][4]: accumulator layout
    float *seg_decay;  // [nseg][B*H_v]
};

// The largest of 32 lanes' values: rotations within rows of 16, then the two rows' exchange.
template <int CTRL>
__device__ __forceinline__ uint32_t max_rotated(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t half_max(uint32_t x) {
    x = max_rotated<0x121>(max_rotated<0x122>(max_rotated<0x124>(max_rotated<0x128>(x))));
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return max(r[0], r[1]);
}

// One wave's 32 columns of a state, D_k rows: register r = 8 kb + e of tile `it` is row
// 32 it + 16 kb + 8 (lane / 32) + e, column map32(lane % 32).
// `base`: the element of the wave's first column in the state's first row.
template <int DK, int ST>
__device__ __forceinline__ void load_state(f32x16 (&S)[DK / 32], const void *pool, long long base, int Dv, int lane) {
    constexpr int kSize = ST == RGDR_F32 ? 4 : 2;
    const char *p = static_cast<const char *>(pool) + base * kSize;
    const uint32_t at = (uint32_t)((lane >> 5) * 8 * Dv + map32(lane & 31)) * kSize;
#pragma unroll
    for (int it = 0; it < DK / 32; ++it) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = it * 32 + (r >> 3) * 16 + (r & 7);
            const char *x = p + (uint32_t)(row * Dv) * kSize;
            if constexpr (ST == RGDR_F32)
                S[it][r] = *reinterpret_cast<const float *>(x + at);
            else
                S[it][r] = bf16_to_f32(*reinterpret_cast<const uint16_t *>(x + at));
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <int DK, int ST>
__device__ __forceinline__ void store_state(const f32x16 (&S)[DK / 32], void *pool, long long base, int Dv, int lane) {
    constexpr int kSize = ST == RGDR_F32 ? 4 : 2;
    char *p = static_cast<char *>(pool) + base * kSize;
    asm volatile("" : "+v"(lane));  // the rows' addresses are formed here, not kept from the prompt's start
    const uint32_t at = (uint32_t)((lane >> 5) * 8 * Dv + map32(lane & 31)) * kSize;
#pragma unroll
    for (int it = 0; it < DK / 32; ++it)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = it * 32 + (r >> 3) * 16 + (r & 7);
            char *x = p + (uint32_t)(row * Dv) * kSize;
            const float y = S[it][r];
            if constexpr (ST == RGDR_F32)
                *reinterpret_cast<float *>(x + at) = y;
            else
                *reinterpret_cast<uint16_t *>(x + at) = f32_to_bf16(y);
            if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // a few rows at a time: registers
        }
}

// 8-bit states go in pieces of 16 bytes (half a block) through LDS that is the wave's own: the codes of
// its D_k blocks, then their scale bytes. (B=16, T=1024, H=16/32, D=128: 141 us; code by code to and
// from memory 160.)
template <int DK>
__device__ __forceinline__ constexpr int mx_lds_bytes() {
    return DK * (kMxBlock + 1);
}
template <int DK>
__device__ __forceinline__ void load_state_mx(f32x16 (&S)[DK / 32], const void *pool, const uint8_t *scales,
                                              long long base, int Dv, char *lds, int lane) {
    const char *p = static_cast<const char *>(pool) + base;
    const uint8_t *sc = scales + base / kMxBlock;
    u32x4 w[DK / 32];
    uint8_t eb[DK / 64];
#pragma unroll
    for (int m = 0; m < DK / 32; ++m)
        w[m] = *reinterpret_cast<const u32x4 *>(p + (uint32_t)((m * 32 + lane / 2) * Dv + lane % 2 * 16));
#pragma unroll
    for (int m = 0; m < DK / 64; ++m) eb[m] = sc[(uint32_t)((m * 64 + lane) * (Dv / kMxBlock))];
#pragma unroll
    for (int m = 0; m < DK / 32; ++m) *reinterpret_cast<u32x4 *>(lds + (m * 64 + lane) * 16) = w[m];
#pragma unroll
    for (int m = 0; m < DK / 64; ++m) lds[DK * kMxBlock + m * 64 + lane] = (char)eb[m];
    wave_in_order();
    const char *const code = lds + (lane >> 5) * 8 * kMxBlock + map32(lane & 31);
    const char *const scale = lds + DK * kMxBlock + (lane >> 5) * 8;
#pragma unroll
    for (int it = 0; it < DK / 32; ++it)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const int row = it * 32 + kb * 16;
            const u32x2 e8 = *reinterpret_cast<const u32x2 *>(scale + row);  // of eight rows
#pragma unroll
            for (int e = 0; e < 8; ++e)
                S[it][kb * 8 + e] =
                    static_cast<float>(*reinterpret_cast<const int8_t *>(code + (row + e) * kMxBlock)) *
                    mx_scale(e8[e / 4] >> (e % 4 * 8) & 255);
        }
    wave_in_order();
}
template <int DK>
__device__ __forceinline__ void store_state_mx(const f32x16 (&S)[DK / 32], void *pool, uint8_t *scales,
                                               long long base, int Dv, char *lds, int lane) {
    asm volatile("" : "+v"(lane));  // as in store_state
    char *const code = lds + (lane >> 5) * 8 * kMxBlock + map32(lane & 31);
    char *const scale = lds + DK * kMxBlock + (lane >> 5) * 8;
#pragma unroll
    for (int it = 0; it < DK / 32; ++it)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = it * 32 + (r >> 3) * 16 + (r & 7);
            const uint32_t eb = mx_exponent(half_max(mx_top_bits(S[it][r])));
            code[row * kMxBlock] = (char)mx_code_bits(S[it][r], mx_inverse(eb));
            scale[row] = (char)eb;  // the same from 32 lanes
            if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
    wave_in_order();
    char *p = static_cast<char *>(pool) + base;
    uint8_t *sc = scales + base / kMxBlock;
#pragma unroll
    for (int m = 0; m < DK / 32; ++m)
        *reinterpret_cast<u32x4 *>(p + (uint32_t)((m * 32 + lane / 2) * Dv + lane % 2 * 16)) =
            *reinterpret_cast<const u32x4 *>(lds + (m * 64 + lane) * 16);
#pragma unroll
    for (int m = 0; m < DK / 64; ++m)
        sc[(uint32_t)((m * 64 + lane) * (Dv / kMxBlock))] = (uint8_t)lds[DK * kMxBlock + m * 64 + lane];
    wave_in_order();
}

// Which (entry, segment, value head, columns) a workgroup works on. A unit is what shares a query/key
// head: its value heads and their columns, which run on one XCD, so that q and k meet in its
// L2. Units go round the XCDs (workgroup ids do), those of the longest entries first: with
// ragged lengths every XCD, and every compute unit's two places, then get long and short ones.
// (B=16, H=16/32, D=128, lengths from 0 to 1024: 101.5 us, against 108.2 with each XCD's units
// contiguous, both before the work between the products below.) Where units do not go round the XCDs
// evenly, each workgroup is a unit of its own (launch_prefill).
struct LaItem {
    int b, seg, h, tile;
    bool live;
};

__device__ __forceinline__ int entry_of_rank(const LaArgs &a, int rank) {
    if (!a.lens || a.B < 2 || a.B > 64) return rank;
    const int lane = threadIdx.x & 63;
    const int L = lane < a.B ? min(max(a.lens[lane], 0), a.T) : -1;
    int r = 0;  // of this lane's entry: how many are longer, or as long and before it
    for (int j = 0; j < a.B; ++j) {
        const int other = __builtin_amdgcn_readlane(L, j);
        r += other > L || (other == L && j < lane);
    }
    return __builtin_ctzll(__ballot(lane < a.B && r == rank));
}

template <bool SEGMENTS>
__device__ __forceinline__ LaItem la_item(const LaArgs &a, const LaPlan &p) {
    const int local = blockIdx.x / kXcds, share = a.group * p.tiles;  // workgroups of a query/key head
    int unit = local / p.per * kXcds + blockIdx.x % kXcds, in_group = local % p.per;
    LaItem m;
    m.live = unit < a.B * a.Hq * (SEGMENTS ? p.nseg : 1) * (share / p.per);
    if (p.per == 1) {
        in_group = unit % share;
        unit /= share;
    }
    m.tile = in_group % p.tiles;
    in_group /= p.tiles;
    const int hq = unit % a.Hq;
    unit /= a.Hq;
    m.seg = SEGMENTS ? unit % p.nseg : 0;
    m.b = entry_of_rank(a, m.live ? (SEGMENTS ? unit / p.nseg : unit) : 0);
    m.h = hq * a.group + in_group;
    return m;
}

template <int N>
struct Count {
    static constexpr int value = N;
};

// One step of a stretch of products: LOADS reads of LDS, then N products with VALU vector
// instructions behind each, which issue while it runs. Left to itself the compiler puts a step's
// products in a row and its vector work behind them (B=16, T=1024, D=128, bf16: 132 us, B=8 80.5; so
// 130 and 78.9).
template <int LOADS, int N, int VALU>
__device__ __forceinline__ void interleave() {
    __builtin_amdgcn_sched_group_barrier(0x100, LOADS, 0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x2, VALU, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// S += sum_s k_s (w_s v_s)^T over the 64 tokens of a chunk: k from LDS, v's operands in registers, one
// weight for each token in LDS.
template <int DK>
__device__ __forceinline__ void add_chunk(f32x16 (&S)[DK / 32], char *lk, const bf16x8 (&vf)[4],
                                          const float *weight, int lane) {
    constexpr int KP = DK / 8;
    constexpr int NI = DK / 32;
    u32x4 kf[2][NI], hi[2], lo[2], lo2[2];
    f32x4 wf[2][2];
    auto load_k = [&](int kb) {
#pragma unroll
        for (int it = 0; it < NI; ++it)
            kf[kb & 1][it] = __builtin_bit_cast(u32x4, lds_read_tr<KP, kTrPad>(lk, kb * 16, it, lane));
    };
    auto load_w = [&](int kb) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            wf[kb & 1][i] = *reinterpret_cast<const f32x4 *>(weight + kb * 16 + (lane >> 5) * 8 + i * 4);
    };
    auto weigh = [&](int kb) {
        float x[8];
        const u32x4 v = __builtin_bit_cast(u32x4, vf[kb]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = bf16_lo(v[e]) * wf[kb & 1][e / 2][2 * e % 4];
            x[2 * e + 1] = bf16_hi(v[e]) * wf[kb & 1][e / 2][2 * e % 4 + 1];
        }
        split2(x, hi[kb & 1], lo[kb & 1]);
        lo2[kb & 1] = split_rest(x, lo[kb & 1]);
    };
    load_w(0);
    load_k(0);
    load_w(1);
    weigh(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
        if (kb < 3) {
            load_k(kb + 1);
            weigh(kb + 1);
        }
        if (kb < 2) load_w(kb + 2);
#pragma unroll
        for (int it = 0; it < NI; ++it) S[it] = mfma(kf[kb & 1][it], __builtin_bit_cast(bf16x8, lo2[kb & 1]), S[it]);
#pragma unroll
        for (int it = 0; it < NI; ++it) S[it] = mfma(kf[kb & 1][it], __builtin_bit_cast(bf16x8, lo[kb & 1]), S[it]);
#pragma unroll
        for (int it = 0; it < NI; ++it) S[it] = mfma(kf[kb & 1][it], __builtin_bit_cast(bf16x8, hi[kb & 1]), S[it]);
        // a step: eight values, weighted and split, 8 instructions each
        interleave<2 * NI, 3 * NI, 64 / (3 * NI)>();
    }
}

// What one segment adds to the state behind it, from a zero state, into the workspace: the first pass
// over a long prompt. Its chunks are taken from the last to the first, each token weighted by the
// decay from it to the segment's end, so nothing is rescaled in between. A segment that another one
// of the entry follows is full. Two chunks are in flight. B=1, H=16/32, T=8192, D=128: 37 us for 16
// segments of 8 chunks, of which the last states' way out and the first loads are a third.
template <int DK, bool FULL>
__global__ __launch_bounds__(256, DK == 256 ? 1 : 2) void la_segment_kernel(const LaArgs a, const LaPlan p) {
    constexpr int KP = DK / 8, NR = kChunk * KP / 256, NV = kChunk * 16 / 256;
    constexpr int RK = lds_row_bytes<KP, kTrPad>(), RV = lds_row_bytes<16, kTrPad>();
    __shared__ __align__(256) char lk[kChunk * RK], lv[kChunk * RV];
    __shared__ __align__(16) float keep[2][kChunk];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const LaItem item = la_item<true>(a, p);
    if (!item.live) return;
    const int tile = item.tile, h = item.h, seg = item.seg, b = item.b;
    const LaEntry en = la_entry(a, b);
    const int t_begin = seg * p.seg_len;
    if (!en.state || t_begin + p.seg_len >= en.L) return;  // no later segment needs it
    const int bh = b * a.Hv + h;
    const bool mine = FULL || tile * kCols + wave * 32 < a.Dv;  // this wave has columns
    const int vpieces = FULL ? 16 : min(16, (a.Dv - tile * kCols) / 8);
    const uint16_t *gk = a.k + b * a.sk.b + h / a.group * a.sk.h + t_begin * a.sk.t;
    const uint16_t *gv = a.v + b * a.sv.b + h * a.sv.h + tile * kCols + t_begin * a.sv.t;
    const float *gg = a.g + b * a.sg.b + h * a.sg.h + t_begin * a.sg.t;
    const uint32_t kt = (uint32_t)a.sk.t * 2, vt = (uint32_t)a.sv.t * 2, g_at = lane * (uint32_t)a.sg.t;
    const uint32_t k0 = tid / KP * kt + tid % KP * 16, v0 = tid / 16 * vt + min(tid % 16, vpieces - 1) * 16;
    const int k_to = lds_at<KP, kTrPad>(tid / KP, tid % KP), v_to = lds_at<16, kTrPad>(tid / 16, tid % 16);

    f32x16 S[DK / 32];
#pragma unroll
    for (int it = 0; it < DK / 32; ++it)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[it][r] = 0.f;

    u32x4 rk[2][NR], rv[2][NV];
    auto fetch = [&](u32x4 (&fk)[NR], u32x4 (&fv)[NV], int c) {
        const char *k = reinterpret_cast<const char *>(gk) + (uint64_t)(c * kChunk) * kt;
        const char *v = reinterpret_cast<const char *>(gv) + (uint64_t)(c * kChunk) * vt;
#pragma unroll
        for (int m = 0; m < NR; ++m) fk[m] = *reinterpret_cast<const u32x4 *>(k + (uint64_t)(m * (256 / KP)) * kt + k0);
#pragma unroll
        for (int m = 0; m < NV; ++m) fv[m] = *reinterpret_cast<const u32x4 *>(v + (uint64_t)(m * 16) * vt + v0);
    };
    auto fetch_g = [&](int c) { return (gg + (long long)(c * kChunk) * a.sg.t)[g_at]; };
    double behind = 0.0;  // wave 3: the log2 decay from the chunk's end to the segment's
    auto weights = [&](float g, int to) {
        constexpr double kLog2e = 1.4426950408889634;
        const double G = wave_scan((double)la_log_decay(g) * kLog2e), end = wave_last(G);
        keep[to][lane] = __builtin_amdgcn_exp2f((float)(behind + (end - G)));
        behind += end;
    };

    int c = p.seg_len / kChunk - 1, buf = 0;
    float g_next = 0.f;
    fetch(rk[0], rv[0], c);
    if (c > 0) fetch(rk[1], rv[1], c - 1);
    if (wave == 3) {
        weights(fetch_g(c), 0);
        if (c > 0) g_next = fetch_g(c - 1);
    }
    auto step = [&](u32x4 (&fk)[NR], u32x4 (&fv)[NV]) {
#pragma unroll
        for (int m = 0; m < NR; ++m) *reinterpret_cast<u32x4 *>(lk + k_to + m * (256 / KP) * RK) = fk[m];
#pragma unroll
        for (int m = 0; m < NV; ++m) *reinterpret_cast<u32x4 *>(lv + v_to + m * 16 * RV) = fv[m];
        __syncthreads();
        if (c > 1) fetch(fk, fv, c - 2);
        if (wave == 3 && c > 0) {
            weights(g_next, buf ^ 1);
            if (c > 1) g_next = fetch_g(c - 2);
        }
        if (mine) {
            bf16x8 vf[4];
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) vf[kb] = lds_read_tr<16, kTrPad>(lv, kb * 16, wave, lane);
            add_chunk<DK>(S, lk, vf, keep[buf], lane);
        }
        __syncthreads();
        buf ^= 1;
    };
    while (true) {
        step(rk[0], rv[0]);
        if (--c < 0) break;
        step(rk[1], rv[1]);
        if (--c < 0) break;
    }
    if (mine) {
        float *const ws = p.seg_state + (((long long)seg * a.B * a.Hv + bh) * (a.Dv / 32) + tile * 4 + wave) * (DK * 32);
#pragma unroll
        for (int it = 0; it < DK / 32; ++it)
#pragma unroll
            for (int m = 0; m < 4; ++m)
                *reinterpret_cast<f32x4 *>(ws + ((it * 4 + m) * 64 + lane) * 4) =
                    f32x4{S[it][m * 4], S[it][m * 4 + 1], S[it][m * 4 + 2], S[it][m * 4 + 3]};
    }
    if (wave == 3 && tile == 0 && lane == 0)
        p.seg_decay[(long long)seg * a.B * a.Hv + bh] = __builtin_amdgcn_exp2f((float)behind);
}

// Bound: latency in each wave. B=16, H=16/32, T=1024, D=128, bf16 155 us (2.8 TB/s, 221 TFLOP/s of the
// recurrence): of the 15,700 cycles that a SIMD's two waves spend on a chunk each, their products take
// 7,600 and the issue of their other vector instructions 8,100, so each of the two pipes is free for
// half of the time. A wave waits for three fifths of it: at the three barriers of a chunk, for results of
// its own chain (scores, their split, their product; the state's split, its product), and for its turn
// to issue.
//
// A workgroup works through the tokens of one (entry, value head, 128 columns): a whole prompt, or
// one segment of it. The 4 waves hold 32 columns of the state each, in accumulator registers; the
// chunk's q, k and v lie in LDS, and the waves share the ten 16 x 16 tiles of the scores, two or three
// each; one with two also sums the next chunk's decays. The next chunk's rows are in flight meanwhile.
//
// FULL: D_v is a multiple of 128, so every wave has columns; a template argument, so that a chunk is a
// few long stretches of code without branches, in which the products and the vector work around them
// can be interleaved.
template <int DK, bool SEGMENTS, bool FULL>
__global__ __launch_bounds__(256, DK == 256 ? 1 : 2) void la_chunk_kernel(const LaArgs a, const LaPlan p) {
    constexpr int KP = DK / 8;                 // 16-byte pieces of a q or k row
    constexpr int NR = kChunk * KP / 256;      // of them in each thread's hands
    constexpr int NV = kChunk * 16 / 256;
    constexpr int RQ = lds_row_bytes<KP>(), RK = lds_row_bytes<KP, kTrPad>(), RV = lds_row_bytes<16, kTrPad>();
    // Scores: 32 rows of the 32 tokens that they may see, then 32 of all 64, each with a spare piece. (Rows of
    // one length for all would take the second workgroup's place on the compute unit at D_k = 128.)
    constexpr int RP0 = 5 * 16, RP1 = 9 * 16, kPlane = 32 * (RP0 + RP1);
    __shared__ __align__(256) char lq[kChunk * RQ];
    __shared__ __align__(256) char lk[kChunk * RK];
    __shared__ __align__(256) char lv[kChunk * RV];
    __shared__ __align__(256) char lp[3][kPlane];
    // Of each token of this chunk and the next: the log2 decay sum in two floats, what a later
    // state keeps of it, and what it keeps of the incoming state (with the scale).
    __shared__ __align__(16) float g_hi[2][kChunk], g_lo[2][kChunk], keep[2][kChunk], carry[2][kChunk];
    __shared__ float whole[2];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const LaItem item = la_item<SEGMENTS>(a, p);
    if (!item.live) return;
    const int tile = item.tile, h = item.h, seg = item.seg, b = item.b;
    const LaEntry en = la_entry(a, b);
    const int t_begin = SEGMENTS ? seg * p.seg_len : 0;
    const int t_stop = SEGMENTS ? min(a.T, t_begin + p.seg_len) : a.T;
    const int t_end = min(en.L, t_stop);
    const int hq = h / a.group, bh = b * a.Hv + h;
    const int col0 = tile * kCols + wave * 32;
    const bool mine = FULL || col0 < a.Dv;  // this wave has columns
    const int vpieces = FULL ? 16 : min(16, (a.Dv - tile * kCols) / 8);

    const uint16_t *gq = a.q + b * a.sq.b + hq * a.sq.h;
    const uint16_t *gk = a.k + b * a.sk.b + hq * a.sk.h;
    const uint16_t *gv = a.v + b * a.sv.b + h * a.sv.h + tile * kCols;
    const float *gg = a.g + b * a.sg.b + h * a.sg.h;
    uint16_t *go = a.out + b * a.so.b + h * a.so.h + col0;

    // rows of tokens past the entry's length
    {
        const int from = max(t_begin, t_end);
        for (int j = tid; j < (t_stop - from) * vpieces; j += 256)
            *reinterpret_cast<u32x4 *>(a.out + b * a.so.b + h * a.so.h + tile * kCols +
                                       (from + j / vpieces) * a.so.t + (j % vpieces) * 8) = u32x4{0, 0, 0, 0};
    }
    if (!en.state) return;
    if (t_begin >= t_end && t_begin != 0) return;  // the first segment commits the state of no token

    // The wave's share of q's place: free before the first chunk, and from the scores on until the next.
    static_assert(4 * mx_lds_bytes<DK>() <= kChunk * RQ, "8-bit states pass through q's rows");
    char *const lmx = lq + wave * mx_lds_bytes<DK>();
    f32x16 S[DK / 32];
    const long long base = ((long long)__builtin_amdgcn_readfirstlane(en.slot) * a.Hv + h) * DK * a.Dv + col0;
    if (mine) {
        if constexpr (SEGMENTS) {
            const float *const ws =
                p.seg_state + (((long long)seg * a.B * a.Hv + bh) * (a.Dv / 32) + tile * 4 + wave) * (DK * 32);
#pragma unroll
            for (int it = 0; it < DK / 32; ++it)
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const f32x4 x = *reinterpret_cast<const f32x4 *>(ws + ((it * 4 + m) * 64 + lane) * 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[it][m * 4 + e] = x[e];
                }
        } else if (p.state_dtype == RGDR_F32) {
            load_state<DK, RGDR_F32>(S, a.pool, base, a.Dv, lane);
        } else if (p.state_dtype == RGDR_BF16) {
            load_state<DK, RGDR_BF16>(S, a.pool, base, a.Dv, lane);
        } else {
            load_state_mx<DK>(S, a.pool, a.scales, base, a.Dv, lmx, lane);
        }
    }
    auto commit = [&]() {
        if (!mine) return;
        if (p.state_dtype == RGDR_F32)
            store_state<DK, RGDR_F32>(S, a.pool_out, base, a.Dv, lane);
        else if (p.state_dtype == RGDR_BF16)
            store_state<DK, RGDR_BF16>(S, a.pool_out, base, a.Dv, lane);
        else
            store_state_mx<DK>(S, a.pool_out, a.scales_out, base, a.Dv, lmx, lane);
    };
    if (t_begin == 0 && en.n == 0 && !a.in_place) commit();
    if (t_begin >= t_end) return;
    if (p.state_dtype == RGDR_MXI8) __syncthreads();  // every wave's state is through q's place

    // A chunk ends after 64 tokens, at the accepted count (whose state is committed) or at the end.
    auto chunk_end = [&](int t) { return min(min(t + kChunk, t_end), t < en.n ? en.n : t_end); };

    u32x4 rq[NR], rk[NR], rv[NV];
    // One row of a token for each 16 (or D_k / 8) threads. Rows past the chunk repeat its last row:
    // they are not padding's (never read), and their weights are zero.
    const uint32_t qt = (uint32_t)a.sq.t * 2, kt = (uint32_t)a.sk.t * 2, vt = (uint32_t)a.sv.t * 2;
    const uint32_t qk_row = tid / KP, qk_at = tid % KP * 16, v_row = tid / 16;
    const uint32_t v_at = min(tid % 16, vpieces - 1) * 16;
    auto fetch = [&](int t0, int n) {
        const char *q = reinterpret_cast<const char *>(gq + t0 * a.sq.t);
        const char *k = reinterpret_cast<const char *>(gk + t0 * a.sk.t);
        const char *v = reinterpret_cast<const char *>(gv + t0 * a.sv.t);
        if (n == kChunk) {  // a lane's offsets are the same for every set of rows
            const uint32_t q0 = qk_row * qt + qk_at, k0 = qk_row * kt + qk_at, v0 = v_row * vt + v_at;
#pragma unroll
            for (int m = 0; m < NR; ++m) {
                rq[m] = *reinterpret_cast<const u32x4 *>(q + (uint64_t)(m * (256 / KP)) * qt + q0);
                rk[m] = *reinterpret_cast<const u32x4 *>(k + (uint64_t)(m * (256 / KP)) * kt + k0);
            }
#pragma unroll
            for (int m = 0; m < NV; ++m) rv[m] = *reinterpret_cast<const u32x4 *>(v + (uint64_t)(m * 16) * vt + v0);
        } else {
#pragma unroll
            for (int m = 0; m < NR; ++m) {
                const uint32_t t = min(m * (256 / KP) + qk_row, (uint32_t)n - 1);
                rq[m] = *reinterpret_cast<const u32x4 *>(q + (t * qt + qk_at));
                rk[m] = *reinterpret_cast<const u32x4 *>(k + (t * kt + qk_at));
            }
#pragma unroll
            for (int m = 0; m < NV; ++m)
                rv[m] = *reinterpret_cast<const u32x4 *>(v + (min(m * 16 + v_row, (uint32_t)n - 1) * vt + v_at));
        }
    };
    const int q_to = lds_at<KP>(tid / KP, tid % KP), k_to = lds_at<KP, kTrPad>(tid / KP, tid % KP);
    const int v_to = lds_at<16, kTrPad>(tid / 16, tid % 16);
    auto stage = [&]() {
#pragma unroll
        for (int m = 0; m < NR; ++m) {
            const int set = m * (256 / KP);  // rows of one set of pieces
            *reinterpret_cast<u32x4 *>(lq + q_to + set * RQ) = rq[m];
            *reinterpret_cast<u32x4 *>(lk + k_to + set * RK) = rk[m];
        }
#pragma unroll
        for (int m = 0; m < NV; ++m) *reinterpret_cast<u32x4 *>(lv + v_to + m * 16 * RV) = rv[m];
    };
    const uint32_t g_at = (uint32_t)a.sg.t, out_at = (uint32_t)(lane & 31) * (uint32_t)a.so.t * 2 + (lane >> 5) * 16;
    auto fetch_g = [&](int t0, int n) { return (gg + (long long)t0 * a.sg.t)[(uint32_t)min(lane, n - 1) * g_at]; };
    // One lane for each token: decay sums of a chunk of n tokens, into buffer `to`.
    auto decays = [&](float x, int n, int to) {
        constexpr double kLog2e = 1.4426950408889634;
        const double G = wave_scan(lane < n ? (double)la_log_decay(x) * kLog2e : 0.0), end = wave_last(G);
        const float hi = (float)G;
        g_hi[to][lane] = hi;
        g_lo[to][lane] = (float)(G - (double)hi);
        keep[to][lane] = lane < n ? __builtin_amdgcn_exp2f((float)(end - G)) : 0.f;
        carry[to][lane] = __builtin_amdgcn_exp2f(hi) * a.scale;
        if (lane == 0) whole[to] = __builtin_amdgcn_exp2f((float)end);
    };

    // The two tiles above the diagonal that the products of 32 tokens by 32 read: zero for good.
    if (tid < 3 * 2 * 16 * 2) {
        const int plane = tid >> 6, half = tid >> 5 & 1, row = tid >> 1 & 15, piece = tid & 1;
        *reinterpret_cast<u32x4 *>(lp[plane] + (half ? 32 * RP0 + row * RP1 + 96 : row * RP0 + 32) + piece * 16) =
            u32x4{0, 0, 0, 0};
    }

    int t0 = t_begin, t1 = chunk_end(t0), buf = 0;
    float g_next = 0.f;
    fetch(t0, t1 - t0);
    if (wave == 3) {
        decays(fetch_g(t0, t1 - t0), t1 - t0, 0);
        if (t1 < t_end) g_next = fetch_g(t1, chunk_end(t1) - t1);
    }
    while (true) {
        const int n = t1 - t0;
        const int t2 = t1 < t_end ? chunk_end(t1) : t1;
        // The lane's number, as if new in each round: the many addresses made of it are cheap to
        // form again, and would not fit the registers if they were kept over the loop.
        int now = tid;
        asm volatile("" : "+v"(now));
        const int lane = now & 63, col = lane & 31, hf = lane >> 5;
        stage();
        __syncthreads();
        // scores of tokens t (lanes) and s (registers), in tiles on and below the diagonal: (3,0..3),
        // (2,0..2), (1,0..1), (0,0); the last two waves have two, and the last one the decays, whose
        // chain the others would wait for.
        auto scores = [&](auto count) {
            constexpr int NS = decltype(count)::value;
            const int l16 = lane & 15, l4 = lane >> 4;
            f32x4 x[NS] = {};
            int ts[NS], ss[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const int i = wave + 4 * j;
                ts[j] = (i < 4 ? 3 : i < 7 ? 2 : i < 9 ? 1 : 0) * 16 + l16;
                ss[j] = (i < 4 ? i : i < 7 ? i - 4 : i < 9 ? i - 7 : 0) * 16;
            }
            bf16x8 kf[2][NS], qf[2][NS];
            auto load = [&](int c) {
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    kf[c & 1][j] = lds_read(lk + lds_at<KP, kTrPad>(ss[j] + l16, c * 4 + l4));
                    qf[c & 1][j] = lds_read(lq + lds_at<KP>(ts[j], c * 4 + l4));
                }
            };
            load(0);
#pragma unroll
            for (int c = 0; c < DK / 32; ++c) {
                if (c + 1 < DK / 32) load(c + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < NS; ++j) x[j] = mfma16(kf[c & 1][j], qf[c & 1][j], x[j]);
            }
            float th[NS], tl[NS];
            f32x4 sh[NS], sl[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                th[j] = g_hi[buf][ts[j]];
                tl[j] = g_lo[buf][ts[j]];
                sh[j] = *reinterpret_cast<const f32x4 *>(&g_hi[buf][ss[j] + l4 * 4]);
                sl[j] = *reinterpret_cast<const f32x4 *>(&g_lo[buf][ss[j] + l4 * 4]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const int t = ts[j], s = ss[j] + l4 * 4;
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float w = __builtin_amdgcn_exp2f((th[j] - sh[j][e]) + (tl[j] - sl[j][e])) * a.scale;
                    asm volatile("" : "+v"(w));  // formed for every lane: no branch around it
                    y[e] = s + e <= t ? x[j][e] * w : 0.f;  // columns t past the chunk are not stored
                }
                const int at = wave + 4 * j < 7 ? 32 * RP0 + (t - 32) * RP1 + s * 2 : t * RP0 + s * 2;
#pragma unroll
                for (int pl = 0; pl < 3; ++pl) {
                    const u32x2 part = {pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
                    *reinterpret_cast<u32x2 *>(lp[pl] + at) = part;
                    bf16_rest(part[0], y[0], y[1]);
                    bf16_rest(part[1], y[2], y[3]);
                }
            }
        };
        if (wave < 2) {
            scores(Count<3>{});
        } else {
            if (wave == 3 && t2 > t1) {
                decays(g_next, t2 - t1, buf ^ 1);
                if (t2 < t_end) g_next = fetch_g(t2, chunk_end(t2) - t2);
            }
            scores(Count<2>{});
        }
        bf16x8 vf[4];
        f32x16 o[2] = {};
        // S^T q; the next chunk's loads go out between the products, since twelve in a row keep each
        // wave waiting 800 cycles for their issue; before them all where that chunk is not whole.
        // (B=16 130 -> 128 us, B=8 78.9 -> 75.2, one prompt of 8192 tokens 120 -> 117, with the
        // scores' share for each wave below.)
        auto incoming = [&](auto loads) {
            constexpr bool LOADS = decltype(loads)::value;
            constexpr int NS = DK / 16, NL = 2 * NR + NV;
            const char *gq1 = reinterpret_cast<const char *>(gq + t1 * a.sq.t);
            const char *gk1 = reinterpret_cast<const char *>(gk + t1 * a.sk.t);
            const char *gv1 = reinterpret_cast<const char *>(gv + t1 * a.sv.t);
            const uint32_t q0 = qk_row * qt + qk_at, k0 = qk_row * kt + qk_at, v0 = v_row * vt + v_at;
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) vf[kb] = lds_read_tr<16, kTrPad>(lv, kb * 16, wave, lane);
            bf16x8 qf[2][2];
            u32x4 hi[2], lo[2], lo2[2];
            auto load = [&](int c) {
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) qf[c & 1][tt] = lds_read(lq + lds_at<KP>(tt * 32 + col, c * 2 + hf));
            };
            auto parts = [&](int c) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = S[c / 2][(c & 1) * 8 + e];
                split2(x, hi[c & 1], lo[c & 1]);
                lo2[c & 1] = split_rest(x, lo[c & 1]);
            };
            load(0);
            parts(0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = 0; c < NS; ++c) {
                if (c + 1 < NS) {
                    load(c + 1);
                    parts(c + 1);
                }
                if constexpr (LOADS)
#pragma unroll
                    for (int i = c * NL / NS; i < (c + 1) * NL / NS; ++i) {
                        const int m = i < 2 * NR ? i / 2 : i - 2 * NR;
                        if (i >= 2 * NR)
                            rv[m] = *reinterpret_cast<const u32x4 *>(gv1 + (uint64_t)(m * 16) * vt + v0);
                        else if (i % 2)
                            rk[m] = *reinterpret_cast<const u32x4 *>(gk1 + (uint64_t)(m * (256 / KP)) * kt + k0);
                        else
                            rq[m] = *reinterpret_cast<const u32x4 *>(gq1 + (uint64_t)(m * (256 / KP)) * qt + q0);
                    }
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) o[tt] = mfma(hi[c & 1], qf[c & 1][tt], o[tt]);
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) o[tt] = mfma(lo[c & 1], qf[c & 1][tt], o[tt]);
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) o[tt] = mfma(lo2[c & 1], qf[c & 1][tt], o[tt]);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
                for (int i = 0; i < 6; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                    if (LOADS && i % 3 == 1) __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x2, 6, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                const float c = carry[buf][tt * 32 + col];
#pragma unroll
                for (int r = 0; r < 16; ++r) o[tt][r] *= c;
            }
        };
        if (mine && t2 - t1 == kChunk) {
            incoming(Count<1>{});
        } else {
            if (t2 > t1) fetch(t1, t2 - t1);
            if (mine) incoming(Count<0>{});
        }
        __syncthreads();
        if (mine) {
            // (second tokens, s block 3), (2), then both halves for blocks 1 and 0
            bf16x8 pf[2][6];
            auto load = [&](int kb) {
#pragma unroll
                for (int tt = kb < 2 ? 0 : 1; tt < 2; ++tt)
#pragma unroll
                    for (int pl = 0; pl < 3; ++pl)
                        pf[kb & 1][tt * 3 + pl] =
                            lds_read(lp[pl] + (tt ? 32 * RP0 + col * RP1 : col * RP0) + (kb * 2 + hf) * 16);
            };
            load(3);
            const float d = whole[buf];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kb = 3; kb >= 0; --kb) {
                if (kb > 0) load(kb - 1);
#pragma unroll
                for (int it = kb * DK / 128; it < (kb + 1) * DK / 128; ++it)
#pragma unroll
                    for (int r = 0; r < 16; ++r) S[it][r] *= d;
#pragma unroll
                for (int it = kb * DK / 128; it < (kb + 1) * DK / 128; ++it)
                    asm volatile("" : "+v"(S[it]));  // here, among the products
#pragma unroll
                for (int pl = 0; pl < 3; ++pl)
#pragma unroll
                    for (int tt = kb < 2 ? 0 : 1; tt < 2; ++tt)
                        o[tt] = mfma(__builtin_bit_cast(u32x4, vf[kb]), pf[kb & 1][tt * 3 + pl], o[tt]);
                if (kb < 2)
                    interleave<6, 6, 3>();
                else
                    interleave<6, 3, 6>();
            }
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
                if (tt * 32 + col < n) {
                    char *row = reinterpret_cast<char *>(go + (long long)(t0 + tt * 32) * a.so.t) + out_at;
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        u32x4 y;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[e] = pack_bf16x2(o[tt][m * 8 + 2 * e], o[tt][m * 8 + 2 * e + 1]);
                        *reinterpret_cast<u32x4 *>(row + m * 32) = y;
                    }
                }
            if (t1 < t_end || t1 == en.n) {
                add_chunk<DK>(S, lk, vf, keep[buf], lane);
            }
        }
        if (t1 == en.n) commit();
        if (t2 == t1) break;
        __syncthreads();
        t0 = t1;
        t1 = t2;
        buf ^= 1;
    }
}

// Segments' own contributions into their incoming states, in place: one thread for four rows of a
// column. The states in the pool are read here and committed by the next kernel, since a slot may
// be updated in place. Bound: the states, in and out (13.3 us for 16 segments of 32 heads at D = 128,
// 4.9 TB/s).
template <int ST>
__global__ __launch_bounds__(256) void la_scan_kernel(const LaArgs a, const LaPlan p, int DK) {
    const int per = a.Dv * DK / 4;  // threads for each (entry, head)
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const int bh = (int)(id / per), x = (int)(id % per);
    if (bh >= a.B * a.Hv) return;
    const int b = bh / a.Hv, h = bh % a.Hv;
    const LaEntry en = la_entry(a, b);
    if (!en.state) return;
    const int lane = x & 63, m = (x >> 6) & 3, it = (x >> 8) % (DK / 32), cb = (x >> 8) / (DK / 32);
    const int row = it * 32 + (m >> 1) * 16 + (lane >> 5) * 8 + (m & 1) * 4;
    const long long e = ((long long)en.slot * a.Hv + h) * DK * a.Dv + (long long)row * a.Dv + cb * 32 +
                        map32(lane & 31);
    f32x4 S;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long at = e + (long long)i * a.Dv;
        if constexpr (ST == RGDR_F32)
            S[i] = static_cast<const float *>(a.pool)[at];
        else if constexpr (ST == RGDR_BF16)
            S[i] = bf16_to_f32(static_cast<const uint16_t *>(a.pool)[at]);
        else
            S[i] = static_cast<float>(static_cast<const int8_t *>(a.pool)[at]) * mx_scale(a.scales[at / kMxBlock]);
    }
    const int last = max(0, (en.L + p.seg_len - 1) / p.seg_len - 1);
    const long long step = (long long)a.B * a.Hv * per;
    f32x4 *ws = reinterpret_cast<f32x4 *>(p.seg_state) + (long long)bh * per + x;
    const float *decay = p.seg_decay + bh;
    constexpr int U = 8;  // segments whose contributions are in flight together
    for (int s0 = 0; s0 < last; s0 += U) {
        f32x4 own[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = min(s0 + u, last - 1);
            own[u] = ws[s * step];
            d[u] = decay[(long long)s * a.B * a.Hv];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u < last) {
                ws[(s0 + u) * step] = S;
                S = S * d[u] + own[u];
            }
    }
    ws[last * step] = S;
}

static int cu_count() {
    static int known[64];  // zero: not asked yet; every writer writes the same number
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 0;
    if (dev >= 0 && dev < 64 && (n = __atomic_load_n(&known[dev], __ATOMIC_RELAXED))) return n;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
    if (dev >= 0 && dev < 64) __atomic_store_n(&known[dev], n, __ATOMIC_RELAXED);
    return n;
}

// How many segments: as many as fill the device's resident workgroups (two on a compute unit, one
// with D_k = 256), of at least two chunks; and whether they pay. With `fill` the share of the
// resident workgroups that the segments take, a chunk of a segment costs about 1.4 + 1.1 fill
// chunks of a call in one pass (both passes over it, two workgroups on a compute unit), and the
// launches and the states 2 + 4 fill. Measured at H = 16/32, D = 128, fp32, one pass against
// segments, us: B=1 T=256 23.3/26.4, T=384 31.7/29.6, T=512 40.0/31.0, T=1024 72/35, T=8192 525/128; B=2
// T=512 41.1/35.6; B=4 T=512 41.8/53.0, T=1024 74.3/78.3, T=4096 271/223; B=5 T=2048 143/154; B=8 T=1024
// 90/130. At D = 64 and 256 what the rule cuts up is faster so too (B=1 T=8192 392/66 and 984/420), but
// some calls that it leaves in one pass would gain (D = 64 B=4 T=1024 54.7/42.8; D = 256 B=1 T=512 74/58).
static bool plan_segments(int B, int H_v, int T, int D_k, int D_v, LaPlan &p, size_t &bytes) {
    bytes = 0;
    p.nseg = 1;
    p.seg_len = T;
    const int cus = cu_count();
    if (cus <= 0) return false;
    const long long tiles = (D_v + kCols - 1) / kCols;
    const long long items = (long long)B * H_v * tiles;
    const long long slots = (long long)cus * (D_k == 256 ? 1 : 2);
    const int chunks = (T + kChunk - 1) / kChunk;
    if (items <= 0) return true;
    const long long most = slots / items < chunks / 2 ? slots / items : chunks / 2;
    if (most < 2) return true;
    const int seg_chunks = (int)((chunks + most - 1) / most);
    const int nseg = (chunks + seg_chunks - 1) / seg_chunks;
    const double fill = (double)items * nseg / slots;
    if (chunks <= seg_chunks * (1.4 + 1.1 * fill) + 2 + 4 * fill) return true;
    p.nseg = nseg;
    p.seg_len = seg_chunks * kChunk;
    const size_t bh = (size_t)B * H_v;
    bytes = (size_t)nseg * bh * (size_t)D_k * D_v * 4 + ((size_t)nseg * bh * 4 + 255) / 256 * 256;
    return true;
}

template <int DK, bool FULL>
static rgdr_status launch_prefill(const LaArgs &a, LaPlan p, hipStream_t stream) {
    p.tiles = (a.Dv + kCols - 1) / kCols;
    const long long units = (long long)a.B * a.Hq * p.nseg, share = (long long)a.group * p.tiles;
    // Units of whole query/key heads leave XCDs idle where there are few of them, and whole rounds of them
    // can be more workgroups than a launch takes; workgroups one by one meet neither, and read q and k
    // into more than one L2. One by one where more than a fifth of the rounds is empty (T=1024, D=128, bf16, heads
    // together / one by one, us: B=1 H=1/128 227/74, B=4 H=1/64 131/82, B=5 131/120, B=12 H=1/32
    // 133/126; with less empty B=13 133/135, B=20 201/207, B=16 H=16/32 154.6/157.7).
    const long long rounds = (units + kXcds - 1) / kXcds * kXcds;  // whole rounds over the XCDs
    const bool even = rounds * 4 <= units * 5 && rounds * share <= kMaxGroups;
    p.per = even ? (int)share : 1;
    const unsigned items = (unsigned)((even ? rounds : units) * share);  // at most kMaxGroups: la_check_sizes
    const dim3 block(256);
    if (p.nseg == 1) {
        hipLaunchKernelGGL((la_chunk_kernel<DK, false, FULL>), dim3(items), block, 0, stream, a, p);
        return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
    }
    const unsigned scan = (unsigned)(((long long)a.B * a.Hv * (a.Dv * DK / 4) + 255) / 256);
    hipLaunchKernelGGL((la_segment_kernel<DK, FULL>), dim3(items), block, 0, stream, a, p);
    if (p.state_dtype == RGDR_F32)
        hipLaunchKernelGGL(la_scan_kernel<RGDR_F32>, dim3(scan), block, 0, stream, a, p, DK);
    else if (p.state_dtype == RGDR_BF16)
        hipLaunchKernelGGL(la_scan_kernel<RGDR_BF16>, dim3(scan), block, 0, stream, a, p, DK);
    else
        hipLaunchKernelGGL(la_scan_kernel<RGDR_MXI8>, dim3(scan), block, 0, stream, a, p, DK);
    hipLaunchKernelGGL((la_chunk_kernel<DK, true, FULL>), dim3(items), block, 0, stream, a, p);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}

template <int DK>
static rgdr_status launch_prefill_dk(const LaArgs &a, const LaPlan &p, hipStream_t stream) {
    return a.Dv % kCols == 0 ? launch_prefill<DK, true>(a, p, stream) : launch_prefill<DK, false>(a, p, stream);
}

}  // namespace rgdr

extern "C" rgdr_status la_prefill_workspace_size(int32_t B, int32_t H_v, int32_t T, int32_t D_k,
                                                 int32_t D_v, size_t *bytes) {
    using namespace rgdr;
    if (!bytes) return RGDR_ERR_NULL;
    if (const rgdr_status st = la_check_sizes(kLaMaxPrompt, B, H_v, T, D_k, D_v)) return st;
    *bytes = 0;
    if (B == 0) return RGDR_OK;
    LaPlan p;
    return plan_segments(B, H_v, T, D_k, D_v, p, *bytes) ? RGDR_OK : RGDR_ERR_HIP;
}

extern "C" rgdr_status la_prefill(const void *query, const la_strides *query_strides,
                                  const void *key, const la_strides *key_strides,
                                  const void *value, const la_strides *value_strides,
                                  const float *g, const la_strides *g_strides,
                                  const void *state_pool, const uint8_t *state_scales,
                                  rgdr_dtype state_dtype, const int32_t *actual_seq_lengths,
                                  const int32_t *ssm_state_indices,
                                  const int32_t *num_accepted_tokens, float scale, int32_t B,
                                  int32_t H_q, int32_t H_v, int32_t T, int32_t D_k, int32_t D_v,
                                  int32_t N_slots, void *out, const la_strides *out_strides,
                                  void *state_out, uint8_t *state_scales_out, void *workspace,
                                  size_t workspace_bytes, hipStream_t stream) {
    using namespace rgdr;
    LaArgs a;
    if (const rgdr_status st = la_check(
            a, kLaMaxPrompt, query, query_strides, key, key_strides, value, value_strides, g,
            g_strides, state_pool, state_scales, state_dtype, actual_seq_lengths,
            ssm_state_indices, num_accepted_tokens, scale, B, H_q, H_v, T, D_k, D_v, N_slots, out,
            out_strides, state_out, state_scales_out))
        return st;
    if (B == 0) return RGDR_OK;
    if (workspace && !aligned(workspace, 256)) return RGDR_ERR_ALIGN;
    LaPlan p = {};
    size_t need = 0;
    if (!plan_segments(B, H_v, T, D_k, D_v, p, need)) return RGDR_ERR_HIP;
    if (!workspace || workspace_bytes < need) {
        p.nseg = 1;
        p.seg_len = T;
    }
    p.state_dtype = state_dtype;
    if (p.nseg > 1) {
        p.seg_state = static_cast<float *>(workspace);
        p.seg_decay = p.seg_state + (size_t)p.nseg * B * H_v * D_k * D_v;
    }
    if (D_k == 64) return launch_prefill_dk<64>(a, p, stream);
    if (D_k == 128) return launch_prefill_dk<128>(a, p, stream);
    return launch_prefill_dk<256>(a, p, stream);
}
