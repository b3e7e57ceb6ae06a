// ssm_prefill.hip -- the selective state space scan over whole prompts.
#include "ssm_common.h"

namespace rgdr {

constexpr int kXcds = 8;        // of the device, each with its own L2
constexpr int kPieces = 256;  // a workgroup's threads: (token, 8 channels) pieces of a chunk

// The sizes that go with WAYS lanes for each channel's states.
template <int N, int WAYS>
struct SsmShape {
    static constexpr int NP = N / WAYS;                // states of a lane
    static constexpr int CW = 64 / WAYS, CH = 4 * CW;  // channels of a wave, of a workgroup
    static constexpr int SHARE = 64 / CH;              // workgroups on a line of 128 bytes (of 16-bit rows)
    static constexpr int TPT = CH / 8, TC = kPieces / TPT;  // threads for each token, tokens of a chunk
    static constexpr int ROW = TC + 4;                 // floats of a channel's row in LDS
    static constexpr int ROWS = CH * ROW + (CH / 8 - 1) * 4;  // rows of 8 channels start 4 floats further
    static constexpr int NV = 2 * N / TPT;             // values of B or C that a thread stages
    static constexpr bool BY_TOKEN = NP >= 4;          // B and C in LDS: [t][n], else [n][t]
    static constexpr int BC = BY_TOKEN ? TC * N : N * ROW;
    static __device__ __forceinline__ int at(int c, int t) { return c * ROW + (c >> 3) * 4 + t; }
    static __device__ __forceinline__ int bc_at(int t, int n) { return BY_TOKEN ? t * N + n : n * ROW + t; }
};

struct SsmPlan {
    int ways, c_blocks;
    bool roles;
    int segs, seg_len;
    float *ends;  // [B][segs][C][N]: a segment's end state from zero, then its incoming state
    float *sums;  // [B][segs][C]: its sum of d
};

enum SsmPass { kSsmWhole, kSsmEnds, kSsmSegment };

// WAYS values of each lane, one for each token; lane l = w CW + c is left with the sum of value w over the
// WAYS lanes of channel c. Each step halves the values: lanes of one half take the first half of them,
// the others the second.
template <int WAYS>
__device__ __forceinline__ float ssm_meet(float (&y)[WAYS]) {
    const auto bits = [](float x) { return __float_as_int(x); };
#pragma unroll
    for (int i = 0; i < WAYS / 2; ++i) {
        const auto r = __builtin_amdgcn_permlane32_swap(bits(y[i]), bits(y[i + WAYS / 2]), false, false);
        y[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
#pragma unroll
    for (int i = 0; i < WAYS / 4; ++i) {
        const auto r = __builtin_amdgcn_permlane16_swap(bits(y[i]), bits(y[i + WAYS / 4]), false, false);
        y[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (WAYS >= 8) {
#pragma unroll
        for (int i = 0; i < WAYS / 8; ++i) {  // lane ^ 8: the first value in lanes without that bit
            const float v = y[i], w = y[i + WAYS / 8];
            y[i] = __int_as_float(__builtin_amdgcn_update_dpp(bits(w), bits(v), 0x128, 0xF, 0x3, false)) +
                   __int_as_float(__builtin_amdgcn_update_dpp(bits(v), bits(w), 0x128, 0xF, 0xC, false));
        }
    }
    if constexpr (WAYS >= 16) {  // lane ^ 4
        const float v = y[0], w = y[1];
        y[0] = __int_as_float(__builtin_amdgcn_update_dpp(bits(w), bits(v), 0x104, 0xF, 0x5, false)) +
               __int_as_float(__builtin_amdgcn_update_dpp(bits(v), bits(w), 0x114, 0xF, 0xA, false));
    }
    return y[0];
}

// The wave's priority by the quarter of the tokens that it still has before it. Of waves alike the oldest
// goes first, so that the last workgroup of a compute unit would run the longer alone, at half of the vector units'
// rate. (This change alone: B=16, T=1024, C=4096 257 us without it and 240 with it, ragged 191 and 183.)
__device__ __forceinline__ void ssm_priority(int now, int &quarter) {
    if (now == quarter) return;
    quarter = now;
    if (now == 3)
        __builtin_amdgcn_s_setprio(3);
    else if (now == 2)
        __builtin_amdgcn_s_setprio(2);
    else if (now == 1)
        __builtin_amdgcn_s_setprio(1);
    else
        __builtin_amdgcn_s_setprio(0);
}

// A workgroup has up to CH channels of one entry and group and works through chunks of TC tokens (of the
// entry, or of one of its segments). What is done once for each token and channel (softplus, d x, the gate) and
// all memory access of them goes by (token, 8 channels) for each thread, whole 16-byte pieces; the states go
// by channel: WAYS lanes hold a channel's N states, so that a lane has N / WAYS of them in registers for all
// tokens. d, d x and the sums over the states pass between the two through LDS, as do B and C in fp32.
//
// A workgroup's four waves do both in turn, and waves of other workgroups fill in: with four on a compute
// unit the vector units are busy for 90 to 97% of the time (B=16, T=1024, C=4096, N=16, bf16: 240 us; ragged
// 164). Where a compute unit has one workgroup at most (ROLES), four waves do the one and four others the other,
// a chunk apart, in two sets of buffers (in one pass, with roles and without: B=1, T=8192, C=512 194 us and 257;
// C=4096 203 and 264; T=300 14.0 and 17.0; with two workgroups there it is the other way round, 443 and 381 for
// C=8192). Workgroups of 16 channels that share lines run on one XCD (C=4096 211 us, and 233 when they go round the
// XCDs, before the first chunk's loads were moved ahead of the barrier).
template <typename E, int N, int WAYS, int PASS, bool ROLES>
__global__ __launch_bounds__(ROLES ? 512 : 256, WAYS == 4 && N <= 16 ? (sizeof(E) == 4 ? 3 : 4) : 2)
void ssm_prefill_kernel(const SsmArgs a, const SsmPlan p, const bool state_f32) {
    using S = SsmShape<N, WAYS>;
    constexpr int NP = S::NP, TC = S::TC;
    constexpr int SETS = ROLES ? 2 : 1;
    __shared__ __align__(16) float sd[SETS][S::ROWS], su[SETS][S::ROWS];
    __shared__ __align__(16) float sB[SETS][S::BC], sC[SETS][S::BC];
    __shared__ __align__(16) float s_bias[S::CH], s_D[S::CH];
    const int role = ROLES ? __builtin_amdgcn_readfirstlane(threadIdx.x / 256) : 0;
    const int tid = ROLES ? threadIdx.x % 256 : threadIdx.x;
    const bool by_channel = !ROLES || role == 0, by_token = !ROLES || role == 1;
    int item = blockIdx.x;
    if constexpr (S::SHARE > 1) {  // workgroups that share lines run on one XCD, and meet in its L2
        const int local = item / kXcds;
        item = (local / S::SHARE * kXcds + item % kXcds) * S::SHARE + local % S::SHARE;
        if (item >= p.c_blocks * a.B) return;
    }
    const int cb = item % p.c_blocks, s = item / p.c_blocks % p.segs;
    const int b = entry_of_rank(a.lens, a.B, a.T, item / p.c_blocks / p.segs);
    const LaEntry e = ssm_entry(a, b);
    const int t_begin = s * p.seg_len, t_end = min(e.L, t_begin + p.seg_len);
    if (PASS == kSsmEnds && t_begin + p.seg_len >= e.L) return;

    // by token and 8 channels: a uniform address, which moves on by chunks, and a thread's own 32-bit offset
    // (127 tokens at strides of at most 2^25 bytes)
    const int st = tid / S::TPT, sc = tid % S::TPT * 8;
    const int Cg = a.C / a.G, per = (Cg - 1) / S::CH + 1, g = cb / per;  // this workgroup's group,
    const int c0 = g * Cg + cb % per * S::CH, channels = min(S::CH, Cg - cb % per * S::CH);  // and channels
    const int cs = c0 + sc;
    const bool c_ok = sc < channels;
    const auto first = [&](const void *p, const LaStrides &s) {
        return static_cast<const char *>(p) + (b * s.b + t_begin * s.t) * (long long)sizeof(E);
    };
    const auto step = [&](const LaStrides &s) { return (uint32_t)s.t * (uint32_t)sizeof(E); };  // a token's bytes
    const uint32_t dx = step(a.sx), ddt = step(a.sdt), dz = step(a.sz), dB = step(a.sB), dC = step(a.sC);
    const char *px = first(a.x, a.sx) + c0 * sizeof(E), *pdt = first(a.dt, a.sdt) + c0 * sizeof(E);
    const char *pz = first(a.z, a.sz) + c0 * sizeof(E);
    const char *pB = first(a.Bm, a.sB) + g * a.sB.h * sizeof(E), *pC = first(a.Cm, a.sC) + g * a.sC.h * sizeof(E);
    E *pout = static_cast<E *>(a.out) + b * a.so.b + cs;
    if (PASS != kSsmEnds && c_ok && by_token) {
        const float none[8] = {};
        for (int t = max(e.L, t_begin); t < min(a.T, t_begin + p.seg_len) - st; t += TC)
            row_put(pout + (t + st) * a.so.t, none);
    }

    // by channel and a part of its states
    const int q = tid % 64 / S::CW, c = tid / 64 * S::CW + tid % S::CW, cc = c0 + c;
    const bool mine = c < channels;
    const size_t slot_at = ((size_t)(e.state ? e.slot : 0) * a.C + cc) * N + q * NP;
    const size_t seg_at = ((size_t)(b * p.segs + s) * a.C + cc) * N + q * NP;
    const auto commit = [&](const float (&h)[NP]) {
        if (!mine) return;
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
    for (int i = 0; i < NP; ++i) h[i] = A[i] = 0.f;
    if (mine && e.state && by_channel) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            A[i] = ssm_log2_decay(a.A[(size_t)cc * N + q * NP + i]);
            if (PASS == kSsmWhole)
                h[i] = state_f32 ? static_cast<const float *>(a.pool)[slot_at + i]
                                 : bf16_to_f32(static_cast<const uint16_t *>(a.pool)[slot_at + i]);
            if (PASS == kSsmSegment && t_begin < max(e.L, 1)) h[i] = p.ends[seg_at + i];
        }
    }
    if (PASS != kSsmEnds && s == 0 && e.state && e.n == 0 && !a.in_place && by_channel) commit(h);

    Row<E, 8> nx, dt, nz;
    nx.zero();
    dt.zero();
    nz.zero();
    Row<E, S::NV> bc;
    bc.zero();
    const bool is_C = tid % S::TPT >= S::TPT / 2;
    const int col = tid % (S::TPT / 2) * S::NV;
    // (a thread without a token or channels keeps what it has: it is masked, or never stored)
    const auto load = [&](int left) {
        if (st >= left) return;
        const auto at = [](const char *p, uint32_t offset) { return reinterpret_cast<const E *>(p + offset); };
        const uint32_t o = sc * (uint32_t)sizeof(E);
        if (c_ok) {
            nx.load(at(px, st * dx + o));
            dt.load(at(pdt, st * ddt + o));
            if (PASS != kSsmEnds && a.z) nz.load(at(pz, st * dz + o));
        }
        if (!is_C)
            bc.load(at(pB, st * dB + col * (uint32_t)sizeof(E)));
        else if (PASS != kSsmEnds)
            bc.load(at(pC, st * dC + col * (uint32_t)sizeof(E)));
    };
    Row<float, 8> bias0, D0;
    bias0.zero();
    D0.zero();
    if (st == 0 && by_token && c_ok) {
        if (a.dt_bias) bias0.load(a.dt_bias + cs);
        if (a.D) D0.load(a.D + cs);
    }
    if (by_token) load(t_end - t_begin);  // on its way before the barrier
    if (st == 0 && by_token) {
        bias0.store(s_bias + sc);
        D0.store(s_D + sc);
    }
    __syncthreads();
    // The chunk of nt tokens that was loaded last into LDS.
    const auto stage = [&](int set, int nt) {
        const bool live = st < nt;
        float d[8], u[8], f[S::NV];
        Row<float, 8> bias;
        bias.load(s_bias + sc);
        if (a.softplus) {
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = ssm_softplus(dt.get(i) + bias.get(i));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = dt.get(i) + bias.get(i);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = d[i] * nx.get(i);
#pragma unroll
        for (int i = 0; i < S::NV; ++i) f[i] = bc.get(i);
        if (nt < TC) {  // tokens past the chunk's end leave the state as it is
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[i] = live ? d[i] : 0.f;
                u[i] = live ? u[i] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < S::NV; ++i) f[i] = live ? f[i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sd[set][S::at(sc + i, st)] = d[i];
            su[set][S::at(sc + i, st)] = u[i];
        }
        float *to = (is_C ? sC[set] : sB[set]) + S::bc_at(st, col);
#pragma unroll
        for (int i = 0; i < S::NV; ++i) to[S::bc_at(0, i)] = f[i];
    };
    const auto advance = [&](int nt) {  // (up to 128 tokens of 2^25 bytes: 2^32)
        px += (size_t)nt * dx;
        pdt += (size_t)nt * ddt;
        pz += (size_t)nt * dz;
        pB += (size_t)nt * dB;
        pC += (size_t)nt * dC;
    };
    float sum = 0.f;
    // The states over nt tokens; the sums over the states take the place of d x.
    const auto scan = [&](int set, int nt) {
        const float *d_row = sd[set] + S::at(c, 0);
        const float *tB = sB[set] + S::bc_at(0, q * NP), *tC = sC[set] + S::bc_at(0, q * NP);
        float *u_row = su[set] + S::at(c, 0);
        float part = 0.f;
        if constexpr (WAYS == 4) {
            // LDS reads go ahead: d and d x by four tokens, B and C by two
            f32x4 d4[2], u4[2];
            float B[4][NP], C[4][NP];
            const auto read = [&](int t) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    B[t % 4][i] = tB[S::bc_at(t, i)];
                    if (PASS != kSsmEnds) C[t % 4][i] = tC[S::bc_at(t, i)];
                }
            };
            d4[0] = *reinterpret_cast<const f32x4 *>(d_row);
            u4[0] = *reinterpret_cast<const f32x4 *>(u_row);
            read(0);
            read(1);
#pragma unroll
            for (int t = 0; t < TC; t += 4) {
                if (t >= nt) break;
                float y[4];
                const int now = t / 4 % 2;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (t + j + 2 < TC) read(t + j + 2);
                    if (j == 0 && t + 4 < TC) {
                        d4[1 - now] = *reinterpret_cast<const f32x4 *>(d_row + t + 4);
                        u4[1 - now] = *reinterpret_cast<const f32x4 *>(u_row + t + 4);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    y[j] = 0.f;
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(d4[now][j] * A[i]), h[i],
                                              u4[now][j] * B[(t + j) % 4][i]);
                        if (PASS != kSsmEnds) y[j] = __builtin_fmaf(C[(t + j) % 4][i], h[i], y[j]);
                    }
                }
                if (PASS == kSsmEnds)
                    part += (d4[now][0] + d4[now][1]) + (d4[now][2] + d4[now][3]);
                else
                    u_row[t + q] = ssm_meet<4>(y);
            }
        } else {
#pragma unroll
            for (int t = 0; t < TC; t += WAYS) {
                if (t >= nt) break;
                float d[WAYS], u[WAYS], B[WAYS][NP], C[WAYS][NP], y[WAYS];
#pragma unroll
                for (int k = 0; k < WAYS; k += 4) {
                    *reinterpret_cast<f32x4 *>(d + k) = *reinterpret_cast<const f32x4 *>(d_row + t + k);
                    *reinterpret_cast<f32x4 *>(u + k) = *reinterpret_cast<const f32x4 *>(u_row + t + k);
                }
#pragma unroll
                for (int i = 0; i < NP; ++i) {
#pragma unroll
                    for (int j = 0; j < WAYS; ++j) {
                        B[j][i] = tB[S::bc_at(t + j, i)];
                        C[j][i] = tC[S::bc_at(t + j, i)];
                    }
                }
#pragma unroll
                for (int j = 0; j < WAYS; ++j) {
                    y[j] = 0.f;
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(d[j] * A[i]), h[i], u[j] * B[j][i]);
                        y[j] = __builtin_fmaf(C[j][i], h[i], y[j]);
                    }
                }
                u_row[t + q] = ssm_meet<WAYS>(y);
            }
        }
        sum += part;
    };
    // The outputs of nt tokens from t0 on.
    const auto finish = [&](int set, int t0, int nt, const Row<E, 8> &x, const Row<E, 8> &z) {
        if (PASS == kSsmEnds || st >= nt || !c_ok) return;
        float y[8];
        Row<float, 8> D;
        D.load(s_D + sc);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = ssm_out(su[set][S::at(sc + i, st)], D.get(i), x.get(i), a.z != nullptr, z.get(i));
        row_put(pout + (t0 + st) * a.so.t, y);
    };
    // (the accepted tokens end a chunk, so that the state after them is the one at its end)
    const auto tokens = [&](int t0) { return min(min(TC, t_end - t0), t0 < e.n ? e.n - t0 : TC); };

    int quarter = -1;
    if constexpr (!ROLES) {
        for (int t0 = t_begin; t0 < t_end;) {
            const int nt = tokens(t0);
            ssm_priority((int)((t_end - t0) * 4LL / (p.seg_len + 1)), quarter);
            stage(0, nt);
            const Row<E, 8> x = nx, z = nz;
            __syncthreads();
            advance(nt);
            load(t_end - t0 - nt);
            scan(0, nt);
            if (PASS != kSsmEnds && t0 + nt == e.n) commit(h);
            __syncthreads();
            finish(0, t0, nt, x, z);  // each thread's own place in LDS, which it alone stages next
            t0 += nt;
        }
    } else if (t_begin < t_end) {
        // While one role scans a chunk, the other finishes the one before it and stages the one behind it, in
        // the same buffers: a thread reads and writes its own place there.
        Row<E, 8> x = nx, z = nz, x1 = nx, z1 = nz;  // of the chunk before, and of the one being scanned
        int nt = tokens(t_begin), nt_before = 0, set = 0;
        if (by_token) {
            stage(0, nt);
            x1 = nx;
            z1 = nz;
            advance(nt);
            load(t_end - t_begin - nt);
        }
        __syncthreads();
        for (int t0 = t_begin; t0 < t_end; set ^= 1) {
            const int next = t0 + nt, nt_next = next < t_end ? tokens(next) : 0;
            if (by_channel) {
                ssm_priority((int)((t_end - t0) * 4LL / (p.seg_len + 1)), quarter);
                scan(set, nt);
                if (next == e.n) commit(h);
            } else {
                if (nt_before) finish(set ^ 1, t0 - nt_before, nt_before, x, z);
                x = x1;
                z = z1;
                if (nt_next) {
                    stage(set ^ 1, nt_next);
                    x1 = nx;
                    z1 = nz;
                    advance(nt_next);
                    load(t_end - next - nt_next);
                }
            }
            __syncthreads();
            t0 = next;
            nt_before = nt;
            nt = nt_next;
        }
        if (by_token) finish(set ^ 1, t_end - nt_before, nt_before, x, z);
    }
    if (PASS == kSsmEnds && mine) {
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
    const int last = max(1, (e.L + p.seg_len - 1) / p.seg_len) - 1;
    const size_t slot_at = ((size_t)e.slot * a.C + c) * N + n0, step = (size_t)a.C * N;
    f32x4 *ends = reinterpret_cast<f32x4 *>(p.ends + ((size_t)b * p.segs * a.C + c) * N + n0);
    const float *sums = p.sums + (size_t)b * p.segs * a.C + c;
    float h[4], A[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[k] = state_f32 ? static_cast<const float *>(a.pool)[slot_at + k]
                         : bf16_to_f32(static_cast<const uint16_t *>(a.pool)[slot_at + k]);
        A[k] = ssm_log2_decay(a.A[(size_t)c * N + n0 + k]);
    }
    constexpr int U = 8;  // loads in flight
    for (int s0 = 0; s0 < last; s0 += U) {
        f32x4 end[U];
        float sum[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int s = min(s0 + k, last - 1);
            end[k] = ends[s * step / 4];
            sum[k] = sums[(size_t)s * a.C];
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (s0 + k >= last) break;
            ends[(s0 + k) * step / 4] = f32x4{h[0], h[1], h[2], h[3]};
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(sum[k] * A[i]), h[i], end[k][i]);
        }
    }
    ends[last * step / 4] = f32x4{h[0], h[1], h[2], h[3]};
}

// The workgroups of a launch: with more than four lanes for a channel, whole rounds of the XCDs of those that
// share lines.
static long long ssm_groups(const SsmPlan &p, int B) {
    const long long round = p.ways > 4 ? (long long)p.ways / 4 * kXcds : 1;
    const __int128 n = (__int128)p.c_blocks * p.segs * B;
    return n > kMaxGroups ? kMaxGroups + 1 : ((long long)n + round - 1) / round * round;
}

template <typename E, int N, int WAYS, int PASS, bool ROLES = false>
static rgdr_status launch_ssm_pass(const SsmArgs &a, const SsmPlan &p, bool f32, hipStream_t stream) {
    const long long groups = ssm_groups(p, a.B);
    if (groups > kMaxGroups) return RGDR_ERR_SHAPE;
    hipLaunchKernelGGL((ssm_prefill_kernel<E, N, WAYS, PASS, ROLES>), dim3((unsigned)groups), dim3(ROLES ? 512 : 256), 0,
                       stream, a, p, f32);
    return hipGetLastError() == hipSuccess ? RGDR_OK : RGDR_ERR_HIP;
}

template <typename E, int N>
static rgdr_status launch_ssm_prefill(const SsmArgs &a, const SsmPlan &p, bool f32, hipStream_t stream) {
    constexpr int MOST = N < 16 ? N : 16;
    if (p.ways == MOST && p.roles) return launch_ssm_pass<E, N, MOST, kSsmWhole, true>(a, p, f32, stream);
    if (p.ways == MOST) return launch_ssm_pass<E, N, MOST, kSsmWhole>(a, p, f32, stream);
    if (p.segs == 1) return launch_ssm_pass<E, N, 4, kSsmWhole>(a, p, f32, stream);
    const long long threads = (long long)a.B * a.C * (N / 4), blocks = (threads + 255) / 256;
    if (blocks > kMaxGroups) return RGDR_ERR_SHAPE;
    rgdr_status rc = launch_ssm_pass<E, N, 4, kSsmEnds>(a, p, f32, stream);
    if (rc != RGDR_OK) return rc;
    hipLaunchKernelGGL(ssm_ends_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a, p, N, f32);
    if (hipGetLastError() != hipSuccess) return RGDR_ERR_HIP;
    return launch_ssm_pass<E, N, 4, kSsmSegment>(a, p, f32, stream);
}

template <typename E>
static rgdr_status launch_ssm_states(const SsmArgs &a, const SsmPlan &p, int N, bool f32, hipStream_t stream) {
    if (N == 8) return launch_ssm_prefill<E, 8>(a, p, f32, stream);
    if (N == 16) return launch_ssm_prefill<E, 16>(a, p, f32, stream);
    return launch_ssm_prefill<E, 32>(a, p, f32, stream);
}

// The plan of a call in `ways` lanes for each channel and segments of seg_len tokens.
static SsmPlan ssm_plan_of(int ways, int seg_len, int T, int C, int G) {
    SsmPlan p;
    const int CH = 256 / ways;
    p.ways = ways;
    p.c_blocks = G * ((C / G - 1) / CH + 1);
    p.seg_len = seg_len;
    p.segs = (T + seg_len - 1) / seg_len;
    p.roles = false;
    p.ends = p.sums = nullptr;
    return p;
}

// What a token takes a workgroup in ns: alone on its compute unit (in roles), and each of several there.
struct SsmRates {
    double alone, roles, beside;
};

// How many lanes for each channel, and how many segments: what costs least by the model below, in ns. A chunk's
// tokens take a workgroup alone on its compute unit 97 ns each with four lanes for each channel and 30 with 16,
// or 26 with roles; the vector units allow 58 for each workgroup there with four lanes, the LDS 20 with 16 (a
// quarter of the channels); the last workgroup is alone for a while. Of a segment's two passes the first takes
// three quarters of the second; they and the scan between them are three launches. Those are N = 16's rates; N = 32
// takes 5 / 3 of them. N = 8 has its own, for its wider form is one of eight lanes with half of the channels and a
// state each: 72 and 42 with four lanes, 39, 32 and 22.5 with eight; in fp32, where a compute unit holds
// fewer workgroups of four lanes, 63 in place of 42, and 30 of 22.5.
// bf16, us, 4 lanes / 16 lanes / 4 lanes in segments (of tokens): B=1, C=4096, T=8192 751/203/220 (512);
// C=8192 760/367/416 (256); C=512 758/194/52 (128); C=2048, T=2048 192/55/44 (128); B=2, T=300, C=4096
// 33/19/30 (64); B=4, T=1024 100/80/108 (256); B=8 137/159; B=16 240/338/375 (256); B=3, C=1448 (273
// workgroups of 16 lanes for each channel), T=6801 628/294/204 (512).
// N=32: B=16, T=1024, C=4096 427/565; B=4 150/138/194 (256); B=1, T=8192 1149/323/378 (512); C=512 1152/315/75 (128).
// N=8, 4 lanes / 8 lanes / segments: B=16, T=1024, C=4096 184/197 (fp32 274/248); B=8 105/93; B=4 78/57/78 (256);
// B=64, T=300, C=1024 56/71 (fp32 87/78); B=1, T=8192, C=4096 585/263/158 (512); C=512 582/249/43 (128).
// The segments go by 16-bit rows' rates, so that the workspace's size does not depend on the type. A form whose
// workgroups are more than a launch may have is no candidate.
static SsmPlan ssm_plan(int B, int T, int C, int N, int G, bool f32, bool one_pass, int cus) {
    const int most = N < 16 ? N : 16;
    const double size = N == 8 ? 1 : (8.0 + N) / 24;  // of a token's work, against N = 16
    const auto wide = [&](bool f32) {
        return N == 8 ? SsmRates{39, 32, f32 ? 30 : 22.5} : SsmRates{30, 26, 20};
    };
    const auto four = [&](bool f32) { return N == 8 ? SsmRates{72, 0, f32 ? 63.0 : 42.0} : SsmRates{97, 0, 58}; };
    const SsmRates parts = N == 8 ? SsmRates{126, 0, 73.5} : SsmRates{97 + 75, 0, 58 + 44};
    const auto cost = [&](const SsmPlan &p, const SsmRates &r) {
        const long long groups = (long long)p.c_blocks * B * p.segs;
        // workgroups for each compute unit; of few, those of the unit that has the most
        const double here = groups < 8LL * cus ? (double)((groups + cus - 1) / cus) : (double)groups / cus;
        const double alone = p.roles ? r.roles : r.alone, token = here * r.beside + (alone - r.beside) / 2;
        return size * p.seg_len * (token > alone ? token : alone);
    };
    SsmPlan in_wide = ssm_plan_of(most, T, T, C, G);
    in_wide.roles = (long long)in_wide.c_blocks * B <= cus && T > 8 * most;  // (one chunk has nothing to overlap)
    const SsmPlan in_four = ssm_plan_of(4, T, T, C, G);
    const bool fits = ssm_groups(in_wide, B) <= kMaxGroups;
    SsmPlan best = fits && cost(in_wide, wide(f32)) <= cost(in_four, four(f32)) ? in_wide : in_four;
    double least = cost(in_four, four(false));
    if (fits && cost(in_wide, wide(false)) < least) least = cost(in_wide, wide(false));
    for (int len = 64; !one_pass && len * 2 <= T; len *= 2) {
        const SsmPlan p = ssm_plan_of(4, len, T, C, G);
        const double c = cost(p, parts) + 4000 + 250.0 * p.segs;
        if (c < least && ssm_groups(p, B) <= kMaxGroups) {
            best = p;
            least = c;
        }
    }
    return best;
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
    *bytes = 0;
    if (B == 0) return RGDR_OK;
    const int cus = la_compute_units();
    if (cus == 0) return RGDR_ERR_HIP;
    *bytes = ssm_workspace(ssm_plan(B, T, C, N, G, false, false, cus), B, C, N);
    return RGDR_OK;
}

// The form that a call of these sizes (with rows of fp32, or of 16 bits) takes on `cus` compute units, for tests:
// lanes for each channel, whether in roles, segments, tokens of a segment.
extern "C" rgdr_status ssm_prefill_form(int32_t B, int32_t T, int32_t C, int32_t N, int32_t G, int32_t f32,
                                        int32_t one_pass, int32_t cus, int32_t form[4]) {
    using namespace rgdr;
    const rgdr_status rc = ssm_check_sizes(65536, B, T, C, N, G);
    if (rc != RGDR_OK) return rc;
    if (B < 1 || cus < 1) return RGDR_ERR_SHAPE;
    const SsmPlan p = ssm_plan(B, T, C, N, G, f32 != 0, one_pass != 0, cus);
    form[0] = p.ways;
    form[1] = p.roles;
    form[2] = p.segs;
    form[3] = p.seg_len;
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
    if (ssm_groups(ssm_plan_of(4, T, T, C, G), B) > kMaxGroups) return RGDR_ERR_SHAPE;
    const int cus = la_compute_units();
    if (cus == 0) return RGDR_ERR_HIP;
    const bool wide_rows = dtype == RGDR_F32;
    SsmPlan p = ssm_plan(B, T, C, N, G, wide_rows, false, cus);
    if (!workspace || workspace_bytes < ssm_workspace(p, B, C, N)) p = ssm_plan(B, T, C, N, G, wide_rows, true, cus);
    if (p.segs > 1) {
        p.ends = static_cast<float *>(workspace);
        p.sums = p.ends + (size_t)B * p.segs * C * N;
    }
    const bool f32 = state_dtype == RGDR_F32;
    if (dtype == RGDR_F32) return launch_ssm_states<float>(a, p, N, f32, stream);
    if (dtype == RGDR_F16) return launch_ssm_states<_Float16>(a, p, N, f32, stream);
    return launch_ssm_states<uint16_t>(a, p, N, f32, stream);
}
