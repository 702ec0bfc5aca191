// The selective state space scan: forward and the single-token step, and what
// the forward shares with the backward pass (seq_scan_backward.cu).
//
//   dt = softplus(delta + bias),  h_t = e^(dt A) h_(t-1) + dt u B_t,
//   o_t = C_t h_t + D u,  y_t = o_t silu(z_t)
//
// Bound: an exponential, a product and three FMAs per state and position
// against 8 bytes per position and channel for 16-bit types, so with 16 states
// the exponentials and the instruction issue bound it, not the memory.
#include <utility>

#include "seq_scan.cuh"

namespace spconv {
namespace seq {
namespace {

// Tiling.  A lane holds SPT states of each of two channels, LPC lanes hold a
// channel, so a position's 2 * SPT values of B and C, read from shared memory,
// serve two channels, and its step sizes, two per channel, SPT states.  A
// broadcast read costs a 4-byte word per lane like any other, and a lane's
// 2 * (2 * SPT) + 4 words per 2 * SPT updates are what shared memory can deliver
// about as fast as the exponentials (32 a clock on an SM) can use them: one channel
// and four states per lane read 2.5 words per update and took 375 us on 4 x
// 4096 channels x 2048 positions x 16 states in bf16.
// A block is one warp: its 64 / LPC channels give as many blocks as there are.
template <typename T, int SPT_, int LPC_>
struct ScanTile {
    static constexpr int SPT = SPT_, LPC = LPC_, SP = SPT * LPC;
    static constexpr int VE = 16 / sizeof(T), TT = 4 * VE;  // positions of a lane's load, of a tile
    static constexpr int PAIRS = 32 / LPC, CW = 2 * PAIRS;  // pairs of channels, channels
    static constexpr int NI = CW * 4 / 32;                  // loads of a lane from each row set
    static constexpr int NB = 2 * SP * 4 / 32;              // from B and C
    // in rows of 16 bytes {dt, dt u} of a pair's channels: one more after every
    // VE positions, and 2 modulo 8, so that neither the lanes that write nor the
    // pairs that read meet in the same banks
    static constexpr int kStepPitch = TT + 10;
    static constexpr int kOutPitch = TT + 4;
    static constexpr int kOutHalf = PAIRS * kOutPitch + 16;  // from the pairs' first channels to
                                                             // their second
    static constexpr int kSteps = PAIRS * kStepPitch * 4;    // floats
    // rows of B and of C: one more after every VE positions here too, and two
    // that are read ahead
    static constexpr int kMatrix = (TT + 6) * SP;
    static constexpr int kBC = 2 * kMatrix;
    static constexpr int kOut = 2 * kOutHalf;
    static constexpr bool kAhead = NB <= 4;  // B and C of the next tile wait in registers
};

// One pass over a chunk of positions with the states in registers.
// ENDS: from zero states, only what the chunk leaves and the sum of its step
// sizes.  Otherwise the outputs.
template <typename T, int SPT, int LPC, bool ENDS>
__global__ void __launch_bounds__(32) scan_kernel(const ScanParams p) {
    using G = ScanTile<T, SPT, LPC>;
    constexpr int VE = G::VE, TT = G::TT, SP = G::SP, NP = Pairs<SPT>::N, NI = G::NI, NB = G::NB;
    __shared__ __align__(16) float steps[G::kSteps];
    __shared__ __align__(16) float bc[G::kBC];       // [B, C][row of TT + 6][SP]
    __shared__ __align__(16) float outs[ENDS ? 4 : G::kOut];
    const int lane = threadIdx.x;
    // as owner of states: pair of channels, lane of the pair
    const int pair = lane / LPC, j = lane % LPC, s0 = j * SPT;
    // as owner of positions: VE * quarter .. of channels lane / 4 + 8 k
    const int quarter = lane & 3, t_mine = quarter * VE;

    const int n = blockIdx.y, chunk = blockIdx.z;
    const int g = blockIdx.x / p.blocks_per_group;
    const int c_first = (blockIdx.x - g * p.blocks_per_group) * G::CW;  // within the group
    const int c_count = min(G::CW, p.per_group - c_first);
    const int64_t c_base = (int64_t)g * p.per_group + c_first;
    const int len = p.lengths ? min(max(p.lengths[n], 0), p.L) : p.L;
    const int first = chunk * p.chunk_len, stop = first + min(p.L - first, p.chunk_len);
    const int end = max(min(len, stop), first);
    const int64_t rows = (int64_t)n * p.channels + c_base;
    const int64_t chunk_rows = ((int64_t)n * p.chunks + chunk) * p.channels + c_base;
    const T *ub = static_cast<const T *>(p.u) + n * p.u_sn + c_base * p.u_sc;
    const T *db = static_cast<const T *>(p.delta) + n * p.d_sn + c_base * p.d_sc;
    const T *zb = !ENDS && p.z ? static_cast<const T *>(p.z) + n * p.z_sn + c_base * p.z_sc
                               : nullptr;
    const T *Bb = static_cast<const T *>(p.B) + n * p.b_sn + g * p.b_sg;
    const T *Cb = static_cast<const T *>(p.C) + n * p.c_sn + g * p.c_sg;

    Pairs<SPT> A[2], h[2];
    int mine[2];  // the pair's channels in the block
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        mine[k] = pair + k * G::PAIRS;
        const int S = mine[k] < c_count ? p.S : 0;
        A[k].load(p.A + (c_base + mine[k]) * p.S, s0, S);
        A[k].scale(kLog2e);
        if (ENDS)
            h[k].fill(0.f);
        else if (p.chunks > 1)
            h[k].load(p.h_chunk + (chunk_rows + mine[k]) * p.S, s0, S);
        else if (p.state)
            h[k].load(p.state + (rows + mine[k]) * p.S, s0, S);
        else
            h[k].fill(0.f);
    }
    float bias[NI], D[NI], total[NI];
    int row_end[NI];
#pragma unroll
    for (int k = 0; k < NI; ++k) {
        const int c = lane / 4 + 8 * k;
        row_end[k] = c < c_count ? end : 0;
        bias[k] = p.delta_bias && c < c_count ? p.delta_bias[c_base + c] : 0.f;
        D[k] = p.D && c < c_count ? p.D[c_base + c] : 0.f;
        total[k] = 0.f;
    }

    Run<T, VE> u[NI], un[NI], dn[NI], z[NI], bcn[NB];
    auto fetch_bc = [&](int t0) {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = lane + 32 * k, s = i % SP, q = (i / SP) % 4, which = i / (SP * 4);
            if (ENDS && which) continue;
            const T *row = which ? Cb + s * p.c_ss : Bb + s * p.b_ss;
            load_run(bcn[k], row, t0 + q * VE, s < p.S ? end : 0, p.vec);
        }
    };
    auto fetch = [&](int t0) {
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            const int c = lane / 4 + 8 * k;
            load_run(dn[k], db + c * p.d_sc, t0 + t_mine, row_end[k], p.vec);
            load_run(un[k], ub + c * p.u_sc, t0 + t_mine, row_end[k], p.vec);
        }
        if (G::kAhead) fetch_bc(t0);
    };
    if (first < end) fetch(first);
    for (int t0 = first; t0 < end; t0 += TT) {
        if (!G::kAhead) fetch_bc(t0);
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = lane + 32 * k, s = i % SP, q = (i / SP) % 4, which = i / (SP * 4);
            if (ENDS && which) continue;
            float *to = bc + which * G::kMatrix + q * (VE + 1) * SP + s;
#pragma unroll
            for (int e = 0; e < VE; ++e) to[e * SP] = bcn[k][e];
        }
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            const int c = lane / 4 + 8 * k;
            float2 *to = reinterpret_cast<float2 *>(steps) +
                         ((c % G::PAIRS) * G::kStepPitch + quarter * (VE + 1)) * 2 + c / G::PAIRS;
            u[k] = un[k];
            float dt[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) dt[e] = dn[k][e] + bias[k];
            if (p.softplus) {
#pragma unroll
                for (int e = 0; e < VE; ++e) dt[e] = softplus(dt[e]);
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                to[2 * e] = make_float2(dt[e], dt[e] * u[k][e]);
                if (ENDS) total[k] += t0 + t_mine + e < row_end[k] ? dt[e] : 0.f;
            }
        }
        if (t0 + TT > end || c_count < G::CW) {
            // behind the end a step of size zero leaves the states as they are
            __syncwarp();
            for (int i = lane; i < G::CW * TT; i += 32) {
                const int c = i / TT, t = i % TT;
                if (t0 + t >= end || c >= c_count)
                    reinterpret_cast<float2 *>(steps)[((c % G::PAIRS) * G::kStepPitch + t + t / VE) * 2 +
                                                      c / G::PAIRS] = make_float2(0.f, 0.f);
            }
        }
        __syncwarp();
        if (t0 + TT < end) fetch(t0 + TT);
        if (!ENDS && zb) {
#pragma unroll
            for (int k = 0; k < NI; ++k)
                load_run(z[k], zb + (lane / 4 + 8 * k) * p.z_sc, t0 + t_mine, row_end[k], p.vec);
        }
        const float4 *step = reinterpret_cast<const float4 *>(steps) + pair * G::kStepPitch;
        // Two positions ahead of the states, what a position needs is read; one
        // ahead, its decays and inputs are formed: a warp has few neighbours to
        // hide a latency behind.  (Behind the tile's last position lie rows that
        // are read and not used.)
        float4 xn = step[0];
        Pairs<SPT> bn, cn, c1;
        bn.read(bc + s0);
        if (!ENDS) cn.read(bc + G::kMatrix + s0);
        f32x2 a1[2][NP], b1[2][NP];
        auto advance = [&](int r) {  // forms the position that was read, reads row r
            const f32x2 dt[2] = {pack2(xn.x, xn.x), pack2(xn.z, xn.z)};
            const f32x2 du[2] = {pack2(xn.y, xn.y), pack2(xn.w, xn.w)};
#pragma unroll
            for (int i = 0; i < NP; ++i) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    a1[q][i] = ex2_2(mul2(dt[q], A[q].v[i]));
                    b1[q][i] = mul2(du[q], bn.v[i]);
                }
            }
            c1 = cn;
            xn = step[r];
            bn.read(bc + r * SP + s0);
            if (!ENDS) cn.read(bc + G::kMatrix + r * SP + s0);
        };
        advance(1);
#pragma unroll 1
        for (int t = 0; t < TT; t += 4) {
            float out[4][2];
            const int r0 = t + t / VE, r4 = t + 4 + (t + 4) / VE;  // rows of t and t + 4
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f32x2 y[2];
#pragma unroll
                for (int i = 0; i < NP; ++i) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        h[q].v[i] = fma2(a1[q][i], h[q].v[i], b1[q][i]);
                        if (!ENDS) y[q] = i ? fma2(h[q].v[i], c1.v[i], y[q]) : mul2(h[q].v[i], c1.v[i]);
                    }
                }
                advance(k < 2 ? r0 + k + 2 : r4 + k - 2);
                if (!ENDS) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float2 f = unpack2(y[q]);
                        out[k][q] = f.x + f.y;
                    }
                }
            }
            if (!ENDS) {
                // even lanes keep the pair's first channel, odd lanes the second
                float w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = (j & 1 ? out[k][1] : out[k][0]) +
                           __shfl_xor_sync(~0u, j & 1 ? out[k][0] : out[k][1], 1);
                if (LPC == 4) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] += __shfl_xor_sync(~0u, w[k], 2);
                }
                if (j < 2)
                    *reinterpret_cast<float4 *>(outs + j * G::kOutHalf + pair * G::kOutPitch + t) =
                        make_float4(w[0], w[1], w[2], w[3]);
            }
        }
        __syncwarp();
        if constexpr (!ENDS) {
#pragma unroll
            for (int k = 0; k < NI; ++k) {
                const int c = lane / 4 + 8 * k;
                const float4 *q = reinterpret_cast<const float4 *>(
                    outs + c / G::PAIRS * G::kOutHalf + c % G::PAIRS * G::kOutPitch + t_mine);
                float o[VE];
#pragma unroll
                for (int e = 0; e < VE; e += 4) {
                    const float4 f = q[e / 4];
                    const float y[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[e + i] = fmaf(D[k], u[k][e + i], y[i]);
                }
                if (zb) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) o[e] *= silu(z[k][e]);
                }
                if (t0 + TT > end)
#pragma unroll
                    for (int e = 0; e < VE; ++e) o[e] = t0 + t_mine + e < end ? o[e] : 0.f;
                Run<T, VE> out;
                out.put(o);
                if (c < c_count)
                    store_run(out, static_cast<T *>(p.y) + (rows + c) * p.L, t0 + t_mine, stop, p.vec_y);
            }
        }
    }
    if (ENDS) {
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            total[k] += __shfl_xor_sync(~0u, total[k], 1);
            total[k] += __shfl_xor_sync(~0u, total[k], 2);
            const int c = lane / 4 + 8 * k;
            if (quarter == 0 && c < c_count) p.dt_chunk[chunk_rows + c] = total[k];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (mine[k] < c_count) h[k].store(p.h_chunk + (chunk_rows + mine[k]) * p.S, s0, p.S);
        return;
    }
    // positions of the chunk behind the last tile
    const int done = first + (end - first + TT - 1) / TT * TT;
    if (done < stop) {
        Run<T, VE> zero;
        zero.clear();
        for (int c = lane / 4; c < c_count; c += 8)
            for (int t = done + t_mine; t < stop; t += TT)
                store_run(zero, static_cast<T *>(p.y) + (rows + c) * p.L, t, stop, p.vec_y);
    }
    if (p.final_state && chunk == p.chunks - 1) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (mine[k] < c_count) h[k].store(p.final_state + (rows + mine[k]) * p.S, s0, p.S);
    }
}

// Joins chunks in their order: on entry h_chunk holds the state that each
// leaves from a zero state (blocks y = 1: g_chunk the gradient that reaches its
// start from its own outputs), on return the state that it starts from (the
// gradient of the state that it leaves).  A chunk's decay is e^(A sum dt).
// Eight chunks are read at a time, so that the reads do not wait for the
// writes before them.
__global__ void __launch_bounds__(256) join_chunks_kernel(const ScanParams p, int h_chunks,
                                                          int g_chunks) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t per = (int64_t)p.channels * p.S;
    if (i >= p.N * per) return;
    const bool back = blockIdx.y;
    const int chunks = back ? g_chunks : h_chunks;
    const int n = (int)(i / per);
    const int64_t cs = i - n * per;
    const float A = p.A[cs] * kLog2e;
    const int64_t base = (int64_t)n * chunks;
    const float *dts = (back ? p.dt_segment : p.dt_chunk) + base * p.channels + cs / p.S;
    float *rows = (back ? p.g_chunk : p.h_chunk) + base * per + cs;
    const float *first = back ? p.dfinal : p.state;
    float v = first ? first[i] : 0.f;
    constexpr int kBatch = 8;
    for (int k0 = 0; k0 < chunks; k0 += kBatch) {
        float left[kBatch], decay[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const int k = back ? chunks - 1 - k0 - e : k0 + e;
            if (k0 + e < chunks) {
                left[e] = rows[k * per];
                decay[e] = dts[(int64_t)k * p.channels];
            }
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const int k = back ? chunks - 1 - k0 - e : k0 + e;
            if (k0 + e < chunks) {
                rows[k * per] = v;
                v = fmaf(ex2(A * decay[e]), v, left[e]);
            }
        }
    }
    if (back && p.dstate) p.dstate[i] = v;
}

// Step: LPC lanes per request and channel, each with SPT of its states, which
// are read and written once.  Bound by that traffic, so by how much of it is
// under way: a thread takes one request after the other for its channel, with
// the next one's states and inputs being read, and its row of A once.  (One
// request per thread, 128 x 4096 x 16 in bf16: 28 us.)
template <typename T, int SPT, int LPC>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanParams p) {
    const int64_t c64 = (int64_t)blockIdx.x * (256 / LPC) + threadIdx.x / LPC;
    // lane j holds states s0 .. s0 + SPT-1; of whole rows, fours of them LPC
    // fours apart, so that a warp's reads and writes are contiguous
    const int j = threadIdx.x % LPC, s0 = j * SPT;
    const bool on = c64 < p.channels;
    const int c = on ? (int)c64 : 0, g = p.groups > 1 ? c / p.per_group : 0;
    const bool whole = SPT % 4 == 0 && p.vec && p.S == LPC * SPT;
    const T *u = static_cast<const T *>(p.u) + c, *d = static_cast<const T *>(p.delta) + c;
    const T *z = static_cast<const T *>(p.z) + c;
    const T *B = static_cast<const T *>(p.B) + g * p.b_sg, *C = static_cast<const T *>(p.C) + g * p.c_sg;
    const float bias = p.delta_bias ? p.delta_bias[c] : 0.f, D = p.D ? p.D[c] : 0.f;
    float A[SPT];
    const float *rowA = p.A + (int64_t)c * p.S;
    auto place = [&](int k) { return whole ? (k / 4 * LPC + j) * 4 + k % 4 : s0 + k; };
#pragma unroll
    for (int k = 0; k < SPT; ++k) A[k] = place(k) < p.S ? rowA[place(k)] : 0.f;
#pragma unroll
    for (int k = 0; k < SPT; ++k) A[k] *= kLog2e;
    struct Inputs {
        float *row;  // the request's states, nullptr without
        float h[SPT], b[SPT], c[SPT], u, d, z;
    } next;
    auto fetch = [&](int n) {
        next.row = nullptr;
        if (n >= p.N || !on) return;
        const int slot = p.slots ? p.slots[n] : n;
        if (slot < 0 || slot >= p.num_slots) return;
        next.row = p.pool + ((int64_t)slot * p.channels + c) * p.S;
        next.u = to_f32(u[n * p.u_sn]);
        next.d = to_f32(d[n * p.d_sn]);
        if (p.z) next.z = to_f32(z[n * p.z_sn]);
        const T *Bn = B + n * p.b_sn, *Cn = C + n * p.c_sn;
        if constexpr (SPT % 4 == 0) {
            if (whole) {
#pragma unroll
                for (int k = 0; k < SPT; k += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(next.row + place(k));
                    next.h[k] = f.x; next.h[k + 1] = f.y; next.h[k + 2] = f.z; next.h[k + 3] = f.w;
                    Run<T, 4> rb, rc;
                    load_run(rb, Bn, place(k), p.S, true);
                    load_run(rc, Cn, place(k), p.S, true);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        next.b[k + i] = rb[i];
                        next.c[k + i] = rc[i];
                    }
                }
                return;
            }
        }
        load_states<SPT>(next.h, next.row, s0, p.S);
#pragma unroll
        for (int k = 0; k < SPT; ++k) {
            next.b[k] = s0 + k < p.S ? to_f32(Bn[s0 + k]) : 0.f;
            next.c[k] = s0 + k < p.S ? to_f32(Cn[s0 + k]) : 0.f;
        }
    };
    fetch(blockIdx.y);
    for (int n = blockIdx.y; n < p.N; n += gridDim.y) {
        Inputs now = next;
        fetch(n + gridDim.y);
        float o = 0.f;
        if (now.row) {
            const float raw = now.d + bias, dt = p.softplus ? softplus(raw) : raw;
            const float du = dt * now.u;
#pragma unroll
            for (int k = 0; k < SPT; ++k) {
                now.h[k] = fmaf(ex2(dt * A[k]), now.h[k], du * now.b[k]);
                o = fmaf(now.h[k], now.c[k], o);
            }
            if constexpr (SPT % 4 == 0) {
                if (whole) {
#pragma unroll
                    for (int k = 0; k < SPT; k += 4)
                        *reinterpret_cast<float4 *>(now.row + place(k)) =
                            make_float4(now.h[k], now.h[k + 1], now.h[k + 2], now.h[k + 3]);
                }
            }
            if (!whole) store_states<SPT>(now.row, now.h, s0, p.S);
        }
        o += __shfl_xor_sync(~0u, o, 1);
        if (LPC == 4) o += __shfl_xor_sync(~0u, o, 2);
        if (on && j == 0) {
            if (now.row) {
                o = fmaf(D, now.u, o);
                if (p.z) o *= silu(now.z);
            }
            static_cast<T *>(p.y)[(int64_t)n * p.channels + c] = from_f32<T>(o);
        }
    }
}

}  // namespace

int scan_check_sizes(const spconv_scan_args *a) {
    if (!a || a->N < 0 || a->channels < 0 || a->L < 0 || a->S < 1 || a->groups < 1)
        return SPCONV_ERR_INVALID_ARG;
    if (a->dtype < SPCONV_F32 || a->dtype > SPCONV_F16 || (a->softplus & ~1))
        return SPCONV_ERR_INVALID_ARG;
    if (a->channels % a->groups) return SPCONV_ERR_INVALID_ARG;
    for (int64_t s : {a->u_stride_n, a->u_stride_c, a->delta_stride_n, a->delta_stride_c,
                      a->z_stride_n, a->z_stride_c, a->dy_stride_n, a->dy_stride_c, a->b_stride_n,
                      a->b_stride_g, a->b_stride_s, a->c_stride_n, a->c_stride_g, a->c_stride_s})
        if (!stride_ok(s)) return SPCONV_ERR_INVALID_ARG;
    return a->S > 64 || a->L > kMaxLength ? SPCONV_ERR_UNSUPPORTED : SPCONV_OK;
}

ScanParams scan_params(const spconv_scan_args *a) {
    const size_t e = dtype_size(a->dtype);
    ScanParams p{};
    p.u = a->u; p.delta = a->delta; p.z = a->z; p.B = a->B; p.C = a->C; p.dy = a->dy;
    p.A = a->A; p.D = a->D; p.delta_bias = a->delta_bias; p.state = a->state;
    p.dfinal = a->dfinal_state; p.lengths = a->lengths; p.slots = a->slots;
    p.y = a->y; p.du = a->du; p.ddelta = a->ddelta; p.dz = a->dz; p.dB = a->dB; p.dC = a->dC;
    p.final_state = a->final_state; p.pool = a->pool; p.dA = a->dA; p.dD = a->dD;
    p.ddelta_bias = a->ddelta_bias; p.dstate = a->dstate;
    p.u_sn = a->u_stride_n; p.u_sc = a->u_stride_c;
    p.d_sn = a->delta_stride_n; p.d_sc = a->delta_stride_c;
    p.z_sn = a->z_stride_n; p.z_sc = a->z_stride_c;
    p.dy_sn = a->dy_stride_n; p.dy_sc = a->dy_stride_c;
    p.b_sn = a->b_stride_n; p.b_sg = a->b_stride_g; p.b_ss = a->b_stride_s;
    p.c_sn = a->c_stride_n; p.c_sg = a->c_stride_g; p.c_ss = a->c_stride_s;
    p.N = a->N; p.channels = a->channels; p.L = a->L; p.S = a->S; p.groups = a->groups;
    p.per_group = a->channels / a->groups;
    p.softplus = a->softplus; p.num_slots = a->num_slots;
    p.chunks = 1;
    p.chunk_len = a->L;
    p.vec = rows_aligned(a->u, p.u_sn, p.u_sc, e) && rows_aligned(a->delta, p.d_sn, p.d_sc, e) &&
            (!a->z || rows_aligned(a->z, p.z_sn, p.z_sc, e)) &&
            rows_aligned(a->B, p.b_sn, p.b_sg, e) && rows_aligned(a->B, 0, p.b_ss, e) &&
            rows_aligned(a->C, p.c_sn, p.c_sg, e) && rows_aligned(a->C, 0, p.c_ss, e) &&
            (!a->dy || rows_aligned(a->dy, p.dy_sn, p.dy_sc, e));
    return p;
}

int scan_join_chunks(const ScanParams &p, bool grad, cudaStream_t stream) {
    const int64_t count = (int64_t)p.N * p.channels * p.S;
    join_chunks_kernel<<<dim3((unsigned)((count + 255) / 256), grad ? 2 : 1), 256, 0, stream>>>(
        p, grad ? p.tiles : p.chunks, p.segments);
    return launch_status();
}

}  // namespace seq
}  // namespace spconv

using namespace spconv::seq;

namespace {

bool words(std::initializer_list<const void *> ps) {
    for (const void *q : ps)
        if (!aligned(q, 4)) return false;
    return true;
}
bool elements(size_t e, std::initializer_list<const void *> ps) {
    for (const void *q : ps)
        if (!aligned(q, e)) return false;
    return true;
}

}  // namespace

namespace {

constexpr int64_t kSplitBelow = 304, kSplitTo = 1216;  // warps

// f(SPT, LPC) for the smallest tile that holds S states.
template <typename F>
int by_tile(int S, bool wide, F f) {
    using std::integral_constant;
    if (S <= 4) return f(integral_constant<int, 2>{}, integral_constant<int, 2>{});
    if (S <= 8) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
    if (S <= 16)
        return wide ? f(integral_constant<int, 8>{}, integral_constant<int, 2>{})
                    : f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
    if (S <= 32) return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
}

// Blocks and chunks of the forward scan.  One pass over a sequence needs a warp
// per 32 channels of each sequence; where that leaves schedulers idle the
// sequence is cut, into chunks of 128 positions at least.  Two more
// passes over the states are the price: what every chunk leaves from zero (no
// outputs), and the join.
void plan_chunks(ScanParams &p) {
    p.wide = (int64_t)p.N * p.channels >= 16 * 4096;
    const int cw = p.S <= 8 || p.S > 16 && p.S <= 32 || p.S <= 16 && p.wide ? 32 : 16;
    p.blocks_per_group = (p.per_group + cw - 1) / cw;
    const int64_t blocks = (int64_t)p.groups * p.blocks_per_group * p.N;
    const int64_t most = p.L / 128;
    p.chunks = 1;
    p.chunk_len = p.L;
    if (blocks >= kSplitBelow || most < 2) return;
    int64_t want = (kSplitTo + blocks - 1) / blocks;
    if (want > most) want = most;
    const int64_t len = ((p.L + want - 1) / want + 31) / 32 * 32;  // whole tiles of either type
    p.chunk_len = (int)len;
    p.chunks = (int)((p.L + len - 1) / len);
}

int64_t state_floats(const ScanParams &p) {
    return ((int64_t)p.N * p.chunks * p.channels * p.S + 3) / 4 * 4;
}

}  // namespace

SPCONV_API int64_t spconv_scan_workspace(const spconv_scan_args *a) {
    if (scan_check_sizes(a) || a->channels == 0 || a->N == 0) return 0;
    ScanParams p = scan_params(a);
    plan_chunks(p);
    return p.chunks == 1 ? 0 : (state_floats(p) + (int64_t)p.N * p.chunks * p.channels) * 4;
}

SPCONV_API int spconv_scan(const spconv_scan_args *a, void *stream) {
    const int st = scan_check_sizes(a);
    if (st) return st;
    if (a->N > 65535) return SPCONV_ERR_UNSUPPORTED;  // sequences go along grid y
    const int64_t rows = (int64_t)a->N * a->channels;
    if (rows == 0) return SPCONV_OK;
    const size_t e = dtype_size(a->dtype);
    if (!a->A || (a->L > 0 && (!a->u || !a->delta || !a->B || !a->C || !a->y)))
        return SPCONV_ERR_INVALID_ARG;
    if (!elements(e, {a->u, a->delta, a->z, a->B, a->C, a->y}) ||
        !words({a->A, a->D, a->delta_bias, a->state, a->lengths, a->final_state}))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t L = a->L, yb = rows * L * e, sb = rows * a->S * 4;
    const int64_t bb = extent(a->N, a->groups, (a->S - 1) * a->b_stride_s + L, a->b_stride_n, a->b_stride_g, e);
    const int64_t cb = extent(a->N, a->groups, (a->S - 1) * a->c_stride_s + L, a->c_stride_n, a->c_stride_g, e);
    if (L > 0)
        for (const auto &o : {std::pair<const void *, int64_t>{a->y, yb}, {a->final_state, sb}})
            if (overlap(o.first, o.second, a->u, extent(a->N, a->channels, L, a->u_stride_n, a->u_stride_c, e)) ||
                overlap(o.first, o.second, a->delta, extent(a->N, a->channels, L, a->delta_stride_n, a->delta_stride_c, e)) ||
                overlap(o.first, o.second, a->z, extent(a->N, a->channels, L, a->z_stride_n, a->z_stride_c, e)) ||
                overlap(o.first, o.second, a->B, bb) || overlap(o.first, o.second, a->C, cb) ||
                overlap(o.first, o.second, a->state, sb))
                return SPCONV_ERR_INVALID_ARG;
    if (overlap(a->y, yb, a->final_state, sb) || overlap(a->state, sb, a->final_state, sb))
        return SPCONV_ERR_INVALID_ARG;
    ScanParams p = scan_params(a);
    plan_chunks(p);
    if (p.chunks > 1) {
        const int64_t need = spconv_scan_workspace(a);
        if (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < need)
            return SPCONV_ERR_INVALID_ARG;
        p.h_chunk = static_cast<float *>(a->workspace);
        p.dt_chunk = p.h_chunk + state_floats(p);
    }
    p.vec_y = rows_aligned(a->y, 0, L, e);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_dtype(a->dtype, [&](auto t) {
        return by_tile(a->S, p.wide, [&](auto spt, auto lpc) {
            using T = decltype(t);
            constexpr int SPT = decltype(spt)::value, LPC = decltype(lpc)::value;
            const dim3 grid(p.groups * p.blocks_per_group, p.N, p.chunks);
            if (p.chunks > 1) {
                scan_kernel<T, SPT, LPC, true><<<grid, 32, 0, s>>>(p);
                if (int rc = launch_status()) return rc;
                if (int rc = scan_join_chunks(p, false, s)) return rc;
            }
            scan_kernel<T, SPT, LPC, false><<<grid, 32, 0, s>>>(p);
            return launch_status();
        });
    });
}

SPCONV_API int spconv_scan_step(const spconv_scan_args *a, void *stream) {
    const int st = scan_check_sizes(a);
    if (st) return st;
    if (a->N > 65535) return SPCONV_ERR_UNSUPPORTED;  // requests go along grid y
    if (a->num_slots < 0 || (!a->slots && a->num_slots != a->N) || a->u_stride_c != 1 ||
        a->delta_stride_c != 1 || (a->z && a->z_stride_c != 1) || a->b_stride_s != 1 ||
        a->c_stride_s != 1)
        return SPCONV_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)a->N * a->channels;
    if (rows == 0) return SPCONV_OK;
    const size_t e = dtype_size(a->dtype);
    if (!a->A || !a->u || !a->delta || !a->B || !a->C || !a->y || (a->num_slots > 0 && !a->pool))
        return SPCONV_ERR_INVALID_ARG;
    if (!elements(e, {a->u, a->delta, a->z, a->B, a->C, a->y}) ||
        !words({a->A, a->D, a->delta_bias, a->pool, a->slots}))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t yb = rows * e, sb = (int64_t)a->num_slots * a->channels * a->S * 4;
    for (const auto &o : {std::pair<const void *, int64_t>{a->y, yb}, {a->pool, sb}})
        if (overlap(o.first, o.second, a->u, extent(a->N, a->channels, 1, a->u_stride_n, 1, e)) ||
            overlap(o.first, o.second, a->delta, extent(a->N, a->channels, 1, a->delta_stride_n, 1, e)) ||
            overlap(o.first, o.second, a->z, extent(a->N, a->channels, 1, a->z_stride_n, 1, e)) ||
            overlap(o.first, o.second, a->B, extent(a->N, a->groups, a->S, a->b_stride_n, a->b_stride_g, e)) ||
            overlap(o.first, o.second, a->C, extent(a->N, a->groups, a->S, a->c_stride_n, a->c_stride_g, e)))
            return SPCONV_ERR_INVALID_ARG;
    if (overlap(a->y, yb, a->pool, sb)) return SPCONV_ERR_INVALID_ARG;
    ScanParams p = scan_params(a);
    p.vec = aligned(a->pool, 16) && aligned(a->A, 16) &&
            rows_aligned(a->B, a->b_stride_n, a->b_stride_g, e) &&
            rows_aligned(a->C, a->c_stride_n, a->c_stride_g, e);
    return by_dtype(a->dtype, [&](auto t) {
        return by_tile(a->S, true, [&](auto spt, auto lpc) {
            constexpr int SPT = decltype(spt)::value, LPC = decltype(lpc)::value, CB = 256 / LPC;
            const int64_t blocks = ((int64_t)a->channels + CB - 1) / CB;
            int64_t side = (4 * kSMs + blocks - 1) / blocks;  // requests side by side: 4 blocks per SM
            if (side > a->N) side = a->N;
            scan_step_kernel<decltype(t), SPT, LPC>
                <<<dim3((unsigned)blocks, (unsigned)side), 256, 0,
                   static_cast<cudaStream_t>(stream)>>>(p);
            return launch_status();
        });
    });
}
