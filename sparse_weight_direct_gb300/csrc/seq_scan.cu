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

// Tiling.  A lane holds SPT states of each of four channels, four lanes hold a
// channel, so a position's 2 * SPT values of B and C, read from shared memory,
// serve four channels.  (A broadcast read costs a 4-byte word per lane like any
// other: with one and two channels per lane the reads were what bounded the
// kernel, at 19 words a lane and position for 16 channels of 16 states.)
// What is left to hide is latency: a sequence of 4096 channels has 128 such
// warps, fewer than there are schedulers.  So a block has one warp for the
// states and two that turn the next tiles' rows into step sizes and the last
// ones' sums into outputs; tiles go through two buffers, each handed over and
// back by a named barrier.  4 x 4096 channels x 2048 positions x 16 states in
// bf16 take 201 us (one warp for all of it: 232; two channels per lane and two
// warps for states: 282, its registers leave three blocks per SM): the warp of states
// issues every second clock, 165 a position.
template <typename T, int SPT_>
struct ScanTile {
    static constexpr int SPT = SPT_, SP = 4 * SPT;
    static constexpr int VE = 16 / sizeof(T), TT = 4 * VE;  // positions of a lane's load, of a tile
    static constexpr int CB = 32;                           // channels of a block
    static constexpr int NI = 2;                            // loads of a lane from each row set
    static constexpr int NB = (2 * SP * 4 + 63) / 64;       // from B and C
    // rows of a position: one more after every VE positions, and three more that
    // are read ahead
    static constexpr int kRows = TT + 7;
    // {dt, dt u} of a quad's four channels: rows of 40 bytes, quads 32 modulo
    // 128 bytes apart, so that neither the lanes that write a channel's positions
    // nor the quads that read a position meet in a bank
    static constexpr int kStepPitch = (5 * kRows + 11) / 16 * 16 + 4;  // of 8 bytes
    static constexpr int kOutPitch = TT + 4;
    static constexpr int kOutPart = 8 * kOutPitch + 8;  // to the quads' next channels
    static constexpr int kSteps = 8 * kStepPitch * 2;   // floats
    static constexpr int kOut = 4 * kOutPart;
    static constexpr int kMatrix = kRows * SP;          // of B, of C
    static constexpr int kBuffer = 2 * kMatrix + kSteps + kOut;
    static constexpr bool kAhead = NB <= 4;  // B and C of the next tile wait in registers
    // decays and inputs of the next position wait in registers
    static constexpr bool kForm = SPT <= 8;
};
constexpr int kScanThreads = 96;

// Barriers between the two kinds of warps, one for each buffer and direction.
// (Their numbers are constants of the instructions, or a block would take all
// sixteen.)
template <int ID>
static __device__ __forceinline__ void barrier_sync() {
    asm volatile("barrier.cta.sync %0, %1;" ::"n"(ID), "n"(kScanThreads) : "memory");
}
template <int ID>
static __device__ __forceinline__ void barrier_arrive() {
    __threadfence_block();
    asm volatile("barrier.cta.arrive %0, %1;" ::"n"(ID), "n"(kScanThreads) : "memory");
}
constexpr int kFull = 1, kEmpty = 3;  // + buffer

// One pass over a chunk of positions with the states in registers.
// ENDS: from zero states, only what the chunk leaves and the sum of its step
// sizes.  Otherwise the outputs.
template <typename T, int SPT, bool ENDS>
__global__ void __launch_bounds__(kScanThreads, SPT <= 4 ? 4 : 2) scan_kernel(const ScanParams p) {
    using G = ScanTile<T, SPT>;
    constexpr int VE = G::VE, TT = G::TT, SP = G::SP, NP = Pairs<SPT>::N, NI = G::NI, NB = G::NB;
    extern __shared__ __align__(16) float sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = blockIdx.y, chunk = blockIdx.z;
    const int g = blockIdx.x / p.blocks_per_group;
    const int c_first = (blockIdx.x - g * p.blocks_per_group) * G::CB;  // within the group
    const int c_count = min(G::CB, p.per_group - c_first);
    const int64_t c_base = (int64_t)g * p.per_group + c_first;
    const int len = p.lengths ? min(max(p.lengths[n], 0), p.L) : p.L;
    const int first = chunk * p.chunk_len, stop = first + min(p.L - first, p.chunk_len);
    const int end = max(min(len, stop), first);
    const int tiles = (end - first + TT - 1) / TT;
    const int64_t rows = (int64_t)n * p.channels + c_base;
    const int64_t chunk_rows = ((int64_t)n * p.chunks + chunk) * p.channels + c_base;

    if (warp == 0) {  // the states
        const int quad = lane >> 2, j = lane & 3, s0 = j * SPT;
        // Lane j holds the quad's channels in the order 0 ^ j, 1 ^ j, 2 ^ j, 3 ^ j: in
        // the sums over two lanes each keeps its even ones, then its first, and
        // gives the others, and ends with channel j.
        int mine[4];
        Pairs<SPT> A[4], h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            mine[q] = quad + 8 * (q ^ j);
            const int S = mine[q] < c_count ? p.S : 0;
            A[q].load(p.A + (c_base + mine[q]) * p.S, s0, S);
            A[q].scale(kLog2e);
            if (ENDS)
                h[q].fill(0.f);
            else if (p.chunks > 1)
                h[q].load(p.h_chunk + (chunk_rows + mine[q]) * p.S, s0, S);
            else if (p.state)
                h[q].load(p.state + (rows + mine[q]) * p.S, s0, S);
            else
                h[q].fill(0.f);
        }
        for (int i = 0; i < tiles; ++i) {
            float *buffer = sm + (i & 1) * G::kBuffer;
            const float *bc = buffer;
            const float2 *step = reinterpret_cast<const float2 *>(buffer + 2 * G::kMatrix) +
                                 quad * G::kStepPitch;
            float *out = buffer + 2 * G::kMatrix + G::kSteps + j * G::kOutPart + quad * G::kOutPitch;
            if (i & 1)
                barrier_sync<kFull + 1>();
            else
                barrier_sync<kFull>();
            // Two positions ahead of the states, what a position needs is read; one
            // ahead, its decays and inputs are formed.  (Behind the tile's last
            // position lie rows that are read and not used.)
            float2 x[4];
            Pairs<SPT> bn, cn, c1;
            constexpr int NF = G::kForm ? NP : 1;
            f32x2 a1[4][NF], b1[4][NF];
            auto read = [&](int r) {
#pragma unroll
                for (int q = 0; q < 4; ++q) x[q] = step[r * 5 + (q ^ j)];
                bn.read(bc + r * SP + s0);
                if (!ENDS) cn.read(bc + G::kMatrix + r * SP + s0);
            };
            auto form = [&]() {
                if constexpr (G::kForm) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x2 dt = pack2(x[q].x, x[q].x), du = pack2(x[q].y, x[q].y);
#pragma unroll
                        for (int k = 0; k < NP; ++k) {
                            a1[q][k] = decay2(dt, A[q].v[k]);
                            b1[q][k] = mul2(du, bn.v[k]);
                        }
                    }
                    c1 = cn;
                }
            };
            read(0);
            if (G::kForm) {
                form();
                read(1);
            }
#pragma unroll 1
            for (int t = 0; t < TT; t += 4) {
                float y[4][4];
                const int r0 = t + t / VE, r4 = t + 4 + (t + 4) / VE;  // rows of t and t + 4
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        f32x2 o = 0;
                        const f32x2 dt = pack2(x[q].x, x[q].x), du = pack2(x[q].y, x[q].y);
#pragma unroll
                        for (int e = 0; e < NP; ++e) {
                            const f32x2 a = G::kForm ? a1[q][G::kForm ? e : 0] : decay2(dt, A[q].v[e]);
                            const f32x2 in = G::kForm ? b1[q][G::kForm ? e : 0] : mul2(du, bn.v[e]);
                            const f32x2 c = G::kForm ? c1.v[e] : cn.v[e];
                            h[q].v[e] = fma2(a, h[q].v[e], in);
                            if (!ENDS) o = e ? fma2(h[q].v[e], c, o) : mul2(h[q].v[e], c);
                        }
                        const float2 f = unpack2(o);
                        y[k][q] = f.x + f.y;
                    }
                    form();
                    if (G::kForm)
                        read(k < 2 ? r0 + k + 2 : r4 + k - 2);
                    else
                        read(k < 3 ? r0 + k + 1 : r4);
                }
                if (!ENDS) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        y[k][0] += __shfl_xor_sync(~0u, y[k][1], 1);
                        y[k][2] += __shfl_xor_sync(~0u, y[k][3], 1);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[k][0] += __shfl_xor_sync(~0u, y[k][2], 2);
                    *reinterpret_cast<float4 *>(out + t) =
                        make_float4(y[0][0], y[1][0], y[2][0], y[3][0]);
                }
            }
            if (i & 1)
                barrier_arrive<kEmpty + 1>();
            else
                barrier_arrive<kEmpty>();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (mine[q] >= c_count) continue;
            if (ENDS)
                h[q].store(p.h_chunk + (chunk_rows + mine[q]) * p.S, s0, p.S);
            else if (p.final_state && chunk == p.chunks - 1)
                h[q].store(p.final_state + (rows + mine[q]) * p.S, s0, p.S);
        }
        return;
    }

    // the rows: a lane has the positions t_mine .. of its warp's channels row, row + 8
    const int quarter = lane & 3, t_mine = quarter * VE, half = warp - 1;
    const int row = half * 16 + (lane >> 2);
    const T *ub = static_cast<const T *>(p.u) + n * p.u_sn + (c_base + row) * p.u_sc;
    const T *db = static_cast<const T *>(p.delta) + n * p.d_sn + (c_base + row) * p.d_sc;
    const T *zb = !ENDS && p.z ? static_cast<const T *>(p.z) + n * p.z_sn + (c_base + row) * p.z_sc
                               : nullptr;
    const T *Bb = static_cast<const T *>(p.B) + n * p.b_sn + g * p.b_sg;
    const T *Cb = static_cast<const T *>(p.C) + n * p.c_sn + g * p.c_sg;
    T *yb = static_cast<T *>(p.y) + (rows + row) * p.L;
    float bias[NI], D[NI], total[NI];
    int row_end[NI];
#pragma unroll
    for (int k = 0; k < NI; ++k) {
        const int c = row + 8 * k;
        row_end[k] = c < c_count ? end : 0;
        bias[k] = p.delta_bias && c < c_count ? p.delta_bias[c_base + c] : 0.f;
        D[k] = p.D && c < c_count ? p.D[c_base + c] : 0.f;
        total[k] = 0.f;
    }
    struct Next {
        Run<T, VE> u[NI], d[NI], bc[NB];
    } next[2];  // on their way: the tiles that the buffers will hold
    struct Kept {
        Run<T, VE> u[NI], z[NI];
    } kept[2];  // of the tiles in the buffers
    auto fetch_bc = [&](int t0, Run<T, VE> (&bc)[NB]) {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = lane + 32 * half + 64 * k, s = i % SP, q = (i / SP) % 4, which = i / (SP * 4);
            if (ENDS && which) continue;
            const T *from = which ? Cb + s * p.c_ss : Bb + s * p.b_ss;
            load_run(bc[k], from, t0 + q * VE, s < p.S && which < 2 ? end : 0, p.vec);
        }
    };
    auto fetch = [&](int t0, Next &to) {
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            load_run(to.d[k], db + 8 * k * p.d_sc, t0 + t_mine, row_end[k], p.vec);
            load_run(to.u[k], ub + 8 * k * p.u_sc, t0 + t_mine, row_end[k], p.vec);
        }
        if (G::kAhead) fetch_bc(t0, to.bc);
    };
    auto stage = [&](int t0, float *buffer, Next &from, Kept &keep) {
        if (!G::kAhead) fetch_bc(t0, from.bc);
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = lane + 32 * half + 64 * k, s = i % SP, q = (i / SP) % 4, which = i / (SP * 4);
            if (which >= (ENDS ? 1 : 2)) continue;
            float *to = buffer + which * G::kMatrix + q * (VE + 1) * SP + s;
#pragma unroll
            for (int e = 0; e < VE; ++e) to[e * SP] = from.bc[k][e];
        }
        float dt[NI][VE];
#pragma unroll
        for (int k = 0; k < NI; ++k)
#pragma unroll
            for (int e = 0; e < VE; ++e) dt[k][e] = from.d[k][e] + bias[k];
        if (p.softplus) {
#pragma unroll
            for (int k = 0; k < NI; ++k)
#pragma unroll
                for (int e = 0; e < VE; ++e) dt[k][e] = softplus(dt[k][e]);
        }
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            float2 *to = reinterpret_cast<float2 *>(buffer + 2 * G::kMatrix) +
                         (lane >> 2) * G::kStepPitch + quarter * (VE + 1) * 5 + 2 * half + k;
            keep.u[k] = from.u[k];
            if (t0 + TT > row_end[k]) {
                // behind the end a step of size zero leaves the states as they are
#pragma unroll
                for (int e = 0; e < VE; ++e) dt[k][e] = t0 + t_mine + e < row_end[k] ? dt[k][e] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                to[5 * e] = make_float2(dt[k][e], dt[k][e] * keep.u[k][e]);
                if (ENDS) total[k] += dt[k][e];
            }
        }
    };
    auto finish = [&](int t0, const float *buffer, const Kept &keep) {
        float o[NI][VE];
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            const float4 *q = reinterpret_cast<const float4 *>(
                buffer + 2 * G::kMatrix + G::kSteps + (2 * half + k) * G::kOutPart +
                (lane >> 2) * G::kOutPitch + t_mine);
#pragma unroll
            for (int e = 0; e < VE; e += 4) {
                const float4 f = q[e / 4];
                const float y[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) o[k][e + i] = fmaf(D[k], keep.u[k][e + i], y[i]);
            }
        }
        if (zb) {
#pragma unroll
            for (int k = 0; k < NI; ++k)
#pragma unroll
                for (int e = 0; e < VE; ++e) o[k][e] *= silu(keep.z[k][e]);
        }
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            if (t0 + TT > end) {
#pragma unroll
                for (int e = 0; e < VE; ++e) o[k][e] = t0 + t_mine + e < end ? o[k][e] : 0.f;
            }
            Run<T, VE> out;
            out.put(o[k]);
            if (row + 8 * k < c_count)
                store_run(out, yb + 8 * k * (int64_t)p.L, t0 + t_mine, stop, p.vec_y);
        }
    };
    if (tiles > 0) fetch(first, next[0]);
    if (tiles > 1) fetch(first + TT, next[1]);
    for (int i0 = 0; i0 < tiles + 2; i0 += 2) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {  // (by pairs, so that what is kept stays in registers)
            const int i = i0 + b, t0 = first + i * TT;
            float *buffer = sm + b * G::kBuffer;
            if (i >= 2 && i - 2 < tiles) {
                if (b)
                    barrier_sync<kEmpty + 1>();
                else
                    barrier_sync<kEmpty>();
                if (!ENDS) finish(t0 - 2 * TT, buffer, kept[b]);
            }
            if (i >= tiles) continue;
            __syncwarp();
            stage(t0, buffer, next[b], kept[b]);
            if (b)
                barrier_arrive<kFull + 1>();
            else
                barrier_arrive<kFull>();
            if (!ENDS && zb) {
#pragma unroll
                for (int k = 0; k < NI; ++k)
                    load_run(kept[b].z[k], zb + 8 * k * p.z_sc, t0 + t_mine, row_end[k], p.vec);
            }
            if (i + 2 < tiles) fetch(t0 + 2 * TT, next[b]);
        }
    }
    if (ENDS) {
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            total[k] += __shfl_xor_sync(~0u, total[k], 1);
            total[k] += __shfl_xor_sync(~0u, total[k], 2);
            if (quarter == 0 && row + 8 * k < c_count) p.dt_chunk[chunk_rows + row + 8 * k] = total[k];
        }
        return;
    }
    // positions of the chunk behind the last tile
    const int done = first + tiles * TT;
    if (done < stop) {
        Run<T, VE> zero;
        zero.clear();
        for (int k = 0; k < NI; ++k)
            for (int t = done + t_mine; t < stop && row + 8 * k < c_count; t += TT)
                store_run(zero, yb + 8 * k * (int64_t)p.L, t, stop, p.vec_y);
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
// the next one's states and inputs being read, and its row of A once.  128 x
// 4096 x 16 in bf16: one request per thread 28 us, two blocks per SM 24, three
// (B and C kept as words) 18, four spill and take 20.  In f32 three spill too (56
// bytes of stack): 26 us.  32 states and more leave one block: 64 in bf16 72 us.
template <typename T, int SPT, int LPC>
__global__ void __launch_bounds__(256, SPT <= 8 ? 3 : 1) scan_step_kernel(const ScanParams p) {
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
    constexpr int kFours = SPT % 4 == 0 ? SPT / 4 : 1;
    struct Inputs {
        float *row;  // the request's states, nullptr without
        float h[SPT];
        T u, d, z;
        Run<T, 4> b[kFours], c[kFours];  // of whole rows (as words: registers are blocks)
    } next;
    auto fetch = [&](int n) {
        next.row = nullptr;
        if (n >= p.N || !on) return;
        const int slot = p.slots ? p.slots[n] : n;
        if (slot < 0 || slot >= p.num_slots) return;
        next.row = p.pool + ((int64_t)slot * p.channels + c) * p.S;
        next.u = u[n * p.u_sn];
        next.d = d[n * p.d_sn];
        if (p.z) next.z = z[n * p.z_sn];
        if constexpr (SPT % 4 == 0) {
            if (whole) {
                const T *Bn = B + n * p.b_sn, *Cn = C + n * p.c_sn;
#pragma unroll
                for (int k = 0; k < SPT; k += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(next.row + place(k));
                    next.h[k] = f.x; next.h[k + 1] = f.y; next.h[k + 2] = f.z; next.h[k + 3] = f.w;
                    load_run(next.b[k / 4], Bn, place(k), p.S, true);
                    load_run(next.c[k / 4], Cn, place(k), p.S, true);
                }
                return;
            }
        }
        load_states<SPT>(next.h, next.row, s0, p.S);
    };
    fetch(blockIdx.y);
    for (int n = blockIdx.y; n < p.N; n += gridDim.y) {
        Inputs now = next;
        fetch(n + gridDim.y);
        float o = 0.f;
        if (now.row) {
            const float raw = to_f32(now.d) + bias, dt = p.softplus ? softplus(raw) : raw;
            const float du = dt * to_f32(now.u);
            if constexpr (SPT % 4 == 0) {
                if (whole) {
#pragma unroll
                    for (int k = 0; k < SPT; ++k) {
                        now.h[k] = fmaf(decay(dt, A[k]), now.h[k], du * now.b[k / 4][k % 4]);
                        o = fmaf(now.h[k], now.c[k / 4][k % 4], o);
                    }
#pragma unroll
                    for (int k = 0; k < SPT; k += 4)
                        *reinterpret_cast<float4 *>(now.row + place(k)) =
                            make_float4(now.h[k], now.h[k + 1], now.h[k + 2], now.h[k + 3]);
                }
            }
            if (!whole) {
                const T *Bn = B + n * p.b_sn, *Cn = C + n * p.c_sn;
#pragma unroll
                for (int k = 0; k < SPT; ++k) {
                    const bool in = s0 + k < p.S;
                    now.h[k] = fmaf(decay(dt, A[k]), now.h[k], du * (in ? to_f32(Bn[s0 + k]) : 0.f));
                    o = fmaf(now.h[k], in ? to_f32(Cn[s0 + k]) : 0.f, o);
                }
            }
            if (!whole) store_states<SPT>(now.row, now.h, s0, p.S);
        }
        o += __shfl_xor_sync(~0u, o, 1);
        if (LPC == 4) o += __shfl_xor_sync(~0u, o, 2);
        if (on && j == 0) {
            if (now.row) {
                o = fmaf(D, to_f32(now.u), o);
                if (p.z) o *= silu(to_f32(now.z));
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
    return a->S > 64 || a->L > kMaxLength || a->channels > kMaxLength ? SPCONV_ERR_UNSUPPORTED
                                                                      : SPCONV_OK;
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

// f(SPT, LPC) for the smallest tile of a step that holds S states.
template <typename F>
int by_lanes(int S, F f) {
    using std::integral_constant;
    if (S <= 4) return f(integral_constant<int, 2>{}, integral_constant<int, 2>{});
    if (S <= 8) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
    if (S <= 16) return f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
    if (S <= 32) return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
}

// Blocks and chunks of the forward scan.  One pass over a sequence needs a block
// per 32 channels of each sequence; where that leaves SMs idle the sequence is
// cut.  The price are two more passes over the states: what every chunk leaves
// from zero (without outputs it takes two thirds of a pass) and the join.
// The time of a plan, in positions of a full GPU: four blocks fit an SM, and
// one takes 0.62 of what it takes among four, two 0.73 (measured: 4096
// channels x 2048 positions of 2, 3 and 4 sequences take 166, 185 and 205 us).
// One sequence of those: 4 chunks (512 blocks, one wave) take 93 us, 5 (640) took
// 131; two sequences whole take 166, in 3 chunks each they took 222.  All of it was
// measured on 16 states in bf16; above 16 states two blocks fit an SM, and a wave
// counted here runs as two.
void plan_chunks(ScanParams &p) {
    p.blocks_per_group = (p.per_group + 31) / 32;
    const int64_t blocks = (int64_t)p.groups * p.blocks_per_group * p.N;
    auto time = [&](int64_t chunks, int64_t len) {
        const int64_t all = blocks * chunks, wave = 4 * kSMs, rest = all % wave;
        const double last = rest ? 0.62 + 0.11 * (double)((rest + kSMs - 1) / kSMs) : 0.;
        return ((double)(all / wave) * 1.06 + last) * (double)len;
    };
    p.chunks = 1;
    p.chunk_len = p.L;
    double best = time(1, p.L);
    for (int64_t k = 2; k <= p.L / 64 && (k - 1) * blocks < 4 * kSMs; ++k) {
        const int64_t len = ((p.L + k - 1) / k + 31) / 32 * 32;  // whole tiles of either type
        const int64_t chunks = (p.L + len - 1) / len;
        const double t = 1.65 * time(chunks, len) + 80.;
        if (t >= best) continue;
        best = t;
        p.chunk_len = (int)len;
        p.chunks = (int)chunks;
    }
}

int64_t state_floats(const ScanParams &p) {
    return ((int64_t)p.N * p.chunks * p.channels * p.S + 3) / 4 * 4;
}

int64_t workspace_bytes(const ScanParams &p) {
    return p.chunks == 1 ? 0 : (state_floats(p) + (int64_t)p.N * p.chunks * p.channels) * 4;
}

}  // namespace

SPCONV_API int64_t spconv_scan_workspace(const spconv_scan_args *a) {
    if (scan_check_sizes(a) || a->channels == 0 || a->N == 0) return 0;
    ScanParams p = scan_params(a);
    plan_chunks(p);
    return workspace_bytes(p);
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
    ScanParams p = scan_params(a);
    plan_chunks(p);
    const int64_t need = workspace_bytes(p);
    const int64_t bb = L ? extent(a->N, a->groups, (a->S - 1) * a->b_stride_s + L, a->b_stride_n, a->b_stride_g, e) : 0;
    const int64_t cb = L ? extent(a->N, a->groups, (a->S - 1) * a->c_stride_s + L, a->c_stride_n, a->c_stride_g, e) : 0;
    if (!apart({{a->y, yb}, {a->final_state, sb}, {a->workspace, need}},
               {{a->u, extent(a->N, a->channels, L, a->u_stride_n, a->u_stride_c, e)},
                {a->delta, extent(a->N, a->channels, L, a->delta_stride_n, a->delta_stride_c, e)},
                {a->z, extent(a->N, a->channels, L, a->z_stride_n, a->z_stride_c, e)},
                {a->B, bb}, {a->C, cb}, {a->state, sb}, {a->lengths, a->N * 4LL},
                {a->A, a->channels * 4LL * a->S}, {a->D, a->channels * 4LL}, {a->delta_bias, a->channels * 4LL}}))
        return SPCONV_ERR_INVALID_ARG;
    if (need) {
        if (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < need)
            return SPCONV_ERR_INVALID_ARG;
        p.h_chunk = static_cast<float *>(a->workspace);
        p.dt_chunk = p.h_chunk + state_floats(p);
    }
    p.vec_y = rows_aligned(a->y, 0, L, e);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_dtype(a->dtype, [&](auto t) {
        return by_states(a->S, [&](auto spt) {
            using T = decltype(t);
            constexpr int SPT = decltype(spt)::value, smem = 2 * ScanTile<T, SPT>::kBuffer * 4;
            static_assert(smem <= 227 * 1024, "two tiles fit shared memory");
            const dim3 grid(p.groups * p.blocks_per_group, p.N, p.chunks);
            auto *ends = scan_kernel<T, SPT, true>;
            auto *full = scan_kernel<T, SPT, false>;
            if (int rc = raise_smem(reinterpret_cast<const void *>(full), smem)) return rc;
            if (p.chunks > 1) {
                if (int rc = raise_smem(reinterpret_cast<const void *>(ends), smem)) return rc;
                ends<<<grid, kScanThreads, smem, s>>>(p);
                if (int rc = launch_status()) return rc;
                if (int rc = scan_join_chunks(p, false, s)) return rc;
            }
            full<<<grid, kScanThreads, smem, s>>>(p);
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
    if (!apart({{a->y, yb}, {a->pool, sb}},
               {{a->u, extent(a->N, a->channels, 1, a->u_stride_n, 1, e)},
                {a->delta, extent(a->N, a->channels, 1, a->delta_stride_n, 1, e)},
                {a->z, extent(a->N, a->channels, 1, a->z_stride_n, 1, e)},
                {a->B, extent(a->N, a->groups, a->S, a->b_stride_n, a->b_stride_g, e)},
                {a->C, extent(a->N, a->groups, a->S, a->c_stride_n, a->c_stride_g, e)},
                {a->A, a->channels * 4LL * a->S}, {a->D, a->channels * 4LL}, {a->delta_bias, a->channels * 4LL},
                {a->slots, a->N * 4LL}}))
        return SPCONV_ERR_INVALID_ARG;
    ScanParams p = scan_params(a);
    p.vec = aligned(a->pool, 16) && aligned(a->A, 16) &&
            rows_aligned(a->B, a->b_stride_n, a->b_stride_g, e) &&
            rows_aligned(a->C, a->c_stride_n, a->c_stride_g, e);
    return by_dtype(a->dtype, [&](auto t) {
        return by_lanes(a->S, [&](auto spt, auto lpc) {
            constexpr int SPT = decltype(spt)::value, LPC = decltype(lpc)::value, CB = 256 / LPC;
            const int64_t blocks = ((int64_t)a->channels + CB - 1) / CB;
            int64_t side = (6 * kSMs + blocks - 1) / blocks;  // requests side by side: 6 blocks per SM
            if (side > a->N) side = a->N;
            scan_step_kernel<decltype(t), SPT, LPC>
                <<<dim3((unsigned)blocks, (unsigned)side), 256, 0,
                   static_cast<cudaStream_t>(stream)>>>(p);
            return launch_status();
        });
    });
}
