// Gradients of the selective state space scan.
//
// With do_t = dy_t silu(z_t) and g_t the gradient that reaches h_t,
//
//   g_t = C_t do_t + a_(t+1) g_(t+1),  a_t = e^(dt A)
//   dz = dy o silu'(z),  dC_t = sum_c do_t h_t,  dB_t = sum_c g_t dt u
//   q_t = a_t g_t h_(t-1),  ddt = u (g_t . B_t) + sum_s q_t A,  dA = sum q_t dt
//   du = dt (g_t . B_t) + D do_t,  dD = sum do_t u,  ddelta = ddt sigmoid(raw)
//
// The sequence is cut into tiles of 32 positions and segments of a few tiles.
// One kernel finds what every tile leaves of h from zero and every segment of g
// towards its start; one joins them over the sequence; one forms every
// segment's gradients from the states that its tiles start with and the
// gradient that it ends with.  So all segments run side by side and nothing is
// kept by the forward call: the states cost a number per tile of traffic, not
// one per position.  Within a tile the gradient kernel runs forwards once, keeping
// the states before every fourth position in shared memory, and then goes back
// by four positions at a time: their states and decays are formed again, in
// registers, and used up backwards.  An exponential three times per state
// and position in all is cheaper than the traffic of keeping it.
// Sums over channels, sequences and segments are joined from the blocks' shares
// in a fixed order.  Bound by instructions (413 per position of 32 channels) and
// latency, two warps on a scheduler: 2 x 2048 channels x 2048 positions x 16 states
// in bf16 take 243 us, 54 of them the ends and 22 the joins.
#include "seq_scan.cuh"

namespace spconv {
namespace seq {
namespace {

constexpr int kBackThreads = 128, kBackWarps = kBackThreads / 32;

// A block owns 64 channels of one group of one sequence, a warp 16 of them, four
// lanes a pair of channels with SPT states of each in every lane: what is
// read of B and C serves two channels (see seq_scan.cu), and the registers
// hold four positions' states and decays.
template <int SPT_>
struct BackTile {
    static constexpr int SPT = SPT_, SP = 4 * SPT, NP = Pairs<SPT>::N;
    static constexpr int VE = SPT <= 4 ? 8 : SPT == 8 ? 4 : 2, TT = 4 * VE;
    static constexpr int Q = SPT <= 4 ? 4 : SPT == 8 ? 2 : 1;  // positions gone back at a time
    static constexpr int CW = 16, CB = CW * kBackWarps;        // channels of a warp, of a block
    static constexpr int NI = 2;  // loads of a lane from each row set
    static constexpr int NB = (2 * SP * 4 + kBackThreads - 1) / kBackThreads;  // from B and C
    // rows: one more after every VE positions, pitches that keep the writers of
    // a position's row and the pairs that read it in different banks
    static constexpr int kStepPitch = TT + 10;  // of 16 bytes {dt, dt u} of a pair
    static constexpr int kDoPitch = TT + 5;     // of 8 bytes {do} of a pair
    static constexpr int kOutPitch = TT + 4;
    static constexpr int kOutHalf = 8 * kOutPitch + 8, kOut = 2 * kOutHalf;
    static constexpr int kKept = 2 * NP * 32 * 2;  // floats: a warp's states before Q positions
    // floats of a block
    static constexpr int kMatrix = (TT + 5) * SP;
    static constexpr int kBC = 2 * kMatrix;
    static constexpr int kSteps = 8 * kStepPitch * 4;  // of a warp, from here
    static constexpr int kDo = 8 * kDoPitch * 2;
    static constexpr int kKeptAll = TT / Q * kKept;
    static constexpr int kOuts = 3 * kOut;
    static constexpr int kWarp = kSteps + kDo + kKeptAll + kOuts;
    static constexpr int kEnds = kBC + kBackWarps * (kSteps + kDo);
    static constexpr int kAll = kBC + kBackWarps * kWarp;
    static __device__ __forceinline__ int row(int t) { return t + t / VE; }
};

// Where a thread works.
template <typename T, int SPT>
struct BackPlace {
    using G = BackTile<SPT>;
    static constexpr int VE = G::VE, TT = G::TT, SP = G::SP, NI = G::NI;
    const ScanParams &p;
    int n, g, len, lane, warp, quarter, c_count;
    int64_t c_base;  // the warp's first channel
    const T *u, *d, *z, *dy, *B, *C;
    float bias[NI];
    float *bc, *steps, *dos;
    Run<T, VE> ru[NI], rd[NI], rz[NI], ry[NI];

    __device__ BackPlace(const ScanParams &p_, float *sm) : p(p_) {
        n = blockIdx.y;
        g = blockIdx.x / p.blocks_per_group;
        lane = threadIdx.x & 31;
        warp = threadIdx.x >> 5;
        quarter = lane & 3;
        const int first = (blockIdx.x - g * p.blocks_per_group) * G::CB + warp * G::CW;
        c_count = min(max(p.per_group - first, 0), G::CW);
        c_base = (int64_t)g * p.per_group + min(first, p.per_group - 1);
        len = p.lengths ? min(max(p.lengths[n], 0), p.L) : p.L;
        u = static_cast<const T *>(p.u) + n * p.u_sn + c_base * p.u_sc;
        d = static_cast<const T *>(p.delta) + n * p.d_sn + c_base * p.d_sc;
        z = p.z ? static_cast<const T *>(p.z) + n * p.z_sn + c_base * p.z_sc : nullptr;
        dy = static_cast<const T *>(p.dy) + n * p.dy_sn + c_base * p.dy_sc;
        B = static_cast<const T *>(p.B) + n * p.b_sn + g * p.b_sg;
        C = static_cast<const T *>(p.C) + n * p.c_sn + g * p.c_sg;
        bc = sm;
        steps = sm + G::kBC + warp * (G::kSteps + G::kDo);
        dos = steps + G::kSteps;
#pragma unroll
        for (int k = 0; k < NI; ++k)
            bias[k] = p.delta_bias && lane / 4 + 8 * k < c_count ? p.delta_bias[c_base + lane / 4 + 8 * k]
                                                                 : 0.f;
    }
    // Reads a tile's rows and leaves B, C, {dt, dt u} and do in shared memory;
    // behind the sequence's end, and for channels that do not exist, all are zero.
    // total: the step sizes' sums of the lane's positions.
    __device__ __forceinline__ void stage(int t0, float (&total)[NI]) {
        const int end = min(len, min(p.L - t0, TT) + t0), mine = t0 + quarter * VE;
        Run<T, VE> rows[G::NB];
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            const int c = lane / 4 + 8 * k, e = c < c_count ? end : 0;
            load_run(ru[k], u + c * p.u_sc, mine, e, p.vec);
            load_run(rd[k], d + c * p.d_sc, mine, e, p.vec);
            load_run(ry[k], dy + c * p.dy_sc, mine, e, p.vec);
            if (z) load_run(rz[k], z + c * p.z_sc, mine, e, p.vec);
        }
#pragma unroll
        for (int k = 0; k < G::NB; ++k) {
            const int i = threadIdx.x + kBackThreads * k, s = i % SP, q = (i / SP) % 4;
            const int which = i / (SP * 4);
            const T *row = which ? C + s * p.c_ss : B + s * p.b_ss;
            load_run(rows[k], row, t0 + q * VE, s < p.S && which < 2 ? end : 0, p.vec);
        }
        __syncthreads();  // the previous tile has been read
#pragma unroll
        for (int k = 0; k < G::NB; ++k) {
            const int i = threadIdx.x + kBackThreads * k, s = i % SP, q = (i / SP) % 4;
            const int which = i / (SP * 4);
            if (which >= 2) break;
            float *to = bc + which * G::kMatrix + q * (VE + 1) * SP + s;
#pragma unroll
            for (int e = 0; e < VE; ++e) to[e * SP] = rows[k][e];
        }
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            const int c = lane / 4, first = quarter * (VE + 1);
            float dt[VE], o[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                dt[e] = rd[k][e] + bias[k];
                o[e] = ry[k][e];
            }
            if (p.softplus) {
#pragma unroll
                for (int e = 0; e < VE; ++e) dt[e] = softplus(dt[e]);
            }
            if (z) {
#pragma unroll
                for (int e = 0; e < VE; ++e) o[e] *= silu(rz[k][e]);
            }
            const bool on = c + 8 * k < c_count;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                dt[e] = on && mine + e < end ? dt[e] : 0.f;
                total[k] += dt[e];
                reinterpret_cast<float2 *>(steps)[(c * G::kStepPitch + first + e) * 2 + k] =
                    make_float2(dt[e], dt[e] * ru[k][e]);
                dos[(c * G::kDoPitch + first + e) * 2 + k] = o[e];
            }
        }
        __syncthreads();
    }
};

// What a tile leaves of h from zero and a segment of g towards its start.
template <typename T, int SPT>
__global__ void __launch_bounds__(kBackThreads) segment_ends_kernel(const ScanParams p) {
    using G = BackTile<SPT>;
    constexpr int TT = G::TT, SP = G::SP, NP = G::NP, NI = G::NI;
    extern __shared__ __align__(16) float sm[];
    BackPlace<T, SPT> at(p, sm);
    const int pair = at.lane >> 2, j = at.lane & 3, s0 = j * SPT, seg = blockIdx.z;
    const float4 *step = reinterpret_cast<const float4 *>(at.steps) + pair * G::kStepPitch;
    const float2 *dos = reinterpret_cast<const float2 *>(at.dos) + pair * G::kDoPitch;
    Pairs<SPT> A[2], h[2], P[2], g[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int c = pair + 8 * q;
        A[q].load(p.A + (at.c_base + c) * p.S, s0, c < at.c_count ? p.S : 0);
        A[q].scale(kLog2e);
        P[q].fill(1.f);
        g[q].fill(0.f);
    }
    float all[NI] = {};
    const int first = seg * p.tiles_per_segment, last = min(p.tiles, first + p.tiles_per_segment);
    for (int tile = first; tile < last; ++tile) {
        float total[NI] = {};
        at.stage(tile * TT, total);
        h[0].fill(0.f);
        h[1].fill(0.f);
#pragma unroll 4
        for (int t = 0; t < TT; ++t) {
            const float4 x = step[G::row(t)];
            const float2 o = dos[G::row(t)];
            Pairs<SPT> b, c;
            b.read(at.bc + G::row(t) * SP + s0);
            c.read(at.bc + G::kMatrix + G::row(t) * SP + s0);
            const f32x2 dt[2] = {pack2(x.x, x.x), pack2(x.z, x.z)};
            const f32x2 du[2] = {pack2(x.y, x.y), pack2(x.w, x.w)};
            const f32x2 od[2] = {pack2(o.x, o.x), pack2(o.y, o.y)};
#pragma unroll
            for (int i = 0; i < NP; ++i) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const f32x2 a = decay2(dt[q], A[q].v[i]);
                    h[q].v[i] = fma2(a, h[q].v[i], mul2(du[q], b.v[i]));
                    P[q].v[i] = mul2(P[q].v[i], a);
                    g[q].v[i] = fma2(mul2(P[q].v[i], c.v[i]), od[q], g[q].v[i]);
                }
            }
        }
        const int64_t rows = ((int64_t)at.n * p.tiles + tile) * p.channels + at.c_base;
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            total[k] += __shfl_xor_sync(~0u, total[k], 1);
            total[k] += __shfl_xor_sync(~0u, total[k], 2);
            all[k] += total[k];
            const int c = at.lane / 4 + 8 * k;
            if (at.quarter == 0 && c < at.c_count) p.dt_chunk[rows + c] = total[k];
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (pair + 8 * q < at.c_count) h[q].store(p.h_chunk + (rows + pair + 8 * q) * p.S, s0, p.S);
    }
    const int64_t rows = ((int64_t)at.n * p.segments + seg) * p.channels + at.c_base;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int c = pair + 8 * q;
        if (c >= at.c_count) continue;
        g[q].store(p.g_chunk + (rows + c) * p.S, s0, p.S);
        if (j == 0) p.dt_segment[rows + c] = all[q];
    }
}

static __device__ __forceinline__ float sum4(float v) {
    v += __shfl_xor_sync(~0u, v, 1);
    return v + __shfl_xor_sync(~0u, v, 2);
}

// Sums v[position][matrix][state] over the eight pairs of a warp (lane bits 4, 3, 2): at
// each bit the lanes give half of what they hold to each other, states first,
// then the matrices, so that every lane ends with its own share of the sums
// (v[k][0 .. MATS)[0 .. N)), the first state of which is `state`, of matrix `mat`.
template <int SPT, int MATS, int N, int BIT, int Q>
struct PairSum {
    static __device__ __forceinline__ void run(float (&v)[Q][2][SPT], int lane, int &state, int &mat) {
        if constexpr (BIT >= 4) {
            const bool up = lane & BIT;
            if constexpr (N > 1) {
#pragma unroll
                for (int k = 0; k < Q; ++k)
#pragma unroll
                    for (int w = 0; w < MATS; ++w)
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) {
                            const float keep = up ? v[k][w][i + N / 2] : v[k][w][i];
                            const float give = up ? v[k][w][i] : v[k][w][i + N / 2];
                            v[k][w][i] = keep + __shfl_xor_sync(~0u, give, BIT);
                        }
                state += up ? N / 2 : 0;
                PairSum<SPT, MATS, N / 2, BIT / 2, Q>::run(v, lane, state, mat);
            } else if constexpr (MATS > 1) {
#pragma unroll
                for (int k = 0; k < Q; ++k) {
                    const float keep = up ? v[k][1][0] : v[k][0][0];
                    const float give = up ? v[k][0][0] : v[k][1][0];
                    v[k][0][0] = keep + __shfl_xor_sync(~0u, give, BIT);
                }
                mat = up;
                PairSum<SPT, 1, 1, BIT / 2, Q>::run(v, lane, state, mat);
            } else {
#pragma unroll
                for (int k = 0; k < Q; ++k) v[k][0][0] += __shfl_xor_sync(~0u, v[k][0][0], BIT);
                PairSum<SPT, 1, 1, BIT / 2, Q>::run(v, lane, state, mat);
            }
        }
    }
};
template <int SPT>
struct PairShare {  // what PairSum leaves in a lane
    static constexpr int N = SPT >= 8 ? SPT / 8 : 1, MATS = SPT >= 8 ? 2 : 1;
};

// The gradients of a segment's tiles, last tile first.
template <typename T, int SPT>
__global__ void __launch_bounds__(kBackThreads) gradient_kernel(const ScanParams p) {
    using G = BackTile<SPT>;
    constexpr int VE = G::VE, TT = G::TT, SP = G::SP, NP = G::NP, NI = G::NI, Q = G::Q;
    constexpr float kLn2 = 0.6931471805599453f;
    extern __shared__ __align__(16) float sm[];
    BackPlace<T, SPT> at(p, sm);
    const int lane = at.lane, pair = lane >> 2, j = lane & 3, s0 = j * SPT, odd = j & 1;
    float *kept_all = sm + G::kBC + kBackWarps * (G::kSteps + G::kDo);
    float *kept = kept_all + at.warp * G::kKeptAll;
    float *outs = kept_all + kBackWarps * G::kKeptAll + at.warp * G::kOuts;
    // Odd lanes hold the pair's channels the other way round: in a sum over two
    // lanes every lane keeps its first and gives its second.
    const int mine[2] = {pair + 8 * odd, pair + 8 * (odd ^ 1)};
    const float2 *step[2];
    const float *dos[2];
    Pairs<SPT> A[2], dA[2], g[2];
    const int seg = blockIdx.z;
    const int64_t seg_rows = ((int64_t)at.n * p.segments + seg) * p.channels + at.c_base;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int S = mine[q] < at.c_count ? p.S : 0;
        A[q].load(p.A + (at.c_base + mine[q]) * p.S, s0, S);
        A[q].scale(kLog2e);
        g[q].load(p.g_chunk + (seg_rows + mine[q]) * p.S, s0, S);
        dA[q].fill(0.f);
        step[q] = reinterpret_cast<const float2 *>(at.steps) + pair * G::kStepPitch * 2 + (odd ^ q);
        dos[q] = at.dos + pair * G::kDoPitch * 2 + (odd ^ q);
    }
    float D[NI], dD[NI] = {}, dbias[NI] = {};
#pragma unroll
    for (int k = 0; k < NI; ++k) {
        const int c = lane / 4 + 8 * k;
        D[k] = p.D && c < at.c_count ? p.D[at.c_base + c] : 0.f;
    }
    const int first = seg * p.tiles_per_segment, last = min(p.tiles, first + p.tiles_per_segment);
    const int64_t rows = (int64_t)at.n * p.channels + at.c_base;
    for (int tile = last - 1; tile >= first; --tile) {
        const int t0 = tile * TT;
        float unused[NI] = {};
        Pairs<SPT> h[2];
        const int64_t tile_rows = ((int64_t)at.n * p.tiles + tile) * p.channels + at.c_base;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            h[q].load(p.h_chunk + (tile_rows + mine[q]) * p.S, s0, mine[q] < at.c_count ? p.S : 0);
        at.stage(t0, unused);
        // forwards: the states before every Q positions
#pragma unroll 1
        for (int m = 0; m < TT / Q; ++m) {
            // (what the positions need is read before the states are stored: a store
            // holds later reads back)
            const int r0 = G::row(m * Q);  // (Q divides VE)
            Pairs<SPT> b[Q];
            float2 x[Q][2];
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                b[k].read(at.bc + (r0 + k) * SP + s0);
#pragma unroll
                for (int q = 0; q < 2; ++q) x[k][q] = step[q][(r0 + k) * 2];
            }
            f32x2 *to = reinterpret_cast<f32x2 *>(kept + m * G::kKept) + lane;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < NP; ++i) to[(q * NP + i) * 32] = h[q].v[i];
#pragma unroll
            for (int k = 0; k < Q; ++k) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const f32x2 dt = pack2(x[k][q].x, x[k][q].x), du = pack2(x[k][q].y, x[k][q].y);
#pragma unroll
                    for (int i = 0; i < NP; ++i)
                        h[q].v[i] = fma2(decay2(dt, A[q].v[i]), h[q].v[i], mul2(du, b[k].v[i]));
                }
            }
        }
        // back, Q positions at a time
#pragma unroll 1
        for (int m = TT / Q - 1; m >= 0; --m) {
            const int r0 = G::row(m * Q);
            f32x2 hs[Q + 1][2][NP], a[Q][2][NP];
            Pairs<SPT> b[Q], c[Q];
            float2 x[Q][2];
            float y[Q][2], of[Q][2];
            const f32x2 *from = reinterpret_cast<const f32x2 *>(kept + m * G::kKept) + lane;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < NP; ++i) hs[0][q][i] = from[(q * NP + i) * 32];
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                b[k].read(at.bc + (r0 + k) * SP + s0);
                c[k].read(at.bc + G::kMatrix + (r0 + k) * SP + s0);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    x[k][q] = step[q][(r0 + k) * 2];
                    of[k][q] = dos[q][(r0 + k) * 2];
                    const f32x2 dt = pack2(x[k][q].x, x[k][q].x), du = pack2(x[k][q].y, x[k][q].y);
                    f32x2 o = 0;
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        a[k][q][i] = decay2(dt, A[q].v[i]);
                        hs[k + 1][q][i] = fma2(a[k][q][i], hs[k][q][i], mul2(du, b[k].v[i]));
                        o = i ? fma2(hs[k + 1][q][i], c[k].v[i], o) : mul2(hs[k + 1][q][i], c[k].v[i]);
                    }
                    const float2 f = unpack2(o);
                    y[k][q] = f.x + f.y;
                }
            }
            // The sums over lanes wait for each other and the stores for them, so they
            // come behind the Q positions, those of all positions side by side.
            float s1[Q][2], s2[Q][2], v[Q][2][SPT];
#pragma unroll
            for (int k = Q - 1; k >= 0; --k) {
                f32x2 vB[NP], vC[NP];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const f32x2 o = pack2(of[k][q], of[k][q]), du = pack2(x[k][q].y, x[k][q].y);
                    const f32x2 dt = pack2(x[k][q].x, x[k][q].x);
                    f32x2 gB = 0, qA = 0;
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        const f32x2 now = fma2(c[k].v[i], o, g[q].v[i]);
                        vC[i] = q ? fma2(o, hs[k + 1][q][i], vC[i]) : mul2(o, hs[k + 1][q][i]);
                        vB[i] = q ? fma2(du, now, vB[i]) : mul2(du, now);
                        gB = i ? fma2(now, b[k].v[i], gB) : mul2(now, b[k].v[i]);
                        g[q].v[i] = mul2(now, a[k][q][i]);
                        const f32x2 w = mul2(g[q].v[i], hs[k][q][i]);
                        qA = i ? fma2(w, A[q].v[i], qA) : mul2(w, A[q].v[i]);
                        dA[q].v[i] = fma2(w, dt, dA[q].v[i]);
                    }
                    const float2 f1 = unpack2(gB), f2 = unpack2(qA);
                    s1[k][q] = f1.x + f1.y;
                    s2[k][q] = f2.x + f2.y;
                }
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const float2 fB = unpack2(vB[i]), fC = unpack2(vC[i]);
                    v[k][0][2 * i < SPT ? 2 * i : 0] = fB.x;
                    v[k][1][2 * i < SPT ? 2 * i : 0] = fC.x;
                    if constexpr (SPT > 1) {
                        v[k][0][2 * i + 1] = fB.y;
                        v[k][1][2 * i + 1] = fC.y;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                y[k][0] += __shfl_xor_sync(~0u, y[k][1], 1);
                s1[k][0] += __shfl_xor_sync(~0u, s1[k][1], 1);
                s2[k][0] += __shfl_xor_sync(~0u, s2[k][1], 1);
            }
            float share[Q];  // lanes 0, 1 of the pair end with g . B, lanes 2, 3 with q . A
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                y[k][0] += __shfl_xor_sync(~0u, y[k][0], 2);
                share[k] = (j & 2 ? s2[k][0] : s1[k][0]) +
                           __shfl_xor_sync(~0u, j & 2 ? s1[k][0] : s2[k][0], 2);
            }
            int state = s0, mat = 0;
            PairSum<SPT, 2, SPT, 16, Q>::run(v, lane, state, mat);
            __syncwarp();  // the kept states of all lanes have been read: their place is used again
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                float *to = kept + m * G::kKept + k * 2 * SP + mat * SP + state;
#pragma unroll
                for (int w = 0; w < PairShare<SPT>::MATS; ++w)
#pragma unroll
                    for (int i = 0; i < PairShare<SPT>::N; ++i) to[w * SP + i] = v[k][w][i];
            }
            float *out = outs + odd * G::kOutHalf + pair * G::kOutPitch + m * Q;
            if (j < 2) {
#pragma unroll
                for (int k = 0; k < Q; ++k) out[k] = y[k][0];
            }
            float *sums = outs + (1 + (j >> 1)) * G::kOut + odd * G::kOutHalf + pair * G::kOutPitch + m * Q;
#pragma unroll
            for (int k = 0; k < Q; ++k) sums[k] = share[k];
        }
        __syncwarp();
        // the rows that the lane read: dz, du, ddelta
        const int stop = t0 + min(p.L - t0, TT), end = min(at.len, stop);
        const int t_lane = at.quarter * VE;
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            const int c = lane / 4, place = k * G::kOutHalf + c * G::kOutPitch + t_lane;
            const bool on = c + 8 * k < at.c_count;
            const int64_t row = (rows + c + 8 * k) * p.L;
            float wz[VE], wu[VE], wd[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const bool in = on && t0 + t_lane + e < end;
                const float uu = at.ru[k][e], raw = at.rd[k][e] + at.bias[k];
                const float dt = reinterpret_cast<const float2 *>(
                    at.steps)[(c * G::kStepPitch + t_lane + at.quarter + e) * 2 + k].x;
                const float o = at.dos[(c * G::kDoPitch + t_lane + at.quarter + e) * 2 + k];
                const float gB = outs[G::kOut + place + e], qA = outs[2 * G::kOut + place + e];
                float ddt = fmaf(gB, uu, qA * kLn2);
                if (p.softplus) ddt *= sigmoid(raw);
                wd[e] = in ? ddt : 0.f;
                wu[e] = in ? fmaf(gB, dt, D[k] * o) : 0.f;
                dbias[k] += wd[e];
                dD[k] = fmaf(o, uu, dD[k]);
                if (at.z)
                    wz[e] = in ? at.ry[k][e] * fmaf(D[k], uu, outs[place + e]) * silu_grad(at.rz[k][e])
                               : 0.f;
            }
            if (on) {
                Run<T, VE> r;
                r.put(wu);
                store_run(r, static_cast<T *>(p.du) + row, t0 + t_lane, stop, p.vec_y);
                r.put(wd);
                store_run(r, static_cast<T *>(p.ddelta) + row, t0 + t_lane, stop, p.vec_y);
                if (at.z) {
                    r.put(wz);
                    store_run(r, static_cast<T *>(p.dz) + row, t0 + t_lane, stop, p.vec_y);
                }
            }
        }
        // this block's share of dB and dC: the warps' in their order
        __syncthreads();
        const int64_t share_rows = ((int64_t)blockIdx.x * p.N + at.n) * p.L + t0;
        const int64_t matrix = (int64_t)gridDim.x * p.N * p.L * p.S;
        for (int i = threadIdx.x; i < TT * 2 * SP; i += kBackThreads) {
            const int t = i / (2 * SP), r = i % (2 * SP), s = r % SP;
            const float *q = kept_all + t / Q * G::kKept + t % Q * (2 * SP) + r;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kBackWarps; ++w) v += q[w * G::kKeptAll];
            if (s < p.S && t0 + t < stop) p.part_bc[r / SP * matrix + (share_rows + t) * p.S + s] = v;
        }
    }
    const int64_t part = ((int64_t)at.n * p.segments + seg) * p.channels + at.c_base;
#pragma unroll
    for (int q = 0; q < 2; ++q)
        if (mine[q] < at.c_count) dA[q].store(p.part_a + (part + mine[q]) * (p.S + 2), s0, p.S);
#pragma unroll
    for (int k = 0; k < NI; ++k) {
        dD[k] = sum4(dD[k]);
        dbias[k] = sum4(dbias[k]);
        const int c = lane / 4 + 8 * k;
        if (at.quarter == 0 && c < at.c_count) {
            p.part_a[(part + c) * (p.S + 2) + p.S] = dD[k];
            p.part_a[(part + c) * (p.S + 2) + p.S + 1] = dbias[k];
        }
    }
}

// Joins the blocks' shares in their order.  The first `weight_blocks` blocks take
// dA, dD and ddelta_bias, the shares of segments; the others dB and dC, the
// shares of blocks, [position][state] to [state][position].
template <typename T>
__global__ void __launch_bounds__(256) join_shares_kernel(const ScanParams p, int weight_blocks) {
    if ((int)blockIdx.x < weight_blocks) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        const int64_t per = (int64_t)p.channels * (p.S + 2);
        if (i >= per) return;
        float v = 0.f;
        const int64_t count = (int64_t)p.N * p.segments;
#pragma unroll 4
        for (int64_t k = 0; k < count; ++k) v += p.part_a[k * per + i];
        const int64_t c = i / (p.S + 2);
        const int s = (int)(i - c * (p.S + 2));
        if (s < p.S)
            p.dA[c * p.S + s] = v;
        else if (s == p.S) {
            if (p.dD) p.dD[c] = v;
        } else if (p.ddelta_bias) {
            p.ddelta_bias[c] = v;
        }
        return;
    }
    const int64_t per = (int64_t)p.N * p.L * p.S;  // of one block and matrix
    const int64_t i = (int64_t)(blockIdx.x - weight_blocks) * 256 + threadIdx.x;
    const int blocks = p.groups * p.blocks_per_group;
    if (i >= 2 * p.groups * per) return;
    const int64_t k = i / per, r = i - k * per;
    const int which = (int)(k / p.groups), g = (int)(k - which * p.groups);
    float v = 0.f;
#pragma unroll 4
    for (int b = 0; b < p.blocks_per_group; ++b)
        v += p.part_bc[((int64_t)which * blocks + g * p.blocks_per_group + b) * per + r];
    const int64_t nt = r / p.S, n = nt / p.L, t = nt - n * p.L;
    const int s = (int)(r - nt * p.S);
    T *to = static_cast<T *>(which ? p.dC : p.dB);
    to[((n * p.groups + g) * p.S + s) * p.L + t] = from_f32<T>(v);
}

struct Layout {
    int64_t h, g, dt, dts, bc, a, total;  // float offsets
};

// Sizes of the backward pass for these arguments: tiles, segments and where
// the workspace's parts start.
Layout plan(ScanParams &p) {
    const int tt = p.S <= 16 ? 32 : p.S <= 32 ? 16 : 8;
    p.blocks_per_group = (p.per_group + 63) / 64;
    p.tiles = (p.L + tt - 1) / tt;
    const int64_t blocks = (int64_t)p.groups * p.blocks_per_group;
    // tiles of a segment: two blocks fit an SM, and the blocks run in waves, so
    // the time goes by waves x tiles; of equals the longest (it has the fewest shares
    // of dA and the fewest of g's states)
    int64_t best = 0;
    p.tiles_per_segment = 8;
    p.segments = (p.tiles + 7) / 8;
    for (int per = 1; per <= 8 && per <= p.tiles; ++per) {
        const int64_t segments = (p.tiles + per - 1) / per;
        if (segments > 65535) continue;  // they go along grid z
        const int64_t waves = (blocks * p.N * segments + 2 * kSMs - 1) / (2 * kSMs);
        if (best && waves * per > best) continue;
        best = waves * per;
        p.tiles_per_segment = per;
        p.segments = (int)segments;
    }
    auto up = [](int64_t v) { return (v + 3) / 4 * 4; };
    const int64_t rows = (int64_t)p.N * p.channels;
    Layout l;
    l.h = 0;
    l.g = l.h + up(rows * p.tiles * p.S);
    l.dt = l.g + up(rows * p.segments * p.S);
    l.dts = l.dt + up(rows * p.tiles);
    l.bc = l.dts + up(rows * p.segments);
    l.a = l.bc + up(2 * blocks * p.N * p.L * p.S);
    l.total = l.a + up(rows * p.segments * (p.S + 2));
    return l;
}

}  // namespace
}  // namespace seq
}  // namespace spconv

using namespace spconv::seq;

SPCONV_API int64_t spconv_scan_backward_workspace(const spconv_scan_args *a) {
    if (scan_check_sizes(a) || a->channels == 0 || a->N == 0 || a->L == 0) return 0;
    ScanParams p = scan_params(a);
    return plan(p).total * 4;
}

SPCONV_API int spconv_scan_backward(const spconv_scan_args *a, void *stream) {
    const int st = scan_check_sizes(a);
    if (st) return st;
    if (a->N > 65535) return SPCONV_ERR_UNSUPPORTED;  // sequences go along grid y
    const int64_t rows = (int64_t)a->N * a->channels, L = a->L;
    const size_t e = dtype_size(a->dtype);
    const int64_t bcb = (int64_t)a->N * a->groups * a->S * L * e;
    if (a->channels == 0) {  // dB and dC are sums over no channel
        if (bcb == 0) return SPCONV_OK;
        if (!a->dB || !a->dC || !aligned(a->dB, e) || !aligned(a->dC, e) ||
            overlap(a->dB, bcb, a->dC, bcb))
            return SPCONV_ERR_INVALID_ARG;
        const bool ok = cudaMemsetAsync(a->dB, 0, bcb, static_cast<cudaStream_t>(stream)) == cudaSuccess &&
                        cudaMemsetAsync(a->dC, 0, bcb, static_cast<cudaStream_t>(stream)) == cudaSuccess;
        if (!ok) cudaGetLastError();
        return ok ? SPCONV_OK : SPCONV_ERR_CUDA;
    }
    const bool any = rows > 0 && L > 0;
    if (!a->A || !a->dA) return SPCONV_ERR_INVALID_ARG;
    if (any && (!a->u || !a->delta || !a->B || !a->C || !a->dy || !a->du || !a->ddelta || !a->dB ||
                !a->dC || !a->z != !a->dz))
        return SPCONV_ERR_INVALID_ARG;
    for (const void *q : {a->u, a->delta, a->z, a->B, a->C, a->dy, (const void *)a->du,
                          (const void *)a->ddelta, (const void *)a->dz, (const void *)a->dB,
                          (const void *)a->dC})
        if (!aligned(q, e)) return SPCONV_ERR_INVALID_ARG;
    for (const void *q : {(const void *)a->A, (const void *)a->D, (const void *)a->delta_bias,
                          (const void *)a->state, (const void *)a->lengths,
                          (const void *)a->dfinal_state, (const void *)a->dA, (const void *)a->dD,
                          (const void *)a->ddelta_bias, (const void *)a->dstate})
        if (!aligned(q, 4)) return SPCONV_ERR_INVALID_ARG;
    const int64_t need = spconv_scan_backward_workspace(a);
    if (need && (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < need))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t act = rows * L * e, sb = rows * a->S * 4;
    const int64_t bb = L ? extent(a->N, a->groups, (a->S - 1) * a->b_stride_s + L, a->b_stride_n, a->b_stride_g, e) : 0;
    const int64_t cb = L ? extent(a->N, a->groups, (a->S - 1) * a->c_stride_s + L, a->c_stride_n, a->c_stride_g, e) : 0;
    const int64_t ab = a->channels * 4LL * a->S, per = a->channels * 4LL;
    if (!apart({{a->du, act}, {a->ddelta, act}, {a->dz, act}, {a->dB, bcb}, {a->dC, bcb}, {a->dstate, sb},
                {a->dA, ab}, {a->dD, per}, {a->ddelta_bias, per}, {a->workspace, need}},
               {{a->u, extent(a->N, a->channels, L, a->u_stride_n, a->u_stride_c, e)},
                {a->delta, extent(a->N, a->channels, L, a->delta_stride_n, a->delta_stride_c, e)},
                {a->z, extent(a->N, a->channels, L, a->z_stride_n, a->z_stride_c, e)},
                {a->dy, extent(a->N, a->channels, L, a->dy_stride_n, a->dy_stride_c, e)},
                {a->B, bb}, {a->C, cb}, {a->state, sb}, {a->dfinal_state, sb}, {a->lengths, a->N * 4LL},
                {a->A, ab}, {a->D, per}, {a->delta_bias, per}}))
        return SPCONV_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ScanParams p = scan_params(a);
    if (!any) {
        // no position: the weights' gradients are zero, the initial state's is
        // the final state's
        auto zero = [&](float *to, int64_t count) {
            return !to || !count || cudaMemsetAsync(to, 0, count * 4, s) == cudaSuccess;
        };
        bool ok = zero(a->dA, (int64_t)a->channels * a->S) && zero(a->dD, a->channels) &&
                  zero(a->ddelta_bias, a->channels);
        if (ok && a->dstate && sb)
            ok = a->dfinal_state ? cudaMemcpyAsync(a->dstate, a->dfinal_state, sb,
                                                   cudaMemcpyDeviceToDevice, s) == cudaSuccess
                                 : zero(a->dstate, sb / 4);
        if (!ok) cudaGetLastError();
        return ok ? SPCONV_OK : SPCONV_ERR_CUDA;
    }
    const Layout l = plan(p);
    float *ws = static_cast<float *>(a->workspace);
    p.h_chunk = ws + l.h; p.g_chunk = ws + l.g; p.dt_chunk = ws + l.dt; p.dt_segment = ws + l.dts;
    p.part_bc = ws + l.bc; p.part_a = ws + l.a;
    p.vec_y = rows_aligned(a->du, 0, L, e) && rows_aligned(a->ddelta, 0, L, e) &&
              (!a->dz || rows_aligned(a->dz, 0, L, e));
    const int64_t weights = (int64_t)p.channels * (p.S + 2), bc = 2LL * p.groups * p.N * L * p.S;
    if (p.segments > 65535 || (weights + bc + 511) / 256 > 0x7fffffff) return SPCONV_ERR_UNSUPPORTED;
    return by_dtype(a->dtype, [&](auto t) {
        return by_states(a->S, [&](auto k) {
            using T = decltype(t);
            constexpr int SPT = decltype(k)::value;
            using G = BackTile<SPT>;
            static_assert(G::kAll * 4 <= 227 * 1024, "a tile fits shared memory");
            const dim3 grid(p.groups * p.blocks_per_group, p.N, p.segments);
            auto *ends = segment_ends_kernel<T, SPT>;
            auto *grad = gradient_kernel<T, SPT>;
            if (int rc = raise_smem(reinterpret_cast<const void *>(ends), G::kEnds * 4)) return rc;
            if (int rc = raise_smem(reinterpret_cast<const void *>(grad), G::kAll * 4)) return rc;
            ends<<<grid, kBackThreads, G::kEnds * 4, s>>>(p);
            if (int rc = launch_status()) return rc;
            if (int rc = scan_join_chunks(p, true, s)) return rc;
            grad<<<grid, kBackThreads, G::kAll * 4, s>>>(p);
            if (int rc = launch_status()) return rc;
            const int64_t first = (weights + 255) / 256;
            join_shares_kernel<T><<<(unsigned)(first + (bc + 255) / 256), 256, 0, s>>>(p, (int)first);
            return launch_status();
        });
    });
}
