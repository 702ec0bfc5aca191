// Gradients of the selective state space scan.
//
// With do_t = dy_t silu(z_t) and g_t the gradient that reaches h_t,
//
//   g_t = C_t do_t + a_(t+1) g_(t+1),  a_t = e^(dt A)
//   dz = dy o silu'(z),  dC_t = sum_c do_t h_t,  dB_t = sum_c g_t dt u
//   q_t = a_t g_t h_(t-1),  ddt = u (g_t . B_t) + sum_s q_t A,  dA = sum q_t dt
//   du = dt (g_t . B_t) + D do_t,  dD = sum do_t u,  ddelta = ddt sigmoid(raw)
//
// Both recurrences are cut into chunks of one tile.  One kernel finds what
// every chunk leaves of h from zero and of g towards its start; one joins the
// chunks over the sequence; one forms every chunk's gradients from the states
// that it starts and ends with, its h_t held in shared memory between its run
// forwards and its run back.  So all chunks run side by side and no state is
// kept by the forward call: the states cost two numbers per chunk of
// traffic, not one per position.  Sums over channels, sequences and chunks
// are joined from the blocks' shares in a fixed order.
#include <utility>

#include "seq_scan.cuh"

namespace spconv {
namespace seq {
namespace {

// Positions of a lane in a tile: the tile's h_t, 32 channels of 4 * SPT states,
// have to fit shared memory.
constexpr int run_of(int SPT) { return SPT <= 4 ? 8 : SPT == 8 ? 4 : 2; }

template <int SPT>
struct BackTile {
    static constexpr int VE = run_of(SPT), TT = 4 * VE, SP = 4 * SPT;
    // words of one position's states; 16 more than the channels need, so that
    // neighbouring positions start in different banks
    static constexpr int kHRow = kScanChannels * SP + 16;
    static constexpr int kPitch = TT + 4;
};

// What a chunk leaves: h from zero, the gradient of its start, its decay.
template <typename T, int SPT>
__global__ void __launch_bounds__(kScanThreads) chunk_ends_kernel(const ScanParams p) {
    using G = BackTile<SPT>;
    constexpr int VE = G::VE, TT = G::TT, SP = G::SP;
    __shared__ __align__(16) float bc[2 * TT * SP];
    __shared__ __align__(16) float4 xs[kScanChannels][TT + 1];  // dt, dt u, do
    const int ch = threadIdx.x >> 2, j = threadIdx.x & 3, s0 = j * SPT;
    const int chunk = blockIdx.z;
    const ScanPlace at(p, blockIdx.y, blockIdx.x);
    const int t0 = chunk * TT;
    const int end = max(min(at.len, t0 + TT), t0), row_end = at.valid ? end : 0;
    const int64_t slot = (int64_t)at.n * p.chunks + chunk;
    float h[SPT], g[SPT];
#pragma unroll
    for (int i = 0; i < SPT; ++i) h[i] = g[i] = 0.f;
    float total = 0.f;
    if (t0 < end) {
        const T *ur = static_cast<const T *>(p.u) + at.n * p.u_sn + at.c * p.u_sc;
        const T *dr = static_cast<const T *>(p.delta) + at.n * p.d_sn + at.c * p.d_sc;
        const T *zr = p.z ? static_cast<const T *>(p.z) + at.n * p.z_sn + at.c * p.z_sc : nullptr;
        const T *yr = static_cast<const T *>(p.dy) + at.n * p.dy_sn + at.c * p.dy_sc;
        Run<T, VE> u, d, z, dy;
        load_run(u, ur, t0 + j * VE, row_end, p.vec);
        load_run(d, dr, t0 + j * VE, row_end, p.vec);
        load_run(dy, yr, t0 + j * VE, row_end, p.vec);
        if (zr) load_run(z, zr, t0 + j * VE, row_end, p.vec);
        ScanBC<T, SPT, VE> rows;
        rows.load(p, at, t0, end);
        const float bias = p.delta_bias ? p.delta_bias[at.c] : 0.f;
        float A[SPT], P[SPT];
        load_states<SPT>(A, p.A + (int64_t)at.c * p.S, s0, p.S);
#pragma unroll
        for (int i = 0; i < SPT; ++i) {
            A[i] *= kLog2e;
            P[i] = 1.f;
        }
        rows.store(bc);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const float dt = t0 + j * VE + e < row_end ? step_size(p, d[e] + bias) : 0.f;
            float o = dy[e];
            if (zr) o *= silu(z[e]);
            xs[ch][j * VE + e] = make_float4(dt, dt * u[e], o, 0.f);
        }
        __syncthreads();
#pragma unroll 4
        for (int t = 0; t < TT; ++t) {
            const float4 x = xs[ch][t];
            total += x.x;
            float b[SPT], c[SPT];
            read_states<SPT>(b, bc + t * SP + s0);
            read_states<SPT>(c, bc + (TT + t) * SP + s0);
#pragma unroll
            for (int i = 0; i < SPT; ++i) {
                const float a = ex2(x.x * A[i]);
                h[i] = fmaf(a, h[i], x.y * b[i]);
                P[i] *= a;
                g[i] = fmaf(P[i] * c[i], x.z, g[i]);
            }
        }
    }
    if (!at.valid) return;
    const int64_t to = (slot * p.channels + at.c) * p.S;
    store_states<SPT>(p.h_chunk + to, h, s0, p.S);
    store_states<SPT>(p.g_chunk + to, g, s0, p.S);
    if (j == 0) p.dt_chunk[slot * p.channels + at.c] = total;
}

static __device__ __forceinline__ float sum4(float v) {
    v += __shfl_xor_sync(~0u, v, 1);
    return v + __shfl_xor_sync(~0u, v, 2);
}

// Shared memory of the gradient kernel, in floats.
template <int SPT>
constexpr int gradient_smem() {
    using G = BackTile<SPT>;
    return G::TT * G::kHRow + 2 * G::TT * G::SP + kScanChannels * (2 * (G::TT + 2) + 2 * G::kPitch);
}

// The gradients of a segment's chunks, last chunk first.
template <typename T, int SPT>
__global__ void __launch_bounds__(kScanThreads) gradient_kernel(const ScanParams p) {
    using G = BackTile<SPT>;
    constexpr int VE = G::VE, TT = G::TT, SP = G::SP;
    extern __shared__ __align__(16) float sm[];
    float *hb = sm;                       // [TT][kHRow]: h_t, then g_t
    float *bc = hb + TT * G::kHRow;       // [2][TT][SP]
    const int ch = threadIdx.x >> 2, j = threadIdx.x & 3, s0 = j * SPT;
    float *dob_all = bc + 2 * TT * SP;    // [channel][kPitch]
    float *dob = dob_all + ch * G::kPitch;
    float *yb = dob_all + kScanChannels * G::kPitch + ch * G::kPitch;
    float *dtu_all = dob_all + 2 * kScanChannels * G::kPitch;  // [channel][TT + 2] of {dt, dt u}
    float2 *dtu = reinterpret_cast<float2 *>(dtu_all) + ch * (TT + 2);

    const int cb = blockIdx.x, seg = blockIdx.z;
    const ScanPlace at(p, blockIdx.y, cb);
    const int64_t row = (int64_t)at.n * p.channels + at.c;
    const T *ur = static_cast<const T *>(p.u) + at.n * p.u_sn + at.c * p.u_sc;
    const T *dr = static_cast<const T *>(p.delta) + at.n * p.d_sn + at.c * p.d_sc;
    const T *zr = p.z ? static_cast<const T *>(p.z) + at.n * p.z_sn + at.c * p.z_sc : nullptr;
    const T *yr = static_cast<const T *>(p.dy) + at.n * p.dy_sn + at.c * p.dy_sc;
    const float bias = p.delta_bias ? p.delta_bias[at.c] : 0.f, D = p.D ? p.D[at.c] : 0.f;
    float A[SPT], dA[SPT], dD = 0.f, dbias = 0.f;
    load_states<SPT>(A, p.A + (int64_t)at.c * p.S, s0, p.S);
#pragma unroll
    for (int i = 0; i < SPT; ++i) dA[i] = 0.f;

    const int first = seg * p.chunks_per_segment;
    const int last = min(p.chunks, first + p.chunks_per_segment) - 1;
    for (int chunk = last; chunk >= first; --chunk) {
        const int t0 = chunk * TT, stop = min(p.L, t0 + TT);
        const int end = max(min(at.len, stop), t0), row_end = at.valid ? end : 0;
        const int mine = t0 + j * VE;
        const int64_t place = (((int64_t)at.n * p.chunks + chunk) * p.channels + at.c) * p.S;
        Run<T, VE> u, d, z, dy;
        load_run(u, ur, mine, row_end, p.vec);
        load_run(d, dr, mine, row_end, p.vec);
        load_run(dy, yr, mine, row_end, p.vec);
        if (zr) load_run(z, zr, mine, row_end, p.vec);
        ScanBC<T, SPT, VE> rows;
        rows.load(p, at, t0, end);
        float h0[SPT], g[SPT], h[SPT];
        load_states<SPT>(h0, p.h_chunk + place, s0, at.valid ? p.S : 0);
        load_states<SPT>(g, p.g_chunk + place, s0, at.valid ? p.S : 0);
        __syncthreads();  // the previous chunk's last reads of shared memory
        rows.store(bc);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const float dt = mine + e < row_end ? step_size(p, d[e] + bias) : 0.f;
            float o = dy[e];
            if (zr) o *= silu(z[e]);
            dtu[j * VE + e] = make_float2(dt, dt * u[e]);
            dob[j * VE + e] = o;
            dD = fmaf(o, u[e], dD);
        }
        __syncthreads();
        // forwards: h_t of every position, and o without D u
#pragma unroll
        for (int i = 0; i < SPT; ++i) h[i] = h0[i];
        float *mine_h = hb + ch * SP + s0;
#pragma unroll 4
        for (int t = 0; t < TT; ++t) {
            const float2 x = dtu[t];
            float b[SPT], c[SPT], o = 0.f;
            read_states<SPT>(b, bc + t * SP + s0);
            read_states<SPT>(c, bc + (TT + t) * SP + s0);
#pragma unroll
            for (int i = 0; i < SPT; ++i) {
                h[i] = fmaf(ex2(x.x * (A[i] * kLog2e)), h[i], x.y * b[i]);
                o = fmaf(h[i], c[i], o);
            }
            write_states<SPT>(mine_h + t * G::kHRow, h);
            o = sum4(o);
            if (j == 0) yb[t] = o;
        }
        __syncthreads();
        // dz, and this block's share of dC
        if (zr) {
            float w[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float o = fmaf(D, u[e], yb[j * VE + e]);
                w[e] = mine + e < end ? dy[e] * o * silu_grad(z[e]) : 0.f;
            }
            Run<T, VE> out;
            out.put(w);
            if (at.valid) store_run(out, static_cast<T *>(p.dz) + row * p.L, mine, stop, p.vec_y);
        }
        // over = the sum over the block's channels of w(channel, t) * hb[t][channel][s]
        auto over_channels = [&](auto w, int which) {
            const int64_t base = ((((int64_t)which * gridDim.x + cb) * p.N + at.n) * p.L + t0) * p.S;
            for (int i = threadIdx.x; i < TT * SP; i += kScanThreads) {
                const int t = i / SP, s = i % SP;
                float v = 0.f;
#pragma unroll 8
                for (int k = 0; k < kScanChannels; ++k)
                    v = fmaf(w(k, t), hb[t * G::kHRow + k * SP + s], v);
                if (s < p.S && t0 + t < stop) p.part_bc[base + (int64_t)t * p.S + s] = v;
            }
        };
        over_channels([&](int k, int t) { return dob_all[k * G::kPitch + t]; }, 1);
        __syncthreads();
        // back: g_t in the place of h_t
        float sums[2][VE];  // of the lane's own positions: g . B and q . A
#pragma unroll
        for (int t = TT - 1; t >= 0; --t) {
            const float2 x = dtu[t];
            const float o = dob[t];
            float b[SPT], c[SPT], before[SPT], sb = 0.f, sa = 0.f;
            read_states<SPT>(b, bc + t * SP + s0);
            read_states<SPT>(c, bc + (TT + t) * SP + s0);
            if (t > 0)
                read_states<SPT>(before, mine_h + (t - 1) * G::kHRow);
            else
#pragma unroll
                for (int i = 0; i < SPT; ++i) before[i] = h0[i];
            float now[SPT];
#pragma unroll
            for (int i = 0; i < SPT; ++i) {
                now[i] = fmaf(c[i], o, g[i]);
                sb = fmaf(now[i], b[i], sb);
                g[i] = now[i] * ex2(x.x * (A[i] * kLog2e));
                const float q = g[i] * before[i];
                sa = fmaf(q, A[i], sa);
                dA[i] = fmaf(q, x.x, dA[i]);
            }
            write_states<SPT>(mine_h + t * G::kHRow, now);
            sb = sum4(sb);
            sa = sum4(sa);
            if (t / VE == j) {
                sums[0][t % VE] = sb;
                sums[1][t % VE] = sa;
            }
        }
        {
            float wu[VE], wd[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float raw = d[e] + bias, uu = u[e];
                const float dt = dtu[j * VE + e].x;
                const bool in = mine + e < end;
                float ddt = fmaf(sums[0][e], uu, sums[1][e]);
                if (p.softplus) ddt *= sigmoid(raw);
                ddt = in ? ddt : 0.f;
                dbias += at.valid ? ddt : 0.f;
                wd[e] = ddt;
                wu[e] = in ? fmaf(sums[0][e], dt, D * dob[j * VE + e]) : 0.f;
            }
            Run<T, VE> du, dd;
            du.put(wu);
            dd.put(wd);
            if (at.valid) {
                store_run(du, static_cast<T *>(p.du) + row * p.L, mine, stop, p.vec_y);
                store_run(dd, static_cast<T *>(p.ddelta) + row * p.L, mine, stop, p.vec_y);
            }
        }
        __syncthreads();
        over_channels([&](int k, int t) { return dtu_all[(k * (TT + 2) + t) * 2 + 1]; }, 0);
    }
    dD = sum4(dD);
    dbias = sum4(dbias);
    if (!at.valid) return;
    float *to = p.part_a + (((int64_t)at.n * p.segments + seg) * p.channels + at.c) * (p.S + 2);
    store_states<SPT>(to, dA, s0, p.S);
    if (j == 0) {
        to[p.S] = dD;
        to[p.S + 1] = dbias;
    }
}

// dA, dD and ddelta_bias: the segments' shares in their order.
__global__ void __launch_bounds__(256) join_weights_kernel(const ScanParams p) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t per = (int64_t)p.channels * (p.S + 2);
    if (i >= per) return;
    float v = 0.f;
    for (int64_t k = 0; k < (int64_t)p.N * p.segments; ++k) v += p.part_a[k * per + i];
    const int64_t c = i / (p.S + 2);
    const int s = (int)(i - c * (p.S + 2));
    if (s < p.S)
        p.dA[c * p.S + s] = v;
    else if (s == p.S) {
        if (p.dD) p.dD[c] = v;
    } else if (p.ddelta_bias) {
        p.ddelta_bias[c] = v;
    }
}

// dB and dC: the blocks' shares in their order, [position][state] to
// [state][position].
template <typename T>
__global__ void __launch_bounds__(256) join_bc_kernel(const ScanParams p) {
    const int64_t per = (int64_t)p.N * p.L * p.S;  // of one block and matrix
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int blocks = p.groups * p.blocks_per_group;
    if (i >= 2 * p.groups * per) return;
    const int64_t k = i / per, r = i - k * per;
    const int which = (int)(k / p.groups), g = (int)(k - which * p.groups);
    float v = 0.f;
    for (int b = 0; b < p.blocks_per_group; ++b)
        v += p.part_bc[((int64_t)which * blocks + g * p.blocks_per_group + b) * per + r];
    const int64_t nt = r / p.S, n = nt / p.L, t = nt - n * p.L;
    const int s = (int)(r - nt * p.S);
    T *to = static_cast<T *>(which ? p.dC : p.dB);
    to[((n * p.groups + g) * p.S + s) * p.L + t] = from_f32<T>(v);
}

struct Layout {
    int64_t h, g, dt, bc, a, total;  // float offsets
};

// Sizes of the backward pass for these arguments: chunks, segments and where
// the workspace's parts start.
Layout plan(ScanParams &p) {
    const int tt = p.S <= 16 ? 32 : p.S <= 32 ? 16 : 8;
    p.chunks = (p.L + tt - 1) / tt;
    p.chunk_len = tt;
    const int64_t blocks = (int64_t)p.groups * p.blocks_per_group;
    // chunks of a segment: as few shares of dA as leave eight blocks per SM
    int64_t per = blocks * p.N * p.chunks / (8 * kSMs);
    per = per < 1 ? 1 : per > 16 ? 16 : per;
    p.chunks_per_segment = (int)per;
    p.segments = (int)((p.chunks + per - 1) / per);
    auto up = [](int64_t v) { return (v + 3) / 4 * 4; };
    Layout l;
    l.h = 0;
    l.g = l.h + up((int64_t)p.N * p.chunks * p.channels * p.S);
    l.dt = l.g + up((int64_t)p.N * p.chunks * p.channels * p.S);
    l.bc = l.dt + up((int64_t)p.N * p.chunks * p.channels);
    l.a = l.bc + up(2 * blocks * p.N * p.L * p.S);
    l.total = l.a + up((int64_t)p.N * p.segments * p.channels * (p.S + 2));
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
    if (a->channels == 0) return SPCONV_OK;
    const int64_t rows = (int64_t)a->N * a->channels, L = a->L;
    const size_t e = dtype_size(a->dtype);
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
    const int64_t act = rows * L * e, sb = rows * a->S * 4, bcb = (int64_t)a->N * a->groups * a->S * L * e;
    using Span = std::pair<const void *, int64_t>;
    const Span in[] = {
        {a->u, extent(a->N, a->channels, L, a->u_stride_n, a->u_stride_c, e)},
        {a->delta, extent(a->N, a->channels, L, a->delta_stride_n, a->delta_stride_c, e)},
        {a->z, extent(a->N, a->channels, L, a->z_stride_n, a->z_stride_c, e)},
        {a->dy, extent(a->N, a->channels, L, a->dy_stride_n, a->dy_stride_c, e)},
        {a->B, extent(a->N, a->groups, (a->S - 1) * a->b_stride_s + L, a->b_stride_n, a->b_stride_g, e)},
        {a->C, extent(a->N, a->groups, (a->S - 1) * a->c_stride_s + L, a->c_stride_n, a->c_stride_g, e)},
        {a->state, sb},
        {a->dfinal_state, sb}};
    const Span out[] = {{a->du, act}, {a->ddelta, act}, {a->dz, act}, {a->dB, bcb}, {a->dC, bcb}, {a->dstate, sb}};
    for (const Span &o : out)
        for (const Span &i : in)
            if (overlap(o.first, o.second, i.first, i.second)) return SPCONV_ERR_INVALID_ARG;
    for (int i = 0; i < 6; ++i)
        for (int k = 0; k < i; ++k)
            if (overlap(out[i].first, out[i].second, out[k].first, out[k].second))
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
    p.h_chunk = ws + l.h; p.g_chunk = ws + l.g; p.dt_chunk = ws + l.dt;
    p.part_bc = ws + l.bc; p.part_a = ws + l.a;
    p.vec_y = rows_aligned(a->du, 0, L, e) && rows_aligned(a->ddelta, 0, L, e) &&
              (!a->dz || rows_aligned(a->dz, 0, L, e));
    const int64_t weights = (int64_t)p.channels * (p.S + 2), bc = 2LL * p.groups * p.N * L * p.S;
    if (p.chunks > 65535 || (bc + 255) / 256 > 0x7fffffff) return SPCONV_ERR_UNSUPPORTED;
    return by_dtype(a->dtype, [&](auto t) {
        return by_states(a->S, [&](auto k) {
            using T = decltype(t);
            constexpr int SPT = decltype(k)::value, smem = gradient_smem<SPT>() * 4;
            static_assert(smem <= 227 * 1024, "a tile fits shared memory");
            const dim3 grid(p.groups * p.blocks_per_group, p.N, p.chunks);
            chunk_ends_kernel<T, SPT><<<grid, kScanThreads, 0, s>>>(p);
            if (int rc = launch_status()) return rc;
            if (int rc = scan_join_chunks(p, true, s)) return rc;
            auto *fn = gradient_kernel<T, SPT>;
            if (int rc = raise_smem(reinterpret_cast<const void *>(fn), smem)) return rc;
            fn<<<dim3(grid.x, grid.y, p.segments), kScanThreads, smem, s>>>(p);
            if (int rc = launch_status()) return rc;
            join_weights_kernel<<<(unsigned)((weights + 255) / 256), 256, 0, s>>>(p);
            join_bc_kernel<T><<<(unsigned)((bc + 255) / 256), 256, 0, s>>>(p);
            return launch_status();
        });
    });
}
