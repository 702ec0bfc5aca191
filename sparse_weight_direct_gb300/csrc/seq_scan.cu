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

// Shared memory of a block, in floats: B and C of two tiles, each channel's
// {dt, dt, dt u, dt u} and each lane's part of its positions' outputs.
constexpr int kTile = 4 * kVec;
constexpr int kStepPitch = kTile + 5;  // rows of 16 bytes: odd, so that eight channels' reads
                                       // of one position meet no bank twice
constexpr int kPartPitch = kTile + 4;
template <int SPT, bool ENDS>
constexpr int scan_smem() {
    return (ENDS ? 2 : 4) * kTile * 4 * SPT + kScanChannels * 4 * kStepPitch +
           (ENDS ? 0 : kScanThreads * kPartPitch);
}

// One pass over a chunk of positions with the states in registers.
// ENDS: from zero states, only what the chunk leaves and the sum of its step
// sizes.  Otherwise the outputs: the y of a position is the sum of the four
// lanes' parts, joined through shared memory once per tile.
template <typename T, int SPT, bool ENDS>
__global__ void __launch_bounds__(kScanThreads) scan_kernel(const ScanParams p) {
    constexpr int VE = kVec, TT = kTile, SP = 4 * SPT, NP = Pairs<SPT>::N;
    extern __shared__ __align__(16) float sm[];
    constexpr int kBuf = (ENDS ? 1 : 2) * TT * SP;
    float *bc = sm;                                   // [2 buffers][B, C][TT][SP]
    const int lane = threadIdx.x & 31, j = lane & 3;
    ulonglong2 *steps = reinterpret_cast<ulonglong2 *>(sm + 2 * kBuf) +
                        (threadIdx.x >> 2) * kStepPitch;
    float *parts = sm + 2 * kBuf + kScanChannels * 4 * kStepPitch;

    const int cb = blockIdx.x, chunk = blockIdx.z;
    const ScanPlace at(p, blockIdx.y, cb);
    const int first = chunk * p.chunk_len, stop = first + min(p.L - first, p.chunk_len);
    const int end = max(min(at.len, stop), first), row_end = at.valid ? end : 0;
    const int64_t row = (int64_t)at.n * p.channels + at.c;
    const T *ur = static_cast<const T *>(p.u) + at.n * p.u_sn + at.c * p.u_sc;
    const T *dr = static_cast<const T *>(p.delta) + at.n * p.d_sn + at.c * p.d_sc;
    const T *zr = !ENDS && p.z ? static_cast<const T *>(p.z) + at.n * p.z_sn + at.c * p.z_sc
                               : nullptr;
    T *yr = static_cast<T *>(p.y) + row * p.L;
    const float bias = p.delta_bias ? p.delta_bias[at.c] : 0.f, D = p.D ? p.D[at.c] : 0.f;
    const int s0 = j * SPT;

    Pairs<SPT> A, h;
    A.load(p.A + (int64_t)at.c * p.S, s0, p.S);
    A.scale(kLog2e);
    const int64_t chunk_row = ((int64_t)at.n * p.chunks + chunk) * p.channels + at.c;
    if (ENDS)
        h.fill(0.f);
    else if (p.chunks > 1)
        h.load(p.h_chunk + chunk_row * p.S, s0, p.S);
    else if (p.state)
        h.load(p.state + row * p.S, s0, p.S);
    else
        h.fill(0.f);

    Run<T> u, d, z, un, dn, zn;
    ScanBC<T, SPT, VE, ENDS> next;
    auto fetch = [&](int t0) {
        load_run(un, ur, t0 + j * VE, row_end, p.vec);
        load_run(dn, dr, t0 + j * VE, row_end, p.vec);
        if (!ENDS && zr) load_run(zn, zr, t0 + j * VE, row_end, p.vec);
        next.load(p, at, t0, end);
    };
    float total = 0.f;
    if (first < end) fetch(first);
    int buf = 0;
    for (int t0 = first; t0 < end; t0 += TT, buf ^= 1) {
        float *tile = bc + buf * kBuf;
        next.store(tile);
        u = un; d = dn; z = zn;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const float dt = t0 + j * VE + e < row_end ? step_size(p, to_f32(d.e[e]) + bias) : 0.f;
            const float du = dt * to_f32(u.e[e]);
            if (ENDS) total += dt;
            steps[j * (VE + 1) + e] = make_ulonglong2(pack2(dt, dt), pack2(du, du));
        }
        // one barrier per tile: the other buffer of B and C was last read before
        // the previous one
        __syncthreads();
        if (t0 + TT < end) fetch(t0 + TT);
#pragma unroll 2
        for (int t = 0; t < TT; t += 4) {
            float yp[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const ulonglong2 x = steps[t + t / VE + k];
                Pairs<SPT> b;
                b.read(tile + (t + k) * SP + s0);
                f32x2 y = 0;
                if (ENDS) {
#pragma unroll
                    for (int i = 0; i < NP; ++i)
                        h.v[i] = fma2(ex2_2(mul2(x.x, A.v[i])), h.v[i], mul2(x.y, b.v[i]));
                } else {
                    Pairs<SPT> c;
                    c.read(tile + (TT + t + k) * SP + s0);
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        h.v[i] = fma2(ex2_2(mul2(x.x, A.v[i])), h.v[i], mul2(x.y, b.v[i]));
                        y = i ? fma2(h.v[i], c.v[i], y) : mul2(h.v[i], c.v[i]);
                    }
                }
                const float2 f = unpack2(y);
                yp[k] = f.x + f.y;
            }
            if (!ENDS)
                *reinterpret_cast<float4 *>(parts + threadIdx.x * kPartPitch + t) =
                    make_float4(yp[0], yp[1], yp[2], yp[3]);
        }
        __syncwarp();
        if (!ENDS) {
            float y[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) y[e] = D * to_f32(u.e[e]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 *q = reinterpret_cast<const float4 *>(
                    parts + ((threadIdx.x & ~3) + k) * kPartPitch + j * VE);
#pragma unroll
                for (int e = 0; e < VE; e += 4) {
                    const float4 f = q[e / 4];
                    y[e] += f.x; y[e + 1] += f.y; y[e + 2] += f.z; y[e + 3] += f.w;
                }
            }
            Run<T> out;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if (zr) y[e] *= silu(to_f32(z.e[e]));
                out.e[e] = from_f32<T>(t0 + j * VE + e < end ? y[e] : 0.f);
            }
            if (at.valid) store_run(out, yr, t0 + j * VE, stop, p.vec_y);
            __syncwarp();
        }
    }
    if (ENDS) {
        total += __shfl_xor_sync(~0u, total, 1);
        total += __shfl_xor_sync(~0u, total, 2);
        if (!at.valid) return;
        h.store(p.h_chunk + chunk_row * p.S, s0, p.S);
        if (j == 0) p.dt_chunk[chunk_row] = total;
        return;
    }
    // positions of the chunk behind the last tile
    if (at.valid) {
        const int done = first + (end - first + TT - 1) / TT * TT;
        Run<T> zero;
#pragma unroll
        for (int e = 0; e < VE; ++e) zero.e[e] = from_f32<T>(0.f);
        for (int t = done + j * VE; t < stop; t += TT) store_run(zero, yr, t, stop, p.vec_y);
        if (p.final_state && chunk == p.chunks - 1) h.store(p.final_state + row * p.S, s0, p.S);
    }
}

// Joins the chunks in their order: on entry h_chunk holds the state that each
// chunk leaves from a zero state (and g_chunk the gradient that reaches its
// start from its own outputs), on return the state that it starts from (the
// gradient of the state that it leaves).  A chunk's decay is e^(A sum dt).
// Eight chunks are read at a time, so that the reads do not wait for the
// writes before them.
__global__ void __launch_bounds__(256) join_chunks_kernel(const ScanParams p, int grad) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t per = (int64_t)p.channels * p.S;
    if (i >= p.N * per) return;
    const int n = (int)(i / per);
    const int64_t cs = i - n * per;
    const float A = p.A[cs] * kLog2e;
    const int64_t base = (int64_t)n * p.chunks;
    const float *dts = p.dt_chunk + base * p.channels + cs / p.S;
    constexpr int kBatch = 8;
    for (int back = 0; back <= grad; ++back) {
        float *rows = (back ? p.g_chunk : p.h_chunk) + base * per + cs;
        const float *first = back ? p.dfinal : p.state;
        float v = first ? first[i] : 0.f;
        for (int k0 = 0; k0 < p.chunks; k0 += kBatch) {
            float left[kBatch], decay[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const int k = back ? p.chunks - 1 - k0 - e : k0 + e;
                if (k0 + e < p.chunks) {
                    left[e] = rows[k * per];
                    decay[e] = dts[(int64_t)k * p.channels];
                }
            }
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const int k = back ? p.chunks - 1 - k0 - e : k0 + e;
                if (k0 + e < p.chunks) {
                    rows[k * per] = v;
                    v = fmaf(ex2(A * decay[e]), v, left[e]);
                }
            }
        }
        if (back && p.dstate) p.dstate[i] = v;
    }
}

// Step: four lanes per request and channel, as in the scan; the states are
// read and written once.
template <typename T, int SPT>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanParams p) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 2;
    const int j = threadIdx.x & 3, s0 = j * SPT;
    const bool on = i < (int64_t)p.N * p.channels;
    const int n = on ? (int)(i / p.channels) : 0, c = on ? (int)(i - (int64_t)n * p.channels) : 0;
    const int slot = !on ? -1 : p.slots ? p.slots[n] : n;
    const bool live = slot >= 0 && slot < p.num_slots;
    float o = 0.f;
    if (live) {
        const int g = c / p.per_group;
        const float u = to_f32(static_cast<const T *>(p.u)[n * p.u_sn + c]);
        const float raw = to_f32(static_cast<const T *>(p.delta)[n * p.d_sn + c]) +
                          (p.delta_bias ? p.delta_bias[c] : 0.f);
        const float dt = step_size(p, raw);
        const T *B = static_cast<const T *>(p.B) + n * p.b_sn + g * p.b_sg;
        const T *C = static_cast<const T *>(p.C) + n * p.c_sn + g * p.c_sg;
        float *row = p.pool + ((int64_t)slot * p.channels + c) * p.S;
        float A[SPT], h[SPT];
        load_states<SPT>(h, row, s0, p.S);
        load_states<SPT>(A, p.A + (int64_t)c * p.S, s0, p.S);
#pragma unroll
        for (int k = 0; k < SPT; ++k) {
            const bool in = s0 + k < p.S;
            const float b = in ? to_f32(B[s0 + k]) : 0.f, cc = in ? to_f32(C[s0 + k]) : 0.f;
            h[k] = fmaf(ex2(dt * (A[k] * kLog2e)), h[k], dt * u * b);
            o = fmaf(h[k], cc, o);
        }
        store_states<SPT>(row, h, s0, p.S);
        if (j == 0 && p.D) o = fmaf(p.D[c], u, o);
    }
    o += __shfl_xor_sync(~0u, o, 1);
    o += __shfl_xor_sync(~0u, o, 2);
    if (on && j == 0) {
        if (p.z && live) o *= silu(to_f32(static_cast<const T *>(p.z)[n * p.z_sn + c]));
        static_cast<T *>(p.y)[i] = from_f32<T>(o);
    }
}

template <typename F>
int raise_smem(F *fn, size_t bytes) {
    if (bytes <= 48 * 1024) return SPCONV_OK;
    return cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)bytes) == cudaSuccess
               ? SPCONV_OK
               : SPCONV_ERR_CUDA;
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
    p.blocks_per_group = (p.per_group + kScanChannels - 1) / kScanChannels;
    p.softplus = a->softplus; p.num_slots = a->num_slots;
    p.chunks = p.segments = p.chunks_per_segment = 1;
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
    join_chunks_kernel<<<(unsigned)((count + 255) / 256), 256, 0, stream>>>(p, grad);
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

// Chunks of the forward scan.  One pass over a sequence needs a block per 32
// channels of each sequence; where that leaves fewer than two blocks per SM,
// the sequence is cut so that there are four, into chunks of four tiles at least.
// Two more passes over the states are the price: what every chunk leaves from
// zero (no outputs), and the join.
void plan_chunks(ScanParams &p) {
    const int64_t blocks = (int64_t)p.groups * p.blocks_per_group * p.N;
    const int64_t tiles = ((int64_t)p.L + kTile - 1) / kTile;
    p.chunks = 1;
    p.chunk_len = p.L;
    if (blocks >= 2 * kSMs || tiles < 8) return;
    int64_t want = (4 * kSMs + blocks - 1) / blocks;
    if (want > tiles / 4) want = tiles / 4;
    const int64_t per = (tiles + want - 1) / want;
    p.chunk_len = (int)(per * kTile);
    p.chunks = (int)((tiles + per - 1) / per);
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
        return by_states(a->S, [&](auto k) {
            using T = decltype(t);
            constexpr int SPT = decltype(k)::value;
            constexpr size_t ends = scan_smem<SPT, true>() * 4, full = scan_smem<SPT, false>() * 4;
            const dim3 grid(p.groups * p.blocks_per_group, p.N, p.chunks);
            if (p.chunks > 1) {
                if (int rc = raise_smem(scan_kernel<T, SPT, true>, ends)) return rc;
                scan_kernel<T, SPT, true><<<grid, kScanThreads, ends, s>>>(p);
                if (int rc = launch_status()) return rc;
                if (int rc = scan_join_chunks(p, false, s)) return rc;
            }
            if (int rc = raise_smem(scan_kernel<T, SPT, false>, full)) return rc;
            scan_kernel<T, SPT, false><<<grid, kScanThreads, full, s>>>(p);
            return launch_status();
        });
    });
}

SPCONV_API int spconv_scan_step(const spconv_scan_args *a, void *stream) {
    const int st = scan_check_sizes(a);
    if (st) return st;
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
    const ScanParams p = scan_params(a);
    const int64_t blocks = (rows * 4 + 255) / 256;
    if (blocks > 0x7fffffff) return SPCONV_ERR_UNSUPPORTED;
    return by_dtype(a->dtype, [&](auto t) {
        return by_states(a->S, [&](auto k) {
            scan_step_kernel<decltype(t), decltype(k)::value>
                <<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
            return launch_status();
        });
    });
}
