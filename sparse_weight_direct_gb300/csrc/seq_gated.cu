// The gated linear recurrence: forward and the single-token step.
//
//   rho = sigmoid(r + r_bias),  a = e^(A rho),  v = sigmoid(i + i_bias) x
//   h_t = a h_(t-1) + sqrt(1 - a^2) v,  y_t = h_t silu(z_t)
//
// Bound: 30 operations, seven of them on the special function unit (32 a clock and
// SM on this chip), against 10 bytes per element for 16-bit types: the memory, with
// the instruction issue close behind.
#include "seq_gated.cuh"

namespace spconv {
namespace seq {
namespace {

namespace cg = cooperative_groups;

// A row's positions lie on the threads of part of a warp, of a block or of a
// cluster, V to a thread, so that one pass reads a row of 2048 positions (16,384
// in a cluster).  A thread runs through its own positions from a zero state and
// keeps what they do to a state (a Link); links are joined over a warp's lanes by
// shuffles, over warps and blocks in shared memory.  Each position then adds what
// is left of the state in front of its thread.
// 8 x 4096 x 2048 in bf16 take 133 us, 0.74 of the measured bandwidth, 1 x 1000 x 8191
// in float32 34 us (0.70).  Element by element, with the exponential of every decay:
// 254 us; three blocks of 80 registers to an SM for 16-bit types (two: 151 us, four
// spill: 156), two for float32 (three spill: 58 us for the long rows).
// CARRY: only the states in front of each round.
// WIDE: a row has more than one warp.
template <typename T, int V, bool I, bool Z, bool CARRY, bool WIDE>
__global__ void __launch_bounds__(kGatedThreads, sizeof(T) == 4 ? 2 : 3) gated_kernel(const GatedParams p) {
    __shared__ Link warps[2][kGatedWarps], blocks[2][kGatedRanks];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = WIDE && p.ranks > 1 ? (int)cluster.block_rank() : 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tx = threadIdx.x & (p.tx - 1);
    const int width = WIDE ? 32 : p.tx, at = tx & (width - 1);
    if (WIDE && p.ranks > 1) cluster.sync();  // the others' shared memory is there
    const GatedRow g =
        gated_row(p, (int64_t)(blockIdx.x / p.ranks) * (kGatedThreads >> p.log_tx) + (threadIdx.x >> p.log_tx));

    RowIn<T, V> x, r, i, z;
    x.set(p.x, p.x_sn, p.x_sc, g);
    r.set(p.r, p.r_sn, p.r_sc, g);
    const int shift = behind<T, V>(x.at);
    x.vec = true;
    r.vec = behind<T, V>(r.at) == shift;
    bool vec = r.vec;
    if (I) {
        i.set(p.i, p.i_sn, p.i_sc, g);
        i.vec = behind<T, V>(i.at) == shift;
        vec = vec && i.vec;
    }
    if (Z && !CARRY) {
        z.set(p.z, p.z_sn, p.z_sc, g);
        z.vec = behind<T, V>(z.at) == shift;
        vec = vec && z.vec;
    }
    T *y = static_cast<T *>(p.y) + g.row * p.L;
    const bool vec_y = behind<T, V>(y) == shift;
    const float A = p.A[g.c] * kLog2e;
    const float rb = p.r_bias ? p.r_bias[g.c] : 0.f, ib = I && p.i_bias ? p.i_bias[g.c] : 0.f;
    const f32x2 unit = pack2(-kLog2e, -kLog2e), rb2 = pack2(-kLog2e * rb, -kLog2e * rb),
                ib2 = pack2(-kLog2e * ib, -kLog2e * ib);
    float carry = p.state ? p.state[g.row] : 0.f;

    Run<T, V> rx, rr, ri, rz;
    const auto load = [&](int t0) {
        if (vec && t0 >= 0 && t0 + V <= g.end) {
            x.load(rx, t0);
            r.load(rr, t0);
            if (I) i.load(ri, t0);
            if (Z && !CARRY) z.load(rz, t0);
        } else {
            x.load(rx, t0, g.end);
            r.load(rr, t0, g.end);
            if (I) i.load(ri, t0, g.end);
            if (Z && !CARRY) z.load(rz, t0, g.end);
        }
    };
    const int mine_at = (rank * p.tx + tx) * V - shift, step = p.ranks * p.tx * V;
    load(mine_at);
    for (int k = 0; k < p.rounds; ++k) {
        const int t0 = k * step + mine_at;
        if (CARRY && g.on && tx == 0 && rank == 0) p.carry[g.row * p.rounds + k] = carry;
        // (the same for the whole warp or cluster that has the row)
        if ((WIDE ? p.tx == kGatedThreads : p.tx == 32) && k * step - shift >= g.end) {
            if (CARRY) continue;
            Run<T, V> none;
            none.clear();
            store_part(none, y, t0, g.L, vec_y);
            continue;
        }
        // each position's decay, input and output gate
        float a[V], b[V], gate[V];
        Link mine{0.f, 0.f};
        bool done = false;
        if (t0 >= 0 && t0 + V <= g.end) {
            f32x2 w_sum = pack2(0.f, 0.f);
            float w_min = A;
            if (A <= Decay::kNear) w_min = 0.f;
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                const f32x2 w = mul2(sigmoid2(pair_of(rr, j), unit, rb2), pack2(A, A));
                const Decay2 k(w);
                const f32x2 v = I ? mul2(sigmoid2(pair_of(ri, j), unit, ib2), pair_of(rx, j)) : pair_of(rx, j);
                w_sum = add2(w_sum, w);
                if (A <= Decay::kNear) w_min = fminf(w_min, fminf(unpack2(w).x, unpack2(w).y));
                float2 f = unpack2(k.a);
                a[j] = f.x, a[j + 1] = f.y;
                f = unpack2(mul2(mul2(k.square, k.inverse), v));
                b[j] = f.x, b[j + 1] = f.y;
                if (Z && !CARRY) {
                    const f32x2 z2 = pair_of(rz, j);
                    f = unpack2(mul2(z2, sigmoid2(z2, unit, pack2(0.f, 0.f))));
                    gate[j] = f.x, gate[j + 1] = f.y;
                }
            }
            mine.w = unpack2(w_sum).x + unpack2(w_sum).y;
            done = w_min > Decay::kNear;
        }
        // the ends of a sequence, decays far from one (formed again, one by one: with A
        // from -8 on instead of -0.1 8 x 4096 x 2048 in bf16 take 193 us instead of 133)
        if (!done) {
            mine.w = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const bool in = t0 + j >= 0 && t0 + j < g.end;
                const float w = in ? A * sigmoid(rr[j] + rb) : 0.f;
                const Decay k(w);
                const float v = I ? sigmoid(ri[j] + ib) * rx[j] : rx[j];
                mine.w += w;
                a[j] = k.a();
                b[j] = in ? k.rest() * v : 0.f;
                if (Z && !CARRY) gate[j] = in ? silu(rz[j]) : 0.f;
            }
        }
        // the next round's runs, while this one's links are joined
        if (k + 1 < p.rounds) load(t0 + step);
        // (A decay's own rounding is taken into account by the exponents from thread
        // to thread: within a thread it counts eight times at most.)
#pragma unroll
        for (int j = 0; j < V; ++j) mine.b = fmaf(a[j], mine.b, b[j]);
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            if (!WIDE && d >= width) break;
            const float w = __shfl_up_sync(~0u, mine.w, d, width), b = __shfl_up_sync(~0u, mine.b, d, width);
            if (at >= d) {
                mine.b = after(b, mine);
                mine.w += w;
            }
        }
        Link before{__shfl_up_sync(~0u, mine.w, 1, width), __shfl_up_sync(~0u, mine.b, 1, width)};
        if (at == 0) before = {0.f, 0.f};
        float in = carry;
        if (WIDE) {
            Link *links = warps[k & 1];
            if (lane == 31) links[warp] = mine;
            __syncthreads();
            const int team = p.tx >> 5, head = warp & ~(team - 1);
            // the row's warps in this block, joined by eight lanes
            Link w = lane < team ? links[head + lane] : Link{0.f, 0.f};
#pragma unroll
            for (int d = 1; d < kGatedWarps; d *= 2) {
                const float u = __shfl_up_sync(~0u, w.w, d), b = __shfl_up_sync(~0u, w.b, d);
                if (lane >= d) {
                    w.b = after(b, w);
                    w.w += u;
                }
            }
            const Link block{__shfl_sync(~0u, w.w, team - 1), __shfl_sync(~0u, w.b, team - 1)};
            const int to_left = max(warp - head - 1, 0);
            Link over{__shfl_sync(~0u, w.w, to_left), __shfl_sync(~0u, w.b, to_left)};
            if (warp == head) over = {0.f, 0.f};
            if (p.ranks > 1) {
                Link *all = blocks[k & 1];
                if (threadIdx.x < p.ranks) *cluster.map_shared_rank(all + rank, threadIdx.x) = block;
                cluster.sync();
                for (int q = 0; q < p.ranks; ++q) {
                    if (q == rank) in = carry;
                    carry = after(carry, all[q]);
                }
            } else {
                carry = after(carry, block);
            }
            in = after(in, over);
        } else {
            const Link all{__shfl_sync(~0u, mine.w, width - 1, width), __shfl_sync(~0u, mine.b, width - 1, width)};
            carry = after(carry, all);
        }
        if (CARRY) continue;
        in = after(in, before);
        float out[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            in = fmaf(a[j], in, b[j]);
            out[j] = Z ? in * gate[j] : in;
        }
        if (t0 + V > g.end)
#pragma unroll
            for (int j = 0; j < V; ++j) out[j] = t0 + j < g.end ? out[j] : 0.f;
        Run<T, V> ry;
        ry.put(out);
        if (vec_y && t0 >= 0 && t0 + V <= g.L)
            *reinterpret_cast<Run<T, V> *>(y + t0) = ry;
        else
            store_part(ry, y, t0, g.L, vec_y);
    }
    if (!CARRY && p.final_state && g.on && tx == 0 && rank == 0) p.final_state[g.row] = carry;
}

// One position of each request, V channels to a thread.
template <typename T, int V, bool I, bool Z>
__global__ void __launch_bounds__(kGatedThreads) gated_step_kernel(const GatedParams p) {
    const int64_t at = ((int64_t)blockIdx.x * kGatedThreads + threadIdx.x) * V;
    if (at >= p.C) return;
    const int c = (int)at, n = blockIdx.y;
    const int slot = p.slots ? p.slots[n] : n;
    T *y = static_cast<T *>(p.y) + (int64_t)n * p.C + c;
    float out[V] = {};
    if (slot >= 0 && slot < p.num_slots) {
        float x[V], r[V], i[V], z[V], h[V], A[V], rb[V] = {}, ib[V] = {};
        float *pool = p.pool + (int64_t)slot * p.C + c;
        take(x, static_cast<const T *>(p.x) + n * p.x_sn + c);
        take(r, static_cast<const T *>(p.r) + n * p.r_sn + c);
        if (I) take(i, static_cast<const T *>(p.i) + n * p.i_sn + c);
        if (Z) take(z, static_cast<const T *>(p.z) + n * p.z_sn + c);
        take(h, pool);
        take(A, p.A + c);
        if (p.r_bias) take(rb, p.r_bias + c);
        if (I && p.i_bias) take(ib, p.i_bias + c);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const Decay a(A[j] * kLog2e * sigmoid(r[j] + rb[j]));
            const float v = I ? sigmoid(i[j] + ib[j]) * x[j] : x[j];
            h[j] = a.of(h[j]) + a.rest() * v;
            out[j] = Z ? h[j] * silu(z[j]) : h[j];
        }
        give(h, pool);
    }
    give(out, y);
}

// ---------------------------------------------------------------- host side

// f(i, z): whether there is an input gate, an output gate.
template <typename F>
int by_gates(const GatedParams &p, F f) {
    if (p.i) return p.z ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
    return p.z ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}

bool on_elements(const spconv_gated_scan_args *a, std::initializer_list<const void *> ps) {
    for (const void *q : ps)
        if (q && !aligned(q, dtype_size(a->dtype))) return false;
    return true;
}
bool on_words(std::initializer_list<const void *> ps) {
    for (const void *q : ps)
        if (q && !aligned(q, 4)) return false;
    return true;
}

}  // namespace

int gated_check(const spconv_gated_scan_args *a) {
    if (!a || a->N < 0 || a->channels < 0 || a->L < 0) return SPCONV_ERR_INVALID_ARG;
    if (a->dtype < SPCONV_F32 || a->dtype > SPCONV_F16) return SPCONV_ERR_INVALID_ARG;
    if (a->N > kMaxLength || a->channels > kMaxLength || a->L > kMaxLength) return SPCONV_ERR_UNSUPPORTED;
    for (int64_t s : {a->x_stride_n, a->x_stride_c, a->r_stride_n, a->r_stride_c, a->i_stride_n, a->i_stride_c,
                      a->z_stride_n, a->z_stride_c, a->dy_stride_n, a->dy_stride_c})
        if (!stride_ok(s)) return SPCONV_ERR_INVALID_ARG;
    // (an empty tensor's pointer may be NULL)
    if ((a->i_bias || a->di_bias) && !a->i && a->N > 0 && a->channels > 0 && a->L > 0) return SPCONV_ERR_INVALID_ARG;
    return SPCONV_OK;
}

GatedParams gated_params(const spconv_gated_scan_args *a) {
    GatedParams p{};
    p.x = a->x; p.r = a->r; p.i = a->i; p.z = a->z; p.dy = a->dy;
    p.A = a->A; p.r_bias = a->r_bias; p.i_bias = a->i_bias;
    p.state = a->state; p.dfinal = a->dfinal_state;
    p.lengths = a->lengths; p.slots = a->slots;
    p.y = a->y; p.dx = a->dx; p.dr = a->dr; p.di = a->di; p.dz = a->dz;
    p.final_state = a->final_state; p.pool = a->pool;
    p.dA = a->dA; p.dr_bias = a->dr_bias; p.di_bias = a->di_bias; p.dstate = a->dstate;
    p.x_sn = a->x_stride_n; p.x_sc = a->x_stride_c;
    p.r_sn = a->r_stride_n; p.r_sc = a->r_stride_c;
    p.i_sn = a->i_stride_n; p.i_sc = a->i_stride_c;
    p.z_sn = a->z_stride_n; p.z_sc = a->z_stride_c;
    p.dy_sn = a->dy_stride_n; p.dy_sc = a->dy_stride_c;
    p.N = a->N; p.C = a->channels; p.L = a->L; p.num_slots = a->num_slots;
    p.rows = (int64_t)a->N * a->channels;
    return p;
}

bool gated_rows_aligned(const spconv_gated_scan_args *a) {
    return rows_aligned(a->x, a->x_stride_n, a->x_stride_c, dtype_size(a->dtype));
}

int gated_launch(void (*fn)(GatedParams), const GatedParams &p, void *stream) {
    const unsigned blocks = gated_blocks(p);
    if (!blocks) return SPCONV_ERR_UNSUPPORTED;
    if (p.ranks == 1) {
        fn<<<blocks, kGatedThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
        return launch_status();
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kGatedThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, p) != cudaSuccess) {
        cudaGetLastError();
        return SPCONV_ERR_CUDA;
    }
    return SPCONV_OK;
}

int gated_carries(const GatedParams &p, int dtype, void *stream) {
    return by_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        // (rows of several rounds are wide)
        return gated_launch(p.i ? gated_kernel<T, kGatedRun, true, false, true, true>
                                : gated_kernel<T, kGatedRun, false, false, true, true>,
                            p, stream);
    });
}

}  // namespace seq
}  // namespace spconv

using namespace spconv::seq;

SPCONV_API int spconv_gated_scan(const spconv_gated_scan_args *a, void *stream) {
    if (int st = gated_check(a)) return st;
    GatedParams p = gated_params(a);
    if (p.rows == 0) return SPCONV_OK;
    const int64_t e = dtype_size(a->dtype), N = a->N, C = a->channels, L = a->L;
    if (!a->A || (L > 0 && (!a->x || !a->r || !a->y))) return SPCONV_ERR_INVALID_ARG;
    if (!on_elements(a, {a->x, a->r, a->i, a->z, a->y}) ||
        !on_words({a->A, a->r_bias, a->i_bias, a->state, a->lengths, a->final_state}))
        return SPCONV_ERR_INVALID_ARG;
    if (!apart({{a->y, p.rows * L * e}, {a->final_state, p.rows * 4}},
               {{a->x, extent(N, C, L, p.x_sn, p.x_sc, e)}, {a->r, extent(N, C, L, p.r_sn, p.r_sc, e)},
                {a->i, extent(N, C, L, p.i_sn, p.i_sc, e)}, {a->z, extent(N, C, L, p.z_sn, p.z_sc, e)},
                {a->A, C * 4}, {a->r_bias, C * 4}, {a->i_bias, C * 4}, {a->state, p.rows * 4},
                {a->lengths, N * 4}}))
        return SPCONV_ERR_INVALID_ARG;
    gated_plan(p, kGatedRun, gated_rows_aligned(a), false);
    return by_dtype(a->dtype, [&](auto t) {
        return by_gates(p, [&](auto i, auto z) {
            using T = decltype(t);
            return gated_launch(p.tx > 32 ? gated_kernel<T, kGatedRun, i.value, z.value, false, true>
                                          : gated_kernel<T, kGatedRun, i.value, z.value, false, false>,
                                p, stream);
        });
    });
}

SPCONV_API int spconv_gated_scan_step(const spconv_gated_scan_args *a, void *stream) {
    if (int st = gated_check(a)) return st;
    if (a->num_slots < 0 || (!a->slots && a->N > 0 && a->num_slots != a->N) || a->x_stride_c != 1 || a->r_stride_c != 1 ||
        (a->i && a->i_stride_c != 1) || (a->z && a->z_stride_c != 1))
        return SPCONV_ERR_INVALID_ARG;
    if (a->N > 65535) return SPCONV_ERR_UNSUPPORTED;  // requests go along grid y
    const GatedParams p = gated_params(a);
    if (p.rows == 0) return SPCONV_OK;
    const int64_t e = dtype_size(a->dtype), N = a->N, C = a->channels;
    if (!a->x || !a->r || !a->A || !a->y || (a->num_slots > 0 && !a->pool)) return SPCONV_ERR_INVALID_ARG;
    if (!on_elements(a, {a->x, a->r, a->i, a->z, a->y}) ||
        !on_words({a->A, a->r_bias, a->i_bias, a->slots, a->pool}))
        return SPCONV_ERR_INVALID_ARG;
    if (!apart({{a->y, p.rows * e}, {a->pool, a->num_slots * C * 4}},
               {{a->x, extent(N, C, 1, p.x_sn, 1, e)}, {a->r, extent(N, C, 1, p.r_sn, 1, e)},
                {a->i, extent(N, C, 1, p.i_sn, 1, e)}, {a->z, extent(N, C, 1, p.z_sn, 1, e)}, {a->A, C * 4},
                {a->r_bias, C * 4}, {a->i_bias, C * 4}, {a->slots, N * 4}}))
        return SPCONV_ERR_INVALID_ARG;
    // four channels to a thread where they are whole vectors in every tensor
    bool four = C % 4 == 0;
    for (const void *q : {a->x, a->r, a->i, a->z, (const void *)a->y}) four = four && aligned(q, 4 * e);
    for (int64_t s : {p.x_sn, p.r_sn, p.i_sn, p.z_sn}) four = four && s % 4 == 0;
    for (const float *q : {a->A, a->r_bias, a->i_bias, (const float *)a->pool}) four = four && aligned(q, 16);
    const int V = four ? 4 : 1;
    const dim3 grid((unsigned)((C + kGatedThreads * V - 1) / (kGatedThreads * V)), (unsigned)N);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_dtype(a->dtype, [&](auto t) {
        return by_gates(p, [&](auto i, auto z) {
            using T = decltype(t);
            if (four)
                gated_step_kernel<T, 4, i.value, z.value><<<grid, kGatedThreads, 0, s>>>(p);
            else
                gated_step_kernel<T, 1, i.value, z.value><<<grid, kGatedThreads, 0, s>>>(p);
            return launch_status();
        });
    });
}
