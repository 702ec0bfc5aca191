// The gradients of the gated linear recurrence.
//
//   rho = sigmoid(r + r_bias),  w = A rho,  a = e^w,  m = sqrt(1 - a^2)
//   iota = sigmoid(i + i_bias),  h_t = a h_(t-1) + m iota x,  y_t = h_t silu(z_t)
//
// With g_t the gradient of h_t,
//
//   g_t = dy_t silu(z_t) + a_(t+1) g_(t+1)        (the final state's beyond the end)
//   dx = g m iota,  di = g m x iota (1 - iota),  dz = dy h silu'(z)
//   dw = g (a h_(t-1) - iota x a^2 / m),  dr = dw w (1 - rho),  dA = sum dw rho
//
// and dr_bias, di_bias the sums of dr and di; a^2 / m is taken as zero where m is.
//
// Bound: nine rows of memory traffic with both gates, against 70 operations.
#include "seq_gated.cuh"

namespace spconv {
namespace seq {
namespace {

namespace cg = cooperative_groups;

// What a thread's, a warp's or a block's positions do to the state that comes
// from the left (h -> 2^w h + b) and to the gradient that comes from the right
// (q -> 2^w q + c).
struct Both {
    float w, b, c;
};

// Rows on threads as in the forward pass.  The two recurrences run against each
// other, but what a stretch does to either depends on its own positions alone: so
// both are joined across the threads at once, and each input is read once where a
// row fits a cluster's threads.  Longer rows take their rounds from the last to
// the first, from states that a forward pass left in front of each.
// 4 x 2048 x 2048 in bf16 take 92 us, 0.48 of the measured bandwidth: instruction issue
// and latency, two blocks of 128 registers to an SM.  A block for each row, its runs
// read when it starts: 107 us; four positions to a thread and two blocks to a row: 262
// (80 registers: 218).
// WIDE: a row has the whole block (or a cluster).
// STREAM (1: rows of one round, 2: of any): a block takes one row after the other, the next one's (or the next round's)
// runs on their way to slots of its threads in shared memory meanwhile: what a
// thread reads it has sent for itself, so that nothing else is waited for.  (A round
// behind the sequence's end has no barrier; such rounds come first in a row, and the
// row before has ended with one.)
template <typename T, int V, bool I, bool Z, bool WIDE, int STREAM>
__global__ void __launch_bounds__(kGatedThreads, 2) gated_backward_kernel(const __grid_constant__ GatedParams p) {
    __shared__ Both warps[2][kGatedWarps], blocks[2][kGatedRanks];
    __shared__ float all_sums[2][kGatedWarps][3];  // (two: an empty row has no other barrier)
    extern __shared__ uint4 slots[];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = WIDE && p.ranks > 1 ? (int)cluster.block_rank() : 0;
    if (WIDE && p.ranks > 1) cluster.sync();  // the others' shared memory is there
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int threads = WIDE ? kGatedThreads : p.tx, tx = threadIdx.x & (threads - 1);
    const int width = min(threads, 32), at = tx & (width - 1);
    const int team = max(threads >> 5, 1), head = warp & ~(team - 1);

    // a row, its scalars and its inputs
    struct Row {
        GatedRow g;
        RowIn<T, V> x, r, i, z, dy;
        int shift;
        bool vec;
        float A, rb, ib, start, q_end;
    };
    const auto row_of = [&](int64_t number) {
        Row w;
        w.g = gated_row(p, number);
        w.x.set(p.x, p.x_sn, p.x_sc, w.g);
        w.r.set(p.r, p.r_sn, p.r_sc, w.g);
        w.dy.set(p.dy, p.dy_sn, p.dy_sc, w.g);
        w.shift = behind<T, V>(w.x.at);
        w.x.vec = true;
        w.r.vec = behind<T, V>(w.r.at) == w.shift;
        w.dy.vec = behind<T, V>(w.dy.at) == w.shift;
        w.vec = w.r.vec && w.dy.vec;
        if (I) {
            w.i.set(p.i, p.i_sn, p.i_sc, w.g);
            w.i.vec = behind<T, V>(w.i.at) == w.shift;
            w.vec = w.vec && w.i.vec;
        }
        if (Z) {
            w.z.set(p.z, p.z_sn, p.z_sc, w.g);
            w.z.vec = behind<T, V>(w.z.at) == w.shift;
            w.vec = w.vec && w.z.vec;
        }
        w.A = p.A[w.g.c];
        w.rb = p.r_bias ? p.r_bias[w.g.c] : 0.f;
        w.ib = I && p.i_bias ? p.i_bias[w.g.c] : 0.f;
        w.start = p.state ? p.state[w.g.row] : 0.f;
        w.q_end = p.dfinal ? p.dfinal[w.g.row] : 0.f;  // the gradient from the right of a round
        return w;
    };
    // a thread's slots: [stage][input][half of a run] of all threads
    constexpr int kHalves = sizeof(Run<T, V>) / 16, kSlots = 5 * kHalves * kGatedThreads;
    const auto slot = [&](int stage, int input) {
        return slots + stage * kSlots + input * kHalves * kGatedThreads + threadIdx.x;
    };
    const auto send = [&](const Row &w, int round, int stage) {
        const int t0 = (round * threads + tx) * V - w.shift;
        const bool whole = w.vec && t0 >= 0 && t0 + V <= w.g.end;
        const auto one = [&](const RowIn<T, V> &in, int input) {
            uint4 *to = slot(stage, input);
            if (whole) {
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     (uint32_t)__cvta_generic_to_shared(to + h * kGatedThreads)),
                                 "l"(in.at + t0 + h * (16 / (int)sizeof(T)))
                                 : "memory");
            } else {
                Run<T, V> run;
                in.load(run, t0, w.g.end);
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                    to[h * kGatedThreads] = make_uint4(run.w[4 * h], run.w[4 * h + 1], run.w[4 * h + 2], run.w[4 * h + 3]);
            }
        };
        one(w.x, 0);
        one(w.r, 1);
        one(w.dy, 2);
        if (I) one(w.i, 3);
        if (Z) one(w.z, 4);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const auto held = [&](Run<T, V> &run, int stage, int input) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            const uint4 u = slot(stage, input)[h * kGatedThreads];
            run.w[4 * h] = u.x, run.w[4 * h + 1] = u.y, run.w[4 * h + 2] = u.z, run.w[4 * h + 3] = u.w;
        }
    };

    const int rounds = STREAM == 1 ? 1 : p.rounds;
    int64_t number = WIDE ? (int64_t)(blockIdx.x / p.ranks)
                          : (int64_t)blockIdx.x * (kGatedThreads >> p.log_tx) + (threadIdx.x >> p.log_tx);
    Row now = row_of(number);
    if (STREAM) send(now, rounds - 1, 0);
    for (int turn = 0, stage = 0;; turn ^= 1) {
        Row next;
        bool more = false;
        const GatedRow &g = now.g;
        auto &sums = all_sums[turn];
        const int shift = now.shift;
        const int64_t to = g.row * p.L;
        const auto give = [&](void *base, const float (&v)[V], int t0) {
            T *row = static_cast<T *>(base) + to;
            Run<T, V> run;
            run.put(v);
            const bool vec_out = behind<T, V>(row) == shift;
            if (vec_out && t0 >= 0 && t0 + V <= g.L)
                *reinterpret_cast<Run<T, V> *>(row + t0) = run;
            else
                store_part(run, row, t0, g.L, vec_out);
        };
        const float A = now.A, A2 = A * kLog2e, rb = now.rb, ib = now.ib, start = now.start;
        float q_end = now.q_end;
        const f32x2 unit = pack2(-kLog2e, -kLog2e), rb2 = pack2(-kLog2e * rb, -kLog2e * rb),
                    ib2 = pack2(-kLog2e * ib, -kLog2e * ib);
        float dA = 0.f, drb = 0.f, dib = 0.f;

        for (int k = rounds - 1; k >= 0; --k, stage ^= 1) {
            if (STREAM) {  // the next round, or the next row's last one
                if (k > 0) {
                    send(now, k - 1, stage ^ 1);
                } else if (number + (int)gridDim.x < p.rows) {
                    more = true;
                    number += gridDim.x;
                    next = row_of(number);
                    send(next, rounds - 1, stage ^ 1);
                }
                if (k > 0 || more)
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                else
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            const int first = k * p.ranks * threads * V - shift;
            const int t0 = first + (rank * threads + tx) * V;
            if (WIDE && first >= g.end) {  // (the same for the whole cluster)
                const float none[V] = {};
                give(p.dx, none, t0);
                give(p.dr, none, t0);
                if (I) give(p.di, none, t0);
                if (Z) give(p.dz, none, t0);
                continue;
            }
            Run<T, V> rx, rr, ri, rz, rd;
            const bool whole = t0 >= 0 && t0 + V <= g.end;
            const auto read = [&]() {
                held(rx, stage, 0);
                held(rr, stage, 1);
                held(rd, stage, 2);
                if (I) held(ri, stage, 3);
                if (Z) held(rz, stage, 4);
            };
            if (STREAM) {
                read();
            } else if (now.vec && whole) {
                now.x.load(rx, t0);
                now.r.load(rr, t0);
                now.dy.load(rd, t0);
                if (I) now.i.load(ri, t0);
                if (Z) now.z.load(rz, t0);
            } else {
                now.x.load(rx, t0, g.end);
                now.r.load(rr, t0, g.end);
                now.dy.load(rd, t0, g.end);
                if (I) now.i.load(ri, t0, g.end);
                if (Z) now.z.load(rz, t0, g.end);
            }
            const float h_round = rounds > 1 ? p.carry[g.row * rounds + k] : start;

            // each position's gates, decay, sqrt(1 - a^2) and its inverse (for 0 replaced
            // below), and the gradient that its own output gives its state
            float rho[V], iota[V], zeta[V], a[V], m[V], inverse[V], dh[V];
            Both mine{0.f, 0.f, 0.f};
            bool done = false;
            if (whole) {
                f32x2 w_sum = pack2(0.f, 0.f);
                float w_min = A2;
                if (A2 <= Decay::kNear) w_min = 0.f;
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    const f32x2 s = sigmoid2(pair_of(rr, j), unit, rb2), w = mul2(s, pack2(A2, A2));
                    const Decay2 k(w);
                    w_sum = add2(w_sum, w);
                    if (A2 <= Decay::kNear) w_min = fminf(w_min, fminf(unpack2(w).x, unpack2(w).y));
                    float2 f = unpack2(s);
                    rho[j] = f.x, rho[j + 1] = f.y;
                    f = unpack2(k.a);
                    a[j] = f.x, a[j + 1] = f.y;
                    f = unpack2(k.inverse);
                    inverse[j] = f.x, inverse[j + 1] = f.y;
                    f = unpack2(mul2(k.square, k.inverse));
                    m[j] = f.x, m[j + 1] = f.y;
                    if (I) {
                        f = unpack2(sigmoid2(pair_of(ri, j), unit, ib2));
                        iota[j] = f.x, iota[j + 1] = f.y;
                    }
                    f = unpack2(pair_of(rd, j));
                    if (Z) {
                        const f32x2 z2 = pair_of(rz, j), sz = sigmoid2(z2, unit, pack2(0.f, 0.f));
                        f = unpack2(sz);
                        zeta[j] = f.x, zeta[j + 1] = f.y;
                        f = unpack2(mul2(pair_of(rd, j), mul2(z2, sz)));
                    }
                    dh[j] = f.x, dh[j + 1] = f.y;
                }
                mine.w = unpack2(w_sum).x + unpack2(w_sum).y;
                done = w_min > Decay::kNear;
            }
            // the ends of a sequence, decays far from one (formed again, one by one: with
            // A from -8 on instead of -0.1 4 x 2048 x 2048 in bf16 take 102 us instead of 92)
            if (!done) {
                mine.w = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const bool in = t0 + j >= 0 && t0 + j < g.end;
                    rho[j] = in ? sigmoid(rr[j] + rb) : 0.f;
                    const float w = in ? A2 * rho[j] : 0.f;
                    const Decay k(w);
                    mine.w += w;
                    a[j] = k.a();
                    m[j] = in ? k.rest() : 0.f;
                    inverse[j] = rcp(m[j]);
                    if (I) iota[j] = sigmoid(ri[j] + ib);
                    if (Z) zeta[j] = sigmoid(rz[j]);
                    dh[j] = in ? (Z ? rd[j] * (rz[j] * zeta[j]) : rd[j]) : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (!(m[j] > 0.f)) inverse[j] = m[j];  // (a slope of zero; NaN stays)
                mine.b = fmaf(a[j], mine.b, m[j] * (I ? iota[j] * rx[j] : rx[j]));
            }
#pragma unroll
            for (int j = V - 1; j >= 0; --j) mine.c = a[j] * (dh[j] + mine.c);
            float wl = mine.w, wr = mine.w;
            for (int d = 1; d < width; d *= 2) {
                const float w = __shfl_up_sync(~0u, wl, d, width), b = __shfl_up_sync(~0u, mine.b, d, width);
                const float u = __shfl_down_sync(~0u, wr, d, width), c = __shfl_down_sync(~0u, mine.c, d, width);
                if (at >= d) {
                    mine.b = fmaf(grown(wl), b, mine.b);
                    wl += w;
                }
                if (at + d < width) {
                    mine.c = fmaf(grown(wr), c, mine.c);
                    wr += u;
                }
            }
            // what lies to the left and to the right within the warp
            Link before{__shfl_up_sync(~0u, wl, 1, width), __shfl_up_sync(~0u, mine.b, 1, width)};
            Link behind_{__shfl_down_sync(~0u, wr, 1, width), __shfl_down_sync(~0u, mine.c, 1, width)};
            if (at == 0) before = {0.f, 0.f};
            if (at == width - 1) behind_ = {0.f, 0.f};
            const Both all{__shfl_sync(~0u, wl, width - 1, width), __shfl_sync(~0u, mine.b, width - 1, width),
                           __shfl_sync(~0u, mine.c, 0, width)};
            float h_in = h_round, q_in = q_end;
            if (threads > 32) {
                Both *links = warps[STREAM ? stage : k & 1];
                if (lane == 0) links[warp] = all;
                __syncthreads();
                // the row's warps in this block, joined from both ends by eight lanes
                const Both l = lane < team ? links[head + lane] : Both{0.f, 0.f, 0.f};
                float bl = l.b, wl2 = l.w, cr = l.c, wr2 = l.w;
#pragma unroll
                for (int d = 1; d < kGatedWarps; d *= 2) {
                    const float w = __shfl_up_sync(~0u, wl2, d), b = __shfl_up_sync(~0u, bl, d);
                    const float u = __shfl_down_sync(~0u, wr2, d), c = __shfl_down_sync(~0u, cr, d);
                    if (lane >= d) {
                        bl = fmaf(grown(wl2), b, bl);
                        wl2 += w;
                    }
                    if (lane + d < kGatedWarps) {  // (lanes behind the team hold links that change nothing)
                        cr = fmaf(grown(wr2), c, cr);
                        wr2 += u;
                    }
                }
                const Both block{__shfl_sync(~0u, wl2, team - 1), __shfl_sync(~0u, bl, team - 1), __shfl_sync(~0u, cr, 0)};
                const int to_left = max(warp - head - 1, 0), to_right = warp - head + 1;
                Link over{__shfl_sync(~0u, wl2, to_left), __shfl_sync(~0u, bl, to_left)};
                Link under{__shfl_sync(~0u, wr2, to_right), __shfl_sync(~0u, cr, to_right)};
                if (warp == head) over = {0.f, 0.f};
                if (warp == head + team - 1) under = {0.f, 0.f};
                if (WIDE && p.ranks > 1) {
                    Both *parts = blocks[k & 1];
                    if (threadIdx.x < p.ranks) *cluster.map_shared_rank(parts + rank, threadIdx.x) = block;
                    cluster.sync();
                    for (int o = 0; o < rank; ++o) h_in = fmaf(grown(parts[o].w), h_in, parts[o].b);
                    for (int o = p.ranks - 1; o >= 0; --o) {
                        if (o == rank) q_in = q_end;
                        q_end = fmaf(grown(parts[o].w), q_end, parts[o].c);
                    }
                } else {
                    q_end = fmaf(grown(block.w), q_end, block.c);
                }
                h_in = after(h_in, over);
                q_in = after(q_in, under);
            } else {
                q_end = fmaf(grown(all.w), q_end, all.c);
            }
            h_in = after(h_in, before);
            q_in = after(q_in, behind_);

            if (STREAM) read();  // (rather than held in registers until here)
            // from the right: what each state's gradient is
#pragma unroll
            for (int j = V - 1; j >= 0; --j) {
                dh[j] += q_in;
                q_in = a[j] * dh[j];
            }
            float dx[V], dr[V], di[V], dz[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float v = I ? iota[j] * rx[j] : rx[j], gm = dh[j] * m[j];
                const float kept = a[j] * h_in;
                h_in = fmaf(m[j], v, kept);
                const float dw = dh[j] * fmaf(-v * inverse[j], a[j] * a[j], kept);
                dx[j] = I ? gm * iota[j] : gm;
                if (I) di[j] = gm * v * (1.f - iota[j]);
                dr[j] = dw * rho[j];
                if (Z) dz[j] = rd[j] * h_in * (zeta[j] * fmaf(rz[j], 1.f - zeta[j], 1.f));
            }
            if (!whole)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (t0 + j < 0 || t0 + j >= g.end) dx[j] = dr[j] = di[j] = dz[j] = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                dA += dr[j];
                dr[j] *= A * (1.f - rho[j]);
                drb += dr[j];
                if (I) dib += di[j];
            }
            give(p.dx, dx, t0);
            give(p.dr, dr, t0);
            if (I) give(p.di, di, t0);
            if (Z) give(p.dz, dz, t0);
        }
        if (p.dstate && g.on && tx == 0 && rank == 0) p.dstate[g.row] = q_end;

        // the row's sums: over a warp's lanes, then over its warps in their order
        for (int d = width >> 1; d; d >>= 1) {
            dA += __shfl_down_sync(~0u, dA, d, width);
            drb += __shfl_down_sync(~0u, drb, d, width);
            dib += __shfl_down_sync(~0u, dib, d, width);
        }
        if (threads > 32) {
            if (lane == 0) {
                sums[warp][0] = dA;
                sums[warp][1] = drb;
                sums[warp][2] = dib;
            }
            __syncthreads();
            for (int o = 1; o < team && tx == 0; ++o) {
                dA += sums[warp + o][0];
                drb += sums[warp + o][1];
                dib += sums[warp + o][2];
            }
        }
        if (g.on && tx == 0) {
            float *part = p.partial + (g.row * p.ranks + rank) * 3;
            part[0] = dA;
            part[1] = drb;
            part[2] = dib;
        }
        if (!more) break;
        now = next;
    }
}

// A warp per channel adds its rows' parts, each lane those of every 32nd.
__global__ void __launch_bounds__(kGatedThreads) gated_join_kernel(const GatedParams p) {
    const int64_t c = (int64_t)blockIdx.x * kGatedWarps + (threadIdx.x >> 5);
    if (c >= p.C) return;
    const int lane = threadIdx.x & 31;
    float s[3] = {0.f, 0.f, 0.f};
    const int64_t parts = (int64_t)p.N * p.ranks;
    for (int64_t o = lane; o < parts; o += 32) {
        const float *part = p.partial + (((o / p.ranks) * p.C + c) * p.ranks + o % p.ranks) * 3;
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k] += part[k];
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
        for (int d = 16; d; d >>= 1) s[k] += __shfl_down_sync(~0u, s[k], d);
    if (lane == 0) {
        p.dA[c] = s[0];
        if (p.dr_bias) p.dr_bias[c] = s[1];
        if (p.di_bias) p.di_bias[c] = s[2];
    }
}

GatedParams backward_plan(const spconv_gated_scan_args *a, bool aligned) {
    GatedParams p = gated_params(a);
    gated_plan(p, kGatedRun, aligned, true);
    return p;
}
// The workspace's size must not depend on pointers: it is for the larger of the
// plans with and without aligned rows.
bool strides_aligned(const spconv_gated_scan_args *a) {
    return rows_aligned(nullptr, a->x_stride_n, a->x_stride_c, dtype_size(a->dtype));
}
int64_t partial_floats(const GatedParams &p) { return (p.rows * p.ranks * 3 + 3) / 4 * 4; }
int64_t workspace_floats(const GatedParams &p) {
    return partial_floats(p) + (p.rounds > 1 ? (p.rows * p.rounds + 3) / 4 * 4 : 0);
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
}  // namespace seq
}  // namespace spconv

using namespace spconv::seq;

SPCONV_API int64_t spconv_gated_scan_backward_workspace(const spconv_gated_scan_args *a) {
    if (gated_check(a) || a->channels == 0) return 0;
    const int64_t off = workspace_floats(backward_plan(a, false)) * 4;
    if (!strides_aligned(a)) return off;
    const int64_t on = workspace_floats(backward_plan(a, true)) * 4;
    return on > off ? on : off;
}

SPCONV_API int spconv_gated_scan_backward(const spconv_gated_scan_args *a, void *stream) {
    if (int st = gated_check(a)) return st;
    if (a->channels == 0) return SPCONV_OK;
    GatedParams p = backward_plan(a, gated_rows_aligned(a));
    const int64_t e = dtype_size(a->dtype), N = a->N, C = a->channels, L = a->L;
    const bool any = p.rows * L > 0;
    if (!a->A || !a->dA || (any && (!a->x || !a->r || !a->dy || !a->dx || !a->dr))) return SPCONV_ERR_INVALID_ARG;
    if (any && (!a->i != !a->di || !a->z != !a->dz)) return SPCONV_ERR_INVALID_ARG;
    if (!on_elements(a, {a->x, a->r, a->i, a->z, a->dy, a->dx, a->dr, a->di, a->dz}) ||
        !on_words({a->A, a->r_bias, a->i_bias, a->state, a->lengths, a->dfinal_state, a->dA, a->dr_bias,
                   a->di_bias, a->dstate}))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t need = spconv_gated_scan_backward_workspace(a);
    if (need && (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < need))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t out = p.rows * L * e;
    if (!apart({{a->dx, out}, {a->dr, out}, {a->di, out}, {a->dz, out}, {a->dA, C * 4}, {a->dr_bias, C * 4},
                {a->di_bias, C * 4}, {a->dstate, p.rows * 4}, {a->workspace, need}},
               {{a->x, extent(N, C, L, p.x_sn, p.x_sc, e)}, {a->r, extent(N, C, L, p.r_sn, p.r_sc, e)},
                {a->i, extent(N, C, L, p.i_sn, p.i_sc, e)}, {a->z, extent(N, C, L, p.z_sn, p.z_sc, e)},
                {a->dy, extent(N, C, L, p.dy_sn, p.dy_sc, e)}, {a->A, C * 4}, {a->r_bias, C * 4},
                {a->i_bias, C * 4}, {a->state, p.rows * 4}, {a->dfinal_state, p.rows * 4},
                {a->lengths, N * 4}}))
        return SPCONV_ERR_INVALID_ARG;
    p.partial = static_cast<float *>(a->workspace);
    p.carry = p.partial + partial_floats(p);
    if (p.rows && !gated_blocks(p)) return SPCONV_ERR_UNSUPPORTED;
    if (p.rows && p.rounds > 1)
        if (int st = gated_carries(p, a->dtype, stream)) return st;
    if (p.rows) {
        const int st = by_dtype(a->dtype, [&](auto t) {
            using T = decltype(t);
            constexpr int V = kGatedRun;
            const auto launch = [&](auto i, auto z) {
                if (p.tx == kGatedThreads && p.ranks == 1 && (p.rounds > 1 || p.rows >= kGatedStream)) {
                    // two blocks to an SM at most, each with every 304th row
                    void (*fn)(GatedParams) = p.rounds == 1 ? gated_backward_kernel<T, V, i.value, z.value, true, 1>
                                                            : gated_backward_kernel<T, V, i.value, z.value, true, 2>;
                    const int bytes = 2 * 5 * kGatedThreads * (int)sizeof(Run<T, V>);
                    if (int rc = raise_smem(reinterpret_cast<const void *>(fn), bytes)) return rc;
                    const unsigned blocks = p.rows < 2 * kSMs ? (unsigned)p.rows : 2 * kSMs;
                    fn<<<blocks, kGatedThreads, bytes, static_cast<cudaStream_t>(stream)>>>(p);
                    return launch_status();
                }
                return gated_launch(p.tx == kGatedThreads ? gated_backward_kernel<T, V, i.value, z.value, true, 0>
                                                          : gated_backward_kernel<T, V, i.value, z.value, false, 0>,
                                    p, stream);
            };
            if (p.i) return p.z ? launch(std::true_type{}, std::true_type{}) : launch(std::true_type{}, std::false_type{});
            return p.z ? launch(std::false_type{}, std::true_type{}) : launch(std::false_type{}, std::false_type{});
        });
        if (st) return st;
    }
    gated_join_kernel<<<(unsigned)((C + kGatedWarps - 1) / kGatedWarps), kGatedThreads, 0,
                        static_cast<cudaStream_t>(stream)>>>(p);
    return launch_status();
}
