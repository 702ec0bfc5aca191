// The gradients of the norms before and after a block.
//
//   b = y silu(z),  q = 1 / rms(b),  n = b q (without post: b),  w = scale post
//   s = x + w n,  t = 1 / rms(s),  out = pre s t
//
// With v = dout pre and means over the channels,
//
//   G = dsum + t v - s t^3 mean(v s),  dx = G,  dpre = sum dout s t
//   u = G w,  db = q u - b q^3 mean(u b)    (without post: u)
//   dy = db silu(z),  dz = db y silu'(z),  dscale = sum G post n,  dpost = sum G scale n
//
// Bound: eight rows of memory traffic, with x, y, z, both gradients, dx, dy and dz.
#include "seq_norm.cuh"

namespace spconv {
namespace seq {
namespace {

// Tiles as in the forward pass, and as there one pass of sums: with w = scale post,
//
//   sum s^2 = sum x^2 + 2 q sum w x b + q^2 sum w^2 b^2
//   sum v s = sum v x + q sum v w b
//   sum u b = sum w b dsum + t sum v w b - t^3 mean(v s) (sum w x b + q sum w^2 b^2)
//
// so that the three norms and means that wait for one another wait for the cluster
// once.  Where x and w q b cancel in s, the sums over s are formed again from its
// terms.  A cluster takes one tile after the other; the weights' gradients are summed
// by the thread that has the channel and written once for each cluster, and a second
// kernel adds the clusters.
//
// 4 x 2048 x 2048 in bf16 take 104 us, 0.38 of the measured bandwidth: 112 instructions
// an element at 0.50 an SMSP and clock, and one tile's copies before its sums.  A pass
// for each of the three sums, unrolled in registers: 626 us, most of it waiting for
// instructions.
template <typename T, int W, bool VEC>
__global__ void __launch_bounds__(kNormThreads, 2) norm_backward_kernel(const __grid_constant__ NormParams p) {
    using Tile = NormTile<T, W, VEC>;
    constexpr int V = Tile::V, H = V / 2, K = 7;
    extern __shared__ uint4 shared[];
    auto &sm = *reinterpret_cast<NormSums<K, W, V> *>(
        shared + p.stages * p.inputs * p.R * (kNormThreads + (VEC ? 0 : Tile::ROWS)));
    // the thread's channels' sums of dout s t and G n
    float2 *held = reinterpret_cast<float2 *>(&sm + 1) + threadIdx.x;
    float2 *block_weights = reinterpret_cast<float2 *>(&sm + 1) + p.R * kNormThreads;
    float2 *weights = block_weights + threadIdx.x / W;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = p.ranks > 1 ? (int)cluster.block_rank() : 0;
    const unsigned id = blockIdx.x / p.ranks;
    Tile tile(p, shared, rank);
    for (int k = 0; k < p.R; ++k) held[k * kNormThreads] = {0.f, 0.f};
    int stage = 0, parity = 0;
    tile.place(id, 0);
    tile.fetch();
    tile.weights(block_weights);
    if (p.ranks > 1) cluster.sync();  // the others' shared memory is there
    const bool gated = p.in[kZ];
    const unsigned jobs = (unsigned)p.jobs, step = (unsigned)p.clusters;
    for (unsigned job = id; job < jobs; job += step) {
        const bool more = p.stages > 1 && job + step < jobs;
        if (more) {
            tile.place(job + step, stage ^ 1);
            tile.fetch();
        }
        tile.place(job, stage);
        tile.arrived(more);
        const auto work = [&]() {
            f32x2 v[K * H] = {};
            for (int k = 0, o = tile.origin; k < p.R; ++k, o += kNormThreads) {
                const float2 w = weights[k * Tile::ROWS];
                f32x2 x[H], b[H], dout[H], dsum[H];
                tile.pairs(b, kY, o);
                if (gated) {
                    f32x2 z[H];
                    tile.pairs(z, kZ, o);
    #pragma unroll
                    for (int j = 0; j < H; ++j) b[j] = mul2(b[j], mul2(z[j], sigmoid2(z[j])));
                }
                tile.pairs(x, kX, o);
                tile.pairs(dout, kDout, o);
                tile.pairs(dsum, kDsum, o);
    #pragma unroll
                for (int j = 0; j < H; ++j) {
                    const f32x2 wb = mul2(both(w.x), b[j]), u = mul2(both(w.y), dout[j]);
                    v[j] = fma2(b[j], b[j], v[j]);
                    v[H + j] = fma2(x[j], x[j], v[H + j]);
                    v[2 * H + j] = fma2(wb, x[j], v[2 * H + j]);
                    v[3 * H + j] = fma2(wb, wb, v[3 * H + j]);
                    v[4 * H + j] = fma2(u, x[j], v[4 * H + j]);
                    v[5 * H + j] = fma2(u, wb, v[5 * H + j]);
                    v[6 * H + j] = fma2(wb, dsum[j], v[6 * H + j]);
                }
            }
            // the factors from q, t, sum v s, sum w b s, sum w b v and sum w b dsum
            const auto set = [&](int at, float q, float t, float vs, float wbs, float wbv, float wbd) {
                const float back = t * t * t * (vs * p.inv_C);
                const float ub = fmaf(t, wbv, wbd) - back * wbs;
                const bool in = tile.first + at < tile.end;
                sm.factors[at] = in ? make_float4(q, t, -back, p.post ? -q * q * q * (ub * p.inv_C) : 0.f)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
            };
            const bool again = sum_tile<K, V, W>(v, sm, p.ranks, rank, parity, [&](int at, const float (&s)[K], bool store) {
                const float q = p.post ? rsqrtf(fmaf(s[0], p.inv_C, p.eps)) : 1.f;
                const float apart = fmaf(q * q, s[3], s[1]), sum = fmaf(2.f * q, s[2], apart);
                const float t = p.pre ? rsqrtf(fmaf(sum, p.inv_C, p.eps)) : 0.f;
                if (store) {
                    set(at, q, t, fmaf(q, s[5], s[4]), fmaf(q, s[3], s[2]), s[5], s[6]);
                    sm.held[at] = make_float2(s[5], s[6]);
                }
                return p.pre && tile.first + at < tile.end && sum < 0.125f * apart;
            });
            parity ^= 1;
            if (again) {
                f32x2 u[3 * H] = {};
                for (int k = 0, o = tile.origin; k < p.R; ++k, o += kNormThreads) {
                    const float2 w = weights[k * Tile::ROWS];
                    f32x2 x[H], y[H], z[H], dout[H];
                    tile.pairs(x, kX, o);
                    tile.pairs(y, kY, o);
                    tile.pairs(z, kZ, o);
                    tile.pairs(dout, kDout, o);
    #pragma unroll
                    for (int j = 0; j < H; ++j) {
                        const f32x2 b = gated ? mul2(y[j], mul2(z[j], sigmoid2(z[j]))) : y[j], wb = mul2(both(w.x), b);
                        const float4 *f = sm.factors + tile.tx * V + 2 * j;
                        const f32x2 s = fma2(wb, pack2(f[0].x, f[1].x), x[j]);
                        u[j] = fma2(s, s, u[j]);
                        u[H + j] = fma2(mul2(both(w.y), dout[j]), s, u[H + j]);
                        u[2 * H + j] = fma2(wb, s, u[2 * H + j]);
                    }
                }
                sum_tile<3, V, W>(u, sm, p.ranks, rank, parity, [&](int at, const float (&s)[3], bool store) {
                    // (of a position's eight lanes only this one reads or writes its factors)
                    if (store)
                        set(at, sm.factors[at].x, rsqrtf(fmaf(s[0], p.inv_C, p.eps)), s[1], s[2], sm.held[at].x,
                            sm.held[at].y);
                    return false;
                });
                parity ^= 1;
            }
            f32x2 q[H], t[H], back[H], back_b[H];
    #pragma unroll
            for (int j = 0; j < H; ++j) {
                const float4 f0 = sm.factors[tile.tx * V + 2 * j], f1 = sm.factors[tile.tx * V + 2 * j + 1];
                q[j] = pack2(f0.x, f1.x), t[j] = pack2(f0.y, f1.y);
                back[j] = pack2(f0.z, f1.z), back_b[j] = pack2(f0.w, f1.w);
            }
            int c = tile.c0;
            int64_t to = tile.out;
            for (int k = 0, o = tile.origin; k < p.R; ++k, o += kNormThreads, c += Tile::ROWS, to += tile.out_step) {
                const float2 w = weights[k * Tile::ROWS];
                f32x2 x[H], y[H], z[H], dout[H], dsum[H];
                tile.pairs(x, kX, o);
                tile.pairs(y, kY, o);
                tile.pairs(z, kZ, o);
                tile.pairs(dout, kDout, o);
                tile.pairs(dsum, kDsum, o);
                f32x2 s0 = 0, s1 = 0;
    #pragma unroll
                for (int j = 0; j < H; ++j) {
                    f32x2 gate, slope, b = y[j];
                    if (gated) {
                        const f32x2 g = sigmoid2(z[j]);
                        gate = mul2(z[j], g);
                        // g (1 + z (1 - g)) = g + gate (1 - g)
                        slope = fma2(gate, fma2(g, both(-1.f), both(1.f)), g);
                        b = mul2(y[j], gate);
                    }
                    const f32x2 bq = mul2(b, q[j]), s = fma2(both(w.x), bq, x[j]);
                    const f32x2 g = fma2(s, back[j], fma2(mul2(t[j], both(w.y)), dout[j], dsum[j]));
                    const f32x2 db = fma2(b, back_b[j], mul2(mul2(g, both(w.x)), q[j]));
                    s0 = fma2(dout[j], mul2(s, t[j]), s0);
                    s1 = fma2(g, bq, s1);
                    x[j] = g;
                    if (gated) {
                        z[j] = mul2(mul2(db, y[j]), slope);
                        y[j] = mul2(db, gate);
                    } else {
                        y[j] = db;
                    }
                }
                const float2 f0 = unpack2(s0), f1 = unpack2(s1);
                float2 sums = held[k * kNormThreads];
                sums.x += f0.x + f0.y;
                sums.y += f1.x + f1.y;
                held[k * kNormThreads] = sums;
                if (p.in[kX]) tile.give(p.dx, x, c, to);
                if (p.in[kY]) tile.give(p.dy, y, c, to);
                if (gated) tile.give(p.dz, z, c, to);
            }
        };
        if (tile.empty()) {
            tile.clear(p.dx);
            tile.clear(p.dy);
            tile.clear(p.dz);
        } else {
            work();
        }
        if (p.stages > 1) {
            stage ^= 1;
        } else if (job + step < jobs) {
            tile.place(job + step, 0);
            tile.fetch();
        }
    }
    float *to = p.partial + (int64_t)id * 2 * p.C;
    for (int k = 0; k < p.R; ++k) {
        float2 s = held[k * kNormThreads];
#pragma unroll
        for (int d = W >> 1; d; d >>= 1) {
            s.x += __shfl_down_sync(~0u, s.x, d, W);
            s.y += __shfl_down_sync(~0u, s.y, d, W);
        }
        const int c = tile.c0 + k * Tile::ROWS;
        if (tile.tx == 0 && c < tile.c_end) {
            to[c] = s.x;
            to[p.C + c] = s.y;
        }
    }
}

// More channels than a cluster holds: a block for 32 positions, whose rows are
// read again for each sum.  A block takes one tile after the other and adds to its
// own part of the weights' gradients.  4 x 8200 x 512 in bf16 take 6.2 ms (8192
// channels, in clusters, 0.166).
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_backward_wide_kernel(const NormParams p) {
    __shared__ float all[2][kNormWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *to_pre = p.partial + (int64_t)blockIdx.x * 2 * p.C, *to_both = to_pre + p.C;
    for (int64_t job = blockIdx.x; job < p.jobs; job += p.clusters) {
        const int n = (int)(job / p.tiles), t = (int)(job - (int64_t)n * p.tiles) * 32 + lane;
        const int end = p.lengths ? min(max(p.lengths[n], 0), p.L) : p.L;
        const bool in = t < end;
        const auto read = [&](int input, int c) {
            return p.in[input] && in
                       ? to_f32(static_cast<const T *>(p.in[input])[n * p.in_sn[input] + c * p.in_sc[input] + t])
                       : 0.f;
        };
        const auto block = [&](int c) {
            const float y = read(kY, c);
            return p.in[kZ] ? y * silu(read(kZ, c)) : y;
        };
        const auto weight = [&](int c) {
            return p.in[kY] ? (p.post ? p.post[c] : 1.f) * (p.scale ? p.scale[c] : 1.f) : 0.f;
        };
        const auto total = [&](const LongSum &x, const LongSum &y) {
            all[0][warp][lane] = x.value();
            all[1][warp][lane] = y.value();
            __syncthreads();
            float2 s{0.f, 0.f};
            for (int w = 0; w < kNormWarps; ++w) {
                s.x += all[0][w][lane];
                s.y += all[1][w][lane];
            }
            __syncthreads();
            return s;
        };
        float q = 1.f, f = 0.f, back = 0.f, back_b = 0.f;
        if (p.post) {
            LongSum s, none;
            for (int c = warp; c < p.C; c += kNormWarps) {
                const float b = block(c);
                s.add(b * b);
            }
            q = total(s, none).x;
            q = in ? rsqrtf(fmaf(q, p.inv_C, p.eps)) : 0.f;
        }
        const auto sum_of = [&](int c) { return fmaf(weight(c), block(c) * q, read(kX, c)); };
        if (p.pre) {
            LongSum squares, slopes;
            for (int c = warp; c < p.C; c += kNormWarps) {
                const float v = sum_of(c);
                squares.add(v * v);
                slopes.add(read(kDout, c) * p.pre[c] * v);
            }
            const float2 s = total(squares, slopes);
            f = in ? rsqrtf(fmaf(s.x, p.inv_C, p.eps)) : 0.f;
            back = f * f * f * (s.y * p.inv_C);
        }
        const auto grad_of = [&](int c, float sum) {
            return fmaf(-sum, back, fmaf(f * (p.pre ? p.pre[c] : 0.f), read(kDout, c), read(kDsum, c)));
        };
        const int64_t to = (int64_t)n * p.C * p.L + t;
        LongSum s;
        for (int c = warp; c < p.C; c += kNormWarps) {
            const float sum = sum_of(c), b = block(c), g = grad_of(c, sum);
            s.add(g * weight(c) * b);
            float a0 = read(kDout, c) * (sum * f), a1 = g * (b * q);
            for (int d = 16; d; d >>= 1) {
                a0 += __shfl_xor_sync(~0u, a0, d);
                a1 += __shfl_xor_sync(~0u, a1, d);
            }
            if (lane == 0) {  // (the same thread for every tile)
                const bool first = job == (int64_t)blockIdx.x;
                to_pre[c] = first ? a0 : to_pre[c] + a0;
                to_both[c] = first ? a1 : to_both[c] + a1;
            }
            if (p.in[kX] && t < p.L) static_cast<T *>(p.dx)[to + (int64_t)c * p.L] = from_f32<T>(in ? g : 0.f);
        }
        if (!p.in[kY]) continue;
        if (p.post) {
            back_b = q * q * q * (total(s, LongSum{}).x * p.inv_C);
        }
        for (int c = warp; c < p.C; c += kNormWarps) {
            const float sum = sum_of(c), b = block(c);
            const float db = fmaf(-b, back_b, grad_of(c, sum) * weight(c) * q);
            if (t >= p.L) continue;
            const float z = read(kZ, c);
            static_cast<T *>(p.dy)[to + (int64_t)c * p.L] = from_f32<T>(!in ? 0.f : p.in[kZ] ? db * silu(z) : db);
            if (p.in[kZ])
                static_cast<T *>(p.dz)[to + (int64_t)c * p.L] = from_f32<T>(in ? db * read(kY, c) * silu_grad(z) : 0.f);
        }
    }
}

// The clusters' parts added: 32 channels of a block, eight threads to each.
__global__ void __launch_bounds__(kNormThreads) norm_join_kernel(const NormParams p) {
    __shared__ float sums[2][8][33];
    const int cx = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;
    float s0 = 0.f, s1 = 0.f;
    if (c < p.C)
        for (int o = part; o < p.clusters; o += 8) {
            s0 += p.partial[(int64_t)o * 2 * p.C + c];
            s1 += p.partial[((int64_t)o * 2 + 1) * p.C + c];
        }
    sums[0][part][cx] = s0;
    sums[1][part][cx] = s1;
    __syncthreads();
    if (part || c >= p.C) return;
    for (int o = 1; o < 8; ++o) {
        s0 += sums[0][o][cx];
        s1 += sums[1][o][cx];
    }
    if (p.dpre) p.dpre[c] = s0;
    if (p.dscale) p.dscale[c] = s1 * (p.post ? p.post[c] : 1.f);
    if (p.dpost) p.dpost[c] = s1 * (p.scale ? p.scale[c] : 1.f);
}

constexpr int kHeld = 8;  // bytes that a thread holds for each of its channels

// W of the tiles, 0 for the wide kernel.
int backward_plan(NormParams &p, int dtype, bool vec) {
    const int W = norm_plan(p, dtype, kHeld, vec);
    if (W == 0) {
        p.ranks = 1;
        p.tiles = (p.L - 1) / 32 + 1;
        p.jobs = (int64_t)p.N * p.tiles;
        p.clusters = (int)(p.jobs < 4 * kSMs ? p.jobs : 4 * kSMs);
    }
    return W;
}

}  // namespace
}  // namespace seq
}  // namespace spconv

using namespace spconv::seq;

SPCONV_API int64_t spconv_residual_norm_backward_workspace(const spconv_residual_norm_args *a) {
    if (norm_check(a) || a->C == 0 || a->N == 0 || a->L == 0) return 0;
    NormParams p = norm_params(a);  // (the larger plan's: whether rows are aligned depends on pointers)
    backward_plan(p, a->dtype, false);
    int most = p.clusters;
    backward_plan(p, a->dtype, true);
    if (p.clusters > most) most = p.clusters;
    return (int64_t)most * 2 * a->C * 4;
}

SPCONV_API int spconv_residual_norm_backward(const spconv_residual_norm_args *a, void *stream) {
    if (int st = norm_check(a)) return st;
    NormParams p = norm_params(a);
    const int64_t e = dtype_size(a->dtype), N = a->N, C = a->C, L = a->L, all = N * C * L;
    if (C == 0) return SPCONV_OK;
    if (!a->post != !a->dpost || !a->scale != !a->dscale || !a->pre != !a->dpre) return SPCONV_ERR_INVALID_ARG;
    if (all > 0 &&
        ((!a->x && !a->y) || (!a->y && (!a->pre || a->z || a->post || a->scale)) || !a->pre != !a->dout ||
         !a->x != !a->dx || !a->y != !a->dy || !a->z != !a->dz))
        return SPCONV_ERR_INVALID_ARG;
    if (!norm_on_elements(a, {a->x, a->y, a->z, a->dsum, a->dout, a->dx, a->dy, a->dz}) ||
        !norm_on_words({a->post, a->scale, a->pre, a->lengths, a->dpost, a->dscale, a->dpre}))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t need = spconv_residual_norm_backward_workspace(a);
    if (need && (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < need))
        return SPCONV_ERR_INVALID_ARG;
    const auto size = [&](int64_t sn, int64_t sc) { return extent(N, C, L, sn, sc, e); };
    if (!apart({{a->dx, all * e}, {a->dy, all * e}, {a->dz, all * e}, {a->dpost, C * 4}, {a->dscale, C * 4},
                {a->dpre, C * 4}, {a->workspace, need}},
               {{a->x, size(a->x_stride_n, a->x_stride_c)}, {a->y, size(a->y_stride_n, a->y_stride_c)},
                {a->z, size(a->z_stride_n, a->z_stride_c)}, {a->dsum, size(a->dsum_stride_n, a->dsum_stride_c)},
                {a->dout, size(a->dout_stride_n, a->dout_stride_c)}, {a->post, C * 4}, {a->scale, C * 4},
                {a->pre, C * 4}, {a->lengths, N * 4}}))
        return SPCONV_ERR_INVALID_ARG;
    p.partial = static_cast<float *>(a->workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (all > 0) {
        bool vec = rows_aligned(a->dx, 0, L, e) && rows_aligned(a->dy, 0, L, e) && rows_aligned(a->dz, 0, L, e);
        for (int i = 0; i < kNormInputs; ++i)
            vec = vec && (!p.in[i] || rows_aligned(p.in[i], p.in_sn[i], p.in_sc[i], e));
        const int W = backward_plan(p, a->dtype, vec);
        const int st = by_dtype(a->dtype, [&](auto t) {
            using T = decltype(t);
            if (W == 0) {
                norm_backward_wide_kernel<T><<<(unsigned)p.clusters, kNormThreads, 0, s>>>(p);
                return launch_status();
            }
            void (*fn)(NormParams) =
                vec ? (W == 8 ? norm_backward_kernel<T, 8, true> : W == 4 ? norm_backward_kernel<T, 4, true>
                                                                          : norm_backward_kernel<T, 2, true>)
                    : (W == 8 ? norm_backward_kernel<T, 8, false> : W == 4 ? norm_backward_kernel<T, 4, false>
                                                                           : norm_backward_kernel<T, 2, false>);
            return norm_launch(fn, p, stream);
        });
        if (st) return st;
    }
    if (!p.dpost && !p.dscale && !p.dpre) return SPCONV_OK;
    norm_join_kernel<<<(unsigned)((C + 31) / 32), kNormThreads, 0, s>>>(p);
    return launch_status();
}
