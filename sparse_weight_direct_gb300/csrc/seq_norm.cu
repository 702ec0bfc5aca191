// The norms before and after a block with its gate and residual scale.
//
//   b = y silu(z),  p = post b / rms(b),  sum = x + scale p,  out = pre sum / rms(sum)
//
// with rms(v) = sqrt(mean of v^2 over the channels + eps) at each position.
//
// Bound: about twenty operations per element against two bytes (four in float32)
// for each of x, y, z, sum and out: the memory bandwidth.
#include "seq_norm.cuh"

namespace spconv {
namespace seq {
namespace {

// Channels-first rows put a position's channels L elements apart, so a cluster of
// blocks takes a tile of positions with all their channels, a part of them in each
// block's shared memory, while the next tile's are on their way.
//
// Both norms come from one pass of sums: with w = scale post and q = 1 / rms(b),
//   sum of (x + w q b)^2 = sum x^2 + 2 q sum w x b + q^2 sum w^2 b^2,
// so that a tile waits for its cluster once.  Where x and w q b cancel to less than
// an eighth of their squares, the sum is formed again from its terms.
//
// 8 x 2048 x 2048 in bf16 take 89 us, 0.55 of the measured bandwidth: 53 instructions
// an element at 0.53 an SMSP and clock, 16 warps to an SM.  The tile in registers and a
// pass for each norm: 190 us; single floats and two more clusters than run at once: 215;
// pairs, and b kept in float32: 97; three blocks of 80 registers: 93.
template <typename T, int W, bool VEC>
__global__ void __launch_bounds__(kNormThreads, 2) norm_tile_kernel(const __grid_constant__ NormParams p) {
    using Tile = NormTile<T, W, VEC>;
    constexpr int V = Tile::V, H = V / 2, K = 4;
    extern __shared__ uint4 shared[];
    auto &sm = *reinterpret_cast<NormSums<K, W, V> *>(
        shared + p.stages * p.inputs * p.R * (kNormThreads + (VEC ? 0 : Tile::ROWS)));
    float2 *weights = reinterpret_cast<float2 *>(&sm + 1) + threadIdx.x / W;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = p.ranks > 1 ? (int)cluster.block_rank() : 0;
    const unsigned id = blockIdx.x / p.ranks;
    Tile tile(p, shared, rank);
    int stage = 0, parity = 0;
    tile.place(id, 0);
    tile.fetch();
    tile.weights(reinterpret_cast<float2 *>(&sm + 1));
    if (p.ranks > 1) cluster.sync();  // the others' shared memory is there
    const bool gated = p.in[kZ];
    // b, as float32 in the slots of y and z
    const auto block = [&](f32x2 (&b)[H], int o) {
        if (gated) {
            const float4 lo = *reinterpret_cast<const float4 *>(tile.at(kY, o));
            b[0] = pack2(lo.x, lo.y), b[1] = pack2(lo.z, lo.w);
            if constexpr (H == 4) {
                const float4 hi = *reinterpret_cast<const float4 *>(tile.at(kZ, o));
                b[2] = pack2(hi.x, hi.y), b[3] = pack2(hi.z, hi.w);
            }
        } else {
            tile.pairs(b, kY, o);
        }
    };
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
                const f32x2 w = both(weights[k * Tile::ROWS].x);
                f32x2 x[H], b[H];
                tile.pairs(x, kX, o);
                tile.pairs(b, kY, o);
                if (gated) {
                    f32x2 z[H];
                    tile.pairs(z, kZ, o);
    #pragma unroll
                    for (int j = 0; j < H; ++j) b[j] = mul2(b[j], mul2(z[j], sigmoid2(z[j])));
                    const float2 f0 = unpack2(b[0]), f1 = unpack2(b[1]);
                    *reinterpret_cast<float4 *>(tile.at(kY, o)) = make_float4(f0.x, f0.y, f1.x, f1.y);
                    if constexpr (H == 4) {
                        const float2 f2 = unpack2(b[2]), f3 = unpack2(b[3]);
                        *reinterpret_cast<float4 *>(tile.at(kZ, o)) = make_float4(f2.x, f2.y, f3.x, f3.y);
                    }
                }
    #pragma unroll
                for (int j = 0; j < H; ++j) {
                    const f32x2 wb = mul2(w, b[j]);
                    v[j] = fma2(b[j], b[j], v[j]);
                    v[H + j] = fma2(x[j], x[j], v[H + j]);
                    v[2 * H + j] = fma2(wb, x[j], v[2 * H + j]);
                    v[3 * H + j] = fma2(wb, wb, v[3 * H + j]);
                }
            }
            const bool again = sum_tile<K, V, W>(v, sm, p.ranks, rank, parity, [&](int t, const float (&s)[K], bool store) {
                const float q = p.post ? rsqrtf(fmaf(s[0], p.inv_C, p.eps)) : 1.f;
                const float apart = fmaf(q * q, s[3], s[1]), sum = fmaf(2.f * q, s[2], apart);
                const bool in = tile.first + t < tile.end;
                if (store) {
                    sm.held[t].x = in ? q : 0.f;
                    sm.held[t].y = in && p.pre ? rsqrtf(fmaf(sum, p.inv_C, p.eps)) : 0.f;
                }
                return p.pre && in && sum < 0.125f * apart;
            });
            parity ^= 1;
            f32x2 q[H], t[H];
            const auto factors = [&]() {
    #pragma unroll
                for (int j = 0; j < H; ++j) {
                    const float4 f = *reinterpret_cast<const float4 *>(&sm.held[tile.tx * V + 2 * j]);
                    q[j] = pack2(f.x, f.z);
                    t[j] = pack2(f.y, f.w);
                }
            };
            factors();
            if (again) {
                f32x2 u[H] = {};
                for (int k = 0, o = tile.origin; k < p.R; ++k, o += kNormThreads) {
                    const f32x2 w = both(weights[k * Tile::ROWS].x);
                    f32x2 x[H], b[H];
                    tile.pairs(x, kX, o);
                    block(b, o);
    #pragma unroll
                    for (int j = 0; j < H; ++j) {
                        const f32x2 s = fma2(mul2(w, q[j]), b[j], x[j]);
                        u[j] = fma2(s, s, u[j]);
                    }
                }
                sum_tile<1, V, W>(u, sm, p.ranks, rank, parity, [&](int at, const float (&s)[1], bool store) {
                    if (store) sm.held[at].y = tile.first + at < tile.end ? rsqrtf(fmaf(s[0], p.inv_C, p.eps)) : 0.f;
                    return false;
                });
                parity ^= 1;
                factors();
            }
            int c = tile.c0;
            int64_t to = tile.out;
            for (int k = 0, o = tile.origin; k < p.R; ++k, o += kNormThreads, c += Tile::ROWS, to += tile.out_step) {
                const float2 w = weights[k * Tile::ROWS];
                f32x2 x[H], s[H];
                tile.pairs(x, kX, o);
                block(s, o);
    #pragma unroll
                for (int j = 0; j < H; ++j) s[j] = fma2(mul2(both(w.x), q[j]), s[j], x[j]);
                if (p.sum) tile.give(p.sum, s, c, to);
                if (p.pre) {
    #pragma unroll
                    for (int j = 0; j < H; ++j) s[j] = mul2(s[j], mul2(both(w.y), t[j]));
                    tile.give(p.out, s, c, to);
                }
            }
        };
        if (tile.empty()) {
            tile.clear(p.sum);
            tile.clear(p.out);
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
}

// Single tokens: a row of contiguous channels to a block.  A thread keeps its
// channels in registers where they are no more than two runs, and reads them again
// for each sum else.
template <typename T, int V>
__global__ void __launch_bounds__(1024) norm_token_kernel(const NormParams p) {
    __shared__ float sums[2][32];
    const int n = blockIdx.x, step = blockDim.x * V, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (p.lengths && p.lengths[n] <= 0) {
        for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
            if (p.sum) static_cast<T *>(p.sum)[(int64_t)n * p.C + c] = from_f32<T>(0.f);
            if (p.pre) static_cast<T *>(p.out)[(int64_t)n * p.C + c] = from_f32<T>(0.f);
        }
        return;
    }
    const auto read = [&](int input, float (&v)[V], int c) {
        if (p.in[input] && c < p.C) take(v, static_cast<const T *>(p.in[input]) + n * p.in_sn[input] + c);
        else
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = 0.f;
    };
    const auto block = [&](float (&b)[V], int c) {
        read(kY, b, c);
        if (p.in[kZ]) {
            float z[V];
            read(kZ, z, c);
#pragma unroll
            for (int j = 0; j < V; ++j) b[j] *= silu(z[j]);
        }
    };
    const auto weight = [&](float (&w)[V], int c) {
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] = p.in[kY] && c < p.C ? 1.f : 0.f;
        for (const float *from : {p.post, p.scale})
            if (from && c < p.C) {
                float f[V];
                take(f, from + c);
#pragma unroll
                for (int j = 0; j < V; ++j) w[j] *= f[j];
            }
    };
    const auto total = [&](float s, int place) {
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        if (lane == 0) sums[place][warp] = s;
        __syncthreads();
        s = lane < (int)blockDim.x / 32 ? sums[place][lane] : 0.f;
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        return s;
    };
    constexpr int kKept = 2;
    const bool kept = p.C <= kKept * step;
    float b[kKept][V], x[kKept][V];
    const int c0 = threadIdx.x * V;
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        read(kX, x[k], c0 + k * step);
        block(b[k], c0 + k * step);
    }
    float q = 1.f;
    if (p.post) {
        float s = 0.f;
        if (kept) {
#pragma unroll
            for (int k = 0; k < kKept; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) s = fmaf(b[k][j], b[k][j], s);
        } else {
            LongSum all;
            for (int c = c0; c < p.C; c += step) {
                block(b[0], c);
                float part = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j) part = fmaf(b[0][j], b[0][j], part);
                all.add(part);
            }
            s = all.value();
        }
        q = rsqrtf(fmaf(total(s, 0), p.inv_C, p.eps));
    }
    // x + w q b in b
    const auto sum_up = [&](float (&to)[V], const float (&from)[V], int c) {
        float w[V];
        weight(w, c);
#pragma unroll
        for (int j = 0; j < V; ++j) to[j] = fmaf(w[j], to[j] * q, from[j]);
        if (p.sum && c < p.C) give(to, static_cast<T *>(p.sum) + (int64_t)n * p.C + c);
    };
    float s = 0.f;
    if (kept) {
#pragma unroll
        for (int k = 0; k < kKept; ++k) {
            sum_up(b[k], x[k], c0 + k * step);
#pragma unroll
            for (int j = 0; j < V; ++j) s = fmaf(b[k][j], b[k][j], s);
        }
    } else {
        LongSum all;
        for (int c = c0; c < p.C; c += step) {
            read(kX, x[0], c);
            block(b[0], c);
            sum_up(b[0], x[0], c);
            float part = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) part = fmaf(b[0][j], b[0][j], part);
            all.add(part);
        }
        s = all.value();
    }
    if (!p.pre) return;
    const float t = rsqrtf(fmaf(total(s, 1), p.inv_C, p.eps));
    const auto out = [&](float (&v)[V], int c) {
        if (c >= p.C) return;
        float w[V];
        take(w, p.pre + c);
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] *= v[j] * t;
        give(w, static_cast<T *>(p.out) + (int64_t)n * p.C + c);
    };
    if (kept) {
#pragma unroll
        for (int k = 0; k < kKept; ++k) out(b[k], c0 + k * step);
    } else {
        for (int c = c0; c < p.C; c += step) {
            read(kX, x[0], c);
            block(b[0], c);
            sum_up(b[0], x[0], c);
            out(b[0], c);
        }
    }
}

// More channels than a cluster holds: a block for 32 positions, whose rows are
// read again (from the cache where they fit) for each sum.  Few blocks, each with one
// load of 64 or 128 bytes a warp on its way: 4 x 15,400 x 512 in bf16 take 3.2 ms (15,360
// channels, in clusters, 0.146).
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_wide_kernel(const NormParams p) {
    __shared__ float sums[kNormWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = (int)(blockIdx.x / p.tiles), t = (int)(blockIdx.x - (unsigned)n * p.tiles) * 32 + lane;
    const int end = p.lengths ? min(max(p.lengths[n], 0), p.L) : p.L;
    const bool in = t < end;
    const auto read = [&](int input, int c) {
        return p.in[input] && in ? to_f32(static_cast<const T *>(p.in[input])[n * p.in_sn[input] + c * p.in_sc[input] + t])
                                 : 0.f;
    };
    const auto block = [&](int c) {
        const float y = read(kY, c);
        return p.in[kZ] ? y * silu(read(kZ, c)) : y;
    };
    const auto total = [&](float s) {
        sums[warp][lane] = s;
        __syncthreads();
        s = 0.f;
        for (int w = 0; w < kNormWarps; ++w) s += sums[w][lane];
        __syncthreads();
        return s;
    };
    float q = 1.f;
    if (p.post) {
        LongSum s;
        for (int c = warp; c < p.C; c += kNormWarps) {
            const float b = block(c);
            s.add(b * b);
        }
        q = rsqrtf(fmaf(total(s.value()), p.inv_C, p.eps));
    }
    const auto sum_of = [&](int c) {
        const float w = p.in[kY] ? (p.post ? p.post[c] : 1.f) * (p.scale ? p.scale[c] : 1.f) : 0.f;
        return in ? fmaf(w, block(c) * q, read(kX, c)) : 0.f;
    };
    const int64_t to = (int64_t)n * p.C * p.L + t;
    LongSum s;
    for (int c = warp; c < p.C; c += kNormWarps) {
        const float v = sum_of(c);
        s.add(v * v);
        if (p.sum && t < p.L) static_cast<T *>(p.sum)[to + (int64_t)c * p.L] = from_f32<T>(v);
    }
    if (!p.pre) return;
    const float f = rsqrtf(fmaf(total(s.value()), p.inv_C, p.eps));
    for (int c = warp; c < p.C; c += kNormWarps) {
        const float v = sum_of(c);
        if (t < p.L) static_cast<T *>(p.out)[to + (int64_t)c * p.L] = from_f32<T>(in ? p.pre[c] * (v * f) : 0.f);
    }
}

}  // namespace

// ---------------------------------------------------------------- host side

int norm_check(const spconv_residual_norm_args *a) {
    if (!a || a->N < 0 || a->C < 0 || a->L < 0) return SPCONV_ERR_INVALID_ARG;
    if (a->dtype < SPCONV_F32 || a->dtype > SPCONV_F16 || !(a->eps >= 0.f)) return SPCONV_ERR_INVALID_ARG;
    if (a->N > kMaxLength || a->L > kMaxLength || a->C > 1 << 26) return SPCONV_ERR_UNSUPPORTED;
    for (int64_t s : {a->x_stride_n, a->x_stride_c, a->y_stride_n, a->y_stride_c, a->z_stride_n, a->z_stride_c,
                      a->dsum_stride_n, a->dsum_stride_c, a->dout_stride_n, a->dout_stride_c})
        if (!stride_ok(s)) return SPCONV_ERR_INVALID_ARG;
    return SPCONV_OK;
}

NormParams norm_params(const spconv_residual_norm_args *a) {
    NormParams p{};
    const int64_t e = dtype_size(a->dtype);
    const void *in[] = {a->x, a->y, a->z, a->dout, a->dsum};
    const int64_t sn[] = {a->x_stride_n, a->y_stride_n, a->z_stride_n, a->dout_stride_n, a->dsum_stride_n};
    const int64_t sc[] = {a->x_stride_c, a->y_stride_c, a->z_stride_c, a->dout_stride_c, a->dsum_stride_c};
    for (int i = 0; i < kNormInputs; ++i) {
        p.in[i] = in[i];
        p.in_sn[i] = sn[i];
        p.in_sc[i] = sc[i];
        p.in_end[i] = in[i] ? static_cast<const char *>(in[i]) + extent(a->N, a->C, a->L, sn[i], sc[i], e) : nullptr;
    }
    p.post = a->post; p.scale = a->scale; p.pre = a->pre; p.lengths = a->lengths;
    p.sum = a->sum; p.out = a->out; p.dx = a->dx; p.dy = a->dy; p.dz = a->dz;
    p.dpost = a->dpost; p.dscale = a->dscale; p.dpre = a->dpre;
    p.eps = a->eps;
    p.N = a->N; p.C = a->C; p.L = a->L;
    return p;
}

bool norm_on_elements(const spconv_residual_norm_args *a, std::initializer_list<const void *> ps) {
    for (const void *q : ps)
        if (q && !aligned(q, dtype_size(a->dtype))) return false;
    return true;
}
bool norm_on_words(std::initializer_list<const void *> ps) {
    for (const void *q : ps)
        if (q && !aligned(q, 4)) return false;
    return true;
}

// A cluster that does not fit beside the others runs its share of the tiles behind
// all of them, so there are no more than run at once (36 of eight blocks where two
// blocks fit an SM, not 38: its SMs come in groups).  Asked once for each kernel,
// size and device.
static int clusters_at_once(void (*fn)(NormParams), const cudaLaunchConfig_t &cfg, int ranks) {
    struct Known {
        void (*fn)(NormParams);
        int device, ranks, shared, count;
    };
    static std::mutex lock;
    static Known known[128];
    static int filled = 0;
    int device = 0, count = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return 0;
    const int shared = (int)cfg.dynamicSmemBytes;
    std::lock_guard<std::mutex> hold(lock);
    for (int i = 0; i < filled; ++i)
        if (known[i].fn == fn && known[i].device == device && known[i].ranks == ranks && known[i].shared == shared)
            return known[i].count;
    if (ranks > 1) {
        if (cudaOccupancyMaxActiveClusters(&count, fn, &cfg) != cudaSuccess) return 0;
    } else {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&count, fn, kNormThreads, shared) != cudaSuccess) return 0;
        count *= kSMs;
    }
    if (filled < 128) known[filled++] = {fn, device, ranks, shared, count};
    return count;
}

int norm_launch(void (*fn)(NormParams), NormParams &p, void *stream) {
    if (int st = raise_smem(reinterpret_cast<const void *>(fn), kNormShared)) return st;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.clusters * p.ranks));
    cfg.blockDim = dim3(kNormThreads);
    cfg.dynamicSmemBytes = p.shared;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.ranks > 1;
    const int most = clusters_at_once(fn, cfg, p.ranks);
    if (most < 1) {
        cudaGetLastError();
        return SPCONV_ERR_CUDA;
    }
    if (p.clusters > most) p.clusters = most;
    cfg.gridDim = dim3((unsigned)(p.clusters * p.ranks));
    if (cudaLaunchKernelEx(&cfg, fn, p) != cudaSuccess) {
        cudaGetLastError();
        return SPCONV_ERR_CUDA;
    }
    return SPCONV_OK;
}

}  // namespace seq
}  // namespace spconv

using namespace spconv::seq;

SPCONV_API int spconv_residual_norm(const spconv_residual_norm_args *a, void *stream) {
    if (int st = norm_check(a)) return st;
    NormParams p = norm_params(a);
    const int64_t e = dtype_size(a->dtype), N = a->N, C = a->C, L = a->L, all = N * C * L;
    if (all == 0) return SPCONV_OK;
    if ((!a->x && !a->y) || (!a->y && (!a->pre || a->z || a->post || a->scale)) || !a->sum != !a->y ||
        !a->out != !a->pre)
        return SPCONV_ERR_INVALID_ARG;
    if (!norm_on_elements(a, {a->x, a->y, a->z, a->sum, a->out}) ||
        !norm_on_words({a->post, a->scale, a->pre, a->lengths}))
        return SPCONV_ERR_INVALID_ARG;
    const auto size = [&](const void *, int64_t sn, int64_t sc) { return extent(N, C, L, sn, sc, e); };
    if (!apart({{a->sum, all * e}, {a->out, all * e}},
               {{a->x, size(a->x, a->x_stride_n, a->x_stride_c)}, {a->y, size(a->y, a->y_stride_n, a->y_stride_c)},
                {a->z, size(a->z, a->z_stride_n, a->z_stride_c)}, {a->post, C * 4}, {a->scale, C * 4},
                {a->pre, C * 4}, {a->lengths, N * 4}}))
        return SPCONV_ERR_INVALID_ARG;
    p.in[kDout] = p.in[kDsum] = nullptr;  // (the backward pass' alone)
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const auto along = [&](const void *q, int64_t sc) { return !q || sc == 1; };
    if (L == 1 && along(a->x, a->x_stride_c) && along(a->y, a->y_stride_c) && along(a->z, a->z_stride_c)) {
        // eight channels to a load (four in float32) where every row allows it
        const int V = 16 / (int)e;
        bool vec = C % V == 0 && aligned(a->sum, 16) && aligned(a->out, 16);
        for (const float *q : {p.post, p.scale, p.pre}) vec = vec && aligned(q, 16);
        for (int i = kX; i <= kZ; ++i) vec = vec && (!p.in[i] || rows_aligned(p.in[i], p.in_sn[i], 0, e));
        p.inv_C = 1.f / (float)C;
        const int64_t want = (C + 2 * (vec ? V : 1) - 1) / (2 * (vec ? V : 1));
        int threads = 32;
        while (threads < 1024 && threads < want) threads *= 2;
        return by_dtype(a->dtype, [&](auto t) {
            using T = decltype(t);
            if (vec)
                norm_token_kernel<T, 16 / sizeof(T)><<<(unsigned)N, threads, 0, s>>>(p);
            else
                norm_token_kernel<T, 1><<<(unsigned)N, threads, 0, s>>>(p);
            return launch_status();
        });
    }
    bool vec = rows_aligned(a->sum, 0, L, e) && rows_aligned(a->out, 0, L, e);
    for (int i = kX; i <= kZ; ++i) vec = vec && (!p.in[i] || rows_aligned(p.in[i], p.in_sn[i], p.in_sc[i], e));
    const int W = norm_plan(p, a->dtype, 0, vec);
    return by_dtype(a->dtype, [&](auto t) {
        using T = decltype(t);
        if (W == 0) {
            p.tiles = (a->L - 1) / 32 + 1;
            if (N * p.tiles > 0x7fffffff) return (int)SPCONV_ERR_UNSUPPORTED;
            norm_wide_kernel<T><<<(unsigned)(N * p.tiles), kNormThreads, 0, s>>>(p);
            return launch_status();
        }
        void (*fn)(NormParams) =
            vec ? (W == 8 ? norm_tile_kernel<T, 8, true> : W == 4 ? norm_tile_kernel<T, 4, true>
                                                                  : norm_tile_kernel<T, 2, true>)
                : (W == 8 ? norm_tile_kernel<T, 8, false> : W == 4 ? norm_tile_kernel<T, 4, false>
                                                                   : norm_tile_kernel<T, 2, false>);
        return norm_launch(fn, p, stream);
    });
}
