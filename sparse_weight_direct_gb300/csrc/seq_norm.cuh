// Internal: what the block norms' forward pass (seq_norm.cu) and their gradients
// (seq_norm_backward.cu) share.
#pragma once

#include <cooperative_groups.h>

#include "seq_common.cuh"

namespace spconv {
namespace seq {

namespace cg = cooperative_groups;

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kNormRanks = 8;             // blocks of a cluster
constexpr int kNormInputs = 5;            // x, y, z, dout, dsum
constexpr int kNormShared = 224 * 1024;   // bytes of a block at most
constexpr int kNormRow = kNormThreads * 16;  // bytes of one load of every thread

struct NormParams {
    // x, y, z and, backward, dout and dsum; NULL where absent
    const void *in[kNormInputs], *in_end[kNormInputs];
    int64_t in_sn[kNormInputs], in_sc[kNormInputs];
    int slot[kNormInputs];  // the input's place in a stage
    const float *post, *scale, *pre;
    const int32_t *lengths;
    void *sum, *out, *dx, *dy, *dz;
    float *dpost, *dscale, *dpre;
    float *partial;      // clusters x 2 x C: sums of dout s t and of G n
    int64_t jobs;        // tiles of all sequences
    float eps, inv_C;
    int N, C, L;
    int tiles;           // of a sequence
    int ranks, per;      // blocks of a cluster; channels of a block
    int inputs;          // how many are given
    int R;               // runs of a thread in a tile
    int stages;          // tiles on their way
    int clusters;        // that share the tiles
    int shared;          // bytes of a block
};
enum { kX, kY, kZ, kDout, kDsum };

// ---------------------------------------------------------------- runs

// Elements behind the first `keep` of a run are zeros.
template <typename T, int V>
static __device__ __forceinline__ void cut(Run<T, V> &run, int keep) {
#pragma unroll
    for (int k = 0; k < Run<T, V>::W; ++k) {
        if constexpr (sizeof(T) == 4)
            run.w[k] = k < keep ? run.w[k] : 0;
        else
            run.w[k] &= (2 * k < keep ? 0xffffu : 0u) | (2 * k + 1 < keep ? 0xffff0000u : 0u);
    }
}

static __device__ __forceinline__ f32x2 both(float v) { return pack2(v, v); }
static __device__ __forceinline__ f32x2 sigmoid2(f32x2 v) {
    const float2 e = unpack2(add2(ex2_2(mul2(v, both(-kLog2e))), both(1.f)));
    return pack2(rcp(e.x), rcp(e.y));
}

// ---------------------------------------------------------------- a tile's sums

// Shared memory behind the stages.
template <int K, int W, int V>
struct NormSums {
    static constexpr int TILE = W * V;
    static constexpr int kRanks = W == 8 ? 1 : kNormRanks;  // (the widest tiles have one block)
    float warps[kNormWarps][K * TILE];
    float ranks[2][kRanks][K * TILE];  // by a tile's parity
    float4 factors[TILE];
    float2 held[TILE];
};

// K sums over the channels at each position of a tile: u[k * V / 2 + j] is a thread's
// part at its positions 2 j and 2 j + 1.  derive(position, sums) is called for each position
// by eight neighbouring lanes with the whole cluster's sums, the last argument
// telling the one that is to store what it makes of them; its values of truth are
// joined over the block, and so alike in the whole cluster.
//
// Lanes of a warp that hold other channels first halve their values among them, so
// that a sum costs about one shuffle; warps, then blocks, are added in a fixed order.
template <int K, int V, int W, typename S, typename F>
static __device__ __forceinline__ bool sum_tile(const f32x2 (&u)[K * V / 2], S &sm, int ranks, int rank, int parity, F derive) {
    constexpr int TILE = W * V, N = K * V;
    constexpr int kHalvings = N % 8 == 0 ? 3 : 2;  // (V is 4 or 8)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tx = lane & (W - 1);
    float v[N];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) v[2 * i] = unpack2(u[i]).x, v[2 * i + 1] = unpack2(u[i]).y;
    int base = 0, d = 16;
    bool writes = true;
    int n = N;
#pragma unroll
    for (int level = 0; level < 5; ++level, d >>= 1) {
        if (d < W) break;
        if (level < kHalvings) {
            const bool up = lane & d;
            n >>= 1;
#pragma unroll
            for (int i = 0; i < (N >> (level + 1)); ++i) {
                const int hi = i + (N >> (level + 1));
                const float give = up ? v[i] : v[hi], keep = up ? v[hi] : v[i];
                v[i] = keep + __shfl_xor_sync(~0u, give, d);
            }
            if (up) base += n;
        } else {
#pragma unroll
            for (int i = 0; i < (N >> kHalvings); ++i) v[i] += __shfl_xor_sync(~0u, v[i], d);
            writes = writes && !(lane & d);
        }
    }
    constexpr int kLevels = W == 8 ? 2 : W == 4 ? 3 : 4;
    constexpr int kLeft = N >> (kLevels < kHalvings ? kLevels : kHalvings);
    if (writes)
#pragma unroll
        for (int i = 0; i < kLeft; ++i) {
            const int o = base + i;
            sm.warps[warp][o / V * TILE + tx * V + o % V] = v[i];
        }
    __syncthreads();
    cg::cluster_group cluster = cg::this_cluster();
    for (int o = threadIdx.x; o < K * TILE; o += kNormThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kNormWarps; ++w) s += sm.warps[w][o];
        float *mine = &sm.ranks[parity][rank][o];
        if (ranks > 1)
            for (int q = 0; q < ranks; ++q) *cluster.map_shared_rank(mine, q) = s;
        else
            *mine = s;
    }
    if (ranks > 1)
        cluster.sync();
    else
        __syncthreads();
    bool flag = false;
    const int r = threadIdx.x & 7;
    for (int t = threadIdx.x >> 3; t < TILE; t += kNormThreads / 8) {  // (a warp has four positions or none)
        float s[K];
#pragma unroll
        for (int k = 0; k < K; ++k) s[k] = r < ranks ? sm.ranks[parity][r][k * TILE + t] : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int o = 4; o; o >>= 1) s[k] += __shfl_xor_sync(~0u, s[k], o);
        flag |= derive(t, s, r == 0);
    }
    return __syncthreads_or(flag);
}

// ---------------------------------------------------------------- a tile's runs

// The stages of a block: the runs that each thread reads, in slots of its own, so
// that nothing but the thread's own copies has to be waited for.
template <typename T, int W, bool VEC>
struct NormTile {
    static constexpr int V = 16 / sizeof(T), TILE = W * V, ROWS = kNormThreads / W;
    const NormParams &p;
    uint4 *slots;
    int off[kNormInputs];  // an input's slots in a stage
    int tx, c0, c_end;
    int64_t out_step;      // between a thread's rows of an output
    // of the tile in work
    int n, first, t0, end;
    int origin;            // the thread's first slot of the stage
    int64_t out;           // its first run of an output

    __device__ __forceinline__ NormTile(const NormParams &p_, uint4 *slots_, int rank) : p(p_), slots(slots_) {
        tx = threadIdx.x & (W - 1);
        c0 = rank * p.per + (int)threadIdx.x / W;
        c_end = min(p.C, (rank + 1) * p.per);
        out_step = (int64_t)ROWS * p.L;
#pragma unroll
        for (int i = 0; i < kNormInputs; ++i) off[i] = p.slot[i] * p.R * kNormThreads;
    }
    __device__ __forceinline__ void place(unsigned job, int stage) {
        n = (int)(job / (unsigned)p.tiles);
        first = (int)(job - (unsigned)n * (unsigned)p.tiles) * TILE;
        t0 = first + tx * V;
        end = p.lengths ? min(max(p.lengths[n], 0), p.L) : p.L;
        origin = stage * p.inputs * p.R * kNormThreads + (int)threadIdx.x;
        out = ((int64_t)n * p.C + c0) * p.L + t0;
    }
    // Slots are numbered by o, `origin` for a thread's first channel (c0) and
    // kNormThreads more for each further one (ROWS more).
    __device__ __forceinline__ uint4 *at(int input, int o) const { return slots + (off[input] + o); }
    // Unaligned rows have one more word, in a slot behind the stages' others.
    __device__ __forceinline__ uint4 *tail(int input) const {
        return slots + p.stages * p.inputs * p.R * kNormThreads +
               ((origin - (int)threadIdx.x + off[input]) / W + (int)threadIdx.x / W);
    }
    // Sends for the tile that was placed.
    __device__ __forceinline__ void fetch() const {
#pragma unroll
        for (int i = 0; i < kNormInputs; ++i) {
            if (!p.in[i] || empty()) continue;
            const T *from = static_cast<const T *>(p.in[i]) + n * p.in_sn[i] + c0 * p.in_sc[i] + t0;
            const int64_t step = ROWS * p.in_sc[i];
            int c = !VEC || t0 < end ? c0 : c_end;
            if (VEC) {
                uint32_t to = (uint32_t)__cvta_generic_to_shared(at(i, origin));
                for (int k = 0; k < p.R; ++k, c += ROWS, from += step, to += kNormRow)
                    // (0 bytes are read, and zeros written, where there is no channel or position)
                    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to),
                                 "l"(c < c_end ? from : static_cast<const T *>(p.in[i])), "r"(c < c_end ? 16 : 0)
                                 : "memory");
                continue;
            }
            const uintptr_t nowhere = reinterpret_cast<uintptr_t>(p.in[i]) & ~(uintptr_t)15;  // (not read)
            // a word that is to be read, or zeros
            const auto send = [&](uint4 *slot, const T *word, int t) {
                const bool on = c < c_end && t < end;
                if (!on || (word >= static_cast<const T *>(p.in[i]) && word + V <= static_cast<const T *>(p.in_end[i]))) {
                    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(
                                     (uint32_t)__cvta_generic_to_shared(slot)),
                                 "l"(on ? reinterpret_cast<uintptr_t>(word) : nowhere), "r"(on ? 16 : 0)
                                 : "memory");
                    return;
                }
                Run<T, V> run;  // across the tensor's ends: what lies inside
                run.clear();
                constexpr int per = 4 / sizeof(T);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (t + j >= 0 && t + j < end) run.w[j / per] |= bits_of(word[j]) << (j % per * 16);
                *reinterpret_cast<Run<T, V> *>(slot) = run;
            };
            uint4 *to = at(i, origin), *to_tail = tail(i);
            for (int k = 0; k < p.R; ++k, c += ROWS, from += step, to += kNormThreads, to_tail += ROWS) {
                const int o = (int)((uintptr_t)from & 15) / (int)sizeof(T);  // the row's place in its words
                send(to, from - o, t0 - o);
                if (tx == W - 1 && o) send(to_tail, from - o + V, t0 - o + V);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // A tile behind its sequence's end (the same for the whole cluster) has zeros alone.
    __device__ __forceinline__ bool empty() const { return first >= end; }
    __device__ __forceinline__ void clear(void *base) const {
        f32x2 none[V / 2] = {};
        int c = c0;
        int64_t to = out;
        for (int k = 0; base && k < p.R; ++k, c += ROWS, to += out_step) give(base, none, c, to);
    }
    // The tile is there; what lies behind the sequence's end is not.  Unaligned rows are
    // put into place: a run lies across the words of its thread and the next one.
    __device__ __forceinline__ void arrived(bool others) const {
        if (others)
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        else
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (empty()) return;
        if (!VEC) __syncwarp();
        if (!VEC || (t0 < end && t0 + V > end))
#pragma unroll
            for (int i = 0; i < kNormInputs; ++i) {
                if (!p.in[i]) continue;
                Run<T, V> *slot = reinterpret_cast<Run<T, V> *>(at(i, origin));
                unsigned off = 0, step = 0;
                const uint4 *last = nullptr;
                if (!VEC) {
                    off = (unsigned)(uintptr_t)(static_cast<const T *>(p.in[i]) + n * p.in_sn[i] + c0 * p.in_sc[i] + t0);
                    step = (unsigned)(ROWS * p.in_sc[i] * sizeof(T));
                    last = tail(i);
                }
#pragma unroll 2
                for (int k = 0; k < p.R; ++k, slot += kNormThreads, off += step, last += ROWS) {
                    Run<T, V> run = *slot;
                    if (!VEC) {
                        const uint4 hi = tx == W - 1 ? *last : reinterpret_cast<const uint4 *>(slot)[1];
                        uint32_t s[8] = {run.w[0], run.w[1], run.w[2], run.w[3], hi.x, hi.y, hi.z, hi.w};
                        run_across(run, s, off & 15);
                        __syncwarp();
                    }
                    if (t0 + V > end) cut(run, end - t0);
                    *slot = run;
                }
            }
    }
    // A run's values, two to a word of 64 bits; zeros of an input that is not there.
    __device__ __forceinline__ void pairs(f32x2 (&v)[V / 2], int input, int o) const {
        if (p.in[input]) {
            const Run<T, V> r = *reinterpret_cast<const Run<T, V> *>(at(input, o));
#pragma unroll
            for (int j = 0; j < V / 2; ++j) v[j] = pair_of(r, 2 * j);
        } else {
#pragma unroll
            for (int j = 0; j < V / 2; ++j) v[j] = 0;
        }
    }
    // The block's weights: w = scale post (0 without y) and pre of each of its channels.
    __device__ __forceinline__ void weights(float2 *to) const {
        for (int o = threadIdx.x; o < ROWS * p.R; o += kNormThreads) {
            const int c = c0 - (int)threadIdx.x / W + o;
            const bool on = c < c_end;
            to[o].x = on && p.in[kY] ? (p.post ? p.post[c] : 1.f) * (p.scale ? p.scale[c] : 1.f) : 0.f;
            to[o].y = on && p.pre ? p.pre[c] : 0.f;
        }
        __syncthreads();
    }
    // A run of an output, N x C x L, of channel c at place `to`.  Unaligned rows are
    // stored as the aligned words that lie within the tile, each from two threads'
    // runs, and single elements at its ends.
    __device__ __forceinline__ void give(void *base, const f32x2 (&v)[V / 2], int c, int64_t to) const {
        Run<T, V> run;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            const float2 f = unpack2(v[j]);
            if constexpr (sizeof(T) == 4)
                run.w[2 * j] = __float_as_uint(f.x), run.w[2 * j + 1] = __float_as_uint(f.y);
            else
                run.w[j] = f32_to_word<T>(f.x, f.y);
        }
        if (t0 + V > end) cut(run, end - t0);
        if (VEC) {
            if (c < c_end && t0 < p.L)
                *reinterpret_cast<Run<T, V> *>(static_cast<T *>(base) + to) = run;
        } else {
            T *at = static_cast<T *>(base) + to;
            const unsigned off = (unsigned)((uintptr_t)at & 15);
            const int o = (int)(off / sizeof(T));
            uint32_t s[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s[k] = __shfl_up_sync(~0u, run.w[k], 1);
                s[k + 4] = run.w[k];
            }
            Run<T, V> word = run;
            if (off) run_across(word, s, 16 - off);
            if (c >= c_end) return;
            const bool whole = (o == 0 || tx > 0) && t0 - o + V <= p.L;
            const bool next = tx + 1 < W && t0 - o + 2 * V <= p.L;
            if (whole) *reinterpret_cast<Run<T, V> *>(at - o) = word;
            if (whole && (next || o == 0)) return;
            using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
            constexpr int per = 4 / sizeof(T);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (t0 + j < p.L && !(j < V - o ? whole : next))
                    reinterpret_cast<Bits *>(at)[j] = (Bits)(run.w[j / per] >> (j % per * 16));
        }
    }
};

// ---------------------------------------------------------------- host side

// The tile's row (W threads of 16 bytes each), the cluster and the runs of a thread
// for C channels; the row becomes narrower down to a sector before a thread takes
// more.  Whole lines are for channels that one block has.  Returns W, or 0 where not
// even eight blocks hold a tile.
//
// What a block takes of a tile at a time decides how often the cluster is waited for
// (some 2 us) and whether the next tile can be on its way.  Aligned rows, forward: 48 KB,
// twice (8 x 2048 x 2048 bf16 89 us; 96 KB once 110 us).  Unaligned ones cost more
// instructions, which hide the copies: 98 KB once (6 x 515 x 785 f32 19 us, 48 KB twice
// 28 us; 3 x 1018 x 2862 f32 87 and 104 us).  Backward: 88 KB once (4 x 2048 x 2048 bf16
// 104 us; 44 KB twice, in rows of one sector, 125 us).
// extra: bytes that the backward pass holds for each run, 0 forward.
inline int norm_plan(NormParams &p, int dtype, int extra, bool vec) {
    const int V = 16 / (int)dtype_size(dtype);
    p.inputs = 0;
    for (int i = 0; i < kNormInputs; ++i)
        if (p.in[i]) p.slot[i] = p.inputs++;
    p.inv_C = 1.f / (float)p.C;
    const int sums = extra ? 7 : 4;
    for (int most : {extra ? 88 * 1024 : vec ? 48 * 1024 : 98 * 1024, kNormShared - 40 * 1024}) {
        for (int W = 8; W >= 2; W /= 2) {
            if (W > 2 && W * V >= 2 * (int64_t)p.L) continue;
            const int rows = kNormThreads / W, run = p.inputs * (vec ? kNormRow : kNormRow + rows * 16);
            const int R = most / (run + extra * kNormThreads);
            if (R < 1) continue;
            // the smallest cluster whose blocks hold their channels beside the sums and weights
            const int tile = W * V;
            int ranks = 1;
            for (; ranks <= (W == 8 ? 1 : kNormRanks); ranks *= 2) {
                p.per = (p.C + ranks - 1) / ranks;
                p.R = (p.per + rows - 1) / rows;
                if (p.R > R) continue;
                const int stage = p.R * run;
                const int rest = (kNormWarps + 2 * (W == 8 ? 1 : kNormRanks)) * sums * tile * 4 + 24 * tile +
                                 extra * p.R * kNormThreads + rows * p.R * 8;
                p.stages = 2 * stage + rest <= kNormShared / 2 || stage + rest > kNormShared / 2 ? 2 : 1;
                if (p.stages * stage + rest > kNormShared) p.stages = 1;
                p.shared = p.stages * stage + rest;
                if (p.shared <= kNormShared) break;
            }
            if (ranks > (W == 8 ? 1 : kNormRanks)) continue;
            p.ranks = ranks;
            p.tiles = (p.L - 1) / tile + 1;
            p.jobs = (int64_t)p.N * p.tiles;
            if (p.jobs > 0x7fff0000) continue;  // (a tile's number and a cluster's step stay within 32 bits)
            // (at most; norm_launch takes as many as run at once)
            const int64_t clusters = (int64_t)kSMs * (kNormShared / p.shared < 4 ? kNormShared / p.shared : 4) / ranks;
            p.clusters = (int)(p.jobs < clusters ? p.jobs : clusters);
            return W;
        }
    }
    return 0;
}

int norm_check(const spconv_residual_norm_args *a);
NormParams norm_params(const spconv_residual_norm_args *a);
bool norm_on_elements(const spconv_residual_norm_args *a, std::initializer_list<const void *> ps);
bool norm_on_words(std::initializer_list<const void *> ps);
int norm_launch(void (*fn)(NormParams), NormParams &p, void *stream);

}  // namespace seq
}  // namespace spconv
