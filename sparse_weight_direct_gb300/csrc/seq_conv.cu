// The short causal convolution along the positions of a channels-first
// sequence, one filter of K = 1..4 taps per channel: forward, backward and the
// single-token step.
//
//   p = (state | x),  v_t = b + sum_k w_k p_(t+k),  y_t = silu(v_t) or v_t
//
// With g_t = dy_t * silu'(v_t) inside the sequence and 0 behind it, the
// gradients are dp_j = sum_k w_k g_(j-k) (dx and dstate are its two parts, and
// a final state's gradient adds to its last K-1 entries), dw_k = sum g_t
// p_(t+k) and db = sum g_t.
//
// Bound: a few FMAs per element against one read and one write, so the memory
// bandwidth bounds it.
#include "seq_common.cuh"

namespace spconv {
namespace seq {
namespace {

constexpr int kThreads = 256;

struct ConvParams {
    const void *x, *state, *dy, *dfinal;
    const float *weight, *bias;
    const int32_t *lengths, *slots;
    void *y, *final_state, *pool, *dx, *dstate;
    float *dweight, *dbias, *partial;
    int64_t x_sn, x_sc, dy_sn, dy_sc;
    int N, C, L, silu, num_slots;
    int runs;    // runs of kVec positions in a row
    int tx;      // threads along a row (power of two)
    int ty;      // rows of a block
    int tiles;   // blocks along a row
    int splits;  // backward: blocks that share a channel
    int vec_x, vec_y, vec_dy;
};

static __device__ __forceinline__ int length_of(const int32_t *lengths, int n, int L) {
    return lengths ? min(max(lengths[n], 0), L) : L;
}

// s[0 .. K-2] = the K-1 entries of p before position t0, oldest first: the end
// of the run to the left (a neighbour has read it: it comes from L1), or the
// state.
template <typename T, int K>
static __device__ __forceinline__ void load_before(float *s, const T *row, const T *state_row,
                                                   int t0, int end, bool vec) {
    if (K == 1) return;
    if (t0 > 0) {
        if (vec) {
            Run<T> left;
            load_run(left, row, t0 - kVec, end, true);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) s[j] = left[kVec - (K - 1) + j];
        } else {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) s[j] = to_f32(row[t0 - (K - 1) + j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) s[j] = state_row ? to_f32(state_row[j]) : 0.f;
    }
}

// s[0 .. K-2] = the K-1 entries of a row from t0, zeros from `end`.
template <typename T, int K>
static __device__ __forceinline__ void load_behind(float *s, const T *row, int t0, int end, bool vec) {
    if (K == 1) return;
    if (vec && t0 + kVec <= end) {
        Run<T> right;
        load_run(right, row, t0, end, true);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) s[j] = right[j];
    } else {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) s[j] = t0 + j < end ? to_f32(row[t0 + j]) : 0.f;
    }
}

// Forward: a thread computes kVec consecutive outputs of one channel in one
// sequence after the other, the next one's inputs on their way; blocks x go
// over the tiles of a row and the channels, y over the sequences.  Its
// instructions are as near a bound as its bytes: a thread per run spent two
// thirds of them on its place and its weights (82 us on 8 x 4096 x 2048 in
// bf16), one loop for every case many on the cases (65 us).  So whole, aligned
// runs of full sequences have a loop of their own (55 us, six blocks per SM, for
// which 16-bit types with 4 taps spill 40 to 52 bytes).
template <typename T, int K, bool SILU>
static __device__ __forceinline__ void conv_whole_runs(const ConvParams &p, const float (&w)[K],
                                                       float b, int c, int t0) {
    const int64_t x_step = gridDim.y * p.x_sn, row_step = (int64_t)gridDim.y * p.C;
    const T *x = static_cast<const T *>(p.x) + blockIdx.y * p.x_sn + c * p.x_sc + t0;
    const int64_t row = (int64_t)blockIdx.y * p.C + c;
    T *y = static_cast<T *>(p.y) + row * p.L + t0;
    const T *state = p.state ? static_cast<const T *>(p.state) + row * (K - 1) : nullptr;
    const int64_t y_step = row_step * p.L;
    Run<T> in, left;
    auto fetch = [&](int n) {
        if (n >= p.N) return;
        load_run(in, x, 0, kVec, true);
        if (K > 1 && t0 > 0) {
            load_run(left, x - kVec, 0, kVec, true);
        } else if (K > 1) {
            float f[kVec] = {};
#pragma unroll
            for (int j = 0; j < K - 1; ++j) f[kVec - (K - 1) + j] = state ? to_f32(state[j]) : 0.f;
            left.put(f);
        }
        x += x_step;
        if (state) state += row_step * (K - 1);
    };
    fetch(blockIdx.y);
    for (int n = blockIdx.y; n < p.N; n += gridDim.y, y += y_step) {
        float s[kVec + K - 1], o[kVec];
#pragma unroll
        for (int i = 0; i < K - 1; ++i) s[i] = left[kVec - (K - 1) + i];
#pragma unroll
        for (int i = 0; i < kVec; ++i) s[K - 1 + i] = in[i];
        fetch(n + gridDim.y);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            o[i] = b;
#pragma unroll
            for (int k = 0; k < K; ++k) o[i] = fmaf(w[k], s[i + k], o[i]);
            if (SILU) o[i] = silu(o[i]);
        }
        Run<T> out;
        out.put(o);
        *reinterpret_cast<Run<T> *>(y) = out;
    }
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 6 : 4) conv_kernel(const ConvParams p) {
    const unsigned cb = blockIdx.x / (unsigned)p.tiles;
    const int tile = (int)(blockIdx.x - cb * p.tiles);
    const int lane = threadIdx.x & (p.tx - 1);
    const int64_t c64 = (int64_t)cb * p.ty + threadIdx.x / p.tx;
    if (c64 >= p.C) return;
    const int c = (int)c64, run = tile * p.tx + lane, t0 = run * kVec;
    float w[K];
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = p.weight[(int64_t)c * K + k];
    const float b = p.bias ? p.bias[c] : 0.f;
    if (p.vec_x && p.vec_y && !p.lengths && t0 + kVec <= p.L) {
        if (p.silu)
            conv_whole_runs<T, K, true>(p, w, b, c, t0);
        else
            conv_whole_runs<T, K, false>(p, w, b, c, t0);
        if (K > 1 && p.final_state && run == 0) {  // (whole runs: L >= K - 1)
            for (int n = blockIdx.y; n < p.N; n += gridDim.y) {
                const T *last = static_cast<const T *>(p.x) + n * p.x_sn + c * p.x_sc + p.L - (K - 1);
                T *fin = static_cast<T *>(p.final_state) + ((int64_t)n * p.C + c) * (K - 1);
#pragma unroll
                for (int j = 0; j < K - 1; ++j) fin[j] = last[j];
            }
        }
        return;
    }
    const int64_t x_step = gridDim.y * p.x_sn, row_step = (int64_t)gridDim.y * p.C;
    const T *x = static_cast<const T *>(p.x) + blockIdx.y * p.x_sn + c * p.x_sc;
    int64_t row = (int64_t)blockIdx.y * p.C + c;
    struct Inputs {
        Run<T> in;
        float left[K > 1 ? K - 1 : 1];
        int len;
    } next;
    auto fetch = [&](int n) {
        if (n >= p.N) return;
        next.len = length_of(p.lengths, n, p.L);
        if (t0 < next.len) {
            load_run(next.in, x, t0, next.len, p.vec_x);
            load_before<T, K>(next.left, x,
                              p.state ? static_cast<const T *>(p.state) + row * (K - 1) : nullptr,
                              t0, next.len, p.vec_x);
        }
    };
    fetch(blockIdx.y);
    for (int n = blockIdx.y; n < p.N; n += gridDim.y) {
        const Inputs now = next;
        const T *xrow = x;
        const int64_t rowi = row;
        x += x_step;
        row += row_step;
        fetch(n + gridDim.y);
        if (run < p.runs) {
            Run<T> out;
            out.clear();
            if (t0 < now.len) {
                float s[kVec + K - 1], o[kVec];
#pragma unroll
                for (int i = 0; i < K - 1; ++i) s[i] = now.left[i];
#pragma unroll
                for (int i = 0; i < kVec; ++i) s[K - 1 + i] = now.in[i];
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    o[i] = b;
#pragma unroll
                    for (int k = 0; k < K; ++k) o[i] = fmaf(w[k], s[i + k], o[i]);
                }
                if (p.silu) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) o[i] = silu(o[i]);
                }
                if (t0 + kVec > now.len) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) o[i] = t0 + i < now.len ? o[i] : 0.f;
                }
                out.put(o);
            }
            store_run(out, static_cast<T *>(p.y) + rowi * p.L, t0, p.L, p.vec_y);
        }
        if (K > 1 && p.final_state && run == 0) {
            const T *st = p.state ? static_cast<const T *>(p.state) + rowi * (K - 1) : nullptr;
            T *fin = static_cast<T *>(p.final_state) + rowi * (K - 1);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                const int t = now.len - (K - 1) + j;
                fin[j] = t >= 0 ? xrow[t] : st ? st[t + K - 1] : from_f32<T>(0.f);
            }
        }
    }
}

// The gradients' loop of a thread whose items are the same whole, aligned run of
// one full sequence after the other: what is special about the first and the
// last run is known before it.
template <typename T, int K, bool SILU>
static __device__ __forceinline__ void back_whole_runs(const ConvParams &p, const float (&w)[K],
                                                       float b, int c, int t0, int n0, int dn,
                                                       float (&sum)[K + 1]) {
    constexpr int kG = kVec + K - 1;
    const bool is_first = t0 == 0, is_last = t0 + kVec == p.L;
    int64_t row = (int64_t)n0 * p.C + c;
    const int64_t row_step = (int64_t)dn * p.C, x_step = dn * p.x_sn, dy_step = dn * p.dy_sn;
    const T *x = static_cast<const T *>(p.x) + n0 * p.x_sn + c * p.x_sc + t0;
    const T *dy = static_cast<const T *>(p.dy) + n0 * p.dy_sn + c * p.dy_sc + t0;
    T *dx = static_cast<T *>(p.dx) + row * p.L + t0;
    const int64_t dx_step = row_step * p.L;
    Run<T> left, right, gright;
    left.clear();
    right.clear();
    gright.clear();
    for (int64_t n = n0; n < p.N; n += dn, x += x_step, dy += dy_step, dx += dx_step, row += row_step) {
        Run<T> in, gin;
        load_run(in, x, 0, kVec, true);
        load_run(gin, dy, 0, kVec, true);
        if (K > 1 && !is_first) load_run(left, x - kVec, 0, kVec, true);
        if (K > 1 && is_first && p.state) {
            float f[kVec] = {};
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
                f[kVec - (K - 1) + j] = to_f32(static_cast<const T *>(p.state)[row * (K - 1) + j]);
            left.put(f);
        }
        if (K > 1 && !is_last) {
            load_run(right, x + kVec, 0, kVec, true);
            load_run(gright, dy + kVec, 0, kVec, true);
        }
        float s[kG + K - 1], g[kG], o[kVec];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            s[j] = left[kVec - (K - 1) + j];
            s[K - 1 + kVec + j] = right[j];
            g[kVec + j] = gright[j];
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            s[K - 1 + j] = in[j];
            g[j] = gin[j];
        }
        if (SILU) {
#pragma unroll
            for (int j = 0; j < kG; ++j) {
                float v = b;
#pragma unroll
                for (int k = 0; k < K; ++k) v = fmaf(w[k], s[j + k], v);
                g[j] *= silu_grad(v);
            }
            if (K > 1 && is_last) {
#pragma unroll
                for (int j = kVec; j < kG; ++j) g[j] = 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            sum[K] += g[j];
            o[j] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                sum[k] = fmaf(g[j], s[j + k], sum[k]);
                o[j] = fmaf(w[k], g[j + K - 1 - k], o[j]);
            }
        }
        if (K > 1 && is_last && p.dfinal) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
                o[kVec - (K - 1) + j] += to_f32(static_cast<const T *>(p.dfinal)[row * (K - 1) + j]);
        }
        Run<T> out;
        out.put(o);
        *reinterpret_cast<Run<T> *>(dx) = out;
        if (K > 1 && is_first && p.dstate) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {  // (a whole run: the sequence is longer than the state)
                float d = 0.f;
#pragma unroll
                for (int k = 0; k <= j; ++k) d = fmaf(w[k], g[j - k], d);
                static_cast<T *>(p.dstate)[row * (K - 1) + j] = from_f32<T>(d);
            }
        }
    }
}

// Backward: a block takes every splits-th group of kThreads runs of one
// channel over all sequences; a thread holds the inputs around its run, forms
// g for its kVec positions and the K-1 behind them (which its right neighbour
// forms too: K-1 in kVec twice is cheaper than an exchange), writes dx and
// adds to its sums for dw and db.  The sums are joined in a fixed order.
// Bound by its instructions: 4 x 2048 x 2048 in bf16 take 28 us, 38 without the
// loop of its own for whole runs (60 instructions an element).  That loop is taken
// where a thread keeps its run from one sequence to the next, so not at every
// length: 2 x 2048 x 4096, the same bytes, take 40 us.
template <typename T, int K>
__global__ void __launch_bounds__(kThreads) conv_backward_kernel(const ConvParams p) {
    const int c = blockIdx.x / p.splits, split = blockIdx.x - c * p.splits;
    float w[K];
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = p.weight[(int64_t)c * K + k];
    const float b = p.bias ? p.bias[c] : 0.f;
    float sum[K + 1];
#pragma unroll
    for (int k = 0; k <= K; ++k) sum[k] = 0.f;
    // (sequence, run) of the thread's items, advanced without dividing
    const int stride = p.splits * kThreads, dn = stride / max(p.runs, 1), dr = stride - dn * p.runs;
    int64_t n = 0;
    int run = 0;
    if (p.runs > 0) {
        const int first = split * kThreads + threadIdx.x;
        n = first / p.runs;
        run = first - (int)n * p.runs;
    }
    if (dr == 0 && p.vec_x && p.vec_dy && p.vec_y && !p.lengths && p.L % kVec == 0 && p.runs > 0) {
        if (n < p.N) {
            if (p.silu)
                back_whole_runs<T, K, true>(p, w, b, c, run * kVec, (int)n, dn, sum);
            else
                back_whole_runs<T, K, false>(p, w, b, c, run * kVec, (int)n, dn, sum);
        }
        n = p.N;
    }
    int64_t rowi = n * p.C + c;
    const T *row = static_cast<const T *>(p.x) + n * p.x_sn + c * p.x_sc;
    const T *drow = static_cast<const T *>(p.dy) + n * p.dy_sn + c * p.dy_sc;
    const int64_t x_step = dn * p.x_sn, dy_step = dn * p.dy_sn, row_step = (int64_t)dn * p.C;
    while (n < p.N && p.runs > 0) {
        const int t0 = run * kVec;
        const int len = length_of(p.lengths, (int)n, p.L);
        const T *st = p.state ? static_cast<const T *>(p.state) + rowi * (K - 1) : nullptr;
        const T *df = p.dfinal ? static_cast<const T *>(p.dfinal) + rowi * (K - 1) : nullptr;
        constexpr int kG = kVec + K - 1;
        float s[kG + K - 1], g[kG];
        if (t0 < len) {
            Run<T> in, gin;
            load_run(in, row, t0, len, p.vec_x);
            load_run(gin, drow, t0, len, p.vec_dy);
            load_before<T, K>(s, row, st, t0, len, p.vec_x);
            load_behind<T, K>(s + K - 1 + kVec, row, t0 + kVec, len, p.vec_x);
            load_behind<T, K>(g + kVec, drow, t0 + kVec, len, p.vec_dy);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                s[K - 1 + j] = in[j];
                g[j] = gin[j];
            }
            if (p.silu) {
#pragma unroll
                for (int j = 0; j < kG; ++j) {
                    float v = b;
#pragma unroll
                    for (int k = 0; k < K; ++k) v = fmaf(w[k], s[j + k], v);
                    g[j] *= silu_grad(v);
                }
                if (t0 + kG > len) {
#pragma unroll
                    for (int j = 0; j < kG; ++j) g[j] = t0 + j < len ? g[j] : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                sum[K] += g[j];
#pragma unroll
                for (int k = 0; k < K; ++k) sum[k] = fmaf(g[j], s[j + k], sum[k]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kG; ++j) g[j] = 0.f;
        }
        float o[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            o[j] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) o[j] = fmaf(w[k], g[j + K - 1 - k], o[j]);
        }
        if (t0 + kG > len) {
            // the sequence's end: what its final state's gradient adds
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const int t = t0 + j, back = t - (len - (K - 1));
                if (K > 1 && df && t < len && back >= 0) o[j] += to_f32(df[back]);
                o[j] = t < len ? o[j] : 0.f;
            }
        }
        Run<T> out;
        out.put(o);
        store_run(out, static_cast<T *>(p.dx) + rowi * p.L, t0, p.L, p.vec_y);
        if (K > 1 && p.dstate && run == 0) {
            T *ds = static_cast<T *>(p.dstate) + rowi * (K - 1);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {  // p_j: position j - (K-1)
                float d = 0.f;
#pragma unroll
                for (int k = 0; k <= j; ++k) d = fmaf(w[k], g[j - k], d);
                if (df && j >= len) d += to_f32(df[j - len]);
                ds[j] = from_f32<T>(d);
            }
        }
        n += dn;
        row += x_step;
        drow += dy_step;
        rowi += row_step;
        run += dr;
        if (run >= p.runs) {
            run -= p.runs;
            ++n;
            row += p.x_sn;
            drow += p.dy_sn;
            rowi += p.C;
        }
    }
    __shared__ float part[kThreads / 32][K + 1];
#pragma unroll
    for (int k = 0; k <= K; ++k) {
#pragma unroll
        for (int o = 16; o; o >>= 1) sum[k] += __shfl_xor_sync(~0u, sum[k], o);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][k] = sum[k];
    }
    __syncthreads();
    if (threadIdx.x <= K) {
        float total = 0.f;
        for (int i = 0; i < kThreads / 32; ++i) total += part[i][threadIdx.x];
        const int k = threadIdx.x;
        if (p.splits > 1)
            p.partial[((int64_t)split * p.C + c) * (K + 1) + k] = total;
        else if (k < K)
            p.dweight[(int64_t)c * K + k] = total;
        else if (p.dbias)
            p.dbias[c] = total;
    }
}

// The blocks' sums of one channel, in their order.
template <int K>
__global__ void __launch_bounds__(kThreads) conv_join_kernel(const ConvParams p) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (int64_t)p.C * (K + 1)) return;
    float total = 0.f;
    for (int s = 0; s < p.splits; ++s) total += p.partial[(int64_t)s * p.C * (K + 1) + i];
    const int64_t c = i / (K + 1);
    const int k = (int)(i - c * (K + 1));
    if (k < K)
        p.dweight[c * K + k] = total;
    else if (p.dbias)
        p.dbias[c] = total;
}

// dstate where L = 0: no run exists, the final state is the initial one.
template <typename T>
__global__ void __launch_bounds__(kThreads) copy_state_kernel(const void *from, void *to,
                                                              int64_t count) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= count) return;
    static_cast<T *>(to)[i] = from ? static_cast<const T *>(from)[i] : from_f32<T>(0.f);
}

// Step: a thread per request and channel.
template <typename T, int K>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvParams p) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int n = blockIdx.y;
    if (c >= p.C) return;
    const int64_t i = (int64_t)n * p.C + c;
    const int slot = p.slots ? p.slots[n] : n;
    T *y = static_cast<T *>(p.y) + i;
    if (slot < 0 || slot >= p.num_slots) {
        *y = from_f32<T>(0.f);
        return;
    }
    const T x = static_cast<const T *>(p.x)[n * p.x_sn + c];
    T s[K];
    T *st = static_cast<T *>(p.pool) + ((int64_t)slot * p.C + c) * (K - 1);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) s[k] = st[k];
    s[K - 1] = x;
    float v = p.bias ? p.bias[c] : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) v = fmaf(p.weight[c * K + k], to_f32(s[k]), v);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) st[k] = s[k + 1];
    *y = from_f32<T>(p.silu ? silu(v) : v);
}

// ---------------------------------------------------------------- host side

template <typename F>
int by_taps(int K, F f) {
    switch (K) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 3: return f(std::integral_constant<int, 3>{});
        case 4: return f(std::integral_constant<int, 4>{});
    }
    return SPCONV_ERR_UNSUPPORTED;
}

int check_sizes(const spconv_short_conv_args *a) {
    if (!a || a->N < 0 || a->C < 0 || a->L < 0 || a->K < 1) return SPCONV_ERR_INVALID_ARG;
    if (a->dtype < SPCONV_F32 || a->dtype > SPCONV_F16 || (a->silu & ~1))
        return SPCONV_ERR_INVALID_ARG;
    if (a->K > 4 || a->L > kMaxLength || a->N > kMaxLength || a->C > kMaxLength)
        return SPCONV_ERR_UNSUPPORTED;
    if (!stride_ok(a->x_stride_n) || !stride_ok(a->x_stride_c) || !stride_ok(a->dy_stride_n) ||
        !stride_ok(a->dy_stride_c))
        return SPCONV_ERR_INVALID_ARG;
    return SPCONV_OK;
}

ConvParams params_of(const spconv_short_conv_args *a) {
    const size_t e = dtype_size(a->dtype);
    ConvParams p{};
    p.x = a->x; p.state = a->state; p.dy = a->dy; p.dfinal = a->dfinal_state;
    p.weight = a->weight; p.bias = a->bias;
    p.lengths = a->lengths; p.slots = a->slots;
    p.y = a->y; p.final_state = a->final_state; p.pool = a->pool; p.dx = a->dx;
    p.dstate = a->dstate; p.dweight = a->dweight; p.dbias = a->dbias;
    p.partial = static_cast<float *>(a->workspace);
    p.x_sn = a->x_stride_n; p.x_sc = a->x_stride_c;
    p.dy_sn = a->dy_stride_n; p.dy_sc = a->dy_stride_c;
    p.N = a->N; p.C = a->C; p.L = a->L; p.silu = a->silu; p.num_slots = a->num_slots;
    p.runs = (a->L + kVec - 1) / kVec;
    p.vec_x = rows_aligned(a->x, a->x_stride_n, a->x_stride_c, e);
    p.vec_dy = rows_aligned(a->dy, a->dy_stride_n, a->dy_stride_c, e);
    return p;
}

// Blocks that share a channel's runs in the backward pass: enough to fill the
// GPU with 8 blocks per SM, none with less than one run per thread.
int backward_splits(const spconv_short_conv_args *a) {
    const int64_t items = (int64_t)a->N * ((a->L + kVec - 1) / kVec);
    const int64_t most = (items + kThreads - 1) / kThreads;
    const int64_t want = (8 * kSMs + a->C - 1) / a->C;
    const int64_t s = want < most ? want : most;
    return s < 1 ? 1 : (int)s;
}

bool on_elements(const spconv_short_conv_args *a, std::initializer_list<const void *> ps) {
    for (const void *q : ps)
        if (q && !aligned(q, dtype_size(a->dtype))) return false;
    return true;
}

Span weights_of(const spconv_short_conv_args *a) { return {a->weight, (int64_t)a->C * a->K * 4}; }
Span bias_of(const spconv_short_conv_args *a) { return {a->bias, a->C * 4LL}; }

bool on_words(std::initializer_list<const void *> ps) {
    for (const void *q : ps)
        if (q && !aligned(q, 4)) return false;
    return true;
}

}  // namespace
}  // namespace seq
}  // namespace spconv

using namespace spconv::seq;

SPCONV_API int spconv_short_conv(const spconv_short_conv_args *a, void *stream) {
    int st = check_sizes(a);
    if (st) return st;
    const int64_t rows = (int64_t)a->N * a->C;
    if (rows == 0) return SPCONV_OK;
    const size_t e = dtype_size(a->dtype);
    if (!a->weight || (a->L > 0 && (!a->x || !a->y))) return SPCONV_ERR_INVALID_ARG;
    if (!on_elements(a, {a->x, a->state, a->y, a->final_state}) ||
        !on_words({a->weight, a->bias, a->lengths}))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t xb = extent(a->N, a->C, a->L, a->x_stride_n, a->x_stride_c, e);
    const int64_t yb = rows * a->L * e, sb = rows * (a->K - 1) * e;
    if (!apart({{a->y, yb}, {a->final_state, sb}},
               {{a->x, xb}, {a->state, sb}, weights_of(a), bias_of(a), {a->lengths, a->N * 4LL}}))
        return SPCONV_ERR_INVALID_ARG;
    ConvParams p = params_of(a);
    p.vec_y = rows_aligned(a->y, 0, a->L, e);
    const int runs = p.runs > 0 ? p.runs : 1;
    p.tx = 1;
    while (p.tx < runs && p.tx < kThreads) p.tx *= 2;
    p.ty = kThreads / p.tx;
    p.tiles = (runs + p.tx - 1) / p.tx;
    const int64_t blocks = ((int64_t)a->C + p.ty - 1) / p.ty * p.tiles;
    if (blocks > 0x7fffffff) return SPCONV_ERR_UNSUPPORTED;
    // sequences side by side as far as 16 blocks per SM need them
    int64_t side = (16 * kSMs + blocks - 1) / blocks;
    if (side > a->N) side = a->N;
    if (side > 65535) side = 65535;
    const dim3 grid((unsigned)blocks, (unsigned)side);
    return by_dtype(a->dtype, [&](auto t) {
        return by_taps(a->K, [&](auto k) {
            conv_kernel<decltype(t), decltype(k)::value>
                <<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
            return launch_status();
        });
    });
}

SPCONV_API int64_t spconv_short_conv_backward_workspace(const spconv_short_conv_args *a) {
    if (check_sizes(a) || a->C == 0) return 0;
    const int s = backward_splits(a);
    return s > 1 ? (int64_t)s * a->C * (a->K + 1) * 4 : 0;
}

SPCONV_API int spconv_short_conv_backward(const spconv_short_conv_args *a, void *stream) {
    int st = check_sizes(a);
    if (st) return st;
    if (a->C == 0) return SPCONV_OK;
    const int64_t rows = (int64_t)a->N * a->C;
    const size_t e = dtype_size(a->dtype);
    if (!a->weight || !a->dweight || (rows * a->L > 0 && (!a->x || !a->dy || !a->dx)))
        return SPCONV_ERR_INVALID_ARG;
    if (!on_elements(a, {a->x, a->state, a->dy, a->dfinal_state, a->dx, a->dstate}) ||
        !on_words({a->weight, a->bias, a->lengths, a->dweight, a->dbias}))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t need = spconv_short_conv_backward_workspace(a);
    if (need && (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < need))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t xb = extent(a->N, a->C, a->L, a->x_stride_n, a->x_stride_c, e);
    const int64_t db = extent(a->N, a->C, a->L, a->dy_stride_n, a->dy_stride_c, e);
    const int64_t yb = rows * a->L * e, sb = rows * (a->K - 1) * e;
    if (!apart({{a->dx, yb}, {a->dstate, sb}, {a->dweight, weights_of(a).bytes},
                {a->dbias, bias_of(a).bytes}, {a->workspace, need}},
               {{a->x, xb}, {a->dy, db}, {a->state, sb}, {a->dfinal_state, sb}, weights_of(a),
                bias_of(a), {a->lengths, a->N * 4LL}}))
        return SPCONV_ERR_INVALID_ARG;
    ConvParams p = params_of(a);
    p.vec_y = rows_aligned(a->dx, 0, a->L, e);
    p.splits = backward_splits(a);
    if ((int64_t)p.splits * a->C > 0x7fffffff) return SPCONV_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_dtype(a->dtype, [&](auto t) {
        return by_taps(a->K, [&](auto k) {
            constexpr int K = decltype(k)::value;
            using T = decltype(t);
            const int64_t states = rows * (K - 1);
            if (a->L == 0 && a->dstate && states > 0)
                copy_state_kernel<T><<<(unsigned)((states + kThreads - 1) / kThreads), kThreads, 0,
                                       s>>>(a->dfinal_state, a->dstate, states);
            conv_backward_kernel<T, K><<<(unsigned)(p.splits * p.C), kThreads, 0, s>>>(p);
            if (p.splits > 1) {
                const int64_t count = (int64_t)p.C * (K + 1);
                conv_join_kernel<K><<<(unsigned)((count + kThreads - 1) / kThreads), kThreads, 0,
                                      s>>>(p);
            }
            return launch_status();
        });
    });
}

SPCONV_API int spconv_short_conv_step(const spconv_short_conv_args *a, void *stream) {
    int st = check_sizes(a);
    if (st) return st;
    if (a->num_slots < 0 || (!a->slots && a->num_slots != a->N) || a->x_stride_c != 1)
        return SPCONV_ERR_INVALID_ARG;
    if (a->N > 65535) return SPCONV_ERR_UNSUPPORTED;  // requests go along grid y
    const int64_t rows = (int64_t)a->N * a->C;
    if (rows == 0) return SPCONV_OK;
    const size_t e = dtype_size(a->dtype);
    if (!a->x || !a->weight || !a->y || (a->K > 1 && a->num_slots > 0 && !a->pool))
        return SPCONV_ERR_INVALID_ARG;
    if (!on_elements(a, {a->x, a->pool, a->y}) || !on_words({a->weight, a->bias, a->slots}))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t xb = extent(a->N, a->C, 1, a->x_stride_n, 1, e), yb = rows * e;
    const int64_t sb = (int64_t)a->num_slots * a->C * (a->K - 1) * e;
    if (!apart({{a->y, yb}, {a->pool, sb}},
               {{a->x, xb}, weights_of(a), bias_of(a), {a->slots, a->N * 4LL}}))
        return SPCONV_ERR_INVALID_ARG;
    const ConvParams p = params_of(a);
    const dim3 grid((unsigned)((a->C - 1) / kThreads + 1), a->N);
    return by_dtype(a->dtype, [&](auto t) {
        return by_taps(a->K, [&](auto k) {
            conv_step_kernel<decltype(t), decltype(k)::value>
                <<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
            return launch_status();
        });
    });
}
