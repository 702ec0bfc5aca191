// Internal: what the gated recurrence's forward pass (seq_gated.cu) and its
// gradients (seq_gated_backward.cu) share.
#pragma once

#include <cooperative_groups.h>

#include "seq_common.cuh"

namespace spconv {
namespace seq {

constexpr int kGatedThreads = 256;
constexpr int kGatedWarps = kGatedThreads / 32;
constexpr int kGatedRanks = 8;  // blocks of a cluster
constexpr int kGatedRun = 8;    // positions of a thread
constexpr int kGatedStream = 2 * kSMs;  // rows from which a block takes one after the other, backward

struct GatedParams {
    const void *x, *r, *i, *z, *dy;
    const float *A, *r_bias, *i_bias, *state, *dfinal;
    const int32_t *lengths, *slots;
    void *y, *dx, *dr, *di, *dz;
    float *final_state, *pool, *dA, *dr_bias, *di_bias, *dstate;
    float *carry;    // rows x rounds: the state in front of each round
    float *partial;  // rows x ranks x 3: a row's part of dA, dr_bias and di_bias
    int64_t x_sn, x_sc, r_sn, r_sc, i_sn, i_sc, z_sn, z_sc, dy_sn, dy_sc;
    int64_t rows;    // N * C
    int N, C, L, num_slots;
    int tx, log_tx;  // threads of a row, 2^log_tx
    int ranks;       // blocks of a row: a cluster
    int rounds;      // passes of a row's threads over its positions
};

// ---------------------------------------------------------------- rows

// A thread's row and its end; a row behind the last one has no positions.
struct GatedRow {
    int64_t row;
    int n, c, L, end;
    bool on;
};
static __device__ __forceinline__ GatedRow gated_row(const GatedParams &p, int64_t row) {
    GatedRow g;
    g.on = row < p.rows;
    g.row = g.on ? row : 0;
    if (p.rows >> 31) {
        g.n = (int)(g.row / p.C);
        g.c = (int)(g.row - (int64_t)g.n * p.C);
    } else {
        g.n = (int)((uint32_t)g.row / (uint32_t)p.C);
        g.c = (int)g.row - g.n * p.C;
    }
    g.L = g.on ? p.L : 0;
    g.end = min(g.L, p.lengths ? max(p.lengths[g.n], 0) : g.L);
    return g;
}

// Elements that an address lies behind a run's alignment.
template <typename T, int V>
static __device__ __forceinline__ int behind(const T *p) {
    constexpr int to = sizeof(Run<T, V>) < 16 ? sizeof(Run<T, V>) : 16;
    return (int)(((uintptr_t)p & (to - 1)) / sizeof(T));
}

// A row of one tensor: its runs are whole vectors where the row is as far
// behind an aligned address as the one that the runs are laid out by.
template <typename T, int V>
struct RowIn {
    const T *at;
    bool vec;
    __device__ __forceinline__ void set(const void *base, int64_t sn, int64_t sc, const GatedRow &g) {
        at = static_cast<const T *>(base) + g.n * sn + g.c * sc;
    }
    // A run inside the row.
    __device__ __forceinline__ void load(Run<T, V> &run, int t0) const {
        run = *reinterpret_cast<const Run<T, V> *>(at + t0);
    }
    // Positions t0.. of the run, zeros outside [0, end).
    __device__ __forceinline__ void load(Run<T, V> &run, int t0, int end) const {
        if (t0 >= 0) {
            load_run(run, at, t0, end, vec);
        } else {
            run.clear();
            constexpr int per = 4 / sizeof(T);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (t0 + j >= 0 && t0 + j < end) run.w[j / per] |= bits_of(at[t0 + j]) << (j % per * 16);
        }
    }
};
template <typename T, int V>
static __device__ __forceinline__ void store_part(const Run<T, V> &run, T *row, int t0, int L, bool vec) {
    if (t0 >= 0) {
        store_run(run, row, t0, L, vec);
    } else {
        using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
        constexpr int per = 4 / sizeof(T);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (t0 + j >= 0 && t0 + j < L)
                reinterpret_cast<Bits *>(row)[t0 + j] = (Bits)(run.w[j / per] >> (j % per * 16));
    }
}

// ---------------------------------------------------------------- the recurrence

// A decay 2^w, w <= 0, with its digits at both ends: next to one as 1 + e, e = 2^w
// - 1 from the degree-5 interpolant of (2^w - 1) / w at the Chebyshev nodes of
// [-0.75, 0] (relative error 2e-9), else as e itself.  A state's decay then costs
// one rounding, and 1 - a^2 keeps its digits.
struct Decay {
    static constexpr float kNear = -0.75f;
    float e;
    bool near;
    __device__ __forceinline__ explicit Decay(float w) {
        near = w > kNear;
        float q = fmaf(w, 1.23557082e-4f, 1.30864489e-3f);
        q = fmaf(w, q, 9.60869808e-3f);
        q = fmaf(w, q, 5.55024669e-2f);
        q = fmaf(w, q, 0.240226403f);
        q = fmaf(w, q, 0.693147182f);
        e = near ? w * q : ex2(w);
    }
    __device__ __forceinline__ Decay() {}
    __device__ __forceinline__ float a() const { return near ? 1.f + e : e; }
    __device__ __forceinline__ float of(float h) const { return fmaf(e, h, near ? h : 0.f); }
    __device__ __forceinline__ float rest() const;  // sqrt(1 - a^2)
};
static __device__ __forceinline__ float root(float v) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}

__device__ __forceinline__ float Decay::rest() const { return root(fmaf(-e, e, near ? -2.f * e : 1.f)); }

// 1 / sqrt(v), of a number from 2^-126 up; finite (and so of no consequence for a
// product with v) below, NaN for a negative one.
static __device__ __forceinline__ float inverse_root(float v) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(v, 1.17549435e-38f)));
    return v >= 0.f ? y : __int_as_float(0x7fffffff);
}

// What a stretch of positions does to a state: h -> 2^w h + b.  Decays are
// joined by their exponents: a product of decays next to one would carry each
// one's rounding, thousands of positions over.
struct Link {
    float w, b;
};
static __device__ __forceinline__ float grown(float w) { return decay(1.f, w); }
static __device__ __forceinline__ float after(float h, Link l) { return fmaf(grown(l.w), h, l.b); }

// ---------------------------------------------------------------- two positions at a time

// Sigmoids of (v + bias), from v, -log2(e) and -log2(e) bias.
static __device__ __forceinline__ f32x2 sigmoid2(f32x2 v, f32x2 unit, f32x2 bias) {
    const float2 e = unpack2(add2(ex2_2(fma2(v, unit, bias)), pack2(1.f, 1.f)));
    return pack2(rcp(e.x), rcp(e.y));
}
// a = 2^w for w in [-0.75, 0], 1 - a^2 and the inverse of its root (for 0 some finite
// number: of no consequence times the square, to be replaced where it stands alone).
// 1 - a comes from Decay's polynomial, so that 1 - a^2 keeps its digits next to a
// decay of one; a itself is rounded once.
struct Decay2 {
    f32x2 a, square, inverse;
    __device__ __forceinline__ explicit Decay2(f32x2 w) {
        f32x2 q = fma2(w, pack2(-1.23557082e-4f, -1.23557082e-4f), pack2(-1.30864489e-3f, -1.30864489e-3f));
        q = fma2(w, q, pack2(-9.60869808e-3f, -9.60869808e-3f));
        q = fma2(w, q, pack2(-5.55024669e-2f, -5.55024669e-2f));
        q = fma2(w, q, pack2(-0.240226403f, -0.240226403f));
        q = fma2(w, q, pack2(-0.693147182f, -0.693147182f));
        const f32x2 less = mul2(w, pack2(-1.f, -1.f)), lost = mul2(w, q);  // 1 - a
        a = fma2(less, q, pack2(1.f, 1.f));
        square = mul2(lost, add2(a, pack2(1.f, 1.f)));
        const float2 s = unpack2(square);
        inverse = pack2(inverse_root(s.x), inverse_root(s.y));
    }
};

// Threads per row, blocks per row and rounds, for runs of V positions.
// Forward, what a row's setup and the joining of warps cost counts for more than
// the number of blocks: a row gets a warp, and more (up to a cluster) only as long as
// the rows leave less than twelve warps to an SM.  (8 x 4096 rows of 2048 in bf16:
// 230 us with a block for each, 133 us with a warp.  1 x 1000 rows of 8191 in float32:
// 34 us with twelve warps to an SM, 37 with twenty.)  Backward (`whole`), a row gets a
// block, and few rows clusters as far as they take a row in one round, since with
// more rounds a third of what it reads is read again.  (160 rows of 8192 in bf16: 17 us in
// clusters, 20 in rounds; 249 of 17,042 in float32, two rounds of a cluster: 138 and 70 us;
// 504 of 27,506 in f16 without gates: 179 and 91 us, with both 132 in rounds.)
inline void gated_plan(GatedParams &p, int V, bool aligned, bool whole) {
    const int64_t runs = ((int64_t)p.L + (aligned ? 0 : V - 1) + V - 1) / V;
    p.log_tx = 2;
    while ((1 << p.log_tx) < runs && (1 << p.log_tx) < kGatedThreads &&
           (whole || p.log_tx < 5 || p.rows << p.log_tx < 12 * 32 * kSMs))
        ++p.log_tx;
    p.tx = 1 << p.log_tx;
    p.ranks = 1;
    // backward: clusters for rows that one takes in a round, or that are too few by far
    const bool split = p.rows < (runs <= kGatedThreads * kGatedRanks ? kGatedStream : kSMs / 2);
    while (p.tx == kGatedThreads && p.ranks < kGatedRanks && (int64_t)p.tx * p.ranks < runs &&
           (whole ? split : p.rows * p.ranks * kGatedWarps < 12 * kSMs))
        p.ranks *= 2;
    p.rounds = (int)((runs + (int64_t)p.tx * p.ranks - 1) / ((int64_t)p.tx * p.ranks));
}

// Blocks of all rows, or 0 where they are more than a grid takes.
inline unsigned gated_blocks(const GatedParams &p) {
    const int64_t ty = kGatedThreads / p.tx, blocks = (p.rows + ty - 1) / ty;
    return blocks > 0x7fffffff / p.ranks ? 0 : (unsigned)(blocks * p.ranks);
}

int gated_check(const spconv_gated_scan_args *a);
GatedParams gated_params(const spconv_gated_scan_args *a);
// Every row of the inputs starts on 16 bytes.
bool gated_rows_aligned(const spconv_gated_scan_args *a);
int gated_launch(void (*fn)(GatedParams), const GatedParams &p, void *stream);
// The states in front of each round (p.carry), by the forward kernel.
int gated_carries(const GatedParams &p, int dtype, void *stream);

}  // namespace seq
}  // namespace spconv
