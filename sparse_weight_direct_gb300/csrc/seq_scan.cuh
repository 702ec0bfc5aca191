// Internal: parameters and staging that the selective scan's forward
// (seq_scan.cu) and backward (seq_scan_backward.cu) kernels share.
//
// A block owns 32 channels of one group of one sequence; four lanes of a warp
// share a channel and hold SPT = ceil(S / 4) of its states each in registers.
// Positions go in tiles of 4 * VE: lane j of a channel's four loads the
// positions VE*j .. VE*j + VE-1 of its rows (16 bytes for 16-bit types with VE = 8),
// so a warp reads eight rows side by side, and turns them into step sizes; the
// four exchange them through shared memory.  B and C of the tile are shared by
// the block's channels and are laid out [position][state] there.
#pragma once

#include "seq_common.cuh"

namespace spconv {
namespace seq {

constexpr int kScanThreads = 128;
constexpr int kScanChannels = kScanThreads / 4;  // channels of a block

struct ScanParams {
    const void *u, *delta, *z, *B, *C, *dy;
    const float *A, *D, *delta_bias, *state, *dfinal;
    const int32_t *lengths, *slots;
    void *y, *du, *ddelta, *dz, *dB, *dC;
    float *final_state, *pool, *dA, *dD, *ddelta_bias, *dstate;
    // chunks of the sequence: what each leaves (N x chunks x channels x S), then,
    // joined, what each starts from
    float *h_chunk, *g_chunk;
    float *dt_chunk;               // N x chunks x channels: sum of its step sizes
    float *part_bc;                // 2 x blocks x N x L x S: a block's share of dB, dC
    float *part_a;                 // N x segments x channels x (S + 2): of dA, dD, ddelta_bias
    int64_t u_sn, u_sc, d_sn, d_sc, z_sn, z_sc, dy_sn, dy_sc;
    int64_t b_sn, b_sg, b_ss, c_sn, c_sg, c_ss;
    int N, channels, L, S, groups, per_group;  // channels of a group
    int blocks_per_group;
    int softplus, num_slots;
    int chunks, chunk_len;         // chunk_len: a multiple of the tile
    int segments, chunks_per_segment;
    int wide;                      // forward: the tile with fewer lanes per channel
    int vec;                       // input rows can be read as vectors
    int vec_y;                     // output rows (N x channels x L) likewise
};

// Where a thread works: sequence, group, channel (valid or not) and rows.
struct ScanPlace {
    int n, g, c, len;
    bool valid;

    __device__ ScanPlace(const ScanParams &p, int n_, int cb) {
        n = n_;
        g = cb / p.blocks_per_group;
        const int in_group = (cb - g * p.blocks_per_group) * kScanChannels + threadIdx.x / 4;
        valid = in_group < p.per_group;
        c = g * p.per_group + (valid ? in_group : 0);
        len = p.lengths ? min(max(p.lengths[n], 0), p.L) : p.L;
    }
};

// The step size of one position.
static __device__ __forceinline__ float step_size(const ScanParams &p, float raw) {
    return p.softplus ? softplus(raw) : raw;
}

// B and C of one tile: a thread holds VE positions of NB (matrix, state) pairs.
// ONLY_B: without C.
template <typename T, int SPT, int VE, bool ONLY_B = false>
struct ScanBC {
    static constexpr int SP = 4 * SPT, TT = 4 * VE;
    static constexpr int kItems = (ONLY_B ? 1 : 2) * SP * 4;
    static constexpr int NB = (kItems + kScanThreads - 1) / kScanThreads;
    Run<T, VE> r[NB];

    __device__ __forceinline__ void load(const ScanParams &p, const ScanPlace &at, int t0, int end) {
        const T *b = static_cast<const T *>(p.B) + at.n * p.b_sn + at.g * p.b_sg;
        const T *c = static_cast<const T *>(p.C) + at.n * p.c_sn + at.g * p.c_sg;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = threadIdx.x + k * kScanThreads;
            const int s = i % SP, q = (i / SP) % 4, which = i / (SP * 4);
            const bool on = i < kItems && s < p.S;
            const T *row = which ? c + s * p.c_ss : b + s * p.b_ss;
            load_run(r[k], row, t0 + q * VE, on ? end : 0, p.vec);
        }
    }
    // to: [2][TT][SP]
    __device__ __forceinline__ void store(float *to) const {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = threadIdx.x + k * kScanThreads;
            if (i >= kItems) break;
            const int s = i % SP, q = (i / SP) % 4, which = i / (SP * 4);
            float *d = to + which * (TT * SP) + q * VE * SP + s;
#pragma unroll
            for (int e = 0; e < VE; ++e) d[e * SP] = r[k][e];
        }
    }
};

// The lane's SPT states as pairs; one state (S <= 4) leaves the second half
// of its pair at zero.
template <int SPT>
struct Pairs {
    static constexpr int N = SPT > 1 ? SPT / 2 : 1;
    f32x2 v[N];

    // from a row of floats in shared memory
    __device__ __forceinline__ void read(const float *row) {
        if constexpr (SPT % 4 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(row + 2 * i);
                v[i] = q.x;
                v[i + 1] = q.y;
            }
        } else if constexpr (SPT == 2) {
            v[0] = *reinterpret_cast<const f32x2 *>(row);
        } else {
            v[0] = pack2(row[0], 0.f);
        }
    }
    __device__ __forceinline__ void write(float *row) const {
        if constexpr (SPT % 4 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 2)
                *reinterpret_cast<ulonglong2 *>(row + 2 * i) = make_ulonglong2(v[i], v[i + 1]);
        } else if constexpr (SPT == 2) {
            *reinterpret_cast<f32x2 *>(row) = v[0];
        } else {
            row[0] = unpack2(v[0]).x;
        }
    }
    // from a row of S floats in global memory, the lane's from s0; zeros behind S
    __device__ __forceinline__ void load(const float *row, int s0, int S) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int s = s0 + 2 * i;
            v[i] = pack2(s < S ? row[s] : 0.f, SPT > 1 && s + 1 < S ? row[s + 1] : 0.f);
        }
    }
    __device__ __forceinline__ void store(float *row, int s0, int S) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int s = s0 + 2 * i;
            const float2 f = unpack2(v[i]);
            if (s < S) row[s] = f.x;
            if (SPT > 1 && s + 1 < S) row[s + 1] = f.y;
        }
    }
    __device__ __forceinline__ void fill(float x) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = pack2(x, x);
    }
    __device__ __forceinline__ void scale(float x) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = mul2(v[i], pack2(x, x));
    }
    // the sum of all
    __device__ __forceinline__ float sum() const {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 f = unpack2(v[i]);
            t += SPT > 1 ? f.x + f.y : f.x;
        }
        return t;
    }
};

// v[0..SPT) = the lane's states of one row of SP floats in shared memory.
template <int SPT>
static __device__ __forceinline__ void read_states(float (&v)[SPT], const float *row) {
    if constexpr (SPT % 4 == 0) {
#pragma unroll
        for (int i = 0; i < SPT; i += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(row + i);
            v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
        }
    } else if constexpr (SPT == 2) {
        const float2 q = *reinterpret_cast<const float2 *>(row);
        v[0] = q.x; v[1] = q.y;
    } else {
        v[0] = row[0];
    }
}
template <int SPT>
static __device__ __forceinline__ void write_states(float *row, const float (&v)[SPT]) {
    if constexpr (SPT % 4 == 0) {
#pragma unroll
        for (int i = 0; i < SPT; i += 4)
            *reinterpret_cast<float4 *>(row + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else if constexpr (SPT == 2) {
        *reinterpret_cast<float2 *>(row) = make_float2(v[0], v[1]);
    } else {
        row[0] = v[0];
    }
}

// A lane's states in global memory: S floats in a row, the lane's from s0.
template <int SPT>
static __device__ __forceinline__ void load_states(float (&v)[SPT], const float *row, int s0, int S) {
#pragma unroll
    for (int i = 0; i < SPT; ++i) v[i] = s0 + i < S ? row[s0 + i] : 0.f;
}
template <int SPT>
static __device__ __forceinline__ void store_states(float *row, const float (&v)[SPT], int s0, int S) {
#pragma unroll
    for (int i = 0; i < SPT; ++i)
        if (s0 + i < S) row[s0 + i] = v[i];
}

// Host: checks of sizes that every entry makes, and the parameters.
int scan_check_sizes(const spconv_scan_args *a);
ScanParams scan_params(const spconv_scan_args *a);
// Host: joins the chunks' ends to their starts (see the kernel).
int scan_join_chunks(const ScanParams &p, bool grad, cudaStream_t stream);

// f(integral_constant<int, SPT>) for the smallest SPT of 1, 2, 4, 8, 16 with
// 4 * SPT >= S.
template <typename F>
inline int by_states(int S, F f) {
    if (S <= 4) return f(std::integral_constant<int, 1>{});
    if (S <= 8) return f(std::integral_constant<int, 2>{});
    if (S <= 16) return f(std::integral_constant<int, 4>{});
    if (S <= 32) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}

}  // namespace seq
}  // namespace spconv
