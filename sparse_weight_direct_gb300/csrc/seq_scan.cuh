// Internal: parameters and pieces that the selective scan's forward
// (seq_scan.cu) and backward (seq_scan_backward.cu) kernels share.
#pragma once

#include "seq_common.cuh"

namespace spconv {
namespace seq {

struct ScanParams {
    const void *u, *delta, *z, *B, *C, *dy;
    const float *A, *D, *delta_bias, *state, *dfinal;
    const int32_t *lengths, *slots;
    void *y, *du, *ddelta, *dz, *dB, *dC;
    float *final_state, *pool, *dA, *dD, *ddelta_bias, *dstate;
    // chunks (backward: tiles for h, segments for g) of the sequence: what each
    // leaves (N x chunks x channels x S), then, joined, what each starts from
    float *h_chunk, *g_chunk;
    float *dt_chunk, *dt_segment;  // N x chunks x channels: sum of its step sizes
    float *part_bc;                // 2 x blocks x N x L x S: a block's share of dB, dC
    float *part_a;                 // N x segments x channels x (S + 2): of dA, dD, ddelta_bias
    int64_t u_sn, u_sc, d_sn, d_sc, z_sn, z_sc, dy_sn, dy_sc;
    int64_t b_sn, b_sg, b_ss, c_sn, c_sg, c_ss;
    int N, channels, L, S, groups, per_group;  // channels of a group
    int blocks_per_group;          // along the channels of a group
    int softplus, num_slots;
    int chunks, chunk_len;         // chunk_len: a multiple of the tile
    int tiles, segments, tiles_per_segment;  // backward
    int vec;                       // input rows can be read as vectors
    int vec_y;                     // output rows (N x channels x L) likewise
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
