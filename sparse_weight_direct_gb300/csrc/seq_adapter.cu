// Low-rank adapters of many requests beside a shared projection:
//
//   out = y + scale_i b_i (a_i x),  i = index[n];  out = y where i is no adapter
//
// Bound: x and y are read once and out written once, and 2 R (C + M)
// operations per position are few beside that, so memory bounds prompts and
// latency bounds tokens.  Both forms are one launch: a thread-block cluster
// takes a tile of one request's positions, its blocks split the C channels of
// v = a x, add their parts of v through distributed shared memory in the
// order of their ranks, and split the M rows of b v.  So x is read once, v
// never leaves the SMs, and the rows of b and y that do not depend on v can be
// fetched before it is there.
//
// Prompts use matrix instructions on registers (mma.sync): with R <= 64 rows
// an operand tile is far too small to keep the tensor memory path busy, and
// the products take a fraction of the time of the reads and writes around them.
// 8 x 1024 positions, 2048 -> 4096, rank 32 in bf16 take 39 us (0.61 of the
// measured bandwidth; rank 64: 60 us): a wave of clusters, whose two phases do not overlap.
#include <cooperative_groups.h>

#include <utility>

#include "seq_common.cuh"

namespace cg = cooperative_groups;

namespace spconv {
namespace seq {
namespace {

struct AdapterParams {
    const void *x, *a, *b, *y;
    const int32_t *index;
    const float *scale;
    void *out;
    int64_t x_sn, x_sc;
    int N, P, C, M, R, adapters;
    int tiles;                     // prompts: tiles of positions of a request
    int row_lanes;                 // tokens: lanes that share a row of b (a power of two)
    int vec_x, vec_a, vec_b, vec_y;  // rows can be read 16 (b of prompts: 4) bytes at a time
};

constexpr int kMaxRanks = 8;  // blocks of a cluster
constexpr int kMaxR = 64;

static __device__ __forceinline__ int adapter_of(const AdapterParams &p, int64_t n) {
    const int i = p.index[n];
    return i >= 0 && i < p.adapters ? i : -1;
}

// ---------------------------------------------------------------- matrix instructions

// d += a b, 16 x 8 x 16 of 16-bit types
template <typename T>
static __device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d += a b, 16 x 8 x 8 of 32-bit values with 11 bits of significand
static __device__ __forceinline__ void mma8(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// v = hi + lo, each of 11 bits: 22 of v's 24 bits at least.
static __device__ __forceinline__ void split_tf32(float v, uint32_t &hi, uint32_t &lo) {
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(v));
    const float rest = v - __uint_as_float(hi);
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(rest));
}
// two values as words of three bfloat16 parts, each what the ones before leave:
// all 24 bits of both
static __device__ __forceinline__ void split_bf16(float a, float b, uint32_t (&parts)[3]) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        parts[k] = f32_to_word<__nv_bfloat16>(a, b);
        const float2 h = word_to_f32<__nv_bfloat16>(parts[k]);
        a -= h.x;
        b -= h.y;
    }
}
// Sums of parts' products are NaN where the whole ones' are an infinity (a part of
// zero, or of the other sign, against it) or near the largest value (whose first
// part rounds beyond it).  So sums that are not finite are formed again from whole
// products.
static __device__ __forceinline__ bool finite4(float a, float b, float c, float d) {
    return fmaf(a, 0.f, b * 0.f) + fmaf(c, 0.f, d * 0.f) == 0.f;
}
static __device__ __forceinline__ bool finite(float v) { return fabsf(v) <= 3.40282347e38f; }

static __device__ __forceinline__ uint32_t smem_address(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
static __device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_address(p)));
}
static __device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_address(p)));
}
// 16 bytes, or zeros
static __device__ __forceinline__ void copy16(void *to, const void *from, bool on) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(smem_address(to)),
                 "l"(from), "r"(on ? 16 : 0)
                 : "memory");
}

// ---------------------------------------------------------------- prompts

constexpr int kPos = 64;    // positions of a tile
constexpr int kStages = 3;
constexpr int kThreads = 128;

template <typename T, int RT>
struct PromptTile {
    static constexpr bool kWide = sizeof(T) == 4;
    static constexpr int RP = 16 * RT;  // rows of a, padded
    static constexpr int kChan = kWide ? 32 : 64;  // channels of a stage
    static constexpr int kVec = 16 / sizeof(T);
    // pitches in elements: the eight rows of a matrix read start in different
    // banks; 32-bit fragments take rows 4 (a) and 8 (x) banks apart
    static constexpr int kXPitch = kPos + 8;
    static constexpr int kAPitch = kWide ? kChan + 4 : kChan + 8;
    static constexpr int kXBytes = kChan * kXPitch * (int)sizeof(T);
    static constexpr int kStage = kXBytes + RP * kAPitch * (int)sizeof(T);
    static constexpr int kVPitch = kPos + 4;
    static constexpr int kV = RP * kVPitch * 4;
    // Behind the products the stages' place is taken by the block's part of v
    // and by rows of y on their way: tiles of 16 x 32 for each warp.
    static constexpr int kDepth = kWide ? 4 : 6;
    static constexpr int kRing = kDepth * (kThreads / 32) * 16 * 32 * (int)sizeof(T);
    static constexpr int kFront =
        kStages * kStage > kV + kRing ? kStages * kStage : kV + kRing;
    static constexpr int kSmem = kFront + kV;
    // Blocks of an SM that registers are held to where the compiler would take more
    // (0: as it likes).
    static constexpr int kBlocks = kWide ? 0 : std::is_same<T, __half>::value ? (RT == 2) * 4 : (RT == 4) * 3;
};

// One stage: kChan channels from c0 of the tile's positions and of a's rows.
template <typename T, int RT>
static __device__ __forceinline__ void fetch_stage(const AdapterParams &p, unsigned char *stage,
                                                   const T *x, const T *a, int c0, int p0) {
    using G = PromptTile<T, RT>;
    constexpr int V = G::kVec, kChan = G::kChan;
    T *xs = reinterpret_cast<T *>(stage), *as = reinterpret_cast<T *>(stage + G::kXBytes);
    if (p.vec_x) {
        for (int i = threadIdx.x; i < kChan * (kPos / V); i += kThreads) {
            const int c = i / (kPos / V), q = i % (kPos / V) * V;
            const bool on = c0 + c < p.C && p0 + q < p.P;  // rows are whole vectors
            copy16(xs + c * G::kXPitch + q, on ? x + (int64_t)(c0 + c) * p.x_sc + p0 + q : x, on);
        }
    } else {
        for (int i = threadIdx.x; i < kChan * kPos; i += kThreads) {
            const int c = i / kPos, q = i % kPos;
            xs[c * G::kXPitch + q] = c0 + c < p.C && p0 + q < p.P
                                         ? x[(int64_t)(c0 + c) * p.x_sc + p0 + q]
                                         : from_f32<T>(0.f);
        }
    }
    if (p.vec_a) {
        for (int i = threadIdx.x; i < G::RP * (kChan / V); i += kThreads) {
            const int r = i / (kChan / V), q = i % (kChan / V) * V;
            const bool on = r < p.R && c0 + q < p.C;
            copy16(as + r * G::kAPitch + q, on ? a + (int64_t)r * p.C + c0 + q : a, on);
        }
    } else {
        for (int i = threadIdx.x; i < G::RP * kChan; i += kThreads) {
            const int r = i / kChan, q = i % kChan;
            as[r * G::kAPitch + q] =
                r < p.R && c0 + q < p.C ? a[(int64_t)r * p.C + c0 + q] : from_f32<T>(0.f);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// Runs of eight positions (16-bit) or four (32-bit) of y, eight positions in
// all, zeros where there are none.
template <typename T>
struct Eight {
    static constexpr int V = 16 / sizeof(T), K = 8 / V;
    Run<T, V> r[K];
    __device__ __forceinline__ void load(const T *row, int at, int end, bool vec) {
#pragma unroll
        for (int k = 0; k < K; ++k) load_run(r[k], row, at + k * V, end, vec);
    }
    __device__ __forceinline__ void read(const T *shared) {
#pragma unroll
        for (int k = 0; k < K; ++k) r[k] = reinterpret_cast<const Run<T, V> *>(shared)[k];
    }
    __device__ __forceinline__ float get(int i) const { return r[i / V][i % V]; }
    __device__ __forceinline__ void store(const float (&v)[8], T *row, int at, int end, bool vec) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[V];
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = v[k * V + i];
            r[k].put(w);
            store_run(r[k], row, at + k * V, end, vec);
        }
    }
};

template <typename T, int RT>
__global__ void __launch_bounds__(kThreads, PromptTile<T, RT>::kBlocks) prompt_kernel(const AdapterParams p) {
    using G = PromptTile<T, RT>;
    constexpr bool kWide = G::kWide;
    constexpr int kChan = G::kChan;
    extern __shared__ __align__(128) unsigned char smem[];
    float *part = reinterpret_cast<float *>(smem);              // [RP][kVPitch]
    float *v = reinterpret_cast<float *>(smem + G::kFront);     // likewise
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int job = blockIdx.x / ranks;
    const int n = job / p.tiles, p0 = (job - n * p.tiles) * kPos;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
    const int id = adapter_of(p, n);
    const T *y = static_cast<const T *>(p.y) + (int64_t)n * p.M * p.P;
    T *out = static_cast<T *>(p.out) + (int64_t)n * p.M * p.P;

    // rows of the output that are this block's; a warp takes 16 at a time of one
    // half of the positions, eight consecutive ones of two rows in each lane
    const int mtiles = (p.M + 15) / 16;
    const int m_first = (int)((int64_t)mtiles * rank / ranks);
    const int m_last = (int)((int64_t)mtiles * (rank + 1) / ranks);
    const int half = p0 + (warp >> 1) * 32, at = half + j * 8;
    if (id < 0) {  // the same for the whole cluster
        if (static_cast<const void *>(out) == y) return;
        constexpr int V = G::kVec, kRow = kPos / V, kBatch = 8;  // reads under way at once
        const int row_end = min(p.M, m_last * 16), pieces = (row_end - m_first * 16) * kRow;
        for (int i0 = threadIdx.x; i0 < pieces; i0 += kThreads * kBatch) {
            Run<T, V> r[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + k * kThreads, row = m_first * 16 + i / kRow;
                load_run(r[k], y + (int64_t)row * p.P, p0 + i % kRow * V, i < pieces ? p.P : 0,
                         p.vec_y);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + k * kThreads, row = m_first * 16 + i / kRow;
                store_run(r[k], out + (int64_t)row * p.P, p0 + i % kRow * V, i < pieces ? p.P : 0,
                          p.vec_y);
            }
        }
        return;
    }
    const T *x = static_cast<const T *>(p.x) + n * p.x_sn;
    const T *a = static_cast<const T *>(p.a) + (int64_t)id * p.R * p.C;
    const T *b = static_cast<const T *>(p.b) + (int64_t)id * p.M * p.R;
    const float scale = p.scale ? p.scale[id] : 1.f;

    // what a warp takes next of b is on its way while it multiplies
    constexpr bool kPairs = !kWide;  // products of 16-bit parts
    constexpr bool kAhead = kPairs || RT <= 2;  // (32-bit rows of more would not fit)
    uint32_t next[kPairs ? RT : kAhead ? 2 * RT : 1][4];
    const int m_own = m_first + (warp & 1);
    const bool whole_b = p.vec_b && p.R == G::RP;
    auto fetch_b = [&](int m) {
        const int r0 = m * 16 + g, r1 = r0 + 8;
        if (kAhead && whole_b && m < m_last && m * 16 + 16 <= p.M) {
            // whole rows of words
            constexpr int kRow = kPairs ? RT * 8 : RT * 16;
            const uint32_t *q = reinterpret_cast<const uint32_t *>(b) + (int64_t)r0 * kRow + j;
#pragma unroll
            for (int k = 0; k < (kPairs ? RT : 2 * RT); ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    next[kAhead ? k : 0][i] =
                        __ldg(q + (i & 1) * (8 * kRow) + k * 8 + (i >> 1) * 4);
        } else if constexpr (kPairs) {
#pragma unroll
            for (int k = 0; k < RT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = i & 1 ? r1 : r0, c = k * 16 + (i >> 1) * 8 + 2 * j;
                    const T *q = b + (int64_t)row * p.R + c;
                    next[k][i] = 0;
                    if (m < m_last && row < p.M) {
                        if (p.vec_b && c + 1 < p.R)
                            next[k][i] = *reinterpret_cast<const uint32_t *>(q);
                        else
                            next[k][i] = (c < p.R ? bits_of(q[0]) : 0u) |
                                         (c + 1 < p.R ? bits_of(q[1]) << 16 : 0u);
                    }
                }
        } else if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < 2 * RT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = i & 1 ? r1 : r0, c = k * 8 + (i >> 1) * 4 + j;
                    next[k][i] = m < m_last && row < p.M && c < p.R
                                     ? bits_of(b[(int64_t)row * p.R + c]) : 0;
                }
        }
    };
    // and of y kDepth tiles are: a lane copies what it will use itself
    constexpr int kDepth = G::kDepth;
    T *ring = reinterpret_cast<T *>(smem + G::kV) + warp * (kDepth * 512) + lane * 8;
    const int64_t y_half = 8 * (int64_t)p.P, y_step = 32 * (int64_t)p.P;
    const T *y_next = y + (int64_t)(m_own * 16 + g) * p.P + at;
    int row_next = m_own * 16 + g;
    auto fetch_y = [&](int slot) {
        if (p.vec_y && row_next - g < m_last * 16) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int k = 0; k < 8; k += G::kVec) {
                    const bool on = row_next + 8 * r < p.M && at + k < p.P;
                    copy16(ring + slot * 512 + r * 256 + k, on ? y_next + r * y_half + k : y, on);
                }
        }
        y_next += y_step;
        row_next += 32;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // v = a x over this block's channels; a warp has 16 of the positions
    {
        const int stages = (p.C + kChan - 1) / kChan;
        const int first = (int)((int64_t)stages * rank / ranks);
        const int last = (int)((int64_t)stages * (rank + 1) / ranks);
        float acc[RT][2][4];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][q][i] = 0.f;
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) {
            if (first + k < last)
                fetch_stage<T, RT>(p, smem + k * G::kStage, x, a, (first + k) * kChan, p0);
            else
                asm volatile("cp.async.commit_group;" ::: "memory");
        }
        for (int s = first; s < last; ++s) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncthreads();  // the stage has arrived, and the one to be fetched is free
            const int ahead = s + kStages - 1;
            if (ahead < last)
                fetch_stage<T, RT>(p, smem + (ahead - first) % kStages * G::kStage, x, a,
                                   ahead * kChan, p0);
            else
                asm volatile("cp.async.commit_group;" ::: "memory");
            const unsigned char *stage = smem + (s - first) % kStages * G::kStage;
            const T *xs = reinterpret_cast<const T *>(stage);
            const T *as = reinterpret_cast<const T *>(stage + G::kXBytes);
            if constexpr (!kWide) {
#pragma unroll
                for (int k = 0; k < kChan; k += 16) {
                    uint32_t xb[4];
                    ldmatrix4_trans(xb, xs + (k + (lane & 15)) * G::kXPitch + warp * 16 + (lane >> 4) * 8);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        uint32_t aa[4];
                        ldmatrix4(aa, as + (r * 16 + (lane & 15)) * G::kAPitch + k + (lane >> 4) * 8);
                        mma16<T>(acc[r][0], aa, xb[0], xb[1]);
                        mma16<T>(acc[r][1], aa, xb[2], xb[3]);
                    }
                }
            } else {
                // The instruction does not round its running sums to nearest: a stage's
                // are added to the others' outside it (2048 channels: an error of 5e-7
                // for 1.6e-6).
                float sum[RT][2][4] = {};
#pragma unroll
                for (int k = 0; k < kChan; k += 8) {
                    uint32_t xh[2][2], xl[2][2];
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            split_tf32(to_f32(xs[(k + j + 4 * i) * G::kXPitch + warp * 16 + q * 8 + g]),
                                       xh[q][i], xl[q][i]);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        uint32_t ah[4], al[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            split_tf32(to_f32(as[(r * 16 + g + 8 * (i & 1)) * G::kAPitch + k + j +
                                                 4 * (i >> 1)]),
                                       ah[i], al[i]);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            mma8(sum[r][q], al, xh[q][0], xh[q][1]);
                            mma8(sum[r][q], ah, xl[q][0], xl[q][1]);
                            mma8(sum[r][q], ah, xh[q][0], xh[q][1]);
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[r][q][i] += sum[r][q][i];
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        fetch_b(m_own);
#pragma unroll
        for (int k = 0; k < kDepth; ++k) fetch_y(k);
        // rows behind R are zero whatever x holds
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = r * 16 + g + 8 * (i >> 1);
                    part[row * G::kVPitch + warp * 16 + q * 8 + 2 * j + (i & 1)] =
                        row < p.R ? acc[r][q][i] : 0.f;
                }
    }
    // four positions of a row of v; 16-bit factors are whole in the instruction
    auto place_of = [](int i) { return i / (kPos / 4) * G::kVPitch + i % (kPos / 4) * 4; };
    auto form_again = [&](int i, float4 &t) {
        if (!kWide || finite4(t.x, t.y, t.z, t.w)) return;
        const int row = i / (kPos / 4), first = p0 + i % (kPos / 4) * 4;
        if (row >= p.R) return;
        float sum[4] = {};
#pragma unroll 4
        for (int c = 0; c < p.C; ++c) {
            const float f = to_f32(a[(int64_t)row * p.C + c]);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (first + q < p.P) sum[q] = fmaf(f, to_f32(x[c * p.x_sc + first + q]), sum[q]);
        }
        t.x = finite(t.x) ? t.x : sum[0];
        t.y = finite(t.y) ? t.y : sum[1];
        t.z = finite(t.z) ? t.z : sum[2];
        t.w = finite(t.w) ? t.w : sum[3];
    };
    if (ranks > 1) {
        cluster.sync();
        // each block adds a share of v over the ranks and hands it to all
        for (int i = rank * kThreads + threadIdx.x; i < G::RP * kPos / 4; i += ranks * kThreads) {
            const int o = place_of(i);
            float4 f[kMaxRanks], t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kMaxRanks; ++k)  // read together, added in their order
                f[k] = k < ranks ? *reinterpret_cast<const float4 *>(cluster.map_shared_rank(part, k) + o)
                                 : t;
#pragma unroll
            for (int k = 0; k < kMaxRanks; ++k) {
                t.x += f[k].x; t.y += f[k].y; t.z += f[k].z; t.w += f[k].w;
            }
            form_again(i, t);
#pragma unroll
            for (int k = 0; k < kMaxRanks; ++k)
                if (k < ranks) *reinterpret_cast<float4 *>(cluster.map_shared_rank(v, k) + o) = t;
        }
        cluster.sync();
    } else {
        v = part;
        __syncthreads();
        if (kWide) {
            for (int i = threadIdx.x; i < G::RP * kPos / 4; i += kThreads)
                form_again(i, *reinterpret_cast<float4 *>(part + place_of(i)));
            __syncthreads();
        }
    }

    // out = y + scale b v.  Column q of the four tiles of eight that a warp
    // multiplies stands for position 8 (q / 2) + 2 tile + q % 2 of its half, so
    // that a lane's results are eight consecutive positions.
    // v keeps its bits between the products.  Against bfloat16 it goes as three parts
    // of that type.  Half precision does not reach as far as sums of its products,
    // and one scale for a position's sums loses those 2^14 below the largest: so its
    // b goes to the 32-bit instruction, which holds it, with v as two parts, and the rows
    // of a step of eight in the order in which b's words hold them (8 x 1024 positions,
    // 2048 -> 4096: rank 32 42 us, rank 64 82, its registers leave two blocks per SM;
    // b as two bfloat16 parts against three of v took 46 and 85).
    constexpr bool kHalf = std::is_same<T, __half>::value, kBf16 = kPairs && !kHalf;
    constexpr int KS = kBf16 ? RT : RT * 2;  // steps of 16 or 8 rows of v
    constexpr int kParts = kBf16 ? 3 : 2;
    uint32_t vp[KS][4][2][kParts];
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float *col = v + (warp >> 1) * 32 + (g >> 1) * 8 + 2 * t + (g & 1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (kBf16) {
                    const float *two = col + (k * 16 + i * 8 + 2 * j) * G::kVPitch;
                    split_bf16(two[0], two[G::kVPitch], vp[k][t][i]);
                } else {
                    const int row = k * 8 + (kHalf ? 2 * j + i : i * 4 + j);
                    split_tf32(col[row * G::kVPitch], vp[k][t][i][0], vp[k][t][i][1]);
                }
            }
        }
    int slot = 0;
    T *o = out + (int64_t)(m_own * 16 + g) * p.P + at;
    int m = m_own;
    for (; m < m_last; m += 2, o += y_step) {
        const int r0 = m * 16 + g, r1 = r0 + 8;
        Eight<T> e0, e1;
        auto read_y = [&]() {
            if (p.vec_y) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
                e0.read(ring + slot * 512);
                e1.read(ring + slot * 512 + 256);
            } else {
                e0.load(y + (int64_t)r0 * p.P, at, r0 < p.M ? p.P : 0, false);
                e1.load(y + (int64_t)r1 * p.P, at, r1 < p.M ? p.P : 0, false);
            }
        };
        auto more_y = [&]() {
            fetch_y(slot);
            slot = slot + 1 < kDepth ? slot + 1 : 0;
        };
        // (behind the products of 16-bit types, where its registers are short: bf16
        // rank 64 68 -> 60 us; before those of 32 bits, which wait for it: rank 64 221 -> 205)
        if (kWide) read_y();
        uint32_t now[kPairs ? RT : kAhead ? 2 * RT : 1][4];
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < (kPairs ? RT : 2 * RT); ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) now[k][i] = next[k][i];
        }
        fetch_b(m + 2);
        if (kWide) more_y();
        float acc[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
        if constexpr (kBf16) {
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = kParts - 1; e >= 0; --e)
                        mma16<T>(acc[t], now[k], vp[k][t][0][e], vp[k][t][1][e]);
        } else if constexpr (kHalf) {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint32_t *w = now[k / 2] + k % 2 * 2;
                const float2 w0 = word_to_f32<T>(w[0]), w1 = word_to_f32<T>(w[1]);
                const uint32_t bh[4] = {bits_of(w0.x), bits_of(w1.x), bits_of(w0.y), bits_of(w1.y)};
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    mma8(acc[t], bh, vp[k][t][0][1], vp[k][t][1][1]);
                    mma8(acc[t], bh, vp[k][t][0][0], vp[k][t][1][0]);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t bh[4], bl[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = i & 1 ? r1 : r0, c = k * 8 + (i >> 1) * 4 + j;
                    const float f = kAhead ? __uint_as_float(now[kAhead ? k : 0][i])
                                    : row < p.M && c < p.R ? to_f32(b[(int64_t)row * p.R + c]) : 0.f;
                    split_tf32(f, bh[i], bl[i]);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    mma8(acc[t], bl, vp[k][t][0][0], vp[k][t][1][0]);
                    mma8(acc[t], bh, vp[k][t][0][1], vp[k][t][1][1]);
                    mma8(acc[t], bh, vp[k][t][0][0], vp[k][t][1][0]);
                }
            }
        }
        if (!kWide) read_y();
        bool fine = true;
#pragma unroll
        for (int t = 0; t < 4; ++t) fine &= finite4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
        if (__any_sync(~0u, !fine)) break;
        if (!kWide) more_y();
        float f0[8], f1[8];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f0[2 * t + i] = fmaf(scale, acc[t][i], e0.get(2 * t + i));
                f1[2 * t + i] = fmaf(scale, acc[t][2 + i], e1.get(2 * t + i));
            }
        if (r0 < p.M) e0.store(f0, o, 0, p.P - at, p.vec_y);
        if (r1 < p.M) e1.store(f1, o + y_half, 0, p.P - at, p.vec_y);
    }
    if (m >= m_last) return;
    // the warp's rows from one on whose sums are not finite, by whole products
    // (behind the loop: in it they cost registers, and with them blocks of an SM)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    const float *col = v + (warp >> 1) * 32 + j * 8;
    for (; m < m_last; m += 2)
        for (int row = m * 16 + g; row < min(m * 16 + 16, p.M); row += 8) {
            const T *q = b + (int64_t)row * p.R;
            float f[8] = {};
            for (int r = 0; r < p.R; ++r) {
                const float w = to_f32(q[r]);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = fmaf(w, col[r * G::kVPitch + i], f[i]);
            }
            Eight<T> e;
            e.load(y + (int64_t)row * p.P, at, p.P, p.vec_y);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = fmaf(scale, f[i], e.get(i));
            e.store(f, out + (int64_t)row * p.P, at, p.P, p.vec_y);
        }
}

// ---------------------------------------------------------------- single tokens

constexpr int kTokenThreads = 256, kTokenWarps = kTokenThreads / 32;

// A cluster per token.  A warp sums two rows of a at a time over the block's
// channels, every block adds the ranks' parts of v, and row_lanes lanes sum a row
// of b, 16 bytes each (with a lane per row a read takes 16 bytes of 32 lines).
// What does not depend on v -- the first rows of b, of y -- is read before it.
// What counts is how many reads are under way: 48 tokens, 4096 x 4096, rank 16,
// bf16 take 6.0 us (two blocks per SM 9.2); 128 of rank 64 take 31 where they
// share 16 adapters, 44 with one each (three blocks took 1.29 times as long, with
// four rows of a at a time 1.13 times).
template <typename T>
__global__ void __launch_bounds__(kTokenThreads, 4) token_kernel(const AdapterParams p) {
    __shared__ float part[kMaxR];
    __shared__ __align__(16) float v[kMaxR];
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int n = blockIdx.x / ranks;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int id = adapter_of(p, n);
    const T *y = static_cast<const T *>(p.y) + (int64_t)n * p.M;
    T *out = static_cast<T *>(p.out) + (int64_t)n * p.M;
    const int m_first = (int)((int64_t)p.M * rank / ranks);
    const int m_last = (int)((int64_t)p.M * (rank + 1) / ranks);
    if (id < 0) {  // the same for the whole cluster
        for (int m = m_first + threadIdx.x; m < m_last; m += kTokenThreads) out[m] = y[m];
        return;
    }
    const T *x = static_cast<const T *>(p.x) + n * p.x_sn;
    const T *a = static_cast<const T *>(p.a) + (int64_t)id * p.R * p.C;
    const T *b = static_cast<const T *>(p.b) + (int64_t)id * p.M * p.R;
    const float scale = p.scale ? p.scale[id] : 1.f;
    constexpr int V = 16 / sizeof(T), RW = 2, kRows = 4;  // kRows: of b that a lane has under way
    // channels in whole vectors, so that a block's slice starts on one
    const int vectors = (p.C + V - 1) / V;
    const int c_first = (int)((int64_t)vectors * rank / ranks) * V;
    const int c_last = min(p.C, (int)((int64_t)vectors * (rank + 1) / ranks) * V);
    const int part_of = threadIdx.x & (p.row_lanes - 1), side = kTokenThreads / p.row_lanes;
    Run<T, V> rows[kRows];
    float ys[kRows];
    auto fetch = [&](int m) {
#pragma unroll
        for (int k = 0; k < kRows; ++k, m += side) {
            load_run(rows[k], b + (int64_t)m * p.R, part_of * V, m < m_last ? p.R : 0, p.vec_b);
            ys[k] = part_of == 0 && m < m_last ? to_f32(y[m]) : 0.f;
        }
    };
    int m = m_first + threadIdx.x / p.row_lanes;
    fetch(m);
    for (int r0 = warp * RW; r0 < p.R; r0 += kTokenWarps * RW) {
        float s[RW] = {};
        const T *row = a + (int64_t)r0 * p.C;
#pragma unroll 2
        for (int c = c_first + lane * V; c < c_last; c += 32 * V) {
            Run<T, V> xr, ar[RW];
            if (p.x_sc == 1) {
                load_run(xr, x, c, c_last, p.vec_x);
            } else {
                float f[V];
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = c + i < c_last ? to_f32(x[(c + i) * p.x_sc]) : 0.f;
                xr.put(f);
            }
#pragma unroll
            for (int k = 0; k < RW; ++k)
                load_run(ar[k], row + (int64_t)k * p.C, c, r0 + k < p.R ? c_last : 0, p.vec_a);
#pragma unroll
            for (int k = 0; k < RW; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) s[k] = fmaf(ar[k][i], xr[i], s[k]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
            for (int k = 0; k < RW; ++k) s[k] += __shfl_xor_sync(~0u, s[k], o);
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < RW; ++k)
                if (r0 + k < p.R) part[r0 + k] = s[k];
        }
    }
    cluster.sync();
    if (threadIdx.x < kMaxR) {
        float t = 0.f;
        if (threadIdx.x < p.R) {
            float f[kMaxRanks];  // read together, added in their order
#pragma unroll
            for (int k = 0; k < kMaxRanks; ++k)
                f[k] = k < ranks ? cluster.map_shared_rank(part, k)[threadIdx.x] : 0.f;
#pragma unroll
            for (int k = 0; k < kMaxRanks; ++k) t += f[k];
        }
        v[threadIdx.x] = t;
    }
    __syncthreads();
    auto left = cluster.barrier_arrive();  // this block has read the others' parts
    float mine[V];  // v against the lane's part of a row
#pragma unroll
    for (int i = 0; i < V; ++i) mine[i] = part_of * V + i < kMaxR ? v[part_of * V + i] : 0.f;
    for (int base = m_first; base < m_last; base += kRows * side) {
        float o[kRows], y0[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            o[k] = 0.f;
            y0[k] = ys[k];
#pragma unroll
            for (int i = 0; i < V; ++i) o[k] = fmaf(rows[k][i], mine[i], o[k]);
        }
        const int at = m;
        m += kRows * side;
        if (base + kRows * side < m_last) fetch(m);
        for (int d = p.row_lanes / 2; d; d >>= 1)
#pragma unroll
            for (int k = 0; k < kRows; ++k) o[k] += __shfl_xor_sync(~0u, o[k], d);
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            if (part_of == 0 && at + k * side < m_last)
                out[at + k * side] = from_f32<T>(fmaf(scale, o[k], y0[k]));
    }
    cluster.barrier_wait(std::move(left));  // its own part may go once all have
}

// ---------------------------------------------------------------- host side

int check_sizes(const spconv_adapter_args *a) {
    if (!a || a->N < 0 || a->P < 0 || a->C < 0 || a->M < 0 || a->R < 1 || a->adapters < 0)
        return SPCONV_ERR_INVALID_ARG;
    if (a->dtype < SPCONV_F32 || a->dtype > SPCONV_F16) return SPCONV_ERR_INVALID_ARG;
    if (!stride_ok(a->x_stride_n) || !stride_ok(a->x_stride_c)) return SPCONV_ERR_INVALID_ARG;
    constexpr int kMost = 1 << 26;  // rows, channels, positions: their products with a tile's
                                    // pieces stay within 32 bits
    return a->R > kMaxR || a->C > kMost || a->M > kMost || a->P > kMost ? SPCONV_ERR_UNSUPPORTED
                                                                       : SPCONV_OK;
}

// Launches `jobs` clusters of `ranks` blocks.
int launch_clusters(void (*fn)(AdapterParams), int64_t jobs, int ranks, int threads, int smem,
                    const AdapterParams &p, cudaStream_t stream) {
    if (jobs * ranks > 0x7fffffff) return SPCONV_ERR_UNSUPPORTED;
    if (int rc = raise_smem(reinterpret_cast<const void *>(fn), smem)) return rc;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(jobs * ranks));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, p) != cudaSuccess) {
        cudaGetLastError();
        return SPCONV_ERR_CUDA;
    }
    return SPCONV_OK;
}

// Blocks of a cluster: twice as many until there are `want` blocks, as long as
// each has `least` of both the channels and the rows.
int ranks_for(const AdapterParams &p, int64_t jobs, int64_t want, int least) {
    int r = 1;
    const int small = p.C < p.M ? p.C : p.M;
    while (r < kMaxRanks && jobs * r < want && small / (2 * r) >= least) r *= 2;
    return r;
}

}  // namespace
}  // namespace seq
}  // namespace spconv

using namespace spconv::seq;

SPCONV_API int spconv_adapter_add(const spconv_adapter_args *a, void *stream) {
    const int st = check_sizes(a);
    if (st) return st;
    const int64_t out = (int64_t)a->N * a->M * a->P;
    if (out == 0) return SPCONV_OK;
    const size_t e = dtype_size(a->dtype);
    if (!a->y || !a->out || !a->index || (a->C > 0 && !a->x) ||
        (a->adapters > 0 && (!a->b || (a->C > 0 && !a->a))))
        return SPCONV_ERR_INVALID_ARG;
    for (const void *q : {a->x, a->a, a->b, a->y, (const void *)a->out})
        if (!aligned(q, e)) return SPCONV_ERR_INVALID_ARG;
    if (!aligned(a->index, 4) || !aligned(a->scale, 4)) return SPCONV_ERR_INVALID_ARG;
    const int64_t ab = (int64_t)a->adapters * a->R * e;
    if ((a->out != a->y && overlap(a->out, out * e, a->y, out * e)) ||
        !apart({{a->out, (int64_t)(out * e)}},
               {{a->x, extent(a->N, a->C, a->P, a->x_stride_n, a->x_stride_c, e)}, {a->a, ab * a->C},
                {a->b, ab * a->M}, {a->index, a->N * 4LL}, {a->scale, a->adapters * 4LL}}))
        return SPCONV_ERR_INVALID_ARG;
    AdapterParams p{};
    p.x = a->x; p.a = a->a; p.b = a->b; p.y = a->y; p.index = a->index; p.scale = a->scale;
    p.out = a->out;
    p.x_sn = a->x_stride_n; p.x_sc = a->x_stride_c;
    p.N = a->N; p.P = a->P; p.C = a->C; p.M = a->M; p.R = a->R; p.adapters = a->adapters;
    p.vec_a = rows_aligned(a->a, 0, a->C, e);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->P == 1) {
        p.vec_x = rows_aligned(a->x, a->x_stride_n, 0, e);
        p.vec_b = rows_aligned(a->b, 0, a->R, e);
        p.row_lanes = 1;
        while (p.row_lanes * 16 < (int)(a->R * e)) p.row_lanes *= 2;
        return by_dtype(a->dtype, [&](auto t) {
            return launch_clusters(token_kernel<decltype(t)>, p.N, ranks_for(p, p.N, 4 * kSMs, 64),
                                   kTokenThreads, 0, p, s);
        });
    }
    p.tiles = (int)(((int64_t)a->P + kPos - 1) / kPos);
    p.vec_x = rows_aligned(a->x, a->x_stride_n, a->x_stride_c, e) && a->P * e % 16 == 0;
    p.vec_y = rows_aligned(a->y, 0, a->P, e) && rows_aligned(a->out, 0, a->P, e);
    p.vec_b = aligned(a->b, 4) && a->R % 2 == 0;
    const int64_t jobs = (int64_t)p.N * p.tiles;
    const int ranks = ranks_for(p, jobs, 2 * kSMs, 64);
    return by_dtype(a->dtype, [&](auto t) {
        using T = decltype(t);
        auto go = [&](auto rt) {
            constexpr int RT = decltype(rt)::value;
            return launch_clusters(prompt_kernel<T, RT>, jobs, ranks, kThreads,
                                   PromptTile<T, RT>::kSmem, p, s);
        };
        if (a->R <= 16) return go(std::integral_constant<int, 1>{});
        if (a->R <= 32) return go(std::integral_constant<int, 2>{});
        return go(std::integral_constant<int, 4>{});
    });
}
