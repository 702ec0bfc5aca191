// Beam search: the selection over beams and vocabulary, and the reordering of the
// states' pools that follows it.
#include "seq_common.cuh"

namespace spconv {
namespace seq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBeams = 32;
constexpr int kVocab = 8;       // logits of a thread's load
constexpr int kMaxLoads = 8;    // loads of a thread in a part of a row
constexpr int kMaxPart = kThreads * kVocab * kMaxLoads;
constexpr int kFound = 1024;    // logits of a part that are ranked
constexpr int kWays = 1024;     // ways of a request that are ranked
constexpr float kLargest = 3.402823466e38f;

struct BeamParams {
    const void *logits;
    const float *scores;
    const uint8_t *ended;
    float *new_scores;
    int32_t *tokens, *parents;
    uint8_t *new_ended;
    float2 *sums;   // N x B x parts: the largest logit and the sum of exponentials over it
    uint64_t *best; // N x B x parts x K: the part's best, largest first
    int64_t sn, sb;
    int N, B, V, K, eos;
    int part, parts;  // tokens of a part, parts of a row
};

// A float's place in the order of floats, as an unsigned number, and back.
static __device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
static __device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// A logit and its token: the larger key is the better one, of equal logits the
// lower token.  Zero is below every key of a logit.
static __device__ __forceinline__ uint64_t key_of(float v, int token) {
    return (uint64_t)ordered(v + 0.f) << 32 | (uint32_t)~token;  // (+ 0: a negative zero is a zero)
}
static __device__ __forceinline__ float finite_or_least(float v) {
    return fminf(fmaxf(v, -INFINITY), kLargest);  // (NaN counts as minus infinity)
}

// The K-th largest of a warp's 32 values (K <= 32): a bitonic sort, largest first.
static __device__ __forceinline__ float kth_of_warp(float v, int K) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int d = size / 2; d; d /= 2) {
            const float o = __shfl_xor_sync(~0u, v, d);
            const bool larger = ((lane & d) == 0) == ((lane & size) == 0);  // (of the pair, this one keeps the larger)
            v = larger ? fmaxf(v, o) : fminf(v, o);
        }
    return __shfl_sync(~0u, v, K - 1);
}

// Part of a row of logits: the largest, the sum of the exponentials over it, and
// the K best.  A thread reads kVocab logits at a time and keeps the largest and the
// sum.  A warp with K lanes whose largest are at least some value has K logits of
// at least that value, so the K-th of a warp's lanes, and the largest of those over
// the warps, bounds the part's K-th best logit from below.  Some four times K logits
// lie above it; the threads that have them are found by their largest, their logits
// read once more by eight lanes, and ranked against one another.
//
// Bound: instruction issue (0.63 an SMSP and clock, some 17 an element) ahead of the
// memory: 64 x 8 beams x 128,000 in bf16 take 45 us, 0.43 of the measured bandwidth.
// Every key ranked against the block's 256 threads' and each element's key formed took
// 117 us; two lanes' worth of logits looked at one thread after the other 47.
template <typename T>
__global__ void __launch_bounds__(kThreads) beam_part_kernel(const BeamParams p) {
    __shared__ float2 warps[kWarps];
    __shared__ float bounds[kWarps];
    __shared__ uint64_t found[kFound];
    __shared__ uint64_t bests[kWarps];
    __shared__ int count;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = blockIdx.x % p.parts;
    const int64_t row = blockIdx.x / p.parts;
    const int n = (int)(row / p.B), b = (int)(row - (int64_t)n * p.B);
    if (p.ended && p.ended[row]) return;
    const T *at = static_cast<const T *>(p.logits) + n * p.sn + b * p.sb;
    const int first = part * p.part, stop = min(p.V, first + p.part);
    // (A thread's tokens do not depend on where the row lies, so that rows of equal
    // logits have equal sums, to the bit, and equal beams tie.)
    const auto load = [&](float (&v)[kVocab], int t0) {
        Run<T, kVocab> run;
        if (load_across(run, at + t0, at + first, at + stop)) {
#pragma unroll
            for (int j = 0; j < kVocab; ++j) v[j] = run[j];
        } else {
#pragma unroll
            for (int j = 0; j < kVocab; ++j) v[j] = t0 + j < stop ? to_f32(at[t0 + j]) : -INFINITY;
        }
    };
    const int start = first + (int)threadIdx.x * kVocab;
    float most = -kLargest, sum = 0.f;
    const auto add = [&](const float (&v)[kVocab]) {
        float top = v[0];
#pragma unroll
        for (int j = 1; j < kVocab; ++j) top = fmaxf(top, v[j]);
        if (top > most) {
            sum *= ex2((most - top) * kLog2e);
            most = top;
        }
        const f32x2 less = pack2(-most, -most), scale = pack2(kLog2e, kLog2e);
        f32x2 s = pack2(sum, 0.f);
#pragma unroll
        for (int j = 0; j < kVocab; j += 2) s = add2(s, ex2_2(mul2(add2(pack2(v[j], v[j + 1]), less), scale)));
        const float2 f = unpack2(s);
        sum = f.x + f.y;
    };
    int next = start;
    if (((uintptr_t)(at + first) & 15) == 0) {
#pragma unroll 8
        for (; next + kVocab <= stop; next += kThreads * kVocab) {
            const Run<T, kVocab> run = *reinterpret_cast<const Run<T, kVocab> *>(at + next);
            float v[kVocab];
#pragma unroll
            for (int j = 0; j < kVocab; ++j) v[j] = run[j];
            add(v);
        }
    }
#pragma unroll 2
    for (; next < stop; next += kThreads * kVocab) {
        float v[kVocab];
        load(v, next);
        add(v);
    }
    if (!(most <= kLargest) || sum != sum) {  // an infinity or NaN among them: again, with what they count as
        most = -kLargest;
        sum = 0.f;
        for (int t0 = start; t0 < stop; t0 += kThreads * kVocab) {
            float v[kVocab];
            load(v, t0);
#pragma unroll
            for (int j = 0; j < kVocab; ++j) v[j] = finite_or_least(v[j]);
            add(v);
        }
    }
    // (a thread with minus infinities alone has a sum of zero: there is nothing to be found)
    const float mine = sum > 0.f ? most : -INFINITY;
    float2 all{most, sum};
    for (int d = 16; d; d >>= 1) {
        const float m = __shfl_xor_sync(~0u, all.x, d), s = __shfl_xor_sync(~0u, all.y, d);
        const float top = fmaxf(all.x, m);
        all.y = all.y * ex2((all.x - top) * kLog2e) + s * ex2((m - top) * kLog2e);
        all.x = top;
    }
    const float kth = kth_of_warp(mine, p.K);
    if (lane == 0) {
        warps[warp] = all;
        bounds[warp] = kth;
    }
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    if (threadIdx.x == 0) {
        float2 s = warps[0];
        for (int w = 1; w < kWarps; ++w) {
            const float top = fmaxf(s.x, warps[w].x);
            s.y = s.y * ex2((s.x - top) * kLog2e) + warps[w].y * ex2((warps[w].x - top) * kLog2e);
            s.x = top;
        }
        p.sums[row * p.parts + part] = s;
    }
    float bound = bounds[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) bound = fmaxf(bound, bounds[w]);
    // the logits of four such threads at a time, a load to each of a thread's eight lanes
    static_assert(kMaxLoads == 8, "eight lanes read a thread's loads");
    unsigned those = __ballot_sync(~0u, mine > -INFINITY && mine >= bound);
    while (those) {
        unsigned left = those;
        for (int o = lane >> 3; o; --o) left &= left - 1;
        const int t0 = first + (warp * 32 + __ffs(left) - 1) * kVocab + (lane & 7) * (kThreads * kVocab);
        if (left && t0 < stop) {
            float v[kVocab];
            load(v, t0);
#pragma unroll
            for (int j = 0; j < kVocab; ++j) {
                const float f = finite_or_least(v[j]);
                if (f > -INFINITY && f >= bound) {
                    const int o = atomicAdd(&count, 1);  // (their order does not matter: they are ranked)
                    if (o < kFound) found[o] = key_of(f, t0 + j);
                }
            }
        }
#pragma unroll
        for (int o = 0; o < 4; ++o) those &= those - 1;
    }
    __syncthreads();
    const int M = count;
    uint64_t *out = p.best + (row * p.parts + part) * p.K;
    if (M <= kFound) {
        for (int o = threadIdx.x; o < M; o += kThreads) {
            const uint64_t k = found[o];
            int up = 0;
            for (int u = 0; u < M; ++u) up += found[u] > k;
            if (up < p.K) out[up] = k;
        }
        for (int o = M + threadIdx.x; o < p.K; o += kThreads) out[o] = 0;
        return;
    }
    // too many alike: one after the other
    uint64_t last = ~(uint64_t)0;
    for (int k = 0; k < p.K; ++k) {
        uint64_t best = 0;
        for (int t0 = start; t0 < stop; t0 += kThreads * kVocab) {
            float v[kVocab];
            load(v, t0);
#pragma unroll
            for (int j = 0; j < kVocab; ++j) {
                const float f = finite_or_least(v[j]);
                const uint64_t key = key_of(f, t0 + j);
                if (f > -INFINITY && key < last && key > best) best = key;
            }
        }
        for (int d = 16; d; d >>= 1) {
            const uint64_t o = __shfl_xor_sync(~0u, best, d);
            best = o > best ? o : best;
        }
        if (lane == 0) bests[warp] = best;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) best = bests[w] > best ? bests[w] : best;
        __syncthreads();
        if (threadIdx.x == 0) out[k] = best;
        last = best;
    }
}

// A way to go on: its total and its place among the request's B * V.
struct Way {
    double total;
    int place;
};
static __device__ __forceinline__ bool better(const Way &a, const Way &b) {
    return a.total > b.total || (a.total == b.total && a.place < b.place);
}
// A total's place in the order of numbers (never NaN; a negative zero is a zero):
// compared as whole numbers, since 64-bit ones of the other kind are slow here.
static __device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.);
    return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}

// A block for each request: the K best of its beams' parts' bests, bounded from
// below as in a part and ranked.  Bound: latency, two reads behind one another, a
// 64-bit logarithm and five block barriers, 8 to 11 us.  (K rounds of a block's maximum:
// 35 us for eight of 512 ways.)
__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamParams p) {
    __shared__ double lse[kMaxBeams], scores[kMaxBeams];
    __shared__ bool ended[kMaxBeams];
    __shared__ float bounds[kWarps];
    __shared__ Way ways[kWays];
    __shared__ uint64_t order[kWays];
    __shared__ Way firsts[kWarps];
    __shared__ int count;
    const int n = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t rows = (int64_t)n * p.B;
    const int per_beam = p.parts * p.K, all = p.B * per_beam;
    const uint64_t *bests = p.best + rows * per_beam;
    // (what an ended beam's lists hold is not used)
    constexpr int kMine = 4;
    uint64_t keys[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int o = threadIdx.x + i * kThreads;
        keys[i] = o < all ? bests[o] : 0;
    }
    if (threadIdx.x < p.B) {
        ended[threadIdx.x] = p.ended && p.ended[rows + threadIdx.x];
        scores[threadIdx.x] = (double)finite_or_least(p.scores[rows + threadIdx.x]);
    }
    for (int b = warp; b < p.B; b += kWarps) {
        const float2 *sums = p.sums + (rows + b) * p.parts;
        float2 s = lane < p.parts ? sums[lane] : make_float2(-kLargest, 0.f);
        LongSum sum_of{s.y};  // (thousands of parts alike would all be rounded to the same side)
        for (int o = lane + 32; o < p.parts; o += 32) {
            const float2 u = sums[o];
            const float top = fmaxf(s.x, u.x), fall = ex2((s.x - top) * kLog2e);
            sum_of.s *= fall;
            sum_of.lost *= fall;
            sum_of.add(u.y * ex2((u.x - top) * kLog2e));
            s.x = top;
        }
        s.y = sum_of.value();
        float most = s.x;
        for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, d));
        float sum = s.y * ex2((s.x - most) * kLog2e);
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
        if (lane == 0) lse[b] = (double)most + log((double)sum);
    }
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    // entry o of the lists, or false
    const auto way = [&](int o, uint64_t key, Way &w) {
        const int b = o / per_beam;
        if (ended[b]) {
            if (o != b * per_beam) return false;
            w = {scores[b], b * p.V + p.eos};
        } else {
            if (!key) return false;
            w = {scores[b] + ((double)unordered((uint32_t)(key >> 32)) - lse[b]), b * p.V + (int)~(uint32_t)key};
        }
        return w.total > -INFINITY;
    };
    // every way of this thread
    const auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int o = threadIdx.x + i * kThreads;
            if (o < all) f(o, keys[i]);
        }
        for (int o = threadIdx.x + kMine * kThreads; o < all; o += kThreads) f(o, bests[o]);
    };
    float most = -INFINITY;
    each([&](int o, uint64_t key) {
        Way w;
        if (way(o, key, w)) most = fmaxf(most, __double2float_rd(w.total));
    });
    const float kth = kth_of_warp(most, p.K);
    if (lane == 0) bounds[warp] = kth;
    __syncthreads();
    float bound = bounds[0];
    for (int w = 1; w < kWarps; ++w) bound = fmaxf(bound, bounds[w]);
    each([&](int o, uint64_t key) {
        Way w;
        if (!way(o, key, w) || w.total < (double)bound) return;
        const int at = atomicAdd(&count, 1);  // (their order does not matter: they are ranked)
        if (at < kWays) {
            ways[at] = w;
            order[at] = ordered(w.total);
        }
    });
    __syncthreads();
    const int M = count;
    const auto store = [&](int k, const Way &w, bool any) {
        const int b = any ? w.place / p.V : k < p.B ? k : 0;
        const int token = any ? w.place - b * p.V : 0;
        const int64_t o = (int64_t)n * p.K + k;
        p.new_scores[o] = any ? (float)w.total : -INFINITY;
        p.tokens[o] = token;
        p.parents[o] = b;
        if (p.new_ended) p.new_ended[o] = ended[b] || token == p.eos;
    };
    if (M <= kWays) {
        for (int o = threadIdx.x; o < M; o += kThreads) {
            const Way w = ways[o];
            const uint64_t mine = order[o];
            int up = 0;
            for (int u = 0; u < M; ++u) up += order[u] > mine || (order[u] == mine && ways[u].place < w.place);
            if (up < p.K) store(up, w, true);
        }
        for (int o = M + threadIdx.x; o < p.K; o += kThreads) store(o, Way{}, false);
        return;
    }
    // too many alike: one after the other
    Way last{INFINITY, -1};
    for (int k = 0; k < p.K; ++k) {
        Way best{-INFINITY, 0x7fffffff};
        each([&](int o, uint64_t key) {
            Way w;
            if (way(o, key, w) && better(last, w) && better(w, best)) best = w;
        });
        for (int d = 16; d; d >>= 1) {
            const Way w{__shfl_xor_sync(~0u, best.total, d), __shfl_xor_sync(~0u, best.place, d)};
            if (better(w, best)) best = w;
        }
        if (lane == 0) firsts[warp] = best;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w)
            if (better(firsts[w], best)) best = firsts[w];
        __syncthreads();
        if (threadIdx.x == 0) store(k, best, best.total > -INFINITY);
        last = best;
    }
}

// ---------------------------------------------------------------- states

constexpr int kMaxPools = 64;    // of a launch
constexpr int kStates = 16384;   // bytes of a state that a block copies

struct ReorderParams {
    char *pools[kMaxPools];
    int64_t bytes[kMaxPools];
    int first[kMaxPools];   // the pool's first block
    uint8_t unit[kMaxPools];  // bytes of a copy: 16, 4, 2 or 1
    const int32_t *parents, *slots;
    int32_t *new_slots;     // NULL: an earlier launch has written them
    int N, B, num_pools, num_slots;
};

template <typename U>
static __device__ __forceinline__ void copy_state(char *to, const char *from, int64_t begin, int64_t end) {
    for (int64_t o = begin + (int64_t)threadIdx.x * sizeof(U); o < end; o += kThreads * sizeof(U))
        *reinterpret_cast<U *>(to + o) = *reinterpret_cast<const U *>(from + o);
}

// Blocks (part of a state, request).  Each warp works out the request's copies
// from its beams' parents, one beam to a lane: no block waits for another's plan,
// and no slot that is read is written.  Bound: memory; 192 copies of 607 KB take 42.6 us,
// 0.81 of the measured bandwidth.
__global__ void __launch_bounds__(kThreads) reorder_kernel(const ReorderParams p) {
    const int n = blockIdx.y, lane = threadIdx.x & 31;
    const bool beam = lane < p.B;
    const int parent = beam ? p.parents[(int64_t)n * p.B + lane] : -1;
    const int mine = beam ? p.slots[(int64_t)n * p.B + lane] : -1;
    const bool valid = beam && parent >= 0 && parent < p.B;
    const unsigned same = __match_any_sync(~0u, valid ? parent : -1 - lane);
    const bool stays = valid && (__ffs(same) - 1) == lane;
    const unsigned taken = __reduce_or_sync(~0u, valid ? 1u << parent : 0u);
    const unsigned moving = __ballot_sync(~0u, beam && !stays);
    unsigned spare = ~taken & (p.B == 32 ? ~0u : (1u << p.B) - 1);
    for (int o = __popc(moving & ((1u << lane) - 1)); o > 0; --o) spare &= spare - 1;
    const int source = __shfl_sync(~0u, mine, valid ? parent : 0);
    const int target_from = beam && !stays ? __ffs(spare) - 1 : valid ? parent : 0;
    const int target = __shfl_sync(~0u, mine, max(target_from, 0));
    if (p.new_slots && blockIdx.x == 0 && threadIdx.x < p.B) p.new_slots[(int64_t)n * p.B + lane] = target;
    unsigned copies = __ballot_sync(~0u, valid && !stays && source >= 0 && source < p.num_slots && target >= 0 &&
                                             target < p.num_slots);
    if (!p.num_pools) return;
    int pool = 0;
    while (pool + 1 < p.num_pools && (int)blockIdx.x >= p.first[pool + 1]) ++pool;
    const int64_t bytes = p.bytes[pool], begin = (int64_t)((int)blockIdx.x - p.first[pool]) * kStates;
    const int64_t end = min(bytes, begin + kStates);
    char *base = p.pools[pool];
    const int unit = p.unit[pool];
    for (; copies; copies &= copies - 1) {
        const int o = __ffs(copies) - 1;
        const char *from = base + __shfl_sync(~0u, source, o) * bytes;
        char *to = base + __shfl_sync(~0u, target, o) * bytes;
        if (unit == 16) copy_state<uint4>(to, from, begin, end);
        else if (unit == 4) copy_state<uint32_t>(to, from, begin, end);
        else if (unit == 2) copy_state<uint16_t>(to, from, begin, end);
        else copy_state<uint8_t>(to, from, begin, end);
    }
}

// ---------------------------------------------------------------- host side

int check_beams(const spconv_beam_select_args *a) {
    if (!a || a->N < 0 || a->B < 1 || a->K < 1 || a->V < 1) return SPCONV_ERR_INVALID_ARG;
    if (a->dtype < SPCONV_F32 || a->dtype > SPCONV_F16 || a->eos < -1 || a->eos >= a->V) return SPCONV_ERR_INVALID_ARG;
    if (!stride_ok(a->logits_stride_n) || !stride_ok(a->logits_stride_b)) return SPCONV_ERR_INVALID_ARG;
    if (a->N > 65535 || a->B > kMaxBeams || a->K > kMaxBeams || (int64_t)a->B * a->V > kMaxLength)
        return SPCONV_ERR_UNSUPPORTED;
    return SPCONV_OK;
}

// Parts of a row: as many as fill the GPU with four blocks per SM, none shorter
// than a load of each thread or longer than kMaxPart.
void beam_plan(BeamParams &p) {
    constexpr int kStep = kThreads * kVocab;
    const int64_t rows = (int64_t)p.N * p.B, most = (p.V + kStep - 1) / kStep;
    int64_t parts = rows ? (4 * kSMs + rows - 1) / rows : 1;
    if (parts > most) parts = most;
    int64_t part = ((p.V + parts - 1) / parts + kStep - 1) / kStep * kStep;
    if (part > kMaxPart) part = kMaxPart;
    p.part = (int)part;
    p.parts = (int)((p.V + part - 1) / part);
}

BeamParams beam_params(const spconv_beam_select_args *a) {
    BeamParams p{};
    p.logits = a->logits; p.scores = a->scores; p.ended = a->ended;
    p.new_scores = a->new_scores; p.tokens = a->tokens; p.parents = a->parents; p.new_ended = a->new_ended;
    p.sn = a->logits_stride_n; p.sb = a->logits_stride_b;
    p.N = a->N; p.B = a->B; p.V = a->V; p.K = a->K; p.eos = a->eos;
    beam_plan(p);
    return p;
}

int64_t sums_bytes(const BeamParams &p) { return ((int64_t)p.N * p.B * p.parts * 8 + 15) / 16 * 16; }

}  // namespace
}  // namespace seq
}  // namespace spconv

using namespace spconv::seq;

SPCONV_API int64_t spconv_beam_select_workspace(const spconv_beam_select_args *a) {
    if (check_beams(a)) return 0;
    const BeamParams p = beam_params(a);
    return sums_bytes(p) + (int64_t)p.N * p.B * p.parts * p.K * 8;
}

SPCONV_API int spconv_beam_select(const spconv_beam_select_args *a, void *stream) {
    if (int st = check_beams(a)) return st;
    if (a->N == 0) return SPCONV_OK;
    const int64_t e = dtype_size(a->dtype), N = a->N, B = a->B, K = a->K;
    if (!a->logits || !a->scores || !a->new_scores || !a->tokens || !a->parents || (a->ended && a->eos < 0))
        return SPCONV_ERR_INVALID_ARG;
    if (!aligned(a->logits, e)) return SPCONV_ERR_INVALID_ARG;
    for (const void *q : {(const void *)a->scores, (const void *)a->new_scores, (const void *)a->tokens,
                          (const void *)a->parents})
        if (!aligned(q, 4)) return SPCONV_ERR_INVALID_ARG;
    const int64_t need = spconv_beam_select_workspace(a);
    if (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < need) return SPCONV_ERR_INVALID_ARG;
    if (!apart({{a->new_scores, N * K * 4}, {a->tokens, N * K * 4}, {a->parents, N * K * 4},
                {a->new_ended, N * K}, {a->workspace, need}},
               {{a->logits, extent(N, B, a->V, a->logits_stride_n, a->logits_stride_b, e)},
                {a->scores, N * B * 4}, {a->ended, N * B}}))
        return SPCONV_ERR_INVALID_ARG;
    BeamParams p = beam_params(a);
    p.sums = static_cast<float2 *>(a->workspace);
    p.best = reinterpret_cast<uint64_t *>(static_cast<char *>(a->workspace) + sums_bytes(p));
    const int64_t blocks = N * B * p.parts;
    if (blocks > 0x7fffffff || B * p.parts * K > kMaxLength) return SPCONV_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_dtype(a->dtype, [&](auto t) {
        beam_part_kernel<decltype(t)><<<(unsigned)blocks, kThreads, 0, s>>>(p);
        beam_join_kernel<<<(unsigned)N, kThreads, 0, s>>>(p);
        return launch_status();
    });
}

SPCONV_API int spconv_reorder_states(const spconv_reorder_args *a, void *stream) {
    if (!a || a->N < 0 || a->B < 1 || a->num_pools < 0 || a->num_slots < 0) return SPCONV_ERR_INVALID_ARG;
    if (a->B > kMaxBeams || a->N > 65535) return SPCONV_ERR_UNSUPPORTED;
    if (a->num_pools && (!a->pools || !a->slot_bytes)) return SPCONV_ERR_INVALID_ARG;
    if (a->N == 0) return SPCONV_OK;
    const int64_t table = (int64_t)a->N * a->B * 4;
    if (!a->parents || !a->slots || !a->new_slots || !aligned(a->parents, 4) || !aligned(a->slots, 4) ||
        !aligned(a->new_slots, 4))
        return SPCONV_ERR_INVALID_ARG;
    const Span in[2] = {{a->parents, table}, {a->slots, table}};
    for (const Span &i : in)
        if (overlap(a->new_slots, table, i.p, i.bytes)) return SPCONV_ERR_INVALID_ARG;
    for (int k = 0; k < a->num_pools; ++k) {
        const int64_t size = a->slot_bytes[k];
        if (size < 0 || size > (int64_t)1 << 40) return SPCONV_ERR_INVALID_ARG;
        const Span pool{a->pools[k], size * a->num_slots};
        if (pool.bytes && !pool.p) return SPCONV_ERR_INVALID_ARG;
        if (size / kStates > 1 << 20) return SPCONV_ERR_UNSUPPORTED;  // (64 pools' blocks fit a grid)
        for (const Span &i : {in[0], in[1], Span{a->new_slots, table}})
            if (overlap(pool.p, pool.bytes, i.p, i.bytes)) return SPCONV_ERR_INVALID_ARG;
        for (int o = 0; o < k; ++o)
            if (overlap(pool.p, pool.bytes, a->pools[o], a->slot_bytes[o] * a->num_slots)) return SPCONV_ERR_INVALID_ARG;
    }
    int done = 0;
    do {
        ReorderParams p{};
        p.parents = a->parents; p.slots = a->slots;
        p.new_slots = done ? nullptr : a->new_slots;
        p.N = a->N; p.B = a->B; p.num_slots = a->num_slots;
        int64_t blocks = 0;
        for (; done < a->num_pools && p.num_pools < kMaxPools; ++done) {
            const int64_t size = a->slot_bytes[done];
            if (size == 0 || a->num_slots == 0) continue;
            const int k = p.num_pools++;
            p.pools[k] = static_cast<char *>(a->pools[done]);
            p.bytes[k] = size;
            p.first[k] = (int)blocks;
            const uint64_t lies = (uint64_t)(uintptr_t)p.pools[k] | (uint64_t)size;
            p.unit[k] = lies % 16 == 0 ? 16 : lies % 4 == 0 ? 4 : lies % 2 == 0 ? 2 : 1;
            blocks += (size + kStates - 1) / kStates;
        }
        if (blocks == 0 && !p.new_slots) break;
        reorder_kernel<<<dim3((unsigned)(blocks ? blocks : 1), (unsigned)a->N), kThreads, 0,
                         static_cast<cudaStream_t>(stream)>>>(p);
        if (int st = launch_status()) return st;
    } while (done < a->num_pools);
    return SPCONV_OK;
}
