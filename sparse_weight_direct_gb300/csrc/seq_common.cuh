// Internal: what the sequence operators (seq_*.cu) share -- element types,
// vector loads of a row's positions, the activations, and the checks of their
// C entries.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <type_traits>
#include <utility>

#include "spconv.h"

#define SPCONV_API extern "C" __attribute__((visibility("default")))

namespace spconv {
namespace seq {

constexpr int kSMs = 152;
constexpr int kVec = 8;  // positions a thread holds of a row
constexpr int kMaxLength = 0x7fff0000;  // positions, sequences, channels: a block's reach, or a
                                        // grid's step (at most 65535), beyond stays within 32 bits

// ---------------------------------------------------------------- elements

static __device__ __forceinline__ float to_f32(float v) { return v; }
static __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
static __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
static __device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two elements as they lie in one word, and back (rounded to nearest).
template <typename T>
static __device__ __forceinline__ float2 word_to_f32(uint32_t w) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <typename T>
static __device__ __forceinline__ uint32_t f32_to_word(float a, float b) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}
static __device__ __forceinline__ uint32_t bits_of(float v) { return __float_as_uint(v); }
static __device__ __forceinline__ uint32_t bits_of(__nv_bfloat16 v) {
    return __bfloat16_as_ushort(v);
}
static __device__ __forceinline__ uint32_t bits_of(__half v) { return __half_as_ushort(v); }

// V consecutive elements of a row, kept as the words they are loaded in (as
// elements, a 16-bit type would take a register each).
template <typename T, int V = kVec>
struct alignas(V * sizeof(T) >= 16 ? 16 : V * sizeof(T)) Run {
    static constexpr bool kWide = sizeof(T) == 4;
    static constexpr int W = V * sizeof(T) / 4;
    uint32_t w[W];

    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (kWide) return __uint_as_float(w[i]);
        else return i & 1 ? word_to_f32<T>(w[i / 2]).y : word_to_f32<T>(w[i / 2]).x;
    }
    __device__ __forceinline__ void put(const float (&v)[V]) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (kWide) w[i] = __float_as_uint(v[i]);
            else w[i] = f32_to_word<T>(v[2 * i], v[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
};

// row[t0, t0 + V) of global memory where t < end, zeros behind (positions behind `end` are not
// read unless the run is whole, so what lies there does not matter).
// vec: the run's address is aligned to the run.
template <typename T, int V>
static __device__ __forceinline__ void load_run(Run<T, V> &r, const T *__restrict__ row, int t0,
                                                int end, bool vec) {
    if (vec && t0 + V <= end) {
        // the rest of the line is the row's next run: have it brought to L2 with this one
        if constexpr (sizeof(r) == 16)
            asm("ld.global.nc.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                : "l"(row + t0));
        else
            r = *reinterpret_cast<const Run<T, V> *>(row + t0);
    } else {
        r.clear();
        constexpr int per = 4 / sizeof(T);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (t0 + i < end) r.w[i / per] |= bits_of(row[t0 + i]) << (i % per * 16);
    }
}

// A run that starts anywhere lies across W / 4 or W / 4 + 1 words of 16 bytes: the
// first one, or NULL where not all of them are within [begin, end).
template <typename T, int V>
static __device__ __forceinline__ const uint4 *words_across(const T *p, const T *begin, const T *end) {
    const unsigned off = (unsigned)((uintptr_t)p & 15);
    const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(p) - off);
    const bool in = reinterpret_cast<uintptr_t>(q) >= reinterpret_cast<uintptr_t>(begin) &&
                    reinterpret_cast<uintptr_t>(q + Run<T, V>::W / 4 + (off != 0)) <= reinterpret_cast<uintptr_t>(end);
    return in ? q : nullptr;
}
// The run that starts `off` bytes (below 16) into the words s[0 .. W + 3].
template <typename T, int V>
static __device__ __forceinline__ void run_across(Run<T, V> &run, uint32_t (&s)[Run<T, V>::W + 4], unsigned off) {
    constexpr int W = Run<T, V>::W;
    if (off & 8)
#pragma unroll
        for (int k = 0; k < W + 2; ++k) s[k] = s[k + 2];
    if (off & 4)
#pragma unroll
        for (int k = 0; k < W + 1; ++k) s[k] = s[k + 1];
    const unsigned half = off & 2 ? 16 : 0;
#pragma unroll
    for (int k = 0; k < W; ++k) run.w[k] = __funnelshift_r(s[k], s[k + 1], half);
}
template <typename T, int V>
static __device__ __forceinline__ bool load_across(Run<T, V> &run, const T *p, const T *begin, const T *end) {
    constexpr int W = Run<T, V>::W;
    const uint4 *q = words_across<T, V>(p, begin, end);
    if (!q) return false;
    uint32_t s[W + 4] = {};
#pragma unroll
    for (int k = 0; k < W / 4 + 1; ++k)
        if (k < W / 4 || ((uintptr_t)p & 15)) {
            const uint4 u = __ldg(q + k);
            s[4 * k] = u.x, s[4 * k + 1] = u.y, s[4 * k + 2] = u.z, s[4 * k + 3] = u.w;
        }
    run_across(run, s, (unsigned)((uintptr_t)p & 15));
    return true;
}

// row[t0, t0 + V) = r where t < L.
template <typename T, int V>
static __device__ __forceinline__ void store_run(const Run<T, V> &r, T *__restrict__ row, int t0,
                                                 int L, bool vec) {
    if (vec && t0 + V <= L) {
        *reinterpret_cast<Run<T, V> *>(row + t0) = r;
    } else {
        using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
        constexpr int per = 4 / sizeof(T);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (t0 + i < L)
                reinterpret_cast<Bits *>(row)[t0 + i] = (Bits)(r.w[i / per] >> (i % per * 16));
    }
}

// V channels of a row, whole vectors or single elements.
template <typename T, int V>
static __device__ __forceinline__ void take(float (&v)[V], const T *p) {
    if constexpr (V == 1) {
        v[0] = to_f32(*p);
    } else {
        const Run<T, V> run = *reinterpret_cast<const Run<T, V> *>(p);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = run[j];
    }
}
template <typename T, int V>
static __device__ __forceinline__ void give(const float (&v)[V], T *p) {
    if constexpr (V == 1) {
        *p = from_f32<T>(v[0]);
    } else {
        Run<T, V> run;
        run.put(v);
        *reinterpret_cast<Run<T, V> *>(p) = run;
    }
}

// A thread's sum of many numbers, with what its additions lost: 131,072 of 1.21 added to
// one float are 3e-3 off.
struct LongSum {
    float s = 0.f, lost = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float t = __fadd_rn(s, v), part = __fsub_rn(t, s);
        lost += __fadd_rn(__fsub_rn(s, __fsub_rn(t, part)), __fsub_rn(v, part));
        s = t;
    }
    __device__ __forceinline__ float value() const { return lost == lost ? s + lost : s; }  // (infinity stays)
};

// ---------------------------------------------------------------- activations

constexpr float kLog2e = 1.4426950408889634f;

// 2^x, relative error about 2^-22.
static __device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / x, relative error about 2^-23; 0 for an infinite x.
static __device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + e^-v)
static __device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(-kLog2e * v)); }
static __device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
// d silu / dv
static __device__ __forceinline__ float silu_grad(float v) {
    const float s = sigmoid(v);
    return s * (1.f + v * (1.f - s));
}
// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v|: nothing overflows.  With
// t = e / (2 + e), log(1 + e) = 2 artanh(t) = t P(t^2), t^2 <= 1/9; P is the
// degree-4 interpolant of 2 artanh(t) / t at the Chebyshev nodes (relative
// error 4e-9), so the small values that step sizes are keep their digits.
static __device__ __forceinline__ float softplus(float v) {
    const float e = ex2(-kLog2e * fabsf(v));
    const float t = e * rcp(2.f + e), x = t * t;
    float q = fmaf(x, 0.28157778f, 0.27965158f);
    q = fmaf(x, q, 0.40024595f);
    q = fmaf(x, q, 0.66666322f);
    q = fmaf(x, q, 2.00000001f);
    return fmaf(t, q, fmaxf(v, 0.f));
}

// ---------------------------------------------------------------- pairs of floats
//
// Two floats in one 64-bit register: one instruction issues two products or
// sums, which is what the scan's loops are short of.

using f32x2 = unsigned long long;

static __device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
static __device__ __forceinline__ float2 unpack2(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
static __device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
static __device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
static __device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
static __device__ __forceinline__ f32x2 ex2_2(f32x2 v) {
    const float2 f = unpack2(v);
    return pack2(ex2(f.x), ex2(f.y));
}

// Two neighbouring elements of a run.
template <typename T, int V>
static __device__ __forceinline__ f32x2 pair_of(const Run<T, V> &r, int j) {
    return pack2(r[j], r[j + 1]);
}

// e^(dt A) of two states, A in units of log2(e).  The fast exponential comes
// out low by 2e-8 on average (measured over the arguments that decays have, -2^-8
// to -1), and a state keeps that from every position: the offset, half a unit in the
// last place, takes it back (states after 100 slow steps: error 1.3e-6 -> 6e-7).
// For a step of size zero the result is one exactly.
constexpr float kDecayUp = 2.98023224e-8f;
static __device__ __forceinline__ f32x2 decay2(f32x2 dt, f32x2 A) {
    return ex2_2(fma2(dt, A, pack2(kDecayUp, kDecayUp)));
}
static __device__ __forceinline__ float decay(float dt, float A) {
    return ex2(fmaf(dt, A, kDecayUp));
}

// ---------------------------------------------------------------- checks of the C entries

inline bool aligned(const void *p, size_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

inline size_t dtype_size(int dtype) { return dtype == SPCONV_F32 ? 4 : 2; }

// Bytes from the first to behind the last element of an N x C x L tensor.
inline int64_t extent(int64_t N, int64_t C, int64_t L, int64_t sn, int64_t sc, int64_t size) {
    if (N <= 0 || C <= 0 || L <= 0) return 0;
    return ((N - 1) * sn + (C - 1) * sc + L) * size;
}

inline bool overlap(const void *a, int64_t an, const void *b, int64_t bn) {
    if (!a || !b || an <= 0 || bn <= 0) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

struct Span {
    const void *p;
    int64_t bytes;
};

// No output lies over another one or over what is read.
inline bool apart(std::initializer_list<Span> out, std::initializer_list<Span> in) {
    for (const Span &o : out) {
        for (const Span &i : in)
            if (overlap(o.p, o.bytes, i.p, i.bytes)) return false;
        for (const Span *k = out.begin(); k != &o; ++k)
            if (overlap(o.p, o.bytes, k->p, k->bytes)) return false;
    }
    return true;
}

// A stride that 64-bit byte offsets can hold for any valid index.
inline bool stride_ok(int64_t s) { return s >= 0 && s <= (int64_t)1 << 40; }

// Rows of runs can be read as vectors: base and strides are multiples of
// 16 bytes.
inline bool rows_aligned(const void *p, int64_t sn, int64_t sc, size_t size) {
    return aligned(p, 16) && (sn * (int64_t)size) % 16 == 0 && (sc * (int64_t)size) % 16 == 0;
}

// Device side of one dtype: f(T{}) with T the element type.
template <typename F>
inline int by_dtype(int dtype, F f) {
    switch (dtype) {
        case SPCONV_F32: return f(float{});
        case SPCONV_BF16: return f(__nv_bfloat16{});
        case SPCONV_F16: return f(__half{});
    }
    return SPCONV_ERR_INVALID_ARG;
}

// Allows a kernel `bytes` of dynamic shared memory, once per kernel and device
// (a call per launch costs host time, and a launch may be under capture).
inline int raise_smem(const void *fn, int bytes) {
    if (bytes <= 48 * 1024) return SPCONV_OK;
    static std::mutex lock;
    static std::pair<const void *, int> done[256];
    static int count = 0;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return SPCONV_ERR_CUDA;
    std::lock_guard<std::mutex> hold(lock);
    for (int i = 0; i < count; ++i)
        if (done[i].first == fn && done[i].second == device) return SPCONV_OK;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return SPCONV_ERR_CUDA;
    }
    if (count < 256) done[count++] = {fn, device};
    return SPCONV_OK;
}

inline int launch_status() {
    return cudaGetLastError() == cudaSuccess ? SPCONV_OK : SPCONV_ERR_CUDA;
}

}  // namespace seq
}  // namespace spconv
