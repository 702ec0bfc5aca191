// Low-rank adapters of many requests beside a shared projection:
//
//   out = y + scale_i b_i (a_i x),  i = index[n];  out = y where i is no adapter
//
// Two kernels: v = a_i x (R x P floats per request, in the workspace), then the
// sum over R beside the read of y.
#include "seq_common.cuh"

namespace spconv {
namespace seq {
namespace {

constexpr int kThreads = 256;

struct AdapterParams {
    const void *x, *a, *b, *y;
    const int32_t *index;
    const float *scale;
    void *out;
    float *v;
    int64_t x_sn, x_sc;
    int N, P, C, M, R, adapters;
};

static __device__ __forceinline__ int adapter_of(const AdapterParams &p, int64_t n) {
    const int i = p.index[n];
    return i >= 0 && i < p.adapters ? i : -1;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) shrink_kernel(const AdapterParams p) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (int64_t)p.N * p.R * p.P) return;
    const int64_t nr = i / p.P, n = nr / p.R;
    const int pos = (int)(i - nr * p.P), r = (int)(nr - n * p.R);
    const int k = adapter_of(p, n);
    if (k < 0) return;
    const T *x = static_cast<const T *>(p.x) + n * p.x_sn + pos;
    const T *a = static_cast<const T *>(p.a) + ((int64_t)k * p.R + r) * p.C;
    float v = 0.f;
    for (int c = 0; c < p.C; ++c) v = fmaf(to_f32(a[c]), to_f32(x[c * p.x_sc]), v);
    p.v[i] = v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) expand_kernel(const AdapterParams p) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (int64_t)p.N * p.M * p.P) return;
    const int64_t nm = i / p.P, n = nm / p.M;
    const int pos = (int)(i - nm * p.P), m = (int)(nm - n * p.M);
    const int k = adapter_of(p, n);
    float o = to_f32(static_cast<const T *>(p.y)[i]);
    if (k >= 0) {
        const T *b = static_cast<const T *>(p.b) + ((int64_t)k * p.M + m) * p.R;
        const float *v = p.v + n * p.R * p.P + pos;
        float s = 0.f;
        for (int r = 0; r < p.R; ++r) s = fmaf(to_f32(b[r]), v[(int64_t)r * p.P], s);
        o = fmaf(p.scale ? p.scale[k] : 1.f, s, o);
    }
    static_cast<T *>(p.out)[i] = from_f32<T>(o);
}

int check_sizes(const spconv_adapter_args *a) {
    if (!a || a->N < 0 || a->P < 0 || a->C < 0 || a->M < 0 || a->R < 1 || a->adapters < 0)
        return SPCONV_ERR_INVALID_ARG;
    if (a->dtype < SPCONV_F32 || a->dtype > SPCONV_F16) return SPCONV_ERR_INVALID_ARG;
    if (!stride_ok(a->x_stride_n) || !stride_ok(a->x_stride_c)) return SPCONV_ERR_INVALID_ARG;
    return a->R > 64 ? SPCONV_ERR_UNSUPPORTED : SPCONV_OK;
}

}  // namespace
}  // namespace seq
}  // namespace spconv

using namespace spconv::seq;

SPCONV_API int64_t spconv_adapter_workspace(const spconv_adapter_args *a) {
    if (check_sizes(a)) return 0;
    return (int64_t)a->N * a->R * a->P * 4;
}

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
    const int64_t need = spconv_adapter_workspace(a);
    if (need && (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < need))
        return SPCONV_ERR_INVALID_ARG;
    const int64_t ab = (int64_t)a->adapters * a->R * e;
    if ((a->out != a->y && overlap(a->out, out * e, a->y, out * e)) ||
        overlap(a->out, out * e, a->x, extent(a->N, a->C, a->P, a->x_stride_n, a->x_stride_c, e)) ||
        overlap(a->out, out * e, a->a, ab * a->C) || overlap(a->out, out * e, a->b, ab * a->M))
        return SPCONV_ERR_INVALID_ARG;
    AdapterParams p{};
    p.x = a->x; p.a = a->a; p.b = a->b; p.y = a->y; p.index = a->index; p.scale = a->scale;
    p.out = a->out; p.v = static_cast<float *>(a->workspace);
    p.x_sn = a->x_stride_n; p.x_sc = a->x_stride_c;
    p.N = a->N; p.P = a->P; p.C = a->C; p.M = a->M; p.R = a->R; p.adapters = a->adapters;
    const int64_t inner = (int64_t)a->N * a->R * a->P;
    const int64_t bi = (inner + kThreads - 1) / kThreads, bo = (out + kThreads - 1) / kThreads;
    if (bi > 0x7fffffff || bo > 0x7fffffff) return SPCONV_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_dtype(a->dtype, [&](auto t) {
        using T = decltype(t);
        shrink_kernel<T><<<(unsigned)bi, kThreads, 0, s>>>(p);
        expand_kernel<T><<<(unsigned)bo, kThreads, 0, s>>>(p);
        return launch_status();
    });
}
