// residual_rmsnorm.cu -- the residual step between two blocks (norm after a block,
// gate, scale, residual add, norm before the next block) and its gradients, declared
// in include/residual_rmsnorm.h.
//
// One block per row, any n: the row is read once for each of its two statistics and
// once more for the outputs.  The backward's sums over rows go to one partial row per
// block and are added up by a second kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "nvtx_range.h"
#include "residual_rmsnorm.h"

namespace rrms {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 304;  // of the backward: two for each of the 152 SMs
constexpr uint32_t kMaxN = 1u << 20;

struct Args {
    const void *f, *x, *gate, *w_post, *w_pre;
    void *h, *y;
    float *rstd;
    const void *dy, *dh;
    void *df, *dx, *dgate;
    float *dw_post, *dw_pre, *partial;
    int m, n, kind, blocks;
    float eps, scale;
};

template <typename T>
__device__ __forceinline__ float to_f(T v) {
    if constexpr (sizeof(T) == 4) {
        return v;
    } else {
        return (float)v;
    }
}
template <typename T>
__device__ __forceinline__ T from_f(float v) {
    if constexpr (sizeof(T) == 4) {
        return v;
    } else {
        return (T)v;
    }
}

// Sum over the block, the same value in every thread; `s` holds one float per warp and is free again after the
// next call's first barrier.
__device__ __forceinline__ float block_sum(float x, float *s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += s[w];
    return t;
}

template <typename T>
__device__ __forceinline__ float gate_at(const Args &a, int64_t row, int j) {
    if (a.kind == RESIDUAL_GATE_NONE) return 1.f;
    const T *g = static_cast<const T *>(a.gate);
    return to_f(a.kind == RESIDUAL_GATE_CHANNEL ? g[j] : g[row * a.n + j]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) forward_row_kernel(const Args a) {
    __shared__ float s[kThreads / 32];
    const int64_t row = blockIdx.x, at = row * a.n;
    const T *f = static_cast<const T *>(a.f) + at, *x = static_cast<const T *>(a.x) + at;
    const T *wp = static_cast<const T *>(a.w_post), *wq = static_cast<const T *>(a.w_pre);
    T *h = static_cast<T *>(a.h) + at, *y = static_cast<T *>(a.y) + at;
    float sum = 0.f;
    for (int j = threadIdx.x; j < a.n; j += kThreads) sum = fmaf(to_f(f[j]), to_f(f[j]), sum);
    const float rp = 1.0f / sqrtf(block_sum(sum, s) / (float)a.n + a.eps);
    auto stream = [&](int j) {
        return fmaf(a.scale * gate_at<T>(a, row, j), to_f(f[j]) * rp * to_f(wp[j]), to_f(x[j]));
    };
    sum = 0.f;
    for (int j = threadIdx.x; j < a.n; j += kThreads) {
        const float v = stream(j);
        sum = fmaf(v, v, sum);
    }
    const float rq = 1.0f / sqrtf(block_sum(sum, s) / (float)a.n + a.eps);
    for (int j = threadIdx.x; j < a.n; j += kThreads) {
        const float v = stream(j);
        h[j] = from_f<T>(v);
        y[j] = from_f<T>(v * rq * to_f(wq[j]));
    }
    if (threadIdx.x == 0 && a.rstd) a.rstd[2 * row] = rp, a.rstd[2 * row + 1] = rq;
}

// Partial sums of block b: partial[b][0] dw_post, [1] dw_pre, [2] dgate (per channel), n values each; thread j % 256
// alone adds to column j.
template <typename T>
__global__ void __launch_bounds__(kThreads) backward_row_kernel(const Args a) {
    __shared__ float s[kThreads / 32];
    const T *wp = static_cast<const T *>(a.w_post), *wq = static_cast<const T *>(a.w_pre);
    float *part = a.partial + (int64_t)blockIdx.x * 3 * a.n;
    for (int j = threadIdx.x; j < 3 * a.n; j += kThreads) part[j] = 0.f;
    __syncthreads();
    for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
        const int64_t at = row * a.n;
        const T *f = static_cast<const T *>(a.f) + at, *h = static_cast<const T *>(a.h) + at;
        const T *dy = static_cast<const T *>(a.dy) + at, *dh = a.dh ? static_cast<const T *>(a.dh) + at : nullptr;
        T *df = static_cast<T *>(a.df) + at, *dx = static_cast<T *>(a.dx) + at;
        const float rp = a.rstd[2 * row], rq = a.rstd[2 * row + 1];
        float sum = 0.f;
        for (int j = threadIdx.x; j < a.n; j += kThreads)
            sum = fmaf(to_f(wq[j]) * to_f(dy[j]), to_f(h[j]), sum);
        const float c = rq * rq * (block_sum(sum, s) / (float)a.n);
        auto total = [&](int j) {  // G
            return rq * (to_f(wq[j]) * to_f(dy[j]) - to_f(h[j]) * c) + (dh ? to_f(dh[j]) : 0.f);
        };
        sum = 0.f;
        for (int j = threadIdx.x; j < a.n; j += kThreads)
            sum = fmaf(to_f(wp[j]) * (a.scale * total(j) * gate_at<T>(a, row, j)), to_f(f[j]), sum);
        const float e = rp * rp * (block_sum(sum, s) / (float)a.n);
        for (int j = threadIdx.x; j < a.n; j += kThreads) {
            const float gj = total(j), u = a.scale * gj, fn = to_f(f[j]) * rp, dz = u * gate_at<T>(a, row, j);
            const float dg = u * fn * to_f(wp[j]);
            df[j] = from_f<T>(rp * (to_f(wp[j]) * dz - to_f(f[j]) * e));
            part[j] += dz * fn;
            part[a.n + j] += to_f(dy[j]) * to_f(h[j]) * rq;
            if (a.kind == RESIDUAL_GATE_CHANNEL) part[2 * a.n + j] += dg;
            if (a.kind == RESIDUAL_GATE_ELEMENT) static_cast<T *>(a.dgate)[at + j] = from_f<T>(dg);
            dx[j] = from_f<T>(gj);  // last: dX may be dH's buffer
        }
    }
}

__global__ void __launch_bounds__(kThreads) partial_sum_kernel(const Args a) {
    const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int rows = a.kind == RESIDUAL_GATE_CHANNEL ? 3 : 2;
    if (j >= (int64_t)rows * a.n) return;
    float t = 0.f;
    for (int b = 0; b < a.blocks; ++b) t += a.partial[(int64_t)b * 3 * a.n + j];
    if (j < a.n)
        a.dw_post[j] = t;
    else if (j < 2 * (int64_t)a.n)
        a.dw_pre[j - a.n] = t;
    else
        static_cast<float *>(a.dgate)[j - 2 * (int64_t)a.n] = t;
}

bool aligned(const void *ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

int validate(const residual_rmsnorm_params *p, int dtype) {
    if (!p) return DGRAD_ERR_INVALID_ARG;
    if (dtype != DGRAD_F32 && dtype != DGRAD_BF16 && dtype != DGRAD_F16) return DGRAD_ERR_INVALID_ARG;
    if (p->gate_kind > RESIDUAL_GATE_ELEMENT || !std::isfinite(p->eps) || p->eps < 0.f || !std::isfinite(p->scale))
        return DGRAD_ERR_INVALID_ARG;
    if (p->m == 0 || p->n == 0) return DGRAD_ERR_SHAPE;
    if (p->n > kMaxN || p->m > (uint32_t)INT32_MAX) return DGRAD_ERR_UNSUPPORTED;
    return DGRAD_OK;
}

// Checks shared by both directions: all of `ptr` given and aligned to the element.
template <typename... P>
int check(const residual_rmsnorm_params *p, int dtype, const void *gate, const P *...ptr) {
    if (((ptr == nullptr) || ...)) return DGRAD_ERR_INVALID_ARG;
    const int v = validate(p, dtype);
    if (v != DGRAD_OK) return v;
    if ((p->gate_kind == RESIDUAL_GATE_NONE) != (gate == nullptr)) return DGRAD_ERR_INVALID_ARG;
    const uintptr_t e = dtype == DGRAD_F32 ? 4 : 2;
    return (aligned(ptr, e) && ...) && aligned(gate, e) ? DGRAD_OK : DGRAD_ERR_ALIGNMENT;
}

int blocks_of(const residual_rmsnorm_params *p) { return p->m < (uint32_t)kMaxBlocks ? (int)p->m : kMaxBlocks; }

size_t workspace_bytes_of(const residual_rmsnorm_params *p) {
    return (size_t)blocks_of(p) * 3 * p->n * sizeof(float);
}

template <typename T>
int forward_t(const Args &a, cudaStream_t st) {
    forward_row_kernel<T><<<a.m, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? DGRAD_OK : DGRAD_ERR_CUDA;
}

template <typename T>
int backward_t(const Args &a, cudaStream_t st) {
    backward_row_kernel<T><<<a.blocks, kThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return DGRAD_ERR_CUDA;
    const int64_t cols = (int64_t)(a.kind == RESIDUAL_GATE_CHANNEL ? 3 : 2) * a.n;
    partial_sum_kernel<<<(unsigned)((cols + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? DGRAD_OK : DGRAD_ERR_CUDA;
}

}  // namespace
}  // namespace rrms

extern "C" {

int residual_rmsnorm_forward(const void *f, const void *x, const void *gate, const void *w_post, const void *w_pre,
                             void *h, void *y, float *rstd, const residual_rmsnorm_params *p, int dtype,
                             struct CUstream_st *stream) {
    using namespace rrms;
    dgrad::NvtxRange range("residual_rmsnorm_forward");
    const int rc = check(p, dtype, gate, f, x, w_post, w_pre, static_cast<const void *>(h), static_cast<const void *>(y));
    if (rc != DGRAD_OK) return rc;
    if (!aligned(rstd, 4)) return DGRAD_ERR_ALIGNMENT;
    Args a{};
    a.f = f, a.x = x, a.gate = gate, a.w_post = w_post, a.w_pre = w_pre, a.h = h, a.y = y, a.rstd = rstd;
    a.m = (int)p->m, a.n = (int)p->n, a.kind = (int)p->gate_kind, a.eps = p->eps, a.scale = p->scale;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == DGRAD_F32) return forward_t<float>(a, st);
    if (dtype == DGRAD_BF16) return forward_t<__nv_bfloat16>(a, st);
    return forward_t<__half>(a, st);
}

size_t residual_rmsnorm_workspace_size(const residual_rmsnorm_params *p, int dtype) {
    return rrms::validate(p, dtype) == DGRAD_OK ? rrms::workspace_bytes_of(p) : 0;
}

int residual_rmsnorm_backward(const void *f, const void *h, const void *gate, const void *w_post, const void *w_pre,
                              const float *rstd, const void *dy, const void *dh, void *df, void *dx, void *dgate,
                              float *dw_post, float *dw_pre, void *workspace, size_t workspace_bytes,
                              const residual_rmsnorm_params *p, int dtype, struct CUstream_st *stream) {
    using namespace rrms;
    dgrad::NvtxRange range("residual_rmsnorm_backward");
    const int rc = check(p, dtype, gate, f, h, w_post, w_pre, dy, static_cast<const void *>(df),
                         static_cast<const void *>(dx));
    if (rc != DGRAD_OK) return rc;
    if (!rstd || !dw_post || !dw_pre || !workspace || (p->gate_kind == RESIDUAL_GATE_NONE) != (dgate == nullptr))
        return DGRAD_ERR_INVALID_ARG;
    const uintptr_t e = dtype == DGRAD_F32 ? 4 : 2;
    if (!aligned(rstd, 4) || !aligned(dw_post, 4) || !aligned(dw_pre, 4) || !aligned(workspace, 16) ||
        !aligned(dh, e) || !aligned(dgate, p->gate_kind == RESIDUAL_GATE_CHANNEL ? 4 : e))
        return DGRAD_ERR_ALIGNMENT;
    if (workspace_bytes < workspace_bytes_of(p)) return DGRAD_ERR_WORKSPACE;
    Args a{};
    a.f = f, a.h = const_cast<void *>(h), a.gate = gate, a.w_post = w_post, a.w_pre = w_pre;
    a.rstd = const_cast<float *>(rstd), a.dy = dy, a.dh = dh, a.df = df, a.dx = dx, a.dgate = dgate;
    a.dw_post = dw_post, a.dw_pre = dw_pre, a.partial = static_cast<float *>(workspace);
    a.m = (int)p->m, a.n = (int)p->n, a.kind = (int)p->gate_kind, a.eps = p->eps, a.scale = p->scale;
    a.blocks = blocks_of(p);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == DGRAD_F32) return backward_t<float>(a, st);
    if (dtype == DGRAD_BF16) return backward_t<__nv_bfloat16>(a, st);
    return backward_t<__half>(a, st);
}

}  // extern "C"
