// residual_rmsnorm.cu -- the residual step between two blocks (norm after a block,
// gate, scale, residual add, norm before the next block) and its gradients, declared
// in include/residual_rmsnorm.h.
//
// Both directions read each row once into registers or shared memory and write their
// results once; the floor is the bytes.  A row belongs to a team of 1 to 16 warps, each
// thread holding ITER pieces of it (16 bytes each, or single elements where n or a
// pointer does not allow 16-byte accesses); the two statistics of a row follow one
// another, each a shuffle reduction plus, for teams of several warps, one barrier of
// that team alone.
//
// Forward: a block of up to 512 threads takes one row per team and ends, so that several
// blocks per SM keep loads in flight while others reduce.
//
// Backward: one persistent block of 16 warps per SM, because the sums over rows (the
// weights' and the channel gate's gradients) stay in registers from row to row.  What
// covers the loads' latency is a ring of kRing / ITER rows per thread in shared memory, filled
// with cp.async: a thread copies and reads its own pieces only, so the ring needs no
// barrier.  At the end teams add up in a fixed order, each block writes one partial row,
// and a second kernel adds those in a fixed order.
//
// Rows too long for that (more than 512 threads x 4 pieces, x 2 in the 16-bit backward,
// x 8 single elements) take kernels that read the row again for each statistic.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "nvtx_range.h"
#include "residual_rmsnorm.h"

namespace rrms {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 152;  // of the backward: one for each SM
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

// ------------------------------------------------- rows held on the chip
__device__ __forceinline__ void team_barrier(int team, int warps) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * warps) : "memory");
}

// Sum over a team of `tw` warps; `red` [2][16] floats, `turn` alternates between its halves: when a half is written
// again, every thread of the team has passed the barrier after which nobody reads it.
__device__ __forceinline__ float team_sum(float x, float *red, int &turn, int tw, int warp) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (tw == 1) return x;
    float *r = red + 16 * turn;
    turn ^= 1;
    const int team = warp / tw, first = team * tw;
    if ((threadIdx.x & 31) == 0) r[warp] = x;
    team_barrier(team, tw);
    float t = 0.f;
    for (int w = 0; w < tw; ++w) t += r[first + w];
    return t;
}

// A piece of a row: V elements, 16 bytes or one element.
template <typename T, bool VEC>
struct Piece {
    static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
    using Raw = typename std::conditional<VEC, uint4, T>::type;
    Raw raw;
    __device__ __forceinline__ void load(const void *base, int64_t piece) {
        raw = __ldg(static_cast<const Raw *>(base) + piece);
    }
    __device__ __forceinline__ void zero() { raw = Raw{}; }
    __device__ __forceinline__ float get(int e) const { return to_f(reinterpret_cast<const T *>(&raw)[e]); }
};
template <typename T, bool VEC>
__device__ __forceinline__ void store_piece(void *base, int64_t piece, const float *x) {
    if constexpr (VEC) {
        uint4 w;
        T *t = reinterpret_cast<T *>(&w);
#pragma unroll
        for (int e = 0; e < 16 / (int)sizeof(T); ++e) t[e] = from_f<T>(x[e]);
        static_cast<uint4 *>(base)[piece] = w;
    } else {
        static_cast<T *>(base)[piece] = from_f<T>(x[0]);
    }
}

// pieces: of a row.  Thread `t` of a team holds pieces t, t + 32 tw, ...
template <typename T, int ITER, bool VEC>
__global__ void __launch_bounds__(512) forward_kernel(const Args a, int tw, int pieces) {
    using P = Piece<T, VEC>;
    __shared__ float red[32];
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, teams = (int)(blockDim.x >> 5) / tw, team = warp / tw;
    const int64_t row = (int64_t)blockIdx.x * teams + team;
    if (row >= a.m) return;  // the whole team
    const int t = (warp - team * tw) * 32 + (threadIdx.x & 31), step = 32 * tw;
    int turn = 0;
    const int64_t at = row * pieces;
    P f[ITER], x[ITER], wp[ITER], g[ITER], wq[ITER];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = t + i * step;
        if (c < pieces) {
            f[i].load(a.f, at + c), x[i].load(a.x, at + c);
            if (a.kind == RESIDUAL_GATE_ELEMENT) g[i].load(a.gate, at + c);
        } else {
            f[i].zero(), x[i].zero(), g[i].zero();
        }
    }
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = t + i * step;
        if (c < pieces) {
            wp[i].load(a.w_post, c), wq[i].load(a.w_pre, c);
            if (a.kind == RESIDUAL_GATE_CHANNEL) g[i].load(a.gate, c);
        } else {
            wp[i].zero(), wq[i].zero(), g[i].zero();
        }
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int e = 0; e < P::V; ++e) sum = fmaf(f[i].get(e), f[i].get(e), sum);
    const float rp = 1.0f / sqrtf(team_sum(sum, red, turn, tw, warp) / (float)a.n + a.eps);
    float h[ITER][P::V];
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int e = 0; e < P::V; ++e) {
            const float gate = a.kind == RESIDUAL_GATE_NONE ? 1.f : g[i].get(e);
            h[i][e] = fmaf(a.scale * gate, f[i].get(e) * rp * wp[i].get(e), x[i].get(e));
            sum = fmaf(h[i][e], h[i][e], sum);
        }
    const float rq = 1.0f / sqrtf(team_sum(sum, red, turn, tw, warp) / (float)a.n + a.eps);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = t + i * step;
        if (c >= pieces) continue;
        float y[P::V];
#pragma unroll
        for (int e = 0; e < P::V; ++e) y[e] = h[i][e] * rq * wq[i].get(e);
        store_piece<T, VEC>(a.h, at + c, h[i]);
        store_piece<T, VEC>(a.y, at + c, y);
    }
    if (t == 0 && a.rstd) a.rstd[2 * row] = rp, a.rstd[2 * row + 1] = rq;
}

// The backward's inputs of one row and piece: 0 f, 1 h, 2 dy, 3 dh, 4 gate (per element).
constexpr int kTensors = 5;
// The ring's rows times ITER: 160 KB of shared memory for 16-byte pieces of 512 threads.
constexpr int kRing = 4;

template <typename T, int ITER, bool VEC>
__global__ void __launch_bounds__(512, 1) backward_kernel(const Args a, int tw, int pieces) {
    using P = Piece<T, VEC>;
    constexpr int V = P::V, RING = VEC ? kRing / ITER : 1;
    extern __shared__ uint4 ring[];  // VEC: [stage][tensor][ITER][512]; then the teams' sums [3][n]
    __shared__ float red[32];
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, teams = 16 / tw, team = warp / tw;
    const int t = (warp - team * tw) * 32 + (threadIdx.x & 31), step = 32 * tw;
    const int64_t first = (int64_t)blockIdx.x * teams + team, stride = (int64_t)gridDim.x * teams;
    const bool channel = a.kind == RESIDUAL_GATE_CHANNEL, element = a.kind == RESIDUAL_GATE_ELEMENT;
    const void *src[kTensors] = {a.f, a.h, a.dy, a.dh, element ? a.gate : nullptr};
    int turn = 0;
    P wp[ITER], wq[ITER], gc[ITER], next[VEC ? 1 : kTensors][VEC ? 1 : ITER];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = t + i * step;
        wp[i].zero(), wq[i].zero(), gc[i].zero();
        if (c < pieces) {
            wp[i].load(a.w_post, c), wq[i].load(a.w_pre, c);
            if (channel) gc[i].load(a.gate, c);
        }
    }
    // Asks for a row: into the ring's slot (one cp.async group per row, empty past the last), or into registers.
    auto fetch = [&](int64_t row, int slot) {
#pragma unroll
        for (int k = 0; k < kTensors; ++k)
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
                const int c = t + i * step;
                const bool in = row < a.m && c < pieces && src[k];
                if constexpr (VEC) {
                    if (in) {
                        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(
                            ring + ((slot * kTensors + k) * ITER + i) * 512 + threadIdx.x);
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
                                     "l"(static_cast<const uint4 *>(src[k]) + row * pieces + c)
                                     : "memory");
                    }
                } else {
                    next[k][i].zero();
                    if (in) next[k][i].load(src[k], row * pieces + c);
                }
            }
        if constexpr (VEC) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float post[ITER][V], pre[ITER][V], gsum[ITER][V];
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) post[i][e] = pre[i][e] = gsum[i][e] = 0.f;
    float2 rstd_next = make_float2(0.f, 0.f);
    auto fetch_rstd = [&](int64_t row) {
        if (row < a.m) rstd_next = make_float2(__ldg(a.rstd + 2 * row), __ldg(a.rstd + 2 * row + 1));
    };
    if constexpr (VEC) {
#pragma unroll
        for (int s = 0; s < (RING > 1 ? RING - 1 : 1); ++s) fetch(first + s * stride, s);
    } else {
        fetch(first, 0);
    }
    fetch_rstd(first);
    int slot = 0;
    for (int64_t row = first; row < a.m; row += stride) {
        P cur[VEC ? 1 : kTensors][VEC ? 1 : ITER];
        if constexpr (VEC) {
            // Rows row .. row + RING - 2 strides are asked for; this one has landed when RING - 2 groups are pending.
            asm volatile("cp.async.wait_group %0;" ::"n"(RING > 2 ? RING - 2 : 0) : "memory");
        } else {
#pragma unroll
            for (int k = 0; k < kTensors; ++k)
#pragma unroll
                for (int i = 0; i < ITER; ++i) cur[k][i] = next[k][i];
        }
        const float rp = rstd_next.x, rq = rstd_next.y;
        // The slot that this fills was read in the last iteration, by this thread alone.
        if (!VEC || RING > 1) fetch(row + (VEC ? RING - 1 : 1) * stride, (slot + RING - 1) % RING);
        fetch_rstd(row + stride);
        auto piece = [&](int k, int i) {
            P p;
            if constexpr (VEC)
                p.raw = ring[((slot * kTensors + k) * ITER + i) * 512 + threadIdx.x];
            else
                p = cur[k][i];
            return p;
        };
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            if (t + i * step >= pieces) continue;
            const P h = piece(1, i), dy = piece(2, i);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float hy = dy.get(e) * h.get(e);
                sum = fmaf(wq[i].get(e), hy, sum);
                pre[i][e] = fmaf(hy, rq, pre[i][e]);
            }
        }
        const float c1 = rq * rq * (team_sum(sum, red, turn, tw, warp) / (float)a.n);
        float g[ITER][V];
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            if (t + i * step >= pieces) continue;
            const P h = piece(1, i), dy = piece(2, i), f = piece(0, i);
            P dh;
            dh.zero();
            if (a.dh) dh = piece(3, i);
            P gate = gc[i];
            if (element) gate = piece(4, i);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                g[i][e] = fmaf(rq, wq[i].get(e) * dy.get(e) - h.get(e) * c1, dh.get(e));
                const float u = a.scale * g[i][e], dz = a.kind == RESIDUAL_GATE_NONE ? u : u * gate.get(e);
                sum = fmaf(wp[i].get(e) * dz, f.get(e), sum);
            }
        }
        const float c2 = rp * rp * (team_sum(sum, red, turn, tw, warp) / (float)a.n);
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = t + i * step;
            if (c >= pieces) continue;
            const P f = piece(0, i);
            P gate = gc[i];
            if (element) gate = piece(4, i);
            float df[V], dg[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float u = a.scale * g[i][e], fn = f.get(e) * rp, w = wp[i].get(e);
                const float dz = a.kind == RESIDUAL_GATE_NONE ? u : u * gate.get(e);
                df[e] = rp * (w * dz - f.get(e) * c2);
                post[i][e] = fmaf(dz, fn, post[i][e]);
                dg[e] = u * fn * w;
                gsum[i][e] += dg[e];
            }
            store_piece<T, VEC>(a.df, row * pieces + c, df);
            store_piece<T, VEC>(a.dx, row * pieces + c, g[i]);
            if (element) store_piece<T, VEC>(a.dgate, row * pieces + c, dg);
        }
        if (VEC && RING == 1) fetch(row + stride, 0);  // the row is read: its place is the next one's
        slot = (slot + 1) % RING;
    }
    // One partial row per block, teams added in their order.
    float *part = a.partial + (int64_t)blockIdx.x * 3 * a.n, *all = reinterpret_cast<float *>(ring);
    if constexpr (VEC) asm volatile("cp.async.wait_group 0;" ::: "memory");
    for (int k = 0; k < teams; ++k) {
        __syncthreads();
        if (team != k) continue;
        float *dst = k == teams - 1 ? part : all;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = t + i * step;
            if (c >= pieces) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int j = c * V + e;
                dst[j] = post[i][e] + (k ? all[j] : 0.f);
                dst[a.n + j] = pre[i][e] + (k ? all[a.n + j] : 0.f);
                if (channel) dst[2 * a.n + j] = gsum[i][e] + (k ? all[2 * a.n + j] : 0.f);
            }
        }
    }
}

// --------------------------------------------------------------- long rows
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

// Columns of the blocks' partial rows added up: 32 columns per block, 8 warps taking every 8th row, then their sums in
// order.
__global__ void __launch_bounds__(kThreads) partial_sum_kernel(const Args a) {
    __shared__ float s[kThreads / 32][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t j = (int64_t)blockIdx.x * 32 + lane, cols = (int64_t)(a.kind == RESIDUAL_GATE_CHANNEL ? 3 : 2) * a.n;
    float t = 0.f;
    if (j < cols) {
#pragma unroll 8
        for (int b = warp; b < a.blocks; b += kThreads / 32) t += __ldcg(a.partial + (int64_t)b * 3 * a.n + j);
    }
    s[warp][lane] = t;
    __syncthreads();
    if (warp != 0 || j >= cols) return;
    t = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += s[w][lane];
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

// A launch that may start while the kernel before it ends (each kernel waits before it touches memory).
template <typename K, typename... A>
int launch(K kern, int64_t blocks, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? DGRAD_OK : DGRAD_ERR_CUDA;
}

// How a row of `pieces` is laid over a team: `warps` (a power of two up to 16) x 32 threads x `iter` pieces, as few
// pieces per thread as 16 warps allow but at least `least`; iter 0 when 4 pieces (8 single elements) do not reach.
struct Layout {
    int warps, iter;
};
Layout layout_of(int64_t pieces, int least, int most) {
    for (int it = least; it <= most; it *= 2)
        for (int w = 1; w <= 16; w *= 2)
            if (pieces <= (int64_t)32 * w * it) return {w, it};
    return {0, 0};
}

template <typename... P>
bool vector_applies(int n, size_t esize, const P *...ptr) {
    return (size_t)n * esize % 16 == 0 && (aligned(ptr, 16) && ...);
}

template <typename T, int ITER, bool VEC>
int forward_iter(const Args &a, int tw, int pieces, cudaStream_t st) {
    const int warps = tw < 8 ? 8 : tw, teams = warps / tw;
    return launch(forward_kernel<T, ITER, VEC>, ((int64_t)a.m + teams - 1) / teams, 32 * warps, 0, st, a, tw, pieces);
}

template <typename T>
int forward_t(const Args &a, cudaStream_t st) {
    const bool vec = vector_applies(a.n, sizeof(T), a.f, a.x, a.gate, a.w_post, a.w_pre, a.h, a.y);
    const int pieces = vec ? a.n * (int)sizeof(T) / 16 : a.n;
    const Layout l = layout_of(pieces, 1, vec ? 4 : 8);
    if (vec && l.iter == 1) return forward_iter<T, 1, true>(a, l.warps, pieces, st);
    if (vec && l.iter == 2) return forward_iter<T, 2, true>(a, l.warps, pieces, st);
    if (vec && l.iter == 4) return forward_iter<T, 4, true>(a, l.warps, pieces, st);
    if (l.iter == 1 || l.iter == 2) return forward_iter<T, 2, false>(a, l.warps, pieces, st);
    if (l.iter == 4 || l.iter == 8) return forward_iter<T, 8, false>(a, l.warps, pieces, st);
    forward_row_kernel<T><<<a.m, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? DGRAD_OK : DGRAD_ERR_CUDA;
}

template <typename T, int ITER, bool VEC>
int backward_iter(const Args &a, int tw, int pieces, cudaStream_t st) {
    const size_t ring = VEC ? (size_t)kRing * kTensors * 512 * 16 : 0;
    const size_t sums = tw < 16 ? (size_t)3 * a.n * sizeof(float) : 0, smem = std::max(ring, sums);
    auto kern = backward_kernel<T, ITER, VEC>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return DGRAD_ERR_CUDA;
    return launch(kern, a.blocks, 512, smem, st, a, tw, pieces);
}

template <typename T>
int backward_rows(Args &a, cudaStream_t st) {
    const void *dgate = a.kind == RESIDUAL_GATE_ELEMENT ? a.dgate : nullptr;
    const bool vec =
        vector_applies(a.n, sizeof(T), a.f, a.h, a.gate, a.w_post, a.w_pre, a.dy, a.dh, a.df, a.dx, dgate);
    const int pieces = vec ? a.n * (int)sizeof(T) / 16 : a.n;
    const Layout l = layout_of(pieces, 1, vec ? (sizeof(T) == 4 ? 4 : 2) : 8);
    if (l.iter) {
        const int64_t teams = 16 / l.warps, need = (a.m + teams - 1) / teams;
        a.blocks = need < a.blocks ? (int)need : a.blocks;
    }
    if (vec && l.iter == 1) return backward_iter<T, 1, true>(a, l.warps, pieces, st);
    if (vec && l.iter == 2) return backward_iter<T, 2, true>(a, l.warps, pieces, st);
    if constexpr (sizeof(T) == 4)
        if (vec && l.iter == 4) return backward_iter<T, 4, true>(a, l.warps, pieces, st);
    if (!vec && (l.iter == 1 || l.iter == 2)) return backward_iter<T, 2, false>(a, l.warps, pieces, st);
    if (!vec && (l.iter == 4 || l.iter == 8)) return backward_iter<T, 8, false>(a, l.warps, pieces, st);
    backward_row_kernel<T><<<a.blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? DGRAD_OK : DGRAD_ERR_CUDA;
}

template <typename T>
int backward_t(Args &a, cudaStream_t st) {
    const int rc = backward_rows<T>(a, st);
    if (rc != DGRAD_OK) return rc;
    const int64_t cols = (int64_t)(a.kind == RESIDUAL_GATE_CHANNEL ? 3 : 2) * a.n;
    return launch(partial_sum_kernel, (cols + 31) / 32, kThreads, 0, st, a);
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
