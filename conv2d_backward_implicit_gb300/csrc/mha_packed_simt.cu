// mha_packed_simt.cu -- CUDA-core kernels of causal attention over packed
// sequences (include/mha_packed.h): every type, any head_dim up to 256, float32
// throughout.
//
// Forward: one block of 256 threads per tile of 64 queries of one head.  Q stays in
// shared memory; the keys pass through in tiles of 64, K then V in one buffer.
// Thread (ty, tx) of a 16 x 16 grid owns queries 4 ty .. 4 ty + 3 and keys tx + 16 j
// of the scores, so a query's statistics live in the 16 lanes of a half-warp; its
// outputs are the same queries and elements 4 tx + 64 c .. + 3.  The running maximum
// and sum of the softmax make it one pass over the keys.
//
// Backward: one kernel for both directions of the pair of products, with resident
// rows R1, R2 and streamed rows X1, X2 (tile of 64, 32 for head_dim above 128):
//   s = R1 X1^T, dp = R2 X2^T, p and ds from the statistics,
//   acc1 += ds X1, and with keys resident also acc2 += p X2;
// queries resident (R = Q, dO; X = K, V) give dQ, keys resident (R = K, V; X = Q, dO,
// over the heads of the group) give dK and dV.  Scores are formed twice, which costs
// 7 products in place of 5 but needs no atomics: results do not change from run to run.
//
// A masked pair has p = ds = 0, and in tiles that the mask crosses its products are
// left out instead of multiplied by zero: infinities and NaN in rows that a query does
// not attend stay out of its results.
#include "mha_packed_internal.cuh"
#include "nvtx_range.h"

namespace mhapk {

__device__ unsigned int g_simt_error_word = 0;

unsigned take_simt_error(cudaError_t &e) {
    unsigned int word = 0;
    const unsigned int zero = 0;
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&word, g_simt_error_word, sizeof(word));
    if (e == cudaSuccess && word) e = cudaMemcpyToSymbol(g_simt_error_word, &zero, sizeof(zero));
    return word;
}

namespace {

constexpr int kThreads = 256;

// rows [r0, r0 + ROWS) of a [..][stride] tensor's head into shared memory as float32, zero past `live` rows and past hd.
template <typename T, int ROWS, int D>
__device__ __forceinline__ void load_tile(float *dst, const T *src, int64_t stride, int live, int hd) {
    constexpr int P = D + 4;
    constexpr int V = 16 / sizeof(T);  // elements of a 16-byte load
    if (hd % V == 0 && stride % V == 0 && (reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
        for (int e = threadIdx.x; e < ROWS * (D / V); e += kThreads) {
            const int r = e / (D / V), d = (e - r * (D / V)) * V;
            float x[V];
            if (r < live && d < hd) {
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(src + (int64_t)r * stride + d));
                const T *h = reinterpret_cast<const T *>(&w);
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = to_f(h[i]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < V; i += 4)
                *reinterpret_cast<float4 *>(dst + r * P + d + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        }
    } else {
        for (int e = threadIdx.x; e < ROWS * D; e += kThreads) {
            const int r = e / D, d = e - r * D;
            dst[r * P + d] = r < live && d < hd ? to_f(src[(int64_t)r * stride + d]) : 0.f;
        }
    }
}

// acc[i][j] += sum over d of a[RT ty + i][d] b[tx + 16 j][d].
template <int RT, int D>
__device__ __forceinline__ void score_tile(const float *a, const float *b, int ty, int tx, float (&acc)[RT][RT]) {
    constexpr int P = D + 4;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 x[RT], y[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) x[i] = *reinterpret_cast<const float4 *>(a + (RT * ty + i) * P + d);
#pragma unroll
        for (int j = 0; j < RT; ++j) y[j] = *reinterpret_cast<const float4 *>(b + (tx + 16 * j) * P + d);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
                acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
                acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
                acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
            }
    }
}

// acc[i][4 c ..] += sum over t of p[RT ty + i][t] x[t][4 tx + 64 c ..]; SKIP leaves out terms with p = 0.
template <int RT, int B, int D, bool SKIP>
__device__ __forceinline__ void add_tile(const float *p, const float *x, int ty, int tx, float (&acc)[RT][D / 16]) {
    constexpr int P = D + 4, PP = B + 4;
#pragma unroll 2
    for (int t = 0; t < B; t += 4) {
        float4 w[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) w[i] = *reinterpret_cast<const float4 *>(p + (RT * ty + i) * PP + t);
#pragma unroll
        for (int z = 0; z < 4; ++z)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const float4 y = *reinterpret_cast<const float4 *>(x + (t + z) * P + 4 * tx + 64 * c);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const float f = z == 0 ? w[i].x : z == 1 ? w[i].y : z == 2 ? w[i].z : w[i].w;
                    if (!SKIP || f != 0.f) {
                        acc[i][4 * c] = fmaf(f, y.x, acc[i][4 * c]);
                        acc[i][4 * c + 1] = fmaf(f, y.y, acc[i][4 * c + 1]);
                        acc[i][4 * c + 2] = fmaf(f, y.z, acc[i][4 * c + 2]);
                        acc[i][4 * c + 3] = fmaf(f, y.w, acc[i][4 * c + 3]);
                    }
                }
            }
    }
}

template <typename T, int RT, int D>
__device__ __forceinline__ void store_rows(T *dst, int64_t stride, int ty, int tx, int live, int hd,
                                           const float (&acc)[RT][D / 16], const float (&factor)[RT]) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int r = RT * ty + i;
        if (r >= live) continue;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int d = 4 * tx + 64 * c + z;
                if (d < hd) dst[(int64_t)r * stride + d] = from_f<T>(acc[i][4 * c + z] * factor[i]);
            }
    }
}

__device__ __forceinline__ float half_warp_max(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float half_warp_sum(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) forward_simt_kernel(const Args a) {
    constexpr int B = 64, RT = 4, P = D + 4, PP = B + 4;
    extern __shared__ float4 sm4[];
    float *sm = reinterpret_cast<float *>(sm4);
    float *q_s = sm, *x_s = q_s + B * P, *p_s = x_s + B * P;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int h = (int)(blockIdx.x % (unsigned)a.nh), g = h / a.hpk;
    const Unit u = find_unit(a, blockIdx.x / (unsigned)a.nh, 6, true, blockIdx.x == 0, &g_simt_error_word);
    if (!u.live) return;
    const int live = u.len - u.p0 < B ? u.len - u.p0 : B;
    const int64_t row0 = (int64_t)u.begin + u.p0;
    T *out = static_cast<T *>(a.out) + (row0 * a.nh + h) * a.hd;
    float acc[RT][D / 16];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
    float top[RT], sum[RT], factor[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) top[i] = -INFINITY, sum[i] = 0.f, factor[i] = 0.f;
    if (u.pad) {
        store_rows<T, RT, D>(out, (int64_t)a.nh * a.hd, ty, tx, live, a.hd, acc, factor);
        if (threadIdx.x < live) {
            float *l = a.lse + ((row0 + threadIdx.x) * a.nh + h) * 2;
            l[0] = 0.f, l[1] = INFINITY;
        }
        return;
    }
    load_tile<T, B, D>(q_s, static_cast<const T *>(a.q) + row0 * a.qs + (int64_t)h * a.hd, a.qs, live, a.hd);
    const int last = u.p0 + live - 1;
    int first = 0;
    if (a.window > 0 && u.p0 - a.window + 1 > 0) first = (u.p0 - a.window + 1) / B * B;
    for (int t0 = first; t0 <= last; t0 += B) {
        const int keys = u.len - t0 < B ? u.len - t0 : B;
        const int64_t t_row = (int64_t)u.begin + t0;
        __syncthreads();  // the last tile's V is read
        load_tile<T, B, D>(x_s, static_cast<const T *>(a.k) + t_row * a.ks + (int64_t)g * a.hd, a.ks, keys, a.hd);
        __syncthreads();
        float s[RT][RT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < RT; ++j) s[i][j] = 0.f;
        score_tile<RT, D>(q_s, x_s, ty, tx, s);
        const bool whole = t0 + B - 1 <= u.p0 && (a.window == 0 || u.p0 + B - 1 < t0 + a.window);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int pos = u.p0 + RT * ty + i;
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const int t = t0 + tx + 16 * j;
                const bool in = whole || (t <= pos && (a.window == 0 || pos - t < a.window));
                s[i][j] = in ? s[i][j] * a.scale : -INFINITY;
                m = fmaxf(m, s[i][j]);
            }
            m = half_warp_max(m);
            const float now = fmaxf(top[i], m);
            // A row whose keys so far are all masked keeps sum 0 and factor 1.
            const float keep = now == -INFINITY ? 1.f : expf(top[i] - now);
            float part = 0.f;
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const int t = t0 + tx + 16 * j;
                const bool in = whole || (t <= pos && (a.window == 0 || pos - t < a.window));
                const float e = in ? expf(s[i][j] - now) : 0.f;
                part += e;
                p_s[(RT * ty + i) * PP + tx + 16 * j] = e;
            }
            sum[i] = sum[i] * keep + half_warp_sum(part);
            top[i] = now;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) acc[i][c] *= keep;
        }
        __syncthreads();  // scores read K, and p is written
        load_tile<T, B, D>(x_s, static_cast<const T *>(a.v) + t_row * a.vs + (int64_t)g * a.hd, a.vs, keys, a.hd);
        __syncthreads();
        if (whole)
            add_tile<RT, B, D, false>(p_s, x_s, ty, tx, acc);
        else
            add_tile<RT, B, D, true>(p_s, x_s, ty, tx, acc);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        factor[i] = 1.0f / sum[i];
        if (tx == 0 && RT * ty + i < live) {
            float *l = a.lse + ((row0 + RT * ty + i) * a.nh + h) * 2;
            l[0] = top[i], l[1] = logf(sum[i]);
        }
    }
    store_rows<T, RT, D>(out, (int64_t)a.nh * a.hd, ty, tx, live, a.hd, acc, factor);
}

// delta = dO . O of every row and head into stats[h][row].y; one warp per row and head.
template <typename T>
__global__ void __launch_bounds__(kThreads) delta_simt_kernel(const Args a) {
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (w >= (int64_t)a.tokens * a.nh) return;
    const T *o = static_cast<const T *>(a.o) + w * a.hd, *go = static_cast<const T *>(a.go) + w * a.hd;
    float s = 0.f;
    for (int d = threadIdx.x & 31; d < a.hd; d += 32) s = fmaf(to_f(o[d]), to_f(go[d]), s);
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) a.stats[(w % a.nh) * a.tokens + w / a.nh].y = s;
}

template <typename T, int D, int B, bool KEYS>
__global__ void __launch_bounds__(kThreads) backward_simt_kernel(const Args a) {
    constexpr int RT = B / 16, P = D + 4, PP = B + 4;
    extern __shared__ float4 sm4[];
    float *sm = reinterpret_cast<float *>(sm4);
    float *r1 = sm, *r2 = r1 + B * P, *x1 = r2 + B * P, *x2 = x1 + B * P;
    float *ds_s = x2 + B * P, *p_s = ds_s + B * PP;  // p_s with KEYS only
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const unsigned heads = KEYS ? a.nkv : a.nh;
    const int head = (int)(blockIdx.x % heads), g = KEYS ? head : head / a.hpk;
    const Unit u = find_unit(a, blockIdx.x / heads, B == 64 ? 6 : 5, !KEYS, blockIdx.x == 0 && KEYS, &g_simt_error_word);
    if (!u.live) return;
    const int live = u.len - u.p0 < B ? u.len - u.p0 : B;
    const int64_t row0 = (int64_t)u.begin + u.p0;
    float acc1[RT][D / 16], acc2[RT][D / 16];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc1[i][c] = acc2[i][c] = 0.f;
    if (!u.pad) {
        if (KEYS) {
            load_tile<T, B, D>(r1, static_cast<const T *>(a.k) + row0 * a.ks + (int64_t)g * a.hd, a.ks, live, a.hd);
            load_tile<T, B, D>(r2, static_cast<const T *>(a.v) + row0 * a.vs + (int64_t)g * a.hd, a.vs, live, a.hd);
        } else {
            load_tile<T, B, D>(r1, static_cast<const T *>(a.q) + row0 * a.qs + (int64_t)head * a.hd, a.qs, live, a.hd);
            load_tile<T, B, D>(r2, static_cast<const T *>(a.go) + (row0 * a.nh + head) * a.hd, (int64_t)a.nh * a.hd,
                               live, a.hd);
        }
        // Streamed rows [lo, hi) of the sequence: the queries that reach these keys, or the keys these queries reach.
        int lo = 0, hi = u.p0 + live;
        if (KEYS) {
            lo = u.p0, hi = u.len;
            if (a.window > 0 && u.p0 + live - 1 < u.len - a.window) hi = u.p0 + live - 1 + a.window;
        } else if (a.window > 0 && u.p0 - a.window + 1 > 0) {
            lo = (u.p0 - a.window + 1) / B * B;
        }
        for (int c0 = lo; c0 < hi; c0 += B)
            for (int r = 0; r < (KEYS ? a.hpk : 1); ++r) {
                const int h = KEYS ? g * a.hpk + r : head;
                const int cols = u.len - c0 < B ? u.len - c0 : B;
                const int64_t c_row = (int64_t)u.begin + c0;
                __syncthreads();  // the last step's tiles are read
                if (KEYS) {
                    load_tile<T, B, D>(x1, static_cast<const T *>(a.q) + c_row * a.qs + (int64_t)h * a.hd, a.qs, cols,
                                       a.hd);
                    load_tile<T, B, D>(x2, static_cast<const T *>(a.go) + (c_row * a.nh + h) * a.hd,
                                       (int64_t)a.nh * a.hd, cols, a.hd);
                } else {
                    load_tile<T, B, D>(x1, static_cast<const T *>(a.k) + c_row * a.ks + (int64_t)g * a.hd, a.ks, cols,
                                       a.hd);
                    load_tile<T, B, D>(x2, static_cast<const T *>(a.v) + c_row * a.vs + (int64_t)g * a.hd, a.vs, cols,
                                       a.hd);
                }
                __syncthreads();
                float s[RT][RT], dp[RT][RT];
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < RT; ++j) s[i][j] = dp[i][j] = 0.f;
                score_tile<RT, D>(r1, x1, ty, tx, s);
                score_tile<RT, D>(r2, x2, ty, tx, dp);
                bool whole;
                if (KEYS)
                    whole = c0 >= u.p0 + B - 1 && cols == B && (a.window == 0 || c0 + B - 1 < u.p0 + a.window);
                else
                    whole = c0 + B - 1 <= u.p0 && (a.window == 0 || u.p0 + B - 1 < c0 + a.window);
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < RT; ++j) {
                        const int row = u.p0 + RT * ty + i, col = c0 + tx + 16 * j;
                        const int pos = KEYS ? col : row, t = KEYS ? row : col;
                        float p = 0.f, d = 0.f;
                        if (pos < u.len && t <= pos && (a.window == 0 || pos - t < a.window)) {
                            const int64_t at = (int64_t)u.begin + pos;
                            const float *l = a.lse_in + (at * a.nh + h) * 2;
                            p = expf(s[i][j] * a.scale - __ldg(l) - __ldg(l + 1));
                            d = p * (dp[i][j] - a.stats[(int64_t)h * a.tokens + at].y);
                        }
                        ds_s[(RT * ty + i) * PP + tx + 16 * j] = d;
                        if (KEYS) p_s[(RT * ty + i) * PP + tx + 16 * j] = p;
                    }
                __syncthreads();
                if (whole) {
                    add_tile<RT, B, D, false>(ds_s, x1, ty, tx, acc1);
                    if (KEYS) add_tile<RT, B, D, false>(p_s, x2, ty, tx, acc2);
                } else {
                    add_tile<RT, B, D, true>(ds_s, x1, ty, tx, acc1);
                    if (KEYS) add_tile<RT, B, D, true>(p_s, x2, ty, tx, acc2);
                }
            }
    }
    float one[RT], scaled[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) one[i] = 1.f, scaled[i] = a.scale;
    const int64_t stride = (int64_t)heads * a.hd, at = (row0 * heads + head) * a.hd;
    store_rows<T, RT, D>(static_cast<T *>(KEYS ? a.dk : a.dq) + at, stride, ty, tx, live, a.hd, acc1, scaled);
    if (KEYS) store_rows<T, RT, D>(static_cast<T *>(a.dv) + at, stride, ty, tx, live, a.hd, acc2, one);
}

// A kernel with its dynamic shared memory; raising the limit is per function and device and cheap to repeat.
template <typename K>
int launch(K kern, int64_t blocks, size_t smem, const Args &a, cudaStream_t st) {
    if (blocks > INT32_MAX) return DGRAD_ERR_UNSUPPORTED;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return DGRAD_ERR_CUDA;
    kern<<<(unsigned)blocks, kThreads, smem, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? DGRAD_OK : DGRAD_ERR_CUDA;
}

template <typename T, int D>
int forward_t(const Args &a, const mha_packed_params *p, cudaStream_t st) {
    const size_t smem = sizeof(float) * (2 * 64 * (D + 4) + 64 * 68);
    return launch(forward_simt_kernel<T, D>, unit_bound(p, 64) * a.nh, smem, a, st);
}

template <typename T, int D, int B>
int backward_t(const Args &a, const mha_packed_params *p, cudaStream_t st) {
    const size_t tiles = sizeof(float) * 4 * B * (D + 4), sq = sizeof(float) * B * (B + 4);
    int rc = launch(delta_simt_kernel<T>, ((int64_t)a.tokens * a.nh + kThreads / 32 - 1) / (kThreads / 32), 0, a, st);
    if (rc == DGRAD_OK)
        rc = launch(backward_simt_kernel<T, D, B, true>, unit_bound(p, B) * a.nkv, tiles + 2 * sq, a, st);
    if (rc == DGRAD_OK) rc = launch(backward_simt_kernel<T, D, B, false>, unit_bound(p, B) * a.nh, tiles + sq, a, st);
    return rc;
}

template <typename T>
int forward_d(const Args &a, const mha_packed_params *p, cudaStream_t st) {
    if (a.hd <= 64) return forward_t<T, 64>(a, p, st);
    if (a.hd <= 128) return forward_t<T, 128>(a, p, st);
    return forward_t<T, 256>(a, p, st);
}
template <typename T>
int backward_d(const Args &a, const mha_packed_params *p, cudaStream_t st) {
    if (a.hd <= 64) return backward_t<T, 64, 64>(a, p, st);
    if (a.hd <= 128) return backward_t<T, 128, 64>(a, p, st);
    return backward_t<T, 256, 32>(a, p, st);
}

}  // namespace

int forward_simt(const Args &a, const mha_packed_params *p, int dtype, cudaStream_t st) {
    if (dtype == DGRAD_F32) return forward_d<float>(a, p, st);
    if (dtype == DGRAD_BF16) return forward_d<__nv_bfloat16>(a, p, st);
    return forward_d<__half>(a, p, st);
}

int backward_simt(const Args &a, const mha_packed_params *p, int dtype, cudaStream_t st) {
    if (dtype == DGRAD_F32) return backward_d<float>(a, p, st);
    if (dtype == DGRAD_BF16) return backward_d<__nv_bfloat16>(a, p, st);
    return backward_d<__half>(a, p, st);
}

}  // namespace mhapk
