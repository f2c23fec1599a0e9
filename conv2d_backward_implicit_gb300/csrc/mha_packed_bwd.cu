// mha_packed_bwd.cu -- tensor-core backward of causal attention over packed
// sequences (include/mha_packed.h): bf16 / fp16, head_dim a multiple of 8 up to 128
// (padded to D = 64 or 128 by the TMA copies' zero fill), sm_103a.
//
// Two launches.  The first makes, per head and position, the folded statistic
// (m + l) log2(e) and delta = dO . O.  The second has one block per work unit of
// 128 resident rows, of two kinds with one body:
//   keys resident (R1 = K, R2 = V; streamed X1 = Q, X2 = dO, over the query blocks that
//   reach them and the heads of the group):  dK = acc1, dV = acc2;
//   queries resident (R1 = Q, R2 = dO; streamed X1 = K, X2 = V):  dQ = acc1.
// For every step of 64 streamed rows (columns below):
//   S = R1 X1^T, G = R2 X2^T      tcgen05 M128 N64 K16, D / 16 steps each
//   P = 2^(S c - stat), dS = P (G - delta), masked, rounded to 16 bits
//   acc1 += dS X1, acc2 += P X2   tcgen05 M128 N(D) K16, 4 steps each, P and dS from
//                                 tensor memory, X as the MN-major operand
// so scores are formed twice (7 products in place of 5), and in return every gradient
// is one block's sum in a fixed order: no atomics, nothing to zero or convert after.
// Tensor memory: acc1 and acc2 (D columns each), and a ring of two (D = 128) or three
// buffers of S and G (64 columns each, P and dS over the first 16 of each 32).
//   * warps 0-7 and 8-15: P and dS of the even and the odd steps, half a resident row
//     (32 columns) per thread; at the end dK / dQ and dV;
//   * warp 16 (converged, lane 0 issuing): S and G of each step, as far ahead as the ring
//     has buffers; warp 17: acc of each step whose P and dS are written.  Two warps,
//     because a warp's waits and commits (about 750 cycles a step) otherwise stand
//     between its products;
//   * warp 18 (one thread): TMA copies of X1 and X2 (128 rows a copy, two steps) and of R1
//     and R2;
//   * warp 19: with keys resident, the statistics of each step's 64 queries.
// fp16 has 5 exponent bits: P is scaled by 2^13 (P <= 1) and dS by the power of two
// that brings 2 max|dO| max|V| (row norms; |dP - delta| cannot be larger) to 2^15 at
// most, both taken out of the sums at the end; the two maxima come from the first launch.
// Streamed rows past the sequence's end are zeroed in shared memory; where a masked row
// inside the sequence is not finite, the product with 0 leaves a NaN in the sums and the
// tile is recomputed row by row over the attended pairs alone.
// Every wait is bounded, as in the forward.
#include "mha_packed_tc.cuh"

namespace mhapk {

__device__ unsigned int g_bwd_error_word = 0;

unsigned take_bwd_error(cudaError_t &e) {
    unsigned int word = 0;
    const unsigned int zero = 0;
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&word, g_bwd_error_word, sizeof(word));
    if (e == cudaSuccess && word) e = cudaMemcpyToSymbol(g_bwd_error_word, &zero, sizeof(zero));
    return word;
}

namespace {

constexpr int kRows = 128;           // resident rows, rows of a streamed copy
constexpr int kCols = 64;            // streamed rows of a step
constexpr uint32_t kHalf = kRows * 128;
constexpr int kSoftWarps = 16, kMmaWarp = 16, kLoadWarp = 18, kStatWarp = 19;
constexpr int kThreads = 32 * 20;
constexpr int kStatSlots = 4;
constexpr uint32_t kStatBytes = kCols * 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 13.0f;     // log2 of fp16's scale of P

template <int D>
struct Cfg {
    static constexpr int kHalves = D / 64;
    static constexpr uint32_t kTile = kHalf * kHalves;
    static constexpr int kStages = D == 64 ? 4 : 2;
    static constexpr int kBufs = D == 64 ? 3 : 2;  // of S and G
    static constexpr uint32_t kColAcc1 = 0, kColAcc2 = D, kColS = 2 * D, kColG = kColS + 64 * kBufs;  // + 64 per buffer
    static constexpr uint32_t kOffStat = 1024, kOffR = kOffStat + kStatSlots * kStatBytes + 1024;
    static constexpr uint32_t kOffX1 = kOffR + 2 * kTile, kOffX2 = kOffX1 + kStages * kTile;
    static constexpr uint32_t kSmem = 1024 + kOffX2 + kStages * kTile;  // + 1 KB alignment slack
    static_assert(kOffR % 1024 == 0, "operand tiles must be 1 KB aligned");
    static_assert(kSmem + 1024 <= 232448, "shared memory over the per-block limit");
};

struct BwdArgs {
    Args a;
    CUtensorMap q_map, k_map, v_map, go_map;
    const unsigned *norms;  // fp16: bits of max |dO row|^2, max |V row|^2
    int64_t key_units;      // blocks [0, key_units) have keys resident
    uint32_t idesc1, idesc2;
};

struct Ctl {
    uint64_t r_full, x_full[4], x_empty[4], st_full[kStatSlots], st_empty[kStatSlots];
    uint64_t s_full[3], g_full[3], p_ready[3], free[3], acc_full, mma_done[2];
    uint32_t tmem_base;
    int abort_flag, bad;
};
static_assert(sizeof(Ctl) <= 1024, "control block too large");

// The streamed rows [lo, hi) of a unit, in copies of 128 and steps of 64; `heads`: query heads per copy position.
struct Walk {
    int lo, hi, heads;
    __device__ __forceinline__ int copies() const { return (hi - lo + kRows - 1) / kRows; }
    __device__ __forceinline__ int steps(int c0) const { return hi - c0 > kCols ? 2 : 1; }
};

template <bool KEYS>
__device__ __forceinline__ Walk walk_of(const Args &a, const Unit &u, int live) {
    Walk w;
    if (KEYS) {
        w.lo = u.p0;
        w.hi = u.len;
        if (a.window > 0 && u.p0 + live - 1 < u.len - a.window) w.hi = u.p0 + live - 1 + a.window;
        w.heads = a.hpk;
    } else {
        w.lo = a.window > 0 && u.p0 - a.window + 1 > 0 ? (u.p0 - a.window + 1) / kCols * kCols : 0;
        w.hi = u.p0 + live;
        w.heads = 1;
    }
    return w;
}

// The scale of dS (a power of two): 1 for bf16.
template <bool F16>
__device__ __forceinline__ float ds_scale(const BwdArgs &p) {
    if constexpr (!F16) return 1.f;
    const float bound = 2.0f * sqrtf(__uint_as_float(p.norms[0])) * sqrtf(__uint_as_float(p.norms[1]));
    if (!(bound > 0.f)) return 1.f;
    // bound <= 2^e, so bound * 2^(15 - e) <= 2^15; kept where the scale and its inverse are normal floats.
    int e = (int)((__float_as_uint(bound) >> 23) & 255u) - 126;
    e = 15 - e;
    e = e > 100 ? 100 : (e < -100 ? -100 : e);
    return __uint_as_float((uint32_t)(127 + e) << 23);
}

// ------------------------------------------------------------ first launch
// One warp per head and run of 32 positions: G = hd / 8 lanes (a power of two at least that) take a row's 16-byte pieces.
template <typename T>
__global__ void __launch_bounds__(256) stats_kernel(const Args a, unsigned *norms, int group) {
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr bool F16 = std::is_same<T, __half>::value;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int runs = (a.tokens + 31) / 32;
    const int64_t own = (int64_t)runs * a.nh;
    const int piece = lane % group, sub = lane / group, per = 32 / group;
    const bool has = piece * 8 < a.hd;
    const int first = F16 ? clamp_row(a.off[0], a.tokens) : 0, last = F16 ? clamp_row(a.off[a.seqs], a.tokens) : 0;
    if (w < own) {
        const int h = (int)(w % a.nh), t0 = (int)(w / a.nh) * 32;
        float mine = 0.f, norm = 0.f;
#pragma unroll 4
        for (int r = 0; r < 32; r += per) {
            const int t = t0 + r + sub;
            float s = 0.f, n = 0.f;
            if (has && t < a.tokens) {
                const int64_t at = ((int64_t)t * a.nh + h) * a.hd + piece * 8;
                const uint4 x = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.o) + at));
                const uint4 y = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.go) + at));
                const T *xs = reinterpret_cast<const T *>(&x), *ys = reinterpret_cast<const T *>(&y);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s = fmaf(to_f(xs[i]), to_f(ys[i]), s);
                    if (F16) n = fmaf(to_f(ys[i]), to_f(ys[i]), n);
                }
            }
            for (int o = group / 2; o > 0; o >>= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, o);
                if (F16) n += __shfl_xor_sync(0xffffffffu, n, o);
            }
            const float got = __shfl_sync(0xffffffffu, s, ((lane - r) & (per - 1)) * group);
            if (lane >= r && lane < r + per) mine = got;
            if (F16 && t >= first && t < last && finite(n)) norm = fmaxf(norm, n);
        }
        const int t = t0 + lane;
        if (t < a.tokens) {
            const float *l = a.lse_in + ((int64_t)t * a.nh + h) * 2;
            a.stats[(int64_t)h * a.tokens + t] = make_float2((l[0] + l[1]) * kLog2e, mine);
        }
        if (F16) {
            for (int o = 16; o > 0; o >>= 1) norm = fmaxf(norm, __shfl_xor_sync(0xffffffffu, norm, o));
            if (lane == 0) atomicMax(norms, __float_as_uint(norm));
        }
    } else if (F16) {  // V's rows, for their largest norm
        const int64_t x = w - own;
        const int g = (int)(x % a.nkv);
        if (x / a.nkv >= runs) return;
        const int t0 = (int)(x / a.nkv) * 32;
        float norm = 0.f;
#pragma unroll 4
        for (int r = 0; r < 32; r += per) {
            const int t = t0 + r + sub;
            float n = 0.f;
            if (has && t < a.tokens) {
                const uint4 y = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.v) + (int64_t)t * a.vs +
                                                                      (int64_t)g * a.hd + piece * 8));
                const T *ys = reinterpret_cast<const T *>(&y);
#pragma unroll
                for (int i = 0; i < 8; ++i) n = fmaf(to_f(ys[i]), to_f(ys[i]), n);
            }
            for (int o = group / 2; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
            if (t >= first && t < last && finite(n)) norm = fmaxf(norm, n);
        }
        for (int o = 16; o > 0; o >>= 1) norm = fmaxf(norm, __shfl_xor_sync(0xffffffffu, norm, o));
        if (lane == 0) atomicMax(norms + 1, __float_as_uint(norm));
    }
}

// ----------------------------------------------------------- second launch
// The loading thread: R1 and R2, then X1 and X2 of every ring slot.
template <int D, bool KEYS>
__device__ void role_load(const BwdArgs &p, Ctl &c, uint32_t smem, const Unit &u, const Walk &k, int head, int g,
                          const Waiter &w) {
    using C = Cfg<D>;
    const CUtensorMap *r1 = KEYS ? &p.k_map : &p.q_map, *r2 = KEYS ? &p.v_map : &p.go_map;
    const CUtensorMap *x1 = KEYS ? &p.q_map : &p.k_map, *x2 = KEYS ? &p.go_map : &p.v_map;
    load_rows<D>(smem + C::kOffR, r1, p.a.hd, head, u.begin + u.p0, kRows, su32(&c.r_full));
    load_rows<D>(smem + C::kOffR + C::kTile, r2, p.a.hd, head, u.begin + u.p0, kRows, su32(&c.r_full));
    const int n = k.copies();
    int it = 0;
    bool ok = true;
    for (int b = 0; b < n && ok; ++b)
        for (int r = 0; r < k.heads; ++r, ++it) {
            const int s = it % C::kStages, h = KEYS ? g * p.a.hpk + r : g, row = u.begin + k.lo + kRows * b;
            if (!wait(su32(&c.x_empty[s]), (uint32_t)(((it / C::kStages) & 1) ^ 1), w)) {
                ok = false;
                break;
            }
            load_rows<D>(smem + C::kOffX1 + (uint32_t)s * C::kTile, x1, p.a.hd, h, row, kRows, su32(&c.x_full[s]));
            load_rows<D>(smem + C::kOffX2 + (uint32_t)s * C::kTile, x2, p.a.hd, h, row, kRows, su32(&c.x_full[s]));
        }
    // Copies still landing must finish before the block exits.
    drain(su32(&c.r_full), 0, w);
    for (int q = it > C::kStages ? it - C::kStages : 0; q < it; ++q)
        drain(su32(&c.x_full[q % C::kStages]), (uint32_t)((q / C::kStages) & 1), w);
}

// Statistics of each step's 64 queries: per pair of columns (-stat, -stat, -delta, -delta).
template <bool F16>
__device__ void role_stats(const BwdArgs &p, Ctl &c, uint32_t smem, const Unit &u, const Walk &k, int g, float kappa,
                           int lane, const Waiter &w) {
    const int n = k.copies();
    int step = 0;
    for (int b = 0; b < n; ++b)
        for (int r = 0; r < k.heads; ++r) {
            const int c0 = k.lo + kRows * b, ns = k.steps(c0);
            const float2 *st = p.a.stats + (int64_t)(g * p.a.hpk + r) * p.a.tokens + u.begin;
            for (int s = 0; s < ns; ++s, ++step) {
                const int slot = step % kStatSlots, col = c0 + kCols * s + 2 * lane;
                const float2 x = col < u.len ? __ldg(st + col) : make_float2(0.f, 0.f);
                const float2 y = col + 1 < u.len ? __ldg(st + col + 1) : make_float2(0.f, 0.f);
                if (!wait_warp(su32(&c.st_empty[slot]), (uint32_t)(((step / kStatSlots) & 1) ^ 1), w)) return;
                const float shift = F16 ? kPShift : 0.f;
                sts128(smem + 1024u + (uint32_t)slot * kStatBytes + (uint32_t)lane * 16u, __float_as_uint(shift - x.x),
                       __float_as_uint(shift - y.x), __float_as_uint(-x.y * kappa), __float_as_uint(-y.y * kappa));
                __syncwarp();
                if (lane == 0) bar_arrive(su32(&c.st_full[slot]));
            }
        }
}

// The ring walk of one product warp: visit(slot, half, step, first use of the slot, last use, first row of the copy)
// for every step, until it returns false.
template <int STAGES, typename F>
__device__ __forceinline__ bool for_steps(const Walk &k, F visit) {
    const int n = k.copies();
    int it = 0, step = 0;
    for (int b = 0; b < n; ++b)
        for (int r = 0; r < k.heads; ++r, ++it) {
            const int c0 = k.lo + kRows * b, ns = k.steps(c0);
            for (int s = 0; s < ns; ++s, ++step)
                if (!visit(it % STAGES, (uint32_t)((it / STAGES) & 1), s, step, s == 0, s == ns - 1, c0)) return false;
        }
    return true;
}

// S and G of every step, into the next buffer once the sums have read what it held.
template <int D, bool KEYS>
__device__ __forceinline__ void issue_scores(const BwdArgs &p, Ctl &c, uint32_t smem, uint32_t tmem, int seq_end,
                                             const Walk &k, int lane, const Waiter &w) {
    using C = Cfg<D>;
    const uint32_t leader = lane == 0;
    const uint64_t r1 = desc_k(smem + C::kOffR), r2 = desc_k(smem + C::kOffR + C::kTile);
    if (!wait_warp(su32(&c.r_full), 0, w)) return;
    for_steps<C::kStages>(k, [&](int slot, uint32_t phase, int s, int step, bool fresh, bool, int c0) {
        const int buf = step % C::kBufs;
        if (fresh) {
            if (!wait_warp(su32(&c.x_full[slot]), phase, w)) return false;
            if (seq_end - c0 < kRows) {
                zero_rows(smem + C::kOffX1 + (uint32_t)slot * C::kTile, seq_end - c0, kRows, C::kHalves, lane);
                if (KEYS) zero_rows(smem + C::kOffX2 + (uint32_t)slot * C::kTile, seq_end - c0, kRows, C::kHalves, lane);
            }
        }
        if (!wait_warp(su32(&c.free[buf]), (uint32_t)(((step / C::kBufs) & 1) ^ 1), w)) return false;
        tc_after();
        const uint32_t at = (uint32_t)slot * C::kTile + (uint32_t)s * (kCols * 128u);
        const uint64_t x1 = desc_k(smem + C::kOffX1 + at), x2 = desc_k(smem + C::kOffX2 + at);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const uint64_t off = 2u * (i % 4) + (uint64_t)(i / 4) * (kHalf >> 4);
            tc_mma_f16_if(tmem + C::kColS + 64u * buf, r1 + off, x1 + off, p.idesc1, i > 0, leader);
        }
        tc_commit_to_if(su32(&c.s_full[buf]), leader);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const uint64_t off = 2u * (i % 4) + (uint64_t)(i / 4) * (kHalf >> 4);
            tc_mma_f16_if(tmem + C::kColG + 64u * buf, r2 + off, x2 + off, p.idesc1, i > 0, leader);
        }
        tc_commit_to_if(su32(&c.g_full[buf]), leader);
        return true;
    });
}

// acc1 += dS X1 and acc2 += P X2 of every step.
template <int D, bool KEYS>
__device__ __forceinline__ void issue_sums(const BwdArgs &p, Ctl &c, uint32_t smem, uint32_t tmem, const Walk &k,
                                           int lane, const Waiter &w) {
    using C = Cfg<D>;
    const uint32_t leader = lane == 0;
    const bool done = for_steps<C::kStages>(k, [&](int slot, uint32_t, int s, int step, bool, bool last, int) {
        const int buf = step % C::kBufs;
        if (!wait_warp(su32(&c.p_ready[buf]), (uint32_t)((step / C::kBufs) & 1), w)) return false;
        tc_after();
        const uint32_t at = (uint32_t)slot * C::kTile + (uint32_t)s * (kCols * 128u);
        const uint64_t x1 = desc_mn(smem + C::kOffX1 + at, kHalf, 1024u), x2 = desc_mn(smem + C::kOffX2 + at, kHalf, 1024u);
        if (KEYS) {
#pragma unroll
            for (int i = 0; i < kCols / 16; ++i)
                tc_mma_f16_ts_if(tmem + C::kColAcc2, tmem + C::kColS + 64u * buf + 32u * (i / 2) + 8u * (i % 2),
                                 x2 + 128u * i, p.idesc2, step > 0 || i > 0, leader);
        }
#pragma unroll
        for (int i = 0; i < kCols / 16; ++i)
            tc_mma_f16_ts_if(tmem + C::kColAcc1, tmem + C::kColG + 64u * buf + 32u * (i / 2) + 8u * (i % 2),
                             x1 + 128u * i, p.idesc2, step > 0 || i > 0, leader);
        tc_commit_to_if(su32(&c.free[buf]), leader);
        if (last) tc_commit_to_if(su32(&c.x_empty[slot]), leader);
        return true;
    });
    if (done) tc_commit_to_if(su32(&c.acc_full), leader);
}

// P and dS of 32 columns.  s, g: this row's scores and dP; columns outside [from, to] are masked when MASK.  With
// KEYS the statistics are per column at shared address `st`, else (nl, nd) of the row.
template <bool F16, bool KEYS, bool MASK>
__device__ __forceinline__ void grad32(const uint32_t (&s)[32], const uint32_t (&g)[32], float cs, float kappa,
                                       uint32_t st, float nl, float nd, int from, int to, uint32_t (&pp)[16],
                                       uint32_t (&pd)[16]) {
    const float2 c2 = make_float2(cs, cs), k2 = make_float2(kappa, kappa);
    float2 l2 = make_float2(nl, nl), d2 = make_float2(nd, nd);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        if (KEYS) {
            const uint4 x = lds128(st + (uint32_t)e * 8u);
            l2 = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
            d2 = make_float2(__uint_as_float(x.z), __uint_as_float(x.w));
        }
        const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, l2);
        float2 y = make_float2(fast_exp2(x.x), fast_exp2(x.y));
        const float2 z = __ffma2_rn(make_float2(__uint_as_float(g[e]), __uint_as_float(g[e + 1])), k2, d2);
        float2 d = __fmul2_rn(y, z);
        if (MASK) {
            if (e < from || e > to) y.x = 0.f, d.x = 0.f;
            if (e + 1 < from || e + 1 > to) y.y = 0.f, d.y = 0.f;
        }
        if (KEYS) pp[e >> 1] = pack2<F16>(y.x, y.y);
        pd[e >> 1] = pack2<F16>(d.x, d.y);
    }
}

// W columns of 32 rows from tensor memory, times `factor`, through this warp's staging rows to dst (a row every
// `stride` elements; `cols` of the columns exist).  Returns whether this lane's row is finite.
template <int W, bool F16>
__device__ __forceinline__ bool store_acc(uint32_t acc_tm, uint32_t stage, float factor, uint16_t *dst, int64_t stride,
                                          int live, int cols, int lane) {
    constexpr int kChunks = W / 8;  // 16-byte chunk j of row r lies at j ^ (r & 7), of 64-byte rows at j ^ (r / 2 & 3)
    auto place = [](int r, int j) { return (uint32_t)((kChunks == 4 ? j ^ ((r >> 1) & 3) : j ^ (r & 7)) << 4); };
    bool good = true;
#pragma unroll
    for (int k = 0; k < W / 32; ++k) {
        uint32_t o[32];
        tc_ld_32x32(acc_tm + 32 * k, o);
        tc_wait_ld(o);
        float x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            x[e] = __uint_as_float(o[e]) * factor;
            good = good && finite(x[e]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sts128(stage + (uint32_t)lane * (2 * W) + place(lane, 4 * k + j), pack2<F16>(x[8 * j], x[8 * j + 1]),
                   pack2<F16>(x[8 * j + 2], x[8 * j + 3]), pack2<F16>(x[8 * j + 4], x[8 * j + 5]),
                   pack2<F16>(x[8 * j + 6], x[8 * j + 7]));
    }
    __syncwarp();
    const int j = lane % kChunks;
    for (int r = lane / kChunks; r < 32; r += 32 / kChunks) {
        if (r >= live || 8 * j >= cols) continue;
        const uint4 x = lds128(stage + (uint32_t)r * (2 * W) + place(r, j));
        *reinterpret_cast<uint4 *>(dst + (int64_t)r * stride + 8 * j) = x;
    }
    return good;
}

template <int D, bool F16, bool KEYS>
__device__ void role_soft(const BwdArgs &p, Ctl &c, uint32_t smem, uint32_t tmem, const Unit &u, const Walk &k, int live,
                          int head, float sigma, int warp, int lane, const Waiter &w) {
    using C = Cfg<D>;
    const Args &a = p.a;
    const int quad = warp & 3, part = (warp >> 2) & 1, grp = warp >> 3, row = u.p0 + 32 * quad + lane;
    const uint32_t lane_tm = (uint32_t)(32 * quad) << 16;
    const float cs = a.scale * kLog2e, kappa = F16 ? sigma * 0x1p-13f : 1.f;
    float nl = 0.f, nd = 0.f;
    if (!KEYS && row < u.len) {
        const float2 st = __ldg(a.stats + (int64_t)head * a.tokens + u.begin + row);
        nl = (F16 ? kPShift : 0.f) - st.x, nd = -st.y * kappa;
    }
    const int n = k.copies();
    int step = 0;
    for (int b = 0; b < n; ++b) {
        const int c0 = k.lo + kRows * b, ns = k.steps(c0);
        for (int r = 0; r < k.heads; ++r)
            for (int s = 0; s < ns; ++s, ++step) {
                if ((step & 1) != grp) continue;
                const int base = c0 + kCols * s + 32 * part, slot = step % kStatSlots, buf = step % C::kBufs;
                const uint32_t phase = (uint32_t)((step / C::kBufs) & 1);
                const uint32_t s_tm = tmem + lane_tm + C::kColS + 64u * buf, g_tm = tmem + lane_tm + C::kColG + 64u * buf;
                int from, to;
                bool whole;
                if (KEYS) {
                    from = row - base;
                    int end = u.len;
                    if (a.window > 0 && row < u.len - a.window) end = row + a.window;
                    to = end - 1 - base;
                    whole = base >= u.p0 + kRows - 1 && base + 32 <= u.len &&
                            (a.window == 0 || base + 31 < u.p0 + a.window);
                    if (!wait_warp(su32(&c.st_full[slot]), (uint32_t)((step / kStatSlots) & 1), w)) return;
                } else {
                    from = a.window > 0 ? row - a.window + 1 - base : 0;
                    to = row - base;
                    whole = base + 31 <= u.p0 && (a.window == 0 || u.p0 + kRows - 1 < base + a.window);
                }
                uint32_t sv[32], gv[32], pp[16], pd[16];
                if (!wait_warp(su32(&c.s_full[buf]), phase, w)) return;
                tc_after();
                tc_ld_32x32(s_tm + 32 * part, sv);
                if (!wait_warp(su32(&c.g_full[buf]), phase, w)) return;
                tc_after();
                tc_ld_32x32(g_tm + 32 * part, gv);
                tc_wait_ld(sv);
                tc_wait_ld(gv);
                // The warp of the other 32 columns may still read its half of S and G: P and dS (16 columns) go over
                // this warp's own half.
                const uint32_t st = smem + 1024u + (uint32_t)slot * kStatBytes + 256u * part;
                if (whole)
                    grad32<F16, KEYS, false>(sv, gv, cs, kappa, st, nl, nd, 0, 0, pp, pd);
                else
                    grad32<F16, KEYS, true>(sv, gv, cs, kappa, st, nl, nd, from, to, pp, pd);
                if (KEYS) tc_st_32x16(s_tm + 32 * part, pp);
                tc_st_32x16(g_tm + 32 * part, pd);
                tc_wait_st();
                tc_before();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(su32(&c.p_ready[buf]));
                    if (KEYS) bar_arrive(su32(&c.st_empty[slot]));
                }
            }
    }
    if (!wait_warp(su32(&c.acc_full), 0, w)) return;
    tc_after();
    // The resident tiles are read by now: group 0 stages dK or dQ in R1, group 1 dV in R2, half of the columns a warp.
    if (!KEYS && grp == 1) return;
    constexpr int W = D / 2;
    const int heads = KEYS ? a.nkv : a.nh;
    const int64_t stride = (int64_t)heads * a.hd;
    const int64_t at = (((int64_t)u.begin + u.p0 + 32 * quad) * heads + head) * a.hd + W * part;
    const float factor = grp == 0 ? a.scale / sigma : (F16 ? 0x1p-13f : 1.f);
    uint16_t *dst = static_cast<uint16_t *>(grp == 0 ? (KEYS ? a.dk : a.dq) : a.dv) + at;
    const uint32_t stage = smem + C::kOffR + (uint32_t)grp * C::kTile + (uint32_t)(warp & 7) * (C::kTile / 8);
    const bool good = store_acc<W, F16>(tmem + lane_tm + (grp == 0 ? C::kColAcc1 : C::kColAcc2) + W * part, stage, factor,
                                        dst, stride, live - 32 * quad, a.hd - W * part, lane);
    if (__any_sync(0xffffffffu, row < u.len && !good) && lane == 0) c.bad = 1;
}

// The unit's rows one by one over the attended pairs alone, one warp per row.
template <int D, bool F16, bool KEYS>
__device__ __noinline__ void recompute(const Args &a, const Unit &u, int live, int head) {
    using T = typename std::conditional<F16, __half, __nv_bfloat16>::type;
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, heads = KEYS ? a.nkv : a.nh;
    const T *q = static_cast<const T *>(a.q), *k = static_cast<const T *>(a.k), *v = static_cast<const T *>(a.v);
    const T *go = static_cast<const T *>(a.go);
    for (int r = threadIdx.x >> 5; r < live; r += warps) {
        const int row = u.p0 + r;
        float acc1[N], acc2[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc1[i] = acc2[i] = 0.f;
        int lo = row, hi = u.len;
        if (KEYS) {
            if (a.window > 0 && row < u.len - a.window) hi = row + a.window;
        } else {
            hi = row + 1;
            lo = a.window > 0 && row - a.window + 1 > 0 ? row - a.window + 1 : 0;
        }
        for (int x = lo; x < hi; ++x)
            for (int z = 0; z < (KEYS ? a.hpk : 1); ++z) {
                const int h = KEYS ? head * a.hpk + z : head, g = h / a.hpk;
                const int64_t pos = (int64_t)u.begin + (KEYS ? x : row), t = (int64_t)u.begin + (KEYS ? row : x);
                const T *qr = q + pos * a.qs + (int64_t)h * a.hd, *kr = k + t * a.ks + (int64_t)g * a.hd;
                const T *vr = v + t * a.vs + (int64_t)g * a.hd, *gr = go + (pos * a.nh + h) * a.hd;
                float s = 0.f, dp = 0.f;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int d = lane + 32 * i;
                    if (d < a.hd) s = fmaf(to_f(qr[d]), to_f(kr[d]), s), dp = fmaf(to_f(gr[d]), to_f(vr[d]), dp);
                }
                s = warp_sum(s), dp = warp_sum(dp);
                const float *l = a.lse_in + (pos * a.nh + h) * 2;
                const float e = expf(s * a.scale - l[0] - l[1]), ds = e * (dp - a.stats[(int64_t)h * a.tokens + pos].y);
                const T *x1 = KEYS ? qr : kr;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int d = lane + 32 * i;
                    if (d < a.hd) {
                        acc1[i] = fmaf(ds, to_f(x1[d]), acc1[i]);
                        if (KEYS) acc2[i] = fmaf(e, to_f(gr[d]), acc2[i]);
                    }
                }
            }
        const int64_t at = (((int64_t)u.begin + row) * heads + head) * a.hd;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int d = lane + 32 * i;
            if (d >= a.hd) continue;
            static_cast<T *>(KEYS ? a.dk : a.dq)[at + d] = from_f<T>(acc1[i] * a.scale);
            if (KEYS) static_cast<T *>(a.dv)[at + d] = from_f<T>(acc2[i]);
        }
    }
}

template <int D, bool F16, bool KEYS>
__device__ __forceinline__ void unit_body(const BwdArgs &p, Ctl &c, uint32_t smem, uint32_t tmem, int64_t index,
                                          bool check, int warp, int lane) {
    using C = Cfg<D>;
    const unsigned heads = KEYS ? p.a.nkv : p.a.nh;
    const int head = (int)(index % heads), g = KEYS ? head : head / p.a.hpk;
    const Unit u = find_unit(p.a, index / heads, kRows, !KEYS, check, &g_bwd_error_word);
    if (!u.live) return;
    const int live = u.len - u.p0 < kRows ? u.len - u.p0 : kRows;
    if (u.pad) {
        for (int r = warp; r < live; r += kThreads / 32) {
            const int64_t at = (((int64_t)u.begin + u.p0 + r) * heads + head) * p.a.hd;
            for (int d = lane; d < p.a.hd; d += 32) {
                static_cast<uint16_t *>(KEYS ? p.a.dk : p.a.dq)[at + d] = 0;
                if (KEYS) static_cast<uint16_t *>(p.a.dv)[at + d] = 0;
            }
        }
        return;
    }
    const Waiter w{&c.abort_flag, &g_bwd_error_word};
    const Walk k = walk_of<KEYS>(p.a, u, live);
    const float sigma = ds_scale<F16>(p);
    if (warp < kSoftWarps) {
        role_soft<D, F16, KEYS>(p, c, smem, tmem, u, k, live, head, sigma, warp, lane, w);
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        const int second = warp - kMmaWarp;
        const uint32_t sm = uniform(smem), tm = uniform(tmem);
        const Walk ku{uniform(k.lo), uniform(k.hi), uniform(k.heads)};
        if (second)
            issue_sums<D, KEYS>(p, c, sm, tm, ku, lane, w);
        else
            issue_scores<D, KEYS>(p, c, sm, tm, uniform(u.len), ku, lane, w);
        tc_commit_to_if(su32(&c.mma_done[second]), lane == 0);  // nothing may still run when tensor memory is released
        drain(su32(&c.mma_done[second]), 0, w);
        __syncwarp();
    } else if (warp < kStatWarp) {
        if (lane == 0) role_load<D, KEYS>(p, c, smem, u, k, head, g, w);
        __syncwarp();
    } else if (KEYS) {
        role_stats<F16>(p, c, smem, u, k, g, F16 ? sigma * 0x1p-13f : 1.f, lane, w);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (c.bad && !c.abort_flag) recompute<D, F16, KEYS>(p.a, u, live, head);
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1) backward_tc_kernel(const __grid_constant__ BwdArgs p) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t smem = (su32(smem_raw) + 1023u) & ~1023u;
    Ctl &c = *reinterpret_cast<Ctl *>(smem_raw + (smem - su32(smem_raw)));
    const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        bar_init(su32(&c.r_full), 2);
        for (int s = 0; s < 4; ++s) {
            bar_init(su32(&c.x_full[s]), 2);
            bar_init(su32(&c.x_empty[s]), 1);
        }
        for (int s = 0; s < kStatSlots; ++s) {
            bar_init(su32(&c.st_full[s]), 1);
            bar_init(su32(&c.st_empty[s]), 8);
        }
        for (int i = 0; i < 3; ++i) {
            bar_init(su32(&c.s_full[i]), 1);
            bar_init(su32(&c.g_full[i]), 1);
            bar_init(su32(&c.p_ready[i]), 8);
            bar_init(su32(&c.free[i]), 1);
        }
        bar_init(su32(&c.acc_full), 1);
        bar_init(su32(&c.mma_done[0]), 1);
        bar_init(su32(&c.mma_done[1]), 1);
        c.abort_flag = 0;
        c.bad = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tc_alloc(su32(&c.tmem_base), 512);
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = c.tmem_base;
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int64_t)blockIdx.x < p.key_units)
        unit_body<D, F16, true>(p, c, smem, tmem, blockIdx.x, blockIdx.x == 0, warp, lane);
    else
        unit_body<D, F16, false>(p, c, smem, tmem, (int64_t)blockIdx.x - p.key_units, false, warp, lane);
    __syncthreads();
    if (warp == kMmaWarp) tc_dealloc(tmem, 512);
}

template <int D, bool F16>
int launch(const BwdArgs &q, int64_t blocks, cudaStream_t st) {
    static std::atomic<uint64_t> configured{0};
    return launch_tc(backward_tc_kernel<D, F16>, blocks, kThreads, Cfg<D>::kSmem, configured, q, st);
}

template <typename T>
int launch_stats(const Args &a, unsigned *norms, cudaStream_t st) {
    int group = 1;
    while (group * 8 < a.hd) group *= 2;
    const int64_t runs = (a.tokens + 31) / 32, warps = runs * (a.nh + (std::is_same<T, __half>::value ? a.nkv : 0));
    if (std::is_same<T, __half>::value && cudaMemsetAsync(norms, 0, 2 * sizeof(unsigned), st) != cudaSuccess)
        return DGRAD_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((warps + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, stats_kernel<T>, a, norms, group) == cudaSuccess ? DGRAD_OK : DGRAD_ERR_CUDA;
}

}  // namespace

int backward_tc(const Args &a, unsigned *norms, const mha_packed_params *p, int dtype, cudaStream_t st) {
    BwdArgs q{};
    q.a = a;
    q.norms = norms;
    const int D = a.hd <= 64 ? 64 : 128;
    q.idesc1 = instr_desc(dtype, kRows, kCols, false);
    q.idesc2 = instr_desc(dtype, kRows, D, true);
    const int64_t dense = (int64_t)a.nh * a.hd;
    if (!encode_rows(&q.q_map, a.q, a.tokens, a.nh, a.hd, a.qs, kRows) ||
        !encode_rows(&q.k_map, a.k, a.tokens, a.nkv, a.hd, a.ks, kRows) ||
        !encode_rows(&q.v_map, a.v, a.tokens, a.nkv, a.hd, a.vs, kRows) ||
        !encode_rows(&q.go_map, a.go, a.tokens, a.nh, a.hd, dense, kRows))
        return DGRAD_ERR_UNSUPPORTED;
    const bool f16 = dtype == DGRAD_F16;
    const int rc = f16 ? launch_stats<__half>(a, norms, st) : launch_stats<__nv_bfloat16>(a, norms, st);
    if (rc != DGRAD_OK) return rc;
    const int64_t units = unit_bound(p, kRows);
    q.key_units = units * a.nkv;
    const int64_t blocks = q.key_units + units * a.nh;
    if (D == 64) return f16 ? launch<64, true>(q, blocks, st) : launch<64, false>(q, blocks, st);
    return f16 ? launch<128, true>(q, blocks, st) : launch<128, false>(q, blocks, st);
}

}  // namespace mhapk
