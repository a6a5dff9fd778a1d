// The end of one block and the start of the next, forward and backward, on gfx950.
//
//   r = x + c sig(z) f,   y = h w + b with h = norm(r);   f = o, or k p + q with k = norm(o)
//   backward, with S() a mean over the row (0 where the norm is not centred, for the first of each):
//     g = dy w,   e = dr + rstd (g - S(g) - h S(g h)) is the gradient of r and of x
//     dz = e c f sig'(z),   d = e c sig(z) is the gradient of f,   do = d, or
//     do = rstd_o (d p - S(d p) - k S(d p k));   sums over rows: dw = dy h, db = dy, dc = e sig(z) f,
//     dp = d k, dq = d
//
// Bound by HBM: every array is read or written once, a row stays in registers and every sum is in
// fp32.  The backward pass forms r again from x, o and z instead of reading it: the same bytes, and
// r without its rounding.  G lanes share a row, a piece of 16 bytes each (KP pieces beyond 512 lanes);
// the next row is on its way while one is summed.  400,000 rows of 512 bfloat16 with a gate: forward 407 us
// (5.0 TB/s), backward 645 (5.1 TB/s); 25,600 ragged rows of 1,024 with everything there 54 and 97, with
// 8 for the parameters' partial sums.  The gradient then has two sums over a row one after the other, each with a
// barrier of the row's two wavefronts, at two wavefronts a SIMD, where the bytes take 68 us.  In float32, where a
// row has twice the bytes, with a gate: 25,600 rows of 1,024 forward 104 us (5.0 TB/s), backward 164 to 169 (5.1).
#include "common.h"
#include "encoder.h"
#include "gates.h"
#include "norm_rows.h"

namespace semicrf {

namespace {

// Pieces a lane up to which the weights stay in registers
constexpr int HOLD = 2;

// Two sums at once
template <int G>
__device__ __forceinline__ void row_sums(float& u, float& v, float* red, int& slot) {
    if constexpr (G <= 64) {
        u = group_reduce<G>(u, OpSum());
        v = group_reduce<G>(v, OpSum());
    } else {
        u = group_reduce<64>(u, OpSum());
        v = group_reduce<64>(v, OpSum());
        float* s = red + slot * 2 * (G / 64);
        slot ^= 1;
        if ((threadIdx.x & 63) == 0) {
            s[(threadIdx.x >> 6) * 2] = u;
            s[(threadIdx.x >> 6) * 2 + 1] = v;
        }
        __syncthreads();
        u = v = 0.0f;
#pragma unroll
        for (int i = 0; i < G / 64; ++i) {
            u += s[2 * i];
            v += s[2 * i + 1];
        }
    }
}

// Where a row starts in the dense arrays and in the strided ones; whether it holds data.
struct At {
    size_t dense;
    int64_t branch, gate;
    bool ok;
};
__device__ __forceinline__ At locate(const semicrf_residual& p, unsigned row, unsigned rows, int32_t* status) {
    At at{};
    at.ok = row < rows;
    if (!at.ok) return at;
    const unsigned b = row / (unsigned)p.T, t = row - b * (unsigned)p.T;
    at.ok = !p.lengths || (int)t < seq_length(p.lengths, b, p.T, status);
    at.dense = (size_t)row * p.N;
    at.branch = b * p.branch_stride[0] + t * p.branch_stride[1];
    at.gate = b * p.gate_stride[0] + t * p.gate_stride[1];
    return at;
}

// V weights from a column as they lie in memory, which takes half the registers in bfloat16; where there
// are none, a factor of 1 or a term of 0.
template <class W, int V>
struct Weights {
    W t[V];
    // Called in a loop: keeps the compiler from converting them once and holding the results
    __device__ __forceinline__ void stay() {
        constexpr int WORDS = V * sizeof(W) / 4;
        uint32_t r[WORDS];
        __builtin_memcpy(r, t, sizeof(r));
#pragma unroll
        for (int i = 0; i < WORDS; ++i) asm volatile("" : "+v"(r[i]));
        __builtin_memcpy(t, r, sizeof(r));
    }
    __device__ __forceinline__ void load(const void* p, int at, int N, float dflt) {
        const W* w = (const W*)p;
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = (W)dflt;
        if (!p) return;
        if (at + V <= N) {
            __builtin_memcpy(t, w + at, sizeof(t));
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (at + i < N) t[i] = w[at + i];
        }
    }
    __device__ __forceinline__ float operator[](int i) const { return (float)t[i]; }
};
template <class W, int V>
struct Params {
    Weights<W, V> w, b, c, p, q;
    __device__ __forceinline__ void stay() {
        w.stay();
        b.stay();
        c.stay();
        p.stay();
        q.stay();
    }
    __device__ __forceinline__ void load(const semicrf_residual& a, int at, bool post) {
        w.load(a.weight, at, a.N, 1.0f);
        b.load(a.bias, at, a.N, 0.0f);
        c.load(a.scale, at, a.N, 1.0f);
        p.load(post ? a.branch_weight : nullptr, at, a.N, 1.0f);
        q.load(post ? a.branch_bias : nullptr, at, a.N, 0.0f);
    }
};

template <class T, class W, int G, int KP, int NT, int MODE, bool POST>
__global__ __launch_bounds__(NT) void k_residual_norm(const ResArgs a) {
    using Pc = Piece<T, MODE == NARROWER>;
    constexpr int V = Pc::V, RPB = NT / G;
    __shared__ float red[2 * (G > 64 ? G / 64 : 1)];
    int slot = 0;
    const semicrf_residual& p = a.p;
    const int N = MODE == EXACT ? G * KP * V : p.N, lane = threadIdx.x % G;
    const unsigned rows = (unsigned)p.B * p.T, step = gridDim.x * RPB;
    const bool gated = p.gate;
    unsigned row = blockIdx.x * RPB + threadIdx.x / G;
    raw_piece xr[KP], br[KP], gr[KP];
    At at;
    auto fetch = [&](unsigned i) {
        at = locate(p, i, rows, a.status);
        if (!at.ok) return;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const Pc pc(k * G + lane, N);
            xr[k] = load_raw((const T*)p.x + at.dense, pc, N);
            br[k] = load_raw((const T*)p.branch + at.branch, pc, N);
            if (gated) gr[k] = load_raw((const T*)p.gate + at.gate, pc, N);
        }
    };
#pragma unroll
    for (int k = 0; k < KP; ++k) xr[k] = br[k] = gr[k] = raw_piece{0, 0, 0, 0};
    fetch(row);
    Params<W, V> par[KP];
    if constexpr (KP <= HOLD)
#pragma unroll
        for (int k = 0; k < KP; ++k) par[k].load(p, Pc(k * G + lane, N).at, POST);
    for (unsigned r0 = blockIdx.x * RPB; r0 < rows; r0 += step, row += step) {
        const bool now = at.ok, in = row < rows;
        const size_t dense = (size_t)row * N;
        float x[KP][V], f[KP][V], own[KP][V];
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const Pc pc(k * G + lane, N);
            if constexpr (KP > HOLD) par[k].load(p, pc.at, POST);
#pragma unroll
            for (int i = 0; i < V; ++i) own[k][i] = MODE == EXACT || counted(pc, i, N) ? 1.0f : 0.0f;
            unpack<T>(xr[k], x[k]);
            unpack<T>(br[k], f[k]);
        }
        float mean_o = 0.0f, rstd_o = 0.0f;
        if constexpr (POST) {
            if (p.center) {
                float s = 0.0f;
#pragma unroll
                for (int k = 0; k < KP; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) s = fmaf(f[k][i], own[k][i], s);
                mean_o = row_sum<G>(s, red, slot) / (float)N;
            }
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    f[k][i] -= mean_o;
                    s = fmaf(f[k][i], f[k][i] * own[k][i], s);
                }
            rstd_o = 1.0f / sqrtf(row_sum<G>(s, red, slot) / (float)N + p.eps);
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) f[k][i] = fmaf(f[k][i] * rstd_o, par[k].p[i], par[k].q[i]);
        }
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            float z[V];
            if (gated) unpack<T>(gr[k], z);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float c = par[k].c[i];
                if (gated) c *= sigmoid(z[i]);
                x[k][i] = fmaf(c, f[k][i], x[k][i]);
                s = fmaf(x[k][i], own[k][i], s);
                f[k][i] = now ? x[k][i] : 0.0f;
            }
        }
        if (r0 + step < rows) fetch(row + step);
        if (in)
#pragma unroll
            for (int k = 0; k < KP; ++k) store_piece<T>((T*)a.r + dense, Pc(k * G + lane, N), N, f[k]);
        float mean = 0.0f;
        if (p.center) mean = row_sum<G>(s, red, slot) / (float)N;
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < KP; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[k][i] -= mean;
                s = fmaf(x[k][i], x[k][i] * own[k][i], s);
            }
        const float rstd = 1.0f / sqrtf(row_sum<G>(s, red, slot) / (float)N + p.eps);
        if (!in) continue;
        if (a.stats && lane == 0) {
            float* st = a.stats + (size_t)row * 4;
            st[0] = now ? mean : 0.0f;
            st[1] = now ? rstd : 0.0f;
            st[2] = now ? mean_o : 0.0f;
            st[3] = now ? rstd_o : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < KP; ++k) {
#pragma unroll
            for (int i = 0; i < V; ++i) x[k][i] = now ? fmaf(x[k][i] * rstd, par[k].w[i], par[k].b[i]) : 0.0f;
            store_piece<T>((T*)a.y + dense, Pc(k * G + lane, N), N, x[k]);
        }
    }
}

// part [workgroup][5][N]: the sums over the workgroup's rows, in the order of grad_params
template <class T, class W, int G, int KP, int NT, int MODE, bool POST>
__global__ __launch_bounds__(NT, KP == 1 && !POST ? 3 : 1) void k_residual_norm_grad(const ResArgs a, float* part) {
    using Pc = Piece<T, MODE == NARROWER>;
    constexpr int V = Pc::V, RPB = NT / G;
    __shared__ float red[4 * (G > 64 ? G / 64 : 1)];
    __shared__ float join[RPB > 1 ? (RPB - 1) * G * V * 5 : 1];
    int slot = 0;
    const semicrf_residual& p = a.p;
    const int N = MODE == EXACT ? G * KP * V : p.N, lane = threadIdx.x % G, sub = threadIdx.x / G;
    const unsigned rows = (unsigned)p.B * p.T, step = gridDim.x * RPB;
    const bool gated = p.gate;
    const float inv = 1.0f / (float)N, cinv = p.center ? inv : 0.0f;
    unsigned row = blockIdx.x * RPB + sub;
    raw_piece xr[KP], br[KP], gr[KP], dr[KP], dy[KP];
    float st[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    At at;
    auto fetch = [&](unsigned i) {
        at = locate(p, i, rows, a.status);
        if (!at.ok) {                                // a row of zeros adds nothing
#pragma unroll
            for (int k = 0; k < KP; ++k) xr[k] = br[k] = gr[k] = dr[k] = dy[k] = raw_piece{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j) st[j] = 0.0f;
            return;
        }
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const Pc pc(k * G + lane, N);
            xr[k] = load_raw((const T*)p.x + at.dense, pc, N);
            br[k] = load_raw((const T*)p.branch + at.branch, pc, N);
            if (gated) gr[k] = load_raw((const T*)p.gate + at.gate, pc, N);
            if (a.grad_r) dr[k] = load_raw((const T*)a.grad_r + at.dense, pc, N);
            if (a.grad_y) dy[k] = load_raw((const T*)a.grad_y + at.dense, pc, N);
        }
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) st[i4] = a.stats_in[(size_t)i * 4 + i4];
    };
#pragma unroll
    for (int k = 0; k < KP; ++k) xr[k] = br[k] = gr[k] = dr[k] = dy[k] = raw_piece{0, 0, 0, 0};
    fetch(row);
    Params<W, V> par[KP];
    if constexpr (KP <= HOLD)
#pragma unroll
        for (int k = 0; k < KP; ++k) par[k].load(p, Pc(k * G + lane, N).at, POST);
    float sum[KP][5][V];
#pragma unroll
    for (int k = 0; k < KP; ++k)
#pragma unroll
        for (int j = 0; j < 5; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) sum[k][j][i] = 0.0f;
    for (unsigned r0 = blockIdx.x * RPB; r0 < rows; r0 += step, row += step) {
        const bool now = at.ok, in = row < rows;
#pragma unroll
        for (int k = 0; k < KP; ++k)
            if (KP <= HOLD && !POST) par[k].stay();
        const size_t dense = (size_t)row * N;
        const float mean = st[0], rstd = st[1], mean_o = st[2], rstd_o = st[3];
        // h: x, then r, then its norm; kh: the branch, then its norm; e: dr, then the gradient of r;
        // g: dy w, then d p; sg, qg: sig(z) and 1 - sig(z)
        float h[KP][V], kh[KP][V], e[KP][V], g[KP][V], sg[KP][V], qg[KP][V];
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const Pc pc(k * G + lane, N);
            if constexpr (KP > HOLD) par[k].load(p, pc.at, POST);
            unpack<T>(xr[k], h[k]);
            unpack<T>(br[k], kh[k]);
            unpack<T>(dr[k], e[k]);
            unpack<T>(dy[k], g[k]);
            float z[V];
            if (gated) unpack<T>(gr[k], z);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sg[k][i] = 1.0f;
                qg[k][i] = 0.0f;
                if (gated) sigmoids(z[i], sg[k][i], qg[k][i]);
                if (POST) kh[k][i] = (kh[k][i] - mean_o) * rstd_o;
                const float f = POST ? fmaf(kh[k][i], par[k].p[i], par[k].q[i]) : kh[k][i];
                h[k][i] = (fmaf(par[k].c[i] * sg[k][i], f, h[k][i]) - mean) * rstd;
                sum[k][0][i] = fmaf(g[k][i], h[k][i], sum[k][0][i]);
                sum[k][1][i] += g[k][i];
                g[k][i] *= par[k].w[i];
                const float t = MODE == EXACT || counted(pc, i, N) ? g[k][i] : 0.0f;
                s0 += t;
                s1 = fmaf(t, h[k][i], s1);
            }
        }
        if (r0 + step < rows) fetch(row + step);
        row_sums<G>(s0, s1, red, slot);
        s0 *= cinv;
        s1 *= inv;
        float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const Pc pc(k * G + lane, N);
            float dz[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                e[k][i] = fmaf(rstd, g[k][i] - s0 - h[k][i] * s1, e[k][i]);
                const float f = POST ? fmaf(kh[k][i], par[k].p[i], par[k].q[i]) : kh[k][i];
                const float es = e[k][i] * sg[k][i], d = es * par[k].c[i];
                dz[i] = now ? d * f * qg[k][i] : 0.0f;
                sum[k][2][i] = fmaf(es, f, sum[k][2][i]);
                e[k][i] = now ? e[k][i] : 0.0f;      // weights that are not finite stay out of padding
                g[k][i] = d;
                if constexpr (POST) {
                    sum[k][3][i] = fmaf(d, kh[k][i], sum[k][3][i]);
                    sum[k][4][i] += d;
                    g[k][i] = d * par[k].p[i];
                    const float t = MODE == EXACT || counted(pc, i, N) ? g[k][i] : 0.0f;
                    t0 += t;
                    t1 = fmaf(t, kh[k][i], t1);
                }
            }
            if (in) {
                store_piece<T>((T*)a.grad_x + dense, pc, N, e[k]);
                if (gated) store_piece<T>((T*)a.grad_gate + dense, pc, N, dz);
            }
        }
        if constexpr (POST) {
            row_sums<G>(t0, t1, red, slot);
            t0 *= cinv;
            t1 *= inv;
        }
        if (!in) continue;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (POST) g[k][i] = rstd_o * (g[k][i] - t0 - kh[k][i] * t1);
                g[k][i] = now ? g[k][i] : 0.0f;
            }
            store_piece<T>((T*)a.grad_branch + dense, Pc(k * G + lane, N), N, g[k]);
        }
    }
    if (!a.grad_params) return;
    // join the row groups of the workgroup in order, then one partial row
    float* out = part + (size_t)blockIdx.x * 5 * N;
#pragma unroll
    for (int k = 0; k < KP; ++k) {
        if constexpr (RPB > 1) {
            if (sub > 0)
#pragma unroll
                for (int j = 0; j < 5; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) join[(((sub - 1) * 5 + j) * V + i) * G + lane] = sum[k][j][i];
            __syncthreads();
            if (sub == 0)
#pragma unroll 1
                for (int q = 0; q < RPB - 1; ++q)
#pragma unroll
                    for (int j = 0; j < 5; ++j)
#pragma unroll
                        for (int i = 0; i < V; ++i) sum[k][j][i] += join[((q * 5 + j) * V + i) * G + lane];
        }
        if (sub == 0) {
            const Pc pc(k * G + lane, N);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (counted(pc, i, N))
#pragma unroll
                    for (int j = 0; j < 5; ++j) out[(size_t)j * N + pc.at + i] = sum[k][j][i];
        }
    }
}

// grid (ceil(5N / 16)), block 256: 16 columns, 16 groups of partial rows, joined in order
template <class W>
__global__ __launch_bounds__(256) void k_residual_partials(const float* part, int nwg, int N, W* out) {
    __shared__ float s[16][17];
    const int c = blockIdx.x * 16 + (threadIdx.x & 15), grp = threadIdx.x >> 4;
    const int per = (nwg + 15) / 16, r1 = min(nwg, (grp + 1) * per);
    float v = 0.0f;
    if (c < 5 * N) {
        constexpr int U = 8;                   // loads in flight
        for (int r = grp * per; r < r1; r += U) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = r + u < r1 ? part[(size_t)(r + u) * 5 * N + c] : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) v += x[u];
        }
    }
    s[grp][threadIdx.x & 15] = v;
    __syncthreads();
    if (grp == 0 && c < 5 * N) {
        for (int i = 1; i < 16; ++i) v += s[i][threadIdx.x];
        out[c] = (W)v;
    }
}

// Lanes per row and pieces per lane: one piece a lane up to 512 lanes.
struct RowShape {
    int G, KP;
};
RowShape row_shape(int N, int V) {
    const int np = (N + V - 1) / V;
    int G = 2, KP = 1;
    while (G < 512 && G < np) G *= 2;
    while (KP * G < np) KP *= 2;
    return {G, KP};
}
constexpr int row_threads(int G) { return G > 64 ? G : 256; }

// Workgroups of NT threads for the rows: at most as many as make `per_simd` wavefronts a SIMD.
int row_wgs(long rows, int G, int per_simd) {
    const int NT = row_threads(G);
    const long need = (rows + NT / G - 1) / (NT / G), most = 1024l * per_simd / (NT / 64);
    return (int)(need < most ? need : most);
}
// As many wavefronts a SIMD as the kernels' registers leave room for: more workgroups than run at once make a
// second, short round, and in the gradient more partial rows (25,600 ragged rows of 1,024 bfloat16, everything
// there: 105 us and 19 for the partials' sum at 4, 97 and 8 at 2; 400,000 of 512 without a norm of the
// branch: 705 and 9 at 4, 645 and 6 at 3).
template <class T>
constexpr int waves(bool norm_branch) { return sizeof(T) == 4 ? (norm_branch ? 6 : 8) : norm_branch ? 4 : 5; }
constexpr int GRAD_WAVES = 2, GRAD_WAVES_PLAIN = 3;

template <int V, class F>
hipError_t with_row_shape(int N, F&& f) {
    const RowShape s = row_shape(N, V);
    if (N < V)
        return f(std::integral_constant<int, 2>(), std::integral_constant<int, 1>(),
                 std::integral_constant<int, NARROWER>());
#define CASE(g, kp)                                                                                                  \
    if (s.G == g && s.KP == kp) {                                                                                    \
        std::integral_constant<int, g> gg;                                                                           \
        std::integral_constant<int, kp> kk;                                                                          \
        if constexpr (kp == 1)                                                                                       \
            if (N == g * V) return f(gg, kk, std::integral_constant<int, EXACT>());                                  \
        return f(gg, kk, std::integral_constant<int, MASKED>());                                                     \
    }
    CASE(2, 1) CASE(4, 1) CASE(8, 1) CASE(16, 1) CASE(32, 1) CASE(64, 1) CASE(128, 1) CASE(256, 1) CASE(512, 1)
    CASE(512, 2) CASE(512, 4)
    if constexpr (V == 4) { CASE(512, 8) }     // rows have at most 16,384 elements
#undef CASE
    return hipErrorInvalidValue;
}

template <class T, class W>
hipError_t run_residual(const ResArgs& a, hipStream_t stream) {
    return with_row_shape<16 / (int)sizeof(T)>(a.p.N, [&](auto g, auto kp, auto mode) {
        constexpr int G = decltype(g)::value, KP = decltype(kp)::value, NT = row_threads(G);
        const int nwg = row_wgs((long)a.p.B * a.p.T, G, waves<T>(a.p.norm_branch));
        if (a.p.norm_branch)
            hipLaunchKernelGGL((k_residual_norm<T, W, G, KP, NT, decltype(mode)::value, true>), dim3(nwg), dim3(NT), 0,
                               stream, a);
        else
            hipLaunchKernelGGL((k_residual_norm<T, W, G, KP, NT, decltype(mode)::value, false>), dim3(nwg), dim3(NT), 0,
                               stream, a);
        return hipGetLastError();
    });
}

template <class T, class W>
hipError_t run_residual_grad(const ResArgs& a, float* part, hipStream_t stream) {
    return with_row_shape<16 / (int)sizeof(T)>(a.p.N, [&](auto g, auto kp, auto mode) {
        constexpr int G = decltype(g)::value, KP = decltype(kp)::value, NT = row_threads(G);
        const int nwg = row_wgs((long)a.p.B * a.p.T, G, a.p.norm_branch ? GRAD_WAVES : GRAD_WAVES_PLAIN);
        if (a.p.norm_branch)
            hipLaunchKernelGGL((k_residual_norm_grad<T, W, G, KP, NT, decltype(mode)::value, true>), dim3(nwg), dim3(NT),
                               0, stream, a, part);
        else
            hipLaunchKernelGGL((k_residual_norm_grad<T, W, G, KP, NT, decltype(mode)::value, false>), dim3(nwg),
                               dim3(NT), 0, stream, a, part);
        if (a.grad_params)
            hipLaunchKernelGGL((k_residual_partials<W>), dim3((5 * a.p.N + 15) / 16), dim3(256), 0, stream, part, nwg,
                               a.p.N, (W*)a.grad_params);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_residual_norm(const ResArgs& a, hipStream_t stream) {
    if (a.p.dtype == SEMICRF_F32) return run_residual<float, float>(a, stream);
    return a.p.wdtype == SEMICRF_F32 ? run_residual<bf16, float>(a, stream) : run_residual<bf16, bf16>(a, stream);
}

size_t residual_norm_grad_bytes(int B, int T, int N, int dtype) {
    const RowShape s = row_shape(N, dtype == SEMICRF_F32 ? 4 : 8);
    return (size_t)row_wgs((long)B * T, s.G, GRAD_WAVES_PLAIN) * 5 * N * sizeof(float);
}

hipError_t launch_residual_norm_grad(const ResArgs& a, void* ws, hipStream_t stream) {
    float* part = (float*)ws;
    if (a.p.dtype == SEMICRF_F32) return run_residual_grad<float, float>(a, part, stream);
    return a.p.wdtype == SEMICRF_F32 ? run_residual_grad<bf16, float>(a, part, stream)
                                     : run_residual_grad<bf16, bf16>(a, part, stream);
}

}  // namespace semicrf
