// Layer norm over the last axis, forward and backward, on gfx950.
//
//   mu = mean_j x_j,  r = 1 / sqrt(mean_j (x_j - mu)^2 + eps),  y_j = (x_j - mu) r w_j + b_j
//   backward, with h_j = (x_j - mu) r and g_j = dy_j w_j:
//     dx_j = r (g_j - mean g - h_j mean(g h)),  dw_j = sum over rows dy_j h_j,  db_j = sum dy_j
//
// Both are bound by HBM: a row is read once and kept in registers (the variance is taken
// about the mean from the registers, not as a difference of sums), and every sum is in fp32.
// G lanes of a workgroup share a row, each with KP pieces of 16 bytes; G grows with the width
// so that a lane keeps few pieces and narrow rows still fill a wavefront.
//
// The weight's gradient sums over all rows.  A workgroup of the backward pass takes every
// nwg-th row block and keeps its columns' sums in registers; its G-groups are joined through
// LDS and written as one partial row, and k_norm_partials adds the partial rows in a fixed
// order (no atomics: the same inputs give the same bits).
#include "common.h"
#include "encoder.h"

namespace semicrf {

namespace {

// Sum over the G lanes of a row (G <= 64: inside a wavefront; else the whole workgroup of G
// threads, through `red`, which alternates between two slots so one barrier is enough).
template <int G>
__device__ __forceinline__ float row_sum(float v, float* red, int& slot) {
    if constexpr (G <= 64) {
        return group_reduce<G>(v, OpSum());
    } else {
        v = group_reduce<64>(v, OpSum());
        float* s = red + slot * (G / 64);
        slot ^= 1;
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < G / 64; ++i) t += s[i];
        return t;
    }
}

// Row -> t < length of its sequence.  Rows are numbered b * T + t, below 2^30.
__device__ __forceinline__ bool row_valid(const NormArgs& a, unsigned row) {
    if (!a.lengths) return true;
    const unsigned b = row / (unsigned)a.T;
    return (int)(row - b * (unsigned)a.T) < seq_length(a.lengths, b, a.T, a.status);
}

// Whether element i of a lane's piece is its own.  Sums take the others times 0: they hold elements
// of the same row, so one that is not finite is in the sum either way.
template <class T, bool NARROW>
__device__ __forceinline__ bool counted(const Piece<T, NARROW>& p, int i, int N) {
    return i >= p.skip && (!NARROW || i < N);
}

// V weights from column c in the element type W of theirs
template <class W, int V>
__device__ __forceinline__ void load_weights(const void* p, int c, int N, float dflt,
                                             float (&w)[V]) {
    if (p) {
        load_elements<W, V>((const W*)p, c, N, w);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = dflt;
    }
}

// One pass over the rows of a workgroup: the next row is on its way while this one is summed, and
// the weights stay in registers.
//
// MODE: rows fill the lanes' pieces exactly (G * KP * V elements), or not, or are narrower than one.
//
// Forward, 25,600 ragged rows of 1,024 bfloat16: 92 MB in 17 us (5.4 TB/s).  128 rows of 333 float32:
// 3.2 us, the launch.  Backward, 400,000 rows of 512 bfloat16: 1.23 GB in 221 us (5.6 TB/s), the sum of
// 1,024 partial rows 6.6 us.
enum { EXACT, MASKED, NARROWER };

template <class T, class W, int G, int KP, int NT, int MODE>
__global__ __launch_bounds__(NT) void k_layer_norm(const NormArgs a) {
    using Pc = Piece<T, MODE == NARROWER>;
    constexpr int V = Pc::V, RPB = NT / G;
    __shared__ float red[2 * (G > 64 ? G / 64 : 1)];
    int slot = 0;
    const int N = MODE == EXACT ? G * KP * V : a.N, lane = threadIdx.x % G;
    const unsigned rows = (unsigned)a.B * a.T, step = gridDim.x * RPB;
    unsigned row = blockIdx.x * RPB + threadIdx.x / G;
    raw_piece x[KP];
    bool ok;
    auto fetch = [&](unsigned at) {
        ok = at < rows && row_valid(a, at);
        if (!ok) return;
        const T* from = (const T*)a.x + (size_t)at * N;
#pragma unroll
        for (int k = 0; k < KP; ++k) x[k] = load_raw(from, Pc(k * G + lane, N), N);
    };
#pragma unroll
    for (int k = 0; k < KP; ++k) x[k] = raw_piece{0, 0, 0, 0};
    fetch(row);
    float w[KP][V], b[KP][V], own[KP][V];
#pragma unroll
    for (int k = 0; k < KP; ++k) {
        const Pc pc(k * G + lane, N);
        load_weights<W, V>(a.weight, pc.at, N, 1.0f, w[k]);
        load_weights<W, V>(a.bias, pc.at, N, 0.0f, b[k]);
#pragma unroll
        for (int i = 0; i < V; ++i) own[k][i] = counted(pc, i, N) ? 1.0f : 0.0f;
    }
    for (unsigned r0 = blockIdx.x * RPB; r0 < rows; r0 += step, row += step) {
        float v[KP][V];
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            unpack<T>(x[k], v[k]);
#pragma unroll
            for (int i = 0; i < V; ++i) s = MODE == EXACT ? s + v[k][i] : fmaf(v[k][i], own[k][i], s);
        }
        const bool now = ok, in = row < rows;
        if (r0 + step < rows) fetch(row + step);
        const float mean = row_sum<G>(s, red, slot) / (float)N;
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < KP; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[k][i] -= mean;
                s = fmaf(v[k][i], MODE == EXACT ? v[k][i] : v[k][i] * own[k][i], s);
            }
        const float var = row_sum<G>(s, red, slot) / (float)N;
        const float r = 1.0f / sqrtf(var + a.eps);
        if (!in) continue;
        if (lane == 0) {
            if (a.mean) a.mean[row] = now ? mean : 0.0f;
            if (a.rstd) a.rstd[row] = now ? r : 0.0f;
        }
        T* y = (T*)a.y + (size_t)row * N;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = now ? fmaf(v[k][i] * r, w[k][i], b[k][i]) : 0.0f;
            store_piece<T>(y, Pc(k * G + lane, N), N, v[k]);
        }
    }
}

template <class T, class W, int G, int KP, int NT, int MODE>
__global__ __launch_bounds__(NT) void k_layer_norm_grad(const NormArgs a, float* part) {
    using Pc = Piece<T, MODE == NARROWER>;
    constexpr int V = Pc::V, RPB = NT / G;
    __shared__ float red[2 * (G > 64 ? G / 64 : 1)];
    __shared__ float join[RPB > 1 ? (RPB - 1) * G * V * 2 : 1];
    int slot = 0;
    const int N = MODE == EXACT ? G * KP * V : a.N, lane = threadIdx.x % G, sub = threadIdx.x / G;
    const unsigned rows = (unsigned)a.B * a.T;
    const float inv = 1.0f / (float)N;
    // own: the weight where the element is the lane's own, else 0
    float w[KP][V], own[KP][V], dw[KP][V], db[KP][V];
#pragma unroll
    for (int k = 0; k < KP; ++k) {
        const Pc pc(k * G + lane, N);
        load_weights<W, V>(a.weight, pc.at, N, 1.0f, w[k]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            own[k][i] = counted(pc, i, N) ? w[k][i] : 0.0f;
            dw[k][i] = db[k][i] = 0.0f;
        }
    }
    const unsigned step = gridDim.x * RPB;
    unsigned row = blockIdx.x * RPB + sub;
    raw_piece xr[KP], gr[KP];
    float mean_r = 0.0f, rstd_r = 0.0f;
    bool ok;
    auto fetch = [&](unsigned at) {            // the next row is on its way while one is summed
        ok = at < rows && row_valid(a, at);
        if (!ok) return;
        const size_t first = (size_t)at * N;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const Pc pc(k * G + lane, N);
            xr[k] = load_raw((const T*)a.x + first, pc, N);
            gr[k] = load_raw((const T*)a.grad_out + first, pc, N);
        }
        mean_r = a.mean_in[at];
        rstd_r = a.rstd_in[at];
    };
#pragma unroll
    for (int k = 0; k < KP; ++k) xr[k] = gr[k] = raw_piece{0, 0, 0, 0};
    fetch(row);
    for (unsigned r0 = blockIdx.x * RPB; r0 < rows; r0 += step, row += step) {
        const bool in = row < rows, now = ok;
        const float mean = mean_r, r = rstd_r;
        float h[KP][V], dy[KP][V];
        float sg = 0.0f, sgh = 0.0f;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            unpack<T>(xr[k], h[k]);
            unpack<T>(gr[k], dy[k]);
        }
        if (r0 + step < rows) fetch(row + step);
        if (now) {
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    h[k][i] = (h[k][i] - mean) * r;
                    const float t = dy[k][i] * (MODE == EXACT ? w[k][i] : own[k][i]);
                    sg += t;
                    sgh += t * h[k][i];
                    dw[k][i] += dy[k][i] * h[k][i];
                    db[k][i] += dy[k][i];
                }
        }
        sg = row_sum<G>(sg, red, slot) * inv;
        sgh = row_sum<G>(sgh, red, slot) * inv;
        if (!in) continue;
        T* dx = (T*)a.grad_x + (size_t)row * N;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                dy[k][i] = now ? r * (dy[k][i] * w[k][i] - sg - h[k][i] * sgh) : 0.0f;
            store_piece<T>(dx, Pc(k * G + lane, N), N, dy[k]);
        }
    }
    // join the row groups of the workgroup in order, then one partial row [2][N]
    float* out = part + (size_t)blockIdx.x * 2 * N;
#pragma unroll
    for (int k = 0; k < KP; ++k) {
        if constexpr (RPB > 1) {
            __syncthreads();
            if (sub > 0) {
                float* j = join + ((sub - 1) * G + lane) * V * 2;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    j[i] = dw[k][i];
                    j[V + i] = db[k][i];
                }
            }
            __syncthreads();
            if (sub == 0)
#pragma unroll 1                               // unrolled, it holds up to 512 registers
                for (int q = 0; q < RPB - 1; ++q) {
                    const float* j = join + (q * G + lane) * V * 2;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        dw[k][i] += j[i];
                        db[k][i] += j[V + i];
                    }
                }
        }
        if (sub == 0) {
            const Pc pc(k * G + lane, N);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (counted(pc, i, N)) {
                    out[pc.at + i] = dw[k][i];
                    out[N + pc.at + i] = db[k][i];
                }
        }
    }
}

// grid (ceil(2N / 16)), block 256: 16 columns, 16 groups of partial rows, joined in order
template <class W>
__global__ __launch_bounds__(256) void k_norm_partials(const float* part, int nwg, int N, W* gw,
                                                       W* gb) {
    __shared__ float s[16][17];
    const int c = blockIdx.x * 16 + (threadIdx.x & 15), grp = threadIdx.x >> 4;
    const int per = (nwg + 15) / 16;
    const int r1 = min(nwg, (grp + 1) * per);
    float v = 0.0f;
    if (c < 2 * N) {
        constexpr int U = 8;                   // loads in flight
        for (int r = grp * per; r < r1; r += U) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = r + u < r1 ? part[(size_t)(r + u) * 2 * N + c] : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) v += x[u];
        }
    }
    s[grp][threadIdx.x & 15] = v;
    __syncthreads();
    if (grp == 0 && c < 2 * N) {
        for (int i = 1; i < 16; ++i) v += s[i][threadIdx.x];
        W* out = c < N ? gw : gb;
        if (out) out[c < N ? c : c - N] = (W)v;
    }
}

// Lanes per row and pieces per lane for a width.  Pieces per lane are kept at two until the
// row takes a whole workgroup of 1024.
struct Shape2 {
    int G, KP;
};
Shape2 norm_shape(int N, int V) {
    const int np = (N + V - 1) / V;
    int G = 2;
    while (G < 64 && G < np) G *= 2;
    if (np > 2 * 64) G = 256;
    if (np > 2 * 256) G = 1024;
    int KP = 1;
    while (KP * G < np) KP *= 2;
    return {G, KP};
}

// Workgroups of NT threads for the rows: at most as many as make `waves` wavefronts a SIMD.
int norm_wgs(long rows, int G, int NT, int waves) {
    const long need = (rows + NT / G - 1) / (NT / G), most = 1024l * waves / (NT / 64);
    return (int)(need < most ? need : most);
}
constexpr int norm_threads(int G) { return G > 256 ? G : 256; }
// The gradient runs at 4 wavefronts a SIMD: the row on its way hides the latency, and every
// workgroup leaves a partial row (400,000 rows of 512 bfloat16, with the partials' sum: 228 us
// at 4; 299 at 6 and 267 at 8 when it took 238 at 4, workgroups of 512 threads 326 at 4).  Narrow
// rows leave little and have little on its way: 8.
constexpr int norm_grad_waves(int G) { return G < 32 ? 8 : 4; }

// Calls f with the shape's G, KP and MODE.
template <int V, class F>
hipError_t with_shape(int N, F&& f) {
    const Shape2 s = norm_shape(N, V);
    using I = std::integral_constant<int, MASKED>;
    if (N < V)
        return f(std::integral_constant<int, 2>(), std::integral_constant<int, 1>(),
                 std::integral_constant<int, NARROWER>());
#define CASE(g, kp)                                                                                                  \
    if (s.G == g && s.KP == kp) {                                                                                    \
        std::integral_constant<int, g> gg;                                                                           \
        std::integral_constant<int, kp> kk;                                                                          \
        return N == g * kp * V ? f(gg, kk, std::integral_constant<int, EXACT>()) : f(gg, kk, I());                   \
    }
    CASE(2, 1) CASE(4, 1) CASE(8, 1) CASE(16, 1) CASE(32, 1) CASE(64, 1) CASE(64, 2) CASE(256, 1) CASE(256, 2)
    CASE(1024, 1) CASE(1024, 2) CASE(1024, 4)
    if constexpr (V == 4) { CASE(1024, 8) }    // rows have at most 32,768 elements
#undef CASE
    return hipErrorInvalidValue;
}

template <class T, class W>
hipError_t run_norm(const NormArgs& a, hipStream_t stream) {
    return with_shape<16 / (int)sizeof(T)>(a.N, [&](auto g, auto kp, auto mode) {
        constexpr int G = decltype(g)::value, KP = decltype(kp)::value, NT = norm_threads(G);
        const int nwg = norm_wgs((long)a.B * a.T, G, NT, 8);
        hipLaunchKernelGGL((k_layer_norm<T, W, G, KP, NT, decltype(mode)::value>), dim3(nwg), dim3(NT), 0, stream, a);
        return hipGetLastError();
    });
}

template <class T, class W>
hipError_t run_norm_grad(const NormArgs& a, float* part, hipStream_t stream) {
    return with_shape<16 / (int)sizeof(T)>(a.N, [&](auto g, auto kp, auto mode) {
        constexpr int G = decltype(g)::value, KP = decltype(kp)::value, NT = norm_threads(G);
        const int nwg = norm_wgs((long)a.B * a.T, G, NT, norm_grad_waves(G));
        hipLaunchKernelGGL((k_layer_norm_grad<T, W, G, KP, NT, decltype(mode)::value>), dim3(nwg), dim3(NT), 0, stream,
                           a, part);
        if (a.grad_weight || a.grad_bias)
            hipLaunchKernelGGL((k_norm_partials<W>), dim3((2 * a.N + 15) / 16), dim3(256), 0, stream,
                               part, nwg, a.N, (W*)a.grad_weight, (W*)a.grad_bias);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t stream) {
    if (a.dtype == SEMICRF_F32) return run_norm<float, float>(a, stream);
    return a.wdtype == SEMICRF_F32 ? run_norm<bf16, float>(a, stream) : run_norm<bf16, bf16>(a, stream);
}

size_t layer_norm_grad_bytes(int B, int T, int N, int dtype) {
    const int V = dtype == SEMICRF_F32 ? 4 : 8;
    const Shape2 s = norm_shape(N, V);
    return (size_t)norm_wgs((long)B * T, s.G, norm_threads(s.G), norm_grad_waves(s.G)) * 2 * N * sizeof(float);
}

hipError_t launch_layer_norm_grad(const NormArgs& a, void* ws, hipStream_t stream) {
    float* part = (float*)ws;
    if (a.dtype == SEMICRF_F32) return run_norm_grad<float, float>(a, part, stream);
    return a.wdtype == SEMICRF_F32 ? run_norm_grad<bf16, float>(a, part, stream)
                                   : run_norm_grad<bf16, bf16>(a, part, stream);
}

}  // namespace semicrf
