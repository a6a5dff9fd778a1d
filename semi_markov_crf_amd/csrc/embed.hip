// Embedding lookup with scaling, and its gradient by sorted tokens, on gfx950.
//
//   y[i, :] = scale * W[tok_i, :]        (0 at padding, NaN for a token outside [0, V))
//   dW[v, :] = scale * sum of dy[i, :] over the positions i with tok_i = v
//
// Both are bound by HBM.  The lookup reads each token once and moves rows in pieces of 16
// bytes.  The gradient has no float atomics: positions are sorted by token (stable, so a
// token's positions stay in order), the sorted list is cut into chunks of equal length, and a
// wavefront adds the rows of its chunk into registers, run by run.  A run inside one chunk is
// written to dW at once; a run that crosses chunk borders leaves one partial row a chunk, and
// k_grad_join adds those in order.  So a token that fills the whole batch and 50,000 tokens
// that appear once cost the same reads, and the same inputs give the same bits.
#include "common.h"
#include "encoder.h"

namespace semicrf {

namespace {

__device__ __forceinline__ long load_token(const EmbedArgs& a, long i) {
    return a.token_bits == 64 ? ((const int64_t*)a.tokens)[i] : (long)((const int32_t*)a.tokens)[i];
}

__device__ __forceinline__ bool position_valid(const EmbedArgs& a, long i) {
    if (!a.lengths) return true;
    const int b = (int)(i / a.T);
    return (int)(i - (long)b * a.T) < seq_length(a.lengths, b, a.T, a.status);
}

// G lanes a row, U rows a lane group.
template <class T, int G, int U>
__global__ __launch_bounds__(256) void k_embed(const EmbedArgs a) {
    constexpr int V = Piece<T>::V, RPB = 256 / G;
    const int N = a.N, lane = threadIdx.x % G;
    const long n = (long)a.B * a.T;
    const long i0 = ((long)blockIdx.x * RPB + threadIdx.x / G) * U;
    const T* src[U];
    float mul[U];
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long i = i0 + u;
        live[u] = false;
        mul[u] = 0.0f;
        src[u] = (const T*)a.table;
        if (i < n && position_valid(a, i)) {
            const long tok = load_token(a, i);
            if (tok >= 0 && tok < a.V) {
                live[u] = true;
                src[u] += tok * N;
            } else {
                mul[u] = __builtin_nanf("");
                if (a.status && lane == 0) atomicOr(a.status, 1);
            }
        }
    }
    for (int c = lane * V; c < N; c += G * V) {
        float x[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) load_piece<T>(src[u] + c, live[u] ? N - c : 0, x[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u >= n) break;
#pragma unroll
            for (int j = 0; j < V; ++j) x[u][j] = live[u] ? x[u][j] * a.scale : mul[u];
            store_piece<T>((T*)a.out + (i0 + u) * N + c, N - c, x[u]);
        }
    }
}

// ------------------------------------------------------------------ sort by token
// Least-significant-digit radix sort of (key, position), 8 bits a pass, stable.  The key of a
// position that counts for nothing (padding, a token outside [0, V)) is V: it sorts last.
constexpr int BINS = 256, TILE = 4096, SORT_NT = 256, PER = TILE / SORT_NT;

__device__ __forceinline__ uint32_t first_key(const EmbedArgs& a, long i) {
    if (!position_valid(a, i)) return (uint32_t)a.V;
    const long tok = load_token(a, i);
    if (tok >= 0 && tok < a.V) return (uint32_t)tok;
    if (a.status) atomicOr(a.status, 1);
    return (uint32_t)a.V;
}

// counts [BINS][nblk] of this pass's digit
__global__ __launch_bounds__(SORT_NT) void k_sort_count(const EmbedArgs a, const uint32_t* keys,
                                                        int n, int shift, int nblk, int* counts) {
    __shared__ int h[BINS];
    h[threadIdx.x] = 0;
    __syncthreads();
    const int base = blockIdx.x * TILE;
    for (int p = 0; p < PER; ++p) {
        const int i = base + p * SORT_NT + threadIdx.x;
        if (i < n) {
            const uint32_t key = keys ? keys[i] : first_key(a, i);
            atomicAdd(&h[(key >> shift) & (BINS - 1)], 1);
        }
    }
    __syncthreads();
    counts[(size_t)threadIdx.x * nblk + blockIdx.x] = h[threadIdx.x];
}

// exclusive scan of one bin's counts over the blocks; totals [BINS].  grid BINS, block 256
__global__ __launch_bounds__(256) void k_sort_scan(int* counts, int nblk, int* totals) {
    __shared__ int wsum[4];
    int* c = counts + (size_t)blockIdx.x * nblk;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int carry = 0;
    for (int j0 = 0; j0 < nblk; j0 += 256) {
        const int j = j0 + threadIdx.x;
        const int v = j < nblk ? c[j] : 0;
        int s = v;
        for (int off = 1; off < 64; off <<= 1) {
            const int t = __shfl_up(s, off, 64);
            if (lane >= off) s += t;
        }
        if (lane == 63) wsum[w] = s;
        __syncthreads();
        int before = carry;
        for (int i = 0; i < w; ++i) before += wsum[i];
        if (j < nblk) c[j] = before + s - v;
        for (int i = 0; i < 4; ++i) carry += wsum[i];
        __syncthreads();
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

// Stable scatter of one tile.  A wavefront takes PER * 64 consecutive items, 64 at a time: the
// lanes with the same digit find each other with one ballot a bit, the lowest of them takes
// their places from the wavefront's running count.
__global__ __launch_bounds__(SORT_NT) void k_sort_scatter(const EmbedArgs a, const uint32_t* keys,
                                                          const int* pos, int n, int shift, int nblk,
                                                          const int* counts, const int* totals,
                                                          uint32_t* keys_out, int* pos_out) {
    __shared__ int run[SORT_NT / 64][BINS];
    __shared__ int wsum[4];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    for (int i = 0; i < SORT_NT / 64; ++i) run[i][tid] = 0;
    __syncthreads();
    const int base = blockIdx.x * TILE + w * PER * 64;
    uint32_t key[PER];
    int rank[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int i = base + p * 64 + lane;
        key[p] = 0;
        if (i < n) key[p] = keys ? keys[i] : first_key(a, i);
        const uint32_t d = (key[p] >> shift) & (BINS - 1);
        uint64_t same = __ballot(i < n);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const bool bit = (d >> b) & 1;
            const uint64_t m = __ballot(bit);
            same &= bit ? m : ~m;
        }
        const int before = __popcll(same & ((1ull << lane) - 1));
        int start = 0;
        if (i < n) start = run[w][d];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (i < n && before == 0) run[w][d] = start + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        rank[p] = start + before;
    }
    __syncthreads();
    // digit start = items of smaller digits + this digit's items in earlier tiles, waves
    {
        const int v = totals[tid];
        int s = v;
        for (int off = 1; off < 64; off <<= 1) {
            const int t = __shfl_up(s, off, 64);
            if (lane >= off) s += t;
        }
        if (lane == 63) wsum[w] = s;
        __syncthreads();
        int at = s - v + counts[(size_t)tid * nblk + blockIdx.x];
        for (int i = 0; i < w; ++i) at += wsum[i];
        for (int i = 0; i < SORT_NT / 64; ++i) {
            const int c = run[i][tid];
            run[i][tid] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int i = base + p * 64 + lane;
        if (i < n) {
            const int to = run[w][(key[p] >> shift) & (BINS - 1)] + rank[p];
            keys_out[to] = key[p];
            pos_out[to] = pos ? pos[i] : i;
        }
    }
}

// ------------------------------------------------------------------ sums over runs
__global__ __launch_bounds__(256) void k_grad_fill(char* out, size_t pieces, int ntail) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    const uint4 zero{0, 0, 0, 0};
    if (i < pieces) __builtin_memcpy(out + i * 16, &zero, 16);
    if (blockIdx.x == 0 && (int)threadIdx.x < ntail) out[pieces * 16 + threadIdx.x] = 0;
}

// One wavefront adds the rows of one chunk over 64 pieces of columns.
// Partial rows: part[chunk][0] = the run that comes from the chunk before, part[chunk][1] =
// the run that starts here and goes on.  grid (ceil(nchunks / 4), column slabs), block 256
template <class T>
__global__ __launch_bounds__(256) void k_grad_chunks(const EmbedArgs a, const uint32_t* keys,
                                                     const int* pos, int n, int R, int nchunks,
                                                     float* part) {
    constexpr int V = Piece<T>::V;
    const int N = a.N, lane = threadIdx.x & 63;
    const int chunk = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    if (chunk >= nchunks) return;
    const int c = (blockIdx.y * 64 + lane) * V;
    const int r0 = chunk * R, r1 = min(n, r0 + R);
    const T* g = (const T*)a.grad_out;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    bool from_before = r0 > 0 && keys[r0 - 1] == keys[r0];
    uint32_t cur = keys[r0];
    for (int r = r0; r < r1; ++r) {
        const uint32_t key = keys[r];
        if (key != cur) {
            if (from_before) {
                float* p = part + (size_t)chunk * 2 * N + c;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (c + i < N) p[i] = acc[i];
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] *= a.scale;
                store_piece<T>((T*)a.out + (size_t)cur * N + c, N - c, acc);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.0f;
            from_before = false;
            cur = key;
        }
        if (key >= (uint32_t)a.V) return;      // the positions that count for nothing
        float x[V];
        load_piece<T>(g + (size_t)pos[r] * N + c, N - c, x);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += x[i];
    }
    const bool goes_on = r1 < n && keys[r1] == cur;
    if (from_before || goes_on) {
        float* p = part + ((size_t)chunk * 2 + (from_before ? 0 : 1)) * N + c;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i < N) p[i] = acc[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= a.scale;
        store_piece<T>((T*)a.out + (size_t)cur * N + c, N - c, acc);
    }
}

// The run that starts in this chunk and goes on: its partial rows, in order.  The 16 wavefronts
// take consecutive shares of them.  grid (nchunks, ceil(N / 64)), block 1024
template <class T>
__global__ __launch_bounds__(1024) void k_grad_join(const EmbedArgs a, const uint32_t* keys, int n,
                                                    int R, int nchunks, const float* part) {
    __shared__ float s[16][64];
    const int chunk = blockIdx.x, N = a.N;
    const int r1 = (chunk + 1) * R;
    if (r1 >= n) return;
    const uint32_t key = keys[r1];
    if (keys[r1 - 1] != key || key >= (uint32_t)a.V) return;
    // started before this chunk: its first chunk joins it
    const int r0 = chunk * R;
    if (r0 > 0 && keys[r0 - 1] == key) return;
    // last row of the run: the first row past it, by halving
    int lo = r1, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (keys[mid] == key) lo = mid + 1; else hi = mid;
    }
    const int last = (lo - 1) / R;             // chunk that holds the run's last row
    const int m = last - chunk;                // partial rows after the first
    const int w = threadIdx.x >> 6, c = blockIdx.y * 64 + (threadIdx.x & 63);
    const int per = (m + 15) / 16;
    float v = 0.0f;
    if (c < N) {
        if (w == 0) v = part[((size_t)chunk * 2 + 1) * N + c];
        const int q1 = min(m, (w + 1) * per);
        for (int q = w * per; q < q1; ++q) v += part[(size_t)(chunk + 1 + q) * 2 * N + c];
    }
    s[w][threadIdx.x & 63] = v;
    __syncthreads();
    if (w == 0 && c < N) {
        for (int i = 1; i < 16; ++i) v += s[i][threadIdx.x];
        ((T*)a.out)[(size_t)key * N + c] = (T)(v * a.scale);
    }
}

struct GradLayout {
    int n, nblk, passes, R, nchunks;
    size_t key[2], pos[2], counts, totals, part, total;
};

GradLayout grad_layout(int B, int T, int V, int N, int dtype) {
    (void)dtype;
    GradLayout l{};
    l.n = B * T;
    l.nblk = (l.n + TILE - 1) / TILE;
    int bits = 1;
    while (((long)V >> bits) != 0) ++bits;
    l.passes = (bits + 7) / 8;
    // rows per chunk: enough chunks to fill the device, few enough partial rows
    l.R = 16;
    while (l.R < 128 && l.n / l.R > 4096) l.R *= 2;
    l.nchunks = (l.n + l.R - 1) / l.R;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off += (bytes + 255) / 256 * 256;
        return o;
    };
    for (int i = 0; i < 2; ++i) {
        l.key[i] = take((size_t)l.n * 4);
        l.pos[i] = take((size_t)l.n * 4);
    }
    l.counts = take((size_t)BINS * l.nblk * 4);
    l.totals = take(BINS * 4);
    l.part = take((size_t)l.nchunks * 2 * N * 4);
    l.total = off;
    return l;
}

template <class T>
hipError_t run_embed(const EmbedArgs& a, hipStream_t stream) {
    constexpr int V = Piece<T>::V;
    const long n = (long)a.B * a.T;
    const int np = (a.N + V - 1) / V;
    auto go = [&](auto g) {
        constexpr int G = decltype(g)::value, U = 4;
        const long per = (256 / G) * U;
        hipLaunchKernelGGL((k_embed<T, G, U>), dim3((unsigned)((n + per - 1) / per)), dim3(256), 0,
                           stream, a);
        return hipGetLastError();
    };
    if (np <= 4) return go(std::integral_constant<int, 4>());
    if (np <= 16) return go(std::integral_constant<int, 16>());
    return go(std::integral_constant<int, 64>());
}

template <class T>
hipError_t run_embed_grad(const EmbedArgs& a, char* ws, hipStream_t stream) {
    constexpr int V = Piece<T>::V;
    const GradLayout l = grad_layout(a.B, a.T, a.V, a.N, a.dtype);
    const size_t bytes = (size_t)a.V * a.N * sizeof(T);
    const size_t pieces = bytes / 16;
    hipLaunchKernelGGL(k_grad_fill, dim3((unsigned)((pieces + 255) / 256 + 1)), dim3(256), 0, stream,
                       (char*)a.out, pieces, (int)(bytes - pieces * 16));
    const uint32_t* keys = nullptr;
    const int* pos = nullptr;
    int* counts = (int*)(ws + l.counts);
    int* totals = (int*)(ws + l.totals);
    for (int p = 0; p < l.passes; ++p) {
        uint32_t* ko = (uint32_t*)(ws + l.key[p & 1]);
        int* po = (int*)(ws + l.pos[p & 1]);
        hipLaunchKernelGGL(k_sort_count, dim3(l.nblk), dim3(SORT_NT), 0, stream, a, keys, l.n, 8 * p,
                           l.nblk, counts);
        hipLaunchKernelGGL(k_sort_scan, dim3(BINS), dim3(256), 0, stream, counts, l.nblk, totals);
        hipLaunchKernelGGL(k_sort_scatter, dim3(l.nblk), dim3(SORT_NT), 0, stream, a, keys, pos, l.n,
                           8 * p, l.nblk, counts, totals, ko, po);
        keys = ko;
        pos = po;
    }
    float* part = (float*)(ws + l.part);
    hipLaunchKernelGGL((k_grad_chunks<T>), dim3((l.nchunks + 3) / 4, (a.N + 64 * V - 1) / (64 * V)),
                       dim3(256), 0, stream, a, keys, pos, l.n, l.R, l.nchunks, part);
    hipLaunchKernelGGL((k_grad_join<T>), dim3(l.nchunks, (a.N + 63) / 64), dim3(1024), 0, stream, a,
                       keys, l.n, l.R, l.nchunks, part);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_embed(const EmbedArgs& a, hipStream_t stream) {
    return a.dtype == SEMICRF_F32 ? run_embed<float>(a, stream) : run_embed<bf16>(a, stream);
}

size_t embed_grad_bytes(int B, int T, int V, int N, int dtype) {
    return grad_layout(B, T, V, N, dtype).total;
}

hipError_t launch_embed_grad(const EmbedArgs& a, void* ws, hipStream_t stream) {
    return a.dtype == SEMICRF_F32 ? run_embed_grad<float>(a, (char*)ws, stream)
                                  : run_embed_grad<bf16>(a, (char*)ws, stream);
}

}  // namespace semicrf
