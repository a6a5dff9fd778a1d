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
// that appear once cost the same reads, and the same inputs give the same bits.  Beyond 2 million
// positions the partial rows of such a token grow with the batch (one a 256 positions), and one
// workgroup a column slab adds them up.
#include "common.h"
#include "encoder.h"

namespace semicrf {

namespace {

// Keys of U positions (b * T + t, below 2^30): the token, V where the position counts for nothing
// (padding, past n), V + 1 for a token outside [0, V).  The loads do not wait for one another.
template <int U>
__device__ __forceinline__ void load_keys(const EmbedArgs& a, const unsigned (&at)[U], unsigned n,
                                          uint32_t (&key)[U]) {
    long tok[U];
    int t[U], L[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        t[u] = 0;
        L[u] = at[u] < n;
    }
    if (a.lengths) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned i = min(at[u], n - 1), b = i / (unsigned)a.T;
            t[u] = (int)(i - b * (unsigned)a.T);
            L[u] = a.lengths[b];
        }
    }
    if (a.token_bits == 64) {
#pragma unroll
        for (int u = 0; u < U; ++u) tok[u] = ((const int64_t*)a.tokens)[min(at[u], n - 1)];
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) tok[u] = ((const int32_t*)a.tokens)[min(at[u], n - 1)];
    }
    bool bad = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool known = tok[u] >= 0 && tok[u] < a.V, in = at[u] < n;
        if (a.lengths) bad |= in && (L[u] < 0 || L[u] > a.T);
        const bool live = in && t[u] < L[u];
        bad |= live && !known;
        key[u] = !live ? (uint32_t)a.V : known ? (uint32_t)tok[u] : (uint32_t)a.V + 1;
    }
    if (bad && a.status) atomicOr(a.status, 1);
}

// G lanes a row, U rows a lane group, a group's rows 256 / G apart.  400,000 rows of 512 bfloat16 from
// a table of 4,096: 410 MB written in 69 us (5.9 TB/s; a fill reaches 6.9, a copy 5.2).
template <class T, int G, int U, bool STREAM, bool NARROW>
__global__ __launch_bounds__(256) void k_embed(const EmbedArgs a) {
    using Pc = Piece<T, NARROW>;
    constexpr int V = Pc::V, RPB = 256 / G;
    const int N = a.N, lane = threadIdx.x % G;
    const unsigned n = (unsigned)a.B * a.T;
    const unsigned i0 = a.first + blockIdx.x * RPB * U + threadIdx.x / G;
    unsigned at[U];
    uint32_t key[U];
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = i0 + u * RPB;
    load_keys<U>(a, at, n, key);
    for (int i = lane; i * V < N; i += G) {
        const Pc pc(i, N);
        raw_piece x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool known = key[u] < (uint32_t)a.V;
            x[u] = load_raw((const T*)a.table + (size_t)(known ? key[u] : 0) * N, pc, N);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (at[u] >= n) break;
            const float fill = key[u] > (uint32_t)a.V ? __builtin_nanf("") : 0.0f;
            float y[V];
            unpack<T>(x[u], y);
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = key[u] < (uint32_t)a.V ? y[j] * a.scale : fill;
            store_piece<T, STREAM>((T*)a.out + (size_t)at[u] * N, pc, N, y);
        }
    }
}

// ------------------------------------------------------------------ sort by token
// Least-significant-digit radix sort of (key, position), 8 bits a pass, stable.  The key of a
// position that counts for nothing is V here, for unknown tokens too: it sorts last.
//
// counts says how many items of each tile have each digit of the pass; the first pass counts in
// k_grad_begin.
// In tiles, beyond what one workgroup sorts.  Up to 64 tiles every scatter workgroup adds the counts
// up by itself and they lie tile by tile; beyond, k_sort_scan does it once, digit by digit.
// 400,000 positions of 6 tokens (one pass) 16 us in three launches, 16,000 of 50,001 (two passes)
// 14 us beside clearing 102 MB of gradient: bound by launches and the latency of a tile.
constexpr int BINS = 256, SCAN_TILES = 64, TILE = 1024, SORT_NT = 256, PER = TILE / SORT_NT;

struct SortArgs {
    const uint32_t* keys;    // NULL: the tokens themselves, positions in order
    const int* pos;          // with keys
    int n, shift, ntiles;
    int by_digit, by_tile;   // strides of the counts
    int* counts;             // counts, or exclusive over the tiles once scanned
    const int* totals;       // NULL: counts are not scanned yet
    uint32_t* keys_out;
    int* pos_out;
};

// One tile's count of a digit.  Each wavefront counts for itself: few distinct tokens make the
// atomics of a counter wait for each other.
__device__ __forceinline__ void count_tile(const uint32_t (&key)[PER], const unsigned (&from)[PER], int n,
                                           int shift, int* counts) {
    __shared__ int h[4][BINS];
    const int w = threadIdx.x >> 6;
    for (int i = 0; i < 4; ++i) h[i][threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < PER; ++p)
        if (from[p] < (unsigned)n) atomicAdd(&h[w][(key[p] >> shift) & (BINS - 1)], 1);
    __syncthreads();
    *counts = h[0][threadIdx.x] + h[1][threadIdx.x] + h[2][threadIdx.x] + h[3][threadIdx.x];
}

// grid ntiles
__global__ __launch_bounds__(256) void k_sort_count(const SortArgs s) {
    uint32_t key[PER];
    unsigned from[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        from[p] = blockIdx.x * TILE + p * SORT_NT + threadIdx.x;
        key[p] = s.keys[min(from[p], (unsigned)s.n - 1)];
    }
    count_tile(key, from, s.n, s.shift, s.counts + (size_t)threadIdx.x * s.by_digit + (size_t)blockIdx.x * s.by_tile);
}

// Clears `bytes` of the gradient (rows of tokens that do not appear stay 0): workgroup `block` of
// `blocks`.
__device__ __forceinline__ void clear_share(void* p, size_t bytes, int block, int blocks) {
    char* out = (char*)p;
    const size_t pieces = bytes / 16, step = (size_t)blocks * blockDim.x;
    const raw_piece zero = {0, 0, 0, 0};
    const size_t first = (size_t)block * blockDim.x + threadIdx.x;
    for (size_t i = first; i < pieces; i += step) *(loose_piece*)(out + i * 16) = zero;
    if (first < bytes - pieces * 16) out[pieces * 16 + first] = 0;
}

// Workgroups 0 .. ntiles - 1 count the first digit of a tile; the others clear the gradient.
__global__ __launch_bounds__(256) void k_grad_begin(const EmbedArgs a, const SortArgs s, size_t bytes) {
    if (blockIdx.x >= (unsigned)s.ntiles) return clear_share(a.out, bytes, blockIdx.x - s.ntiles, gridDim.x - s.ntiles);
    uint32_t key[PER];
    unsigned from[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) from[p] = blockIdx.x * TILE + p * SORT_NT + threadIdx.x;
    load_keys<PER>(a, from, s.n, key);
#pragma unroll
    for (int p = 0; p < PER; ++p) key[p] = min(key[p], (uint32_t)a.V);
    count_tile(key, from, s.n, 0, s.counts + (size_t)threadIdx.x * s.by_digit + (size_t)blockIdx.x * s.by_tile);
}

// Ranks of a wavefront's items among its items of the same digit, 64 at a time: the lanes with the
// same digit find each other with one ballot a bit, the lowest of them takes their places from
// the wavefront's running count `run` [BINS].
template <int N>
__device__ __forceinline__ void rank_items(const uint32_t (&key)[N], const bool (&live)[N], int shift, int* run,
                                           int (&rank)[N]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int p = 0; p < N; ++p) {
        const uint32_t d = (key[p] >> shift) & (BINS - 1);
        uint64_t same = __ballot(live[p]);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const bool bit = (d >> b) & 1;
            const uint64_t m = __ballot(bit);
            same &= bit ? m : ~m;
        }
        const int before = __popcll(same & ((1ull << lane) - 1));
        int start = 0;
        if (live[p]) start = run[d];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (live[p] && before == 0) run[d] = start + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        rank[p] = start + before;
    }
}

// Up to 4,096 positions: workgroup 0 sorts them all in LDS, a pass after the other, while the others
// clear the gradient (310 positions, two digits: 12.5 us in one launch against 15.3 in four; 16,384 this way
// would take 37 us against 28, its LDS keeping the clearing workgroups out).
constexpr int ONE_NT = 1024, ONE_N = 4, ONE_MAX = ONE_N * ONE_NT;
template <int N>
__global__ __launch_bounds__(ONE_NT) void k_grad_sort_one(const EmbedArgs a, int n, int passes, uint32_t* keys_out,
                                                          int* pos_out, size_t bytes) {
    if (blockIdx.x > 0) return clear_share(a.out, bytes, blockIdx.x - 1, gridDim.x - 1);
    constexpr int NW = ONE_NT / 64;
    __shared__ uint32_t keys[N * ONE_NT];
    __shared__ int pos[N * ONE_NT];
    __shared__ int run[NW][BINS];
    __shared__ int wsum[4];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    uint32_t key[N];
    unsigned from[N];
    bool live[N];
    int rank[N];
#pragma unroll
    for (int p = 0; p < N; ++p) {
        from[p] = w * N * 64 + p * 64 + lane;
        live[p] = from[p] < (unsigned)n;
    }
    load_keys<N>(a, from, n, key);
#pragma unroll
    for (int p = 0; p < N; ++p) key[p] = min(key[p], (uint32_t)a.V);
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = 8 * pass;
        for (int i = tid; i < NW * BINS; i += ONE_NT) (&run[0][0])[i] = 0;
        __syncthreads();
        rank_items<N>(key, live, shift, run[w], rank);
        __syncthreads();
        // start of each digit, then of each wavefront's share of it
        int total = 0, sum = 0;
        if (tid < BINS) {
            for (int i = 0; i < NW; ++i) total += run[i][tid];
            sum = total;
            for (int off = 1; off < 64; off <<= 1) {
                const int t = __shfl_up(sum, off, 64);
                if (lane >= off) sum += t;
            }
            if (lane == 63) wsum[w] = sum;
        }
        __syncthreads();
        if (tid < BINS) {
            int at = sum - total;
            for (int i = 0; i < w; ++i) at += wsum[i];
            for (int i = 0; i < NW; ++i) {
                const int v = run[i][tid];
                run[i][tid] = at;
                at += v;
            }
        }
        __syncthreads();
#pragma unroll
        for (int p = 0; p < N; ++p)
            if (live[p]) {
                const int to = run[w][(key[p] >> shift) & (BINS - 1)] + rank[p];
                keys[to] = key[p];
                pos[to] = (int)from[p];
            }
        __syncthreads();
#pragma unroll
        for (int p = 0; p < N; ++p) {
            const int i = w * N * 64 + p * 64 + lane;
            if (live[p]) {
                key[p] = keys[i];
                from[p] = pos[i];
            }
        }
    }
#pragma unroll
    for (int p = 0; p < N; ++p) {
        const int i = w * N * 64 + p * 64 + lane;
        if (live[p]) {
            keys_out[i] = key[p];
            pos_out[i] = (int)from[p];
        }
    }
}

// exclusive scan of one digit's counts over the tiles; totals [BINS].  grid BINS, block 256
__global__ __launch_bounds__(256) void k_sort_scan(int* counts, int ntiles, int* totals) {
    __shared__ int wsum[4];
    int* c = counts + (size_t)blockIdx.x * ntiles;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int carry = 0;
    for (int j0 = 0; j0 < ntiles; j0 += 256) {
        const int j = j0 + threadIdx.x;
        const int v = j < ntiles ? c[j] : 0;
        int s = v;
        for (int off = 1; off < 64; off <<= 1) {
            const int t = __shfl_up(s, off, 64);
            if (lane >= off) s += t;
        }
        if (lane == 63) wsum[w] = s;
        __syncthreads();
        int before = carry;
        for (int i = 0; i < w; ++i) before += wsum[i];
        if (j < ntiles) c[j] = before + s - v;
        for (int i = 0; i < 4; ++i) carry += wsum[i];
        __syncthreads();
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

// Stable scatter of one tile.  A wavefront takes PER * 64 consecutive items.
__global__ __launch_bounds__(SORT_NT) void k_sort_scatter(const EmbedArgs a, const SortArgs s) {
    __shared__ int run[SORT_NT / 64][BINS];
    __shared__ int wsum[4];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, n = s.n;
    for (int i = 0; i < SORT_NT / 64; ++i) run[i][tid] = 0;
    __syncthreads();
    const int base = blockIdx.x * TILE + w * PER * 64;
    uint32_t key[PER];
    unsigned from[PER];
    int rank[PER];
    bool live[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        from[p] = base + p * 64 + lane;
        live[p] = from[p] < (unsigned)n;
    }
    if (s.keys) {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const unsigned i = min(from[p], (unsigned)n - 1);
            key[p] = s.keys[i];
            from[p] = s.pos[i];
        }
    } else {
        load_keys<PER>(a, from, n, key);
#pragma unroll
        for (int p = 0; p < PER; ++p) key[p] = min(key[p], (uint32_t)a.V);
    }
    // this tile's share of its digit: items of the digit in earlier tiles
    int before_tile = 0, total = 0;
    if (s.totals) {
        before_tile = s.counts[(size_t)tid * s.by_digit + blockIdx.x];
        total = s.totals[tid];
    } else {
        constexpr int U = 16;                  // loads in flight
        for (int j0 = 0; j0 < s.ntiles; j0 += U) {
            int v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = s.counts[min(j0 + u, s.ntiles - 1) * BINS + tid];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                before_tile += j0 + u < (int)blockIdx.x ? v[u] : 0;
                total += j0 + u < s.ntiles ? v[u] : 0;
            }
        }
    }
    rank_items<PER>(key, live, s.shift, run[w], rank);
    // digit start = items of smaller digits + this digit's items in earlier tiles, wavefronts
    int sum = total;
    for (int off = 1; off < 64; off <<= 1) {
        const int t = __shfl_up(sum, off, 64);
        if (lane >= off) sum += t;
    }
    if (lane == 63) wsum[w] = sum;
    __syncthreads();
    int at = sum - total + before_tile;
    for (int i = 0; i < w; ++i) at += wsum[i];
    for (int i = 0; i < SORT_NT / 64; ++i) {
        const int v = run[i][tid];
        run[i][tid] = at;
        at += v;
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        if (live[p]) {
            const int to = run[w][(key[p] >> s.shift) & (BINS - 1)] + rank[p];
            s.keys_out[to] = key[p];
            s.pos_out[to] = from[p];
        }
    }
}

// ------------------------------------------------------------------ sums over runs
// G lanes add the rows of one chunk over G pieces of columns, U rows on their way at a time; G is 64
// but for narrow rows.  Partial rows: part[chunk][0] = the run that comes from the chunk before,
// part[chunk][1] = the run that starts here and goes on.
// Bound by HBM: 400,000 rows of 256 float32, 410 MB in 77 us (5.3 TB/s); 16,000 rows of 1,024 bfloat16
// over 50,001 tokens, 33 MB, 12 us.
// grid (ceil(nchunks / (256 / G)), column slabs), block 256
template <class T, int G, bool NARROW>
__global__ __launch_bounds__(256) void k_grad_chunks(const EmbedArgs a, const uint32_t* keys,
                                                     const int* pos, int n, int R, int nchunks,
                                                     float* part) {
    using Pc = Piece<T, NARROW>;
    constexpr int V = Pc::V, U = 8;
    const int N = a.N, lane = threadIdx.x & (G - 1);
    int chunk = blockIdx.x * (256 / G) + threadIdx.x / G;
    if constexpr (G == 64) chunk = __builtin_amdgcn_readfirstlane(chunk);
    if (chunk >= nchunks) return;
    const Pc pc(blockIdx.y * G + lane, N);
    const int r0 = chunk * R, r1 = min(n, r0 + R);
    const T* g = (const T*)a.grad_out;
    const uint32_t key_before = r0 > 0 ? keys[r0 - 1] : ~0u, key_after = r1 < n ? keys[r1] : ~0u;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    uint32_t cur = keys[r0];
    if (cur >= (uint32_t)a.V) return;          // the positions that count for nothing come last
    bool from_before = key_before == cur;
    auto flush = [&](bool goes_on) {
        if (from_before || goes_on) {
            if (pc.skip < V) store_elements(part + ((size_t)chunk * 2 + (from_before ? 0 : 1)) * N, pc.at, N, acc);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] *= a.scale;
            store_piece<T>((T*)a.out + (size_t)cur * N, pc, N, acc);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
        from_before = false;
    };
    for (int b0 = r0; b0 < r1; b0 += G) {
        // every lane keeps one row's key and position; row r of the block is read from lane r
        const int m = min(r1 - b0, G);
        const uint32_t my_key = lane < m ? keys[b0 + lane] : (uint32_t)a.V;
        const int my_pos = lane < m ? pos[b0 + lane] : 0;
        const uint64_t mask = __ballot(my_key < (uint32_t)a.V);
        const int live = G == 64 ? __popcll(mask)
                                 : __popcll((mask >> (threadIdx.x & 63 & ~(G - 1))) & ((1ull << (G & 63)) - 1));
        auto from_lane = [&](int v, int r) {
            return G == 64 ? __builtin_amdgcn_readlane(v, r) : __shfl(v, r & (G - 1), G);
        };
        raw_piece x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const T* row = g + (size_t)(unsigned)from_lane(my_pos, u) * N;
            if (u < live) x[u] = load_raw(row, pc, N);
        }
        for (int r = 0; r < live; r += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = r + U + u;
                const T* row = g + (size_t)(unsigned)from_lane(my_pos, q & (G - 1)) * N;
                if (q < live) y[u] = load_raw(row, pc, N);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t key = (uint32_t)from_lane((int)my_key, (r + u) & (G - 1));
                if (r + u < live) {
                    if (key != cur) {
                        flush(false);
                        cur = key;
                    }
                    float f[V];
                    unpack<T>(x[u], f);
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] += f[i];
                }
                x[u] = y[u];
            }
        }
        if (live < m) break;
    }
    flush(key_after == cur);
}

// The runs that start in a chunk and go on: their partial rows, in order.  A workgroup looks at `per`
// chunks (at most 64, a lane each) and takes the runs it finds one by one; CL lanes take four
// columns each, the 512 / CL groups consecutive shares of the partial rows.  Bound by latency (keys,
// search, partial rows, join): 1,563 chunks of six tokens 11 us, 16,000 rows of 1,024 columns 7 us.
// grid (ceil(nchunks / per), ceil(N / (4 CL))), block 512
template <class T, int CL>
__global__ __launch_bounds__(512) void k_grad_join(const EmbedArgs a, const uint32_t* keys, int n,
                                                   int R, int nchunks, int per, const float* part) {
    constexpr int GR = 512 / CL, U = 8;
    __shared__ float s[GR][CL][4];
    const int N = a.N, lane64 = threadIdx.x & 63, c0 = blockIdx.x * per;
    const int lane = threadIdx.x % CL, grp = threadIdx.x / CL, c = (blockIdx.y * CL + lane) * 4;
    // only a run that starts in its chunk and goes on: an earlier start is joined by its first chunk
    bool starts = false;
    uint32_t my_key = 0;
    {
        const int chunk = c0 + lane64, r0 = chunk * R, r1 = r0 + R;
        if (lane64 < per && chunk < nchunks && r1 < n) {
            my_key = keys[r1];
            const uint32_t last = keys[r1 - 1], before = r0 > 0 ? keys[r0 - 1] : ~0u;
            starts = last == my_key && my_key < (uint32_t)a.V && before != my_key;
        }
    }
    // the same in every wavefront
    for (uint64_t found = __ballot(starts); found; found &= found - 1) {
        const int i = __builtin_ctzll(found), chunk = c0 + i;
        const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)my_key, i);
        // chunks lo .. hi - 1 may end with the key, those before lo do: 64 of them asked at a time
        int lo = chunk + 1, hi = nchunks;
        while (lo < hi) {
            const int step = (hi - lo + 63) / 64, q = lo + (lane64 + 1) * step - 1;
            const bool has = q < hi && keys[min(n, (q + 1) * R) - 1] == key;
            const int yes = __popcll(__ballot(has));
            lo += yes * step;
            hi = min(hi, lo + step - 1);
        }
        // chunk lo (if any) ends with another key: the run reaches into it if its first row has the key
        const int last = lo < nchunks && keys[lo * R] == key ? lo : lo - 1;
        const int m = last - chunk;            // partial rows after the first
        const int share = (m + GR - 1) / GR;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (c < N) {
            if (grp == 0) load_elements(part + ((size_t)chunk * 2 + 1) * N, c, N, v);
            const int q1 = min(m, (grp + 1) * share);
            const float* p = part + (size_t)(chunk + 1) * 2 * N;
            for (int q = grp * share; q < q1; q += U) {
                float x[U][4];
#pragma unroll
                for (int u = 0; u < U; ++u) load_elements(p + (size_t)(q + u) * 2 * N, c, q + u < q1 ? N : 0, x[u]);
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] += x[u][j];
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) s[grp][lane][j] = v[j];
        __syncthreads();
        if (grp == 0 && c < N) {
#pragma unroll 8
            for (int q = 1; q < GR; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] += s[q][lane][j];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < N) ((T*)a.out)[(size_t)key * N + c + j] = (T)(v[j] * a.scale);
        }
    }
}

struct GradLayout {
    int n, ntiles, passes, R, nchunks;
    size_t key[2], pos[2], counts, totals, part, total;
};

GradLayout grad_layout(int B, int T, int V, int N, int es) {
    GradLayout l{};
    l.n = B * T;
    l.ntiles = (l.n + TILE - 1) / TILE;
    int bits = 1;
    while (((long)V >> bits) != 0) ++bits;
    l.passes = (bits + 7) / 8;
    // rows per chunk: about 2,048 wavefronts over the chunks and column slabs fill the device; longer
    // chunks leave fewer partial rows.  A narrow row takes a part of a wavefront; its chunks are at most
    // 8,192 up to 2 million positions (256 rows a chunk at most), so that the join has no more to do than
    // the sums (400,000 rows, sums + join: 17 + 18 us for 16 float32 columns, 13 + 28 with 16,384
    // chunks, 29 + 11 with 4,096).
    const long np = ((long)N * es + 15) / 16, G = np <= 8 ? 8 : np <= 16 ? 16 : np <= 32 ? 32 : 64;
    l.R = 8;
    while (l.R < 256 && (l.n * ((np + G - 1) / G) * G / 64 / l.R > 2048 || l.n / l.R > 8192)) l.R *= 2;
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
    l.counts = take((size_t)BINS * l.ntiles * 4);
    l.totals = take(BINS * 4);
    l.part = take((size_t)l.nchunks * 2 * N * 4);
    l.total = off;
    return l;
}

template <class T>
hipError_t run_embed(const EmbedArgs& a, hipStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const long n = (long)a.B * a.T;
    const int np = (a.N + V - 1) / V;
    // Outputs past the memory-side cache (256 MB) are written as a stream: what reads them finds
    // nothing of them in a cache either way, and the table stays there.  Measured in bfloat16, the
    // lookup alone and followed by two layer norms: 410 MB 67 against 107 us, 403 against 432; 52 MB
    // 14 against 15, but 59 against 53, so smaller outputs are written as usual.
    const bool stream_out = (size_t)n * a.N * sizeof(T) > (size_t)256 << 20;
    auto go = [&](auto g) {
        constexpr int G = decltype(g)::value, U = 2;
        const long per = (256 / G) * U, most = per << 22;    // a launch holds less than 2^32 threads
        const dim3 block(256);
        EmbedArgs part = a;
        for (long first = 0; first < n; first += most) {
            part.first = (unsigned)first;
            const long rows = n - first < most ? n - first : most;
            const dim3 grid((unsigned)((rows + per - 1) / per));
            if (a.N < V) hipLaunchKernelGGL((k_embed<T, 4, U, false, true>), grid, block, 0, stream, part);
            else if (stream_out) hipLaunchKernelGGL((k_embed<T, G, U, true, false>), grid, block, 0, stream, part);
            else hipLaunchKernelGGL((k_embed<T, G, U, false, false>), grid, block, 0, stream, part);
        }
        return hipGetLastError();
    };
    if (np <= 4) return go(std::integral_constant<int, 4>());
    if (np <= 8) return go(std::integral_constant<int, 8>());
    if (np <= 16) return go(std::integral_constant<int, 16>());
    if (np <= 32) return go(std::integral_constant<int, 32>());
    return go(std::integral_constant<int, 64>());
}

template <class T>
hipError_t run_embed_grad(const EmbedArgs& a, char* ws, hipStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const GradLayout l = grad_layout(a.B, a.T, a.V, a.N, sizeof(T));
    const size_t bytes = (size_t)a.V * a.N * sizeof(T);
    SortArgs s{};
    s.n = l.n;
    s.ntiles = l.ntiles;
    s.counts = (int*)(ws + l.counts);
    const bool scan = l.ntiles > SCAN_TILES;
    s.by_digit = scan ? l.ntiles : 1;
    s.by_tile = scan ? 1 : BINS;
    const size_t fill = bytes / (256 * 64) + 1;    // four pieces a thread, up to 4,096 workgroups
    if (l.n <= ONE_MAX) {
        s.keys_out = (uint32_t*)(ws + l.key[0]);
        s.pos_out = (int*)(ws + l.pos[0]);
        const size_t share = bytes / (ONE_NT * 64) + 1;
        const dim3 grid(1 + (unsigned)(share < 1024 ? share : 1024)), block(ONE_NT);
        hipLaunchKernelGGL((k_grad_sort_one<ONE_N>), grid, block, 0, stream, a, l.n, l.passes, s.keys_out,
                           s.pos_out, bytes);
        s.keys = s.keys_out;
        s.pos = s.pos_out;
    } else {
        hipLaunchKernelGGL(k_grad_begin, dim3(l.ntiles + (unsigned)(fill < 4096 ? fill : 4096)), dim3(256), 0,
                           stream, a, s, bytes);
        for (int p = 0; p < l.passes; ++p) {
            s.shift = 8 * p;
            if (p > 0) hipLaunchKernelGGL(k_sort_count, dim3(l.ntiles), dim3(256), 0, stream, s);
            if (scan) {
                s.totals = (const int*)(ws + l.totals);
                hipLaunchKernelGGL(k_sort_scan, dim3(BINS), dim3(256), 0, stream, s.counts, l.ntiles,
                                   (int*)(ws + l.totals));
            }
            s.keys_out = (uint32_t*)(ws + l.key[p & 1]);
            s.pos_out = (int*)(ws + l.pos[p & 1]);
            hipLaunchKernelGGL(k_sort_scatter, dim3(l.ntiles), dim3(SORT_NT), 0, stream, a, s);
            s.keys = s.keys_out;
            s.pos = s.pos_out;
        }
    }
    float* part = (float*)(ws + l.part);
    auto chunks = [&](auto g) {
        constexpr int G = decltype(g)::value, CPB = 256 / G;
        const dim3 grid((l.nchunks + CPB - 1) / CPB, (a.N + G * V - 1) / (G * V));
        if (a.N < V)
            hipLaunchKernelGGL((k_grad_chunks<T, 8, true>), grid, dim3(256), 0, stream, a, s.keys, s.pos, l.n, l.R,
                               l.nchunks, part);
        else
            hipLaunchKernelGGL((k_grad_chunks<T, G, false>), grid, dim3(256), 0, stream, a, s.keys, s.pos, l.n, l.R,
                               l.nchunks, part);
    };
    const int np = (a.N + V - 1) / V;
    if (np <= 8) chunks(std::integral_constant<int, 8>());
    else if (np <= 16) chunks(std::integral_constant<int, 16>());
    else if (np <= 32) chunks(std::integral_constant<int, 32>());
    else chunks(std::integral_constant<int, 64>());
    if (l.nchunks > 1) {
        auto join = [&](auto cl) {
            constexpr int CL = decltype(cl)::value;
            const int slabs = (a.N + 4 * CL - 1) / (4 * CL);
            // about 2,048 workgroups: most chunks have no run, and one that has keeps its workgroup for
            // 5 us (12,500 chunks, each a workgroup: 93 us; 1,024 workgroups 70; 2,048 as here 28)
            const long want = ((long)l.nchunks * slabs + 2047) / 2048;
            const int per = (int)(want < 64 ? want : 64);
            hipLaunchKernelGGL((k_grad_join<T, CL>), dim3((l.nchunks + per - 1) / per, slabs), dim3(512), 0, stream, a,
                               s.keys, l.n, l.R, l.nchunks, per, part);
        };
        // narrow rows leave more groups for the partial rows
        if (a.N <= 64) join(std::integral_constant<int, 16>());
        else if (a.N <= 128) join(std::integral_constant<int, 32>());
        else if (a.N <= 256) join(std::integral_constant<int, 64>());
        else join(std::integral_constant<int, 256>());
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_embed(const EmbedArgs& a, hipStream_t stream) {
    return a.dtype == SEMICRF_F32 ? run_embed<float>(a, stream) : run_embed<bf16>(a, stream);
}

size_t embed_grad_bytes(int B, int T, int V, int N, int dtype) {
    return grad_layout(B, T, V, N, dtype == SEMICRF_F32 ? 4 : 2).total;
}

hipError_t launch_embed_grad(const EmbedArgs& a, void* ws, hipStream_t stream) {
    return a.dtype == SEMICRF_F32 ? run_embed_grad<float>(a, (char*)ws, stream)
                                  : run_embed_grad<bf16>(a, (char*)ws, stream);
}

}  // namespace semicrf
