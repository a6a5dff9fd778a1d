// Negative log-likelihood of tokens over a vocabulary, and its gradients, on gfx950.
//
//   z_mv = scale x_m . W_v,   loss_m = log sum_v exp z_mv - z_m,t(m)
//   p_mv = exp(z_mv - lse_m) - [v = t(m)]
//   dx_m = g_m scale sum_v p_mv W_v,   dW_v = scale sum_m g_m p_mv x_m
//
// The rows that have something to predict are listed and gathered first, padded with zeros to whole
// tiles, so that masked positions and padding cost nothing; their number stays on the GPU, and the
// grids are fixed: a workgroup takes tiles until none is left.
//
// Three products, one core: a tile of BA x BB results over rows of A and B that are both dense along
// the contracted axis, 128 bytes of each row a step, through LDS.
//   scores    A = W,   B = x        the log sum (k_nll_scores<false>), p in pieces of the vocabulary (<true>)
//   dx        A = W^T, B = p
//   dW        A = x^T, B = p^T
// Scores are summed and exponentiated in registers; a lane holds scores of the same rows of x for all
// tiles of the vocabulary it sees, so that maximum and sum run along without an exchange.
//
// Rounding (bfloat16): scores are exact products summed in fp32.  p, W and x enter the second
// products in fp16, scaled by powers of two to the top of its range: W and x lose nothing within 2^29
// of their largest value, and p has 11 bits down to 2^-29, so that the gradients' own rounding is
// what is seen (p in bfloat16 would add an error as large as that).  In float32 everything is float32.
#include "common.h"
#include "encoder.h"

namespace semicrf {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
using f16 = _Float16;

constexpr float LOG2EF = 1.44269504088896f, LN2F = 0.69314718055994531f;
constexpr int ROW_TILE = 256;        // rows of x are padded to it
constexpr int STEP = 128;            // bytes of a row a step of a product takes

// what the second products' operands are held in
template <class T> struct Held { using type = float; };
template <> struct Held<bf16> { using type = f16; };

// 16 bytes of 16 rows of A and of B: lane l = 16 g + r holds, of row r, elements that both operands
// take in the same order.  The result tile holds column (row of B) r, rows (of A) 4 g .. 4 g + 3.
__device__ __forceinline__ f32x4 mma(const bf16*, raw_piece a, raw_piece b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
__device__ __forceinline__ f32x4 mma(const f16*, raw_piece a, raw_piece b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}
__device__ __forceinline__ f32x4 mma(const float*, raw_piece a, raw_piece b, f32x4 c) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], c, 0, 0, 0);
    return c;
}

// A tile: BA rows of A, BB rows of B, WA x WB wavefronts.  A step's rows lie in LDS 128 bytes apart;
// 16-byte chunk c of row r lies at place c ^ (r mod 8), so that the 16 rows a fragment is read
// from fall on different banks.
template <class T, int BA_, int BB_, int WA_, int WB_>
struct Tile {
    static constexpr int BA = BA_, BB = BB_, WA = WA_, WB = WB_;
    static constexpr int NW = WA * WB, NT = 64 * NW, MA = BA / WA / 16, MB = BB / WB / 16;
    static constexpr int LOADS_A = BA / 8 / NW, LOADS_B = BB / 8 / NW;
    static constexpr int STAGE = (BA + BB) * STEP;

    f32x4 acc[MA][MB];

    // acc = A . B over nk steps.  A and B point to the tile's first rows; rows of A past rowsA - 1 are
    // taken as that one.
    __device__ __forceinline__ void product(const char* A, unsigned lda, int rowsA, const char* B, unsigned ldb,
                                            int nk, char* lds) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int wa = wave / WB, wb = wave % WB;
        unsigned oa[LOADS_A], ob[LOADS_B];
#pragma unroll
        for (int i = 0; i < LOADS_A; ++i) {
            const int r = (i * NW + wave) * 8 + lane / 8;
            oa[i] = (unsigned)min(r, rowsA - 1) * lda + ((lane & 7) ^ (r & 7)) * 16;
        }
#pragma unroll
        for (int i = 0; i < LOADS_B; ++i) {
            const int r = (i * NW + wave) * 8 + lane / 8;
            ob[i] = (unsigned)r * ldb + ((lane & 7) ^ (r & 7)) * 16;
        }
#pragma unroll
        for (int i = 0; i < MA; ++i)
#pragma unroll
            for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        raw_piece ra[LOADS_A], rb[LOADS_B];
        const int to = (wave * 8 + lane / 8) * STEP + (lane & 7) * 16;
        for (int k = 0; k < nk; ++k) {
#pragma unroll
            for (int i = 0; i < LOADS_A; ++i) ra[i] = *(const raw_piece*)(A + (size_t)k * STEP + oa[i]);
#pragma unroll
            for (int i = 0; i < LOADS_B; ++i) rb[i] = *(const raw_piece*)(B + (size_t)k * STEP + ob[i]);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < LOADS_A; ++i) *(raw_piece*)(lds + i * NW * 8 * STEP + to) = ra[i];
#pragma unroll
            for (int i = 0; i < LOADS_B; ++i) *(raw_piece*)(lds + BA * STEP + i * NW * 8 * STEP + to) = rb[i];
            __syncthreads();
            const int r = lane & 15;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int c = ((half * 4 + lane / 16) ^ (r & 7)) * 16;
                raw_piece b[MB];
#pragma unroll
                for (int j = 0; j < MB; ++j)
                    b[j] = *(const raw_piece*)(lds + (BA + wb * (BB / WB) + j * 16 + r) * STEP + c);
#pragma unroll
                for (int i = 0; i < MA; ++i) {
                    const raw_piece a = *(const raw_piece*)(lds + (wa * (BA / WA) + i * 16 + r) * STEP + c);
#pragma unroll
                    for (int j = 0; j < MB; ++j) acc[i][j] = mma((const T*)nullptr, a, b[j], acc[i][j]);
                }
            }
        }
        __syncthreads();
    }
};

// ------------------------------------------------------------------ rows that have a target
// What stays on the GPU between the launches of a call
struct Control {
    int rows;                // listed rows
    unsigned max_x, max_w, max_g;      // bits of the largest finite |x|, |W| and |grad_loss|
};

__device__ __forceinline__ int64_t target_at(const NllArgs& a, unsigned row) {
    return a.target_bits == 64 ? ((const int64_t*)a.targets)[row] : ((const int32_t*)a.targets)[row];
}

// Row -> whether it is listed; NaN: its target is out of range
__device__ __forceinline__ bool listed(const NllArgs& a, unsigned row, bool& beyond, int& target) {
    const unsigned b = row / (unsigned)a.T, t = row - b * (unsigned)a.T;
    beyond = false;
    if (a.lengths && (int)t >= seq_length(a.lengths, b, a.T, a.status)) return false;
    const int64_t v = target_at(a, row);
    beyond = v >= a.V;
    target = (int)v;
    return v >= 0 && !beyond;
}

constexpr int LIST = 4096, LIST_THREADS = 1024, LIST_EACH = LIST / LIST_THREADS;

// counts[block] = listed rows of the block's 4,096; clears the control block
__global__ __launch_bounds__(LIST_THREADS) void k_nll_count(const NllArgs a, Control* ctl, int* counts) {
    __shared__ int s[LIST_THREADS / 64];
    const unsigned rows = (unsigned)a.B * a.T, first = blockIdx.x * (unsigned)LIST + threadIdx.x * LIST_EACH;
    int n = 0;
    for (int i = 0; i < LIST_EACH; ++i) {
        bool beyond;
        int target;
        if (first + i < rows) n += listed(a, first + i, beyond, target);
    }
    for (int off = 32; off >= 1; off >>= 1) n += __shfl_xor(n, off, 64);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
        n = 0;
        for (int i = 0; i < LIST_THREADS / 64; ++i) n += s[i];
        counts[blockIdx.x] = n;
        if (blockIdx.x == 0) *ctl = Control{0, 0, 0, 0};
    }
}

// What a listed row carries into the products
struct Listed {
    int* row;                // its place among all rows
    int* target;
    float *lse, *grad;       // gradients only
    int* place;              // [all rows] its number in the list, or -1 (gradients only)
};

template <bool GRAD>
__global__ __launch_bounds__(LIST_THREADS) void k_nll_list(const NllArgs a, Control* ctl, const int* counts,
                                                           Listed list) {
    __shared__ int s[LIST_THREADS / 64], before[LIST_THREADS / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const unsigned rows = (unsigned)a.B * a.T, first = blockIdx.x * (unsigned)LIST + threadIdx.x * LIST_EACH;
    int n = 0, prev = 0, target[LIST_EACH];
    bool is[LIST_EACH];
    for (unsigned i = threadIdx.x; i < blockIdx.x; i += LIST_THREADS) prev += counts[i];
    for (int off = 32; off >= 1; off >>= 1) prev += __shfl_xor(prev, off, 64);
#pragma unroll
    for (int i = 0; i < LIST_EACH; ++i) {
        const unsigned row = first + i;
        bool beyond = false;
        is[i] = row < rows && listed(a, row, beyond, target[i]);
        n += is[i];
        if (row >= rows) continue;
        if (beyond && a.status) atomicOr(a.status, 1);
        if (GRAD) {
            if (!is[i]) list.place[row] = -1;
        } else if (!is[i]) {
            a.loss[row] = beyond ? __builtin_nanf("") : 0.0f;
            if (a.lse) a.lse[row] = 0.0f;
        }
    }
    int upto = n;
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(upto, off, 64);
        if (lane >= off) upto += v;
    }
    if (lane == 63) s[wave] = upto;
    if (lane == 0) before[wave] = prev;
    __syncthreads();
    int at = upto - n;
    for (int i = 0; i < LIST_THREADS / 64; ++i) {
        at += before[i];
        if (i < wave) at += s[i];
    }
    unsigned most = 0;
#pragma unroll
    for (int i = 0; i < LIST_EACH; ++i) {
        const unsigned row = first + i;
        if (!is[i]) continue;
        list.row[at] = (int)row;
        list.target[at] = target[i];
        if (GRAD) {
            const float g = a.grad_loss[row];
            list.lse[at] = a.lse_in[row] * LOG2EF;
            list.grad[at] = g;
            list.place[row] = at;
            const unsigned bits = __float_as_uint(g) & 0x7fffffffu;
            if (bits < 0x7f800000u) most = max(most, bits);
        }
        ++at;
    }
    if (GRAD) {
        for (int off = 32; off >= 1; off >>= 1) most = max(most, (unsigned)__shfl_xor((int)most, off, 64));
        if (lane == 0 && most) atomicMax(&ctl->max_g, most);
    }
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == LIST_THREADS - 1) ctl->rows = at;
}

__host__ __device__ __forceinline__ int tiles(int rows, int tile) { return (rows + tile - 1) / tile; }

// dst [rows][ld] = src rows (index: which; NULL: in order) of N elements, zeros beyond N and in rows
// past the last up to a whole tile.  A wavefront a row.  max: the largest finite magnitude.
template <class T>
__global__ __launch_bounds__(256) void k_nll_rows(const T* src, const int* index, const Control* ctl, int rows, int N,
                                                  T* dst, int ld, int pad) {
    constexpr int V = 16 / sizeof(T);
    if (ctl) rows = ctl->rows;
    const int r = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (r >= tiles(rows, pad) * pad) return;
    T* to = dst + (size_t)r * ld;
    const T* from = src + (size_t)(r < rows ? (index ? index[r] : r) : 0) * N;
    for (int c = lane * V; c < ld; c += 64 * V) {
        raw_piece x = {0, 0, 0, 0};
        if (r < rows) {
            if (c + V <= N) {
                x = *(const loose_piece*)(from + c);
            } else {
                T t[V];
#pragma unroll
                for (int i = 0; i < V; ++i) t[i] = c + i < N ? from[c + i] : (T)0.0f;
                __builtin_memcpy(&x, t, 16);
            }
        }
        *(raw_piece*)(to + c) = x;
    }
}

// The largest finite magnitude of `rows` rows of N elements: a fixed grid
template <class T>
__global__ __launch_bounds__(256) void k_nll_max(const T* src, const Control* ctl, long n, int N, unsigned* out) {
    if (ctl) n = (long)ctl->rows * N;
    constexpr int V = 16 / sizeof(T);
    unsigned most = 0;
    auto see = [&](float x) {
        const unsigned bits = __float_as_uint(x) & 0x7fffffffu;
        if (bits < 0x7f800000u) most = max(most, bits);
    };
    const long step = (long)gridDim.x * 256 * V;
    long i = ((long)blockIdx.x * 256 + threadIdx.x) * V;
    for (; i + V <= n; i += step) {
        const raw_piece r = *(const loose_piece*)(src + i);
        float x[V];
        unpack<T>(r, x);
#pragma unroll
        for (int j = 0; j < V; ++j) see(x[j]);
    }
    for (; i < n; ++i) see((float)src[i]);
    for (int off = 32; off >= 1; off >>= 1) most = max(most, (unsigned)__shfl_xor((int)most, off, 64));
    if ((threadIdx.x & 63) == 0 && most) atomicMax(out, most);
}

// The power of two that brings a largest magnitude to [2^14, 2^15)
template <class H>
__device__ __forceinline__ float held_scale(unsigned bits) {
    if (sizeof(H) == 4 || bits == 0) return 1.0f;
    const int e = max((int)(bits >> 23) - 126, -100);
    return __uint_as_float((unsigned)(127 + 15 - e) << 23);
}
// p's scale: |p| <= 1
template <class H>
constexpr float P_SCALE = sizeof(H) == 4 ? 1.0f : 32768.0f;

// What the rows' gradients are divided by in p^T: the largest one
__device__ __forceinline__ float grad_unit(unsigned bits) { return fmaxf(__uint_as_float(bits), 0x1p-120f); }

// dst [N][ldd] = the transpose of src [rows][ld], scaled, zeros in columns past the rows up to a whole tile
template <class T, class H>
__global__ __launch_bounds__(256) void k_nll_transpose(const T* src, const Control* ctl, bool listed_rows, int rows,
                                                       int N, int ld, const unsigned* most, H* dst, size_t ldd,
                                                       int pad) {
    __shared__ H s[64][64 + 8 / sizeof(H) * 1];
    if (listed_rows) rows = ctl->rows;
    const int r0 = blockIdx.x * 64, c0 = blockIdx.y * 64;
    if (r0 >= tiles(rows, pad) * pad) return;
    const float f = held_scale<H>(*most);
    const int cx = threadIdx.x & 63, ry = threadIdx.x >> 6;
    for (int r = ry; r < 64; r += 4) {
        const bool in = r0 + r < rows && c0 + cx < N;
        s[r][cx] = (H)(in ? (float)src[(size_t)(r0 + r) * ld + c0 + cx] * f : 0.0f);
    }
    __syncthreads();
    for (int c = ry; c < 64; c += 4)
        if (c0 + c < N) dst[(size_t)(c0 + c) * ldd + r0 + cx] = s[cx][c];
}

// ------------------------------------------------------------------ scores
// Workgroups in the order in which their tiles share rows: each of the 8 chiplets (which have an L2
// cache each, and to which consecutive workgroups go in turn) takes consecutive numbers.
__device__ __forceinline__ int ordered_block() {
    return (blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8;
}

// How many workgroups share the vocabulary of a tile of rows: the number that leaves the least for the
// busiest one.  All lanes get the same.
__device__ __forceinline__ int vocab_split(int mt, int vt, int wgs) {
    const int s = (threadIdx.x & 63) + 1;
    unsigned cost = 0xffffffffu;
    if (s <= vt && (s == 1 || mt * s <= 4 * wgs)) cost = (unsigned)(tiles(mt * s, wgs) * tiles(vt, s));
    unsigned long long key = ((unsigned long long)cost << 8) | (unsigned)s;
    for (int off = 32; off >= 1; off >>= 1) {
        const unsigned long long o = __shfl_xor(key, off, 64);
        key = o < key ? o : key;
    }
    return __builtin_amdgcn_readfirstlane((int)(key & 0xff));
}

struct Scores {
    const char *w, *x;
    unsigned ldw, ldx;       // bytes
    int V, nk;
    float scale;             // to log2 units
};

// part[(item, wavefront row)][BB] = (maximum, sum) of the scores of a share of the vocabulary, item =
// tile of rows * split + share; at_target[row] = the target's score.  All in log2 units.
template <class T, class Tl>
__global__ __launch_bounds__(Tl::NT) void k_nll_scores(const Scores p, const Control* ctl, const int* target,
                                                       float2* part, float* at_target) {
    __shared__ __align__(16) char lds[Tl::STAGE];
    const int mt = tiles(ctl->rows, Tl::BB), vt = tiles(p.V, Tl::BA), S = vocab_split(mt, vt, gridDim.x);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wa = wave / Tl::WB, wb = wave % Tl::WB;
    for (int item = ordered_block(); item < mt * S; item += gridDim.x) {
        const int m0 = item / S * Tl::BB, share = item % S;
        const int col = wb * (Tl::BB / Tl::WB) + (lane & 15);
        float top[Tl::MB], sum[Tl::MB];
        int tgt[Tl::MB];
#pragma unroll
        for (int j = 0; j < Tl::MB; ++j) {
            top[j] = -__builtin_inff();
            sum[j] = 0.0f;
            const int m = m0 + col + j * 16;
            tgt[j] = m < ctl->rows ? target[m] : -1;
        }
        for (int v = share * vt / S; v < (share + 1) * vt / S; ++v) {
            Tl t;
            t.product(p.w + (size_t)v * Tl::BA * p.ldw, p.ldw, p.V - v * Tl::BA, p.x + (size_t)m0 * p.ldx, p.ldx, p.nk,
                      lds);
            const int first = v * Tl::BA + wa * (Tl::BA / Tl::WA) + lane / 16 * 4;
#pragma unroll
            for (int j = 0; j < Tl::MB; ++j) {
                float z[Tl::MA][4], most = top[j];
#pragma unroll
                for (int i = 0; i < Tl::MA; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int at = first + i * 16 + k;
                        z[i][k] = at < p.V ? t.acc[i][j][k] * p.scale : -__builtin_inff();
                        most = fmaxf(most, z[i][k]);
                        if (at == tgt[j]) at_target[m0 + col + j * 16] = z[i][k];
                    }
                const float ref = most == -__builtin_inff() ? 0.0f : most;
                float s = sum[j] * fast_exp2(top[j] - ref);
#pragma unroll
                for (int i = 0; i < Tl::MA; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s += fast_exp2(z[i][k] - ref);
                sum[j] = s;
                top[j] = most;
            }
        }
#pragma unroll
        for (int j = 0; j < Tl::MB; ++j) {       // the four lanes of a row
#pragma unroll
            for (int off = 16; off < 64; off <<= 1) {
                const float om = __shfl_xor(top[j], off, 64), os = __shfl_xor(sum[j], off, 64);
                const float most = fmaxf(top[j], om), ref = most == -__builtin_inff() ? 0.0f : most;
                sum[j] = sum[j] * fast_exp2(top[j] - ref) + os * fast_exp2(om - ref);
                top[j] = most;
            }
            if (lane < 16)
                part[((size_t)item * Tl::WA + wa) * Tl::BB + wb * (Tl::BB / Tl::WB) + j * 16 + lane] =
                    float2{top[j], sum[j]};
        }
    }
}

// A thread a listed row: loss = log sum - score of the target
__global__ __launch_bounds__(256) void k_nll_loss(const Control* ctl, const int* row, const float2* part,
                                                  const float* at_target, int V, int BA, int BB, int WA, int wgs,
                                                  float* loss, float* lse) {
    const int rows = ctl->rows, mt = tiles(rows, BB), S = vocab_split(mt, tiles(V, BA), wgs);
    const int m = blockIdx.x * 256 + threadIdx.x;
    if (m >= rows) return;
    float top = -__builtin_inff();
    const float2* p = part + (size_t)(m / BB) * S * WA * BB + m % BB;
    for (int i = 0; i < S * WA; ++i) top = fmaxf(top, p[(size_t)i * BB].x);
    const float ref = top == -__builtin_inff() ? 0.0f : top;
    float sum = 0.0f;
    for (int i = 0; i < S * WA; ++i) sum += p[(size_t)i * BB].y * fast_exp2(p[(size_t)i * BB].x - ref);
    const float l = fast_log2(sum);
    loss[row[m]] = (l + (ref - at_target[m])) * LN2F;
    if (lse) lse[row[m]] = (l + ref) * LN2F;
}

// ------------------------------------------------------------------ gradients
// p of a piece of the vocabulary, [rows][ldp] and its transpose [piece][ldt] times the row's gradient
// over the largest one.  Zero for rows and words past the last.
template <class T, class H, class Tl>
__global__ __launch_bounds__(Tl::NT) void k_nll_p(const Scores s, const Control* ctl, const int* target,
                                                  const float* lse, const float* grad, int v0, int vt, H* p,
                                                  size_t ldp, H* pt, size_t ldt) {
    __shared__ __align__(16) char lds[Tl::STAGE];
    const int rows = ctl->rows, mt = tiles(rows, ROW_TILE) * (ROW_TILE / Tl::BB);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wa = wave / Tl::WB, wb = wave % Tl::WB;
    const float over = 1.0f / grad_unit(ctl->max_g);
    for (int tile = ordered_block(); tile < mt * vt; tile += gridDim.x) {
        // eight tiles of rows by all of the vocabulary at a time
        const int group = tile / (8 * vt), in = tile - group * 8 * vt, width = min(8, mt - group * 8);
        const int m0 = (group * 8 + in % width) * Tl::BB, v = in / width;
        Tl t;
        const int w0 = min(v0 + v * Tl::BA, s.V - 1);         // pieces may end past the vocabulary
        t.product(s.w + (size_t)w0 * s.ldw, s.ldw, s.V - w0, s.x + (size_t)m0 * s.ldx, s.ldx, s.nk, lds);
        const int first = v * Tl::BA + wa * (Tl::BA / Tl::WA) + lane / 16 * 4;
#pragma unroll
        for (int j = 0; j < Tl::MB; ++j) {
            const int m = m0 + wb * (Tl::BB / Tl::WB) + j * 16 + (lane & 15);
            const bool in_rows = m < rows;
            const float l = in_rows ? lse[m] : 0.0f, g = in_rows ? grad[m] * over : 0.0f;
            const int tgt = in_rows ? target[m] - v0 : -1;
#pragma unroll
            for (int i = 0; i < Tl::MA; ++i) {
                H out[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int at = first + i * 16 + k;
                    float q = fast_exp2(fmaf(t.acc[i][j][k], s.scale, -l));
                    if (at == tgt) q -= 1.0f;
                    if (!in_rows || v0 + at >= s.V) q = 0.0f;
                    out[k] = (H)(q * P_SCALE<H>);
                    pt[(size_t)at * ldt + m] = (H)(in_rows ? q * g * P_SCALE<H> : 0.0f);
                }
                __builtin_memcpy(p + (size_t)m * ldp + first + i * 16, out, sizeof(out));
            }
        }
    }
}

// How the contracted axis of dx is shared out: as many shares as fill the workgroups
__device__ __forceinline__ int dx_split(int mt, int at, int wgs, int nk) {
    return max(1, min(min(wgs / max(1, mt * at), nk), 16));
}

// out[share][row of B][ldo] (+)= A . B over a share of the contracted axis, fp32.  dx: the rows of B are
// the listed ones, dW: the contracted axis is theirs.
template <class H, class Tl, bool DX>
__global__ __launch_bounds__(Tl::NT) void k_nll_product(const char* A, unsigned lda, int rowsA, const char* B,
                                                        unsigned ldb, const Control* ctl, int bt, int nk, int S,
                                                        bool add, float* out, int ldo) {
    __shared__ __align__(16) char lds[Tl::STAGE];
    const int padded = tiles(ctl->rows, ROW_TILE) * ROW_TILE, at = tiles(rowsA, Tl::BA);
    if (DX) {
        bt = padded / Tl::BB;
        S = dx_split(bt, at, gridDim.x, nk);
    } else {
        nk = padded / (int)(STEP / sizeof(H));
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wa = wave / Tl::WB, wb = wave % Tl::WB;
    for (int item = ordered_block(); item < at * bt * S; item += gridDim.x) {
        const int share = item / (at * bt), tile = item - share * at * bt;
        const int group = tile / (8 * at), in = tile - group * 8 * at, width = min(8, bt - group * 8);
        const int b0 = (group * 8 + in % width) * Tl::BB, a0 = in / width * Tl::BA;
        const int k0 = (int)((long)share * nk / S), k1 = (int)((long)(share + 1) * nk / S);
        Tl t;
        t.product(A + (size_t)a0 * lda + (size_t)k0 * STEP, lda, rowsA - a0, B + (size_t)b0 * ldb + (size_t)k0 * STEP,
                  ldb, k1 - k0, lds);
#pragma unroll
        for (int j = 0; j < Tl::MB; ++j) {
            const int b = b0 + wb * (Tl::BB / Tl::WB) + j * 16 + (lane & 15);
            float* row = out + ((size_t)share * bt * Tl::BB + b) * ldo;
#pragma unroll
            for (int i = 0; i < Tl::MA; ++i) {
                const int a = a0 + wa * (Tl::BA / Tl::WA) + i * 16 + lane / 16 * 4;
                if (a >= ldo) continue;              // ldo: N up to a multiple of 4
                f32x4 x = t.acc[i][j];
                if (add) x += *(const f32x4*)(row + a);
                *(f32x4*)(row + a) = x;
            }
        }
    }
}

// A wavefront a row of x: zeros where it is not listed, else the shares' sum times the row's gradient
template <class T, class H>
__global__ __launch_bounds__(256) void k_nll_dx(const Control* ctl, const int* place, const float* grad, float scale,
                                                const float* part, int ldo, int BA, int BB, int wgs, int nk, int rows,
                                                int N, T* out) {
    const int r = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (r >= rows) return;
    const int i = place[r], bt = tiles(ctl->rows, ROW_TILE) * (ROW_TILE / BB);
    T* to = out + (size_t)r * N;
    if (i < 0) {
        for (int c = lane; c < N; c += 64) to[c] = (T)0.0f;
        return;
    }
    const int S = dx_split(bt, tiles(N, BA), wgs, nk);
    const float back = 1.0f / held_scale<H>(ctl->max_w), g = grad[i] * scale;
    for (int c = lane; c < N; c += 64) {
        float v = 0.0f;
        for (int s = 0; s < S; ++s) v += part[((size_t)s * bt * BB + i) * ldo + c];
        to[c] = (T)(v * (1.0f / P_SCALE<H>) * back * g);
    }
}

// A wavefront a word of a piece
template <class T, class H>
__global__ __launch_bounds__(256) void k_nll_dw(const Control* ctl, const float* part, int ldo, int piece, int S,
                                                float scale, int words, int N, T* out) {
    const int r = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (r >= words) return;
    const float back = 1.0f / held_scale<H>(ctl->max_x), g = grad_unit(ctl->max_g) * scale;
    for (int c = lane; c < N; c += 64) {
        float v = 0.0f;
        for (int s = 0; s < S; ++s) v += part[((size_t)s * piece + r) * ldo + c];
        out[(size_t)r * N + c] = (T)(v * (1.0f / P_SCALE<H>) * back * g);
    }
}

// ------------------------------------------------------------------ host
template <class T> using Large = Tile<T, 256, 256, 2, 4>;
template <class T> using Small = Tile<T, 128, 128, 2, 2>;

long up(long n, long m) { return (n + m - 1) / m * m; }

// Everything a call lays out in its workspace
struct Plan {
    bool large, copy_w;
    int wgs, BA, BB, WA;
    long rows, padded, V, N, ld;       // ld: elements of a padded row of x (and of W)
    long piece, pieces, vpad, ldo;
    int dw_split;
    size_t ctl, counts, list_row, list_target, list_lse, list_grad, place, x, w, part, score;
    size_t xt, wt, p, pt, dx, dw, total;
};

size_t region(size_t& at, size_t bytes) {
    const size_t r = at;
    at += (bytes + 255) / 256 * 256;
    return r;
}

// `table`: the array, or NULL where only the size is asked for (then it is taken as unaligned)
Plan make_plan(int dtype, int B, int T, int V, int N, bool grad, const void* table) {
    Plan p{};
    const long e = dtype == SEMICRF_F32 ? 4 : 2;
    p.rows = (long)B * T;
    p.padded = up(p.rows, ROW_TILE);
    p.V = V;
    p.N = N;
    p.ld = up(N, STEP / e);
    p.large = tiles((int)p.rows, 256) * (long)tiles(V, 256) >= 256;
    p.BA = p.BB = p.large ? 256 : 128;
    p.WA = 2;
    p.wgs = p.large ? 256 : 512;
    p.copy_w = N * e % STEP != 0 || !table || (uintptr_t)table % 16;
    size_t at = 0;
    p.ctl = region(at, sizeof(Control));
    p.counts = region(at, (size_t)up(p.rows, LIST) / LIST * 4);
    p.list_row = region(at, p.padded * 4);
    p.list_target = region(at, p.padded * 4);
    p.x = region(at, p.padded * p.ld * e);
    if (!grad) {
        const long items = p.padded / p.BB > 4l * p.wgs ? p.padded / p.BB : 4l * p.wgs;
        p.part = region(at, items * p.WA * p.BB * sizeof(float2));
        p.score = region(at, p.padded * 4);
    } else {
        p.list_lse = region(at, p.padded * 4);
        p.list_grad = region(at, p.padded * 4);
        p.place = region(at, p.rows * 4);
        p.vpad = up(V, 256);
        // pieces of the vocabulary: p and its transpose take at most 1 GB together, or one tile of words
        const long most = (512l << 20) / (p.padded * e) / 256 * 256;
        p.pieces = most < 256 ? p.vpad / 256 : tiles((int)p.vpad, (int)(most < p.vpad ? most : p.vpad));
        p.piece = up((p.vpad + p.pieces - 1) / p.pieces, 256);
        p.pieces = (p.vpad + p.piece - 1) / p.piece;
        p.vpad = p.piece * p.pieces;
        p.ldo = up(N, 4);
        const long nt = tiles(N, p.BA);
        const long shares = p.wgs / ((p.piece / p.BB) * nt);
        p.dw_split = (int)(shares < 1 ? 1 : shares > 16 ? 16 : shares);
        const long k = p.padded * e / STEP;
        if (p.dw_split > k) p.dw_split = (int)k;
        p.xt = region(at, p.N * p.padded * e);
        p.wt = region(at, p.N * p.vpad * e);
        p.p = region(at, p.padded * p.piece * e);
        p.pt = region(at, p.padded * p.piece * e);
        const long dx_rows = p.padded > p.wgs * p.BB / nt ? p.padded : p.wgs * p.BB / nt;
        p.dx = region(at, dx_rows * p.ldo * 4);
        p.dw = region(at, (size_t)p.dw_split * p.piece * p.ldo * 4);
    }
    p.w = region(at, p.copy_w ? (size_t)V * p.ld * e : 0);
    p.total = at;
    return p;
}

template <class P>
P* in(void* ws, size_t at) { return (P*)((char*)ws + at); }

// The listed rows and the padded copies of x and, where its rows are no whole steps, of W.
template <class T, bool GRAD>
Scores gather(const NllArgs& a, const Plan& p, const Listed& list, void* ws, hipStream_t stream) {
    Control* ctl = in<Control>(ws, p.ctl);
    int* counts = in<int>(ws, p.counts);
    const int blocks = (int)(up(p.rows, LIST) / LIST);
    hipLaunchKernelGGL(k_nll_count, dim3(blocks), dim3(LIST_THREADS), 0, stream, a, ctl, counts);
    hipLaunchKernelGGL(k_nll_list<GRAD>, dim3(blocks), dim3(LIST_THREADS), 0, stream, a, ctl, counts, list);
    T* x = in<T>(ws, p.x);
    hipLaunchKernelGGL(k_nll_rows<T>, dim3((unsigned)(p.padded / 4)), dim3(256), 0, stream, (const T*)a.x, list.row, ctl,
                       0, a.N, x, (int)p.ld, ROW_TILE);
    const T* w = (const T*)a.table;
    if (p.copy_w) {
        T* copy = in<T>(ws, p.w);
        hipLaunchKernelGGL(k_nll_rows<T>, dim3((unsigned)((p.V + 3) / 4)), dim3(256), 0, stream, w, (const int*)nullptr,
                           (const Control*)nullptr, a.V, a.N, copy, (int)p.ld, 1);
        w = copy;
    }
    Scores s{};
    s.w = (const char*)w;
    s.x = (const char*)x;
    s.ldw = s.ldx = (unsigned)(p.ld * sizeof(T));
    s.V = a.V;
    s.nk = (int)(p.ld * sizeof(T) / STEP);
    s.scale = a.scale * LOG2EF;
    return s;
}

template <class T, class Tl>
hipError_t run_nll(const NllArgs& a, const Plan& p, void* ws, hipStream_t stream) {
    Listed list{in<int>(ws, p.list_row), in<int>(ws, p.list_target), nullptr, nullptr, nullptr};
    const Scores s = gather<T, false>(a, p, list, ws, stream);
    const Control* ctl = in<Control>(ws, p.ctl);
    float2* part = in<float2>(ws, p.part);
    float* score = in<float>(ws, p.score);
    hipLaunchKernelGGL((k_nll_scores<T, Tl>), dim3(p.wgs), dim3(Tl::NT), 0, stream, s, ctl, list.target, part, score);
    hipLaunchKernelGGL(k_nll_loss, dim3((unsigned)((p.rows + 255) / 256)), dim3(256), 0, stream, ctl, list.row, part,
                       score, a.V, p.BA, p.BB, p.WA, p.wgs, a.loss, a.lse);
    return hipGetLastError();
}

template <class T, class Tl, class Tg>
hipError_t run_nll_grad(const NllArgs& a, const Plan& p, void* ws, hipStream_t stream) {
    using H = typename Held<T>::type;
    Listed list{in<int>(ws, p.list_row), in<int>(ws, p.list_target), in<float>(ws, p.list_lse),
                in<float>(ws, p.list_grad), in<int>(ws, p.place)};
    const Scores s = gather<T, true>(a, p, list, ws, stream);
    Control* ctl = in<Control>(ws, p.ctl);
    H *xt = in<H>(ws, p.xt), *wt = in<H>(ws, p.wt), *pp = in<H>(ws, p.p), *pt = in<H>(ws, p.pt);
    float *dx = in<float>(ws, p.dx), *dw = in<float>(ws, p.dw);
    const unsigned nb = (unsigned)((a.N + 63) / 64);
    if (a.grad_table) {
        if (sizeof(H) == 2)
            hipLaunchKernelGGL(k_nll_max<T>, dim3(256), dim3(256), 0, stream, (const T*)s.x, ctl, 0l, (int)p.ld,
                               &ctl->max_x);
        hipLaunchKernelGGL((k_nll_transpose<T, H>), dim3((unsigned)(p.padded / 64), nb), dim3(256), 0, stream,
                           (const T*)s.x, ctl, true, 0, a.N, (int)p.ld, &ctl->max_x, xt, (size_t)p.padded, ROW_TILE);
    }
    if (a.grad_x) {
        if (sizeof(H) == 2)
            hipLaunchKernelGGL(k_nll_max<T>, dim3(1024), dim3(256), 0, stream, (const T*)a.table, (const Control*)nullptr,
                               (long)a.V * a.N, a.N, &ctl->max_w);
        hipLaunchKernelGGL((k_nll_transpose<T, H>), dim3((unsigned)(p.vpad / 64), nb), dim3(256), 0, stream,
                           (const T*)a.table, ctl, false, a.V, a.N, a.N, &ctl->max_w, wt, (size_t)p.vpad, (int)p.vpad);
    }
    const int nk_dx = (int)(p.piece * sizeof(H) / STEP);
    for (long i = 0; i < p.pieces; ++i) {
        const int v0 = (int)(i * p.piece);
        const int words = (int)(p.V - v0 < p.piece ? p.V - v0 : p.piece);
        if (words <= 0) break;
        hipLaunchKernelGGL((k_nll_p<T, H, Tl>), dim3(p.wgs), dim3(Tl::NT), 0, stream, s, ctl, list.target, list.lse,
                           list.grad, v0, (int)(p.piece / Tl::BA), pp, (size_t)p.piece, pt, (size_t)p.padded);
        if (a.grad_x)
            hipLaunchKernelGGL((k_nll_product<H, Tg, true>), dim3(p.wgs), dim3(Tg::NT), 0, stream,
                               (const char*)(wt + v0), (unsigned)(p.vpad * sizeof(H)), a.N, (const char*)pp,
                               (unsigned)(p.piece * sizeof(H)), ctl, 0, nk_dx, 0, i > 0, dx, (int)p.ldo);
        if (a.grad_table) {
            hipLaunchKernelGGL((k_nll_product<H, Tg, false>), dim3(p.wgs), dim3(Tg::NT), 0, stream, (const char*)xt,
                               (unsigned)(p.padded * sizeof(H)), a.N, (const char*)pt,
                               (unsigned)(p.padded * sizeof(H)), ctl, (int)(p.piece / Tg::BB), 0, p.dw_split, false, dw,
                               (int)p.ldo);
            hipLaunchKernelGGL((k_nll_dw<T, H>), dim3((unsigned)((words + 3) / 4)), dim3(256), 0, stream, ctl, dw,
                               (int)p.ldo, (int)p.piece, p.dw_split, a.scale, words, a.N,
                               (T*)a.grad_table + (size_t)v0 * a.N);
        }
    }
    if (a.grad_x)
        hipLaunchKernelGGL((k_nll_dx<T, H>), dim3((unsigned)((p.rows + 3) / 4)), dim3(256), 0, stream, ctl, list.place,
                           list.grad, a.scale, dx, (int)p.ldo, p.BA, p.BB, p.wgs, nk_dx, (int)p.rows, a.N,
                           (T*)a.grad_x);
    return hipGetLastError();
}

}  // namespace

size_t token_nll_bytes(int dtype, int B, int T, int V, int N, bool grad) {
    return make_plan(dtype, B, T, V, N, grad, nullptr).total;
}

hipError_t launch_token_nll(const NllArgs& a, void* ws, hipStream_t stream) {
    const Plan p = make_plan(a.dtype, a.B, a.T, a.V, a.N, false, a.table);
    if (a.dtype == SEMICRF_F32)
        return p.large ? run_nll<float, Large<float>>(a, p, ws, stream) : run_nll<float, Small<float>>(a, p, ws, stream);
    return p.large ? run_nll<bf16, Large<bf16>>(a, p, ws, stream) : run_nll<bf16, Small<bf16>>(a, p, ws, stream);
}

hipError_t launch_token_nll_grad(const NllArgs& a, void* ws, hipStream_t stream) {
    const Plan p = make_plan(a.dtype, a.B, a.T, a.V, a.N, true, a.table);
    if (a.dtype == SEMICRF_F32)
        return p.large ? run_nll_grad<float, Large<float>, Large<float>>(a, p, ws, stream)
                       : run_nll_grad<float, Small<float>, Small<float>>(a, p, ws, stream);
    return p.large ? run_nll_grad<bf16, Large<bf16>, Large<f16>>(a, p, ws, stream)
                   : run_nll_grad<bf16, Small<bf16>, Small<f16>>(a, p, ws, stream);
}

}  // namespace semicrf
