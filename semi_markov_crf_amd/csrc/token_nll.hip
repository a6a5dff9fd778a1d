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
// Three products, one core: a tile of BA x BB results, 128 bytes of the contracted axis a step, through
// two stages of LDS that are filled without passing through registers.
//   scores    A = W,            B = x            the log sum (k_nll_scores); p of a piece of words (k_nll_p)
//   dx        A = W by columns, B = p
//   dW        A = x by columns, B = p by columns
// Scores are summed and exponentiated in registers; a lane holds scores of the same rows of x for all
// tiles of the vocabulary it sees, so that maximum and sum run along without an exchange.
//
// Rounding (bfloat16): scores are exact products summed in fp32.  The second products' operands are in
// fp16, each scaled by a power of two to the top of its range: 11 bits down to 2^-28 of the largest, fewer
// below, 0 from 2^-39 on.  W has 8 bits of its own and loses nothing down to 2^-28 of its largest value.  p
// (at most 1) has 11 bits down to 2^-29, and is 0 below 2^-40: a word that is nowhere more likely, nor a target,
// has no gradient.  x enters dW times its row's gradient, rounded to 11 bits; the largest |x| times the
// largest |gradient| is the top.  So the gradients' own rounding is what is seen (p in bfloat16 would add an
// error as large as that): off by 0.00167 in the 2-norm, as with everything in fp32.  In float32 everything is
// float32.
//
// Bound by the matrix cores.  16,000 rows of 1,024 over 50,001 words in bfloat16, 1.64 * 10^12 operations a
// product (a large product of the library reaches 1,230 TFLOP/s): scores 1,400 us (1,170 TFLOP/s), p 1,560 to
// 1,600 (1,040: it stores 1.6 GB), dx 1,290 (1,270), dW 1,360 (1,200); all else of a loss and its gradient 140.  The
// gradient forms the scores a second time: the forward pass would have to keep 1.6 GB for it.  In float32 (a large
// product: 153 TFLOP/s) 16,000 rows of 1,024 over 8,192 words take 1,958 us (137 TFLOP/s), their gradient 5,834 (138).
#include "common.h"
#include "encoder.h"

namespace semicrf {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
using f16 = _Float16;

// log2 e and ln 2 with what their floats leave over: a log sum of 10 loses 2^-21 to one of them
constexpr float LOG2EF = 1.44269504088896f, LOG2E_REST = (float)(1.4426950408889634074 - (double)LOG2EF);
constexpr float LN2F = 0.69314718055994531f, LN2_REST = (float)(0.69314718055994530942 - (double)LN2F);
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

// Four columns of 16 lanes of an LDS tile of rows of the contracted axis, as a fragment: lane 16 g + r gets
// column r, rows 8 g .. 8 g + 7 of the step half (the order of a fragment read along a row).  The transposing
// read gives lane 16 g + i the i-th column of the 4 x 16 block whose row j is what lanes 16 g + 4 j .. + 3
// point at.
typedef __fp16 half4 __attribute__((__vector_size__(8)));
typedef __attribute__((address_space(3))) half4 LdsHalf4;

// How an operand lies in memory: ROWS: dense along the contracted axis, a step takes 128 bytes of each row;
// COLUMNS: dense along the other axis, a step takes 64 (fp16) or 32 (fp32) rows of as many elements as the
// tile has.  In LDS a step's bytes keep that form; 16-byte chunks are permuted within a row so that the
// lanes of a read fall on different banks.
enum Form { ROWS, COLUMNS };

template <class T>
__device__ __forceinline__ int column_swizzle(int k) {
    return sizeof(T) == 2 ? (k & 3) * 2 : (k >> 2 & 3) * 4;
}

// One operand of a tile: SIZE rows (or columns) shared out to NW wavefronts
template <class T, Form F, int SIZE, int NW>
struct Operand {
    static constexpr int ELEMENTS = STEP / sizeof(T);            // of the contracted axis a step
    static constexpr int CHUNKS = F == ROWS ? STEP / 16 : SIZE * (int)sizeof(T) / 16;   // of a row in LDS
    static constexpr int BYTES = SIZE * STEP, LOADS = BYTES / 1024 / NW;
    const char* base;
    size_t step;                                                 // bytes from one step to the next
    unsigned at[LOADS];

    // rows: how many of the tile's rows exist (ROWS), or bytes of a row from the tile's first column
    // (COLUMNS); what lies beyond is taken as the last
    __device__ __forceinline__ void point(const void* p, unsigned ld, int limit) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        base = (const char*)p;
        step = F == ROWS ? STEP : (size_t)ELEMENTS * ld;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int chunk = (i * NW + wave) * 64 + lane, r = chunk / CHUNKS, c = chunk % CHUNKS;
            if (F == ROWS) at[i] = (unsigned)min(r, limit - 1) * ld + (c ^ (r & 7)) * 16;
            else at[i] = (unsigned)r * ld + min((c ^ column_swizzle<T>(r)) * 16, limit - 16);
        }
    }
    // To LDS directly, 1,024 bytes an instruction from the address in m0 on.  As assembly without results: the
    // compiler would wait for such loads before any transposing read of LDS, whichever half of it they fill
    // (the 25,088-word product of dW took 1,120 us so).  step_barrier() waits for them.
    __device__ __forceinline__ void fetch(int k, char* lds) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const char* from = base + k * step;
        const unsigned to = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)lds + wave * 1024;
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"          // m0 is reserved; nothing else here uses it
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                         :
                         : "s"(to + i * NW * 1024), "v"(at[i]), "s"(from)
                         : "memory", "m0");
#pragma clang diagnostic pop
    }
    // Of half a step, the 16 rows (or columns) from `first`
    __device__ __forceinline__ static raw_piece fragment(const char* lds, int first, int half) {
        const int lane = threadIdx.x & 63, g = lane / 16, r = lane & 15;
        if constexpr (F == ROWS) {
            return *(const raw_piece*)(lds + (first + r) * STEP + (((half * 4 + g) ^ (r & 7)) * 16));
        } else if constexpr (sizeof(T) == 2) {
            const int k = half * 32 + 8 * g + (r >> 2), c = first / 8 + (r & 3) / 2, in = (r & 1) * 8;
            const char* p = lds + k * (CHUNKS * 16) + in + (c ^ column_swizzle<T>(k)) * 16;
            const half4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4f16((LdsHalf4*)p);
            const half4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4f16((LdsHalf4*)(p + 4 * CHUNKS * 16));
            return __builtin_bit_cast(raw_piece, __builtin_shufflevector(__builtin_bit_cast(f16x4, lo),
                                                                         __builtin_bit_cast(f16x4, hi), 0, 1, 2, 3, 4,
                                                                         5, 6, 7));
        } else {
            f32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = half * 16 + 4 * g + j, c = (first + r) / 4;
                v[j] = *(const float*)(lds + k * (CHUNKS * 16) + (c ^ column_swizzle<T>(k)) * 16 + (r & 3) * 4);
            }
            return __builtin_bit_cast(raw_piece, v);
        }
    }
};

// All fetches are there, and all wavefronts have read what the next ones overwrite
__device__ __forceinline__ void step_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// A tile: BA rows of A, BB rows of B, WA x WB wavefronts, two steps in LDS: one is multiplied while the
// next is on its way.
template <class T, Form FA, Form FB, int BA_, int BB_, int WA_, int WB_>
struct Tile {
    static constexpr int BA = BA_, BB = BB_, WA = WA_, WB = WB_;
    static constexpr int NW = WA * WB, NT = 64 * NW, MA = BA / WA / 16, MB = BB / WB / 16;
    static constexpr int STAGE = (BA + BB) * STEP;
    using OpA = Operand<T, FA, BA, NW>;
    using OpB = Operand<T, FB, BB, NW>;

    f32x4 acc[MA][MB];
    OpA a;
    OpB b;
    int turn = 0;                        // which half of LDS the next step goes to

    __device__ __forceinline__ void fetch(int k, char* lds) {
        a.fetch(k, lds + turn * STAGE);
        b.fetch(k, lds + turn * STAGE + BA * STEP);
        turn ^= 1;
    }
    __device__ __forceinline__ void point(const void* pa, unsigned lda, int limit_a, const void* pb, unsigned ldb,
                                          int limit_b) {
        a.point(pa, lda, limit_a);
        b.point(pb, ldb, limit_b);
    }
    // acc = A . B over steps k0 .. k1 - 1, of which the first was fetched.  next(k): points at the tile to
    // come and sets k to its first step, which is fetched during the last one here; false: there is none.
    template <class Next>
    __device__ __forceinline__ void product(int k0, int k1, char* lds, Next&& next) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wa = wave / WB, wb = wave % WB;
#pragma unroll
        for (int i = 0; i < MA; ++i)
#pragma unroll
            for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = k0; k < k1; ++k) {
            step_barrier();
            const char* now = lds + (turn ^ 1) * STAGE;
            int to = k + 1;
            bool more = true;
            if (to == k1) more = next(to);
            if (more) fetch(to, lds);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                raw_piece fb[MB];
#pragma unroll
                for (int j = 0; j < MB; ++j)
                    fb[j] = OpB::fragment(now + BA * STEP, wb * (BB / WB) + j * 16, half);
#pragma unroll
                for (int i = 0; i < MA; ++i) {
                    const raw_piece fa = OpA::fragment(now, wa * (BA / WA) + i * 16, half);
#pragma unroll
                    for (int j = 0; j < MB; ++j) acc[i][j] = mma((const T*)nullptr, fa, fb[j], acc[i][j]);
                }
            }
            // In this order: the first two fragments of A and those of B, then a read ahead of each row of products
            // (products of a step alone leave half of the matrix cores' time to waits for LDS).
            if constexpr (sizeof(T) == 2) {
                constexpr int RA = FA == ROWS ? 1 : 2, RB = FB == ROWS ? 1 : 2;
                __builtin_amdgcn_sched_group_barrier(0x100, MB * RB + 2 * RA, 0);
#pragma unroll
                for (int i = 0; i < 2 * MA; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, MB, 0);
                    if (i + 2 < 2 * MA) __builtin_amdgcn_sched_group_barrier(0x100, RA, 0);
                    if (i >= MA - 1 - MB && i < MA - 1) __builtin_amdgcn_sched_group_barrier(0x100, RB, 0);
                }
            }
        }
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

// Row -> whether it is listed; beyond: its target is out of range
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

// counts[block] = listed rows of the block's 4,096
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

// The listed rows in order, then the others from the end on, and what listed rows carry into the products
struct Listed {
    int* row;                // place among all rows
    int* target;
    float *lse, *grad;       // gradients only
};

// counts NULL: one workgroup, which also clears the control block
template <bool GRAD>
__global__ __launch_bounds__(LIST_THREADS) void k_nll_list(const NllArgs a, Control* ctl, const int* counts,
                                                           Listed list) {
    __shared__ int s[LIST_THREADS / 64], before[LIST_THREADS / 64];
    __shared__ unsigned top;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const unsigned rows = (unsigned)a.B * a.T, first = blockIdx.x * (unsigned)LIST + threadIdx.x * LIST_EACH;
    int n = 0, prev = 0, target[LIST_EACH];
    bool is[LIST_EACH];
    if (threadIdx.x == 0) top = 0;
    if (counts)
        for (unsigned i = threadIdx.x; i < blockIdx.x; i += LIST_THREADS) prev += counts[i];
    for (int off = 32; off >= 1; off >>= 1) prev += __shfl_xor(prev, off, 64);
#pragma unroll
    for (int i = 0; i < LIST_EACH; ++i) {
        const unsigned row = first + i;
        bool beyond = false;
        is[i] = row < rows && listed(a, row, beyond, target[i]);
        n += is[i];
        if (beyond && a.status) atomicOr(a.status, 1);
        if (!GRAD && row < rows && !is[i]) {
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
        if (!is[i]) {
            if (row < rows) list.row[rows - 1 - (row - at)] = (int)row;
            continue;
        }
        list.row[at] = (int)row;
        list.target[at] = target[i];
        if (GRAD) {
            const float g = a.grad_loss[row];
            list.lse[at] = a.lse_in[row];
            list.grad[at] = g;
            const unsigned bits = __float_as_uint(g) & 0x7fffffffu;
            if (bits < 0x7f800000u) most = max(most, bits);
        }
        ++at;
    }
    if (GRAD) {
        for (int off = 32; off >= 1; off >>= 1) most = max(most, (unsigned)__shfl_xor((int)most, off, 64));
        if (lane == 0 && most) atomicMax(&top, most);
        __syncthreads();
        if (counts && threadIdx.x == 0 && top) atomicMax(&ctl->max_g, top);
    }
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == LIST_THREADS - 1) {
        ctl->rows = at;
        if (!counts) {
            ctl->max_x = ctl->max_w = 0;
            ctl->max_g = top;
        }
    }
}

__host__ __device__ __forceinline__ int tiles(int rows, int tile) { return (rows + tile - 1) / tile; }

constexpr int MAX_WGS = 512, MAX_THREADS = 1024;

// The largest finite magnitude of n elements, by blocks `first` .. of the grid's `blocks`
template <class T>
__device__ __forceinline__ unsigned largest(const T* src, long n, int block, int blocks) {
    constexpr int V = 16 / sizeof(T);
    unsigned most = 0;
    auto see = [&](float x) {
        const unsigned bits = __float_as_uint(x) & 0x7fffffffu;
        if (bits < 0x7f800000u) most = max(most, bits);
    };
    const long step = (long)blocks * MAX_THREADS * V;
    long i = ((long)block * MAX_THREADS + threadIdx.x) * V;
    for (; i + V <= n; i += step) {
        const raw_piece r = *(const loose_piece*)(src + i);
        float x[V];
        unpack<T>(r, x);
#pragma unroll
        for (int j = 0; j < V; ++j) see(x[j]);
    }
    for (; i < n; ++i) see((float)src[i]);
    return most;
}

// max_x over the listed rows, by the first x_wgs workgroups, and max_w over the table
template <class T>
__global__ __launch_bounds__(MAX_THREADS) void k_nll_max(const NllArgs a, Control* ctl, const int* row, int x_wgs) {
    const int lane = threadIdx.x & 63, rows = ctl->rows;
    const bool of_x = (int)blockIdx.x < x_wgs;
    unsigned most = 0;
    if (of_x) {
        // a wavefront a row
        constexpr int V = 16 / sizeof(T);
        for (int r = blockIdx.x * (MAX_THREADS / 64) + (threadIdx.x >> 6); r < rows; r += x_wgs * (MAX_THREADS / 64)) {
            const T* from = (const T*)a.x + (size_t)row[r] * a.N;
            for (int c = lane * V; c < a.N; c += 64 * V) {
                if (c + V <= a.N) {
                    float x[V];
                    const raw_piece v = *(const loose_piece*)(from + c);
                    unpack<T>(v, x);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const unsigned bits = __float_as_uint(x[j]) & 0x7fffffffu;
                        if (bits < 0x7f800000u) most = max(most, bits);
                    }
                } else {
                    for (int j = c; j < a.N; ++j) {
                        const unsigned bits = __float_as_uint((float)from[j]) & 0x7fffffffu;
                        if (bits < 0x7f800000u) most = max(most, bits);
                    }
                }
            }
        }
    } else {
        most = largest((const T*)a.table, (long)a.V * a.N, blockIdx.x - x_wgs, gridDim.x - x_wgs);
    }
    // one atomic a workgroup at most: on one address they take some 20 ns each, one after another
    __shared__ unsigned s[MAX_THREADS / 64];
    for (int off = 32; off >= 1; off >>= 1) most = max(most, (unsigned)__shfl_xor((int)most, off, 64));
    if (lane == 0) s[threadIdx.x >> 6] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < MAX_THREADS / 64; ++i) most = max(most, s[i]);
        unsigned* to = of_x ? &ctl->max_x : &ctl->max_w;
        if (most > __hip_atomic_load(to, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(to, most);
    }
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
template <class H>
constexpr float P_EXPONENT = sizeof(H) == 4 ? 0.0f : 15.0f;
// What the rows' gradients are divided by where x carries them into dW: the largest one
__device__ __forceinline__ float grad_unit(unsigned bits) { return fmaxf(__uint_as_float(bits), 0x1p-120f); }

// What the products read, laid out once a call.  Rows of ld elements, zeros past N.
struct Layout {
    void* x;                 // [rows up to a whole tile][ld]: the listed rows
    void* w;                 // the table, or its copy with rows of ld elements where the table's own are no
                             // whole steps
    void* xg;                // as x, times the row's gradient over the largest one (dW)
    void* wh;                // [words up to whole pieces][ld] (dx)
    int ld, words;           // rows of the copies of W
    bool copy_w;
};

// Blocks of 64 rows by 64 columns: first those of x, then those of W; rows without a target get their zeros in grad_x
template <class T, class H, bool GRAD>
__global__ __launch_bounds__(256) void k_nll_lay(const NllArgs a, const Control* ctl, Listed list, Layout l,
                                                 int x_blocks) {
    constexpr int V = 16 / sizeof(T), ACROSS = 64 / V, DOWN = 256 / ACROSS;
    const int cols = l.ld / 64, M = a.B * a.T, rows = ctl->rows, padded = tiles(rows, ROW_TILE) * ROW_TILE;
    const bool of_x = (int)blockIdx.x < x_blocks;
    const int block = of_x ? blockIdx.x : blockIdx.x - x_blocks;
    const int c = block % cols * 64 + threadIdx.x % ACROSS * V, r0 = block / cols * 64;
    if (of_x && r0 >= padded && !(GRAD && a.grad_x && r0 < M)) return;
    float unit = 0.0f, sx = 1.0f, sw = 1.0f;
    if (GRAD) {
        unit = 1.0f / grad_unit(ctl->max_g);
        sx = held_scale<H>(ctl->max_x);
        sw = held_scale<H>(ctl->max_w);
    }
    for (int r = r0 + threadIdx.x / ACROSS; r < r0 + 64; r += DOWN) {
        const int n = of_x ? rows : a.V;
        raw_piece v = {0, 0, 0, 0};
        if (r < n) {
            const T* from = of_x ? (const T*)a.x + (size_t)list.row[r] * a.N : (const T*)a.table + (size_t)r * a.N;
            if (c + V <= a.N) {
                v = *(const loose_piece*)(from + c);
            } else {
                T t[V];
#pragma unroll
                for (int i = 0; i < V; ++i) t[i] = c + i < a.N ? from[c + i] : (T)0.0f;
                __builtin_memcpy(&v, t, 16);
            }
        }
        const size_t at = (size_t)r * l.ld + c;
        auto held = [&](float f, void* to) {
            float x[V];
            H h[V];
            unpack<T>(v, x);
#pragma unroll
            for (int i = 0; i < V; ++i) h[i] = (H)(x[i] * f);
            __builtin_memcpy((H*)to + at, h, sizeof(h));
        };
        if (of_x) {
            if (r < padded) {
                *(raw_piece*)((T*)l.x + at) = v;
                if (GRAD && a.grad_table) held(r < rows ? list.grad[r] * unit * sx : 0.0f, l.xg);
            }
            if (GRAD && a.grad_x && r >= rows && r < M) {
                T* to = (T*)a.grad_x + (size_t)list.row[r] * a.N;
                if (c + V <= a.N) {
                    *(loose_piece*)(to + c) = raw_piece{0, 0, 0, 0};
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (c + i < a.N) to[c + i] = (T)0.0f;
                }
            }
        } else {
            if (l.copy_w && r < l.words) *(raw_piece*)((T*)l.w + at) = v;
            if (GRAD && sizeof(H) == 2 && a.grad_x && r < l.words) held(sw, l.wh);
        }
    }
}

// ------------------------------------------------------------------ scores
// Workgroups in the order in which their tiles share rows: each of the 8 chiplets (which have an L2
// cache each, and to which consecutive workgroups go in turn) takes consecutive numbers.
__device__ __forceinline__ int ordered_block() {
    return (blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8;
}
// Tile number -> row tile and column tile: eight tiles of rows by all columns at a time
__device__ __forceinline__ void in_groups(int tile, int rows, int cols, int& r, int& c) {
    const int group = tile / (8 * cols), in = tile - group * 8 * cols, width = min(8, rows - group * 8);
    r = group * 8 + in % width;
    c = in / width;
}

// How many workgroups share the vocabulary of a tile of rows: the number that leaves the least for the
// busiest one, of up to four rounds of items.  All lanes get the same.  25,600 rows of 1,024 over 50,001 words:
// one round at most 2,566 us, 2, 4 or 8 2,204 to 2,213; 100 to 16,000 rows within 2 % whichever.
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
    unsigned ld;             // bytes
    int V, nk;
    float scale, rest;       // to log2 units, and what the float leaves over (of use in float32 only)
};

// part[(item, wavefront row)][BB] = (maximum, sum) of the scores of a share of the vocabulary, item =
// tile of rows * split + share; at_target[row] = the target's score.  All in log2 units.
template <class T, class Tl>
__global__ __launch_bounds__(Tl::NT) void k_nll_scores(const Scores p, const Control* ctl, const int* target,
                                                       float2* part, float* at_target) {
    __shared__ __align__(16) char lds[2 * Tl::STAGE];
    __shared__ int words[2][Tl::BB];         // targets of a tile's rows, by turns
    const int rows = __builtin_amdgcn_readfirstlane(ctl->rows);
    const int mt = tiles(rows, Tl::BB), vt = tiles(p.V, Tl::BA), S = vocab_split(mt, vt, gridDim.x);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wa = wave / Tl::WB, wb = wave % Tl::WB;
    const int col = wb * (Tl::BB / Tl::WB) + (lane & 15);
    Tl t;
    auto point = [&](int item, int v) {
        t.point(p.w + (size_t)v * Tl::BA * p.ld, p.ld, p.V - v * Tl::BA, p.x + (size_t)(item / S) * Tl::BB * p.ld, p.ld,
                Tl::BB);
    };
    int item = ordered_block();
    if (item < mt * S) {
        point(item, item % S * vt / S);
        t.fetch(0, lds);
    }
    for (int turn = 0; item < mt * S; item += gridDim.x, turn ^= 1) {
        const int m0 = item / S * Tl::BB, v1 = (item % S + 1) * vt / S;
        // seen by all after the first step of a product; the turn before may still be read
        if ((int)threadIdx.x < Tl::BB) {
            const int m = m0 + threadIdx.x;
            words[turn][threadIdx.x] = m < rows ? target[m] : -1;
        }
        float top[Tl::MB], sum[Tl::MB];
#pragma unroll
        for (int j = 0; j < Tl::MB; ++j) {
            top[j] = -__builtin_inff();
            sum[j] = 0.0f;
        }
        for (int v = item % S * vt / S; v < v1; ++v) {
            t.product(0, p.nk, lds, [&](int& k) {
                const int after = v + 1 < v1 ? item : item + (int)gridDim.x;
                if (after >= mt * S) return false;
                point(after, v + 1 < v1 ? v + 1 : after % S * vt / S);
                k = 0;
                return true;
            });
            const int first = v * Tl::BA + wa * (Tl::BA / Tl::WA) + lane / 16 * 4;
            const bool whole = (v + 1) * Tl::BA <= p.V;
#pragma unroll
            for (int j = 0; j < Tl::MB; ++j) {
                float most = top[j];
#pragma unroll
                for (int i = 0; i < Tl::MA; ++i) {
                    f32x4& z = t.acc[i][j];
                    if constexpr (sizeof(T) == 4)
#pragma unroll
                        for (int k = 0; k < 4; ++k) z[k] = fmaf(z[k], p.scale, z[k] * p.rest);
                    else
                        z *= p.scale;
                    if (!whole)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (first + i * 16 + k >= p.V) z[k] = -__builtin_inff();
                    most = fmaxf(most, fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])));
                }
                const int m = m0 + col + j * 16;
                const int hit = words[turn][col + j * 16] - first;        // the target is one of the lane's words
                if (hit >= 0 && hit < Tl::MA * 16 && hit % 16 < 4) {
#pragma unroll
                    for (int i = 0; i < Tl::MA; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (hit == i * 16 + k) at_target[m] = t.acc[i][j][k];
                }
                const float ref = most == -__builtin_inff() ? 0.0f : most;
                // The tile's words first: added to the running sum one by one, V / 8 roundings in a row, those
                // below half a step of it would be lost however many they are.
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < Tl::MA; ++i) {
                    float e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) e[k] = fast_exp2(t.acc[i][j][k] - ref);
                    s += (e[0] + e[1]) + (e[2] + e[3]);
                }
                sum[j] = fmaf(sum[j], fast_exp2(top[j] - ref), s);
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
    if (lse) lse[row[m]] = fmaf(ref, LN2F, fmaf(ref, LN2_REST, l * LN2F));
}

// ------------------------------------------------------------------ gradients
// p of a piece of the vocabulary, [rows up to a whole tile][ldp], times P_SCALE.  Zero for rows and words past
// the last.
template <class T, class H, class Tl>
__global__ __launch_bounds__(Tl::NT) void k_nll_p(const Scores s, const Control* ctl, const int* target,
                                                  const float* lse, int v0, int vt, H* p, int ldp) {
    __shared__ __align__(16) char lds[2 * Tl::STAGE];
    const int rows = __builtin_amdgcn_readfirstlane(ctl->rows), mt = tiles(rows, ROW_TILE) * (ROW_TILE / Tl::BB);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wa = wave / Tl::WB, wb = wave % Tl::WB;
    Tl t;
    auto point = [&](int tile) {
        int m, v;
        in_groups(tile, mt, vt, m, v);
        const int w0 = min(v0 + v * Tl::BA, s.V - 1);         // pieces may end past the vocabulary
        t.point(s.w + (size_t)w0 * s.ld, s.ld, s.V - w0, s.x + (size_t)m * Tl::BB * s.ld, s.ld, Tl::BB);
    };
    int tile = ordered_block();
    if (tile < mt * vt) {
        point(tile);
        t.fetch(0, lds);
    }
    for (; tile < mt * vt; tile += gridDim.x) {
        int mi, v;
        in_groups(tile, mt, vt, mi, v);
        // read and waited for here, where the product's first step waits as well: after the product they would
        // wait for what it has fetched ahead
        float log_sum[Tl::MB];
        int word[Tl::MB];
#pragma unroll
        for (int j = 0; j < Tl::MB; ++j) {
            const int m = mi * Tl::BB + wb * (Tl::BB / Tl::WB) + j * 16 + (lane & 15);
            // a row past the last has an infinite log sum: its p is 0
            log_sum[j] = m < rows ? lse[m] : __builtin_inff();
            word[j] = m < rows ? target[m] : -1;
        }
#pragma unroll
        for (int j = 0; j < Tl::MB; ++j) asm volatile("" : "+v"(log_sum[j]), "+v"(word[j]));
        t.product(0, s.nk, lds, [&](int& k) {
            const int after = tile + gridDim.x;
            if (after >= mt * vt) return false;
            point(after);
            k = 0;
            return true;
        });
        const int first = v * Tl::BA + wa * (Tl::BA / Tl::WA) + lane / 16 * 4;
        const bool whole = v0 + (v + 1) * Tl::BA <= s.V;
#pragma unroll
        for (int j = 0; j < Tl::MB; ++j) {
            const int m = mi * Tl::BB + wb * (Tl::BB / Tl::WB) + j * 16 + (lane & 15);
            float l = log_sum[j] * LOG2EF, rest = 0.0f;
            if (sizeof(H) == 4 && fabsf(l) < 1e30f)
                rest = fmaf(log_sum[j], LOG2EF, -l) + log_sum[j] * LOG2E_REST;
            l -= P_EXPONENT<H>;                                // p's scale goes into the exponent
            const int hit = word[j] - v0 - first;             // a row past the last: negative
            auto words = [&](int i, auto seen, H (&out)[4]) __attribute__((always_inline)) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float z = t.acc[i][j][k];
                    float q = fmaf(z, s.scale, -l);
                    if (sizeof(H) == 4) q += fmaf(z, s.rest, -rest);
                    q = fast_exp2(q);
                    if (decltype(seen)::value && hit == i * 16 + k) q -= P_SCALE<H>;
                    if (!whole && v0 + first + i * 16 + k >= s.V) q = 0.0f;
                    out[k] = (H)q;
                }
            };
            auto tiles = [&](auto seen) __attribute__((always_inline)) {
                if constexpr (sizeof(H) == 2) {
                    // Two tiles at a time, so that a lane has 16 bytes of its row and four lanes 64: lane 16 g + r
                    // gives up words 4 g .. 4 g + 3 of either tile for words 8 g .. 8 g + 7 of both.  (8 bytes a lane
                    // and 32 a row: 1,790 us in place of 1,630 for 16,000 rows over 50,001 words.)
                    H* to = p + (size_t)m * ldp + first - lane / 16 * 4 + lane / 16 * 8;
#pragma unroll
                    for (int i = 0; i < Tl::MA; i += 2) {
                        H one[4], two[4];
                        words(i, seen, one);
                        words(i + 1, seen, two);
                        unsigned x[2], y[2];
                        __builtin_memcpy(x, one, 8);
                        __builtin_memcpy(y, two, 8);
                        raw_piece v;
#pragma unroll
                        for (int d = 0; d < 2; ++d) {
                            const auto half = __builtin_amdgcn_permlane32_swap(x[d], y[d], false, false);
                            const auto row = __builtin_amdgcn_permlane16_swap(half[0], half[1], false, false);
                            v[d] = row[0];
                            v[2 + d] = row[1];
                        }
                        *(raw_piece*)(to + i * 16) = v;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < Tl::MA; ++i) {
                        H out[4];
                        words(i, seen, out);
                        __builtin_memcpy(p + (size_t)m * ldp + first + i * 16, out, sizeof(out));
                    }
                }
            };
            // few tiles hold the target of a row: the others compare nothing
            if (__any(hit >= 0 && hit < Tl::MA * 16)) tiles(std::true_type());
            else tiles(std::false_type());
        }
    }
}

// Where a product's results go: rows of N elements of type T times the factors, or, from tiles whose
// contracted axis is shared out, partial sums in fp32 that k_nll_join adds.  dx over several pieces of the
// vocabulary is added up in fp32 rows instead.
struct Product {
    const char *A, *B;
    unsigned lda, ldb;       // bytes
    int N;                   // columns of the result
    int b_tiles, b_rows;     // dW: tiles of words, and words
    int nk;                  // dx: steps
    bool pieces, add, last;  // dx: several pieces; some before this one; none after it
    float* part;             // [share][tile][BB][BA], or [rows][ldo] over several pieces
    int ldo;
    const int* row;          // dx: of a listed row
    const float* grad;       // dx: the row's gradient
    float scale;
    void* out;
};

// Tiles are taken whole, a round of all workgroups after the other; those of the last round, if they are
// few, are shared out along the contracted axis, in at most 16 shares of at least eight steps.  The gradient of
// 15,000 rows of 512 over 4,096 words in bfloat16: 284 us, 436 without shares; of 6,000 of 768 over 1,000 125 and
// 163, 126 with at most 8 shares, 124 with 32.  Shares of 4 or 16 steps: 121 and 112 there, but 2,000 of 512 over
// 3,000 words 85 with either in place of 81, 500 of 256 over 2,000 in float32 85 and 120 in place of 94.
struct Rounds {
    int whole, rest, shares, total;      // whole tiles, tiles shared out, shares of each, items
};
__host__ __device__ __forceinline__ Rounds rounds(int tiles, int wgs, int nk, bool split) {
    Rounds r{tiles, 0, 1, tiles};
    const int rest = tiles % wgs;
    if (!split || !rest) return r;
    int s = wgs / rest;
    if (s > nk / 8) s = nk / 8;
    if (s > 16) s = 16;
    if (s < 2) return r;
    r.whole = tiles - rest;
    r.rest = rest;
    r.shares = s;
    r.total = r.whole + rest * s;
    return r;
}

template <class T, class H, class Tl, bool DX>
__global__ __launch_bounds__(Tl::NT) void k_nll_product(const Product p, const Control* ctl) {
    __shared__ __align__(16) char lds[2 * Tl::STAGE];
    const int rows = __builtin_amdgcn_readfirstlane(ctl->rows), padded = tiles(rows, ROW_TILE) * ROW_TILE;
    const int at = tiles(p.N, Tl::BA), bt = DX ? padded / Tl::BB : p.b_tiles;
    const int nk = DX ? p.nk : padded / (int)(STEP / sizeof(H));
    const Rounds rd = rounds(at * bt, gridDim.x, nk, !p.pieces);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wa = wave / Tl::WB, wb = wave % Tl::WB;
    Tl t;
    auto where = [&](int item, int& a0, int& b0, int& k0, int& k1) {
        const int j = item - rd.whole, share = j / max(1, rd.rest);
        int ai, bi;
        in_groups(j < 0 ? item : rd.whole + j - share * rd.rest, bt, at, bi, ai);
        a0 = ai * Tl::BA;
        b0 = bi * Tl::BB;
        k0 = j < 0 ? 0 : (int)((long)share * nk / rd.shares);
        k1 = j < 0 ? nk : (int)((long)(share + 1) * nk / rd.shares);
    };
    // whether an item has steps; its first
    auto point = [&](int item, int& k) {
        int a0, b0, k1;
        where(item, a0, b0, k, k1);
        if (k >= k1) return false;
        t.point(p.A + a0 * sizeof(H), p.lda, (int)p.lda - a0 * (int)sizeof(H),
                DX ? p.B + (size_t)b0 * p.ldb : p.B + b0 * sizeof(H), p.ldb,
                DX ? Tl::BB : (int)p.ldb - b0 * (int)sizeof(H));
        return true;
    };
    // the scales of the operands are taken out one at a time: their product may be out of range
    const float back = 1.0f / held_scale<H>(DX ? ctl->max_w : ctl->max_x);
    int item = ordered_block(), k = 0;
    if (item < rd.total && point(item, k)) t.fetch(k, lds);
    for (; item < rd.total; item += gridDim.x) {
        int a0, b0, k0, k1;
        where(item, a0, b0, k0, k1);
        auto next = [&](int& k) {
            const int after = item + gridDim.x;
            return after < rd.total && point(after, k);
        };
        t.product(k0, k1, lds, next);
        if (k0 >= k1 && next(k)) t.fetch(k, lds);            // no listed rows
        const int a1 = wa * (Tl::BA / Tl::WA) + lane / 16 * 4;
#pragma unroll
        for (int j = 0; j < Tl::MB; ++j) {
            const int b1 = wb * (Tl::BB / Tl::WB) + j * 16 + (lane & 15), b = b0 + b1;
            if (item >= rd.whole) {
                float* to = p.part + ((size_t)(item - rd.whole) * Tl::BB + b1) * Tl::BA;
#pragma unroll
                for (int i = 0; i < Tl::MA; ++i) *(f32x4*)(to + a1 + i * 16) = t.acc[i][j];
            } else if (DX && p.pieces) {
                float* to = p.part + (size_t)b * p.ldo;
#pragma unroll
                for (int i = 0; i < Tl::MA; ++i) {
                    const int a = a0 + a1 + i * 16;
                    if (a >= p.ldo) continue;              // ldo: N up to a multiple of 4
                    f32x4 x = t.acc[i][j];
                    if (p.add) x += *(const f32x4*)(to + a);
                    *(f32x4*)(to + a) = x;
                }
            } else {
                const bool in = b < (DX ? rows : p.b_rows);
                const float g = DX ? (in ? p.grad[b] * p.scale : 0.0f) : grad_unit(ctl->max_g) * p.scale;
                T* to = (T*)p.out + (size_t)(in ? (DX ? p.row[b] : b) : 0) * p.N;
#pragma unroll
                for (int i = 0; i < Tl::MA; ++i) {
                    const int a = a0 + a1 + i * 16;
                    T v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = (T)(t.acc[i][j][k] * (1.0f / P_SCALE<H>) * back * g);
                    if (!in) continue;
                    if (a + 4 <= p.N) {
                        __builtin_memcpy(to + a, v, sizeof(v));
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (a + k < p.N) to[a + k] = v[k];
                    }
                }
            }
        }
    }
}

// Partial sums to results, in the order of the shares.  Shared-out tiles: grid (tiles of a round, BB * BA /
// 1024), four columns a thread.
template <class T, class H, bool DX>
__global__ __launch_bounds__(256) void k_nll_join(const Product p, const Control* ctl, int BA, int BB, int wgs) {
    const int rows = ctl->rows, padded = tiles(rows, ROW_TILE) * ROW_TILE;
    const int at = tiles(p.N, BA), bt = DX ? padded / BB : p.b_tiles;
    const Rounds rd = rounds(at * bt, wgs, DX ? p.nk : padded / (int)(STEP / sizeof(H)), true);
    if ((int)blockIdx.x >= rd.rest) return;
    int ai, bi;
    in_groups(rd.whole + blockIdx.x, bt, at, bi, ai);
    const int e = (blockIdx.y * 256 + threadIdx.x) * 4, b = bi * BB + e / BA, a = ai * BA + e % BA;
    if (b >= (DX ? rows : p.b_rows) || a >= p.N) return;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < rd.shares; ++s)
        v += *(const f32x4*)(p.part + ((size_t)s * rd.rest + blockIdx.x) * BB * BA + e);
    const float back = 1.0f / held_scale<H>(DX ? ctl->max_w : ctl->max_x);
    const float g = (DX ? p.grad[b] : grad_unit(ctl->max_g)) * p.scale;
    T* to = (T*)p.out + (size_t)(DX ? p.row[b] : b) * p.N + a;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (a + k < p.N) to[k] = (T)(v[k] * (1.0f / P_SCALE<H>) * back * g);
}

// dx over several pieces: a wavefront a listed row
template <class T, class H>
__global__ __launch_bounds__(256) void k_nll_dx(const Product p, const Control* ctl) {
    const int r = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (r >= ctl->rows) return;
    const float back = 1.0f / held_scale<H>(ctl->max_w), g = p.grad[r] * p.scale;
    T* to = (T*)p.out + (size_t)p.row[r] * p.N;
    const float* from = p.part + (size_t)r * p.ldo;
    for (int c = lane; c < p.N; c += 64) to[c] = (T)(from[c] * (1.0f / P_SCALE<H>) * back * g);
}

// ------------------------------------------------------------------ host
// Three sizes of tile.  Each holds its workgroups' LDS: 1, 2 and 4 workgroups a CU.
enum Size { LARGE, MEDIUM, SMALL };
struct Config {
    int tile, wgs;
};
constexpr Config CONFIG[3] = {{256, 256}, {128, 512}, {64, 1024}};
template <class T, Form FA, Form FB> using Large = Tile<T, FA, FB, 256, 256, 2, 4>;
template <class T, Form FA, Form FB> using Medium = Tile<T, FA, FB, 128, 128, 2, 2>;
template <class T, Form FA, Form FB> using Small = Tile<T, FA, FB, 64, 64, 2, 2>;

long up(long n, long m) { return (n + m - 1) / m * m; }

// The size whose busiest workgroup is done first: steps of the tiles and shares it takes, times what a step
// takes with the CU's workgroups at work (a large tile's as unit).  Scores of 16,384 rows of 1,024 over 16,384 words
// in bfloat16, whole rounds at every size, take 498, 665 and 849 us: 1, 0.67 and 0.43 a step.  What is picked is the
// fastest or within 2 % of it: 4,096 x 1,024 x 4,096 60 us (71 and 81 with the others), gradient of x at 1,024 x
// 512 x 2,048 49 (58, 78), in float32 85 (138, 239); but scores of 300 x 256 x 1,000 27 where medium takes 25.
Size pick(long a, long b, long nk, bool split) {
    constexpr double step[3] = {1.0, 0.6, 0.4};
    Size best = LARGE;
    double least = 1e300;
    for (int s = 0; s < 3; ++s) {
        const long t = up(a, CONFIG[s].tile) / CONFIG[s].tile * (up(b, CONFIG[s].tile) / CONFIG[s].tile);
        const Rounds r = rounds((int)(t < 1l << 30 ? t : 1l << 30), CONFIG[s].wgs, (int)nk, split);
        const double whole = (double)((r.whole + CONFIG[s].wgs - 1) / CONFIG[s].wgs);
        const double time = step[s] * (whole * (nk + 2.0) + (r.rest ? (double)nk / r.shares + 2.0 : 0.0));
        if (time < least) {
            least = time;
            best = (Size)s;
        }
    }
    return best;
}

// Everything a call lays out in its workspace
struct Plan {
    bool copy_w;
    Size scores, dx, dw;
    long rows, padded, ld;       // ld: elements of a padded row of x and W
    long piece, pieces, vpad, ldo;
    int nk, nk_dx;
    size_t ctl, counts, row, target, lse, grad, x, w, part, score, xg, wh, p, dx_part, dw_part, total;
};

size_t region(size_t& at, size_t bytes) {
    const size_t r = at;
    at += (bytes + 255) / 256 * 256;
    return r;
}

// `table`: the array, or NULL where the size for any is asked for (then it is taken as unaligned)
Plan make_plan(int dtype, int B, int T, int V, int N, bool grad, const void* table) {
    Plan p{};
    const long e = dtype == SEMICRF_F32 ? 4 : 2;
    p.rows = (long)B * T;
    p.padded = up(p.rows, ROW_TILE);
    p.ld = up(N, 64);
    p.nk = (int)(up(N * e, STEP) / STEP);
    p.copy_w = N % 64 || !table || (uintptr_t)table % 16 || (grad && e == 4);
    p.scores = pick(V, p.rows, p.nk, false);
    size_t at = 0;
    p.ctl = region(at, sizeof(Control));
    p.counts = region(at, (size_t)up(p.rows, LIST) / LIST * 4);
    p.row = region(at, p.padded * 4);
    p.target = region(at, p.padded * 4);
    p.x = region(at, p.padded * p.ld * e);
    p.vpad = V;
    if (!grad) {
        const Config c = CONFIG[p.scores];
        const long items = p.padded / c.tile > 4l * c.wgs ? p.padded / c.tile : 4l * c.wgs;
        p.part = region(at, items * 2 * c.tile * sizeof(float2));
        p.score = region(at, p.padded * 4);
    } else {
        p.lse = region(at, p.padded * 4);
        p.grad = region(at, p.padded * 4);
        p.vpad = up(V, 256);
        // pieces of the vocabulary: p takes at most 2 GB, or one large tile of words
        const long most = (2048l << 20) / (p.padded * e) / 256 * 256;
        p.pieces = most < 256 ? p.vpad / 256 : (p.vpad + most - 1) / most;
        p.piece = up((p.vpad + p.pieces - 1) / p.pieces, 256);
        p.pieces = (V + p.piece - 1) / p.piece;
        p.vpad = p.piece * p.pieces;
        p.ldo = up(N, 4);
        p.nk_dx = (int)(p.piece * e / STEP);
        p.dx = pick(N, p.rows, p.nk_dx, p.pieces == 1);
        p.dw = pick(N, p.piece, p.padded * e / STEP, true);
        p.xg = region(at, p.padded * p.ld * e);
        p.wh = region(at, e == 2 ? p.vpad * p.ld * e : 0);
        p.p = region(at, p.padded * p.piece * e);
        // shares of the last round's tiles: at most one a workgroup
        const Config cx = CONFIG[p.dx], cw = CONFIG[p.dw];
        p.dx_part = region(at, p.pieces > 1 ? p.padded * p.ldo * 4 : (size_t)cx.wgs * cx.tile * cx.tile * 4);
        p.dw_part = region(at, (size_t)cw.wgs * cw.tile * cw.tile * 4);
    }
    p.w = region(at, p.copy_w ? (size_t)p.vpad * p.ld * e : 0);
    p.total = at;
    return p;
}

template <class P>
P* in(void* ws, size_t at) { return (P*)((char*)ws + at); }

// f(tile type) of a size
template <class T, Form FA, Form FB, class F>
void with_size(Size s, F&& f) {
    if (s == LARGE) f((Large<T, FA, FB>*)nullptr);
    else if (s == MEDIUM) f((Medium<T, FA, FB>*)nullptr);
    else f((Small<T, FA, FB>*)nullptr);
}

// Lists the rows and lays out what the products read
template <class T, class H, bool GRAD>
Scores gather(const NllArgs& a, const Plan& p, const Listed& list, Layout& l, void* ws, hipStream_t stream) {
    Control* ctl = in<Control>(ws, p.ctl);
    int* counts = in<int>(ws, p.counts);
    const int blocks = (int)(up(p.rows, LIST) / LIST);
    if (blocks > 1)
        hipLaunchKernelGGL(k_nll_count, dim3(blocks), dim3(LIST_THREADS), 0, stream, a, ctl, counts);
    hipLaunchKernelGGL(k_nll_list<GRAD>, dim3(blocks), dim3(LIST_THREADS), 0, stream, a, ctl,
                       blocks > 1 ? counts : nullptr, list);
    if (GRAD && sizeof(H) == 2) {
        // shared out by rows, a quarter at least to either: a row of x waits for its place in the list
        // (15,000 of 100,000 rows of 512, 4,096 words: 19 us, 26 where x always has a quarter; and 11 with 512
        // workgroups of 1,024 threads in place of 2,048 of 256, by fewer atomics)
        const long share = MAX_WGS * p.rows / (p.rows + a.V);
        hipLaunchKernelGGL(k_nll_max<T>, dim3(MAX_WGS), dim3(MAX_THREADS), 0, stream, a, ctl, list.row,
                           (int)(share < MAX_WGS / 4 ? MAX_WGS / 4 : share > MAX_WGS * 3 / 4 ? MAX_WGS * 3 / 4 : share));
    }
    l.x = in<T>(ws, p.x);
    l.w = p.copy_w ? in<T>(ws, p.w) : (void*)a.table;
    l.ld = (int)p.ld;
    l.words = (int)p.vpad;
    l.copy_w = p.copy_w;
    const unsigned cols = (unsigned)(p.ld / 64), x_blocks = (unsigned)(p.padded / 64) * cols;
    const bool w_too = p.copy_w || (GRAD && a.grad_x);
    const unsigned w_blocks = w_too ? (unsigned)((p.vpad + 63) / 64) * cols : 0;
    hipLaunchKernelGGL((k_nll_lay<T, H, GRAD>), dim3(x_blocks + w_blocks), dim3(256), 0, stream, a, ctl, list, l,
                       (int)x_blocks);
    Scores s{};
    s.w = (const char*)l.w;
    s.x = (const char*)l.x;
    s.ld = (unsigned)(p.ld * sizeof(T));
    s.V = a.V;
    s.nk = p.nk;
    const double log2_scale = (double)a.scale * 1.4426950408889634074;
    s.scale = (float)log2_scale;
    s.rest = (float)(log2_scale - s.scale);
    return s;
}

template <class T>
hipError_t run_nll(const NllArgs& a, void* ws, hipStream_t stream) {
    const Plan p = make_plan(a.dtype, a.B, a.T, a.V, a.N, false, a.table);
    Listed list{in<int>(ws, p.row), in<int>(ws, p.target), nullptr, nullptr};
    Layout l{};
    const Scores s = gather<T, T, false>(a, p, list, l, ws, stream);
    const Control* ctl = in<Control>(ws, p.ctl);
    float2* part = in<float2>(ws, p.part);
    float* score = in<float>(ws, p.score);
    with_size<T, ROWS, ROWS>(p.scores, [&](auto* t) {
        using Tl = std::remove_pointer_t<decltype(t)>;
        const int wgs = CONFIG[p.scores].wgs;
        hipLaunchKernelGGL((k_nll_scores<T, Tl>), dim3(wgs), dim3(Tl::NT), 0, stream, s, ctl, list.target, part, score);
        hipLaunchKernelGGL(k_nll_loss, dim3((unsigned)((p.rows + 255) / 256)), dim3(256), 0, stream, ctl, list.row, part,
                           score, a.V, Tl::BA, Tl::BB, Tl::WA, wgs, a.loss, a.lse);
    });
    return hipGetLastError();
}

template <class T>
hipError_t run_nll_grad(const NllArgs& a, void* ws, hipStream_t stream) {
    using H = typename Held<T>::type;
    const Plan p = make_plan(a.dtype, a.B, a.T, a.V, a.N, true, a.table);
    Listed list{in<int>(ws, p.row), in<int>(ws, p.target), in<float>(ws, p.lse), in<float>(ws, p.grad)};
    Layout l{};
    l.xg = in<H>(ws, p.xg);
    l.wh = sizeof(H) == 2 ? (void*)in<H>(ws, p.wh) : (void*)in<T>(ws, p.w);
    const Scores s = gather<T, H, true>(a, p, list, l, ws, stream);
    const Control* ctl = in<Control>(ws, p.ctl);
    H* pp = in<H>(ws, p.p);
    const int ldp = (int)p.piece;
    for (long i = 0; i < p.pieces; ++i) {
        const int v0 = (int)(i * p.piece), words = (int)(a.V - v0 < p.piece ? a.V - v0 : p.piece);
        with_size<T, ROWS, ROWS>(p.scores, [&](auto* t) {
            using Tl = std::remove_pointer_t<decltype(t)>;
            hipLaunchKernelGGL((k_nll_p<T, H, Tl>), dim3(CONFIG[p.scores].wgs), dim3(Tl::NT), 0, stream, s, ctl,
                               list.target, list.lse, v0, ldp / Tl::BA, pp, ldp);
        });
        Product q{};
        q.B = (const char*)pp;
        q.lda = (unsigned)(p.ld * sizeof(H));
        q.ldb = (unsigned)(p.piece * sizeof(H));
        q.N = a.N;
        q.ldo = (int)p.ldo;
        q.scale = a.scale;
        if (a.grad_x)
            with_size<H, COLUMNS, ROWS>(p.dx, [&](auto* t) {
                using Tl = std::remove_pointer_t<decltype(t)>;
                const int wgs = CONFIG[p.dx].wgs;
                Product d = q;
                d.A = (const char*)((H*)l.wh + (size_t)v0 * p.ld);
                d.nk = p.nk_dx;
                d.pieces = p.pieces > 1;
                d.add = i > 0;
                d.last = i + 1 == p.pieces;
                d.part = in<float>(ws, p.dx_part);
                d.row = list.row;
                d.grad = list.grad;
                d.out = a.grad_x;
                hipLaunchKernelGGL((k_nll_product<T, H, Tl, true>), dim3(wgs), dim3(Tl::NT), 0, stream, d, ctl);
                if (!d.pieces && p.nk_dx >= 16)             // else no tile is shared out, whatever the rows
                    hipLaunchKernelGGL((k_nll_join<T, H, true>), dim3(wgs, Tl::BA * Tl::BB / 1024), dim3(256), 0, stream,
                                       d, ctl, Tl::BA, Tl::BB, wgs);
                if (d.pieces && d.last)
                    hipLaunchKernelGGL((k_nll_dx<T, H>), dim3((unsigned)((p.rows + 3) / 4)), dim3(256), 0, stream, d,
                                       ctl);
            });
        if (a.grad_table)
            with_size<H, COLUMNS, COLUMNS>(p.dw, [&](auto* t) {
                using Tl = std::remove_pointer_t<decltype(t)>;
                const int wgs = CONFIG[p.dw].wgs;
                Product d = q;
                d.A = (const char*)l.xg;
                d.b_tiles = ldp / Tl::BB;
                d.b_rows = words;
                d.part = in<float>(ws, p.dw_part);
                d.out = (T*)a.grad_table + (size_t)v0 * a.N;
                hipLaunchKernelGGL((k_nll_product<T, H, Tl, false>), dim3(wgs), dim3(Tl::NT), 0, stream, d, ctl);
                const Rounds rd = rounds(tiles(a.N, Tl::BA) * d.b_tiles, wgs, (int)(p.padded * sizeof(H) / STEP), true);
                if (rd.rest)                                // fewer rows may mean no shares, never more
                    hipLaunchKernelGGL((k_nll_join<T, H, false>), dim3(rd.rest, Tl::BA * Tl::BB / 1024), dim3(256), 0,
                                       stream, d, ctl, Tl::BA, Tl::BB, wgs);
            });
    }
    return hipGetLastError();
}

}  // namespace

size_t token_nll_bytes(int dtype, int B, int T, int V, int N, const void* table, bool grad) {
    return make_plan(dtype, B, T, V, N, grad, table).total;
}

hipError_t launch_token_nll(const NllArgs& a, void* ws, hipStream_t stream) {
    return a.dtype == SEMICRF_F32 ? run_nll<float>(a, ws, stream) : run_nll<bf16>(a, ws, stream);
}

hipError_t launch_token_nll_grad(const NllArgs& a, void* ws, hipStream_t stream) {
    return a.dtype == SEMICRF_F32 ? run_nll_grad<float>(a, ws, stream) : run_nll_grad<bf16>(a, ws, stream);
}

}  // namespace semicrf
