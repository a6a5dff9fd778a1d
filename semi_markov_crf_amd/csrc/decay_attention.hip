// Linear attention with a decay for each head, on gfx950: whole sequences in chunks, forward
// and backward, and one token at a time.
//
//   S_t = gamma S_{t-1} + k_t v_t^T,   o_t = scale q_t^T S_t,   gamma = exp(log_decay[h])
//
// One sweep does it all.  It takes three roles a, b [., Da] and c [., Dc] and a state
// S [Da, Dc], and for each chunk of C positions (i, j local)
//
//   out_i = scale sum_{j <= i} gamma^(i-j) (a_i . b_j) c_j + si gamma^(i+1-e) a_i S
//   S     = gamma^C S + su sum_j gamma^(C-1-j+e) b_j c_j^T
//
//   forward  a, b, c = q, k, v          in order,  state S,   e = 0, si = scale, su = 1
//   dq       a, b, c = do, v, k         in order,  state S^T, e = 0, si = scale, su = 1
//   dv       a, b, c = k, q, do         reversed,  state R,   e = 1, si = 1, su = scale
//   dk       a, b, c = v, do, q         reversed,  state R^T, e = 1, si = 1, su = scale
//
// R is what the later positions send back, R = sum gamma^(i-j) scale q_i do_i^T, and starts
// from the gradient of the final state; at the end it is the gradient of the initial one.
//
// A long sequence is cut into segments: k_attn_state sweeps every segment's state alone from
// zero, k_attn_scan joins them in order, and the sweep then runs over all segments at once,
// each from its own start.
//
// The products run on the matrix cores.  A wavefront owns VT columns tiles of c (and of the
// state, which stays in fp32 accumulators for the whole sweep) and all rows; the masked
// products a.b^T of a chunk are shared out by rows and exchanged through LDS.
//
// Rounding (bfloat16): inputs are exact.  The masked products enter the second product, and the
// state the rows that read it, as the sum of two bfloat16 numbers (16 bits): their error is 2^-8 of
// the output's own rounding to 8 bits.  One number instead of two would add an error as large as
// the output's.  c scaled by its decay is the sum of three (24 bits) when the state is updated, so
// that the state itself keeps fp32 accuracy.
#include "common.h"
#include "encoder.h"

namespace semicrf {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// raw buffer: no stride, no swizzle, 32-bit data format, out of range reads 0 and drops writes
constexpr int BUFFER_FLAGS = 0x00027000;

// ------------------------------------------------------------------ matrix products
// A product step contracts KS indices.  Lane l = 16 g + r holds, of row (or column) r, the E
// contraction indices that `order` lists; both operands list the same ones, so any order gives
// the same product.  The result tile holds column r, rows 4 g .. 4 g + 3.  The order used is the
// one in which result tiles lie in registers, four rows of a 16-row tile after four of the
// next: the state's accumulators are an operand as they are, and the transposing LDS read
// fetches four rows at a time.
template <class T>
struct Mma;

template <>
struct Mma<bf16> {
    static constexpr int E = 8, KS = 32;
    typedef bf16x8 Frag;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

template <>
struct Mma<float> {
    static constexpr int E = 4, KS = 16;
    typedef f32x4 Frag;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
};

// Where index i of a row stands when it is stored in the order of product steps: in blocks of
// 32, 8 g + e holds index 4 g + e, 8 g + 4 + e index 16 + 4 g + e (fp32 steps take 16: no change).
template <class T>
__device__ __forceinline__ constexpr int ordered(int i) {
    return sizeof(T) == 4 ? i : (i & ~31) + 8 * ((i & 15) >> 2) + 4 * ((i & 31) >> 4) + (i & 3);
}

// Row `row + r` of a buffer whose rows are stored in the order of product steps
template <class T>
__device__ __forceinline__ typename Mma<T>::Frag frag_ordered(const T* buf, int ld, int row, int k0) {
    const int l = threadIdx.x & 63;
    return *(const typename Mma<T>::Frag*)(buf + (row + (l & 15)) * ld + k0 + (l >> 4) * Mma<T>::E);
}
// ... and of one whose rows are stored as they are
__device__ __forceinline__ bf16x8 frag_row(const bf16* buf, int ld, int row, int k0) {
    const int l = threadIdx.x & 63;
    const bf16* at = buf + (row + (l & 15)) * ld + k0 + (l >> 4) * 4;
    return __builtin_shufflevector(*(const bf16x4*)at, *(const bf16x4*)(at + 16), 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ f32x4 frag_row(const float* buf, int ld, int row, int k0) {
    return frag_ordered<float>(buf, ld, row, k0);
}

// Column c0 + r, rows k0 .. of a step
__device__ __forceinline__ bf16x8 frag_col(const bf16* buf, int ld, int k0, int c0) {
    // the transposing read gives lane 16 g + i the i-th column of the 4 x 16 block whose row j
    // is what lanes 16 g + 4 j .. + 3 point at, four elements each
    const int l = threadIdx.x & 63, g = l >> 4, p = l & 15;
    typedef __attribute__((address_space(3))) bf16x4 Lds;
    const bf16* at = buf + (k0 + 4 * g + (p >> 2)) * ld + c0 + 4 * (p & 3);
    const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((Lds*)at);
    const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((Lds*)(at + 16 * ld));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ f32x4 frag_col(const float* buf, int ld, int k0, int c0) {
    const int l = threadIdx.x & 63, g = l >> 4, r = l & 15;
    const float* at = buf + (k0 + 4 * g) * ld + c0 + r;
    return f32x4{at[0], at[ld], at[2 * ld], at[3 * ld]};
}
// Row of a step that element j of this lane's fragment holds
template <class T>
__device__ __forceinline__ int step_row(int j) {
    const int g = (threadIdx.x & 63) >> 4;
    return sizeof(T) == 4 ? 4 * g + j : 4 * g + (j & 3) + 16 * (j >> 2);
}

// Elements between rows in LDS.  Measured on row reads, transposing reads and piece writes: 16
// bfloat16 of padding cost no bank conflicts in any of them, 8 do in all.
template <class T>
constexpr int lds_pitch(int width) { return width + (sizeof(T) == 4 ? 4 : 16); }

// Parts of an fp32 fragment that add up to it: one in fp32, n in bfloat16 (8 bits each).  Two
// elements at a time, as the conversion takes them.
template <class T, int N>
struct Parts {
    typename Mma<T>::Frag f[N];
    __device__ __forceinline__ void set(int j, float x, float y) {
        if constexpr (sizeof(T) == 4) {
            f[0][j] = x;
            f[0][j + 1] = y;
        } else {
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            f32x2 r = {x, y};
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const bf16x2 h = __builtin_convertvector(r, bf16x2);
                f[n][j] = h[0];
                f[n][j + 1] = h[1];
                if (n + 1 < N) {
                    const uint32_t u = __builtin_bit_cast(uint32_t, h);
                    r[0] -= __builtin_bit_cast(float, u << 16);
                    r[1] -= __builtin_bit_cast(float, u & 0xffff0000u);
                }
            }
        }
    }
};
template <class T>
constexpr int state_parts() { return sizeof(T) == 4 ? 1 : 2; }
template <class T>
constexpr int masked_parts() { return sizeof(T) == 4 ? 1 : 2; }
template <class T>
constexpr int update_parts() { return sizeof(T) == 4 ? 1 : 3; }
// Whether a chunk's update is summed up by itself before the state takes it.  Every product added
// to the state is rounded at the state's size; with slow decays 8 and more a chunk made the errors of
// fp32 outputs 6e-7 to 9e-7, where 2.7e-7 are left with one.  In bfloat16 they are far below the output's
// rounding.
template <class T>
constexpr bool update_apart() { return sizeof(T) == 4; }

// Four consecutive masked products as parts that add up to them, each part's array `stride`
// elements after the one before.
__device__ __forceinline__ void put_masked(float* to, int, f32x4 x) { *(f32x4*)to = x; }
__device__ __forceinline__ void put_masked(bf16* to, int stride, f32x4 x) {
    Parts<bf16, masked_parts<bf16>()> p;
    p.set(0, x[0], x[1]);
    p.set(2, x[2], x[3]);
#pragma unroll
    for (int n = 0; n < masked_parts<bf16>(); ++n)
        *(bf16x4*)(to + n * stride) = __builtin_shufflevector(p.f[n], p.f[n], 0, 1, 2, 3);
}

// ------------------------------------------------------------------ a sweep
struct Role {
    const void* p;
    long sb, st, sh;         // strides in elements
    int group;               // query heads that share a head of this role
};

struct Sweep {
    Role a, b, c;
    int B0, B1;              // sequences of a launch
    int T, H, Da, Dc;        // H: query heads
    const int32_t* lengths;
    const float* log_decay;
    float scale, si, su;
    int e, reverse;
    int seg, nseg;           // positions per segment (a multiple of the chunk), segments
    const float* state;      // start of every segment [B, H, nseg, ...] or NULL for zeros
    int state_nseg;          // segments of `state`
    int transposed;          // the state in memory is [Dc, Da]
    float* state_out;        // after the last position (one segment only), or NULL
    float* local;            // k_attn_state: state of each segment alone
    void* out;               // [B, T, H, Dc] in T, or fp32 where `out32`
    int out32;
    int32_t* status;
};

// Sweeps of one shape that run in one launch.
template <int N>
struct Sweeps {
    Sweep s[N];
};

// Workgroup -> (sweep, batch row, query head, segment).  What shares a key / value head and a
// segment reads the same rows, so it runs at the same time on the same chiplet: consecutive
// workgroups go to the 8 chiplets in turn, and members of a unit are 8 apart.
struct Place {
    int sweep, b, h, seg;
};
constexpr int CHIPLETS = 8;
__device__ __forceinline__ bool place(const Sweep& w, int sweeps, int group, Place& p) {
    const int members = sweeps * group;
    const int id = blockIdx.x, lane = id % CHIPLETS, rest = id / CHIPLETS;
    const int m = rest % members;
    int u = rest / members * CHIPLETS + lane;
    p.sweep = m / group;
    const int hk = w.H / group;
    p.seg = u % w.nseg;
    u /= w.nseg;
    p.h = u % hk * group + m % group;
    p.b = w.B0 + u / hk;
    return p.b < w.B1;
}

__device__ __forceinline__ float power(float g2, int n) {
    return n == 0 ? 1.0f : __builtin_amdgcn_exp2f(g2 * (float)n);
}

// How a kernel reads its rows and what it leaves out.
//   FULL: rows fill the padded width P exactly, by buffer descriptors.
//   PART: by buffer descriptors; tiles of products past Da and columns past Dc are left out.
//   LOOSE: rows of any width, stride and alignment, by pointers; the same left out.
// A descriptor spans exactly the chunk's valid rows, less than 2^29 bytes, so that rows and columns
// out of range read as zeros with no branch (bit 31 of the offset puts a column out of range); rows
// are then whole pieces of 16 bytes from dword addresses.  Measured in bfloat16: 32 x 800 positions,
// 8 heads of 64 columns 34 us FULL, 44 LOOSE; 16 x 800 of 40 and 48 columns 33 PART, 41 LOOSE; of 128
// and 64 columns 48 PART, 51 FULL with 128 and 128.
enum { FULL, PART, LOOSE };

// A chunk's rows of one role on their way from memory to LDS, in 16-byte pieces; a thread's
// column piece is the same in all its rows.
template <class T, int P, int C, int NT, int MODE>
struct Tile {
    static constexpr int V = 16 / sizeof(T), PPR = P / V, LD = lds_pitch<T>(P), RPS = NT / PPR;
    static constexpr int NP = C / RPS;
    static_assert(NT % PPR == 0 && C % RPS == 0, "pieces per thread");
    u32x4 x[NP];
    int shift;               // LOOSE: bits that the row's last piece starts early

    // m valid rows from sweep index t0 (position L - t0 - m is the lowest of a reversed chunk)
    __device__ __forceinline__ void load(const Role& w, const T* seq, int D, int t0, int m, int L, int reverse) {
        const int row0 = threadIdx.x / PPR, c = (threadIdx.x % PPR) * V;
        if constexpr (MODE != LOOSE) {
            const int stb = (int)w.st * (int)sizeof(T);
            const T* base = seq + (long)(reverse ? L - t0 - m : t0) * w.st;
            const __amdgpu_buffer_rsrc_t buf = __builtin_amdgcn_make_buffer_rsrc(
                (void*)base, 0, m > 0 ? (m - 1) * stb + D * (int)sizeof(T) : 0, BUFFER_FLAGS);
            const int step = reverse ? -stb : stb;
            uint32_t off = (c < D ? c * (uint32_t)sizeof(T) : 0x80000000u) + (uint32_t)(row0 * step) +
                           (uint32_t)(reverse ? (m - 1) * stb : 0);
#pragma unroll
            for (int n = 0; n < NP; ++n) x[n] = __builtin_amdgcn_raw_buffer_load_b128(buf, off + n * RPS * step, 0, 0);
        } else {
            // a last piece past the row's end is read from D - V on and shifted when it is put
            const int at = D < V ? 0 : min(c, D - V);
            shift = D < V ? 0 : (c - at) * 8 * (int)sizeof(T);
            const long st = reverse ? -w.st : w.st;
            const T* p = seq + (long)(reverse ? L - 1 - t0 : t0) * w.st + row0 * st + at;
#pragma unroll
            for (int n = 0; n < NP; ++n, p += RPS * st) {
                x[n] = u32x4{0, 0, 0, 0};
                if (row0 + n * RPS < m && c < D) {
                    if (D >= V) {
                        x[n] = *(const loose_piece*)p;
                    } else {
                        T e[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) e[i] = i < D ? p[i] : (T)0.0f;
                        __builtin_memcpy(&x[n], e, 16);
                    }
                }
            }
        }
    }
    __device__ __forceinline__ u32x4 piece(int n) const {
        if constexpr (MODE != LOOSE) return x[n];
        const uint64_t lo = (uint64_t)x[n][1] << 32 | x[n][0], hi = (uint64_t)x[n][3] << 32 | x[n][2];
        const int s = shift & 63;
        const uint64_t l = shift & 64 ? hi : lo, h = shift & 64 ? 0 : hi;
        const uint64_t a = l >> s | h << 1 << (63 - s), b = h >> s;
        return shift < 128 ? u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)} : u32x4{0, 0, 0, 0};
    }
    // ORDERED: columns in the order of product steps
    template <bool ORDERED>
    __device__ __forceinline__ void put(T* buf) const {
        const int row0 = threadIdx.x / PPR, c = (threadIdx.x % PPR) * V;
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            T* row = buf + (row0 + n * RPS) * LD;
            const u32x4 y = piece(n);
            if constexpr (ORDERED && sizeof(T) == 2) {
                *(u32x2*)(row + ordered<T>(c)) = u32x2{y[0], y[1]};
                *(u32x2*)(row + ordered<T>(c + 4)) = u32x2{y[2], y[3]};
            } else {
                *(u32x4*)(row + c) = y;
            }
        }
    }
};

template <class T>
__device__ __forceinline__ const T* role_base(const Role& r, int b, int h) {
    return (const T*)r.p + (long)b * r.sb + (long)(h / r.group) * r.sh;
}

// One wavefront for each 16 columns of the state.
constexpr int sweep_waves(int P) { return P / 16; }
// Wavefronts a SIMD that the sweep's registers are held to: as many as run with no more than a
// dozen values spilled, and in bfloat16 of width 32 as the LDS lets run.
template <class T, int P>
constexpr int sweep_occupancy() { return P == 128 || (sizeof(T) == 2 && P == 32) ? 2 : sizeof(T) == 2 ? 3 : 4; }

// gamma^m of the state.  Near 1 it is applied as S + (gamma^m - 1) S: over thousands of chunks, or
// of single tokens, a factor rounded once would bend every old contribution the same way.
struct Decay {
    float f;
    int near1;               // the same in every lane
    __device__ __forceinline__ void set(float g, int m) {
        f = m == 0 ? 1.0f : expf(g * (float)m);
        near1 = __builtin_amdgcn_readfirstlane(f > 0.5f);
        if (near1) f = m == 0 ? 0.0f : expm1f(g * (float)m);
    }
};

// With e = 1 every weight of the update has a factor gamma.  A power of two near 1 / gamma, at most
// 2^60, is kept in the state while it lies in registers, so that the low parts of c times its
// weight do not underflow.
__device__ __forceinline__ float state_scale(float g2, int e) {
    return e ? __builtin_amdgcn_exp2f(fminf(60.0f, fmaxf(-60.0f, rintf(-g2)))) : 1.0f;
}

// State tiles of a wavefront: all rows, its own columns.
template <class T, int P>
struct State {
    static constexpr int NW = sweep_waves(P), VT = P / 16 / NW, ST = P / 16;
    static constexpr int KS = Mma<T>::KS, E = Mma<T>::E, TPK = KS / 16;   // state tiles a step
    f32x4 s[ST][VT];

    __device__ __forceinline__ int col(int vt) const {
        return ((threadIdx.x >> 6) * VT + vt) * 16 + (threadIdx.x & 15);
    }
    __device__ __forceinline__ int row(int t, int r) const {
        return 16 * t + 4 * ((threadIdx.x & 63) >> 4) + r;
    }
    __device__ __forceinline__ void load(const float* p, int Da, int Dc, bool transposed, float scale) {
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int v = 0; v < VT; ++v)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = row(t, r), j = col(v);
                    s[t][v][r] = p && i < Da && j < Dc ? p[transposed ? j * Da + i : i * Dc + j] * scale : 0.0f;
                }
    }
    __device__ __forceinline__ void store(float* p, int Da, int Dc, bool transposed, float scale) const {
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int v = 0; v < VT; ++v)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = row(t, r), j = col(v);
                    if (i < Da && j < Dc) p[transposed ? j * Da + i : i * Dc + j] = s[t][v][r] * scale;
                }
    }
    __device__ __forceinline__ void decay(Decay d) {
        if (d.near1) {
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int v = 0; v < VT; ++v)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[t][v][r] = fmaf(s[t][v][r], d.f, s[t][v][r]);
        } else {
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int v = 0; v < VT; ++v)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[t][v][r] *= d.f;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int v = 0; v < VT; ++v) s[t][v] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // gamma^m S + u
    __device__ __forceinline__ void add(Decay d, const State& u) {
        if (d.near1) {
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int v = 0; v < VT; ++v)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[t][v][r] += fmaf(s[t][v][r], d.f, u.s[t][v][r]);
        } else {
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int v = 0; v < VT; ++v)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[t][v][r] = fmaf(s[t][v][r], d.f, u.s[t][v][r]);
        }
    }
    // S += sum_j w_j b_j c_j^T over one product step from row k0; `c` the columns' fragments.  Rows
    // of S from `rows` on are left out, 32 at a time.
    struct Step {
        typename Mma<T>::Frag a[ST];
        Parts<T, update_parts<T>()> p[VT];
        __device__ __forceinline__ void prepare(const T* bbuf, int ld, int k0, const typename Mma<T>::Frag (&c)[VT],
                                                const float (&w)[E]) {
#pragma unroll
            for (int t = 0; t < ST; ++t) a[t] = frag_col(bbuf, ld, k0, 16 * t);
#pragma unroll
            for (int v = 0; v < VT; ++v)
#pragma unroll
                for (int j = 0; j < E; j += 2) p[v].set(j, (float)c[v][j] * w[j], (float)c[v][j + 1] * w[j + 1]);
        }
    };
    template <int MODE>
    __device__ __forceinline__ void update(const Step& x, int rows) {
        constexpr int TG = MODE == FULL ? ST : 2;
#pragma unroll
        for (int t0 = 0; t0 < ST; t0 += TG)
            if (MODE == FULL || 16 * t0 < rows)
#pragma unroll
                for (int n = 0; n < update_parts<T>(); ++n)
#pragma unroll
                    for (int t = t0; t < t0 + TG; ++t)
#pragma unroll
                        for (int v = 0; v < VT; ++v) s[t][v] = Mma<T>::mma(x.a[t], x.p[v].f[n], s[t][v]);
    }
};

// su gamma^(m-1-j+e) for the rows j this lane holds of the step from row k0 (0 past m).
template <class T>
__device__ __forceinline__ void update_weights(float g2, float su, int k0, int m, int e, float (&w)[Mma<T>::E]) {
#pragma unroll
    for (int j = 0; j < Mma<T>::E; ++j) {
        const int i = k0 + step_row<T>(j);
        w[j] = i < m ? su * power(g2, m - 1 - i + e) : 0.0f;
    }
}

// The update of full chunks: weights of the last product step (earlier steps are gamma^KS
// apart) and the state's decay.  A sequence's last, partial chunk is left out of it (`skip`) and
// added by update_rest after the loop, where it matters.
template <class T, int C>
struct Update {
    static constexpr int KS = Mma<T>::KS, E = Mma<T>::E;
    float last[E], step;
    Decay d;
    __device__ __forceinline__ void set(float g, float g2, float su, int e) {
        update_weights<T>(g2, su, 0, KS, e, last);
        step = power(g2, KS);
        d.set(g, C);
    }
    __device__ __forceinline__ void skip() {
#pragma unroll
        for (int j = 0; j < E; ++j) last[j] = 0.0f;
        d.set(0.0f, 0);
    }
    __device__ __forceinline__ void get(int k0, float (&w)[E]) const {
        float f = 1.0f;
#pragma unroll
        for (int k = k0 + KS; k < C; k += KS) f *= step;
#pragma unroll
        for (int j = 0; j < E; ++j) w[j] = last[j] * f;
    }
};
template <class T, int P, int C>
__device__ __forceinline__ void update_rest(State<T, P>& S, const T* sb, const T* sc, int m, float g, float g2,
                                            float su, int e) {
    constexpr int LD = lds_pitch<T>(P), VT = State<T, P>::VT;
    Decay d;
    d.set(g, m);
    S.decay(d);
#pragma unroll 1
    for (int k0 = 0; k0 < C; k0 += Mma<T>::KS) {
        typename Mma<T>::Frag c[VT];
#pragma unroll
        for (int v = 0; v < VT; ++v) c[v] = frag_col(sc, LD, k0, ((threadIdx.x >> 6) * VT + v) * 16);
        float u[Mma<T>::E];
        update_weights<T>(g2, su, k0, m, e, u);
        typename State<T, P>::Step x;
        x.prepare(sb, LD, k0, c, u);
        S.template update<FULL>(x, P);
    }
}

// The state of every segment alone, from zero: S = sum_j su gamma^(m-1-j+e) b_j c_j^T, a chunk at a
// time.  Bound by HBM where segments are many: 4 x 100,000 positions, 8 heads of 64 columns, 0.82 GB
// of bfloat16 in 175 us (4.7 TB/s).  fp32 takes the slower matrix instructions: 100,001 positions, 6
// heads, both states of the gradients, 0.61 GB in 152 us (4.0 TB/s).
template <class T, int P, int C, int MODE, int N>
__global__ __launch_bounds__(64 * sweep_waves(P), P == 128 ? 2 : 4) void
k_attn_state(const Sweeps<N> set, int group) {
    using M = Mma<T>;
    using St = State<T, P>;
    constexpr int NT = 64 * St::NW, VT = St::VT;
    using Tl = Tile<T, P, C, NT, MODE>;
    __shared__ __align__(16) T sb[C * Tl::LD], sc[C * Tl::LD];
    Place at;
    if (!place(set.s[0], N, group, at)) return;
    const Sweep w = set.s[N == 1 ? 0 : at.sweep];
    const int seg = at.seg, h = at.h, b = at.b;
    const int L = __builtin_amdgcn_readfirstlane(seq_length(w.lengths, b, w.T, w.status));
    const int t_begin = seg * w.seg, t_end = min(L, t_begin + w.seg);
    const float g = w.log_decay[h], g2 = g * (float)LOG2E, sigma = state_scale(g2, w.e), su = w.su * sigma;
    const T* pb = role_base<T>(w.b, b, h);
    const T* pc = role_base<T>(w.c, b, h);
    Tl tb, tc;
    tb.load(w.b, pb, w.Da, t_begin, min(C, t_end - t_begin), L, w.reverse);
    tc.load(w.c, pc, w.Dc, t_begin, min(C, t_end - t_begin), L, w.reverse);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool mine = MODE == FULL || wave * VT * 16 < w.Dc;     // columns of this wavefront
    St S;
    S.load(nullptr, 0, 0, false, 1.0f);
    Update<T, C> up;
    up.set(g, g2, su, w.e);
    for (int t0 = t_begin; t0 < t_end; t0 += C) {
        const int m = min(C, t_end - t0);
        __syncthreads();
        tb.template put<false>(sb);
        tc.template put<false>(sc);
        __syncthreads();
        if (t0 + C < t_end) {
            const int mn = min(C, t_end - t0 - C);
            tb.load(w.b, pb, w.Da, t0 + C, mn, L, w.reverse);
            tc.load(w.c, pc, w.Dc, t0 + C, mn, L, w.reverse);
        }
        if (!mine) continue;
        if (m < C) up.skip();
        St chunk;
        St& sum = update_apart<T>() ? chunk : S;
        if constexpr (update_apart<T>()) chunk.clear();
        else S.decay(up.d);
#pragma unroll
        for (int k0 = 0; k0 < C; k0 += M::KS) {
            typename M::Frag c[VT];
#pragma unroll
            for (int v = 0; v < VT; ++v) c[v] = frag_col(sc, Tl::LD, k0, (wave * VT + v) * 16);
            float u[M::E];
            up.get(k0, u);
            typename St::Step x;
            x.prepare(sb, Tl::LD, k0, c, u);
            __builtin_amdgcn_sched_barrier(0);
            sum.template update<MODE>(x, w.Da);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (update_apart<T>()) S.add(up.d, chunk);
    }
    if (t_end > t_begin && (t_end - t_begin) % C)
        update_rest<T, P, C>(S, sb, sc, (t_end - t_begin) % C, g, g2, su, w.e);
    S.store(w.local + (((size_t)b * w.H + h) * w.nseg + seg) * w.Da * w.Dc, w.Da, w.Dc, false, 1.0f / sigma);
}

// As Decay, of the many positions of a segment
struct Decay64 {
    float f;
    bool near1;
    __device__ __forceinline__ Decay64(double g, int m) {
        const double e = m == 0 ? 1.0 : exp(g * m);
        near1 = e > 0.5;
        f = (float)(m == 0 ? 0.0 : near1 ? expm1(g * m) : e);
    }
};

// Start of every segment from the segments' own states, in place, in order; the state after
// the last position to `out`.  One or two states: blockIdx.y = state * H + head.  Bound by the
// latency of its loads, 16 segments at a time: 23 segments of 32 heads, 12 MB, 9.5 us.
// grid (ceil(D / 256), states * H, B), D = Da Dc
struct Scan {
    float* local[2];
    const float* init[2];
    float* out[2];
    const int32_t* lengths;
    const float* log_decay;
    int T, H, seg, nseg, D;
};
__global__ __launch_bounds__(256) void k_attn_scan(const Scan a) {
    const int i = blockIdx.x * 256 + threadIdx.x, which = blockIdx.y / a.H, h = blockIdx.y % a.H, b = blockIdx.z;
    const int T = a.T, H = a.H, seg = a.seg, nseg = a.nseg, D = a.D;
    float* const local = a.local[which];
    const float* const init = a.init[which];
    float* const out = a.out[which];
    if (i >= D) return;
    const size_t bh = (size_t)b * H + h;
    const int L = seq_length(a.lengths, b, T, nullptr);
    const double g = a.log_decay[h];
    float cur = init ? init[bh * D + i] : 0.0f;
    const Decay64 full(g, seg);
    float* p = local + bh * nseg * D + i;
    // the loads do not wait for one another: U at a time
    constexpr int U = 16;
    for (int s0 = 0; s0 < nseg; s0 += U) {
        float own[U];
#pragma unroll
        for (int n = 0; n < U; ++n) own[n] = s0 + n < nseg ? p[(size_t)(s0 + n) * D] : 0.0f;
#pragma unroll
        for (int n = 0; n < U; ++n) {
            const int s = s0 + n;
            if (s >= nseg) break;
            p[(size_t)s * D] = cur;
            const int m = min(seg, max(0, L - s * seg));
            const Decay64 d = m == seg ? full : Decay64(g, m);
            cur = (d.near1 ? cur : 0.0f) + fmaf(cur, d.f, own[n]);
        }
    }
    if (out) out[bh * D + i] = cur;
}

// Four consecutive columns of an output row.
template <class O>
__device__ __forceinline__ void store4(const __amdgpu_buffer_rsrc_t& buf, uint32_t off, const f32x4& x) {
    if constexpr (sizeof(O) == 4) {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), buf, off, 0, 0);
    } else {
        const bf16x4 h = {(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]};
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, h), buf, off, 0, 0);
    }
}

// Rows i < m of a chunk from result tiles that hold column i = 16 it + r, rows (of the tile)
// four consecutive output columns from `col`.
template <class O, int MODE, int IT, int VT>
__device__ __forceinline__ void store_rows(const Sweep& w, O* seq, int t0, int m, int L, int col,
                                           const f32x4 (&acc)[IT][VT]) {
    const int r16 = threadIdx.x & 15;
    const long ost = (long)w.H * w.Dc;
    if constexpr (MODE != LOOSE) {
        const int stb = (int)ost * (int)sizeof(O), step = w.reverse ? -stb : stb;
        O* base = seq + (long)(w.reverse ? L - t0 - m : t0) * ost;
        const __amdgpu_buffer_rsrc_t buf = __builtin_amdgcn_make_buffer_rsrc(
            (void*)base, 0, (m - 1) * stb + w.Dc * (int)sizeof(O), BUFFER_FLAGS);
        const uint32_t off = (uint32_t)(r16 * step) + (uint32_t)(w.reverse ? (m - 1) * stb : 0);
#pragma unroll
        for (int v = 0; v < VT; ++v) {
            const int c = col + 16 * v;
            const uint32_t at = off + (c < w.Dc ? c * (uint32_t)sizeof(O) : 0x80000000u);
#pragma unroll
            for (int it = 0; it < IT; ++it) store4<O>(buf, at + it * 16 * step, acc[it][v]);
        }
    } else {
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int i = 16 * it + r16;
            if (i < m) {
                O* p = seq + (long)(w.reverse ? L - 1 - t0 - i : t0 + i) * ost;
#pragma unroll
                for (int v = 0; v < VT; ++v) {
                    const int c = col + 16 * v;
                    O y[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[r] = (O)acc[it][v][r];
                    if (c + 4 <= w.Dc) {
                        __builtin_memcpy(p + c, y, sizeof(y));
                    } else {
#pragma unroll
                        for (int r = 0; r < 3; ++r)
                            if (c + r < w.Dc) p[c + r] = y[r];
                    }
                }
            }
        }
    }
}

// The sweep over every segment from its start.  A chunk: its rows go from registers to LDS (the next
// chunk's loads leave at once), the masked products are shared out and exchanged through LDS, then
// each wavefront has its columns to itself: the state's part, the chunk's own part, the update.  The
// fragments of a product step are read and split ahead of its products (scheduling barriers keep
// them there), and products that add to one tile are apart.
// Medians of a few calls after a start: 4 x 100,000 positions, 8 heads of 64 columns in bfloat16:
// 1.64 GB in 397 us (4.1 TB/s), bound by HBM; 32 x 800 positions, 8 heads on 256 workgroups: 36 us (34
// in many calls), bound by the latency of 13 chunks in order, some 5,500 cycles each (rows into LDS
// 650, next loads 450, masked products 1,000, state's part 650, own part and update 1,800, stores and
// the wait for loads 750).  The three sweeps of the gradients in fp32, 100,001 positions, 6 heads: 40
// GFLOP of matrix instructions in 476 us (387 to 552), 84 of the 155 TFLOP/s that a large product
// reaches.
template <class T, int P, int C, int MODE, int N>
__global__ __launch_bounds__(64 * sweep_waves(P), (sweep_occupancy<T, P>())) void
k_attn_sweep(const Sweeps<N> set, int group) {
    using M = Mma<T>;
    using St = State<T, P>;
    constexpr int NW = St::NW, NT = 64 * NW, VT = St::VT, IT = C / 16, KS = M::KS, E = M::E;
    using Tl = Tile<T, P, C, NT, MODE>;
    constexpr int LDM = lds_pitch<T>(C), MP = masked_parts<T>();
    __shared__ __align__(16) T sa[C * Tl::LD], sb[C * Tl::LD], sc[C * Tl::LD], sm[MP * C * LDM];
    Place at;
    if (!place(set.s[0], N, group, at)) return;
    const Sweep w = set.s[N == 1 ? 0 : at.sweep];
    const int seg = at.seg, h = at.h, b = at.b;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int gr = lane >> 4, r16 = lane & 15;
    const int L = __builtin_amdgcn_readfirstlane(seq_length(w.lengths, b, w.T, w.status));
    const int t_begin = seg * w.seg, t_last = min(w.T, t_begin + w.seg), t_end = min(L, t_last);
    const float g = w.log_decay[h], g2 = g * (float)LOG2E, sigma = state_scale(g2, w.e), su = w.su * sigma;
    const size_t bh = (size_t)b * w.H + h;
    const size_t D = (size_t)w.Da * w.Dc;
    const size_t out0 = (size_t)b * w.T * w.H * w.Dc + (size_t)h * w.Dc;
    const T* pa = role_base<T>(w.a, b, h);
    const T* pb = role_base<T>(w.b, b, h);
    const T* pc = role_base<T>(w.c, b, h);
    Tl ta, tb, tc;
    {
        const int m = min(C, t_end - t_begin);
        ta.load(w.a, pa, w.Da, t_begin, m, L, w.reverse);
        tb.load(w.b, pb, w.Da, t_begin, m, L, w.reverse);
        tc.load(w.c, pc, w.Dc, t_begin, m, L, w.reverse);
    }
    // padding: positions from the length on
    for (int t = max(t_begin, L) + threadIdx.x / 16; t < t_last; t += NT / 16)
        for (int j = r16; j < w.Dc; j += 16) {
            const size_t to = out0 + (size_t)t * w.H * w.Dc + j;
            if (w.out32) ((float*)w.out)[to] = 0.0f;
            else ((T*)w.out)[to] = (T)0.0f;
        }
    St S;
    S.load(w.state ? w.state + (bh * w.state_nseg + (w.state_nseg > 1 ? seg : 0)) * D : nullptr, w.Da,
           w.Dc, w.transposed, sigma);
    // Weights of the masked products, scale gamma^(i-j) where i >= j.  BIG: three tiles of 32 x 32, a
    // wavefront each; lanes hold column i = r32, rows j = 8 q + 4 h32 + r.  Otherwise in tiles of 16
    // (rows j = 4 gr + r, column i = r16): on the diagonal, and one tile off it.  16 x 800 positions, 8
    // heads of 128 columns: 50.5 us against 52.8 in tiles of 16, the gradients 99.9 against 104.7.
    constexpr bool BIG = sizeof(T) == 2 && NW >= 4;
    const int r32 = lane & 31, h32 = lane >> 5;
    float own[BIG ? 16 : 1], diag[4], below[4], inter[IT];
    if constexpr (BIG) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int d = r32 - 8 * (i / 4) - 4 * h32 - i % 4 + (wave == 2 ? 32 : 0);
            own[i] = d >= 0 ? w.scale * power(g2, d) : 0.0f;
        }
    } else {
        // products above the diagonal stay zero
        for (int i = threadIdx.x; i < MP * C * LDM; i += NT) sm[i] = (T)0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = r16 - 4 * gr - r;
            diag[r] = d >= 0 ? w.scale * power(g2, d) : 0.0f;
            below[r] = w.scale * power(g2, 16 + d);
        }
    }
#pragma unroll
    for (int it = 0; it < IT; ++it) inter[it] = w.si / sigma * power(g2, 16 * it + r16 + 1 - w.e);
    const float g16 = power(g2, 16);
    const bool mine = MODE == FULL || wave * VT * 16 < w.Dc;     // columns of this wavefront
    Update<T, C> up;
    up.set(g, g2, su, w.e);
    wait_loads();
    for (int t0 = t_begin; t0 < t_end; t0 += C) {
        const int m = min(C, t_end - t0);
        __syncthreads();
        ta.template put<true>(sa);
        tb.template put<false>(sb);
        tc.template put<false>(sc);
        __syncthreads();
        if (t0 + C < t_end) {
            const int mn = min(C, t_end - t0 - C);
            ta.load(w.a, pa, w.Da, t0 + C, mn, L, w.reverse);
            tb.load(w.b, pb, w.Da, t0 + C, mn, L, w.reverse);
            tc.load(w.c, pc, w.Dc, t0 + C, mn, L, w.reverse);
        }
        // masked products: the tiles on and below the diagonal, dealt out to the wavefronts
        if constexpr (BIG) {
            if (wave < 3) {
                const int it = wave > 0 ? 32 : 0, jt = wave == 1 ? 32 : 0;
                const bf16* rb = (const bf16*)sb + (jt + r32) * Tl::LD + 4 * h32;
                const bf16* ra = (const bf16*)sa + (it + r32) * Tl::LD + 8 * h32;
                f32x16 acc = {};
#pragma unroll
                for (int k1 = 0; k1 < P; k1 += 32)
                    if (MODE == FULL || k1 < w.Da)
#pragma unroll
                        for (int s = 0; s < 2; ++s)
                            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                __builtin_shufflevector(*(const bf16x4*)(rb + k1 + 8 * s),
                                                        *(const bf16x4*)(rb + k1 + 8 * s + 16), 0, 1, 2, 3, 4, 5, 6, 7),
                                *(const bf16x8*)(ra + k1 + 16 * s), acc, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    T* to = sm + (it + r32) * LDM + ordered<T>(jt + 8 * q + 4 * h32);
                    put_masked(to, C * LDM, f32x4{acc[4 * q] * own[4 * q], acc[4 * q + 1] * own[4 * q + 1],
                                                  acc[4 * q + 2] * own[4 * q + 2], acc[4 * q + 3] * own[4 * q + 3]});
                }
            }
        } else {
            // the products of all its tiles do not wait for one another
            constexpr int NT2 = IT * (IT + 1) / 2, ROUNDS = (NT2 + NW - 1) / NW;
            f32x4 acc[ROUNDS];
            auto tile = [&](int n, int& it, int& jt) {
                it = n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3;
                jt = n - it * (it + 1) / 2;
            };
#pragma unroll
            for (int k = 0; k < ROUNDS; ++k) {
                const int n = k * NW + wave;
                acc[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                if ((k + 1) * NW <= NT2 || n < NT2) {
                    int it, jt;
                    tile(n, it, jt);
#pragma unroll
                    for (int k1 = 0; k1 < P; k1 += 32)
                        if (MODE == FULL || k1 < w.Da)
#pragma unroll
                            for (int k0 = k1; k0 < k1 + 32; k0 += KS)
                                acc[k] = M::mma(frag_row(sb, Tl::LD, 16 * jt, k0), frag_ordered<T>(sa, Tl::LD, 16 * it, k0), acc[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < ROUNDS; ++k) {
                const int n = k * NW + wave;
                if ((k + 1) * NW <= NT2 || n < NT2) {
                    int it, jt;
                    tile(n, it, jt);
                    const float step = it - jt <= 1 ? 1.0f : it - jt == 2 ? g16 : g16 * g16;
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[k][r] *= jt < it ? below[r] * step : diag[r];
                    put_masked(sm + (16 * it + r16) * LDM + ordered<T>(16 * jt + 4 * gr), C * LDM, acc[k]);
                }
            }
        }
        __syncthreads();
        if (!mine) continue;
        // what the state gives each row; result tiles hold columns of c by rows
        f32x4 acc[IT][VT];
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
            for (int v = 0; v < VT; ++v) acc[it][v] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb < P / KS; ++kb) {
            if (MODE != FULL && kb * KS / 32 * 32 >= w.Da) break;
            Parts<T, state_parts<T>()> p[VT];
#pragma unroll
            for (int v = 0; v < VT; ++v)
#pragma unroll
                for (int j = 0; j < E; j += 2)
                    p[v].set(j, S.s[kb * St::TPK + j / 4][v][j % 4], S.s[kb * St::TPK + j / 4][v][j % 4 + 1]);
            typename M::Frag a[IT];
#pragma unroll
            for (int it = 0; it < IT; ++it) a[it] = frag_ordered<T>(sa, Tl::LD, 16 * it, kb * KS);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n = 0; n < state_parts<T>(); ++n)
#pragma unroll
                for (int it = 0; it < IT; ++it)
#pragma unroll
                    for (int v = 0; v < VT; ++v) acc[it][v] = M::mma(p[v].f[n], a[it], acc[it][v]);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
            for (int v = 0; v < VT; ++v)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[it][v][r] *= inter[it];
        // what the chunk's own rows give, and the state's update
        if (m < C) up.skip();
        St chunk;
        St& sum = update_apart<T>() ? chunk : S;
        if constexpr (update_apart<T>()) chunk.clear();
        else S.decay(up.d);
#pragma unroll
        for (int k0 = 0; k0 < C; k0 += KS) {
            typename M::Frag c[VT];
#pragma unroll
            for (int v = 0; v < VT; ++v) c[v] = frag_col(sc, Tl::LD, k0, (wave * VT + v) * 16);
#pragma unroll
            for (int n = 0; n < MP; ++n) {
                typename M::Frag a[IT];
#pragma unroll
                for (int it = k0 / 16; it < IT; ++it) a[it] = frag_ordered<T>(sm + n * C * LDM, LDM, 16 * it, k0);
#pragma unroll
                for (int it = k0 / 16; it < IT; ++it)
#pragma unroll
                    for (int v = 0; v < VT; ++v) acc[it][v] = M::mma(c[v], a[it], acc[it][v]);
            }
            __builtin_amdgcn_sched_barrier(0);
            float u[E];
            up.get(k0, u);
            typename St::Step x;
            x.prepare(sb, Tl::LD, k0, c, u);
            __builtin_amdgcn_sched_barrier(0);
            sum.template update<MODE>(x, w.Da);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (update_apart<T>()) S.add(up.d, chunk);
        const int col = wave * VT * 16 + 4 * gr;
        wait_loads();
        if (w.out32) store_rows<float, MODE, IT, VT>(w, (float*)w.out + out0, t0, m, L, col, acc);
        else store_rows<T, MODE, IT, VT>(w, (T*)w.out + out0, t0, m, L, col, acc);
    }
    if (w.state_out) {
        if (t_end > t_begin && (t_end - t_begin) % C)
            update_rest<T, P, C>(S, sb, sc, (t_end - t_begin) % C, g, g2, su, w.e);
        S.store(w.state_out + bh * D, w.Da, w.Dc, w.transposed, 1.0f / sigma);
    }
}

// Sums over the query heads of a group, in order: out[row, hk, :] = sum of x[row, hk, 0 .. group).
// blockIdx.y: 0 sums dk, 1 sums dv.  One piece of a row a thread.  Bound by memory: 25,600 rows of
// 8 heads to 2, 64 columns, 118 MB in 17 us (6.9 TB/s: the sums' terms are still in the memory-side cache).
struct GroupSum {
    const float* x[2];
    void* out[2];
    int D[2];
    long first, end;         // heads of a launch, of rows * Hk
    int group;
};
template <class T>
__global__ __launch_bounds__(256) void k_attn_group(const GroupSum a) {
    constexpr int V = 4;
    const int which = blockIdx.y, D = a.D[which], pieces = (D + V - 1) / V;
    const long i = (long)blockIdx.x * 256 + threadIdx.x;
    const long head = a.first + i / pieces;
    if (head >= a.end) return;
    const int c = (int)(i % pieces) * V;
    const float* p = a.x[which] + head * a.group * D + c;
    float s[V] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int q = 0; q < a.group; ++q) {
        float x[V];
        load_elements<float>(p + (long)q * D, 0, D - c, x);
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] += x[j];
    }
    T* out = (T*)a.out[which] + head * D + c;
    T y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = (T)s[j];
    if (D - c >= V) {
        __builtin_memcpy(out, y, sizeof(y));
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < D) out[j] = y[j];
    }
}

// ------------------------------------------------------------------ one token
// S = gamma S + k v^T, o = scale q S: a state is read and written once, so HBM bounds a batch (256
// streams, 16 heads of 128 x 128, 0.46 GB in 98 us, 4.7 TB/s) and the launch a single stream (8 heads
// of 64 x 64 4.9 us).  A workgroup a head, so that one stream still spreads over compute units and no sum
// leaves a workgroup.
// grid (Hq, B), block 256: LR lanes take 4 columns each of a state row, 256 / LR row groups.
template <class T>
__global__ __launch_bounds__(256) void k_attn_step(const semicrf_attention p, const int32_t* slots,
                                                   int pool, T* out, float* state_out, int LR) {
    __shared__ float sq[ATTN_MAX_D], sk[ATTN_MAX_D];
    __shared__ float part[256 * 4];
    const int h = blockIdx.x, b = blockIdx.y, Dk = p.Dk, Dv = p.Dv, hk = h / (p.Hq / p.Hk);
    const int tid = threadIdx.x;
    const int slot = slots ? slots[b] : b;
    T* o = out + ((size_t)b * p.Hq + h) * Dv;
    if (slot < 0 || slot >= pool) {
        for (int j = tid; j < Dv; j += 256) o[j] = (T)0.0f;
        return;
    }
    const T* q = (const T*)p.q + b * p.q_stride[0] + h * p.q_stride[2];
    const T* k = (const T*)p.k + b * p.k_stride[0] + hk * p.k_stride[2];
    const T* v = (const T*)p.v + b * p.v_stride[0] + hk * p.v_stride[2];
    if (tid < Dk) {
        sq[tid] = (float)q[tid] * p.scale;
        sk[tid] = (float)k[tid];
    }
    __syncthreads();
    const int lr = tid & (LR - 1), grp = tid / LR, ng = 256 / LR, c = lr * 4;
    Decay gamma;
    gamma.set(p.log_decay[h], 1);
    float vv[4], acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) vv[i] = c + i < Dv ? (float)v[c + i] : 0.0f;
    const size_t base = ((size_t)slot * p.Hq + h) * Dk * Dv;
    for (int r = grp; r < Dk; r += ng) {
        float s[4];
        load_elements<float>(p.state + base + (size_t)r * Dv, c, Dv, s);
        const float kr = sk[r], qr = sq[r];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[i] = (gamma.near1 ? s[i] : 0.0f) + fmaf(s[i], gamma.f, kr * vv[i]);
            acc[i] = fmaf(qr, s[i], acc[i]);
        }
        store_elements(state_out + base + (size_t)r * Dv, c, Dv, s);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) part[tid * 4 + i] = acc[i];
    __syncthreads();
    if (tid < Dv) {
        float s = 0.0f;
        for (int n = 0; n < ng; ++n) s += part[n * LR * 4 + tid];
        o[tid] = (T)s;
    }
}

// ------------------------------------------------------------------ host
int head_pad(const semicrf_attention& p) {
    const int d = p.Dk > p.Dv ? p.Dk : p.Dv;
    return d <= 32 ? 32 : d <= 64 ? 64 : 128;
}
int chunk_of(const semicrf_attention& p) { return p.dtype == SEMICRF_F32 ? 32 : 64; }

// Workgroups of the sweep that run at once on 256 compute units, by registers (sweep_occupancy)
// and, for bfloat16 of width 32, by LDS (38 KB of 160).
int sweep_slots(const semicrf_attention& p) {
    const int P = head_pad(p);
    const bool f32 = p.dtype == SEMICRF_F32;
    return 256 * (P == 128 ? 1 : P == 64 ? (f32 ? 4 : 3) : (f32 ? 8 : 4));
}

// Positions per segment.  Segments shorten the chain of chunks that one workgroup takes in order, at
// the price of the pass over the states, its launches and the join.  The times are modelled in
// units of one chunk of the sweep where a compute unit has one workgroup (2 us at width 64, 64
// bfloat16 or 32 fp32 positions); with w workgroups a unit it takes 0.4 + 0.6 w, the state's pass 0.4
// of that, launches and prologues 6 (9 with gradients), the join 0.06 a segment.  Measured at width
// 64, one segment against the choice: 1 x 3,000 positions, 2 heads, bfloat16 94 and 24 us; 8 x 800, 8
// heads 31 and 30 us, fp32 57 and 44; but bfloat16 gradients 32 and (4 segments) 44 us: one is kept.
// The constants are those of width 64 at widths 32 and 128 too.  The members of a unit are to run at
// once on one chiplet; more query heads on one than it holds (gradients: from 11 at width 128, from
// 33 at width 64 in bfloat16) get one segment: 100,000 positions, 16 heads on one of 128 columns, 11.3 ms,
// in four segments 3.6.
int segment(const semicrf_attention& p, bool grad) {
    const int C = chunk_of(p), sweeps = grad ? 3 : 1, states = grad ? 2 : 1, group = p.Hq / p.Hk;
    const long bh = (long)p.B * p.Hq, n = ((long)p.T + C - 1) / C;
    // workgroups go to the chiplets in turn: as many units (place()) as run at once on each of them
    const long most = CHIPLETS * (sweep_slots(p) / CHIPLETS / (group * sweeps)) / ((long)p.B * p.Hk);
    auto load = [](long workgroups) {
        const double w = (double)workgroups / 256;
        return w > 1.0 ? 0.4 + 0.6 * w : 1.0;
    };
    long best = 1;
    double cost = n * load(bh * sweeps);
    for (long k = 2; k <= most && k <= n; ++k) {
        const long len = (n + k - 1) / k;
        const double c = len * (load(bh * k * sweeps) + 0.4 * load(bh * k * states)) + (grad ? 9 : 6) + 0.06 * k;
        if (c < cost) {
            cost = c;
            best = k;
        }
    }
    return (int)((n + best - 1) / best * C);
}

struct AttnLayout {
    int seg, nseg;
    size_t S, R, gk, gv, total;
};

AttnLayout attn_layout(const semicrf_attention& p, bool grad) {
    AttnLayout l{};
    l.seg = segment(p, grad);
    l.nseg = (p.T + l.seg - 1) / l.seg;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off += (bytes + 255) / 256 * 256;
        return o;
    };
    const size_t st = l.nseg > 1 ? (size_t)p.B * p.Hq * l.nseg * p.Dk * p.Dv * 4 : 0;
    l.S = take(st);
    if (grad) {
        l.R = take(st);
        const size_t rows = p.Hq > p.Hk ? (size_t)p.B * p.T * p.Hq * 4 : 0;
        l.gk = take(rows * p.Dk);
        l.gv = take(rows * p.Dv);
    }
    l.total = off ? off : 256;
    return l;
}

template <class F>
hipError_t with_kernel(const semicrf_attention& p, F&& f) {
    const int P = head_pad(p);
    using I32 = std::integral_constant<int, 32>;
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    if (p.dtype == SEMICRF_F32) {
        if (P == 32) return f(0.0f, I32(), I32());
        if (P == 64) return f(0.0f, I64(), I32());
        return f(0.0f, I128(), I32());
    }
    if (P == 32) return f((bf16)0.0f, I32(), I64());
    if (P == 64) return f((bf16)0.0f, I64(), I64());
    return f((bf16)0.0f, I128(), I64());
}

Sweep base_sweep(const AttnArgs& a, const AttnLayout& l) {
    const semicrf_attention& p = a.p;
    Sweep w{};
    w.T = p.T; w.H = p.Hq;
    w.lengths = p.lengths;
    w.log_decay = p.log_decay;
    w.scale = p.scale;
    w.seg = l.seg; w.nseg = l.nseg;
    w.status = a.status;
    return w;
}

Role role(const void* p, const int64_t* s, int group) { return Role{p, (long)s[0], (long)s[1], (long)s[2], group}; }

// Whether a role's rows can be read through buffer descriptors, addresses being whole dwords, and
// whether the output's rows can be written so.
bool fast_role(const Role& r, int D, int es) {
    return (uintptr_t)r.p % 4 == 0 && r.sb * es % 4 == 0 && r.st * es % 4 == 0 && r.sh * es % 4 == 0 &&
           D * es % 16 == 0 && r.st >= D && r.st * es * 64 < (1l << 29);
}
bool fast_out(const Sweep& w, int es) {
    return (uintptr_t)w.out % 4 == 0 && w.Dc % 4 == 0 && (long)w.H * w.Dc * (w.out32 ? 4 : es) * 64 < (1l << 29);
}

// Launches over all sequences, as many at a time as a grid of less than 2^32 threads holds:
// f(set, workgroups).
template <int N, class F>
hipError_t by_sequences(const semicrf_attention& p, Sweeps<N> set, int threads, F&& f) {
    const long group = p.Hq / p.Hk, units = (long)p.Hk * set.s[0].nseg;      // of a sequence
    const long most = (1l << 32) / threads / (N * group) / CHIPLETS * CHIPLETS - CHIPLETS, step = most / units;
    for (long b = 0; b < p.B; b += step) {
        const long end = b + step < p.B ? b + step : p.B;
        for (Sweep& w : set.s) {
            w.B0 = (int)b;
            w.B1 = (int)end;
        }
        f(set, (unsigned)(((end - b) * units + CHIPLETS - 1) / CHIPLETS * CHIPLETS * N * group));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int N>
hipError_t run_state(const semicrf_attention& p, const Sweeps<N>& set, hipStream_t stream) {
    return with_kernel(p, [&](auto t, auto pp, auto cc) {
        using T = decltype(t);
        constexpr int P = decltype(pp)::value, C = decltype(cc)::value, es = sizeof(T);
        const int group = p.Hq / p.Hk, threads = 64 * sweep_waves(P);
        bool fast = true;
        for (const Sweep& w : set.s) fast = fast && fast_role(w.b, w.Da, es) && fast_role(w.c, w.Dc, es);
        return by_sequences(p, set, threads, [&](const Sweeps<N>& part, unsigned grid) {
            if (!fast)
                hipLaunchKernelGGL((k_attn_state<T, P, C, LOOSE, N>), grid, threads, 0, stream, part, group);
            else if (p.Dk == P && p.Dv == P)
                hipLaunchKernelGGL((k_attn_state<T, P, C, FULL, N>), grid, threads, 0, stream, part, group);
            else
                hipLaunchKernelGGL((k_attn_state<T, P, C, PART, N>), grid, threads, 0, stream, part, group);
        });
    });
}

template <int N>
hipError_t run_sweep(const semicrf_attention& p, const Sweeps<N>& set, hipStream_t stream) {
    return with_kernel(p, [&](auto t, auto pp, auto cc) {
        using T = decltype(t);
        constexpr int P = decltype(pp)::value, C = decltype(cc)::value, es = sizeof(T);
        const int group = p.Hq / p.Hk, threads = 64 * sweep_waves(P);
        bool fast = true;
        for (const Sweep& w : set.s)
            fast = fast && fast_role(w.a, w.Da, es) && fast_role(w.b, w.Da, es) && fast_role(w.c, w.Dc, es) &&
                   fast_out(w, es);
        return by_sequences(p, set, threads, [&](const Sweeps<N>& part, unsigned grid) {
            if (!fast)
                hipLaunchKernelGGL((k_attn_sweep<T, P, C, LOOSE, N>), grid, threads, 0, stream, part, group);
            else if (p.Dk == P && p.Dv == P)
                hipLaunchKernelGGL((k_attn_sweep<T, P, C, FULL, N>), grid, threads, 0, stream, part, group);
            else
                hipLaunchKernelGGL((k_attn_sweep<T, P, C, PART, N>), grid, threads, 0, stream, part, group);
        });
    });
}

hipError_t run_scan(const semicrf_attention& p, const AttnLayout& l, Scan s, int states, hipStream_t stream) {
    s.lengths = p.lengths; s.log_decay = p.log_decay;
    s.T = p.T; s.H = p.Hq; s.seg = l.seg; s.nseg = l.nseg; s.D = p.Dk * p.Dv;
    hipLaunchKernelGGL(k_attn_scan, dim3((s.D + 255) / 256, states * p.Hq, p.B), dim3(256), 0, stream, s);
    return hipGetLastError();
}

#define TRY(x)                              \
    do {                                    \
        const hipError_t e_ = (x);          \
        if (e_ != hipSuccess) return e_;    \
    } while (0)

}  // namespace

size_t decay_attention_bytes(const semicrf_attention& p, bool grad) { return attn_layout(p, grad).total; }

hipError_t launch_decay_attention(const AttnArgs& a, void* ws, hipStream_t stream) {
    const semicrf_attention& p = a.p;
    const AttnLayout l = attn_layout(p, false);
    const int group = p.Hq / p.Hk;
    Sweep w = base_sweep(a, l);
    w.a = role(p.q, p.q_stride, 1);
    w.b = role(p.k, p.k_stride, group);
    w.c = role(p.v, p.v_stride, group);
    w.Da = p.Dk; w.Dc = p.Dv;
    w.si = p.scale; w.su = 1.0f;
    w.out = a.out;
    w.state = p.state;
    w.state_nseg = 1;
    if (l.nseg > 1) {
        w.local = (float*)((char*)ws + l.S);
        TRY(run_state(p, Sweeps<1>{{w}}, stream));
        TRY(run_scan(p, l, Scan{{w.local}, {p.state}, {a.state_out}}, 1, stream));
        w.state = w.local;
        w.state_nseg = l.nseg;
    } else {
        w.state_out = a.state_out;
    }
    return run_sweep(p, Sweeps<1>{{w}}, stream);
}

hipError_t launch_decay_attention_grad(const AttnArgs& a, void* ws, hipStream_t stream) {
    const semicrf_attention& p = a.p;
    const AttnLayout l = attn_layout(p, true);
    const int group = p.Hq / p.Hk;
    const int64_t gs[3] = {(int64_t)p.T * p.Hq * p.Dv, (int64_t)p.Hq * p.Dv, p.Dv};
    const Role q = role(p.q, p.q_stride, 1), k = role(p.k, p.k_stride, group),
               v = role(p.v, p.v_stride, group), g = role(a.grad_out, gs, 1);
    float* S = (float*)((char*)ws + l.S);
    float* R = (float*)((char*)ws + l.R);
    Sweep w = base_sweep(a, l);
    w.state_nseg = l.nseg;
    Sweep f = w, r = w;
    f.si = p.scale; f.su = 1.0f;
    r.si = 1.0f; r.su = p.scale; r.e = 1; r.reverse = 1;
    f.state = p.state;
    r.state = a.grad_state_out;
    if (l.nseg > 1) {
        f.b = k; f.c = v; f.Da = p.Dk; f.Dc = p.Dv; f.local = S;
        r.b = q; r.c = g; r.Da = p.Dk; r.Dc = p.Dv; r.local = R;
        TRY(run_state(p, Sweeps<2>{{f, r}}, stream));
        TRY(run_scan(p, l, Scan{{S, R}, {p.state, a.grad_state_out}, {nullptr, a.grad_state}}, 2, stream));
        f.state = S;
        r.state = R;
    }
    // dq
    f.a = g; f.b = v; f.c = k; f.Da = p.Dv; f.Dc = p.Dk; f.transposed = 1;
    f.out = a.grad_q;
    // dv, and the gradient of the initial state
    r.a = k; r.b = q; r.c = g; r.Da = p.Dk; r.Dc = p.Dv; r.transposed = 0;
    r.out32 = group > 1;
    r.out = group > 1 ? (void*)((char*)ws + l.gv) : a.grad_v;
    r.state_out = l.nseg > 1 ? nullptr : a.grad_state;
    const Sweep dv = r;
    // dk
    r.a = v; r.b = g; r.c = q; r.Da = p.Dv; r.Dc = p.Dk; r.transposed = 1;
    r.out = group > 1 ? (void*)((char*)ws + l.gk) : a.grad_k;
    r.state_out = nullptr;
    TRY(run_sweep(p, Sweeps<3>{{dv, r, f}}, stream));
    if (group > 1) {
        GroupSum s{{(const float*)((char*)ws + l.gk), (const float*)((char*)ws + l.gv)},
                   {a.grad_k, a.grad_v}, {p.Dk, p.Dv}, 0, 0, group};
        const long heads = (long)p.B * p.T * p.Hk, pieces = ((p.Dk > p.Dv ? p.Dk : p.Dv) + 3) / 4;
        const long most = (1l << 31) / pieces;           // a launch holds less than 2^32 threads
        for (; s.first < heads; s.first = s.end) {
            s.end = s.first + most < heads ? s.first + most : heads;
            const dim3 grid((unsigned)(((s.end - s.first) * pieces + 255) / 256), 2);
            if (p.dtype == SEMICRF_F32) hipLaunchKernelGGL((k_attn_group<float>), grid, dim3(256), 0, stream, s);
            else hipLaunchKernelGGL((k_attn_group<bf16>), grid, dim3(256), 0, stream, s);
            TRY(hipGetLastError());
        }
    }
    return hipSuccess;
}

hipError_t launch_decay_attention_step(const semicrf_attention& p, const int32_t* slots, int pool,
                                       void* out, float* state_out, hipStream_t stream) {
    int LR = 1;
    while (LR * 4 < p.Dv) LR *= 2;
    if (p.dtype == SEMICRF_F32)
        hipLaunchKernelGGL((k_attn_step<float>), dim3(p.Hq, p.B), dim3(256), 0, stream, p, slots, pool,
                           (float*)out, state_out, LR);
    else
        hipLaunchKernelGGL((k_attn_step<bf16>), dim3(p.Hq, p.B), dim3(256), 0, stream, p, slots, pool,
                           (bf16*)out, state_out, LR);
    return hipGetLastError();
}

}  // namespace semicrf
