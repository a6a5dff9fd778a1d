// Gated linear recurrence, forward, backward and one token at a time, on gfx950.
//
//   s = log_decay sig(r),  a = exp(s),  b = sqrt(1 - a^2),  u = sig(i) x,  h_t = a_t h_{t-1} + b_t u_t
//   backward, with E_t = g_t + a_{t+1} E_{t+1} the gradient of h_t:
//     ds = E (a h_{t-1} - a^2 / b u),  dr = ds s (1 - sig r),  dlog_decay = sum ds sig(r)
//     du = E b,  dx = du sig(i),  di = du u (1 - sig i),  dh_0 = a_1 E_1
//
// A decay next to 1 is kept as its distance from 1: m = a - 1 = expm1(s) has a relative rounding
// error, where a = 1 + m would lose what is below 2^-24 and with it time constants of many
// positions.  h_t = h_{t-1} + m h_{t-1} + b u, and 1 - a^2 = -m (m + 2).  A strong decay is kept as a itself,
// h_t = a h_{t-1} + b u: by its distance from 1 the state before would leave an error of 2^-24 of its own
// size, however little of it is left.
#include "common.h"
#include "encoder.h"
#include "gates.h"

namespace semicrf {

namespace {

constexpr int SPAN = SEMICRF_RECURRENCE_SPAN;

// A decay factor exp(s), s <= 0, as c: a - 1 where the decay is weak (s >= -1/4), else a.  m = a - 1 and e = a in
// any case.  Below -1/4 the difference costs at most two bits; above, five terms of the series leave
// s^6 / 5040 < 2^-24.  WEAK: s is known to be -1/4 or more.
template <bool WEAK = false>
__device__ __forceinline__ float decay(float s, bool& weak, float& m, float& e) {
    float p = fmaf(s, 1.0f / 720.0f, 1.0f / 120.0f);
    p = fmaf(s, p, 1.0f / 24.0f);
    p = fmaf(s, p, 1.0f / 6.0f);
    p = fmaf(s, p, 0.5f);
    p = fmaf(s * s, p, s);
    const float full = WEAK ? 0.0f : fast_exp2(s * LOG2EF);
    weak = WEAK || s >= -0.25f;
    e = weak ? 1.0f + p : full;
    m = weak ? p : full - 1.0f;
    return weak ? p : full;
}
// a v + add, a v
__device__ __forceinline__ float decayed(bool weak, float c, float v, float add) {
    return (weak ? v : 0.0f) + fmaf(c, v, add);
}
__device__ __forceinline__ float decayed(bool weak, float c, float v) { return fmaf(c, v, weak ? v : 0.0f); }

__device__ __forceinline__ float root(float x) { return __builtin_amdgcn_sqrtf(x); }

template <bool V>
struct Flag {
    static constexpr bool value = V;
};

template <class T>
__device__ __forceinline__ const T* row(const void* p, const int64_t (&stride)[2], int b, int t) {
    return (const T*)p + b * stride[0] + t * stride[1];
}

// ------------------------------------------------------------------ elements of a lane
// A wavefront takes a span of 16 positions of 32 CH channels: lane 32 q + l holds CH neighbouring
// channels at positions 8 q .. 8 q + 7.  Where N is no multiple of CH the last lanes start early, at
// N - CH, and compute channels that a neighbour has too (of the same wavefront: a width that leaves one
// channel to the last takes CH = 1).
constexpr int POS = 8, LANES = 32;

// As loaded, two bfloat16 to a register
template <class T, int CH>
struct Raw {
    unsigned w[(CH * sizeof(T) + 3) / 4];
    __device__ __forceinline__ float operator[](int c) const {
        if (sizeof(T) == 4) return __uint_as_float(w[c]);
        return __uint_as_float(c % 2 ? w[c / 2] & 0xffff0000u : w[c / 2] << 16);
    }
    __device__ __forceinline__ void fill(unsigned bits) {
#pragma unroll
        for (unsigned& v : w) v = bits;
    }
};
template <class T, int CH>
__device__ __forceinline__ Raw<T, CH> load(const T* base, unsigned at) {
    Raw<T, CH> r{};
    __builtin_memcpy(r.w, (const char*)base + at * (unsigned)sizeof(T), CH * sizeof(T));
    return r;
}
// True where no channel of the wavefront decays by more than 1/4 a position
template <int CH>
__device__ __forceinline__ bool all_weak(const Raw<float, CH>& lam) {
    bool strong = false;
#pragma unroll
    for (int c = 0; c < CH; ++c) strong |= lam[c] < -0.25f;
    return !__any(strong);
}
// Positions past the length: a gate that is closed for good keeps the state, whatever else is there
template <class T, int CH>
__device__ __forceinline__ void close(Raw<T, CH> (&x)[POS], Raw<T, CH> (&r)[POS], Raw<T, CH> (&g)[POS], int first,
                                      int count) {
#pragma unroll
    for (int i = 0; i < POS; ++i)
        if (first + i >= count) {
            r[i].fill(sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u);      // -infinity
            x[i].fill(0);
            g[i].fill(0);
        }
}
template <class T, int CH>
__device__ __forceinline__ void store(T* base, unsigned at, const float (&x)[CH]) {
    T r[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) r[c] = (T)x[c];
    __builtin_memcpy((char*)base + at * (unsigned)sizeof(T), r, sizeof(r));
}

// ------------------------------------------------------------------ joins
// The state goes through a stretch of positions as A h + H, A the product of the a and H what the stretch
// makes of 0.  M stands for A as c does for a; a weak one has its sign bit set, also where A = 1.
struct Map {
    float M, H;
};
constexpr Map SAME{-0.0f, 0.0f};
__device__ __forceinline__ bool is_weak(float c) { return (int)__float_as_uint(c) < 0; }
__device__ __forceinline__ float mark(bool weak, float c) { return weak ? __builtin_copysignf(c, -1.0f) : c; }
// The product of decays whose logarithms add up to s
__device__ __forceinline__ float product_of(float s) {
    bool weak;
    float m, e;
    const float c = decay(s, weak, m, e);
    return mark(weak, c);
}
__device__ __forceinline__ float apply(Map a, float h) { return decayed(is_weak(a.M), a.M, h, a.H); }
__device__ __forceinline__ Map then(Map a, Map b) {          // a first
    const bool wa = is_weak(a.M), wb = is_weak(b.M);
    const float p = decayed(wb, b.M, a.M, wa ? b.M : 0.0f);
    // many weak ones make a strong one
    return {wa && wb ? (p < -0.25f ? 1.0f + p : mark(true, p)) : p, apply(b, a.H)};
}

// The lower half's value, or the upper's
template <int UPPER>
__device__ __forceinline__ float of_half(float v) {
    const int i = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, (int)__builtin_amdgcn_permlane32_swap(i, i, false, false)[UPPER]);
}

// Maps of the two halves, in order of position (REVERSED: from the last): what comes before the lane's
// half, and both.
template <bool REVERSED>
__device__ __forceinline__ void join_halves(Map own, Map& before, Map& all) {
    const bool later = ((threadIdx.x & 63) / LANES) != REVERSED;
    const Map first{of_half<REVERSED>(own.M), of_half<REVERSED>(own.H)};
    all = then(first, Map{of_half<!REVERSED>(own.M), of_half<!REVERSED>(own.H)});
    before = Map{later ? first.M : SAME.M, later ? first.H : SAME.H};
}

// ------------------------------------------------------------------ tiles in order
// A tile is W spans, a span a wavefront; a chain is the tiles of 32 CH channels of a sequence.  Every tile
// finds its map by itself and then needs the state it starts from.  A workgroup serves one chain and takes
// its tiles in order by a ticket, so that whoever waits waits for tiles that are at work already or done.
// (One ticket for all chains costs 24 ns a tile, on one after another: more than the tile's bytes.)
// Tile k publishes its map, and the last of each GROUP tiles the state it ends with; tile k reads the
// state of the group before and the maps since, and joins them in order: the same additions on every
// call.  A publication is one 8-byte store, with a pattern that no map has as "not there yet".
// Where there are chains enough a workgroup of the backward pass has its chain to itself and publishes nothing.
constexpr int GROUP = 16;
constexpr unsigned long long EMPTY = ~0ull;

struct Chain {
    unsigned long long* words;   // [sequence x columns][tiles][channels of a tile]: maps
    unsigned long long* states;  // [sequence x columns][groups][channels of a tile]: (0, state)
    unsigned* tickets;           // [sequence x columns][TICKET], or NULL where a workgroup has the whole chain
    int tiles, groups, cols;
    unsigned chains;
};
constexpr int TICKET = 32;       // a line each

__device__ __forceinline__ unsigned long long pack(Map m) {
    if (m.M != m.M) m.M = __builtin_nanf("");            // never the pattern of EMPTY
    return ((unsigned long long)__float_as_uint(m.H) << 32) | __float_as_uint(m.M);
}
__device__ __forceinline__ Map unpack_map(unsigned long long v) {
    return {__uint_as_float((unsigned)v), __uint_as_float((unsigned)(v >> 32))};
}
__device__ __forceinline__ void publish(unsigned long long* p, unsigned long long v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long peek(const unsigned long long* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The next n <= U words of each lane, once all of them are there.  The wait ends: what is waited for
// is held by a workgroup that waits for earlier tiles only.  Should another call write to the same
// workspace meanwhile, it ends all the same, after a second or so, and the outputs are NaN.
constexpr int PATIENCE = 1 << 20;
template <int U>
__device__ __forceinline__ void await(const unsigned long long* p, size_t stride, int n,
                                      unsigned long long (&v)[U]) {
#pragma unroll 1
    for (int i = 0; i < PATIENCE; ++i) {
        bool missing = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = u < n ? peek(p + u * stride) : 0;
            missing |= v[u] == EMPTY;
        }
        if (!__any(missing)) return;
        __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (v[u] == EMPTY) v[u] = pack(Map{__builtin_nanf(""), __builtin_nanf("")});
}

// What a workgroup shares while it joins its spans and finds the state it starts from
template <int CW, int W>
struct Shared {
    Map part[W][CW];             // maps of the spans, in the order in which the state goes through them
    float logs[W][CW];           // and the logarithms of their decays
    Map look[W][CW];             // maps of a wavefront's share of the tiles since the last group
    float base[2][CW];           // the state at the end of the last group, or of the last tile, by turns
    float start[W][CW];          // the state each span starts from
    unsigned slot;
};

// The state before each span of tile k of chain `seq`, into sh.start: `order` is the wavefront's place in
// part, `first` the state before tile 0 at a channel.  A lane takes whole channels here.  Waits for all
// wavefronts' writes of part.  CARRY: the workgroup may have the chain to itself.
template <bool CARRY, int CW, int W, class F>
__device__ __forceinline__ void find_starts(const Chain& ch, Shared<CW, W>& sh, long seq, int k, bool last, int order,
                                            F&& first) {
    constexpr int U = (GROUP + W - 1) / W, PER = (CW + 63) / 64;
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));                      // addresses are made anew
    const int g = k / GROUP, j = k - g * GROUP;
    float h[PER];
    // The first state is read before the barrier, and so before anything is published: the chain's last
    // wavefront may overwrite it after that.
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        h[i] = (!CARRY || ch.tickets ? g == 0 : k == 0) && lane + i * 64 < CW ? first(lane + i * 64) : 0.0f;
        asm volatile("" : "+v"(h[i]));
    }
    __syncthreads();
    if (W > 1 && ch.tickets) {
        unsigned long long* words = ch.words + (size_t)seq * ch.tiles * CW;
        unsigned long long* states = ch.states + (size_t)seq * ch.groups * CW;
        Map own[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = lane + i * 64;
            own[i] = SAME;
            if (CW % 64 && c >= CW) continue;
            if (order == 0 && !last) {
                float log = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    log += sh.logs[w][c];
                    own[i].H = apply(sh.part[w][c], own[i].H);
                }
                own[i].M = product_of(log);
                if (j < GROUP - 1) publish(words + (size_t)k * CW + c, pack(own[i]));
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = lane + i * 64;
            if (CW % 64 && c >= CW) continue;
            unsigned long long v[U];
            const int n = min(U, j - order * U);
            Map m = SAME;
            if (n > 0) await(words + (size_t)(g * GROUP + order * U) * CW + c, CW, n, v);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u < n) m = then(m, unpack_map(v[u]));
            sh.look[order][c] = m;
            if (order == W - 1 && g > 0) {
                unsigned long long s[1];
                await(states + (size_t)(g - 1) * CW + c, 0, 1, s);
                sh.base[0][c] = unpack_map(s[0]).H;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = lane + i * 64;
            if (CW % 64 && c >= CW) continue;
            if (g > 0) h[i] = sh.base[0][c];
#pragma unroll
            for (int w = 0; w < W; ++w) h[i] = apply(sh.look[w][c], h[i]);
            if (order == 0 && !last && j == GROUP - 1)
                publish(states + (size_t)g * CW + c, pack(Map{0.0f, apply(own[i], h[i])}));
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = lane + i * 64;
        if (CW % 64 && c >= CW) continue;
        if (CARRY && W > 1 && !ch.tickets && k > 0) h[i] = sh.base[k & 1][c];
#pragma unroll
        for (int w = 0; w < W - 1; ++w)
            if (w < order) h[i] = apply(sh.part[w][c], h[i]);
        sh.start[order][c] = h[i];
        if (CARRY && W > 1 && !ch.tickets && order == W - 1) sh.base[(k + 1) & 1][c] = apply(sh.part[W - 1][c], h[i]);
    }
    // read by the same wavefront only
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__global__ __launch_bounds__(256) void k_recurrence_clear(unsigned long long* p, size_t n, unsigned* tickets,
                                                          size_t m) {
    const size_t at = blockIdx.x * 256ul + threadIdx.x, step = gridDim.x * 256ul;
    for (size_t i = at; i < n; i += step) p[i] = EMPTY;
    for (size_t i = at; i < m; i += step) tickets[i] = 0;
}

// The chain that a workgroup serves: sequence b, channels from column col on
struct Place {
    unsigned seq;
    int b, col, L, last;
};
template <int W>
__device__ __forceinline__ Place place(const semicrf_recurrence& p, const Chain& ch, int32_t* status) {
    Place o;
    o.seq = blockIdx.x % ch.chains;
    o.b = (int)(o.seq / ch.cols);
    o.col = (int)(o.seq - o.b * ch.cols);
    o.L = __builtin_amdgcn_readfirstlane(seq_length(p.lengths, o.b, p.T, status));
    o.last = o.L > 0 ? (o.L - 1) / (W * SPAN) : 0;
    return o;
}

// The workgroup's first tile; the next ones' tickets are drawn while a tile is worked on
__device__ __forceinline__ unsigned draw(const Chain& ch, unsigned seq, unsigned none) {
    return ch.tickets && threadIdx.x == 0 ? atomicAdd(ch.tickets + (size_t)seq * TICKET, 1u) : none;
}
__device__ __forceinline__ int first_tile(const Chain& ch, unsigned seq, unsigned& slot) {
    if (!ch.tickets) return 0;
    const unsigned k = draw(ch, seq, 0);
    if (threadIdx.x == 0) slot = k;
    __syncthreads();
    const int got = __builtin_amdgcn_readfirstlane((int)slot);
    __syncthreads();
    return got;
}

// Forward.  Reads x and the gates once: the positions' decays and b u stay in registers while the state before
// them is found.
//
// Bound by neither alone: an element is about 35 instructions of a cycle a lane row and five of four (two
// sigmoids and the root), which is 300 us for 4 x 100,000 x 512 in bfloat16, and its 1.7 GB are 327 us; it takes
// 475 (3.6 TB/s).  A workgroup's loads wait for its arithmetic and the other way round, and three on a compute
// unit make up for a part of it only.  1 x 250,001 x 256 in float32 takes 245 to 300 on different cards (4.2 to
// 3.4 TB/s).  Strong decays in all channels cost 5 % on long sequences, 503 us for the first (32 x 800 x 1,024: 65
// against 59).
//   Two rows of 32 lanes with two channels each, not four of 16 with four: half the maps to make and
// one join in place of two.  Where no decay of the wavefront's channels is strong the exponential of
// decay is not taken: both together 525 -> 497 us.  Three workgroups a compute unit (80 registers):
// 497 -> 470.  Loading the next tile while the state is found needs 128 registers and gained nothing
// (537), nor did tiles of 12 or 16 wavefronts (467 and 502; 32 x 800 x 1,024: 57 and 69 in place of 55).
template <class T, int CH, int W>
__global__ __launch_bounds__(64 * W, W == 1 ? 2 : 6) void k_recurrence(const RecArgs a, const Chain ch) {
    constexpr int CW = CH * LANES;
    __shared__ Shared<CW, W> sh;
    const semicrf_recurrence& p = a.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int q = lane / LANES;
    const int l = lane % LANES;
    const int spans = (p.T + SPAN - 1) / SPAN;
    const Place o = place<W>(p, ch, a.status);
    unsigned n = min((o.col * LANES + l) * CH, p.N - CH);
    const bool mine = (o.col * LANES + l) * CH < p.N;
    const Raw<float, CH> lam = load<float, CH>(p.log_decay, n);
    Raw<T, CH> x[POS], r[POS], g[POS];
    auto fetch = [&](int tile) __attribute__((always_inline)) {      // rows past the length: the last one again
        const int end = max(o.L, 1) - 1, t0 = min((tile * W + wave) * SPAN, end);
        const T* px = row<T>(p.x, p.x_stride, o.b, t0);
        const T* pr = row<T>(p.decay_gate, p.decay_stride, o.b, t0);
        const T* pg = row<T>(p.input_gate, p.input_stride, o.b, t0);
#pragma unroll
        for (int i = 0; i < POS; ++i) {
            const unsigned at = min(q * POS + i, end - t0);
            x[i] = load<T, CH>(px, at * (unsigned)p.x_stride[1] + n);
            r[i] = load<T, CH>(pr, at * (unsigned)p.decay_stride[1] + n);
            g[i] = load<T, CH>(pg, at * (unsigned)p.input_stride[1] + n);
        }
    };
    auto tiles = [&](auto w) __attribute__((always_inline)) {
        int k = first_tile(ch, o.seq, sh.slot);
        while (k < ch.tiles) {
            asm volatile("" : "+v"(n), "+v"(q));        // addresses are made anew: no registers to spare for them
            const unsigned ticket = draw(ch, o.seq, k + 1);
            const int t0 = (k * W + wave) * SPAN, count = max(0, min(SPAN, o.L - t0));
            T* out = (T*)a.out + ((size_t)o.b * p.T + t0) * p.N;
            if (k > o.last) {                           // all padding
                const float zero[CH] = {};
                if (mine)
                    for (int i = q; i < SPAN && t0 + i < p.T; i += 2) store<T, CH>(out, i * p.N + n, zero);
                __syncthreads();                        // all have read the ticket
                if (threadIdx.x == 0) sh.slot = ticket;
                __syncthreads();
                k = __builtin_amdgcn_readfirstlane((int)sh.slot);
                continue;
            }
            fetch(k);
            __builtin_amdgcn_sched_barrier(0);          // the loads first, then a few elements at a time
            float a1[POS][CH], bu[POS][CH], sum[CH], H[CH];
            bool weak[POS][CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) sum[c] = H[c] = 0.0f;
            if (count < SPAN) close(x, r, g, q * POS, count);
#pragma unroll
            for (int i = 0; i < POS; ++i) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const float s = lam[c] * sigmoid(r[i][c]);
                    float m, e;
                    a1[i][c] = decay<w.value>(s, weak[i][c], m, e);
                    bu[i][c] = root(-m * (m + 2.0f)) * (sigmoid(g[i][c]) * x[i][c]);
                    sum[c] += s;
                    H[c] = decayed(weak[i][c], a1[i][c], H[c], bu[i][c]);
                }
                __builtin_amdgcn_sched_barrier(0);      // a few elements at a time
            }
            Map before[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                Map all;
                join_halves<false>(Map{product_of(sum[c]), H[c]}, before[c], all);
                sum[c] = of_half<0>(sum[c]) + of_half<1>(sum[c]);
                if (q == 0) {
                    sh.part[wave][l * CH + c] = all;
                    sh.logs[wave][l * CH + c] = sum[c];
                }
            }
            find_starts<false>(ch, sh, o.seq, k, k == o.last, wave, [&](int c) __attribute__((always_inline)) {
                const int at = min((o.col * LANES + c / CH) * CH, p.N - CH) + c % CH;
                return p.state ? p.state[(size_t)o.b * p.N + at] : 0.0f;
            });
            if (mine) {
                float h[CH];
#pragma unroll
                for (int c = 0; c < CH; ++c) h[c] = sh.start[wave][l * CH + c];
                if (a.starts && count > 0 && q == 0)
                    store<float, CH>(a.starts + ((size_t)o.b * spans + t0 / SPAN) * p.N, n, h);
#pragma unroll
                for (int c = 0; c < CH; ++c) h[c] = apply(before[c], h[c]);
#pragma unroll
                for (int i = 0; i < POS; ++i) {
                    float y[CH];
                    const int at = q * POS + i;
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        h[c] = decayed(weak[i][c], a1[i][c], h[c], bu[i][c]);
                        y[c] = at < count ? h[c] : 0.0f;
                    }
                    if (t0 + at < p.T) store<T, CH>(out, at * p.N + n, y);
                }
                if (a.state_out && k == o.last && wave == W - 1 && q == 1)
                    store<float, CH>(a.state_out + (size_t)o.b * p.N, n, h);
            }
            if (threadIdx.x == 0) sh.slot = ticket;
            __syncthreads();                            // before the next tile's part
            k = __builtin_amdgcn_readfirstlane((int)sh.slot);
        }
    };
    if (all_weak<CH>(lam)) tiles(Flag<true>{});
    else tiles(Flag<false>{});
}

// Backward, from the last tile to the first.  What later positions pass on to earlier ones, f_t = a_t (g_t +
// f_{t+1}), goes through a tile as h does in the forward pass.  Before a position's f is known its
// factors of it are: with e = g + f the gradient of h,
//   dx = e kx,  di = e ki,  dr = e kr,  dlog_decay += e kl
// kx = b sig(i), ki = kx x (1 - sig i), kl = a (h' - a u / b) sig(r), kr = kl log_decay (1 - sig r); h' runs
// forward from the span's stored start.  dpart [tile x sequence][N]: the tile's share of dlog_decay.
//
// Five factors an element stay in registers (168), so that inputs are read and exponentials taken once.
// About 80 instructions an element, of them six of four cycles: 510 us for 4 x 100,000 x 512 in bfloat16, where
// the bytes take 565; with one workgroup of 12 wavefronts a compute unit, whose loads and arithmetic take turns,
// 858 (3.4 TB/s), and 925 with strong decays in all channels.  (Before those were held as factors 840, against 890
// with 8 wavefronts and 1,110 with two workgroups of 6.)
template <class T, int CH, int W>
__global__ __launch_bounds__(64 * W, W == 1 ? 2 : 3) void k_recurrence_grad(const RecArgs a, const Chain ch,
                                                                                  float* dpart) {
    constexpr int CW = CH * LANES;
    __shared__ Shared<CW, W> sh;
    __shared__ float dl[W][CW];
    const semicrf_recurrence& p = a.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int q = lane / LANES;
    const int l = lane % LANES;
    const int spans = (p.T + SPAN - 1) / SPAN;
    const Place o = place<W>(p, ch, a.status);
    unsigned n = min((o.col * LANES + l) * CH, p.N - CH);
    const bool mine = (o.col * LANES + l) * CH < p.N;
    const Raw<float, CH> lam = load<float, CH>(p.log_decay, n);
    Raw<T, CH> x[POS], r[POS], g[POS], d[POS];
    Raw<float, CH> first;
    auto fetch = [&](int tile) __attribute__((always_inline)) {      // rows past the length: the last one again
        const int end = max(o.L, 1) - 1, t0 = min((tile * W + wave) * SPAN, end);
        const T* px = row<T>(p.x, p.x_stride, o.b, t0);
        const T* pr = row<T>(p.decay_gate, p.decay_stride, o.b, t0);
        const T* pg = row<T>(p.input_gate, p.input_stride, o.b, t0);
        const T* po = (const T*)a.grad_out + ((size_t)o.b * p.T + t0) * p.N;
#pragma unroll
        for (int i = 0; i < POS; ++i) {
            const unsigned at = min(q * POS + i, end - t0);
            x[i] = load<T, CH>(px, at * (unsigned)p.x_stride[1] + n);
            r[i] = load<T, CH>(pr, at * (unsigned)p.decay_stride[1] + n);
            g[i] = load<T, CH>(pg, at * (unsigned)p.input_stride[1] + n);
            d[i] = load<T, CH>(po, at * (unsigned)p.N + n);
        }
        first = load<float, CH>(a.starts_in + ((size_t)o.b * spans + t0 / SPAN) * p.N, n);
    };
    auto tiles = [&](auto w) __attribute__((always_inline)) {
        int k = first_tile(ch, o.seq, sh.slot);
        while (k < ch.tiles) {
            asm volatile("" : "+v"(n), "+v"(q));        // addresses are made anew: no registers to spare for them
            const unsigned ticket = draw(ch, o.seq, k + 1);
            const int tile = k <= o.last ? o.last - k : k;  // tiles of padding come last
            const int t0 = (tile * W + wave) * SPAN, count = max(0, min(SPAN, o.L - t0));
            const size_t at0 = ((size_t)o.b * p.T + t0) * p.N;
            T *gx = (T*)a.grad_x + at0, *gr = (T*)a.grad_decay + at0, *gi = (T*)a.grad_input + at0;
            float* dout = dpart + ((size_t)tile * p.B + o.b) * p.N;
            if (k > o.last) {
                const float zero[CH] = {};
                if (mine) {
                    for (int i = q; i < SPAN && t0 + i < p.T; i += 2) {
                        store<T, CH>(gx, i * p.N + n, zero);
                        store<T, CH>(gr, i * p.N + n, zero);
                        store<T, CH>(gi, i * p.N + n, zero);
                    }
                    if (wave == 0 && q == 0) store<float, CH>(dout, n, zero);
                }
                __syncthreads();                        // all have read the ticket
                if (threadIdx.x == 0) sh.slot = ticket;
                __syncthreads();
                k = __builtin_amdgcn_readfirstlane((int)sh.slot);
                continue;
            }
            fetch(tile);
            __builtin_amdgcn_sched_barrier(0);
            float a1[POS][CH], kx[POS][CH], ki[POS][CH], kr[POS][CH], kl[POS][CH], M[CH], F[CH];
            if (count < SPAN) {
                close(x, r, g, q * POS, count);
#pragma unroll
                for (int i = 0; i < POS; ++i)
                    if (q * POS + i >= count) d[i].fill(0);
                if (count == 0) first = Raw<float, CH>{};   // a span without a stored start
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float sum = 0.0f, H = 0.0f, bu[POS], av[POS], aub[POS], sr[POS], qr[POS];
#pragma unroll
                for (int i = 0; i < POS; ++i) {
                    float si, qi;
                    sigmoids(r[i][c], sr[i], qr[i]);
                    sigmoids(g[i][c], si, qi);
                    const float s = lam[c] * sr[i];
                    float m;
                    bool weak;
                    a1[i][c] = decay<w.value>(s, weak, m, av[i]);
                    if (!w.value) a1[i][c] = mark(weak, a1[i][c]);      // masks would take 32 scalar registers
                    const float bb = -m * (m + 2.0f), bv = root(bb);
                    const float ib = bb > 0x1p-123f ? __builtin_amdgcn_rsqf(bb) : 0.0f;
                    const float xv = x[i][c], u = si * xv;
                    bu[i] = bv * u;
                    sum += s;
                    H = decayed(w.value || is_weak(a1[i][c]), a1[i][c], H, bu[i]);
                    aub[i] = av[i] * ib * u;
                    kx[i][c] = bv * si;
                    ki[i][c] = kx[i][c] * xv * qi;
                }
                M[c] = product_of(sum);
                sum = of_half<0>(sum) + of_half<1>(sum);
                if (q == 0) sh.logs[W - 1 - wave][l * CH + c] = sum;
                Map before, all;
                join_halves<false>(Map{M[c], H}, before, all);
                float h = apply(before, first[c]);
#pragma unroll
                for (int i = 0; i < POS; ++i) {
                    kl[i][c] = av[i] * (h - aub[i]) * sr[i];
                    kr[i][c] = kl[i][c] * lam[c] * qr[i];
                    h = decayed(w.value || is_weak(a1[i][c]), a1[i][c], h, bu[i]);
                }
                float f = 0.0f;
#pragma unroll
                for (int i = POS - 1; i >= 0; --i) {
                    const float e = f + d[i][c];
                    f = decayed(w.value || is_weak(a1[i][c]), a1[i][c], e);
                    // held until f is known: not moved to where they are used, with what they are made of
                    asm volatile("" : "+v"(a1[i][c]), "+v"(kx[i][c]), "+v"(ki[i][c]), "+v"(kl[i][c]), "+v"(kr[i][c]));
                }
                F[c] = f;
                __builtin_amdgcn_sched_barrier(0);
            }
            Map before[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                Map all;
                join_halves<true>(Map{M[c], F[c]}, before[c], all);
                if (q == 0) sh.part[W - 1 - wave][l * CH + c] = all;
            }
            find_starts<true>(ch, sh, o.seq, k, k == o.last, W - 1 - wave, [&](int c) __attribute__((always_inline)) {
                const int at = min((o.col * LANES + c / CH) * CH, p.N - CH) + c % CH;
                return a.grad_state_out ? a.grad_state_out[(size_t)o.b * p.N + at] : 0.0f;
            });
            float f[CH], dlam[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                f[c] = apply(before[c], sh.start[W - 1 - wave][l * CH + c]);
                dlam[c] = 0.0f;
            }
#pragma unroll
            for (int i = POS - 1; i >= 0; --i) {
                float dx[CH], dr[CH], di[CH];
                const int at = q * POS + i;
                const bool in = at < count;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const float e = f[c] + d[i][c];
                    dx[c] = in ? e * kx[i][c] : 0.0f;
                    di[c] = in ? e * ki[i][c] : 0.0f;
                    dr[c] = in ? e * kr[i][c] : 0.0f;
                    dlam[c] += in ? e * kl[i][c] : 0.0f;
                    f[c] = decayed(w.value || is_weak(a1[i][c]), a1[i][c], e);
                }
                if (mine && t0 + at < p.T) {
                    store<T, CH>(gx, at * p.N + n, dx);
                    store<T, CH>(gr, at * p.N + n, dr);
                    store<T, CH>(gi, at * p.N + n, di);
                }
            }
            if (mine && a.grad_state && k == o.last && wave == 0 && q == 0)
                store<float, CH>(a.grad_state + (size_t)o.b * p.N, n, f);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                dlam[c] = of_half<0>(dlam[c]) + of_half<1>(dlam[c]);
                if (q == 0) dl[wave][l * CH + c] = dlam[c];
            }
            if (threadIdx.x == 0) sh.slot = ticket;
            __syncthreads();
            if (wave == 0 && q == 0 && mine) {
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int w = 1; w < W; ++w) dlam[c] += dl[w][l * CH + c];
                store<float, CH>(dout, n, dlam);
            }
            k = __builtin_amdgcn_readfirstlane((int)sh.slot);
        }
    };
    if (all_weak<CH>(lam)) tiles(Flag<true>{});
    else tiles(Flag<false>{});
}

// grid (ceil(N / 16)), block 1024: 16 columns, 64 groups of partial rows, joined in order
__global__ __launch_bounds__(1024) void k_recurrence_partials(const float* part, long rows, int N, float* out) {
    __shared__ float s[64][17];
    const int n = blockIdx.x * 16 + (threadIdx.x & 15), grp = threadIdx.x >> 4;
    const long per = (rows + 63) / 64, r1 = min(rows, (grp + 1) * per);
    float v = 0.0f;
    if (n < N) {
        constexpr int U = 8;                            // loads in flight
        for (long r = grp * per; r < r1; r += U) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = r + u < r1 ? part[(r + u) * N + n] : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) v += x[u];
        }
    }
    s[grp][threadIdx.x & 15] = v;
    __syncthreads();
    if (grp == 0 && n < N) {
        for (int i = 1; i < 64; ++i) v += s[i][threadIdx.x];
        out[n] = v;
    }
}

// One token: grid (ceil(N / 256), B).
template <class T>
__global__ __launch_bounds__(256) void k_recurrence_step(const semicrf_recurrence p, const int32_t* slots, int pool,
                                                         T* out, float* state_out) {
    const int n = blockIdx.x * 256 + threadIdx.x, b = blockIdx.y;
    if (n >= p.N) return;
    const int slot = slots ? slots[b] : b;
    const size_t o = (size_t)b * p.N + n;
    if (slot < 0 || slot >= pool) {
        out[o] = (T)0.0f;
        return;
    }
    const size_t at = (size_t)slot * p.N + n;
    const float x = (float)row<T>(p.x, p.x_stride, b, 0)[n];
    const float r = (float)row<T>(p.decay_gate, p.decay_stride, b, 0)[n];
    const float i = (float)row<T>(p.input_gate, p.input_stride, b, 0)[n];
    bool weak;
    float m, e;
    const float c = decay(p.log_decay[n] * sigmoid(r), weak, m, e);
    const float h = decayed(weak, c, p.state[at], root(-m * (m + 2.0f)) * (sigmoid(i) * x));
    state_out[at] = h;
    out[o] = (T)h;
}

// ------------------------------------------------------------------ host
constexpr int WIDE = 8, WIDE_GRAD = 12;      // wavefronts a workgroup: measured at the kernels
// Workgroups of a launch: 32 x 800 x 1,024 forward 56 us with 1,024 to 4,096, 63 with 512; longer sequences
// within 3 % of one another, but 1 x 250,001 x 256 in float32 forward (260 with 512, 292 to 297 with more).
constexpr int SERVE = 2048;

// Backward, whether each chain is one workgroup's, which carries what it passes on along and waits for no one:
// where there are chains for all compute units, and their last round leaves few of them idle.  In bfloat16 16 x
// 5,000 x 1,024 (256 chains) 297 us against 350 and 5 to clear what tiles wait for, 32 x 800 114 against 132
// and 5.  Chains of 800 and of 3,000 positions: 240 (all at once, 6 % idle) 61 against 72 and 181 against 211; 480
// (6 % of the last round idle) 117 against 137 and 343 against 397; 384 (25 %) 110 against 112, but 334 against
// 322; 272 (47 %) 98 against 100, but 318 against 293.  Forward, with three workgroups a compute unit to wait on
// one another, it is 112 against 118 and 5 at 64 x 800, but 202 against 172 at 16 x 5,000 and 56 against 50 and 5
// at 32 x 800 ragged: not taken there.
bool alone(long chains, bool grad) {
    return grad && chains >= 256 && ((chains + 255) / 256 * 256 - chains) * 10 <= chains;
}

// How a call is laid out: channels a lane, wavefronts a workgroup, and the workspace
struct Plan {
    int CH, W;
    Chain chain;
    int grid;
    bool fits, shared;           // whether workgroups share a chain
    size_t words, states, ticket, part, total;
};

Plan make_plan(const semicrf_recurrence& p, bool grad) {
    Plan q{};
    // One channel left over would be computed beside a neighbour that another workgroup has as well, whose final
    // state may be there already, over the initial one
    q.CH = p.N % (2 * LANES) == 1 ? 1 : 2;
    q.W = p.T <= SPAN ? 1 : grad ? WIDE_GRAD : WIDE;
    Chain& c = q.chain;
    c.tiles = (p.T + q.W * SPAN - 1) / (q.W * SPAN);
    c.groups = (c.tiles + GROUP - 1) / GROUP;
    c.cols = (p.N + LANES * q.CH - 1) / (LANES * q.CH);
    const long seqs = (long)p.B * c.cols;
    q.fits = seqs < (1l << 22);          // launches hold less than 2^32 threads
    c.chains = (unsigned)seqs;
    // enough workgroups on a chain that all of them together fill the GPU a few times over (chains of
    // short sequences end early)
    const bool single = alone(seqs, grad);
    long serve = single ? 1 : (SERVE + seqs - 1) / seqs;
    serve = serve < c.tiles ? serve : c.tiles;
    q.grid = (int)(seqs * serve);
    size_t at = 0;
    auto region = [&](size_t bytes) {
        const size_t r = at;
        at += (bytes + 255) / 256 * 256;
        return r;
    };
    q.shared = c.tiles > 1 && !single;
    q.ticket = region(q.shared ? seqs * TICKET * sizeof(unsigned) : 1);
    if (q.shared) {
        q.words = region(seqs * c.tiles * q.CH * LANES * 8);
        q.states = region(seqs * c.groups * q.CH * LANES * 8);
    }
    if (grad) q.part = region((size_t)c.tiles * p.B * p.N * sizeof(float));
    q.total = at;
    return q;
}

// Binds the plan to its workspace and clears what tiles wait for
void prepare(Plan& q, void* ws, hipStream_t stream) {
    if (!q.shared) return;
    char* w = (char*)ws;
    q.chain.tickets = (unsigned*)(w + q.ticket);
    q.chain.words = (unsigned long long*)(w + q.words);
    q.chain.states = (unsigned long long*)(w + q.states);
    const size_t n = (size_t)q.chain.chains * (q.chain.tiles + q.chain.groups) * q.CH * LANES;
    const size_t blocks = (n + 2047) / 2048;
    hipLaunchKernelGGL(k_recurrence_clear, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, stream,
                       q.chain.words, n, q.chain.tickets, (size_t)q.chain.chains * TICKET);
}

}  // namespace

size_t gated_recurrence_bytes(const semicrf_recurrence& p, bool grad) {
    const Plan q = make_plan(p, grad);
    return q.fits ? q.total : 0;
}

hipError_t launch_gated_recurrence(const RecArgs& a, void* ws, hipStream_t stream) {
    Plan q = make_plan(a.p, false);
    prepare(q, ws, stream);
#define RUN(T, CH)                                                                                             \
    if (q.W == 1)                                                                                              \
        hipLaunchKernelGGL((k_recurrence<T, CH, 1>), dim3(q.grid), dim3(64), 0, stream, a, q.chain);           \
    else                                                                                                       \
        hipLaunchKernelGGL((k_recurrence<T, CH, WIDE>), dim3(q.grid), dim3(64 * WIDE), 0, stream, a, q.chain);
    if (a.p.dtype == SEMICRF_F32) {
        if (q.CH == 2) { RUN(float, 2) } else { RUN(float, 1) }
    } else {
        if (q.CH == 2) { RUN(bf16, 2) } else { RUN(bf16, 1) }
    }
#undef RUN
    return hipGetLastError();
}

hipError_t launch_gated_recurrence_grad(const RecArgs& a, void* ws, hipStream_t stream) {
    Plan q = make_plan(a.p, true);
    prepare(q, ws, stream);
    float* part = (float*)((char*)ws + q.part);
#define RUN(T, CH)                                                                                             \
    if (q.W == 1)                                                                                              \
        hipLaunchKernelGGL((k_recurrence_grad<T, CH, 1>), dim3(q.grid), dim3(64), 0, stream, a, q.chain, part); \
    else                                                                                                       \
        hipLaunchKernelGGL((k_recurrence_grad<T, CH, WIDE_GRAD>), dim3(q.grid), dim3(64 * WIDE_GRAD), 0, stream, a, \
                           q.chain, part);
    if (a.p.dtype == SEMICRF_F32) {
        if (q.CH == 2) { RUN(float, 2) } else { RUN(float, 1) }
    } else {
        if (q.CH == 2) { RUN(bf16, 2) } else { RUN(bf16, 1) }
    }
#undef RUN
    if (a.grad_log_decay)
        hipLaunchKernelGGL(k_recurrence_partials, dim3((a.p.N + 15) / 16), dim3(1024), 0, stream, part,
                           (long)q.chain.tiles * a.p.B, a.p.N, a.grad_log_decay);
    return hipGetLastError();
}

hipError_t launch_gated_recurrence_step(const semicrf_recurrence& p, const int32_t* slots, int pool, void* out,
                                        float* state_out, hipStream_t stream) {
    const dim3 grid((p.N + 255) / 256, p.B);
    if (p.dtype == SEMICRF_F32)
        hipLaunchKernelGGL(k_recurrence_step<float>, grid, dim3(256), 0, stream, p, slots, pool, (float*)out,
                           state_out);
    else
        hipLaunchKernelGGL(k_recurrence_step<bf16>, grid, dim3(256), 0, stream, p, slots, pool, (bf16*)out,
                           state_out);
    return hipGetLastError();
}

}  // namespace semicrf
