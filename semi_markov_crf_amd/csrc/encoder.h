// Shared by the encoder operators (embedding, layer norm, decayed linear attention, gated
// recurrence, residual norm, token loss): element types, 16-byte pieces of rows, and the
// interfaces between encoder_api.cpp and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/semicrf.h"

namespace semicrf {

using bf16 = __bf16;

// A row of N elements is taken in pieces of 16 bytes, V elements.  Global loads and stores of 16
// bytes need no 16-byte alignment on gfx950, so rows of any width take the same path: where N is
// no multiple of V the last piece starts early, at N - V, and its first `skip` elements are the
// piece before's too (loaded and stored twice with the same values, added up once).  A lane past
// the row's pieces holds the last one with skip = V.  NARROW: N < V, element by element.
template <class T, bool NARROW = false>
struct Piece {
    static constexpr int V = 16 / sizeof(T);
    int at, skip;
    __device__ __forceinline__ Piece(int i, int N) {
        const int c = i * V;
        at = NARROW ? 0 : min(c, N - V);
        skip = NARROW ? (c < N ? 0 : V) : min(c - at, V);
    }
};

typedef uint32_t raw_piece __attribute__((ext_vector_type(4)));
typedef raw_piece loose_piece __attribute__((aligned(1)));

template <class T, bool NARROW>
__device__ __forceinline__ raw_piece load_raw(const T* __restrict__ row, const Piece<T, NARROW>& p, int N) {
    if constexpr (!NARROW) {
        return *(const loose_piece*)(row + p.at);
    } else {
        constexpr int V = 16 / sizeof(T);
        T t[V];
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = i < N ? row[i] : (T)0.0f;
        raw_piece x;
        __builtin_memcpy(&x, t, 16);
        return x;
    }
}
template <class T>
__device__ __forceinline__ void unpack(const raw_piece& r, float (&x)[16 / sizeof(T)]) {
    T t[16 / sizeof(T)];
    __builtin_memcpy(t, &r, 16);
#pragma unroll
    for (int i = 0; i < 16 / (int)sizeof(T); ++i) x[i] = (float)t[i];
}
// STREAM: the store does not keep its line in the caches.
template <class T, bool STREAM = false, bool NARROW>
__device__ __forceinline__ void store_piece(T* __restrict__ row, const Piece<T, NARROW>& p, int N,
                                            const float (&x)[16 / sizeof(T)]) {
    constexpr int V = 16 / sizeof(T);
    T t[V];
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = (T)x[i];
    if (p.skip == V) return;
    if constexpr (!NARROW) {
        raw_piece r;
        __builtin_memcpy(&r, t, 16);
        if constexpr (STREAM) __builtin_nontemporal_store(r, (loose_piece*)(row + p.at));
        else *(loose_piece*)(row + p.at) = r;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < N) row[i] = t[i];
    }
}

// V elements of type W from element `at` of a row, zeros past N
template <class W, int V>
__device__ __forceinline__ void load_elements(const W* __restrict__ row, int at, int N, float (&x)[V]) {
    W t[V];
    if (at + V <= N) {
        __builtin_memcpy(t, row + at, sizeof(t));
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = (float)t[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = at + i < N ? (float)row[at + i] : 0.0f;
    }
}
template <int V>
__device__ __forceinline__ void store_elements(float* __restrict__ row, int at, int N, const float (&x)[V]) {
    if (at + V <= N) {
        __builtin_memcpy(row + at, x, sizeof(x));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (at + i < N) row[at + i] = x[i];
    }
}

// Loads and stores are counted together, in order.  A loop that fetches its next input, then stores
// its output, would wait at its top for the stores too (the first round has none to allow for).
// Waiting for the fetch before the loop and before the stores leaves the stores in flight.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }   // vmcnt(0)

// Length of sequence b, clamped to [0, T]; a length outside raises the caller's status word.
__device__ __forceinline__ int seq_length(const int32_t* __restrict__ lengths, int b, int T,
                                          int32_t* status) {
    if (!lengths) return T;
    const int L = lengths[b];
    if (L >= 0 && L <= T) return L;
    if (status) atomicOr(status, 1);
    return L < 0 ? 0 : T;
}

// ------------------------------------------------------------------ launch interfaces
struct EmbedArgs {
    const void* tokens;
    int token_bits;
    const int32_t* lengths;
    const void* table;       // embed
    const void* grad_out;    // embed_grad
    int dtype, B, T, V, N;
    unsigned first;          // embed: first row of a launch
    float scale;
    void* out;               // y, or the gradient of the table
    int32_t* status;
};
constexpr int EMBED_GRAD_MAX_N = 1 << 23;      // slabs of columns are the second grid dimension, below 2^16
hipError_t launch_embed(const EmbedArgs& a, hipStream_t stream);
size_t embed_grad_bytes(int B, int T, int V, int N, int dtype);
hipError_t launch_embed_grad(const EmbedArgs& a, void* ws, hipStream_t stream);

struct NormArgs {
    const void *x, *grad_out, *weight, *bias;
    const float *mean_in, *rstd_in;
    const int32_t* lengths;
    int dtype, wdtype, B, T, N;
    float eps;
    void *y, *grad_x, *grad_weight, *grad_bias;
    float *mean, *rstd;
    int32_t* status;
};
constexpr int NORM_MAX_N = 32768;
hipError_t launch_layer_norm(const NormArgs& a, hipStream_t stream);
size_t layer_norm_grad_bytes(int B, int T, int N, int dtype);
hipError_t launch_layer_norm_grad(const NormArgs& a, void* ws, hipStream_t stream);

struct AttnArgs {
    semicrf_attention p;
    void* out;               // [B, T, Hq, Dv]
    float* state_out;
    const void* grad_out;
    const float* grad_state_out;
    void *grad_q, *grad_k, *grad_v;
    float* grad_state;
    int32_t* status;
};
constexpr int ATTN_MAX_D = 128;
size_t decay_attention_bytes(const semicrf_attention& p, bool grad);
hipError_t launch_decay_attention(const AttnArgs& a, void* ws, hipStream_t stream);
hipError_t launch_decay_attention_grad(const AttnArgs& a, void* ws, hipStream_t stream);
hipError_t launch_decay_attention_step(const semicrf_attention& p, const int32_t* slots, int pool,
                                       void* out, float* state_out, hipStream_t stream);

struct RecArgs {
    semicrf_recurrence p;
    const float* starts_in;
    const void* grad_out;
    const float* grad_state_out;
    void* out;               // h
    float *state_out, *starts;
    void *grad_x, *grad_decay, *grad_input;
    float *grad_log_decay, *grad_state;
    int32_t* status;
};
constexpr int REC_MAX_N = 1 << 20;
size_t gated_recurrence_bytes(const semicrf_recurrence& p, bool grad);
hipError_t launch_gated_recurrence(const RecArgs& a, void* ws, hipStream_t stream);
hipError_t launch_gated_recurrence_grad(const RecArgs& a, void* ws, hipStream_t stream);
hipError_t launch_gated_recurrence_step(const semicrf_recurrence& p, const int32_t* slots, int pool,
                                        void* out, float* state_out, hipStream_t stream);

struct ResArgs {
    semicrf_residual p;
    void *r, *y;
    float* stats;
    const float* stats_in;
    const void *grad_r, *grad_y;
    void *grad_x, *grad_branch, *grad_gate, *grad_params;
    int32_t* status;
};
constexpr int RES_MAX_N = 16384;
hipError_t launch_residual_norm(const ResArgs& a, hipStream_t stream);
size_t residual_norm_grad_bytes(int B, int T, int N, int dtype);
hipError_t launch_residual_norm_grad(const ResArgs& a, void* ws, hipStream_t stream);

struct NllArgs {
    const void *x, *table, *targets;
    const int32_t* lengths;
    const float *grad_loss, *lse_in;
    int dtype, target_bits, B, T, V, N;
    float scale;
    float *loss, *lse;
    void *grad_x, *grad_table;
    int32_t* status;
};
constexpr long NLL_MAX_ROWS = 1l << 22;        // of x and of the table: 256 rows of p span at most 2^32 bytes
constexpr int NLL_MAX_N = 32768;
// table: the array, or NULL for what is enough for any
size_t token_nll_bytes(int dtype, int B, int T, int V, int N, const void* table, bool grad);
hipError_t launch_token_nll(const NllArgs& a, void* ws, hipStream_t stream);
hipError_t launch_token_nll_grad(const NllArgs& a, void* ws, hipStream_t stream);

}  // namespace semicrf
