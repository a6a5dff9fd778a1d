// Shared by the encoder operators (embedding, layer norm, decayed linear attention): element
// types, 16-byte pieces of rows, and the interfaces between encoder_api.cpp and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/semicrf.h"

namespace semicrf {

using bf16 = __bf16;

// A row of N elements is taken in pieces of 16 bytes.  Global loads and stores of 16 bytes
// need no 16-byte alignment on gfx950, so rows of any width take the same path; only the
// last piece of a row whose width is no multiple of V goes element by element.
template <class T>
struct Piece {
    static constexpr int V = 16 / sizeof(T);
};

template <class T>
__device__ __forceinline__ void load_piece(const T* __restrict__ p, int valid,
                                           float (&x)[Piece<T>::V]) {
    constexpr int V = Piece<T>::V;
    if (valid >= V) {
        T t[V];
        __builtin_memcpy(t, p, 16);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = (float)t[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i < valid ? (float)p[i] : 0.0f;
    }
}

typedef uint32_t raw_piece __attribute__((ext_vector_type(4)));
typedef raw_piece loose_piece __attribute__((aligned(1)));

// STREAM: the store does not keep its line in the caches.
template <class T, bool STREAM = false>
__device__ __forceinline__ void store_piece(T* __restrict__ p, int valid,
                                            const float (&x)[Piece<T>::V]) {
    constexpr int V = Piece<T>::V;
    if (valid >= V) {
        T t[V];
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = (T)x[i];
        raw_piece r;
        __builtin_memcpy(&r, t, 16);
        if constexpr (STREAM) __builtin_nontemporal_store(r, (loose_piece*)p);
        else *(loose_piece*)p = r;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < valid) p[i] = (T)x[i];
    }
}

// Loads and stores are counted together, in order.  A loop that fetches its next input, then stores
// its output, would wait at its top for the stores too (the first round has none to allow for).
// Waiting for the fetch before the loop and before the stores leaves the stores in flight.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }   // vmcnt(0)

// A piece as it lies in memory; what is past `valid` elements is zero.
template <class T>
__device__ __forceinline__ raw_piece load_raw(const T* __restrict__ p, int valid) {
    constexpr int V = Piece<T>::V;
    raw_piece x = {0, 0, 0, 0};
    if (valid >= V) {
        __builtin_memcpy(&x, p, 16);
    } else if (valid > 0) {
        T t[V];
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = i < valid ? p[i] : (T)0.0f;
        __builtin_memcpy(&x, t, 16);
    }
    return x;
}
template <class T>
__device__ __forceinline__ void unpack(const raw_piece& r, float (&x)[Piece<T>::V]) {
    T t[Piece<T>::V];
    __builtin_memcpy(t, &r, 16);
#pragma unroll
    for (int i = 0; i < Piece<T>::V; ++i) x[i] = (float)t[i];
}

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
    float scale;
    void* out;               // y, or the gradient of the table
    int32_t* status;
};
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

}  // namespace semicrf
