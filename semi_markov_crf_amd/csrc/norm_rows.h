// Rows of a norm shared out over lanes: what layer norm and the residual norm have in common.
#pragma once

#include "common.h"
#include "encoder.h"

namespace semicrf {

// How rows lie in the lanes' pieces: they fill them exactly (G * KP * V elements), or not, or are
// narrower than one.
enum { EXACT, MASKED, NARROWER };

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

}  // namespace semicrf
