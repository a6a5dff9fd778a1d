// Gated linear recurrence, forward, backward and one token at a time, on gfx950.
//
//   s = log_decay sig(r),  a = exp(s),  b = sqrt(1 - a^2),  u = sig(i) x,  h_t = a_t h_{t-1} + b_t u_t
//   backward, with E_t = g_t + a_{t+1} E_{t+1} the gradient of h_t:
//     ds = E (a h_{t-1} - a^2 / b u),  dr = ds s (1 - sig r),  dlog_decay = sum ds sig(r)
//     du = E b,  dx = du sig(i),  di = du u (1 - sig i),  dh_0 = a_1 E_1
//
// A decay next to 1 is kept as its distance from 1: m = a - 1 = expm1(s) has a relative rounding
// error, where a = 1 + m would lose what is below 2^-24 and with it time constants of many
// positions.  h_t = h_{t-1} + m h_{t-1} + b u, and 1 - a^2 = -m (m + 2).  The gradient's factor a, which
// may be far below 1, is the exponential itself.
#include "common.h"
#include "encoder.h"
#include "gates.h"

namespace semicrf {

namespace {

constexpr int SPAN = SEMICRF_RECURRENCE_SPAN;

// expm1 for s <= 0, and exp(s).  Below -1/4 the difference costs at most two bits; above, five terms
// of the series leave s^6 / 5040 < 2^-24.
__device__ __forceinline__ float expm1_neg(float s, float& e) {
    float p = fmaf(s, 1.0f / 720.0f, 1.0f / 120.0f);
    p = fmaf(s, p, 1.0f / 24.0f);
    p = fmaf(s, p, 1.0f / 6.0f);
    p = fmaf(s, p, 0.5f);
    p = fmaf(s * s, p, s);
    e = fast_exp2(s * LOG2EF);
    return s > -0.25f ? p : e - 1.0f;
}
__device__ __forceinline__ float expm1_neg(float s) {
    float e;
    return expm1_neg(s, e);
}

__device__ __forceinline__ float root(float x) { return __builtin_amdgcn_sqrtf(x); }

template <class T>
__device__ __forceinline__ const T* row(const void* p, const int64_t (&stride)[2], int b, int t) {
    return (const T*)p + b * stride[0] + t * stride[1];
}

// grid (ceil(N / 64), B), block 64: a channel a thread
template <class T>
__global__ __launch_bounds__(64) void k_recurrence(const RecArgs a) {
    const semicrf_recurrence& p = a.p;
    const int n = blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
    const int L = seq_length(p.lengths, b, p.T, a.status);
    if (n >= p.N) return;
    const float lam = p.log_decay[n];
    float h = p.state ? p.state[(size_t)b * p.N + n] : 0.0f;
    const size_t spans = (p.T + SPAN - 1) / SPAN;
    for (int t = 0; t < p.T; ++t) {
        T* out = (T*)a.out + ((size_t)b * p.T + t) * p.N + n;
        if (t >= L) {
            *out = (T)0.0f;
            continue;
        }
        if (a.starts && t % SPAN == 0) a.starts[((size_t)b * spans + t / SPAN) * p.N + n] = h;
        const float x = (float)row<T>(p.x, p.x_stride, b, t)[n];
        const float r = (float)row<T>(p.decay_gate, p.decay_stride, b, t)[n];
        const float i = (float)row<T>(p.input_gate, p.input_stride, b, t)[n];
        const float m = expm1_neg(lam * sigmoid(r));
        h = fmaf(m, h, root(-m * (m + 2.0f)) * (sigmoid(i) * x)) + h;
        *out = (T)h;
    }
    if (a.state_out) a.state_out[(size_t)b * p.N + n] = h;
}

// the same grid; part [B][N]: the sequence's share of the gradient of log_decay
template <class T>
__global__ __launch_bounds__(64) void k_recurrence_grad(const RecArgs a, float* part) {
    const semicrf_recurrence& p = a.p;
    const int n = blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
    const int L = seq_length(p.lengths, b, p.T, a.status);
    if (n >= p.N) return;
    const float lam = p.log_decay[n];
    const size_t spans = (p.T + SPAN - 1) / SPAN, at = (size_t)b * p.T * p.N + n;
    float e = a.grad_state_out ? a.grad_state_out[(size_t)b * p.N + n] : 0.0f, dlam = 0.0f;
    for (int j = (int)spans - 1; j >= 0; --j) {
        const int t0 = j * SPAN;
        float h[SPAN], m[SPAN], av[SPAN];
        if (t0 < L) h[0] = a.starts_in[((size_t)b * spans + j) * p.N + n];
#pragma unroll
        for (int k = 0; k < SPAN; ++k) {
            const int t = t0 + k;
            m[k] = 0.0f;
            float bu = 0.0f;
            if (t < L) {
                m[k] = expm1_neg(lam * sigmoid((float)row<T>(p.decay_gate, p.decay_stride, b, t)[n]), av[k]);
                bu = root(-m[k] * (m[k] + 2.0f)) * sigmoid((float)row<T>(p.input_gate, p.input_stride, b, t)[n]) *
                     (float)row<T>(p.x, p.x_stride, b, t)[n];
            }
            if (k + 1 < SPAN) h[k + 1] = fmaf(m[k], h[k], bu) + h[k];
        }
#pragma unroll
        for (int k = SPAN - 1; k >= 0; --k) {
            const int t = t0 + k;
            if (t >= p.T) continue;
            const size_t o = at + (size_t)t * p.N;
            float dx = 0.0f, dr = 0.0f, di = 0.0f;
            if (t < L) {
                float sr, qr, si, qi;
                sigmoids((float)row<T>(p.decay_gate, p.decay_stride, b, t)[n], sr, qr);
                sigmoids((float)row<T>(p.input_gate, p.input_stride, b, t)[n], si, qi);
                const float x = (float)row<T>(p.x, p.x_stride, b, t)[n], s = lam * sr, u = si * x;
                const float bb = -m[k] * (m[k] + 2.0f), ib = bb > 0x1p-123f ? __builtin_amdgcn_rsqf(bb) : 0.0f;
                e += (float)((const T*)a.grad_out)[o];
                const float ds = e * av[k] * (h[k] - av[k] * ib * u), du = e * root(bb);
                dx = du * si;
                di = du * u * qi;
                dr = ds * s * qr;
                dlam += ds * sr;
                e = fmaf(m[k], e, e);
            }
            ((T*)a.grad_x)[o] = (T)dx;
            ((T*)a.grad_decay)[o] = (T)dr;
            ((T*)a.grad_input)[o] = (T)di;
        }
    }
    if (a.grad_state) a.grad_state[(size_t)b * p.N + n] = e;
    part[(size_t)b * p.N + n] = dlam;
}

__global__ __launch_bounds__(64) void k_recurrence_partials(const float* part, int rows, int N, float* out) {
    const int n = blockIdx.x * 64 + threadIdx.x;
    if (n >= N) return;
    float v = 0.0f;
    for (int r = 0; r < rows; ++r) v += part[(size_t)r * N + n];
    out[n] = v;
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
    const float m = expm1_neg(p.log_decay[n] * sigmoid(r)), h0 = p.state[at];
    const float h = fmaf(m, h0, root(-m * (m + 2.0f)) * (sigmoid(i) * x)) + h0;
    state_out[at] = h;
    out[o] = (T)h;
}

}  // namespace

size_t gated_recurrence_bytes(const semicrf_recurrence& p, bool grad) {
    return grad ? ((size_t)p.B * p.N * sizeof(float) + 255) / 256 * 256 : 256;
}

hipError_t launch_gated_recurrence(const RecArgs& a, void*, hipStream_t stream) {
    const dim3 grid((a.p.N + 63) / 64, a.p.B);
    if (a.p.dtype == SEMICRF_F32) hipLaunchKernelGGL(k_recurrence<float>, grid, dim3(64), 0, stream, a);
    else hipLaunchKernelGGL(k_recurrence<bf16>, grid, dim3(64), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_gated_recurrence_grad(const RecArgs& a, void* ws, hipStream_t stream) {
    const dim3 grid((a.p.N + 63) / 64, a.p.B);
    float* part = (float*)ws;
    if (a.p.dtype == SEMICRF_F32) hipLaunchKernelGGL(k_recurrence_grad<float>, grid, dim3(64), 0, stream, a, part);
    else hipLaunchKernelGGL(k_recurrence_grad<bf16>, grid, dim3(64), 0, stream, a, part);
    if (a.grad_log_decay)
        hipLaunchKernelGGL(k_recurrence_partials, dim3(grid.x), dim3(64), 0, stream, part, a.p.B, a.p.N,
                           a.grad_log_decay);
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
