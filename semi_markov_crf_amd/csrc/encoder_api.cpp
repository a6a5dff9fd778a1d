// C ABI of the encoder operators: argument checks and launches.  See include/semicrf.h for the
// contract.
#include <hip/hip_runtime.h>

#include "../../include/semicrf.h"
#include "encoder.h"

using namespace semicrf;

namespace {

constexpr long MAX_ROWS = 1l << 30;      // positions of a batch, rows of a table

bool type_ok(int dtype) { return dtype == SEMICRF_F32 || dtype == SEMICRF_BF16; }

int check_rows(int B, int T, int N) {
    if (B < 1 || T < 1 || N < 1) return SEMICRF_ERR_INVALID;
    return (long)B * T < MAX_ROWS ? SEMICRF_OK : SEMICRF_ERR_UNSUPPORTED;
}

int check_ws(const void* ws, size_t have, size_t need) {
    return !ws || have < need || (uintptr_t)ws % 256 ? SEMICRF_ERR_WORKSPACE : SEMICRF_OK;
}

int done(hipError_t e) { return e == hipSuccess ? SEMICRF_OK : SEMICRF_ERR_DEVICE; }

int check_embed(const void* tokens, int token_bits, int dtype, int B, int T, int V, int N) {
    if (!tokens || (token_bits != 32 && token_bits != 64) || !type_ok(dtype) || V < 1)
        return SEMICRF_ERR_INVALID;
    const int rc = check_rows(B, T, N);
    if (rc) return rc;
    return V < MAX_ROWS && N < MAX_ROWS ? SEMICRF_OK : SEMICRF_ERR_UNSUPPORTED;
}

int check_norm(const void* x, int dtype, int wdtype, int B, int T, int N) {
    if (!x || !type_ok(dtype) || (wdtype != dtype && wdtype != SEMICRF_F32))
        return SEMICRF_ERR_INVALID;
    const int rc = check_rows(B, T, N);
    if (rc) return rc;
    return N <= NORM_MAX_N ? SEMICRF_OK : SEMICRF_ERR_UNSUPPORTED;
}

int check_shape(const semicrf_attention* p) {
    if (!p || !type_ok(p->dtype) || p->Hq < 1 || p->Hk < 1 || p->Dk < 1 || p->Dv < 1 || p->Hq % p->Hk)
        return SEMICRF_ERR_INVALID;
    const int rc = check_rows(p->B, p->T, 1);
    if (rc) return rc;
    if (p->Dk > ATTN_MAX_D || p->Dv > ATTN_MAX_D || p->B >= 65536 || p->Hq >= 32768)
        return SEMICRF_ERR_UNSUPPORTED;
    return SEMICRF_OK;
}

int check_attention(const semicrf_attention* p) {
    const int rc = check_shape(p);
    if (rc) return rc;
    return p->q && p->k && p->v && p->log_decay ? SEMICRF_OK : SEMICRF_ERR_INVALID;
}

}  // namespace

extern "C" {

int semicrf_embed(const void* tokens, int token_bits, const int32_t* lengths, const void* table,
                  int dtype, int B, int T, int V, int N, float scale, hipStream_t stream,
                  void* out, int32_t* status) {
    const int rc = check_embed(tokens, token_bits, dtype, B, T, V, N);
    if (rc) return rc;
    if (!table || !out) return SEMICRF_ERR_INVALID;
    EmbedArgs a{};
    a.tokens = tokens; a.token_bits = token_bits; a.lengths = lengths; a.table = table;
    a.dtype = dtype; a.B = B; a.T = T; a.V = V; a.N = N; a.scale = scale;
    a.out = out; a.status = status;
    return done(launch_embed(a, stream));
}

size_t semicrf_embed_grad_bytes(int dtype, int B, int T, int V, int N) {
    if (!type_ok(dtype) || check_rows(B, T, N) || V < 1 || V >= MAX_ROWS || N > EMBED_GRAD_MAX_N) return 0;
    return embed_grad_bytes(B, T, V, N, dtype);
}

int semicrf_embed_grad(const void* tokens, int token_bits, const int32_t* lengths,
                       const void* grad_out, int dtype, int B, int T, int V, int N, float scale,
                       hipStream_t stream, void* workspace, size_t workspace_bytes,
                       void* grad_table, int32_t* status) {
    int rc = check_embed(tokens, token_bits, dtype, B, T, V, N);
    if (rc) return rc;
    if (N > EMBED_GRAD_MAX_N) return SEMICRF_ERR_UNSUPPORTED;
    if (!grad_out || !grad_table) return SEMICRF_ERR_INVALID;
    if ((rc = check_ws(workspace, workspace_bytes, embed_grad_bytes(B, T, V, N, dtype)))) return rc;
    EmbedArgs a{};
    a.tokens = tokens; a.token_bits = token_bits; a.lengths = lengths; a.grad_out = grad_out;
    a.dtype = dtype; a.B = B; a.T = T; a.V = V; a.N = N; a.scale = scale;
    a.out = grad_table; a.status = status;
    return done(launch_embed_grad(a, workspace, stream));
}

int semicrf_layer_norm(const void* x, int dtype, const void* weight, const void* bias, int wdtype,
                       const int32_t* lengths, int B, int T, int N, float eps, hipStream_t stream,
                       void* y, float* mean, float* rstd, int32_t* status) {
    const int rc = check_norm(x, dtype, wdtype, B, T, N);
    if (rc) return rc;
    if (!y || !(eps >= 0.0f)) return SEMICRF_ERR_INVALID;
    NormArgs a{};
    a.x = x; a.weight = weight; a.bias = bias; a.lengths = lengths;
    a.dtype = dtype; a.wdtype = wdtype; a.B = B; a.T = T; a.N = N; a.eps = eps;
    a.y = y; a.mean = mean; a.rstd = rstd; a.status = status;
    return done(launch_layer_norm(a, stream));
}

size_t semicrf_layer_norm_grad_bytes(int dtype, int B, int T, int N) {
    if (!type_ok(dtype) || check_rows(B, T, N) || N > NORM_MAX_N) return 0;
    return layer_norm_grad_bytes(B, T, N, dtype);
}

int semicrf_layer_norm_grad(const void* grad_out, const void* x, int dtype, const void* weight,
                            int wdtype, const float* mean, const float* rstd,
                            const int32_t* lengths, int B, int T, int N, hipStream_t stream,
                            void* workspace, size_t workspace_bytes, void* grad_x,
                            void* grad_weight, void* grad_bias, int32_t* status) {
    int rc = check_norm(x, dtype, wdtype, B, T, N);
    if (rc) return rc;
    if (!grad_out || !mean || !rstd || !grad_x) return SEMICRF_ERR_INVALID;
    if ((rc = check_ws(workspace, workspace_bytes, layer_norm_grad_bytes(B, T, N, dtype)))) return rc;
    NormArgs a{};
    a.x = x; a.grad_out = grad_out; a.weight = weight; a.mean_in = mean; a.rstd_in = rstd;
    a.lengths = lengths; a.dtype = dtype; a.wdtype = wdtype; a.B = B; a.T = T; a.N = N;
    a.grad_x = grad_x; a.grad_weight = grad_weight; a.grad_bias = grad_bias; a.status = status;
    return done(launch_layer_norm_grad(a, workspace, stream));
}

size_t semicrf_decay_attention_bytes(const semicrf_attention* attention, int grad) {
    return check_shape(attention) ? 0 : decay_attention_bytes(*attention, grad != 0);
}

int semicrf_decay_attention(const semicrf_attention* attention, hipStream_t stream,
                            void* workspace, size_t workspace_bytes, void* out,
                            float* state_out, int32_t* status) {
    int rc = check_attention(attention);
    if (rc) return rc;
    if (!out) return SEMICRF_ERR_INVALID;
    if ((rc = check_ws(workspace, workspace_bytes, decay_attention_bytes(*attention, false)))) return rc;
    AttnArgs a{};
    a.p = *attention; a.out = out; a.state_out = state_out; a.status = status;
    return done(launch_decay_attention(a, workspace, stream));
}

int semicrf_decay_attention_grad(const semicrf_attention* attention, const void* grad_out,
                                 const float* grad_state_out, hipStream_t stream, void* workspace,
                                 size_t workspace_bytes, void* grad_q, void* grad_k, void* grad_v,
                                 float* grad_state, int32_t* status) {
    int rc = check_attention(attention);
    if (rc) return rc;
    if (!grad_out || !grad_q || !grad_k || !grad_v) return SEMICRF_ERR_INVALID;
    if ((rc = check_ws(workspace, workspace_bytes, decay_attention_bytes(*attention, true)))) return rc;
    AttnArgs a{};
    a.p = *attention; a.grad_out = grad_out; a.grad_state_out = grad_state_out;
    a.grad_q = grad_q; a.grad_k = grad_k; a.grad_v = grad_v; a.grad_state = grad_state;
    a.status = status;
    return done(launch_decay_attention_grad(a, workspace, stream));
}

int semicrf_decay_attention_step(const semicrf_attention* attention, const int32_t* slots,
                                 int pool, hipStream_t stream, void* out, float* state_out) {
    const int rc = check_attention(attention);
    if (rc) return rc;
    if (!out || !state_out || !attention->state || attention->T != 1 || attention->lengths || pool < 1 ||
        (!slots && pool < attention->B))
        return SEMICRF_ERR_INVALID;
    return done(launch_decay_attention_step(*attention, slots, pool, out, state_out, stream));
}

}  // extern "C"
