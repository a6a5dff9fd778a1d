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

int check_recurrence_shape(const semicrf_recurrence* p) {
    if (!p || !type_ok(p->dtype)) return SEMICRF_ERR_INVALID;
    const int rc = check_rows(p->B, p->T, p->N);
    if (rc) return rc;
    // 16 positions of a row are addressed by 32 bits
    const int64_t s[3] = {p->x_stride[1], p->decay_stride[1], p->input_stride[1]};
    for (int i = 0; i < 3; ++i)
        if (p->T > 1 && (s[i] < 0 || s[i] >= 1 << 25)) return SEMICRF_ERR_UNSUPPORTED;
    return p->N <= REC_MAX_N && p->B < 65536 ? SEMICRF_OK : SEMICRF_ERR_UNSUPPORTED;
}

int check_recurrence(const semicrf_recurrence* p) {
    const int rc = check_recurrence_shape(p);
    if (rc) return rc;
    return p->x && p->decay_gate && p->input_gate && p->log_decay ? SEMICRF_OK : SEMICRF_ERR_INVALID;
}

int check_residual(const semicrf_residual* p) {
    if (!p || !p->branch || !(p->eps >= 0.0f)) return SEMICRF_ERR_INVALID;
    const int rc = check_norm(p->x, p->dtype, p->wdtype, p->B, p->T, p->N);
    if (rc) return rc;
    return p->N <= RES_MAX_N ? SEMICRF_OK : SEMICRF_ERR_UNSUPPORTED;
}

int check_nll_shape(int dtype, int B, int T, int V, int N) {
    if (!type_ok(dtype) || V < 1) return SEMICRF_ERR_INVALID;
    const int rc = check_rows(B, T, N);
    if (rc) return rc;
    if ((long)B * T > NLL_MAX_ROWS || V > NLL_MAX_ROWS || N > NLL_MAX_N) return SEMICRF_ERR_UNSUPPORTED;
    // x and the table are laid out by blocks of 64 x 64 in one launch, of less than 2^32 threads; pieces of the
    // vocabulary, rounded up, add less than 2^16 words
    return (((long)B * T + V) / 64 + 1040) * ((N + 63) / 64) < (1l << 24) ? SEMICRF_OK : SEMICRF_ERR_UNSUPPORTED;
}

int check_nll(const void* x, const void* table, const void* targets, int target_bits, int dtype, int B,
              int T, int V, int N, float scale) {
    if (!x || !table || !targets || (target_bits != 32 && target_bits != 64) || !(scale - scale == 0.0f))
        return SEMICRF_ERR_INVALID;
    return check_nll_shape(dtype, B, T, V, N);
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

size_t semicrf_gated_recurrence_bytes(const semicrf_recurrence* recurrence, int grad) {
    return check_recurrence_shape(recurrence) ? 0 : gated_recurrence_bytes(*recurrence, grad != 0);
}

int semicrf_gated_recurrence(const semicrf_recurrence* recurrence, hipStream_t stream,
                             void* workspace, size_t workspace_bytes, void* out, float* state_out,
                             float* starts, int32_t* status) {
    int rc = check_recurrence(recurrence);
    if (rc) return rc;
    if (!out) return SEMICRF_ERR_INVALID;
    const size_t need = gated_recurrence_bytes(*recurrence, false);
    if (!need) return SEMICRF_ERR_UNSUPPORTED;
    if ((rc = check_ws(workspace, workspace_bytes, need))) return rc;
    RecArgs a{};
    a.p = *recurrence; a.out = out; a.state_out = state_out; a.starts = starts; a.status = status;
    return done(launch_gated_recurrence(a, workspace, stream));
}

int semicrf_gated_recurrence_grad(const semicrf_recurrence* recurrence, const float* starts,
                                  const void* grad_out, const float* grad_state_out,
                                  hipStream_t stream, void* workspace, size_t workspace_bytes,
                                  void* grad_x, void* grad_decay_gate, void* grad_input_gate,
                                  float* grad_log_decay, float* grad_state, int32_t* status) {
    int rc = check_recurrence(recurrence);
    if (rc) return rc;
    if (!starts || !grad_out || !grad_x || !grad_decay_gate || !grad_input_gate) return SEMICRF_ERR_INVALID;
    const size_t need = gated_recurrence_bytes(*recurrence, true);
    if (!need) return SEMICRF_ERR_UNSUPPORTED;
    if ((rc = check_ws(workspace, workspace_bytes, need))) return rc;
    RecArgs a{};
    a.p = *recurrence; a.starts_in = starts; a.grad_out = grad_out; a.grad_state_out = grad_state_out;
    a.grad_x = grad_x; a.grad_decay = grad_decay_gate; a.grad_input = grad_input_gate;
    a.grad_log_decay = grad_log_decay; a.grad_state = grad_state; a.status = status;
    return done(launch_gated_recurrence_grad(a, workspace, stream));
}

int semicrf_gated_recurrence_step(const semicrf_recurrence* recurrence, const int32_t* slots,
                                  int pool, hipStream_t stream, void* out, float* state_out) {
    const int rc = check_recurrence(recurrence);
    if (rc) return rc;
    if (!out || !state_out || !recurrence->state || recurrence->T != 1 || recurrence->lengths || pool < 1 ||
        (!slots && pool < recurrence->B))
        return SEMICRF_ERR_INVALID;
    return done(launch_gated_recurrence_step(*recurrence, slots, pool, out, state_out, stream));
}

int semicrf_residual_norm(const semicrf_residual* residual, hipStream_t stream, void* r, void* y,
                          float* stats, int32_t* status) {
    const int rc = check_residual(residual);
    if (rc) return rc;
    if (!r || !y) return SEMICRF_ERR_INVALID;
    ResArgs a{};
    a.p = *residual; a.r = r; a.y = y; a.stats = stats; a.status = status;
    return done(launch_residual_norm(a, stream));
}

size_t semicrf_residual_norm_grad_bytes(int dtype, int B, int T, int N) {
    if (!type_ok(dtype) || check_rows(B, T, N) || N > RES_MAX_N) return 0;
    return residual_norm_grad_bytes(B, T, N, dtype);
}

int semicrf_residual_norm_grad(const semicrf_residual* residual, const float* stats,
                               const void* grad_r, const void* grad_y, hipStream_t stream,
                               void* workspace, size_t workspace_bytes, void* grad_x,
                               void* grad_branch, void* grad_gate, void* grad_params,
                               int32_t* status) {
    int rc = check_residual(residual);
    if (rc) return rc;
    if (!stats || !grad_x || !grad_branch || (residual->gate && !grad_gate)) return SEMICRF_ERR_INVALID;
    const size_t need = residual_norm_grad_bytes(residual->B, residual->T, residual->N, residual->dtype);
    if ((rc = check_ws(workspace, workspace_bytes, need))) return rc;
    ResArgs a{};
    a.p = *residual; a.stats_in = stats; a.grad_r = grad_r; a.grad_y = grad_y; a.grad_x = grad_x;
    a.grad_branch = grad_branch; a.grad_gate = grad_gate; a.grad_params = grad_params; a.status = status;
    return done(launch_residual_norm_grad(a, workspace, stream));
}

size_t semicrf_token_nll_bytes(int dtype, int B, int T, int V, int N, int grad) {
    return semicrf_token_nll_table_bytes(dtype, B, T, V, N, nullptr, grad);
}

size_t semicrf_token_nll_table_bytes(int dtype, int B, int T, int V, int N, const void* table, int grad) {
    return check_nll_shape(dtype, B, T, V, N) ? 0 : token_nll_bytes(dtype, B, T, V, N, table, grad != 0);
}

int semicrf_token_nll(const void* x, const void* table, int dtype, const void* targets,
                      int target_bits, const int32_t* lengths, int B, int T, int V, int N,
                      float scale, hipStream_t stream, void* workspace, size_t workspace_bytes,
                      float* loss, float* lse, int32_t* status) {
    int rc = check_nll(x, table, targets, target_bits, dtype, B, T, V, N, scale);
    if (rc) return rc;
    if (!loss) return SEMICRF_ERR_INVALID;
    if ((rc = check_ws(workspace, workspace_bytes, token_nll_bytes(dtype, B, T, V, N, table, false)))) return rc;
    NllArgs a{};
    a.x = x; a.table = table; a.targets = targets; a.target_bits = target_bits; a.lengths = lengths;
    a.dtype = dtype; a.B = B; a.T = T; a.V = V; a.N = N; a.scale = scale;
    a.loss = loss; a.lse = lse; a.status = status;
    return done(launch_token_nll(a, workspace, stream));
}

int semicrf_token_nll_grad(const float* grad_loss, const void* x, const void* table, int dtype,
                           const void* targets, int target_bits, const int32_t* lengths,
                           const float* lse, int B, int T, int V, int N, float scale,
                           hipStream_t stream, void* workspace, size_t workspace_bytes,
                           void* grad_x, void* grad_table, int32_t* status) {
    int rc = check_nll(x, table, targets, target_bits, dtype, B, T, V, N, scale);
    if (rc) return rc;
    if (!grad_loss || !lse || (!grad_x && !grad_table)) return SEMICRF_ERR_INVALID;
    if ((rc = check_ws(workspace, workspace_bytes, token_nll_bytes(dtype, B, T, V, N, table, true)))) return rc;
    NllArgs a{};
    a.x = x; a.table = table; a.targets = targets; a.target_bits = target_bits; a.lengths = lengths;
    a.grad_loss = grad_loss; a.lse_in = lse;
    a.dtype = dtype; a.B = B; a.T = T; a.V = V; a.N = N; a.scale = scale;
    a.grad_x = grad_x; a.grad_table = grad_table; a.status = status;
    return done(launch_token_nll_grad(a, workspace, stream));
}

}  // extern "C"
