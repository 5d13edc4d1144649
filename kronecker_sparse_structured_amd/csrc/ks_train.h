// ks_train.h -- shared declarations of the operators around the product:
// adapters, the preference loss and the optimizer step (ks_train_api.cpp
// validates and calls these launchers).
#pragma once

#include "ks_internal.h"

namespace ks {

// ---- adapters (ks_adapter.hip, ks_adapter_grad.hip)

struct AdapterCall {
    const void* A;
    const void* B;
    const float* scale;
    const int32_t* ids;
    int n_in, n_out, rank, count;
    int xt, wt;              // ElemType of X and of A and B
    int64_t batch;
    hipStream_t stream;
    int num_cus;
};

// Whether a batch runs as one launch (launch_adapter_rows, H optional) or as
// the two products, H = X A^T and Y += H B^T.
bool adapter_one_launch(int64_t batch);
ks_status_t launch_adapter_rows(const AdapterCall& c, const void* X, float* Y, float* H);
ks_status_t launch_adapter_down(const AdapterCall& c, const void* X, float* H);
ks_status_t launch_adapter_up(const AdapterCall& c, const float* H, float* Y);

size_t adapter_grad_workspace(int n_in, int n_out, int rank, int count, int64_t batch);
ks_status_t launch_adapter_grad(const AdapterCall& c, const float* dY, const void* X, const float* H, float* dX,
                                float* dA, float* dB, void* ws);

// ---- preference loss (ks_preference.hip)

struct LogitsCall {
    ks_logits_t x;
    hipStream_t stream;
};

// Rows of sequences [s0, s0 + n) and, if pairs > 0, of [s0 + half, s0 + half + n).
ks_status_t launch_token_logp(const LogitsCall& c, int64_t s0, int64_t n, int64_t half, float* tokens, float* stats);
ks_status_t launch_sequence_sum(const LogitsCall& c, const float* tokens, float* total);
ks_status_t launch_pair_loss(const LogitsCall& c, int64_t p0, int64_t n, const float* tokens, const float* ref,
                             int64_t ref_stride, float beta, float smoothing, float* loss, float* rewards,
                             float* grad);
ks_status_t launch_logit_grad(const LogitsCall& c, int64_t s0, int64_t n, int64_t half, const float* stats,
                              const float* grad, const float* upstream, void* d, int64_t d_seq, int64_t d_row);

// ---- optimizer (ks_adamw.hip)

size_t grad_norm_workspace(const ks_adamw_tensor_t* t, int n);
ks_status_t launch_grad_norm(const ks_adamw_tensor_t* t, int n, float* norm, void* ws, hipStream_t stream);
ks_status_t launch_adamw(const ks_adamw_tensor_t* t, int n, const ks_adamw_options_t& o, const float* norm,
                         hipStream_t stream);
ks_status_t launch_adamw_values(const ks_adamw_tensor_t* t, int n, float* const* m, float* const* v,
                                hipStream_t stream);

}  // namespace ks
