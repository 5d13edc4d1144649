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

// One row of logits a workgroup (none: nothing is launched); the pair loss is
// one workgroup.
ks_status_t launch_token_logp(const ks_logits_t& x, float* tokens, float* stats, hipStream_t stream);
ks_status_t launch_sequence_sum(const ks_logits_t& x, const float* tokens, float* total, hipStream_t stream);
ks_status_t launch_pair_loss(const ks_logits_t& x, const float* tokens, const float* ref, int64_t ref_stride,
                             float beta, float smoothing, float* loss, float* rewards, float* grad,
                             hipStream_t stream);
ks_status_t launch_logit_grad(const ks_logits_t& x, const float* stats, const float* grad, const float* upstream,
                              void* d, int64_t d_seq, int64_t d_row, hipStream_t stream);

// ---- optimizer (ks_adamw.hip)

size_t grad_norm_workspace(const ks_adamw_tensor_t* t, int n);
ks_status_t launch_grad_norm(const ks_adamw_tensor_t* t, int n, float* norm, void* ws, hipStream_t stream);
ks_status_t launch_adamw(const ks_adamw_tensor_t* t, int n, const ks_adamw_options_t& o, const float* norm,
                         hipStream_t stream);
ks_status_t launch_adamw_values(const ks_adamw_tensor_t* t, int n, float* const* m, float* const* v,
                                hipStream_t stream);

}  // namespace ks
