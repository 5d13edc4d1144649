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

// Rows by adapter (stable; rows without an adapter left out), cut into blocks
// of `block` rows of one adapter each.
struct AdapterSlot {
    int adapter, start, len, reserved;   // rows order[start .. start + len); len 0: empty
};
struct AdapterSegment {
    int start, len;                      // an adapter's rows in the order
};
struct AdapterOrder {
    int* order;
    AdapterSegment* segs;
    AdapterSlot* slots;
    int block, n_slots;
};
// Blocks of adapter g start at slot floor(start / block) + g: at most one slot
// an adapter is left empty, and no slot is claimed twice.
inline int adapter_slots(int64_t batch, int block, int count) { return static_cast<int>(batch / block) + count; }
// Bytes and layout (from `ws`) of an order for this batch.
size_t adapter_order_layout(int64_t batch, int block, int count, char* ws, AdapterOrder* out);
ks_status_t launch_adapter_order(const AdapterCall& c, const AdapterOrder& o);

// How a batch runs: one launch for few rows (H optional); the two products
// H = X A^T and Y += H B^T over rows sorted by adapter for more; over rows as
// they lie for many.
enum AdapterPath : int { kAdapterRows = 0, kAdapterSorted = 1, kAdapterRuns = 2 };
AdapterPath adapter_path(int64_t batch);
size_t adapter_workspace(int64_t batch, int count);
ks_status_t launch_adapter(const AdapterCall& c, const void* X, float* H, float* Y, void* ws);

// The first product alone, over rows as they lie: H, its values in parts as the
// fused pair takes them, and the adapters of each kPairGroup rows (none where they
// change more than once); then the second product for those groups' rows.
ks_status_t launch_adapter_down(const AdapterCall& c, const void* X, float* H, void* parts, PairGroup* groups);
ks_status_t launch_adapter_rest(const AdapterCall& c, const float* H, float* Y);

// Adapters beside a chain: chain_matmul (ks_chain_matmul with the dtype as an int)
// runs them around its last launch where that is a fused pair that adds them
// (added); the caller runs them otherwise.
struct ChainAdapters {
    AdapterCall call;
    PairAdapters pair;
    float* H;
    bool added;
};
ks_status_t chain_matmul(const ks_pattern_t* p, int n, const void* const* W, const void* X, void* Y, int64_t batch,
                         int dt, void* ws, size_t ws_bytes, unsigned flags, hipStream_t stream, ChainAdapters* extra);

// dX of a pair of factors (1, b0, 16, 64), (b0, 8, 8, 8) with bf16 weights in one
// launch (ks_pair_grad.hip).
bool pair_dx_supports(const Shape& s0, const Shape& s1, int wt, const void* W0, const void* W1, const float* dY);
ks_status_t launch_pair_dx(const Shape& s0, const void* W0, const void* W1, const float* dY, float* dX, int64_t batch,
                           hipStream_t stream, int num_cus);

// fits: whether the launches' grids can hold it.
bool adapter_grad_fits(int n_in, int n_out, int rank, int count, int64_t batch);
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
