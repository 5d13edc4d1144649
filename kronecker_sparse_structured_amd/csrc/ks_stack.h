// ks_stack.h -- declarations of the operators between and behind the layers:
// residual norms, distillation, beam search (ks_stack_api.cpp validates and
// calls these launchers).
#pragma once

#include "ks_internal.h"

namespace ks {

// Workgroups of 256 threads a launch (a quarter of 1024): a grid counts its threads
// in 32 bits.
constexpr int64_t kMaxGrid = int64_t(1) << 23;

// ---- residual norms (ks_norm.hip)

// How a backward pass cuts its rows: `workers` contiguous ranges of `per`. With a
// gate of several rows a group either `chunks` workers share a group (and their
// parts of its gradient are added up later) or a worker has whole groups.
struct NormSplit {
    int64_t workers, per;
    int64_t group_rows;       // rows that share a gate (0: no gate)
    int chunks;
    int workers_a_group;      // workers a workgroup
    int64_t workgroups;
};
NormSplit norm_split(int64_t width, int64_t rows, int64_t groups);
size_t norm_workspace(const ks_residual_norm_t& n, const NormSplit& s, int64_t rows, int64_t groups);
ks_status_t launch_norm(const ks_residual_norm_t& n, const void* x, const void* y, const void* gate, int64_t groups,
                        void* z, void* h, float* stats, int64_t rows, hipStream_t stream);
ks_status_t launch_norm_grad(const ks_residual_norm_t& n, const NormSplit& s, const void* dz, const void* dh,
                             const void* x, const void* y, const void* gate, int64_t groups, const float* stats,
                             void* dx, void* dy, const ks_residual_norm_grads_t& g, void* dgate, int64_t rows, void* ws,
                             hipStream_t stream);

// ---- distillation (ks_distil.hip)

struct Distil {
    double weight, temperature;
};
// inv: 1 / (unmasked rows).
ks_status_t launch_distil_count(const ks_logits_t& x, float* inv, hipStream_t stream);
// Loss and gradient at once (d null: tokens and stats), of rows that a workgroup
// holds; of few rows the launch counts them as well.
bool distil_holds(const ks_logits_t& x, bool gradient);
bool distil_counts(const ks_logits_t& x);
ks_status_t launch_distil_rows(const ks_logits_t& x, const ks_teacher_t& t, const Distil& o, float* tokens, float* inv,
                               float* stats, void* d, int64_t d_seq, int64_t d_row, hipStream_t stream);
// Of longer rows, in two launches.
ks_status_t launch_distil_tokens(const ks_logits_t& x, const ks_teacher_t& t, const Distil& o, float* tokens,
                                 float* stats, hipStream_t stream);
// The loss; count: and inv.
ks_status_t launch_distil_sum(const ks_logits_t& x, const float* tokens, float* inv, bool count, float* loss,
                              hipStream_t stream);
ks_status_t launch_distil_grad(const ks_logits_t& x, const ks_teacher_t& t, const Distil& o, const float* stats,
                               const float* inv, const float* upstream, void* d, int64_t d_seq, int64_t d_row,
                               hipStream_t stream);

// ---- beam search (ks_beam.hip)

struct BeamOut {
    int beams;
    float* scores;
    int64_t* tokens;
    int32_t* parents;
    uint8_t* done;
    int32_t* lengths;
};
size_t beam_workspace(const ks_beams_t& x, int out_beams);
ks_status_t launch_beam_select(const ks_beams_t& x, const BeamOut& out, void* ws, hipStream_t stream);
ks_status_t launch_beam_reorder(const ks_state_t* states, int n, const int32_t* parents, int64_t requests, int beams,
                                int out_beams, hipStream_t stream);

}  // namespace ks
