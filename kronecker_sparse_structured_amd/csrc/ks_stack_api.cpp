// ks_stack_api.cpp -- the C ABI of the operators between and behind the layers:
// residual norms, distillation, beam search. Validation is pure host code and
// returns before any HIP call, as in ks_api.cpp; see include/ks.h for the
// operations.

#include <algorithm>
#include <cmath>
#include <exception>
#include <vector>

#include "ks_check.h"
#include "ks_stack.h"

using namespace ks;

namespace {

int size_of(int elem) { return elem == KS_ELEM_BF16 ? 2 : 4; }
bool known(int elem) { return elem == KS_ELEM_F32 || elem == KS_ELEM_BF16; }

// ---------------------------------------------------------------- distillation

ks_status_t check_teacher(const ks_logits_t* x, const ks_teacher_t* t) {
    if (!t) return KS_ERR_NULL;
    if (!known(t->elem)) return KS_ERR_DTYPE;
    if (t->reserved != 0 || (t->id_bytes != 4 && t->id_bytes != 8)) return KS_ERR_INVALID;
    if (t->count < 1 || t->count > KS_TEACHER_MAX_COUNT) return KS_ERR_INVALID;
    for (const int64_t* p : {&t->id_seq_stride, &t->top_seq_stride}) {
        const int64_t seq = p[0], row = p[1];
        if (row < t->count || row >= kLimit || seq >= (int64_t(1) << 40)) return KS_ERR_INVALID;
        if (x->tokens > 0 && seq < (x->tokens - 1) * row + t->count) return KS_ERR_INVALID;
    }
    if (x->sequences > 0 && x->tokens > 0) {
        if (!t->ids || !t->top) return KS_ERR_NULL;
        if (!aligned(t->ids, t->id_bytes) || !aligned(t->top, size_of(t->elem))) return KS_ERR_ALIGN;
    }
    return KS_OK;
}

bool valid_options(double weight, double temperature) {
    return weight >= 0.0 && weight <= 1.0 && temperature > 0.0 && std::isfinite(temperature) &&
           std::isfinite(static_cast<float>(1.0 / (temperature * temperature))) &&
           std::isfinite(static_cast<float>(temperature * temperature));
}

Range id_range(const ks_logits_t* x, const ks_teacher_t* t) {
    return {t->ids, span_bytes(x->sequences, t->id_seq_stride, x->tokens, t->id_row_stride, t->count, t->id_bytes)};
}
Range top_range(const ks_logits_t* x, const ks_teacher_t* t) {
    return {t->top,
            span_bytes(x->sequences, t->top_seq_stride, x->tokens, t->top_row_stride, t->count, size_of(t->elem))};
}

// ---------------------------------------------------------------- beams

ks_status_t check_beams(const ks_beams_t* x, int out_beams) {
    if (!x) return KS_ERR_NULL;
    if (!known(x->elem)) return KS_ERR_DTYPE;
    if (x->beams < 1 || x->beams > KS_BEAM_MAX || out_beams < 1 || out_beams > KS_BEAM_MAX) return KS_ERR_INVALID;
    if (x->requests < 0 || x->vocab < 1 || x->vocab >= kLimit || x->beams * x->vocab >= kLimit) return KS_ERR_INVALID;
    if (x->requests >= kLimit || x->requests * std::max<int64_t>(x->beams, out_beams) >= kLimit) return KS_ERR_INVALID;
    if (x->beam_stride < x->vocab || x->beam_stride >= kLimit || x->request_stride >= (int64_t(1) << 40) ||
        x->request_stride < (x->beams - 1) * x->beam_stride + x->vocab)
        return KS_ERR_INVALID;
    if (x->eos >= x->vocab || (x->eos < 0 && x->done)) return KS_ERR_INVALID;
    if (!(x->length_penalty >= 0.0) || !std::isfinite(x->length_penalty)) return KS_ERR_INVALID;
    if (x->length_penalty != 0.0 && !x->lengths && x->requests > 0) return KS_ERR_NULL;
    return KS_OK;
}

// ---------------------------------------------------------------- norms

ks_status_t check_norm(const ks_residual_norm_t* n, int64_t rows, int64_t groups) {
    if (!n) return KS_ERR_NULL;
    if (!known(n->elem) || !known(n->x_elem) || !known(n->y_elem) || !known(n->h_elem) || !known(n->gate_elem))
        return KS_ERR_DTYPE;
    if (n->kind != KS_NORM_RMS && n->kind != KS_NORM_LAYER) return KS_ERR_INVALID;
    if (rows < 0 || rows >= kLimit) return KS_ERR_BATCH;
    if (n->width < 1) return KS_ERR_INVALID;
    if (n->width > KS_NORM_MAX_WIDTH) return KS_ERR_UNSUPPORTED;
    if (!(n->eps > 0.0) || !std::isfinite(n->eps) || !(static_cast<float>(n->eps) > 0.0f) ||
        !std::isfinite(static_cast<float>(n->eps)) || !std::isfinite(static_cast<float>(n->residual)))
        return KS_ERR_INVALID;
    if (groups < 0 || groups >= kLimit || (groups > 0 && rows % groups != 0)) return KS_ERR_INVALID;
    if ((n->pre_bias && !n->pre_weight) || (n->post_bias && !n->post_weight)) return KS_ERR_INVALID;
    for (const void* v : {n->pre_weight, n->pre_bias, n->post_weight, n->post_bias, n->scale})
        if (!aligned(v, size_of(n->elem))) return KS_ERR_ALIGN;
    return KS_OK;
}

}  // namespace

extern "C" {

ks_status_t ks_distil_loss(const ks_logits_t* x, const ks_teacher_t* teacher, double weight, double temperature,
                           float* loss, float* tokens, float* stats, void* dlogits, int64_t d_seq_stride,
                           int64_t d_row_stride, hipStream_t stream) {
    ks_status_t st = check_logits(x);
    if (st == KS_OK) st = check_teacher(x, teacher);
    if (st != KS_OK) return st;
    if (!valid_options(weight, temperature)) return KS_ERR_INVALID;
    const uint64_t rows = static_cast<uint64_t>(x->sequences) * x->tokens;
    if (!loss || !stats || (rows > 0 && !tokens)) return KS_ERR_NULL;
    if (!aligned(loss, 4) || !aligned(tokens, 4) || !aligned(stats, 4)) return KS_ERR_ALIGN;
    if (dlogits) {
        st = check_dlogits(x, dlogits, d_seq_stride, d_row_stride);
        if (st != KS_OK) return st;
    }
    const Range data{x->data, logit_bytes(x)}, labels{x->labels, label_bytes(x)}, ids = id_range(x, teacher),
        top = top_range(x, teacher);
    const Range d{dlogits, dlogits ? dlogit_bytes(x, d_seq_stride, d_row_stride) : 0};
    if (any_overlap({{loss, 4}, {tokens, rows * 4}, {stats, rows * 12 + 4}}, {data, labels, ids, top, d}))
        return KS_ERR_OVERLAP;
    if (any_overlap({d}, {labels, ids, top})) return KS_ERR_OVERLAP;
    if (dlogits && !in_place(x, dlogits, d_seq_stride, d_row_stride) && overlap(d.p, d.bytes, data.p, data.bytes))
        return KS_ERR_OVERLAP;
    const Distil o{weight, temperature};
    float* inv = stats + 3 * rows;
    // the gradient's factor is 1 / N, so that comes first; without one it can come last
    const bool held = rows > 0 && distil_holds(*x, dlogits != nullptr), counted = held && distil_counts(*x);
    if (dlogits && !counted) st = launch_distil_count(*x, inv, stream);
    if (st != KS_OK) return st;
    if (held) {
        st = launch_distil_rows(*x, *teacher, o, tokens, inv, dlogits ? nullptr : stats, dlogits, d_seq_stride,
                                d_row_stride, stream);
    } else {
        st = launch_distil_tokens(*x, *teacher, o, tokens, stats, stream);
        if (st == KS_OK && dlogits)
            st = launch_distil_grad(*x, *teacher, o, stats, inv, nullptr, dlogits, d_seq_stride, d_row_stride, stream);
    }
    return st != KS_OK ? st : launch_distil_sum(*x, tokens, inv, !dlogits && !counted, loss, stream);
}

ks_status_t ks_distil_backward(const ks_logits_t* x, const ks_teacher_t* teacher, double weight, double temperature,
                               const float* stats, const float* upstream, void* dlogits, int64_t d_seq_stride,
                               int64_t d_row_stride, hipStream_t stream) {
    ks_status_t st = check_logits(x);
    if (st == KS_OK) st = check_teacher(x, teacher);
    if (st != KS_OK) return st;
    if (!valid_options(weight, temperature)) return KS_ERR_INVALID;
    const uint64_t rows = static_cast<uint64_t>(x->sequences) * x->tokens;
    if (rows == 0) return KS_OK;
    if (!stats || !dlogits) return KS_ERR_NULL;
    if (!aligned(stats, 4) || !aligned(upstream, 4)) return KS_ERR_ALIGN;
    st = check_dlogits(x, dlogits, d_seq_stride, d_row_stride);
    if (st != KS_OK) return st;
    const Range data{x->data, logit_bytes(x)}, d{dlogits, dlogit_bytes(x, d_seq_stride, d_row_stride)};
    if (any_overlap({d}, {{x->labels, label_bytes(x)}, id_range(x, teacher), top_range(x, teacher),
                          {stats, rows * 12 + 4}, {upstream, 4}}))
        return KS_ERR_OVERLAP;
    if (!in_place(x, dlogits, d_seq_stride, d_row_stride) && overlap(d.p, d.bytes, data.p, data.bytes))
        return KS_ERR_OVERLAP;
    return launch_distil_grad(*x, *teacher, Distil{weight, temperature}, stats, stats + 3 * rows, upstream, dlogits,
                              d_seq_stride, d_row_stride, stream);
}

ks_status_t ks_beam_workspace_size(const ks_beams_t* x, int out_beams, size_t* bytes) {
    if (!bytes) return KS_ERR_NULL;
    const ks_status_t st = check_beams(x, out_beams);
    if (st != KS_OK) return st;
    *bytes = beam_workspace(*x, out_beams);
    return KS_OK;
}

ks_status_t ks_beam_select(const ks_beams_t* x, int out_beams, float* scores, int64_t* tokens, int32_t* parents,
                           uint8_t* done, int32_t* lengths, void* ws, size_t ws_bytes, hipStream_t stream) {
    const ks_status_t st = check_beams(x, out_beams);
    if (st != KS_OK) return st;
    if (x->eos < 0 && done) return KS_ERR_INVALID;
    if (x->requests == 0) return KS_OK;
    if (!x->data || !x->scores || !scores || !tokens || !parents || (x->eos >= 0 && !done)) return KS_ERR_NULL;
    if (!x->lengths != !lengths) return KS_ERR_NULL;
    const size_t need = beam_workspace(*x, out_beams);
    if (!ws || ws_bytes < need) return KS_ERR_WORKSPACE;
    if (!aligned(x->data, size_of(x->elem)) || !aligned(x->scores, 4) || !aligned(x->lengths, 4) || !aligned(scores, 4) ||
        !aligned(tokens, 8) || !aligned(parents, 4) || !aligned(lengths, 4) || !aligned(ws, 16))
        return KS_ERR_ALIGN;
    const uint64_t in = static_cast<uint64_t>(x->requests) * x->beams, out = static_cast<uint64_t>(x->requests) * out_beams;
    const uint64_t data = (static_cast<uint64_t>(x->requests - 1) * x->request_stride +
                           static_cast<uint64_t>(x->beams - 1) * x->beam_stride + x->vocab) * size_of(x->elem);
    if (any_overlap({{scores, out * 4}, {tokens, out * 8}, {parents, out * 4}, {done, out}, {lengths, out * 4}, {ws, need}},
                    {{x->data, data}, {x->scores, in * 4}, {x->done, in}, {x->lengths, in * 4}}))
        return KS_ERR_OVERLAP;
    return launch_beam_select(*x, BeamOut{out_beams, scores, tokens, parents, done, lengths}, ws, stream);
}

ks_status_t ks_beam_reorder(const ks_state_t* states, int n, const int32_t* parents, int64_t requests, int beams,
                            int out_beams, hipStream_t stream) {
    if (n < 0 || requests < 0 || requests >= kLimit || beams < 1 || beams > KS_BEAM_MAX || out_beams < 1 ||
        out_beams > KS_BEAM_MAX || requests * std::max(beams, out_beams) >= kLimit)
        return KS_ERR_INVALID;
    if (n > 0 && !states) return KS_ERR_NULL;
    struct Span {
        uintptr_t from, to;
        bool written;
    };
    std::vector<Span> spans;
    try {
        spans.reserve(2 * static_cast<size_t>(n) + 1);
    } catch (const std::exception&) {      // no exception passes a C entry
        return KS_ERR_INVALID;
    }
    for (int i = 0; i < n; ++i) {
        const ks_state_t& s = states[i];
        if (s.row_bytes < 0 || s.row_bytes >= (int64_t(1) << 40)) return KS_ERR_INVALID;
        if (s.row_bytes == 0 || requests == 0) continue;
        if (!s.src || !s.dst) return KS_ERR_NULL;
        const uintptr_t a = reinterpret_cast<uintptr_t>(s.src), b = reinterpret_cast<uintptr_t>(s.dst);
        spans.push_back({a, a + static_cast<uint64_t>(requests) * beams * s.row_bytes, false});
        spans.push_back({b, b + static_cast<uint64_t>(requests) * out_beams * s.row_bytes, true});
    }
    if (spans.empty()) return KS_OK;
    if (!parents) return KS_ERR_NULL;
    if (!aligned(parents, 4)) return KS_ERR_ALIGN;
    const uintptr_t p = reinterpret_cast<uintptr_t>(parents);
    spans.push_back({p, p + static_cast<uint64_t>(requests) * out_beams * 4, false});
    // in order of their starts: a written one may meet nothing, a read one nothing written
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.from < b.from; });
    uintptr_t read = 0, written = 0;
    for (const Span& s : spans) {
        if (s.from < written || (s.written && s.from < read)) return KS_ERR_OVERLAP;
        (s.written ? written : read) = std::max(s.written ? written : read, s.to);
    }
    return launch_beam_reorder(states, n, parents, requests, beams, out_beams, stream);
}

ks_status_t ks_residual_norm(const ks_residual_norm_t* n, const void* x, const void* y, const void* gate,
                             int64_t groups, void* z, void* h, float* stats, int64_t rows, hipStream_t stream) {
    const ks_status_t st = check_norm(n, rows, groups);
    if (st != KS_OK) return st;
    if ((groups > 0) != (gate != nullptr) || (!y && (gate || z)) || (n->pre_weight == nullptr) != (h == nullptr))
        return rows == 0 ? KS_OK : KS_ERR_INVALID;
    if (rows == 0) return KS_OK;
    if (!x || (y && !z) || (!y && !h)) return KS_ERR_NULL;
    const int xs = size_of(n->x_elem), ys = size_of(n->y_elem), hs = size_of(n->h_elem), gs = size_of(n->gate_elem);
    if (!aligned(x, xs) || !aligned(z, xs) || !aligned(y, ys) || !aligned(h, hs) || !aligned(gate, gs) ||
        !aligned(stats, 16))
        return KS_ERR_ALIGN;
    const uint64_t values = static_cast<uint64_t>(rows) * n->width, w = static_cast<uint64_t>(n->width) * size_of(n->elem);
    const Range rx{x, values * xs}, rz{z, values * xs};
    if (any_overlap({rz, {h, values * hs}, {stats, static_cast<uint64_t>(rows) * 16}},
                    {z == x ? Range{nullptr, 0} : rx, {y, values * ys},
                     {gate, static_cast<uint64_t>(groups) * n->width * gs}, {n->pre_weight, w}, {n->pre_bias, w},
                     {n->post_weight, w}, {n->post_bias, w}, {n->scale, w}}) ||
        any_overlap({{h, values * hs}, {stats, static_cast<uint64_t>(rows) * 16}}, {rx}))
        return KS_ERR_OVERLAP;
    return launch_norm(*n, x, y, gate, groups, z, h, stats, rows, stream);
}

ks_status_t ks_residual_norm_backward_workspace_size(const ks_residual_norm_t* n, int64_t rows, int64_t groups,
                                                     size_t* bytes) {
    if (!bytes) return KS_ERR_NULL;
    const ks_status_t st = check_norm(n, rows, groups);
    if (st != KS_OK) return st;
    *bytes = norm_workspace(*n, norm_split(n->width, rows, groups), rows, groups);
    return KS_OK;
}

ks_status_t ks_residual_norm_backward(const ks_residual_norm_t* n, const void* dz, const void* dh, const void* x,
                                      const void* y, const void* gate, int64_t groups, const float* stats, void* dx,
                                      void* dy, const ks_residual_norm_grads_t* g, void* dgate, int64_t rows, void* ws,
                                      size_t ws_bytes, hipStream_t stream) {
    const ks_status_t st = check_norm(n, rows, groups);
    if (st != KS_OK) return st;
    const ks_residual_norm_grads_t none{};
    if (!g) g = &none;
    if ((g->pre_weight && !n->pre_weight) || (g->pre_bias && !n->pre_bias) || (g->post_weight && !n->post_weight) ||
        (g->post_bias && !n->post_bias) || (g->scale && !n->scale) || (dgate && groups == 0) || (dh && !n->pre_weight))
        return KS_ERR_INVALID;
    const bool normed = n->pre_weight || n->post_weight;
    if (rows > 0) {
        if ((groups > 0) != (gate != nullptr) || (y == nullptr) != (dy == nullptr) || (!y && gate)) return KS_ERR_INVALID;
        if (!x || !dx || (normed && !stats)) return KS_ERR_NULL;
    }
    const NormSplit split = norm_split(n->width, rows, groups);
    const size_t need = norm_workspace(*n, split, rows, groups);
    if (need > 0 && (!ws || ws_bytes < need)) return KS_ERR_WORKSPACE;
    const int xs = size_of(n->x_elem), ys = size_of(n->y_elem), hs = size_of(n->h_elem), gs = size_of(n->gate_elem);
    if (!aligned(x, xs) || !aligned(dz, xs) || !aligned(dx, xs) || !aligned(y, ys) || !aligned(dy, ys) ||
        !aligned(dh, hs) || !aligned(gate, gs) || !aligned(dgate, gs) || !aligned(stats, 16) ||
        (need > 0 && !aligned(ws, 16)))
        return KS_ERR_ALIGN;
    for (const float* p : {g->pre_weight, g->pre_bias, g->post_weight, g->post_bias, g->scale})
        if (!aligned(p, 4)) return KS_ERR_ALIGN;
    const uint64_t values = static_cast<uint64_t>(rows) * n->width, w = static_cast<uint64_t>(n->width) * size_of(n->elem);
    const uint64_t f = static_cast<uint64_t>(n->width) * 4, gates = static_cast<uint64_t>(groups) * n->width * gs;
    if (any_overlap({{dx, values * xs}, {dy, values * ys}, {dgate, gates}, {g->pre_weight, f}, {g->pre_bias, f},
               {g->post_weight, f}, {g->post_bias, f}, {g->scale, f}, {need > 0 ? ws : nullptr, need}},
              {{dz, values * xs}, {dh, values * hs}, {x, values * xs}, {y, values * ys}, {gate, gates},
               {stats, static_cast<uint64_t>(rows) * 16}, {n->pre_weight, w}, {n->pre_bias, w}, {n->post_weight, w},
               {n->post_bias, w}, {n->scale, w}}))
        return KS_ERR_OVERLAP;
    return launch_norm_grad(*n, split, dz, dh, x, y, gate, groups, stats, dx, dy, *g, dgate, rows, ws, stream);
}

}  // extern "C"
