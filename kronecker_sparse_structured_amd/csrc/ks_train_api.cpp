// ks_train_api.cpp -- the C ABI of the operators around the product: adapters
// beside a projection, the preference loss, the optimizer step. Validation is
// pure host code and returns before any HIP call, as in ks_api.cpp; see
// include/ks.h for the operations.

#include <algorithm>
#include <cmath>
#include <vector>

#include "ks_check.h"
#include "ks_train.h"

using namespace ks;

namespace {

// ---------------------------------------------------------------- adapters

ks_status_t adapter_types(int dt, int* xt, int* wt) {
    switch (dt) {
        case KS_DTYPE_F32: *xt = ks::kF32; *wt = ks::kF32; return KS_OK;
        case KS_DTYPE_BF16: *xt = ks::kBF16; *wt = ks::kBF16; return KS_OK;
        case KS_DTYPE_BF16W: *xt = ks::kF32; *wt = ks::kBF16; return KS_OK;
        default: return KS_ERR_DTYPE;
    }
}

ks_status_t check_adapters(const ks_adapters_t* ad, int64_t batch) {
    if (!ad) return KS_ERR_NULL;
    if (batch < 0 || batch >= kLimit) return KS_ERR_BATCH;
    if (ad->rank < 1 || ad->rank > KS_ADAPTER_MAX_RANK || ad->count < 1 || ad->count > KS_ADAPTER_MAX_COUNT)
        return KS_ERR_INVALID;
    if (ad->n_in < 1 || ad->n_out < 1 || ad->n_in >= kLimit || ad->n_out >= kLimit) return KS_ERR_INVALID;
    if (ad->rank * ad->n_in >= kLimit || ad->rank * ad->n_out >= kLimit) return KS_ERR_INVALID;
    if (ad->count * ad->rank * ad->n_in >= kLimit || ad->count * ad->rank * ad->n_out >= kLimit) return KS_ERR_INVALID;
    if (batch * ad->rank >= kLimit) return KS_ERR_INVALID;
    return KS_OK;
}

uint64_t a_bytes(const ks_adapters_t* ad, int wt) {
    return static_cast<uint64_t>(ad->count) * ad->rank * ad->n_in * ks::elem_bytes(wt);
}
uint64_t b_bytes(const ks_adapters_t* ad, int wt) {
    return static_cast<uint64_t>(ad->count) * ad->rank * ad->n_out * ks::elem_bytes(wt);
}

ks::AdapterCall adapter_call(const ks_adapters_t* ad, const int32_t* ids, int xt, int wt, int64_t batch,
                             hipStream_t stream, int cus) {
    ks::AdapterCall c;
    c.A = ad->A; c.B = ad->B; c.scale = ad->scale; c.ids = ids;
    c.n_in = static_cast<int>(ad->n_in); c.n_out = static_cast<int>(ad->n_out);
    c.rank = ad->rank; c.count = ad->count;
    c.xt = xt; c.wt = wt; c.batch = batch; c.stream = stream; c.num_cus = cus;
    return c;
}

// Pointers of the adapters and of a forward call (batch > 0), and its
// workspace.
ks_status_t check_forward(const ks_adapters_t* ad, const int32_t* ids, const void* X, const float* Y, const float* H,
                          int64_t batch, int xt, int wt, const void* ws, size_t ws_bytes, size_t need) {
    if (!ad->A || !ad->B || !ad->scale || !ids || !X || !Y) return KS_ERR_NULL;
    if (need > 0 && (!ws || ws_bytes < need)) return KS_ERR_WORKSPACE;
    if (!aligned(ad->A, ks::elem_bytes(wt)) || !aligned(ad->B, ks::elem_bytes(wt)) || !aligned(ad->scale, 4) ||
        !aligned(ids, 4) || !aligned(X, ks::elem_bytes(xt)) || !aligned(Y, 4) || !aligned(H, 4) ||
        (need > 0 && !aligned(ws, 16)))
        return KS_ERR_ALIGN;
    const uint64_t n = static_cast<uint64_t>(batch);
    if (any_overlap({{Y, n * ad->n_out * 4}, {H, n * ad->rank * 4}, {need > 0 ? ws : nullptr, need}},
                    {{X, n * ad->n_in * ks::elem_bytes(xt)}, {ids, n * 4}, {ad->A, a_bytes(ad, wt)},
                     {ad->B, b_bytes(ad, wt)}, {ad->scale, static_cast<uint64_t>(ad->count) * 4}}))
        return KS_ERR_OVERLAP;
    return KS_OK;
}

ks_status_t check_backward(const ks_adapters_t* ad, const int32_t* ids, const float* dY, const void* X, const float* H,
                           const float* dX, const float* dA, const float* dB, int64_t batch, int xt, int wt,
                           const void* ws, size_t need) {
    if (!dA != !dB) return KS_ERR_NULL;
    const uint64_t n = static_cast<uint64_t>(batch);
    if (batch > 0) {
        if (!ad->A || !ad->B || !ad->scale || !ids || !dY) return KS_ERR_NULL;
        if (dA && (!X || !H)) return KS_ERR_NULL;
        if (!aligned(ad->A, ks::elem_bytes(wt)) || !aligned(ad->B, ks::elem_bytes(wt)) || !aligned(ad->scale, 4) ||
            !aligned(ids, 4) || !aligned(dY, 4) || !aligned(X, ks::elem_bytes(xt)) || !aligned(H, 4))
            return KS_ERR_ALIGN;
    }
    if (!aligned(dX, 4) || !aligned(dA, 4) || !aligned(dB, 4) || !aligned(ws, 16)) return KS_ERR_ALIGN;
    if (any_overlap({{dX, n * ad->n_in * 4},
                     {dA, static_cast<uint64_t>(ad->count) * ad->rank * ad->n_in * 4},
                     {dB, static_cast<uint64_t>(ad->count) * ad->rank * ad->n_out * 4},
                     {ws, need}},
                    {{X, n * ad->n_in * ks::elem_bytes(xt)}, {H, n * ad->rank * 4}, {dY, n * ad->n_out * 4},
                     {ids, n * 4}, {ad->A, a_bytes(ad, wt)}, {ad->B, b_bytes(ad, wt)},
                     {ad->scale, static_cast<uint64_t>(ad->count) * 4}}))
        return KS_ERR_OVERLAP;
    return KS_OK;
}

// Whether a chain's last launch may add the adapters, and the bytes of H in parts.
// It is for rows whose requests lie together, as those of prompts and of training
// do (1024 -> 4096, rank 16, chain and adapters, against the sorted rows or the
// rows as they lie: 1024 rows 18 us for 33, 2048 rows 22 for 40, 4096 rows 30 for
// 58, 16384 rows 78 for 157; rank 32: 16384 rows 97 for 180). Up to this many rows the batch may as well be the next
// tokens of as many requests in any order, which the other launch has to take (1024
// rows 66 us for 36 sorted, 4096 rows 117 for 61).
constexpr int64_t kLooseRows = 1024;
bool takes_parts(int rank, int64_t batch) { return batch > kLooseRows && rank <= ks::kLowPartsRank; }
uint64_t parts_bytes(int rank, int64_t batch) {
    return round256(static_cast<uint64_t>(batch) * ks::low_parts_bytes(rank));
}

ks_status_t chain_widths(const ks_pattern_t* p, int n, const ks_adapters_t* ad) {
    const int64_t in = static_cast<int64_t>(p[0].a) * p[0].c * p[0].d;
    const int64_t out = static_cast<int64_t>(p[n - 1].a) * p[n - 1].b * p[n - 1].d;
    return in == ad->n_in && out == ad->n_out ? KS_OK : KS_ERR_CHAIN_MISMATCH;
}

// dX = dY W_{n-1} ... W_0 is the chain of the factors in reverse, each with its
// blocks transposed (pattern (a, c, b, d)): it runs as ks_chain_matmul does, with
// its fused launches. dY is fp32, so it runs with the weights' type alone.
struct ChainGrad {
    std::vector<ks_pattern_t> p;     // in application order
    std::vector<size_t> at;          // of each factor's transposed blocks, in application order
    size_t blocks;                   // bytes of all of them
    ks_dtype_t dt;
    int wt;
};

ks_status_t reversed_chain(const ks_pattern_t* p, int n, int64_t batch, int dt, ChainGrad* out) {
    size_t bytes = 0;
    // the chain's own checks of patterns, batch and type
    ks_status_t st = ks_chain_workspace_size(p, n, batch, static_cast<ks_dtype_t>(dt), KS_CHAIN_NO_FUSE, &bytes);
    if (st != KS_OK) return st;
    int xt = 0;
    st = adapter_types(dt, &xt, &out->wt);
    if (st != KS_OK) return st;
    out->dt = out->wt == ks::kBF16 ? KS_DTYPE_BF16W : KS_DTYPE_F32;
    out->blocks = 0;
    for (int k = n - 1; k >= 0; --k) {
        st = ks_matmul_dx_workspace_size(p[k], out->dt, &bytes);
        if (st != KS_OK) return st;
        out->p.push_back({p[k].a, p[k].c, p[k].b, p[k].d});
        out->at.push_back(out->blocks);
        out->blocks += bytes;
    }
    return KS_OK;
}

ks::Shape shape_of(const ks_pattern_t& p) {
    ks::Shape s;
    s.a = p.a; s.b = p.b; s.c = p.c; s.d = p.d;
    s.n_in = static_cast<int64_t>(p.a) * p.c * p.d;
    s.n_out = static_cast<int64_t>(p.a) * p.b * p.d;
    s.nnz = s.n_in * p.b;
    return s;
}

// W's blocks transposed into Wt, in the order of the reversed chain.
ks_status_t transpose_chain(const ks_pattern_t* p, int n, const void* const* W, const ChainGrad& g, char* wt,
                            hipStream_t stream) {
    for (int k = 0; k < n; ++k) {
        const ks_status_t st =
            ks::launch_transpose_blocks(shape_of(p[n - 1 - k]), g.wt, W[n - 1 - k], wt + g.at[k], stream);
        if (st != KS_OK) return st;
    }
    return KS_OK;
}

// Workspace of the chain's part of a backward call: transposed blocks, unless
// the caller has them, then the reversed chain's own.
struct ChainGradWs {
    size_t chain, adapters, total;
};

ks_status_t chain_grad_ws(const ChainGrad& g, const ks_adapters_t* ad, int64_t batch, bool have_blocks,
                          ChainGradWs* out) {
    ks_status_t st = ks_chain_workspace_size(g.p.data(), static_cast<int>(g.p.size()), batch, g.dt, KS_CHAIN_AUTO,
                                             &out->chain);
    if (st != KS_OK) return st;
    st = ks_adapter_backward_workspace_size(ad, batch, &out->adapters);
    if (st != KS_OK) return st;
    // the adapters run after the chain, over the same memory
    out->total = std::max((have_blocks ? 0 : g.blocks) + round256(out->chain), out->adapters);
    return KS_OK;
}

// ---------------------------------------------------------------- optimizer

ks_status_t check_tensors(const ks_adamw_tensor_t* t, int n) {
    if (n < 0) return KS_ERR_INVALID;
    if (n > 0 && !t) return KS_ERR_NULL;
    int64_t total = 0;
    for (int i = 0; i < n; ++i) {
        if (t[i].n < 0 || t[i].n >= kLimit) return KS_ERR_INVALID;
        if (t[i].g_elem != KS_ELEM_F32 && t[i].g_elem != KS_ELEM_BF16) return KS_ERR_DTYPE;
        total += t[i].n;
    }
    return total >= (int64_t(1) << 44) ? KS_ERR_INVALID : KS_OK;
}

int elem_size(int e) { return e == KS_ELEM_BF16 ? 2 : 4; }

// State pointers of an 8- or 32-bit tensor; p and g as well if `step`.
ks_status_t check_states(const ks_adamw_tensor_t& t, int bits, bool step) {
    if (t.n == 0) return KS_OK;
    if (step && (!t.p || !t.g)) return KS_ERR_NULL;
    if (step && t.p_elem != KS_ELEM_F32 && t.p_elem != KS_ELEM_BF16) return KS_ERR_DTYPE;
    if (!t.m || !t.v || (bits == 8 && !t.scales)) return KS_ERR_NULL;
    const int size = bits == 8 ? 1 : 4;
    if (!aligned(t.m, size) || !aligned(t.v, size) || (bits == 8 && !aligned(t.scales, 4))) return KS_ERR_ALIGN;
    if (step && (!aligned(t.p, elem_size(t.p_elem)) || !aligned(t.g, elem_size(t.g_elem)))) return KS_ERR_ALIGN;
    if (!step) return KS_OK;
    const uint64_t n = static_cast<uint64_t>(t.n);
    return any_overlap({{t.p, n * elem_size(t.p_elem)}, {t.m, n * size}, {t.v, n * size},
                        {bits == 8 ? t.scales : nullptr, (n + 255) / 256 * 8}},
                       {{t.g, n * elem_size(t.g_elem)}})
               ? KS_ERR_OVERLAP
               : KS_OK;
}

}  // namespace

extern "C" {

ks_status_t ks_adapter_workspace_size(const ks_adapters_t* ad, int64_t batch, size_t* bytes) {
    if (!bytes) return KS_ERR_NULL;
    const ks_status_t st = check_adapters(ad, batch);
    if (st != KS_OK) return st;
    *bytes = ks::adapter_workspace(batch, ad->count);
    return KS_OK;
}

ks_status_t ks_adapter_matmul(const ks_adapters_t* ad, const int32_t* ids, const void* X, float* Y, float* H,
                              int64_t batch, ks_dtype_t dt, void* ws, size_t ws_bytes, hipStream_t stream) {
    size_t need = 0;
    ks_status_t st = ks_adapter_workspace_size(ad, batch, &need);
    if (st != KS_OK) return st;
    int xt = 0, wt = 0;
    st = adapter_types(enum_value(&dt), &xt, &wt);
    if (st != KS_OK) return st;
    if (batch == 0) return KS_OK;
    if (!H) return KS_ERR_NULL;
    st = check_forward(ad, ids, X, Y, H, batch, xt, wt, ws, ws_bytes, need);
    if (st != KS_OK) return st;
    int cus = 0;
    st = current_cus(&cus);
    if (st != KS_OK) return st;
    return ks::launch_adapter(adapter_call(ad, ids, xt, wt, batch, stream, cus), X, H, Y, ws);
}

ks_status_t ks_adapter_backward_workspace_size(const ks_adapters_t* ad, int64_t batch, size_t* bytes) {
    if (!bytes) return KS_ERR_NULL;
    const ks_status_t st = check_adapters(ad, batch);
    if (st != KS_OK) return st;
    const int n_in = static_cast<int>(ad->n_in), n_out = static_cast<int>(ad->n_out);
    if (!ks::adapter_grad_fits(n_in, n_out, ad->rank, ad->count, batch)) return KS_ERR_UNSUPPORTED;
    *bytes = ks::adapter_grad_workspace(n_in, n_out, ad->rank, ad->count, batch);
    return KS_OK;
}

ks_status_t ks_adapter_backward(const ks_adapters_t* ad, const int32_t* ids, const float* dY, const void* X,
                                const float* H, float* dX, float* dA, float* dB, int64_t batch, ks_dtype_t dt,
                                void* ws, size_t ws_bytes, hipStream_t stream) {
    size_t need = 0;
    ks_status_t st = ks_adapter_backward_workspace_size(ad, batch, &need);
    if (st != KS_OK) return st;
    int xt = 0, wt = 0;
    st = adapter_types(enum_value(&dt), &xt, &wt);
    if (st != KS_OK) return st;
    if (!dA && !dB && (batch == 0 || !dX)) return KS_OK;
    if (need > 0 && (!ws || ws_bytes < need)) return KS_ERR_WORKSPACE;
    st = check_backward(ad, ids, dY, X, H, dX, dA, dB, batch, xt, wt, ws, need);
    if (st != KS_OK) return st;
    int cus = 0;
    st = current_cus(&cus);
    if (st != KS_OK) return st;
    return ks::launch_adapter_grad(adapter_call(ad, ids, xt, wt, batch, stream, cus), dY, X, H, dX, dA, dB, ws);
}

ks_status_t ks_chain_adapter_workspace_size(const ks_pattern_t* p, int n, const ks_adapters_t* ad, int64_t batch,
                                            ks_dtype_t dt, size_t* bytes) {
    if (!bytes) return KS_ERR_NULL;
    size_t need = 0;
    const int code = enum_value(&dt);
    ks_status_t st = ks_chain_workspace_size(p, n, batch, static_cast<ks_dtype_t>(code), KS_CHAIN_AUTO, &need);
    if (st != KS_OK) return st;
    st = check_adapters(ad, batch);
    if (st != KS_OK) return st;
    st = chain_widths(p, n, ad);
    if (st != KS_OK) return st;
    // the adapters' own, H for callers that do not keep it, and what a last launch
    // that adds the adapters reads
    *bytes = round256(need) + round256(ks::adapter_workspace(batch, ad->count)) +
             (ks::adapter_path(batch) == ks::kAdapterRows ? 0 : round256(static_cast<uint64_t>(batch) * ad->rank * 4)) +
             (takes_parts(ad->rank, batch) ? parts_bytes(ad->rank, batch) + round256((static_cast<uint64_t>(batch) + 3) / 4 * 8) : 0);
    return KS_OK;
}

ks_status_t ks_chain_adapter_matmul(const ks_pattern_t* p, int n, const void* const* W, const ks_adapters_t* ad,
                                    const int32_t* ids, const void* X, float* Y, float* H, int64_t batch,
                                    ks_dtype_t dt, void* ws, size_t ws_bytes, hipStream_t stream) {
    size_t need = 0, chain_ws = 0;
    const int code = enum_value(&dt);
    ks_status_t st = ks_chain_adapter_workspace_size(p, n, ad, batch, static_cast<ks_dtype_t>(code), &need);
    if (st != KS_OK) return st;
    int xt = 0, wt = 0;
    st = adapter_types(code, &xt, &wt);
    if (st != KS_OK) return st;
    if (batch == 0) return KS_OK;
    st = check_forward(ad, ids, X, Y, H, batch, xt, wt, ws, ws_bytes, need);
    if (st != KS_OK) return st;
    for (int k = 0; W && k < n; ++k) {
        // the chain's own checks take in Y and its part of the workspace
        const uint64_t bytes = static_cast<uint64_t>(shape_of(p[k]).nnz) * ks::elem_bytes(wt);
        if (any_overlap({{H, static_cast<uint64_t>(batch) * ad->rank * 4}, {need > 0 ? ws : nullptr, need}}, {{W[k], bytes}}))
            return KS_ERR_OVERLAP;
    }
    st = ks_chain_workspace_size(p, n, batch, static_cast<ks_dtype_t>(code), KS_CHAIN_AUTO, &chain_ws);
    if (st != KS_OK) return st;
    char* rest = static_cast<char*>(ws) + round256(chain_ws);
    char* low = rest + round256(ks::adapter_workspace(batch, ad->count));
    if (!H && ks::adapter_path(batch) != ks::kAdapterRows) H = reinterpret_cast<float*>(low);
    char* parts = low + round256(static_cast<uint64_t>(batch) * ad->rank * 4);
    ks::ChainAdapters extra;
    extra.call = adapter_call(ad, ids, xt, wt, batch, stream, 0);
    extra.pair = {parts, reinterpret_cast<ks::PairGroup*>(parts + parts_bytes(ad->rank, batch)), ad->B, ad->rank};
    extra.H = H;
    extra.added = false;
    // the chain's own checks (weights, alignment, overlaps) come first: an
    // argument error launches nothing
    st = ks::chain_matmul(p, n, W, X, Y, batch, code, ws, chain_ws, KS_CHAIN_AUTO, stream,
                          takes_parts(ad->rank, batch) ? &extra : nullptr);
    if (st != KS_OK || extra.added) return st;
    st = current_cus(&extra.call.num_cus);
    if (st != KS_OK) return st;
    return ks::launch_adapter(extra.call, X, H, Y, rest);
}

ks_status_t ks_chain_transpose_size(const ks_pattern_t* p, int n, ks_dtype_t dt, size_t* bytes) {
    if (!bytes) return KS_ERR_NULL;
    ChainGrad g;
    const ks_status_t st = reversed_chain(p, n, 0, enum_value(&dt), &g);
    if (st != KS_OK) return st;
    *bytes = g.blocks;
    return KS_OK;
}

ks_status_t ks_chain_transpose(const ks_pattern_t* p, int n, const void* const* W, void* Wt, ks_dtype_t dt,
                               hipStream_t stream) {
    ChainGrad g;
    const ks_status_t st = reversed_chain(p, n, 0, enum_value(&dt), &g);
    if (st != KS_OK) return st;
    if (!W || !Wt) return KS_ERR_NULL;
    if (!aligned(Wt, 16)) return KS_ERR_ALIGN;
    for (int k = 0; k < n; ++k) {
        if (!W[k]) return KS_ERR_NULL;
        if (!aligned(W[k], ks::elem_bytes(g.wt))) return KS_ERR_ALIGN;
        if (overlap(Wt, g.blocks, W[k], static_cast<uint64_t>(shape_of(p[k]).nnz) * ks::elem_bytes(g.wt)))
            return KS_ERR_OVERLAP;
    }
    return transpose_chain(p, n, W, g, static_cast<char*>(Wt), stream);
}

ks_status_t ks_chain_adapter_backward_workspace_size(const ks_pattern_t* p, int n, const ks_adapters_t* ad,
                                                     int64_t batch, ks_dtype_t dt, int have_transposed,
                                                     size_t* bytes) {
    if (!bytes) return KS_ERR_NULL;
    ChainGrad g;
    ChainGradWs w;
    ks_status_t st = reversed_chain(p, n, batch, enum_value(&dt), &g);
    if (st == KS_OK) st = check_adapters(ad, batch);
    if (st == KS_OK) st = chain_widths(p, n, ad);
    if (st == KS_OK) st = chain_grad_ws(g, ad, batch, have_transposed != 0, &w);
    if (st != KS_OK) return st;
    *bytes = w.total;
    return KS_OK;
}

ks_status_t ks_chain_adapter_backward(const ks_pattern_t* p, int n, const void* const* W, const void* Wt,
                                      const ks_adapters_t* ad, const int32_t* ids, const float* dY, const void* X,
                                      const float* H, float* dX, float* dA, float* dB, int64_t batch, ks_dtype_t dt,
                                      void* ws, size_t ws_bytes, hipStream_t stream) {
    ChainGrad g;
    ChainGradWs w;
    const int code = enum_value(&dt);
    ks_status_t st = reversed_chain(p, n, batch, code, &g);
    if (st == KS_OK) st = check_adapters(ad, batch);
    if (st == KS_OK) st = chain_widths(p, n, ad);
    if (st == KS_OK) st = chain_grad_ws(g, ad, batch, Wt != nullptr, &w);
    if (st != KS_OK) return st;
    int xt = 0, wt = 0;
    st = adapter_types(code, &xt, &wt);
    if (st != KS_OK) return st;
    if (batch > 0 && ((!W && !Wt) || !dX)) return KS_ERR_NULL;
    if (batch == 0 && !dA && !dB) return KS_OK;
    if (w.total > 0 && (!ws || ws_bytes < w.total)) return KS_ERR_WORKSPACE;
    st = check_backward(ad, ids, dY, X, H, dX, dA, dB, batch, xt, wt, ws, w.total);
    if (st != KS_OK) return st;
    if (!aligned(Wt, 16)) return KS_ERR_ALIGN;
    char* base = static_cast<char*>(ws);
    int cus = 0;
    if (batch > 0) {
        const uint64_t dx_bytes = static_cast<uint64_t>(batch) * ad->n_in * 4;
        const uint64_t each = static_cast<uint64_t>(ad->count) * ad->rank * 4;
        const Range da{dA, each * ad->n_in}, db{dB, each * ad->n_out};
        if (Wt && any_overlap({{dX, dx_bytes}, da, db, {ws, w.total}}, {{Wt, g.blocks}})) return KS_ERR_OVERLAP;
        bool have = W != nullptr;                            // every factor as it is
        for (int k = 0; k < n && W; ++k) {
            have = have && W[k];
            if (!W[k] && !Wt) return KS_ERR_NULL;
            if (!W[k]) continue;
            if (!aligned(W[k], ks::elem_bytes(wt))) return KS_ERR_ALIGN;
            const uint64_t bytes = static_cast<uint64_t>(shape_of(p[k]).nnz) * ks::elem_bytes(wt);
            if (any_overlap({{dX, dx_bytes}, da, db, {ws, w.total}}, {{W[k], bytes}})) return KS_ERR_OVERLAP;
        }
        st = current_cus(&cus);
        if (st != KS_OK) return st;
        if (n == 2 && have && ks::pair_dx_supports(shape_of(p[0]), shape_of(p[1]), wt, W[0], W[1], dY)) {
            st = ks::launch_pair_dx(shape_of(p[0]), W[0], W[1], dY, dX, batch, stream, cus);
        } else {
            const char* blocks = static_cast<const char*>(Wt);
            char* chain_ws = base;
            if (!blocks) {
                st = transpose_chain(p, n, W, g, base, stream);
                if (st != KS_OK) return st;
                blocks = base;
                chain_ws = base + g.blocks;
            }
            std::vector<const void*> factors(n);
            for (int k = 0; k < n; ++k) factors[k] = blocks + g.at[k];
            st = ks_chain_matmul(g.p.data(), n, factors.data(), dY, dX, batch, g.dt, chain_ws, w.chain, KS_CHAIN_AUTO,
                                 stream);
        }
        if (st != KS_OK) return st;
    }
    st = current_cus(&cus);
    if (st != KS_OK) return st;
    return ks::launch_adapter_grad(adapter_call(ad, ids, xt, wt, batch, stream, cus), dY, X, H,
                                   batch > 0 ? dX : nullptr, dA, dB, ws);
}

ks_status_t ks_sequence_logp(const ks_logits_t* x, float* tokens, float* total, float* stats, hipStream_t stream) {
    const ks_status_t st = check_logits(x);
    if (st != KS_OK) return st;
    if (x->sequences == 0) return KS_OK;
    const uint64_t rows = static_cast<uint64_t>(x->sequences) * x->tokens;
    if (!total || (rows > 0 && !tokens)) return KS_ERR_NULL;
    if (!aligned(tokens, 4) || !aligned(total, 4) || !aligned(stats, 4)) return KS_ERR_ALIGN;
    if (any_overlap({{tokens, rows * 4}, {total, static_cast<uint64_t>(x->sequences) * 4}, {stats, rows * 8}},
                    {{x->data, logit_bytes(x)}, {x->labels, label_bytes(x)}}))
        return KS_ERR_OVERLAP;
    const ks_status_t run = ks::launch_token_logp(*x, tokens, stats, stream);
    return run != KS_OK ? run : ks::launch_sequence_sum(*x, tokens, total, stream);
}

ks_status_t ks_preference_loss(const ks_logits_t* x, const float* ref, int64_t ref_stride, float beta, float smoothing,
                               float* loss, float* rewards, float* tokens, float* grad, float* stats, void* dlogits,
                               int64_t d_seq_stride, int64_t d_row_stride, hipStream_t stream) {
    ks_status_t st = check_logits(x);
    if (st != KS_OK) return st;
    if (x->sequences % 2 != 0 || ref_stride < x->tokens || ref_stride >= kLimit) return KS_ERR_INVALID;
    if (!(beta > 0.0f) || !std::isfinite(beta) || !(smoothing >= 0.0f) || !(smoothing <= 1.0f)) return KS_ERR_INVALID;
    const uint64_t rows = static_cast<uint64_t>(x->sequences) * x->tokens;
    if (!loss || (x->sequences > 0 && (!rewards || !grad)) || (rows > 0 && (!ref || !tokens || !stats)))
        return KS_ERR_NULL;
    if (!aligned(loss, 4) || !aligned(rewards, 4) || !aligned(grad, 4) || !aligned(ref, 4) || !aligned(tokens, 4) ||
        !aligned(stats, 4))
        return KS_ERR_ALIGN;
    const uint64_t seqs = static_cast<uint64_t>(x->sequences) * 4;
    uint64_t db = 0;
    bool same = false;
    if (dlogits) {
        st = check_dlogits(x, dlogits, d_seq_stride, d_row_stride);
        if (st != KS_OK) return st;
        db = dlogit_bytes(x, d_seq_stride, d_row_stride);
        same = in_place(x, dlogits, d_seq_stride, d_row_stride);
    }
    const Range logits{x->data, logit_bytes(x)};
    const Range none{nullptr, 0};
    if (any_overlap({{loss, 4}, {rewards, seqs}, {grad, seqs}, {tokens, rows * 4}, {stats, rows * 8}, {dlogits, db}},
                    {same ? none : logits, {x->labels, label_bytes(x)},
                     {ref, span_bytes(x->sequences, ref_stride, 1, 0, x->tokens, 4)}}) ||
        any_overlap({{loss, 4}, {rewards, seqs}, {grad, seqs}, {tokens, rows * 4}, {stats, rows * 8}}, {logits}))
        return KS_ERR_OVERLAP;
    st = ks::launch_token_logp(*x, tokens, stats, stream);
    if (st == KS_OK) st = ks::launch_pair_loss(*x, tokens, ref, ref_stride, beta, smoothing, loss, rewards, grad, stream);
    if (st == KS_OK && dlogits)
        st = ks::launch_logit_grad(*x, stats, grad, nullptr, dlogits, d_seq_stride, d_row_stride, stream);
    return st;
}

ks_status_t ks_preference_backward(const ks_logits_t* x, const float* stats, const float* grad, const float* upstream,
                                   void* dlogits, int64_t d_seq_stride, int64_t d_row_stride, hipStream_t stream) {
    ks_status_t st = check_logits(x);
    if (st != KS_OK) return st;
    const uint64_t rows = static_cast<uint64_t>(x->sequences) * x->tokens;
    if (rows == 0) return KS_OK;
    if (!stats || !grad || !dlogits) return KS_ERR_NULL;
    if (!aligned(stats, 4) || !aligned(grad, 4) || !aligned(upstream, 4)) return KS_ERR_ALIGN;
    st = check_dlogits(x, dlogits, d_seq_stride, d_row_stride);
    if (st != KS_OK) return st;
    const Range logits{x->data, logit_bytes(x)};
    const Range none{nullptr, 0};
    if (any_overlap({{dlogits, dlogit_bytes(x, d_seq_stride, d_row_stride)}},
                    {in_place(x, dlogits, d_seq_stride, d_row_stride) ? none : logits, {x->labels, label_bytes(x)},
                     {stats, rows * 8}, {grad, static_cast<uint64_t>(x->sequences) * 4}, {upstream, 4}}))
        return KS_ERR_OVERLAP;
    return ks::launch_logit_grad(*x, stats, grad, upstream, dlogits, d_seq_stride, d_row_stride, stream);
}

ks_status_t ks_grad_norm_workspace_size(const ks_adamw_tensor_t* t, int n, size_t* bytes) {
    if (!bytes) return KS_ERR_NULL;
    const ks_status_t st = check_tensors(t, n);
    if (st != KS_OK) return st;
    *bytes = ks::grad_norm_workspace(t, n);
    return KS_OK;
}

ks_status_t ks_grad_norm(const ks_adamw_tensor_t* t, int n, float* norm, void* ws, size_t ws_bytes,
                         hipStream_t stream) {
    size_t need = 0;
    const ks_status_t st = ks_grad_norm_workspace_size(t, n, &need);
    if (st != KS_OK) return st;
    if (!norm) return KS_ERR_NULL;
    if (need > 0 && (!ws || ws_bytes < need)) return KS_ERR_WORKSPACE;
    if (!aligned(norm, 4) || !aligned(ws, 16)) return KS_ERR_ALIGN;
    if (any_overlap({{norm, 4}, {ws, need}}, {})) return KS_ERR_OVERLAP;
    for (int i = 0; i < n; ++i) {
        if (t[i].n == 0) continue;
        if (!t[i].g) return KS_ERR_NULL;
        if (!aligned(t[i].g, elem_size(t[i].g_elem))) return KS_ERR_ALIGN;
        if (any_overlap({{norm, 4}, {ws, need}}, {{t[i].g, static_cast<uint64_t>(t[i].n) * elem_size(t[i].g_elem)}}))
            return KS_ERR_OVERLAP;
    }
    return ks::launch_grad_norm(t, n, norm, ws, stream);
}

ks_status_t ks_adamw_step(const ks_adamw_tensor_t* t, int n, const ks_adamw_options_t* o, const float* norm,
                          hipStream_t stream) {
    ks_status_t st = check_tensors(t, n);
    if (st != KS_OK) return st;
    if (!o) return KS_ERR_NULL;
    if (o->state_bits != 8 && o->state_bits != 32) return KS_ERR_INVALID;
    if (o->step < 1) return KS_ERR_INVALID;
    if (!(o->beta1 >= 0.0 && o->beta1 < 1.0) || !(o->beta2 >= 0.0 && o->beta2 < 1.0)) return KS_ERR_INVALID;
    if (!(o->eps >= 0.0) || !std::isfinite(o->eps) || !std::isfinite(o->lr) || !std::isfinite(o->weight_decay))
        return KS_ERR_INVALID;
    if (!(o->max_norm >= 0.0) || !std::isfinite(o->max_norm)) return KS_ERR_INVALID;
    if (o->max_norm > 0.0 && !norm) return KS_ERR_NULL;
    if (!aligned(norm, 4)) return KS_ERR_ALIGN;
    for (int i = 0; i < n; ++i) {
        st = check_states(t[i], o->state_bits, true);
        if (st != KS_OK) return st;
    }
    return ks::launch_adamw(t, n, *o, norm, stream);
}

ks_status_t ks_adamw_state_values(const ks_adamw_tensor_t* t, int n, float* const* m_out, float* const* v_out,
                                  hipStream_t stream) {
    ks_status_t st = check_tensors(t, n);
    if (st != KS_OK) return st;
    if (n > 0 && (!m_out || !v_out)) return KS_ERR_NULL;
    for (int i = 0; i < n; ++i) {
        if (t[i].n == 0) continue;
        st = check_states(t[i], 8, false);
        if (st != KS_OK) return st;
        if (!m_out[i] || !v_out[i]) return KS_ERR_NULL;
        if (!aligned(m_out[i], 4) || !aligned(v_out[i], 4)) return KS_ERR_ALIGN;
        const uint64_t k = static_cast<uint64_t>(t[i].n);
        if (any_overlap({{m_out[i], k * 4}, {v_out[i], k * 4}}, {{t[i].m, k}, {t[i].v, k}, {t[i].scales, (k + 255) / 256 * 8}}))
            return KS_ERR_OVERLAP;
    }
    return ks::launch_adamw_values(t, n, m_out, v_out, stream);
}

}  // extern "C"
