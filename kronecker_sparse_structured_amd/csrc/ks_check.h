// ks_check.h -- argument checks shared by the C entry points of the operators
// around the product. Host code only, no HIP call but the device query.
#pragma once

#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <vector>

#include "ks_internal.h"

namespace ks {

constexpr int64_t kLimit = int64_t(1) << 31;

// The integer a C caller passed for an enum parameter (any int is allowed
// there in C; loading it as the enum type would be undefined).
template <typename E>
inline int enum_value(const E* e) {
    static_assert(sizeof(E) == sizeof(int), "C enums are int-sized");
    int v;
    std::memcpy(&v, e, sizeof v);
    return v;
}

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Half-open byte ranges [p, p + pb) and [q, q + qb) intersect.
inline bool overlap(const void* p, uint64_t pb, const void* q, uint64_t qb) {
    if (!p || !q || pb == 0 || qb == 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + qb && b < a + pb;
}

struct Range {
    const void* p;
    uint64_t bytes;
};

// Whether range i of `written` meets a later one of it or one of `read`.
inline bool any_overlap(std::initializer_list<Range> written, std::initializer_list<Range> read) {
    for (const Range* w = written.begin(); w != written.end(); ++w) {
        for (const Range* v = w + 1; v != written.end(); ++v)
            if (overlap(w->p, w->bytes, v->p, v->bytes)) return true;
        for (const Range& r : read)
            if (overlap(w->p, w->bytes, r.p, r.bytes)) return true;
    }
    return false;
}

inline size_t round256(uint64_t bytes) { return static_cast<size_t>((bytes + 255) / 256 * 256); }

inline ks_status_t current_cus(int* cus) {
    static std::mutex mu;
    static std::vector<int> cache;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return KS_ERR_HIP;
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= static_cast<int>(cache.size())) cache.resize(dev + 1, 0);
    if (cache[dev] == 0 &&
        (hipDeviceGetAttribute(&cache[dev], hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cache[dev] <= 0)) {
        cache[dev] = 0;
        return KS_ERR_HIP;
    }
    *cus = cache[dev];
    return KS_OK;
}

// ---------------------------------------------------------------- logits

inline ks_status_t check_logits(const ks_logits_t* x) {
    if (!x) return KS_ERR_NULL;
    if (x->elem != KS_ELEM_F32 && x->elem != KS_ELEM_BF16) return KS_ERR_DTYPE;
    if (x->reserved != 0) return KS_ERR_INVALID;
    if (x->sequences < 0 || x->tokens < 0 || x->vocab < 1) return KS_ERR_INVALID;
    if (x->sequences >= kLimit || x->tokens >= kLimit || x->vocab >= kLimit) return KS_ERR_INVALID;
    if (x->sequences * x->tokens >= kLimit) return KS_ERR_INVALID;
    if (x->row_stride < x->vocab || x->label_stride < x->tokens) return KS_ERR_INVALID;
    if (x->row_stride >= kLimit || x->label_stride >= kLimit) return KS_ERR_INVALID;
    if (x->tokens > 0 && x->seq_stride < (x->tokens - 1) * x->row_stride + x->vocab) return KS_ERR_INVALID;
    if (x->seq_stride >= (int64_t(1) << 40)) return KS_ERR_INVALID;
    if (x->sequences > 0 && x->tokens > 0) {
        if (!x->data || !x->labels) return KS_ERR_NULL;
        if (!aligned(x->data, x->elem == KS_ELEM_BF16 ? 2 : 4) || !aligned(x->labels, 8)) return KS_ERR_ALIGN;
    }
    return KS_OK;
}

inline uint64_t span_bytes(int64_t seqs, int64_t seq, int64_t tokens, int64_t row, int64_t width, int size) {
    if (seqs == 0 || tokens == 0) return 0;
    return (static_cast<uint64_t>(seqs - 1) * seq + static_cast<uint64_t>(tokens - 1) * row + width) * size;
}

inline uint64_t logit_bytes(const ks_logits_t* x) {
    return span_bytes(x->sequences, x->seq_stride, x->tokens, x->row_stride, x->vocab,
                      x->elem == KS_ELEM_BF16 ? 2 : 4);
}
inline uint64_t label_bytes(const ks_logits_t* x) {
    return span_bytes(x->sequences, x->label_stride, 1, 0, x->tokens, 8);
}

inline ks_status_t check_dlogits(const ks_logits_t* x, const void* d, int64_t d_seq, int64_t d_row) {
    if (d_row < x->vocab || d_row >= kLimit || d_seq >= (int64_t(1) << 40)) return KS_ERR_INVALID;
    if (x->tokens > 0 && d_seq < (x->tokens - 1) * d_row + x->vocab) return KS_ERR_INVALID;
    if (!aligned(d, x->elem == KS_ELEM_BF16 ? 2 : 4)) return KS_ERR_ALIGN;
    return KS_OK;
}

inline uint64_t dlogit_bytes(const ks_logits_t* x, int64_t d_seq, int64_t d_row) {
    return span_bytes(x->sequences, d_seq, x->tokens, d_row, x->vocab, x->elem == KS_ELEM_BF16 ? 2 : 4);
}

// Logits and their gradient may be the same memory with the same strides.
inline bool in_place(const ks_logits_t* x, const void* d, int64_t d_seq, int64_t d_row) {
    return d == x->data && d_row == x->row_stride && (x->sequences <= 1 || d_seq == x->seq_stride);
}

}  // namespace ks
