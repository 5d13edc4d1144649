// ks_preference.hip -- log probabilities of labelled tokens, the paired
// preference loss on them, and its gradient with respect to the logits.
//
//   l = x[label] - log sum_v exp x[v]          for each unmasked row
//   R[s] = beta sum_t (l - ref),  z_i = R[i] - R[P + i]
//   loss = mean (1-e) log(1 + exp(-z)) + e log(1 + exp(z))
//   dx[v] = c[s] (1[v = label] - exp(x[v] - max) / sum)
//
// A row of logits is 8 KB to 200 KB and everything else is small, so the work
// is one stream over the logits for l and a second one for dx: the gradient's
// factor c[s] depends on every row of both sequences of a pair, so no row can
// be finished in the first stream. The second stream takes the rows in the
// opposite order and finds those read last in the 256 MB last cache. (Ranges of
// pairs small enough for that cache, one after another, were slower: a launch
// of 1024 rows of 100 KB reached 3.8 TB/s where one of 8192 reaches 5.4.)
//
// One workgroup a row. The maximum and the sum of exponentials are kept
// together in one pass: each lane keeps its own running pair (m, s), rescales
// s when m grows, and the lanes' pairs are joined at the end. Rows start at
// any element (an odd vocabulary in bf16 puts them at any even byte), so a
// row's head up to the next 128-byte line and its tail go element-wise, one
// value a thread, and the rest in 16-byte vectors that fill whole lines.
//
// exp(x - m) is exp2((x - m) log2 e): the difference is taken first, so that a
// maximum at the type's lowest value (a fully masked vocabulary) cannot
// overflow. The logarithm and l are settled in double, once a row.

#include <algorithm>

#include "ks_device.h"
#include "ks_train.h"

namespace ks {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxRows = int64_t(1) << 23;   // workgroups a launch: a grid counts its threads in 32 bits
constexpr int kWaves = kThreads / 64;
// log2 e in two parts: the fp32 value alone is 1.3e-8 too small, which a sum of
// terms near exp(-6) shows as 8e-8, the same way in every row
constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.92596299e-8f;
constexpr float kLowest = -3.402823466e38f;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));   // elements in 16 bytes

template <typename T>
__device__ __forceinline__ void widen(u32x4 w, float (&x)[kVec<T>]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            x[i] = __uint_as_float(w[i]);
        } else {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}

template <typename T>
__device__ __forceinline__ T narrow(float x) {
    if constexpr (sizeof(T) == 4) return x;
    else return to_bf16(x);
}

template <typename T>
__device__ __forceinline__ u32x4 pack(const float (&x)[kVec<T>]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x[i]);
        else w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    }
    return w;
}

// Elements before the first 128-byte line that starts at or after p, at most n.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int n) {
    const int bytes = static_cast<int>((128 - reinterpret_cast<uintptr_t>(p) % 128) % 128);
    return min(n, bytes / static_cast<int>(sizeof(T)));
}

__device__ __forceinline__ float exp_of(float d) {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(d, kLog2e, d * kLog2eLow));
}

// Joins (m2, s2) to (m, s).
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    s = s * exp_of(m - top) + s2 * exp_of(m2 - top);
    m = top;
}

// KEEP: a gradient may follow and read these logits again; else they go past the
// last cache (16 x 512 rows of 32000 in bf16: 74 us, 80 through it).
template <typename T, bool KEEP>
__global__ __launch_bounds__(kThreads) void token_logp_kernel(const ks_logits_t x_, int64_t row0, float* tokens, float* stats) {
    __shared__ float wave_m[kWaves], wave_s[kWaves];
    constexpr int E = kVec<T>;
    const int64_t at = row0 + blockIdx.x, s_ = at / x_.tokens, t_ = at - s_ * x_.tokens;
    const int64_t label = x_.labels[s_ * x_.label_stride + t_];
    if (label < 0) {
        if (threadIdx.x == 0) {
            tokens[at] = 0.0f;
            if (stats) {
                stats[2 * at] = 0.0f;
                stats[2 * at + 1] = 1.0f;
            }
        }
        return;
    }
    const T* row = static_cast<const T*>(x_.data) + s_ * x_.seq_stride + t_ * x_.row_stride;
    const int V = static_cast<int>(x_.vocab);
    const int head = head_of(row, V);
    const int vecs = (V - head) / E;
    const int tail = head + vecs * E;
    const u32x4* body = reinterpret_cast<const u32x4*>(row + head);
    // the maximum starts at the lowest finite value: a row of -inf then sums to
    // 0 instead of computing inf - inf on the way
    float m = kLowest, s = 0.0f;
    const int tid = threadIdx.x;
    if (tid < head) {
        const float x = to_f32(row[tid]);
        join(m, s, fmaxf(x, kLowest), exp_of(x - fmaxf(x, kLowest)));
    }
    if (tid < V - tail) {
        const float x = to_f32(row[tail + tid]);
        join(m, s, fmaxf(x, kLowest), exp_of(x - fmaxf(x, kLowest)));
    }
    constexpr int U = 4;    // vectors in flight a lane
    int v = tid;
    for (; v + (U - 1) * kThreads < vecs; v += U * kThreads) {
        u32x4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            w[u] = KEEP ? body[v + u * kThreads] : __builtin_nontemporal_load(&body[v + u * kThreads]);
        float x[U][E], top = m;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            widen<T>(w[u], x[u]);
#pragma unroll
            for (int i = 0; i < E; ++i) top = fmaxf(top, x[u][i]);
        }
        s *= exp_of(m - top);
        m = top;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float part = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) part += exp_of(x[u][i] - m);
            s += part;
        }
    }
    for (; v < vecs; v += kThreads) {
        float x[E], top = m;
        widen<T>(body[v], x);
#pragma unroll
        for (int i = 0; i < E; ++i) top = fmaxf(top, x[i]);
        s *= exp_of(m - top);
        m = top;
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) part += exp_of(x[i] - m);
        s += part;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const float m2 = __shfl_xor(m, d, 64), s2 = __shfl_xor(s, d, 64);
        join(m, s, m2, s2);
    }
    if (tid % 64 == 0) {
        wave_m[tid / 64] = m;
        wave_s[tid / 64] = s;
    }
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < kWaves; ++w) join(m, s, wave_m[w], wave_s[w]);
        const float x = label < x_.vocab ? to_f32(row[label]) : __builtin_nanf("");
        tokens[at] = static_cast<float>((static_cast<double>(x) - static_cast<double>(m)) -
                                        log(static_cast<double>(s)));
        if (stats) {
            stats[2 * at] = m;
            stats[2 * at + 1] = s;
        }
    }
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
    return x;
}

// total[s] = sum_t tokens: one wave a sequence.
__global__ __launch_bounds__(kThreads) void sequence_sum_kernel(const float* tokens, int64_t T, int64_t s0, int64_t S,
                                                               float* total) {
    const int64_t s = s0 + static_cast<int64_t>(blockIdx.x) * kWaves + threadIdx.x / 64;
    if (s >= S) return;
    double x = 0.0;
    for (int64_t t = threadIdx.x % 64; t < T; t += 64) x += static_cast<double>(tokens[s * T + t]);
    x = wave_sum(x);
    if (threadIdx.x % 64 == 0) total[s] = static_cast<float>(x);
}

// Rewards, the loss and the gradient's factors. One workgroup, a wave a
// sequence at a time and eight tokens a lane in flight: a few thousand values
// beside megabytes of logits (4 us at 16 x 512 tokens).
__global__ __launch_bounds__(1024) void pair_loss_kernel(const ks_logits_t x, const float* tokens, const float* ref,
                                                         int64_t ref_stride, float beta, float smoothing, float* loss,
                                                         float* rewards, float* grad) {
    __shared__ double sums[16];
    const int64_t S = x.sequences, P = S / 2, T = x.tokens;
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    constexpr int U = 8;
    for (int64_t s = wave; s < S; s += 16) {
        const int64_t* labels = x.labels + s * x.label_stride;
        const float* l = tokens + s * T;
        const float* r = ref + s * ref_stride;
        double sum = 0.0;
        for (int64_t t0 = 0; t0 < T; t0 += 64 * U) {
            int64_t label[U];
            float a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t t = t0 + 64 * u + lane, in = t < T ? t : 0;
                label[u] = t < T ? labels[in] : -1;
                a[u] = l[in];
                b[u] = r[in];
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (label[u] >= 0) sum += static_cast<double>(a[u]) - static_cast<double>(b[u]);
        }
        sum = wave_sum(sum);
        if (lane == 0) rewards[s] = static_cast<float>(static_cast<double>(beta) * sum);
    }
    __syncthreads();
    double sum = 0.0;
    for (int64_t p = threadIdx.x; p < P; p += 1024) {
        const double z = static_cast<double>(rewards[p]) - static_cast<double>(rewards[p + P]), e = smoothing;
        // exp(-|z|) gives both sigmoids and both logarithms without overflow
        const double d = exp(-fabs(z)), near = 1.0 / (1.0 + d), far = d / (1.0 + d), more = log1p(d);
        const double up = z >= 0.0 ? near : far, un = z >= 0.0 ? far : near;
        // a side of weight 0 is left out: its logarithm may be infinite
        if (e < 1.0) sum += (1.0 - e) * (more + fmax(-z, 0.0));
        if (e > 0.0) sum += e * (more + fmax(z, 0.0));
        const double c = static_cast<double>(beta) * (e * up - (1.0 - e) * un) / static_cast<double>(P);
        grad[p] = static_cast<float>(c);
        grad[p + P] = static_cast<float>(-c);
    }
    sum = wave_sum(sum);
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double total = 0.0;
        for (int w = 0; w < 16; ++w) total += sums[w];
        *loss = P > 0 ? static_cast<float>(total / static_cast<double>(P)) : 0.0f;
    }
}

// dx of one row, stored past the last cache: it leaves that to the logits still
// to come (8192 x 50257 in bf16: 370 us a call, 402 with ordinary stores). The
// output row may start at another place of a 16-byte
// granule than the input row: then it goes element-wise.
template <typename T>
__global__ __launch_bounds__(kThreads) void logit_grad_kernel(const ks_logits_t x_, int64_t row0, const float* stats, const float* grad,
                                                              const float* upstream, T* d, int64_t d_seq,
                                                              int64_t d_row) {
    constexpr int E = kVec<T>;
    // the rows that the first stream read last come first: the last cache still
    // holds some 200 MB of them
    const int64_t at = row0 + gridDim.x - 1 - blockIdx.x, s_ = at / x_.tokens, t_ = at - s_ * x_.tokens;
    const int64_t label = x_.labels[s_ * x_.label_stride + t_];
    const T* row = static_cast<const T*>(x_.data) + s_ * x_.seq_stride + t_ * x_.row_stride;
    T* out = d + s_ * d_seq + t_ * d_row;
    const int V = static_cast<int>(x_.vocab);
    const int head = head_of(out, V);
    const int vecs = (V - head) / E;
    const int tail = head + vecs * E;
    u32x4* obody = reinterpret_cast<u32x4*>(out + head);
    const int tid = threadIdx.x;
    if (label < 0) {
        if (tid < head) out[tid] = narrow<T>(0.0f);
        if (tid < V - tail) out[tail + tid] = narrow<T>(0.0f);
        const u32x4 none = {0u, 0u, 0u, 0u};
        for (int v = tid; v < vecs; v += kThreads) __builtin_nontemporal_store(none, &obody[v]);
        return;
    }
    const float m = stats[2 * at];
    float c = grad[s_];
    if (upstream) c *= *upstream;
    const float scale = -c / stats[2 * at + 1];
    // a label outside the vocabulary has no place to go: the whole row says so
    const float c_label = label < x_.vocab ? c : __builtin_nanf("");
    const int place = label < x_.vocab ? static_cast<int>(label) : 0;
    auto one = [&](int v) {
        float y = scale * exp_of(to_f32(row[v]) - m);
        if (v == place) y += c_label;
        out[v] = narrow<T>(y);
    };
    if (tid < head) one(tid);
    if (tid < V - tail) one(tail + tid);
    if (head_of(row, V) != head) {
        for (int v = head + tid; v < tail; v += kThreads) one(v);
        return;
    }
    const u32x4* body = reinterpret_cast<const u32x4*>(row + head);
    auto vec = [&](int v, u32x4 w) {
        float x[E];
        widen<T>(w, x);
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = scale * exp_of(x[i] - m);
        const int in = place - head - v * E;
        if (in >= 0 && in < E) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (i == in) x[i] += c_label;
        }
        __builtin_nontemporal_store(pack<T>(x), &obody[v]);
    };
    constexpr int U = 4;
    int v = tid;
    for (; v + (U - 1) * kThreads < vecs; v += U * kThreads) {
        u32x4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = body[v + u * kThreads];
#pragma unroll
        for (int u = 0; u < U; ++u) vec(v + u * kThreads, w[u]);
    }
    for (; v < vecs; v += kThreads) vec(v, body[v]);
}

}  // namespace

ks_status_t launch_token_logp(const ks_logits_t& x, float* tokens, float* stats, hipStream_t stream) {
    void (*kernel)(ks_logits_t, int64_t, float*, float*);
    if (x.elem == KS_ELEM_BF16) kernel = stats ? token_logp_kernel<bf16_t, true> : token_logp_kernel<bf16_t, false>;
    else kernel = stats ? token_logp_kernel<float, true> : token_logp_kernel<float, false>;
    const int64_t rows = x.sequences * x.tokens;
    for (int64_t r = 0; r < rows; r += kMaxRows) {
        const ks_status_t st = launch_kernel(kernel, dim3(static_cast<unsigned>(std::min(kMaxRows, rows - r))),
                                             dim3(kThreads), 0, stream, x, r, tokens, stats);
        if (st != KS_OK) return st;
    }
    return KS_OK;
}

ks_status_t launch_sequence_sum(const ks_logits_t& x, const float* tokens, float* total, hipStream_t stream) {
    for (int64_t s = 0; s < x.sequences; s += kMaxRows * kWaves) {
        const int64_t groups = std::min(kMaxRows, (x.sequences - s + kWaves - 1) / kWaves);
        const ks_status_t st = launch_kernel(sequence_sum_kernel, dim3(static_cast<unsigned>(groups)), dim3(kThreads), 0,
                                             stream, tokens, x.tokens, s, x.sequences, total);
        if (st != KS_OK) return st;
    }
    return KS_OK;
}

ks_status_t launch_pair_loss(const ks_logits_t& x, const float* tokens, const float* ref, int64_t ref_stride,
                             float beta, float smoothing, float* loss, float* rewards, float* grad,
                             hipStream_t stream) {
    return launch_kernel(pair_loss_kernel, dim3(1), dim3(1024), 0, stream, x, tokens, ref, ref_stride, beta, smoothing,
                         loss, rewards, grad);
}

ks_status_t launch_logit_grad(const ks_logits_t& x, const float* stats, const float* grad, const float* upstream,
                              void* d, int64_t d_seq, int64_t d_row, hipStream_t stream) {
    const int64_t rows = x.sequences * x.tokens;
    for (int64_t end = rows; end > 0; end -= std::min(kMaxRows, end)) {
        const int64_t n = std::min(kMaxRows, end);
        const dim3 grid(static_cast<unsigned>(n));
        const ks_status_t st =
            x.elem == KS_ELEM_BF16
                ? launch_kernel(logit_grad_kernel<bf16_t>, grid, dim3(kThreads), 0, stream, x, end - n, stats, grad,
                                upstream, static_cast<bf16_t*>(d), d_seq, d_row)
                : launch_kernel(logit_grad_kernel<float>, grid, dim3(kThreads), 0, stream, x, end - n, stats, grad,
                                upstream, static_cast<float*>(d), d_seq, d_row);
        if (st != KS_OK) return st;
    }
    return KS_OK;
}

}  // namespace ks
