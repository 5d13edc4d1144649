// ks_distil.hip -- distillation from a teacher's highest logits, with the
// gradient of the student's.
//
//   q = softmax(top / T) over a row's K entries, p = softmax(x / T), p1 = softmax(x)
//   token = w T^2 sum_k q_k (log q_k - log p[id_k]) - (1 - w) log p1[label]
//   dx_v = (w T (p_v - q_v) + (1 - w) (p1_v - 1[v = label])) / N
//
// A row of logits is 8 KB to 200 KB, its entries at most a few KB: one
// workgroup a row. The factor of a row's gradient is known before any row is, so
// where loss and gradient are asked for together a row is read once and written
// once: a workgroup holds it in registers (up to 256 KB) while its maximum, its
// sums and its entries' part are formed. Longer rows, and a gradient that is
// asked for later, go through the row again; there the maximum and both sums of
// exponentials are kept in one pass, as in ks_preference.hip.
//
// The gradient goes out in two steps: the whole row as if there were no entries, in
// 16-byte nontemporal stores (8192 rows of 50257 in bf16 329 us a call, 333 with ordinary
// ones), and behind a barrier the few values at the entries' and the label's tokens
// again.
//
// What bounds it: the row's read and write. 8192 rows of 50257 in bf16 (1.65 GB)
// with one exponential a value 313 us a call, 5.3 TB/s, a device copy of as much 320;
// with two, 332 (temperature 2) and 367: there the exponentials' arithmetic shows. In
// fp32, 8192 rows of 32000 (2.1 GB), 393 us either way. With the gradient in a call of
// its own 170 and 338 us, 4096 rows of 70000 in fp32 (1.15 GB a pass), which no
// workgroup holds, 205 and 452. What a row needs beside its vectors (its
// entries, what lies before and behind them) is on its way with them: a load whose
// value is converted in a branch is waited for in that branch (8192 rows of 16000 in
// bf16 110 us, 124 with such loads).

#include <algorithm>
#include <cmath>

#include "ks_logit.h"
#include "ks_stack.h"

namespace ks {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxTop = KS_TEACHER_MAX_COUNT;
// Positions up to which each workgroup counts the unmasked ones itself (a launch
// less): 2 to 8 labels a thread.
constexpr int kCountRows = 2048;
static_assert(kMaxTop <= kThreads, "an entry a thread");

// 16 bytes of values that no maximum and no sum sees.
template <typename T>
__device__ __forceinline__ u32x4 lowest() {
    const uint32_t w = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;      // -inf
    return u32x4{w, w, w, w};
}

// Keeps a row's values as they were loaded: without it the compiler widens them
// once for all phases, which takes twice their registers.
template <int U>
__device__ __forceinline__ void keep_narrow(u32x4 (&w)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) asm volatile("" : "+v"(w[u]));
}

// exp((x - m) / T) as exp2((x - m) hi + (x - m) lo): log2 e / T in two parts, both
// positive, so that a difference of -inf gives 0 and not -inf + inf.
struct Scale {
    float hi, lo;
};
__device__ __forceinline__ float exp_of(float d, Scale s) {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(d, s.hi, d * s.lo));
}

// The same for a value that is rounded to T: for bf16 without the second part, which
// is 1e-6 of it at most.
template <typename T>
__device__ __forceinline__ float short_exp(float d, Scale s) {
    if constexpr (sizeof(T) == 4) return exp_of(d, s);
    else return __builtin_amdgcn_exp2f(d * s.hi);
}
constexpr Scale kNatural{kLog2e, kLog2eLow};

struct DistilArgs {
    ks_logits_t x;
    ks_teacher_t t;
    double inverse;       // 1 / T
    Scale scale;          // log2 e / T
    double kl;            // w T^2
    double ce;            // 1 - w
    float slope;          // w T
    int64_t row0;
};

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
    return x;
}
__device__ __forceinline__ float wave_sum32(float x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
    return x;
}

__device__ __forceinline__ float uniform(float x) {
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
}
// Of the W waves' values: a lane reads one, W lanes exchange them.
template <int W>
__device__ __forceinline__ float waves_max(const float (&v)[W]) {
    float x = v[threadIdx.x % W];
#pragma unroll
    for (int d = 1; d < W; d <<= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
    return uniform(x);
}
template <int W>
__device__ __forceinline__ float waves_sum(const float (&v)[W]) {
    float x = v[threadIdx.x % W];
#pragma unroll
    for (int d = 1; d < W; d <<= 1) x += __shfl_xor(x, d, 64);
    return uniform(x);
}

// A row's entry of this thread: q, its logarithm and its token (-1: none).
struct Entry {
    int64_t id;
    float q, logq;
};

__device__ __forceinline__ uint32_t bits_of(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t bits_of(bf16_t x) { return x; }
template <typename T>
__device__ __forceinline__ float value_of(uint32_t bits) {
    return __uint_as_float(sizeof(T) == 4 ? bits : bits << 16);
}

// Entry k of a row as it is loaded, with nothing that depends on the values: the
// loads stay on their way (what is converted in a branch is waited for there).
// Both words of an id and both halves of a value, of the short types the same twice.
struct RawEntry {
    uint32_t lo, hi, first, second;
};
__device__ __forceinline__ RawEntry ask_entry(const DistilArgs& a, int64_t s, int64_t t, int k) {
    k = min(k, a.t.count - 1);
    const int64_t i = s * a.t.id_seq_stride + t * a.t.id_row_stride + k;
    const int64_t v = s * a.t.top_seq_stride + t * a.t.top_row_stride + k;
    const int iw = a.t.id_bytes / 4, vw = a.t.elem == KS_ELEM_BF16 ? 1 : 2;
    const uint32_t* ids = static_cast<const uint32_t*>(a.t.ids) + i * iw;
    const uint16_t* top = static_cast<const uint16_t*>(a.t.top) + v * vw;
    return {ids[0], ids[iw - 1], top[0], top[vw - 1]};
}
__device__ __forceinline__ int64_t id_of(const DistilArgs& a, const RawEntry& e) {
    return a.t.id_bytes == 8 ? static_cast<int64_t>(static_cast<uint64_t>(e.hi) << 32 | e.lo) : static_cast<int32_t>(e.lo);
}
__device__ __forceinline__ float top_of(const DistilArgs& a, const RawEntry& e) {
    const uint32_t high = e.second << 16;
    return __uint_as_float(a.t.elem == KS_ELEM_BF16 ? high : high | e.first);
}

// buf: 2 kWaves values.
__device__ __forceinline__ Entry teacher_entry(const DistilArgs& a, int64_t s, int64_t t, float* buf) {
    Entry e{-1, 0.0f, 0.0f};
    const int k = threadIdx.x, wave = k / 64;
    float v = -INFINITY;
    if (k < a.t.count) {
        const RawEntry raw = ask_entry(a, s, t, k);
        e.id = id_of(a, raw);
        if (e.id >= 0) v = top_of(a, raw);
    }
    float m = wave_max(v);
    if (k % 64 == 0) buf[wave] = m;
    __syncthreads();
    m = buf[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, buf[w]);
    if (m == -INFINITY) m = 0.0f;            // no entry that weighs anything
    const float d = v - m, p = exp_of(d, a.scale);
    const float part = wave_sum32(p);
    if (k % 64 == 0) buf[kWaves + wave] = part;
    __syncthreads();
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += buf[kWaves + w];
    if (e.id >= 0 && sum != 0.0f) {
        e.q = p / sum;
        e.logq = static_cast<float>(static_cast<double>(d) * a.inverse - log(static_cast<double>(sum)));
    }
    if (e.id >= a.x.vocab) e.q = __builtin_nanf("");
    return e;
}

// The label of row `at`, of rows below 2^31.
__device__ __forceinline__ int64_t label_at(const ks_logits_t& x, int64_t at) {
    const uint32_t s = static_cast<uint32_t>(at) / static_cast<uint32_t>(x.tokens);
    return x.labels[s * x.label_stride + (at - static_cast<int64_t>(s) * x.tokens)];
}

// The workgroup's sum of x, in thread 0.
__device__ __forceinline__ double group_sum(double x) {
    __shared__ double sums[16];
    x = wave_sum(x);
    if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = x;
    __syncthreads();
    double total = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < 16; ++w) total += sums[w];
    __syncthreads();
    return total;
}

__device__ __forceinline__ float inverse_of(double count) { return static_cast<float>(1.0 / fmax(count, 1.0)); }

// SUM: loss = the tokens' sum times inv. COUNT: inv = 1 / (unmasked positions), at
// least one, before that. Of one workgroup: what it reads is asked for 8 at a time.
template <bool SUM, bool COUNT>
__global__ __launch_bounds__(1024) void distil_sum_kernel(const ks_logits_t x, const float* tokens, float* inv,
                                                          float* loss) {
    const int64_t n = x.sequences * x.tokens;
    const float given = COUNT ? 0.0f : *inv;
    double s = 0.0;
    int count = 0;
    constexpr int U = 8;
    for (int64_t i0 = threadIdx.x; i0 < n; i0 += 1024 * U) {
        float v[U];
        int64_t label[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = min(i0 + 1024 * u, n - 1);
            v[u] = SUM ? tokens[i] : 0.0f;
            label[u] = COUNT ? label_at(x, i) : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = i0 + 1024 * u < n;
            s += in ? static_cast<double>(v[u]) : 0.0;
            count += in && label[u] >= 0;
        }
    }
    const float scale = COUNT ? inverse_of(group_sum(static_cast<double>(count))) : given;
    if (SUM) s = group_sum(s);
    if (threadIdx.x != 0) return;
    if (COUNT) *inv = scale;
    if (SUM) *loss = static_cast<float>(s * static_cast<double>(scale));
}

// A running maximum with its two sums: exp((x - m) / T), and exp(x - m) if TWO.
template <bool TWO>
struct Running {
    float m = kLowest, s = 0.0f, s1 = 0.0f;
    __device__ __forceinline__ void raise(float top, Scale c) {
        s *= exp_of(m - top, c);
        if (TWO) s1 *= ks::exp_of(m - top);
        m = top;
    }
    __device__ __forceinline__ void add(float x, Scale c) {
        s += exp_of(x - m, c);
        if (TWO) s1 += ks::exp_of(x - m);
    }
    __device__ __forceinline__ void join(float m2, float s2, float s12, Scale c) {
        const float top = fmaxf(m, m2);
        raise(top, c);
        s += s2 * exp_of(m2 - top, c);
        if (TWO) s1 += s12 * ks::exp_of(m2 - top);
    }
};

template <typename T, bool TWO>
__global__ __launch_bounds__(kThreads) void distil_tokens_kernel(const DistilArgs a, float* tokens, float* stats) {
    __shared__ float buf[2 * kWaves], wave_stats[kWaves][3];
    __shared__ double parts[kWaves];
    constexpr int E = kVec<T>;
    const int64_t at = a.row0 + blockIdx.x, s = at / a.x.tokens, t = at - s * a.x.tokens;
    const int64_t label = a.x.labels[s * a.x.label_stride + t];
    const int tid = threadIdx.x;
    if (label < 0) {
        if (tid == 0) tokens[at] = 0.0f;
        if (tid < 3) stats[3 * at + tid] = tid == 0 ? 0.0f : 1.0f;
        return;
    }
    const T* row = static_cast<const T*>(a.x.data) + s * a.x.seq_stride + t * a.x.row_stride;
    const int V = static_cast<int>(a.x.vocab);
    const int head = head_of(row, V), vecs = (V - head) / E, tail = head + vecs * E;
    const u32x4* body = reinterpret_cast<const u32x4*>(row + head);
    Running<TWO> run;
    if (tid < head) {
        const float x = to_f32(row[tid]);
        run.raise(fmaxf(x, run.m), a.scale);
        run.add(x, a.scale);
    }
    if (tid < V - tail) {
        const float x = to_f32(row[tail + tid]);
        run.raise(fmaxf(x, run.m), a.scale);
        run.add(x, a.scale);
    }
    for (int v = tid; v < vecs; v += kThreads) {
        float x[E], top = run.m;
        widen<T>(body[v], x);
#pragma unroll
        for (int i = 0; i < E; ++i) top = fmaxf(top, x[i]);
        run.raise(top, a.scale);
#pragma unroll
        for (int i = 0; i < E; ++i) run.add(x[i], a.scale);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const float m2 = __shfl_xor(run.m, d, 64), s2 = __shfl_xor(run.s, d, 64), s12 = __shfl_xor(run.s1, d, 64);
        run.join(m2, s2, s12, a.scale);
    }
    if (tid % 64 == 0) {
        wave_stats[tid / 64][0] = run.m;
        wave_stats[tid / 64][1] = run.s;
        wave_stats[tid / 64][2] = run.s1;
    }
    const Entry e = teacher_entry(a, s, t, buf);      // its barriers cover wave_stats as well
    Running<TWO> all;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) all.join(wave_stats[w][0], wave_stats[w][1], wave_stats[w][2], a.scale);
    if (!TWO) all.s1 = all.s;
    // a weight of 0 leaves its side out, whatever it is
    double part = 0.0;
    if (a.kl > 0.0 && !(e.q == 0.0f)) {
        const float x = e.id < a.x.vocab ? to_f32(row[e.id]) : 0.0f;
        const double logp = (static_cast<double>(x) - all.m) * a.inverse - log(static_cast<double>(all.s));
        part = e.q * (e.logq - logp);
    }
    part = wave_sum(part);
    if (tid % 64 == 0) parts[tid / 64] = part;
    __syncthreads();
    if (tid == 0) {
        double token = 0.0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) token += parts[w];
        if (a.kl > 0.0) token *= a.kl;
        if (a.ce > 0.0) {
            const float x = label < a.x.vocab ? to_f32(row[label]) : __builtin_nanf("");
            token -= a.ce * ((static_cast<double>(x) - all.m) - log(static_cast<double>(all.s1)));
        }
        tokens[at] = static_cast<float>(token);
        stats[3 * at] = all.m;
        stats[3 * at + 1] = all.s;
        stats[3 * at + 2] = all.s1;
    }
}

// The exponentials of a row: exp((x - m) / T) and, where both sides weigh and T is
// not 1, exp(x - m): by an exponential of its own, or for T = 2 (the usual choice)
// as the square of the first (8192 rows of 50257 in bf16 332 us a call; 367 at
// temperature 3, with an exponential of its own).
enum Exps : int { kOne = 0, kBoth = 1, kSquare = 2 };

// dx of one row: first as if there were no entries, then the values at the
// entries' and the label's tokens again. Logits and gradient may be one memory,
// so those logits are read before anything is written. Two entries of one token
// are looked for in a bit a token (`bits`: there is room for one), and added up
// where there are any; over wider vocabularies that is done for every row.
constexpr int kSeenVocab = 1 << 17;
template <typename T, int MODE>
__global__ __launch_bounds__(kThreads) void distil_grad_kernel(const DistilArgs a, const float* stats, const float* inv,
                                                               const float* upstream, T* d_, int64_t d_seq,
                                                               int64_t d_row, bool bits) {
    extern __shared__ uint32_t seen[];
    __shared__ float buf[2 * kWaves];
    __shared__ int ids[kMaxTop], any, twice, label_in, outside;
    __shared__ float qs[kMaxTop];
    constexpr int E = kVec<T>;
    const int64_t at = a.row0 + blockIdx.x, s = at / a.x.tokens, t = at - s * a.x.tokens;
    const int64_t label = a.x.labels[s * a.x.label_stride + t];
    const T* row = static_cast<const T*>(a.x.data) + s * a.x.seq_stride + t * a.x.row_stride;
    T* out = d_ + s * d_seq + t * d_row;
    const int V = static_cast<int>(a.x.vocab), tid = threadIdx.x, entries = a.t.count;
    const int head = head_of(out, V), vecs = (V - head) / E, tail = head + vecs * E;
    typedef typename Access<T, 4>::vec access;
    u32x4* obody = reinterpret_cast<u32x4*>(out + head);
    if (label < 0) {
        if (tid < head) out[tid] = narrow<T>(0.0f);
        if (tid < V - tail) out[tail + tid] = narrow<T>(0.0f);
        const u32x4 none = {0u, 0u, 0u, 0u};
        for (int v = tid; v < vecs; v += kThreads) __builtin_nontemporal_store(none, &obody[v]);
        return;
    }
    const bool kl = a.kl > 0.0, ce = a.ce > 0.0;
    const float m = uniform(stats[3 * at]), sum = stats[3 * at + 1], sum1 = stats[3 * at + 2];
    float c = *inv;
    if (upstream) c *= *upstream;
    if (tid == 0) {
        any = label_in = 0;
        twice = !bits;
        outside = ce && label >= V;
    }
    for (int i = tid; bits && i < (V + 31) / 32; i += kThreads) seen[i] = 0;
    Entry e{-1, 0.0f, 0.0f};
    if (kl) e = teacher_entry(a, s, t, buf);       // its barriers cover what was cleared
    const bool in = e.id >= 0 && e.id < V;
    const float xe = in ? to_f32(row[e.id]) : 0.0f;
    const float xl = ce && tid == 0 ? to_f32(row[label < V ? label : 0]) : 0.0f;
    if (in) {
        const int k = static_cast<int>(e.id);
        if (bits && atomicOr(&seen[k / 32], 1u << k % 32) >> k % 32 & 1) twice = 1;
        if (e.id == label) label_in = 1;
    }
    if (e.id >= V) outside = 1;
    if (!(e.q == 0.0f)) any = 1;
    if (tid < entries) ids[tid] = in ? static_cast<int>(e.id) : -1;
    __syncthreads();
    // where nothing in the row weighs anything, that side is not there
    const float slope = any ? a.slope * c : 0.0f, hard = static_cast<float>(a.ce) * c;
    // a token outside the vocabulary makes its whole row NaN
    const float c0 = uniform(outside ? __builtin_nanf("") : MODE != kOne ? slope / sum : (slope + hard) / sum);
    const float c1 = uniform(hard / sum1);
    if (tid < entries) qs[tid] = slope * e.q;
    auto value = [&](float x) {
        const float y = short_exp<T>(x - m, a.scale);
        if (MODE == kBoth) return c0 * y + c1 * short_exp<T>(x - m, kNatural);
        if (MODE == kSquare) return y * (c0 + c1 * y);
        return c0 * y;
    };
    if (tid < head) out[tid] = narrow<T>(value(to_f32(row[tid])));
    if (tid < V - tail) out[tail + tid] = narrow<T>(value(to_f32(row[tail + tid])));
    auto put = [&](int v, u32x4 w) {
        float x[E];
        widen<T>(w, x);
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = value(x[i]);
        __builtin_nontemporal_store(pack<T>(x), &obody[v]);
    };
    constexpr int U = 4;
    int v = tid;
    for (; v + (U - 1) * kThreads < vecs; v += U * kThreads) {
        u32x4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = *reinterpret_cast<const access*>(row + head + (v + u * kThreads) * E);
#pragma unroll
        for (int u = 0; u < U; ++u) put(v + u * kThreads, w[u]);
    }
    for (; v < vecs; v += kThreads) put(v, *reinterpret_cast<const access*>(row + head + v * E));
    __syncthreads();
    if (tid < entries && in) {
        float taken = qs[tid];
        bool first = true;
        if (twice) {
            taken = 0.0f;
            for (int j = 0; j < entries; ++j) {
                if (ids[j] != ids[tid]) continue;
                first = first && j >= tid;
                taken += qs[j];
            }
        }
        if (ce && e.id == label) taken += hard;
        if (first) out[e.id] = narrow<T>(value(xe) - taken);
    }
    if (tid == 0 && ce && label < V && !label_in) out[label] = narrow<T>(value(xl) - hard);
}

// Loss and gradient (d_ null: the loss alone, and stats for a later gradient) of a
// row that the workgroup holds, U 16-byte vectors a lane.
// Rows of logits and of their gradient may start at any element: the vectors
// start where the gradient's lines do, so that stores fill them; what lies before
// the first and behind the last goes element-wise. COUNT: the workgroup counts
// the unmasked positions itself.
template <typename T, int MODE, int NT, int U, bool COUNT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(U <= 4 ? 8 : U == 8 ? 6 : 4))) void distil_row_kernel(
    const DistilArgs a, float* tokens, float* inv, float* stats, T* d_, int64_t d_seq, int64_t d_row) {
    constexpr int E = kVec<T>, W = NT / 64, EN = NT < kMaxTop ? kMaxTop / NT : 1;    // entries a thread
    constexpr bool TWO = MODE != kOne;
    extern __shared__ uint32_t seen[];        // a bit a token: whether an entry has it
    __shared__ float maxima[2][W], sums[3][W];
    __shared__ double parts[W];
    __shared__ int counts[W], twice, label_in, outside;
    __shared__ int ids[kMaxTop];
    __shared__ float qs[kMaxTop];
    const int64_t at = a.row0 + blockIdx.x, s = at / a.x.tokens, t = at - s * a.x.tokens;
    const int64_t label = a.x.labels[s * a.x.label_stride + t];
    const T* row = static_cast<const T*>(a.x.data) + s * a.x.seq_stride + t * a.x.row_stride;
    T* out = d_ + s * d_seq + t * d_row;
    const int V = static_cast<int>(a.x.vocab), tid = threadIdx.x, wave = tid / 64, entries = a.t.count;
    const int head = head_of(d_ ? out : row, V), vecs = (V - head) / E, tail = head + vecs * E;
    typedef typename Access<T, 4>::vec access;
    u32x4* obody = reinterpret_cast<u32x4*>(out + head);
    if (label < 0 && !(COUNT && at == 0)) {
        if (tid == 0) tokens[at] = 0.0f;
        if (stats && tid < 3) stats[3 * at + tid] = tid == 0 ? 0.0f : 1.0f;
        if (!d_) return;
        if (tid < head) out[tid] = narrow<T>(0.0f);
        if (tid < V - tail) out[tail + tid] = narrow<T>(0.0f);
        const u32x4 none = {0u, 0u, 0u, 0u};
        for (int v = tid; v < vecs; v += NT) __builtin_nontemporal_store(none, &obody[v]);
        return;
    }
    const bool kl = a.kl > 0.0, ce = a.ce > 0.0;
    int64_t id[EN];
    float top[EN], xe[EN];
    RawEntry raw[EN] = {};
    // the row, then what else it needs (before it: 4096 rows of 32000 in fp32, the loss
    // alone, 96 us for 94)
    u32x4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int v = u * NT + tid;
        w[u] = lowest<T>();
        if (v < vecs) w[u] = *reinterpret_cast<const access*>(row + head + v * E);
    }
#pragma unroll
    for (int n = 0; n < EN; ++n)
        if (n * NT + wave * 64 < entries) raw[n] = ask_entry(a, s, t, n * NT + tid);
    uint32_t rh = 0, rt = 0, rl = 0;
    if (wave == 0) {
        rh = bits_of(row[min(tid, V - 1)]);
        rt = bits_of(row[min(tail + tid, V - 1)]);
        rl = bits_of(row[label >= 0 && label < V ? label : 0]);
    }
    for (int i = tid; i < (V + 31) / 32; i += NT) seen[i] = 0;
    if (tid == 0) {
        twice = label_in = 0;
        outside = ce && label >= V;
    }
    int count = 0;
    if (COUNT) {
        const int n = static_cast<int>(a.x.sequences * a.x.tokens);
        int64_t labels[kCountRows / NT];
#pragma unroll
        for (int k = 0; k < kCountRows / NT; ++k) labels[k] = label_at(a.x, min(k * NT + tid, n - 1));
#pragma unroll
        for (int k = 0; k < kCountRows / NT; ++k) count += k * NT + tid < n && labels[k] >= 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) count += __shfl_xor(count, d, 64);
    }
    // maxima
    float m = kLowest, tm = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float x[E];
        widen<T>(w[u], x);
#pragma unroll
        for (int i = 0; i < E; ++i) m = fmaxf(m, x[i]);
    }
    // what came beside the row: not looked at before, in whatever order it is built
    asm volatile("" : "+v"(rh), "+v"(rt), "+v"(rl));
    const float xh = tid < head ? value_of<T>(rh) : -INFINITY, xt = tid < V - tail ? value_of<T>(rt) : -INFINITY;
    float xl = value_of<T>(rl);
    m = fmaxf(m, fmaxf(xh, xt));
    // the logits at the entries are on their way through the sums
    uint32_t re[EN] = {};
#pragma unroll
    for (int n = 0; n < EN; ++n) {
        asm volatile("" : "+v"(raw[n].lo), "+v"(raw[n].hi), "+v"(raw[n].first), "+v"(raw[n].second));
        id[n] = kl && n * NT + tid < entries ? id_of(a, raw[n]) : -1;
        top[n] = id[n] < 0 ? -INFINITY : top_of(a, raw[n]);
        tm = fmaxf(tm, top[n]);
        if (n * NT + wave * 64 < entries) re[n] = bits_of(row[id[n] >= 0 && id[n] < V ? id[n] : 0]);
    }
    m = wave_max(m);
    tm = wave_max(tm);
    if (tid % 64 == 0) {
        maxima[0][wave] = m;
        maxima[1][wave] = tm;
        if (COUNT) counts[wave] = count;
    }
    __syncthreads();
    m = waves_max(maxima[0]);
    tm = waves_max(maxima[1]);
    float scale;
    if (COUNT) {
        count = 0;
        for (int k = 0; k < W; ++k) count += counts[k];
        scale = static_cast<float>(1.0 / static_cast<double>(max(count, 1)));
        if (at == 0 && tid == 0) *inv = scale;
        if (label < 0) {                     // row 0, which stayed to count
            if (tid == 0) tokens[at] = 0.0f;
            if (stats && tid < 3) stats[3 * at + tid] = tid == 0 ? 0.0f : 1.0f;
            for (int v = tid; d_ && v < V; v += NT) out[v] = narrow<T>(0.0f);
            return;
        }
    } else {
        scale = d_ ? *inv : 0.0f;
    }
    // sums
    keep_narrow(w);
    if (tm == -INFINITY) tm = 0.0f;          // no entry that weighs anything
    float p[EN], tsum = 0.0f;
#pragma unroll
    for (int n = 0; n < EN; ++n) {
        p[n] = exp_of(top[n] - tm, a.scale);
        tsum += p[n];
        if (id[n] >= V) outside = 1;
        if (id[n] < 0 || id[n] >= V) continue;
        // duplicates are rare: looked for here, added up below if there is one
        const int k = static_cast<int>(id[n]);
        if (atomicOr(&seen[k / 32], 1u << k % 32) >> k % 32 & 1) twice = 1;
        if (id[n] == label) label_in = 1;
    }
    float sum = 0.0f, sum1 = 0.0f;
    auto add = [&](float x, float& s0, float& s1) {
        const float e = exp_of(x - m, a.scale);
        s0 += e;
        if (MODE == kBoth) s1 += ks::exp_of(x - m);
        if (MODE == kSquare) s1 += e * e;
    };
    add(xh, sum, sum1);
    add(xt, sum, sum1);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (u * NT >= vecs) continue;        // the same for all threads
        float x[E], part = 0.0f, part1 = 0.0f;
        widen<T>(w[u], x);
#pragma unroll
        for (int i = 0; i < E; ++i) add(x[i], part, part1);
        sum += part;
        sum1 += part1;
    }
    // here at the latest: behind the barrier the gradient may take the logits' place
#pragma unroll
    for (int n = 0; n < EN; ++n) {
        asm volatile("" : "+v"(re[n]));
        xe[n] = value_of<T>(re[n]);
    }
    sum = wave_sum32(sum);
    if (TWO) sum1 = wave_sum32(sum1);
    tsum = wave_sum32(tsum);
    if (tid % 64 == 0) {
        sums[0][wave] = sum;
        sums[1][wave] = sum1;
        sums[2][wave] = tsum;
    }
    __syncthreads();
    sum = waves_sum(sums[0]);
    sum1 = TWO ? waves_sum(sums[1]) : sum;
    tsum = waves_sum(sums[2]);
    // what the gradient needs of the entries
    const bool any = kl && tsum != 0.0f;     // else that side is not there
    const float slope = any ? a.slope * scale : 0.0f, hard = static_cast<float>(a.ce) * scale;
    float q[EN];
#pragma unroll
    for (int n = 0; n < EN; ++n) {
        const int k = n * NT + tid;
        q[n] = id[n] >= 0 && any ? p[n] / tsum : 0.0f;
        if (id[n] >= V) q[n] = __builtin_nanf("");
        if (k < entries) {
            ids[k] = id[n] >= 0 && id[n] < V ? static_cast<int>(id[n]) : -1;      // an id of 64 bits is no token by its lower 32
            qs[k] = slope * q[n];
        }
    }
    keep_narrow(w);
    // the gradient as if there were no entries
    // a token outside the vocabulary makes its whole row NaN
    const float c0 = uniform(outside ? __builtin_nanf("") : TWO ? slope / sum : (slope + hard) / sum);
    const float c1 = uniform(hard / sum1);
    auto value = [&](float x) {
        const float e = short_exp<T>(x - m, a.scale);
        if (MODE == kBoth) return c0 * e + c1 * short_exp<T>(x - m, kNatural);
        if (MODE == kSquare) return e * (c0 + c1 * e);
        return c0 * e;
    };
    if (d_ && tid < head) out[tid] = narrow<T>(value(xh));
    if (d_ && tid < V - tail) out[tail + tid] = narrow<T>(value(xt));
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int v = u * NT + tid;
        if (!d_ || v >= vecs) continue;
        float x[E];
        widen<T>(w[u], x);
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = value(x[i]);
        __builtin_nontemporal_store(pack<T>(x), &obody[v]);
    }
    // the entries' part of the loss
    double part = 0.0;
#pragma unroll
    for (int n = 0; n < EN; ++n) {
        if (q[n] == 0.0f) continue;
        const double logq = static_cast<double>(top[n] - tm) * a.inverse - log(static_cast<double>(tsum));
        const double logp = (static_cast<double>(xe[n]) - m) * a.inverse - log(static_cast<double>(sum));
        part += q[n] * (logq - logp);
    }
    if (wave * 64 < entries) part = wave_sum(part);
    if (tid % 64 == 0) parts[wave] = part;
    __syncthreads();
    // the values at the entries' tokens again, and at the label's if it is none of them
#pragma unroll
    for (int n = 0; n < EN; ++n) {
        const int k = n * NT + tid;
        if (!d_ || k >= entries || id[n] < 0 || id[n] >= V) continue;
        float taken = qs[k];
        bool first = true;
        if (twice) {
            taken = 0.0f;
            for (int j = 0; j < entries; ++j) {
                if (ids[j] != ids[k]) continue;
                first = first && j >= k;
                taken += qs[j];
            }
        }
        if (ce && id[n] == label) taken += hard;
        if (first) out[id[n]] = narrow<T>(value(xe[n]) - taken);
    }
    if (tid != 0) return;
    if (d_ && ce && label < V && !label_in) out[label] = narrow<T>(value(xl) - hard);
    double token = 0.0;
    for (int k = 0; k < W && k * 64 < entries; ++k) token += parts[k];
    token = kl ? token * a.kl : 0.0;
    if (ce) {
        const double x = label < V ? xl : __builtin_nanf("");
        token -= a.ce * ((x - m) - log(static_cast<double>(sum1)));
    }
    tokens[at] = static_cast<float>(token);
    if (!stats) return;
    stats[3 * at] = m;
    stats[3 * at + 1] = sum;
    stats[3 * at + 2] = sum1;
}

DistilArgs distil_args(const ks_logits_t& x, const ks_teacher_t& t, const Distil& o) {
    DistilArgs a;
    a.x = x;
    a.t = t;
    // a side of weight 0 may have any temperature: one exponential serves
    const double T = o.weight > 0.0 ? o.temperature : 1.0, c = 1.44269504088896340736 / T;
    a.inverse = 1.0 / T;
    a.scale.hi = static_cast<float>(c);
    if (a.scale.hi > c) a.scale.hi = std::nextafter(a.scale.hi, 0.0f);
    a.scale.lo = static_cast<float>(std::max(c - a.scale.hi, c * 1e-12));
    a.kl = o.weight * T * T;
    a.ce = 1.0 - o.weight;
    a.slope = static_cast<float>(o.weight * T);
    a.row0 = 0;
    return a;
}

int exps_of(const Distil& o) {
    if (!(o.weight > 0.0 && o.weight < 1.0 && o.temperature != 1.0)) return kOne;
    return o.temperature == 2.0 ? kSquare : kBoth;
}

}  // namespace

ks_status_t launch_distil_count(const ks_logits_t& x, float* inv, hipStream_t stream) {
    return launch_kernel(distil_sum_kernel<false, true>, dim3(1), dim3(1024), 0, stream, x, nullptr, inv, nullptr);
}

ks_status_t launch_distil_sum(const ks_logits_t& x, const float* tokens, float* inv, bool count, float* loss,
                              hipStream_t stream) {
    return launch_kernel(count ? distil_sum_kernel<true, true> : distil_sum_kernel<true, false>, dim3(1), dim3(1024), 0, stream, x,
                         tokens, inv, loss);
}

ks_status_t launch_distil_tokens(const ks_logits_t& x, const ks_teacher_t& t, const Distil& o, float* tokens,
                                 float* stats, hipStream_t stream) {
    DistilArgs a = distil_args(x, t, o);
    const bool two = exps_of(o) != kOne;
    const auto kernel = x.elem == KS_ELEM_BF16
                            ? (two ? distil_tokens_kernel<bf16_t, true> : distil_tokens_kernel<bf16_t, false>)
                            : (two ? distil_tokens_kernel<float, true> : distil_tokens_kernel<float, false>);
    const int64_t rows = x.sequences * x.tokens;
    for (a.row0 = 0; a.row0 < rows; a.row0 += kMaxGrid) {
        const ks_status_t st = launch_kernel(kernel, dim3(static_cast<unsigned>(std::min(kMaxGrid, rows - a.row0))),
                                             dim3(kThreads), 0, stream, a, tokens, stats);
        if (st != KS_OK) return st;
    }
    return KS_OK;
}

ks_status_t launch_distil_grad(const ks_logits_t& x, const ks_teacher_t& t, const Distil& o, const float* stats,
                               const float* inv, const float* upstream, void* d, int64_t d_seq, int64_t d_row,
                               hipStream_t stream) {
    DistilArgs a = distil_args(x, t, o);
    const bool bits = x.vocab <= kSeenVocab;
    const size_t lds = bits ? static_cast<size_t>((x.vocab + 31) / 32 * 4) : 0;
    const int mode = exps_of(o);
    const int64_t rows = x.sequences * x.tokens;
    for (a.row0 = 0; a.row0 < rows; a.row0 += kMaxGrid) {
        const dim3 grid(static_cast<unsigned>(std::min(kMaxGrid, rows - a.row0)));
        const auto run = [&](auto type, auto kernel) {
            typedef decltype(type) T;
            return launch_kernel(kernel, grid, dim3(kThreads), lds, stream, a, stats, inv, upstream, static_cast<T*>(d), d_seq,
                                 d_row, bits);
        };
        const ks_status_t st =
            x.elem == KS_ELEM_BF16
                ? run(bf16_t{}, mode == kOne ? distil_grad_kernel<bf16_t, kOne> : mode == kBoth
                                ? distil_grad_kernel<bf16_t, kBoth> : distil_grad_kernel<bf16_t, kSquare>)
                : run(float{}, mode == kOne ? distil_grad_kernel<float, kOne> : mode == kBoth
                               ? distil_grad_kernel<float, kBoth> : distil_grad_kernel<float, kSquare>);
        if (st != KS_OK) return st;
    }
    return KS_OK;
}

namespace {

template <typename T, int MODE, int NT, int U, bool COUNT>
ks_status_t run_rows(const DistilArgs& a, int64_t n, float* tokens, float* inv, float* stats, void* d, int64_t d_seq, int64_t d_row,
                     hipStream_t stream) {
    return launch_kernel(distil_row_kernel<T, MODE, NT, U, COUNT>, dim3(static_cast<unsigned>(n)), dim3(NT),
                         static_cast<size_t>((a.x.vocab + 31) / 32 * 4), stream, a, tokens, inv, stats, static_cast<T*>(d),
                         d_seq, d_row);
}

// The workgroup that holds a row's vectors: of few rows as many threads as it
// takes, for the time of one row; of many rows 8 or 16 vectors a lane, so that the
// card has more rows on their way (16384 rows of 4096 in bf16 63 us, 71 with 2).
template <typename T, int MODE>
ks_status_t pick_rows(const DistilArgs& a, int64_t n, float* tokens, float* inv, float* stats, void* d, int64_t d_seq, int64_t d_row,
                      hipStream_t stream) {
    const int64_t vecs = a.x.vocab / kVec<T>;
    const auto run =
        distil_counts(a.x)
            ? (vecs <= 256 ? run_rows<T, MODE, 256, 1, true> : vecs <= 512 ? run_rows<T, MODE, 256, 2, true>
               : vecs <= 1024 ? run_rows<T, MODE, 256, 4, true> : vecs <= 2048 ? run_rows<T, MODE, 256, 8, true>
               : vecs <= 4096 ? run_rows<T, MODE, 256, 16, true> : vecs <= 8192 ? run_rows<T, MODE, 512, 16, true>
               : run_rows<T, MODE, 1024, 16, true>)
            : (vecs <= 512 ? run_rows<T, MODE, 64, 8, false> : vecs <= 1024 ? run_rows<T, MODE, 128, 8, false>
               : vecs <= 2048 ? run_rows<T, MODE, 256, 8, false> : vecs <= 4096 ? run_rows<T, MODE, 256, 16, false>
               : vecs <= 8192 ? run_rows<T, MODE, 512, 16, false> : run_rows<T, MODE, 1024, 16, false>);
    return run(a, n, tokens, inv, stats, d, d_seq, d_row, stream);
}

}  // namespace

// With a gradient as long as registers reach. The loss alone up to 32768 values:
// of longer rows a workgroup that goes through the row keeps more bytes on their way
// (8192 rows of 50257 in bf16 161 us, 191 held; 4096 of them in fp32 150, 205 held;
// 4096 rows of 32000 in fp32 100, 95 held).
bool distil_holds(const ks_logits_t& x, bool gradient) {
    return gradient ? x.vocab / (x.elem == KS_ELEM_BF16 ? 8 : 4) <= 16384 : x.vocab <= 32768;
}

bool distil_counts(const ks_logits_t& x) { return x.sequences * x.tokens <= kCountRows; }

ks_status_t launch_distil_rows(const ks_logits_t& x, const ks_teacher_t& t, const Distil& o, float* tokens, float* inv,
                               float* stats, void* d, int64_t d_seq, int64_t d_row, hipStream_t stream) {
    DistilArgs a = distil_args(x, t, o);
    const int mode = exps_of(o);
    const auto pick = x.elem == KS_ELEM_BF16 ? (mode == kOne ? pick_rows<bf16_t, kOne> : mode == kBoth ? pick_rows<bf16_t, kBoth>
                                                : pick_rows<bf16_t, kSquare>)
                                             : (mode == kOne ? pick_rows<float, kOne> : mode == kBoth ? pick_rows<float, kBoth>
                                                : pick_rows<float, kSquare>);
    const int64_t rows = x.sequences * x.tokens;
    for (a.row0 = 0; a.row0 < rows; a.row0 += kMaxGrid / 4) {
        const ks_status_t st = pick(a, std::min(kMaxGrid / 4, rows - a.row0), tokens, inv, stats, d, d_seq, d_row, stream);
        if (st != KS_OK) return st;
    }
    return KS_OK;
}

}  // namespace ks
