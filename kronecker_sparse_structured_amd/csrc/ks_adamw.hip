// ks_adamw.hip -- one AdamW step over many tensors in few launches, with the
// two moments in fp32 or in 8 bits, and the global norm of the gradients.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// Every element is read and written once: the step is a stream of 28 bytes an
// element in fp32, 14 with bf16 gradients and 8-bit moments. A layer of KS
// factors has many small tensors, so one launch takes up to kTensors of them:
// their pointers travel as a kernel argument (no table in device memory, no
// copy that a captured graph would have to keep alive) and each workgroup
// finds its tensor by its first workgroup's number.
//
// Moments in 8 bits: blocks of 256 values with one scale a moment, m as
// s k|k| / 127^2 and v as s k^4 / 255^4. The square and the fourth power give
// the small values of a block steps as fine as the large ones' (v spans 4e9 in
// a block). A step changes v by 1 - b2 = 0.1 %, less than half a code (0.8 %
// at the top): rounding to the nearest code would never let it fall. So a
// value between two codes takes the upper one with the probability that keeps
// its mean; the random number is a hash of the seed and the value's index.
// Codes are settled by fp32 products without contraction, so they do not
// depend on how the square roots that find the lower code are rounded.

#include <algorithm>
#include <cmath>

#include "ks_device.h"
#include "ks_train.h"

#pragma clang fp contract(off)

namespace ks {
namespace {

constexpr int kTensors = 60;      // a launch: 60 * 56 bytes + options stay under 4 KB of arguments
constexpr int kThreads = 256;
constexpr int64_t kMaxGroups = int64_t(1) << 23;   // workgroups a launch: a grid counts its threads in 32 bits
constexpr int kBlock = 256;       // values that share a scale
constexpr int kLane = 8;          // consecutive values a lane holds: half a wave covers a block
constexpr int kStep = kThreads * kLane;

constexpr float kTopM = 16129.0f, kTopV = 4228250625.0f;             // 127^2, 255^4
constexpr float kUnitM = 1.0f / kTopM, kUnitV = 1.0f / kTopV;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct Entry {
    void* p;
    const void* g;
    void* m;
    void* v;
    float* scales;
    int32_t n;
    int32_t first;     // first workgroup of this tensor in the launch
    uint32_t base;     // index of its first value in the random stream
    uint32_t flags;    // kPBF16, kGBF16, kWide
};
enum : uint32_t { kPBF16 = 1, kGBF16 = 2, kWide = 4 };

struct Table {
    Entry e[kTensors];
    int32_t count;
};

struct Step {
    float b1, c1, b2, c2;      // beta and 1 - beta
    float decay;               // lr wd
    float rate;                // lr / (1 - b1^t)
    float root;                // 1 / sqrt(1 - b2^t)
    float eps;
    float max_norm;            // 0: no clip
    uint32_t seed;
    const float* norm;
};

// The tensor of a workgroup: the last entry whose first workgroup is not
// after it. The table is in scalar registers' reach: a search of six steps.
__device__ __forceinline__ int find_entry(const Table& t, int wg) {
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.e[mid].first <= wg) lo = mid;
        else hi = mid;
    }
    return lo;
}

// kLane values from element i on, `valid` of them inside the tensor.
template <typename T>
__device__ __forceinline__ void load_lane(const T* src, int valid, bool wide, float (&x)[kLane]) {
    if (wide && valid == kLane) {
        if constexpr (sizeof(T) == 4) {
            const f32x4 a = reinterpret_cast<const f32x4*>(src)[0], b = reinterpret_cast<const f32x4*>(src)[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = a[i];
                x[4 + i] = b[i];
            }
        } else {
            const u32x4 a = *reinterpret_cast<const u32x4*>(src);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16_lo(a[i]);
                x[2 * i + 1] = bf16_hi(a[i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kLane; ++i) x[i] = i < valid ? to_f32(src[i]) : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void store_lane(T* dst, int valid, bool wide, const float (&x)[kLane]) {
    if (wide && valid == kLane) {
        if constexpr (sizeof(T) == 4) {
            f32x4 a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = x[i];
                b[i] = x[4 + i];
            }
            reinterpret_cast<f32x4*>(dst)[0] = a;
            reinterpret_cast<f32x4*>(dst)[1] = b;
        } else {
            u32x4 a;
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
            *reinterpret_cast<u32x4*>(dst) = a;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kLane; ++i) {
            if (i < valid) {
                if constexpr (sizeof(T) == 4) dst[i] = x[i];
                else dst[i] = to_bf16(x[i]);
            }
        }
    }
}

// Eight byte codes of a lane (8-byte vectors where the tensor allows it).
__device__ __forceinline__ u32x2 load_codes(const uint8_t* src, int valid, bool wide) {
    if (wide && valid == kLane) return *reinterpret_cast<const u32x2*>(src);
    u32x2 w = {0u, 0u};
#pragma unroll
    for (int i = 0; i < kLane; ++i)
        if (i < valid) w[i / 4] |= static_cast<uint32_t>(src[i]) << (8 * (i % 4));
    return w;
}

__device__ __forceinline__ void store_codes(uint8_t* dst, int valid, bool wide, u32x2 w) {
    if (wide && valid == kLane) {
        *reinterpret_cast<u32x2*>(dst) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < kLane; ++i)
        if (i < valid) dst[i] = static_cast<uint8_t>(w[i / 4] >> (8 * (i % 4)));
}

__device__ __forceinline__ float signed_code(u32x2 w, int i) {
    return static_cast<float>(static_cast<int32_t>(w[i / 4] << (24 - 8 * (i % 4))) >> 24);
}
__device__ __forceinline__ float plain_code(u32x2 w, int i) {
    return static_cast<float>((w[i / 4] >> (8 * (i % 4))) & 0xffu);
}

__device__ __forceinline__ float m_value(float k, float unit) { return (k * fabsf(k)) * unit; }
__device__ __forceinline__ float v_value(float k, float unit) {
    const float q = k * k;
    return (q * q) * unit;
}

// 32 random bits for an index: a multiplicative (golden ratio) sequence and
// two rounds of multiply and shift; the multipliers were picked among random
// odd numbers for an even avalanche.
__device__ __forceinline__ uint32_t hash(uint32_t x) {
    x ^= x >> 16;
    x *= 0xaadde6a9u;
    x ^= x >> 15;
    x *= 0xbede544du;
    return x ^ (x >> 16);
}

// The largest bit pattern among the 32 lanes of a half wave: for values that
// are not negative this is their maximum, and a NaN wins.
__device__ __forceinline__ float half_wave_max(float x) {
    uint32_t u = __float_as_uint(x);
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) u = max(u, static_cast<uint32_t>(__shfl_xor(static_cast<int>(u), s, 64)));
    return __uint_as_float(u);
}

__device__ __forceinline__ float clip_of(const Step& s, bool* skip) {
    *skip = false;
    if (s.max_norm <= 0.0f) return 1.0f;
    const float norm = *s.norm;
    *skip = !(norm < __builtin_inff());
    return fminf(1.0f, s.max_norm / (norm + 1e-6f));
}

template <int BITS, typename P, typename G>
__device__ __forceinline__ void step_lane(const Entry& e, const Step& s, float clip, int64_t i, int valid) {
    const bool wide = e.flags & kWide;
    P* p = static_cast<P*>(e.p) + i;
    float g[kLane], x[kLane], m[kLane], v[kLane];
    load_lane(static_cast<const G*>(e.g) + i, valid, wide, g);
    load_lane(p, valid, wide, x);
    float* scales = e.scales + 2 * (i / kBlock);
    if constexpr (BITS == 32) {
        load_lane(static_cast<const float*>(e.m) + i, valid, wide, m);
        load_lane(static_cast<const float*>(e.v) + i, valid, wide, v);
    } else {
        const u32x2 mc = load_codes(static_cast<const uint8_t*>(e.m) + i, valid, wide);
        const u32x2 vc = load_codes(static_cast<const uint8_t*>(e.v) + i, valid, wide);
        const float mu = valid > 0 ? scales[0] * kUnitM : 0.0f;
        const float vu = valid > 0 ? scales[1] * kUnitV : 0.0f;
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            m[j] = m_value(signed_code(mc, j), mu);
            v[j] = v_value(plain_code(vc, j), vu);
        }
    }
    float mtop = 0.0f, vtop = 0.0f;
#pragma unroll
    for (int j = 0; j < kLane; ++j) {
        const float gj = g[j] * clip;
        m[j] = m[j] * s.b1 + gj * s.c1;
        v[j] = v[j] * s.b2 + (gj * gj) * s.c2;
        const float root = __builtin_amdgcn_sqrtf(v[j]) * s.root + s.eps;
        // the small terms first: p itself is rounded once
        x[j] = x[j] - (x[j] * s.decay + (m[j] * __builtin_amdgcn_rcpf(root)) * s.rate);
    }
    store_lane(p, valid, wide, x);
    if constexpr (BITS == 32) {
        store_lane(static_cast<float*>(e.m) + i, valid, wide, m);
        store_lane(static_cast<float*>(e.v) + i, valid, wide, v);
    } else {
        uint32_t mb = 0, vb = 0;
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            if (j < valid) {
                mb = max(mb, __float_as_uint(fabsf(m[j])));
                vb = max(vb, __float_as_uint(v[j]));
            }
        }
        mtop = half_wave_max(__uint_as_float(mb));
        vtop = half_wave_max(__uint_as_float(vb));
        if (mtop < 1e-30f) mtop = 1e-30f;
        if (vtop < 1e-28f) vtop = 1e-28f;
        const float mi = (1.0f / mtop) * kTopM, vi = (1.0f / vtop) * kTopV;
        u32x2 mc = {0u, 0u}, vc = {0u, 0u};
        uint32_t at = (e.base + static_cast<uint32_t>(i)) * 0x9e3779b1u + s.seed;
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            const uint32_t bits = hash(at);
            at += 0x9e3779b1u;
            const float mr = static_cast<float>(bits & 0xffffu) * (1.0f / 65536.0f);
            const float vr = static_cast<float>(bits >> 16) * (1.0f / 65536.0f);
            const float mu = fabsf(m[j]) * mi, vu = v[j] * vi;
            float k = fminf(floorf(__builtin_amdgcn_sqrtf(mu)), 127.0f);
            if (mr * (2.0f * k + 1.0f) < mu - k * k) k += 1.0f;
            k = copysignf(fminf(k, 127.0f), m[j]);
            mc[j / 4] |= (static_cast<uint32_t>(static_cast<int32_t>(k)) & 0xffu) << (8 * (j % 4));
            float q = fminf(floorf(__builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf(vu))), 255.0f);
            const float low = v_value(q, 1.0f), high = v_value(q + 1.0f, 1.0f);
            if (vr * (high - low) < vu - low) q += 1.0f;
            if (q < 1.0f && v[j] > 0.0f) q = 1.0f;
            vc[j / 4] |= static_cast<uint32_t>(fminf(q, 255.0f)) << (8 * (j % 4));
        }
        store_codes(static_cast<uint8_t*>(e.m) + i, valid, wide, mc);
        store_codes(static_cast<uint8_t*>(e.v) + i, valid, wide, vc);
        if (i % kBlock == 0 && valid > 0) {
            scales[0] = mtop;
            scales[1] = vtop;
        }
    }
}

// Workgroup w of a tensor takes values [w kStep, (w + 1) kStep): one step, as
// two or four were 1 to 9 % slower.
template <int BITS>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const Table t, const Step s) {
    bool skip;
    const float clip = clip_of(s, &skip);
    if (skip) return;
    const int wg = blockIdx.x;
    const Entry& e = t.e[find_entry(t, wg)];
    const int64_t i = static_cast<int64_t>(wg - e.first) * kStep + threadIdx.x * kLane;
    // whole half waves go on together: their maxima need every lane
    if (i / kBlock * kBlock >= e.n) return;
    const int64_t left = e.n - i;
    const int valid = static_cast<int>(left < 0 ? 0 : (left < kLane ? left : kLane));
    const uint32_t types = e.flags & (kPBF16 | kGBF16);
    if (types == 0) step_lane<BITS, float, float>(e, s, clip, i, valid);
    else if (types == kPBF16) step_lane<BITS, bf16_t, float>(e, s, clip, i, valid);
    else if (types == kGBF16) step_lane<BITS, float, bf16_t>(e, s, clip, i, valid);
    else step_lane<BITS, bf16_t, bf16_t>(e, s, clip, i, valid);
}

// Values of 8-bit states: p and g of the entries are the fp32 outputs.
__global__ __launch_bounds__(kThreads) void values_kernel(const Table t) {
    const int wg = blockIdx.x;
    const Entry& e = t.e[find_entry(t, wg)];
    const int64_t i = static_cast<int64_t>(wg - e.first) * kStep + threadIdx.x * kLane;
    if (i >= e.n) return;
    const int valid = static_cast<int>(e.n - i < kLane ? e.n - i : kLane);
    const bool wide = e.flags & kWide;
    const u32x2 mc = load_codes(static_cast<const uint8_t*>(e.m) + i, valid, wide);
    const u32x2 vc = load_codes(static_cast<const uint8_t*>(e.v) + i, valid, wide);
    const float mu = e.scales[2 * (i / kBlock)] * kUnitM;
    const float vu = e.scales[2 * (i / kBlock) + 1] * kUnitV;
    float m[kLane], v[kLane];
#pragma unroll
    for (int j = 0; j < kLane; ++j) {
        m[j] = m_value(signed_code(mc, j), mu);
        v[j] = v_value(plain_code(vc, j), vu);
    }
    store_lane(static_cast<float*>(e.p) + i, valid, wide, m);
    store_lane(static_cast<float*>(const_cast<void*>(e.g)) + i, valid, wide, v);
}

constexpr int kNormIters = 8;     // 16384 values a workgroup

// Sum of a workgroup's 256 values, in a fixed order; the result is in thread 0.
__device__ __forceinline__ float group_sum(float x) {
    __shared__ float part[kThreads / 64];
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) x += __shfl_xor(x, s, 64);
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = x;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

__global__ __launch_bounds__(kThreads) void square_sum_kernel(const Table t, float* out) {
    const int wg = blockIdx.x;
    const Entry& e = t.e[find_entry(t, wg)];
    const int64_t start = static_cast<int64_t>(wg - e.first) * (kStep * kNormIters) + threadIdx.x * kLane;
    const bool wide = e.flags & kWide;
    float sum = 0.0f;
    const bool whole = wide && start - threadIdx.x * kLane + kStep * kNormIters <= e.n;
    if (whole && !(e.flags & kGBF16)) {
        // every load of the workgroup's share in flight, each in whole lines and
        // past the last cache: 206 MB in 34 us (68 with ordinary loads, which
        // first push other tensors' changed lines out to memory)
        const f32x4* g = reinterpret_cast<const f32x4*>(static_cast<const float*>(e.g) + (start - threadIdx.x * kLane)) +
                         threadIdx.x;
        f32x4 x[2 * kNormIters];
#pragma unroll
        for (int it = 0; it < 2 * kNormIters; ++it) x[it] = __builtin_nontemporal_load(&g[it * kThreads]);
#pragma unroll
        for (int it = 0; it < 2 * kNormIters; ++it) {
            float part = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) part += x[it][j] * x[it][j];
            sum += part;
        }
    } else for (int it = 0; it < kNormIters; ++it) {
        const int64_t i = start + it * kStep;
        if (i < e.n) {
            const int valid = static_cast<int>(e.n - i < kLane ? e.n - i : kLane);
            float g[kLane];
            if (e.flags & kGBF16) load_lane(static_cast<const bf16_t*>(e.g) + i, valid, wide, g);
            else load_lane(static_cast<const float*>(e.g) + i, valid, wide, g);
            float part = 0.0f;
#pragma unroll
            for (int j = 0; j < kLane; ++j) part += g[j] * g[j];
            sum += part;
        }
    }
    sum = group_sum(sum);
    if (threadIdx.x == 0) out[wg] = sum;
}

// The partial sums of all workgroups, added in double.
__global__ __launch_bounds__(1024) void norm_kernel(const float* part, int n, float* norm) {
    __shared__ double sums[16];
    double x = 0.0;
    for (int i = threadIdx.x; i < n; i += 1024) x += static_cast<double>(part[i]);
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) x += __shfl_xor(x, s, 64);
    if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
        double total = 0.0;
        for (int i = 0; i < 16; ++i) total += sums[i];
        *norm = static_cast<float>(sqrt(total));
    }
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Runs f(table, workgroups) for every kTensors tensors; chunk = values a workgroup.
template <typename Fill, typename Run>
ks_status_t for_tables(const ks_adamw_tensor_t* t, int n, int64_t chunk, Fill fill, Run run) {
    Table table;
    table.count = 0;
    int64_t wgs = 0;
    uint64_t base = 0;
    for (int i = 0; i < n; ++i) {
        const int64_t groups = (t[i].n + chunk - 1) / chunk;
        if (groups > 0) {
            if (table.count == kTensors || wgs + groups > kMaxGroups) {
                const ks_status_t st = run(table, static_cast<unsigned>(wgs));
                if (st != KS_OK) return st;
                table.count = 0;
                wgs = 0;
            }
            Entry& e = table.e[table.count++];
            e.n = static_cast<int32_t>(t[i].n);
            e.first = static_cast<int32_t>(wgs);
            e.base = static_cast<uint32_t>(base);
            e.scales = t[i].scales;
            e.m = t[i].m;
            e.v = t[i].v;
            e.p = t[i].p;
            e.g = t[i].g;
            e.flags = (t[i].p_elem == KS_ELEM_BF16 ? kPBF16 : 0u) | (t[i].g_elem == KS_ELEM_BF16 ? kGBF16 : 0u);
            fill(e, i);
            wgs += groups;
        }
        base += static_cast<uint64_t>((t[i].n + kBlock - 1) / kBlock) * kBlock;
    }
    return table.count > 0 ? run(table, static_cast<unsigned>(wgs)) : KS_OK;
}

}  // namespace

size_t grad_norm_workspace(const ks_adamw_tensor_t* t, int n) {
    int64_t wgs = 0;
    for (int i = 0; i < n; ++i) wgs += (t[i].n + kStep * kNormIters - 1) / (kStep * kNormIters);
    return static_cast<size_t>((wgs * 4 + 255) / 256 * 256);
}

ks_status_t launch_grad_norm(const ks_adamw_tensor_t* t, int n, float* norm, void* ws, hipStream_t stream) {
    float* part = static_cast<float*>(ws);
    int total = 0;
    const ks_status_t st = for_tables(
        t, n, kStep * kNormIters, [](Entry& e, int) { e.flags |= on16(e.g) ? kWide : 0u; },
        [&](const Table& table, unsigned wgs) {
            const ks_status_t s = launch_kernel(square_sum_kernel, dim3(wgs), dim3(kThreads), 0, stream, table,
                                                part + total);
            total += static_cast<int>(wgs);
            return s;
        });
    if (st != KS_OK) return st;
    return launch_kernel(norm_kernel, dim3(1), dim3(1024), 0, stream, part, total, norm);
}

ks_status_t launch_adamw(const ks_adamw_tensor_t* t, int n, const ks_adamw_options_t& o, const float* norm,
                         hipStream_t stream) {
    Step s;
    s.b1 = static_cast<float>(o.beta1);
    s.c1 = static_cast<float>(1.0 - o.beta1);
    s.b2 = static_cast<float>(o.beta2);
    s.c2 = static_cast<float>(1.0 - o.beta2);
    s.decay = static_cast<float>(o.lr * o.weight_decay);
    s.rate = static_cast<float>(o.lr / (1.0 - std::pow(o.beta1, static_cast<double>(o.step))));
    s.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(o.beta2, static_cast<double>(o.step))));
    s.eps = static_cast<float>(o.eps);
    s.max_norm = static_cast<float>(o.max_norm);
    s.seed = o.seed;
    s.norm = norm;
    const bool small = o.state_bits == 8;
    return for_tables(
        t, n, kStep,
        [&](Entry& e, int) {
            e.flags |= (on16(e.p) && on16(e.g) && on16(e.m) && on16(e.v)) ? kWide : 0u;
        },
        [&](const Table& table, unsigned wgs) {
            return launch_kernel(small ? adamw_kernel<8> : adamw_kernel<32>, dim3(wgs),
                                 dim3(kThreads), 0, stream, table, s);
        });
}

ks_status_t launch_adamw_values(const ks_adamw_tensor_t* t, int n, float* const* m, float* const* v,
                                hipStream_t stream) {
    return for_tables(
        t, n, kStep,
        [&](Entry& e, int i) {
            e.p = m[i];
            e.g = v[i];
            e.flags = (on16(e.p) && on16(e.g) && on16(e.m) && on16(e.v)) ? kWide : 0u;
        },
        [&](const Table& table, unsigned wgs) {
            return launch_kernel(values_kernel, dim3(wgs), dim3(kThreads), 0, stream, table);
        });
}

}  // namespace ks
