// ks_norm.hip -- the norms around a block with its gate and the residual, and
// their gradients.
//
//   u = post(y),  z = x + c s . g . u,  h = pre(z)
//
// Forward, a row at a time: x and y are read once and held in registers while
// the sums for the norms are formed, z and h are written once. Backward, with
// the statistics of the forward pass and zn, yn the normed values:
//   dx = dz + r1 (dn - zn mean(dn zn) - mean(dn)),   dn = dh . w1
//   du = c s . g . dx
//   dy = r2 (dm - yn mean(dm yn) - mean(dm)),        dm = du . w2
// (the plain means only for a norm that takes the mean off), and over the rows
//   dw1 = sum dh zn, db1 = sum dh, dw2 = sum du yn, db2 = sum du,
//   ds = sum c dx g u, and per gate dg = sum c dx s u.
// z is formed again from x and y, which costs the same read as a saved z and
// keeps what its type would have rounded away. A worker goes through a range of
// rows with its columns' sums in registers; a second launch adds up the workers'
// parts in a fixed order.
//
// A worker is 1 to 16 waves with 4 or 8 values a lane. Sums over a row are formed
// in the wave and then, for more than one wave, over LDS. The variance is the mean
// of squared differences from the mean, not a difference of two large sums. The
// vectors stay in registers from row to row and the next row is on its way while
// this one's sums are formed.
//
// What bounds it: memory, at the rate of a large copy (4.9 TB/s) or, with the last
// cache's help, above it. Forward 16384 x 1024 (fp32 in, bf16 h, 235 MB) 37 us, 6.4
// TB/s; 4096 x 4096 in bf16 (134 MB) 28 us, 4.8 TB/s (a second row ahead the same,
// and 43 for 39 in fp32). Backward 25216 x 384 in fp32 with a gate of 197 rows (232
// MB) 51 us, 4.5 TB/s; 4096 x 4096 in bf16 (201 MB) 47 us, 4.3 TB/s; 2048 x 8192 in
// bf16 (201 MB) 60 us, 3.3 TB/s: one row a compute unit, and none ahead. The parts'
// launch takes 5 to 7 us.
//
// The gradients of post's vectors and of the scale need two sums, not three:
// with t = c dx . g,  P = sum t yn  and  Q = sum t,
//   dw2 = s P,  db2 = s Q,  ds = w2 P + b2 Q.

#include <algorithm>

#include "ks_device.h"
#include "ks_stack.h"
#include "ks_stream.h"

namespace ks {
namespace {

// Waves of a worker of which a lane holds `lane` values: a power of two, so that
// workers fill a workgroup.
int worker_waves(int64_t width, int lane) {
    int w = 1;
    while (w * 64 * lane < width) w *= 2;
    return w;
}

// The values that a lane holds. Forward: 8 keep more bytes on their way (4096 x
// 4096 in bf16 27 us, 54 with 4), unless one wave of 4 would do. Backward: 4, as
// long as 16 waves reach (8192 x 2048 46 us; as many values as 2048 x 8192, with 8,
// 60 us: its vectors and sums do not fit the registers).
int forward_lane(int64_t width) { return width <= 256 ? 4 : 8; }
int backward_lane(int64_t width) { return width <= 4096 ? 4 : 8; }

// A lane's L values of a row as they are loaded: neighbours, in accesses of up to
// 16 bytes that may start at any element (a row of an odd width does), the last
// lane's one by one if the row ends among them.
template <typename T, int L>
struct Raw {
    static constexpr int kWords = L * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return i % 2 == 0 ? bf16_lo(w[i / 2]) : bf16_hi(w[i / 2]);
    }
};

template <int L>
struct Lanes {
    int t, left;            // the lane in its worker; columns from its first on, none below 0
    __device__ __forceinline__ bool in(int i) const { return i < left; }

    template <typename T>
    __device__ __forceinline__ void load(const T* row, Raw<T, L>& r) const {
        constexpr int W = Raw<T, L>::kWords, V = W < 4 ? W : 4;
        typedef typename Access<T, V>::vec vec;
        const T* p = row + t * L;
#pragma unroll
        for (int k = 0; k < W; ++k) r.w[k] = 0u;
        if (left >= L) {
#pragma unroll
            for (int k = 0; k < W; k += V) {
                const vec v = *reinterpret_cast<const vec*>(p + k * 4 / static_cast<int>(sizeof(T)));
#pragma unroll
                for (int i = 0; i < V; ++i) r.w[k + i] = v[i];
            }
        } else if (left > 0) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (!in(i)) continue;
                if constexpr (sizeof(T) == 4) r.w[i] = __float_as_uint(p[i]);
                else r.w[i / 2] |= static_cast<uint32_t>(p[i]) << (i % 2 * 16);
            }
        }
    }
    template <typename T>
    __device__ __forceinline__ void load(const T* row, float (&v)[L]) const {
        Raw<T, L> r;
        load(row, r);
#pragma unroll
        for (int i = 0; i < L; ++i) v[i] = r.get(i);
    }
    __device__ __forceinline__ void load(const void* row, int elem, float (&v)[L]) const {
        if (elem == KS_ELEM_BF16) load(static_cast<const bf16_t*>(row), v);
        else load(static_cast<const float*>(row), v);
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, const float (&v)[L]) const {
        constexpr int W = Raw<T, L>::kWords, V = W < 4 ? W : 4;
        typedef typename Access<T, V>::vec vec;
        T* p = row + t * L;
        if (left >= L) {
#pragma unroll
            for (int k = 0; k < W; k += V) {
                vec w;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[k + i]);
                    else w[i] = pack_bf16(v[2 * (k + i)], v[2 * (k + i) + 1]);
                }
                *reinterpret_cast<vec*>(p + k * 4 / static_cast<int>(sizeof(T))) = w;
            }
        } else if (left > 0) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (!in(i)) continue;
                if constexpr (sizeof(T) == 4) p[i] = v[i];
                else p[i] = to_bf16(v[i]);
            }
        }
    }
};

// Row `row` of a matrix whose type is known at run time.
__device__ __forceinline__ const void* row_of(const void* rows, int64_t row, int width, int elem) {
    return static_cast<const char*>(rows) + row * width * (elem == KS_ELEM_BF16 ? 2 : 4);
}

template <int L>
__device__ __forceinline__ void fill(float (&v)[L], float x) {
#pragma unroll
    for (int i = 0; i < L; ++i) v[i] = x;
}

// The wave's sums of a and b, in every lane. Exchanges within 16 lanes, then
// lane 15 of a row of 16 to the next row, lane 31 to the upper half.
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ void wave_sums(float& a, float& b) {
    a += moved<0xb1, 0xf>(a);       // lane ^ 1
    b += moved<0xb1, 0xf>(b);
    a += moved<0x4e, 0xf>(a);       // lane ^ 2
    b += moved<0x4e, 0xf>(b);
    a += moved<0x141, 0xf>(a);      // mirrored in 8 lanes
    b += moved<0x141, 0xf>(b);
    a += moved<0x140, 0xf>(a);      // mirrored in 16
    b += moved<0x140, 0xf>(b);
    a += moved<0x142, 0xa>(a);      // lane 15 to rows 1 and 3
    b += moved<0x142, 0xa>(b);
    a += moved<0x143, 0xc>(a);      // lane 31 to rows 2 and 3
    b += moved<0x143, 0xc>(b);
    a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(a), 63));
    b = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(b), 63));
}

// Sums over the waves of a worker. Two buffers in turn: a wave that writes one
// for the next sum but one has passed the barrier that all waves reach after
// they read it.
struct RowSums {
    float2 (*buf)[16];
    int wave, first, waves, turn;   // of the workgroup; of the worker; its waves
    __device__ __forceinline__ void operator()(float& a, float& b) {
        wave_sums(a, b);
        if (waves == 1) return;
        if (threadIdx.x % 64 == 0) buf[turn][wave] = make_float2(a, b);
        lds_barrier();
        const float2 v = buf[turn][first + (threadIdx.x & (waves - 1))];
        a = v.x + moved<0xb1, 0xf>(v.x);
        b = v.y + moved<0xb1, 0xf>(v.y);
        if (waves > 2) {
            a += moved<0x4e, 0xf>(a);
            b += moved<0x4e, 0xf>(b);
        }
        if (waves > 4) {
            a += moved<0x141, 0xf>(a);
            b += moved<0x141, 0xf>(b);
        }
        if (waves > 8) {
            a += moved<0x140, 0xf>(a);
            b += moved<0x140, 0xf>(b);
        }
        turn ^= 1;
    }
};

struct NormArgs {
    ks_residual_norm_t n;
    const void* x;
    const void* y;
    const void* gate;
    int64_t group_rows;     // 0: no gate
    int64_t rows;
    int waves;              // a worker
    float eps, residual, inverse;   // inverse: 1 / width
};

// Mean (layer norm) and 1 / deviation of the row's values.
template <int L>
__device__ __forceinline__ void deviation(const Lanes<L>& l, RowSums& sums, const NormArgs& a, const float (&v)[L],
                                          float& mean, float& r) {
    mean = 0.0f;
    float none = 0.0f;
    if (a.n.kind == KS_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < L; ++i) mean += v[i];
        sums(mean, none);
        mean *= a.inverse;
    }
    float square = 0.0f;
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const float d = l.in(i) ? v[i] - mean : 0.0f;
        square += d * d;
    }
    sums(square, none);
    r = 1.0f / sqrtf(square * a.inverse + a.eps);
}

template <int L>
__device__ __forceinline__ void vector(const Lanes<L>& l, const void* v, int elem, float none, float (&to)[L]) {
    fill(to, none);
    if (v) l.load(v, elem, to);
}

// s u = w yn + b with the scale in post's vectors: two products and 8 registers a
// lane less in every row (4096 x 4096 in bf16 26.0 us for 26.7; backward the same
// costs 3 to 10 us: its sums need s by itself too).
template <int L>
__device__ __forceinline__ void scaled_post(const Lanes<L>& l, const ks_residual_norm_t& n, float (&w)[L], float (&b)[L]) {
    float s[L];
    vector(l, n.scale, n.elem, 1.0f, s);
    vector(l, n.post_weight, n.elem, 1.0f, w);
    vector(l, n.post_bias, n.elem, 0.0f, b);
#pragma unroll
    for (int i = 0; i < L; ++i) {
        w[i] *= s[i];
        b[i] *= s[i];
    }
}

template <typename XT, typename YT, typename HT, int L>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs a, XT* z, HT* h, float* stats) {
    __shared__ float2 buf[2][16];
    const int wave = threadIdx.x / 64, worker = wave / a.waves;
    const int width = static_cast<int>(a.n.width);
    const int t = static_cast<int>(threadIdx.x) - worker * a.waves * 64;
    const Lanes<L> l{t, width - t * L};
    RowSums sums{buf, wave, worker * a.waves, a.waves, 0};
    const int each = blockDim.x / 64 / a.waves;
    const int64_t step = static_cast<int64_t>(gridDim.x) * each;
    const XT* X = static_cast<const XT*>(a.x);
    const YT* Y = static_cast<const YT*>(a.y);
    int64_t first = static_cast<int64_t>(blockIdx.x) * each;       // of the workgroup's rows
    Raw<XT, L> nx;
    Raw<YT, L> ny = {};
    float gate[L], w1[L], b1[L], w2[L], b2[L];
    // a worker without a row goes through the barriers with the last one
    auto fetch = [&](int64_t row) {
        l.load(X + row * width, nx);
        if (Y) l.load(Y + row * width, ny);
    };
    fetch(min(first + worker, a.rows - 1));
    fill(gate, 1.0f);
    scaled_post(l, a.n, w2, b2);
    vector(l, a.n.pre_weight, a.n.elem, 0.0f, w1);
    vector(l, a.n.pre_bias, a.n.elem, 0.0f, b1);
    for (; first < a.rows; first += step) {
        const int64_t row = min(first + worker, a.rows - 1);
        const bool on = first + worker < a.rows;
        float v[L], u[L], mean1 = 0.0f, r1 = 1.0f, mean2 = 0.0f, r2 = 1.0f;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            v[i] = nx.get(i);
            u[i] = ny.get(i);
        }
        if (a.gate) l.load(row_of(a.gate, row / a.group_rows, width, a.n.gate_elem), a.n.gate_elem, gate);
        if (first + step < a.rows) fetch(min(row + step, a.rows - 1));
        if (Y) {
            if (a.n.post_weight) deviation(l, sums, a, u, mean2, r2);
#pragma unroll
            for (int i = 0; i < L; ++i) v[i] += a.residual * (((u[i] - mean2) * r2 * w2[i] + b2[i]) * gate[i]);
            if (on) l.store(z + row * width, v);
        }
        if (a.n.pre_weight) {
            deviation(l, sums, a, v, mean1, r1);
#pragma unroll
            for (int i = 0; i < L; ++i) v[i] = (v[i] - mean1) * r1 * w1[i] + b1[i];
            if (on) l.store(h + row * width, v);
        }
        if (stats && on && t == 0) *reinterpret_cast<float4*>(stats + 4 * row) = make_float4(mean1, r1, mean2, r2);
    }
}

// The workgroups' parts of the vectors' sums: dw1, db1, P and Q, those that are
// wanted, one after another, each workgroups x width; then, where workers share
// a gate, theirs of the gate's, workers x width.
struct NormParts {
    float* sums;
    float* gates;
    int64_t workgroups;
    int want;               // bit k: the k-th sum
};
constexpr int kSums = 4;

struct NormGrad {
    const void* dz;
    const void* dh;
    const float* stats;
    void* dx;
    void* dy;
    void* dgate;
    NormSplit split;
    NormParts parts;
};

template <typename XT, typename YT, typename HT, int L, bool GATE>
__global__ __launch_bounds__(1024) void norm_grad_kernel(const NormArgs a, const NormGrad g) {
    extern __shared__ float join[];                // a row of the worker's columns, or its sums
    __shared__ float2 buf[2][16];
    const int wave = threadIdx.x / 64, worker = wave / a.waves, workers = blockDim.x / 64 / a.waves;
    const int width = static_cast<int>(a.n.width);
    const int t = static_cast<int>(threadIdx.x) - worker * a.waves * 64;
    const Lanes<L> l{t, width - t * L};
    RowSums sums{buf, wave, worker * a.waves, a.waves, 0};
    const int64_t id = static_cast<int64_t>(blockIdx.x) * workers + worker;
    // the worker's rows, and the one at which its gate's sum is complete
    int64_t row = id * g.split.per, end = row + g.split.per;
    if (g.split.chunks > 1) {
        const int64_t group = id / g.split.chunks, chunk = id - group * g.split.chunks;
        row = group * g.split.group_rows + chunk * g.split.per;
        end = min(row + g.split.per, (group + 1) * g.split.group_rows);
    }
    if (id >= g.split.workers) row = end = 0;
    end = min(end, a.rows);
    int64_t gate_end = g.split.chunks > 1 ? end : row + g.split.group_rows;
    const bool layer = a.n.kind == KS_NORM_LAYER;
    const XT* X = static_cast<const XT*>(a.x);
    const YT* Y = static_cast<const YT*>(a.y);
    const XT* DZ = static_cast<const XT*>(g.dz);
    const HT* DH = static_cast<const HT*>(g.dh);
    Raw<XT, L> nx, nz = {};
    Raw<YT, L> ny = {};
    Raw<HT, L> nh = {};
    float4 next = make_float4(0.0f, 1.0f, 0.0f, 1.0f);
    auto fetch = [&](int64_t at) {
        l.load(X + at * width, nx);
        if (Y) l.load(Y + at * width, ny);
        if (g.stats) next = *reinterpret_cast<const float4*>(g.stats + 4 * at);
        if (DZ) l.load(DZ + at * width, nz);
        if (DH) l.load(DH + at * width, nh);
    };
    // with 8 values a lane 16 waves have no registers for the vectors, for a row
    // ahead and for the sums: the vectors are loaded where they are used, a row when
    // it begins, the sums are in LDS
    constexpr bool kAhead = L == 4;
    if (kAhead) fetch(row < end ? row : 0);
    float held[kAhead ? kSums : 1][L], dg[L];
    auto sum = [&](int k, int i) -> float& {
        if constexpr (kAhead) return held[k][i];
        else return join[(k * L + i) * 1024 + threadIdx.x];      // 16 waves: a constant stride takes no registers
    };
#pragma unroll
    for (int k = 0; k < kSums; ++k)
#pragma unroll
        for (int i = 0; i < L; ++i) sum(k, i) = 0.0f;
    fill(dg, 0.0f);
    float w1[L], w2[L], b2[L], s[L], gate[L];
    auto hold = [&](const void* v, float none, float (&to)[L], bool now) {
        if (!now) return;
        fill(to, none);
        if (v) l.load(v, a.n.elem, to);
    };
    hold(a.n.pre_weight, 0.0f, w1, kAhead);
    hold(a.n.post_weight, 1.0f, w2, kAhead);
    hold(a.n.post_bias, 0.0f, b2, kAhead);
    hold(a.n.scale, 1.0f, s, kAhead);
    fill(gate, 1.0f);
    // every worker goes through as many rounds: they meet at barriers
    for (int64_t k = 0; k < g.split.per; ++k, ++row) {
        const bool on = row < end;
        const int64_t here = on ? row : 0;
        if (!kAhead) fetch(here);
        float z[L], yn[L], d[L], dh[L];
        const float4 st = next;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            z[i] = nx.get(i);
            yn[i] = ny.get(i);
            d[i] = nz.get(i);
            dh[i] = nh.get(i);
        }
        if (GATE && a.gate) l.load(row_of(a.gate, here / g.split.group_rows, width, a.n.gate_elem), a.n.gate_elem, gate);
        if (kAhead && row + 1 < end) fetch(row + 1);
        if (Y) {
            hold(a.n.post_weight, 1.0f, w2, !kAhead);
            hold(a.n.post_bias, 0.0f, b2, !kAhead);
            hold(a.n.scale, 1.0f, s, !kAhead);
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (a.n.post_weight) yn[i] = (yn[i] - st.z) * st.w;
                z[i] += a.residual * ((yn[i] * w2[i] + b2[i]) * s[i] * gate[i]);
            }
        }
        if (DH) {
            float dot = 0.0f, plain = 0.0f;
            hold(a.n.pre_weight, 0.0f, w1, !kAhead);
#pragma unroll
            for (int i = 0; i < L; ++i) {
                z[i] = l.in(i) ? (z[i] - st.x) * st.y : 0.0f;
                if (on) {
                    sum(0, i) += dh[i] * z[i];
                    if (kAhead || a.n.pre_bias) sum(1, i) += dh[i];
                }
                dh[i] *= w1[i];
                dot += dh[i] * z[i];
                plain += dh[i];
            }
            sums(dot, plain);
            dot *= a.inverse;
            plain = layer ? plain * a.inverse : 0.0f;
#pragma unroll
            for (int i = 0; i < L; ++i) d[i] += st.y * (dh[i] - z[i] * dot - plain);
        }
        if (on) l.store(static_cast<XT*>(g.dx) + row * width, d);
        if (!Y) continue;
        float dot = 0.0f, plain = 0.0f;
        hold(a.n.post_weight, 1.0f, w2, !kAhead);
        hold(a.n.post_bias, 0.0f, b2, !kAhead);
        hold(a.n.scale, 1.0f, s, !kAhead);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const float t = a.residual * d[i], tg = t * gate[i];
            if (on) {
                sum(2, i) += tg * yn[i];
                if (kAhead || a.n.post_bias) sum(3, i) += tg;
                if (GATE) dg[i] += t * (yn[i] * w2[i] + b2[i]) * s[i];
            }
            d[i] = l.in(i) ? tg * s[i] * w2[i] : 0.0f;
            dot += d[i] * yn[i];
            plain += d[i];
        }
        if (a.n.post_weight) {
            sums(dot, plain);
            dot *= a.inverse;
            plain = layer ? plain * a.inverse : 0.0f;
#pragma unroll
            for (int i = 0; i < L; ++i) d[i] = st.w * (d[i] - yn[i] * dot - plain);
        }
        if (on) l.store(static_cast<YT*>(g.dy) + row * width, d);
        if (GATE && g.dgate && on && row + 1 == gate_end) {
            if (g.split.chunks > 1) l.store(g.parts.gates + id * width, dg);
            else if (a.n.gate_elem == KS_ELEM_BF16) l.store(static_cast<bf16_t*>(g.dgate) + row / g.split.group_rows * width, dg);
            else l.store(static_cast<float*>(g.dgate) + row / g.split.group_rows * width, dg);
            fill(dg, 0.0f);
            gate_end += g.split.group_rows;
        }
    }
    // the workers of a workgroup, one after another
    float* to = g.parts.sums + static_cast<int64_t>(blockIdx.x) * width;
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
        if (!(g.parts.want >> k & 1)) continue;
        float mine[L];
#pragma unroll
        for (int i = 0; i < L; ++i) mine[i] = sum(k, i);
        for (int w = workers - 1; w > 0; --w) {
            if (w == worker) {
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    float* p = join + i * a.waves * 64 + t;
                    *p = w == workers - 1 ? mine[i] : *p + mine[i];
                }
            }
            lds_barrier();
        }
        if (worker == 0) {
            if (workers > 1) {
#pragma unroll
                for (int i = 0; i < L; ++i) mine[i] += join[i * a.waves * 64 + t];
            }
            l.store(to, mine);
        }
        if (workers > 1) lds_barrier();
        to += g.parts.workgroups * width;
    }
}

// Sums of parts, added in the same order every time. Of the vectors' sums, 32
// columns a workgroup and 32 parts at a time: job 0 takes dw1, job 1 db1, job 2 P
// and Q, from which it forms the gradients. Of the gates', which have few parts
// each, 128 columns of one gate a workgroup and 8 parts at a time.
struct NormJoin {
    ks_residual_norm_t n;
    ks_residual_norm_grads_t out;
    NormParts parts;
    void* dgate;
    int chunks;              // parts of a gate
    int64_t vector_groups;   // workgroups of the vectors, before those of the gates
};
constexpr int kVectorJobs = 3, kVectorCols = 32, kGateCols = 128;

__device__ __forceinline__ double vector_at(const void* v, int elem, int column, double none) {
    if (!v) return none;
    return elem == KS_ELEM_BF16 ? to_f32(static_cast<const bf16_t*>(v)[column]) : static_cast<const float*>(v)[column];
}

// A thread's share of a column's parts: `from`, from + STEP, ... of `count`.
template <int STEP>
__device__ __forceinline__ double some_parts(const float* p, int64_t from, int64_t count, int width) {
    double s = 0.0;
    int64_t k = from;
    for (; k + 7 * STEP < count; k += 8 * STEP) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = p[(k + STEP * u) * width];
#pragma unroll
        for (int u = 0; u < 8; ++u) s += static_cast<double>(v[u]);
    }
    for (; k < count; k += STEP) s += static_cast<double>(p[k * width]);
    return s;
}

__global__ __launch_bounds__(1024) void norm_join_kernel(const NormJoin j, int64_t group0) {
    __shared__ double buf[1056];
    const int width = static_cast<int>(j.n.width), tid = threadIdx.x;
    const int64_t group = blockIdx.x + group0;
    if (group >= j.vector_groups) {
        const int blocks = (width + kGateCols - 1) / kGateCols;
        const int64_t gate = (group - j.vector_groups) / blocks;
        const int column = static_cast<int>((group - j.vector_groups) % blocks) * kGateCols + tid % kGateCols;
        double s = 0.0;
        if (column < width) s = some_parts<8>(j.parts.gates + gate * j.chunks * width + column, tid / kGateCols, j.chunks, width);
        buf[tid] = s;
        __syncthreads();
        if (tid >= kGateCols || column >= width) return;
        for (int i = 1; i < 8; ++i) s += buf[i * kGateCols + tid];
        if (j.n.gate_elem == KS_ELEM_BF16)
            static_cast<bf16_t*>(j.dgate)[gate * width + column] = to_bf16(static_cast<float>(s));
        else
            static_cast<float*>(j.dgate)[gate * width + column] = static_cast<float>(s);
        return;
    }
    const int blocks = (width + kVectorCols - 1) / kVectorCols, job = static_cast<int>(group / blocks);
    const int first = static_cast<int>(group % blocks) * kVectorCols, low = tid % 32, high = tid / 32;
    // the sum k for column first + high, in that column's 32 threads
    auto total = [&](int k) {
        const float* p = j.parts.sums + __builtin_popcount(j.parts.want & ((1 << k) - 1)) * j.parts.workgroups * width;
        double s = 0.0;
        if (first + low < width) s = some_parts<32>(p + first + low, high, j.parts.workgroups, width);
        __syncthreads();
        buf[high * 33 + low] = s;
        __syncthreads();
        s = buf[low * 33 + high];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) s += __shfl_xor(s, d, 64);
        return s;
    };
    const int column = first + high;
    const bool writes = low == 0 && column < width;
    if (job < 2) {
        float* out = job == 0 ? j.out.pre_weight : j.out.pre_bias;
        if (!out) return;
        const double s = total(job);
        if (writes) out[column] = static_cast<float>(s);
    } else {
        if (!j.out.post_weight && !j.out.post_bias && !j.out.scale) return;
        const double P = j.parts.want & 4 ? total(2) : 0.0, Q = j.parts.want & 8 ? total(3) : 0.0;
        if (!writes) return;
        const double s = vector_at(j.n.scale, j.n.elem, column, 1.0),
                     w2 = vector_at(j.n.post_weight, j.n.elem, column, 1.0),
                     b2 = vector_at(j.n.post_bias, j.n.elem, column, 0.0);
        if (j.out.post_weight) j.out.post_weight[column] = static_cast<float>(s * P);
        if (j.out.post_bias) j.out.post_bias[column] = static_cast<float>(s * Q);
        if (j.out.scale) j.out.scale[column] = static_cast<float>(w2 * P + b2 * Q);
    }
}

NormArgs norm_args(const ks_residual_norm_t& n, const void* x, const void* y, const void* gate, int64_t groups,
                   int64_t rows, int lane) {
    NormArgs a;
    a.n = n;
    a.x = x;
    a.y = y;
    a.gate = gate;
    a.group_rows = groups > 0 ? rows / groups : 0;
    a.rows = rows;
    a.waves = worker_waves(n.width, lane);
    a.eps = static_cast<float>(n.eps);
    a.residual = static_cast<float>(n.residual);
    a.inverse = static_cast<float>(1.0 / static_cast<double>(n.width));
    return a;
}

template <typename XT, typename YT, typename HT, int L>
ks_status_t run_norm(const NormArgs& a, void* z, void* h, float* stats, dim3 grid, dim3 block,
                     hipStream_t stream) {
    return launch_kernel(norm_kernel<XT, YT, HT, L>, grid, block, 0, stream, a, static_cast<XT*>(z), static_cast<HT*>(h),
                         stats);
}

template <typename XT, typename YT, typename HT, int L>
ks_status_t run_grad(const NormArgs& a, const NormGrad& g, dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
    // with 8 values a lane the gate and its sum spill registers (2048 x 8192 in bf16
    // 81 us with a gate a row; without one 60, 67 if one kernel had both): a kernel
    // without them. With 4 values they fit and the same split gains nothing.
    if constexpr (L == 8)
        if (!a.gate) return launch_kernel(norm_grad_kernel<XT, YT, HT, L, false>, grid, block, lds, stream, a, g);
    return launch_kernel(norm_grad_kernel<XT, YT, HT, L, true>, grid, block, lds, stream, a, g);
}

// f(XT{}, YT{}, HT{}) for the types of n.
template <typename XT, typename YT, typename F>
ks_status_t with_h(const ks_residual_norm_t& n, F f) {
    return n.h_elem == KS_ELEM_BF16 ? f(XT{}, YT{}, bf16_t{}) : f(XT{}, YT{}, float{});
}
template <typename XT, typename F>
ks_status_t with_y(const ks_residual_norm_t& n, F f) {
    return n.y_elem == KS_ELEM_BF16 ? with_h<XT, bf16_t>(n, f) : with_h<XT, float>(n, f);
}
template <typename F>
ks_status_t with_types(const ks_residual_norm_t& n, F f) {
    return n.x_elem == KS_ELEM_BF16 ? with_y<bf16_t>(n, f) : with_y<float>(n, f);
}

// The sums that a backward pass may need: dw1, db1, P, Q.
int wanted(const ks_residual_norm_t& n) {
    return (n.pre_weight ? 1 : 0) | (n.pre_bias ? 2 : 0) | (n.post_weight || n.scale ? 4 : 0) | (n.post_bias ? 8 : 0);
}

int64_t sum_parts(const ks_residual_norm_t& n, const NormSplit& s) {
    return (__builtin_popcount(wanted(n)) * s.workgroups * n.width + 63) / 64 * 64;
}

}  // namespace

ks_status_t launch_norm(const ks_residual_norm_t& n, const void* x, const void* y, const void* gate, int64_t groups,
                        void* z, void* h, float* stats, int64_t rows, hipStream_t stream) {
    const int lane = forward_lane(n.width);
    const NormArgs a = norm_args(n, x, y, gate, groups, rows, lane);
    const int waves = std::max(4, a.waves);
    const int64_t each = waves / a.waves;
    // 16 waves a compute unit: what it holds at once with 8 values a lane
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((rows + each - 1) / each, 256 * 16 / waves)));
    return with_types(n, [&](auto xt, auto yt, auto ht) {
        typedef decltype(xt) XT;
        typedef decltype(yt) YT;
        typedef decltype(ht) HT;
        return lane == 4 ? run_norm<XT, YT, HT, 4>(a, z, h, stats, grid, dim3(waves * 64), stream)
                         : run_norm<XT, YT, HT, 8>(a, z, h, stats, grid, dim3(waves * 64), stream);
    });
}

NormSplit norm_split(int64_t width, int64_t rows, int64_t groups) {
    NormSplit s;
    const int waves = worker_waves(width, backward_lane(width));
    s.workers_a_group = std::max(1, 8 / waves);
    // 16 waves a compute unit
    const int64_t target = int64_t(256 * 16 / waves);
    const int64_t per = std::max<int64_t>(1, (rows + target - 1) / target);
    s.group_rows = groups > 0 ? rows / groups : 0;
    s.chunks = 1;
    if (rows == 0) {
        s.per = s.workers = 0;
    } else if (groups == 0) {
        s.per = per;
        s.workers = (rows + per - 1) / per;
    } else if (s.group_rows > per) {
        const int64_t chunks = (s.group_rows + per - 1) / per;
        s.per = (s.group_rows + chunks - 1) / chunks;
        s.chunks = static_cast<int>((s.group_rows + s.per - 1) / s.per);
        s.workers = groups * s.chunks;
    } else {
        const int64_t units = (per + s.group_rows - 1) / s.group_rows;    // whole groups a worker
        s.per = units * s.group_rows;
        s.workers = (groups + units - 1) / units;
    }
    s.workgroups = (s.workers + s.workers_a_group - 1) / s.workers_a_group;
    return s;
}

size_t norm_workspace(const ks_residual_norm_t& n, const NormSplit& s, int64_t rows, int64_t groups) {
    if (rows == 0) return 0;
    int64_t values = sum_parts(n, s);
    if (groups > 0 && s.chunks > 1) values += s.workers * n.width;
    return static_cast<size_t>(values) * 4;
}

ks_status_t launch_norm_grad(const ks_residual_norm_t& n, const NormSplit& s, const void* dz, const void* dh,
                             const void* x, const void* y, const void* gate, int64_t groups, const float* stats,
                             void* dx, void* dy, const ks_residual_norm_grads_t& out, void* dgate, int64_t rows, void* ws,
                             hipStream_t stream) {
    const bool any = out.pre_weight || out.pre_bias || out.post_weight || out.post_bias || out.scale;
    NormGrad g;
    g.dz = dz;
    g.dh = dh;
    g.stats = stats;
    g.dx = dx;
    g.dy = dy;
    g.dgate = dgate;
    g.split = s;
    g.parts = {static_cast<float*>(ws), static_cast<float*>(ws) + sum_parts(n, s), s.workgroups, any ? wanted(n) : 0};
    const int lane = backward_lane(n.width);
    const NormArgs a = norm_args(n, x, y, gate, groups, rows, lane);
    ks_status_t st = KS_OK;
    if (rows > 0) {
        const dim3 grid(static_cast<unsigned>(s.workgroups)), block(s.workers_a_group * a.waves * 64);
        const size_t row = static_cast<size_t>(a.waves) * 64 * lane * 4;
        const size_t lds = lane == 8 ? kSums * row : s.workers_a_group > 1 ? row : 0;
        st = with_types(n, [&](auto xt, auto yt, auto ht) {
            typedef decltype(xt) XT;
            typedef decltype(yt) YT;
            typedef decltype(ht) HT;
            return lane == 4 ? run_grad<XT, YT, HT, 4>(a, g, grid, block, lds, stream)
                             : run_grad<XT, YT, HT, 8>(a, g, grid, block, lds, stream);
        });
    }
    // the vectors and the gates that workers share (of no rows: zeros), in one launch
    const bool shared = dgate && groups > 0 && (rows == 0 || s.chunks > 1);
    const int64_t vectors = any ? kVectorJobs * ((n.width + kVectorCols - 1) / kVectorCols) : 0;
    const int64_t total = vectors + (shared ? groups * ((n.width + kGateCols - 1) / kGateCols) : 0);
    const NormJoin j{n, out, g.parts, dgate, rows > 0 ? s.chunks : 0, vectors};
    for (int64_t at = 0; st == KS_OK && at < total; at += kMaxGrid / 4)
        st = launch_kernel(norm_join_kernel, dim3(static_cast<unsigned>(std::min(kMaxGrid / 4, total - at))), dim3(1024), 0,
                           stream, j, at);
    return st;
}

}  // namespace ks
