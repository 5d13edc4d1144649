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
// A worker is 1 to 16 waves, 8 values a lane (width <= 512 a wave). Sums over a
// row are formed in the wave and then, for more than one wave, over LDS. The
// variance is the mean of squared differences from the mean, not a difference
// of two large sums.

#include <algorithm>

#include "ks_device.h"
#include "ks_stack.h"
#include "ks_stream.h"

namespace ks {
namespace {

constexpr int kLane = 8;        // values a lane holds
constexpr int kWaveCols = 64 * kLane;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Where a lane's values lie in a row. WIDE: eight neighbours, in 16-byte
// accesses. Else (a row of any width at any address) one value of each stretch
// of the row as long as the worker is wide.
template <bool WIDE>
struct Lanes {
    int t, threads, width;
    __device__ __forceinline__ int at(int i) const { return WIDE ? t * kLane + i : i * threads + t; }
    __device__ __forceinline__ bool in(int i) const { return WIDE ? t * kLane < width : at(i) < width; }

    template <typename T>
    __device__ __forceinline__ void load(const T* row, float (&v)[kLane]) const {
        if constexpr (WIDE) {
            load8<true>(row + t * kLane, t * kLane < width ? kLane : 0, v);
        } else {
#pragma unroll
            for (int i = 0; i < kLane; ++i) v[i] = in(i) ? to_f32(row[at(i)]) : 0.0f;
        }
    }
    __device__ __forceinline__ void load(const void* row, int elem, float (&v)[kLane]) const {
        if (elem == KS_ELEM_BF16) load(static_cast<const bf16_t*>(row), v);
        else load(static_cast<const float*>(row), v);
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, const float (&v)[kLane]) const {
        if constexpr (WIDE) {
            if (t * kLane >= width) return;
            if constexpr (sizeof(T) == 4) {
                f32x4* p = reinterpret_cast<f32x4*>(row + t * kLane);
                p[0] = f32x4{v[0], v[1], v[2], v[3]};
                p[1] = f32x4{v[4], v[5], v[6], v[7]};
            } else {
                u32x4 w;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
                *reinterpret_cast<u32x4*>(row + t * kLane) = w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kLane; ++i) {
                if (!in(i)) continue;
                if constexpr (sizeof(T) == 4) row[at(i)] = v[i];
                else row[at(i)] = to_bf16(v[i]);
            }
        }
    }
    __device__ __forceinline__ void store(void* row, int elem, const float (&v)[kLane]) const {
        if (elem == KS_ELEM_BF16) store(static_cast<bf16_t*>(row), v);
        else store(static_cast<float*>(row), v);
    }
};

// Sums over the waves of a worker. Two buffers in turn: a wave that writes one
// for the next sum but one has passed the barrier that all waves reach after
// they read it.
struct RowSums {
    float (*buf)[16][2];
    int wave, first, waves, turn;   // of the workgroup; of the worker; its waves
    __device__ __forceinline__ void operator()(float& a, float& b) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            a += __shfl_xor(a, d, 64);
            b += __shfl_xor(b, d, 64);
        }
        if (waves == 1) return;
        if (threadIdx.x % 64 == 0) {
            buf[turn][wave][0] = a;
            buf[turn][wave][1] = b;
        }
        lds_barrier();
        a = b = 0.0f;
        for (int w = first; w < first + waves; ++w) {
            a += buf[turn][w][0];
            b += buf[turn][w][1];
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
    int64_t row0, rows;     // rows of this launch: row0 .. rows - 1
    int waves;              // a worker
    float eps, residual, inverse;   // inverse: 1 / width
};

// Mean (layer norm) and 1 / deviation of the row's values.
template <bool WIDE>
__device__ __forceinline__ void deviation(const Lanes<WIDE>& l, RowSums& sums, const NormArgs& a,
                                          const float (&v)[kLane], float& mean, float& r) {
    mean = 0.0f;
    float none = 0.0f;
    if (a.n.kind == KS_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < kLane; ++i) mean += v[i];
        sums(mean, none);
        mean *= a.inverse;
    }
    float square = 0.0f;
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
        const float d = l.in(i) ? v[i] - mean : 0.0f;
        square += d * d;
    }
    sums(square, none);
    r = 1.0f / sqrtf(square * a.inverse + a.eps);
}

template <typename XT, typename YT, typename HT, bool WIDE>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs a, XT* z, HT* h, float* stats) {
    __shared__ float buf[2][16][2];
    const int wave = threadIdx.x / 64, worker = wave / a.waves;
    const int width = static_cast<int>(a.n.width);
    const Lanes<WIDE> l{static_cast<int>(threadIdx.x) - worker * a.waves * 64, a.waves * 64, width};
    RowSums sums{buf, wave, worker * a.waves, a.waves, 0};
    const int64_t at = a.row0 + static_cast<int64_t>(blockIdx.x) * (blockDim.x / 64 / a.waves) + worker;
    const bool on = at < a.rows;
    const int64_t row = on ? at : a.rows - 1;       // a worker without a row goes through the barriers
    float v[kLane], mean1 = 0.0f, r1 = 1.0f, mean2 = 0.0f, r2 = 1.0f;
    l.load(static_cast<const XT*>(a.x) + row * width, v);
    if (a.y) {
        float u[kLane], w[kLane];
        l.load(static_cast<const YT*>(a.y) + row * width, u);
        if (a.n.post_weight) {
            deviation(l, sums, a, u, mean2, r2);
            l.load(a.n.post_weight, a.n.elem, w);
#pragma unroll
            for (int i = 0; i < kLane; ++i) u[i] = (u[i] - mean2) * r2 * w[i];
            if (a.n.post_bias) {
                l.load(a.n.post_bias, a.n.elem, w);
#pragma unroll
                for (int i = 0; i < kLane; ++i) u[i] += w[i];
            }
        }
        if (a.n.scale) {
            l.load(a.n.scale, a.n.elem, w);
#pragma unroll
            for (int i = 0; i < kLane; ++i) u[i] *= w[i];
        }
        if (a.gate) {
            const int64_t g = row / a.group_rows;
            l.load(static_cast<const char*>(a.gate) + g * width * (a.n.gate_elem == KS_ELEM_BF16 ? 2 : 4),
                   a.n.gate_elem, w);
#pragma unroll
            for (int i = 0; i < kLane; ++i) u[i] *= w[i];
        }
#pragma unroll
        for (int i = 0; i < kLane; ++i) v[i] += a.residual * u[i];
        if (on) l.store(z + row * width, v);
    }
    if (a.n.pre_weight) {
        float w[kLane];
        deviation(l, sums, a, v, mean1, r1);
        l.load(a.n.pre_weight, a.n.elem, w);
#pragma unroll
        for (int i = 0; i < kLane; ++i) v[i] = (v[i] - mean1) * r1 * w[i];
        if (a.n.pre_bias) {
            l.load(a.n.pre_bias, a.n.elem, w);
#pragma unroll
            for (int i = 0; i < kLane; ++i) v[i] += w[i];
        }
        if (on) l.store(h + row * width, v);
    }
    if (stats && on && l.t == 0) {
        *reinterpret_cast<f32x4*>(stats + 4 * row) = f32x4{mean1, r1, mean2, r2};
    }
}

// The workers' parts of the vectors' gradients, one vector after another, each
// workgroups x width; then, where workers share a gate, theirs of the gate's,
// workers x width.
struct NormParts {
    float* vectors;
    float* gates;
    int64_t workgroups;
    int want;               // bit k: the k-th vector's gradient
};
constexpr int kVectors = 5;

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

template <typename XT, typename YT, typename HT, bool WIDE>
__global__ __launch_bounds__(1024) void norm_grad_kernel(const NormArgs a, const NormGrad g) {
    extern __shared__ float lds[];
    float (*buf)[16][2] = reinterpret_cast<float (*)[16][2]>(lds);
    float* join = lds + 2 * 16 * 2;                // a row of the worker's columns
    const int wave = threadIdx.x / 64, worker = wave / a.waves, workers = blockDim.x / 64 / a.waves;
    const int width = static_cast<int>(a.n.width);
    const Lanes<WIDE> l{static_cast<int>(threadIdx.x) - worker * a.waves * 64, a.waves * 64, width};
    RowSums sums{buf, wave, worker * a.waves, a.waves, 0};
    const int64_t id = static_cast<int64_t>(blockIdx.x) * workers + worker;
    // the worker's rows, and the one at which its gate's sum is complete
    int64_t row = id * g.split.per, end = row + g.split.per, gate_end = 0;
    if (g.split.chunks > 1) {
        const int64_t group = id / g.split.chunks, chunk = id - group * g.split.chunks;
        row = group * g.split.group_rows + chunk * g.split.per;
        end = min(row + g.split.per, (group + 1) * g.split.group_rows);
    }
    if (id >= g.split.workers) row = end = 0;
    end = min(end, a.rows);
    gate_end = g.split.chunks > 1 ? end : row + g.split.group_rows;
    const bool layer = a.n.kind == KS_NORM_LAYER;
    float sum[kVectors][kLane], dg[kLane];
#pragma unroll
    for (int k = 0; k < kVectors; ++k) zero(sum[k]);
    zero(dg);
    float w1[kLane], w2[kLane], b2[kLane], s[kLane], gate[kLane];
    zero(w1);
    zero(b2);
#pragma unroll
    for (int i = 0; i < kLane; ++i) w2[i] = s[i] = gate[i] = 1.0f;
    if (a.n.pre_weight) l.load(a.n.pre_weight, a.n.elem, w1);
    if (a.n.post_weight) l.load(a.n.post_weight, a.n.elem, w2);
    if (a.n.post_bias) l.load(a.n.post_bias, a.n.elem, b2);
    if (a.n.scale) l.load(a.n.scale, a.n.elem, s);
    const int gate_size = a.n.gate_elem == KS_ELEM_BF16 ? 2 : 4;
    // every worker goes through as many rounds: they meet at barriers
    for (int64_t k = 0; k < g.split.per; ++k, ++row) {
        const bool on = row < end;
        const int64_t at = (on ? row : 0) * width;
        float z[kLane], yn[kLane], u[kLane], d[kLane];
        f32x4 st = {0.0f, 1.0f, 0.0f, 1.0f};
        if (g.stats) st = *reinterpret_cast<const f32x4*>(g.stats + 4 * (on ? row : 0));
        l.load(static_cast<const XT*>(a.x) + at, z);
        if (a.y) {
            l.load(static_cast<const YT*>(a.y) + at, yn);
            if (a.gate) {
                const int64_t group = on ? row / g.split.group_rows : 0;
                l.load(static_cast<const char*>(a.gate) + group * width * gate_size, a.n.gate_elem, gate);
            }
#pragma unroll
            for (int i = 0; i < kLane; ++i) {
                if (a.n.post_weight) yn[i] = (yn[i] - st[2]) * st[3];
                u[i] = yn[i] * w2[i] + b2[i];
                z[i] += a.residual * u[i] * s[i] * gate[i];
            }
        }
        zero(d);
        if (g.dz) l.load(static_cast<const XT*>(g.dz) + at, d);
        if (g.dh) {
            float dh[kLane], dot = 0.0f, plain = 0.0f;
            l.load(static_cast<const HT*>(g.dh) + at, dh);
#pragma unroll
            for (int i = 0; i < kLane; ++i) {
                z[i] = l.in(i) ? (z[i] - st[0]) * st[1] : 0.0f;
                if (on) {
                    sum[0][i] += dh[i] * z[i];
                    sum[1][i] += dh[i];
                }
                dh[i] *= w1[i];
                dot += dh[i] * z[i];
                plain += dh[i];
            }
            sums(dot, plain);
            dot *= a.inverse;
            plain = layer ? plain * a.inverse : 0.0f;
#pragma unroll
            for (int i = 0; i < kLane; ++i) d[i] += st[1] * (dh[i] - z[i] * dot - plain);
        }
        if (on) l.store(static_cast<XT*>(g.dx) + at, d);
        if (!a.y) continue;
        float dot = 0.0f, plain = 0.0f;
#pragma unroll
        for (int i = 0; i < kLane; ++i) {
            const float t = a.residual * d[i], tu = t * u[i];
            const float du = t * s[i] * gate[i];
            if (on) {
                sum[4][i] += tu * gate[i];
                sum[2][i] += du * yn[i];
                sum[3][i] += du;
                dg[i] += tu * s[i];
            }
            d[i] = l.in(i) ? du * w2[i] : 0.0f;
            dot += d[i] * yn[i];
            plain += d[i];
        }
        if (a.n.post_weight) {
            sums(dot, plain);
            dot *= a.inverse;
            plain = layer ? plain * a.inverse : 0.0f;
#pragma unroll
            for (int i = 0; i < kLane; ++i) d[i] = st[3] * (d[i] - yn[i] * dot - plain);
        }
        if (on) l.store(static_cast<YT*>(g.dy) + at, d);
        if (g.dgate && on && row + 1 == gate_end) {
            if (g.split.chunks > 1) l.store(g.parts.gates + id * width, dg);
            else l.store(static_cast<char*>(g.dgate) + row / g.split.group_rows * width * gate_size, a.n.gate_elem, dg);
            zero(dg);
            gate_end += g.split.group_rows;
        }
    }
    // the workers of a workgroup, one after another
    for (int k = 0; k < kVectors; ++k) {
        if (!(g.parts.want >> k & 1)) continue;
        float mine[kLane];
#pragma unroll
        for (int i = 0; i < kLane; ++i) mine[i] = k == 0 ? sum[0][i] : k == 1 ? sum[1][i] : k == 2 ? sum[2][i] : k == 3 ? sum[3][i] : sum[4][i];
        for (int w = 0; w < workers; ++w) {
            if (w == worker) {
#pragma unroll
                for (int i = 0; i < kLane; ++i) {
                    float* p = join + i * l.threads + l.t;
                    *p = w == 0 ? mine[i] : *p + mine[i];
                }
            }
            if (workers > 1) lds_barrier();
        }
        if (worker == 0) {
#pragma unroll
            for (int i = 0; i < kLane; ++i) mine[i] = join[i * l.threads + l.t];
            l.store(g.parts.vectors + (__builtin_popcount(g.parts.want & ((1 << k) - 1)) * g.parts.workgroups + blockIdx.x) * width, mine);
        }
        if (workers > 1) lds_barrier();
    }
}

// out[column] = sum of `count` parts `width` apart: 32 columns a workgroup, 8
// parts at a time, added in the same order every time.
__device__ __forceinline__ float part_sum(const float* p, int64_t count, int64_t width, int column, int row,
                                          double (&buf)[8][32]) {
    double s = 0.0;
    if (column < width)
        for (int64_t k = row; k < count; k += 8) s += static_cast<double>(p[k * width + column]);
    buf[row][threadIdx.x % 32] = s;
    __syncthreads();
    s = 0.0;
    for (int k = 0; k < 8; ++k) s += buf[k][threadIdx.x % 32];
    return static_cast<float>(s);
}

struct VectorOut {
    float* p[kVectors];     // those that are wanted, in order
};

__global__ __launch_bounds__(256) void norm_vectors_kernel(const NormParts parts, int width, VectorOut out) {
    __shared__ double buf[8][32];
    const int column = blockIdx.x * 32 + threadIdx.x % 32, row = threadIdx.x / 32, k = blockIdx.y;
    const float s = part_sum(parts.vectors + k * parts.workgroups * width, parts.workgroups, width, column, row, buf);
    if (row == 0 && column < width) out.p[k][column] = s;
}

__global__ __launch_bounds__(256) void norm_gates_kernel(const float* parts, int chunks, int width, int64_t group0,
                                                         void* dgate, int elem) {
    __shared__ double buf[8][32];
    const int blocks = (width + 31) / 32;
    const int64_t group = group0 + blockIdx.x / blocks;
    const int column = static_cast<int>(blockIdx.x % blocks) * 32 + threadIdx.x % 32, row = threadIdx.x / 32;
    const float s = part_sum(parts + group * chunks * width, chunks, width, column, row, buf);
    if (row != 0 || column >= width) return;
    if (elem == KS_ELEM_BF16) static_cast<bf16_t*>(dgate)[group * width + column] = to_bf16(s);
    else static_cast<float*>(dgate)[group * width + column] = s;
}

// Waves of a worker: a power of two, so that workers fill a workgroup.
int worker_waves(int64_t width) {
    int w = 1;
    while (static_cast<int64_t>(w) * kWaveCols < width) w *= 2;
    return w;
}

NormArgs norm_args(const ks_residual_norm_t& n, const void* x, const void* y, const void* gate, int64_t groups,
                   int64_t rows) {
    NormArgs a;
    a.n = n;
    a.x = x;
    a.y = y;
    a.gate = gate;
    a.group_rows = groups > 0 ? rows / groups : 0;
    a.row0 = 0;
    a.rows = rows;
    a.waves = worker_waves(n.width);
    a.eps = static_cast<float>(n.eps);
    a.residual = static_cast<float>(n.residual);
    a.inverse = static_cast<float>(1.0 / static_cast<double>(n.width));
    return a;
}

bool aligned16(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
    return true;
}

template <typename XT, typename YT, typename HT>
ks_status_t run_norm(const NormArgs& a, bool wide, void* z, void* h, float* stats, dim3 grid, dim3 block,
                     hipStream_t stream) {
    return launch_kernel(wide ? norm_kernel<XT, YT, HT, true> : norm_kernel<XT, YT, HT, false>, grid, block, 0, stream,
                         a, static_cast<XT*>(z), static_cast<HT*>(h), stats);
}

template <typename XT, typename YT, typename HT>
ks_status_t run_grad(const NormArgs& a, const NormGrad& g, bool wide, dim3 grid, dim3 block, size_t lds,
                     hipStream_t stream) {
    return launch_kernel(wide ? norm_grad_kernel<XT, YT, HT, true> : norm_grad_kernel<XT, YT, HT, false>, grid, block,
                         lds, stream, a, g);
}

// f.template operator()<XT, YT, HT>() for the types of n.
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

}  // namespace

ks_status_t launch_norm(const ks_residual_norm_t& n, const void* x, const void* y, const void* gate, int64_t groups,
                        void* z, void* h, float* stats, int64_t rows, hipStream_t stream) {
    NormArgs a = norm_args(n, x, y, gate, groups, rows);
    const int waves = std::max(4, a.waves);
    const int64_t each = waves / a.waves;
    const bool wide = n.width % kLane == 0 && aligned16({x, y, gate, z, h, n.pre_weight, n.pre_bias, n.post_weight,
                                                         n.post_bias, n.scale});
    for (int64_t r = 0; r < rows; r += kMaxGrid / 4 * each) {
        a.row0 = r;
        const dim3 grid(static_cast<unsigned>(std::min(kMaxGrid / 4, (rows - r + each - 1) / each))), block(waves * 64);
        const ks_status_t st = with_types(n, [&](auto xt, auto yt, auto ht) {
            return run_norm<decltype(xt), decltype(yt), decltype(ht)>(a, wide, z, h, stats, grid, block, stream);
        });
        if (st != KS_OK) return st;
    }
    return KS_OK;
}

NormSplit norm_split(int64_t width, int64_t rows, int64_t groups) {
    NormSplit s;
    const int waves = worker_waves(width);
    s.groups_of_waves = std::max(1, 8 / waves);
    // two workgroups a compute unit
    const int64_t target = int64_t(512) * s.groups_of_waves;
    const int64_t per = std::max<int64_t>(1, (rows + target - 1) / target);
    s.group_rows = groups > 0 ? rows / groups : 0;
    s.chunks = 1;
    s.units = 1;
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
        const int64_t units = (per + s.group_rows - 1) / s.group_rows;
        s.units = static_cast<int>(units);
        s.per = units * s.group_rows;
        s.workers = (groups + units - 1) / units;
    }
    s.workgroups = (s.workers + s.groups_of_waves - 1) / s.groups_of_waves;
    return s;
}

namespace {

int wanted(const ks_residual_norm_t& n) {
    return (n.pre_weight ? 1 : 0) | (n.pre_bias ? 2 : 0) | (n.post_weight ? 4 : 0) | (n.post_bias ? 8 : 0) |
           (n.scale ? 16 : 0);
}

int64_t vector_parts(const ks_residual_norm_t& n, const NormSplit& s) {
    return __builtin_popcount(wanted(n)) * s.workgroups * n.width;
}

}  // namespace

size_t norm_workspace(const ks_residual_norm_t& n, const NormSplit& s, int64_t rows, int64_t groups) {
    if (rows == 0) return 0;
    int64_t values = (vector_parts(n, s) + 63) / 64 * 64;
    if (groups > 0 && s.chunks > 1) values += s.workers * n.width;
    return static_cast<size_t>(values) * 4;
}

ks_status_t launch_norm_grad(const ks_residual_norm_t& n, const NormSplit& s, const void* dz, const void* dh,
                             const void* x, const void* y, const void* gate, int64_t groups, const float* stats,
                             void* dx, void* dy, const ks_residual_norm_grads_t& out, void* dgate, int64_t rows, void* ws,
                             hipStream_t stream) {
    float* const outs[kVectors] = {out.pre_weight, out.pre_bias, out.post_weight, out.post_bias, out.scale};
    VectorOut vectors{};
    int count = 0;
    NormGrad g;
    g.dz = dz;
    g.dh = dh;
    g.stats = stats;
    g.dx = dx;
    g.dy = dy;
    g.dgate = dgate;
    g.split = s;
    g.parts = {static_cast<float*>(ws), static_cast<float*>(ws) + (vector_parts(n, s) + 63) / 64 * 64, s.workgroups, 0};
    for (int k = 0; k < kVectors; ++k) {
        if (!outs[k]) continue;
        g.parts.want |= 1 << k;
        vectors.p[count++] = outs[k];
    }
    const NormArgs a = norm_args(n, x, y, gate, groups, rows);
    ks_status_t st = KS_OK;
    if (rows > 0) {
        const bool wide = n.width % kLane == 0 && aligned16({x, y, gate, dz, dh, dx, dy, dgate, ws, n.pre_weight,
                                                             n.post_weight, n.post_bias, n.scale});
        const size_t lds = (2 * 16 * 2 + static_cast<size_t>(a.waves) * kWaveCols) * 4;
        st = with_types(n, [&](auto xt, auto yt, auto ht) {
            return run_grad<decltype(xt), decltype(yt), decltype(ht)>(
                a, g, wide, dim3(static_cast<unsigned>(s.workgroups)), dim3(s.groups_of_waves * a.waves * 64), lds,
                stream);
        });
    }
    if (st == KS_OK && count > 0)
        st = launch_kernel(norm_vectors_kernel, dim3(static_cast<unsigned>((n.width + 31) / 32), count), dim3(256), 0,
                           stream, g.parts, static_cast<int>(n.width), vectors);
    if (!dgate || groups == 0 || (rows > 0 && s.chunks == 1)) return st;
    const int64_t blocks = (n.width + 31) / 32, most = kMaxGrid / blocks;
    for (int64_t first = 0; st == KS_OK && first < groups; first += most)
        st = launch_kernel(norm_gates_kernel, dim3(static_cast<unsigned>(std::min(most, groups - first) * blocks)),
                           dim3(256), 0, stream, g.parts.gates, rows > 0 ? s.chunks : 0, static_cast<int>(n.width), first,
                           dgate, n.gate_elem);
    return st;
}

}  // namespace ks
