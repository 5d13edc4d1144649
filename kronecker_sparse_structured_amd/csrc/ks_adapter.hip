// ks_adapter.hip -- low-rank adapters of many requests beside a shared
// projection: Y[n] += H[n] B[g]^T with H[n] = scale[g] X[n] A[g]^T, g = ids[n].
//
// Two kernels, by the number of rows.
//
// Few rows (decoding: each row a request of its own): adapter_rows_kernel, one
// row and one slice of the outputs a workgroup. Every workgroup computes the
// row's H by itself (rank dot products of n_in values: A[g] is read from L2 by
// the slices after the first), keeps it in LDS and finishes its slice, so that
// one launch does both products. What counts is latency: all loads of a phase
// are independent.
//
// Many rows: both products on the matrix cores, in two launches. A tile of 16
// rows holds rows of one request most of the time; where it holds several
// adapters they are gone through one after another and each row takes its own
// adapter's values.
//   adapter_down_kernel, H = X A^T: the four waves of a workgroup split n_in,
//     their partial sums are added in LDS. bf16 operands use the bf16 matrix
//     instruction (products of two bf16 values are exact in fp32), others the
//     fp32 one.
//   adapter_up_kernel, Y += H B^T: fp32 matrix instructions on B widened to
//     fp32, so that H is never rounded to fewer bits.
// The operands go from global memory straight to registers: A and B are read
// by many workgroups and come from L2, X and Y are used once.

#include <algorithm>

#include "ks_device.h"
#include "ks_train.h"

namespace ks {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kRowsMax = 1024;   // rows up to which the one-row kernel runs
constexpr int kTile = 16;        // rows of a tile

struct Args {
    const void* A;
    const void* B;
    const float* scale;
    const int32_t* ids;
    const void* X;
    float* Y;
    float* H;
    int64_t batch;
    int n_in, n_out, rank, count;
};

// Four consecutive values from an address that is aligned to them (WIDE), or
// element-wise; values at or after `valid` are 0.
template <bool WIDE, typename T>
__device__ __forceinline__ void load4(const T* p, int valid, float (&x)[4]) {
    if (WIDE && valid >= 4) {
        load4_f32(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = i < valid ? to_f32(p[i]) : 0.0f;
    }
}

// Ranks r .. r + 3 of a row of `rank` values. WIDE (rank a multiple of 4): one
// unconditional load, so that the loads of a wave go out together.
template <bool WIDE, typename T>
__device__ __forceinline__ void load_ranks(const T* row, int r, int rank, float (&x)[4]) {
    if constexpr (WIDE) {
        load4_f32(row + min(r, rank - 4), x);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = r < rank ? x[i] : 0.0f;
    } else {
        load4<false>(row + r, rank - r, x);
    }
}

// ---------------------------------------------------------------- few rows

// Eight consecutive values: 16-byte loads (WIDE), or element-wise with zeros
// from `valid` on.
template <bool WIDE, typename T>
__device__ __forceinline__ void load8(const T* p, int valid, float (&x)[8]) {
    if (WIDE && valid >= 8) {
        if constexpr (sizeof(T) == 4) {
            const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = a[i];
                x[4 + i] = b[i];
            }
        } else {
            const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16_lo(a[i]);
                x[2 * i + 1] = bf16_hi(a[i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < valid ? to_f32(p[i]) : 0.0f;
    }
}

template <typename TX, typename TW, bool WIDE>
__global__ __launch_bounds__(kThreads) void adapter_rows_kernel(const Args a, int slice) {
    __shared__ float h[KS_ADAPTER_MAX_RANK];
    const int64_t n = blockIdx.x;
    const int g = a.ids[n];
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    if (g < 0 || g >= a.count) {
        if (a.H && blockIdx.y == 0)
            for (int r = tid; r < a.rank; r += kThreads) a.H[n * a.rank + r] = 0.0f;
        return;
    }
    const TX* x = static_cast<const TX*>(a.X) + n * a.n_in;
    const TW* A = static_cast<const TW*>(a.A) + static_cast<int64_t>(g) * a.rank * a.n_in;
    const TW* B = static_cast<const TW*>(a.B) + static_cast<int64_t>(g) * a.n_out * a.rank;
    const float scale = a.scale[g];
    const int o0 = blockIdx.y * slice;
    const int o1 = min(a.n_out, o0 + slice);
    float* y = a.Y + n * a.n_out;
    // the first output's values of B and Y are on their way during the dot
    // products
    constexpr int kAhead = 2;
    float ahead[kAhead][8], y0 = 0.0f;
    {
        const int o = min(o0 + tid, o1 - 1);
        y0 = y[o];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) load8<WIDE>(B + static_cast<int64_t>(o) * a.rank + 8 * q, a.rank - 8 * q, ahead[q]);
    }
    // h: a wave takes four ranks at a time, its lanes the inputs
    for (int r0 = wave * 4; r0 < a.rank; r0 += 16) {
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
        for (int k = lane * 8; k < a.n_in; k += 512) {
            float xv[8], av[4][8];
            load8<WIDE>(x + k, a.n_in - k, xv);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                load8<WIDE>(A + static_cast<int64_t>(min(r0 + j, a.rank - 1)) * a.n_in + k, a.n_in - k, av[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[j] += xv[i] * av[j][i];
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], d, 64);
        if (lane == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (r0 + j < a.rank) {
                    const float v = scale * acc[j];
                    h[r0 + j] = v;
                    if (a.H && blockIdx.y == 0) a.H[n * a.rank + r0 + j] = v;
                }
            }
        }
    }
    __syncthreads();
    for (int o = o0 + tid; o < o1; o += kThreads) {
        const TW* b = B + static_cast<int64_t>(o) * a.rank;
        const bool first = o < o0 + kThreads;
        float sum = 0.0f;
        if (first) {
#pragma unroll
            for (int q = 0; q < kAhead; ++q)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (8 * q + i < a.rank) sum += ahead[q][i] * h[8 * q + i];
        }
        for (int r = first ? 8 * kAhead : 0; r < a.rank; r += 8) {
            float bv[8];
            load8<WIDE>(b + r, a.rank - r, bv);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r + i < a.rank) sum += bv[i] * h[r + i];
        }
        y[o] = (first ? y0 : y[o]) + sum;
    }
}

// ---------------------------------------------------------------- many rows

// Inputs of one step of a wave's dot products: four fp32 instructions or one
// bf16 instruction.
template <typename T>
constexpr int kStepK = sizeof(T) == 2 ? 32 : 16;

// The adapters of 16 rows, one a lane (repeated in the four lane groups), and
// the rows not yet done. A wave takes the adapters one after another: next()
// gives one of them and the mask of its rows.
struct Mix {
    int id;             // this lane's row's adapter, -1 for none
    uint64_t left;      // rows (lanes 0..15) with adapters still to do
    __device__ __forceinline__ Mix(const int32_t* ids, int64_t row0, int rows, int count) {
        const int li = threadIdx.x % 16;
        id = li < rows ? ids[row0 + li] : -1;
        if (id >= count) id = -1;
        left = __ballot(id >= 0) & 0xffffu;
    }
    __device__ __forceinline__ int next() {
        const int g = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        left &= ~__ballot(id == g);
        return g;
    }
};

// H of 16 rows a workgroup. RT: rank tiles of 16 that a pass over X keeps in
// registers.
template <typename TX, typename TW, int RT, bool WIDE>
__global__ __launch_bounds__(kThreads) void adapter_down_kernel(const Args a) {
    constexpr bool kBf16 = sizeof(TX) == 2 && sizeof(TW) == 2;
    constexpr int kPart = 16 * RT + 1;                 // odd: no bank conflicts between rows
    __shared__ float part[4][kTile][kPart];
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    const int li = lane % 16, lg = lane / 16;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const int rows = static_cast<int>(a.batch - row0 < kTile ? a.batch - row0 : kTile);
    Mix mix(a.ids, row0, rows, a.count);
    const int my_row = li < rows ? li : rows - 1;      // rows beyond the batch repeat the last one
    const TX* x = static_cast<const TX*>(a.X) + (row0 + my_row) * a.n_in;
    const int quarter = (a.n_in + 4 * kStepK<TX> - 1) / (4 * kStepK<TX>) * kStepK<TX>;
    const int k0 = wave * quarter, k1 = min(a.n_in, k0 + quarter);
    float* H = a.H + row0 * a.rank;
    if (__ballot(li < rows && mix.id < 0) != 0) {
        // rows without an adapter
        for (int i = tid; i < rows * a.rank; i += kThreads) {
            const int row = i / a.rank, id = a.ids[row0 + row];
            if (id < 0 || id >= a.count) H[i] = 0.0f;
        }
    }
    while (mix.left) {
        const int g = mix.next();
        const TW* A = static_cast<const TW*>(a.A) + static_cast<int64_t>(g) * a.rank * a.n_in;
        const float scale = a.scale[g];
        for (int r0 = 0; r0 < a.rank; r0 += 16 * RT) {
            f32x4 acc[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (kBf16 && WIDE) {
                constexpr int U = 4;                   // steps whose loads are in flight together
                for (int kb = k0; kb < k1; kb += 32 * U) {
                    u32x4 xw[U], aw[U][RT];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int k = kb + 32 * u + 8 * lg;
                        const bool in = k < k1;
                        xw[u] = *reinterpret_cast<const u32x4*>(x + (in ? k : 0));
#pragma unroll
                        for (int t = 0; t < RT; ++t) {
                            const int r = min(r0 + t * 16 + li, a.rank - 1);
                            aw[u][t] = *reinterpret_cast<const u32x4*>(A + static_cast<int64_t>(r) * a.n_in + (in ? k : 0));
                        }
                        if (!in) {
                            xw[u] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                            for (int t = 0; t < RT; ++t) aw[u][t] = u32x4{0u, 0u, 0u, 0u};
                        }
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int t = 0; t < RT; ++t)
                            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xw[u]),
                                                                            __builtin_bit_cast(bf16x8, aw[u][t]), acc[t],
                                                                            0, 0, 0);
                }
            } else {
                constexpr int U = 2;
                for (int kb = k0; kb < k1; kb += 16 * U) {
                    float xv[U][4], av[U][RT][4];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int k = kb + 16 * u + 4 * lg;
                        load4<WIDE>(x + k, k1 - k, xv[u]);
#pragma unroll
                        for (int t = 0; t < RT; ++t) {
                            const int r = min(r0 + t * 16 + li, a.rank - 1);
                            load4<WIDE>(A + static_cast<int64_t>(r) * a.n_in + k, k1 - k, av[u][t]);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int t = 0; t < RT; ++t)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(xv[u][i], av[u][t][i], acc[t], 0, 0, 0);
                }
            }
            // D: row 4 lg + i is the tile's row, column li the rank (ranks
            // beyond the adapter's repeat its last and are not kept)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[wave][4 * lg + i][t * 16 + li] = acc[t][i];
            __syncthreads();
            for (int i = tid; i < kTile * 16 * RT; i += kThreads) {
                const int row = i / (16 * RT), r = i % (16 * RT);
                if (row < rows && r0 + r < a.rank && a.ids[row0 + row] == g)
                    H[row * a.rank + r0 + r] =
                        scale * ((part[0][row][r] + part[1][row][r]) + (part[2][row][r] + part[3][row][r]));
            }
            __syncthreads();
        }
    }
}

// Y += H B^T: 16 rows and 64 outputs a wave, 256 outputs a workgroup. The
// products are formed transposed, outputs along the instruction's rows: lane
// (li, lg) holds outputs 4 lg .. 4 lg + 3 of tile row li, 64 bytes of 16 rows an
// instruction. They cross a small LDS tile of the wave's own, so that Y is read
// and written in runs of 256 bytes: lane (li, lg) takes rows 4 q + lg, outputs
// 4 li .. + 3. Y's values are on their way from the start. Bound by HBM: Y is
// read and written once, 5.7 TB/s at 16384 x 4096 (64 rows a wave: 5.4, and a
// third slower on 4099 rows, where a round of waves does not fill the card).
constexpr int kUpCols = 256, kUpPitch = 68;

// Orders the wave's LDS accesses before and after it: its lanes exchange values.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <typename TW, int RT, bool WIDE>
__global__ __launch_bounds__(kThreads) void adapter_up_kernel(const Args a) {
    __shared__ __align__(16) float cross[4][16 * kUpPitch];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int li = lane % 16, lg = lane / 16;
    // neighbouring workgroups take neighbouring columns of the same rows: with
    // rows fastest, all that run together would meet in a few memory channels
    const unsigned slabs = (a.n_out + kUpCols - 1) / kUpCols;
    const int o0 = blockIdx.x % slabs * kUpCols + wave * 64;
    if (o0 >= a.n_out) return;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / slabs) * kTile;
    const int rows = static_cast<int>(a.batch - row0 < kTile ? a.batch - row0 : kTile);
    float* mine = cross[wave];
    const int left = a.n_out - (o0 + 4 * li);          // this lane's outputs of Y inside the matrix
    const bool whole = WIDE && rows == kTile && o0 + 64 <= a.n_out;      // every lane's vectors, for the whole wave
    f32x4 y[4];
    if (whole) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            y[q] = *reinterpret_cast<const f32x4*>(a.Y + (row0 + 4 * q + lg) * a.n_out + o0 + 4 * li);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v[4];
            load4<WIDE>(a.Y + (row0 + 4 * q + lg) * a.n_out + o0 + 4 * li, 4 * q + lg < rows ? left : 0, v);
            y[q] = f32x4{v[0], v[1], v[2], v[3]};
        }
    }
    const float* h = a.H + (row0 + (li < rows ? li : rows - 1)) * a.rank;
    float hv[RT][4];                                   // H of the first ranks: all of them up to 16 RT
#pragma unroll
    for (int t = 0; t < RT; ++t) load_ranks<WIDE>(h, 16 * t + 4 * lg, a.rank, hv[t]);
    Mix mix(a.ids, row0, rows, a.count);
    if (!mix.left) return;
    f32x4 all[4];
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) all[ct] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    while (mix.left) {
        const int g = mix.next();
        f32x4 sum[4];
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) sum[ct] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int r0 = 0; r0 < a.rank; r0 += 16 * RT) {
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const int r = r0 + 16 * t + 4 * lg;
                float hr[4], bv[4][4];
                if (r0 == 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) hr[i] = hv[t][i];
                } else {
                    load_ranks<WIDE>(h, r, a.rank, hr);
                }
#pragma unroll
                for (int ct = 0; ct < 4; ++ct) {
                    const int o = min(o0 + 16 * ct + li, a.n_out - 1);
                    load_ranks<WIDE>(static_cast<const TW*>(a.B) + (static_cast<int64_t>(g) * a.n_out + o) * a.rank, r,
                                     a.rank, bv[ct]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int ct = 0; ct < 4; ++ct)
                        sum[ct] = __builtin_amdgcn_mfma_f32_16x16x4f32(bv[ct][i], hr[i], sum[ct], 0, 0, 0);
            }
        }
        // a lane's column of the product is one row of Y: a row takes its own
        // adapter's, and nothing of the others', not even their NaN
#pragma unroll
        for (int ct = 0; ct < 4; ++ct)
            if (mix.id == g) all[ct] = sum[ct];
    }
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) *reinterpret_cast<f32x4*>(mine + li * kUpPitch + 16 * ct + 4 * lg) = all[ct];
    wave_fence();
    const uint64_t on = __ballot(mix.id >= 0);         // bit r: row r has an adapter
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int r = 4 * q + lg;
        const f32x4 add = *reinterpret_cast<const f32x4*>(mine + r * kUpPitch + 4 * li);
        if (!(on >> r & 1)) continue;
        float* dst = a.Y + (row0 + r) * a.n_out + o0 + 4 * li;
        if (whole || (WIDE && left >= 4)) {
            *reinterpret_cast<f32x4*>(dst) = y[q] + add;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < left) dst[i] = y[q][i] + add[i];
        }
    }
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename TX, typename TW>
ks_status_t launch_rows(const Args& a, hipStream_t stream, int num_cus) {
    const bool wide = on16(a.X) && on16(a.A) && on16(a.B) && a.n_in % 8 == 0 && a.rank % 8 == 0;
    // slices of the outputs until the card has about four workgroups a unit;
    // at most one output a thread
    int slices = static_cast<int>(std::max<int64_t>(1, 4 * num_cus / a.batch));
    slices = std::min(slices, (a.n_out + kThreads - 1) / kThreads);
    const int slice = (a.n_out + slices - 1) / slices;
    const dim3 grid(static_cast<unsigned>(a.batch), static_cast<unsigned>((a.n_out + slice - 1) / slice));
    return launch_kernel(wide ? adapter_rows_kernel<TX, TW, true> : adapter_rows_kernel<TX, TW, false>, grid, dim3(kThreads), 0,
                         stream, a, slice);
}

template <typename TX, typename TW>
ks_status_t launch_down(const Args& a, hipStream_t stream) {
    const bool wide = on16(a.X) && on16(a.A) && a.n_in % (16 / sizeof(TX)) == 0 && a.n_in % (16 / sizeof(TW)) == 0;
    const dim3 grid(static_cast<unsigned>((a.batch + kTile - 1) / kTile));
    void (*kernel)(Args);
    if (a.rank <= 16) kernel = wide ? adapter_down_kernel<TX, TW, 1, true> : adapter_down_kernel<TX, TW, 1, false>;
    else kernel = wide ? adapter_down_kernel<TX, TW, 2, true> : adapter_down_kernel<TX, TW, 2, false>;
    return launch_kernel(kernel, grid, dim3(kThreads), 0, stream, a);
}

template <typename TW>
ks_status_t launch_up(const Args& a, hipStream_t stream) {
    const bool wide = on16(a.B) && on16(a.H) && on16(a.Y) && a.rank % 4 == 0 && a.n_out % 4 == 0;
    const int64_t blocks = (a.batch + kTile - 1) / kTile * ((a.n_out + kUpCols - 1) / kUpCols);
    if (blocks >= int64_t(1) << 31) return KS_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(blocks));
    void (*kernel)(Args);
    if (a.rank <= 16) kernel = wide ? adapter_up_kernel<TW, 1, true> : adapter_up_kernel<TW, 1, false>;
    else kernel = wide ? adapter_up_kernel<TW, 2, true> : adapter_up_kernel<TW, 2, false>;
    return launch_kernel(kernel, grid, dim3(kThreads), 0, stream, a);
}

Args args_of(const AdapterCall& c, const void* X, float* Y, float* H) {
    return Args{c.A, c.B, c.scale, c.ids, X, Y, H, c.batch, c.n_in, c.n_out, c.rank, c.count};
}

}  // namespace

bool adapter_one_launch(int64_t batch) { return batch <= kRowsMax; }

ks_status_t launch_adapter_rows(const AdapterCall& c, const void* X, float* Y, float* H) {
    const Args a = args_of(c, X, Y, H);
    if (c.xt == kBF16) return launch_rows<bf16_t, bf16_t>(a, c.stream, c.num_cus);
    if (c.wt == kBF16) return launch_rows<float, bf16_t>(a, c.stream, c.num_cus);
    return launch_rows<float, float>(a, c.stream, c.num_cus);
}

ks_status_t launch_adapter_down(const AdapterCall& c, const void* X, float* H) {
    const Args a = args_of(c, X, nullptr, H);
    if (c.xt == kBF16) return launch_down<bf16_t, bf16_t>(a, c.stream);
    if (c.wt == kBF16) return launch_down<float, bf16_t>(a, c.stream);
    return launch_down<float, float>(a, c.stream);
}

ks_status_t launch_adapter_up(const AdapterCall& c, const float* H, float* Y) {
    const Args a = args_of(c, nullptr, Y, const_cast<float*>(H));
    return c.wt == kBF16 ? launch_up<bf16_t>(a, c.stream) : launch_up<float>(a, c.stream);
}

}  // namespace ks
