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
// More rows: both products on the matrix cores, in two launches over tiles of 16
// rows. Up to some thousand rows, where requests of one row each may come in any
// order, the rows are sorted by adapter first and a tile has one adapter. Above
// that the rows of a request lie together and tiles are taken as they are: where
// one holds several adapters they are gone through one after another and each
// row takes its own adapter's values.
//   adapter_down_kernel, H = X A^T: the four waves of a workgroup split n_in,
//     their partial sums are added in LDS. bf16 operands use the bf16 matrix
//     instruction (products of two bf16 values are exact in fp32), others the
//     fp32 one.
//   adapter_up_kernel, Y += H B^T: fp32 matrix instructions on B widened to
//     fp32, so that H is never rounded to fewer bits.
// Beside a chain whose last launch adds the adapters itself (ks_fused.hip), the down
// kernel gives H in the parts that it reads, and the up kernel takes the rows it
// leaves.
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
constexpr int kRowsMax = 128;    // rows up to which the one-row kernel runs
constexpr int kSortMax = 4096;   // rows up to which the tiles are of sorted rows
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
    bf16_t* parts;           // H in three parts, chunks of 4 ranks (null: not wanted)
    PairGroup* groups;       // with parts: the adapters of each group of rows
    int64_t first;           // first workgroup of a launch among all of the batch's
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

// Sum over the wave's 64 lanes, in lane 63: four steps inside rows of 16 lanes,
// then the rows' totals from one to the next.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_total(float x) {
    x = dpp_add<0x111>(x);   // row_shr 1
    x = dpp_add<0x112>(x);   // row_shr 2
    x = dpp_add<0x114>(x);   // row_shr 4
    x = dpp_add<0x118>(x);   // row_shr 8
    x = dpp_add<0x142>(x);   // row_bcast 15: each row's last lane to the next row
    x = dpp_add<0x143>(x);   // row_bcast 31: lane 31 to the upper half
    return x;
}

template <typename TX, typename TW, bool WIDE>
__global__ __launch_bounds__(kThreads) void adapter_rows_kernel(const Args a, int slice) {
    __shared__ float h[KS_ADAPTER_MAX_RANK];
    const int64_t n = blockIdx.x;
    const int g = adapter_of(a.ids[n], a.count);
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    if (g < 0) {
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
        for (int j = 0; j < 4; ++j) acc[j] = wave_total(acc[j]);
        if (lane == 63) {
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

// Sixteen rows of a tile: rows as they lie, with their adapters' mix, or a
// block of sorted rows with one adapter.
struct Tile {
    int rows;                // rows of the tile
    int64_t row;             // this lane's row (lanes repeat in groups of 16; past `rows`: the last one)
    int id;                  // its adapter, -1 for none or past `rows`
    uint64_t left;           // rows with adapters still to do (bits 0..15)

    __device__ __forceinline__ Tile(const int32_t* ids, int64_t batch, int count, int64_t row0) {
        const int li = threadIdx.x % 16;
        rows = static_cast<int>(batch - row0 < kTile ? batch - row0 : kTile);
        row = row0 + min(li, rows - 1);
        id = li < rows ? adapter_of(ids[row], count) : -1;
        left = __ballot(id >= 0) & 0xffffu;
    }
    __device__ __forceinline__ Tile(const int* order, const AdapterSlot& slot) {
        const int li = threadIdx.x % 16;
        rows = slot.len;
        row = rows > 0 ? order[slot.start + min(li, rows - 1)] : 0;
        id = li < rows ? slot.adapter : -1;
        left = __ballot(id >= 0) & 0xffffu;
    }
    // Whether the adapters of this lane's group of kPairGroup rows change at most
    // once, and them (none if not).
    __device__ __forceinline__ bool plain(PairGroup* g) const {
        constexpr unsigned kAll = (1u << kPairGroup) - 1;
        const int lane = threadIdx.x % 64, base = lane & ~(kPairGroup - 1);
        const int last = max(min(kPairGroup, rows - base % 16) - 1, 0);
        const int first = __shfl(id, base, 64), then = __shfl(id, base + last, 64);
        const bool past = lane % 16 >= rows;
        const unsigned as_first = __ballot(past || id == first) >> base & kAll;
        const unsigned as_then = __ballot(past || id == then) >> base & kAll;
        const int split = as_first == kAll ? kPairGroup : __builtin_ctz(~as_first);
        const bool ok = as_then >> split == kAll >> split;
        *g = PairGroup::of(ok ? first : -1, ok ? split : kPairGroup, then);
        return ok;
    }
    // The rows' adapters one after another.
    __device__ __forceinline__ int next() {
        const int g = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        left &= ~__ballot(id == g);
        return g;
    }
};

// A value of H as three bf16 values, each the leading bits of what the ones before
// leave: their sum is the value exactly. Infinity and NaN stay in the first.
__device__ __forceinline__ void keep_parts(const Args& a, int64_t row, int r, float h) {
    bf16_t* to = a.parts + row * (low_parts_bytes(a.rank) / 2) + r / 4 * 12 + r % 4;
    float first = __uint_as_float(__float_as_uint(h) & 0xffff0000u), rest = h - first;
    if (!(fabsf(h) < __builtin_inff())) {
        first = h;
        rest = 0.0f;
    }
    const float second = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
    to[0] = to_bf16(first);
    to[4] = to_bf16(second);
    to[8] = to_bf16(rest - second);
}

// H of 16 rows a workgroup. RT: rank tiles of 16 that a pass over X keeps in
// registers. With sorted rows, workgroups past the slots look for rows without
// an adapter, 256 each.
template <typename TX, typename TW, int RT, bool WIDE>
__global__ __launch_bounds__(kThreads) void adapter_down_kernel(const Args a, const AdapterOrder o) {
    constexpr bool kBf16 = sizeof(TX) == 2 && sizeof(TW) == 2;
    constexpr int kPart = 16 * RT + 1;                 // odd: no bank conflicts between rows
    __shared__ float part[4][kTile][kPart];
    __shared__ int64_t row_of[kTile];
    __shared__ int id_of[kTile];
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    const int li = lane % 16, lg = lane / 16;
    const int64_t block = a.first + blockIdx.x;
    if (o.order && block >= o.n_slots) {
        // a row a thread; a wave clears the rows it has found
        const int64_t row0 = (block - o.n_slots) * kThreads + wave * 64, i = row0 + lane;
        const bool none = i < a.batch && adapter_of(a.ids[i], a.count) < 0;
        for (uint64_t off = __ballot(none); off; off &= off - 1)
            for (int r = lane; r < a.rank; r += 64) a.H[(row0 + __builtin_ctzll(off)) * a.rank + r] = 0.0f;
        return;
    }
    Tile tile = o.order ? Tile(o.order, o.slots[block]) : Tile(a.ids, a.batch, a.count, block * kTile);
    if (tile.rows == 0) return;
    if (tid < kTile) {
        row_of[tid] = tile.row;
        id_of[tid] = tile.id;
    }
    __syncthreads();
    const int rows = tile.rows;
    const TX* x = static_cast<const TX*>(a.X) + tile.row * a.n_in;
    const int quarter = (a.n_in + 4 * kStepK<TX> - 1) / (4 * kStepK<TX>) * kStepK<TX>;
    const int k0 = wave * quarter, k1 = min(a.n_in, k0 + quarter);
    if (a.parts) {
        PairGroup g;
        tile.plain(&g);
        if (tid < rows && tid % kPairGroup == 0) a.groups[(block * kTile + tid) / kPairGroup] = g;
    }
    if (!o.order) {
        // rows without an adapter
        for (int i = tid; i < rows * a.rank; i += kThreads)
            if (id_of[i / a.rank] < 0) a.H[row_of[i / a.rank] * a.rank + i % a.rank] = 0.0f;
    }
    while (tile.left) {
        const int g = tile.next();
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
                if (id_of[row] != g) continue;
                const bool in = r0 + r < a.rank;
                const float h = scale * ((part[0][row][r] + part[1][row][r]) + (part[2][row][r] + part[3][row][r]));
                if (in) a.H[row_of[row] * a.rank + r0 + r] = h;
                if (a.parts) keep_parts(a, row_of[row], r0 + r, in ? h : 0.0f);
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
// read and written once, 6.4 TB/s at 16384 x 4096 with both past the last cache
// (5.9 through it; 64 rows a wave: 5.4, and a third slower on 4099 rows, where a
// round of waves does not fill the card).
constexpr int kUpCols = 256, kUpPitch = 68;

// Orders the wave's LDS accesses before and after it: its lanes exchange values.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// kRest: only rows of groups whose adapters change more than once (a fused launch
// has added the others'), kRestTiles tiles a workgroup: mostly there are few or none, and the
// launch costs its workgroups' starts. 16384 rows in runs of whole groups: 82 us
// the whole chain with one tile each, 77 with 4, 75 with 16; 4099 rows in random
// order: 104, 105, 138.
constexpr int kRestTiles = 4;

template <typename TW, int RT, bool WIDE, bool kRest>
__global__ __launch_bounds__(kThreads) void adapter_up_kernel(const Args a, const AdapterOrder o) {
    __shared__ __align__(16) float cross[4][16 * kUpPitch];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int li = lane % 16, lg = lane / 16;
    // neighbouring workgroups take neighbouring columns of the same rows: with
    // rows fastest, all that run together would meet in a few memory channels
    const unsigned slabs = (a.n_out + kUpCols - 1) / kUpCols;
    const int64_t group = a.first + blockIdx.x;
    const int o0 = static_cast<int>(group % slabs) * kUpCols + wave * 64;
    if (o0 >= a.n_out) return;
    const int64_t first = group / slabs * (kRest ? kRestTiles : 1);
    uint64_t todo = 1;                                 // a bit a tile; with kRest kTile / kPairGroup bits, a group each
    constexpr int kBits = kRest ? kTile / kPairGroup : 1;
    if (kRest) {
        static_assert(kRestTiles * kTile <= 64 * kPairGroup, "a group a lane");
        const int64_t n = first * kTile + lane * kPairGroup;
        int id[kPairGroup];                            // all loads first: compared as they come, 6.5 us for 5.2
#pragma unroll
        for (int i = 0; i < kPairGroup; ++i) id[i] = a.ids[min(n + i, a.batch - 1)];
        const int64_t end = min(a.batch, (first + kRestTiles) * kTile);
        int changes = 0;
#pragma unroll
        for (int i = 0; i < kPairGroup; ++i) {
            id[i] = adapter_of(id[i], a.count);
            if (i > 0 && n + i < end && id[i] != id[i - 1]) ++changes;
        }
        todo = __ballot(changes > 1);
    }
    while (todo) {
        const int at = __builtin_ctzll(todo) / kBits;
        todo &= ~(((uint64_t(1) << kBits) - 1) << (at * kBits));
        const int64_t block = first + at;
        Tile tile = o.order ? Tile(o.order, o.slots[block]) : Tile(a.ids, a.batch, a.count, block * kTile);
        if (kRest) {
            PairGroup g;
            if (tile.plain(&g)) tile.id = -1;
            tile.left = __ballot(tile.id >= 0) & 0xffffu;
        }
        if (!tile.left) continue;
        const int rows = tile.rows;
        int64_t row_of[4];                                 // of this lane's runs of Y
#pragma unroll
        for (int q = 0; q < 4; ++q)
            row_of[q] = o.order ? __shfl(static_cast<int>(tile.row), 4 * q + lg, 64) : block * kTile + 4 * q + lg;
        float* mine = cross[wave];
        const int left = a.n_out - (o0 + 4 * li);          // this lane's outputs of Y inside the matrix
        const bool whole = WIDE && rows == kTile && o0 + 64 <= a.n_out;      // every lane's vectors, for the whole wave
        f32x4 y[4];
        if (whole) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                y[q] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(a.Y + row_of[q] * a.n_out + o0 + 4 * li));
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
                load4<WIDE>(a.Y + row_of[q] * a.n_out + o0 + 4 * li, 4 * q + lg < rows ? left : 0, v);
                y[q] = f32x4{v[0], v[1], v[2], v[3]};
            }
        }
        const float* h = a.H + tile.row * a.rank;
        float hv[RT][4];                                   // H of the first ranks: all of them up to 16 RT
#pragma unroll
        for (int t = 0; t < RT; ++t) load_ranks<WIDE>(h, 16 * t + 4 * lg, a.rank, hv[t]);
        f32x4 all[4];
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) all[ct] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        while (tile.left) {
            const int g = tile.next();
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
                        const int c = min(o0 + 16 * ct + li, a.n_out - 1);
                        load_ranks<WIDE>(static_cast<const TW*>(a.B) + (static_cast<int64_t>(g) * a.n_out + c) * a.rank, r,
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
                if (tile.id == g) all[ct] = sum[ct];
        }
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) *reinterpret_cast<f32x4*>(mine + li * kUpPitch + 16 * ct + 4 * lg) = all[ct];
        wave_fence();
        const uint64_t on = __ballot(tile.id >= 0);         // bit r: row r has an adapter
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = 4 * q + lg;
            const f32x4 add = *reinterpret_cast<const f32x4*>(mine + r * kUpPitch + 4 * li);
            if (!(on >> r & 1)) continue;
            float* dst = a.Y + row_of[q] * a.n_out + o0 + 4 * li;
            if (whole || (WIDE && left >= 4)) {
                __builtin_nontemporal_store(y[q] + add, reinterpret_cast<f32x4*>(dst));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < left) dst[i] = y[q][i] + add[i];
            }
        }
        wave_fence();
    }
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename TX, typename TW>
ks_status_t launch_rows(const Args& a, hipStream_t stream, int num_cus) {
    const bool wide = on16(a.X) && on16(a.A) && on16(a.B) && a.n_in % 8 == 0 && a.rank % 8 == 0;
    // slices of the outputs until the card has about two workgroups a unit;
    // at most one output a thread
    int slices = static_cast<int>(std::max<int64_t>(1, 2 * num_cus / a.batch));
    slices = std::min(slices, (a.n_out + kThreads - 1) / kThreads);
    const int slice = (a.n_out + slices - 1) / slices;
    const dim3 grid(static_cast<unsigned>(a.batch), static_cast<unsigned>((a.n_out + slice - 1) / slice));
    return launch_kernel(wide ? adapter_rows_kernel<TX, TW, true> : adapter_rows_kernel<TX, TW, false>, grid, dim3(kThreads), 0,
                         stream, a, slice);
}

// A grid counts its threads in 32 bits: at most 2^23 workgroups a launch.
ks_status_t launch_groups(void (*kernel)(Args, AdapterOrder), int64_t blocks, Args a, const AdapterOrder& o,
                          hipStream_t stream) {
    constexpr int64_t kMost = int64_t(1) << 23;
    for (a.first = 0; a.first < blocks; a.first += kMost) {
        const ks_status_t st = launch_kernel(kernel, dim3(static_cast<unsigned>(std::min(kMost, blocks - a.first))),
                                             dim3(kThreads), 0, stream, a, o);
        if (st != KS_OK) return st;
    }
    return KS_OK;
}

template <typename TX, typename TW>
ks_status_t launch_down(const Args& a, const AdapterOrder& o, hipStream_t stream) {
    const bool wide = on16(a.X) && on16(a.A) && a.n_in % (16 / sizeof(TX)) == 0 && a.n_in % (16 / sizeof(TW)) == 0;
    const int64_t blocks = o.order ? o.n_slots + (a.batch + kThreads - 1) / kThreads : (a.batch + kTile - 1) / kTile;
    void (*kernel)(Args, AdapterOrder);
    if (a.rank <= 16) kernel = wide ? adapter_down_kernel<TX, TW, 1, true> : adapter_down_kernel<TX, TW, 1, false>;
    else kernel = wide ? adapter_down_kernel<TX, TW, 2, true> : adapter_down_kernel<TX, TW, 2, false>;
    return launch_groups(kernel, blocks, a, o, stream);
}

bool up_wide(const Args& a) {
    return on16(a.B) && on16(a.H) && on16(a.Y) && a.rank % 4 == 0 && a.n_out % 4 == 0;
}

template <typename TW>
ks_status_t launch_up(const Args& a, const AdapterOrder& o, hipStream_t stream) {
    const bool wide = up_wide(a);
    const int64_t tiles = o.order ? o.n_slots : (a.batch + kTile - 1) / kTile;
    const int64_t blocks = tiles * ((a.n_out + kUpCols - 1) / kUpCols);
    void (*kernel)(Args, AdapterOrder);
    if (a.rank <= 16) kernel = wide ? adapter_up_kernel<TW, 1, true, false> : adapter_up_kernel<TW, 1, false, false>;
    else kernel = wide ? adapter_up_kernel<TW, 2, true, false> : adapter_up_kernel<TW, 2, false, false>;
    return launch_groups(kernel, blocks, a, o, stream);
}

template <typename TX, typename TW>
ks_status_t launch_types(const AdapterCall& c, const Args& a, void* ws) {
    const AdapterPath path = adapter_path(c.batch);
    if (path == kAdapterRows) return launch_rows<TX, TW>(a, c.stream, c.num_cus);
    AdapterOrder o = {};
    if (path == kAdapterSorted) {
        adapter_order_layout(c.batch, kTile, c.count, static_cast<char*>(ws), &o);
        const ks_status_t st = launch_adapter_order(c, o);
        if (st != KS_OK) return st;
    }
    const ks_status_t st = launch_down<TX, TW>(a, o, c.stream);
    return st != KS_OK ? st : launch_up<TW>(a, o, c.stream);
}

}  // namespace

// Measured at 1024 -> 4096, rank 16, bf16, 32 adapters in random order (us;
// in parentheses: the rows of a request together). 64 rows: one launch 8 (8),
// sorted tiles 14, tiles as they lie 46 (29); 200 rows: 17 (20), 14, 46 (18);
// 1024 rows: 58 (58), 20, 68 (12). From 4096 rows on the rows of a request are
// taken to lie together (prompts, training: 34 against 40 sorted); if they do
// not, a tile takes its adapters one after another (133).
AdapterPath adapter_path(int64_t batch) {
    return batch <= kRowsMax ? kAdapterRows : batch <= kSortMax ? kAdapterSorted : kAdapterRuns;
}

size_t adapter_workspace(int64_t batch, int count) {
    AdapterOrder o;
    return adapter_path(batch) == kAdapterSorted ? adapter_order_layout(batch, kTile, count, nullptr, &o) : 0;
}

ks_status_t launch_adapter(const AdapterCall& c, const void* X, float* H, float* Y, void* ws) {
    const Args a{c.A, c.B, c.scale, c.ids, X, Y, H, c.batch, c.n_in, c.n_out, c.rank, c.count, nullptr, nullptr, 0};
    if (c.xt == kBF16) return launch_types<bf16_t, bf16_t>(c, a, ws);
    if (c.wt == kBF16) return launch_types<float, bf16_t>(c, a, ws);
    return launch_types<float, float>(c, a, ws);
}

ks_status_t launch_adapter_down(const AdapterCall& c, const void* X, float* H, void* parts, PairGroup* groups) {
    const Args a{c.A, c.B, c.scale, c.ids, X, nullptr, H, c.batch, c.n_in, c.n_out, c.rank, c.count,
                 static_cast<bf16_t*>(parts), groups, 0};
    if (c.xt == kBF16) return launch_down<bf16_t, bf16_t>(a, {}, c.stream);
    if (c.wt == kBF16) return launch_down<float, bf16_t>(a, {}, c.stream);
    return launch_down<float, float>(a, {}, c.stream);
}

ks_status_t launch_adapter_rest(const AdapterCall& c, const float* H, float* Y) {
    if (c.wt != kBF16 || c.rank > kLowPartsRank) return KS_ERR_UNSUPPORTED;
    const Args a{c.A, c.B, c.scale, c.ids, nullptr, Y, const_cast<float*>(H), c.batch, c.n_in, c.n_out, c.rank,
                 c.count, nullptr, nullptr, 0};
    constexpr int kRows = kRestTiles * kTile;
    return launch_groups(up_wide(a) ? adapter_up_kernel<bf16_t, 1, true, true> : adapter_up_kernel<bf16_t, 1, false, true>,
                         (c.batch + kRows - 1) / kRows * ((c.n_out + kUpCols - 1) / kUpCols), a, {}, c.stream);
}

}  // namespace ks
