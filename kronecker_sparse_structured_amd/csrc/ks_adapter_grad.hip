// ks_adapter_grad.hip -- gradients of the adapters beside a shared projection.
// With g = ids[n] and E[n] = scale[g] dY[n] B[g]:
//   dX[n] += E[n] A[g],  dA[g] = sum_{n of g} E[n]^T X[n],  dB[g] = sum_{n of g} dY[n]^T H[n]
//
// What it cannot do without: dY and X read once, dX read and written once (the
// projection's own dX is there already). E needs a whole row of dY and dB a
// whole column, so a pass that reads dY once leaves partial sums of one of
// them: workgroups take up to 256 rows x 256 columns and leave both, E over
// column ranges and dB over row ranges, a few percent of dY's bytes each.
//   1. sort    rows by adapter (stable), cut into blocks of rows that belong
//              to one adapter each: the rest never meets a mixed block.
//   2. grad_y  a pass over dY: partial E and dB.
//   3. sum     dB and E from their partial sums, in order.
//   4. grad_x  a pass over X and dX: dX, partial dA.
//   5. sum     dA.
// For few rows the same in two launches without sorting: E and dX row by row, then
// dA and dB, each adapter's columns over its rows. No atomics; the order of every
// sum is fixed by ids alone.
//
// The products run on the fp32 matrix instruction (16 x 16 x 4), whose operands
// hold one value a lane: E, dA and dB are sums over thousands of values and stay
// in fp32 throughout. The order of the instruction's inner index is free as long
// as both operands agree on it.

#include <algorithm>

#include "ks_device.h"
#include "ks_train.h"

namespace ks {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kFewRows = 64;     // most rows of the two small launches
constexpr int kMaxRows = 256;    // most rows of a block
constexpr int kColsY = 256;      // columns of dY a workgroup takes
constexpr int kColsX = 64;       // columns of X a workgroup takes (25216 x 384: 108 us a call, 118 with 128)
constexpr int kPitch = 72;       // LDS row of a 64-wide tile: 16-byte runs of a row for the row operand, and
                                 // 4 rows x 16 columns over all banks, two lanes each, for the column operand

using Slot = AdapterSlot;
using Segment = AdapterSegment;

__device__ __forceinline__ int first_slot(Segment s, int g, int block) { return s.start / block + g; }

// One workgroup an adapter: its rows' places in the order are the rows of
// smaller adapters plus its own before them. Each wave counts a run of the
// ids, 64 at a time.
__global__ __launch_bounds__(1024) void sort_kernel(const int32_t* ids, int batch, int count, int block, int* order,
                                                    Segment* segs, Slot* slots, int n_slots) {
    __shared__ int wave_own[16], wave_less[16];
    const int g = blockIdx.x, tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    const int64_t per = ((static_cast<int64_t>(batch) + 15) / 16 + 63) / 64 * 64;
    const int64_t i0 = min(static_cast<int64_t>(batch), wave * per), i1 = min(static_cast<int64_t>(batch), i0 + per);
    constexpr int kHeld = 32;       // ids a lane holds: one read of up to 32768 rows
    int own = 0, less = 0, id[kHeld];
    for (int64_t i = i0; i < i1; i += 64 * kHeld) {
#pragma unroll
        for (int u = 0; u < kHeld; ++u) id[u] = i + 64 * u + lane < i1 ? ids[i + 64 * u + lane] : -1;
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            own += __popcll(__ballot(id[u] == g));
            less += __popcll(__ballot(id[u] >= 0 && id[u] < g));
        }
    }
    if (lane == 0) {
        wave_own[wave] = own;
        wave_less[wave] = less;
    }
    __syncthreads();
    int start = 0, total = 0, at = 0;
    for (int w = 0; w < 16; ++w) {
        start += wave_less[w];
        at += w < wave ? wave_own[w] : 0;
        total += wave_own[w];
    }
    at += start;
    if (own) {
        const bool held = i1 - i0 <= 64 * kHeld;
        for (int64_t i = i0; i < i1; i += 64 * kHeld) {
            if (!held) {
#pragma unroll
                for (int u = 0; u < kHeld; ++u) id[u] = i + 64 * u + lane < i1 ? ids[i + 64 * u + lane] : -1;
            }
#pragma unroll
            for (int u = 0; u < kHeld; ++u) {
                const uint64_t all = __ballot(id[u] == g);
                if (id[u] == g) order[at + __popcll(all & ((uint64_t(1) << lane) - 1))] = static_cast<int>(i + 64 * u + lane);
                at += __popcll(all);
            }
        }
    }
    const Segment seg = {start, total};
    if (tid == 0) segs[g] = seg;
    const int s0 = first_slot(seg, g, block);
    const int s1 = g + 1 < count ? first_slot(Segment{start + total, 0}, g + 1, block) : n_slots;
    for (int s = s0 + tid; s < s1; s += 1024) {
        const int done = (s - s0) * block;
        const int len = max(0, min(block, total - done));
        slots[s] = Slot{g, start + done, len, 0};
    }
}

// A value at row `row` of a matrix, 0 where the place is outside.
template <typename T>
__device__ __forceinline__ float value_at(const T* p, int64_t row, int64_t width, int col, bool inside) {
    const float x = to_f32(p[inside ? row * width + col : 0]);
    return inside ? x : 0.0f;
}

// Partial E and dB of one block of rows and 256 columns of dY. RT: tiles of 16
// ranks; blockIdx.z: which group of 16 RT ranks.
//
// dY goes through LDS in tiles of 64 x 64, the next tile's loads in flight
// while this one is multiplied. A wave takes 16 rows of the tile for E (inner
// index: the columns, 16 lg + j for lane group lg) and 16 columns for dB (inner
// index: the rows, 4 j + lg).
// PAST: dY goes past the last cache.
template <typename TW, int RT, bool PAST>
__global__ __launch_bounds__(kThreads) void grad_y_kernel(const float* dY, const TW* B, const float* H,
                                                          const float* scale, const int* order, const Slot* slots,
                                                          int64_t batch, int n_out, int rank, unsigned splits, float* e_part,
                                                          float* db_part) {
    constexpr int kR = 16 * RT + 1;
    constexpr int kB = 16 * RT + (sizeof(TW) == 4 ? 1 : 2);   // bf16 pairs: an odd number of 4-byte words
    __shared__ __align__(16) float tile[64 * kPitch];
    __shared__ __align__(4) TW bt[kColsY * kB];         // B[o][r], all columns of the workgroup
    __shared__ float ht[64 * kR];          // H[n][r], the row tile's
    __shared__ int row_of[kMaxRows];
    // neighbouring workgroups take neighbouring columns of the same rows
    const int split = blockIdx.x % splits, slot = blockIdx.x / splits;
    const Slot s = slots[slot];
    if (s.len == 0) return;
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64, li = lane % 16, lg = lane / 16;
    const int r0 = blockIdx.z * 16 * RT, base = split * kColsY;
    const TW* b = B + static_cast<int64_t>(s.adapter) * n_out * rank;
    const bool wide = n_out % 4 == 0 && reinterpret_cast<uintptr_t>(dY) % 16 == 0;
    const float factor = scale[s.adapter];
    const int row_tiles = (s.len + 63) / 64, col_tiles = min(kColsY / 64, (n_out - base + 63) / 64);
    for (int i = tid; i < kMaxRows; i += kThreads) row_of[i] = order[s.start + min(i, s.len - 1)];
    __syncthreads();
    // thread: rows tid / 16 + 16 q of a tile, four columns from 4 (tid % 16)
    float next[4][4], hnext[4 * RT];
    auto load = [&](int rt, int ct) {
        const int o = base + ct * 64 + 4 * (tid % 16);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int at = rt * 64 + tid / 16 + 16 * q;
            const float* src = dY + static_cast<int64_t>(row_of[at]) * n_out + o;
            const int valid = at < s.len ? n_out - o : 0;
            if (wide && valid >= 4) {
                const f32x4 v = PAST ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(src))
                                     : *reinterpret_cast<const f32x4*>(src);
#pragma unroll
                for (int i = 0; i < 4; ++i) next[q][i] = v[i];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) next[q][i] = i < valid ? src[i] : 0.0f;
            }
        }
        if (ct == 0 && db_part) {
#pragma unroll
            for (int q = 0; q < 4 * RT; ++q) {
                const int n = (q * kThreads + tid) / (16 * RT), r = (q * kThreads + tid) % (16 * RT);
                const int at = rt * 64 + n;
                hnext[q] = value_at(H, row_of[at], rank, r0 + r, at < s.len && r0 + r < rank);
            }
        }
    };
    f32x4 d[kColsY / 64][RT];
#pragma unroll
    for (int c = 0; c < kColsY / 64; ++c)
#pragma unroll
        for (int t = 0; t < RT; ++t) d[c][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    load(0, 0);
    // B of all columns: 16-byte vectors of ranks where they are whole
    constexpr int kV = 16 / static_cast<int>(sizeof(TW)), kVecs = kColsY * 16 * RT / kV / kThreads;
    if (rank % kV == 0 && reinterpret_cast<uintptr_t>(B) % 16 == 0) {
        u32x4 w[kVecs];
#pragma unroll
        for (int q = 0; q < kVecs; ++q) {
            const int v = q * kThreads + tid, o = v / (16 * RT / kV), r = v % (16 * RT / kV) * kV;
            const bool in = base + o < n_out && r0 + r < rank;
            w[q] = *reinterpret_cast<const u32x4*>(b + (in ? static_cast<int64_t>(base + o) * rank + r0 + r : 0));
            if (!in) w[q] = u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int q = 0; q < kVecs; ++q) {
            const int v = q * kThreads + tid, o = v / (16 * RT / kV), r = v % (16 * RT / kV) * kV;
            uint32_t* dst = reinterpret_cast<uint32_t*>(bt + o * kB + r);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = w[q][i];
        }
    } else {
#pragma unroll 8
        for (int i = tid; i < kColsY * 16 * RT; i += kThreads) {
            const int o = i / (16 * RT), r = i % (16 * RT);
            const bool in = base + o < n_out && r0 + r < rank;
            const TW w = b[in ? static_cast<int64_t>(base + o) * rank + r0 + r : 0];
            bt[o * kB + r] = in ? w : TW(0);
        }
    }
    for (int rt = 0; rt < row_tiles; ++rt) {
        f32x4 e[RT];
        float hv[RT][16];                  // H with inner index n, for all column tiles
#pragma unroll
        for (int t = 0; t < RT; ++t) e[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ct = 0; ct < kColsY / 64; ++ct) {
            if (ct >= col_tiles) break;
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4*>(tile + (tid / 16 + 16 * q) * kPitch + 4 * (tid % 16)) =
                    f32x4{next[q][0], next[q][1], next[q][2], next[q][3]};
            if (ct == 0 && db_part) {
#pragma unroll
                for (int q = 0; q < 4 * RT; ++q)
                    ht[(q * kThreads + tid) / (16 * RT) * kR + (q * kThreads + tid) % (16 * RT)] = hnext[q];
            }
            __syncthreads();
            if (ct + 1 < col_tiles) load(rt, ct + 1);
            else if (rt + 1 < row_tiles) load(rt + 1, 0);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(tile + (16 * wave + li) * kPitch + 16 * lg + 4 * q);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        e[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                            x[j], to_f32(bt[(ct * 64 + 16 * lg + 4 * q + j) * kB + 16 * t + li]), e[t], 0, 0, 0);
            }
            if (db_part) {
                if (ct == 0) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
#pragma unroll
                        for (int t = 0; t < RT; ++t) hv[t][j] = ht[(4 * j + lg) * kR + 16 * t + li];
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float x = tile[(4 * j + lg) * kPitch + 16 * wave + li];
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        d[ct][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(x, hv[t][j], d[ct][t], 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = rt * 64 + 16 * wave + 4 * lg + i, r = r0 + 16 * t + li;
                if (at < s.len && r < rank)
                    e_part[(static_cast<int64_t>(split) * batch + s.start + at) * rank + r] = factor * e[t][i];
            }
    }
    if (!db_part) return;
#pragma unroll
    for (int ct = 0; ct < kColsY / 64; ++ct)
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int o = base + ct * 64 + 16 * wave + 4 * lg + i, r = r0 + 16 * t + li;
                if (o < n_out && r < rank)
                    db_part[(static_cast<int64_t>(slot) * n_out + o) * rank + r] = d[ct][t][i];
            }
}

// Orders the wave's LDS accesses before and after it: its lanes exchange values.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// dX and partial dA of one block of rows and 64 columns of X, in tiles of
// 64 x 64. X goes through LDS for dA (inner index: the rows; a wave takes 16
// columns); for dX a wave takes 16 rows, forms its product with the columns
// along the instruction's rows and turns it in LDS, so that dX is read and
// written in runs of 256 bytes. (Two waves a SIMD at least: without that bound the
// compiler takes more registers, 38 us against 27 at 25216 x 384 in fp32.)
template <typename TX, typename TW, int RT>
__global__ __launch_bounds__(kThreads, 2) void grad_x_kernel(const TX* X, const TW* A, const float* E, const int* order,
                                                          const Slot* slots, int n_in, int rank, unsigned splits,
                                                          float* dX, float* da_part) {
    constexpr int kR = 16 * RT + 1, kTiles = kColsX / 64, kTurn = 68;
    __shared__ __align__(16) float tile[64 * kPitch];   // X; after its use for dA, a quarter for each wave's turn
    __shared__ float et[64 * kR];                       // E[n][r] of the row tile
    __shared__ int row_of[kMaxRows];
    const int split = blockIdx.x % splits, slot = blockIdx.x / splits;
    const Slot s = slots[slot];
    if (s.len == 0) return;
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64, li = lane % 16, lg = lane / 16;
    const TW* a = A + static_cast<int64_t>(s.adapter) * rank * n_in;
    const bool wide_x = n_in % 4 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0;
    const bool wide_d = n_in % 4 == 0 && reinterpret_cast<uintptr_t>(dX) % 16 == 0;
    const int row_tiles = (s.len + 63) / 64, base = split * kColsX;
    const int col_tiles = min(kTiles, (n_in - base + 63) / 64);
    for (int i = tid; i < kMaxRows; i += kThreads) row_of[i] = order[s.start + min(i, s.len - 1)];
    __syncthreads();
    for (int r0 = 0; r0 < rank; r0 += 16 * RT) {
        // A[r][k], inner index r, of both column tiles
        float av[kTiles][4][RT][4];
        if (dX) {
#pragma unroll
            for (int ct = 0; ct < kTiles; ++ct)
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int t = 0; t < RT; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = r0 + 16 * t + 4 * lg + j, k = base + ct * 64 + 16 * c + li;
                            av[ct][c][t][j] = value_at(a, r, n_in, k, r < rank && k < n_in);
                        }
        }
        // thread: rows tid / 16 + 16 q of a tile, four columns from 4 (tid % 16)
        float next[4][4], enext[4 * RT];
        auto load = [&](int rt, int ct) {
            if (ct == 0) {
#pragma unroll
                for (int q = 0; q < 4 * RT; ++q) {
                    const int n = (q * kThreads + tid) / (16 * RT), r = r0 + (q * kThreads + tid) % (16 * RT);
                    const int at = rt * 64 + n;
                    enext[q] = value_at(E, s.start + at, rank, r, at < s.len && r < rank);
                }
            }
            if (!da_part) return;
            const int k = base + ct * 64 + 4 * (tid % 16);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int at = rt * 64 + tid / 16 + 16 * q;
                const TX* src = X + static_cast<int64_t>(row_of[at]) * n_in + k;
                const int valid = at < s.len ? n_in - k : 0;
                if (wide_x && valid >= 4) {
                    load4_f32(src, next[q]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) next[q][i] = i < valid ? to_f32(src[i]) : 0.0f;
                }
            }
        };
        f32x4 d[kTiles][RT];
#pragma unroll
        for (int c = 0; c < kTiles; ++c)
#pragma unroll
            for (int t = 0; t < RT; ++t) d[c][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        load(0, 0);
        for (int rt = 0; rt < row_tiles; ++rt) {
#pragma unroll
            for (int ct = 0; ct < kTiles; ++ct) {
                if (ct >= col_tiles) break;
                // this wave's rows of dX, four runs of 256 bytes
                f32x4 y[4];
                const int k = base + ct * 64 + 4 * li;
                if (dX) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int at = rt * 64 + 16 * wave + 4 * q + lg;
                        const float* src = dX + static_cast<int64_t>(row_of[at]) * n_in + k;
                        const int valid = at < s.len ? n_in - k : 0;
                        y[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                        if (wide_d && valid >= 4) {
                            y[q] = *reinterpret_cast<const f32x4*>(src);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (i < valid) y[q][i] = src[i];
                        }
                    }
                }
                __syncthreads();
                if (da_part) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<f32x4*>(tile + (tid / 16 + 16 * q) * kPitch + 4 * (tid % 16)) =
                            f32x4{next[q][0], next[q][1], next[q][2], next[q][3]};
                }
                if (ct == 0) {
#pragma unroll
                    for (int q = 0; q < 4 * RT; ++q)
                        et[(q * kThreads + tid) / (16 * RT) * kR + (q * kThreads + tid) % (16 * RT)] = enext[q];
                }
                __syncthreads();
                if (ct + 1 < col_tiles) load(rt, ct + 1);
                else if (rt + 1 < row_tiles) load(rt + 1, 0);
                if (da_part) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float x = tile[(4 * j + lg) * kPitch + 16 * wave + li];
#pragma unroll
                        for (int t = 0; t < RT; ++t)
                            d[ct][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(et[(4 * j + lg) * kR + 16 * t + li], x,
                                                                            d[ct][t], 0, 0, 0);
                    }
                }
                if (dX) {
                    if (da_part) __syncthreads();
                    float* cross = tile + wave * 16 * kPitch;
                    f32x4 sum[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) sum[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int t = 0; t < RT; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float ev = et[(16 * wave + li) * kR + 16 * t + 4 * lg + j];
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                sum[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[ct][c][t][j], ev, sum[c], 0, 0, 0);
                        }
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<f32x4*>(cross + li * kTurn + 16 * c + 4 * lg) = sum[c];
                    wave_fence();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int at = rt * 64 + 16 * wave + 4 * q + lg;
                        const f32x4 add = *reinterpret_cast<const f32x4*>(cross + (4 * q + lg) * kTurn + 4 * li);
                        float* dst = dX + static_cast<int64_t>(row_of[at]) * n_in + k;
                        const int valid = at < s.len ? n_in - k : 0;
                        if (wide_d && valid >= 4) {
                            *reinterpret_cast<f32x4*>(dst) = y[q] + add;
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (i < valid) dst[i] = y[q][i] + add[i];
                        }
                    }
                    wave_fence();
                }
            }
        }
        if (da_part) {
#pragma unroll
            for (int ct = 0; ct < kTiles; ++ct)
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = r0 + 16 * t + 4 * lg + i;
                        const int k = base + ct * 64 + 16 * wave + li;
                        if (r < rank && k < n_in)
                            da_part[(static_cast<int64_t>(slot) * rank + r) * n_in + k] = d[ct][t][i];
                    }
        }
        __syncthreads();   // the next ranks' tiles go over these
    }
}

// n values `stride` apart, added in order; eight loads in flight.
__device__ __forceinline__ float sum_of(const float* p, int64_t stride, int n) {
    float sum = 0.0f;
    int i = 0;
    for (; i + 8 <= n; i += 8) {
        float x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = p[(i + u) * stride];
#pragma unroll
        for (int u = 0; u < 8; ++u) sum += x[u];
    }
    for (; i < n; ++i) sum += p[i * stride];
    return sum;
}

// Gradient of the adapters' weights (`size` values each): the sum over an
// adapter's blocks of rows, zeros without any; and, in the workgroups past
// those (part_e not NULL), E as the sum over the column ranges: `planes` of
// `n_e` values.
__global__ __launch_bounds__(kThreads) void sum_kernel(const float* part, const Segment* segs, int64_t size, int block,
                                                       int per_adapter, int count, float* out, const float* part_e,
                                                       int64_t n_e, int planes, float* E) {
    const int64_t wg = blockIdx.x, weights = static_cast<int64_t>(per_adapter) * count;
    if (wg >= weights) {
        const int64_t i = (wg - weights) * kThreads + threadIdx.x;
        if (i < n_e) E[i] = sum_of(part_e + i, n_e, planes);
        return;
    }
    const int g = static_cast<int>(wg / per_adapter);
    const int64_t i = wg % per_adapter * kThreads + threadIdx.x;
    if (i >= size) return;
    const Segment seg = segs[g];
    out[g * size + i] = sum_of(part + first_slot(seg, g, block) * size + i, size, (seg.len + block - 1) / block);
}

// ---------------------------------------------------------------- few rows

constexpr int kFewThreads = 1024;

// E and dX of one row a workgroup: E[r] = scale sum_o dY[o] B[o][r], then
// dX[k] += sum_r E[r] A[r][k]. A thread takes eight ranks of every so many
// outputs (16-byte loads of B with WIDE); the threads' sums of a rank are added
// in LDS, sixteen at a time, in a fixed order.
template <typename TW, bool WIDE>
__global__ __launch_bounds__(kFewThreads) void few_rows_kernel(const float* dY, const TW* A, const TW* B,
                                                               const float* scale, const int32_t* ids, int n_in,
                                                               int n_out, int rank, int count, float* E, float* dX) {
    __shared__ float part[kFewThreads * 9];
    __shared__ float part2[16 * KS_ADAPTER_MAX_RANK];
    __shared__ float e[KS_ADAPTER_MAX_RANK];
    const int64_t n = blockIdx.x;
    const int g = adapter_of(ids[n], count), tid = threadIdx.x;
    if (g < 0) return;                                 // nothing reads its E
    const TW* a = A + static_cast<int64_t>(g) * rank * n_in;
    const TW* b = B + static_cast<int64_t>(g) * n_out * rank;
    const float* dy = dY + n * n_out;
    const int eights = (rank + 7) / 8, groups = kFewThreads / eights;
    const int r8 = tid % eights * 8, group = tid / eights;
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (group < groups) {
#pragma unroll 4
        for (int o = group; o < n_out; o += groups) {
            const float y = dy[o];
            float x[8];
            load8<WIDE>(b + static_cast<int64_t>(o) * rank + r8, rank - r8, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += y * x[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[tid * 9 + i] = acc[i];
    __syncthreads();
    for (int v = tid; v < 16 * rank; v += kFewThreads) {
        const int r = v % rank, c = v / rank;
        float sum = 0.0f;
        for (int q = c; q < groups; q += 16) sum += part[(q * eights + r / 8) * 9 + r % 8];
        part2[c * rank + r] = sum;
    }
    __syncthreads();
    if (tid < rank) {
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < 16; ++c) sum += part2[c * rank + tid];
        e[tid] = scale[g] * sum;
        E[n * rank + tid] = e[tid];
    }
    __syncthreads();
    if (!dX) return;
    for (int k = tid; k < n_in; k += kFewThreads) {
        float sum = dX[n * n_in + k];
#pragma unroll 8
        for (int r = 0; r < rank; ++r) sum += e[r] * to_f32(a[static_cast<int64_t>(r) * n_in + k]);
        dX[n * n_in + k] = sum;
    }
}

// dA and dB of one adapter and 256 columns: a thread a column, sixteen ranks at a
// time, over the adapter's rows in order, eight loads in flight. blockIdx.x: the adapter; blockIdx.y:
// column groups of X, then of dY.
template <typename TX>
__global__ __launch_bounds__(kThreads) void few_weights_kernel(const float* dY, const TX* X, const float* H,
                                                               const float* E, const int32_t* ids, int batch, int n_in,
                                                               int n_out, int rank, float* dA, float* dB) {
    __shared__ int row_of[kFewRows + 1], wave_rows[4];
    __shared__ __attribute__((aligned(16))) float low[(kFewRows + 7) / 8 * 8 * 16 + 16];
    const int g = blockIdx.x, tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    int rows = 0;
    for (int i0 = 0; i0 < batch; i0 += kThreads) {
        const bool mine = i0 + tid < batch && ids[i0 + tid] == g;
        const uint64_t all = __ballot(mine);
        if (lane == 0) wave_rows[wave] = __popcll(all);
        __syncthreads();
        int at = rows + __popcll(all & ((uint64_t(1) << lane) - 1));
        for (int w = 0; w < 4; ++w) {
            at += w < wave ? wave_rows[w] : 0;
            rows += wave_rows[w];
        }
        if (mine) row_of[at] = i0 + tid;
        __syncthreads();
    }
    const int groups_in = (n_in + kThreads - 1) / kThreads;
    const bool first = static_cast<int>(blockIdx.y) < groups_in;
    const int col = (first ? blockIdx.y : blockIdx.y - groups_in) * kThreads + tid, width = first ? n_in : n_out;
    const float* other = first ? E : H;
    for (int r0 = 0; r0 < rank; r0 += 16) {
        __syncthreads();
        for (int v = tid; v < (rows + 7) / 8 * 8 * 16; v += kThreads) {
            const int i = v / 16, r = r0 + v % 16;
            low[v] = i < rows && r < rank ? other[static_cast<int64_t>(row_of[i]) * rank + r] : 0.0f;
        }
        __syncthreads();
        float acc[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
        for (int i0 = 0; i0 < rows; i0 += 8) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t at = static_cast<int64_t>(row_of[min(i0 + i, rows - 1)]) * width + min(col, width - 1);
                x[i] = first ? to_f32(X[at]) : dY[at];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xi = i0 + i < rows ? x[i] : 0.0f;
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[r] += xi * low[(i0 + i) * 16 + r];
            }
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            if (r0 + r >= rank || col >= width) break;
            if (first) dA[(static_cast<int64_t>(g) * rank + r0 + r) * n_in + col] = acc[r];
            else dB[(static_cast<int64_t>(g) * n_out + col) * rank + r0 + r] = acc[r];
        }
    }
}

template <typename TX, typename TW>
ks_status_t run_few(const AdapterCall& c, const float* dY, const void* X, const float* H, float* dX, float* dA,
                    float* dB, void* ws) {
    float* E = static_cast<float*>(ws);
    const bool wide = c.rank % 8 == 0 && reinterpret_cast<uintptr_t>(c.B) % 16 == 0;
    if (c.batch > 0) {
        const ks_status_t st = launch_kernel(
            wide ? few_rows_kernel<TW, true> : few_rows_kernel<TW, false>, dim3(static_cast<unsigned>(c.batch)),
            dim3(kFewThreads), 0, c.stream, dY, static_cast<const TW*>(c.A), static_cast<const TW*>(c.B), c.scale,
            c.ids, c.n_in, c.n_out, c.rank, c.count, E, dX);
        if (st != KS_OK) return st;
    }
    if (!dA) return KS_OK;
    const unsigned groups =
        static_cast<unsigned>((c.n_in + kThreads - 1) / kThreads + (c.n_out + kThreads - 1) / kThreads);
    return launch_kernel(few_weights_kernel<TX>, dim3(static_cast<unsigned>(c.count), groups), dim3(kThreads), 0,
                         c.stream, dY, static_cast<const TX*>(X), H, E, c.ids, static_cast<int>(c.batch), c.n_in,
                         c.n_out, c.rank, dA, dB);
}

// ---------------------------------------------------------------- many rows

// Few rows: two launches. The weights' one walks an adapter's rows for every
// sixteen ranks, 0.3 us a row, in place of three more launches, so the limit is on
// rows times those passes. A call from the host, 1024 x 4096, against the sorted
// path: 64 rows of rank 16, 22 us against 34 with 16 adapters and 26 against 32
// with one; 128 rows 22 against 36 and 42 against 32. The column groups are a
// grid's second dimension.
bool few_rows(int n_in, int n_out, int rank, int64_t batch) {
    return batch * ((rank + 15) / 16) <= kFewRows &&
           (n_in + kThreads - 1) / kThreads + (n_out + kThreads - 1) / kThreads <= 65535;
}

struct Layout {
    AdapterOrder o;
    size_t e, e_part, w_part, total;
    int splits;
};

// Rows of a block: as many as leave the passes about two and one workgroups a
// compute unit of the card's 256 (fewer partial sums against loads in flight).
int block_rows(int n_in, int n_out, int64_t batch) {
    int block = kMaxRows;
    while (block > 64 && (batch / block * ((n_out + kColsY - 1) / kColsY) < 512 ||
                          batch / block * ((n_in + kColsX - 1) / kColsX) < 256))
        block /= 2;
    return block;
}

Layout layout_of(int n_in, int n_out, int rank, int count, int64_t batch, char* ws) {
    Layout l;
    size_t at = adapter_order_layout(batch, block_rows(n_in, n_out, batch), count, ws, &l.o);
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    l.splits = (n_out + kColsY - 1) / kColsY;
    l.e = take(static_cast<size_t>(batch) * rank * 4);
    l.e_part = take(l.splits > 1 ? static_cast<size_t>(l.splits) * batch * rank * 4 : 0);
    // dB's partial sums are added before dA's are written
    l.w_part = take(static_cast<size_t>(l.o.n_slots) * rank * std::max(n_in, n_out) * 4);
    l.total = at;
    return l;
}

template <typename TX, typename TW, int RT>
ks_status_t run(const AdapterCall& c, const float* dY, const void* X, const float* H, float* dX, float* dA, float* dB,
                char* ws) {
    const Layout l = layout_of(c.n_in, c.n_out, c.rank, c.count, c.batch, ws);
    const int* order = l.o.order;
    const Segment* segs = l.o.segs;
    const Slot* slots = l.o.slots;
    float* E = reinterpret_cast<float*>(ws + l.e);
    float* e_part = l.splits > 1 ? reinterpret_cast<float*>(ws + l.e_part) : E;
    float* w_part = reinterpret_cast<float*>(ws + l.w_part);
    const TW* A = static_cast<const TW*>(c.A);
    const TW* B = static_cast<const TW*>(c.B);
    ks_status_t st = launch_adapter_order(c, l.o);
    if (st != KS_OK) return st;
    // one launch for dB (or dA) and, with planes > 1, for E
    auto sum = [&](int64_t size, float* out, int planes) {
        const int64_t per = out ? (size + kThreads - 1) / kThreads : 0, n_e = planes > 1 ? c.batch * c.rank : 0;
        const int64_t blocks = per * c.count + (n_e + kThreads - 1) / kThreads;
        if (blocks == 0) return KS_OK;
        return launch_kernel(sum_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, c.stream, w_part, segs,
                             size, l.o.block, static_cast<int>(per), out ? c.count : 0, out, e_part, n_e, planes, E);
    };
    if (c.batch > 0) {
        const dim3 gy(static_cast<unsigned>(l.o.n_slots) * l.splits, 1,
                      static_cast<unsigned>((c.rank + 16 * RT - 1) / (16 * RT)));
        // a dY that the last cache cannot hold goes past it (16384 x 4096: 130 us a
        // call, 155 through it; smaller ones are there from the projection's pass)
        const bool past_cache = c.batch * c.n_out * 4 > int64_t(192) << 20;
        st = launch_kernel(past_cache ? grad_y_kernel<TW, RT, true> : grad_y_kernel<TW, RT, false>, gy, dim3(kThreads),
                           0, c.stream, dY, B, H, c.scale, order, slots, c.batch, c.n_out, c.rank,
                           static_cast<unsigned>(l.splits), e_part, dB ? w_part : static_cast<float*>(nullptr));
        if (st != KS_OK) return st;
    }
    st = sum(static_cast<int64_t>(c.n_out) * c.rank, dB, c.batch > 0 ? l.splits : 0);
    if (st != KS_OK) return st;
    if (c.batch > 0) {
        const unsigned splits = static_cast<unsigned>((c.n_in + kColsX - 1) / kColsX);
        const dim3 gx(static_cast<unsigned>(l.o.n_slots) * splits);
        st = launch_kernel(grad_x_kernel<TX, TW, RT>, gx, dim3(kThreads), 0, c.stream, static_cast<const TX*>(X), A, E,
                           order, slots, c.n_in, c.rank, splits, dX, dA ? w_part : static_cast<float*>(nullptr));
        if (st != KS_OK) return st;
    }
    return sum(static_cast<int64_t>(c.n_in) * c.rank, dA, 0);
}

template <typename TX, typename TW>
ks_status_t run_rank(const AdapterCall& c, const float* dY, const void* X, const float* H, float* dX, float* dA,
                     float* dB, char* ws) {
    if (c.rank <= 16) return run<TX, TW, 1>(c, dY, X, H, dX, dA, dB, ws);
    return run<TX, TW, 2>(c, dY, X, H, dX, dA, dB, ws);
}

}  // namespace

size_t adapter_order_layout(int64_t batch, int block, int count, char* ws, AdapterOrder* out) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* here = ws ? ws + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    out->block = block;
    out->n_slots = adapter_slots(batch, block, count);
    out->order = reinterpret_cast<int*>(take(static_cast<size_t>(batch) * 4));
    out->segs = reinterpret_cast<Segment*>(take(static_cast<size_t>(count) * sizeof(Segment)));
    out->slots = reinterpret_cast<Slot*>(take(static_cast<size_t>(out->n_slots) * sizeof(Slot)));
    return at;
}

ks_status_t launch_adapter_order(const AdapterCall& c, const AdapterOrder& o) {
    return launch_kernel(sort_kernel, dim3(static_cast<unsigned>(c.count)), dim3(1024), 0, c.stream, c.ids,
                         static_cast<int>(c.batch), c.count, o.block, o.order, o.segs, o.slots, o.n_slots);
}

bool adapter_grad_fits(int n_in, int n_out, int rank, int count, int64_t batch) {
    if (few_rows(n_in, n_out, rank, batch)) return true;
    // a grid counts its threads in 32 bits: 2^24 workgroups of 256 are one too many
    const int64_t most = (int64_t(1) << 24) - 1, wide = std::max(n_in, n_out);
    const int64_t slots = adapter_slots(batch, block_rows(n_in, n_out, batch), count);
    return slots * ((wide + kColsX - 1) / kColsX) <= most &&
           (wide * rank + kThreads - 1) / kThreads * count + (batch * rank + kThreads - 1) / kThreads <= most;
}

size_t adapter_grad_workspace(int n_in, int n_out, int rank, int count, int64_t batch) {
    if (few_rows(n_in, n_out, rank, batch)) return static_cast<size_t>((batch * rank * 4 + 255) / 256 * 256);
    return layout_of(n_in, n_out, rank, count, batch, nullptr).total;
}

ks_status_t launch_adapter_grad(const AdapterCall& c, const float* dY, const void* X, const float* H, float* dX,
                                float* dA, float* dB, void* ws) {
    if (few_rows(c.n_in, c.n_out, c.rank, c.batch)) {
        if (c.xt == kBF16) return run_few<bf16_t, bf16_t>(c, dY, X, H, dX, dA, dB, ws);
        if (c.wt == kBF16) return run_few<float, bf16_t>(c, dY, X, H, dX, dA, dB, ws);
        return run_few<float, float>(c, dY, X, H, dX, dA, dB, ws);
    }
    char* w = static_cast<char*>(ws);
    if (c.xt == kBF16) return run_rank<bf16_t, bf16_t>(c, dY, X, H, dX, dA, dB, w);
    if (c.wt == kBF16) return run_rank<float, bf16_t>(c, dY, X, H, dX, dA, dB, w);
    return run_rank<float, float>(c, dY, X, H, dX, dA, dB, w);
}

}  // namespace ks
