// ks_fused.hip -- two KS factors in one launch, the intermediate kept in LDS.
//
// Chains of KS factors are how Butterfly- and Monarch-type layers are built
// (KS abstract page, taxoreview.com "dblp:303/4794", first paragraph). A pair
// F0 = (1, b0, c0, d0) followed by F1 = (a1, b1, c1, d1) with a1 = b0 and
// c1 * d1 = d0 has a simple joint structure: F1 reads F0's output row
// Z[beta0][delta0] as Z[alpha1][gamma1][delta1], i.e. alpha1 = beta0 and
// delta0 = gamma1 * d1 + delta1. Hence a fixed set of beta0 values (= alpha1
// values) needs all of X's row, produces a contiguous slab of Y's row
// (Y[alpha1][beta1][delta1]), and touches only its own slices of both weight
// tensors. The GPT-2-medium MLP shape (1, 64, 16, 64) -> (64, 8, 8, 8) is of
// this kind.
//
// Workgroup: BT consecutive beta0 (= alpha1) values (32, 16 or 8, the
// largest that divides b0) and a range of rows; one loader wave streams whole
// rows of X into an LDS ring (ks_stream.h), each row followed by 32 bytes of
// padding so that the four rows a matrix-core instruction reads start in
// different banks; the b0 / BT workgroups that share rows run on the same
// XCD, so X is fetched from HBM once and served to the others from L2. Per
// stage of 4 rows, eight consumer waves
//  (A) compute Z[r][beta0][delta0] into LDS on the matrix cores: for a fixed
//      delta0 it is a (rows x c0) by (c0 x beta0) product, and the 16-block
//      4x4x1 fp32 MFMA does 16 such delta0 at once (weights in registers),
//  (B) compute Y[r][alpha1][beta1][delta1] of the previous stage from the
//      other Z buffer on the VALU: runs of 4 delta1 per thread (c1 FMAs per
//      value, weights in registers), stored as 16-byte vectors.
// One LDS barrier per stage separates the two. A wide tile (BT = 32 for
// GPT-2-medium's b0 = 64) cuts the L2 re-reads of X to b0 / BT per row and
// keeps more X bytes in flight per byte of Y than two narrow workgroups
// per compute unit would.
// Z never leaves the chip: the pair moves |X| + |Y| + weights through HBM
// instead of |X| + 2|Z| + |Y|.
//
// Adapters. With bf16 operands the same launch can add the low-rank adapters of
// the rows' requests, Y[n] += H[n] B[g]^T with g = ids[n], H from an earlier launch,
// for stages whose four rows share an adapter or pass once from one to another:
// there Y is written once and never read. H comes as three bf16 values whose sum
// is the fp32 value exactly, so its products with a finite B are those of fp32 (a part
// may be 0: an infinite B can give NaN); the loader
// streams the stage's rows of them and the stage's adapters along with X. A thread of phase B keeps its four outputs'
// values of B in registers, and the products run on the 16-block 4x4x4 bf16 MFMA,
// whose lanes are given their own outputs as the columns: each receives the stage's
// four rows of its own output, which is where phase B has them. Phase A uses the
// same instruction there, four gammas at a time (products of bf16 values are exact
// in fp32): the kernel is bound by its two phases on the chip more than by HBM, and
// that saves 17 us of 16384 rows. With H, 16384 rows take 78 us at rank 16 and 97 at
// 32 (63 for the chain alone); with the adapters added by a pass over Y, 157 and 180.
// Weights stay packed in registers: nine waves leave 168 a wave, and spilled ones
// come back through the vector-memory counter behind the stores.
// Other stages are left to another launch: going through all of a stage's adapters
// here, each loading its B, took 524 us on 16384 rows in random order of 8 adapters,
// 368 now.
//
// Alignment. X and Y need only be aligned to their element size. When X
// starts xshift elements past a 16-byte boundary, the loader streams the
// 16-byte granules that cover each row, from the boundary below it (a
// granule never crosses a page, so the extra bytes are always readable), one
// granule more per row (it lands in the row's padding), and the consumers
// read every element xshift places further on. When Y is not 16-byte
// aligned, phase B stores single elements.

#include <algorithm>
#include <cstdio>

#include "ks_device.h"
#include "ks_internal.h"
#include "ks_stream.h"

namespace ks {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));

// Shape family handled: F0 = (1, b0, 16, 64), F1 = (b0, 8, 8, 8), b0 % 8 == 0.
constexpr int kC0 = 16, kD0 = 64;          // first factor: gamma0, delta0 extents
constexpr int kB1 = 8, kC1 = 8, kD1 = 8;   // second factor: beta1, gamma1, delta1 extents
constexpr int kRows = 4;                   // rows per stage
constexpr int kXPadBytes = 32;             // LDS pad after each row of X: rows start 8 banks apart
constexpr int kZPitch = kD0 + 8;           // Z pitch per beta0 (floats): beta0 neighbours 8 banks apart
constexpr int kZBufs = 2;                  // Z double buffer: phase B of stage s - 1 runs beside phase A of stage s
constexpr int kFusedConsumers = 8;         // consumer waves per workgroup
constexpr int kFusedThreads = kFusedConsumers * 64 + 64;   // + one loader wave

// Geometry of a tile of BT beta0 (= alpha1) values.
template <int BT>
struct FusedTile {
    static constexpr int kZRow = BT * kZPitch + 8;       // Z pitch per row (floats): rows 8 banks apart
    static constexpr int kZFloats = kRows * kZRow;       // one Z buffer
    static constexpr int kSetsPerWave = BT / kFusedConsumers;   // phase A: groups of 4 beta0 per wave
    static constexpr int kRowsPerPass = kFusedConsumers * 64 / (BT * kB1 * 2);   // phase B: rows per pass
    static_assert(BT == 8 || BT == 16 || BT == 32, "tile widths");
    static_assert(kRowsPerPass >= 1 && kRows % kRowsPerPass == 0 && (kZPitch * 4) % 16 == 0 &&
                      (kZRow * 4) % 16 == 0,
                  "phase B covers whole rows per pass, Z in 16-byte runs");
    // phase A: wave w takes delta0 in [16 (w % 4), +16) and the beta0 groups
    // [(w / 4) * kSetsPerWave * 4, +kSetsPerWave * 4)
    static_assert(kRows == 4 && kD0 == 64 && kFusedConsumers == 8 && (kFusedConsumers / 4) * kSetsPerWave * 4 == BT,
                  "phase A: 4x4 MFMA blocks of rows x beta0, 16 delta0 per block group");
};

static_assert(kRows == kPairGroup, "an adapter a stage");

// Loader instructions (1 KB each) for one stage of rows of elem_bytes-wide
// elements with kXPadBytes after each row.
constexpr int stage_insts(int eb) { return (kRows * (kC0 * kD0 * eb + kXPadBytes) + 1023) / 1024; }
constexpr int stage_bytes(int eb) { return stage_insts(eb) * 1024; }
constexpr int kStagesF32 = 3;              // LDS ring depth for fp32 rows
constexpr int kStagesBF16 = 4;             // ... and for bf16 rows (half the bytes)
constexpr int stages_for(int eb) { return eb == 4 ? kStagesF32 : kStagesBF16; }
// With adapters, a ring of the stages' rows of H and ids, one loader instruction
// each. Phase B reads them one stage after phase A has read X: one slot more.
constexpr int kLowBytes = 1024 + 256;
constexpr size_t fused_lds_bytes(int eb, int bt, bool low) {
    return size_t(stages_for(eb)) * stage_bytes(eb) + (low ? size_t(stages_for(eb) + 1) * kLowBytes : 0) +
           size_t(kZBufs) * kRows * (bt * kZPitch + 8) * sizeof(float);
}

struct FusedArgs {
    int b0;                 // beta0 extent (= alpha1 extent)
    int64_t n_in, n_mid, n_out;
    int64_t batch;
    int n_tiles;            // b0 / BT
    int rows_per_split;     // multiple of kRows
    int xshift;             // elements from the 16-byte boundary below X to X (the same in every row)
};

// N weights of a thread: fp32 values, or the packed words of bf16 ones, widened
// where they are used (hold: widened once, ahead of the loop over the stages, they
// would take twice the registers).
template <int N, bool PACKED>
struct Weights {
    float v[N];
    template <typename TW>
    __device__ __forceinline__ void load(const TW* p) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = to_f32(p[i]);
    }
    __device__ __forceinline__ float at(int i) const { return v[i]; }
    __device__ __forceinline__ void hold() {}
};
typedef short short4v __attribute__((ext_vector_type(4)));
__device__ __forceinline__ short4v four_bf16(uint32_t lo, uint32_t hi) {
    return __builtin_bit_cast(short4v, uint64_t(lo) | uint64_t(hi) << 32);
}
template <int N>
struct Weights<N, true> {
    uint32_t w[N / 2];
    __device__ __forceinline__ void load(const bf16_t* p) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = uint32_t(p[2 * i]) | uint32_t(p[2 * i + 1]) << 16;
    }
    __device__ __forceinline__ float at(int i) const { return i % 2 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]); }
    __device__ __forceinline__ void hold() {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) asm volatile("" : "+v"(w[i]));
    }
    __device__ __forceinline__ short4v four(int c) const { return four_bf16(w[2 * c], w[2 * c + 1]); }
};

// The byte limit of issue_stage when rows start xshift elements past a
// 16-byte boundary: the granule holding the last elements of the stage's last
// row is one past the usual limit.
__device__ __forceinline__ uint32_t shifted_limit(uint32_t limit, int xshift) {
    return (xshift == 0 || limit > kNoVector - 16u) ? limit : limit + 16u;
}

// kYVec: Y is 16-byte aligned (vector stores in phase B); BT: beta0 per tile;
// RT: tiles of 16 ranks of adapters that are added (0: none).
template <typename TX, typename TW, bool kYVec, int BT, int RT>
__device__ __forceinline__ void fused_pair(const TX* __restrict__ X, const TW* __restrict__ K0, const TW* __restrict__ K1,
                                           float* __restrict__ Y, const FusedArgs& args, const PairAdapters& ad) {
    static_assert(RT == 0 || (sizeof(TX) == 2 && sizeof(TW) == 2 && BT == 32), "adapters: bf16, a thread all rows of a stage");
    constexpr int EB = int(sizeof(TX));
    constexpr int VW = 16 / EB;
    constexpr int INSTS = stage_insts(EB);
    constexpr int kLowRow = low_parts_bytes(16 * RT);                  // bytes of a row's parts of H
    constexpr int kLoads = INSTS + (RT > 0 ? 2 : 0);            // loader instructions of a stage
    constexpr int kStageBytes = stage_bytes(EB);
    constexpr int kStages = stages_for(EB);
    constexpr int kRowBytes = kC0 * kD0 * EB + kXPadBytes;   // LDS pitch of a row of X
    using Tile = FusedTile<BT>;
    constexpr int kZRow = Tile::kZRow;
    constexpr int kZFloats = Tile::kZFloats;
    constexpr int kSetsPerWave = Tile::kSetsPerWave;
    constexpr int kRowsPerPass = Tile::kRowsPerPass;
    extern __shared__ __align__(16) unsigned char lds[];
    float* const zs = reinterpret_cast<float*>(lds + kStages * kStageBytes);   // kZBufs x [kRows][BT][kZPitch]
    unsigned char* const lows = reinterpret_cast<unsigned char*>(zs + kZBufs * kZFloats);   // kStages + 1 slots (RT > 0)

    const int t = threadIdx.x;
    const int blk = xcd_logical_block(blockIdx.x, gridDim.x);
    const int tile = blk % args.n_tiles;
    const int split = blk / args.n_tiles;
    const int beta0 = tile * BT;                           // first beta0 (= alpha1) of the tile

    const int64_t row_begin = int64_t(split) * args.rows_per_split;
    if (row_begin >= args.batch) return;
    const int64_t row_end = min(args.batch, row_begin + int64_t(args.rows_per_split));
    const int nsteps = static_cast<int>((row_end - row_begin + kRows - 1) / kRows);

    if (t >= kFusedConsumers * 64) {
        // ------------------------------------------------------ loader wave
        StageMap m;
        m.rows = kRows;
        m.blocks = 1;
        // one whole row of X, and the granule past it when X is not 16-byte
        // aligned (it takes the first vector of the row's padding)
        const int extra = args.xshift != 0 ? 1 : 0;
        m.blk_vec = kC0 * kD0 / VW + extra;
        m.pad_vec = kXPadBytes / 16 - extra;
        m.row_vec = m.blk_vec + m.pad_vec;
        m.gstride = 0;
        LoaderPlan<INSTS> lp;
        make_loader_plan<INSTS>(m, INSTS, VW, EB, args.n_in, 1, m.blk_vec, t - kFusedConsumers * 64, &lp);
        const TX* xbase = X - args.xshift;                 // 16-byte aligned
        auto issue = [&](int s) {
            const int64_t n0 = row_begin + int64_t(s) * kRows;
            issue_stage<INSTS>(lp, INSTS, xbase + n0 * args.n_in,
                               shifted_limit(stage_limit(n0, row_end, args.n_in, EB), args.xshift),
                               lds + (s % kStages) * kStageBytes);
            if constexpr (RT > 0) {
                // the rows' parts of H, one after another, and their adapters; lanes past
                // the last row read its end again, which nobody uses
                const int lane = t - kFusedConsumers * 64;
                unsigned char* low = lows + (s % (kStages + 1)) * kLowBytes;
                const int bytes = static_cast<int>(min(row_end - n0, int64_t(kRows))) * kLowRow;
                __builtin_amdgcn_global_load_lds(
                    reinterpret_cast<const void*>(reinterpret_cast<const char*>(ad.H) + n0 * kLowRow +
                                                  min(lane * 16, bytes - 16)),
                    low, 16, 0, 0);
                __builtin_amdgcn_global_load_lds(
                    reinterpret_cast<const void*>(&ad.groups[n0 / kRows].first + min(lane, 1)), low + 1024, 4, 0, 0);
            }
        };
        for (int s = 0; s < kStages - 1 && s < nsteps; ++s) issue(s);
        for (int s = 0; s <= nsteps; ++s) {
            if (s < nsteps) wait_vmcnt_upto(min(kStages - 2, nsteps - 1 - s) * kLoads);
            lds_barrier();                                   // stage s ready, Z of stage s - 1 written
            if (s + kStages - 1 < nsteps) issue(s + kStages - 1);
        }
        return;
    }

    // ---------------------------------------------------------- consumers
    // Phase A is a batched 4x4 outer product on the matrix cores: in
    // v_mfma_f32_4x4x1f32 lane l belongs to block l / 4, supplies row l % 4
    // of that block's A column and column l % 4 of its B row, and receives
    // D[i][l % 4] of its block in accumulator register i. One instruction
    // per gamma and group of 4 output columns.
    const int lane = t & 63;
    const int wave = t >> 6;
    const int q = lane & 3;                                // A: row; B and D: column within a group of 4
    // (A) block = delta0, A = X[row][gamma0][delta0], B = K0[0][delta0][beta0][gamma0];
    // wave w -> delta0 in [16 (w % 4), 16 (w % 4) + 16) and kSetsPerWave
    // groups of 4 beta0, all kRows rows
    const int a_d0 = 16 * (wave & 3) + (lane >> 2);        // delta0 of this lane's block
    const int a_b0 = (wave >> 2) * kSetsPerWave * 4;       // first beta0 (within the tile) of the wave
    Weights<kC0, (RT > 0)> k0r[kSetsPerWave];
#pragma unroll
    for (int j = 0; j < kSetsPerWave; ++j)                  // K0[0][d0][beta][:]
        k0r[j].load(K0 + (int64_t(a_d0) * args.b0 + beta0 + a_b0 + 4 * j + q) * kC0);

    // (A) Z[r][beta0][d0] = sum_g K0[0][d0][beta0][g] * X[r][g][d0] for stage s
    auto phase_a = [&](int s, float* zb) {
        const unsigned char* xs = lds + (s % kStages) * kStageBytes;
        if constexpr (RT > 0) {
            static_assert(kRows == 4, "one row a lane of a block");
            const TX* xa = reinterpret_cast<const TX*>(xs + q * kRowBytes) + args.xshift + a_d0;
            short4v x[kC0 / 4];
#pragma unroll
            for (int g = 0; g < kC0; ++g) x[g / 4][g % 4] = static_cast<short>(xa[g * kD0]);
            floatx4 z[kSetsPerWave];
#pragma unroll
            for (int j = 0; j < kSetsPerWave; ++j) z[j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < kC0 / 4; ++c)
#pragma unroll
                for (int j = 0; j < kSetsPerWave; ++j)
                    z[j] = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(x[c], k0r[j].four(c), z[j], 0, 0, 0);
#pragma unroll
            for (int j = 0; j < kSetsPerWave; ++j) {
                float* zw = zb + (a_b0 + 4 * j + q) * kZPitch + a_d0;
#pragma unroll
                for (int i = 0; i < 4; ++i) zw[i * kZRow] = z[j][i];
            }
            return;
        } else {
#pragma unroll
        for (int rg = 0; rg < kRows; rg += 4) {
            const TX* xa = reinterpret_cast<const TX*>(xs + (rg + q) * kRowBytes) + args.xshift + a_d0;
            floatx4 z[kSetsPerWave];
#pragma unroll
            for (int j = 0; j < kSetsPerWave; ++j) z[j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int g = 0; g < kC0; ++g) {
                const float x = to_f32(xa[g * kD0]);
#pragma unroll
                for (int j = 0; j < kSetsPerWave; ++j)
                    z[j] = __builtin_amdgcn_mfma_f32_4x4x1f32(x, k0r[j].at(g), z[j], 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < kSetsPerWave; ++j) {
                float* zw = zb + rg * kZRow + (a_b0 + 4 * j + q) * kZPitch + a_d0;   // lane's beta0 and delta0
#pragma unroll
                for (int i = 0; i < 4; ++i) zw[i * kZRow] = z[j][i];
            }
        }
        }
    };

    // one barrier per stage: phase A of stage s and phase B of stage s - 1
    // share an iteration, on alternate Z buffers
    auto pipeline = [&](auto&& phase_b) {
        for (int s = 0; s <= nsteps; ++s) {
            lds_barrier();                                   // stage s ready, Z of stage s - 1 written
            if (s < nsteps) phase_a(s, zs + (s & 1) * kZFloats);
            if (s > 0) phase_b(s - 1, zs + ((s - 1) & 1) * kZFloats);
        }
    };

    // (B) thread -> one row of a pass, (alpha1, beta1) and a run of 4 delta1:
    // lanes in (alpha1, beta1, run) order store 16-byte vectors that tile
    // the row's slab of Y contiguously
    const int rsub = t / (BT * kB1 * 2);               // row within a pass
    const int run = t & 1;
    const int b1 = (t >> 1) & (kB1 - 1);
    const int a1 = (t >> 4) & (BT - 1);                // alpha1 within the tile
    const int e10 = run * 4;                           // first delta1 of the run
    Weights<kC1, (RT > 0)> k1r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)                              // K1[a][e][b][:]
        k1r[k].load(K1 + ((int64_t(beta0 + a1) * kD1 + e10 + k) * kB1 + b1) * kC1);
    const int64_t yoff = int64_t(beta0 + a1) * (kB1 * kD1) + b1 * kD1 + e10;
    // low[k][r]: the adapters' part of output k of the run in row r of the stage. An
    // adapter's B of these four outputs stays from stage to stage.
    uint32_t bw[4][RT > 0 ? 8 * RT : 1];
    int held = -1;
    auto adapters = [&](int s, floatx4 (&low)[4]) {
        const unsigned char* at = lows + (s % (kStages + 1)) * kLowBytes;
        const uint4* h = reinterpret_cast<const uint4*>(at + q * kLowRow);   // of row q: [chunk of 4 ranks][part][4]
        PairGroup rows;
        rows.first = __builtin_amdgcn_readfirstlane(reinterpret_cast<const int*>(at + 1024)[0]);
        rows.second = __builtin_amdgcn_readfirstlane(reinterpret_cast<const int*>(at + 1024)[1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) low[k] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        int g = rows.first, row = 0, end = rows.split();         // rows [row, end) are adapter g's
        for (;;) {
            if (g >= 0) {
                if (g != held) {
                    held = g;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const bf16_t* b = static_cast<const bf16_t*>(ad.B) + (int64_t(g) * args.n_out + yoff + k) * ad.rank;
#pragma unroll
                        for (int w = 0; w < 8 * RT; w += 2) {
                            uint2 v = *reinterpret_cast<const uint2*>(b + min(2 * w, ad.rank - 4));
                            if (2 * w >= ad.rank) v = uint2{0u, 0u};
                            bw[k][w] = v.x;
                            bw[k][w + 1] = v.y;
                        }
                    }
                }
                floatx4 sum[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[k] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < 4 * RT; c += 2) {              // two chunks of 4 ranks
                    const uint4 v[3] = {h[3 * c / 2], h[3 * c / 2 + 1], h[3 * c / 2 + 2]};
                    const short4v part[6] = {four_bf16(v[0].x, v[0].y), four_bf16(v[0].z, v[0].w),
                                             four_bf16(v[1].x, v[1].y), four_bf16(v[1].z, v[1].w),
                                             four_bf16(v[2].x, v[2].y), four_bf16(v[2].z, v[2].w)};
#pragma unroll
                    for (int i = 0; i < 6; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            sum[k] = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(
                                part[i], four_bf16(bw[k][2 * (c + i / 3)], bw[k][2 * (c + i / 3) + 1]), sum[k], 0, 0, 0);
                }
                // a row takes its own adapter's, nothing of the other's NaN
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int k = 0; k < 4; ++k) low[k][r] = r >= row && r < end ? sum[k][r] : low[k][r];
            }
            if (end >= kRows) return;
            g = rows.then();
            row = end;
            end = kRows;
        }
    };
    auto phase_b = [&](int s, const float* zb) {
        const int64_t n0 = row_begin + int64_t(s) * kRows;
        const int rows = static_cast<int>(min(int64_t(kRows), row_end - n0));
        if constexpr (RT > 0) {
            // on top of the adapter's part, all rows of a gamma1 together: what
            // the other order holds at a time does not fit the registers
            floatx4 y[4];
            adapters(s, y);
#pragma unroll
            for (int k = 0; k < 4; ++k) k1r[k].hold();
#pragma unroll
            for (int g = 0; g < kC1; ++g)
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const floatx4 z = *reinterpret_cast<const floatx4*>(zb + r * kZRow + a1 * kZPitch + e10 + g * kD1);
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[k][r] = fmaf(k1r[k].at(g), z[k], y[k][r]);
                }
            // Every row is finished here: sunk into the tests below, as the compiler
            // would have them, the sums of rows 1 to 3 keep all that they need in
            // registers (rank 32: spilled, 64 us on 4099 rows for 38).
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int k = 0; k < 4; ++k) asm volatile("" : "+v"(y[k][r]));
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (r >= rows) break;
                const floatx4 out = {y[0][r], y[1][r], y[2][r], y[3][r]};
                float* yr = Y + (n0 + r) * args.n_out + yoff;
                if constexpr (kYVec) {
                    __builtin_nontemporal_store(out, reinterpret_cast<floatx4*>(yr));
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) __builtin_nontemporal_store(out[k], yr + k);
                }
            }
            return;
        }
#pragma unroll
        for (int r0 = 0; r0 < kRows; r0 += kRowsPerPass) {
            const int r = r0 + rsub;
            const float* zr = zb + r * kZRow + a1 * kZPitch + e10;
            floatx4 y = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int g = 0; g < kC1; ++g) {
                const floatx4 z = *reinterpret_cast<const floatx4*>(zr + g * kD1);
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = fmaf(k1r[k].at(g), z[k], y[k]);
            }
            if (r < rows) {
                float* yr = Y + (n0 + r) * args.n_out + yoff;
                if constexpr (kYVec) {
                    __builtin_nontemporal_store(y, reinterpret_cast<floatx4*>(yr));
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) __builtin_nontemporal_store(y[k], yr + k);
                }
            }
        }
    };
    pipeline(phase_b);
}

template <typename TX, typename TW, bool kYVec, int BT>
__global__ __launch_bounds__(kFusedThreads) void fused_pair_kernel(const TX* __restrict__ X,
                                                                   const TW* __restrict__ K0,
                                                                   const TW* __restrict__ K1,
                                                                   float* __restrict__ Y, FusedArgs args) {
    fused_pair<TX, TW, kYVec, BT, 0>(X, K0, K1, Y, args, PairAdapters{});
}

// LDS holds one workgroup a compute unit, three waves on a SIMD at most: registers
// for more waves would only hold back reads of Z (16384 rows of rank 16: 92 us with
// four in the compiler's mind, 78 with three).
template <bool kYVec, int RT>
__global__ __launch_bounds__(kFusedThreads)
    __attribute__((amdgpu_waves_per_eu(3, 3))) void fused_pair_adapters_kernel(const bf16_t* __restrict__ X,
                                                                               const bf16_t* __restrict__ K0,
                                                                               const bf16_t* __restrict__ K1,
                                                                               float* __restrict__ Y, FusedArgs args,
                                                                               PairAdapters ad) {
    fused_pair<bf16_t, bf16_t, kYVec, 32, RT>(X, K0, K1, Y, args, ad);
}

bool shape_ok(const Shape& s0, const Shape& s1) {
    return s0.a == 1 && s0.c == kC0 && s0.d == kD0 && s0.b % 8 == 0 && s1.a == s0.b && s1.b == kB1 &&
           s1.c == kC1 && s1.d == kD1;
}

template <typename TX, typename TW, int BT, int RT>
ks_status_t launch_tile(const Shape& s0, const Shape& s1, const void* W0, const void* W1, const void* X,
                        float* Y, int64_t batch, const PairAdapters& ad, hipStream_t stream, int num_cus) {
    FusedArgs args;
    args.b0 = s0.b;
    args.n_in = s0.n_in;
    args.n_mid = s0.n_out;
    args.n_out = s1.n_out;
    args.batch = batch;
    args.n_tiles = s0.b / BT;
    args.xshift = static_cast<int>((reinterpret_cast<uintptr_t>(X) & 15u) / sizeof(TX));
    // about one resident wave of workgroups (as many per compute unit as fit its 160 KB of LDS)
    const size_t lds = fused_lds_bytes(int(sizeof(TX)), BT, RT > 0);
    const int per_cu = std::max(1, std::min(4, int((160 * 1024) / lds)));
    const int64_t steps_total = (batch + kRows - 1) / kRows;
    const int64_t splits = std::max<int64_t>(1, int64_t(std::max(num_cus, 1)) * per_cu / args.n_tiles);
    const int64_t steps = std::max<int64_t>(1, (steps_total + splits - 1) / splits);
    args.rows_per_split = static_cast<int>(steps * kRows);
    const int64_t nsplit = (batch + args.rows_per_split - 1) / args.rows_per_split;
    const int64_t blocks = nsplit * args.n_tiles;
    if (blocks > 0x7fffffff) return KS_ERR_UNSUPPORTED;
    const bool y_vec = (reinterpret_cast<uintptr_t>(Y) & 15u) == 0;
    const dim3 grid(static_cast<unsigned>(blocks)), block(kFusedThreads);
    const TX* x = static_cast<const TX*>(X);
    const TW *w0 = static_cast<const TW*>(W0), *w1 = static_cast<const TW*>(W1);
    if constexpr (RT > 0) {
        return launch_kernel(y_vec ? fused_pair_adapters_kernel<true, RT> : fused_pair_adapters_kernel<false, RT>, grid,
                             block, lds, stream, x, w0, w1, Y, args, ad);
    } else {
        return launch_kernel(y_vec ? fused_pair_kernel<TX, TW, true, BT> : fused_pair_kernel<TX, TW, false, BT>, grid,
                             block, lds, stream, x, w0, w1, Y, args);
    }
}

// The widest tile that divides b0: 32 beta0 per workgroup on GPT-2-medium's
// b0 = 64 (fp32 64 vs 72 us, bf16 61 vs 68 us against 8 beta0 and four
// compute waves, measured A/B in one process).
template <typename TX, typename TW>
ks_status_t launch_typed(const Shape& s0, const Shape& s1, const void* W0, const void* W1, const void* X,
                         float* Y, int64_t batch, hipStream_t stream, int num_cus) {
    if (s0.b % 32 == 0) return launch_tile<TX, TW, 32, 0>(s0, s1, W0, W1, X, Y, batch, {}, stream, num_cus);
    if (s0.b % 16 == 0) return launch_tile<TX, TW, 16, 0>(s0, s1, W0, W1, X, Y, batch, {}, stream, num_cus);
    return launch_tile<TX, TW, 8, 0>(s0, s1, W0, W1, X, Y, batch, {}, stream, num_cus);
}

}  // namespace

bool fused_pair_supports(const Shape& s0, const Shape& s1, int xt, int wt0, int wt1) {
    if (wt0 != wt1) return false;
    if (!(xt == kF32 || xt == kBF16)) return false;
    if (!shape_ok(s0, s1)) return false;
    // the loader addresses a stage with 32-bit byte offsets
    return int64_t(kRows) * s0.n_in * elem_bytes(xt) < (int64_t(1) << 31);
}

ks_status_t launch_fused_pair(const Shape& s0, const Shape& s1, int xt, int wt0, int wt1, const void* W0,
                              const void* W1, const void* X, float* Y, int64_t batch, hipStream_t stream,
                              int num_cus) {
    if (!fused_pair_supports(s0, s1, xt, wt0, wt1)) return KS_ERR_UNSUPPORTED;
    // X and Y aligned to their element size (checked by the caller); rows
    // are whole 16-byte granules apart, so every row has X's misalignment
    if ((reinterpret_cast<uintptr_t>(X) % elem_bytes(xt)) != 0 || (reinterpret_cast<uintptr_t>(Y) & 3u) != 0 ||
        (s0.n_in * elem_bytes(xt)) % 16 != 0)
        return KS_ERR_UNSUPPORTED;
    if (xt == kF32 && wt0 == kF32) return launch_typed<float, float>(s0, s1, W0, W1, X, Y, batch, stream, num_cus);
    if (xt == kBF16 && wt0 == kBF16) return launch_typed<bf16_t, bf16_t>(s0, s1, W0, W1, X, Y, batch, stream, num_cus);
    if (xt == kF32 && wt0 == kBF16) return launch_typed<float, bf16_t>(s0, s1, W0, W1, X, Y, batch, stream, num_cus);
    return KS_ERR_UNSUPPORTED;
}

bool fused_pair_adds(const Shape& s0, const Shape& s1, int xt, int wt, const void* B, int rank) {
    return xt == kBF16 && wt == kBF16 && s0.b % 32 == 0 && fused_pair_supports(s0, s1, xt, wt, wt) &&
           rank <= kLowPartsRank && rank % 4 == 0 && reinterpret_cast<uintptr_t>(B) % 8 == 0;
}

ks_status_t launch_fused_pair_adapters(const Shape& s0, const Shape& s1, const void* W0, const void* W1,
                                       const void* X, float* Y, int64_t batch, const PairAdapters& ad,
                                       hipStream_t stream, int num_cus) {
    if (!fused_pair_adds(s0, s1, kBF16, kBF16, ad.B, ad.rank)) return KS_ERR_UNSUPPORTED;
    return ad.rank <= 16 ? launch_tile<bf16_t, bf16_t, 32, 1>(s0, s1, W0, W1, X, Y, batch, ad, stream, num_cus)
                         : launch_tile<bf16_t, bf16_t, 32, 2>(s0, s1, W0, W1, X, Y, batch, ad, stream, num_cus);
}

}  // namespace ks
