// ks_pair_grad.hip -- dX of a GPT-2-type pair of factors in one launch.
//
// The pair F0 = (1, b0, 16, 64), F1 = (b0, 8, 8, 8) (ks_fused.hip) has the gradient
//   dZ[alpha][gamma1][delta1] = sum_beta1  K1[alpha][delta1][beta1][gamma1] dY[alpha][beta1][delta1]
//   dX[gamma0][delta0]        = sum_beta0  K0[delta0][beta0][gamma0] dZ[beta0][delta0]
// with alpha = beta0 and delta0 = 8 gamma1 + delta1. As a chain of transposed
// factors it is two launches with dZ, as wide as dY, written and read between
// them (and W's blocks transposed first); here dZ stays on the chip and W is read
// as it lies: 28 us for 66 (and 9 for the transposes) at 4099 x 4096.
//
// Workgroup: whole rows, four at a time, eight waves, one workgroup a compute
// unit. All weights of the pair stay in its registers, two bf16 values a word (96
// words a thread at b0 = 64), loaded once through LDS. Two buffers of dZ take 133 of
// the 160 KB of LDS at b0 = 64 and would take 166 at 80: wider pairs run as a chain.
//  (A) on the 16-block 4x4x1 fp32 MFMA: lane 4 i + q supplies row q of block i's
//      left operand, column q of its right one, and receives column q of the
//      block's product, the rows in its four registers. Wave w takes alpha in
//      [8 w, 8 w + 8); block = (alpha, half of delta1), an instruction for each
//      delta1 of the half, beta1, and parity of gamma1 (column q: gamma1 = 2 q +
//      parity). dY comes from global memory as 16-byte runs of delta1, one stage
//      ahead. The products, four rows in a vector, go to LDS.
//  (B) on the VALU: a thread takes delta0 16 (w % 4) + lane / 4 and two gamma0, and
//      goes through all of beta0, four rows a read of dZ.
// One barrier a stage on alternate buffers of dZ: phase B of one wave runs beside
// phase A of the next stage in another. Bound by the stream of dY (phase B on the
// MFMA as well, the waves of a SIMD in opposite phases, or two stages of dY ahead:
// the same times): 16384 x 4096 85 us, 4.0 TB/s with the start, mostly weights,
// that takes 8 of them.

#include <algorithm>

#include "ks_device.h"
#include "ks_stream.h"
#include "ks_train.h"

namespace ks {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kC0 = 16, kD0 = 64;        // first factor
constexpr int kB1 = 8, kC1 = 8, kD1 = 8; // second factor
constexpr int kRows = 4;                 // rows a stage
constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kMaxB0 = 64;
constexpr int kK0Pad = 16, kK1Row = kB1 * kC1 * 2 + 16;   // bytes: LDS rows of a delta0's and of an (alpha, delta1)'s weights

constexpr int z_pitch(int b0) { return b0 + 1; }          // vectors of four rows: delta0 neighbours 4 banks apart
constexpr size_t z_bytes(int b0) { return size_t(kD0) * z_pitch(b0) * 16; }
constexpr size_t lds_bytes(int b0) {
    return std::max({2 * z_bytes(b0), size_t(kD0) * (b0 * kC0 * 2 + kK0Pad), size_t(b0) * kD1 * kK1Row});
}

// Packed words are widened where they are used: widened once, ahead of the loop
// over the stages, they would take twice the registers. The shift and the mask are
// new to the compiler in every stage.
struct Widen {
    uint32_t shift = 16, mask = 0xffff0000u;
    __device__ __forceinline__ Widen() { asm volatile("" : "+s"(shift), "+s"(mask)); }
    __device__ __forceinline__ float lo(uint32_t w) const { return __uint_as_float(w << shift); }
    __device__ __forceinline__ float hi(uint32_t w) const { return __uint_as_float(w & mask); }
};

template <int B0>
__global__ __launch_bounds__(kThreads) void pair_dx_kernel(const float* __restrict__ dY, const bf16_t* __restrict__ K0,
                                                           const bf16_t* __restrict__ K1, float* __restrict__ dX,
                                                           int64_t batch) {
    extern __shared__ __align__(16) unsigned char lds[];
    constexpr int64_t kOut = int64_t(B0) * kB1 * kD1, kIn = kC0 * kD0;
    constexpr int P = z_pitch(B0);
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int q = lane & 3, block = lane >> 2;
    // the workgroups take neighbouring rows at a time
    const int64_t row0 = int64_t(blockIdx.x) * kRows, step = int64_t(gridDim.x) * kRows;
    // phase A: this lane's alpha and first delta1
    const bool first = wave * 8 < B0;
    const int alpha = min(wave * 8 + (block >> 1), B0 - 1), d1 = (block & 1) * 4;
    // phase B: its delta0 and first gamma0
    const int d0 = 16 * (wave & 3) + block, g0 = 8 * (wave >> 2) + 2 * q;

    f32x4 y[kB1];
    auto fetch = [&](int64_t n0) {
        const float* at = dY + min(n0 + q, batch - 1) * kOut + alpha * (kB1 * kD1) + d1;
#pragma unroll
        for (int b = 0; b < kB1; ++b) y[b] = *reinterpret_cast<const f32x4*>(at + b * kD1);
    };
    if (first) fetch(row0);

    // weights: through LDS, where rows are padded, into registers
    uint32_t k0[B0], k1[4][kB1];
    {
        constexpr int kRow = B0 * kC0 * 2 / 16;               // 16-byte vectors of a delta0
        constexpr int kVec = kB1 * kC1 * 2 / 16;              // of an (alpha, delta1)
        constexpr int N0 = kD0 * kRow / kThreads, N1 = B0 * kD1 * kVec / kThreads;
        static_assert(kD0 * kRow % kThreads == 0 && B0 * kD1 * kVec % kThreads == 0, "whole vectors a thread");
        u32x4 v0[N0], v1[N1];                                 // all on their way at once
#pragma unroll
        for (int i = 0; i < N0; ++i) v0[i] = reinterpret_cast<const u32x4*>(K0)[i * kThreads + t];
#pragma unroll
        for (int i = 0; i < N1; ++i) v1[i] = reinterpret_cast<const u32x4*>(K1)[i * kThreads + t];
#pragma unroll
        for (int i = 0; i < N0; ++i) {
            const int v = i * kThreads + t;
            *reinterpret_cast<u32x4*>(lds + v / kRow * (kRow * 16 + kK0Pad) + v % kRow * 16) = v0[i];
        }
        lds_barrier();
#pragma unroll
        for (int b = 0; b < B0; ++b)
            k0[b] = *reinterpret_cast<const uint32_t*>(lds + d0 * (kRow * 16 + kK0Pad) + (b * kC0 + g0) * 2);
        lds_barrier();
#pragma unroll
        for (int i = 0; i < N1; ++i) {
            const int v = i * kThreads + t;
            *reinterpret_cast<u32x4*>(lds + v / kVec * kK1Row + v % kVec * 16) = v1[i];
        }
        lds_barrier();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int b = 0; b < kB1; ++b)
                k1[j][b] = *reinterpret_cast<const uint32_t*>(lds + (alpha * kD1 + d1 + j) * kK1Row + (b * kC1 + 2 * q) * 2);
        lds_barrier();
    }

    int s = 0;
    for (int64_t n0 = row0; n0 < batch; n0 += step, ++s) {
        f32x4* const z = reinterpret_cast<f32x4*>(lds + (s & 1) * z_bytes(B0));    // [delta0][beta0], four rows
        const Widen widen;
        if (first) {
            f32x4 even[4], odd[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) even[j] = odd[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int b = 0; b < kB1; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    even[j] = __builtin_amdgcn_mfma_f32_4x4x1f32(y[b][j], widen.lo(k1[j][b]), even[j], 0, 0, 0);
                    odd[j] = __builtin_amdgcn_mfma_f32_4x4x1f32(y[b][j], widen.hi(k1[j][b]), odd[j], 0, 0, 0);
                }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = (2 * q * kD1 + d1 + j) * P + alpha;
                z[at] = even[j];
                z[at + kD1 * P] = odd[j];
            }
            if (n0 + step < batch) fetch(n0 + step);
        }
        lds_barrier();
        f32x4 acc0 = {0.0f, 0.0f, 0.0f, 0.0f}, acc1 = acc0;   // four rows of gamma0 and the next
        const f32x4* const zb = z + d0 * P;
        // a run's reads of dZ are on their way during the one before
        constexpr int kRun = 4;
        f32x4 x[2][kRun];
#pragma unroll
        for (int b = 0; b < kRun; ++b) x[0][b] = zb[b];
#pragma unroll
        for (int b0 = 0; b0 < B0; b0 += kRun) {
            const int half = b0 / kRun & 1;
            if (b0 + kRun < B0) {
#pragma unroll
                for (int b = 0; b < kRun; ++b) x[half ^ 1][b] = zb[b0 + kRun + b];
            }
#pragma unroll
            for (int b = 0; b < kRun; ++b) {
                const float lo = widen.lo(k0[b0 + b]), hi = widen.hi(k0[b0 + b]);
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    acc0[r] = fmaf(x[half][b][r], lo, acc0[r]);
                    acc1[r] = fmaf(x[half][b][r], hi, acc1[r]);
                }
            }
        }
        // every row here: sunk into the tests below, the sums of rows 1 to 3 would
        // keep all of dZ and the weights waiting
#pragma unroll
        for (int r = 0; r < kRows; ++r) asm volatile("" : "+v"(acc0[r]), "+v"(acc1[r]));
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (n0 + r >= batch) break;
            float* out = dX + (n0 + r) * kIn + g0 * kD0 + d0;
            out[0] = acc0[r];
            out[kD0] = acc1[r];
        }
    }
}

}  // namespace

bool pair_dx_supports(const Shape& s0, const Shape& s1, int wt, const void* W0, const void* W1, const float* dY) {
    return wt == kBF16 && s0.a == 1 && s0.c == kC0 && s0.d == kD0 && s1.a == s0.b && s1.b == kB1 && s1.c == kC1 &&
           s1.d == kD1 && s0.b % 16 == 0 && s0.b <= kMaxB0 && reinterpret_cast<uintptr_t>(W0) % 16 == 0 &&
           reinterpret_cast<uintptr_t>(W1) % 16 == 0 && reinterpret_cast<uintptr_t>(dY) % 16 == 0;
}

ks_status_t launch_pair_dx(const Shape& s0, const void* W0, const void* W1, const float* dY, float* dX, int64_t batch,
                           hipStream_t stream, int num_cus) {
    const int64_t stages = (batch + kRows - 1) / kRows;
    void (*kernel)(const float*, const bf16_t*, const bf16_t*, float*, int64_t) =
        s0.b == 16 ? pair_dx_kernel<16> : s0.b == 32 ? pair_dx_kernel<32> : s0.b == 48 ? pair_dx_kernel<48> : pair_dx_kernel<64>;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(std::min<int64_t>(stages, std::max(num_cus, 1)))),
                         dim3(kThreads), lds_bytes(s0.b), stream, dY, static_cast<const bf16_t*>(W0),
                         static_cast<const bf16_t*>(W1), dX, batch);
}

}  // namespace ks
