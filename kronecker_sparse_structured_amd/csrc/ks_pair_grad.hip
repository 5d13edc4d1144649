// ks_pair_grad.hip -- dX of a GPT-2-type pair of factors in one launch.
//
// The pair F0 = (1, b0, 16, 64), F1 = (b0, 8, 8, 8) (ks_fused.hip) has the gradient
//   dZ[alpha][gamma1][delta1] = sum_beta1  K1[alpha][delta1][beta1][gamma1] dY[alpha][beta1][delta1]
//   dX[gamma0][delta0]        = sum_beta0  K0[delta0][beta0][gamma0] dZ[beta0][delta0]
// with alpha = beta0 and delta0 = 8 gamma1 + delta1. As a chain of transposed
// factors it is two launches with dZ, as wide as dY, written and read between
// them (and W's blocks transposed first); here dZ stays on the chip and W is read
// as it lies: 4099 x 4096 @@US@@.
//
// Workgroup: whole rows, four at a time, eight waves, one workgroup a compute
// unit. All weights of the pair stay in its registers, two bf16 values a word (96
// words a thread at b0 = 64), loaded once through LDS. Both phases run on the
// 16-block 4x4x1 fp32 MFMA: lane 4 i + q supplies row q of block i's left operand,
// column q of its right one, and receives column q of the block's product, the
// rows in its four registers.
//  (A) wave w takes alpha in [8 w, 8 w + 8); block = (alpha, half of delta1), an
//      instruction for each delta1 of the half, beta1, and parity of gamma1 (column
//      q: gamma1 = 2 q + parity). dY comes from global memory as 16-byte runs of
//      delta1, one stage ahead. The products, four rows in a vector, go to LDS.
//  (B) wave w takes delta0 in [16 (w % 4), + 16), a block each, and gamma0 in
//      [8 (w / 4), + 8), two a column, and goes through all of beta0.
// One barrier a stage on alternate buffers of dZ: phase B of one wave runs beside
// phase A of the next stage in another.

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

template <int B0>
__global__ __launch_bounds__(kThreads) void pair_dx_kernel(const float* __restrict__ dY, const bf16_t* __restrict__ K0,
                                                           const bf16_t* __restrict__ K1, float* __restrict__ dX,
                                                           int64_t batch, int rows_per_group) {
    extern __shared__ __align__(16) unsigned char lds[];
    constexpr int64_t kOut = int64_t(B0) * kB1 * kD1, kIn = kC0 * kD0;
    constexpr int P = z_pitch(B0);
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int q = lane & 3, block = lane >> 2;
    const int64_t row0 = int64_t(blockIdx.x) * rows_per_group;
    const int64_t row1 = min(batch, row0 + rows_per_group);
    // phase A: this lane's alpha and first delta1
    const bool first = wave * 8 < B0;
    const int alpha = min(wave * 8 + (block >> 1), B0 - 1), d1 = (block & 1) * 4;
    // phase B: its delta0 and first gamma0
    const int d0 = 16 * (wave & 3) + block, g0 = 8 * (wave >> 2) + 2 * q;

    f32x4 y[kB1];
    auto fetch = [&](int64_t n0) {
        const float* at = dY + min(n0 + q, row1 - 1) * kOut + alpha * (kB1 * kD1) + d1;
#pragma unroll
        for (int b = 0; b < kB1; ++b) y[b] = *reinterpret_cast<const f32x4*>(at + b * kD1);
    };
    if (first) fetch(row0);

    // weights: through LDS, where rows are padded, into registers
    uint32_t k0[B0], k1[4][kB1];
    {
        constexpr int kRow = B0 * kC0 * 2 / 16;               // 16-byte vectors of a delta0
        for (int v = t; v < kD0 * kRow; v += kThreads)
            *reinterpret_cast<u32x4*>(lds + v / kRow * (kRow * 16 + kK0Pad) + v % kRow * 16) =
                reinterpret_cast<const u32x4*>(K0)[v];
        __syncthreads();
#pragma unroll
        for (int b = 0; b < B0; ++b)
            k0[b] = *reinterpret_cast<const uint32_t*>(lds + d0 * (kRow * 16 + kK0Pad) + (b * kC0 + g0) * 2);
        __syncthreads();
        constexpr int kVec = kB1 * kC1 * 2 / 16;              // of an (alpha, delta1)
        for (int v = t; v < B0 * kD1 * kVec; v += kThreads)
            *reinterpret_cast<u32x4*>(lds + v / kVec * kK1Row + v % kVec * 16) = reinterpret_cast<const u32x4*>(K1)[v];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int b = 0; b < kB1; ++b)
                k1[j][b] = *reinterpret_cast<const uint32_t*>(lds + (alpha * kD1 + d1 + j) * kK1Row + (b * kC1 + 2 * q) * 2);
        __syncthreads();
    }

    int s = 0;
    for (int64_t n0 = row0; n0 < row1; n0 += kRows, ++s) {
        f32x4* const z = reinterpret_cast<f32x4*>(lds + (s & 1) * z_bytes(B0));    // [delta0][beta0], four rows
        if (first) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f32x4 even = {0.0f, 0.0f, 0.0f, 0.0f}, odd = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int b = 0; b < kB1; ++b) {
                    // widened where they are used, not ahead of the loop
                    asm volatile("" : "+v"(k1[j][b]));
                    even = __builtin_amdgcn_mfma_f32_4x4x1f32(y[b][j], bf16_lo(k1[j][b]), even, 0, 0, 0);
                    odd = __builtin_amdgcn_mfma_f32_4x4x1f32(y[b][j], bf16_hi(k1[j][b]), odd, 0, 0, 0);
                }
                const int at = (2 * q * kD1 + d1 + j) * P + alpha;
                z[at] = even;
                z[at + kD1 * P] = odd;
            }
            if (n0 + kRows < row1) fetch(n0 + kRows);
        }
        lds_barrier();
        f32x4 acc[4];                                         // gamma0 parity, beta0 parity
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const float* const zq = reinterpret_cast<const float*>(z + d0 * P) + q;
#pragma unroll
        for (int b = 0; b < B0; ++b) {
            asm volatile("" : "+v"(k0[b]));
            const float x = zq[4 * b];
            acc[b & 1] = __builtin_amdgcn_mfma_f32_4x4x1f32(x, bf16_lo(k0[b]), acc[b & 1], 0, 0, 0);
            acc[2 + (b & 1)] = __builtin_amdgcn_mfma_f32_4x4x1f32(x, bf16_hi(k0[b]), acc[2 + (b & 1)], 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (n0 + r >= row1) break;
            float* out = dX + (n0 + r) * kIn + g0 * kD0 + d0;
            out[0] = acc[0][r] + acc[1][r];
            out[kD0] = acc[2][r] + acc[3][r];
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
    const int64_t stages = (batch + kRows - 1) / kRows, cus = std::max(num_cus, 1);
    const int64_t rows = (stages + cus - 1) / cus * kRows;
    if (rows > 0x7fffffff) return KS_ERR_UNSUPPORTED;
    void (*kernel)(const float*, const bf16_t*, const bf16_t*, float*, int64_t, int) =
        s0.b == 16 ? pair_dx_kernel<16> : s0.b == 32 ? pair_dx_kernel<32> : s0.b == 48 ? pair_dx_kernel<48> : pair_dx_kernel<64>;
    return launch_kernel(kernel, dim3(static_cast<unsigned>((batch + rows - 1) / rows)), dim3(kThreads), lds_bytes(s0.b),
                         stream, dY, static_cast<const bf16_t*>(W0), static_cast<const bf16_t*>(W1), dX, batch,
                         static_cast<int>(rows));
}

}  // namespace ks
