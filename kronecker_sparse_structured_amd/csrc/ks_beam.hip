// ks_beam.hip -- beam search: the best continuations of each request's beams,
// and their states.
//
//   score(w, v) = scores[w] + x[w][v] - log sum_u exp x[w][u]
//
// The logits are read once, by as many waves as there are slices of kSlice
// values: one row or a few have to fill the card as well as hundreds. A wave
// holds its slice in registers, forms its maximum and its sum of exponentials,
// and finds its best `keep` values (keep = min(out_beams, vocab)) without a
// barrier:
//   1. the keep-th largest of the 64 lanes' own maxima is a bound: at least keep
//      values of the slice reach it, and only keep lanes hold any,
//   2. the values that reach it go to a list in LDS (at most keep times what a
//      lane holds; keep or a few more of random values),
//   3. each of them counts how many of the list are before it: its place.
// Values are compared as 64-bit keys, their order's 32 bits and then the lower
// token, so that no two are equal and every choice is the same each time.
//
// Then one workgroup a request joins the slices of each beam (its lists in the
// same way, its sums in double) and picks from the beams' lists, which are
// sorted, the best head out_beams times.

#include <algorithm>

#include "ks_logit.h"
#include "ks_stack.h"

namespace ks {
namespace {

constexpr int kMaxBeams = KS_BEAM_MAX;
constexpr int kHold = 4;                 // 16-byte vectors a lane holds of a slice
constexpr int kSliceBytes = 64 * 16 * kHold;
constexpr int kSelectWaves = 4;          // a workgroup of the first launch
constexpr int kJoinWaves = 8;            // of the second, at most
constexpr int kJoinHold = 8;             // keys a lane holds there

// The order of fp32 values as unsigned numbers; -0 is 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// 0 is below every value's key.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t token) {
    return static_cast<uint64_t>(ordered(x)) << 32 | (0xffffffffu - token);
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t x, int d) {
    const uint32_t lo = __shfl_xor(static_cast<uint32_t>(x), d, 64), hi = __shfl_xor(static_cast<uint32_t>(x >> 32), d, 64);
    return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t y = shfl_xor64(x, d);
        x = y > x ? y : x;
    }
    return x;
}

// The keep-th largest of the lanes' keys (0 if fewer lanes have one).
__device__ __forceinline__ uint64_t bound_of(uint64_t mine, int keep) {
    uint64_t top = 0;
    for (int k = 0; k < keep; ++k) {
        top = wave_max64(mine);
        if (mine == top) mine = 0;
    }
    return top;
}

// What the wave's lanes wrote to LDS is there for all of them.
__device__ __forceinline__ void wave_lds_fence() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Sorts the best of list[0 .. n) to out[0 .. keep), the rest of which become 0.
// Of one wave; n is at least the number of keys that are looked for.
__device__ __forceinline__ void sort_best(const uint64_t* list, int n, int keep, uint64_t* out) {
    const int lane = threadIdx.x % 64;
    for (int i = lane; i < keep; i += 64)
        if (i >= n) out[i] = 0;
    for (int i = lane; i < n; i += 64) {
        const uint64_t mine = list[i];
        int place = 0;
        for (int j = 0; j < n; ++j) place += list[j] > mine;
        if (place < keep) out[place] = mine;
    }
}

// What the first launch leaves of a slice: {maximum, sum of exp(x - maximum)},
// and its best keys.
struct Slices {
    float2* stats;       // rows x slices
    uint64_t* keys;      // rows x slices x keep
    int slices, keep;
};

template <typename T>
__global__ __launch_bounds__(kSelectWaves * 64) void beam_slices_kernel(const ks_beams_t x, Slices s, int64_t unit0) {
    constexpr int E = kVec<T>, kHeld = E * kHold, kSlice = 64 * kHeld;
    extern __shared__ uint64_t lists[];                    // kSelectWaves x keep x kHeld
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int64_t unit = unit0 + static_cast<int64_t>(blockIdx.x) * kSelectWaves + wave;
    const int64_t row = unit / s.slices;
    if (row >= x.requests * x.beams) return;
    if (x.done && x.done[row]) return;
    const uint32_t slice = static_cast<uint32_t>(unit - row * s.slices);
    const int64_t r = row / x.beams;
    const T* data = static_cast<const T*>(x.data) + r * x.request_stride + (row - r * x.beams) * x.beam_stride;
    const uint32_t first = slice * kSlice, V = static_cast<uint32_t>(x.vocab);   // below 2^31 + kSlice
    float v[kHold][E];
    const bool wide = reinterpret_cast<uintptr_t>(data) % 16 == 0;
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
        const uint32_t at = first + (u * 64 + lane) * E;
        if (wide && at + E <= V) {
            widen<T>(*reinterpret_cast<const u32x4*>(data + at), v[u]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) v[u][i] = at + i < V ? to_f32(data[at + i]) : -INFINITY;
        }
    }
    float top = kLowest;
    uint64_t best = 0;
#pragma unroll
    for (int u = 0; u < kHold; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const uint32_t at = first + (u * 64 + lane) * E + i;
            top = fmaxf(top, v[u][i]);
            const uint64_t k = key_of(v[u][i], at);
            if (at < V && k > best) best = k;
        }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < kHold; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) sum += exp_of(v[u][i] - top);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    if (lane == 0) s.stats[unit] = make_float2(top, sum);
    const uint64_t bound = bound_of(best, s.keep);
    uint64_t* list = lists + static_cast<size_t>(wave) * s.keep * kHeld;
    int n = 0;
#pragma unroll
    for (int u = 0; u < kHold; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const uint32_t at = first + (u * 64 + lane) * E + i;
            const uint64_t k = key_of(v[u][i], at);
            const bool in = at < V && k >= bound;
            const uint64_t mask = __ballot(in);
            if (in) list[n + __popcll(mask & ((1ull << lane) - 1))] = k;
            n += __popcll(mask);
        }
    wave_lds_fence();
    sort_best(list, n, s.keep, s.keys + unit * s.keep);
}

// x is better than y: a higher rank, or an equal one earlier.
__device__ __forceinline__ bool better(double x, int at, double y, int other) {
    return x > y || (x == y && at < other);
}

// The best candidates of one request.
__global__ __launch_bounds__(kJoinWaves * 64) void beam_join_kernel(const ks_beams_t x, Slices s, BeamOut out,
                                                                    int64_t request0) {
    extern __shared__ uint64_t lds[];
    const int waves = blockDim.x / 64, wave = threadIdx.x / 64, lane = threadIdx.x % 64, W = x.beams, keep = s.keep;
    uint64_t* best = lds;                                             // W x keep
    uint64_t* list = best + W * keep + wave * keep * kJoinHold;
    __shared__ double base[kMaxBeams], divisor[kMaxBeams];            // score = base + x, rank = score / divisor
    __shared__ int length[kMaxBeams];
    const int64_t request = request0 + blockIdx.x;
    for (int w = wave; w < W; w += waves) {
        const int64_t row = request * W + w;
        const double score = x.scores[row];
        const bool done = x.done && x.done[row];
        const int len = x.lengths ? x.lengths[row] + (done ? 0 : 1) : 0;
        double shift = 0.0;
        bool live = score - score == 0.0;                             // finite
        if (!done) {
            const float2* st = s.stats + row * s.slices;
            double top = kLowest, sum = 0.0;
            for (int i = lane; i < s.slices; i += 64) top = fmax(top, static_cast<double>(st[i].x));
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) top = fmax(top, __shfl_xor(top, d, 64));
            for (int i = lane; i < s.slices; i += 64)
                sum += static_cast<double>(st[i].y) * exp(static_cast<double>(st[i].x) - top);
            sum = wave_sum(sum);
            shift = -top - log(sum);
            live = live && sum > 0.0 && sum - sum == 0.0;
            // the slices' keys, as many at a time as the list has room for beside
            // the best of those before
            const uint64_t* keys = s.keys + row * s.slices * keep;
            const int n = s.slices * keep;
            uint64_t mine[kJoinHold];
            for (int first = 0; first < n; first += 64 * (kJoinHold - 1)) {
                uint64_t high = mine[0] = first > 0 && lane < keep ? best[w * keep + lane] : 0;
#pragma unroll
                for (int u = 1; u < kJoinHold; ++u) {
                    const int i = first + (u - 1) * 64 + lane;
                    mine[u] = i < n ? keys[i] : 0;
                    high = mine[u] > high ? mine[u] : high;
                }
                const uint64_t bound = bound_of(high, keep);
                int count = 0;
#pragma unroll
                for (int u = 0; u < kJoinHold; ++u) {
                    const bool in = mine[u] != 0 && mine[u] >= bound;
                    const uint64_t mask = __ballot(in);
                    if (in) list[count + __popcll(mask & ((1ull << lane) - 1))] = mine[u];
                    count += __popcll(mask);
                }
                wave_lds_fence();
                sort_best(list, count, keep, best + w * keep);
                wave_lds_fence();
            }
        } else {
            for (int i = lane; i < keep; i += 64)
                best[w * keep + i] = i == 0 ? key_of(0.0f, static_cast<uint32_t>(x.eos)) : 0;
        }
        if (lane == 0) {
            base[w] = live ? score + shift : -INFINITY;
            length[w] = len;
            divisor[w] = x.length_penalty == 0.0 ? 1.0 : pow(static_cast<double>(max(len, 1)), x.length_penalty);
        }
    }
    __syncthreads();
    if (wave != 0) return;
    // lane w goes down beam w's list
    int next = 0, token = 0;
    double score = -INFINITY, rank = -INFINITY;
    auto take = [&]() {
        score = rank = -INFINITY;
        if (lane >= W || next >= keep) return;
        const uint64_t k = best[lane * keep + next];
        ++next;
        if (k == 0 || !(base[lane] > -INFINITY)) return;
        token = static_cast<int>(0xffffffffu - static_cast<uint32_t>(k));
        score = base[lane] + static_cast<double>(value_of(static_cast<uint32_t>(k >> 32)));
        rank = score > -INFINITY ? score / divisor[lane] : score;
    };
    take();
    const int64_t to = request * out.beams;
    for (int j = 0; j < out.beams; ++j) {
        double high = rank;
        int at = lane < W ? lane : 64;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double other = __shfl_xor(high, d, 64);
            const int from = __shfl_xor(at, d, 64);
            if (better(other, from, high, at)) {
                high = other;
                at = from;
            }
        }
        if (!(high > -INFINITY)) {                                    // none is left
            if (lane == 0) {
                out.scores[to + j] = -INFINITY;
                out.tokens[to + j] = x.eos >= 0 ? x.eos : 0;
                out.parents[to + j] = 0;
                if (out.done) out.done[to + j] = 1;
                if (out.lengths) out.lengths[to + j] = 0;
            }
            continue;
        }
        if (lane == at) {
            out.scores[to + j] = static_cast<float>(score);
            out.tokens[to + j] = token;
            out.parents[to + j] = lane;
            if (out.done) out.done[to + j] = token == x.eos;
            if (out.lengths) out.lengths[to + j] = length[lane];
            take();
        }
    }
}

// ---------------------------------------------------------------- states

constexpr int kStates = 60;              // a launch: their table is a kernel argument
constexpr int kPiece = 16;               // accesses of a wave
struct StateEntry {
    const char* src;
    char* dst;
    int64_t row_bytes;
    int64_t first;                       // first wave of this state
    int64_t pieces;                      // waves a row
    int64_t size;                        // bytes of an access: 16, 4 or 1
};
struct StateTable {
    StateEntry e[kStates];
    int32_t count;
};

// A wave copies one piece of one row.
template <typename V>
__device__ __forceinline__ void copy_piece(const StateEntry& e, int64_t row, int64_t from, int64_t piece, bool valid) {
    const int lane = threadIdx.x % 64;
    const int64_t n = e.row_bytes / static_cast<int64_t>(sizeof(V));
    V* dst = reinterpret_cast<V*>(e.dst + row * e.row_bytes);
    const V* src = reinterpret_cast<const V*>(e.src + (valid ? from : 0) * e.row_bytes);
    for (int k = 0; k < kPiece; ++k) {
        const int64_t i = (piece * kPiece + k) * 64 + lane;
        if (i < n) dst[i] = valid ? src[i] : V{};
    }
}

__global__ __launch_bounds__(256) void beam_reorder_kernel(const StateTable t, const int32_t* parents, int beams,
                                                           int out_beams, int64_t wave0, int64_t waves) {
    const int64_t unit = wave0 + static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 64;
    if (unit >= waves) return;
    int k = 0;
    for (int i = 1; i < t.count; ++i)
        if (t.e[i].first <= unit) k = i;
    const StateEntry& e = t.e[k];
    const int64_t at = unit - e.first, row = at / e.pieces, piece = at - row * e.pieces, request = row / out_beams;
    const int parent = parents[row];
    const bool valid = parent >= 0 && parent < beams;
    const int64_t from = request * beams + parent;
    if (e.size == 16) copy_piece<u32x4>(e, row, from, piece, valid);
    else if (e.size == 4) copy_piece<uint32_t>(e, row, from, piece, valid);
    else copy_piece<uint8_t>(e, row, from, piece, valid);
}

int slice_count(const ks_beams_t& x) {
    const int64_t slice = kSliceBytes / (x.elem == KS_ELEM_BF16 ? 2 : 4);
    return static_cast<int>((x.vocab + slice - 1) / slice);
}

Slices slices_of(const ks_beams_t& x, int out_beams, void* ws) {
    Slices s;
    s.slices = slice_count(x);
    s.keep = static_cast<int>(std::min<int64_t>(out_beams, x.vocab));
    const int64_t units = x.requests * x.beams * s.slices;
    s.keys = static_cast<uint64_t*>(ws);
    s.stats = reinterpret_cast<float2*>(s.keys + units * s.keep);
    return s;
}

}  // namespace

size_t beam_workspace(const ks_beams_t& x, int out_beams) {
    const Slices s = slices_of(x, out_beams, nullptr);
    return static_cast<size_t>(x.requests * x.beams * s.slices) * (static_cast<size_t>(s.keep) * 8 + 8);
}

ks_status_t launch_beam_select(const ks_beams_t& x, const BeamOut& out, void* ws, hipStream_t stream) {
    const Slices s = slices_of(x, out.beams, ws);
    const int64_t units = x.requests * x.beams * s.slices;
    const bool bf16 = x.elem == KS_ELEM_BF16;
    const size_t lds = static_cast<size_t>(kSelectWaves) * s.keep * kHold * (bf16 ? 8 : 4) * 8;
    const int64_t groups = (units + kSelectWaves - 1) / kSelectWaves;
    for (int64_t g = 0; g < groups; g += kMaxGrid) {
        const ks_status_t st = launch_kernel(bf16 ? beam_slices_kernel<bf16_t> : beam_slices_kernel<float>,
                                             dim3(static_cast<unsigned>(std::min(kMaxGrid, groups - g))),
                                             dim3(kSelectWaves * 64), lds, stream, x, s, g * kSelectWaves);
        if (st != KS_OK) return st;
    }
    const int waves = std::min(kJoinWaves, x.beams);
    const size_t join = static_cast<size_t>(x.beams * s.keep + waves * s.keep * kJoinHold) * 8;
    for (int64_t r = 0; r < x.requests; r += kMaxGrid) {
        const ks_status_t st = launch_kernel(beam_join_kernel,
                                             dim3(static_cast<unsigned>(std::min(kMaxGrid, x.requests - r))),
                                             dim3(waves * 64), join, stream, x, s, out, r);
        if (st != KS_OK) return st;
    }
    return KS_OK;
}

ks_status_t launch_beam_reorder(const ks_state_t* states, int n, const int32_t* parents, int64_t requests, int beams,
                                int out_beams, hipStream_t stream) {
    for (int i = 0; i < n;) {
        StateTable t;
        t.count = 0;
        int64_t waves = 0;
        for (; i < n && t.count < kStates; ++i) {
            if (states[i].row_bytes == 0) continue;
            StateEntry& e = t.e[t.count++];
            e.src = static_cast<const char*>(states[i].src);
            e.dst = static_cast<char*>(states[i].dst);
            e.row_bytes = states[i].row_bytes;
            const uint64_t bits = reinterpret_cast<uintptr_t>(e.src) | reinterpret_cast<uintptr_t>(e.dst) |
                                  static_cast<uint64_t>(e.row_bytes);
            e.size = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
            e.pieces = (e.row_bytes / e.size + 64 * kPiece - 1) / (64 * kPiece);
            e.first = waves;
            waves += requests * out_beams * e.pieces;
        }
        if (waves == 0) continue;
        const int64_t groups = (waves + 3) / 4;
        for (int64_t g = 0; g < groups; g += kMaxGrid) {
            const ks_status_t st = launch_kernel(beam_reorder_kernel, dim3(static_cast<unsigned>(std::min(kMaxGrid, groups - g))),
                                                 dim3(256), 0, stream, t, parents, beams, out_beams, g * 4, waves);
            if (st != KS_OK) return st;
        }
    }
    return KS_OK;
}

}  // namespace ks
