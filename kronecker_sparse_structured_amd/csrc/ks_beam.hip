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
//      values of the slice reach it,
//   2. those that do go to a list in LDS: keep or a few more of random values. Only
//      keep lanes have any, so the list has room for all, unless lanes' maxima are
//      (nearly) equal: then the bound is taken again over values with their
//      tokens, of which no two are,
//   3. each of them counts how many of the list are before it: its place.
// Values are ordered as 64-bit keys, their order's 32 bits and then the lower
// token, so that no two are equal and every choice is the same each time.
//
// Then one workgroup a request joins the slices of each beam (its lists in the
// same way, its sums in double), ranks every beam's list and picks from the lists,
// which are sorted, the best head out_beams times.
//
// What bounds it: many rows the arithmetic of the first launch beside its reads
// (32 x 16 beams of 32000 in fp32, 66 MB, 15 us, and 64 x 4 of 50257 in bf16, 26 MB,
// 10 us: 4.4 and 2.6 TB/s), few rows the two launches' latency, 6 us each. The second
// launch is a chain of dependent steps, 6 to 7 us for 4 beams and 11 for 16.

#include <algorithm>

#include "ks_logit.h"
#include "ks_stack.h"

namespace ks {
namespace {

constexpr int kMaxBeams = KS_BEAM_MAX;
constexpr int kHeld = 32;                // values a lane holds of a slice
constexpr int kSlice = 64 * kHeld;
constexpr int kSelectWaves = 4;          // a workgroup of the first launch
constexpr int kJoinWaves = 16;           // of the second, at most
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

__device__ __forceinline__ bool finite(float x) { return x - x == 0.0f; }

// The wave's largest x, in every lane: exchanges within 16 lanes, then lane 15 of a
// row of 16 to the next row, lane 31 to the upper half.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t max_with(uint32_t x) {
    return max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, ROWS, 0xf, false)));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = max_with<0xb1, 0xf>(x);
    x = max_with<0x4e, 0xf>(x);
    x = max_with<0x141, 0xf>(x);
    x = max_with<0x140, 0xf>(x);
    x = max_with<0x142, 0xa>(x);
    x = max_with<0x143, 0xc>(x);
    return __builtin_amdgcn_readlane(x, 63);
}

// The upper BITS bits of the keep-th largest of the lanes' x, the others 0: bit by
// bit, by how many lanes reach it (keep rounds of a maximum instead: 32 x 16 beams
// of 32000 in 26 us for 22).
template <int BITS, typename K>
__device__ __forceinline__ K bound_of(K x, int keep) {
    constexpr int kAll = 8 * sizeof(K);
    K t = 0;
#pragma unroll
    for (int b = kAll - 1; b >= kAll - BITS; --b) {
        const K higher = t | K(1) << b;
        if (__popcll(__ballot(x >= higher)) >= keep) t = higher;
    }
    return t;
}

// Appends the lanes' keys that are `in` to a list of n with room for `most`; n
// counts those without room too.
__device__ __forceinline__ void append(uint64_t* list, int& n, int most, bool in, uint64_t key) {
    const uint64_t mask = __ballot(in);
    if (mask == 0) return;
    const int at = n + __popcll(mask & ((1ull << (threadIdx.x % 64)) - 1));
    if (in && at < most) list[at] = key;
    n += __popcll(mask);
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
#pragma unroll 8
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
    constexpr int E = kVec<T>, kHold = kHeld / E;
    extern __shared__ uint64_t lists[];                    // kSelectWaves x keep x kHeld
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int64_t unit = unit0 + static_cast<int64_t>(blockIdx.x) * kSelectWaves + wave;
    const int64_t row = unit / s.slices;
    if (row >= x.requests * x.beams) return;
    if (!finite(x.scores[row]) || (x.done && x.done[row])) return;       // no candidates of its logits
    const uint32_t slice = static_cast<uint32_t>(unit - row * s.slices);
    const int64_t r = row / x.beams;
    const T* data = static_cast<const T*>(x.data) + r * x.request_stride + (row - r * x.beams) * x.beam_stride;
    const uint32_t first = slice * kSlice, V = static_cast<uint32_t>(x.vocab);   // below 2^31 + kSlice
    // 16-byte accesses that may start at any element: rows of an odd vocabulary do
    typedef typename Access<T, 4>::vec access;
    float v[kHold][E];
    if (first + kSlice <= V) {
        u32x4 w[kHold];
#pragma unroll
        for (int u = 0; u < kHold; ++u) w[u] = *reinterpret_cast<const access*>(data + first + (u * 64 + lane) * E);
#pragma unroll
        for (int u = 0; u < kHold; ++u) widen<T>(w[u], v[u]);
    } else {
#pragma unroll
        for (int u = 0; u < kHold; ++u) {
            const uint32_t at = first + (u * 64 + lane) * E;
            if (at + E <= V) {
                widen<T>(*reinterpret_cast<const access*>(data + at), v[u]);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) v[u][i] = at + i < V ? to_f32(data[at + i]) : -INFINITY;
            }
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kHold; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) top = fmaxf(top, v[u][i]);
    const uint32_t mine = ordered(top);
    top = fmaxf(value_of(wave_max(mine)), kLowest);
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) part += exp_of(v[u][i] - top);
        sum += part;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    if (lane == 0) s.stats[unit] = make_float2(top, sum);
    // 16 bits of the bound will do: a few more values reach it
    const float bound = value_of(max(bound_of<16>(mine, s.keep), ordered(-INFINITY)));
    const int most = s.keep * kHeld;
    uint64_t* list = lists + static_cast<size_t>(wave) * most;
    auto key = [&](int u, int i) {
        const uint32_t at = first + (u * 64 + lane) * E + i;
        return at < V ? key_of(v[u][i], at) : 0;
    };
    auto collect = [&](uint64_t least) {
        int n = 0;
#pragma unroll
        for (int u = 0; u < kHold; ++u)
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (__ballot(v[u][i] >= bound)) append(list, n, most, v[u][i] >= bound && key(u, i) >= least, key(u, i));
        return n;
    };
    int n = collect(1);
    if (n > most) {
        uint64_t best = 0;
#pragma unroll
        for (int u = 0; u < kHold; ++u)
#pragma unroll
            for (int i = 0; i < E; ++i) best = max(best, key(u, i));
        n = collect(max(bound_of<64>(best, s.keep), uint64_t(1)));
    }
    wave_lds_fence();
    sort_best(list, n, s.keep, s.keys + unit * s.keep);
}

// The order of doubles as unsigned numbers above 0; -0 is 0.
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x + 0.0);
    return b >> 63 ? ~b : b | 1ull << 63;
}

__device__ __forceinline__ double beam_score(double base, double total, uint64_t key) {
    return base - log(total) + static_cast<double>(value_of(static_cast<uint32_t>(key >> 32)));
}

// The best candidates of one request: a wave joins a beam's slices, all rank the
// beams' candidates, and the first picks.
__global__ __launch_bounds__(kJoinWaves * 64) void beam_join_kernel(const ks_beams_t x, Slices s, BeamOut out,
                                                                    int64_t request0) {
    extern __shared__ uint64_t lds[];
    const int waves = blockDim.x / 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int W = x.beams, keep = s.keep;
    uint64_t* best = lds;                                             // W x keep
    uint64_t* ranks = best + W * keep;                                // W x keep
    uint64_t* list = ranks + W * keep + wave * keep * kJoinHold;
    // score = base + x - log total, rank = score / divisor
    __shared__ double base[kMaxBeams], total[kMaxBeams], divisor[kMaxBeams];
    __shared__ int length[kMaxBeams], chosen[kMaxBeams];
    const int64_t request = request0 + blockIdx.x;
    for (int w = wave; w < W; w += waves) {
        const int64_t row = request * W + w;
        // everything that may be needed is asked for at once (a beam that is done, or
        // whose score is not finite, has written nothing, and it is not used)
        const float score = x.scores[row];
        const bool done = x.done && x.done[row];
        const uint64_t* keys = s.keys + row * s.slices * keep;
        const int n = s.slices * keep;
        uint64_t mine[kJoinHold];
#pragma unroll
        for (int u = 1; u < kJoinHold; ++u) {
            const int i = (u - 1) * 64 + lane;
            mine[u] = i < n ? keys[i] : 0;
        }
        const float2* st = s.stats + row * s.slices;
        const float2 own = lane < s.slices ? st[lane] : make_float2(kLowest, 0.0f);
        // while the keys are on their way: one wave for all beams, since 16 waves that take
        // a power (or a logarithm: below) each are in each other's way (32 x 16 beams 26 us
        // for 27.6)
        if (w == waves - 1 && lane < W) {
            const int64_t beam = request * W + lane;
            const int len = x.lengths ? x.lengths[beam] + (x.done && x.done[beam] ? 0 : 1) : 0;
            length[lane] = len;
            divisor[lane] = x.length_penalty == 0.0 ? 1.0 : pow(static_cast<double>(max(len, 1)), x.length_penalty);
        }
        double shift = 0.0, all = 1.0;
        bool live = finite(score);
        if (done || !live) {
            for (int i = lane; i < keep; i += 64)
                best[w * keep + i] = i == 0 && live ? key_of(0.0f, static_cast<uint32_t>(x.eos)) : 0;
        } else {
            float top = own.x;
            for (int i = 64 + lane; i < s.slices; i += 64) top = fmaxf(top, st[i].x);
            top = value_of(wave_max(ordered(top)));
            double sum = static_cast<double>(own.y) * exp(static_cast<double>(own.x) - top);
            for (int i = 64 + lane; i < s.slices; i += 64)
                sum += static_cast<double>(st[i].y) * exp(static_cast<double>(st[i].x) - top);
            sum = wave_sum(sum);
            shift = -top;
            all = sum;
            live = live && sum > 0.0 && sum - sum == 0.0;
            // the slices' keys, as many at a time as the list has room for beside
            // the best of those before
            for (int first = 0; first < n; first += 64 * (kJoinHold - 1)) {
                mine[0] = first > 0 && lane < keep ? best[w * keep + lane] : 0;
                uint64_t high = mine[0];
#pragma unroll
                for (int u = 1; u < kJoinHold; ++u) {
                    const int i = first + (u - 1) * 64 + lane;
                    if (first > 0) mine[u] = i < n ? keys[i] : 0;
                    high = max(high, mine[u]);
                }
                // as in a slice: by 16 bits of the values, and with the tokens if too many reach it
                uint64_t least = static_cast<uint64_t>(bound_of<16>(static_cast<uint32_t>(high >> 32), keep)) << 32;
                const int most = keep * kJoinHold;
                auto collect = [&]() {
                    int count = 0;
                    least = max(least, uint64_t(1));
#pragma unroll
                    for (int u = 0; u < kJoinHold; ++u) append(list, count, most, mine[u] >= least, mine[u]);
                    return count;
                };
                int count = collect();
                if (count > most) {
                    least = bound_of<64>(high, keep);
                    count = collect();
                }
                wave_lds_fence();
                sort_best(list, count, keep, best + w * keep);
                wave_lds_fence();
            }
        }
        if (lane == 0) {
            base[w] = live ? static_cast<double>(score) + shift : -INFINITY;
            total[w] = all;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < W * keep; i += blockDim.x) {
        const uint64_t k = best[i];
        const int w = i / keep;
        const double score = beam_score(base[w], total[w], k);
        // no candidate: below every rank
        ranks[i] = k != 0 && base[w] > -INFINITY && score > -INFINITY ? ordered(score / divisor[w]) : 0;
    }
    __syncthreads();
    if (wave != 0) return;
    // lane w goes down beam w's list, the rank after the next at hand
    const uint64_t* mine = ranks + lane * keep;
    int at = 0, found = 0;
    uint64_t rank = lane < W ? mine[0] : 0, after = lane < W && keep > 1 ? mine[1] : 0;
    for (; found < out.beams; ++found) {
        // by their upper halves, and by the lower ones where those are equal
        const uint32_t upper = static_cast<uint32_t>(rank >> 32), high = wave_max(upper);
        if (high == 0) break;                                         // none is left
        unsigned long long best_lanes = __ballot(upper == high);
        if (best_lanes & (best_lanes - 1)) {
            const uint32_t lower = upper == high ? static_cast<uint32_t>(rank) : 0, most = wave_max(lower);
            best_lanes &= __ballot(lower == most);
        }
        if (lane == __ffsll(best_lanes) - 1) {                        // the lowest beam of equal rank
            chosen[found] = lane * keep + at;
            ++at;
            rank = after;
            after = at + 1 < keep ? mine[at + 1] : 0;
        }
    }
    wave_lds_fence();
    if (lane >= out.beams) return;
    const int64_t to = request * out.beams + lane;
    const bool is = lane < found;
    const int pick = is ? chosen[lane] : 0, w = pick / keep;
    const uint64_t k = best[pick];
    const int64_t token = is ? static_cast<int64_t>(0xffffffffu - static_cast<uint32_t>(k)) : x.eos >= 0 ? x.eos : 0;
    out.scores[to] = is ? static_cast<float>(beam_score(base[w], total[w], k)) : -INFINITY;
    out.tokens[to] = token;
    out.parents[to] = is ? w : 0;
    if (out.done) out.done[to] = !is || token == x.eos;
    if (out.lengths) out.lengths[to] = is ? length[w] : 0;
}

// ---------------------------------------------------------------- states
//
// A copy of rows, bound by memory: 64 beams of 2 MB, 268 MB in and out, 36 us
// (7.4 TB/s: a part of it is still in the last cache). Where addresses or rows are no
// multiple of 4 bytes a lane copies one byte at a time and the accesses bound it: rows
// 2 bytes longer take 105 us.

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
template <int N>
struct StateTable {
    StateEntry e[N];
    int32_t count;
};

// A wave copies one piece of one row.
template <typename V>
__device__ __forceinline__ void copy_piece(const StateEntry& e, int64_t row, int64_t from, int64_t piece, bool valid) {
    const int lane = threadIdx.x % 64;
    const int64_t n = e.row_bytes / static_cast<int64_t>(sizeof(V)), at = piece * kPiece * 64 + lane;
    V* dst = reinterpret_cast<V*>(e.dst + row * e.row_bytes) + at;
    const V* src = reinterpret_cast<const V*>(e.src + (valid ? from : 0) * e.row_bytes) + at;
    const int left = static_cast<int>(min(n - at, int64_t(kPiece) * 64));
    constexpr int U = 4;         // on their way at once
#pragma unroll 1
    for (int k0 = 0; k0 < kPiece; k0 += U) {
        V v[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            v[k] = V{};
            if (valid && (k0 + k) * 64 < left) v[k] = src[(k0 + k) * 64];
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if ((k0 + k) * 64 < left) dst[(k0 + k) * 64] = v[k];
    }
}

template <int N>
__global__ __launch_bounds__(256) void beam_reorder_kernel(const StateTable<N> t, const int32_t* parents, int beams,
                                                           int out_beams, int64_t wave0, int64_t waves) {
    const int64_t unit = wave0 + static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
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
    return static_cast<int>((x.vocab + kSlice - 1) / kSlice);
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
    const size_t lds = static_cast<size_t>(kSelectWaves) * s.keep * kHeld * 8;
    const int64_t groups = (units + kSelectWaves - 1) / kSelectWaves;
    for (int64_t g = 0; g < groups; g += kMaxGrid) {
        const ks_status_t st = launch_kernel(bf16 ? beam_slices_kernel<bf16_t> : beam_slices_kernel<float>,
                                             dim3(static_cast<unsigned>(std::min(kMaxGrid, groups - g))),
                                             dim3(kSelectWaves * 64), lds, stream, x, s, g * kSelectWaves);
        if (st != KS_OK) return st;
    }
    const int waves = std::min(kJoinWaves, x.beams);
    const size_t join = static_cast<size_t>(2 * x.beams * s.keep + waves * s.keep * kJoinHold) * 8;
    for (int64_t r = 0; r < x.requests; r += kMaxGrid / 4) {
        const ks_status_t st = launch_kernel(beam_join_kernel,
                                             dim3(static_cast<unsigned>(std::min(kMaxGrid / 4, x.requests - r))),
                                             dim3(waves * 64), join, stream, x, s, out, r);
        if (st != KS_OK) return st;
    }
    return KS_OK;
}

namespace {

// Up to N states a launch, from states[i] on.
template <int N>
ks_status_t reorder_some(const ks_state_t* states, int n, int& i, const int32_t* parents, int64_t requests, int beams,
                         int out_beams, hipStream_t stream) {
    StateTable<N> t;
    t.count = 0;
    int64_t waves = 0;
    for (; i < n && t.count < N; ++i) {
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
    const int64_t groups = (waves + 3) / 4;
    for (int64_t g = 0; g < groups; g += kMaxGrid) {
        const ks_status_t st = launch_kernel(beam_reorder_kernel<N>, dim3(static_cast<unsigned>(std::min(kMaxGrid, groups - g))),
                                             dim3(256), 0, stream, t, parents, beams, out_beams, g * 4, waves);
        if (st != KS_OK) return st;
    }
    return KS_OK;
}

}  // namespace

ks_status_t launch_beam_reorder(const ks_state_t* states, int n, const int32_t* parents, int64_t requests, int beams,
                                int out_beams, hipStream_t stream) {
    ks_status_t st = KS_OK;
    for (int i = 0; i < n && st == KS_OK;)
        st = n <= 8 ? reorder_some<8>(states, n, i, parents, requests, beams, out_beams, stream)
                    : reorder_some<kStates>(states, n, i, parents, requests, beams, out_beams, stream);
    return st;
}

}  // namespace ks
