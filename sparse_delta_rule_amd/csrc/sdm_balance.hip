// A route's balance (include/sdm_train.h): sdm_route_balance and its gradient.
//
// A row's scores as shares of their sum: with o an offset that keeps the largest term
// near 1, e_i = exp(x_i - o) for a softmax, o the largest x, and for a sigmoid e_i = s_i,
// or, where even the largest x is below -64 and 1 + exp(x) rounds to 1, exp(x_i - o).
// Then p_i = e_i / sum e, and parts of a row with offsets of their own are put together
// as parts of a softmax are: the part's sum times exp(its o - the largest o).

#include <type_traits>

#include "sdm_route_device.h"
#include "sdm_train.h"

namespace sdm {

namespace {

constexpr float kDeep = -64.0f;

__device__ __forceinline__ uint32_t live_limit(const BalanceParams& p, uint32_t chunk) {
    const int32_t v = p.chunk_valid != nullptr ? p.chunk_valid[chunk] : int32_t(p.valid);
    return uint32_t(max(v, 0));
}
__device__ __forceinline__ bool is_live(const BalanceParams& p, uint32_t t) {
    const uint32_t c = t / p.chunk;
    return t - c * p.chunk < live_limit(p, c);
}

// The tokens of a workgroup's piece.
struct Piece {
    uint32_t sequence, first, end;
};
__device__ __forceinline__ Piece this_piece(const BalanceParams& p, uint32_t number) {
    Piece r;
    r.sequence = number / p.pieces;
    const uint32_t at = (number - r.sequence * p.pieces) * uint32_t(p.piece), begin = r.sequence * p.sequence;
    r.first = begin + at;
    r.end = begin + min(at + uint32_t(p.piece), p.sequence);
    return r;
}

// VPT keys a lane of THREADS, as they are in memory: loaded ahead of their use.
template <typename E, int THREADS, int VPT, bool VEC> struct RawRow {
    using Row = RowKeys<E, THREADS, VPT, VEC>;
    static constexpr int kN = Row::kN;
    using T = typename std::conditional<VEC, uint4, E>::type;
    T raw[VPT / kN];

    __device__ __forceinline__ void load(const E* row, int keys, int tid) {
#pragma unroll
        for (int i = 0; i < VPT / kN; ++i)
            raw[i] = *reinterpret_cast<const T*>(row + min(Row::key_of(i * kN, tid), keys - kN));
    }
    // Clean logits; -inf past the row's end.
    __device__ __forceinline__ void values(int keys, int tid, float (&c)[VPT]) const {
#pragma unroll
        for (int i = 0; i < VPT / kN; ++i) {
            E e[kN];
            __builtin_memcpy(e, &raw[i], sizeof e);
            const bool in = Row::key_of(i * kN, tid) < keys;
#pragma unroll
            for (int j = 0; j < kN; ++j) c[i * kN + j] = in ? clean(widen(e[j])) : -INFINITY;
        }
    }
};

// The terms of one lane's keys, c[i] -> e_i, given the largest of the part's logits; returns the offset.
template <int N> __device__ __forceinline__ float terms(int score, float largest, float (&c)[N]) {
    if (score == SDM_SOFTMAX) {
        const float o = max32(largest, -FLT_MAX);
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = exp32(c[i] - o);
        return o;
    }
    const bool deep = largest <= kDeep;
    const float o = deep ? max32(largest, -FLT_MAX) : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float e = exp32(deep ? c[i] - o : -c[i]);
        c[i] = deep ? e : __builtin_amdgcn_rcpf(1.0f + e);
    }
    return o;
}

template <int N> __device__ __forceinline__ float sum_of(const float (&x)[N]) {
    float s = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) s += x[i];
    return s;
}

// Counts of the keys [base, base + most) that the piece's live tokens chose, two to a word.
__device__ __forceinline__ void count_choices(const BalanceParams& p, const Piece& r, int base, int most, uint32_t* words) {
    const uint32_t entries = (r.end - r.first) * uint32_t(p.k);
    for (uint32_t e = threadIdx.x; e < entries; e += blockDim.x) {
        const uint32_t t = r.first + e / uint32_t(p.k);
        const int64_t o = int64_t(r.first) * p.k + e;
        const int64_t slot = p.idx64 ? static_cast<const int64_t*>(p.idx)[o] : int64_t(static_cast<const int32_t*>(p.idx)[o]);
        const int64_t key = slot - int64_t(t % p.streams) * p.stream_slots;
        if (key < base || key >= int64_t(base) + most || !is_live(p, t)) continue;
        atomicAdd(words + (uint32_t(key) - uint32_t(base)) / 2, key & 1 ? 0x10000u : 1u);
    }
}

// ------------------------------------------------------------------ first pass: pieces

constexpr int kSmallKeys = 1024;
constexpr int kSmallThreads = 512;

// Rows of at most 1024 keys: LANES lanes a row, VPT keys a lane, whose sums over the piece
// stay in registers and are put together over the workgroup's rows at its end.
template <typename E, int LANES, int VPT, bool VEC>
__global__ __launch_bounds__(kSmallThreads) void balance_small_kernel(BalanceParams p) {
    using Row = RowKeys<E, LANES, VPT, VEC>;
    constexpr int kRows = kSmallThreads / LANES;
    constexpr int kWide = LANES * VPT;  // keys at most
    __shared__ float sums[kRows][kWide];
    __shared__ uint32_t words[kSmallKeys / 2];
    ieee_mode_off();
    const int tid = threadIdx.x, lane = tid % LANES, row = tid / LANES;
    const Piece r = this_piece(p, blockIdx.x);
    const E* logits = static_cast<const E*>(p.logits);
    // Two rows ahead, the first of them before everything else.
    RawRow<E, LANES, VPT, VEC> next[2];
    auto load = [&](uint32_t t, RawRow<E, LANES, VPT, VEC>& to) {
        to.load(logits + int64_t(min(t, r.end - 1)) * p.keys, p.keys, lane);
    };
    load(r.first + row, next[0]);
    load(r.first + row + kRows, next[1]);
    if (blockIdx.x == 0 && tid == 0) *p.done = 0;
    for (int i = tid; i < (p.keys + 1) / 2; i += kSmallThreads) words[i] = 0;
    const int live = __syncthreads_count(r.first + tid < r.end && is_live(p, r.first + tid));
    if (tid == 0) p.live[blockIdx.x] = uint32_t(live);
    count_choices(p, r, 0, p.keys, words);
    float acc[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) acc[i] = 0.0f;
    for (uint32_t t0 = r.first; t0 < r.end; t0 += kRows) {  // the same rounds in every wavefront
        const uint32_t t = t0 + row;
        float c[VPT];
        next[0].values(p.keys, lane, c);
        next[0] = next[1];
        load(t + 2 * kRows, next[1]);
        const float largest = lanes_reduce<LANES>(max_of(c, -INFINITY), [](float a, float b) { return max32(a, b); });
        terms(p.score, largest, c);
        const float sum = lanes_reduce<LANES>(sum_of(c), [](float a, float b) { return a + b; });
        const float f = sum > 0 && t < r.end && is_live(p, t) ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) acc[i] = fmaf(c[i], f, acc[i]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) sums[row][Row::key_of(i, lane)] = acc[i];
    __syncthreads();
    for (int key = tid; key < p.keys; key += kSmallThreads) {
        float s = 0;
        for (int i = 0; i < kRows; ++i) s += sums[i][key];
        p.part[int64_t(blockIdx.x) * p.keys + key] = s;
    }
    const int stride = (p.keys + 1) / 2;
    for (int i = tid; i < stride; i += kSmallThreads) p.part_count[int64_t(blockIdx.x) * stride + i] = words[i];
}

constexpr int kBigThreads = 1024;
constexpr int kCountKeys = 16384;  // keys counted in LDS at a time

// Longer rows: the workgroup takes one row after another, its sums in registers. A wavefront's
// terms have an offset of their own, so a row needs one barrier.
template <typename E, int VPT, bool VEC>
__global__ __launch_bounds__(kBigThreads) void balance_big_kernel(BalanceParams p) {
    using Row = RowKeys<E, kBigThreads, VPT, VEC>;
    constexpr int kWaves = kBigThreads / 64;
    constexpr bool kAhead = VPT * sizeof(E) <= 64;  // the next row is loaded while one is taken
    __shared__ float offset[2][kWaves], total[2][kWaves];
    __shared__ uint32_t words[kCountKeys / 2];
    ieee_mode_off();
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const Piece r = this_piece(p, blockIdx.x);
    const E* logits = static_cast<const E*>(p.logits);
    RawRow<E, kBigThreads, VPT, VEC> next;
    if (kAhead) next.load(logits + int64_t(r.first) * p.keys, p.keys, tid);
    if (blockIdx.x == 0 && tid == 0) *p.done = 0;
    const int live = __syncthreads_count(r.first + tid < r.end && is_live(p, r.first + tid));
    if (tid == 0) p.live[blockIdx.x] = uint32_t(live);
    const int stride = (p.keys + 1) / 2;
    for (int base = 0; base < p.keys; base += kCountKeys) {
        for (int i = tid; i < kCountKeys / 2; i += kBigThreads) words[i] = 0;
        __syncthreads();
        count_choices(p, r, base, kCountKeys, words);
        __syncthreads();
        uint32_t* to = p.part_count + int64_t(blockIdx.x) * stride + base / 2;
        for (int i = tid; i < min(kCountKeys / 2, stride - base / 2); i += kBigThreads) to[i] = words[i];
        __syncthreads();
    }
    float acc[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) acc[i] = 0.0f;
    int buffer = 0;
    for (uint32_t t = r.first; t < r.end; ++t) {
        float c[VPT];
        if (kAhead) {
            next.values(p.keys, tid, c);
            next.load(logits + int64_t(min(t + 1, r.end - 1)) * p.keys, p.keys, tid);
        }
        if (!is_live(p, t)) continue;  // of the whole workgroup
        if (!kAhead) {
            next.load(logits + int64_t(t) * p.keys, p.keys, tid);
            next.values(p.keys, tid, c);
        }
        const float largest = lanes_reduce<64>(max_of(c, -INFINITY), [](float a, float b) { return max32(a, b); });
        const float o = terms(p.score, largest, c);
        const float sum = lanes_reduce<64>(sum_of(c), [](float a, float b) { return a + b; });
        if (lane == 0) {
            offset[buffer][wave] = o;
            total[buffer][wave] = sum;
        }
        __syncthreads();
        float most = -FLT_MAX, z = 0;
        for (int w = 0; w < kWaves; ++w) most = max32(most, offset[buffer][w]);
        for (int w = 0; w < kWaves; ++w) z = fmaf(total[buffer][w], exp32(offset[buffer][w] - most), z);
        const float f = z > 0 ? exp32(o - most) / z : 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) acc[i] = fmaf(c[i], f, acc[i]);
        buffer ^= 1;
    }
    float* out = p.part + int64_t(blockIdx.x) * p.keys;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (Row::key_of(i, tid) < p.keys) out[Row::key_of(i, tid)] = acc[i];
}

// ------------------------------------------------------------------ second pass: sequences

constexpr int kJoinThreads = 1024;
constexpr int kJoinKeys = 64;  // keys of an item

template <typename T> __device__ __forceinline__ T wave_sum(T v) {
    for (int n = 1; n < 64; n *= 2) v += __shfl_xor(v, n);
    return v;
}
template <typename T> __device__ __forceinline__ T join_sum(T v, T* lds) {
    v = wave_sum(v);
    __syncthreads();
    if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
    __syncthreads();
    v = lds[0];
    for (int w = 1; w < kJoinThreads / 64; ++w) v += lds[w];
    return v;
}

// An item is 64 keys of a sequence: the pieces' sums and counts in order, in float64. 16 lanes take
// a piece's keys, four each, so that a workgroup reads 64 pieces at a time. The workgroup that ends
// last puts the items' parts of the loss together.
__global__ __launch_bounds__(kJoinThreads) void balance_join_kernel(BalanceParams p) {
    constexpr int kRows = kJoinThreads / 16, kWaves = kJoinThreads / 64;
    __shared__ double sums[kRows][kJoinKeys];
    __shared__ int32_t counts[kRows][kJoinKeys];
    __shared__ double scratch[kWaves];
    __shared__ uint32_t ticket;
    const int tid = threadIdx.x, row = tid / 16, k0 = tid % 16 * 4;
    const uint32_t blocks = uint32_t(p.keys + kJoinKeys - 1) / kJoinKeys;
    const uint64_t items = uint64_t(p.sequences) * blocks;
    const int stride = (p.keys + 1) / 2;
    const bool vec = p.keys % 4 == 0;  // the pieces' rows are 16-byte vectors of sums, and 8-byte ones of counts
    for (uint64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t g = uint32_t(item / blocks), b = uint32_t(item % blocks);
        const uint64_t first = uint64_t(g) * p.pieces;
        const int key = int(b) * kJoinKeys + k0;
        double n = 0;
        for (uint32_t i = tid; i < p.pieces; i += kJoinThreads) n += p.live[first + i];
        double sum[4] = {};
        int32_t count[4] = {};
        if (key < p.keys) {
#pragma unroll 8
            for (uint32_t i = row; i < p.pieces; i += kRows) {
                const float* part = p.part + (first + i) * p.keys + key;
                const uint32_t* words = p.part_count + (first + i) * stride + key / 2;
                float4 v = {};
                uint2 c = {};
                if (vec) {
                    v = *reinterpret_cast<const float4*>(part);
                    c = *reinterpret_cast<const uint2*>(words);
                } else {
                    v.x = part[0];
                    if (key + 1 < p.keys) v.y = part[1];
                    if (key + 2 < p.keys) v.z = part[2];
                    if (key + 3 < p.keys) v.w = part[3];
                    c.x = words[0];
                    if (key + 2 < p.keys) c.y = words[1];
                }
                sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
                count[0] += c.x & 0xffff, count[1] += c.x >> 16, count[2] += c.y & 0xffff, count[3] += c.y >> 16;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sums[row][k0 + j] = sum[j];
            counts[row][k0 + j] = count[j];
        }
        const uint32_t live = uint32_t(join_sum(n, scratch));  // and a barrier
        if (tid < kJoinKeys) {
            const int key = int(b) * kJoinKeys + tid, rows = int(min(p.pieces, uint32_t(kRows)));
            double s = 0;
            int32_t c = 0;
            for (int r = 0; r < rows; ++r) {
                s += sums[r][tid];
                c += counts[r][tid];
            }
            if (key < p.keys) {
                p.counts[int64_t(g) * p.keys + key] = c;
                p.mean[int64_t(g) * p.keys + key] = live > 0 ? float(s / live) : 0.0f;
            }
            const double part = wave_sum(double(c) * s);
            if (tid == 0) {
                p.loss_part[item] = part;
                if (b == 0) p.live_all[g] = live;
            }
        }
        __syncthreads();
    }
    if (tid == 0) {
        __threadfence();
        ticket = __hip_atomic_fetch_add(p.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (ticket != gridDim.x - 1) return;
    __threadfence();
    double with = 0;
    for (uint32_t g = tid; g < p.sequences; g += kJoinThreads) with += p.live_all[g] > 0;
    const double sequences = join_sum(with, scratch);
    auto coef = [&](uint32_t g) {
        const double n = p.live_all[g];
        return n > 0 ? p.scale * p.keys / (double(p.k) * n * n * sequences) : 0.0;
    };
    double loss = 0;
    for (uint64_t item = tid; item < items; item += kJoinThreads) loss += coef(uint32_t(item / blocks)) * p.loss_part[item];
    for (uint32_t g = tid; g < p.sequences; g += kJoinThreads) p.coef[g] = float(coef(g));
    loss = join_sum(loss, scratch);
    if (tid == 0) *p.loss = float(loss);
}

// No tokens: the one sequence of a call that does not take chunks apart is empty.
__global__ __launch_bounds__(256) void balance_nothing_kernel(BalanceParams p) {
    const int64_t n = int64_t(p.sequences) * p.keys;
    for (int64_t i = threadIdx.x; i < n; i += 256) {
        p.counts[i] = 0;
        p.mean[i] = 0.0f;
    }
    if (threadIdx.x < p.sequences) p.coef[threadIdx.x] = 0.0f;
    if (threadIdx.x == 0) *p.loss = 0.0f;
}

// ------------------------------------------------------------------ backward

// The difference of two counts as float32 (a difference past 2^31 cannot be: a sequence has
// fewer choices).
__device__ __forceinline__ float apart(int32_t a, int32_t b) { return float(int32_t(uint32_t(a) - uint32_t(b))); }

// A lane's VPT gradients: p_i ((c_i - top) - d), and for a sigmoid times 1 - s_i, times f.
template <int N>
__device__ __forceinline__ void gradients(int score, const float (&x)[N], const float (&e)[N], const int32_t (&count)[N],
                                          int32_t top, float share, float d, float f, float (&out)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float s = e[i] * share;
        float v = s * (apart(count[i], top) - d) * f;
        if (score == SDM_SIGMOID) v *= __builtin_amdgcn_rcpf(1.0f + exp32(x[i]));
        out[i] = s > 0 ? v : 0.0f;  // also where f is not finite
    }
}

template <typename E, typename Row, int VPT, bool VEC>
__device__ __forceinline__ void store_row(E* out, int keys, int tid, const float (&g)[VPT], bool add) {
    constexpr int kN = Row::kN;
#pragma unroll
    for (int i = 0; i < VPT; i += kN) {
        const int key = Row::key_of(i, tid);
        if (key >= keys) continue;
        if constexpr (VEC) {
            float v[kN];
#pragma unroll
            for (int j = 0; j < kN; ++j) v[j] = g[i + j];
            if (add) {
                const uint4 raw = *reinterpret_cast<const uint4*>(out + key);
                E old[kN];
                __builtin_memcpy(old, &raw, 16);
#pragma unroll
                for (int j = 0; j < kN; ++j) v[j] += widen(old[j]);
            }
            *reinterpret_cast<uint4*>(out + key) = Pack<E, 16>::of(v);
        } else {
            out[key] = narrow<E>(add ? widen(out[key]) + g[i] : g[i]);
        }
    }
}

__device__ __forceinline__ float row_factor(const BalanceParams& p, uint32_t sequence) {
    return p.coef[sequence] * (p.dloss != nullptr ? *p.dloss : 1.0f);
}

template <typename Row, int VPT>
__device__ __forceinline__ void load_counts(const BalanceParams& p, uint32_t sequence, int tid, int32_t (&count)[VPT]) {
    const int32_t* counts = p.counts + int64_t(sequence) * p.keys;
#pragma unroll
    for (int i = 0; i < VPT; ++i) count[i] = counts[min(Row::key_of(i, tid), p.keys - 1)];
}

template <typename E, int LANES, int VPT, bool VEC>
__global__ __launch_bounds__(kSmallThreads) void balance_backward_small_kernel(BalanceParams p) {
    using Row = RowKeys<E, LANES, VPT, VEC>;
    constexpr int kRows = kSmallThreads / LANES;
    ieee_mode_off();
    const int tid = threadIdx.x, lane = tid % LANES, row = tid / LANES;
    const Piece r = this_piece(p, blockIdx.x);
    const E* logits = static_cast<const E*>(p.logits);
    E* dlogits = static_cast<E*>(p.dlogits);
    RawRow<E, LANES, VPT, VEC> next[2];  // two rows ahead
    auto load = [&](uint32_t t, RawRow<E, LANES, VPT, VEC>& to) {
        to.load(logits + int64_t(min(t, r.end - 1)) * p.keys, p.keys, lane);
    };
    load(r.first + row, next[0]);
    load(r.first + row + kRows, next[1]);
    int32_t count[VPT];
    load_counts<Row>(p, r.sequence, lane, count);
    const float f = row_factor(p, r.sequence);
    for (uint32_t t = r.first + row; t < r.end; t += kRows) {
        const bool live = is_live(p, t);
        float x[VPT], e[VPT], g[VPT];
        next[0].values(p.keys, lane, x);
        next[0] = next[1];
        load(t + 2 * kRows, next[1]);
        const float largest = lanes_reduce<LANES>(max_of(x, -INFINITY), [](float a, float b) { return max32(a, b); });
        int32_t top = INT32_MIN;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            e[i] = x[i];
            top = x[i] == largest && Row::key_of(i, lane) < p.keys ? max(top, count[i]) : top;
        }
        top = lanes_reduce<LANES>(top, [](int32_t a, int32_t b) { return max(a, b); });
        terms(p.score, largest, e);
        float z = 0, d = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            z += e[i];
            d = fmaf(e[i], apart(count[i], top), d);
        }
        z = lanes_reduce<LANES>(z, [](float a, float b) { return a + b; });
        d = lanes_reduce<LANES>(d, [](float a, float b) { return a + b; });
        const float share = z > 0 && live ? 1.0f / z : 0.0f;
        gradients(p.score, x, e, count, top, share, d * share, f, g);
        if (live || !p.accumulate) store_row<E, Row, VPT, VEC>(dlogits + int64_t(t) * p.keys, p.keys, lane, g, p.accumulate);
    }
}

template <typename E, int VPT, bool VEC>
__global__ __launch_bounds__(kBigThreads) void balance_backward_big_kernel(BalanceParams p) {
    using Row = RowKeys<E, kBigThreads, VPT, VEC>;
    constexpr int kWaves = kBigThreads / 64;
    __shared__ float largest_of[2][kWaves], offset[2][kWaves], total[2][kWaves], dot[2][kWaves];
    __shared__ int32_t top_of[2][kWaves];
    ieee_mode_off();
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const Piece r = this_piece(p, blockIdx.x);
    const E* logits = static_cast<const E*>(p.logits);
    E* dlogits = static_cast<E*>(p.dlogits);
    constexpr bool kAhead = VPT * sizeof(E) <= 64;  // the next row is loaded while one is taken
    RawRow<E, kBigThreads, VPT, VEC> next;
    if (kAhead) next.load(logits + int64_t(r.first) * p.keys, p.keys, tid);
    int32_t count[VPT];
    load_counts<Row>(p, r.sequence, tid, count);
    const float f = row_factor(p, r.sequence);
    int buffer = 0;
    for (uint32_t t = r.first; t < r.end; ++t) {
        E* out = dlogits + int64_t(t) * p.keys;
        float x[VPT], e[VPT], g[VPT];
        if (kAhead) {
            next.values(p.keys, tid, x);
            next.load(logits + int64_t(min(t + 1, r.end - 1)) * p.keys, p.keys, tid);
        }
        if (!is_live(p, t)) {  // of the whole workgroup
            if (!p.accumulate) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) g[i] = 0.0f;
                store_row<E, Row, VPT, VEC>(out, p.keys, tid, g, false);
            }
            continue;
        }
        if (!kAhead) {
            next.load(logits + int64_t(t) * p.keys, p.keys, tid);
            next.values(p.keys, tid, x);
        }
        const float largest = lanes_reduce<64>(max_of(x, -INFINITY), [](float a, float b) { return max32(a, b); });
        int32_t mine = INT32_MIN;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            e[i] = x[i];
            mine = x[i] == largest && Row::key_of(i, tid) < p.keys ? max(mine, count[i]) : mine;
        }
        mine = lanes_reduce<64>(mine, [](int32_t a, int32_t b) { return max(a, b); });
        const float o = terms(p.score, largest, e);
        float z = 0, d = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            z += e[i];
            d = fmaf(e[i], apart(count[i], mine), d);
        }
        z = lanes_reduce<64>(z, [](float a, float b) { return a + b; });
        d = lanes_reduce<64>(d, [](float a, float b) { return a + b; });
        if (lane == 0) {
            largest_of[buffer][wave] = largest;
            offset[buffer][wave] = o;
            total[buffer][wave] = z;
            dot[buffer][wave] = d;
            top_of[buffer][wave] = mine;
        }
        __syncthreads();
        float most = -FLT_MAX, highest = -INFINITY;
        int32_t top = INT32_MIN;
        for (int w = 0; w < kWaves; ++w) {
            most = max32(most, offset[buffer][w]);
            highest = max32(highest, largest_of[buffer][w]);
        }
        for (int w = 0; w < kWaves; ++w) top = largest_of[buffer][w] == highest ? max(top, top_of[buffer][w]) : top;
        z = 0;
        d = 0;
        for (int w = 0; w < kWaves; ++w) {
            const float part = exp32(offset[buffer][w] - most), sum = total[buffer][w] * part;
            z += sum;
            d += fmaf(sum, apart(top_of[buffer][w], top), dot[buffer][w] * part);
        }
        const float share = z > 0 ? 1.0f / z : 0.0f;
        gradients(p.score, x, e, count, top, share * exp32(o - most), d * share, f, g);
        store_row<E, Row, VPT, VEC>(out, p.keys, tid, g, p.accumulate);
        buffer ^= 1;
    }
}

// ------------------------------------------------------------------ launches

constexpr int64_t kPieces = 512, kBigPieces = 256;  // pieces wanted of a call with many tokens

template <typename E, int LANES, int VPT> void run_small(const BalanceParams& p, bool vec, bool backward, hipStream_t s) {
    const dim3 grid{unsigned(p.sequences * p.pieces)}, block{kSmallThreads};
    if (vec && backward) hipLaunchKernelGGL((balance_backward_small_kernel<E, LANES, VPT, true>), grid, block, 0, s, p);
    else if (backward) hipLaunchKernelGGL((balance_backward_small_kernel<E, LANES, VPT, false>), grid, block, 0, s, p);
    else if (vec) hipLaunchKernelGGL((balance_small_kernel<E, LANES, VPT, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((balance_small_kernel<E, LANES, VPT, false>), grid, block, 0, s, p);
}
template <typename E, int VPT> void run_big(const BalanceParams& p, bool vec, bool backward, hipStream_t s) {
    const dim3 grid{unsigned(p.sequences * p.pieces)}, block{kBigThreads};
    if (vec && backward) hipLaunchKernelGGL((balance_backward_big_kernel<E, VPT, true>), grid, block, 0, s, p);
    else if (backward) hipLaunchKernelGGL((balance_backward_big_kernel<E, VPT, false>), grid, block, 0, s, p);
    else if (vec) hipLaunchKernelGGL((balance_big_kernel<E, VPT, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((balance_big_kernel<E, VPT, false>), grid, block, 0, s, p);
}
template <typename E> void run_rows(const BalanceParams& p, bool backward, hipStream_t s) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.logits) | (backward ? reinterpret_cast<uintptr_t>(p.dlogits) : 0);
    const bool vec = at % 16 == 0 && p.keys * sizeof(E) % 16 == 0;
    if (p.keys <= 128) run_small<E, 16, 8>(p, vec, backward, s);
    else if (p.keys <= 256) run_small<E, 32, 8>(p, vec, backward, s);
    else if (p.keys <= 512) run_small<E, 64, 8>(p, vec, backward, s);
    else if (p.keys <= 1024) run_small<E, 64, 16>(p, vec, backward, s);
    else if (p.keys <= 8192) run_big<E, 8>(p, vec, backward, s);
    else if (p.keys <= 16384) run_big<E, 16>(p, vec, backward, s);
    else if (p.keys <= 32768) run_big<E, 32>(p, vec, backward, s);
    else run_big<E, 64>(p, vec, backward, s);
}

}  // namespace

int64_t balance_layout(BalanceParams* p, void* workspace) {
    p->sequence = p->per_chunk ? p->chunk : p->tokens;
    p->sequences = p->per_chunk ? p->tokens / p->chunk : 1;
    const int64_t wanted = p->keys > kSmallKeys ? kBigPieces : kPieces;
    int64_t piece = (int64_t(p->tokens) + wanted - 1) / wanted;
    if (piece > kMaxPiece) piece = kMaxPiece;
    if (piece > p->sequence) piece = p->sequence;
    if (piece < 1) piece = 1;
    p->piece = int(piece);
    p->pieces = uint32_t((p->sequence + piece - 1) / piece);
    const int64_t pieces = int64_t(p->sequences) * p->pieces, blocks = (p->keys + kJoinKeys - 1) / kJoinKeys;
    char* base = static_cast<char*>(workspace);
    int64_t used = 0;
    auto place = [&](int64_t bytes) {
        char* at = base != nullptr ? base + used : nullptr;
        used += (bytes + 15) / 16 * 16;
        return at;
    };
    p->done = reinterpret_cast<uint32_t*>(place(4));
    p->live = reinterpret_cast<uint32_t*>(place(4 * pieces));
    p->live_all = reinterpret_cast<uint32_t*>(place(4 * int64_t(p->sequences)));
    p->loss_part = reinterpret_cast<double*>(place(8 * int64_t(p->sequences) * blocks));
    p->part = reinterpret_cast<float*>(place(4 * pieces * p->keys));
    p->part_count = reinterpret_cast<uint32_t*>(place(4 * pieces * ((p->keys + 1) / 2)));
    return used;
}

hipError_t launch_balance(const BalanceParams& p, bool bf16, hipStream_t stream) {
    if (p.tokens == 0) {
        hipLaunchKernelGGL(balance_nothing_kernel, dim3(1), dim3(256), 0, stream, p);
        return hipGetLastError();
    }
    if (bf16) run_rows<uint16_t>(p, false, stream);
    else run_rows<float>(p, false, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    int64_t items = int64_t(p.sequences) * ((p.keys + kJoinKeys - 1) / kJoinKeys);
    if (items > 65536) items = 65536;
    hipLaunchKernelGGL(balance_join_kernel, dim3(unsigned(items)), dim3(kJoinThreads), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceParams& p, bool bf16, hipStream_t stream) {
    if (bf16) run_rows<uint16_t>(p, true, stream);
    else run_rows<float>(p, true, stream);
    return hipGetLastError();
}

}  // namespace sdm
