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
    const uint32_t c = divide(t, p.by_chunk);
    return t - c * p.chunk < live_limit(p, c);
}

struct Larger {
    __device__ __forceinline__ float operator()(float a, float b) const { return max32(a, b); }
};
struct Plus {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
constexpr Larger larger{};
constexpr Plus plus{};

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
        constexpr uint32_t kMinusInf = sizeof(E) == 2 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
        for (int i = 0; i < VPT / kN; ++i) {
            E e[kN];
            if constexpr (VEC) {
                const uint32_t in = uint32_t((Row::key_of(i * kN, tid) - keys) >> 31);  // all ones where the row has the vector
                uint4 v = raw[i];
                v.x = (v.x & in) | (kMinusInf & ~in), v.y = (v.y & in) | (kMinusInf & ~in);
                v.z = (v.z & in) | (kMinusInf & ~in), v.w = (v.w & in) | (kMinusInf & ~in);
                opaque(v);  // four words chosen, not each key
                __builtin_memcpy(e, &v, 16);
            } else {
                e[0] = raw[i];
            }
#pragma unroll
            for (int j = 0; j < kN; ++j) c[i * kN + j] = clean(VEC || Row::key_of(i, tid) < keys ? widen(e[j]) : -INFINITY);
        }
    }
};

// f over the LANES (16, 32 or 64) neighbouring lanes of a row, without LDS: gfx950 swaps rows of 16
// and halves of 32 lanes between two registers.
template <int LANES, typename T, typename F> __device__ __forceinline__ T reduce(T v, F f) {
    v = lanes_reduce<16>(v, f);
    auto both = [&](auto pair) {
        const uint32_t a = pair[0], b = pair[1];
        T x, y;
        __builtin_memcpy(&x, &a, 4);
        __builtin_memcpy(&y, &b, 4);
        v = f(x, y);
    };
    auto bits = [&] {
        uint32_t u;
        __builtin_memcpy(&u, &v, 4);
        return u;
    };
    if constexpr (LANES >= 32) both(__builtin_amdgcn_permlane16_swap(bits(), bits(), false, false));
    if constexpr (LANES >= 64) both(__builtin_amdgcn_permlane32_swap(bits(), bits(), false, false));
    return v;
}

// What holds for all lanes of a row or for none: a branch of the wavefront where that is the row's. (Of
// more rows it is not: a row's path, and so its bits, would be its neighbours'.)
template <int LANES> __device__ __forceinline__ bool all_of(bool holds) {
    return LANES == 64 ? __ballot(!holds) == 0 : holds;
}

// The terms of one lane's keys, c[i] -> e_i, given the largest of the part's logits; returns the
// offset. scale: what every e_i is to be multiplied by to be relative to that offset: an exponential
// by one fused operation, 2^(x L - q) with q = o L rounded, has what q's rounding puts into all of
// them, 2^(o L - q), taken out there. rest (may be NULL): 1 - s_i of a sigmoid, for positive x the
// exponential's own share, so that it is as precise as s_i is for negative x.
template <int LANES, int N>
__device__ __forceinline__ float terms(int score, float largest, float (&c)[N], float* rest, float& scale) {
    constexpr float kL = 1.44269504f;
    scale = 1.0f;
    if (score == SDM_SOFTMAX) {
        const float o = max32(largest, -FLT_MAX);
        if (all_of<LANES>(fabsf(o) < 65536.0f)) {
            const float q = o * kL;
#pragma unroll
            for (int i = 0; i < N; ++i) c[i] = __builtin_amdgcn_exp2f(fmaf(c[i], kL, -q));
            scale = __builtin_amdgcn_exp2f(-fmaf(o, kL, -q));
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) c[i] = exp32(c[i] - o);
        }
        return o;
    }
    const bool deep = largest <= kDeep;
    const float o = deep ? max32(largest, -FLT_MAX) : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float e = exp32(deep ? c[i] - o : -c[i]), s = __builtin_amdgcn_rcpf(1.0f + e);
        if (rest != nullptr) rest[i] = deep ? 1.0f : c[i] > 0 ? e * s : 1.0f - s;
        c[i] = deep ? e : s;
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
        const uint32_t t = r.first + divide(e, p.by_k);
        const int64_t o = int64_t(r.first) * p.k + e;
        const int64_t slot = p.idx64 ? static_cast<const int64_t*>(p.idx)[o] : int64_t(static_cast<const int32_t*>(p.idx)[o]);
        const int64_t key = p.stream_slots == 0 ? slot : slot - int64_t(t % p.streams) * p.stream_slots;
        if (key < base || key >= int64_t(base) + most || !is_live(p, t)) continue;
        atomicAdd(words + (uint32_t(key) - uint32_t(base)) / 2, key & 1 ? 0x10000u : 1u);
    }
}

// ------------------------------------------------------------------ first pass: pieces

constexpr int kSmallKeys = 1024;
constexpr int kSmallThreads = 512;

// Rows of at most 1024 keys: LANES lanes a row, VPT keys a lane, whose sums over the piece
// stay in registers and are put together over the workgroup's rows at its end. 32768 x 256 float32
// keys, 30 MB of live rows, take 10.6 us and the second pass 7.6: both bound by the latency of
// their steps (5 us are the bytes'), as 512 pieces are two workgroups a compute unit.
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
        const float largest = reduce<LANES>(max_of(c, -INFINITY), larger);
        float scale;  // of all of the row's terms
        terms<LANES>(p.score, largest, c, nullptr, scale);
        const float sum = reduce<LANES>(sum_of(c), plus);
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

constexpr int kCountKeys = 16384;  // keys counted in LDS at a time

// Longer rows: the workgroup takes one row after another, its sums in registers. A wavefront's
// terms have an offset of their own, so a row needs one barrier. Rows of more than 32768 keys are
// taken in parts, which are read again for their shares: a lane's 64 keys and 64 sums do not fit its
// registers (1024 rows of 65536 bfloat16 keys: 228 us with both there, 194 in parts). 4096 rows of
// 16384 bfloat16 keys take 35 us, 3.9 TB/s: the instructions (200 for a wavefront's part of a row)
// are 24 us of it, one barrier a row with 16 wavefronts a compute unit the rest.
template <typename E, int THREADS, int VPT, int PARTS, bool VEC>
__global__ __launch_bounds__(THREADS) void balance_big_kernel(BalanceParams p) {
    using Row = RowKeys<E, THREADS, VPT, VEC>;
    constexpr int kWaves = THREADS / 64, kPart = THREADS * VPT;
    constexpr bool kAhead = PARTS == 1 && VPT * sizeof(E) <= 64;  // the next row is loaded while one is taken
    __shared__ float offset[2][kWaves], total[2][kWaves];
    __shared__ uint32_t words[kCountKeys / 2];
    ieee_mode_off();
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const Piece r = this_piece(p, blockIdx.x);
    const E* logits = static_cast<const E*>(p.logits);
    RawRow<E, THREADS, VPT, VEC> next;
    if (kAhead) next.load(logits + int64_t(r.first) * p.keys, p.keys, tid);
    if (blockIdx.x == 0 && tid == 0) *p.done = 0;
    const int live = __syncthreads_count(r.first + tid < r.end && is_live(p, r.first + tid));
    if (tid == 0) p.live[blockIdx.x] = uint32_t(live);
    const int stride = (p.keys + 1) / 2;
    for (int base = 0; base < p.keys; base += kCountKeys) {
        for (int i = tid; i < kCountKeys / 2; i += THREADS) words[i] = 0;
        __syncthreads();
        count_choices(p, r, base, kCountKeys, words);
        __syncthreads();
        uint32_t* to = p.part_count + int64_t(blockIdx.x) * stride + base / 2;
        for (int i = tid; i < min(kCountKeys / 2, stride - base / 2); i += THREADS) to[i] = words[i];
        __syncthreads();
    }
    float acc[PARTS][VPT];
#pragma unroll
    for (int h = 0; h < PARTS; ++h)
#pragma unroll
        for (int i = 0; i < VPT; ++i) acc[h][i] = 0.0f;
    int buffer = 0;
    for (uint32_t t = r.first; t < r.end; ++t) {
        const E* row = logits + int64_t(t) * p.keys;
        float c[VPT];
        if (kAhead) {
            next.values(p.keys, tid, c);
            next.load(logits + int64_t(min(t + 1, r.end - 1)) * p.keys, p.keys, tid);
        }
        if (!is_live(p, t)) continue;  // of the whole workgroup
        // A part's terms, relative to an offset of its own.
        float o, scale;
        auto take = [&](int h) {
            if (!kAhead) {
                next.load(row + h * kPart, p.keys - h * kPart, tid);
                next.values(p.keys - h * kPart, tid, c);
            }
            o = terms<64>(p.score, reduce<64>(max_of(c, -INFINITY), larger), c, nullptr, scale);
        };
        float mine = -FLT_MAX, its = 0;
#pragma unroll 1
        for (int h = 0; h < PARTS; ++h) {
            take(h);
            const float sum = reduce<64>(sum_of(c), plus) * scale, most = max32(mine, o);
            its = PARTS == 1 ? sum : its * exp32(mine - most) + sum * exp32(o - most);
            mine = most;
        }
        if (lane == 0) {
            offset[buffer][wave] = mine;
            total[buffer][wave] = its;
        }
        __syncthreads();
        // A lane for each wavefront's part, in every 16 lanes.
        const int w = lane % 16 % kWaves;
        const float part = offset[buffer][w], most = lanes_reduce<16>(part, larger);
        const float z = lanes_reduce<16>(lane % 16 < kWaves ? total[buffer][w] * exp32(part - most) : 0.0f, plus);
#pragma unroll
        for (int h = 0; h < PARTS; ++h) {
            if (PARTS > 1) take(h);
            const float f = z > 0 ? scale * exp32(o - most) / z : 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) acc[h][i] = fmaf(c[i], f, acc[h][i]);
        }
        buffer ^= 1;
    }
    float* out = p.part + int64_t(blockIdx.x) * p.keys;
#pragma unroll
    for (int h = 0; h < PARTS; ++h) {
#pragma unroll
        for (int i = 0; i < VPT; i += VEC ? 4 : 1) {
            const int key = h * kPart + Row::key_of(i, tid);
            if (key >= p.keys) continue;
            if constexpr (VEC) *reinterpret_cast<float4*>(out + key) = make_float4(acc[h][i], acc[h][i + 1], acc[h][i + 2], acc[h][i + 3]);
            else out[key] = acc[h][i];
        }
    }
}

// ------------------------------------------------------------------ second pass: sequences

constexpr int kJoinKeys = 64;  // keys of an item

template <typename T> __device__ __forceinline__ T wave_sum(T v) {
    for (int n = 1; n < 64; n *= 2) v += __shfl_xor(v, n);
    return v;
}
template <int THREADS, typename T> __device__ __forceinline__ T join_sum(T v, T* lds) {
    v = wave_sum(v);
    __syncthreads();
    if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
    __syncthreads();
    v = lds[0];
    for (int w = 1; w < THREADS / 64; ++w) v += lds[w];
    return v;
}

// An item is 64 keys of a sequence: the pieces' sums and counts in order, in float64. 16 lanes take
// a piece's keys, four each, so that a workgroup reads THREADS / 16 pieces at a time. The workgroup
// that ends last puts the items' parts of the loss together.
template <int THREADS> __global__ __launch_bounds__(THREADS) void balance_join_kernel(BalanceParams p) {
    constexpr int kRows = THREADS / 16, kWaves = THREADS / 64;
    __shared__ double sums[kWaves][kJoinKeys];
    __shared__ int32_t counts[kWaves][kJoinKeys];
    __shared__ double scratch[kWaves];
    __shared__ uint32_t ticket;
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, row = tid / 16, k0 = tid % 16 * 4;
    const uint32_t blocks = uint32_t(p.keys + kJoinKeys - 1) / kJoinKeys;
    const uint64_t items = uint64_t(p.sequences) * blocks;
    const int stride = (p.keys + 1) / 2;
    const bool vec = p.keys % 4 == 0;  // the pieces' rows are 16-byte vectors of sums, and 8-byte ones of counts
    for (uint64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t g = uint32_t(item / blocks), b = uint32_t(item % blocks);
        const uint64_t first = uint64_t(g) * p.pieces;
        const int key = int(b) * kJoinKeys + k0;
        double n = 0;
        for (uint32_t i = tid; i < p.pieces; i += THREADS) n += p.live[first + i];
        double sum[4] = {};
        int32_t count[4] = {};
        if (key < p.keys) {
#pragma unroll 4
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
            sum[j] += __shfl_xor(sum[j], 16);
            sum[j] += __shfl_xor(sum[j], 32);
            count[j] += __shfl_xor(count[j], 16);
            count[j] += __shfl_xor(count[j], 32);
        }
        if (lane < 16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sums[wave][k0 + j] = sum[j];
                counts[wave][k0 + j] = count[j];
            }
        }
        const uint32_t live = uint32_t(join_sum<THREADS>(n, scratch));  // and a barrier
        if (wave == 0) {
            const int mine = int(b) * kJoinKeys + lane;
            double s = 0;
            int32_t c = 0;
            for (int w = 0; w < kWaves; ++w) {
                s += sums[w][lane];
                c += counts[w][lane];
            }
            if (mine < p.keys) {
                p.counts[int64_t(g) * p.keys + mine] = c;
                p.mean[int64_t(g) * p.keys + mine] = live > 0 ? float(s / live) : 0.0f;
            }
            const double part = wave_sum(double(c) * s);
            if (lane == 0) {
                p.loss_part[item] = part;
                if (b == 0) p.live_all[g] = live;
            }
        }
        __syncthreads();
    }
    // Thread 0's own stores are what the last workgroup reads: its release, and the other thread 0's
    // acquire and the barrier behind it, are all that this needs.
    if (tid == 0) ticket = __hip_atomic_fetch_add(p.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (ticket != gridDim.x - 1) return;
    double with = 0;
    for (uint32_t g = tid; g < p.sequences; g += THREADS) with += p.live_all[g] > 0;
    const double sequences = join_sum<THREADS>(with, scratch);
    auto coef = [&](uint32_t g) {
        const double n = p.live_all[g];
        return n > 0 ? p.scale * p.keys / (double(p.k) * n * n * sequences) : 0.0;
    };
    double loss = 0;
    for (uint64_t item = tid; item < items; item += THREADS) loss += coef(uint32_t(item / blocks)) * p.loss_part[item];
    for (uint32_t g = tid; g < p.sequences; g += THREADS) p.coef[g] = float(coef(g));
    loss = join_sum<THREADS>(loss, scratch);
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
//
// With p_i = e_i / z a row's gradient is p_i (f_i - sum_j f_j p_j), and as the p_i sum to 1 it stays
// the same when a constant is taken from all f_i. The counts are taken relative to their mean, which
// keeps them small where a route is balanced; in a row where one key has nearly all of the share,
// relative to that key's count, so that its own gradient, a sum over the others, loses nothing.

constexpr float kMostShare = 0.8f;

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

// A lane's counts; returns their sum. (In float64: counts that were added up over many devices may sum
// to more than an integer of 32 bits holds.)
template <typename Row, int VPT>
__device__ __forceinline__ double load_counts(const int32_t* counts, int keys, int tid, int32_t (&count)[VPT]) {
    if (Row::kN > 1 && reinterpret_cast<uintptr_t>(counts) % 16 == 0) {  // rows of whole vectors
#pragma unroll
        for (int i = 0; i + 3 < VPT; i += 4) {
            const int4 v = *reinterpret_cast<const int4*>(counts + min(Row::key_of(i, tid), keys - 4));
            count[i] = v.x, count[i + 1] = v.y, count[i + 2] = v.z, count[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) count[i] = counts[min(Row::key_of(i, tid), keys - 1)];
    }
    double sum = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) sum += Row::key_of(i, tid) < keys ? double(count[i]) : 0.0;
    return sum;
}
template <int LANES> __device__ __forceinline__ double lanes_sum(double v) {
    for (int n = 1; n < LANES; n *= 2) v += __shfl_xor(v, n);
    return v;
}
// The differences to `from`, exact below 2^24.
template <int N> __device__ __forceinline__ void apart(const int32_t (&count)[N], int32_t from, float (&c)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = float(int32_t(uint32_t(count[i]) - uint32_t(from)));
}

// sum_i e_i (c_i - top) of one lane.
template <int N> __device__ __forceinline__ float dot_of(const float (&e)[N], const float (&c)[N], float top) {
    float d = 0;
    if (top == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) d = fmaf(e[i], c[i], d);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) d = fmaf(e[i], c[i] - top, d);
    }
    return d;
}

// A lane's gradients, e[i] -> e_i share ((c_i - top) - d) f, and for a sigmoid times 1 - s_i.
template <int LANES, int N>
__device__ __forceinline__ void gradients(int score, const float (&rest)[N], const float (&c)[N], float top, float share, float d,
                                          float f, float (&e)[N]) {
    const float k = share * f;
    // Differences of counts are below 2^33, so that a product of k and one is finite. Otherwise a key's own
    // share comes first, whose product is infinite only where the gradient is; one of score 0 has the
    // gradient 0 all the same.
    if (!all_of<LANES>(fabsf(k) < 0x1p90f && fabsf(d) < INFINITY)) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float s = e[i] * share, v = s * (score == SDM_SIGMOID ? rest[i] : 1.0f) * ((c[i] - top) - d) * f;
            e[i] = s > 0 ? v : 0.0f;
        }
        return;
    }
    if (top == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] *= k * (c[i] - d);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] *= k * ((c[i] - top) - d);
    }
    if (score == SDM_SIGMOID) {
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] *= rest[i];
    }
}

// The largest term that a part with this largest logit and offset has (relative to that offset).
__device__ __forceinline__ float largest_term(int score, float largest, float o) {
    if (score == SDM_SIGMOID && largest > kDeep) return __builtin_amdgcn_rcpf(1.0f + exp32(-largest));
    return exp32(largest - o);  // 1, or 0 where no key has a score
}
// The count of one lane's keys that have the row's largest term.
template <typename Row, int VPT>
__device__ __forceinline__ float count_of_largest(const float (&e)[VPT], const float (&c)[VPT], float largest, int keys, int tid) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPT; ++i) top = e[i] == largest && Row::key_of(i, tid) < keys ? max32(top, c[i]) : top;
    return top;
}

// 32768 x 256 float32 keys: 15 us. A copy of as many bytes takes 9 (the caches hold a part), the 5.1 M
// vector instructions some 9; neither fills the other's gaps, with two workgroups a compute unit.
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
    float c[VPT];
    {
        int32_t count[VPT];
        const double sum = lanes_sum<LANES>(load_counts<Row>(p.counts + int64_t(r.sequence) * p.keys, p.keys, lane, count));
        apart(count, int32_t(sum / p.keys), c);
    }
    const float f = row_factor(p, r.sequence);
    for (uint32_t t0 = r.first; t0 < r.end; t0 += kRows) {  // the same rounds in every wavefront
        const uint32_t t = t0 + row;
        const bool there = t < r.end, live = there && is_live(p, t);
        float e[VPT], rest[VPT], scale;
        next[0].values(p.keys, lane, e);
        next[0] = next[1];
        load(t + 2 * kRows, next[1]);
        const float largest = reduce<LANES>(max_of(e, -INFINITY), larger);
        const float o = terms<LANES>(p.score, largest, e, rest, scale);
        const float z = reduce<LANES>(sum_of(e), plus);
        const float share = z > 0 && live ? 1.0f / z : 0.0f;
        float top = 0;
        const bool confident = share * largest_term(p.score, largest, o) > kMostShare;
        if (__ballot(confident) != 0) {  // of any row of the wavefront; the others keep the mean
            const float most = reduce<LANES>(max_of(e, 0.0f), larger);
            const float its = reduce<LANES>(count_of_largest<Row>(e, c, most, p.keys, lane), larger);
            top = confident ? its : 0.0f;
        }
        const float d = reduce<LANES>(dot_of(e, c, top), plus);
        gradients<LANES>(p.score, rest, c, top, share, d * share, f, e);
        if (there && (live || !p.accumulate))
            store_row<E, Row, VPT, VEC>(dlogits + int64_t(t) * p.keys, p.keys, lane, e, p.accumulate);
    }
}

// A row at a time, the counts in registers. 4096 rows of 16384 bfloat16 keys: 59 to 63 us, 4.3 to 4.5
// TB/s read and written, with 41 us of instructions. Rows of more than
// 16384 keys, and of more than 8192 that are not whole vectors, do not fit the registers (32768 float32
// keys spill 32, or 118).
template <typename E, int THREADS, int VPT, bool VEC>
__global__ __launch_bounds__(THREADS) void balance_backward_big_kernel(BalanceParams p) {
    using Row = RowKeys<E, THREADS, VPT, VEC>;
    constexpr int kWaves = THREADS / 64;
    constexpr bool kAhead = VPT * sizeof(E) <= 64;  // the next row is loaded while one is taken
    __shared__ float offset[2][kWaves], total[2][kWaves], dot[2][kWaves], term[2][kWaves];
    __shared__ float again[2][kWaves];
    __shared__ double sums[kWaves];
    ieee_mode_off();
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const Piece r = this_piece(p, blockIdx.x);
    const E* logits = static_cast<const E*>(p.logits);
    E* dlogits = static_cast<E*>(p.dlogits);
    RawRow<E, THREADS, VPT, VEC> next;
    if (kAhead) next.load(logits + int64_t(r.first) * p.keys, p.keys, tid);
    float c[VPT];
    {
        int32_t count[VPT];
        const double mine = lanes_sum<64>(load_counts<Row>(p.counts + int64_t(r.sequence) * p.keys, p.keys, tid, count));
        if (lane == 0) sums[wave] = mine;
        __syncthreads();
        double sum = 0;
        for (int w = 0; w < kWaves; ++w) sum += sums[w];
        apart(count, int32_t(sum / p.keys), c);
    }
    const float f = row_factor(p, r.sequence);
    int buffer = 0;
    for (uint32_t t = r.first; t < r.end; ++t) {
        E* out = dlogits + int64_t(t) * p.keys;
        float e[VPT], rest[VPT], scale;
        if (kAhead) {
            next.values(p.keys, tid, e);
            next.load(logits + int64_t(min(t + 1, r.end - 1)) * p.keys, p.keys, tid);
        }
        if (!is_live(p, t)) {  // of the whole workgroup
            if (!p.accumulate) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) e[i] = 0.0f;
                store_row<E, Row, VPT, VEC>(out, p.keys, tid, e, false);
            }
            continue;
        }
        if (!kAhead) {
            next.load(logits + int64_t(t) * p.keys, p.keys, tid);
            next.values(p.keys, tid, e);
        }
        const float largest = reduce<64>(max_of(e, -INFINITY), larger);
        const float o = terms<64>(p.score, largest, e, rest, scale);
        const float mine = reduce<64>(sum_of(e), plus) * scale, its_dot = reduce<64>(dot_of(e, c, 0.0f), plus) * scale;
        if (lane == 0) {
            offset[buffer][wave] = o;
            total[buffer][wave] = mine;
            dot[buffer][wave] = its_dot;
            term[buffer][wave] = largest_term(p.score, largest, o);
        }
        __syncthreads();
        // A lane for each wavefront's part, in every 16 lanes.
        const int w = lane % 16 % kWaves;
        const float at = offset[buffer][w], most = lanes_reduce<16>(at, larger);
        const float part = lane % 16 < kWaves ? exp32(at - most) : 0.0f;
        const float z = lanes_reduce<16>(total[buffer][w] * part, plus);
        float d = lanes_reduce<16>(dot[buffer][w] * part, plus), top = 0;
        const float biggest = lanes_reduce<16>(term[buffer][w] * part, larger);
        const float share = z > 0 ? 1.0f / z : 0.0f, own = scale * exp32(o - most);
        if (biggest * share > kMostShare) {  // of the whole workgroup
            // The count of the key of the largest term (one that has more than kMostShare of the share is
            // alone above half of it), then the sum relative to that.
            const float here = reduce<64>(max_of(e, 0.0f), larger);
            float its = reduce<64>(count_of_largest<Row>(e, c, here, p.keys, tid), larger);
            if (!(here * own * share > 0.5f)) its = -INFINITY;
            if (lane == 0) again[0][wave] = its;
            __syncthreads();
            top = lanes_reduce<16>(again[0][w], larger);
            its = reduce<64>(dot_of(e, c, top), plus) * own;
            if (lane == 0) again[1][wave] = its;
            __syncthreads();
            d = lanes_reduce<16>(lane % 16 < kWaves ? again[1][w] : 0.0f, plus);
        }
        gradients<64>(p.score, rest, c, top, share * own, d * share, f, e);
        store_row<E, Row, VPT, VEC>(out, p.keys, tid, e, p.accumulate);
        buffer ^= 1;
    }
}

// Rows of more than 32768 keys, in parts that are read, with their counts, for each of their uses: a
// lane's 64 keys and counts do not fit its registers (1024 rows of 65536 keys, float32: 467 us with
// both there, 205 in parts; bfloat16 and sigmoid: 625 and 142 us).
template <typename E, int THREADS, int VPT, int PARTS, bool VEC>
__global__ __launch_bounds__(THREADS) void balance_backward_long_kernel(BalanceParams p) {
    using Row = RowKeys<E, THREADS, VPT, VEC>;
    constexpr int kWaves = THREADS / 64, kPart = THREADS * VPT;
    __shared__ float offset[2][kWaves], total[2][kWaves], dot[2][kWaves], term[2][kWaves];
    __shared__ float again[2][kWaves];
    __shared__ double sums[kWaves];
    ieee_mode_off();
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const Piece r = this_piece(p, blockIdx.x);
    const E* logits = static_cast<const E*>(p.logits);
    E* dlogits = static_cast<E*>(p.dlogits);
    RawRow<E, THREADS, VPT, VEC> next;
    const int32_t* counts = p.counts + int64_t(r.sequence) * p.keys;
    int32_t mean = 0;
    float c[VPT];
    auto load_part = [&](int h) {
        int32_t count[VPT];
        const double sum = load_counts<Row>(counts + h * kPart, p.keys - h * kPart, tid, count);
        apart(count, mean, c);
        return sum;
    };
    {
        double mine = 0;
#pragma unroll 1
        for (int h = 0; h < PARTS; ++h) mine += load_part(h);
        mine = lanes_sum<64>(mine);
        if (lane == 0) sums[wave] = mine;
        __syncthreads();
        double sum = 0;
        for (int w = 0; w < kWaves; ++w) sum += sums[w];
        mean = int32_t(sum / p.keys);
    }
    const float f = row_factor(p, r.sequence);
    int buffer = 0;
    for (uint32_t t = r.first; t < r.end; ++t) {
        const E* row = logits + int64_t(t) * p.keys;
        E* out = dlogits + int64_t(t) * p.keys;
        float e[VPT], rest[VPT], o, scale, largest;
        if (!is_live(p, t)) {  // of the whole workgroup
            if (!p.accumulate) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) e[i] = 0.0f;
#pragma unroll 1
                for (int h = 0; h < PARTS; ++h)
                    store_row<E, Row, VPT, VEC>(out + h * kPart, p.keys - h * kPart, tid, e, false);
            }
            continue;
        }
        // A part's terms, relative to an offset of its own, and its counts.
        auto take = [&](int h) {
            next.load(row + h * kPart, p.keys - h * kPart, tid);
            next.values(p.keys - h * kPart, tid, e);
            load_part(h);
            largest = reduce<64>(max_of(e, -INFINITY), larger);
            o = terms<64>(p.score, largest, e, rest, scale);
        };
        float mine = -FLT_MAX, its_total = 0, its_dot = 0, its_term = 0;
#pragma unroll 1
        for (int h = 0; h < PARTS; ++h) {
            take(h);
            const float sum = reduce<64>(sum_of(e), plus) * scale, products = reduce<64>(dot_of(e, c, 0.0f), plus) * scale;
            const float most = max32(mine, o), before = exp32(mine - most), now = exp32(o - most);
            its_total = its_total * before + sum * now;
            its_dot = its_dot * before + products * now;
            its_term = max32(its_term * before, largest_term(p.score, largest, o) * now);
            mine = most;
        }
        if (lane == 0) {
            offset[buffer][wave] = mine;
            total[buffer][wave] = its_total;
            dot[buffer][wave] = its_dot;
            term[buffer][wave] = its_term;
        }
        __syncthreads();
        // A lane for each wavefront's part, in every 16 lanes.
        const int w = lane % 16 % kWaves;
        const float at = offset[buffer][w], most = lanes_reduce<16>(at, larger);
        const float part = lane % 16 < kWaves ? exp32(at - most) : 0.0f;
        const float z = lanes_reduce<16>(total[buffer][w] * part, plus);
        float d = lanes_reduce<16>(dot[buffer][w] * part, plus), top = 0;
        const float biggest = lanes_reduce<16>(term[buffer][w] * part, larger);
        const float share = z > 0 ? 1.0f / z : 0.0f;
        if (biggest * share > kMostShare) {  // of the whole workgroup
            // The count of the key of the largest term (one that has more than kMostShare of the share is
            // alone above half of it), then the sum relative to that.
            float its = -INFINITY;
#pragma unroll 1
            for (int h = 0; h < PARTS; ++h) {
                take(h);
                const float own = scale * exp32(o - most), here = reduce<64>(max_of(e, 0.0f), larger);
                if (here * own * share > 0.5f)
                    its = max32(its, reduce<64>(count_of_largest<Row>(e, c, here, p.keys - h * kPart, tid), larger));
            }
            if (lane == 0) again[0][wave] = its;
            __syncthreads();
            top = lanes_reduce<16>(again[0][w], larger);
            its = 0;
#pragma unroll 1
            for (int h = 0; h < PARTS; ++h) {
                take(h);
                its += reduce<64>(dot_of(e, c, top), plus) * scale * exp32(o - most);
            }
            if (lane == 0) again[1][wave] = its;
            __syncthreads();
            d = lanes_reduce<16>(lane % 16 < kWaves ? again[1][w] : 0.0f, plus);
        }
#pragma unroll 1
        for (int h = 0; h < PARTS; ++h) {
            take(h);
            gradients<64>(p.score, rest, c, top, share * scale * exp32(o - most), d * share, f, e);
            store_row<E, Row, VPT, VEC>(out + h * kPart, p.keys - h * kPart, tid, e, p.accumulate);
        }
        buffer ^= 1;
    }
}

// ------------------------------------------------------------------ launches

// Pieces wanted of a call with many tokens. More leave the second pass more to add, fewer leave compute
// units idle. Up to 1024 keys 512: the gradient of 32768 x 256 in 14.4 us, with 256 in 16.9, with 1024 in
// 15.8; of 32768 x 1024 in 47.1, 45.8 and 53.8, its first pass 36.4, 32.2 and 40.6. Beyond 256: 4096 x
// 16384 in 50.1 us, with 128 in 67.5, with 512 in 58.7; 1024 x 65536 float32 in 234, 278 and 293; only
// 8192 x 4096 would take 512 (52.2, 87.0 and 46.8).
constexpr int64_t kPieces = 512, kBigPieces = 256;

template <typename E, int LANES, int VPT> void run_small(const BalanceParams& p, bool vec, bool backward, hipStream_t s) {
    const dim3 grid{unsigned(p.sequences * p.pieces)}, block{kSmallThreads};
    if (vec && backward) hipLaunchKernelGGL((balance_backward_small_kernel<E, LANES, VPT, true>), grid, block, 0, s, p);
    else if (backward) hipLaunchKernelGGL((balance_backward_small_kernel<E, LANES, VPT, false>), grid, block, 0, s, p);
    else if (vec) hipLaunchKernelGGL((balance_small_kernel<E, LANES, VPT, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((balance_small_kernel<E, LANES, VPT, false>), grid, block, 0, s, p);
}
template <typename E, int VPT, int PARTS> void run_big(const BalanceParams& p, bool vec, bool backward, hipStream_t s) {
    const dim3 grid{unsigned(p.sequences * p.pieces)}, block{1024};
    if (backward) {
        if constexpr (PARTS == 1) {
            if (vec) hipLaunchKernelGGL((balance_backward_big_kernel<E, 1024, VPT, true>), grid, block, 0, s, p);
            else hipLaunchKernelGGL((balance_backward_big_kernel<E, 1024, VPT, false>), grid, block, 0, s, p);
        } else {
            // Vectors of bfloat16 spill (65536 keys, sigmoid: 285 us; key by key 142); of float32 they pay
            // (205 us; key by key 312).
            constexpr bool kVec = sizeof(E) == 4;
            if (kVec && vec) hipLaunchKernelGGL((balance_backward_long_kernel<E, 1024, VPT, PARTS, kVec>), grid, block, 0, s, p);
            else hipLaunchKernelGGL((balance_backward_long_kernel<E, 1024, VPT, PARTS, false>), grid, block, 0, s, p);
        }
    } else if (vec) {
        hipLaunchKernelGGL((balance_big_kernel<E, 1024, VPT, PARTS, true>), grid, block, 0, s, p);
    } else {
        hipLaunchKernelGGL((balance_big_kernel<E, 1024, VPT, PARTS, false>), grid, block, 0, s, p);
    }
}
template <typename E> void run_rows(const BalanceParams& p, bool backward, hipStream_t s) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.logits) | (backward ? reinterpret_cast<uintptr_t>(p.dlogits) : 0);
    const bool vec = at % 16 == 0 && p.keys * sizeof(E) % 16 == 0;
    if (p.keys <= 128) run_small<E, 16, 8>(p, vec, backward, s);
    else if (p.keys <= 256) run_small<E, 32, 8>(p, vec, backward, s);
    else if (p.keys <= 512) run_small<E, 64, 8>(p, vec, backward, s);
    else if (p.keys <= 1024) run_small<E, 64, 16>(p, vec, backward, s);
    else if (p.keys <= 8192) run_big<E, 8, 1>(p, vec, backward, s);
    else if (p.keys <= 16384) run_big<E, 16, 1>(p, vec, backward, s);
    else if (p.keys <= 32768) run_big<E, 32, 1>(p, vec, backward, s);
    else run_big<E, 16, 4>(p, vec, backward, s);
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
    p->by_chunk = divisor(p->chunk);
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
    if (items > 1024) items = 1024;  // workgroups: each adds to one counter, some 20 ns after the other
    // Many short sequences have few pieces each.
    if (p.pieces <= 16) hipLaunchKernelGGL(balance_join_kernel<256>, dim3(unsigned(items)), dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(balance_join_kernel<1024>, dim3(unsigned(items)), dim3(1024), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceParams& p, bool bf16, hipStream_t stream) {
    if (bf16) run_rows<uint16_t>(p, true, stream);
    else run_rows<float>(p, true, stream);
    return hipGetLastError();
}

}  // namespace sdm
