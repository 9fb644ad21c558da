// Device code that the slot router's kernels share.
#pragma once

#include <float.h>
#include <math.h>

#include "../../include/sdm_memory.h"
#include "sdm_kernels.h"
#include "sdm_memory.h"

namespace sdm {

// Largest and smallest as single instructions: the compiler adds moves that quieten
// NaN operands first, and there are none here.
__device__ __forceinline__ float max32(float a, float b) {
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ float max32(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float median32(float a, float b, float c) {
    float r;
    asm("v_med3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
template <int N> __device__ __forceinline__ float max_of(const float (&x)[N], float v) {
    if constexpr (N % 2 == 1) v = max32(v, x[N - 1]);
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) v = max32(v, x[i], x[i + 1]);
    return v;
}
// A logit as the definition reads it: NaN counts as -inf, +inf as the largest float32.
// A median of three with a NaN among them is the least of the other two, of a
// signalling NaN too while the wavefront's IEEE mode is off.
__device__ __forceinline__ float clean(float x) { return median32(x, -INFINITY, FLT_MAX); }
__device__ __forceinline__ void ieee_mode_off() { __builtin_amdgcn_s_setreg(1 | 9 << 6 | 0 << 11, 0); }  // MODE, bit 9
// Bits of a ballot by 32-bit shifts: gfx950 has given wrong results, other ones on each
// run, for a 64-bit shift whose amount the compiler had put into the last vector register
// that the kernel allocates (v79 of 80).
__device__ __forceinline__ uint32_t half_of(uint64_t bits, int i) { return i & 32 ? uint32_t(bits >> 32) : uint32_t(bits); }
__device__ __forceinline__ bool bit_of(uint64_t bits, int i) { return half_of(bits, i) >> (i & 31) & 1; }
// Those of the LANES lanes that lane `tid` belongs to.
template <int LANES> __device__ __forceinline__ uint64_t row_bits(uint64_t bits, int tid) {
    if constexpr (LANES == 64) return bits;
    if constexpr (LANES == 32) return half_of(bits, tid);
    return half_of(bits, tid) >> (tid & 16) & 0xffff;
}
template <typename E> __device__ __forceinline__ float logit_at(const E* row, int64_t i) { return clean(widen(row[i])); }

__device__ __forceinline__ bool bias_excludes(float b) { return !(b > -INFINITY); }

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }
// Within (4 + 2 |x|) 2^-24 of its value: the hardware's base-2 exponential, of a product that is
// rounded, with a rounded constant.
__device__ __forceinline__ float exp32(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
// Sum of exp(x[i] - v), v the largest x of the row's lanes or -FLT_MAX.
template <int N> __device__ __forceinline__ float exp_sum(const float (&x)[N], float v) {
    constexpr float kL = 1.44269504f;
    float sum = 0;
    if (__ballot(!(fabsf(v) < 65536.0f)) == 0) {  // a branch of the wavefront
        // 2^(x L - c) with c = v L rounded: one operation less a term, and what c's rounding
        // puts into every term, 2^(v L - c) (at most 2^(2^-8) for such v), is taken out of
        // the sum.
        const float c = v * kL;
#pragma unroll
        for (int i = 0; i < N; ++i) sum += __builtin_amdgcn_exp2f(fmaf(x[i], kL, -c));
        return sum * __builtin_amdgcn_exp2f(-fmaf(v, kL, -c));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) sum += exp32(x[i] - v);
    return sum;
}
__device__ __forceinline__ float sigmoid32(float x) { return __builtin_amdgcn_rcpf(1.0f + exp32(-x)); }

// float32 as an unsigned integer of the same order (-0 as +0), and back.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float(u ^ (~uint32_t(int32_t(u) >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t ordered64(double x) {
    const uint64_t u = uint64_t(__double_as_longlong(x + 0.0));
    return u ^ (uint64_t(int64_t(u) >> 63) | 1ull << 63);
}
__device__ __forceinline__ double from_ordered64(uint64_t u) {
    return __longlong_as_double(int64_t(u ^ (~uint64_t(int64_t(u) >> 63) | 1ull << 63)));
}
constexpr uint64_t kOut64 = 0x000fffffffffffffull;  // ordered64(-inf)
constexpr uint32_t kOut = 0x007fffffu;  // ordered(-inf): a key that is not eligible
constexpr uint32_t kAbsent = 0;         // a key that cannot be chosen at all

__device__ __forceinline__ void store_choice(const RouteParams& p, int64_t t, int j, int key, double u) {
    const int64_t o = t * p.k + j, slot = int64_t(uint32_t(t) % p.streams) * p.stream_slots + key;
    if (p.idx64) static_cast<int64_t*>(p.idx)[o] = slot;
    else static_cast<int32_t*>(p.idx)[o] = int32_t(slot);
    const float w = float(p.scale * u);
    if (p.w_bf16) static_cast<uint16_t*>(p.w)[o] = to_bf16_rne(w);
    else static_cast<float*>(p.w)[o] = w;
}

// ------------------------------------------------------------------ any row, exactly

// A key's rank among the keys of its row: the larger value first, then the lower key.
struct Ranked {
    double c;
    int key;
};
__device__ __forceinline__ bool before(const Ranked& a, const Ranked& b) {
    return a.c > b.c || (a.c == b.c && a.key < b.key);
}

// Whether the order of two values v and w, scores that are `apart` plus a bias each, may be another
// one with a softmax's sum in float64 than with one that is off by half of `off` of itself: that
// moves the values by so much of `apart` against each other. Four roundings to float64, two
// values' with either sum, make equal or unequal what is nearer yet.
__device__ __forceinline__ bool near(double v, double w, double apart, double off) {
    return w > -INFINITY && apart > 0 && fabs(v - w) <= off * apart + 0x1p-50 * fmin(fabs(v), fabs(w));
}

template <int THREADS, typename T, typename F> __device__ __forceinline__ T block_reduce(T v, T* lds, F f) {
    __syncthreads();
    lds[threadIdx.x] = v;
    __syncthreads();
    for (int n = THREADS / 2; n > 0; n /= 2) {
        if (int(threadIdx.x) < n) lds[threadIdx.x] = f(lds[threadIdx.x], lds[threadIdx.x + n]);
        __syncthreads();
    }
    return lds[0];
}

template <int THREADS> struct ExactLds {
    union {
        Ranked ranked[THREADS];
        double value[THREADS];
    };
    double worth[SDM_MAX_GROUPS];
    unsigned long long most[SDM_MAX_GROUPS], next[SDM_MAX_GROUPS];
    uint8_t kept[SDM_MAX_GROUPS];
    int chosen[SDM_MAX_WIDTH];
};

// One row by one workgroup, every value in float64: k rounds of a reduction over
// the keys that come after the last one chosen. The kernels below use it for the
// rows whose order float32 cannot tell.
template <typename E, int THREADS>
__device__ __forceinline__ void exact_row(const RouteParams& p, int64_t t, ExactLds<THREADS>& lds) {
    const int tid = threadIdx.x;
    const E* row = static_cast<const E*>(p.logits) + t * p.keys;
    const auto larger = [](double a, double b) { return fmax(a, b); };
    const auto plus = [](double a, double b) { return a + b; };

    double m = 0, z = 1;
    if (p.score == SDM_SOFTMAX) {
        double v = -INFINITY;
        for (int i = tid; i < p.keys; i += THREADS) v = fmax(v, double(logit_at(row, i)));
        m = fmax(block_reduce<THREADS>(v, lds.value, larger), -double(FLT_MAX));
        v = 0;
        for (int i = tid; i < p.keys; i += THREADS) v += exp(double(logit_at(row, i)) - m);
        z = block_reduce<THREADS>(v, lds.value, plus);
    }
    auto eligible = [&](int i) {
        return logit_at(row, i) > -INFINITY && !(p.bias != nullptr && bias_excludes(p.bias[i]));
    };
    auto score = [&](int i) {
        const double x = logit_at(row, i);
        return p.score == SDM_SOFTMAX ? (z > 0 ? exp(x - m) / z : 0.0) : sigmoid64(x);
    };
    const int size = p.keys / p.groups;
    if (p.groups > 1) {
        for (int g = tid; g < p.groups; g += THREADS) lds.most[g] = lds.next[g] = 0;
        __syncthreads();
        for (int i = tid; i < p.keys; i += THREADS) {  // the two largest of each group
            if (!eligible(i)) continue;
            const unsigned long long c = ordered64(score(i) + (p.bias != nullptr ? double(p.bias[i]) : 0.0));
            const unsigned long long less = min(c, atomicMax(&lds.most[i / size], c));
            if (less > kOut64) atomicMax(&lds.next[i / size], less);
        }
        __syncthreads();
        for (int g = tid; g < p.groups; g += THREADS) {
            double v = lds.most[g] > kOut64 ? from_ordered64(lds.most[g]) : -INFINITY;
            if (p.top == 2 && lds.next[g] > kOut64) v += from_ordered64(lds.next[g]);
            lds.worth[g] = v;
        }
        __syncthreads();
        for (int g = tid; g < p.groups; g += THREADS) {
            int rank = 0;
            for (int h = 0; h < p.groups; ++h)
                rank += lds.worth[h] > lds.worth[g] || (lds.worth[h] == lds.worth[g] && h < g);
            lds.kept[g] = rank < p.kept;
        }
        __syncthreads();
    }
    Ranked last = {INFINITY, -1};
    for (int j = 0; j < p.k; ++j) {
        Ranked best = {-INFINITY, 0x7fffffff};
        for (int i = tid; i < p.keys; i += THREADS) {
            if (p.groups > 1 && !lds.kept[i / size]) continue;
            Ranked r = {-INFINITY, i};
            if (eligible(i)) r.c = p.bias != nullptr ? score(i) + double(p.bias[i]) : double(logit_at(row, i));
            if (before(last, r) && before(r, best)) best = r;
        }
        last = block_reduce<THREADS>(best, lds.ranked, [](Ranked a, Ranked b) { return before(b, a) ? b : a; });
        if (tid == 0) lds.chosen[j] = last.key;
    }
    __syncthreads();
    double top = -INFINITY, total = 0;
    const bool relative = p.normalise && p.score == SDM_SOFTMAX;
    if (relative) {
        for (int j = tid; j < p.k; j += THREADS)
            if (eligible(lds.chosen[j])) top = fmax(top, double(logit_at(row, lds.chosen[j])));
        top = fmax(block_reduce<THREADS>(top, lds.value, larger), -double(FLT_MAX));
    }
    auto part = [&](int key) {
        if (!eligible(key)) return 0.0;
        return relative ? exp(double(logit_at(row, key)) - top) : score(key);
    };
    if (p.normalise) {
        for (int j = tid; j < p.k; j += THREADS) total += part(lds.chosen[j]);
        total = block_reduce<THREADS>(total, lds.value, plus);
    }
    for (int j = tid; j < p.k; j += THREADS) {
        const double u = part(lds.chosen[j]);
        store_choice(p, t, j, lds.chosen[j], !p.normalise ? u : total > 0 ? u / total : 0.0);
    }
    __syncthreads();
}

// ------------------------------------------------------------------ lanes

// Lane i's value of the lane that `ctrl` names within its row of 16 lanes.
template <int ctrl> __device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), ctrl, 0xf, 0xf, true));
}
template <int ctrl> __device__ __forceinline__ float dpp(float v) { return __uint_as_float(dpp<ctrl>(__float_as_uint(v))); }
constexpr int kXor1 = 0xb1, kXor2 = 0x4e;            // quad_perm [1,0,3,2] and [2,3,0,1]
constexpr int kHalfMirror = 0x141, kMirror = 0x140;  // lane i of 8, of 16 <- lane 7 - i, 15 - i

// f over the LANES (16, 32 or 64) neighbouring lanes of a row, of 32-bit values.
template <int LANES, typename T, typename F> __device__ __forceinline__ T lanes_reduce(T v, F f) {
    auto with = [&](uint32_t other) {
        T o;
        __builtin_memcpy(&o, &other, 4);
        v = f(v, o);
    };
    auto bits = [&] {
        uint32_t u;
        __builtin_memcpy(&u, &v, 4);
        return u;
    };
    with(dpp<kXor1>(bits()));
    with(dpp<kXor2>(bits()));
    with(dpp<kHalfMirror>(bits()));
    with(dpp<kMirror>(bits()));
    if constexpr (LANES >= 32) with(uint32_t(__shfl_xor(int(bits()), 16)));
    if constexpr (LANES >= 64) with(uint32_t(__shfl_xor(int(bits()), 32)));
    return v;
}

// ------------------------------------------------------------------ a row in a workgroup's registers

// VPT keys a lane of a workgroup of THREADS: vectors of 16 bytes, the lanes' side by
// side (VEC), or one by one.
template <typename E, int THREADS, int VPT, bool VEC> struct RowKeys {
    static constexpr int kN = VEC ? 16 / int(sizeof(E)) : 1;
    static __device__ __forceinline__ int key_of(int i, int tid) { return ((i / kN) * THREADS + tid) * kN + i % kN; }

    // Clean logits; -inf past the row's end.
    static __device__ __forceinline__ void load(const E* row, int keys, int tid, float (&c)[VPT]) {
        constexpr uint32_t kMinusInf = sizeof(E) == 2 ? 0xff80ff80u : 0xff800000u;
        if constexpr (VEC) {
            uint4 raw[VPT / kN];
#pragma unroll
            for (int i = 0; i < VPT / kN; ++i)
                raw[i] = *reinterpret_cast<const uint4*>(row + min(key_of(i * kN, tid), keys - kN));
#pragma unroll
            for (int i = 0; i < VPT / kN; ++i) {
                const uint32_t in = uint32_t((key_of(i * kN, tid) - keys) >> 31);  // all ones where the row has the vector
                uint4 v = raw[i];
                v.x = (v.x & in) | (kMinusInf & ~in), v.y = (v.y & in) | (kMinusInf & ~in);
                v.z = (v.z & in) | (kMinusInf & ~in), v.w = (v.w & in) | (kMinusInf & ~in);
                opaque(v);  // four words chosen, not each key
                E e[kN];
                __builtin_memcpy(e, &v, 16);
#pragma unroll
                for (int j = 0; j < kN; ++j) c[i * kN + j] = widen(e[j]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i) c[i] = widen(row[min(key_of(i, tid), keys - 1)]);
#pragma unroll
            for (int i = 0; i < VPT; ++i) c[i] = key_of(i, tid) < keys ? c[i] : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) c[i] = clean(c[i]);
    }
};

}  // namespace sdm
