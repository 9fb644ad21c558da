// sdm_route (include/sdm_memory.h): the k best keys of each token and their weights.

#include "sdm_route_device.h"

namespace sdm {

namespace {

// ------------------------------------------------------------------ few keys: several rows of a wavefront

constexpr int kSpare = 4;  // candidates beyond k

// A bound on how far a float32 score + bias near c may be from its value, at least
// twice what its roundings come to: a sigmoid's 2^-22 (exponential, sum and
// reciprocal), a softmax's 2^-18 (its sum of at most 1024 terms, in lanes of 16
// and 6 levels, above all), and the rounding of the sum.
__device__ __forceinline__ float value_slack(bool softmax, float c) {
    return (softmax ? 0x1p-17f : 0x1p-21f) + 0x1p-23f * fabsf(c);
}
// And relatively, of a score's own, x from where its exponent is 0.
__device__ __forceinline__ float score_slack(float x) { return (4.0f + fabsf(x)) * 0x1p-22f; }

// One row by one wavefront, KEYS / 64 keys a lane, every value in float64 and in LDS:
// it runs for few rows, and its registers would cost all of them occupancy.
template <int KEYS> struct ExactSmallLds {
    double value[KEYS];  // score + bias, or the score
    float x[KEYS];       // -inf where the key is not eligible
};
template <typename E, int KEYS>
__device__ __forceinline__ void exact_small_row(const RouteParams& p, int64_t t, ExactSmallLds<KEYS>& lds) {
    constexpr int N = KEYS / 64;
    const int lane = threadIdx.x, size = p.keys / p.groups;
    const E* row = static_cast<const E*>(p.logits) + t * p.keys;
    const bool biased = p.bias != nullptr, softmax = p.score == SDM_SOFTMAX;
    auto all = [](double v, auto f) {
#pragma unroll 1
        for (int n = 1; n < 64; n *= 2) v = f(v, __shfl_xor(v, n));
        return v;
    };
    const auto larger = [](double a, double b) { return fmax(a, b); };
    const auto plus = [](double a, double b) { return a + b; };
    // A lane reads and writes its own keys alone.
    auto x = [&](int i) -> float& { return lds.x[i * 64 + lane]; };
    auto v = [&](int i) -> double& { return lds.value[i * 64 + lane]; };
    uint32_t gone = 0;  // bit i: key i of the lane cannot be chosen (any more)
    double m = -FLT_MAX, z = 0;
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
        const int n = i * 64 + lane;
        x(i) = n < p.keys ? logit_at(row, n) : -INFINITY;
        if (n >= p.keys) gone |= 1u << i;
        m = fmax(m, double(x(i)));
    }
    m = all(m, larger);
    auto raw_score = [&](float a) { return softmax ? exp(double(a) - m) : sigmoid64(a); };
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
        v(i) = raw_score(x(i));
        z += v(i);
    }
    z = softmax ? all(z, plus) : 1.0;
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
        const float b = biased ? p.bias[min(i * 64 + lane, p.keys - 1)] : 0.0f;
        if (bias_excludes(b)) x(i) = -INFINITY;
        v(i) = x(i) > -INFINITY ? v(i) / z + double(b) : -INFINITY;
    }
    if (p.groups > 1) {
        double mine = 0;
#pragma unroll 1
        for (int g = 0; g < p.groups; ++g) {
            double hi = -INFINITY, lo = -INFINITY;
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
                const int n = i * 64 + lane;
                if (n / size == g && n < p.keys) {
                    lo = fmax(lo, fmin(hi, v(i)));
                    hi = fmax(hi, v(i));
                }
            }
#pragma unroll 1
            for (int n = 1; n < 64; n *= 2) {
                const double h = __shfl_xor(hi, n), w = __shfl_xor(lo, n);
                lo = fmax(fmax(lo, w), fmin(hi, h));
                hi = fmax(hi, h);
            }
            if (lane == g) mine = p.top == 2 && lo > -INFINITY ? hi + lo : hi;
        }
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const double other = __shfl(mine, g);
            rank += other > mine || (other == mine && g < lane);
        }
        const uint64_t kept = __ballot(lane < p.groups && rank < p.kept);
#pragma unroll 1
        for (int i = 0; i < N; ++i)
            if (i * 64 + lane < p.keys && !bit_of(kept, (i * 64 + lane) / size)) gone |= 1u << i;
    }
    int key = 0;
    float xk = -INFINITY;  // of the lane's choice: lane j has the j-th
#pragma unroll 1
    for (int j = 0; j < p.k; ++j) {
        Ranked best = {-INFINITY, 0x7fffffff};
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
            const Ranked r = {biased ? v(i) : double(x(i)), i * 64 + lane};
            if (!(gone >> i & 1) && before(r, best)) best = r;
        }
#pragma unroll 1
        for (int n = 1; n < 64; n *= 2) {
            const Ranked o = {__shfl_xor(best.c, n), __shfl_xor(best.key, n)};
            if (before(o, best)) best = o;
        }
        float xb = 0;
#pragma unroll 1
        for (int i = 0; i < N; ++i)
            if (best.key == i * 64 + lane) {
                gone |= 1u << i;
                xb = x(i);
            }
        xb = __shfl(xb, best.key % 64);
        if (lane == j) {
            key = best.key;
            xk = xb;
        }
    }
    double sk = xk > -INFINITY ? raw_score(xk) / z : 0.0;
    if (p.normalise) {
        if (softmax) {
            const double top = all(fmax(double(xk), -double(FLT_MAX)), larger);
            sk = xk > -INFINITY ? exp(double(xk) - top) : 0.0;
        }
        const double total = all(sk, plus);
        sk = total > 0 ? sk / total : 0.0;
    }
    if (lane < p.k) store_choice(p, t, lane, key, sk);
}

template <int KEYS> struct SmallLds {
    union {
        struct {
            double value[64], score[64];
            int key[64];
            float worth[64], slack[64];
            uint32_t group_max[64], group_next[64];
        };
        ExactSmallLds<KEYS> exact;
    };
};

// One wavefront a workgroup, 64 / LANES rows of it, VPT consecutive keys a lane.
// The keys are put in order by an integer that holds the value's leading bits and
// the key below them, so that one maximum gives both and a round of the selection
// is a subtraction and a maximum for each key held. kSpare candidates more than k
// are taken that way, and put in exact order by their float64 values. Where the
// leading bits cannot show that the candidates hold the k best, or the order of groups
// that are not whole lanes is in doubt, the row is done again by exact_small_row.
//
// What bounds it, at 32768 rows of 256 float32 keys, 8 chosen of 4 of 8 groups with a
// bias (26 us; the logits and the choice alone take 6 at a copy's rate): 1410 VALU
// instructions for four rows, a third of them the twelve rounds, 19 us of issue.
template <typename E, int VPT, int LANES, bool VEC>
__global__ __launch_bounds__(64, 6) void route_small_kernel(RouteParams p) {
    constexpr int kRows = 64 / LANES;
    constexpr int kKeys = VPT * LANES;
    __shared__ SmallLds<kKeys> lds;
    constexpr int kBits = kKeys <= 64 ? 6 : kKeys <= 128 ? 7 : kKeys <= 256 ? 8 : kKeys <= 512 ? 9 : 10;
    constexpr uint32_t kMask = (1u << kBits) - 1;
    ieee_mode_off();
    const int tid = threadIdx.x, l = tid % LANES, first = tid - l;
    const bool biased = p.bias != nullptr, softmax = p.score == SDM_SOFTMAX;
    const int size = p.keys / p.groups;
    const int available = p.kept * size;
    const bool exact_keys = !biased && sizeof(E) == 2;  // the leading bits are all there are
    const int rounds = min(p.k + (exact_keys ? 0 : kSpare), available);
    const int64_t t0 = int64_t(blockIdx.x) * kRows;
    const int64_t t = t0 + tid / LANES;
    const bool row_there = t < p.tokens;
    const E* row = static_cast<const E*>(p.logits) + (row_there ? t : t0) * p.keys;
    // Keys past the row's end repeat its last ones here and are left out below.
    float x[VPT], b[VPT];
    if constexpr (VEC) {
        constexpr int kN = 16 / int(sizeof(E));
        uint4 raw[VPT / kN];
#pragma unroll
        for (int i = 0; i < VPT / kN; ++i)
            raw[i] = *reinterpret_cast<const uint4*>(row + min(l * VPT + i * kN, p.keys - kN));
#pragma unroll
        for (int i = 0; i < VPT / kN; ++i) {
            E e[kN];
            __builtin_memcpy(e, &raw[i], 16);
#pragma unroll
            for (int j = 0; j < kN; ++j) x[i * kN + j] = widen(e[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) x[i] = widen(row[min(l * VPT + i, p.keys - 1)]);
    }
    if (biased) {
        if (VEC && reinterpret_cast<uintptr_t>(p.bias) % 16 == 0) {
#pragma unroll
            for (int i = 0; i < VPT / 4; ++i) {
                const float4 v = *reinterpret_cast<const float4*>(p.bias + min(l * VPT + i * 4, p.keys - 4));
                b[4 * i] = v.x, b[4 * i + 1] = v.y, b[4 * i + 2] = v.z, b[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i) b[i] = p.bias[min(l * VPT + i, p.keys - 1)];
        }
    }
    const int held = p.keys - l * VPT;  // of this lane's keys, those that there are
#pragma unroll
    for (int i = 0; i < VPT; ++i) x[i] = i < held ? clean(x[i]) : -INFINITY;
    float m = 0, z = 1;
    if (softmax && (biased || !p.normalise)) {
        m = lanes_reduce<LANES>(max_of(x, -FLT_MAX), [](float a, float c) { return max32(a, c); });
        z = lanes_reduce<LANES>(exp_sum(x, m), [](float a, float c) { return a + c; });
    }
    // What the keys are chosen by: the value, or what has its order.
    float c[VPT];
    if (biased) {
        const float inv = 1.0f / max32(z, FLT_MIN);
#pragma unroll
        for (int i = 0; i < VPT; ++i) c[i] = (softmax ? exp32(x[i] - m) * inv : sigmoid32(x[i])) + b[i];
#pragma unroll
        for (int i = 0; i < VPT; ++i) c[i] = (x[i] > -INFINITY) & (b[i] > -INFINITY) ? c[i] : -INFINITY;
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) c[i] = x[i];
    }
    bool doubt = false;
    bool mine_kept = true;         // this lane's keys, where a group is whole lanes
    uint64_t kept_groups = ~0ull;  // of the row, where it is not
    // A group of whole lanes, a power of two of them, is put together by those lanes;
    // others in LDS, and lane g of the row has group g.
    const bool whole = size % VPT == 0 && (size / VPT & (size / VPT - 1)) == 0;
    const float per_size = 1.0f / float(size);
    auto group_of = [&](int n) { return int((float(n) + 0.5f) * per_size); };  // exact: n is far below 2^16
    if (p.groups > 1) {
        const int of_group = whole ? size / VPT : 1;  // lanes of a group
        float hi = -INFINITY, lo = -INFINITY;          // the two largest
        auto add = [&](float v) {
            lo = median32(hi, lo, v);
            hi = max32(hi, v);
        };
        auto merge = [&](float h, float w) {
            add(h);
            lo = max32(lo, w);  // w <= h: above hi only if h was
        };
        if (whole) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) add(c[i]);
            if (of_group > 1) merge(dpp<kXor1>(hi), dpp<kXor1>(lo));
            if (of_group > 2) merge(dpp<kXor2>(hi), dpp<kXor2>(lo));
            if (of_group > 4) merge(dpp<kHalfMirror>(hi), dpp<kHalfMirror>(lo));
            if (of_group > 8) merge(dpp<kMirror>(hi), dpp<kMirror>(lo));
            if (of_group > 16) merge(__shfl_xor(hi, 16), __shfl_xor(lo, 16));
        } else {
            lds.group_max[tid] = lds.group_next[tid] = 0;
            __syncthreads();
            int at = group_of(l * VPT);
            // Every value but the largest is at some time the smaller of a maximum and what
            // it replaced, so the second largest gets there too.
            auto put_down = [&] {
                if (hi > -INFINITY) {
                    const uint32_t h = ordered(hi);
                    const uint32_t w = max(ordered(lo), min(h, atomicMax(&lds.group_max[first + at], h)));
                    if (w > kOut) atomicMax(&lds.group_next[first + at], w);
                }
                hi = lo = -INFINITY;
            };
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int g = group_of(l * VPT + i);  // past the end only -inf is added, and put down nowhere
                if (g != at) {
                    put_down();
                    at = g;
                }
                add(c[i]);
            }
            put_down();
            __syncthreads();
            hi = lds.group_max[tid] > kOut ? from_ordered(lds.group_max[tid]) : -INFINITY;
            lo = lds.group_next[tid] > kOut ? from_ordered(lds.group_next[tid]) : -INFINITY;
        }
        // Groups are compared by their scores, also without a bias: logits whose float64 scores
        // are equal (of a sigmoid, all above 37) are equal here.
        float slack = 0;
        if (biased) {
            slack = value_slack(softmax, hi) + (lo > -INFINITY ? value_slack(softmax, lo) : 0.0f);
            if (!(slack < INFINITY)) slack = 1.0f;  // of an infinite value: equal ones are in doubt
        } else {
            const float top = softmax ? lanes_reduce<LANES>(max32(hi, -FLT_MAX), [](float a, float d) { return max32(a, d); }) : 0.0f;
            slack = hi > -INFINITY ? 2 * score_slack(hi - top) : 0.0f;
            if (lo > -INFINITY) slack = 2 * score_slack(max32(fabsf(hi - top), fabsf(lo - top)));
            hi = hi > -INFINITY ? (softmax ? exp32(hi - top) : sigmoid32(hi)) : hi;
            lo = lo > -INFINITY ? (softmax ? exp32(lo - top) : sigmoid32(lo)) : lo;
            slack = slack * (max32(hi, 0.0f) + max32(lo, 0.0f)) + 0x1p-120f;  // and below that, of nothing
        }
        // Two of the lowest values add up to -inf in float32, which is a group's without a key;
        // at the lowest finite one its slack keeps them apart and in doubt.
        const float worth = p.top == 2 && lo > -INFINITY ? max32(hi + lo, -FLT_MAX) : hi;
        const int g = l / of_group;
        __syncthreads();
        if (l % of_group == 0 && g < p.groups) {
            lds.worth[first + g] = worth;
            lds.slack[first + g] = slack;
        }
        __syncthreads();
        int above = 0, not_below = 0;  // groups that surely, that perhaps go before this one
        for (int h = 0; h < p.groups; ++h) {
            const float other = lds.worth[first + h], far = slack + lds.slack[first + h];
            const bool exact = !(max32(other, worth) > -INFINITY);
            const bool ahead = (other > worth) | ((other == worth) & (h < g));
            above += (h != g) & (exact ? ahead : other > worth + far);
            not_below += (h != g) & (exact ? ahead : !(other < worth - far));
        }
        mine_kept = not_below < p.kept;
        const bool unsure = g < p.groups && not_below >= p.kept && above < p.kept;
        if (!whole) {
            kept_groups = row_bits<LANES>(__ballot(g < p.groups && not_below < p.kept), tid);
            mine_kept = true;
            doubt = unsure;
        } else if (__ballot(unsure) != 0) {
            // Some group of the wavefront's rows is in doubt (of 32768 rows in 8 groups, 5): the
            // same in float64, a softmax's sum with it.
            double sum = 0, most = -INFINITY, next = -INFINITY;
            const double at = softmax ? lanes_reduce<LANES>(max_of(x, -FLT_MAX), [](float a, float d) { return max32(a, d); }) : 0.0f;
            auto score = [&](float a) { return softmax ? exp(double(a) - at) : sigmoid64(a); };
            if (biased && softmax) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) sum += score(x[i]);
                for (int n = 1; n < LANES; n *= 2) sum += __shfl_xor(sum, n);
            } else {
                sum = 1;
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const double v = c[i] > -INFINITY ? score(x[i]) / sum + (biased ? double(b[i]) : 0.0) : -INFINITY;
                next = fmax(next, fmin(most, v));
                most = fmax(most, v);
            }
            for (int n = 1; n < of_group; n *= 2) {
                const double h = __shfl_xor(most, n), w = __shfl_xor(next, n);
                next = fmax(fmax(next, w), fmin(most, h));
                most = fmax(most, h);
            }
            const double exactly = p.top == 2 && next > -INFINITY ? most + next : most;
            __syncthreads();
            if (l % of_group == 0 && g < p.groups) lds.value[first + g] = exactly;
            __syncthreads();
            int rank = 0;
            for (int h = 0; h < p.groups; ++h) {
                const double other = lds.value[first + h];
                rank += (other > exactly) | ((other == exactly) & (h < g));
            }
            mine_kept = rank < p.kept;
        }
    }
    uint32_t key[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const uint32_t k = (ordered(c[i]) >> 1 & ~kMask) | (kMask - uint32_t(l * VPT + i));
        const bool kept = mine_kept & (whole || bit_of(kept_groups, group_of(l * VPT + i) & 63));
        key[i] = (i < held) & kept ? k : kAbsent;
    }
    uint32_t last = 0x80000000u, mine = 0, at_k = 0;
    for (int r = 0; r < rounds; ++r) {
        uint32_t best = 0;  // of key - last: those after the last one are past 2^31
#pragma unroll
        for (int i = 0; i < VPT; ++i) best = max(best, key[i] - last);
        best = lanes_reduce<LANES>(best, [](uint32_t a, uint32_t d) { return max(a, d); });
        last += best;
        if (l == r) mine = last;
        if (r == p.k - 1) at_k = last;
    }
    // Every key outside the candidates has leading bits of at most `last`'s.
    if (!exact_keys && rounds < available) {
        const uint32_t qk = at_k & ~kMask, ql = last & ~kMask;
        if (ql != (kOut >> 1 & ~kMask)) {  // else: what is eligible is all in, the rest goes by the key
            if (!biased) {
                doubt |= qk == ql;
            } else {
                const float low_k = from_ordered(qk << 1), high_last = from_ordered((ql | kMask) << 1 | 1);
                doubt |= !(low_k - high_last > value_slack(softmax, low_k) + value_slack(softmax, high_last));
            }
        }
    }
    const int n = min(int(kMask - (mine & kMask)), p.keys - 1);
    float xn = -INFINITY, bn = 0;
    if (l < rounds) {
        xn = logit_at(row, n);
        if (biased) bn = p.bias[n];
    }
    const bool ok = xn > -INFINITY && bn > -INFINITY;
    double s = 0;  // the score, where something needs it
    if (biased || !p.normalise || !softmax) {
        if (ok) s = softmax ? exp(double(xn) - double(m)) / double(z) : sigmoid64(xn);
    }
    int rank = l;
    if (!exact_keys) {
        const double v = !ok ? -INFINITY : biased ? s + double(bn) : double(xn);
        __syncthreads();
        lds.value[tid] = v;
        lds.score[tid] = s;
        lds.key[tid] = n;
        __syncthreads();
        rank = 0;
        for (int r = 0; r < rounds; ++r) {
            const double o = lds.value[first + r];
            rank += (o > v) | ((o == v) & (lds.key[first + r] < n));
            // The scores of a softmax are off by 2^-18, its float32 sum, of themselves, all by the same.
            if (softmax && biased && l < rounds && ok) doubt |= near(v, o, fabs(s - lds.score[first + r]), 0x1p-17);
        }
    }
    double u = s;
    const bool chosen = l < rounds && rank < p.k;
    if (p.normalise) {
        if (softmax) {
            float top = chosen && ok ? xn : -FLT_MAX;
            top = lanes_reduce<LANES>(top, [](float a, float d) { return fmaxf(a, d); });
            u = ok ? exp(double(xn) - double(top)) : 0.0;
        }
        __syncthreads();
        lds.value[tid] = chosen ? u : 0.0;
        __syncthreads();
        double total = 0;
        for (int r = 0; r < rounds; ++r) total += lds.value[first + r];
        u = total > 0 ? u / total : 0.0;
    }
    constexpr uint64_t kRow = LANES == 64 ? ~0ull : (1ull << (LANES % 64)) - 1;
    const uint64_t in_doubt = __ballot(doubt && row_there);
    if (chosen && row_there && row_bits<LANES>(in_doubt, tid) == 0) store_choice(p, t, rank, n, u);
    for (int r = 0; r < kRows; ++r)
        if (in_doubt >> (r * LANES) & kRow) {
            __syncthreads();
            exact_small_row<E, kKeys>(p, t0 + r, lds.exact);
        }
}

template <typename E, int VPT, int LANES> void run_small(const RouteParams& p, bool vec, hipStream_t stream) {
    const dim3 grid{unsigned((p.tokens + 64 / LANES - 1) / (64 / LANES))}, block{64};
    if constexpr (VPT * sizeof(E) % 16 == 0) {
        if (vec) {
            hipLaunchKernelGGL((route_small_kernel<E, VPT, LANES, true>), grid, block, 0, stream, p);
            return;
        }
    }
    hipLaunchKernelGGL((route_small_kernel<E, VPT, LANES, false>), grid, block, 0, stream, p);
}

template <typename E, int LANES> void run_small(const RouteParams& p, int vpt, bool vec, hipStream_t stream) {
    if (vpt == 4) run_small<E, 4, LANES>(p, vec, stream);
    else if (vpt == 8) run_small<E, 8, LANES>(p, vec, stream);
    else run_small<E, 16, LANES>(p, vec, stream);
}

constexpr int64_t kFewTokens = 1024;

template <typename E> void run_route(const RouteParams& p, hipStream_t stream) {
    // A lane for each candidate, and 16 keys a lane at most; of few tokens, 4 keys a lane:
    // a wavefront alone is as fast as its lanes are short (one token of 256 keys: 7.5 us
    // with 16 lanes of 16 keys, 6.3 with 64 of 4), and the card is not full either way.
    const int most = p.tokens <= kFewTokens ? 4 : 16;
    int lanes = 16;
    while (lanes < 64 && (lanes * most < p.keys || lanes < p.k + kSpare)) lanes *= 2;
    int vpt = 4;
    while (vpt < 16 && lanes * vpt < p.keys) vpt *= 2;
    if (lanes * vpt >= p.keys && lanes >= p.k + kSpare && p.groups <= lanes) {
        const bool vec = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && p.keys * sizeof(E) % 16 == 0;
        if (lanes == 16) run_small<E, 16>(p, vpt, vec, stream);
        else if (lanes == 32) run_small<E, 32>(p, vpt, vec, stream);
        else run_small<E, 64>(p, vpt, vec, stream);
        return;
    }
    launch_route_block(p, sizeof(E) == 2, stream);
}

}  // namespace

hipError_t launch_route(const RouteParams& p, bool bf16, hipStream_t stream) {
    if (bf16) run_route<uint16_t>(p, stream);
    else run_route<float>(p, stream);
    return hipGetLastError();
}

}  // namespace sdm
