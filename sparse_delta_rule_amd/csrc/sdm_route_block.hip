// sdm_route for rows of any size: a workgroup a row (include/sdm_memory.h).

#include "sdm_route_device.h"

namespace sdm {

namespace {

constexpr int kCandidates = 1024;  // held in LDS at most

// A bound on how far a float32 score + bias near c may be from its value, at least
// twice what its roundings come to (a softmax's sum: 64 terms a lane, 6 levels
// of lanes and 16 wavefronts: 2^-17 of the score).
__device__ __forceinline__ float block_slack(bool softmax, float c) {
    return (softmax ? 0x1p-16f : 0x1p-21f) + 0x1p-23f * fabsf(c);
}

template <int THREADS> struct BlockLds {
    union {
        struct {
            uint32_t lane_max[THREADS];
            uint32_t group_max[SDM_MAX_GROUPS], group_next[SDM_MAX_GROUPS];
            double worth[SDM_MAX_GROUPS];
            float slack[SDM_MAX_GROUPS];
            uint8_t kept[SDM_MAX_GROUPS];
        } first;
        struct {
            double value[kCandidates];
            double sorted[SDM_MAX_WIDTH + 1], score[SDM_MAX_WIDTH + 1];
        } second;
        ExactLds<THREADS> exact;
    };
    uint32_t cand_key[kCandidates];
    int cand[kCandidates];
    int chosen[SDM_MAX_WIDTH];
    float wave_max[THREADS / 64], wave_sum[THREADS / 64];
    double wave_value[THREADS / 64];
    uint32_t threshold;
    int found, count[2], doubt;
};

// VPT keys a lane, held as ordered integers of what they are chosen by. The k-th
// largest of the lanes' own maxima (or a number a little below it) is a bound that
// at least k keys reach and, with twice as many lanes as k, about 1.1 to 1.4 k do:
// those are put in LDS, given their exact values and ranked by counting. Where more
// reach it than LDS holds (ties, masked rows, large keys all in a few lanes) the
// exact k-th key is found by bisection over its bits. Rows that stay in doubt with
// a bias (more near-ties than LDS holds, groups or softmax values that float32 cannot
// tell apart) go to exact_row.
template <typename E, int THREADS, int VPT, bool VEC>
__global__ __launch_bounds__(THREADS) void route_block_kernel(RouteParams p) {
    __shared__ BlockLds<THREADS> lds;
    constexpr int kWaves = THREADS / 64;
    constexpr int kN = VEC ? 16 / int(sizeof(E)) : 1;
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const int64_t t = blockIdx.x;
    const E* row = static_cast<const E*>(p.logits) + t * p.keys;
    const bool biased = p.bias != nullptr, softmax = p.score == SDM_SOFTMAX;
    const int size = p.keys / p.groups;
    auto key_of = [&](int i) { return ((i / kN) * THREADS + tid) * kN + i % kN; };

    float x[VPT];
#pragma unroll
    for (int i = 0; i < VPT; i += kN) {
        if constexpr (VEC) {
            const uint4 raw = *reinterpret_cast<const uint4*>(row + min(key_of(i), p.keys - kN));
            E e[kN];
            __builtin_memcpy(e, &raw, 16);
#pragma unroll
            for (int j = 0; j < kN; ++j) x[i + j] = widen(e[j]);
        } else {
            x[i] = widen(row[min(key_of(i), p.keys - 1)]);
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) x[i] = key_of(i) < p.keys ? clean(x[i]) : -INFINITY;
    if (tid == 0) {
        lds.found = 0;
        lds.doubt = 0;
    }
    const bool stats = softmax && (biased || !p.normalise);
    float m = 0, z = 1;
    if (stats) {
        float v = -FLT_MAX, sum = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) v = max32(v, x[i]);
        v = lanes_reduce<64>(v, [](float a, float b) { return max32(a, b); });
#pragma unroll
        for (int i = 0; i < VPT; ++i) sum += exp32(x[i] - v);
        sum = lanes_reduce<64>(sum, [](float a, float b) { return a + b; });
        if (lane == 0) {
            lds.wave_max[wave] = v;
            lds.wave_sum[wave] = sum;
        }
    }
    auto row_stats = [&] {  // after a barrier
        m = -FLT_MAX, z = 0;
        for (int w = 0; w < kWaves; ++w) m = max32(m, lds.wave_max[w]);
        for (int w = 0; w < kWaves; ++w) z += lds.wave_sum[w] * exp32(lds.wave_max[w] - m);
    };
    uint32_t u[VPT];
    if (biased) {
        if (stats) {
            __syncthreads();
            row_stats();
        }
        const float inv = 1.0f / max32(z, FLT_MIN);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const float b = p.bias[min(key_of(i), p.keys - 1)];
            const float c = (softmax ? exp32(x[i] - m) * inv : sigmoid32(x[i])) + b;
            u[i] = (x[i] > -INFINITY) & (b > -INFINITY) ? ordered(c) : kOut;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) u[i] = ordered(x[i]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) u[i] = key_of(i) < p.keys ? u[i] : kAbsent;

    if (p.groups > 1) {
        auto& f = lds.first;
        for (int g = tid; g < p.groups; g += THREADS) f.group_max[g] = f.group_next[g] = 0;
        __syncthreads();
        // The two largest of each group. Every value but the largest is at some time the
        // smaller of a maximum and what it replaced, so the second largest gets there too.
        auto add = [&](int n, uint32_t hi, uint32_t lo) {
            if (hi <= kOut) return;
            const int g = n / size;
            lo = max(lo, min(hi, atomicMax(&f.group_max[g], hi)));
            if (lo > kOut) atomicMax(&f.group_next[g], lo);
        };
        const bool whole = size % kN == 0;  // a vector of keys is of one group
#pragma unroll
        for (int i = 0; i < VPT; i += kN) {
            if (whole) {
                uint32_t hi = 0, lo = 0;
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    lo = max(lo, min(hi, u[i + j]));
                    hi = max(hi, u[i + j]);
                }
                add(key_of(i), hi, lo);
            } else {
#pragma unroll
                for (int j = 0; j < kN; ++j) add(key_of(i + j), u[i + j], 0);
            }
        }
        __syncthreads();
        uint32_t top = 0;
        if (softmax && !biased)
            for (int g = 0; g < p.groups; ++g) top = max(top, f.group_max[g]);
        const double from = top > kOut ? double(from_ordered(top)) : 0.0;
        for (int g = tid; g < p.groups; g += THREADS) {
            const bool any = f.group_max[g] > kOut, two = p.top == 2 && f.group_next[g] > kOut;
            double hi = any ? double(from_ordered(f.group_max[g])) : -INFINITY;
            double lo = two ? double(from_ordered(f.group_next[g])) : 0.0;
            float slack = 0;
            if (biased) {
                slack = block_slack(softmax, float(hi)) + (two ? block_slack(softmax, float(lo)) : 0.0f);
                if (!(slack < INFINITY)) slack = 1.0f;
            } else if (p.top == 2) {  // by the scores, from the two logits, in float64
                if (any) hi = softmax ? exp(hi - from) : sigmoid64(hi);
                if (two) lo = softmax ? exp(lo - from) : sigmoid64(lo);
            }
            f.worth[g] = hi + lo;
            f.slack[g] = slack;
        }
        __syncthreads();
        for (int g = tid; g < p.groups; g += THREADS) {
            const double worth = f.worth[g];
            int above = 0, not_below = 0;  // groups that surely, that perhaps go before this one
            for (int h = 0; h < p.groups; ++h) {
                const double other = f.worth[h];
                const bool exact = !biased | !(fmax(other, worth) > -INFINITY);
                const bool ahead = (other > worth) | ((other == worth) & (h < g));
                const double far = f.slack[g] + f.slack[h];
                above += (h != g) & (exact ? ahead : other > worth + far);
                not_below += (h != g) & (exact ? ahead : !(other < worth - far));
            }
            f.kept[g] = not_below < p.kept;
            if (not_below >= p.kept && above < p.kept) lds.doubt = 1;
        }
        __syncthreads();
        if (lds.doubt) {
            __syncthreads();
            exact_row<E, THREADS>(p, t, lds.exact);
            return;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (key_of(i) < p.keys && !f.kept[key_of(i) / size]) u[i] = kAbsent;
    }

    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) most = max(most, u[i]);
    lds.first.lane_max[tid] = most;
    __syncthreads();
    if (wave == 0) {
        uint32_t v[kWaves], bound = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) v[i] = lds.first.lane_max[i * 64 + lane];
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t trial = bound | 1u << bit;
            int n = 0;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) n += __popcll(__ballot(v[i] >= trial));
            if (n < p.k) continue;
            bound = trial;
            if (n <= p.k + p.k / 8) break;
        }
        if (lane == 0) lds.threshold = bound;
    }
    __syncthreads();
    // With a bias, the keys that may be among the k best are those within twice the
    // slack of a bound that k keys reach.
    auto widened = [&](uint32_t bound) {
        if (!biased || bound <= kOut) return bound;
        const float c = from_ordered(bound);
        return c < INFINITY ? max(ordered(c - 2 * block_slack(softmax, c)), kOut + 1) : bound;
    };
    auto collect = [&](auto takes) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (takes(u[i], key_of(i))) {
                const int at = atomicAdd(&lds.found, 1);
                if (at < kCandidates) {
                    lds.cand_key[at] = u[i];
                    lds.cand[at] = key_of(i);
                }
            }
    };
    const uint32_t low = max(widened(lds.threshold), 1u);
    if (most >= low) collect([&](uint32_t k, int) { return k >= low; });
    __syncthreads();
    if (lds.found > kCandidates) {
        int turn = 0;
        auto count = [&](auto counts) {  // over the row
            int n = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) n += __popcll(__ballot(counts(u[i], key_of(i))));
            if (tid == 0) lds.count[turn] = 0;
            __syncthreads();
            if (lane == 0) atomicAdd(&lds.count[turn], n);
            __syncthreads();
            n = lds.count[turn];
            turn ^= 1;
            return n;
        };
        uint32_t kth = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t trial = kth | 1u << bit;
            if (count([&](uint32_t k, int) { return k >= trial; }) >= p.k) kth = trial;
        }
        if (tid == 0) lds.found = 0;
        if (biased && kth > kOut) {
            const uint32_t least = widened(kth);
            const int n = count([&](uint32_t k, int) { return k >= least; });
            if (n > kCandidates) {
                __syncthreads();
                exact_row<E, THREADS>(p, t, lds.exact);
                return;
            }
            collect([&](uint32_t k, int) { return k >= least; });
        } else {
            const int need = p.k - count([&](uint32_t k, int) { return k > kth; });
            int last = 0;  // the lowest keys among those equal to the k-th, up to this one
            for (int bit = 15; bit >= 0; --bit) {
                const int trial = last | 1 << bit;
                if (count([&](uint32_t k, int n) { return k == kth && n < trial; }) < need) last = trial;
            }
            collect([&](uint32_t k, int n) { return k > kth || (k == kth && n <= last); });
        }
        __syncthreads();
    }
    const int found = lds.found;
    auto& f = lds.second;
    if (biased) {
        for (int i = tid; i < found; i += THREADS) {
            double v = -INFINITY;
            if (lds.cand_key[i] > kOut) {
                const double a = logit_at(row, lds.cand[i]);
                v = (softmax ? exp(a - double(m)) / double(z) : sigmoid64(a)) + double(p.bias[lds.cand[i]]);
            }
            f.value[i] = v;
        }
        __syncthreads();
        for (int i = tid; i < found; i += THREADS) {
            const double v = f.value[i];
            const int n = lds.cand[i];
            int rank = 0;
            for (int j = 0; j < found; ++j) rank += (f.value[j] > v) | ((f.value[j] == v) & (lds.cand[j] < n));
            if (rank < p.k) lds.chosen[rank] = n;
            if (softmax && rank <= p.k) {
                f.sorted[rank] = v;
                f.score[rank] = v > -INFINITY ? exp(double(logit_at(row, n)) - double(m)) / double(z) : 0.0;
            }
        }
        __syncthreads();
        if (softmax) {
            // The scores are off by 2^-17, their float32 sum, of themselves, all by the same.
            if (tid < p.k && tid + 1 < found && f.sorted[tid + 1] > -INFINITY) {
                const double apart = fabs(f.score[tid] - f.score[tid + 1]);
                if (apart > 0 && f.sorted[tid] - f.sorted[tid + 1] <= 0x1p-16 * apart) lds.doubt = 1;
            }
            __syncthreads();
            if (lds.doubt) {
                exact_row<E, THREADS>(p, t, lds.exact);
                return;
            }
        }
    } else {
        for (int i = tid; i < found; i += THREADS) {
            const uint32_t k = lds.cand_key[i];
            const int n = lds.cand[i];
            int rank = 0;
            for (int j = 0; j < found; ++j) rank += (lds.cand_key[j] > k) | ((lds.cand_key[j] == k) & (lds.cand[j] < n));
            if (rank < p.k) lds.chosen[rank] = n;
        }
        __syncthreads();
        if (stats) row_stats();
    }
    const int key = tid < p.k ? lds.chosen[tid] : 0;
    const float xk = tid < p.k ? logit_at(row, key) : -INFINITY;
    const bool ok = xk > -INFINITY && !(biased && bias_excludes(p.bias[key]));
    auto block = [&](double v, auto op) {  // over the lanes, then over the wavefronts in order
        for (int n = 1; n < 64; n *= 2) v = op(v, __shfl_xor(v, n));
        __syncthreads();
        if (lane == 0) lds.wave_value[wave] = v;
        __syncthreads();
        v = lds.wave_value[0];
        for (int w = 1; w < kWaves; ++w) v = op(v, lds.wave_value[w]);
        return v;
    };
    double s = 0;
    if (p.normalise && softmax) {
        const double top = block(ok ? double(xk) : -double(FLT_MAX), [](double a, double b) { return fmax(a, b); });
        if (ok) s = exp(double(xk) - top);
    } else if (ok) {
        s = softmax ? exp(double(xk) - double(m)) / double(z) : sigmoid64(xk);
    }
    if (p.normalise) {
        const double total = block(s, [](double a, double b) { return a + b; });
        s = total > 0 ? s / total : 0.0;
    }
    if (tid < p.k) store_choice(p, t, tid, key, s);
}

template <typename E, int THREADS, int VPT> void run(const RouteParams& p, bool vec, hipStream_t stream) {
    const dim3 grid{unsigned(p.tokens)}, block{THREADS};
    if constexpr (VPT * sizeof(E) % 16 == 0) {
        if (vec) {
            hipLaunchKernelGGL((route_block_kernel<E, THREADS, VPT, true>), grid, block, 0, stream, p);
            return;
        }
    }
    hipLaunchKernelGGL((route_block_kernel<E, THREADS, VPT, false>), grid, block, 0, stream, p);
}

template <typename E> void run_route(const RouteParams& p, hipStream_t stream) {
    const bool vec = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && p.keys * sizeof(E) % 16 == 0;
    if (p.k <= 128 && p.keys <= 4096) {
        if (p.keys <= 1024) run<E, 256, 4>(p, vec, stream);
        else if (p.keys <= 2048) run<E, 256, 8>(p, vec, stream);
        else run<E, 256, 16>(p, vec, stream);
    } else if (p.keys <= 16384) {
        if (p.keys <= 512) run<E, 512, 1>(p, vec, stream);
        else if (p.keys <= 2048) run<E, 512, 4>(p, vec, stream);
        else if (p.keys <= 4096) run<E, 512, 8>(p, vec, stream);
        else if (p.keys <= 8192) run<E, 512, 16>(p, vec, stream);
        else run<E, 512, 32>(p, vec, stream);
    } else if (p.keys <= 32768) {
        run<E, 1024, 32>(p, vec, stream);
    } else {
        run<E, 1024, 64>(p, vec, stream);
    }
}

}  // namespace

void launch_route_block(const RouteParams& p, bool bf16, hipStream_t stream) {
    if (bf16) run_route<uint16_t>(p, stream);
    else run_route<float>(p, stream);
}

}  // namespace sdm
