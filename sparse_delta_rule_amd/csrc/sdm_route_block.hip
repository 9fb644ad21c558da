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

template <int THREADS, bool GENERAL> struct BlockLds {
    static constexpr int kGroups = GENERAL ? SDM_MAX_GROUPS : 1, kChosen = GENERAL ? SDM_MAX_WIDTH : 1;
    union {
        struct {
            uint32_t lane_max[THREADS];
            uint32_t group_max[kGroups], group_next[kGroups];
            double worth[kGroups];
            unsigned long long exact_max[kGroups], exact_next[kGroups];
            float slack[kGroups];
            uint8_t kept[kGroups];
        } first;
        struct {
            uint64_t value[GENERAL ? kCandidates : 1];  // with a bias: float64 values, as ordered integers
            double sorted[kChosen], score[kChosen];
        } second;
        ExactLds<GENERAL ? THREADS : 1> exact;
    };
    alignas(16) uint64_t cand[kCandidates];  // what it is chosen by, as an ordered integer, and its key's complement
    int rank[kCandidates];
    int chosen[SDM_MAX_WIDTH];
    float chosen_value[SDM_MAX_WIDTH];
    float wave_max[THREADS / 64], wave_sum[THREADS / 64];
    double wave_value[THREADS / 64];
    uint32_t threshold;
    int found, count[2], doubt;
};

// VPT keys a lane, held as what they are chosen by. The k-th
// largest of the lanes' own maxima (or a number a little below it) is a bound that
// at least k keys reach and, with twice as many lanes as k, about 1.1 to 1.4 k do:
// those are put in LDS, given their exact values and ranked by counting. Where more
// reach it than LDS holds (ties, masked rows, large keys all in a few lanes) the
// exact k-th key is found by bisection over its bits. With a bias, a row of more near-ties
// at its k-th key than LDS holds goes to exact_row (a softmax's slack does not shrink with its
// scores, so 16384 flat ones, of logits of a spread of 0.2, are near-ties: about 100 times as long).
//
// What bounds it, at 4096 rows of 16384 bfloat16 keys with their softmax (53 us; the
// logits alone take 22 at a copy's rate): 537 VALU instructions for each 64 x 32 keys,
// 31 us of issue, and the phases between the barriers, which three rows of a CU
// cover only in part. 512 rows of 2048 keys, 256 chosen (18 us) are two rows a CU and
// the latency of their phases.
//
// GENERAL: with a bias or groups. Without either nothing is ever in doubt, and the
// kernel needs half the registers.
template <typename E, int THREADS, int VPT, bool VEC, bool GENERAL>
__global__ __launch_bounds__(THREADS, THREADS == 1024 || GENERAL ? 4 : VPT <= 8 ? 8 : 6) void route_block_kernel(RouteParams p) {
    __shared__ BlockLds<THREADS, GENERAL> lds;
    constexpr int kWaves = THREADS / 64;
    constexpr int kN = RowKeys<E, THREADS, VPT, VEC>::kN;
    ieee_mode_off();
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const int64_t t = blockIdx.x;
    const E* row = static_cast<const E*>(p.logits) + t * p.keys;
    const bool biased = GENERAL && p.bias != nullptr, softmax = p.score == SDM_SOFTMAX;
    const int size = GENERAL ? p.keys / p.groups : p.keys;
    using Row = RowKeys<E, THREADS, VPT, VEC>;
    auto key_of = [&](int i) { return Row::key_of(i, tid); };
    float c[VPT];  // the logits, and then what they are chosen by
    Row::load(row, p.keys, tid, c);
    if (tid == 0) {
        lds.found = 0;
        lds.doubt = 0;
    }
    const bool stats = softmax && (biased || !p.normalise);
    float m = 0, z = 1;
    float most = max_of(c, -INFINITY);
    if (stats) {
        const float v = lanes_reduce<64>(max32(most, -FLT_MAX), [](float a, float b) { return max32(a, b); });
        const float sum = lanes_reduce<64>(exp_sum(c, v), [](float a, float b) { return a + b; });
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
    if (biased) {
        if (stats) {
            __syncthreads();
            row_stats();
        }
        const float inv = 1.0f / max32(z, FLT_MIN);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const float b = p.bias[min(key_of(i), p.keys - 1)];
            const float v = (softmax ? exp32(c[i] - m) * inv : sigmoid32(c[i])) + b;
            c[i] = (c[i] > -INFINITY) & (b > -INFINITY) ? v : -INFINITY;
        }
        most = max_of(c, -INFINITY);
    }
    auto block = [&](double v, auto op) {  // over the lanes, then over the wavefronts in order
        for (int n = 1; n < 64; n *= 2) v = op(v, __shfl_xor(v, n));
        __syncthreads();
        if (lane == 0) lds.wave_value[wave] = v;
        __syncthreads();
        v = lds.wave_value[0];
        for (int w = 1; w < kWaves; ++w) v = op(v, lds.wave_value[w]);
        return v;
    };
    auto block_sum = [&](double v) { return block(v, [](double a, double b) { return a + b; }); };
    // A key's group: (n + 1/2) / size is at least 1 / (2 size) from a whole number, and a
    // float32's roundings are less than 2^-7 / size there.
    const float per_size = 1.0f / float(size);
    auto group_of = [&](int n) { return int((float(n) + 0.5f) * per_size); };
    double exact_z = 0;  // a softmax's sum in float64, where float32's leaves something in doubt
    auto exact_sum = [&] {
        double v = 0;
        for (int n = tid; n < p.keys; n += THREADS) v += exp(double(logit_at(row, n)) - double(m));
        exact_z = block_sum(v);
    };
    auto exact_score = [&](float a) { return softmax ? exp(double(a) - double(m)) / exact_z : sigmoid64(a); };
    if (GENERAL && p.groups > 1) {
        auto& f = lds.first;
        for (int g = tid; g < p.groups; g += THREADS) f.group_max[g] = f.group_next[g] = 0;
        __syncthreads();
        // The two largest of each group. Every value but the largest is at some time the
        // smaller of a maximum and what it replaced, so the second largest gets there too.
        auto put = [&](int g, float hi, float lo) {
            if (!(hi > -INFINITY)) return;
            const uint32_t h = ordered(hi);
            const uint32_t l = max(ordered(lo), min(h, atomicMax(&f.group_max[g], h)));
            if (l > kOut) atomicMax(&f.group_next[g], l);
        };
        // A lane's keys ascend, so its groups do: it keeps the two largest of the group it is
        // in, and the wavefront puts them down when some lane comes to another one, once
        // for all its lanes where they are in one group.
        int at = group_of(key_of(0));
        float hi = -INFINITY, lo = -INFINITY;
        auto add = [&](float v) {
            lo = median32(hi, lo, v);
            hi = max32(hi, v);
        };
        auto put_down = [&] {
            if (__ballot(at != __builtin_amdgcn_readfirstlane(at)) == 0) {
                auto merge = [&](float h, float w) {
                    add(h);
                    lo = max32(lo, w);
                };
                merge(dpp<kXor1>(hi), dpp<kXor1>(lo));
                merge(dpp<kXor2>(hi), dpp<kXor2>(lo));
                merge(dpp<kHalfMirror>(hi), dpp<kHalfMirror>(lo));
                merge(dpp<kMirror>(hi), dpp<kMirror>(lo));
                merge(__shfl_xor(hi, 16), __shfl_xor(lo, 16));
                merge(__shfl_xor(hi, 32), __shfl_xor(lo, 32));
                if (lane == 0) put(at, hi, lo);
            } else {
                put(at, hi, lo);
            }
            hi = lo = -INFINITY;
        };
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int g = group_of(min(key_of(i), p.keys - 1));  // past the end: -inf, in no way of the last group's
            if (__ballot(g != at) != 0) {
                put_down();
                at = g;
            }
            add(c[i]);
        }
        put_down();
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
                if (!(slack < INFINITY)) slack = 1.0f;  // of an infinite value: equal ones are in doubt
            } else {  // by the scores, from the logits, in float64
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
        if (lds.doubt) {  // a bias, and groups that float32 cannot tell apart: the same in float64
            if (softmax) exact_sum();
            for (int g = tid; g < p.groups; g += THREADS) f.exact_max[g] = f.exact_next[g] = 0;
            __syncthreads();
            for (int n = tid; n < p.keys; n += THREADS) {
                const float a = logit_at(row, n);
                if (!(a > -INFINITY) || bias_excludes(p.bias[n])) continue;
                const unsigned long long h = ordered64(exact_score(a) + double(p.bias[n]));
                const int g = group_of(n);
                const unsigned long long l = min(h, atomicMax(&f.exact_max[g], h));
                if (l > kOut64) atomicMax(&f.exact_next[g], l);
            }
            __syncthreads();
            for (int g = tid; g < p.groups; g += THREADS) {
                double v = f.exact_max[g] > kOut64 ? from_ordered64(f.exact_max[g]) : -INFINITY;
                if (p.top == 2 && f.exact_next[g] > kOut64) v += from_ordered64(f.exact_next[g]);
                f.worth[g] = v;
            }
            __syncthreads();
            for (int g = tid; g < p.groups; g += THREADS) {
                int rank = 0;
                for (int h = 0; h < p.groups; ++h)
                    rank += (f.worth[h] > f.worth[g]) | ((f.worth[h] == f.worth[g]) & (h < g));
                f.kept[g] = rank < p.kept;
            }
            __syncthreads();
            if (tid == 0) lds.doubt = 0;
        }
        most = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const bool kept = f.kept[group_of(min(key_of(i), p.keys - 1))];
            if (kept) most = max32(most, c[i]);
            c[i] = kept ? c[i] : NAN;  // NaN: reaches no bound
        }
    }

    lds.first.lane_max[tid] = ordered(most);
    for (int i = tid; i < kCandidates; i += THREADS) lds.rank[i] = 0;
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
        if (lane == 0) lds.threshold = max(bound, kOut);  // -inf: every key that there is
    }
    __syncthreads();
    // With a bias, the keys that may be among the k best are those within twice the
    // slack of a bound that k keys reach.
    auto widened = [&](uint32_t bound) {
        const float v = from_ordered(bound);
        return biased && fabsf(v) < INFINITY ? max32(v - 2 * block_slack(softmax, v), -FLT_MAX) : v;
    };
    uint32_t zero = 0;
    opaque(zero);  // an address that may differ between lanes: few add at a time, one by one is best
    auto collect = [&](auto takes) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (takes(c[i], key_of(i))) {
                uint32_t n = uint32_t(key_of(i));
                opaque(n);  // compared here, and not for all keys beforehand
                if (int(n) >= p.keys) continue;
                const int at = atomicAdd(&lds.found + zero, 1);
                if (at < kCandidates) lds.cand[at] = uint64_t(ordered(c[i])) << 32 | ~n;
            }
    };
    auto value_of = [](uint64_t cand) { return from_ordered(uint32_t(cand >> 32)); };
    const float low = widened(lds.threshold);
    if (most >= low) collect([&](float v, int) { return v >= low; });
    __syncthreads();
    if (lds.found > kCandidates) {
        int turn = 0;
        auto count = [&](auto counts) {  // over the row
            int n = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float v = c[i];
                uint32_t key = uint32_t(key_of(i));
                opaque(v);  // else the loops below would hold another integer and a mask for each key
                opaque(key);
                n += __popcll(__ballot(v == v && int(key) < p.keys && counts(ordered(v), int(key))));
            }
            if (tid == 0) lds.count[turn] = 0;
            __syncthreads();
            if (lane == 0) atomicAdd(&lds.count[turn], n);
            __syncthreads();
            n = lds.count[turn];
            turn ^= 1;
            return n;
        };
        uint32_t kth = 0;
#pragma unroll 1
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t trial = kth | 1u << bit;
            if (count([&](uint32_t k, int) { return k >= trial; }) >= p.k) kth = trial;
        }
        if (tid == 0) lds.found = 0;
        if (biased && kth > kOut) {
            const uint32_t least = ordered(widened(kth));
            const int n = count([&](uint32_t k, int) { return k >= least; });
            if (n > kCandidates) {
                __syncthreads();
                if constexpr (GENERAL) exact_row<E, THREADS>(p, t, lds.exact);
                return;
            }
            collect([&](float v, int) { return ordered(v) >= least && v == v; });
        } else {
            const int need = p.k - count([&](uint32_t k, int) { return k > kth; });
            int last = 0;  // the lowest keys among those equal to the k-th, up to this one
#pragma unroll 1
            for (int bit = 15; bit >= 0; --bit) {
                const int trial = last | 1 << bit;
                if (count([&](uint32_t k, int n) { return k == kth && n < trial; }) < need) last = trial;
            }
            collect([&](float v, int n) { return v == v && (ordered(v) > kth || (ordered(v) == kth && n <= last)); });
        }
        __syncthreads();
    }
    const int found = lds.found;
    auto& f = lds.second;
    // Each candidate's rank is the number of those that go before it, counted by as
    // many threads as there are for it.
    auto rank_all = [&] {
        int per = 64;
        while (per < found && per < THREADS) per *= 2;
        const int parts = THREADS / per, part = tid / per;
        for (int i = tid % per; i < found; i += per) {
            const uint64_t mine = lds.cand[i];
            int rank = 0;
            if (biased) {
                const uint64_t v = f.value[i];
                for (int j = part; j < found; j += parts)
                    rank += (f.value[j] > v) | ((f.value[j] == v) & (uint32_t(lds.cand[j]) > uint32_t(mine)));
            } else {
#pragma unroll 4
                for (int j = 2 * part; j < found; j += 2 * parts) {
                    const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(&lds.cand[j]);
                    rank += (two.x > mine) + (two.y > mine);
                }
            }
            if (rank != 0) atomicAdd(&lds.rank[i], rank);
        }
    };
    if (biased) {
        // The candidates' exact values. A softmax's float32 sum is off by up to 2^-17 of itself,
        // by the same for all scores, so two values change places if they are nearer than that of
        // their scores' difference. If none of the k chosen may have done so with the next, and
        // none of the others with the last of them, the choice stands; else the sum is taken in
        // float64 and the order again.
        exact_z = double(z);
        for (int turn = 0; turn < 2; ++turn) {
            for (int i = tid; i < found; i += THREADS) {
                const int n = int(~uint32_t(lds.cand[i]));
                double v = -INFINITY;
                if (value_of(lds.cand[i]) > -INFINITY) v = exact_score(logit_at(row, n)) + double(p.bias[n]);
                f.value[i] = ordered64(v);
                lds.rank[i] = 0;
            }
            __syncthreads();
            rank_all();
            __syncthreads();
            if (!softmax || turn == 1) break;
            auto score_of = [&](int i) { return exact_score(logit_at(row, int(~uint32_t(lds.cand[i])))); };
            for (int i = tid; i < found; i += THREADS)
                if (lds.rank[i] < p.k) {
                    f.sorted[lds.rank[i]] = from_ordered64(f.value[i]);
                    f.score[lds.rank[i]] = score_of(i);
                }
            __syncthreads();
            if (tid + 1 < p.k && near(f.sorted[tid], f.sorted[tid + 1], fabs(f.score[tid] - f.score[tid + 1]), 0x1p-16))
                lds.doubt = 1;
            for (int i = tid; i < found; i += THREADS)
                if (lds.rank[i] >= p.k && near(f.sorted[p.k - 1], from_ordered64(f.value[i]),
                                               fabs(f.score[p.k - 1] - score_of(i)), 0x1p-16))
                    lds.doubt = 1;
            __syncthreads();
            if (!lds.doubt) break;
            exact_sum();
        }
    } else if (tid == 0 && found < kCandidates) {
        lds.cand[found] = 0;  // the list in pairs; everything goes before a 0
    }
    if (!biased) {
        __syncthreads();
        rank_all();
        __syncthreads();
    }
    for (int i = tid; i < found; i += THREADS) {
        const int rank = lds.rank[i], n = int(~uint32_t(lds.cand[i]));
        const float v = value_of(lds.cand[i]);
        if (rank < p.k) {
            lds.chosen[rank] = n;
            lds.chosen_value[rank] = v;
        }
    }
    __syncthreads();
    if (tid / 64 * 64 >= p.k && !p.normalise) return;  // the other wavefronts have no part in the weights
    if (stats && !biased) row_stats();
    const int key = tid < p.k ? lds.chosen[tid] : 0;
    // What a key was chosen by is its logit, or -inf, where there is no bias.
    float xk = tid < p.k ? lds.chosen_value[tid] : -INFINITY;
    const bool ok = xk > -INFINITY;
    if (biased && ok) xk = logit_at(row, key);
    double s = 0;
    if (p.normalise && softmax) {
        const double top = block(ok ? double(xk) : -double(FLT_MAX), [](double a, double b) { return fmax(a, b); });
        if (ok) s = exp(double(xk) - top);
    } else if (ok) {
        s = softmax ? exp(double(xk) - double(m)) / (biased ? exact_z : double(z)) : sigmoid64(xk);
    }
    if (p.normalise) {
        const double total = block_sum(s);
        s = total > 0 ? s / total : 0.0;
    }
    if (tid < p.k) store_choice(p, t, tid, key, s);
}

template <typename E, int THREADS, int VPT> void run(const RouteParams& p, bool vec, hipStream_t stream) {
    const dim3 grid{unsigned(p.tokens)}, block{THREADS};
    const bool general = p.bias != nullptr || p.groups > 1;
    if constexpr (VPT * sizeof(E) % 16 == 0) {
        if (vec) {
            if (general) hipLaunchKernelGGL((route_block_kernel<E, THREADS, VPT, true, true>), grid, block, 0, stream, p);
            else hipLaunchKernelGGL((route_block_kernel<E, THREADS, VPT, true, false>), grid, block, 0, stream, p);
            return;
        }
    }
    if (general) hipLaunchKernelGGL((route_block_kernel<E, THREADS, VPT, false, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((route_block_kernel<E, THREADS, VPT, false, false>), grid, block, 0, stream, p);
}

// Lanes at least twice k, so that few keys reach the lanes' bound; of those, few
// lanes of many keys: what a wavefront does besides its keys is then shared by more
// of them. 32 keys a lane are the most that leave three workgroups of 512 to a CU
// (4096 rows of 16384, 64 chosen: 53 us; 256 lanes of 64 keys take as long and spill).
template <typename E> void run_route(const RouteParams& p, hipStream_t stream) {
    const bool vec = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && p.keys * sizeof(E) % 16 == 0;
    if (p.k <= 128 && p.keys <= 8192) {
        if (p.keys <= 1024) run<E, 256, 4>(p, vec, stream);
        else if (p.keys <= 2048) run<E, 256, 8>(p, vec, stream);
        else if (p.keys <= 4096) run<E, 256, 16>(p, vec, stream);
        else run<E, 256, 32>(p, vec, stream);
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
