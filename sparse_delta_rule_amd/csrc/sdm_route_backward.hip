// sdm_route_backward (include/sdm_memory.h).

#include "sdm_route_device.h"

namespace sdm {

namespace {

// A chosen key of a token as the backward pass reads it: -1 where it is not one of
// the token's keys, x = -inf and dw = 0 where it has no part in anything.
struct Choice {
    int key;
    float x;
    double dw;
};
template <typename E> __device__ __forceinline__ Choice choice_at(const RouteBackwardParams& p, int64_t t, int j) {
    const int64_t o = t * p.k + j;
    const int64_t slot = p.idx64 ? static_cast<const int64_t*>(p.idx)[o] : int64_t(static_cast<const int32_t*>(p.idx)[o]);
    const int64_t key = slot - int64_t(uint32_t(t) % p.streams) * p.stream_slots;
    Choice c = {-1, -INFINITY, 0.0};
    if (key >= 0 && key < p.keys) {
        c.key = int(key);
        if (!(p.bias != nullptr && bias_excludes(p.bias[key])))
            c.x = logit_at(static_cast<const E*>(p.logits) + t * p.keys, key);
    }
    if (c.x > -INFINITY)
        c.dw = p.w_bf16 ? widen(static_cast<const uint16_t*>(p.dw)[o]) : static_cast<const float*>(p.dw)[o];
    return c;
}

// ------------------------------------------------------------------ zeros but for the chosen keys

constexpr int kTile = 2048;  // gradients that a wavefront assembles in LDS at a time
constexpr int kWaves = 4;    // wavefronts of a workgroup

// Renormalised weights, and sigmoid scores: a wavefront takes `rows` consecutive
// tokens, `lanes` of its lanes the chosen keys of each (in float64: they are few),
// PER keys a lane. The rows are then assembled in LDS and written as one run of
// memory. What bounds it is that writing.
template <typename E, int PER>
__global__ __launch_bounds__(64 * kWaves) void route_backward_sparse_kernel(RouteBackwardParams p, int rows, int lanes) {
    __shared__ alignas(16) float tiles[kWaves][kTile];
    ieee_mode_off();
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t t0 = (int64_t(blockIdx.x) * kWaves + wave) * rows;
    if (t0 >= p.tokens) return;
    const int there = int(min(int64_t(rows), p.tokens - t0));
    float* tile = tiles[wave];
    const int r = lane / lanes, j0 = lane % lanes;
    Choice c[PER];
    double u[PER];
    auto over_row = [&](double v, auto f) {
        for (int n = 1; n < lanes; n *= 2) v = f(v, __shfl_xor(v, n));
        return v;
    };
    const auto plus = [](double a, double b) { return a + b; };
    float most = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        c[i] = Choice{-1, -INFINITY, 0.0};
        if (r < there && j0 + i * lanes < p.k) c[i] = choice_at<E>(p, t0 + r, j0 + i * lanes);
        most = max32(most, c[i].x);
    }
    if (p.score == SDM_SOFTMAX)
        for (int n = 1; n < lanes; n *= 2) most = max32(most, __shfl_xor(most, n));
    double total = 0, dot = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        u[i] = c[i].x > -INFINITY ? (p.score == SDM_SIGMOID ? sigmoid64(c[i].x) : exp(double(c[i].x) - double(most))) : 0.0;
        total += u[i];
    }
    if (p.normalise) {
        total = over_row(total, plus);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            u[i] = total > 0 ? u[i] / total : 0.0;
            dot += c[i].dw * u[i];
        }
        dot = over_row(dot, plus);
    }
    float g[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        double d = p.scale * u[i] * (c[i].dw - dot);
        if (p.score == SDM_SIGMOID) d /= 1.0 + exp(double(c[i].x));  // 1 - s; x = -inf gives 1
        g[i] = c[i].x > -INFINITY && !(p.normalise && total == 0) ? float(d) : 0.0f;
    }
    E* out = static_cast<E*>(p.dlogits) + t0 * p.keys;
    const int whole = there * p.keys;  // of one row where it does not fit the tile
    for (int a = 0; a < whole; a += kTile) {
        const int n = min(kTile, whole - a);
        for (int i = lane * 4; i < n; i += 256) *reinterpret_cast<float4*>(tile + i) = make_float4(0, 0, 0, 0);
        wave_lds_order();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = r * p.keys + c[i].key - a;
            if (c[i].key >= 0 && at >= 0 && at < n) atomicAdd(tile + at, g[i]);
        }
        wave_lds_order();
        constexpr int kN = 16 / int(sizeof(E));
        E* to = out + a;
        if (reinterpret_cast<uintptr_t>(to) % 16 == 0) {
            for (int i = lane * kN; i + kN <= n; i += 64 * kN) {
                float v[kN];
#pragma unroll
                for (int j = 0; j < kN; ++j) v[j] = tile[i + j];
                store_stream(reinterpret_cast<uint4*>(to + i), Pack<E, 16>::of(v));
            }
            if (lane < n % kN) to[n - n % kN + lane] = narrow<E>(tile[n - n % kN + lane]);
        } else {
            for (int i = lane; i < n; i += 64) to[i] = narrow<E>(tile[i]);
        }
        wave_lds_order();
    }
}

// ------------------------------------------------------------------ a full softmax

template <int THREADS> struct WholeLds {
    float wave_max[THREADS / 64];
    double wave_sum[THREADS / 64], wave_value[THREADS / 64];
    int head[THREADS];  // a lane's list of the chosen keys it holds: -1, or the first's number
    int next[SDM_MAX_WIDTH];
    int key[SDM_MAX_WIDTH];
    double s[SDM_MAX_WIDTH], du[SDM_MAX_WIDTH];
};

// A workgroup a token, the row in its registers: read once, written once. Every key
// gets -s_i sum_j du_j s_j, and each lane then stores its chosen keys' own gradients,
// computed in float64, over that: a lane's stores to one address happen in order.
// Bound by its memory traffic: 4096 rows of 16384 bfloat16 keys in 51 us, 5.3 TB/s of
// bytes read and written (a large copy: 6.2; with a float32 sum over the row 50 us).
template <typename E, int THREADS, int VPT, bool VEC>
__global__ __launch_bounds__(THREADS) void route_backward_whole_kernel(RouteBackwardParams p) {
    using Row = RowKeys<E, THREADS, VPT, VEC>;
    constexpr int kN = Row::kN;
    __shared__ WholeLds<THREADS> lds;
    ieee_mode_off();
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const int64_t t = blockIdx.x;
    const E* row = static_cast<const E*>(p.logits) + t * p.keys;
    E* out = static_cast<E*>(p.dlogits) + t * p.keys;
    float c[VPT];
    Row::load(row, p.keys, tid, c);
    Choice mine = {-1, -INFINITY, 0.0};
    if (tid < p.k) mine = choice_at<E>(p, t, tid);
    lds.head[tid] = -1;
    const float v = lanes_reduce<64>(max_of(c, -FLT_MAX), [](float a, float b) { return max32(a, b); });
    // The largest term is exactly 1 and the others are added to it in float64, so that 1 - s
    // of a key far above the rest has the precision of the others' terms.
    double sum = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) sum += double(exp32(c[i] - v));
    for (int n = 1; n < 64; n *= 2) sum += __shfl_xor(sum, n);
    if (lane == 0) {
        lds.wave_max[wave] = v;
        lds.wave_sum[wave] = sum;
    }
    __syncthreads();
    float m = -FLT_MAX;
    double z = 0;
    for (int w = 0; w < THREADS / 64; ++w) m = max32(m, lds.wave_max[w]);
    for (int w = 0; w < THREADS / 64; ++w) z += lds.wave_sum[w] * double(exp32(lds.wave_max[w] - m));
    const double du = p.scale * mine.dw;
    const double s = mine.x > -INFINITY ? exp(double(mine.x) - double(m)) / z : 0.0;
    double dot = du * s;
    if (wave * 64 < p.k) {
        for (int n = 1; n < 64; n *= 2) dot += __shfl_xor(dot, n);
        if (mine.x > -INFINITY) {
            const int owner = VEC ? mine.key / kN % THREADS : mine.key % THREADS;
            lds.key[tid] = mine.key;
            lds.s[tid] = s;
            lds.du[tid] = du;
            lds.next[tid] = atomicExch(&lds.head[owner], tid);
        }
    }
    if (lane == 0) lds.wave_value[wave] = dot;
    __syncthreads();
    dot = 0;
    for (int w = 0; w * 64 < p.k; ++w) dot += lds.wave_value[w];
    const double factor = z > 0 ? -dot / z : 0.0;
    const float f = float(factor);
#pragma unroll
    for (int i = 0; i < VPT; ++i) c[i] = exp32(c[i] - m) * f;
#pragma unroll
    for (int i = 0; i < VPT; i += kN) {
        if constexpr (VEC) {
            float part[kN];
#pragma unroll
            for (int j = 0; j < kN; ++j) part[j] = c[i + j];
            if (Row::key_of(i, tid) < p.keys) *reinterpret_cast<uint4*>(out + Row::key_of(i, tid)) = Pack<E, 16>::of(part);
        } else {
            if (Row::key_of(i, tid) < p.keys) out[Row::key_of(i, tid)] = narrow<E>(c[i]);
        }
    }
    if (!(fabsf(f) < INFINITY)) {
        // Past float32, or not finite: the row again with the factor in float64. A masked key's
        // gradient is 0 all the same.
#pragma unroll 1
        for (int i = 0; i < VPT; ++i) {
            const int n = Row::key_of(i, tid);
            if (n >= p.keys) continue;
            const float x = logit_at(row, n);
            out[n] = narrow<E>(x > -INFINITY ? float(factor * exp32(x - m)) : 0.0f);
        }
    }
    for (int j = lds.head[tid]; j >= 0; j = lds.next[j]) {
        double all = 0;  // of the key, should it have been given more than once
        for (int i = lds.head[tid]; i >= 0; i = lds.next[i])
            if (lds.key[i] == lds.key[j]) all += lds.du[i];
        out[lds.key[j]] = narrow<E>(float(lds.s[j] * (all - dot)));
    }
}

template <typename E, int THREADS, int VPT> void run_whole(const RouteBackwardParams& p, bool vec, hipStream_t stream) {
    const dim3 grid{unsigned(p.tokens)}, block{THREADS};
    if constexpr (VPT * sizeof(E) % 16 == 0) {
        if (vec) {
            hipLaunchKernelGGL((route_backward_whole_kernel<E, THREADS, VPT, true>), grid, block, 0, stream, p);
            return;
        }
    }
    hipLaunchKernelGGL((route_backward_whole_kernel<E, THREADS, VPT, false>), grid, block, 0, stream, p);
}

template <typename E, int PER> void run_sparse(const RouteBackwardParams& p, int rows, int lanes, hipStream_t stream) {
    const int64_t waves = (p.tokens + rows - 1) / rows;
    const dim3 grid{unsigned((waves + kWaves - 1) / kWaves)}, block{64 * kWaves};
    hipLaunchKernelGGL((route_backward_sparse_kernel<E, PER>), grid, block, 0, stream, p, rows, lanes);
}

template <typename E> void run_backward(const RouteBackwardParams& p, hipStream_t stream) {
    if (p.score == SDM_SOFTMAX && !p.normalise) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p.logits) | reinterpret_cast<uintptr_t>(p.dlogits);
        const bool vec = at % 16 == 0 && p.keys * sizeof(E) % 16 == 0;
        // At least a thread for each chosen key.
        if (p.keys <= 2048) run_whole<E, 256, 8>(p, vec, stream);
        else if (p.keys <= 8192) run_whole<E, 256, 32>(p, vec, stream);
        else if (p.keys <= 16384) run_whole<E, 256, 64>(p, vec, stream);
        else run_whole<E, 1024, 64>(p, vec, stream);
        return;
    }
    int lanes = 1;
    while (lanes < 64 && lanes < p.k) lanes *= 2;
    int rows = 64 / lanes;
    while (rows > 1 && rows * p.keys > kTile) rows /= 2;
    if (p.k <= 64) run_sparse<E, 1>(p, rows, lanes, stream);
    else run_sparse<E, 4>(p, rows, lanes, stream);
}

}  // namespace

hipError_t launch_route_backward(const RouteBackwardParams& p, bool bf16, hipStream_t stream) {
    if (bf16) run_backward<uint16_t>(p, stream);
    else run_backward<float>(p, stream);
    return hipGetLastError();
}

}  // namespace sdm
