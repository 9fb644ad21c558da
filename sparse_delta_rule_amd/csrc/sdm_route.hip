// The slot router: sdm_route (the k best keys of each token, and their weights)
// and sdm_route_backward (include/sdm_memory.h).

#include <float.h>
#include <math.h>

#include "../../include/sdm_memory.h"
#include "sdm_kernels.h"
#include "sdm_memory.h"

namespace sdm {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 20;  // a grid's workgroups; more tokens are looped over

// A logit as the definition reads it: NaN counts as -inf, +inf as the largest float32.
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : fminf(x, FLT_MAX); }
template <typename E> __device__ __forceinline__ float logit_at(const E* row, int64_t i) { return clean(widen(row[i])); }

__device__ __forceinline__ bool bias_excludes(float b) { return !(b > -INFINITY); }

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// A key's rank among the keys of its row: the larger value first, then the lower key.
struct Ranked {
    double c;
    int key;
};
__device__ __forceinline__ bool before(const Ranked& a, const Ranked& b) {
    return a.c > b.c || (a.c == b.c && a.key < b.key);
}

template <typename T, typename F> __device__ __forceinline__ T block_reduce(T v, T* lds, F f) {
    __syncthreads();
    lds[threadIdx.x] = v;
    __syncthreads();
    for (int n = kThreads / 2; n > 0; n /= 2) {
        if (int(threadIdx.x) < n) lds[threadIdx.x] = f(lds[threadIdx.x], lds[threadIdx.x + n]);
        __syncthreads();
    }
    return lds[0];
}

// One workgroup per token; every value in float64, k rounds of a reduction over
// the keys that come after the last one chosen.
template <typename E>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteParams p) {
    __shared__ Ranked red[kThreads];
    __shared__ double redd[kThreads];
    __shared__ double worth[SDM_MAX_GROUPS];
    __shared__ uint8_t kept[SDM_MAX_GROUPS];
    __shared__ int chosen[SDM_MAX_WIDTH];
    const int tid = threadIdx.x;
    for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
        const E* row = static_cast<const E*>(p.logits) + t * p.keys;

        double m = 0, z = 1;
        if (p.score == SDM_SOFTMAX) {
            double v = -INFINITY;
            for (int i = tid; i < p.keys; i += kThreads) v = fmax(v, double(logit_at(row, i)));
            m = fmax(block_reduce(v, redd, [](double a, double b) { return fmax(a, b); }), -double(FLT_MAX));
            v = 0;
            for (int i = tid; i < p.keys; i += kThreads) v += exp(double(logit_at(row, i)) - m);
            z = block_reduce(v, redd, [](double a, double b) { return a + b; });
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
            for (int g = tid; g < p.groups; g += kThreads) {
                double a = -INFINITY, b = -INFINITY;  // the two largest
                for (int i = g * size; i < (g + 1) * size; ++i) {
                    if (!eligible(i)) continue;
                    const double c = score(i) + (p.bias != nullptr ? double(p.bias[i]) : 0.0);
                    b = fmax(b, fmin(a, c));
                    a = fmax(a, c);
                }
                worth[g] = p.top == 2 && b > -INFINITY ? a + b : a;
            }
            __syncthreads();
            for (int g = tid; g < p.groups; g += kThreads) {
                int rank = 0;
                for (int h = 0; h < p.groups; ++h) rank += worth[h] > worth[g] || (worth[h] == worth[g] && h < g);
                kept[g] = rank < p.kept;
            }
            __syncthreads();
        }
        Ranked last = {INFINITY, -1};
        for (int j = 0; j < p.k; ++j) {
            Ranked best = {-INFINITY, 0x7fffffff};
            for (int i = tid; i < p.keys; i += kThreads) {
                if (p.groups > 1 && !kept[i / size]) continue;
                Ranked r = {-INFINITY, i};
                if (eligible(i)) r.c = p.bias != nullptr ? score(i) + double(p.bias[i]) : double(logit_at(row, i));
                if (before(last, r) && before(r, best)) best = r;
            }
            last = block_reduce(best, red, [](Ranked a, Ranked b) { return before(b, a) ? b : a; });
            if (tid == 0) chosen[j] = last.key;
        }
        __syncthreads();
        const int key = tid < p.k ? chosen[tid] : 0;
        const bool mine = tid < p.k && eligible(key);
        double u = 0;
        if (p.normalise && p.score == SDM_SOFTMAX) {
            const double x = mine ? double(logit_at(row, key)) : -INFINITY;
            const double top = fmax(block_reduce(x, redd, [](double a, double b) { return fmax(a, b); }), -double(FLT_MAX));
            u = exp(x - top);
        } else if (mine) {
            u = score(key);
        }
        if (p.normalise) {
            const double total = block_reduce(u, redd, [](double a, double b) { return a + b; });
            u = total > 0 ? u / total : 0.0;
        }
        if (tid < p.k) {
            const int64_t o = t * p.k + tid, slot = (t % p.streams) * p.stream_slots + key;
            if (p.idx64) static_cast<int64_t*>(p.idx)[o] = slot;
            else static_cast<int32_t*>(p.idx)[o] = int32_t(slot);
            const float w = float(p.scale * u);
            if (p.w_bf16) static_cast<uint16_t*>(p.w)[o] = to_bf16_rne(w);
            else static_cast<float*>(p.w)[o] = w;
        }
    }
}

constexpr int kTile = 4096;  // gradients assembled in LDS at a time

// One workgroup per token: the chosen keys' part in float64, then the row in
// tiles, each assembled in LDS from the chosen keys and written whole.
template <typename E>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(RouteBackwardParams p) {
    __shared__ double redd[kThreads];
    __shared__ float redf[kThreads];
    __shared__ float tile[kTile];
    const int tid = threadIdx.x;
    for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
        const E* row = static_cast<const E*>(p.logits) + t * p.keys;
        E* drow = static_cast<E*>(p.dlogits) + t * p.keys;
        const bool whole = p.score == SDM_SOFTMAX && !p.normalise;

        float m = 0, z = 1;
        if (whole) {
            float v = -INFINITY;
            for (int i = tid; i < p.keys; i += kThreads) v = fmaxf(v, logit_at(row, i));
            m = fmaxf(block_reduce(v, redf, [](float a, float b) { return fmaxf(a, b); }), -FLT_MAX);
            v = 0;
            for (int i = tid; i < p.keys; i += kThreads) v += expf(logit_at(row, i) - m);
            z = block_reduce(v, redf, [](float a, float b) { return a + b; });
        }
        int64_t key = -1;
        double x = -INFINITY, dw = 0;
        if (tid < p.k) {
            const int64_t o = t * p.k + tid;
            key = (p.idx64 ? static_cast<const int64_t*>(p.idx)[o] : int64_t(static_cast<const int32_t*>(p.idx)[o])) -
                  (t % p.streams) * p.stream_slots;
            if (key < 0 || key >= p.keys) key = -1;
            if (key >= 0 && !(p.bias != nullptr && bias_excludes(p.bias[key]))) x = logit_at(row, key);
            dw = p.w_bf16 ? widen(static_cast<const uint16_t*>(p.dw)[o]) : static_cast<const float*>(p.dw)[o];
        }
        const bool mine = x > -INFINITY;
        if (!mine) dw = 0;  // no part in anything, whatever its gradient holds
        double u = 0;  // score, up to a factor of the row where the weights are normalised
        if (p.score == SDM_SIGMOID) {
            if (mine) u = sigmoid64(x);
        } else if (p.normalise) {
            const double top = fmax(block_reduce(x, redd, [](double a, double b) { return fmax(a, b); }), -double(FLT_MAX));
            u = exp(x - top);
        } else if (mine) {
            u = exp(x - double(m)) / double(z);
        }
        double d = p.scale * dw;
        if (p.normalise) {
            const double total = block_reduce(u, redd, [](double a, double b) { return a + b; });
            u = total > 0 ? u / total : 0.0;
        }
        float sum = 0;
        if (p.normalise || whole) {
            const double dot = block_reduce(d * u, redd, [](double a, double b) { return a + b; });
            if (whole) sum = float(dot);
            else d -= dot;
        }
        float g = float(d);  // full softmax: the row below multiplies by s
        if (!whole) {
            d *= u;
            if (p.score == SDM_SIGMOID && mine) d /= 1.0 + exp(x);
            g = float(d);
        }
        for (int a = 0; a < p.keys; a += kTile) {
            const int n = min(kTile, p.keys - a);
            __syncthreads();
            for (int i = tid; i < n; i += kThreads) tile[i] = 0;
            __syncthreads();
            if (mine && key >= a && key < a + n) atomicAdd(&tile[key - a], g);
            __syncthreads();
            for (int i = tid; i < n; i += kThreads) {
                float v = tile[i];
                if (whole) v = z > 0 ? expf(logit_at(row, a + i) - m) / z * (v - sum) : 0.0f;
                drow[a + i] = narrow<E>(v);
            }
        }
    }
}

}  // namespace

hipError_t launch_route(const RouteParams& p, bool bf16, hipStream_t stream) {
    const dim3 grid{unsigned(p.tokens < kMaxBlocks ? p.tokens : kMaxBlocks)}, block{unsigned(kThreads)};
    if (bf16) hipLaunchKernelGGL(route_kernel<uint16_t>, grid, block, 0, stream, p);
    else hipLaunchKernelGGL(route_kernel<float>, grid, block, 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardParams& p, bool bf16, hipStream_t stream) {
    const dim3 grid{unsigned(p.tokens < kMaxBlocks ? p.tokens : kMaxBlocks)}, block{unsigned(kThreads)};
    if (bf16) hipLaunchKernelGGL(route_backward_kernel<uint16_t>, grid, block, 0, stream, p);
    else hipLaunchKernelGGL(route_backward_kernel<float>, grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace sdm
