// Vectors of a row's columns as float32, of every element type.
#pragma once

#include "../../include/sdm_memory.h"
#include "sdm_kernels.h"

namespace sdm {

// Eight consecutive columns of a row as float32, VB bytes a load; columns at or
// past `left` are 0.
template <typename E, int VB> __device__ __forceinline__ void load_octet(const E* p, int left, float (&x)[8]) {
    constexpr int VEC = VB / int(sizeof(E));
    if (left >= 8) {
        typename RawVec<VB>::T raw[8 / VEC];
#pragma unroll
        for (int i = 0; i < 8 / VEC; ++i) raw[i] = reinterpret_cast<const typename RawVec<VB>::T*>(p)[i];
        E e[8];
        __builtin_memcpy(e, raw, sizeof e);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = widen(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < left ? widen(p[i]) : 0.0f;
    }
}

// Store eight columns of a row, VB bytes a store; columns at or past `left` are not stored.
template <typename E, int VB> __device__ __forceinline__ void store_octet(E* p, int left, const float (&x)[8]) {
    constexpr int VEC = VB / int(sizeof(E));
    if (left >= 8) {
#pragma unroll
        for (int i = 0; i < 8; i += VEC) {
            float v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = x[i + j];
            store_stream(reinterpret_cast<typename RawVec<VB>::T*>(p + i), Pack<E, VB>::of(v));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = narrow<E>(x[i]);
    }
}

// N consecutive columns of a packed row (16, 8 or 4): their codes, and their values as float32.
template <bool MX4, int N> struct Codes {
    static constexpr int kBytes = MX4 ? N / 2 : N;
    using Raw = typename RawVec<kBytes>::T;
    static __device__ __forceinline__ void values(const Raw& v, float s, float (&x)[N]) {
        uint32_t w[kBytes < 4 ? 1 : kBytes / 4] = {};
        __builtin_memcpy(w, &v, kBytes);
        if constexpr (MX4) {
#pragma unroll
            for (int i = 0; i < (N + 7) / 8; ++i) {
                const F32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], s, 0);
                const F32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], s, 1);
                x[8 * i] = a.x, x[8 * i + 1] = a.y, x[8 * i + 2] = b.x, x[8 * i + 3] = b.y;
                if constexpr (N >= 8) {
                    const F32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], s, 2);
                    const F32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], s, 3);
                    x[8 * i + 4] = c.x, x[8 * i + 5] = c.y, x[8 * i + 6] = d.x, x[8 * i + 7] = d.y;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const F32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i], s, false);
                const F32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i], s, true);
                x[4 * i] = a.x, x[4 * i + 1] = a.y, x[4 * i + 2] = b.x, x[4 * i + 3] = b.y;
            }
        }
    }
};

}  // namespace sdm
