// The columns that a lookup's dropout keeps: Philox4x32-10 (Salmon, Moraes, Dror, Shaw,
// 2011), a block cipher of ten rounds that turns a counter into four random words.
#pragma once

#include "sdm_train.h"

namespace sdm {

struct PhiloxKey {
    uint32_t k0, k1, c2, c3;  // the key, and the half of the counter that a call has in common
};
__device__ __forceinline__ PhiloxKey philox_key(const Dropout& d) {
    const uint64_t seed = d.rng[0], offset = d.rng[1];
    return {uint32_t(seed), uint32_t(seed >> 32), uint32_t(offset), uint32_t(offset >> 32)};
}

// Bit j: column 8 * octet + j of row `row` stays.
__device__ __forceinline__ uint32_t kept_columns(const PhiloxKey& key, uint32_t octet, uint32_t row, uint32_t threshold) {
    uint32_t c0 = octet, c1 = row, c2 = key.c2, c3 = key.c3, k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = uint64_t(c0) * 0xD2511F53u, p1 = uint64_t(c2) * 0xCD9E8D57u;
        c0 = uint32_t(p1 >> 32) ^ c1 ^ k0;
        c1 = uint32_t(p1);
        c2 = uint32_t(p0 >> 32) ^ c3 ^ k1;
        c3 = uint32_t(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    const uint32_t words[4] = {c0, c1, c2, c3};
    uint32_t kept = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) kept |= uint32_t((words[j / 2] >> (j % 2 * 16) & 0xffffu) >= threshold) << j;
    return kept;
}

}  // namespace sdm
