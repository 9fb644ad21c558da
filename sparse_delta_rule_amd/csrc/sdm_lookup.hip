// sdm_lookup (include/sdm_train.h).

#include "sdm_dropout.h"
#include "sdm_rows.h"

namespace sdm {

namespace {

constexpr int kThreads = 256;

// Eight columns of a row of any bank as float32; columns past the row's end may hold anything.
template <int KIND, int VB> struct OctetOf;
template <int VB> struct OctetOf<SDM_F32, VB> {
    static __device__ __forceinline__ void load(const LookupParams& p, int64_t slot, int o, float (&x)[8]) {
        load_octet<float, VB>(static_cast<const float*>(p.bank) + slot * p.hd + 8 * o, p.hd - 8 * o, x);
    }
};
template <int VB> struct OctetOf<SDM_BF16, VB> {
    static __device__ __forceinline__ void load(const LookupParams& p, int64_t slot, int o, float (&x)[8]) {
        load_octet<uint16_t, VB>(static_cast<const uint16_t*>(p.bank) + slot * p.hd + 8 * o, p.hd - 8 * o, x);
    }
};
template <bool MX4> struct PackedOctet {
    static __device__ __forceinline__ void load(const LookupParams& p, int64_t slot, int o, float (&x)[8]) {
        using C = Codes<MX4, 8>;
        const auto raw = reinterpret_cast<const typename C::Raw*>(static_cast<const char*>(p.bank) + slot * p.row_bytes)[o];
        const uint32_t s = p.scales[slot * p.scale_bytes + o / 4];
        C::values(raw, __uint_as_float(s << 23), x);
    }
};
template <> struct OctetOf<SDM_MX8, 16> : PackedOctet<false> {};
template <> struct OctetOf<SDM_MX4, 16> : PackedOctet<true> {};

// A thread takes eight columns of ROWS rows, a row's threads are neighbours. 32768 rows of 1024
// bfloat16 take 15.5 us, 6.5 TB/s of rows fetched (each by the XCDs that read it) and written; with
// dropout 20, as the ten rounds of the generator, though one run serves eight columns, are 10.4 M vector
// instructions, some 17 us, that the loads only in part hide. A launch of few rows is bound by two
// dependent loads (64 rows: 2.6 us).
template <int KIND, int VB, typename E, int OVB, bool DROP, int ROWS>
__global__ __launch_bounds__(kThreads) void lookup_kernel(LookupParams p) {
    const int octets = (p.hd + 7) / 8;
    const int per_row = min(octets, kThreads), rows = kThreads / per_row;
    const int r = int(threadIdx.x) / per_row, o = int(blockIdx.y) * kThreads + int(threadIdx.x) % per_row;
    if (r >= rows || o >= octets) return;
    const int64_t i0 = p.first + int64_t(blockIdx.x) * (rows * ROWS) + r;
    int64_t slot[ROWS];
    float x[ROWS][8];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        slot[u] = slot_at(p.idx, min(i0 + u * rows, p.n - 1), p.idx64 ? 8 : 4);
        if (uint64_t(slot[u]) >= uint64_t(p.num_slots)) slot[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < ROWS; ++u) OctetOf<KIND, VB>::load(p, max(slot[u], int64_t(0)), o, x[u]);
    PhiloxKey key = {};
    if (DROP) key = philox_key(p.dropout);
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        const int64_t i = i0 + u * rows;
        if (i >= p.n) break;
        uint32_t kept = slot[u] >= 0 ? 0xff : 0;
        if (DROP) kept &= kept_columns(key, uint32_t(o), uint32_t(i), p.dropout.threshold);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[u][j] = kept >> j & 1 ? x[u][j] * p.factor : 0.0f;
        store_octet<E, OVB>(static_cast<E*>(p.out) + i * p.hd + 8 * o, p.hd - 8 * o, x[u]);
    }
}

struct LookupGrid {
    int64_t groups;
    int slices, rows;  // rows of a thread
    int group_rows;
};
LookupGrid lookup_grid(const LookupParams& p) {
    const int octets = (p.hd + 7) / 8, rows = kThreads / (octets < kThreads ? octets : kThreads);
    LookupGrid g{(p.n + rows - 1) / rows, (octets + kThreads - 1) / kThreads, 1, rows};
    // Several rows a thread where that leaves 1024 workgroups: with dropout 32768 x 1024 in 19.4 us, with
    // one row a thread 21.9; 131072 x 8192 in 613, with one 775. Fewer workgroups have one (65521 rows of
    // 100 4-bit columns: 8.8 us, with four 9.3). Rows that are not whole vectors would take one too
    // (32768 x 1001: 38.1 us, with one 22.5), and 8-bit ones (50.7, with one 41.4).
    if (g.groups * g.slices >= 4096) {
        g.rows = 4;
        g.groups = (g.groups + 3) / 4;
        g.group_rows = 4 * rows;
    }
    return g;
}

// Rows past what a grid holds along one axis, 2^32 threads, are a launch of their own.
constexpr int64_t kMostGroups = 0xffffffffLL / kThreads;
template <int KIND, int VB, typename E, int OVB, bool DROP> void run(const LookupParams& call, hipStream_t stream) {
    const LookupGrid g = lookup_grid(call);
    LookupParams p = call;
    for (int64_t at = 0; at < g.groups; at += kMostGroups) {
        const dim3 grid{unsigned(g.groups - at < kMostGroups ? g.groups - at : kMostGroups), unsigned(g.slices)}, block{kThreads};
        p.first = at * g.group_rows;
        if (g.rows == 4) hipLaunchKernelGGL((lookup_kernel<KIND, VB, E, OVB, DROP, 4>), grid, block, 0, stream, p);
        else hipLaunchKernelGGL((lookup_kernel<KIND, VB, E, OVB, DROP, 1>), grid, block, 0, stream, p);
    }
}

template <int KIND, int VB, typename E, int OVB> void run_drop(const LookupParams& p, hipStream_t stream) {
    if (p.dropout.threshold != 0) run<KIND, VB, E, OVB, true>(p, stream);
    else run<KIND, VB, E, OVB, false>(p, stream);
}
template <int KIND, int VB> void run_out(const LookupParams& p, bool out_bf16, hipStream_t stream) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.out) | uintptr_t(p.hd) * (out_bf16 ? 2 : 4);
    if (out_bf16 && at % 16 == 0) run_drop<KIND, VB, uint16_t, 16>(p, stream);
    else if (out_bf16) run_drop<KIND, VB, uint16_t, 2>(p, stream);
    else if (at % 16 == 0) run_drop<KIND, VB, float, 16>(p, stream);
    else run_drop<KIND, VB, float, 4>(p, stream);
}

}  // namespace

int64_t lookup_groups(const LookupParams& p) { return lookup_grid(p).groups; }

hipError_t launch_lookup(const LookupParams& p, int bank_dtype, bool out_bf16, hipStream_t stream) {
    const bool vec = (reinterpret_cast<uintptr_t>(p.bank) | uintptr_t(p.row_bytes)) % 16 == 0;
    if (bank_dtype == SDM_MX8) run_out<SDM_MX8, 16>(p, out_bf16, stream);
    else if (bank_dtype == SDM_MX4) run_out<SDM_MX4, 16>(p, out_bf16, stream);
    else if (bank_dtype == SDM_BF16 && vec) run_out<SDM_BF16, 16>(p, out_bf16, stream);
    else if (bank_dtype == SDM_BF16) run_out<SDM_BF16, 2>(p, out_bf16, stream);
    else if (vec) run_out<SDM_F32, 16>(p, out_bf16, stream);
    else run_out<SDM_F32, 4>(p, out_bf16, stream);
    return hipGetLastError();
}

}  // namespace sdm
