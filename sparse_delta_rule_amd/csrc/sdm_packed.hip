// Packed banks (include/sdm_memory.h): sdm_bank_pack, sdm_gather_packed and
// sdm_gather_weight_grad.

#include "../../include/sdm_memory.h"
#include "sdm_kernels.h"
#include "sdm_memory.h"
#include "sdm_rows.h"

namespace sdm {

namespace {

constexpr int kThreads = 256;

// Lane i's value of the lane that `ctrl` names within its row of 16 lanes.
template <int ctrl> __device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), ctrl, 0xf, 0xf, true));
}
template <int ctrl> __device__ __forceinline__ float dpp(float v) { return __uint_as_float(dpp<ctrl>(__float_as_uint(v))); }
constexpr int kXor1 = 0xb1, kXor2 = 0x4e;               // quad_perm [1,0,3,2] and [2,3,0,1]
constexpr int kHalfMirror = 0x141, kMirror = 0x140;     // lane i of 8, of 16 <- lane 7 - i, 15 - i

// ------------------------------------------------------------------ pack

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;

// The largest |x| (as bits) of four lanes' octets: of a block.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
    m = max(m, dpp<kXor1>(m));
    return max(m, dpp<kXor2>(m));
}

// A thread takes eight columns of a row, four neighbouring lanes a block of 32;
// a row's threads are neighbours. The scale comes from the largest magnitude's own
// bits, and the conversions divide by it and round to nearest even, exactly. Bound by
// its memory traffic: 1048576 rows of 100 float32 columns to 4 bits in 87 us, 5.5 TB/s
// of bytes read and written (a large copy: 6.2); 262144 rows of 256 bytes to scattered
// slots in 21 us, 4.9 TB/s.
template <typename E, int VB, bool MX4>
__global__ __launch_bounds__(kThreads) void pack_kernel(PackParams p) {
    const int blocks = (p.hd + SDM_PACK_BLOCK - 1) / SDM_PACK_BLOCK;
    const int per_row = min(4 * blocks, kThreads);  // threads of a row
    const int rows = kThreads / per_row;            // rows of a workgroup
    const int r = int(threadIdx.x) / per_row, o0 = int(threadIdx.x) % per_row;
    if (r >= rows) return;
    const int64_t stride = int64_t(gridDim.x) * rows;
    for (int64_t i = int64_t(blockIdx.x) * rows + r; i < p.n; i += stride) {
        const int64_t src = p.row_idx != nullptr ? slot_at(p.row_idx, i, p.idx64 ? 8 : 4) : i;
        const int64_t dst = p.slots != nullptr ? slot_at(p.slots, i, p.idx64 ? 8 : 4) : i;
        if (src < 0 || src >= p.num_rows || dst < 0 || dst >= p.num_slots) continue;
        const E* row = static_cast<const E*>(p.rows) + src * p.hd;
        uint8_t* codes = p.codes + dst * p.row_bytes;
        uint8_t* scales = p.scales + dst * p.scale_bytes;
        for (int o = o0; o < 4 * blocks; o += per_row) {
            float x[8];
            load_octet<E, VB>(row + 8 * o, p.hd - 8 * o, x);
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, abs_bits(x[j]));
            m = block_max(m);
            uint32_t bad = 0;  // bit j: element j is not finite
            if (m >= kInfBits) {
                m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (abs_bits(x[j]) >= kInfBits) {
                        bad |= 1u << j;
                        x[j] = 0;
                    }
                    m = max(m, abs_bits(x[j]));
                }
                m = block_max(m);
            }
            // The least e with m <= 448 2^e (6 2^e), as e + 127, from m's own exponent.
            uint32_t scale = MX4 ? (m >> 23) + ((m & 0x7fffffu) > 0x400000u) : (m >> 23) + ((m & 0x7fffffu) > 0x600000u);
            constexpr uint32_t kTop = MX4 ? 2 : 8;
            scale = scale > kTop ? scale - kTop : 0;
            const float s = __uint_as_float(scale << 23);  // the conversions read the exponent field alone
            if constexpr (MX4) {
                uint32_t any = bad;
                any |= dpp<kXor1>(any);
                any |= dpp<kXor2>(any);
                uint32_t c = 0;
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], s, 0);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], s, 2);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], s, 3);
                if (any != 0) {
                    c = 0;
                    scale = 255;
                }
                if (4 * o < p.row_bytes) *reinterpret_cast<uint32_t*>(codes + 4 * o) = c;
            } else {
                typedef short Short2 __attribute__((ext_vector_type(2)));
                uint32_t c[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    Short2 v = {0, 0};
                    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, x[4 * h], x[4 * h + 1], s, false);
                    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, x[4 * h + 2], x[4 * h + 3], s, true);
                    __builtin_memcpy(&c[h], &v, 4);
                }
                if (bad != 0) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (bad >> j & 1) c[j / 4] |= 0x7fu << (8 * (j % 4));
                }
                if (8 * o < p.row_bytes) *reinterpret_cast<uint2*>(codes + 8 * o) = make_uint2(c[0], c[1]);
            }
            if (o % 4 == 0) {
                scales[o / 4] = uint8_t(scale);
                if (o / 4 == blocks - 1)
                    for (int b = blocks; b < p.scale_bytes; ++b) scales[b] = 0;
            }
        }
    }
}

// ------------------------------------------------------------------ gather

__device__ __forceinline__ bool is_live(const MemoryGatherParams& p, int64_t t) {
    const int64_t c = t / p.chunk;
    const int64_t limit = p.chunk_valid != nullptr ? int64_t(p.chunk_valid[c]) : p.valid;
    return t - c * p.chunk < limit;
}

constexpr int kFlight = 8;  // rows of a pair whose loads are in flight together

// What a pair (token, operand) needs of an entry, put into LDS by the pair's own
// lanes, kStage entries a lane: where its row begins, its weight, and the scales of
// a row of at most four blocks. So a lane's slots, weights and scales cost one load
// each for a whole row of lanes, and a row one LDS read.
struct Entry {
    int64_t row;      // where the row begins (FOUR, and a float bank); else its slot
    float w;
    uint32_t scales;  // FOUR: of the row's blocks
};
constexpr int kStage = 8;

struct Pair {
    int64_t t;
    int op, lane, lanes, width;
    Entry* entries;  // of this pair: kStage * lanes
};

__device__ __forceinline__ Pair this_pair(const MemoryGatherParams& p, int lanes, Entry* lds) {
    Pair r;
    const int in_block = int(threadIdx.x) / lanes;
    const int64_t q = int64_t(blockIdx.x) * (int(blockDim.x) / lanes) + in_block;
    r.t = p.operands == 2 ? q >> 1 : q;
    r.op = p.operands == 2 ? int(q & 1) : 0;
    r.lane = int(threadIdx.x) % lanes;
    r.lanes = lanes;
    r.width = r.op == 0 ? p.width[0] : p.width[1];
    r.entries = lds + in_block * (kStage * lanes);
    return r;
}

// Put the pair's entries from n0 up to `end` into LDS (at most kStage * lanes of them);
// returns how many. The lanes of a pair are in one wavefront.
template <bool WEIGHTS, bool FOUR, bool OFFSETS>
__device__ __forceinline__ int stage(const MemoryGatherParams& p, const Pair& r, int n0, int end) {
    const int count = min(end - n0, kStage * r.lanes);
    const void* idx = r.op == 0 ? p.idx[0] : p.idx[1];
    const void* w = r.op == 0 ? p.w[0] : p.w[1];
    const int64_t first = r.t * r.width + n0;
    int64_t slot[kStage] = {};
    float v[kStage] = {};
    uint32_t sc[kStage] = {};
    if (p.idx64) {
#pragma unroll
        for (int i = 0; i < kStage; ++i)
            slot[i] = static_cast<const int64_t*>(idx)[first + min(i * r.lanes + r.lane, count - 1)];
    } else {
#pragma unroll
        for (int i = 0; i < kStage; ++i)
            slot[i] = static_cast<const int32_t*>(idx)[first + min(i * r.lanes + r.lane, count - 1)];
    }
    if (WEIGHTS && p.w_bf16) {
#pragma unroll
        for (int i = 0; i < kStage; ++i)
            v[i] = widen(static_cast<const uint16_t*>(w)[first + min(i * r.lanes + r.lane, count - 1)]);
    } else if (WEIGHTS) {
#pragma unroll
        for (int i = 0; i < kStage; ++i)
            v[i] = static_cast<const float*>(w)[first + min(i * r.lanes + r.lane, count - 1)];
    }
    if (FOUR) {
#pragma unroll
        for (int i = 0; i < kStage; ++i) sc[i] = reinterpret_cast<const uint32_t*>(p.scales)[slot[i]];
    }
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
        const int n = i * r.lanes + r.lane;
        if (n < count) r.entries[n] = Entry{OFFSETS ? slot[i] * p.row_bytes : slot[i], v[i], sc[i]};
    }
    wave_lds_order();
    return count;
}

// The scale of a row's block as the conversions take it, from an entry's four bytes.
__device__ __forceinline__ float scale_of(uint32_t four, int block) {
    return __uint_as_float(four >> (8 * block) << 23 & 0x7f800000u);
}

// A pair takes `lanes` neighbouring lanes, N columns each. FOUR: a row has at most
// four blocks, whose scales come with the entry.
//
// Bound, over a large bank, by requests: a row's codes and its scales are a request
// each, 3.13 M rows of 128 columns (24466 tokens, 128 entries each) take 143 us over
// 2^24 slots, 43.8 G requests/s, and reads of random rows of up to 128 bytes alone reach
// 42-45 G/s on this card. Where the scales stay in the L2 caches the codes' requests are
// left (2^17 slots: 70 us), and in caches altogether (2^14 slots: 53 us) the VALU
// instructions, 37 for each row of a wavefront's eight.
template <bool MX4, bool FOUR, int N>
__global__ __launch_bounds__(kThreads) void gather_packed_kernel(MemoryGatherParams p, int lanes) {
    using C = Codes<MX4, N>;
    constexpr int kAhead = N == 16 ? kFlight : 2 * kFlight;  // rows in flight
    extern __shared__ Entry lds[];
    const Pair r = this_pair(p, lanes, lds);
    if (r.t >= p.tokens) return;
    const int c0 = N * (int(blockIdx.y) * lanes + r.lane);
    const int block = c0 / SDM_PACK_BLOCK;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    if (is_live(p, r.t)) {
        // A lane past the row's end reads its last columns.
        const int vec = min(c0 / N, (p.hd - 1) / N);
        const char* codes = static_cast<const char*>(p.bank) + vec * C::kBytes;
        const uint8_t* scales = p.scales + min(block, (p.hd - 1) / SDM_PACK_BLOCK);
        for (int s0 = 0; s0 < r.width; s0 += kStage * lanes) {
            const int count = stage<true, FOUR, FOUR>(p, r, s0, r.width);
            for (int n0 = 0; n0 < count; n0 += kAhead) {
                typename C::Raw raw[kAhead];
                Entry e[kAhead];
                float s[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) e[u] = r.entries[min(n0 + u, count - 1)];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) raw[u] = *reinterpret_cast<const typename C::Raw*>(codes + e[u].row * (FOUR ? 1 : p.row_bytes));
                if constexpr (!FOUR) {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u)
                        s[u] = __uint_as_float(uint32_t(scales[e[u].row * p.scale_bytes]) << 23);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (n0 + u < count) {
                        float x[N];
                        C::values(raw[u], FOUR ? scale_of(e[u].scales, block) : s[u], x);
#pragma unroll
                        for (int i = 0; i < N; ++i) acc[i] = fmaf(e[u].w, x[i], acc[i]);
                    }
                }
            }
        }
    }
    if (c0 >= p.hd) return;
    float* out = (r.op == 0 ? p.out[0] : p.out[1]) + r.t * p.hd + c0;
    if (c0 + N <= p.hd && p.out_vec) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            reinterpret_cast<float4*>(out)[i] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c0 + i < p.hd) out[i] = acc[i];
    }
}

// ------------------------------------------------------------------ weight gradient

// A row's vector of a bank: of kN columns, read by one lane.
template <int KIND, int VB> struct BankVec;
template <int VB> struct BankVec<SDM_F32, VB> {
    using Raw = typename RawVec<VB>::T;
    static constexpr int kN = VB / 4;
    static constexpr bool kPacked = false;
    static __device__ __forceinline__ void values(const Raw& v, float, float (&x)[kN]) { __builtin_memcpy(x, &v, VB); }
};
template <int VB> struct BankVec<SDM_BF16, VB> {
    using Raw = typename RawVec<VB>::T;
    static constexpr int kN = VB / 2;
    static constexpr bool kPacked = false;
    static __device__ __forceinline__ void values(const Raw& v, float, float (&x)[kN]) {
        uint16_t e[kN];
        __builtin_memcpy(e, &v, VB);
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = widen(e[i]);
    }
};
template <> struct BankVec<SDM_MX8, 16> : Codes<false, 16> {
    static constexpr int kN = 16;
    static constexpr bool kPacked = true;
};
template <> struct BankVec<SDM_MX4, 8> : Codes<true, 16> {
    static constexpr int kN = 16;
    static constexpr bool kPacked = true;
};

// Sum over the `lanes` (a power of two) neighbouring lanes of a pair.
__device__ __forceinline__ float lane_sum(float v, int lanes) {
    if (lanes > 1) v += dpp<kXor1>(v);
    if (lanes > 2) v += dpp<kXor2>(v);
    if (lanes > 4) v += dpp<kHalfMirror>(v);
    if (lanes > 8) v += dpp<kMirror>(v);
    if (lanes > 16) v += __shfl_xor(v, 16);
    if (lanes > 32) v += __shfl_xor(v, 32);
    return v;
}

// A pair takes `lanes` neighbouring lanes, a vector of the row each (or several in
// turn, rows of more than 64 vectors), for the entries of one segment of the width.
// WHOLE: a lane has one vector at most, so its
// part of dout stays in registers. Bound as the gather is: 1.57 M rows of 128 8-bit
// columns over 2^24 slots in 74 us, 42.3 G requests/s.
template <int KIND, int VB, bool FOUR, bool WHOLE>
__global__ __launch_bounds__(kThreads) void weight_grad_kernel(MemoryGatherParams p, int lanes, int per_segment) {
    using V = BankVec<KIND, VB>;
    constexpr bool kOffsets = FOUR || !V::kPacked;
    extern __shared__ Entry lds[];
    const Pair r = this_pair(p, lanes, lds);
    if (r.t >= p.tokens) return;
    const int begin = int(blockIdx.y) * per_segment, end = min(begin + per_segment, r.width);
    const bool live = is_live(p, r.t);
    const int vecs = (p.hd + V::kN - 1) / V::kN;
    const char* bank = static_cast<const char*>(p.bank);
    const float* dout = (r.op == 0 ? p.dout[0] : p.dout[1]) + r.t * p.hd;
    void* dw = r.op == 0 ? p.dw[0] : p.dw[1];
    float g[V::kN] = {};
    auto load_dout = [&](int v) {
        const int c0 = v * V::kN;
#pragma unroll
        for (int i = 0; i < V::kN; ++i) g[i] = c0 + i < p.hd ? dout[c0 + i] : 0.0f;
    };
    if (WHOLE && live && r.lane < vecs) load_dout(r.lane);
    for (int s0 = begin; s0 < end; s0 += kStage * lanes) {
        const int count = live ? stage<false, FOUR, kOffsets>(p, r, s0, end) : min(end - s0, kStage * lanes);
        for (int n0 = 0; n0 < count; n0 += kFlight) {
            float sum[kFlight];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) sum[u] = 0.0f;
            if (live) {
                Entry e[kFlight];
#pragma unroll
                for (int u = 0; u < kFlight; ++u) e[u] = r.entries[min(n0 + u, count - 1)];
                for (int v = r.lane; v < (WHOLE ? lanes : vecs); v += lanes) {
                    const int c0 = v * V::kN;
                    const int at = WHOLE ? min(v, vecs - 1) : v;  // a lane past the row's end has only zeros in g
                    if (!WHOLE) load_dout(v);
                    typename V::Raw raw[kFlight];
                    float s[kFlight];
#pragma unroll
                    for (int u = 0; u < kFlight; ++u)
                        raw[u] = *reinterpret_cast<const typename V::Raw*>(bank + e[u].row * (kOffsets ? 1 : p.row_bytes) + int64_t(at) * VB);
                    if constexpr (V::kPacked && !FOUR) {
#pragma unroll
                        for (int u = 0; u < kFlight; ++u)
                            s[u] = __uint_as_float(uint32_t(p.scales[e[u].row * p.scale_bytes + at * V::kN / SDM_PACK_BLOCK]) << 23);
                    }
#pragma unroll
                    for (int u = 0; u < kFlight; ++u) {
                        float x[V::kN];
                        V::values(raw[u], FOUR ? scale_of(e[u].scales, c0 / SDM_PACK_BLOCK) : s[u], x);
                        float part = 0;
                        if (c0 + V::kN <= p.hd) {
#pragma unroll
                            for (int i = 0; i < V::kN; ++i) part = fmaf(g[i], x[i], part);
                        } else {  // columns past the row's end are not looked at: they may hold anything
#pragma unroll
                            for (int i = 0; i < V::kN; ++i)
                                if (c0 + i < p.hd) part = fmaf(g[i], x[i], part);
                        }
                        sum[u] += part;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kFlight; ++u) sum[u] = lane_sum(sum[u], lanes);
            // Lane u stores entry u, of fewer lanes each its share.
            for (int at = r.lane; at < kFlight; at += lanes) {
                float total = sum[0];
#pragma unroll
                for (int u = 1; u < kFlight; ++u) total = at == u ? sum[u] : total;
                if (n0 + at < count) {
                    const int64_t n = r.t * r.width + s0 + n0 + at;
                    if (p.w_bf16) static_cast<uint16_t*>(dw)[n] = to_bf16_rne(total);
                    else static_cast<float*>(dw)[n] = total;
                }
            }
        }
    }
}

int pow2_lanes(int64_t vecs) {
    int lanes = 1;
    while (lanes < vecs && lanes < 64) lanes *= 2;
    return lanes;
}

// Wavefronts that a launch wants at least: 4 on each of the 256 CUs.
constexpr int64_t kManyWaves = 1024;

struct PairGrid {
    dim3 grid, block;
    size_t lds;
};
// Workgroups of one wavefront where there are few, so that they spread over the card.
PairGrid pair_grid(const MemoryGatherParams& p, int lanes, int rows_of_grid) {
    const int64_t waves = (p.tokens * p.operands * lanes + 63) / 64 * rows_of_grid;
    const int threads = waves < 2 * kManyWaves ? 64 : kThreads, per = threads / lanes;
    return {dim3(unsigned((p.tokens * p.operands + per - 1) / per), unsigned(rows_of_grid)), dim3(unsigned(threads)),
            size_t(threads) * kStage * sizeof(Entry)};
}

template <int KIND, int VB, bool FOUR> void run_weight_grad(const MemoryGatherParams& p, hipStream_t stream) {
    using V = BankVec<KIND, VB>;
    const int vecs = (p.hd + V::kN - 1) / V::kN, lanes = pow2_lanes(vecs);
    // Few pairs: the entries of each are split over wavefronts, kFlight at least a piece.
    const int widest = p.operands == 2 && p.width[1] > p.width[0] ? p.width[1] : p.width[0];
    const int64_t waves = (p.tokens * p.operands * lanes + 63) / 64;
    int segments = (widest + kFlight - 1) / kFlight;
    if (waves * segments > kManyWaves) segments = waves >= kManyWaves ? 1 : int(kManyWaves / waves);
    const int per_segment = ((widest + segments - 1) / segments + kFlight - 1) / kFlight * kFlight;
    const PairGrid g = pair_grid(p, lanes, (widest + per_segment - 1) / per_segment);
    if (vecs <= lanes)
        hipLaunchKernelGGL((weight_grad_kernel<KIND, VB, FOUR, true>), g.grid, g.block, g.lds, stream, p, lanes, per_segment);
    else
        hipLaunchKernelGGL((weight_grad_kernel<KIND, VB, FOUR, false>), g.grid, g.block, g.lds, stream, p, lanes, per_segment);
}

template <int N> void run_gather_packed(const MemoryGatherParams& p, bool mx4, hipStream_t stream) {
    const int lanes = pow2_lanes((p.hd + N - 1) / N);
    const PairGrid g = pair_grid(p, lanes, (p.hd + N * lanes - 1) / (N * lanes));
    const bool four = p.scale_bytes == 4;
    if (mx4 && four) hipLaunchKernelGGL((gather_packed_kernel<true, true, N>), g.grid, g.block, g.lds, stream, p, lanes);
    else if (mx4) hipLaunchKernelGGL((gather_packed_kernel<true, false, N>), g.grid, g.block, g.lds, stream, p, lanes);
    else if (four) hipLaunchKernelGGL((gather_packed_kernel<false, true, N>), g.grid, g.block, g.lds, stream, p, lanes);
    else hipLaunchKernelGGL((gather_packed_kernel<false, false, N>), g.grid, g.block, g.lds, stream, p, lanes);
}

template <typename E, int VB> void run_pack(const PackParams& p, bool mx4, hipStream_t stream) {
    const int blocks = (p.hd + SDM_PACK_BLOCK - 1) / SDM_PACK_BLOCK;
    const int rows = kThreads / (4 * blocks < kThreads ? 4 * blocks : kThreads);
    int64_t grid = (p.n + rows - 1) / rows;
    if (grid > (1 << 20)) grid = 1 << 20;
    if (mx4) hipLaunchKernelGGL((pack_kernel<E, VB, true>), dim3(unsigned(grid)), dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL((pack_kernel<E, VB, false>), dim3(unsigned(grid)), dim3(kThreads), 0, stream, p);
}

}  // namespace

hipError_t launch_pack(const PackParams& p, bool bf16, bool mx4, hipStream_t stream) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.rows) | uintptr_t(p.hd) * (bf16 ? 2 : 4);
    const int vb = at % 16 == 0 ? 16 : at % 8 == 0 ? 8 : at % 4 == 0 ? 4 : 2;
    if (bf16) {
        if (vb == 16) run_pack<uint16_t, 16>(p, mx4, stream);
        else if (vb == 8) run_pack<uint16_t, 8>(p, mx4, stream);
        else if (vb == 4) run_pack<uint16_t, 4>(p, mx4, stream);
        else run_pack<uint16_t, 2>(p, mx4, stream);
    } else {
        if (vb == 16) run_pack<float, 16>(p, mx4, stream);
        else if (vb == 8) run_pack<float, 8>(p, mx4, stream);
        else run_pack<float, 4>(p, mx4, stream);
    }
    return hipGetLastError();
}

hipError_t launch_gather_packed(const MemoryGatherParams& p, bool mx4, hipStream_t stream) {
    // Few pairs: 4 columns a lane instead of 16, four times the wavefronts and twice the
    // rows in flight (an element's chain of additions is one lane's in either).
    const int64_t waves = p.tokens * p.operands * ((p.hd + 15) / 16) / 64;
    if (waves < kManyWaves && p.hd <= 4096) run_gather_packed<4>(p, mx4, stream);
    else run_gather_packed<16>(p, mx4, stream);
    return hipGetLastError();
}

hipError_t launch_weight_grad(const MemoryGatherParams& p, int bank_dtype, hipStream_t stream) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.bank) | uintptr_t(p.row_bytes);
    const int vb = at % 16 == 0 ? 16 : at % 8 == 0 ? 8 : at % 4 == 0 ? 4 : 2;
    const bool four = p.scale_bytes == 4;
    if (bank_dtype == SDM_MX8 && four) run_weight_grad<SDM_MX8, 16, true>(p, stream);
    else if (bank_dtype == SDM_MX8) run_weight_grad<SDM_MX8, 16, false>(p, stream);
    else if (bank_dtype == SDM_MX4 && four) run_weight_grad<SDM_MX4, 8, true>(p, stream);
    else if (bank_dtype == SDM_MX4) run_weight_grad<SDM_MX4, 8, false>(p, stream);
    else if (bank_dtype == SDM_F32 && vb == 16) run_weight_grad<SDM_F32, 16, false>(p, stream);
    else if (bank_dtype == SDM_F32 && vb == 8) run_weight_grad<SDM_F32, 8, false>(p, stream);
    else if (bank_dtype == SDM_F32) run_weight_grad<SDM_F32, 4, false>(p, stream);
    else if (vb == 16) run_weight_grad<SDM_BF16, 16, false>(p, stream);
    else if (vb == 8) run_weight_grad<SDM_BF16, 8, false>(p, stream);
    else if (vb == 4) run_weight_grad<SDM_BF16, 4, false>(p, stream);
    else run_weight_grad<SDM_BF16, 2, false>(p, stream);
    return hipGetLastError();
}

}  // namespace sdm
