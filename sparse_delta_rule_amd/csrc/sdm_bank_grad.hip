// Gradients to a bank (include/sdm_train.h): sdm_lookup_grad and sdm_gather_bank_grad.
//
// An entry is a named row: a lookup's row, or a (token, place) of a gather's operand. The
// entries that count are sorted by slot, equal slots in the order of the entries (a stable
// radix sort), and each slot's terms are then added in that order: no float atomics, so
// the same inputs give the same bits.

#include "sdm_dropout.h"
#include "sdm_memory.h"
#include "sdm_rows.h"

namespace sdm {

namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ entries

__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor& d) {
    return uint32_t(uint64_t(n) * d.mul >> d.shift);
}

// Where an entry's token is: its operand and number.
struct Place {
    uint32_t op, token, at;  // at: the entry's number in its operand
};
template <bool LOOKUP> __device__ __forceinline__ Place place_of(const BankGradParams& p, uint32_t e) {
    if (LOOKUP) return {0, e, e};
    const uint32_t op = e >= p.first_entries, at = op ? e - p.first_entries : e;
    const Divisor d = op ? p.by_width[1] : p.by_width[0];
    return {op, divide(at, d), at};
}

constexpr uint32_t kNone = 0xffffffffu;
// An entry's slot, or kNone where it does not count. All of its loads are made whatever the others
// bring, so that those of many entries are in flight together.
template <bool LOOKUP> __device__ __forceinline__ uint32_t slot_of(const BankGradParams& p, uint32_t e) {
    const Place r = place_of<LOOKUP>(p, e);
    const int64_t s = slot_at(r.op ? p.idx[1] : p.idx[0], r.at, p.idx64 ? 8 : 4);
    bool counts = uint64_t(s) < uint64_t(p.num_slots);
    if (!LOOKUP) {
        const uint32_t c = divide(r.token, p.by_chunk);
        int32_t limit = int32_t(p.valid);
        if (p.chunk_valid != nullptr) limit = p.chunk_valid[c];
        counts &= int32_t(r.token - c * p.chunk) < limit;
    }
    return counts ? uint32_t(s) : kNone;
}

// ------------------------------------------------------------------ sort

constexpr int kMaxBits = 9;  // of a digit
constexpr int kMaxDigits = 1 << kMaxBits;

__device__ __forceinline__ uint32_t digit_of(uint32_t slot, int pass, int bits) {
    return slot >> (pass * bits) & ((1u << bits) - 1);
}

// Among the lanes of a wavefront that hold a digit: those with this lane's.
__device__ __forceinline__ uint64_t lanes_with(uint32_t digit, bool has, int bits) {
    uint64_t same = __ballot(has);
    for (int b = 0; b < bits; ++b) {
        const bool one = digit >> b & 1;
        const uint64_t ones = __ballot(one);
        same &= one ? ones : ~ones;
    }
    return same;
}
__device__ __forceinline__ uint32_t lanes_below(uint64_t lanes) {
    return __builtin_amdgcn_mbcnt_hi(uint32_t(lanes >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(lanes), 0));
}

// Each of a wavefront's ITEMS entries (64 neighbours at a time): how many of its earlier ones have
// the same digit. count: the wavefront's own, of each digit, 0 before and its sum after.
template <int ITEMS>
__device__ __forceinline__ void rank_items(const uint32_t (&slot)[ITEMS], int pass, int bits, uint32_t* count,
                                           uint32_t (&rank)[ITEMS]) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const bool has = slot[i] != kNone;
        const uint32_t digit = digit_of(slot[i], pass, bits);
        const uint64_t same = lanes_with(digit, has, bits);
        const uint32_t below = lanes_below(same);
        rank[i] = 0;
        if (has) {
            const uint32_t before = count[digit];
            rank[i] = before + below;
            wave_lds_order();
            if (below == 0) count[digit] = before + uint32_t(__popcll(same));
        }
        wave_lds_order();
    }
}

// Sums of the values of lower threads, over a workgroup of THREADS; *all: of all threads.
template <int THREADS> __device__ __forceinline__ uint32_t sum_below(uint32_t v, uint32_t* lds, uint32_t* all) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    uint32_t sum = v;
    for (int n = 1; n < 64; n *= 2) {
        const uint32_t o = __shfl_up(sum, n);
        if (lane >= n) sum += o;
    }
    if (lane == 63) lds[wave] = sum;
    __syncthreads();
    uint32_t below = sum - v, total = 0;
    for (int w = 0; w < THREADS / 64; ++w) {
        below += w < wave ? lds[w] : 0;
        total += lds[w];
    }
    *all = total;
    return below;
}

// Few entries: one workgroup sorts them in LDS, all passes in one launch.
constexpr int kOneThreads = 1024;
constexpr int kOneWaves = kOneThreads / 64;
constexpr int kOneItems = 8;
constexpr uint32_t kOneEntries = kOneThreads * kOneItems;

template <bool LOOKUP, int ITEMS> __global__ __launch_bounds__(kOneThreads) void sort_one_kernel(BankGradParams p) {
    __shared__ Record records[kOneThreads * ITEMS];
    __shared__ uint32_t count[kOneWaves][kMaxDigits];
    __shared__ uint32_t scratch[kOneWaves];
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, digits = 1 << p.bits;
    uint32_t slot[ITEMS], entry[ITEMS], rank[ITEMS], n = p.entries;
    const uint32_t first = wave * (64 * ITEMS) + lane;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        entry[i] = first + i * 64;
        slot[i] = slot_of<LOOKUP>(p, min(entry[i], n - 1));
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) slot[i] = entry[i] < n ? slot[i] : kNone;
    for (int pass = 0; pass < p.passes; ++pass) {
        for (int i = tid; i < kOneWaves * digits; i += kOneThreads) count[i / digits][i % digits] = 0;
        __syncthreads();
        rank_items<ITEMS>(slot, pass, p.bits, count[wave], rank);
        __syncthreads();
        uint32_t all = 0;
        if (tid < digits)
            for (int w = 0; w < kOneWaves; ++w) all += count[w][tid];
        uint32_t base = sum_below<kOneThreads>(all, scratch, &n);
        if (tid < digits) {
            for (int w = 0; w < kOneWaves; ++w) {
                const uint32_t v = count[w][tid];
                count[w][tid] = base;
                base += v;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (slot[i] != kNone) records[count[wave][digit_of(slot[i], pass, p.bits)] + rank[i]] = Record{slot[i], entry[i]};
        __syncthreads();
        if (pass == p.passes - 1) break;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const Record r = records[min(first + i * 64, uint32_t(kOneThreads * ITEMS - 1))];
            slot[i] = first + i * 64 < n ? r.slot : kNone;
            entry[i] = r.entry;
        }
    }
    Record* to = p.records[(p.passes - 1) & 1];
    for (uint32_t i = tid; i < n; i += kOneThreads) to[i] = records[i];
    if (tid == 0) *p.n = n;
}

constexpr int kWaves = kThreads / 64;

// The slots of a thread's entries of a tile, `stride` apart; kNone past the end.
template <bool FIRST, bool LOOKUP, int ITEMS>
__device__ __forceinline__ void load_slots(const BankGradParams& p, int pass, uint32_t first, uint32_t stride, uint32_t n,
                                           uint32_t (&slot)[ITEMS], uint32_t (&entry)[ITEMS]) {
    if (n == 0) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) slot[i] = kNone, entry[i] = 0;
        return;
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        entry[i] = min(first + i * stride, n - 1);
        if (FIRST) {
            slot[i] = slot_of<LOOKUP>(p, entry[i]);
        } else {
            const Record r = p.records[(pass - 1) & 1][entry[i]];
            slot[i] = r.slot;
            entry[i] = r.entry;
        }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) slot[i] = first + i * stride < n ? slot[i] : kNone;
}

__device__ __forceinline__ uint32_t* hist_of(const BankGradParams& p, int pass, uint32_t tile) {
    return p.hist + (int64_t(pass) * p.tiles + tile) * (1 << p.bits);
}

// How many entries of each tile have each digit.
template <bool FIRST, bool LOOKUP, int ITEMS>
__global__ __launch_bounds__(kThreads) void sort_count_kernel(BankGradParams p, int pass) {
    __shared__ uint32_t count[kMaxDigits];
    const int digits = 1 << p.bits;
    for (int d = threadIdx.x; d < digits; d += kThreads) count[d] = 0;
    __syncthreads();
    const uint32_t n = FIRST ? p.entries : *p.n;
    uint32_t slot[ITEMS], entry[ITEMS];
    load_slots<FIRST, LOOKUP, ITEMS>(p, pass, blockIdx.x * uint32_t(kThreads * ITEMS) + threadIdx.x, kThreads, n, slot, entry);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        if (slot[i] != kNone) atomicAdd(&count[digit_of(slot[i], pass, p.bits)], 1u);
    __syncthreads();
    uint32_t* hist = hist_of(p, pass, blockIdx.x);
    for (int d = threadIdx.x; d < digits; d += kThreads) hist[d] = count[d];
}

// For each digit, the entries of lower tiles that have it, in place, and of all of them.
constexpr int kScanDigits = 32, kScanParts = 32;
__global__ __launch_bounds__(kScanDigits * kScanParts) void sort_scan_kernel(BankGradParams p, int pass) {
    __shared__ uint32_t sums[kScanParts][kScanDigits];
    const int d = threadIdx.x % kScanDigits, part = threadIdx.x / kScanDigits;
    const int digits = 1 << p.bits, digit = min(int(blockIdx.x) * kScanDigits + d, digits - 1);
    uint32_t* hist = hist_of(p, pass, 0) + digit;
    const int64_t each = (int64_t(p.tiles) + kScanParts - 1) / kScanParts;
    const int64_t begin = min(part * each, int64_t(p.tiles)), end = min(begin + each, int64_t(p.tiles));
    uint32_t sum = 0;
#pragma unroll 8
    for (int64_t i = begin; i < end; ++i) sum += hist[i * digits];
    sums[part][d] = sum;
    __syncthreads();
    if (int(blockIdx.x) * kScanDigits + d >= digits) return;
    uint32_t before = 0, all = 0;
    for (int i = 0; i < kScanParts; ++i) {
        before += i < part ? sums[i][d] : 0;
        all += sums[i][d];
    }
#pragma unroll 8
    for (int64_t i = begin; i < end; ++i) {
        const uint32_t v = hist[i * digits];
        hist[i * digits] = before;
        before += v;
    }
    if (part == 0) p.total[pass * digits + digit] = all;
}

// Puts each entry of a tile in its place of the order by this pass's digit. A wavefront takes
// 64 neighbours at a time; the lanes of the same digit find one another by ballots.
template <bool FIRST, bool LOOKUP, int ITEMS>
__global__ __launch_bounds__(kThreads) void sort_place_kernel(BankGradParams p, int pass) {
    __shared__ uint32_t count[kWaves][kMaxDigits];
    __shared__ uint32_t scratch[kWaves];
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, digits = 1 << p.bits;
    const uint32_t n = FIRST ? p.entries : *p.n;
    uint32_t slot[ITEMS], entry[ITEMS], rank[ITEMS];
    load_slots<FIRST, LOOKUP, ITEMS>(p, pass, blockIdx.x * uint32_t(kThreads * ITEMS) + wave * (64 * ITEMS) + lane, 64, n, slot,
                                     entry);
    // Where each digit's entries of this tile begin: a thread takes digits 2 tid and 2 tid + 1.
    uint32_t total[2], before[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int d = 2 * tid + j;
        total[j] = d < digits ? p.total[pass * digits + d] : 0;
        before[j] = d < digits ? hist_of(p, pass, blockIdx.x)[d] : 0;
        for (int w = 0; w < kWaves; ++w) count[w][d] = 0;
    }
    uint32_t all;
    const uint32_t below = sum_below<kThreads>(total[0] + total[1], scratch, &all);
    if (FIRST && blockIdx.x == 0 && tid == 0) *p.n = all;
    rank_items<ITEMS>(slot, pass, p.bits, count[wave], rank);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t base = below + (j == 1 ? total[0] : 0) + before[j];
        for (int w = 0; w < kWaves; ++w) {
            const uint32_t v = count[w][2 * tid + j];
            count[w][2 * tid + j] = base;
            base += v;
        }
    }
    __syncthreads();
    Record* to = p.records[pass & 1];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        if (slot[i] != kNone) to[count[wave][digit_of(slot[i], pass, p.bits)] + rank[i]] = Record{slot[i], entry[i]};
}

// ------------------------------------------------------------------ sums

// The sorted entries are cut into blocks, a lane group each; a workgroup takes neighbours. A run
// of equal slots that ends within `spill` entries past a block's end is taken by that block to
// its end, and the next begins behind it; of a longer one each block makes a partial sum, which
// join_kernel adds up. cont: block b's first run began in an earlier block and is not that
// block's alone. `at`: the slot of a sorted entry.
template <typename F> __device__ __forceinline__ bool cont(const BankGradParams& p, F at, uint32_t n, uint64_t begin) {
    return begin > 0 && begin + p.spill < n && at(begin - 1) == at(begin + p.spill);
}

// N neighbouring columns of a row.
template <typename E, int VB, int N> __device__ __forceinline__ void load_columns(const E* p, int left, float (&x)[N]) {
    constexpr int VEC = VB / int(sizeof(E));
    if (left >= N) {
        typename RawVec<VB>::T raw[N / VEC];
#pragma unroll
        for (int i = 0; i < N / VEC; ++i) raw[i] = reinterpret_cast<const typename RawVec<VB>::T*>(p)[i];
        E e[N];
        __builtin_memcpy(e, raw, sizeof e);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = widen(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = i < left ? widen(p[i]) : 0.0f;
    }
}
template <typename E, int VB, int N> __device__ __forceinline__ void store_columns(E* p, int left, const float (&x)[N]) {
    constexpr int VEC = VB / int(sizeof(E));
    if (left >= N) {
#pragma unroll
        for (int i = 0; i < N; i += VEC) {
            float v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = x[i + j];
            store_stream(reinterpret_cast<typename RawVec<VB>::T*>(p + i), Pack<E, VB>::of(v));
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) p[i] = narrow<E>(x[i]);
    }
}

template <typename E, int VB, int N>
__device__ __forceinline__ void finish(const BankGradParams& p, uint32_t slot, int c0, const float (&acc)[N]) {
    E* row = static_cast<E*>(p.dbank) + int64_t(slot) * p.hd + c0;
    float v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = acc[j] * p.factor;
    if (p.add) {
        float old[N];
        load_columns<E, VB, N>(row, p.hd - c0, old);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] += old[j];
    }
    store_columns<E, VB, N>(row, p.hd - c0, v);
}

constexpr int kMaxBlock = 64;
constexpr int kMaxSpill = 16;
constexpr int kMinLanes = 8;
constexpr int kFlight = 8;  // rows whose loads are in flight together

struct Term {
    uint32_t slot, token, op;
    float w;
};

template <typename D, int DVB, typename E, int VB, bool WEIGHTS, bool DROP>
__global__ __launch_bounds__(kThreads) void sum_kernel(BankGradParams p, int lanes, int slices) {
    constexpr int N = 16 / int(sizeof(D));  // columns of a lane
    constexpr int EVB = VB == 16 ? (N * int(sizeof(E)) < 16 ? N * int(sizeof(E)) : 16) : VB;
    extern __shared__ Term lds[];
    const int groups = kThreads / lanes, lane = int(threadIdx.x) % lanes, group = int(threadIdx.x) / lanes;
    const int c0 = (int(blockIdx.x % slices) * lanes + lane) * N;
    const int columns = (p.hd + 7) / 8 * 8;
    const uint64_t range = uint64_t(groups) * p.block, start = blockIdx.x / slices * range;
    const Record* records = p.records[(p.passes - 1) & 1];
    const uint32_t n = *p.n;
    if (start >= n) return;
    // terms[i]: entry start - 1 + i, so that the one before the range is there
    const Term* terms = lds;
    const int there = int(min(range + p.spill + 2, n - start + 1));
    for (int i = threadIdx.x; i < there; i += kThreads) {
        const Record r = records[start + i > 0 ? start + i - 1 : 0];
        const Place e = place_of<!WEIGHTS>(p, r.entry);
        Term t = {r.slot, e.token, e.op, 1.0f};
        if (WEIGHTS) t.w = value_at(e.op ? p.w[1] : p.w[0], e.at, p.w_bf16 ? 2 : 4);
        lds[i] = t;
    }
    __syncthreads();
    const uint32_t b = uint32_t(blockIdx.x / slices) * groups + group;
    const uint64_t begin = uint64_t(b) * p.block;
    if (begin >= n || c0 >= p.hd) return;
    auto slot_of_sorted = [&](uint64_t i) { return terms[int(i + 1 - start)].slot; };
    const bool from_before = cont(p, slot_of_sorted, n, begin), goes_on = cont(p, slot_of_sorted, n, begin + p.block);
    int at = int(begin + 1 - start), end = min(at + p.block, there);
    const uint32_t last = terms[end - 1].slot;
    if (begin > 0 && !from_before)
        for (const uint32_t before = terms[at - 1].slot; at < end && terms[at].slot == before;) ++at;
    if (!goes_on)
        while (end < there && terms[end].slot == last) ++end;
    PhiloxKey key = {};
    if (DROP) key = philox_key(p.dropout);
    float acc[N] = {};
    bool open = from_before;  // the run being added up began in an earlier block
    while (at < end) {
        const int count = min(end - at, kFlight);
        float x[kFlight][N];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const Term& t = terms[at + min(u, count - 1)];
            const D* row = static_cast<const D*>(t.op ? p.dout[1] : p.dout[0]) + int64_t(t.token) * p.hd;
            load_columns<D, DVB, N>(row + c0, p.hd - c0, x[u]);
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (u >= count) break;
            const Term t = terms[at + u];
            const uint32_t kept = DROP ? kept_columns(key, uint32_t(c0) / 8, t.token, p.dropout.threshold) >> (c0 & 7) : 0xff;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (WEIGHTS) acc[j] = fmaf(t.w, x[u][j], acc[j]);
                else acc[j] += kept >> j & 1 ? x[u][j] : 0.0f;
            }
            const bool is_last = at + u + 1 == end;
            if (is_last || terms[at + u + 1].slot != t.slot) {
                if (open || (is_last && goes_on)) {
                    float* to = (open ? p.first : p.last) + int64_t(b) * columns + c0;
#pragma unroll
                    for (int j = 0; j < N; j += 4)
                        *reinterpret_cast<float4*>(to + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
                } else {
                    finish<E, EVB, N>(p, t.slot, c0, acc);
                }
                open = false;
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] = 0.0f;
            }
        }
        at += count;
    }
}

// Runs over several blocks. A workgroup looks at kJoinBlocks blocks; the partial sums of each
// run that begins in one of them are added by its lane groups in turn, and theirs in order.
constexpr int kJoinThreads = 1024;
constexpr int kJoinBlocks = 64;

template <typename E, int VB> __global__ __launch_bounds__(kJoinThreads) void join_kernel(BankGradParams p, int lanes) {
    constexpr int N = 4;
    constexpr int EVB = VB == 16 ? N * int(sizeof(E)) : VB;
    __shared__ uint64_t begins;
    __shared__ float sums[kJoinThreads][N];
    const int tid = threadIdx.x, groups = kJoinThreads / lanes, lane = tid % lanes, group = tid / lanes;
    const int c0 = (int(blockIdx.y) * lanes + lane) * N;
    const int64_t columns = (p.hd + 7) / 8 * 8;
    const Record* records = p.records[(p.passes - 1) & 1];
    const uint32_t n = *p.n;
    const uint32_t b0 = blockIdx.x * uint32_t(kJoinBlocks);
    if (uint64_t(b0) * p.block >= n) return;
    auto at = [&](uint64_t i) { return records[i].slot; };
    if (tid < 64) {
        const uint64_t begin = uint64_t(b0 + tid) * p.block;
        bool is = cont(p, at, n, begin + p.block);
        if (is && begin > 0) is = at(begin - 1) != at(begin + p.block - 1);
        const uint64_t found = __ballot(is);
        if (tid == 0) begins = found;
    }
    __syncthreads();
    for (uint64_t left = begins; left != 0; left &= left - 1) {
        const uint32_t b = b0 + uint32_t(__ffsll(static_cast<unsigned long long>(left))) - 1;
        const uint32_t slot = at(uint64_t(b) * p.block + p.block - 1);
        // The blocks after b whose first run is this one.
        uint32_t more = 0, found;
        do {
            const uint64_t begin = (uint64_t(b) + 1 + more + tid) * p.block;
            const bool is = cont(p, at, n, begin) && at(begin) == slot;
            found = uint32_t(__syncthreads_count(is));
            more += found;
        } while (found == kJoinThreads);
        float acc[N] = {};
        if (c0 < p.hd) {
            if (group == 0) load_columns<float, 16, N>(p.last + b * columns + c0, N, acc);
#pragma unroll 8
            for (uint32_t c = group; c < more; c += groups) {
                float x[N];
                load_columns<float, 16, N>(p.first + (int64_t(b) + 1 + c) * columns + c0, N, x);
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += x[j];
            }
        }
        *reinterpret_cast<float4*>(sums[tid]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        __syncthreads();
        if (group == 0 && c0 < p.hd) {
            for (int g = 1; g < min(groups, int(min(more, uint32_t(kJoinThreads)))); ++g) {
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += sums[g * lanes + lane][j];
            }
            finish<E, EVB, N>(p, slot, c0, acc);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ rows that no entry names

constexpr int kZeroBytes = 65536;  // of a workgroup's rows
constexpr int kZeroRows = 1024;    // at most

__device__ __forceinline__ uint32_t lower_bound(const Record* records, uint32_t n, uint64_t slot) {
    uint32_t lo = 0, hi = n;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (records[mid].slot < slot) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

template <int VB> __global__ __launch_bounds__(kThreads) void zero_kernel(BankGradParams p, int rows, int64_t row_bytes) {
    __shared__ uint8_t named[kZeroRows];
    __shared__ uint32_t bounds[2];
    const Record* records = p.records[(p.passes - 1) & 1];
    const uint32_t n = p.entries > 0 ? *p.n : 0;
    const int64_t first = int64_t(blockIdx.x) * rows;
    const int count = int(min(int64_t(rows), int64_t(p.num_slots) - first));
    for (int i = threadIdx.x; i < count; i += kThreads) named[i] = 0;
    if (threadIdx.x < 2) bounds[threadIdx.x] = lower_bound(records, n, uint64_t(first) + (threadIdx.x == 0 ? 0 : count));
    __syncthreads();
    for (uint32_t i = bounds[0] + threadIdx.x; i < bounds[1]; i += kThreads) named[records[i].slot - uint32_t(first)] = 1;
    __syncthreads();
    const int per_row = int(row_bytes / VB);
    char* base = static_cast<char*>(p.dbank) + first * row_bytes;
    using T = typename RawVec<VB>::T;
    for (int64_t v = threadIdx.x; v < int64_t(count) * per_row; v += kThreads)
        if (!named[v / per_row]) store_stream(reinterpret_cast<T*>(base) + v, T{});
}

// ------------------------------------------------------------------ launches

template <typename D, int DVB, typename E, int VB> void run_sums(const BankGradParams& p, hipStream_t stream) {
    constexpr int N = 16 / int(sizeof(D));
    const int vecs = (p.hd + N - 1) / N;
    int lanes = kMinLanes;
    while (lanes < 64 && lanes < vecs) lanes *= 2;
    const int groups = kThreads / lanes, slices = (vecs + lanes - 1) / lanes;
    const dim3 grid{unsigned((p.blocks + groups - 1) / groups * slices)}, block{kThreads};
    const size_t lds = size_t(groups * p.block + p.spill + 2) * sizeof(Term);
    if (p.w[0] != nullptr) {
        if constexpr (sizeof(D) == 4)
            hipLaunchKernelGGL((sum_kernel<D, DVB, E, VB, true, false>), grid, block, lds, stream, p, lanes, slices);
    } else if (p.dropout.threshold != 0) {
        hipLaunchKernelGGL((sum_kernel<D, DVB, E, VB, false, true>), grid, block, lds, stream, p, lanes, slices);
    } else {
        hipLaunchKernelGGL((sum_kernel<D, DVB, E, VB, false, false>), grid, block, lds, stream, p, lanes, slices);
    }
    int join_lanes = kMinLanes;
    while (join_lanes < 64 && join_lanes < (p.hd + 3) / 4) join_lanes *= 2;
    const dim3 join{unsigned((p.blocks + kJoinBlocks - 1) / kJoinBlocks), unsigned(((p.hd + 3) / 4 + join_lanes - 1) / join_lanes)};
    if (p.blocks > 1) hipLaunchKernelGGL((join_kernel<E, VB>), join, dim3(kJoinThreads), 0, stream, p, join_lanes);
}

template <typename D, int DVB> void run_bank(const BankGradParams& p, bool bank_bf16, bool vec, hipStream_t stream) {
    if (bank_bf16 && vec) run_sums<D, DVB, uint16_t, 16>(p, stream);
    else if (bank_bf16) run_sums<D, DVB, uint16_t, 2>(p, stream);
    else if (vec) run_sums<D, DVB, float, 16>(p, stream);
    else run_sums<D, DVB, float, 4>(p, stream);
}

int64_t zero_rows(int64_t row_bytes) {
    const int64_t rows = kZeroBytes / row_bytes;
    return rows < 1 ? 1 : rows > kZeroRows ? kZeroRows : rows;
}
template <int VB> void run_zero(const BankGradParams& p, int64_t row_bytes, hipStream_t stream) {
    const int64_t rows = zero_rows(row_bytes);
    hipLaunchKernelGGL(zero_kernel<VB>, dim3(unsigned((p.num_slots + rows - 1) / rows)), dim3(kThreads), 0, stream, p,
                       int(rows), row_bytes);
}

template <bool LOOKUP> void run_sort_one(const BankGradParams& p, hipStream_t stream) {
    const dim3 grid{1}, block{kOneThreads};
    if (p.entries <= kOneThreads) hipLaunchKernelGGL((sort_one_kernel<LOOKUP, 1>), grid, block, 0, stream, p);
    else if (p.entries <= 2 * kOneThreads) hipLaunchKernelGGL((sort_one_kernel<LOOKUP, 2>), grid, block, 0, stream, p);
    else if (p.entries <= 4 * kOneThreads) hipLaunchKernelGGL((sort_one_kernel<LOOKUP, 4>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((sort_one_kernel<LOOKUP, kOneItems>), grid, block, 0, stream, p);
}

template <bool LOOKUP, int ITEMS> void run_sort_many(const BankGradParams& p, hipStream_t stream) {
    const dim3 tiles{p.tiles}, block{kThreads};
    const dim3 scans{unsigned(((1 << p.bits) + kScanDigits - 1) / kScanDigits)};
    for (int pass = 0; pass < p.passes; ++pass) {
        if (pass == 0) hipLaunchKernelGGL((sort_count_kernel<true, LOOKUP, ITEMS>), tiles, block, 0, stream, p, pass);
        else hipLaunchKernelGGL((sort_count_kernel<false, LOOKUP, ITEMS>), tiles, block, 0, stream, p, pass);
        hipLaunchKernelGGL(sort_scan_kernel, scans, dim3(kScanDigits * kScanParts), 0, stream, p, pass);
        if (pass == 0) hipLaunchKernelGGL((sort_place_kernel<true, LOOKUP, ITEMS>), tiles, block, 0, stream, p, pass);
        else hipLaunchKernelGGL((sort_place_kernel<false, LOOKUP, ITEMS>), tiles, block, 0, stream, p, pass);
    }
}

template <bool LOOKUP> void run_sort(const BankGradParams& p, hipStream_t stream) {
    if (p.items == 0) run_sort_one<LOOKUP>(p, stream);
    else if (p.items == 4) run_sort_many<LOOKUP, 4>(p, stream);
    else run_sort_many<LOOKUP, 16>(p, stream);
}

Divisor divisor(uint32_t d) {
    Divisor r{0, 31};
    if (d == 0) return r;  // never divided by
    while ((uint64_t(1) << (r.shift - 31)) < d) ++r.shift;
    r.mul = uint32_t(((uint64_t(1) << r.shift) + d - 1) / d);
    return r;
}

}  // namespace

int64_t bank_grad_layout(BankGradParams* p, void* workspace) {
    const int64_t entries = p->entries, octets = (int64_t(p->hd) + 7) / 8;
    int bits = 1;
    while (bits < 31 && (uint64_t(p->num_slots - 1) >> bits) != 0) ++bits;
    p->passes = (bits + kMaxBits - 1) / kMaxBits;
    p->bits = (bits + p->passes - 1) / p->passes;
    p->items = entries <= kOneEntries ? 0 : entries <= 262144 ? 4 : 16;
    p->tiles = p->items > 0 ? uint32_t((entries + kThreads * p->items - 1) / (kThreads * p->items)) : 0;
    // Entries of a lane group: enough groups for four wavefronts on each SIMD of 256 CUs.
    const int64_t threads = entries * (octets < kMinLanes ? kMinLanes : octets);
    int block = 8;
    while (block < kMaxBlock && threads / block > 4096 * 64) block *= 2;
    p->block = block;
    p->spill = block / 2 < kMaxSpill ? block / 2 : kMaxSpill;
    p->blocks = uint32_t((entries + block - 1) / block);
    char* base = static_cast<char*>(workspace);
    int64_t used = 0;
    auto place = [&](int64_t bytes) {
        char* at = base != nullptr ? base + used : nullptr;
        used += (bytes + 15) / 16 * 16;
        return at;
    };
    const int64_t digits = int64_t(1) << p->bits;
    p->n = reinterpret_cast<uint32_t*>(place(4));
    p->total = reinterpret_cast<uint32_t*>(place(4 * p->passes * digits));
    p->hist = reinterpret_cast<uint32_t*>(place(4 * p->passes * p->tiles * digits));
    for (int i = 0; i < 2; ++i) p->records[i] = reinterpret_cast<Record*>(place(8 * entries));
    p->first = reinterpret_cast<float*>(place(32 * octets * p->blocks));
    p->last = reinterpret_cast<float*>(place(32 * octets * p->blocks));
    return used;
}

int64_t bank_grad_groups(const BankGradParams& p, int bank_size) {
    const int64_t rows = zero_rows(int64_t(p.hd) * bank_size);
    return p.add ? 0 : (p.num_slots + rows - 1) / rows;  // those over entries are at most 2^31 / 64
}

hipError_t launch_bank_grad(const BankGradParams& call, bool dout_bf16, bool bank_bf16, hipStream_t stream) {
    BankGradParams p = call;
    p.first_entries = p.tokens * p.width[0];
    p.by_width[0] = divisor(p.width[0]);
    p.by_width[1] = divisor(p.width[1]);
    p.by_chunk = divisor(p.chunk);
    const int64_t row_bytes = int64_t(p.hd) * (bank_bf16 ? 2 : 4);
    const bool bank_vec = (reinterpret_cast<uintptr_t>(p.dbank) | uintptr_t(row_bytes)) % 16 == 0;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.dout[0]) | (p.width[1] != 0 ? reinterpret_cast<uintptr_t>(p.dout[1]) : 0) |
                         uintptr_t(p.hd) * (dout_bf16 ? 2 : 4);
    if (p.entries > 0 && p.w[0] == nullptr) run_sort<true>(p, stream);
    else if (p.entries > 0) run_sort<false>(p, stream);
    if (!p.add) {
        if (bank_vec) run_zero<16>(p, row_bytes, stream);
        else if (bank_bf16) run_zero<2>(p, row_bytes, stream);
        else run_zero<4>(p, row_bytes, stream);
    }
    if (p.entries > 0) {
        if (dout_bf16 && at % 16 == 0) run_bank<uint16_t, 16>(p, bank_bf16, bank_vec, stream);
        else if (dout_bf16) run_bank<uint16_t, 2>(p, bank_bf16, bank_vec, stream);
        else if (at % 16 == 0) run_bank<float, 16>(p, bank_bf16, bank_vec, stream);
        else run_bank<float, 4>(p, bank_bf16, bank_vec, stream);
    }
    return hipGetLastError();
}

}  // namespace sdm
