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

// Columns are summed in turns, which use the same memory, where the sums of blocks would take more than
// this: up to hd / 4 bytes an entry, far more than dout where its tokens have many entries (32768 tokens of
// 512 x 8192: 1.5 GB of workspace, at once 34.8). A turn reads the entries again, 12 bytes for 256 or more
// of dout, and finds more of its columns in the caches (8192 tokens of 256 x 8192 into 32768 slots, four
// turns: 10.4 ms, at once 11.2).
constexpr int64_t kTurnBytes = 1LL << 30;
constexpr int kMinTurn = 64;  // columns: whole lines of dout and of dbank

// ------------------------------------------------------------------ entries

constexpr uint32_t kNone = 0xffffffffu;
struct Entry {
    Record r;  // slot kNone: does not count
    float w;
};

// Entry e of the call. All of its loads are made whatever the others bring, so that those of many
// entries are in flight together.
template <bool LOOKUP> __device__ __forceinline__ Entry entry_of(const BankGradParams& p, uint32_t e) {
    const bool second = !LOOKUP && e >= p.first_entries;
    const uint32_t at = second ? e - p.first_entries : e;
    const int64_t s = slot_at(second ? p.idx[1] : p.idx[0], at, p.idx64 ? 8 : 4);
    bool counts = uint64_t(s) < uint64_t(p.num_slots);
    uint32_t token = e;
    float w = 1.0f;
    if (!LOOKUP) {
        const Divisor by_width = second ? p.by_width[1] : p.by_width[0];
        token = divide(at, by_width);
        const uint32_t c = divide(token, p.by_chunk);
        int32_t limit = int32_t(p.valid);
        if (p.chunk_valid != nullptr) limit = p.chunk_valid[c];
        counts &= int32_t(token - c * p.chunk) < limit;
        w = value_at(second ? p.w[1] : p.w[0], at, p.w_bf16 ? 2 : 4);
    }
    return {{counts ? uint32_t(s) : kNone, token | (second ? kSecond : 0)}, w};
}

// ------------------------------------------------------------------ zeros

// Part `part` of `parts` of the bank's bytes, kZeroBytes a workgroup: the sort's launches leave most
// of the card idle.
constexpr int64_t kZeroBytes = 65536;
__device__ __host__ __forceinline__ int64_t zero_groups(int64_t bytes, int parts) {  // of a part
    return ((bytes + kZeroBytes - 1) / kZeroBytes + parts - 1) / parts;
}
__device__ __forceinline__ void zero_part(const BankGradParams& p, int part, int parts, uint32_t group) {
    const int64_t begin = (part * zero_groups(p.zero_bytes, parts) + group) * kZeroBytes, end = min(begin + kZeroBytes, p.zero_bytes);
    char* to = static_cast<char*>(p.dbank);
    const int threads = blockDim.x;
    if (reinterpret_cast<uintptr_t>(to) % 16 == 0) {
        for (int64_t i = begin + threadIdx.x * 16; i + 16 <= end; i += threads * 16)
            store_stream(reinterpret_cast<uint4*>(to + i), uint4{});
        for (int64_t i = end - end % 16 + threadIdx.x * 2; i < end; i += threads * 2) *reinterpret_cast<uint16_t*>(to + i) = 0;
    } else {
        for (int64_t i = begin + threadIdx.x * 2; i < end; i += threads * 2) *reinterpret_cast<uint16_t*>(to + i) = 0;
    }
}
__global__ __launch_bounds__(kThreads) void zero_kernel(BankGradParams p) { zero_part(p, 0, 1, blockIdx.x); }

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
__device__ __forceinline__ void rank_items(const Entry (&e)[ITEMS], int pass, int bits, uint16_t* count, uint32_t (&rank)[ITEMS]) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const bool has = e[i].r.slot != kNone;
        const uint32_t digit = digit_of(e[i].r.slot, pass, bits);
        const uint64_t same = lanes_with(digit, has, bits);
        const uint32_t below = lanes_below(same);
        rank[i] = 0;
        if (has) {
            const uint32_t before = count[digit];
            rank[i] = before + below;
            wave_lds_order();
            if (below == 0) count[digit] = uint16_t(before + uint32_t(__popcll(same)));
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

// Few entries, up to 4096: one workgroup sorts them in LDS, all passes in one launch (500 entries: 5 us).
// With 8 entries a thread it took 25 us for 8192 in two passes, as long as the four launches of many
// workgroups, which zero the bank beside it.
constexpr int kOneThreads = 1024;
constexpr int kOneWaves = kOneThreads / 64;

template <bool LOOKUP, int ITEMS> __global__ __launch_bounds__(kOneThreads) void sort_one_kernel(BankGradParams p) {
    constexpr uint32_t kMost = kOneThreads * ITEMS;
    __shared__ Record records[kMost];
    __shared__ float weights[LOOKUP ? 1 : kMost];
    __shared__ uint16_t count[kOneWaves][kMaxDigits];  // of all entries, at most kMost
    __shared__ uint32_t scratch[kOneWaves];
    if (blockIdx.x > 0) return zero_part(p, 0, 1, blockIdx.x - 1);
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, digits = 1 << p.bits;
    uint32_t rank[ITEMS], n = p.entries;
    Entry e[ITEMS];
    const uint32_t first = wave * (64 * ITEMS) + lane;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) e[i] = entry_of<LOOKUP>(p, min(first + i * 64, n - 1));
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) e[i].r.slot = first + i * 64 < n ? e[i].r.slot : kNone;
    for (int pass = 0; pass < p.passes; ++pass) {
        for (int i = tid; i < kOneWaves << p.bits; i += kOneThreads) count[i >> p.bits][i & (digits - 1)] = 0;
        __syncthreads();
        rank_items<ITEMS>(e, pass, p.bits, count[wave], rank);
        __syncthreads();
        uint32_t all = 0;
        if (tid < digits)
            for (int w = 0; w < kOneWaves; ++w) all += count[w][tid];
        uint32_t base = sum_below<kOneThreads>(all, scratch, &n);
        if (tid < digits) {
            for (int w = 0; w < kOneWaves; ++w) {
                const uint32_t v = count[w][tid];
                count[w][tid] = uint16_t(base);
                base += v;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (e[i].r.slot == kNone) continue;
            const uint32_t to = count[wave][digit_of(e[i].r.slot, pass, p.bits)] + rank[i];
            records[to] = e[i].r;
            if (!LOOKUP) weights[to] = e[i].w;
        }
        __syncthreads();
        if (pass == p.passes - 1) break;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t from = min(first + i * 64, kMost - 1);
            e[i] = {records[from], LOOKUP ? 1.0f : weights[from]};
            e[i].r.slot = first + i * 64 < n ? e[i].r.slot : kNone;
        }
    }
    const int to = (p.passes - 1) & 1;
    for (uint32_t i = tid; i < n; i += kOneThreads) {
        p.records[to][i] = records[i];
        if (!LOOKUP) p.weights[to][i] = weights[i];
    }
    if (tid == 0) *p.n = n;
}

constexpr int kWaves = kThreads / 64;

// A thread's entries of a tile, `stride` apart: what is there, before it is known how many count.
template <bool FIRST, bool LOOKUP, bool WEIGHTS, int ITEMS>
__device__ __forceinline__ void load_entries(const BankGradParams& p, int pass, uint32_t first, uint32_t stride, Entry (&e)[ITEMS]) {
    const int from = (pass - 1) & 1;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const uint32_t at = min(first + i * stride, p.entries - 1);
        if (FIRST) e[i] = entry_of<LOOKUP>(p, at);
        else e[i] = {p.records[from][at], WEIGHTS ? p.weights[from][at] : 1.0f};
    }
}
// Slot kNone past the end.
template <int ITEMS> __device__ __forceinline__ void cut_entries(uint32_t first, uint32_t stride, uint32_t n, Entry (&e)[ITEMS]) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) e[i].r.slot = first + i * stride < n ? e[i].r.slot : kNone;
}

// The count of a tile's entries that have a digit: tiles side by side where they are scanned, digits
// where every workgroup adds the tiles up.
template <bool SUMS> __device__ __forceinline__ uint32_t* hist_of(const BankGradParams& p, int pass, uint32_t tile, int digit) {
    if (SUMS) return p.hist + ((int64_t(pass) * p.tiles + tile) << p.bits) + digit;
    return p.hist + ((int64_t(pass) << p.bits) + digit) * p.stride + tile;
}

// How many entries of each tile have each digit.
template <bool FIRST, bool LOOKUP, int ITEMS, bool SUMS>
__global__ __launch_bounds__(kThreads) void sort_count_kernel(BankGradParams p, int pass) {
    __shared__ uint32_t count[kMaxDigits];
    if (blockIdx.x >= p.tiles) return zero_part(p, 2 * pass, 2 * p.passes, blockIdx.x - p.tiles);
    const int digits = 1 << p.bits;
    const uint32_t n = FIRST ? p.entries : *p.n, first = blockIdx.x * uint32_t(kThreads * ITEMS) + threadIdx.x;
    Entry e[ITEMS];
    load_entries<FIRST, LOOKUP, false, ITEMS>(p, pass, first, kThreads, e);
    for (int d = threadIdx.x; d < digits; d += kThreads) count[d] = 0;
    __syncthreads();
    cut_entries(first, kThreads, n, e);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        if (e[i].r.slot != kNone) atomicAdd(&count[digit_of(e[i].r.slot, pass, p.bits)], 1u);
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kThreads) *hist_of<SUMS>(p, pass, blockIdx.x, d) = count[d];
}

// For each digit, the entries of lower tiles that have it, in place, and of all of them: a
// workgroup a digit, kScanTiles tiles at a time.
constexpr uint32_t kScanEach = 4, kScanTiles = kThreads * kScanEach;
__global__ __launch_bounds__(kThreads) void sort_scan_kernel(BankGradParams p, int pass) {
    __shared__ uint32_t scratch[2][kWaves];
    const int digits = 1 << p.bits;
    uint32_t* hist = p.hist + (int64_t(pass) * digits + blockIdx.x) * p.stride;
    uint32_t before = 0;
    int buffer = 0;
    for (uint32_t i0 = 0; i0 < p.tiles; i0 += kScanTiles, buffer ^= 1) {
        const uint32_t i = i0 + threadIdx.x * kScanEach;  // p.stride is a multiple of kScanEach
        uint4 v = {};
        if (i < p.tiles) v = *reinterpret_cast<const uint4*>(hist + i);
        v.y = i + 1 < p.tiles ? v.y : 0;
        v.z = i + 2 < p.tiles ? v.z : 0;
        v.w = i + 3 < p.tiles ? v.w : 0;
        uint32_t all;
        uint32_t at = before + sum_below<kThreads>(v.x + v.y + v.z + v.w, scratch[buffer], &all);
        if (i < p.tiles) *reinterpret_cast<uint4*>(hist + i) = make_uint4(at, at + v.x, at + v.x + v.y, at + v.x + v.y + v.z);
        before += all;
    }
    if (threadIdx.x == 0) p.total[pass * digits + blockIdx.x] = before;
}

// Puts each entry of a tile in its place of the order by this pass's digit. A wavefront takes
// 64 neighbours at a time; the lanes of the same digit find one another by ballots. The tile's
// entries are put in order in LDS first, so that those of a digit leave as one run of memory.
// SUMS: the tiles are few, and a workgroup adds up the lower ones' counts by itself.
// Bound by a tile's chain of steps, with five tiles on a compute unit at a time: 3.14 M entries of
// 12 bytes read and written in 23 us, 3.2 TB/s; directly to their places, without LDS, 37 us.
template <bool FIRST, bool LOOKUP, int ITEMS, bool SUMS>
__global__ __launch_bounds__(kThreads) void sort_place_kernel(BankGradParams p, int pass) {
    constexpr uint32_t kTile = kThreads * ITEMS;
    __shared__ Record records[kTile];
    __shared__ float weights[LOOKUP ? 1 : kTile];
    __shared__ uint16_t count[kWaves][kMaxDigits];  // of the tile's entries
    __shared__ uint32_t go[kMaxDigits];  // where a digit's entries of this tile go, less where they are in `records`
    __shared__ uint32_t scratch[2][kWaves];
    if (blockIdx.x >= p.tiles) return zero_part(p, 2 * pass + 1, 2 * p.passes, blockIdx.x - p.tiles);
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, digits = 1 << p.bits;
    const uint32_t n = FIRST ? p.entries : *p.n, first = blockIdx.x * kTile + wave * (64 * ITEMS) + lane;
    Entry e[ITEMS];
    uint32_t rank[ITEMS];
    load_entries<FIRST, LOOKUP, !LOOKUP, ITEMS>(p, pass, first, 64, e);
    // A thread takes digits 2 tid and 2 tid + 1: those of all tiles, and of the lower ones.
    uint32_t total[2] = {}, before[2] = {};
    if (2 * tid < digits) {
        if (SUMS) {
#pragma unroll 16
            for (uint32_t i = 0; i < p.tiles; ++i) {
                const uint2 v = *reinterpret_cast<const uint2*>(hist_of<SUMS>(p, pass, i, 2 * tid));
                total[0] += v.x;
                total[1] += v.y;
                before[0] += i < blockIdx.x ? v.x : 0;
                before[1] += i < blockIdx.x ? v.y : 0;
            }
        } else {
            const uint2 a = *reinterpret_cast<const uint2*>(p.total + pass * digits + 2 * tid);
            total[0] = a.x, total[1] = a.y;
            before[0] = *hist_of<SUMS>(p, pass, blockIdx.x, 2 * tid);
            before[1] = *hist_of<SUMS>(p, pass, blockIdx.x, 2 * tid + 1);
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
        for (int w = 0; w < kWaves; ++w) count[w][2 * tid + j] = 0;
    if (!FIRST && blockIdx.x * kTile >= n) return;  // of the whole workgroup
    cut_entries(first, 64, n, e);
    uint32_t all, here;
    const uint32_t below = sum_below<kThreads>(total[0] + total[1], scratch[0], &all);
    if (FIRST && blockIdx.x == 0 && tid == 0) *p.n = all;
    rank_items<ITEMS>(e, pass, p.bits, count[wave], rank);
    __syncthreads();
    uint32_t mine[2] = {};
#pragma unroll
    for (int j = 0; j < 2; ++j)
        for (int w = 0; w < kWaves; ++w) mine[j] += count[w][2 * tid + j];
    uint32_t base = sum_below<kThreads>(mine[0] + mine[1], scratch[1], &here);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        go[2 * tid + j] = below + (j == 1 ? total[0] : 0) + before[j] - base;
        for (int w = 0; w < kWaves; ++w) {
            const uint32_t v = count[w][2 * tid + j];
            count[w][2 * tid + j] = uint16_t(base);
            base += v;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        if (e[i].r.slot == kNone) continue;
        const uint32_t to = count[wave][digit_of(e[i].r.slot, pass, p.bits)] + rank[i];
        records[to] = e[i].r;
        if (!LOOKUP) weights[to] = e[i].w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const uint32_t from = i * kThreads + tid;
        if (from >= here) break;
        const Record r = records[from];
        const uint32_t to = go[digit_of(r.slot, pass, p.bits)] + from;
        p.records[pass & 1][to] = r;
        if (!LOOKUP) p.weights[pass & 1][to] = weights[from];
    }
}

// ------------------------------------------------------------------ sums

// The sorted entries are cut into blocks, a lane group each. A run of equal slots that ends within
// `spill` entries past the end of the block it begins in, or the next one's, is that block's to its
// end, and the next begins behind it. Of a longer run each block makes a partial sum, which
// join_kernel adds up. cont: the block of sorted entries that begins at `begin` continues such a
// long run. at(i): the slot of sorted entry i.
template <typename F> __device__ __forceinline__ bool cont(const BankGradParams& p, F at, uint32_t n, uint64_t begin) {
    return begin > 0 && begin + p.spill < n && at(begin - 1) == at(begin + p.spill);
}

__device__ __forceinline__ bool bit_at(uint64_t bits, int i) {
    return (i & 32 ? uint32_t(bits >> 32) : uint32_t(bits)) >> (i & 31) & 1;
}

// N neighbouring columns of a row of hd, from column c. VEC: rows are whole vectors of N; else a
// column at a time, those past the row's end 0.
template <typename D, int N, bool VEC> __device__ __forceinline__ void load_columns(const D* row, int c, int hd, float (&x)[N]) {
    if constexpr (VEC) {
        constexpr int VB = N * int(sizeof(D)) < 16 ? N * int(sizeof(D)) : 16, M = VB / int(sizeof(D));
#pragma unroll
        for (int i = 0; i < N; i += M) {
            const typename RawVec<VB>::T raw = *reinterpret_cast<const typename RawVec<VB>::T*>(row + c + i);
            D e[M];
            __builtin_memcpy(e, &raw, VB);
#pragma unroll
            for (int j = 0; j < M; ++j) x[i + j] = widen(e[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = c + i < hd ? widen(row[c + i]) : 0.0f;
    }
}
// The row's new values: the sums times `factor`, and (ADD) what was there.
template <typename E, int N, bool VEC, bool ADD>
__device__ __forceinline__ void store_columns(E* row, int c, int hd, float factor, const float (&x)[N]) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x[i] * factor;
    if (ADD) {
        float old[N];
        load_columns<E, N, VEC>(row, c, hd, old);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += old[i];
    }
    if constexpr (VEC) {
        constexpr int VB = N * int(sizeof(E)) < 16 ? N * int(sizeof(E)) : 16, M = VB / int(sizeof(E));
#pragma unroll
        for (int i = 0; i < N; i += M) {
            float part[M];
#pragma unroll
            for (int j = 0; j < M; ++j) part[j] = v[i + j];
            store_stream(reinterpret_cast<typename RawVec<VB>::T*>(row + c + i), Pack<E, VB>::of(part));
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + i < hd) row[c + i] = narrow<E>(v[i]);
    }
}

// What the sums need of an entry, put into LDS.
struct Term {
    const void* row;  // of dout
    uint32_t token;
    float w;
};

constexpr int kFlight = 8;  // rows whose loads are in flight together

// What the two kinds of sums share. A lane has N columns of a row's slice, 16 bytes of dout; the
// lanes of a group read theirs in one run of memory.
template <typename D, typename E, bool VEC, bool WEIGHTS, bool DROP> struct Sums {
    static constexpr int N = 16 / int(sizeof(D));

    const BankGradParams& p;
    const Record* records;
    const float* weights;
    uint32_t n;
    int c;  // the lane's first column
    PhiloxKey key;

    __device__ __forceinline__ Sums(const BankGradParams& p, int lanes, int lane, uint32_t slice) : p(p) {
        const int last = (p.passes - 1) & 1;
        records = p.records[last];
        weights = p.weights[last];
        n = *p.n;
        c = (p.line * (kMinTurn / N) + int(slice) * lanes + lane) * N;  // a multiple of N that the compiler sees
        key = {};
        if (DROP) key = philox_key(p.dropout);
    }
    __device__ __forceinline__ Term term(uint64_t i) const {
        const uint32_t token = records[i].token;
        const void* dout = WEIGHTS && (token & kSecond) ? p.dout[1] : p.dout[0];
        return {static_cast<const D*>(dout) + int64_t(token & ~kSecond) * p.hd, token, WEIGHTS ? weights[i] : 1.0f};
    }
    __device__ __forceinline__ void load(const Term& t, float (&x)[N]) const {
        // A lane past the row's end reads the row's last columns.
        load_columns<D, N, VEC>(static_cast<const D*>(t.row), VEC ? min(c, p.hd - N) : c, p.hd, x);
    }
    __device__ __forceinline__ void add(const Term& t, const float (&x)[N], float (&acc)[N]) const {
        const uint32_t kept = DROP ? kept_columns(key, uint32_t(c) / 8, t.token, p.dropout.threshold) >> (c & 7) : 0xff;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (WEIGHTS) acc[j] = fmaf(t.w, x[j], acc[j]);
            else if (DROP) acc[j] += kept >> j & 1 ? x[j] : 0.0f;
            else acc[j] += x[j];
        }
    }
    static __device__ __forceinline__ void clear(float (&acc)[N]) {
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    }
    template <bool ADD> __device__ __forceinline__ void finish(uint32_t slot, const float (&acc)[N]) const {
        E* row = static_cast<E*>(p.dbank) + int64_t(slot) * p.hd;
        store_columns<E, N, VEC, ADD>(row, c, p.hd, WEIGHTS ? 1.0f : p.factor, acc);
    }
    __device__ __forceinline__ void zero(uint32_t slot) const {  // no entry names it: +0, whatever the factor's sign
        float none[N];
        clear(none);
        store_columns<E, N, VEC, false>(static_cast<E*>(p.dbank) + int64_t(slot) * p.hd, c, p.hd, 1.0f, none);
    }
};

// The grid of the sums, workgroups in eights, one on each XCD: `sums` eights for the blocks of entries,
// then `rows` eights for the bank's rows. (With the blocks' workgroups, most of which end at once, and
// the rows' taken in turn, 3.14 M entries of 2^21 x 128 took 459 us instead of 332.)
struct SumGrid {
    int lanes, slices, shift;  // lanes of a group; groups that share a row's columns; log2 of p.block
    uint32_t ranges;           // workgroups of a slice, for the blocks
    uint32_t group_rows;       // rows of a lane group
    uint32_t row_ranges;       // workgroups of a slice, for the rows
    uint32_t sums, rows;
};

// ------------------------------------------------------------------ whole banks: sums of rows

constexpr int kMinLanes = 4;
constexpr int kMaxRows = 2048;       // of a workgroup
constexpr uint32_t kStaged = 1024;   // entries of a workgroup that fit LDS
constexpr uint32_t kScanned = 4096;  // entries that are looked at one by one for where the rows begin

// The first of the sorted entries whose slot is at least `slot`: a wavefront looks at 64 places at once.
__device__ __forceinline__ uint32_t lower_bound(const Record* records, uint32_t n, uint64_t slot) {
    uint32_t lo = 0, len = n;
    while (len > 0) {
        const uint32_t step = (len + 63) / 64, q = (threadIdx.x % 64 + 1) * step - 1;
        const uint32_t less = uint32_t(__popcll(__ballot(q < len && records[lo + min(q, len - 1)].slot < slot)));
        lo += less * step;
        len = min(step - 1, len - less * step);
    }
    return lo;
}

// A workgroup takes neighbouring rows of the bank and writes each: the sum of its entries, or 0. So
// the bank is written once and in order. Rows of long runs are left to the blocks' sums.
// Bound by what leaves and enters the L2 caches: 4.19 M entries (3.14 M that count) of 2^21 x 128
// float32 in 332 us, 1.07 GB written and 1.19 GB fetched (9.27 M misses of 128 bytes), 6.8 TB/s, of which
// dout, 34 MB, comes from the cache behind the L2s. 56% of the L2s' reads hit. Without slices of the
// columns 376 us, 1.64 GB fetched. The entries' rows first and the zeros in a pass of its own 342.
template <typename S>
__device__ __forceinline__ void sum_rows(const S& s, const SumGrid& g, uint32_t range, uint32_t* lds) {
    constexpr int N = S::N;
    const BankGradParams& p = s.p;
    const int tid = threadIdx.x, groups = kThreads / g.lanes, group = tid / g.lanes;
    const uint64_t first = uint64_t(range) * groups * g.group_rows;
    const uint32_t rows = uint32_t(min(uint64_t(groups) * g.group_rows, uint64_t(p.num_slots) - first));
    Term* terms = reinterpret_cast<Term*>(lds);        // [kStaged]
    uint32_t* starts = lds + kStaged * sizeof(Term) / 4;  // [rows + 1] where a row's entries begin, from the first row's
    uint32_t* bounds = starts + groups * g.group_rows + 1;  // [2]
    if (tid < 128) {
        const uint32_t at = lower_bound(s.records, s.n, first + (tid < 64 ? 0 : rows));
        if (tid % 64 == 0) bounds[tid / 64] = at;
    }
    __syncthreads();
    const uint32_t lo = bounds[0], count = bounds[1] - lo;
    if (count <= kScanned) {
        for (uint32_t r = tid; r <= rows; r += kThreads) starts[r] = count;
        __syncthreads();
        for (uint32_t i = tid; i < count; i += kThreads) {
            const int row = int(s.records[lo + i].slot - uint32_t(first));
            const int before = i > 0 ? int(s.records[lo + i - 1].slot - uint32_t(first)) : -1;
            for (int k = before + 1; k <= row; ++k) starts[k] = i;
            if (i < kStaged) terms[i] = s.term(lo + i);
        }
    } else {
        for (uint32_t r = tid; r <= rows; r += kThreads) {
            uint32_t a = 0, b = count;
            while (a < b) {
                const uint32_t m = a + (b - a) / 2;
                if (s.records[lo + m].slot < first + r) a = m + 1;
                else b = m;
            }
            starts[r] = a;
        }
    }
    __syncthreads();
    if (s.c >= p.columns) return;
    const bool staged = count <= kStaged;
    auto is_long = [&](uint32_t r) {
        const uint32_t a = lo + starts[r], b = lo + starts[r + 1];
        return b - a > uint32_t(p.spill) && (((a >> g.shift) + 1) << g.shift) + uint32_t(p.spill) < b;
    };
    const uint32_t r0 = min(group * g.group_rows, rows), r1 = min(r0 + g.group_rows, rows);
    for (uint32_t r = r0; r < r1; ++r)
        if (starts[r] == starts[r + 1]) s.zero(uint32_t(first) + r);
    float acc[N];
    s.clear(acc);
    for (uint32_t r = r0; r < r1;) {
        if (is_long(r)) {
            ++r;
            continue;
        }
        uint32_t to = r + 1;  // rows r .. to have no long run
        while (to < r1 && !is_long(to)) ++to;
        uint32_t at = starts[r];
        const uint32_t end = starts[to];
        while (r < to && starts[r + 1] == at) ++r;
        uint32_t row_end = starts[min(r + 1, to)];
        while (at < end) {
            const uint32_t some = min(end - at, uint32_t(kFlight));
            float x[kFlight][N];
            Term t[kFlight];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                const uint32_t i = at + min(uint32_t(u), some - 1);
                if (staged) t[u] = terms[i];
                else t[u] = s.term(lo + i);
            }
#pragma unroll
            for (int u = 0; u < kFlight; ++u) s.load(t[u], x[u]);
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                if (u >= int(some)) break;
                s.add(t[u], x[u], acc);
                if (at + u + 1 == row_end) {
                    s.template finish<false>(uint32_t(first) + r, acc);
                    s.clear(acc);
                    do {
                        ++r;
                        row_end = starts[min(r + 1, to)];
                    } while (r < to && row_end == at + u + 1);
                }
            }
            at += some;
        }
        r = to;
    }
}

// ------------------------------------------------------------------ sums of blocks

constexpr int kMaxBlock = 32;
constexpr int kMaxSpill = 16;

// The words of LDS between the entries of a block and the next's: the groups' reads then fall on
// different banks.
__device__ __host__ __forceinline__ int lds_place(int i, int shift) { return i + (i >> shift); }

// How the sums are made: a row of the bank at a time, and the long runs by blocks; or all by blocks of
// entries, stored to rows that are zero, or added to what is there.
enum { kByRows, kStore, kAdd };

// What the entries of a range of blocks add to their rows; by rows, the long runs' alone.
template <int MODE, typename S>
__device__ __forceinline__ void sum_blocks(const S& s, const SumGrid& g, uint32_t range_number, uint32_t* lds) {
    constexpr int N = S::N;
    constexpr bool ALL = MODE != kByRows;
    const BankGradParams& p = s.p;
    const int groups = kThreads / g.lanes, group = int(threadIdx.x) / g.lanes;
    const uint64_t range = uint64_t(groups) * p.block, start = range_number * range;
    const uint32_t n = s.n;
    if (start >= n) return;
    if (!ALL) {
        auto at = [&](uint64_t i) { return s.records[i].slot; };
        const bool some = int(threadIdx.x) <= groups && cont(p, at, n, start + uint64_t(threadIdx.x) * p.block);
        if (!__syncthreads_or(some)) return;
    }
    // In LDS entry start - 1 + i has number i, so that the one before the range is there.
    const int most = int(range) + p.spill + 2;
    auto place = [&](int i) { return lds_place(i, g.shift); };
    Term* terms = reinterpret_cast<Term*>(lds);
    uint32_t* slots = lds + (place(most) + 1) * int(sizeof(Term) / 4);
    const int there = int(min(uint64_t(most), n - start + 1));
    for (int i = threadIdx.x; i < there; i += kThreads) {
        const uint64_t from = start + i > 0 ? start + i - 1 : 0;
        slots[place(i)] = s.records[from].slot;
        terms[place(i)] = s.term(from);
    }
    __syncthreads();
    const uint32_t b = range_number * groups + group;
    const uint64_t begin = uint64_t(b) * p.block;
    if (begin >= n || s.c >= p.columns) return;
    auto slot_of_sorted = [&](uint64_t i) { return slots[place(int(i + 1 - start))]; };
    const bool from_before = cont(p, slot_of_sorted, n, begin), goes_on = cont(p, slot_of_sorted, n, begin + p.block);
    int at = int(begin + 1 - start), end = min(at + p.block, there);
    const uint32_t last = slots[place(end - 1)];
    if (begin > 0 && !from_before)
        for (const uint32_t earlier = slots[place(at - 1)]; at < end && slots[place(at)] == earlier;) ++at;
    if (!goes_on)
        while (end < there && slots[place(end)] == last) ++end;
    auto add_up = [&](int at, int end, bool open) {  // open: the first run began in an earlier block
        float acc[N];
        s.clear(acc);
        uint32_t slot = at < end ? slots[place(at)] : 0;
        while (at < end) {
            const int some = min(end - at, kFlight);
            float x[kFlight][N];
            Term t[kFlight];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) t[u] = terms[place(at + min(u, some - 1))];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) s.load(t[u], x[u]);
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                if (u >= some) break;
                s.add(t[u], x[u], acc);
                const bool is_last = at + u + 1 == end;
                const uint32_t next = is_last ? kNone : slots[place(at + u + 1)];
                if (next != slot) {
                    if (open || (is_last && goes_on)) {
                        float* to = (open ? p.first : p.last) + int64_t(b) * p.turn + s.c;
#pragma unroll
                        for (int j = 0; j < N; j += 4)
                            *reinterpret_cast<float4*>(to + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
                    } else {
                        s.template finish<MODE == kAdd>(slot, acc);
                    }
                    open = false;
                    slot = next;
                    s.clear(acc);
                }
            }
            at += some;
        }
    };
    if (ALL) {
        add_up(at, end, from_before);
        return;
    }
    // The block's first run, or its last, or both, should they be long.
    int head = at, tail = end;
    if (from_before)
        for (const uint32_t first = slots[place(at)]; head < end && slots[place(head)] == first;) ++head;
    if (goes_on)
        while (tail > head && slots[place(tail - 1)] == last) --tail;
    if (from_before) add_up(at, head, true);
    if (tail < end) add_up(tail, end, false);
}

// All of a gradient's sums but the long runs' totals. The slices of a row's columns lie on XCDs of
// their own (workgroup i runs on XCD i mod 8), so that what an XCD's L2 cache holds of dout is that
// slice alone.
template <typename D, typename E, bool VEC, bool WEIGHTS, bool DROP, int MODE>
__global__ __launch_bounds__(kThreads) void sum_kernel(BankGradParams p, SumGrid g) {
    extern __shared__ uint4 lds16[];
    uint32_t* lds = reinterpret_cast<uint32_t*>(lds16);
    const bool blocks = MODE != kByRows || blockIdx.x < 8 * g.sums;
    const uint32_t number = blockIdx.x - (blocks ? 0 : 8 * g.sums), range = number / g.slices;
    if (range >= (blocks ? g.ranges : g.row_ranges)) return;
    const Sums<D, E, VEC, WEIGHTS, DROP> s(p, g.lanes, int(threadIdx.x) % g.lanes, number % g.slices);
    if (blocks) sum_blocks<MODE>(s, g, range, lds);
    else sum_rows(s, g, range, lds);
}

// ------------------------------------------------------------------ sums of blocks' sums

// Runs over several blocks, 14 us for a most frequent token of 2100 in 32768: a chain of loads. A
// workgroup looks at 64 blocks. Of the runs that begin there each lane group adds up some of the short
// ones that end there, in order; another's blocks are dealt out to all lane groups, each of which adds its own, and
// then the groups' sums are added. As many as a batch has rows may come together there, so that these
// additions are float64.
constexpr int kJoinThreads = 1024;
constexpr int kJoinBlocks = 64;

constexpr uint32_t kShort = 16;  // blocks of a run that one lane group adds up

template <typename E, bool VEC, bool ADD>
__global__ __launch_bounds__(kJoinThreads, 8) void join_kernel(BankGradParams p, int lanes) {  // 64 registers: two workgroups a compute unit
    constexpr int N = 4;
    __shared__ uint64_t masks[2];
    __shared__ uint32_t slots[64];  // of the blocks' last entries
    __shared__ double sums[kJoinThreads][N];
    const int tid = threadIdx.x, groups = kJoinThreads / lanes, lane = tid % lanes, group = tid / lanes;
    const int c0 = p.line * kMinTurn + (int(blockIdx.y) * lanes + lane) * N;
    const int64_t columns = p.turn;
    const Record* records = p.records[(p.passes - 1) & 1];
    const uint32_t n = *p.n;
    const uint32_t b0 = blockIdx.x * uint32_t(kJoinBlocks);
    if (uint64_t(b0) * p.block >= n) return;
    auto at = [&](uint64_t i) { return records[i].slot; };
    if (tid < 64) {
        // Bit i of the first: a run of several blocks begins in block b0 + i; of the second: block
        // b0 + 1 + i is in the middle of one. All of the slots that this takes are loaded at once.
        const uint64_t begin = uint64_t(b0 + tid) * p.block, end = begin + p.block;
        auto any = [&](uint64_t i) { return records[min(i, uint64_t(p.entries - 1))].slot; };
        const uint32_t earlier = any(begin > 0 ? begin - 1 : 0), last = any(end - 1), first = any(end), spill = any(end + p.spill);
        const uint32_t next_last = any(end + p.block - 1), next_spill = any(end + p.block + p.spill);
        const bool goes_on = end + p.spill < n && last == spill;
        const bool further = goes_on && end + p.block + p.spill < n && next_last == next_spill;
        const bool is_new = goes_on && (begin == 0 || earlier != last);
        const uint64_t b = __ballot(is_new), m = __ballot(further && first == next_last);
        slots[tid] = last;
        if (tid == 0) {
            masks[0] = b;
            masks[1] = m;
        }
    }
    __syncthreads();
    const uint64_t begins = masks[0], middles = masks[1];
    auto add = [&](auto (&acc)[N], uint32_t b, uint32_t from, uint32_t more, uint32_t stride) {
        for (uint32_t c = from; c < more; c += kFlight * stride) {
            float x[kFlight][N];
#pragma unroll
            for (int u = 0; u < kFlight; ++u)
                load_columns<float, N, true>(p.first + (int64_t(b) + 1 + min(c + u * stride, more - 1)) * columns, c0, p.hd, x[u]);
#pragma unroll
            for (int u = 0; u < kFlight; ++u)
                if (c + u * stride < more)
#pragma unroll
                    for (int j = 0; j < N; ++j) acc[j] += x[u][j];
        }
    };
    auto finish = [&](uint32_t slot, const float (&acc)[N]) {
        E* row = static_cast<E*>(p.dbank) + int64_t(slot) * p.hd;
        store_columns<E, N, VEC, ADD>(row, c0, p.hd, p.factor, acc);
    };
    // The run's blocks after its first, as far as the masks tell: the middle ones, and its last.
    auto known = [&](int i) {
        uint32_t more = 1;
        while (i < 64 && bit_at(middles, i)) ++i, ++more;
        return more;
    };
    int turn = 0;
    for (uint64_t left = begins; left != 0; left &= left - 1, ++turn) {
        if (turn % groups != group) continue;
        const int i = __ffsll(static_cast<unsigned long long>(left)) - 1;
        const uint32_t b = b0 + uint32_t(i), more = known(i);
        if (more > kShort || i + more > 64 || c0 >= p.columns) continue;
        float acc[N];
        load_columns<float, N, true>(p.last + b * columns, c0, p.hd, acc);
        add(acc, b, 0, more, 1);
        finish(slots[i], acc);
    }
    for (uint64_t left = begins; left != 0; left &= left - 1) {
        const int i = __ffsll(static_cast<unsigned long long>(left)) - 1;
        uint32_t more = known(i);
        if (more <= kShort && i + more <= 64) continue;  // of the whole workgroup
        const uint32_t b = b0 + uint32_t(i), slot = slots[i];
        if (i + more > 64) {  // perhaps further than the masks
            uint32_t found;
            do {
                const uint64_t begin = (uint64_t(b) + 1 + more + tid) * p.block;
                const bool is = cont(p, at, n, begin) && at(begin) == slot;
                found = uint32_t(__syncthreads_count(is));
                more += found;
            } while (found == kJoinThreads);
        }
        double acc[N] = {};
        if (c0 < p.columns) {
            if (group == 0) {
                float begun[N];
                load_columns<float, N, true>(p.last + b * columns, c0, p.hd, begun);
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] = begun[j];
            }
            add(acc, b, group, more, groups);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) sums[tid][j] = acc[j];
        __syncthreads();
        if (group == 0 && c0 < p.columns) {
            for (int g = 1; g < min(groups, int(min(more, uint32_t(kJoinThreads)))); ++g) {
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += sums[g * lanes + lane][j];
            }
            float total[N];
#pragma unroll
            for (int j = 0; j < N; ++j) total[j] = float(acc[j]);
            finish(slot, total);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ launches

int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

// Whether a written bank's sums are made a row at a time. With few entries for its rows it is zeroed
// beside the sort instead, which takes as long without it, and only the rows that entries name are
// written again: 32768 tokens of 50000 x 1024 in 81 us instead of 88, 8192 entries of 131072 x 128 in
// 37 instead of 44. Where most rows are named that would write them twice, 130 us for 3.1 M entries of
// 2^21 x 128, as long as their sort.
bool by_rows(const BankGradParams& p) { return !p.add && p.entries > p.num_slots; }

SumGrid sum_grid(const BankGradParams& p, int dout_size, int bank_size) {
    const int width = p.columns - p.line * kMinTurn, n = 16 / dout_size, vecs = (width + n - 1) / n;
    SumGrid g{};
    // A gather reads each token's dout once for every entry: slices of the columns, so that an XCD's 4 MB
    // of L2 hold more of what its entries read, but of whole 128-byte lines of dbank (c3's entries: the
    // call 490 us with one slice, 471 with two, 440 with four, 609 with eight).
    g.slices = 1;
    const int64_t bytes = (p.width[1] != 0 ? 2 : 1) * int64_t(p.tokens) * width * dout_size;
    if (p.width[0] + p.width[1] >= 8)
        while (g.slices < 8 && bytes / g.slices > (3 << 20) && width * bank_size / g.slices >= 256) g.slices *= 2;
    if (vecs > 64 * g.slices) g.slices = (vecs + 63) / 64;
    g.lanes = kMinLanes;
    while (g.lanes * g.slices < vecs) g.lanes *= 2;
    const int groups = kThreads / g.lanes;
    g.shift = log2_of(p.block);
    g.ranges = (p.blocks + groups - 1) / groups;
    g.sums = uint32_t((int64_t(g.ranges) * g.slices + 7) / 8);
    if (by_rows(p)) {
        // Rows of a lane group: 32 KB of the bank a workgroup. (1563 tiles of 64 KB are one and a half
        // rounds of the compute units: 32768 tokens of 50000 x 1024, 123 against 89 us for the call; with
        // 16 KB, 101 us.)
        g.group_rows = 1;
        while (g.group_rows < 32 && 2 * g.group_rows * groups <= kMaxRows &&
               int64_t(g.group_rows) * kThreads * n * bank_size < 32768)
            g.group_rows *= 2;
        const int64_t rows = int64_t(groups) * g.group_rows;
        g.row_ranges = uint32_t((p.num_slots + rows - 1) / rows);
        g.rows = uint32_t((int64_t(g.row_ranges) * g.slices + 7) / 8);
    }
    return g;
}

template <typename D, typename E, bool VEC, bool WEIGHTS, bool DROP>
void run_sum(const BankGradParams& p, const SumGrid& g, hipStream_t stream) {
    const int groups = kThreads / g.lanes, most = groups * p.block + p.spill + 2;
    size_t lds = size_t(lds_place(most, g.shift) + 1) * (sizeof(Term) + 4);
    const size_t for_rows = kStaged * sizeof(Term) + size_t(groups * g.group_rows + 3) * 4;
    if (by_rows(p) && for_rows > lds) lds = for_rows;
    const dim3 grid{8 * (g.sums + g.rows)}, block{kThreads};
    if (p.add) hipLaunchKernelGGL((sum_kernel<D, E, VEC, WEIGHTS, DROP, kAdd>), grid, block, lds, stream, p, g);
    else if (by_rows(p)) hipLaunchKernelGGL((sum_kernel<D, E, VEC, WEIGHTS, DROP, kByRows>), grid, block, lds, stream, p, g);
    else hipLaunchKernelGGL((sum_kernel<D, E, VEC, WEIGHTS, DROP, kStore>), grid, block, lds, stream, p, g);
}

template <typename D, typename E, bool VEC> void run_turn(const BankGradParams& p, hipStream_t stream) {
    const SumGrid g = sum_grid(p, int(sizeof(D)), int(sizeof(E)));
    if (p.w[0] != nullptr) {
        if constexpr (sizeof(D) == 4) run_sum<D, E, VEC, true, false>(p, g, stream);
    } else if (p.dropout.threshold != 0) {
        run_sum<D, E, VEC, false, true>(p, g, stream);
    } else {
        run_sum<D, E, VEC, false, false>(p, g, stream);
    }
    if (p.blocks <= 1) return;
    const int vecs = (p.columns - p.line * kMinTurn + 3) / 4;
    int lanes = kMinLanes;
    while (lanes < 64 && lanes < vecs) lanes *= 2;
    const dim3 join{unsigned((p.blocks + kJoinBlocks - 1) / kJoinBlocks), unsigned((vecs + lanes - 1) / lanes)};
    if (p.add) hipLaunchKernelGGL((join_kernel<E, VEC, true>), join, dim3(kJoinThreads), 0, stream, p, lanes);
    else hipLaunchKernelGGL((join_kernel<E, VEC, false>), join, dim3(kJoinThreads), 0, stream, p, lanes);
}

template <typename D, typename E, bool VEC> void run_sums(const BankGradParams& call, hipStream_t stream) {
    BankGradParams p = call;
    for (int first = 0; first < p.hd; first += p.turn) {
        p.line = first / kMinTurn;
        p.first = call.first - first;  // where column 0 would be
        p.last = call.last - first;
        p.columns = p.hd - first < p.turn ? p.hd : first + p.turn;
        run_turn<D, E, VEC>(p, stream);
    }
}

template <typename D, typename E> void run_types(const BankGradParams& p, hipStream_t stream) {
    // Whole vectors of 16 / sizeof(D) columns in every row of dout and of dbank.
    constexpr int kN = 16 / int(sizeof(D)), kBank = kN * int(sizeof(E)) < 16 ? kN * int(sizeof(E)) : 16;
    const uintptr_t dout = reinterpret_cast<uintptr_t>(p.dout[0]) | (p.width[1] != 0 ? reinterpret_cast<uintptr_t>(p.dout[1]) : 0);
    if (p.hd % kN == 0 && dout % 16 == 0 && reinterpret_cast<uintptr_t>(p.dbank) % kBank == 0) run_sums<D, E, true>(p, stream);
    else run_sums<D, E, false>(p, stream);
}

// Up to this many entries one workgroup sorts them all.
constexpr int64_t kOneEntries = 4 * kOneThreads;
template <bool LOOKUP> void run_sort_one(const BankGradParams& p, hipStream_t stream) {
    const dim3 grid{unsigned(1 + zero_groups(p.zero_bytes, 1))}, block{kOneThreads};
    if (p.entries <= kOneThreads) hipLaunchKernelGGL((sort_one_kernel<LOOKUP, 1>), grid, block, 0, stream, p);
    else if (p.entries <= 2 * kOneThreads) hipLaunchKernelGGL((sort_one_kernel<LOOKUP, 2>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((sort_one_kernel<LOOKUP, 4>), grid, block, 0, stream, p);
}

// Up to this many tiles every workgroup that places entries adds their counts up by itself.
constexpr uint32_t kSumTiles = 64;

template <bool FIRST, bool LOOKUP, int ITEMS, bool SUMS> void run_pass(const BankGradParams& p, int pass, hipStream_t stream) {
    const dim3 tiles{unsigned(p.tiles + zero_groups(p.zero_bytes, 2 * p.passes))}, block{kThreads};
    hipLaunchKernelGGL((sort_count_kernel<FIRST, LOOKUP, ITEMS, SUMS>), tiles, block, 0, stream, p, pass);
    if (!SUMS) hipLaunchKernelGGL(sort_scan_kernel, dim3(1u << p.bits), block, 0, stream, p, pass);
    hipLaunchKernelGGL((sort_place_kernel<FIRST, LOOKUP, ITEMS, SUMS>), tiles, block, 0, stream, p, pass);
}
template <bool LOOKUP, int ITEMS, bool SUMS> void run_sort_many(const BankGradParams& p, hipStream_t stream) {
    run_pass<true, LOOKUP, ITEMS, SUMS>(p, 0, stream);
    for (int pass = 1; pass < p.passes; ++pass) run_pass<false, LOOKUP, ITEMS, SUMS>(p, pass, stream);
}

template <bool LOOKUP> void run_sort(const BankGradParams& p, hipStream_t stream) {
    if (p.items == 0) run_sort_one<LOOKUP>(p, stream);
    else if (p.items == 4) run_sort_many<LOOKUP, 4, true>(p, stream);
    else run_sort_many<LOOKUP, 8, false>(p, stream);
}

}  // namespace

int64_t bank_grad_layout(BankGradParams* p, void* workspace) {
    const int64_t entries = p->entries, octets = (int64_t(p->hd) + 7) / 8;
    int bits = 1;  // at least: a thread of the sort takes pairs of digits
    while (bits < 31 && (uint64_t(p->num_slots - 1) >> bits) != 0) ++bits;
    p->passes = (bits + kMaxBits - 1) / kMaxBits;
    p->bits = (bits + p->passes - 1) / p->passes;
    p->items = entries <= kOneEntries ? 0 : entries <= int64_t(kSumTiles) * kThreads * 4 ? 4 : 8;
    p->tiles = p->items > 0 ? uint32_t((entries + kThreads * p->items - 1) / (kThreads * p->items)) : 0;
    // Entries of a lane group: enough groups for four wavefronts on each SIMD of 256 CUs.
    const int64_t threads = entries * (octets < kMinLanes ? kMinLanes : octets);
    int block = 16;
    while (block < kMaxBlock && threads / block > 4096 * 64) block *= 2;
    p->block = block;
    p->spill = block / 2 < kMaxSpill ? block / 2 : kMaxSpill;
    p->blocks = uint32_t((entries + block - 1) / block);
    p->turn = int(8 * octets);
    const int64_t column_bytes = 8 * int64_t(p->blocks);  // of both arrays
    if (column_bytes * p->turn > kTurnBytes) {
        const int64_t most = kTurnBytes / column_bytes / kMinTurn * kMinTurn;
        p->turn = int(most > kMinTurn ? most : kMinTurn);
        if (p->turn > 8 * octets) p->turn = int(8 * octets);
    }
    p->line = 0;
    p->columns = p->hd < p->turn ? p->hd : p->turn;
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
    p->stride = (p->tiles + kScanEach - 1) / kScanEach * kScanEach;
    p->hist = reinterpret_cast<uint32_t*>(place(4 * p->passes * p->stride * digits));
    for (int i = 0; i < 2; ++i) p->records[i] = reinterpret_cast<Record*>(place(8 * entries));
    for (int i = 0; i < 2; ++i) p->weights[i] = reinterpret_cast<float*>(place(4 * entries));
    p->first = reinterpret_cast<float*>(place(4 * int64_t(p->turn) * p->blocks));
    p->last = reinterpret_cast<float*>(place(4 * int64_t(p->turn) * p->blocks));
    return used;
}

int64_t bank_grad_groups(const BankGradParams& p, int dout_size, int bank_size) {
    const SumGrid g = sum_grid(p, dout_size, bank_size);
    const int64_t zeroed = p.add || by_rows(p) ? 0 : int64_t(p.num_slots) * p.hd * bank_size;
    // In workgroups of 256 threads: one workgroup's sort has 1024, the bank's part beside it too.
    const int64_t sort = p.items == 0 ? 4 * (1 + zero_groups(zeroed, 1)) : p.tiles + zero_groups(zeroed, 2 * p.passes);
    const int64_t sums = 8 * (int64_t(g.sums) + g.rows);
    return sort > sums ? sort : sums;
}

hipError_t launch_bank_grad(const BankGradParams& call, bool dout_bf16, bool bank_bf16, hipStream_t stream) {
    BankGradParams p = call;
    p.first_entries = p.tokens * p.width[0];
    p.by_width[0] = divisor(p.width[0]);
    p.by_width[1] = divisor(p.width[1]);
    p.by_chunk = divisor(p.chunk);
    if (!by_rows(p) && !p.add) p.zero_bytes = int64_t(p.num_slots) * p.hd * (bank_bf16 ? 2 : 4);
    if (p.entries == 0) {
        if (!p.add) hipLaunchKernelGGL(zero_kernel, dim3(unsigned(zero_groups(p.zero_bytes, 1))), dim3(kThreads), 0, stream, p);
        return hipGetLastError();
    }
    if (p.w[0] == nullptr) run_sort<true>(p, stream);
    else run_sort<false>(p, stream);
    if (dout_bf16 && bank_bf16) run_types<uint16_t, uint16_t>(p, stream);
    else if (dout_bf16) run_types<uint16_t, float>(p, stream);
    else if (bank_bf16) run_types<float, uint16_t>(p, stream);
    else run_types<float, float>(p, stream);
    return hipGetLastError();
}

}  // namespace sdm
