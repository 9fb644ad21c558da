// Gradients to a bank (include/sdm_train.h): sdm_lookup_grad and sdm_gather_bank_grad.
//
// An entry is a named row: a lookup's row, or a (token, place) of a gather's operand. The
// entries that count are sorted by slot, equal slots in the order of the entries (a radix
// sort by 8 bits at a time, stable), and each slot's terms are then added in that order:
// no float atomics, so the same inputs give the same bits.

#include "sdm_dropout.h"
#include "sdm_rows.h"

namespace sdm {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kItems = 16;                 // entries of a thread of the sort
constexpr int kTile = kThreads * kItems;   // entries of a workgroup
constexpr int kDigits = 256;

// Between a wavefront's LDS writes and its reads of what other lanes wrote: its LDS accesses
// happen in order by themselves, so only the compiler has to keep to it.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ------------------------------------------------------------------ entries

// Entry e's operand and token.
__device__ __forceinline__ uint32_t token_of(const BankGradParams& p, uint32_t e, uint32_t& op) {
    const uint32_t first = p.tokens * p.width[0];
    op = e >= first;
    return op == 0 ? e / p.width[0] : (e - first) / p.width[1];
}
constexpr uint32_t kNone = 0xffffffffu;
// Its slot, or kNone where it does not count.
__device__ __forceinline__ uint32_t slot_of(const BankGradParams& p, uint32_t e) {
    uint32_t op;
    const uint32_t t = token_of(p, e, op), c = t / p.chunk;
    const int32_t limit = p.chunk_valid != nullptr ? p.chunk_valid[c] : int32_t(p.valid);
    if (int32_t(t - c * p.chunk) >= limit) return kNone;
    const uint32_t at = op == 0 ? e : e - p.tokens * p.width[0];
    const int64_t s = slot_at(op == 0 ? p.idx[0] : p.idx[1], at, p.idx64 ? 8 : 4);
    return uint64_t(s) < uint64_t(p.num_slots) ? uint32_t(s) : kNone;
}

// ------------------------------------------------------------------ sort

// Entry `at` (of the first pass: of the call; else of the sorted ones) and its slot.
template <bool FIRST>
__device__ __forceinline__ uint32_t key_at(const BankGradParams& p, int from, uint32_t at, uint32_t n) {
    if (at >= n) return kNone;
    return FIRST ? slot_of(p, at) : p.keys[from][at];
}

// How many entries of each tile have each digit.
template <bool FIRST> __global__ __launch_bounds__(kThreads) void sort_count_kernel(BankGradParams p, int pass) {
    __shared__ uint32_t count[kDigits];
    count[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t n = FIRST ? p.entries : *p.n;
    const int from = (pass - 1) & 1;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t key = key_at<FIRST>(p, from, blockIdx.x * uint32_t(kTile) + i * kThreads + threadIdx.x, n);
        if (key != kNone) atomicAdd(&count[key >> (8 * pass) & 255], 1u);
    }
    __syncthreads();
    p.hist[(int64_t(pass) * p.tiles + blockIdx.x) * kDigits + threadIdx.x] = count[threadIdx.x];
}

// For each digit, the entries of lower tiles that have it, in place, and of all of them.
constexpr int kScanDigits = 32, kScanParts = 32;
__global__ __launch_bounds__(kScanDigits * kScanParts) void sort_scan_kernel(BankGradParams p, int pass) {
    __shared__ uint32_t sums[kScanParts][kScanDigits];
    const int d = threadIdx.x % kScanDigits, part = threadIdx.x / kScanDigits;
    const int digit = int(blockIdx.x) * kScanDigits + d;
    uint32_t* hist = p.hist + int64_t(pass) * p.tiles * kDigits + digit;
    const int64_t each = (int64_t(p.tiles) + kScanParts - 1) / kScanParts;
    const int64_t begin = min(part * each, int64_t(p.tiles)), end = min(begin + each, int64_t(p.tiles));
    uint32_t sum = 0;
    for (int64_t i = begin; i < end; ++i) sum += hist[i * kDigits];
    sums[part][d] = sum;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int i = 0; i < kScanParts; ++i) {
        before += i < part ? sums[i][d] : 0;
        all += sums[i][d];
    }
    for (int64_t i = begin; i < end; ++i) {
        const uint32_t v = hist[i * kDigits];
        hist[i * kDigits] = before;
        before += v;
    }
    if (part == 0) p.total[pass * kDigits + digit] = all;
}

// Puts each entry of a tile in its place of the order by this pass's digit. A wavefront takes
// 64 neighbours at a time; the lanes of the same digit find one another by eight ballots.
template <bool FIRST> __global__ __launch_bounds__(kThreads) void sort_place_kernel(BankGradParams p, int pass) {
    __shared__ uint32_t count[kWaves][kDigits];
    __shared__ uint32_t wave_total[kWaves];
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    for (int w = 0; w < kWaves; ++w) count[w][tid] = 0;
    // Where each digit's entries of this tile begin.
    const uint32_t total = p.total[pass * kDigits + tid];
    uint32_t scan = total;
    for (int n = 1; n < 64; n *= 2) {
        const uint32_t o = __shfl_up(scan, n);
        if (lane >= n) scan += o;
    }
    if (lane == 63) wave_total[wave] = scan;
    __syncthreads();
    uint32_t all = 0, base = scan - total;
    for (int w = 0; w < kWaves; ++w) {
        base += w < wave ? wave_total[w] : 0;
        all += wave_total[w];
    }
    if (FIRST && blockIdx.x == 0 && tid == 0) *p.n = all;
    base += p.hist[(int64_t(pass) * p.tiles + blockIdx.x) * kDigits + tid];

    const uint32_t n = FIRST ? p.entries : all;
    const int from = (pass - 1) & 1, to = pass & 1;
    const uint32_t first = blockIdx.x * uint32_t(kTile) + wave * (64 * kItems) + lane;
    uint32_t key[kItems], id[kItems], rank[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t at = first + i * 64;
        key[i] = key_at<FIRST>(p, from, at, n);
        id[i] = FIRST || at >= n ? at : p.ids[from][at];
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t digit = key[i] >> (8 * pass) & 255;
        uint64_t same = __ballot(key[i] != kNone);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const uint64_t has = __ballot(digit >> b & 1);
            same &= digit >> b & 1 ? has : ~has;
        }
        const uint32_t below = __builtin_amdgcn_mbcnt_hi(uint32_t(same >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(same), 0));
        if (key[i] != kNone) {
            const uint32_t before = count[wave][digit];
            rank[i] = before + below;
            wave_lds_order();
            if (below == 0) count[wave][digit] = before + uint32_t(__popcll(same));
        }
        wave_lds_order();
    }
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) {
        const uint32_t v = count[w][tid];
        count[w][tid] = base;
        base += v;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (key[i] == kNone) continue;
        const uint32_t at = count[wave][key[i] >> (8 * pass) & 255] + rank[i];
        p.keys[to][at] = key[i];
        p.ids[to][at] = id[i];
    }
}

// ------------------------------------------------------------------ sums

// The sorted entries are cut into blocks, a lane group (a row's octets, or 64 of them) each.
// A run of equal slots that ends within `spill` entries past a block's end is taken by that
// block to its end, and the next begins behind it; of a longer one each block makes a partial
// sum, which join_kernel adds up. cont: block b's first run began in an earlier block and is
// not that block's alone.
__device__ __forceinline__ bool cont(const BankGradParams& p, const uint32_t* keys, uint32_t n, uint32_t b) {
    const uint64_t at = uint64_t(b) * p.block;
    return at > 0 && at + p.spill < n && keys[at - 1] == keys[at + p.spill];
}

template <typename E, int VB>
__device__ __forceinline__ void finish(const BankGradParams& p, uint32_t slot, int o, const float (&acc)[8]) {
    E* row = static_cast<E*>(p.dbank) + int64_t(slot) * p.hd + 8 * o;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = acc[j] * p.factor;
    if (p.add) {
        float old[8];
        load_octet<E, VB>(row, p.hd - 8 * o, old);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += old[j];
    }
    store_octet<E, VB>(row, p.hd - 8 * o, v);
}

__device__ __forceinline__ void store_partial(float* rows, uint32_t b, int octets, int o, const float (&acc)[8]) {
    float4* to = reinterpret_cast<float4*>(rows + (int64_t(b) * octets + o) * 8);
    to[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    to[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
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
__global__ __launch_bounds__(kThreads) void sum_kernel(BankGradParams p, int lanes) {
    extern __shared__ Term lds[];
    const int octets = (p.hd + 7) / 8;
    const int lane = int(threadIdx.x) % lanes, o = int(blockIdx.y) * lanes + lane;
    const uint32_t b = blockIdx.x * uint32_t(kThreads / lanes) + threadIdx.x / lanes;
    const uint32_t* keys = p.keys[(p.passes - 1) & 1];
    const uint32_t* ids = p.ids[(p.passes - 1) & 1];
    const uint32_t n = *p.n;
    const uint64_t begin = uint64_t(b) * p.block;
    if (begin >= n) return;
    const int staged = p.block + p.spill + 1;
    Term* terms = lds + int(threadIdx.x) / lanes * staged;
    const int there = int(min(uint64_t(staged), n - begin));
    for (int i = lane; i < there; i += lanes) {
        Term t;
        t.slot = keys[begin + i];
        const uint32_t e = ids[begin + i];
        t.token = token_of(p, e, t.op);
        t.w = 1.0f;
        if (WEIGHTS) t.w = value_at(t.op == 0 ? p.w[0] : p.w[1], t.op == 0 ? e : e - p.tokens * p.width[0], p.w_bf16 ? 2 : 4);
        terms[i] = t;
    }
    wave_lds_order();
    const bool from_before = cont(p, keys, n, b), goes_on = cont(p, keys, n, b + 1);
    int at = 0, end = min(p.block, there);
    if (begin > 0 && !from_before) {
        const uint32_t before = keys[begin - 1];
        while (at < there && terms[at].slot == before) ++at;
    }
    if (!goes_on)
        while (end < there && terms[end].slot == terms[p.block - 1].slot) ++end;
    if (o >= octets) return;
    PhiloxKey key = {};
    if (DROP) key = philox_key(p.dropout);
    float acc[8] = {};
    bool open = from_before;  // the run being added up began in an earlier block
    while (at < end) {
        const int count = min(end - at, kFlight);
        float x[kFlight][8];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const Term& t = terms[at + min(u, count - 1)];
            const D* row = static_cast<const D*>(t.op == 0 ? p.dout[0] : p.dout[1]) + int64_t(t.token) * p.hd;
            load_octet<D, DVB>(row + 8 * o, p.hd - 8 * o, x[u]);
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (u >= count) break;
            const Term t = terms[at + u];
            const uint32_t kept = DROP ? kept_columns(key, uint32_t(o), t.token, p.dropout.threshold) : 0xff;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (WEIGHTS) acc[j] = fmaf(t.w, x[u][j], acc[j]);
                else acc[j] += kept >> j & 1 ? x[u][j] : 0.0f;
            }
            const bool is_last = at + u + 1 == end;
            if (is_last || terms[at + u + 1].slot != t.slot) {
                if (open) store_partial(p.first, b, octets, o, acc);
                else if (is_last && goes_on) store_partial(p.last, b, octets, o, acc);
                else finish<E, VB>(p, t.slot, o, acc);
                open = false;
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
            }
        }
        at += count;
    }
}

// Runs over several blocks: the lane group of the block where one begins adds its partial sums.
template <typename E, int VB> __global__ __launch_bounds__(kThreads) void join_kernel(BankGradParams p, int lanes) {
    const int octets = (p.hd + 7) / 8;
    const int o = int(blockIdx.y) * lanes + int(threadIdx.x) % lanes;
    const uint32_t b = blockIdx.x * uint32_t(kThreads / lanes) + threadIdx.x / lanes;
    const uint32_t* keys = p.keys[(p.passes - 1) & 1];
    const uint32_t n = *p.n;
    const uint64_t begin = uint64_t(b) * p.block;
    if (begin >= n || o >= octets || !cont(p, keys, n, b + 1)) return;
    const uint32_t slot = keys[begin + p.block - 1];
    if (begin > 0 && keys[begin - 1] == slot) return;  // began in an earlier block
    float acc[8];
    load_octet<float, 16>(p.last + (int64_t(b) * octets + o) * 8, 8, acc);
    for (uint32_t c = b + 1; cont(p, keys, n, c) && keys[uint64_t(c) * p.block] == slot; ++c) {
        float x[8];
        load_octet<float, 16>(p.first + (int64_t(c) * octets + o) * 8, 8, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += x[j];
    }
    finish<E, VB>(p, slot, o, acc);
}

// ------------------------------------------------------------------ rows that no entry names

constexpr int kZeroBytes = 65536;  // of a workgroup's rows
constexpr int kZeroRows = 1024;    // at most

__device__ __forceinline__ uint32_t lower_bound(const uint32_t* keys, uint32_t n, uint64_t key) {
    uint32_t lo = 0, hi = n;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (keys[mid] < key) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

template <int VB> __global__ __launch_bounds__(kThreads) void zero_kernel(BankGradParams p, int rows, int64_t row_bytes) {
    __shared__ uint8_t named[kZeroRows];
    __shared__ uint32_t bounds[2];
    const uint32_t* keys = p.keys[(p.passes - 1) & 1];
    const uint32_t n = p.entries > 0 ? *p.n : 0;
    const int64_t first = int64_t(blockIdx.x) * rows;
    const int count = int(min(int64_t(rows), int64_t(p.num_slots) - first));
    for (int i = threadIdx.x; i < count; i += kThreads) named[i] = 0;
    if (threadIdx.x < 2) bounds[threadIdx.x] = lower_bound(keys, n, uint64_t(first) + (threadIdx.x == 0 ? 0 : count));
    __syncthreads();
    for (uint32_t i = bounds[0] + threadIdx.x; i < bounds[1]; i += kThreads) named[keys[i] - uint32_t(first)] = 1;
    __syncthreads();
    const int per_row = int(row_bytes / VB);
    char* base = static_cast<char*>(p.dbank) + first * row_bytes;
    using T = typename RawVec<VB>::T;
    for (int64_t v = threadIdx.x; v < int64_t(count) * per_row; v += kThreads)
        if (!named[v / per_row]) store_stream(reinterpret_cast<T*>(base) + v, T{});
}

// ------------------------------------------------------------------ launches

template <typename D, int DVB, typename E, int VB> void run_sums(const BankGradParams& p, hipStream_t stream) {
    const int octets = (p.hd + 7) / 8;
    int lanes = kMinLanes;
    while (lanes < 64 && lanes < octets) lanes *= 2;
    const int groups = kThreads / lanes;
    const dim3 grid{unsigned((p.blocks + groups - 1) / groups), unsigned((octets + lanes - 1) / lanes)}, block{kThreads};
    const size_t lds = size_t(groups) * size_t(p.block + p.spill + 1) * sizeof(Term);
    if (p.w[0] != nullptr) {
        if constexpr (sizeof(D) == 4) hipLaunchKernelGGL((sum_kernel<D, DVB, E, VB, true, false>), grid, block, lds, stream, p, lanes);
    } else if (p.dropout.threshold != 0) {
        hipLaunchKernelGGL((sum_kernel<D, DVB, E, VB, false, true>), grid, block, lds, stream, p, lanes);
    } else {
        hipLaunchKernelGGL((sum_kernel<D, DVB, E, VB, false, false>), grid, block, lds, stream, p, lanes);
    }
    hipLaunchKernelGGL((join_kernel<E, VB>), grid, block, 0, stream, p, lanes);
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

void run_sort(const BankGradParams& p, hipStream_t stream) {
    const dim3 tiles{p.tiles}, block{kThreads};
    for (int pass = 0; pass < p.passes; ++pass) {
        if (pass == 0) hipLaunchKernelGGL(sort_count_kernel<true>, tiles, block, 0, stream, p, pass);
        else hipLaunchKernelGGL(sort_count_kernel<false>, tiles, block, 0, stream, p, pass);
        hipLaunchKernelGGL(sort_scan_kernel, dim3(kDigits / kScanDigits), dim3(kScanDigits * kScanParts), 0, stream, p, pass);
        if (pass == 0) hipLaunchKernelGGL(sort_place_kernel<true>, tiles, block, 0, stream, p, pass);
        else hipLaunchKernelGGL(sort_place_kernel<false>, tiles, block, 0, stream, p, pass);
    }
}

}  // namespace

int64_t bank_grad_layout(BankGradParams* p, void* workspace) {
    const int64_t entries = p->entries, octets = (int64_t(p->hd) + 7) / 8;
    p->passes = 1;
    while (p->passes < 4 && (uint64_t(p->num_slots - 1) >> (8 * p->passes)) != 0) ++p->passes;
    p->tiles = uint32_t((entries + kTile - 1) / kTile);
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
    p->n = reinterpret_cast<uint32_t*>(place(4));
    p->total = reinterpret_cast<uint32_t*>(place(4 * int64_t(p->passes) * kDigits));
    p->hist = reinterpret_cast<uint32_t*>(place(4 * int64_t(p->passes) * p->tiles * kDigits));
    for (int i = 0; i < 2; ++i) {
        p->keys[i] = reinterpret_cast<uint32_t*>(place(4 * entries));
        p->ids[i] = reinterpret_cast<uint32_t*>(place(4 * entries));
    }
    p->first = reinterpret_cast<float*>(place(32 * octets * p->blocks));
    p->last = reinterpret_cast<float*>(place(32 * octets * p->blocks));
    return used;
}

int64_t bank_grad_groups(const BankGradParams& p, int bank_size) {
    const int64_t rows = zero_rows(int64_t(p.hd) * bank_size);
    return p.add ? 0 : (p.num_slots + rows - 1) / rows;  // those over entries are at most 2^31 / 64
}

hipError_t launch_bank_grad(const BankGradParams& p, bool dout_bf16, bool bank_bf16, hipStream_t stream) {
    const int64_t row_bytes = int64_t(p.hd) * (bank_bf16 ? 2 : 4);
    const bool bank_vec = (reinterpret_cast<uintptr_t>(p.dbank) | uintptr_t(row_bytes)) % 16 == 0;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.dout[0]) | (p.width[1] != 0 ? reinterpret_cast<uintptr_t>(p.dout[1]) : 0) |
                         uintptr_t(p.hd) * (dout_bf16 ? 2 : 4);
    if (p.entries > 0) run_sort(p, stream);
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
