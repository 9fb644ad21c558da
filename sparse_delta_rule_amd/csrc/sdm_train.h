// Internal declarations of what trains a router and a bank: launch parameter blocks,
// the layouts of the workspaces, and the launchers that the C ABI calls.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdm {

// n / d of n < 2^31 by a product: mul = ceil(2^shift / d), shift = 31 + ceil(log2 d), is
// less than 2^32 and near enough for every such n (Granlund and Montgomery, 1994).
struct Divisor {
    uint32_t mul, shift;
};
inline Divisor divisor(uint32_t d) {
    Divisor r{0, 31};
    if (d == 0) return r;  // never divided by
    while ((uint64_t(1) << (r.shift - 31)) < d) ++r.shift;
    r.mul = uint32_t(((uint64_t(1) << r.shift) + d - 1) / d);
    return r;
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor& d) {
    return uint32_t(uint64_t(n) * d.mul >> d.shift);
}


// ------------------------------------------------------------------ balance
// A piece is a run of tokens of one sequence, which one workgroup reads: at most 255, so
// that a key's count in it fits 16 bits (255 * SDM_MAX_WIDTH < 2^16).
constexpr int kMaxPiece = 255;

struct BalanceParams {
    const void* logits;
    const int32_t* chunk_valid;
    uint32_t tokens, chunk, valid;
    Divisor by_chunk, by_k;
    int keys, k, score;
    int per_chunk, piece;
    uint32_t sequence;  // tokens of a sequence
    uint32_t sequences, pieces;  // pieces of each sequence
    double scale;
    uint32_t streams;
    int64_t stream_slots;
    const void* idx;
    int idx64;
    int32_t* counts;
    float* mean;
    float* coef;
    float* loss;
    // workspace
    uint32_t* done;       // [1] workgroups of the second pass that have ended
    uint32_t* live;       // [sequences * pieces]
    uint32_t* live_all;   // [sequences]
    double* loss_part;    // [sequences * key blocks]
    float* part;          // [sequences * pieces, keys] sums of shares
    uint32_t* part_count; // [sequences * pieces, (keys + 1) / 2] counts, two of 16 bits a word
    // backward
    const float* dloss;
    void* dlogits;
    int accumulate;
};
// Splits the tokens into pieces and, where `workspace` is given, places its arrays; returns the
// workspace's bytes.
int64_t balance_layout(BalanceParams* p, void* workspace);
hipError_t launch_balance(const BalanceParams& p, bool bf16, hipStream_t stream);
hipError_t launch_balance_backward(const BalanceParams& p, bool bf16, hipStream_t stream);

// ------------------------------------------------------------------ lookup
// The random bits of a lookup's columns; see sdm_lookup.
struct Dropout {
    const uint64_t* rng;
    uint32_t threshold;  // 0: none
};

struct LookupParams {
    const void* bank;
    const uint8_t* scales;
    int64_t num_slots, n;
    int64_t first;  // of the launch's rows
    int hd;
    int64_t row_bytes;
    int scale_bytes;
    const void* idx;
    int idx64;
    float factor;
    Dropout dropout;
    void* out;
};
int64_t lookup_groups(const LookupParams& p);  // workgroups for a slice of the columns
hipError_t launch_lookup(const LookupParams& p, int bank_dtype, bool out_bf16, hipStream_t stream);

// ------------------------------------------------------------------ gradient to a bank
// An entry as it is sorted: its slot, and its token with its operand in the top bit.
struct Record {
    uint32_t slot, token;
};
constexpr uint32_t kSecond = 0x80000000u;  // operand 1

struct BankGradParams {
    const void* idx[2];
    const void* w[2];     // NULL: 1 (a lookup)
    const void* dout[2];
    uint32_t width[2];    // width[1] = 0: one operand
    uint32_t tokens, chunk, valid;
    const int32_t* chunk_valid;
    int idx64, w_bf16;
    float factor;
    Dropout dropout;
    void* dbank;
    uint32_t num_slots;
    int hd;
    int add;
    // from the sizes
    uint32_t entries;
    uint32_t first_entries;  // of operand 0
    Divisor by_width[2], by_chunk;
    int passes, bits;     // of the sort, and of a slot in a pass
    int items;            // entries of a thread of the sort; 0: one workgroup sorts them all
    uint32_t tiles;       // of 256 * items entries
    int block, spill;     // entries of a lane group; how far it may go past their end
    uint32_t blocks;
    int64_t zero_bytes;   // of dbank, zeroed beside the sort
    int turn;             // columns that are summed at a time: all, or a multiple of 64
    int line, columns;    // the first of this turn's, in 64s, and the end of them
    // workspace
    uint32_t* n;          // [1] entries that count
    int64_t stride;       // of the counts of a digit
    uint32_t* hist;       // [passes, tiles, 2^bits], or [passes, 2^bits, stride] where they are scanned
    uint32_t* total;      // [passes, 2^bits]
    Record* records[2];   // [entries]
    float* weights[2];    // [entries] (a gather)
    float* first;         // [blocks, turn] sums of a run that began in an earlier block
    float* last;          // [blocks, turn] of one that goes on in the next
};
// From entries, num_slots and hd: the other sizes and, where `workspace` is given, the places of
// its arrays; returns the workspace's bytes.
int64_t bank_grad_layout(BankGradParams* p, void* workspace);
// Workgroups of the largest launch; the sizes are set.
int64_t bank_grad_groups(const BankGradParams& p, int dout_size, int bank_size);
hipError_t launch_bank_grad(const BankGradParams& p, bool dout_bf16, bool bank_bf16, hipStream_t stream);

}  // namespace sdm
