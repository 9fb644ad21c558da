// The C ABI of the slot router and the packed bank (include/sdm_memory.h):
// argument checks and launches. Everything cheap is checked on the host before
// the first HIP call.

#include <math.h>

#include <new>
#include <unordered_map>
#include <vector>

#include "../../include/sdm_memory.h"
#include "sdm_host.h"
#include "sdm_memory.h"

namespace {

using namespace sdm;

using i64 = long long;

constexpr int64_t kMaxGatherColumns = 65535LL * 1024;  // column slices of a gather's grid, of 1024 columns at the widest
constexpr int64_t kMaxGridThreads = 0xffffffffLL;  // threads of a launch along one axis

bool is_value(int dtype) { return dtype == SDM_F32 || dtype == SDM_BF16; }
bool is_index(int dtype) { return dtype == SDM_I32 || dtype == SDM_I64; }
bool is_packed(int dtype) { return dtype == SDM_MX8 || dtype == SDM_MX4; }

struct Named {
    const void* p;
    const char* name;
    int64_t bytes;
};

int check_device_ptrs(const Named* list, size_t n) {
    for (size_t i = 0; i < n; ++i) {
        if (list[i].p == nullptr) continue;
        const int rc = check_device_ptr(list[i].p, list[i].name);
        if (rc != SDM_OK) return rc;
    }
    return SDM_OK;
}

// No written array shares memory with another array of the call.
int check_apart(const char* fn, const Named* written, size_t nw, const Named* read, size_t nr) {
    for (size_t i = 0; i < nw; ++i) {
        for (size_t j = i + 1; j < nw; ++j)
            if (overlap(written[i].p, written[i].bytes, written[j].p, written[j].bytes))
                return fail(SDM_E_OVERLAP, "%s: %s and %s share memory", fn, written[i].name, written[j].name);
        for (size_t j = 0; j < nr; ++j)
            if (overlap(written[i].p, written[i].bytes, read[j].p, read[j].bytes))
                return fail(SDM_E_OVERLAP, "%s: %s and %s share memory", fn, written[i].name, read[j].name);
    }
    return SDM_OK;
}

int launched(const char* fn, hipError_t e) {
    if (e != hipSuccess) return fail(SDM_E_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
    return ok();
}

// The checks that both directions of a route share. *run: there is something to launch.
int check_route(const char* fn, int logit_dtype, int64_t tokens, int64_t keys, int32_t k, int score, float scale,
                int64_t streams, int64_t stream_slots, int idx_dtype, int w_dtype, int64_t choice) {
    if (!is_value(logit_dtype))
        return fail(SDM_E_DTYPE, "%s: logits must be float32 or bfloat16 (dtype %d)", fn, logit_dtype);
    if (!is_index(idx_dtype)) return fail(SDM_E_DTYPE, "%s: idx must be int32 or int64 (dtype %d)", fn, idx_dtype);
    if (!is_value(w_dtype))
        return fail(SDM_E_DTYPE, "%s: weights must be float32 or bfloat16 (dtype %d)", fn, w_dtype);
    if (tokens < 0) return fail(SDM_E_SHAPE, "%s: tokens = %lld < 0", fn, (i64)tokens);
    if (tokens > SDM_MAX_ROUTE_TOKENS)
        return fail(SDM_E_SHAPE, "%s: at most 2^21 tokens per call, got %lld", fn, (i64)tokens);
    if (keys < 1 || keys > SDM_MAX_KEYS)
        return fail(SDM_E_RANGE, "%s: keys must be in 1..%d, got %lld", fn, SDM_MAX_KEYS, (i64)keys);
    if (k < 1 || k > SDM_MAX_WIDTH || k > choice)
        return fail(SDM_E_RANGE, "%s: k must be in 1..%d and at most the %lld keys to choose from, got %d", fn,
                    SDM_MAX_WIDTH, (i64)choice, k);
    if (score != SDM_SOFTMAX && score != SDM_SIGMOID)
        return fail(SDM_E_RANGE, "%s: score must be SDM_SOFTMAX or SDM_SIGMOID, got %d", fn, score);
    if (!std::isfinite(scale)) return fail(SDM_E_RANGE, "%s: scale must be finite", fn);
    if (streams < 1 || stream_slots < 0)
        return fail(SDM_E_SHAPE, "%s: streams = %lld, stream_slots = %lld: at least 1 and 0 are needed", fn,
                    (i64)streams, (i64)stream_slots);
    if (!mul_fits(streams, stream_slots))
        return fail(SDM_E_SHAPE, "%s: sizes overflow 64-bit byte counts", fn);
    const int64_t used = tokens < streams ? (tokens > 0 ? tokens : 1) : streams;  // streams that occur
    const int64_t last = (used - 1) * stream_slots;
    if (last > INT64_MAX - keys || (idx_dtype == SDM_I32 && last + keys - 1 > INT32_MAX))
        return fail(SDM_E_RANGE, "%s: the last slot does not fit idx's type", fn);
    return SDM_OK;
}

// The checks and the parameter block that the two passes over a gather's rows
// share: sdm_gather_packed and sdm_gather_weight_grad. `in` and `out` are each
// operand's value arrays, read and written, of in_bytes and out_bytes per token.
struct Rows {
    const void* bank;
    const void* scales;
    int dtype;
    int64_t num_slots, head_dim, tokens, chunk, valid;
    const int32_t* chunk_valid;
    int idx_dtype, w_dtype;
    const void* idx[2];
    const void* in[2];
    void* out[2];
    int32_t width[2];
    const char* names[3];  // of idx, in and out, without the operand's number
    bool in_is_weights;
};

int rows_call(const char* fn, const Rows& r, MemoryGatherParams* p, bool* run, hipStream_t stream) {
    *run = false;
    const bool packed = is_packed(r.dtype);
    if (!is_index(r.idx_dtype)) return fail(SDM_E_DTYPE, "%s: slots must be int32 or int64 (dtype %d)", fn, r.idx_dtype);
    if (!is_value(r.w_dtype))
        return fail(SDM_E_DTYPE, "%s: weights must be float32 or bfloat16 (dtype %d)", fn, r.w_dtype);
    if (r.num_slots < 1 || r.head_dim < 1)
        return fail(SDM_E_SHAPE, "%s: empty bank [%lld, %lld]: num_slots and head_dim must both be positive", fn,
                    (i64)r.num_slots, (i64)r.head_dim);
    if (r.head_dim > SDM_MAX_ROW_BYTES / 4)
        return fail(SDM_E_RANGE, "%s: head_dim %lld: a float32 row would exceed %lld bytes", fn, (i64)r.head_dim,
                    (i64)SDM_MAX_ROW_BYTES);
    if (r.tokens < 0 || r.chunk < 1 || r.tokens % r.chunk != 0 || r.valid < 0 || r.valid > r.chunk)
        return fail(SDM_E_SHAPE, "%s: tokens must be a whole number of chunks and valid lie in [0, chunk]: tokens=%lld "
                    "chunk=%lld valid=%lld", fn, (i64)r.tokens, (i64)r.chunk, (i64)r.valid);
    const int operands = r.idx[1] != nullptr || r.in[1] != nullptr || r.out[1] != nullptr || r.width[1] != 0 ? 2 : 1;
    for (int o = 0; o < operands; ++o) {
        if (o == 1 && r.tokens > 0 && (r.idx[1] == nullptr || r.in[1] == nullptr || r.out[1] == nullptr))
            return fail(SDM_E_NULL, "%s: operand 1 is given in part: pass %s1, %s1 and %s1 all, or none", fn, r.names[0],
                        r.names[1], r.names[2]);
        if (r.width[o] < 1 || r.width[o] > SDM_MAX_WIDTH)
            return fail(SDM_E_RANGE, "%s: width%d must be in 1..%d, got %d", fn, o, SDM_MAX_WIDTH, r.width[o]);
    }
    const int64_t row_bytes = packed ? sdm_packed_row_bytes(r.dtype, r.head_dim) : r.head_dim * elem_size(r.dtype);
    const int64_t scale_bytes = packed ? sdm_packed_scale_bytes(r.dtype, r.head_dim) : 0;
    if (!mul_fits(r.num_slots, row_bytes) || !mul_fits(r.num_slots, r.head_dim, 4) ||
        !mul_fits(r.tokens, SDM_MAX_WIDTH, r.head_dim * 8))
        return fail(SDM_E_SHAPE, "%s: sizes overflow 64-bit byte counts", fn);
    if (r.tokens == 0) return SDM_OK;
    if (r.bank == nullptr || (packed && r.scales == nullptr) || r.idx[0] == nullptr || r.in[0] == nullptr ||
        r.out[0] == nullptr)
        return fail(SDM_E_NULL, "%s: the bank, %s0, %s0 and %s0 are required", fn, r.names[0], r.names[1], r.names[2]);
    const int is = elem_size(r.idx_dtype), ws = elem_size(r.w_dtype);
    const int in_size = r.in_is_weights ? ws : 4, out_size = r.in_is_weights ? 4 : ws;
    if (!aligned(r.bank, packed ? 16 : elem_size(r.dtype)) || (packed && !aligned(r.scales, 4)))
        return fail(SDM_E_ALIGN, packed ? "%s: codes must be 16-byte and scales 4-byte aligned"
                                        : "%s: a pointer is not aligned to its element size", fn);
    bool fine = aligned(r.chunk_valid, 4);
    Named read[7] = {{r.bank, packed ? "codes" : "bank", r.num_slots * row_bytes},
                     {r.scales, "scales", r.num_slots * scale_bytes},
                     {r.chunk_valid, "chunk_valid", r.tokens / r.chunk * 4}};
    Named written[2] = {};
    for (int o = 0; o < operands; ++o) {
        const int64_t entries = r.tokens * r.width[o], dense = r.tokens * r.head_dim;
        fine = fine && aligned(r.idx[o], is) && aligned(r.in[o], in_size) && aligned(r.out[o], out_size);
        read[3 + 2 * o] = {r.idx[o], r.names[0], entries * is};
        read[4 + 2 * o] = {r.in[o], r.names[1], (r.in_is_weights ? entries : dense) * in_size};
        written[o] = {r.out[o], r.names[2], (r.in_is_weights ? dense : entries) * out_size};
    }
    if (!fine) return fail(SDM_E_ALIGN, "%s: a pointer is not aligned to its element size", fn);
    int rc = check_apart(fn, written, size_t(operands), read, size_t(3 + 2 * operands));
    if (rc != SDM_OK) return rc;
    if (debug_validate()) {
        try {
            rc = check_device_ptrs(read, size_t(3 + 2 * operands));
            if (rc == SDM_OK) rc = check_device_ptrs(written, size_t(operands));
            if (rc == SDM_OK)
                rc = validate_gather_slots(r.num_slots, r.tokens, r.chunk, r.valid, r.chunk_valid, r.idx[0], r.width[0],
                                           operands == 2 ? r.idx[1] : nullptr, r.width[1], r.idx_dtype, stream);
        } catch (const std::bad_alloc&) {
            rc = fail(SDM_E_HIP, "%s: no host memory to check the slots", fn);
        }
        if (rc != SDM_OK) return rc;
    }
    *p = MemoryGatherParams{};
    p->bank = r.bank;
    p->scales = static_cast<const uint8_t*>(r.scales);
    p->chunk_valid = r.chunk_valid;
    for (int o = 0; o < operands; ++o) {
        p->idx[o] = r.idx[o];
        p->width[o] = r.width[o];
        if (r.in_is_weights) {
            p->w[o] = r.in[o];
            p->out[o] = static_cast<float*>(r.out[o]);
        } else {
            p->dout[o] = static_cast<const float*>(r.in[o]);
            p->dw[o] = r.out[o];
        }
    }
    p->tokens = r.tokens;
    p->chunk = r.chunk;
    p->valid = r.valid;
    p->num_slots = r.num_slots;
    p->hd = int(r.head_dim);
    p->row_bytes = row_bytes;
    p->scale_bytes = int(scale_bytes);
    p->operands = operands;
    p->idx64 = r.idx_dtype == SDM_I64;
    p->w_bf16 = r.w_dtype == SDM_BF16;
    p->out_vec = r.head_dim % 4 == 0 && aligned(r.out[0], 16) && (operands == 1 || aligned(r.out[1], 16));
    // A pair of a token and an operand takes at most 64 threads of a launch.
    if (r.tokens > (kMaxGridThreads - 256) / (64 * operands))
        return fail(SDM_E_SHAPE, "%s: %lld tokens exceed the grid", fn, (i64)r.tokens);
    *run = true;
    return SDM_OK;
}

// A slot given twice is given the same row each time.
int validate_pack(int64_t n, const void* row_idx, const void* slots, int idx_dtype, int64_t num_rows, int64_t num_slots,
                  hipStream_t stream) {
    std::vector<int64_t> from, to;
    int rc = fetch_slots(slots, idx_dtype, n, to, stream, "slots");
    if (rc == SDM_OK && row_idx != nullptr) rc = fetch_slots(row_idx, idx_dtype, n, from, stream, "row_idx");
    if (rc != SDM_OK) return rc;
    std::unordered_map<int64_t, int64_t> owner;
    for (int64_t i = 0; i < n; ++i) {
        const int64_t s = to[size_t(i)], r = row_idx != nullptr ? from[size_t(i)] : i;
        if (s < 0 || s >= num_slots || r < 0 || r >= num_rows) continue;
        const auto it = owner.emplace(s, r).first;
        if (it->second != r)
            return fail(SDM_E_RANGE, "sdm_bank_pack: slot %lld is given rows %lld and %lld", (i64)s, (i64)it->second,
                        (i64)r);
    }
    return SDM_OK;
}

}  // namespace

extern "C" {

int64_t sdm_packed_row_bytes(int packed_dtype, int64_t head_dim) {
    if (!is_packed(packed_dtype) || head_dim < 1 || head_dim > SDM_MAX_ROW_BYTES) return 0;
    const int64_t bytes = packed_dtype == SDM_MX8 ? head_dim : (head_dim + 1) / 2;
    return (bytes + 15) / 16 * 16;
}

int64_t sdm_packed_scale_bytes(int packed_dtype, int64_t head_dim) {
    if (!is_packed(packed_dtype) || head_dim < 1 || head_dim > SDM_MAX_ROW_BYTES) return 0;
    return ((head_dim + SDM_PACK_BLOCK - 1) / SDM_PACK_BLOCK + 3) / 4 * 4;
}

int sdm_route(const void* logits, int logit_dtype, int64_t tokens, int64_t keys, int32_t k, int score,
              const float* bias, int32_t groups, int32_t kept_groups, int32_t group_top, int32_t normalise,
              float scale, int64_t streams, int64_t stream_slots, void* idx, int idx_dtype, void* w, int w_dtype,
              void* hip_stream) {
    const char* fn = "sdm_route";
    if (groups < 1 || groups > SDM_MAX_GROUPS || kept_groups < 1 || kept_groups > groups)
        return fail(SDM_E_RANGE, "%s: groups must be in 1..%d and kept_groups in 1..groups, got %d and %d", fn,
                    SDM_MAX_GROUPS, groups, kept_groups);
    if (group_top != 1 && group_top != 2) return fail(SDM_E_RANGE, "%s: group_top must be 1 or 2, got %d", fn, group_top);
    const int64_t choice = keys < 1 || keys > SDM_MAX_KEYS ? 0 : keys / groups * kept_groups;
    if (keys >= 1 && keys <= SDM_MAX_KEYS && keys % groups != 0)
        return fail(SDM_E_SHAPE, "%s: %d groups do not divide %lld keys", fn, groups, (i64)keys);
    int rc = check_route(fn, logit_dtype, tokens, keys, k, score, scale, streams, stream_slots, idx_dtype, w_dtype,
                         choice);
    if (rc != SDM_OK) return rc;
    if (tokens == 0) return ok();
    if (logits == nullptr || idx == nullptr || w == nullptr)
        return fail(SDM_E_NULL, "%s: logits, idx and w are required", fn);
    const int es = elem_size(logit_dtype), is = elem_size(idx_dtype), ws = elem_size(w_dtype);
    if (!aligned(logits, es) || !aligned(bias, 4) || !aligned(idx, is) || !aligned(w, ws))
        return fail(SDM_E_ALIGN, "%s: a pointer is not aligned to its element size", fn);
    const Named read[] = {{logits, "logits", tokens * keys * es}, {bias, "bias", keys * 4}};
    const Named written[] = {{idx, "idx", tokens * k * is}, {w, "w", tokens * k * ws}};
    rc = check_apart(fn, written, 2, read, 2);
    if (rc != SDM_OK) return rc;
    if (debug_validate()) {
        rc = check_device_ptrs(read, 2);
        if (rc == SDM_OK) rc = check_device_ptrs(written, 2);
        if (rc != SDM_OK) return rc;
    }
    RouteParams p{};
    p.logits = logits;
    p.bias = bias;
    p.tokens = tokens;
    p.keys = int(keys);
    p.k = k;
    p.score = score;
    p.groups = groups;
    p.kept = kept_groups;
    p.top = group_top;
    p.normalise = normalise != 0;
    p.scale = scale;
    p.streams = uint32_t(streams < UINT32_MAX ? streams : UINT32_MAX);
    p.stream_slots = stream_slots;
    p.idx = idx;
    p.w = w;
    p.idx64 = idx_dtype == SDM_I64;
    p.w_bf16 = w_dtype == SDM_BF16;
    return launched(fn, launch_route(p, logit_dtype == SDM_BF16, static_cast<hipStream_t>(hip_stream)));
}

int sdm_route_backward(const void* logits, int logit_dtype, int64_t tokens, int64_t keys, int32_t k, int score,
                       const float* bias, int32_t normalise, float scale, int64_t streams, int64_t stream_slots,
                       const void* idx, int idx_dtype, const void* dw, int w_dtype, void* dlogits, void* hip_stream) {
    const char* fn = "sdm_route_backward";
    int rc = check_route(fn, logit_dtype, tokens, keys, k, score, scale, streams, stream_slots, idx_dtype, w_dtype,
                         keys);
    if (rc != SDM_OK) return rc;
    if (tokens == 0) return ok();
    if (logits == nullptr || idx == nullptr || dw == nullptr || dlogits == nullptr)
        return fail(SDM_E_NULL, "%s: logits, idx, dw and dlogits are required", fn);
    const int es = elem_size(logit_dtype), is = elem_size(idx_dtype), ws = elem_size(w_dtype);
    if (!aligned(logits, es) || !aligned(bias, 4) || !aligned(idx, is) || !aligned(dw, ws) || !aligned(dlogits, es))
        return fail(SDM_E_ALIGN, "%s: a pointer is not aligned to its element size", fn);
    const Named read[] = {{logits, "logits", tokens * keys * es},
                          {bias, "bias", keys * 4},
                          {idx, "idx", tokens * k * is},
                          {dw, "dw", tokens * k * ws}};
    const Named written[] = {{dlogits, "dlogits", tokens * keys * es}};
    rc = check_apart(fn, written, 1, read, 4);
    if (rc != SDM_OK) return rc;
    if (debug_validate()) {
        rc = check_device_ptrs(read, 4);
        if (rc == SDM_OK) rc = check_device_ptrs(written, 1);
        if (rc != SDM_OK) return rc;
    }
    RouteBackwardParams p{};
    p.logits = logits;
    p.bias = bias;
    p.tokens = tokens;
    p.keys = int(keys);
    p.k = k;
    p.score = score;
    p.normalise = normalise != 0;
    p.scale = scale;
    p.streams = uint32_t(streams < UINT32_MAX ? streams : UINT32_MAX);
    p.stream_slots = stream_slots;
    p.idx = idx;
    p.dw = dw;
    p.dlogits = dlogits;
    p.idx64 = idx_dtype == SDM_I64;
    p.w_bf16 = w_dtype == SDM_BF16;
    return launched(fn, launch_route_backward(p, logit_dtype == SDM_BF16, static_cast<hipStream_t>(hip_stream)));
}

int sdm_bank_pack(void* codes, void* scales, int packed_dtype, int64_t num_slots, int64_t head_dim, const void* rows,
                  int row_dtype, int64_t num_rows, int64_t n, const void* row_idx, const void* slots, int idx_dtype,
                  void* hip_stream) {
    const char* fn = "sdm_bank_pack";
    hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    if (!is_packed(packed_dtype))
        return fail(SDM_E_DTYPE, "%s: the bank must be SDM_MX8 or SDM_MX4 (dtype %d)", fn, packed_dtype);
    if (!is_value(row_dtype)) return fail(SDM_E_DTYPE, "%s: rows must be float32 or bfloat16 (dtype %d)", fn, row_dtype);
    if (!is_index(idx_dtype))
        return fail(SDM_E_DTYPE, "%s: row_idx and slots must be int32 or int64 (dtype %d)", fn, idx_dtype);
    if (num_slots < 1 || head_dim < 1)
        return fail(SDM_E_SHAPE, "%s: empty bank [%lld, %lld]: num_slots and head_dim must both be positive", fn,
                    (i64)num_slots, (i64)head_dim);
    if (head_dim > SDM_MAX_ROW_BYTES / 4)
        return fail(SDM_E_RANGE, "%s: head_dim %lld: a float32 row would exceed %lld bytes", fn, (i64)head_dim,
                    (i64)SDM_MAX_ROW_BYTES);
    if (num_rows < 0 || n < 0) return fail(SDM_E_SHAPE, "%s: num_rows = %lld, n = %lld < 0", fn, (i64)num_rows, (i64)n);
    if (!mul_fits(num_slots, head_dim, 4) || !mul_fits(num_rows, head_dim, 4) || !mul_fits(n, 8))
        return fail(SDM_E_SHAPE, "%s: sizes overflow 64-bit byte counts", fn);
    if (row_idx == nullptr && n > num_rows)
        return fail(SDM_E_SHAPE, "%s: n = %lld rows of %lld", fn, (i64)n, (i64)num_rows);
    if (slots == nullptr && n > num_slots)
        return fail(SDM_E_SHAPE, "%s: n = %lld rows into %lld slots", fn, (i64)n, (i64)num_slots);
    if (n == 0 || num_rows == 0) return ok();
    if (codes == nullptr || scales == nullptr || rows == nullptr)
        return fail(SDM_E_NULL, "%s: codes, scales and rows are required", fn);
    const int es = elem_size(row_dtype), is = elem_size(idx_dtype);
    if (!aligned(codes, 16) || !aligned(scales, 4))
        return fail(SDM_E_ALIGN, "%s: codes must be 16-byte and scales 4-byte aligned", fn);
    if (!aligned(rows, es) || !aligned(row_idx, is) || !aligned(slots, is))
        return fail(SDM_E_ALIGN, "%s: a pointer is not aligned to its element size", fn);
    const int64_t row_bytes = sdm_packed_row_bytes(packed_dtype, head_dim);
    const int64_t scale_bytes = sdm_packed_scale_bytes(packed_dtype, head_dim);
    const Named read[] = {{rows, "rows", num_rows * head_dim * es}, {row_idx, "row_idx", n * is}, {slots, "slots", n * is}};
    const Named written[] = {{codes, "codes", num_slots * row_bytes}, {scales, "scales", num_slots * scale_bytes}};
    int rc = check_apart(fn, written, 2, read, 3);
    if (rc != SDM_OK) return rc;
    if (debug_validate()) {
        try {
            rc = check_device_ptrs(read, 3);
            if (rc == SDM_OK) rc = check_device_ptrs(written, 2);
            if (rc == SDM_OK && slots != nullptr)
                rc = validate_pack(n, row_idx, slots, idx_dtype, num_rows, num_slots, stream);
        } catch (const std::bad_alloc&) {
            rc = fail(SDM_E_HIP, "%s: no host memory to check the slots", fn);
        }
        if (rc != SDM_OK) return rc;
    }
    PackParams p{};
    p.codes = static_cast<uint8_t*>(codes);
    p.scales = static_cast<uint8_t*>(scales);
    p.rows = rows;
    p.row_idx = row_idx;
    p.slots = slots;
    p.num_slots = num_slots;
    p.num_rows = num_rows;
    p.n = n;
    p.hd = int(head_dim);
    p.row_bytes = int(row_bytes);
    p.scale_bytes = int(scale_bytes);
    p.idx64 = idx_dtype == SDM_I64;
    return launched(fn, launch_pack(p, row_dtype == SDM_BF16, packed_dtype == SDM_MX4, stream));
}

int sdm_gather_packed(const void* codes, const void* scales, int packed_dtype, int64_t num_slots, int64_t head_dim,
                      int64_t tokens, int64_t chunk, int64_t valid, const int32_t* chunk_valid, int idx_dtype,
                      int w_dtype, const void* idx0, const void* w0, int32_t width0, float* out0, const void* idx1,
                      const void* w1, int32_t width1, float* out1, void* hip_stream) {
    const char* fn = "sdm_gather_packed";
    if (!is_packed(packed_dtype))
        return fail(SDM_E_DTYPE, "%s: the bank must be SDM_MX8 or SDM_MX4 (dtype %d)", fn, packed_dtype);
    const Rows r = {codes, scales, packed_dtype, num_slots, head_dim, tokens, chunk, valid, chunk_valid, idx_dtype,
                    w_dtype, {idx0, idx1}, {w0, w1}, {out0, out1}, {width0, width1}, {"idx", "w", "out"}, true};
    if (head_dim > kMaxGatherColumns)
        return fail(SDM_E_RANGE, "%s: head_dim %lld exceeds the grid's %lld columns", fn, (i64)head_dim,
                    (i64)kMaxGatherColumns);
    hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    MemoryGatherParams p;
    bool run;
    const int rc = rows_call(fn, r, &p, &run, stream);
    if (rc != SDM_OK || !run) return rc == SDM_OK ? ok() : rc;
    return launched(fn, launch_gather_packed(p, packed_dtype == SDM_MX4, stream));
}

int sdm_gather_weight_grad(const void* bank, const void* scales, int bank_dtype, int64_t num_slots, int64_t head_dim,
                           int64_t tokens, int64_t chunk, int64_t valid, const int32_t* chunk_valid, int idx_dtype,
                           int w_dtype, const void* idx0, const float* dout0, int32_t width0, void* dw0,
                           const void* idx1, const float* dout1, int32_t width1, void* dw1, void* hip_stream) {
    const char* fn = "sdm_gather_weight_grad";
    if (!is_packed(bank_dtype) && !is_value(bank_dtype))
        return fail(SDM_E_DTYPE, "%s: the bank must be float32, bfloat16, SDM_MX8 or SDM_MX4 (dtype %d)", fn, bank_dtype);
    const Rows r = {bank, is_packed(bank_dtype) ? scales : nullptr, bank_dtype, num_slots, head_dim, tokens, chunk,
                    valid, chunk_valid, idx_dtype, w_dtype, {idx0, idx1}, {dout0, dout1}, {dw0, dw1},
                    {width0, width1}, {"idx", "dout", "dw"}, false};
    hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    MemoryGatherParams p;
    bool run;
    const int rc = rows_call(fn, r, &p, &run, stream);
    if (rc != SDM_OK || !run) return rc == SDM_OK ? ok() : rc;
    return launched(fn, launch_weight_grad(p, bank_dtype, stream));
}

}  // extern "C"
