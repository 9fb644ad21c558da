// The C ABI of a route's balance, of lookups and of the gradients to a bank
// (include/sdm_train.h): argument checks and launches. Everything cheap is checked on the
// host before the first HIP call.

#include <math.h>

#include "../../include/sdm_train.h"
#include "sdm_check.h"
#include "sdm_host.h"
#include "sdm_train.h"

namespace {

using namespace sdm;

using i64 = long long;

constexpr int64_t kMaxColumns = 65535LL * 256;  // slices along y of a grid: 256 columns where runs are joined
constexpr int64_t kMaxGroups = 0xffffffffLL / 256;  // workgroups of 256 threads along one axis
constexpr int64_t kMaxLookupGroups = 1LL << 26;  // of a lookup's launches: 288 GiB of 2-byte outputs take 3.8e7 at most

// The workspace is there, large enough and apart from the call's arrays (`read` and `written`
// hold them; the workspace becomes the last of `written`).
int check_workspace(const char* fn, const void* workspace, int64_t bytes, int64_t needed, Named* written, size_t nw,
                    const Named* read, size_t nr) {
    if (workspace == nullptr) return fail(SDM_E_NULL, "%s: workspace is required", fn);
    if (bytes < needed)
        return fail(SDM_E_SHAPE, "%s: the workspace has %lld bytes, %lld are needed", fn, (i64)bytes, (i64)needed);
    if (!aligned(workspace, 16)) return fail(SDM_E_ALIGN, "%s: workspace must be 16-byte aligned", fn);
    written[nw] = {workspace, "workspace", needed};
    return check_apart(fn, written, nw + 1, read, nr);
}

// ------------------------------------------------------------------ balance

int check_balance(const char* fn, int logit_dtype, int64_t tokens, int64_t keys, int score, int64_t chunk, int64_t valid) {
    if (!is_value(logit_dtype))
        return fail(SDM_E_DTYPE, "%s: logits must be float32 or bfloat16 (dtype %d)", fn, logit_dtype);
    if (tokens < 0) return fail(SDM_E_SHAPE, "%s: tokens = %lld < 0", fn, (i64)tokens);
    if (tokens > SDM_MAX_ROUTE_TOKENS)
        return fail(SDM_E_SHAPE, "%s: at most 2^21 tokens per call, got %lld", fn, (i64)tokens);
    if (keys < 1 || keys > SDM_MAX_KEYS)
        return fail(SDM_E_RANGE, "%s: keys must be in 1..%d, got %lld", fn, SDM_MAX_KEYS, (i64)keys);
    if (score != SDM_SOFTMAX && score != SDM_SIGMOID)
        return fail(SDM_E_RANGE, "%s: score must be SDM_SOFTMAX or SDM_SIGMOID, got %d", fn, score);
    if (chunk < 1 || tokens % chunk != 0 || valid < 0 || valid > chunk)
        return fail(SDM_E_SHAPE, "%s: tokens must be a whole number of chunks and valid lie in [0, chunk]: tokens=%lld "
                    "chunk=%lld valid=%lld", fn, (i64)tokens, (i64)chunk, (i64)valid);
    return SDM_OK;
}

BalanceParams balance_params(const void* logits, int64_t tokens, int64_t keys, int score, int64_t chunk, int64_t valid,
                             const int32_t* chunk_valid, int32_t per_chunk) {
    BalanceParams p{};
    p.logits = logits;
    p.chunk_valid = chunk_valid;
    p.tokens = uint32_t(tokens);
    p.chunk = uint32_t(chunk < UINT32_MAX ? chunk : UINT32_MAX);  // past the tokens only where there are none
    p.valid = uint32_t(valid < INT32_MAX ? valid : INT32_MAX);
    p.keys = int(keys);
    p.score = score;
    p.per_chunk = per_chunk != 0;
    return p;
}

// ------------------------------------------------------------------ lookups

// *threshold: of 65536 equally likely values, those that drop a column; *factor: what the others are scaled by.
int check_dropout(const char* fn, float scale, float dropout, const uint64_t* rng, bool run, uint32_t* threshold,
                  float* factor) {
    if (!std::isfinite(scale)) return fail(SDM_E_RANGE, "%s: scale must be finite", fn);
    if (!(dropout >= 0.0f && dropout <= 1.0f - 0x1p-16f))
        return fail(SDM_E_RANGE, "%s: dropout must be in [0, 1 - 2^-16], got %g", fn, double(dropout));
    *threshold = uint32_t(nearbyint(double(dropout) * 65536.0));
    *factor = float(double(scale) * 65536.0 / (65536.0 - double(*threshold)));
    if (!std::isfinite(*factor))
        return fail(SDM_E_RANGE, "%s: scale / (1 - dropout) must be finite in float32, got %g / (1 - %g)", fn, double(scale),
                    double(dropout));
    if (*threshold != 0 && run && rng == nullptr) return fail(SDM_E_NULL, "%s: dropout needs rng", fn);
    if (!aligned(rng, 8)) return fail(SDM_E_ALIGN, "%s: rng must be 8-byte aligned", fn);
    return SDM_OK;
}

int check_bank(const char* fn, int64_t num_slots, int64_t head_dim) {
    if (num_slots < 1 || head_dim < 1)
        return fail(SDM_E_SHAPE, "%s: empty bank [%lld, %lld]: num_slots and head_dim must both be positive", fn,
                    (i64)num_slots, (i64)head_dim);
    if (head_dim > kMaxColumns)
        return fail(SDM_E_RANGE, "%s: head_dim must be at most %lld, got %lld", fn, (i64)kMaxColumns, (i64)head_dim);
    if (!mul_fits(num_slots, head_dim, 4)) return fail(SDM_E_SHAPE, "%s: sizes overflow 64-bit byte counts", fn);
    return SDM_OK;
}

int check_grad(const char* fn, int bank_dtype, int64_t num_slots, int64_t head_dim, int mode) {
    if (!is_value(bank_dtype))
        return fail(SDM_E_DTYPE, "%s: dbank must be float32 or bfloat16 (dtype %d)", fn, bank_dtype);
    const int rc = check_bank(fn, num_slots, head_dim);
    if (rc != SDM_OK) return rc;
    if (num_slots > SDM_MAX_GRAD_ENTRIES)
        return fail(SDM_E_RANGE, "%s: at most 2^31 - 1 slots, got %lld", fn, (i64)num_slots);
    if (mode != SDM_GRAD_WRITE && mode != SDM_GRAD_ADD)
        return fail(SDM_E_RANGE, "%s: mode must be SDM_GRAD_WRITE or SDM_GRAD_ADD, got %d", fn, mode);
    return SDM_OK;
}

}  // namespace

extern "C" {

int64_t sdm_route_balance_workspace(int64_t tokens, int64_t keys, int64_t chunk, int32_t per_chunk) {
    if (tokens < 0 || tokens > SDM_MAX_ROUTE_TOKENS || keys < 1 || keys > SDM_MAX_KEYS || chunk < 1 || tokens % chunk != 0)
        return 0;
    BalanceParams p = balance_params(nullptr, tokens, keys, SDM_SOFTMAX, chunk, 0, nullptr, per_chunk);
    return balance_layout(&p, nullptr);
}

int sdm_route_balance(const void* logits, int logit_dtype, int64_t tokens, int64_t keys, int32_t k, int score,
                      int64_t chunk, int64_t valid, const int32_t* chunk_valid, int32_t per_chunk, float scale,
                      int64_t streams, int64_t stream_slots, const void* idx, int idx_dtype, int32_t* counts,
                      float* mean, float* coef, float* loss, void* workspace, int64_t workspace_bytes,
                      void* hip_stream) {
    const char* fn = "sdm_route_balance";
    int rc = check_balance(fn, logit_dtype, tokens, keys, score, chunk, valid);
    if (rc != SDM_OK) return rc;
    if (!is_index(idx_dtype)) return fail(SDM_E_DTYPE, "%s: idx must be int32 or int64 (dtype %d)", fn, idx_dtype);
    if (k < 1 || k > SDM_MAX_WIDTH || k > keys)
        return fail(SDM_E_RANGE, "%s: k must be in 1..%d and at most the %lld keys, got %d", fn, SDM_MAX_WIDTH, (i64)keys, k);
    if (!std::isfinite(scale)) return fail(SDM_E_RANGE, "%s: scale must be finite", fn);
    if (streams < 1 || stream_slots < 0)
        return fail(SDM_E_SHAPE, "%s: streams = %lld, stream_slots = %lld: at least 1 and 0 are needed", fn,
                    (i64)streams, (i64)stream_slots);
    if (!mul_fits(streams, stream_slots)) return fail(SDM_E_SHAPE, "%s: sizes overflow 64-bit byte counts", fn);
    BalanceParams p = balance_params(logits, tokens, keys, score, chunk, valid, chunk_valid, per_chunk);
    const int64_t needed = balance_layout(&p, workspace);
    if (loss == nullptr || (p.sequences > 0 && (counts == nullptr || mean == nullptr || coef == nullptr)) ||
        (tokens > 0 && (logits == nullptr || idx == nullptr)))
        return fail(SDM_E_NULL, "%s: logits, idx, counts, mean, coef and loss are required", fn);
    const int es = elem_size(logit_dtype), is = elem_size(idx_dtype);
    if (!aligned(logits, es) || !aligned(idx, is) || !aligned(chunk_valid, 4) || !aligned(counts, 4) || !aligned(mean, 4) ||
        !aligned(coef, 4) || !aligned(loss, 4))
        return fail(SDM_E_ALIGN, "%s: a pointer is not aligned to its element size", fn);
    const int64_t table = int64_t(p.sequences) * keys * 4;
    const Named read[] = {{logits, "logits", tokens * keys * es},
                          {idx, "idx", tokens * k * is},
                          {chunk_valid, "chunk_valid", tokens / chunk * 4}};
    Named written[5] = {{counts, "counts", table}, {mean, "mean", table}, {coef, "coef", int64_t(p.sequences) * 4},
                        {loss, "loss", 4}};
    rc = check_workspace(fn, workspace, workspace_bytes, needed, written, 4, read, 3);
    if (rc != SDM_OK) return rc;
    if (debug_validate()) {
        rc = check_device_ptrs(read, tokens > 0 ? 3 : 0);
        if (rc == SDM_OK) rc = check_device_ptrs(written, 5);
        if (rc != SDM_OK) return rc;
    }
    p.k = k;
    p.by_k = divisor(uint32_t(k));
    p.scale = scale;
    p.streams = uint32_t(streams < UINT32_MAX ? streams : UINT32_MAX);
    p.stream_slots = stream_slots;
    p.idx = idx;
    p.idx64 = idx_dtype == SDM_I64;
    p.counts = counts;
    p.mean = mean;
    p.coef = coef;
    p.loss = loss;
    return launched(fn, launch_balance(p, logit_dtype == SDM_BF16, static_cast<hipStream_t>(hip_stream)));
}

int sdm_route_balance_backward(const void* logits, int logit_dtype, int64_t tokens, int64_t keys, int score,
                               int64_t chunk, int64_t valid, const int32_t* chunk_valid, int32_t per_chunk,
                               const int32_t* counts, const float* coef, const float* dloss, int32_t accumulate,
                               void* dlogits, void* hip_stream) {
    const char* fn = "sdm_route_balance_backward";
    int rc = check_balance(fn, logit_dtype, tokens, keys, score, chunk, valid);
    if (rc != SDM_OK) return rc;
    if (tokens == 0) return ok();
    if (logits == nullptr || counts == nullptr || coef == nullptr || dlogits == nullptr)
        return fail(SDM_E_NULL, "%s: logits, counts, coef and dlogits are required", fn);
    const int es = elem_size(logit_dtype);
    if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(chunk_valid, 4) || !aligned(counts, 4) ||
        !aligned(coef, 4) || !aligned(dloss, 4))
        return fail(SDM_E_ALIGN, "%s: a pointer is not aligned to its element size", fn);
    BalanceParams p = balance_params(logits, tokens, keys, score, chunk, valid, chunk_valid, per_chunk);
    balance_layout(&p, nullptr);
    const Named read[] = {{logits, "logits", tokens * keys * es},
                          {chunk_valid, "chunk_valid", tokens / chunk * 4},
                          {counts, "counts", int64_t(p.sequences) * keys * 4},
                          {coef, "coef", int64_t(p.sequences) * 4},
                          {dloss, "dloss", 4}};
    const Named written[] = {{dlogits, "dlogits", tokens * keys * es}};
    rc = check_apart(fn, written, 1, read, 5);
    if (rc != SDM_OK) return rc;
    if (debug_validate()) {
        rc = check_device_ptrs(read, 5);
        if (rc == SDM_OK) rc = check_device_ptrs(written, 1);
        if (rc != SDM_OK) return rc;
    }
    p.counts = const_cast<int32_t*>(counts);
    p.coef = const_cast<float*>(coef);
    p.dloss = dloss;
    p.dlogits = dlogits;
    p.accumulate = accumulate != 0;
    return launched(fn, launch_balance_backward(p, logit_dtype == SDM_BF16, static_cast<hipStream_t>(hip_stream)));
}

int sdm_lookup(const void* bank, const void* scales, int bank_dtype, int64_t num_slots, int64_t head_dim, int64_t n,
               const void* idx, int idx_dtype, float scale, float dropout, const uint64_t* rng, void* out, int out_dtype,
               void* hip_stream) {
    const char* fn = "sdm_lookup";
    const bool packed = is_packed(bank_dtype);
    if (!packed && !is_value(bank_dtype))
        return fail(SDM_E_DTYPE, "%s: the bank must be float32, bfloat16, SDM_MX8 or SDM_MX4 (dtype %d)", fn, bank_dtype);
    if (!is_index(idx_dtype)) return fail(SDM_E_DTYPE, "%s: idx must be int32 or int64 (dtype %d)", fn, idx_dtype);
    if (!is_value(out_dtype)) return fail(SDM_E_DTYPE, "%s: out must be float32 or bfloat16 (dtype %d)", fn, out_dtype);
    int rc = check_bank(fn, num_slots, head_dim);
    if (rc != SDM_OK) return rc;
    if (n < 0 || n > SDM_MAX_LOOKUP_ROWS) return fail(SDM_E_SHAPE, "%s: n must be in 0..2^31 - 1, got %lld", fn, (i64)n);
    const int64_t row_bytes = packed ? sdm_packed_row_bytes(bank_dtype, head_dim) : head_dim * elem_size(bank_dtype);
    const int64_t scale_bytes = packed ? sdm_packed_scale_bytes(bank_dtype, head_dim) : 0;
    if (!mul_fits(num_slots, row_bytes) || !mul_fits(n, head_dim, 4))
        return fail(SDM_E_SHAPE, "%s: sizes overflow 64-bit byte counts", fn);
    LookupParams p{};
    rc = check_dropout(fn, scale, dropout, rng, n > 0, &p.dropout.threshold, &p.factor);
    if (rc != SDM_OK) return rc;
    if (n == 0) return ok();
    p.n = n;
    p.hd = int(head_dim);
    if (lookup_groups(p) > kMaxLookupGroups) return fail(SDM_E_SHAPE, "%s: %lld rows exceed the grid", fn, (i64)n);
    if (bank == nullptr || (packed && scales == nullptr) || idx == nullptr || out == nullptr)
        return fail(SDM_E_NULL, "%s: the bank, idx and out are required", fn);
    const int is = elem_size(idx_dtype), os = elem_size(out_dtype);
    if (packed && (!aligned(bank, 16) || !aligned(scales, 4)))
        return fail(SDM_E_ALIGN, "%s: codes must be 16-byte and scales 4-byte aligned", fn);
    if ((!packed && !aligned(bank, elem_size(bank_dtype))) || !aligned(idx, is) || !aligned(out, os))
        return fail(SDM_E_ALIGN, "%s: a pointer is not aligned to its element size", fn);
    const Named read[] = {{bank, packed ? "codes" : "bank", num_slots * row_bytes},
                          {packed ? scales : nullptr, "scales", num_slots * scale_bytes},
                          {idx, "idx", n * is},
                          {p.dropout.threshold != 0 ? rng : nullptr, "rng", 16}};
    const Named written[] = {{out, "out", n * head_dim * os}};
    rc = check_apart(fn, written, 1, read, 4);
    if (rc != SDM_OK) return rc;
    if (debug_validate()) {
        rc = check_device_ptrs(read, 4);
        if (rc == SDM_OK) rc = check_device_ptrs(written, 1);
        if (rc != SDM_OK) return rc;
    }
    p.bank = bank;
    p.scales = static_cast<const uint8_t*>(scales);
    p.num_slots = num_slots;
    p.row_bytes = row_bytes;
    p.scale_bytes = int(scale_bytes);
    p.idx = idx;
    p.idx64 = idx_dtype == SDM_I64;
    p.dropout.rng = rng;
    p.out = out;
    return launched(fn, launch_lookup(p, bank_dtype, out_dtype == SDM_BF16, static_cast<hipStream_t>(hip_stream)));
}

int64_t sdm_bank_grad_workspace(int64_t entries, int64_t num_slots, int64_t head_dim) {
    if (entries < 0 || entries > SDM_MAX_GRAD_ENTRIES || num_slots < 1 || num_slots > SDM_MAX_GRAD_ENTRIES ||
        head_dim < 1 || head_dim > kMaxColumns)
        return 0;
    BankGradParams p{};
    p.entries = uint32_t(entries);
    p.num_slots = uint32_t(num_slots);
    p.hd = int(head_dim);
    return bank_grad_layout(&p, nullptr);
}

int sdm_lookup_grad(int64_t n, const void* idx, int idx_dtype, const void* dout, int dout_dtype, float scale,
                    float dropout, const uint64_t* rng, void* dbank, int bank_dtype, int64_t num_slots,
                    int64_t head_dim, int mode, void* workspace, int64_t workspace_bytes, void* hip_stream) {
    const char* fn = "sdm_lookup_grad";
    if (!is_index(idx_dtype)) return fail(SDM_E_DTYPE, "%s: idx must be int32 or int64 (dtype %d)", fn, idx_dtype);
    if (!is_value(dout_dtype)) return fail(SDM_E_DTYPE, "%s: dout must be float32 or bfloat16 (dtype %d)", fn, dout_dtype);
    int rc = check_grad(fn, bank_dtype, num_slots, head_dim, mode);
    if (rc != SDM_OK) return rc;
    if (n < 0 || n > SDM_MAX_GRAD_ENTRIES) return fail(SDM_E_SHAPE, "%s: n must be in 0..2^31 - 1, got %lld", fn, (i64)n);
    if (!mul_fits(n, head_dim, 4)) return fail(SDM_E_SHAPE, "%s: sizes overflow 64-bit byte counts", fn);
    BankGradParams p{};
    rc = check_dropout(fn, scale, dropout, rng, n > 0, &p.dropout.threshold, &p.factor);
    if (rc != SDM_OK) return rc;
    if (n == 0 && mode == SDM_GRAD_ADD) return ok();
    if (dbank == nullptr || (n > 0 && (idx == nullptr || dout == nullptr)))
        return fail(SDM_E_NULL, "%s: idx, dout and dbank are required", fn);
    const int is = elem_size(idx_dtype), ds = elem_size(dout_dtype), bs = elem_size(bank_dtype);
    if (!aligned(idx, is) || !aligned(dout, ds) || !aligned(dbank, bs))
        return fail(SDM_E_ALIGN, "%s: a pointer is not aligned to its element size", fn);
    p.entries = p.tokens = p.chunk = p.valid = uint32_t(n);
    p.width[0] = 1;
    p.num_slots = uint32_t(num_slots);
    p.hd = int(head_dim);
    p.add = mode == SDM_GRAD_ADD;
    const int64_t needed = bank_grad_layout(&p, workspace);
    if (bank_grad_groups(p, ds, bs) > kMaxGroups)
        return fail(SDM_E_SHAPE, "%s: the bank or the entries exceed the grid", fn);
    const Named read[] = {{idx, "idx", n * is},
                          {dout, "dout", n * head_dim * ds},
                          {p.dropout.threshold != 0 ? rng : nullptr, "rng", 16}};
    Named written[2] = {{dbank, "dbank", num_slots * head_dim * bs}};
    rc = check_workspace(fn, workspace, workspace_bytes, needed, written, 1, read, 3);
    if (rc != SDM_OK) return rc;
    if (debug_validate()) {
        rc = check_device_ptrs(read, n > 0 ? 3 : 0);
        if (rc == SDM_OK) rc = check_device_ptrs(written, 2);
        if (rc != SDM_OK) return rc;
    }
    p.idx[0] = idx;
    p.dout[0] = dout;
    p.idx64 = idx_dtype == SDM_I64;
    p.dropout.rng = rng;
    p.dbank = dbank;
    return launched(fn, launch_bank_grad(p, dout_dtype == SDM_BF16, bank_dtype == SDM_BF16,
                                         static_cast<hipStream_t>(hip_stream)));
}

int sdm_gather_bank_grad(int64_t tokens, int64_t chunk, int64_t valid, const int32_t* chunk_valid, int idx_dtype,
                         int w_dtype, const void* idx0, const void* w0, const float* dout0, int32_t width0,
                         const void* idx1, const void* w1, const float* dout1, int32_t width1, void* dbank,
                         int bank_dtype, int64_t num_slots, int64_t head_dim, int mode, void* workspace,
                         int64_t workspace_bytes, void* hip_stream) {
    const char* fn = "sdm_gather_bank_grad";
    const void* const idx[2] = {idx0, idx1};
    const void* const w[2] = {w0, w1};
    const float* const dout[2] = {dout0, dout1};
    const int32_t width[2] = {width0, width1};
    if (!is_index(idx_dtype)) return fail(SDM_E_DTYPE, "%s: slots must be int32 or int64 (dtype %d)", fn, idx_dtype);
    if (!is_value(w_dtype))
        return fail(SDM_E_DTYPE, "%s: weights must be float32 or bfloat16 (dtype %d)", fn, w_dtype);
    int rc = check_grad(fn, bank_dtype, num_slots, head_dim, mode);
    if (rc != SDM_OK) return rc;
    if (tokens < 0 || chunk < 1 || tokens % chunk != 0 || valid < 0 || valid > chunk)
        return fail(SDM_E_SHAPE, "%s: tokens must be a whole number of chunks and valid lie in [0, chunk]: tokens=%lld "
                    "chunk=%lld valid=%lld", fn, (i64)tokens, (i64)chunk, (i64)valid);
    const int operands = idx1 != nullptr || w1 != nullptr || dout1 != nullptr || width1 != 0 ? 2 : 1;
    for (int o = 0; o < operands; ++o) {
        if (o == 1 && tokens > 0 && (idx1 == nullptr || w1 == nullptr || dout1 == nullptr))
            return fail(SDM_E_NULL, "%s: operand 1 is given in part: pass idx1, w1 and dout1 all, or none", fn);
        if (width[o] < 1 || width[o] > SDM_MAX_WIDTH)
            return fail(SDM_E_RANGE, "%s: width%d must be in 1..%d, got %d", fn, o, SDM_MAX_WIDTH, width[o]);
    }
    const int64_t all = int64_t(width0) + (operands == 2 ? width1 : 0);
    if (tokens > SDM_MAX_GRAD_ENTRIES / all)
        return fail(SDM_E_SHAPE, "%s: at most 2^31 - 1 entries per call, got %lld tokens of %lld", fn, (i64)tokens, (i64)all);
    if (!mul_fits(tokens, head_dim, 4)) return fail(SDM_E_SHAPE, "%s: sizes overflow 64-bit byte counts", fn);
    if (tokens == 0 && mode == SDM_GRAD_ADD) return ok();
    if (dbank == nullptr || (tokens > 0 && (idx0 == nullptr || w0 == nullptr || dout0 == nullptr)))
        return fail(SDM_E_NULL, "%s: idx0, w0, dout0 and dbank are required", fn);
    const int is = elem_size(idx_dtype), ws = elem_size(w_dtype), bs = elem_size(bank_dtype);
    bool fine = aligned(dbank, bs) && aligned(chunk_valid, 4);
    Named read[7] = {{chunk_valid, "chunk_valid", tokens / chunk * 4}};
    for (int o = 0; o < operands; ++o) {
        fine = fine && aligned(idx[o], is) && aligned(w[o], ws) && aligned(dout[o], 4);
        read[1 + 3 * o] = {idx[o], "idx", tokens * width[o] * is};
        read[2 + 3 * o] = {w[o], "w", tokens * width[o] * ws};
        read[3 + 3 * o] = {dout[o], "dout", tokens * head_dim * 4};
    }
    if (!fine) return fail(SDM_E_ALIGN, "%s: a pointer is not aligned to its element size", fn);
    BankGradParams p{};
    p.entries = uint32_t(tokens * all);
    p.tokens = uint32_t(tokens);
    for (int o = 0; o < operands; ++o) p.width[o] = uint32_t(width[o]);
    p.num_slots = uint32_t(num_slots);
    p.hd = int(head_dim);
    p.add = mode == SDM_GRAD_ADD;
    const int64_t needed = bank_grad_layout(&p, workspace);
    if (bank_grad_groups(p, 4, bs) > kMaxGroups)
        return fail(SDM_E_SHAPE, "%s: the bank or the entries exceed the grid", fn);
    Named written[2] = {{dbank, "dbank", num_slots * head_dim * bs}};
    rc = check_workspace(fn, workspace, workspace_bytes, needed, written, 1, read, size_t(1 + 3 * operands));
    if (rc != SDM_OK) return rc;
    if (debug_validate()) {
        rc = check_device_ptrs(read, tokens > 0 ? size_t(1 + 3 * operands) : 0);
        if (rc == SDM_OK) rc = check_device_ptrs(written, 2);
        if (rc != SDM_OK) return rc;
    }
    for (int o = 0; o < operands; ++o) {
        p.idx[o] = idx[o];
        p.w[o] = w[o];
        p.dout[o] = dout[o];
    }
    p.chunk = uint32_t(chunk < UINT32_MAX ? chunk : UINT32_MAX);  // past the tokens only where there are none
    p.valid = uint32_t(valid < INT32_MAX ? valid : INT32_MAX);
    p.chunk_valid = chunk_valid;
    p.idx64 = idx_dtype == SDM_I64;
    p.w_bf16 = w_dtype == SDM_BF16;
    p.factor = 1.0f;
    p.dbank = dbank;
    return launched(fn, launch_bank_grad(p, false, bank_dtype == SDM_BF16, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
