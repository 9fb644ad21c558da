// Host-side helpers of the C ABI, shared by its files: the calling thread's error
// message and the checks that every entry point makes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <vector>

namespace sdm {

// Store a message for sdm_last_error() and return `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clear the message and return SDM_OK.
int ok();

int elem_size(int dtype);                      // of SDM_F32, SDM_BF16, SDM_I32, SDM_I64; 0 for another
bool aligned(const void* p, int bytes);
bool overlap(const void* a, int64_t na, const void* b, int64_t nb);  // of two byte ranges
bool mul_fits(int64_t a, int64_t b, int64_t c = 1);                  // a * b * c (none negative) fits in int64

bool debug_validate();  // SDM_DEBUG_VALIDATE is set
int check_device_ptr(const void* p, const char* name);
int device_cus(int* cus);  // compute units of the current device

// Copy a device slot list to the host as int64 (SDM_DEBUG_VALIDATE only).
int fetch_slots(const void* dev, int dtype, int64_t n, std::vector<int64_t>& out, hipStream_t stream,
                const char* name);
// The gather's slot preconditions; see the definition.
int validate_gather_slots(int64_t num_slots, int64_t rows, int64_t chunk, int64_t valid, const int32_t* chunk_valid,
                          const void* idx0, int width0, const void* idx1, int width1, int idx_dtype,
                          hipStream_t stream);

}  // namespace sdm
