// Checks of an entry point's arguments that files of the C ABI share.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/sdm_memory.h"
#include "sdm_host.h"

namespace sdm {

inline bool is_value(int dtype) { return dtype == SDM_F32 || dtype == SDM_BF16; }
inline bool is_index(int dtype) { return dtype == SDM_I32 || dtype == SDM_I64; }
inline bool is_packed(int dtype) { return dtype == SDM_MX8 || dtype == SDM_MX4; }

struct Named {
    const void* p;
    const char* name;
    int64_t bytes;
};

inline int check_device_ptrs(const Named* list, size_t n) {
    for (size_t i = 0; i < n; ++i) {
        if (list[i].p == nullptr) continue;
        const int rc = check_device_ptr(list[i].p, list[i].name);
        if (rc != SDM_OK) return rc;
    }
    return SDM_OK;
}

// No written array shares memory with another array of the call.
inline int check_apart(const char* fn, const Named* written, size_t nw, const Named* read, size_t nr) {
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

inline int launched(const char* fn, hipError_t e) {
    if (e != hipSuccess) return fail(SDM_E_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
    return ok();
}

}  // namespace sdm
