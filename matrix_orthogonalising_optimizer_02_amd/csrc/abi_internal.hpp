// Host-side entry points shared between the C-ABI source files of libmuon_rocm.so.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <exception>
#include <functional>
#include <new>
#include <string>
#include <vector>

#include "../../include/muon_rocm.h"

namespace muon {

// Sets this thread's muon_last_error() text and returns `code`; an empty text clears it.
int set_last_error(int code, const std::string& what);

// Byte range of a buffer of a call, for the overlap check.
struct Range {
    uintptr_t lo, hi;
    bool write;
};

// MUON_ERR_ALIAS (with the error text set) when a written range overlaps another one.
// Sorts the ranges.
int check_overlaps(std::vector<Range>& ranges);

// Runs `launch`, bracketed by events of kernel class `cls` while timing is enabled;
// MUON_ERR_HIP (with the error text set) when it fails.
int run_timed(int cls, hipStream_t stream, const char* name, const std::function<hipError_t()>& launch);

// Runs the body of a C entry point; no C++ exception leaves it (the lists of a call that do
// not fit the host's memory give MUON_ERR_TOO_LARGE).
template <class F>
int guarded(F&& body) {
    try {
        set_last_error(MUON_OK, "");
        return body();
    } catch (const std::bad_alloc&) {
        return set_last_error(MUON_ERR_TOO_LARGE, "out of host memory");
    } catch (const std::exception& e) {
        return set_last_error(MUON_ERR_INVALID_ARG, e.what());
    }
}

// rownorm_update on a scratch buffer of scratch_cap bytes that get_scratch returns for
// the current device (NULL with *error set on failure). Validates and plans on the host
// before get_scratch is called; rejects matrices whose RowNorm workspace exceeds
// scratch_cap with MUON_ERR_WORKSPACE. Enqueues no timing events.
int rownorm_noalloc_impl(const muon_matrix* mats, int32_t count, const muon_hparams* hp, float* update_rms,
                         void* stream, size_t scratch_cap, void* (*get_scratch)(std::string* error));

}  // namespace muon
