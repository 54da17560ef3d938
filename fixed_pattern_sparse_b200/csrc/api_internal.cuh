// api_internal.cuh -- host helpers that the entry points of skiparse_api.cu share with those of
// other files: geometry, the device status word, test hooks and error recording.
#pragma once

#include <cstddef>

#include "skiparse_internal.cuh"

namespace skiparse {
namespace api {

int cuda_fail(int err);  // records a failed CUDA call's message; returns SKIPARSE_ERR_CUDA
int geometry(int dims, int B, int T, int H, int W, int heads, int d, int P, int mode, Geometry& g);
int* status_word();      // the current device's; nullptr (recorded) on a CUDA failure
long long debug_bound(long long rows);
int pending_fault(int kind);
unsigned long long wait_limit_ns();
bool ranges_overlap(const void* a, size_t abytes, const void* b, size_t bbytes);

}  // namespace api
}  // namespace skiparse
