// sscan_host.h -- host helpers that the API translation units share: the per-thread
// error line and launch count behind sscan_last_error / sscan_last_launch_count
// (defined in sscan_api.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include "sscan.h"

namespace sscan {

// Start of an API call: clears the error line and the launch count of this thread.
void api_begin();
// Records the reason for a failed call and returns its status.
sscan_status api_fail(sscan_status s, const char* fmt, ...);
void api_count_launch();
// SSCAN_OK, or SSCAN_ERR_CUDA with the pending launch error's text.
sscan_status api_launched(const char* what);
// SSCAN_ERR_WORKSPACE unless ws holds `need` bytes on a 256-byte boundary.
sscan_status api_workspace(size_t need, const void* ws, size_t bytes);
// SSCAN_ERR_UNSUPPORTED above 2^37 elements of a (batch, L, D) tensor (or of batch x D):
// more than a device holds, and what keeps the block counts of the kernels below 2^31.
sscan_status api_elements(int64_t batch, int64_t L, int64_t D);

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }
inline bool aligned_to(const void* p, size_t n) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace sscan
