// Host-side helpers shared by the C ABI's translation units: error reporting and the
// argument checks (api.cu defines them).
#pragma once

#include "internal.h"

#define VQ_API extern "C" __attribute__((visibility("default")))

namespace vq {

// Record the calling thread's message and return the status.
vq_status fail(vq_status st, const char* fmt, ...);
vq_status cuda_fail(cudaError_t e, const char* what);

bool aligned16(const void* p);
vq_status check_ptr(const void* p, const char* name);
vq_status validate_desc(const vq_linear_desc* d);
vq_status validate_planes(const vq_linear_desc& d, const vq_planes* p);
vq_status validate_codebooks(const vq_linear_desc& d, const vq_codebooks* cb, const void* scales);
LayerArgs make_args(const vq_linear_desc& d, const vq_planes* p, const vq_codebooks* cb, const void* scales);

// The current device, which must be sm_100.
vq_status query_device(DeviceInfo* dev);
vq_status check_current_device(int device);
// VQ_ERR_NOMEM where the test hook VQ_TEST_FAIL_ALLOC=1 is set.
vq_status refuse_alloc();
// Waits for all work of `device` and frees a and b (either may be NULL) there.
cudaError_t free_on_device(int device, void* a, void* b = nullptr);
// Whether the byte ranges [a, a + na) and [b, b + nb) meet.
bool overlaps(const void* a, size_t na, const void* b, size_t nb);
// VQ_ERR_INVALID_ARG where y's yb bytes meet a plane, codebook or scale that a call with these (valid)
// arguments reads: those of E layers after one another, with `sets` sets of codebooks.  Of the sparse
// correction's entries only the first counts, for their number is on the device.
vq_status check_output(const vq_linear_desc& d, const vq_planes& p, const vq_codebooks& cb, const void* scales, int E,
                       int sets, const void* y, size_t yb);

}  // namespace vq
