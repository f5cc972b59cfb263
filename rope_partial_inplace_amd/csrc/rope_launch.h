// rope_launch.h -- launching and error text shared by the entry points of librope_amd.so
// (library-internal).
#pragma once

#include <hip/hip_runtime.h>

#include <string>

#define ROPE_API extern "C" __attribute__((visibility("default")))

namespace ropeamd {

// Text of the calling thread's last failing call.
extern thread_local std::string g_last_error;

// One launch of a kernel that takes its plan by value; a failed launch sets the error text.
int launch_kernel(const void *fn, dim3 blocks, int threads, size_t lds, void *stream, void *plan);

}  // namespace ropeamd
