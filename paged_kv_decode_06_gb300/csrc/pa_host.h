// Host helpers shared by the translation units that implement entry points
// (defined in pa_host.cu): error details, descriptor checks, per-device state
// and the split workspace.
#pragma once

#include <cuda_runtime.h>

#include <exception>
#include <mutex>

#include "paged_attn.h"

namespace pa {

constexpr int kMaxSeqsHost = 8192;     // sequences (block-table rows) of a call

// Set the thread's error detail and return `status`.
int host_fail(int status, const char* fmt, ...);
int host_cuda_fail(cudaError_t e, const char* what);
void host_clear_error();

// Descriptor pointer, data pointer, rank, non-negative shape and strides.
int host_check_tensor(const pa_tensor_t* t, const char* name, int ndim, bool allow_null);
bool host_aligned(const void* ptr, size_t a);

// What a launch needs of the current device, set up on first use.
struct HostDevice {
  int num_sms;
  int smem_optin;      // dynamic shared memory a kernel may ask for
  uint32_t* status;    // device status word
};

// Serialises the library's host state.  Hold it across host_device,
// host_workspace and the launches that use their results.
std::unique_lock<std::mutex> host_lock();
int host_device(HostDevice* out);

// The caller's workspace from `opts` (size and alignment checked) or the
// device's library-owned one, grown outside stream capture.
int host_workspace(const pa_options_t* opts, size_t bytes, cudaStream_t stream, const char* reserve_fn, void** ws);
int host_reserve(size_t bytes);

// Runs the body of an entry point: no exception crosses the C boundary.
template <typename F>
int host_entry(F body) noexcept {
  try {
    host_clear_error();
    return body();
  } catch (const std::exception& e) {
    try {
      return host_fail(PA_ERR_CUDA, "host error: %s", e.what());
    } catch (...) {
    }
  } catch (...) {
  }
  return PA_ERR_CUDA;
}

}  // namespace pa
