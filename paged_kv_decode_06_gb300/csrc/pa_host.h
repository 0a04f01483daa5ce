// Host helpers shared by the translation units that implement entry points
// (defined in pa_host.cu): error details, descriptor checks, per-device state
// and the split workspace.
#pragma once

#include <cuda_runtime.h>

#include <exception>
#include <mutex>

#include "pa_kernels.h"
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
  cudaError_t shared_prefix;   // whether the prefix kernel can run
};

// Serialises the library's host state.  Hold it across host_device,
// host_workspace and the launches that use their results.
std::unique_lock<std::mutex> host_lock();
int host_device(HostDevice* out);

// The caller's workspace from `opts` (size and alignment checked) or the
// device's library-owned one, grown outside stream capture.
int host_workspace(const pa_options_t* opts, size_t bytes, cudaStream_t stream, const char* reserve_fn, void** ws);
int host_reserve(size_t bytes);

// Launch plan of the mma.sync split kernel (at most 64 query rows a KV head), `seq_ints`
// int32 a sequence in its shared memory: sp has the plan's fields, the rest zero; `rows`
// partial rows are left by cut units.
struct HostSplitPlan {
  SplitParams sp;
  int threads, grid, smem;
  size_t rows;
};
int host_split_plan(int B, int Hq, int Hkv, int D, int kv_dtype, int max_qlen, const pa_options_t* opts, int seq_ints,
                    const HostDevice& dev, HostSplitPlan* out);
// TMA map over a cache for boxes of HC heads of a page.
int host_cache_map(CUtensorMap* map, const pa_tensor_t* t, int esz, int D, int Hkv, int HC, int64_t NB);
// TMA map for a shared prefix's loads; *split: a page comes in four boxes.
int host_prefix_map(CUtensorMap* map, const pa_tensor_t* t, int esz, int D, int Hkv, int64_t NB, bool* split);

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
