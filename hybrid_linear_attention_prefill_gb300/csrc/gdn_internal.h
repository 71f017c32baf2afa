// Host-side internals shared by the library's entry points (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include <mutex>

namespace gdn {

// The calling thread's record of the CUDA error behind its last GDN_ERR_LAUNCH or
// GDN_ERR_ALLOC (what gdn_last_cuda_error returns).  set_cuda_error records `e` and
// returns `code`; clear_cuda_error resets the record at the start of a call.
int set_cuda_error(cudaError_t e, int code);
void clear_cuda_error();

// Take the calling thread's pending gdn_set_phase_events hook (and clear it).
void take_phase_events(cudaEvent_t (&ev)[3]);

// Device address of the fixed scratch array behind gdn_prefill_static on device `dev`,
// or nullptr while no call on that device has looked it up.
void* static_scratch_address(int dev);

// Test hook behind gdn_debug_fail_allocations: true when the next library allocation
// is to fail (and counts it down).
bool take_injected_alloc_failure();

// SMs of the current device (0 without one).
int device_sms();

// gdn_ssm_scan's library-owned workspace on device `dev`, grown to at least `need` bytes (its first
// 256 bytes are status words, cleared on stream `st` when new but for bits already set): GDN_OK or the error code to
// return.
int ensure_ssm_workspace(int dev, size_t need, cudaStream_t st, void** ws);

// The library's own workspace of an attention call: the device's status words, and for `need` bytes (0: none) a place of
// the stream's own, zero where it has not been used.  GDN_OK, or the error code to return; GDN_ERR_SCRATCH while the
// stream is being captured, where something would have to be allocated or a place of the stream's given to a graph that
// any stream may run.  The library's buffers are held as they are until `hold` goes: after the launch.
struct AttnOwn {
  int* status = nullptr;
  void* ws = nullptr;
  std::unique_lock<std::mutex> hold;
};
int own_attn_workspace(int dev, size_t need, cudaStream_t st, AttnOwn& own);

// Where a kernel's dynamic shared memory starts on the current device, if it has no other: the bytes that the system keeps
// before it, or what gdn_debug_attn_smem_base says.
cudaError_t attn_smem_base(int* bytes);

}  // namespace gdn
