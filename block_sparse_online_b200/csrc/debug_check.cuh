// debug_check.cuh -- the bounds checks of the debug build, shared by every kernel.
#pragma once

namespace solattn {

constexpr int kStatusBounds = -6;  // a debug-build bounds check failed

// Debug builds (-DSOLATTN_DEBUG) check the indices each role derives from shared state
// before it uses them for a copy, an MMA operand or a store. A failed check records
// kStatusBounds (if no error is recorded yet) and raises the abort flag; the role then
// leaves as it does after a timeout, and the other roles follow at their next wait.
// Release builds compile every check to `true`.
__device__ __forceinline__ bool debug_fail(int *abort_flag, int *status) {
  atomicCAS(status, 0, kStatusBounds);
  *reinterpret_cast<volatile int *>(abort_flag) = 1;
  return false;
}
// Kernels without an abort flag (the routing pass) record the status only; the routing-only
// entry point runs without a status word (null), and then a failed check only skips the access.
__device__ __forceinline__ bool debug_fail_status(int *status) {
  if (status) atomicCAS(status, 0, kStatusBounds);
  return false;
}
#ifdef SOLATTN_DEBUG
#define SOLATTN_DCHECK(cond, abort_flag, status) ((cond) ? true : debug_fail((abort_flag), (status)))
#define SOLATTN_DCHECK_STATUS(cond, status) ((cond) ? true : debug_fail_status(status))
#else
#define SOLATTN_DCHECK(cond, abort_flag, status) true
#define SOLATTN_DCHECK_STATUS(cond, status) true
#endif

}  // namespace solattn
