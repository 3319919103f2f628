// device_errors.h -- the bits of the sticky device error word, which kernels set
// and ssm_check_device_errors() reads and clears.  One bit per cause, so that the
// word of a failed run tells which kernels gave up.
#pragma once

namespace ssm {

constexpr unsigned kErrWait = 1u;       // STREAM, the tiled backward: a copy did not land in time
constexpr unsigned kErrSsdWait = 2u;    // SSD form: a copy or product did not finish in time
constexpr unsigned kErrSsdAlign = 4u;   // SSD form: shared memory not 1024-byte aligned, nothing computed
constexpr unsigned kErrWaitTm = 8u;     // STREAM-TM: a copy or product did not finish in time
constexpr unsigned kErrConvWait = 16u;  // short convolution: a copy did not land in time
constexpr unsigned kErrXentWait = 32u;  // cross entropy: a copy or product did not finish in time

}  // namespace ssm
