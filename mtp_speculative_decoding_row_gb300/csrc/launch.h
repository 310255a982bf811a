// launch.h -- the device's SMs, the resident CTAs of a kernel, and launches, for
// the C ABI of the tree and step operators.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mtp_rs.h"

namespace mtp {

inline bool good_dtype(int d) { return d == MTP_DTYPE_F32 || d == MTP_DTYPE_BF16; }

// The current device and its SMs; false on a CUDA error.
bool device_sms(int &dev, int &sms);
// Resident CTAs per SM of a kernel, its shared-memory limit raised first; 0
// where it does not fit.
int resident(int dev, const void *func, uint32_t smem, int threads);
// Launch programmatically; args, map1 and map2 are the kernel's parameters.
// cluster: thread blocks of a cluster (the grid is a multiple of it).
int launch(const void *func, dim3 grid, int threads, uint32_t smem, const void *args, mtp_stream_t stream,
           const void *map1 = nullptr, const void *map2 = nullptr, int cluster = 1);

}  // namespace mtp
