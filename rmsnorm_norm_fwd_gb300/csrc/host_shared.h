// host_shared.h -- what api.cu offers the library's other host units: the
// device cache, the grid cap and the second stage of the backward.
#pragma once

#include <stdint.h>

#include <cuda_runtime.h>

namespace gbn {

struct HostDevice {
    int dev;         // current device
    int sms;
    int smem_optin;  // largest dynamic shared memory of a block
    int *fault;      // the device's fault word (gbnorm_read_fault)
};
constexpr int kHostMaxDev = 64;  // HostDevice::dev is below this

// The current device, checked to be one the kernels run on; a gbnorm_status_t.
int host_device(HostDevice *d);
// Cap on the persistent grid (gbnorm_set_grid_limit), 0 for none.
int64_t host_grid_limit();
// Column sums of the P partial rows of ws ([2][P][N], the second block with
// is_ln) into dgamma / dbeta; P = 0 writes zeros, a NULL output is skipped.
// after_rows: the launch before it on `stream` is the row kernel.
int host_colreduce(int is_ln, const float *ws, int64_t P, int64_t N, float *dgamma, float *dbeta, bool after_rows,
                   cudaStream_t stream);

}  // namespace gbn
