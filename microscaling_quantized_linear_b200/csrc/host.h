// host.h -- what the library's translation units share on the host: the
// current device's facts, the tensor-map encoder and the wait limit, all
// kept in nvq.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace nvq {

struct HostDevice {
    int index;
    int num_sms;
    unsigned int* status;      // device status word (NVQ_STATUS_* bits)
};

// The current device; NVQ_OK, NVQ_ERR_ARCH or NVQ_ERR_CUDA.
int host_device(HostDevice* out);

using HostEncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                       const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                       CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                       CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder; null when it cannot be reached.
HostEncodeTiledFn host_encoder();

// Limit in ns of the kernels' pipeline waits (nvq_set_wait_limit), `dflt` if unset.
uint64_t host_wait_ns(uint64_t dflt);

}  // namespace nvq
