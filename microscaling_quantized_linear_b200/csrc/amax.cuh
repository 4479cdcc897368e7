// amax.cuh -- largest magnitudes of BF16 values, shared by the quantizers.
#pragma once
#include <cstdint>

namespace nvq {

constexpr float kAmaxFloor = 0x1p-100f;       // below this a tensor (NVFP4) or a block (FP8) quantizes to zero

// Bits of the device status word (the NVQ_STATUS_* values of nvq.h).
constexpr unsigned int kStatusTimeout = 1u;
constexpr unsigned int kStatusNonfinite = 2u;
constexpr unsigned int kStatusWorkspace = 4u;

// max over the two 16-bit magnitudes packed in u
__device__ __forceinline__ uint32_t absmax2(uint32_t acc, uint32_t u) {
    return __vmaxu2(acc, u & 0x7FFF7FFFu);
}

__device__ __forceinline__ uint32_t fold2(uint32_t m2) {
    return max(m2 & 0xFFFFu, m2 >> 16);
}

// Block-wide max of one value per thread; result valid in every thread.
template <int THREADS>
__device__ __forceinline__ uint32_t block_max_u32(uint32_t v, uint32_t* red /* THREADS/32 */) {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    uint32_t w = (lane < THREADS / 32) ? red[lane] : 0u;
    w = __reduce_max_sync(0xFFFFFFFFu, w);
    __syncthreads();
    return w;
}

}  // namespace nvq
