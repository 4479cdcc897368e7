// fp8_gemm.cuh -- products of E4M3 operands with one FP32 scale per block of 128.
//
//   out[r, c] = sum over blocks t of 128 of the contracted axis:
//                 sa(r, t) * sb(c, t) * sum_{k in t} a(r, k) * b(c, k)      (+ bias[c])
//
// linear    a = activations [M, K] row-wise, b = weights [N, K] tile-wise
// dgrad     a = dY [M, N] row-wise, b = the same weights read along N
// wgrad     a = dY [M, N], b = X [M, K], both column-wise and read along M
// gated     linear onto gate and up; H = SiLU(gate) * up quantized row-wise
// The inner sum of a block is a sum of products of codes; the scales are FP32,
// so they are applied to each block's sum as it is added to the FP32 total.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include "debug.cuh"
#include "fp8_gated.cuh"
#include "ptx.cuh"

namespace nvq {

enum Fp8Op { kFp8Linear = 0, kFp8Dgrad = 1, kFp8Wgrad = 2, kFp8Gated = 3 };

struct Fp8GemmParams {
    const uint8_t* a;
    const float* sa;
    const uint8_t* b;
    const float* sb;
    const __nv_bfloat16* bias;
    void* out;                  // BF16 (linear, dgrad), FP32 (wgrad), BF16 gate and up or null (gated)
    uint8_t* h_codes;           // gated: [R, C] and [C / 128, R]
    float* h_scales;
    uint32_t R, C, T;           // output rows, columns (gated: F), contracted length
    uint32_t ldo;
    uint32_t accumulate;        // wgrad: add to out
    unsigned int* status;
};

__device__ __forceinline__ float e4m3_value(uint8_t code) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}

template <int OP>
__device__ __forceinline__ float fp8_a(const Fp8GemmParams& p, uint32_t r, uint32_t t) {
    if (r >= p.R || t >= p.T) return 0.0f;
    return e4m3_value(OP == kFp8Wgrad ? p.a[(size_t)t * p.R + r] : p.a[(size_t)r * p.T + t]);
}

template <int OP>
__device__ __forceinline__ float fp8_b(const Fp8GemmParams& p, uint32_t c, uint32_t rows, uint32_t t) {
    if (c >= rows || t >= p.T) return 0.0f;
    return e4m3_value(OP == kFp8Wgrad || OP == kFp8Dgrad ? p.b[(size_t)t * rows + c] : p.b[(size_t)c * p.T + t]);
}

template <int OP>
__device__ __forceinline__ float fp8_sb(const Fp8GemmParams& p, uint32_t c, uint32_t rows, uint32_t tb) {
    if (c >= rows) return 0.0f;
    if (OP == kFp8Wgrad) return p.sb[(size_t)tb * rows + c];
    if (OP == kFp8Dgrad) return p.sb[(size_t)tb * ((rows + 127) / 128) + c / 128];
    return p.sb[(size_t)(c / 128) * ((p.T + 127) / 128) + tb];
}

// 32 x 128 output tile (gated: of both projections), 256 threads, thread = rows
// 4w..4w+3 of the tile (warp w) x columns 4l..4l+3 (lane l), blocks of 16 staged
// in shared memory as FP32.
template <int OP>
__global__ void __launch_bounds__(256) fp8_gemm_simple_kernel(const Fp8GemmParams p) {
    constexpr int P = OP == kFp8Gated ? 2 : 1;
    __shared__ float s_a[16][32];
    __shared__ float s_b[P][16][128];
    griddep_wait();
    griddep_launch();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t cblocks = (p.C + 127) / 128;
    const uint32_t c0 = (blockIdx.x % cblocks) * 128, r0 = (blockIdx.x / cblocks) * 32;
    const uint32_t brows = P * p.C;
    float acc[P][4][4] = {};
    for (uint32_t tb = 0; tb * 128 < p.T; ++tb) {
        float part[P][4][4] = {};
        for (uint32_t k0 = tb * 128; k0 < tb * 128 + 128; k0 += 16) {
            __syncthreads();
            for (uint32_t i = threadIdx.x; i < 512; i += 256) s_a[i & 15][i >> 4] = fp8_a<OP>(p, r0 + (i >> 4), k0 + (i & 15));
            for (int q = 0; q < P; ++q)
                for (uint32_t i = threadIdx.x; i < 2048; i += 256) {
                    const uint32_t k = OP == kFp8Linear || OP == kFp8Gated ? i & 15 : i >> 7;
                    const uint32_t c = OP == kFp8Linear || OP == kFp8Gated ? i >> 4 : i & 127;
                    s_b[q][k][c] = c0 + c < p.C ? fp8_b<OP>(p, q * p.C + c0 + c, brows, k0 + k) : 0.0f;
                }
            __syncthreads();
            for (int k = 0; k < 16; ++k)
                for (int q = 0; q < P; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            part[q][i][j] = __fmaf_rn(s_a[k][warp * 4 + i], s_b[q][k][lane * 4 + j], part[q][i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r = r0 + warp * 4 + i;
            const float sa = r < p.R ? p.sa[(size_t)tb * p.R + r] : 0.0f;
#pragma unroll
            for (int q = 0; q < P; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t c = c0 + lane * 4 + j;
                    const float sb = c < p.C ? fp8_sb<OP>(p, q * p.C + c, brows, tb) : 0.0f;
                    if (r < p.R && c < p.C) acc[q][i][j] = __fmaf_rn(part[q][i][j], sa * sb, acc[q][i][j]);
                }
        }
    }
    for (int i = 0; i < 4; ++i) {
        const uint32_t r = r0 + warp * 4 + i;
        if (r >= p.R) continue;
        if (OP == kFp8Gated) {
            float hv[4];
            uint32_t m = 0;
            for (int j = 0; j < 4; ++j) {
                const float gate = acc[0][i][j], up = acc[P - 1][i][j];
                hv[j] = gate * sigmoid_f32(gate) * up;
                m = max(m, abs_bits(hv[j]));
                if (p.out) {
                    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + (size_t)r * p.ldo + c0 + lane * 4 + j;
                    o[0] = __float2bfloat16_rn(gate);
                    o[p.C] = __float2bfloat16_rn(up);
                }
            }
            m = __reduce_max_sync(0xFFFFFFFFu, m);
            const Fp8Scale s = fp8_block_scale(m, p.status);
            *reinterpret_cast<uint32_t*>(p.h_codes + (size_t)r * p.C + c0 + lane * 4) =
                cvt_e4m3x4(hv[0] * s.factor, hv[1] * s.factor, hv[2] * s.factor, hv[3] * s.factor);
            if (lane == 0) p.h_scales[(size_t)(c0 / 128) * p.R + r] = s.scale;
            continue;
        }
        for (int j = 0; j < 4; ++j) {
            const uint32_t c = c0 + lane * 4 + j;
            if (c >= p.C) continue;
            float v = acc[0][i][j];
            if (p.bias) v = __fadd_rn(v, __bfloat162float(p.bias[c]));
            if (OP == kFp8Wgrad) {
                float* o = static_cast<float*>(p.out) + (size_t)r * p.ldo + c;
                *o = p.accumulate ? __fadd_rn(*o, v) : v;
            } else {
                static_cast<__nv_bfloat16*>(p.out)[(size_t)r * p.ldo + c] = __float2bfloat16_rn(v);
            }
        }
    }
}

}  // namespace nvq
