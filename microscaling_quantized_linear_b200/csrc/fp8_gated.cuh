// fp8_gated.cuh -- backward pass of H = SiLU(G) * U between the products of a
// gated feed-forward block, quantized for the products that follow.
//
//   sigma = 1 / (1 + exp(-G))
//   dG = dH * U * sigma * (1 + G * (1 - sigma)),  dU = dH * G * sigma,  H = G * sigma * U
//
// in FP32 from BF16 inputs, unrounded until the E4M3 codes.  [dG | dU] is one
// [M, 2F] matrix, quantized row-wise (for dX, which contracts 2F) and
// column-wise (for dW, which contracts M); H is quantized column-wise (for the
// second projection's dW).
#pragma once
#include <cstdint>
#include "debug.cuh"
#include "fp8_quantize.cuh"
#include "ptx.cuh"

namespace nvq {

constexpr int kGatedBwdThreads = 512;

struct GatedBwdParams {
    const uint16_t* dh;         // [rows, F], pitch ld_dh
    const uint16_t* gu;         // [rows, 2F], pitch ld_gu
    uint32_t rows, F, ld_dh, ld_gu;
    uint8_t* row_codes;         // [rows, 2F]; scales [2F / 128, rows]
    float* row_scales;
    uint8_t* col_codes;         // [rows, 2F]; scales [ceil(rows / 128), 2F]
    float* col_scales;
    uint8_t* h_codes;           // [rows, F]; scales [ceil(rows / 128), F]
    float* h_scales;
    unsigned int* status;
};

// sigma(g) = 1 / (1 + e), e = exp(-g), within about two units: e = 2^hi (1 + lo ln 2)
// with hi + lo = -g log2(e) carried in two floats, so that a large |g| costs no
// precision.  e overflows to infinity for g < -88, which gives 0.
struct Sigmoid {
    float s, one_minus;         // sigma(g), 1 - sigma(g)
};

__device__ __forceinline__ float exp_neg(float g) {
    const float hi = __fmul_rn(g, -1.4426950216f);
    const float lo = __fmaf_rn(g, -1.9259630e-8f, __fmaf_rn(g, -1.4426950216f, -hi));
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(hi));
    return fabsf(hi) < 126.0f ? __fmaf_rn(e, __fmul_rn(lo, 0.6931471806f), e) : e;
}

// 1 / (1 + e) to about half a unit: the approximate reciprocal and one Newton step
// (not where 1 + e nears the largest floats, whose reciprocal needs no more).
__device__ __forceinline__ float sigmoid_of_exp(float e) {
    const float d = __fadd_rn(1.0f, e);
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
    return e < 1e30f ? __fmaf_rn(r, __fmaf_rn(-d, r, 1.0f), r) : r;
}

__device__ __forceinline__ float sigmoid_f32(float g) { return sigmoid_of_exp(exp_neg(g)); }

__device__ __forceinline__ Sigmoid sigmoid_both(float g) {
    const float e = exp_neg(g), s = sigmoid_of_exp(e);
    return {s, e > 1e30f ? 1.0f : __fmul_rn(e, s)};
}

__device__ __forceinline__ uint2 fp8_codes8(const float* v, const float (&f)[8]) {
    return make_uint2(cvt_e4m3x4(v[0] * f[0], v[1] * f[1], v[2] * f[2], v[3] * f[3]),
                      cvt_e4m3x4(v[4] * f[4], v[5] * f[5], v[6] * f[6], v[7] * f[7]));
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// One CTA = a tile of 128 rows x 128 of F.  Thread: rows g + 32 i (i < 4) x 8 columns.
__global__ void __launch_bounds__(kGatedBwdThreads)
fp8_gated_backward_kernel(const GatedBwdParams p) {
    __shared__ uint32_t s_max[16][3][128];
    __shared__ float s_factor[3][128];
    griddep_wait();
    griddep_launch();
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t h = lane & 15, g = threadIdx.x >> 4;
    const uint32_t fblocks = p.F / 128;
    const uint32_t fb = blockIdx.x % fblocks, rb = blockIdx.x / fblocks, r0 = rb * 128;
    const uint32_t c = fb * 128 + h * 8;
    const uint32_t F2 = 2 * p.F, mblocks = (p.rows + 127) / 128;
    const uint64_t n2 = (uint64_t)p.rows * F2;
    float d[3][4][8];                                   // dG, dU, H
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t r = r0 + g + 32 * i;
        uint4 vh = make_uint4(0, 0, 0, 0), vg = vh, vu = vh;
        if (r < p.rows && in_bounds((uint64_t)r * p.ld_dh + c, 8, pitched_extent(p.rows, p.F, p.ld_dh), p.status) &&
            in_bounds((uint64_t)r * p.ld_gu + p.F + c, 8, pitched_extent(p.rows, F2, p.ld_gu), p.status)) {
            vh = __ldg(reinterpret_cast<const uint4*>(p.dh + (size_t)r * p.ld_dh + c));
            vg = __ldg(reinterpret_cast<const uint4*>(p.gu + (size_t)r * p.ld_gu + c));
            vu = __ldg(reinterpret_cast<const uint4*>(p.gu + (size_t)r * p.ld_gu + p.F + c));
        }
        const uint32_t wh[4] = {vh.x, vh.y, vh.z, vh.w}, wg[4] = {vg.x, vg.y, vg.z, vg.w}, wu[4] = {vu.x, vu.y, vu.z, vu.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const auto pick = [&](const uint32_t (&w)[4]) {
                return __uint_as_float((e & 1) ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
            };
            const float dh = pick(wh), gate = pick(wg), up = pick(wu);
            const Sigmoid sg = sigmoid_both(gate);
            // products of two BF16 values are exact in FP32: they come first
            d[0][i][e] = __fmul_rn(__fmul_rn(dh, up), __fmul_rn(sg.s, __fmaf_rn(gate, sg.one_minus, 1.0f)));
            d[1][i][e] = __fmul_rn(__fmul_rn(dh, gate), sg.s);
            d[2][i][e] = __fmul_rn(__fmul_rn(gate, up), sg.s);
        }
    }
    // row-wise: dG and dU
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        const uint32_t kb = fb + a * fblocks;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, abs_bits(d[a][i][e]));
#pragma unroll
            for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const Fp8Scale s = fp8_block_scale(m, p.status);
            const uint32_t r = r0 + g + 32 * i;
            if (r < p.rows) {
                const float f[8] = {s.factor, s.factor, s.factor, s.factor, s.factor, s.factor, s.factor, s.factor};
                const uint64_t at = (uint64_t)r * F2 + a * p.F + c;
                if (in_bounds(at, 8, n2, p.status))
                    *reinterpret_cast<uint2*>(p.row_codes + at) = fp8_codes8(d[a][i], f);
                if (h == 0 && in_bounds((uint64_t)kb * p.rows + r, 1, (uint64_t)2 * fblocks * p.rows, p.status))
                    p.row_scales[(size_t)kb * p.rows + r] = s.scale;
            }
        }
    }
    // column-wise: dG, dU and H
#pragma unroll
    for (int a = 0; a < 3; ++a)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max(m, abs_bits(d[a][i][e]));
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
            if (lane < 16) s_max[warp][a][h * 8 + e] = m;
        }
    __syncthreads();
    if (threadIdx.x < 384) {
        const uint32_t a = threadIdx.x >> 7, k = threadIdx.x & 127;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) m = max(m, s_max[w][a][k]);
        const Fp8Scale s = fp8_block_scale(m, p.status);
        s_factor[a][k] = s.factor;
        const uint32_t col = fb * 128 + k;
        if (a < 2) {
            const uint64_t at = (uint64_t)rb * F2 + a * p.F + col;
            if (in_bounds(at, 1, (uint64_t)mblocks * F2, p.status)) p.col_scales[at] = s.scale;
        } else {
            const uint64_t at = (uint64_t)rb * p.F + col;
            if (in_bounds(at, 1, (uint64_t)mblocks * p.F, p.status)) p.h_scales[at] = s.scale;
        }
    }
    __syncthreads();
#pragma unroll
    for (int a = 0; a < 3; ++a) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = s_factor[a][h * 8 + e];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r = r0 + g + 32 * i;
            if (r >= p.rows) continue;
            const uint64_t at = a < 2 ? (uint64_t)r * F2 + a * p.F + c : (uint64_t)r * p.F + c;
            if (!in_bounds(at, 8, a < 2 ? n2 : n2 / 2, p.status)) continue;
            *reinterpret_cast<uint2*>((a < 2 ? p.col_codes : p.h_codes) + at) = fp8_codes8(d[a][i], f);
        }
    }
}

}  // namespace nvq
