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
#include "fp8_ptx.cuh"

namespace nvq {

template <bool V>
struct Flag {
    static constexpr bool value = V;
};

constexpr int kGatedBwdThreads = 512;
constexpr int kGatedBwdSmem = 2 * 3 * 4 * 512 * 16 + 16 * 3 * 128 * 4 + 3 * 128 * 4 + 16;

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

// sigma(g) and 1 - sigma(g) of two values.  exp(-g) = 2^i 2^f with i the integer
// nearest to -g log2(e), f the rest to about 2^-25 (Cody and Waite's reduction: log2(e) in two floats, so that
// a large |g| costs no precision), and 2^f, |f| <= 1/2, by its Taylor series to the
// seventh power (the next term is below 2^-27): 0.44 units rms against 0.67 for
// expf and 0.97 for one ex2.approx.  The reciprocal is the approximate one and a
// Newton step.  WIDE takes any g: it is limited to +-87, and beyond, the smaller of the two (less than
// 2^-125) is taken as 0, so that no large g brings it back; otherwise |g| <= 43, where the product of two 1 + exp(-g) is
// below 2^125 and one reciprocal serves both (141.1 -> 138.3 us at 4608 x 12288).
template <bool WIDE>
__device__ __forceinline__ void sigmoid2(uint64_t g, uint64_t& sigma, uint64_t& one_minus) {
    const auto two = [](float v) { return f32x2_pack(v, v); };
    const float2 gv = f32x2_unpack(g);
    const uint64_t gc = WIDE ? f32x2_pack(fminf(fmaxf(gv.x, -87.0f), 87.0f), fminf(fmaxf(gv.y, -87.0f), 87.0f)) : g;
    const uint64_t i = f32x2_fma3(gc, two(-1.4426950216f), two(12582912.0f));       // 1.5 2^23: the integer lands in the low bits
    uint64_t f = f32x2_fma3(i, two(-1.0f), two(12582912.0f));
    f = f32x2_fma3(gc, two(-1.9259630e-8f), f32x2_fma3(gc, two(-1.4426950216f), f));
    uint64_t p = two(1.5252733804e-5f);                                             // (ln 2)^k / k!, k = 7 .. 0
    p = f32x2_fma3(p, f, two(1.5403530394e-4f));
    p = f32x2_fma3(p, f, two(1.3333558146e-3f));
    p = f32x2_fma3(p, f, two(9.6181291076e-3f));
    p = f32x2_fma3(p, f, two(5.5504108665e-2f));
    p = f32x2_fma3(p, f, two(0.2402265070f));
    p = f32x2_fma3(p, f, two(0.6931471806f));
    p = f32x2_fma3(p, f, two(1.0f));
    const float2 pv = f32x2_unpack(p), iv = f32x2_unpack(i);
    const uint64_t e = f32x2_pack(__uint_as_float(__float_as_uint(pv.x) + (__float_as_uint(iv.x) << 23)),
                                  __uint_as_float(__float_as_uint(pv.y) + (__float_as_uint(iv.y) << 23)));
    const uint64_t neg = f32x2_fma3(e, two(-1.0f), two(-1.0f));
    const float2 nv = f32x2_unpack(neg);
    uint64_t r;
    if (WIDE) {
        float rx, ry;
        asm("rcp.approx.f32 %0, %1;" : "=f"(rx) : "f"(-nv.x));
        asm("rcp.approx.f32 %0, %1;" : "=f"(ry) : "f"(-nv.y));
        r = f32x2_pack(rx, ry);
    } else {                                             // 1 / x = y / (x y): one reciprocal for two
        float rxy;
        asm("rcp.approx.f32 %0, %1;" : "=f"(rxy) : "f"(__fmul_rn(nv.x, nv.y)));
        r = f32x2_mul(two(-rxy), f32x2_pack(nv.y, nv.x));
    }
    sigma = f32x2_fma3(r, f32x2_fma3(neg, r, two(1.0f)), r);
    one_minus = f32x2_mul(e, sigma);
    if (WIDE) {
        const float2 sv = f32x2_unpack(sigma);
        sigma = f32x2_pack(gv.x < -87.0f ? 0.0f : sv.x, gv.y < -87.0f ? 0.0f : sv.y);
        const float2 ov = f32x2_unpack(one_minus);
        one_minus = f32x2_pack(gv.x > 87.0f ? 0.0f : ov.x, gv.y > 87.0f ? 0.0f : ov.y);
    }
}

// sigma(g) of one value in fewer registers, for the products' epilogues: ex2.approx of
// the same two-float argument (0.81 units rms against 0.63).
__device__ __forceinline__ float sigmoid1(float g) {
    const float gc = fminf(fmaxf(g, -87.0f), 87.0f);
    const float hi = __fmul_rn(gc, -1.4426950216f);
    const float lo = __fmaf_rn(gc, -1.9259630e-8f, __fmaf_rn(gc, -1.4426950216f, -hi));
    float e, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(hi));
    const float d = __fadd_rn(1.0f, __fmaf_rn(e, __fmul_rn(lo, 0.6931471806f), e));
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
    return g < -87.0f ? 0.0f : __fmaf_rn(r, __fmaf_rn(-d, r, 1.0f), r);
}

// SiLU(g) * u; the argument's NaN comes through the product.  g * sigma(g) is at most |g|, so nothing
// overflows that the result does not.
__device__ __forceinline__ float silu_mul(float g, float u) { return __fmul_rn(__fmul_rn(g, sigmoid1(g)), u); }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// a * b * f, f at most 1.1, where a * b may pass FP32's range though the result does not.  Both are at least 1
// then (BF16 ends at 2^128): their product is taken 2^-128 times as large, exactly, and brought back last.
__device__ __forceinline__ float careful_mul(float a, float b, float f) {
    const float p = __fmul_rn(a, b);
    if (abs_bits(p) < 0x7F800000u) return __fmul_rn(p, f);
    return __fmul_rn(__fmul_rn(__fmul_rn(__fmul_rn(__fmul_rn(a, 0x1p-64f), __fmul_rn(b, 0x1p-64f)), f), 0x1p64f), 0x1p64f);
}

// v where it is finite, w elsewhere.
__device__ __forceinline__ uint64_t or_finite(uint64_t v, uint64_t w) {
    const float2 a = f32x2_unpack(v), b = f32x2_unpack(w);
    return f32x2_pack(abs_bits(a.x) < 0x7F800000u ? a.x : b.x, abs_bits(a.y) < 0x7F800000u ? a.y : b.y);
}

// The larger magnitude, NaN if either is.
__device__ __forceinline__ float amax_nan(float m, float v) {
    float o;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(m), "f"(fabsf(v)));
    return o;
}

// Eight values (four pairs) times factors -> eight codes.
__device__ __forceinline__ uint2 fp8_codes8(const uint64_t (&v)[4], const uint64_t (&f)[4]) {
    const float2 a = f32x2_unpack(f32x2_mul(v[0], f[0])), b = f32x2_unpack(f32x2_mul(v[1], f[1]));
    const float2 c = f32x2_unpack(f32x2_mul(v[2], f[2])), d = f32x2_unpack(f32x2_mul(v[3], f[3]));
    return make_uint2(cvt_e4m3x4(a.x, a.y, b.x, b.y), cvt_e4m3x4(c.x, c.y, d.x, d.y));
}

// Persistent, one CTA per SM, over tiles of 128 rows x 128 of F; thread: rows
// g + 32 i (i < 4) x 8 columns, its 96 results in registers.  The next tile's
// inputs come in meanwhile (16-byte copies, each thread its own, no barrier).  11 bytes
// a value move, which HBM does in 97 us at 4608 x 12288; measured 138 in short runs (4.6 TB/s), 139 to 149 over
// seconds on different boxes.  The arithmetic sets the pace, 53 instructions a value with packed pairs throughout: issue
// slots are 60 % full, and multiply-adds (41 % of their unit), maxima (49 %) and
// conversions take turns, as the two barriers of a tile keep the 16 warps in step.
// Three-operand maxima changed nothing (141.1 -> 140.9 us); a second
// CTA has no registers left, the 96 results of a thread hold them.
//
// A product of two BF16 values is exact in FP32, so it comes first.  It may pass FP32's range though the result does
// not: a CTA does its tiles that met a result which is not finite once more at the end (AGAIN), carefully for the values
// where that is so, and the others keep their bits.  (Looking at the inputs' magnitudes first cost every tile 3 %,
// doing such a tile again inside the loop 17 %, by its spills.)
template <bool AGAIN>
__device__ __forceinline__ void gated_backward_tiles(const GatedBwdParams& p, uint8_t* smem) {
    uint4* in = reinterpret_cast<uint4*>(smem);                     // [2][12][512]
    float* s_max = reinterpret_cast<float*>(smem + 2 * 12 * 512 * 16);          // [16 warps][3][128]
    float* s_factor = s_max + 16 * 3 * 128;                                     // [3][128]
    uint32_t* s_again = reinterpret_cast<uint32_t*>(s_factor + 3 * 128);        // bit n % 128: the CTA's tile n is to be done again
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t h = lane & 15, g = tid >> 4;
    const uint32_t fblocks = p.F / 128, mblocks = (p.rows + 127) / 128, tiles = fblocks * mblocks;
    const uint32_t F2 = 2 * p.F;
    const uint32_t n2 = p.rows * F2;                                // below 2^31
    const uint64_t dh_n = pitched_extent(p.rows, p.F, p.ld_dh), gu_n = pitched_extent(p.rows, F2, p.ld_gu);
    const auto load = [&](uint32_t tile, uint32_t b) {
        const uint32_t c = tile % fblocks * 128 + h * 8, r0 = tile / fblocks * 128 + g;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r = r0 + 32 * i;
            const uint64_t at_dh = (uint64_t)r * p.ld_dh + c, at_gu = (uint64_t)r * p.ld_gu + c;
            const bool ok = r < p.rows && in_bounds(at_dh, 8, dh_n, p.status) && in_bounds(at_gu + p.F, 8, gu_n, p.status);
            const uint32_t dst = smem_u32(in + (b * 12 + 3 * i) * 512 + tid), bytes = ok ? 16 : 0;
            cp_async16_zfill(dst, ok ? p.dh + at_dh : p.dh, bytes);
            cp_async16_zfill(dst + 512 * 16, ok ? p.gu + at_gu : p.gu, bytes);
            cp_async16_zfill(dst + 1024 * 16, ok ? p.gu + at_gu + p.F : p.gu, bytes);
        }
    };
    uint32_t b = 0;
    if (!AGAIN && blockIdx.x < tiles) load(blockIdx.x, 0);
    cp_async_commit();
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, b ^= 1) {
        if (AGAIN) {
            const uint32_t n = tile / gridDim.x;
            if (!(s_again[(n >> 5) & 3] >> (n & 31) & 1)) continue;
            load(tile, b);
        } else if (tile + gridDim.x < tiles) {
            load(tile + gridDim.x, b ^ 1);
        }
        cp_async_commit();
        cp_async_wait<AGAIN ? 0 : 1>();
        const uint32_t fb = tile % fblocks, rb = tile / fblocks;
        const uint32_t c = fb * 128 + h * 8, r0 = rb * 128 + g;
        uint64_t d[3][4][4];                            // dG, dU, H: pairs of columns
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4* src = in + (b * 12 + 3 * i) * 512 + tid;
            const uint4 vh = src[0], vg = src[512], vu = src[1024];
            const uint32_t wh[4] = {vh.x, vh.y, vh.z, vh.w}, wg[4] = {vg.x, vg.y, vg.z, vg.w}, wu[4] = {vu.x, vu.y, vu.z, vu.w};
            const auto pair = [](uint32_t w) { return f32x2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); };
            const auto values = [&](auto wide, auto careful) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t dh = pair(wh[e]), gate = pair(wg[e]), up = pair(wu[e]);
                    uint64_t s, om, k;                               // k = 1 + gate (1 - s)
                    sigmoid2<decltype(wide)::value>(gate, s, om);
                    const uint64_t one = f32x2_pack(1.0f, 1.0f);
                    // Around gate = -1.28, where k is 0, s is small beside 1 - s: (1 + gate) - gate s, with 1 + gate exact there,
                    // takes k's error from that of 1 - s = e s to that of s (dG 13.1 -> 5.6 units of 2^-24 rms, the FP32
                    // formula in separate operations 7.1, gates of standard deviation 1.5; 1 % slower)
                    if (decltype(wide)::value) k = f32x2_fma3(gate, om, one);
                    else k = f32x2_fma3(pair(wg[e] ^ 0x80008000u), s, f32x2_add(gate, one));
                    const uint64_t f = f32x2_mul(s, k);
                    if (decltype(careful)::value) {
                        const float2 h = f32x2_unpack(dh), u = f32x2_unpack(up), fv = f32x2_unpack(f);
                        const uint64_t silu = f32x2_mul(gate, s);                   // at most |gate|
                        d[0][i][e] = or_finite(d[0][i][e], f32x2_pack(careful_mul(h.x, u.x, fv.x), careful_mul(h.y, u.y, fv.y)));
                        d[1][i][e] = or_finite(d[1][i][e], f32x2_mul(dh, silu));
                        d[2][i][e] = or_finite(d[2][i][e], f32x2_mul(up, silu));
                    } else {
                        d[0][i][e] = f32x2_mul(f32x2_mul(dh, up), f);
                        d[1][i][e] = f32x2_mul(f32x2_mul(dh, gate), s);
                        d[2][i][e] = f32x2_mul(f32x2_mul(gate, up), s);
                    }
                }
            };
            if (fold2(absmax2(absmax2(absmax2(absmax2(0, wg[0]), wg[1]), wg[2]), wg[3])) <= 0x422Cu) values(Flag<false>(), Flag<false>());   // 43
            else values(Flag<true>(), Flag<false>());
            if (AGAIN) {
                float x = 0.0f;
#pragma unroll
                for (int e = 0; e < 12; ++e) {
                    const float2 v = f32x2_unpack(d[e / 4][i][e % 4]);
                    x = amax_nan(amax_nan(x, v.x), v.y);
                }
                if (abs_bits(x) >= 0x7F800000u) values(Flag<true>(), Flag<true>());
            }
        }
        // row-wise: dG and dU.  Lane j of a half-warp divides for the half-warp's block j (4 rows x 2).
        float m[8];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 v = f32x2_unpack(d[a][i][e]);
                    x = amax_nan(amax_nan(x, v.x), v.y);
                }
                m[4 * a + i] = x;
            }
#pragma unroll
        for (int o = 8; o; o >>= 1)
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = amax_nan(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], o));
        {
            const float m0 = h & 1 ? m[1] : m[0], m1 = h & 1 ? m[3] : m[2], m2 = h & 1 ? m[5] : m[4], m3 = h & 1 ? m[7] : m[6];
            const float x = h & 4 ? (h & 2 ? m3 : m2) : (h & 2 ? m1 : m0);
            const Fp8Scale s = fp8_block_scale(__float_as_uint(x), AGAIN ? p.status : nullptr);
            const uint32_t r = r0 + 32 * (h & 3), kb = fb + ((h >> 2) & 1) * fblocks;
            if (h < 8 && r < p.rows && in_bounds((uint64_t)kb * p.rows + r, 1, (uint64_t)2 * fblocks * p.rows, p.status))
                p.row_scales[(size_t)kb * p.rows + r] = s.scale;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = __shfl_sync(0xFFFFFFFFu, s.factor, (lane & 16) + 4 * a + i);
                    const uint64_t ff = f32x2_pack(f, f);
                    const uint64_t f4[4] = {ff, ff, ff, ff};
                    const uint32_t row = r0 + 32 * i;
                    const uint32_t at = row * F2 + a * p.F + c;
                    if (row < p.rows && in_bounds(at, 8, n2, p.status))
                        *reinterpret_cast<uint2*>(p.row_codes + at) = fp8_codes8(d[a][i], f4);
                }
        }
        // column-wise: dG, dU and H
#pragma unroll
        for (int a = 0; a < 3; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = 0.0f, y = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = f32x2_unpack(d[a][i][e]);
                    x = amax_nan(x, v.x);
                    y = amax_nan(y, v.y);
                }
                x = amax_nan(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                y = amax_nan(y, __shfl_xor_sync(0xFFFFFFFFu, y, 16));
                if (lane < 16) *reinterpret_cast<float2*>(s_max + (warp * 3 + a) * 128 + h * 8 + 2 * e) = make_float2(x, y);
            }
        __syncthreads();
        if (tid < 384) {
            const uint32_t a = tid >> 7, k = tid & 127;
            float x = 0.0f;
#pragma unroll
            for (int w = 0; w < 16; ++w) x = amax_nan(x, s_max[(w * 3 + a) * 128 + k]);
            const Fp8Scale s = fp8_block_scale(__float_as_uint(x), AGAIN ? p.status : nullptr);
            s_factor[a * 128 + k] = s.factor;
            if (!AGAIN && abs_bits(x) >= 0x7F800000u) {                 // the columns' maxima are over all that the rows' are
                const uint32_t n = tile / gridDim.x;
                atomicOr(s_again + ((n >> 5) & 3), 1u << (n & 31));
            }
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
            uint64_t f4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f4[e] = *reinterpret_cast<const uint64_t*>(s_factor + a * 128 + h * 8 + 2 * e);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t r = r0 + 32 * i;
                const uint32_t at = a < 2 ? r * F2 + a * p.F + c : r * p.F + c;
                if (r < p.rows && in_bounds(at, 8, a < 2 ? n2 : n2 / 2, p.status))
                    *reinterpret_cast<uint2*>((a < 2 ? p.col_codes : p.h_codes) + at) = fp8_codes8(d[a][i], f4);
            }
        }
    }
}

__global__ void __launch_bounds__(kGatedBwdThreads, 1)
fp8_gated_backward_kernel(const GatedBwdParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    uint4* s_again = reinterpret_cast<uint4*>(smem + kGatedBwdSmem - 16);
    if (threadIdx.x == 0) *s_again = make_uint4(0, 0, 0, 0);
    griddep_wait();
    griddep_launch();
    __syncthreads();
    gated_backward_tiles<false>(p, smem);
    __syncthreads();
    const uint4 again = *s_again;
    if (again.x | again.y | again.z | again.w) gated_backward_tiles<true>(p, smem);
}

}  // namespace nvq
