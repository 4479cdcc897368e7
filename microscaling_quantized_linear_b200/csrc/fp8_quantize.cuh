// fp8_quantize.cuh -- BF16 -> E4M3 codes with one FP32 scale per block of 128.
//
// A block is 1 x 128 (row-wise: the operand of a product that contracts the
// columns), 128 x 1 (column-wise: contracts the rows) or 128 x 128 (weights).
// With b the block's largest magnitude, in FP32 round-to-nearest-even:
//   scale = b / 448, r = 448 / b, code = E4M3(x * r)   (to nearest even)
// A block with b < 2^-100 (zero included) gets the scale 0 and codes +-0, which
// also keeps r finite.  A NaN in a block makes its scale NaN, an infinity makes
// it infinite with the infinity's own code NaN, so whatever reads the block is
// NaN; the status word reports either.
//
// One CTA of 256 threads holds a 128 x 128 tile in registers (64 values per
// thread: 8 rows x 8 columns, a half-warp across one row's 128 columns), so x
// is read once whatever orientations are asked for.  Row maxima are shuffles
// within the half-warp on packed pairs of BF16 magnitudes; column maxima go
// through 2 KB of shared memory.  The divisions are shared out, one block per
// lane, and the factors handed round.  Bound by HBM: 2 bytes read and 1 (or 2)
// written per value; 4608 x 12288 both ways takes 38.4 to 40.6 us on different boxes (87 to 92 % of the copy
// rate), a weight of 9224 x 4112 18.8 to 19.6 us (89 to 93 %).  One token is all launch:
// 10 us a call, of which the kernel's own time is hidden behind the next call's checks.
#pragma once
#include <cstdint>
#include "amax.cuh"
#include "debug.cuh"
#include "ptx.cuh"

namespace nvq {

constexpr int kFp8QuantThreads = 256;

struct Fp8Scale {
    float scale, factor;
};

// Scale and factor of a block from the FP32 bits of its largest magnitude; one that is not finite is reported
// (status null: not reported).
__device__ __forceinline__ Fp8Scale fp8_block_scale(uint32_t amax_bits, unsigned int* status) {
    const float b = __uint_as_float(amax_bits);
    if (amax_bits >= 0x7F800000u && status) atomicOr(status, kStatusNonfinite);
    if (b < kAmaxFloor) return {0.0f, 0.0f};
    return {__fdiv_rn(b, 448.0f), __fdiv_rn(448.0f, b)};
}

// Eight BF16 values (packed in v) times per-value factors -> eight codes.
__device__ __forceinline__ uint2 fp8_codes8(const uint4& v, const float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float p[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[2 * i] = __fmul_rn(__uint_as_float(w[i] << 16), f[2 * i]);
        p[2 * i + 1] = __fmul_rn(__uint_as_float(w[i] & 0xFFFF0000u), f[2 * i + 1]);
    }
    return make_uint2(cvt_e4m3x4(p[0], p[1], p[2], p[3]), cvt_e4m3x4(p[4], p[5], p[6], p[7]));
}

__device__ __forceinline__ uint2 fp8_codes8(const uint4& v, float f) {
    const float2 a = bf16x2_mul(v.x, f), b = bf16x2_mul(v.y, f), c = bf16x2_mul(v.z, f), d = bf16x2_mul(v.w, f);
    return make_uint2(cvt_e4m3x4(a.x, a.y, b.x, b.y), cvt_e4m3x4(c.x, c.y, d.x, d.y));
}

struct Fp8QuantParams {
    const uint16_t* x;          // [rows, cols] BF16, pitch ld
    uint32_t rows, cols, ld;
    uint8_t* row_codes;         // [rows, cols], scales [ceil(cols / 128), rows]
    float* row_scales;
    uint8_t* col_codes;         // [rows, cols], scales [ceil(rows / 128), cols]
    float* col_scales;
    unsigned int* status;
};

// KIND bit 0: row-wise, bit 1: column-wise; 4: tile-wise (row_codes, row_scales
// = [ceil(rows / 128), ceil(cols / 128)]).
template <int KIND>
__global__ void __launch_bounds__(kFp8QuantThreads)
fp8_block_quantize_kernel(const Fp8QuantParams p) {
    constexpr bool kRows = KIND & 1, kCols = KIND & 2, kTile = KIND == 4;
    __shared__ uint4 s_max[8][16];        // per warp: BF16 magnitudes of 128 column maxima
    __shared__ float s_factor[128];
    griddep_wait();
    griddep_launch();
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t h = lane & 15;                       // column octet
    const uint32_t g = threadIdx.x >> 4;                // first row of the thread
    const uint32_t kblocks = (p.cols + 127) / 128;
    const uint32_t kb = blockIdx.x % kblocks, rb = blockIdx.x / kblocks, r0 = rb * 128;
    const uint32_t c = kb * 128 + h * 8;
    const bool col_ok = c < p.cols;
    const uint64_t x_elems = pitched_extent(p.rows, p.cols, p.ld);
    const uint64_t n_codes = (uint64_t)p.rows * p.cols;
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t r = r0 + g + 16 * i;
        v[i] = make_uint4(0, 0, 0, 0);
        if (col_ok && r < p.rows && in_bounds((uint64_t)r * p.ld + c, 8, x_elems, p.status))
            v[i] = __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)r * p.ld + c));
    }
    if (kRows) {
        uint32_t m[4];                                  // rows 2j (low half) and 2j + 1 of the thread
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 a = v[2 * j], b = v[2 * j + 1];
            const uint32_t lo = fold2(absmax2(absmax2(absmax2(absmax2(0, a.x), a.y), a.z), a.w));
            const uint32_t hi = fold2(absmax2(absmax2(absmax2(absmax2(0, b.x), b.y), b.z), b.w));
            m[j] = lo | (hi << 16);
        }
#pragma unroll
        for (int o = 8; o; o >>= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) m[j] = __vmaxu2(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], o));
        // lane h of the half-warp divides for the thread's row h & 7
        const uint32_t pair = (h & 4) ? ((h & 2) ? m[3] : m[2]) : ((h & 2) ? m[1] : m[0]);
        const Fp8Scale s = fp8_block_scale(((h & 1) ? pair >> 16 : pair & 0xFFFFu) << 16, p.status);
        const uint32_t sr = r0 + g + 16 * (h & 7);
        if (h < 8 && sr < p.rows &&
            in_bounds((uint64_t)kb * p.rows + sr, 1, (uint64_t)kblocks * p.rows, p.status))
            p.row_scales[(size_t)kb * p.rows + sr] = s.scale;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = __shfl_sync(0xFFFFFFFFu, s.factor, (lane & 16) + i);
            const uint32_t r = r0 + g + 16 * i;
            if (col_ok && r < p.rows && in_bounds((uint64_t)r * p.cols + c, 8, n_codes, p.status))
                *reinterpret_cast<uint2*>(p.row_codes + (size_t)r * p.cols + c) = fp8_codes8(v[i], f);
        }
    }
    if (kCols || kTile) {
        uint4 m = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m.x = absmax2(m.x, v[i].x);
            m.y = absmax2(m.y, v[i].y);
            m.z = absmax2(m.z, v[i].z);
            m.w = absmax2(m.w, v[i].w);
        }
        if (kTile) {
            const uint32_t t = block_max_u32<kFp8QuantThreads>(fold2(absmax2(absmax2(absmax2(m.x, m.y), m.z), m.w)),
                                                               reinterpret_cast<uint32_t*>(&s_max[0][0]));
            const Fp8Scale s = fp8_block_scale(t << 16, p.status);
            if (threadIdx.x == 0 && in_bounds((uint64_t)rb * kblocks + kb, 1,
                                              (uint64_t)((p.rows + 127) / 128) * kblocks, p.status))
                p.row_scales[(size_t)rb * kblocks + kb] = s.scale;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t r = r0 + g + 16 * i;
                if (col_ok && r < p.rows && in_bounds((uint64_t)r * p.cols + c, 8, n_codes, p.status))
                    *reinterpret_cast<uint2*>(p.row_codes + (size_t)r * p.cols + c) = fp8_codes8(v[i], s.factor);
            }
            return;
        }
        m.x = __vmaxu2(m.x, __shfl_xor_sync(0xFFFFFFFFu, m.x, 16));
        m.y = __vmaxu2(m.y, __shfl_xor_sync(0xFFFFFFFFu, m.y, 16));
        m.z = __vmaxu2(m.z, __shfl_xor_sync(0xFFFFFFFFu, m.z, 16));
        m.w = __vmaxu2(m.w, __shfl_xor_sync(0xFFFFFFFFu, m.w, 16));
        if (lane < 16) s_max[warp][lane] = m;
        __syncthreads();
        if (threadIdx.x < 128) {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(&s_max[0][0]) + threadIdx.x;
            uint32_t t = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) t = max(t, (uint32_t)q[128 * w]);
            const Fp8Scale s = fp8_block_scale(t << 16, p.status);
            s_factor[threadIdx.x] = s.factor;
            const uint32_t cc = kb * 128 + threadIdx.x;
            if (cc < p.cols && in_bounds((uint64_t)rb * p.cols + cc, 1,
                                         (uint64_t)((p.rows + 127) / 128) * p.cols, p.status))
                p.col_scales[(size_t)rb * p.cols + cc] = s.scale;
        }
        __syncthreads();
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = s_factor[h * 8 + e];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t r = r0 + g + 16 * i;
            if (col_ok && r < p.rows && in_bounds((uint64_t)r * p.cols + c, 8, n_codes, p.status))
                *reinterpret_cast<uint2*>(p.col_codes + (size_t)r * p.cols + c) = fp8_codes8(v[i], f);
        }
    }
}

}  // namespace nvq
