// fp8_block.cu -- C ABI of the FP8 block-scaled operators (see include/nvq.h):
// host-side checks (nothing is launched when one fails) and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8_gated.cuh"
#include "fp8_gemm.cuh"
#include "fp8_quantize.cuh"
#include "host.h"
#include "nvq.h"

namespace nvq {
namespace {

bool misaligned(const void* p, uintptr_t bytes = 16) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

// A dense [rows, cols] code matrix whose rows are a multiple of `bytes` (16: read
// through a tensor map).
bool bad_codes(int64_t rows, int64_t cols, int64_t bytes = 16) {
    return rows < 0 || cols <= 0 || cols % bytes || rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31) ||
           rows * cols >= (int64_t(1) << 31);
}

// A [rows, cols] matrix of 16-byte vectors of `per` elements, row pitch ld.
bool bad_pitch(int64_t rows, int64_t cols, int64_t ld, int64_t per) {
    return ld < cols || ld % per || ld >= (int64_t(1) << 31) || rows * ld >= (int64_t(1) << 40);
}

// Launch with programmatic stream serialization (every kernel executes
// griddepcontrol.wait before it touches global memory).
template <typename... KArgs, typename... Args>
int launch(void (*kernel)(KArgs...), uint32_t grid, uint32_t block, size_t smem, nvq_stream_t stream, uint32_t cluster,
           const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return NVQ_ERR_CUDA;
    }
    return NVQ_OK;
}

template <int OP>
int launch_gemm(const HostDevice& d, Fp8GemmParams& p, nvq_stream_t stream) {
    p.status = d.status;
    const uint64_t tiles = (uint64_t)blocks_of(p.C) * ((p.R + 31) / 32);
    return launch(fp8_gemm_simple_kernel<OP>, (uint32_t)tiles, 256, 0, stream, 1, p);
}

}  // namespace
}  // namespace nvq

using namespace nvq;

extern "C" {

size_t fp8_block_scales(int kind, int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0) return 0;
    switch (kind) {
        case NVQ_FP8_ROWS: return (size_t)(blocks_of(cols) * rows);
        case NVQ_FP8_COLUMNS: return (size_t)(blocks_of(rows) * cols);
        case NVQ_FP8_TILES: return (size_t)(blocks_of(rows) * blocks_of(cols));
        default: return 0;
    }
}

int fp8_block_quantize(const void* x, int64_t M, int64_t K, int64_t ldx, uint8_t* row_codes, float* row_scales,
                       uint8_t* col_codes, float* col_scales, nvq_stream_t stream) {
    if (bad_codes(M, K, 8) || bad_pitch(M, K, ldx, 8)) return NVQ_ERR_SHAPE;
    if (M == 0) return NVQ_OK;
    const bool rows = row_codes || row_scales, cols = col_codes || col_scales;
    if (!x || (!rows && !cols) || (rows && (!row_codes || !row_scales)) || (cols && (!col_codes || !col_scales)))
        return NVQ_ERR_NULL;
    if (misaligned(x) || misaligned(row_codes) || misaligned(row_scales) || misaligned(col_codes) ||
        misaligned(col_scales))
        return NVQ_ERR_ALIGN;
    HostDevice d;
    if (int rc = host_device(&d)) return rc;
    const Fp8QuantParams p = {static_cast<const uint16_t*>(x), (uint32_t)M, (uint32_t)K, (uint32_t)ldx, row_codes,
                              row_scales, col_codes, col_scales, d.status};
    const uint32_t grid = (uint32_t)(blocks_of(M) * blocks_of(K));
    auto kern = rows && cols ? fp8_block_quantize_kernel<3> : rows ? fp8_block_quantize_kernel<1> : fp8_block_quantize_kernel<2>;
    return launch(kern, grid, kFp8QuantThreads, 0, stream, 1, p);
}

int fp8_block_quantize_weight(const void* w, int64_t N, int64_t K, int64_t ldw, uint8_t* codes, float* scales,
                              nvq_stream_t stream) {
    if (bad_codes(N, K, 8) || bad_pitch(N, K, ldw, 8)) return NVQ_ERR_SHAPE;
    if (N == 0) return NVQ_OK;
    if (!w || !codes || !scales) return NVQ_ERR_NULL;
    if (misaligned(w) || misaligned(codes) || misaligned(scales)) return NVQ_ERR_ALIGN;
    HostDevice d;
    if (int rc = host_device(&d)) return rc;
    const Fp8QuantParams p = {static_cast<const uint16_t*>(w), (uint32_t)N, (uint32_t)K, (uint32_t)ldw, codes,
                              scales, nullptr, nullptr, d.status};
    return launch(fp8_block_quantize_kernel<4>, (uint32_t)(blocks_of(N) * blocks_of(K)), kFp8QuantThreads, 0, stream, 1, p);
}

int fp8_block_linear(const uint8_t* a_codes, const float* a_scales, const uint8_t* w_codes, const float* w_scales,
                     const void* bias, void* out, int64_t ldo, int64_t M, int64_t N, int64_t K, nvq_stream_t stream) {
    if (bad_codes(M, K) || N <= 0 || bad_codes(N, K) || N % 8 || bad_pitch(M, N, ldo, 8)) return NVQ_ERR_SHAPE;
    if (M == 0) return NVQ_OK;
    if (!a_codes || !a_scales || !w_codes || !w_scales || !out) return NVQ_ERR_NULL;
    if (misaligned(a_codes) || misaligned(a_scales) || misaligned(w_codes) || misaligned(w_scales) || misaligned(out) ||
        misaligned(bias, 4))
        return NVQ_ERR_ALIGN;
    HostDevice d;
    if (int rc = host_device(&d)) return rc;
    Fp8GemmParams p = {a_codes, a_scales, w_codes, w_scales, static_cast<const __nv_bfloat16*>(bias), out, nullptr,
                       nullptr, (uint32_t)M, (uint32_t)N, (uint32_t)K, (uint32_t)ldo, 0, nullptr};
    return launch_gemm<kFp8Linear>(d, p, stream);
}

int fp8_block_linear_dgrad(const uint8_t* dy_codes, const float* dy_scales, const uint8_t* w_codes,
                           const float* w_scales, void* dx, int64_t lddx, int64_t M, int64_t N, int64_t K,
                           nvq_stream_t stream) {
    if (bad_codes(M, N, 8) || bad_codes(N, K) || bad_pitch(M, K, lddx, 8)) return NVQ_ERR_SHAPE;
    if (M == 0) return NVQ_OK;
    if (!dy_codes || !dy_scales || !w_codes || !w_scales || !dx) return NVQ_ERR_NULL;
    if (misaligned(dy_codes) || misaligned(dy_scales) || misaligned(w_codes) || misaligned(w_scales) || misaligned(dx))
        return NVQ_ERR_ALIGN;
    HostDevice d;
    if (int rc = host_device(&d)) return rc;
    Fp8GemmParams p = {dy_codes, dy_scales, w_codes, w_scales, nullptr, dx, nullptr, nullptr, (uint32_t)M, (uint32_t)K,
                       (uint32_t)N, (uint32_t)lddx, 0, nullptr};
    return launch_gemm<kFp8Dgrad>(d, p, stream);
}

int fp8_block_linear_wgrad(const uint8_t* dy_codes, const float* dy_scales, const uint8_t* x_codes,
                           const float* x_scales, float* dw, int64_t lddw, int accumulate, int64_t M, int64_t N,
                           int64_t K, nvq_stream_t stream) {
    if (bad_codes(M, N, 8) || bad_codes(M, K) || N * K >= (int64_t(1) << 31) || bad_pitch(N, K, lddw, 4)) return NVQ_ERR_SHAPE;
    if (!dw || (M > 0 && (!dy_codes || !dy_scales || !x_codes || !x_scales))) return NVQ_ERR_NULL;
    if (misaligned(dy_codes) || misaligned(dy_scales) || misaligned(x_codes) || misaligned(x_scales) || misaligned(dw))
        return NVQ_ERR_ALIGN;
    HostDevice d;
    if (int rc = host_device(&d)) return rc;
    if (M == 0) {               // no rows: the gradient is zero
        if (!accumulate && cudaMemset2DAsync(dw, lddw * 4, 0, K * 4, N, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
            cudaGetLastError();
            return NVQ_ERR_CUDA;
        }
        return NVQ_OK;
    }
    Fp8GemmParams p = {dy_codes, dy_scales, x_codes, x_scales, nullptr, dw, nullptr, nullptr, (uint32_t)N, (uint32_t)K,
                       (uint32_t)M, (uint32_t)lddw, accumulate != 0, nullptr};
    return launch_gemm<kFp8Wgrad>(d, p, stream);
}

int fp8_block_gated_linear(const uint8_t* a_codes, const float* a_scales, const uint8_t* w_codes,
                           const float* w_scales, uint8_t* h_codes, float* h_scales, void* gate_up, int64_t ldgu,
                           int64_t M, int64_t F, int64_t K, nvq_stream_t stream) {
    if (bad_codes(M, K) || F <= 0 || F % 128 || bad_codes(2 * F, K) || bad_codes(M, 2 * F)) return NVQ_ERR_SHAPE;
    if (gate_up && bad_pitch(M, 2 * F, ldgu, 8)) return NVQ_ERR_SHAPE;
    if (M == 0) return NVQ_OK;
    if (!a_codes || !a_scales || !w_codes || !w_scales || !h_codes || !h_scales) return NVQ_ERR_NULL;
    if (misaligned(a_codes) || misaligned(a_scales) || misaligned(w_codes) || misaligned(w_scales) ||
        misaligned(h_codes) || misaligned(h_scales) || misaligned(gate_up))
        return NVQ_ERR_ALIGN;
    HostDevice d;
    if (int rc = host_device(&d)) return rc;
    Fp8GemmParams p = {a_codes, a_scales, w_codes, w_scales, nullptr, gate_up, h_codes, h_scales, (uint32_t)M,
                       (uint32_t)F, (uint32_t)K, (uint32_t)ldgu, 0, nullptr};
    return launch_gemm<kFp8Gated>(d, p, stream);
}

int fp8_block_gated_backward(const void* dh, int64_t lddh, const void* gate_up, int64_t ldgu, uint8_t* row_codes,
                             float* row_scales, uint8_t* col_codes, float* col_scales, uint8_t* h_codes,
                             float* h_scales, int64_t M, int64_t F, nvq_stream_t stream) {
    if (F <= 0 || F % 128 || bad_codes(M, 2 * F) || bad_pitch(M, F, lddh, 8) || bad_pitch(M, 2 * F, ldgu, 8))
        return NVQ_ERR_SHAPE;
    if (M == 0) return NVQ_OK;
    if (!dh || !gate_up || !row_codes || !row_scales || !col_codes || !col_scales || !h_codes || !h_scales)
        return NVQ_ERR_NULL;
    if (misaligned(dh) || misaligned(gate_up) || misaligned(row_codes) || misaligned(row_scales) ||
        misaligned(col_codes) || misaligned(col_scales) || misaligned(h_codes) || misaligned(h_scales))
        return NVQ_ERR_ALIGN;
    HostDevice d;
    if (int rc = host_device(&d)) return rc;
    const GatedBwdParams p = {static_cast<const uint16_t*>(dh), static_cast<const uint16_t*>(gate_up), (uint32_t)M,
                              (uint32_t)F, (uint32_t)lddh, (uint32_t)ldgu, row_codes, row_scales, col_codes,
                              col_scales, h_codes, h_scales, d.status};
    return launch(fp8_gated_backward_kernel, (uint32_t)(blocks_of(M) * (F / 128)), kGatedBwdThreads, 0, stream, 1, p);
}

}  // extern "C"
