// fp8_block.cu -- C ABI of the FP8 block-scaled operators (see include/nvq.h):
// host-side checks (nothing is launched when one fails) and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "fp8_gated.cuh"
#include "fp8_gemm.cuh"
#include "fp8_quantize.cuh"
#include "fp8_short.cuh"
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

// A dense [rows, cols] code matrix in tiles of 128 rows x 128 bytes, swizzled as
// the MMA reads them; what lies outside reads as zeros.
int codes_map(HostEncodeTiledFn encode, CUtensorMap* map, const void* codes, int64_t rows, int64_t cols, uint32_t box_rows = 128) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols};
    const cuuint32_t box[2] = {128u, box_rows}, estr[2] = {1u, 1u};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS ? NVQ_OK : NVQ_ERR_CUDA;
}

// The output in chunks of 32 rows x 64 bytes; stores outside are dropped.
int out_map(HostEncodeTiledFn encode, CUtensorMap* map, void* out, bool f32, int64_t rows, int64_t cols, int64_t ld) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * (f32 ? 4 : 2)};
    const cuuint32_t box[2] = {f32 ? 16u : 32u, 32u}, estr[2] = {1u, 1u};
    return encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS ? NVQ_OK : NVQ_ERR_CUDA;
}

struct Fp8Gemm {
    const uint8_t *a, *b;
    void* out;
    int64_t ldo;
    Fp8GemmParams p;
};

// Raise a kernel's shared-memory limit, once per device (`opted`: bit per device).
template <typename Kernel>
int opt_in(Kernel kern, int bytes, int device, std::atomic<uint64_t>& opted) {
    if (opted.load(std::memory_order_acquire) >> device & 1) return NVQ_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return NVQ_ERR_CUDA;
    }
    opted.fetch_or(uint64_t(1) << device, std::memory_order_release);
    return NVQ_OK;
}

Fp8GemmParams gemm_params(const float* sa, const float* sb, int64_t R, int64_t C, int64_t T) {
    Fp8GemmParams p = {};
    p.sa = sa;
    p.sb = sb;
    p.R = (uint32_t)R;
    p.C = (uint32_t)C;
    p.T = (uint32_t)T;
    return p;
}

template <int OP, bool PLAIN_A>
int launch_pair(const HostDevice& d, Fp8Gemm& g, nvq_stream_t stream) {
    using C = Fp8PairCfg<OP, PLAIN_A>;
    const HostEncodeTiledFn encode = host_encoder();
    if (!encode) return NVQ_ERR_CUDA;
    Fp8GemmParams& p = g.p;
    const int64_t brows = OP == kFp8Gated ? 2 * (int64_t)p.C : p.C;
    CUtensorMap ma, mb, mo;
    int rc;
    if ((rc = codes_map(encode, &mb, g.b, C::B_MN ? p.T : brows, C::B_MN ? brows : p.T))) return rc;
    if (PLAIN_A) ma = mb;                                // not read
    else if ((rc = codes_map(encode, &ma, g.a, C::A_MN ? p.T : p.R, C::A_MN ? p.R : p.T))) return rc;
    if (!g.out) mo = mb;                                 // not written
    else if ((rc = out_map(encode, &mo, g.out, OP == kFp8Wgrad, p.R, brows, g.ldo))) return rc;
    auto kern = fp8_gemm_pair_kernel<OP, PLAIN_A>;
    static std::atomic<uint64_t> opted{0};
    if ((rc = opt_in(kern, C::SMEM_BYTES, d.index, opted))) return rc;
    p.a = g.a;
    p.status = d.status;
    p.wait_ns = (uint32_t)host_wait_ns(kFp8WaitNs);
    p.row_tiles = (p.R + 255) / 256;
    p.col_tiles = OP == kFp8Gated ? p.C / 128 : (p.C + 255) / 256;
    p.save = OP == kFp8Gated && g.out != nullptr;
    const uint32_t tiles = p.row_tiles * p.col_tiles, pairs = (uint32_t)d.num_sms / 2;
    return launch(kern, 2 * (tiles < pairs ? tiles : pairs), C::THREADS, C::SMEM_BYTES, stream, 2, ma, mb, mo, p);
}

// The split of the contracted axis: the largest that makes no more than `room` CTAs and leaves each at least
// two blocks, so that the weight streams through as many SMs as possible.
uint32_t short_log_split(uint64_t tiles, uint64_t blocks, uint64_t room) {
    uint32_t log = 3;
    while (log > 0 && (tiles << log > room || blocks < 2u << log)) --log;
    return log;
}

// Few tokens: one cluster of `split` CTAs per 128 output columns and TN tokens.
template <int OP, int TN>
int launch_short(const HostDevice& d, const Fp8Gemm& g, nvq_stream_t stream) {
    using C = Fp8ShortCfg<OP, TN>;
    const HostEncodeTiledFn encode = host_encoder();
    if (!encode) return NVQ_ERR_CUDA;
    const int64_t wrows = C::P * (int64_t)g.p.C;
    CUtensorMap mw, ma;
    int rc;
    if ((rc = codes_map(encode, &mw, g.b, C::W_MN ? g.p.T : wrows, C::W_MN ? wrows : g.p.T))) return rc;
    if ((rc = codes_map(encode, &ma, g.a, g.p.R, g.p.T, TN))) return rc;
    auto kern = fp8_short_kernel<OP, TN>;
    static std::atomic<uint64_t> opted{0};
    if ((rc = opt_in(kern, C::SMEM_BYTES, d.index, opted))) return rc;
    Fp8ShortParams p = {};
    p.sa = g.p.sa;
    p.sw = g.p.sb;
    p.bias = g.p.bias;
    p.out = static_cast<__nv_bfloat16*>(g.out);
    p.h_codes = g.p.h_codes;
    p.h_scales = g.p.h_scales;
    p.status = d.status;
    p.M = g.p.R;
    p.C = g.p.C;
    p.T = g.p.T;
    p.ldo = (uint32_t)g.ldo;
    const uint64_t tiles = (uint64_t)blocks_of(p.C) * ((p.M + TN - 1) / TN);
    // Where two CTAs fit an SM, as many as fill half of the SMs twice: at 8 tokens (us, cold weights; columns x
    // contracted) 1, 3/2 and 2 CTAs an SM took 14.6, 12.7 and 12.7 (12288 x 4096), 10.6, 10.6 and 14.2 (9224 x
    // 4112), 12.9, 12.9 and 11.3 (4096 x 12288), 6.7 each (4096 x 4096).
    p.log_split = short_log_split(tiles, blocks_of(p.T), C::PER_SM == 2 ? (uint64_t)d.num_sms * 3 / 2 : d.num_sms);
    p.wait_ns = (uint32_t)host_wait_ns(kFp8WaitNs);
    return launch(kern, (uint32_t)tiles << p.log_split, C::THREADS, C::SMEM_BYTES, stream, 1u << p.log_split, mw, ma, p);
}

// Whether a product runs on the few-tokens kernel: always up to 32 tokens; above, on tiles of 64 tokens,
// where that is estimated faster than 256-row tiles on CTA pairs.  The estimates (ns) are fits: a wave of CTA
// pairs takes 550 a block and 2500, a wave of few-tokens CTAs 360 a block (gated: 1000) and 3500.  Measured
// (us, cold weights; columns x contracted, tokens: pairs / few-tokens):
//   linear 4096 x 4096, 64: 21.2 / 8.4, 256: 21.6 / 16.3, 384: 21.8 / 31.2;  12288 x 4096, 64: 22.7 / 16.4, 96: 23.1 / 28.4
//   linear 4096 x 12288, 256: 54.0 / 39.2, 384: 54.2 / 77.1;  1024 x 8192, 512: 37.4 / 16.3
//   dgrad 4096 x 12288, 64: 52.6 / 14.4, 256: 53.1 / 39.0, 384: 53.4 / 76.8;  12288 x 4096, 64: 21.6 / 16.7, 96: 21.8 / 28.6
//   gated 12288 x 4096, 64: 44.9 / 34.0, 96: 45.3 / 52.6;  2048 x 4096, 256: 23.7 / 19.5, 384: 23.9 / 32.0
// Of 144 cases (16 shapes, 33 to 512 tokens) it takes the faster one in 143, in the other one 1 % slower.
bool use_short(bool gated, int64_t R, int64_t C, int64_t T, int64_t num_sms) {
    if (R <= 32) return true;
    const int64_t blocks = blocks_of(T), tiles = blocks_of(C) * ((R + 63) / 64);
    const uint32_t log = short_log_split(tiles, blocks, num_sms);
    const int64_t waves = ((tiles << log) + num_sms - 1) / num_sms, share = (blocks + (1 << log) - 1) >> log;
    const int64_t pair_tiles = (R + 255) / 256 * (gated ? C / 128 : (C + 255) / 256), pairs = num_sms / 2;
    return waves * (share * (gated ? 1000 : 360) + 3500) < (pair_tiles + pairs - 1) / pairs * blocks * 550 + 2500;
}

template <int OP>
int launch_gemm(const HostDevice& d, Fp8Gemm& g, nvq_stream_t stream) {
    if constexpr (OP != kFp8Wgrad) {
        if (g.p.T % 16 == 0 && use_short(OP == kFp8Gated, g.p.R, g.p.C, g.p.T, d.num_sms)) {
            if (g.p.R <= 16) return launch_short<OP, 16>(d, g, stream);
            if (g.p.R <= 32) return launch_short<OP, 32>(d, g, stream);
            return launch_short<OP, 64>(d, g, stream);
        }
    }
    // dY's rows may be 8 bytes past a multiple of 16, which a tensor map cannot describe.  Against 8 columns more, short
    // runs, us: dgrad 4608 x 4104 x 4096 111 / 83, 300 x 12296 x 4096 81 / 53, 8 x 4104 x 4096 26.5 / 5.0 (the few-tokens
    // kernel has no such loads); wgrad 4608 x 4104 x 4096 140 / 134, 300 x 12296 x 4096 65 / 62.
    if constexpr (OP == kFp8Dgrad || OP == kFp8Wgrad)
        if ((OP == kFp8Wgrad ? g.p.R : g.p.T) % 16) return launch_pair<OP, true>(d, g, stream);
    return launch_pair<OP, false>(d, g, stream);
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
    Fp8Gemm g = {a_codes, w_codes, out, ldo, gemm_params(a_scales, w_scales, M, N, K)};
    g.p.bias = static_cast<const __nv_bfloat16*>(bias);
    return launch_gemm<kFp8Linear>(d, g, stream);
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
    Fp8Gemm g = {dy_codes, w_codes, dx, lddx, gemm_params(dy_scales, w_scales, M, K, N)};
    return launch_gemm<kFp8Dgrad>(d, g, stream);
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
    Fp8Gemm g = {dy_codes, x_codes, dw, lddw, gemm_params(dy_scales, x_scales, N, K, M)};
    g.p.accumulate = accumulate != 0;
    return launch_gemm<kFp8Wgrad>(d, g, stream);
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
    Fp8Gemm g = {a_codes, w_codes, gate_up, ldgu, gemm_params(a_scales, w_scales, M, F, K)};
    g.p.h_codes = h_codes;
    g.p.h_scales = h_scales;
    return launch_gemm<kFp8Gated>(d, g, stream);
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
    static std::atomic<uint64_t> opted{0};
    if (int rc = opt_in(fp8_gated_backward_kernel, kGatedBwdSmem, d.index, opted)) return rc;
    const int64_t tiles = blocks_of(M) * (F / 128);
    return launch(fp8_gated_backward_kernel, (uint32_t)(tiles < d.num_sms ? tiles : d.num_sms), kGatedBwdThreads,
                  kGatedBwdSmem, stream, 1, p);
}

}  // extern "C"
