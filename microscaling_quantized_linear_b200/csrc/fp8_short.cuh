// fp8_short.cuh -- the FP8 block-scaled products of few tokens: the weight's rows
// take the MMA's 128-row side and the tokens its narrow one.
//
//   out[m, c] = sum_t sa(m, t) sw(c, t) sum_{k in t} a(m, k) w(c, k)
//
// (linear, dgrad; gated: for gate and up, then H, as in fp8_gemm.cuh).  What such
// a call costs is reading the weight once, so the work is cut for the most bytes
// in flight: one cluster of `split` CTAs per 128 weight rows (gated: 128 of gate
// and the same of up) and TN tokens, each CTA with a share of the contracted axis
// and as many 128 x 128-byte stages as shared memory holds (asking L2 for the
// share while the previous grid still runs, as gemm.cuh does, measured slower: 13.9
// against 11.9 us at 29 x 9224 x 4112).  Every block's sum goes to its own TN columns of
// tensor memory (512 / TN of them in turn); 8 epilogue warps, a thread per weight
// row, scale it into registers.  The CTAs of a cluster then hand their partial
// sums to each token's owner through distributed shared memory, which adds them
// in rank order.  Measured back to back in a graph, with the weight in HBM (weights rotated over more than L2)
// and in L2: 29 x 9224 x 4112 11.8 and 8.7 us (3.2 TB/s from HBM; stream 5.8, first tile 1.1, exchange and output
// 2.5, start 1), 1 x 4096 x 4096 6.4 and 4.4 us (9 through the binding), 29 x 12288 x 4096 14.1 and 10.1, dgrad 8 x
// 4096 x 12288 11.7 and 8.5, gated 1 x 12288 x 4096 18.7 and 17.5 us (5.4 TB/s from HBM).
// Warps 0-7: epilogue (linear: half of the tokens each group of four; gated: gate
// and up); 8: loads; 9, 10: MMAs, units in turn.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "debug.cuh"
#include "fp8_gated.cuh"
#include "fp8_gemm.cuh"
#include "fp8_ptx.cuh"

namespace nvq {

struct Fp8ShortParams {
    const float* sa;            // [T / 128][M]
    const float* sw;            // linear, gated: [rows / 128][T / 128]; dgrad: [T / 128][C / 128]
    const __nv_bfloat16* bias;
    __nv_bfloat16* out;         // linear, dgrad: [M, C]; gated: gate and up [M, 2 C] or null
    uint8_t* h_codes;
    float* h_scales;
    unsigned int* status;
    uint32_t M, C, T;           // tokens, output columns (gated: F), contracted length
    uint32_t ldo, log_split, wait_ns;
};

template <int OP, int TN_>
struct Fp8ShortCfg {
    static constexpr int TN = TN_;
    static constexpr bool GATED = OP == kFp8Gated;
    static constexpr bool W_MN = OP == kFp8Dgrad;                       // the weight's contiguous axis is the output's
    static constexpr int P = GATED ? 2 : 1;                             // projections
    static constexpr int NT = GATED ? TN : TN / 2;                      // tokens of an epilogue thread
    static constexpr int THREADS = 352;
    static constexpr int W_BYTES = 128 * 128, A_BYTES = TN * 128;
    static constexpr int STAGE_BYTES = W_BYTES + A_BYTES;               // of one unit (block and projection)
    // Two CTAs to an SM: the next launch's start (barriers, tensor memory) then overlaps this one's end.  For
    // more tokens the exchange area leaves no room for that.
    static constexpr int PER_SM = !GATED && TN <= 32 ? 2 : 1;
    static constexpr int TM_COLS = 512 / PER_SM;
    static constexpr int NBUF = TM_COLS / TN;                           // accumulators; unit u uses u % NBUF
    static constexpr int CHUNK = 512 / TN;                              // blocks of scales held at once
    static constexpr int SCALE_BYTES = P * CHUNK * TN * 4;
    static constexpr int RECV_BYTES = P * TN * 128 * 4;
    static constexpr int BAR_BYTES = 1024;
    static constexpr int SMEM_LIMIT = PER_SM == 2 ? 115712 : 232448;
    static constexpr int FIT = (SMEM_LIMIT - 1024 - BAR_BYTES - SCALE_BYTES - RECV_BYTES) / STAGE_BYTES;
    // an MMA warp takes every other unit: with an even number of stages it sees every phase of theirs
    static constexpr int STAGES = (FIT > 12 ? 12 : FIT) & ~1;
    static constexpr int OFF_RECV = STAGES * STAGE_BYTES;
    static constexpr int OFF_SCALE = OFF_RECV + RECV_BYTES;
    static constexpr int OFF_BAR = OFF_SCALE + SCALE_BYTES;
    static constexpr int SMEM_BYTES = OFF_BAR + BAR_BYTES + 1024;
    static constexpr uint32_t IDESC = (1u << 4) | ((W_MN ? 1u : 0u) << 15) | ((uint32_t)(TN >> 3) << 17) | ((128u >> 4) << 24);
    static constexpr uint32_t W_STEP = W_MN ? 4096 : 32;
    static_assert(TN == 16 || TN == 32 || TN == 64, "token tile");
    static_assert(STAGES >= 4 && SMEM_BYTES <= SMEM_LIMIT, "shared memory");
    static_assert((2 * STAGES + 2 * NBUF + 2) * 8 + 48 <= BAR_BYTES, "barriers");
};

template <int OP, int TN>
__global__ void __launch_bounds__(Fp8ShortCfg<OP, TN>::THREADS, Fp8ShortCfg<OP, TN>::PER_SM)
fp8_short_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a,
                 const Fp8ShortParams p) {
    using C = Fp8ShortCfg<OP, TN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    // full[s], empty[s]: the stages; tfull[b], tempty[b]: the accumulators
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::STAGES;
    const uint32_t tfull0 = empty0 + 8 * C::STAGES, tempty0 = tfull0 + 8 * C::NBUF, drain0 = tempty0 + 8 * C::NBUF;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * C::STAGES + 2 * C::NBUF + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    volatile int* never = abort_flag + 1;
    uint32_t* s_amax = tmem_holder + 4;                  // gated: [2][4] warp maxima
    float* s_scale = reinterpret_cast<float*>(smem + C::OFF_SCALE);
    float* recv = reinterpret_cast<float*>(smem + C::OFF_RECV);

    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();             // its share of the contracted axis
    const uint32_t ctiles = (p.C + 127) / 128;
    const uint32_t cb = (blockIdx.x >> p.log_split) % ctiles;       // 128 output columns
    const uint32_t m0 = (blockIdx.x >> p.log_split) / ctiles * TN;
    const uint32_t mt = min(p.M - m0, (uint32_t)TN);     // tokens of this tile
    const uint32_t blocks = (p.T + 127) / 128;
    const uint32_t t0 = (uint32_t)((uint64_t)blocks * rank >> p.log_split);
    const uint32_t nb = (uint32_t)((uint64_t)blocks * (rank + 1) >> p.log_split) - t0;
    const uint32_t log_per = 31 - __clz(TN) - p.log_split;          // tokens that a CTA finishes
    const auto load_w = [&](uint32_t j, uint32_t pr, auto fn) {      // block t0 + j of projection pr
        const int32_t k = (int32_t)((t0 + j) * 128), c = (int32_t)(cb * 128 + pr * p.C);
        fn(C::W_MN ? c : k, C::W_MN ? k : c);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < C::NBUF; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, C::GATED ? 4 : 8);
        }
        mbar_init(drain0, 1);
        mbar_init(drain0 + 8, 1);
        *abort_flag = 0;
        *never = 0;
        fence_mbarrier_init();
    }
    if (warp == 8 && lane == 0) {
        prefetch_tensormap(&tmap_w);
        prefetch_tensormap(&tmap_a);
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_holder), C::TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    cluster_arrive_relaxed();                            // this CTA runs: its shared memory may be written
    griddep_wait();
    griddep_launch();
    const auto gave_up = [&] {
        *abort_flag = 1;
        atomicOr(p.status, kStatusTimeout);
    };

    if (warp == 8) {
        // ---------------------------------------------------------- loads
        if (lane == 0) {
            bool ok = true;
            uint32_t u = 0;
            for (; u < nb * C::P; ++u) {
                const uint32_t s = u % C::STAGES, use = u / C::STAGES, j = u / C::P;
                if (use > 0 && !fp8_wait(empty0 + 8 * s, (use - 1) & 1, abort_flag, p.wait_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t st = smem_u32(smem + s * C::STAGE_BYTES);
                mbar_arrive_expect_tx(full0 + 8 * s, C::STAGE_BYTES);
                load_w(j, u % C::P, [&](int32_t x, int32_t y) { tma_load_2d(st, &tmap_w, full0 + 8 * s, x, y); });
                tma_load_2d(st + C::W_BYTES, &tmap_a, full0 + 8 * s, (int32_t)((t0 + j) * 128), (int32_t)m0);
            }
            if (!ok) gave_up();
            for (uint32_t i = u > (uint32_t)C::STAGES ? u - C::STAGES : 0; i < u; ++i)     // no load left in flight
                fp8_wait(full0 + 8 * (i % C::STAGES), (i / C::STAGES) & 1, never, kFp8WaitNs);
        }
    } else if (warp == 9 || warp == 10) {
        // ---------------------------------------------------------- MMAs: unit u = block * P + projection
        if (lane == 0) {
            const uint32_t w = warp - 9;
            bool ok = true;
            for (uint32_t u = w; u < nb * C::P; u += 2) {
                const uint32_t s = u % C::STAGES, b = u % C::NBUF, use = u / C::NBUF;
                if (!fp8_wait(full0 + 8 * s, (u / C::STAGES) & 1, abort_flag, p.wait_ns) ||
                    (use > 0 && !fp8_wait(tempty0 + 8 * b, (use - 1) & 1, abort_flag, p.wait_ns))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = smem_u32(smem + s * C::STAGE_BYTES);
                const uint32_t ws = st, as = st + C::W_BYTES;
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k)
                    tc_mma_f8(tmem + b * TN, smem_desc(ws + k * C::W_STEP, 1024, 1024, 2), smem_desc(as + k * 32, 1024, 1024, 2),
                              C::IDESC, k != 0);
                tc_commit(tfull0 + 8 * b);
                tc_commit(empty0 + 8 * s);
            }
            if (!ok) gave_up();
            tc_commit(drain0 + 8 * w);
            fp8_wait(drain0 + 8 * w, 0, never, kFp8WaitNs);
        }
    } else {
        // ---------------------------------------------------------- epilogue: thread = weight row 32 q + lane
        const uint32_t q = warp & 3, g = warp >> 2, n = 32 * q + lane;
        const uint32_t first = C::GATED ? 0 : g * C::NT;             // first token of the thread
        const uint32_t lanes = tmem + ((32 * q) << 16) + first;
        const uint32_t kb_all = (p.T + 127) / 128;
        uint64_t acc[C::NT / 2] = {};
        bool ok = true;
        for (uint32_t j = 0; j < nb; ++j) {
            const uint32_t jc = j % C::CHUNK;
            if (jc == 0) {
                // scales of the next CHUNK blocks: the token's times the weight tile's
                if (j > 0) named_barrier_sync(1, 256);
                const uint32_t count = min(nb - j, (uint32_t)C::CHUNK) * TN;
                for (uint32_t i = threadIdx.x; i < C::P * count; i += 256) {
                    const uint32_t pr = i / count, e = i % count, t = t0 + j + e / TN, m = e % TN;
                    const uint64_t sw_at = OP == kFp8Dgrad ? (uint64_t)t * ctiles + cb : (uint64_t)(cb + pr * ctiles) * kb_all + t;
                    float v = 0.0f;
                    if (m < mt && in_bounds((uint64_t)t * p.M + m0 + m, 1, (uint64_t)kb_all * p.M, p.status) &&
                        in_bounds(sw_at, 1, (uint64_t)C::P * ctiles * kb_all, p.status))
                        v = __fmul_rn(__ldg(p.sa + (size_t)t * p.M + m0 + m), __ldg(p.sw + sw_at));
                    s_scale[pr * C::CHUNK * TN + e] = v;
                }
                named_barrier_sync(1, 256);
            }
            const uint32_t u = j * C::P + (C::GATED ? g : 0), b = u % C::NBUF;
            // every warp comes to the barriers above, whether its wait has given up or not
            if (ok && !fp8_wait_warp(tfull0 + 8 * b, (u / C::NBUF) & 1, abort_flag, p.wait_ns)) {
                ok = false;
                if (lane == 0) gave_up();
            }
            if (!ok) continue;
            tc_fence_after();
            const uint32_t sc = smem_u32(s_scale + (C::GATED ? g * C::CHUNK * TN : 0) + jc * TN + first);
            constexpr int CS = C::NT < 16 ? 8 : 16;
#pragma unroll
            for (int c = 0; c < C::NT; c += CS) {
                uint32_t v[CS];
                if constexpr (CS == 8) {
                    tc_ld_32x32b_x8(lanes + b * TN + c, v);
                } else {
                    tc_ld_32x32b_x16(lanes + b * TN + c, v);
                }
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < CS / 2; i += 2) {
                    uint64_t s0, s1;
                    lds_2xf32x2(sc + 4 * (c + 2 * i), s0, s1);
                    tmem_fma2(acc[c / 2 + i], v[2 * i], v[2 * i + 1], s0);
                    tmem_fma2(acc[c / 2 + i + 1], v[2 * i + 2], v[2 * i + 3], s1);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(tempty0 + 8 * b);
        }
        cluster_wait();                                  // every CTA of the cluster runs
        // token m's partial sums go to its owner, rank m >> log_per:
        // recv[(source rank * tokens per owner + m) * P + projection][row]
        const uint32_t mine = smem_u32(recv + n) + (((rank << log_per) * C::P) + (C::GATED ? g : 0)) * 512;
        uint32_t owner = ~0u, dst = 0;
#pragma unroll
        for (int i = 0; i < C::NT; ++i) {
            const uint32_t m = first + i;
            if (m >> log_per != owner) {
                owner = m >> log_per;
                dst = mapa_shared(mine, owner);
            }
            const float2 x = f32x2_unpack(acc[i / 2]);
            if (m < mt) st_shared_cluster_u32(dst + (m & ((1u << log_per) - 1)) * (C::P * 512), __float_as_uint(i & 1 ? x.y : x.x));
        }
    }
    __syncwarp();
    if (warp >= 8) cluster_wait();
    // the bias comes in while the partial sums travel
    const uint32_t bcol = cb * 128 + 32 * (warp & 3) + lane;
    const float bias = OP == kFp8Linear && warp < 8 && p.bias && bcol < p.C ? __bfloat162float(p.bias[bcol]) : 0.0f;
    cluster_sync();                                      // every partial sum has arrived
    if (warp < 8) {
        const uint32_t q = warp & 3, g = warp >> 2, n = 32 * q + lane;
        const uint32_t per = 1u << log_per, col = cb * 128 + n, split = 1u << p.log_split;
#pragma unroll 4
        for (uint32_t i = g; i < per; i += 2) {
            const uint32_t m = (rank << log_per) + i;
            if (m >= mt) break;
            float v[C::P];
#pragma unroll
            for (uint32_t pr = 0; pr < (uint32_t)C::P; ++pr) {
                v[pr] = recv[(i * C::P + pr) * 128 + n];
                for (uint32_t r = 1; r < split; ++r) v[pr] = __fadd_rn(v[pr], recv[(((r << log_per) + i) * C::P + pr) * 128 + n]);
            }
            const size_t row = m0 + m;
            if (C::GATED) {
                const float gate = v[0], up = v[C::P - 1];
                const float y = silu_mul(gate, up);
                const uint64_t at = row * p.ldo + col, gu_n = pitched_extent(p.M, 2 * p.C, p.ldo);
                if (p.out && in_bounds(at, 1, gu_n, p.status) && in_bounds(at + p.C, 1, gu_n, p.status)) {
                    p.out[at] = __float2bfloat16_rn(gate);
                    p.out[at + p.C] = __float2bfloat16_rn(up);
                }
                const uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, abs_bits(y));
                named_barrier_sync(2 + g, 128);          // the last token's maxima have been read
                if (lane == 0) s_amax[4 * g + q] = mx;
                named_barrier_sync(2 + g, 128);
                const Fp8Scale s = fp8_block_scale(max(max(s_amax[4 * g], s_amax[4 * g + 1]), max(s_amax[4 * g + 2], s_amax[4 * g + 3])),
                                                   p.status);
                if (in_bounds(row * p.C + col, 1, (uint64_t)p.M * p.C, p.status))
                    p.h_codes[row * p.C + col] = (uint8_t)cvt_e4m3x2(0.0f, __fmul_rn(y, s.factor));
                if (n == 0 && in_bounds((uint64_t)cb * p.M + row, 1, (uint64_t)ctiles * p.M, p.status))
                    p.h_scales[(size_t)cb * p.M + row] = s.scale;
            } else if (col < p.C && in_bounds(row * p.ldo + col, 1, pitched_extent(p.M, p.C, p.ldo), p.status)) {
                float y = v[0];
                if (OP == kFp8Linear && p.bias) y = __fadd_rn(y, bias);
                p.out[row * p.ldo + col] = __float2bfloat16_rn(y);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TM_COLS);
    }
}

}  // namespace nvq
