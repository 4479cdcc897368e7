// fp8_gemm.cuh -- products of E4M3 operands with one FP32 scale per block of 128.
//
//   out[r, c] = sum over blocks t of 128 of the contracted axis:
//                 sa(r, t) * sb(c, t) * sum_{k in t} a(r, k) * b(c, k)      (+ bias[c])
//
// linear    a = activations [M, K] row-wise, b = weights [N, K] tile-wise
// dgrad     a = dY [M, N] row-wise, b = the same weights read along N
// wgrad     a = dY [M, N], b = X [M, K], both column-wise and read along M
// gated     linear onto gate and up; H = SiLU(gate) * up quantized row-wise
//
// The scales are FP32, so the tensor core cannot apply them (its own block
// scales are powers of two): each block's sum is taken by MMAs into tensor
// memory, and 8 epilogue warps read it, multiply by the scales and add it to
// the FP32 total in their registers while the MMAs go on.
//
// CTA pairs, one per two SMs, persistent over 256 x 256 output tiles (gated: 256
// rows x 128 columns of H, gate's 128 columns and up's as one 256-wide B tile).
// CTA r stages rows [128 r, 128 r + 128) of the A tile and of the B tile (128
// bytes of the contracted axis, one block, per stage), holds output rows
// [128 r, 128 r + 128) and drains them.  Operands whose contracted axis is not
// the contiguous one (wgrad's, dgrad's weight) are staged as they lie in memory,
// 128 of the contracted axis x 128 contiguous bytes, and read "MN-major" by the
// MMA: no transposed copies.
//
// A block is two units, h = 0 and 1: the MMA of unit h reads rows [64 h, 64 h +
// 64) of each CTA's B tile, so its 128 accumulator columns are tile columns
// 64 h .. + 63 and 128 + 64 h .. + 63.  Tensor memory holds four units, two of
// each h.  From an accumulator's completion to the MMA that may overwrite it lie
// three hand-overs between threads (200 to 400 cycles each) and the drain; with two
// 256-wide accumulators the tensor pipe stood idle for half of that time (906 cycles
// a block without the multiply-adds, 727 with units; the MMAs alone take 512).
// Warps 0-7: epilogue, warp w reads tensor-memory lanes 32 (w % 4) .. + 31 of
// units h = w / 4; 8: tile loads; 9: scales, by 4-byte copies into a ring that runs
// as far ahead as the tiles (L2 answers after some 2,000 cycles while the tiles
// stream in: reading them two blocks ahead in the epilogue cost 80 us of 298);
// 10-13: MMAs (in the leader CTA), a warp per accumulator.  One thread spends at
// least 86 cycles on issuing an MMA that takes the tensor pipe 64, and 130 on a
// commit: four MMAs and two commits alone measured 390 cycles a unit from two
// warps, 276 from four, where the pipe needs 256.
// The totals take 128 registers of an epilogue thread; a spill in its loop goes
// through a first-level cache that shared memory has left almost nothing of, and
// cost up to a third of the kernel's time, hence the register split.
//
// Measured at 4608 x 12288 x 4096, values from normal ones, on several boxes: 230 to 236 us in
// short runs (1,970 to 2,017 TFLOP/s, SM clock 1.7 GHz), 276 to 284 us over seconds (1,630 to
// 1,680 TFLOP/s, at the power limit; a BF16 library product reaches 1,360 there); in short runs dgrad
// 4608 x 4096 x 12288 224 to 232 us, wgrad 355 us (its column scales are one more multiply and a
// shared-memory read for each pair of values), gated with gate and up kept 524 us (590 to 610 over seconds).
// What bounds it is the epilogue: about 1,010 cycles a block, of which 500 drain and
// add, 200 the scales, 100 to 200 each the accumulator's barrier and the release, and
// 200 a tile's share of output; shared memory answers slowly beside the tensor core's
// operand reads.  Tried and not kept: 16 epilogue warps of 64 columns (1,240 cycles), 32-byte
// stores from registers in place of the staged tensor-map stores (1,230), the next block's
// scales read before the last chunk is added (244 us against 230), longer chunks (spills).
// Every wait is bounded (status word and abort flag), as in gemm_pair.cuh; warps that share a barrier, and
// the lanes of a warp, leave together when one runs out.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "debug.cuh"
#include "fp8_gated.cuh"
#include "fp8_ptx.cuh"

namespace nvq {

enum Fp8Op { kFp8Linear = 0, kFp8Dgrad = 1, kFp8Wgrad = 2, kFp8Gated = 3 };

constexpr uint32_t kFp8WaitNs = 4000000000u;            // 4 s per pipeline wait
// What a load in flight is given once its CTA has aborted, when its barrier's other arrivals may never come:
// a thousand times what it takes to land.  Without an abort it has the full limit.
constexpr uint32_t kFp8AbortNs = 10000000u;

struct Fp8GemmParams {
    const uint8_t* a;           // plain A loads only
    const float* sa;            // [T / 128][R]
    const float* sb;            // linear, gated: [B rows / 128][T / 128]; dgrad: [T / 128][C / 128]; wgrad: [T / 128][C]
    const __nv_bfloat16* bias;
    uint8_t* h_codes;           // gated: [R, C] and [C / 128][R]
    float* h_scales;
    unsigned int* status;
    uint32_t R, C, T;           // output rows, columns (gated: F), contracted length
    uint32_t row_tiles, col_tiles;
    uint32_t accumulate;        // wgrad: add to out
    uint32_t save;              // gated: store gate and up
    uint32_t wait_ns;
};

template <int OP, bool PLAIN_A = false>
struct Fp8PairCfg {
    static constexpr bool A_MN = OP == kFp8Wgrad;                       // A's contiguous axis is its row axis
    static constexpr bool B_MN = OP == kFp8Wgrad || OP == kFp8Dgrad;
    static constexpr bool SB_COL = OP == kFp8Wgrad;                     // one B scale per column
    static constexpr int EPI_WARPS = 8;
    static constexpr int LOAD_WARP = EPI_WARPS, SCALE_WARP = LOAD_WARP + 1, MMA_WARP = LOAD_WARP + 2;
    static constexpr int MMA_WARPS = PLAIN_A ? 2 : 4;                   // plain loads need the warps
    static constexpr int THREADS = 32 * (EPI_WARPS + 8);                // four warpgroups
    // registers a thread: 512 x 128 at launch, shared out 256 x 208 + 256 x 48
    static constexpr int EPI_REGS = 208, OTHER_REGS = 48;
    static_assert(32 * EPI_WARPS * EPI_REGS + 256 * OTHER_REGS <= THREADS * 128, "register split");
    static constexpr int TILE_BYTES = 128 * 128;                        // 128 rows x 128 bytes
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;                  // A and B tile of one CTA
    static constexpr int STAGES = PLAIN_A ? 4 : 6;                       // plain loads: one for each of their warps
    static constexpr int STAGING = 32 * 64;                             // per epilogue warp: one chunk
    // scale slot of a block: 128 row scales, then 256 column scales or the two tile scales; slots are
    // filled GROUP blocks at a time, with one barrier a group
    static constexpr int SLOT_BYTES = 512 + (SB_COL ? 1024 : 16);
    static constexpr int GROUP = SB_COL ? 2 : 4;
    static constexpr int GROUPS = SB_COL ? 5 : 4;
    static constexpr int SLOTS = GROUP * GROUPS;
    static constexpr int AMAX_BYTES = OP == kFp8Gated ? 2 * 256 * 4 : 0;
    static constexpr int BAR_BYTES = 384;
    static constexpr int SMEM_LIMIT = 232448;
    static constexpr int OFF_STAGING = STAGES * STAGE_BYTES;
    static constexpr int OFF_AMAX = OFF_STAGING + EPI_WARPS * STAGING;
    static constexpr int OFF_SCALE = OFF_AMAX + AMAX_BYTES;
    static constexpr int OFF_BAR = OFF_SCALE + SLOTS * SLOT_BYTES;
    static constexpr int SMEM_BYTES = OFF_BAR + BAR_BYTES + 1024;
    // instruction descriptor of kind::f8f6f4: FP32 accumulator, E4M3 x E4M3, major-ness, N / 8, M / 16
    static constexpr uint32_t IDESC = (1u << 4) | ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) |
                                      ((128u >> 3) << 17) | ((256u >> 4) << 24);
    // K step of 32 within a stage: 32 bytes along a row, or 32 rows of 128 bytes
    static constexpr uint32_t A_STEP = A_MN ? 4096 : 32, B_STEP = B_MN ? 4096 : 32;
    static constexpr uint32_t B_UNIT = B_MN ? 64 : 64 * 128;            // from unit 0's B to unit 1's
    static_assert(SMEM_BYTES <= SMEM_LIMIT, "shared memory");
    static_assert(EPI_WARPS + 2 + MMA_WARPS + (PLAIN_A ? 4 : 0) <= THREADS / 32, "warps");
    static_assert((2 * STAGES + 8 + MMA_WARPS + 2 * GROUPS) * 8 + 16 <= BAR_BYTES, "barriers");
};

// Bounded wait of the pipeline: gives up after limit_ns or when *abort is set.
// The clock is read on every 64th attempt only (each attempt suspends the
// thread for a while), so a wait that is about to end costs no timer reads;
// where the limit is shorter than those attempts may take, on every one.
constexpr uint64_t kFp8ShortLimitNs = 1000000u;

template <bool CLUSTER = false>
__device__ __forceinline__ bool fp8_wait(uint32_t bar, uint32_t parity, const volatile int* abort, uint64_t limit_ns) {
    uint64_t t0 = 0;
    const uint32_t mask = limit_ns < kFp8ShortLimitNs ? 0 : 63;
    for (uint32_t n = 0;; ++n) {
        uint32_t ok;
        if (CLUSTER)
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        else
            ok = mbar_try_wait(bar, parity);
        if (ok) return true;
        if ((n & mask) == mask) {
            if (*abort) return false;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            else if (t - t0 > limit_ns) return false;
        }
    }
}

// The same for a whole warp, with one decision: each lane reads the abort flag and the clock for itself, and
// what follows a wait (tensor-memory loads, barriers, __syncwarp) takes every lane.
__device__ __forceinline__ bool fp8_wait_warp(uint32_t bar, uint32_t parity, const volatile int* abort, uint64_t limit_ns) {
    return __all_sync(0xFFFFFFFFu, fp8_wait(bar, parity, abort, limit_ns));
}

// Warps of plain loads, each with a stage of its own: the proxy fence that publishes
// a stage's copies waits for all that its warp has in flight, so more than one at a
// time would come one after the other (dgrad of 1111 x 2056 x 1552: a quarter of each
// of six stages to a warp 24.2 us, three warps with two stages each 19.5, this 17.9).
constexpr uint32_t kFp8PlainWarps = 4;

// Stage a 128-row x 128-byte tile of a matrix whose pitch is not a multiple of 16
// bytes (a tensor map cannot describe it) with one warp: 8-byte copies, laid out
// in the 128-byte swizzle that a tensor-map load would write (16-byte chunk c of
// row r at chunk c ^ (r % 8)), zeros outside the matrix.
__device__ __forceinline__ void fp8_plain_tile(uint32_t dst, const uint8_t* src, uint32_t rows, uint32_t cols, uint32_t r0,
                                               uint32_t c0, uint32_t lane, unsigned int* status) {
    const uint32_t c = c0 + (lane & 15) * 8;
    const uint64_t end = (uint64_t)rows * cols;
#pragma unroll
    for (uint32_t part = 0; part < 4; ++part) {
        const uint32_t i0 = 2 * part + (lane >> 4);                                       // rows i0 + 8 j
        const uint32_t live = c < cols && r0 + i0 < rows ? (rows - r0 - i0 + 7) / 8 : 0;  // of them inside
        const uint32_t d = dst + i0 * 128 + ((((lane & 15) >> 1) ^ (i0 & 7)) << 4) + (lane & 1) * 8;
        uint64_t at = (uint64_t)(r0 + i0) * cols + c;
#pragma unroll
        for (uint32_t j = 0; j < 16; ++j, at += 8 * (uint64_t)cols) {
            const bool in = j < live && in_bounds(at, 8, end, status);
            cp_async8_zfill(d + j * 1024, in ? src + at : src, in ? 8 : 0);
        }
    }
}

// Writes one 32-row x 64-byte chunk (v: this thread's row) through the warp's
// staging buffer: 64-byte swizzle, then a tensor-map store, or an addition.
__device__ __forceinline__ void fp8_store_chunk(const uint32_t (&v)[16], uint8_t* buf, const CUtensorMap* map, int32_t c,
                                                int32_t r, uint32_t lane, bool add) {
    const uint32_t swz = (lane >> 1) & 3;
    if (lane == 0) bulk_wait_group_read<0>();            // the previous store has read the buffer
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(buf + lane * 64 + 16 * ((uint32_t)i ^ swz)) =
            make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (add) tma_reduce_add_2d(map, smem_u32(buf), c, r);
        else tma_store_2d(map, smem_u32(buf), c, r);
        bulk_commit_group();
    }
}

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    const __nv_bfloat162 o = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&o);
}

template <int OP, bool PLAIN_A>
__global__ void __launch_bounds__(Fp8PairCfg<OP, PLAIN_A>::THREADS, 1)
fp8_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                     const __grid_constant__ CUtensorMap tmap_out, const Fp8GemmParams p) {
    using C = Fp8PairCfg<OP, PLAIN_A>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    // full[s]:   the stage's tiles of both CTAs landed (leader's barrier)
    // empty[s]:  both units' MMAs of the stage completed (commits multicast to both CTAs)
    // tfull[b]:  accumulator b (of unit b % 2) holds a block's sums (both CTAs)
    // tempty[b]: both CTAs' epilogue warps have read accumulator b (leader's barrier)
    // sfull[i]:  group i of scale slots is filled (each lane of the scale warp arrives)
    // sempty[i]: this CTA's epilogue warps are past group i
    const uint32_t full0 = smem_u32(bars);
    const uint32_t empty0 = full0 + 8 * C::STAGES;
    const uint32_t tfull0 = empty0 + 8 * C::STAGES;
    const uint32_t tempty0 = tfull0 + 32;
    const uint32_t drain0 = tempty0 + 32;
    const uint32_t sfull0 = drain0 + 8 * C::MMA_WARPS;
    const uint32_t sempty0 = sfull0 + 8 * C::GROUPS;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * C::STAGES + 8 + C::MMA_WARPS + 2 * C::GROUPS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    volatile int* never = abort_flag + 1;

    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();             // 0 = leader
    const uint32_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full0 + 8 * s, PLAIN_A ? 3 : 1);
            mbar_init(empty0 + 8 * s, 2);
        }
        for (int b = 0; b < 4; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, 8);                 // four epilogue warps of each CTA
        }
        for (int m = 0; m < C::MMA_WARPS; ++m) mbar_init(drain0 + 8 * m, 1);
        for (int i = 0; i < C::GROUPS; ++i) {
            mbar_init(sfull0 + 8 * i, 32);
            mbar_init(sempty0 + 8 * i, C::EPI_WARPS);
        }
        *abort_flag = 0;
        *never = 0;
        fence_mbarrier_init();
    }
    if (warp == C::LOAD_WARP && lane == 0) {
        if (!PLAIN_A) prefetch_tensormap(&tmap_a);
        prefetch_tensormap(&tmap_b);
        prefetch_tensormap(&tmap_out);
    }
    if (warp == C::MMA_WARP) {
        tmem_alloc_pair(smem_u32(tmem_holder), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();                                      // barriers of both CTAs initialised
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    griddep_wait();
    griddep_launch();
    const uint32_t num_tiles = p.row_tiles * p.col_tiles;
    const uint32_t blocks = (p.T + 127) / 128;
    const auto gave_up = [&] {
        *abort_flag = 1;
        atomicOr(p.status, kStatusTimeout);
    };

    if (warp >= C::EPI_WARPS) {
        regs_dec<C::OTHER_REGS>();
        if (warp == C::LOAD_WARP) {
            // ---------------------------------------------------------- tile loads (both CTAs)
            if (lane == 0) {
                uint32_t it = 0;
                bool ok = true;
                for (uint32_t tile = pair; tile < num_tiles && ok; tile += npairs) {
                    const uint32_t cb = tile / p.row_tiles;
                    const int32_t r0 = (int32_t)((tile % p.row_tiles) * 256 + 128 * rank);
                    const int32_t c0 = OP == kFp8Gated ? (int32_t)(cb * 128 + rank * p.C) : (int32_t)(cb * 256 + 128 * rank);
                    for (uint32_t t = 0; t < blocks; ++t, ++it) {
                        const uint32_t s = it % C::STAGES, use = it / C::STAGES;
                        if (use > 0 && !fp8_wait(empty0 + 8 * s, (use - 1) & 1, abort_flag, p.wait_ns)) {
                            ok = false;
                            break;
                        }
                        const uint32_t st = smem_u32(smem + s * C::STAGE_BYTES);
                        const int32_t k0 = (int32_t)(t * 128);
                        const uint32_t fb = mapa_shared(full0 + 8 * s, 0);
                        if (rank == 0)
                            mbar_arrive_expect_tx(full0 + 8 * s, 2 * (PLAIN_A ? C::TILE_BYTES : C::STAGE_BYTES));
                        if (!PLAIN_A) tma_load_2d_pair(st, &tmap_a, fb, C::A_MN ? r0 : k0, C::A_MN ? k0 : r0);
                        tma_load_2d_pair(st + C::TILE_BYTES, &tmap_b, fb, C::B_MN ? c0 : k0, C::B_MN ? k0 : c0);
                    }
                }
                if (!ok) gave_up();
                // Neither CTA leaves while a load it issued may be in flight: the leader's
                // barriers count both CTAs' bytes; the peer learns of its own through the
                // commits of the MMAs that consumed them.
                for (uint32_t j = it > (uint32_t)C::STAGES ? it - C::STAGES : 0; j < it; ++j) {
                    const uint32_t bar = (rank == 0 ? full0 : empty0) + 8 * (j % C::STAGES), phase = (j / C::STAGES) & 1;
                    // an abort, at its start or on the way, leaves it kFp8AbortNs
                    if (!fp8_wait(bar, phase, abort_flag, kFp8WaitNs)) fp8_wait(bar, phase, never, kFp8AbortNs);
                }
            }
        } else if (PLAIN_A && warp >= C::THREADS / 32 - kFp8PlainWarps) {
            // ---------------------------------------------------------- plain A tiles (both CTAs)
            static_assert(!PLAIN_A || C::STAGES % kFp8PlainWarps == 0, "a warp sees every phase of its stages' barriers");
            uint32_t it = 0, turn = warp - (C::THREADS / 32 - kFp8PlainWarps);
            bool ok = true;
            for (uint32_t tile = pair; tile < num_tiles && ok; tile += npairs) {
                const uint32_t r0 = (tile % p.row_tiles) * 256 + 128 * rank;
                for (uint32_t t = 0; t < blocks; ++t, ++it) {
                    if (it != turn) continue;
                    turn += kFp8PlainWarps;
                    const uint32_t s = it % C::STAGES, use = it / C::STAGES;
                    if (use > 0 && !fp8_wait_warp(empty0 + 8 * s, (use - 1) & 1, abort_flag, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = smem_u32(smem + s * C::STAGE_BYTES);
                    if (C::A_MN) fp8_plain_tile(st, p.a, p.T, p.R, t * 128, r0, lane, p.status);
                    else fp8_plain_tile(st, p.a, p.R, p.T, r0, t * 128, lane, p.status);
                    cp_async_commit();
                    cp_async_wait<0>();
                    // publish the copies to the leader's MMAs
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(mapa_shared(full0 + 8 * s, 0));
                }
            }
            if (!ok && lane == 0) gave_up();
        } else if (warp == C::SCALE_WARP) {
            // ---------------------------------------------------------- scales (both CTAs)
            const uint32_t cblocks = (p.C + 127) / 128;
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t tile = pair; tile < num_tiles && ok; tile += npairs) {
                const uint32_t r0 = (tile % p.row_tiles) * 256 + 128 * rank, cb = tile / p.row_tiles;
                const uint32_t nb = OP == kFp8Gated ? cb + (lane & 1) * cblocks : min(2 * cb + (lane & 1), cblocks - 1);
                for (uint32_t t = 0; t < blocks; ++t, ++it) {
                    if (it % C::GROUP == 0) {
                        const uint32_t n = it / C::GROUP;
                        if (n > 0) cp_async_arrive(sfull0 + 8 * ((n - 1) % C::GROUPS));
                        if (n >= (uint32_t)C::GROUPS &&
                            !fp8_wait_warp(sempty0 + 8 * (n % C::GROUPS), (n / C::GROUPS - 1) & 1, abort_flag, p.wait_ns)) {
                            ok = false;
                            break;
                        }
                    }
                    const uint32_t slot = smem_u32(smem + C::OFF_SCALE + (it % C::SLOTS) * C::SLOT_BYTES);
                    const float* sa = p.sa + (size_t)t * p.R;
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) {
                        const uint32_t r = r0 + lane + 32 * i;
                        const bool in = r < p.R && in_bounds((uint64_t)t * p.R + r, 1, (uint64_t)blocks * p.R, p.status);
                        cp_async4_zfill(slot + 4 * (lane + 32 * i), in ? sa + r : p.sa, in ? 4 : 0);
                    }
                    if (C::SB_COL) {
                        const float* sb = p.sb + (size_t)t * p.C;
#pragma unroll
                        for (uint32_t i = 0; i < 2; ++i) {              // C is a multiple of 16
                            const uint32_t c = cb * 256 + 4 * (lane + 32 * i);
                            const bool in = c < p.C && in_bounds((uint64_t)t * p.C + c, 4, (uint64_t)blocks * p.C, p.status);
                            cp_async16_zfill(slot + 512 + 16 * (lane + 32 * i), in ? sb + c : p.sb, in ? 16 : 0);
                        }
                    } else if (lane < 2) {
                        const uint64_t at = OP == kFp8Dgrad ? (uint64_t)t * cblocks + nb : (uint64_t)nb * blocks + t;
                        const bool in = in_bounds(at, 1, (uint64_t)blocks * (OP == kFp8Gated ? 2 : 1) * cblocks, p.status);
                        cp_async4_zfill(slot + 512 + 4 * lane, in ? p.sb + at : p.sb, in ? 4 : 0);
                    }
                }
            }
            if (it > 0) cp_async_arrive(sfull0 + 8 * ((it - 1) / C::GROUP % C::GROUPS));   // the last group, whole or not
            if (!ok && lane == 0) gave_up();
            cp_async_commit();
            cp_async_wait<0>();
        } else if (warp < C::MMA_WARP + C::MMA_WARPS) {
            // ---------------------------------------------------------- MMAs (leader), a warp per accumulator
            // Warp m fills accumulator m: unit m % 2 of every other block, and so of every other stage
            // (two warps: both accumulators of unit m).
            static_assert(C::STAGES % 2 == 0, "a warp sees every phase of its stages' barriers");
            if (lane == 0 && rank == 0) {
                const uint32_t m = warp - C::MMA_WARP;
                const uint32_t my_tiles = num_tiles > pair ? (num_tiles - pair + npairs - 1) / npairs : 0;
                const uint32_t total = my_tiles * blocks;
                bool ok = true;
                for (uint32_t it = m >> 1; it < total; it += C::MMA_WARPS / 2) {
                    const uint32_t s = it % C::STAGES, b = (m & 1) + 2 * (it & 1);
                    if (!fp8_wait<PLAIN_A>(full0 + 8 * s, (it / C::STAGES) & 1, abort_flag, p.wait_ns) ||
                        (it >= 2 && !fp8_wait(tempty0 + 8 * b, ((it >> 1) - 1) & 1, abort_flag, p.wait_ns))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = smem_u32(smem + s * C::STAGE_BYTES), bt = st + C::TILE_BYTES + (m & 1) * C::B_UNIT;
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k)
                        tc_mma_f8_pair(tmem + b * 128, smem_desc(st + k * C::A_STEP, 1024, 1024, 2),
                                       smem_desc(bt + k * C::B_STEP, 1024, 1024, 2), C::IDESC, k != 0);
                    tc_commit_pair_mc(tfull0 + 8 * b, 0x3);
                    tc_commit_pair_mc(empty0 + 8 * s, 0x3);
                }
                if (!ok) gave_up();
                tc_commit_pair(drain0 + 8 * m);
                fp8_wait(drain0 + 8 * m, 0, never, kFp8WaitNs);
            }
        }
    } else {
        regs_inc<C::EPI_REGS>();
        // ---------------------------------------------------------- epilogue (both CTAs)
        const uint32_t q = warp & 3, h = warp >> 2;
        uint8_t* staging = smem + C::OFF_STAGING + warp * C::STAGING;
        uint32_t* s_amax = reinterpret_cast<uint32_t*>(smem + C::OFF_AMAX);
        // column i of a unit (i < 64: of the first 128 of the tile, gated: of gate) is tile column
        // 64 h + i, or 64 h + 64 + i
        const uint32_t lanes = tmem + ((32 * q) << 16);
        const uint32_t cblocks = (p.C + 127) / 128;
        const uint32_t scales = smem_u32(smem + C::OFF_SCALE);
        // where this CTA's releases go: the leader's barriers
        const uint32_t release0 = mapa_shared(tempty0 + 8 * h, 0), release1 = mapa_shared(tempty0 + 8 * (h + 2), 0);
        uint32_t it = 0, slot = 0, sslot = 0, sphase = 0;
        bool ok = true, ready = false;
        for (uint32_t tile = pair; tile < num_tiles && ok; tile += npairs) {
            const uint32_t rw = (tile % p.row_tiles) * 256 + 128 * rank + 32 * q;      // the warp's first row
            const uint32_t cb = tile / p.row_tiles;
            const uint32_t r = rw + lane;
            const uint32_t n0 = cb * (OP == kFp8Gated ? 128 : 256);                    // the tile's first column
            uint64_t acc[64] = {};                          // columns 2i, 2i + 1 of the unit
            for (uint32_t t = 0; t < blocks; ++t, ++it) {
                const uint32_t b = h + 2 * (it & 1);
                // A lane whose wait for scales gives up says so and goes on with what the slot holds; the warp leaves at
                // its next wait for an accumulator that is not there yet (a vote here cost 1 to 2 % of the kernel).
                if (sslot % C::GROUP == 0) {
                    if (!fp8_wait(sfull0 + 8 * (sslot / C::GROUP), sphase, abort_flag, p.wait_ns)) gave_up();
                    __syncwarp();
                }
                const uint32_t block_scale = scales + sslot * C::SLOT_BYTES;
                if (++sslot == (uint32_t)C::SLOTS) {
                    sslot = 0;
                    sphase ^= 1;
                }
                const float sa = lds_f32(block_scale + 4 * (32 * q + lane));
                const float f0 = C::SB_COL ? sa : __fmul_rn(sa, lds_f32(block_scale + 512));
                const float f1 = C::SB_COL ? sa : __fmul_rn(sa, lds_f32(block_scale + 516));
                const uint64_t s0 = f32x2_pack(f0, f0), s1 = f32x2_pack(f1, f1);
                if (!ready && !fp8_wait_warp(tfull0 + 8 * b, (it >> 1) & 1, abort_flag, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // a chunk's load runs while the chunk before it is added
                const uint32_t src = lanes + b * 128;
                uint32_t v[2][16];
                const auto add = [&](int j) {
                    const uint32_t(&x)[16] = v[j & 1];
                    const uint64_t s = j < 4 ? s0 : s1;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (C::SB_COL) {
                            uint64_t c0, c1;
                            lds_2xf32x2(block_scale + 512 + 4 * (64 * h + 16 * j + (j < 4 ? 0 : 64) + 4 * i), c0, c1);
                            tmem_fma2(acc[8 * j + 2 * i], x[4 * i], x[4 * i + 1], c0, s);
                            tmem_fma2(acc[8 * j + 2 * i + 1], x[4 * i + 2], x[4 * i + 3], c1, s);
                        } else {
                            tmem_fma2(acc[8 * j + 2 * i], x[4 * i], x[4 * i + 1], s);
                            tmem_fma2(acc[8 * j + 2 * i + 1], x[4 * i + 2], x[4 * i + 3], s);
                        }
                    }
                };
                tc_ld_32x32b_x16(src, v[0]);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 7; ++j) {
                    tc_ld_32x32b_x16(src + 16 * (j + 1), v[(j + 1) & 1]);
                    add(j);
                    tc_wait_ld();
                }
                tc_fence_before();
                __syncwarp();
                // the loads have returned, and the signal publishes no memory writes
                if (lane == 0) mbar_arrive_relaxed_cluster(b == h ? release0 : release1);
                // look at the next block's accumulator while the last chunk is added (a vote at the wait itself, ready or
                // not, cost 2 to 3 % of the kernel; going on after any lost wait and voting once a group of scales 2 to 5 %)
                ready = __all_sync(0xFFFFFFFFu, mbar_test(tfull0 + 8 * (b ^ 2), ((it + 1) >> 1) & 1));
                add(7);
                if (sslot % C::GROUP == 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sempty0 + 8 * ((sslot == 0 ? C::GROUPS : sslot / C::GROUP) - 1));
                }
            }
            if (OP != kFp8Gated && !ok) break;
            if (OP == kFp8Gated) {
                const uint64_t h_n = (uint64_t)p.R * p.C;
                if (ok && p.save && rw < p.R) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t o[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 x = f32x2_unpack(acc[16 * j + i]);
                            o[i] = bf16x2_of(x.x, x.y);
                        }
                        fp8_store_chunk(o, staging, &tmap_out, (int32_t)(n0 + (j >> 1) * p.C + 64 * h + 32 * (j & 1)), (int32_t)rw,
                                        lane, false);
                    }
                }
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {             // acc[i] becomes H
                    const float2 x = f32x2_unpack(acc[i]), u = f32x2_unpack(acc[32 + i]);
                    const float y0 = silu_mul(x.x, u.x), y1 = silu_mul(x.y, u.y);
                    m = max(m, max(abs_bits(y0), abs_bits(y1)));
                    acc[i] = f32x2_pack(y0, y1);
                }
                // The row's block of 128 columns is shared by the two warps of this lane quarter.  They wait for
                // different accumulators, so one may have given up where the other has not: it says so in place of
                // its maximum, both come to the barrier once a tile and leave after the same one, before they make
                // anything of what a lost wait left.
                constexpr uint32_t kGaveUp = 0xFFFFFFFFu;  // magnitudes are below 2^31
                uint32_t* am = s_amax + 256 * slot + 32 * q + lane;
                if (!ok || *abort_flag) m = kGaveUp;
                am[128 * h] = m;
                named_barrier_sync(1 + q, 64);
                const uint32_t other = am[128 * (h ^ 1)];
                slot ^= 1;                                 // the next tile's writes may pass this one's reads
                m = max(m, other);
                if (__any_sync(0xFFFFFFFFu, m == kGaveUp)) {
                    ok = false;
                    break;
                }
                if (r < p.R) {
                    const Fp8Scale s = fp8_block_scale(m, p.status);
                    const uint64_t at = (uint64_t)r * p.C + n0 + 64 * h;
                    if (in_bounds(at, 64, h_n, p.status)) {
                        uint4* d = reinterpret_cast<uint4*>(p.h_codes + at);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 x = f32x2_unpack(acc[8 * i + 2 * e]), y = f32x2_unpack(acc[8 * i + 2 * e + 1]);
                                w[e] = cvt_e4m3x4(x.x * s.factor, x.y * s.factor, y.x * s.factor, y.y * s.factor);
                            }
                            d[i] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    if (h == 0 && in_bounds((uint64_t)cb * p.R + r, 1, (uint64_t)cblocks * p.R, p.status))
                        p.h_scales[(size_t)cb * p.R + r] = s.scale;
                }
            } else if (rw < p.R) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t c = n0 + 128 * (j >> 1) + 64 * h + 32 * (j & 1);
                    if (c >= p.C) continue;
                    uint32_t o[16];
                    if (OP == kFp8Wgrad) {
#pragma unroll
                        for (int part = 0; part < 2; ++part) {          // 16 FP32 columns a chunk
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float2 x = f32x2_unpack(acc[16 * j + 8 * part + i]);
                                o[2 * i] = __float_as_uint(x.x);
                                o[2 * i + 1] = __float_as_uint(x.y);
                            }
                            if (c + 16 * part < p.C)
                                fp8_store_chunk(o, staging, &tmap_out, (int32_t)(c + 16 * part), (int32_t)rw, lane,
                                                p.accumulate);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 x = f32x2_unpack(acc[16 * j + i]);
                            // C is a multiple of 8, so a pair of columns is inside or outside
                            if (OP == kFp8Linear && p.bias && c + 2 * i < p.C) {
                                const __nv_bfloat162 bb = *reinterpret_cast<const __nv_bfloat162*>(p.bias + c + 2 * i);
                                x.x = __fadd_rn(x.x, __bfloat162float(bb.x));
                                x.y = __fadd_rn(x.y, __bfloat162float(bb.y));
                            }
                            o[i] = bf16x2_of(x.x, x.y);
                        }
                        fp8_store_chunk(o, staging, &tmap_out, (int32_t)c, (int32_t)rw, lane, false);
                    }
                }
            }
        }
        if (!ok && lane == 0) gave_up();
        if (lane == 0) bulk_wait_group_all();
        __syncwarp();
    }

    tc_fence_before();
    cluster_sync();                                      // both CTAs done with the pair's resources
    if (warp == C::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

}  // namespace nvq
