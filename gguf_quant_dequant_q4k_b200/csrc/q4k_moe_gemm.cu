// q4k_moe_gemm.cu -- expert-grouped products of fp16 activations with Q4_K
// matrices (q4k_moe_gemm_f16, q4k_moe_gemm_swiglu_f16): y = x16 * W16_e^T, W16
// the fp16 mirror's values (the f32 weight d*sc*q - dmin*m rounded to
// binary16), formed inside the kernel from the superblocks.
//
// * Tiles. A pair of CTAs (one cluster, tensor cores joined by cta_group::2)
//   owns a tile of y^T: 256 rows of W_e (the MMA's M, 128 per CTA) by a block of
//   expert e's slots (N). An expert's slots are cut into equal blocks of at most
//   MoeShape::slots; N is the block's slots rounded up to 16. SwiGLU: 128 gate
//   and 128 up rows, per CTA 64 and 64, so that TMEM lanes 32q + l and 32q + 16 +
//   l (l < 16) hold gate and up of one feature. 74 persistent pairs walk the
//   tiles of all experts, the blocks of a row tile one after another.
// * A (weights). A producer streams 128 rows x 144 bytes per superblock into a
//   shared-memory ring (TMA). Three sets of four decode warps (a warp per TMEM
//   lane quarter, a lane per row) take the steps (two 64-weight quant groups) in
//   turn: the quants become f32 through binary16 subnormals, the weight is one
//   packed fma, rounded once, then cvt to fp16 pairs, stored to TMEM. The decoded
//   step feeds all N slots: its MMAs take 4 N cycles, at least 390 (reading A),
//   its decoding about 750 (500 on an SM that does nothing else), so blocks of
//   about 190 slots and more hide it.
// * B (activations). 128 elements of N / 2 rows per CTA and step, by TMA in the
//   128-byte-swizzled layout; the pair's tensor cores share the two halves. x
//   in slot order is read in place; otherwise a copy in slot order is made
//   first (a launch of its own into a stream-ordered workspace). Measured on
//   2048 tokens, top 2, 14336x4096: fetching each row inside the kernel with
//   16-byte async copies took 54 cycles per 512 bytes (1.23 ms in all), with
//   four-row TMA gathers about 90 cycles (2.8 ms).
// * D. The tensor core adds to D by truncation (measured 1.7e-5 relative over K =
//   14336); every kPlainChunk superblocks the plain form therefore moves D into
//   f32 registers, rounding to nearest (under 1e-6). The SwiGLU form rounds to
//   fp16 and keeps D for the whole row.
// * Measured (times are of calls back to back; the clock falls to about 1.5 GHz
//   under the large cases): 2048 tokens, 8 experts, top 2: gate/up 14336 x 4096
//   0.83-0.94 ms = 1030-1160 TFLOP/s (cuBLAS bf16, sustained: 1428), bound by
//   the MMAs, 1088 cycles per step of about 910; down 4096 x 14336 0.50-0.56 ms,
//   bound by the drains of D, which the MMAs wait for, and by 6 tiles per pair
//   where 5.2 are due. 777 tokens, 64 experts, top 4 (about 48 slots each): gate/up
//   1536 x 2048 111-121 us, down 56-61 us, bound by the latency of each decode
//   warp's chain, load - decode - store - wait - arrival (785 cycles per step, 624
//   without its arithmetic, 390 for the MMAs alone; issue slots 0.68).
// * Waits are bounded; a role that gives up raises Q4K_FAULT_COPY_TIMEOUT and
//   the CTA lets its copies and MMAs land before shared memory and TMEM go. The
//   longest wait in order is the SwiGLU epilogue's for a whole row, about 0.7 us per
//   step of 128 elements: 0.1 s for the longest row accepted, of about 1 s.
#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>

#include "q4k_internal.h"
#include "q4k_moe.h"
#include "q4k_pair.cuh"
#include "q4k_per_device.h"
#include "q4k_superblock.cuh"
#include "q4k_tensor_map.h"

namespace q4k {

__device__ unsigned int g_moe_gemm_fault_flags = 0;

namespace {

constexpr int kCtaRows = 128;                // W rows per CTA (TMEM lanes)
constexpr int kWStageBytes = kCtaRows * kBlockBytes;
constexpr int kGroup = 64;                   // weights of one quant group of a superblock
constexpr int kStep = 2 * kGroup;            // K per step
constexpr int kBBoxRows = 32;                // rows per TMA box of x
constexpr int kMoeTmemCols = 512;
constexpr int kPlainChunk = 3;               // superblocks per accumulation in D, plain form
constexpr int kMaxWStages = 4, kMaxBStages = 8;
constexpr int kDecodeWarp0 = 4;

// The shapes of the kernel. Warps: 0 weight copies, 1 activation copies, 2 MMA, 3
// TMEM; 4-15 decode (three sets of a warp per lane quarter: a step's two groups
// take 626 cycles on 8 warps alone, 507 on 12, 499 on 16); 16-23 epilogue (two
// per lane quarter).
// * Wide (large groups): blocks of 256 slots (plain: 192), so that a step's MMAs
//   (4 cycles per slot) cover the decoding of its weights and the issue of the
//   MMAs. One accumulator, taken into registers by the epilogue, 64 columns per
//   thread at a time (SwiGLU), or added to the registers' sums (plain).
// * Narrow (groups of about a hundred or fewer): blocks of 128 slots, two
//   accumulators; the decoding sets the pace.
// All keep four steps of decoded weights in TMEM: with two, the chain
// MMAs done -> store -> MMAs issued (about 1500 cycles) set the pace (2048
// tokens, 14336 x 4096: 1080 cycles per step of 704).
// Registers move from the copy and decode warps to the epilogue: 768 x 80 = 128 x
// 48 + 384 x 64 + 256 x 120 (plain, wide) >= 128 x 48 + 384 x 72 + 256 x 104.
template <bool SWIGLU, bool WIDE>
struct MoeShape {
    static constexpr int slots = !WIDE ? 128 : SWIGLU ? 256 : 192;   // most slots per tile: MMA N
    static constexpr int d_bufs = WIDE ? 1 : 2;
    static constexpr int a_col0 = slots * d_bufs;            // TMEM: D, then A
    static constexpr int a_steps = 4;                        // decoded steps
    static constexpr int sets = 3;
    static constexpr int epi_warp0 = kDecodeWarp0 + 4 * sets;
    static constexpr int threads = 32 * (epi_warp0 + 8);
    static constexpr int regs_launch = 80, regs_copy = 48, regs_decode = WIDE && !SWIGLU ? 64 : 72,
                         regs_epi = WIDE && !SWIGLU ? 120 : 104;
    static constexpr int b_stages = WIDE ? 4 : 8, w_stages = 4;   // powers of two: the decode warps index by masks
    static constexpr int b_half = slots / 2 * kGroup * 2;    // 64 elements of the CTA's rows of B
    static constexpr int b_stage = 2 * b_half;
    static constexpr int smem = 1024 + b_stages * b_stage + w_stages * kWStageBytes;
    static_assert(threads * regs_launch <= 65536 &&
                      128 * regs_copy + 128 * sets * regs_decode + 256 * regs_epi <= threads * regs_launch,
                  "register split");
    static_assert(a_col0 + a_steps * kStep / 2 <= kMoeTmemCols, "TMEM");
    static_assert(b_stages >= a_steps, "a step's barrier is reused behind its A buffers");
    static_assert(smem <= 227 * 1024 - 4096, "shared memory");
};
// At most this many pairs per expert on average: narrow. Measured, narrow against wide, us, for 64 / 96 / 128 / 192 /
// 256 / 384 pairs per expert (a router that prefers some experts; the groups differ by a factor of about four):
//   gate/up, 64 experts 1536 x 2048:  108/116, 132/133, 157/153, 207/195, 261/238, 367/328
//   gate/up, 8 experts 14336 x 4096:  214/222, 264/260, 328/287, 425/371, 536/459, 741/617
//   plain, 64 experts 2048 x 1536:    61/76, 71/86, 84/99, 110/118, 139/147, 191/199
//   plain, 8 experts 4096 x 14336:    117/125, 140/152, 168/166, 222/219, 281/285, 395/380
// In the plain form the narrow shape fills its second accumulator while the first is drained, which the wide one waits
// for; beyond 128 pairs, where wide has one block and narrow two, it depends on the tiles' number (6 experts 2048 x 4096,
// 160 pairs: 36/29; 4 experts 3900 x 9984: 75/97). The average decides: an expert far above it runs in blocks of 128.
constexpr int kNarrowPairsGated = 96, kNarrowPairsPlain = 128;

struct MoeShared {
    uint64_t w_full[kMaxWStages], w_empty[kMaxWStages];
    uint64_t full[kMaxBStages];                     // the first CTA's: both CTAs' A and B of the step are there
    uint64_t done[kMaxBStages];                     // the step's MMAs are complete: B stage and A buffers free
    uint64_t d_full[2], d_empty[2];                 // d_empty: the first CTA's
    uint64_t mma_done;
    uint32_t tmem;
    int abort;
    int warp_tiles[8];
    int tile0[Q4K_MOE_MAX_EXPERTS + 1];             // first tile of each expert
    int first[Q4K_MOE_MAX_EXPERTS], count[Q4K_MOE_MAX_EXPERTS];   // its slots
};

struct MoeGemmParams {
    MoeGroups g;
    void* y;
    int n, nsb, row_tiles;
};

// A completed barrier passes in about 90 cycles (mbar_wait_bounded's loop: 160).
__device__ __forceinline__ bool moe_wait(uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait_now(bar, parity)) return true;
    return mbar_wait_bounded(bar, parity, &g_moe_gemm_fault_flags);
}

// A walk over the pair's tiles, blocks of at most SLOTS slots.
template <int SLOTS>
struct TileWalk {
    int tile, e;            // current tile and its expert
    int slot0, slots, cols; // its slots, and their number rounded up to 16 (N)
    int row_tile;

    __device__ __forceinline__ void start() {
        tile = static_cast<int>(blockIdx.x >> 1);
        e = 0;
    }
    // Fills in the current tile; false past the last.
    __device__ __forceinline__ bool open(const MoeShared& sh, int experts) {
        if (tile >= sh.tile0[experts]) return false;
        while (tile >= sh.tile0[e + 1]) ++e;
        const int cnt = sh.count[e];
        const int blocks = (cnt + SLOTS - 1) / SLOTS;
        const int local = tile - sh.tile0[e];
        row_tile = local / blocks;
        const int b = local - row_tile * blocks;
        const int s0 = static_cast<int>(static_cast<long long>(cnt) * b / blocks);
        const int s1 = static_cast<int>(static_cast<long long>(cnt) * (b + 1) / blocks);
        slot0 = sh.first[e] + s0;
        slots = s1 - s0;
        cols = (slots + 15) & ~15;
        return true;
    }
    __device__ __forceinline__ void next() { tile += static_cast<int>(gridDim.x >> 1); }
};

// silu(g) * u for a result that is rounded to fp16 (silu_mul, q4k_swiglu.cuh, is
// the f32 form): __expf is off by at most 2 + 1.173 |g| ulp and __fdividef by 2,
// together under 2^-16 relative for |g| <= 88 against fp16's half step of 2^-11;
// below -88 the exponential overflows and the quotient is 0.
__device__ __forceinline__ float silu_mul_fast(float g, float u) {
    return __fdividef(g, 1.0f + __expf(-g)) * u;
}

__device__ __forceinline__ uint32_t pack_half2(float2 v) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 widen_half2(uint32_t bits) {
    return __half22float2(*reinterpret_cast<const __half2*>(&bits));
}

// One quant group of a row on its way to fp16: 64 quants, and for its two
// sub-blocks (low nibbles, high nibbles) the factor and the negated minimum.
struct QuantGroup {
    uint4 q0, q1;
    float s0, c0, s1, c1;   // 2^24 d sc_2g, -dmin m_2g, 2^20 d sc_2g+1, -dmin m_2g+1
};

// Half a superblock header, for the two groups of a step: the six-bit fields of
// a word become f32 as binary16 subnormals (times 2^-24), so the powers of two go
// to d, dmin.
struct StepHeader {
    uint32_t sc, mn;        // four sub-blocks' fields, a byte each
    float d48, d44, m24;    // 2^48 d, 2^44 d, -2^24 dmin (exact)

    __device__ __forceinline__ void load(const uint8_t* block, bool second) {
        const uint4 h = *reinterpret_cast<const uint4*>(block);
        const float2 d = widen_half2(h.x);
        if (second) {
            sc = (h.w & 0x0F0F0F0Fu) | (h.y >> 2 & 0x30303030u);
            mn = (h.w >> 4 & 0x0F0F0F0Fu) | (h.z >> 2 & 0x30303030u);
        } else {
            sc = h.y & 0x3F3F3F3Fu;
            mn = h.z & 0x3F3F3F3Fu;
        }
        d48 = d.x * 281474976710656.f;
        d44 = d.x * 17592186044416.f;
        m24 = d.y * -16777216.f;
    }
    __device__ __forceinline__ QuantGroup group(const uint8_t* quants, bool second) const {
        QuantGroup r;
        r.q0 = *reinterpret_cast<const uint4*>(quants);
        r.q1 = *reinterpret_cast<const uint4*>(quants + 16);
        const uint32_t pick = second ? 0x4342u : 0x4140u;   // two bytes, widened to 16 bits
        const float2 s = widen_half2(__byte_perm(sc, 0u, pick)), m = widen_half2(__byte_perm(mn, 0u, pick));
        r.s0 = d48 * s.x;
        r.s1 = d44 * s.y;
        r.c0 = m24 * m.x;
        r.c1 = m24 * m.y;
        return r;
    }
};

// The group's 64 weights as 32 fp16 pairs in K order. A masked quant word is a
// pair of subnormal binary16 values, q * 2^-24 (low nibbles) or q * 2^-20 (high
// nibbles), which widen to f32 exactly; one fma gives the weight dsc*q - dm
// rounded once, and cvt its binary16.
__device__ __forceinline__ void decode_group(const QuantGroup& in, uint32_t (&out)[32]) {
    const float2 s0 = make_float2(in.s0, in.s0), c0 = make_float2(in.c0, in.c0);
    const float2 s1 = make_float2(in.s1, in.s1), c1 = make_float2(in.c1, in.c1);
    const uint32_t w[8] = {in.q0.x, in.q0.y, in.q0.z, in.q0.w, in.q1.x, in.q1.y, in.q1.z, in.q1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = w[i] >> 8;
        const float2 a = widen_half2(w[i] & 0x000F000Fu), b = widen_half2(u & 0x000F000Fu);   // bytes 0 2, 1 3
        const float2 c = widen_half2(w[i] & 0x00F000F0u), d = widen_half2(u & 0x00F000F0u);
        const float2 l0 = ffma2(make_float2(a.x, b.x), s0, c0), l1 = ffma2(make_float2(a.y, b.y), s0, c0);
        const float2 h0 = ffma2(make_float2(c.x, d.x), s1, c1), h1 = ffma2(make_float2(c.y, d.y), s1, c1);
        out[2 * i] = pack_half2(l0);
        out[2 * i + 1] = pack_half2(l1);
        out[16 + 2 * i] = pack_half2(h0);
        out[16 + 2 * i + 1] = pack_half2(h1);
    }
}

template <bool SWIGLU, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(MoeShape<SWIGLU, WIDE>::threads, 1)
q4k_moe_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_w2,
                    const __grid_constant__ CUtensorMap map_x, const MoeGemmParams p) {
    using S = MoeShape<SWIGLU, WIDE>;
    constexpr int kBStages = S::b_stages, kWStages = S::w_stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sb = smem;                                  // [stages][2][slots / 2][64] fp16, swizzled
    uint8_t* sw = smem + kBStages * S::b_stage;          // [stages][128][144]
    __shared__ MoeShared sh;
    volatile int* abort_flag = &sh.abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int experts = p.g.experts, nsb = p.nsb;

    if (threadIdx.x == 0) {
        sh.abort = 0;
        for (int i = 0; i < kWStages; ++i) {
            mbar_init(&sh.w_full[i], 1);
            mbar_init(&sh.w_empty[i], 8);                // its two steps' decode warps
        }
        for (int i = 0; i < kBStages; ++i) {
            mbar_init(&sh.full[i], 9);                   // B's bytes; the step's decode warps in both CTAs
            mbar_init(&sh.done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.d_full[i], 1);
            mbar_init(&sh.d_empty[i], 16);               // epilogue warps of both CTAs
        }
        mbar_init(&sh.mma_done, 1);
        fence_mbar_init();
        tma_prefetch_map(&map_w);
        if (SWIGLU) tma_prefetch_map(&map_w2);
        tma_prefetch_map(&map_x);
    }
    if (warp == 3) tmem_alloc_pair(&sh.tmem, kMoeTmemCols);
    pdl_launch_dependents();
    pdl_wait();
    // Experts' slots and first tiles (a block-wide scan over up to 256 experts).
    {
        int tiles = 0;
        const int e = threadIdx.x;
        if (e < experts) {
            const int a = p.g.offsets[e], b = p.g.offsets[e + 1];
            const bool ok = a >= 0 && a <= b && b <= p.g.pairs;
            if (!ok && blockIdx.x == 0) atomicOr(&g_moe_gemm_fault_flags, Q4K_FAULT_ROUTE_RANGE);
            const int cnt = ok ? b - a : 0;
            sh.first[e] = a;
            sh.count[e] = cnt;
            tiles = (cnt + S::slots - 1) / S::slots * p.row_tiles;
        }
        int scan = tiles;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, scan, off);
            if (lane >= off) scan += v;
        }
        if (warp < 8 && lane == 31) sh.warp_tiles[warp] = scan;
        __syncthreads();
        if (e < experts) {
            int before = 0;
            for (int w = 0; w < warp; ++w) before += sh.warp_tiles[w];
            sh.tile0[e + 1] = before + scan;
            if (e == 0) sh.tile0[0] = 0;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem;

    if (warp < 4) {
        regs_lower<S::regs_copy>();
        if (warp == 0) {
            // ------------------------------------------------ weight copies
            if (lane == 0) {
                int it = 0;
                TileWalk<S::slots> t;
                for (t.start(); !*abort_flag && t.open(sh, experts); t.next()) {
                    const int per = SWIGLU ? 64 : kCtaRows;
                    const int row = t.e * p.n + (t.row_tile * 2 + static_cast<int>(rank)) * per;
                    for (int b = 0; b < nsb && !*abort_flag; ++b, ++it) {
                        const int s = it % kWStages;
                        if (it >= kWStages && !moe_wait(&sh.w_empty[s], static_cast<uint32_t>((it / kWStages - 1) & 1))) {
                            *abort_flag = 1;
                            break;
                        }
                        uint8_t* dst = sw + s * kWStageBytes;
                        mbar_arrive_expect_tx(&sh.w_full[s], kWStageBytes);
                        tma_load_3d(dst, &map_w, 0, b, row, &sh.w_full[s]);
                        if (SWIGLU) tma_load_3d(dst + kWStageBytes / 2, &map_w2, 0, b, row, &sh.w_full[s]);
                    }
                }
                if (*abort_flag)   // copies in flight land before shared memory goes
                    for (int i = it > kWStages ? it - kWStages : 0; i < it; ++i)
                        moe_wait(&sh.w_full[i % kWStages], static_cast<uint32_t>((i / kWStages) & 1));
            }
        } else if (warp == 2) {
            // ------------------------------------------------ MMA
            // The warp runs converged and one elected lane issues, so that the
            // operands stay in uniform registers. All 512 TMEM columns are the
            // pair's: its base address is 0.
            if (rank == 0) {
                const int chunk = SWIGLU ? nsb : kPlainChunk;   // superblocks per accumulation
                int s = 0, abuf = 0, chunk_no = 0;   // B stage, A buffer; accumulations so far
                uint32_t par = 0;
                bool ok = tmem == 0u;
                const uint64_t desc0 = sw128_kmajor_desc(smem_addr(sb));
                TileWalk<S::slots> t;
                for (t.start(); ok && t.open(sh, experts); t.next()) {
                    const uint32_t idesc = mma_f16_idesc(256, t.cols);
                    for (int b = 0; ok && b < nsb; b += chunk, ++chunk_no) {
                        const int dbuf = chunk_no % S::d_bufs;
                        if (chunk_no >= S::d_bufs)
                            ok = moe_wait(&sh.d_empty[dbuf], static_cast<uint32_t>((chunk_no / S::d_bufs - 1) & 1));
                        const uint32_t dcol = static_cast<uint32_t>(dbuf * S::slots);
                        const int steps = 2 * min(chunk, nsb - b);
#pragma unroll 1
                        for (int i = 0; i < steps; ++i) {
                            ok = __all_sync(0xFFFFFFFFu, ok && moe_wait(&sh.full[s], par));
                            if (!ok) break;
                            tc_fence_after_sync();
                            if (elect_one()) {
                                const uint64_t bd = desc0 + static_cast<uint64_t>(s * (S::b_stage >> 4));
                                const uint32_t acol = S::a_col0 + abuf * (kStep / 2);
#pragma unroll
                                for (int kk = 0; kk < kStep / 16; ++kk)
                                    mma_f16_tmem_a_pair(dcol, acol + 8 * kk,
                                                        bd + static_cast<uint64_t>((kk >> 2) * (S::b_half >> 4) + 2 * (kk & 3)),
                                                        idesc, i == 0 && kk == 0 ? 0u : 1u);
                                mma_commit_pair(&sh.done[s]);
                                if (i + 1 == steps) mma_commit_pair(&sh.d_full[dbuf]);
                            }
                            __syncwarp();
                            if (++s == kBStages) {
                                s = 0;
                                par ^= 1u;
                            }
                            if (++abuf == S::a_steps) abuf = 0;
                        }
                    }
                }
                if (!ok) *abort_flag = 1;
                if (elect_one()) {
                    mma_commit_pair_local(&sh.mma_done);
                    moe_wait(&sh.mma_done, 0u);
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------ activation copies
            int s = 0, it = 0;
            uint32_t par = 1;
            bool ok = true;
            TileWalk<S::slots> t;
            const uint32_t bar0 = map_to_rank(&sh.full[0], 0);
            for (t.start(); ok && !*abort_flag && t.open(sh, experts); t.next()) {
                const int half = t.cols / 2;
                const int boxes = (half + kBBoxRows - 1) / kBBoxRows;
                const int row = t.slot0 + static_cast<int>(rank) * half;
                for (int i = 0; i < 2 * nsb; ++i, ++it) {
                    if (it >= kBStages) {
                        ok = __all_sync(0xFFFFFFFFu, moe_wait(&sh.done[s], par));
                        if (!ok) break;
                    }
                    if (elect_one()) {
                        if (rank == 0)   // both CTAs' bytes
                            mbar_arrive_expect_tx(&sh.full[s], 2u * 2u * boxes * kBBoxRows * kGroup * 2);
                        uint8_t* dst = sb + s * S::b_stage;
                        for (int j = 0; j < boxes; ++j) {
                            tma_load_2d_pair(dst + j * kBBoxRows * kGroup * 2, &map_x, i * kStep, row + j * kBBoxRows,
                                             bar0 + 8 * s);
                            tma_load_2d_pair(dst + S::b_half + j * kBBoxRows * kGroup * 2, &map_x, i * kStep + kGroup,
                                             row + j * kBBoxRows, bar0 + 8 * s);
                        }
                    }
                    __syncwarp();
                    if (++s == kBStages) {
                        s = 0;
                        par ^= 1u;
                    }
                }
            }
            if (!ok) *abort_flag = 1;
            if (*abort_flag) {   // copies in flight land before shared memory goes: their bytes are
                                 // counted on barriers that may now miss arrivals, so wait them out
                for (int i = 0; i < 64; ++i) __nanosleep(1000000);
            }
        }
    } else if (warp < S::epi_warp0) {
        // ---------------------------------------------------- decode
        // The pair's steps in the order of its tiles are numbered through: step i,
        // two quant groups of a superblock, is decoded by set i % sets into TMEM
        // buffer i % a_steps. (A set per group instead: three headers in four groups
        // and twice the barriers; 777 tokens 109 us.)
        regs_lower<S::regs_decode>();
        const int quarter = warp & 3;
        const int row = SWIGLU ? (lane < 16 ? 0 : 64) + 16 * quarter + (lane & 15) : 32 * quarter + lane;
        const uint32_t lane_addr = tmem + S::a_col0 + (static_cast<uint32_t>(32 * quarter) << 16);
        const uint32_t full0 = map_to_rank(&sh.full[0], 0);
        const int pairs = static_cast<int>(gridDim.x >> 1), pair = static_cast<int>(blockIdx.x >> 1);
        const int tiles = sh.tile0[experts] > pair ? (sh.tile0[experts] - pair - 1) / pairs + 1 : 0;
        const uint32_t steps = 2u * static_cast<uint32_t>(tiles) * static_cast<uint32_t>(nsb);
        StepHeader hd;
        bool ok = true;
        const uint8_t* quants;
        auto fetch = [&](uint32_t i) {       // step i's header, its first group's quants and factors
            const uint32_t b = i >> 1, ws = b % kWStages;
            const uint8_t* block = sw + ws * kWStageBytes + row * kBlockBytes;
            ok = __all_sync(0xFFFFFFFFu, moe_wait(&sh.w_full[ws], (b / kWStages) & 1u));
            if (!ok) return QuantGroup{};
            hd.load(block, (i & 1u) != 0u);
            quants = block + kQsOffset + ((i & 1u) != 0u ? 64 : 0);
            return hd.group(quants, false);
        };
        uint32_t i = (warp - kDecodeWarp0) >> 2;
        QuantGroup q{};
        if (i < steps) q = fetch(i);
#pragma unroll 1
        for (; ok && i < steps; i += S::sets) {
            // the buffer's last step: its barrier is polled ahead of the decoding, which covers the poll's latency
            const uint32_t last = i - S::a_steps;
            uint64_t* free_bar = &sh.done[last % kBStages];
            const uint32_t free_par = (last / kBStages) & 1u;
            const bool free = i < S::a_steps || mbar_try_wait_now(free_bar, free_par);
            const uint32_t addr = lane_addr + (i % S::a_steps) * (kStep / 2);
            uint32_t r[32];
            decode_group(q, r);
            q = hd.group(quants + 32, true);
            if (!__all_sync(0xFFFFFFFFu, free)) {
                ok = __all_sync(0xFFFFFFFFu, moe_wait(free_bar, free_par));
                if (!ok) break;
            }
            tc_fence_after_sync();
            tmem_store_32cols(addr, r);
            decode_group(q, r);
            tmem_store_32cols(addr + kGroup / 2, r);
            __syncwarp();                    // the superblock's quants are read
            if (lane == 0) mbar_arrive(&sh.w_empty[(i >> 1) % kWStages]);
            if (i + S::sets < steps) q = fetch(i + S::sets);
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(full0 + 8 * (i % kBStages));
        }
        if (!ok) *abort_flag = 1;
    } else {
        // ---------------------------------------------------- epilogue
        regs_raise<S::regs_epi>();
        const int quarter = warp & 3, part = (warp - S::epi_warp0) >> 2;
        constexpr int kPart = S::slots / 2;                // columns per warp
        const int c0 = part * kPart;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + c0;
        int chunk_no = 0;
        bool ok = true;
        TileWalk<S::slots> t;
        for (t.start(); ok && t.open(sh, experts); t.next()) {
            // the pairs of this warp's columns, a column per lane and 32-column piece; -1: not stored
            int pair[kPart / 32];
#pragma unroll
            for (int j = 0; j < kPart / 32; ++j) {
                const int c = c0 + 32 * j + lane;
                pair[j] = -1;
                if (c < t.slots) {
                    const int v = p.g.order[t.slot0 + c];
                    if (v >= 0 && v < p.g.pairs) pair[j] = v;
                    else if (t.row_tile == 0) atomicOr(&g_moe_gemm_fault_flags, Q4K_FAULT_ROUTE_RANGE);
                }
            }
            if constexpr (SWIGLU) {
                const int dbuf = chunk_no % S::d_bufs;
                ok = !*abort_flag && moe_wait(&sh.d_full[dbuf], static_cast<uint32_t>((chunk_no / S::d_bufs) & 1));
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) {
                    *abort_flag = 1;
                    break;
                }
                ++chunk_no;
                tc_fence_after_sync();
                const int feature = (t.row_tile * 2 + static_cast<int>(rank)) * 64 + 16 * quarter + (lane & 15);
                const bool gate = lane < 16;
                // lanes with gate rows finish even columns, lanes with up rows odd ones
                __half* y = static_cast<__half*>(p.y) + static_cast<size_t>(t.slot0 + c0 + (gate ? 0 : 1)) * p.n + feature;
#pragma unroll
                for (int pass = 0; pass < kPart / 64; ++pass) {
                    uint32_t acc[2][32];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (c0 + 64 * pass + 32 * j < t.cols)
                            tmem_load_32cols_async(lane_addr + dbuf * S::slots + 64 * pass + 32 * j, acc[j]);
                    tmem_wait_ld();
                    if (pass + 1 == kPart / 64) {       // D is in registers: the MMAs may go on
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(map_to_rank(&sh.d_empty[dbuf], 0));
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t stored = __ballot_sync(0xFFFFFFFFu, pair[2 * pass + j] >= 0);
                        const uint32_t mine = feature < p.n ? stored >> (gate ? 0 : 1) : 0u;
                        if (stored == 0u) continue;
#pragma unroll
                        for (int c8 = 0; c8 < 32; c8 += 8) {
                            if ((stored >> c8 & 0xFFu) == 0u) continue;   // eight columns without a pair
#pragma unroll
                            for (int c = c8; c < c8 + 8; c += 2) {
                                const float a = __uint_as_float(acc[j][c]), d = __uint_as_float(acc[j][c + 1]);
                                const float other = __shfl_xor_sync(0xFFFFFFFFu, gate ? d : a, 16);
                                if (mine & (1u << c))
                                    y[static_cast<size_t>(64 * pass + 32 * j + c) * p.n] =
                                        __float2half_rn(silu_mul_fast(gate ? a : other, gate ? other : d));
                            }
                        }
                    }
                }
            } else {
                float acc[kPart];
#pragma unroll
                for (int c = 0; c < kPart; ++c) acc[c] = 0.f;
                for (int b = 0; b < nsb; b += kPlainChunk) {
                    const int dbuf = chunk_no % S::d_bufs;
                    ok = !*abort_flag && moe_wait(&sh.d_full[dbuf], static_cast<uint32_t>((chunk_no / S::d_bufs) & 1));
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    ++chunk_no;
                    tc_fence_after_sync();
#pragma unroll
                    for (int j = 0; j < kPart / 16; ++j) {
                        if (c0 + 16 * j < t.cols) {
                            uint32_t r[16];
                            tmem_load_16cols(lane_addr + dbuf * S::slots + 16 * j, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 16; ++c) acc[16 * j + c] += __uint_as_float(r[c]);
                        }
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(map_to_rank(&sh.d_empty[dbuf], 0));
                }
                if (!ok) {
                    *abort_flag = 1;
                    break;
                }
                const int row = (t.row_tile * 2 + static_cast<int>(rank)) * kCtaRows + 32 * quarter + lane;
                float* y = static_cast<float*>(p.y) + row;
#pragma unroll
                for (int j = 0; j < kPart / 32; ++j) {
                    if (__ballot_sync(0xFFFFFFFFu, pair[j] >= 0) == 0u) continue;
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const int pr = __shfl_sync(0xFFFFFFFFu, pair[j], c);
                        if (pr >= 0 && row < p.n) y[static_cast<size_t>(pr) * p.n] = acc[32 * j + c];
                    }
                }
            }
        }
    }

    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();   // no arrival or MMA on either CTA's memory is left
    if (warp == 3) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, kMoeTmemCols);
    }
}

// out[s] = x[order[s] / per_row] for every slot whose entry is a pair: a warp per
// row, four 16-byte loads per lane in flight. All entries are looked at, not those
// below offsets[experts]: where some expert's offsets are bad, another's slots may
// lie behind that. A slot without a pair is not copied (the product does not store
// it, and a column of B reaches no other column of D).
constexpr int kGatherThreads = 256;

__global__ void __launch_bounds__(kGatherThreads)
q4k_moe_gather_kernel(const uint4* x, uint4* __restrict__ out, const MoeGroups g, int row16) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int warps = static_cast<int>(gridDim.x) * (kGatherThreads / 32);
    for (int s = static_cast<int>(blockIdx.x) * (kGatherThreads / 32) + static_cast<int>(threadIdx.x >> 5); s < g.pairs;
         s += warps) {
        const int pair = g.order[s];
        if (pair < 0 || pair >= g.pairs) continue;
        const uint4* src = x + static_cast<size_t>(pair / g.per_row) * row16;
        uint4* dst = out + static_cast<size_t>(s) * row16;
        for (int c0 = lane; c0 < row16; c0 += 128) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c0 + 32 * i < row16) v[i] = src[c0 + 32 * i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c0 + 32 * i < row16) dst[c0 + 32 * i] = v[i];
        }
    }
}

// (byte of a superblock, superblock, row) of all experts' rows, boxes of one
// superblock by box_rows rows.
bool make_moe_weight_map(CUtensorMap* map, const void* w, long long rows, int nsb, int box_rows) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kBlockBytes), static_cast<cuuint64_t>(nsb),
                                static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kBlockBytes), static_cast<cuuint64_t>(nsb) * kBlockBytes};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(kBlockBytes), 1u, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(w), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row-major fp16 [rows][k], boxes of 64 elements by box_rows rows, 128-byte
// swizzle.
bool make_moe_x_map(CUtensorMap* map, const void* x, int rows, int k, int box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(k) * 2};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kGroup), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(x), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The current device's pool for the copies of x: it keeps up to kPoolKeepBytes
// between calls (the default pool gives all back whenever the device is
// synchronised, and the next allocation then takes 0.5-1.6 ms). Allocations and
// frees are stream-ordered and captured into graphs as their own nodes, so no
// two calls that may overlap share a copy.
constexpr uint64_t kPoolKeepBytes = 512ull << 20;

cudaError_t workspace_pool(cudaMemPool_t* pool) {
    static PerDevice<cudaMemPool_t> pools;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return pools.get(dev, pool, [dev](cudaMemPool_t* made) {
        // the first call may be inside a capture, which a pool's creation would end in the default mode
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        cudaError_t status = cudaThreadExchangeStreamCaptureMode(&mode);
        if (status != cudaSuccess) return status;
        cudaMemPoolProps props = {};
        props.allocType = cudaMemAllocationTypePinned;
        props.location.type = cudaMemLocationTypeDevice;
        props.location.id = dev;
        status = cudaMemPoolCreate(made, &props);
        if (status == cudaSuccess) {
            uint64_t keep = kPoolKeepBytes;
            status = cudaMemPoolSetAttribute(*made, cudaMemPoolAttrReleaseThreshold, &keep);
            if (status != cudaSuccess) cudaMemPoolDestroy(*made);
        }
        const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
        if (status == cudaSuccess && back != cudaSuccess) {
            cudaMemPoolDestroy(*made);
            status = back;
        }
        return status;
    });
}

// The kernels' attributes, set by the device's first call (not with the library's
// other kernels, so that programs without experts load none of this).
cudaError_t gemm_ready() {
    static PerDevice<bool> ready;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    bool set;
    return ready.get(dev, &set, [](bool* made) {
        constexpr cudaFuncAttribute smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
        cudaError_t status = cudaFuncSetAttribute(q4k_moe_gemm_kernel<true, true>, smem, MoeShape<true, true>::smem);
        if (status == cudaSuccess)
            status = cudaFuncSetAttribute(q4k_moe_gemm_kernel<true, false>, smem, MoeShape<true, false>::smem);
        if (status == cudaSuccess)
            status = cudaFuncSetAttribute(q4k_moe_gemm_kernel<false, true>, smem, MoeShape<false, true>::smem);
        if (status == cudaSuccess)
            status = cudaFuncSetAttribute(q4k_moe_gemm_kernel<false, false>, smem, MoeShape<false, false>::smem);
        *made = true;
        return status;
    });
}

}  // namespace

int launch_moe_gemm(const DeviceInfo& dev, const void* w, const void* w2, const void* x_f16, const MoeGroups& g, void* y,
                    int n, int k, cudaStream_t stream) {
    const bool swiglu = w2 != nullptr;
    const int nsb = k / kQK;
    const long long rows = static_cast<long long>(g.experts) * n;
    if (encode_tiled() == nullptr) return cuda_failure(cudaErrorInvalidValue);
    cudaError_t e = gemm_ready();
    if (e != cudaSuccess) return cuda_failure(e);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;

    const void* xs = x_f16;      // rows in slot order
    void* work = nullptr;
    if (g.per_row > 0) {
        cudaMemPool_t pool = nullptr;
        e = workspace_pool(&pool);
        if (e == cudaSuccess)
            e = cudaMallocFromPoolAsync(&work, static_cast<size_t>(g.pairs) * static_cast<size_t>(k) * 2, pool, stream);
        if (e != cudaSuccess) return cuda_failure(e);
        const int per_cta = kGatherThreads / 32;
        const long long blocks = (static_cast<long long>(g.pairs) + per_cta - 1) / per_cta;
        cfg.gridDim = dim3(static_cast<unsigned>(blocks < dev.sm_count * 8 ? blocks : dev.sm_count * 8));
        cfg.blockDim = dim3(kGatherThreads);
        e = cudaLaunchKernelEx(&cfg, q4k_moe_gather_kernel, static_cast<const uint4*>(x_f16), static_cast<uint4*>(work), g,
                               k / 8);
        xs = work;
    }
    CUtensorMap mw, mw2, mx;
    if (e == cudaSuccess &&
        (!make_moe_weight_map(&mw, w, rows, nsb, swiglu ? 64 : kCtaRows) ||
         !make_moe_weight_map(&mw2, swiglu ? w2 : w, rows, nsb, 64) || !make_moe_x_map(&mx, xs, g.pairs, k, kBBoxRows)))
        e = cudaErrorInvalidValue;
    if (e == cudaSuccess) {
        MoeGemmParams p{};
        p.g = g;
        p.y = y;
        p.n = n;
        p.nsb = nsb;
        const int tile_rows = swiglu ? kCtaRows : 2 * kCtaRows;
        p.row_tiles = (n + tile_rows - 1) / tile_rows;
        const bool wide = g.pairs > static_cast<long long>(swiglu ? kNarrowPairsGated : kNarrowPairsPlain) * g.experts;
        cfg.gridDim = dim3(static_cast<unsigned>(dev.sm_count / 2 * 2));
        cfg.blockDim = dim3(MoeShape<true, true>::threads);
        cfg.dynamicSmemBytes = swiglu ? (wide ? MoeShape<true, true>::smem : MoeShape<true, false>::smem)
                                      : (wide ? MoeShape<false, true>::smem : MoeShape<false, false>::smem);
        auto* kernel = swiglu ? (wide ? q4k_moe_gemm_kernel<true, true> : q4k_moe_gemm_kernel<true, false>)
                              : (wide ? q4k_moe_gemm_kernel<false, true> : q4k_moe_gemm_kernel<false, false>);
        e = cudaLaunchKernelEx(&cfg, kernel, mw, mw2, mx, p);
    }
    if (work != nullptr) {
        const cudaError_t f = cudaFreeAsync(work, stream);
        if (e == cudaSuccess) e = f;
    }
    return e == cudaSuccess ? Q4K_OK : cuda_failure(e);
}

int read_moe_gemm_fault_flags(unsigned* flags) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_moe_gemm_fault_flags, sizeof(v));
    if (e != cudaSuccess) return cuda_failure(e);
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(g_moe_gemm_fault_flags, &zero, sizeof(zero));
    if (e != cudaSuccess) return cuda_failure(e);
    *flags = v;
    return Q4K_OK;
}

}  // namespace q4k
