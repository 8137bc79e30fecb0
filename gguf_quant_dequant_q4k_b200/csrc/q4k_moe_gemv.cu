// q4k_moe_gemv.cu -- expert-grouped products of a few f32 vectors per expert
// with Q4_K matrices (q4k_moe_gemv, q4k_moe_gemv_swiglu): every pair (slot) of a
// decode batch with its own expert's matrix, each matrix row read once per
// group of up to four vectors.
//
// * Arithmetic (that of the integer GEMV for several vectors). Per 256-element
//   block b of a vector X = round(x * 2^(30 - E_b)), E_b the exponent of the
//   block's largest |x|, in four balanced base-256 digits X = sum_l 256^l X_l.
//   For every sub-block j the tensor cores form D_j[row][l] = sum q * X_l from
//   the raw quants (unsigned bytes w & 0x0F0F0F0F; the high nibbles as 16 q),
//   exact in 32 bits. P_l = sum_j sc_j D_j[l] and, with S0_j = sum of X over the
//   sub-block, M = sum_j m_j S0_j are exact integers too, and the row's f64
//   total gets 2^(E_b - 30) * (d * sum_l 256^l P_l - dmin * M); y is that total
//   rounded once.
// * Tensor cores. mma.sync m16n8k32 (u8 x s8 -> s32): one MMA is 16 rows x one
//   sub-block x the digits of two vectors. It issues 0.49 per cycle and SM
//   (measured) against 0.16 that the HBM rate needs for two vectors; unlike
//   tcgen05 it takes the quants from registers and returns the sums there,
//   which keeps a call's start and end short where a CTA has only a few tiles.
// * Weights. A warp streams boxes of 16 rows x 2 superblocks (4608 bytes, TMA)
//   through its own shared-memory stages; lane 4 g + t holds rows g, g + 8 and
//   the bytes 8 t .. 8 t + 7 of each 32-byte quant group (a permutation of K
//   inside the sub-block that the digit image repeats). Rows 288 bytes apart
//   make those 8-byte loads free of bank conflicts.
// * Work. A unit is 16 rows x one group of vectors; clusters of CTAs own equal
//   contiguous ranges of units, the CTAs of a cluster equal parts of K (one CTA
//   where the digit image of the whole row fits), the warps of a CTA equal
//   ranges of the (unit, box) items of a round. With one CTA per cluster a
//   round is all its units of a group: a warp stores the units it has whole, and
//   the units cut between warps (at most one per warp) meet in shared memory.
//   With several, a round is up to kRoundUnits units and all pieces meet in the
//   cluster's shared memory. Pieces are added in a fixed order.
// * Bound: HBM for one and two vectors; the issue slots for four.
#include <cstdint>
#include <cuda.h>
#include <mutex>
#include <type_traits>

#include "q4k_internal.h"
#include "q4k_moe.h"
#include "q4k_pair.cuh"
#include "q4k_superblock.cuh"
#include "q4k_swiglu.cuh"

namespace q4k {

__device__ unsigned int g_moe_gemv_fault_flags = 0;

namespace {

constexpr int kVWarps = 16;
constexpr int kVThreads = 32 * kVWarps;
constexpr int kVStages = 2;                       // boxes in flight per warp
constexpr int kVRows = 16;                        // rows per unit: the MMA's M
constexpr int kVBoxCols = 2;                      // superblocks per box
constexpr int kVRowPitch = kVBoxCols * kBlockBytes;
constexpr int kVBoxBytes = kVRows * kVRowPitch;
constexpr int kVMaxVec = 4;                       // vectors per group
constexpr int kRoundUnits = 16;                   // most units of a round in a cluster of several CTAs
// Pieces of units in shared memory. Several CTAs: every piece of a round,
// numbered unit + warp (unique: of two neighbouring pieces one or both grow).
// One CTA: a warp's first piece if it starts inside a unit (2 warp), its last if
// it ends inside one (2 warp + 1).
constexpr int kVPieces = 2 * kVWarps;
static_assert(kRoundUnits + kVWarps <= kVPieces, "pieces of a round");
constexpr int kVMaxCluster = 8;
// Digit image of one superblock and two vectors: [sub-block pair][lane][2][8
// bytes]; metadata per vector: 2^(E-30), from byte 16 l_0..7, from byte 48 h_0..7
// with S0_j = 2^18 h_j + l_j.
constexpr int kVImageBytes = 2048;
constexpr int kVMetaBytes = 80;
__host__ __device__ constexpr int v_meta_offset(int cap) { return cap / 2 * kVImageBytes; }
__host__ __device__ constexpr int v_sb_bytes(int cap) { return v_meta_offset(cap) + cap * kVMetaBytes; }
// [matrix][vector][row]
__host__ __device__ constexpr int v_piece_doubles(int cap, bool swiglu) { return kVRows * cap * (swiglu ? 2 : 1); }
// Shared memory of groups of up to `cap` vectors (4, or 2 for long K) and parts
// of `sbs` superblocks; the most superblocks that fit.
constexpr int v_smem(int sbs, int cap, bool swiglu) {
    return 128 + kVWarps * kVStages * kVBoxBytes + sbs * v_sb_bytes(cap) + kVPieces * v_piece_doubles(cap, swiglu) * 8;
}
constexpr int kVSmemLimit = 227 * 1024 - 4096;    // less the static part
constexpr int v_max_sbs(int cap, bool swiglu) { return (kVSmemLimit - v_smem(0, cap, swiglu)) / v_sb_bytes(cap); }
static_assert(v_max_sbs(2, true) * kVMaxCluster * kQK >= Q4K_MOE_GEMV_MAX_K, "every accepted K fits");

struct MoeGemvParams {
    MoeGroups g;
    const float* x;
    float* y;
    int n, k, nsb;
    int units;      // row tiles of one matrix
    int part_sbs;   // superblocks of a CTA's part of K (the last one's may be fewer)
    int cap;        // most vectors per group: 4 or 2
};

struct GemvShared {
    uint64_t full[kVWarps][kVStages];
    int warp_sum[kVWarps];
    int chunk0[Q4K_MOE_MAX_EXPERTS + 1];            // first vector group of each expert
    int first[Q4K_MOE_MAX_EXPERTS], count[Q4K_MOE_MAX_EXPERTS];
    int abort;
};

__device__ __forceinline__ void imma(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}

// A 32-bit integer as f64, exactly: 2^52 + 2^31 + v less 2^52 + 2^31.
__device__ __forceinline__ double int_to_f64(int v) {
    return __hiloint2double(0x43300000, v ^ static_cast<int>(0x80000000u)) - 4503601774854144.0;
}

// The digits of one vector's block: lane holds K positions 8 lane .. + 7.
__device__ __forceinline__ void block_digits(const float* __restrict__ x, int vec, uint8_t* sb_image, int meta_offset,
                                             int lane) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(x) + 2 * lane);
    const float4 c = __ldg(reinterpret_cast<const float4*>(x) + 2 * lane + 1);
    const float v[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
    bool finite = true;
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        finite = finite && isfinite(v[e]);
        amax = fmaxf(amax, fabsf(v[e]));
    }
    finite = __all_sync(0xFFFFFFFFu, finite);
    amax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax)));   // non-negative: ordered as integers
    const bool scaled = finite && amax > 0.f;
    int ex = 0;
    if (scaled) frexpf(amax, &ex);                       // amax in [2^(ex-1), 2^ex)
    const double up = scaled ? __longlong_as_double(static_cast<long long>(1023 + 30 - ex) << 52) : 0.0;
    int r[8];
    long long sum = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        r[e] = scaled ? __double2int_rn(static_cast<double>(v[e]) * up) : 0;
        sum += r[e];
    }
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);         // S0 of sub-block j: lanes 4j .. 4j + 3
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
    uint8_t* meta = sb_image + meta_offset + vec * kVMetaBytes;
    const int j = lane >> 2, t = lane & 3;
    if (t == 0) {
        reinterpret_cast<int*>(meta + 16)[j] = static_cast<int>(sum & 0x3FFFF);
        reinterpret_cast<int*>(meta + 48)[j] = static_cast<int>(sum >> 18);
    }
    if (lane == 0)
        *reinterpret_cast<double*>(meta) =
            finite ? (scaled ? __longlong_as_double(static_cast<long long>(1023 + ex - 30) << 52) : 0.0)
                   : __longlong_as_double(0x7FF8000000000000LL);
    uint8_t* img = sb_image + (vec >> 1) * kVImageBytes + (j >> 1) * 512 + (j & 1) * 8;
#pragma unroll
    for (int l = 0; l < 4; ++l) {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int dig = l < 3 ? ((r[e] + 128) & 255) - 128 : r[e];
            r[e] = (r[e] - dig) >> 8;
            w[e >> 2] |= (static_cast<uint32_t>(dig) & 0xFFu) << (8 * (e & 3));
        }
        const int col = 4 * (vec & 1) + l;
        *reinterpret_cast<uint2*>(img + (4 * col + t) * 16) = make_uint2(w[0], w[1]);
    }
}

// Adds one superblock of 16 rows to the lane's totals: acc[nt][0] for row g,
// acc[nt][1] for row g + 8, each the lane's two digit columns of vector 2 nt +
// t / 2 (digits 0, 1 for even t, 2, 3 for odd t) and its half of the M term.
template <int NT>
__device__ __forceinline__ void superblock_rows(const uint8_t* rows, const uint8_t* sb_image, int meta_offset, int lane,
                                                double (&acc)[NT][2]) {
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* ra = rows + g * kVRowPitch;
    const uint8_t* rb = ra + 8 * kVRowPitch;
    const Header ha = decode_header(*reinterpret_cast<const uint4*>(ra));
    const Header hb = decode_header(*reinterpret_cast<const uint4*>(rb));
    int pe[NT][4], po[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) pe[i][c] = po[i][c] = 0;
#pragma unroll
    for (int jp = 0; jp < 4; ++jp) {
        const uint2 qa = *reinterpret_cast<const uint2*>(ra + kQsOffset + 32 * jp + 8 * t);
        const uint2 qb = *reinterpret_cast<const uint2*>(rb + kQsOffset + 32 * jp + 8 * t);
        const uint32_t wa = jp < 2 ? ha.sc_lo : ha.sc_hi, wb = jp < 2 ? hb.sc_lo : hb.sc_hi;
        const int sae = static_cast<int>(byte_of(wa, (2 * jp) & 3)), sao = static_cast<int>(byte_of(wa, (2 * jp + 1) & 3));
        const int sbe = static_cast<int>(byte_of(wb, (2 * jp) & 3)), sbo = static_cast<int>(byte_of(wb, (2 * jp + 1) & 3));
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const uint4 dg = *reinterpret_cast<const uint4*>(sb_image + i * kVImageBytes + jp * 512 + lane * 16);
            int d[4];
            imma(d, qa.x & 0x0F0F0F0Fu, qb.x & 0x0F0F0F0Fu, qa.y & 0x0F0F0F0Fu, qb.y & 0x0F0F0F0Fu, dg.x, dg.y);
            pe[i][0] += sae * d[0];
            pe[i][1] += sae * d[1];
            pe[i][2] += sbe * d[2];
            pe[i][3] += sbe * d[3];
            imma(d, qa.x & 0xF0F0F0F0u, qb.x & 0xF0F0F0F0u, qa.y & 0xF0F0F0F0u, qb.y & 0xF0F0F0F0u, dg.z, dg.w);
            po[i][0] += sao * d[0];    // sixteen times the sums
            po[i][1] += sao * d[1];
            po[i][2] += sbo * d[2];
            po[i][3] += sbo * d[3];
        }
    }
    const bool low = (t & 1) == 0;
    const double fs = low ? 1.0 : 65536.0, fm = low ? -1.0 : -262144.0;
    const double da = ha.d * fs, db = hb.d * fs, ma = ha.dmin * fm, mb = hb.dmin * fm;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const uint8_t* meta = sb_image + meta_offset + (2 * i + (t >> 1)) * kVMetaBytes;
        const int4 x0 = *reinterpret_cast<const int4*>(meta + (low ? 16 : 48));
        const int4 x1 = *reinterpret_cast<const int4*>(meta + (low ? 16 : 48) + 16);
        const int xs[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        int sa = 0, sb = 0;            // |m l| sums < 8 * 63 * 2^18, |m h| sums < 8 * 63 * 2^17
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sa += static_cast<int>(byte_of(j < 4 ? ha.m_lo : ha.m_hi, j & 3)) * xs[j];
            sb += static_cast<int>(byte_of(j < 4 ? hb.m_lo : hb.m_hi, j & 3)) * xs[j];
        }
        const double scale = *reinterpret_cast<const double*>(meta);
        const double pa = fma(256.0, int_to_f64(pe[i][1] + (po[i][1] >> 4)), int_to_f64(pe[i][0] + (po[i][0] >> 4)));
        const double pb = fma(256.0, int_to_f64(pe[i][3] + (po[i][3] >> 4)), int_to_f64(pe[i][2] + (po[i][2] >> 4)));
        acc[i][0] = fma(scale, fma(da, pa, ma * int_to_f64(sa)), acc[i][0]);
        acc[i][1] = fma(scale, fma(db, pb, mb * int_to_f64(sb)), acc[i][1]);
    }
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kVThreads, 1)
q4k_moe_gemv_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_w2,
                    const MoeGemvParams p) {
    constexpr int R = SWIGLU ? 2 : 1;                      // matrices
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                               ~static_cast<uintptr_t>(127));
    uint8_t* ring = smem;
    uint8_t* image = ring + kVWarps * kVStages * kVBoxBytes;
    const int sb_bytes = v_sb_bytes(p.cap), meta_offset = v_meta_offset(p.cap);
    double* parts = reinterpret_cast<double*>(image + p.part_sbs * sb_bytes);
    __shared__ GemvShared sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t csize, rank, cid, nclusters;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(csize));
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(cid));
    asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(nclusters));
    rank = cluster_rank();
    const int experts = p.g.experts;
    const int sb0 = static_cast<int>(rank) * p.part_sbs;
    const int sbs = max(0, min(p.part_sbs, p.nsb - sb0));  // this CTA's superblocks
    const int boxes = (p.part_sbs + kVBoxCols - 1) / kVBoxCols;   // per unit and matrix, the same in every CTA

    if (lane == 0)
        for (int s = 0; s < kVStages; ++s) mbar_init(&sh.full[warp][s], 1);
    if (threadIdx.x == 0) {
        sh.abort = 0;
        tma_prefetch_map(&map_w);
        if (SWIGLU) tma_prefetch_map(&map_w2);
    }
    fence_mbar_init();
    pdl_launch_dependents();
    pdl_wait();
    // Experts' slots and first vector groups.
    {
        const int e = threadIdx.x;
        int chunks = 0;
        if (e < experts) {
            const int a = __ldg(p.g.offsets + e), b = __ldg(p.g.offsets + e + 1);
            const bool ok = a >= 0 && a <= b && b <= p.g.pairs;
            if (!ok && blockIdx.x == 0) atomicOr(&g_moe_gemv_fault_flags, Q4K_FAULT_ROUTE_RANGE);
            const int cnt = ok ? b - a : 0;
            sh.first[e] = a;
            sh.count[e] = cnt;
            chunks = (cnt + p.cap - 1) / p.cap;
        }
        int scan = chunks;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, scan, off);
            if (lane >= off) scan += v;
        }
        if (lane == 31) sh.warp_sum[warp] = scan;
        __syncthreads();
        if (e < experts) {
            int before = 0;
            for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
            sh.chunk0[e + 1] = before + scan;
            if (e == 0) sh.chunk0[0] = 0;
        }
        __syncthreads();
    }
    const long long total = static_cast<long long>(sh.chunk0[experts]) * p.units;
    const long long u0 = total * cid / nclusters, u1 = total * (cid + 1) / nclusters;

    // The rounds of this cluster: up to kRoundUnits units of one vector group.
    struct Round {
        long long u;         // first unit
        int count;           // units; 0 behind the last round
        int e, chunk, tile;  // expert, vector group, row tile of the first unit
    };
    auto open_round = [&](long long u, int e) {
        Round r{u, 0, e, 0, 0};
        if (u >= u1) return r;
        r.chunk = static_cast<int>(u / p.units);
        r.tile = static_cast<int>(u - static_cast<long long>(r.chunk) * p.units);
        while (r.chunk >= sh.chunk0[r.e + 1]) ++r.e;
        const long long left = min(u1 - u, static_cast<long long>(p.units - r.tile));
        r.count = static_cast<int>(csize > 1 ? min(left, static_cast<long long>(kRoundUnits)) : left);
        return r;
    };
    auto item_begin = [&](int count, int w) {
        return static_cast<int>(static_cast<long long>(count) * boxes * w / kVWarps);
    };
    const int piece = v_piece_doubles(p.cap, SWIGLU);

    // This warp's boxes in order, requested kVStages ahead of use.
    Round pr = open_round(u0, 0);
    int p_item = item_begin(pr.count, warp), p_mat = 0, p_stage = 0;
    auto request = [&] {
        while (pr.count > 0 && p_item >= item_begin(pr.count, warp + 1)) {
            pr = open_round(pr.u + pr.count, pr.e);
            p_item = item_begin(pr.count, warp);
        }
        if (pr.count == 0) return;
        if (lane == 0) {
            const int unit = p_item / boxes, box = p_item - unit * boxes;
            mbar_arrive_expect_tx(&sh.full[warp][p_stage], kVBoxBytes);
            tma_load_3d(ring + (warp * kVStages + p_stage) * kVBoxBytes, p_mat == 0 ? &map_w : &map_w2, 0,
                        sb0 + box * kVBoxCols, pr.e * p.n + (pr.tile + unit) * kVRows, &sh.full[warp][p_stage]);
        }
        if (++p_mat == R) {
            p_mat = 0;
            ++p_item;
        }
        p_stage = (p_stage + 1) % kVStages;
    };
    for (int s = 0; s < kVStages; ++s) request();

    int stage = 0;
    uint32_t par = 0;
    int chunk_of_image = -1;
    bool parts_free = true;      // no CTA still reads this one's pieces
    for (Round r = open_round(u0, 0); r.count > 0; r = open_round(r.u + r.count, r.e)) {
        const int cnt = sh.count[r.e], chunks = sh.chunk0[r.e + 1] - sh.chunk0[r.e], c = r.chunk - sh.chunk0[r.e];
        const int v0 = static_cast<int>(static_cast<long long>(cnt) * c / chunks);
        const int vecs = static_cast<int>(static_cast<long long>(cnt) * (c + 1) / chunks) - v0;
        const int slot0 = sh.first[r.e] + v0;
        if (r.chunk != chunk_of_image) {
            // every warp has left the previous group's image (the barrier behind its last round)
            for (int job = warp; job < sbs * p.cap; job += kVWarps) {
                const int b = job / p.cap, v = job % p.cap;
                uint8_t* img = image + b * sb_bytes;
                if (v < vecs) {
                    const int s = slot0 + v, pair = __ldg(p.g.order + s);
                    const bool ok = pair >= 0 && pair < p.g.pairs;
                    const int row = p.g.per_row == 0 ? s : ok ? pair / p.g.per_row : 0;
                    block_digits(p.x + static_cast<size_t>(row) * p.k + static_cast<size_t>(sb0 + b) * kQK, v, img, meta_offset,
                                 lane);
                } else if (v == 1 || v == 3) {
                    // the other half of a pair of vectors: columns that are never read back, kept finite
                    *reinterpret_cast<double*>(img + meta_offset + v * kVMetaBytes) = 0.0;
                }
            }
            chunk_of_image = r.chunk;
            __syncthreads();
        }
        const int i0 = item_begin(r.count, warp), i1 = item_begin(r.count, warp + 1);
        bool ok = *static_cast<volatile int*>(&sh.abort) == 0;
        // the group's pairs: vector v's in lane v (-1: not stored)
        int my_pair = -1;
        if (lane < vecs) {
            const int v = __ldg(p.g.order + slot0 + lane);
            if (v >= 0 && v < p.g.pairs) my_pair = v;
            else if (warp == 0) atomicOr(&g_moe_gemv_fault_flags, Q4K_FAULT_ROUTE_RANGE);
        }
        // y of vector v's pair (v's own lane's, by shuffle) and a row of W
        auto store = [&](int pair, int v, int grow, double a, double b) {
            if (pair < 0 || grow >= p.n) return;
            if constexpr (SWIGLU)
                p.y[static_cast<size_t>(slot0 + v) * p.n + grow] = silu_mul(static_cast<float>(a), static_cast<float>(b));
            else
                p.y[static_cast<size_t>(pair) * p.n + grow] = static_cast<float>(a);
        };
        auto run = [&](auto nt_tag) {
            constexpr int NT = decltype(nt_tag)::value;
            double acc[R][NT][2];
            int unit = i0 / boxes, box = i0 - unit * boxes;
            bool whole = true;       // the piece starts at its unit's first box
            for (int it = i0; it < i1 && ok; ++it) {
                if (it == i0 || box == 0) {
                    whole = box == 0;
#pragma unroll
                    for (int m = 0; m < R; ++m)
#pragma unroll
                        for (int i = 0; i < NT; ++i) acc[m][i][0] = acc[m][i][1] = 0.0;
                }
#pragma unroll
                for (int m = 0; m < R; ++m) {
                    ok = __all_sync(0xFFFFFFFFu,
                                    mbar_try_wait_now(&sh.full[warp][stage], par) ||
                                        mbar_wait_bounded(&sh.full[warp][stage], par, &g_moe_gemv_fault_flags));
                    if (!ok) break;
                    const uint8_t* rows = ring + (warp * kVStages + stage) * kVBoxBytes;
#pragma unroll 1
                    for (int b = box * kVBoxCols; b < min(sbs, (box + 1) * kVBoxCols); ++b)
                        superblock_rows<NT>(rows + (b & (kVBoxCols - 1)) * kBlockBytes, image + b * sb_bytes, meta_offset, lane,
                                            acc[m]);
                    __syncwarp();              // every lane has read the box
                    request();
                    if (++stage == kVStages) {
                        stage = 0;
                        par ^= 1u;
                    }
                }
                const bool ends = box + 1 == boxes;
                if (ends || it + 1 == i1) {    // the piece of this unit
                    if (!parts_free) {
                        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
                        parts_free = true;
                    }
                    const int t = lane & 3;
                    double* out = parts + static_cast<size_t>(csize > 1 ? unit + warp : 2 * warp + (whole ? 1 : 0)) * piece;
                    const int row = (lane >> 2) + 8 * (t & 1);      // even t takes rows 0..7, odd t rows 8..15
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        double v[2];
#pragma unroll
                        for (int m = 0; m < R; ++m) {
                            const double lo = acc[m][i][0] + __shfl_xor_sync(0xFFFFFFFFu, acc[m][i][0], 1);
                            const double hi = acc[m][i][1] + __shfl_xor_sync(0xFFFFFFFFu, acc[m][i][1], 1);
                            v[m] = (t & 1) ? hi : lo;
                        }
                        const int vec = 2 * i + (t >> 1);
                        const int pair = __shfl_sync(0xFFFFFFFFu, my_pair, vec);
                        if (csize == 1 && whole && ends) {
                            store(pair, vec, (r.tile + unit) * kVRows + row, v[0], v[R - 1]);
                        } else {
#pragma unroll
                            for (int m = 0; m < R; ++m) out[(m * p.cap + vec) * kVRows + row] = v[m];
                        }
                    }
                }
                if (++box == boxes) {
                    box = 0;
                    ++unit;
                }
            }
        };
        if (vecs <= 2) run(std::integral_constant<int, 1>{});
        else run(std::integral_constant<int, 2>{});
        if (!ok) sh.abort = 1;
        if (!parts_free) {       // a warp without items in this round
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            parts_free = true;
        }
        __syncwarp();
        if (csize > 1) cluster_sync();
        else __syncthreads();
        const bool sound = *static_cast<volatile int*>(&sh.abort) == 0;
        if (csize == 1) {
            // Units cut between warps: warp w adds the unit its range starts inside, if no earlier warp's does: the
            // tail of the warp before (with items), then the heads of w, w + 1, ...; lane = 16 (vector & 1) + row.
            const int unit = i0 / boxes;
            const int prev = i0 > 0 ? static_cast<int>((static_cast<long long>(i0) * kVWarps - 1) / (r.count * boxes)) : 0;
            if (sound && i0 < i1 && i0 > unit * boxes && item_begin(r.count, prev) <= unit * boxes) {
                const int row = lane & 15;
                for (int v = lane >> 4; v - (lane >> 4) < vecs; v += 2) {
                    double sum[2] = {0.0, 0.0};
#pragma unroll
                    for (int m = 0; m < R; ++m) {
                        const int at = (m * p.cap + v) * kVRows + row;
                        double d = v < vecs ? parts[(2 * prev + 1) * piece + at] : 0.0;
                        for (int w = warp; w < kVWarps && item_begin(r.count, w) < (unit + 1) * boxes; ++w)
                            if (v < vecs && item_begin(r.count, w) < item_begin(r.count, w + 1)) d += parts[2 * w * piece + at];
                        sum[m] = d;
                    }
                    const int pair = __shfl_sync(0xFFFFFFFFu, my_pair, v & 31);
                    store(v < vecs ? pair : -1, v, (r.tile + unit) * kVRows + row, sum[0], sum[R - 1]);
                }
            }
            __syncthreads();
        } else {
            // Totals: thread = (unit, vector, row), the cluster's CTAs take alternate units; pieces in order of CTA and warp.
            const int items = r.count * boxes;
            for (int i = threadIdx.x; i < r.count * p.cap * kVRows; i += kVThreads) {
                const int unit = i / (p.cap * kVRows), v = i / kVRows % p.cap, row = i % kVRows;
                if (unit % csize != rank || v >= vecs || !sound) continue;
                const int pair = __ldg(p.g.order + slot0 + v);
                // the warps whose items touch the unit
                const int wa = ((unit * boxes + 1) * kVWarps - 1) / items, wb = ((unit + 1) * boxes * kVWarps - 1) / items;
                double sum[2] = {0.0, 0.0};
                for (uint32_t cta = 0; cta < csize; ++cta)
                    for (int w = wa; w <= wb; ++w) {
                        if (item_begin(r.count, w) == item_begin(r.count, w + 1)) continue;   // no items
#pragma unroll
                        for (int m = 0; m < R; ++m) {
                            const double* src = parts + static_cast<size_t>(unit + w) * piece + (m * p.cap + v) * kVRows + row;
                            double d;
                            asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(d) : "r"(map_to_rank(src, cta)) : "memory");
                            sum[m] += d;
                        }
                    }
                store(pair < p.g.pairs ? pair : -1, v, (r.tile + unit) * kVRows + row, sum[0], sum[R - 1]);
            }
            __syncwarp();
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            parts_free = false;
        }
    }
    if (*static_cast<volatile int*>(&sh.abort) != 0)       // copies in flight land before shared memory goes
        for (int i = 0; i < 64; ++i) __nanosleep(1000000);
    if (csize > 1) {
        __syncwarp();
        if (!parts_free) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        cluster_sync();
    }
}

bool make_gemv_map(CUtensorMap* map, const void* w, long long rows, int nsb) {
    using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                       const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                       CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static EncodeTiledFn fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kBlockBytes), static_cast<cuuint64_t>(nsb),
                                static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kBlockBytes), static_cast<cuuint64_t>(nsb) * kBlockBytes};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(kBlockBytes), static_cast<cuuint32_t>(kVBoxCols),
                               static_cast<cuuint32_t>(kVRows)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(w), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of csize CTAs that the current device holds at once: a cluster lies
// in one GPC, so several SMs may stay without one, and a cluster more than fits
// would run after all others.
int gemv_clusters(int csize, int num_sms) {
    if (csize == 1) return num_sms;
    constexpr int kDevices = 64;
    static std::once_flag once[kDevices];
    static int fit[kDevices][4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
    std::call_once(once[dev], [dev] {
        for (int i = 1; i <= 3; ++i) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(1u << i);
            cfg.blockDim = dim3(kVThreads);
            cfg.dynamicSmemBytes = kVSmemLimit;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << i;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&fit[dev][i], q4k_moe_gemv_kernel<true>, &cfg) != cudaSuccess) fit[dev][i] = 0;
        }
    });
    const int got = fit[dev][csize == 2 ? 1 : csize == 4 ? 2 : 3];
    return got < num_sms / csize ? got : num_sms / csize;
}

}  // namespace

int launch_moe_gemv(const DeviceInfo& dev, const void* w, const void* w2, const float* x, const MoeGroups& g, float* y,
                    int n, int k, cudaStream_t stream) {
    const bool swiglu = w2 != nullptr;
    const int nsb = k / kQK;
    const long long rows = static_cast<long long>(g.experts) * n;
    CUtensorMap mw, mw2;
    if (!make_gemv_map(&mw, w, rows, nsb) || !make_gemv_map(&mw2, swiglu ? w2 : w, rows, nsb))
        return cuda_failure(cudaErrorInvalidValue);
    // Groups of up to four vectors, or of two where an expert has one pair on
    // average (the image is half as large). The smallest cluster whose CTAs'
    // parts of K fit (groups of two if none does).
    int csize = 1, cap = g.pairs <= g.experts ? 2 : kVMaxVec;
    while (csize < kVMaxCluster && (nsb + csize - 1) / csize > v_max_sbs(cap, swiglu)) csize *= 2;
    if ((nsb + csize - 1) / csize > v_max_sbs(cap, swiglu)) cap = 2;
    const int clusters = gemv_clusters(csize, dev.sm_count);
    if (clusters <= 0) return cuda_failure(cudaErrorInvalidConfiguration);
    MoeGemvParams p{};
    p.g = g;
    p.x = x;
    p.y = y;
    p.n = n;
    p.k = k;
    p.nsb = nsb;
    p.units = (n + kVRows - 1) / kVRows;
    p.part_sbs = (nsb + csize - 1) / csize;
    p.cap = cap;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * csize));
    cfg.blockDim = dim3(kVThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(v_smem(p.part_sbs, cap, swiglu));
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(csize);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = swiglu ? cudaLaunchKernelEx(&cfg, q4k_moe_gemv_kernel<true>, mw, mw2, p)
                                 : cudaLaunchKernelEx(&cfg, q4k_moe_gemv_kernel<false>, mw, mw2, p);
    return e == cudaSuccess ? Q4K_OK : cuda_failure(e);
}

int moe_gemv_set_attributes() {
    constexpr cudaFuncAttribute attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(q4k_moe_gemv_kernel<true>, attr, kVSmemLimit);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(q4k_moe_gemv_kernel<false>, attr, kVSmemLimit);
    return e == cudaSuccess ? Q4K_OK : cuda_failure(e);
}

int read_moe_gemv_fault_flags(unsigned* flags) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_moe_gemv_fault_flags, sizeof(v));
    if (e != cudaSuccess) return cuda_failure(e);
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(g_moe_gemv_fault_flags, &zero, sizeof(zero));
    if (e != cudaSuccess) return cuda_failure(e);
    *flags = v;
    return Q4K_OK;
}

}  // namespace q4k
