// q4k_moe_gemv.cu -- expert-grouped products of a few f32 vectors per expert
// with Q4_K matrices (q4k_moe_gemv, q4k_moe_gemv_swiglu): every pair (slot) of a
// decode batch with its own expert's matrix, each matrix row read once per
// group of up to four vectors.
//
// * Arithmetic (that of the integer GEMV for several vectors). Per 256-element
//   block b of a vector X = round(x * 2^(30 - E_b)), E_b the exponent of the
//   block's largest |x|, in four balanced base-256 digits X = sum_l 256^l X_l.
//   For every sub-block j the tensor cores form D_j[row][l] = sum q * X_l from
//   the raw quants (unsigned bytes; the high nibbles in place, as 16 q), exact in
//   32 bits, P_l = sum_j sc_j D_j[l], and with the digits' sums over the
//   sub-blocks M_l = sum_j m_j sum X_l; the row's f64 total gets 2^(E_b - 30) *
//   sum_l 256^l (d * P_l - dmin * M_l); y is that total rounded once.
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
// * Work. A unit is 16 rows x one group of vectors; clusters of CTAs own
//   contiguous ranges of units of equal cost (a group of three or four vectors
//   is two columns of MMAs and costs half as much again as one of two: 24 tokens
//   56 -> 52 us and 31 -> 29), the CTAs of a cluster equal parts of K (one CTA
//   where the digit image of the whole row fits), the warps of a CTA equal ranges
//   of the columns of a round's units. With one CTA per cluster a round is all
//   its units of a group: a warp stores the units it has whole, and the units cut
//   between warps (at most one per warp) meet in shared memory. With several, a
//   round is up to kRoundUnits units and all pieces meet in the cluster's shared
//   memory. Pieces are added in a fixed order.
// * Bound and measured. One token, 8 experts, top 2: gate/up 14336 x 4096 33 us
//   (4.0 TB/s; twice the rows take 24 us more, 5.5 TB/s), down 4096 x 14336 20
//   us; 24 tokens, 64 experts, top 4: gate/up 1536 x 2048 49 us, down 28 us.
//   Of the one-token call about 6 us are its start (planning, digits, the first
//   boxes). No unit is full in the loop: issue slots 0.60 and 0.58 used, DRAM 4.0
//   and 3.6 TB/s; warps wait on their own chain (wait 21-23 % of the stalls) and,
//   with several groups, at the barriers around the one digit image.
#include <cstdint>
#include <cuda.h>
#include <type_traits>

#include "q4k_internal.h"
#include "q4k_moe.cuh"
#include "q4k_moe.h"
#include "q4k_pair.cuh"
#include "q4k_per_device.h"
#include "q4k_superblock.cuh"
#include "q4k_swiglu.cuh"
#include "q4k_tensor_map.h"

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
constexpr int kCost2 = 2, kCost4 = 3;             // of a unit of up to two, and of four vectors
constexpr int kRoundUnits = 16;                   // most units of a round in a cluster of several CTAs
// Pieces of units in shared memory. Several CTAs: every piece of a round,
// numbered unit + warp (unique: of two neighbouring pieces one or both grow).
// One CTA: a warp's first piece if it starts inside a unit (its head), which the
// warp with the unit's first boxes adds when it comes to its own range's end.
__host__ __device__ constexpr int v_pieces(bool one_cta) { return one_cta ? kVWarps : kRoundUnits + kVWarps; }
constexpr int kVMaxCluster = 8;
// Digit image of one superblock and two vectors: [sub-block pair][lane][2][8
// bytes]; behind the images per vector 2^(E-30), and from byte 16 the sums of
// each digit over the sub-blocks, 16 bits each: [digit][sub-block].
constexpr int kVImageBytes = 2048;
constexpr int kVMetaBytes = 80;
__host__ __device__ constexpr int v_meta_offset(int cap) { return cap / 2 * kVImageBytes; }
__host__ __device__ constexpr int v_sb_bytes(int cap) { return v_meta_offset(cap) + cap * kVMetaBytes; }
// [matrix][vector][row]
__host__ __device__ constexpr int v_piece_doubles(int cap, bool swiglu) { return kVRows * cap * (swiglu ? 2 : 1); }
// Shared memory of groups of up to `cap` vectors (4, or 2 for long K) and parts
// of `sbs` superblocks; the most superblocks that fit.
constexpr int v_smem(int sbs, int cap, bool swiglu, bool one_cta) {
    return 128 + kVWarps * kVStages * kVBoxBytes + sbs * v_sb_bytes(cap) +
           v_pieces(one_cta) * v_piece_doubles(cap, swiglu) * 8;
}
constexpr int kVSmemLimit = 227 * 1024 - 6144;    // less the static part
constexpr int v_max_sbs(int cap, bool swiglu, bool one_cta) {
    return (kVSmemLimit - v_smem(0, cap, swiglu, one_cta)) / v_sb_bytes(cap);
}
static_assert(v_max_sbs(2, true, false) * kVMaxCluster * kQK >= Q4K_MOE_GEMV_MAX_K, "every accepted K fits");

struct MoeGemvParams {
    MoeGroups g;
    const float* x;
    float* y;
    int n, k, nsb;
    int units;      // row tiles of one matrix
    int part_sbs;   // superblocks of a CTA's part of K (the last one's may be fewer)
    int cap;        // most vectors per group: 4 or 2
};

struct GemvShared {   // static: below the 6 KB that kVSmemLimit leaves
    uint64_t full[kVWarps][kVStages];
    int chunk0[Q4K_MOE_MAX_EXPERTS + 1];            // first vector group of each expert
    int first[Q4K_MOE_MAX_EXPERTS], count[Q4K_MOE_MAX_EXPERTS];
    int cost0[Q4K_MOE_MAX_EXPERTS + 1];             // cost of a row tile of all groups before the expert's
    short order[kVThreads];                         // of the first pairs; -1: out of range
    long long range[2];
    int head[kVWarps];                              // rounds whose head piece the warp has left, plus one
    int abort;
};

static_assert(sizeof(GemvShared) <= 6144 - 256, "shared memory");

// What a unit of an expert's groups costs: three or four vectors are two columns
// of MMAs.
__device__ __forceinline__ int unit_cost(int cnt, int chunks) { return cnt > 2 * chunks ? kCost4 : kCost2; }

// d = A B^T: A 16 x 32 unsigned bytes (a0, a2: row g, a1, a3: row g + 8), B 8 x 32 signed.
__device__ __forceinline__ void imma(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}

// c + the products of the two signed 16-bit halves of a with bytes 0, 1 (lo) or
// 2, 3 (hi) of b.
__device__ __forceinline__ int dp2a_lo(int a, uint32_t b, int c) {
    int d;
    asm("dp2a.lo.s32.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ int dp2a_hi(int a, uint32_t b, int c) {
    int d;
    asm("dp2a.hi.s32.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// A 32-bit integer as f64, exactly: 2^52 + 2^31 + v less 2^52 + 2^31.
__device__ __forceinline__ double int_to_f64(int v) {
    return __hiloint2double(0x43300000, v ^ static_cast<int>(0x80000000u)) - 4503601774854144.0;
}

// a + 256 b as f64, exactly: as a 64-bit integer added to the bits of 2^52 + 2^51.
__device__ __forceinline__ double digits_to_f64(int a, int b) {
    const long long base = static_cast<long long>(static_cast<unsigned long long>(static_cast<uint32_t>(0x43380000 + (a >> 31))) << 32 |
                                                  static_cast<uint32_t>(a));
    long long v;
    asm("mad.wide.s32 %0, %1, 256, %2;" : "=l"(v) : "r"(b), "l"(base));
    return __longlong_as_double(v) - 6755399441055744.0;
}

// The digits of one vector's block (lane: K positions 8 lane .. + 7, v). E is
// taken from the exponent field of the largest |x| (-125 at least).
__device__ __forceinline__ void block_digits(const float (&v)[8], int vec, uint8_t* sb_image, int meta_offset, int lane) {
    uint32_t top = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xFFFFFFFFu, top);             // non-negative floats are ordered as integers
    const bool finite = top < 0x7F800000u;
    const int ex = max(static_cast<int>(top >> 23), 1) - 126;   // |x| < 2^ex
    // x 2^(30 - ex) in two exact steps (the power may lie outside f32; a step that underflows belongs to a digit 0)
    const int s1 = (30 - ex) / 2, s2 = 30 - ex - s1;
    const float up1 = __int_as_float((127 + s1) << 23), up2 = __int_as_float((127 + s2) << 23);
    int r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = finite ? __float2int_rn(v[e] * up1 * up2) : 0;
    const int j = lane >> 2, t = lane & 3;
    if (lane == 0)
        *reinterpret_cast<double*>(sb_image + meta_offset + vec * kVMetaBytes) =
            __longlong_as_double(finite ? static_cast<long long>(1023 + ex - 30) << 52 : 0x7FF8000000000000LL);
    // With 128 (1 + 256 + 256^2) added, the lower three bytes are the balanced digits plus 128: flipping their top
    // bits leaves the four signed digits as bytes. Then bytes l of four elements are brought together.
    uint32_t z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = (static_cast<uint32_t>(r[e]) + 0x00808080u) ^ 0x00808080u;
    uint8_t* img = sb_image + (vec >> 1) * kVImageBytes + (j >> 1) * 512 + (j & 1) * 8 + (16 * (vec & 1) + t) * 16;
    uint32_t w[4][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t lo01 = __byte_perm(z[4 * h], z[4 * h + 1], 0x5140), hi01 = __byte_perm(z[4 * h], z[4 * h + 1], 0x7362);
        const uint32_t lo23 = __byte_perm(z[4 * h + 2], z[4 * h + 3], 0x5140);
        const uint32_t hi23 = __byte_perm(z[4 * h + 2], z[4 * h + 3], 0x7362);
        w[0][h] = __byte_perm(lo01, lo23, 0x5410);
        w[1][h] = __byte_perm(lo01, lo23, 0x7632);
        w[2][h] = __byte_perm(hi01, hi23, 0x5410);
        w[3][h] = __byte_perm(hi01, hi23, 0x7632);
    }
#pragma unroll
    for (int l = 0; l < 4; ++l) {
        *reinterpret_cast<uint2*>(img + l * 64) = make_uint2(w[l][0], w[l][1]);
        int sum = __dp4a(static_cast<int>(w[l][0]), 0x01010101, __dp4a(static_cast<int>(w[l][1]), 0x01010101, 0));
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);        // sub-block j: lanes 4j .. 4j + 3
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
        if (t == l)
            reinterpret_cast<int16_t*>(sb_image + meta_offset + vec * kVMetaBytes + 16)[8 * l + j] = static_cast<int16_t>(sum);
    }
}

// Adds one superblock of 16 rows to the lane's totals: acc[nt][0] for row g,
// acc[nt][1] for row g + 8, each over the lane's two digits of vector 2 nt +
// t / 2 (digits 0, 1 for even t; 2, 3, in units of 256^2, for odd t).
template <int NT>
__device__ __forceinline__ void superblock_rows(const uint8_t* rows, const uint8_t* sb_image, int meta_offset, int lane,
                                                double (&acc)[NT][2]) {
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* ra = rows + g * kVRowPitch;
    const uint8_t* rb = ra + 8 * kVRowPitch;
    const Header ha = decode_header(*reinterpret_cast<const uint4*>(ra));
    const Header hb = decode_header(*reinterpret_cast<const uint4*>(rb));
    int ps[NT][4];      // 16 P_l: even sub-blocks with 16 sc_j, odd ones with 16 q (the high nibbles in place)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) ps[i][c] = 0;
#pragma unroll
    for (int jp = 0; jp < 4; ++jp) {
        const uint2 qa = *reinterpret_cast<const uint2*>(ra + kQsOffset + 32 * jp + 8 * t);
        const uint2 qb = *reinterpret_cast<const uint2*>(rb + kQsOffset + 32 * jp + 8 * t);
        const uint32_t wa = jp < 2 ? ha.sc_lo : ha.sc_hi, wb = jp < 2 ? hb.sc_lo : hb.sc_hi;
        const int sae = static_cast<int>(__byte_perm(wa, 0u, 0x4440u + ((2 * jp) & 3)) << 4), sao = static_cast<int>(__byte_perm(wa, 0u, 0x4440u + ((2 * jp + 1) & 3)));
        const int sbe = static_cast<int>(__byte_perm(wb, 0u, 0x4440u + ((2 * jp) & 3)) << 4), sbo = static_cast<int>(__byte_perm(wb, 0u, 0x4440u + ((2 * jp + 1) & 3)));
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const uint4 dg = *reinterpret_cast<const uint4*>(sb_image + i * kVImageBytes + jp * 512 + lane * 16);
            int d[4];
            imma(d, qa.x & 0x0F0F0F0Fu, qb.x & 0x0F0F0F0Fu, qa.y & 0x0F0F0F0Fu, qb.y & 0x0F0F0F0Fu, dg.x, dg.y);
            ps[i][0] += sae * d[0];
            ps[i][1] += sae * d[1];
            ps[i][2] += sbe * d[2];
            ps[i][3] += sbe * d[3];
            imma(d, qa.x & 0xF0F0F0F0u, qb.x & 0xF0F0F0F0u, qa.y & 0xF0F0F0F0u, qb.y & 0xF0F0F0F0u, dg.z, dg.w);
            ps[i][0] += sao * d[0];
            ps[i][1] += sao * d[1];
            ps[i][2] += sbo * d[2];
            ps[i][3] += sbo * d[3];
        }
    }
    const double da = ha.d * 0.0625f, db = hb.d * 0.0625f, ma = -ha.dmin, mb = -hb.dmin;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const uint8_t* meta = sb_image + meta_offset + (2 * i + (t >> 1)) * kVMetaBytes;
        const double scale = *reinterpret_cast<const double*>(meta);
        const int4 s0 = *reinterpret_cast<const int4*>(meta + 16 + 32 * (t & 1));        // the lane's lower digit
        const int4 s1 = *reinterpret_cast<const int4*>(meta + 16 + 32 * (t & 1) + 16);
        // M of two digits: |M_l| <= 8 * 63 * 4096, so M_0 + 256 M_1 fits 32 bits
        auto mins = [](const int4& s, uint32_t lo, uint32_t hi) {
            return dp2a_lo(s.x, lo, dp2a_hi(s.y, lo, dp2a_lo(s.z, hi, dp2a_hi(s.w, hi, 0))));
        };
        const int m_a = mins(s0, ha.m_lo, ha.m_hi) + 256 * mins(s1, ha.m_lo, ha.m_hi);
        const int m_b = mins(s0, hb.m_lo, hb.m_hi) + 256 * mins(s1, hb.m_lo, hb.m_hi);
        // |16 P_l| <= 16 * 8 * 63 * 32 * 15 * 128 < 2^29
        const double pa = digits_to_f64(ps[i][0], ps[i][1]);
        const double pb = digits_to_f64(ps[i][2], ps[i][3]);
        acc[i][0] = fma(scale, fma(da, pa, ma * int_to_f64(m_a)), acc[i][0]);
        acc[i][1] = fma(scale, fma(db, pb, mb * int_to_f64(m_b)), acc[i][1]);
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
    // The warps' shares are counted in columns of kItem superblocks: of one for two matrices (24 tokens: 52 -> 50 us),
    // of a box for one matrix (half boxes: 28.5 -> 29.5 us). Columns per unit, the same in every CTA:
    constexpr int kItem = SWIGLU ? 1 : kVBoxCols;
    const int cols = (p.part_sbs + kItem - 1) / kItem;

    if (lane == 0) {
        for (int s = 0; s < kVStages; ++s) mbar_init(&sh.full[warp][s], 1);
        sh.head[warp] = 0;
    }
    if (threadIdx.x == 0) {
        sh.abort = 0;
        tma_prefetch_map(&map_w);
        if (SWIGLU) tma_prefetch_map(&map_w2);
    }
    fence_mbar_init();
    pdl_launch_dependents();
    pdl_wait();
    // Experts' slots and first vector groups (warp 0; the others' redundant scans would fill the issue slots).
    // All first loads are requested before any is used: behind one another they take 0.7-1.5 us of a call.
    const int my_order = threadIdx.x < p.g.pairs ? load_i32(p.g.order + threadIdx.x) : -1;
    int2 bounds = make_int2(0, 0);                         // of expert `lane`, then of the next 32
    auto load_bounds = [&](int e) {
        return e < experts ? make_int2(load_i32(p.g.offsets + e), load_i32(p.g.offsets + e + 1)) : make_int2(0, 0);
    };
    if (warp == 0) bounds = load_bounds(lane);
    if (threadIdx.x < p.g.pairs)
        sh.order[threadIdx.x] = static_cast<short>(my_order >= 0 && my_order < p.g.pairs ? my_order : -1);
    if (warp == 0) {
        const bool even = p.cap == 2;         // every unit costs the same
        int chunks_before = 0, cost_before = 0;
        for (int e0 = 0; e0 < experts; e0 += 32) {
            const int e = e0 + lane;
            int chunks = 0, cost = 0;
            const int a = bounds.x, b = bounds.y;
            bounds = load_bounds(e + 32);
            if (e < experts) {
                const bool ok = a >= 0 && a <= b && b <= p.g.pairs;
                if (!ok && blockIdx.x == 0) atomicOr(&g_moe_gemv_fault_flags, Q4K_FAULT_ROUTE_RANGE);
                const int cnt = ok ? b - a : 0;
                sh.first[e] = a;
                sh.count[e] = cnt;
                chunks = (cnt + p.cap - 1) >> (even ? 1 : 2);
                cost = chunks * unit_cost(cnt, chunks);
            }
            int scan = chunks;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, scan, off);
                if (lane >= off) scan += v;
            }
            if (e < experts) sh.chunk0[e + 1] = chunks_before + scan;
            chunks_before += __shfl_sync(0xFFFFFFFFu, scan, 31);
            if (!even) {
                scan = cost;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int v = __shfl_up_sync(0xFFFFFFFFu, scan, off);
                    if (lane >= off) scan += v;
                }
                if (e < experts) sh.cost0[e + 1] = cost_before + scan;
                cost_before += __shfl_sync(0xFFFFFFFFu, scan, 31);
            }
        }
        if (lane == 0) sh.chunk0[0] = sh.cost0[0] = 0;
        __syncwarp();
        // This cluster's units, [range[0], range[1]): an equal share of the cost.
        const long long total = static_cast<long long>(even ? chunks_before : cost_before) * p.units;
        auto share = [&](int i) {
            return total < (1 << 23)          // at most 148 clusters: 32-bit division
                       ? static_cast<long long>(static_cast<uint32_t>(total) * (cid + i) / nclusters)
                       : total * (cid + i) / nclusters;
        };
        if (even) {
            if (lane < 2) sh.range[lane] = share(lane);
        } else {
            // a bound lies in the expert whose costs it falls into, or behind them all; neighbours find the same one
            const long long bound[2] = {share(0), share(1)};
            if (lane < 2 && bound[lane & 1] >= total) sh.range[lane] = static_cast<long long>(chunks_before) * p.units;
            for (int e = lane; e < experts; e += 32) {
                const int c0 = sh.chunk0[e], each = unit_cost(sh.count[e], sh.chunk0[e + 1] - c0);
                const long long lo = static_cast<long long>(sh.cost0[e]) * p.units;
                const long long hi = static_cast<long long>(sh.cost0[e + 1]) * p.units;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (bound[i] < lo || bound[i] >= hi) continue;
                    const long long in = bound[i] - lo;
                    sh.range[i] = static_cast<long long>(c0) * p.units + (each == kCost2 ? in / kCost2 : in / kCost4);
                }
            }
        }
    }
    __syncthreads();
    const long long u0 = sh.range[0], u1 = sh.range[1];

    // The rounds of this cluster: up to kRoundUnits units of one vector group.
    struct Round {
        long long u;         // first unit
        int count;           // units; 0 behind the last round
        int e, chunk, tile;  // expert, vector group, row tile of the first unit
    };
    auto open_round = [&](long long u, int e) {
        Round r{u, 0, e, 0, 0};
        if (u >= u1) return r;
        r.chunk = u1 < (1 << 23) ? static_cast<int>(static_cast<uint32_t>(u) / static_cast<uint32_t>(p.units))
                                    : static_cast<int>(u / p.units);
        r.tile = static_cast<int>(u - static_cast<long long>(r.chunk) * p.units);
        while (r.chunk >= sh.chunk0[r.e + 1]) ++r.e;
        const long long left = min(u1 - u, static_cast<long long>(p.units - r.tile));
        r.count = static_cast<int>(csize > 1 ? min(left, static_cast<long long>(kRoundUnits)) : left);
        return r;
    };
    auto item_begin = [&](int count, int w) {
        return static_cast<int>(static_cast<unsigned long long>(static_cast<uint32_t>(count) * static_cast<uint32_t>(cols)) *
                                static_cast<uint32_t>(w) / kVWarps);
    };
    const int piece = v_piece_doubles(p.cap, SWIGLU);

    // This warp's boxes in order, requested kVStages ahead of use.
    const Round first_round = open_round(u0, 0);
    Round pr = first_round;
    int p_left = 0, p_col = 0, p_row = 0, p_mat = 0, p_stage = 0;   // columns left in the round, the next one and its row
    // Columns of the box that starts at col: up to the unit's or the range's end.
    auto box_cols = [&](int col, int left) { return min(min(kVBoxCols / kItem, cols - col), left); };
    auto enter = [&] {
        const int i0 = item_begin(pr.count, warp);
        p_left = item_begin(pr.count, warp + 1) - i0;
        const int unit = i0 / cols;
        p_col = i0 - unit * cols;
        p_row = pr.e * p.n + (pr.tile + unit) * kVRows;
    };
    enter();
    auto request = [&] {
        while (p_left == 0) {
            if (pr.count == 0) return;
            pr = open_round(pr.u + pr.count, pr.e);
            enter();
        }
        if (lane == 0) {
            mbar_arrive_expect_tx(&sh.full[warp][p_stage], kVBoxBytes);
            tma_load_3d(ring + (warp * kVStages + p_stage) * kVBoxBytes, p_mat == 0 ? &map_w : &map_w2, 0,
                        sb0 + p_col * kItem, p_row, &sh.full[warp][p_stage]);
        }
        if (++p_mat == R) {
            p_mat = 0;
            const int take = box_cols(p_col, p_left);
            p_left -= take;
            p_col += take;
            if (p_col == cols) {
                p_col = 0;
                p_row += kVRows;
            }
        }
        p_stage = (p_stage + 1) % kVStages;
    };

    // A round's vector group: its slots, and vector v's pair in lane v (-1: not stored).
    struct Group {
        int slot0, vecs, pair;
    };
    auto open_group = [&](const Round& r) {
        const int cnt = sh.count[r.e], chunks = sh.chunk0[r.e + 1] - sh.chunk0[r.e], c = r.chunk - sh.chunk0[r.e];
        int v0 = 0, v1 = cnt;        // an expert's vectors in equal groups
        if (chunks > 1) {
            v0 = static_cast<int>(static_cast<uint32_t>(cnt) * static_cast<uint32_t>(c) / static_cast<uint32_t>(chunks));
            v1 = static_cast<int>(static_cast<uint32_t>(cnt) * static_cast<uint32_t>(c + 1) / static_cast<uint32_t>(chunks));
        }
        Group g;
        g.vecs = v1 - v0;
        g.slot0 = sh.first[r.e] + v0;
        g.pair = -1;
        if (lane < g.vecs) {
            const int slot = g.slot0 + lane;
            const int v = slot < kVThreads ? sh.order[slot] : p.g.order[slot];
            if (v >= 0 && v < p.g.pairs) g.pair = v;
        }
        return g;
    };
    // Block `job` = (superblock, vector) of the group's digit image: this lane's eight elements.
    auto block_of = [](int job, int vecs) { return vecs == 3 ? job * 43691 >> 17 : job >> (vecs >> 1); };   // job / vecs
    auto fetch = [&](const Group& g, int job, float (&v)[8]) {
        const int b = block_of(job, g.vecs), vec = job - b * g.vecs;
        const int pair = __shfl_sync(0xFFFFFFFFu, g.pair, vec);
        const int row = p.g.per_row == 0 ? g.slot0 + vec : pair >= 0 ? pair / p.g.per_row : 0;
        const float4* src =
            reinterpret_cast<const float4*>(p.x + static_cast<size_t>(row) * p.k + static_cast<size_t>(sb0 + b) * kQK) + 2 * lane;
        const float4 lo = load_f4(src), hi = load_f4(src + 1);
        v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
        v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    };

    int stage = 0;
    uint32_t par = 0;
    int chunk_of_image = -1;
    bool parts_free = true;      // no CTA still reads this one's pieces
    int round_no = 0;
    // A warp's head piece of a round is in shared memory (its writes released, acquired by the reader).
    auto publish_head = [&](int round) {
        asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(smem_addr(&sh.head[warp])), "r"(round + 1) : "memory");
    };
    auto wait_head = [&](int w, int round) {
        for (unsigned i = 0; i < kSpinLimit; ++i) {
            int v;
            asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(v) : "r"(smem_addr(&sh.head[w])) : "memory");
            if (v == round + 1) return true;
            __nanosleep(64);
        }
        atomicOr(&g_moe_gemv_fault_flags, kFaultCopyTimeout);
        return false;
    };
    for (Round r = first_round; r.count > 0; r = open_round(r.u + r.count, r.e)) {
        const Group grp = open_group(r);
        const int vecs = grp.vecs, slot0 = grp.slot0, my_pair = grp.pair;
        if (warp == 0 && lane < vecs && my_pair < 0) atomicOr(&g_moe_gemv_fault_flags, Q4K_FAULT_ROUTE_RANGE);
        if (r.chunk != chunk_of_image) {
            // every warp has left the previous group's image (the barrier behind its last round); a warp's next block
            // is requested before the digits of the one at hand. The first weights are requested behind the first
            // digits: beside a full ring of copies everything else that comes from L2, instructions too, waits
            // microseconds
            const int jobs = sbs * vecs;
            float cur[8], nxt[8];
            if (warp < jobs) fetch(grp, warp, cur);
            for (int job = warp; job < jobs; job += kVWarps) {
                if (job + kVWarps < jobs) fetch(grp, job + kVWarps, nxt);
                const int b = block_of(job, vecs);
                block_digits(cur, job - b * vecs, image + b * sb_bytes, meta_offset, lane);
#pragma unroll
                for (int e = 0; e < 8; ++e) cur[e] = nxt[e];
            }
            if (chunk_of_image < 0)
                for (int s = 0; s < kVStages; ++s) request();
            if (vecs & 1)      // the other half of a pair of vectors: never read back, kept finite
                for (int b = threadIdx.x; b < sbs; b += kVThreads)
                    *reinterpret_cast<double*>(image + b * sb_bytes + meta_offset + vecs * kVMetaBytes) = 0.0;
            chunk_of_image = r.chunk;
            __syncthreads();
        }
        const int i0 = item_begin(r.count, warp), i1 = item_begin(r.count, warp + 1);
        bool ok = *static_cast<volatile int*>(&sh.abort) == 0;
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
            // totals of the matrix at hand and of the other one (swapped after every box: one copy of the loop's code)
            double acc[NT][2], other[NT][2];
            int unit = i0 / cols, col = i0 - unit * cols;
            bool whole = true;       // the piece starts at its unit's first superblock
            for (int it = i0; it < i1 && ok;) {
                const int take = box_cols(col, i1 - it);
                if (it == i0 || col == 0) {
                    whole = col == 0;
#pragma unroll
                    for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = other[i][0] = other[i][1] = 0.0;
                }
#pragma unroll 1
                for (int m = 0; m < R; ++m) {
                    ok = __all_sync(0xFFFFFFFFu,
                                    mbar_try_wait_now(&sh.full[warp][stage], par) ||
                                        mbar_wait_bounded(&sh.full[warp][stage], par, &g_moe_gemv_fault_flags));
                    if (!ok) break;
                    const uint8_t* rows = ring + (warp * kVStages + stage) * kVBoxBytes;
#pragma unroll 1
                    for (int b = 0; b < min(take * kItem, sbs - col * kItem); ++b)
                        superblock_rows<NT>(rows + b * kBlockBytes, image + (col * kItem + b) * sb_bytes, meta_offset, lane, acc);
                    __syncwarp();              // every lane has read the box
                    request();
                    if (++stage == kVStages) {
                        stage = 0;
                        par ^= 1u;
                    }
                    if constexpr (R == 2) {
#pragma unroll
                        for (int i = 0; i < NT; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const double v = acc[i][h];
                                acc[i][h] = other[i][h];
                                other[i][h] = v;
                            }
                    }
                }
                it += take;
                col += take;
                const bool ends = col == cols;
                if (ok && (ends || it == i1)) {        // the piece of this unit
                    if (!parts_free) {
                        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
                        parts_free = true;
                    }
                    const int t = lane & 3;
                    // even t holds digits 0 and 1, odd t 2 and 3; even t goes on with row g, odd t with g + 8
                    const int row = (lane >> 2) + 8 * (t & 1);
                    const bool head = csize > 1 || !whole;     // goes to shared memory
                    double* out = parts + static_cast<size_t>(csize > 1 ? unit + warp : warp) * piece + row;
                    if (csize == 1 && whole && !ends) {        // the rest of the unit: the next warps' heads
                        for (int w = warp + 1; w < kVWarps && item_begin(r.count, w) < (unit + 1) * cols; ++w)
                            if (item_begin(r.count, w) < item_begin(r.count, w + 1)) ok = wait_head(w, round_no) && ok;
                    }
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const int vec = 2 * i + (t >> 1);
                        double v[2];
#pragma unroll
                        for (int m = 0; m < R; ++m) {
                            const double a0 = m == 0 ? acc[i][0] : other[i][0], a1 = m == 0 ? acc[i][1] : other[i][1];
                            const double mine = (t & 1) ? a1 * 65536.0 : a0, give = (t & 1) ? a0 * 65536.0 : a1;
                            v[m] = mine + __shfl_xor_sync(0xFFFFFFFFu, give, 1);
                            if (head) out[(m * p.cap + vec) * kVRows] = v[m];
                        }
                        const int pair = __shfl_sync(0xFFFFFFFFu, my_pair, vec);
                        if (!head) {
                            if (!ends)
                                for (int w = warp + 1; w < kVWarps && item_begin(r.count, w) < (unit + 1) * cols; ++w)
                                    if (item_begin(r.count, w) < item_begin(r.count, w + 1)) {
#pragma unroll
                                        for (int m = 0; m < R; ++m)
                                            v[m] += parts[static_cast<size_t>(w) * piece + (m * p.cap + vec) * kVRows + row];
                                    }
                            if (ok) store(pair, vec, (r.tile + unit) * kVRows + row, v[0], v[R - 1]);
                        }
                    }
                    if (head && csize == 1) {
                        __syncwarp();
                        if (lane == 0) publish_head(round_no);
                    }
                }
                if (ends) {
                    col = 0;
                    ++unit;
                }
            }
        };
        if (vecs <= 2) run(std::integral_constant<int, 1>{});
        else run(std::integral_constant<int, 2>{});
        if (!ok) sh.abort = 1;
        ++round_no;
        if (csize == 1) {
            __syncthreads();         // every warp has left the image and the heads
        } else {
            if (!parts_free) {       // a warp without items in this round
                asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
                parts_free = true;
            }
            __syncwarp();
            cluster_sync();
            const bool sound = *static_cast<volatile int*>(&sh.abort) == 0;
            // Totals: thread = (unit, vector, row), the cluster's CTAs take alternate units; pieces in order of CTA and warp.
            const int items = r.count * cols;
            for (int i = threadIdx.x; i < r.count * p.cap * kVRows; i += kVThreads) {
                const int unit = i / (p.cap * kVRows), v = i / kVRows % p.cap, row = i % kVRows;
                if (unit % csize != rank || v >= vecs || !sound) continue;
                const int pair = p.g.order[slot0 + v];
                // the warps whose items touch the unit
                const int wa = ((unit * cols + 1) * kVWarps - 1) / items, wb = ((unit + 1) * cols * kVWarps - 1) / items;
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
    if (encode_tiled() == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kBlockBytes), static_cast<cuuint64_t>(nsb),
                                static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kBlockBytes), static_cast<cuuint64_t>(nsb) * kBlockBytes};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(kBlockBytes), static_cast<cuuint32_t>(kVBoxCols),
                               static_cast<cuuint32_t>(kVRows)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(w), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of csize CTAs that the current device holds at once: a cluster lies
// in one GPC, so several SMs may stay without one, and a cluster more than fits
// would run after all others. The device's first call also sets the kernels'
// attributes (here, so that programs without experts load none of this).
cudaError_t gemv_clusters(int csize, int num_sms, int* clusters) {
    struct Fit {
        int of[4];   // by the logarithm of the size
    };
    static PerDevice<Fit> fits;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    Fit fit;
    e = fits.get(dev, &fit, [](Fit* made) {
        constexpr cudaFuncAttribute smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
        cudaError_t set = cudaFuncSetAttribute(q4k_moe_gemv_kernel<true>, smem, kVSmemLimit);
        if (set == cudaSuccess) set = cudaFuncSetAttribute(q4k_moe_gemv_kernel<false>, smem, kVSmemLimit);
        if (set != cudaSuccess) return set;
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
            const cudaError_t query = cudaOccupancyMaxActiveClusters(&made->of[i], q4k_moe_gemv_kernel<true>, &cfg);
            if (query != cudaSuccess) return query;
        }
        return cudaSuccess;
    });
    if (e != cudaSuccess) return e;
    *clusters = num_sms;
    if (csize == 1) return cudaSuccess;
    const int got = fit.of[csize == 2 ? 1 : csize == 4 ? 2 : 3];
    *clusters = got < num_sms / csize ? got : num_sms / csize;
    return *clusters > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
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
    // average (the image is half as large). Measured, groups of two / of four, us,
    // gate/up then down: 8 experts 14336 x 4096, 2 pairs 33/39, 20/27; 8 pairs 76/85,
    // 44/49; 16 pairs 122/132, 71/77 (four vectors of K = 4096 need two CTAs). 64
    // experts 1536 x 2048, 16 pairs 24/27, 15/16; 48 pairs 36/39, 21/23; 64 pairs
    // 42/36, 24/22; 128 pairs 61/58, 33/33; 256 pairs 98/88, 51/46. The smallest
    // cluster whose CTAs' parts of K fit (groups of two if none does).
    int csize = 1, cap = g.pairs <= g.experts ? 2 : kVMaxVec;
    while (csize < kVMaxCluster && (nsb + csize - 1) / csize > v_max_sbs(cap, swiglu, csize == 1)) csize *= 2;
    if ((nsb + csize - 1) / csize > v_max_sbs(cap, swiglu, csize == 1)) cap = 2;
    int clusters = 0;
    cudaError_t e = gemv_clusters(csize, dev.sm_count, &clusters);
    if (e != cudaSuccess) return cuda_failure(e);
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
    cfg.dynamicSmemBytes = static_cast<size_t>(v_smem(p.part_sbs, cap, swiglu, csize == 1));
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
    e = swiglu ? cudaLaunchKernelEx(&cfg, q4k_moe_gemv_kernel<true>, mw, mw2, p)
               : cudaLaunchKernelEx(&cfg, q4k_moe_gemv_kernel<false>, mw, mw2, p);
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
