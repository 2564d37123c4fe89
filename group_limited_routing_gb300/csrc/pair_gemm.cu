// Dense products of the training operators on CTA pairs (tcgen05 cta_group::2,
// TMEM accumulators, TMA): the vocabulary loss's logits, and the gradient
// products of the loss and of the router.
//
// A pair computes 256 x 256 tiles, K in blocks of 64: each CTA loads its own
// 128 rows of A and 128 of the 256 columns of B (16 + 16 KB per block, six
// blocks in flight), the even CTA issues M = 256, N = 256 MMAs over both CTAs'
// shared memory, and each CTA's TMEM receives its 128 rows of the accumulator.
// Two accumulators fit in TMEM, so one tile's epilogue overlaps the next
// tile's MMAs.  Either operand may be K-major (rows of K) or MN-major (rows
// of M or N, as a gradient's transposed operand lies in memory): no operand is
// ever transposed in memory.  The products are bound by the tensor cores; the
// softmax work of the loss (PG_STATS, PG_DLOGITS) is in the epilogue, so the
// [rows, vocabulary] logits exist in TMEM only.
//
// The tensor core does not round its running fp32 sum to nearest: over a long K
// the sum drifts by several times an fp32 product's error.  Where the result
// stays fp32 (the loss, the router weight's gradient), K is cut into parts:
// each part has an accumulator of its own, and the epilogue warps add the
// parts in registers, rounding to nearest.
//
// A CTA takes 32 KB of operands for each 512 cycles of MMAs, 64 bytes a cycle,
// which is also what an SM was measured to draw from L2 (loads alone, no MMAs:
// 18.8 TB/s over 152 SMs): long products run at the tensor cores' rate only while
// every stage is full.  Measured on one GB300 (bf16 peak 1957 TFLOP/s in a burst,
// 1758 sustained under the power cap): T = 8192, H = 2048, V = 131072 loss 2.45 ms,
// 1705 TFLOP/s; V = 65536 gradient 3.75-3.84 ms, 1630-1670 TFLOP/s; the
// router's weight gradient at T = 32768 59 us, tensor pipe 84% active.
//
// Roles (320 threads): warp 0 lane 0 loads, warp 1 lane 0 of the even CTA
// issues the MMAs, warps 2..9 run the epilogue: TMEM lanes 32 (w % 4) .. + 31, the
// tile's left or right 128 columns.
// Every wait is bounded; when one runs out, every role leaves its loop, copies
// in flight are waited for (bounded), TMEM is freed and the status word gets
// MOE_STATUS_TIMEOUT.
#include <cuda_bf16.h>

#include <float.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace glr {

namespace {

constexpr int PG_EPI_WARPS = 8;
constexpr int PG_THREADS = 64 + 32 * PG_EPI_WARPS;
constexpr int PG_BM = 256, PG_BN = 256;          // a pair's tile
constexpr int PG_HALF = PG_BN / 2;               // an epilogue warp's columns
constexpr float LOG2E = 1.44269504088896341f;

constexpr int PG_ATOM = 64 * GEMM_BK * 2;        // 64 x 64 bf16, 8 KB
constexpr int PG_B_BYTES = 2 * PG_ATOM;          // a CTA's 128 columns of B
constexpr int PG_SLOTS = 2;                      // accumulators in TMEM
constexpr int PG_TMEM_COLS = 512;

template <int EPI>
constexpr bool IS_STATS = EPI == PG_STATS || EPI == PG_STATS_FEW;

// Shared memory: a ring of operand stages, and per epilogue warp the 4 KB
// box its output leaves through (none for the statistics; two more where an
// addend arrives, a tile ahead).  A sixth stage is worth more than a second
// output box: with five, the long products of the loss's gradient took 3% more.
// Storing from registers instead, without boxes and with a seventh stage, took
// 24% more for the gradients' outputs (a warp's store then touches 32 rows).
// PG_STATS_FEW is for at most PAIR_FEW_ROWS rows, where the product streams B
// from memory: a stage holds those rows of A only, and the shared memory this
// frees goes to a deeper ring of B.  The MMA still reads 128 rows per CTA; the
// rest alias the bytes behind and reach accumulator rows that nobody reads.
// SPLIT: fp32 operands as bf16 parts, SPLIT of A and 4 - SPLIT of B, of which
// three products are formed: four loads for three products.  A stage is then one
// part's K block (16 KB), released by the last product that reads it; a stage of
// all four left the tensor core waiting for memory (two fit beside the boxes).
//   2: the parts in order A middle, B high, A high, B middle, and the products
//      middle x high, high x high, high x middle
//   3: B, A low, A middle, A high, and each A x B as its A arrives
//   1: the same with the operands' roles exchanged
template <int EPI, int SPLIT>
struct PgCfg {
    static constexpr bool FEW = EPI == PG_STATS_FEW;
    static constexpr int A_ROWS = FEW ? PAIR_FEW_ROWS : 128;
    static constexpr int A_BYTES = A_ROWS * GEMM_BK * 2;
    static constexpr int STAGE_BYTES = SPLIT ? PG_B_BYTES : A_BYTES + PG_B_BYTES;
    static constexpr int BUFS = IS_STATS<EPI> ? 0 : EPI == PG_BF16_ADD ? 3 : 1;
    static constexpr int STAGING = BUFS * PG_EPI_WARPS * 4096;
    static constexpr int STAGES = (230400 - STAGING) / STAGE_BYTES;
    static constexpr int NBARS = 2 * STAGES + 2 * PG_SLOTS + 1 + PG_EPI_WARPS;
    static constexpr int SMEM = STAGES * STAGE_BYTES + STAGING + 1024 /*align*/ + NBARS * 8 + 16;
    static_assert(SMEM <= 232448, "more than 227 KB of shared memory");
    static_assert(STAGE_BYTES % 1024 == 0, "swizzle atoms need 1024-B alignment");
};

// fp32 box added to global memory from shared memory (bulk-group completion)
__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap *map, uint32_t src, int c0, int c1)
{
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(c0), "r"(c1)
                 : "memory");
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// One unit of work: a tile and its K blocks, in parts of at most p.part_blocks.
struct Unit {
    int m0, n0, nt, split;
    int k0, k1;
    int parts;
};

struct Shape {
    int M, m_tiles, n_tiles, kblocks, part_blocks, splits, split_rows, units;
};

__device__ __forceinline__ Shape shape_of(const PairGemmParams &p)
{
    Shape sh;
    const int rows = p.meta ? p.meta->rows : 0;
    sh.M = p.m_from_rows ? rows : p.M;
    sh.kblocks = p.k_from_rows ? (rows + GEMM_BK - 1) / GEMM_BK : p.kblocks;
    sh.part_blocks = p.few_part_blocks && rows <= p.few_rows ? p.few_part_blocks : p.part_blocks;
    sh.m_tiles = (sh.M + PG_BM - 1) / PG_BM;
    sh.n_tiles = (p.N + PG_BN - 1) / PG_BN;
    sh.splits = p.splits ? p.splits : p.meta->splits;
    sh.split_rows = p.split_rows ? p.split_rows : sh.m_tiles * PG_BM;
    sh.units = sh.m_tiles * sh.n_tiles * sh.splits;
    return sh;
}

__device__ __forceinline__ Unit unit_of(const PairGemmParams &p, const Shape &sh, int u)
{
    Unit t;
    const int tiles = sh.m_tiles * sh.n_tiles;
    t.split = u / tiles;
    const int tile = u - t.split * tiles;
    const int per = p.group_m * sh.n_tiles;
    const int g = tile / per, in = tile - g * per;
    const int gm = min(p.group_m, sh.m_tiles - g * p.group_m);
    t.nt = in / gm;
    t.m0 = (g * p.group_m + in % gm) * PG_BM;
    t.n0 = t.nt * PG_BN;
    t.k0 = (int)((long long)sh.kblocks * t.split / sh.splits);
    t.k1 = (int)((long long)sh.kblocks * (t.split + 1) / sh.splits);
    t.parts = (t.k1 - t.k0 + sh.part_blocks - 1) / sh.part_blocks;
    return t;
}

// Writes 128 bytes of each of this warp's 32 rows (lane = row, eight 16-byte
// pieces in v) into a staging box, as the 128-byte swizzle lays them out.
__device__ __forceinline__ void fill_box(uint8_t *box, const uint4 (&v)[8], int lane)
{
#pragma unroll
    for (int q = 0; q < 8; ++q)
        *reinterpret_cast<uint4 *>(box + lane * 128 + ((q ^ (lane & 7)) << 4)) = v[q];
    fence_proxy_async_smem();
    __syncwarp();
}

// Sends a filled box to the output map.  Boxes outside the map are skipped; TMA
// clips those that cross its edge.
template <bool ADD>
__device__ __forceinline__ void send_box(const PairGemmParams &p, const uint8_t *box, int lane, int col, int row)
{
    if (lane == 0) {
        if (col < p.out_cols && row < p.out_rows) {
            if (ADD)
                tma_reduce_add_2d(&p.tmOut, smem_u32(box), col, row);
            else
                tma_store_2d(&p.tmOut, smem_u32(box), col, row);
        }
        bulk_commit_group();
    }
}

// through the warp's only box: free once the store before has read it
template <bool ADD>
__device__ __forceinline__ void store_box(const PairGemmParams &p, uint8_t *box, const uint4 (&v)[8], int lane,
                                          int col, int row)
{
    if (lane == 0)
        bulk_wait_group_read<0>();
    __syncwarp();
    fill_box(box, v, lane);
    send_box<ADD>(p, box, lane, col, row);
}

// Softmax statistics of this lane's row over the warp's 128 columns: a base b
// (in log2) and s = sum 2^(z log2 e - b).  The exponentials' base is finite even
// when the largest logit is not, so that an infinite or NaN logit shows in s.  With
// +inf it is the largest fp32, which no other block's base exceeds when the blocks are
// joined; columns of -inf alone leave the join's neutral element (-inf, 0).
__device__ __forceinline__ void epilogue_stats(const PairGemmParams &p, const Shape &sh, const Unit &t,
                                               uint32_t (&z)[PG_HALF], int half, int row)
{
    const int col0 = t.n0 + half * PG_HALF;
    const int ncols = min(PG_HALF, p.N - col0);
    if (ncols <= 0)
        return;
    if (ncols < PG_HALF)
#pragma unroll
        for (int i = 0; i < PG_HALF; ++i)
            if (i >= ncols)
                z[i] = 0xff800000u;
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < PG_HALF; ++i)
        m[i & 3] = fmaxf(m[i & 3], __uint_as_float(z[i]));
    const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * LOG2E;
    float base = top > -INFINITY ? fminf(top, FLT_MAX) : 0.0f;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < PG_HALF; ++i)
        s[i & 3] += ex2_approx(fmaf(__uint_as_float(z[i]), LOG2E, -base));
    const float sum = (s[0] + s[1]) + (s[2] + s[3]);
    if (!(top > -INFINITY) && sum == 0.0f)          // (a NaN among them is in the sum)
        base = -INFINITY;
    const bool valid = row < sh.M;
    const int at = valid ? p.target[row] - (p.n0 + col0) : -1;
    const bool mine = at >= 0 && at < ncols;
    float zt = 0.0f;
    if (__any_sync(0xffffffffu, mine)) {
#pragma unroll
        for (int i = 0; i < PG_HALF; ++i)
            if (at == i)
                zt = __uint_as_float(z[i]);
    }
    if (valid) {
        p.stats[(size_t)(2 * t.nt + half) * p.ld_stats + row] = make_float2(base, sum);
        if (mine)
            p.target_logit[row] = zt;
    }
}

// dz of the warp's columns in bf16, 64 at a time.  The rounding (half a step,
// 2^-8 of each value) makes dz an operand of the tensor core; the rows' weights
// are divided by the largest of them first, so that a mean's equal weights
// are 1 exactly and add no rounding of their own, common to every value.  A few
// rows' gradient is mostly that of their targets, whose roundings (of p - 1) do not
// average out; there the rows repeat (VocabMeta) and the second time give what the
// first rounding left.
__device__ __forceinline__ void epilogue_dlogits(const PairGemmParams &p, const Shape &sh, const Unit &t,
                                                 uint32_t tacc, int half, int row, int row0, int lane, uint8_t *box)
{
    const bool valid = row < sh.M;
    const float nl = valid ? -p.lse[row] * LOG2E : 0.0f;
    const float w = valid ? p.weight[row] : 0.0f;
    const int target = valid ? p.target[row] - p.n0 : -1;
    const bool low = valid && row >= p.meta->counted, any_low = __any_sync(0xffffffffu, low);
#pragma unroll 1
    for (int c = t.n0 + half * PG_HALF; c < min(t.n0 + (half + 1) * PG_HALF, p.N); c += 64) {
        uint32_t r[64];
        tmem_load64(tacc + (c - t.n0), r);
        const int at = target - c;
        float f[64];
#pragma unroll
        for (int i = 0; i < 64; ++i)
            f[i] = ex2_approx(fmaf(__uint_as_float(r[i]), LOG2E, nl));
        if (__any_sync(0xffffffffu, at >= 0 && at < 64)) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (at == i)
                    f[i] -= 1.0f;
        }
#pragma unroll
        for (int i = 0; i < 64; ++i)
            f[i] = valid ? f[i] * w : 0.0f;
        if (p.N - c < 64)
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (i >= p.N - c)
                    f[i] = 0.0f;
        uint4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            v[q] = make_uint4(bf16x2(f[8 * q], f[8 * q + 1]), bf16x2(f[8 * q + 2], f[8 * q + 3]),
                              bf16x2(f[8 * q + 4], f[8 * q + 5]), bf16x2(f[8 * q + 6], f[8 * q + 7]));
        if (any_low) {
            auto rest = [&](uint32_t hi, float a, float b) {
                return low ? bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u)) : hi;
            };
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = make_uint4(rest(v[q].x, f[8 * q], f[8 * q + 1]), rest(v[q].y, f[8 * q + 2], f[8 * q + 3]),
                                  rest(v[q].z, f[8 * q + 4], f[8 * q + 5]), rest(v[q].w, f[8 * q + 6], f[8 * q + 7]));
        }
        store_box<false>(p, box, v, lane, c, row0);
    }
}

// The warp's fp32 sums into the split's slice.  Each element is stored or added
// to once per launch, so the sums' order is that of the launches.
__device__ __forceinline__ void epilogue_partial(const PairGemmParams &p, const Shape &sh, const Unit &t,
                                                 const uint32_t (&z)[PG_HALF], int half, int row0, int lane, uint8_t *box)
{
    const int row = t.split * sh.split_rows + row0;
#pragma unroll
    for (int c = 0; c < PG_HALF; c += 32) {
        const int col = t.n0 + half * PG_HALF + c;
        if (col < p.N) {
            uint4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = make_uint4(z[c + 4 * q], z[c + 4 * q + 1], z[c + 4 * q + 2], z[c + 4 * q + 3]);
            if (p.accumulate)
                store_box<true>(p, box, v, lane, col, row);
            else
                store_box<false>(p, box, v, lane, col, row);
        }
    }
}

// One 64-column box of a bf16 output, scaled, plus the addend that lies in the
// box (as TMA laid it out there) if there is one; one rounding.
template <bool ADD>
__device__ __forceinline__ void bf16_box(uint32_t tacc, bool empty, float scale, const uint8_t *box, int lane,
                                         uint4 (&v)[8])
{
    uint32_t r[64];
    if (empty) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
            r[i] = 0u;
    } else {
        tmem_load64(tacc, r);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = __uint_as_float(r[8 * q + i]) * scale;
        if (ADD) {
            const uint4 a = *reinterpret_cast<const uint4 *>(box + lane * 128 + ((q ^ (lane & 7)) << 4));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] += __uint_as_float(w[i] << 16);
                f[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
            }
        }
        v[q] = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
    }
}

template <int EPI, bool A_MN, bool B_MN, int SPLIT>
__global__ void __launch_bounds__(PG_THREADS, 1) pair_gemm_kernel(const __grid_constant__ PairGemmParams p)
{
    using C = PgCfg<EPI, SPLIT>;
    constexpr uint32_t IDESC = idesc_bf16_f32(PG_BM, PG_BN, A_MN, B_MN);
    extern __shared__ uint8_t dsmem[];
    const uint32_t raw = smem_u32(dsmem);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *staging = dsmem + (base - raw) + C::STAGES * C::STAGE_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(staging + C::STAGING);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + C::NBARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = (rank == 0);
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int st) { return bar0 + 8u * st; };
    auto empty_bar = [&](int st) { return bar0 + 8u * (C::STAGES + st); };
    const uint32_t tfull0 = bar0 + 8u * (2 * C::STAGES);
    const uint32_t tempty0 = tfull0 + 8u * PG_SLOTS;
    const uint32_t fin_bar = tempty0 + 8u * PG_SLOTS;
    const uint32_t add_bar0 = fin_bar + 8u;

    if (threadIdx.x == 0) {
        for (int st = 0; st < C::STAGES; ++st) {
            mbar_init(full_bar(st), 1);
            mbar_init(empty_bar(st), 1);
        }
        for (int a = 0; a < PG_SLOTS; ++a) {
            mbar_init(tfull0 + 8u * a, 1);
            mbar_init(tempty0 + 8u * a, 2 * PG_EPI_WARPS);    // (the leader's: both CTAs' epilogue warps)
        }
        mbar_init(fin_bar, 1);
        for (int w = 0; w < PG_EPI_WARPS; ++w)
            mbar_init(add_bar0 + 8u * w, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_map(&p.tmA);
        tma_prefetch_map(&p.tmB);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_holder), PG_TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();            // both CTAs' barriers initialised and TMEM allocated
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // Operands and row counts come from earlier kernels; of a product beside the one
    // launched before it, from the kernels that that one waited for before it let
    // this one start (so this one need only outlast it).
    if (p.beside != PG_SECOND)
        pdl_wait();
    if (p.beside == PG_FIRST)
        pdl_trigger();

    const int npairs = (int)gridDim.x / 2;
    const int pair = (int)blockIdx.x / 2;
    const Shape sh = shape_of(p);
    const bool packed = p.meta && p.meta->packed;
    const unsigned long long limit = p.wait_limit_ns ? p.wait_limit_ns : WAIT_LIMIT_NS;
    bool aborted_peer_loads = false;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- TMA producer
            const CUtensorMap *ma = (packed && (IS_STATS<EPI> || EPI == PG_DLOGITS)) ? &p.tmHidden : &p.tmA;
            const CUtensorMap *mb = (packed && EPI == PG_BF16) ? &p.tmHidden : &p.tmB;
            const uint32_t full_leader0 = mapa_shared(full_bar(0), 0);
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_parity = 0;
            bool ok = !p.inject_withhold;
            for (int u = pair; ok && u < sh.units; u += npairs) {
                const Unit t = unit_of(p, sh, u);
                const int m = t.m0 + rank * 128, n = t.n0 + rank * 128;
                for (int kb = t.k0; ok && kb < t.k1; ++kb) {
                    const int k = kb * GEMM_BK;
                    uint32_t to = 0, fb = 0;
                    // the next stage, free, its bytes announced
                    auto take = [&]() {
                        if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, limit))
                            return false;
                        to = base + stage * C::STAGE_BYTES;
                        fb = full_leader0 + 8u * stage;
                        if (leader)
                            mbar_arrive_expect_tx(full_bar(stage),
                                                  C::FEW ? C::A_BYTES + 2 * PG_B_BYTES : 2 * C::STAGE_BYTES);
                        issued |= 1u << stage;
                        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                        if (++stage == C::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        return true;
                    };
                    auto load = [&](const CUtensorMap *map, bool mn_major, int mn, int off, uint32_t dst) {
                        if (mn_major) {
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                tma_load_2d_pair(dst + q * PG_ATOM, map, fb, mn + q * 64, k + off);
                        } else {
                            tma_load_2d_pair(dst, map, fb, k, mn + off);
                        }
                    };
                    if constexpr (SPLIT == 0) {
                        if (!(ok = take()))
                            break;
                        if (!C::FEW || leader)
                            load(ma, A_MN, m, p.a_off[0], to);
                        load(mb, B_MN, n, p.b_off[0], to + C::A_BYTES);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (!(ok = take()))
                                break;
                            if (SPLIT == 2 ? (j & 1) != 0 : (j == 0) == (SPLIT == 3))
                                load(mb, B_MN, n, p.b_off[SPLIT == 2 ? j >> 1 : SPLIT == 3 ? 0 : 3 - j], to);
                            else
                                load(ma, A_MN, m, p.a_off[SPLIT == 2 ? 1 - (j >> 1) : SPLIT == 1 ? 0 : 3 - j], to);
                        }
                    }
                }
            }
            if (!ok) {
                if (leader) {
                    for (int st = 0; st < C::STAGES; ++st)
                        if ((issued >> st) & 1u)
                            mbar_drain(full_bar(st), (issued_parity >> st) & 1u);
                } else {
                    aborted_peer_loads = issued != 0;
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            // ------------------------------------------------------ MMA issuer
            int stage = 0;
            uint32_t phase = 0, ctr = 0;      // ctr: accumulators used so far
            bool ok = true;
            for (int u = pair; ok && u < sh.units; u += npairs) {
                const Unit t = unit_of(p, sh, u);
                for (int part = 0; ok && part < t.parts; ++part) {
                    const int kp = t.k0 + part * sh.part_blocks, ke = min(kp + sh.part_blocks, t.k1);
                    const uint32_t slot = ctr % PG_SLOTS, par = (ctr / PG_SLOTS) & 1u;
                    // (the peer's epilogue warps arrive here across the pair)
                    if (!mbar_wait_cluster(tempty0 + 8u * slot, par ^ 1u, abort_flag, limit)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + slot * 256;
                    // the next stage, once its bytes are there (0: gave up)
                    auto take = [&](int &st) {
                        st = stage;
                        if (!mbar_wait(full_bar(stage), phase, abort_flag, limit))
                            return false;
                        tc_fence_after();
                        if (++stage == C::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        return true;
                    };
                    auto multiply = [&](uint32_t a, uint32_t b, bool first) {
#pragma unroll
                        for (int kk = 0; kk < GEMM_BK / 16; ++kk)
                            // 16 K: 32 B along a K-major row, 2048 B (two 8-row atoms) of an MN-major operand
                            umma_bf16_pair(d,
                                           A_MN ? sdesc_mnmajor_sw128(a + kk * 2048, PG_ATOM)
                                                : sdesc_kmajor_sw128(a + kk * 32),
                                           B_MN ? sdesc_mnmajor_sw128(b + kk * 2048, PG_ATOM)
                                                : sdesc_kmajor_sw128(b + kk * 32),
                                           IDESC, (!first || kk > 0) ? 1u : 0u);
                    };
                    auto at = [&](int st) { return base + st * C::STAGE_BYTES; };
                    for (int kb = kp; ok && kb < ke; ++kb) {
                        int s0, s1, s2, s3;
                        if constexpr (SPLIT == 0) {
                            if (!(ok = take(s0)))
                                break;
                            multiply(at(s0), at(s0) + C::A_BYTES, kb == kp);
                            umma_commit_pair(empty_bar(s0), 0x3);     // both CTAs' stage is read
                        } else {
                            if (!(ok = take(s0) && take(s1)))
                                break;
                            if (SPLIT == 3)
                                multiply(at(s1), at(s0), kb == kp);   // A low, B
                            else
                                multiply(at(s0), at(s1), kb == kp);   // A middle, B high (A, B low)
                            umma_commit_pair(empty_bar(SPLIT == 2 ? s0 : s1), 0x3);
                            if (!(ok = take(s2)))
                                break;
                            if (SPLIT == 2)
                                multiply(at(s2), at(s1), false);      // A high, B high
                            else if (SPLIT == 3)
                                multiply(at(s2), at(s0), false);      // A middle, B
                            else
                                multiply(at(s0), at(s2), false);      // A, B middle
                            umma_commit_pair(empty_bar(SPLIT == 2 ? s1 : s2), 0x3);
                            if (!(ok = take(s3)))
                                break;
                            if (SPLIT == 2)
                                multiply(at(s2), at(s3), false);      // A high, B middle
                            else if (SPLIT == 3)
                                multiply(at(s3), at(s0), false);      // A high, B
                            else
                                multiply(at(s0), at(s3), false);      // A, B high
                            umma_commit_pair(empty_bar(SPLIT == 2 ? s2 : s0), 0x3);
                            umma_commit_pair(empty_bar(s3), 0x3);
                        }
                    }
                    if (ok) {
                        umma_commit_pair(tfull0 + 8u * slot, 0x3);    // accumulator ready in both TMEMs
                        ++ctr;
                    }
                }
            }
            umma_commit_pair(fin_bar, 0x1);
            mbar_drain(fin_bar, 0);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int ew = warp - 2, quad = warp & 3, half = ew >> 2;
        uint8_t *boxes = staging + ew * (C::BUFS * 4096);
        const uint32_t add_bar = add_bar0 + 8u * ew;
        const float scale = (EPI == PG_BF16 && p.meta) ? p.meta->scale : 1.0f;
        uint32_t ctr = 0, add_phase = 0;
        bool ok = true, add_pending = false;
        // waits for the next accumulator (the whole warp gets the answer)
        auto accumulator = [&]() {
            int got = 1;
            if (lane == 0)
                got = mbar_wait(tfull0 + 8u * (ctr % PG_SLOTS), (ctr / PG_SLOTS) & 1u, abort_flag, limit) ? 1 : 0;
            got = __shfl_sync(0xffffffffu, got, 0);
            __syncwarp();
            tc_fence_after();
            return got != 0;
        };
        auto tacc = [&]() {
            return tmem + ((uint32_t)(quad * 32) << 16) + (ctr % PG_SLOTS) * 256 + half * PG_HALF;
        };
        // gives the accumulator back to the MMA issuer, in the even CTA
        const uint32_t tempty_leader = mapa_shared(tempty0, 0);
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(tempty_leader + 8u * (ctr % PG_SLOTS));
            ++ctr;
        };
        // the addend's two boxes of unit u
        auto fetch_add = [&](int u) {
            if (lane == 0 && u < sh.units) {
                const Unit t = unit_of(p, sh, u);
                const int col = t.n0 + half * PG_HALF, row = t.m0 + rank * 128 + quad * 32;
                mbar_arrive_expect_tx(add_bar, 2 * 4096);
                tma_load_2d(smem_u32(boxes), &p.tmHidden, add_bar, col, row);
                tma_load_2d(smem_u32(boxes + 4096), &p.tmHidden, add_bar, col + 64, row);
                add_pending = true;
            }
        };
        if (EPI == PG_BF16_ADD)
            fetch_add(pair);
        for (int u = pair; ok && u < sh.units; u += npairs) {
            const Unit t = unit_of(p, sh, u);
            const int row0 = t.m0 + rank * 128 + quad * 32, col0 = t.n0 + half * PG_HALF;
            if constexpr (IS_STATS<EPI> || EPI == PG_PARTIAL) {
                uint32_t z[PG_HALF];
                if (t.parts == 0) {
#pragma unroll
                    for (int i = 0; i < PG_HALF; ++i)
                        z[i] = 0u;
                }
                for (int part = 0; part < t.parts; ++part) {
                    if (!accumulator()) {
                        ok = false;
                        break;
                    }
                    if (IS_STATS<EPI> && row0 >= sh.M) {
                        // (a short tile's empty rows)
                    } else if (part == 0) {
#pragma unroll
                        for (int c = 0; c < PG_HALF; c += 32)
                            tmem_load32(tacc() + c, z + c);
                    } else {
#pragma unroll
                        for (int c = 0; c < PG_HALF; c += 32) {
                            uint32_t r[32];
                            tmem_load32(tacc() + c, r);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                z[c + i] = __float_as_uint(__uint_as_float(z[c + i]) + __uint_as_float(r[i]));
                        }
                    }
                    release();
                }
                if (!ok)
                    break;
                if constexpr (IS_STATS<EPI>) {
                    if (row0 < sh.M)
                        epilogue_stats(p, sh, t, z, half, row0 + lane);
                } else
                    epilogue_partial(p, sh, t, z, half, row0, lane, boxes);
            } else {
                // (one part: the accumulator's values are used as they are)
                const bool empty = t.parts == 0;
                if (!empty && !accumulator()) {
                    ok = false;
                    break;
                }
                if constexpr (EPI == PG_BF16_ADD) {
                    int got = 1;
                    if (lane == 0) {
                        got = mbar_wait(add_bar, add_phase, abort_flag, limit) ? 1 : 0;
                        add_pending = got == 0;
                    }
                    got = __shfl_sync(0xffffffffu, got, 0);
                    __syncwarp();
                    if (!got) {
                        ok = false;
                        break;
                    }
                    add_phase ^= 1u;
                    uint4 v[2][8];
                    bf16_box<true>(tacc(), empty, 1.0f, boxes, lane, v[0]);
                    bf16_box<true>(tacc() + 64, empty, 1.0f, boxes + 4096, lane, v[1]);
                    if (!empty)
                        release();
                    __syncwarp();                // (every lane has read its row of the boxes)
                    fetch_add(u + npairs);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        store_box<false>(p, boxes + 2 * 4096, v[i], lane, col0 + 64 * i, row0 + p.out_row0);
                } else if constexpr (EPI == PG_BF16) {
                    uint4 v[2][8];
                    bf16_box<false>(tacc(), empty, scale, nullptr, lane, v[0]);
                    bf16_box<false>(tacc() + 64, empty, scale, nullptr, lane, v[1]);
                    if (!empty)
                        release();
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        store_box<false>(p, boxes, v[i], lane, col0 + 64 * i, row0 + p.out_row0);
                } else {
                    epilogue_dlogits(p, sh, t, tacc() - half * PG_HALF, half, row0 + lane, row0, lane, boxes);
                    release();
                }
            }
        }
        if (lane == 0) {
            if (EPI == PG_BF16_ADD && add_pending)
                mbar_drain(add_bar, add_phase);
            bulk_wait_group_all();              // this warp's output stores have completed
        }
    }

    __syncwarp();
    if (aborted_peer_loads) {
        // the leader's barrier counts this CTA's copies; give them time to land
        const unsigned long long t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 100000ull) {
        }
    }
    if (p.beside == PG_SECOND)
        pdl_wait();
    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, PG_TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag && p.status)
        atomicOr(p.status, ST_TIMEOUT);
}

template <int EPI, bool A_MN, bool B_MN, int SPLIT = 0>
cudaError_t launch_one(const PairGemmParams &p, int max_units, cudaStream_t s)
{
    auto kernel = pair_gemm_kernel<EPI, A_MN, B_MN, SPLIT>;
    static int configured_device = -1;
    static int max_clusters = 0;
    int dev = 0;
    cudaGetDevice(&dev);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.blockDim = dim3(PG_THREADS);
    cfg.dynamicSmemBytes = PgCfg<EPI, SPLIT>::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (configured_device != dev) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PgCfg<EPI, SPLIT>::SMEM);
        if (e != cudaSuccess)
            return e;
        cfg.gridDim = dim3(2);
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess)
            return e;
        if (n < 1)
            return cudaErrorInvalidConfiguration;
        max_clusters = n;
        configured_device = dev;
    }
    cfg.gridDim = dim3(2 * std::max(1, std::min(max_units, max_clusters)));
    const cudaError_t le = cudaLaunchKernelEx(&cfg, kernel, p);
    return le != cudaSuccess ? le : cudaPeekAtLastError();
}

}  // namespace

// max_units: tiles times splits if every row counts
cudaError_t launch_pair_gemm(PairEpilogue epi, PairProduct product, const PairGemmParams &p, int max_units,
                             cudaStream_t s)
{
    switch (product) {
    case PP_LOGITS:
        if (epi == PG_STATS)
            return launch_one<PG_STATS, false, false>(p, max_units, s);
        if (epi == PG_STATS_FEW)
            return launch_one<PG_STATS_FEW, false, false>(p, max_units, s);
        if (epi == PG_DLOGITS)
            return launch_one<PG_DLOGITS, false, false>(p, max_units, s);
        break;
    case PP_DX:
        if (epi == PG_PARTIAL)
            return launch_one<PG_PARTIAL, false, true>(p, max_units, s);
        break;
    case PP_DW:
        if (epi == PG_BF16)
            return launch_one<PG_BF16, true, true>(p, max_units, s);
        break;
    case PP_LOGITS_PARTS:
        if (epi == PG_PARTIAL)
            return launch_one<PG_PARTIAL, false, false, 1>(p, max_units, s);
        break;
    case PP_DX_PARTS:
        if (epi == PG_BF16)
            return launch_one<PG_BF16, false, true, 2>(p, max_units, s);
        if (epi == PG_BF16_ADD)
            return launch_one<PG_BF16_ADD, false, true, 2>(p, max_units, s);
        break;
    case PP_DW_PARTS:
        if (epi == PG_PARTIAL)
            return launch_one<PG_PARTIAL, true, true, 3>(p, max_units, s);
        break;
    }
    return cudaErrorInvalidValue;
}

}  // namespace glr
