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
// Roles (192 threads): warp 0 lane 0 loads, warp 1 lane 0 of the even CTA
// issues the MMAs (of the odd one, forwards its epilogue's arrivals to the
// even one), warps 2..5 run the epilogue on the TMEM lanes 32 (w % 4) .. + 31.
// Every wait is bounded; when one runs out, every role leaves its loop, copies
// in flight are waited for (bounded), TMEM is freed and the status word gets
// MOE_STATUS_TIMEOUT.
#include <cuda_bf16.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace glr {

namespace {

constexpr int PG_THREADS = 64 + 32 * 4;
constexpr int PG_BM = 256, PG_BN = 256;          // a pair's tile
constexpr float LOG2E = 1.44269504088896341f;

struct PgCfg {
    static constexpr int ATOM = 64 * GEMM_BK * 2;            // 64 x 64 bf16, 8 KB
    static constexpr int A_BYTES = 2 * ATOM, B_BYTES = 2 * ATOM;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = 6;
    static constexpr int SLOTS = 2;
    static constexpr int TMEM_COLS = 512;
    static constexpr int STAGING = 2 * 4 * 4096;             // two 4 KB buffers per epilogue warp
    static constexpr int NBARS = 2 * STAGES + 2 * SLOTS + 1;
    static constexpr int SMEM = STAGES * STAGE_BYTES + STAGING + 1024 /*align*/ + NBARS * 8 + 16;
    static_assert(SMEM <= 232448, "more than 227 KB of shared memory");
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

// One unit of work: a tile and its K blocks (the same range of every segment).
struct Unit {
    int m0, n0, nt, split;
    int k0, k1;              // blocks of each segment
};

struct Shape {
    int M, m_tiles, n_tiles, kblocks, units;
};

__device__ __forceinline__ Shape shape_of(const PairGemmParams &p)
{
    Shape sh;
    const int rows = p.meta ? p.meta->rows : 0;
    sh.M = p.m_from_rows ? rows : p.M;
    sh.kblocks = p.k_from_rows ? (rows + GEMM_BK - 1) / GEMM_BK : p.kblocks;
    sh.m_tiles = (sh.M + PG_BM - 1) / PG_BM;
    sh.n_tiles = (p.N + PG_BN - 1) / PG_BN;
    sh.units = sh.m_tiles * sh.n_tiles * p.splits;
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
    t.k0 = (int)((long long)sh.kblocks * t.split / p.splits);
    t.k1 = (int)((long long)sh.kblocks * (t.split + 1) / p.splits);
    return t;
}

// This warp's 32 rows x 128 bytes (lane = row, eight 16-byte pieces in v) to
// the output map, through one of the warp's two staging buffers.  Boxes
// outside the map are skipped; TMA clips those that cross its edge.
template <bool ADD>
__device__ __forceinline__ void store_box(const PairGemmParams &p, uint8_t *stage2, int &buf, const uint4 (&v)[8],
                                          int lane, int col, int row)
{
    uint8_t *stage = stage2 + buf * 4096;
    if (lane == 0)
        bulk_wait_group_read<1>();              // the store before the last has left this buffer
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q)
        *reinterpret_cast<uint4 *>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) = v[q];
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (col < p.out_cols && row < p.out_rows) {
            if (ADD)
                tma_reduce_add_2d(&p.tmOut, smem_u32(stage), col, row);
            else
                tma_store_2d(&p.tmOut, smem_u32(stage), col, row);
        }
        bulk_commit_group();
    }
    buf ^= 1;
}

// Softmax statistics of this lane's row over the tile's columns: a base b (in
// log2) and s = sum 2^(z log2 e - b), 64 columns at a time, s rescaled when a
// later 64 hold a larger value.  b is finite even when the largest logit is
// not, so that an infinite or NaN logit shows in s.
__device__ __forceinline__ void epilogue_stats(const PairGemmParams &p, const Shape &sh, const Unit &t, uint32_t tacc,
                                               int row)
{
    const bool valid = row < sh.M;
    const int rel = valid ? p.target[row] - (p.n0 + t.n0) : -1;
    const int ncols = min(PG_BN, p.N - t.n0);
    float b = -INFINITY, s = 0.0f, zt = 0.0f;
    bool found = false;
#pragma unroll 1
    for (int c = 0; c < ncols; c += 64) {
        uint32_t r[64];
        tmem_load64(tacc + c, r);
        if (ncols - c < 64)
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (i >= ncols - c)
                    r[i] = 0xff800000u;
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
            m0 = fmaxf(m0, __uint_as_float(r[i]));
            m1 = fmaxf(m1, __uint_as_float(r[i + 1]));
        }
        float base = fmaxf(b, fmaxf(m0, m1) * LOG2E);
        if (!(fabsf(base) < INFINITY))
            base = 0.0f;
        float s0 = s * ex2_approx(b - base), s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
            s0 += ex2_approx(fmaf(__uint_as_float(r[i]), LOG2E, -base));
            s1 += ex2_approx(fmaf(__uint_as_float(r[i + 1]), LOG2E, -base));
        }
        s = s0 + s1;
        b = base;
        const int at = rel - c;
        if (__any_sync(0xffffffffu, at >= 0 && at < 64)) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (at == i) {
                    zt = __uint_as_float(r[i]);
                    found = true;
                }
        }
    }
    if (valid) {
        p.stats[(size_t)t.nt * p.ld_stats + row] = make_float2(b, s);
        if (found)
            p.target_logit[row] = zt;
    }
}

// dz of the tile in bf16, 64 columns at a time.  The rounding (half a step,
// 2^-8 of each value) makes dz an operand of the tensor core; the rows' weights
// are divided by the largest of them first, so that a mean's equal weights
// are 1 exactly and add no rounding of their own, common to every value.
__device__ __forceinline__ void epilogue_dlogits(const PairGemmParams &p, const Shape &sh, const Unit &t,
                                                 uint32_t tacc, int row, int row0, int lane, uint8_t *stage, int &buf)
{
    const bool valid = row < sh.M;
    const int rel = valid ? p.target[row] - (p.n0 + t.n0) : -1;
    const float nl = valid ? -p.lse[row] * LOG2E : 0.0f;
    const float w = valid ? p.weight[row] : 0.0f;
    const int ncols = min(PG_BN, p.N - t.n0);
#pragma unroll 1
    for (int c = 0; c < PG_BN; c += 64) {
        if (c >= ncols)
            break;
        uint32_t r[64];
        tmem_load64(tacc + c, r);
        const int at = rel - c;
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
            f[i] = valid && i < ncols - c ? f[i] * w : 0.0f;
        uint4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            v[q] = make_uint4(bf16x2(f[8 * q], f[8 * q + 1]), bf16x2(f[8 * q + 2], f[8 * q + 3]),
                              bf16x2(f[8 * q + 4], f[8 * q + 5]), bf16x2(f[8 * q + 6], f[8 * q + 7]));
        store_box<false>(p, stage, buf, v, lane, t.n0 + c, row0);
    }
}

// fp32 tile into the split's slice.  Each element is stored or added to once
// per launch, so the sums' order is that of the launches.
__device__ __forceinline__ void epilogue_partial(const PairGemmParams &p, const Unit &t, uint32_t tacc, bool empty,
                                                 int row0, int lane, uint8_t *stage, int &buf)
{
    const int ncols = min(PG_BN, p.N - t.n0);
#pragma unroll 1
    for (int c = 0; c < ncols; c += 32) {
        uint32_t r[32];
        if (empty) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                r[i] = 0u;
        } else {
            tmem_load32(tacc + c, r);
        }
        uint4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            v[q] = make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
        const int row = t.split * p.split_rows + row0;
        if (p.accumulate)
            store_box<true>(p, stage, buf, v, lane, t.n0 + c, row);
        else
            store_box<false>(p, stage, buf, v, lane, t.n0 + c, row);
    }
}

// bf16 tile, scaled, with an optional bf16 addend; one rounding.
__device__ __forceinline__ void epilogue_bf16(const PairGemmParams &p, const Unit &t, uint32_t tacc, bool empty,
                                              int row, int row0, int lane, uint8_t *stage, int &buf)
{
    const int ncols = min(PG_BN, p.N - t.n0);
    const float scale = p.meta ? p.meta->scale : 1.0f;
    const bool has_add = p.add && row < p.out_rows;
#pragma unroll 1
    for (int c = 0; c < ncols; c += 64) {
        uint32_t r[64];
        if (empty) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
                r[i] = 0u;
        } else {
            tmem_load64(tacc + c, r);
        }
        uint4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = __uint_as_float(r[8 * q + i]) * scale;
            if (has_add && c + 8 * q < ncols) {           // (N is a multiple of 8)
                const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p.add + (size_t)row * p.N + t.n0 + c + 8 * q));
                const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[2 * i] += __uint_as_float(w[i] << 16);
                    f[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
                }
            }
            v[q] = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
        }
        store_box<false>(p, stage, buf, v, lane, t.n0 + c, row0 + p.out_row0);
    }
}

template <int EPI, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(PG_THREADS, 1) pair_gemm_kernel(const __grid_constant__ PairGemmParams p)
{
    using C = PgCfg;
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
    const uint32_t tempty0 = tfull0 + 8u * C::SLOTS;
    const uint32_t fin_bar = tempty0 + 8u * C::SLOTS;

    if (threadIdx.x == 0) {
        for (int st = 0; st < C::STAGES; ++st) {
            mbar_init(full_bar(st), 1);
            mbar_init(empty_bar(st), 1);
        }
        for (int a = 0; a < C::SLOTS; ++a) {
            mbar_init(tfull0 + 8u * a, 1);
            // this CTA's epilogue warps; the leader's also counts the peer's forwarder
            mbar_init(tempty0 + 8u * a, 4 + (leader ? 1 : 0));
        }
        mbar_init(fin_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_map(&p.tmA);
        tma_prefetch_map(&p.tmB);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_holder), C::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();            // both CTAs' barriers initialised and TMEM allocated
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_wait();                // operands and row counts come from earlier kernels

    const int npairs = (int)gridDim.x / 2;
    const int pair = (int)blockIdx.x / 2;
    const Shape sh = shape_of(p);
    const bool packed = p.meta && p.meta->rows < p.T;
    bool aborted_peer_loads = false;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- TMA producer
            const CUtensorMap *ma = (packed && (EPI == PG_STATS || EPI == PG_DLOGITS)) ? &p.tmHidden : &p.tmA;
            const CUtensorMap *mb = (packed && EPI == PG_BF16) ? &p.tmHidden : &p.tmB;
            const uint32_t full_leader0 = mapa_shared(full_bar(0), 0);
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_parity = 0;
            bool ok = true;
            for (int u = pair; ok && u < sh.units; u += npairs) {
                const Unit t = unit_of(p, sh, u);
                const int m = t.m0 + rank * 128, n = t.n0 + rank * 128;
                for (int seg = 0; ok && seg < p.nseg; ++seg) {
                    for (int kb = t.k0; kb < t.k1; ++kb) {
                        if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag)) {
                            ok = false;
                            break;
                        }
                        const uint32_t sA = base + stage * C::STAGE_BYTES, sB = sA + C::A_BYTES;
                        if (leader)
                            mbar_arrive_expect_tx(full_bar(stage), 2 * C::STAGE_BYTES);
                        const uint32_t fb = full_leader0 + 8u * stage;
                        const int k = kb * GEMM_BK;
                        if (A_MN) {
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                tma_load_2d_pair(sA + q * C::ATOM, ma, fb, m + q * 64, k + p.a_off[seg]);
                        } else {
                            tma_load_2d_pair(sA, ma, fb, k, m + p.a_off[seg]);
                        }
                        if (B_MN) {
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                tma_load_2d_pair(sB + q * C::ATOM, mb, fb, n + q * 64, k + p.b_off[seg]);
                        } else {
                            tma_load_2d_pair(sB, mb, fb, k, n + p.b_off[seg]);
                        }
                        issued |= 1u << stage;
                        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                        if (++stage == C::STAGES) {
                            stage = 0;
                            phase ^= 1u;
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
                const int nkb = (t.k1 - t.k0) * p.nseg;
                if (nkb == 0)
                    continue;
                const uint32_t slot = ctr % C::SLOTS, par = (ctr / C::SLOTS) & 1u;
                // (the peer's forwarder arrives here across the pair)
                if (!mbar_wait_cluster(tempty0 + 8u * slot, par ^ 1u, abort_flag))
                    break;
                tc_fence_after();
                const uint32_t d = tmem + slot * 256;
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!mbar_wait(full_bar(stage), phase, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sA = base + stage * C::STAGE_BYTES, sB = sA + C::A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < GEMM_BK / 16; ++kk)
                        // 16 K: 32 B along a K-major row, 2048 B (two 8-row atoms) of an MN-major operand
                        umma_bf16_pair(d,
                                       A_MN ? sdesc_mnmajor_sw128(sA + kk * 2048, C::ATOM)
                                            : sdesc_kmajor_sw128(sA + kk * 32),
                                       B_MN ? sdesc_mnmajor_sw128(sB + kk * 2048, C::ATOM)
                                            : sdesc_kmajor_sw128(sB + kk * 32),
                                       IDESC, (kb > 0 || kk > 0) ? 1u : 0u);
                    umma_commit_pair(empty_bar(stage), 0x3);          // both CTAs' stage is read
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) {
                    umma_commit_pair(tfull0 + 8u * slot, 0x3);        // accumulator ready in both TMEMs
                    ++ctr;
                }
            }
            umma_commit_pair(fin_bar, 0x1);
            mbar_drain(fin_bar, 0);
        } else if (lane == 0) {
            // ------------------------------------------- the peer's forwarder
            const uint32_t tempty_leader = mapa_shared(tempty0, 0);
            uint32_t ctr = 0;
            for (int u = pair; u < sh.units; u += npairs) {
                const Unit t = unit_of(p, sh, u);
                if (t.k0 == t.k1)
                    continue;
                const uint32_t slot = ctr % C::SLOTS, par = (ctr / C::SLOTS) & 1u;
                if (!mbar_wait(tempty0 + 8u * slot, par, abort_flag))
                    break;
                mbar_arrive_cluster(tempty_leader + 8u * slot);
                ++ctr;
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int quad = warp & 3;
        uint8_t *stage = staging + (warp - 2) * (2 * 4096);
        int buf = 0;
        uint32_t ctr = 0;
        for (int u = pair; u < sh.units; u += npairs) {
            const Unit t = unit_of(p, sh, u);
            const bool empty = t.k0 == t.k1;
            const uint32_t slot = ctr % C::SLOTS, par = (ctr / C::SLOTS) & 1u;
            if (!empty) {
                int ok = 1;
                if (lane == 0)
                    ok = mbar_wait(tfull0 + 8u * slot, par, abort_flag) ? 1 : 0;
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok)
                    break;
                __syncwarp();
                tc_fence_after();
            }
            const uint32_t tacc = tmem + ((uint32_t)(quad * 32) << 16) + slot * 256;
            const int row0 = t.m0 + rank * 128 + quad * 32;
            if (EPI == PG_STATS)
                epilogue_stats(p, sh, t, tacc, row0 + lane);
            else if (EPI == PG_DLOGITS)
                epilogue_dlogits(p, sh, t, tacc, row0 + lane, row0, lane, stage, buf);
            else if (EPI == PG_PARTIAL)
                epilogue_partial(p, t, tacc, empty, row0, lane, stage, buf);
            else
                epilogue_bf16(p, t, tacc, empty, row0 + lane, row0, lane, stage, buf);
            if (!empty) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(tempty0 + 8u * slot);   // (the peer's forwarder passes it on to the leader)
                ++ctr;
            }
        }
        if (lane == 0)
            bulk_wait_group_all();              // this warp's output stores have completed
    }

    __syncwarp();
    if (aborted_peer_loads) {
        // the leader's barrier counts this CTA's copies; give them time to land
        const unsigned long long t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 100000ull) {
        }
    }
    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, C::TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag && p.status)
        atomicOr(p.status, ST_TIMEOUT);
}

template <int EPI, bool A_MN, bool B_MN>
cudaError_t launch_one(const PairGemmParams &p, int max_units, cudaStream_t s)
{
    auto kernel = pair_gemm_kernel<EPI, A_MN, B_MN>;
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
    cfg.dynamicSmemBytes = PgCfg::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (configured_device != dev) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PgCfg::SMEM);
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
cudaError_t launch_pair_gemm(PairEpilogue epi, bool a_mn, bool b_mn, const PairGemmParams &p, int max_units,
                             cudaStream_t s)
{
    if (epi == PG_STATS && !a_mn && !b_mn)
        return launch_one<PG_STATS, false, false>(p, max_units, s);
    if (epi == PG_DLOGITS && !a_mn && !b_mn)
        return launch_one<PG_DLOGITS, false, false>(p, max_units, s);
    if (epi == PG_PARTIAL && !a_mn && b_mn)
        return launch_one<PG_PARTIAL, false, true>(p, max_units, s);
    if (epi == PG_PARTIAL && a_mn && b_mn)
        return launch_one<PG_PARTIAL, true, true>(p, max_units, s);
    if (epi == PG_BF16 && !a_mn && b_mn)
        return launch_one<PG_BF16, false, true>(p, max_units, s);
    if (epi == PG_BF16 && a_mn && b_mn)
        return launch_one<PG_BF16, true, true>(p, max_units, s);
    return cudaErrorInvalidValue;
}

}  // namespace glr
