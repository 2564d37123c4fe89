// Matrix products of 8-bit operands with a scale for each 128 of the sum
// (tcgen05 kind::mxf8f6f4 with block scales, TMEM accumulators, TMA):
//
//   out[m, n] = sum_b sA[b, m] sB[b, n] sum_{k in block b} A[m, k] B[n, k]
//
// dense; with the rows of A grouped (sorted by expert) and a B for each group; or
// with the sum grouped (the gradient of each expert's weight).
//
// The scales are powers of two, which the tensor core applies itself while it
// multiplies: it wants them in TMEM, a 32-bit word for each row, of which the
// instruction names one byte.  A block of 128 has one scale, so the four MMAs of a
// block name the same byte and a word serves four blocks.  Four warps fetch the
// scale bytes of four blocks from shared memory and write their words to TMEM
// (tcgen05.st) in the layout of the MMA: row r in lane r % 32 (the same in all four
// lane quarters), column r / 32.
//
// Tiles: 256 rows and 256 or 224 columns on a pair of CTAs (cta_group::2), where each
// loads its 128 rows of A and half of B's; or 128 x 128 or 64 on one CTA.  There are
// two accumulators, so that a tile's epilogue runs beside the next one's MMAs.  With
// 256 columns they and the scales do not fit into TMEM's 512 side by side: they
// overlap by 64 columns, which the epilogue empties first and hands back at once.
//
// The scales have rings of their own in shared memory and in TMEM, four blocks to a
// slot, and run well ahead of the operands: a write to TMEM and its handshake take
// more than a thousand cycles while MMAs run, an operand stage's MMAs 550.  With words of
// four equal bytes, one for each stage, in the operands' ring a pair reached 2910 TFLOP/s
// (8192 x 8192 x 8192), with words of four blocks on this ring 3020, all else alike.
//
// The tensor core cuts its running sum to fp32 instead of rounding it, so it drifts
// towards zero as it grows: by 4e-6 over 8192 of K of one sign, 2.4e-5 over 32768.
// Where the result stays fp32, K is therefore cut into parts of 2048 with an
// accumulator each, which the epilogue adds in the output, rounding to nearest
// (5e-7).
//
// Roles: warp 0 lane 0 loads operands, warp 1 lane 0 (of the pair's even CTA)
// issues the MMAs, warp 2 lane 0 loads scales, warps 4 to 7 write them to TMEM, the
// rest store the output.
// Every wait is bounded; when one runs out, every role leaves its loop, copies in
// flight are waited for (bounded), TMEM is freed and the status word gets
// MOE_STATUS_TIMEOUT.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "expert_ops.h"
#include "kernels.h"
#include "ptx.cuh"

namespace glr {

namespace {

constexpr int SG_BM = 128, SG_BK = 128;            // a CTA's rows of A, K per stage
constexpr int SG_TMEM_COLS = 512, SG_SCALE_COL = 448;
constexpr int SG_CHUNK = SCALED_CHUNK;             // blocks of 128 whose scales come at once
constexpr int SG_CHUNKS = 4;                       // slots for them in shared memory
static_assert(SG_CHUNK == 4, "a byte of a word for each block");

// F32: fp32 output, which leaves through shared memory.
template <int BN, bool PAIR, bool F32>
struct SgCfg {
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int A_BYTES = SG_BM * SG_BK, B_ROWS = BN / CTAS, B_BYTES = B_ROWS * SG_BK;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int SA_BOX = SCALED_SA_BOX * SG_CHUNK, SB_BOX = BN * SG_CHUNK;
    static constexpr int SA_BYTES = (SA_BOX + 127) / 128 * 128, SB_BYTES = SB_BOX;
    static constexpr int SCALE_BYTES = SA_BYTES + SB_BYTES;
    static constexpr int SCALE_COLS = (4 + BN / 32 + 3) / 4 * 4;         // TMEM columns of a slot: 4 and BN / 32
    static constexpr int SLOTS = (SG_TMEM_COLS - SG_SCALE_COL) / SCALE_COLS;
    static constexpr int EPI_WARPS = 8, EPI_WARP0 = 8;
    static constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
    static constexpr int BOXES = F32 ? EPI_WARPS * 4096 : 0;
    static constexpr int MOST_STAGES = 8;
    static constexpr int PART = F32 ? 16 : 1 << 24;                      // blocks of 128 in an accumulator at most (fp32)
    static constexpr int REST = BOXES + SG_CHUNKS * SCALE_BYTES + 1024 /*align*/ +
                                (2 * MOST_STAGES + 2 * SLOTS + 2 * SG_CHUNKS + 5) * 8 + 16 + (SCALED_MAX_E + 1) * 4;
    static constexpr int FIT = (232448 - REST) / STAGE_BYTES;
    static constexpr int STAGES = FIT < MOST_STAGES ? FIT : MOST_STAGES;
    static constexpr int NBARS = 2 * STAGES + 2 * SLOTS + 2 * SG_CHUNKS + 2 + 2 + 1;
    static constexpr int SMEM = STAGES * STAGE_BYTES + REST;
    static_assert(SMEM <= 232448 && STAGES >= 4, "shared memory");
    static constexpr int SLOT_STEP = BN == 256 ? 192 : BN;               // TMEM columns between the two accumulators
    static constexpr bool OVERLAP = SLOT_STEP < BN;
    static_assert(SLOT_STEP + BN <= SG_SCALE_COL, "accumulators over the scales");
    static_assert(BN % 32 == 0 && B_BYTES % 1024 == 0, "swizzle atoms need 1024-B alignment");
    static_assert(SA_BYTES % 128 == 0 && SCALE_BYTES % 128 == 0, "TMA boxes on 128-byte boundaries");
};

// kind::mxf8f6f4, scales in bytes 2^(b - 127); K-major operands
__host__ __device__ constexpr uint32_t idesc_scaled(int M, int N, bool a_e5m2, bool b_e5m2)
{
    return ((a_e5m2 ? 1u : 0u) << 7) | ((b_e5m2 ? 1u : 0u) << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
           ((uint32_t)(M >> 4) << 24);
}

// The low words of two K-major, 128-byte-swizzled operands' descriptors (the high
// ones are constant); `first`: the accumulator starts from zero.
constexpr uint32_t SG_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | (1u << 16); }

template <bool PAIR>
__device__ __forceinline__ void umma_scaled(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                            uint32_t accumulate)
{
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %7};\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], da, db, %3, [%5], [%6], p;\n\t}\n"
            ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb), "n"(SG_DESC_HI)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %7};\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], da, db, %3, [%5], [%6], p;\n\t}\n"
            ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb), "n"(SG_DESC_HI)
            : "memory");
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t pred;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(pred));
    return pred != 0;
}

// N words of each of this warp's 32 TMEM lanes (no wait)
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t *r)
{
    if constexpr (N >= 4) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                     "r"(r[2]), "r"(r[3])
                     : "memory");
        tmem_store<N - 4>(taddr + 4, r + 4);
    } else if constexpr (N >= 2) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(r[0]), "r"(r[1]) : "memory");
        tmem_store<N - 2>(taddr + 2, r + 2);
    } else if constexpr (N == 1) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r[0]) : "memory");
    }
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(uint32_t lo, uint32_t hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// One tile of work: output rows m0 .. (of the tensor), those below m_end exist,
// columns n0 .. below N.
struct Tile {
    int a_row, m_end, out_row;      // first row of A; first row past the tile's in the output; output row
    int n0, b_row, sb_row0;         // B: first row of the map, first row of its scales' map
    int k0, k1;                     // blocks of 128
};

// Walks the tiles u = first, first + step, .. in order (groups come in order too).
template <int BM, int BN>
struct Tiles {
    const ScaledGemmParams &p;
    const int *pre;                 // [E + 1] tiles of the groups before, in units of n-tiles (SM_ROWS)
    int n_tiles, m_tiles, total, e;
    __device__ Tiles(const ScaledGemmParams &p_, const int *pre_) : p(p_), pre(pre_), e(0)
    {
        n_tiles = (p.N + BN - 1) / BN;
        m_tiles = (p.M + BM - 1) / BM;
        total = p.mode == SM_ROWS ? pre[p.E] * n_tiles : m_tiles * n_tiles * (p.mode == SM_SUM && p.E ? p.E : 1);
    }
    __device__ __forceinline__ int bound(int i, int most) const { return min(max(p.bounds[i], 0), most); }
    __device__ Tile at(int u)
    {
        Tile t;
        int g = 0, mt, nt;
        if (p.mode == SM_ROWS) {
            while (u >= pre[e + 1] * n_tiles)
                ++e;
            g = e;
            const int mine = pre[e + 1] - pre[e], in = u - pre[e] * n_tiles;
            mt = in % mine;
            nt = in / mine;
            const int a = bound(g, p.M), b = bound(g + 1, p.M);
            t.a_row = a + mt * BM;
            t.m_end = b;
            t.out_row = t.a_row;
        } else {
            g = u / (m_tiles * n_tiles);
            const int tile = u - g * m_tiles * n_tiles, per = p.band * n_tiles;
            const int b0 = tile / per, in = tile - b0 * per, rows = min(p.band, m_tiles - b0 * p.band);
            nt = in / rows;
            mt = b0 * p.band + in - nt * rows;
            t.a_row = mt * BM;
            t.out_row = (p.mode == SM_SUM ? g * p.M : 0) + t.a_row;
            t.m_end = t.out_row - t.a_row + p.M;
        }
        t.n0 = nt * BN;
        t.b_row = (p.mode == SM_ROWS ? g * p.N : 0) + t.n0;
        t.k0 = 0;
        t.k1 = p.kblocks;
        if (p.mode == SM_SUM && p.E) {
            t.k0 = bound(g, p.kblocks);
            t.k1 = max(t.k0, bound(g + 1, p.kblocks));
        }
        t.sb_row0 = p.mode == SM_ROWS ? g * p.kblocks : 0;
        return t;
    }
};

// pre[e] = row tiles of the groups before e (one warp)
template <int BM>
__device__ __forceinline__ void count_tiles(const ScaledGemmParams &p, int *pre, int lane)
{
    int run = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        int n = 0;
        if (e < p.E) {
            const int a = min(max(p.bounds[e], 0), p.M), b = min(max(p.bounds[e + 1], 0), p.M);
            n = (max(b - a, 0) + BM - 1) / BM;
        }
        int incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off)
                incl += y;
        }
        if (e < p.E)
            pre[e] = run + incl - n;
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0)
        pre[p.E] = run;
}

// 32 accumulator columns (from TMEM column `acc`; zeros without) of a warp's 32 rows
// (lane = row) to the output; read() is called when they have left TMEM.  `add`: to what
// the part of K before left there (fp32; the same lane wrote it).
// bf16 goes straight from registers, 32 bytes, a whole sector, per lane and store where
// the rows allow it (`wide`), else 16: shared memory is busy with operands.  fp32, whose
// products write more than they read, passes through the warp's 4 KB box, so that
// eight lanes write a row's 128 bytes: 256 weight gradients of 1024 x 2048 over 65536
// rows took 392 us, 475 from registers and 460 through TMA (box by box).
template <bool F32, typename Read>
__device__ __forceinline__ void store_piece(const ScaledGemmParams &p, uint32_t acc, bool empty, bool add, uint8_t *box,
                                            int col, int row0, int m_end, int lane, Read read)
{
    uint32_t z[32];
    if (empty) {
#pragma unroll
        for (int q = 0; q < 32; ++q)
            z[q] = 0u;
    } else {
        tmem_load32(acc, z);
    }
    read();
    if (row0 >= m_end || col >= p.N)
        return;
    if (F32) {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4 *>(box + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                make_uint4(z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]);
        __syncwarp();
        const int piece = lane & 7, r0 = lane >> 3, c = col + 4 * piece;
        float *dst = static_cast<float *>(p.out) + (size_t)(row0 + r0) * p.N + c;
        const size_t step = (size_t)4 * p.N;
        const int rows = c < p.N ? m_end - row0 - r0 : 0;        // 4 i below it exist
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = 4 * i + r0;
            v[i] = *reinterpret_cast<const float4 *>(box + row * 128 + ((piece ^ (row & 7)) << 4));
        }
        if (add) {
            float4 o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (4 * i < rows)
                    o[i] = *reinterpret_cast<const float4 *>(dst + i * step);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = make_float4(o[i].x + v[i].x, o[i].y + v[i].y, o[i].z + v[i].z, o[i].w + v[i].w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (4 * i < rows)
                *reinterpret_cast<float4 *>(dst + i * step) = v[i];
        return;
    }
    const int row = row0 + lane;
    if (row >= m_end)
        return;
    uint8_t *dst = static_cast<uint8_t *>(p.out) + ((size_t)row * p.N + col) * 2;
#pragma unroll
    for (int q = 0; q < 2; ++q) {                    // 16 columns each
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = pack_bf16(z[16 * q + 2 * i], z[16 * q + 2 * i + 1]);
        const int c = col + 16 * q;
        if (p.wide) {
            if (c < p.N)
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 32 * q), "r"(v[0]),
                             "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                             : "memory");
        } else {
            if (c < p.N)
                *reinterpret_cast<uint4 *>(dst + 32 * q) = make_uint4(v[0], v[1], v[2], v[3]);
            if (c + 8 < p.N)
                *reinterpret_cast<uint4 *>(dst + 32 * q + 16) = make_uint4(v[4], v[5], v[6], v[7]);
        }
    }
}

template <int BN, bool PAIR, bool F32>
__global__ void __launch_bounds__(SgCfg<BN, PAIR, F32>::THREADS) scaled_gemm_kernel(const __grid_constant__ ScaledGemmParams p)
{
    using C = SgCfg<BN, PAIR, F32>;
    constexpr int BM = SG_BM * C::CTAS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t base = smem_u32(smem);
    uint8_t *boxes = smem + C::STAGES * C::STAGE_BYTES;
    uint8_t *scales = boxes + C::BOXES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(scales + SG_CHUNKS * C::SCALE_BYTES);
    const uint32_t bar0 = smem_u32(bars);
    // of a pair, the even CTA's: full (both CTAs' operands), scaled (scales in both
    // TMEMs), tempty; each CTA has its own of the others (used: a slot of scales)
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
    auto scaled_bar = [&](int s) { return bar0 + 8u * (2 * C::STAGES + s); };
    auto used_bar = [&](int s) { return bar0 + 8u * (2 * C::STAGES + C::SLOTS + s); };
    auto sload_bar = [&](int s) { return bar0 + 8u * (2 * C::STAGES + 2 * C::SLOTS + s); };
    auto sfree_bar = [&](int s) { return bar0 + 8u * (2 * C::STAGES + 2 * C::SLOTS + SG_CHUNKS + s); };
    const uint32_t tfull0 = bar0 + 8u * (2 * C::STAGES + 2 * C::SLOTS + 2 * SG_CHUNKS), tempty0 = tfull0 + 16, fin_bar = tempty0 + 16;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + C::NBARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *pre = reinterpret_cast<int *>(tmem_holder + 2);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_ctarank() : 0;
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int s = 0; s < C::SLOTS; ++s) {
            mbar_init(scaled_bar(s), 4 * C::CTAS);
            mbar_init(used_bar(s), 1);
        }
        for (int s = 0; s < SG_CHUNKS; ++s) {
            mbar_init(sload_bar(s), 1);
            mbar_init(sfree_bar(s), 4);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull0 + 8u * a, 1);
            mbar_init(tempty0 + 8u * a, C::EPI_WARPS * C::CTAS);
        }
        mbar_init(fin_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_map(&p.tmA);
        tma_prefetch_map(&p.tmB);
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(smem_u32(tmem_holder), SG_TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tmem_holder), SG_TMEM_COLS);
            tmem_relinquish();
        }
    }
    pdl_wait();
    if (p.mode == SM_ROWS && warp == 0)
        count_tiles<BM>(p, pre, lane);
    tc_fence_before();
    if (PAIR)
        cluster_sync();              // both CTAs' barriers initialised and TMEM allocated
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const unsigned long long limit = p.wait_limit_ns ? p.wait_limit_ns : WAIT_LIMIT_NS;
    const int first = (int)blockIdx.x / C::CTAS, step = (int)gridDim.x / C::CTAS;
    Tiles<BM, BN> tiles(p, pre);
    // the accumulator of tile number i (of this CTA's or pair's)
    auto acc_col = [&](uint32_t i) { return tmem + (i & 1u) * C::SLOT_STEP; };
    // An arrival at a barrier of the even CTA.  It hands over TMEM, whose accesses have
    // completed before it (wait::st, wait::ld), and no memory, so it needs no release
    // at cluster scope.  With one: 8192 x 8192 x 8192 2990 TFLOP/s instead of 3400, 65536 x
    // 2048 x 1024 1840 instead of 2520.
    auto arrive_leader = [&](uint32_t bar) {
        if (PAIR)
            asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(bar, 0)) : "memory");
        else
            mbar_arrive(bar);
    };
    // ... and a wait there for both CTAs' threads
    auto wait_both = [&](uint32_t bar, uint32_t parity) {
        return PAIR ? mbar_wait_cluster(bar, parity, abort_flag, limit) : mbar_wait(bar, parity, abort_flag, limit);
    };
    // a wait of a whole warp
    auto warp_wait = [&](uint32_t bar, uint32_t parity) {
        int got = 1;
        if (lane == 0)
            got = mbar_wait(bar, parity, abort_flag, limit) ? 1 : 0;
        return __shfl_sync(0xffffffffu, got, 0) != 0;
    };
    bool aborted_peer_loads = false;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------- operands
            const uint32_t full_leader0 = PAIR ? mapa_shared(full_bar(0), 0) : full_bar(0);
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_parity = 0;
            bool ok = !p.inject_withhold;
            for (int u = first; ok && u < tiles.total; u += step) {
                const Tile t = tiles.at(u);
                const int a_row = t.a_row + rank * SG_BM, b_row = t.b_row + rank * C::B_ROWS;
                for (int kb = t.k0; kb < t.k1; ++kb) {
                    if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full_leader0 + 8u * stage, to = base + stage * C::STAGE_BYTES;
                    if (leader)
                        mbar_arrive_expect_tx(full_bar(stage), C::CTAS * C::STAGE_BYTES);
                    issued |= 1u << stage;
                    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                    if (PAIR) {
                        tma_load_2d_pair(to, &p.tmA, fb, kb * SG_BK, a_row);
                        tma_load_2d_pair(to + C::A_BYTES, &p.tmB, fb, kb * SG_BK, b_row);
                    } else {
                        tma_load_2d(to, &p.tmA, fb, kb * SG_BK, a_row);
                        tma_load_2d(to + C::A_BYTES, &p.tmB, fb, kb * SG_BK, b_row);
                    }
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                if (leader) {
                    for (int s = 0; s < C::STAGES; ++s)
                        if ((issued >> s) & 1u)
                            mbar_drain(full_bar(s), (issued_parity >> s) & 1u);
                } else {
                    aborted_peer_loads = issued != 0;
                }
            }
        }
    } else if (warp == 1) {
        if (leader) {
            // ------------------------------------------------------ MMA issuer
            // The whole warp walks the loop and one lane issues: what the instructions
            // take is then the same in all lanes and stays in uniform registers.
            const uint32_t idesc = idesc_scaled(BM, BN, p.a_e5m2, p.b_e5m2);
            auto commit = [&](uint32_t bar) {
                if (PAIR)
                    umma_commit_pair(bar, 0x3);
                else
                    umma_commit(bar);
            };
            const uint32_t lo0 = desc_lo(base);
            const bool one = elect_one();
            int stage = 0, slot = 0;
            uint32_t phase = 0, slot_phase = 0, ctr = 0;
            bool ok = true;
            for (int u = first; ok && u < tiles.total; u += step) {
                const Tile t = tiles.at(u);
                if (t.k0 == t.k1)
                    continue;
                const int blocks = t.k1 - t.k0;
                for (int kp = 0; ok && kp < blocks; kp += C::PART) {
                    // the accumulator's last use has left it, or, where they overlap, the
                    // other's the shared columns
                    if (C::OVERLAP)
                        ok = ctr == 0 || wait_both(tempty0 + 8u * ((ctr - 1) & 1u), ((ctr - 1) >> 1) & 1u);
                    else
                        ok = wait_both(tempty0 + 8u * (ctr & 1u), ((ctr >> 1) & 1u) ^ 1u);
                    ok = __all_sync(0xffffffffu, ok);
                    tc_fence_after();
                    const uint32_t d = acc_col(ctr);
                    const int ke = min(kp + C::PART, blocks);
                    for (int kb = kp; ok && kb < ke; ++kb) {
                        const uint32_t byte = (uint32_t)kb & (SG_CHUNK - 1);
                        ok = (byte != 0 || wait_both(scaled_bar(slot), slot_phase)) &&
                             mbar_wait(full_bar(stage), phase, abort_flag, limit);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok)
                            break;
                        tc_fence_after();
                        const uint32_t a = lo0 + stage * (C::STAGE_BYTES >> 4), b = a + (C::A_BYTES >> 4);
                        const uint32_t sa = tmem + SG_SCALE_COL + slot * C::SCALE_COLS, sb = sa + 4;
                        const uint32_t id = idesc | (byte << 4) | (byte << 29);      // which byte, of B and of A
                        const bool last = byte == SG_CHUNK - 1 || kb + 1 == blocks;
                        if (one) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)           // (32 bytes of K)
                                umma_scaled<PAIR>(d, a + 2 * kk, b + 2 * kk, id, sa, sb,
                                                  kk > 0 ? 1u : (uint32_t)(kb - kp));
                            commit(empty_bar(stage));
                            if (last)
                                commit(used_bar(slot));
                        }
                        __syncwarp();
                        if (++stage == C::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        if (last && ++slot == C::SLOTS) {
                            slot = 0;
                            slot_phase ^= 1u;
                        }
                    }
                    if (ok) {
                        if (one)
                            commit(tfull0 + 8u * (ctr & 1u));
                        __syncwarp();
                        ++ctr;
                    }
                    if (!F32)
                        break;
                }
            }
            if (one) {
                if (PAIR)
                    umma_commit_pair(fin_bar, 0x1);
                else
                    umma_commit(fin_bar);
                mbar_drain(fin_bar, 0);
            }
        }
    } else if (warp == 2) {
        if (lane == 0) {
            // ------------------------------------------------ scales to shared memory
            int slot = 0;
            uint32_t phase = 0, issued = 0, issued_parity = 0;
            bool ok = !p.inject_withhold;
            for (int u = first; ok && u < tiles.total; u += step) {
                const Tile t = tiles.at(u);
                for (int kc = t.k0; kc < t.k1; kc += SG_CHUNK) {
                    if (!mbar_wait(sfree_bar(slot), phase ^ 1u, abort_flag, limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t to = smem_u32(scales + slot * C::SCALE_BYTES);
                    mbar_arrive_expect_tx(sload_bar(slot), C::SA_BOX + C::SB_BOX);
                    issued |= 1u << slot;
                    issued_parity = (issued_parity & ~(1u << slot)) | (phase << slot);
                    tma_load_2d(to, &p.tmSA, sload_bar(slot), (t.a_row + rank * SG_BM) & ~15, kc);
                    tma_load_2d(to + C::SA_BYTES, &p.tmSB, sload_bar(slot), t.n0, t.sb_row0 + kc);
                    if (++slot == SG_CHUNKS) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok)
                for (int s = 0; s < SG_CHUNKS; ++s)
                    if ((issued >> s) & 1u)
                        mbar_drain(sload_bar(s), (issued_parity >> s) & 1u);
        }
    } else if (warp >= 4 && warp < C::EPI_WARP0) {
        // ---------------------------------------------------------- scales to TMEM
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        int slot = 0, chunk = 0;
        uint32_t slot_phase = 0, chunk_phase = 0;
        bool ok = true;
        for (int u = first; ok && u < tiles.total; u += step) {
            const Tile t = tiles.at(u);
            const int rem = t.a_row & 15;
            for (int kc = t.k0; kc < t.k1; kc += SG_CHUNK) {
                if (!warp_wait(sload_bar(chunk), chunk_phase)) {
                    ok = false;
                    break;
                }
                // the bytes of four blocks side by side in a row's word (those past the
                // tile's last block are never named)
                const uint8_t *sa = scales + chunk * C::SCALE_BYTES + rem + lane;
                const uint8_t *sb = scales + chunk * C::SCALE_BYTES + C::SA_BYTES + lane;
                uint32_t wa[4], wb[BN / 32];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    wa[c] = sa[32 * c] | (sa[32 * c + SCALED_SA_BOX] << 8) | (sa[32 * c + 2 * SCALED_SA_BOX] << 16) |
                            ((uint32_t)sa[32 * c + 3 * SCALED_SA_BOX] << 24);
#pragma unroll
                for (int c = 0; c < BN / 32; ++c)
                    wb[c] = sb[32 * c] | (sb[32 * c + BN] << 8) | (sb[32 * c + 2 * BN] << 16) |
                            ((uint32_t)sb[32 * c + 3 * BN] << 24);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(sfree_bar(chunk));
                if (!warp_wait(used_bar(slot), slot_phase ^ 1u)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t to = tmem + quarter + SG_SCALE_COL + slot * C::SCALE_COLS;
                tmem_store<4>(to, wa);
                tmem_store<BN / 32>(to + 4, wb);
                tmem_store_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    arrive_leader(scaled_bar(slot));
                if (++slot == C::SLOTS) {
                    slot = 0;
                    slot_phase ^= 1u;
                }
                if (++chunk == SG_CHUNKS) {
                    chunk = 0;
                    chunk_phase ^= 1u;
                }
            }
        }
    } else if (warp >= C::EPI_WARP0) {
        // ------------------------------------------------------------ epilogue
        // TMEM lanes 32 (warp % 4) .. + 31, the left or right part of the columns
        constexpr int PIECES = BN / 32, LEFT = (PIECES + 1) / 2;
        const int quad = warp & 3, half = (warp - C::EPI_WARP0) >> 2;
        uint8_t *box = boxes + (warp - C::EPI_WARP0) * 4096;
        uint32_t ctr = 0;
        bool ok = true;
        for (int u = first; ok && u < tiles.total; u += step) {
            const Tile t = tiles.at(u);
            const bool empty = t.k0 == t.k1;
            const int row0 = t.out_row + rank * SG_BM + quad * 32;
            for (int kp = t.k0; ok && (kp == t.k0 || kp < t.k1); kp += C::PART) {
                if (!empty) {
                    if (!warp_wait(tfull0 + 8u * (ctr & 1u), (ctr >> 1) & 1u)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                const uint32_t acc = acc_col(ctr) + ((uint32_t)(quad * 32) << 16);
                auto release = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        arrive_leader(tempty0 + 8u * (ctr & 1u));
                };
                // Of overlapping accumulators the last two pieces of the lower and the first
                // two of the upper are the shared ones; who has none hands back at once (its
                // accumulator before is done).
                const bool lower = (ctr & 1u) == 0, shares = half == (lower ? 1 : 0);
                if (C::OVERLAP && !empty && !shares)
                    release();
                const int n = half ? PIECES - LEFT : LEFT, shift = C::OVERLAP && lower && half ? 2 : 0;
                const int after = C::OVERLAP ? (shares ? 1 : -1) : n - 1;
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    const int piece = half * LEFT + (C::OVERLAP ? (i + shift) & 3 : i);
                    store_piece<F32>(p, acc + piece * 32, empty, kp > t.k0, box, t.n0 + piece * 32, row0, t.m_end, lane,
                                     [&]() {
                                         if (!empty && i == after)
                                             release();
                                     });
                }
                if (!empty)
                    ++ctr;
                if (!F32)
                    break;
            }
        }
    }

    __syncwarp();
    if (aborted_peer_loads) {
        // the even CTA's barrier counts this CTA's copies; give them time to land
        const unsigned long long t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 100000ull) {
        }
    }
    tc_fence_before();
    if (PAIR)
        cluster_sync();
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if (PAIR)
            tmem_dealloc_pair(tmem, SG_TMEM_COLS);
        else
            tmem_dealloc(tmem, SG_TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag && p.status)
        atomicOr(p.status, ST_TIMEOUT);
}

template <int BN, bool PAIR, bool F32>
cudaError_t launch_as(const ScaledGemmParams &p, int units, cudaStream_t s)
{
    using C = SgCfg<BN, PAIR, F32>;
    auto kernel = scaled_gemm_kernel<BN, PAIR, F32>;
    static std::atomic<int> most[64];          // CTAs or pairs resident at once, for each device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C::CTAS;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(C::CTAS);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    int n = most[dev & 63].load();
    if (n == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess)
            return e;
        if (PAIR) {
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            if (e != cudaSuccess)
                return e;
        } else {
            n = 1 << 30;                       // (one to an SM: the caller's units)
        }
        if (n < 1)
            return cudaErrorInvalidConfiguration;
        most[dev & 63].store(n);
    }
    cfg.gridDim = dim3(C::CTAS * std::max(1, std::min(units, n)));
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int BN, bool PAIR>
cudaError_t launch_one(const ScaledGemmParams &p, int units, cudaStream_t s)
{
    return p.out_f32 ? launch_as<BN, PAIR, true>(p, units, s) : launch_as<BN, PAIR, false>(p, units, s);
}

}  // namespace

// The tile: a pair of CTAs with 256 or 224 columns, or one CTA with 128 or 64, by an
// estimate of the cycles that the tiles take, round by round: a tile's MMAs (545 for
// 256 columns and 128 of K), the loads of its operands (64 bytes a cycle) or its
// stores, whichever is longest, and what it costs by itself (256 columns: the wait for
// the shared part of the accumulators).  TFLOP/s with 256 and 224 columns: 8192 x
// 4096 x 2048 2800 and 2970; grouped, 262144 x 1024 x 2048 2680 and 2550.
ScaledTile scaled_tile(int mode, int M, int N, int E, int kblocks, bool f32, int sms)
{
    static const ScaledTile tiles[] = {{256, true}, {224, true}, {128, false}, {64, false}};
    ScaledTile best = tiles[0];
    double cost = -1.0;
    const double blocks = mode == SM_SUM && E ? (double)kblocks / E : kblocks;
    for (const ScaledTile &t : tiles) {
        const int rows = t.pair ? 256 : 128, slots = t.pair ? sms / 2 : sms, columns = t.columns;
        double m_tiles = (M + rows - 1) / rows;
        if (mode == SM_ROWS)             // each group's last tile is half full (the device knows)
            m_tiles = (double)M / rows + 0.5 * std::min(E, M);
        if (mode == SM_SUM && E)
            m_tiles *= E;
        const double units = m_tiles * ((N + columns - 1) / columns);
        const double rounds = units <= slots ? 1.0 : units / slots + (units < 4 * slots ? 0.5 : 0.0);
        const double mma = blocks * columns * (545.0 / 256), load = blocks * 128 * (128 + columns / (t.pair ? 2 : 1)) / 64;
        const double store = 128.0 * columns * (f32 ? 4 : 2) / 20;
        const double c = rounds * std::max(std::max(mma, load) + (columns == 256 ? 1100 : 400), store + 300);
        if (cost < 0.0 || c < cost) {
            cost = c;
            best = t;
        }
    }
    return best;
}

cudaError_t launch_scaled_gemm(const ScaledGemmParams &p, ScaledTile tile, int max_units, cudaStream_t s)
{
    return tile.columns == 256   ? launch_one<256, true>(p, max_units, s)
           : tile.columns == 224 ? launch_one<224, true>(p, max_units, s)
           : tile.columns == 128 ? launch_one<128, false>(p, max_units, s)
                                 : launch_one<64, false>(p, max_units, s);
}

}  // namespace glr
