// Norms around a block of a decoder layer, fused with the block's gate and the
// residual scale, and their backward.  With x the residual stream, y the
// block's output and RMSNorm(z) = z / sqrt(mean_h z^2 + eps):
//
//   u = RMSNorm(y),  r = alpha x + gate (u w_post)      the new residual stream
//   q = RMSNorm(r),  n = q w_pre                        the next block's input
//
// (y absent: r = alpha x, and only the second norm remains.)  n is formed from
// r before r is rounded for storage; every sum and statistic is fp32.
//
// Backward, from d_r (through the stream) and d_n (through the norm), with
// sigma = 1/sqrt(mean r^2 + eps), rho = 1/sqrt(mean y^2 + eps), dq = d_n w_pre:
//   dr = d_r + sigma (dq - q mean(dq q)),  d_x = alpha dr
//   du = dr gate w_post,  d_y = rho (du - u mean(du u))
//   dw_pre = sum_t d_n q,  dw_post = sum_t dr gate u,  d_gate = sum_t dr w_post u
// x and y are read again and r, u, q formed again: reading them costs what
// reading saved statistics and r would, and the forward need not keep anything.
//
// Bound by memory: forward 2 reads + 2 writes of [T, H], backward 4 + 2; what
// decides how near they come is the instructions per column and the loads in
// flight.  Each thread copies the bytes that it will read itself into shared
// memory of its own (cp.async), so loads in flight cost no registers and no
// thread waits for another's copies, and the arithmetic runs on pairs of fp32
// values (f32x2).
//   Forward: a row belongs to one warp up to H = 2048, so that 64 columns per
//   lane share each reduction and none needs a barrier; a row's piece is
//   fetched for the next row as soon as it has been read.  Wider rows belong to
//   a block, 16 columns per thread (two or four warps per row with 64 columns
//   per lane measured slower: 117 against 99 us at T = 16384, H = 4096, 142
//   against 87 us at T = 8192, H = 8192).
//   Backward: a row belongs to a block, 16 columns per thread, because the
//   column sums of all its rows stay in the threads' registers; rows are
//   fetched three (fp32 stream: two) ahead.  One warp per row with 64 columns
//   per lane measured slower (194 against 148 us at T = 32768, H = 2048): its
//   column sums leave registers for eight warps per SM.
// Measured on one GB300 (copy rate 6.79 TB/s): T = 32768, H = 2048 in bf16
// forward 92 us, 5.8 TB/s (0.86 of the copy rate); backward with the column sums
// 150 us, 5.4 TB/s (0.79), its two reductions per row and their barriers being
// the rest; with an fp32 stream 191 us (0.62) and 271 us (0.66; two rows in flight).
// T = 4095, H = 1536, fp32 stream, backward 39 us (0.43: five rows per block do not
// outlast a block's start and the column sums' kernel).
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace glr {

namespace {

constexpr int BN_WARPS = 8;          // forward, a warp per row: rows of a block at a time
constexpr int BN_BWD_WARPS = 16;     // a block per row: its warps at most

// two fp32 values in one register pair
struct F2 {
    uint64_t v;
};

__device__ __forceinline__ F2 f2(float lo, float hi)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 get(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ float sum2(F2 a)
{
    const float2 f = get(a);
    return f.x + f.y;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ void unpack8(const uint4 &q, F2 *f)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const F2 *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = get(f[i]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Eight consecutive values of a row: 16 bytes of bf16 or 32 of fp32, in 16-byte
// pieces.  In shared memory the pieces of the block's threads lie side by side.
constexpr int BN_THREADS = 32 * BN_WARPS;

template <bool F32>
struct Vec8;

template <>
struct Vec8<false> {
    static constexpr int PIECES = 1;
    static __device__ __forceinline__ void read(const uint4 *sm, int, F2 *f) { unpack8(*sm, f); }
    static __device__ __forceinline__ void store(void *p, size_t i, const F2 *f)
    {
        static_cast<uint4 *>(p)[i] = pack8(f);
    }
};

template <>
struct Vec8<true> {
    static constexpr int PIECES = 2;
    static __device__ __forceinline__ void read(const uint4 *sm, int threads, F2 *f)
    {
        const uint4 a = sm[0], b = sm[threads];
        f[0] = f2(__uint_as_float(a.x), __uint_as_float(a.y));
        f[1] = f2(__uint_as_float(a.z), __uint_as_float(a.w));
        f[2] = f2(__uint_as_float(b.x), __uint_as_float(b.y));
        f[3] = f2(__uint_as_float(b.z), __uint_as_float(b.w));
    }
    static __device__ __forceinline__ void store(void *p, size_t i, const F2 *f)
    {
        const float2 a = get(f[0]), b = get(f[1]), c = get(f[2]), d = get(f[3]);
        static_cast<float4 *>(p)[2 * i] = make_float4(a.x, a.y, b.x, b.y);
        static_cast<float4 *>(p)[2 * i + 1] = make_float4(c.x, c.y, d.x, d.y);
    }
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Sums over the block, the same bits in every thread (warp sums by butterfly,
// then the warps' sums in warp order).  `slot` alternates between calls, so one
// barrier per call suffices: a slot is written again only after the barrier of
// the call between, which every reader of it has passed.
__device__ __forceinline__ float block_sum(float v, float (*sm)[BN_BWD_WARPS], int &slot)
{
    v = warp_sum(v);
    const int nw = blockDim.x >> 5;
    if (nw == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        sm[slot][threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < nw; ++w)
        v += sm[slot][w];
    slot ^= 1;
    return v;
}

// The same for five values.  Each of the first three butterfly steps halves the
// values a lane carries (lane bits 4, 3, 2 choose which), 9 exchanges in all
// instead of 25.
__device__ __forceinline__ void block_sums5(float *t, float (*sm)[BN_BWD_WARPS][8], int &slot)
{
    const int lane = threadIdx.x & 31;
    float a[4];
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float hi = i == 0 ? t[4] : 0.0f;
        a[i] = (b4 ? hi : t[i]) + __shfl_xor_sync(0xffffffffu, b4 ? t[i] : hi, 16);
    }
    float c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        c[i] = (b3 ? a[2 + i] : a[i]) + __shfl_xor_sync(0xffffffffu, b3 ? a[i] : a[2 + i], 8);
    float d = (b2 ? c[1] : c[0]) + __shfl_xor_sync(0xffffffffu, b2 ? c[0] : c[1], 4);
    d += __shfl_xor_sync(0xffffffffu, d, 2);
    d += __shfl_xor_sync(0xffffffffu, d, 1);
    // lane 4 i holds value i
    const int nw = blockDim.x >> 5;
    if (nw == 1) {
#pragma unroll
        for (int i = 0; i < 5; ++i)
            t[i] = __shfl_sync(0xffffffffu, d, 4 * i);
        return;
    }
    if ((lane & 3) == 0)
        sm[slot][threadIdx.x >> 5][lane >> 2] = d;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 5; ++i)
        t[i] = 0.0f;
    for (int w = 0; w < nw; ++w) {
        const float4 q = *reinterpret_cast<const float4 *>(sm[slot][w]);
        t[0] += q.x; t[1] += q.y; t[2] += q.z; t[3] += q.w;
        t[4] += sm[slot][w][4];
    }
    slot ^= 1;
}

// eight fp32 weights, from shared or global memory (NULL: 1)
__device__ __forceinline__ void load_vec(const float *w, int v, F2 *f)
{
    if (!w) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = f2(1.0f);
        return;
    }
    const float4 a = reinterpret_cast<const float4 *>(w)[2 * v];
    const float4 b = reinterpret_cast<const float4 *>(w)[2 * v + 1];
    f[0] = f2(a.x, a.y); f[1] = f2(a.z, a.w); f[2] = f2(b.x, b.y); f[3] = f2(b.z, b.w);
}

// gate * w_post for one vector of columns
__device__ __forceinline__ void load_gw(const float *gate, const float *w_post, int v, F2 *f)
{
    F2 w[4];
    load_vec(gate, v, f);
    load_vec(w_post, v, w);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = mul2(f[i], w[i]);
}

// gate * w_post for this thread's columns
template <int VPT>
__device__ __forceinline__ void load_gw_columns(const BlockNormParams &p, int group, int nv, F2 (*gw)[4])
{
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        if (v >= nv)
            continue;
        load_gw(p.gate ? p.gate + (size_t)group * p.H : nullptr, p.w_post, v, gw[k]);
    }
}

// 16-byte pieces per vector of one row's inputs (x, y, backward also d_n, d_r),
// and the backward's rows in flight: what lets four blocks of a 2048-wide row
// share an SM's shared memory (48 KB each)
template <bool F32, bool HAS_Y, bool BWD>
struct Slots {
    static constexpr int X = F32 ? 2 : 1;
    static constexpr int AT_Y = X, AT_DN = X + (HAS_Y ? 1 : 0), AT_DR = AT_DN + 1;
    static constexpr int PIECES = BWD ? AT_DR + X : AT_DN;
    static constexpr int ROWS = (F32 ? 2 : 3) + (BWD ? 0 : 1);
};

// The weights' copies in shared memory, behind the rows' slots.
__device__ __forceinline__ void stage_weights(const BlockNormParams &p, uint4 *after, const float *&w_post,
                                              const float *&w_pre)
{
    w_post = p.w_post;
    w_pre = p.w_pre;
    float *post = reinterpret_cast<float *>(after), *pre = post + p.H;
    for (int h = threadIdx.x; h < p.H; h += BN_THREADS) {
        if (w_post)
            post[h] = w_post[h];
        if (w_pre)
            pre[h] = w_pre[h];
    }
    __syncthreads();
    w_post = w_post ? post : nullptr;
    w_pre = w_pre ? pre : nullptr;
}

}  // namespace

// A warp per row: warp w of block b takes rows w grid + b, and every (warps grid)-th
// after.
template <int VPT, bool F32, bool HAS_Y>
__global__ void __launch_bounds__(BN_THREADS) block_norm_kernel(const BlockNormParams p)
{
    using X = Vec8<F32>;
    using S = Slots<F32, HAS_Y, false>;
    extern __shared__ uint4 dyn[];       // [VPT][PIECES][threads], weights
    pdl_wait();
    const int nv = p.H / 8;
    const float inv_h = 1.0f / (float)p.H;
    const F2 alpha = f2(p.alpha);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int step = BN_WARPS * gridDim.x;
    uint4 *mine = dyn + threadIdx.x;
    const uint32_t mine_s = smem_u32(mine);
    auto fetch = [&](int k, int row) {
        const int v = lane + k * 32;
        if (row < p.T && v < nv) {
            const size_t at = (size_t)row * nv + v;
            const uint32_t dst = mine_s + k * S::PIECES * BN_THREADS * 16;
#pragma unroll
            for (int i = 0; i < S::X; ++i)
                cp_async16(dst + i * BN_THREADS * 16, static_cast<const uint4 *>(p.x) + at * S::X + i);
            if (HAS_Y)
                cp_async16(dst + S::AT_Y * BN_THREADS * 16, reinterpret_cast<const uint4 *>(p.y) + at);
        }
    };
    int row = warp * gridDim.x + blockIdx.x;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
        fetch(k, row);
    const float *w_post, *w_pre;
    stage_weights(p, dyn + VPT * S::PIECES * BN_THREADS, w_post, w_pre);
    for (; row < p.T; row += step) {
        cp_async_wait_all();
        const float *gate = p.gate ? p.gate + (size_t)(row / p.rows_per_gate) * p.H : nullptr;
        F2 rho = f2(0.0f);
        if (HAS_Y) {
            F2 s = f2(0.0f);
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (lane + k * 32 < nv) {
                    F2 y[4];
                    unpack8(mine[(k * S::PIECES + S::AT_Y) * BN_THREADS], y);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s = fma2(y[i], y[i], s);
                }
            rho = f2(rsqrtf(warp_sum(sum2(s)) * inv_h + p.eps));
        }
        F2 r[VPT][4];
        F2 s = f2(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = lane + k * 32;
            if (v < nv) {
                const uint4 *at = mine + k * S::PIECES * BN_THREADS;
                X::read(at, BN_THREADS, r[k]);
                if (HAS_Y) {
                    F2 y[4], gw[4];
                    unpack8(at[S::AT_Y * BN_THREADS], y);
                    load_gw(gate, w_post, v, gw);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        r[k][i] = fma2(alpha, r[k][i], mul2(gw[i], mul2(y[i], rho)));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        r[k][i] = mul2(alpha, r[k][i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s = fma2(r[k][i], r[k][i], s);
                fetch(k, row + step);
            }
        }
        const F2 sigma = f2(rsqrtf(warp_sum(sum2(s)) * inv_h + p.eps));
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = lane + k * 32;
            if (v < nv) {
                if (p.r)
                    X::store(p.r, (size_t)row * nv + v, r[k]);
                F2 w[4];
                load_vec(w_pre, v, w);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = mul2(mul2(r[k][i], sigma), w[i]);
                Vec8<false>::store(p.n, (size_t)row * nv + v, w);
            }
        }
    }
}

// Rows wider than a warp's registers hold (H > 2048): a block per row, rows
// fetched four (fp32 stream: three) ahead.  Block b takes rows [b T / grid, (b + 1) T / grid).
template <int VPT, bool F32, bool HAS_Y>
__global__ void __launch_bounds__(512) block_norm_wide_kernel(const BlockNormParams p)
{
    using X = Vec8<F32>;
    using At = Slots<F32, HAS_Y, false>;
    constexpr int P = At::PIECES, S = At::ROWS;
    extern __shared__ uint4 ring[];      // [S][VPT][P][threads]
    __shared__ float sm[2][BN_BWD_WARPS];
    pdl_wait();
    const int nt = blockDim.x;
    const int nv = p.H / 8;
    const int row0 = (int)((long long)blockIdx.x * p.T / gridDim.x);
    const int row1 = (int)((long long)(blockIdx.x + 1) * p.T / gridDim.x);
    const float inv_h = 1.0f / (float)p.H;
    const F2 alpha = f2(p.alpha);
    int slot = 0, group = -1;
    uint4 *mine = ring + threadIdx.x;
    auto fetch = [&](int row, int st) {
        if (row < row1)
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = threadIdx.x + k * nt;
                if (v < nv) {
                    const size_t at = (size_t)row * nv + v;
                    const uint32_t dst = smem_u32(mine + (st * VPT + k) * P * nt);
#pragma unroll
                    for (int i = 0; i < X::PIECES; ++i)
                        cp_async16(dst + i * nt * 16, static_cast<const uint4 *>(p.x) + at * X::PIECES + i);
                    if (HAS_Y)
                        cp_async16(dst + X::PIECES * nt * 16, reinterpret_cast<const uint4 *>(p.y) + at);
                }
            }
        cp_async_commit();
    };
#pragma unroll
    for (int st = 0; st < S; ++st)
        fetch(row0 + st, st);
    F2 gw[VPT][4], wpre[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * nt;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            gw[k][i] = wpre[k][i] = f2(0.0f);
        if (v < nv)
            load_vec(p.w_pre, v, wpre[k]);
    }
    int st = 0;
    for (int row = row0; row < row1; ++row) {
        if (HAS_Y && row / p.rows_per_gate != group) {
            group = row / p.rows_per_gate;
            load_gw_columns<VPT>(p, group, nv, gw);
        }
        cp_async_wait<S - 1>();
        F2 r[VPT][4], y[VPT][4];
        F2 s = f2(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r[k][i] = y[k][i] = f2(0.0f);
            if (threadIdx.x + k * nt < nv) {
                const uint4 *at = mine + (st * VPT + k) * P * nt;
                X::read(at, nt, r[k]);
                if (HAS_Y) {
                    unpack8(at[X::PIECES * nt], y[k]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s = fma2(y[k][i], y[k][i], s);
                }
            }
        }
        fetch(row + S, st);
        st = st + 1 == S ? 0 : st + 1;
        F2 rho = f2(0.0f);
        if (HAS_Y)
            rho = f2(rsqrtf(block_sum(sum2(s), sm, slot) * inv_h + p.eps));
        s = f2(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (HAS_Y)
                    r[k][i] = fma2(alpha, r[k][i], mul2(gw[k][i], mul2(y[k][i], rho)));
                else
                    r[k][i] = mul2(alpha, r[k][i]);
                s = fma2(r[k][i], r[k][i], s);
            }
        const F2 sigma = f2(rsqrtf(block_sum(sum2(s), sm, slot) * inv_h + p.eps));
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = threadIdx.x + k * nt;
            if (v >= nv)
                continue;
            if (p.r)
                X::store(p.r, (size_t)row * nv + v, r[k]);
            F2 n[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                n[i] = mul2(mul2(r[k][i], sigma), wpre[k][i]);
            Vec8<false>::store(p.n, (size_t)row * nv + v, n);
        }
    }
    cp_async_wait<0>();
}

// Chunk c holds rows of one gate group only: group c / cpg, its part c % cpg of
// cpg.  Block b takes chunks [b C / grid, (b + 1) C / grid).  Per chunk it
// leaves A[c] = sum_t dr u (the finish kernel's d_gate and dw_post), and per
// block B[b] = sum_t d_n q (dw_pre).
template <int VPT, bool F32, bool HAS_Y>
__global__ void __launch_bounds__(512) block_norm_backward_kernel(const BlockNormParams p)
{
    using X = Vec8<F32>;
    using At = Slots<F32, HAS_Y, true>;
    constexpr int P = At::PIECES, S = At::ROWS, AT_DN = At::AT_DN, AT_DR = At::AT_DR, AT_Y = At::AT_Y;
    extern __shared__ uint4 ring[];      // [S][VPT][P][threads]
    __shared__ float sm1[2][BN_BWD_WARPS];
    __shared__ __align__(16) float sm5[2][BN_BWD_WARPS][8];
    pdl_wait();
    const int nt = blockDim.x;
    const int nv = p.H / 8;
    const float inv_h = 1.0f / (float)p.H;
    const F2 alpha = f2(p.alpha);
    const int chunks = p.groups * p.cpg;
    const int c0 = (int)((long long)blockIdx.x * chunks / gridDim.x);
    const int c1 = (int)((long long)(blockIdx.x + 1) * chunks / gridDim.x);
    auto chunk_begin = [&](int c) {
        return (c / p.cpg) * p.rows_per_gate + (int)((long long)(c % p.cpg) * p.rows_per_gate / p.cpg);
    };
    const int row_end = chunk_begin(c1);   // (chunks are contiguous)
    int slot1 = 0, slot5 = 0;
    uint4 *mine = ring + threadIdx.x;
    auto fetch = [&](int row, int st) {
        if (row < row_end)
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = threadIdx.x + k * nt;
                if (v < nv) {
                    const size_t at = (size_t)row * nv + v;
                    const uint32_t dst = smem_u32(mine + (st * VPT + k) * P * nt);
                    if (HAS_Y)
                        cp_async16(dst + AT_Y * nt * 16, reinterpret_cast<const uint4 *>(p.y) + at);
#pragma unroll
                    for (int i = 0; i < X::PIECES; ++i)
                        cp_async16(dst + i * nt * 16, static_cast<const uint4 *>(p.x) + at * X::PIECES + i);
                    cp_async16(dst + AT_DN * nt * 16, reinterpret_cast<const uint4 *>(p.d_n) + at);
                    if (p.d_r)
#pragma unroll
                        for (int i = 0; i < X::PIECES; ++i)
                            cp_async16(dst + (AT_DR + i) * nt * 16,
                                       static_cast<const uint4 *>(p.d_r) + at * X::PIECES + i);
                }
            }
        cp_async_commit();
    };
    const int first = chunk_begin(c0);
#pragma unroll
    for (int st = 0; st < S; ++st)
        fetch(first + st, st);
    F2 gw[VPT][4], wpre[VPT][4], accA[VPT][4], accB[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * nt;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            gw[k][i] = wpre[k][i] = accB[k][i] = f2(0.0f);
        if (v < nv)
            load_vec(p.w_pre, v, wpre[k]);
    }
    int st = 0;
    for (int c = c0; c < c1; ++c) {
        const int begin = chunk_begin(c), end = chunk_begin(c + 1);
        if (HAS_Y && (c == c0 || c % p.cpg == 0))
            load_gw_columns<VPT>(p, c / p.cpg, nv, gw);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                accA[k][i] = f2(0.0f);
        for (int row = begin; row < end; ++row) {
            cp_async_wait<S - 1>();
            const uint4 *stage = mine + st * VPT * P * nt;
            F2 r[VPT][4], u[VPT][4];
            F2 s = f2(0.0f);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    r[k][i] = u[k][i] = f2(0.0f);
                if (threadIdx.x + k * nt < nv) {
                    X::read(stage + k * P * nt, nt, r[k]);
                    if (HAS_Y) {
                        unpack8(stage[(k * P + AT_Y) * nt], u[k]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s = fma2(u[k][i], u[k][i], s);
                    }
                }
            }
            float rho = 0.0f;
            if (HAS_Y)
                rho = rsqrtf(block_sum(sum2(s), sm1, slot1) * inv_h + p.eps);
            // sum r^2, sum dq r, and the three parts of sum du u
            F2 t[5];
#pragma unroll
            for (int i = 0; i < 5; ++i)
                t[i] = f2(0.0f);
            const F2 rho2 = f2(rho);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                F2 dr[4], dn[4];
                if (threadIdx.x + k * nt < nv) {
                    unpack8(stage[(k * P + AT_DN) * nt], dn);
                    if (p.d_r && HAS_Y)
                        X::read(stage + (k * P + AT_DR) * nt, nt, dr);
                    else
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dr[i] = f2(0.0f);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dr[i] = dn[i] = f2(0.0f);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const F2 dq = mul2(dn[i], wpre[k][i]);
                    if (HAS_Y) {
                        u[k][i] = mul2(u[k][i], rho2);
                        const F2 a = mul2(gw[k][i], u[k][i]);
                        r[k][i] = fma2(alpha, r[k][i], a);
                        t[2] = fma2(a, dr[i], t[2]);
                        t[3] = fma2(a, dq, t[3]);
                        t[4] = fma2(a, r[k][i], t[4]);
                    } else {
                        r[k][i] = mul2(alpha, r[k][i]);
                    }
                    t[0] = fma2(r[k][i], r[k][i], t[0]);
                    t[1] = fma2(dq, r[k][i], t[1]);
                }
            }
            float q5[5] = {sum2(t[0]), sum2(t[1]), sum2(t[2]), sum2(t[3]), sum2(t[4])};
            block_sums5(q5, sm5, slot5);
            const float sigma = rsqrtf(q5[0] * inv_h + p.eps);
            // dr = d_r + sigma dq - c_r r, c_r = sigma^2 mean(dq q) = sigma (sigma (sigma mean(dq r))):
            // from the inside each factor stays near the gradient's size, while sigma^3 leaves
            // fp32's range from RMS(r) = 1e-13 down, where sigma^2 is at 1e26
            const float c_r = sigma * (sigma * (sigma * (q5[1] * inv_h)));
            const float c_u = (q5[2] + sigma * q5[3] - c_r * q5[4]) * inv_h;   // mean(du u)
            const F2 sigma2 = f2(sigma), ncr = f2(-c_r), ncu = f2(-c_u);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = threadIdx.x + k * nt;
                if (v >= nv)
                    continue;
                F2 dx[4], dy[4], dr[4], dn[4];
                unpack8(stage[(k * P + AT_DN) * nt], dn);
                if (p.d_r)
                    X::read(stage + (k * P + AT_DR) * nt, nt, dr);
                else
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dr[i] = f2(0.0f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const F2 sdn = mul2(sigma2, dn[i]);
                    accB[k][i] = fma2(sdn, r[k][i], accB[k][i]);
                    const F2 g = fma2(ncr, r[k][i], fma2(sdn, wpre[k][i], dr[i]));
                    dx[i] = mul2(alpha, g);
                    if (HAS_Y) {
                        accA[k][i] = fma2(g, u[k][i], accA[k][i]);
                        dy[i] = mul2(rho2, fma2(ncu, u[k][i], mul2(g, gw[k][i])));
                    }
                }
                X::store(p.d_x, (size_t)row * nv + v, dx);
                if (HAS_Y)
                    Vec8<false>::store(p.d_y, (size_t)row * nv + v, dy);
            }
            fetch(row + S, st);
            st = st + 1 == S ? 0 : st + 1;
        }
        if (HAS_Y)
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = threadIdx.x + k * nt;
                if (v < nv)
                    Vec8<true>::store(p.part_a, (size_t)c * nv + v, accA[k]);
            }
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * nt;
        if (v < nv)
            Vec8<true>::store(p.part_b, (size_t)blockIdx.x * nv + v, accB[k]);
    }
    cp_async_wait<0>();
}

// The column sums from the chunks' and blocks' partial sums, in a fixed order:
// dw_pre = sum_b B[b], d_gate[g] = w_post sum_c A[g, c], dw_post = sum_g gate[g]
// sum_c A[g, c].  A block takes FIN_COLS columns: FIN_LANES threads of four
// columns each (a sector of a row), FIN_SLICES partial sums at a time, all loads of
// a thread in flight at once.  32 columns and 1024 threads left most SMs idle: the
// whole backward 40.1 against 39.0 us at T = 4095, H = 1536; 16 columns 39.6.
constexpr int FIN_COLS = 8, FIN_THREADS = 512;
constexpr int FIN_LANES = FIN_COLS / 4, FIN_SLICES = FIN_THREADS / FIN_LANES, FIN_WARPS = FIN_THREADS / 32;
__global__ void __launch_bounds__(FIN_THREADS) block_norm_finish_kernel(const BlockNormParams p, int blocks)
{
    __shared__ __align__(16) float sm[FIN_WARPS][FIN_COLS];
    pdl_wait();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = (lane % FIN_LANES) * 4, slice = threadIdx.x / FIN_LANES;
    const int h = blockIdx.x * FIN_COLS + col;
    const bool in = h < p.H;                      // (H is a multiple of 8)
    auto add = [](float4 &a, const float4 &b) { a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w; };
    // sum of partial sums row0 .. row0 + n - 1 by `many` slices, this thread being number `at` of them
    auto some = [&](const float *part, size_t row0, int n, int at, int many) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = at; i < n; i += many)
            add(a, *reinterpret_cast<const float4 *>(part + (row0 + i) * p.H + h));
        return a;
    };
    // the warp's slices, then the warps in order; warp 0's first lanes get column `lane`
    auto across = [&](float4 a) {
#pragma unroll
        for (int off = FIN_LANES; off <= 16; off <<= 1) {
            a.x += __shfl_xor_sync(0xffffffffu, a.x, off);
            a.y += __shfl_xor_sync(0xffffffffu, a.y, off);
            a.z += __shfl_xor_sync(0xffffffffu, a.z, off);
            a.w += __shfl_xor_sync(0xffffffffu, a.w, off);
        }
        __syncthreads();
        if (lane < FIN_LANES)
            *reinterpret_cast<float4 *>(&sm[w][col]) = a;
        __syncthreads();
        float t = 0.0f;
        if (w == 0 && lane < FIN_COLS)
#pragma unroll
            for (int i = 0; i < FIN_WARPS; ++i)
                t += sm[i][lane];
        return t;
    };
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const int out = blockIdx.x * FIN_COLS + lane; // warp 0's column
    const bool mine = w == 0 && lane < FIN_COLS && out < p.H;
    constexpr int FEW = 4;
    const bool few = p.part_a && p.groups <= FEW;  // a few long groups: the whole block takes each
    float4 part[1 + FEW];
    part[0] = in ? some(p.part_b, 0, blocks, slice, FIN_SLICES) : zero;
#pragma unroll
    for (int g = 0; g < FEW; ++g)
        part[1 + g] = in && few && g < p.groups ? some(p.part_a, (size_t)g * p.cpg, p.cpg, slice, FIN_SLICES) : zero;
    const float pre = across(part[0]);
    if (mine && p.dw_pre)
        p.dw_pre[out] = pre;
    if (!p.part_a)
        return;
    if (few) {
        const float wp = mine && p.w_post ? p.w_post[out] : 1.0f;
        float post = 0.0f;
#pragma unroll
        for (int g = 0; g < FEW; ++g) {
            if (g >= p.groups)
                break;
            const float a = across(part[1 + g]);
            if (mine) {
                if (p.d_gate)
                    p.d_gate[(size_t)g * p.H + out] = wp * a;
                post = fmaf(p.gate ? p.gate[(size_t)g * p.H + out] : 1.0f, a, post);
            }
        }
        if (mine && p.dw_post)
            p.dw_post[out] = post;
        return;
    }
    // many groups: each by one slice, a group's chunks in sequence.  T = 32768, H = 2048:
    // 165 us with 8 groups, 159 with 16 and 64, against 152 with one; T = 65536, H = 256,
    // where a group has the most chunks: 88 us with 8, 48 with 64, against 42 with one.
    float4 wp = make_float4(1.f, 1.f, 1.f, 1.f), post = zero;
    if (in && p.w_post)
        wp = *reinterpret_cast<const float4 *>(p.w_post + h);
    if (in)
        for (int g = slice; g < p.groups; g += FIN_SLICES) {
            const float4 a = some(p.part_a, (size_t)g * p.cpg, p.cpg, 0, 1);
            const size_t at = (size_t)g * p.H + h;
            if (p.d_gate) {
                p.d_gate[at] = wp.x * a.x;
                p.d_gate[at + 1] = wp.y * a.y;
                p.d_gate[at + 2] = wp.z * a.z;
                p.d_gate[at + 3] = wp.w * a.w;
            }
            float4 q = make_float4(1.f, 1.f, 1.f, 1.f);
            if (p.gate)
                q = *reinterpret_cast<const float4 *>(p.gate + at);
            post.x = fmaf(q.x, a.x, post.x);
            post.y = fmaf(q.y, a.y, post.y);
            post.z = fmaf(q.z, a.z, post.z);
            post.w = fmaf(q.w, a.w, post.w);
        }
    const float total = across(post);
    if (mine && p.dw_post)
        p.dw_post[out] = total;
}

namespace {

// Forward, a warp per row: vectors per lane.
int lane_vectors(int H)
{
    const int nv = H / 8;
    return nv <= 32 ? 1 : nv <= 64 ? 2 : nv <= 128 ? 4 : 8;
}

constexpr int BN_WARP_MAX_H = 2048;

// A block per row: vectors per thread, threads.
struct RowShape {
    int vpt, threads;
};

RowShape row_shape(int H)
{
    const int nv = H / 8;
    const int vpt = nv <= 32 ? 1 : 2;
    const int per = (nv + vpt - 1) / vpt;
    return {vpt, (per + 31) / 32 * 32};
}

cudaError_t launch(void (*kernel)(BlockNormParams), const BlockNormParams &p, int blocks, int threads, size_t smem,
                   cudaStream_t s)
{
    if (smem > 40 * 1024) {          // (with the static arrays, past the 48 KB that need no opting in)
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
    }
    const cudaError_t e = launch_pdl(kernel, dim3(blocks), dim3(threads), smem, s, p);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

template <int VPT>
cudaError_t launch_fwd(const BlockNormParams &p, bool f32, int blocks, cudaStream_t s)
{
    const bool y = p.y != nullptr;
    const int pieces = (f32 ? 2 : 1) + (y ? 1 : 0);
    // the rows' slots, then the weights' copies (112 KB at most)
    const size_t smem = (size_t)VPT * pieces * BN_THREADS * 16 + 8ull * p.H;
    return launch(f32 ? (y ? block_norm_kernel<VPT, true, true> : block_norm_kernel<VPT, true, false>)
                      : (y ? block_norm_kernel<VPT, false, true> : block_norm_kernel<VPT, false, false>),
                  p, blocks, BN_THREADS, smem, s);
}

cudaError_t launch_wide(const BlockNormParams &p, bool f32, int blocks, int threads, cudaStream_t s)
{
    const bool y = p.y != nullptr;
    const int pieces = (f32 ? 2 : 1) + (y ? 1 : 0);
    const size_t smem = (size_t)(f32 ? Slots<true, true, false>::ROWS : Slots<false, true, false>::ROWS) * 2 * pieces *
                        threads * 16;
    return launch(f32 ? (y ? block_norm_wide_kernel<2, true, true> : block_norm_wide_kernel<2, true, false>)
                      : (y ? block_norm_wide_kernel<2, false, true> : block_norm_wide_kernel<2, false, false>),
                  p, blocks, threads, smem, s);
}

template <int VPT>
cudaError_t launch_bwd(const BlockNormParams &p, bool f32, int blocks, int threads, cudaStream_t s)
{
    const bool y = p.y != nullptr;
    const int pieces = (f32 ? 4 : 2) + (y ? 2 : 1);
    const size_t smem = (size_t)(f32 ? Slots<true, true, true>::ROWS : Slots<false, true, true>::ROWS) * VPT * pieces *
                        threads * 16;
    return launch(f32 ? (y ? block_norm_backward_kernel<VPT, true, true> : block_norm_backward_kernel<VPT, true, false>)
                      : (y ? block_norm_backward_kernel<VPT, false, true>
                           : block_norm_backward_kernel<VPT, false, false>),
                  p, blocks, threads, smem, s);
}

}  // namespace

// Forward: rows go round the blocks first, so that a few rows spread over the
// SMs; narrow rows leave room for several blocks per SM.  A block per row: 512
// threads per SM, as backward.
int block_norm_blocks(int T, int H, int sms)
{
    const int vpt = lane_vectors(H);
    const int n = sms * (H > BN_WARP_MAX_H ? 512 / row_shape(H).threads : vpt >= 8 ? 2 : vpt >= 4 ? 3 : 6);
    return T < n ? T : n;
}

// Backward: 512 threads per SM (at the 128 registers that the launch bounds
// allow, what the register file holds).  The chunks per gate group are those
// with the fewest rows in the longest-working block, and of equal ones the most.
BlockNormPlan block_norm_plan(int T, int H, int groups, int sms)
{
    const int rows = T / groups;
    const int most = sms * (512 / row_shape(H).threads);
    BlockNormPlan best = {};
    long long least = -1;
    for (int m = 0; m <= 4; ++m) {       // one chunk per group, or as many as fill the blocks m times
        const long long want = m ? (long long)m * most / groups : 1;
        const int cpg = (int)(want < 1 ? 1 : want > rows ? rows : want);
        const long long chunks = (long long)groups * cpg;
        const long long cost = (chunks + most - 1) / most * ((rows + cpg - 1) / cpg);
        if (least < 0 || cost < least || (cost == least && chunks <= most)) {
            least = cost;
            best.cpg = cpg;
            best.blocks = (int)(chunks < most ? chunks : most);
        }
    }
    return best;
}

cudaError_t launch_block_norm(const BlockNormParams &p, bool stream_f32, int blocks, cudaStream_t s)
{
    if (p.H > BN_WARP_MAX_H)
        return launch_wide(p, stream_f32, blocks, row_shape(p.H).threads, s);
    switch (lane_vectors(p.H)) {
    case 1: return launch_fwd<1>(p, stream_f32, blocks, s);
    case 2: return launch_fwd<2>(p, stream_f32, blocks, s);
    case 4: return launch_fwd<4>(p, stream_f32, blocks, s);
    default: return launch_fwd<8>(p, stream_f32, blocks, s);
    }
}

cudaError_t launch_block_norm_backward(const BlockNormParams &p, bool stream_f32, int blocks, cudaStream_t s)
{
    const RowShape sh = row_shape(p.H);
    return sh.vpt == 1 ? launch_bwd<1>(p, stream_f32, blocks, sh.threads, s)
                       : launch_bwd<2>(p, stream_f32, blocks, sh.threads, s);
}

cudaError_t launch_block_norm_finish(const BlockNormParams &p, int blocks, cudaStream_t s)
{
    const cudaError_t e = launch_pdl(block_norm_finish_kernel, dim3((p.H + FIN_COLS - 1) / FIN_COLS),
                                     dim3(FIN_THREADS), 0, s, p, blocks);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace glr
