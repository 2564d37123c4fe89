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
// Bound by memory: forward 2 reads + 2 writes of [T, H], backward 4 + 2.  One
// block holds one row, up to sixteen columns per thread, so a row's values stay
// in registers and shared memory between the two reductions that it needs.
// Each thread copies the bytes that it will read itself, rows ahead, into
// shared memory of its own (cp.async): the loads in flight do not cost
// registers, and no thread waits for another's copies.  The arithmetic runs on
// pairs of fp32 values (f32x2): one value at a time, the instructions issued
// take as long as the memory.
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace glr {

namespace {

constexpr int BN_MAX_WARPS = 16;

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

// Eight consecutive values of a row: 16 bytes of bf16 or 32 of fp32.  In shared
// memory the 16-byte pieces of the block's threads lie side by side.
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

// Sums over the block, the same bits in every thread (warp sums by butterfly,
// then the warps' sums in warp order).  `slot` alternates between calls, so one
// barrier per call suffices: a slot is written again only after the barrier of
// the call between, which every reader of it has passed.
__device__ __forceinline__ float block_sum(float v, float (*sm)[BN_MAX_WARPS], int &slot)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
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
__device__ __forceinline__ void block_sums5(float *t, float (*sm)[BN_MAX_WARPS][8], int &slot)
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

// eight weights (NULL: 1)
__device__ __forceinline__ void load_vec(const float *w, int v, F2 *f)
{
    if (!w) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = f2(1.0f);
        return;
    }
    const float4 a = __ldg(reinterpret_cast<const float4 *>(w) + 2 * v);
    const float4 b = __ldg(reinterpret_cast<const float4 *>(w) + 2 * v + 1);
    f[0] = f2(a.x, a.y); f[1] = f2(a.z, a.w); f[2] = f2(b.x, b.y); f[3] = f2(b.z, b.w);
}

// gate * w_post for this thread's columns
template <int VPT>
__device__ __forceinline__ void load_gw(const BlockNormParams &p, int group, int nv, F2 (*gw)[4])
{
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        if (v >= nv)
            continue;
        F2 g[4], w[4];
        load_vec(p.gate ? p.gate + (size_t)group * p.H : nullptr, v, g);
        load_vec(p.w_post, v, w);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            gw[k][i] = mul2(g[i], w[i]);
    }
}

// 16-byte pieces per thread and vector of one row's inputs, and the rows in
// flight: what lets four blocks of a 2048-wide row share an SM's shared memory
// (48 KB each, 32 KB forward)
template <bool F32, bool HAS_Y, bool BWD>
struct Ring {
    static constexpr int X = F32 ? 2 : 1;
    static constexpr int PIECES = X + (HAS_Y ? 1 : 0) + (BWD ? X + 1 : 0);
    static constexpr int ROWS = BWD ? (F32 ? 2 : 3) : (F32 ? 3 : 4);
};

}  // namespace

// Rows [b T / grid, (b + 1) T / grid) of block b.
template <int VPT, bool F32, bool HAS_Y>
__global__ void __launch_bounds__(512) block_norm_kernel(const BlockNormParams p)
{
    using X = Vec8<F32>;
    constexpr int P = Ring<F32, HAS_Y, false>::PIECES, S = Ring<F32, HAS_Y, false>::ROWS;
    extern __shared__ uint4 ring[];      // [S][VPT][P][threads]
    __shared__ float sm[2][BN_MAX_WARPS];
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
            load_gw<VPT>(p, group, nv, gw);
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
            rho = f2(1.0f / sqrtf(block_sum(sum2(s), sm, slot) * inv_h + p.eps));
        s = f2(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r[k][i] = mul2(alpha, r[k][i]);
                if (HAS_Y)
                    r[k][i] = fma2(gw[k][i], mul2(y[k][i], rho), r[k][i]);
                s = fma2(r[k][i], r[k][i], s);
            }
        const F2 sigma = f2(1.0f / sqrtf(block_sum(sum2(s), sm, slot) * inv_h + p.eps));
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
    constexpr int P = Ring<F32, HAS_Y, true>::PIECES, S = Ring<F32, HAS_Y, true>::ROWS;
    constexpr int AT_DN = X::PIECES, AT_DR = X::PIECES + 1, AT_Y = 2 * X::PIECES + 1;
    extern __shared__ uint4 ring[];      // [S][VPT][P][threads]
    __shared__ float sm1[2][BN_MAX_WARPS];
    __shared__ __align__(16) float sm5[2][BN_MAX_WARPS][8];
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
            load_gw<VPT>(p, c / p.cpg, nv, gw);
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
                rho = 1.0f / sqrtf(block_sum(sum2(s), sm1, slot1) * inv_h + p.eps);
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
                    r[k][i] = mul2(alpha, r[k][i]);
                    if (HAS_Y) {
                        u[k][i] = mul2(u[k][i], rho2);
                        const F2 a = mul2(gw[k][i], u[k][i]);
                        r[k][i] = fma2(gw[k][i], u[k][i], r[k][i]);
                        t[2] = fma2(a, dr[i], t[2]);
                        t[3] = fma2(a, dq, t[3]);
                        t[4] = fma2(a, r[k][i], t[4]);
                    }
                    t[0] = fma2(r[k][i], r[k][i], t[0]);
                    t[1] = fma2(dq, r[k][i], t[1]);
                }
            }
            float q5[5] = {sum2(t[0]), sum2(t[1]), sum2(t[2]), sum2(t[3]), sum2(t[4])};
            block_sums5(q5, sm5, slot5);
            const float sigma = 1.0f / sqrtf(q5[0] * inv_h + p.eps);
            // dr = d_r + sigma dq - (sigma^3 mean(dq r)) r
            const float c_r = sigma * sigma * sigma * (q5[1] * inv_h);
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
// sum_c A[g, c].  32 columns per block, 32 rows of the partial sums at a time.
__global__ void __launch_bounds__(1024) block_norm_finish_kernel(const BlockNormParams p, int blocks)
{
    __shared__ float sm[32][33];
    pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int h = blockIdx.x * 32 + lane;
    const bool in = h < p.H;
    auto across = [&](float v) {      // sum over the 32 warps, in warp order; thread (0, lane) gets it
        __syncthreads();
        sm[w][lane] = v;
        __syncthreads();
        float t = 0.0f;
        if (w == 0)
            for (int i = 0; i < 32; ++i)
                t += sm[i][lane];
        return t;
    };
    float s = 0.0f;
#pragma unroll 8
    for (int b = w; b < blocks; b += 32)
        if (in)
            s += p.part_b[(size_t)b * p.H + h];
    s = across(s);
    if (w == 0 && in && p.dw_pre)
        p.dw_pre[h] = s;
    if (!p.part_a)
        return;
    const float wp = (in && p.w_post) ? p.w_post[h] : 1.0f;
    float post = 0.0f;
    if (p.cpg == 1) {
        // whole groups: one per warp and step
        for (int g = w; g < p.groups; g += 32)
            if (in) {
                const float a = p.part_a[(size_t)g * p.H + h];
                if (p.d_gate)
                    p.d_gate[(size_t)g * p.H + h] = wp * a;
                post = fmaf(p.gate ? p.gate[(size_t)g * p.H + h] : 1.0f, a, post);
            }
    } else {
        // up to 32 groups at a time, the 32 warps shared out among them
        const int at_once = min(32, p.groups), wpg = 32 / at_once;
        const int gi = w / wpg, sub = w % wpg;
        for (int g0 = 0; g0 < p.groups; g0 += at_once) {
            const int g = g0 + gi;
            const bool mine = in && gi < at_once && g < p.groups;
            float a = 0.0f;
#pragma unroll 8
            for (int c = sub; c < p.cpg; c += wpg)
                if (mine)
                    a += p.part_a[((size_t)g * p.cpg + c) * p.H + h];
            __syncthreads();
            sm[w][lane] = a;
            __syncthreads();
            if (mine && sub == 0) {
                for (int i = 1; i < wpg; ++i)
                    a += sm[w + i][lane];
                if (p.d_gate)
                    p.d_gate[(size_t)g * p.H + h] = wp * a;
                post = fmaf(p.gate ? p.gate[(size_t)g * p.H + h] : 1.0f, a, post);
            }
        }
    }
    post = across(post);
    if (w == 0 && in && p.dw_post)
        p.dw_post[h] = post;
}

namespace {

struct Shape {
    int vpt, threads;
};

// Sixteen columns per thread (eight where a warp then covers the row): a
// thread's share of the reductions costs half as much per column.
Shape shape_of(int H)
{
    const int nv = H / 8;
    const int vpt = nv <= 32 ? 1 : 2;
    const int per = (nv + vpt - 1) / vpt;
    return {vpt, (per + 31) / 32 * 32};
}

template <int VPT, bool F32, bool HAS_Y>
cudaError_t launch_one(const BlockNormParams &p, bool bwd, int threads, int blocks, cudaStream_t s)
{
    auto kernel = bwd ? block_norm_backward_kernel<VPT, F32, HAS_Y> : block_norm_kernel<VPT, F32, HAS_Y>;
    using B = Ring<F32, HAS_Y, true>;
    using A = Ring<F32, HAS_Y, false>;
    const size_t smem = (size_t)(bwd ? B::ROWS * B::PIECES : A::ROWS * A::PIECES) * VPT * threads * 16;
    if (smem > 40 * 1024) {      // (with the kernels' static 1.2 KB, past the 48 KB that need no opting in)
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
    }
    const cudaError_t e = launch_pdl(kernel, dim3(blocks), dim3(threads), smem, s, p);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

cudaError_t launch_any(const BlockNormParams &p, bool f32, bool bwd, int blocks, cudaStream_t s)
{
    const Shape sh = shape_of(p.H);
    const bool y = p.y != nullptr;
    if (sh.vpt == 1)
        return f32 ? (y ? launch_one<1, true, true>(p, bwd, sh.threads, blocks, s)
                        : launch_one<1, true, false>(p, bwd, sh.threads, blocks, s))
                   : (y ? launch_one<1, false, true>(p, bwd, sh.threads, blocks, s)
                        : launch_one<1, false, false>(p, bwd, sh.threads, blocks, s));
    return f32 ? (y ? launch_one<2, true, true>(p, bwd, sh.threads, blocks, s)
                    : launch_one<2, true, false>(p, bwd, sh.threads, blocks, s))
               : (y ? launch_one<2, false, true>(p, bwd, sh.threads, blocks, s)
                    : launch_one<2, false, false>(p, bwd, sh.threads, blocks, s));
}

}  // namespace

// Blocks that a launch fills the GPU with: 512 threads per SM (at the 128
// registers that the launch bounds allow, what the register file holds), so
// that a block's rows are contiguous and its weights are loaded once.
int block_norm_blocks(int T, int H, int sms)
{
    const Shape sh = shape_of(H);
    const int per_sm = 512 / sh.threads;
    const int n = sms * (per_sm < 1 ? 1 : per_sm);
    return T < n ? T : n;
}

int block_norm_cpg(int T, int groups, int blocks)
{
    const int rows = T / groups;
    int cpg = (blocks + groups - 1) / groups;
    return cpg < 1 ? 1 : cpg > rows ? rows : cpg;
}

cudaError_t launch_block_norm(const BlockNormParams &p, bool stream_f32, int blocks, cudaStream_t s)
{
    return launch_any(p, stream_f32, false, blocks, s);
}

cudaError_t launch_block_norm_backward(const BlockNormParams &p, bool stream_f32, int blocks, cudaStream_t s)
{
    return launch_any(p, stream_f32, true, blocks, s);
}

cudaError_t launch_block_norm_finish(const BlockNormParams &p, int blocks, cudaStream_t s)
{
    const cudaError_t e = launch_pdl(block_norm_finish_kernel, dim3((p.H + 31) / 32), dim3(1024), 0, s, p, blocks);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace glr
