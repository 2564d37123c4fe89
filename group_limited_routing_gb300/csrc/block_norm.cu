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
// CTA holds one row, eight columns (16 bytes of bf16) per thread and vector,
// so a row's values stay in registers between the two reductions that it
// needs, and the next row's loads are issued before this row's reductions.
#include <cuda_bf16.h>

#include "kernels.h"

namespace glr {

namespace {

constexpr int BN_MAX_WARPS = 16;

__device__ __forceinline__ void unpack8(const uint4 &q, float *f)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// eight consecutive values of a row as loaded: 16 bytes of bf16 or 32 of fp32
template <bool F32>
struct Raw8;

template <>
struct Raw8<false> {
    uint4 a;
    __device__ __forceinline__ void load(const void *p, size_t i) { a = __ldcs(static_cast<const uint4 *>(p) + i); }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float *f) const { unpack8(a, f); }
    static __device__ __forceinline__ void store(void *p, size_t i, const float *f)
    {
        static_cast<uint4 *>(p)[i] = pack8(f);
    }
};

template <>
struct Raw8<true> {
    float4 a, b;
    __device__ __forceinline__ void load(const void *p, size_t i)
    {
        a = __ldcs(static_cast<const float4 *>(p) + 2 * i);
        b = __ldcs(static_cast<const float4 *>(p) + 2 * i + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float *f) const
    {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    static __device__ __forceinline__ void store(void *p, size_t i, const float *f)
    {
        static_cast<float4 *>(p)[2 * i] = make_float4(f[0], f[1], f[2], f[3]);
        static_cast<float4 *>(p)[2 * i + 1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// Sums of N values over the block, the same bits in every thread (warp sums by
// butterfly, then the warps' sums in warp order).  `slot` alternates between
// calls, so one barrier per call suffices: a slot is written again only after
// the barrier of the call between, which every reader of it has passed.
template <int N>
__device__ __forceinline__ void block_sums(float *v, float (*sm)[BN_MAX_WARPS][N], int &slot)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    const int nw = blockDim.x >> 5;
    if (nw == 1)
        return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            sm[slot][threadIdx.x >> 5][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = 0.0f;
    for (int w = 0; w < nw; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += sm[slot][w][i];
    slot ^= 1;
}

// gate * w_post for this thread's columns (NULL: 1)
__device__ __forceinline__ void load_vec(const float *w, int v, float *f)
{
    if (!w) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = 1.0f;
        return;
    }
    const float4 a = __ldg(reinterpret_cast<const float4 *>(w) + 2 * v);
    const float4 b = __ldg(reinterpret_cast<const float4 *>(w) + 2 * v + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

template <int VPT>
__device__ __forceinline__ void load_gw(const BlockNormParams &p, int group, int nv, float (*gw)[8])
{
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        if (v >= nv)
            continue;
        float g[8], w[8];
        load_vec(p.gate ? p.gate + (size_t)group * p.H : nullptr, v, g);
        load_vec(p.w_post, v, w);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            gw[k][i] = g[i] * w[i];
    }
}

}  // namespace

// Rows [b T / grid, (b + 1) T / grid) of block b.
template <int VPT, bool F32, bool HAS_Y>
__global__ void __launch_bounds__(512) block_norm_kernel(const BlockNormParams p)
{
    __shared__ float sm[2][BN_MAX_WARPS][1];
    pdl_wait();
    const int nv = p.H / 8;
    const int row0 = (int)((long long)blockIdx.x * p.T / gridDim.x);
    const int row1 = (int)((long long)(blockIdx.x + 1) * p.T / gridDim.x);
    const float inv_h = 1.0f / (float)p.H;
    int slot = 0, group = -1;
    float gw[VPT][8], wpre[VPT][8];
    Raw8<F32> xr[VPT];
    Raw8<false> yr[VPT];
    auto fetch = [&](int row) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            xr[k].zero();
            yr[k].zero();
            if (v < nv) {
                xr[k].load(p.x, (size_t)row * nv + v);
                if (HAS_Y)
                    yr[k].load(p.y, (size_t)row * nv + v);
            }
        }
    };
    if (row0 < row1)
        fetch(row0);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            gw[k][i] = 0.0f, wpre[k][i] = 0.0f;
        if (v < nv)
            load_vec(p.w_pre, v, wpre[k]);
    }
    for (int row = row0; row < row1; ++row) {
        if (HAS_Y && row / p.rows_per_gate != group) {
            group = row / p.rows_per_gate;
            load_gw<VPT>(p, group, nv, gw);
        }
        float r[VPT][8], y[VPT][8];
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            xr[k].get(r[k]);
            if (HAS_Y) {
                yr[k].get(y[k]);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s[0] = fmaf(y[k][i], y[k][i], s[0]);
            }
        }
        if (row + 1 < row1)
            fetch(row + 1);
        float rho = 0.0f;
        if (HAS_Y) {
            block_sums<1>(s, sm, slot);
            rho = 1.0f / sqrtf(s[0] * inv_h + p.eps);
        }
        s[0] = 0.0f;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                r[k][i] = HAS_Y ? fmaf(p.alpha, r[k][i], gw[k][i] * (y[k][i] * rho)) : p.alpha * r[k][i];
                s[0] = fmaf(r[k][i], r[k][i], s[0]);
            }
        block_sums<1>(s, sm, slot);
        const float sigma = 1.0f / sqrtf(s[0] * inv_h + p.eps);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v >= nv)
                continue;
            if (p.r)
                Raw8<F32>::store(p.r, (size_t)row * nv + v, r[k]);
            float n[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                n[i] = r[k][i] * sigma * wpre[k][i];
            Raw8<false>::store(p.n, (size_t)row * nv + v, n);
        }
    }
}

// Chunk c holds rows of one gate group only: group c / cpg, its part c % cpg of
// cpg.  Block b takes chunks [b C / grid, (b + 1) C / grid).  Per chunk it
// leaves A[c] = sum_t dr u (the finish kernel's d_gate and dw_post), and per
// block B[b] = sum_t d_n q (dw_pre).
template <int VPT, bool F32, bool HAS_Y>
__global__ void __launch_bounds__(512) block_norm_backward_kernel(const BlockNormParams p)
{
    __shared__ float sm1[2][BN_MAX_WARPS][1];
    __shared__ float sm5[2][BN_MAX_WARPS][5];
    pdl_wait();
    const int nv = p.H / 8;
    const float inv_h = 1.0f / (float)p.H;
    const int chunks = p.groups * p.cpg;
    const int c0 = (int)((long long)blockIdx.x * chunks / gridDim.x);
    const int c1 = (int)((long long)(blockIdx.x + 1) * chunks / gridDim.x);
    auto chunk_begin = [&](int c) {
        return (c / p.cpg) * p.rows_per_gate + (int)((long long)(c % p.cpg) * p.rows_per_gate / p.cpg);
    };
    int slot1 = 0, slot5 = 0;
    float gw[VPT][8], wpre[VPT][8], accA[VPT][8], accB[VPT][8];
    Raw8<F32> xr[VPT], drr[VPT];
    Raw8<false> yr[VPT], dnr[VPT];
    auto fetch = [&](int row) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            xr[k].zero();
            yr[k].zero();
            drr[k].zero();
            dnr[k].zero();
            if (v < nv) {
                const size_t at = (size_t)row * nv + v;
                if (HAS_Y)
                    yr[k].load(p.y, at);
                xr[k].load(p.x, at);
                dnr[k].load(p.d_n, at);
                if (p.d_r)
                    drr[k].load(p.d_r, at);
            }
        }
    };
    const int row_end = chunk_begin(c1);   // (chunks are contiguous)
    if (c0 < c1)
        fetch(chunk_begin(c0));
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            gw[k][i] = 0.0f, wpre[k][i] = 0.0f, accB[k][i] = 0.0f;
        if (v < nv)
            load_vec(p.w_pre, v, wpre[k]);
    }
    for (int c = c0; c < c1; ++c) {
        const int begin = chunk_begin(c), end = chunk_begin(c + 1);
        if (HAS_Y && (c == c0 || c % p.cpg == 0))
            load_gw<VPT>(p, c / p.cpg, nv, gw);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                accA[k][i] = 0.0f;
        for (int row = begin; row < end; ++row) {
            float r[VPT][8], u[VPT][8], dr[VPT][8], dn[VPT][8];
            float s[1] = {0.0f};
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                xr[k].get(r[k]);
                drr[k].get(dr[k]);
                dnr[k].get(dn[k]);
                if (HAS_Y) {
                    yr[k].get(u[k]);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        s[0] = fmaf(u[k][i], u[k][i], s[0]);
                }
            }
            if (row + 1 < row_end)
                fetch(row + 1);
            float rho = 0.0f;
            if (HAS_Y) {
                block_sums<1>(s, sm1, slot1);
                rho = 1.0f / sqrtf(s[0] * inv_h + p.eps);
            }
            // sum r^2, sum dq r, and the three parts of sum du u
            float t[5] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float dq = dn[k][i] * wpre[k][i];
                    if (HAS_Y) {
                        u[k][i] *= rho;
                        const float a = gw[k][i] * u[k][i];
                        r[k][i] = fmaf(p.alpha, r[k][i], a);
                        t[2] = fmaf(a, dr[k][i], t[2]);
                        t[3] = fmaf(a, dq, t[3]);
                        t[4] = fmaf(a, r[k][i], t[4]);
                    } else {
                        r[k][i] *= p.alpha;
                    }
                    t[0] = fmaf(r[k][i], r[k][i], t[0]);
                    t[1] = fmaf(dq, r[k][i], t[1]);
                }
            block_sums<5>(t, sm5, slot5);
            const float sigma = 1.0f / sqrtf(t[0] * inv_h + p.eps);
            // dr = d_r + sigma dq - (sigma^3 mean(dq r)) r
            const float c_r = sigma * sigma * sigma * (t[1] * inv_h);
            const float c_u = (t[2] + sigma * t[3] - c_r * t[4]) * inv_h;   // mean(du u)
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = threadIdx.x + k * blockDim.x;
                float dx[8], dy[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float q = r[k][i] * sigma;
                    accB[k][i] = fmaf(dn[k][i], q, accB[k][i]);
                    const float g = fmaf(-c_r, r[k][i], fmaf(sigma, dn[k][i] * wpre[k][i], dr[k][i]));
                    dx[i] = p.alpha * g;
                    if (HAS_Y) {
                        accA[k][i] = fmaf(g, u[k][i], accA[k][i]);
                        dy[i] = rho * fmaf(-c_u, u[k][i], g * gw[k][i]);
                    }
                }
                if (v < nv) {
                    Raw8<F32>::store(p.d_x, (size_t)row * nv + v, dx);
                    if (HAS_Y)
                        Raw8<false>::store(p.d_y, (size_t)row * nv + v, dy);
                }
            }
        }
        if (HAS_Y)
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = threadIdx.x + k * blockDim.x;
                if (v < nv)
                    Raw8<true>::store(p.part_a, (size_t)c * nv + v, accA[k]);
            }
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        if (v < nv)
            Raw8<true>::store(p.part_b, (size_t)blockIdx.x * nv + v, accB[k]);
    }
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

// Eight columns per thread up to H = 4096, sixteen up to BLOCK_NORM_MAX_H.
Shape shape_of(int H)
{
    const int nv = H / 8;
    const int vpt = nv <= 512 ? 1 : 2;
    const int per = (nv + vpt - 1) / vpt;
    return {vpt, (per + 31) / 32 * 32};
}

template <int VPT, bool BWD>
auto pick(bool f32, bool has_y)
{
    if constexpr (BWD)
        return f32 ? (has_y ? block_norm_backward_kernel<VPT, true, true> : block_norm_backward_kernel<VPT, true, false>)
                   : (has_y ? block_norm_backward_kernel<VPT, false, true>
                            : block_norm_backward_kernel<VPT, false, false>);
    else
        return f32 ? (has_y ? block_norm_kernel<VPT, true, true> : block_norm_kernel<VPT, true, false>)
                   : (has_y ? block_norm_kernel<VPT, false, true> : block_norm_kernel<VPT, false, false>);
}

}  // namespace

// Blocks that a launch fills the GPU with: as many as the register file of the
// SMs holds of this shape (the kernels' launch bounds keep them at 128
// registers per thread at most), so that a block's rows are contiguous and its
// weights are loaded once.
int block_norm_blocks(int T, int H, int sms)
{
    const Shape sh = shape_of(H);
    const int per_sm = sh.threads <= 32 ? 16 : 512 / sh.threads;
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
    const Shape sh = shape_of(p.H);
    auto k = sh.vpt == 1 ? pick<1, false>(stream_f32, p.y != nullptr) : pick<2, false>(stream_f32, p.y != nullptr);
    const cudaError_t e = launch_pdl(k, dim3(blocks), dim3(sh.threads), 0, s, p);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

cudaError_t launch_block_norm_backward(const BlockNormParams &p, bool stream_f32, int blocks, cudaStream_t s)
{
    const Shape sh = shape_of(p.H);
    auto k = sh.vpt == 1 ? pick<1, true>(stream_f32, p.y != nullptr) : pick<2, true>(stream_f32, p.y != nullptr);
    const cudaError_t e = launch_pdl(k, dim3(blocks), dim3(sh.threads), 0, s, p);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

cudaError_t launch_block_norm_finish(const BlockNormParams &p, int blocks, cudaStream_t s)
{
    const cudaError_t e = launch_pdl(block_norm_finish_kernel, dim3((p.H + 31) / 32), dim3(1024), 0, s, p, blocks);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace glr
