// The router's gradient: from the gradient of the routing weights (and of the
// balance loss) to that of the logits, in the form the tensor-core products
// of pair_gemm.cu read.
//
// With s = sigmoid(L), S the chosen experts of a token and D = sum_S s + eps,
// w_j = rsf s_j / D, so  ds_j = rsf / D (dw_j - sum_i dw_i s_i / D)
//                            = rsf / D^2 (sum_i (dw_j - dw_i) s_i + dw_j eps),
// the second form without the first's cancellation (equal dw, or a single
// expert, leave eps alone).  The balance
// loss E sum_e f_e mean_t(s_te / Z_t), Z_t = sum_e s_te, f_e = counts_e / (k T)
// fixed, adds  ds_e += d_aux E / T (f_e - sum_e' f_e' s_e' / Z) / Z.  Then
// dL = ds s (1 - s), with 1 - s formed as exp(-L) s where L > 0, which keeps its
// digits near s = 1.
//
// dL is written as three bf16 parts (high, middle, low: 24 bits, as the router
// weight is split for the forward), so that the products with the bf16 hidden
// rows are exact and the gradient of the fp32 router weight keeps fp32 accuracy.
//
// One warp per token, the next token's loads in flight; 2.5 KB per token read
// and written.  Measured at T = 32768, E = 256: 22 us (0.55 of the copy rate), of
// the 232 us of the whole gradient.
#include <cuda_bf16.h>

#include "kernels.h"

namespace glr {

namespace {

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

}  // namespace

// One warp per token; a lane holds EPL = E / 32 neighbouring experts.
template <int EPL>
__global__ void __launch_bounds__(256) route_grad_kernel(const float *__restrict__ logits, int nparts,
                                                         long long stride,
                                                         const int32_t *__restrict__ idx,
                                                         const float *__restrict__ d_w,
                                                         const int32_t *__restrict__ counts,
                                                         const float *__restrict__ d_aux, int T, int k, float rsf,
                                                         float eps, uint16_t *parts, int *status)
{
    constexpr int E = EPL * 32;
    __shared__ __align__(16) float scatter[8][E];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (blockDim.x >> 5);
    float f[EPL];
    const float aux = d_aux ? *d_aux * ((float)E / (float)T) : 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        f[i] = d_aux ? (float)counts[lane * EPL + i] / ((float)k * (float)T) : 0.0f;
    // a token's logits, chosen experts and their gradients, loaded a token ahead
    float4 ahead[EPL / 4];
    int e_ahead = -1;
    float dw_ahead = 0.0f;
    auto fetch = [&](int t) {
        if (t >= T)
            return;
        const float *row = logits + (size_t)t * E + lane * EPL;
#pragma unroll
        for (int i = 0; i < EPL / 4; ++i)
            ahead[i] = reinterpret_cast<const float4 *>(row)[i];
        for (int part = 1; part < nparts; ++part)
#pragma unroll
            for (int i = 0; i < EPL / 4; ++i) {
                const float4 q = reinterpret_cast<const float4 *>(row + part * stride)[i];
                ahead[i].x += q.x; ahead[i].y += q.y; ahead[i].z += q.z; ahead[i].w += q.w;
            }
        if (lane < k) {
            e_ahead = idx[(size_t)t * k + lane];
            dw_ahead = d_w[(size_t)t * k + lane];
        }
    };
    float *mine = scatter[threadIdx.x >> 5];
    int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    fetch(t);
    for (; t < T; t += warps) {
        float L[EPL], ds[EPL], s[EPL], slope[EPL];
#pragma unroll
        for (int i = 0; i < EPL / 4; ++i) {
            L[4 * i] = ahead[i].x; L[4 * i + 1] = ahead[i].y; L[4 * i + 2] = ahead[i].z; L[4 * i + 3] = ahead[i].w;
        }
        // lane j < k: the chosen expert j
        int e = e_ahead;
        float dw = dw_ahead;
        fetch(t + warps);
        if (lane < k && (e < 0 || e >= E)) {
            atomicOr(status, ST_BAD_INDEX);
            e = -1;
        }
        if (e < 0)
            dw = 0.0f;
        float Z = 0.0f, F = 0.0f, zero = 0.0f;          // zero: 0 unless a logit is not finite
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            float x;                                  // exp(-L)
            s[i] = router_sigmoid(L[i], x);
            slope[i] = s[i] * (L[i] > 0.0f ? x * s[i] : 1.0f - s[i]);
            Z += s[i];
            F = fmaf(f[i], s[i], F);
            zero = fmaf(L[i], 0.0f, zero);
        }
        if (!__all_sync(0xffffffffu, zero == 0.0f) && lane == 0)
            atomicOr(status, ST_NONFINITE);
        // scores to the lanes whose expert they are, through shared memory; the
        // gradients back the same way
#pragma unroll
        for (int i = 0; i < EPL; i += 4)
            *reinterpret_cast<float4 *>(mine + lane * EPL + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
        __syncwarp();
        const float sj = e >= 0 ? mine[e] : 0.0f;
        const float D = warp_sum(sj) + eps;
        float dsj = dw * eps;
        for (int i = 0; i < k; ++i)
            dsj = fmaf(dw - __shfl_sync(0xffffffffu, dw, i), __shfl_sync(0xffffffffu, sj, i), dsj);
        const float per_d = __fdividef(1.0f, D);
        dsj = dsj * per_d * (rsf * per_d);
        // (an id that a token names more than once, never the router's, adds up
        // in the first lane that names it)
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const bool first = e >= 0 && __ffs(same) - 1 == lane;
        if (__any_sync(0xffffffffu, e >= 0 && !first)) {
            float sum = 0.0f;
            for (int j = 0; j < k; ++j) {
                const float v = __shfl_sync(0xffffffffu, dsj, j);
                if ((same >> j) & 1u)
                    sum += v;
            }
            dsj = sum;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < EPL; i += 4)
            *reinterpret_cast<float4 *>(mine + lane * EPL + i) = make_float4(0.f, 0.f, 0.f, 0.f);
        __syncwarp();
        if (first)
            mine[e] = dsj;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < EPL; i += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(mine + lane * EPL + i);
            ds[i] = q.x; ds[i + 1] = q.y; ds[i + 2] = q.z; ds[i + 3] = q.w;
        }
        __syncwarp();
        if (d_aux) {
            Z = warp_sum(Z);
            F = warp_sum(F);
            const float c = __fdividef(aux, Z), mean = __fdividef(F, Z);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                ds[i] = fmaf(c, f[i] - mean, ds[i]);
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            ds[i] *= slope[i];
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            uint32_t o[EPL / 2];
#pragma unroll
            for (int i = 0; i < EPL / 2; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(ds[2 * i], ds[2 * i + 1]);
                o[i] = *reinterpret_cast<const uint32_t *>(&b);
                ds[2 * i] -= __uint_as_float(o[i] << 16);
                ds[2 * i + 1] -= __uint_as_float(o[i] & 0xffff0000u);
            }
            uint16_t *dst = parts + ((size_t)q * T + t) * E + lane * EPL;
            if constexpr (EPL == 8)
                *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            else
                *reinterpret_cast<uint2 *>(dst) = make_uint2(o[0], o[1]);
        }
    }
}

__global__ void __launch_bounds__(256) sum_splits_kernel(const float *__restrict__ part, int splits, long long stride,
                                                         long long n4, float *out)
{
    pdl_wait();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n4)
        return;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
        const float4 q = __ldcs(reinterpret_cast<const float4 *>(part + s * stride) + i);
        a.x += q.x; a.y += q.y; a.z += q.z; a.w += q.w;
    }
    reinterpret_cast<float4 *>(out)[i] = a;
}

cudaError_t launch_route_grad(const float *logits, int nparts, long long part_stride, const int32_t *idx,
                              const float *d_w, const int32_t *counts, const float *d_aux, int T, int E, int k, float rsf,
                              float eps, uint16_t *parts, int *status, cudaStream_t s)
{
    const int want = (T + 7) / 8, most = 152 * 5;      // (what the SMs hold at once)
    const dim3 grid(want < most ? want : most);
    const cudaError_t e = E == 256 ? launch_pdl(route_grad_kernel<8>, grid, dim3(256), 0, s, logits, nparts, part_stride,
                                                idx, d_w, counts, d_aux, T, k, rsf, eps, parts, status)
                                   : launch_pdl(route_grad_kernel<4>, grid, dim3(256), 0, s, logits, nparts, part_stride,
                                                idx, d_w, counts, d_aux, T, k, rsf, eps, parts, status);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

cudaError_t launch_sum_splits(const float *part, int splits, long long stride, long long n, float *out,
                              cudaStream_t s)
{
    const long long n4 = n / 4;
    const cudaError_t e = launch_pdl(sum_splits_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, s, part,
                                     splits, stride, n4, out);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace glr
