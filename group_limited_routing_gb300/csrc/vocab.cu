// Vocabulary loss: the kernels around the dense products of pair_gemm.cu.
//
//   z[t, v] = <hidden_t, W_v>,  lse_t = log sum_v exp z[t, v],
//   loss_t = lse_t - z[t, target_t]
//
// The products run over the rows that count only (a target in [0, V) that is
// not the ignored one): their row numbers are packed here, and their hidden
// rows too where some row does not count, so that masked rows (prompts,
// padding) cost nothing and a NaN in one reaches no gradient.  All of these
// kernels move a few percent of the products' bytes; they are bound by launch
// and memory latency (T = 8192, V = 131072: rows 13 us, join 21 us of 2.45 ms; T = 16:
// 4 us each of 100).
#include <cuda_bf16.h>

#include "kernels.h"

namespace glr {

namespace {

__device__ __forceinline__ long long target_at(const VocabRowsParams &p, int t)
{
    return p.target_bits == 64 ? static_cast<const long long *>(p.target)[t]
                               : (long long)static_cast<const int *>(p.target)[t];
}

constexpr int ROWS_THREADS = 1024;

}  // namespace

// Which rows count, and their packed order.  Block b owns rows [b T / grid,
// (b + 1) T / grid).  It counts those before them and all of them (every block
// reads every target: a few coalesced loads per thread, and no block waits for
// another), packs its own rows behind the ones before, and, where some row of
// the batch does not count, copies its rows' hidden states side by side.  Rows
// of zeros follow up to a multiple of 64 (a K block of the weight gradient).
// Where every row counts the products read `hidden` itself.
__global__ void __launch_bounds__(ROWS_THREADS) vocab_rows_kernel(const VocabRowsParams p)
{
    __shared__ int sums[32], befores[32], own[32];
    __shared__ float tops[32];
    __shared__ int list[ROWS_THREADS];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int blocks = gridDim.x;
    const int t0 = (int)((long long)blockIdx.x * p.T / blocks), t1 = (int)((long long)(blockIdx.x + 1) * p.T / blocks);
    auto counts = [&](long long v) { return v != p.ignore && v >= 0 && v < p.V; };
    int n = 0, before = 0;
    bool bad = false;
    float top = 0.0f;
#pragma unroll 8
    for (int t = threadIdx.x; t < p.T; t += ROWS_THREADS) {
        const long long v = target_at(p, t);
        const bool c = counts(v);
        const float g = p.d_loss ? fabsf(p.d_loss[t]) : 0.0f;
        bad |= !c && v != p.ignore;
        n += c;
        before += c && t < t0;
        if (c)
            top = g > top || g != g ? g : top;          // a NaN stays
    }
    if (bad && blockIdx.x == 0)
        atomicOr(p.status, ST_BAD_TARGET);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        n += __shfl_xor_sync(0xffffffffu, n, off);
        before += __shfl_xor_sync(0xffffffffu, before, off);
        const float f = __shfl_xor_sync(0xffffffffu, top, off);
        top = f > top || f != f ? f : top;
    }
    if (lane == 0) {
        sums[w] = n;
        befores[w] = before;
        tops[w] = top;
    }
    __syncthreads();
    // (each warp for itself: lane i takes warp i's sums)
    n = sums[lane];
    before = befores[lane];
    top = tops[lane];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        n += __shfl_xor_sync(0xffffffffu, n, off);
        before += __shfl_xor_sync(0xffffffffu, before, off);
        const float f = __shfl_xor_sync(0xffffffffu, top, off);
        top = f > top || f != f ? f : top;
    }
    const int total = n;
    const float scale = top > 0.0f && top < INFINITY ? top : 1.0f;
    const bool twice = p.packed_of && total <= VOCAB_TWICE_ROWS;
    const int rows = twice ? 2 * total : total;
    const bool packed = twice || total < p.T;
    if (blockIdx.x == 0 && w == 0) {
        if (lane == 0) {
            p.meta->rows = rows;
            p.meta->counted = total;
            p.meta->packed = packed;
            p.meta->scale = scale;
        }
        if (p.packed_of) {
            // choose_splits, a candidate per lane
            const int c = lane + 1, tiles = (rows + 255) / 256 * ((p.H + 255) / 256);
            const bool may = c <= VOCAB_MAX_SPLITS && may_split(tiles, p.dx_kblocks, c, VOCAB_MIN_SPLIT_BLOCKS);
            long long key = may ? split_cost(tiles, p.dx_kblocks, (long long)rows * p.H, c) * 64 + c
                                : 0x7fffffffffffffffll;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                key = min(key, __shfl_xor_sync(0xffffffffu, key, off));
            if (lane == 0)
                p.meta->splits = (int)(key & 63);
        }
    }
    const int nv = p.H / 8;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.hidden);
    uint4 *dst = reinterpret_cast<uint4 *>(p.packed);
    for (int first = t0; first < t1; first += ROWS_THREADS) {
        const int t = first + threadIdx.x;
        const long long v = t < t1 ? target_at(p, t) : p.ignore;
        const bool c = t < t1 && counts(v);
        const unsigned mask = __ballot_sync(0xffffffffu, c);
        __syncthreads();                                 // (the pass before has read own and list)
        if (lane == 0)
            own[w] = __popc(mask);
        __syncthreads();
        int mine = own[lane];                            // the warps' sums: inclusive scan over the lanes
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, mine, off);
            if (lane >= off)
                mine += o;
        }
        const int here = __shfl_sync(0xffffffffu, mine, 31);
        const int rank = (w ? __shfl_sync(0xffffffffu, mine, w - 1) : 0) + __popc(mask & ((1u << lane) - 1u));
        const int q = before + rank;
        if (t < t1 && p.packed_of)
            p.packed_of[t] = c ? q : -1;
        if (c) {
            list[rank] = t;
            p.row_of[q] = t;
            p.packed_target[q] = (int)v;
            if (p.d_loss) {
                p.packed_lse[q] = p.lse[t];
                p.packed_weight[q] = p.d_loss[t] / scale;
                if (twice) {
                    p.packed_target[total + q] = (int)v;
                    p.packed_lse[total + q] = p.lse[t];
                    p.packed_weight[total + q] = p.d_loss[t] / scale;
                }
            }
        } else if (t < t1 && p.loss) {
            p.loss[t] = 0.0f;
            p.lse_out[t] = 0.0f;
        }
        __syncthreads();
        if (packed)
            for (int i = w; i < here; i += 32) {
                const size_t from = (size_t)list[i] * nv, to = (size_t)(before + i) * nv;
                for (int v0 = lane; v0 < nv; v0 += 8 * 32) {
                    uint4 q8[8];                         // (loads before stores: the compiler may not assume it)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (v0 + 32 * j < nv)
                            q8[j] = __ldcs(src + from + v0 + 32 * j);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (v0 + 32 * j < nv)
                            dst[to + v0 + 32 * j] = q8[j];
                    if (twice)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (v0 + 32 * j < nv)
                                dst[to + (size_t)total * nv + v0 + 32 * j] = q8[j];
                }
            }
        before += here;
    }
    if (packed)
        for (int q = rows + blockIdx.x; q < min(p.packed_rows, (rows + 63) / 64 * 64); q += blocks)
            for (int v = threadIdx.x; v < nv; v += ROWS_THREADS)
                dst[(size_t)q * nv + v] = make_uint4(0, 0, 0, 0);
}

// Joins the 128-column blocks' softmax statistics of each row.  A block takes R
// rows and shares their column blocks among its 1024 / R threads per row, so
// that a few rows' many statistics are loaded at once too.  The bases are
// log2 values, so the sums are over powers of two; pairs are joined in a fixed
// order (a thread's own in column order, then lanes, then warps by halves).
template <int R>
__global__ void __launch_bounds__(1024) vocab_join_kernel(const float2 *__restrict__ stats, int nstats, int ld,
                                                          const float *__restrict__ target_logit,
                                                          const VocabMeta *meta, const int *row_of, float *loss,
                                                          float *lse)
{
    constexpr int SHARE = 1024 / R;
    __shared__ float2 sm[R][33];
    pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int r = threadIdx.x % R, part = threadIdx.x / R;
    const int rows = meta->rows;               // (forward: rows that count)
    const bool in = (int)blockIdx.x * R + r < rows;
    auto join = [](float2 a, float2 b) {
        const float top = fmaxf(a.x, b.x);
        if (!(top > -INFINITY))
            return a;
        return make_float2(top, a.y * exp2f(a.x - top) + b.y * exp2f(b.x - top));
    };
    auto halves = [&](float2 a, int from, int to) {
        for (int off = from; off >= to; off >>= 1)
            a = join(a, make_float2(__shfl_xor_sync(0xffffffffu, a.x, off), __shfl_xor_sync(0xffffffffu, a.y, off)));
        return a;
    };
    float2 acc = make_float2(-INFINITY, 0.0f);
    if (in)
        for (int i = part; i < nstats; i += 4 * SHARE) {
            float2 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = i + j * SHARE < nstats ? stats[(size_t)(i + j * SHARE) * ld + blockIdx.x * R + r]
                                              : make_float2(-INFINITY, 0.0f);
            acc = join(acc, join(join(v[0], v[1]), join(v[2], v[3])));
        }
    acc = halves(acc, 16, R);              // the warp's threads of one row
    if (lane < R)
        sm[lane][w] = acc;
    __syncthreads();
    const int row = blockIdx.x * R + w;    // warp w < R: the warps' sums of row w
    if (w >= R || row >= rows)
        return;
    acc = halves(sm[w][lane], 16, 1);
    if (lane == 0) {
        const float l = (acc.x + log2f(acc.y)) * 0.69314718055994531f;
        const int t = row_of[row];
        lse[t] = l;
        loss[t] = l - target_logit[row];
    }
}

// d_hidden[t] = bf16( scale sum_s part[s][packed row of t] ), zero where the
// row does not count.  Splits in order; a low part's sums after the high part's.
__global__ void __launch_bounds__(128) vocab_dx_join_kernel(const float *__restrict__ part, const VocabMeta *meta,
                                                            const int *packed_of, int T, int H, uint16_t *d_hidden)
{
    pdl_wait();
    const float scale = meta->scale;
    const int splits = meta->splits;
    const int counted = meta->counted, twice = meta->rows > counted;
    const size_t split_stride = (size_t)((meta->rows + 255) / 256 * 256) * H;
    const int nv = H / 8;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        const int r = packed_of[t];
        for (int v = threadIdx.x; v < nv; v += blockDim.x) {
            float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (r >= 0)
                for (int s = 0; s < splits << twice; ++s) {
                    const bool low = s >= splits;
                    const size_t at = (low ? s - splits : s) * split_stride + (size_t)(low ? r + counted : r) * H;
                    const float4 *q = reinterpret_cast<const float4 *>(part + at) + 2 * v;
                    const float4 a = __ldcs(q), b = __ldcs(q + 1);
                    f[0] += a.x; f[1] += a.y; f[2] += a.z; f[3] += a.w;
                    f[4] += b.x; f[5] += b.y; f[6] += b.z; f[7] += b.w;
                }
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i] * scale, f[2 * i + 1] * scale);
                o[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
            reinterpret_cast<uint4 *>(d_hidden)[(size_t)t * nv + v] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

cudaError_t launch_vocab_rows(const VocabRowsParams &p, cudaStream_t s)
{
    // an SM per block at most, and a block per eight rows: copying is spread,
    // counting is not worth more blocks
    const int want = (p.T + 7) / 8;
    const cudaError_t e = launch_pdl(vocab_rows_kernel, dim3(want < 152 ? want : 152), dim3(ROWS_THREADS), 0, s, p);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

cudaError_t launch_vocab_join(const float2 *stats, int nstats, int ld, const float *target_logit,
                              const VocabMeta *meta, const int *row_of, int T, float *loss, float *lse,
                              cudaStream_t s)
{
    // 32 rows per block read whole lines; fewer rows than fill the SMs so are
    // spread, four to a block
    const cudaError_t e = T > 2048 ? launch_pdl(vocab_join_kernel<32>, dim3((T + 31) / 32), dim3(1024), 0, s, stats,
                                                nstats, ld, target_logit, meta, row_of, loss, lse)
                                   : launch_pdl(vocab_join_kernel<4>, dim3((T + 3) / 4), dim3(1024), 0, s, stats,
                                                nstats, ld, target_logit, meta, row_of, loss, lse);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

cudaError_t launch_vocab_dx_join(const float *part, const VocabMeta *meta, const int *packed_of, int T, int H,
                                 uint16_t *d_hidden, cudaStream_t s)
{
    const int blocks = T < 2432 ? T : 2432;
    const cudaError_t e = launch_pdl(vocab_dx_join_kernel, dim3(blocks), dim3(128), 0, s, part, meta,
                                     packed_of, T, H, d_hidden);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace glr
