// The AdamW step over many tensors in one launch, with states in fp32 or in 8
// bits, and the global norm of the gradients (SIMT, sm_103a).
//
//   m <- beta1 m + (1 - beta1) g,  v <- beta2 v + (1 - beta2) g^2
//   p <- p (1 - lr decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// in fp32, each operation correctly rounded by itself in this order (no fused
// multiply-adds), so that the results do not depend on how a compiler groups them: an
// ulp would put a few of the values that are then rounded stochastically on the other
// side of a border.  (A quotient under 2^-126 is not rounded to a subnormal number.)
//
// 8-bit states hold m and sqrt(v) as e4m3 with a power-of-two scale for each 128
// elements.  The root halves the range of v's exponents: within a block e4m3
// reaches down to 2^-18 of the largest root.  Rounding is stochastic (up with the
// probability of the fraction): a moving average whose steps are smaller than
// half a step of the format would otherwise stand still.  A root that is not zero is
// never stored as zero, or a state that rounded down would divide by eps alone.
// A bf16 parameter without fp32 master weights is rounded stochastically for the
// same reason.  The random bits are a hash of the element's index, the tensor's
// ordinal, the step and a seed, so a step is reproducible.
//
// With fp32 states the step is bound by memory: per element the parameter, the gradient
// and the states, read and written once; with 8-bit states by the instructions an element
// takes (adamw_kernel).  A warp takes 512 elements of one tensor, all
// of whose loads it issues before the first is used.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "expert_ops.h"
#include "kernels.h"
#include "scaled_convert.cuh"

namespace glr {

namespace {

constexpr int K_S8 = 1, K_PB = 2, K_GB = 4, K_MASTER = 8, K_VEC = 16;
constexpr int ADAM_THREADS = 128;
constexpr int WARP_UNIT = ADAM_UNIT / (ADAM_THREADS / 32);      // a warp's elements

struct Step {
    float b1, one_b1, b2, one_b2, eps, size, inv, scale, one;
    float decay;
    bool scaled, plain;
    uint32_t step_key;
};

// Two fp32 values in one register pair: one instruction for both.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 of(F2 p)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
// a + b of a product a, with one = 1 that the compiler does not know: the assembler makes
// one instruction of mul.rn.f32x2 and add.rn.f32x2, with one rounding
__device__ __forceinline__ F2 add2_apart(F2 a, F2 b, F2 one) { return fma2(a, one, b); }
__device__ __forceinline__ F2 add2_cut(F2 a, F2 b)
{
    F2 r;
    asm("add.rz.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 sub2(F2 a, F2 b)
{
    F2 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ float rsqrt_approx(float x)
{
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Correctly rounded square roots of two values under 2^62, by Goldschmidt's iteration
// with the correction of Markstein (1990): from y = 1 / sqrt(x) to 2^-22, g = x y and
// h = y / 2 are refined together, then the residual x - g^2, exact in a fused
// multiply-add, times h corrects g.  It all happens at 2^64 times the value, whose
// residual does not underflow (2^-126 more for the rsqrt is nothing there, but keeps
// zero's finite); a value past 2^64 gives NaN or is past 2^32.
__device__ __forceinline__ F2 root2(F2 v)
{
    const F2 x = mul2(v, f2(0x1p64f));
    const float2 a = of(add2(x, f2(0x1p-126f)));
    const F2 y = f2(rsqrt_approx(a.x), rsqrt_approx(a.y));
    F2 g = mul2(x, y), h = mul2(y, f2(-0.5f));
    const F2 r = fma2(g, h, f2(0.5f));
    g = fma2(g, r, g);
    h = fma2(h, r, h);
    return mul2(fma2(fma2(g, g, mul2(x, f2(-1.0f))), h, g), f2(0x1p-32f));
}

// Correctly rounded m / -a of two values each (Markstein 1990): a reciprocal refined
// until it is the rounded one, then the quotient corrected by its exact residual.
// 2^-85 <= |m| < 2^74 or m = 0, 2^-50 <= -a < 2^41.
__device__ __forceinline__ F2 quotient2(F2 m, F2 a)
{
    const float2 n = of(a);
    F2 z = f2(rcp_approx(-n.x), rcp_approx(-n.y));
    z = fma2(z, fma2(a, z, f2(1.0f)), z);
    const F2 q = mul2(m, z);
    return fma2(fma2(a, q, m), z, q);
}

// Both for any value (the zeros of a gradient that never came are common).
__device__ __forceinline__ float root_of(float v)
{
    const float r = __fsqrt_rn(v == 0.0f ? 1.0f : v);
    return v == 0.0f ? v : r;
}
__device__ __forceinline__ float quotient(float m, float den)
{
    const bool zero = m == 0.0f && den > 0.0f;
    const float q = __fdiv_rn(zero ? 1.0f : m, zero ? 1.0f : den);
    return zero ? m : q;
}

// Odd multipliers from the fractional parts of the golden ratio and of the square
// roots of 2 and 3.
// start: the element's index times the first of them, plus the key
__device__ __forceinline__ uint32_t random_bits(uint32_t start)
{
    uint32_t x = start;
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x ^ (x >> 16);
}

// V elements at element i behind `base`, of which `left` exist: fp32, or bf16 as
// patterns, two to a word (those past the end are zero).  WHOLE: all exist and lie on
// a 16-byte boundary (four bf16: 8 bytes).
template <int V, bool BF16, bool WHOLE>
__device__ __forceinline__ void load(const void *base, int i, int left, uint32_t (&f)[V])
{
    if (BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(base) + i;
        if (WHOLE && V == 8) {
            const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
            f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
        } else if (WHOLE) {
            const uint2 u = __ldcs(reinterpret_cast<const uint2 *>(p));
            f[0] = u.x, f[1] = u.y;
        } else {
#pragma unroll
            for (int q = 0; q < V / 2; ++q)
                f[q] = (2 * q < left ? (uint32_t)p[2 * q] : 0u) | (2 * q + 1 < left ? (uint32_t)p[2 * q + 1] << 16 : 0u);
        }
    } else {
        const uint32_t *p = static_cast<const uint32_t *>(base) + i;
#pragma unroll
        for (int q = 0; q < V; q += 4) {
            if (WHOLE) {
                const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p + q));
                f[q] = u.x, f[q + 1] = u.y, f[q + 2] = u.z, f[q + 3] = u.w;
            } else {
#pragma unroll
                for (int j = q; j < q + 4; ++j)
                    f[j] = j < left ? p[j] : 0u;
            }
        }
    }
}

// elements 2 h and 2 h + 1
template <int V, bool BF16>
__device__ __forceinline__ F2 pair_of(const uint32_t (&f)[V], int h)
{
    return BF16 ? f2(__uint_as_float(f[h] << 16), __uint_as_float(f[h] & 0xffff0000u))
                : f2(__uint_as_float(f[(2 * h) % V]), __uint_as_float(f[(2 * h + 1) % V]));
}

template <int V, bool WHOLE>
__device__ __forceinline__ void store(void *base, int i, int left, const float (&f)[V])
{
    float *p = static_cast<float *>(base) + i;
#pragma unroll
    for (int q = 0; q < V; q += 4) {
        if (WHOLE) {
            __stcs(reinterpret_cast<float4 *>(p + q), make_float4(f[q], f[q + 1], f[q + 2], f[q + 3]));
        } else {
#pragma unroll
            for (int j = q; j < q + 4; ++j)
                if (j < left)
                    p[j] = f[j];
        }
    }
}

// words of two 16-bit patterns
template <int V, bool WHOLE>
__device__ __forceinline__ void store_bf16(void *base, int i, int left, const uint32_t (&w)[V / 2])
{
    uint16_t *p = static_cast<uint16_t *>(base) + i;
    if (WHOLE && V == 8) {
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2 % (V / 2)], w[3 % (V / 2)]));
    } else if (WHOLE) {
        __stcs(reinterpret_cast<uint2 *>(p), make_uint2(w[0], w[1]));
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < left)
                p[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
    }
}

// 8 bytes
template <bool WHOLE>
__device__ __forceinline__ uint2 load_bytes(const void *base, int i, int left)
{
    const uint8_t *p = static_cast<const uint8_t *>(base) + i;
    if (WHOLE)
        return __ldcs(reinterpret_cast<const uint2 *>(p));
    uint32_t u[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < left)
            u[j / 4] |= (uint32_t)p[j] << (8 * (j & 3));
    return make_uint2(u[0], u[1]);
}

template <bool WHOLE>
__device__ __forceinline__ void store_bytes(void *base, int i, int left, uint2 u)
{
    uint8_t *p = static_cast<uint8_t *>(base) + i;
    if (WHOLE) {
        __stcs(reinterpret_cast<uint2 *>(p), u);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left)
                p[j] = (uint8_t)((j < 4 ? u.x : u.y) >> (8 * (j & 3)));
    }
}

// 4 e4m3 values, exactly
__device__ __forceinline__ void unpack_e4m3(uint32_t u, float *f)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> (16 * h)), __NV_E4M3);
        const float2 v = __half22float2(__half2(r));
        f[2 * h] = v.x;
        f[2 * h + 1] = v.y;
    }
}

// 2^(b - 127); infinity for 255 (whose values are NaN, and so are their products)
__device__ __forceinline__ float scale_value(uint32_t b)
{
    return __uint_as_float(max(b << 23, 0x00400000u));
}

// the largest magnitude, or NaN if one is
template <int V>
__device__ __forceinline__ float largest(const float (&x)[V])
{
    float t = x[0];
#pragma unroll
    for (int i = 1; i < V; i += 2)
        asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(t) : "f"(fabsf(t)), "f"(fabsf(x[i])), "f"(fabsf(x[(i + 1) % V])));
    return t;
}

// What the scale of a block follows from, in 9 bits and in order of the magnitude:
// block_scale's byte is the key - 9 (0 at least); 0 for zero, 511 for an infinity or a
// NaN.  (A carry out of the mantissa past 0.875.)
__device__ __forceinline__ uint32_t scale_key(float t)
{
    const uint32_t top = __float_as_uint(t);
    return top >= 0x7f800000u ? 511u : top ? ((top + 0x1fffffu) >> 23) + 1u : 0u;
}

// Two t (|t| <= 448) to the e4m3 grid, away from zero where the fraction of a step
// exceeds 1 - u (v = u 2^-23): the largest multiple of the step at most |t| + u
// step.  `far` is 2^23 steps (the step is an eighth of the power of two at or below
// |t|, which counts as 2^-6 at least: the grid is even below), of t's sign: added to
// it fp32 holds whole steps, cut towards zero, which is the floor.
template <bool ROOT>
__device__ __forceinline__ float2 round_e4m3(F2 t, F2 v)
{
    const float2 x = of(t);
    auto beyond = [](float f) {
        const uint32_t b = __float_as_uint(f), e = max((b & 0x7f800000u) + (20u << 23), 141u << 23);
        return __uint_as_float(ROOT ? e : e | (b & 0x80000000u));
    };
    const F2 far = f2(beyond(x.x), beyond(x.y));
    float2 q = of(sub2(add2_cut(fma2(v, far, t), far), far));
    if (ROOT) {                                  // (one that is not zero stays so)
        if (x.x > 0.0f)
            q.x = fmaxf(q.x, 0x1p-9f);
        if (x.y > 0.0f)
            q.y = fmaxf(q.y, 0x1p-9f);
    }
    return q;
}

__device__ __forceinline__ uint32_t pack_e4m3(const float *f)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Eight of a block's values as 8 bits with the scale of its key, rounded by the low
// (m) or high (ROOT) half of each element's random bits (tiny: 2^-16).
template <bool ROOT>
__device__ __forceinline__ void quantize(const float (&x)[8], const uint32_t (&bits)[8], uint32_t key, F2 tiny, uint2 &q,
                                         uint32_t &scale)
{
    scale = (uint32_t)max((int)key - 9, 0);
    if (key - 1u >= 256u) {                      // zeros, an infinity or a NaN
        scale = key ? 255u : 127u;
        q = key ? make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu) : make_uint2(0u, 0u);
        return;
    }
    const F2 mul = f2(__uint_as_float(0x7f000000u - scale * (1u << 23)));
    float r[8];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        // 2^-16 + u 2^-23: fp32's last place there is 2^-39
        uint32_t f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            f[i] = ROOT ? __byte_perm(bits[2 * h + i], 0x3780u, 0x5432) : (bits[2 * h + i] & 0xffffu) | 0x37800000u;
        const F2 v = sub2(f2(__uint_as_float(f[0]), __uint_as_float(f[1])), tiny);
        const float2 c = round_e4m3<ROOT>(mul2(f2(x[2 * h], x[2 * h + 1]), mul), v);
        r[2 * h] = c.x;
        r[2 * h + 1] = c.y;
    }
    q = make_uint2(pack_e4m3(r), pack_e4m3(r + 4));
}

// A warp's elements, V to a lane at a time: four, or with 8-bit states eight, so that 16
// lanes hold a block of 128 and what belongs to a block (its scales, their keys) is
// done once for eight elements.
// WHOLE: all of them exist, on vector boundaries.  FAST: by root2 and quotient2; the
// result has a bit for each piece with a value that these are not for, of which nothing
// is written.  Otherwise the pieces of `pieces`, any value.
template <int KIND, bool WHOLE, bool FAST>
__device__ __forceinline__ uint32_t step_unit(const AdamTensor &t, const Step &c, long long i0, uint32_t pieces)
{
    constexpr bool S8 = KIND & K_S8, PB = KIND & K_PB, GB = KIND & K_GB, MASTER = KIND & K_MASTER;
    constexpr int V = S8 ? 8 : 4, PIECES = WARP_UNIT / (32 * V);
    const int lane = threadIdx.x & 31;
    // the lane's first element of each tensor; everything else is a constant away
    const long long il = i0 + V * lane;
    const int rest = WHOLE ? 0 : (int)min(t.n - il, (long long)ADAM_UNIT);
    const int there = WHOLE ? 0 : (int)min(t.n - i0, (long long)ADAM_UNIT);      // from the warp's first
    auto at = [il](auto *q, int size) { return (char *)q + il * size; };
    const char *pg = at(t.g, GB ? 2 : 4);
    char *pw = MASTER ? at(t.master, 4) : nullptr, *pp = at(t.p, PB ? 2 : 4);
    char *pm = at(t.m, S8 ? 1 : 4), *pv = at(t.v, S8 ? 1 : 4);
    uint8_t *ps = S8 ? t.m_scale + (il >> 7) : nullptr, *pr = S8 ? t.v_scale + (il >> 7) : nullptr;
    uint32_t g[PIECES][V], w[PIECES][V], m[PIECES][V], v[PIECES][V], sm[PIECES], sv[PIECES];
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
        const int i = 32 * V * k, left = rest - i;
        if (!WHOLE && (i >= there || (!FAST && !(pieces >> k & 1))))
            continue;
        load<V, GB, WHOLE>(pg, i, left, g[k]);
        if (MASTER)
            load<V, false, WHOLE>(pw, i, left, w[k]);
        else
            load<V, PB, WHOLE>(pp, i, left, w[k]);
        if (S8) {
            const uint2 a = load_bytes<WHOLE>(pm, i, left), b = load_bytes<WHOLE>(pv, i, left);
            m[k][0] = a.x, m[k][1] = a.y;
            v[k][0] = b.x, v[k][1] = b.y;
            sm[k] = sv[k] = 127;
            if (WHOLE || left > 0) {
                sm[k] = ps[2 * k];
                sv[k] = pr[2 * k];
            }
        } else {
            load<V, false, WHOLE>(pm, i, left, m[k]);
            load<V, false, WHOLE>(pv, i, left, v[k]);
        }
    }
    uint32_t odd = 0;
    const uint32_t start = (uint32_t)il * 0x9E3779B9u + (t.key + c.step_key);
    const F2 one_b1 = f2(c.one_b1), one_b2 = f2(c.one_b2), ninv = f2(-c.inv), neps = f2(-c.eps),
             size = f2(c.size * -0x1p-64f), decay = f2(c.decay), tiny = f2(0x1p-16f), one = f2(c.one);
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
        const int i = 32 * V * k, left = rest - i;
        if (!WHOLE && (i >= there || (!FAST && !(pieces >> k & 1))))
            continue;
        float mk[V], vk[V], wk[V], root[V];
        uint32_t bits[V];
        const F2 b1 = f2(c.b1), b2 = f2(c.b2);
        F2 mp[V / 2], vp[V / 2];
        if (S8) {
            // the states' values, exactly (a root of 4 bits has an exact square, if not
            // under 2^-149); times beta only then: a small scale may leave no bits for it
#pragma unroll
            for (int h = 0; h < V / 4; ++h) {
                unpack_e4m3(m[k][h], mk + 4 * h);
                unpack_e4m3(v[k][h], vk + 4 * h);
            }
            const F2 r = f2(scale_value(sv[k])), q = f2(scale_value(sm[k]));
#pragma unroll
            for (int h = 0; h < V / 2; ++h) {
                mp[h] = mul2(f2(mk[2 * h], mk[2 * h + 1]), q);
                vp[h] = mul2(f2(vk[2 * h], vk[2 * h + 1]), r);
                vp[h] = mul2(vp[h], vp[h]);
            }
        } else {
#pragma unroll
            for (int h = 0; h < V / 2; ++h) {
                mp[h] = pair_of<V, false>(m[k], h);
                vp[h] = pair_of<V, false>(v[k], h);
            }
        }
#pragma unroll
        for (int h = 0; h < V / 2; ++h) {
            F2 gr = pair_of<V, GB>(g[k], h);
            if (c.scaled)
                gr = mul2(gr, f2(c.scale));
            mp[h] = add2_apart(mul2(mp[h], b1), mul2(gr, one_b1), one);
            vp[h] = add2_apart(mul2(vp[h], b2), mul2(mul2(gr, gr), one_b2), one);
            const float2 mn = of(mp[h]), vn = of(vp[h]);
            const float2 rn = FAST ? of(root2(vp[h])) : make_float2(root_of(vn.x), root_of(vn.y));
            mk[2 * h] = mn.x, mk[2 * h + 1] = mn.y;
            vk[2 * h] = vn.x, vk[2 * h + 1] = vn.y;
            root[2 * h] = rn.x, root[2 * h + 1] = rn.y;
        }
        if (!WHOLE)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j >= left)
                    mk[j] = root[j] = 0.0f;          // (past the end: no part of the block's largest)
        const float mtop = largest(mk), rtop = largest(root);
        const bool mine = !FAST || __all_sync(0xffffffffu, c.plain && mtop < 0x1p10f && rtop < 0x1p30f);
        odd |= mine ? 0u : 1u << k;
#pragma unroll
        for (int h = 0; h < V / 2; ++h) {
            const F2 wo = pair_of<V, PB && !MASTER>(w[k], h), rt = f2(root[2 * h], root[2 * h + 1]);
            if (FAST) {
                const F2 u = quotient2(mul2(mp[h], f2(0x1p64f)), add2_apart(mul2(rt, ninv), neps, one));
                const float2 wn = of(add2_apart(mul2(u, size), mul2(wo, decay), one));
                wk[2 * h] = wn.x, wk[2 * h + 1] = wn.y;
            } else {
                const float2 wf = of(wo);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int q = 2 * h + j;
                    const float u = quotient(mk[q], __fadd_rn(__fmul_rn(root[q], c.inv), c.eps));
                    wk[q] = __fsub_rn(__fmul_rn(j ? wf.y : wf.x, c.decay), __fmul_rn(u, c.size));
                }
            }
        }
#pragma unroll
        for (int q = 0; q < V; ++q)
            if (S8 || (PB && !MASTER))
                bits[q] = random_bits(start + (uint32_t)(i + q) * 0x9E3779B9u);
        if constexpr (S8) {
            uint2 q;
            uint32_t s;
            // both keys of the block over its 16 lanes
            uint32_t keys = scale_key(mtop) | (scale_key(rtop) << 16);
#pragma unroll
            for (int off = 8; off; off >>= 1)
                keys = __vmaxu2(keys, __shfl_xor_sync(0xffffffffu, keys, off));
            const bool writes = mine && (lane & 15) == 0 && (WHOLE || left > 0);
            quantize<false>(mk, bits, keys & 0xffffu, tiny, q, s);
            if (mine)
                store_bytes<WHOLE>(pm, i, left, q);
            if (writes)
                ps[2 * k] = (uint8_t)s;
            quantize<true>(root, bits, keys >> 16, tiny, q, s);
            if (mine)
                store_bytes<WHOLE>(pv, i, left, q);
            if (writes)
                pr[2 * k] = (uint8_t)s;
        } else {
            if (mine)
                store<V, WHOLE>(pm, i, left, mk);
            if (mine)
                store<V, WHOLE>(pv, i, left, vk);
        }
        if (MASTER && mine)
            store<V, WHOLE>(pw, i, left, wk);
        if (PB) {
            uint32_t h[V / 2];
            if (MASTER) {
#pragma unroll
                for (int q = 0; q < V / 2; ++q) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(wk[2 * q], wk[2 * q + 1]);
                    h[q] = *reinterpret_cast<const uint32_t *>(&b);
                }
            } else {
                // up as often as the cut half is large: a fraction of a step is added at
                // random (an infinity stays one, and so does a NaN)
                uint32_t x[V];
                float sum = 0.0f;
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    x[q] = __float_as_uint(wk[q]) + ((bits[q] * 0x9E3779B9u) >> 16);
                    sum += wk[q];
                }
                if (!(fabsf(sum) < INFINITY))
#pragma unroll
                    for (int q = 0; q < V; ++q)
                        if (wk[q] != wk[q])
                            x[q] = 0x7fc00000u;
#pragma unroll
                for (int q = 0; q < V / 2; ++q)
                    h[q] = __byte_perm(x[2 * q], x[2 * q + 1], 0x7632);
            }
            if (mine)
                store_bf16<V, WHOLE>(pp, i, left, h);
        } else if (mine) {
            store<V, WHOLE>(pp, i, left, wk);
        }
    }
    return odd;
}

// (a call, so that the 8-bit kernel's registers go to what all but such pieces need)
template <int KIND>
__device__ __noinline__ void step_rest(const AdamTensor &t, const Step &c, long long i0, uint32_t pieces)
{
    step_unit<KIND, false, false>(t, c, i0, pieces);
}

template <int KIND>
__device__ __forceinline__ void step_any(const AdamTensor &t, const Step &c, long long i0)
{
    const uint32_t rest = (t.kind & K_VEC) && i0 + WARP_UNIT <= t.n ? step_unit<KIND, true, true>(t, c, i0, 0)
                                                                    : step_unit<KIND, false, true>(t, c, i0, 0);
    if (__builtin_expect(rest == 0, 1))
        return;
    if constexpr (KIND & K_S8)
        step_rest<KIND>(t, c, i0, rest);
    else
        step_unit<KIND, false, false>(t, c, i0, rest);
}

// A kernel for each kind of state.  Blocks of 128 threads.  With 8-bit states 2^26
// elements take 176 us with 6 blocks to an SM, of which 21 are for rounding every
// operation as the formula does (155 with an approximate root and reciprocal; with the
// compiler's root and quotient in their place 190).  Counters: 85 instructions an element,
// issue slots 81% used, and the pipe of paired fp32 and integer products nearly as much.
// Before those 21: 169 with 4 blocks, 161 with 5; blocks of 1024 elements 162 to 173, a
// block that loops over four times the elements 344; four elements to a lane instead of
// eight 158.  With fp32 states (286 us with a master copy) 3 to 6 blocks make no
// difference: memory bounds them, and rounding costs nothing.
template <int N, bool S8>
__global__ void __launch_bounds__(ADAM_THREADS, S8 ? 6 : 4) adamw_kernel(const __grid_constant__ AdamTable<N> tab)
{
    pdl_wait();
    const AdamScalars &k = tab.c;
    Step c;
    c.b1 = k.b1;
    c.one_b1 = k.one_b1;
    c.b2 = k.b2;
    c.one_b2 = k.one_b2;
    c.eps = k.eps;
    c.size = k.size;
    c.inv = k.inv;
    c.one = k.one;
    c.step_key = k.step_key;
    c.scaled = k.grad_scale != nullptr;
    c.scale = c.scaled ? *k.grad_scale : 1.0f;
    int lo = 0, hi = tab.count - 1;              // the tensor of this block's unit
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.unit0[mid] <= (int)blockIdx.x)
            lo = mid;
        else
            hi = mid - 1;
    }
    const AdamTensor &t = tab.t[lo];
    c.decay = t.decay;
    if (k.lr_dev || k.step) {
        // the step's number and lr as they are on the device now
        __shared__ float sh[3];
        if (threadIdx.x == 0) {
            const double lr = k.lr_dev ? (double)*k.lr_dev : k.lr;
            const double n = (double)(k.step ? *k.step : k.step_host);
            sh[0] = (float)(lr / (1.0 - pow(k.beta1, n)));
            sh[1] = (float)(1.0 / sqrt(1.0 - pow(k.beta2, n)));
            sh[2] = (float)__dsub_rn(1.0, __dmul_rn(lr, t.weight_decay));
        }
        __syncthreads();
        c.size = sh[0];
        c.inv = sh[1];
        c.decay = sh[2];
        if (k.step)
            c.step_key = (uint32_t)*k.step * 0x85A308D3u;
    }
    // (what root2, quotient2 and the factor 2^-64 of size are for)
    c.plain = c.inv < 0x1p10f && c.eps >= 0x1p-50f && c.eps < 0x1p30f && (c.size == 0.0f || fabsf(c.size) >= 0x1p-62f);
    if (!(fabsf(c.scale) <= 3.402823466e38f))
        return;                                  // (a step whose gradients' norm is not finite is left out)
    const long long i0 = (long long)((int)blockIdx.x - tab.unit0[lo]) * ADAM_UNIT + (threadIdx.x >> 5) * WARP_UNIT;
    if (i0 >= t.n)
        return;
    constexpr int S = S8 ? K_S8 : 0;
    switch (t.kind & (K_PB | K_GB | K_MASTER)) {
    case 0: step_any<S>(t, c, i0); break;
    case K_GB: step_any<S | K_GB>(t, c, i0); break;
    case K_PB: step_any<S | K_PB>(t, c, i0); break;
    case K_PB | K_GB: step_any<S | K_PB | K_GB>(t, c, i0); break;
    case K_PB | K_MASTER: step_any<S | K_PB | K_MASTER>(t, c, i0); break;
    case K_PB | K_GB | K_MASTER: step_any<S | K_PB | K_GB | K_MASTER>(t, c, i0); break;
    default: break;
    }
}

// Squares of a thread's elements, V at a time, in 64 bits: those that fp32 cannot hold.
template <int V, bool BF16>
__device__ __noinline__ double squares_64(const void *g, int n)
{
    double sum = 0.0;
    for (int i = threadIdx.x * V; i < n; i += 256 * V)
        for (int j = 0; j < V; ++j) {
            const float x = BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(g)[i + j] << 16)
                                 : static_cast<const float *>(g)[i + j];
            if (x != 0.0f)
                sum = fma((double)x, (double)x, sum);
        }
    return sum;
}

// Sum of squares of every tensor: a thread adds at most 32 squares in fp32
// before they join a 64-bit sum, so the norm is as exact over 10^9 elements as over
// a few; the blocks' sums are added in a fixed order.  Where the 32 overflow, or
// their sum is so small that some may have vanished (`any`: bits of those that are not
// zero), the thread takes them again in 64 bits.
__global__ void __launch_bounds__(256) grad_norm_kernel(const __grid_constant__ NormTable tab, double *__restrict__ partial)
{
    pdl_wait();
    __shared__ double wsum[8];
    __shared__ int which;
    double sum = 0.0;
    int at = 0;
    for (int u = blockIdx.x; u < tab.units; u += gridDim.x) {
        if (threadIdx.x == 0) {
            while (at + 1 < tab.count && tab.t[at + 1].unit0 <= u)
                ++at;
            which = at;
        }
        __syncthreads();
        const NormTensor &t = tab.t[which];
        __syncthreads();
        const long long i0 = (long long)(u - t.unit0) * NORM_UNIT;
        const long long n = min(t.n - i0, (long long)NORM_UNIT);
        float acc[4] = {};
        uint32_t any = 0;
        const bool whole = t.aligned && n == NORM_UNIT;
        if (t.bf16) {
            const uint16_t *g = static_cast<const uint16_t *>(t.g) + i0;
            if (whole) {
                uint4 v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[q] = __ldcs(reinterpret_cast<const uint4 *>(g) + threadIdx.x + 256 * q);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t x[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a = __uint_as_float(x[j] << 16), b = __uint_as_float(x[j] & 0xffff0000u);
                        acc[q] = fmaf(b, b, fmaf(a, a, acc[q]));
                        any |= x[j] & 0x7fff7fffu;
                    }
                }
            } else {
                for (int i = threadIdx.x; i < n; i += 256) {
                    const float a = __uint_as_float((uint32_t)g[i] << 16);
                    acc[0] = fmaf(a, a, acc[0]);
                    any |= g[i] & 0x7fffu;
                }
            }
        } else {
            const float *g = static_cast<const float *>(t.g) + i0;
            if (whole) {
                float4 v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    v[q] = __ldcs(reinterpret_cast<const float4 *>(g) + threadIdx.x + 256 * q);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    acc[q & 3] += fmaf(v[q].x, v[q].x, v[q].y * v[q].y) + fmaf(v[q].z, v[q].z, v[q].w * v[q].w);
                    any |= __float_as_uint(v[q].x) | __float_as_uint(v[q].y) | __float_as_uint(v[q].z) | __float_as_uint(v[q].w);
                }
            } else {
                for (int i = threadIdx.x; i < n; i += 256) {
                    acc[0] = fmaf(g[i], g[i], acc[0]);
                    any |= __float_as_uint(g[i]);
                }
            }
            any &= 0x7fffffffu;
        }
        const float all = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        double more = (double)acc[0] + (double)acc[1] + ((double)acc[2] + (double)acc[3]);
        if (any && !(all >= 0x1p-90f && all < INFINITY)) {
            const void *g = static_cast<const char *>(t.g) + i0 * (t.bf16 ? 2 : 4);
            more = t.bf16 ? whole ? squares_64<8, true>(g, (int)n) : squares_64<1, true>(g, (int)n)
                          : whole ? squares_64<4, false>(g, (int)n) : squares_64<1, false>(g, (int)n);
        }
        sum += more;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if ((threadIdx.x & 31) == 0)
        wsum[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int q = 0; q < 8; ++q)
            s += wsum[q];
        partial[tab.first + blockIdx.x] = s;
    }
}

__global__ void __launch_bounds__(256) grad_norm_finish_kernel(const double *__restrict__ partial, int n, float max_norm,
                                                               float *__restrict__ norm, float *__restrict__ scale)
{
    pdl_wait();
    __shared__ double wsum[8];
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += 256)
        s += partial[i];
#pragma unroll
    for (int off = 16; off; off >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, off);
    if ((threadIdx.x & 31) == 0)
        wsum[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int q = 0; q < 8; ++q)
            t += wsum[q];
        t = sqrt(t);
        *norm = (float)t;
        if (scale) {
            const bool finite = (float)t < INFINITY;
            *scale = !finite ? __uint_as_float(0x7fc00000u) : t > (double)max_norm ? (float)((double)max_norm / t) : 1.0f;
        }
    }
}

}  // namespace

cudaError_t launch_adamw(const AdamTable<ADAM_TABLE> &t, bool states_8, cudaStream_t s)
{
    return launch_pdl(states_8 ? adamw_kernel<ADAM_TABLE, true> : adamw_kernel<ADAM_TABLE, false>, dim3(t.units), dim3(ADAM_THREADS),
                      0, s, t);
}

cudaError_t launch_adamw(const AdamTable<ADAM_TABLE_SMALL> &t, bool states_8, cudaStream_t s)
{
    return launch_pdl(states_8 ? adamw_kernel<ADAM_TABLE_SMALL, true> : adamw_kernel<ADAM_TABLE_SMALL, false>,
                      dim3(t.units), dim3(ADAM_THREADS), 0, s, t);
}

cudaError_t launch_grad_norm(const NormTable &t, double *partial, cudaStream_t s)
{
    return launch_pdl(grad_norm_kernel, dim3(t.blocks), dim3(256), 0, s, t, partial);
}

cudaError_t launch_grad_norm_finish(const double *partial, int n, float max_norm, float *norm, float *scale, cudaStream_t s)
{
    return launch_pdl(grad_norm_finish_kernel, dim3(1), dim3(256), 0, s, partial, n, max_norm, norm, scale);
}

}  // namespace glr
