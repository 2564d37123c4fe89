// C-ABI entry points of token order, the 8-bit products and the AdamW step
// (include/moe.h), each with its argument checks and launch sequence.  As in
// api.cu, every check runs on the host before any CUDA call.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "expert_ops.h"
#include "host.h"

using namespace glr;
using namespace glr::host;

namespace {

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// ------------------------------------------------------------ token order
constexpr int MAX_K = 4096;
constexpr long long MAX_PAIRS = (1ll << 31) - (1ll << 20);

int check_pairs(int32_t T, int32_t k)
{
    if (T < 0 || k < 1)
        return MOE_ERR_INVALID_ARG;
    return (long long)T * k > MAX_PAIRS || k > MAX_K ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}

int check_order(int32_t T, int32_t k, int32_t E)
{
    const int rc = check_pairs(T, k);
    if (rc != MOE_OK)
        return rc;
    if (E < 1)
        return MOE_ERR_INVALID_ARG;
    return E > ORDER_MAX_E ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}

size_t order_bytes(int32_t T, int32_t k, int32_t E)
{
    const OrderPlan plan = order_plan((long long)T * k);
    return sizeof(WsHeader) + (plan.blocks > 1 ? align_up(4ull * plan.blocks * order_ld(E), 256) : 0);
}

// a kernel's grid over this many threads or warps
bool grid_fits(long long blocks) { return blocks <= 0x7fffffffll; }

int check_rows(int32_t T, int32_t k, int32_t H, int32_t f32, int64_t rows)
{
    const int rc = check_pairs(T, k);
    if (rc != MOE_OK)
        return rc;
    if (H < 1 || rows < 0 || (f32 != 0 && f32 != 1))
        return MOE_ERR_INVALID_ARG;
    if (H % (f32 ? 4 : 8) != 0 || !grid_fits(((long long)T * H + 255) / 256))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// --------------------------------------------------------- 8-bit operands
int check_format(int32_t f) { return f == 0 || f == 1 ? MOE_OK : MOE_ERR_INVALID_ARG; }

int check_quantize(int32_t R, int32_t K, int32_t f32, int32_t e5m2)
{
    if (R < 0 || K < 1 || (f32 != 0 && f32 != 1) || check_format(e5m2) != MOE_OK)
        return MOE_ERR_INVALID_ARG;
    return K % 16 != 0 || K > (1 << 24) ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}

// ------------------------------------------------------------ the products
int scaled_gemm(int kid, ScaledGemmParams &p, const uint8_t *A, const uint8_t *sA, uint64_t a_ld, const uint8_t *B,
                const uint8_t *sB, uint64_t b_ld, uint64_t K, uint64_t b_rows, uint64_t sb_rows, void *out,
                void *ws, cudaStream_t s, int &launches)
{
    int sms = 0;
    const int rc = device_check(&sms);
    if (rc != MOE_OK)
        return rc;
    const ScaledTile tile = scaled_tile(p.mode, p.M, p.N, p.E, p.kblocks, p.out_f32, sms);
    const int rows = tile.pair ? 256 : 128;
    const bool maps = make_map_bytes(&p.tmA, A, p.M, K, 128, 128, true) &&
                      make_map_bytes(&p.tmB, B, b_rows, K, 128, tile.pair ? tile.columns / 2 : tile.columns, true) &&
                      make_map_bytes(&p.tmSA, sA, p.kblocks, a_ld, SCALED_SA_BOX, SCALED_CHUNK, false) &&
                      make_map_bytes(&p.tmSB, sB, sb_rows, b_ld, tile.columns, SCALED_CHUNK, false);
    if (!maps)
        return MOE_ERR_CUDA;
    // Bands of A that stay in L2 while their column tiles pass (an eighth of it: the
    // dies keep copies, and the output passes too).  65536 x 2048 x 1024: 125 us with
    // all rows in one band, whose 67 MB were read again for every column tile.
    p.band = p.E ? ceil_div(p.M, rows) : (int)std::max<uint64_t>(1, (16u << 20) / (rows * std::max<uint64_t>(K, 1)));
    p.out = out;
    p.wide = aligned(out, 32) && (size_t)p.N * (p.out_f32 ? 4 : 2) % 32 == 0;
    p.status = &header(ws)->status;
    if (take_injected_timeout()) {
        p.inject_withhold = 1;
        p.wait_limit_ns = 50000000ull;
    }
    const long long n_tiles = ceil_div(p.N, tile.columns);
    long long units = n_tiles * ceil_div(p.M, rows);
    if (p.mode == SM_ROWS)
        units = n_tiles * (ceil_div(p.M, rows) + (long long)std::min(p.E, p.M));
    if (p.mode == SM_SUM && p.E)
        units *= p.E;
    GLR_LAUNCH(kid, launch_scaled_gemm(p, tile, (int)std::min<long long>(units, tile.pair ? sms / 2 : sms), s));
    return MOE_OK;
}

int check_product(int32_t M, int32_t N, int64_t K, int32_t E, int32_t a_format, int32_t b_format, int32_t out_f32)
{
    if (M < 0 || N < 1 || K < 0 || E < 0 || check_format(a_format) != MOE_OK || check_format(b_format) != MOE_OK ||
        (out_f32 != 0 && out_f32 != 1))
        return MOE_ERR_INVALID_ARG;
    if (K % 16 != 0 || N % 8 != 0 || E > SCALED_MAX_E || M > (1 << 28) || N > (1 << 24) || K > (1 << 30) ||
        (long long)std::max(E, 1) * N > (1ll << 31) - 256 ||
        ((long long)ceil_div(M, 128) + E) * ceil_div(N, 64) * std::max(E, 1) > (1ll << 30))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// ------------------------------------------------------------- the optimiser
int check_tensors(int32_t count, const moe_adamw_tensor *t, bool step)
{
    if (count < 0 || (count && !t))
        return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor &a = t[i];
        if (a.n < 0 || (a.flags & ~7))
            return MOE_ERR_INVALID_ARG;
        if (a.n > (1ll << 40))
            return MOE_ERR_UNSUPPORTED_SHAPE;
        if (a.n == 0)
            continue;
        if (!a.g)
            return MOE_ERR_INVALID_ARG;
        if (!aligned(a.g, a.flags & MOE_ADAMW_GRAD_BF16 ? 2 : 4))
            return MOE_ERR_MISALIGNED;
        if (!step)
            continue;
        const bool bytes = a.flags & MOE_ADAMW_STATES_IN_BYTES, bf16 = a.flags & MOE_ADAMW_PARAM_BF16;
        if (!a.p || !a.m || !a.v || (bytes && (!a.m_scale || !a.v_scale)) || (!bytes && (a.m_scale || a.v_scale)) ||
            (a.master && !bf16) || !(a.weight_decay >= 0.0) || !isfinite(a.weight_decay))
            return MOE_ERR_INVALID_ARG;
        if (!aligned(a.p, bf16 ? 2 : 4) || !aligned(a.master, 4) || (!bytes && (!aligned(a.m, 4) || !aligned(a.v, 4))))
            return MOE_ERR_MISALIGNED;
    }
    return MOE_OK;
}

template <int N>
cudaError_t adamw_chunk(const moe_adamw_tensor *t, int count, const AdamScalars &c, uint32_t seed, cudaStream_t s,
                        bool &empty)
{
    AdamTable<N> tab;
    tab.c = c;
    tab.count = 0;
    long long units = 0;
    for (int i = 0; i < count; ++i) {
        if (t[i].n == 0)
            continue;
        AdamTensor &a = tab.t[tab.count++];
        const bool bytes = t[i].flags & MOE_ADAMW_STATES_IN_BYTES, pb = t[i].flags & MOE_ADAMW_PARAM_BF16,
                   gb = t[i].flags & MOE_ADAMW_GRAD_BF16;
        a.p = t[i].p;
        a.g = t[i].g;
        a.master = t[i].master;
        a.m = t[i].m;
        a.v = t[i].v;
        a.m_scale = t[i].m_scale;
        a.v_scale = t[i].v_scale;
        a.n = t[i].n;
        a.weight_decay = t[i].weight_decay;
        const volatile double shrink = c.lr * t[i].weight_decay;     // (two roundings, on every host)
        a.decay = (float)(1.0 - shrink);
        a.key = seed + t[i].ordinal * 0x13198A2Fu;
        const bool vec = aligned(a.p, pb && !bytes ? 8 : 16) && aligned(a.g, gb && !bytes ? 8 : 16) &&
                         aligned(a.master, 16) && aligned(a.m, bytes ? 8 : 16) && aligned(a.v, bytes ? 8 : 16);
        a.kind = (bytes ? 1 : 0) | (pb ? 2 : 0) | (gb ? 4 : 0) | (a.master ? 8 : 0) | (vec ? 16 : 0);
        a.pad = 0;
        tab.unit0[tab.count - 1] = (int)units;
        units += (t[i].n + ADAM_UNIT - 1) / ADAM_UNIT;
    }
    tab.units = (int)units;
    empty = units == 0;
    return empty ? cudaSuccess : launch_adamw(tab, (t[0].flags & MOE_ADAMW_STATES_IN_BYTES) != 0, s);
}

long long adam_units(const moe_adamw_tensor &t) { return (t.n + ADAM_UNIT - 1) / ADAM_UNIT; }

}  // namespace

extern "C" {

size_t moe_sort_tokens_workspace_bytes(int32_t T, int32_t k, int32_t E)
{
    return check_order(T, k, E) == MOE_OK ? order_bytes(T, k, E) : 0;
}

int moe_sort_tokens(int32_t T, int32_t k, int32_t E, const int32_t *topk_idx, int32_t *offsets, int32_t *slot_of,
                    void *ws, size_t ws_bytes, void *stream)
{
    ProfCall prof_call_;
    int rc = check_order(T, k, E);
    if (rc != MOE_OK)
        return rc;
    if ((T && (!topk_idx || !slot_of)) || !offsets)
        return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(ws, ws_bytes, order_bytes(T, k, E))) != MOE_OK)
        return rc;
    if (!aligned(topk_idx, 4) || !aligned(offsets, 4) || !aligned(slot_of, 4))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long pairs = (long long)T * k;
    const OrderPlan plan = order_plan(pairs);
    int32_t *hist = plan.blocks > 1 ? at<int32_t>(ws, sizeof(WsHeader)) : nullptr;
    int launches = 0;
    if (hist)
        GLR_LAUNCH(KID_SORT_ORDER, launch_order_count(topk_idx, pairs, E, plan, hist, s));
    GLR_LAUNCH(KID_SORT_ORDER,
               launch_order_assign(topk_idx, pairs, E, plan, hist, offsets, slot_of, &header(ws)->status, s));
    set_last_launches(launches);
    return MOE_OK;
}

int moe_sort_rows(int32_t T, int32_t k, int64_t row_bytes, int64_t rows, const void *x, const int32_t *slot_of,
                  void *out, void *stream)
{
    ProfCall prof_call_;
    int rc = check_pairs(T, k);
    if (rc != MOE_OK)
        return rc;
    if (row_bytes < 1 || rows < 0)
        return MOE_ERR_INVALID_ARG;
    if (row_bytes % 16 != 0 || row_bytes > (1ll << 30) || !grid_fits((T * (row_bytes / 16) + 255) / 256))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || rows == 0) {
        set_last_launches(0);
        return MOE_OK;
    }
    if (!x || !slot_of || !out)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(slot_of, 4))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    GLR_LAUNCH(KID_SORT_ROWS, launch_sort_rows(x, T, k, row_bytes / 16, rows, slot_of, out, s));
    set_last_launches(launches);
    return MOE_OK;
}

int moe_unsort_rows(int32_t T, int32_t k, int32_t H, int32_t f32, int64_t rows, const void *y, const int32_t *slot_of,
                    const float *topk_w, void *out, void *stream)
{
    ProfCall prof_call_;
    int rc = check_rows(T, k, H, f32, rows);
    if (rc != MOE_OK)
        return rc;
    if (T == 0) {
        set_last_launches(0);
        return MOE_OK;
    }
    if ((rows && !y) || !slot_of || !out)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(out, 16) || !aligned(slot_of, 4) || !aligned(topk_w, 4))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    GLR_LAUNCH(KID_UNSORT, launch_unsort_rows(y, f32 != 0, T, k, H, rows, slot_of, topk_w, out, sms, s));
    set_last_launches(launches);
    return MOE_OK;
}

int moe_unsort_rows_backward(int32_t T, int32_t k, int32_t H, int32_t f32, int64_t rows, const void *d_out,
                             const void *y, const int32_t *slot_of, const float *topk_w, void *d_y, float *d_topk_w,
                             void *stream)
{
    ProfCall prof_call_;
    int rc = check_rows(T, k, H, f32, rows);
    if (rc != MOE_OK)
        return rc;
    if (T == 0) {
        set_last_launches(0);
        return MOE_OK;
    }
    if (!d_out || (rows && (!y || !d_y)) || !slot_of || !topk_w)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(d_out, 16) || !aligned(y, 16) || !aligned(d_y, 16) || !aligned(slot_of, 4) || !aligned(topk_w, 4) ||
        !aligned(d_topk_w, 4))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    GLR_LAUNCH(KID_UNSORT_BWD,
               launch_unsort_backward(d_out, y, f32 != 0, T, k, H, rows, slot_of, topk_w, d_y, d_topk_w, s));
    set_last_launches(launches);
    return MOE_OK;
}

int moe_scaled_quantize(int32_t batch, int32_t R, int32_t K, int32_t f32, int32_t e_five_m_two, const void *x,
                        uint8_t *q, uint8_t *scale, uint8_t *qt, uint8_t *scale_t, int32_t E, const int32_t *offsets,
                        int32_t *starts, int64_t P, void *stream)
{
    ProfCall prof_call_;
    int rc = check_quantize(R, K, f32, e_five_m_two);
    if (rc != MOE_OK)
        return rc;
    if (batch < 1 || E < 0 || !q != !scale || !qt != !scale_t || (!q && !qt) || (E > 0 && (!offsets || !starts || batch != 1 || !qt)) ||
        (E == 0 && (offsets || starts)))
        return MOE_ERR_INVALID_ARG;
    const long long blocks = E > 0 ? (long long)R / 128 + E : ((long long)R + 127) / 128;
    if (qt && (E > 0 ? P % 128 != 0 || P < 128 * blocks : P != (int64_t)align_up(R, 16)))
        return MOE_ERR_INVALID_ARG;
    if (batch > 65535 || blocks > 65535 || P > 128ll * 65535 || E > SCALED_MAX_E)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (R && !x)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(qt, 16) || !aligned(offsets, 4) || !aligned(starts, 4))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    if (E > 0)
        GLR_LAUNCH(KID_STARTS, launch_column_starts(offsets, E, R, starts, s));
    if (R > 0) {
        QuantParams p = {};
        p.x = x;
        p.R = R;
        p.K = K;
        p.kblocks = ceil_div(K, 128);
        p.f32 = f32 != 0;
        p.e5m2 = e_five_m_two != 0;
        p.q = q;
        p.scale = scale;
        p.ld = (long long)align_up(R, 16);
        p.qt = qt;
        p.scale_t = scale_t;
        p.P = P;
        p.ld_t = (long long)align_up(K, 16);
        p.starts = starts;
        p.offsets = offsets;
        p.E = E;
        p.batch = batch;
        GLR_LAUNCH(KID_QUANTIZE, launch_quantize_tiles(p, q != nullptr, qt != nullptr, s));
    }
    set_last_launches(launches);
    return MOE_OK;
}

int moe_scaled_quantize_rows(int32_t T, int32_t k, int32_t K, int32_t f32, int32_t e_five_m_two, int64_t rows,
                             const void *x, const int32_t *slot_of, uint8_t *q, uint8_t *scale, void *stream)
{
    ProfCall prof_call_;
    int rc = check_quantize(T, K, f32, e_five_m_two);
    if (rc == MOE_OK)
        rc = check_pairs(T, k);
    if (rc != MOE_OK)
        return rc;
    if (rows < 0)
        return MOE_ERR_INVALID_ARG;
    if (rows > (1ll << 31) - 256 || !grid_fits(((long long)T * ceil_div(K, 128) + 15) / 16))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || rows == 0) {
        set_last_launches(0);
        return MOE_OK;
    }
    if (!x || !slot_of || !q || !scale)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(slot_of, 4))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    QuantParams p = {};
    p.x = x;
    p.R = T;
    p.K = K;
    p.kblocks = ceil_div(K, 128);
    p.f32 = f32 != 0;
    p.e5m2 = e_five_m_two != 0;
    p.q = q;
    p.scale = scale;
    p.ld = (long long)align_up(rows, 16);
    p.slot_of = slot_of;
    p.k = k;
    p.rows = rows;
    int launches = 0;
    GLR_LAUNCH(KID_QUANTIZE, launch_quantize_slots(p, s));
    set_last_launches(launches);
    return MOE_OK;
}

int moe_scaled_product(int32_t M, int32_t N, int32_t K, int32_t E, int32_t a_format, int32_t b_format, int32_t out_f32,
                       const uint8_t *A, const uint8_t *A_scale, const uint8_t *B, const uint8_t *B_scale,
                       const int32_t *offsets, void *out, void *ws, size_t ws_bytes, void *stream)
{
    ProfCall prof_call_;
    int rc = check_product(M, N, K, E, a_format, b_format, out_f32);
    if (rc != MOE_OK)
        return rc;
    if (K < 1 || (E > 0) != (offsets != nullptr))
        return MOE_ERR_INVALID_ARG;
    if (M == 0) {
        set_last_launches(0);
        return MOE_OK;
    }
    if (!A || !A_scale || !B || !B_scale || !out)
        return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(ws, ws_bytes, sizeof(WsHeader))) != MOE_OK)
        return rc;
    if (!aligned(A, 16) || !aligned(A_scale, 16) || !aligned(B, 16) || !aligned(B_scale, 16) || !aligned(out, 16) ||
        !aligned(offsets, 4))
        return MOE_ERR_MISALIGNED;
    ScaledGemmParams p;
    memset(&p, 0, sizeof(p));
    p.mode = E > 0 ? SM_ROWS : SM_DENSE;
    p.M = M;
    p.N = N;
    p.kblocks = ceil_div(K, 128);
    p.E = E;
    p.bounds = offsets;
    p.out_f32 = out_f32 != 0;
    p.a_e5m2 = a_format != 0;
    p.b_e5m2 = b_format != 0;
    const uint64_t groups = std::max(E, 1);
    int launches = 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    rc = scaled_gemm(KID_SCALED_PRODUCT, p, A, A_scale, align_up(M, 16), B, B_scale, align_up(N, 16), K, groups * N,
                     groups * p.kblocks, out, ws, s, launches);
    if (rc == MOE_OK)
        set_last_launches(launches);
    return rc;
}

int moe_scaled_weight_gradient(int32_t M, int32_t N, int64_t P, int32_t E, int32_t a_format, int32_t b_format,
                               int32_t out_f32, const uint8_t *A, const uint8_t *A_scale, const uint8_t *B,
                               const uint8_t *B_scale, const int32_t *starts, void *out, void *ws, size_t ws_bytes,
                               void *stream)
{
    ProfCall prof_call_;
    int rc = check_product(M, N, P, E, a_format, b_format, out_f32);
    if (rc != MOE_OK)
        return rc;
    if (M < 1 || P < 1 || (E > 0 && P % 128 != 0) || (E > 0) != (starts != nullptr))
        return MOE_ERR_INVALID_ARG;
    if (!A || !A_scale || !B || !B_scale || !out)
        return MOE_ERR_INVALID_ARG;
    if ((long long)std::max(E, 1) * M > (1ll << 31) - 256)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if ((rc = check_ws(ws, ws_bytes, sizeof(WsHeader))) != MOE_OK)
        return rc;
    if (!aligned(A, 16) || !aligned(A_scale, 16) || !aligned(B, 16) || !aligned(B_scale, 16) || !aligned(out, 16) ||
        !aligned(starts, 4))
        return MOE_ERR_MISALIGNED;
    ScaledGemmParams p;
    memset(&p, 0, sizeof(p));
    p.mode = SM_SUM;
    p.M = M;
    p.N = N;
    p.kblocks = ceil_div(P, 128);
    p.E = E;
    p.bounds = starts;
    p.out_f32 = out_f32 != 0;
    p.a_e5m2 = a_format != 0;
    p.b_e5m2 = b_format != 0;
    int launches = 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    rc = scaled_gemm(KID_SCALED_WGRAD, p, A, A_scale, align_up(M, 16), B, B_scale, align_up(N, 16), P, N, p.kblocks,
                     out, ws, s, launches);
    if (rc == MOE_OK)
        set_last_launches(launches);
    return rc;
}

int moe_debug_scaled_tile(int32_t weight_gradient, int32_t M, int32_t N, int64_t K, int32_t E, int32_t out_f32,
                          int32_t sms, int32_t *rows, int32_t *columns)
{
    const int rc = check_product(M, N, K, E, 0, 0, out_f32);
    if (rc != MOE_OK)
        return rc;
    if (M < 1 || K < 1 || sms < 2 || !rows || !columns)
        return MOE_ERR_INVALID_ARG;
    const ScaledTile t = scaled_tile(weight_gradient ? SM_SUM : E > 0 ? SM_ROWS : SM_DENSE, M, N, E, ceil_div(K, 128), out_f32 != 0, sms);
    *rows = t.pair ? 256 : 128;
    *columns = t.columns;
    return MOE_OK;
}

int moe_adamw(int32_t count, const moe_adamw_tensor *tensors, const moe_adamw_cfg *cfg, const float *grad_scale,
              const int64_t *step_on_device, const float *lr_on_device, void *stream)
{
    ProfCall prof_call_;
    int rc = check_tensors(count, tensors, true);
    if (rc != MOE_OK)
        return rc;
    if (!cfg || !isfinite(cfg->lr) || !(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0) || !(cfg->beta2 >= 0.0 && cfg->beta2 < 1.0) ||
        !(cfg->eps >= 0.0) || !isfinite(cfg->eps) || (!step_on_device && cfg->step < 1) || cfg->reserved != 0)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(grad_scale, 4) || !aligned(step_on_device, 8) || !aligned(lr_on_device, 4))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    AdamScalars c = {};
    c.lr = cfg->lr;
    c.beta1 = cfg->beta1;
    c.beta2 = cfg->beta2;
    c.b1 = (float)cfg->beta1;
    c.one_b1 = (float)(1.0 - cfg->beta1);
    c.b2 = (float)cfg->beta2;
    c.one_b2 = (float)(1.0 - cfg->beta2);
    c.eps = (float)cfg->eps;
    c.one = 1.0f;
    const double step = (double)std::max<int64_t>(cfg->step, 1);
    c.step_host = std::max<int64_t>(cfg->step, 1);
    c.size = (float)(cfg->lr / (1.0 - pow(cfg->beta1, step)));
    c.inv = (float)(1.0 / sqrt(1.0 - pow(cfg->beta2, step)));
    c.step_key = step_on_device ? 0 : (uint32_t)cfg->step * 0x85A308D3u;
    c.grad_scale = grad_scale;
    c.step = step_on_device;
    c.lr_dev = lr_on_device;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    for (int i = 0; i < count;) {
        // as many tensors, with states of one kind, as a launch's table and its grid take
        int n = 0;
        long long units = 0;
        while (i + n < count && n < ADAM_TABLE &&
               ((tensors[i + n].flags ^ tensors[i].flags) & MOE_ADAMW_STATES_IN_BYTES) == 0 && (n == 0 || units + adam_units(tensors[i + n]) < (1ll << 30)))
            units += adam_units(tensors[i + n++]);
        bool empty = false;
        ProfScope prof(KID_ADAMW, s);
        const cudaError_t e = n <= ADAM_TABLE_SMALL ? adamw_chunk<ADAM_TABLE_SMALL>(tensors + i, n, c, cfg->seed, s, empty)
                                                    : adamw_chunk<ADAM_TABLE>(tensors + i, n, c, cfg->seed, s, empty);
        if (e != cudaSuccess)
            return MOE_ERR_CUDA;
        prof.done();
        launches += !empty;
        i += n;
    }
    set_last_launches(launches);
    return MOE_OK;
}

size_t moe_grad_norm_workspace_bytes(int32_t count)
{
    return count < 0 ? 0 : sizeof(WsHeader) + align_up(8ull * NORM_MAX_BLOCKS * std::max(1, ceil_div(count, NORM_TABLE)), 256);
}

int moe_grad_norm(int32_t count, const moe_adamw_tensor *tensors, float max_norm, float *norm, float *scale, void *ws,
                  size_t ws_bytes, void *stream)
{
    ProfCall prof_call_;
    int rc = check_tensors(count, tensors, false);
    if (rc != MOE_OK)
        return rc;
    if (!norm || (scale && !(max_norm > 0.0f)))
        return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(ws, ws_bytes, moe_grad_norm_workspace_bytes(count))) != MOE_OK)
        return rc;
    if (!aligned(norm, 4) || !aligned(scale, 4))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    double *partial = at<double>(ws, sizeof(WsHeader));
    int launches = 0, first = 0;
    for (int i = 0; i < count; i += NORM_TABLE) {
        NormTable tab;
        tab.count = 0;
        tab.first = first;
        long long units = 0;
        for (int j = i; j < std::min(count, i + NORM_TABLE); ++j) {
            if (tensors[j].n == 0)
                continue;
            NormTensor &t = tab.t[tab.count++];
            t.g = tensors[j].g;
            t.n = tensors[j].n;
            t.bf16 = (tensors[j].flags & MOE_ADAMW_GRAD_BF16) != 0;
            t.aligned = aligned(t.g, 16);
            t.unit0 = (int)units;
            t.pad = 0;
            units += (t.n + NORM_UNIT - 1) / NORM_UNIT;
            if (units > (1ll << 30))
                return MOE_ERR_UNSUPPORTED_SHAPE;
        }
        if (units == 0)
            continue;
        tab.units = (int)units;
        tab.blocks = (int)std::min<long long>(units, NORM_MAX_BLOCKS);
        GLR_LAUNCH(KID_GRAD_NORM, launch_grad_norm(tab, partial, s));
        first += tab.blocks;
    }
    GLR_LAUNCH(KID_GRAD_NORM, launch_grad_norm_finish(partial, first, max_norm, norm, scale, s));
    set_last_launches(launches);
    return MOE_OK;
}

}  // extern "C"
