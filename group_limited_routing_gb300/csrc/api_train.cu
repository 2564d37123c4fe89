// C-ABI entry points of the training operators (include/moe.h): the norms
// around a block, the vocabulary loss and the router's gradient, each with
// its argument checks, workspace layout and launch sequence.  As in api.cu,
// every check runs on the host before any CUDA call.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "host.h"

using namespace glr;
using namespace glr::host;

namespace {

// ------------------------------------------------------------- block norm
int check_block_norm(int32_t T, int32_t H, int32_t groups, int32_t stream_f32, float alpha, float eps)
{
    if (T < 1 || H < 8 || groups < 1 || T % groups != 0 || (stream_f32 != 0 && stream_f32 != 1) ||
        !isfinite(alpha) || !isfinite(eps) || eps < 0.0f)
        return MOE_ERR_INVALID_ARG;
    if (H % 8 != 0 || H > BLOCK_NORM_MAX_H || T > (1 << 24))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// The grid is that of a full GB300 whatever the device, so that the workspace
// size and the order of the column sums depend on the shape alone.
constexpr int NORM_SMS = 152;

struct NormLayout {
    size_t part_a, part_b, total;
    BlockNormPlan plan;
};

NormLayout norm_layout(int T, int H, int groups)
{
    NormLayout L;
    L.plan = block_norm_plan(T, H, groups, NORM_SMS);
    L.part_a = sizeof(WsHeader);
    L.part_b = L.part_a + align_up(sizeof(float) * (size_t)groups * L.plan.cpg * H, 256);
    L.total = L.part_b + align_up(sizeof(float) * (size_t)L.plan.blocks * H, 256);
    return L;
}

// ------------------------------------------------------------ dense products
int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

cudaError_t pair_product(PairEpilogue epi, PairProduct product, PairGemmParams p, int max_units, cudaStream_t s)
{
    if (take_injected_timeout()) {
        p.inject_withhold = 1;
        p.wait_limit_ns = 50000000ull;
    }
    return launch_pair_gemm(epi, product, p, max_units, s);
}

// K blocks per accumulator of the loss's logits (704 of K, evened out over the
// parts): the tensor core's own running sum then stays about as close to the
// exact one as an fp32 product's.  Measured at T = 8192, H = 2048, V = 131072,
// 2-norm of the losses' error over theirs, and time: one part 1.7e-6, 2.37 ms; two
// 8.2e-7, 2.42 ms; three 5.3e-7, 2.45 ms; four 4.0e-7, 2.49 ms; an fp32 matrix
// product 4.7e-7.
constexpr int LOGIT_PART_BLOCKS = 11;
// At most this many rows that count (of however many; the device knows) take
// shorter parts: T = 3, H = 3144, V = 87989 1.3e-6 -> 5e-7 at worst (an fp32 product,
// there a sum per element, 3e-7), for a quarter more time (T = 16, H = 2048, V =
// 131072: 96 -> 119 us).  That price is why more rows keep the longer parts, whose
// errors, as large row by row, partly cancel in a sum over the rows.
constexpr int LOGIT_EXACT_ROWS = 8, LOGIT_EXACT_BLOCKS = 4;

// ---------------------------------------------------------- vocabulary loss
int check_vocab(int32_t T, int32_t H, int32_t V, int32_t target_bits)
{
    if (T < 0 || H < 1 || V < 1 || (target_bits != 32 && target_bits != 64))
        return MOE_ERR_INVALID_ARG;
    if (H % 8 != 0 || H > (1 << 16) || T > (1 << 24) || V > (1 << 24) ||
        (long long)ceil_div(T, 256) * ceil_div(V, 256) > (1ll << 30))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// Backward: dlogits of one vocabulary piece [T, piece] bf16 live in the
// workspace, at most this many bytes (and 256 columns at least).
constexpr size_t VOCAB_PIECE_BYTES = 1ull << 30;

struct VocabLayout {
    size_t meta, row_of, target, packed_of, lse, weight, logit, stats, hidden, dz, part, total;
    int ntiles, nstats, piece, part_rows;
    int rows;                  // packed rows at most: T, or the repeated ones of a few
};

VocabLayout vocab_layout(int T, int H, int V, bool backward)
{
    VocabLayout L = {};
    T = std::max(T, 1);
    size_t off = sizeof(WsHeader);
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += align_up(bytes, 256);
        return at;
    };
    L.ntiles = ceil_div(V, 256);
    L.nstats = ceil_div(V, 128);
    L.rows = backward ? std::max(T, 2 * std::min(T, VOCAB_TWICE_ROWS)) : T;
    L.meta = take(sizeof(VocabMeta));
    L.row_of = take(4ull * T);
    L.target = take(4ull * L.rows);
    L.hidden = take(2ull * L.rows * H);
    if (backward) {
        L.packed_of = take(4ull * T);
        L.lse = take(4ull * L.rows);
        L.weight = take(4ull * L.rows);
        const size_t most = std::max<size_t>(1, VOCAB_PIECE_BYTES / (512ull * L.rows));   // 256-column blocks
        L.piece = (int)std::min<size_t>(L.ntiles, most) * 256;
        // (never less than fewer rows' piece takes, which may fill its bytes better)
        L.dz = take(std::min(512ull * L.rows * L.ntiles, std::max<unsigned long long>(VOCAB_PIECE_BYTES, 512ull * L.rows)));
        // fp32 sums of d_hidden: one slice per split, and as few rows as count
        // (which the host does not know) may be split the most
        const int h_tiles = ceil_div(H, 256), m_tiles = ceil_div(L.rows, 256);
        L.part_rows = 256 * std::max(m_tiles, std::min(VOCAB_MAX_SPLITS * m_tiles, SPLIT_MAX_UNITS / h_tiles));
        L.part = take(4ull * L.part_rows * H);
    } else {
        L.logit = take(4ull * T);
        L.stats = take(sizeof(float2) * (size_t)L.nstats * T);
    }
    L.total = off;
    return L;
}

// m-tiles per group of the products over [rows, vocabulary]: a group's hidden
// rows (32 MB) stay in L2 while the vocabulary's weight streams past them.
int vocab_group(int H) { return std::max(1, (32 << 20) / (256 * 2 * H)); }

// The logits product's operands: rows of hidden (packed or not), rows of W.
bool vocab_logits_maps(PairGemmParams &p, const VocabLayout &L, int T, int H, int V, const moe_bf16 *hidden,
                       const moe_bf16 *W, void *ws, int a_rows)
{
    return make_map_bf16(&p.tmA, hidden, T, H, GEMM_BK, a_rows) &&
           make_map_bf16(&p.tmHidden, at<uint16_t>(ws, L.hidden), L.rows, H, GEMM_BK, a_rows) &&
           make_map_bf16(&p.tmB, W, V, H, GEMM_BK, 128);
}

// ------------------------------------------------------- the router's gradient
struct RouteBwdLayout {
    size_t split, parts, part, logits, total;
    int splits;
    int logit_splits;          // 0: the logits come from the forward's router
};

// The logits again.  The forward's router keeps one accumulator over its part of
// K, whose additions the tensor core truncates: that is most of the error of
// d_W_router (relative 2-norm 1.1e-6 at H = 2048, at any T).  A batch of one tile
// of rows (and more than the CUDA-core router takes) forms the logits with the
// pair product instead, the hidden rows against the weight's three parts, K cut
// into splits for the SMs and into accumulators of ROUTE_LOGIT_BLOCKS blocks that
// are added in fp32 registers: 3.4e-7, what an fp32 product on the CUDA cores has.
// It costs 3 us (T = 104: 35.5 against 32.6, T = 4096: 58.8 against 56.0, E = 256,
// 4 blocks per accumulator: 35.3 and 9.0e-7); from 256 rows up a library's fp32
// product is at 1.0e-6 as well, and the forward's router serves.
constexpr int ROUTE_PAIR_LOGITS_MAX_T = 256, ROUTE_LOGIT_BLOCKS = 2;

// 64-token blocks per accumulator of the weight gradient (its K is the tokens)
constexpr int ROUTE_DW_BLOCKS = 4;

RouteBwdLayout route_bwd_layout(const moe_cfg &c)
{
    RouteBwdLayout L;
    size_t off = align_up(route_region_bytes(c), 256);
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += align_up(bytes, 256);
        return at;
    };
    L.split = take(3ull * c.E * c.H * 2);
    L.parts = take(3ull * c.T * c.E * 2);
    L.splits = choose_splits(ceil_div(c.H, 256), 3 * ceil_div(c.T, GEMM_BK), 256ll * c.H, 64, 3);
    L.part = take(L.splits > 1 ? 4ull * L.splits * 256 * c.H : 0);
    L.logit_splits = 0;
    if (c.T > ROUTER_SIMT_MAX_T && c.T <= ROUTE_PAIR_LOGITS_MAX_T) {
        L.logit_splits = choose_splits(1, 3 * (c.H / GEMM_BK), 256ll * c.E, 8, 6);
        L.logits = take(4ull * L.logit_splits * 256 * c.E);
    }
    L.total = off;
    return L;
}

}  // namespace

extern "C" {

int moe_block_norm(int32_t T, int32_t H, int32_t groups, int32_t stream_f32, const void *x, const moe_bf16 *y,
                   const float *gate, const float *w_post, const float *w_pre, float alpha, float eps, void *r,
                   moe_bf16 *n, void *stream)
{
    ProfCall prof_call_;
    int rc = check_block_norm(T, H, groups, stream_f32, alpha, eps);
    if (rc != MOE_OK)
        return rc;
    if (!x || !n || (y && !r) || (!y && (gate || w_post)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(gate, 16) || !aligned(w_post, 16) || !aligned(w_pre, 16) ||
        !aligned(r, 16) || !aligned(n, 16))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    BlockNormParams p = {};
    p.T = T;
    p.H = H;
    p.groups = groups;
    p.rows_per_gate = T / groups;
    p.alpha = alpha;
    p.eps = eps;
    p.x = x;
    p.y = y;
    p.gate = gate;
    p.w_post = w_post;
    p.w_pre = w_pre;
    p.r = r;
    p.n = n;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    GLR_LAUNCH(KID_BLOCK_NORM, launch_block_norm(p, stream_f32 != 0, block_norm_blocks(T, H, NORM_SMS), s));
    set_last_launches(launches);
    return MOE_OK;
}

size_t moe_block_norm_workspace_bytes(int32_t T, int32_t H, int32_t groups)
{
    return check_block_norm(T, H, groups, 0, 1.0f, 0.0f) == MOE_OK ? norm_layout(T, H, groups).total : 0;
}

int moe_block_norm_backward(int32_t T, int32_t H, int32_t groups, int32_t stream_f32, const void *x,
                            const moe_bf16 *y, const float *gate, const float *w_post, const float *w_pre,
                            float alpha, float eps, const void *d_r, const moe_bf16 *d_n, void *d_x, moe_bf16 *d_y,
                            float *d_gate, float *dw_post, float *dw_pre, void *ws, size_t ws_bytes, void *stream)
{
    ProfCall prof_call_;
    int rc = check_block_norm(T, H, groups, stream_f32, alpha, eps);
    if (rc != MOE_OK)
        return rc;
    if (!x || !d_n || !d_x || (y && !d_y) || (!y && (gate || w_post || d_y || d_gate || dw_post)))
        return MOE_ERR_INVALID_ARG;
    const NormLayout L = norm_layout(T, H, groups);
    if ((rc = check_ws(ws, ws_bytes, L.total)) != MOE_OK)
        return rc;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(gate, 16) || !aligned(w_post, 16) || !aligned(w_pre, 16) ||
        !aligned(d_r, 16) || !aligned(d_n, 16) || !aligned(d_x, 16) || !aligned(d_y, 16) || !aligned(d_gate, 4) ||
        !aligned(dw_post, 4) || !aligned(dw_pre, 4))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    BlockNormParams p = {};
    p.T = T;
    p.H = H;
    p.groups = groups;
    p.rows_per_gate = T / groups;
    p.cpg = L.plan.cpg;
    p.alpha = alpha;
    p.eps = eps;
    p.x = x;
    p.y = y;
    p.gate = gate;
    p.w_post = w_post;
    p.w_pre = w_pre;
    p.d_r = d_r;
    p.d_n = d_n;
    p.d_x = d_x;
    p.d_y = d_y;
    p.part_a = y ? at<float>(ws, L.part_a) : nullptr;
    p.part_b = at<float>(ws, L.part_b);
    p.d_gate = d_gate;
    p.dw_post = dw_post;
    p.dw_pre = dw_pre;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    GLR_LAUNCH(KID_BLOCK_NORM_BWD, launch_block_norm_backward(p, stream_f32 != 0, L.plan.blocks, s));
    if (d_gate || dw_post || dw_pre)
        GLR_LAUNCH(KID_BLOCK_NORM_BWD, launch_block_norm_finish(p, L.plan.blocks, s));
    set_last_launches(launches);
    return MOE_OK;
}

size_t moe_vocab_loss_workspace_bytes(int32_t T, int32_t H, int32_t V, int backward)
{
    return check_vocab(T, H, V, 32) == MOE_OK ? vocab_layout(T, H, V, backward != 0).total : 0;
}

int moe_vocab_loss(int32_t T, int32_t H, int32_t V, const moe_bf16 *hidden, const moe_bf16 *W_vocab,
                   const void *target, int32_t target_bits, int64_t ignore_index, float *loss, float *lse, void *ws,
                   size_t ws_bytes, void *stream)
{
    ProfCall prof_call_;
    int rc = check_vocab(T, H, V, target_bits);
    if (rc != MOE_OK)
        return rc;
    if (T == 0) {
        set_last_launches(0);
        return MOE_OK;
    }
    if (!hidden || !W_vocab || !target || !loss || !lse)
        return MOE_ERR_INVALID_ARG;
    const VocabLayout L = vocab_layout(T, H, V, false);
    if ((rc = check_ws(ws, ws_bytes, L.total)) != MOE_OK)
        return rc;
    if (!aligned(hidden, 16) || !aligned(W_vocab, 16) || !aligned(target, target_bits / 8) || !aligned(loss, 4) ||
        !aligned(lse, 4))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    VocabMeta *meta = at<VocabMeta>(ws, L.meta);
    int *status = &header(ws)->status;
    VocabRowsParams rp = {};
    rp.T = T;
    rp.V = V;
    rp.target_bits = target_bits;
    rp.target = target;
    rp.ignore = ignore_index;
    rp.meta = meta;
    rp.row_of = at<int>(ws, L.row_of);
    rp.packed_target = at<int>(ws, L.target);
    rp.status = status;
    rp.hidden = hidden;
    rp.packed = at<uint16_t>(ws, L.hidden);
    rp.packed_rows = L.rows;
    rp.H = H;
    rp.loss = loss;
    rp.lse_out = lse;
    GLR_LAUNCH(KID_VOCAB_ROWS, launch_vocab_rows(rp, s));
    const bool few = T <= PAIR_FEW_ROWS;
    PairGemmParams p;
    memset(&p, 0, sizeof(p));
    if (!vocab_logits_maps(p, L, T, H, V, hidden, W_vocab, ws, few ? PAIR_FEW_ROWS : 128))
        return MOE_ERR_CUDA;
    p.meta = meta;
    p.m_from_rows = 1;
    p.N = V;
    p.kblocks = ceil_div(H, GEMM_BK);
    p.part_blocks = ceil_div(p.kblocks, ceil_div(p.kblocks, LOGIT_PART_BLOCKS));
    p.few_rows = LOGIT_EXACT_ROWS;
    p.few_part_blocks = ceil_div(p.kblocks, ceil_div(p.kblocks, LOGIT_EXACT_BLOCKS));
    p.splits = 1;
    p.group_m = vocab_group(H);
    p.target = rp.packed_target;
    p.stats = at<float2>(ws, L.stats);
    p.ld_stats = T;
    p.target_logit = at<float>(ws, L.logit);
    p.status = status;
    GLR_LAUNCH(KID_VOCAB_LOGITS, pair_product(few ? PG_STATS_FEW : PG_STATS, PP_LOGITS, p, ceil_div(T, 256) * L.ntiles,
                                                   s));
    GLR_LAUNCH(KID_VOCAB_JOIN, launch_vocab_join(p.stats, L.nstats, T, p.target_logit, meta, rp.row_of, T, loss, lse,
                                                 s));
    set_last_launches(launches);
    return MOE_OK;
}

int moe_vocab_loss_backward(int32_t T, int32_t H, int32_t V, const moe_bf16 *hidden, const moe_bf16 *W_vocab,
                            const void *target, int32_t target_bits, int64_t ignore_index, const float *lse,
                            const float *d_loss, moe_bf16 *d_hidden, moe_bf16 *dW_vocab, void *ws, size_t ws_bytes,
                            void *stream)
{
    ProfCall prof_call_;
    int rc = check_vocab(T, H, V, target_bits);
    if (rc != MOE_OK)
        return rc;
    if (!W_vocab || !dW_vocab || (T > 0 && (!hidden || !target || !lse || !d_loss || !d_hidden)))
        return MOE_ERR_INVALID_ARG;
    const VocabLayout L = vocab_layout(T, H, V, true);
    if ((rc = check_ws(ws, ws_bytes, L.total)) != MOE_OK)
        return rc;
    if (!aligned(hidden, 16) || !aligned(W_vocab, 16) || !aligned(target, target_bits / 8) || !aligned(lse, 4) ||
        !aligned(d_loss, 4) || !aligned(d_hidden, 16) || !aligned(dW_vocab, 16))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    if (T == 0) {
        set_last_launches(0);
        return cudaMemsetAsync(dW_vocab, 0, 2ull * V * H, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    VocabMeta *meta = at<VocabMeta>(ws, L.meta);
    int *status = &header(ws)->status;
    VocabRowsParams rp = {};
    rp.T = T;
    rp.V = V;
    rp.target_bits = target_bits;
    rp.target = target;
    rp.ignore = ignore_index;
    rp.meta = meta;
    rp.row_of = at<int>(ws, L.row_of);
    rp.packed_target = at<int>(ws, L.target);
    rp.status = status;
    rp.hidden = hidden;
    rp.packed = at<uint16_t>(ws, L.hidden);
    rp.packed_rows = L.rows;
    rp.H = H;
    rp.packed_of = at<int>(ws, L.packed_of);
    rp.dx_kblocks = L.piece / GEMM_BK;
    rp.lse = lse;
    rp.d_loss = d_loss;
    rp.packed_lse = at<float>(ws, L.lse);
    rp.packed_weight = at<float>(ws, L.weight);
    GLR_LAUNCH(KID_VOCAB_ROWS, launch_vocab_rows(rp, s));

    uint16_t *dz = at<uint16_t>(ws, L.dz);
    float *part = at<float>(ws, L.part);
    const int m_tiles = ceil_div(L.rows, 256), h_tiles = ceil_div(H, 256);
    // z again, piece by piece, turned into dz in the epilogue
    PairGemmParams pz, px, pw;
    memset(&pz, 0, sizeof(pz));
    if (!vocab_logits_maps(pz, L, T, H, V, hidden, W_vocab, ws, 128) ||
        !make_map_bf16(&pz.tmOut, dz, L.rows, L.piece, 64, 32))
        return MOE_ERR_CUDA;
    pz.meta = meta;
    pz.m_from_rows = 1;
    pz.kblocks = pz.part_blocks = ceil_div(H, GEMM_BK);
    pz.splits = 1;
    pz.group_m = vocab_group(H);
    pz.out_rows = L.rows;
    pz.target = rp.packed_target;
    pz.lse = rp.packed_lse;
    pz.weight = rp.packed_weight;
    pz.status = status;
    // d_hidden partial sums [splits][rows, H] += dz W
    memset(&px, 0, sizeof(px));
    if (!make_map_bf16(&px.tmA, dz, L.rows, L.piece, GEMM_BK, 128) || !make_map_bf16(&px.tmB, W_vocab, V, H, 64, GEMM_BK) ||
        !make_map_f32(&px.tmOut, part, L.part_rows, H, 32, 32))
        return MOE_ERR_CUDA;
    px.meta = meta;
    px.m_from_rows = 1;
    px.N = H;
    px.group_m = 1;
    px.out_rows = L.part_rows;
    px.out_cols = H;
    px.beside = PG_FIRST;
    px.status = status;
    // dW piece = dz^T hidden
    memset(&pw, 0, sizeof(pw));
    if (!make_map_bf16(&pw.tmA, dz, L.rows, L.piece, 64, GEMM_BK) || !make_map_bf16(&pw.tmB, hidden, T, H, 64, GEMM_BK) ||
        !make_map_bf16(&pw.tmHidden, at<uint16_t>(ws, L.hidden), L.rows, H, 64, GEMM_BK) ||
        !make_map_bf16(&pw.tmOut, dW_vocab, V, H, 64, 32))
        return MOE_ERR_CUDA;
    pw.meta = meta;
    pw.k_from_rows = 1;
    pw.part_blocks = ceil_div(L.rows, GEMM_BK);
    pw.N = H;
    pw.splits = 1;
    pw.group_m = 1;
    pw.out_rows = V;
    pw.out_cols = H;
    pw.beside = PG_SECOND;
    pw.status = status;
    for (int v0 = 0; v0 < V; v0 += L.piece) {
        const int n = std::min(L.piece, V - v0);
        pz.N = pz.out_cols = n;
        pz.n0 = v0;
        pz.b_off[0] = v0;
        GLR_LAUNCH(KID_VOCAB_DLOGITS,
                   pair_product(PG_DLOGITS, PP_LOGITS, pz, m_tiles * ceil_div(n, 256), s));
        px.kblocks = px.part_blocks = ceil_div(n, GEMM_BK);
        px.b_off[0] = v0;
        px.accumulate = v0 > 0;
        GLR_LAUNCH(KID_VOCAB_DX, pair_product(PG_PARTIAL, PP_DX, px, PAIRS, s));
        pw.M = n;
        pw.out_row0 = v0;
        GLR_LAUNCH(KID_VOCAB_DW, pair_product(PG_BF16, PP_DW, pw, ceil_div(n, 256) * h_tiles, s));
    }
    GLR_LAUNCH(KID_VOCAB_DX, launch_vocab_dx_join(part, meta, rp.packed_of, T, H, d_hidden, s));
    set_last_launches(launches);
    return MOE_OK;
}

size_t moe_route_backward_workspace_bytes(const moe_cfg *cfg)
{
    return check_route_cfg(cfg) == MOE_OK ? route_bwd_layout(*cfg).total : 0;
}

int moe_route_backward(const moe_cfg *cfg, const moe_bf16 *hidden, const float *W_router, const moe_bf16 *W_split,
                       const int32_t *topk_idx, const float *d_topk_w, const int32_t *expert_counts,
                       const float *d_aux_loss, const moe_bf16 *d_hidden_add, moe_bf16 *d_hidden, float *dW_router,
                       void *ws, size_t ws_bytes, void *stream)
{
    ProfCall prof_call_;
    int rc = check_route_cfg(cfg);
    if (rc != MOE_OK)
        return rc;
    if (!hidden || !W_router || !topk_idx || !d_topk_w || !d_hidden || !dW_router || (d_aux_loss && !expert_counts))
        return MOE_ERR_INVALID_ARG;
    const moe_cfg &c = *cfg;
    const RouteBwdLayout L = route_bwd_layout(c);
    if ((rc = check_ws(ws, ws_bytes, L.total)) != MOE_OK)
        return rc;
    if (!aligned(hidden, 16) || !aligned(W_router, 4) || !aligned(W_split, 16) || !aligned(topk_idx, 4) ||
        !aligned(d_topk_w, 4) || !aligned(expert_counts, 4) || !aligned(d_aux_loss, 4) || !aligned(d_hidden_add, 16) ||
        !aligned(d_hidden, 16) || !aligned(dW_router, 16))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((rc = device_check(&sms)) != MOE_OK)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    int *status = &header(ws)->status;
    const uint16_t *W3 = W_split;
    if (!W3) {
        uint16_t *own = at<uint16_t>(ws, L.split);
        GLR_LAUNCH(KID_SPLIT, launch_split_router(W_router, own, c.E, c.H, nullptr, s));
        W3 = own;
    }
    float *logits = nullptr;
    int nparts = 1;
    long long part_stride = (long long)c.T * c.E;
    if (L.logit_splits) {
        logits = at<float>(ws, L.logits);
        nparts = L.logit_splits;
        const int rows = 256;
        part_stride = (long long)rows * c.E;
        PairGemmParams p;
        memset(&p, 0, sizeof(p));
        if (!make_map_bf16(&p.tmA, hidden, c.T, c.H, GEMM_BK, 128) ||
            !make_map_bf16(&p.tmB, W3, 3ull * c.E, c.H, GEMM_BK, 128) ||
            !make_map_f32(&p.tmOut, logits, (uint64_t)nparts * rows, c.E, 32, 32))
            return MOE_ERR_CUDA;
        p.M = c.T;
        p.N = c.E;
        p.kblocks = c.H / GEMM_BK;
        p.part_blocks = ROUTE_LOGIT_BLOCKS;
        p.b_off[1] = c.E;
        p.b_off[2] = 2 * c.E;
        p.splits = nparts;
        p.group_m = 1;
        p.out_rows = nparts * rows;
        p.out_cols = c.E;
        p.split_rows = rows;
        p.status = status;
        GLR_LAUNCH(KID_ROUTER_GEMM, pair_product(PG_PARTIAL, PP_LOGITS_PARTS, p, nparts, s));
    } else if ((rc = route_region_logits(c, hidden, W_router, W3, ws, sms, s, launches, &logits, &nparts)) != MOE_OK) {
        return rc;
    }
    uint16_t *parts = at<uint16_t>(ws, L.parts);
    GLR_LAUNCH(KID_ROUTE_BWD_SCORES, launch_route_grad(logits, nparts, part_stride, topk_idx, d_topk_w, expert_counts,
                                                       d_aux_loss, c.T, c.E, c.k, c.rsf, c.eps, parts, status, s));
    const int h_tiles = ceil_div(c.H, 256);
    // d_hidden = dL W: of the parts' products the three largest (the rest is
    // below 2^-16 of the result, which is rounded to bf16)
    PairGemmParams p;
    memset(&p, 0, sizeof(p));
    if (!make_map_bf16(&p.tmA, parts, 3ull * c.T, c.E, GEMM_BK, 128) ||
        !make_map_bf16(&p.tmB, W3, 3ull * c.E, c.H, 64, GEMM_BK) || !make_map_bf16(&p.tmOut, d_hidden, c.T, c.H, 64, 32))
        return MOE_ERR_CUDA;
    p.M = c.T;
    p.N = c.H;
    p.kblocks = p.part_blocks = c.E / GEMM_BK;
    p.a_off[1] = c.T;              // the middle parts
    p.b_off[1] = c.E;
    p.splits = 1;
    p.group_m = 1;
    p.out_rows = c.T;
    p.out_cols = c.H;
    p.beside = PG_FIRST;
    p.status = status;
    if (d_hidden_add && !make_map_bf16(&p.tmHidden, d_hidden_add, c.T, c.H, 64, 32))
        return MOE_ERR_CUDA;
    GLR_LAUNCH(KID_ROUTE_BWD_DX, pair_product(d_hidden_add ? PG_BF16_ADD : PG_BF16, PP_DX_PARTS, p, ceil_div(c.T, 256) * h_tiles, s));
    // dW = dL^T hidden, exact products: low, middle, high part of dL
    float *part = at<float>(ws, L.part);
    memset(&p, 0, sizeof(p));
    if (!make_map_bf16(&p.tmA, parts, 3ull * c.T, c.E, 64, GEMM_BK) ||
        !make_map_bf16(&p.tmB, hidden, c.T, c.H, 64, GEMM_BK) ||
        !(L.splits == 1 ? make_map_f32(&p.tmOut, dW_router, c.E, c.H, 32, 32)
                        : make_map_f32(&p.tmOut, part, 256ull * L.splits, c.H, 32, 32)))
        return MOE_ERR_CUDA;
    p.M = c.E;
    p.N = c.H;
    p.kblocks = ceil_div(c.T, GEMM_BK);
    p.part_blocks = ROUTE_DW_BLOCKS;
    p.a_off[1] = c.T;
    p.a_off[2] = 2 * c.T;
    p.splits = L.splits;
    p.group_m = 1;
    p.out_rows = L.splits == 1 ? c.E : 256 * L.splits;
    p.out_cols = c.H;
    p.split_rows = 256;
    p.beside = PG_SECOND;
    p.status = status;
    GLR_LAUNCH(KID_ROUTE_BWD_DW, pair_product(PG_PARTIAL, PP_DW_PARTS, p, h_tiles * L.splits, s));
    if (L.splits > 1)
        GLR_LAUNCH(KID_ROUTE_BWD_DW, launch_sum_splits(part, L.splits, 256ll * c.H, (long long)c.E * c.H, dW_router, s));
    set_last_launches(launches);
    return MOE_OK;
}

}  // extern "C"
