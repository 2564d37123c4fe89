// Internal interface between api_expert_ops.cu and the kernels of the operators
// around a layer's experts: token order (tokens.cu), 8-bit products (scaled.cu,
// scaled_gemm.cu) and the optimiser (optim.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace glr {

// ------------------------------------------------------------ token order
constexpr int ORDER_MAX_E = 512;
constexpr int ORDER_THREADS = 512;
constexpr int ORDER_CHUNK = 2048;       // pairs per block at least
constexpr int ORDER_MAX_BLOCKS = 128;   // ... and blocks at most (each reads every block's counts)

inline __host__ __device__ int order_ld(int E) { return (E + 3) / 4 * 4; }

struct OrderPlan {
    int blocks;
    long long chunk;    // pairs per block
};

inline OrderPlan order_plan(long long pairs)
{
    long long chunk = (pairs + ORDER_MAX_BLOCKS - 1) / ORDER_MAX_BLOCKS;
    chunk = chunk < ORDER_CHUNK ? ORDER_CHUNK : (chunk + ORDER_THREADS - 1) / ORDER_THREADS * ORDER_THREADS;
    const long long blocks = (pairs + chunk - 1) / chunk;
    return {blocks < 1 ? 1 : (int)blocks, chunk};
}

cudaError_t launch_order_count(const int32_t *idx, long long pairs, int E, OrderPlan plan, int32_t *hist, cudaStream_t s);
cudaError_t launch_order_assign(const int32_t *idx, long long pairs, int E, OrderPlan plan, const int32_t *hist,
                                int32_t *offsets, int32_t *slot_of, int *status, cudaStream_t s);
// rows of `vecs` 16-byte vectors
cudaError_t launch_sort_rows(const void *x, long long T, int k, long long vecs, long long R, const int32_t *slot_of,
                             void *rows, cudaStream_t s);
cudaError_t launch_unsort_rows(const void *y, bool f32, long long T, int k, int H, long long R, const int32_t *slot_of,
                               const float *w, void *out, int sms, cudaStream_t s);
cudaError_t launch_unsort_backward(const void *d_out, const void *y, bool f32, long long T, int k, int H, long long R,
                                   const int32_t *slot_of, const float *w, void *d_y, float *d_w, cudaStream_t s);

// --------------------------------------------------------- 8-bit operands
constexpr int SCALED_BLOCK = 128;
constexpr int SCALED_MAX_E = 1024;

struct QuantParams {
    const void *x;            // [R, K] bf16 or fp32
    long long R;
    int K, kblocks;           // kblocks = ceil(K / 128)
    bool f32, e5m2;
    // rows form
    uint8_t *q, *scale;       // [rows, K]; [kblocks, ld]
    long long ld;
    // rows form, each row to its slots
    const int32_t *slot_of;   // [R, k] or null
    int k;
    long long rows;           // rows of q
    // columns form: [K, P] and [P / 128, ld_t]
    uint8_t *qt, *scale_t;
    long long P, ld_t;
    const int32_t *starts;    // [E + 1] blocks, with offsets; null: one group of R rows
    const int32_t *offsets;   // [E + 1] rows
    int E;
    int batch;                // x is [batch, R, K] and the outputs as many (no groups then)
};

cudaError_t launch_quantize_slots(const QuantParams &p, cudaStream_t s);
cudaError_t launch_quantize_tiles(const QuantParams &p, bool rows, bool columns, cudaStream_t s);
cudaError_t launch_column_starts(const int32_t *offsets, int E, long long R, int32_t *starts, cudaStream_t s);

// --------------------------------------------------------- 8-bit products
enum ScaledMode { SM_DENSE = 0, SM_ROWS = 1, SM_SUM = 2 };

struct ScaledGemmParams {
    CUtensorMap tmA, tmB, tmSA, tmSB;
    int mode;
    int M, N;                 // of the output (a group's, with SM_SUM)
    int kblocks;              // 128 of K each (SM_SUM: from starts)
    int E;                    // groups (0: none)
    int band;                 // row tiles that are taken together for all columns
    const int32_t *bounds;    // SM_ROWS: offsets; SM_SUM: starts ([E + 1])
    void *out;
    bool out_f32;
    bool wide;                // the output's rows start on 32-byte boundaries
    bool a_e5m2, b_e5m2;
    int *status;
    unsigned long long wait_limit_ns;
    int inject_withhold;
};

// rows of SA's box: 128 and a start that is not on a 16-byte boundary
constexpr int SCALED_SA_BOX = 144;
constexpr int SCALED_CHUNK = 4;         // blocks of 128 whose scales a box holds
struct ScaledTile {
    int columns;
    bool pair;                // 256 rows on two CTAs, else 128 on one
};
ScaledTile scaled_tile(int mode, int M, int N, int E, int kblocks, bool f32, int sms);
cudaError_t launch_scaled_gemm(const ScaledGemmParams &p, ScaledTile tile, int max_units, cudaStream_t s);

// -------------------------------------------------------------- optimiser
constexpr int ADAM_UNIT = 2048;         // elements per block of the step
constexpr int ADAM_TABLE = 128;         // tensors per launch
constexpr int ADAM_TABLE_SMALL = 16;

struct AdamTensor {
    void *p;
    const void *g;
    float *master;
    void *m, *v;
    uint8_t *m_scale, *v_scale;
    long long n;
    double weight_decay;
    float decay;              // 1 - lr weight_decay
    uint32_t key;             // of its random numbers, without the step's share
    int kind;                 // bit 0: 8-bit states, 1: p bf16, 2: g bf16, 3: master; bit 4: vectors are aligned
    int pad;
};

struct AdamScalars {
    double lr, beta1, beta2;
    float b1, one_b1, b2, one_b2, eps;
    float size, inv;          // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
    float one;                // 1 (its value is not for the compiler to know)
    uint32_t step_key;
    long long step_host;
    const float *grad_scale;
    const int64_t *step;      // on the device, or null
    const float *lr_dev;
};

template <int N>
struct AdamTable {
    AdamScalars c;
    int count, units;
    int unit0[N];             // each tensor's first unit (side by side: every block searches them)
    AdamTensor t[N];
};

cudaError_t launch_adamw(const AdamTable<ADAM_TABLE> &t, bool states_8, cudaStream_t s);
cudaError_t launch_adamw(const AdamTable<ADAM_TABLE_SMALL> &t, bool states_8, cudaStream_t s);

constexpr int NORM_UNIT = 8192;
constexpr int NORM_TABLE = 128;
constexpr int NORM_MAX_BLOCKS = 608;    // per launch

struct NormTensor {
    const void *g;
    long long n;
    int bf16, aligned;
    int unit0, pad;
};

struct NormTable {
    int count, units, blocks, first;    // first: of this launch's partial sums
    NormTensor t[NORM_TABLE];
};

cudaError_t launch_grad_norm(const NormTable &t, double *partial, cudaStream_t s);
cudaError_t launch_grad_norm_finish(const double *partial, int n, float max_norm, float *norm, float *scale, cudaStream_t s);

}  // namespace glr
