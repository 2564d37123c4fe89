// What the C-ABI files (api.cu, api_train.cu) share: argument checks, the
// per-launch profiling records, tensor maps and the workspace header.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "moe.h"

namespace glr {
namespace host {

// ids of moe_profile_read / moe_kernel_name
enum KernelId {
    KID_SPLIT = 0, KID_ROUTER_GEMM, KID_SELECT, KID_FINALIZE, KID_HIST, KID_SCAN, KID_SCATTER,
    KID_GEMM_GATE_UP, KID_GEMM_DOWN, KID_COMBINE, KID_DENSE_TILES, KID_BWD_RECOMPUTE, KID_BWD_DGRAD,
    KID_BWD_DX, KID_BWD_WGRAD, KID_BWD_MISC, KID_ROUTE_FUSED, KID_TILES,
    KID_STAGE_ROUTE_PERMUTE,  // (per-stage timing) the routing and bucketing kernels as one interval
    KID_BLOCK_NORM = MOE_KERNEL_TRAIN_FIRST, KID_BLOCK_NORM_BWD, KID_VOCAB_ROWS, KID_VOCAB_LOGITS, KID_VOCAB_JOIN, KID_VOCAB_DLOGITS,
    KID_VOCAB_DX, KID_VOCAB_DW, KID_ROUTE_BWD_SCORES, KID_ROUTE_BWD_DX, KID_ROUTE_BWD_DW, KID_END
};
static_assert(KID_STAGE_ROUTE_PERMUTE == MOE_KERNEL_STAGE_ROUTE_PERMUTE &&
              KID_STAGE_ROUTE_PERMUTE + 1 == MOE_KERNEL_COUNT &&
              KID_END == MOE_KERNEL_TRAIN_FIRST + MOE_KERNEL_TRAIN_COUNT, "ids are part of the ABI");

// whether a launch is to be sabotaged (moe_debug_inject_timeout); counts it
bool take_injected_timeout();

// kernels the last call of this thread enqueued (moe_last_launch_count)
void set_last_launches(int n);

struct ProfRecord {
    cudaEvent_t start, stop;
    int kid;
};

// brackets one launch with events while profiling is on
struct ProfScope {
    bool on;
    ProfRecord r;
    cudaStream_t s;
    ProfScope(int kid, cudaStream_t st);
    void done();
};

// At the end of every public call that launches kernels: closes the stage
// left open by its last launch.
struct ProfCall {
    ~ProfCall();
};

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline WsHeader *header(void *ws) { return static_cast<WsHeader *>(ws); }

template <typename T>
T *at(void *ws, size_t off)
{
    return reinterpret_cast<T *>(static_cast<char *>(ws) + off);
}

int check_route_cfg(const moe_cfg *c);
int check_ws(void *ws, size_t ws_bytes, size_t need);
int device_check(int *sms);

// 2D tensor [rows, cols] (row-major), box [box_rows, box_cols] of 128 bytes,
// 128-byte swizzle, zero fill outside the tensor
bool make_map_bf16(CUtensorMap *m, const void *ptr, uint64_t rows, uint64_t cols, uint32_t box_cols,
                   uint32_t box_rows);
bool make_map_f32(CUtensorMap *m, const void *ptr, uint64_t rows, uint64_t cols, uint32_t box_cols,
                  uint32_t box_rows);

// The routing region at the start of a workspace (header first) and the fp32
// logits [T, E] computed into it with the weight's bf16 x 3 split W_split, as
// *nparts buffers T E floats apart whose sum they are (the router GEMM's K parts).
size_t route_region_bytes(const moe_cfg &c);
int route_region_logits(const moe_cfg &c, const moe_bf16 *hidden, const float *W, const moe_bf16 *W_split, void *ws,
                        int sms, cudaStream_t s, int &launches, float **logits, int *nparts);

}  // namespace host
}  // namespace glr

#define GLR_LAUNCH(kid, expr)                  \
    do {                                       \
        ProfScope prof_scope_((kid), s);       \
        if ((expr) != cudaSuccess)             \
            return MOE_ERR_CUDA;               \
        prof_scope_.done();                    \
        ++launches;                            \
    } while (0)
