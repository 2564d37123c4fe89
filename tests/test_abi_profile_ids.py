"""Ids of moe_profile_read and moe_kernel_name are part of the ABI: those of the
layer's kernels keep their values, and the training operators' kernels have a
range of their own."""
import ctypes

import pytest

from group_limited_routing_gb300 import _lib, build, moe

LAYER = ["split_router", "router_gemm", "route_select", "route_finalize", "bucket_hist", "bucket_scan",
         "bucket_scatter", "gemm_gate_up_swiglu", "gemm_down", "combine", "dense_tiles", "bwd_gate_up_recompute",
         "bwd_dgrad_down_swiglu", "bwd_dgrad_x", "bwd_weight_grads", "bwd_pad_and_dw", "router_route_bucket",
         "bucket_tiles", "router_plus_permute"]
TRAIN = ["block_norm", "block_norm_backward", "vocab_rows", "vocab_logits", "vocab_join", "vocab_dlogits",
         "vocab_d_hidden", "vocab_d_weight", "route_backward_scores", "route_backward_d_hidden",
         "route_backward_d_weight"]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_layer_ids(lib):
    assert _lib.MOE_KERNEL_COUNT == 19 and _lib.MOE_KERNEL_STAGE_ROUTE_PERMUTE == 18
    assert [lib.moe_kernel_name(i).decode() for i in range(19)] == LAYER


def test_training_ids(lib):
    first, n = _lib.MOE_KERNEL_TRAIN_FIRST, _lib.MOE_KERNEL_TRAIN_COUNT
    assert first > _lib.MOE_KERNEL_COUNT
    assert [lib.moe_kernel_name(i).decode() for i in range(first, first + n)] == TRAIN
    ms, launches = ctypes.c_double(), ctypes.c_int32()
    ids = set(range(19)) | set(range(first, first + n))
    for i in range(-2, first + n + 2):
        rc = lib.moe_profile_read(i, ctypes.byref(ms), ctypes.byref(launches), 0)
        assert rc == (_lib.MOE_OK if i in ids else _lib.MOE_ERR_INVALID_ARG), i
        assert bool(lib.moe_kernel_name(i)) == (i in ids)


def test_binding_reads_both_ranges(lib):
    assert set(moe.profile_read()) == set(LAYER + TRAIN)
