"""Sizes that no launch can take are refused before anything is launched (CPU)."""
import ctypes

import mx_block_scaled_amax_amd as qf8

SHAPE = -3
F = ctypes.c_void_p(0x10000)


def test_more_tiles_than_a_launch_holds():
    """A launch has fewer than 2^32 threads."""
    lib = qf8._load()

    def mm(m, n, k=4, kind=0, out=0):
        return lib.matmul_block(F, F, F, F, m, n, k, 0, 0, kind, 0, F, out, F, 1 << 40, None)
    assert mm((1 << 31) - 1, 128) == SHAPE and mm(1 << 30, 4096, out=1) == SHAPE and mm(1 << 30, 4096, kind=1) == SHAPE
    assert mm(1 << 30, 1 << 20, kind=2) == SHAPE
    assert lib.matmul_block_experts(F, F, 64, F, F, F, 8, F, (1 << 31) - 1, 256, 4, 0, 0, 0, 0, F, 0, None) == SHAPE
    assert lib.matmul_block_experts_wgrad(F, F, F, F, F, 1024, 128, 1 << 20, 1 << 20, 0, 0, 0, F, 1, None) == SHAPE


def test_more_tokens_than_a_launch_holds():
    lib = qf8._load()

    def route(t, k=2):
        return lib.route_experts(F, 0, t, 8, k, 0, None, 1, 1, 1, 1.0, F, F, None)

    def route_backward(t):
        return lib.route_experts_backward(F, 0, t, 8, F, F, 2, 0, 1, 1.0, F, None)

    def combine(t, r=64):
        return lib.combine_experts(F, 0, r, 8, F, F, t, 2, F, None)

    def combine_backward(t, r):
        return lib.combine_experts_backward(F, F, 0, r, 8, F, F, F, t, 2, F, F, None)
    assert route(1 << 26) == SHAPE and route_backward(1 << 26) == SHAPE
    assert combine(1 << 24) == SHAPE and combine_backward(1 << 24, 64) == SHAPE
    assert combine_backward(64, 1 << 30) == SHAPE and combine_backward((1 << 24) - 64, 1 << 12) == SHAPE
    # the largest that is taken: past the checks of sizes, where a missing pointer is found
    assert lib.combine_experts(F, 0, 64, 8, F, F, (1 << 24) - 1, 2, None, None) == -1
    assert lib.route_experts(F, 0, (1 << 26) - 1, 8, 2, 0, None, 1, 1, 1, 1.0, F, None, None) == -1
    assert lib.combine_experts_backward(F, F, 0, 1 << 12, 8, F, F, F, (1 << 24) - 65, 2, None, F, None) == -1


def test_flags_of_products():
    """fp32 sums for BF16 results are bit 16; other bits are refused. Their workspace is that of FP32 results."""
    lib = qf8._load()

    def mm(flags, ws_bytes):
        return lib.matmul_block(F, F, F, F, 8, 128, 65536, 0, 0, 0, flags, None, 0, F, ws_bytes, None)
    assert mm(32, 1 << 40) == -2 and mm(16 | 4, 1 << 40) == -2
    assert mm(16, 1 << 40) == -1 and mm(17, 1 << 40) == -1                                       # only y is missing

    def short(flags, out):
        need = lib.matmul_block_workspace_bytes(8, 128, 65536, 0, 1)
        return lib.matmul_block(F, F, F, F, 8, 128, 65536, 0, 0, 0, flags, F, out, F, need - 1, None)
    assert short(16, 0) == -5 and short(0, 1) == -5
