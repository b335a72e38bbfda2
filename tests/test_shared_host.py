"""The shared expert's and the 4-bit products' entry points without a GPU: size
queries, and bad arguments rejected before any device work."""
import ctypes

import pytest

import mixture_experts_routing_gb300 as moe


@pytest.fixture(scope="module")
def L():
    from mixture_experts_routing_gb300 import _build
    _build.build()
    return moe.lib()


def test_workspace_sizes(L):
    for n, h, i in [(1, 8, 32), (77, 520, 160), (4096, 7168, 2048)]:
        assert moe.shared_backward_workspace_bytes(moe.SharedConfig(n, h, i)) >= 6 * n * i
        assert moe.w4_workspace_bytes(moe.W4Config(n % 100, 128, 8, 8, i // 32 * 32, 32)) >= 2 * (n % 100) * 8 * i
    assert moe.shared_backward_workspace_bytes(moe.SharedConfig(0, 8, 32)) == 0
    assert moe.shared_backward_workspace_bytes(moe.SharedConfig(1 << 22, 8, 1 << 14)) == 6 << 36  # past 32 bits


@pytest.mark.parametrize("field,value,status", [
    ("n_tokens", -1, -1), ("hidden", 0, -1), ("inter", 0, -1), ("activation", 2, -1), ("grad_f32", 2, -1),
    ("hidden", 12, -2), ("inter", 48, -2), ("n_tokens", 1 << 25, -2), ("hidden", 1 << 25, -2), ("inter", 1 << 24, -2)])
def test_shared_config_checks(L, field, value, status):
    cfg = moe.SharedConfig(4, 64, 64)
    setattr(cfg, field, value)
    assert L.moe_shared_backward_workspace_bytes(ctypes.byref(cfg)) == status
    assert L.moe_shared_forward(ctypes.byref(cfg), *[256] * 6, None) == status
    assert L.moe_shared_forward_train(ctypes.byref(cfg), *[256] * 8, None) == status
    assert L.moe_shared_backward(ctypes.byref(cfg), *[256] * 11, 1 << 30, None) == status


def test_shared_pointer_checks(L):
    cfg = moe.SharedConfig(4, 64, 64)
    c = ctypes.byref(cfg)
    need = moe.shared_backward_workspace_bytes(cfg)
    for at in (0, 1, 2, 4, 5):  # x, w13, w2, h, y (add may be missing)
        for bad in (None, 264):
            args = [256] * 6
            args[at] = bad
            assert L.moe_shared_forward(c, *args, None) == -1
    assert L.moe_shared_forward(c, 256, 256, 256, 264, 256, 256, None) == -1  # add misaligned
    for at in range(8):
        args = [256] * 8
        args[at] = 264
        assert L.moe_shared_forward_train(c, *args, None) == -1
    for at in (6, 7):
        args = [256] * 8
        args[at] = None
        assert L.moe_shared_forward_train(c, *args, None) == -1
    # x, w13, w2, ck, ck_sf, dy, dx_add, dx, dw13, dw2, workspace
    for at in range(10):
        args = [256] * 11
        args[at] = 264
        assert L.moe_shared_backward(c, *args, need, None) == -1
    for at in (0, 1, 2, 3, 4, 5, 7, 8, 9):
        args = [256] * 11
        args[at] = None
        assert L.moe_shared_backward(c, *args, need, None) == -1
    for ws, size in ((None, need), (264, need), (256, need - 1)):
        assert L.moe_shared_backward(c, *[256] * 10, ws, size, None) == -3
    assert L.moe_shared_forward(None, *[256] * 6, None) == -1


@pytest.mark.parametrize("field,value,status", [
    ("n_tokens", -1, -1), ("hidden", 0, -1), ("n_experts", 0, -1), ("top_k", 0, -1), ("inter", 0, -1), ("group", 16, -1), ("group", 48, -1), ("group", 0, -1),
    ("activation", 3, -1), ("n_experts", 257, -2), ("top_k", 17, -2), ("hidden", 96, -2), ("inter", 96, -2), ("n_tokens", 513, -2)])
def test_w4_config_checks(L, field, value, status):
    cfg = moe.W4Config(4, 128, 8, 2, 128, 64)
    setattr(cfg, field, value)
    assert L.moe_w4_workspace_bytes(ctypes.byref(cfg)) == status
    assert L.moe_w4_ffn_forward(ctypes.byref(cfg), *[256] * 10, 1 << 30, None) == status


def test_w4_pointer_checks(L):
    cfg = moe.W4Config(4, 128, 8, 2, 128, 64)
    c, need = ctypes.byref(cfg), moe.w4_workspace_bytes(cfg)
    # topk_ids, topk_p, x, w13q, w13_scale, w2q, w2_scale, add, y, workspace
    for at in (0, 1, 2, 3, 4, 5, 6, 8):
        args = [256] * 10
        args[at] = None
        assert L.moe_w4_ffn_forward(c, *args, need, None) == -1
    for at in range(2, 9):
        args = [256] * 10
        args[at] = 264
        assert L.moe_w4_ffn_forward(c, *args, need, None) == -1
    for ws, size in ((None, need), (264, need), (256, need - 1)):
        assert L.moe_w4_ffn_forward(c, *[256] * 9, ws, size, None) == -3
    good = [256, 256, 256, 2, 16, 128, 64, 256]  # x, q, scale, n, rows, cols, group, y
    for at, bad, status in ((0, None, -1), (1, 264, -1), (2, None, -1), (3, -1, -1), (3, 1025, -2), (4, 0, -1), (5, 96, -1), (6, 16, -1), (7, None, -1)):
        args = list(good)
        args[at] = bad
        assert L.moe_w4_matvec(*args, None) == status
    for args in ((256, -1, 128, 64, 256, 256), (256, 4, 96, 64, 256, 256), (256, 4, 128, 16, 256, 256), (None, 4, 128, 64, 256, 256), (264, 4, 128, 64, 256, 256)):
        assert L.moe_w4_quantize(*args, None) == -1
    assert L.moe_w4_quantize(None, 0, 128, 64, None, None, None) == 0
    assert L.moe_w4_matvec(None, None, None, 0, 16, 128, 64, None, None) == 0
