"""Refusals of the few-token layer, layer norm and AdamW: the library's argument checks
(no GPU work happens before them) and the binding's, without a GPU."""
import ctypes
import math

import pytest
import torch

import mixture_experts_routing_gb300 as moe

INVALID, SHAPE, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module", autouse=True)
def library():
    from mixture_experts_routing_gb300 import _build
    _build.build()


def few(**over):
    cfg = moe.FewConfig(4, 128, 8, 2, 64)
    for k, v in over.items():
        setattr(cfg, k, v)
    return cfg


@pytest.mark.parametrize("field,value,status", [
    ("n_tokens", -1, INVALID), ("n_tokens", 65, SHAPE), ("hidden", 0, INVALID), ("hidden", 96, SHAPE), ("hidden", 16448, SHAPE),
    ("n_experts", 0, INVALID), ("n_experts", 257, SHAPE), ("top_k", 0, INVALID), ("top_k", 9, INVALID), ("inter", 32, SHAPE),
    ("inter", -64, INVALID), ("inter", 16448, SHAPE), ("renorm", 2, INVALID), ("activation", 2, INVALID),
])
def test_few_config(field, value, status):
    cfg = few(**{field: value})
    assert moe.lib().moe_few_workspace_bytes(ctypes.byref(cfg)) == status
    with pytest.raises(moe.MoEError) as e:
        moe.few_workspace_bytes(cfg)
    assert e.value.status == status
    args = [16] * 10 + [16, 1 << 30, None]
    assert moe.lib().moe_few_forward(ctypes.byref(cfg), *args) == status


def test_few_top_k_over_16():
    cfg = few(n_experts=32, top_k=17)
    assert moe.lib().moe_few_workspace_bytes(ctypes.byref(cfg)) == SHAPE


# x, w_router, bias, w13, w2, add, n_valid, y, topk_ids, topk_p
@pytest.mark.parametrize("at,value", [(0, None), (1, None), (3, None), (4, None), (7, None), (0, 8), (1, 2), (2, 2), (3, 8), (4, 8), (5, 8), (6, 2), (7, 8), (8, 2), (9, 1)])
def test_few_pointers(at, value):
    args = [1024] * 10
    args[at] = value
    assert moe.lib().moe_few_forward(ctypes.byref(few()), *args, 1024, 1 << 30, None) == INVALID


def test_few_workspace():
    L, cfg = moe.lib(), few()
    need = moe.few_workspace_bytes(cfg)
    assert need > 0
    for ws, size in ((None, need), (1024, need - 1), (1032, need), (1024, 0)):
        assert L.moe_few_forward(ctypes.byref(cfg), *[1024] * 10, ws, size, None) == WORKSPACE
    assert L.moe_few_forward(ctypes.byref(few(n_tokens=0)), *[None] * 11, 0, None) == 0


def norm(**over):
    cfg = moe.NormConfig(4, 64)
    for k, v in over.items():
        setattr(cfg, k, v)
    return cfg


@pytest.mark.parametrize("field,value,status", [
    ("n_tokens", -1, INVALID), ("hidden", 0, INVALID), ("hidden", 60, SHAPE), ("hidden", 16392, SHAPE), ("kind", 2, INVALID),
    ("eps", -1e-5, INVALID), ("eps", math.inf, INVALID), ("eps", math.nan, INVALID),
])
def test_norm_config(field, value, status):
    L, cfg = moe.lib(), norm(**{field: value})
    assert L.moe_norm_backward_workspace_bytes(ctypes.byref(cfg)) == status
    assert L.moe_norm_forward(ctypes.byref(cfg), *[1024] * 8, None) == status
    assert L.moe_norm_backward(ctypes.byref(cfg), *[1024] * 10, 1 << 30, None) == status


# x, add, weight, bias, sum, y, mean, rstd
@pytest.mark.parametrize("change", [
    {0: None}, {2: None}, {5: None}, {1: None}, {4: None}, {0: 8}, {1: 8}, {2: 8}, {3: 8}, {4: 8}, {5: 8}, {6: 2}, {7: 2}, {4: 2048, 5: 2048},
])
def test_norm_forward_pointers(change):
    args = [1024, 1024, 1024, 1024, 2048, 4096, 1024, 1024]
    for at, value in change.items():
        args[at] = value
    assert moe.lib().moe_norm_forward(ctypes.byref(norm()), *args, None) == INVALID


def test_norm_forward_rms_has_no_mean():
    assert moe.lib().moe_norm_forward(ctypes.byref(norm(kind=1)), *[1024, 1024, 1024, 1024, 2048, 4096, 1024, 1024], None) == INVALID


# x, weight, mean, rstd, dy, dx_add, dx, dweight, dbias
@pytest.mark.parametrize("change", [
    {0: None}, {1: None}, {2: None}, {3: None}, {4: None}, {6: None}, {7: None}, {0: 8}, {1: 8}, {2: 2}, {3: 1}, {4: 8}, {5: 8}, {6: 8}, {7: 8}, {8: 8},
])
def test_norm_backward_pointers(change):
    args = [1024] * 9
    for at, value in change.items():
        args[at] = value
    assert moe.lib().moe_norm_backward(ctypes.byref(norm()), *args, 1024, 1 << 30, None) == INVALID


def test_norm_backward_rms_has_no_mean_and_needs_its_workspace():
    L = moe.lib()
    assert L.moe_norm_backward(ctypes.byref(norm(kind=1)), *[1024] * 9, 1024, 1 << 30, None) == INVALID
    need = moe.norm_backward_workspace_bytes(norm())
    for ws, size in ((None, need), (1024, need - 1), (1032, need)):
        assert L.moe_norm_backward(ctypes.byref(norm()), *[1024] * 9, ws, size, None) == WORKSPACE


def adamw(**over):
    cfg = moe.AdamWConfig(0.9, 0.999, 1e-3, 1e-8, 8, 0)
    for k, v in over.items():
        setattr(cfg, k, v)
    return cfg


@pytest.mark.parametrize("field,value", [
    ("beta1", 1.0), ("beta1", -0.1), ("beta2", math.nan), ("beta2", 1.5), ("lr", math.inf), ("lr", math.nan), ("eps", 0.0), ("eps", 1e-31), ("eps", -1.0),
    ("eps", math.inf), ("state_bits", 16),
])
def test_adamw_config(field, value):
    assert moe.lib().moe_adamw_step(ctypes.byref(adamw(**{field: value})), None, 0, None, None, 1024, None) == INVALID


@pytest.mark.parametrize("change", [
    dict(param=None), dict(param=8), dict(master=8), dict(grad=None), dict(grad=8), dict(m=None), dict(m=8), dict(v=None), dict(v=8),
    dict(m_scale=None), dict(m_scale=2), dict(v_scale=None), dict(n=-1), dict(n=1 << 41), dict(first=-1), dict(first=8), dict(weight_decay=math.nan),
    dict(weight_decay=math.inf), dict(grad_bf16=2),
])
def test_adamw_tensors(change):
    good = dict(param=1024, master=1024, grad=1024, m=1024, v=1024, m_scale=1024, v_scale=1024, n=8, first=0, weight_decay=0.0, grad_bf16=0)
    table = (moe._AdamWTensorC * 2)(moe._AdamWTensorC(**good), moe._AdamWTensorC(**{**good, **change}))
    L = moe.lib()
    assert L.moe_adamw_step(ctypes.byref(adamw()), ctypes.byref(table), 2, None, None, 1024, None) == INVALID


def test_adamw_call():
    L = moe.lib()
    for n, table, lr, scale, steps in ((-1, None, None, None, 1024), (1, None, None, None, 1024), ((1 << 20) + 1, 1024, None, None, 1024),
                                       (0, None, None, None, None), (0, None, None, None, 1026), (0, None, 2, None, 1024), (0, None, None, 2, 1024)):
        assert L.moe_adamw_step(ctypes.byref(adamw()), table, n, lr, scale, steps, None) == INVALID
    assert L.moe_adamw_step(None, None, 0, None, None, 1024, None) == INVALID


def test_bindings_refuse_host_tensors():
    bf, f32 = torch.bfloat16, torch.float32
    x, w = torch.zeros((4, 64), dtype=bf), torch.ones(64)
    with pytest.raises(ValueError, match="x must be"):
        moe.norm_forward(moe.NormConfig(4, 64), x, w, x)
    with pytest.raises(ValueError, match="x must be"):
        moe.norm_backward(moe.NormConfig(4, 64, kind=moe.NORM_RMS), x, w, None, torch.ones(4), x, x, w, torch.zeros(256, dtype=torch.uint8))
    x = torch.zeros((4, 128), dtype=bf)
    with pytest.raises(ValueError, match="x must be"):
        moe.few_forward(few(), x, torch.zeros((128, 8), dtype=f32), None, torch.zeros((8, 128, 128), dtype=bf), torch.zeros((8, 128, 64), dtype=bf), x,
                        torch.zeros(256, dtype=torch.uint8))
    p = torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        moe.AdamW([p], [p.clone()], lr=1e-3)
    for kw in (dict(params=[], grads=[]), dict(params=[p], grads=[]), dict(params=[p], grads=[p], weight_decay=[0.1, 0.1]), dict(params=[p], grads=[p], state_bits=4)):
        with pytest.raises(ValueError):
            moe.AdamW(lr=1e-3, **kw)
