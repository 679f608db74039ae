"""What the fine-tuning entry points refuse, on the host and before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

import grouped_gemm_03_b200 as gg

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P, NULL, BIG = ctypes.c_void_p(0x10000), None, 1 << 40
ODD = ctypes.c_void_p(0x10004)
Q = ctypes.c_void_p(0x90000)


@pytest.fixture(scope="module")
def L():
    from grouped_gemm_03_b200.build import build
    build()
    return gg.lib()


def _loss(L, logits=P, dtype=0, idx=P, T=16, E=8, k=2, off=NULL, S=1, loss=P, counts=P, coef=P, ws=P, n=BIG):
    return L.moe_balance_loss(logits, dtype, idx, T, E, k, off, S, NULL, 0.1, loss, counts, NULL, coef, ws, n, NULL)


def test_balance_loss(L):
    assert _loss(L, k=9) == INVALID and _loss(L, E=0) == INVALID and _loss(L, E=2000) == INVALID
    assert _loss(L, T=-1) == INVALID and _loss(L, S=0) == INVALID and _loss(L, dtype=3) == INVALID
    assert _loss(L, S=2) == INVALID                      # several sequences need offsets
    assert _loss(L, off=P, S=(1 << 20) + 1) == UNSUPPORTED and _loss(L, T=1 << 29) == UNSUPPORTED
    assert _loss(L, logits=NULL) == INVALID and _loss(L, idx=NULL) == INVALID and _loss(L, logits=ODD) == INVALID
    assert _loss(L, loss=NULL) == INVALID and _loss(L, counts=NULL) == INVALID and _loss(L, coef=NULL) == INVALID
    assert _loss(L, ws=NULL) == WORKSPACE and _loss(L, ws=ctypes.c_void_p(0x10010)) == WORKSPACE
    need = L.moe_balance_loss_workspace_size(16, 8, 1)
    assert need >= 256 and _loss(L, n=need - 1) == WORKSPACE
    assert L.moe_balance_loss_workspace_size(-1, 8, 1) == 0


def _grad(L, logits=P, dtype=0, idx=P, dw=P, T=16, E=8, k=2, off=NULL, S=1, counts=NULL, coef=NULL, out=Q, odt=0):
    return L.moe_router_backward(logits, dtype, idx, dw, T, E, k, 0, off, S, NULL, counts, coef, NULL, out, odt, NULL)


def test_router_backward(L):
    assert _grad(L, dw=NULL) == INVALID                  # nothing to differentiate
    assert _grad(L, counts=P) == INVALID and _grad(L, coef=P) == INVALID
    assert _grad(L, k=9) == INVALID and _grad(L, dtype=4) == INVALID and _grad(L, odt=3) == INVALID
    assert _grad(L, out=NULL) == INVALID and _grad(L, out=ODD) == INVALID and _grad(L, out=P, odt=2) == INVALID
    assert _grad(L, T=1 << 29) == UNSUPPORTED and _grad(L, S=3) == INVALID


def test_adapter_plan(L):
    call = L.moe_adapter_plan
    assert call(P, 10, 0, P, P, P, BIG, NULL) == INVALID and call(P, -1, 2, P, P, P, BIG, NULL) == INVALID
    assert call(P, 10, 1025, P, P, P, BIG, NULL) == UNSUPPORTED
    assert call(P, (1 << 30) + 1, 2, P, P, P, BIG, NULL) == UNSUPPORTED
    assert call(NULL, 10, 2, P, P, P, BIG, NULL) == INVALID and call(P, 10, 2, NULL, P, P, BIG, NULL) == INVALID
    assert call(P, 10, 2, P, P, P, L.moe_adapter_plan_workspace_size(10, 2) - 1, NULL) == WORKSPACE


def _lora(L, x=P, A=P, B=P, off=P, order=P, n=2, rows=10, d=64, N=64, R=8, base=NULL, out=Q, dt=2, ws=NULL,
          nb=0):
    return L.moe_lora(x, A, B, NULL, off, order, n, rows, d, N, R, base, out, dt, NULL, ws, nb, NULL)


def test_lora(L):
    for R in (4, 12, 136):
        assert _lora(L, R=R) == UNSUPPORTED
    assert _lora(L, R=0) == INVALID and _lora(L, d=68) == UNSUPPORTED and _lora(L, N=60) == UNSUPPORTED
    assert _lora(L, d=(1 << 20) + 8) == UNSUPPORTED and _lora(L, N=(1 << 20) + 8) == UNSUPPORTED
    assert _lora(L, n=0) == INVALID and _lora(L, n=1025) == UNSUPPORTED and _lora(L, rows=-1) == INVALID
    assert _lora(L, dt=1) == INVALID and _lora(L, out=P) == INVALID      # out must not be x
    for name in ("x", "A", "B", "off", "order", "out"):
        assert _lora(L, **{name: NULL}) == INVALID
    for name in ("x", "A", "B", "base", "out"):
        assert _lora(L, **{name: ODD}) == INVALID
    big = dict(rows=8192, n=2, d=7168, N=4096, R=32)   # two launches, with h between them
    need = L.moe_lora_workspace_size(8192, 2, 7168, 4096, 32)
    assert need > 0 and L.moe_lora_workspace_size(10, 2, 64, 64, 8) == 0
    assert L.moe_lora_workspace_size(8192, 2, 7168, 4096, 20) == 0
    assert _lora(L, **big) == WORKSPACE and _lora(L, ws=P, nb=need - 1, **big) == WORKSPACE
    assert _lora(L, ws=ODD, nb=BIG, **big) == WORKSPACE


def _back(L, dC=P, x=P, h=P, n=2, rows=10, d=64, N=64, R=8, dx=Q, dxt=2, dA=Q, dB=Q, gt=0, ws=P, nb=BIG):
    return L.moe_lora_backward(dC, x, h, P, P, NULL, P, P, n, rows, d, N, R, NULL, dx, dxt, dA, dB, gt, ws, nb, NULL)


def test_lora_backward(L):
    assert _back(L, dx=NULL, dA=NULL, dB=NULL) == INVALID
    assert _back(L, R=20) == UNSUPPORTED and _back(L, d=4) == UNSUPPORTED and _back(L, gt=1) == INVALID
    assert _back(L, dxt=1) == INVALID and _back(L, h=NULL) == INVALID and _back(L, dx=P) == INVALID
    assert _back(L, dA=ODD) == INVALID and _back(L, ws=NULL) == WORKSPACE
    assert _back(L, nb=L.moe_lora_backward_workspace_size(10, 2, 64, 64, 8) - 1) == WORKSPACE
    assert L.moe_lora_backward_workspace_size(10, 2, 64, 64, 20) == 0


def _comb(L, g=P, dt=2, Y=P, t2r=P, w=P, off=NULL, E=0, T=10, d=64, k=2, dY=Q, dw=Q):
    return L.moe_combine_backward(g, dt, Y, t2r, w, off, E, 0, T, d, k, dY, dw, NULL)


def test_combine_backward(L):
    assert _comb(L, dY=NULL, dw=NULL) == INVALID and _comb(L, Y=NULL) == INVALID
    assert _comb(L, dY=P) == INVALID and _comb(L, dt=1) == INVALID and _comb(L, k=33) == INVALID
    assert _comb(L, d=60) == UNSUPPORTED and _comb(L, T=1 << 29) == UNSUPPORTED and _comb(L, off=P, E=0) == INVALID
    assert _comb(L, g=NULL) == INVALID and _comb(L, t2r=NULL) == INVALID and _comb(L, dY=ODD) == INVALID


def test_binding_refuses_host_tensors():
    t, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gg.balance_loss(t, i, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        gg.router_backward(t, i, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        gg.combine_backward(t, t, i, torch.zeros(4, 2), False)
    with pytest.raises(ValueError, match="CUDA"):
        gg.adapter_plan(i[:, 0].contiguous(), 2)
    b = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        gg.lora(b, b[None], b[None], i[:, 0], i[:, 0])


def test_binding_refuses_what_is_no_tensor():
    with pytest.raises(TypeError, match="logits"):
        gg.balance_loss([1.0], torch.zeros(4, 2, dtype=torch.int32), 0.1)
    with pytest.raises(TypeError, match="row_adapter"):
        gg.adapter_plan(None, 2)
    with pytest.raises(TypeError):
        gg.lora(1, 2, 3, 4, 5)


@pytest.mark.parametrize("n", [(1 << 31), (1 << 32) + 5, -(1 << 32) + 5, -(1 << 31) - 1])
def test_binding_refuses_adapters_past_32_bits(n):
    # a number cut to 32 bits would pass for another one, and offsets is made for the one that was asked for
    with pytest.raises(ValueError, match="adapters"):
        gg.adapter_plan(torch.zeros(4, dtype=torch.int32), n)
