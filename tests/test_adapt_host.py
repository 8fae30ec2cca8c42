"""Host-side checks of the router-gradient and adapter entry points, without a
GPU: argument checks of the C ABI, refusals of the binding."""
import ctypes

import pytest
import torch

import fp8_blockwise_routed_b200 as fm
from test_abi_host import A, MIS, L  # noqa: F401  (stand-in addresses and the library fixture)

f1 = ctypes.c_float(1.0)


def test_balance_loss_validation(L):  # noqa: F811
    ws = L.moe_balance_loss_workspace_bytes(100, 8)
    assert ws >= 7 * (8 + 4 + 8 * 4)
    assert L.moe_balance_loss_workspace_bytes(-1, 8) == 0
    assert L.moe_balance_loss(A, 100, 0, A, A, A, A, A, ws, None) == 1
    assert L.moe_balance_loss(A, 100, 1025, A, A, A, A, A, ws, None) == 1
    assert L.moe_balance_loss(A, -1, 8, A, A, A, A, A, ws, None) == 1
    assert L.moe_balance_loss(None, 100, 8, A, A, A, A, A, ws, None) == 1
    assert L.moe_balance_loss(A, 100, 8, None, A, A, A, A, ws, None) == 1
    assert L.moe_balance_loss(A, 100, 8, A, A, MIS, A, A, ws, None) == 3
    assert L.moe_balance_loss(A, 100, 8, A, A, A, A, A, ws - 1, None) == 4
    assert L.moe_balance_loss(A, 1 << 31, 8, A, A, A, A, A, 1 << 40, None) == 2
    assert L.moe_balance_loss(A, 100, 8, A, A, A, A, A, ws, None) == 5      # no device here


def test_balance_workspace_is_bounded(L):  # noqa: F811
    # the number of partial sums stops growing with T
    assert L.moe_balance_loss_workspace_bytes(1 << 20, 256) == L.moe_balance_loss_workspace_bytes(1 << 24, 256)


def _route_bwd(L, T=4, E=8, k=2, y=A, dout=A, H=256, counts=A, d_loss=A, out=A, logits=A):  # noqa: F811
    return L.moe_route_backward(logits, T, E, A, A, k, y, dout, H, f1, counts, d_loss, out, None)


def test_route_backward_validation(L):  # noqa: F811
    assert _route_bwd(L, E=0) == 1
    assert _route_bwd(L, k=0) == 1
    assert _route_bwd(L, k=33) == 1
    assert _route_bwd(L, H=200) == 1
    assert _route_bwd(L, H=32768) == 1
    assert _route_bwd(L, y=None, d_loss=None) == 1        # nothing to differentiate
    assert _route_bwd(L, dout=None) == 1
    assert _route_bwd(L, counts=None) == 1
    assert _route_bwd(L, out=None) == 1
    assert _route_bwd(L, y=MIS) == 3
    assert _route_bwd(L, out=MIS) == 3
    assert _route_bwd(L, T=1 << 31) == 2
    assert _route_bwd(L, T=0) == 0                        # T = 0: no-op
    assert _route_bwd(L, y=None, dout=None, k=0, H=0) == 5   # balance terms alone: valid, no device here
    assert _route_bwd(L, counts=None, d_loss=None) == 5      # routing weights alone


def _lora(L, T=4, K=256, N=128, n=3, R=16, ld_x=None, ld_base=None, ld_out=None, x=A, base=A, out=A, v=A):  # noqa: F811
    return L.moe_lora(x, ld_x or K, T, K, A, A, A, n, R, N, A, A, base, ld_base or N, v, out, ld_out or N, None, None)


def test_lora_validation(L):  # noqa: F811
    for bad in (dict(T=-1), dict(K=0), dict(K=16392), dict(N=0), dict(N=16392), dict(n=0), dict(n=1025), dict(R=0),
                dict(R=129), dict(ld_x=248), dict(ld_x=260), dict(ld_out=124), dict(ld_out=130), dict(ld_base=120),
                dict(x=None), dict(out=None), dict(v=None)):
        assert _lora(L, **bad) == 1, bad
    assert _lora(L, K=252) == 2 and _lora(L, N=132) == 2 and _lora(L, T=(1 << 24) + 1) == 2
    assert _lora(L, x=MIS) == 3 and _lora(L, base=MIS) == 3 and _lora(L, v=MIS) == 3
    assert _lora(L, T=0) == 0
    assert _lora(L) == 5 and _lora(L, base=None) == 5


def _lora_bwd(L, T=4, K=256, N=128, n=3, R=16, ws=None, dx=A, dx_base=A, d_a=A, ld_dout=None):  # noqa: F811
    ws = L.moe_lora_backward_workspace_bytes(T, R) if ws is None else ws
    return L.moe_lora_backward(A, K, T, K, A, A, A, n, R, N, A, A, A, A, ld_dout or N, dx_base, K, dx, K, d_a, A, A,
                               ws, None)


def test_lora_backward_validation(L):  # noqa: F811
    assert L.moe_lora_backward_workspace_bytes(100, 16) >= 100 * 16 * 4
    assert L.moe_lora_backward_workspace_bytes(-1, 16) == 0
    for bad in (dict(R=0), dict(R=129), dict(n=0), dict(d_a=None), dict(dx=None), dict(ld_dout=132)):
        assert _lora_bwd(L, **bad) == 1, bad
    assert _lora_bwd(L, K=100) == 2
    assert _lora_bwd(L, d_a=MIS) == 3
    assert _lora_bwd(L, ws=64) == 4
    assert _lora_bwd(L) == 5
    assert _lora_bwd(L, dx=None, dx_base=None) == 5          # no gradient of x: valid


def _refused(call, *args):
    with pytest.raises(fm.MoeError) as e:
        call(*args)
    assert e.value.code == 1
    return str(e.value)


def test_binding_refuses_host_tensors():
    z = torch.zeros
    lg = z((4, 8))
    assert "logits" in _refused(fm.moe_balance_loss, lg, z(9, dtype=torch.int32), z(2), z(9, dtype=torch.int32), z(8),
                                z(4096, dtype=torch.uint8))
    assert "logits" in _refused(fm.moe_route_backward, lg, None, None, None, None, 1.0, None, z(2), z((4, 8)))
    x = z((4, 16), dtype=torch.bfloat16)
    a = z((1, 2, 16), dtype=torch.bfloat16)
    off, tok = z(2, dtype=torch.int32), z(4, dtype=torch.int32)
    assert "x is on" in _refused(fm.moe_lora, x, a, a, None, off, tok, None, z((4, 2)), z((4, 16)))
    assert "x is on" in _refused(fm.moe_lora_backward, x, a, a, None, off, tok, z((4, 2)), x, None, None,
                                 z((1, 2, 16)), z((1, 2, 16)), z(256, dtype=torch.uint8))
