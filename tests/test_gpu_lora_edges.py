"""moe_lora and moe_lora_backward at the edges of their ranges and behind one
another on a stream."""
import pytest
import torch

import fp8_blockwise_routed_b200 as fm
from fp8_blockwise_routed_b200.adapters import LoraBatch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [16, 64])
def test_gradient_without_tokens_waits_for_the_call_before(R):
    """A backward call of no tokens writes zeros where the forward call before
    it on the stream wrote its rows: the memory holds the zeros afterwards."""
    T, K, N, n = 6000, 64, 4096, 2
    g = torch.Generator(device="cuda").manual_seed(R)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    a, b = rnd(n, R, K), rnd(n, R, N)
    batch = LoraBatch(n, T).assign(torch.arange(T, dtype=torch.int32, device="cuda") % n)
    v, out = torch.empty((T, R), device="cuda"), torch.empty((T, N), device="cuda")
    none = LoraBatch(n, 0)
    d_a, d_b = out.view(-1)[:n * R * K].view(n, R, K), out.view(-1)[-n * R * N:].view(n, R, N)
    ws = torch.empty((fm.moe_lora_backward_workspace_bytes(0, R),), dtype=torch.uint8, device="cuda")
    x = rnd(T, K)
    for _ in range(10):
        fm.moe_lora(x, a, b, None, batch.offsets, batch.sorted, None, v, out)
        fm.moe_lora_backward(x[:0], a, b, None, none.offsets, none.sorted, v[:0], rnd(0, N), None, None, d_a, d_b, ws)
        assert not d_a.any() and not d_b.any()
        assert bool(out[T // 2].any())
