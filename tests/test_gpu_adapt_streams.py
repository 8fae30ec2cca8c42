"""Buffers that the layer and the adapters allocate for a call on another
stream than the current one: they belong to the stream that writes them."""
import pytest
import torch

import fp8_blockwise_routed_b200 as fm
import moe_inputs as mi
from fp8_blockwise_routed_b200.adapters import LoraAdapters, LoraBatch

pytestmark = pytest.mark.gpu


def _layer(T, seed=3):
    wl = mi.WORKLOADS["tiny"].with_(T=T)
    d = mi.make_inputs(wl, seed, "cuda")
    layer = fm.RoutedMoE(d["w_gate"], d["s_gate"], d["w_up"], d["s_up"], d["w_down"], d["s_down"], wl.k, 2.0, T)
    layer.forward(d["x"], d["logits"])
    return wl, d, layer


def _late_writes(numel, stream):
    """Memory of `numel` floats given back to the allocator while work queued
    on `stream` has still to write it."""
    with torch.cuda.stream(stream):
        t = torch.empty((numel,), device="cuda")
        m = torch.randn((4096, 4096), device="cuda")
        for _ in range(20):
            torch.mm(m, m)
        t.fill_(-7.0)
        del t


@pytest.mark.parametrize("handle", [False, True])
def test_router_backward_on_another_stream(handle):
    """d_logits neither takes over memory that the current stream has still to
    write, nor gives its own to the current stream before it is written."""
    T = 2048
    wl, d, layer = _layer(T)
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    arg = side.cuda_stream if handle else side
    dout = torch.randn((T, wl.H), device="cuda").to(torch.bfloat16)
    want = layer.router_backward(d["logits"], dout).clone()
    torch.cuda.synchronize()
    _late_writes(want.numel(), main)
    got = layer.router_backward(d["logits"], dout, stream=arg)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del got
    _late_writes(want.numel(), side)                       # keeps the side stream busy
    layer.router_backward(d["logits"], dout, stream=arg)   # dropped at once
    other = torch.full_like(want, 5.0)
    torch.cuda.synchronize()
    assert bool((other == 5.0).all())


def test_result_used_on_the_current_stream():
    """A result is not handed out on the side stream while the current one
    still reads it."""
    T = 2048
    wl, d, layer = _layer(T)
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    dout = torch.randn((T, wl.H), device="cuda").to(torch.bfloat16)
    want = layer.router_backward(d["logits"], dout).clone()
    torch.cuda.synchronize()
    got = layer.router_backward(d["logits"], dout, stream=side)
    main.wait_stream(side)
    m = torch.randn((4096, 4096), device="cuda")
    for _ in range(20):
        torch.mm(m, m)
    kept = got.clone()
    del got
    with torch.cuda.stream(side):
        torch.full_like(want, 9.0)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_first_balance_loss_on_another_stream():
    T = 4096
    wl, d, layer = _layer(T)
    wl2, d2, plain = _layer(T)
    loss, counts = plain.balance_loss(d2["logits"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for numel in (2, wl.E + 1, wl.E, (plain.ws_loss.numel() + 3) // 4):
        _late_writes(numel, torch.cuda.current_stream())
    l2, c2 = layer.balance_loss(d["logits"], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(l2, loss) and torch.equal(c2, counts)


def test_first_adapter_gradient_on_another_stream():
    T, K, N, R, n = 900, 512, 1024, 16, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    x, a, b, dout = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
                     for s in ((T, K), (n, R, K), (n, R, N), (T, N)))
    batch = LoraBatch(n, T).assign(torch.arange(T, dtype=torch.int32, device="cuda") % n)
    out = torch.empty((T, N), device="cuda")
    pair = [LoraAdapters(a, b, None, T) for _ in range(2)]
    for ad in pair:
        ad.forward(batch, x, None, out)
    want = pair[0].backward(batch, x, dout)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for t in want:
        _late_writes(t.numel(), torch.cuda.current_stream())
    got = pair[1].backward(batch, x, dout, stream=side)
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)


def test_gradient_after_a_replayed_forward():
    """A replay is not seen by the layer: after it the gradient of the captured
    batch is taken, whatever batch was routed eagerly in between."""
    wl, d, layer = _layer(50)
    dout = torch.randn((50, wl.H), device="cuda").to(torch.bfloat16)
    d_loss = torch.tensor([0.01, 0.001], device="cuda")
    layer.balance_loss(d["logits"])
    want = layer.router_backward(d["logits"], dout, d_loss).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(d["x"], d["logits"])
        layer.balance_loss(d["logits"])
    layer.forward(d["x"][:30], d["logits"][:30])
    graph.replay()
    assert torch.equal(layer.router_backward(d["logits"], dout, d_loss), want)
