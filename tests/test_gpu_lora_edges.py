"""moe_lora and moe_lora_backward at the edges of their ranges and behind one
another on a stream."""
import pytest
import torch

import fp8_blockwise_routed_b200 as fm
from fp8_blockwise_routed_b200.adapters import LoraAdapters, LoraBatch

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


# barriers of moe_debug_waits
EXPAND_SLAB, EXPAND_FREE, SHRINK_FULL, SHRINK_EMPTY, OUTER_FULL, OUTER_EMPTY = 1, 2, 4, 8, 16, 32
LIMIT_NS = 50_000_000


@pytest.fixture
def held():
    yield lambda mask: fm.moe_debug_waits(LIMIT_NS, mask)
    torch.cuda.synchronize()
    fm.moe_debug_waits(0, 0)


@pytest.mark.parametrize("R", [64, 100])
@pytest.mark.parametrize("barrier", [EXPAND_SLAB, EXPAND_FREE])
def test_expand_whose_wait_runs_out(held, barrier, R):
    """Where a wait of the wide expand runs out the rows' columns say so, in
    FP32 and BF16; the others are right, and the next call is."""
    T, K, N, n = 4200, 64, 4096, 2
    g = torch.Generator(device="cuda").manual_seed(R)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    x, a, b = rnd(T, K), rnd(n, R, K), rnd(n, R, N)
    base = torch.randn((T, N), generator=g, device="cuda")
    batch = LoraBatch(n, T).assign(torch.arange(T, dtype=torch.int32, device="cuda") % n)

    def forward():
        v = torch.empty((T, R), device="cuda")
        out, o16 = torch.full((T, N), -7.0, device="cuda"), torch.full((T, N), -7.0, device="cuda").to(torch.bfloat16)
        fm.moe_lora(x, a, b, None, batch.offsets, batch.sorted, base, v, out, o16)
        return v, out, o16

    v, out, o16 = forward()
    held(barrier)
    v1, out1, o161 = forward()
    torch.cuda.synchronize()
    fm.moe_debug_waits(0, 0)
    assert torch.equal(v1, v)                              # the first product has no part in it
    gone = torch.isnan(out1)
    assert torch.equal(torch.isnan(o161), gone) and bool(gone.any())
    assert torch.equal(out1[~gone], out[~gone]) and torch.equal(o161[~gone], o16[~gone])
    if barrier == EXPAND_SLAB:                             # no product without its rank rows
        assert bool(gone.all())
    for p, q in zip(forward(), (v, out, o16)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("T,R", [(600, 16), (600, 64), (700, 100), (9000, 64)])
@pytest.mark.parametrize("barrier", [SHRINK_FULL, SHRINK_EMPTY])
def test_shrink_whose_wait_runs_out(held, barrier, T, R):
    """Where a wait of the tiled shrink runs out, v and all that is made of it
    are NaN; rows without an adapter stay, and the next call is right."""
    K, N, n = 4096, 264, 3
    g = torch.Generator(device="cuda").manual_seed(T + R)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    x, a, b = rnd(T, K), rnd(n, R, K), rnd(n, R, N)
    ids = torch.arange(T, dtype=torch.int32, device="cuda") % (n + 1) - 1
    batch = LoraBatch(n, T).assign(ids)
    base, has = torch.randn((T, N), generator=g, device="cuda"), ids >= 0

    def forward():
        v, out = torch.full((T, R), -7.0, device="cuda"), base.clone()
        fm.moe_lora(x, a, b, None, batch.offsets, batch.sorted, out, v, out)
        return v, out

    v, out = forward()
    held(barrier)
    v1, out1 = forward()
    torch.cuda.synchronize()
    fm.moe_debug_waits(0, 0)
    P = int(has.sum())
    assert torch.isnan(v1[:P]).all() and torch.equal(v1[P:], v[P:])
    assert torch.isnan(out1[has]).all() and torch.equal(out1[~has], base[~has])
    for p, q in zip(forward(), (v, out)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("T,K,R,n", [(9000, 512, 64, 3), (9000, 1024, 64, 40), (3000, 256, 100, 2), (16000, 256, 8, 4)])
@pytest.mark.parametrize("barrier", [OUTER_FULL, OUTER_EMPTY])
def test_gradient_product_whose_wait_runs_out(held, barrier, T, K, R, n):
    """Where a wait of the gradient product runs out the entries concerned are
    NaN; the others and dx are right, and so is the next call."""
    g = torch.Generator(device="cuda").manual_seed(T + R)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    x, dout, a, b = rnd(T, K), rnd(T, K), rnd(n, R, K), rnd(n, R, K)
    batch = LoraBatch(n, T).assign(torch.arange(T, dtype=torch.int32, device="cuda") % n)
    v = torch.randn((T, R), generator=g, device="cuda")

    def backward():
        dx = torch.full((T, K), -7.0, device="cuda")
        d_a, d_b = torch.full((n, R, K), -7.0, device="cuda"), torch.full((n, R, K), -7.0, device="cuda")
        ws = torch.empty((fm.moe_lora_backward_workspace_bytes(T, R),), dtype=torch.uint8, device="cuda")
        fm.moe_lora_backward(x, a, b, None, batch.offsets, batch.sorted, v, dout, None, dx, d_a, d_b, ws)
        return dx, d_a, d_b

    want = backward()
    held(barrier)
    got = backward()
    torch.cuda.synchronize()
    fm.moe_debug_waits(0, 0)
    assert torch.equal(got[0], want[0])
    for p, q in zip(got[1:], want[1:]):
        gone = torch.isnan(p)
        assert bool(gone.any()) and torch.equal(p[~gone], q[~gone])
        if barrier == OUTER_FULL:                          # no stage ever comes in
            assert bool(gone.all())
    for p, q in zip(backward(), want):
        assert torch.equal(p, q)


def test_micro_batches_add_up():
    """Gradients of two micro-batches in buffers of their own add up to those
    of the whole batch (rounded apart: 2^-24 each, over at most 3 * 40 / 16 + 64
    additions of either side, relative to the sums of absolute products)."""
    K, N, R, n = 64, 48, 8, 2
    g = torch.Generator(device="cuda").manual_seed(2)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    x, dout, a, b = rnd(80, K), rnd(80, N), rnd(n, R, K), rnd(n, R, N)
    ids = torch.arange(80, dtype=torch.int32, device="cuda") % n
    ad = LoraAdapters(a, b, None, 80)
    batch, out = LoraBatch(n, 80), torch.empty((80, N), device="cuda")
    got = []
    for lo in (0, 40):
        batch.assign(ids[lo:lo + 40])
        ad.forward(batch, x[lo:lo + 40], None, out[:40])
        got.append(ad.backward(batch, x[lo:lo + 40], dout[lo:lo + 40], d_a=torch.empty(a.shape, device="cuda"),
                               d_b=torch.empty(b.shape, device="cuda")))
    batch.assign(ids)
    ad.forward(batch, x, None, out)
    whole = ad.backward(batch, x, dout)
    u = 2.0 ** -24
    for i in range(n):
        t = ids == i
        xa, da = x[t].double().abs(), dout[t].double().abs()
        dv, v = da @ b[i].double().abs().T, xa @ a[i].double().abs().T
        for w, p, q, mag in ((whole[0], got[0][0], got[1][0], dv.T @ xa), (whole[1], got[0][1], got[1][1], v.T @ da)):
            diff = (w[i].double() - p[i].double() - q[i].double()).abs()
            assert bool((diff <= 4 * (72 + 72) * 2 * u * mag).all())
