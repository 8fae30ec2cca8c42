"""moe_balance_loss and moe_route_backward at the edges of their ranges and
beside other work."""
import numpy as np
import pytest
import torch

import fp8_blockwise_routed_b200 as fm
from test_gpu_route_grad import U, _exact_grad, _exact_probs, _gamma, _grad_case, _loss, _route

pytestmark = pytest.mark.gpu


def _offsets(T, E, k):
    """Offsets of T * k pairs spread over the experts."""
    return torch.div(torch.arange(E + 1, device="cuda") * T * k, E, rounding_mode="floor").to(torch.int32)


def _loss_buffers(T, E):
    return (torch.full((2,), -7.0, device="cuda"), torch.full((E + 1,), -7, dtype=torch.int32, device="cuda"),
            torch.full((E,), -7.0, device="cuda"),
            torch.full((fm.moe_balance_loss_workspace_bytes(T, E),), 255, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("T,E", [(4096, 256), (3001, 257), (66667, 4)])
def test_blocks_that_start_apart_join_alike(T, E):
    """The blocks that join the partial sums get their SMs one by one when
    another stream keeps the GPU busy; the losses keep their bits."""
    z = torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    off = _offsets(T, E, 2)
    want = _loss_buffers(T, E)
    fm.moe_balance_loss(z, off, *want)
    assert torch.isfinite(want[0]).all()
    busy = torch.cuda.Stream()
    work = torch.randn((1 << 24,), device="cuda")
    m = torch.randn((2048, 2048), device="cuda")
    busy.wait_stream(torch.cuda.current_stream())
    got = [_loss_buffers(T, E) for _ in range(40)]
    for i, g in enumerate(got):
        with torch.cuda.stream(busy):
            work.mul_(1.0)
            torch.mm(m, m)
        fm.moe_balance_loss(z, off, *g)
    torch.cuda.synchronize()
    for g in got:
        for p, q in zip(g[:3], want[:3]):
            assert torch.equal(p, q)


# barriers of moe_debug_waits
LOSS, GRAD_FULL, GRAD_EMPTY = 64, 128, 256
LIMIT_NS = 50_000_000


@pytest.fixture
def held():
    yield lambda mask: fm.moe_debug_waits(LIMIT_NS, mask)
    torch.cuda.synchronize()
    fm.moe_debug_waits(0, 0)


@pytest.mark.parametrize("T,E", [(4096, 256), (70001, 8), (2500, 512)])
def test_loss_whose_wait_runs_out(held, T, E):
    """Losses of rows that did not come in say so, and so does the gradient
    that is taken with their counts; the pairs per expert do not depend on
    them.  The next call is right."""
    z = torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    off = _offsets(T, E, 2)
    want = _loss_buffers(T, E)
    fm.moe_balance_loss(z, off, *want)
    held(LOSS)
    loss, counts, mean, ws = _loss_buffers(T, E)
    fm.moe_balance_loss(z, off, loss, counts, mean, ws)
    torch.cuda.synchronize()
    fm.moe_debug_waits(0, 0)
    assert torch.isnan(loss).all() and torch.isnan(mean).all()
    assert torch.equal(counts[:E], want[1][:E]) and int(counts[E]) == -2 ** 30
    counts[E] += T          # as summed with another rank's
    d = torch.zeros_like(z)
    fm.moe_route_backward(z, None, None, None, None, 1.0, counts, torch.ones((2,), device="cuda"), d)
    assert torch.isnan(d).all()
    fm.moe_balance_loss(z, off, loss, counts, mean, ws)
    for p, q in zip((loss, counts, mean), want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("T,E,k,H", [(600, 64, 8, 5120), (450, 300, 10, 2048), (1000, 16, 2, 4096)])
@pytest.mark.parametrize("barrier", [GRAD_FULL, GRAD_EMPTY])
def test_routing_gradient_whose_wait_runs_out(held, barrier, T, E, k, H):
    """A token whose slot rows did not come in has NaN at its chosen experts;
    everything else of the gradient is right, and so is the next call."""
    g = torch.Generator(device="cuda").manual_seed(T)
    z = torch.randn((T, E), generator=g, device="cuda")
    w, ids = torch.softmax(z, 1).topk(k, 1)
    ids = ids.to(torch.int32)
    ids[::5] = -1                                          # tokens without experts
    y = torch.randn((T, k, H), generator=g, device="cuda")
    dout = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    off, (loss, counts, mean, ws) = _offsets(T, E, k), _loss_buffers(T, E)
    fm.moe_balance_loss(z, off, loss, counts, mean, ws)
    d_loss = torch.ones((2,), device="cuda")

    def backward():
        d = torch.full((T, E), -7.0, device="cuda")
        fm.moe_route_backward(z, ids, w, y, dout, 1.5, counts, d_loss, d)
        return d

    want = backward()
    assert torch.isfinite(want).all()
    held(barrier)
    got = backward()
    torch.cuda.synchronize()
    fm.moe_debug_waits(0, 0)
    chosen = torch.zeros((T, E), dtype=torch.bool, device="cuda")
    t, j = torch.nonzero(ids >= 0, as_tuple=True)
    chosen[t, ids[t, j].long()] = True
    gone = torch.isnan(got)
    assert bool(gone.any()) and not bool((gone & ~chosen).any()) and torch.equal(got[~gone], want[~gone])
    if barrier == GRAD_FULL:
        assert torch.equal(gone, chosen)
    assert torch.equal(backward(), want)


# Logits far out: whole rows of one value (a padded token masked with it), one
# such logit beside ordinary ones, and it beside its negative.  The bounds are
# those of the ordinary ranges (imported): an exponential is off by its
# argument's rounding (u |z - max|, exact for logits within a factor two) and
# by 4 u, so a row's probabilities do not lose by where its maximum lies; what
# lies 104 or more below it is 0 in both.
FAR = [1e9, 3e9, -1e9, 1e10, -1e10, -65504.0, 1e20, -1e20, 1e30, -1e30, 2e38, -2e38, 3.3e38]
FAR_SHAPES = [(65, 8), (40, 24), (50, 48), (33, 130), (70, 256), (41, 300), (21, 1024), (4096, 256), (40001, 8),
              (3001, 257)]


def _far(z, val):
    T, E = z.shape
    z[::4] = val
    z[1::8, E // 3] = val
    z[5::8] = -val
    z[5::8, E // 2] = val
    return z


@pytest.mark.parametrize("val", FAR)
@pytest.mark.parametrize("T,E", FAR_SHAPES)
def test_losses_of_far_logits(T, E, val):
    g = torch.Generator(device="cuda").manual_seed(T)
    z = _far(torch.randn((T, E), generator=g, device="cuda") * 3, val)
    ids, w, off = _route(z, 2)
    assert torch.isfinite(w).all()                         # the router takes them
    loss, counts, mean = _loss(z, off, fill=255)
    p, lse, some, ep = _exact_probs(z)
    c = counts[:-1].double().cpu().numpy()
    assert int(counts[-1]) == T
    want = p.mean(0)
    tol = ep.mean(0) + (_gamma(T / 16 + 17) + U) * want
    assert np.all(np.abs(mean.double().cpu().numpy() - want) <= tol)
    wl = E * (c * want).sum() / c.sum()
    assert abs(float(loss[0]) - wl) <= E * (c * tol).sum() / c.sum() + 2 * U * wl
    wz = (lse ** 2).mean()
    if wz < 1e38 and np.abs(lse).max() < 1e18:             # (beyond FP32's range: below)
        el = U * (np.abs(lse) + 5 * np.log(max(E, 2)) + E / 32 + 32)
        assert abs(float(loss[1]) - wz) <= (2 * np.abs(lse) * el + el ** 2).mean() + 18 * U * wz
    elif wz > 4e38:
        assert float(loss[1]) == np.inf


@pytest.mark.parametrize("val", FAR)
@pytest.mark.parametrize("T,E,k,H", [(45, 8, 2, 128), (33, 130, 3, 256), (40, 256, 8, 128), (29, 300, 4, 128),
                                     (17, 1024, 9, 128)])
def test_gradient_of_far_logits(T, E, k, H, val):
    z, ids, w, off, y, dout = _grad_case(T, E, k, H, "plain", 2.5, seed=T)
    _far(z, val)
    ids, w, off = _route(z, k)
    _, counts, _ = _loss(z, off)
    d_loss = torch.tensor([0.7, -0.3], device="cuda")
    for use_y, use_loss in ((True, True), (True, False), (False, True)):
        d = torch.full((T, E), -7.0, device="cuda")
        fm.moe_route_backward(z, ids if use_y else None, w if use_y else None, y if use_y else None,
                              dout if use_y else None, 2.5, counts if use_loss else None,
                              d_loss if use_loss else None, d)
        want, tol = _exact_grad(z, ids, w, y if use_y else None, dout, 2.5, counts, d_loss if use_loss else None)
        got = d.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol), (use_y, use_loss)


def test_without_losses_no_softmax_takes_part():
    """d_loss None leaves the routing weights' part alone: a +Inf logit, whose
    softmax is NaN, reaches the chosen experts of its own row only (through
    the router's NaN weights)."""
    T, E, k, H = 23, 40, 3, 256
    z, ids, w, off, y, dout = _grad_case(T, E, k, H, "plain", 2.5, seed=5)
    z[3, 7] = torch.inf
    ids, w, off = _route(z, k)
    assert torch.isnan(w[3]).all()
    d = torch.full((T, E), -7.0, device="cuda")
    fm.moe_route_backward(z, ids, w, y, dout, 2.5, None, None, d)
    keep = torch.arange(T, device="cuda") != 3
    want, tol = _exact_grad(z[keep], ids[keep], w[keep], y[keep], dout[keep], 2.5, None, None)
    assert np.all(np.abs(d[keep].double().cpu().numpy() - want) <= tol)
    others = torch.ones((E,), dtype=torch.bool, device="cuda")
    others[ids[3].long()] = False
    assert torch.isnan(d[3][~others]).all() and not d[3][others].any()


@pytest.mark.parametrize("T,E", [(4096, 256), (1000, 16), (3001, 257), (40001, 8)])
def test_z_loss_of_a_few_far_rows(T, E):
    """Squares beyond FP32's range do not lose a mean within it.  lse is off by
    u (|lse| + ...) as above: relative 2 u + u from far rows, and the sum of 16
    ordinary ones in FP32 does not matter beside them."""
    z = torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(9), device="cuda")
    z[5], z[T - 2] = -1e20, 3e19
    ids, w, off = _route(z, 2)
    loss, counts, _ = _loss(z, off)
    want = ((z[5, 0].double() ** 2 + z[T - 2, 0].double() ** 2) / T).item()
    assert 1e34 < want < 1e38 and abs(float(loss[1]) - want) <= 8 * U * want


def test_gradient_where_the_z_slope_is_beyond_fp32():
    """2 d1 lse / N beyond FP32's range: its products with the probabilities
    are finite where they lie within it, and 0 at logits that are not
    selectable.  Relative bound: p as above (E / 32 + 32 units) and three
    products; the balance term, 1e-6 of it at most, is included in `want`."""
    T, E = 6, 1024
    z = torch.full((T, E), -3e38, device="cuda")
    z[:, ::2] = -torch.inf
    z[4:] = torch.randn((2, E), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    counts = torch.full((E + 1,), 12, dtype=torch.int32, device="cuda")
    counts[E] = T
    d_loss = torch.tensor([0.5, 700.0], device="cuda")
    d = torch.full((T, E), -7.0, device="cuda")
    fm.moe_route_backward(z, None, None, None, None, 1.0, counts, d_loss, d)
    want, tol = _exact_grad(z, None, None, None, None, 1.0, counts, d_loss)
    slope = 2 * 700.0 / T * 3e38
    assert slope > 3.5e38 and np.abs(want).max() < 3e38
    assert not d[:4, ::2].any()
    got = d.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= np.maximum(tol, (E / 32 + 48) * U * np.abs(want)))
