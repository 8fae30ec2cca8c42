"""moe_balance_loss and moe_route_backward against the definitions in 64 bits,
with tolerances derived from FP32 rounding (u = 2^-24):

  expf is within 2 ulp and z - max is rounded once, so an exponential is off
  by a relative u (|z - max| + 4); a sum of E positive ones in at most
  E / 32 + 5 additions, its reciprocal and the product add E / 32 + 8:
  relative error of p[t, e] <= u (|z - max| + |z - max|_p + E / 32 + 16),
  where the sum's own error is at most that of its largest contributions
  (bounded by 4 + E / 32 + 5 plus the mean |z - max| under p).
  prob_mean adds at most T / 16 + 16 additions of positive terms per block
  (FP64 across blocks).  The squares of lse are summed 16 at a time in FP32
  (at most 16 u of the sum of these positive terms), beyond that in FP64.
  Dots of H terms run in at most H / 256 + 64 steps.
"""
import numpy as np
import pytest
import torch

import fp8_blockwise_routed_b200 as fm
import moe_inputs as mi

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _gamma(m):
    return m * U / (1 - m * U)


def _logits(T, E, kind, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn((T, E), generator=g, device="cuda") * 3
    if kind == "masked":
        z[torch.rand((T, E), generator=g, device="cuda") < 0.5] = -torch.inf
        z[torch.rand((T, E), generator=g, device="cuda") < 0.1] = torch.nan
        z[::7] = -torch.inf
        z[3::11] = torch.nan
        if T > 4:
            z[4] = -torch.inf
            z[4, E // 2] = 2.5          # one selectable expert
    elif kind == "lowest":              # the type's lowest value is selectable, unlike -Inf
        z[:, ::2] = torch.finfo(torch.float32).min
    elif kind == "wide":
        z *= 1000.0
    elif kind == "equal":
        z[:] = 0.5
    return z


def _route(z, k):
    T, E = z.shape
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    off = torch.empty((E + 1,), dtype=torch.int32, device="cuda")
    sp = torch.empty((max(T * k, 1),), dtype=torch.int32, device="cuda")
    ws = torch.empty((fm.moe_route_workspace_bytes(T, E, k),), dtype=torch.uint8, device="cuda")
    fm.moe_route(z, k, ids, w, off, sp, ws)
    return ids, w, off


def _loss(z, off, fill=0):
    T, E = z.shape
    loss = torch.full((2,), -7.0, device="cuda")
    counts = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    mean = torch.full((E,), -7.0, device="cuda")
    ws = torch.full((fm.moe_balance_loss_workspace_bytes(T, E),), fill, dtype=torch.uint8, device="cuda")
    fm.moe_balance_loss(z, off, loss, counts, mean, ws)
    return loss, counts, mean


def _exact_probs(z):
    """p [T, E], lse [T], counted rows and the error bound of p, in 64 bits."""
    z = z.double().cpu().numpy()
    ok = ~np.isnan(z) & (z > -np.inf)
    some = ok.any(1)
    m = np.where(some, np.max(np.where(ok, z, -np.inf), axis=1, initial=-np.inf), 0.0)
    d = np.where(ok, z - m[:, None], 0.0)
    ex = np.where(ok, np.exp(d), 0.0)
    tot = np.where(some, ex.sum(1), 1.0)
    p = ex / tot[:, None]
    dist = np.abs(d)
    rel = U * (dist + (p * dist).sum(1, keepdims=True) + z.shape[1] / 32 + 32)
    # FP32's smallest positive values: below them p rounds to 0
    return p, np.where(some, m + np.log(tot), 0.0), some, rel * p + 1e-37


SHAPES = [(1, 1, 1), (1, 5, 2), (3, 8, 8), (33, 64, 2), (130, 65, 6), (257, 256, 8), (1000, 257, 4), (37, 1024, 32),
          (5003, 8, 2), (70, 30, 3), (9, 6, 2)]
# beyond one cluster's share: bulk copies (whole 16-byte rows) and plain loads
LARGE = [(4096, 256, 8), (1029, 256, 8), (70001, 8, 2), (30011, 12, 2), (4444, 64, 4), (3333, 100, 4), (2500, 512, 8),
         (1500, 1024, 8), (3001, 257, 4), (66667, 7, 2), (9001, 30, 2), (2111, 130, 3), (300, 1023, 5), (40000, 20, 3)]


@pytest.mark.parametrize("kind", ["plain", "masked", "lowest", "wide", "equal"])
@pytest.mark.parametrize("T,E,k", SHAPES + LARGE)
def test_balance_loss(T, E, k, kind):
    z = _logits(T, E, kind, seed=T + E)
    ids, w, off = _route(z, k)
    loss, counts, mean = _loss(z, off, fill=255)
    p, lse, some, ep = _exact_probs(z)
    n = int(some.sum())
    i = ids.cpu().numpy()
    c = np.bincount(i[i >= 0], minlength=E)
    assert np.array_equal(counts.cpu().numpy(), np.append(c, n))
    nn = max(n, 1)
    adds = _gamma(T / 16 + 17) + U
    want = p.sum(0) / nn
    tol = ep.sum(0) / nn + adds * want
    got = mean.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol)
    P = max(int(c.sum()), 1)
    wl = E * (c * want).sum() / P
    got_l = loss.double().cpu().numpy()
    assert abs(got_l[0] - wl) <= E * (c * tol).sum() / P + 2 * U * wl
    with np.errstate(over="ignore"):
        wz = np.float64(np.float32((lse[some] ** 2).sum() / nn)) if n else 0.0
    # log(sum) is within 2 ulp of the log of a sum off by U (E / 32 + 16 + mean distance); max added with one rounding
    entropy = -(p * np.log(np.maximum(p, 1e-300))).sum(1)
    el = U * (np.abs(lse) + 5 * np.log(max(E, 2)) + E / 32 + 16 + entropy)
    if np.isfinite(wz):
        assert abs(got_l[1] - wz) <= (2 * np.abs(lse[some]) * el[some] + el[some] ** 2).sum() / nn + 18 * U * wz + 1e-37
    else:
        assert got_l[1] == wz


def test_balance_of_nothing():
    """No rows, or rows without a selectable expert: zeros, not NaN."""
    for z in (torch.empty((0, 8), device="cuda"), torch.full((5, 8), -torch.inf, device="cuda"),
              torch.full((2, 300), torch.nan, device="cuda")):
        E = z.shape[1]
        loss, counts, mean = _loss(z, torch.zeros((E + 1,), dtype=torch.int32, device="cuda"))
        assert torch.equal(loss, torch.zeros_like(loss)) and torch.equal(mean, torch.zeros_like(mean))
        assert torch.equal(counts, torch.zeros_like(counts))
        d = torch.full(z.shape, -7.0, device="cuda")
        fm.moe_route_backward(z, None, None, None, None, 1.0, counts, torch.ones((2,), device="cuda"), d)
        assert torch.equal(d, torch.zeros_like(d))


def test_uniform_routing_has_loss_one():
    z = torch.zeros((64, 8), device="cuda")
    off = torch.arange(0, 9, dtype=torch.int32, device="cuda") * 16
    loss, _, mean = _loss(z, off)
    assert torch.equal(mean, torch.full((8,), 0.125, device="cuda")) and loss[0].item() == 1.0


def test_infinite_logit_gives_nan_as_in_the_router():
    z = _logits(9, 16, "plain")
    z[5, 3] = torch.inf
    ids, w, off = _route(z, 2)
    assert torch.isnan(w[5]).all()
    loss, _, _ = _loss(z, off)
    assert torch.isnan(loss).all()


def _grad_case(T, E, k, H, kind, rs, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 17)
    z = _logits(T, E, kind, seed)
    ids, w, off = _route(z, k)
    y = torch.randn((T, k, H), generator=g, device="cuda") * w.unsqueeze(2)
    y[ids < 0] = torch.nan                      # rows of unfilled slots were never written
    dout = (torch.randn((T, H), generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    dout[(ids < 0).all(1)] = torch.nan          # nothing of a token without experts counts
    return z, ids, w, off, y, dout


def _exact_grad(z, ids, w, y, dout, rs, counts, d_loss):
    p, lse, some, ep = _exact_probs(z)
    T, E = p.shape
    out, tol = np.zeros((T, E)), np.zeros((T, E))
    if d_loss is not None:
        c = counts.cpu().numpy().astype(np.float64)
        n, P = max(c[-1], 1), max(c[:-1].sum(), 1)
        d0, d1 = (float(v) for v in d_loss)
        gg = d0 * E * c[:-1] / (P * n)
        zc = 2 * d1 / n
        inner = (p * gg).sum(1) - zc * lse
        el = U * (8 * np.abs(lse) + 8 * np.log(max(E, 2)) + E / 32 + 48)
        e_in = (ep * np.abs(gg)).sum(1) + _gamma(E / 32 + 12) * (p * np.abs(gg)).sum(1) + abs(zc) * el
        diff = gg - inner[:, None]
        out += p * diff
        tol += ep * np.abs(diff) + (p + ep) * (e_in[:, None] + 4 * U * np.abs(gg) + 4 * U * np.abs(inner)[:, None])
    if y is not None:
        i, ww = ids.cpu().numpy(), w.double().cpu().numpy()
        yy, dd = y.double().cpu().numpy(), dout.double().cpu().numpy()
        H = yy.shape[2]
        filled = (i >= 0) & (i < E)
        with np.errstate(invalid="ignore"):
            s = np.where(filled, rs * (yy * dd[:, None, :]).sum(2), 0.0)
            sa = np.where(filled, abs(rs) * np.abs(yy * dd[:, None, :]).sum(2), 0.0)
        es = _gamma(H / 256 + 66) * sa
        ww = np.where(filled, ww, 0.0)
        d = s - ww * s.sum(1, keepdims=True)
        e = es + ww * (es.sum(1, keepdims=True) + _gamma(8) * np.abs(s).sum(1, keepdims=True)) + 2 * U * (np.abs(s) + np.abs(d))
        t, j = np.nonzero(filled)
        np.add.at(out, (t, i[t, j]), d[t, j])
        np.add.at(tol, (t, i[t, j]), e[t, j])
    return out, tol + 2 * U * np.abs(out) + 1e-37


@pytest.mark.parametrize("T,E", [(4096, 256), (3001, 257), (300, 64), (70001, 8)])
def test_loss_again_on_a_stream_and_in_a_graph(T, E):
    """The same bits from one launch or two, on another stream beside other
    work, and from a captured graph with new logits."""
    z = _logits(T, E, "masked", seed=3)
    ids, w, off = _route(z, 2)
    want = [t.clone() for t in _loss(z, off)]
    other = _logits(T, E, "plain", seed=4)
    o_ids, o_w, o_off = _route(other, 2)
    o_want = [t.clone() for t in _loss(other, o_off)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s1):
        got = _loss(z, off)
    with torch.cuda.stream(s2):
        o_got = _loss(other, o_off)
    torch.cuda.synchronize()
    for p, q in zip((*got, *o_got), (*want, *o_want)):
        assert torch.equal(p, q)
    zz, zoff = z.clone(), off.clone()
    out = [torch.empty_like(t) for t in want]
    ws = torch.empty((fm.moe_balance_loss_workspace_bytes(T, E),), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fm.moe_balance_loss(zz, zoff, *out, ws)
    for src, src_off, ref in ((other, o_off, o_want), (z, off, want)):
        zz.copy_(src)
        zoff.copy_(src_off)
        graph.replay()
        for p, q in zip(out, ref):
            assert torch.equal(p, q)


GRADS = [(1, 5, 2, 128), (600, 12, 3, 1152), (450, 130, 9, 2048), (3, 8, 8, 256), (33, 64, 2, 640), (130, 65, 6, 128), (65, 256, 8, 1152), (21, 257, 9, 384),
         (7, 1024, 32, 256), (2, 40, 17, 16384)]


@pytest.mark.parametrize("kind", ["plain", "masked", "lowest"])
@pytest.mark.parametrize("T,E,k,H", GRADS)
def test_route_backward(T, E, k, H, kind):
    z, ids, w, off, y, dout = _grad_case(T, E, k, H, kind, 2.5, seed=T)
    _, counts, _ = _loss(z, off)
    # the z term of logits at the type's lowest value is beyond FP32
    d_loss = torch.tensor([0.7, 0.0 if kind == "lowest" else -0.3], device="cuda")
    for use_y, use_loss in ((True, True), (True, False), (False, True)):
        d = torch.full((T, E), -7.0, device="cuda")
        fm.moe_route_backward(z, ids if use_y else None, w if use_y else None, y if use_y else None,
                              dout if use_y else None, 2.5, counts if use_loss else None,
                              d_loss if use_loss else None, d)
        want, tol = _exact_grad(z, ids, w, y if use_y else None, dout, 2.5, counts, d_loss if use_loss else None)
        got = d.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol), (use_y, use_loss, np.nanmax(np.abs(got - want) / tol))
        off_limits = ~(z > -torch.inf).cpu().numpy()
        assert np.all(got[off_limits] == 0.0)


def test_shared_slot_and_foreign_ids_are_skipped():
    """Ids outside [0, E) (the shared expert's slot, unfilled ones) take no
    part, and an id that a token holds twice gets both parts."""
    T, E, k, H = 9, 16, 4, 256
    z, ids, w, off, y, dout = _grad_case(T, E, k, H, "plain", 1.0)
    ids[:, 3] = E
    ids[2, 1] = -1
    ids[3, 1] = 77
    ids[4, 1] = ids[4, 0]
    w[:, 3] = 1.0
    y[:, 3] = torch.nan
    d = torch.empty((T, E), device="cuda")
    fm.moe_route_backward(z, ids, w, y, dout, 1.0, None, None, d)
    want, tol = _exact_grad(z, ids, w, y, dout, 1.0, None, None)
    assert np.all(np.abs(d.double().cpu().numpy() - want) <= tol)


def test_gradient_against_differences():
    """Central differences of the 64-bit loss, the experts' outputs and the
    counts held fixed; step 1e-5, so the difference quotient is off by about
    1e-10 (third derivatives of order one) + 1e-16 / 1e-5."""
    T, E, k, H, rs = 5, 12, 3, 128, 1.5
    z, ids, w, off, y, dout = _grad_case(T, E, k, H, "plain", rs)
    _, counts, _ = _loss(z, off)
    d_loss = torch.tensor([2.0, 0.5], device="cuda")
    d = torch.empty((T, E), device="cuda")
    fm.moe_route_backward(z, ids, w, y, dout, rs, counts, d_loss, d)
    o = (y / w.unsqueeze(2)).double().cpu().numpy()
    dd, i = dout.double().cpu().numpy(), ids.cpu().numpy()
    c = counts.cpu().numpy().astype(np.float64)

    def total(zz):
        sel = np.take_along_axis(zz, i, 1)
        ww = np.exp(sel - sel.max(1, keepdims=True))
        ww /= ww.sum(1, keepdims=True)
        ex = np.exp(zz)
        p = ex / ex.sum(1, keepdims=True)
        lb = E * (c[:-1] / c[:-1].sum() * p.mean(0)).sum()
        lz = (np.log(ex.sum(1)) ** 2).mean()
        return rs * np.einsum("th,tkh,tk->", dd, o, ww) + 2.0 * lb + 0.5 * lz

    zz = z.double().cpu().numpy()
    got = d.double().cpu().numpy()
    scale = np.abs(got).max()
    for t in range(T):
        for e in range(E):
            hi, lo = zz.copy(), zz.copy()
            hi[t, e] += 1e-5
            lo[t, e] -= 1e-5
            assert abs((total(hi) - total(lo)) / 2e-5 - got[t, e]) <= 1e-5 * scale


def test_layer_methods_and_repeatability():
    """balance_loss and router_backward after RoutedMoE.forward: the separate
    calls' bits; the same bits on a second call, on another stream, and when
    replayed from a captured graph with new inputs."""
    wl = mi.WORKLOADS["tiny"].with_(T=50)
    d = mi.make_inputs(wl, 3, "cuda")
    layer = fm.RoutedMoE(d["w_gate"], d["s_gate"], d["w_up"], d["s_up"], d["w_down"], d["s_down"], wl.k, 2.0, 64)
    layer.forward(d["x"], d["logits"])
    dout = torch.randn((wl.T, wl.H), device="cuda").to(torch.bfloat16)
    d_loss = torch.tensor([0.01, 0.001], device="cuda")
    loss, counts = layer.balance_loss(d["logits"])
    grad = layer.router_backward(d["logits"], dout, d_loss).clone()
    l2, c2, _ = _loss(d["logits"], layer.offsets)
    g2 = torch.empty_like(grad)
    fm.moe_route_backward(d["logits"], layer.ids[:wl.T], layer.tw[:wl.T], layer.y[:wl.T], dout, 2.0, c2, d_loss, g2)
    assert torch.equal(loss, l2) and torch.equal(counts, c2) and torch.equal(grad, g2)
    want, tol = _exact_grad(d["logits"], layer.ids[:wl.T], layer.tw[:wl.T], layer.y[:wl.T], dout, 2.0, counts, d_loss)
    assert np.all(np.abs(grad.double().cpu().numpy() - want) <= tol)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g3 = torch.full_like(grad, -7.0)
    layer.balance_loss(d["logits"], stream=side)
    layer.router_backward(d["logits"], dout, d_loss, g3, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(g3, grad)

    graph = torch.cuda.CUDAGraph()
    lg = d["logits"].clone()
    with torch.cuda.graph(graph):
        layer.forward(d["x"], lg)
        layer.balance_loss(lg)
        layer.router_backward(lg, dout, d_loss, g3)
    for seed in (5, 6):
        lg.copy_(mi.make_logits(wl, seed, "cuda"))
        graph.replay()
        replayed = g3.clone()
        layer.forward(d["x"], lg)
        layer.balance_loss(lg)
        assert torch.equal(layer.router_backward(lg, dout, d_loss), replayed)
    assert layer.device_status() == 0


def test_binding_refusals():
    z = _logits(6, 8, "plain")
    ids, w, off = _route(z, 2)
    loss, counts, mean = _loss(z, off)
    y, dout = torch.zeros((6, 2, 128), device="cuda"), torch.zeros((6, 128), dtype=torch.bfloat16, device="cuda")
    d, dl = torch.empty_like(z), torch.ones((2,), device="cuda")
    ws = torch.empty((1 << 16,), dtype=torch.uint8, device="cuda")

    def refused(code, fn, *a):
        with pytest.raises(fm.MoeError) as e:
            fn(*a)
        assert e.value.code == code

    refused(1, fm.moe_balance_loss, z.double(), off, loss, counts, mean, ws)
    refused(1, fm.moe_balance_loss, z.t(), off, loss, counts, mean, ws)
    refused(1, fm.moe_balance_loss, z, off.long(), loss, counts, mean, ws)
    refused(1, fm.moe_balance_loss, z, off, loss, counts[:8], mean, ws)
    refused(1, fm.moe_balance_loss, z, off, loss.cpu(), counts, mean, ws)
    refused(4, fm.moe_balance_loss, z, off, loss, counts, mean, ws[:16])
    refused(1, fm.moe_route_backward, z, ids, w, None, None, 1.0, None, None, d)
    refused(1, fm.moe_route_backward, z, ids, w, y, dout.float(), 1.0, None, None, d)
    refused(1, fm.moe_route_backward, z, ids.long(), w, y, dout, 1.0, None, None, d)
    refused(1, fm.moe_route_backward, z, ids, w, y[:5], dout, 1.0, None, None, d)
    refused(1, fm.moe_route_backward, z, ids, w, y, dout, 1.0, counts[:8], dl, d)
    refused(1, fm.moe_route_backward, z, ids, w, y, dout, 1.0, counts, dl, d[:, :7])
