"""moe_lora and moe_lora_backward against the definitions in 64 bits.

Tolerances (u = 2^-24).  The BF16 products are exact; a sum of C of them on
the tensor core is taken in groups of 16 whose additions are only assumed
faithful (2u each), so in any order of the groups its error is at most
gamma(C / 16 + 64; 2u) times the sum of the absolute products (64: the
additions inside a group, the joins of warps and blocks, and a scale).
v and dv enter the second product as three BF16 terms whose sum is v to
within u |v|; that product has 3 C / 16 groups.  A BF16 output adds half of
a BF16 step, 2^-8 relative.
"""
import numpy as np
import pytest
import torch

import fp8_blockwise_routed_b200 as fm
import moe_inputs as mi
from fp8_blockwise_routed_b200.adapters import LoraAdapters, LoraBatch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _g(c):
    m = (c / 16 + 64) * 2 * U
    return m / (1 - m)


def _ids(T, n, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "mixed":                       # tokens of any adapter, some without one
        return rng.integers(-1, n, T)
    if kind == "own":                         # every token its own adapter
        return np.arange(T) % n
    if kind == "one":                         # all tokens on the last adapter
        return np.full(T, n - 1)
    if kind == "none":
        return np.full(T, -1)
    cuts = np.sort(rng.integers(0, T + 1, 6))  # contiguous requests, some of length zero
    return (np.searchsorted(cuts, np.arange(T), side="right") * 3) % (n + 1) - 1


def _case(T, K, N, R, n, kind, seed=0, scales=True):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)

    def rnd(shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    ids = torch.from_numpy(_ids(T, n, kind, seed).astype(np.int32)).cuda()
    c = dict(T=T, K=K, N=N, R=R, n=n, ids=ids, x=rnd((T, K)).to(torch.bfloat16),
             a=rnd((n, R, K), K ** -0.5).to(torch.bfloat16), b=rnd((n, R, N), R ** -0.5).to(torch.bfloat16),
             scales=rnd((n,)) if scales else None, base=rnd((T, N)), dout=rnd((T, N), 0.1).to(torch.bfloat16),
             dx_base=rnd((T, K)))
    c["batch"] = LoraBatch(n, T).assign(ids)
    return c


def _forward(c, base="base", bf16=False, fill=-7.0):
    v = torch.full((c["T"], c["R"]), fill, device="cuda")
    out = torch.full((c["T"], c["N"]), fill, device="cuda")
    o16 = torch.full((c["T"], c["N"]), fill, device="cuda", dtype=torch.bfloat16) if bf16 else None
    b = None if base is None else c[base]
    fm.moe_lora(c["x"], c["a"], c["b"], c["scales"], c["batch"].offsets, c["batch"].sorted, b, v, out, o16)
    return v, out, o16


def _exact_forward(c, base):
    """v by token, out and their error bounds, in 64 bits."""
    x, a, b = c["x"].double(), c["a"].double(), c["b"].double()
    T, N, R, K = c["T"], c["N"], c["R"], c["K"]
    out = torch.zeros((T, N), dtype=torch.float64, device="cuda") if base is None else base.double().clone()
    e_out, v, e_v = torch.zeros_like(out), out.new_zeros((T, R)), out.new_zeros((T, R))
    for i in range(c["n"]):
        t = torch.nonzero(c["ids"] == i)[:, 0]
        if not t.numel():
            continue
        f = 1.0 if c["scales"] is None else float(c["scales"][i])
        v[t] = x[t] @ a[i].T
        e_v[t] = _g(K) * (x[t].abs() @ a[i].T.abs())
        d = f * (v[t] @ b[i])
        e = abs(f) * (e_v[t] @ b[i].abs() + (_g(3 * R) + 2 * U) * ((v[t].abs() + e_v[t]) @ b[i].abs()))
        out[t] += d
        e_out[t] = e + U * (out[t].abs() + e + d.abs())
    return v, e_v, out, e_out


def _close(got, want, tol, what):
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), (what, float((err / tol.clamp_min(1e-300)).max()))


def _check_forward(c, v, out, o16, base, fill=-7.0):
    ve, e_v, oe, e_o = _exact_forward(c, base)
    has = c["ids"] >= 0
    P = int(has.sum())
    tok = c["batch"].sorted[:P].long()
    _close(v[:P], ve[tok], e_v[tok] + 1e-37, "v")
    assert bool((v[P:] == fill).all())
    _close(out[has], oe[has], e_o[has] + 1e-37, "out")
    assert bool((out[~has] == fill).all())
    if o16 is not None:
        assert torch.equal(o16[has], out[has].to(torch.bfloat16))
        assert bool((o16[~has] == fill).all())


SHAPES = [(1, 8, 8, 1, 1, "one"), (1, 5120, 640, 16, 8, "one"), (5, 24, 40, 3, 2, "mixed"),
          (70, 264, 520, 13, 5, "mixed"), (129, 1024, 72, 33, 7, "requests"), (300, 136, 1000, 100, 3, "one"),
          (64, 512, 512, 64, 64, "own"), (17, 5120, 264, 128, 4, "mixed"), (513, 328, 320, 17, 1024, "mixed"),
          (1030, 256, 248, 32, 3, "requests"), (2100, 1536, 1096, 64, 2, "requests"), (40, 64, 64, 8, 4, "none"),
          (700, 2048, 136, 48, 2, "mixed"), (333, 200, 2056, 24, 300, "own"), (16, 16384, 16384, 8, 3, "mixed"),
          # rows enough for the wide kernel of ranks above 32, in each direction
          (4100, 136, 4104, 64, 3, "requests"), (4111, 4120, 136, 100, 2, "mixed"), (4200, 72, 4096, 33, 4, "own"),
          # every size of cluster of the few-token kernel, one adapter or many
          (2, 5120, 72, 64, 1024, "own"), (40, 2048, 2048, 16, 2, "mixed"), (200, 1024, 1024, 40, 64, "mixed"),
          (1000, 256, 256, 8, 500, "own"), (255, 8, 8, 4, 3, "mixed"), (256, 8, 8, 4, 3, "mixed"),
          # uneven adapters over many column blocks
          (1500, 2048, 1536, 16, 17, "requests"), (900, 640, 640, 8, 56, "mixed"),
          # ranks that are no multiple of four, or above 64, behind the tiled first product
          (900, 264, 520, 13, 5, "mixed"), (600, 264, 520, 100, 2, "requests"), (520, 72, 2056, 127, 1, "one"),
          (385, 512, 512, 64, 48, "mixed"), (513, 512, 512, 32, 21, "mixed")]


@pytest.mark.parametrize("T,K,N,R,n,kind", SHAPES)
def test_lora(T, K, N, R, n, kind):
    c = _case(T, K, N, R, n, kind, seed=T + R)
    _check_forward(c, *_forward(c, "base", bf16=True), c["base"])
    v, out, _ = _forward(c, None)
    _check_forward(c, v, out, None, None)


def _backward(c, v, dx_base="dx_base", dx=True, fill=-7.0):
    d_a = torch.full(c["a"].shape, fill, device="cuda")
    d_b = torch.full(c["b"].shape, fill, device="cuda")
    gx = torch.full((c["T"], c["K"]), fill, device="cuda") if dx else None
    ws = torch.full((fm.moe_lora_backward_workspace_bytes(c["T"], c["R"]),), 255, dtype=torch.uint8, device="cuda")
    fm.moe_lora_backward(c["x"], c["a"], c["b"], c["scales"], c["batch"].offsets, c["batch"].sorted, v, c["dout"],
                         None if dx_base is None else c[dx_base], gx, d_a, d_b, ws)
    return gx, d_a, d_b


def _check_backward(c, v, gx, d_a, d_b, dx_base, fill=-7.0):
    x, a, b, dout = c["x"].double(), c["a"].double(), c["b"].double(), c["dout"].double()
    off, tok = c["batch"].offsets.tolist(), c["batch"].sorted.long()
    for i in range(c["n"]):
        t = tok[off[i]:off[i + 1]]
        f = 1.0 if c["scales"] is None else float(c["scales"][i])
        vi = v[off[i]:off[i + 1]].double()
        dv = f * (dout[t] @ b[i].T)
        e_dv = (_g(c["N"]) + U) * abs(f) * (dout[t].abs() @ b[i].T.abs())
        if gx is not None and len(t):
            want = dv @ a[i] + (0.0 if dx_base is None else dx_base[t].double())
            e = e_dv @ a[i].abs() + (_g(3 * c["R"]) + 2 * U) * ((dv.abs() + e_dv) @ a[i].abs())
            _close(gx[t], want, e + U * (want.abs() + e) + 1e-37, "dx")
        steps = 3 * len(t)
        want = dv.T @ x[t]
        e = e_dv.T @ x[t].abs() + (_g(steps) + 2 * U) * ((dv.abs() + e_dv).T @ x[t].abs())
        _close(d_a[i], want, e + U * want.abs() + 1e-37, "d_a")
        want = f * (vi.T @ dout[t])
        e = (_g(steps) + 2 * U) * abs(f) * (vi.abs().T @ dout[t].abs())
        _close(d_b[i], want, e + U * want.abs() + 1e-37, "d_b")
    if gx is not None:
        assert bool((gx[c["ids"] < 0] == fill).all())


@pytest.mark.parametrize("T,K,N,R,n,kind", SHAPES)
def test_lora_backward(T, K, N, R, n, kind):
    c = _case(T, K, N, R, n, kind, seed=T + R)
    v, _, _ = _forward(c)
    _check_backward(c, v, *_backward(c, v), c["dx_base"])
    _check_backward(c, v, *_backward(c, v, None), None)
    gx, d_a, d_b = _backward(c, v, None, dx=False)
    _check_backward(c, v, None, d_a, d_b, None)


def test_no_tokens():
    c = _case(0, 64, 32, 8, 3, "none")
    _forward(c)
    gx, d_a, d_b = _backward(c, torch.empty((0, 8), device="cuda"))
    assert not d_a.any() and not d_b.any()


def test_no_scales_is_one():
    c = _case(50, 128, 64, 8, 3, "mixed", scales=False)
    v, out, _ = _forward(c)
    gx = _backward(c, v)
    c["scales"] = torch.ones((3,), device="cuda")
    v1, out1, _ = _forward(c)
    assert torch.equal(out, out1)
    for p, q in zip(gx, _backward(c, v)):
        assert torch.equal(p, q)


def test_linear_in_each_adapter_entry():
    """Differences: out is linear in one entry of lora_b and of lora_a, so
    <dout, out> at two values of an entry gives its gradient exactly in 64 bits;
    the tolerance is the kernels' own."""
    c = _case(37, 64, 48, 5, 3, "mixed", seed=4)
    v, _, _ = _forward(c)
    gx, d_a, d_b = _backward(c, v, None)
    _, _, o0, _ = _exact_forward(c, None)
    dout = c["dout"].double()
    base_loss = (dout * o0).sum()
    for name, grad, at in (("a", d_a, (1, 2, 30)), ("a", d_a, (2, 4, 63)), ("b", d_b, (0, 0, 0)), ("b", d_b, (1, 3, 47))):
        w = c[name].clone()
        c2 = dict(c)
        c2[name] = w
        w[at] = w[at] + 1.0
        step = float(w[at].double() - c[name][at].double())
        _, _, o1, _ = _exact_forward(c2, None)
        want = float(((dout * o1).sum() - base_loss) / step)
        assert abs(want - float(grad[at])) <= 1e-5 * float(grad.abs().max())
    # and in x, one token
    t, k = int(torch.nonzero(c["ids"] >= 0)[0]), 11
    x = c["x"].clone()
    x[t, k] += 1.0
    step = float(x[t, k].double() - c["x"][t, k].double())
    _, _, o1, _ = _exact_forward(dict(c, x=x), None)
    assert abs(float(((dout * o1).sum() - base_loss) / step) - float(gx[t, k])) <= 1e-5 * float(gx.abs().max())


def test_in_place_and_strided_rows():
    """base = out, rows inside wider buffers (a slot of y, a slice of x): the
    bits of the contiguous call, and nothing else of the buffers touched."""
    c = _case(201, 256, 136, 20, 4, "requests", seed=9)
    v, out, o16 = _forward(c, bf16=True)
    has = c["ids"] >= 0
    y = torch.full((201, 3, 136), -7.0, device="cuda")
    y[:, 2] = c["base"]
    xw = torch.full((201, 256 + 64), 9.0, device="cuda", dtype=torch.bfloat16)
    xw[:, 8:264] = c["x"]
    v2 = torch.empty_like(v)
    fm.moe_lora(xw[:, 8:264], c["a"], c["b"], c["scales"], c["batch"].offsets, c["batch"].sorted, y[:, 2], v2,
                y[:, 2])
    P = int(has.sum())
    assert torch.equal(v2[:P], v[:P])
    assert torch.equal(y[has, 2], out[has]) and torch.equal(y[~has, 2], c["base"][~has])
    assert bool((y[:, :2] == -7.0).all())
    gx, d_a, d_b = _backward(c, v)
    dw = torch.full((201, 5, 136), 9.0, device="cuda", dtype=torch.bfloat16)
    dw[:, 4] = c["dout"]
    gw = torch.full((201, 264), -7.0, device="cuda")
    gw[:, :256] = c["dx_base"]
    d_a2, d_b2 = torch.empty_like(d_a), torch.empty_like(d_b)
    ws = torch.empty((fm.moe_lora_backward_workspace_bytes(201, 20),), dtype=torch.uint8, device="cuda")
    fm.moe_lora_backward(xw[:, 8:264], c["a"], c["b"], c["scales"], c["batch"].offsets, c["batch"].sorted, v,
                         dw[:, 4], gw[:, :256], gw[:, :256], d_a2, d_b2, ws)
    assert torch.equal(d_a, d_a2) and torch.equal(d_b, d_b2)
    assert torch.equal(gw[has, :256], gx[has]) and torch.equal(gw[~has, :256], c["dx_base"][~has])
    assert bool((gw[:, 256:] == -7.0).all())


def test_other_rows_do_not_matter():
    """NaN and Inf in the rows of one request, and in tokens without an
    adapter, stay there; the other rows keep their bits.  An Inf in v is
    carried as an Inf."""
    c = _case(90, 128, 96, 16, 3, "mixed", seed=2)
    v, out, _ = _forward(c)
    gx, d_a, d_b = _backward(c, v)
    bad = (c["ids"] == 1) | (c["ids"] < 0)
    c2 = dict(c, x=c["x"].clone(), dout=c["dout"].clone())
    c2["x"][bad] = torch.nan
    c2["dout"][bad] = torch.inf
    v2, out2, _ = _forward(c2)
    gx2, d_a2, d_b2 = _backward(c2, v2)
    ok = ~bad
    assert torch.equal(out[ok], out2[ok]) and torch.equal(gx[ok], gx2[ok])
    for i in (0, 2):
        assert torch.equal(d_a[i], d_a2[i]) and torch.equal(d_b[i], d_b2[i])
    assert torch.isnan(out2[c["ids"] == 1]).all()
    one = _case(3, 8, 16, 1, 1, "one")
    one["x"][1, 0] = torch.inf
    one["x"][1, 1:] = 0
    _, o, _ = _forward(one)
    want = one["base"] + one["scales"] * (one["x"].float() @ one["a"][0].float().T) @ one["b"][0].float()
    assert torch.equal(torch.isinf(o), torch.isinf(want)) and torch.equal(torch.sign(o[1]), torch.sign(want[1]))


def test_entries_outside_the_batch_are_skipped():
    c = _case(60, 64, 64, 8, 3, "mixed", seed=3)
    tok = c["batch"].sorted.clone()
    P = int((c["ids"] >= 0).sum())
    lost = tok[[1, P - 1]].long()
    tok[1], tok[P - 1] = -5, 60
    v, out, _ = _forward(c)
    v2, out2 = torch.zeros_like(v), torch.full_like(out, -7.0)
    fm.moe_lora(c["x"], c["a"], c["b"], c["scales"], c["batch"].offsets, tok, c["base"], v2, out2)
    keep = torch.ones((60,), dtype=torch.bool, device="cuda")
    keep[lost] = False
    assert torch.equal(out2[keep], out[keep]) and bool((out2[lost] == -7.0).all())


@pytest.mark.parametrize("T", [333, 1333])
def test_repeatable_streams_graph(T):
    """Another batch in the same buffers, replayed from a graph and run on another
    stream: the same bits, and right."""
    c = _case(T, 520, 264, 24, 6, "requests", seed=8)
    ad = LoraAdapters(c["a"], c["b"], c["scales"], 1400)
    batch = LoraBatch(6, 1400)
    out, gx = c["base"].clone(), torch.zeros((T, 520), device="cuda")
    graph = torch.cuda.CUDAGraph()
    ids, x = c["ids"].clone(), c["x"].clone()
    ad.backward(batch.assign(ids), x, c["dout"], None, gx)   # buffers exist before the capture
    with torch.cuda.graph(graph):
        batch.assign(ids)
        ad.forward(batch, x, c["base"], out)
        g_a, g_b = ad.backward(batch, x, c["dout"], None, gx)
    for seed in (1, 2):
        ids.copy_(torch.from_numpy(_ids(T, 6, "mixed", seed).astype(np.int32)))
        x.copy_(torch.randn((T, 520), device="cuda"))
        out.copy_(c["base"])
        gx.zero_()
        graph.replay()
        got = [t.clone() for t in (out, gx, g_a, g_b)]
        out.copy_(c["base"])
        gx.zero_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        batch.assign(ids, stream=side)
        ad.forward(batch, x, c["base"], out, stream=side)
        ad.backward(batch, x, c["dout"], None, gx, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for p, q in zip(got, (out, gx, g_a, g_b)):
            assert torch.equal(p, q)
        c2 = dict(c, ids=ids, x=x, batch=batch)
        has = ids >= 0
        _, _, want, tol = _exact_forward(c2, c["base"])
        _close(out[has], want[has], tol[has] + 1e-37, "out")


@pytest.mark.parametrize("T,n", [(61, 7), (500, 3), (900, 3)])
def test_two_calls_at_once(T, n):
    """Two batches on two streams side by side, each with buffers of its own,
    give the bits of one after the other."""
    cs = [_case(T, 1024, 512, 24, n, "mixed", seed=s) for s in (1, 2)]
    want = []
    for c in cs:
        v, out, _ = _forward(c)
        want.append((v, out, *_backward(c, v)))
    streams = [torch.cuda.Stream() for _ in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(3):
        for i, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                v, out, _ = _forward(c)
                got[i] = (v, out, *_backward(c, v))
    torch.cuda.synchronize()
    for i in range(2):
        for p, q in zip(got[i], want[i]):
            assert torch.equal(p, q)


def test_first_use_inside_a_capture():
    """A graph may capture the first call of a shape: nothing in a call
    allocates, synchronises or runs on another stream."""
    c = _case(4500, 72, 4096, 72, 2, "requests", seed=12)
    v, out = torch.zeros((4500, 72), device="cuda"), c["base"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fm.moe_lora(c["x"], c["a"], c["b"], c["scales"], c["batch"].offsets, c["batch"].sorted, c["base"], v, out)
    graph.replay()
    has = c["ids"] >= 0
    _, _, want, tol = _exact_forward(c, c["base"])
    _close(out[has], want[has], tol[has] + 1e-37, "out")


def test_binding_refusals():
    c = _case(20, 64, 32, 4, 2, "mixed")
    v, out = torch.empty((20, 4), device="cuda"), torch.empty((20, 32), device="cuda")
    b = c["batch"]
    good = dict(x=c["x"], lora_a=c["a"], lora_b=c["b"], scales=c["scales"], adapter_offsets=b.offsets,
                sorted_tokens=b.sorted, base=c["base"], v=v, out=out)
    for name, bad in (("x", c["x"].float()), ("x", c["x"].t()), ("out", out[:1].expand(20, 32)), ("lora_a", c["a"][:, :3]), ("lora_b", c["b"].float()),
                      ("scales", c["scales"].double()), ("adapter_offsets", b.offsets[:2]),
                      ("sorted_tokens", b.sorted.long()), ("base", c["base"][:, :31]), ("v", v[:19]),
                      ("out", out.cpu()), ("out_bf16", out)):
        with pytest.raises(fm.MoeError) as e:
            fm.moe_lora(**dict(good, **{name: bad}))
        assert e.value.code == 1 and name in str(e.value)
    for name in ("lora_a", "adapter_offsets", "sorted_tokens", "v", "out"):
        with pytest.raises(fm.MoeError) as e:
            fm.moe_lora(**dict(good, **{name: None}))
        assert e.value.code == 1 and f"{name} is missing" in str(e.value)
    with pytest.raises(fm.MoeError) as e:   # rows that start off a 16-byte boundary
        fm.moe_lora(**dict(good, base=torch.zeros((20, 33), device="cuda")[:, 1:]))
    assert e.value.code in (1, 3)
    d_a, d_b = torch.empty((2, 4, 64), device="cuda"), torch.empty((2, 4, 32), device="cuda")
    with pytest.raises(fm.MoeError) as e:
        fm.moe_lora_backward(c["x"], c["a"], c["b"], None, b.offsets, b.sorted, v, c["dout"], None, None, d_a, d_b,
                             torch.empty((16,), dtype=torch.uint8, device="cuda"))
    assert e.value.code == 4


def test_infinite_rows_stay_infinite():
    """An infinite x gives infinite or NaN elements where the formula does, in
    its own row only, on the few-token and the tiled paths."""
    for T, R in ((20, 8), (900, 64)):
        c = _case(T, 64, 32, R, 2, "mixed")
        c["x"][3, 5] = float("inf")
        v, out = torch.empty((T, R), device="cuda"), c["base"].clone()
        b = c["batch"]
        fm.moe_lora(c["x"], c["a"], c["b"], c["scales"], b.offsets, b.sorted, c["base"], v, out)
        clean = c["x"].clone()
        clean[3] = 0
        v2, out2 = torch.empty((T, R), device="cuda"), c["base"].clone()
        fm.moe_lora(clean, c["a"], c["b"], c["scales"], b.offsets, b.sorted, c["base"], v2, out2)
        rest = torch.arange(T, device="cuda") != 3
        assert torch.equal(out[rest], out2[rest])
        a = int(c["ids"][3])
        if a >= 0:
            want = (c["x"][3].double() @ c["a"][a].double().t()) @ c["b"][a].double() * float(
                1 if c["scales"] is None else c["scales"][a]) + c["base"][3].double()
            assert not want.isfinite().any()
            assert torch.equal(out[3].isnan(), want.isnan()) and torch.equal(out[3].isposinf(), want.isposinf())


@pytest.mark.parametrize("mx", [False, True])
def test_adapted_layer_as_used(mx):
    """A fine-tuning step of one layer with frozen FP8 experts: forward with
    adapters, router losses, router gradient, adapter gradients; against the
    layer without adapters and the definitions."""
    wl = mi.WORKLOADS["tiny"].with_(T=61)
    d = mi.make_inputs_mx(wl, 1, "cuda") if mx else mi.make_inputs(wl, 1, "cuda")
    cls = fm.RoutedMoEMX if mx else fm.RoutedMoE
    layer = cls(d["w_gate"], d["s_gate"], d["w_up"], d["s_up"], d["w_down"], d["s_down"], wl.k, 1.5, 64)
    c = _case(wl.T, wl.H, wl.H, 12, 4, "requests", seed=6)
    c["x"] = d["x"]
    ad, batch = LoraAdapters(c["a"], c["b"], c["scales"], 64), LoraBatch(4, 64).assign(c["ids"])
    o16 = torch.empty((wl.T, wl.H), dtype=torch.bfloat16, device="cuda")
    plain = layer.forward(d["x"], d["logits"], out_bf16=o16).clone()
    plain16 = o16.clone()
    out = layer.forward(d["x"], d["logits"], out_bf16=o16, adapters=ad, batch=batch)
    has = c["ids"] >= 0
    _, _, want, tol = _exact_forward(c, plain)
    _close(out[has], want[has], tol[has] + 1e-37, "out")
    assert torch.equal(out[~has], plain[~has]) and torch.equal(o16[~has], plain16[~has])
    assert torch.equal(o16, out.to(torch.bfloat16))
    loss, counts = layer.balance_loss(d["logits"])
    d_logits = layer.router_backward(d["logits"], c["dout"], torch.tensor([0.1, 0.01], device="cuda"))
    gx = torch.full((wl.T, wl.H), -7.0, device="cuda")
    d_a, d_b = ad.backward(batch, d["x"], c["dout"], None, gx)
    _check_backward(c, ad.v, gx, d_a, d_b, None)
    assert int(counts[:-1].sum()) == wl.T * wl.k and int(counts[-1]) == wl.T
    assert torch.isfinite(d_logits).all() and torch.isfinite(loss).all()
    assert layer.device_status() == 0


def test_adapters_on_the_shared_slot():
    """Adapters beside the shared expert: its slot of y, [T, k+1, H], takes the
    adapters' rows in place before the combine."""
    wl = mi.WORKLOADS["tiny"].with_(T=40)
    d = mi.make_inputs(wl, 2, "cuda")
    T, H, E, k = wl.T, wl.H, wl.E, wl.k
    c = _case(T, H, H, 9, 3, "mixed", seed=5)
    c["x"] = d["x"]
    ids = torch.empty((T, k + 1), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k + 1), device="cuda")
    off = torch.empty((E + 1,), dtype=torch.int32, device="cuda")
    sp = torch.empty((T * (k + 1),), dtype=torch.int32, device="cuda")
    ws = torch.empty((fm.moe_route_workspace_bytes(T, E, k + 1),), dtype=torch.uint8, device="cuda")
    fm.moe_route_shared(d["logits"], k, ids, w, off, sp, ws)
    y = torch.zeros((T, k + 1, H), device="cuda")
    y[:, k] = c["base"][:, :H]
    slot = y[:, k]
    fm.moe_lora(d["x"], c["a"], c["b"], c["scales"], c["batch"].offsets, c["batch"].sorted, slot,
                torch.empty((T, 9), device="cuda"), slot)
    out = torch.empty((T, H), device="cuda")
    wsc = torch.empty((fm.moe_combine_workspace_bytes(),), dtype=torch.uint8, device="cuda")
    fm.moe_combine_shared(y, ids, E, 2.0, out, None, wsc)
    _, _, want, tol = _exact_forward(c, c["base"])
    _close(out, want, tol + U * want.abs() + 1e-37, "out")
