"""Timed cases of the operators that adapt a routed layer whose experts stay
frozen in FP8: the router's balance loss with per-expert counts, the gradient
of the routing, and low-rank adapters of many requests with their gradients.

``run`` computes an operator in elementary torch operations, or, with ``own``
set, by the framework's calls.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest routed layer of the workload list: launch latency
        dict(name="balance_tiny", op="balance", T=64, E=8, k=2, masked=0.0, empty=0.0),
        # one prefill-sized micro-batch of the GLM-class router
        dict(name="balance_glm", op="balance", T=4096, E=256, k=8, masked=0.0, empty=0.02),
        # a whole optimizer step's tokens at once (logits larger than L2)
        dict(name="balance_step", op="balance", T=131072, E=256, k=8, masked=0.2, empty=0.01),
        # router gradient of the small workload's layer
        dict(name="route_grad_small", op="route", T=1024, H=2048, E=64, k=8, rs=2.5, masked=0.0, empty=0.0),
        # router gradient of the GLM-class layer: 671 MB of slot rows
        dict(name="route_grad_glm", op="route", T=4096, H=5120, E=256, k=8, rs=1.0, masked=0.0, empty=0.0),
        # a padded, partly masked batch: unfilled slots and tokens with no expert
        dict(name="route_grad_masked", op="route", T=777, H=640, E=160, k=6, rs=1.8, masked=0.96, empty=0.05),
        # one decoded token of one request
        dict(name="lora_token", op="lora", T=1, K=5120, N=5120, R=16, n=8, requests=1, bf16=False),
        # a decode batch: one token of each of 64 requests over 48 adapters
        dict(name="lora_decode", op="lora", T=64, K=5120, N=5120, R=64, n=48, requests=64, bf16=True),
        # a mixed prefill batch beside the shared expert's up projection
        dict(name="lora_prefill", op="lora", T=4096, K=5120, N=1536, R=32, n=32, requests=57, bf16=False),
        # the long prefill: few long prompts, H -> H
        dict(name="lora_long", op="lora", T=16384, K=6144, N=6144, R=64, n=8, requests=13, bf16=False),
        # adapter gradients of a small fine-tuning batch of odd sizes
        dict(name="lora_grad_small", op="lora_grad", T=1021, K=2048, N=512, R=8, n=5, requests=9),
        # adapter gradients of the GLM-class layer, H -> H
        dict(name="lora_grad_glm", op="lora_grad", T=4096, K=5120, N=5120, R=64, n=16, requests=24),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("balance", "route", "lora", "lora_grad"))
    if op == "balance":
        E = _log(rng, 4, 1024)
        T = _log(rng, 1, min(131072, 131072 * 256 // E))
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 10)), masked=rng.choice((0.0, 0.2, 0.9)),
                    empty=rng.choice((0.0, 0.05)))
    if op == "route":
        H, k = 128 * rng.randint(2, 48), rng.randint(1, 9)
        T = _log(rng, 1, min(8192, 4096 * 8 * 5120 // (H * k)))
        return dict(op=op, T=T, H=H, E=rng.randint(max(k, 8), 384), k=k, rs=rng.choice((1.0, 2.5)),
                    masked=rng.choice((0.0, 0.3, 0.95)), empty=rng.choice((0.0, 0.05)))
    K, N = 128 * rng.randint(2, 48), 128 * rng.randint(2, 48)
    R, n = rng.choice((4, 8, 13, 16, 24, 32, 48, 64)), _log(rng, 1, 64)
    if op == "lora":
        T = _log(rng, 1, 8192)
        requests = T if T <= 128 and rng.random() < 0.7 else rng.randint(1, max(1, min(T, 64)))
        return dict(op=op, T=T, K=K, N=N, R=R, n=n, requests=requests, bf16=rng.random() < 0.5)
    T = _log(rng, 16, 4096)
    return dict(op=op, T=T, K=min(K, 5120), N=min(N, 5120), R=R, n=min(n, 16), requests=rng.randint(1, min(T, 32)))


# ------------------------------------------------------------------ inputs

def _router_inputs(case, g):
    """Logits with some experts masked per token and some tokens masked
    whole, and the routing that the framework's router gives for them."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn((T, E), generator=g, device="cuda")
    logits += 1.5 * torch.randn((1, E), generator=g, device="cuda")  # popular and unpopular experts
    if case["masked"]:
        logits[torch.rand((T, E), generator=g, device="cuda") < case["masked"]] = -math.inf
    if case["empty"]:
        logits[torch.rand((T,), generator=g, device="cuda") < case["empty"]] = -math.inf
    top, ids = torch.topk(logits, k, dim=1)
    filled = top > -math.inf
    ex = torch.where(filled, torch.exp(top - top[:, :1]), 0.0)
    w = torch.where(filled, ex / ex.sum(1, keepdim=True), 0.0)
    ids = torch.where(filled, ids, -1).to(torch.int32)
    counts = torch.bincount(ids[filled].long(), minlength=E)
    offsets = torch.zeros((E + 1,), dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    tokens = (logits > -math.inf).any(1).sum().reshape(1)
    return logits, ids, w, offsets, torch.cat([counts, tokens]).to(torch.int32)


def _requests(case, g):
    """Adapter of each token: requests of uneven lengths, one adapter each,
    about one in twelve without."""
    T, n, requests = case["T"], case["n"], case["requests"]
    pick = torch.randint(0, n, (requests,), generator=g, device="cuda")
    pick[torch.rand((requests,), generator=g, device="cuda") < 1 / 12] = -1
    if requests <= 3:
        pick.clamp_(min=0)
    if requests == T:
        ids = pick
    else:
        cuts = torch.randperm(T - 1, generator=g, device="cuda")[:requests - 1].sort().values + 1
        ids = pick[torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)]
    # the permutation of the tokens by adapter (one per batch, kept for every
    # projection that the batch passes), as the framework's moe_permute gives
    # it for [T, 1] ids
    order = torch.sort(torch.where(ids < 0, n, ids), stable=True).indices
    counts = torch.bincount(ids[ids >= 0], minlength=n)
    offsets = torch.zeros((n + 1,), dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    P = int(offsets[-1])
    tokens = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    tokens[:P] = order[:P].to(torch.int32)
    return offsets, tokens, P, int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    s = {"op": op}
    if op in ("balance", "route"):
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"], s["ids"], s["w"], s["offsets"], s["counts"] = _router_inputs(case, g)
        if op == "balance":
            s["loss"] = torch.empty((2,), device="cuda")
            s["counts"] = torch.empty((E + 1,), dtype=torch.int32, device="cuda")
            s["prob_mean"] = torch.empty((E,), device="cuda")
            # scratch of the call: its size does not depend on the inputs
            s["ws"] = torch.zeros((1 << 22,), dtype=torch.uint8, device="cuda")
            return s
        H = case["H"]
        # slot rows as the experts leave them: routing weight times an expert
        # output; rows of unfilled slots were never written
        y = normal((T, k, H))
        y *= s["w"].unsqueeze(2)
        y[s["ids"] < 0] = math.nan
        s["y"], s["rs"] = y, case["rs"]
        s["dout"] = normal((T, H), 0.02, torch.bfloat16)
        s["d_loss"] = torch.tensor([0.01, 0.001], device="cuda")
        s["d_logits"] = torch.empty((T, E), device="cuda")
        return s
    T, K, N, R, n = (case[c] for c in ("T", "K", "N", "R", "n"))
    s["offsets"], s["tokens"], s["P"], s["most"] = _requests(case, g)
    s["x"] = normal((T, K), 1.0, torch.bfloat16)
    s["a"] = normal((n, R, K), K ** -0.5, torch.bfloat16)
    s["b"] = normal((n, R, N), R ** -0.5, torch.bfloat16)
    s["scales"] = 0.25 + 2 * torch.rand((n,), generator=g, device="cuda")
    if op == "lora":
        s["base"] = normal((T, N))
        s["out"] = s["base"].clone()
        s["out_bf16"] = s["base"].to(torch.bfloat16) if case["bf16"] else None
        s["v"] = torch.zeros((T, R), device="cuda")
        return s
    s["dout"] = normal((T, N), 0.02, torch.bfloat16)
    s["v"] = torch.zeros((T, R), device="cuda")
    at, tok = _placed(s)
    s["v"][:s["P"]] = _rows(s["x"].double(), at, tok, s).bmm(s["a"].double().mT).flatten(0, 1)[at].float()
    s["dx_base"] = normal((T, K), 0.02)
    s["dx"] = s["dx_base"].clone()
    s["d_a"] = torch.empty((n, R, K), device="cuda")
    s["d_b"] = torch.empty((n, R, N), device="cuda")
    s["ws"] = torch.zeros(((1 << 20) + 16 * T * R,), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------- plain forms

def _balance(logits, offsets):
    E = logits.shape[1]
    ok = logits > -math.inf
    some = ok.any(1)
    top = torch.where(some, logits.amax(1), 0.0)
    ex = torch.exp(logits - top[:, None])  # 0 at the masked experts
    total = torch.where(some, ex.sum(1), 1.0)
    probs = ex / total[:, None]
    lse = torch.where(some, top + torch.log(total), 0.0)
    tokens = some.sum()
    each = (offsets[1:] - offsets[:-1])
    mean = probs.sum(0, dtype=torch.float64) / tokens.clamp(min=1)
    share = each.double() / offsets[-1].clamp(min=1)
    loss = torch.stack([E * (share * mean).sum(), lse.double().square().sum() / tokens.clamp(min=1)])
    return {"loss": loss.float(), "counts": torch.cat([each, tokens.reshape(1).to(torch.int32)]),
            "prob_mean": mean.float()}


def _route(s):
    logits, ids, w, counts = s["logits"], s["ids"].long(), s["w"], s["counts"]
    E = logits.shape[1]
    filled = ids >= 0
    # routing weights: weighted dots of the slot rows, then the softmax over
    # the selected experts
    dots = s["rs"] * (s["y"] * s["dout"].float().unsqueeze(1)).sum(2)
    dots = torch.where(filled, dots, 0.0)
    d_top = dots - w * dots.sum(1, keepdim=True)
    # balance and z terms: the softmax over all experts
    some = (logits > -math.inf).any(1)
    top = torch.where(some, logits.amax(1), 0.0)
    ex = torch.exp(logits - top[:, None])
    total = torch.where(some, ex.sum(1), 1.0)
    probs = ex / total[:, None]
    lse = top + torch.log(total)
    tokens = counts[-1].clamp(min=1)
    g = s["d_loss"][0] * E * counts[:-1].float() / (counts[:-1].sum().clamp(min=1).float() * tokens)
    inner = (probs * g).sum(1) - 2 * s["d_loss"][1] * lse / tokens
    d = probs * (g - inner[:, None])
    return d.scatter_add(1, ids.clamp(min=0), torch.where(filled, d_top, 0.0))


def _placed(s):
    """Place of each sorted token in a [adapters, most tokens] batch, and the
    tokens themselves."""
    p = torch.arange(s["P"], device="cuda", dtype=torch.int32)
    a = torch.searchsorted(s["offsets"][1:], p, right=True)
    return a * s["most"] + (p - s["offsets"][a]), s["tokens"][:s["P"]].long()


def _rows(rows, at, tok, s):
    """Rows of the tokens as a padded batch [adapters, most tokens, width]."""
    n = s["a"].shape[0]
    out = torch.zeros((n * s["most"], rows.shape[1]), dtype=rows.dtype, device="cuda")
    out[at] = rows[tok]
    return out.view(n, s["most"], -1)


def _lora(s):
    at, tok = _placed(s)
    v = _rows(s["x"].float(), at, tok, s).bmm(s["a"].float().mT)
    delta = v.bmm(s["b"].float()) * s["scales"][:, None, None]
    out = s["base"].clone()
    out[tok] += delta.flatten(0, 1)[at]
    got = {"out": out, "v": torch.zeros_like(s["v"])}
    got["v"][:s["P"]] = v.flatten(0, 1)[at]
    if s["out_bf16"] is not None:
        got["out_bf16"] = out.to(torch.bfloat16)
    return got


def _lora_grad(s):
    at, tok = _placed(s)
    x, dout = _rows(s["x"].float(), at, tok, s), _rows(s["dout"].float(), at, tok, s)
    v = _rows(s["v"], at, torch.arange(s["P"], device="cuda"), s)
    dv = dout.bmm(s["b"].float().mT) * s["scales"][:, None, None]
    dx = s["dx_base"].clone()
    dx[tok] += dv.bmm(s["a"].float()).flatten(0, 1)[at]
    return {"dx": dx, "d_a": dv.mT.bmm(x), "d_b": v.mT.bmm(dout) * s["scales"][:, None, None]}


def run(state):
    s = state
    if own:
        import fp8_blockwise_routed_b200 as fm

        if s["op"] == "balance":
            fm.moe_balance_loss(s["logits"], s["offsets"], s["loss"], s["counts"], s["prob_mean"], s["ws"])
            return {c: s[c] for c in ("loss", "counts", "prob_mean")}
        if s["op"] == "route":
            fm.moe_route_backward(s["logits"], s["ids"], s["w"], s["y"], s["dout"], s["rs"], s["counts"],
                                  s["d_loss"], s["d_logits"])
            return s["d_logits"]
        if s["op"] == "lora":
            fm.moe_lora(s["x"], s["a"], s["b"], s["scales"], s["offsets"], s["tokens"], s["base"], s["v"], s["out"],
                        s["out_bf16"])
            got = {"out": s["out"], "v": s["v"]}
            if s["out_bf16"] is not None:
                got["out_bf16"] = s["out_bf16"]
            return got
        fm.moe_lora_backward(s["x"], s["a"], s["b"], s["scales"], s["offsets"], s["tokens"], s["v"], s["dout"],
                             s["dx_base"], s["dx"], s["d_a"], s["d_b"], s["ws"])
        return {c: s[c] for c in ("dx", "d_a", "d_b")}
    if s["op"] == "balance":
        return _balance(s["logits"], s["offsets"])
    if s["op"] == "route":
        return _route(s)
    return _lora(s) if s["op"] == "lora" else _lora_grad(s)


# ------------------------------------------------------------ work, exact

def work(case):
    op, T = case["op"], case["T"]
    if op == "balance":
        E = case["E"]
        return {"bytes": 4 * T * E + 4 * (E + 1) * 2 + 4 * E + 8, "flops": 6 * T * E}
    if op == "route":
        E, k, H = case["E"], case["k"], case["H"]
        return {"bytes": 4 * T * k * H + 2 * T * H + 8 * T * E + 8 * T * k + 4 * E, "flops": 2 * T * k * H + 12 * T * E}
    K, N, R = case["K"], case["N"], case["R"]
    weights = 2 * min(case["n"], case["requests"]) * R * (K + N)
    if op == "lora":
        return {"bytes": 2 * T * K + weights + 8 * T * N + 4 * T * R + (2 * T * N if case["bf16"] else 0),
                "flops": 2 * T * R * (K + N)}
    return {"bytes": 2 * T * (K + N) + 8 * T * K + weights + 2 * weights + 4 * T * R, "flops": 4 * T * R * (K + N)}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "balance":
        z = s["logits"].double()
        some = torch.isfinite(z).any(1)
        z = z[some]
        probs, lse = torch.softmax(z, 1), torch.logsumexp(z, 1)
        c = (s["offsets"][1:] - s["offsets"][:-1]).double()
        E, tokens = z.shape[1], max(1, z.shape[0])
        mean = probs.sum(0) / tokens
        return {"loss": torch.stack([E * torch.dot(c, mean) / max(1.0, float(c.sum())), lse.pow(2).sum() / tokens]),
                "counts": None, "prob_mean": mean}
    if s["op"] == "route":
        # by differentiation of the layer's loss, the experts' outputs held fixed
        some = (s["ids"] >= 0).any(1)
        z = s["logits"][some].double().requires_grad_()
        ids, w = s["ids"][some].long(), s["w"][some].double()
        filled = ids >= 0
        y = torch.where(filled.unsqueeze(2), s["y"][some], 0.0)
        dots = torch.einsum("tkh,th->tk", y.double(), s["dout"][some].double())
        slope = torch.where(w > 0, dots / torch.where(w > 0, w, 1.0), 0.0)  # of the loss in each routing weight
        picked = torch.where(filled, z.gather(1, ids.clamp(min=0)), -math.inf)
        c = s["counts"].double()
        E, tokens = z.shape[1], float(c[-1])
        balance = E * (torch.softmax(z, 1).sum(0) * c[:-1]).sum() / (float(c[:-1].sum()) * tokens)
        zloss = torch.logsumexp(z, 1).pow(2).sum() / tokens
        total = (s["rs"] * (torch.softmax(picked, 1) * slope).sum() + s["d_loss"][0].double() * balance
                 + s["d_loss"][1].double() * zloss)
        d = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
        d[some] = torch.autograd.grad(total, z)[0] if z.numel() else 0.0
        return d
    off, tok = s["offsets"].tolist(), s["tokens"].long()
    x, a, b = s["x"].double(), s["a"].double(), s["b"].double()
    n = len(off) - 1
    if s["op"] == "lora":
        out, v = s["base"].double(), torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
        for i in range(n):
            t = tok[off[i]:off[i + 1]]
            v[off[i]:off[i + 1]] = x[t] @ a[i].T
            out[t] = out[t] + float(s["scales"][i]) * (v[off[i]:off[i + 1]] @ b[i])
        got = {"out": out, "v": v}
        if s["out_bf16"] is not None:
            got["out_bf16"] = out
        return got
    dx, da, db = s["dx_base"].double(), torch.zeros_like(a), torch.zeros_like(b)
    for i in range(n):
        t, f = tok[off[i]:off[i + 1]], float(s["scales"][i])
        dv = f * (s["dout"][t].double() @ b[i].T)
        da[i] = dv.T @ x[t]
        db[i] = f * (s["v"][off[i]:off[i + 1]].double().T @ s["dout"][t].double())
        dx[t] = dx[t] + dv @ a[i]
    return {"dx": dx, "d_a": da, "d_b": db}
