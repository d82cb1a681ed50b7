"""Measured cases of the router, the few-token expert layer and the routed low-rank adapters.

Each case is one pass through an operator as a program calls it: with ``own``
false its plain form in elementary torch operations, with ``own`` true the
calls of ``combine_topk_idx_amd.ep``.
"""

import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one decoding token: 256 experts in 8 groups of which 4 are kept, biased sigmoid scores
        dict(name="router_one", op="router", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4, top=2,
             renorm=True, scale=2.5, logits="float32", ids="int64", masked=0.0, train=False),
        # a decoding batch with bf16 logits, plain softmax scores
        dict(name="router_decode", op="router", T=128, E=256, k=8, score="softmax", bias=False, groups=1, keep=1,
             top=1, renorm=True, scale=1.0, logits="bfloat16", ids="int64", masked=0.0, train=False),
        # a whole prefill batch through the grouped, biased router
        dict(name="router_large", op="router", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4,
             top=2, renorm=True, scale=2.5, logits="float32", ids="int32", masked=0.0, train=False),
        # a training step's router, an odd expert count, some experts masked out: forward and gradient
        dict(name="router_train", op="router", T=8191, E=60, k=4, score="softmax", bias=False, groups=1, keep=1,
             top=1, renorm=False, scale=1.0, logits="float32", ids="int64", masked=0.05, train=True),
        # the expert layer for one token of a large model (8 of 256 experts)
        dict(name="layer_one", op="layer", T=1, H=7168, I=2048, E=256, k=8, weights="mxfp8", ids="int64", neg=0.0,
             skew=0.0),
        # a small batch on a small model with unquantised weights
        dict(name="layer_small_bf16", op="layer", T=13, H=2048, I=768, E=64, k=6, weights="none", ids="int32",
             neg=0.0, skew=0.5),
        # an odd batch with four-bit weights
        dict(name="layer_mxfp4", op="layer", T=33, H=4096, I=1408, E=128, k=4, weights="mxfp4", ids="int64",
             neg=0.1, skew=0.5),
        # a full decoding batch: nearly every expert is read
        dict(name="layer_decode", op="layer", T=128, H=7168, I=2048, E=256, k=8, weights="mxfp8", ids="int64",
             neg=0.1, skew=0.0),
        # three requests, one token each, a narrow projection
        dict(name="lora_few", op="lora", T=3, IN=2048, OUT=1024, R=8, N=4, none=0.0, skew=0.0, train=False),
        # a decoding batch over many adapters, a quarter of the requests without one
        dict(name="lora_decode", op="lora", T=128, IN=7168, OUT=7168, R=16, N=64, none=0.25, skew=0.5, train=False),
        # prefill of several requests at a higher rank
        dict(name="lora_prefill", op="lora", T=4099, IN=7168, OUT=2048, R=64, N=8, none=0.1, skew=1.0, train=False),
        # a training step of a few adapters: forward and every gradient
        dict(name="lora_train", op="lora", T=8192, IN=7168, OUT=7168, R=16, N=4, none=0.0, skew=0.5, train=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["router", "layer", "lora"])
    if op == "router":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(2, 32 // groups), 512 // groups)
        keep = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(16, E // groups * keep))
        train = rng.random() < 0.4
        T = _log_int(rng, 1, min(16384, 16384 * 256 // E))
        return dict(op="router", T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    groups=groups, keep=keep, top=rng.choice([1, 2]), renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), logits=rng.choice(["float32", "bfloat16", "float16"]),
                    ids=rng.choice(["int32", "int64"]), masked=rng.choice([0.0, 0.05]), train=train)
    if op == "layer":
        H = 64 * _log_int(rng, 8, 96)
        inter = 64 * _log_int(rng, 4, 32)
        E = _log_int(rng, 4, 128)
        k = rng.randint(1, min(8, E))
        return dict(op="layer", T=_log_int(rng, 1, 128), H=H, I=inter, E=E, k=k,
                    weights=rng.choice(["none", "mxfp8", "mxfp4"]), ids=rng.choice(["int32", "int64"]),
                    neg=rng.choice([0.0, 0.1]), skew=rng.choice([0.0, 0.5]))
    return dict(op="lora", T=_log_int(rng, 1, 8192), IN=32 * _log_int(rng, 16, 224), OUT=32 * _log_int(rng, 16, 224),
                R=8 * rng.choice([1, 2, 3, 4, 5, 8, 16]), N=_log_int(rng, 1, 128), none=rng.choice([0.0, 0.25]),
                skew=rng.choice([0.0, 0.5, 1.0]), train=rng.random() < 0.4)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _popular(g, n, skew):
    """Log probabilities of n choices, the r-th most popular one r**-skew, in a random order."""
    p = -skew * torch.log(torch.arange(1, n + 1, device=DEV, dtype=torch.float32))
    return p[torch.randperm(n, generator=g, device=DEV)]


def _gumbel(g, *shape):
    u = torch.rand(*shape, generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
    return -torch.log(-torch.log(u))


def _router_inputs(c, seed):
    g = _gen(seed)
    z = torch.randn(c["T"], c["E"], generator=g, device=DEV) * 1.5
    z = z + torch.randn(c["E"], generator=g, device=DEV) * 0.5
    if c["masked"]:
        z = z.masked_fill(torch.rand(c["T"], c["E"], generator=g, device=DEV) < c["masked"], -math.inf)
    s = dict(logits=z.to(getattr(torch, c["logits"])))
    if c["bias"]:
        s["bias"] = torch.randn(c["E"], generator=g, device=DEV) * 0.1
    if c["train"]:
        s["grad_weights"] = torch.randn(c["T"], c["k"], generator=g, device=DEV)
    return s


def _mx_scales(g, K, *shape):
    base = 127 - int(round(math.log2(K) / 2))
    return torch.randint(base - 1, base + 2, (*shape, K // 32), generator=g, device=DEV, dtype=torch.uint8)


def _weights(g, kind, E, N, K):
    """Expert weights whose rows give products of order one: bf16, or codes with a scale byte per 32."""
    if kind == "none":
        return (torch.randn(E, N, K, generator=g, device=DEV) / math.sqrt(K)).to(torch.bfloat16), None
    if kind == "mxfp4":
        codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        return codes, _mx_scales(g, 4 * K, E, N)[..., : K // 32].contiguous()
    # e4m3 with exponent fields 4..7: magnitudes 0.125 .. 1.875, never NaN
    codes = torch.randint(0, 256, (E, N, K), generator=g, device=DEV, dtype=torch.uint8)
    codes = codes.bitwise_and_(0x9F).bitwise_or_(0x20)
    return codes, _mx_scales(g, K, E, N)


def _layer_inputs(c, seed):
    g = _gen(seed)
    T, H, inter, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    s = dict(x=torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16))
    pick = _popular(g, E, c["skew"]) + _gumbel(g, T, E)
    idx = torch.topk(pick, k, dim=1).indices
    if c["neg"]:
        idx = idx.masked_fill(torch.rand(T, k, generator=g, device=DEV) < c["neg"], -1)
    s["topk_idx"] = idx.to(getattr(torch, c["ids"])).contiguous()
    s["topk_weights"] = torch.softmax(torch.randn(T, k, generator=g, device=DEV), dim=1)
    s["w1"], s["w1_scales"] = _weights(g, c["weights"], E, 2 * inter, H)
    s["w2"], s["w2_scales"] = _weights(g, c["weights"], E, H, inter)
    return s


def _lora_inputs(c, seed):
    g = _gen(seed)
    T, IN, OUT, R, N = c["T"], c["IN"], c["OUT"], c["R"], c["N"]
    ids = torch.argmax(_popular(g, N, c["skew"]) + _gumbel(g, T, N), dim=1)
    if c["none"]:
        ids = ids.masked_fill(torch.rand(T, generator=g, device=DEV) < c["none"], -1)

    def rows(*shape, by=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * by).to(torch.bfloat16)

    s = dict(ids=ids.to(torch.int32).view(T, 1), x=rows(T, IN), base=rows(T, OUT), a=rows(N, R, IN, by=IN ** -0.5),
             b=rows(N, OUT, R, by=R ** -0.5), scale=torch.rand(N, generator=g, device=DEV) + 0.5)
    if c["train"]:
        s["grad_out"], s["grad_base"] = rows(T, OUT), rows(T, IN)
    return s


def _inputs(case, seed):
    s = {"router": _router_inputs, "layer": _layer_inputs, "lora": _lora_inputs}[case["op"]](case, seed)
    s["case"] = case
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _keep(case, s)
    return s


def _keep(c, s):
    """What a program using the library keeps between calls: output buffers, workspaces, packed weights, the
    layout of the requests' adapters (one layout serves every projection of a step)."""
    from combine_topk_idx_amd import ep

    def new(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=DEV)

    if c["op"] == "router":
        s["topk_idx"] = new(c["T"], c["k"], dtype=getattr(torch, c["ids"]))
        s["topk_weights"] = new(c["T"], c["k"])
        if c["train"]:
            s["grad_logits"] = torch.empty_like(s["logits"])
    elif c["op"] == "layer":
        s["p1"] = ep.pack_moe_weights(s["w1"], s["w1_scales"], True, quant=c["weights"])
        s["p2"] = ep.pack_moe_weights(s["w2"], s["w2_scales"], False, quant=c["weights"])
        s["workspace"] = new(ep.ep_moe_layer_workspace_bytes(c["T"], c["k"], c["E"], c["H"], c["I"]),
                             dtype=torch.uint8)
        s["out"] = new(c["T"], c["H"], dtype=torch.bfloat16)
    else:
        T, R, N = c["T"], c["R"], c["N"]
        s["layout_workspace"] = new(ep.ep_workspace_bytes(T, 1, N), dtype=torch.uint8)
        s["handle"] = ep.ep_layout(s["ids"], N, T, new(N, dtype=torch.int64), s["layout_workspace"])
        s["out"], s["down"] = new(T, c["OUT"], dtype=torch.bfloat16), new(T, R)
        if c["train"]:
            s["grad_x"] = new(T, c["IN"], dtype=torch.bfloat16)
            s["grad_a"], s["grad_b"] = new(N, R, c["IN"]), new(N, c["OUT"], R)
        s["workspace"] = new(ep.ep_lora_workspace_bytes(T, c["IN"], c["OUT"], R, N, c["train"]), dtype=torch.uint8)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"router": _router_own, "layer": _layer_own, "lora": _lora_own}[op](state)
    return {"router": _router_plain, "layer": _layer_plain, "lora": _lora_plain}[op](state)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------


def _router_own(s):
    from combine_topk_idx_amd import ep
    c = s["case"]
    ep.ep_router(s["logits"], s["topk_idx"], s["topk_weights"], score=c["score"], bias=s.get("bias"),
                 num_groups=c["groups"], topk_groups=c["keep"], group_top=c["top"], renormalize=c["renorm"],
                 scale=c["scale"])
    if not c["train"]:
        return s["topk_idx"], s["topk_weights"]
    ep.ep_router_backward(s["logits"], s["topk_idx"], s["grad_weights"], s["grad_logits"], score=c["score"],
                          renormalize=c["renorm"], scale=c["scale"])
    return s["topk_idx"], s["topk_weights"], s["grad_logits"]


def _layer_own(s):
    from combine_topk_idx_amd import ep
    c = s["case"]
    ep.ep_moe_layer(s["x"], s["topk_idx"], s["topk_weights"], c["E"], c["I"], c["weights"], *s["p1"], *s["p2"],
                    s["workspace"], s["out"])
    return s["out"]


def _lora_own(s):
    from combine_topk_idx_amd import ep
    c = s["case"]
    ep.ep_lora(s["handle"], s["x"], s["a"], s["b"], s["out"], s["down"], s["workspace"], scale=s["scale"],
               base=s["base"])
    if not c["train"]:
        return s["out"]
    ep.ep_lora_backward(s["handle"], s["grad_out"], s["x"], s["a"], s["b"], s["down"], s["grad_x"], s["grad_a"],
                        s["grad_b"], s["workspace"], scale=s["scale"], grad_base=s["grad_base"])
    return s["out"], s["grad_x"], s["grad_a"], s["grad_b"]


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _router_plain(s):
    # keys in 64 bits: two experts' keys may lie closer than 32-bit rounding
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    z = s["logits"].double()
    ok = z > -math.inf                                    # false for NaN
    zm = z.masked_fill(~ok, -math.inf)
    if c["score"] == "softmax":
        top = zm.amax(1, keepdim=True)
        p = torch.exp(zm - top.masked_fill(top == -math.inf, 0.0))
        score = p / p.sum(1, keepdim=True).clamp_min(1e-300)
        log_score = zm
    else:
        score = 1.0 / (1.0 + torch.exp(-zm))
        log_score = -torch.log1p(torch.exp(-zm))
    biased = "bias" in s
    by_score = score + s["bias"].double() if biased else score
    by_score = by_score.masked_fill(~ok, -math.inf)
    key = by_score if biased else zm                      # the scores rise with the logits
    if c["groups"] > 1:
        G = c["groups"]
        per = (zm if c["top"] == 1 and not biased else by_score).view(T, G, E // G)
        rank = torch.sort(per, dim=2, descending=True).values[:, :, :c["top"]].sum(2)
        kept = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        allowed = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        key = key.view(T, G, E // G).masked_fill(~allowed[:, :, None], -math.inf).view(T, E)
    val, idx = torch.sort(key, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    used = val > -math.inf
    weights = _router_weights(c, torch.gather(score, 1, idx), torch.gather(log_score, 1, idx), used)
    out_idx = idx.masked_fill(~used, -1).to(getattr(torch, c["ids"]))
    if not c["train"]:
        return out_idx, (weights * c["scale"]).float()
    grad = s["grad_weights"].double().masked_fill(~used, 0.0) * c["scale"]
    if c["renorm"]:
        d = weights * (grad - (weights * grad).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d * (1.0 - torch.gather(score, 1, idx))
        dz = torch.zeros_like(z).scatter_add_(1, idx, d.masked_fill(~used, 0.0))
    else:
        dz = torch.zeros_like(z).scatter_add_(1, idx, grad)
        if c["score"] == "sigmoid":
            dz = dz * score * (1.0 - score)
        else:
            dz = score * (dz - (weights * grad).sum(1, keepdim=True))
    return out_idx, (weights * c["scale"]).float(), dz.to(s["logits"].dtype)


def _router_weights(c, score, log_score, used):
    if not c["renorm"]:
        return score.masked_fill(~used, 0.0)
    ls = log_score.masked_fill(~used, -math.inf)
    top = ls.amax(1, keepdim=True)
    e = torch.exp(ls - top.masked_fill(top == -math.inf, 0.0))
    return e / e.sum(1, keepdim=True).clamp_min(1e-300)


def _decode(kind, w, scales):
    """Expert weights in float32."""
    if kind == "none":
        return w.float()
    if kind == "mxfp4":
        one = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=w.device)
        byte = torch.arange(256, device=w.device)
        v = torch.stack((one[byte & 15], one[byte >> 4]), dim=1)[w.int()].flatten(-2)
    else:
        v = w.view(torch.float8_e4m3fn).float()
    v.view(*v.shape[:-1], -1, 32).mul_(torch.exp2(scales.float() - 127.0)[..., None])
    return v


def _take(t, i):
    return None if t is None else t[i]


def _layer_plain(s):
    c = s["case"]
    T, H, inter, k = c["T"], c["H"], c["I"], c["k"]
    flat = s["topk_idx"].long().view(-1)
    pairs = torch.nonzero(flat >= 0).view(-1)
    rows = torch.zeros(T * k, H, device=flat.device)
    if pairs.numel():
        experts, at, count = torch.unique(flat[pairs], return_inverse=True, return_counts=True)
        order = torch.argsort(at, stable=True)
        place = torch.empty_like(at)
        place[order] = torch.arange(at.numel(), device=at.device) - (torch.cumsum(count, 0) - count)[at[order]]
        x = torch.zeros(experts.numel(), int(count.max()), H, device=flat.device)
        x[at, place] = s["x"].float()[pairs // k]
        w1 = _decode(c["weights"], s["w1"][experts], _take(s["w1_scales"], experts))
        gu = torch.bmm(x, w1.transpose(1, 2))
        del w1
        gate, up = gu[..., :inter], gu[..., inter:]
        act = gate / (1.0 + torch.exp(-gate)) * up
        w2 = _decode(c["weights"], s["w2"][experts], _take(s["w2_scales"], experts))
        y = torch.bmm(act, w2.transpose(1, 2))
        rows[pairs] = y[at, place]
    return (rows.view(T, k, H) * s["topk_weights"][:, :, None]).sum(1).to(torch.bfloat16)


def _lora_plain(s):
    # every adapter's down product of every row, the row's own one picked: cheap while the rank is low
    c = s["case"]
    T, IN, OUT, R, N = c["T"], c["IN"], c["OUT"], c["R"], c["N"]
    ids = s["ids"].view(T).long()
    mine = torch.zeros(T, N, device=ids.device).scatter_(1, ids.clamp_min(0)[:, None], (ids >= 0).float()[:, None])
    a, b = s["a"].float(), s["b"].float()
    x = s["x"].float()
    rows = torch.arange(T, device=ids.device)
    down = (x @ a.view(N * R, IN).t()).view(T, N, R)[rows, ids.clamp_min(0)]
    scaled = mine * s["scale"]
    b_in = b.permute(0, 2, 1).reshape(N * R, OUT)
    out = s["base"].float() + (scaled[:, :, None] * down[:, None, :]).view(T, N * R) @ b_in
    out = out.to(torch.bfloat16)
    if not c["train"]:
        return out
    dy = s["grad_out"].float()
    u = (dy @ b_in.t()).view(T, N, R) * scaled[:, :, None]
    grad_x = (s["grad_base"].float() + u.view(T, N * R) @ a.view(N * R, IN)).to(torch.bfloat16)
    grad_a = (u.view(T, N * R).t() @ x).view(N, R, IN)
    placed = (scaled[:, :, None] * down[:, None, :]).view(T, N * R)
    grad_b = (placed.t() @ dy).view(N, R, OUT).permute(0, 2, 1).contiguous()
    return out, grad_x, grad_a, grad_b


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "router":
        z = c["T"] * c["E"] * (4 if c["logits"] == "float32" else 2)
        pair = c["T"] * c["k"] * ((8 if c["ids"] == "int64" else 4) + 4)
        n = z + pair + (4 * c["E"] if c["bias"] else 0)
        if c["train"]:
            n += z + c["T"] * c["k"] * 4
        return {"bytes": n, "flops": (20 if c["train"] else 10) * c["T"] * c["E"]}
    if c["op"] == "layer":
        # the experts that so many uniform draws leave in use
        pairs = c["T"] * c["k"] * (1.0 - c["neg"])
        used = c["E"] * (1.0 - (1.0 - c["k"] * (1.0 - c["neg"]) / c["E"]) ** c["T"])
        one = {"none": 2.0, "mxfp8": 1.0 + 1 / 32, "mxfp4": 0.5 + 1 / 32}[c["weights"]]
        n = used * 3 * c["H"] * c["I"] * one + c["T"] * (4 * c["H"] + 12 * c["k"])
        return {"bytes": int(n), "flops": int(6 * pairs * c["H"] * c["I"])}
    T, IN, OUT, R = c["T"], c["IN"], c["OUT"], c["R"]
    rows = T * (1.0 - c["none"])
    used = c["N"] * (1.0 - (1.0 - (1.0 - c["none"]) / c["N"]) ** T)
    n = rows * 2 * IN + T * 4 * OUT + used * 2 * R * (IN + OUT)
    flops = 2 * rows * R * (IN + OUT)
    if c["train"]:
        n += rows * 2 * OUT + T * 4 * IN + c["N"] * 4 * R * (IN + OUT)
        flops *= 3
    return {"bytes": int(n), "flops": int(flops)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    s = _inputs(case, seed)
    return {"router": _router_exact, "layer": _layer_exact, "lora": _lora_exact}[case["op"]](case, s)


def _router_exact(c, s):
    """From the chosen experts of the definition: a host sort per row, the weights and gradients by formula."""
    import numpy as np
    z = s["logits"].double().cpu().numpy()
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    bias = s["bias"].double().cpu().numpy() if c["bias"] else None
    with np.errstate(all="ignore"):
        ok = z > -np.inf
        if c["score"] == "softmax":
            m = np.where(ok, z, -np.inf).max(1, keepdims=True)
            e = np.where(ok, np.exp(z - m), 0.0)
            total = e.sum(1, keepdims=True)
            score = np.where(total > 0, e / total, 0.0)
        else:
            score = np.where(ok, 1.0 / (1.0 + np.exp(-z)), 0.0)
        key = np.where(ok, z if bias is None else score + bias, -np.inf)
        if G > 1:
            of = np.where(ok, score if bias is None else score + bias, -np.inf) if c["top"] == 2 else key
            best = -np.sort(-of.reshape(T, G, -1), axis=2)
            rank = best[:, :, 0] if c["top"] == 1 else best[:, :, 0] + best[:, :, 1]
            place = np.argsort(np.argsort(-rank, axis=1, kind="stable"), axis=1)
            key = np.where(np.repeat(place < c["keep"], E // G, axis=1), key, -np.inf)
        idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
        used = np.take_along_axis(key, idx, 1) > -np.inf
        w = np.where(used, np.take_along_axis(score, idx, 1), 0.0)
        if c["renorm"]:
            sums = w.sum(1, keepdims=True)
            w = np.where(sums > 0, w / sums, 0.0)
        weights = w * c["scale"]
        if not c["train"]:
            return None, torch.from_numpy(weights)
        g = np.where(used, s["grad_weights"].double().cpu().numpy(), 0.0) * c["scale"]
        # d(weight_j)/d(z_e) = weight_j (d log s_j / d z_e - [renormalised] sum_i weight_i d log s_i / d z_e)
        at = np.where(used, idx, 0)
        wg = w * g
        pull = wg - w * wg.sum(1, keepdims=True) if c["renorm"] else wg     # d(loss) / d(log s_j)
        if c["score"] == "sigmoid":
            pull = pull * (1.0 - np.take_along_axis(score, at, 1))
        dz = np.zeros_like(z)
        np.add.at(dz, (np.arange(T)[:, None], at), np.where(used, pull, 0.0))
        if c["score"] == "softmax":
            dz -= score * pull.sum(1, keepdims=True)
        return None, torch.from_numpy(weights), torch.from_numpy(dz)


def _value64(kind, w, scales):
    if kind == "none":
        return w.double()
    if kind == "mxfp4":
        code = torch.empty(*w.shape[:-1], 2 * w.shape[-1], dtype=torch.uint8, device=w.device)
        code[..., 0::2], code[..., 1::2] = w % 16, w // 16
        sign, mag = 1.0 - 2.0 * (code // 8).double(), (code % 8).double()
        e, m = torch.floor(mag / 2), mag % 2
        v = sign * torch.where(e == 0, m * 0.5, torch.pow(2.0, e - 1) * (1.0 + 0.5 * m))
    else:
        sign, e, m = 1.0 - 2.0 * (w // 128).double(), (w % 128 // 8).double(), (w % 8).double()
        v = sign * torch.where(e == 0, m * 2.0 ** -9, torch.pow(2.0, e - 7) * (1.0 + m / 8))
    return v * torch.pow(2.0, scales.double() - 127.0).repeat_interleave(32, dim=-1)


def _layer_exact(c, s):
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV)
    x, weights = s["x"].double(), s["topk_weights"].double()
    for e in torch.unique(s["topk_idx"]).tolist():
        if e < 0:
            continue
        t, j = torch.nonzero(s["topk_idx"] == e, as_tuple=True)
        h = x[t] @ _value64(c["weights"], s["w1"][e], _take(s["w1_scales"], e)).t()
        gate, up = h[:, : c["I"]], h[:, c["I"]:]
        y = (gate * torch.sigmoid(gate) * up) @ _value64(c["weights"], s["w2"][e], _take(s["w2_scales"], e)).t()
        out.index_add_(0, t, y * weights[t, j][:, None])
    return out


def _lora_exact(c, s):
    ids = s["ids"].view(-1)
    out = s["base"].double()
    grads = [s["grad_base"].double(), torch.zeros(s["a"].shape, dtype=torch.float64, device=DEV),
             torch.zeros(s["b"].shape, dtype=torch.float64, device=DEV)] if c["train"] else None
    for n in range(c["N"]):
        t = torch.nonzero(ids == n).view(-1)
        a, b, by = s["a"][n].double(), s["b"][n].double(), s["scale"][n].double()
        x = s["x"][t].double()
        v = x @ a.t()
        out[t] += by * (v @ b.t())
        if grads:
            dy = s["grad_out"][t].double()
            u = by * (dy @ b)
            grads[0][t] += u @ a
            grads[1][n] = u.t() @ x
            grads[2][n] = by * (dy.t() @ v)
    return (out, *grads) if grads else out
