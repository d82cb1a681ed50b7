"""Measured cases of the gated feed-forward block of expert rows, its 8-bit checkpoints and the block-scaled product.

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
        # a few requests through a small expert block, no training: latency
        dict(name="ffn_few", op="ffn", T=5, k=2, E=8, H=1024, I=512, align=1, neg=0.0, skew=0.0, act="silu",
             train=False, ckpt="none"),
        # a decoding batch over every expert of a small model: about twelve rows an expert, the weights bound it
        dict(name="ffn_decode", op="ffn", T=128, k=6, E=64, H=2048, I=768, align=1, neg=0.0, skew=0.5, act="silu",
             train=False, ckpt="none"),
        # prefill: many rows an expert, inference
        dict(name="ffn_prefill", op="ffn", T=4096, k=4, E=32, H=4096, I=1408, align=1, neg=0.1, skew=0.5, act="silu",
             train=False, ckpt="none"),
        # a small training step, odd token count, GELU gate, bf16 checkpoint
        dict(name="ffn_train_small", op="ffn", T=509, k=4, E=16, H=1024, I=448, align=1, neg=0.0, skew=1.0,
             act="gelu", train=True, ckpt="none"),
        # a training step over aligned expert blocks with the 8-bit checkpoint, some pairs without an expert
        dict(name="ffn_train_fp8", op="ffn", T=1531, k=6, E=64, H=2048, I=768, align=16, neg=0.1, skew=0.5,
             act="silu", train=True, ckpt="fp8_b128"),
        # a training step of one dense block (a shared expert): every token, one pair of weights
        dict(name="ffn_train_dense", op="ffn", T=8192, k=1, E=1, H=4096, I=1408, align=1, neg=0.0, skew=0.0,
             act="silu", train=True, ckpt="none"),
        # the largest training step: the experts of a large model that fall to one GPU, 8-bit checkpoint
        dict(name="ffn_train_large", op="ffn", T=4096, k=8, E=32, H=7168, I=2048, align=1, neg=0.0, skew=0.5,
             act="silu", train=True, ckpt="fp8_b128"),
        # a few requests through a small block-scaled product
        dict(name="gmm_few", op="gmm", T=5, k=2, E=8, K=1024, N=1024, align=1, neg=0.0, skew=0.0, act="none",
             transposed=False, rows="fp8_b128"),
        # a decoding batch of a large model through gate and up projection: four rows an expert
        dict(name="gmm_decode", op="gmm", T=128, k=8, E=256, K=7168, N=4096, align=1, neg=0.0, skew=0.0, act="silu",
             transposed=False, rows="fp8_b128"),
        # an odd batch through the down projection, power-of-two scales as bytes
        dict(name="gmm_odd", op="gmm", T=1001, k=6, E=64, K=1408, N=4096, align=16, neg=0.1, skew=0.5, act="none",
             transposed=False, rows="fp8_b128_ue8m0"),
        # prefill through gate and up projection
        dict(name="gmm_prefill", op="gmm", T=4096, k=8, E=32, K=7168, N=4096, align=1, neg=0.0, skew=0.5, act="silu",
             transposed=False, rows="fp8_b128"),
        # the gradient of the rows through the same weights
        dict(name="gmm_gradient", op="gmm", T=4096, k=8, E=32, K=4096, N=7168, align=1, neg=0.0, skew=0.5,
             act="none", transposed=True, rows="fp8_b128"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    k = rng.randint(1, 8)
    c = dict(op=rng.choice(["ffn", "gmm"]), T=_log_int(rng, 1, 4096), k=k, align=rng.choice([1, 1, 16, 128]),
             neg=rng.choice([0.0, 0.1]), skew=rng.choice([0.0, 0.5, 1.0]))
    if c["op"] == "ffn":
        c.update(E=_log_int(rng, k, 32), H=64 * _log_int(rng, 4, 112), act=rng.choice(["silu", "gelu"]),
                 train=rng.random() < 0.6, ckpt=rng.choice(["none", "fp8_b128"]))
        # an 8-bit checkpoint has a scale for each 128 channels
        c["I"] = 128 * _log_int(rng, 1, 16) if c["ckpt"] != "none" else 64 * _log_int(rng, 3, 32)
        return c
    c.update(E=_log_int(rng, k, 128), K=128 * _log_int(rng, 2, 56), N=128 * _log_int(rng, 2, 32),
             transposed=rng.random() < 0.3, rows=rng.choice(["fp8_b128", "fp8_b128_pow2", "fp8_b128_ue8m0"]))
    c["act"] = "none" if c["transposed"] or c["N"] % 256 else rng.choice(["none", "silu", "gelu"])
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _max_rows(c):
    return c["T"] * c["k"] + c["E"] * (c["align"] - 1)


def _routing(g, c):
    """Ids of a batch whose r-th most popular expert is drawn r**-skew times as often as the first."""
    T, k, E = c["T"], c["k"], c["E"]
    p = -c["skew"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    u = torch.rand(T, E, generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
    pick = p[torch.randperm(E, generator=g, device=DEV)] - torch.log(-torch.log(u))
    idx = torch.topk(pick, k, dim=1).indices
    if c["neg"]:
        idx = idx.masked_fill(torch.rand(T, k, generator=g, device=DEV) < c["neg"], -1)
    return idx.contiguous()


def _blocks(c, topk_idx):
    """Rows of every expert and the first row of its block."""
    flat = topk_idx.reshape(-1)
    count = torch.zeros(c["E"], dtype=torch.int64, device=flat.device)
    count.scatter_add_(0, flat.clamp_min(0), (flat >= 0).long())
    block = (count + c["align"] - 1) // c["align"] * c["align"]
    return count, torch.cumsum(block, 0) - block


def _held(c, count, start):
    """Which rows of the buffers hold a pair."""
    held = torch.zeros(_max_rows(c) + 1, dtype=torch.int64, device=count.device)
    held.scatter_add_(0, start, (count > 0).long())
    held.scatter_add_(0, start + count, -(count > 0).long())
    return torch.cumsum(held, 0)[:-1] > 0


def _ffn_inputs(c, seed):
    g = _gen(seed)
    E, H, inter = c["E"], c["H"], c["I"]
    s = dict(topk_idx=_routing(g, c))
    empty = ~_held(c, *_blocks(c, s["topk_idx"]))[:, None]

    def rows(width, by=1.0):      # rows that hold no pair are whatever was there: not a number, to be sure
        return (torch.randn(_max_rows(c), width, generator=g, device=DEV) * by).masked_fill_(empty, math.nan).to(
            torch.bfloat16)

    def weights(n, k):
        w = torch.empty(E, n, k, dtype=torch.bfloat16, device=DEV)
        for e in range(E):
            w[e] = torch.randn(n, k, generator=g, device=DEV) * k ** -0.5
        return w

    s["x"], s["w1"], s["w2"] = rows(H), weights(2 * inter, H), weights(H, inter)
    s["out"] = torch.zeros_like(s["x"])
    if c["train"]:
        s["grad_out"] = rows(H, 0.1)
        s["grad_x"] = torch.zeros_like(s["x"])
    return s


def _gmm_inputs(c, seed):
    g = _gen(seed)
    E, K, N, R = c["E"], c["K"], c["N"], _max_rows(c)
    s = dict(topk_idx=_routing(g, c))
    empty = ~_held(c, *_blocks(c, s["topk_idx"]))[:, None]
    x = torch.randn(R, K // 128, 128, generator=g, device=DEV).mul_(
        torch.rand(R, K // 128, 1, generator=g, device=DEV) * 2 + 0.1)
    top = x.abs().amax(2, keepdim=True)
    scale = top / 448.0
    if c["rows"] != "fp8_b128":
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    codes = (x / scale).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(R, K)
    s["codes"] = codes.masked_fill_(empty, 0x7F)
    scale = scale.view(R, K // 128)
    if c["rows"] == "fp8_b128_ue8m0":
        s["scales"] = (torch.log2(scale).round_() + 127).to(torch.uint8).masked_fill_(empty, 0xFF)
    else:
        s["scales"] = scale.masked_fill(empty, math.nan)
    n, k = (K, N) if c["transposed"] else (N, K)       # the weights lie as the forward pass has them
    w = torch.randint(0, 256, (E, n, k), generator=g, device=DEV, dtype=torch.uint8)
    # e4m3 with exponent fields 4..7: magnitudes 0.125 .. 1.875, never NaN
    s["w"] = w.bitwise_and_(0x9F).bitwise_or_(0x20)
    s["w_scales"] = (torch.rand(E, n // 128, k // 128, generator=g, device=DEV) + 0.5) * (1.5 * K) ** -0.5
    s["out"] = torch.zeros(R, N // 2 if c["act"] != "none" else N, dtype=torch.bfloat16, device=DEV)
    return s


def _inputs(case, seed):
    s = {"ffn": _ffn_inputs, "gmm": _gmm_inputs}[case["op"]](case, seed)
    s["case"] = case
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _keep(case, s)
    return s


def _keep(c, s):
    """What a program using the library has before the call: the layout of the step's routing, workspaces, the
    buffers that the dispatch filled."""
    from combine_topk_idx_amd import ep

    def new(*shape, dtype=torch.uint8):
        return torch.empty(*shape, dtype=dtype, device=DEV)

    T, k, E, R = c["T"], c["k"], c["E"], _max_rows(c)
    s["layout_workspace"] = new(ep.ep_workspace_bytes_ex(T, k, E, c["align"], 0))
    s["count"] = new(E, dtype=torch.int64)
    s["handle"] = ep.ep_layout_ex(s["topk_idx"], E, T, c["align"], 0, s["count"], s["layout_workspace"])
    if c["op"] == "ffn":
        s["workspace"] = new(ep.ep_ffn_workspace_bytes(R, c["H"], c["I"], E, c["train"]))
        if c["train"]:
            s["checkpoint"] = new(ep.ep_buffer_bytes(R, 2 * c["I"], c["ckpt"])[0])
            s["grad_w1"], s["grad_w2"] = torch.empty_like(s["w1"]), torch.empty_like(s["w2"])
    else:
        total, at = ep.ep_buffer_bytes(R, c["K"], c["rows"])
        s["buf"] = new(total)
        s["buf"][: R * c["K"]] = s["codes"].view(-1)
        s["buf"][at:] = s["scales"].view(-1).view(torch.uint8)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"ffn": _ffn_own, "gmm": _gmm_own}[op](state)
    return {"ffn": _ffn_plain, "gmm": _gmm_plain}[op](state)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------


def _ffn_own(s):
    from combine_topk_idx_amd import ep
    c = s["case"]
    if not c["train"]:
        ep.ep_ffn(s["handle"], s["x"], s["w1"], s["w2"], s["workspace"], s["out"], act=c["act"],
                  recv_count=s["count"])
        return s["out"]
    ep.ep_ffn(s["handle"], s["x"], s["w1"], s["w2"], s["workspace"], s["out"], act=c["act"], recv_count=s["count"],
              checkpoint=s["checkpoint"], checkpoint_quant=c["ckpt"])
    ep.ep_ffn_backward(s["handle"], s["grad_out"], s["x"], s["w1"], s["w2"], s["checkpoint"], s["workspace"],
                       s["grad_x"], s["grad_w1"], s["grad_w2"], act=c["act"], checkpoint_quant=c["ckpt"],
                       recv_count=s["count"])
    return s["out"], s["grad_x"], s["grad_w1"], s["grad_w2"]


def _gmm_own(s):
    from combine_topk_idx_amd import ep
    c = s["case"]
    ep.ep_moe_gmm_b128(s["handle"], s["buf"], c["rows"], c["K"], c["N"], s["w"], s["w_scales"], s["out"],
                       act=c["act"], transposed=c["transposed"], recv_count=s["count"])
    return s["out"]


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _places(s):
    """Row of each place of a [experts, most rows] grid, and which places hold one."""
    count, start = _blocks(s["case"], s["topk_idx"])
    at = torch.arange(max(1, int(count.max())), device=count.device)
    ok = at < count[:, None]
    return (start[:, None] + at).masked_fill(~ok, 0), ok


def _grid(rows, place, ok):
    return rows[place].float().masked_fill(~ok[:, :, None], 0.0)


def _act(kind, z):
    """The gate's activation and its derivative."""
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    p = 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5))
    return z * p, p + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5


def _checkpoint(c, v):
    """What the checkpoint's values stand for: e4m3 codes with a scale for each 128 channels."""
    if c["ckpt"] == "none":
        return v
    b = v.view(*v.shape[:-1], -1, 128)
    top = b.abs().amax(-1, keepdim=True)
    codes = (b * (448.0 / top.clamp_min(1e-30))).clamp(-448, 448).to(torch.float8_e4m3fn)
    return (codes.float() * (top / 448.0)).view(v.shape)


def _ffn_plain(s):
    c = s["case"]
    inter = c["I"]
    place, ok = _places(s)
    x, w1, w2 = _grid(s["x"], place, ok), s["w1"].float(), s["w2"].float()
    gu = torch.bmm(x, w1.transpose(1, 2))
    y = torch.bmm(_act(c["act"], gu[..., :inter])[0] * gu[..., inter:], w2.transpose(1, 2))
    s["out"][place[ok]] = y[ok].to(torch.bfloat16)
    if not c["train"]:
        return s["out"]
    gu = _checkpoint(c, gu)
    gate, up = gu[..., :inter], gu[..., inter:]
    f, df = _act(c["act"], gate)
    dy = _grid(s["grad_out"], place, ok)
    dh = torch.bmm(dy, w2)
    d = torch.cat((dh * up * df, dh * f), dim=2)
    s["grad_x"][place[ok]] = torch.bmm(d, w1)[ok].to(torch.bfloat16)
    grad_w1 = torch.bmm(d.transpose(1, 2), x).to(torch.bfloat16)
    grad_w2 = torch.bmm(dy.transpose(1, 2), f * up).to(torch.bfloat16)
    return s["out"], s["grad_x"], grad_w1, grad_w2


def _gmm_plain(s):
    c = s["case"]
    place, ok = _places(s)
    scale = s["scales"] if c["rows"] != "fp8_b128_ue8m0" else torch.exp2(s["scales"].float() - 127.0)
    x = s["codes"][place].view(torch.float8_e4m3fn).float()
    x = (x.view(*place.shape, -1, 128) * scale[place][..., None]).view(*place.shape, -1)
    x = x.masked_fill(~ok[:, :, None], 0.0)
    w = s["w"].view(torch.float8_e4m3fn).float()
    w.view(c["E"], w.shape[1] // 128, 128, w.shape[2] // 128, 128).mul_(s["w_scales"][:, :, None, :, None])
    y = torch.bmm(x, w if c["transposed"] else w.transpose(1, 2))
    if c["act"] != "none":
        y = _act(c["act"], y[..., : c["N"] // 2])[0] * y[..., c["N"] // 2:]
    s["out"][place[ok]] = y[ok].to(torch.bfloat16)
    return s["out"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    c = case
    rows = c["T"] * c["k"] * (1.0 - c["neg"])
    # the experts that so many uniform draws leave in use
    used = c["E"] * (1.0 - (1.0 - c["k"] * (1.0 - c["neg"]) / c["E"]) ** c["T"])
    if c["op"] == "gmm":
        out = c["N"] // 2 if c["act"] != "none" else c["N"]
        one = 1 + (1 if c["rows"] == "fp8_b128_ue8m0" else 4) / 128
        n = used * c["K"] * c["N"] * (1 + 4 / 128 ** 2) + rows * (c["K"] * one + 2 * out)
        return {"bytes": int(n), "flops": int(2 * rows * c["K"] * c["N"])}
    H, inter = c["H"], c["I"]
    n, flops = used * 6 * H * inter + rows * 4 * H, 6 * rows * H * inter
    if c["train"]:
        # a backward pass of its own: the weights and the rows again, the checkpoint out and in
        n += used * 6 * H * inter + c["E"] * 6 * H * inter + rows * 6 * H
        n += 2 * rows * 2 * inter * (2 if c["ckpt"] == "none" else 1 + 4 / 128)
        flops *= 3
    return {"bytes": int(n), "flops": int(flops)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    s = _inputs(case, seed)
    return {"ffn": _ffn_exact, "gmm": _gmm_exact}[case["op"]](case, s)


def _spans(c, topk_idx):
    """(expert, first row, rows) of every expert with rows."""
    at = 0
    for e in range(c["E"]):
        n = int((topk_idx == e).sum())
        if n:
            yield e, at, n
        at += -(-n // c["align"]) * c["align"]


def _exact_act(kind, z):
    if kind == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    p = torch.special.ndtr(z)
    return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def _exact_checkpoint(v):
    """e4m3 codes and scales by 128 channels, in float32 as the format has them, from values in 64 bits."""
    n, wide = v.shape
    b = v.view(n, wide // 128, 128)
    top = b.abs().max(dim=2, keepdim=True).values
    q = torch.where(top > 0, b * 448.0 / top, torch.zeros_like(b))
    # the codes' spacing: 2^-3 of the power of two at or below the value, 2^-9 at least
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(q / step) * step * (top / 448.0)).view(n, wide)


def _ffn_exact(c, s):
    inter = c["I"]
    out = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
    if c["train"]:
        grad_x = torch.zeros_like(out)
        grad_w1 = torch.zeros(s["w1"].shape, dtype=torch.float64, device=DEV)
        grad_w2 = torch.zeros(s["w2"].shape, dtype=torch.float64, device=DEV)
    for e, at, n in _spans(c, s["topk_idx"]):
        x, w1, w2 = s["x"][at:at + n].double(), s["w1"][e].double(), s["w2"][e].double()
        gate, up = x @ w1[:inter].t(), x @ w1[inter:].t()
        out[at:at + n] = (_exact_act(c["act"], gate)[0] * up) @ w2.t()
        if not c["train"]:
            continue
        if c["ckpt"] != "none":
            both = _exact_checkpoint(torch.cat((gate, up), dim=1))
            gate, up = both[:, :inter], both[:, inter:]
        f, df = _exact_act(c["act"], gate)
        dy = s["grad_out"][at:at + n].double()
        dh = dy @ w2
        d_gate, d_up = dh * up * df, dh * f
        grad_x[at:at + n] = d_gate @ w1[:inter] + d_up @ w1[inter:]
        grad_w1[e, :inter], grad_w1[e, inter:] = d_gate.t() @ x, d_up.t() @ x
        grad_w2[e] = dy.t() @ (f * up)
    return (out, grad_x, grad_w1, grad_w2) if c["train"] else out


def _value64(code):
    """What an e4m3 code stands for."""
    sign, e, m = 1.0 - 2.0 * (code // 128).double(), (code % 128 // 8).double(), (code % 8).double()
    return sign * torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e - 7) * (1.0 + m / 8))


def _gmm_exact(c, s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for e, at, n in _spans(c, s["topk_idx"]):
        scale = s["scales"][at:at + n].double()
        if c["rows"] == "fp8_b128_ue8m0":
            scale = torch.exp2(scale - 127)
        x = _value64(s["codes"][at:at + n]) * scale.repeat_interleave(128, dim=1)
        w = _value64(s["w"][e]) * s["w_scales"][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        y = x @ w if c["transposed"] else x @ w.t()
        if c["act"] != "none":
            y = _exact_act(c["act"], y[:, : c["N"] // 2])[0] * y[:, c["N"] // 2:]
        out[at:at + n] = y
    return out
