"""The operators around the recurrence of a linear-attention layer, as measured cases: the short causal convolution
before it (and its gradient), the selective state space scan (the recurrence with a scalar decay and no erase) for
prompts and for single tokens, and the layer norm after it, gated or not (and its gradient)."""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------------------------------
# Sequences: B of them, lengths drawn from T .. T_hi by `lens`, packed one after the other; with T == T_hi the batch is
# dense. wide: the input rows are a slice of rows that are this many values longer.
#   conv, conv_back: D channels, width taps.
#   scan, step: nk heads of keys and queries (dk values), nv heads of values (dv values).
#   norm, norm_back: rows of `groups` groups of dim values; kind "layer" or "rms"; gate "none", "after" (the norm's
#   result times silu(gate)) or "before" (the norm of x silu(gate)).


def _conv(name, op, B, T, T_hi, D, width=4, type="bf16", wide=0, carried=True, lens=1):
    return dict(name=name, op=op, B=B, T=T, T_hi=T_hi, D=D, width=width, type=type, wide=wide, carried=carried, lens=lens)


def _scan(name, op, B, T, T_hi, nk, nv, dk, dv, wide=0, lens=1):
    return dict(name=name, op=op, B=B, T=T, T_hi=T_hi, nk=nk, nv=nv, dk=dk, dv=dv, wide=wide, lens=lens)


def _norm(name, op, rows, groups, dim, kind="layer", gate="none", type="bf16", wide=0):
    return dict(name=name, op=op, rows=rows, groups=groups, dim=dim, kind=kind, gate=gate, type=type, wide=wide)


def listed():
    return [
        # one decode step of a serving batch: 16 + 16 heads of queries and keys, 32 of values, 128 each
        _conv("conv, 1 token of 64", "conv", 64, 1, 1, 8192),
        # ragged prompts, some of them continuing an earlier chunk; q, k, v a slice of the layer's projection
        _conv("conv, 8 ragged prompts", "conv", 8, 100, 16000, 8192, wide=4096),
        # the training batch of the benchmark: 4 sequences of 8192 tokens
        _conv("conv backward, 4 x 8192", "conv_back", 4, 8192, 8192, 8192, carried=False),
        # a small ragged fp32 batch, as gradient checks and small models use
        _conv("conv backward, odd fp32", "conv_back", 5, 1, 301, 1112, width=3, type="fp32"),
        # the prefill batch of the benchmark, with the delta rule's head counts and sizes
        _scan("scan, 4 x 8192", "scan", 4, 8192, 8192, 16, 32, 128, 128),
        # ragged prompts, all heads on one group of queries and keys, which are slices of the convolution's rows
        _scan("scan, 8 ragged prompts", "scan", 8, 100, 16000, 1, 64, 128, 64, wide=4352),
        # one short prompt: latency
        _scan("scan, 1 x 333", "scan", 1, 333, 333, 2, 24, 64, 64),
        # one decode step of a serving batch (the benchmark's decode workload)
        _scan("step, 256 sequences", "step", 256, 1, 1, 16, 32, 128, 128),
        # one decode step of a few sequences: latency
        _scan("step, 3 sequences", "step", 3, 1, 1, 1, 24, 128, 64),
        # the layer's output norm: every head of 128 values, gated; a training or prefill batch
        _norm("norm, 32768 x 32 heads gated", "norm", 32768, 32, 128, "rms", "after"),
        # a training batch's rows of the model
        _norm("norm backward, 32768 x 4096", "norm_back", 32768, 1, 4096),
        # odd rows and sizes, the gate inside the norm
        _norm("norm backward, odd fp16", "norm_back", 1999, 1, 1000, "rms", "before", "fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng, rng.choice(["conv", "conv_back", "scan", "scan", "step", "norm", "norm_back"]))
        w = work(c)
        if max(w["bytes"] / 6.7e12, w["flops"] / 1.9e15) <= 1.5e-4 and _held(c) < 6e9:
            return c


def _held(c):
    """Bytes of the plain scan's largest arrays."""
    if c["op"] != "scan":
        return 0
    chunks = c["B"] * -(-c["T_hi"] // 128)
    return 8 * chunks * c["nv"] * (128 * 128 + 2 * c["dk"] * c["dv"]) + 8 * chunks * chunks // c["B"] * c["nv"]


def _draw(rng, op):
    type = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    wide = rng.choice([0, 0, 8 * rng.randrange(1, 64)])
    lens = rng.randrange(1000)
    if op in ("conv", "conv_back"):
        T = 1 if op == "conv" and rng.random() < 0.3 else _log(rng, 1, 16384)
        c = _conv("", op, _log(rng, 1, 256), T, rng.choice([T, 2 * T]), 8 * _log(rng, 1, 1536), rng.choice([2, 3, 4, 4]), type,
                  wide, rng.random() < 0.6, lens)
    elif op == "scan":
        T, nk = _log(rng, 1, 16384), rng.choice([1, 1, 2, 4, 8, 16])
        c = _scan("", op, _log(rng, 1, 64), T, rng.choice([T, 2 * T]), nk, nk * rng.choice([1, 2, 3, 4, 7, 8]),
                  rng.choice([64, 128, 128]), rng.choice([64, 64, 128]), wide, lens)
    elif op == "step":
        nk = rng.choice([1, 1, 2, 4, 8, 16])
        c = _scan("", op, _log(rng, 1, 512), 1, 1, nk, nk * rng.choice([1, 2, 3, 4, 7, 8]), rng.choice([64, 128, 128]),
                  rng.choice([64, 64, 128]), wide, lens)
    else:
        groups = rng.choice([1, 1, _log(rng, 1, 48)])
        dim = 8 * _log(rng, 1, 1024) if groups == 1 else 8 * _log(rng, 1, 64)
        c = _norm("", op, _log(rng, 1, 32768), groups, dim, rng.choice(["layer", "rms"]),
                  rng.choice(["none", "after", "before"]), type, wide)
    del c["name"]
    return c


def _lengths(c):
    """The sequences' lengths: part of the case."""
    r = random.Random(c["lens"])
    return [r.randint(c["T"], c["T_hi"]) for _ in range(c["B"])]


def work(c):
    e = 4 if c.get("type") == "fp32" else 2
    if c["op"] in ("norm", "norm_back"):
        n, gated, back = c["rows"] * c["groups"] * c["dim"], c["gate"] != "none", c["op"] == "norm_back"
        arrays = (3 if back else 2) + gated * (2 if back else 1)
        return {"bytes": arrays * e * n + (16 if back else 8) * c["dim"], "flops": (20 if back else 10) * n}
    rows = sum(_lengths(c))
    if c["op"] in ("conv", "conv_back"):
        n, back, kept = rows * c["D"], c["op"] == "conv_back", c["B"] * (c["width"] - 1) * c["D"] * c["carried"]
        return {"bytes": (3 if back else 2) * e * n + (3 if back else 2) * e * kept + (2 if back else 1) * 4 * c["D"] * (c["width"] + 1),
                "flops": (6 if back else 2) * c["width"] * n + 10 * n}
    key, value = c["nk"] * c["dk"], c["nv"] * c["dv"]
    # the state once in and once out, an update and a read-out of it for every token
    return {"bytes": 2 * rows * (2 * key + 2 * value) + 4 * rows * c["nv"] + 8 * c["B"] * value * c["dk"],
            "flops": 4 * rows * value * c["dk"]}


# ---- inputs --------------------------------------------------------------------------------------------------------


def prepare(c, seed):
    dev, t = torch.device("cuda"), _TYPES[c.get("type", "bf16")]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, type=t):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32 if type == torch.float32 else torch.bfloat16).to(type)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=gen, device=dev)

    def rows_of(rows, width):
        """Rows of `width` values, each a slice of a longer one where the case says so."""
        return normal(rows, width + c["wide"])[:, c["wide"]:]

    # scratch memory, reserved once by such a program: more than any case asks for
    s = dict(c=c, scratch=torch.empty(1 << 30, dtype=torch.uint8, device=dev))
    if c["op"] in ("norm", "norm_back"):
        rows, width = c["rows"], c["groups"] * c["dim"]
        s["x"] = rows_of(rows, width) + normal(rows, 1)  # rows with a mean of their own
        s["w"], s["b"] = 1.0 + 0.1 * normal(c["dim"], type=torch.float32), 0.1 * normal(c["dim"], type=torch.float32)
        if c["kind"] == "rms":
            s["b"] = None
        s["gate"] = rows_of(rows, width) if c["gate"] != "none" else None
        s["out"] = torch.empty(rows, width, dtype=t, device=dev)
        if c["op"] == "norm_back":
            s["dout"] = normal(rows, width)
            s["dgate"] = torch.empty_like(s["out"]) if s["gate"] is not None else None
            s["dw"] = torch.empty_like(s["w"])
            s["db"] = torch.empty_like(s["w"]) if s["b"] is not None else None
        return s

    lens, B = _lengths(c), c["B"]
    rows = sum(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
    ragged = c["T"] != c["T_hi"]
    s["cu"] = cu
    s["batch"] = dict(cu_seqlens=cu) if ragged else dict(B=B, T=c["T"])
    if c["op"] in ("conv", "conv_back"):
        D, width, r = c["D"], c["width"], c["width"] ** -0.5
        s["x"] = rows_of(rows, D)
        s["w"], s["b"] = uniform(-r, r, D, width), uniform(-r, r, D)
        s["state"] = normal(B, width - 1, D) if c["carried"] else None
        s["out"] = torch.empty(rows, D, dtype=t, device=dev)
        if c["op"] == "conv_back":
            s["dout"] = normal(rows, D)
            s["dw"], s["db"] = torch.empty_like(s["w"]), torch.empty_like(s["b"])
            s["dlast"] = normal(B, width - 1, D) if c["carried"] else None
            s["dstate"] = torch.empty_like(s["state"]) if c["carried"] else None
        return s

    nk, nv, dk, dv = c["nk"], c["nv"], c["dk"], c["dv"]

    def heads(n, d):
        """As they leave the convolution and its silu."""
        x = rows_of(rows, n * d)
        return x * torch.sigmoid(x)

    s["q"], s["k"], s["v"] = heads(nk, dk), heads(nk, dk), heads(nv, dv)
    if c["wide"]:  # still slices of longer rows
        for name in ("q", "k", "v"):
            s[name] = torch.cat([s[name].new_zeros(rows, c["wide"]), s[name]], 1)[:, c["wide"]:]
    # steps of 0.001 to 0.1 around a bias, decay rates of 1 to 16
    step = torch.exp(uniform(math.log(1e-3), math.log(0.1), nv))
    s["bias"] = step + torch.log(-torch.expm1(-step))
    s["dt"] = 0.5 * normal(rows, nv, type=torch.float32)
    s["a"] = -uniform(1.0, 16.0, nv)
    s["skip"] = 1.0 + 0.1 * normal(nv, type=torch.float32)
    s["state"] = 0.1 * normal(B, nv, dk, dv, type=torch.float32)
    s["out"] = torch.empty(rows, nv * dv, dtype=t, device=dev)
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------


def run(s):
    return (_own if own else _plain)[s["c"]["op"]](s)


def _own_conv(s):
    import gated_delta_rule_17_gb300 as gdn
    gdn.causal_conv(s["x"], s["w"], s["out"], bias=s["b"], state=s["state"], silu=True, **s["batch"])
    return [t for t in (s["out"], s["state"]) if t is not None]


def _own_conv_back(s):
    import gated_delta_rule_17_gb300 as gdn
    gdn.causal_conv_backward(s["x"], s["w"], s["dout"], s["out"], s["dw"], s["db"], bias=s["b"], h0=s["state"], dST=s["dlast"],
                             dh0=s["dstate"], silu=True, workspace=s["scratch"], **s["batch"])
    return [t for t in (s["out"], s["dw"], s["db"], s["dstate"]) if t is not None]


def _own_scan(s):
    import gated_delta_rule_17_gb300 as gdn
    c = s["c"]
    gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], s["state"], s["out"], nk=c["nk"], nv=c["nv"], dk=c["dk"], dv=c["dv"],
                 dt_bias=s["bias"], softplus=True, skip=s["skip"], workspace=s["scratch"], **s["batch"])
    return s["out"], s["state"]


def _own_step(s):
    import gated_delta_rule_17_gb300 as gdn
    c = s["c"]
    gdn.ssm_decode(s["q"], s["k"], s["v"], s["dt"], s["a"], s["state"], s["out"], nk=c["nk"], nv=c["nv"], dk=c["dk"], dv=c["dv"],
                   dt_bias=s["bias"], softplus=True, skip=s["skip"])
    return s["out"], s["state"]


def _own_norm(s):
    import gated_delta_rule_17_gb300 as gdn
    c = s["c"]
    gdn.layer_norm(s["x"], s["out"], dim=c["dim"], weight=s["w"], bias=s["b"], gate=s["gate"], gate_first=c["gate"] == "before",
                   rms=c["kind"] == "rms", eps=1e-5)
    return s["out"]


def _own_norm_back(s):
    import gated_delta_rule_17_gb300 as gdn
    c = s["c"]
    gdn.layer_norm_backward(s["x"], s["dout"], s["out"], s["dw"], s["db"], dim=c["dim"], weight=s["w"], bias=s["b"],
                            gate=s["gate"], dgate=s["dgate"], gate_first=c["gate"] == "before", rms=c["kind"] == "rms",
                            eps=1e-5, workspace=s["scratch"])
    return [t for t in (s["out"], s["dw"], s["db"], s["dgate"]) if t is not None]


def _extended(s):
    """All sequences' inputs, each behind the width - 1 rows before it; the places of the inputs in it, those of the rows
    before each sequence, and those of each sequence's last width - 1 rows."""
    c, cu = s["c"], s["cu"].long()
    before = c["width"] - 1
    rows = s["x"].shape[0]
    row = torch.arange(rows, device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    at = row + (seq + 1) * before
    lag = torch.arange(before, device=cu.device)
    first = cu[:-1, None] + torch.arange(c["B"], device=cu.device)[:, None] * before + lag
    last = cu[1:, None] + torch.arange(c["B"], device=cu.device)[:, None] * before + lag
    x = torch.zeros(rows + c["B"] * before, c["D"], device=cu.device)
    x[at] = s["x"].float()
    if s["state"] is not None:
        x[first] = s["state"].float()
    return x, at, first, last


def _plain_conv(s):
    c = s["c"]
    x, at, _, last = _extended(s)
    y = s["b"] + sum(x[at - (c["width"] - 1) + j] * s["w"][:, j] for j in range(c["width"]))
    s["out"].copy_(y / (1.0 + torch.exp(-y)))
    if s["state"] is None:
        return [s["out"]]
    s["state"].copy_(x[last])
    return [s["out"], s["state"]]


def _plain_conv_back(s):
    c, w = s["c"], s["w"]
    x, at, first, last = _extended(s)
    taps = range(c["width"])
    y = s["b"] + sum(x[at - (c["width"] - 1) + j] * w[:, j] for j in taps)
    g = 1.0 / (1.0 + torch.exp(-y))
    dy = s["dout"].float() * (g + y * g * (1.0 - g))
    del y, g
    s["dw"].copy_(torch.stack([(x[at - (c["width"] - 1) + j] * dy).sum(0) for j in taps], 1))
    s["db"].copy_(dy.sum(0))
    # the gradient of input i: what the outputs i .. i + width - 1 of its own sequence have of it
    wide = torch.zeros(x.shape[0] + c["width"] - 1, c["D"], device=x.device)
    wide[at] = dy
    dx = sum(wide[c["width"] - 1 - j:][:x.shape[0]] * w[:, j] for j in taps)
    if s["dlast"] is not None:
        dx[last] += s["dlast"].float()
    s["out"].copy_(dx[at])
    if s["dstate"] is None:
        return [s["out"], s["dw"], s["db"]]
    s["dstate"].copy_(dx[first])
    return [s["out"], s["dw"], s["db"], s["dstate"]]


def _steps(s):
    """The steps dt, after bias and softplus."""
    z = s["dt"] + s["bias"]
    return torch.clamp(z, min=0.0) + torch.log1p(torch.exp(-z.abs()))


def _plain_scan(s):
    c, L = s["c"], 128
    B, nk, nv, dk, dv = c["B"], c["nk"], c["nv"], c["dk"], c["dv"]
    cu, T, group = s["cu"].long(), -(-c["T_hi"] // L) * L, nv // nk
    t = torch.arange(T, device=cu.device)
    held = t < (cu[1:] - cu[:-1])[:, None]  # [B, T]
    at = (cu[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
    dt = torch.where(held[..., None], _steps(s)[at], 0.0)

    def chunks(x, n, d):
        return x[at].float().view(B, T // L, L, n, d).transpose(2, 3)  # [B, chunks, heads, L, d]

    q, k, v = chunks(s["q"], nk, dk), chunks(s["k"], nk, dk), chunks(s["v"], nv, dv)
    dt = dt.view(B, T // L, L, nv).transpose(2, 3)  # [B, chunks, nv, L]
    g = torch.cumsum((dt * s["a"][:, None]).double(), -1)  # within the chunk: differences of far tokens stay exact
    i = torch.arange(L, device=cu.device)
    decay = torch.exp(torch.where(i[:, None] >= i, g[..., :, None] - g[..., None, :], float("-inf")).float())
    scores = torch.matmul(q, k.transpose(3, 4)).repeat_interleave(group, 2) * decay
    dv_ = v * dt[..., None]
    out = torch.matmul(scores, dv_)
    del scores, decay
    # each chunk's own part of the state at its end, and the states before all chunks from those
    left = torch.exp((g[..., -1:] - g).float())
    part = torch.matmul(k.transpose(3, 4).repeat_interleave(group, 2), dv_ * left[..., None])
    part = torch.cat([s["state"][:, None], part], 1)
    total = torch.cat([g.new_zeros(B, 1, nv), torch.cumsum(g[..., -1], 1)], 1).transpose(1, 2)  # [B, nv, chunks + 1]
    n = torch.arange(T // L + 1, device=cu.device)
    pass_on = torch.exp(torch.where(n[:, None] >= n, total[..., :, None] - total[..., None, :], float("-inf")).float())
    states = torch.matmul(pass_on, part.transpose(1, 2).flatten(3)).view(B, nv, -1, dk, dv).transpose(1, 2)
    out = out + torch.matmul(q.repeat_interleave(group, 2), states[:, :-1]) * torch.exp(g.float())[..., None]
    out = out + s["skip"][:, None, None] * v
    out = out.transpose(2, 3).reshape(B, T, nv * dv)
    s["out"].copy_(out[held])
    s["state"].copy_(states[:, -1])
    return s["out"], s["state"]


def _plain_step(s):
    c = s["c"]
    B, nk, nv, dk, dv = c["B"], c["nk"], c["nv"], c["dk"], c["dv"]
    q, k = (s[n].float().view(B, nk, dk).repeat_interleave(nv // nk, 1) for n in ("q", "k"))
    v, dt = s["v"].float().view(B, nv, dv), _steps(s)
    new = torch.exp(dt * s["a"])[..., None, None] * s["state"] + k[..., None] * (dt[..., None] * v)[..., None, :]
    s["state"].copy_(new)
    out = (new * q[..., None]).sum(2) + s["skip"][:, None] * v
    s["out"].copy_(out.view(B, nv * dv))
    return s["out"], s["state"]


def _grouped(x, c):
    return x.unflatten(1, (c["groups"], c["dim"])).float()


def _plain_norm(s):
    c = s["c"]
    x = _grouped(s["x"], c)
    if s["gate"] is not None:
        z = _grouped(s["gate"], c)
        z = z / (1.0 + torch.exp(-z))
        if c["gate"] == "before":
            x = x * z
    if c["kind"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    if c["gate"] == "after":
        y = y * z
    s["out"].copy_(y.flatten(1))
    return s["out"]


def _plain_norm_back(s):
    c = s["c"]
    x, dy = _grouped(s["x"], c), _grouped(s["dout"], c)
    u, z = x, None
    if s["gate"] is not None:
        z = _grouped(s["gate"], c)
        sig = 1.0 / (1.0 + torch.exp(-z))
        slope = sig + z * sig * (1.0 - sig)
        if c["gate"] == "before":
            u = x * z * sig
    if c["kind"] == "layer":
        u = u - u.mean(-1, keepdim=True)
    r = torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-5)
    n = u * r
    if c["gate"] == "after":
        y = n * s["w"] if s["b"] is None else n * s["w"] + s["b"]
        s["dgate"].copy_((dy * y * slope).flatten(1))
        dy = dy * z * sig
        del y
    s["dw"].copy_((dy * n).sum((0, 1)))
    if s["db"] is not None:
        s["db"].copy_(dy.sum((0, 1)))
    dn = dy * s["w"]
    du = dn - n * (dn * n).mean(-1, keepdim=True)
    if c["kind"] == "layer":
        du = du - dn.mean(-1, keepdim=True)
    du = du * r
    if c["gate"] == "before":
        s["dgate"].copy_((du * x * slope).flatten(1))
        du = du * z * sig
    s["out"].copy_(du.flatten(1))
    return [t for t in (s["out"], s["dw"], s["db"], s["dgate"]) if t is not None]


_own = {"conv": _own_conv, "conv_back": _own_conv_back, "scan": _own_scan, "step": _own_step, "norm": _own_norm,
        "norm_back": _own_norm_back}
_plain = {"conv": _plain_conv, "conv_back": _plain_conv_back, "scan": _plain_scan, "step": _plain_step, "norm": _plain_norm,
          "norm_back": _plain_norm_back}


# ---- in 64 bits ----------------------------------------------------------------------------------------------------


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("norm", "norm_back"):
        return _exact_norm(c, s)
    if c["op"] in ("conv", "conv_back"):
        return _exact_conv(c, s)
    return _exact_scan(c, s)


def _exact_norm(c, s):
    back, parts, sums = c["op"] == "norm_back", [], []
    step = max(1, (1 << 25) // (c["groups"] * c["dim"]))
    for a in range(0, c["rows"], step):  # in pieces: the gradient keeps many copies
        leaf = {n: s[n][a:a + step].double().unflatten(1, (c["groups"], c["dim"])) for n in ("x", "gate") if s[n] is not None}
        leaf.update({n: s[n].double() for n in ("w", "b") if s[n] is not None})
        leaf = {n: t.clone().requires_grad_(back) for n, t in leaf.items()}
        gate = torch.nn.functional.silu(leaf["gate"]) if "gate" in leaf else 1.0
        u = leaf["x"] * gate if c["gate"] == "before" else leaf["x"]
        mean = u.mean(-1, keepdim=True) if c["kind"] == "layer" else 0.0
        y = (u - mean) / torch.sqrt(((u - mean) ** 2).mean(-1, keepdim=True) + 1e-5) * leaf["w"] + leaf.get("b", 0.0)
        y = y * gate if c["gate"] == "after" else y
        if not back:
            parts.append(y.flatten(1))
            continue
        y.backward(s["dout"][a:a + step].double().view_as(y))
        parts.append((leaf["x"].grad.flatten(1), leaf["gate"].grad.flatten(1) if "gate" in leaf else None))
        sums.append([leaf[n].grad for n in ("w", "b") if n in leaf])
    if not back:
        return torch.cat(parts)
    out = [torch.cat([p[0] for p in parts])] + [sum(t) for t in zip(*sums)]
    return out + ([torch.cat([p[1] for p in parts])] if s["gate"] is not None else [])


def _exact_conv(c, s):
    back, D, width = c["op"] == "conv_back", c["D"], c["width"]
    w, b = s["w"].double().requires_grad_(back), s["b"].double().requires_grad_(back)
    outs, states, row = [], [], 0
    for n, length in enumerate(_lengths(c)):
        x = s["x"][row:row + length].double().clone().requires_grad_(back)
        first = s["state"][n].double().clone() if c["carried"] else torch.zeros(width - 1, D, dtype=torch.float64, device=x.device)
        first.requires_grad_(back)
        z = torch.cat([first, x])
        y = torch.nn.functional.silu(torch.nn.functional.conv1d(z.T[None], w[:, None], b, groups=D)[0].T)
        if back:
            total = (y * s["dout"][row:row + length].double()).sum()
            if c["carried"]:
                total = total + (z[length:] * s["dlast"][n].double()).sum()
            total.backward()
        outs.append(x.grad if back else y)
        states.append(first.grad if back else z[length:])
        row += length
    kept = [torch.stack(states)] if c["carried"] else []
    return [torch.cat(outs)] + ([w.grad, b.grad] if back else []) + kept


def _exact_scan(c, s):
    B, nk, nv, dk, dv = c["B"], c["nk"], c["nv"], c["dk"], c["dv"]
    lens, cu = torch.tensor(_lengths(c), device="cuda"), s["cu"].long()
    dt = torch.nn.functional.softplus(s["dt"].double() + s["bias"].double(), threshold=1e3)
    state, out = s["state"].double(), torch.empty_like(s["out"], dtype=torch.float64)
    a, skip = s["a"].double(), s["skip"].double()
    for t in range(max(_lengths(c))):  # token by token, all sequences that still have one
        b = (lens > t).nonzero()[:, 0] if c["T"] != c["T_hi"] else slice(None)
        row = cu[:-1][b] + t
        q, k = (s[n][row].double().view(-1, nk, 1, dk, 1) for n in ("q", "k"))
        v = s["v"][row].double().view(-1, nk, nv // nk, 1, dv)
        d = dt[row].view(-1, nk, nv // nk, 1, 1)
        now = torch.exp(d * a.view(nk, -1, 1, 1)) * state[b].view(-1, nk, nv // nk, dk, dv) + k * (d * v)
        state[b] = now.view(-1, nv, dk, dv)
        out[row] = ((q * now).sum(3) + skip.view(nk, -1, 1) * v[:, :, :, 0]).view(-1, nv * dv)
    return out, state
