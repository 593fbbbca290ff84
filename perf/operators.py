"""The operators of a softmax-attention layer in a hybrid model, next to the gated delta rule, as measured cases:
the norm and rotation of query and key heads (and its gradient), the append to a paged cache, and the attention of
a tree of drafted tokens (or of one decode token) over that cache."""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------------------------------
# Fields: op; type; nq, nkv heads of d values; rot: rotated values of a head; pairs: "half" (i, i + rot/2) or
# "next" (2i, 2i+1).
#   norm, norm_back: rows tokens.
#   append, attend: B sequences, each with n new rows (n_hi > n: ragged, n .. n_hi) behind a context of
#   ctx .. ctx_hi tokens, drawn by `lens`; page: tokens to a page; tree: drafted tokens form a random tree.


def _norm(name, op, rows, nq, nkv, d=128, rot=128, type="bf16", pairs="half"):
    return dict(name=name, op=op, rows=rows, nq=nq, nkv=nkv, d=d, rot=rot, type=type, pairs=pairs)


def _append(name, B, n, n_hi, ctx, ctx_hi, nkv, page, d=128, rot=128, type="bf16", pairs="half", normed=True, lens=1):
    return dict(name=name, op="append", B=B, n=n, n_hi=n_hi, ctx=ctx, ctx_hi=ctx_hi, nq=nkv, nkv=nkv, page=page, d=d,
                rot=rot, type=type, pairs=pairs, normed=normed, lens=lens)


def _attend(name, B, n, n_hi, ctx, ctx_hi, nq, nkv, page, tree, d=128, type="bf16", lens=1):
    return dict(name=name, op="attend", B=B, n=n, n_hi=n_hi, ctx=ctx, ctx_hi=ctx_hi, nq=nq, nkv=nkv, page=page,
                tree=tree, d=d, type=type, lens=lens)


def listed():
    return [
        # one decode step of a few sequences: the latency of the call
        _norm("norm, 4 tokens", "norm", 4, 16, 2),
        # a training or prefill batch: 4 sequences of 8192 tokens
        _norm("norm, 4 x 8192 tokens", "norm", 32768, 32, 8),
        # odd head counts, partial rotation of neighbouring pairs, small heads
        _norm("norm, odd fp16", "norm", 1999, 15, 5, d=64, rot=32, type="fp16", pairs="next"),
        # the backward pass of the training batch
        _norm("norm backward, 4 x 8192 tokens", "norm_back", 32768, 32, 8),
        # a short fp32 batch with partial rotation, as gradient checks and small models use
        _norm("norm backward, odd fp32", "norm_back", 777, 6, 3, rot=64, type="fp32"),
        # one decode step of a serving batch, each sequence at its own length
        _append("append, decode of 64", 64, 1, 1, 100, 16000, 8, 64),
        # prefill of 8 ragged prompts, some continuing a cached context that ends inside a page
        _append("append, 8 ragged prompts", 8, 100, 16000, 0, 1000, 8, 16),
        # a single sequence's decode token over a short context: latency
        _attend("attend, 1 token over 257", 1, 1, 1, 257, 257, 32, 8, 64, False),
        # decode step of a serving batch with ragged contexts
        _attend("attend, decode of 64", 64, 1, 1, 100, 16000, 32, 8, 64, False),
        # verifying small ragged draft trees for a serving batch
        _attend("attend, trees of 3..16", 16, 3, 16, 500, 8192, 32, 8, 16, True),
        # verifying one draft tree over a very long context
        _attend("attend, tree of 33 over 65536", 1, 33, 33, 65536, 65536, 16, 2, 64, True, type="fp16"),
        # large draft trees over long contexts, where the products bound
        _attend("attend, trees of 64 over 32768", 8, 64, 64, 32000, 32768, 32, 4, 64, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "append", "attend", "attend"])
    c = _draw(rng, op)
    while max(work(c)["bytes"] / 6.7e12, work(c)["flops"] / 1.9e15) > 1.9e-4 or 3072 in _sizes(c):
        c = _draw(rng, op)
    return c


def _sizes(c):
    return [c.get("rows"), c.get("n"), c.get("n_hi"), c.get("ctx"), c.get("ctx_hi"), c["nq"] * c["d"], c["nkv"] * c["d"]]


def _draw(rng, op):
    d = rng.choice([64, 128, 128])
    nkv = rng.choice([1, 2, 3, 4, 5, 8])
    nq = nkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    rot = rng.choice([d, d, d // 2, 16, 48])
    pairs = rng.choice(["half", "half", "next"])
    if op in ("norm", "norm_back"):
        c = _norm("", op, _log(rng, 1, 32768), min(nq, 40), nkv, d, rot, rng.choice(["bf16", "bf16", "fp16", "fp32"]), pairs)
    elif op == "append":
        n = _log(rng, 1, 8192) if rng.random() < 0.5 else 1
        ctx = rng.choice([0, _log(rng, 1, 16000)])
        c = _append("", _log(rng, 1, 128), n, rng.choice([n, 2 * n]), ctx, rng.choice([ctx, 2 * ctx + 1]), nkv,
                    rng.choice([1, 16, 17, 64, 256]), d, rot, rng.choice(["bf16", "bf16", "fp16"]), pairs,
                    rng.random() < 0.5, rng.randrange(1000))
    else:
        n = _log(rng, 1, 128) if rng.random() < 0.7 else 1
        ctx = rng.choice([0] + 9 * [_log(rng, 1, 65536)])
        c = _attend("", _log(rng, 1, 128), n, rng.choice([n, 2 * n]), ctx, rng.choice([ctx, 2 * ctx]), nq, nkv,
                    rng.choice([16, 16, 17, 64, 64, 256]), rng.random() < 0.7, d, rng.choice(["bf16", "bf16", "fp16"]),
                    rng.randrange(1000))
        if nq > 64 or 2.0 * c["B"] * c["n_hi"] ** 2 * nq > 2e9 or c["B"] * c["n_hi"] * nq * c["ctx_hi"] > 6e8:
            return _draw(rng, op)  # the plain form's score matrices would not fit
    del c["name"]
    return c


def _lengths(c):
    """The context lengths and new rows of every sequence: part of the case."""
    r = random.Random(c["lens"])
    ctx = [r.randint(c["ctx"], c["ctx_hi"]) for _ in range(c["B"])]
    new = [r.randint(c["n"], c["n_hi"]) for _ in range(c["B"])]
    return ctx, new


def work(c):
    e, d = (4 if c["type"] == "fp32" else 2), c["d"]
    if c["op"] in ("norm", "norm_back"):
        back = c["op"] == "norm_back"
        heads = c["rows"] * (c["nq"] + c["nkv"])
        return {"bytes": (3 if back else 2) * e * heads * d + 4 * c["rows"] * (1 + c["rot"]) + (16 if back else 8) * d,
                "flops": (20 if back else 10) * heads * d}
    ctx, new = _lengths(c)
    rows = sum(new)
    if c["op"] == "append":
        return {"bytes": 4 * e * rows * c["nkv"] * d + 4 * rows * (1 + c["rot"]), "flops": 10 * rows * c["nkv"] * d}
    tokens = sum(ctx) + rows
    return {"bytes": 2 * e * tokens * c["nkv"] * d + 2 * e * rows * c["nq"] * d,
            "flops": 4 * c["nq"] * d * sum(n * (t + n) for t, n in zip(ctx, new))}


# ---- inputs --------------------------------------------------------------------------------------------------------


def _tables(c, count, device):
    """cos and sin of position * base^(-2i/rot), fp32 [count, rot/2]."""
    f = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=device, dtype=torch.float64) / c["rot"])
    a = torch.arange(count, device=device, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def _trees(rng, new):
    """Random draft trees: parent[i] < i or none (the context); each row's ancestors and itself, as 64-bit words."""
    words = (max(new) + 63) // 64
    rows, depths = [], []
    for n in new:
        sees, depth = np.zeros((n, words * 64), dtype=bool), np.zeros(n, dtype=np.int64)
        parent = (rng.random(n) * (np.arange(n) + 1)).astype(np.int64) - 1
        for i in range(n):
            if parent[i] >= 0:
                sees[i] = sees[parent[i]]
                depth[i] = depth[parent[i]] + 1
            sees[i, i] = True
        rows.append(sees)
        depths.append(depth)
    bits = np.packbits(np.concatenate(rows), axis=1, bitorder="little").view("<i8")
    return np.ascontiguousarray(bits.reshape(-1, words)), np.concatenate(depths)


def prepare(c, seed):
    dev, t = torch.device("cuda"), _TYPES[c["type"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    d, nq, nkv = c["d"], c["nq"], c["nkv"]

    def normal(*shape, type=t):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32 if type == torch.float32 else torch.bfloat16).to(type)

    def weight():
        return 1.0 + 0.1 * torch.randn(d, generator=gen, device=dev)

    # scratch memory, reserved once by such a program: more than any case asks for
    s = dict(c=c, scratch=torch.empty(64 << 20, dtype=torch.uint8, device=dev))
    if c["op"] in ("norm", "norm_back"):
        rows, span = c["rows"], max(c["rows"], 4096)
        s["q"], s["k"] = normal(rows, nq * d), normal(rows, nkv * d)
        s["qw"], s["kw"] = weight(), weight()
        s["cos"], s["sin"] = _tables(c, span, dev)
        # packed sequences: positions count up from somewhere
        s["pos"] = ((torch.arange(rows, device=dev) + int(rng.integers(span))) % span).int()
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        if c["op"] == "norm_back":
            s["dyq"], s["dyk"] = normal(rows, nq * d), normal(rows, nkv * d)
            s["dqw"], s["dkw"] = torch.empty_like(s["qw"]), torch.empty_like(s["kw"])
        return s

    ctx, new = _lengths(c)
    B, rows, page = c["B"], sum(new), c["page"]
    need = [(a + n + page - 1) // page for a, n in zip(ctx, new)]
    pages = sum(need) + 3
    ids = rng.permutation(pages)[:sum(need)].astype(np.int32)
    table = np.full((B, max(need)), -1, dtype=np.int32)
    table[np.arange(max(need))[None, :] < np.array(need)[:, None]] = ids
    s["table"] = torch.from_numpy(table).to(dev)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=dev)
    s["k_cache"], s["v_cache"] = normal(pages, page, nkv, d), normal(pages, page, nkv, d)
    drafted = max(new) <= 64 if c["op"] == "append" else c["tree"]
    bits, depth = _trees(rng, new) if drafted else (None, None)
    if c["op"] == "append":
        s["k"], s["v"], s["kw"] = normal(rows, nkv * d), normal(rows, nkv * d), weight()
        first = np.repeat(ctx, new)
        # drafted tokens stand at their depth in the tree, a prompt's at their place
        at = first + (depth if drafted else np.arange(rows) - np.repeat(np.cumsum(new) - new, new))
        s["pos"] = torch.from_numpy(at.astype(np.int32)).to(dev)
        s["cos"], s["sin"] = _tables(c, max(a + n for a, n in zip(ctx, new)), dev)
    else:
        s["q"] = 2.0 * normal(rows, nq * d)  # scores of standard deviation 2: some tokens count far more than others
        s["out"] = torch.empty_like(s["q"])
        s["mask"] = torch.from_numpy(bits).to(dev) if c["tree"] else None
        s["max_rows"] = max(new)
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------


def run(s):
    return (_own if own else _plain)[s["c"]["op"]](s)


def _own_norm(s):
    import gated_delta_rule_17_gb300 as gdn
    c = s["c"]
    gdn.head_norm_rope(s["q"], s["k"], s["pos"], s["cos"], s["sin"], s["q_out"], s["k_out"], nq=c["nq"], nkv=c["nkv"],
                       head_dim=c["d"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS, interleaved=c["pairs"] == "next")
    return s["q_out"], s["k_out"]


def _own_norm_back(s):
    import gated_delta_rule_17_gb300 as gdn
    c = s["c"]
    gdn.head_norm_rope_backward(s["q"], s["k"], s["pos"], s["cos"], s["sin"], s["dyq"], s["dyk"], s["q_out"], s["k_out"],
                                s["dqw"], s["dkw"], nq=c["nq"], nkv=c["nkv"], head_dim=c["d"], q_weight=s["qw"],
                                k_weight=s["kw"], eps=EPS, interleaved=c["pairs"] == "next", workspace=s["scratch"])
    return s["q_out"], s["k_out"], s["dqw"], s["dkw"]


def _own_append(s):
    import gated_delta_rule_17_gb300 as gdn
    c = s["c"]
    gdn.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], nkv=c["nkv"], head_dim=c["d"],
                     cu_rows=s["cu"], positions=s["pos"], cos=s["cos"], sin=s["sin"], norm=c["normed"],
                     k_weight=s["kw"] if c["normed"] else None, eps=EPS, interleaved=c["pairs"] == "next")
    return s["k_cache"], s["v_cache"]


def _own_attend(s):
    import gated_delta_rule_17_gb300 as gdn
    c = s["c"]
    gdn.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["out"], nq=c["nq"], nkv=c["nkv"],
                       head_dim=c["d"], cu_rows=s["cu"], mask=s["mask"], max_rows=s["max_rows"], workspace=s["scratch"])
    return s["out"]


def _heads(x, d):
    return x.view(x.shape[0], -1, d).float()


def _pairs(z, rot, pairs):
    """The two halves of the rotated values, and the rest."""
    r = z[..., :rot]
    a, b = (r[..., :rot // 2], r[..., rot // 2:]) if pairs == "half" else (r[..., 0::2], r[..., 1::2])
    return a, b, z[..., rot:]


def _join(a, b, rest, pairs):
    r = torch.cat([a, b], -1) if pairs == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([r, rest], -1)


def _rotate(z, cos, sin, rot, pairs):
    a, b, rest = _pairs(z, rot, pairs)
    return _join(a * cos - b * sin, b * cos + a * sin, rest, pairs)


def _plain_norm(s):
    c = s["c"]
    cos, sin = s["cos"][s["pos"].long(), None], s["sin"][s["pos"].long(), None]

    def one(x, w):
        x = _heads(x, c["d"])
        z = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        return _rotate(z, cos, sin, c["rot"], c["pairs"]).flatten(1).to(_TYPES[c["type"]])

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _plain_norm_back(s):
    c = s["c"]
    cos, sin = s["cos"][s["pos"].long(), None], s["sin"][s["pos"].long(), None]

    def one(x, dy, w):
        x, dy = _heads(x, c["d"]), _heads(dy, c["d"])
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        dz = _rotate(dy, cos, -sin, c["rot"], c["pairs"])
        xr = x * r
        t = dz * w
        dx = r * (t - xr * (t * xr).mean(-1, keepdim=True))
        return dx.flatten(1).to(_TYPES[c["type"]]), (dz * xr).sum((0, 1))

    (dq, dqw), (dk, dkw) = one(s["q"], s["dyq"], s["qw"]), one(s["k"], s["dyk"], s["kw"])
    return dq, dk, dqw, dkw


def _slots(s):
    """Page, offset in the page and sequence of every new row."""
    page, cu = s["c"]["page"], s["cu"].long()
    row = torch.arange(s["k"].shape[0], device=cu.device)
    b = torch.searchsorted(cu, row, right=True) - 1
    slot = s["ctx"].long()[b] + row - cu[b]
    return s["table"].long()[b, slot // page], slot % page


def _plain_append(s):
    c = s["c"]
    k = _heads(s["k"], c["d"])
    if c["normed"]:
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * s["kw"]
    at = s["pos"].long()
    k = _rotate(k, s["cos"][at, None], s["sin"][at, None], c["rot"], c["pairs"])
    page, off = _slots(s)
    s["k_cache"][page, off] = k.to(s["k_cache"].dtype)
    s["v_cache"][page, off] = s["v"].view(k.shape)
    return s["k_cache"], s["v_cache"]


def _plain_attend(s):
    c = s["c"]
    B, d, nq, nkv, n = c["B"], c["d"], c["nq"], c["nkv"], s["max_rows"]
    cu, ctx, table = s["cu"].long(), s["ctx"].long()[:, None, None], s["table"].long()
    new = (cu[1:] - cu[:-1])[:, None]
    i = torch.arange(n, device=cu.device)
    held = i < new  # [B, n]: the rows that there are
    at = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].view(-1, nkv, nq // nkv, d)[at].float()  # [B, n, nkv, group, d]
    q = q.permute(0, 2, 3, 1, 4).reshape(B, nkv, -1, d)
    k, v = (x[table.clamp(min=0)].flatten(1, 2).permute(0, 2, 1, 3).float() for x in (s["k_cache"], s["v_cache"]))
    j = torch.arange(k.shape[2], device=cu.device) - ctx  # [B, 1, tokens]: the place among the new rows
    if s["mask"] is None:
        sees = j <= i[:, None]
    else:
        word = torch.gather(s["mask"][at], 2, (j.clamp(0, n - 1) // 64).expand(-1, n, -1))
        sees = (j < 0) | (((word >> (j.clamp(0, n - 1) % 64)) & 1) == 1)
    sees = (sees & (j < new[:, None]))[:, None, None]  # [B, 1, 1, n, tokens]
    x = torch.matmul(q, k.transpose(2, 3)).view(B, nkv, nq // nkv, n, -1) / math.sqrt(d)
    x = torch.where(sees, x, float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == float("-inf"), 0.0, top))
    del x
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, nkv, -1, p.shape[-1]), v).view(B, nkv, nq // nkv, n, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4)  # [B, n, nkv, group, d]
    return o[held].reshape(-1, nq * d).to(s["q"].dtype)


_own = {"norm": _own_norm, "norm_back": _own_norm_back, "append": _own_append, "attend": _own_attend}
_plain = {"norm": _plain_norm, "norm_back": _plain_norm_back, "append": _plain_append, "attend": _plain_attend}


# ---- in 64 bits ----------------------------------------------------------------------------------------------------


def _turn(x, c, angle_cos, angle_sin, w=None):
    """Norm (with w) and rotation of heads x [rows, heads, d], as products of complex numbers."""
    d, rot = c["d"], c["rot"]
    if w is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS) * w.double()
    turn = torch.complex(angle_cos.double(), angle_sin.double())[:, None, :]
    i = torch.arange(rot // 2, device=x.device)
    one, two = (i, i + rot // 2) if c["pairs"] == "half" else (2 * i, 2 * i + 1)
    z = torch.complex(x[..., one], x[..., two]) * turn
    at = torch.argsort(torch.cat([one, two]))
    return torch.cat([torch.cat([z.real, z.imag], -1)[..., at], x[..., rot:]], -1)


def exact(c, seed):
    s = prepare(c, seed)
    d = c["d"]
    if c["op"] in ("norm", "norm_back"):
        cos, sin = s["cos"][s["pos"].long()], s["sin"][s["pos"].long()]
        outs, sums = [], []
        for x, w, dy in ((s["q"], s["qw"], s.get("dyq")), (s["k"], s["kw"], s.get("dyk"))):
            parts, dw = [], 0
            for a in range(0, c["rows"], 2048):  # in pieces: the gradient keeps many copies
                xs = x[a:a + 2048].double().view(-1, x.shape[1] // d, d).requires_grad_(dy is not None)
                ws = w.double().requires_grad_(dy is not None)
                y = _turn(xs, c, cos[a:a + 2048], sin[a:a + 2048], ws)
                if dy is None:
                    parts.append(y.flatten(1))
                else:
                    y.backward(dy[a:a + 2048].double().view_as(y))
                    parts.append(xs.grad.flatten(1))
                    dw = dw + ws.grad
            outs.append(torch.cat(parts))
            sums.append(dw)
        return tuple(outs) if c["op"] == "norm" else tuple(outs + sums)

    ctx, new = _lengths(c)
    page = c["page"]
    if c["op"] == "append":
        at = s["pos"].long()
        k = _turn(s["k"].double().view(-1, c["nkv"], d), c, s["cos"][at], s["sin"][at], s["kw"] if c["normed"] else None)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        row = 0
        for b in range(c["B"]):
            slot = torch.arange(ctx[b], ctx[b] + new[b], device=k.device)
            flat = s["table"][b].long()[slot // page] * page + slot % page
            kc.view(-1, c["nkv"], d)[flat] = k[row:row + new[b]]
            vc.view(-1, c["nkv"], d)[flat] = s["v"][row:row + new[b]].double().view(-1, c["nkv"], d)
            row += new[b]
        return kc, vc

    group, out, row = c["nq"] // c["nkv"], [], 0
    for b in range(c["B"]):
        n, total = new[b], ctx[b] + new[b]
        slot = torch.arange(total, device=s["q"].device)
        flat = s["table"][b].long()[slot // page] * page + slot % page
        sees = torch.ones(n, total, dtype=torch.bool, device=slot.device)
        if c["tree"]:
            words = np.ascontiguousarray(s["mask"][row:row + n].cpu().numpy())
            bits = np.unpackbits(words.view(np.uint8), axis=1, bitorder="little")[:, :n]
            sees[:, ctx[b]:] = torch.from_numpy(bits.astype(bool)).to(sees.device)
        else:
            sees[:, ctx[b]:] = torch.ones(n, n, device=slot.device).tril().bool()
        q = s["q"][row:row + n].double().view(n, c["nkv"], group, d)
        o = torch.empty_like(q)
        for h in range(c["nkv"]):
            kh = s["k_cache"].view(-1, c["nkv"], d)[flat, h].double()
            vh = s["v_cache"].view(-1, c["nkv"], d)[flat, h].double()
            p = torch.softmax((q[:, h] @ kh.T / math.sqrt(d)).masked_fill(~sees[:, None], float("-inf")), -1)
            o[:, h] = p @ vh
        out.append(o.reshape(n, -1))
        row += n
    return torch.cat(out)
